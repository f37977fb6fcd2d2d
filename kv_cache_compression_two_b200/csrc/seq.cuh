// seq.cuh -- packed sequences: bounds read from device arrays, and the even
// split of ragged work over a fixed number of CTAs that the two sequence
// attentions share.
//
// The work of one call is a line of unit steps: sequences in order, each
// sequence's items (a query tile of a head) in order, each item's KV tiles in
// order.  CTA c of n takes the stretch [c * total / n, (c + 1) * total / n), so
// every SM gets the same number of steps whatever the lengths are.  An item
// that a boundary cuts is finished from partial results: each CTA leaves at
// most two (the end of an item that began before its stretch, slot 2c, and the
// start of one that goes on behind it, slot 2c + 1), and a second launch
// merges them.  A boundary that would leave fewer than min_head steps before it
// or fewer than min_tail behind it in its item moves to the item's edge.
#pragma once

#include "common.cuh"

namespace ispa {

// Rows [begin, begin + n) of sequence b, clamped to the T rows that exist.
struct SeqRows {
  int begin, n;
};

__device__ __forceinline__ SeqRows seq_rows(const int *cu, int b, int T) {
  const int c0 = min(max(__ldg(cu + b), 0), T), c1 = min(max(__ldg(cu + b + 1), 0), T);
  return {c0, max(0, c1 - c0)};
}

__device__ __forceinline__ bool seq_rows_bad(const int *cu, int b, int T) {
  const int c0 = __ldg(cu + b), c1 = __ldg(cu + b + 1);
  return c0 < 0 || c1 < c0 || c1 > T;
}

// Records a value of sequence b that is out of range (err: the device error word).
__device__ __forceinline__ void report_seq(int *err, int b) {
  if (atomicCAS(err, 0, ISPA_ERR_INVALID_ARG) == 0) atomicExch(err + 1, b);
}

__device__ __forceinline__ int seq_len(const int *lens, int b, int cap) {
  return min(max(__ldg(lens + b), 0), cap);
}

// The sequence that owns packed row t, or -1; executed by a whole warp with a
// uniform t.  Each round narrows the candidates 32-fold by a ballot, so that
// 1024 sequences cost two dependent loads.  (The last check holds for every t
// unless bounds decrease: the search may then end at a sequence without the row.)
__device__ __forceinline__ int seq_of_row(const int *cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the first b in [lo, lo + n) with cu[b + 1] > t
  while (n > 0) {
    const int step = (n + 31) >> 5;
    const int b = lo + min((lane + 1) * step, n) - 1;  // last candidate of this lane's part
    const unsigned past = __ballot_sync(0xffffffffu, __ldg(cu + b + 1) <= t);
    const int k = __popc(past);  // parts that end at or before t
    if (k == 32) return -1;
    const int skip = min(k * step, n);
    lo += skip;
    n = min(step, n - skip);
    if (step == 1) break;
  }
  return n > 0 && lo < B && __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -1;
}

// a b / n and a / b; in 32 bits where they fit (64-bit division is a long routine, and these
// stand in front of a call's first load).
__device__ __forceinline__ long long mul_div(int a, long long b, int n) {
  if (b < (1LL << 32) / 2048 && a < 2048) return (uint32_t)a * (uint32_t)b / (uint32_t)n;
  return a * b / n;
}
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (a < (1LL << 32) && b < (1LL << 32)) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct SplitRange {
  int b;             // sequence that holds the first step
  int tag;           // f.item()'s name of the item
  long long off;     // the step's place in the sequence's line
  long long begin;   // and the item's
  long long x0, x1;  // the stretch [x0, x1) of the whole line
};

// This CTA's stretch.  f.cost(b): steps of sequence b; f.item(b, off, &s, &e)
// (called by a whole warp): the item [s, e) that holds step off of sequence b.
// At most ceil(total / min_unit) CTAs get work.  Called by all NT threads; sw:
// NT / 32 + 8 values of scratch.
template <int NT, class F>
__device__ void split_range(const F &f, int B, int nc, int c, int min_unit, int min_head, int min_tail, SplitRange *r,
                            long long *sw) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + NT - 1) / NT;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += f.cost(b);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) sw[warp] = inc;
  long long *found = sw + NT / 32;  // per boundary: sequence (-1: none), place in it, place of the sequence
  if (tid < 2) found[3 * tid] = -1;
  __syncthreads();
  if (warp == 0) {  // the warps' sums to prefixes; the line's length; the two boundaries, before they
                    // move to an item's edge (none: 0 or the end of the line)
    const long long own = lane < NT / 32 ? sw[lane] : 0;
    long long up_to = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, up_to, o);
      if (lane >= o) up_to += up;
    }
    const long long total = __shfl_sync(0xffffffffu, up_to, 31);
    if (lane < NT / 32) sw[lane] = up_to - own;
    const long long want = min_unit == 1 ? total : div_pos(total + min_unit - 1, min_unit);
    const int n = (int)(want < nc ? (want > 0 ? want : 1) : nc);
    if (lane < 2) found[6 + lane] = c < n ? mul_div(c + lane, total, n) : total;
    if (lane == 0) {
      r->b = 0;
      r->tag = 0;
      r->off = 0;
      r->begin = 0;
      r->x0 = c < n ? 0 : total;
      r->x1 = total;
    }
  }
  __syncthreads();
  const long long pre = sw[warp] + inc - mine, total = r->x1;
  if (mine > 0) {
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const long long x = found[6 + k];
      if (x <= 0 || x >= total || x < pre || x >= pre + mine) continue;
      long long p = pre;
      for (int b = b0; b < b1; ++b) {
        const long long cb = b1 - b0 == 1 ? mine : f.cost(b);
        if (x < p + cb) {
          found[3 * k] = b;
          found[3 * k + 1] = x - p;
          found[3 * k + 2] = p;
          break;
        }
        p += cb;
      }
    }
  }
  __syncthreads();
  if (warp < 2 && found[3 * warp] >= 0) {
    const int b = (int)found[3 * warp];
    long long off = found[3 * warp + 1], s, e;
    const int tag = f.item(b, off, &s, &e);
    if (off - s < min_head) off = s;
    else if (e - off < min_tail) off = e;
    if (lane == 0) {
      if (warp == 0) {
        r->b = b;
        r->tag = tag;
        r->off = off;
        r->begin = s;
        r->x0 = found[2] + off;
      } else {
        r->x1 = found[5] + off;
      }
    }
  }
  __syncthreads();
}

// What a CTA records of its two partial results (slots 2c and 2c + 1), and of the
// item that slot 2c + 1 starts: all that the merge needs, in one load.
struct __align__(16) PartMeta {
  int state;  // 0: none, 1: the item goes on in the next CTA, 2: the item ends here
  int row;    // packed row of the sequence's (tile's) first token
  int first, count;  // the item's rows: their first (from `row`, in token * group + head), their number
  int head;   // K/V head
  int spare[3];
};

// A stretch's first CTA owns an item that slot 2c + 1 starts; its parts are
// that slot and slots 2c' of the CTAs behind it up to the first with state 2.
// part_count returns their number (0: nothing to merge), parts_from the same when
// an item is known to start there; part i > 0 is in slot 2 (c + i).
// Called by a whole warp: 32 states are read at a time.
__device__ __forceinline__ int parts_from(const PartMeta *meta, int nc, int c) {
  const int lane = threadIdx.x & 31;
  for (int n = 1; c + n < nc; n += 32) {
    const int at = c + n + lane;
    const int st = at < nc ? *const_cast<const volatile int *>(&meta[2 * at].state) : 2;
    const unsigned stop = __ballot_sync(0xffffffffu, st != 1);
    if (stop) {
      const int k = __ffs(stop) - 1;
      return n + k + (__shfl_sync(0xffffffffu, at < nc ? st : 0, k) == 2 ? 1 : 0);
    }
  }
  return nc - c;
}

__device__ __forceinline__ int part_count(const PartMeta *meta, int nc, int c) {
  return *const_cast<const volatile int *>(&meta[2 * c + 1].state) == 0 ? 0 : parts_from(meta, nc, c);
}

__device__ __forceinline__ int part_slot(int c, int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); }

// 16-byte stores of eight fp32 values in the output's type.
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(__half *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]),
                                             pack_half2(x[6], x[7]));
}

// Sixteen values of a row that lies far from the neighbouring lanes' rows: whole 32-byte
// sectors at a time when the address allows it (wide), else in 16-byte pieces.
__device__ __forceinline__ void store32b(void *p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16], bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
    store32b(p + 8 * h, w, wide);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  store32b(p, w, wide);
}
// A prompt's output is a mean of fp16 values: where rounded weights (off by 2^-11) carry it past the
// largest number of the type, it is that one and not infinity.  (NaN stays NaN.)
__device__ __forceinline__ uint32_t pack_half2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store16(__half *p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_half2_sat(x[2 * i], x[2 * i + 1]);
  store32b(p, w, wide);
}

__device__ __forceinline__ float2 unpack16(uint32_t w, const __half *) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack16(uint32_t w, const __nv_bfloat16 *) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

}  // namespace ispa

// kvq.cu -- writing rows into the quantised paged cache and reading them back.
//
// Both are one pass over their bytes.  Reading 23400 tokens of 12 heads takes 36.5 us in
// e4m3, 37 in int8 (218 MB, 5.9 TB/s, 0.9 of the measured copy rate) and 40 us in int4 (184 MB,
// 4.6 TB/s, 0.7): there the issue slots (75 % busy) and the integer pipe (71 %) bind, 474
// instructions a warp for 1024 values.  Writing as many is bound by its arithmetic: 46 us in
// int8, 51 in e4m3, 55 in int4 (662 instructions a warp for 1024 values, issue slots 76 % busy;
// 4680 tokens 10.7, 12.2 and 12.3 us).  A decoding step's few rows are bound by the launch.
// A row (one token of one head) is handled by d / 16 lanes, 16 values each: with 8 a
// lane the reductions and reciprocals of a row cost as much as its values.  A warp takes
// one token and up to kHeads heads of K and of V, whose loads are all issued before the
// first is used.
//
// The codes are those of real arithmetic, ties included, without a division an
// element.  A quotient a / b lies on a border t between two codes or on one side
// of it; with an approximate reciprocal it is first found to about 2^-22, rounded
// to the grid that holds the borders (halves for the integer codes, 5 significant
// bits for e4m3) as t, and then taken as t + (a - t b) / b: a - t b is exact in one
// fused operation (a = x times 127/128, 49/64 or 7/8 has at most 18 significant
// bits, b = amax times a 4-bit factor 15, t 9, and the difference is small), so the
// correction has the right sign, is zero exactly on the border, and otherwise at
// least 2^-20 of t, which the last addition keeps.
#include "kvq.cuh"
#include "seq.cuh"

namespace ispa {

namespace {

constexpr int kThreads = 256;
constexpr float kLeast = 0x1p-96f;  // rows below this are stored as zeros: their reciprocal scales overflow

struct RowParams {
  KvqView c;
  int B, T, H_kv;
  const int *cu, *lens, *begin;  // lens: write; begin: read (may be NULL)
  const void *k, *v;             // write: inputs
  void *ko, *vo;                 // read: outputs
  long long ks, vs;              // row strides in elements
  int *err;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 1 / b to about 2^-23, for b in [2^-120, 2^125]: the largest is int4's amax / 512 * g / 8 =
// 0.11 amax of the largest bf16 rows, and leaves one power of two to where the result is flushed.
__device__ __forceinline__ float reciprocal(float b) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
  return r;
}

// a / b to fp32, exactly on, or on the right side of, every multiple of 1 / 2 (|a / b| < 2^21).
__device__ __forceinline__ float exact_half(float a, float b, float inv) {
  const float t = __fadd_rn(fmaf(a, inv, 6291456.f), -6291456.f);  // 1.5 * 2^22: rounds to halves
  return fmaf(fmaf(-t, b, a), inv, t);
}
// The same for every number of 5 significant bits: the borders of e4m3.
__device__ __forceinline__ float exact_e4m3(float a, float b, float inv) {
  const float t = __uint_as_float((__float_as_uint(a * inv) + 0x40000u) & 0xfff80000u);
  return copysignf(fmaf(fmaf(-t, b, a), inv, t), a);  // (the sign of zero is kept)
}

// Sixteen codes rint(49 / 64 x / b) + 8, clamped if they may pass 7.  Two nibbles are joined
// as floats (n0 + 16 n1 + 136 in the last byte of 1.5 * 2^23 + that): integer operations are scarcer.
template <bool CLAMP>
__device__ __forceinline__ uint4 nibbles(const float (&x)[16], float b, float inv) {
  uint32_t byte[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float n[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float y = exact_half(x[2 * i + k] * (49.f / 64.f), b, inv);
      if (CLAMP) y = fminf(fmaxf(y, -7.f), 7.f);
      n[k] = __fadd_rn(y, 12582912.f);  // 1.5 * 2^23: rounds to the nearest even integer
    }
    byte[i] = __float_as_uint(fmaf(__fadd_rn(n[1], -12582912.f), 16.f, __fadd_rn(n[0], 136.f)));
  }
  return make_uint4(__byte_perm(__byte_perm(byte[0], byte[1], 0x40), __byte_perm(byte[2], byte[3], 0x40), 0x5410),
                    __byte_perm(__byte_perm(byte[4], byte[5], 0x40), __byte_perm(byte[6], byte[7], 0x40), 0x5410), 0u, 0u);
}

// Sixteen values of a row of W lanes: codes (16 or 8 bytes) and the row's scale record.
template <int FMT, int W>
__device__ __forceinline__ void quantise16(const float (&x)[16], uint4 &code, uint2 &rec) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) am = fmaxf(am, fabsf(x[i]));
  float group = am;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (o == 1) group = am;  // the two lanes of 32 channels
  }
  const bool some = am >= kLeast;
  const float div = some ? am : 1.f;
  if (FMT == ISPA_KVQ_INT4) {
    const float gb = div * (1.f / 512.f), ga = group * 0.875f;  // 448 group / amax = ga / gb
    const float ginv = reciprocal(gb);
    const uint32_t g8 = some ? e4m3x2(exact_e4m3(ga, gb, ginv), 0.f) & 0xffu : 0u;
    const bool on = g8 != 0;
    const float b = on ? gb * e4m3x2_to_float(g8).x * 0.125f : 1.f;  // 3136 x / (amax g) = (49 / 64 x) / b
    const float inv = on ? reciprocal(b) : 0.f;                      // (0: every n is 0)
    // |n| <= 7 / (1 - 2^-4) < 7.5 unless g is below its type's normal numbers
    code = __any_sync(0xffffffffu, g8 - 1u < 7u) ? nibbles<true>(x, b, inv) : nibbles<false>(x, b, inv);
    // the factors of the row's groups (two lanes hold each)
    uint32_t factors = g8 << (8 * ((threadIdx.x & (W - 1)) >> 1));
#pragma unroll
    for (int o = 2; o < W; o <<= 1) factors |= __shfl_xor_sync(0xffffffffu, factors, o);
    rec = make_uint2(__float_as_uint(some ? am / 3136.f : 0.f), factors);
  } else if (FMT == ISPA_KVQ_INT8) {
    const float b = div * (1.f / 128.f), inv = reciprocal(b);  // 127 x / amax = (127 / 128 x) / b, at most 127
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        n[i] = __float_as_uint(exact_half(x[4 * q + i] * (127.f / 128.f), b, inv) + 12582912.f);
      w[q] = some ? __byte_perm(__byte_perm(n[0], n[1], 0x40), __byte_perm(n[2], n[3], 0x40), 0x5410) : 0u;
    }
    code = make_uint4(w[0], w[1], w[2], w[3]);
    rec = make_uint2(__float_as_uint(some ? am / 127.f : 0.f), 0u);
  } else {
    const float b = div * (1.f / 512.f), inv = reciprocal(b);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = some ? e4m3x2(exact_e4m3(x[2 * i] * 0.875f, b, inv), exact_e4m3(x[2 * i + 1] * 0.875f, b, inv)) : 0u;
    code = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    rec = make_uint2(__float_as_uint(some ? am / 448.f : 0.f), 0u);
  }
}

// The last block of a launch has no rows: it looks over every sequence's bounds, those
// that no row falls in among them, beside the rows' way and not in front of it.
__device__ __forceinline__ bool bounds_block(const RowParams &P) {
  if (blockIdx.x + 1 != gridDim.x) return false;
  for (int b = threadIdx.x; b < P.B; b += kThreads)
    if (seq_rows_bad(P.cu, b, P.T)) report_seq(P.err, b);
  return true;
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kvq_write_kernel(RowParams P) {
  constexpr int W = D / 16;                       // lanes of a row
  constexpr int kRows = 32 / W;                   // rows of a pass: K and V of kStep heads
  constexpr int kHeads = 4, kStep = kRows / 2;    // heads of a warp, heads of a pass
  constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D, REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  if (bounds_block(P)) return;
  const int lane = threadIdx.x & 31;
  const int h_parts = (P.H_kv + kHeads - 1) / kHeads;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(item / h_parts), h0 = (int)(item % h_parts) * kHeads;
  if (t >= P.T) return;
  const int b = seq_of_row(P.cu, P.B, t);
  if (b < 0) return;
  const int sub = lane / W, l = lane % W;
  const bool is_v = sub >= kStep;
  const T *src = static_cast<const T *>(is_v ? P.v : P.k) + (long long)t * (is_v ? P.vs : P.ks) + l * 16;
  uint4 in[kHeads / kStep][2];
#pragma unroll
  for (int i = 0; i < kHeads / kStep; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      in[i][k] = h < P.H_kv ? __ldg(reinterpret_cast<const uint4 *>(src + (long long)h * D) + k) : make_uint4(0, 0, 0, 0);
  }
  const int c0 = __ldg(P.cu + b), c1 = __ldg(P.cu + b + 1);
  const long long pos = (long long)__ldg(P.lens + b) - (c1 - c0) + (t - c0);
  const int page = P.c.page(b, pos);
  if (page < 0) {
    if (lane == 0) report_seq(P.err, b);
    return;
  }
  const int place = (int)(pos & ((1 << P.c.page_log2) - 1));
  unsigned char *codes = is_v ? P.c.v_code : P.c.k_code, *scales = is_v ? P.c.v_scale : P.c.k_scale;
#pragma unroll
  for (int i = 0; i < kHeads / kStep; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    const uint32_t w[8] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w, in[i][1].x, in[i][1].y, in[i][1].z, in[i][1].w};
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = unpack16(w[j], static_cast<const T *>(nullptr));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
    uint4 code;
    uint2 rec;
    quantise16<FMT, W>(x, code, rec);
    if (h >= P.H_kv) continue;
    const long long row = P.c.row(page, h, place);
    if (FMT == ISPA_KVQ_INT4) {
      *reinterpret_cast<uint2 *>(codes + row * ROW + l * 8) = make_uint2(code.x, code.y);
      if (l == 0) *reinterpret_cast<uint2 *>(scales + row * REC) = rec;
    } else {
      *reinterpret_cast<uint4 *>(codes + row * ROW + l * 16) = code;
      if (l == 0) *reinterpret_cast<uint32_t *>(scales + row * REC) = rec.x;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) { return pack_half2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }

// Reading: a warp takes one token of up to four heads, all loads first.  Eight values a
// lane here, so that a warp's stores are whole lines (sixteen a lane: 43 us instead of 38 to 40
// for 23400 tokens of 12 heads in int4; two or four tokens a warp, or streaming stores: no change).
template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kvq_read_kernel(RowParams P) {
  constexpr int W = D / 8;
  constexpr int kRows = 32 / W;
  constexpr int kHeads = 4, kStep = kRows / 2, kN = kHeads / kStep;
  constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D, REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  if (bounds_block(P)) return;
  const int lane = threadIdx.x & 31;
  const int h_parts = (P.H_kv + kHeads - 1) / kHeads;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(item / h_parts), h0 = (int)(item % h_parts) * kHeads;
  if (t >= P.T) return;
  const int b = seq_of_row(P.cu, P.B, t);
  if (b < 0) return;
  const long long pos = (long long)(P.begin ? __ldg(P.begin + b) : 0) + (t - __ldg(P.cu + b));
  const int page = P.c.page(b, pos);
  if (page < 0 && lane == 0) report_seq(P.err, b);
  const int place = (int)(pos & ((1 << P.c.page_log2) - 1));
  const int sub = lane / W, l = lane % W;
  const bool is_v = sub >= kStep;
  const unsigned char *codes = is_v ? P.c.v_code : P.c.k_code, *scales = is_v ? P.c.v_scale : P.c.k_scale;
  uint2 code[kN], rec[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    code[i] = make_uint2(0u, 0u);
    rec[i] = make_uint2(0u, 0u);
    if (h >= P.H_kv || page < 0) continue;
    const long long row = P.c.row(page, h, place);
    if (FMT == ISPA_KVQ_INT4) {
      code[i].x = __ldg(reinterpret_cast<const uint32_t *>(codes + row * ROW + l * 4));
      rec[i] = __ldg(reinterpret_cast<const uint2 *>(scales + row * REC));
    } else {
      code[i] = __ldg(reinterpret_cast<const uint2 *>(codes + row * ROW + l * 8));
      rec[i].x = __ldg(reinterpret_cast<const uint32_t *>(scales + row * REC));
    }
  }
  T *dst = static_cast<T *>(is_v ? P.vo : P.ko) + (long long)t * P.H_kv * D + l * 8;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    if (h >= P.H_kv) continue;
    const float s = __uint_as_float(rec[i].x);
    const uint32_t w[2] = {code[i].x, code[i].y};
    float x[8];
    if (FMT == ISPA_KVQ_INT4) {
      const float sg = s * e4m3x2_to_float((rec[i].y >> (8 * (l >> 2))) & 0xffu).x;
      // 1.5 * 2^23 + n has n in its last bits: the conversion is one subtraction
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (__uint_as_float(0x4b400000u | ((w[0] >> (4 * j)) & 15u)) - 12582920.f) * sg;
    } else if (FMT == ISPA_KVQ_INT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (float)(int)(signed char)((w[j >> 2] >> (8 * (j & 3))) & 0xffu) * s;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_to_float((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
        x[2 * j] = f.x * s;
        x[2 * j + 1] = f.y * s;
      }
    }
    *reinterpret_cast<uint4 *>(dst + (long long)h * D) =
        page < 0 ? make_uint4(0u, 0u, 0u, 0u)
                 : make_uint4(pack16<T>(x[0], x[1]), pack16<T>(x[2], x[3]), pack16<T>(x[4], x[5]), pack16<T>(x[6], x[7]));
  }
}

template <int FMT, int D, typename T>
void launch_rows(const RowParams &P, bool write, unsigned grid, cudaStream_t s) {
  if (write)
    kvq_write_kernel<FMT, D, T><<<grid, kThreads, 0, s>>>(P);
  else
    kvq_read_kernel<FMT, D, T><<<grid, kThreads, 0, s>>>(P);
}

template <int FMT, int D>
void launch_rows_typed(const RowParams &P, bool write, ispa_dtype dt, unsigned grid, cudaStream_t s) {
  if (dt == ISPA_BF16)
    launch_rows<FMT, D, __nv_bfloat16>(P, write, grid, s);
  else
    launch_rows<FMT, D, __half>(P, write, grid, s);
}

template <int FMT>
void launch_rows_fmt(const RowParams &P, bool write, int d, ispa_dtype dt, unsigned grid, cudaStream_t s) {
  if (d == 128)
    launch_rows_typed<FMT, 128>(P, write, dt, grid, s);
  else
    launch_rows_typed<FMT, 64>(P, write, dt, grid, s);
}

ispa_status launch_kvq(const ispa_kvq_desc &d, RowParams P, bool write, ispa_dtype dt, cudaStream_t s) {
  DevErr e;
  ispa_status st = device_err(&e);
  if (st != ISPA_OK) return st;
  P.err = e.word;
  const long long items = (long long)P.T * ((d.H_kv + 3) / 4);
  const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32)) + 1;  // (and bounds_block)
  if (d.fmt == ISPA_KVQ_E4M3)
    launch_rows_fmt<ISPA_KVQ_E4M3>(P, write, d.head_dim, dt, grid, s);
  else if (d.fmt == ISPA_KVQ_INT8)
    launch_rows_fmt<ISPA_KVQ_INT8>(P, write, d.head_dim, dt, grid, s);
  else
    launch_rows_fmt<ISPA_KVQ_INT4>(P, write, d.head_dim, dt, grid, s);
  note_launch();
  return cuda_status(cudaGetLastError(), write ? "kvq_write launch" : "kvq_read launch");
}

}  // namespace

ispa_status launch_kvq_write(const ispa_kvq_desc &d, int B, int T, const int *table, int max_pages, const int *lens,
                             const int *cu, const void *k, long long ks, const void *v, long long vs, ispa_dtype dt,
                             void *kvq, cudaStream_t s) {
  RowParams P = {kvq_view(d, kvq, table, max_pages), B, T, d.H_kv, cu, lens, nullptr, k, v, nullptr, nullptr, ks, vs,
                 nullptr};
  return launch_kvq(d, P, true, dt, s);
}

ispa_status launch_kvq_read(const ispa_kvq_desc &d, int B, int T, const int *table, int max_pages, const int *begin,
                            const int *cu, const void *kvq, void *ko, void *vo, ispa_dtype dt, cudaStream_t s) {
  RowParams P = {kvq_view(d, kvq, table, max_pages), B, T, d.H_kv, cu, nullptr, begin, nullptr, nullptr, ko, vo, 0, 0,
                 nullptr};
  return launch_kvq(d, P, false, dt, s);
}

}  // namespace ispa

// attn_prompt.cu -- attention of packed prompts on tcgen05 tensor cores (bf16 or fp16, d = 64 or 128).
//
// A persistent CTA per SM walks an even stretch of the call's work (seq.cuh);
// an item is a pair of 128-row query tiles of one K/V head, a step one
// 128-key tile for both.  The rows of a tile are tokens x the H / H_kv heads
// that share the K/V head (row = token * group + head), so grouped heads share
// every K/V tile, short sequences fill the tiles better, and a causal tile's
// diagonal is 128 / group tokens wide.
//
// Warps (640 threads):
//   0-7    softmax and output of tile A: two threads a row (TMEM lane = row), 64 keys and
//          half of O's columns each; they exchange maxima and sums through shared memory
//   8-15   the same for tile B
//   16     TMA producer: the pair's Q tiles, then K_0, V_0, K_1, V_1, ... through one ring
//   17     TMEM allocator and MMA issuer (warp-uniform code, an elected lane issues)
//   18     scheduler: walks the stretch and hands the items on through a ring in shared
//          memory, so that no role on the critical path holds the walk's state (when every role
//          walked for itself, the spilled registers went to L2 -- shared memory leaves no
//          L1 -- and a step took 14 k cycles)
//   19     idle
// TMEM: S of A [0,128), S of B [128,256), O of A [256,256+d), O of B [384,384+d).
// P overwrites the first half of each thread's 64 score columns and is published in two
// parts (16-key steps 0 1 4 5, then 2 3 6 7), so that the second product starts while the
// second part is formed.  The issuer's order is
//   S_A0 S_B0 | PV_A0 S_A1 | PV_B0 S_B1 | PV_A1 S_A2 | ...
// so while one tile's warps work on its scores the tensor cores run the other tile's two
// products: the softmax's latency chain, which bounds a kernel with one tile in flight, is
// hidden behind the other tile.  Q and K come from shared memory (S is SS, PV is TS): a
// probe of the pair S + PV of a 128 x 128 x 128 tile back to back takes 1025 cycles, the
// nominal rate, with the TMEM loads and copies of the other roles running or not.
//
// What bounds it: a step takes about 3300 cycles for 2050 of MMAs.  The chain of a tile
// is 410 (scores in, maximum, exchange) + 190 + 2 x 680 (exponentials of 32 columns, two
// warps an SM sub-partition: 0.75 of the MUFU rate) + 230 until the weights are published,
// then 100 to the issuer and about 1000 for the products; the two tiles' exponentials
// nearly fill the MUFU.  Tried: an eighth to a half of the exponentials as polynomials on
// the FMA pipe (the same to 10 % slower), one thread a row with the scores in registers
// (spills), spinning waits, one pass over the scores with a late correction (spills).
//
// Measured (bf16, d = 128), in a graph of a few calls / in long runs at the power cap: 8192
// causal tokens, 32 heads on 8, 450 to 463 / 535 us, 1190 to 1220 / 1030 TFLOP/s (0.71 to 0.72 of
// the measured burst peak / 0.73 of the sustained one); 4680 queries over 32760 keys, 12 heads, 742
// to 843 / 875 us, 1270 to 1120 / 1080 TFLOP/s; six prompts of 545 to 2815 tokens 158 / 184 us, 890 /
// 760 TFLOP/s; 24 prompts of 1 to 300 tokens (d = 64) 13.7 us.  8192 tokens in fp16: 530 us; with
// d = 64 484 (bf16) and 435 us (fp16), 565 and 630 TFLOP/s: half the products for as many exponentials.
//
// Ordering (MMAs of one thread execute in order; a commit fires when all
// earlier ones have completed): S_{j+1} is issued after PV_j of the same tile,
// so it may overwrite P_j, and s_full(j + 1) says that O holds PV_0..PV_j: a
// softmax warp that has seen it may rescale O without a further wait, PV_{j+1}
// being held back by p_half(j + 1), which every warp of the tile signs.  The last
// PV of an item commits o_final; the next item's first PV overwrites O after the
// p_half that the same warps publish behind their reading of O.
//
// Keys: a tile past the end of its sequence holds rows of the next one, or
// zeros.  Scores there are replaced by -inf; in the second product only the
// 16-key steps that hold a visible key are issued, and the issuing warp zeroes
// the rows that remain of the last one (0 * Inf would not be 0).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "seq.cuh"

namespace ispa {

namespace {

constexpr int kThreads = 640;
constexpr int kTile = 128;
constexpr int kBox = 128 * 128;  // bytes of 128 rows x 64 columns
constexpr int kItem = 2;         // steps counted for an item besides its own: filling the pipeline, the output
constexpr int kMinPart = 6;      // steps that are worth cutting off
constexpr int kSegs = 4;         // items handed on ahead
constexpr int kSegReaders = 18;  // producer, issuer, sixteen softmax warps
// A row's reference lies `behind` below its largest score (log2) and moves when one passes it by
// more than `limit`, so that weights are at most 2^limit.  bf16 has fp32's range.  fp16 weights use
// what theirs has upwards (2^15), and the small ones of a long row keep their bits: a weight is
// off by at most 2^-25 where fp16's normal numbers end, 2^-32 of the row's largest.
template <typename T>
struct Ref {
  static constexpr float behind = 0.f, limit = 8.f;
};
template <>
struct Ref<__half> {
  static constexpr float behind = 7.f, limit = 15.f;
};
constexpr uint32_t kColS = 0, kColO = 256;

struct PromptParams {
  int B, H, H_kv, G, TQ;  // G = H / H_kv heads per K/V head, TQ = 128 / G tokens per tile
  int Tq, Tk, causal, nc;
  int wide;  // o is 32-byte aligned
  float scale_log2;
  const int *cu_q, *cu_k;
  void *o;
  float *lse;
  float *part;     // [2 nc][2 tiles][m 128 | l 128 | O as float4 [d / 4][128 rows]]
  PartMeta *meta;  // [2 nc]
  DevErr err;
};

template <int D>
constexpr int tile_floats() { return kTile * (D + 2); }

// sum over i < n of floor((a i + b) / m)
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += (long long)n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += (long long)n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return ans;
}

// What a step-line needs to know of one sequence.
struct PromptSeq {
  int q0, n, k0, len, past, pairs;  // past = len - n: keys before the first query (negative: fewer keys)
};

struct PromptCost {
  const int *cu_q, *cu_k;
  int Tq, Tk, TQ, H_kv, causal;
  __device__ PromptSeq seq(int b) const {
    const SeqRows q = seq_rows(cu_q, b, Tq), k = seq_rows(cu_k, b, Tk);
    return {q.begin, q.n, k.begin, k.n, k.n - q.n, (q.n + 2 * TQ - 1) / (2 * TQ)};
  }
  // keys that the queries below token index t of the sequence see at most
  __device__ int limit(const PromptSeq &s, int t) const { return causal ? s.past + min(t, s.n) : s.len; }
  // steps of a pair: kItem and its KV tiles
  __device__ int steps(const PromptSeq &s, int pair) const {
    return kItem + max(1, (limit(s, (pair + 1) * 2 * TQ) + kTile - 1) >> 7);
  }
  // steps of the pairs before `pair` (< s.pairs), all of them full
  __device__ long long before(const PromptSeq &s, int pair) const {
    return (long long)kItem * pair + tiles_before(s, pair);
  }
  __device__ long long tiles_before(const PromptSeq &s, int pair) const {
    if (!causal) return (long long)pair * max(1, (s.len + kTile - 1) >> 7);
    const int R = 2 * TQ;
    const bool pow2 = (R & (R - 1)) == 0;  // (as for every group of 2^k heads; the general sum is several divisions)
    const int lg = 31 - __clz(R);
    const int room = kTile - s.past;
    const int ones = min(pair, room <= 0 ? 0 : pow2 ? room >> lg : room / R);  // pairs of one step
    const int n = pair - ones;
    if (n == 0) return ones;
    const uint32_t b = s.past + (ones + 1) * R + kTile - 1;
    if (pow2) {
      if (R >= kTile) return ones + (long long)(R >> 7) * n * (n - 1) / 2 + (long long)n * (b >> 7);
      const int per = 7 - lg;  // floor((R i + b) / 128) = floor((i + floor(b / R)) / 2^per)
      auto sum = [per](long long x) {  // of floor(j / 2^per) over j < x
        const long long q = x >> per;
        return ((q * (q - 1) / 2) << per) + q * (x - (q << per));
      };
      return ones + sum((b >> lg) + n) - sum(b >> lg);
    }
    return ones + floor_sum(n, kTile, R, b);
  }
  __device__ long long head(const PromptSeq &s) const {
    return s.pairs ? before(s, s.pairs - 1) + steps(s, s.pairs - 1) : 0;
  }
  __device__ long long cost(int b) const { return head(seq(b)) * H_kv; }
  // whole warp: 32-way search for the last pair that starts at or before off; tag = the pair's number h * pairs + pair
  __device__ int item(int b, long long off, long long *s, long long *e) const {
    const PromptSeq q = seq(b);
    const long long line = head(q);
    const int h = (int)div_pos(off, line);
    const long long rem = off - h * line;
    int lo = 0, n = q.pairs;
    const int lane = threadIdx.x & 31;
    while (n > 1) {
      const int step = (n + 31) >> 5;
      const int at = min(lane * step, n - 1);
      const unsigned le = __ballot_sync(0xffffffffu, before(q, lo + at) <= rem);
      const int k = (__popc(le) - 1) * step;  // lane 0 always is
      const int skip = min(k, n - 1);
      lo += skip;
      n = min(step, n - skip);
    }
    *s = h * line + before(q, lo);
    *e = *s + steps(q, lo);
    return h * q.pairs + lo;
  }
};

// One item, or the part of it that falls in this CTA's stretch, as the roles see it.
struct PromptSeg {
  int mode;             // -1: no more work, 0: a part (result to `slot`), 1: the whole item
  int slot, h;
  int q_row, n_tok;     // first row of the pair's tokens, tokens of the pair (up to 2 TQ)
  int k_row, len, lim;  // first key row, keys, keys that the pair's first token sees
  int j0, end[2];       // KV tiles [j0, end[w]) of tile w
};

// The scheduler's walk over the stretch.
struct PromptWalk {
  long long left;
  int b, h, pair, j;
  int whole, id, stride;  // whole items id, id + stride, ... to take before the stretch (sequences all alike)
  PromptSeq s;
  __device__ void start(const PromptCost &c, const SplitRange &r) {
    left = r.x1 - r.x0;
    b = r.b;
    if (left <= 0) return;
    s = c.seq(b);
    h = s.pairs ? r.tag / s.pairs : 0;
    pair = s.pairs ? r.tag % s.pairs : 0;
    j = (int)(r.off - r.begin);
  }
  // (not inlined, with its state in shared memory: its registers would be taken from the roles' loops)
  __device__ __noinline__ bool next(const PromptCost &c, int B, const SplitRange &r, PromptSeg &g, PartMeta *meta) {
    if (whole > 0) {
      s = c.seq(0);
      const int line = c.H_kv * s.pairs;
      b = id / line;
      h = id % line / s.pairs;
      pair = id % s.pairs;
      s = c.seq(b);
      j = 0;
      left = c.steps(s, pair);
      id += stride;
    }
    if (left <= 0) return false;
    int total = pair < s.pairs ? c.steps(s, pair) : 0;
    while (j >= total) {  // on to the next item that has steps
      j = 0;
      if (++pair >= s.pairs) {
        pair = 0;
        if (++h >= c.H_kv || s.pairs == 0) {
          h = 0;
          do {
            if (++b >= B) return false;
            s = c.seq(b);
          } while (s.pairs == 0);
        }
      }
      total = c.steps(s, pair);
    }
    // step x of an item is its tile x - kItem (a boundary lies at x = 0 or well behind kItem)
    const int x1 = (int)min((long long)total, j + left);
    const int j0 = max(0, j - kItem), j1 = max(0, x1 - kItem);
    const int t0 = pair * 2 * c.TQ;
    g.h = h;
    g.q_row = s.q0 + t0;
    g.n_tok = min(2 * c.TQ, s.n - t0);
    g.k_row = s.k0;
    g.len = s.len;
    g.lim = c.causal ? s.past + t0 + 1 : s.len;
    g.j0 = j0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int lim = g.n_tok > w * c.TQ ? c.limit(s, t0 + (w + 1) * c.TQ) : 0;
      g.end[w] = max(j0, min(j1, (lim + kTile - 1) >> 7));
    }
    g.slot = j == 0 ? 1 : 0;
    g.mode = j == 0 && x1 == total ? 1 : 0;
    if (g.mode == 0) {
      const PartMeta m = {x1 == total ? 2 : 1, g.q_row, 0, g.n_tok, h, {}};
      meta[g.slot] = m;
    }
    left -= x1 - j;
    j = x1;
    if (whole > 0 && --whole == 0) start(c, r);
    return true;
  }
};

// The work of CTA c of nc when every item has the same steps (see the kernel).
__device__ __noinline__ void split_alike(const PromptCost &f, int B, int nc, int c, SplitRange *r, PromptWalk *w) {
  const PromptSeq s = f.seq(0);
  const int steps = f.steps(s, 0);
  const long long items = (long long)B * f.H_kv * s.pairs;
  w->whole = (int)(items / nc);
  w->id = c;
  w->stride = nc;
  const long long first = items / nc * nc, total = (items - first) * steps;
  const int n = (int)min((long long)nc, max(1LL, total));
  long long x[2];
  for (int k = 0; k < 2; ++k) {
    x[k] = (long long)min(c + k, n) * total / n;
    const long long off = x[k] % steps;
    if (off > 0 && off < kItem + kMinPart) x[k] -= off;
    else if (off > 0 && steps - off < kMinPart) x[k] += steps - off;
  }
  const long long item = first + x[0] / steps;
  const int line = f.H_kv * s.pairs;
  r->x0 = x[0];
  r->x1 = c < n ? x[1] : x[0];
  r->b = (int)min(item / line, (long long)B - 1);
  r->tag = (int)(item % line);
  r->off = x[0] % steps;
  r->begin = 0;
}

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = HALVES * kBox;
  static constexpr int STAGES = D == 128 ? 5 : 8;
};

template <int D>
struct PromptSmem {
  uint8_t q[2][Cfg<D>::TILE];
  uint8_t ring[Cfg<D>::STAGES][Cfg<D>::TILE];
  uint64_t full[Cfg<D>::STAGES], empty[Cfg<D>::STAGES];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], o_final[2], swapped[2];
  uint64_t drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  float swap[2][2][kTile];  // per tile: what the two threads of a row tell each other
  PromptSeg seg[kSegs];
  PromptWalk walk;
  long long scratch[kThreads / 32 + 8];
  SplitRange range;
  uint32_t tmem_base;
  int abort;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) { return pack_half2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// MMAs issued from warp-uniform code: every lane executes the statement with the
// same operands and the elected one issues, so that descriptors and addresses stay in
// uniform registers (inside an `if (lane == 0)` each of them had to be moved there,
// about 100 cycles an MMA beside two busy softmax warps).  Descriptors are given by
// their low words; the high word (stride 1024, version 1, 128-byte swizzle) is constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss_u(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%2, %6};\n\tmov.b64 db, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], da, db, %4, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_u(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%3, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], db, %4, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_commit_u(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
      "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *m, uint64_t *bar, int x, int y, int z, int w,
                                            int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
      : "memory");
}

template <int D, typename T, typename TO>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, PromptParams P) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PromptSmem<D> &sm = *reinterpret_cast<PromptSmem<D> *>(smem_raw);
  if (smem_u32(smem_raw) & 1023u) {  // the operand tiles need it; nothing static lies in front
    if (threadIdx.x == 0) report_error(P.err, ISPA_ERR_CUDA, 48);
    return;
  }
  volatile int *abort = &sm.abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const PromptCost cost = {P.cu_q, P.cu_k, P.Tq, P.Tk, P.TQ, P.H_kv, P.causal};

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sm.s_full[w], 1);
      mbar_init(&sm.p_half[w], 8);
      mbar_init(&sm.p_full[w], 8);
      mbar_init(&sm.swapped[w], 8);
      mbar_init(&sm.o_final[w], 1);
    }
    mbar_init(&sm.drain, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&sm.seg_full[i], 1);
      mbar_init(&sm.seg_empty[i], kSegReaders);
    }
    sm.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    asm volatile("griddepcontrol.launch_dependents;");  // the merge may take its place on the SMs; it waits for this grid
    P.meta[2 * blockIdx.x].state = 0;
    P.meta[2 * blockIdx.x + 1].state = 0;
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < P.B; b += kThreads)
      if (seq_rows_bad(P.cu_q, b, P.Tq) || seq_rows_bad(P.cu_k, b, P.Tk)) report_error(P.err, ISPA_ERR_INVALID_ARG, b);
  if (warp == 17) tmem_alloc(&sm.tmem_base, 512);
  // Sequences that are all alike and see every key (the chunks of a batch of instances): as many
  // whole items as there are for every CTA come first, one each a round, so that the CTAs of
  // one head read the same keys at the same time and the L2 holds them (4680 queries over 32760
  // keys, 12 heads, 201 MB of K and V: 881 -> 742 us); only the rest is cut into stretches.
  bool alike = !P.causal;
  if (alike) {
    const PromptSeq s0 = cost.seq(0);
    for (int b = threadIdx.x; b < P.B; b += kThreads) {
      const PromptSeq s1 = cost.seq(b);
      alike = alike && s1.n == s0.n && s1.len == s0.len;
    }
    alike = __syncthreads_and(alike) && s0.n > 0;
  }
  if (alike) {
    if (threadIdx.x == 0) split_alike(cost, P.B, P.nc, blockIdx.x, &sm.range, &sm.walk);
  } else {
    if (threadIdx.x == 0) sm.walk.whole = 0;
    split_range<kThreads>(cost, P.B, P.nc, blockIdx.x, 1, kItem + kMinPart, kMinPart, &sm.range, sm.scratch);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
  // item i of the stretch, for the roles: seg_wait, read, seg_done
  uint32_t n_seg = 0;
  auto seg_wait = [&]() -> const PromptSeg * {
    const uint32_t i = n_seg % kSegs;
    return wait_parity(&sm.seg_full[i], (n_seg / kSegs) & 1, P.err, abort, 50) ? &sm.seg[i] : nullptr;
  };
  auto seg_done = [&]() {  // one lane of each reading warp
    mbar_arrive(&sm.seg_empty[n_seg % kSegs]);
    ++n_seg;
  };

  if (warp >= 16) {
    // 128 x 64 + 512 x 104 registers: the 640 x 96 of the launch, and no spill in the softmax's loop
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 18) {
      // ---------------------------------------------------------- scheduler
      if (lane == 0) {
        if (sm.walk.whole == 0) sm.walk.start(cost, sm.range);
        for (bool more = true; more; ++n_seg) {
          const uint32_t i = n_seg % kSegs;
          if (!wait_parity(&sm.seg_empty[i], ((n_seg / kSegs) & 1) ^ 1, P.err, abort, 49)) break;
          more = sm.walk.next(cost, P.B, sm.range, sm.seg[i], P.meta + 2 * blockIdx.x);
          if (!more) sm.seg[i].mode = -1;
          mbar_arrive(&sm.seg_full[i]);
        }
      }
    } else if (warp == 16) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        uint32_t n_ring = 0, pend = 0, ph_bits = 0, n_q = 0;
        bool ok = true;
        auto load = [&](const CUtensorMap *m, int row, int h) {
          const uint32_t st = n_ring % C::STAGES, ph = (n_ring / C::STAGES) & 1;
          ++n_ring;
          if (!wait_parity(&sm.empty[st], ph ^ 1, P.err, abort, 51)) return false;
          mbar_arrive_expect_tx(&sm.full[st], C::TILE);
          tma_load_4d(sm.ring[st], m, &sm.full[st], 0, row, 0, h);
          pend |= 1u << st;
          ph_bits = (ph_bits & ~(1u << st)) | (ph << st);
          return true;
        };
        while (ok) {
          const PromptSeg *g = seg_wait();
          if (!g || g->mode < 0) break;
          const int j0 = g->j0, end = max(g->end[0], g->end[1]), h = g->h, k_row = g->k_row, q_row = g->q_row;
          seg_done();
          if (end == j0) continue;  // no key in sight: nothing to load
          ok = wait_parity(&sm.q_empty, (n_q & 1) ^ 1, P.err, abort, 52);
          if (!ok) break;
          mbar_arrive_expect_tx(&sm.q_full, 2 * C::HALVES * P.G * P.TQ * 128);
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int f = 0; f < C::HALVES; ++f)
              tma_load_5d(sm.q[w] + f * kBox, &tq, &sm.q_full, 0, 0, q_row + w * P.TQ, f, h);
          ++n_q;
          for (int j = j0; ok && j < end; ++j) {
            ok = load(&tk, k_row + j * kTile, h);
            if (ok) ok = load(&tv, k_row + j * kTile, h);
          }
        }
        if (*abort) {  // let copies in flight land before the CTA exits
          for (int st = 0; st < C::STAGES; ++st)
            if (pend & (1u << st)) wait_parity_drain(&sm.full[st], (ph_bits >> st) & 1, P.err);
          if (n_q) wait_parity_drain(&sm.q_full, (n_q - 1) & 1, P.err);
        }
      }
    } else if (warp == 17) {
      // ---------------------------------------------------------- MMA issuer
      constexpr int fmt = std::is_same<T, __half>::value ? 0 : 1;
      constexpr uint32_t idesc_s = make_idesc(128, 128, fmt, 0, 0);   // Q (K-major) x K (K-major)
      constexpr uint32_t idesc_pv = make_idesc(128, D, fmt, 0, 1);    // P (TMEM) x V (MN-major)
      const uint32_t leader = elect_one();
      const uint32_t dq = ((smem_u32(sm.q[0]) >> 4) & 0x3fffu) | (1u << 16);
      const uint32_t dk = ((smem_u32(sm.ring[0]) >> 4) & 0x3fffu) | (1u << 16);
      const uint32_t dv = ((smem_u32(sm.ring[0]) >> 4) & 0x3fffu) | ((uint32_t)(kBox >> 4) << 16);
      uint32_t st = 0, ph = 0;    // ring stage of the next tile to be consumed, and its phase
      uint32_t n_q = 0, ph_p = 0;  // phases of q_full and, one bit a tile, of p_full
      bool ok = true;
      auto advance = [&](uint32_t &s, uint32_t &p) {
        if (++s == C::STAGES) {
          s = 0;
          p ^= 1;
        }
      };
      auto issue_s = [&](int w, uint32_t stage) {
        const uint32_t qd = dq + ((w * C::TILE) >> 4), kd = dk + stage * (C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
          mma_ss_u(leader, tmem + kColS + w * 128, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit_u(leader, &sm.s_full[w]);
      };
      while (true) {
        const PromptSeg *g = seg_wait();
        ok = __all_sync(0xffffffffu, g != nullptr);
        if (!ok) break;
        // (through a shuffle: uniform for the compiler too)
        auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const int mode = uni(g->mode), j0 = uni(g->j0), end0 = uni(g->end[0]), end1 = uni(g->end[1]);
        const int len = uni(g->len), n_tok = uni(g->n_tok), lim = uni(g->lim);
        if (mode < 0) break;
        const int end = max(end0, end1);
        // keys that the rows of each tile see at most
        const int lim0 = P.causal ? lim + min(P.TQ, n_tok) - 1 : len;
        const int lim1 = P.causal ? lim + min(2 * P.TQ, n_tok) - 1 : len;
        if (lane == 0) seg_done();
        else ++n_seg;
        __syncwarp();
        if (end == j0) continue;
        ok = wait_parity(&sm.q_full, n_q, P.err, abort, 53) && wait_parity(&sm.full[st], ph, P.err, abort, 54);
        n_q ^= 1;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (j0 < end0) issue_s(0, st);
        if (j0 < end1) issue_s(1, st);
        mma_commit_u(leader, &sm.empty[st]);
        if (end == j0 + 1) mma_commit_u(leader, &sm.q_empty);
        advance(st, ph);
#pragma unroll 1
        for (int j = j0; j < end; ++j) {
          const uint32_t sv = st;
          ok = wait_parity(&sm.full[st], ph, P.err, abort, 55);
          advance(st, ph);
          const uint32_t sk = st;
          if (j + 1 < end) {
            if (ok) ok = wait_parity(&sm.full[st], ph, P.err, abort, 56);
            advance(st, ph);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int left = len - j * kTile;  // keys of the sequence in this tile
          if (left < kTile && (left & 15)) {
            // rows left .. the end of their 16-key step belong to the next sequence
            uint8_t *v = sm.ring[sv];
            const int n16 = (16 - (left & 15)) * 8;
            for (int i = lane; i < n16 * C::HALVES; i += 32)
              *reinterpret_cast<uint4 *>(v + (i / n16) * kBox + left * 128 + (i % n16) * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          const uint32_t vd = dv + sv * (C::TILE >> 4);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int my_end = w ? end1 : end0;
            if (j < my_end) {
              const int k_steps = (min(kTile, (w ? lim1 : lim0) - j * kTile) + 15) >> 4;
              const uint32_t a_p = tmem + kColS + w * 128, d_o = tmem + kColO + w * 128;
#pragma unroll
              for (int part = 0; part < 2; ++part) {  // the weights come in two parts: 16-key steps 0 1 4 5, then 2 3 6 7
                ok = wait_parity(part ? &sm.p_full[w] : &sm.p_half[w], (ph_p >> w) & 1, P.err, abort, 57 + w);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int kk = (i >> 1) * 4 + part * 2 + (i & 1);
                  if (kk < k_steps)
                    mma_ts_u(leader, d_o, a_p + kk * 8 + (kk >> 2) * 32, vd + kk * (2048 >> 4), idesc_pv,
                             kk > 0 || j > j0 ? 1u : 0u);
                }
              }
              ph_p ^= 1u << w;
              if (!ok) break;
              if (j + 1 < my_end)
                issue_s(w, sk);
              else
                mma_commit_u(leader, &sm.o_final[w]);
            }
          }
          if (!ok) break;
          mma_commit_u(leader, &sm.empty[sv]);
          if (j + 1 < end) mma_commit_u(leader, &sm.empty[sk]);
          if (j + 2 == end) mma_commit_u(leader, &sm.q_empty);
        }
        if (!ok) break;
      }
      if (!ok) {
        mma_commit_u(leader, &sm.drain);
        wait_parity_drain(&sm.drain, 0, P.err);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int w = warp >> 3, half = (warp >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;  // row of the tile == TMEM lane
    const int tok = r / P.G, head = r % P.G;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = lane_base + kColS + w * 128 + half * 64;        // this thread's 64 scores
    const uint32_t col_o = lane_base + kColO + w * 128 + half * (D / 2);   // and its half of O
    float *mine = &sm.swap[w][half][r], *theirs = &sm.swap[w][half ^ 1][r];
    uint32_t n_s = 0, n_o = 0, n_x = 0;
    auto swap_sync = [&]() {  // the tile's eight warps; bounded like every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.swapped[w]);
      const bool ok = wait_parity(&sm.swapped[w], n_x & 1, P.err, abort, 65 + w);
      ++n_x;
      return (bool)__all_sync(0xffffffffu, ok);
    };
    bool ok = true;
    while (ok) {
      const PromptSeg *g = seg_wait();
      if (!__all_sync(0xffffffffu, g != nullptr) || g->mode < 0) break;
      const int t = w * P.TQ + tok;  // this row's token in the pair
      const bool row_ok = tok < P.TQ && t < g->n_tok;
      const int lim = P.causal ? g->lim + t : g->len;
      const int lim_first = P.causal ? g->lim + w * P.TQ : g->len;
      const int j0 = g->j0, end = g->end[w], mode = g->mode, slot = 2 * blockIdx.x + g->slot;
      const int out_row = g->q_row + (row_ok ? t : 0), out_head = g->h * P.G + head;
      __syncwarp();
      if (lane == 0) seg_done();
      else ++n_seg;
      float m_ref = 0.f, l = 0.f;
      for (int j = j0; j < end; ++j) {
        ok = wait_parity(&sm.s_full[w], n_s & 1, P.err, abort, 61 + w);
        ++n_s;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // the scores are read twice, 32 columns at a time: registers are scarcer than that bandwidth
        const bool edge = (j + 1) * kTile > lim_first;  // the diagonal, or the sequence's end
        const int valid = lim - j * kTile - half * 64;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t x[32];
          tmem_ld32(col_s + c * 32, x);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int t = 0; t < 32; ++t)
              if (c * 32 + t >= valid) x[t] = 0xff800000u;
          }
#pragma unroll
          for (int t = 0; t < 32; t += 2)
            mx[(t >> 1) & 3] = max3(mx[(t >> 1) & 3], __uint_as_float(x[t]), __uint_as_float(x[t + 1]));
        }
        float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        *mine = mt;
        ok = swap_sync();
        if (!ok) break;
        mt = fmaxf(mt, *theirs) * P.scale_log2;
        if (j == j0) {
          m_ref = mt == -INFINITY ? 0.f : mt - Ref<T>::behind;
        } else if (__any_sync(0xffffffffu, row_ok && mt > m_ref + Ref<T>::limit)) {
          // (rows that are none hold what lies behind the sequence, or in shared memory behind TQ G rows:
          // they must not move the others, whose roundings would depend on it)
          const float m_new = fmaxf(m_ref, mt - Ref<T>::behind);
          const float f = exp2_fast(m_ref - m_new);
          m_ref = m_new;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 16) {
            uint32_t o[16];
            tmem_ld16(col_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
            tmem_st16(col_o + c, o);
          }
        }
        // P = 2^(s scale log2e - m_ref) in the input type, over the first 64 columns of S
        const float2 sc2 = make_float2(P.scale_log2, P.scale_log2), nm2 = make_float2(-m_ref, -m_ref);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t y[32], pk[16];
          tmem_ld32(col_s + c * 32, y);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int t = 0; t < 32; ++t)
              if (c * 32 + t >= valid) y[t] = 0xff800000u;
          }
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const float2 x =
                fma2(make_float2(__uint_as_float(y[2 * t]), __uint_as_float(y[2 * t + 1])), sc2, nm2);
            const float2 pp = make_float2(exp2_fast(x.x), exp2_fast(x.y));
            ls[t & 1] = add2(ls[t & 1], pp);
            pk[t] = pack2<T>(pp.x, pp.y);
          }
          tmem_st16(col_s + c * 16, pk);  // over scores that have been read
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(c == 0 ? &sm.p_half[w] : &sm.p_full[w]);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      }
      if (!ok) break;
      // ---- the segment's output
      if (end > j0) {
        ok = wait_parity(&sm.o_final[w], n_o & 1, P.err, abort, 63 + w);
        ++n_o;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        *mine = l;
        ok = swap_sync();
        if (!ok) break;
        l += *theirs;
        ok = swap_sync();  // read before the next item's first maximum takes its place
        if (!ok) break;
      }
      const bool some = l != 0.f;  // (a sum that is NaN stays so)
      if (mode == 1) {
        const float inv = some ? 1.f / l : 0.f;
        const long long out = (long long)out_row * P.H + out_head;
        TO *dst = static_cast<TO *>(P.o) + out * D + half * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t raw[16];
          if (end > j0) {
            tmem_ld16(col_o + c, raw);
            tmem_wait_ld();
          }
          if (!row_ok) continue;
          float x[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) x[t] = some ? __uint_as_float(raw[t]) * inv : 0.f;
          store16(dst + c, x, P.wide);
        }
        if (row_ok && half == 0 && P.lse) P.lse[out] = some ? (m_ref + log2f(l)) * 0.69314718055994530942f : -INFINITY;
      } else {
        float *part = P.part + ((size_t)slot * 2 + w) * tile_floats<D>();
        if (half == 0) {
          part[r] = some ? m_ref : -INFINITY;
          part[kTile + r] = l;
        }
        float4 *po = reinterpret_cast<float4 *>(part + 2 * kTile) + half * (D / 8) * kTile + r;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t raw[16];
          if (end > j0) {
            tmem_ld16(col_o + c, raw);
            tmem_wait_ld();
          }
#pragma unroll
          for (int v = 0; v < 4; ++v)
            po[(c / 4 + v) * kTile] =
                some ? make_float4(__uint_as_float(raw[4 * v]), __uint_as_float(raw[4 * v + 1]),
                                   __uint_as_float(raw[4 * v + 2]), __uint_as_float(raw[4 * v + 3]))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      tc_fence_before();  // O is read before the p_half that lets the next item overwrite it
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// Joins the parts of the item that slot 2c + 1 starts: block (c, tile, 32 columns), one row per thread.
template <int D, typename TO>
__global__ void __launch_bounds__(kTile) prompt_merge_kernel(PromptParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, w = blockIdx.y, c0 = blockIdx.z * 32, r = threadIdx.x;
  const int n = part_count(P.meta, P.nc, c);
  if (n == 0) return;
  const PartMeta own = P.meta[2 * c + 1];
  const int tok = r / P.G, head = r % P.G, t = w * P.TQ + tok;
  if (tok >= P.TQ || t >= own.count) return;
  auto at = [&](int k) { return P.part + ((size_t)part_slot(c, k) * 2 + w) * tile_floats<D>(); };
  float mm = -INFINITY, ll = 0.f, x[32] = {};
#pragma unroll 2
  for (int k = 0; k < n; ++k) {
    const float *p = at(k);
    const float mk = p[r], lk = p[kTile + r];
    const float4 *po = reinterpret_cast<const float4 *>(p + 2 * kTile) + (c0 / 4) * kTile + r;
    float4 a[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) a[v] = po[v * kTile];
    const float to = fmaxf(mm, mk), ref = to == -INFINITY ? 0.f : to;
    const float f0 = exp2_fast(mm - ref), f = exp2_fast(mk - ref);
    mm = to;
    ll = ll * f0 + lk * f;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      x[4 * v] = x[4 * v] * f0 + a[v].x * f, x[4 * v + 1] = x[4 * v + 1] * f0 + a[v].y * f;
      x[4 * v + 2] = x[4 * v + 2] * f0 + a[v].z * f, x[4 * v + 3] = x[4 * v + 3] * f0 + a[v].w * f;
    }
  }
  const long long out = (long long)(own.row + t) * P.H + own.head * P.G + head;
  const float inv = ll == 0.f ? 0.f : 1.f / ll;  // (a sum that is NaN stays so)
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float y[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) y[t] = x[16 * v + t] * inv;
    store16(static_cast<TO *>(P.o) + out * D + c0 + v * 16, y, P.wide);
  }
  if (P.lse && c0 == 0) P.lse[out] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
}

template <int D, typename T, typename TO>
ispa_status launch_one(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PromptParams &P,
                       cudaStream_t s) {
  auto kern = attn_prompt_kernel<D, T, TO>;
  constexpr int smem = sizeof(PromptSmem<D>);
  static_assert(smem <= 232448, "shared memory of a block");
  static std::atomic<void *> prepared{nullptr};
  ispa_status st = allow_smem(reinterpret_cast<const void *>(kern), smem, prepared, "attn_prompt shared memory");
  if (st != ISPA_OK) return st;
  kern<<<P.nc, kThreads, smem, s>>>(tq, tk, tv, P);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e, "attn_prompt launch");
  // no item is cut when none can have two parts' worth of KV tiles
  if ((P.Tk + kTile - 1) / kTile < 2 * kMinPart) return ISPA_OK;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.nc, 2, D / 32);
  cfg.blockDim = dim3(kTile);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prompt_merge_kernel<D, TO>, P);
  note_launch();
  return cuda_status(e, "prompt_merge launch");
}

template <int D>
ispa_status launch_typed(const ispa_attn_seq_desc &d, const CUtensorMap &tq, const CUtensorMap &tk,
                         const CUtensorMap &tv, const PromptParams &P, cudaStream_t s) {
  const bool f32 = d.out_dtype == ISPA_F32;
  if (d.in_dtype == ISPA_BF16)
    return f32 ? launch_one<D, __nv_bfloat16, float>(tq, tk, tv, P, s)
               : launch_one<D, __nv_bfloat16, __nv_bfloat16>(tq, tk, tv, P, s);
  return f32 ? launch_one<D, __half, float>(tq, tk, tv, P, s) : launch_one<D, __half, __half>(tq, tk, tv, P, s);
}

}  // namespace

size_t attn_prompt_workspace_bytes(int head_dim) {
  const size_t nc = sm_count();
  return 2 * nc * (sizeof(PartMeta) + (size_t)2 * kTile * (head_dim + 2) * 4);
}

ispa_status launch_attn_prompt(const ispa_attn_seq_desc &d, float scale, int Tq, int Tk, const int *cu_q,
                               const int *cu_k, const void *q, long long qs, const void *k, long long ks,
                               const void *v, long long vs, void *o, float *lse, void *workspace, cudaStream_t s) {
  PromptParams P;
  ispa_status st = device_err(&P.err);
  if (st != ISPA_OK) return st;
  P.B = d.B;
  P.H = d.H;
  P.H_kv = d.H_kv;
  P.G = d.H / d.H_kv;
  P.TQ = kTile / P.G;
  P.Tq = Tq;
  P.Tk = Tk;
  P.causal = d.causal;
  P.nc = sm_count();
  P.wide = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  P.scale_log2 = scale * 1.4426950408889634f;
  P.cu_q = cu_q;
  P.cu_k = cu_k;
  P.o = o;
  P.lse = lse;
  P.meta = static_cast<PartMeta *>(workspace);
  P.part = reinterpret_cast<float *>(P.meta + 2 * P.nc);
  const CUtensorMapDataType dt =
      d.in_dtype == ISPA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int D = d.head_dim;
  CUtensorMap tq, tk, tv;
  {
    // 64 columns | heads of the group | tokens | column halves | K/V heads
    const uint64_t dims[5] = {64, (uint64_t)P.G, (uint64_t)Tq, (uint64_t)D / 64, (uint64_t)d.H_kv};
    const uint64_t str[4] = {(uint64_t)D * 2, (uint64_t)qs * 2, 128, (uint64_t)P.G * D * 2};
    const uint32_t box[5] = {64, (uint32_t)P.G, (uint32_t)P.TQ, 1, 1};
    st = make_tmap(&tq, dt, 5, q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != ISPA_OK) return st;
  }
  for (int i = 0; i < 2; ++i) {
    // without a key (Tk == 0) no tile is loaded: the maps then describe q's first rows
    const uint64_t dims[4] = {64, (uint64_t)std::max(Tk, 1), (uint64_t)D / 64, (uint64_t)d.H_kv};
    const uint64_t str[3] = {(uint64_t)(i ? vs : ks) * 2, 128, (uint64_t)D * 2};
    const uint32_t box[4] = {64, (uint32_t)kTile, (uint32_t)D / 64, 1};
    st = make_tmap(i ? &tv : &tk, dt, 4, Tk == 0 ? q : (i ? v : k), dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != ISPA_OK) return st;
  }
  return D == 128 ? launch_typed<128>(d, tq, tk, tv, P, s) : launch_typed<64>(d, tq, tk, tv, P, s);
}

}  // namespace ispa

// attn_kvq.cu -- attention of a sequence's newest tokens over its quantised paged cache.
//
// For one sequence and one K/V head the query rows are the n new tokens times
// the group's H / H_kv heads (row = token * group + head), taken 16 at a time:
// one 16-row operand of the m16n8k16 matrix instruction, so that a decoding
// step's grouped heads share every byte of the cache.  The work is bound by
// the cache's bytes; the matrix instructions only have to keep up with them
// (16 rows x 2 d flop a byte), which the register-fed form does without the
// 128-row tiles and tensor-memory round trips of the prompt kernel.
//
// A CTA's eight warps work on the same 16 rows and each on every eighth
// 32-token tile, with a private softmax state and a private ring of tiles in
// shared memory, filled by asynchronous 16-byte copies straight from the pages
// (the page of a tile is looked up one tile ahead; tokens past the length are
// filled with zeros, so nothing that lies there matters).  No barrier is
// needed until the states are merged at the end of the CTA's stretch of an
// item (seq.cuh); parts of an item that other CTAs hold are merged by
// kvq_merge_kernel.
//
// Codes go into fp16 exactly: e4m3 and int8 values as they are, int4 values
// times the group's e4m3 factor (7 significant bits).  The per-token scales
// are applied outside the products: K's to the scores in fp32, V's to the
// softmax weights before they are rounded to fp16 (relative to the largest V
// scale seen, as a power of two, so that the weights stay in fp16's range).
// Channels are assigned to operand positions so that each lane's bytes of a
// row are contiguous: Q is permuted to match, and O comes out in runs of d/8.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kvq.cuh"
#include "seq.cuh"

namespace ispa {

namespace {

constexpr int kRows = 16;   // query rows of an item
constexpr int kTile = 32;   // tokens of a warp's tile
constexpr int kMinUnit = 8;       // tiles a CTA gets at least
constexpr int kMinPart = 4;
constexpr float kRescale = 8.f;   // the reference maximum moves when passed by more than this (log2)
constexpr float kNegInf = -INFINITY;

struct KvqParams {
  KvqView c;
  int B, T, H, G;             // G = H / H_kv
  int cap;                    // max_pages * page_tokens: bound of a length
  int causal, nc;
  float scale_log2;
  const int *cu, *lens;
  const void *q;
  long long qs;
  void *o;
  float *lse;
  float *part;                // [2 nc][part_floats]
  PartMeta *meta;             // [2 nc]
  int *err;
};

template <int D>
constexpr int part_floats() { return kRows * (D + 2); }

// Steps of a sequence: tiles x row blocks x heads.
struct KvqCost {
  const int *cu, *lens;
  int T, cap, G, H_kv;
  __device__ int blocks(int b) const { return (int)(((long long)seq_rows(cu, b, T).n * G + kRows - 1) / kRows); }
  __device__ int tiles(int b) const { return max(1, (seq_len(lens, b, cap) + kTile - 1) / kTile); }
  __device__ long long cost(int b) const { return (long long)blocks(b) * H_kv * tiles(b); }
  __device__ int item(int b, long long off, long long *s, long long *e) const {
    const int t = tiles(b);
    *s = off / t * t;
    *e = *s + t;
    return 0;
  }
};

template <int FMT, int D>
struct Geo {
  static constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D;
  static constexpr int REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  static constexpr int CPR = ROW / 16;  // 16-byte chunks of a row
  static constexpr int CODE = kTile * ROW, SCALE = kTile * REC;
  static constexpr int STAGE = 2 * (CODE + SCALE);
  // As many warps and stages as shared memory holds, two stages at least: the chain of
  // a tile (scores, maximum, weights, product) has to be hidden by other warps.
  // (168 registers a thread with 12 warps, 128 with 16: d = 128 needs the former for O's 64.)
  static constexpr int WARPS = D == 128 ? 12 : 16;
  static constexpr int STAGES = (220 << 10) / (WARPS * STAGE) < 4 ? (220 << 10) / (WARPS * STAGE) : 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int KS = D / 16;  // k steps of the first product
  static constexpr int NB = D / 8;   // n blocks of the second
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int MERGE = WARPS * kRows * (D + 2) * 4;
  static constexpr int QBYTES = KS * 32 * 16;
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + QBYTES + 256;

  // Byte offset of a 16-byte chunk of a K row / V row in its tile.  K is read
  // by lanes (row lane / 4, chunk lane % 4 [+ 4]), V by lanes (rows 2 (lane % 4)
  // + {0, 1, 8, 9}, d / 8 channels from (lane / 4) d / 8); the swaps put each
  // group of lanes that the shared memory serves together on distinct banks.
  static __device__ __forceinline__ int k_off(int row, int ch) {
    return row * ROW + (CPR == 8 ? ch ^ ((row & 1) << 2) : ch) * 16;
  }
  static __device__ __forceinline__ int v_off(int row, int ch) {
    if (CPR == 8) return row * ROW + (ch ^ (row & 6)) * 16;
    const int pos = (row & ~7) | ((row & 1) << 2) | ((row >> 1) & 3);
    return pos * ROW + (CPR == 4 ? ch ^ (pos & 2) : ch) * 16;
  }
  // Operand position of channel ch of Q: k step, lane % 4, half of the step, element.
  static __device__ __forceinline__ void q_pos(int ch, int &ks, int &t, int &half, int &e) {
    if (FMT == ISPA_KVQ_INT4) {  // a lane has d / 4 channels; nibbles c and c + 4 of a word make a pair
      t = ch / (D / 4);
      const int w = ch % (D / 4) / 8, c = ch % 8;
      e = c >> 2;
      ks = w * 2 + ((c & 3) >> 1);
      half = c & 1;
    } else {  // a lane has chunks t and t + 4 (d = 128) or chunk t (d = 64)
      const int chunk = ch / 16;
      t = chunk & 3;
      ks = (chunk >> 2) * 4 + (ch % 16) / 4;
      half = (ch >> 1) & 1;
      e = ch & 1;
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// Four code bytes as two pairs of fp16 (bytes 0, 1 and bytes 2, 3).
template <int FMT>
__device__ __forceinline__ void four_codes(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (FMT == ISPA_KVQ_INT8) {  // 1024 + 128 + x as fp16 bits, then minus 1152: exact
    w ^= 0x80808080u;
    lo = hsub2(prmt(w, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2(prmt(w, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    lo = e4m3x2_to_half2(w & 0xffffu);
    hi = e4m3x2_to_half2(w >> 16);
  }
}
// Nibble i of both 16-bit halves of a word as fp16 values (n - 8) f, exactly: with the nibble
// in mantissa bits 4..7 of 1024 the fp16 number is 1024 + 16 n, and (1024 + 16 n) (f / 16) - 72 f
// is one fused operation whose operands (f has 4 significant bits) and result (7) are fp16 numbers.
struct Factor {
  uint32_t sixteenth, minus72;  // pairs f / 16 and -72 f
  __device__ __forceinline__ explicit Factor(uint32_t f) : sixteenth(hmul2(f, 0x2c002c00u)), minus72(hmul2(f, 0xd480d480u)) {}
};
__device__ __forceinline__ uint32_t two_nibbles(uint32_t w, int i, const Factor &f) {
  const uint32_t at4 = i == 0 ? w << 4 : i == 1 ? w : w >> (4 * (i - 1));
  return hfma2((at4 & 0x00f000f0u) | 0x64006400u, f.sixteenth, f.minus72);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One 32-token tile of K and V (codes and scale records) into a ring stage.
template <int FMT, int D>
__device__ __forceinline__ void load_tile(const KvqView &c, uint32_t dst, int h, int tok0, int len, int pg0, int pg1) {
  using Ge = Geo<FMT, D>;
  const int lane = threadIdx.x & 31;
  const int mask = (1 << c.page_log2) - 1;
  constexpr int RPI = 32 / Ge::CPR;  // rows of one pass of the warp
  const int ch = lane % Ge::CPR, r0 = lane / Ge::CPR;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int pg = half ? pg1 : pg0, t0 = tok0 + half * 16;
    const long long row0 = c.row(pg < 0 ? 0 : pg, h, t0 & mask);
    const unsigned char *ks = c.k_code + row0 * Ge::ROW, *vs = c.v_code + row0 * Ge::ROW;
#pragma unroll
    for (int i = 0; i < 16 / RPI; ++i) {
      const int r = i * RPI + r0;
      const bool on = pg >= 0 && t0 + r < len;
      const int off = on ? r * Ge::ROW + ch * 16 : 0;
      cp_async16(dst + Ge::k_off(half * 16 + r, ch), ks + off, on ? 16 : 0);
      cp_async16(dst + Ge::CODE + Ge::v_off(half * 16 + r, ch), vs + off, on ? 16 : 0);
    }
    // scale records: 16 REC bytes of each half, lanes 0.. of K then of V
    constexpr int SC = 16 * Ge::REC / 16;
    if (lane < 2 * SC) {
      const int i = lane % SC;
      const int tok = t0 + i * (16 / Ge::REC);
      const int bytes = pg >= 0 ? min(16, max(0, (len - tok) * Ge::REC)) : 0;
      const unsigned char *s = (lane < SC ? c.k_scale : c.v_scale) + row0 * Ge::REC + (bytes ? i * 16 : 0);
      cp_async16(dst + 2 * Ge::CODE + (lane < SC ? 0 : Ge::SCALE) + half * 16 * Ge::REC + i * 16, s, bytes);
    }
  }
}

// fp32 scales of tokens nb * 8 + 2t and + 1 of a tile.
template <int REC>
__device__ __forceinline__ float2 two_scales(const unsigned char *rec, int tok) {
  if (REC == 4) return *reinterpret_cast<const float2 *>(rec + tok * 4);
  const float4 f = *reinterpret_cast<const float4 *>(rec + tok * 8);
  return make_float2(f.x, f.z);
}

template <int FMT, int D, typename T, typename TO>
__global__ void __launch_bounds__(Geo<FMT, D>::THREADS, 1) attn_kvq_kernel(KvqParams P) {
  using Ge = Geo<FMT, D>;
  constexpr int kWarps = Ge::WARPS, kThreads = Ge::THREADS;
  // fp16 outputs are as fine as fp16 weights: these then enter as a sum of two fp16 numbers
  constexpr bool kTwoParts = std::is_same<T, __half>::value;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ SplitRange range;
  __shared__ long long scratch[kWarps + 6];
  __shared__ float q_unscale[kRows];
  unsigned char *qh = smem + (Ge::RING > Ge::MERGE ? Ge::RING : Ge::MERGE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const KvqCost cost = {P.cu, P.lens, P.T, P.cap, P.G, P.c.H_kv};
  if (threadIdx.x < 2) P.meta[2 * blockIdx.x + threadIdx.x].state = 0;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < P.B; b += kThreads)
      if (seq_rows_bad(P.cu, b, P.T) || __ldg(P.lens + b) != seq_len(P.lens, b, P.cap)) report_seq(P.err, b);
  split_range<kThreads>(cost, P.B, P.nc, blockIdx.x, kMinUnit, kMinPart, &range, scratch);

  long long left = range.x1 - range.x0;
  int b = range.b;
  long long off = range.off;
  unsigned char *ring = smem + warp * Ge::STAGES * Ge::STAGE;
  const uint32_t ring_u = smem_u32(ring);

  while (left > 0) {
    // ---- the next item of the stretch
    const SeqRows rows = seq_rows(P.cu, b, P.T);
    const int blocks = cost.blocks(b), tiles = cost.tiles(b);
    if (off >= (long long)blocks * P.c.H_kv * tiles) {
      ++b;
      off = 0;
      continue;
    }
    const int len = seq_len(P.lens, b, P.cap);
    const int item = (int)(off / tiles), t_begin = (int)(off % tiles);
    const int t_end = (int)min((long long)tiles, t_begin + left);
    const int h = item / blocks, rb = item % blocks;
    const int n_rows = min(kRows, rows.n * P.G - rb * kRows);
    // ---- this warp's first tiles are on their way while Q is laid out
    const int my0 = t_begin + warp;
    int bad = 0;
    auto pages = [&](int tile, int &p0, int &p1) {
      p0 = p1 = -1;
      if (tile < t_end && tile * kTile < len) {
        p0 = P.c.page(b, tile * kTile);
        bad |= p0 < 0;
        if (tile * kTile + 16 < len) {
          p1 = P.c.page(b, tile * kTile + 16);
          bad |= p1 < 0;
        }
      }
    };
    int np0, np1;
#pragma unroll
    for (int s = 0; s < Ge::STAGES - 1; ++s) {
      const int tile = my0 + s * kWarps;
      pages(tile, np0, np1);
      if (tile < t_end) load_tile<FMT, D>(P.c, ring_u + s * Ge::STAGE, h, tile * kTile, len, np0, np1);
      cp_commit();
    }
    pages(my0 + (Ge::STAGES - 1) * kWarps, np0, np1);

    // ---- Q: 16 rows as fp16, scaled by a power of two per row, in operand order
    for (int r = warp; r < kRows; r += kWarps) {
      constexpr int PER = D / 32;
      float x[PER];
      float am = 0.f;
      const int rr = rb * kRows + r;
      if (r < n_rows) {
        const int tok = rows.begin + rr / P.G, head = h * P.G + rr % P.G;
        const T *src = static_cast<const T *>(P.q) + (long long)tok * P.qs + (long long)head * D + lane * PER;
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
          const float2 f = unpack16(__ldg(reinterpret_cast<const uint32_t *>(src) + i), static_cast<const T *>(nullptr));
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) am = fmaxf(am, fabsf(x[i]));
      am = warp_max(am);
      // largest entry in [2^14, 2^15); rows of zeros and non-finite rows stay as they are
      const int e = am > 0.f && am < INFINITY ? min(14 - ilogbf(am), 126) : 0;
      const float up = ldexpf(1.f, e);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        int ks, t, half, el;
        Ge::q_pos(lane * PER + i, ks, t, half, el);
        const int reg = half * 2 + (r >> 3);
        reinterpret_cast<__half *>(qh)[((ks * 32 + (r & 7) * 4 + t) * 4 + reg) * 2 + el] = __float2half_rn(x[i] * up);
      }
      if (lane == 0) q_unscale[r] = P.scale_log2 * ldexpf(1.f, -e);
    }
    __syncthreads();
    const uint4 *qf = reinterpret_cast<const uint4 *>(qh) + lane;  // operand of k step ks: qf[32 ks]
    const float un0 = q_unscale[g], un1 = q_unscale[g + 8];
    // keys that rows g and g + 8 may see
    const int past = len - rows.n + 1;
    const int lim0 = P.causal ? min(len, past + (rb * kRows + g) / P.G) : len;
    const int lim1 = P.causal ? min(len, past + (rb * kRows + g + 8) / P.G) : len;
    const int lim_all = P.causal ? min(len, past + (rb * kRows) / P.G) : len;  // the first row sees the fewest

    float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
    int ve = -200;  // exponent of the largest V scale so far: weights enter the product times 2^(6 - ve)
    float acc[Ge::NB][4];
#pragma unroll
    for (int j = 0; j < Ge::NB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

    int stage = 0;
    for (int tile = my0; tile < t_end; tile += kWarps) {
      cp_wait<Ge::STAGES - 2>();
      __syncwarp();
      {  // refill the stage read in the last round
        const int nt = tile + (Ge::STAGES - 1) * kWarps;
        const int ns = stage == 0 ? Ge::STAGES - 1 : stage - 1;
        if (nt < t_end) load_tile<FMT, D>(P.c, ring_u + ns * Ge::STAGE, h, nt * kTile, len, np0, np1);
        cp_commit();
        pages(nt + kWarps, np0, np1);
      }
      const unsigned char *kc = ring + stage * Ge::STAGE, *vc = kc + Ge::CODE, *kr = vc + Ge::CODE,
                          *vr = kr + Ge::SCALE;
      stage = stage + 1 == Ge::STAGES ? 0 : stage + 1;

      // ---- scores: 16 rows x 32 tokens, times K's scale (the row's factor comes with the exponent)
      float s[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nb][i] = 0.f;
      if (FMT == ISPA_KVQ_INT4) {
        constexpr int WORDS = D / 32;  // words of this lane's D / 4 channels
#pragma unroll
        for (int np = 0; np < 4; np += 2) {
          uint32_t w[2][WORDS];
          uint32_t f[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int row = (np + n) * 8 + g;
            if (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4 *>(kc + Ge::k_off(row, t4));
              w[n][0] = v.x, w[n][1] = v.y, w[n][WORDS - 2] = v.z, w[n][WORDS - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(kc + row * Ge::ROW + t4 * 8);
              w[n][0] = v.x, w[n][1] = v.y;
            }
            f[n] = kr[row * 8 + 4 + t4 * (D / 4) / 32];
          }
          const Factor fa(e4m3x2_to_half2(f[0] | f[0] << 8)), fb(e4m3x2_to_half2(f[1] | f[1] << 8));
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            const uint4 q0 = qf[64 * i], q1 = qf[64 * i + 32];
            mma16816(s[np], q0, two_nibbles(w[0][i], 0, fa), two_nibbles(w[0][i], 1, fa));
            mma16816(s[np + 1], q0, two_nibbles(w[1][i], 0, fb), two_nibbles(w[1][i], 1, fb));
            mma16816(s[np], q1, two_nibbles(w[0][i], 2, fa), two_nibbles(w[0][i], 3, fa));
            mma16816(s[np + 1], q1, two_nibbles(w[1][i], 2, fb), two_nibbles(w[1][i], 3, fb));
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 v[4];
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) v[nb] = *reinterpret_cast<const uint4 *>(kc + Ge::k_off(nb * 8 + g, t4 + 4 * c));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 q0 = qf[32 * (4 * c + i)];
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              uint32_t b0, b1;
              four_codes<FMT>(i == 0 ? v[nb].x : i == 1 ? v[nb].y : i == 2 ? v[nb].z : v[nb].w, b0, b1);
              mma16816(s[nb], q0, b0, b1);
            }
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const float2 ksc = two_scales<Ge::REC>(kr, nb * 8 + 2 * t4);
        s[nb][0] *= ksc.x;
        s[nb][1] *= ksc.y;
        s[nb][2] *= ksc.x;
        s[nb][3] *= ksc.y;
      }
      if (tile * kTile + kTile > lim_all) {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          const int tok = tile * kTile + nb * 8 + 2 * t4;
          if (tok >= lim0) s[nb][0] = kNegInf;
          if (tok + 1 >= lim0) s[nb][1] = kNegInf;
          if (tok >= lim1) s[nb][2] = kNegInf;
          if (tok + 1 >= lim1) s[nb][3] = kNegInf;
        }
      }
      if (bad) {  // tokens whose page does not exist are left out
        int p0, p1;
        const int keep = bad;
        pages(tile, p0, p1);
        bad = keep;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          if ((nb < 2 ? p0 : p1) < 0) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = kNegInf;
      }

      // ---- running maximum and V scale; O follows when they move
      float mx0 = kNegInf, mx1 = kNegInf, vmx = 0.f;
      float2 vsc[4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        mx0 = fmaxf(mx0, fmaxf(s[nb][0], s[nb][1]));
        mx1 = fmaxf(mx1, fmaxf(s[nb][2], s[nb][3]));
        vsc[nb] = two_scales<Ge::REC>(vr, nb * 8 + 2 * t4);
        vmx = fmaxf(vmx, fmaxf(vsc[nb].x, vsc[nb].y));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        vmx = fmaxf(vmx, __shfl_xor_sync(0xffffffffu, vmx, o));
      }
      mx0 *= un0;
      mx1 *= un1;
      const int et = (int)(__float_as_uint(vmx) >> 23) - 127;  // floor(log2), -127 for zeros
      if (__any_sync(0xffffffffu, mx0 > m0 + kRescale || mx1 > m1 + kRescale || (m0 == kNegInf && mx0 > kNegInf) ||
                                      (m1 == kNegInf && mx1 > kNegInf) || et > ve)) {
        const float n0 = mx0 > m0 ? mx0 : m0, n1 = mx1 > m1 ? mx1 : m1;
        const float f0 = m0 == kNegInf ? 0.f : exp2_fast(m0 - n0), f1 = m1 == kNegInf ? 0.f : exp2_fast(m1 - n1);
        const int nv = max(ve, et);
        const float fv = ve == -200 ? 0.f : exp2_fast((float)(ve - nv));
        m0 = n0;
        m1 = n1;
        ve = nv;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < Ge::NB; ++j) {
          acc[j][0] *= f0 * fv;
          acc[j][1] *= f0 * fv;
          acc[j][2] *= f1 * fv;
          acc[j][3] *= f1 * fv;
        }
      }
      const float r0 = m0 == kNegInf ? 0.f : m0, r1 = m1 == kNegInf ? 0.f : m1;
      const float vup = __uint_as_float((uint32_t)(min(127 + 6 - ve, 254)) << 23);  // 2^(6 - ve)
      uint32_t pa[2][4], pl[2][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const float p0 = exp2_fast(fmaf(s[nb][0], un0, -r0)), p1 = exp2_fast(fmaf(s[nb][1], un0, -r0));
        const float p2 = exp2_fast(fmaf(s[nb][2], un1, -r1)), p3 = exp2_fast(fmaf(s[nb][3], un1, -r1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        const float va = vsc[nb].x * vup, vb = vsc[nb].y * vup;
        const float w0 = p0 * va, w1 = p1 * vb, w2 = p2 * va, w3 = p3 * vb;
        const uint32_t h0 = pack_half2(w0, w1), h1 = pack_half2(w2, w3);
        pa[nb >> 1][(nb & 1) * 2] = h0;
        pa[nb >> 1][(nb & 1) * 2 + 1] = h1;
        if (kTwoParts) {
          const float2 f0 = unpack16(h0, static_cast<const __half *>(nullptr));
          const float2 f1 = unpack16(h1, static_cast<const __half *>(nullptr));
          pl[nb >> 1][(nb & 1) * 2] = pack_half2(w0 - f0.x, w1 - f0.y);
          pl[nb >> 1][(nb & 1) * 2 + 1] = pack_half2(w2 - f1.x, w3 - f1.y);
        }
      }
      auto product = [&](float(&c)[4], int kb, uint32_t b0, uint32_t b1) {
        mma16816(c, make_uint4(pa[kb][0], pa[kb][1], pa[kb][2], pa[kb][3]), b0, b1);
        if (kTwoParts) mma16816(c, make_uint4(pl[kb][0], pl[kb][1], pl[kb][2], pl[kb][3]), b0, b1);
      };

      // ---- O += P V
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const int r = kb * 16 + 2 * t4;
        if (FMT == ISPA_KVQ_INT4) {
          constexpr int WORDS = D / 64;
          uint32_t w[4][WORDS];
          uint32_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = r + (i & 1) + (i >> 1) * 8;
            if (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2 *>(vc + Ge::v_off(row, g >> 1) + (g & 1) * 8);
              w[i][0] = v.x, w[i][WORDS - 1] = v.y;
            } else {
              w[i][0] = *reinterpret_cast<const uint32_t *>(vc + Ge::v_off(row, g >> 2) + (g & 3) * 4);
            }
            f[i] = vr[row * 8 + 4 + g * (D / 8) / 32];
          }
          const Factor fa(e4m3x2_to_half2(f[0] | f[1] << 8)), fb(e4m3x2_to_half2(f[2] | f[3] << 8));
#pragma unroll
          for (int i = 0; i < WORDS; ++i)
#pragma unroll
            for (int hw = 0; hw < 2; ++hw) {  // 16-bit halves of the words: channels 0-3, 4-7
              const uint32_t xa = prmt(w[0][i], w[1][i], hw ? 0x7632 : 0x5410);
              const uint32_t xb = prmt(w[2][i], w[3][i], hw ? 0x7632 : 0x5410);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                product(acc[i * 8 + hw * 4 + c], kb, two_nibbles(xa, c, fa), two_nibbles(xb, c, fb));
            }
        } else {
          constexpr int WORDS = D / 32;
          uint32_t w[4][WORDS];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = r + (i & 1) + (i >> 1) * 8;
            if (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4 *>(vc + Ge::v_off(row, g));
              w[i][0] = v.x, w[i][1] = v.y, w[i][WORDS - 2] = v.z, w[i][WORDS - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(vc + Ge::v_off(row, g >> 1) + (g & 1) * 8);
              w[i][0] = v.x, w[i][1] = v.y;
            }
          }
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
            four_codes<FMT>(prmt(w[0][i], w[1][i], 0x5140), a0, a1);
            four_codes<FMT>(prmt(w[0][i], w[1][i], 0x7362), a2, a3);
            four_codes<FMT>(prmt(w[2][i], w[3][i], 0x5140), b0, b1);
            four_codes<FMT>(prmt(w[2][i], w[3][i], 0x7362), b2, b3);
            product(acc[4 * i], kb, a0, b0);
            product(acc[4 * i + 1], kb, a1, b1);
            product(acc[4 * i + 2], kb, a2, b2);
            product(acc[4 * i + 3], kb, a3, b3);
          }
        }
      }
    }
    if (bad && lane == 0) report_seq(P.err, b);

    // ---- merge the warps' states (the rings are idle now)
    cp_wait<0>();
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);  // [warp][m 16 | l 16 | O 16 x D]
    {
      float *mine = mg + warp * kRows * (D + 2);
      if (t4 == 0) {
        mine[g] = m0;
        mine[g + 8] = m1;
        mine[kRows + g] = l0;
        mine[kRows + g + 8] = l1;
      }
      const float vdown = ve == -200 ? 0.f : __uint_as_float((uint32_t)(max(127 + ve - 6, 0)) << 23);
      float *oo = mine + 2 * kRows;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < Ge::NB; j += 4) {
          const int ch = (2 * t4 + e) * Ge::NB + j;
          *reinterpret_cast<float4 *>(oo + g * D + ch) =
              make_float4(acc[j][e] * vdown, acc[j + 1][e] * vdown, acc[j + 2][e] * vdown, acc[j + 3][e] * vdown);
          *reinterpret_cast<float4 *>(oo + (g + 8) * D + ch) = make_float4(
              acc[j][2 + e] * vdown, acc[j + 1][2 + e] * vdown, acc[j + 2][2 + e] * vdown, acc[j + 3][2 + e] * vdown);
        }
    }
    __syncthreads();
    const bool whole = t_begin == 0 && t_end == tiles;
    const int slot = 2 * blockIdx.x + (t_begin == 0 ? 1 : 0);
    float *part = P.part + (size_t)slot * part_floats<D>();
    for (int i = threadIdx.x; i < n_rows * (D / 8); i += kThreads) {
      const int r = i / (D / 8), c8 = i % (D / 8) * 8;
      float mm = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, mg[w * kRows * (D + 2) + r]);
      const float ref = mm == kNegInf ? 0.f : mm;
      float ll = 0.f, x[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float *st = mg + w * kRows * (D + 2);
        const float f = exp2_fast(st[r] - ref);
        ll += st[kRows + r] * f;
        const float4 a = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8);
        const float4 c = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8 + 4);
        x[0] += a.x * f, x[1] += a.y * f, x[2] += a.z * f, x[3] += a.w * f;
        x[4] += c.x * f, x[5] += c.y * f, x[6] += c.z * f, x[7] += c.w * f;
      }
      if (whole) {
        const int rr = rb * kRows + r;
        const long long out = (long long)(rows.begin + rr / P.G) * P.H + h * P.G + rr % P.G;
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv;
        store8(static_cast<TO *>(P.o) + out * D + c8, x);
        if (P.lse && c8 == 0) P.lse[out] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994530942f : kNegInf;
      } else {
        if (c8 == 0) {
          part[r] = mm;
          part[kRows + r] = ll;
        }
        store8(part + 2 * kRows + r * D + c8, x);
      }
    }
    if (!whole && threadIdx.x == 0) {
      PartMeta *m = P.meta + slot;
      m->b = b;
      m->item = item;
      m->state = t_end == tiles ? 2 : 1;
    }
    __syncthreads();  // the merge area is the next item's ring
    left -= t_end - t_begin;
    off += t_end - t_begin;
  }
}

// Joins the parts of the item that slot 2c + 1 starts (c = blockIdx.x).
template <int D, typename TO>
__global__ void __launch_bounds__(256) kvq_merge_kernel(KvqParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int n = part_count(P.meta, P.nc, c);
  if (n == 0) return;
  const int b = P.meta[2 * c + 1].b, item = P.meta[2 * c + 1].item;
  const SeqRows rows = seq_rows(P.cu, b, P.T);
  const int blocks = (int)(((long long)rows.n * P.G + kRows - 1) / kRows);
  const int h = item / blocks, rb = item % blocks;
  const int n_rows = min(kRows, rows.n * P.G - rb * kRows);
  for (int i = threadIdx.x; i < n_rows * (D / 8); i += blockDim.x) {
    const int r = i / (D / 8), c8 = i % (D / 8) * 8;
    float mm = kNegInf;
    for (int k = 0; k < n; ++k) mm = fmaxf(mm, P.part[(size_t)part_slot(c, k) * part_floats<D>() + r]);
    const float ref = mm == kNegInf ? 0.f : mm;
    float ll = 0.f, x[8] = {};
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float *st = P.part + (size_t)part_slot(c, k) * part_floats<D>();
      const float f = exp2_fast(st[r] - ref);
      ll += st[kRows + r] * f;
      const float4 a = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8);
      const float4 d = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8 + 4);
      x[0] += a.x * f, x[1] += a.y * f, x[2] += a.z * f, x[3] += a.w * f;
      x[4] += d.x * f, x[5] += d.y * f, x[6] += d.z * f, x[7] += d.w * f;
    }
    const int rr = rb * kRows + r;
    const long long out = (long long)(rows.begin + rr / P.G) * P.H + h * P.G + rr % P.G;
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] *= inv;
    store8(static_cast<TO *>(P.o) + out * D + c8, x);
    if (P.lse && c8 == 0) P.lse[out] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994530942f : kNegInf;
  }
}

template <int FMT, int D, typename T, typename TO>
ispa_status launch_one(const KvqParams &P, cudaStream_t s) {
  using Ge = Geo<FMT, D>;
  auto kern = attn_kvq_kernel<FMT, D, T, TO>;
  static std::atomic<void *> prepared{nullptr};
  ispa_status st = allow_smem(reinterpret_cast<const void *>(kern), Ge::SMEM, prepared, "attn_kvq shared memory");
  if (st != ISPA_OK) return st;
  kern<<<P.nc, Ge::THREADS, Ge::SMEM, s>>>(P);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e, "attn_kvq launch");
  // the merge is launched ahead of the kernel's end and waits for it on the device
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.nc);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kvq_merge_kernel<D, TO>, P);
  note_launch();
  return cuda_status(e, "kvq_merge launch");
}

template <int FMT, int D>
ispa_status launch_typed(const KvqParams &P, ispa_dtype in, ispa_dtype out, cudaStream_t s) {
  if (in == ISPA_BF16)
    return out == ISPA_F32 ? launch_one<FMT, D, __nv_bfloat16, float>(P, s)
                           : launch_one<FMT, D, __nv_bfloat16, __nv_bfloat16>(P, s);
  return out == ISPA_F32 ? launch_one<FMT, D, __half, float>(P, s) : launch_one<FMT, D, __half, __half>(P, s);
}

}  // namespace

size_t attn_kvq_workspace_bytes(int head_dim) {
  const size_t nc = sm_count();
  return 2 * nc * (sizeof(PartMeta) + (size_t)kRows * (head_dim + 2) * 4);
}

ispa_status launch_attn_kvq(const ispa_attn_seq_desc &d, const ispa_kvq_desc &c, float scale, int T, const int *cu_q,
                            const int *table, int max_pages, const int *lens, const void *q, long long qs,
                            const void *kvq, void *o, float *lse, void *workspace, cudaStream_t s) {
  DevErr e;
  ispa_status st = device_err(&e);
  if (st != ISPA_OK) return st;
  KvqParams P;
  P.c = kvq_view(c, kvq, table, max_pages);
  P.B = d.B;
  P.T = T;
  P.H = d.H;
  P.G = d.H / d.H_kv;
  P.cap = (int)std::min<long long>((long long)max_pages * c.page_tokens, 1LL << 30);
  P.causal = d.causal;
  P.nc = sm_count();
  P.scale_log2 = scale * 1.4426950408889634f;
  P.cu = cu_q;
  P.lens = lens;
  P.q = q;
  P.qs = qs;
  P.o = o;
  P.lse = lse;
  P.meta = static_cast<PartMeta *>(workspace);
  P.part = reinterpret_cast<float *>(P.meta + 2 * P.nc);
  P.err = e.word;
  const int f = c.fmt * 2 + (c.head_dim == 128 ? 1 : 0);
  switch (f) {
    case ISPA_KVQ_E4M3 * 2: return launch_typed<ISPA_KVQ_E4M3, 64>(P, d.in_dtype, d.out_dtype, s);
    case ISPA_KVQ_E4M3 * 2 + 1: return launch_typed<ISPA_KVQ_E4M3, 128>(P, d.in_dtype, d.out_dtype, s);
    case ISPA_KVQ_INT8 * 2: return launch_typed<ISPA_KVQ_INT8, 64>(P, d.in_dtype, d.out_dtype, s);
    case ISPA_KVQ_INT8 * 2 + 1: return launch_typed<ISPA_KVQ_INT8, 128>(P, d.in_dtype, d.out_dtype, s);
    case ISPA_KVQ_INT4 * 2: return launch_typed<ISPA_KVQ_INT4, 64>(P, d.in_dtype, d.out_dtype, s);
    default: return launch_typed<ISPA_KVQ_INT4, 128>(P, d.in_dtype, d.out_dtype, s);
  }
}

}  // namespace ispa

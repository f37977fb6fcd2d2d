// attn_kvq.cu -- attention of a sequence's newest tokens over its quantised paged cache.
//
// For one sequence and one K/V head the query rows are the n new tokens times
// the group's H / H_kv heads (row = token * group + head), taken 8 or 16 at a
// time.  The work is bound by the cache's bytes and, close behind, by the
// instructions that turn codes into operands, so the rows are the narrow side of
// the matrix instruction (m16n8k16): 16 tokens of K (or 16 channels of V) times
// 16 channels (tokens) are one operand, 8 rows the other.  Scores are formed as
// S^T = K Q^T, and O^T = V^T P^T; P^T is S^T transposed in 8 x 8 blocks by
// movmatrix.
//
// A CTA's four warps work on the same rows and each on every fourth 32-token
// tile, with a private softmax state and a private ring of tiles in shared memory,
// filled by asynchronous 16-byte copies straight from the pages (the page of a tile
// is looked up one tile ahead; tokens past the length are filled with zeros, so
// nothing that lies there matters).  No barrier is needed until the states are merged
// at the end of the CTA's stretch of an item (seq.cuh); parts of an item that other
// CTAs hold are merged by kvq_merge_kernel.  Two to four CTAs share an SM, so that
// an item's start and end in one are covered by the others: 48 sequences of 200 to
// 16000 tokens took 137 us with one CTA of 12 warps an SM and items counted by their
// tiles, 78 us (71 now) with four warps and an item's fixed cost counted.
//
// Measured: those 48 sequences (406 MB, e4m3, 8 heads of 128, groups of 4) 71 us,
// 5.7 TB/s, 0.87 of the measured copy rate; 102960 tokens of 40 heads in int4 (593 MB)
// 145 us, 4.1 TB/s, 0.62, bound by issue slots and the integer pipe (800 instructions
// a 32-token tile, of which 160 unpack nibbles; issue slots 64 % busy, integer pipe 51 %,
// DRAM 47 %); one sequence of 999 tokens 10.4 us, of 16000 18.7 us.
//
// No kernel spills but int4's with d = 128, fp16 inputs and blocks of 8 rows (16 bytes a thread).
//
// Codes go into fp16 exactly: e4m3 and int8 values as they are, int4 values
// times the group's e4m3 factor (7 significant bits).  The per-token scales
// are applied outside the products: K's to the scores in fp32, V's to the
// softmax weights before they are rounded to fp16.  A weight times its V scale
// enters the product times a power of two of its row, which puts the largest such
// product among the row's own visible keys so far between 2^9 and 2^15: keys that a row
// does not see, or gives no weight, do not move it, however large their V.  A weight is
// then off by at most 2^-34 of the row's largest product where fp16 has no 11 bits left.
// Channels are assigned to operand positions so that each lane's bytes of a
// row are contiguous: Q is permuted to match, and O comes out in runs of d/8.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kvq.cuh"
#include "seq.cuh"

namespace ispa {

namespace {

constexpr int kMaxRows = 16;  // query rows of an item: 8 NR, NR = 1 or 2 blocks of 8
constexpr int kTile = 32;   // tokens of a warp's tile
constexpr int kMinUnit = 4;       // tiles a CTA gets at least: one per warp
constexpr int kMaxCtas = 4;       // CTAs per SM at most (Geo::CTAS)
constexpr int kItem = 8;          // steps counted for an item besides its tiles
constexpr int kMinTail = 4;       // tiles that are worth cutting off
constexpr int kMinHead = kItem + kMinTail;
// A row's softmax reference is put kAhead (log2) above its largest score and moves when a score
// passes it by as much: weights are at most 2^4, so that their products with V's scales (below
// 2^121) stay in fp32's range.  The row's power of two puts its largest product into [2^9, 2^10)
// (kUpTo: 127 + 9) and moves when one comes to kUpLimit = 2^15; its exponent field is kUpMax at most.
constexpr float kAhead = 4.f, kUpLimit = 32768.f;
constexpr int kUpTo = 127 + 9, kUpMax = 253;
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

template <int D, int NR>
constexpr int part_floats() { return 8 * NR * (D + 2); }

// Steps of a sequence: tiles x row blocks x heads.
struct KvqCost {
  const int *cu, *lens;
  int T, cap, G, H_kv, rows_log2;  // rows of a block
  __device__ int blocks(int b) const {
    return (int)(((long long)seq_rows(cu, b, T).n * G + (1 << rows_log2) - 1) >> rows_log2);
  }
  __device__ int tiles(int b) const { return max(1, (seq_len(lens, b, cap) + kTile - 1) / kTile); }
  // An item costs its tiles and about kItem more: the first tiles' latency, laying out Q, merging the warps.
  __device__ int steps(int b) const { return tiles(b) + kItem; }
  __device__ long long cost(int b) const { return (long long)blocks(b) * H_kv * steps(b); }
  __device__ int item(int b, long long off, long long *s, long long *e) const {
    const int t = steps(b);
    *s = div_pos(off, t) * t;
    *e = *s + t;
    return 0;
  }
};

template <int FMT, int D, int NR>
struct Geo {
  static constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D;
  static constexpr int REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  static constexpr int CPR = ROW / 16;  // 16-byte chunks of a row
  static constexpr int CODE = kTile * ROW, SCALE = kTile * REC;
  static constexpr int STAGE = 2 * (CODE + SCALE);
  static constexpr int ROWS = 8 * NR;
  // CTAs of four warps, as many to an SM as shared memory and registers hold without spills (255 a
  // thread with two CTAs, 168 with three, 128 with four).  Blocks of 16 rows with one CTA more
  // spilled 8 to 224 bytes a thread: 16 sequences of 24 rows over 3000 to 9000 tokens, d = 128, took
  // 50 (e4m3), 55 (int8) and 53 us (int4) instead of 45, 49 and 48, in fp16 62, 62 and 59 instead of 50,
  // 55 and 54; d = 64 34, 36 and 37 instead of 32, 34 and 35 (64 sequences: up to 2 % the other way).
  static constexpr int WARPS = 4;
  static constexpr int CTAS = D == 128 && NR == 2 ? 2 : STAGE > 8192 || NR == 2 ? 3 : 4;
  static constexpr int QBYTES = (D / 16) * NR * 32 * 8;
  static constexpr int FIT = (233472 / CTAS - 2048 - QBYTES) / (WARPS * STAGE);
  static constexpr int STAGES = FIT < 4 ? FIT : 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int KS = D / 16;  // k steps of the first product
  static constexpr int MB = D / 16;  // blocks of 16 channels of the second
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int MERGE = WARPS * ROWS * (D + 2) * 4;
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
template <int OFF>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
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
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}
// The four nibbles of both 16-bit halves of a word as fp16 values (n - 8) f, exactly.
// A nibble in mantissa bits 4..7 of 1024 makes the fp16 number 1024 + 16 n, and
// (1024 + 16 n) (f / 16) - 72 f is one fused operation whose operands (f has 4
// significant bits) and result (7) are fp16 numbers; one in bits 0..3 makes 1024 + n, and
// (1024 + n) - 1032, then times f, are two.  Taking nibbles 0 and 2 the second way costs one
// shift a word instead of three: the integer pipe is the scarcer one here.
struct Factor {
  uint32_t one, sixteenth, minus72;  // pairs f, f / 16 and -72 f
  __device__ __forceinline__ explicit Factor(uint32_t f)
      : one(f), sixteenth(hmul2(f, 0x2c002c00u)), minus72(hmul2(f, 0xd480d480u)) {}
};
__device__ __forceinline__ uint32_t nibble_bits(uint32_t w, uint32_t mask) {
  uint32_t r;  // (w & mask) | 0x64006400 in one operation
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
  return r;
}
__device__ __forceinline__ void four_nibbles(uint32_t w, const Factor &f, uint32_t (&n)[4]) {
  const uint32_t u = w >> 8;
  n[0] = hmul2(hsub2(nibble_bits(w, 0x000f000fu), 0x64086408u), f.one);
  n[1] = hfma2(nibble_bits(w, 0x00f000f0u), f.sixteenth, f.minus72);
  n[2] = hmul2(hsub2(nibble_bits(u, 0x000f000fu), 0x64086408u), f.one);
  n[3] = hfma2(nibble_bits(u, 0x00f000f0u), f.sixteenth, f.minus72);
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
// Tiles that lie wholly below the length take copies with constant offsets from
// one address a half; the others fill what is missing with zeros.
template <int FMT, int D, int I>
__device__ __forceinline__ void copy_rows(uint32_t dst, int half, const unsigned char *ks, const unsigned char *vs,
                                          int ch, int r0) {
  using Ge = Geo<FMT, D, 1>;
  constexpr int RPI = 32 / Ge::CPR;  // rows of one pass of the warp
  if constexpr (I < 16 / RPI) {
    cp_async16_at<I * RPI * Ge::ROW>(dst + Ge::k_off(half * 16 + I * RPI + r0, ch), ks);
    cp_async16_at<I * RPI * Ge::ROW>(dst + Ge::CODE + Ge::v_off(half * 16 + I * RPI + r0, ch), vs);
    copy_rows<FMT, D, I + 1>(dst, half, ks, vs, ch, r0);
  }
}

// Where one head's tiles lie: addresses of page 0, this lane's bytes; a page's stride.
struct TileSource {
  const unsigned char *k, *v, *rec;
  uint32_t code_page, rec_page;
  int mask;
};

template <int FMT, int D>
__device__ __forceinline__ TileSource tile_source(const KvqView &c, int h) {
  using Ge = Geo<FMT, D, 1>;
  constexpr int SC = Ge::REC;  // 16-byte pieces of 16 scale records
  const int lane = threadIdx.x & 31;
  const long long row = (long long)h << c.page_log2;
  const uint32_t rows = (uint32_t)c.H_kv << c.page_log2;
  return {c.k_code + row * Ge::ROW + lane * 16, c.v_code + row * Ge::ROW + lane * 16,
          (lane < SC ? c.k_scale : c.v_scale) + row * Ge::REC + (lane % SC) * 16, rows * Ge::ROW, rows * Ge::REC,
          (1 << c.page_log2) - 1};
}

template <int FMT, int D>
__device__ __forceinline__ void load_tile(const TileSource &src, uint32_t dst, int tok0, int len, int pg0, int pg1) {
  using Ge = Geo<FMT, D, 1>;
  constexpr int RPI = 32 / Ge::CPR, SC = Ge::REC;
  const int lane = threadIdx.x & 31;
  const int ch = lane % Ge::CPR, r0 = lane / Ge::CPR;
  const uint32_t rec_dst = dst + 2 * Ge::CODE + (lane < SC ? 0 : Ge::SCALE) + (lane % SC) * 16;
  const bool full = tok0 + kTile <= len && (pg0 | pg1) >= 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int pg = half ? pg1 : pg0, t0 = tok0 + half * 16;
    const uint32_t page = pg < 0 ? 0u : (uint32_t)pg, place = t0 & src.mask;
    const unsigned long long at = (unsigned long long)page * src.code_page + place * Ge::ROW;
    const unsigned char *rec = src.rec + ((unsigned long long)page * src.rec_page + place * Ge::REC);
    if (full) {
      copy_rows<FMT, D, 0>(dst, half, src.k + at, src.v + at, ch, r0);
      if (lane < 2 * SC) cp_async16(rec_dst + half * 16 * Ge::REC, rec, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const int r = i * RPI + r0;
        const bool on = pg >= 0 && t0 + r < len;
        const unsigned long long off = on ? at + i * RPI * Ge::ROW : 0ull;
        cp_async16(dst + Ge::k_off(half * 16 + r, ch), src.k + off, on ? 16 : 0);
        cp_async16(dst + Ge::CODE + Ge::v_off(half * 16 + r, ch), src.v + off, on ? 16 : 0);
      }
      if (lane < 2 * SC) {
        const int tok = t0 + (lane % SC) * (16 / Ge::REC);
        const int bytes = pg >= 0 ? min(16, max(0, (len - tok) * Ge::REC)) : 0;
        cp_async16(rec_dst + half * 16 * Ge::REC, bytes ? rec : src.rec, bytes);
      }
    }
  }
}

// An 8 x 8 block of 16-bit values, one row of pairs per four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int FMT, int D, int NR, typename T, typename TO>
__global__ void __launch_bounds__(Geo<FMT, D, NR>::THREADS, Geo<FMT, D, NR>::CTAS) attn_kvq_kernel(KvqParams P) {
  using Ge = Geo<FMT, D, NR>;
  constexpr int kWarps = Ge::WARPS, kThreads = Ge::THREADS, kRows = Ge::ROWS;
  // fp16 outputs are as fine as fp16 weights: these then enter as a sum of two fp16 numbers
  constexpr bool kTwoParts = std::is_same<T, __half>::value;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ SplitRange range;
  __shared__ long long scratch[kWarps + 8];
  __shared__ float q_unscale[kRows];
  unsigned char *qh = smem + (Ge::RING > Ge::MERGE ? Ge::RING : Ge::MERGE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const KvqCost cost = {P.cu, P.lens, P.T, P.cap, P.G, P.c.H_kv, NR == 1 ? 3 : 4};
  asm volatile("griddepcontrol.launch_dependents;");  // the merge may take its place on the SMs; it waits for this grid
  if (threadIdx.x < 2) P.meta[2 * blockIdx.x + threadIdx.x].state = 0;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < P.B; b += kThreads)
      if (seq_rows_bad(P.cu, b, P.T) || __ldg(P.lens + b) != seq_len(P.lens, b, P.cap)) report_seq(P.err, b);
  split_range<kThreads>(cost, P.B, P.nc, blockIdx.x, kMinUnit, kMinHead, kMinTail, &range, scratch);

  long long left = range.x1 - range.x0;
  int b = range.b;
  long long off = range.off;
  unsigned char *ring = smem + warp * Ge::STAGES * Ge::STAGE;
  const uint32_t ring_u = smem_u32(ring);

  while (left > 0) {
    // ---- the next item of the stretch
    const SeqRows rows = seq_rows(P.cu, b, P.T);
    const int blocks = cost.blocks(b), tiles = cost.tiles(b), steps = tiles + kItem;
    if (off >= (long long)blocks * P.c.H_kv * steps) {
      ++b;
      off = 0;
      continue;
    }
    const int len = seq_len(P.lens, b, P.cap);
    // step x of an item is its tile x - kItem (a boundary lies at x = 0 or well behind kItem)
    const int item = (int)div_pos(off, steps), x_begin = (int)(off - (long long)item * steps);
    const int x_end = (int)min((long long)steps, x_begin + left);
    const int t_begin = max(0, x_begin - kItem), t_end = max(0, x_end - kItem);
    const int h = item / blocks, rb = item % blocks;
    const int n_rows = min(kRows, rows.n * P.G - rb * kRows);
    // ---- all loads of the start are issued together: Q's rows, the first tiles' pages, then the tiles,
    // which are on their way while Q is laid out
    constexpr int PER = D / 32, kMine = kRows / kWarps;  // values of a row per lane, rows of a warp
    uint32_t qw[kMine][PER / 2];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = warp + i * kWarps, rr = rb * kRows + r;
      const T *src = static_cast<const T *>(P.q) + (long long)(rows.begin + rr / P.G) * P.qs +
                     (long long)(h * P.G + rr % P.G) * D + lane * PER;
#pragma unroll
      for (int k = 0; k < PER / 2; ++k) qw[i][k] = r < n_rows ? __ldg(reinterpret_cast<const uint32_t *>(src) + k) : 0u;
    }
    const int my0 = t_begin + warp;
    int bad = 0;
    // pages of a tile's two halves, -1 where there is none (a tile below the length lies inside the table)
    const int *table = P.c.table + (long long)b * P.c.max_pages;
    const int page_log2 = P.c.page_log2;
    const unsigned n_pages = P.c.n_pages;
    auto pages = [&](int tile, int &p0, int &p1) {
      p0 = p1 = -1;
      const int tok = tile * kTile;
      if (tile < t_end && tok < len) {
        const int *at = table + (tok >> page_log2);
        p0 = __ldg(at);
        if ((unsigned)p0 >= n_pages) p0 = -1;
        bad |= p0;
        if (tok + 16 < len) {
          p1 = p0;
          if (page_log2 == 4) {
            p1 = __ldg(at + 1);
            if ((unsigned)p1 >= n_pages) p1 = -1;
            bad |= p1;
          }
        }
      }
    };
    const TileSource src = tile_source<FMT, D>(P.c, h);
    int fp[Ge::STAGES][2];
#pragma unroll
    for (int s = 0; s < Ge::STAGES; ++s) pages(my0 + s * kWarps, fp[s][0], fp[s][1]);
#pragma unroll
    for (int s = 0; s < Ge::STAGES - 1; ++s) {
      const int tile = my0 + s * kWarps;
      if (tile < t_end) load_tile<FMT, D>(src, ring_u + s * Ge::STAGE, tile * kTile, len, fp[s][0], fp[s][1]);
      cp_commit();
    }
    int np0 = fp[Ge::STAGES - 1][0], np1 = fp[Ge::STAGES - 1][1];

    // ---- Q: the rows as fp16, scaled by a power of two per row, in operand order
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int r = warp + j * kWarps;
      float x[PER];
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < PER / 2; ++i) {
        const float2 f = unpack16(qw[j][i], static_cast<const T *>(nullptr));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
        am = fmaxf(am, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      am = warp_max(am);
      // largest entry in [2^14, 2^15) (the exponent field; 2^126 at most); rows of zeros and
      // non-finite rows stay as they are
      const int e = am > 0.f && am < INFINITY ? min(14 + 127 - (int)(__float_as_uint(am) >> 23), 126) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        int ks, t, half, el;
        Ge::q_pos(lane * PER + i, ks, t, half, el);
        reinterpret_cast<__half *>(qh)[(((ks * NR + (r >> 3)) * 32 + (r & 7) * 4 + t) * 2 + half) * 2 + el] =
            __float2half_rn(x[i] * up);
      }
      // (never 0, which would make NaN of a masked score: the scores that it scales are below 2^128, so that
      // 2^-149 leaves them as good as 0 too)
      if (lane == 0) q_unscale[r] = fmaxf(P.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 0x1p-149f);
    }
    __syncthreads();
    uint2 qb[Ge::KS][NR];
#pragma unroll
    for (int ks = 0; ks < Ge::KS; ++ks)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) qb[ks][nr] = reinterpret_cast<const uint2 *>(qh)[(ks * NR + nr) * 32 + lane];
    // this lane's rows: 8 nr + 2 t4 + e; the keys that each may see
    const int past = len - rows.n + 1;
    float un[NR][2], m[NR][2], l[NR][2], up[NR][2];
    int lim[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nr * 8 + 2 * t4 + e;
        un[nr][e] = q_unscale[r];
        lim[nr][e] = P.causal ? min(len, past + (rb * kRows + r) / P.G) : len;
        m[nr][e] = kNegInf;
        l[nr][e] = 0.f;
        up[nr][e] = __uint_as_float((uint32_t)kUpMax << 23);
      }
    const int lim_all = P.causal ? min(len, past + (rb * kRows) / P.G) : len;  // the first row sees the fewest

    float acc[Ge::MB][NR][4];
#pragma unroll
    for (int j = 0; j < Ge::MB; ++j)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][nr][i] = 0.f;

    int stage = 0;
    for (int tile = my0; tile < t_end; tile += kWarps) {
      cp_wait<Ge::STAGES - 2>();
      __syncwarp();
      {  // refill the stage read in the last round
        const int nt = tile + (Ge::STAGES - 1) * kWarps;
        const int ns = stage == 0 ? Ge::STAGES - 1 : stage - 1;
        if (nt < t_end) load_tile<FMT, D>(src, ring_u + ns * Ge::STAGE, nt * kTile, len, np0, np1);
        cp_commit();
        pages(nt + kWarps, np0, np1);
      }
      const unsigned char *kc = ring + stage * Ge::STAGE, *vc = kc + Ge::CODE, *kr = vc + Ge::CODE,
                          *vr = kr + Ge::SCALE;
      stage = stage + 1 == Ge::STAGES ? 0 : stage + 1;

      // ---- scores of 2 x 16 tokens (lane: tokens g and g + 8 of each) for its rows, times K's scale
      float s[2][NR][4];
      float vs[2][2];  // V's scales of the same tokens
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[tb][nr][i] = 0.f;
        const int row0 = tb * 16 + g, row1 = row0 + 8;
        float ks0, ks1;
        if (FMT == ISPA_KVQ_INT4) {
          constexpr int WORDS = D / 32;  // words of this lane's D / 4 channels
          uint32_t w[2][WORDS];
          const uint2 rec0 = *reinterpret_cast<const uint2 *>(kr + row0 * 8);
          const uint2 rec1 = *reinterpret_cast<const uint2 *>(kr + row1 * 8);
          ks0 = __uint_as_float(rec0.x);
          ks1 = __uint_as_float(rec1.x);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4 *>(kc + Ge::k_off(n ? row1 : row0, t4));
              w[n][0] = v.x, w[n][1] = v.y, w[n][WORDS - 2] = v.z, w[n][WORDS - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(kc + (n ? row1 : row0) * Ge::ROW + t4 * 8);
              w[n][0] = v.x, w[n][1] = v.y;
            }
          }
          const uint32_t pick = (uint32_t)(t4 * (D / 4) / 32) * 0x11u;  // the factor's byte, twice
          const Factor f0(e4m3x2_to_half2(prmt(rec0.y, 0u, pick))), f1(e4m3x2_to_half2(prmt(rec1.y, 0u, pick)));
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            uint32_t n0[4], n1[4];
            four_nibbles(w[0][i], f0, n0);
            four_nibbles(w[1][i], f1, n1);
            const uint4 a0 = make_uint4(n0[0], n1[0], n0[1], n1[1]), a1 = make_uint4(n0[2], n1[2], n0[3], n1[3]);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              mma16816(s[tb][nr], a0, qb[2 * i][nr].x, qb[2 * i][nr].y);
              mma16816(s[tb][nr], a1, qb[2 * i + 1][nr].x, qb[2 * i + 1][nr].y);
            }
          }
        } else {
          ks0 = *reinterpret_cast<const float *>(kr + row0 * 4);
          ks1 = *reinterpret_cast<const float *>(kr + row1 * 4);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 u = *reinterpret_cast<const uint4 *>(kc + Ge::k_off(row0, t4 + 4 * c));
            const uint4 v = *reinterpret_cast<const uint4 *>(kc + Ge::k_off(row1, t4 + 4 * c));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 a;
              four_codes<FMT>(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w, a.x, a.z);
              four_codes<FMT>(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w, a.y, a.w);
#pragma unroll
              for (int nr = 0; nr < NR; ++nr) mma16816(s[tb][nr], a, qb[4 * c + i][nr].x, qb[4 * c + i][nr].y);
            }
          }
        }
        vs[tb][0] = *reinterpret_cast<const float *>(vr + row0 * Ge::REC);
        vs[tb][1] = *reinterpret_cast<const float *>(vr + row1 * Ge::REC);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          s[tb][nr][0] *= ks0;
          s[tb][nr][1] *= ks0;
          s[tb][nr][2] *= ks1;
          s[tb][nr][3] *= ks1;
        }
      }
      if (tile * kTile + kTile > lim_all) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
          const int tok = tile * kTile + tb * 16 + g;
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tok + (i >> 1) * 8 >= lim[nr][i & 1]) s[tb][nr][i] = kNegInf;
        }
      }
      if (bad < 0) {  // tokens whose page does not exist are left out
        int p0, p1;
        const int keep = bad;
        pages(tile, p0, p1);
        bad = keep;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
          if ((tb ? p1 : p0) < 0) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) s[tb][nr][0] = s[tb][nr][1] = s[tb][nr][2] = s[tb][nr][3] = kNegInf;
          }
      }

      // ---- the running maximum moves only when some lane's tokens pass it
      float mx[NR][2];
      bool move = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nr][e] = fmaxf(fmaxf(s[0][nr][e], s[0][nr][2 + e]), fmaxf(s[1][nr][e], s[1][nr][2 + e])) * un[nr][e];
          move |= mx[nr][e] > m[nr][e] + kAhead;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[nr][e] = fmaxf(mx[nr][e], __shfl_xor_sync(0xffffffffu, mx[nr][e], o));
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float to = fmaxf(m[nr][e], mx[nr][e] + kAhead);
            const float f = m[nr][e] == kNegInf ? 0.f : exp2_fast(m[nr][e] - to);
            m[nr][e] = to;
            l[nr][e] *= f;
            // the earlier products shrink by f: the power of two grows by as much, so that small V scales
            // among the keys that now matter keep their bits
            const int was = (int)(__float_as_uint(up[nr][e]) >> 23);
            const int now = min(was + 127 - (int)(__float_as_uint(f) >> 23), kUpMax);
            up[nr][e] = __uint_as_float((uint32_t)now << 23);
            const float g = f * __uint_as_float((uint32_t)(127 + now - was) << 23);
#pragma unroll
            for (int j = 0; j < Ge::MB; ++j) {
              acc[j][nr][e] *= g;
              acc[j][nr][2 + e] *= g;
            }
          }
      }

      // ---- weights: exp2, times V's scale
      bool over = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[nr][e] == kNegInf ? 0.f : m[nr][e];
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float &w = s[k >> 1][nr][2 * (k & 1) + e];
            const float p = exp2_fast(fmaf(w, un[nr][e], -ref));
            l[nr][e] += p;
            w = p * vs[k >> 1][k & 1];
            top = fmaxf(top, w);
          }
          mx[nr][e] = top;
          over |= top * up[nr][e] >= kUpLimit;
        }
      if (__any_sync(0xffffffffu, over)) {  // the first tile, and where a row's products grow 32-fold
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[nr][e] = fmaxf(mx[nr][e], __shfl_xor_sync(0xffffffffu, mx[nr][e], o));
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (mx[nr][e] * up[nr][e] >= kUpLimit) {
              const int was = (int)(__float_as_uint(up[nr][e]) >> 23);
              const int now = min(127 + kUpTo - (int)(__float_as_uint(mx[nr][e]) >> 23), kUpMax);
              up[nr][e] = __uint_as_float((uint32_t)now << 23);
              const float g = __uint_as_float((uint32_t)max(127 + now - was, 0) << 23);
#pragma unroll
              for (int j = 0; j < Ge::MB; ++j) {
                acc[j][nr][e] *= g;
                acc[j][nr][2 + e] *= g;
              }
            }
      }

      // ---- to fp16, transposed
      uint2 pb[2][NR], pl[2][NR];
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = s[tb][nr][i] * up[nr][i & 1];
          const uint32_t h0 = pack_half2(w[0], w[1]), h1 = pack_half2(w[2], w[3]);
          pb[tb][nr] = make_uint2(transpose8(h0), transpose8(h1));
          if (kTwoParts) {
            const float2 f0 = unpack16(h0, static_cast<const __half *>(nullptr));
            const float2 f1 = unpack16(h1, static_cast<const __half *>(nullptr));
            pl[tb][nr] = make_uint2(transpose8(pack_half2(w[0] - f0.x, w[1] - f0.y)),
                                    transpose8(pack_half2(w[2] - f1.x, w[3] - f1.y)));
          }
        }
      }
      auto product = [&](int j, int kb, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          mma16816(acc[j][nr], make_uint4(a0, a1, a2, a3), pb[kb][nr].x, pb[kb][nr].y);
          if (kTwoParts) mma16816(acc[j][nr], make_uint4(a0, a1, a2, a3), pl[kb][nr].x, pl[kb][nr].y);
        }
      };

      // ---- O^T += V^T P^T
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
              uint32_t na[4], nb[4];
              four_nibbles(xa, fa, na);
              four_nibbles(xb, fb, nb);
              product(i * 4 + hw * 2, kb, na[0], na[1], nb[0], nb[1]);
              product(i * 4 + hw * 2 + 1, kb, na[2], na[3], nb[2], nb[3]);
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
            product(2 * i, kb, a0, a1, b0, b1);
            product(2 * i + 1, kb, a2, a3, b2, b3);
          }
        }
      }
    }
    if (bad < 0 && lane == 0) report_seq(P.err, b);

    // ---- merge the warps' states (the rings are idle now)
    cp_wait<0>();
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], o);
    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);  // [warp][m | l | O rows x D]
    {
      float *mine = mg + warp * kRows * (D + 2);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nr * 8 + 2 * t4 + e;
          const float down = __uint_as_float((254u << 23) - __float_as_uint(up[nr][e]));  // 1 / up, exactly
          if (g == 0) {
            mine[r] = m[nr][e];
            mine[kRows + r] = l[nr][e];
          }
          float4 *oo = reinterpret_cast<float4 *>(mine + 2 * kRows + r * D + g * (D / 8));
#pragma unroll
          for (int j = 0; j < Ge::MB; j += 2)
            oo[j / 2] = make_float4(acc[j][nr][e] * down, acc[j][nr][2 + e] * down, acc[j + 1][nr][e] * down,
                                    acc[j + 1][nr][2 + e] * down);
        }
    }
    __syncthreads();
    const bool whole = t_begin == 0 && t_end == tiles;
    const int slot = 2 * blockIdx.x + (t_begin == 0 ? 1 : 0);
    float *part = P.part + (size_t)slot * part_floats<D, NR>();
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
        const float inv = ll == 0.f ? 0.f : 1.f / ll;  // (a sum that is NaN stays so)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv;
        store8(static_cast<TO *>(P.o) + out * D + c8, x);
        if (P.lse && c8 == 0) P.lse[out] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718055994530942f;
      } else {
        if (c8 == 0) {
          part[r] = mm;
          part[kRows + r] = ll;
        }
        store8(part + 2 * kRows + r * D + c8, x);
      }
    }
    if (!whole && threadIdx.x == 0) {
      PartMeta m = {t_end == tiles ? 2 : 1, rows.begin, rb * kRows, n_rows, h, {}};
      P.meta[slot] = m;
    }
    __syncthreads();  // the merge area is the next item's ring
    left -= x_end - x_begin;
    off += x_end - x_begin;
  }
}

// Who joins which columns of a cut item.  CTA c takes the item that its slot 2c + 1 starts; when
// that has many parts, the CTAs c + 1 .. c + shares - 1, whose slots the item runs through, take
// equal shares of its values: two from 16 parts on, four from 32 (shares <= parts / 8, so that a
// helper never is the item's last CTA).  4 sequences of 30000 tokens of one head, 150 parts each: 34
// -> 24 us, 16 with pending tokens: 23.2 -> 22.1 (512 threads a CTA instead: 27 and 23.4; sharing from
// 8 parts on: 0.5 us more for one sequence of 999 tokens; up to eight CTAs: no gain).
constexpr int kMaxShares = 4, kShareParts = 16;
struct MergeRole {
  int head, share, shares, n;  // n: the item's parts, 0: nothing to do
};
__device__ __forceinline__ MergeRole merge_role(const PartMeta *meta, int nc, int c) {  // by a whole warp
  const int lane = threadIdx.x & 31, at = c - lane;
  const bool see = lane < kMaxShares && at >= 0;
  const int through = see ? *const_cast<const volatile int *>(&meta[2 * at].state) : 0;
  const int starts = see ? *const_cast<const volatile int *>(&meta[2 * at + 1].state) : 0;
  const unsigned heads = __ballot_sync(0xffffffffu, starts != 0), runs = __ballot_sync(0xffffffffu, through == 1);
  MergeRole m = {0, 0, 1, 0};
  if (heads == 0) return m;
  m.share = __ffs(heads) - 1;
  const unsigned below = (1u << m.share) - 1;
  if ((runs & below) != below) return m;  // (the item ended before c)
  m.head = c - m.share;
  const int n = parts_from(meta, nc, m.head);
  while (m.shares < kMaxShares && n >= kShareParts * m.shares) m.shares *= 2;
  m.n = m.share < m.shares ? n : 0;
  return m;
}

// Joins the parts of the cut items.
// (A launch of its own, made ahead and waiting on the device: joining in the attention's kernel, by
// the last of an item's CTAs to arrive at a counter, took 12.6 us instead of 10.2 for one sequence
// of 999 tokens and 27 instead of 23.2 for 16 sequences with pending tokens.)
template <int D, int NR, typename TO>
__global__ void __launch_bounds__(256) kvq_merge_kernel(KvqParams P) {
  constexpr int kRows = 8 * NR;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ MergeRole role;
  if (threadIdx.x < 32) {
    const MergeRole m = merge_role(P.meta, P.nc, blockIdx.x);
    if (threadIdx.x == 0) role = m;
  }
  __syncthreads();
  const int n = role.n, c = role.head;
  if (n == 0) return;
  const PartMeta own = P.meta[2 * c + 1];
  const int h = own.head, n_rows = own.count;
  // a thread takes a row's eight columns; with fewer rows, several threads take every split-th
  // part of the same columns and are added up in shared memory
  __shared__ float red[256][11];
  const int all = n_rows * (D / 8);
  const int first = all * role.share / role.shares, items = all * (role.share + 1) / role.shares;
  int split = 1;
  while (split * 2 * (items - first) <= 256 && split < n) split *= 2;
  for (int i0 = first; i0 < items; i0 += 256 / split) {
    const int i = i0 + threadIdx.x / split, sub = threadIdx.x % split;
    const int r = i / (D / 8), c8 = i % (D / 8) * 8;
    float mm = kNegInf, ll = 0.f, x[8] = {};
    if (i < items) {
#pragma unroll 4
      for (int k = sub; k < n; k += split) {  // (one pass: the loads of several parts are in flight together)
        const float *st = P.part + (size_t)part_slot(c, k) * part_floats<D, NR>();
        const float mk = st[r], lk = st[kRows + r];
        const float4 a = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8);
        const float4 d = *reinterpret_cast<const float4 *>(st + 2 * kRows + r * D + c8 + 4);
        const float to = fmaxf(mm, mk), ref = to == kNegInf ? 0.f : to;
        const float f0 = exp2_fast(mm - ref), f = exp2_fast(mk - ref);
        mm = to;
        ll = ll * f0 + lk * f;
        x[0] = x[0] * f0 + a.x * f, x[1] = x[1] * f0 + a.y * f, x[2] = x[2] * f0 + a.z * f, x[3] = x[3] * f0 + a.w * f;
        x[4] = x[4] * f0 + d.x * f, x[5] = x[5] * f0 + d.y * f, x[6] = x[6] * f0 + d.z * f, x[7] = x[7] * f0 + d.w * f;
      }
    }
    if (split > 1) {
#pragma unroll
      for (int k = 0; k < 8; ++k) red[threadIdx.x][k] = x[k];
      red[threadIdx.x][8] = ll;
      red[threadIdx.x][9] = mm;
      __syncthreads();
      if (sub == 0)
        for (int o = 1; o < split; ++o) {
          const float *other = red[threadIdx.x + o];
          const float to = fmaxf(mm, other[9]), ref = to == kNegInf ? 0.f : to;
          const float f0 = exp2_fast(mm - ref), f = exp2_fast(other[9] - ref);
          mm = to;
          ll = ll * f0 + other[8] * f;
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] * f0 + other[k] * f;
        }
      __syncthreads();
    }
    if (i >= items || sub != 0) continue;
    const int rr = own.first + r;
    const long long out = (long long)(own.row + rr / P.G) * P.H + h * P.G + rr % P.G;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;  // (a sum that is NaN stays so)
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] *= inv;
    store8(static_cast<TO *>(P.o) + out * D + c8, x);
    if (P.lse && c8 == 0) P.lse[out] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718055994530942f;
  }
}

template <int FMT, int D, int NR, typename T, typename TO>
ispa_status launch_rows(KvqParams P, cudaStream_t s) {
  using Ge = Geo<FMT, D, NR>;
  static_assert(Ge::STAGES >= 2 && Ge::CTAS <= kMaxCtas, "ring");
  P.nc *= Ge::CTAS;
  auto kern = attn_kvq_kernel<FMT, D, NR, T, TO>;
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
  e = cudaLaunchKernelEx(&cfg, kvq_merge_kernel<D, NR, TO>, P);
  note_launch();
  return cuda_status(e, "kvq_merge launch");
}

// Row blocks of 8 when a sequence's rows fit one, else of 16, which read and unpack the cache half
// as often.  The number of rows is an average over the call, rows of padding counted (the arrays
// are on the device), so the line lies at 11: 8 rows and up to three of padding for eight sequences.
// 16 sequences of 3000 to 9000 tokens, 4 K/V heads, us with blocks of 8 / of 16:
//   rows a sequence      4            8            9            16           32
//   e4m3, d = 128    27.0 / 30.0  28.0 / 31.9  34.0 / 32.9  35.0 / 32.9  53.2 / 45.7
//   int8, d = 128    28.0 / 32.3  29.4 / 34.3  39.1 / 34.6  39.6 / 34.6  63.1 / 49.3
//   int4, d = 128    29.0 / 31.7  29.4 / 33.3  39.6 / 33.8  40.1 / 33.3  62.6 / 49.2
//   e4m3, d = 64     22.0 / 24.6  23.2 / 24.6  27.1 / 25.7  27.1 / 25.1  40.3 / 33.1
// (With the line at 8, one row of padding took a batch of 8 rows a sequence to the right side.)
template <int FMT, int D, typename T, typename TO>
ispa_status launch_one(const KvqParams &P, cudaStream_t s) {
  return (long long)P.G * P.T <= 11LL * P.B ? launch_rows<FMT, D, 1, T, TO>(P, s) : launch_rows<FMT, D, 2, T, TO>(P, s);
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
  const size_t nc = (size_t)sm_count() * kMaxCtas;
  return 2 * nc * (sizeof(PartMeta) + (size_t)kMaxRows * (head_dim + 2) * 4);
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
  P.part = reinterpret_cast<float *>(P.meta + 2 * P.nc * kMaxCtas);
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

// kvq.cu -- writing rows into the quantised paged cache and reading them back.
//
// Both are one pass over their bytes and bound by memory (and, for a decoding
// step's few rows, by the launch).  A row (one token of one head) is handled
// by d / 8 lanes, 16 bytes of 16-bit values each; a warp takes one token and
// up to kHeads heads of K and of V, whose loads are all issued before the
// first is used.
//
// The codes are decided by quotients with exact operands: 127 x, 448 x and
// 3136 x / 4096 fit fp32 for 16-bit x, as does amax * g, and the powers of two
// that keep the quotient in range are exact too.  The quotient of two such
// numbers is either on a border between two codes or further from it than
// half an fp32 step (numerator and denominator have at most 18 and 15
// significant bits, the border 8), so one correctly rounded division gives the
// code of real arithmetic, ties included.
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

// Eight values of a row of W lanes: codes (8 or 4 bytes) and the row's scale record.
template <int FMT, int W>
__device__ __forceinline__ void quantise8(const float (&x)[8], uint2 &code, uint2 &rec) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[i]));
  float group = am;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    if (o == 4) group = am;  // the four lanes of 32 channels
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  }
  const bool some = am >= kLeast;
  const float div = some ? am : 1.f;
  if (FMT == ISPA_KVQ_INT4) {
    const uint32_t g8 = some ? e4m3x2(group * 0.875f / div * 512.f, 0.f) & 0xffu : 0u;
    const float step = div * (e4m3x2_to_float(g8).x * (1.f / 512.f));
    const bool on = g8 != 0;
    const float over = on ? step : 1.f;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = fminf(fmaxf(rintf(x[i] * (49.f / 64.f) / over * 8.f), -7.f), 7.f);
      c |= (uint32_t)((on ? (int)n : 0) + 8) << (4 * i);
    }
    code = make_uint2(c, 0u);
    // the factors of the row's groups, gathered from the first lane of each
    uint32_t factors = 0;
#pragma unroll
    for (int g = 0; g < W / 4; ++g) factors |= __shfl_sync(0xffffffffu, g8, g * 4, W) << (8 * g);
    rec = make_uint2(__float_as_uint(some ? am / 3136.f : 0.f), factors);
  } else if (FMT == ISPA_KVQ_INT8) {
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = fminf(fmaxf(rintf(x[i] * (127.f / 128.f) / div * 128.f), -127.f), 127.f);
      c[i >> 2] |= ((uint32_t)(some ? (int)n : 0) & 0xffu) << (8 * (i & 3));
    }
    code = make_uint2(c[0], c[1]);
    rec = make_uint2(__float_as_uint(some ? am / 127.f : 0.f), 0u);
  } else {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = some ? x[i] * 0.875f / div * 512.f : 0.f;
    code = make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16, e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
    rec = make_uint2(__float_as_uint(some ? am / 448.f : 0.f), 0u);
  }
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kvq_write_kernel(RowParams P) {
  constexpr int W = D / 8;                        // lanes of a row
  constexpr int kRows = 32 / W;                   // rows of a pass: K and V, and two heads each for d = 64
  constexpr int kHeads = 4, kStep = kRows / 2;    // heads of a warp, heads of a pass
  constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D, REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const int h_parts = (P.H_kv + kHeads - 1) / kHeads;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(item / h_parts), h0 = (int)(item % h_parts) * kHeads;
  if (t >= P.T) return;
  const int b = seq_of_row(P.cu, P.B, t);
  if (b < 0) return;
  const int sub = lane / W, l = lane % W;
  const bool is_v = sub >= kStep;
  const T *src = static_cast<const T *>(is_v ? P.v : P.k) + (long long)t * (is_v ? P.vs : P.ks) + l * 8;
  uint4 in[kHeads / kStep];
#pragma unroll
  for (int i = 0; i < kHeads / kStep; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    in[i] = h < P.H_kv ? __ldg(reinterpret_cast<const uint4 *>(src + (long long)h * D)) : make_uint4(0, 0, 0, 0);
  }
  const int c0 = __ldg(P.cu + b), c1 = __ldg(P.cu + b + 1);
  const long long pos = (long long)__ldg(P.lens + b) - (c1 - c0) + (t - c0);
  const int page = P.c.page(b, pos);
  if (page < 0 || seq_rows_bad(P.cu, b, P.T)) {
    if (lane == 0) report_seq(P.err, b);
    if (page < 0) return;
  }
  const int place = (int)(pos & ((1 << P.c.page_log2) - 1));
  unsigned char *codes = is_v ? P.c.v_code : P.c.k_code, *scales = is_v ? P.c.v_scale : P.c.k_scale;
#pragma unroll
  for (int i = 0; i < kHeads / kStep; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(w[j], static_cast<const T *>(nullptr));
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
    uint2 code, rec;
    quantise8<FMT, W>(x, code, rec);
    if (h >= P.H_kv) continue;
    const long long row = P.c.row(page, h, place);
    if (FMT == ISPA_KVQ_INT4) {
      *reinterpret_cast<uint32_t *>(codes + row * ROW + l * 4) = code.x;
      if (l == 0) *reinterpret_cast<uint2 *>(scales + row * REC) = rec;
    } else {
      *reinterpret_cast<uint2 *>(codes + row * ROW + l * 8) = code;
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

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kvq_read_kernel(RowParams P) {
  constexpr int W = D / 8;
  constexpr int kRows = 32 / W;
  constexpr int kHeads = 4, kStep = kRows / 2;
  constexpr int ROW = FMT == ISPA_KVQ_INT4 ? D / 2 : D, REC = FMT == ISPA_KVQ_INT4 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const int h_parts = (P.H_kv + kHeads - 1) / kHeads;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(item / h_parts), h0 = (int)(item % h_parts) * kHeads;
  if (t >= P.T) return;
  const int b = seq_of_row(P.cu, P.B, t);
  if (b < 0) return;
  const long long pos = (long long)(P.begin ? __ldg(P.begin + b) : 0) + (t - __ldg(P.cu + b));
  const int page = P.c.page(b, pos);
  if ((page < 0 || seq_rows_bad(P.cu, b, P.T)) && lane == 0) report_seq(P.err, b);
  const int place = (int)(pos & ((1 << P.c.page_log2) - 1));
  const int sub = lane / W, l = lane % W;
  const bool is_v = sub >= kStep;
  const unsigned char *codes = is_v ? P.c.v_code : P.c.k_code, *scales = is_v ? P.c.v_scale : P.c.k_scale;
  uint2 code[kHeads / kStep], rec[kHeads / kStep];
#pragma unroll
  for (int i = 0; i < kHeads / kStep; ++i) {
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
  for (int i = 0; i < kHeads / kStep; ++i) {
    const int h = h0 + i * kStep + sub % kStep;
    if (h >= P.H_kv) continue;
    const float s = __uint_as_float(rec[i].x);
    float x[8];
    if (FMT == ISPA_KVQ_INT4) {
      const float sg = s * e4m3x2_to_float((rec[i].y >> (8 * (l >> 2))) & 0xffu).x;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (float)((int)((code[i].x >> (4 * j)) & 15u) - 8) * sg;
      if (page < 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
      }
    } else if (FMT == ISPA_KVQ_INT8) {
      const uint32_t w[2] = {code[i].x, code[i].y};
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (float)(int)(signed char)((w[j >> 2] >> (8 * (j & 3))) & 0xffu) * s;
    } else {
      const uint32_t w[2] = {code[i].x, code[i].y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_to_float((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
        x[2 * j] = f.x * s;
        x[2 * j + 1] = f.y * s;
      }
    }
    *reinterpret_cast<uint4 *>(dst + (long long)h * D) =
        make_uint4(pack16<T>(x[0], x[1]), pack16<T>(x[2], x[3]), pack16<T>(x[4], x[5]), pack16<T>(x[6], x[7]));
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
  const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
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

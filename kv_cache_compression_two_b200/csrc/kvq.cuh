// kvq.cuh -- the bytes of the quantised paged cache (see ispa_kvq_desc).
#pragma once

#include "internal.h"

namespace ispa {

struct KvqLayout {
  size_t rows;               // n_pages * H_kv * page_tokens
  size_t k_code, v_code, k_scale, v_scale, bytes;
  int row, rec;              // bytes of a row's codes and of its scale record
  int page_log2;
};

inline int kvq_log2(int page_tokens) {
  for (int l = 4; l <= 8; ++l)
    if (page_tokens == 1 << l) return l;
  return -1;
}

inline KvqLayout kvq_layout(const ispa_kvq_desc &d) {
  KvqLayout L;
  const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  L.rows = (size_t)d.n_pages * d.H_kv * d.page_tokens;
  L.row = d.fmt == ISPA_KVQ_INT4 ? d.head_dim / 2 : d.head_dim;
  L.rec = d.fmt == ISPA_KVQ_INT4 ? 8 : 4;
  L.k_code = 0;
  L.v_code = up(L.rows * L.row);
  L.k_scale = L.v_code + up(L.rows * L.row);
  L.v_scale = L.k_scale + up(L.rows * L.rec);
  L.bytes = L.v_scale + up(L.rows * L.rec);
  L.page_log2 = kvq_log2(d.page_tokens);
  return L;
}

// Device view of one cache with the block table that addresses it.
struct KvqView {
  unsigned char *k_code, *v_code, *k_scale, *v_scale;
  const int *table;
  int max_pages, n_pages, H_kv, page_log2;

  // Page of position pos of sequence b, or -1 when the table has none.
  __device__ __forceinline__ int page(int b, long long pos) const {
    const long long i = pos >> page_log2;
    if (pos < 0 || i >= max_pages) return -1;
    const int p = __ldg(table + (long long)b * max_pages + i);
    return (unsigned)p < (unsigned)n_pages ? p : -1;
  }
  // Row number of (page, head, place in the page).
  __device__ __forceinline__ long long row(int p, int h, int place) const {
    return ((((long long)p * H_kv + h) << page_log2) + place);
  }
};

inline KvqView kvq_view(const ispa_kvq_desc &d, const void *kvq, const int *table, int max_pages) {
  const KvqLayout L = kvq_layout(d);
  unsigned char *p = static_cast<unsigned char *>(const_cast<void *>(kvq));
  return {p + L.k_code, p + L.v_code, p + L.k_scale, p + L.v_scale, table, max_pages, d.n_pages, d.H_kv, L.page_log2};
}

}  // namespace ispa

// The attention layers' paged cache as the kernels see it, and its host-side
// check (contract: include/gdn.h).
#pragma once

#include "gdn_internal.cuh"
#include "hostcheck.cuh"

namespace gdn {
namespace kv {

using namespace hostcheck;

inline bool page_ok(int32_t page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }
inline int32_t log2_of(int32_t page) {
  int32_t n = 0;
  while ((1 << n) < page) ++n;
  return n;
}
inline bool dim_ok(int32_t d) { return d == 64 || d == 128; }

inline size_t pool_bytes(const gdn_kv_cache& c) {
  return (size_t)c.layers * c.pages * c.kv_heads * c.page * c.d * (c.dtype == GDN_BF16 ? 2 : 1);
}
inline size_t scale_bytes(const gdn_kv_cache& c) {
  return c.dtype == GDN_BF16 ? 0 : (size_t)c.layers * c.pages * c.kv_heads * c.page * 4;
}

// GDN_OK, or what is wrong with a cache's description.
inline int check_cache(const gdn_kv_cache* c) {
  if (!c) return GDN_ERR_INVALID_ARG;
  if (c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->rows < 1 || c->max_pages < 1)
    return GDN_ERR_INVALID_ARG;
  if (c->dtype != GDN_BF16 && c->dtype != GDN_E4M3) return GDN_ERR_UNSUPPORTED;
  if (!page_ok(c->page) || !dim_ok(c->d)) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->table || !c->lengths || !c->refs) return GDN_ERR_INVALID_ARG;
  const bool scales = c->k_scale && c->v_scale;
  if (c->dtype == GDN_E4M3 ? !scales : (c->k_scale || c->v_scale)) return GDN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16) || !aligned(c->refs, 16) || !aligned(c->table, 4) ||
      !aligned(c->lengths, 4))
    return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

// What a cache occupies; nothing of it may overlap.
struct Spans {
  Span s[7];
};
inline Spans spans_of(const gdn_kv_cache& c) {
  return {{span_of(c.k, pool_bytes(c)), span_of(c.v, pool_bytes(c)),
           span_of(c.k_scale, scale_bytes(c)), span_of(c.v_scale, scale_bytes(c)),
           span_of(c.table, (size_t)c.rows * c.max_pages * 4), span_of(c.lengths, (size_t)c.rows * 4),
           span_of(c.refs, (size_t)c.pages * 4)}};
}

}  // namespace kv
}  // namespace gdn

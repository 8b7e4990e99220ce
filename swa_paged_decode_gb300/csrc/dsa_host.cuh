// dsa_host.cuh -- host-side helpers shared by the entry points: argument
// checks, record sizes, the cache descriptor's rules and the NVTX range.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <cstdlib>

#include "dsa_internal.cuh"

namespace dsa {

// NVTX range over one entry point (host side: argument checks and launches),
// so a profiler timeline shows each call.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
inline int record_bytes(int32_t fmt) {
  if (fmt == DSA_REC_FP8_528 || fmt == DSA_REC_FP8_528_UE8M0) return 528;
  if (fmt == DSA_REC_MODEL1_584) return 584;
  if (fmt == DSA_REC_V32_656) return 656;
  return fmt == DSA_REC_NVFP4_288 ? 288 : -1;
}
inline dsa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

// The cache descriptor's own rules, and the list's cache fields from it.
inline dsa_status fill_cache(const dsa_cache_desc *c, ListArgs &L) {
  if (!c || !c->base) return DSA_ERR_INVALID_ARG;
  const int rb = record_bytes(c->format);
  if (rb < 0) return DSA_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || !pow2(c->page_size)) return DSA_ERR_INVALID_ARG;
  if (c->page_stride_bytes < (int64_t)c->page_size * rb) return DSA_ERR_INVALID_ARG;
  if (c->num_pages > ((int64_t)INT32_MAX + 1) / c->page_size) return DSA_ERR_UNSUPPORTED;
  if (!aligned(c->base, 16) || c->page_stride_bytes % 16 != 0) return DSA_ERR_ALIGNMENT;
  L.base = static_cast<const uint8_t *>(c->base);
  L.num_slots = c->num_pages * (int64_t)c->page_size;
  L.page_stride = c->page_stride_bytes;
  int sh = 0;
  while ((1 << sh) < c->page_size) ++sh;
  L.page_shift = sh;
  L.page_mask = c->page_size - 1;
  L.fmt = c->format;
  L.rec = rb;
  L.extent = c->num_pages * c->page_stride_bytes;
#ifdef DSA_DEBUG
  // Checking build only: a smaller extent for the record checks (a test
  // knob: records past it are reported and skipped, never read).
  if (const char *cap = std::getenv("DSA_DEBUG_CHECK_EXTENT")) {
    const long long v = std::atoll(cap);
    if (v > 0 && v < L.extent) L.extent = v;
  }
#endif
  L.aligned32 = (aligned(c->base, 32) && c->page_stride_bytes % 32 == 0 && rb % 32 == 0) ? 1 : 0;
  L.sectors32 = (aligned(c->base, 32) && c->page_stride_bytes % 32 == 0) ? 1 : 0;
  return DSA_OK;
}

}  // namespace dsa

// dsa_cache.cu -- the cache side of the decode: rows of keys quantized into
// the paged records as they are written (dsa_cache_write), and records read
// back as dense rows (dsa_cache_read).
//
// Both are one pass over memory: a row of 512 or 576 values in 16 or 32 bits
// against a record of 288 to 656 bytes. A warp takes a row, a lane 16
// consecutive dims of it (and 2 of the 64 key dims that a V3.2 row has more),
// so that every block of every format (16, 32, 64 or 128 dims sharing a
// scale) lies in 1, 2, 4 or 8 neighbouring lanes and its largest magnitude is
// found with at most three shuffles; the row is held in registers from the
// load to the store.
#include <cmath>
#include <cstring>

#include "dsa_host.cuh"
#include "dsa_rows.cuh"

namespace dsa {

template <int FMT, int TY, bool kRope>
__global__ void __launch_bounds__(32 * kCacheWarps, 5) cache_write_kernel(CacheParams p) {
  write_rows<FMT, TY, kRope>(p, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------ read
// 32 bytes in one store (p 32-byte aligned), or two of 16.
__device__ __forceinline__ void store32(void *p, bool wide, const uint32_t (&w)[8]) {
  const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
  if (wide) {
    tc::stg_v8(p, a, b);
  } else {
    static_cast<uint4 *>(p)[0] = a;
    static_cast<uint4 *>(p)[1] = b;
  }
}
template <int TY>
__device__ __forceinline__ void store16(char *row, int lane, bool wide, const float (&v)[16]) {
  char *d = row + 16 * lane * kTypeBytes<TY>;
  uint32_t w[8];
  if constexpr (TY == DSA_TYPE_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[8 * h + k]);
      store32(d + 32 * h, wide, w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack2<TY>(v[2 * k], v[2 * k + 1]);
    store32(d, wide, w);
  }
}

template <int FMT, int TY>
__global__ void __launch_bounds__(32 * kCacheWarps) cache_read_kernel(CacheParams p) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const int32_t sid = __ldg(p.L.ids + i);
  const int64_t stride = p.stride * kTypeBytes<TY>;
  char *row = static_cast<char *>(p.dst) + i * stride;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.dst) | (uintptr_t)stride) & 31u) == 0;
  float v[16], t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = 0.f;
  const uint8_t *rec = nullptr;
  if (sid >= 0 && (int64_t)sid < p.L.num_slots) rec = record_ptr(p.L, sid);
  if (kDebug && rec && rec + p.L.rec > p.L.base + p.L.extent) rec = nullptr;
  if (rec) decode_record<FMT>(rec, lane, v, t0, t1);   // a slot outside the cache: zeros
  store16<TY>(row, lane, wide, v);
  if constexpr (kV32) {
    char *d = row + (kD + 2 * lane) * kTypeBytes<TY>;
    if constexpr (TY == DSA_TYPE_F32) *reinterpret_cast<float2 *>(d) = make_float2(t0, t1);
    else *reinterpret_cast<uint32_t *>(d) = pack2<TY>(t0, t1);
  }
}

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::CacheParams;

template <int FMT>
cudaError_t launch(const CacheParams &p, int32_t type, bool write, cudaStream_t st) {
  using namespace dsa;
  const int64_t blocks = (p.n + kCacheWarps - 1) / kCacheWarps;
  const unsigned grid = (unsigned)(write && blocks > kCacheBlocks ? kCacheBlocks : blocks);
  constexpr int kT = 32 * kCacheWarps;
#define DSA_CACHE_CASE(TY)                                        \
  case TY:                                                        \
    if (write && p.cos_sin) cache_write_kernel<FMT, TY, true><<<grid, kT, 0, st>>>(p); \
    else if (write) cache_write_kernel<FMT, TY, false><<<grid, kT, 0, st>>>(p); \
    else cache_read_kernel<FMT, TY><<<grid, kT, 0, st>>>(p);        \
    break;
  switch (type) {
    DSA_CACHE_CASE(DSA_TYPE_BF16)
    DSA_CACHE_CASE(DSA_TYPE_F16)
    DSA_CACHE_CASE(DSA_TYPE_F32)
  }
#undef DSA_CACHE_CASE
  return cudaGetLastError();
}

// Checks that both calls share; launches.
dsa_status cache_rows(CacheParams &p, const dsa_cache_desc *cache, const int32_t *slots,
                      int64_t num_rows, const void *rows, int64_t row_stride, int32_t row_type,
                      bool write, dsa_stream_t stream) {
  if (num_rows < 0) return DSA_ERR_INVALID_ARG;
  if (row_type != DSA_TYPE_BF16 && row_type != DSA_TYPE_F16 && row_type != DSA_TYPE_F32)
    return DSA_ERR_UNSUPPORTED;
  const dsa_status s = dsa::fill_cache(cache, p.L);
  if (s != DSA_OK) return s;
  if (num_rows == 0) return DSA_OK;
  if (!slots || !rows) return DSA_ERR_INVALID_ARG;
  const int64_t dims = cache->format == DSA_REC_V32_656 ? 576 : dsa::kD;
  if (row_stride < dims) return DSA_ERR_INVALID_ARG;
  if (num_rows > (int64_t)INT32_MAX * dsa::kCacheWarps) return DSA_ERR_UNSUPPORTED;
  if (!aligned(rows, 16) || row_stride % (row_type == DSA_TYPE_F32 ? 4 : 8) != 0 ||
      !aligned(slots, 4))
    return DSA_ERR_ALIGNMENT;
  p.L.ids = slots;
  p.n = num_rows;
  p.stride = row_stride;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache->format) {
    case DSA_REC_FP8_528: e = launch<DSA_REC_FP8_528>(p, row_type, write, st); break;
    case DSA_REC_NVFP4_288: e = launch<DSA_REC_NVFP4_288>(p, row_type, write, st); break;
    case DSA_REC_FP8_528_UE8M0: e = launch<DSA_REC_FP8_528_UE8M0>(p, row_type, write, st); break;
    case DSA_REC_MODEL1_584: e = launch<DSA_REC_MODEL1_584>(p, row_type, write, st); break;
    case DSA_REC_V32_656: e = launch<DSA_REC_V32_656>(p, row_type, write, st); break;
  }
  return dsa::cuda_status(e);
}

}  // namespace

extern "C" {

dsa_status dsa_cache_write(const dsa_cache_desc *cache, const int32_t *slots, int64_t num_rows,
                           const void *rows, int64_t row_stride, int32_t row_type,
                           const float *norm_weight, float norm_eps, const int64_t *positions,
                           const float *cos_sin, int64_t cos_sin_rows, int32_t rope_style,
                           int32_t *device_status, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_cache_write");
  CacheParams p;
  std::memset(&p, 0, sizeof(p));
  if (rope_style != DSA_ROPE_NEOX && rope_style != DSA_ROPE_GPTJ) return DSA_ERR_INVALID_ARG;
  // (no rows have no positions: an empty array may have no address)
  if (num_rows > 0 && (positions == nullptr) != (cos_sin == nullptr)) return DSA_ERR_INVALID_ARG;
  if (cos_sin && cos_sin_rows < 1) return DSA_ERR_INVALID_ARG;
  if (norm_weight && !(std::isfinite(norm_eps) && norm_eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  if ((cos_sin && (!aligned(cos_sin, 16) || !aligned(positions, 8))) ||
      (norm_weight && !aligned(norm_weight, 16)) || (device_status && !aligned(device_status, 4)))
    return DSA_ERR_ALIGNMENT;
  p.src = rows;
  p.norm_w = norm_weight;
  p.eps = norm_eps;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.cs_rows = cos_sin_rows;
  p.gptj = rope_style == DSA_ROPE_GPTJ ? 1 : 0;
  p.status = device_status;
  return cache_rows(p, cache, slots, num_rows, rows, row_stride, row_type, true, stream);
}

dsa_status dsa_cache_read(const dsa_cache_desc *cache, const int32_t *slots, int64_t num_rows,
                          void *rows, int64_t row_stride, int32_t row_type, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_cache_read");
  CacheParams p;
  std::memset(&p, 0, sizeof(p));
  p.dst = rows;
  return cache_rows(p, cache, slots, num_rows, rows, row_stride, row_type, false, stream);
}

}  // extern "C"

// dsa_qk.cu -- what stands between a layer's projections and its attention
// (dsa_qk_norm): every query head and every token's key normed over their first
// 512 dims,
//
//   y = x w / sqrt(mean x^2 + eps),
//
// and their last 64 dims rotated; queries leave as bf16 rows, keys as records of
// the cache (the arithmetic of dsa_cache_write, whose rows these are).
//
// One pass over memory, a warp per row, lane l on dims 16 l .. 16 l + 15, the
// next row on its way while one is worked on. What bounds it is memory and issue
// together (49 % of the issue slots, 214 instructions a row): the rotation takes
// a pair per lane, through shared memory, as in the cache write (in the four lanes
// that hold the last 64 dims it was a third of the instructions). The first blocks
// take the keys, which cost about two query rows each. 8192 tokens x 128 heads: 375
// us, 5.8 TB/s, 0.85 of the measured copy rate (418 us with rows strided over the
// grid and the rotation in four lanes).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "dsa_host.cuh"
#include "dsa_rows.cuh"

namespace dsa {

struct QkParams {
  CacheParams k;             // the keys (k.n = 0: none); eps, positions, table and status are the queries' too
  int32_t key_blocks;
  const void *q;
  int64_t q_st, q_sh;        // elements
  __nv_bfloat16 *out;
  int64_t o_st, o_sh;
  const float *w;            // [512], or one per head; null: no norm
  int64_t w_sh;              // elements between heads' weights, 0: shared
  int32_t T, H;
};

template <int TY>
__device__ __forceinline__ float one_value(const void *p) {
  if constexpr (TY == DSA_TYPE_F32) return __ldg(static_cast<const float *>(p));
  else if constexpr (TY == DSA_TYPE_F16) return __half2float(__ldg(static_cast<const __half *>(p)));
  else return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(p)));
}
// A query row as loaded, and of a 576-dim row the lane's pair of the last 64 dims.
template <int TY>
struct QueryRaw {
  RowRaw<TY> r;
  float t0, t1;
};

// r with r ~ 1 / sqrt(mean of the row's 512 squares + eps), and v scaled
// alongside where the squares leave fp32 no room (as norm_row: the quotient is the
// same). The outputs are bf16, so the plain fp32 sum (2^-21 of it at most) only
// counts next to a tie.
__device__ __forceinline__ float norm_factor(F2 (&v)[8], float eps) {
  float me;
#pragma unroll 1
  for (bool again = false;; again = true) {   // (the lanes agree)
    F2 sq[2] = {f2_mul(v[0], v[0]), f2_mul(v[1], v[1])};
#pragma unroll
    for (int k = 2; k < 8; ++k) sq[k & 1] = f2_fma(v[k], v[k], sq[k & 1]);
    float s0, s1;
    f2_get(f2_add(sq[0], sq[1]), s0, s1);
    float ss = s0 + s1;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    me = fmaf(ss, 1.0f / kD, eps);
    if (again || (me >= 8.673617379884035e-19f && ss <= 1.2676506002282294e30f)) break;
    uint32_t m = 0;                                // largest magnitude, as bits
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      f2_get(v[k], a, b);
      m = max(m, max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (m >= 0x7F800000u) break;                   // an infinity or a NaN: as it is
    int e = max((int)(m >> 23) - 127, -126);
    if (eps > 0.f) e = max(e, ((int)(__float_as_uint(eps) >> 23) - 126) >> 1);
    const float d = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
    eps = (eps * d) * d;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f2_mul(v[k], f2(d, d));
  }
  return rsqrtf(me);
}

template <int TY, bool kV32, bool kRope>
__device__ __forceinline__ void query_rows(const QkParams &p, int64_t block, int64_t blocks) {
  const int lane = threadIdx.x & 31;
  const bool gptj = p.k.gptj;
  // the lane's pair of the last 64 dims
  const int ia = gptj ? 2 * lane : lane, ib = gptj ? 2 * lane + 1 : lane + 32;
  constexpr bool kStage = kRope && !kV32;
  __shared__ __align__(16) float last_s[kStage ? kCacheWarps : 1][64];
  float *last = last_s[kStage ? threadIdx.x >> 5 : 0];
  // A run of rows to a warp: the heads of a token find its position and table row
  // in L1 (rows strided over the grid each waited for theirs: 418 us).
  const int64_t rows = (int64_t)p.T * p.H, warps = blocks * kCacheWarps, per = (rows + warps - 1) / warps;
  const int64_t first = (block * kCacheWarps + (threadIdx.x >> 5)) * per, end = min(rows, first + per);
  uint32_t t = (uint32_t)(first / p.H), h = (uint32_t)(first % p.H);
  const char *src = static_cast<const char *>(p.q);
  const bool wide_in = (((uintptr_t)src | (uintptr_t)(p.q_st * kTypeBytes<TY>) | (uintptr_t)(p.q_sh * kTypeBytes<TY>)) & 31u) == 0;
  const bool wide_out = (((uintptr_t)p.out | (uintptr_t)(p.o_st * 2) | (uintptr_t)(p.o_sh * 2)) & 31u) == 0;
  F2 w[8];
  auto weights = [&](const float *from) {
    const float4 *w4 = reinterpret_cast<const float4 *>(from) + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = __ldg(w4 + k);
      w[2 * k] = f2(x.x, x.y);
      w[2 * k + 1] = f2(x.z, x.w);
    }
  };
  if (p.w && p.w_sh == 0) weights(p.w);
  QueryRaw<TY> next;
  auto fetch = [&](uint32_t ft, uint32_t fh) {
    const char *row = src + ((int64_t)ft * p.q_st + (int64_t)fh * p.q_sh) * kTypeBytes<TY>;
    load_row<TY, false>(row, lane, wide_in, next.r);
    if constexpr (kV32) {
      next.t0 = one_value<TY>(row + (kD + ia) * kTypeBytes<TY>);
      next.t1 = one_value<TY>(row + (kD + ib) * kTypeBytes<TY>);
    }
  };
  if (first < end) fetch(t, h);
#pragma unroll 1
  for (int64_t i = first; i < end; ++i) {   // whole warps
    const QueryRaw<TY> raw = next;
    const uint32_t ct = t, ch = h;
    if (++h == (uint32_t)p.H) {
      h = 0;
      ++t;
    }
    if (i + 1 < end) fetch(t, h);
    float co = 0.f, si = 0.f;
    if constexpr (kRope) {
      const int64_t pos = __ldg(p.k.positions + ct);
      if (pos < 0 || pos >= p.k.cs_rows) {   // outside the table: the token is not written
        if (p.k.status && lane == 0) report_status(p.k.status, DSA_ERR_INVALID_ARG);
        continue;
      }
      co = __ldg(p.k.cos_sin + pos * 64 + lane);
      si = __ldg(p.k.cos_sin + pos * 64 + 32 + lane);
    }
    F2 v[8];
    float u0, u1;
    unpack_row<TY, false>(raw.r, v, u0, u1);
    if (p.w) {
      if (p.w_sh != 0) weights(p.w + (int64_t)ch * p.w_sh);
      const float r = norm_factor(v, p.k.eps);
      const F2 r2 = f2(r, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = f2_mul(f2_mul(v[k], r2), w[k]);
    }
    __nv_bfloat16 *dst = p.out + (int64_t)ct * p.o_st + (int64_t)ch * p.o_sh;
    if (kStage && lane >= 28) {   // on their way to a pair per lane
      ulonglong2 *d = reinterpret_cast<ulonglong2 *>(last + 16 * (lane - 28));
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = make_ulonglong2(v[2 * k].v, v[2 * k + 1].v);
    } else {
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float a, b;
        f2_get(v[k], a, b);
        o[k] = bf16x2_bits(a, b);
      }
      const uint4 oa = make_uint4(o[0], o[1], o[2], o[3]), ob = make_uint4(o[4], o[5], o[6], o[7]);
      if (wide_out) {
        tc::stg_v8(dst + 16 * lane, oa, ob);
      } else {
        *reinterpret_cast<uint4 *>(dst + 16 * lane) = oa;
        *reinterpret_cast<uint4 *>(dst + 16 * lane + 8) = ob;
      }
    }
    if constexpr (kStage || kV32) {
      float a = raw.t0, b = raw.t1;
      if constexpr (kStage) {
        __syncwarp();
        a = last[ia];
        b = last[ib];
      }
      if constexpr (kRope) {
        const float ra = fmaf(a, co, -(b * si)), rb = fmaf(b, co, a * si);
        a = ra;
        b = rb;
      }
      __nv_bfloat16 *tail = dst + (kV32 ? kD : kD - 64);
      if (gptj) {
        *reinterpret_cast<uint32_t *>(tail + ia) = bf16x2_bits(a, b);
      } else {
        tail[ia] = __float2bfloat16_rn(a);
        tail[ib] = __float2bfloat16_rn(b);
      }
      if constexpr (kStage) __syncwarp();   // the stage is free again
    }
  }
}

template <int FMT, int TY, bool kRope>
__global__ void __launch_bounds__(32 * kCacheWarps, 5) qk_norm_kernel(const __grid_constant__ QkParams p) {
  if ((int32_t)blockIdx.x < p.key_blocks) write_rows<FMT, TY, kRope>(p.k, blockIdx.x, p.key_blocks);
  else query_rows<TY, FMT == DSA_REC_V32_656, kRope>(p, blockIdx.x - p.key_blocks, gridDim.x - p.key_blocks);
}

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::QkParams;

template <int FMT>
cudaError_t launch(QkParams &p, int32_t type, cudaStream_t st) {
  using namespace dsa;
  // A warp per row while all blocks are resident; past that the resident ones,
  // divided as the work is, a key counting as two query rows.
  const int64_t kb = (p.k.n + kCacheWarps - 1) / kCacheWarps, qb = ((int64_t)p.T * p.H + kCacheWarps - 1) / kCacheWarps;
  int64_t keys = kb, blocks = kb + qb;
  if (blocks > kCacheBlocks) {
    blocks = kCacheBlocks;
    keys = kb == 0 ? 0 : std::min<int64_t>(kb, std::max<int64_t>(1, kCacheBlocks * 2 * kb / (2 * kb + qb)));
  }
  p.key_blocks = (int32_t)keys;
  const unsigned grid = (unsigned)blocks;
  constexpr int kT = 32 * kCacheWarps;
#define DSA_QK_CASE(TY)                                                      \
  case TY:                                                                   \
    if (p.k.cos_sin) qk_norm_kernel<FMT, TY, true><<<grid, kT, 0, st>>>(p);  \
    else qk_norm_kernel<FMT, TY, false><<<grid, kT, 0, st>>>(p);             \
    break;
  switch (type) {
    DSA_QK_CASE(DSA_TYPE_BF16)
    DSA_QK_CASE(DSA_TYPE_F16)
    DSA_QK_CASE(DSA_TYPE_F32)
  }
#undef DSA_QK_CASE
  return cudaGetLastError();
}

}  // namespace

extern "C" {

dsa_status dsa_qk_norm(int32_t num_tokens, int32_t num_heads, int32_t dims, int32_t row_type, const void *q,
                       int64_t q_stride_t, int64_t q_stride_h, const float *q_weight, int64_t q_weight_stride_h,
                       void *out, int64_t out_stride_t, int64_t out_stride_h, const void *keys, int64_t key_stride,
                       const float *key_weight, const dsa_cache_desc *cache, const int32_t *slots, float eps,
                       const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, int32_t rope_style,
                       int32_t *device_status, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_qk_norm");
  if (num_tokens < 0 || num_heads < 1 || (dims != 512 && dims != 576)) return DSA_ERR_INVALID_ARG;
  if (row_type != DSA_TYPE_BF16 && row_type != DSA_TYPE_F16 && row_type != DSA_TYPE_F32) return DSA_ERR_UNSUPPORTED;
  if (rope_style != DSA_ROPE_NEOX && rope_style != DSA_ROPE_GPTJ) return DSA_ERR_INVALID_ARG;
  if (!(std::isfinite(eps) && eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  if ((int64_t)num_tokens * num_heads > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  QkParams p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  int32_t fmt = dims == 576 ? DSA_REC_V32_656 : DSA_REC_FP8_528;
  if (keys || cache || slots || key_weight) {
    const dsa_status s = dsa::fill_cache(cache, p.k.L);
    if (s != DSA_OK) return s;
    fmt = cache->format;
    if ((fmt == DSA_REC_V32_656) != (dims == 576)) return DSA_ERR_UNSUPPORTED;
    if (num_tokens > 0 && (!keys || !slots)) return DSA_ERR_INVALID_ARG;
    p.k.n = num_tokens;
  }
  if (num_tokens == 0) return DSA_OK;
  if (!q || !out) return DSA_ERR_INVALID_ARG;
  if ((positions == nullptr) != (cos_sin == nullptr)) return DSA_ERR_INVALID_ARG;
  if (cos_sin && cos_sin_rows < 1) return DSA_ERR_INVALID_ARG;
  const int64_t H = num_heads;
  if (q_stride_h < dims || q_stride_t < (H - 1) * q_stride_h + dims || out_stride_h < dims ||
      out_stride_t < (H - 1) * out_stride_h + dims || (p.k.n && key_stride < dims) ||
      (q_weight && q_weight_stride_h != 0 && q_weight_stride_h < 512))
    return DSA_ERR_INVALID_ARG;
  const int64_t per = row_type == DSA_TYPE_F32 ? 4 : 8;   // elements in 16 bytes
  if (!aligned(q, 16) || q_stride_t % per != 0 || q_stride_h % per != 0 || !aligned(out, 16) || out_stride_t % 8 != 0 ||
      out_stride_h % 8 != 0 || (q_weight && (!aligned(q_weight, 16) || q_weight_stride_h % 4 != 0)) ||
      (p.k.n && (!aligned(keys, 16) || key_stride % per != 0 || !aligned(slots, 4))) ||
      (key_weight && !aligned(key_weight, 16)) || (cos_sin && (!aligned(cos_sin, 16) || !aligned(positions, 8))) ||
      (device_status && !aligned(device_status, 4)))
    return DSA_ERR_ALIGNMENT;
  // In place only row for row: the queries' own type and strides.
  if (out == q && (row_type != DSA_TYPE_BF16 || out_stride_t != q_stride_t || out_stride_h != q_stride_h))
    return DSA_ERR_INVALID_ARG;
  p.k.L.ids = slots;
  p.k.src = keys;
  p.k.stride = key_stride;
  p.k.norm_w = key_weight;
  p.k.eps = eps;
  p.k.positions = positions;
  p.k.cos_sin = cos_sin;
  p.k.cs_rows = cos_sin_rows;
  p.k.gptj = rope_style == DSA_ROPE_GPTJ ? 1 : 0;
  p.k.status = device_status;
  p.q = q;
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.o_st = out_stride_t;
  p.o_sh = out_stride_h;
  p.w = q_weight;
  p.w_sh = q_weight_stride_h;
  p.T = num_tokens;
  p.H = num_heads;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (fmt) {
    case DSA_REC_FP8_528: e = launch<DSA_REC_FP8_528>(p, row_type, st); break;
    case DSA_REC_NVFP4_288: e = launch<DSA_REC_NVFP4_288>(p, row_type, st); break;
    case DSA_REC_FP8_528_UE8M0: e = launch<DSA_REC_FP8_528_UE8M0>(p, row_type, st); break;
    case DSA_REC_MODEL1_584: e = launch<DSA_REC_MODEL1_584>(p, row_type, st); break;
    case DSA_REC_V32_656: e = launch<DSA_REC_V32_656>(p, row_type, st); break;
  }
  return dsa::cuda_status(e);
}

}  // extern "C"

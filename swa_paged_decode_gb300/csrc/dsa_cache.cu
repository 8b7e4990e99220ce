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
#include "dsa_records.cuh"

namespace dsa {

struct CacheParams {
  ListArgs L;                // the cache (ids: slot of each row)
  int64_t n;                 // rows
  const void *src;           // write: rows in
  void *dst;                 // read: rows out
  int64_t stride;            // elements between rows
  const float *norm_w;       // write: RMS norm of dims 0..511, or null
  float eps;
  const int64_t *positions;  // write: RoPE of the last 64 dims, or null
  const float *cos_sin;
  int64_t cs_rows;
  int32_t gptj;
  int32_t *status;           // optional status word
};

constexpr int kCacheWarps = 4;   // rows per block (a row has no shared state)

// Type TY's 16 values at p (16-byte aligned) -> fp32.
template <int TY>
__device__ __forceinline__ void load16(const void *p, float (&v)[16]) {
  if constexpr (TY == DSA_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = ld_row(static_cast<const uint4 *>(p) + i);
      v[4 * i] = __uint_as_float(w.x);
      v[4 * i + 1] = __uint_as_float(w.y);
      v[4 * i + 2] = __uint_as_float(w.z);
      v[4 * i + 3] = __uint_as_float(w.w);
    }
  } else {
    const uint4 a = ld_row(p), b = ld_row(static_cast<const uint4 *>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (TY == DSA_TYPE_BF16) {
        v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}
template <int TY>
__device__ __forceinline__ void load2(const void *p, float &a, float &b) {
  if constexpr (TY == DSA_TYPE_F32) {
    const float2 f = __ldg(static_cast<const float2 *>(p));
    a = f.x;
    b = f.y;
  } else {
    const uint32_t w = __ldg(static_cast<const uint32_t *>(p));
    if constexpr (TY == DSA_TYPE_BF16) {
      a = bf16_bits_to_f32(w & 0xFFFFu);
      b = bf16_bits_to_f32(w >> 16);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
      a = f.x;
      b = f.y;
    }
  }
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <int TY>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (TY == DSA_TYPE_BF16) return bf16x2_bits(lo, hi);
  else return tc::pack_f16x2(lo, hi);
}
template <int TY>
constexpr int kTypeBytes = TY == DSA_TYPE_F32 ? 4 : 2;

// Largest magnitude of 16 values as bits: magnitudes order as their bits, a
// NaN above every number, so a NaN among the values is not lost.
__device__ __forceinline__ uint32_t amax16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}
// ... over the block's neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
  for (int off = 1; off < LANES; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}
// ue8m0 byte of a block: the smallest power of two 2^ex with amax / 448 <=
// 2^ex. 448 = 1.75 * 2^8, so with amax = m * 2^e, ex = e - 8, plus one when
// m > 1.75; exact, no logarithm. ex is clamped to [-127, 127], a block of
// zeros takes 2^0, an infinity 254 and a NaN 255 (the E8M0 NaN).
__device__ __forceinline__ uint32_t ue8m0_of(uint32_t amax) {
  if (amax == 0u) return 127u;
  if (amax >= 0x7F800000u) return amax == 0x7F800000u ? 254u : 255u;
  const int b = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(b, 0);
}
// 2^(127 - byte), exact (byte 254 gives the subnormal 2^-127).
__device__ __forceinline__ float ue8m0_down(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(byte == 254u ? 0x00400000u : (254u - byte) << 23);
}
// 16 values times a power of two -> e4m3 codes.
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float down) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2_rn_sat(v[4 * i] * down, v[4 * i + 1] * down) |
           (e4m3x2_rn_sat(v[4 * i + 2] * down, v[4 * i + 3] * down) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Eight fp32 values -> e2m1 codes (nearest even, saturating at 6), element i
// in nibble i; a zero code has no sign.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[16], int o) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[o]), "f"(y[o + 1]), "f"(y[o + 2]), "f"(y[o + 3]), "f"(y[o + 4]), "f"(y[o + 5]),
        "f"(y[o + 6]), "f"(y[o + 7]));
  const uint32_t nz = (w | (w >> 1) | (w >> 2)) & 0x11111111u;
  return w & (nz * 15u);
}

// ------------------------------------------------------------ write
// x -> (norm) -> (rotation) -> codes and scales, all in fp32 from the loaded
// values to the codes: nothing is rounded to 16 bits in between.
template <int FMT, int TY>
__global__ void __launch_bounds__(32 * kCacheWarps) cache_write_kernel(CacheParams p) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;   // whole warps
  const int32_t sid = __ldg(p.L.ids + i);
  const char *row = static_cast<const char *>(p.src) + i * p.stride * kTypeBytes<TY>;
  float v[16], t0 = 0.f, t1 = 0.f;
  load16<TY>(row + 16 * lane * kTypeBytes<TY>, v);
  if constexpr (kV32) load2<TY>(row + (kD + 2 * lane) * kTypeBytes<TY>, t0, t1);
  if (sid < 0 || (int64_t)sid >= p.L.num_slots) return;   // padding: nothing is written
  // x * w / sqrt(mean x^2 + eps) over dims 0..511, each result its exact
  // value rounded to fp32 (but for a few in a hundred off by one step): a
  // relative error of 2^-23 in front of the quantization would move the codes
  // of four elements in a million. The squares are summed as a tree and the
  // lanes' sums with their rounding errors; the root's reciprocal carries a
  // correction r1, and the products theirs. 90 instructions more for a row
  // than the plain fp32 form.
  if (p.norm_w) {
    float sq[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) sq[k] = fmaf(v[2 * k], v[2 * k], v[2 * k + 1] * v[2 * k + 1]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < o; ++k) sq[k] += sq[k + o];
    float ss = sq[0], sl = 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, ss, off), ol = __shfl_xor_sync(0xffffffffu, sl, off);
      const float t = ss + o, z = t - ss;          // ss + o = t + the error of t
      sl += ol + ((ss - (t - z)) + (o - z));
      ss = t;
    }
    const float ms = ss * (1.0f / kD), me = ms + p.eps, mz = me - ms;
    const float ml = fmaf(sl, 1.0f / kD, (ms - (me - mz)) + (p.eps - mz));
    // 1 / sqrt(me + ml) = r0 + r1: one Newton step, its residual 1 - (me + ml) r0^2 by FMAs
    const float r0 = 1.0f / sqrtf(me);
    const float h = me * r0, hl = fmaf(me, r0, -h) + ml * r0;
    const float r1 = 0.5f * r0 * fmaf(-hl, r0, fmaf(-h, r0, 1.0f));
    const float4 *w4 = reinterpret_cast<const float4 *>(p.norm_w) + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 w = __ldg(w4 + k);
      const float wk[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float &x = v[4 * k + e];
        const float q = x * wk[e], ql = fmaf(x, wk[e], -q);
        x = fmaf(q, r0, fmaf(q, r1, ql * r0));
      }
    }
  }
  // (a, b) -> (a cos - b sin, b cos + a sin) on the last 64 dims
  if (p.cos_sin) {
    const int64_t pos = __ldg(p.positions + i);
    if (pos < 0 || pos >= p.cs_rows) {   // outside the table: the row is not written
      if (p.status && lane == 0) report_status(p.status, DSA_ERR_INVALID_ARG);
      return;
    }
    const float *cs = p.cos_sin + pos * 64;
    if constexpr (kV32) {   // dims 512 + 2 lane, + 1
      if (p.gptj) {         // one pair
        const float c = __ldg(cs + lane), s = __ldg(cs + 32 + lane);
        const float a = t0, b = t1;
        t0 = fmaf(a, c, -(b * s));
        t1 = fmaf(b, c, a * s);
      } else {              // the partners of two pairs sit 16 lanes away
        const float2 c = __ldg(reinterpret_cast<const float2 *>(cs) + (lane & 15));
        const float2 s = __ldg(reinterpret_cast<const float2 *>(cs) + 16 + (lane & 15));
        const float o0 = __shfl_xor_sync(0xffffffffu, t0, 16), o1 = __shfl_xor_sync(0xffffffffu, t1, 16);
        const float sg = lane < 16 ? -1.f : 1.f;
        t0 = fmaf(t0, c.x, sg * (o0 * s.x));
        t1 = fmaf(t1, c.y, sg * (o1 * s.y));
      }
    } else {                // lanes 28..31
      const int r = lane - 28;
      if (p.gptj) {
        if (r >= 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float c = __ldg(cs + 8 * r + k), s = __ldg(cs + 32 + 8 * r + k);
            const float a = v[2 * k], b = v[2 * k + 1];
            v[2 * k] = fmaf(a, c, -(b * s));
            v[2 * k + 1] = fmaf(b, c, a * s);
          }
        }
      } else {              // partners two lanes away
        const float sg = r < 2 ? -1.f : 1.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float o = __shfl_xor_sync(0xffffffffu, v[k], 2);
          if (r >= 0) {
            const float c = __ldg(cs + 16 * (r & 1) + k), s = __ldg(cs + 32 + 16 * (r & 1) + k);
            v[k] = fmaf(v[k], c, sg * (o * s));
          }
        }
      }
    }
  }
  uint8_t *rec = const_cast<uint8_t *>(record_ptr(p.L, sid));
  if (kDebug && (rec < p.L.base || rec + p.L.rec > p.L.base + p.L.extent)) {
    if (p.status) report_status(p.status, DSA_ERR_BOUNDS);
    return;
  }
  const uint32_t am = amax16(v);
  if constexpr (FMT == DSA_REC_FP8_528 || kV32) {
    const uint32_t m = block_max<8>(am);
    const float s = __fdiv_rn(__uint_as_float(m), 448.0f);
    const float d = s > 0.f || !(s == s) ? s : 1.0f;   // zero blocks divide by one
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = e4m3x2_rn_sat(__fdiv_rn(v[4 * k], d), __fdiv_rn(v[4 * k + 1], d)) |
             (e4m3x2_rn_sat(__fdiv_rn(v[4 * k + 2], d), __fdiv_rn(v[4 * k + 3], d)) << 16);
    *reinterpret_cast<uint4 *>(rec + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 7) == 0) *reinterpret_cast<float *>(rec + 512 + (lane >> 1)) = s;
    if constexpr (kV32) *reinterpret_cast<uint32_t *>(rec + 528 + 4 * lane) = bf16x2_bits(t0, t1);
  } else if constexpr (FMT == DSA_REC_FP8_528_UE8M0) {
    const uint32_t e = ue8m0_of(block_max<2>(am));
    *reinterpret_cast<uint4 *>(rec + 16 * lane) = codes16(v, ue8m0_down(e));
    if ((lane & 1) == 0) rec[512 + (lane >> 1)] = (uint8_t)e;
  } else if constexpr (FMT == DSA_REC_MODEL1_584) {
    const uint32_t e = ue8m0_of(block_max<4>(am));
    if (lane < 28) {         // 8-byte aligned records
      const uint4 w = codes16(v, ue8m0_down(e));
      uint2 *d = reinterpret_cast<uint2 *>(rec + 16 * lane);
      d[0] = make_uint2(w.x, w.y);
      d[1] = make_uint2(w.z, w.w);
      if ((lane & 3) == 0) rec[576 + (lane >> 2)] = (uint8_t)e;
    } else {                 // the bf16 part, and the unused byte
      uint2 *d = reinterpret_cast<uint2 *>(rec + 448 + 32 * (lane - 28));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        d[k] = make_uint2(bf16x2_bits(v[4 * k], v[4 * k + 1]), bf16x2_bits(v[4 * k + 2], v[4 * k + 3]));
      if (lane == 28) rec[583] = 0;
    }
  } else {                   // NVFP4: a block is one lane's 16 dims
    const float a6 = fminf(__fdiv_rn(__uint_as_float(am), 6.0f), 448.0f);
    const uint32_t sb = am > 0x7F800000u ? 0x7Fu : (e4m3x2_rn_sat(a6, 0.f) & 0xFFu);
    const float s = e4m3_to_f32(sb);
    uint2 w = make_uint2(0u, 0u);
    if (sb != 0u && sb != 0x7Fu) {
      float y[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) y[k] = __fdiv_rn(v[k], s);
      w = make_uint2(e2m1x8(y, 0), e2m1x8(y, 8));
    }
    *reinterpret_cast<uint2 *>(rec + 8 * lane) = w;
    rec[256 + lane] = (uint8_t)sb;
  }
}

// ------------------------------------------------------------ read
template <int TY>
__device__ __forceinline__ void store16(char *row, int lane, const float (&v)[16]) {
  uint4 *d = reinterpret_cast<uint4 *>(row + 16 * lane * kTypeBytes<TY>);
  if constexpr (TY == DSA_TYPE_F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      d[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                        __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      d[k] = make_uint4(pack2<TY>(v[8 * k], v[8 * k + 1]), pack2<TY>(v[8 * k + 2], v[8 * k + 3]),
                        pack2<TY>(v[8 * k + 4], v[8 * k + 5]), pack2<TY>(v[8 * k + 6], v[8 * k + 7]));
  }
}
template <int FMT, int TY>
__global__ void __launch_bounds__(32 * kCacheWarps) cache_read_kernel(CacheParams p) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const int32_t sid = __ldg(p.L.ids + i);
  char *row = static_cast<char *>(p.dst) + i * p.stride * kTypeBytes<TY>;
  float v[16], t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = 0.f;
  const uint8_t *rec = nullptr;
  if (sid >= 0 && (int64_t)sid < p.L.num_slots) rec = record_ptr(p.L, sid);
  if (kDebug && rec && rec + p.L.rec > p.L.base + p.L.extent) rec = nullptr;
  if (rec) decode_record<FMT>(rec, lane, v, t0, t1);   // a slot outside the cache: zeros
  store16<TY>(row, lane, v);
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
  const unsigned grid = (unsigned)((p.n + kCacheWarps - 1) / kCacheWarps);
  constexpr int kT = 32 * kCacheWarps;
#define DSA_CACHE_CASE(TY)                                        \
  case TY:                                                        \
    if (write) cache_write_kernel<FMT, TY><<<grid, kT, 0, st>>>(p); \
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
  if ((positions == nullptr) != (cos_sin == nullptr)) return DSA_ERR_INVALID_ARG;
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

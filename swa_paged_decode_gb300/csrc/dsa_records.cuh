// dsa_records.cuh -- a record's values in fp32, a warp per record: lane l
// holds dims 16 l .. 16 l + 15 (and of a V3.2 record dims 512 + 2 l, + 1).
#pragma once

#include "dsa_internal.cuh"
#include "tc_ptx.cuh"

namespace dsa {

// 16 bytes of a row that is read once.
__device__ __forceinline__ uint4 ld_row(const void *p) { return tc::ldg_nc_v4(p); }

__device__ __forceinline__ void decode16_e4m3(const uint4 &w, float s, float (&v)[16]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t lo, hi;
    tc::e4m3x4_to_f16x4(u[k], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v[4 * k] = a.x * s;
    v[4 * k + 1] = a.y * s;
    v[4 * k + 2] = b.x * s;
    v[4 * k + 3] = b.y * s;
  }
}

template <int FMT>
__device__ __forceinline__ void decode_record(const uint8_t *rec, int lane, float (&v)[16], float &t0,
                                              float &t1) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  if constexpr (FMT == DSA_REC_FP8_528 || kV32) {
    const uint4 w = ld_row(rec + 16 * lane);
    const float s = __ldg(reinterpret_cast<const float *>(rec + 512) + (lane >> 3));
    decode16_e4m3(w, s, v);
    if constexpr (kV32) {
      const uint32_t b = __ldg(reinterpret_cast<const uint32_t *>(rec + 528) + lane);
      t0 = bf16_bits_to_f32(b & 0xFFFFu);
      t1 = bf16_bits_to_f32(b >> 16);
    }
  } else if constexpr (FMT == DSA_REC_FP8_528_UE8M0) {
    const uint4 w = ld_row(rec + 16 * lane);
    decode16_e4m3(w, ue8m0_to_f32(__ldg(rec + 512 + (lane >> 1))), v);
  } else if constexpr (FMT == DSA_REC_MODEL1_584) {
    if (lane < 28) {
      const uint2 a = tc::ldg_nc_v2(rec + 16 * lane), b = tc::ldg_nc_v2(rec + 16 * lane + 8);
      decode16_e4m3(make_uint4(a.x, a.y, b.x, b.y), ue8m0_to_f32(__ldg(rec + 576 + (lane >> 2))), v);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint2 a = tc::ldg_nc_v2(rec + 448 + 32 * (lane - 28) + 8 * k);
        v[4 * k] = bf16_bits_to_f32(a.x & 0xFFFFu);
        v[4 * k + 1] = bf16_bits_to_f32(a.x >> 16);
        v[4 * k + 2] = bf16_bits_to_f32(a.y & 0xFFFFu);
        v[4 * k + 3] = bf16_bits_to_f32(a.y >> 16);
      }
    }
  } else {
    const uint2 w = tc::ldg_nc_v2(rec + 8 * lane);
    const uint32_t sb = __ldg(rec + 256 + lane);
    const float s = (sb & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_to_f32(sb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[4];
      tc::e2m1x8_to_f16x8(h ? w.y : w.x, f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&f[k]));
        v[8 * h + 2 * k] = a.x * s;
        v[8 * h + 2 * k + 1] = a.y * s;
      }
    }
  }
}

}  // namespace dsa

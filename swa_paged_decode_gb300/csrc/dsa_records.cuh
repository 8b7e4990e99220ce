// dsa_records.cuh -- a record's values in fp32, a warp per record: lane l
// holds dims 16 l .. 16 l + 15 (and of a V3.2 record dims 512 + 2 l, + 1).
#pragma once

#include <cuda_fp16.h>

#include "dsa_internal.cuh"
#include "pair_ptx.cuh"

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

// A lane's share of a record as loaded (words not used by a format cost
// nothing).
struct RawRecord {
  uint32_t w[8];   // codes (fp8: 4 words, NVFP4: 2; MODEL1 lanes 28..31: 16 bf16 values)
  uint32_t s;      // the scale of the lane's block, as stored
  uint32_t t;      // V3.2: 2 bf16 values
};

template <int FMT>
__device__ __forceinline__ void load_record(const uint8_t *rec, int lane, RawRecord &r) {
  if constexpr (FMT == DSA_REC_NVFP4_288) {
    const uint2 a = tc::ldg_nc_v2(rec + 8 * lane);
    r.w[0] = a.x;
    r.w[1] = a.y;
    r.s = __ldg(rec + 256 + lane);
  } else if constexpr (FMT == DSA_REC_MODEL1_584) {   // 8-byte aligned; lanes 28..31: 32 bytes
    const uint8_t *p = lane < 28 ? rec + 16 * lane : rec + 448 + 32 * (lane - 28);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint2 a = tc::ldg_nc_v2(p + 8 * k);
      r.w[2 * k] = a.x;
      r.w[2 * k + 1] = a.y;
    }
    if (lane >= 28) {
#pragma unroll
      for (int k = 2; k < 4; ++k) {
        const uint2 a = tc::ldg_nc_v2(p + 8 * k);
        r.w[2 * k] = a.x;
        r.w[2 * k + 1] = a.y;
      }
    }
    r.s = __ldg(rec + 576 + min(lane >> 2, 6));
  } else {
    const uint4 a = ld_row(rec + 16 * lane);
    r.w[0] = a.x;
    r.w[1] = a.y;
    r.w[2] = a.z;
    r.w[3] = a.w;
    if constexpr (FMT == DSA_REC_FP8_528_UE8M0) {
      r.s = __ldg(rec + 512 + (lane >> 1));
    } else {
      r.s = __ldg(reinterpret_cast<const uint32_t *>(rec + 512) + (lane >> 3));
      if constexpr (FMT == DSA_REC_V32_656) r.t = __ldg(reinterpret_cast<const uint32_t *>(rec + 528) + lane);
    }
  }
}

template <int FMT>
__device__ __forceinline__ void expand_record(const RawRecord &r, int lane, float (&v)[16], float &t0, float &t1) {
  if constexpr (FMT == DSA_REC_NVFP4_288) {
    const float s = (r.s & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_to_f32(r.s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[4];
      tc::e2m1x8_to_f16x8(r.w[h], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&f[k]));
        v[8 * h + 2 * k] = a.x * s;
        v[8 * h + 2 * k + 1] = a.y * s;
      }
    }
  } else {
    if (FMT == DSA_REC_MODEL1_584 && lane >= 28) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[2 * k] = bf16_bits_to_f32(r.w[k] & 0xFFFFu);
        v[2 * k + 1] = bf16_bits_to_f32(r.w[k] >> 16);
      }
    } else {
      const float s = (FMT == DSA_REC_FP8_528 || FMT == DSA_REC_V32_656) ? __uint_as_float(r.s) : ue8m0_to_f32(r.s);
      decode16_e4m3(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), s, v);
    }
    if constexpr (FMT == DSA_REC_V32_656) {
      t0 = bf16_bits_to_f32(r.t & 0xFFFFu);
      t1 = bf16_bits_to_f32(r.t >> 16);
    }
  }
}

// e with every value of the lane's share below 2^(e + 1): from the block's
// scale (its largest code is 448 or 6) and the bf16 parts. kZeroShare where all
// codes are zero: the scale says nothing then (ue8m0 blocks of zeros carry
// 2^0, which in front of small values would cost them their low bits).
constexpr int kZeroShare = -127;
template <int FMT>
__device__ __forceinline__ int record_exponent(const RawRecord &r, int lane) {
  if constexpr (FMT == DSA_REC_NVFP4_288) {   // 6 s < 2^(k + 4), s < 2^(k + 1)
    const uint32_t b = r.s & 0x7Fu;
    if (((r.w[0] | r.w[1]) & 0x77777777u) == 0u || b == 0u) return kZeroShare;
    return (b < 8u ? -6 : (int)(b >> 3) - 7) + 3;
  } else {
    if (FMT == DSA_REC_MODEL1_584 && lane >= 28) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __vmaxu2(m, r.w[k] & 0x7FFF7FFFu);
      return (int)(max(m & 0xFFFFu, m >> 16) >> 7) - 127;
    }
    const bool zero = ((r.w[0] | r.w[1] | r.w[2] | r.w[3]) & 0x7F7F7F7Fu) == 0u;
    int e = kZeroShare;
    if constexpr (FMT == DSA_REC_FP8_528 || FMT == DSA_REC_V32_656) {   // 448 s < 2^(k + 10)
      if (!zero && (r.s & 0x7FFFFFFFu) != 0u) e = (int)((r.s >> 23) & 0xFFu) - 127 + 9;
    } else {
      if (!zero) e = (int)(r.s & 0xFFu) - 127 + 8;                      // 448 * 2^k < 2^(k + 9)
    }
    if constexpr (FMT == DSA_REC_V32_656) {
      const uint32_t m = __vmaxu2(r.t & 0x7FFF7FFFu, 0u);
      e = max(e, (int)(max(m & 0xFFFFu, m >> 16) >> 7) - 127);
    }
    return e;
  }
}

template <int FMT>
__device__ __forceinline__ void decode_record(const uint8_t *rec, int lane, float (&v)[16], float &t0,
                                              float &t1) {
  RawRecord r;
  load_record<FMT>(rec, lane, r);
  expand_record<FMT>(r, lane, v, t0, t1);
}

}  // namespace dsa

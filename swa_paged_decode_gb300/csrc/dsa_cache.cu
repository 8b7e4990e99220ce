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

constexpr int kCacheWarps = 4;      // warps per block (a row has no shared state)
constexpr int kCacheBlocks = 760;   // 5 per SM of 152, all resident: more rows than that make the warps loop

// ------------------------------------------------------------ packed fp32
// Two fp32 values in a register pair: one instruction for both (each result
// rounded as the scalar instruction rounds it).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_get(F2 a, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// ------------------------------------------------------------ rows
template <int TY>
constexpr int kTypeBytes = TY == DSA_TYPE_F32 ? 4 : 2;

// A lane's 16 values of a row as loaded: 32 or 64 bytes, in 32-byte loads where
// the rows allow it (`wide`: they start on 32 bytes), else 16-byte ones.
template <int TY>
struct RowRaw {
  uint4 q[TY == DSA_TYPE_F32 ? 4 : 2];
  uint32_t t[TY == DSA_TYPE_F32 ? 2 : 1];   // V3.2: dims 512 + 2 lane, + 1
};
template <int TY, bool kV32>
__device__ __forceinline__ void load_row(const char *row, int lane, bool wide, RowRaw<TY> &r) {
  constexpr int kN = TY == DSA_TYPE_F32 ? 4 : 2;
  const char *p = row + 16 * lane * kTypeBytes<TY>;
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    if (wide) {
      tc::ldg_nc_v8(p + 16 * i, r.q[i], r.q[i + 1]);
    } else {
      r.q[i] = ld_row(p + 16 * i);
      r.q[i + 1] = ld_row(p + 16 * i + 16);
    }
  }
  if constexpr (kV32) {
    const uint32_t *p2 = reinterpret_cast<const uint32_t *>(row + (kD + 2 * lane) * kTypeBytes<TY>);
#pragma unroll
    for (int i = 0; i < kTypeBytes<TY> / 2; ++i) r.t[i] = __ldg(p2 + i);
  }
}
template <int TY>
__device__ __forceinline__ F2 unpack2(uint32_t w) {
  if constexpr (TY == DSA_TYPE_BF16) return f2(bf16_bits_to_f32(w & 0xFFFFu), __uint_as_float(w & 0xFFFF0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return f2(f.x, f.y);
}
template <int TY, bool kV32>
__device__ __forceinline__ void unpack_row(const RowRaw<TY> &r, F2 (&v)[8], float &t0, float &t1) {
#pragma unroll
  for (int i = 0; i < (TY == DSA_TYPE_F32 ? 4 : 2); ++i) {
    const uint32_t w[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
    if constexpr (TY == DSA_TYPE_F32) {
      v[2 * i] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      v[2 * i + 1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * i + k] = unpack2<TY>(w[k]);
    }
  }
  if constexpr (kV32) {
    if constexpr (TY == DSA_TYPE_F32) {
      t0 = __uint_as_float(r.t[0]);
      t1 = __uint_as_float(r.t[1]);
    } else {
      f2_get(unpack2<TY>(r.t[0]), t0, t1);
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

// ------------------------------------------------------------ blocks
// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest magnitude of a block: this lane's 16 values, then the block's
// neighbouring lanes. As bits: magnitudes order as their bits, a NaN above
// every number.
template <int LANES>
__device__ __forceinline__ uint32_t block_amax(const float (&v)[16]) {
  float a = max_nan(fabsf(v[0]), fabsf(v[1])), b = max_nan(fabsf(v[2]), fabsf(v[3]));
#pragma unroll
  for (int i = 4; i < 16; i += 2) {
    a = max_nan(a, fabsf(v[i]));
    b = max_nan(b, fabsf(v[i + 1]));
  }
  uint32_t m = __float_as_uint(max_nan(a, b));
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
// y = -x / s for 16 values, each rounded to nearest (the codes' signs are
// flipped back in packed form). With inv = 1 / s rounded to nearest, q = -x inv
// and the exact remainder x + q s, q - inv (x + q s) rounds to the quotient
// (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000", 1990): 3 packed instructions for two values, and a zero keeps
// its sign. The remainder is exact while it stays clear of the subnormals,
// which a scale in 2^-60 .. 2^60 sees to wherever the quotient matters (below
// 2^-10 every code is 0); other scales, and blocks with an infinity, divide.
__device__ __forceinline__ void divide16_neg(const F2 (&x)[8], float s, bool finite, float (&y)[16]) {
  if (finite && s >= 8.673617379884035e-19f && s <= 1.152921504606847e18f) {
    const float inv = __frcp_rn(s);
    const F2 ni = f2(-inv, -inv), s2 = f2(s, s);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const F2 q = f2_mul(x[k], ni);
      f2_get(f2_fma(f2_fma(q, s2, x[k]), ni, q), y[2 * k], y[2 * k + 1]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      f2_get(x[k], a, b);
      y[2 * k] = __fdiv_rn(a, -s);
      y[2 * k + 1] = __fdiv_rn(b, -s);
    }
  }
}
// 16 values -> e4m3 codes.
__device__ __forceinline__ uint4 codes16(const float (&y)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2_rn_sat(y[4 * i], y[4 * i + 1]) | (e4m3x2_rn_sat(y[4 * i + 2], y[4 * i + 3]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 codes16_scaled(const F2 (&x)[8], float down) {
  const F2 d2 = f2(down, down);
  float y[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) f2_get(f2_mul(x[k], d2), y[2 * k], y[2 * k + 1]);
  return codes16(y);
}
// Eight negated fp32 values -> e2m1 codes (nearest even, saturating at 6),
// element i in nibble i; a zero code has no sign.
__device__ __forceinline__ uint32_t e2m1x8_neg(const float (&y)[16], int o) {
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
  return (w ^ 0x88888888u) & (nz * 15u);
}

// ------------------------------------------------------------ norm
// x * w / sqrt(mean x^2 + eps) over dims 0..511, each result its exact value
// rounded to fp32 (but for a few in a hundred off by one step): a relative
// error of 2^-23 in front of the quantization would move the codes of four
// elements in a million. The squares are summed as a tree and the lanes' sums
// with their rounding errors; the root's reciprocal carries a correction r1,
// and the products theirs. A row whose squares leave that no room (a mean below
// 2^-60 or a sum above 2^100, which fp32 may not hold at all) is taken again
// times a power of two, eps with it: the quotient is the same.
// With kStage `stage` receives lanes 28..31's 64 results and behind them what
// their rounding left off, for the rotation.
template <bool kStage>
__device__ __forceinline__ void norm_row(F2 (&v)[8], const F2 (&w)[8], float eps, int lane, float *stage) {
  float me, ml;
#pragma unroll 1
  for (bool again = false;; again = true) {   // (the lanes agree)
    F2 sq[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sq[k] = f2_fma(v[2 * k], v[2 * k], f2_mul(v[2 * k + 1], v[2 * k + 1]));
    float s0, s1;
    f2_get(f2_add(f2_add(sq[0], sq[1]), f2_add(sq[2], sq[3])), s0, s1);
    float ss = s0 + s1, sl = 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, ss, off), ol = __shfl_xor_sync(0xffffffffu, sl, off);
      const float t = ss + o, z = t - ss;          // ss + o = t + the error of t
      sl += ol + ((ss - (t - z)) + (o - z));
      ss = t;
    }
    const float ms = ss * (1.0f / kD);
    me = ms + eps;
    const float mz = me - ms;
    ml = fmaf(sl, 1.0f / kD, (ms - (me - mz)) + (eps - mz));
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
    // 2^e about the larger of the row and the root of eps
    int e = max((int)(m >> 23) - 127, -126);
    if (eps > 0.f) e = max(e, ((int)(__float_as_uint(eps) >> 23) - 126) >> 1);
    const float d = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
    eps = (eps * d) * d;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f2_mul(v[k], f2(d, d));
  }
  // 1 / sqrt(me + ml) = r0 + r1: an approximation and one Newton step, its
  // residual 1 - (me + ml) r0^2 by FMAs (none where me is 0 or infinite)
  const float r0 = rsqrtf(me);
  const float h = me * r0, hl = fmaf(me, r0, -h) + ml * r0;
  const float r1 = h == h ? 0.5f * r0 * fmaf(-hl, r0, fmaf(-h, r0, 1.0f)) : 0.f;
  const F2 a = f2(r0, r0), b = f2(r1, r1), na = f2(-r0, -r0), minus = f2(-1.f, -1.f);
  F2 lo[2];
#pragma unroll
  for (int k = 0; k < 8; ++k) {   // x w = q + ql
    const F2 q = f2_mul(v[k], w[k]), ql = f2_fma(v[k], w[k], f2_mul(q, minus));
    const F2 c = f2_fma(ql, a, f2_mul(q, b));
    v[k] = f2_fma(q, a, c);
    if constexpr (kStage) {
      lo[k & 1] = f2_fma(f2_fma(q, na, v[k]), minus, c);
      if ((k & 1) && lane >= 28) {
        ulonglong2 *d = reinterpret_cast<ulonglong2 *>(stage + 16 * (lane - 28) + 2 * k - 2);
        d[0] = make_ulonglong2(v[k - 1].v, v[k].v);
        d[16] = make_ulonglong2(lo[0].v, lo[1].v);
      }
    }
  }
}

// ------------------------------------------------------------ rotation
// (a, b) and its low part turned by (c, s): (a c - b s, b c + a s), nearly
// always the exact values rounded to fp32: the products' and the sums' rounding
// errors are added at the end (Dekker, "A floating-point technique for extending
// the available precision", 1971, with the products' errors by FMAs). In plain
// fp32 one bf16 value in 80000 behind it fell on the other side of a tie. Zeros
// keep their sign, infinities stay.
__device__ __forceinline__ void turn(float &a, float &b, F2 low, float c, float s) {
  float al, bl, t0, t1, d0, d1;
  f2_get(low, al, bl);
  const F2 x = f2(a, b), y = f2(b, a), yl = f2(bl, al), c2 = f2(c, c), s2 = f2(-s, s), minus = f2(-1.f, -1.f);
  const F2 p = f2_mul(x, c2), q = f2_mul(y, s2), t = f2_add(p, q);
  const F2 z = f2_fma(p, minus, t), u = f2_fma(z, minus, t);                          // t - p, t - (t - p)
  const F2 e = f2_add(f2_fma(u, minus, p), f2_fma(z, minus, q));                      // p + q - t
  const F2 ep = f2_fma(x, c2, f2_mul(p, minus)), eq = f2_fma(y, s2, f2_mul(q, minus));
  f2_get(f2_fma(low, c2, f2_fma(yl, s2, f2_add(e, f2_add(ep, eq)))), d0, d1);
  f2_get(t, t0, t1);
  a = d0 != 0.f && fabsf(t0) < INFINITY ? t0 + d0 : t0;
  b = d1 != 0.f && fabsf(t1) < INFINITY ? t1 + d1 : t1;
}

// ------------------------------------------------------------ write
// x -> (norm) -> (rotation) -> codes and scales, all in fp32 from the loaded
// values to the codes: nothing is rounded to 16 bits in between. A warp's next
// row is loaded before its present one is worked on. The rotation takes a pair
// per lane, through shared memory, so that its exact arithmetic is the work of
// 32 lanes and not of the 4 that hold the last 64 dims: 65536 normed MODEL1 rows
// take 35 us, 33 with a rotation in plain fp32 in those 4. Without a table none
// of it is compiled in (65536 plain fp8 rows 17 us, 22 with it skipped).
template <int FMT, int TY, bool kRope>
__global__ void __launch_bounds__(32 * kCacheWarps, 5) cache_write_kernel(CacheParams p) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kCacheWarps;
  const char *src = static_cast<const char *>(p.src);
  const int64_t stride = p.stride * kTypeBytes<TY>;
  const bool wide = ((reinterpret_cast<uintptr_t>(src) | (uintptr_t)stride) & 31u) == 0;
  F2 w[8];
  if (p.norm_w) {
    const float4 *w4 = reinterpret_cast<const float4 *>(p.norm_w) + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = __ldg(w4 + k);
      w[2 * k] = f2(x.x, x.y);
      w[2 * k + 1] = f2(x.z, x.w);
    }
  }
  // A row's last 64 dims on their way to a pair per lane and back (V3.2 rows
  // hold theirs so already): values, then the norm's low parts.
  constexpr bool kStage = kRope && !kV32;
  __shared__ __align__(16) float rot_s[kStage ? kCacheWarps : 1][128];
  float *stage = rot_s[kStage ? threadIdx.x >> 5 : 0];
  // the lane's pair: dims k, 32 + k (NeoX) or 2 k, 2 k + 1 (GPT-J)
  const int pair = kV32 && !p.gptj ? (lane & 15) * 2 + (lane >> 4) : lane;
  const int ia = p.gptj ? 2 * pair : pair, ib = p.gptj ? 2 * pair + 1 : pair + 32;
  RowRaw<TY> next;
  int32_t next_sid = -1;
  int64_t next_pos = 0;
  auto fetch = [&](int64_t i) {
    if (i >= p.n) return;
    next_sid = __ldg(p.L.ids + i);
    if constexpr (kRope) next_pos = __ldg(p.positions + i);
    load_row<TY, kV32>(src + i * stride, lane, wide, next);
  };
  int64_t i = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  fetch(i);
#pragma unroll 1
  for (; i < p.n; i += step) {   // whole warps
    const RowRaw<TY> raw = next;
    const int32_t sid = next_sid;
    const int64_t pos = next_pos;
    fetch(i + step);
    if (sid < 0 || (int64_t)sid >= p.L.num_slots) continue;   // padding: nothing is written
    float co = 0.f, si = 0.f;
    if constexpr (kRope) {
      if (pos < 0 || pos >= p.cs_rows) {   // outside the table: the row is not written
        if (p.status && lane == 0) report_status(p.status, DSA_ERR_INVALID_ARG);
        continue;
      }
      const float *cs = p.cos_sin + pos * 64;
      co = __ldg(cs + pair);
      si = __ldg(cs + 32 + pair);
    }
    F2 v[8];
    float t0 = 0.f, t1 = 0.f;
    unpack_row<TY, kV32>(raw, v, t0, t1);
    if constexpr (kStage) __syncwarp();   // the row before has left the stage
    if (p.norm_w) norm_row<kStage>(v, w, p.eps, lane, stage);
    // (a, b) -> (a cos - b sin, b cos + a sin) on the last 64 dims
    float ra = 0.f, rb = 0.f;
    if constexpr (kRope) {
      if constexpr (kV32) {     // dims 512 + 2 lane, + 1; NeoX partners sit 16 lanes away
        float a = t0, b = t1;
        if (!p.gptj) {          // lower lanes take the even pairs, upper lanes the odd ones
          const float x = __shfl_xor_sync(0xffffffffu, lane < 16 ? t1 : t0, 16);
          (lane < 16 ? b : a) = x;
        }
        turn(a, b, f2(0.f, 0.f), co, si);
        t0 = a;
        t1 = b;
        if (!p.gptj) {
          const float x = __shfl_xor_sync(0xffffffffu, lane < 16 ? t1 : t0, 16);
          (lane < 16 ? t1 : t0) = x;
        }
      } else {
        if (!p.norm_w && lane >= 28) {
          ulonglong2 *d = reinterpret_cast<ulonglong2 *>(stage + 16 * (lane - 28));
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = make_ulonglong2(v[2 * k].v, v[2 * k + 1].v);
        }
        __syncwarp();
        ra = stage[ia];
        rb = stage[ib];
        turn(ra, rb, p.norm_w ? f2(stage[64 + ia], stage[64 + ib]) : f2(0.f, 0.f), co, si);
        if constexpr (FMT != DSA_REC_MODEL1_584) {
          stage[ia] = ra;
          stage[ib] = rb;
          __syncwarp();
          if (lane >= 28) {
            const ulonglong2 *d = reinterpret_cast<const ulonglong2 *>(stage + 16 * (lane - 28));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const ulonglong2 x = d[k];
              v[2 * k].v = x.x;
              v[2 * k + 1].v = x.y;
            }
          }
        }
      }
    }
    uint8_t *rec = const_cast<uint8_t *>(record_ptr(p.L, sid));
    if (kDebug && (rec < p.L.base || rec + p.L.rec > p.L.base + p.L.extent)) {
      if (p.status) report_status(p.status, DSA_ERR_BOUNDS);
      continue;
    }
    float x[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) f2_get(v[k], x[2 * k], x[2 * k + 1]);
    if constexpr (FMT == DSA_REC_FP8_528 || kV32) {
      const uint32_t m = block_amax<8>(x);
      const float s = __fdiv_rn(__uint_as_float(m), 448.0f);
      float y[16];
      divide16_neg(v, s > 0.f || s != s ? s : 1.0f, true, y);   // zero blocks divide by one
      const uint4 c = codes16(y);
      *reinterpret_cast<uint4 *>(rec + 16 * lane) =
          make_uint4(c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u);
      if ((lane & 7) == 0) *reinterpret_cast<float *>(rec + 512 + (lane >> 1)) = s;
      if constexpr (kV32) *reinterpret_cast<uint32_t *>(rec + 528 + 4 * lane) = bf16x2_bits(t0, t1);
    } else if constexpr (FMT == DSA_REC_FP8_528_UE8M0) {
      const uint32_t e = ue8m0_of(block_amax<2>(x));
      *reinterpret_cast<uint4 *>(rec + 16 * lane) = codes16_scaled(v, ue8m0_down(e));
      if ((lane & 1) == 0) rec[512 + (lane >> 1)] = (uint8_t)e;
    } else if constexpr (FMT == DSA_REC_MODEL1_584) {
      const uint32_t e = ue8m0_of(block_amax<4>(x));
      if (lane < 28) {         // 8-byte aligned records
        const uint4 c = codes16_scaled(v, ue8m0_down(e));
        uint2 *d = reinterpret_cast<uint2 *>(rec + 16 * lane);
        d[0] = make_uint2(c.x, c.y);
        d[1] = make_uint2(c.z, c.w);
        if ((lane & 3) == 0) rec[576 + (lane >> 2)] = (uint8_t)e;
      } else if constexpr (!kRope) {   // the bf16 part
        uint2 *d = reinterpret_cast<uint2 *>(rec + 448 + 32 * (lane - 28));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[k] = make_uint2(bf16x2_bits(x[4 * k], x[4 * k + 1]), bf16x2_bits(x[4 * k + 2], x[4 * k + 3]));
      }
      if constexpr (kRope) {   // the bf16 part, a pair per lane
        const uint32_t r = bf16x2_bits(ra, rb);
        if (p.gptj) {
          *reinterpret_cast<uint32_t *>(rec + 448 + 4 * lane) = r;
        } else {
          *reinterpret_cast<uint16_t *>(rec + 448 + 2 * lane) = (uint16_t)r;
          *reinterpret_cast<uint16_t *>(rec + 512 + 2 * lane) = (uint16_t)(r >> 16);
        }
      }
      if (lane == 28) rec[583] = 0;   // the unused byte
    } else {                   // NVFP4: a block is one lane's 16 dims
      const uint32_t m = block_amax<1>(x);
      const float a6 = fminf(__fdiv_rn(__uint_as_float(m), 6.0f), 448.0f);
      const uint32_t sb = m > 0x7F800000u ? 0x7Fu : (e4m3x2_rn_sat(a6, 0.f) & 0xFFu);
      uint2 c = make_uint2(0u, 0u);
      if (sb != 0u && sb != 0x7Fu) {
        float y[16];
        divide16_neg(v, e4m3_to_f32(sb), m < 0x7F800000u, y);
        c = make_uint2(e2m1x8_neg(y, 0), e2m1x8_neg(y, 8));
      }
      *reinterpret_cast<uint2 *>(rec + 8 * lane) = c;
      rec[256 + lane] = (uint8_t)sb;
    }
  }
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

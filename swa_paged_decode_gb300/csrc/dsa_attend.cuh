// dsa_attend.cuh -- the kernels behind dsa_prefix_run and dsa_chunk_run: records
// gathered once into f16 tile images, CTA pairs that attend 128 query rows to
// them, and the merge of rows whose keys were split over pairs. A shared-prefix
// call has one list for all rows; a chunk call (kChunk) has sequences, each with
// its list, its rows and the keys that its rows may see (dsa_chunk.cu).
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "dsa_chunk_index.cuh"
#include "dsa_host.cuh"
#include "dsa_records.cuh"

namespace dsa {

constexpr int kPfTile = 256;                   // keys per tile
constexpr int kPfGroup = 32;                   // keys that share an exponent
constexpr int kPfSpread = 5;                   // log2 spread of their magnitudes up to which they do
constexpr int kPfTop = 14;                     // the largest value's exponent in the f16 tile
// The row's reference m of its weights P = 2^(score + exponent - m) in f16: the
// largest one stands at 2^kPfLift, and m moves once one exceeds 2^kPfMove (f16
// ends at 2^16). Lifted, weights keep 11 bits down to 2^-21 of the largest and
// are off by 2^-32 of it below (half of f16's smallest step, 2^-25). With the
// largest at 2^0 keys of 2^-25 of its weight counted for nothing, a million of
// them 3 % of the row.
constexpr int kPfLift = 7;
constexpr int kPfMove = 15;
constexpr int kPfRange = 48;                   // exponents of the keys' magnitudes: -48..48
constexpr int32_t kPfNoKey = INT32_MAX;        // exponent of a key that is not kept
constexpr int32_t kPfZeroKey = -kPfRange - 1;  // of a key of zeros: any other key's will do
constexpr int32_t kPfMixed = INT32_MIN;        // group exponent: one per key instead
// Chunk: exponent of a key with an infinity, a NaN or an element of 2^49 or more
// (with the range's largest exponent f16 ends at 2^50). Its image holds zeros and
// its scores are NaN, so that rows that may not see it do not meet it as 0 * NaN. A
// multiple of 2^9: as an exponent field it reads 2^0.
constexpr int32_t kPfNanKey = 1 << 20;

struct PrefixParams {
  ListArgs L;                  // the cache; ids: the prefix list, lens: its length, width
  const __nv_bfloat16 *q;
  int64_t q_st, q_sh;
  const float *sink;
  const int64_t *positions;
  const float *cos_sin;
  int64_t cs_rows;
  int32_t gptj;
  float scale_log2;
  const __nv_bfloat16 *tail_out;   // [T, H, 512] state of the token's own list, or null
  const float *tail_lse;
  __nv_bfloat16 *out;
  float *lse;
  int32_t H, rows;             // heads; query rows T H
  int32_t R;                   // 128-row tiles
  int64_t halves;              // 128-key halves of the images
  int32_t C;                   // CTA pairs
  long long wait_budget;
  // workspace
  int32_t *status;
  int2 *info;                  // [groups] (exponent or kPfMixed, mask of kept keys)
  int32_t *key_e;              // [keys] exponent of each key
  uint8_t *image;              // [128 keys][64-dim block][8-key group][1 KiB]
  int2 *tile;                  // [R] (pair of the tile's first units, * 2, + 1 if not its first tile; of its last)
  float *part_lse;             // [C][2][128]
  float *part_o;               // [C][2][128][512]
  // checking build: the rows that out and lse, and the partials, may be touched in
  int64_t check_rows, check_parts;
};

// The checking build's bounds of the rows of out, lse and the tail, of the
// partials, and of the images' halves (two from this one on).
__device__ __forceinline__ bool row_ok(const PrefixParams &p, int64_t gr) {
  return dbg_ok(p.status, gr >= 0 && gr < p.check_rows, kDbgOut);
}
__device__ __forceinline__ bool part_ok(const PrefixParams &p, int64_t slot) {
  return dbg_ok(p.status, slot >= 0 && slot < p.check_parts, kDbgPartial);
}
__device__ __forceinline__ bool halves_ok(const PrefixParams &p, int64_t half) {
  return dbg_ok(p.status, half >= 0 && half + 2 <= p.halves, kDbgPartial);
}

// A chunk call: rows of several sequences, each over its own list and with its
// own range of it (dsa_chunk.cu). The gather leaves where the work is.
struct ChunkParams : PrefixParams {
  const int32_t *starts;       // [B + 1] first token of every sequence
  int32_t T, B;
  int32_t window;              // keys that a token sees, itself among them; 0: all before it
  int32_t seq_halves;          // halves of a sequence's images
  // workspace
  int4 *row_tile;              // [R][2] of each row tile: (first row, rows, units, -), (first unit's half, its first
                               // key's list position, list position of row g's token - g / H, -)
  int32_t *seq_tile;           // [B] first row tile of every sequence
  int2 *begin;                 // [C + 1] (row tile, unit of it) at which a pair begins; the last: (row tiles with units, 0)
  int32_t *n_merge, *merge;    // [R] the row tiles that pairs share, or that have no keys
};
template <bool kChunk>
using AttendParams = std::conditional_t<kChunk, ChunkParams, PrefixParams>;

// min(len, width) of the prefix list, and its key tiles
__device__ __forceinline__ int32_t prefix_tiles(const PrefixParams &p, int32_t &len) {
  len = list_limit(p.L, 0);
  return (len + kPfTile - 1) / kPfTile;
}
// Weights of a row's prefix state (normalized, lse) and of its tail state in
// the output, and the lse of both: M = the larger lse, den = e^{lse - M} +
// e^{lse' - M} (+ e^{z - M}); a state with lse = -inf weighs nothing.
struct RowWeights {
  float o, tail, lse;
};
__device__ __forceinline__ RowWeights row_weights(float lse, float lt, bool sink, float sk) {
  const float M = fmaxf(lse, lt);
  RowWeights w = {0.f, 0.f, -INFINITY};
  if (!(M > -INFINITY)) {
    if (lse != lse || lt != lt) w.o = w.tail = w.lse = __uint_as_float(0x7FC00000u);
    return w;
  }
  const float a = expf(lse - M), b = expf(lt - M), z = a + b;
  w.lse = M + logf(z);
  float den = z;
  if (sink) den = sk == INFINITY ? INFINITY : z + expf(sk - M);
  w.o = a / den;
  w.tail = b / den;
  return w;
}
// 4 dims of a row's output: o (weighted) + wt * tail (4 bf16 values), as bf16.
// A tail that weighs nothing does not count, whatever it holds.
__device__ __forceinline__ void store_out4(const PrefixParams &p, int64_t gr, int d, float4 o, float wt, uint2 t) {
  if (!row_ok(p, gr)) return;
  if (wt != 0.f) {
    o.x = fmaf(wt, bf16_bits_to_f32(t.x & 0xFFFFu), o.x);
    o.y = fmaf(wt, bf16_bits_to_f32(t.x >> 16), o.y);
    o.z = fmaf(wt, bf16_bits_to_f32(t.y & 0xFFFFu), o.z);
    o.w = fmaf(wt, bf16_bits_to_f32(t.y >> 16), o.w);
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
  *reinterpret_cast<uint2 *>(p.out + gr * kD + d) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// ------------------------------------------------------------ gather
// Whether the lane's share of a record holds a value that is not finite.
template <int FMT>
__device__ __forceinline__ bool share_not_finite(const RawRecord &r, int lane) {
  if constexpr (FMT == DSA_REC_NVFP4_288) return (r.s & 0x7Fu) == 0x7Fu;
  auto bf16_bad = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
  bool bad = false;
  if (FMT == DSA_REC_MODEL1_584 && lane >= 28) {
#pragma unroll
    for (int k = 0; k < 8; ++k) bad |= bf16_bad(r.w[k]);
    return bad;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) bad |= __vcmpeq4(r.w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
  if constexpr (FMT == DSA_REC_FP8_528 || FMT == DSA_REC_V32_656) bad |= (r.s & 0x7F800000u) == 0x7F800000u;
  else bad |= (r.s & 0xFFu) == 0xFFu;
  if constexpr (FMT == DSA_REC_V32_656) bad |= bf16_bad(r.t);
  return bad;
}

// 32 records (a group) of a list of `len` into the images: positions key0 .. of
// the list become group `group`. The warp's 4 slots come in lanes 0..3; e_s is
// shared scratch.
template <int FMT, bool kChunk>
__device__ __forceinline__ void gather_group(const PrefixParams &p, int32_t slot, int32_t key0, int32_t len, int64_t group,
                                             int32_t (&e_s)[kPfGroup]) {
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  constexpr int kDB = kV32 ? 9 : 8;   // 64-dim blocks of a key
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // 4 keys per warp, their loads in flight together and kept as loaded until
  // the 32 keys' exponent is known
  RawRecord raw[4];
  bool ok[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t r = key0 + 4 * warp + i;
    const int32_t sid = __shfl_sync(0xffffffffu, slot, i);
    ok[i] = slot_valid(p.L, r, len, sid);
    const uint8_t *rec = record_ptr(p.L, ok[i] ? sid : 0);
    if (ok[i]) ok[i] = dbg_ok(p.status, rec >= p.L.base && rec + p.L.rec <= p.L.base + p.L.extent, kDbgRecord);
    if (ok[i]) load_record<FMT>(rec, lane, raw[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = __reduce_max_sync(0xffffffffu, ok[i] ? record_exponent<FMT>(raw[i], lane) : 0);
    int share = !ok[i] ? kPfNoKey : e == kZeroShare ? kPfZeroKey : min(max(e, -kPfRange), kPfRange);
    if constexpr (kChunk) {
      bool bad = ok[i] && share_not_finite<FMT>(raw[i], lane);
      if (ok[i] && e > kPfRange) {   // by its scale; its codes may be small (the warp agrees)
        float v[16], t0 = 0.f, t1 = 0.f;
        expand_record<FMT>(raw[i], lane, v, t0, t1);
        float most = fmaxf(fabsf(t0), fabsf(t1));
#pragma unroll
        for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(v[k]));
        bad |= most >= 562949953421312.f;   // 2^49
      }
      if (__any_sync(0xffffffffu, bad)) share = kPfNanKey;
    }
    if (lane == 0) e_s[4 * warp + i] = share;
  }
  __syncthreads();
  const int raw_e = e_s[lane], my = max(raw_e, -kPfRange);   // lane's key of the 32
  const bool kept = raw_e != kPfNoKey;
  const bool nan_key = kChunk && raw_e == kPfNanKey, usual = kept && !nan_key;
  const int hi = __reduce_max_sync(0xffffffffu, usual ? my : -kPfRange);
  const int lo = __reduce_min_sync(0xffffffffu, usual && raw_e != kPfZeroKey ? my : kPfRange);
  const uint32_t mask = __ballot_sync(0xffffffffu, kept);
  // (no key but zeros: hi = -kPfRange, lo = kPfRange)
  const bool mixed = hi - lo > kPfSpread || (kChunk && __any_sync(0xffffffffu, nan_key));
  if (warp == 0) {
    p.key_e[group * kPfGroup + lane] = nan_key ? kPfNanKey : (usual && mixed ? my : hi) - kPfTop;
    if (lane == 0) p.info[group] = make_int2(mixed ? kPfMixed : hi - kPfTop, (int)mask);
  }
  // image: key r of the tile in row r % 8 of 8-key group r / 8, 16-byte
  // chunk c of its 128 bytes at c ^ (r % 8)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (int)(group & 3) * kPfGroup + 4 * warp + i;   // of the half's 128 keys
    const int es = e_s[4 * warp + i];
    const bool zeros = kChunk && es == kPfNanKey;
    const int E = ((mixed && es != kPfNoKey && !zeros) ? max(es, -kPfRange) : hi) - kPfTop;
    const float down = __uint_as_float((uint32_t)(127 - E) << 23);
    const int g = r >> 3, x = r & 7;
    uint8_t *base = p.image + (group >> 2) * (kDB * 16384) + g * 1024 + x * 128;
    float v[16], t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = 0.f;
    if (ok[i] && !zeros) expand_record<FMT>(raw[i], lane, v, t0, t1);
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = tc::pack_f16x2(v[2 * k] * down, v[2 * k + 1] * down);
    // the lane's chunks c and c + 1 (c even) share a 32-byte sector, in either
    // order: one store of it (65536 MODEL1 records: 21 us, 28 with two stores,
    // each of half a sector)
    const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
    tc::stg_v8(base + (lane >> 2) * 16384 + (((2 * (lane & 3)) ^ (x & 6)) << 4), (x & 1) ? b : a, (x & 1) ? a : b);
    if constexpr (kV32)
      *reinterpret_cast<uint32_t *>(base + 8 * 16384 + (((lane >> 2) ^ x) << 4) + 4 * (lane & 3)) =
          tc::pack_f16x2(t0 * down, t1 * down);
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) prefix_gather_kernel(PrefixParams p) {
  __shared__ int32_t e_s[kPfGroup];
  // (the checking build clears the word before this launch instead)
  if (!kDebug && blockIdx.x == 0 && threadIdx.x == 0) *p.status = DSA_OK;
  pdl_launch_dependents();
  int32_t len;
  const int32_t tiles = prefix_tiles(p, len);
  const int32_t key0 = blockIdx.x * kPfGroup;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (loaded along with the length)
  int32_t slot = -1;
  if (lane < 4 && key0 + 4 * warp + lane < p.L.width) slot = __ldg(p.L.ids + key0 + 4 * warp + lane);
  if (key0 >= tiles * kPfTile || !halves_ok(p, key0 / kPfTile * 2)) return;   // (whole blocks)
  gather_group<FMT, false>(p, slot, key0, len, blockIdx.x, e_s);
}

// ------------------------------------------------------------ attend
// A pair of CTAs works on 128 query rows x 256 keys at a time:
//   S[128, 256] = Q . K^T   M = 128 over the pair (64 query rows in each
//       CTA), N = 256 keys (128 keys' rows of the operand in each CTA);
//   O[128, 512] += P . V    two N = 256 halves, 128 dims of each in either
//       CTA's shared memory; the accumulator takes 256 of the 512 TMEM
//       columns, S twice 128.
// One CTA alone cannot hold this: O for 128 rows fills all of its TMEM. In
// the pair's layout lane l of CTA r holds row 64 r + l % 64, and the upper
// half of each product's columns sits in lanes 64..127. (N = 128 for S, the
// largest that a 128-key tile allows, runs at half the rate: measured 62
// cycles per instruction of 128 x 128 x 16 against 71 for 128 x 256 x 16.)
//
// K and V of a unit come as 16 KiB chunks of the tile images, 128 keys x 64
// dims each (the same bytes read K-major as K and MN-major as V), one copy a
// chunk, through one ring in the order of their use: QK of unit i + 1 is
// issued before PV of unit i, so the softmax of a unit overlaps the products
// around it. V goes by two chunks (the 128 dims of an N = 256 half).
//
// Roles: warps 0-7 softmax (a row is held by 4 threads, 64 keys each), Q
// staging and the epilogue; warp 8 of the leader issues the MMAs; warps 9-11
// copy. Warp 8 runs its loop converged, one elected lane issuing: with uniform
// operands an instruction goes out in fewer cycles than the tensor core takes
// for it. Every wait is bounded as in the decode kernel.
//
// What bounds it: the products' shared-memory operands and the issue of a
// chunk every 270 cycles. 16384 rows x 16384 keys (550 GFLOP), gather and merge
// included: 326 to 335 us for one call alone, by the box (1640 to 1690 TFLOP/s of
// 1918); 313 us without the copies, measured at 342.
// The steps there, calls alone: N = 128 tiles with a relay of the chunks' arrival
// 1272; arrivals released at CTA scope 914;
// N = 256, one copy a chunk, converged issue 561; three copying warps and
// single-test waits 438; merge and gather 413; copies that complete on the
// leader's barrier 380; Q staging, epilogue, merge and ranges 348; tails
// prefetched 342; the rotation a pair per lane, rows out by bulk copies 335;
// queries' pieces over all banks 328. Two pairs that share their key copies by
// multicast were no faster (L2 gives 11 TB/s) and leave 4 of 76 pairs without a
// place. Few rows are latency: 32 rows x 512 keys take 15 us (gather 2.3, set-up
// and Q 4, a unit 5, epilogue 2, merge 2).
constexpr int kPfThreads = 384;
constexpr int kPfCopyWarps = 3;
constexpr long long kPfWait = 4000000000ll;   // SM cycles (~2 s) per wait
constexpr long long kPfCopyWait = 20000000ll; // ~10 ms: copies in flight after a timeout

template <bool V32>
struct PfCfg {
  static constexpr int kDB = V32 ? 9 : 8;
  static constexpr int kKChunks = V32 ? 10 : 8;   // V3.2: the tenth is empty, so that V starts on an even slot
  static constexpr int kSlots = V32 ? 6 : 8;      // even: the two chunks of a V half lie side by side
  static constexpr uint32_t kQ = 0;                          // [kDB][64 rows x 64 dims] f16
  static constexpr uint32_t kP = kDB * 8192;                 // [4][64 rows x 64 keys] f16
  static constexpr uint32_t kRing = kP + 32768;
  static constexpr uint32_t kRed = kRing + kSlots * 16384;   // [4][64] f32
  static constexpr uint32_t kHeadF = kRed + 1024;            // [64] f32: scale log2(e) 2^e of a row
  static constexpr uint32_t kRowW = kHeadF + 256;            // [2][64] f32 epilogue weights
  static constexpr uint32_t kMisc = kRowW + 512;
  static constexpr uint32_t kBytes = kMisc + 512;
  static constexpr uint32_t kSmem = kBytes + 1024 > 232448u ? 232448u : kBytes + 1024;
  static constexpr uint32_t kIdQK = tc::idesc_f16(128, 256, false, false);
  static constexpr uint32_t kIdPV = tc::idesc_f16(128, 256, false, true);
  static constexpr uint32_t kColO = 0, kColS = 256;
  // barriers (8 bytes each) in the misc area
  static constexpr int kFull = 0, kEmpty = kSlots, kSFull = 2 * kSlots,
                       kPFull = kSFull + 2, kPvDone = kPFull + 1, kQReady = kPvDone + 1,
                       kDrain = kQReady + 1, kBars = kDrain + 1;
  static constexpr uint32_t kAbort = 8 * kBars, kTmem = kAbort + 4;
  static_assert(kTmem + 4 <= 512, "misc area");
  static_assert(kBytes <= 232448u, "shared memory layout exceeds 227 KiB");
};

// The segments of a pair's range, in order.
template <bool kChunk>
struct Walk;
template <>
struct Walk<false> {
  int64_t u, u1;
  int32_t KT, rows;
  __device__ __forceinline__ Walk(const PrefixParams &p, int pair) : rows(p.rows) {
    int32_t len;
    KT = prefix_tiles(p, len);
    const Schedule sched = make_schedule(p.R, KT, p.C);
    u = sched.begin(pair);
    u1 = sched.begin(pair + 1);   // (a pair may have no units)
  }
  __device__ __forceinline__ bool empty() const { return u >= u1; }
  __device__ __forceinline__ bool next(TileRun &s) {
    if (u >= u1) return false;
    const int64_t qt = u / KT, kt = u - qt * KT, end = min((qt + 1) * KT, u1);
    s.qt = (int32_t)qt;
    s.g0 = qt * 128;
    s.n = (int32_t)min((int64_t)128, rows - s.g0);
    s.half = 2 * kt;
    s.units = (int32_t)(end - u);
    s.head = kt == 0;
    s.tail = end == (qt + 1) * KT;
    s.key0 = s.shift = 0;
    u = end;
    return true;
  }
  // rows of the next segment's tile (0: none)
  __device__ __forceinline__ int32_t peek(const TileRun &s, int64_t &g0) const {
    g0 = s.g0 + 128;
    return u < u1 ? (int32_t)min((int64_t)128, rows - g0) : 0;
  }
};
struct LoadRowTile {
  const int4 *tiles;
  __device__ __forceinline__ void operator()(int32_t t, RowTile &r) const {
    const int4 a = __ldcg(tiles + 2 * (int64_t)t), b = __ldcg(tiles + 2 * (int64_t)t + 1);
    r = {a.x, a.y, a.z, b.x, b.y, b.z};
  }
};
template <>
struct Walk<true> : TileWalk<LoadRowTile> {
  __device__ __forceinline__ Walk(const ChunkParams &p, int pair)
      : Walk(p, __ldcg(p.begin + pair), __ldcg(p.begin + pair + 1)) {}
  __device__ __forceinline__ Walk(const ChunkParams &p, int2 from, int2 to)
      : TileWalk<LoadRowTile>({p.row_tile}, from.x, from.y, to.x, to.y) {}
};

template <bool kV32, bool kChunk>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPfThreads, 1)
    prefix_attend_kernel(AttendParams<kChunk> p, const __grid_constant__ CUtensorMap image) {
  using Cfg = PfCfg<kV32>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = tc::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sbase = raw_base + pad;
  const uint32_t q_base = sbase + Cfg::kQ, p_base = sbase + Cfg::kP, ring = sbase + Cfg::kRing;
  float *red_s = reinterpret_cast<float *>(smem + Cfg::kRed);
  float *headf_s = reinterpret_cast<float *>(smem + Cfg::kHeadF);
  float *roww_s = reinterpret_cast<float *>(smem + Cfg::kRowW);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kMisc);
  volatile int32_t *abort_s = reinterpret_cast<volatile int32_t *>(smem + Cfg::kMisc + Cfg::kAbort);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kMisc + Cfg::kTmem);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t side = tc::cluster_rank();   // CTA of its pair; 0 leads
  const int pair = blockIdx.x >> 1;
  if (pad + Cfg::kBytes > Cfg::kSmem) {       // every CTA alike
    if (tid == 0) report_status(p.status, DSA_ERR_UNSUPPORTED);
    return;
  }
  if (warp == 0) tc::tmem_alloc_pair(tmem_slot, 512);
  if (tid == 32) {
    for (int b = 0; b < Cfg::kBars; ++b)
      tc::mbar_init(&bars[b], (b == Cfg::kPFull || b == Cfg::kQReady) ? 16u : 1u);
    tc::fence_mbar_init();
    *abort_s = 0;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (kChunk) pdl_wait_primary();   // (the pairs' ranges)
  Walk<kChunk> walk(p, pair);

  // Bounded wait on a phase, after any timeout of the CTA a mere test; false:
  // given up. What is there already passes in one test: at a chunk every 270
  // cycles the issuing and copying threads have no time for more.
  auto wait = [&](int b, uint32_t phase) -> bool {
    if (tc::mbar_test_wait(&bars[b], phase)) return true;
    if (*abort_s) return false;
    const long long budget = p.wait_budget > 0 ? p.wait_budget : kPfWait;
    if (tc::mbar_wait(&bars[b], phase, budget)) return true;
    if (!*abort_s) {
      *abort_s = 1;
      report_status(p.status, DSA_ERR_TIMEOUT);
    }
    return false;
  };
  const uint32_t lead_pfull = tc::mapa(tc::smem_u32(&bars[Cfg::kPFull]), 0);
  const uint32_t lead_qready = tc::mapa(tc::smem_u32(&bars[Cfg::kQReady]), 0);

  if (warp >= 9) {
    // ======================================================== copies
    // The warps take turns, chunk by chunk: one thread issues a chunk in
    // about 300 cycles, too slow for a chunk every 270. The bytes of both
    // CTAs complete on the leader's barrier, which its own warps arm.
    if (lane == 0) {
      if constexpr (!kChunk) pdl_wait_primary();   // the images are complete
      uint32_t slot = 0, ph = 1;   // the first round finds every slot empty
      int turn = warp - 9;         // 0: this warp's
      bool ok = true;
      uint32_t filled = 0, fill_ph = 0;   // slots this warp has filled, and the phase of their latest fill
      const uint32_t full0 = tc::mapa(tc::smem_u32(&bars[Cfg::kFull]), 0);
      constexpr int32_t kHalf = Cfg::kDB * 32;   // map rows (512 bytes) of 128 keys; a chunk has 32
      const int64_t map_rows = p.halves * kHalf;
      auto chunk = [&](int32_t y, bool some) {
        if (some) dbg_ok(p.status, y >= 0 && y + 32 <= map_rows, kDbgSmemKv);   // (the map gives zeros past its end)
        if (turn == 0) {
          turn = kPfCopyWarps;
          ok = wait(Cfg::kEmpty + slot, ph);
          if (!ok) return;
          if (side == 0) {
            tc::mbar_expect_tx(&bars[Cfg::kFull + slot], some ? 32768u : 0u);
            filled |= 1u << slot;
            fill_ph = (fill_ph & ~(1u << slot)) | ((ph ^ 1u) << slot);
          }
          if (some) tc::tma_load_pair(ring + slot * 16384, &image, 0, y, full0 + 8 * slot);
        }
        --turn;
        if (++slot == Cfg::kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      };
      auto load_k = [&](int64_t half) {   // this CTA's 128 keys, 64 dims a chunk
        const int32_t y = (int32_t)(half + side) * kHalf;
#pragma unroll 1
        for (int c = 0; c < Cfg::kKChunks && ok; ++c) chunk(y + c * 32, c < Cfg::kDB);
      };
      auto load_v = [&](int64_t half) {   // 128 keys, then the others; dims 128 side .. of either half
        const int32_t y = (int32_t)half * kHalf + 64 * side;
#pragma unroll 1
        for (int c = 0; c < 8 && ok; ++c) chunk(y + (c >> 2) * kHalf + ((c >> 1) & 1) * 128 + (c & 1) * 32, true);
      };
      TileRun seg;
      while (ok && walk.next(seg)) {
        load_k(seg.half);
        for (int32_t i = 0; i < seg.units && ok; ++i) {
          if (i + 1 < seg.units) load_k(seg.half + 2 * (i + 1));
          if (ok) load_v(seg.half + 2 * i);
        }
      }
      // The slots' last releases have arrived: no commit of the leader
      // reaches this CTA's barriers after its end. (A slot that was never
      // filled passes at once.)
      for (int k = 0; k < Cfg::kSlots && ok; ++k) {
        ok = wait(Cfg::kEmpty + slot, ph);
        if (++slot == Cfg::kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
      // After a timeout no copy may be in flight into shared memory when the
      // pair ends: the leader waits for the chunks it has armed (both CTAs'
      // bytes, unless the other gave up before); then either thread lets a
      // thousand times the latency of a copy pass.
      if (!ok) {
        for (int k = 0; k < Cfg::kSlots; ++k)
          if ((filled >> k) & 1u) tc::mbar_wait(&bars[Cfg::kFull + k], (fill_ph >> k) & 1u, kPfCopyWait);
        const long long t0 = clock64();
        while (clock64() - t0 < kPfCopyWait / 10) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    uint32_t slot = 0, ph = 0;
    auto next = [&]() {
      if (++slot == Cfg::kSlots) {
        slot = 0;
        ph ^= 1u;
      }
    };
    if (side == 0) {
      // ====================================================== MMA issue
      constexpr uint16_t kBoth = 3;
      constexpr uint32_t kHi = tc::sdesc_hi(1024, tc::kSwz128);
      const uint32_t dq = tc::sdesc_lo(q_base, 16), dp = tc::sdesc_lo(p_base, 16);
      const uint32_t dk0 = tc::sdesc_lo(ring, 16), dv0 = tc::sdesc_lo(ring, 16384);
      uint32_t ph_p = 0, ph_q = 0, nqk = 0;
      bool issued = false;
      auto here = [&](bool x) { return __all_sync(0xffffffffu, x); };
      auto qk = [&]() -> bool {
        const uint32_t d = tmem + Cfg::kColS + (nqk & 1u) * 128u;
#pragma unroll
        for (int c = 0; c < Cfg::kKChunks; ++c) {
          if (!here(wait(Cfg::kFull + slot, ph))) return false;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint32_t dk = dk0 + slot * 1024u;
            if (c < Cfg::kDB) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_f16_pair(d, dq + ((c * 8192 + ks * 32) >> 4), dk + ((ks * 32) >> 4), kHi, Cfg::kIdQK,
                                 (c | ks) ? 1u : 0u);
            }
            tc::mma_commit_to(&bars[Cfg::kEmpty + slot], kBoth);
            if (c == Cfg::kKChunks - 1) tc::mma_commit_to(&bars[Cfg::kSFull + (nqk & 1u)], kBoth);
          }
          __syncwarp();
          next();
        }
        ++nqk;
        return true;
      };
      auto pv = [&](bool first) -> bool {
        if (!here(wait(Cfg::kPFull, ph_p))) return false;
        ph_p ^= 1u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {    // (128 keys, half of the dims)
          if (!here(wait(Cfg::kFull + slot, ph) && wait(Cfg::kFull + slot + 1, ph))) return false;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint32_t dv = dv0 + slot * 1024u, d = tmem + Cfg::kColO + 128 * (c & 1);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc::mma_f16_pair(d, dp + (((c >> 1) * 16384 + (ks >> 2) * 8192 + (ks & 3) * 32) >> 4),
                               dv + ((ks * 2048) >> 4), kHi, Cfg::kIdPV, (c >> 1) | ks ? 1u : (first ? 0u : 1u));
            tc::mma_commit_to(&bars[Cfg::kEmpty + slot], kBoth);
            tc::mma_commit_to(&bars[Cfg::kEmpty + slot + 1], kBoth);
            if (c == 3) tc::mma_commit_to(&bars[Cfg::kPvDone], kBoth);
          }
          __syncwarp();
          next();
          next();
        }
        return true;
      };
      bool ok = true;
      TileRun seg;
      while (ok && walk.next(seg)) {
        ok = here(wait(Cfg::kQReady, ph_q));
        ph_q ^= 1u;
        if (ok) {
          issued = true;   // (qk may give up after some of its products)
          ok = qk();
        }
        for (int32_t i = 0; i < seg.units && ok; ++i) {
          if (i + 1 < seg.units) ok = qk();
          if (ok) ok = pv(i == 0);
        }
      }
      // MMAs issued before a timeout end before TMEM is freed
      if (issued && !ok && tc::elect_one()) {
        tc::mma_commit_one(&bars[Cfg::kDrain]);
        tc::mbar_wait(&bars[Cfg::kDrain], 0u, kPfWait);
      }
    }
    __syncwarp();
  } else {
    // ======================================================== softmax
    const int q4 = warp & 3, half = warp >> 2;
    const int lr = 32 * q4 + lane;             // TMEM lane
    const int row = lr & 63, kh = lr >> 6;     // query row of this CTA, half of the tile's keys
    const int part = 2 * kh + half;            // this thread's 64 keys of the tile: two 32-key groups
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16);
    auto sm_bar = [&]() { asm volatile("barrier.sync 1, 256;" ::: "memory"); };
    auto sm_bar_or = [&](bool x) {
      int r;
      asm volatile(
          "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\t"
          "barrier.red.or.pred b, 1, 256, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
          : "=r"(r) : "r"((int)x) : "memory");
      return r != 0;
    };
    // 16 bytes into the Q tile (also the epilogue's staging area)
    auto st_q = [&](uint32_t off, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      if (dbg_ok(p.status, off + 16u <= Cfg::kP - Cfg::kQ, kDbgSmemQ)) tc::st_shared_v4(q_base + off, a, b, c, d);
    };
    bool bad_pos = false;   // reported once the gather, which clears the status word, is done
    // Row lane % 8 of the warp's 8 of a tile: its queries, its table row (found
    // before the epilogue of the tile before: its position is a load of its own).
    const __nv_bfloat16 *qp = nullptr;
    const float *cp = p.cos_sin;
    auto find_rows = [&](int64_t g0, int32_t rows) {
      const uint32_t in = side * 64u + 8u * warp + (lane & 7), gl = (uint32_t)g0 + in;
      qp = nullptr;
      cp = p.cos_sin;
      if ((int32_t)in < rows) {
        const uint32_t t = gl / (uint32_t)p.H, h = gl - t * (uint32_t)p.H;
        if (dbg_ok(p.status, (int64_t)t * p.H + h < (int64_t)p.rows, kDbgQ))
          qp = p.q + (int64_t)t * p.q_st + (int64_t)h * p.q_sh;
        if (cp) {
          const int64_t pos = __ldg(p.positions + t);
          if (pos >= 0 && pos < p.cs_rows) cp += pos * 64;
          else bad_pos = true;   // outside the table: flag, row 0
        }
      }
    };
    bool leaving = false;   // rows of the tile before are on their way out of the Q tile
    // Q rows of this CTA -> f16 K-major tile: RoPE in fp32, times a power of
    // two per row so that its largest unrotated magnitude lies in [1, 2) (a
    // rotation adds half a bit at most). A warp takes 8 rows, 2 or 4 at a time
    // with the next ones in flight; the loop stays rolled and a row's address is
    // found once, by a lane of its own: this code runs once per 128 rows, so
    // its size is its time (8 rows unrolled took 9700 cycles, 700 a row). A lane
    // takes the 16-byte pieces l and 32 + l: 8 lanes fill the 128 bytes of a row of
    // the image, all banks (with pieces 2 l and 2 l + 1 half of them twice: 5400
    // cycles a tile against 4500).
    auto stage_q = [&]() {
      const bool rope = p.cos_sin != nullptr;
      // The rotation takes a pair per lane, through the P tile, which no product
      // reads now (in the four lanes that hold the last 64 dims it was a third of
      // the instructions).
      const int ia = p.gptj ? 2 * lane : lane, ib = p.gptj ? 2 * lane + 1 : lane + 32;
      float *turn_s = reinterpret_cast<float *>(smem + Cfg::kP) + 256 * warp;   // [rows at a time][64]
      constexpr int kIn = kChunk ? 4 : 2;   // rows at a time (chunks: many short tiles)
      uint4 na[kIn], nb[kIn], nc[kIn];
      float nco[kIn], nsi[kIn];
      auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          const uint4 *r = reinterpret_cast<const uint4 *>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(qp), i0 + i));
          na[i] = nb[i] = nc[i] = make_uint4(0, 0, 0, 0);
          if (r) {
            na[i] = __ldg(r + lane);
            nb[i] = __ldg(r + 32 + lane);
            if constexpr (kV32)
              if (lane < 8) nc[i] = __ldg(r + 64 + lane);   // dims 512 + 8 lane ..
          }
          if (rope) {
            const float *c = reinterpret_cast<const float *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(cp), i0 + i));
            const int64_t at = c - p.cos_sin;
            if (dbg_ok(p.status, at >= 0 && at + 64 <= p.cs_rows * 64, kDbgTable)) {
              nco[i] = __ldg(c + lane);
              nsi[i] = __ldg(c + 32 + lane);
            }
          }
        }
      };
      fetch(0);
      if (leaving) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        sm_bar();
        leaving = false;
      }
#pragma unroll 1
      for (int i0 = 0; i0 < 8; i0 += kIn) {
        uint4 qa[kIn], qb[kIn], qc[kIn];
        float co[kIn], si[kIn];
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          qa[i] = na[i];
          qb[i] = nb[i];
          qc[i] = nc[i];
          co[i] = nco[i];
          si[i] = nsi[i];
        }
        if (i0 + kIn < 8) fetch(i0 + kIn);
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          const int r = 8 * warp + i0 + i;
          const uint32_t w[8] = {qa[i].x, qa[i].y, qa[i].z, qa[i].w, qb[i].x, qb[i].y, qb[i].z, qb[i].w};
          const uint32_t wc[4] = {qc[i].x, qc[i].y, qc[i].z, qc[i].w};
          // largest magnitude, from the bf16 bits
          uint32_t mb = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) mb = __vmaxu2(mb, w[k] & 0x7FFF7FFFu);
          if constexpr (kV32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mb = __vmaxu2(mb, wc[k] & 0x7FFF7FFFu);
          }
          mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
          int e = mb ? (int)(mb >> 7) - 127 : 0;
          e = e < -126 ? -126 : (e > 126 ? 126 : e);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          if (lane == 0) headf_s[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
          float v[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[2 * k] = bf16_bits_to_f32(w[k] & 0xFFFFu) * down;
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * down;
          }
          const uint32_t ro = (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u;
          const uint32_t at = (uint32_t)(lane >> 3) * 8192u + ro + (((lane & 7) ^ (r & 7)) << 4);
          uint32_t f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = tc::pack_f16x2(v[2 * k], v[2 * k + 1]);
          st_q(at, f[0], f[1], f[2], f[3]);
          if (rope && lane >= 24) {
            float4 *d = reinterpret_cast<float4 *>(turn_s + 64 * i + 8 * (lane - 24));
            d[0] = make_float4(v[8], v[9], v[10], v[11]);
            d[1] = make_float4(v[12], v[13], v[14], v[15]);
          } else {
            st_q(at + 4 * 8192u, f[4], f[5], f[6], f[7]);
          }
          if constexpr (kV32) {
            if (lane < 8) {
              uint32_t fc[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                fc[k] = tc::pack_f16x2(bf16_bits_to_f32(wc[k] & 0xFFFFu) * down, bf16_bits_to_f32(wc[k] >> 16) * down);
              st_q(8 * 8192 + ro + ((lane ^ (r & 7)) << 4), fc[0], fc[1], fc[2], fc[3]);
            }
          }
        }
        if (rope) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kIn; ++i) {
            const int r = 8 * warp + i0 + i;
            const float x1 = turn_s[64 * i + ia], x2 = turn_s[64 * i + ib];
            const uint32_t f = tc::pack_f16x2(fmaf(x1, co[i], -(x2 * si[i])), fmaf(x2, co[i], x1 * si[i]));
            uint8_t *q = smem + Cfg::kQ + 7 * 8192 + (r >> 3) * 1024 + (r & 7) * 128;
            uint8_t *qa = q + (((ia >> 3) ^ (r & 7)) << 4) + 2 * (ia & 7);
            if (p.gptj) {
              *reinterpret_cast<uint32_t *>(qa) = f;
            } else {
              *reinterpret_cast<uint16_t *>(qa) = (uint16_t)f;
              *reinterpret_cast<uint16_t *>(q + (((ib >> 3) ^ (r & 7)) << 4) + 2 * (ib & 7)) = (uint16_t)(f >> 16);
            }
          }
          __syncwarp();   // the stage is free again
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_remote(lead_qready);
    };

    if (walk.empty() && tid < 64 && part_ok(p, (int64_t)pair * 256 + side * 64 + tid))
      p.part_lse[(int64_t)pair * 256 + side * 64 + tid] = -INFINITY;
    uint32_t ph_s = 0, nqk = 0, ph_pv = 0;
    const uint32_t prow = p_base + part * 8192 + (uint32_t)(row >> 3) * 1024u + (uint32_t)(row & 7) * 128u;
    TileRun seg;
    for (bool begun = false; walk.next(seg); begun = true) {
      const int32_t late = begun ? 1 : 0;   // (a later tile than the pair's first)
      const int4 *info = reinterpret_cast<const int4 *>(p.info) + part;   // (exponent, mask) of two groups
      auto load_info = [&](int64_t half) { return halves_ok(p, half) ? __ldcg(info + half * 2) : make_int4(0, 0, 0, 0); };
      int4 inf = make_int4(0, 0, 0, 0);
      if (kChunk || begun) inf = load_info(seg.half);
      if (!begun) find_rows(seg.g0, seg.n);
      stage_q();
      if (!kChunk && !begun) {
        pdl_wait_primary();   // group records of the gather
        inf = load_info(seg.half);
      }
      if (bad_pos) report_status(p.status, DSA_ERR_INVALID_ARG);
      sm_bar();   // headf_s
      int64_t next_g0;
      if (const int32_t nn = walk.peek(seg, next_g0)) {   // the next tile's queries on their way to L2
        const int32_t in = side * 64 + 8 * warp + (lane & 7);
        const int64_t nr = next_g0 + in;
        if (in < nn) {
          const uint32_t t = (uint32_t)nr / (uint32_t)p.H, h = (uint32_t)nr - t * (uint32_t)p.H;
          const char *qr = reinterpret_cast<const char *>(p.q + (int64_t)t * p.q_st + (int64_t)h * p.q_sh);
          for (int b = 128 * (lane >> 3); b < Cfg::kDB * 128; b += 512)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(qr + b));
        }
      }
      const bool whole = seg.head && seg.tail;
      if (p.tail_out && whole) {   // and the tails that this one's epilogue adds
        for (int b = tid; b < 512; b += 256) {
          const int64_t gr = seg.g0 + side * 64 + (b >> 3);
          if ((int)side * 64 + (b >> 3) < seg.n)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.tail_out + gr * kD + 64 * (b & 7)));
        }
      }
      const float hf = headf_s[row];
      float m = -1e30f, l = 0.f;
      // chunk: the row's own place among the keys of this thread, moved on with the units
      int32_t place = 0;
      if constexpr (kChunk) place = (int32_t)((uint32_t)(seg.g0 + side * 64 + row) / (uint32_t)p.H) + seg.shift - seg.key0 - 64 * part;
      for (int32_t i_u = 0; i_u < seg.units; ++i_u) {
        const int64_t half_u = seg.half + 2 * i_u;
        int4 cur = inf;
        if (i_u + 1 < seg.units) inf = load_info(half_u + 2);
        const bool mixed = cur.x == kPfMixed || cur.z == kPfMixed;   // one exponent per key
        bool full = ((uint32_t)cur.y & (uint32_t)cur.w) == 0xFFFFFFFFu;
        if constexpr (kChunk) {   // keys place - window + 1 .. place of the 64
          uint64_t seen = place >= 63 ? ~0ull : place < 0 ? 0ull : (2ull << place) - 1ull;
          if (p.window > 0 && place >= p.window) {
            const int32_t lo = place - p.window + 1;
            seen &= lo > 63 ? 0ull : ~((1ull << lo) - 1ull);
          }
          cur.y &= (int)(uint32_t)seen;
          cur.w &= (int)(uint32_t)(seen >> 32);
          full = __all_sync(0xffffffffu, full && seen == ~0ull);
          place -= kPfTile;
        }
        const int32_t *ke = p.key_e + half_u * 128 + part * 64;
        float x[64];
        // x = score in log2 units + exponent of the key - mm (-inf: not kept)
        auto load_t = [&](float mm) {
          const uint32_t c = tl + Cfg::kColS + (nqk & 1u) * 128u + half * 64;
          uint32_t r4[4][16];
          DSA_TMEM_LD16_NOWAIT(c, r4[0]);
          DSA_TMEM_LD16_NOWAIT(c + 16, r4[1]);
          DSA_TMEM_LD16_NOWAIT(c + 32, r4[2]);
          DSA_TMEM_LD16_NOWAIT(c + 48, r4[3]);
          DSA_TMEM_WAIT32(r4[0], r4[1]);
          DSA_TMEM_WAIT32(r4[2], r4[3]);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t(&ra)[16] = r4[2 * g], (&rb)[16] = r4[2 * g + 1];
            const int e = g ? cur.z : cur.x;
            if (!mixed) {
              const float a = hf * __uint_as_float((uint32_t)(127 + e) << 23), b = (float)e - mm;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[32 * g + i] = fmaf(__uint_as_float(ra[i]), a, b);
                x[32 * g + 16 + i] = fmaf(__uint_as_float(rb[i]), a, b);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int ei = __ldcg(ke + 32 * g + i);
                if (kChunk && ei == kPfNanKey) {
                  x[32 * g + i] = __uint_as_float(0x7FC00000u);
                  continue;
                }
                x[32 * g + i] = fmaf(__uint_as_float(i < 16 ? ra[i & 15] : rb[i & 15]),
                                     hf * __uint_as_float((uint32_t)(127 + ei) << 23), (float)ei - mm);
              }
            }
            if (!full) {
              const uint32_t mask = (uint32_t)(g ? cur.w : cur.y);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((mask >> i) & 1u)) x[32 * g + i] = -INFINITY;
            }
          }
        };
        wait(Cfg::kSFull + (nqk & 1u), ph_s);
        tc::tc_fence_after();
        // Scores against the running reference; where a row's exceed it by
        // kPfMove (or it has none yet: its scores stand alone) the references,
        // O and the sums of the whole CTA move.
        const bool unset = m < -1e29f;
        const float mm = unset ? 0.f : m;
        load_t(mm);
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < 64; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
        top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool moved = sm_bar_or(top[0] > (unset ? -INFINITY : (float)kPfMove));
        if (moved) {
          red_s[part * 64 + row] = top[0];
          sm_bar();
          const float tm = fmaxf(fmaxf(red_s[row], red_s[64 + row]), fmaxf(red_s[128 + row], red_s[192 + row]));
          const float mn = fmaxf(m, mm + tm - (float)kPfLift);
          const float f = tc::ex2(m - mn);   // 0 with the first kept key
          const float d = mn - mm;
          m = mn;
          l *= f;
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] -= d;
          if (i_u > 0) {   // (zero on a row without a key: 0 * 0)
            wait(Cfg::kPvDone, ph_pv);
            tc::tc_fence_after();
#pragma unroll 1
            for (int g = 0; g < 8; ++g) {
              const uint32_t ta = tl + Cfg::kColO + half * 128 + 16 * g;
              float o[16];
              tc::tmem_ld<16>(ta, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tc::tmem_st<16>(ta, o);
            }
          }
          sm_bar();   // red_s free again
        }
        // P = 2^x; the sums take P 2^-E = 2^(score - m)
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = tc::ex2(x[i]);
        if (!mixed) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i & 3] += x[32 * g + i];
            l = fmaf((s[0] + s[1]) + (s[2] + s[3]), __uint_as_float((uint32_t)(127 - (g ? cur.z : cur.x)) << 23), l);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) l = fmaf(x[i], __uint_as_float((uint32_t)(127 - __ldcg(ke + i)) << 23), l);
        }
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = tc::pack_f16x2(x[2 * i], x[2 * i + 1]);
        // P of the unit before has been read (a segment's first unit follows
        // an epilogue, which waited for that)
        if (i_u > 0) {
          if (!moved) wait(Cfg::kPvDone, ph_pv);
          ph_pv ^= 1u;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = prow + ((k ^ (row & 7)) << 4);
          if (dbg_ok(p.status, at >= p_base && at + 16u <= ring, kDbgSmemP))
            tc::st_shared_v4(at, pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        }
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(lead_pfull);
        ++nqk;
        if ((nqk & 1u) == 0) ph_s ^= 1u;
      }
      // ---- epilogue
      {   // (the next tile's rows, while the last products run)
        int64_t g;
        const int32_t n = walk.peek(seg, g);
        if (n) find_rows(g, n);
      }
      red_s[part * 64 + row] = l;
      const int64_t g0 = seg.g0 + side * 64;       // this CTA's first row
      const int32_t rows_here = seg.n - side * 64; // and how many it has of the tile's (none: <= 0)
      const int64_t ps = (2 * (int64_t)pair + late) * 128 + side * 64;
      if (side == 0 && tid == 0 && dbg_ok(p.status, seg.qt >= 0 && seg.qt < p.R, kDbgPartial)) {   // where the merge finds this tile
        if (seg.head) p.tile[seg.qt].x = 2 * pair + late;
        if (seg.tail) p.tile[seg.qt].y = pair;
      }
      sm_bar();
      if (tid < 64) {   // row tid: lane tid of the lower half holds it
        const int64_t gr = g0 + row;
        const float lt = (red_s[row] + red_s[64 + row]) + (red_s[128 + row] + red_s[192 + row]);
        // (a NaN among the scores or values stays one)
        const float lse = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
        float wo = lt == 0.f ? 0.f : 1.f / lt, wt = 0.f;
        if (row < rows_here) {
          if (whole) {
            const RowWeights w =
                row_weights(lse, p.tail_lse && row_ok(p, gr) ? p.tail_lse[gr] : -INFINITY, p.sink != nullptr,
                            p.sink ? __ldg(p.sink + (uint32_t)gr % (uint32_t)p.H) : 0.f);
            wo *= w.o;
            wt = w.tail;
            if (row_ok(p, gr)) p.lse[gr] = w.lse;
          } else if (part_ok(p, ps + row)) {
            p.part_lse[ps + row] = lse;
          }
        }
        roww_s[row] = wo;
        roww_s[64 + row] = wt;
      }
      wait(Cfg::kPvDone, ph_pv);
      ph_pv ^= 1u;
      tc::tc_fence_after();
      sm_bar();
      // O leaves in two passes of 256 dims (64 of each thread's 128) through
      // the Q tile, whose products are done: rows of 1 KiB, 16-byte piece i
      // at i ^ (row % 8); then a warp stores whole runs of 8 rows. (Straight
      // from the threads, 16 bytes to a row at a time, an epilogue took 11000
      // cycles.)
      const float wo = roww_s[row];
      if (whole && !p.tail_out) {
        // Nothing to add: the tile fits as bf16, in one pass, and its rows leave
        // by bulk copies, 1 KiB each, that the next tile's queries wait for
        // (5000 cycles with the two passes of fp32 below). Rows lie 1040 bytes
        // apart, the last ones in the P tile: 8 rows' pieces in 8 bank groups.
        constexpr uint32_t kPitch = 1040;
        const uint32_t dst = q_base + row * kPitch + (half * 32 + kh * 16) * 16, c = tl + Cfg::kColO + half * 128;
        static_assert(Cfg::kQ + 64 * kPitch <= Cfg::kRing, "rows on their way out");
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t o[2][16];
          DSA_TMEM_LD16_NOWAIT(c + 32 * g, o[0]);
          DSA_TMEM_LD16_NOWAIT(c + 32 * g + 16, o[1]);
          DSA_TMEM_WAIT32(o[0], o[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * (i & 1) + 2 * k;
              const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[i >> 1][e]) * wo, __uint_as_float(o[i >> 1][e + 1]) * wo);
              w[k] = *reinterpret_cast<const uint32_t *>(&h);
            }
            tc::st_shared_v4(dst + (4 * g + i) * 16, w[0], w[1], w[2], w[3]);
          }
        }
        tc::fence_async_smem();
        tc::tc_fence_before();   // O read before the next product
        sm_bar();
        const int r = 8 * warp + lane;
        if (lane < 8 && r < rows_here && row_ok(p, g0 + r)) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 1024;" ::"l"(p.out + (g0 + r) * kD),
                       "r"(q_base + r * kPitch)
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        leaving = true;
        continue;
      }
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        const uint32_t dst = row * 1024, c = tl + Cfg::kColO + half * 128 + pass * 64;
        uint32_t o[4][16];
        DSA_TMEM_LD16_NOWAIT(c, o[0]);
        DSA_TMEM_LD16_NOWAIT(c + 16, o[1]);
        DSA_TMEM_LD16_NOWAIT(c + 32, o[2]);
        DSA_TMEM_LD16_NOWAIT(c + 48, o[3]);
        DSA_TMEM_WAIT32(o[0], o[1]);
        DSA_TMEM_WAIT32(o[2], o[3]);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(o[g][4 * i + k]) * wo);
            st_q(dst + ((((half * 2 + kh) * 16 + 4 * g + i) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
        sm_bar();
        // lane's two 4-dim pieces of a row of the pass
        const int d0 = (lane >> 4) * 128 + pass * 64 + (lane & 15) * 4, d1 = d0 + 256;
        auto piece = [&](int r, int k) {
          return *reinterpret_cast<const float4 *>(smem + Cfg::kQ + r * 1024 + (((lane + 32 * k) ^ (r & 7)) << 4));
        };
        const int n = min(8, rows_here - 8 * warp);   // the warp's rows that exist
        if (!whole) {
#pragma unroll 2
          for (int i = 0; i < n; ++i) {
            const int r = 8 * warp + i;
            if (!part_ok(p, ps + r)) continue;
            float *dst = p.part_o + (ps + r) * kD;
            __stcg(reinterpret_cast<float4 *>(dst + d0), piece(r, 0));
            __stcg(reinterpret_cast<float4 *>(dst + d1), piece(r, 1));
          }
        } else {
          // The tails of 4 rows are in flight before the first store, which
          // might be to the same memory (with a load after each store, as the
          // compiler must keep them, a pass took 16800 cycles).
#pragma unroll 1
          for (int i0 = 0; i0 < n; i0 += 4) {
            uint2 tail[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              tail[i][0] = tail[i][1] = make_uint2(0, 0);
              if (p.tail_out && i0 + i < n && row_ok(p, g0 + 8 * warp + i0 + i)) {
                const __nv_bfloat16 *src = p.tail_out + (g0 + 8 * warp + i0 + i) * kD;
                tail[i][0] = *reinterpret_cast<const uint2 *>(src + d0);
                tail[i][1] = *reinterpret_cast<const uint2 *>(src + d1);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * warp + i0 + i;
              if (i0 + i < n) {   // (wt = 0 without a tail)
                store_out4(p, g0 + r, d0, piece(r, 0), roww_s[64 + r], tail[i][0]);
                store_out4(p, g0 + r, d1, piece(r, 1), roww_s[64 + r], tail[i][1]);
              }
            }
          }
        }
        sm_bar();   // the tile is free again
      }
      tc::tc_fence_before();   // O read before the next product
    }
  }

  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // (rows that left by bulk copies have arrived)
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();   // no MMA, commit or arrive of the other CTA reaches this one any more
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------ merge
// Parts of a row are the pairs whose ranges meet the row tile's units; M =
// max_i lse_i, w_i = e^{lse_i - M}. kGroups groups of kTh threads per row:
// group g takes parts g, g + kGroups, ... (thread t of it dims 4 (t + kTh q)
// ..), the groups' sums are added in their order, so the result does not
// depend on who finishes first. The attend kernel leaves each tile's pairs in
// `tile` (found anew by every thread they took longer than all the rest: 64-bit
// divisions), and the first values are loaded along with the lse.
// A row in few parts takes a warp (<32, 1>: 2048 rows in 5 parts 5 us, with a
// block of 512 threads per row 27), a row in many a block (<128, 2>: 512 rows
// in 19 parts 6 us, with 512 threads 9, with 128 threads 8).

template <int kTh, int kGroups, bool kChunk>
__device__ __forceinline__ void merge_row(const AttendParams<kChunk> &p, int64_t block) {
  constexpr int kBlock = kTh * kGroups < 128 ? 128 : kTh * kGroups;
  constexpr int kRow = kTh * kGroups;            // threads of a row
  constexpr int kQ = kD / 4 / kTh;               // float4 per thread and part
  constexpr int kIn = kTh == 32 ? 2 : 8;         // parts of a group in flight
  constexpr int kW = kRow;                       // parts whose weights are held at a time
  __shared__ float w_sh[kBlock / kRow][kW];
  __shared__ float red_s[kBlock / 32];
  __shared__ float4 sum_s[kGroups > 1 ? (kGroups - 1) * kTh : 1];
  const int rt = threadIdx.x % kRow, t = rt % kTh, g = rt / kTh, lane = threadIdx.x & 31;
  float *w_s = w_sh[threadIdx.x / kRow];
  auto row_sync = [&]() {
    if constexpr (kRow == 32) __syncwarp();
    else __syncthreads();
  };
  const int64_t ir = block * (kBlock / kRow) + threadIdx.x / kRow;   // row ir % 128 of a row tile
  int64_t gr = ir, tile = ir >> 7;
  int32_t units, len;
  if constexpr (!kChunk) {
    units = prefix_tiles(p, len);
    pdl_wait_primary();
    if (gr >= p.rows) return;                    // (whole warps; a block has one row where it syncs)
  } else {
    tile = __ldcg(p.merge + tile);
    const int4 rec = __ldcg(p.row_tile + 2 * tile);
    if ((ir & 127) >= rec.y) return;
    gr = rec.x + (ir & 127);
    units = rec.z;
  }
  RowParts parts = {0, -1, 0, (int32_t)(ir & 127)};   // no parts: no keys
  if (units > 0) {
    const int2 tl = __ldcg(p.tile + tile);
    parts.c0 = tl.x >> 1;
    parts.c1 = tl.y;
    parts.late = (tl.x & 1) * 128;
    if (parts.c0 == parts.c1) return;            // written by its pair
  }
  float lt = -INFINITY, sk = 0.f;
  uint2 tail[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) tail[q] = make_uint2(0, 0);
  if (p.tail_lse && row_ok(p, gr)) {
    lt = p.tail_lse[gr];
    if (g == 0) {
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        tail[q] = reinterpret_cast<const uint2 *>(p.tail_out + gr * kD)[t + kTh * q];
    }
  }
  if (p.sink) sk = __ldg(p.sink + (uint32_t)gr % (uint32_t)p.H);
  const int n_all = parts.count();
  auto part_lse = [&](int i) {
    return i < n_all && part_ok(p, parts.slot(i)) ? __ldcg(p.part_lse + parts.slot(i)) : -INFINITY;
  };
  float4 o[kIn][kQ];
  auto fetch = [&](int i0) {         // the group's parts i0, i0 + kGroups, .. (the last one again past the end)
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const int64_t from = parts.loaded(i0 + kGroups * i);
      const float4 *src = reinterpret_cast<const float4 *>(p.part_o + from * kD) + t;
      const bool ok = part_ok(p, from);
#pragma unroll
      for (int q = 0; q < kQ; ++q) o[i][q] = ok ? __ldcg(src + kTh * q) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  const float first = part_lse(rt);
  if (n_all > 0) fetch(g);
  float M = first;
  bool nan = first != first;
#pragma unroll 1
  for (int i = rt + kRow; i < n_all; i += kRow) {
    const float x = part_lse(i);
    nan |= x != x;
    M = fmaxf(M, x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (__any_sync(0xffffffffu, nan)) M = __uint_as_float(0x7FC00000u);   // a NaN stays one
  if constexpr (kRow > 32) {
    if (lane == 0) red_s[threadIdx.x >> 5] = M;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kRow / 32; ++i) {
      const float x = red_s[i];
      M = (x != x || M != M) ? __uint_as_float(0x7FC00000u) : fmaxf(M, x);
    }
  }
  float4 acc[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;                                 // (every thread adds all weights: no exchange)
#pragma unroll 1
  for (int cb = 0; cb < n_all && M != -INFINITY; cb += kW) {   // (M: a row without a kept key)
    const int n = min(kW, n_all - cb);
    row_sync();
    if (rt < n) {
      const float x = cb == 0 ? first : part_lse(cb + rt);
      w_s[rt] = x == -INFINITY ? 0.f : expf(x - M);
    }
    row_sync();
#pragma unroll 4
    for (int i = 0; i < n; ++i) z += w_s[i];
#pragma unroll 1
    for (int i0 = g; i0 < n; i0 += kGroups * kIn) {
      if (cb + i0 > g) fetch(cb + i0);
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int j = i0 + kGroups * i;
        const float w = j < n ? w_s[j] : 0.f;
        if (w == 0.f) continue;                  // (a pair without units left its slot as it was)
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          acc[q].x = fmaf(w, o[i][q].x, acc[q].x);
          acc[q].y = fmaf(w, o[i][q].y, acc[q].y);
          acc[q].z = fmaf(w, o[i][q].z, acc[q].z);
          acc[q].w = fmaf(w, o[i][q].w, acc[q].w);
        }
      }
    }
  }
  if constexpr (kGroups > 1) {
    if (g > 0) sum_s[(g - 1) * kTh + t] = acc[0];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 x = sum_s[k * kTh + t];
      acc[0].x += x.x;
      acc[0].y += x.y;
      acc[0].z += x.z;
      acc[0].w += x.w;
    }
  }
  const float lse = z == 0.f ? -INFINITY : M + logf(z);
  const RowWeights w = row_weights(lse, lt, p.sink != nullptr, sk);
  const float wo = z == 0.f ? 0.f : w.o / z;
  // (out may alias the tail, which its own thread has read; lse too, which
  // every thread of the row has read before a barrier above or this one)
  if constexpr (kRow == 32) __syncwarp();
  if (rt == 0 && row_ok(p, gr)) p.lse[gr] = w.lse;
#pragma unroll
  for (int q = 0; q < kQ; ++q)
    store_out4(p, gr, 4 * (t + kTh * q), make_float4(acc[q].x * wo, acc[q].y * wo, acc[q].z * wo, acc[q].w * wo),
               w.tail, tail[q]);
}

// A chunk call's blocks take the listed tiles' rows in turn: at most a tile per
// pair but for those without keys (a grid over all rows took 86 us of 323 for
// 1770 tiles of a window of 128, 75 of them shared).
template <int kTh, int kGroups, bool kChunk>
__global__ void __launch_bounds__(kTh *kGroups < 128 ? 128 : kTh * kGroups)
    prefix_merge_kernel(AttendParams<kChunk> p) {
  if constexpr (!kChunk) {
    merge_row<kTh, kGroups, kChunk>(p, blockIdx.x);
  } else {
    constexpr int kRows = kTh * kGroups < 128 ? 128 / (kTh * kGroups) : 1;   // of a block
    pdl_wait_primary();
    const int64_t blocks = (int64_t)__ldcg(p.n_merge) * (128 / kRows);
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
      merge_row<kTh, kGroups, kChunk>(p, b);
      __syncthreads();   // its shared memory
    }
  }
}

// ------------------------------------------------------------ launching
template <bool V32, bool kChunk>
cudaError_t attend_setup(void *) {
  return cudaFuncSetAttribute(prefix_attend_kernel<V32, kChunk>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)PfCfg<V32>::kSmem);
}
template <bool V32, bool kChunk>
cudaError_t attend_ready() {
  return dsa_configure_once((kChunk ? kOnceChunk : kOncePrefix) + (V32 ? 1 : 0), &attend_setup<V32, kChunk>, nullptr);
}

inline cudaLaunchConfig_t config(unsigned grid, unsigned block, size_t smem, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  return c;
}
// As the programmatic dependent of the launch before it on the stream.
template <typename... K, typename... A>
cudaError_t launch_dependent(cudaLaunchConfig_t c, void (*kernel)(K...), const A &...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// CTA pairs that run at the same time on the current device (a GPC's odd SM
// takes none), from the kernel's occupancy.
template <bool V32, bool kChunk>
cudaError_t resident_pairs(int *pairs) {
  cudaError_t e = attend_ready<V32, kChunk>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = config(2, kPfThreads, PfCfg<V32>::kSmem, nullptr);
  return cudaOccupancyMaxActiveClusters(pairs, prefix_attend_kernel<V32, kChunk>, &c);
}

// The driver's tensor map encoder, looked up once (no link to libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);
inline EncodeTiled tensor_map_encoder() {
  static const EncodeTiled f = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}
// The images as rows of 512 bytes, 32 of them (a 16 KiB chunk, contiguous) to
// a box.
inline bool image_map(void *image, int64_t bytes, CUtensorMap *map) {
  const EncodeTiled encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {256, (cuuint64_t)(bytes / 512)}, strides[1] = {512};
  const cuuint32_t box[2] = {256, 32}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, image, dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dsa

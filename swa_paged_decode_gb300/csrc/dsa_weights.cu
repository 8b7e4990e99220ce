// dsa_weights.cu -- the attention weight that cached records receive from new
// tokens (dsa_weights_plan / dsa_weights_run): for every sequence b and entry j
// of its list
//
//   out[b][j] = in[b][j] + sum_r e^{s_rj} / (e^{lse_r} + e^{z}),  s_rj = scale q_r . k_j,
//
// over the query rows r (token, head) that see the entry (dsa_chunk.cu says
// which), lse_r as their attention left it and z the head's sink.
//
// The product is taken with the keys as rows, D[key, query row] = K . Q^T, so
// that a thread holds one key and runs along the queries: the sum over r is a sum
// in its own registers and needs no exchange, and a query row's constants are the
// same for the whole warp. A weight is one exponential of (D factor_key)
// factor_row - lse_row.
//
// Precision. The results are fp32 and a weight is off by what its score is off,
// so no operand is rounded: queries are bf16 (8 bits) in f16 (11), with a power
// of two per row; NVFP4, ue8m0 and MODEL1 values are exact in f16 with one per
// key; the e4m3 codes of records with fp32 scales (FP8_528, V3.2) enter without
// their scales, one accumulator per 128-dim block, and the scales are applied in
// fp32 to the four sums (rounding code * scale to f16 first would cost 1e-4 of a
// weight). That halves the tensor core's rate (N = 128 for the room of four
// accumulators) and is hidden by the records' loads at single tokens.
//
// Two or three launches:
//   prepare  queries to f16 tile images (128 rows x 64 dims, 128-byte swizzle),
//            each row's constants, the list of items: (sequence, 128 or 256 keys,
//            a range of its row tiles);
//   weigh    CTA pairs (cta_group::2) take items in turn: 8 warps dequantize the
//            next item's records into one of two key tiles while the products of
//            the present one run; query chunks come through a ring, three warps
//            copying; 8 warps take the exponentials of one step (up to 256 query
//            rows) while the next one's product runs;
//   add      where items had to share the rows of their keys (few keys, many
//            rows): the parts in order, so that the result does not depend on
//            timing.
//
// What bounds it. Many rows: the queries' way from L2. With 64 keys in each CTA
// (M = 128) a step's 256 KiB feed 2048 cycles of products, more than L2's 12 TB/s:
// leaving out half of the products or all exponentials changed nothing (64 tokens
// x 128 heads over 65536 MODEL1 records 408 us). With 128 keys in each (WIDE, M =
// 256, one key tile in place of two) the same bytes feed twice the work: 296 us,
// 1855 TFLOP/s, 0.97 of the measured peak; an item's set-up then stands alone, so
// few rows keep to 64 (dsa_weights_plan). Single tokens: latency, 5 us to prepare,
// then roles of 3000 cycles per 128 keys beside one another (32 tokens x 64 heads
// over 98000 records 26 us, 2.0 TB/s). The steps there: block-wide staging of the
// rows' constants and one warp per key's loads 60 and 653 us; constants a step
// ahead, packed arithmetic 48, 528; records converted in f16 by 8 warps, addresses
// found a lane per key, products unrolled 44, 452; items in shared memory 34;
// constants by bulk copies and no barrier per step 33, 408; images by blocks of 32
// rows, the pairs set up before they wait for them 26, 304 (wide); items counted in
// 32 bits 26, 296. Records of the next item loaded as those of this one are
// converted: no faster.
#include "dsa_attend.cuh"
#include "dsa_rows.cuh"

namespace dsa {

constexpr int32_t kWeightsMagic = 0x57415344;   // "DSAW"

struct WeightsParams {
  ListArgs L;                  // lists: ids, lens, width, idx_stride
  const int32_t *starts;       // [B + 1]
  int32_t T, B, H, window, splits, max_items, tiles;   // tiles: of the query images
  int32_t span;                // keys of an item: 128, or 256 (wide)
  const __nv_bfloat16 *q;
  int64_t q_st, q_sh;
  const float *lse, *sink;
  float scale_log2;
  const float *in;             // or null: zeros
  int64_t in_st;
  float *out;
  int64_t out_st;
  long long wait_budget;
  // workspace
  int32_t *status;
  int32_t *n_items;
  int4 *item;                  // [max_items][2]
  uint8_t *image;              // [tiles][64-dim block][8-row group][1 KiB]
  float *row;                  // [tiles][2][128] scale log2(e) 2^e, and - log2 of the denominator
  float *part;                 // [splits][B][width]
};

constexpr int kWtPrep = 256;
__device__ __forceinline__ Sequence weights_sequence(const WeightsParams &p, int32_t b) {
  const int32_t s0 = __ldg(p.starts + b), s1 = __ldg(p.starts + b + 1), len = __ldg(p.L.lens + b);
  return {s0, s1 - s0, min(max(len, 0), p.L.width), p.window};
}
// First image tile of a sequence: those of any two do not meet.
__device__ __forceinline__ int32_t image_tile(const WeightsParams &p, int32_t b, int32_t s0) {
  return (int32_t)((int64_t)s0 * p.H >> 7) + b;
}
// The row tiles [lo, hi) of a sequence that see any of an item's keys.
__device__ __forceinline__ void seeing_tiles(const WeightsParams &p, const Sequence &s, int32_t key0, int32_t &lo, int32_t &hi) {
  const int64_t before = s.len - s.n;   // position of its first token
  const int64_t t0 = max((int64_t)0, key0 - before);
  int64_t t1 = s.n;
  if (p.window > 0) t1 = min(t1, (int64_t)key0 + p.span - 1 + p.window - before);
  lo = (int32_t)(t0 * p.H >> 7);
  hi = t1 > t0 ? (int32_t)((t1 * p.H + 127) >> 7) : lo;
}

// ------------------------------------------------------------ prepare
template <bool kV32>
__global__ void __launch_bounds__(kWtPrep) weights_prepare_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int kDB = kV32 ? 9 : 8;
  __shared__ int32_t w_s[kWtPrep / 32], upto_s[kWtPrep];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!kDebug && blockIdx.x == 0 && tid == 0) *p.status = DSA_OK;
  pdl_launch_dependents();
  bool bad = false;
  for (int32_t b = tid; b < p.B; b += kWtPrep) {
    const int32_t s0 = __ldg(p.starts + b), s1 = __ldg(p.starts + b + 1);
    bad |= s0 < 0 || s1 < s0 || s1 > p.T;
  }
  if (__syncthreads_or(bad)) {   // starts that do not ascend: no work, as in a chunk call
    if (blockIdx.x == 0 && tid == 0) {
      *p.n_items = 0;
      report_status(p.status, DSA_ERR_INVALID_ARG);
    }
    return;
  }
  if (blockIdx.x == 0) {
    // items: `span` keys that any token of a sequence sees, its row
    // tiles cut in `splits`; 256 sequences at a time, then an item to a thread
    int32_t n = 0;
    for (int32_t b0 = 0; b0 < p.B; b0 += kWtPrep) {
      int32_t mine = 0;
      if (b0 + tid < p.B) {
        const Sequence s = weights_sequence(p, b0 + tid);
        if (s.any()) mine = (s.len - s.gather_begin() * 128 + p.span - 1) / p.span * p.splits;
      }
      int32_t v = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
      }
      __syncthreads();
      if (lane == 31) w_s[warp] = v;
      __syncthreads();
      int32_t sum = 0;
      for (int k = 0; k < kWtPrep / 32; ++k) {
        if (k < warp) v += w_s[k];
        sum += w_s[k];
      }
      upto_s[tid] = v;
      __syncthreads();
      for (int32_t x = tid; x < sum && n + x < p.max_items; x += kWtPrep) {
        int lo = 0, hi = min(kWtPrep, p.B - b0) - 1;   // the sequence of item x
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (upto_s[mid] > x) hi = mid; else lo = mid + 1;
        }
        const int32_t b = b0 + lo, i = x - (lo > 0 ? upto_s[lo - 1] : 0);
        const Sequence s = weights_sequence(p, b);
        const int32_t u = i / p.splits, part = i - u * p.splits, key0 = s.gather_begin() * 128 + u * p.span;
        int32_t r0, r1;
        seeing_tiles(p, s, key0, r0, r1);
        const int64_t steps = (r1 - r0 + 1) >> 1;   // (cut between steps of two tiles)
        const int32_t t0 = min(r1, r0 + 2 * (int32_t)(steps * part / p.splits)), t1 = min(r1, r0 + 2 * (int32_t)(steps * (part + 1) / p.splits));
        p.item[2 * (int64_t)(n + x)] = make_int4(b, key0, s.len, s.n);
        // whether every row of the range sees every key (bit 31: none need be masked)
        const int64_t first = s.row_position(p.H, 128 * (int64_t)t0), last = s.row_position(p.H, min(128 * (int64_t)t1, (int64_t)s.n * p.H) - 1);
        const bool all = t1 > t0 && first >= key0 + p.span - 1 && (p.window == 0 || last - p.window < key0);
        p.item[2 * (int64_t)(n + x) + 1] = make_int4(image_tile(p, b, s.s0), t0, t1, part | (all ? INT32_MIN : 0));
      }
      n += sum;
    }
    if (tid == 0) *p.n_items = min(n, p.max_items);
    return;
  }
  // entries that no token sees keep what they had: a list's share of the blocks
  // takes 256 of them in turn
  if (p.in != p.out) {
    const int32_t blocks = gridDim.x - 1, share = max(1, blocks / p.B);
    for (int32_t u = blockIdx.x - 1; u < p.B * share; u += blocks) {
      const int32_t b = u / share;
      const Sequence s = weights_sequence(p, b);
      const int32_t end = s.any() ? min(s.gather_begin() * 128, s.len) : s.len;
#pragma unroll 4
      for (int32_t j = (u - b * share) * kWtPrep + tid; j < end; j += share * kWtPrep)
        p.out[b * p.out_st + j] = p.in ? __ldg(p.in + b * p.in_st + j) : 0.f;
    }
  }
  // query images, a block per 32 rows of a 128-row tile, 4 to a warp with their
  // loads in flight together (a block per tile, a row after the other, took 8 us
  // longer)
  for (int32_t unit = blockIdx.x - 1; unit < 4 * p.tiles; unit += gridDim.x - 1) {
    const int32_t tile = unit >> 2;
    int32_t b = 0, hi = p.B - 1;   // the last sequence whose tiles begin at or before this one
    while (b < hi) {
      const int32_t mid = (b + hi + 1) >> 1;
      if (image_tile(p, mid, __ldg(p.starts + mid)) <= tile) b = mid; else hi = mid - 1;
    }
    const Sequence s = weights_sequence(p, b);
    const int32_t i = tile - image_tile(p, b, s.s0);
    if (i < 0 || i >= s.tiles(p.H)) continue;
    const int32_t rows = s.tile_rows(p.H, i), first = 32 * (unit & 3) + warp;
    if (i == 0 && rows <= 64 && first >= 64) continue;   // (a sequence of one step of 64 rows)
    uint8_t *base = p.image + (int64_t)tile * (kDB * 16384);
    uint4 qa[4], qb[4];
    uint32_t qc[4];
    float lse[4], sink[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t r = first + 8 * k;
      qa[k] = qb[k] = make_uint4(0, 0, 0, 0);
      qc[k] = 0;
      lse[k] = sink[k] = 0.f;
      if (r >= rows) continue;
      const uint32_t gr = (uint32_t)s.s0 * p.H + 128u * i + r, t = gr / (uint32_t)p.H, h = gr - t * (uint32_t)p.H;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)t * p.q_st + (int64_t)h * p.q_sh);
      qa[k] = ld_row(src + 2 * lane);
      qb[k] = ld_row(src + 2 * lane + 1);
      if constexpr (kV32) qc[k] = __ldg(reinterpret_cast<const uint32_t *>(src + 64) + lane);
      lse[k] = __ldg(p.lse + gr);
      if (p.sink) sink[k] = __ldg(p.sink + h);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t r = first + 8 * k;
      const uint32_t w[8] = {qa[k].x, qa[k].y, qa[k].z, qa[k].w, qb[k].x, qb[k].y, qb[k].z, qb[k].w};
      uint32_t mb = qc[k] & 0x7FFF7FFFu;
#pragma unroll
      for (int j = 0; j < 8; ++j) mb = __vmaxu2(mb, w[j] & 0x7FFF7FFFu);
      mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
      int e = mb ? (int)(mb >> 7) - 127 : 0;
      e = e < -126 ? -126 : (e > 126 ? 126 : e);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      auto half2 = [&](uint32_t x) { return tc::pack_f16x2(bf16_bits_to_f32(x & 0xFFFFu) * down, bf16_bits_to_f32(x >> 16) * down); };
      uint32_t f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = half2(w[j]);
      const int x = r & 7;
      uint8_t *row = base + (r >> 3) * 1024 + x * 128;
      const uint4 lo = make_uint4(f[0], f[1], f[2], f[3]), up = make_uint4(f[4], f[5], f[6], f[7]);
      tc::stg_v8(row + (lane >> 2) * 16384 + (((2 * (lane & 3)) ^ (x & 6)) << 4), (x & 1) ? up : lo, (x & 1) ? lo : up);
      if constexpr (kV32)
        *reinterpret_cast<uint32_t *>(row + 8 * 16384 + (((lane >> 2) ^ x) << 4) + 4 * (lane & 3)) = half2(qc[k]);
      if (lane == 0) {
        // log2(e^lse + e^z); a row that attended nothing weighs nothing, nor do the
        // zeros behind the sequence's last row
        float l = lse[k] == -INFINITY ? INFINITY : lse[k];
        if (p.sink && lse[k] != -INFINITY) {
          const float z = sink[k], m = fmaxf(lse[k], z), d = -fabsf(lse[k] - z);
          l = lse[k] != lse[k] || z != z ? lse[k] + z : m == INFINITY ? INFINITY : z == -INFINITY ? lse[k] : m + log1pf(expf(d));
        }
        const bool in = r < rows;
        p.row[(int64_t)tile * 256 + r] = in ? p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23) : 0.f;
        p.row[(int64_t)tile * 256 + 128 + r] = in ? -l * kLog2e : -INFINITY;
      }
    }
  }
}

// ------------------------------------------------------------ weigh
constexpr int kWtThreads = 640;   // warps 0-7 exponentials, 8 MMA, 9-11 copies, 12-19 records
constexpr int kWtCopies = 3, kWtRecords = 8;

// A lane's 16 values of a record with one factor 2^E per key, in f16 and exact as
// far as the header says: codes times a power of two (or an e4m3 scale), so the
// products are taken in f16 (a third of the instructions of the way through
// fp32, which bf16 parts take, and blocks whose scale is no f16 in units of 2^E:
// far below the row's largest, or with small codes above the range of E). -> E
template <int FMT>
__device__ __forceinline__ int key_halves(const RawRecord &r, int lane, uint32_t (&f)[8]) {
  const int share = record_exponent<FMT>(r, lane);
  const int E = min(max(__reduce_max_sync(0xffffffffu, share), -kPfRange), kPfRange) - kPfTop;
  if constexpr (FMT == DSA_REC_NVFP4_288) {
    const bool nan = (r.s & 0x7Fu) == 0x7Fu;
    const float m = nan ? __uint_as_float(0x7FC00000u) : e4m3_to_f32(r.s) * __uint_as_float((uint32_t)(127 - E) << 23);
    const uint32_t m2 = share == kZeroShare && !nan ? 0u : tc::pack_f16x2(m, m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[4];
      tc::e2m1x8_to_f16x8(r.w[h], c);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[4 * h + k] = tc::hmul2(c[k], m2);
    }
  } else {
    const bool bf16_part = FMT == DSA_REC_MODEL1_584 && lane >= 28;
    const int k = (int)(r.s & 0xFFu) - 127 - E;   // the block's power of two, in units of 2^E
    const bool far = !bf16_part && share != kZeroShare && (k < -24 || k > 15);
    if (__any_sync(0xffffffffu, far)) {
      float v[16], t0, t1;
      expand_record<FMT>(r, lane, v, t0, t1);
      const float down = __uint_as_float((uint32_t)(127 - E) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = tc::pack_f16x2(v[2 * i] * down, v[2 * i + 1] * down);
    } else if (bf16_part) {
      const float down = __uint_as_float((uint32_t)(127 - E) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = tc::pack_f16x2(bf16_bits_to_f32(r.w[i] & 0xFFFFu) * down, __uint_as_float(r.w[i] & 0xFFFF0000u) * down);
    } else {
      uint32_t m = (r.s & 0xFFu) == 0xFFu ? 0x7E00u : share == kZeroShare ? 0u : k >= -14 ? (uint32_t)(k + 15) << 10 : 1u << (k + 24);
      m |= m << 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        tc::e4m3x4_to_f16x4(r.w[i], lo, hi);
        f[2 * i] = tc::hmul2(lo, m);
        f[2 * i + 1] = tc::hmul2(hi, m);
      }
    }
  }
  return E;
}

// Waits for the warp's outstanding TMEM loads; v is tied to the wait.
#define DSA_TMEM_WAIT16(v)                                                                                            \
  asm volatile("tcgen05.wait::ld.sync.aligned;"                                                                       \
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),      \
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]) \
               :                                                                                                      \
               : "memory")

template <int FMT, bool WIDE>
struct WtCfg {
  static constexpr int kKeys = WIDE ? 128 : 64;                     // of an item, to a CTA
  static constexpr int kBufs = WIDE ? 1 : 2;                        // key tiles
  static constexpr bool kV32 = FMT == DSA_REC_V32_656;
  static constexpr bool kBlocks = FMT == DSA_REC_FP8_528 || kV32;   // fp32 scales: an accumulator per block
  static constexpr int kAcc = kV32 ? 5 : kBlocks ? 4 : 1;
  static constexpr int kDB = kV32 ? 9 : 8;
  static constexpr int kN = kBlocks ? 128 : 256;                    // query rows of a step at most
  static constexpr int kCols = WIDE ? kN : kN / 2;                  // TMEM columns of an accumulator
  static constexpr int kSets = 512 / (kAcc * kCols);                // steps whose accumulators it holds
  // Query rows wait in slots of 16 KiB: of a step of N rows one, two or four
  // 64-dim blocks of this CTA's N / 2 (so that a step of few rows takes few waits).
  static constexpr int kSlots = kV32 ? 4 : 5;
  static constexpr uint32_t kBlock = kKeys * 128;                   // 64 dims of the CTA's keys
  static constexpr uint32_t kTile = kDB * kBlock;                   // a key tile: [kDB][kKeys x 64 dims] f16
  static constexpr uint32_t kRing = kBufs * kTile;
  static constexpr int kConst = 4;                                  // steps whose rows' constants are held
  static constexpr uint32_t kColS = kRing + kSlots * 16384;         // [kConst][kN / 128][2][128] f32
  static constexpr uint32_t kFac = kColS + kConst * 8 * kN;         // [kBufs][8][kKeys] f32 a key's factors; the last: kept or not
  static constexpr uint32_t kRed = kFac + 4096;                     // [2][256] f32
  static constexpr uint32_t kItems = kRed + 2048;                   // [kWtHeld][2] int4
  static constexpr uint32_t kMisc = kItems + 2048;
  static constexpr int kFull = 0, kEmpty = kSlots, kAFull = 2 * kSlots, kAEmpty = kAFull + kSets,
                       kKFull = kAEmpty + kSets, kKReady = kKFull + 2, kKEmpty = kKReady + 2, kCFull = kKEmpty + 2, kCEmpty = kCFull + kConst,
                       kDrain = kCEmpty + kConst, kBars = kDrain + 1;
  static constexpr uint32_t kAbort = 8 * kBars, kTmem = kAbort + 4;
  static constexpr uint32_t kBytes = kMisc + 512;
  static_assert(kTmem + 4 <= 512, "misc area");
  static_assert(kBytes + 1024 <= 232448u, "shared memory layout exceeds 227 KiB");
  // rows of the step that starts with `left` rows to go, and 64-dim blocks to a slot
  static __device__ __forceinline__ int rows(int32_t left) { return left > 128 && kN == 256 ? 256 : left > 64 ? 128 : 64; }
  static __device__ __forceinline__ int per_slot(int N) { return 256 / N; }
};

// The items of a pair (its first kWtHeld ones in shared memory: a role that went
// to the L2 for each would wait for it), and the steps of an item (up to kN
// query rows each).
constexpr int kWtHeld = 64;
template <class Cfg>
struct Items {
  const WeightsParams &p;
  const int4 *held;      // [kWtHeld][2]
  int32_t i, n, pair, pairs;   // the next one, of how many of this pair
  int4 a, c;
  int32_t tile, end;     // next row tile of the item, and the row tile past its last
  int32_t past;          // the row past its last (rows are counted in 31 bits less 128)
  __device__ __forceinline__ Items(const WeightsParams &q, const int4 *h, int pr, int prs) : p(q), held(h), i(0), pair(pr), pairs(prs) {
    const int32_t all = __ldcg(p.n_items);
    n = all > pair ? (all - pair + pairs - 1) / pairs : 0;
  }
  __device__ __forceinline__ int4 half(int32_t k, int h) const {
    return k < kWtHeld ? held[2 * k + h] : __ldcg(p.item + 2 * ((int64_t)pair + (int64_t)k * pairs) + h);
  }
  __device__ __forceinline__ bool next() {   // the next item
    if (i >= n) return false;
    a = half(i, 0);
    c = half(i, 1);
    ++i;
    tile = c.y;
    end = c.z;
    past = min(a.w * p.H, end * 128);
    return true;
  }
  __device__ __forceinline__ bool empty() const { return c.y >= c.z; }
  __device__ __forceinline__ int32_t left() const { return past - tile * 128; }
  __device__ __forceinline__ bool next_step(int &N) {   // tile is the step's until advance
    if (tile >= end) return false;
    N = Cfg::rows(left());
    return true;
  }
  __device__ __forceinline__ void advance(int N) { tile += N == 256 ? 2 : 1; }
};

template <int FMT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWtThreads, 1)
    weights_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap map16,
                   const __grid_constant__ CUtensorMap map8, const __grid_constant__ CUtensorMap map4) {
  using Cfg = WtCfg<FMT, WIDE>;
  constexpr bool kV32 = Cfg::kV32;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = tc::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sbase = raw_base + pad, ring = sbase + Cfg::kRing;
  float *col_s = reinterpret_cast<float *>(smem + Cfg::kColS);
  float *fac_s = reinterpret_cast<float *>(smem + Cfg::kFac);
  float *red_s = reinterpret_cast<float *>(smem + Cfg::kRed);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kMisc);
  volatile int32_t *abort_s = reinterpret_cast<volatile int32_t *>(smem + Cfg::kMisc + Cfg::kAbort);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kMisc + Cfg::kTmem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t side = tc::cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (warp == 0) tc::tmem_alloc_pair(tmem_slot, 512);
  if (tid == 32) {
    for (int b = 0; b < Cfg::kBars; ++b) {
      const bool a = b >= Cfg::kAEmpty && b < Cfg::kKFull, k = b >= Cfg::kKFull && b < Cfg::kKReady,
                 r = b >= Cfg::kKReady && b < Cfg::kKEmpty, e = b >= Cfg::kKEmpty && b < Cfg::kCFull, c = b >= Cfg::kCEmpty && b < Cfg::kDrain;
      tc::mbar_init(&bars[b], a ? 16u : k ? 2u * kWtRecords : r ? kWtRecords : e ? 9u : c ? 8u : 1u);
    }
    tc::fence_mbar_init();
    *abort_s = 0;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_primary();
  int4 *held = reinterpret_cast<int4 *>(smem + Cfg::kItems);
  if (tid < 2 * kWtHeld) {   // (past the last item: not looked at)
    const int64_t at = (int64_t)pair + (int64_t)(tid >> 1) * pairs;
    if (at < p.max_items) held[tid] = __ldcg(p.item + 2 * at + (tid & 1));
  }
  Items<Cfg> items(p, held, pair, pairs);
  __syncthreads();
  auto wait = [&](int b, uint32_t phase) -> bool {   // bounded, as in the attend kernel
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
  auto lead = [&](int b) { return tc::mapa(tc::smem_u32(&bars[b]), 0); };

  // 640 threads leave 96 registers each; the exponentials want more (spilled, a
  // load on its way to a register would be waited for), the copies need fewer:
  // 256 x 112 + 128 x 80 + 256 x 88 = 640 x 96.
  if (warp >= 12) {
    tc::setmaxnreg_dec<88>();
    // ======================================================== records
    // kKeys keys of an item to this CTA, 8 or 16 to a warp, 8 records' loads in
    // flight together. The slots of the next two items are known ahead, and the
    // records of the next one are on their way to L2 for a whole item's time. A
    // warp runs one instruction in five cycles or so at best, so what a lane per
    // key can find (addresses) it does.
    const int pw = warp - 12;
    constexpr int kPer = Cfg::kKeys / kWtRecords;
    bool ok = true;
    uint32_t turn = 0;
    auto item_at = [&](int32_t i) { return i < items.n ? items.half(i, 0) : make_int4(0, 0, 0, 0); };
    auto slot_of = [&](const int4 &a) {   // lane l < kPer: the slot of key kPer pw + l (a list of length 0 has none)
      const int32_t j = a.y + Cfg::kKeys * (int32_t)side + kPer * pw + lane;
      return lane < kPer && j < a.z ? __ldg(p.L.ids + (int64_t)a.x * p.L.idx_stride + j) : -1;
    };
    // its record, and whether it is kept; one that is not reads slot 0's, which counts for nothing
    auto record_of = [&](int32_t slot, uint32_t &kept) {
      bool k = slot >= 0 && (int64_t)slot < p.L.num_slots;
      const uint8_t *rec = record_ptr(p.L, k ? slot : 0);
      if (k && !dbg_ok(p.status, rec + p.L.rec <= p.L.base + p.L.extent, kDbgRecord)) {
        k = false;
        rec = p.L.base;
      }
      kept = __ballot_sync(0xffffffffu, k);
      return rec;
    };
    int32_t slot2 = slot_of(item_at(1));
    uint32_t kept1;
    const uint8_t *rec1 = record_of(slot_of(item_at(0)), kept1);
    const uint32_t lane_at = (uint32_t)(lane >> 2) * Cfg::kBlock + (uint32_t)pw * (kPer * 128u);
    while (ok && items.next()) {
      const uint8_t *rec0 = rec1;
      const uint32_t kept0 = kept1;
      constexpr int kDeep = FMT == DSA_REC_MODEL1_584 ? 4 : 8;   // records in flight (a MODEL1 share takes 9 registers)
      RawRecord raw[kDeep];
      auto load = [&](int i) {
        const uint8_t *rec = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rec0), i));
        load_record<FMT>(rec, lane, raw[i % kDeep]);
      };
      if (!items.empty()) {
#pragma unroll
        for (int i = 0; i < kDeep; ++i) load(i);
      }
      rec1 = record_of(slot2, kept1);
      slot2 = slot_of(item_at(items.i + 1));
      if (items.empty()) continue;
      {   // the next records to L2, a line of 128 bytes to a lane
        constexpr int kLanes = 32 / kPer;   // to a key
        const int key = lane / kLanes;
        const uint8_t *rec = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rec1), key));
#pragma unroll
        for (int b = 0; b < 6; b += kLanes) {
          const int line = 128 * (lane % kLanes + b);
          if (line < p.L.rec && ((kept1 >> key) & 1u)) asm volatile("prefetch.global.L2 [%0];" ::"l"(rec + line));
        }
      }
      const int buf = turn % Cfg::kBufs;
      ok = wait(Cfg::kKEmpty + buf, ((turn / Cfg::kBufs) & 1u) ^ 1u);
      ++turn;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float *fac = fac_s + buf * (8 * Cfg::kKeys) + kPer * pw;
      const uint32_t tile = sbase + buf * Cfg::kTile + lane_at;
      if (lane < kPer) fac[7 * Cfg::kKeys + lane] = (kept0 >> lane) & 1u ? 1.f : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {   // row i % 8 of the warp's 8-row group i / 8
        const RawRecord &rr = raw[i % kDeep];
        uint32_t f[8];
        if constexpr (Cfg::kBlocks) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::e4m3x4_to_f16x4(rr.w[k], f[2 * k], f[2 * k + 1]);
          if ((lane & 7) == 0) fac[(lane >> 3) * Cfg::kKeys + i] = __uint_as_float(rr.s);
          if constexpr (kV32) {
            const uint32_t m = rr.t & 0x7FFF7FFFu;
            const uint32_t mb = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
            const int E = min(max((int)(mb >> 7) - 127, -kPfRange), kPfRange) - kPfTop;
            const float down = __uint_as_float((uint32_t)(127 - E) << 23);
            if (lane == 0) fac[4 * Cfg::kKeys + i] = __uint_as_float((uint32_t)(127 + E) << 23);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + buf * Cfg::kTile + 8 * Cfg::kBlock + pw * (kPer * 128) + i * 128 +
                                                        (((lane >> 2) ^ (i & 7)) << 4) + 4 * (lane & 3)),
                         "r"(tc::pack_f16x2(bf16_bits_to_f32(rr.t & 0xFFFFu) * down, bf16_bits_to_f32(rr.t >> 16) * down))
                         : "memory");
          }
        } else {
          const int E = key_halves<FMT>(rr, lane, f);
          if (lane == 0) fac[i] = __uint_as_float((uint32_t)(127 + E) << 23);
        }
        if (i + kDeep < kPer) load(i + kDeep);
        tc::st_shared_v4(tile + i * 128 + (((2 * (lane & 3)) ^ (i & 7)) << 4), f[0], f[1], f[2], f[3]);
        tc::st_shared_v4(tile + i * 128 + (((2 * (lane & 3) + 1) ^ (i & 7)) << 4), f[4], f[5], f[6], f[7]);
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive_remote(tc::mapa(tc::smem_u32(&bars[Cfg::kKReady + buf]), side));
        tc::mbar_arrive_remote(lead(Cfg::kKFull + buf));
      }
    }
    // the tiles' last releases have arrived before the pair ends
    for (int k = 0; k < Cfg::kBufs && ok; ++k, ++turn) ok = wait(Cfg::kKEmpty + turn % Cfg::kBufs, ((turn / Cfg::kBufs) & 1u) ^ 1u);
  } else if (warp >= 8) {
    tc::setmaxnreg_dec<80>();
    if (warp >= 9) {
      // ======================================================== query chunks
      if (lane == 0) {
        uint32_t slot = 0, ph = 1;
        int turn = warp - 9;   // 0: this warp's slot (one thread would take longer for a slot than its products do)
        bool ok = true;
        uint32_t filled = 0, fill_ph = 0;
        const uint32_t full0 = lead(Cfg::kFull);
        uint32_t cs = 0, ph_c = 1;
        while (ok && items.next()) {
          int N;
          while (ok && items.next_step(N)) {
            if (warp == 9) {   // the constants of the step's rows, to either CTA its own copy
              ok = wait(Cfg::kCEmpty + cs, ph_c);
              if (!ok) break;
              const uint32_t bytes = N == 256 ? 2048u : 1024u;
              tc::mbar_expect_tx(&bars[Cfg::kCFull + cs], bytes);
              asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                               sbase + Cfg::kColS + cs * (8 * Cfg::kN)),
                           "l"(p.row + ((int64_t)items.c.x + items.tile) * 256), "r"(bytes), "r"(tc::smem_u32(&bars[Cfg::kCFull + cs]))
                           : "memory");
              if (++cs == Cfg::kConst) {
                cs = 0;
                ph_c ^= 1u;
              }
            }
            // this CTA's N / 2 rows: of a tile of its own with N = 256
            const int64_t tile = items.c.x + items.tile + (N == 256 ? side : 0);
            const int32_t y0 = (int32_t)(tile * (Cfg::kDB * 32)) + (N == 256 ? 0 : (int32_t)side * (N / 8));
            const bool in = dbg_ok(p.status, tile >= 0 && tile < p.tiles, kDbgPartial);
            const int per = Cfg::per_slot(N);
            const uint32_t block = (uint32_t)N * 64u;   // bytes of this CTA's rows of a 64-dim block
            for (int c = 0; c < Cfg::kDB && ok; c += per) {
              if (turn == 0) {
                turn = kWtCopies;
                ok = wait(Cfg::kEmpty + slot, ph);
                if (!ok) break;
                const int n = min(per, Cfg::kDB - c);
                if (side == 0) {
                  tc::mbar_expect_tx(&bars[Cfg::kFull + slot], 2u * n * block);   // both CTAs' bytes
                  filled |= 1u << slot;
                  fill_ph = (fill_ph & ~(1u << slot)) | ((ph ^ 1u) << slot);
                }
                const uint32_t dst = ring + slot * 16384, bar = full0 + 8 * slot;
                const void *map = N == 256 ? &map16 : N == 128 ? &map8 : &map4;
                for (int j = 0; j < n; ++j) tc::tma_load_pair(dst + j * block, map, 0, in ? y0 + (c + j) * 32 : 0, bar);
              }
              --turn;
              if (++slot == Cfg::kSlots) {
                slot = 0;
                ph ^= 1u;
              }
            }
            items.advance(N);
          }
        }
        // no commit reaches this CTA's barriers after its end; after a timeout no
        // copy is in flight (as in the attend kernel)
        for (int k = 0; k < Cfg::kSlots && ok; ++k) {
          ok = wait(Cfg::kEmpty + slot, ph);
          if (++slot == Cfg::kSlots) {
            slot = 0;
            ph ^= 1u;
          }
        }
        if (!ok) {
          for (int k = 0; k < Cfg::kSlots; ++k)
            if ((filled >> k) & 1u) tc::mbar_wait(&bars[Cfg::kFull + k], (fill_ph >> k) & 1u, kPfCopyWait);
          const long long t0 = clock64();
          while (clock64() - t0 < kPfCopyWait / 10) __nanosleep(1000);
        }
      }
      __syncwarp();
    } else {
      // ======================================================== MMA issue
      if (side == 0) {
        constexpr uint16_t kBoth = 3;
        constexpr uint32_t kHi = tc::sdesc_hi(1024, tc::kSwz128);
        const uint32_t dk0 = tc::sdesc_lo(sbase, 16), dq0 = tc::sdesc_lo(ring, 16);
        uint32_t slot = 0, ph = 0, set = 0, ph_a = 1, turn = 0;
        bool ok = true, issued = false;
        auto here = [&](bool x) { return __all_sync(0xffffffffu, x); };
        while (ok && items.next()) {
          if (items.empty()) continue;
          const uint32_t buf = turn % Cfg::kBufs, dk = dk0 + buf * (Cfg::kTile >> 4);
          ok = here(wait(Cfg::kKFull + buf, (turn / Cfg::kBufs) & 1u));
          ++turn;
          int N;
          while (ok && items.next_step(N)) {
            items.advance(N);
            const bool last = items.tile >= items.end;
            ok = here(wait(Cfg::kAEmpty + set, ph_a));
            if (!ok) break;
            tc::tc_fence_after();
            issued = true;
            const uint32_t d0 = tmem + set * (Cfg::kAcc * Cfg::kCols);
            auto products = [&](auto rows) {   // unrolled for each N: a slot is to go out in less time than its products take
              constexpr int kRows = decltype(rows)::value, kPer = 256 / kRows;
              constexpr uint32_t kId = tc::idesc_f16(2 * Cfg::kKeys, kRows, false, false);
#pragma unroll
              for (int c0 = 0; c0 < Cfg::kDB; c0 += kPer) {
                if (!here(wait(Cfg::kFull + slot, ph))) return false;
                tc::tc_fence_after();
                if (tc::elect_one()) {
                  const uint32_t q = dq0 + slot * 1024u;
#pragma unroll
                  for (int j = 0; j < kPer && c0 + j < Cfg::kDB; ++j) {
                    const int c = c0 + j;
                    const uint32_t d = Cfg::kBlocks ? d0 + (c >> 1) * Cfg::kCols : d0;
                    const bool first = Cfg::kBlocks ? (c & 1) == 0 : c == 0;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                      tc::mma_f16_pair(d, dk + c * (Cfg::kBlock >> 4) + 2 * ks, q + j * (kRows * 4u) + 2 * ks, kHi, kId, !first || ks ? 1u : 0u);
                  }
                  tc::mma_commit_to(&bars[Cfg::kEmpty + slot], kBoth);
                  if (c0 + kPer >= Cfg::kDB) {
                    tc::mma_commit_to(&bars[Cfg::kAFull + set], kBoth);
                    if (last) tc::mma_commit_to(&bars[Cfg::kKEmpty + buf], kBoth);
                  }
                }
                __syncwarp();
                if (++slot == Cfg::kSlots) {
                  slot = 0;
                  ph ^= 1u;
                }
              }
              return true;
            };
            if (N == 64) ok = products(std::integral_constant<int, 64>());
            else if (Cfg::kN == 128 || N == 128) ok = products(std::integral_constant<int, 128>());
            else ok = products(std::integral_constant<int, Cfg::kN>());
            if (++set == Cfg::kSets) {
              set = 0;
              ph_a ^= 1u;
            }
          }
        }
        if (issued && !ok && tc::elect_one()) {   // MMAs issued before a timeout end before TMEM is freed
          tc::mma_commit_one(&bars[Cfg::kDrain]);
          tc::mbar_wait(&bars[Cfg::kDrain], 0u, kPfWait);
        }
      }
      __syncwarp();
    }
  } else {
    // ======================================================== exponentials
    tc::setmaxnreg_inc<112>();
    const int q4 = warp & 3, half = warp >> 2;
    // TMEM lane; the key of this CTA's; which part of the rows its two (wide) or
    // four threads take: with 64 keys the upper lanes hold the upper half of N
    const int lr = 32 * q4 + lane, key = lr % Cfg::kKeys, part = WIDE ? half : 2 * (lr >> 6) + half;
    constexpr int kParts = WIDE ? 2 : 4;
    const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16);
    auto sm_bar = [&]() { asm volatile("barrier.sync 1, 256;" ::: "memory"); };
    const uint32_t aempty0 = lead(Cfg::kAEmpty), kempty0 = tc::mapa(tc::smem_u32(&bars[Cfg::kKEmpty]), side);
    const uint32_t cempty0 = tc::mapa(tc::smem_u32(&bars[Cfg::kCEmpty]), side);
    uint32_t set = 0, ph_a = 0, turn = 0, cs = 0, ph_c = 0, rb = 0;
    while (items.next()) {
      const int32_t at = items.a.y + Cfg::kKeys * (int32_t)side + key;   // list position of the thread's key
      const bool writes = part == 0 && at < items.a.z;
      float total = 0.f, before = 0.f;
      if (writes && p.splits == 1 && p.in) before = p.in[(int64_t)items.a.x * p.in_st + at];
      const bool all = items.c.w < 0;                            // every row sees every key
      // the query rows that see the key: see0 .. see0 + seen - 1
      uint32_t see0 = 0, seen = 0xFFFFFFFFu;
      if (!all) {
        const int32_t place = at - (items.a.z - items.a.w);      // of the tokens, the key's own
        const int32_t past = p.window > 0 && p.window < items.a.z - at ? max(place + p.window, 0) : items.a.w;
        see0 = (uint32_t)max(0, place) * (uint32_t)p.H;
        seen = (uint32_t)max(past - max(0, place), 0) * (uint32_t)p.H;
      }
      bool kept = false;
      if (!items.empty()) {
        const int buf = turn % Cfg::kBufs;
        wait(Cfg::kKReady + buf, (turn / Cfg::kBufs) & 1u);
        ++turn;
        const float *fac = fac_s + buf * (8 * Cfg::kKeys) + key;
        kept = fac[7 * Cfg::kKeys] != 0.f;
        F2 s[Cfg::kAcc];
#pragma unroll
        for (int b = 0; b < Cfg::kAcc; ++b) {
          const float f = kept ? fac[b * Cfg::kKeys] : 0.f;
          s[b] = f2(f, f);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(kempty0 + 8 * buf);   // the factors are read
        int N;
        while (items.next_step(N)) {
          // the thread's rows, `mine` of them from `first` (128 and up: in the second tile)
          const int mine = N / kParts, first = part * mine;
          const float *col = col_s + cs * (2 * Cfg::kN) + (first >> 7) * 256 + (first & 127);
          const uint32_t row0 = (uint32_t)items.tile * 128u + first;
          items.advance(N);
          wait(Cfg::kCFull + cs, ph_c);
          wait(Cfg::kAFull + set, ph_a);
          tc::tc_fence_after();
          const uint32_t c0 = tl + set * (Cfg::kAcc * Cfg::kCols) + half * mine;
          F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
          // 16 rows, their scores x (in units of the rows' factors)
          auto weigh = [&](auto masked, const F2 (&x)[8], int g) {
            const float4 *ca = reinterpret_cast<const float4 *>(col + g), *cl = ca + 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 ka = ca[i], kl = cl[i];
              const F2 y0 = f2_fma(x[2 * i], f2(ka.x, ka.y), f2(kl.x, kl.y));
              const F2 y1 = f2_fma(x[2 * i + 1], f2(ka.z, ka.w), f2(kl.z, kl.w));
              float e[4];
              f2_get(y0, e[0], e[1]);
              f2_get(y1, e[2], e[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) e[j] = tc::ex2(e[j]);
              if constexpr (decltype(masked)::value) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (row0 + g + 4 * i + j - see0 >= seen) e[j] = 0.f;
              }
              sum[0] = f2_add(sum[0], f2(e[0], e[1]));
              sum[1] = f2_add(sum[1], f2(e[2], e[3]));
            }
          };
          auto release = [&]() {   // the accumulators are read
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(aempty0 + 8 * set);
          };
          // (a branch for each four rows inside would keep their loads and
          // exponentials from overlapping: 430 cycles for 16 rows)
          auto step = [&](auto masked) {
            if constexpr (Cfg::kAcc == 1) {   // the next 16 rows' load in flight
              uint32_t d[2][16];
              auto take = [&](uint32_t (&v)[16], uint32_t (&next)[16], int g) {   // false: these were the last
                DSA_TMEM_WAIT16(v);
                const bool more = g + 16 < mine;
                if (more) DSA_TMEM_LD16_NOWAIT(c0 + g + 16, next);
                else release();
                F2 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = f2_mul(f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s[0]);
                weigh(masked, x, g);
                return more;
              };
              DSA_TMEM_LD16_NOWAIT(c0, d[0]);
#pragma unroll 1
              for (int g = 0;; g += 32)
                if (!take(d[0], d[1], g) || !take(d[1], d[0], g + 16)) break;
            } else {
#pragma unroll 1
              for (int g = 0; g < mine; g += 16) {
                uint32_t d[2][16];
                F2 x[8];
#pragma unroll
                for (int k = 0; k < Cfg::kAcc; k += 2) {
                  const int k1 = k + 1 < Cfg::kAcc ? k + 1 : k;
                  DSA_TMEM_LD16_NOWAIT(c0 + k * Cfg::kCols + g, d[0]);
                  DSA_TMEM_LD16_NOWAIT(c0 + k1 * Cfg::kCols + g, d[1]);
                  DSA_TMEM_WAIT32(d[0], d[1]);
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const F2 v = f2(__uint_as_float(d[0][2 * i]), __uint_as_float(d[0][2 * i + 1]));
                    x[i] = k == 0 ? f2_mul(v, s[0]) : f2_fma(v, s[k], x[i]);
                    if (k1 > k) x[i] = f2_fma(f2(__uint_as_float(d[1][2 * i]), __uint_as_float(d[1][2 * i + 1])), s[k1], x[i]);
                  }
                }
                if (g + 16 >= mine) release();
                weigh(masked, x, g);
              }
            }
          };
          if (all) step(std::false_type());
          else step(std::true_type());
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_remote(cempty0 + 8 * cs);   // the constants are read
          if (++cs == Cfg::kConst) {
            cs = 0;
            ph_c ^= 1u;
          }
          if (++set == Cfg::kSets) {
            set = 0;
            ph_a ^= 1u;
          }
          float a0, a1;
          f2_get(f2_add(sum[0], sum[1]), a0, a1);
          total += a0 + a1;
        }
      }
      // the threads of a key (the sums of the item before have been read: a barrier ago)
      float *red = red_s + rb * 256;
      rb ^= 1u;
      red[part * Cfg::kKeys + key] = total;
      sm_bar();
      if (writes) {
        float t = red[key];
#pragma unroll
        for (int k = 1; k < kParts; ++k) t += red[k * Cfg::kKeys + key];
        t = kept ? t : 0.f;
        const int64_t b = items.a.x;
        if (p.splits > 1) __stcg(p.part + ((int64_t)(items.c.w & INT32_MAX) * p.B + b) * p.L.width + at, t);
        else p.out[b * p.out_st + at] = before + t;
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------ add
__global__ void __launch_bounds__(256) weights_add_kernel(const __grid_constant__ WeightsParams p) {
  const int32_t b = blockIdx.y, j = (int32_t)(blockIdx.x * 256 + threadIdx.x);
  pdl_wait_primary();
  if (__ldcg(p.n_items) == 0) return;
  const Sequence s = weights_sequence(p, b);
  if (!s.any() || j >= s.len || j < s.gather_begin() * 128) return;
  float t = 0.f;
  for (int32_t k = 0; k < p.splits; ++k) t += __ldcg(p.part + ((int64_t)k * p.B + b) * p.L.width + j);
  p.out[b * p.out_st + j] = (p.in ? p.in[b * p.in_st + j] : 0.f) + t;
}

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::WeightsParams;

template <int FMT, bool WIDE>
cudaError_t weights_setup(void *) {
  return cudaFuncSetAttribute(dsa::weights_kernel<FMT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)(dsa::WtCfg<FMT, WIDE>::kBytes + 1024));
}
template <int FMT, bool WIDE>
cudaError_t weights_ready() {
  static_assert(!WIDE || (FMT >= DSA_REC_NVFP4_288 && FMT <= DSA_REC_MODEL1_584), "a wide kernel without a bit of its own");
  constexpr int bit = WIDE ? dsa::kOnceWeightsWide + FMT - 1 : dsa::kOnceWeights + FMT;
  return dsa::dsa_configure_once(bit, &weights_setup<FMT, WIDE>, nullptr);
}
// CTA pairs that run at the same time on the current device.
template <int FMT>
cudaError_t weights_pairs(int *pairs) {
  cudaError_t e = weights_ready<FMT, false>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = dsa::config(2, dsa::kWtThreads, dsa::WtCfg<FMT, false>::kBytes + 1024, nullptr);
  return cudaOccupancyMaxActiveClusters(pairs, dsa::weights_kernel<FMT, false>, &c);
}

// The query images as rows of 512 bytes, `rows` of them to a box.
bool chunk_map(void *image, int64_t bytes, uint32_t rows, CUtensorMap *map) {
  const dsa::EncodeTiled encode = dsa::tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {256, (cuuint64_t)(bytes / 512)}, strides[1] = {512};
  const cuuint32_t box[2] = {256, rows}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, image, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, bool WIDE>
cudaError_t launch_weigh(const WeightsParams &p, int32_t pairs, cudaStream_t st) {
  using namespace dsa;
  using Cfg = WtCfg<FMT, WIDE>;
  cudaError_t e = weights_ready<FMT, WIDE>();
  if (e != cudaSuccess) return e;
  CUtensorMap map16, map8, map4;
  const int64_t bytes = (int64_t)p.tiles * Cfg::kDB * 16384;
  if (!chunk_map(p.image, bytes, 32, &map16) || !chunk_map(p.image, bytes, 16, &map8) || !chunk_map(p.image, bytes, 8, &map4))
    return cudaErrorNotSupported;
  return launch_dependent(config(2u * pairs, kWtThreads, Cfg::kBytes + 1024, st), weights_kernel<FMT, WIDE>, p, map16, map8, map4);
}

template <int FMT>
cudaError_t launch_weights(const WeightsParams &p, int32_t pairs, int32_t num_sms, cudaStream_t st) {
  using namespace dsa;
  // a block to 32 rows of queries, or to 4096 entries to copy where those are more
  const int64_t copies = p.in != p.out ? p.B * (((int64_t)p.L.width + 4095) / 4096) : 1;
  const unsigned blocks = 1 + (unsigned)std::min(std::max(4 * (int64_t)p.tiles, copies), 8 * (int64_t)num_sms);
  weights_prepare_kernel<FMT == DSA_REC_V32_656><<<blocks, kWtPrep, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.T == 0) return e;   // (no tokens: the scores are copied, nothing is weighed)
  constexpr bool kCanWiden = !WtCfg<FMT, false>::kBlocks;
  e = p.span == 256 ? launch_weigh<FMT, kCanWiden>(p, pairs, st) : launch_weigh<FMT, false>(p, pairs, st);
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t c = config((unsigned)((p.L.width + 255) / 256), 256, 0, st);
  c.gridDim.y = (unsigned)p.B;
  return launch_dependent(c, weights_add_kernel, p);
}

}  // namespace

extern "C" {

dsa_status dsa_weights_plan(int32_t num_tokens, int32_t num_seqs, int32_t num_heads, int32_t width, int32_t num_sms,
                            int32_t d_qk, dsa_weights_plan_t *plan, size_t *workspace_bytes) {
  if (!plan || !workspace_bytes) return DSA_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_seqs < 0 || num_heads < 1 || width < 1 || num_sms < 0) return DSA_ERR_INVALID_ARG;
  if (d_qk != 512 && d_qk != 576) return DSA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)num_tokens * num_heads, halves = ((int64_t)width + 127) / 128;
  // an image tile more than the sequences': the second half of the last step
  const int64_t tiles = dsa::chunk_row_tiles(num_tokens, num_heads, num_seqs) + num_seqs + 2;
  // (rows and images' 512-byte rows, 288 to a tile, are counted in 31 bits, the
  // adding kernel's grid has 2^16 - 1 lists)
  if (rows > INT32_MAX - 128 || num_seqs > 65535 || width > (1 << 29) || tiles > INT32_MAX / 288)
    return DSA_ERR_UNSUPPORTED;
  int most_pairs = num_sms / 2;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        (d_qk == 576 ? weights_pairs<DSA_REC_V32_656>(&most_pairs) : weights_pairs<DSA_REC_FP8_528>(&most_pairs)) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->magic = dsa::kWeightsMagic;
  plan->abi_version = DSA_DECODE_ABI_VERSION;
  plan->num_tokens = num_tokens;
  plan->num_seqs = num_seqs;
  plan->num_heads = num_heads;
  plan->width = width;
  plan->d_qk = d_qk;
  plan->num_sms = num_sms;
  // How to cut the work, by what it takes about: a pair's items one after the
  // other, an item a set-up (its records) and its steps of 256 rows, of the mean
  // sequence. In microseconds: 3.5 and 1.6 for 128 keys, 8 and 2.2 for 256
  // (wide), 3 to add parts up. Measured (ue8m0, 8 lists of 8192): 1024 rows 63.8
  // narrow, 61.6 wide, 71.3 wide in two parts; 4096 rows 203, 171, 169; a list of
  // 32768 and 4096 rows 115, 85.5, 95.9; 4 lists of 6000 and 2048 rows 51.7, 51.9,
  // 50.1.
  const int64_t steps = num_seqs > 0 ? std::max<int64_t>(1, (rows / num_seqs + 255) / 256) : 1;
  const int64_t pairs = most_pairs < 1 ? 1 : most_pairs, units = halves * num_seqs;
  auto cut = [&](int64_t items, double setup, double step, int32_t &splits) {
    double best = 0;
    for (int64_t n = 1; n <= std::min<int64_t>(steps, 16); ++n) {
      const double t = (double)((items * n + pairs - 1) / pairs) * (setup + step * (double)((steps + n - 1) / n)) + (n > 1 ? 3.0 : 0.0);
      if (n == 1 || t < best) {
        best = t;
        splits = (int32_t)n;
      }
    }
    return best;
  };
  int32_t wide_splits = 1;
  const double narrow = cut(units, 3.5, 1.6, plan->splits);
  if (cut((halves + 1) / 2 * num_seqs, 8.0, 2.2, wide_splits) < narrow) plan->wide_splits = wide_splits;
  const int64_t splits = std::max(plan->splits, plan->wide_splits);
  if (units * splits > INT32_MAX / 2) return DSA_ERR_UNSUPPORTED;
  plan->tiles = (int32_t)tiles;
  plan->pairs = (int32_t)(units * splits < pairs ? (units < 1 ? 1 : units * splits) : pairs);
  int64_t off = 256;
  auto take = [&](int64_t &at, int64_t bytes) {
    at = off;
    off = dsa::align_up(off + bytes, 256);
  };
  take(plan->ws_item_offset, 32 * units * splits);
  take(plan->ws_image_offset, tiles * 128 * d_qk * 2);
  take(plan->ws_row_offset, tiles * 128 * 8);
  take(plan->ws_part_offset, splits > 1 ? splits * num_seqs * (int64_t)width * 4 : 0);
  plan->workspace_bytes = num_tokens == 0 || num_seqs == 0 ? 0 : off;
  // Test knob, read only here, as in dsa_decode_plan.
  if (const char *wb = std::getenv("DSA_DECODE_WAIT_BUDGET")) {
    const long long v = std::atoll(wb);
    if (v > 0) plan->wait_budget_cycles = v;
  }
  *workspace_bytes = (size_t)plan->workspace_bytes;
  return DSA_OK;
}

dsa_status dsa_weights_run(const dsa_weights_plan_t *plan, void *workspace, size_t workspace_bytes, const void *q,
                           int64_t q_stride_t, int64_t q_stride_h, const dsa_cache_desc *cache, const int32_t *slots,
                           int64_t slots_stride, const int32_t *lengths, const int32_t *starts, int32_t window,
                           float scale, const float *sink, const float *lse, const float *scores_in,
                           int64_t in_stride, float *scores_out, int64_t out_stride, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_weights_run");
  if (!plan || plan->magic != dsa::kWeightsMagic || plan->abi_version != DSA_DECODE_ABI_VERSION) return DSA_ERR_PLAN;
  // A step without tokens still copies the scores; a plan of one asks for no
  // workspace, without which there is no status word to report to.
  const bool tokens = plan->num_tokens > 0;
  if (plan->num_seqs == 0 || (!tokens && (!workspace || workspace_bytes < 256))) return DSA_OK;
  if (!slots || !lengths || !starts || !scores_out || (tokens && (!q || !lse))) return DSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || window < 0 || slots_stride < plan->width || out_stride < plan->width ||
      (scores_in && in_stride < plan->width) || (scores_in == scores_out && in_stride != out_stride))
    return DSA_ERR_INVALID_ARG;
  if (tokens && (q_stride_h < plan->d_qk || q_stride_t < (int64_t)(plan->num_heads - 1) * q_stride_h + plan->d_qk))
    return DSA_ERR_INVALID_ARG;
  if ((tokens && (!aligned(q, 16) || q_stride_t % 8 != 0 || q_stride_h % 8 != 0 || !aligned(lse, 4))) ||
      !aligned(slots, 4) || !aligned(lengths, 4) || !aligned(starts, 4) || (sink && !aligned(sink, 4)) || (scores_in && !aligned(scores_in, 4)) ||
      !aligned(scores_out, 4))
    return DSA_ERR_ALIGNMENT;
  if (!workspace || (int64_t)workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256))
    return DSA_ERR_WORKSPACE;
  WeightsParams p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  const dsa_status s = dsa::fill_cache(cache, p.L);
  if (s != DSA_OK) return s;
  if ((cache->format == DSA_REC_V32_656) != (plan->d_qk == 576)) return DSA_ERR_UNSUPPORTED;
  p.L.ids = slots;
  p.L.idx_stride = slots_stride;
  p.L.lens = lengths;
  p.L.width = plan->width;
  p.starts = starts;
  p.T = plan->num_tokens;
  p.B = plan->num_seqs;
  p.H = plan->num_heads;
  p.window = window;
  p.tiles = tokens ? plan->tiles : 0;
  // (records with fp32 scales take products half as fast: the queries' way from L2 keeps up)
  const bool wide = plan->wide_splits > 0 && cache->format != DSA_REC_FP8_528 && cache->format != DSA_REC_V32_656;
  p.span = wide ? 256 : 128;
  p.splits = wide ? plan->wide_splits : plan->splits;
  p.max_items = (int32_t)(((int64_t)plan->width + 127) / 128 * plan->num_seqs * p.splits);
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.lse = lse;
  p.sink = sink;
  p.scale_log2 = scale * dsa::kLog2e;
  p.in = scores_in;
  p.in_st = in_stride;
  p.out = scores_out;
  p.out_st = out_stride;
  p.wait_budget = plan->wait_budget_cycles;
  char *w = static_cast<char *>(workspace);
  p.status = reinterpret_cast<int32_t *>(w);
  p.n_items = p.status + 2;
  p.item = reinterpret_cast<int4 *>(w + plan->ws_item_offset);
  p.image = reinterpret_cast<uint8_t *>(w + plan->ws_image_offset);
  p.row = reinterpret_cast<float *>(w + plan->ws_row_offset);
  p.part = reinterpret_cast<float *>(w + plan->ws_part_offset);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dsa::kDebug && cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return DSA_ERR_CUDA;
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache->format) {
    case DSA_REC_FP8_528: e = launch_weights<DSA_REC_FP8_528>(p, plan->pairs, plan->num_sms, st); break;
    case DSA_REC_NVFP4_288: e = launch_weights<DSA_REC_NVFP4_288>(p, plan->pairs, plan->num_sms, st); break;
    case DSA_REC_FP8_528_UE8M0: e = launch_weights<DSA_REC_FP8_528_UE8M0>(p, plan->pairs, plan->num_sms, st); break;
    case DSA_REC_MODEL1_584: e = launch_weights<DSA_REC_MODEL1_584>(p, plan->pairs, plan->num_sms, st); break;
    case DSA_REC_V32_656: e = launch_weights<DSA_REC_V32_656>(p, plan->pairs, plan->num_sms, st); break;
  }
  return dsa::cuda_status(e);
}

}  // extern "C"

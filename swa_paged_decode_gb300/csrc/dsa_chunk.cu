// dsa_chunk.cu -- attention of chunks of new tokens over paged lists
// (dsa_chunk_plan / dsa_chunk_run): sequence b brings n_b tokens, the last n_b
// entries of its list of L_b records. Token i sits at list position p = L_b -
// n_b + i and attends positions max(0, p - window + 1) .. p:
//
//   s_j = scale q . k_j,  lse = log sum_j e^{s_j},  O = sum_j e^{s_j - lse} v_j,
//
// with the state of another list and the sink as in dsa_prefix_run. The kernels
// are those of dsa_attend.cuh, and so are the roundings to 16 bits. What differs
// is where the work is, found on the device, since lengths and starts are there:
//
//   gather  the records that some token of their sequence attends, by blocks that
//           stay and take groups of 32 in turn (a block per group of every
//           list's width would mostly start for nothing); block 0 lays out the
//           row tiles (128 query rows of one sequence), their units (256 keys)
//           and the pairs' ranges, equal in cost, instead;
//   attend  units start at the half tile of the tile's first key; the keys that
//           a row may not see are masked like unused slots, by two words per
//           thread and unit;
//   merge   the rows of tiles that pairs share and of tiles without keys, from a
//           list that block 0 leaves too.
//
// What bounds it. Long lists: as the shared prefix, the products (1024 tokens x 128
// heads over 16384 records 2.37 ms alone, 1800 TFLOP/s, 0.94 of the measured
// peak). Windows: the chain of one tile after the other on a pair, 17000 cycles for
// 2 tokens x 64 heads and 128 keys, of which the products are 4500 (3400 tokens 235
// us; 361 with the output through fp32 in shared memory, the rotation in four
// lanes and a merge over all rows). Few tokens: three dependent kernels (21.1 us).
#include "dsa_attend.cuh"

namespace dsa {

constexpr int32_t kChunkMagic = 0x43415344;   // "DSAC"
constexpr int kChThreads = 256;

__device__ __forceinline__ Sequence load_sequence(const ChunkParams &p, int32_t b) {
  const int32_t s0 = __ldg(p.starts + b), s1 = __ldg(p.starts + b + 1), len = __ldg(p.L.lens + b);
  return {s0, s1 - s0, min(max(len, 0), p.L.width), p.window};
}
// Starts ascend within [0, T]; a call whose starts do not has no work.
__device__ __forceinline__ bool starts_ok(const ChunkParams &p) {
  bool bad = false;
  for (int32_t b = threadIdx.x; b < p.B; b += kChThreads) {
    const int32_t s0 = __ldg(p.starts + b), s1 = __ldg(p.starts + b + 1);
    bad |= s0 < 0 || s1 < s0 || s1 > p.T;
  }
  return !__syncthreads_or(bad);
}
// Sums of the threads up to this one, and of all; w: shared, a word per warp.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *w, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t v = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += y;
  }
  __syncthreads();   // (w free)
  if (lane == 31) w[warp] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int k = 0; k < kChThreads / 32; ++k) {
    if (k < warp) v += w[k];
    total += w[k];
  }
  return v;
}

// Row tiles (those with keys first), their units, and the pairs' ranges: block 0
// of the gather. A unit costs 1 and a tile with any `tile_cost` more
// (dsa_prefix_index.cuh).
__device__ void lay_out(const ChunkParams &p, bool ok) {
  __shared__ int64_t w_s[kChThreads / 32];
  const int tid = threadIdx.x;
  int64_t tiles = 0;
  if (tid == 0) *p.n_merge = 0;
  __syncthreads();
  if (ok) {
    for (int32_t b0 = 0; b0 < p.B; b0 += kChThreads) {
      const int32_t b = b0 + tid;
      const int32_t n = b < p.B ? load_sequence(p, b).tiles(p.H) : 0;
      int64_t sum;
      const int64_t upto = block_scan(n, w_s, sum);
      if (b < p.B) p.seq_tile[b] = (int32_t)(tiles + upto - n);
      tiles += sum;
    }
    __syncthreads();   // seq_tile
  }
  // (a bound of the plan, which starts that ascend keep)
  const int32_t R = (int32_t)min(tiles, (int64_t)p.R);
  const int32_t t0 = (int32_t)((int64_t)R * tid / kChThreads), t1 = (int32_t)((int64_t)R * (tid + 1) / kChThreads);
  int32_t b_first = 0;   // the last sequence that starts at or before tile t0 (those without tiles come before it)
  if (t0 < t1) {
    int32_t hi = p.B - 1;
    while (b_first < hi) {
      const int32_t mid = (b_first + hi + 1) >> 1;
      if (p.seq_tile[mid] <= t0) b_first = mid; else hi = mid - 1;
    }
  }
  // Twice over the thread's tiles: their costs, then, with the costs before
  // them known, their records and the pairs that begin in them.
  int64_t units = 0, live = 0;
  auto each = [&](auto &&f) {
    if (t0 >= t1) return;
    int32_t b = b_first, first = p.seq_tile[b];
    Sequence s = load_sequence(p, b);
    for (int32_t t = t0; t < t1; ++t) {
      while (t >= first + s.tiles(p.H)) {
        s = load_sequence(p, ++b);
        first = p.seq_tile[b];
      }
      int32_t half;
      const int32_t u = s.tile_units(p.H, t - first, half);
      f(t, b, s, t - first, half, u);
    }
  };
  each([&](int32_t, int32_t, const Sequence &, int32_t, int32_t, int32_t u) {
    units += u;
    live += u > 0 ? 1 : 0;
  });
  int64_t all_units, all_live;
  const int64_t before_u = block_scan(units, w_s, all_units) - units;
  const int64_t before_l = block_scan(live, w_s, all_live) - live;
  const int64_t tile_cost = all_units >= 2 * (int64_t)p.C ? 2 : 0, total = all_units + tile_cost * all_live;
  int64_t at = before_u + tile_cost * before_l, l = before_l;
  each([&](int32_t t, int32_t b, const Sequence &s, int32_t i, int32_t half, int32_t u) {
    const int32_t to = tile_place(t, u, l, all_live);
    p.row_tile[2 * (int64_t)to] = make_int4(s.s0 * p.H + 128 * i, s.tile_rows(p.H, i), u, 0);
    p.row_tile[2 * (int64_t)to + 1] = make_int4(b * p.seq_halves + half, half * 128, s.len - s.n - s.s0, 0);
    if (u == 0) {
      p.merge[atomicAdd(p.n_merge, 1)] = to;
      return;
    }
    ++l;
    bool shared = false;   // (the list's order does not matter)
    pairs_in_tile(at, u, tile_cost, total, p.C, [&](int32_t c, int32_t w) {
      p.begin[c] = make_int2(to, w);
      shared |= w > 0;
    });
    if (shared) p.merge[atomicAdd(p.n_merge, 1)] = to;
    at += u + tile_cost;
  });
  if (total == 0)
    for (int32_t c = tid; c < p.C; c += kChThreads) p.begin[c] = make_int2(0, 0);
  if (tid == 0) p.begin[p.C] = make_int2((int32_t)all_live, 0);
}

template <int FMT>
__global__ void __launch_bounds__(kChThreads) chunk_gather_kernel(ChunkParams p) {
  __shared__ int32_t e_s[kPfGroup];
  __shared__ int64_t w_s[kChThreads / 32];
  __shared__ int64_t upto_s[kChThreads];
  __shared__ int2 seq_s[kChThreads];   // (first group, list length)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!kDebug && blockIdx.x == 0 && tid == 0) *p.status = DSA_OK;
  pdl_launch_dependents();
  const bool ok = starts_ok(p);
  if (blockIdx.x == 0) {
    if (!ok && tid == 0) report_status(p.status, DSA_ERR_INVALID_ARG);
    lay_out(p, ok);
    return;
  }
  if (!ok) return;
  // groups of 32 keys of 256 sequences at a time; this block takes every
  // (gridDim.x - 1)th of all
  int64_t item = blockIdx.x - 1, before = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kChThreads) {
    int64_t mine = 0, sum;
    if (b0 + tid < p.B) {
      const Sequence s = load_sequence(p, b0 + tid);
      if (s.any()) mine = 4 * (s.gather_end() - s.gather_begin());
      seq_s[tid] = make_int2(s.any() ? 4 * s.gather_begin() : 0, s.len);
    }
    upto_s[tid] = block_scan(mine, w_s, sum);
    __syncthreads();
    for (; item < before + sum; item += gridDim.x - 1) {
      const int64_t x = item - before;
      int lo = 0, hi = min(kChThreads, p.B - b0) - 1;   // the sequence whose groups hold x
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto_s[mid] > x) hi = mid; else lo = mid + 1;
      }
      const int2 q = seq_s[lo];
      const int32_t g = q.x + (int32_t)(x - (lo > 0 ? upto_s[lo - 1] : 0)), key0 = g * kPfGroup;
      const int32_t *ids = p.L.ids + (int64_t)(b0 + lo) * p.L.idx_stride;
      int32_t slot = -1;
      if (lane < 4 && key0 + 4 * warp + lane < q.y) slot = __ldg(ids + key0 + 4 * warp + lane);
      const int64_t group = (int64_t)(b0 + lo) * p.seq_halves * 4 + g;
      if (dbg_ok(p.status, group >= 0 && group < 4 * p.halves, kDbgPartial))
        gather_group<FMT, true>(p, slot, key0, q.y, group, e_s);
      __syncthreads();   // e_s
    }
    before += sum;
  }
}

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::ChunkParams;

template <int FMT>
cudaError_t launch_chunk(const ChunkParams &p, int32_t num_sms, cudaStream_t st) {
  using namespace dsa;
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  cudaError_t e = attend_ready<kV32, true>();
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!image_map(p.image, p.halves * 128 * (kV32 ? 1152 : 1024), &map)) return cudaErrorNotSupported;
  const int64_t groups = 4 * p.halves;
  const unsigned blocks = (unsigned)std::min<int64_t>(groups, 8 * (int64_t)num_sms);
  chunk_gather_kernel<FMT><<<blocks + 1, kChThreads, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(config(2u * p.C, kPfThreads, PfCfg<kV32>::kSmem, st), prefix_attend_kernel<kV32, true>, p, map);
  if (e != cudaSuccess) return e;
  // as for a prefix: few parts to a row by a warp, many by a block
  const unsigned most = (unsigned)std::min(p.R, p.C);
  if (p.C < 8 * p.R) return launch_dependent(config(32u * most, 128, 0, st), prefix_merge_kernel<32, 1, true>, p);
  return launch_dependent(config(128u * most, 256, 0, st), prefix_merge_kernel<128, 2, true>, p);
}

}  // namespace

extern "C" {

dsa_status dsa_chunk_plan(int32_t num_tokens, int32_t num_seqs, int32_t num_heads, int32_t width, int32_t num_sms,
                          int32_t d_qk, dsa_chunk_plan_t *plan, size_t *workspace_bytes) {
  if (!plan || !workspace_bytes) return DSA_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_seqs < 0 || num_heads < 1 || width < 1 || num_sms < 0) return DSA_ERR_INVALID_ARG;
  if (d_qk != 512 && d_qk != 576) return DSA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)num_tokens * num_heads, seq_halves = dsa::chunk_seq_halves(width);
  // (rows are counted in 31 bits; the images' map counts 512-byte rows in them,
  // 288 to a half; 2^24 row tiles keep the merge's grid within its limit)
  if (rows > INT32_MAX - 128 || num_seqs > (1 << 24) || width > (1 << 29) ||
      seq_halves * (num_seqs > 0 ? num_seqs : 1) > INT32_MAX / 288 - 2)
    return DSA_ERR_UNSUPPORTED;
  const int64_t row_tiles = dsa::chunk_row_tiles(num_tokens, num_heads, num_seqs);
  if (row_tiles >= 1 << 24) return DSA_ERR_UNSUPPORTED;
  int pairs = num_sms / 2;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        (d_qk == 576 ? dsa::resident_pairs<true, true>(&pairs) : dsa::resident_pairs<false, true>(&pairs)) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->magic = dsa::kChunkMagic;
  plan->abi_version = DSA_DECODE_ABI_VERSION;
  plan->num_tokens = num_tokens;
  plan->num_seqs = num_seqs;
  plan->num_heads = num_heads;
  plan->width = width;
  plan->d_qk = d_qk;
  plan->num_sms = num_sms;
  plan->row_tiles = (int32_t)row_tiles;
  plan->seq_halves = (int32_t)seq_halves;
  // one pair per unit at most
  const int64_t units = row_tiles * ((width + dsa::kPfTile - 1) / dsa::kPfTile);
  pairs = pairs < 1 ? 1 : pairs;
  plan->pairs = units < pairs ? (int32_t)(units < 1 ? 1 : units) : pairs;
  // Workspace: status | group info | key exponents | images | row tiles | their
  // sequences' first | ranges | tile | part_lse | part_o
  const int64_t keys = 128 * seq_halves * num_seqs, slots = 2 * (int64_t)plan->pairs * 128;
  int64_t off = 256;
  auto take = [&](int64_t &at, int64_t bytes) {
    at = off;
    off = dsa::align_up(off + bytes, 256);
  };
  take(plan->ws_info_offset, 8 * (keys / dsa::kPfGroup));
  take(plan->ws_key_e_offset, 4 * keys);
  take(plan->ws_image_offset, keys * d_qk * 2);
  take(plan->ws_row_tile_offset, 32 * row_tiles);
  take(plan->ws_seq_tile_offset, 4 * (int64_t)num_seqs);
  take(plan->ws_begin_offset, 8 * ((int64_t)plan->pairs + 1));
  take(plan->ws_tile_offset, 12 * row_tiles);   // (and the list of tiles to merge)
  take(plan->ws_part_lse_offset, 4 * slots);
  take(plan->ws_part_o_offset, 4 * slots * dsa::kD);
  plan->workspace_bytes = num_tokens == 0 || num_seqs == 0 ? 0 : off;
  // Test knob, read only here, as in dsa_decode_plan.
  if (const char *wb = std::getenv("DSA_DECODE_WAIT_BUDGET")) {
    const long long v = std::atoll(wb);
    if (v > 0) plan->wait_budget_cycles = v;
  }
  *workspace_bytes = (size_t)plan->workspace_bytes;
  return DSA_OK;
}

dsa_status dsa_chunk_run(const dsa_chunk_plan_t *plan, void *workspace, size_t workspace_bytes, const void *q,
                         int64_t q_stride_t, int64_t q_stride_h, const dsa_cache_desc *cache, const int32_t *slots,
                         int64_t slots_stride, const int32_t *lengths, const int32_t *starts, int32_t window,
                         const float *sink, const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows,
                         int32_t rope_style, float scale, const void *tail_out, const float *tail_lse, void *out,
                         float *lse, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_chunk_run");
  if (!plan || plan->magic != dsa::kChunkMagic || plan->abi_version != DSA_DECODE_ABI_VERSION) return DSA_ERR_PLAN;
  if (plan->num_tokens == 0 || plan->num_seqs == 0) return DSA_OK;
  if (!q || !slots || !lengths || !starts || !out || !lse) return DSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || window < 0 || slots_stride < plan->width) return DSA_ERR_INVALID_ARG;
  if (rope_style != DSA_ROPE_NEOX && rope_style != DSA_ROPE_GPTJ) return DSA_ERR_INVALID_ARG;
  if (q_stride_h < plan->d_qk || q_stride_t < (int64_t)(plan->num_heads - 1) * q_stride_h + plan->d_qk)
    return DSA_ERR_INVALID_ARG;
  if ((positions == nullptr) != (cos_sin == nullptr)) return DSA_ERR_INVALID_ARG;
  if (cos_sin && cos_sin_rows < 1) return DSA_ERR_INVALID_ARG;
  if ((tail_out == nullptr) != (tail_lse == nullptr)) return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride_t % 8 != 0 || q_stride_h % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(slots, 4) || !aligned(lengths, 4) || !aligned(starts, 4) || (sink && !aligned(sink, 4)) ||
      (cos_sin && (!aligned(cos_sin, 16) || !aligned(positions, 8))) ||
      (tail_out && (!aligned(tail_out, 16) || !aligned(tail_lse, 4))))
    return DSA_ERR_ALIGNMENT;
  if (!workspace || (int64_t)workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256))
    return DSA_ERR_WORKSPACE;
  ChunkParams p;
  std::memset(static_cast<void *>(&p), 0, sizeof(p));
  const dsa_status s = dsa::fill_cache(cache, p.L);
  if (s != DSA_OK) return s;
  // V3.2 records go with 576-dim queries and no table, as in dsa_decode_run
  if ((cache->format == DSA_REC_V32_656) != (plan->d_qk == 576)) return DSA_ERR_UNSUPPORTED;
  if (plan->d_qk == 576 && cos_sin) return DSA_ERR_UNSUPPORTED;
  p.L.ids = slots;
  p.L.idx_stride = slots_stride;
  p.L.lens = lengths;
  p.L.width = plan->width;
  p.starts = starts;
  p.T = plan->num_tokens;
  p.B = plan->num_seqs;
  p.window = window;
  p.seq_halves = plan->seq_halves;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.sink = sink;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.cs_rows = cos_sin_rows;
  p.gptj = rope_style == DSA_ROPE_GPTJ ? 1 : 0;
  p.scale_log2 = scale * dsa::kLog2e;
  p.tail_out = static_cast<const __nv_bfloat16 *>(tail_out);
  p.tail_lse = tail_lse;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.H = plan->num_heads;
  p.rows = plan->num_tokens * plan->num_heads;
  p.R = plan->row_tiles;
  p.halves = (int64_t)plan->seq_halves * plan->num_seqs;
  p.C = plan->pairs;
  p.wait_budget = plan->wait_budget_cycles;
  char *w = static_cast<char *>(workspace);
  p.status = reinterpret_cast<int32_t *>(w);
  p.info = reinterpret_cast<int2 *>(w + plan->ws_info_offset);
  p.key_e = reinterpret_cast<int32_t *>(w + plan->ws_key_e_offset);
  p.image = reinterpret_cast<uint8_t *>(w + plan->ws_image_offset);
  p.row_tile = reinterpret_cast<int4 *>(w + plan->ws_row_tile_offset);
  p.seq_tile = reinterpret_cast<int32_t *>(w + plan->ws_seq_tile_offset);
  p.begin = reinterpret_cast<int2 *>(w + plan->ws_begin_offset);
  p.tile = reinterpret_cast<int2 *>(w + plan->ws_tile_offset);
  p.merge = reinterpret_cast<int32_t *>(p.tile + p.R);
  p.n_merge = p.status + 2;
  p.part_lse = reinterpret_cast<float *>(w + plan->ws_part_lse_offset);
  p.part_o = reinterpret_cast<float *>(w + plan->ws_part_o_offset);
  p.check_rows = p.rows;
  p.check_parts = 256 * (int64_t)p.C;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dsa::kDebug && cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return DSA_ERR_CUDA;
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache->format) {
    case DSA_REC_FP8_528: e = launch_chunk<DSA_REC_FP8_528>(p, plan->num_sms, st); break;
    case DSA_REC_NVFP4_288: e = launch_chunk<DSA_REC_NVFP4_288>(p, plan->num_sms, st); break;
    case DSA_REC_FP8_528_UE8M0: e = launch_chunk<DSA_REC_FP8_528_UE8M0>(p, plan->num_sms, st); break;
    case DSA_REC_MODEL1_584: e = launch_chunk<DSA_REC_MODEL1_584>(p, plan->num_sms, st); break;
    case DSA_REC_V32_656: e = launch_chunk<DSA_REC_V32_656>(p, plan->num_sms, st); break;
  }
  return dsa::cuda_status(e);
}

}  // extern "C"

// dsa_prefix.cu -- attention of a whole decode batch over one shared list of
// records (dsa_prefix_plan / dsa_prefix_run): T tokens x H heads = `rows`
// query rows against P keys, every key gathered and dequantized once.
//
//   s_rj = scale q_r . k_j,  lse_r = log sum_j e^{s_rj},
//   O_r = sum_j e^{s_rj - lse_r} v_j     (v_j = dims 0..511 of k_j)
//
// and, with the state (O', lse') of the token's own list and the sink z,
//   lse = log(e^{lse_r} + e^{lse'}),
//   out = (e^{lse_r} O_r + e^{lse'} O') / (e^lse + e^z).
//
// Three launches, each the programmatic dependent of the one before it:
//   gather  32 records per block -> f16 tile images in the workspace, each
//           value times 2^-E, E the exponent of the 32 keys' largest value
//           (one per key where their magnitudes differ by more than 2^5);
//   attend  pairs of CTAs (tcgen05 cta_group::2) on 128 query rows, a range
//           of (row tile, key tile) units per pair;
//   merge   the rows whose key tiles were split over pairs, and the rows of
//           an empty prefix.
//
// Roundings to 16 bits, as in the decode kernel: keys, queries and weights are
// f16 operands of the tensor core (11 bits; bf16 has 8, and tf32 runs at half
// the rate with operands twice the size), each with a power of two of its own
// (a key or 32 of them, a query row, a row's weights) so that f16's range is no
// limit. Codes times a power of two or an e4m3 scale are exact in them, and
// unrotated queries but for elements below 2^-17 of the row's largest; codes
// times an fp32 scale are off by 2^-11, which shows as 1 to 2e-6 of lse. Scores,
// sums, partials and lse are fp32. The tail is the bf16 output of the decode.
#include "dsa_attend.cuh"

namespace dsa {

constexpr int32_t kPrefixMagic = 0x50415344;   // "DSAP"

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::PrefixParams;

bool prefix_plan_ok(const dsa_prefix_plan_t *plan) {
  return plan && plan->magic == dsa::kPrefixMagic && plan->abi_version == DSA_DECODE_ABI_VERSION;
}

template <int FMT>
cudaError_t launch_prefix(const PrefixParams &p, cudaStream_t st) {
  using namespace dsa;
  constexpr bool kV32 = FMT == DSA_REC_V32_656;
  cudaError_t e = attend_ready<kV32, false>();
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)((p.L.width + kPfTile - 1) / kPfTile);
  CUtensorMap map;
  if (!image_map(p.image, (int64_t)tiles * kPfTile * (kV32 ? 1152 : 1024), &map)) return cudaErrorNotSupported;
  prefix_gather_kernel<FMT><<<tiles * (kPfTile / kPfGroup), 256, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(config(2u * p.C, kPfThreads, PfCfg<kV32>::kSmem, st), prefix_attend_kernel<kV32, false>, p, map);
  if (e != cudaSuccess) return e;
  // about C / R + 1 parts to a row: up to 9 by a warp, more by a block
  if (p.C < 8 * p.R)
    return launch_dependent(config((unsigned)((p.rows + 3) / 4), 128, 0, st), prefix_merge_kernel<32, 1, false>, p);
  return launch_dependent(config((unsigned)p.rows, 256, 0, st), prefix_merge_kernel<128, 2, false>, p);
}

}  // namespace

extern "C" {

dsa_status dsa_prefix_plan(int32_t num_tokens, int32_t num_heads, int32_t width, int32_t num_sms,
                           int32_t d_qk, dsa_prefix_plan_t *plan, size_t *workspace_bytes) {
  if (!plan || !workspace_bytes) return DSA_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_heads < 1 || width < 1 || num_sms < 0) return DSA_ERR_INVALID_ARG;
  if (d_qk != 512 && d_qk != 576) return DSA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)num_tokens * num_heads;
  // (the images' map counts 512-byte rows in 31 bits)
  if (rows > INT32_MAX - 128 || width > (1 << 29)) return DSA_ERR_UNSUPPORTED;
  int pairs = num_sms / 2;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        (d_qk == 576 ? dsa::resident_pairs<true, false>(&pairs) : dsa::resident_pairs<false, false>(&pairs)) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->magic = dsa::kPrefixMagic;
  plan->abi_version = DSA_DECODE_ABI_VERSION;
  plan->num_tokens = num_tokens;
  plan->num_heads = num_heads;
  plan->width = width;
  plan->d_qk = d_qk;
  plan->num_sms = num_sms;
  plan->row_tiles = (int32_t)((rows + 127) / 128);
  plan->key_tiles = (width + dsa::kPfTile - 1) / dsa::kPfTile;
  // one pair per unit at most
  const int64_t units = (int64_t)plan->row_tiles * plan->key_tiles;
  pairs = pairs < 1 ? 1 : pairs;
  plan->pairs = units < pairs ? (int32_t)(units < 1 ? 1 : units) : pairs;
  // Workspace: status | group info | key exponents | images | tile | part_lse | part_o
  const int64_t keys = (int64_t)plan->key_tiles * dsa::kPfTile, slots = 2 * (int64_t)plan->pairs * 128;
  int64_t off = 256;
  plan->ws_info_offset = off;
  off = dsa::align_up(off + 8 * (keys / dsa::kPfGroup), 256);
  plan->ws_key_e_offset = off;
  off = dsa::align_up(off + 4 * keys, 256);
  plan->ws_image_offset = off;
  off += keys * d_qk * 2;
  plan->ws_tile_offset = off;
  off = dsa::align_up(off + 8 * (int64_t)plan->row_tiles, 256);
  plan->ws_part_lse_offset = off;
  off = dsa::align_up(off + 4 * slots, 256);
  plan->ws_part_o_offset = off;
  off += 4 * slots * dsa::kD;
  plan->workspace_bytes = num_tokens == 0 ? 0 : off;
  // Test knob, read only here, as in dsa_decode_plan.
  if (const char *wb = std::getenv("DSA_DECODE_WAIT_BUDGET")) {
    const long long v = std::atoll(wb);
    if (v > 0) plan->wait_budget_cycles = v;
  }
  *workspace_bytes = (size_t)plan->workspace_bytes;
  return DSA_OK;
}

dsa_status dsa_prefix_run(const dsa_prefix_plan_t *plan, void *workspace, size_t workspace_bytes,
                          const void *q, int64_t q_stride_t, int64_t q_stride_h,
                          const dsa_cache_desc *cache, const int32_t *slots, const int32_t *length,
                          const float *sink, const int64_t *positions, const float *cos_sin,
                          int64_t cos_sin_rows, int32_t rope_style, float scale,
                          const void *tail_out, const float *tail_lse, void *out, float *lse,
                          dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_prefix_run");
  if (!prefix_plan_ok(plan)) return DSA_ERR_PLAN;
  if (plan->num_tokens == 0) return DSA_OK;
  if (!q || !slots || !length || !out || !lse) return DSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return DSA_ERR_INVALID_ARG;
  if (rope_style != DSA_ROPE_NEOX && rope_style != DSA_ROPE_GPTJ) return DSA_ERR_INVALID_ARG;
  if (q_stride_h < plan->d_qk || q_stride_t < (int64_t)(plan->num_heads - 1) * q_stride_h + plan->d_qk)
    return DSA_ERR_INVALID_ARG;
  if ((positions == nullptr) != (cos_sin == nullptr)) return DSA_ERR_INVALID_ARG;
  if (cos_sin && cos_sin_rows < 1) return DSA_ERR_INVALID_ARG;
  if ((tail_out == nullptr) != (tail_lse == nullptr)) return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride_t % 8 != 0 || q_stride_h % 8 != 0 || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(slots, 4) || !aligned(length, 4) || (sink && !aligned(sink, 4)) ||
      (cos_sin && (!aligned(cos_sin, 16) || !aligned(positions, 8))) ||
      (tail_out && (!aligned(tail_out, 16) || !aligned(tail_lse, 4))))
    return DSA_ERR_ALIGNMENT;
  if (!workspace || (int64_t)workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256))
    return DSA_ERR_WORKSPACE;
  PrefixParams p;
  std::memset(&p, 0, sizeof(p));
  const dsa_status s = dsa::fill_cache(cache, p.L);
  if (s != DSA_OK) return s;
  // V3.2 records go with 576-dim queries and no table, as in dsa_decode_run
  if ((cache->format == DSA_REC_V32_656) != (plan->d_qk == 576)) return DSA_ERR_UNSUPPORTED;
  if (plan->d_qk == 576 && cos_sin) return DSA_ERR_UNSUPPORTED;
  p.L.ids = slots;
  p.L.lens = length;
  p.L.width = plan->width;
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
  p.halves = 2 * (int64_t)plan->key_tiles;
  p.C = plan->pairs;
  p.wait_budget = plan->wait_budget_cycles;
  char *w = static_cast<char *>(workspace);
  p.status = reinterpret_cast<int32_t *>(w);
  p.info = reinterpret_cast<int2 *>(w + plan->ws_info_offset);
  p.key_e = reinterpret_cast<int32_t *>(w + plan->ws_key_e_offset);
  p.image = reinterpret_cast<uint8_t *>(w + plan->ws_image_offset);
  p.tile = reinterpret_cast<int2 *>(w + plan->ws_tile_offset);
  p.part_lse = reinterpret_cast<float *>(w + plan->ws_part_lse_offset);
  p.part_o = reinterpret_cast<float *>(w + plan->ws_part_o_offset);
  p.check_rows = p.rows;
  p.check_parts = 256 * (int64_t)p.C;
#ifdef DSA_DEBUG
  // Checking build only, test knobs: fewer rows than there are; the accesses
  // past them are reported and left out.
  if (const char *v = std::getenv("DSA_DEBUG_CHECK_ROWS")) p.check_rows = std::min<int64_t>(p.check_rows, std::atoll(v));
  if (const char *v = std::getenv("DSA_DEBUG_CHECK_PARTS")) p.check_parts = std::min<int64_t>(p.check_parts, std::atoll(v));
#endif
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dsa::kDebug && cudaMemsetAsync(workspace, 0, 8, st) != cudaSuccess) return DSA_ERR_CUDA;
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache->format) {
    case DSA_REC_FP8_528: e = launch_prefix<DSA_REC_FP8_528>(p, st); break;
    case DSA_REC_NVFP4_288: e = launch_prefix<DSA_REC_NVFP4_288>(p, st); break;
    case DSA_REC_FP8_528_UE8M0: e = launch_prefix<DSA_REC_FP8_528_UE8M0>(p, st); break;
    case DSA_REC_MODEL1_584: e = launch_prefix<DSA_REC_MODEL1_584>(p, st); break;
    case DSA_REC_V32_656: e = launch_prefix<DSA_REC_V32_656>(p, st); break;
  }
  return dsa::cuda_status(e);
}

}  // extern "C"

// dsa_evict.cu -- every list cut to a budget of records by their accumulated
// weights (dsa_evict): of a list of n > budget entries the first keep_first and
// the last keep_last stay, and of those between the ones with the largest
// scores, in the list's order; the others' slots are given back.
//
// A cluster of CTAs per list, each with a run of it. Scores are read once, into
// shared memory where the run fits there (else again from the L2 in every pass).
// The place of the cut is found by a radix selection over their bits (11, 11 and
// 10 of them: three histograms, each added up over the cluster in the shared memory
// of its first CTA), then every warp walks its own run of entries with ballots,
// knowing from the counts before it where its entries go: no CTA waits for another
// one there, and the order does not depend on timing. All of it is latency: a
// launch, three histograms and two walks for 32 lists of 2048 (8.8 us), eight
// cluster barriers and 512 entries to a warp for 16 of 65521 (23 us; 51 with
// scores compared as floats, every CTA reading the sums and slots loaded 32 at a
// time).
#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>

#include "dsa_host.cuh"

namespace dsa {
namespace cg = cooperative_groups;

constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;   // (two CTAs to an SM: clusters of 8 find a place each)
constexpr int kEvBins = 2048;
constexpr int kEvCached = 40960;   // scores that a CTA holds (160 KiB)

struct EvictParams {
  const int32_t *slots;
  int64_t slots_st;
  const int32_t *lengths;
  const float *scores;
  int64_t scores_st;
  int32_t width, budget, first, last;
  int32_t *kept;
  int64_t kept_st;
  float *kept_scores;
  int64_t kept_scores_st;
  int32_t *kept_lengths;
  int32_t *freed;          // null: not wanted
  int64_t freed_st;
  int32_t *freed_counts;
};

// Scores in the order of their ranks: a NaN below all numbers, -0 as 0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  if ((b & 0x7FFFFFFFu) == 0u) return 0x80000000u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The score of a rank, but for NaN and -0, which are read again.
__device__ __forceinline__ float score_of(uint32_t r, const float *score) {
  if (r == 0u || r == 0x80000000u) return __ldg(score);
  return __uint_as_float((r & 0x80000000u) ? r ^ 0x80000000u : ~r);
}

// kHeld: the ranks of the CTA's scores lie in its shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(kEvThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t cache_s[];
  __shared__ uint32_t hist_s[kEvBins];          // this CTA's
  __shared__ __align__(16) uint32_t total_s[3][kEvBins];   // first CTA: the cluster's, per pass
  __shared__ uint32_t scan_s[kEvWarps];
  __shared__ uint32_t pick_s[3][2];             // first CTA: chosen bin, entries above it, per pass
  __shared__ uint32_t count_s[kEvWarps][2];     // per warp: entries above the cut, at the cut
  __shared__ uint32_t sum_s[2];                 // and of the CTA
  cg::cluster_group cluster = cg::this_cluster();
  const int32_t rank = (int32_t)cluster.block_rank(), size = (int32_t)cluster.num_blocks();
  const int32_t seq = blockIdx.x / size;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t n = min(max(__ldg(p.lengths + seq), 0), p.width), keep = min(p.budget, n);
  const int32_t *slots = p.slots + seq * p.slots_st;
  const float *scores = p.scores + seq * p.scores_st;
  int32_t *kept = p.kept + seq * p.kept_st;
  float *kept_scores = p.kept_scores + seq * p.kept_scores_st;
  int32_t *freed = p.freed ? p.freed + seq * p.freed_st : nullptr;
  if (rank == 0 && tid == 0) {
    p.kept_lengths[seq] = keep;
    if (p.freed_counts) p.freed_counts[seq] = n - keep;
  }
  if (n <= p.budget) {   // the whole cluster: everything stays
    for (int32_t i = rank * kEvThreads + tid; i < n; i += size * kEvThreads) {
      kept[i] = __ldg(slots + i);
      kept_scores[i] = __ldg(scores + i);
    }
    return;
  }
  const int32_t lo = min(p.first, keep), hi = n - min(p.last, keep - lo);   // entries lo .. hi - 1 compete
  const uint32_t want = (uint32_t)(keep - lo - (n - hi));                   // for this many places
  // this CTA's run, and of it the warp's
  const int32_t c0 = (int32_t)((int64_t)n * rank / size), c1 = (int32_t)((int64_t)n * (rank + 1) / size);
  const int32_t w0 = c0 + (int32_t)((int64_t)(c1 - c0) * warp / kEvWarps);
  const int32_t w1 = c0 + (int32_t)((int64_t)(c1 - c0) * (warp + 1) / kEvWarps);
  auto rank_at = [&](int32_t i) { return kHeld ? cache_s[i - c0] : rank_of(__ldg(scores + i)); };
  constexpr int kBatch = 8;
  int32_t slot[kBatch];
  auto fetch = [&](int32_t i8) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t i = i8 + 32 * k + lane;
      slot[k] = i < w1 ? __ldg(slots + i) : 0;
    }
  };
  fetch(w0);
  for (int k = tid; k < kEvBins; k += kEvThreads) {
    hist_s[k] = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) total_s[pass][k] = 0;
  }
  if constexpr (kHeld) {
#pragma unroll 8
    for (int32_t i = w0 + lane; i < w1; i += 32) cache_s[i - c0] = rank_of(__ldg(scores + i));
  }
  cluster.sync();
  uint32_t cut = 0, left = want;   // the cut's bits so far; places below what lies above them
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t mask = (1u << bits) - 1u;
#pragma unroll 8
      for (int32_t i = max(w0, lo) + lane; i < min(w1, hi); i += 32) {
        const uint32_t r = rank_at(i);
        // (bits above this pass's: none in the first)
        if (pass == 0 || (r >> (shift + bits)) == (cut >> (shift + bits))) atomicAdd(&hist_s[(r >> shift) & mask], 1u);
      }
      __syncthreads();
      uint32_t *total = cluster.map_shared_rank(&total_s[pass][0], 0);
      for (int k = tid; k < kEvBins; k += kEvThreads) {
        const uint32_t x = hist_s[k];
        if (x) atomicAdd(total + k, x);
        hist_s[k] = 0;
      }
      cluster.sync();
      if (rank == 0) {
        // the bin that holds the `left`th entry from the top: thread t has bins
        // 2047 - 4 t .. 2044 - 4 t (found once: 8 CTAs reading the sums took 3000
        // cycles)
        const uint4 t4 = reinterpret_cast<const uint4 *>(total_s[pass])[kEvBins / 4 - 1 - tid];
        const uint32_t b[4] = {t4.w, t4.z, t4.y, t4.x}, mine = (b[0] + b[1]) + (b[2] + b[3]);
        uint32_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        if (lane == 31) scan_s[warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? scan_s[lane] : 0u);
        uint32_t above = upto - mine;
        if (above < left && left <= upto) {   // one thread
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (above < left && left <= above + b[k]) {
              pick_s[pass][0] = kEvBins - 1 - 4 * tid - k;
              pick_s[pass][1] = above;
            }
            above += b[k];
          }
        }
      }
      cluster.sync();
      const uint32_t *pick = cluster.map_shared_rank(&pick_s[pass][0], 0);
      cut |= pick[0] << shift;
      left -= pick[1];
    }
  }
  // `left` of the entries at the cut stay, the first ones; none with want = 0
  // (cut 0 would let all in: nothing is above a cut that nothing reaches).
  auto above_cut = [&](int32_t i, uint32_t r) { return i < lo || i >= hi || (want > 0 && r > cut); };
  uint32_t n_above = 0, n_at = 0;
#pragma unroll 8
  for (int32_t i = w0 + lane; i < w1; i += 32) {
    const uint32_t r = rank_at(i);
    const bool a = above_cut(i, r);
    n_above += a ? 1 : 0;
    n_at += !a && want > 0 && r == cut ? 1 : 0;
  }
  n_above = __reduce_add_sync(0xffffffffu, n_above);
  n_at = __reduce_add_sync(0xffffffffu, n_at);
  if (lane == 0) {
    count_s[warp][0] = n_above;
    count_s[warp][1] = n_at;
  }
  __syncthreads();
  if (warp < 2) {
    const uint32_t x = __reduce_add_sync(0xffffffffu, lane < kEvWarps ? count_s[lane][warp] : 0u);
    if (lane == 0) sum_s[warp] = x;
  }
  cluster.sync();
  uint32_t above = 0, at = 0;   // before the warp's run
  for (int32_t k = 0; k < rank; ++k) {
    const uint32_t *s = cluster.map_shared_rank(sum_s, k);
    above += s[0];
    at += s[1];
  }
  cluster.barrier_arrive();     // (no CTA ends while another one reads its counts)
  above += __reduce_add_sync(0xffffffffu, lane < warp ? count_s[lane][0] : 0u);
  at += __reduce_add_sync(0xffffffffu, lane < warp ? count_s[lane][1] : 0u);
  const uint32_t before = (1u << lane) - 1u;
  // 8 x 32 entries at a time, their slots' loads in flight together (the first
  // ones since the beginning)
#pragma unroll 1
  for (int32_t i8 = w0; i8 < w1; i8 += 32 * kBatch) {
    if (i8 > w0) fetch(i8);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i8 + 32 * k >= w1) break;
      const int32_t i = i8 + 32 * k + lane;
      const bool in = i < w1;
      const uint32_t r = in ? rank_at(i) : 0u;
      const bool a = in && above_cut(i, r), e = in && !a && want > 0 && r == cut;
      const uint32_t ma = __ballot_sync(0xffffffffu, a), me = __ballot_sync(0xffffffffu, e);
      const uint32_t e_before = at + __popc(me & before);
      const bool stays = a || (e && e_before < left);
      if (in) {
        const uint32_t to = above + __popc(ma & before) + min(e_before, left);
        if (stays) {
          kept[to] = slot[k];
          kept_scores[to] = score_of(r, scores + i);
        } else if (freed) {
          freed[i - to] = slot[k];
        }
      }
      above += __popc(ma);
      at += __popc(me);
    }
  }
  cluster.barrier_wait();
}

}  // namespace dsa

namespace {

using dsa::aligned;
using dsa::EvictParams;

cudaError_t evict_setup(void *) {
  return cudaFuncSetAttribute(dsa::evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * dsa::kEvCached);
}

}  // namespace

extern "C" dsa_status dsa_evict(int32_t num_seqs, int32_t width, const int32_t *slots, int64_t slots_stride,
                                const int32_t *lengths, const float *scores, int64_t scores_stride, int32_t budget,
                                int32_t keep_first, int32_t keep_last, int32_t *kept_slots, int64_t kept_slots_stride,
                                float *kept_scores, int64_t kept_scores_stride, int32_t *kept_lengths, int32_t *freed,
                                int64_t freed_stride, int32_t *freed_counts, dsa_stream_t stream) {
  dsa::NvtxRange range("dsa_evict");
  if (num_seqs < 0 || width < 1 || budget < 1 || keep_first < 0 || keep_last < 0) return DSA_ERR_INVALID_ARG;
  // (lists no wider than the budget free nothing: an empty array may have no address)
  if ((freed == nullptr) != (freed_counts == nullptr) && !(freed_counts && width <= budget)) return DSA_ERR_INVALID_ARG;
  if (num_seqs > (1 << 24) || width > (1 << 30)) return DSA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return DSA_OK;
  if (!slots || !lengths || !scores || !kept_slots || !kept_scores || !kept_lengths) return DSA_ERR_INVALID_ARG;
  const int32_t most = std::min(budget, width);
  if (slots_stride < width || scores_stride < width || kept_slots_stride < most || kept_scores_stride < most ||
      (freed && freed_stride < width - most))
    return DSA_ERR_INVALID_ARG;
  if (kept_slots == slots || kept_scores == scores || kept_lengths == lengths || freed_counts == lengths ||
      freed_counts == kept_lengths || (freed && (freed == slots || freed == kept_slots)))
    return DSA_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(lengths, 4) || !aligned(scores, 4) || !aligned(kept_slots, 4) ||
      !aligned(kept_scores, 4) || !aligned(kept_lengths, 4) || (freed && (!aligned(freed, 4) || !aligned(freed_counts, 4))))
    return DSA_ERR_ALIGNMENT;
  // CTAs to a list: 1024 entries each at least, 8 at most (16 lists of 65521:
  // 4 CTAs 26 us, 8 25, 16, which find no place together, 49).
  int cluster = 1;
  while (cluster < 8 && width > 1024 * cluster) cluster *= 2;
  EvictParams p = {slots,       slots_stride,       lengths,      scores, scores_stride, width,       budget, keep_first, keep_last,
                   kept_slots,  kept_slots_stride,  kept_scores,  kept_scores_stride,    kept_lengths, freed, freed_stride,
                   freed_counts};
  const int64_t run = ((int64_t)width + cluster - 1) / cluster;
  const bool held = run <= dsa::kEvCached;
  cudaError_t e = dsa::dsa_configure_once(dsa::kOnceEvict, &evict_setup, nullptr);
  if (e != cudaSuccess) return dsa::cuda_status(e);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)num_seqs * cluster);
  c.blockDim = dim3(dsa::kEvThreads);
  c.dynamicSmemBytes = held ? 4 * (size_t)run : 0;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return dsa::cuda_status(cudaLaunchKernelEx(&c, held ? dsa::evict_kernel<true> : dsa::evict_kernel<false>, (const EvictParams)p));
}

// evict.cu - eviction from a paged cache by accumulated attention weight: per sequence and
// KV head, the last tokens and the best-scored others stay, in order, and their K/V rows
// move to other pages. The library's planner (kv_plan.cu) evicts whole anchors; this cuts
// an anchor or a conversation down to a budget.
//
// 1. evict_select_kernel  a thread-block cluster per (sequence, KV head) finds the k-th
//    largest score by a radix select over 32-bit keys (digits of 11, 11 and 10 bits,
//    histograms of the cluster's CTAs added through distributed shared memory) and writes
//    the kept positions in order. The keys stay in shared memory between the passes: the
//    scores are read once. It also marks the pages that are read and written.
// 2. evict_copy_kernel    moves the kept rows: a block looks up the places of 256 (token,
//    head) rows first, then moves them, 16 bytes a thread and eight in flight.
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kSelThreads;  // 4
constexpr int kKeyCap = 20480;                       // keys a CTA holds (80 KB): two CTAs an SM
constexpr int kLoads = 8;                            // scores in flight per thread
constexpr int kMaxCluster = 8;

constexpr int kMarkRead = 1, kMarkWritten = 2;       // a page's uses: bit 0, and 2 per write

__device__ __forceinline__ int evict_len(const PagedEvictArgs& a, int b) {
  const int n = __ldg(a.lens + b);
  return n >= 0 && n <= a.max_len ? n : -1;
}

// Orders like the scores; NaN counts as -inf and -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

constexpr uint32_t kKeyZero = 0x80000000u, kKeyLowest = 0x007FFFFFu;  // of +-0; of -inf and NaN
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ uint4 ld_cluster_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const PagedEvictArgs a,
                                                                   int cluster, int key_cap) {
  extern __shared__ uint32_t s_keys[];  // [key_cap]
  __shared__ __align__(16) uint32_t s_hist[3][kBins];  // one per pass
  __shared__ uint32_t s_warp[kSelWarps];
  __shared__ uint32_t s_found[2];       // digit, and how many are above it
  __shared__ __align__(16) uint32_t s_count[4];  // this CTA's keys above / at the threshold
  __shared__ uint32_t s_gt[kSelWarps], s_eq[kSelWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x / cluster;
  const int b = pair / a.hkv, g = pair % a.hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = evict_len(a, b);
  const int fresh = n < 0 ? 0 : min(n, a.budget);     // tokens kept
  const int recent = min(a.recent, fresh);
  const int elig = (n < 0 ? 0 : n) - recent;          // tokens that compete
  const int k = fresh - recent;                       // for so many places
  const int64_t out_row = static_cast<int64_t>(pair);
  int32_t* kept = a.kept + out_row * a.budget;
  const float* score = a.score + out_row * a.score_stride;
  float* score_out = a.score_out != nullptr ? a.score_out + out_row * a.score_out_stride : nullptr;
  const int tid = rank * kSelThreads + threadIdx.x, threads = cluster * kSelThreads;

  if (g == 0) {  // the sequence's pages and its new length, once
    if (tid == 0) {
      a.new_lens[b] = n < 0 ? -1 : fresh;
      if (n < 0) atomicOr(a.err_word, kErrDeviceBounds);
    }
    const int page = 1 << a.page_shift;
    if (a.same_pool && n > 0)
      for (int j = tid; j < (n + page - 1) >> a.page_shift; j += threads) {
        const int p = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + j);
        if (p >= 0 && p < a.num_pages) atomicOr(a.marks + p, kMarkRead);
      }
    for (int j = tid; j < (fresh + page - 1) >> a.page_shift; j += threads) {
      const int p = __ldg(a.dst_table + static_cast<int64_t>(b) * a.dst_max_pages + j);
      if (p >= 0 && p < a.dst_num_pages) atomicAdd(a.marks + p, kMarkWritten);
    }
  }
  // the recent tokens, and what follows the last kept one
  for (int i = tid; i < recent; i += threads) {
    kept[k + i] = elig + i;
    if (score_out != nullptr) score_out[k + i] = __ldg(score + elig + i);
  }
  for (int i = fresh + tid; i < a.budget; i += threads) kept[i] = -1;
  if (score_out != nullptr)
    for (int64_t i = fresh + tid; i < a.score_out_stride; i += threads) score_out[i] = 0.f;
  if (k == 0) return;  // the same for every CTA of the cluster
  for (int i = threadIdx.x; i < 3 * kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  // this CTA's part of the competing tokens
  const int per = (elig + cluster - 1) / cluster;
  const int e0 = min(rank * per, elig), e1 = min(e0 + per, elig);
  const int count = e1 - e0;
  auto key_at = [&](int i) { return i < key_cap ? s_keys[i] : score_key(__ldg(score + e0 + i)); };

  uint32_t threshold = 0, need = 0;   // keys above it stay, and `need` of those at it
  if (k < elig) {
    need = static_cast<uint32_t>(k);
    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = s_hist[pass];
      if (pass == 0) {
        for (int i0 = threadIdx.x; i0 < count; i0 += kSelThreads * kLoads) {
          float x[kLoads];
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            const int i = i0 + j * kSelThreads;
            x[j] = i < count ? __ldg(score + e0 + i) : 0.f;
          }
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            const int i = i0 + j * kSelThreads;
            const uint32_t key = score_key(x[j]);
            if (i < count && i < key_cap) s_keys[i] = key;
            if (i < count) atomicAdd(&hist[key >> 21], 1u);
          }
        }
      } else {
        const int above = pass == 1 ? 21 : 10;
#pragma unroll 4
        for (int i = threadIdx.x; i < count; i += kSelThreads) {
          const uint32_t key = key_at(i);
          if (key >> above == prefix) atomicAdd(&hist[(key >> shift) & mask], 1u);
        }
      }
      if (cluster > 1) cluster_sync(); else __syncthreads();
      uint32_t bin[kBinsPerThread] = {0, 0, 0, 0};
      if (cluster == 1) {
        const uint4 v = *reinterpret_cast<const uint4*>(&hist[kBinsPerThread * threadIdx.x]);
        bin[0] = v.x;
        bin[1] = v.y;
        bin[2] = v.z;
        bin[3] = v.w;
      } else {
        uint4 v[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < cluster) v[c] = ld_cluster_u4(cluster_map(&hist[kBinsPerThread * threadIdx.x], c));
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < cluster) {
            bin[0] += v[c].x;
            bin[1] += v[c].y;
            bin[2] += v[c].z;
            bin[3] += v[c].w;
          }
      }
      // how many keys lie in the bins of the threads after this one
      const uint32_t mine = bin[0] + bin[1] + bin[2] + bin[3];
      uint32_t x = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_down_sync(0xFFFFFFFFu, x, off);
        if (lane + off < 32) x += y;
      }
      if (lane == 0) s_warp[warp] = x;
      __syncthreads();
      uint32_t above = x - mine;
      for (int w = warp + 1; w < kSelWarps; ++w) above += s_warp[w];
#pragma unroll
      for (int j = kBinsPerThread - 1; j >= 0; --j) {
        if (above < need && need <= above + bin[j]) {
          s_found[0] = kBinsPerThread * threadIdx.x + j;
          s_found[1] = above;
        }
        above += bin[j];
      }
      __syncthreads();
      prefix = pass == 2 ? prefix << 10 | s_found[0] : prefix << 11 | s_found[0];
      need -= s_found[1];
    }
    threshold = prefix;
  }

  // positions of the kept keys: contiguous runs of the warps, in order
  const int run = (count + 32 * kSelWarps - 1) / (32 * kSelWarps) * 32;
  const int w0 = min(warp * run, count), w1 = min(w0 + run, count);
  const bool all = k >= elig;
  uint32_t gt = 0, eq = 0;
  if (!all) {
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t key = key_at(i);
      gt += key > threshold;
      eq += key == threshold;
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  } else {
    gt = static_cast<uint32_t>(max(0, w1 - w0));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t tg = 0, te = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      tg += s_gt[w];
      te += s_eq[w];
    }
    s_count[0] = tg;
    s_count[1] = te;
  }
  if (cluster > 1) cluster_sync(); else __syncthreads();
  uint32_t base_gt = 0, base_eq = 0;
  for (int c = 0; c < rank; ++c) {
    const uint4 v = ld_cluster_u4(cluster_map(s_count, c));
    base_gt += v.x;
    base_eq += v.y;
  }
  for (int w = 0; w < warp; ++w) {
    base_gt += s_gt[w];
    base_eq += s_eq[w];
  }
  const uint32_t before = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t key = in && !all ? key_at(i) : 0u;
    const bool is_gt = in && (all || key > threshold), is_eq = in && !all && key == threshold;
    const uint32_t bg = __ballot_sync(0xFFFFFFFFu, is_gt);
    const uint32_t be = __ballot_sync(0xFFFFFFFFu, is_eq);
    const uint32_t eq_rank = base_eq + __popc(be & before);
    if (is_gt || (is_eq && eq_rank < need)) {
      const uint32_t at = base_gt + __popc(bg & before) + min(eq_rank, need);
      if (at < static_cast<uint32_t>(k)) {  // else the scores changed meanwhile
        kept[at] = e0 + i;
        if (score_out != nullptr) {
          // the key gives the score back, but for the values that share one
          score_out[at] = all || key == kKeyZero || key == kKeyLowest ? __ldg(score + e0 + i)
                                                                     : key_score(key);
        }
      }
    }
    base_gt += __popc(bg);
    base_eq += __popc(be);
  }
  if (cluster > 1) cluster_sync();  // no CTA leaves while others read its counts
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;   // rows' pieces in flight per thread, K and V each

// A block moves 256 consecutive (kept place, head) rows of one sequence, K and V.
__global__ void __launch_bounds__(kCopyThreads, 4) evict_copy_kernel(const PagedEvictArgs a,
                                                                     int chunks) {
  __shared__ int64_t s_src[kCopyThreads], s_dst[kCopyThreads];  // byte offsets; < 0: none
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / chunks;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x % chunks) * kCopyThreads;
  const int n = evict_len(a, b);
  const int fresh = min(n, a.budget);
  const int64_t rows = static_cast<int64_t>(fresh) * a.hkv;
  if (r0 >= rows) return;
  const int count = static_cast<int>(min(static_cast<int64_t>(kCopyThreads), rows - r0));
  if (threadIdx.x < count) {
    const int64_t r = r0 + threadIdx.x;
    const int i = static_cast<int>(r / a.hkv), g = static_cast<int>(r % a.hkv);
    const int mask = (1 << a.page_shift) - 1;
    const int pos = a.kept[(static_cast<int64_t>(b) * a.hkv + g) * a.budget + i];
    const int to = __ldg(a.dst_table + static_cast<int64_t>(b) * a.dst_max_pages +
                         (i >> a.page_shift));
    // the destination page is written once, by this sequence, and read by none
    bool ok = to >= 0 && to < a.dst_num_pages && a.marks[to] == kMarkWritten;
    int from = -1;
    if (pos >= 0 && pos < n) {
      from = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift));
      ok = ok && from >= 0 && from < a.num_pages;
    } else {
      ok = false;
    }
    if (!ok) {
      atomicOr(a.err_word, kErrDeviceBounds);
      a.new_lens[b] = -1;
    }
    s_src[threadIdx.x] =
        ok ? (((static_cast<int64_t>(from) << a.page_shift) + (pos & mask)) * a.hkv + g) * a.row_bytes
           : -1;
    s_dst[threadIdx.x] =
        ok ? (((static_cast<int64_t>(to) << a.page_shift) + (i & mask)) * a.hkv + g) * a.row_bytes
           : -1;
  }
  __syncthreads();
  const int shift = a.row_bytes == 256 ? 4 : a.row_bytes == 128 ? 3 : 2;  // 16-byte pieces a row
  const int pieces = count << shift;
  for (int u0 = threadIdx.x; u0 < pieces; u0 += kCopyThreads * kCopyUnroll) {
    uint4 x[kCopyUnroll], y[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
      const int u = u0 + j * kCopyThreads;
      const int64_t s = u < pieces ? s_src[u >> shift] : -1;
      if (s >= 0) {
        const int64_t at = s + 16 * (u & ((1 << shift) - 1));
        x[j] = *reinterpret_cast<const uint4*>(a.k_pages + at);
        y[j] = *reinterpret_cast<const uint4*>(a.v_pages + at);
      }
    }
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
      const int u = u0 + j * kCopyThreads;
      const int64_t s = u < pieces ? s_dst[u >> shift] : -1;
      if (s >= 0) {
        const int64_t at = s + 16 * (u & ((1 << shift) - 1));
        *reinterpret_cast<uint4*>(a.k_dst + at) = x[j];
        *reinterpret_cast<uint4*>(a.v_dst + at) = y[j];
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e =
      cudaMemsetAsync(a.marks, 0, static_cast<size_t>(a.dst_num_pages) * sizeof(int32_t), stream);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, head): enough to hold the keys, and more while SMs are idle and a
  // CTA has thousands of keys
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  int cluster = 1;
  while (cluster < kMaxCluster &&
         (a.max_len > kKeyCap * cluster ||
          (pairs * cluster * 2 <= num_sms && a.max_len > 2048 * cluster)))
    cluster *= 2;
  int cap = (a.max_len + cluster - 1) / cluster;
  if (cap > kKeyCap) cap = kKeyCap;
  const size_t smem = static_cast<size_t>(cap < 4 ? 4 : cap) * 4;
  static std::atomic<uint64_t> ready{0};
  e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel), kKeyCap * 4, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cluster, cap);
  if (e != cudaSuccess) return e;
  const int chunks = static_cast<int>(
      (static_cast<int64_t>(a.budget) * a.hkv + kCopyThreads - 1) / kCopyThreads);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * chunks));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, evict_copy_kernel, a, chunks);
}

}  // namespace quail

// evict.cu - eviction from a paged cache by accumulated attention weight: per sequence and
// KV head, the last tokens and the best-scored others stay, in order, and their K/V rows
// move to other pages. The library's planner (kv_plan.cu) evicts whole anchors; this cuts
// an anchor or a conversation down to a budget.
//
// 1. evict_select_kernel  a thread-block cluster per (sequence, KV head) finds the k-th
//    largest score by a radix select over 32-bit keys (digits of 11, 11 and 10 bits,
//    histograms of the cluster's CTAs added through distributed shared memory; it stops
//    early where a digit settles it, which distinct scores mostly do after two) and writes
//    the kept positions in order. The keys stay in registers between the passes: the scores
//    are read once, up to 16,384 per CTA. It also notes who writes and who holds each page.
//    Bound by latency: about ten barriers and dependent steps of a microsecond or less.
// 2. evict_copy_kernel    moves the kept rows: a block looks up the places of 256 (token,
//    head) rows first, then moves them, 16 bytes a thread and eight in flight.
// Small calls do both in one launch (FUSED): each CTA compares its sequence's destination pages
// with every other page of the call itself, and moves the tokens of its own part that stay.
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kSelThreads;  // 4
constexpr int kSub = 4;                              // copies of the first histogram
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 32;                         // keys a thread holds at most

__device__ __forceinline__ int evict_len(const PagedEvictArgs& a, int b) {
  const int n = a.lens[b];
  return n >= 0 && n <= a.max_len ? n : -1;
}

// Byte offset in a pool of the row of KV head g at place `at` of a page; fp4: of its codes, and of
// its block scales (a head's codes lie together, and behind them its block scales).
__device__ __forceinline__ int64_t row_at(const PagedEvictArgs& a, int page, int at, int g) {
  if (a.block_bytes == 0)
    return (((static_cast<int64_t>(page) << a.page_shift) + at) * a.hkv + g) * a.row_bytes;
  return (static_cast<int64_t>(page) * a.hkv + g) *
             (static_cast<int64_t>(a.row_bytes + a.block_bytes) << a.page_shift) +
         static_cast<int64_t>(at) * a.row_bytes;
}
__device__ __forceinline__ int64_t blocks_at(const PagedEvictArgs& a, int page, int at, int g) {
  return row_at(a, page, 0, g) + (static_cast<int64_t>(a.row_bytes) << a.page_shift) +
         at * a.block_bytes;
}
// log2 of a row's 16-byte pieces
__device__ __forceinline__ int row_shift(const PagedEvictArgs& a) {
  return a.row_bytes == 256 ? 4 : a.row_bytes == 128 ? 3 : a.row_bytes == 64 ? 2 : 1;
}
// A row's block scales, 8 bytes of them or 4.
__device__ __forceinline__ uint2 load_blocks(const uint8_t* p, int bytes) {
  return bytes == 8 ? *reinterpret_cast<const uint2*>(p)
                    : make_uint2(*reinterpret_cast<const uint32_t*>(p), 0u);
}
__device__ __forceinline__ void store_blocks(uint8_t* p, int bytes, uint2 x) {
  if (bytes == 8) *reinterpret_cast<uint2*>(p) = x;
  else *reinterpret_cast<uint32_t*>(p) = x.x;
}

__device__ __forceinline__ int pages_of(const PagedEvictArgs& a, int tokens) {
  return (tokens + (1 << a.page_shift) - 1) >> a.page_shift;
}

// Notes about a destination page p, in a workspace that nobody clears: the notes name entries
// of the tables, and one that its table does not confirm is what was there before.
//   claim[p]  an entry of dst_table that names p (the last to claim it)
//   dup[p]    -1 once claimed; the entry that found p claimed by another
//   hold[p]   an entry of block_table that names p (same pool only; any of them)
__device__ __forceinline__ bool is_claim(const PagedEvictArgs& a, int entry, int p) {
  if (entry < 0 || entry >= a.num_seqs * a.dst_max_pages || a.dst_table[entry] != p)
    return false;
  const int n = evict_len(a, entry / a.dst_max_pages);
  return entry % a.dst_max_pages < pages_of(a, min(n, a.budget));
}
__device__ __forceinline__ bool is_held(const PagedEvictArgs& a, int entry, int p) {
  if (entry < 0 || entry >= a.num_seqs * a.max_pages || a.table[entry] != p) return false;
  return entry % a.max_pages < pages_of(a, evict_len(a, entry / a.max_pages));
}

// Orders like the scores; NaN counts as -inf and -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// Sum of the lower lanes' values.
__device__ __forceinline__ uint32_t scan_excl(uint32_t v) {
  const int lane = threadIdx.x & 31;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, off);
    if (lane >= off) x += y;
  }
  return x - v;
}

__device__ __forceinline__ uint4 ld_cluster_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster_u4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_cluster_u2(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// The notes about the pages of all sequences, a warp for 32 places of a sequence's table.
__device__ void write_notes(const PagedEvictArgs& a, int warp, int warps, int chunks) {
  const int lane = threadIdx.x & 31;
  for (int64_t item = warp; item < static_cast<int64_t>(a.num_seqs) * chunks; item += warps) {
    const int b = static_cast<int>(item / chunks), j = static_cast<int>(item % chunks) * 32 + lane;
    const int n = evict_len(a, b);
    if (a.same_pool && j < pages_of(a, n)) {
      const int p = a.table[b * a.max_pages + j];
      if (p >= 0 && p < a.num_pages) a.hold[p] = b * a.max_pages + j;
    }
    if (j < pages_of(a, min(n, a.budget))) {
      const int entry = b * a.dst_max_pages + j;
      const int p = a.dst_table[entry];
      if (p < 0 || p >= a.dst_num_pages) continue;
      // of several entries that claim p the last one to do so sees another's claim, and its
      // note follows every clearing
      a.dup[p] = -1;
      __threadfence();
      const int old = atomicExch(a.claim + p, entry);
      __threadfence();
      if (old != entry && is_claim(a, old, p)) a.dup[p] = entry;
    }
  }
}

// KPT: keys a thread holds, in registers, or (SHARED) in shared memory: 32 in registers leave
// room for one CTA per SM, and then only 15 clusters of eight fit the GPU at once (36 with
// two). A CTA's part of the competing tokens is walked in rounds of
// kSelThreads * KPT (one, unless the part is longer: then the scores are read again in every
// pass); in a round each warp has a contiguous run, lane by lane, so that the order of the
// tokens is (round, warp, i, lane).
constexpr int kSmallKeys = 4 * kSelThreads;   // FUSED: tokens per CTA at most
constexpr int kSmallKept = 512;               // kept tokens of a sequence that fits one CTA, at most
constexpr int kSmallShare = 128;              // kept ones per CTA of longer sequences' clusters
constexpr int kSmallPages =                   // the kept ones' pages at most (of 16 tokens or more)
    (kSmallKept > kMaxCluster * kSmallShare ? kSmallKept : kMaxCluster * kSmallShare) / 16;
template <int KPT, bool SHARED, bool FUSED>
__global__ void __launch_bounds__(kSelThreads, 2)
    evict_select_kernel(const PagedEvictArgs a, int cluster, int note_blocks, int note_chunks) {
  // Scores of one octave share few first digits, so lanes often add to the same bin: four
  // copies, by lane, keep those additions from queueing.
  __shared__ __align__(16) uint32_t s_first[kSub][kBins];
  __shared__ __align__(16) uint32_t s_second[kBins], s_third[kBins / 2];
  __shared__ uint32_t s_warp[kSelWarps];
  __shared__ uint32_t s_found[3];       // digit, how many are above it, how many have it
  __shared__ __align__(16) uint32_t s_count[kMaxCluster][2];  // the CTAs' keys above / at the threshold
  __shared__ uint32_t s_gt[kSelWarps], s_eq[kSelWarps];
  int* s_kept = reinterpret_cast<int*>(s_first);  // FUSED, after the passes: this CTA's kept ones
  __shared__ int s_to[FUSED ? kSmallPages : 1], s_bad[FUSED ? kSmallPages + 1 : 1];
  after_stream();
  if (!FUSED) let_next_start();  // the copy
  if (!FUSED && static_cast<int>(blockIdx.x) < note_blocks) {
    write_notes(a, blockIdx.x * kSelWarps + (threadIdx.x >> 5), note_blocks * kSelWarps, note_chunks);
    return;
  }
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int pair = (blockIdx.x - note_blocks) / cluster;
  const int b = pair / a.hkv, g = pair % a.hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = evict_len(a, b);
  const int fresh = n < 0 ? 0 : min(n, a.budget);     // tokens kept
  const int recent = min(a.recent, fresh);
  const int elig = (n < 0 ? 0 : n) - recent;          // tokens that compete
  const int k = fresh - recent;                       // for so many places
  const float* score = a.score + static_cast<int64_t>(pair) * a.score_stride;

  // this CTA's part of the competing tokens
  const int per = (elig + cluster - 1) / cluster;
  const int e0 = min(rank * per, elig), count = min(per, elig - e0);
  constexpr int kRound = kSelThreads * KPT;
  const int rounds = (per + kRound - 1) / kRound;
  extern __shared__ uint32_t s_keys[];  // SHARED: [KPT][kSelThreads], each thread its own
  uint32_t reg[SHARED ? 1 : KPT] = {};
  auto key = [&](int i) {               // 0: none (every score's key is larger)
    return SHARED ? s_keys[i * kSelThreads + threadIdx.x] : reg[SHARED ? 0 : i];
  };
  int w0 = 0;                           // the warp's first token of the round
  auto load = [&](int round) {
    const int left = max(0, min(kRound, count - round * kRound));
    const int run = (left + 32 * kSelWarps - 1) / (32 * kSelWarps) * 32;
    const int end = round * kRound + left;
    w0 = round * kRound + warp * run;
    const int w1 = min(w0 + run, end);
    constexpr int kBatch = KPT < 16 ? KPT : 16;  // loads in flight
#pragma unroll
    for (int i0 = 0; i0 < KPT; i0 += kBatch) {
      float x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = w0 + 32 * (i0 + i) + lane;
        x[i] = at < w1 ? score[e0 + at] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t u = w0 + 32 * (i0 + i) + lane < w1 ? score_key(x[i]) : 0u;
        if (SHARED)
          s_keys[(i0 + i) * kSelThreads + threadIdx.x] = u;
        else
          reg[SHARED ? 0 : i0 + i] = u;
      }
    }
  };
  if (k > 0) load(0);

  int32_t* kept = a.kept + static_cast<int64_t>(pair) * a.budget;
  float* score_out =
      a.score_out != nullptr ? a.score_out + static_cast<int64_t>(pair) * a.score_out_stride : nullptr;
  const int tid = rank * kSelThreads + threadIdx.x, threads = cluster * kSelThreads;
  // the first recent token's score comes with the others, not after the barrier below
  const float recent_score = score_out != nullptr && tid < recent ? score[elig + tid] : 0.f;
  if constexpr (FUSED) {
    const int mine = pages_of(a, fresh);
    for (int j = threadIdx.x; j <= mine; j += kSelThreads) {
      const int p = j < mine ? a.dst_table[b * a.dst_max_pages + j] : 0;
      if (j < mine) s_to[j] = p;
      s_bad[j] = j < mine && (p < 0 || p >= a.dst_num_pages);  // the last: the source pages
    }
    __syncthreads();
    auto meet = [&](int p, int entry) {  // page p is claimed (entry of dst_table) or held (-1)
      for (int j = 0; j < mine; ++j)
        if (s_to[j] == p && b * a.dst_max_pages + j != entry) s_bad[j] = 1;
    };
    const int claims = pages_of(a, min(a.budget, a.max_len));
    for (int e = threadIdx.x; e < a.num_seqs * claims; e += kSelThreads) {
      const int seq = e / claims, j = e % claims, len = evict_len(a, seq);
      if (j < pages_of(a, min(len, a.budget)))
        meet(a.dst_table[seq * a.dst_max_pages + j], seq * a.dst_max_pages + j);
    }
    if (a.same_pool) {
      const int held = pages_of(a, a.max_len);
      for (int e = threadIdx.x; e < a.num_seqs * held; e += kSelThreads) {
        const int seq = e / held, j = e % held;
        if (j < pages_of(a, evict_len(a, seq))) meet(a.table[seq * a.max_pages + j], -1);
      }
    }
    if (g == 0 && rank == 0)
      for (int j = threadIdx.x; j < pages_of(a, n); j += kSelThreads) {
        const int p = a.table[b * a.max_pages + j];
        if (p < 0 || p >= a.num_pages) s_bad[mine] = 1;
      }
  } else if (g == 0 && tid == 0) {  // the new length, once
    a.new_lens[b] = n < 0 ? -1 : fresh;
    if (n < 0) atomicOr(a.err_word, kErrDeviceBounds);
  }
  // the recent tokens, and what follows the last kept one
  for (int i = tid; i < recent; i += threads) {
    kept[k + i] = elig + i;
    if (score_out != nullptr) score_out[k + i] = i == tid ? recent_score : score[elig + i];
  }
  for (int i = fresh + tid; i < a.budget; i += threads) kept[i] = -1;
  if (score_out != nullptr)
    for (int64_t i = fresh + tid; i < a.score_out_stride; i += threads) score_out[i] = 0.f;
  if (!FUSED && k == 0) return;  // the same for every CTA of the cluster
  int first_kept = 0, kept_here = 0;    // FUSED: this CTA's places, without the recent tokens
  if (k > 0) {

  // keys above the threshold stay, and `need` of those at it; k >= elig: every key
  uint32_t threshold = 0, need = 0;
  if (k < elig) {
    for (int i = threadIdx.x; i < kSub * kBins / 4; i += kSelThreads)
      reinterpret_cast<uint4*>(s_first)[i] = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4*>(s_second)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x < kBins / 8) reinterpret_cast<uint4*>(s_third)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    need = static_cast<uint32_t>(k);
    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      uint32_t* hist = pass == 0 ? s_first[0] : pass == 1 ? s_second : s_third;
      for (int round = 0; round < rounds; ++round) {
        if (rounds > 1 && (pass > 0 || round > 0)) load(round);
        if (pass == 0) {
          uint32_t* mine = s_first[lane & (kSub - 1)];
#pragma unroll
          for (int i = 0; i < KPT; ++i)
            if (key(i) != 0) atomicAdd(mine + (key(i) >> 21), 1u);
        } else {
          const int above = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0;
          const uint32_t mask = pass == 1 ? 2047u : 1023u;
#pragma unroll
          for (int i = 0; i < KPT; ++i)
            if (key(i) >> above == prefix) atomicAdd(hist + ((key(i) >> shift) & mask), 1u);
        }
      }
      __syncthreads();
      const bool has = pass < 2 || threadIdx.x < kSelThreads / 2;  // the last has half the bins
      uint4 sum = make_uint4(0u, 0u, 0u, 0u);
      if (has) sum = *reinterpret_cast<const uint4*>(hist + kBinsPerThread * threadIdx.x);
      if (pass == 0) {
#pragma unroll
        for (int c = 1; c < kSub; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(&s_first[c][kBinsPerThread * threadIdx.x]);
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
      }
      if (cluster > 1) {
        // Each CTA adds up its share of the bins and hands the sums to all. (All bins read
        // by all, 57 KB through distributed shared memory per CTA, took 3-4 us a pass.)
        if (pass == 0) *reinterpret_cast<uint4*>(hist + kBinsPerThread * threadIdx.x) = sum;
        cluster_sync();
        const int share = (pass < 2 ? kBins : kBins / 2) / cluster;
        if (threadIdx.x < share / 4) {
          uint32_t* at = hist + rank * share + 4 * threadIdx.x;
          uint4 v[kMaxCluster];
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c)
            if (c < cluster) v[c] = ld_cluster_u4(cluster_map(at, (rank + c) & (cluster - 1)));
#pragma unroll
          for (int c = 1; c < kMaxCluster; ++c)
            if (c < cluster) {
              v[0].x += v[c].x;
              v[0].y += v[c].y;
              v[0].z += v[c].z;
              v[0].w += v[c].w;
            }
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c)  // nobody else reads this share
            if (c < cluster) st_cluster_u4(cluster_map(at, (rank + c) & (cluster - 1)), v[0]);
        }
        cluster_sync();
        if (has) sum = *reinterpret_cast<const uint4*>(hist + kBinsPerThread * threadIdx.x);
      }
      // how many keys lie in the bins of the threads after this one
      const uint32_t bin[kBinsPerThread] = {sum.x, sum.y, sum.z, sum.w};
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
      const uint32_t others = lane > warp && lane < kSelWarps ? s_warp[lane] : 0u;
      above += __reduce_add_sync(0xFFFFFFFFu, others);
#pragma unroll
      for (int j = kBinsPerThread - 1; j >= 0; --j) {
        if (above < need && need <= above + bin[j]) {
          s_found[0] = kBinsPerThread * threadIdx.x + j;
          s_found[1] = above;
          s_found[2] = bin[j];
        }
        above += bin[j];
      }
      __syncthreads();
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      prefix = pass == 2 ? prefix << 10 | s_found[0] : prefix << 11 | s_found[0];
      need -= s_found[1];
      if (s_found[2] == need) {  // every key of the digit stays
        threshold = (prefix << shift) - 1;
        need = 0;
        break;
      }
      threshold = prefix;
    }
  }

  // Positions of the kept keys. Lane i holds the votes on the warp's i-th 32 tokens: which
  // are above the threshold, which at it.
  uint32_t above = 0, at_it = 0;
  auto vote = [&]() {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const uint32_t u = key(i);
      const uint32_t bg = __ballot_sync(0xFFFFFFFFu, u > threshold);
      const uint32_t be = __ballot_sync(0xFFFFFFFFu, u != 0 && u == threshold);
      if (lane == i) {
        above = bg;
        at_it = be;
      }
    }
  };
  uint32_t gt = 0, eq = 0;
  for (int round = 0; round < rounds; ++round) {
    if (rounds > 1) load(round);
    vote();
    gt += __reduce_add_sync(0xFFFFFFFFu, __popc(above));
    eq += __reduce_add_sync(0xFFFFFFFFu, __popc(at_it));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  const uint32_t lane_gt = lane < kSelWarps ? s_gt[lane] : 0u;
  const uint32_t lane_eq = lane < kSelWarps ? s_eq[lane] : 0u;
  uint32_t base_gt = 0, base_eq = 0;    // kept / at the threshold before this CTA's
  const uint32_t all_gt = __reduce_add_sync(0xFFFFFFFFu, lane_gt);
  const uint32_t all_eq = __reduce_add_sync(0xFFFFFFFFu, lane_eq);
  if (k >= elig) {
    base_gt = e0;
  } else if (cluster > 1) {
    // to all of them (which run: the passes had a barrier), so that none has to stay for reads
    if (threadIdx.x < cluster) st_cluster_u2(cluster_map(s_count[rank], threadIdx.x), all_gt, all_eq);
    cluster_sync();
    base_gt = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? s_count[lane][0] : 0u);
    base_eq = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? s_count[lane][1] : 0u);
  }
  first_kept = base_gt + min(base_eq, need);
  kept_here = base_gt + all_gt + min(base_eq + all_eq, need) - first_kept;
  for (int round = 0; round < rounds; ++round) {
    uint32_t warp_gt, warp_eq;          // before this warp's
    if (rounds > 1) {  // the round's own counts
      load(round);
      vote();
      gt = __reduce_add_sync(0xFFFFFFFFu, __popc(above));
      eq = __reduce_add_sync(0xFFFFFFFFu, __popc(at_it));
      __syncthreads();  // the last round's were read
      if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
      }
      __syncthreads();
      const uint32_t x = lane < kSelWarps ? s_gt[lane] : 0u, y = lane < kSelWarps ? s_eq[lane] : 0u;
      warp_gt = base_gt + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0u);
      warp_eq = base_eq + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0u);
      base_gt += __reduce_add_sync(0xFFFFFFFFu, x);
      base_eq += __reduce_add_sync(0xFFFFFFFFu, y);
    } else {
      warp_gt = base_gt + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? lane_gt : 0u);
      warp_eq = base_eq + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? lane_eq : 0u);
    }
    // the kept ones of each 32: all above, and the first `allowed` of the warp at it
    const uint32_t allowed = need > warp_eq ? min(need - warp_eq, eq) : 0u;
    uint32_t sel = above;
    if (allowed == eq) {
      sel |= at_it;
    } else if (allowed > 0) {
      const int room = static_cast<int>(allowed) - static_cast<int>(scan_excl(__popc(at_it)));
      uint32_t some = room > 0 ? at_it : 0u;
      while (__popc(some) > room && some != 0) some &= ~(0x80000000u >> __clz(some));
      sel |= some;
    }
    // The warp's kept tokens, 32 at a time: the o-th lies in the 32 of lane i, where the lanes
    // before it have at most o, and is the r-th of its votes. (A store under each vote, 32 of
    // them one after the other, measured 46 us instead of 43: two caches of 100,000-131,000.)
    const uint32_t first = scan_excl(__popc(sel));
    const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, __popc(sel));
    const uint32_t base = warp_gt + min(warp_eq, need);
    for (uint32_t o0 = 0; o0 < total; o0 += 32) {
      const uint32_t o = o0 + lane;
      int i = 0;
#pragma unroll
      for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xFFFFFFFFu, first, i + step) <= o) i += step;
      const uint32_t votes = __shfl_sync(0xFFFFFFFFu, sel, i);
      uint32_t r = o - __shfl_sync(0xFFFFFFFFu, first, i);
      int bit = 0;
#pragma unroll
      for (int step = 16; step > 0; step >>= 1) {
        const uint32_t c = __popc((votes >> bit) & ((1u << step) - 1u));
        if (r >= c) {
          r -= c;
          bit += step;
        }
      }
      const uint32_t at = base + o;
      if (o < total && at < static_cast<uint32_t>(k)) {  // (more only if the scores change meanwhile)
        const int pos = e0 + w0 + 32 * i + bit;
        kept[at] = pos;
        if (FUSED) s_kept[at - first_kept] = pos;
        if (score_out != nullptr) score_out[at] = score[pos];
      }
    }
  }
  }

  if constexpr (FUSED) {
    __syncthreads();
    const int mine = pages_of(a, fresh);
    if (g == 0 && rank == 0 && threadIdx.x < 32) {
      bool bad = n < 0;
      for (int j = lane; j <= mine; j += 32) bad |= s_bad[j] != 0;
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        a.new_lens[b] = bad ? -1 : fresh;
        if (bad) atomicOr(a.err_word, kErrDeviceBounds);
      }
    }
    const int shift = row_shift(a);
    const int mask = (1 << a.page_shift) - 1;
    // the recent tokens are dealt out evenly
    const int r0 = rank * recent / cluster, r1 = (rank + 1) * recent / cluster;
    const int items = kept_here + r1 - r0;
#pragma unroll 4
    for (int u = threadIdx.x; u < items << shift; u += kSelThreads) {
      const int at = u >> shift, c = u & ((1 << shift) - 1);
      const bool old = at < kept_here;
      const int i = old ? first_kept + at : k + r0 + at - kept_here;
      const int pos = old ? s_kept[at] : elig + r0 + at - kept_here;
      if (pos < 0 || pos >= n) continue;  // only if the scores changed meanwhile
      const int from = a.table[b * a.max_pages + (pos >> a.page_shift)];
      if (s_bad[i >> a.page_shift] || from < 0 || from >= a.num_pages) continue;
      const int to = s_to[i >> a.page_shift];
      const int64_t src = row_at(a, from, pos & mask, g) + 16 * c;
      const int64_t dst = row_at(a, to, i & mask, g) + 16 * c;
      const uint4 x = *reinterpret_cast<const uint4*>(a.k_pages + src);
      const uint4 y = *reinterpret_cast<const uint4*>(a.v_pages + src);
      if (a.block_bytes != 0 && c < 2) {  // one lane K's, one V's
        const uint8_t* from_pages = c == 0 ? a.k_pages : a.v_pages;
        store_blocks((c == 0 ? a.k_dst : a.v_dst) + blocks_at(a, to, i & mask, g), a.block_bytes,
                     load_blocks(from_pages + blocks_at(a, from, pos & mask, g), a.block_bytes));
      }
      *reinterpret_cast<uint4*>(a.k_dst + dst) = x;
      *reinterpret_cast<uint4*>(a.v_dst + dst) = y;
    }
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;   // rows' pieces in flight per thread, K and V each

// A block moves 256 consecutive (kept place, head) rows of one sequence, K and V.
__global__ void __launch_bounds__(kCopyThreads, 4) evict_copy_kernel(const PagedEvictArgs a,
                                                                     int chunks) {
  __shared__ int64_t s_src[kCopyThreads], s_dst[kCopyThreads];  // byte offsets; < 0: none
  const int b = blockIdx.x / chunks;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x % chunks) * kCopyThreads;
  const int n = evict_len(a, b);
  const int fresh = min(n, a.budget);
  const int64_t rows = static_cast<int64_t>(fresh) * a.hkv;
  if (r0 >= rows) {
    after_stream();  // also where nothing is to be moved: the call ends with its selection
    return;
  }
  const int count = static_cast<int>(min(static_cast<int64_t>(kCopyThreads), rows - r0));
  const bool has = threadIdx.x < count;
  const int64_t r = r0 + threadIdx.x;
  const int i = static_cast<int>(r / a.hkv), g = static_cast<int>(r % a.hkv);
  // what the selection does not write is read before its end
  const int to = has ? a.dst_table[static_cast<int64_t>(b) * a.dst_max_pages + (i >> a.page_shift)] : -1;
  after_stream();
  if (has) {
    const int mask = (1 << a.page_shift) - 1;
    const bool to_ok = to >= 0 && to < a.dst_num_pages;
    // (three loads side by side, then two: not one after the other)
    const int pos = a.kept[(static_cast<int64_t>(b) * a.hkv + g) * a.budget + i];
    const int dup = to_ok ? a.dup[to] : 0;
    const int hold = to_ok && a.same_pool ? a.hold[to] : -1;
    const bool pos_ok = pos >= 0 && pos < n;
    const int from =
        pos_ok ? a.table[static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift)] : -1;
    // the destination page is written once, by this sequence, and held by none
    const bool ok = to_ok && dup == -1 && pos_ok && from >= 0 && from < a.num_pages &&
                    !is_held(a, hold, to);
    if (!ok) {
      atomicOr(a.err_word, kErrDeviceBounds);
      a.new_lens[b] = -1;
    }
    s_src[threadIdx.x] = ok ? row_at(a, from, pos & mask, g) : -1;
    s_dst[threadIdx.x] = ok ? row_at(a, to, i & mask, g) : -1;
    if (ok && a.block_bytes != 0) {
      const int64_t src = blocks_at(a, from, pos & mask, g), dst = blocks_at(a, to, i & mask, g);
      const uint2 x = load_blocks(a.k_pages + src, a.block_bytes);
      const uint2 y = load_blocks(a.v_pages + src, a.block_bytes);
      store_blocks(a.k_dst + dst, a.block_bytes, x);
      store_blocks(a.v_dst + dst, a.block_bytes, y);
    }
  }
  __syncthreads();
  const int shift = row_shift(a);
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
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  const int page = 1 << a.page_shift;
  const int most = a.budget < a.max_len ? a.budget : a.max_len;
  const int64_t own = (most + page - 1) / page;
  const int64_t others = a.num_seqs * (own + (a.same_pool ? (a.max_len + page - 1) / page : 0));
  cudaError_t e = cudaSuccess;
  int cluster = 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kSelThreads);
  // One launch: up to 2,048 tokens per CTA. Few tokens that stay may lie in one CTA's hands, whose
  // moving them alone is slow, so with clusters at most 128 per CTA stay, and idle SMs join in.
  // Measured against two launches (8 KV heads, d = 128): one sequence of 4,000 to 128 10.5 us
  // and 11.9, to 1,000 12.7 and 13.0, one of 16,000 to 500 11.2 and 12.8, four of 16,000 (e4m3)
  // to 1,000 15.8 and 20.1; past the rule, one of 8,000 to 2,000 15.4 and 13.5, of 16,000 to
  // 4,000 26 and 18; and 2 us less on the host.
  const bool brief = a.max_len <= kSmallKeys && most <= kSmallKept;
  while (cluster < kMaxCluster && (a.max_len > kSmallKeys * cluster ||
                                   (pairs * cluster * 2 <= num_sms && most > kSmallShare * cluster)))
    cluster *= 2;
  // (every CTA compares its `own` pages with all the `others`)
  if (a.max_len <= kSmallKeys * cluster && (brief || most <= kSmallShare * cluster) &&
      (cluster == 1 || pairs * cluster <= 2 * num_sms) && others <= 1024 && own * others <= 65536) {
    attr[1].val.clusterDim.x = cluster;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cfg.gridDim = dim3(static_cast<unsigned>(pairs * cluster));
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<4, false, true>, a, cluster, 0, 0);
  }
  // CTAs per (sequence, head): enough to hold the keys, and more while SMs are idle and a
  // CTA has thousands of keys
  cluster = 1;
  while (cluster < kMaxCluster &&
         (a.max_len > static_cast<int64_t>(kSelThreads) * kMaxKeys * cluster ||
          (pairs * cluster * 2 <= num_sms && a.max_len > 2048 * cluster)))
    cluster *= 2;
  const int per = (a.max_len + cluster - 1) / cluster;
  attr[1].val.clusterDim.x = cluster;
  cfg.numAttrs = 2;
  // The notes have blocks of their own in front, up to 32 (the claims' fences and exchanges
  // would keep one head's selection, and so its cluster, 2 us longer).
  const int64_t places = a.same_pool ? (a.max_len + page - 1) / page : own;
  const int note_chunks = static_cast<int>((places + 31) / 32);
  int note_blocks = 0;
  while (note_blocks < 32 && note_blocks * kSelWarps < a.num_seqs * static_cast<int64_t>(note_chunks))
    note_blocks += cluster;
  cfg.gridDim = dim3(static_cast<unsigned>(note_blocks + pairs * cluster));
  if (per <= 4 * kSelThreads) {
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<4, false, false>, a, cluster, note_blocks,
                           note_chunks);
  } else if (per <= 16 * kSelThreads) {
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<16, false, false>, a, cluster, note_blocks,
                           note_chunks);
  } else {
    constexpr int kBytes = kSelThreads * kMaxKeys * 4;
    static std::atomic<uint64_t> ready{0};
    e = allow_smem(reinterpret_cast<const void*>(evict_select_kernel<kMaxKeys, true, false>), kBytes, ready);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = kBytes;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<kMaxKeys, true, false>, a, cluster, note_blocks,
                           note_chunks);
    cfg.dynamicSmemBytes = 0;
  }
  if (e != cudaSuccess) return e;
  const int chunks = static_cast<int>(
      (static_cast<int64_t>(a.budget) * a.hkv + kCopyThreads - 1) / kCopyThreads);
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * chunks));
  cfg.blockDim = dim3(kCopyThreads);
  return cudaLaunchKernelEx(&cfg, evict_copy_kernel, a, chunks);
}

}  // namespace quail

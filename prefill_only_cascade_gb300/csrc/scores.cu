// scores.cu - the attention weight that every cached token receives from a set of queries:
//   score[s, g, j] = sum over queries i that see key j, and heads h of group g, of
//                    exp(c q_ih . k_jg - lse_ih)
// i.e. the column sums of softmax attention, whose row statistics (lse) the attention call
// has already written ("Motor de inferência Quail atinge 1 bilhão de tokens por minuto por
// GPU", section "Como funciona": the anchor is prefilled once and kept; these sums say which
// of its tokens are worth keeping). No second softmax pass is needed, and no V.
//
// The product runs transposed, S^T = K Q^T, one 128-key tile of a (sequence, KV head) per
// CTA: a key is one TMEM lane, so the sum over queries stays in one thread's registers and
// nothing is reduced across lanes, and the result does not depend on any order of atomics.
// K stays in shared memory, 128-row query tiles (128 / G tokens x G heads, as one TMA box)
// stream through a ring, and S^T is double-buffered in TMEM: the tensor cores fill one tile
// while four warps exponentiate the other. Bound: with many queries the exponentials (one
// per (query row, key); ~30 results/clk/SM) and the MMA (~512 clk per 128 x 128 x 128) are
// about equal, with few (a window) reading K once from HBM.
#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kBM = 128;            // keys per tile (TMEM lanes)
constexpr int kBN = 128;            // query rows per tile (TMEM columns)
constexpr int kThreads = 192;       // 4 softmax warps, the TMA warp, the MMA warp
constexpr int kWarpLoad = 4, kWarpMma = 5;
constexpr uint32_t kTmemCols = 256;  // two S^T tiles; two CTAs share an SM
constexpr int kBlock = 128 * 128;   // bytes of 128 rows x 64 columns of bf16

template <int D>
struct Cfg {
  static constexpr int kKB = D / 64;               // 64-column blocks
  static constexpr int kTileBytes = kKB * kBlock;  // of K, and of a query stage
  static constexpr int kStages = 256 / D;
  static constexpr int kSmem = kTileBytes * (1 + kStages) + 1024;  // + alignment slack
};

struct Shared {
  alignas(16) float nlse[2][kBN];   // -lse * log2(e) of the tile's query rows (16-byte loads)
  alignas(16) float part[8][kBM];   // rank 0: the other CTAs' sums
  uint64_t k_full, drain;
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2], s_empty[2];
  uint32_t tmem;
  int abort_flag;
};
static_assert(offsetof(Shared, nlse) % 16 == 0 && alignof(Shared) == 16, "16-byte loads of nlse");

// Waits until `bar` reaches the phase, at most until `deadline`: before leaving, no copy or
// MMA of this CTA may be in flight.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t deadline) {
  while (!mbar_try_wait(smem_u32(bar), parity))
    if (global_timer_ns() > deadline) return;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 columns of S^T: adds exp2(s c + nlse[n]) over the columns n in [lo, hi) (MASK), or all.
template <bool MASK>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const float* nlse, uint64_t c2,
                                            int lo, int hi, uint64_t (&acc)[4]) {
#pragma unroll
  for (int n = 0; n < 32; n += 4) {
    const uint4 l = *reinterpret_cast<const uint4*>(nlse + n);
    const uint64_t x0 = f2_fma(f2(__uint_as_float(s[n]), __uint_as_float(s[n + 1])), c2,
                               f2(__uint_as_float(l.x), __uint_as_float(l.y)));
    const uint64_t x1 = f2_fma(f2(__uint_as_float(s[n + 2]), __uint_as_float(s[n + 3])), c2,
                               f2(__uint_as_float(l.z), __uint_as_float(l.w)));
    float a, b, c, d;
    f2_split(x0, a, b);
    f2_split(x1, c, d);
    a = ex2(a);
    b = ex2(b);
    c = ex2(c);
    d = ex2(d);
    if (MASK) {  // select, not multiply: rows past the end may hold anything
      a = n >= lo && n < hi ? a : 0.f;
      b = n + 1 >= lo && n + 1 < hi ? b : 0.f;
      c = n + 2 >= lo && n + 2 < hi ? c : 0.f;
      d = n + 3 >= lo && n + 3 < hi ? d : 0.f;
    }
    acc[(n >> 1) & 3] = f2_add(acc[(n >> 1) & 3], f2(a, b));
    acc[((n >> 1) + 1) & 3] = f2_add(acc[((n >> 1) + 1) & 3], f2(c, d));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    attn_scores_kernel(const AttnScoresArgs a, const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map, int cluster) {
  using C = Cfg<D>;
  extern __shared__ uint8_t dyn[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~1023ull);
  uint8_t* s_k = smem;
  uint8_t* s_q = smem + C::kTileBytes;
  const int warp = threadIdx.x >> 5;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  // blocks in the order key tile, sequence, head: with causal masking the first key tiles
  // have the most queries, so the long CTAs start first
  int id = blockIdx.x / cluster;
  const int g = id % a.hkv;
  id /= a.hkv;
  const int s = id % a.num_seqs, tile = id / a.num_seqs;
  const int64_t k0 = __ldg(a.k_offsets + s), nk64 = __ldg(a.k_offsets + s + 1) - k0;
  const int64_t q0 = __ldg(a.q_offsets + s), nq64 = __ldg(a.q_offsets + s + 1) - q0;
  if (k0 < 0 || nk64 < 0 || nk64 > a.max_k || k0 + nk64 > a.total_k || q0 < 0 || nq64 < 0 ||
      nq64 > a.max_q || q0 + nq64 > a.total_q) {
    if (threadIdx.x == 0) atomicOr(a.err_word, kErrDeviceBounds);
    return;
  }
  const int nk = static_cast<int>(nk64), nq = static_cast<int>(nq64);
  const int j0 = tile * kBM;
  if (j0 >= nk) return;

  const int G = a.group, tok = kBN / G;
  const int w = a.window > 0 ? min(a.window, nq) : nq;
  const int f = nq - w;               // first query token of the window
  const int off = nk - nq;            // causal: query i sees keys 0 .. i + off
  const int tiles = (w + tok - 1) / tok;
  int t_first = 0;                    // first query tile that sees the key tile
  if (a.causal) {
    const int first_query = j0 - off;  // may be negative
    if (first_query > f) t_first = min(tiles, (first_query - f) / tok);
  }
  // the CTAs of a cluster take the query tiles in turn
  const int mine = tiles - t_first > rank ? (tiles - t_first - rank + cluster - 1) / cluster : 0;

  if (threadIdx.x == 0) {
    mbar_init(&sh.k_full, 1);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 128);
    }
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sh.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (cluster > 1) cluster_sync();  // the others run: their shared memory may be written
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const WaitCtl wc{a.timeout_ns, &sh.abort_flag, a.err_word};

  float total = 0.f;
  if (warp == kWarpLoad) {
    if (mine > 0) {
      const bool leader = elect_one();
      const uint64_t keep = l2_policy_evict_last();  // queries: read by every key tile
      const uint64_t once = l2_policy_evict_first();
      if (leader) {
        mbar_arrive_expect_tx(&sh.k_full, C::kTileBytes);
        for (int kb = 0; kb < C::kKB; ++kb)
          tma_load_3d_hint(&k_map, &sh.k_full, s_k + kb * kBlock, kb * 64, g,
                           static_cast<int>(k0) + j0, once);
      }
      __syncwarp();
      bool ok = true;
      int armed = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const int st = i % C::kStages;
        ok = wait_parity_warp(wc, &sh.q_empty[st], ((i / C::kStages) & 1) ^ 1u);
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(&sh.q_full[st], C::kTileBytes);
          const int t = static_cast<int>(q0) + f + (t_first + rank + i * cluster) * tok;
          for (int kb = 0; kb < C::kKB; ++kb)
            tma_load_3d_hint(&q_map, &sh.q_full[st], s_q + st * C::kTileBytes + kb * kBlock,
                             kb * 64, g * G, t, keep);
        }
        __syncwarp();
        ++armed;
      }
      const uint64_t deadline = global_timer_ns() + 100000000ull;
      drain(&sh.k_full, 0, deadline);
      for (int i = armed > C::kStages ? armed - C::kStages : 0; i < armed; ++i)
        drain(&sh.q_full[i % C::kStages], (i / C::kStages) & 1u, deadline);
    }
  } else if (warp == kWarpMma) {
    if (mine > 0) {
      const bool leader = elect_one();
      constexpr uint32_t kIdesc = idesc_f16(kBM, kBN, 1, 0);
      constexpr uint32_t kDescHi = sw128_desc_hi(1024);  // 8-row groups 1024 bytes apart
      const uint32_t k_lo = sw128_desc_lo(smem_u32(s_k), 16);
      const uint32_t q_lo0 = sw128_desc_lo(smem_u32(s_q), 16);
      bool ok = wait_parity_warp(wc, &sh.k_full, 0);
      for (int i = 0; i < mine && ok; ++i) {
        const int st = i % C::kStages, buf = i & 1;
        ok = wait_parity_warp(wc, &sh.q_full[st], (i / C::kStages) & 1u) &&
             wait_parity_warp(wc, &sh.s_empty[buf], ((i >> 1) & 1) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t q_lo = q_lo0 + st * (C::kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t adv = (kk >> 2) * (kBlock >> 4) + (kk & 3) * 2;
            mma_ss_lohi(tmem + 128u * buf, k_lo + adv, kDescHi, q_lo + adv, kDescHi, kIdesc,
                        kk > 0 ? 1u : 0u);
          }
          mma_commit(&sh.q_empty[st]);
          mma_commit(&sh.s_full[buf]);
        }
        __syncwarp();
      }
      if (leader) mma_commit(&sh.drain);
      __syncwarp();
      drain(&sh.drain, 0, global_timer_ns() + 100000000ull);
    }
  } else {
    const int row = threadIdx.x;      // key j0 + row, TMEM lane `row`
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint64_t c2 = f2(a.scale_log2, a.scale_log2);
    float lost = 0.f;                 // what the running sum has rounded away
    bool ok = true;
    // lse of this thread's query row of tile i, loaded a tile ahead
    auto row_lse = [&](int i) {
      const int t = f + (t_first + rank + i * cluster) * tok + row / G;
      return i < mine && t < nq ? __ldg(a.lse + (q0 + t) * a.hq + g * G + row % G) : 0.f;
    };
    float l = row_lse(0);
    for (int i = 0; i < mine; ++i) {
      const int buf = i & 1;
      // a row that saw nothing (-inf) gives no weight
      sh.nlse[buf][row] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      l = row_lse(i + 1);
      // after a wait that ran out every warp still takes part in the barriers
      ok = ok && __all_sync(0xFFFFFFFFu, wait_parity(wc, &sh.s_full[buf], (i >> 1) & 1u));
      if (!ok) continue;
      tc_fence_after();
      const int t0 = f + (t_first + rank + i * cluster) * tok;
      // query rows [lo, hi) of the tile see this thread's key
      const int hi = nq - t0 >= tok ? kBN : (nq - t0) * G;
      int lo = 0;
      if (a.causal) {
        const int64_t first = (static_cast<int64_t>(j0) + row - off - t0) * G;
        lo = first < 0 ? 0 : first > kBN ? kBN : static_cast<int>(first);
      }
      const bool masked = hi < kBN || (a.causal && j0 + kBM - 1 > t0 + off);
      uint64_t acc[4] = {0, 0, 0, 0};
      uint32_t v[2][32];
      tmem_ld32(t_lane + 128u * buf, v[0]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        tmem_wait_ld_dep(v[q & 1]);
        if (q < 3) {
          tmem_ld32(t_lane + 128u * buf + 32 * (q + 1), v[(q + 1) & 1]);
        } else {  // the tile is in registers: its TMEM may be overwritten
          tc_fence_before();
          mbar_arrive(&sh.s_empty[buf]);
        }
        if (masked)
          add_columns<true>(v[q & 1], &sh.nlse[buf][32 * q], c2, lo - 32 * q, hi - 32 * q, acc);
        else
          add_columns<false>(v[q & 1], &sh.nlse[buf][32 * q], c2, 0, 0, acc);
      }
      float x0, x1, y0, y1;
      f2_split(f2_add(acc[0], acc[1]), x0, x1);
      f2_split(f2_add(acc[2], acc[3]), y0, y1);
      // compensated: thousands of tiles may add up (Kahan)
      const float y = ((x0 + x1) + (y0 + y1)) - lost;
      const float t = total + y;
      lost = fabsf(t) < INFINITY ? (t - total) - y : 0.f;
      total = t;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (cluster > 1) {  // the cluster's sums, added in rank order by its first CTA
    if (rank > 0 && threadIdx.x < kBM)
      st_cluster_f32(cluster_map(&sh.part[rank][threadIdx.x], 0), total);
    cluster_sync();
    if (rank > 0) return;
    if (threadIdx.x < kBM)
      for (int r = 1; r < cluster; ++r) total += sh.part[r][threadIdx.x];
  }
  if (threadIdx.x < kBM && j0 + static_cast<int>(threadIdx.x) < nk) {
    const int64_t at = (static_cast<int64_t>(s) * a.hkv + g) * a.score_stride + j0 + threadIdx.x;
    a.score_out[at] = a.score_in != nullptr ? a.score_in[at] + total : total;
  }
}

template <int D>
cudaError_t launch_t(const AttnScoresArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map,
                     int num_sms, cudaStream_t stream) {
  using C = Cfg<D>;
  cudaError_t e = cudaFuncSetAttribute(attn_scores_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks =
      static_cast<int64_t>((a.max_k + kBM - 1) / kBM) * a.num_seqs * a.hkv;
  // Few key tiles: the query tiles of each are split over a cluster, at least four apiece.
  const int most = a.window > 0 && a.window < a.max_q ? a.window : a.max_q;
  const int64_t tiles = (static_cast<int64_t>(most) * a.group + kBN - 1) / kBN;
  int cluster = 1;
  while (cluster < 8 && blocks * cluster < 2 * num_sms && tiles >= 8 * cluster) cluster *= 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_scores_kernel<D>, a, q_map, k_map, cluster);
}

}  // namespace

cudaError_t launch_attn_scores(const AttnScoresArgs& a, const CUtensorMap& q_map,
                               const CUtensorMap& k_map, int head_dim, int num_sms,
                               cudaStream_t stream) {
  return head_dim == 128 ? launch_t<128>(a, q_map, k_map, num_sms, stream)
                         : launch_t<64>(a, q_map, k_map, num_sms, stream);
}

}  // namespace quail

// scores.cu - the attention weight that every cached token receives from a set of queries:
//   score[s, g, j] = sum over queries i that see key j, and heads h of group g, of
//                    exp(c q_ih . k_jg - lse_ih)
// i.e. the column sums of softmax attention, whose row statistics (lse) the attention call
// has already written ("Motor de inferência Quail atinge 1 bilhão de tokens por minuto por
// GPU", section "Como funciona": the anchor is prefilled once and kept; these sums say which
// of its tokens are worth keeping). No second softmax pass is needed, and no V.
//
// The product runs transposed, S^T = K Q^T, in 128 x 128 tiles: a key is one TMEM lane, so
// the sum over queries stays in one thread's registers, nothing is reduced across lanes and
// the result does not depend on any order of atomics. Two kernels:
//   attn_scores_kernel   a CTA keeps 256 keys of a (sequence, KV head) in shared memory and
//     streams 128-row query tiles (128 / G tokens x G heads, as one TMA box) past them. Per
//     tile and SM the MMA (2 x ~512 clk) and the exponentials (2 x 512 clk of the MUFU) are
//     about equal: 16 softmax warps (four warpgroups, one per key tile and parity of the query
//     tile, each with its own S^T in TMEM) exponentiate while the tensor cores fill the other
//     parity. What bounds it is the hand-over MMA -> softmax -> MMA of each S^T tile, whose
//     latency four tiles in TMEM do not hide (about 1,700 clk per two products instead of
//     1,030): hence an MMA warp per key tile and a warp of its own for the lse. 256 keys and
//     not 128, so that a query tile is read from L2 once per two products (~9 TB/s at full rate
//     instead of 18).
//   attn_scores_window_kernel   where the queries of a (sequence, KV head) fit four tiles (the
//     last 128 tokens at G = 4), they stay in shared memory and the keys stream past them, a
//     warpgroup per key tile: bound by reading K once from HBM with one query tile, by the
//     exponentials with four.

#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kBM = 128;            // keys per tile (TMEM lanes)
constexpr int kBN = 128;            // query rows per tile (TMEM columns)
constexpr int kBlock = 128 * 128;   // bytes of 128 rows x 64 columns of bf16
constexpr int kMaxCluster = 8;

// attn_scores_kernel
constexpr int kKeyTiles = 2;        // key tiles of a CTA
constexpr int kGroups = 2 * kKeyTiles;  // softmax warpgroups: (key tile, query tile parity)
constexpr int kThreads = 128 * kGroups + 128;  // + TMA, an MMA warp per key tile, lse
constexpr int kWarpLoad = 4 * kGroups, kWarpMma = 4 * kGroups + 1, kWarpLse = 4 * kGroups + 3;
constexpr int kQStages = 4;

// attn_scores_window_kernel
constexpr int kWinMaxQ = 4;                 // query tiles kept at most
// QT query tiles kept: the warpgroups that take the key tiles in turn, key tiles in flight,
// and S^T tiles of a warpgroup. One: two CTAs share an SM. Two: four warpgroups keep the MUFU
// busier than two. Four: shared memory has no room for more than two key tiles.
template <int QT>
struct Win {
  static constexpr int kGroups = QT == 2 ? 4 : 2;
  static constexpr int kStages = kGroups;
  static constexpr int kBufs = QT == 4 ? 2 : 1;
  static constexpr int kTmem = 128 * kGroups * kBufs;
  static constexpr int kThreads = 128 * kGroups + 64;  // + the TMA warp and the MMA warp
  static constexpr int kLoad = 4 * kGroups, kMma = 4 * kGroups + 1;
};

template <int D>
struct Cfg {
  static constexpr int kKB = D / 64;               // 64-column blocks
  static constexpr int kTileBytes = kKB * kBlock;  // 128 rows of K or Q
  static constexpr int kSmem = kTileBytes * (kKeyTiles + kQStages) + 1024;  // + alignment slack
  static constexpr int win_smem(int q_tiles, int stages) {
    return kTileBytes * (q_tiles + stages) + 1024;
  }
};

struct Shared {
  alignas(16) float nlse[kQStages][kBN];    // -lse * log2(e) of a tile's query rows
  alignas(16) float part[kMaxCluster][kKeyTiles * kBM];  // others' sums: rank 0's own odd
                                            // tiles in row 0, the cluster's CTAs behind
  uint64_t k_full, drain[kKeyTiles];
  uint64_t q_full[kQStages], q_empty[kQStages], l_full[kQStages], l_empty[kQStages];
  uint64_t s_full[kGroups], s_empty[kGroups];
  uint32_t tmem;
  int abort_flag;
  uint32_t others_failed;                   // rank 0: a wait ran out in another CTA
  int dead[kQStages];                       // the tile has rows whose lse is -inf
};
struct WinShared {
  alignas(16) float nlse[kWinMaxQ * kBN];
  uint64_t q_full, drain;
  uint64_t k_full[4], k_empty[4];
  uint64_t s_full[4][2], s_empty[4][2];     // [warpgroup][buffer]
  uint32_t tmem;
  int abort_flag;
};
static_assert(offsetof(Shared, nlse) % 16 == 0 && offsetof(WinShared, nlse) % 16 == 0 &&
                  alignof(Shared) == 16 && alignof(WinShared) == 16,
              "16-byte loads of nlse");

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

// 16 columns of S^T: adds exp2(s c + nlse[n]) over the columns n in [lo, hi) (MASK), of them
// those whose nlse is not -inf (DEAD), or all.
template <bool MASK, bool DEAD>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[16], const float* nlse, uint64_t c2,
                                            int lo, int hi, uint64_t (&acc)[4]) {
#pragma unroll
  for (int n = 0; n < 16; n += 4) {
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
    // select, not multiply: rows past the end, or of no weight, may hold anything
    if (MASK) {
      a = n >= lo && n < hi && (!DEAD || __uint_as_float(l.x) != -INFINITY) ? a : 0.f;
      b = n + 1 >= lo && n + 1 < hi && (!DEAD || __uint_as_float(l.y) != -INFINITY) ? b : 0.f;
      c = n + 2 >= lo && n + 2 < hi && (!DEAD || __uint_as_float(l.z) != -INFINITY) ? c : 0.f;
      d = n + 3 >= lo && n + 3 < hi && (!DEAD || __uint_as_float(l.w) != -INFINITY) ? d : 0.f;
    }
    acc[(n >> 1) & 3] = f2_add(acc[(n >> 1) & 3], f2(a, b));
    acc[((n >> 1) + 1) & 3] = f2_add(acc[((n >> 1) + 1) & 3], f2(c, d));
  }
}

// What sequence s asks for: key and query ranges, and the queries of the window.
struct SeqRange {
  int64_t k0, q0;
  int nk, nq;
  int w;    // queries of the window
  int f;    // the first of them
  int off;  // causal: query i sees keys 0 .. i + off
};
__device__ __forceinline__ bool seq_range(const AttnScoresArgs& a, int s, SeqRange& r) {
  r.k0 = __ldg(a.k_offsets + s);
  r.q0 = __ldg(a.q_offsets + s);
  const int64_t nk = __ldg(a.k_offsets + s + 1) - r.k0, nq = __ldg(a.q_offsets + s + 1) - r.q0;
  if (r.k0 < 0 || nk < 0 || nk > a.max_k || r.k0 + nk > a.total_k || r.q0 < 0 || nq < 0 ||
      nq > a.max_q || r.q0 + nq > a.total_q)
    return false;
  r.nk = static_cast<int>(nk);
  r.nq = static_cast<int>(nq);
  r.w = a.window > 0 ? min(a.window, r.nq) : r.nq;
  r.f = r.nq - r.w;
  r.off = r.nk - r.nq;
  return true;
}

// The sequence with the slot-th most queries in its window (of up to 32; every warp for itself).
__device__ __forceinline__ int seq_by_queries(const AttnScoresArgs& a, int slot) {
  const int lane = threadIdx.x & 31;
  int w = -1;
  if (lane < a.num_seqs) {
    w = max(0, __ldg(a.q_offsets + lane + 1) - __ldg(a.q_offsets + lane));
    if (a.window > 0) w = min(w, a.window);
  }
  int rank = 0;
  for (int i = 0; i < a.num_seqs; ++i) {
    const int other = __shfl_sync(0xFFFFFFFFu, w, i);
    rank += other > w || (other == w && i < lane);
  }
  return __ffs(__ballot_sync(0xFFFFFFFFu, rank == slot && lane < a.num_seqs)) - 1;
}

// Adds the weights of one S^T tile (in TMEM at t_tile, this thread's lane) that this thread's
// key receives: those of the query rows [lo, hi). lo_first and lo_last are the warp's first
// and last lanes' lo: 16 columns that no lane sees are skipped, those that all see take no
// mask unless the tile has dead rows (lse -inf; telling them apart from the others costs 0.6 %
// of 4 x 4,096 tokens, 1.5 % where every tile would otherwise be without a mask). Pieces of 16
// columns, the next one loading while one is worked on (32 at a time without that measured
// 222 us instead of 217, 4 x 4,096 tokens). Releases the TMEM tile as soon as it is in
// registers.
__device__ __forceinline__ float tile_weight(uint32_t t_tile, const float* nlse, uint64_t c2, int lo,
                                             int lo_first, int lo_last, int hi, bool dead,
                                             uint64_t* s_empty) {
  uint64_t acc[4] = {0, 0, 0, 0};
  if (lo_last == 0 && hi == kBN && !dead) {  // most tiles
    uint32_t v[2][16];
    tmem_ld16(t_tile, v[0]);
#pragma unroll
    for (int q = 0; q < kBN / 16; ++q) {
      tmem_wait_ld16_dep(v[q & 1]);
      if (q < kBN / 16 - 1) {
        tmem_ld16(t_tile + 16 * (q + 1), v[(q + 1) & 1]);
      } else {
        tc_fence_before();
        mbar_arrive(s_empty);
      }
      add_columns<false, false>(v[q & 1], nlse + 16 * q, c2, 0, 0, acc);
    }
  } else {
    const int q0 = lo_first >> 4, q1 = (hi + 15) >> 4;
    if (q0 >= q1) mbar_arrive(s_empty);
#pragma unroll 1
    for (int q = q0; q < q1; ++q) {
      uint32_t v[16];
      tmem_ld16(t_tile + 16 * q, v);
      tmem_wait_ld16_dep(v);
      if (q == q1 - 1) {
        tc_fence_before();
        mbar_arrive(s_empty);
      }
      if (lo_last <= 16 * q && 16 * q + 16 <= hi && !dead)
        add_columns<false, false>(v, nlse + 16 * q, c2, 0, 0, acc);
      else if (!dead)
        add_columns<true, false>(v, nlse + 16 * q, c2, lo - 16 * q, hi - 16 * q, acc);
      else
        add_columns<true, true>(v, nlse + 16 * q, c2, lo - 16 * q, hi - 16 * q, acc);
    }
  }
  float x0, x1, y0, y1;
  f2_split(f2_add(acc[0], acc[1]), x0, x1);
  f2_split(f2_add(acc[2], acc[3]), y0, y1);
  return (x0 + x1) + (y0 + y1);
}

// First query row of the tile at query token t0 that sees key j.
__device__ __forceinline__ int first_row(int j, int off, int t0, int G) {
  const int64_t n = (static_cast<int64_t>(j) - off - t0) * G;
  return n < 0 ? 0 : n > kBN ? kBN : static_cast<int>(n);
}

template <int D>
__device__ __forceinline__ void mma_tile(uint32_t d_tmem, uint32_t k_lo, uint32_t q_lo) {
  constexpr uint32_t kIdesc = idesc_f16(kBM, kBN, 1, 0);
  constexpr uint32_t kDescHi = sw128_desc_hi(1024);  // 8-row groups 1024 bytes apart
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t adv = (kk >> 2) * (kBlock >> 4) + (kk & 3) * 2;
    mma_ss_lohi(d_tmem, k_lo + adv, kDescHi, q_lo + adv, kDescHi, kIdesc, kk > 0 ? 1u : 0u);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_scores_kernel(const AttnScoresArgs a, const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap k_map, int cluster, int key_blocks) {
  using C = Cfg<D>;
  extern __shared__ uint8_t dyn[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~1023ull);
  uint8_t* s_k = smem;
  uint8_t* s_q = smem + kKeyTiles * C::kTileBytes;
  const int warp = threadIdx.x >> 5;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  // The long CTAs start first: with causal masking the first keys, which have the most queries,
  // of all sequences, otherwise the sequences by their queries, as found here (8 anchors, 2,000
  // to 4,000 queries each: 157 us instead of 163; it costs a CTA 0.5 us).
  int id = blockIdx.x / cluster;
  const int g = id % a.hkv;
  id /= a.hkv;
  int s, j0;
  if (a.causal) {
    s = id % a.num_seqs;
    j0 = id / a.num_seqs * (kKeyTiles * kBM);
  } else {
    s = id / key_blocks;
    j0 = id % key_blocks * (kKeyTiles * kBM);
    if (a.num_seqs <= 32) s = seq_by_queries(a, s);
  }
  SeqRange sr;
  if (!seq_range(a, s, sr)) {
    if (threadIdx.x == 0) atomicOr(a.err_word, kErrDeviceBounds);
    return;
  }
  if (j0 >= sr.nk) return;

  const int G = a.group, tok = kBN / G;
  const int tiles = (sr.w + tok - 1) / tok;
  // first query tile that sees each key tile (tiles: none, or no such keys)
  int t_first[kKeyTiles];
#pragma unroll
  for (int kt = 0; kt < kKeyTiles; ++kt) {
    const int query = j0 + kt * kBM - sr.off - sr.f;  // of the window; may be negative
    t_first[kt] = a.causal && query > 0 ? min(tiles, query / tok) : 0;
    if (j0 + kt * kBM >= sr.nk) t_first[kt] = tiles;
  }
  // the CTAs of a cluster take the query tiles in turn: this one's i-th is tile_at(i)
  const int left = tiles - t_first[0];
  const int mine = left > rank ? (left - rank + cluster - 1) / cluster : 0;
  auto tile_at = [&](int i) { return t_first[0] + rank + i * cluster; };

  // fault injection: the first keys never reach the last CTA of a cluster
  const bool skip_k = a.inject_skip_first_kv != 0 && j0 == 0 && rank == cluster - 1;
  const uint64_t keep = l2_policy_evict_last();   // queries: read by every key tile
  const uint64_t once = l2_policy_evict_first();
  auto load_q = [&](int i) {
    const int st = i % kQStages, t = static_cast<int>(sr.q0) + sr.f + tile_at(i) * tok;
    mbar_arrive_expect_tx(&sh.q_full[st], C::kTileBytes);
    for (int kb = 0; kb < C::kKB; ++kb)
      tma_load_3d_hint(&q_map, &sh.q_full[st], s_q + st * C::kTileBytes + kb * kBlock, kb * 64,
                       g * G, t, keep);
  };
  if (threadIdx.x == 32 * kWarpLoad) {
    mbar_init(&sh.k_full, 1);
    for (int i = 0; i < kKeyTiles; ++i) mbar_init(&sh.drain[i], 1);
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], kKeyTiles);  // both MMA warps
      mbar_init(&sh.l_full[i], 32);
      mbar_init(&sh.l_empty[i], 4 * kKeyTiles);  // the warps that read it
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 128);
    }
    sh.abort_flag = 0;
    sh.others_failed = 0;
    fence_mbar_init();
    if (mine > 0) {  // the first loads do not wait for the rest of the set-up
      if (!skip_k) mbar_arrive_expect_tx(&sh.k_full, kKeyTiles * C::kTileBytes);
      for (int kt = 0; kt < (skip_k ? 0 : kKeyTiles); ++kt)  // keys past the tensor read as zeros
        for (int kb = 0; kb < C::kKB; ++kb)
          tma_load_3d_hint(&k_map, &sh.k_full, s_k + kt * C::kTileBytes + kb * kBlock, kb * 64, g,
                           static_cast<int>(sr.k0) + j0 + kt * kBM, once);
      for (int i = 0; i < min(mine, kQStages); ++i) load_q(i);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sh.tmem, 128 * kGroups);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  // Waited for at the end, when the TMEM columns are free again: all 512 of an SM are taken here,
  // and a CTA that kept them while it waits for its cluster could keep another cluster's CTA from
  // theirs, which that cluster's other CTAs wait for in turn.
  if (cluster > 1) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const WaitCtl wc{a.timeout_ns, &sh.abort_flag, a.err_word};

  float total = 0.f;
  if (warp == kWarpLoad) {
    if (mine > 0) {
      bool ok = true;
      int armed = min(mine, kQStages);
      for (int i = armed; i < mine && ok; ++i) {
        ok = wait_parity_warp(wc, &sh.q_empty[i % kQStages], ((i / kQStages) & 1) ^ 1u);
        if (!ok) break;
        if ((threadIdx.x & 31) == 0) load_q(i);
        __syncwarp();
        ++armed;
      }
      const uint64_t deadline = global_timer_ns() + 100000000ull;
      if (!skip_k) drain(&sh.k_full, 0, deadline);
      for (int i = armed > kQStages ? armed - kQStages : 0; i < armed; ++i)
        drain(&sh.q_full[i % kQStages], (i / kQStages) & 1u, deadline);
    }
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    if (mine > 0) {
      const int kt = warp - kWarpMma;  // each issues the products of one key tile
      const bool leader = elect_one();
      const uint32_t k_lo = sw128_desc_lo(smem_u32(s_k), 16);
      const uint32_t q_lo = sw128_desc_lo(smem_u32(s_q), 16);
      const int from = kt == 0 ? t_first[0] : t_first[1];
      uint32_t used[2] = {0, 0};
      bool ok = wait_parity_warp(wc, &sh.k_full, 0);
      for (int i = 0; i < mine && ok; ++i) {
        const int st = i % kQStages;
        ok = wait_parity_warp(wc, &sh.q_full[st], (i / kQStages) & 1u);
        if (!ok) break;
        if (tile_at(i) >= from) {
          const int grp = 2 * kt + (i & 1);
          const uint32_t parity = ((i & 1) ? used[1] : used[0]) & 1u;
          ok = wait_parity_warp(wc, &sh.s_empty[grp], parity ^ 1u);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            mma_tile<D>(tmem + 128u * grp, k_lo + kt * (C::kTileBytes >> 4),
                        q_lo + st * (C::kTileBytes >> 4));
            mma_commit(&sh.s_full[grp]);
          }
          __syncwarp();
          if (i & 1) ++used[1]; else ++used[0];
        }
        if (leader) mma_commit(&sh.q_empty[st]);
        __syncwarp();
      }
      if (leader) mma_commit(&sh.drain[kt]);
      __syncwarp();
      drain(&sh.drain[kt], 0, global_timer_ns() + 100000000ull);
    }
  } else if (warp == kWarpLse) {
    // -lse log2(e) of every tile's query rows, four tiles ahead. G divides 128, so the rows
    // lane + 32 j of a tile are tokens and heads at fixed places of it.
    const int lane = threadIdx.x & 31;
    int dt[4];
    const float* at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dt[j] = (lane + 32 * j) / G;
      at[j] = a.lse + (sr.q0 + sr.f + dt[j]) * a.hq + g * G + (lane + 32 * j) % G;
    }
    const int64_t per_token = a.hq;
    float l[4][4];
    auto load = [&](int i, float (&x)[4]) {
      const int t = tile_at(i) * tok, left = i < mine ? sr.w - t : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = dt[j] < left ? __ldg(at[j] + t * per_token) : 0.f;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) load(k, l[k]);
    bool ok = true;
    for (int i0 = 0; i0 < mine && ok; i0 += 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k, st = i % kQStages;
        if (i >= mine || !ok) break;
        ok = wait_parity_warp(wc, &sh.l_empty[st], ((i / kQStages) & 1) ^ 1u);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sh.nlse[st][lane + 32 * j] =
              l[k][j] == -INFINITY ? -INFINITY : l[k][j] * -1.4426950408889634f;
        const bool dead = __any_sync(0xFFFFFFFFu, l[k][0] == -INFINITY || l[k][1] == -INFINITY ||
                                                      l[k][2] == -INFINITY || l[k][3] == -INFINITY);
        if (lane == 0) sh.dead[st] = dead;
        mbar_arrive(&sh.l_full[st]);
        load(i + 4, l[k]);
      }
    }
  } else {
    const int grp = warp >> 2, kt = grp >> 1;
    const int row = threadIdx.x & 127;  // key j0 + 128 kt + row, TMEM lane `row`
    const int key = j0 + kt * kBM + row;
    const uint32_t t_tile = tmem + 128u * grp + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t c2 = f2(a.scale_log2, a.scale_log2);
    const int from = kt == 0 ? t_first[0] : t_first[1];
    float lost = 0.f;                   // what the running sum has rounded away
    uint32_t n = 0;                     // S^T tiles of this group so far
    for (int i = grp & 1; i < mine; i += 2) {
      const int st = i % kQStages;
      // also where it sees no key: one release of a stage per tile, in the tiles' order
      bool ok = wait_parity_warp(wc, &sh.l_full[st], (i / kQStages) & 1u);
      if (!ok) break;
      const bool dead = sh.dead[st] != 0;
      if (tile_at(i) >= from) {
        ok = wait_parity_warp(wc, &sh.s_full[grp], n & 1u);
        if (!ok) break;
        ++n;
        tc_fence_after();
        const int t0 = sr.f + tile_at(i) * tok;
        const int hi = sr.nq - t0 >= tok ? kBN : (sr.nq - t0) * G;
        int lo = 0, lo_first = 0, lo_last = 0;
        if (a.causal && j0 + (kt + 1) * kBM - 1 > t0 + sr.off) {
          lo = first_row(key, sr.off, t0, G);
          lo_first = __shfl_sync(0xFFFFFFFFu, lo, 0);
          lo_last = __shfl_sync(0xFFFFFFFFu, lo, 31);
        }
        // compensated: thousands of tiles may add up (Kahan)
        const float y =
            tile_weight(t_tile, sh.nlse[st], c2, lo, lo_first, lo_last, hi, dead,
                        &sh.s_empty[grp]) - lost;
        const float sum = total + y;
        lost = fabsf(sum) < INFINITY ? (sum - total) - y : 0.f;
        total = sum;
      }
      __syncwarp();  // the warp has read nlse
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.l_empty[st]);
    }
    if (grp & 1) sh.part[0][kt * kBM + row] = total;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 128 * kGroups);
  }
  const bool owner = warp < kWarpLoad && !((warp >> 2) & 1);  // the even groups
  const int at = (warp >> 3) * kBM + (threadIdx.x & 127);     // key of the thread
  if (owner) total += sh.part[0][at];
  bool failed = sh.abort_flag != 0;  // a wait ran out: the sums are not whole
  if (cluster > 1) {  // the cluster's sums, added in rank order by its first CTA
    cluster_wait();   // the others run: their shared memory may be written
    if (rank > 0 && owner) st_cluster_f32(cluster_map(&sh.part[rank][at], 0), total);
    if (rank > 0 && failed && threadIdx.x == 0) st_cluster_u32(cluster_map(&sh.others_failed, 0), 1u);
    cluster_sync();
    if (rank > 0) return;
    failed |= sh.others_failed != 0;
    if (owner)
      for (int r = 1; r < cluster; ++r) total += sh.part[r][at];
  }
  if (owner && !failed && j0 + at < sr.nk) {
    const int64_t out = (static_cast<int64_t>(s) * a.hkv + g) * a.score_stride + j0 + at;
    a.score_out[out] = a.score_in != nullptr ? a.score_in[out] + total : total;
  }
}

// QT: query tiles that fit (1, 2 or 4).
template <int D, int QT>
__global__ void __launch_bounds__(Win<QT>::kThreads, QT == 1 ? 2 : 1)
    attn_scores_window_kernel(const AttnScoresArgs a, const __grid_constant__ CUtensorMap q_map,
                              const __grid_constant__ CUtensorMap k_map, int run) {
  using C = Cfg<D>;
  using W = Win<QT>;
  extern __shared__ uint8_t dyn[];
  __shared__ WinShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~1023ull);
  uint8_t* s_q = smem;
  uint8_t* s_k = smem + QT * C::kTileBytes;
  const int warp = threadIdx.x >> 5;
  int id = blockIdx.x;
  const int g = id % a.hkv;
  id /= a.hkv;
  const int s = id % a.num_seqs;
  const int j0 = id / a.num_seqs * run * kBM;
  SeqRange sr;
  if (!seq_range(a, s, sr)) {
    if (threadIdx.x == 0) atomicOr(a.err_word, kErrDeviceBounds);
    return;
  }
  if (j0 >= sr.nk) return;
  const int G = a.group;
  const int count = min(run, (sr.nk - j0 + kBM - 1) / kBM);  // key tiles of this CTA
  const int64_t out0 = (static_cast<int64_t>(s) * a.hkv + g) * a.score_stride;
  if (sr.w == 0) {  // no queries
    for (int j = j0 + threadIdx.x; j < min(sr.nk, j0 + count * kBM); j += W::kThreads)
      a.score_out[out0 + j] = a.score_in != nullptr ? a.score_in[out0 + j] : 0.f;
    return;
  }

  const int tok = kBN / G, q_tiles = (sr.w + tok - 1) / tok;  // at most QT
  const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
  const int k_skip = a.inject_skip_first_kv != 0 && j0 == 0;  // fault injection: without tile 0
  auto load_k = [&](int i) {
    const int st = i % W::kStages;
    mbar_arrive_expect_tx(&sh.k_full[st], C::kTileBytes);
    for (int kb = 0; kb < C::kKB; ++kb)
      tma_load_3d_hint(&k_map, &sh.k_full[st], s_k + st * C::kTileBytes + kb * kBlock, kb * 64, g,
                       static_cast<int>(sr.k0) + j0 + i * kBM, once);
  };
  if (threadIdx.x == 32 * W::kLoad) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.drain, 1);
    for (int i = 0; i < W::kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < 2 * W::kGroups; ++i) {
      mbar_init(&sh.s_full[i >> 1][i & 1], 1);
      mbar_init(&sh.s_empty[i >> 1][i & 1], 128);
    }
    sh.abort_flag = 0;
    fence_mbar_init();
    // the first loads do not wait for the rest of the set-up
    mbar_arrive_expect_tx(&sh.q_full, q_tiles * C::kTileBytes);
    for (int qt = 0; qt < q_tiles; ++qt)
      for (int kb = 0; kb < C::kKB; ++kb)
        tma_load_3d_hint(&q_map, &sh.q_full, s_q + qt * C::kTileBytes + kb * kBlock, kb * 64, g * G,
                         static_cast<int>(sr.q0) + sr.f + qt * tok, keep);
    for (int i = k_skip; i < min(count, W::kStages); ++i) load_k(i);
  }
  if (warp == W::kMma) {
    tmem_alloc(&sh.tmem, W::kTmem);
    tmem_relinquish();
  }
  bool mine = false;  // of this thread's rows one has an lse of -inf
  for (int r = threadIdx.x; r < q_tiles * kBN; r += W::kThreads) {
    const int t = sr.f + r / G;
    const float l = t < sr.nq ? __ldg(a.lse + (sr.q0 + t) * a.hq + g * G + r % G) : 0.f;
    sh.nlse[r] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
    mine |= l == -INFINITY;
  }
  tc_fence_before();
  const bool dead = __syncthreads_or(mine);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const WaitCtl wc{a.timeout_ns, &sh.abort_flag, a.err_word};

  if (warp == W::kLoad) {
    bool ok = true;
    int armed = min(count, W::kStages);
    for (int i = armed; i < count && ok; ++i) {
      ok = wait_parity_warp(wc, &sh.k_empty[i % W::kStages], ((i / W::kStages) & 1) ^ 1u);
      if (!ok) break;
      if ((threadIdx.x & 31) == 0) load_k(i);
      __syncwarp();
      ++armed;
    }
    const uint64_t deadline = global_timer_ns() + 100000000ull;
    drain(&sh.q_full, 0, deadline);
    for (int i = armed > W::kStages ? armed - W::kStages : k_skip; i < armed; ++i)
      drain(&sh.k_full[i % W::kStages], (i / W::kStages) & 1u, deadline);
  } else if (warp == W::kMma) {
    const bool leader = elect_one();
    const uint32_t k_lo = sw128_desc_lo(smem_u32(s_k), 16);
    const uint32_t q_lo = sw128_desc_lo(smem_u32(s_q), 16);
    bool ok = wait_parity_warp(wc, &sh.q_full, 0);
    // the warpgroups' key tiles side by side, query tile by query tile
    for (int i0 = 0, n = 0; i0 < count && ok; i0 += W::kGroups) {
      for (int qt = 0; qt < q_tiles && ok; ++qt, ++n) {
        const int buf = n % W::kBufs;
        const uint32_t parity = ((n / W::kBufs) & 1u) ^ 1u;
        for (int grp = 0; grp < W::kGroups && i0 + grp < count && ok; ++grp) {
          const int st = (i0 + grp) % W::kStages;
          ok = (qt > 0 || wait_parity_warp(wc, &sh.k_full[st], ((i0 + grp) / W::kStages) & 1u)) &&
               wait_parity_warp(wc, &sh.s_empty[grp][buf], parity);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            mma_tile<D>(tmem + 128u * (grp * W::kBufs + buf), k_lo + st * (C::kTileBytes >> 4),
                        q_lo + qt * (C::kTileBytes >> 4));
            if (qt == q_tiles - 1) mma_commit(&sh.k_empty[st]);
            mma_commit(&sh.s_full[grp][buf]);
          }
          __syncwarp();
        }
      }
    }
    if (leader) mma_commit(&sh.drain);
    __syncwarp();
    drain(&sh.drain, 0, global_timer_ns() + 100000000ull);
  } else {
    const int grp = warp >> 2, row = threadIdx.x & 127;
    const uint32_t t_lane =
        tmem + 128u * grp * W::kBufs + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t c2 = f2(a.scale_log2, a.scale_log2);
    int n = 0;                          // S^T tiles so far
    bool ok = true;
    for (int i = grp; i < count && ok; i += W::kGroups) {
      const int key = j0 + i * kBM + row;
      const bool real = key < sr.nk;
      const float base = real && a.score_in != nullptr ? a.score_in[out0 + key] : 0.f;
      float w = 0.f;
      for (int qt = 0; qt < q_tiles; ++qt, ++n) {
        const int buf = n % W::kBufs;
        ok = __all_sync(0xFFFFFFFFu, wait_parity(wc, &sh.s_full[grp][buf], (n / W::kBufs) & 1u));
        if (!ok) break;
        tc_fence_after();
        const int t0 = sr.f + qt * tok, rows = min(kBN, (sr.w - qt * tok) * G);
        int lo = 0, lo_first = 0, lo_last = 0;
        if (a.causal && j0 + (i + 1) * kBM - 1 > t0 + sr.off) {
          lo = first_row(key, sr.off, t0, G);
          lo_first = __shfl_sync(0xFFFFFFFFu, lo, 0);
          lo_last = __shfl_sync(0xFFFFFFFFu, lo, 31);
        }
        w += tile_weight(t_lane + 128u * buf, sh.nlse + qt * kBN, c2, lo, lo_first, lo_last, rows, dead,
                         &sh.s_empty[grp][buf]);
      }
      if (real && ok) a.score_out[out0 + key] = base + w;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, W::kTmem);
  }
}

template <int D, int QT>
cudaError_t launch_window(const AttnScoresArgs& a, const CUtensorMap& q_map,
                          const CUtensorMap& k_map, int num_sms, cudaStream_t stream) {
  constexpr int kBytes = Cfg<D>::win_smem(QT, Win<QT>::kStages);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(
      reinterpret_cast<const void*>(attn_scores_window_kernel<D, QT>), kBytes, ready);
  if (e != cudaSuccess) return e;
  // Runs of key tiles, as long as there are two blocks per SM: a block costs 4-5 us besides
  // its tiles. Runs of 2, 4, 8 and 16 tiles measured 47, 37, 32 and 32 us (64 prompts of
  // 128-2,048 tokens, the last 32 tokens of each).
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  const int key_tiles = (a.max_k + kBM - 1) / kBM;
  int run = 16;
  while (run > 1 && pairs * ((key_tiles + run - 1) / run) < 2 * num_sms) run /= 2;
  const unsigned blocks = static_cast<unsigned>(pairs * ((key_tiles + run - 1) / run));
  attn_scores_window_kernel<D, QT><<<blocks, Win<QT>::kThreads, kBytes, stream>>>(a, q_map, k_map, run);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_t(const AttnScoresArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map,
                     int num_sms, cudaStream_t stream) {
  using C = Cfg<D>;
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  const int most = a.window > 0 && a.window < a.max_q ? a.window : a.max_q;
  const int64_t tiles = (static_cast<int64_t>(most) * a.group + kBN - 1) / kBN;
  if (tiles <= 1) return launch_window<D, 1>(a, q_map, k_map, num_sms, stream);
  if (tiles <= 2) return launch_window<D, 2>(a, q_map, k_map, num_sms, stream);
  if (tiles <= kWinMaxQ) return launch_window<D, kWinMaxQ>(a, q_map, k_map, num_sms, stream);
  cudaError_t e;
  static std::atomic<uint64_t> ready{0};
  e = allow_smem(reinterpret_cast<const void*>(attn_scores_kernel<D>), C::kSmem, ready);
  if (e != cudaSuccess) return e;
  const int key_blocks = (a.max_k + kKeyTiles * kBM - 1) / (kKeyTiles * kBM);
  const int64_t blocks = key_blocks * pairs;
  // Few blocks for the GPU: the query tiles of each are split over a cluster, until there
  // are two blocks per SM, at least eight tiles apiece. A block costs about 5 us besides its
  // tiles (~1 us each): four per SM measured 260 us against 242 (4 x 4,096 tokens, all
  // queries) and 199 against 178 (8 anchors of 1,024 tokens, ~3,000 queries each).
  int cluster = 1;
  while (cluster < kMaxCluster && blocks * cluster < 2 * num_sms && tiles >= 16 * cluster)
    cluster *= 2;
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
  return cudaLaunchKernelEx(&cfg, attn_scores_kernel<D>, a, q_map, k_map, cluster, key_blocks);
}

}  // namespace

cudaError_t launch_attn_scores(const AttnScoresArgs& a, const CUtensorMap& q_map,
                               const CUtensorMap& k_map, int head_dim, int num_sms,
                               cudaStream_t stream) {
  return head_dim == 128 ? launch_t<128>(a, q_map, k_map, num_sms, stream)
                         : launch_t<64>(a, q_map, k_map, num_sms, stream);
}

}  // namespace quail

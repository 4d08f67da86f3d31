// paged_decode.cuh - what the attention kernels over a paged key/value cache share, whatever
// form the pages hold their values in: how a batch's tiles are dealt out, the pieces of a run,
// the join of their parts, the weights of cached tokens, and the launches.
#pragma once
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;

constexpr int kOneCluster = 8;                       // CTAs that share a small call's head
constexpr int kStages = 3;                           // steps in a warp's ring

// 16 bytes from global to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t smem, const uint8_t* p, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(p),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x = hi + lo in f16: 22 bits, down to f16's smallest step.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack2<true>(x0, x1);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack2<true>(x0 - h.x, x1 - h.y);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// x = hi + mid + lo in bf16: all 24 bits, 8 at a time from the top. Where mid and lo are zero they
// take 2^-30 of hi (far under fp32's rounding), so that all three of a positive x are positive: an
// infinite V times zero would be NaN.
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& mid,
                                           uint32_t& lo) {
  auto top = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
  auto tops = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); };
  hi = tops(x0, x1);
  x0 -= top(x0);
  x1 -= top(x1);
  const uint32_t least = mul_bf16x2(hi, 0x30803080u);
  mid = max_bf16x2(tops(x0, x1), least);
  lo = max_bf16x2(tops(x0 - top(x0), x1 - top(x1)), least);
}

// First tile of CTA c when `total` tiles are dealt to n CTAs.
__device__ __forceinline__ int64_t first_tile(int c, int64_t total, int n) {
  return static_cast<int64_t>(c) * total / n;
}

// The length of sequence b if it is one the call allows, else -1.
__device__ __forceinline__ int checked_len(const PagedDecodeArgs& a, int b) {
  const int n = a.lens[b];
  return n >= 0 && n <= a.max_len ? n : -1;
}

// Where a CTA's run of tiles begins.
struct RunStart {
  int64_t total;      // tiles of the batch
  int64_t begin;      // first tile of this CTA
  int64_t end;        // one past its last
  int seq;            // sequence of tile `begin`
  int64_t seq_tile0;  // first tile of that sequence
};

// Every warp scans the lengths for itself (a few KB from L2, 32 at a time), which costs less
// than a launch before this one, or a barrier.
__device__ RunStart find_run(const PagedDecodeArgs& a, int tile, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  auto tiles_of = [&](int b) {
    const int n = b < a.num_seqs ? checked_len(a, b) : 0;
    return n > 0 ? static_cast<unsigned>((n + tile - 1) / tile) : 0u;
  };
  int64_t total = 0;
#pragma unroll 4
  for (int base = 0; base < a.num_seqs; base += 32)
    total += __reduce_add_sync(0xFFFFFFFFu, tiles_of(base + lane));
  total *= a.hkv;
  RunStart run{total, first_tile(cta, total, ctas), first_tile(cta + 1, total, ctas), 0, 0};
  if (run.begin >= run.end) return run;
  int64_t at = 0;  // tiles of one head before `base`
  for (int base = 0; base < a.num_seqs; base += 32) {
    const unsigned t = tiles_of(base + lane);
    const unsigned sum = __reduce_add_sync(0xFFFFFFFFu, t);
    if (run.begin < (at + sum) * a.hkv) {
      unsigned x = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, off);
        if (lane >= off) x += y;
      }
      const int hit = __ffs(__ballot_sync(0xFFFFFFFFu, run.begin < (at + x) * a.hkv)) - 1;
      run.seq = base + hit;
      run.seq_tile0 = (at + __shfl_sync(0xFFFFFFFFu, x - t, hit)) * a.hkv;
      break;
    }
    at += sum;
  }
  return run;
}

// A piece of the run: keys [kb, ke) of sequence b and KV head g.
struct Piece {
  int b, g, len, kb, ke;
  int64_t at;      // its first tile
  int64_t piece0;  // first tile of (b, g)
  int64_t stop;    // one past its last tile
  bool whole;      // all of (b, g)
};

template <int TILE>
__device__ __forceinline__ void set_piece(const PagedDecodeArgs& a, int64_t end, Piece& p) {
  const int tiles = (p.len + TILE - 1) / TILE;
  p.stop = min(end, p.piece0 + tiles);
  p.kb = static_cast<int>(p.at - p.piece0) * TILE;
  p.ke = min(p.len, static_cast<int>(p.stop - p.piece0) * TILE);
  p.whole = p.at == p.piece0 && p.stop == p.piece0 + tiles;
}

// The next piece; false at the end of the run.
template <int TILE>
__device__ __forceinline__ bool next_piece(const PagedDecodeArgs& a, int64_t end, Piece& p) {
  if (p.stop >= end) return false;
  p.at = p.piece0 = p.stop;
  if (++p.g == a.hkv) {
    p.g = 0;
    do {
      p.len = checked_len(a, ++p.b);
    } while (p.len <= 0);
  }
  set_piece<TILE>(a, end, p);
  return true;
}

// The outputs of heads h0 .. h1 of a sequence of n tokens: none, or fewer (a length out of range).
__device__ __forceinline__ void write_empty(const PagedDecodeArgs& a, int b, int n, int h0, int h1,
                                            int D, int thread, int threads) {
  const float nan = __int_as_float(0x7FFFFFFF);
  if (n < 0 && thread == 0) atomicOr(a.err_word, kErrDeviceBounds);
  const int64_t row = static_cast<int64_t>(b) * a.hq;
  for (int i = h0 * D + thread; i < h1 * D; i += threads)
    a.out[row * D + i] = __float2bfloat16(n < 0 ? nan : 0.f);
  if (a.lse != nullptr)
    for (int i = h0 + thread; i < h1; i += threads) a.lse[row + i] = n < 0 ? nan : -INFINITY;
}
__device__ __forceinline__ void write_empty(const PagedDecodeArgs& a, int b, int n, int h0, int h1,
                                            int D) {
  write_empty(a, b, n, h0, h1, D, threadIdx.x, kDecThreads);
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// How the tiles are dealt out.
enum DecMode {
  kSplit,  // runs of CTA tiles, a run per CTA
  kOne,    // one launch: a cluster per (sequence, head)
  kWarps,  // runs of a warp's steps, a run per warp: no warp waits for another
  kPairs   // one launch: a warp per (sequence, head), and on to the next
};

// Joins the partials of every (sequence, head) that more than one CTA worked on. Its CTAs
// are c0 (where it begins, with its record) .. c1; their blocks here share its query heads:
// block c0 + k takes heads k, k + (c1 - c0 + 1), ... A block so has at most two such jobs
// (the piece that begins in its CTA, and the one that began before); each of their heads is
// a task for one warp, or for several where there are fewer tasks than warps. What counts is
// latency: records of the candidates in one load, eight partials per warp in flight.
constexpr int kJoinWarps = 8;
constexpr int kFinishThreads = 32 * kJoinWarps;
template <int D>
__device__ __forceinline__ void join_parts(const PagedDecodeArgs& a, int ctas, float l_shift) {
  constexpr int V = D / 32;  // values of a lane
  __shared__ alignas(16) float s_acc[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int G = a.group, block = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  DecodeRec rec{-1, 0, 0, 0};
  if (lane < G && lane <= block) rec = a.rec[block - lane];
  const unsigned begun = __ballot_sync(0xFFFFFFFFu, rec.seq >= 0);
  // job 0: begins here; job 1: the nearest before that reaches this block
  int from[2], job_seq[2], job_head[2], last[2], step[2], first[2], tasks[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const unsigned mask = j == 0 ? begun & 1u : begun & ~1u;
    const int back = mask ? __ffs(mask) - 1 : 0;
    job_seq[j] = __shfl_sync(0xFFFFFFFFu, rec.seq, back);
    job_head[j] = __shfl_sync(0xFFFFFFFFu, rec.head, back);
    last[j] = __shfl_sync(0xFFFFFFFFu, rec.last, back);
    from[j] = block - back;
    first[j] = back;
    step[j] = last[j] - from[j] + 1;
    tasks[j] = mask && block <= last[j] && back < G ? (G - back + step[j] - 1) / step[j] : 0;
  }
  const int sparse = __shfl_sync(0xFFFFFFFFu, rec.sparse, begun ? __ffs(begun) - 1 : 0);
  const int total = tasks[0] + tasks[1];
  int wpt = 1;  // warps of a task
  while (wpt < kJoinWarps && 2 * wpt * total <= kJoinWarps) wpt *= 2;
  const int sub = warp % wpt;
  for (int t0 = 0; t0 < total; t0 += kJoinWarps / wpt) {
    const int task = t0 + warp / wpt;
    const int j = task < tasks[0] ? 0 : 1;
    const bool active = task < total;
    const int c0 = j ? from[1] : from[0], c1 = j ? last[1] : last[0];
    const int h = j ? first[1] + (task - tasks[0]) * step[1] : first[0] + task * step[0];
    float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int base = c0 + sub; active && base <= c1; base += 8 * wpt) {
      float2 ml[8];
      float x[8][V];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = base + u * wpt;
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) x[u][v] = 0.f;
        // with fewer tiles than CTAs some have none
        if (c <= c1 && (sparse == 0 || first_tile(c, sparse, ctas) != first_tile(c + 1, sparse, ctas))) {
          const int64_t part = (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * G + h;
          ml[u] = a.part_ml[part];
          const float* p = a.part_o + part * D + V * lane;
          if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4*>(p);
            x[u][0] = y.x;
            x[u][1] = y.y;
            x[u][2] = y.z;
            x[u][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(p);
            x[u][0] = y.x;
            x[u][1] = y.y;
          }
        }
      }
      float to = top;
#pragma unroll
      for (int u = 0; u < 8; ++u) to = fmaxf(to, ml[u].x);
      const float f = top == -INFINITY ? 0.f : ex2(top - to);
      sum *= f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // a bad page's sum is NaN and stays it
        const float e = ml[u].x == -INFINITY ? 0.f : ex2(ml[u].x - to);
        sum = fmaf(ml[u].y, e, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(x[u][v], e, acc[v]);
      }
      top = to;
    }
    if (wpt > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) s_acc[warp][V * lane + v] = acc[v];
      if (lane == 0) s_ml[warp] = make_float2(top, sum);
      __syncthreads();
      if (sub == 0) {
        float to = top;
        for (int w = 1; w < wpt; ++w) to = fmaxf(to, s_ml[warp + w].x);
        const float f = top == -INFINITY ? 0.f : ex2(top - to);
        sum *= f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= f;
        for (int w = 1; w < wpt; ++w) {
          const float2 ml = s_ml[warp + w];
          const float e = ml.x == -INFINITY ? 0.f : ex2(ml.x - to);
          sum = fmaf(ml.y, e, sum);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(s_acc[warp + w][V * lane + v], e, acc[v]);
        }
        top = to;
      }
    }
    if (active && sub == 0) {
      const int seq = j ? job_seq[1] : job_seq[0], head = j ? job_head[1] : job_head[0];
      const int64_t row = static_cast<int64_t>(seq) * a.hq + head * G + h;
      const float vs = a.v_scale != nullptr
                           ? a.v_scale[static_cast<int64_t>(seq) * a.hkv + head] : 1.f;
      uint32_t packed[V / 2];
#pragma unroll
      for (int v = 0; v < V; v += 2)
        packed[v / 2] = pack2<false>(acc[v] / sum * vs, acc[v + 1] / sum * vs);
      uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * D + V * lane);
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[1]);
      else
        out[0] = packed[0];
      if (lane == 0) {
        const float lse2 = top + (log2f(sum) - l_shift);
        if (a.lse != nullptr) a.lse[row] = lse2 * 0.6931471805599453f;
      }
    }
  }
}

// score_out[b, g, j] = score_in + sum over the group's heads of exp2(x - lse2) for 1,024 keys,
// from the scores that the attention left in the workspace (4 bytes per (head, token)
// against 4 d or 2 d bytes of K and V per G of them, and mostly still in L2). lse2 is the
// attention's own, or formed here from the (max, sum) of its parts.
constexpr int kWeightPer = 4;
constexpr int kWeightKeys = kFinishThreads * kWeightPer;
__device__ __forceinline__ void add_weights(const PagedDecodeArgs& a, int ctas, float l_shift,
                                            int pair, int chunk, int chunks) {
  __shared__ float s_lse2[16];
  const int b = pair / a.hkv;
  const int n = checked_len(a, b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(pair) * a.group;  // = b * Hq + g * G
  const int64_t out_row = static_cast<int64_t>(pair) * a.score_stride;
  const int64_t first = static_cast<int64_t>(chunk) * kWeightKeys;
  if (first >= n) {
    after_stream();
    return;
  }
  // the inputs of the call, which the attention does not write, and what does not depend on lse2 first
  float base[kWeightPer];
#pragma unroll
  for (int k = 0; k < kWeightPer; ++k) {
    const int64_t j = first + k * kFinishThreads + threadIdx.x;
    base[k] = a.score_in != nullptr && j < n ? a.score_in[out_row + j] : 0.f;
  }
  after_stream();
  let_next_start();  // (here it gives 0.5 us of 52: 32 sequences of 2,048-8,192 tokens in 4-bit pages)
  // the first heads' scores are on their way while lse2 is worked out
  float x[4][kWeightPer];
  auto load_raw = [&](int h0, int64_t j0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* raw = a.raw + (row + h0 + u) * a.raw_stride;
#pragma unroll
      for (int k = 0; k < kWeightPer; ++k) {
        const int64_t j = j0 + k * kFinishThreads + threadIdx.x;
        x[u][k] = h0 + u < a.group && j < n ? raw[j] : -INFINITY;
      }
    }
  };
  load_raw(0, first);
  const int c0 = a.begun[pair];
  if (c0 < 0) {
    if (threadIdx.x < a.group) s_lse2[threadIdx.x] = a.lse2[row + threadIdx.x];
  } else {
    const DecodeRec rec = a.rec[c0];
    for (int h = warp; h < a.group; h += kJoinWarps) {
      float top = -INFINITY, sum = 0.f;
      for (int c = c0 + lane; c <= rec.last; c += 32) {
        if (rec.sparse != 0 &&
            first_tile(c, rec.sparse, ctas) == first_tile(c + 1, rec.sparse, ctas))
          continue;
        const float2 ml = a.part_ml[(2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * a.group + h];
        const float to = fmaxf(top, ml.x);
        sum = sum * (top == -INFINITY ? 0.f : ex2(top - to)) +
              ml.y * (ml.x == -INFINITY ? 0.f : ex2(ml.x - to));
        top = to;
      }
      float all = top;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) all = fmaxf(all, __shfl_xor_sync(0xFFFFFFFFu, all, off));
      sum *= top == -INFINITY ? 0.f : ex2(top - all);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
      if (lane == 0) s_lse2[h] = all + (log2f(sum) - l_shift);
    }
  }
  __syncthreads();
  for (int64_t j0 = first; j0 < n; j0 += static_cast<int64_t>(chunks) * kWeightKeys) {
    float add[kWeightPer] = {0.f, 0.f, 0.f, 0.f};
    if (j0 != first) {
#pragma unroll
      for (int k = 0; k < kWeightPer; ++k) {
        const int64_t j = j0 + k * kFinishThreads + threadIdx.x;
        base[k] = a.score_in != nullptr && j < n ? a.score_in[out_row + j] : 0.f;
      }
    }
    for (int h0 = 0; h0 < a.group; h0 += 4) {
      if (h0 > 0 || j0 != first) load_raw(h0, j0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float lse2 = h0 + u < a.group ? s_lse2[h0 + u] : -INFINITY;
#pragma unroll
        for (int k = 0; k < kWeightPer; ++k)  // a head whose lse is -inf or NaN adds nothing
          add[k] += lse2 > -INFINITY ? ex2(x[u][k] - lse2) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < kWeightPer; ++k) {
      const int64_t j = j0 + k * kFinishThreads + threadIdx.x;
      if (j < n) a.score_out[out_row + j] = base[k] + add[k];
    }
  }
}

// What follows the attention: blocks 0 .. ctas - 1 join, the others form the weights.
template <int D>
__global__ void __launch_bounds__(kFinishThreads, 4)
    paged_finish_kernel(const PagedDecodeArgs a, int ctas, float l_shift, int chunks) {
  if (static_cast<int>(blockIdx.x) < ctas) {
    // (without let_next_start: with it the next attention's CTAs came 2 us later, 46.1 us for 64
    // sequences of 128-4,096 tokens in 4-bit pages instead of 43.9)
    after_stream();
    join_parts<D>(a, ctas, l_shift);
  } else {
    const int i = static_cast<int>(blockIdx.x) - ctas;
    add_weights(a, ctas, l_shift, i / chunks, i % chunks, chunks);
  }
}

// A kernel and how it is launched: K has the sizes that DecCfg has, the pages' form (kForm), the CTAs
// per SM (kPerSm), the power of two by which its sums are scaled (kShift), tiles per CTA in one launch
// of clusters (kOneTiles), the steps up to which a warp takes a (sequence, head) alone (kPairSteps; < 0:
// it has no such instance), the threads of a CTA with a run (kSplitThreads) and fn(mode), its instances.

// One launch where clusters of up to eight CTAs, a few tiles each at most, all fit the GPU
// at once: there a launch less is worth more than an even division (measured beside kOneTiles).
template <class K>
int one_cluster(const PagedDecodeArgs& a) {
  const int tiles = (a.max_len + K::kTile - 1) / K::kTile;
  int cluster = 1;
  while (cluster < kOneCluster && cluster < tiles) cluster *= 2;
  return cluster;
}
template <class K>
bool decode_in_one(const PagedDecodeArgs& a, int num_sms) {
  const int tiles = (a.max_len + K::kTile - 1) / K::kTile, cluster = one_cluster<K>(a);
  return tiles <= K::kOneTiles * cluster &&
         static_cast<int64_t>(a.num_seqs) * a.hkv * cluster <= K::kPerSm * num_sms;
}
// A warp per (sequence, head).
template <class K>
cudaError_t launch_pairs(const PagedDecodeArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(K::fn(kPairs)), K::kRing, ready);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * (a.hkv << a.split);
  const int64_t all = (pairs + kDecWarps - 1) / kDecWarps, fit = static_cast<int64_t>(K::kPerSm) * num_sms;
  return launch_early(K::fn(kPairs), dim3(static_cast<unsigned>(all < fit ? all : fit)), dim3(kDecThreads),
                      K::kRing, stream, 0, a, 1);
}

template <class K>
cudaError_t launch_decode(PagedDecodeArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e;
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  const int cluster = one_cluster<K>(a);
  if (decode_in_one<K>(a, num_sms)) {
    static std::atomic<uint64_t> one_ready{0};
    e = allow_smem(reinterpret_cast<const void*>(K::fn(kOne)), K::kSmem, one_ready);
    if (e != cudaSuccess) return e;
    return launch_early(K::fn(kOne), dim3(static_cast<unsigned>(pairs * cluster)), dim3(kDecThreads),
                        K::kSmem, stream, cluster, a, cluster);
  }
  if constexpr (K::kPairSteps > 0) {
    if (a.max_len <= K::kPairSteps * K::kKeys) return launch_pairs<K>(a, num_sms, stream);
  }
  // runs of warps or of CTAs
  const bool warps = decode_by_warps(K::kForm, a.group, a.num_seqs, a.hkv, a.max_len, K::kTile);
  const int tile = warps ? K::kKeys : K::kTile;
  const int ctas = decode_ctas(num_sms, K::kPerSm, a.num_seqs, a.hkv, a.max_len, K::kTile);
  const int runs = warps ? ctas * kDecWarps : ctas;
  static std::atomic<uint64_t> ready[2] = {};
  const int smem = warps ? K::kRing : K::kSmem;
  const auto fn = K::fn(warps ? kWarps : kSplit);
  e = allow_smem(reinterpret_cast<const void*>(fn), smem, ready[warps]);
  if (e != cudaSuccess) return e;
  e = launch_early(fn, dim3(ctas), dim3(warps ? kDecThreads : K::kSplitThreads), smem, stream, 0, a, 1);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // left out where no (sequence, head) can have more than one tile and no weights are wanted
  if (e == cudaSuccess && (a.max_len > tile || (a.raw != nullptr && a.max_len > 0))) {
    int64_t blocks = runs;
    int chunks = 1;
    if (a.raw != nullptr) {
      const int most = (a.max_len + kWeightKeys - 1) / kWeightKeys;
      // Blocks of 1,024 keys as long as there are not many thousands of them (the lengths may
      // be far below max_seq_len); beyond that a block takes several chunks.
      const int64_t room = 8192 / pairs;
      chunks = static_cast<int>(most < room ? most : room < 1 ? 1 : room);
      blocks += pairs * chunks;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kFinishThreads);
    e = cudaLaunchKernelEx(&cfg, paged_finish_kernel<K::kDim>, a, runs, K::kShift, chunks);
  }
  return e;
}

}  // namespace

}  // namespace quail

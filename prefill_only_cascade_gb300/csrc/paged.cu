// paged.cu - a paged key/value cache: rows written into pages, and attention of one new
// token per sequence over them. "Motor de inferência Quail atinge 1 bilhão de tokens por
// minuto por GPU", section "Como funciona", keeps anchor KV between prefills; pages let it
// be kept, grown and cut token by token. A page is [page_size, Hkv, d], the token-row
// layout of every K/V tensor of the library, so a contiguous [T, Hkv, d] tensor is itself
// a pool whose pages follow one another.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

// ------------------------------------------------------------------ append
// One block takes `tok` consecutive new tokens: its first threads find each token's
// sequence and slot, then all threads move 16-byte source vectors (8 values), K and V of
// one token row after the other. Bound by HBM (2 bytes read, 2 or 1 written per value).
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTok = 64;

// Eight bf16 -> eight E4M3 codes of RN32(x / s), rounded to nearest even, saturating at
// +-448. r = RN(1/s). For an ordinary scale the quotient is RN(x r) with one FMA correction
// by its exact residual (Markstein, "IA-64 and Elementary Functions", 2000), which is the
// IEEE quotient wherever a code can be other than zero: |x| >= 2^-10 |s| keeps the residual
// out of the subnormals for s in [2^-60, 2^60]. An infinite quotient (x infinite, or x / s
// past fp32) has no residual and is used as it is. Other scales divide.
__device__ __forceinline__ uint2 encode_bf16x8(const uint4& raw, float s, float r, bool plain) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t packed[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x[2] = {__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (plain) {
        const float q = x[j] * r;
        const float c = fmaf(fmaf(-q, s, x[j]), r, q);
        // x's sign restores -0 / s, which the correction rounds to +0
        x[j] = fabsf(q) < 1e30f ? copysignf(c, x[j]) : q;
      } else {
        x[j] = __fdiv_rn(x[j], s);
      }
    }
    const __nv_fp8x2_storage_t c =
        __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    packed[k >> 1] |= static_cast<uint32_t>(c) << (16 * (k & 1));
  }
  return make_uint2(packed[0], packed[1]);
}

template <bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppendArgs a,
                                                                      int tok) {
  __shared__ int64_t s_slot[kAppendMaxTok];
  __shared__ int s_seq[kAppendMaxTok];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int n = static_cast<int>(min(static_cast<int64_t>(tok), a.total_new - t0));
  if (threadIdx.x < n) {
    const int64_t t = t0 + threadIdx.x;
    int b = static_cast<int>(t);
    int64_t i = 0;
    bool ok = true;
    if (a.new_offsets != nullptr) {
      int lo = 0, hi = a.num_seqs;  // the last sequence that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.new_offsets + mid) <= t) lo = mid; else hi = mid;
      }
      b = lo;
      const int64_t o0 = __ldg(a.new_offsets + b);
      i = t - o0;
      ok = o0 <= t && t < __ldg(a.new_offsets + b + 1);
    }
    int64_t slot = -1;
    if (ok) {
      const int64_t start = __ldg(a.start_pos + b);
      const int64_t pos = start + i;
      if (start >= 0 && pos < a.max_len) {
        const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages +
                               (pos >> a.page_shift));
        if (page >= 0 && page < a.num_pages)
          slot = (static_cast<int64_t>(page) << a.page_shift) +
                 (pos & ((1 << a.page_shift) - 1));
      }
    }
    if (slot < 0) atomicOr(a.err_word, kErrDeviceBounds);
    s_slot[threadIdx.x] = slot;
    s_seq[threadIdx.x] = b;
  }
  // the offsets as a whole: increasing from 0 to the number of new rows
  if (blockIdx.x == 0 && a.new_offsets != nullptr) {
    for (int b = threadIdx.x; b <= a.num_seqs; b += kAppendThreads) {
      const int64_t o = __ldg(a.new_offsets + b);
      const int64_t next = b < a.num_seqs ? __ldg(a.new_offsets + b + 1) : a.total_new;
      if ((b == 0 && o != 0) || (b < a.num_seqs ? next < o : next != o))
        atomicOr(a.err_word, kErrDeviceBounds);
    }
  }
  __syncthreads();
  const int vecs = a.row_elems / 8;  // 16-byte source vectors of a token row
  const int total = n * 2 * vecs;
  for (int u = threadIdx.x; u < total; u += kAppendThreads) {
    const int row = u / vecs, c = u - row * vecs;
    const int t = row >> 1, is_v = row & 1;
    const int64_t slot = s_slot[t];
    if (slot < 0) continue;
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(
        (is_v ? a.v_new : a.k_new) + (t0 + t) * (is_v ? a.v_stride : a.k_stride) + 8 * c));
    if (FP8) {
      const int g = (8 * c) / a.head_dim;
      const float s = __ldg((is_v ? a.v_scale : a.k_scale) +
                            static_cast<int64_t>(s_seq[t]) * a.hkv + g);
      const bool plain = s >= 8.673617379884035e-19f && s <= 1.152921504606847e18f;  // 2^-60, 2^60
      *reinterpret_cast<uint2*>((is_v ? a.v_pages : a.k_pages) + slot * a.row_elems + 8 * c) =
          encode_bf16x8(x, s, __frcp_rn(s), plain);
    } else {
      *reinterpret_cast<uint4*>((is_v ? a.v_pages : a.k_pages) + 2 * (slot * a.row_elems + 8 * c)) =
          x;
    }
  }
}

// ------------------------------------------------------------------ decode attention
// o[b, h] = sum_j w_j v_j with w_j = exp(c q.k_j - lse) over the j < len[b] cached tokens;
// every K and V byte is read once for the G query heads that share it, so HBM bounds it.
//
// The tiles (kTile keys of one sequence and KV head) of the whole batch are numbered in
// the order sequence, head, position, and each CTA takes an equal run of them, whatever
// the lengths are: short sequences share a CTA, long ones spread over many. A sequence's
// head that lies inside one CTA is finished there; the others leave (max, sum, O) partials
// that paged_finish_kernel rescales and adds. Small calls (ONE) do all of it in one launch:
// a thread-block cluster per (sequence, head) divides its tiles, joins through distributed
// shared memory and forms the weights.
//
// Each warp walks its own keys of its CTA's run with a running max and sum. Their K and V
// rows come through a ring of its own in shared memory, filled by 16-byte asynchronous
// copies two steps (16 KB a warp, 128 KB an SM) ahead, also over the borders between
// sequences and heads, so the loads never wait for the arithmetic. No warp waits for
// another but where the parts of a (sequence, head) are put together. Where there are many and
// none can be long, the runs are dealt to the warps themselves (kWarps), and none waits at all.
//
// Both products run on mma.sync m16n8k16: one new token gives at most 16 query rows per KV
// head, so the padded products do not bound it but with 16 heads over e4m3 pages (see below).
// Since sums over d (scores) and the order of d (output rows) may be permuted freely,
// 16-byte pieces of plain rows ARE the operand fragments:
//   S  [16 heads x 8 keys]  A = Q (rows: heads), B = K: lane (r, q) holds key r, piece q + 4i
//   O^T [16 d x 8 heads]    A = V^T: lane (r, q) holds keys 2q, 2q+1, 2q+8, 2q+9, piece r
//                           (two keys' values interleaved by byte permutes), B = P, whose
//                           fragment is the score fragment packed in place
// bf16 pages: bf16 products, P as the sum of three bf16 (all 24 bits of P). e4m3 pages: f16
// products (codes are exact in f16), P as the sum of two f16 (22 bits, scaled by 2^14 so that
// weights down to 2^-38 of the largest count), Q scaled per head by a power of two into f16's
// range: q bits below 2^-38 of the head's largest |q| are lost, under fp32's own rounding.
// Against fewer terms of P (two bf16, 16 bits; one f16, 11 bits), whose errors showed in the last
// bit of one output in a few hundred: 64 sequences of 128-4,096 tokens (G = 4, bf16) 90.4 -> 90.8 us,
// one of 131,007 86.7 -> 87.2, of 777 5.9 -> 6.1, 32 of 2,048-8,192 (e4m3) 69.1 -> 69.7; the tensor
// pipe shows with 16 heads per KV head only: 117 -> 120.5 (bf16), 77.6 -> 87 (e4m3).
constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;

constexpr int kOneCluster = 8;                       // CTAs that share a small call's head
constexpr int kStages = 3;                           // steps in a warp's ring
constexpr int kStepBytes = 4096;                     // of K, and of V, in one step

template <int D, bool FP8>
struct DecCfg {
  static constexpr int kRB = D * (FP8 ? 1 : 2);      // bytes of a (token, head) row
  static constexpr int kNC = kRB / 16;               // its 16-byte pieces
  static constexpr int kKeys = kStepBytes / kRB;     // keys per warp step: 16, 32 or 64
  static constexpr int kKG = kKeys / 8;              // in groups of 8 (score tiles)
  static constexpr int kKChunks = kRB / 64;          // K pieces per lane and key
  static constexpr int kSteps16 = kKeys / 16;        // in 16s (products with V)
  static constexpr int kTile = kDecWarps * kKeys;    // keys per CTA tile
  static constexpr int kMT = D / 16;                 // 16-row tiles of O^T
  static constexpr int kQS = D / 16;                 // k-steps of the score product
  static constexpr int kTerms = FP8 ? 2 : 3;         // P as a sum of so many 16-bit values
  static constexpr int kRing = kDecWarps * kStages * 2 * kStepBytes;
  static constexpr int kSmem = kRing + kDecWarps * 8 * D * 4;  // + the warps' O, 8 heads
};

// Places of piece c of row `row` in a step's K and V buffers (in 16-byte units). A warp's
// 16-byte reads go in phases of 8 lanes: two K rows x 4 pieces, or four V row pairs x 2
// pieces; the exclusive-ors spread each phase over all banks.
template <int NC>
__device__ __forceinline__ int k_place(int row, int c) {
  return NC >= 8 ? (row * NC + c) ^ ((row & 1) << 2) : row * NC + c;
}
template <int NC>
__device__ __forceinline__ int v_place(int row, int c) {
  return (row * NC + c) ^ (((row >> 1) & 3) << 1);
}

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
// Two e4m3 codes (the low or the high half of w) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(h)
      : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(h)
      : "r"(w));
  return h;
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

// The d of lane row r's first output row in tile t (its second is the next d).
template <int D, bool FP8>
__device__ __forceinline__ int out_d(int r, int t) {
  if (D == 128 && !FP8) return (r + 8 * (t >> 2)) * 8 + 2 * (t & 3);
  if (D == 128) return r * 16 + 2 * t;
  return r * 8 + 2 * t;
}

// First tile of CTA c when `total` tiles are dealt to n CTAs.
__device__ __forceinline__ int64_t first_tile(int c, int64_t total, int n) {
  return static_cast<int64_t>(c) * total / n;
}

// The length of sequence b if it is one the call allows, else -1.
__device__ __forceinline__ int checked_len(const PagedDecodeArgs& a, int b) {
  const int n = __ldg(a.lens + b);
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

__device__ __forceinline__ void write_empty(const PagedDecodeArgs& a, int b, int n, int h0, int h1,
                                            int D) {
  const float nan = __int_as_float(0x7FFFFFFF);
  if (n < 0 && threadIdx.x == 0) atomicOr(a.err_word, kErrDeviceBounds);
  const int64_t row = static_cast<int64_t>(b) * a.hq;
  for (int i = h0 * D + threadIdx.x; i < h1 * D; i += kDecThreads)
    a.out[row * D + i] = __float2bfloat16(n < 0 ? nan : 0.f);
  if (a.lse != nullptr)
    for (int i = h0 + threadIdx.x; i < h1; i += kDecThreads) a.lse[row + i] = n < 0 ? nan : -INFINITY;
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
  kWarps   // runs of a warp's steps, a run per warp: no warp waits for another
};

template <int D, bool FP8, int NT, DecMode MODE>
__global__ void __launch_bounds__(kDecThreads, 2)
    paged_decode_kernel(const PagedDecodeArgs a, int cluster) {
  using C = DecCfg<D, FP8>;
  constexpr bool ONE = MODE == kOne, WARPS = MODE == kWarps;
  constexpr int kTile = WARPS ? C::kKeys : C::kTile;  // keys that a run is counted in
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float s_m[kDecWarps][8 * NT], s_l[kDecWarps][8 * NT];
  __shared__ int s_bad[kDecWarps];
  float(*s_o)[8][D] = reinterpret_cast<float(*)[8][D]>(dyn + C::kRing);  // [warp][head][d]
  float* s_part = reinterpret_cast<float*>(dyn);  // ONE, at the end: [head][d]
  __shared__ float2 s_pml[ONE ? 8 * NT : 1];
  __shared__ float s_lse2[ONE ? 8 * NT : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, q4 = lane & 3;
  const int G = a.group;
  // who takes a run (a CTA, a warp), or ONE: the rank
  const int cta = ONE ? static_cast<int>(blockIdx.x) % cluster
                      : WARPS ? static_cast<int>(blockIdx.x) * kDecWarps + warp : blockIdx.x;
  const int ctas = WARPS ? static_cast<int>(gridDim.x) * kDecWarps : gridDim.x;
  Piece cur;
  int64_t run_end, run_total = 0;
  if constexpr (ONE) {
    const int pair = static_cast<int>(blockIdx.x) / cluster;
    cur.b = pair / a.hkv;
    cur.g = pair % a.hkv;
    cur.len = checked_len(a, cur.b);
    if (cur.len <= 0) {  // the same for every CTA of the cluster
      if (cta == 0) write_empty(a, cur.b, cur.len, cur.g * G, (cur.g + 1) * G, D);
      return;
    }
    const int tiles = (cur.len + C::kTile - 1) / C::kTile;
    cur.piece0 = 0;
    cur.at = first_tile(cta, tiles, cluster);
    run_end = first_tile(cta + 1, tiles, cluster);
  } else {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // sequences without tokens (0 and -inf) and with lengths out of range (NaN)
    for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
      const int n = checked_len(a, b);
      if (n <= 0) write_empty(a, b, n, 0, a.hq, D);
    }
    const RunStart run = find_run(a, kTile, cta, ctas);
    if (WARPS ? lane == 0 : threadIdx.x == 0) a.rec[cta] = DecodeRec{-1, 0, 0, 0};
    if (run.begin >= run.end) return;
    cur.b = run.seq;
    cur.len = checked_len(a, cur.b);
    const int tiles = (cur.len + kTile - 1) / kTile;
    cur.g = static_cast<int>((run.begin - run.seq_tile0) / tiles);
    cur.piece0 = run.seq_tile0 + static_cast<int64_t>(cur.g) * tiles;
    cur.at = run.begin;
    run_end = run.end;
    run_total = run.total;
  }
  set_piece<kTile>(a, run_end, cur);

  // ------------------------------------------------------ loads: a cursor of their own
  const int64_t row_stride = static_cast<int64_t>(a.hkv) * C::kRB;
  const uint32_t ring = smem_u32(dyn) + warp * (kStages * 2 * kStepBytes);
  Piece ld = cur;
  const int own = WARPS ? 0 : warp * C::kKeys;  // the warp's first key in a tile
  int ld_key = ld.kb + own;              // first key of the next step to load
  bool ld_more = true;
  int page[C::kSteps16];                 // pages of its 16-key blocks
  uint32_t bad_steps = 0;                // bit s: a page of the step in stage s is no page
  auto seek = [&]() {                    // on to a piece that has a step for this warp
    while (ld_more && ld_key >= ld.ke) {
      ld_more = next_piece<kTile>(a, run_end, ld);
      ld_key = ld.kb + own;
    }
    if (ld_more) {
      const int32_t* table = a.table + static_cast<int64_t>(ld.b) * a.max_pages;
#pragma unroll
      for (int i = 0; i < C::kSteps16; ++i)
        page[i] = ld_key + 16 * i < ld.ke ? __ldg(table + ((ld_key + 16 * i) >> a.page_shift)) : 0;
    }
  };
  auto issue = [&](int stage) {
    if (ld_more) {
      const uint32_t kdst = ring + stage * 2 * kStepBytes, vdst = kdst + kStepBytes;
      bool bad = false;
      // lane + 32 j is the j-th piece of this lane: C::kNC pieces a row
      const int row0 = lane / C::kNC, c = lane % C::kNC;
      constexpr int kRows = 32 / C::kNC;  // rows per round of the warp
      int64_t base[C::kSteps16];
#pragma unroll
      for (int i = 0; i < C::kSteps16; ++i) {
        const int pos = ld_key + 16 * i;
        const bool ok = page[i] >= 0 && page[i] < a.num_pages;
        if (pos < ld.ke && !ok) bad = true;
        base[i] = pos < ld.ke && ok
                      ? ((static_cast<int64_t>(page[i]) << a.page_shift) +
                         (pos & ((1 << a.page_shift) - 1))) * row_stride +
                            static_cast<int64_t>(ld.g) * C::kRB + 16 * c
                      : -1;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = row0 + j * kRows;
        const int64_t at = base[(j * kRows) >> 4];
        const bool real = at >= 0 && ld_key + row < ld.ke;
        const int64_t off = real ? at + (row & 15) * row_stride : 0;
        copy16(kdst + 16 * k_place<C::kNC>(row, c), a.k_pages + off, real);
        copy16(vdst + 16 * v_place<C::kNC>(row, c), a.v_pages + off, real);
      }
      bad_steps = bad ? bad_steps | (1u << stage) : bad_steps & ~(1u << stage);
      ld_key += kTile;
      seek();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // Q of a piece as it is in memory: 4 values of d per k-step; heads past the group: zeros
  uint2 qraw[NT][C::kQS];
  constexpr int EC = FP8 ? 16 : 8;  // values per K piece
  auto load_q = [&](int b, int g) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = r + 8 * n;
      const __nv_bfloat16* qp =
          a.q + static_cast<int64_t>(b) * a.q_stride + static_cast<int64_t>(g * G + h) * D;
#pragma unroll
      for (int ks = 0; ks < C::kQS; ++ks) {
        const int off = (q4 + 4 * (ks / (EC / 4))) * EC + 4 * (ks % (EC / 4));
        qraw[n][ks] = h < G ? __ldg(reinterpret_cast<const uint2*>(qp + off)) : make_uint2(0u, 0u);
      }
    }
  };

  seek();
  load_q(cur.b, cur.g);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  int stage = 0;

  while (true) {
    // ---------------------------------------------------- one piece
    uint32_t qa[C::kQS][2 * NT];
    float c_log2[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      c_log2[n] = a.scale_log2;
      if (FP8) {
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < C::kQS; ++ks)
          top = absmax_bf16x2(absmax_bf16x2(top, qraw[n][ks].x), qraw[n][ks].y);
        float mx = absmax_bf16x2_value(top);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        // 2^e with mx 2^e in [2^14, 2^15); zero, infinite and NaN rows are left as they are
        int e = mx > 0.f && mx < INFINITY ? 14 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127) : 0;
        e = min(e, 126);  // a power of two that is a normal float, as is its inverse
        const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        c_log2[n] *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        c_log2[n] *= __ldg(a.k_scale + static_cast<int64_t>(cur.b) * a.hkv + cur.g);
#pragma unroll
        for (int ks = 0; ks < C::kQS; ++ks) {
          const uint2 w = qraw[n][ks];
          qa[ks][2 * n] = pack2<true>(__uint_as_float(w.x << 16) * up,
                                      __uint_as_float(w.x & 0xFFFF0000u) * up);
          qa[ks][2 * n + 1] = pack2<true>(__uint_as_float(w.y << 16) * up,
                                          __uint_as_float(w.y & 0xFFFF0000u) * up);
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < C::kQS; ++ks) {
          qa[ks][2 * n] = qraw[n][ks].x;
          qa[ks][2 * n + 1] = qraw[n][ks].y;
        }
      }
    }

    float o[NT][C::kMT][4];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.f;
#pragma unroll
      for (int t = 0; t < C::kMT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][t][j] = 0.f;
    }
    bool bad = false;

    for (int key0 = cur.kb + own; key0 < cur.ke; key0 += kTile) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // every lane's copies are there, and the stage before was read
      bad |= (bad_steps >> stage) & 1u;
      issue(stage == 0 ? kStages - 1 : stage - 1);
      const uint32_t kbuf = ring + stage * 2 * kStepBytes, vbuf = kbuf + kStepBytes;
      stage = stage == kStages - 1 ? 0 : stage + 1;

      // ---- scores of this step's keys
      float s[C::kKG][4];
#pragma unroll
      for (int kg = 0; kg < C::kKG; ++kg) {
        s[kg][0] = s[kg][1] = s[kg][2] = s[kg][3] = 0.f;
#pragma unroll
        for (int i = 0; i < C::kKChunks; ++i) {
          const uint4 v = ld_shared16(kbuf + 16 * k_place<C::kNC>(8 * kg + r, q4 + 4 * i));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if (FP8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int ks = 4 * i + j;
              mma16816<true>(s[kg], qa[ks][0], NT == 2 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                             NT == 2 ? qa[ks][2 * NT - 1] : 0u, e4m3_lo(w[j]), e4m3_hi(w[j]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int ks = 2 * i + j;
              mma16816<false>(s[kg], qa[ks][0], NT == 2 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                              NT == 2 ? qa[ks][2 * NT - 1] : 0u, w[2 * j], w[2 * j + 1]);
            }
          }
        }
      }

      // ---- running max and sum; x = score in log2 units
      float p[NT][C::kKG][2];
      float mx[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mx[n] = -INFINITY;
#pragma unroll
        for (int kg = 0; kg < C::kKG; ++kg)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool see = key0 + 8 * kg + 2 * q4 + j < cur.ke;
            const float x = see ? s[kg][2 * n + j] * c_log2[n] : -INFINITY;
            p[n][kg][j] = x;
            mx[n] = fmaxf(mx[n], x);
          }
        if (a.raw != nullptr && r + 8 * n < G) {
          float* row =
              a.raw + (static_cast<int64_t>(cur.b) * a.hq + cur.g * G + r + 8 * n) * a.raw_stride;
#pragma unroll
          for (int kg = 0; kg < C::kKG; ++kg)  // rows are padded to whole tiles
            *reinterpret_cast<float2*>(row + key0 + 8 * kg + 2 * q4) =
                make_float2(p[n][kg][0], p[n][kg][1]);
        }
        mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 1));
        mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 2));
      }
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) grew |= mx[n] > m[n];
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float to = fmaxf(m[n], mx[n]);
          const float f = m[n] == -INFINITY ? 0.f : ex2(m[n] - to);
          l[n] *= f;
          m[n] = to;
          const float f0 = __shfl_sync(0xFFFFFFFFu, f, 8 * q4);
          const float f1 = __shfl_sync(0xFFFFFFFFu, f, 8 * q4 + 4);
#pragma unroll
          for (int t = 0; t < C::kMT; ++t) {
            o[n][t][0] *= f0;
            o[n][t][1] *= f1;
            o[n][t][2] *= f0;
            o[n][t][3] *= f1;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // a row that has seen nothing but -inf takes 0 as its reference: its weights are 0
        const float ref = (m[n] == -INFINITY ? 0.f : m[n]) - (FP8 ? 14.f : 0.f);
#pragma unroll
        for (int kg = 0; kg < C::kKG; ++kg)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[n][kg][j] = ex2(p[n][kg][j] - ref);
            l[n] += p[n][kg][j];
          }
      }

      // ---- O^T += V^T P^T
      constexpr int kTerms = C::kTerms;
#pragma unroll
      for (int i = 0; i < C::kSteps16; ++i) {
        uint32_t ps[NT][kTerms][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float* x = p[n][2 * i + h];
            if constexpr (FP8) {
              split_f16(x[0], x[1], ps[n][0][h], ps[n][1][h]);
            } else {
              split_bf16(x[0], x[1], ps[n][0][h], ps[n][1][h], ps[n][2][h]);
            }
          }
        constexpr int kParts = C::kNC == 16 ? 2 : 1;  // 16-byte (or one 8-byte) parts of a lane
        constexpr int kWords = C::kNC == 4 ? 2 : 4;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          uint32_t w[4][kWords];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 16 * i + 2 * q4 + (j & 1) + 8 * (j >> 1);
            if constexpr (C::kNC == 4) {
              const uint2 x =
                  ld_shared8(vbuf + 16 * v_place<C::kNC>(row, r >> 1) + 8 * (r & 1));
              w[j][0] = x.x;
              w[j][1] = x.y;
            } else {
              const uint4 x = ld_shared16(vbuf + 16 * v_place<C::kNC>(row, r + 8 * part));
              w[j][0] = x.x;
              w[j][1] = x.y;
              w[j][2] = x.z;
              w[j][3] = x.w;
            }
          }
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            if (FP8) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h == 0 ? 0x5140u : 0x7362u;
                const uint32_t x = __byte_perm(w[0][k], w[1][k], sel);
                const uint32_t y = __byte_perm(w[2][k], w[3][k], sel);
#pragma unroll
                for (int t = 0; t < kTerms; ++t)
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma16816<true>(o[n][2 * k + h], e4m3_lo(x), e4m3_hi(x), e4m3_lo(y), e4m3_hi(y),
                                   ps[n][t][0], ps[n][t][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(w[0][k], w[1][k], 0x5410);
              const uint32_t a1 = __byte_perm(w[0][k], w[1][k], 0x7632);
              const uint32_t a2 = __byte_perm(w[2][k], w[3][k], 0x5410);
              const uint32_t a3 = __byte_perm(w[2][k], w[3][k], 0x7632);
#pragma unroll
              for (int t = 0; t < kTerms; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma16816<false>(o[n][4 * part + k], a0, a1, a2, a3, ps[n][t][0], ps[n][t][1]);
            }
          }
        }
      }
    }

    // the next piece's queries are on their way while this one is put together
    Piece nxt = cur;
    const bool more = !ONE && next_piece<kTile>(a, run_end, nxt);
    if (more) load_q(nxt.b, nxt.g);

    // ---------------------------------------------------- the four warps' parts together
    const float vs = FP8 ? __ldg(a.v_scale + static_cast<int64_t>(cur.b) * a.hkv + cur.g) : 1.f;
    // slot 0: the run began inside this (b, g); slot 1: the run's last, begun here
    const int64_t part = 2 * static_cast<int64_t>(cta) + (cur.at == cur.piece0 ? 1 : 0);
    auto note = [&](bool any_bad) {      // by one thread, about (b, g)
      if (any_bad) atomicOr(a.err_word, kErrDeviceBounds);
      if (ONE || cur.at != cur.piece0) return;
      if (a.begun != nullptr)
        a.begun[static_cast<int64_t>(cur.b) * a.hkv + cur.g] = cur.whole ? -1 : cta;
      if (!cur.whole) {  // goes on in the next runs: the join's entry
        const int64_t end = cur.piece0 + (cur.len + kTile - 1) / kTile;
        // the last run of (b, g) is the one that holds tile end - 1
        a.rec[cta] = DecodeRec{cur.b, cur.g, static_cast<int>((end * ctas - 1) / run_total),
                               run_total < ctas ? static_cast<int>(run_total) : 0};
      }
    };
    if constexpr (WARPS) {
      if (lane == 0) note(bad);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 1);
        l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 2);
        if (bad) l[n] = __int_as_float(0x7FFFFFFF);
        const int64_t row = static_cast<int64_t>(cur.b) * a.hq + cur.g * G + 8 * n;
        if (q4 == 0 && r + 8 * n < G) {
          if (cur.whole) {
            const float lse2 = m[n] + (log2f(l[n]) - (FP8 ? 14.f : 0.f));
            if (a.lse != nullptr) a.lse[row + r] = lse2 * 0.6931471805599453f;
            if (a.lse2 != nullptr) a.lse2[row + r] = lse2;
          } else {
            a.part_ml[part * G + 8 * n + r] = make_float2(m[n], l[n]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the lane's output rows are heads 2 q4 and 2 q4 + 1
          const float sum = __shfl_sync(0xFFFFFFFFu, l[n], 8 * q4 + 4 * h);
          const int hh = 2 * q4 + h;
          if (8 * n + hh >= G) continue;
          const float inv = vs / sum;
#pragma unroll
          for (int t = 0; t < C::kMT; t += 4) {  // eight neighbouring d
            const int d = out_d<D, FP8>(r, t);
            if (cur.whole) {
              uint4 x;
              x.x = pack2<false>(o[n][t][h] * inv, o[n][t][h + 2] * inv);
              x.y = pack2<false>(o[n][t + 1][h] * inv, o[n][t + 1][h + 2] * inv);
              x.z = pack2<false>(o[n][t + 2][h] * inv, o[n][t + 2][h + 2] * inv);
              x.w = pack2<false>(o[n][t + 3][h] * inv, o[n][t + 3][h + 2] * inv);
              *reinterpret_cast<uint4*>(a.out + (row + hh) * D + d) = x;
            } else {
              float4* to = reinterpret_cast<float4*>(a.part_o + (part * G + 8 * n + hh) * D + d);
              to[0] = make_float4(o[n][t][h], o[n][t][h + 2], o[n][t + 1][h], o[n][t + 1][h + 2]);
              to[1] = make_float4(o[n][t + 2][h], o[n][t + 2][h + 2], o[n][t + 3][h],
                                  o[n][t + 3][h + 2]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < (WARPS ? 0 : NT); ++n) {
      l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 1);
      l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 2);
      if (q4 == 0) {
        s_m[warp][8 * n + r] = m[n];
        s_l[warp][8 * n + r] = l[n];
      }
      if (lane == 0) s_bad[warp] = bad;
#pragma unroll
      for (int t = 0; t < C::kMT; ++t) {
        const int d = out_d<D, FP8>(r, t);
        *reinterpret_cast<float2*>(&s_o[warp][2 * q4][d]) = make_float2(o[n][t][0], o[n][t][2]);
        *reinterpret_cast<float2*>(&s_o[warp][2 * q4 + 1][d]) = make_float2(o[n][t][1], o[n][t][3]);
      }
      __syncthreads();
      const bool any_bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
      const int heads = min(8, G - 8 * n);
      for (int i = threadIdx.x; i < heads * D; i += kDecThreads) {
        const int h = i / D, d = i % D, hh = 8 * n + h;
        float top = s_m[0][hh];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_m[w][hh]);
        float sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float f = s_m[w][hh] == -INFINITY ? 0.f : ex2(s_m[w][hh] - top);
          sum = fmaf(s_l[w][hh], f, sum);
          acc = fmaf(s_o[w][h][d], f, acc);
        }
        if (any_bad) sum = __int_as_float(0x7FFFFFFF);
        const int64_t row = static_cast<int64_t>(cur.b) * a.hq + cur.g * G + hh;
        if constexpr (ONE) {  // over the ring: every warp has used its last step
          s_part[hh * D + d] = acc;
          if (d == 0) s_pml[hh] = make_float2(top, sum);
        } else if (cur.whole) {
          a.out[row * D + d] = __float2bfloat16(acc / sum * vs);
          if (d == 0) {
            const float lse2 = top + (log2f(sum) - (FP8 ? 14.f : 0.f));
            if (a.lse != nullptr) a.lse[row] = lse2 * 0.6931471805599453f;
            if (a.lse2 != nullptr) a.lse2[row] = lse2;
          }
        } else {
          a.part_o[(part * G + hh) * D + d] = acc;
          if (d == 0) a.part_ml[part * G + hh] = make_float2(top, sum);
        }
      }
      if (n == 0 && threadIdx.x == 0) note(any_bad);
      __syncthreads();  // the shared parts may be overwritten
    }
    if constexpr (ONE) break;
    if (!more) break;
    cur = nxt;
  }

  if constexpr (ONE) {
    // ---------------------------------------------------- the cluster's parts together
    constexpr float kShift = FP8 ? 14.f : 0.f;
    if (cluster > 1) cluster_sync(); else __syncthreads();
    const float vs = FP8 ? __ldg(a.v_scale + static_cast<int64_t>(cur.b) * a.hkv + cur.g) : 1.f;
    const int64_t row0 = static_cast<int64_t>(cur.b) * a.hq + cur.g * G;
    for (int h = cta; h < G; h += cluster) {
      float2 ml[kOneCluster];
      float x[kOneCluster];
      const int d = threadIdx.x;
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < kOneCluster; ++c) {
        ml[c] = make_float2(-INFINITY, 0.f);
        x[c] = 0.f;
        if (c < cluster) {
          ml[c] = ld_cluster_f32x2(cluster_map(&s_pml[h], c));
          if (d < D) x[c] = ld_cluster_f32(cluster_map(&s_part[h * D + d], c));
          top = fmaxf(top, ml[c].x);
        }
      }
      float sum = 0.f, acc = 0.f;
#pragma unroll
      for (int c = 0; c < kOneCluster; ++c) {
        const float f = ml[c].x == -INFINITY ? 0.f : ex2(ml[c].x - top);
        sum = fmaf(ml[c].y, f, sum);
        acc = fmaf(x[c], f, acc);
      }
      if (d < D) a.out[(row0 + h) * D + d] = __float2bfloat16(acc / sum * vs);
      if (d == 0 && a.lse != nullptr)
        a.lse[row0 + h] = (top + (log2f(sum) - kShift)) * 0.6931471805599453f;
    }
    if (a.raw != nullptr) {
      if (threadIdx.x < G) {
        float top = -INFINITY, sum = 0.f;
        for (int c = 0; c < cluster; ++c)
          top = fmaxf(top, ld_cluster_f32x2(cluster_map(&s_pml[threadIdx.x], c)).x);
        for (int c = 0; c < cluster; ++c) {
          const float2 ml = ld_cluster_f32x2(cluster_map(&s_pml[threadIdx.x], c));
          sum = fmaf(ml.y, ml.x == -INFINITY ? 0.f : ex2(ml.x - top), sum);
        }
        s_lse2[threadIdx.x] = top + (log2f(sum) - kShift);
      }
      __syncthreads();
      const int64_t out_row = (static_cast<int64_t>(cur.b) * a.hkv + cur.g) * a.score_stride;
      for (int j = cur.kb + threadIdx.x; j < cur.ke; j += kDecThreads) {  // this CTA's own keys
        float w = 0.f;
        for (int h = 0; h < G; ++h) {
          const float lse2 = s_lse2[h];
          const float x = a.raw[(row0 + h) * a.raw_stride + j];
          if (lse2 > -INFINITY) w += ex2(x - lse2);
        }
        a.score_out[out_row + j] = (a.score_in != nullptr ? a.score_in[out_row + j] : 0.f) + w;
      }
    }
    if (cluster > 1) cluster_sync();  // no CTA leaves while others read its part
  }
}

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
                           ? __ldg(a.v_scale + static_cast<int64_t>(seq) * a.hkv + head) : 1.f;
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
  if (first >= n) return;
  // the inputs of the call and what does not depend on lse2 first
  float base[kWeightPer];
#pragma unroll
  for (int k = 0; k < kWeightPer; ++k) {
    const int64_t j = first + k * kFinishThreads + threadIdx.x;
    base[k] = a.score_in != nullptr && j < n ? a.score_in[out_row + j] : 0.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    join_parts<D>(a, ctas, l_shift);
  } else {
    const int i = static_cast<int>(blockIdx.x) - ctas;
    add_weights(a, ctas, l_shift, i / chunks, i % chunks, chunks);
  }
}

template <int D, bool FP8, int NT>
cudaError_t launch_decode_t(PagedDecodeArgs& a, int num_sms, cudaStream_t stream) {
  using C = DecCfg<D, FP8>;
  cudaError_t e;
  // One launch where clusters of up to eight CTAs, eight tiles each at most, all fit the GPU
  // at once: there a launch less is worth more than an even division. Measured against the
  // divided runs (8 KV heads, d = 128): one sequence of 777 tokens 6.0 us and 7.6, four of
  // 2,000 9.2 and 12.9, four of 4,000 15.7 and 20.7, four of 1,000-4,000 with weights 19.5 and
  // 18.4; past the rule, one of 8,000 15.8 and 13.1, sixteen of 2,000 39.5 and 30.4.
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
  const int tiles = (a.max_len + C::kTile - 1) / C::kTile;
  int cluster = 1;
  while (cluster < kOneCluster && cluster < tiles) cluster *= 2;
  if (tiles <= 8 * cluster && pairs * cluster <= 2 * num_sms) {
    static std::atomic<uint64_t> one_ready{0};
    e = allow_smem(reinterpret_cast<const void*>(paged_decode_kernel<D, FP8, NT, kOne>), C::kSmem,
                   one_ready);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute dims;
    dims.id = cudaLaunchAttributeClusterDimension;
    dims.val.clusterDim.x = cluster;
    dims.val.clusterDim.y = 1;
    dims.val.clusterDim.z = 1;
    cudaLaunchConfig_t one{};
    one.gridDim = dim3(static_cast<unsigned>(pairs * cluster));
    one.blockDim = dim3(kDecThreads);
    one.dynamicSmemBytes = C::kSmem;
    one.stream = stream;
    one.attrs = &dims;
    one.numAttrs = 1;
    return cudaLaunchKernelEx(&one, paged_decode_kernel<D, FP8, NT, kOne>, a, cluster);
  }
  // runs of warps or of CTAs
  const bool warps = decode_by_warps(a.num_seqs, a.hkv, a.max_len, C::kTile);
  const int tile = warps ? C::kKeys : C::kTile;
  const int ctas = decode_ctas(num_sms, a.num_seqs, a.hkv, a.max_len, C::kTile);
  const int runs = warps ? ctas * kDecWarps : ctas;
  if (warps) {
    static std::atomic<uint64_t> warps_ready{0};
    e = allow_smem(reinterpret_cast<const void*>(paged_decode_kernel<D, FP8, NT, kWarps>), C::kRing,
                   warps_ready);
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, FP8, NT, kWarps><<<ctas, kDecThreads, C::kRing, stream>>>(a, 1);
  } else {
    static std::atomic<uint64_t> ready{0};
    e = allow_smem(reinterpret_cast<const void*>(paged_decode_kernel<D, FP8, NT, kSplit>), C::kSmem,
                   ready);
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, FP8, NT, kSplit><<<ctas, kDecThreads, C::kSmem, stream>>>(a, 1);
  }
  e = cudaGetLastError();
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
      const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.hkv;
      const int most = (a.max_len + kWeightKeys - 1) / kWeightKeys;
      // Blocks of 1,024 keys as long as there are not many thousands of them (the lengths may
      // be far below max_seq_len); beyond that a block takes several chunks.
      const int64_t room = 8192 / pairs;
      chunks = static_cast<int>(most < room ? most : room < 1 ? 1 : room);
      blocks += pairs * chunks;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kFinishThreads);
    e = cudaLaunchKernelEx(&cfg, paged_finish_kernel<D>, a, runs, FP8 ? 14.f : 0.f, chunks);
  }
  return e;
}

}  // namespace

int decode_tile_keys(int head_dim, bool fp8) {
  return kDecWarps * kStepBytes / (head_dim * (fp8 ? 1 : 2));
}

// Where a CTA has several short pieces in its run, putting its warps' parts together is what
// takes the time (8 us a piece). Measured against runs of CTAs: 181 sequences of 20-83 tokens
// (8 KV heads, G = 16, e4m3) 27.0 us and 40.8, 256 of 16-128 (8, G = 4) 29.2 and 38.7, 100 of
// 100-500 (8, G = 8) 33.6 and 39.8, 128 of 300-600 (8, G = 4, e4m3) 35.0 and 37.8; past the rule,
// 93 of 431-589 43.9 and 41.9, 128 of 500-1,000 73.6 and 70.7 (parts of more runs to join).
bool decode_by_warps(int num_seqs, int hkv, int max_len, int tile) {
  return static_cast<int64_t>(num_seqs) * hkv >= 2 * kDecodeMaxCtas && max_len <= 8 * tile;
}

int decode_ctas(int num_sms, int num_seqs, int hkv, int max_len, int tile) {
  const int64_t most = static_cast<int64_t>(num_seqs) * hkv * ((max_len + tile - 1) / tile);
  int64_t full = static_cast<int64_t>(num_sms) * 2;
  if (full > kDecodeMaxCtas) full = kDecodeMaxCtas;  // the workspace holds so many partials
  return static_cast<int>(most < 1 ? 1 : most < full ? most : full);
}

cudaError_t launch_paged_decode(PagedDecodeArgs& a, int head_dim, bool fp8, int num_sms,
                                cudaStream_t stream) {
  const bool two = a.group > 8;
  if (head_dim == 128) {
    if (fp8) return two ? launch_decode_t<128, true, 2>(a, num_sms, stream)
                        : launch_decode_t<128, true, 1>(a, num_sms, stream);
    return two ? launch_decode_t<128, false, 2>(a, num_sms, stream)
               : launch_decode_t<128, false, 1>(a, num_sms, stream);
  }
  if (fp8) return two ? launch_decode_t<64, true, 2>(a, num_sms, stream)
                      : launch_decode_t<64, true, 1>(a, num_sms, stream);
  return two ? launch_decode_t<64, false, 2>(a, num_sms, stream)
             : launch_decode_t<64, false, 1>(a, num_sms, stream);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, int num_sms,
                                cudaStream_t stream) {
  // about 2,048 vectors per block where there are enough tokens, else one block per token
  int64_t tok = 2048 / (2 * (a.row_elems / 8));
  const int64_t spread = (a.total_new + 2 * num_sms - 1) / (2 * num_sms);
  if (tok > spread) tok = spread;
  if (tok > kAppendMaxTok) tok = kAppendMaxTok;
  if (tok < 1) tok = 1;
  const unsigned blocks = static_cast<unsigned>((a.total_new + tok - 1) / tok);
  if (fp8)
    paged_append_kernel<true><<<blocks, kAppendThreads, 0, stream>>>(a, static_cast<int>(tok));
  else
    paged_append_kernel<false><<<blocks, kAppendThreads, 0, stream>>>(a, static_cast<int>(tok));
  return cudaGetLastError();
}

}  // namespace quail

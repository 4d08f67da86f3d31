// fp4_decode.cu - attention of one new token per sequence over a paged key/value cache held in
// 4 bits. "Motor de inferência Quail atinge 1 bilhão de tokens por minuto por GPU", section
// "Como funciona", keeps anchor KV between prefills; in 4 bits 3.6 times as many anchors fit.
//
//   out = S_v sum_j w_j v_j,  w_j = exp2(c S_k q.k_j - lse2),  k_j, v_j = code * block scale
//
// How the batch is divided and joined is as over the other forms of pages (see paged.cu), but that short
// sequences take a warp per head (kPairs). A warp walks its keys with a running max and sum. HBM gives
// 144 bytes per (token, KV head) at d = 128, 24 issue slots of an SM's quarter at the measured copy rate,
// into which 256 codes have to go through conversion (two cycles of the ALU for 32 pairs), scaling and
// two products (eight cycles of the tensor pipe each); so every step's instructions count:
//   S^T [16 keys x 8 heads]  A = K: keys fill the 16 rows (heads would fill 1 to 8 of them), half the
//            products. Lane (r, q) holds pieces q of two keys as they lie in memory: sums over d may run
//            in any order, so its codes ARE its fragments, and they belong to one (d = 64) or two block
//            scales.
//   O^T [16 d x 8 heads]     A = V^T: lane (r, q) holds one block (d = 64: half of one) of four keys.
//            Their nibbles are interleaved before the conversion (4 operations for 8 pairs; permuting the
//            converted halves would take 8); B = P^T, the score fragment transposed in 8 x 8 blocks. The
//            heads of a lane's scores are those of its outputs, so the running max needs no exchange
//            while no score passes it.
// With up to four heads the other four columns are the same heads again: their P^T holds the second term
// of P's sum, and one product does both (64 sequences of 8,000-16,000 tokens: 189 -> 175 us).
// Loads are bulk copies of whole pieces of pages into a ring of two steps, issued by a warp of its own or
// by the warp that computes.
// Products of code and block scale are exact in f16. Q is scaled per head by a power of two into
// f16's range (bits below 2^-38 of the head's largest |q| are lost, under fp32's own rounding); P,
// scaled by 2^14, is the sum of two f16 (22 bits, weights down to 2^-38 of the largest).
// Measured (8 KV heads, G = 4, d = 128, in a graph, of the measured copy rate): one sequence of 131,007
// tokens 38.6 us (58 %), 64 of 8,000-16,000 172 us (75 %), 64 of 128-4,096 44 us (51 %). About 650
// instructions per warp and 32 keys, 0.6 a cycle and quarter with three CTAs on an SM; two took 206 us
// instead of 189 for the second case, four (128 registers) 196, a ring of three steps the same as two.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "paged_decode.cuh"
#include "ptx.cuh"
#include "step_ring.cuh"

namespace quail {

namespace {

constexpr int kFp4PerSm = 3;  // CTAs per SM
constexpr int kSide = 2;      // 16-key blocks whose scores are worked out side by side

template <int D>
struct Fp4Cfg {
  static constexpr int kStages = 2;                  // steps in a warp's ring
  static constexpr int kCB = D / 2;                  // code bytes of a (token, head) row
  static constexpr int kSB = D / 16;                 // its block scales
  static constexpr int kKeys = fp4_tile_keys(D) / kDecWarps;  // keys per warp step: 32 or 64
  static constexpr int kG16 = kKeys / 16;
  static constexpr int kCodes = kKeys * kCB;         // 2,048 bytes of K, and of V, in one step
  static constexpr int kScales = kKeys * kSB;        // 256
  static constexpr int kStep = 2 * (kCodes + kScales);
  static constexpr int kTile = kDecWarps * kKeys;
  static constexpr int kMT = D / 16;                 // 16-row tiles of O^T
  static constexpr int kQS = D / 16;                 // k-steps of the score product
  static constexpr int kWords = D / 64;              // words of V per lane and key
  static constexpr int kRing = kDecWarps * kStages * kStep;
  static constexpr int kSmem = kRing + kDecWarps * 8 * D * 4;  // + the warps' O, 8 heads
};

// The step's data is read only here, and every read is volatile like the wait before it: no clobber of
// memory, so that reads may pass other memory operations.
__device__ __forceinline__ uint4 step16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 step8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void st_shared_u8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// `bytes` (a multiple of 16, both addresses too) to shared memory, counted at mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t smem, const uint8_t* p, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem),
      "l"(p), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for a phase; false past the limit (the device error word is set, and *abort), or once a wait
// of another warp has set *abort.
__device__ __noinline__ bool fp4_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                      unsigned* err_word, volatile int* abort) {
  const uint64_t deadline = global_timer_ns() + timeout_ns;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) != 0) continue;
    if (abort != nullptr && *abort != 0) return false;
    if (global_timer_ns() > deadline) {
      atomicOr(err_word, kErrTimeout);
      if (abort != nullptr) *abort = 1;
      return false;
    }
  }
}
// The four warps that compute.
__device__ __forceinline__ void team_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kDecThreads) : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An 8 x 8 matrix of 16-bit values, transposed: lane (r, q) gives row r's 2q, 2q + 1 and takes
// column r's.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t both(uint32_t h2, int high) {
  return __byte_perm(h2, h2, high ? 0x3232 : 0x1010);
}

// Runs of CTAs have a fifth warp that loads their tiles. With 16 heads the registers that it takes from
// the others cost more than it saves (32 sequences of 1,000-4,096 tokens: 49.4 us against 45.5; with 4
// and 8 heads 64 of 128-4,096: 44.1 against 45.9, 48.7 against 51.0).
template <int H, DecMode MODE>
constexpr bool kFp4Loader = MODE == kSplit && H <= 8;
template <int H, DecMode MODE>
constexpr int kFp4Threads = kDecThreads + (kFp4Loader<H, MODE> ? 32 : 0);

template <int D, int H, DecMode MODE>
__global__ void __launch_bounds__(kFp4Threads<H, MODE>, H <= 8 ? kFp4PerSm : 2)
    fp4_decode_kernel(const PagedDecodeArgs a, int cluster) {
  using C = Fp4Cfg<D>;
  constexpr bool PROD = kFp4Loader<H, MODE>;
  constexpr bool ONE = MODE == kOne, PAIRS = MODE == kPairs;
  constexpr bool WARPS = MODE == kWarps || PAIRS;  // no warp waits for another
  constexpr int NT = H <= 8 ? 1 : 2;     // tiles of 8 heads
  constexpr bool FOLD = H == 4;          // columns 4 to 7 are the same heads: there P's second term
  constexpr int kTile = WARPS ? C::kKeys : C::kTile;  // keys that a run is counted in
  constexpr float kShift = 14.f;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ float s_m[kDecWarps][8 * NT], s_l[kDecWarps][8 * NT];
  __shared__ int s_bad[kDecWarps], s_bad_tile[C::kStages];
  __shared__ volatile int s_abort;       // PROD: a wait ran out
  // pieces and run of each warp: read at their borders, not worth registers in between
  __shared__ Piece s_piece[kDecWarps], s_ld[kDecWarps];
  __shared__ int64_t s_run[kDecWarps][2];
  // [warp][stage] a step's copies have landed; PROD: [0] a tile's have, [1] its warps have read it
  __shared__ uint64_t s_full[kDecWarps][C::kStages];
  float(*s_o)[8][D] = reinterpret_cast<float(*)[8][D]>(dyn + C::kRing);  // [warp][head][d]
  float* s_part = reinterpret_cast<float*>(dyn);  // ONE, at the end: [head][d]
  __shared__ float2 s_pml[ONE ? 8 * NT : 1];
  __shared__ float s_lse2[ONE ? 8 * NT : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, q4 = lane & 3;
  const int G = a.group;
  after_stream();
  if constexpr (!ONE && !PAIRS) let_next_start();  // the join
  // who takes a run (a CTA, a warp), or ONE: the rank
  const int cta = ONE ? static_cast<int>(blockIdx.x) % cluster
                      : WARPS ? static_cast<int>(blockIdx.x) * kDecWarps + warp : blockIdx.x;
  const int ctas = WARPS ? static_cast<int>(gridDim.x) * kDecWarps : gridDim.x;
  const int split = PAIRS ? a.split : 0;  // of the pages' heads it is g >> split
  // PAIRS: the next (sequence, head) with tokens of this warp's, from p.at on; what the others get
  // is written on one of the two walks over them
  auto next_pair = [&](Piece& p, bool write) {
    const int heads = a.hkv << split;
    for (; p.at < static_cast<int64_t>(a.num_seqs) * heads; p.at += ctas) {
      p.b = static_cast<int>(p.at / heads);
      p.g = static_cast<int>(p.at % heads);
      p.len = p.ke = checked_len(a, p.b);
      if (p.len > 0) return true;
      if (write) write_empty(a, p.b, p.len, p.g * G, (p.g + 1) * G, D, lane, 32);
    }
    return false;
  };
  Piece first;
  int64_t run_end = 0, run_total = 0;
  if constexpr (ONE) {
    const int pair = static_cast<int>(blockIdx.x) / cluster;
    first.b = pair / a.hkv;
    first.g = pair % a.hkv;
    first.len = checked_len(a, first.b);
    if (first.len <= 0) {  // the same for every CTA of the cluster
      if (cta == 0) write_empty(a, first.b, first.len, first.g * G, (first.g + 1) * G, D);
      return;
    }
    const int tiles = (first.len + C::kTile - 1) / C::kTile;
    first.piece0 = 0;
    first.at = first_tile(cta, tiles, cluster);
    run_end = first_tile(cta + 1, tiles, cluster);
  } else if constexpr (PAIRS) {
    first.at = cta;
    first.kb = 0;
    first.whole = true;
    if (!next_pair(first, true)) return;
  } else {
    // sequences without tokens (0 and -inf) and with lengths out of range (NaN)
    for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
      const int n = checked_len(a, b);
      if (n <= 0) write_empty(a, b, n, 0, a.hq, D, threadIdx.x, kFp4Threads<H, MODE>);
    }
    const RunStart run = find_run(a, kTile, cta, ctas);
    if (WARPS ? lane == 0 : threadIdx.x == 0) a.rec[cta] = DecodeRec{-1, 0, 0, 0};
    if (run.begin >= run.end) return;
    first.b = run.seq;
    first.len = checked_len(a, first.b);
    const int tiles = (first.len + kTile - 1) / kTile;
    first.g = static_cast<int>((run.begin - run.seq_tile0) / tiles);
    first.piece0 = run.seq_tile0 + static_cast<int64_t>(first.g) * tiles;
    first.at = run.begin;
    run_end = run.end;
    run_total = run.total;
  }
  if constexpr (!PAIRS) set_piece<kTile>(a, run_end, first);

  // ------------------------------------------------------ loads
  // A tile's (PROD) or step's keys of one page lie together in memory and in the ring: four copies,
  // issued by one lane.
  constexpr int kStages = C::kStages;
  constexpr int kShare = PROD ? kDecWarps : 1;  // warps whose steps a stage holds
  const int slot = PROD ? 0 : warp;
  const uint32_t ring = smem_u32(dyn) + slot * (kStages * C::kStep);
  const uint32_t full = smem_u32(&s_full[slot][0]);
  const uint32_t empty = smem_u32(&s_full[1][0]);  // PROD
  if (PROD ? threadIdx.x == 0 : lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_full[slot][i], 1);
      if constexpr (PROD) mbar_init(&s_full[1][i], kDecWarps);
    }
    fence_mbar_init();
  }
  if (lane == 0 && warp < kDecWarps) {
    s_piece[warp] = s_ld[warp] = first;
    s_run[warp][0] = run_end;
    s_run[warp][1] = run_total;
  }
  if (PROD && threadIdx.x == 0) s_abort = 0;
  if constexpr (PROD) __syncthreads(); else __syncwarp();
  const int64_t head_bytes = static_cast<int64_t>(C::kCB + C::kSB) << a.page_shift;
  const int64_t page_bytes = head_bytes * a.hkv;
  const int64_t scales_at = static_cast<int64_t>(C::kCB) << a.page_shift;
  const int page_mask = (1 << a.page_shift) - 1;
  // `keys` from key `pos` on, in page pg, to place `from` of the stage at `to`
  auto load = [&](uint32_t to, uint32_t bar, int pg, int64_t head, int pos, int from, int keys) {
    const int64_t base = pg * page_bytes + head;
    const int at = pos & page_mask;
    const int64_t c = base + at * C::kCB, sc = base + scales_at + at * C::kSB;
    const uint32_t codes = to + from * C::kCB, scales = to + 2 * kShare * C::kCodes + from * C::kSB;
    bulk_load(codes, a.k_pages + c, keys * C::kCB, bar);
    bulk_load(codes + kShare * C::kCodes, a.v_pages + c, keys * C::kCB, bar);
    bulk_load(scales, a.k_pages + sc, keys * C::kSB, bar);
    bulk_load(scales + kShare * C::kScales, a.v_pages + sc, keys * C::kSB, bar);
  };
  if constexpr (PROD) {
    if (warp == kDecWarps) {
      const int part = min(page_mask + 1, C::kTile);  // keys of a tile in one page
      Piece ld = first;
      int key = ld.kb, st = 0;
      uint32_t lap = 0;
      auto page_of = [&]() {             // lane i: of the tile's i-th part
        const int pos = key + lane * part;
        return lane * part < C::kTile && pos < ld.ke
                   ? a.table[static_cast<int64_t>(ld.b) * a.max_pages + (pos >> a.page_shift)] : -1;
      };
      int page = page_of();
      bool more = true;
      while (more) {
        const int keys = min(C::kTile, ld.ke - key), from_key = key, my_page = page;
        const int64_t head = ld.g * head_bytes;
        key += C::kTile;
        if (key >= ld.ke) {
          more = next_piece<kTile>(a, run_end, ld);
          key = ld.kb;
        }
        if (more) page = page_of();      // the next tile's, on its way while the stage is waited for
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(empty + 8 * st, lap ^ 1)) &&
            !__all_sync(0xFFFFFFFFu, fp4_wait(empty + 8 * st, lap ^ 1, a.timeout_ns, a.err_word, &s_abort)))
          break;
        const bool held = lane * part < keys;
        const bool ok = held && static_cast<unsigned>(my_page) < static_cast<unsigned>(a.num_pages);
        // whole 16s: a page holds no fewer
        const int mine = ok ? min(part, (keys - lane * part + 15) / 16 * 16) : 0;
        unsigned todo = __ballot_sync(0xFFFFFFFFu, ok);
        const bool bad = todo != __ballot_sync(0xFFFFFFFFu, held);
        const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(mine));
        const uint32_t bar = full + 8 * st, to = ring + st * (kShare * C::kStep);
        if (lane == 0) {
          s_bad_tile[st] = bad;
          mbar_expect_tx(bar, sum * (2 * (C::kCB + C::kSB)));
        }
        __syncwarp();
        if (a.inject_skip_loads != 0) todo = 0;
        for (; todo != 0; todo &= todo - 1) {
          const int i = __ffs(todo) - 1;
          const int pg = __shfl_sync(0xFFFFFFFFu, my_page, i), n = __shfl_sync(0xFFFFFFFFu, mine, i);
          if (elect_one()) load(to, bar, pg, head, from_key + i * part, i * part, n);
        }
        if (++st == kStages) {
          st = 0;
          lap ^= 1;
        }
      }
      // what is on its way lands before the CTA's memory is given up, or the limit passes
      for (int i = 0; i < kStages; ++i)
        fp4_wait(full + 8 * i, i < st ? lap : lap ^ 1, a.timeout_ns, a.err_word, nullptr);
      return;
    }
  }
  // the others: a cursor of their own
  const int own = WARPS ? 0 : warp * C::kKeys;  // the warp's first key in a tile
  int ld_key = first.kb + own;           // first key of the next step to load
  int ld_ke = first.ke;
  const int32_t* ld_table = a.table + static_cast<int64_t>(first.b) * a.max_pages;
  int64_t ld_head = (first.g >> split) * head_bytes;
  int page = 0;                          // page of ld_key; where a step has several, lane i has the i-th
  bool ld_more = true, late = false;     // late: a wait ran out, the results are NaN
  uint32_t bad_steps = 0;                // bit s: a page of the step in stage s is no page
  auto seek = [&]() {                    // on to a piece that has a step for this warp
    while (ld_key >= ld_ke) {
      Piece ld = s_ld[warp];
      if constexpr (PAIRS) {
        ld.at += ctas;
        ld_more = next_pair(ld, false);
      } else {
        ld_more = next_piece<kTile>(a, s_run[warp][0], ld);
      }
      if (!ld_more) return;
      __syncwarp();
      if (lane == 0) s_ld[warp] = ld;
      __syncwarp();
      ld_key = ld.kb + own;
      ld_ke = ld.ke;
      ld_table = a.table + static_cast<int64_t>(ld.b) * a.max_pages;
      ld_head = (ld.g >> split) * head_bytes;
    }
    const int last = (min(C::kKeys, ld_ke - ld_key) - 1 + (ld_key & page_mask)) >> a.page_shift;
    page = ld_table[(ld_key >> a.page_shift) + min(lane, last)];
  };
  auto issue = [&](int stage) {          // the stage's last step has been read by every lane
    if (!ld_more) return;
    const uint32_t bar = full + 8 * stage, to = ring + stage * C::kStep;
    const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
    bool bad;
    if (page_mask >= C::kKeys - 1) {     // a step is in one page (whose rows past the last key come too)
      bad = !ok;
      if (elect_one()) {
        mbar_expect_tx(bar, ok ? C::kStep : 0);
        if (ok && a.inject_skip_loads == 0) load(to, bar, page, ld_head, ld_key, 0, C::kKeys);
      }
    } else {
      const int parts = (min(C::kKeys, ld_ke - ld_key) + page_mask) >> a.page_shift;
      unsigned todo = __ballot_sync(0xFFFFFFFFu, ok && lane < parts);
      bad = __popc(todo) != parts;
      if (elect_one())
        mbar_expect_tx(bar, __popc(todo) * (2 * (C::kCB + C::kSB) << a.page_shift));
      __syncwarp();
      if (a.inject_skip_loads != 0) todo = 0;
      for (; todo != 0; todo &= todo - 1) {
        const int i = __ffs(todo) - 1, pg = __shfl_sync(0xFFFFFFFFu, page, i);
        const int from = i << a.page_shift;
        if (elect_one()) load(to, bar, pg, ld_head, ld_key + from, from, page_mask + 1);
      }
    }
    bad_steps = bad ? bad_steps | (1u << stage) : bad_steps & ~(1u << stage);
    ld_key += kTile;
    seek();
  };

  // Q of a piece as it is in memory: the D / 4 values from d = q4 D / 4 of head r (+ 8)
  uint4 qraw[NT][D / 32];
  float k_scale, v_scale;                // of the same (sequence, head)
  auto load_q = [&](int b, int g) {
    k_scale = a.k_scale[static_cast<int64_t>(b) * a.hkv + (g >> split)];
    v_scale = a.v_scale[static_cast<int64_t>(b) * a.hkv + (g >> split)];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = FOLD ? r & 3 : r + 8 * n;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(b) * a.q_stride + static_cast<int64_t>(g * G + h) * D +
          q4 * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        qraw[n][i] = h < G ? qp[i] : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  // Row i of a product's 8 keys is key i ^ (i / 2 % 2): the rows that a read of V's takes at once
  // lie half on even and half on odd keys, on different banks.
  const int kr = r ^ ((r >> 1) & 1);
  const int v_row[2] = {2 * q4 + (q4 & 1), 2 * q4 + (~q4 & 1)};

  if constexpr (!PROD) seek();
  load_q(first.b, first.g);
  if constexpr (!PROD) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s);
  }
  StepRing<kStages> due;                 // the step that is waited for

  while (true) {
    // ---------------------------------------------------- one piece
    const int key_end = s_piece[warp].ke, key_begin = s_piece[warp].kb;
    uint32_t qb[NT][C::kQS][2];
    float c_log2[NT][2];                 // of heads 2 q4, 2 q4 + 1 (+ 8 n)
    {
      const float ks = k_scale;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          top = absmax_bf16x2(absmax_bf16x2(top, qraw[n][i].x), qraw[n][i].y);
          top = absmax_bf16x2(absmax_bf16x2(top, qraw[n][i].z), qraw[n][i].w);
        }
        float mx = absmax_bf16x2_value(top);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        // 2^e with mx 2^e in [2^14, 2^15); zero, infinite and NaN rows are left as they are
        int e = mx > 0.f && mx < INFINITY ? 14 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127) : 0;
        e = min(e, 126);  // a power of two that is a normal float, as is its inverse
        const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        const float c = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * ks;
        c_log2[n][0] = __shfl_sync(0xFFFFFFFFu, c, 8 * q4);
        c_log2[n][1] = __shfl_sync(0xFFFFFFFFu, c, 8 * q4 + 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t w[4] = {qraw[n][i].x, qraw[n][i].y, qraw[n][i].z, qraw[n][i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qb[n][2 * i + (j >> 1)][j & 1] = pack2<true>(__uint_as_float(w[j] << 16) * up,
                                                         __uint_as_float(w[j] & 0xFFFF0000u) * up);
        }
      }
    }

    float o[NT][C::kMT][4];
    float m[NT][2], l[NT][2];            // of heads 2 q4, 2 q4 + 1; l of this lane's keys
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < C::kMT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][t][j] = 0.f;
    }
    bool bad = false;

    // (PROD: every warp goes through all tiles, also one that has no keys in the last)
    for (int key0 = key_begin + own; key0 - (PROD ? own : 0) < key_end; key0 += kTile) {
      const bool next_too = ld_more;     // the next step is issued as well
      if constexpr (!PROD) {
        __syncwarp();  // the stage before was read by every lane
        issue(due.ahead());
      }
      const int stage = due.stage;
      if (!late && !__all_sync(0xFFFFFFFFu, mbar_try_wait(full + 8 * stage, due.parity))) {
        late = !__all_sync(0xFFFFFFFFu,
                           fp4_wait(full + 8 * stage, due.parity, a.timeout_ns, a.err_word,
                                    PROD ? &s_abort : nullptr));
        if (!PROD && late) {
          // Nothing more is loaded, and what is on its way lands before the ring's memory is used for
          // anything else or given up, or the limit passes.
          static_assert(kStages == 2, "this step and the next one are all that can be on their way");
          ld_more = false;
          due.drain(next_too ? 2 : 1, [&](int s, uint32_t parity) {
            fp4_wait(full + 8 * s, parity, a.timeout_ns, a.err_word, nullptr);
          });
        }
      }
      bad |= late || (PROD ? s_bad_tile[stage] != 0 : (bad_steps >> stage) & 1u);
      const uint32_t step = ring + stage * (kShare * C::kStep), share = PROD ? warp : 0;
      const uint32_t kbuf = step + share * C::kCodes, vbuf = kbuf + kShare * C::kCodes;
      const uint32_t ksc = step + 2 * kShare * C::kCodes + share * C::kScales, vsc = ksc + kShare * C::kScales;
      const uint32_t read = empty + 8 * stage;
      due.next();
      if (PROD && key0 >= key_end) {
        __syncwarp();  // every lane has read s_bad_tile
        if (lane == 0 && !late) mbar_arrive_at(read);
        continue;
      }
      const bool tail = key0 + C::kKeys > key_end;
      if (tail) {  // what a page holds behind the last key may be no number: scales of zero
        __syncwarp();
        for (int i = (key_end - key0) * C::kSB + lane; i < C::kScales; i += 32) st_shared_u8(vsc + i, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later copy there
        __syncwarp();
      }

      // ---- scores of this step's keys: s[i][n] = keys r, r + 8 of block i by heads 2 q4, + 1
      float s[C::kG16][NT][4];
#pragma unroll
      for (int i0 = 0; i0 < C::kG16; i0 += kSide) {  // blocks of keys side by side
        uint32_t w[kSide][2][D / 32], sc[kSide][2][D / 64];
#pragma unroll
        for (int i = 0; i < kSide; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = 16 * (i0 + i) + 8 * u + kr;
            if constexpr (D == 128) {
              const uint4 x = step16(kbuf + key * C::kCB + 16 * q4);
              w[i][u][0] = x.x;
              w[i][u][1] = x.y;
              w[i][u][2] = x.z;
              w[i][u][3] = x.w;
              const uint32_t h2 = e4m3_lo(ld_shared_u16(ksc + key * C::kSB + 2 * q4));
              sc[i][u][0] = both(h2, 0);
              sc[i][u][1] = both(h2, 1);
            } else {
              const uint2 x = step8(kbuf + key * C::kCB + 8 * q4);
              w[i][u][0] = x.x;
              w[i][u][1] = x.y;
              sc[i][u][0] = both(e4m3_lo(ld_shared_u8(ksc + key * C::kSB + q4)), 0);
            }
          }
#pragma unroll
        for (int i = 0; i < kSide; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            s[i0 + i][n][0] = s[i0 + i][n][1] = s[i0 + i][n][2] = s[i0 + i][n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)  // 8 codes of each key: two k-steps
#pragma unroll
          for (int i = 0; i < kSide; ++i) {
            uint32_t x[4], y[4];
            e2m1x8(w[i][0][j], x);
            e2m1x8(w[i][1][j], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = mul_f16x2(x[k], sc[i][0][j >> 1]);
              y[k] = mul_f16x2(y[k], sc[i][1][j >> 1]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(s[i0 + i][n], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1],
                               qb[n][2 * j + k][0], qb[n][2 * j + k][1]);
          }
      }

      // ---- running max and sum; x = score in log2 units
#pragma unroll
      for (int i = 0; i < C::kG16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][n][j] *= c_log2[n][j & 1];
      if (tail) {
#pragma unroll
        for (int i = 0; i < C::kG16; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (key0 + 16 * i + 8 * u + kr >= key_end) {
#pragma unroll
              for (int n = 0; n < NT; ++n) s[i][n][2 * u] = s[i][n][2 * u + 1] = -INFINITY;
            }
      }
      if (a.raw != nullptr) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = 8 * n + 2 * q4 + j;
            if (h < G) {
              float* row =
                  a.raw + (static_cast<int64_t>(s_piece[warp].b) * a.hq + s_piece[warp].g * G + h) * a.raw_stride;
#pragma unroll
              for (int i = 0; i < C::kG16; ++i) {  // rows are padded to whole tiles
                row[key0 + 16 * i + kr] = s[i][n][j];
                row[key0 + 16 * i + 8 + kr] = s[i][n][2 + j];
              }
            }
          }
      }
      float mx[NT][2];
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[n][j] = s[0][n][j];
#pragma unroll
          for (int i = 0; i < C::kG16; ++i) {
            if (i > 0) mx[n][j] = fmaxf(mx[n][j], s[i][n][j]);
            mx[n][j] = fmaxf(mx[n][j], s[i][n][2 + j]);
          }
          grew |= mx[n][j] > m[n][j];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float to = fmaxf(m[n][j], mx[n][j]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              to = fmaxf(to, __shfl_xor_sync(0xFFFFFFFFu, to, off));
            const float f = m[n][j] == -INFINITY ? 0.f : ex2(m[n][j] - to);
            l[n][j] *= f;
            m[n][j] = to;
#pragma unroll
            for (int t = 0; t < C::kMT; ++t) {
              o[n][t][j] *= f;
              o[n][t][2 + j] *= f;
            }
          }
      }
      // a row that has seen nothing but -inf takes 0 as its reference: its weights are 0
      float ref[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) ref[n][j] = (m[n][j] == -INFINITY ? 0.f : m[n][j]) - kShift;

      // ---- O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < C::kG16; ++i) {
        constexpr int kTerms = FOLD ? 1 : 2;
        uint32_t ps[NT][kTerms][2];      // [head tile][f16 term][8 keys]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x0 = ex2(s[i][n][2 * u] - ref[n][0]), x1 = ex2(s[i][n][2 * u + 1] - ref[n][1]);
            l[n][0] += x0;
            l[n][1] += x1;
            uint32_t hi, lo;
            split_f16(x0, x1, hi, lo);
            ps[n][0][u] = transpose8(FOLD && q4 >= 2 ? lo : hi);
            if constexpr (!FOLD) ps[n][1][u] = transpose8(lo);
          }
        uint32_t w[4][C::kWords], sb[4];  // codes and scales of keys 2 q4, 2 q4 + 1, and 8 on
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * i + 8 * (j >> 1) + v_row[j & 1];
          if constexpr (D == 128) {
            const uint2 x = step8(vbuf + row * C::kCB + 8 * r);
            w[j][0] = x.x;
            w[j][1] = x.y;
            sb[j] = ld_shared_u8(vsc + row * C::kSB + r);
          } else {
            w[j][0] = ld_shared4(vbuf + row * C::kCB + 4 * r);
            sb[j] = ld_shared_u8(vsc + row * C::kSB + (r >> 1));
          }
        }
        const uint32_t sc0 = e4m3_lo(sb[0] | sb[1] << 8), sc1 = e4m3_lo(sb[2] | sb[3] << 8);
#pragma unroll
        for (int k = 0; k < C::kWords; ++k) {
          auto even = [](uint32_t x, uint32_t y) { return (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u); };
          auto odd = [](uint32_t x, uint32_t y) { return ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u); };
          uint32_t a0[4], a1[4], a2[4], a3[4];
          e2m1x8(even(w[0][k], w[1][k]), a0);
          e2m1x8(odd(w[0][k], w[1][k]), a1);
          e2m1x8(even(w[2][k], w[3][k]), a2);
          e2m1x8(odd(w[2][k], w[3][k]), a3);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            a0[b] = mul_f16x2(a0[b], sc0);
            a1[b] = mul_f16x2(a1[b], sc0);
            a2[b] = mul_f16x2(a2[b], sc1);
            a3[b] = mul_f16x2(a3[b], sc1);
          }
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[n][4 * k + b], a0[b], a1[b], a2[b], a3[b], ps[n][t][0], ps[n][t][1]);
        }
      }
      if constexpr (PROD) {
        __syncwarp();
        if (lane == 0 && !late) mbar_arrive_at(read);
      }
    }

    bad = __any_sync(0xFFFFFFFFu, bad);

    // the next piece's queries are on their way while this one is put together
    const Piece cur = s_piece[warp];
    const float vs = v_scale;
    Piece nxt = cur;
    bool more = false;
    if constexpr (PAIRS) {
      nxt.at += ctas;
      more = next_pair(nxt, true);
    } else if constexpr (!ONE) {
      more = next_piece<kTile>(a, s_run[warp][0], nxt);
    }
    if (more) load_q(nxt.b, nxt.g);

    // ---------------------------------------------------- the four warps' parts together
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], off);
    // slot 0: the run began inside this (b, g); slot 1: the run's last, begun here
    const int64_t part = 2 * static_cast<int64_t>(cta) + (cur.at == cur.piece0 ? 1 : 0);
    auto note = [&](bool any_bad) {      // by one thread, about (b, g)
      if (any_bad) atomicOr(a.err_word, kErrDeviceBounds);
      if (ONE || PAIRS || cur.at != cur.piece0) return;
      if (a.begun != nullptr)
        a.begun[static_cast<int64_t>(cur.b) * a.hkv + cur.g] = cur.whole ? -1 : cta;
      if (!cur.whole) {  // goes on in the next runs: the join's entry
        const int64_t end = cur.piece0 + (cur.len + kTile - 1) / kTile;
        // the last run of (b, g) is the one that holds tile end - 1
        const int64_t total = s_run[warp][1];
        a.rec[cta] = DecodeRec{cur.b, cur.g, static_cast<int>((end * ctas - 1) / total),
                               total < ctas ? static_cast<int>(total) : 0};
      }
    };
    // d of tile t's row r; row r + 8 is the next d
    auto out_d = [&](int t) { return r * (D / 8) + 2 * t; };
    if constexpr (WARPS) {
      if constexpr (FOLD) {
#pragma unroll
        for (int t = 0; t < C::kMT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[0][t][j] += __shfl_xor_sync(0xFFFFFFFFu, o[0][t][j], 2);
      }
      if (lane == 0) note(bad);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = 8 * n + 2 * q4 + j;
          if (h >= G) continue;
          const float sum = bad ? __int_as_float(0x7FFFFFFF) : l[n][j];
          const int64_t row = static_cast<int64_t>(cur.b) * a.hq + cur.g * G + h;
          if (r == 0) {
            if (cur.whole) {
              const float lse2 = m[n][j] + (log2f(sum) - kShift);
              if (a.lse != nullptr) a.lse[row] = lse2 * 0.6931471805599453f;
              if (!PAIRS && a.lse2 != nullptr) a.lse2[row] = lse2;
            } else {
              a.part_ml[part * G + h] = make_float2(m[n][j], sum);
            }
          }
          // (small scales apart: the quotient could have few bits left, or none, where the output has all)
          const bool small = fabsf(vs) < 8.673617379884035e-19f;  // 2^-60
          const float inv = (small ? 1.f : vs) / sum, rest = small ? vs : 1.f;
#pragma unroll
          for (int t = 0; t < C::kMT; t += 4) {  // eight neighbouring d
            if (cur.whole) {
              uint4 x;
              x.x = pack2<false>(o[n][t][j] * inv * rest, o[n][t][2 + j] * inv * rest);
              x.y = pack2<false>(o[n][t + 1][j] * inv * rest, o[n][t + 1][2 + j] * inv * rest);
              x.z = pack2<false>(o[n][t + 2][j] * inv * rest, o[n][t + 2][2 + j] * inv * rest);
              x.w = pack2<false>(o[n][t + 3][j] * inv * rest, o[n][t + 3][2 + j] * inv * rest);
              *reinterpret_cast<uint4*>(a.out + row * D + out_d(t)) = x;
            } else {
              float4* to = reinterpret_cast<float4*>(a.part_o + (part * G + h) * D + out_d(t));
              to[0] = make_float4(o[n][t][j], o[n][t][2 + j], o[n][t + 1][j], o[n][t + 1][2 + j]);
              to[1] = make_float4(o[n][t + 2][j], o[n][t + 2][2 + j], o[n][t + 3][j],
                                  o[n][t + 3][2 + j]);
            }
          }
        }
    }
    if constexpr (PAIRS) {  // the weights of these keys, from the scores that the warp has stored
      if (a.raw != nullptr) {
        float lse2[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            lse2[n][j] = bad ? __int_as_float(0x7FFFFFFF) : m[n][j] + (log2f(l[n][j]) - kShift);
        __syncwarp();
        const int64_t pair = static_cast<int64_t>(cur.b) * a.hkv + cur.g;
        const float* raw = a.raw + pair * G * a.raw_stride;
        for (int k0 = 0; k0 < cur.len; k0 += 32) {
          const int k = k0 + lane;
          float w = 0.f;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float z = __shfl_sync(0xFFFFFFFFu, lse2[h >> 3][h & 1], (h & 7) >> 1);
            if (h < G && k < cur.len && z > -INFINITY) w += ex2(raw[h * a.raw_stride + k] - z);
          }
          if (k < cur.len)
            a.score_out[pair * a.score_stride + k] =
                (a.score_in != nullptr ? a.score_in[pair * a.score_stride + k] : 0.f) + w;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < (WARPS ? 0 : NT); ++n) {
      if (r == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s_m[warp][8 * n + 2 * q4 + j] = m[n][j];
          s_l[warp][8 * n + 2 * q4 + j] = l[n][j];
        }
      }
      if (lane == 0) s_bad[warp] = bad;
#pragma unroll
      for (int t = 0; t < C::kMT; t += 2)
#pragma unroll
        for (int j = 0; j < 2; ++j)  // 16-byte units, spread over the banks by the heads' pairs
          *reinterpret_cast<float4*>(&s_o[warp][2 * q4 + j][4 * ((out_d(t) / 4) ^ q4)]) =
              make_float4(o[n][t][j], o[n][t][2 + j], o[n][t + 1][j], o[n][t + 1][2 + j]);
      team_sync();
      const bool any_bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
      const int heads = min(FOLD ? 4 : 8, G - 8 * n);
      const int d = 4 * (threadIdx.x % (D / 4));
      for (int h = threadIdx.x / (D / 4); h < heads; h += 4 * kDecThreads / D) {
        const int hh = 8 * n + h;
        float top = s_m[0][hh];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, s_m[w][hh]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](int w, int row, float f) {
          const float4 x = *reinterpret_cast<const float4*>(&s_o[w][row][4 * ((d / 4) ^ ((row >> 1) & 3))]);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        };
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float f = s_m[w][hh] == -INFINITY ? 0.f : ex2(s_m[w][hh] - top);
          sum = fmaf(s_l[w][hh], f, sum);
          add(w, h, f);
          if constexpr (FOLD) add(w, h + 4, f);
        }
        if (any_bad) sum = __int_as_float(0x7FFFFFFF);
        const int64_t row = static_cast<int64_t>(cur.b) * a.hq + cur.g * G + hh;
        if constexpr (ONE) {  // over the ring: every warp has used its last step
          *reinterpret_cast<float4*>(&s_part[hh * D + d]) = acc;
          if (d == 0) s_pml[hh] = make_float2(top, sum);
        } else if (cur.whole) {
          *reinterpret_cast<uint2*>(a.out + row * D + d) = make_uint2(
              pack2<false>(acc.x / sum * vs, acc.y / sum * vs), pack2<false>(acc.z / sum * vs, acc.w / sum * vs));
          if (d == 0) {
            const float lse2 = top + (log2f(sum) - kShift);
            if (a.lse != nullptr) a.lse[row] = lse2 * 0.6931471805599453f;
            if (a.lse2 != nullptr) a.lse2[row] = lse2;
          }
        } else {
          *reinterpret_cast<float4*>(a.part_o + (part * G + hh) * D + d) = acc;
          if (d == 0) a.part_ml[part * G + hh] = make_float2(top, sum);
        }
      }
      if (n == 0 && threadIdx.x == 0) note(any_bad);
      team_sync();  // the shared parts may be overwritten
    }
    if constexpr (ONE) break;
    if (!more) break;
    __syncwarp();
    if (lane == 0) s_piece[warp] = nxt;
    __syncwarp();
  }
  if constexpr (ONE) {
    const Piece cur = s_piece[warp];
    constexpr bool kScaled = true;
#include "join_cluster.inc"
  }
}

// Which way (see launch_decode), both sides measured in a graph (8 KV heads, d = 128, G = 4 unless said):
//   one launch of clusters, up to four tiles a CTA: one sequence of 777 tokens 5.5 us, four of 2,000
//       7.5 and 10.9, four of 4,000 9.8 and 13.4; past the rule (eight tiles) two of 8,000 15.1 and 14.1,
//       one of 8,000 13.0 and 11.8
//   a warp per (sequence, head), up to eight steps: 181 sequences of 20-83 tokens (4 KV heads, G = 16)
//       10.3 and 20.8, 256 of 16-128 17.0 and 26.9, 256 of 200-256 26.4 and 34.9; past the rule (16 steps)
//       64 of 256-512 19.2 and 17.8, 256 of 300-512 43.7 and 45.0
//   runs of warps with 16 heads only: 100 of 300-600 36.9 and 43.3 (runs of CTAs); with fewer heads 128 of
//       300-600 33.2 and 31.3, 100 of 300-900 with weights 37.8 and 33.5, 256 of 300-512 45.3 and 46.9
template <int D, int H>
struct Fp4Kernel : Fp4Cfg<D> {
  static constexpr int kDim = D, kForm = kFp4, kPerSm = H <= 8 ? kFp4PerSm : 2, kOneTiles = 4;
  static constexpr int kPairSteps = 8, kSplitThreads = kFp4Threads<H, kSplit>;
  static constexpr float kShift = 14.f;
  static auto fn(DecMode mode) {
    if constexpr (H > 8) {
      if (mode == kWarps) return fp4_decode_kernel<D, H, kWarps>;
    }
    return mode == kOne ? fp4_decode_kernel<D, H, kOne>
           : mode == kPairs ? fp4_decode_kernel<D, H, kPairs>
                            : fp4_decode_kernel<D, H, kSplit>;
  }
};
template <int D>
cudaError_t launch_fp4_decode_t(PagedDecodeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.group <= 4) return launch_decode<Fp4Kernel<D, 4>>(a, num_sms, stream);
  if (a.group <= 8) return launch_decode<Fp4Kernel<D, 8>>(a, num_sms, stream);
  // Short sequences with 16 heads: two warps with 8 each, who both read the pages, are done sooner than
  // one where all run at once (181 sequences of 20-83 tokens, 4 KV heads, 9.4 us and 10.2; 100 of 100-256,
  // 8 KV heads, 17.5 and 18.7; past the rule, 300 of 150-256 46.9 and 36.3). The weights need all heads in
  // one warp.
  using Half = Fp4Kernel<D, 8>;
  if (a.raw == nullptr && a.max_len <= Half::kPairSteps * Half::kKeys &&
      2 * static_cast<int64_t>(a.num_seqs) * a.hkv <= kDecWarps * Half::kPerSm * num_sms &&
      !decode_in_one<Fp4Kernel<D, 16>>(a, num_sms)) {
    PagedDecodeArgs half = a;
    half.group = 8;
    half.split = 1;
    return launch_pairs<Half>(half, num_sms, stream);
  }
  return launch_decode<Fp4Kernel<D, 16>>(a, num_sms, stream);
}

}  // namespace

bool fp4_warp_runs(int group) { return group > 8; }
int fp4_decode_per_sm(int group) { return group > 8 ? 2 : kFp4PerSm; }

cudaError_t launch_fp4_decode(PagedDecodeArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  return head_dim == 128 ? launch_fp4_decode_t<128>(a, num_sms, stream)
                         : launch_fp4_decode_t<64>(a, num_sms, stream);
}

}  // namespace quail

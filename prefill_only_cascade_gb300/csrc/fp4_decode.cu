// fp4_decode.cu - attention of one new token per sequence over a paged key/value cache held in
// 4 bits. "Motor de inferência Quail atinge 1 bilhão de tokens por minuto por GPU", section
// "Como funciona", keeps anchor KV between prefills; in 4 bits 3.6 times as many anchors fit.
//
//   out = S_v sum_j w_j v_j,  w_j = exp2(c S_k q.k_j - lse2),  k_j, v_j = code * block scale
//
// How the batch is divided and joined is as over the other forms of pages (see paged.cu); a warp
// walks its keys with a running max and sum. What bounds it: 144 bytes of HBM per (token, KV head)
// at d = 128, 24 issue slots of an SM's quarter at the measured copy rate, into which 256 codes
// have to go through conversion, scaling and two products. So every step's instructions count:
//   S^T [16 keys x 8 heads]  A = K: keys fill the 16 rows (heads would fill 1 to 8 of them), half the
//            products. Lane (r, q) holds pieces q of keys r and r + 8 as they lie in memory: sums
//            over d may run in any order, so its codes ARE its fragments, and they belong to one
//            (d = 64) or two block scales.
//   O^T [16 d x 8 heads]     A = V^T: lane (r, q) holds one block (d = 64: half of one) of keys 2q, 2q + 1,
//            2q + 8, 2q + 9. Their nibbles are interleaved before the conversion (4 operations for 8
//            pairs; permuting the converted halves would take 8); B = P^T, the score fragment
//            transposed in 8 x 8 blocks. The heads of a lane's scores are those of its outputs, so
//            the running max needs no exchange while no score passes it.
// Products of code and block scale are exact in f16. Q is scaled per head by a power of two into
// f16's range (bits below 2^-38 of the head's largest |q| are lost, under fp32's own rounding); P,
// scaled by 2^14, is the sum of two f16 (22 bits, weights down to 2^-38 of the largest).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "kernels.h"
#include "paged_decode.cuh"
#include "ptx.cuh"

namespace quail {

namespace {

template <int D>
struct Fp4Cfg {
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

// Place of 16-byte piece c of V row `row`: the rows 2q of a read's lanes on different banks.
template <int D>
__device__ __forceinline__ int fp4_v_place(int row, int c) {
  return D == 128 ? (row * 4 + c) ^ (((row >> 1) & 3) << 1) : (row * 2 + c) ^ (((row >> 2) & 1) << 1);
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .b16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
               : "=r"(v)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// 16 bytes of which `real` come from global memory and the others are zeros.
__device__ __forceinline__ void copy16_part(uint32_t smem, const uint8_t* p, int real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(p), "r"(real)
               : "memory");
}
// An 8 x 8 matrix of 16-bit values, transposed: lane (r, q) gives row r's 2q, 2q + 1 and takes
// column r's.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t both(uint32_t h2, int high) {
  return __byte_perm(h2, h2, high ? 0x3232 : 0x1010);
}

template <int D, int NT, DecMode MODE>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 3 : 2)
    fp4_decode_kernel(const PagedDecodeArgs a, int cluster) {
  using C = Fp4Cfg<D>;
  constexpr bool ONE = MODE == kOne, WARPS = MODE == kWarps;
  constexpr int kTile = WARPS ? C::kKeys : C::kTile;  // keys that a run is counted in
  constexpr float kShift = 14.f;
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
  const uint32_t ring = smem_u32(dyn) + warp * (kStages * C::kStep);
  Piece ld = cur;
  const int own = WARPS ? 0 : warp * C::kKeys;  // the warp's first key in a tile
  int ld_key = ld.kb + own;              // first key of the next step to load
  bool ld_more = true;
  int page[C::kG16];                     // pages of its 16-key blocks
  uint32_t bad_steps = 0;                // bit s: a page of the step in stage s is no page
  auto seek = [&]() {                    // on to a piece that has a step for this warp
    while (ld_more && ld_key >= ld.ke) {
      ld_more = next_piece<kTile>(a, run_end, ld);
      ld_key = ld.kb + own;
    }
    if (ld_more) {
      const int32_t* table = a.table + static_cast<int64_t>(ld.b) * a.max_pages;
#pragma unroll
      for (int i = 0; i < C::kG16; ++i)
        page[i] = ld_key + 16 * i < ld.ke ? __ldg(table + ((ld_key + 16 * i) >> a.page_shift)) : 0;
    }
  };
  const int64_t head_bytes = static_cast<int64_t>(C::kCB + C::kSB) << a.page_shift;
  const int page_mask = (1 << a.page_shift) - 1;
  // lanes 0-15 copy K's block scales, 16-31 V's: 16 bytes each, of kPieceKeys keys
  constexpr int kPieceKeys = 16 / C::kSB;
  const int sc_key = (lane & 15) * kPieceKeys;
  const uint8_t* const sc_pages = lane < 16 ? a.k_pages : a.v_pages;
  auto issue = [&](int stage) {
    if (ld_more) {
      // K codes, V codes, K scales, V scales
      const uint32_t kdst = ring + stage * C::kStep, vdst = kdst + C::kCodes;
      const uint32_t sdst = kdst + 2 * C::kCodes + 16 * lane;
      bool bad = false;
      int64_t base[C::kG16];             // codes of the block's first key
      int64_t sc_at = -1;
#pragma unroll
      for (int i = 0; i < C::kG16; ++i) {
        const int pos = ld_key + 16 * i;
        const bool ok = page[i] >= 0 && page[i] < a.num_pages;
        if (pos < ld.ke && !ok) bad = true;
        const int at = pos & page_mask;
        const int64_t head = (static_cast<int64_t>(page[i]) * a.hkv + ld.g) * head_bytes;
        base[i] = pos < ld.ke && ok ? head + at * C::kCB + 16 * lane : -1;
        if ((sc_key >> 4) == i && pos < ld.ke && ok)
          sc_at = head + (static_cast<int64_t>(C::kCB) << a.page_shift) +
                  (at + (sc_key & 15)) * C::kSB;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int kPieces = C::kCB / 16;  // of a row
        const int row = lane / kPieces + j * (32 / kPieces), c = lane % kPieces;
        const int64_t at = base[j * (32 / kPieces) >> 4];
        const bool real = at >= 0 && ld_key + row < ld.ke;
        const int64_t off = real ? at + (D == 128 ? (j & 1) * 512 : 0) : 0;
        copy16(kdst + 16 * (lane + 32 * j), a.k_pages + off, real);
        copy16(vdst + 16 * fp4_v_place<D>(row, c), a.v_pages + off, real);
      }
      const int keys = sc_at >= 0 ? max(0, min(kPieceKeys, ld.ke - ld_key - sc_key)) : 0;
      copy16_part(sdst, sc_pages + (keys > 0 ? sc_at : 0), keys * C::kSB);
      bad_steps = bad ? bad_steps | (1u << stage) : bad_steps & ~(1u << stage);
      ld_key += kTile;
      seek();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // Q of a piece as it is in memory: the D / 4 values from d = q4 D / 4 of head r (+ 8)
  uint4 qraw[NT][D / 32];
  auto load_q = [&](int b, int g) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = r + 8 * n;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(b) * a.q_stride + static_cast<int64_t>(g * G + h) * D +
          q4 * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        qraw[n][i] = h < G ? __ldg(qp + i) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  seek();
  load_q(cur.b, cur.g);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  int stage = 0;

  while (true) {
    // ---------------------------------------------------- one piece
    uint32_t qb[NT][C::kQS][2];
    float c_log2[NT][2];                 // of heads 2 q4, 2 q4 + 1 (+ 8 n)
    {
      const float ks = __ldg(a.k_scale + static_cast<int64_t>(cur.b) * a.hkv + cur.g);
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

    for (int key0 = cur.kb + own; key0 < cur.ke; key0 += kTile) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // every lane's copies are there, and the stage before was read
      bad |= (bad_steps >> stage) & 1u;
      issue(stage == 0 ? kStages - 1 : stage - 1);
      const uint32_t kbuf = ring + stage * C::kStep, vbuf = kbuf + C::kCodes;
      const uint32_t ksc = kbuf + 2 * C::kCodes, vsc = ksc + C::kScales;
      stage = stage == kStages - 1 ? 0 : stage + 1;

      // ---- scores of this step's keys: s[i][n] = keys r, r + 8 of block i by heads 2 q4, + 1
      float s[C::kG16][NT][4];
#pragma unroll
      for (int i = 0; i < C::kG16; ++i) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.f;
        uint32_t w[2][D / 32], sc[2][D / 64];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = 16 * i + 8 * u + r;
          if constexpr (D == 128) {
            const uint4 x = ld_shared16(kbuf + key * C::kCB + 16 * q4);
            w[u][0] = x.x;
            w[u][1] = x.y;
            w[u][2] = x.z;
            w[u][3] = x.w;
            const uint32_t h2 = e4m3_lo(ld_shared_u16(ksc + key * C::kSB + 2 * q4));
            sc[u][0] = both(h2, 0);
            sc[u][1] = both(h2, 1);
          } else {
            const uint2 x = ld_shared8(kbuf + key * C::kCB + 8 * q4);
            w[u][0] = x.x;
            w[u][1] = x.y;
            sc[u][0] = both(e4m3_lo(ld_shared_u8(ksc + key * C::kSB + q4)), 0);
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {  // 8 codes of each key: two k-steps
          uint32_t x[4], y[4];
          e2m1x8(w[0][j], x);
          e2m1x8(w[1][j], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] = mul_f16x2(x[k], sc[0][j >> 1]);
            y[k] = mul_f16x2(y[k], sc[1][j >> 1]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816<true>(s[i][n], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1],
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
      if (key0 + C::kKeys > cur.ke) {
#pragma unroll
        for (int i = 0; i < C::kG16; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (key0 + 16 * i + 8 * u + r >= cur.ke) {
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
                  a.raw + (static_cast<int64_t>(cur.b) * a.hq + cur.g * G + h) * a.raw_stride;
#pragma unroll
              for (int i = 0; i < C::kG16; ++i) {  // rows are padded to whole tiles
                row[key0 + 16 * i + r] = s[i][n][j];
                row[key0 + 16 * i + 8 + r] = s[i][n][2 + j];
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
        uint32_t ps[NT][2][2];           // [head tile][f16 term][8 keys]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x0 = ex2(s[i][n][2 * u] - ref[n][0]), x1 = ex2(s[i][n][2 * u + 1] - ref[n][1]);
            l[n][0] += x0;
            l[n][1] += x1;
            uint32_t hi, lo;
            split_f16(x0, x1, hi, lo);
            ps[n][0][u] = transpose8(hi);
            ps[n][1][u] = transpose8(lo);
          }
        uint32_t w[4][C::kWords], sb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 16 * i + 2 * q4 + (j & 1) + 8 * (j >> 1);
          if constexpr (D == 128) {
            const uint2 x = ld_shared8(vbuf + 16 * fp4_v_place<D>(row, r >> 1) + 8 * (r & 1));
            w[j][0] = x.x;
            w[j][1] = x.y;
            sb[j] = ld_shared_u8(vsc + row * C::kSB + r);
          } else {
            w[j][0] = ld_shared4(vbuf + 16 * fp4_v_place<D>(row, r >> 2) + 4 * (r & 3));
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
            const uint32_t f0 = mul_f16x2(a0[b], sc0), f1 = mul_f16x2(a1[b], sc0);
            const uint32_t f2 = mul_f16x2(a2[b], sc1), f3 = mul_f16x2(a3[b], sc1);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<true>(o[n][4 * k + b], f0, f1, f2, f3, ps[n][t][0], ps[n][t][1]);
          }
        }
      }
    }

    // the next piece's queries are on their way while this one is put together
    Piece nxt = cur;
    const bool more = !ONE && next_piece<kTile>(a, run_end, nxt);
    if (more) load_q(nxt.b, nxt.g);

    // ---------------------------------------------------- the four warps' parts together
    const float vs = __ldg(a.v_scale + static_cast<int64_t>(cur.b) * a.hkv + cur.g);
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
    // d of tile t's row r; row r + 8 is the next d
    auto out_d = [&](int t) { return r * (D / 8) + 2 * t; };
    if constexpr (WARPS) {
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
              if (a.lse2 != nullptr) a.lse2[row] = lse2;
            } else {
              a.part_ml[part * G + h] = make_float2(m[n][j], sum);
            }
          }
          const float inv = vs / sum;
#pragma unroll
          for (int t = 0; t < C::kMT; t += 4) {  // eight neighbouring d
            if (cur.whole) {
              uint4 x;
              x.x = pack2<false>(o[n][t][j] * inv, o[n][t][2 + j] * inv);
              x.y = pack2<false>(o[n][t + 1][j] * inv, o[n][t + 1][2 + j] * inv);
              x.z = pack2<false>(o[n][t + 2][j] * inv, o[n][t + 2][2 + j] * inv);
              x.w = pack2<false>(o[n][t + 3][j] * inv, o[n][t + 3][2 + j] * inv);
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
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(&s_o[warp][2 * q4 + j][out_d(t)]) =
              make_float4(o[n][t][j], o[n][t][2 + j], o[n][t + 1][j], o[n][t + 1][2 + j]);
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
            const float lse2 = top + (log2f(sum) - kShift);
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

  if constexpr (ONE) join_cluster<D>(a, cur, cluster, cta, s_part, s_pml, s_lse2, kShift, true);
}

template <int D, int NT>
struct Fp4Kernel : Fp4Cfg<D> {
  static constexpr int kDim = D, kPerSm = NT == 1 ? 3 : 2, kOneTiles = 8;
  static constexpr float kShift = 14.f;
  static auto fn(DecMode mode) {
    return mode == kOne ? fp4_decode_kernel<D, NT, kOne>
           : mode == kWarps ? fp4_decode_kernel<D, NT, kWarps>
                            : fp4_decode_kernel<D, NT, kSplit>;
  }
};

}  // namespace

int fp4_decode_per_sm(int group) { return group > 8 ? 2 : 3; }

cudaError_t launch_fp4_decode(PagedDecodeArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  const bool two = a.group > 8;
  if (head_dim == 128)
    return two ? launch_decode<Fp4Kernel<128, 2>>(a, num_sms, stream)
               : launch_decode<Fp4Kernel<128, 1>>(a, num_sms, stream);
  return two ? launch_decode<Fp4Kernel<64, 2>>(a, num_sms, stream)
             : launch_decode<Fp4Kernel<64, 1>>(a, num_sms, stream);
}

}  // namespace quail

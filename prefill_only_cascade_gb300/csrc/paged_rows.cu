// paged_rows.cu - token rows of a paged key/value cache: quantised to 4 bits as they are
// written, and read back as dense bf16 rows from pages of every form. "Motor de inferência
// Quail atinge 1 bilhão de tokens por minuto por GPU", section "Como funciona", keeps anchor
// KV between prefills; in 4 bits 3.6 times as many anchors fit, and the rows come back where
// a cascade over dense anchors, or the weights of a window of queries, wants them.
//
// The 4-bit form (fp4 pages): blocks of 16 values of one (token, KV head) share an e4m3 scale,
// and a sequence's head shares an fp32 scale S:
//   t = max|x| / (6 S)   (6 S and the quotient rounded to fp32)
//   b = e4m3(t)          nearest, ties to even, at most 448 in size; NaN if the block holds one
//   code = e2m1(x / (b S))  (b S and the quotient rounded to fp32) nearest, ties to even, at
//                        most 6 in size; 0 in a block whose scale is 0 or NaN
//   value = code b S
// e2m1's values are 0, 0.5, 1, 1.5, 2, 3, 4, 6: products with an e4m3 number are exact in f16.
// A page is [Hkv][codes of page_size tokens, d / 2 bytes each | their block scales, d / 16
// bytes each]: a head's tokens follow one another, so that the attention reads whole lines.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace quail {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowMaxTok = 16;  // most tokens of a block
constexpr int kAppendPerSm = 6;  // blocks on an SM: with four 96 prompts took 223 us, read back too, with six 207

// Slot of each of the block's token rows in the pool (page * page_size + place), kNoSlot where
// its position or page is out of range, kNoSeq where no sequence holds it; and its sequence.
constexpr int64_t kNoSlot = -1, kNoSeq = -2;

__device__ __forceinline__ void find_slots(const PagedRows& p, int64_t t0, int n, int64_t* s_slot,
                                           int* s_seq) {
  for (int k = threadIdx.x; k < n; k += kRowThreads) {
    const int64_t t = t0 + k;
    int b = static_cast<int>(t);
    int64_t i = 0, slot = kNoSeq;
    bool ok = true;
    if (p.offsets != nullptr) {
      int lo = 0, hi = p.num_seqs;  // the last sequence that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.offsets[mid] <= t) lo = mid; else hi = mid;
      }
      b = lo;
      const int64_t o0 = p.offsets[b];
      i = t - o0;
      ok = o0 <= t && t < p.offsets[b + 1];
    }
    if (ok) {
      slot = kNoSlot;
      const int64_t start = p.start_pos[b];
      const int64_t pos = start + i;
      if (start >= 0 && pos < p.max_len) {
        const int page = p.table[static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift)];
        if (page >= 0 && page < p.num_pages)
          slot = (static_cast<int64_t>(page) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
      }
    }
    if (slot < 0) atomicOr(p.err_word, kErrDeviceBounds);
    s_slot[k] = slot;
    s_seq[k] = b;
  }
  // the offsets as a whole: increasing from 0 to the number of rows
  if (blockIdx.x == 0 && p.offsets != nullptr) {
    for (int b = threadIdx.x; b <= p.num_seqs; b += kRowThreads) {
      const int64_t o = p.offsets[b];
      const int64_t next = b < p.num_seqs ? p.offsets[b + 1] : p.total;
      if ((b == 0 && o != 0) || (b < p.num_seqs ? next < o : next != o))
        atomicOr(p.err_word, kErrDeviceBounds);
    }
  }
  __syncthreads();
}

// Byte offsets in an fp4 pool of a block's 8 bytes of codes and of its scale.
__device__ __forceinline__ void fp4_place(const PagedRows& p, int D, int64_t slot, int g, int blk,
                                          int64_t& code, int64_t& scale) {
  const int64_t page = slot >> p.page_shift;
  const int at = static_cast<int>(slot & ((1 << p.page_shift) - 1));
  const int64_t head = (page * p.hkv + g) * (static_cast<int64_t>(D / 2 + D / 16) << p.page_shift);
  code = head + static_cast<int64_t>(at) * (D / 2) + 8 * blk;
  scale = head + (static_cast<int64_t>(D / 2) << p.page_shift) + at * (D / 16) + blk;
}

// Eight fp32 -> eight e2m1 codes, x[0] in the low bits.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\tmov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ float rcp_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The codes of a block as the definition has them: an IEEE division per value.
__device__ __noinline__ uint2 divide_block(uint4 lo, uint4 hi, float D) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t v = w[4 * h + k / 2];
      x[k] = __fdiv_rn(__uint_as_float(k & 1 ? v & 0xFFFF0000u : v << 16), D);
      if (x[k] != x[k]) x[k] = 0.f;  // 0 / 0
    }
    c[h] = e2m1x8_of(x);
  }
  return make_uint2(c[0], c[1]);
}

// A block of 16 bf16 values under S: its codes and its scale. r6 is about 1 / (6 S); `plain` says that
// S and 6 S are ordinary numbers (2^-60 to 2^60).
// Quotients are taken as products with a reciprocal, a few units in the last place from the
// definition's. That matters where a quotient is next to a border between two codes, and there the
// definition's own divisions are made:
//   the scale   fp32 bits of t whose low 20 (e4m3 keeps 3 of 23) are within 8 of a half step
//   the codes   the borders are odd multiples m = 1, 3, 5, 7 of powers of two; a bf16 x can be within
//               16 units of m D only where the last 16 bits of m D are: D decides for the whole block
// Random scales send one block in 500 there, scales that are powers of two all of them.
// (Divisions everywhere, by one FMA correction each: 186 us for 96 prompts of 128-2,048 tokens, 8
// heads, d = 128; this way 100, with 64 tokens per block and five blocks an SM 125.)
__device__ __forceinline__ void encode_block(const uint4& lo, const uint4& hi, float S, float r6, bool plain,
                                             uint2& codes, uint8_t& scale) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = absmax_bf16x2(top, w[k]);  // a NaN is above all numbers
  const float amax = absmax_bf16x2_value(top);
  float t = amax * r6;
  bool near = !plain || t < 0.015625f ||  // e4m3 has fewer bits below 2^-6
              ((__float_as_uint(t) + 8 - 0x80000u) & 0xFFFFFu) < 16u;
  if (near) t = __fdiv_rn(amax, __fmul_rn(6.f, S));
  scale = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  const uint32_t h2 = e4m3_lo(scale);
  const float b = __low2float(*reinterpret_cast<const __half2*>(&h2));
  const float D = __fmul_rn(b, S);
  codes = make_uint2(0u, 0u);
  if (!(fabsf(b) > 0.f)) return;
  auto off = [&](float m) { return (__float_as_uint(m * D) + 16u) & 0xFFFFu; };
  if (!plain || min(min(off(1.f), off(3.f)), min(off(5.f), off(7.f))) < 32u) {
    codes = divide_block(lo, hi, D);
    return;
  }
  const float r = rcp_near(D);
  float x[2][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[k >> 2][2 * (k & 3)] = __uint_as_float(w[k] << 16) * r;
    x[k >> 2][2 * (k & 3) + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * r;
  }
  codes = make_uint2(e2m1x8_of(x[0]), e2m1x8_of(x[1]));
}

// Bound by HBM: 2 bytes read and 0.5625 written per value. A warp takes 32 blocks: the blocks
// of one KV head in 4 (d = 128) or 8 tokens, which are whole sectors on both sides. The next K rows
// are on their way while V's are encoded, the first while the slots are looked up.
template <int D>
__global__ void __launch_bounds__(kRowThreads, kAppendPerSm) fp4_append_kernel(const PagedRows p, int tok) {
  __shared__ int64_t s_slot[kRowMaxTok];
  __shared__ int s_seq[kRowMaxTok];
  constexpr int kBlocks = D / 16, kGroup = 32 / kBlocks;
  after_stream();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int n = static_cast<int>(min(static_cast<int64_t>(tok), p.total - t0));
  const int lane = threadIdx.x & 31, blk = lane % kBlocks;
  const int pairs = (n + kGroup - 1) / kGroup * p.hkv;
  const int warp = threadIdx.x >> 5, heads_on = kRowWarps % p.hkv, groups_on = kRowWarps / p.hkv;
  int g = warp % p.hkv, t = warp / p.hkv * kGroup + lane / kBlocks, u = warp;
  uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0;
  auto load_k = [&]() {
    if (t >= n) return;
    const uint4* x = reinterpret_cast<const uint4*>(p.k_new + (t0 + t) * p.k_stride + g * D + 16 * blk);
    k0 = x[0];
    k1 = x[1];
  };
  load_k();
  find_slots(p, t0, n, s_slot, s_seq);
  while (u < pairs) {
    const int64_t slot = t < n ? s_slot[t] : kNoSlot;
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
    float sk = 1.f, sv = 1.f;
    int64_t code, scale;
    if (slot >= 0) {
      const uint4* x = reinterpret_cast<const uint4*>(p.v_new + (t0 + t) * p.v_stride + g * D + 16 * blk);
      v0 = x[0];
      v1 = x[1];
      const int64_t sc = static_cast<int64_t>(s_seq[t]) * p.hkv + g;
      sk = p.k_scale[sc];
      sv = p.v_scale[sc];
      fp4_place(p, D, slot, g, blk, code, scale);
    }
    auto ordinary = [](float S) { return S >= 8.673617379884035e-19f && S <= 1.152921504606847e18f; };
    uint2 c;
    uint8_t b;
    encode_block(k0, k1, sk, rcp_near(6.f * sk), ordinary(sk), c, b);
    if (slot >= 0) {
      *reinterpret_cast<uint2*>(p.k_pages + code) = c;
      p.k_pages[scale] = b;
    }
    u += kRowWarps;
    g += heads_on;
    t += groups_on * kGroup;
    if (g >= p.hkv) {
      g -= p.hkv;
      t += kGroup;
    }
    load_k();
    encode_block(v0, v1, sv, rcp_near(6.f * sv), ordinary(sv), c, b);
    if (slot >= 0) {
      *reinterpret_cast<uint2*>(p.v_pages + code) = c;
      p.v_pages[scale] = b;
    }
  }
}

// Sixteen values of one (token, KV head) as the cache holds them -> bf16: code times block scale
// (exact in f16), times S in fp32, rounded to bf16.
template <int D, KvForm F>
struct Held {
  uint4 a, b;  // bf16: the values; e4m3: a, the codes; fp4: a.x and a.y, the codes, a.z the scale
  __device__ __forceinline__ void load(const PagedRows& p, const uint8_t* pages, int64_t slot, int g,
                                       int blk) {
    if constexpr (F == kFp4) {
      int64_t code, scale;
      fp4_place(p, D, slot, g, blk, code, scale);
      const uint2 x = *reinterpret_cast<const uint2*>(pages + code);
      a = make_uint4(x.x, x.y, pages[scale], 0u);
    } else {
      const uint4* x = reinterpret_cast<const uint4*>(
          pages + (F == kBf16 ? 2 : 1) * ((slot * p.hkv + g) * D + 16 * blk));
      a = x[0];
      if constexpr (F == kBf16) b = x[1];
    }
  }
  __device__ __forceinline__ void decode(float S) {
    if constexpr (F != kBf16) {
      uint32_t h[8];
      if constexpr (F == kFp4) {
        uint32_t x[4];
        const uint32_t s = e4m3_lo(__byte_perm(a.z, a.z, 0x0000));
        e2m1x8(a.x, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = mul_f16x2(x[k], s);
        e2m1x8(a.y, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[4 + k] = mul_f16x2(x[k], s);
      } else {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) h[2 * k] = e4m3_lo(w[k]), h[2 * k + 1] = e4m3_hi(w[k]);
      }
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        o[k] = pack_bf16x2(__fmul_rn(f.x, S), __fmul_rn(f.y, S));
      }
      a = make_uint4(o[0], o[1], o[2], o[3]);
      b = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
};

// Bound by HBM: 0.5625, 1 or 2 bytes read and 2 written per value; a warp takes the same 32
// blocks as when they were written.
template <int D, KvForm F>
__global__ void __launch_bounds__(kRowThreads) paged_read_kernel(const PagedRows p, int tok) {
  __shared__ int64_t s_slot[kRowMaxTok];
  __shared__ int s_seq[kRowMaxTok];
  constexpr int kBlocks = D / 16, kGroup = 32 / kBlocks;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int n = static_cast<int>(min(static_cast<int64_t>(tok), p.total - t0));
  after_stream();
  find_slots(p, t0, n, s_slot, s_seq);
  const int lane = threadIdx.x & 31, blk = lane % kBlocks;
  const int pairs = (n + kGroup - 1) / kGroup * p.hkv;
  const int warp = threadIdx.x >> 5, heads_on = kRowWarps % p.hkv, groups_on = kRowWarps / p.hkv;
  int group = warp / p.hkv, g = warp % p.hkv;
  for (int u = warp; u < pairs; u += kRowWarps, group += groups_on, g += heads_on) {
    if (g >= p.hkv) {
      g -= p.hkv;
      ++group;
    }
    const int t = group * kGroup + lane / kBlocks;
    const int64_t slot = t < n ? s_slot[t] : kNoSeq;
    if (slot == kNoSeq) continue;
    const int64_t sc = static_cast<int64_t>(s_seq[t]) * p.hkv + g;
    const int col = g * D + 16 * blk;
    Held<D, F> k, v;
    const uint32_t nan = 0x7FFF7FFFu;
    k.a = k.b = v.a = v.b = make_uint4(nan, nan, nan, nan);
    if (slot >= 0) {
      if (p.k_out != nullptr) k.load(p, p.k_pages, slot, g, blk);
      if (p.v_out != nullptr) v.load(p, p.v_pages, slot, g, blk);
      k.decode(F == kBf16 || p.k_out == nullptr ? 1.f : p.k_scale[sc]);
      v.decode(F == kBf16 || p.v_out == nullptr ? 1.f : p.v_scale[sc]);
    }
    if (p.k_out != nullptr) {
      uint4* to = reinterpret_cast<uint4*>(p.k_out + (t0 + t) * p.k_stride + col);
      to[0] = k.a;
      to[1] = k.b;
    }
    if (p.v_out != nullptr) {
      uint4* to = reinterpret_cast<uint4*>(p.v_out + (t0 + t) * p.v_stride + col);
      to[0] = v.a;
      to[1] = v.b;
    }
  }
}

// Token rows per block: 16 where there are enough (64 x 4,096 rows of 8 heads read back 213 us; 64 a
// block 220, 8 a block 230), fewer so that two blocks per SM have some.
int tokens_per_block(int64_t total, int num_sms) {
  const int64_t spread = (total + 2 * num_sms - 1) / (2 * num_sms);
  return static_cast<int>(spread < 1 ? 1 : spread < kRowMaxTok ? spread : kRowMaxTok);
}

}  // namespace

cudaError_t launch_fp4_append(const PagedRows& p, int head_dim, int num_sms, cudaStream_t stream) {
  const int tok = tokens_per_block(p.total, num_sms);
  const unsigned blocks = static_cast<unsigned>((p.total + tok - 1) / tok);
  return launch_early(head_dim == 128 ? fp4_append_kernel<128> : fp4_append_kernel<64>, dim3(blocks),
                      dim3(kRowThreads), 0, stream, 0, p, tok);
}

cudaError_t launch_paged_read(const PagedRows& p, int head_dim, int kv_dtype, int num_sms,
                              cudaStream_t stream) {
  const int tok = tokens_per_block(p.total, num_sms);
  const unsigned blocks = static_cast<unsigned>((p.total + tok - 1) / tok);
  const auto fn = head_dim == 128
                      ? (kv_dtype == kFp4 ? paged_read_kernel<128, kFp4>
                         : kv_dtype == kE4m3 ? paged_read_kernel<128, kE4m3> : paged_read_kernel<128, kBf16>)
                      : (kv_dtype == kFp4 ? paged_read_kernel<64, kFp4>
                         : kv_dtype == kE4m3 ? paged_read_kernel<64, kE4m3> : paged_read_kernel<64, kBf16>);
  return launch_early(fn, dim3(blocks), dim3(kRowThreads), 0, stream, 0, p, tok);
}

}  // namespace quail

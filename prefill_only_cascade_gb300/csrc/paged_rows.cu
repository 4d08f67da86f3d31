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
constexpr int kRowMaxTok = 64;

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
        if (__ldg(p.offsets + mid) <= t) lo = mid; else hi = mid;
      }
      b = lo;
      const int64_t o0 = __ldg(p.offsets + b);
      i = t - o0;
      ok = o0 <= t && t < __ldg(p.offsets + b + 1);
    }
    if (ok) {
      slot = kNoSlot;
      const int64_t start = __ldg(p.start_pos + b);
      const int64_t pos = start + i;
      if (start >= 0 && pos < p.max_len) {
        const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift));
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
      const int64_t o = __ldg(p.offsets + b);
      const int64_t next = b < p.num_seqs ? __ldg(p.offsets + b + 1) : p.total;
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

// Two fp32 -> two e2m1 codes in a byte, x0 in the low bits.
__device__ __forceinline__ uint32_t e2m1x2(float x0, float x1) {
  uint16_t r;
  asm("{\n\t.reg .b8 b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b16 %0, {b, 0};\n\t}"
      : "=h"(r)
      : "f"(x0), "f"(x1));
  return r;
}

// A block of 16 bf16 values under S: its codes and its scale.
__device__ __forceinline__ void encode_block(const uint4& lo, const uint4& hi, float S, uint2& codes,
                                             uint8_t& scale) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = absmax_bf16x2(top, w[k]);  // a NaN is above all numbers
  const float amax = absmax_bf16x2_value(top);
  scale = __nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(6.f, S)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t h2 = e4m3_lo(scale);
  const float b = __low2float(*reinterpret_cast<const __half2*>(&h2));
  const float D = __fmul_rn(b, S);
  codes = make_uint2(0u, 0u);
  if (!(fabsf(b) > 0.f)) return;
  // The IEEE quotient x / D for an ordinary D is RN(x r) with one FMA correction by its exact
  // residual (Markstein, "IA-64 and Elementary Functions", 2000), wherever a code can be other
  // than zero; an infinite one has no residual.
  const bool plain = D >= 8.673617379884035e-19f && D <= 1.152921504606847e18f;  // 2^-60, 2^60
  const float r = __frcp_rn(D);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float x[2] = {__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (plain) {
        const float q = x[j] * r;
        const float c = fmaf(fmaf(-q, D, x[j]), r, q);
        x[j] = fabsf(q) < 1e30f ? copysignf(c, x[j]) : q;
      } else {
        x[j] = __fdiv_rn(x[j], D);
        if (x[j] != x[j]) x[j] = 0.f;  // 0 / 0
      }
    }
    const uint32_t two = e2m1x2(x[0], x[1]) << (8 * (k & 3));
    if (k < 4) codes.x |= two; else codes.y |= two;
  }
}

// Bound by HBM: 2 bytes read and 0.5625 written per value. A warp takes 32 blocks: the blocks
// of one KV head in 4 (d = 128) or 8 tokens, which are whole sectors on both sides.
template <int D>
__global__ void __launch_bounds__(kRowThreads) fp4_append_kernel(const PagedRows p, int tok) {
  __shared__ int64_t s_slot[kRowMaxTok];
  __shared__ int s_seq[kRowMaxTok];
  constexpr int kBlocks = D / 16, kGroup = 32 / kBlocks;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int n = static_cast<int>(min(static_cast<int64_t>(tok), p.total - t0));
  find_slots(p, t0, n, s_slot, s_seq);
  const int lane = threadIdx.x & 31, blk = lane % kBlocks;
  const int pairs = (n + kGroup - 1) / kGroup * p.hkv;
  for (int u = threadIdx.x >> 5; u < pairs; u += kRowWarps) {
    const int group = u / p.hkv, g = u - group * p.hkv;
    const int t = group * kGroup + lane / kBlocks;
    const int64_t slot = t < n ? s_slot[t] : kNoSlot;
    if (slot < 0) continue;
    const int col = g * D + 16 * blk;
    const uint4* ks = reinterpret_cast<const uint4*>(p.k_new + (t0 + t) * p.k_stride + col);
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + (t0 + t) * p.v_stride + col);
    const uint4 k0 = __ldg(ks), k1 = __ldg(ks + 1), v0 = __ldg(vs), v1 = __ldg(vs + 1);
    const int64_t sc = static_cast<int64_t>(s_seq[t]) * p.hkv + g;
    int64_t code, scale;
    fp4_place(p, D, slot, g, blk, code, scale);
    uint2 c;
    uint8_t b;
    encode_block(k0, k1, __ldg(p.k_scale + sc), c, b);
    *reinterpret_cast<uint2*>(p.k_pages + code) = c;
    p.k_pages[scale] = b;
    encode_block(v0, v1, __ldg(p.v_scale + sc), c, b);
    *reinterpret_cast<uint2*>(p.v_pages + code) = c;
    p.v_pages[scale] = b;
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
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(pages + code));
      a = make_uint4(x.x, x.y, __ldg(pages + scale), 0u);
    } else {
      const uint4* x = reinterpret_cast<const uint4*>(
          pages + (F == kBf16 ? 2 : 1) * ((slot * p.hkv + g) * D + 16 * blk));
      a = __ldg(x);
      if constexpr (F == kBf16) b = __ldg(x + 1);
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
  find_slots(p, t0, n, s_slot, s_seq);
  const int lane = threadIdx.x & 31, blk = lane % kBlocks;
  const int pairs = (n + kGroup - 1) / kGroup * p.hkv;
  for (int u = threadIdx.x >> 5; u < pairs; u += kRowWarps) {
    const int group = u / p.hkv, g = u - group * p.hkv;
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
      k.decode(F == kBf16 || p.k_out == nullptr ? 1.f : __ldg(p.k_scale + sc));
      v.decode(F == kBf16 || p.v_out == nullptr ? 1.f : __ldg(p.v_scale + sc));
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

// Token rows per block: 64 where there are enough, fewer so that two blocks per SM have some.
int tokens_per_block(int64_t total, int num_sms) {
  const int64_t spread = (total + 2 * num_sms - 1) / (2 * num_sms);
  return static_cast<int>(spread < 1 ? 1 : spread < kRowMaxTok ? spread : kRowMaxTok);
}

}  // namespace

cudaError_t launch_fp4_append(const PagedRows& p, int head_dim, int num_sms, cudaStream_t stream) {
  const int tok = tokens_per_block(p.total, num_sms);
  const unsigned blocks = static_cast<unsigned>((p.total + tok - 1) / tok);
  if (head_dim == 128)
    fp4_append_kernel<128><<<blocks, kRowThreads, 0, stream>>>(p, tok);
  else
    fp4_append_kernel<64><<<blocks, kRowThreads, 0, stream>>>(p, tok);
  return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedRows& p, int head_dim, int kv_dtype, int num_sms,
                              cudaStream_t stream) {
  const int tok = tokens_per_block(p.total, num_sms);
  const unsigned blocks = static_cast<unsigned>((p.total + tok - 1) / tok);
  auto run = [&](auto kernel) { kernel<<<blocks, kRowThreads, 0, stream>>>(p, tok); };
  if (head_dim == 128)
    run(kv_dtype == kFp4 ? paged_read_kernel<128, kFp4>
        : kv_dtype == kE4m3 ? paged_read_kernel<128, kE4m3> : paged_read_kernel<128, kBf16>);
  else
    run(kv_dtype == kFp4 ? paged_read_kernel<64, kFp4>
        : kv_dtype == kE4m3 ? paged_read_kernel<64, kE4m3> : paged_read_kernel<64, kBf16>);
  return cudaGetLastError();
}

}  // namespace quail

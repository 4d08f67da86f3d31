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
#include "paged_decode.cuh"
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

}  // namespace

int decode_tile_keys(int head_dim, int kv_dtype) {
  if (kv_dtype == kFp4) return DecCfg<128, kFp4>::kTile;  // the same for 64
  if (head_dim == 128) return kv_dtype == kE4m3 ? DecCfg<128, kE4m3>::kTile : DecCfg<128, kBf16>::kTile;
  return kv_dtype == kE4m3 ? DecCfg<64, kE4m3>::kTile : DecCfg<64, kBf16>::kTile;
}

int decode_ctas_per_sm(int kv_dtype) {
  return kv_dtype == kFp4 ? DecCfg<128, kFp4>::kPerSm : DecCfg<128, kBf16>::kPerSm;
}

// Where a CTA has several short pieces in its run, putting its warps' parts together is what
// takes the time (8 us a piece). Measured against runs of CTAs: 181 sequences of 20-83 tokens
// (8 KV heads, G = 16, e4m3) 27.0 us and 40.8, 256 of 16-128 (8, G = 4) 29.2 and 38.7, 100 of
// 100-500 (8, G = 8) 33.6 and 39.8, 128 of 300-600 (8, G = 4, e4m3) 35.0 and 37.8; past the rule,
// 93 of 431-589 43.9 and 41.9, 128 of 500-1,000 73.6 and 70.7 (parts of more runs to join).
bool decode_by_warps(int num_seqs, int hkv, int max_len, int tile) {
  return static_cast<int64_t>(num_seqs) * hkv >= 4 * kDecodeMaxSms && max_len <= 8 * tile;
}

int decode_ctas(int num_sms, int per_sm, int num_seqs, int hkv, int max_len, int tile) {
  const int64_t most = static_cast<int64_t>(num_seqs) * hkv * ((max_len + tile - 1) / tile);
  const int64_t full = static_cast<int64_t>(num_sms < kDecodeMaxSms ? num_sms : kDecodeMaxSms) * per_sm;
  return static_cast<int>(most < 1 ? 1 : most < full ? most : full);
}

cudaError_t launch_paged_decode(PagedDecodeArgs& a, int head_dim, int kv_dtype, int num_sms,
                                cudaStream_t stream) {
  if (kv_dtype == kFp4) return launch_paged_decode_fp4(a, head_dim, num_sms, stream);
  const bool two = a.group > 8, fp8 = kv_dtype == kE4m3;
  if (head_dim == 128) {
    if (fp8) return two ? launch_decode_t<128, kE4m3, 2>(a, num_sms, stream)
                        : launch_decode_t<128, kE4m3, 1>(a, num_sms, stream);
    return two ? launch_decode_t<128, kBf16, 2>(a, num_sms, stream)
               : launch_decode_t<128, kBf16, 1>(a, num_sms, stream);
  }
  if (fp8) return two ? launch_decode_t<64, kE4m3, 2>(a, num_sms, stream)
                      : launch_decode_t<64, kE4m3, 1>(a, num_sms, stream);
  return two ? launch_decode_t<64, kBf16, 2>(a, num_sms, stream)
             : launch_decode_t<64, kBf16, 1>(a, num_sms, stream);
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

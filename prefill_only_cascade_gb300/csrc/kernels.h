// kernels.h - internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "quail.h"

namespace quail {

// Status (a quail_status value) of the current device for the library: QUAIL_OK on a
// GB300 after the one-time set-up, else the same code every entry point returns.
int current_device_status();

struct HeadArgs {
  int64_t n_rows;
  int hidden;
  float eps;
  const void* h;
  int64_t h_rows;
  int64_t h_row_stride;
  const int32_t* row_index;
  const void* gamma;
  const void* w8;
  float* logits;
  int32_t* argmax;
  unsigned* err_word;  // the library's device error word (bounds failures)
};
size_t restricted_head_smem_bytes(int hidden);
cudaError_t launch_restricted_head(const HeadArgs& a, int num_sms, cudaStream_t stream);

struct QuantArgs {
  int num_anchors;
  const int32_t* anchor_offsets;
  int64_t total_tokens;
  int num_kv_heads;
  int head_dim;
  const void* kv;
  void* codes;
  float* scale;
  CUtensorMap map;     // 2-D bf16 map over kv [T_A, Hkv * d], box (hg * d, 32 rows)
  unsigned* err_word;
  uint64_t timeout_ns;
};
// Heads per slab of the quantiser (the tensor map's box is hg * d wide).
int quantize_heads_per_slab(int num_kv_heads, int head_dim);
cudaError_t launch_quantize_kv_fp8(const QuantArgs& q, int num_sms, cudaStream_t stream);
// With the amax of every (anchor, KV head) given ([A, Hkv] fp32, device).
cudaError_t launch_quantize_kv_fp8_scaled(const QuantArgs& q, const float* amax, int num_sms,
                                          cudaStream_t stream);

struct JoinSelectArgs {
  int num_anchors;
  int64_t num_suffixes;
  const int32_t* anchor_suffix_ptr;
  const int32_t* argmax;
  int32_t true_index;
  uint8_t* verdict;
  int32_t* selected;
  int32_t* num_selected;
  int32_t* anchor_count;
  int32_t* chunk_work;  // workspace: one int32 per chunk of suffixes
};
size_t join_select_workspace_bytes(int64_t num_suffixes);
cudaError_t launch_join_select(const JoinSelectArgs& j, cudaStream_t stream);

// Everything the cascade kernels need besides the tensor maps.
struct CascadeParams {
  int num_anchors, num_suffixes;
  int64_t total_anchor_tokens, total_suffix_tokens;
  int max_anchor_len, max_suffix_len;
  int hq, hkv, group;        // group = hq / hkv
  int tok_per_tile;          // 128 / group suffix tokens per 128-row query tile
  int item_bound;            // host-known upper bound of work items
  float scale_log2;          // softmax_scale * log2(e)
  bool fp8;
  const int32_t* anchor_offsets;
  const int32_t* anchor_suffix_ptr;
  const int32_t* suffix_offsets;
  const float* k_scale;
  const float* v_scale;
  const void* q_suf;
  const void* k_anc;         // bf16, or e4m3 codes with FP8 anchor KV
  const void* v_anc;
  const void* k_suf;
  const void* v_suf;
  void* out;
  float* lse;
  // workspace (see cascade_workspace_layout)
  int32_t* flag;             // nonzero: a suffix offset check failed
  int32_t* prefix;           // [A+1] work-item prefix over the anchor order; [A] = total
  int32_t* order;            // [A] anchors by decreasing anchor-tile count
  int32_t* seg;              // [T_S] first token of the suffix that holds each token
  int32_t* items;            // [item_bound][12] one record per work item (8 or 12 ints)
  int32_t* redo_count;       // items the speculative kernel handed to the exact one
  int32_t* redo_flag;        // [item_bound] nonzero: item is in redo_list
  int32_t* redo_list;        // [item_bound] item indices, redo_count of them valid
  void* k_anc_bf16;          // FP8 anchor KV: [T_A, Hkv, D] bf16 copies of the codes
  void* v_anc_bf16;
  // Which part of the cascade one launch sequence computes:
  //   kFused       anchor and suffix keys in one online softmax (out, lse)
  //   kAnchorPass  anchor keys only: fp32 normalised O_a -> o_part, lse_a -> lse_part
  //                (anchors of length 0 get no work items; lse_part must hold -inf there)
  //   kSuffixPass  the suffix's own keys only: out / lse as kFused, or with merge != 0
  //                the LSE merge with (o_part, lse_part) done in the epilogue
  int mode;
  int merge;
  // 2: work items of two 128-row query tiles (one CTA each); 4: "quads" of four query
  // tiles for the CTA-pair kernel (the exact kernel then walks quad halves)
  int tiles_per_item;
  float* o_part;             // [T_S, Hq, D] fp32
  float* lse_part;           // [T_S, Hq] fp32 (natural log)
  // Optional (causal prefill): max |x| of the suffix K and V per (suffix, KV head),
  // [S, Hkv] fp32, formed from the K/V tiles already in shared memory via per-row
  // maxima rowmax [T_S, Hkv, 2] (bf16 bit patterns of max |k|, max |v|).
  float* k_amax;
  float* v_amax;
  uint16_t* rowmax;
  unsigned* err_word;
  uint64_t timeout_ns;
  int inject_skip_first_kv;
};

// Byte offsets of the workspace regions; `total` is the size to allocate.
struct CascadeWorkspace {
  size_t flag, redo_count, prefix, order, seg, items, redo_flag, redo_list, k_anc_bf16,
      v_anc_bf16, total;
};
// anchor_bf16_bytes: T_A * Hkv * D * 2 with FP8 anchor KV (each of the two staged
// copies), else 0.
CascadeWorkspace cascade_workspace_layout(int num_anchors, int64_t total_suffix_tokens,
                                          int64_t item_bound, int64_t anchor_bf16_bytes);
int64_t cascade_item_bound(int num_anchors, int64_t total_suffix_tokens, int hkv, int group);

// Tensor maps over q_suf, k/v anchor and k/v suffix (bf16, 3-D: d, head, token).
struct CascadeMaps {
  CUtensorMap q, k_anc, v_anc, k_suf, v_suf;
  CUtensorMap k_anc64, k_suf64;  // the same K tensors with 64-row boxes (CTA-pair halves)
  // bf16 output [T_S, Hq, d] for the epilogue's TMA stores: box (32 of d, G heads, 32 / G
  // tokens) = one warp's rows, 64-byte swizzle (fused mode only)
  CUtensorMap out;
};

// Which d = 128 fused calls run the CTA-pair kernel: QUAIL_CTA_PAIRS_OFF / _AUTO (the
// default) / _ALWAYS.
void set_cta_pairs(int mode);

// ---- paged cache (paged.cu, scores.cu, evict.cu)
// Allows kernel `fn` `bytes` of dynamic shared memory on the current device, once per device
// (`ready`: the devices done so far, kept by the caller).
inline cudaError_t allow_smem(const void* fn, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (ready.load(std::memory_order_relaxed) >> dev & 1u)) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}
// What the entry points outside api.cu need of the current device.
struct DeviceInfo {
  int num_sms;
  unsigned* err_word;
  uint64_t timeout_ns;
  int inject_skip_first_kv;
};
// A quail_status; `info` is filled when it is QUAIL_OK.
int current_device_info(DeviceInfo* info);
// 3-D bf16 tensor map over [tokens, heads, d] rows `row_stride` elements apart, 128-byte
// swizzle, box (64 of d, box_heads, box_rows); out-of-range rows read as zero.
bool encode_rows_bf16(CUtensorMap* m, const void* base, int64_t tokens, int64_t row_stride,
                      int heads, int d, int box_heads, int box_rows);

struct PagedAppendArgs {
  int num_seqs, hkv, head_dim, row_elems;  // row_elems = hkv * head_dim
  int max_len, page_shift, max_pages, num_pages;
  int64_t total_new, k_stride, v_stride;   // elements between token rows
  const uint16_t* k_new;                   // bf16
  const uint16_t* v_new;
  const int32_t* new_offsets;              // NULL: one token per sequence
  const int32_t* start_pos;
  const int32_t* table;
  const float* k_scale;
  const float* v_scale;
  uint8_t* k_pages;
  uint8_t* v_pages;
  unsigned* err_word;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, int num_sms,
                                cudaStream_t stream);
// How pages hold their values (quail_dtype's numbers).
enum KvForm {
  kBf16,
  kE4m3,  // codes, a scale per sequence and KV head
  kFp4    // e2m1 codes, an e4m3 scale per 16 values and a scale per sequence and KV head
};
// A launch that may begin before the kernel ahead of it in the stream has ended: the kernel itself waits
// for that (after_stream, with the rules beside it).
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         int cluster, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Token rows written into fp4 pages, or read back from pages of any form.
struct PagedRows {
  int num_seqs, hkv;
  int max_len, page_shift, max_pages, num_pages;
  int64_t total, k_stride, v_stride;       // token rows; elements between them
  const uint16_t* k_new;                   // append: bf16
  const uint16_t* v_new;
  uint16_t* k_out;                         // read: bf16; one of the two may be NULL
  uint16_t* v_out;
  const int32_t* offsets;                  // NULL: one token per sequence
  const int32_t* start_pos;
  const int32_t* table;
  const float* k_scale;
  const float* v_scale;
  uint8_t* k_pages;
  uint8_t* v_pages;
  unsigned* err_word;
};
cudaError_t launch_fp4_append(const PagedRows& p, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedRows& p, int head_dim, int kv_dtype, int num_sms,
                              cudaStream_t stream);

// What a CTA (or a warp, see decode_by_warps) of the decode attention leaves for the join: the (sequence, head) that begins
// in it and goes on in the next CTAs (seq < 0: none) up to CTA `last`; sparse: the number of
// tiles where there are fewer than CTAs (some then have none), else 0.
struct DecodeRec {
  int seq, head, last, sparse;
};
struct PagedDecodeArgs {
  int num_seqs, hq, hkv, group;
  int max_len, page_shift, max_pages, num_pages;
  float scale_log2;                 // softmax scale * log2(e)
  const __nv_bfloat16* q;
  int64_t q_stride;                 // elements between the sequences' rows
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const int32_t* table;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;
  float* lse;
  const float* score_in;
  float* score_out;
  int64_t score_stride;
  // workspace
  DecodeRec* rec;                   // [CTAs]
  float2* part_ml;                  // [2 CTAs][group] max (log2 units) and sum
  float* part_o;                    // [2 CTAs][group][d]
  float* lse2;                      // [B, Hq], with scores only: of what one CTA finished
  int32_t* begun;                   // [B, Hkv], with scores only: the CTA in which a (sequence,
                                    // head) of several CTAs begins, or -1
  float* raw;                       // [B, Hq, raw_stride] scores in log2 units, or NULL
  int64_t raw_stride;
  unsigned* err_word;
  // fp4 pages: a KV head counts as 2^split of them with a part of its group each; how long a wait for a
  // step's copies may block; no copies, so that it does
  int split;
  uint64_t timeout_ns;
  int inject_skip_loads;
};
constexpr int kDecodeMaxSms = 160;  // the workspace holds the parts of so many SMs' CTAs
int decode_tile_keys(int head_dim, int kv_dtype);
int decode_ctas_per_sm(int kv_dtype, int group);
int decode_ctas(int num_sms, int per_sm, int num_seqs, int hkv, int max_len, int tile);
// Whether runs are dealt to warps, four per CTA (the workspace then holds four times the parts).
bool decode_by_warps(int kv_dtype, int group, int num_seqs, int hkv, int max_len, int tile);
cudaError_t launch_paged_decode(PagedDecodeArgs& a, int head_dim, int kv_dtype, int num_sms,
                                cudaStream_t stream);
// Keys of a CTA's tile over fp4 pages: 8 KB of codes.
constexpr int fp4_tile_keys(int head_dim) { return 16384 / head_dim; }
int fp4_decode_per_sm(int group);
bool fp4_warp_runs(int group);
cudaError_t launch_fp4_decode(PagedDecodeArgs& a, int head_dim, int num_sms, cudaStream_t stream);

struct AttnScoresArgs {
  int num_seqs, hq, hkv, group;
  int64_t total_q, total_k;
  int max_q, max_k, window;
  bool causal;
  float scale_log2;
  const float* lse;
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  const float* score_in;
  float* score_out;
  int64_t score_stride;
  unsigned* err_word;
  uint64_t timeout_ns;
  int inject_skip_first_kv;
};
cudaError_t launch_attn_scores(const AttnScoresArgs& a, const CUtensorMap& q_map,
                               const CUtensorMap& k_map, int head_dim, int num_sms,
                               cudaStream_t stream);

struct PagedEvictArgs {
  int num_seqs, hkv, row_bytes;      // row_bytes of one (token, head); fp4: of its codes
  int block_bytes;                   // fp4: of its block scales, 0 otherwise
  int max_len, page_shift, max_pages, num_pages;
  int budget, recent;
  int dst_max_pages, dst_num_pages;
  bool same_pool;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const int32_t* table;
  const int32_t* lens;
  const float* score;
  int64_t score_stride;
  const int32_t* dst_table;
  uint8_t* k_dst;
  uint8_t* v_dst;
  int32_t* kept;
  int32_t* new_lens;
  float* score_out;
  int64_t score_out_stride;
  int32_t* claim;                    // workspace: [dst_num_pages] each, not cleared
  int32_t* dup;
  int32_t* hold;
  unsigned* err_word;
};
cudaError_t launch_paged_evict(const PagedEvictArgs& a, int num_sms, cudaStream_t stream);

constexpr int kFused = 0, kAnchorPass = 1, kSuffixPass = 2;

// quail_cascade_attn plus the max |x| of the suffix K and V per (suffix, KV head) into
// k_amax / v_amax ([S, Hkv] fp32), formed by the fast kernel from the tiles it loads.
// rowmax: [T_S, Hkv, 2] uint16 scratch for the per-row maxima.
quail_status cascade_attn_with_amax(const quail_cascade_desc* desc, const void* q_suf,
                                    const void* k_anc, const void* v_anc, const void* k_suf,
                                    const void* v_suf, const int32_t* anchor_offsets,
                                    const int32_t* anchor_suffix_ptr,
                                    const int32_t* suffix_offsets, void* out, float* lse,
                                    float* k_amax, float* v_amax, uint16_t* rowmax,
                                    void* workspace, size_t workspace_bytes,
                                    quail_stream_t stream);

cudaError_t launch_cascade(const CascadeParams& p, const CascadeMaps& maps, int head_dim,
                           bool fp8, int num_sms, cudaStream_t stream);

// Two-pass helpers: lse_part[0, n) = -inf; and the LSE merge of the anchor partial
// (o_part, lse_part) with the suffix partial (out, lse_s) in place into out (and lse).
cudaError_t launch_fill_neg_inf(float* x, int64_t n, int num_sms, cudaStream_t stream);
cudaError_t launch_lse_merge(int64_t rows, int head_dim, const float* o_part,
                             const float* lse_part, const float* lse_s, void* out, float* lse,
                             int num_sms, cudaStream_t stream);

}  // namespace quail

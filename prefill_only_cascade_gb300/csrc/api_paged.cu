// api_paged.cu - the C ABI of the paged cache (declared in include/quail.h): argument
// validation on the host and launches on the caller's stream. No call allocates.
#include <cmath>
#include <cstring>

#include "kernels.h"
#include "quail.h"

namespace {

constexpr int64_t kInt32Max = (1ll << 31) - 1;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool valid_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8 || g == 16; }

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Whether [p, p + n) meets one of `rows` rows of `row` bytes that lie `stride` bytes apart.
bool meets_rows(const void* p, size_t n, const void* base, int64_t rows, int64_t row, int64_t stride) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(base);
  if (n == 0 || rows <= 0 || row <= 0) return false;
  // the first row that ends past p
  const int64_t i = a < b + row ? 0 : static_cast<int64_t>((a - b - row) / stride + 1);
  return i < rows && b + static_cast<uintptr_t>(i) * stride < a + n;
}

// score_in and score_out, rows of both `stride` entries apart: one buffer, or two that do not meet.
bool scores_apart(const float* in, const float* out, int64_t rows, int64_t stride) {
  const size_t n = 4 * static_cast<size_t>(rows) * static_cast<size_t>(stride);
  return in == nullptr || in == out || !overlap(in, n, out, n);
}

// The checks of every paged call.
quail_status check_desc(const quail_paged_desc* desc) {
  if (desc == nullptr) return QUAIL_ERR_INVALID_ARG;
  const quail_paged_desc& d = *desc;
  if (d.num_seqs < 0 || d.max_seq_len < 0 || d.num_pages < 0 || d.max_pages_per_seq < 0 ||
      d.page_size <= 0)
    return QUAIL_ERR_INVALID_ARG;
  if (d.num_q_heads <= 0 || d.num_kv_heads <= 0 || d.num_q_heads % d.num_kv_heads != 0)
    return QUAIL_ERR_INVALID_ARG;
  if (!(d.softmax_scale >= 0.0f) || !std::isfinite(d.softmax_scale)) return QUAIL_ERR_INVALID_ARG;
  if (d.kv_dtype != QUAIL_BF16 && d.kv_dtype != QUAIL_FP8_E4M3) return QUAIL_ERR_INVALID_ARG;
  if (d.head_dim != 64 && d.head_dim != 128) return QUAIL_ERR_UNSUPPORTED;
  if (!valid_group(d.num_q_heads / d.num_kv_heads)) return QUAIL_ERR_UNSUPPORTED;
  if (d.page_size < 16 || d.page_size > 256 || (d.page_size & (d.page_size - 1)) != 0)
    return QUAIL_ERR_UNSUPPORTED;
  if (d.max_seq_len > (1 << 30)) return QUAIL_ERR_UNSUPPORTED;
  if (d.max_seq_len > static_cast<int64_t>(d.max_pages_per_seq) * d.page_size)
    return QUAIL_ERR_INVALID_ARG;
  if (static_cast<int64_t>(d.num_seqs) * d.max_pages_per_seq > kInt32Max) return QUAIL_ERR_UNSUPPORTED;
  // work counted in 32 bits: 8 blocks per (sequence, query head)
  if (static_cast<int64_t>(d.num_seqs) * d.num_q_heads > kInt32Max / 8) return QUAIL_ERR_UNSUPPORTED;
  return QUAIL_OK;
}

// e4m3 pages come with scales, bf16 pages without.
bool scales_ok(const quail_paged_desc& d, const float* k_scale, const float* v_scale) {
  if (d.kv_dtype == QUAIL_FP8_E4M3)
    return k_scale != nullptr && v_scale != nullptr && aligned(k_scale, 4) && aligned(v_scale, 4);
  return k_scale == nullptr && v_scale == nullptr;
}

int elem_bytes(const quail_paged_desc& d) { return d.kv_dtype == QUAIL_FP8_E4M3 ? 1 : 2; }

float scale_log2_of(float softmax_scale, int head_dim) {
  const float s = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  return s * 1.4426950408889634f;
}

struct DecodeLayout {
  size_t rec, part_ml, part_o, lse2, begun, raw, total;
  int64_t raw_stride;
};
DecodeLayout decode_layout(const quail_paged_desc& d, bool with_scores) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const bool fp8 = d.kv_dtype == QUAIL_FP8_E4M3;
  const int group = d.num_q_heads / d.num_kv_heads;
  const int tile = quail::decode_tile_keys(d.head_dim, fp8);
  const size_t parts = 2 * static_cast<size_t>(quail::decode_ctas(
                               quail::kDecodeMaxCtas, d.num_seqs, d.num_kv_heads, d.max_seq_len,
                               tile)) *
                       (quail::decode_by_warps(d.num_seqs, d.num_kv_heads, d.max_seq_len, tile) ? 4 : 1);
  DecodeLayout l;
  l.raw_stride = (static_cast<int64_t>(d.max_seq_len) + tile - 1) / tile * tile;
  l.rec = 0;
  l.part_ml = up(parts / 2 * sizeof(quail::DecodeRec));
  l.part_o = up(l.part_ml + parts * group * sizeof(float2));
  l.lse2 = up(l.part_o + parts * group * d.head_dim * 4);
  const size_t rows = static_cast<size_t>(d.num_seqs) * d.num_q_heads;
  l.begun = up(l.lse2 + (with_scores ? rows * 4 : 0));
  l.raw = up(l.begun + (with_scores ? rows / group * 4 : 0));
  l.total = up(l.raw + (with_scores ? rows * l.raw_stride * 4 : 0));
  return l;
}

}  // namespace

extern "C" {

quail_status quail_paged_kv_append(const quail_paged_desc* desc, int64_t num_new,
                                   const void* k_new, const void* v_new, int64_t k_row_stride,
                                   int64_t v_row_stride, const int32_t* new_offsets,
                                   const int32_t* start_pos, const int32_t* block_table,
                                   const float* k_scale, const float* v_scale, void* k_pages,
                                   void* v_pages, quail_stream_t stream) {
  const quail_status c = check_desc(desc);
  if (c != QUAIL_OK) return c;
  const quail_paged_desc& d = *desc;
  const int row = d.num_kv_heads * d.head_dim;
  if (num_new < 0 || num_new > kInt32Max || (d.num_seqs == 0 && num_new != 0))
    return QUAIL_ERR_INVALID_ARG;
  if (new_offsets == nullptr && num_new != d.num_seqs) return QUAIL_ERR_INVALID_ARG;
  if (k_row_stride < row || v_row_stride < row || k_row_stride % 8 != 0 || v_row_stride % 8 != 0)
    return QUAIL_ERR_INVALID_ARG;
  if (!scales_ok(d, k_scale, v_scale) || !aligned(new_offsets, 4)) return QUAIL_ERR_INVALID_ARG;
  if (num_new > 0) {
    if (k_new == nullptr || v_new == nullptr || start_pos == nullptr || block_table == nullptr ||
        k_pages == nullptr || v_pages == nullptr)
      return QUAIL_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) ||
        !aligned(v_pages, 16) || !aligned(start_pos, 4) || !aligned(block_table, 4))
      return QUAIL_ERR_INVALID_ARG;
    const size_t pool = static_cast<size_t>(d.num_pages) * d.page_size * row * elem_bytes(d);
    if (overlap(k_pages, pool, v_pages, pool)) return QUAIL_ERR_INVALID_ARG;
  }
  quail::DeviceInfo info;
  const int ds = quail::current_device_info(&info);
  if (ds != QUAIL_OK) return static_cast<quail_status>(ds);
  if (num_new == 0) return QUAIL_OK;
  quail::PagedAppendArgs a{};
  a.num_seqs = d.num_seqs;
  a.hkv = d.num_kv_heads;
  a.head_dim = d.head_dim;
  a.row_elems = row;
  a.max_len = d.max_seq_len;
  a.page_shift = log2_of(d.page_size);
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages;
  a.total_new = num_new;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.new_offsets = new_offsets;
  a.start_pos = start_pos;
  a.table = block_table;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_pages = static_cast<uint8_t*>(k_pages);
  a.v_pages = static_cast<uint8_t*>(v_pages);
  a.err_word = info.err_word;
  const cudaError_t e = quail::launch_paged_append(a, d.kv_dtype == QUAIL_FP8_E4M3, info.num_sms,
                                                   reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QUAIL_OK : QUAIL_ERR_CUDA;
}

size_t quail_paged_decode_workspace_size(const quail_paged_desc* desc, int32_t with_scores) {
  return check_desc(desc) == QUAIL_OK ? decode_layout(*desc, with_scores != 0).total : 0;
}

quail_status quail_paged_decode_attn(const quail_paged_desc* desc, const void* q,
                                     int64_t q_row_stride, const void* k_pages,
                                     const void* v_pages, const int32_t* block_table,
                                     const int32_t* seq_lens, const float* k_scale,
                                     const float* v_scale, void* out, float* lse,
                                     const float* score_in, float* score_out,
                                     int64_t score_stride, void* workspace,
                                     size_t workspace_bytes, quail_stream_t stream) {
  const quail_status c = check_desc(desc);
  if (c != QUAIL_OK) return c;
  const quail_paged_desc& d = *desc;
  const bool scored = score_out != nullptr;
  if (!scales_ok(d, k_scale, v_scale)) return QUAIL_ERR_INVALID_ARG;
  if (q_row_stride < static_cast<int64_t>(d.num_q_heads) * d.head_dim || q_row_stride % 8 != 0)
    return QUAIL_ERR_INVALID_ARG;
  if (score_in != nullptr && !scored) return QUAIL_ERR_INVALID_ARG;
  if (scored && score_stride < d.max_seq_len) return QUAIL_ERR_INVALID_ARG;
  // written by some blocks while others read
  const int64_t row = static_cast<int64_t>(d.num_q_heads) * d.head_dim * 2;
  if (meets_rows(out, static_cast<size_t>(d.num_seqs) * row, q, d.num_seqs, row, 2 * q_row_stride) ||
      !scores_apart(score_in, score_out, static_cast<int64_t>(d.num_seqs) * d.num_kv_heads, score_stride))
    return QUAIL_ERR_INVALID_ARG;
  if (d.num_seqs > 0) {
    if (q == nullptr || seq_lens == nullptr || out == nullptr || !aligned(q, 16) ||
        !aligned(seq_lens, 4) || !aligned(out, 16))
      return QUAIL_ERR_INVALID_ARG;
    if (d.max_seq_len > 0 && (k_pages == nullptr || v_pages == nullptr || block_table == nullptr))
      return QUAIL_ERR_INVALID_ARG;
  }
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4) ||
      !aligned(lse, 4) || !aligned(score_in, 4) || !aligned(score_out, 4))
    return QUAIL_ERR_INVALID_ARG;
  const DecodeLayout l = decode_layout(d, scored);
  if (workspace == nullptr || workspace_bytes < l.total || !aligned(workspace, 16))
    return QUAIL_ERR_INVALID_ARG;
  quail::DeviceInfo info;
  const int ds = quail::current_device_info(&info);
  if (ds != QUAIL_OK) return static_cast<quail_status>(ds);
  if (d.num_seqs == 0) return QUAIL_OK;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  quail::PagedDecodeArgs a{};
  a.num_seqs = d.num_seqs;
  a.hq = d.num_q_heads;
  a.hkv = d.num_kv_heads;
  a.group = d.num_q_heads / d.num_kv_heads;
  a.max_len = d.max_seq_len;
  a.page_shift = log2_of(d.page_size);
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages;
  a.scale_log2 = scale_log2_of(d.softmax_scale, d.head_dim);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_row_stride;
  a.k_pages = static_cast<const uint8_t*>(k_pages);
  a.v_pages = static_cast<const uint8_t*>(v_pages);
  a.table = block_table;
  a.lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.score_in = score_in;
  a.score_out = score_out;
  a.score_stride = score_stride;
  a.rec = reinterpret_cast<quail::DecodeRec*>(w + l.rec);
  a.part_ml = reinterpret_cast<float2*>(w + l.part_ml);
  a.part_o = reinterpret_cast<float*>(w + l.part_o);
  a.lse2 = scored ? reinterpret_cast<float*>(w + l.lse2) : nullptr;
  a.begun = scored ? reinterpret_cast<int32_t*>(w + l.begun) : nullptr;
  a.raw = scored ? reinterpret_cast<float*>(w + l.raw) : nullptr;
  a.raw_stride = l.raw_stride;
  a.err_word = info.err_word;
  const cudaError_t e =
      quail::launch_paged_decode(a, d.head_dim, d.kv_dtype == QUAIL_FP8_E4M3, info.num_sms,
                                 reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QUAIL_OK : QUAIL_ERR_CUDA;
}

quail_status quail_attn_scores(int32_t num_seqs, int64_t total_q_tokens, int64_t total_k_tokens,
                               int32_t max_q_len, int32_t max_k_len, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim, float softmax_scale,
                               int32_t causal, int32_t window, const void* q,
                               int64_t q_row_stride, const void* k, int64_t k_row_stride,
                               const float* lse, const int32_t* q_offsets,
                               const int32_t* k_offsets, const float* score_in, float* score_out,
                               int64_t score_stride, quail_stream_t stream) {
  if (num_seqs < 0 || total_q_tokens < 0 || total_k_tokens < 0 || total_q_tokens > kInt32Max ||
      total_k_tokens > kInt32Max || max_q_len < 0 || max_k_len < 0 || window < 0 ||
      (causal != 0 && causal != 1))
    return QUAIL_ERR_INVALID_ARG;
  if (num_seqs == 0 && (total_q_tokens != 0 || total_k_tokens != 0)) return QUAIL_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0)
    return QUAIL_ERR_INVALID_ARG;
  if (!(softmax_scale >= 0.0f) || !std::isfinite(softmax_scale)) return QUAIL_ERR_INVALID_ARG;
  const int group = num_q_heads / num_kv_heads;
  if (head_dim != 64 && head_dim != 128) return QUAIL_ERR_UNSUPPORTED;
  if (!valid_group(group)) return QUAIL_ERR_UNSUPPORTED;
  if (q_row_stride < static_cast<int64_t>(num_q_heads) * head_dim || q_row_stride % 8 != 0 ||
      k_row_stride < static_cast<int64_t>(num_kv_heads) * head_dim || k_row_stride % 8 != 0)
    return QUAIL_ERR_INVALID_ARG;
  if (score_stride < max_k_len) return QUAIL_ERR_INVALID_ARG;
  if (num_seqs > 0 && (q_offsets == nullptr || k_offsets == nullptr || !aligned(q_offsets, 4) ||
                       !aligned(k_offsets, 4)))
    return QUAIL_ERR_INVALID_ARG;
  if (total_q_tokens > 0 && (q == nullptr || lse == nullptr || !aligned(q, 16) || !aligned(lse, 4)))
    return QUAIL_ERR_INVALID_ARG;
  if (total_k_tokens > 0 && (k == nullptr || score_out == nullptr || !aligned(k, 16)))
    return QUAIL_ERR_INVALID_ARG;
  if (!aligned(score_in, 4) || !aligned(score_out, 4)) return QUAIL_ERR_INVALID_ARG;
  if (!scores_apart(score_in, score_out, static_cast<int64_t>(num_seqs) * num_kv_heads, score_stride))
    return QUAIL_ERR_INVALID_ARG;
  // TMA coordinates and key numbers run up to two tiles past the last token
  if (total_q_tokens > kInt32Max - 1024 || total_k_tokens > kInt32Max - 1024 ||
      max_k_len > kInt32Max - 1024)
    return QUAIL_ERR_UNSUPPORTED;
  // 8 blocks at most per (sequence, KV head, 128 keys)
  if ((static_cast<int64_t>(max_k_len) + 127) / 128 * num_seqs > kInt32Max / 8 / num_kv_heads)
    return QUAIL_ERR_UNSUPPORTED;
  quail::DeviceInfo info;
  const int ds = quail::current_device_info(&info);
  if (ds != QUAIL_OK) return static_cast<quail_status>(ds);
  if (num_seqs == 0 || total_k_tokens == 0 || max_k_len == 0) return QUAIL_OK;
  CUtensorMap q_map, k_map;
  if (!quail::encode_rows_bf16(&k_map, k, total_k_tokens, k_row_stride, num_kv_heads, head_dim, 1,
                               128))
    return QUAIL_ERR_CUDA;
  q_map = k_map;  // without queries nothing is loaded through it
  if (total_q_tokens > 0 &&
      !quail::encode_rows_bf16(&q_map, q, total_q_tokens, q_row_stride, num_q_heads, head_dim,
                               group, 128 / group))
    return QUAIL_ERR_CUDA;
  quail::AttnScoresArgs a{};
  a.num_seqs = num_seqs;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.group = group;
  a.total_q = total_q_tokens;
  a.total_k = total_k_tokens;
  a.max_q = max_q_len;
  a.max_k = max_k_len;
  a.window = window;
  a.causal = causal != 0;
  a.scale_log2 = scale_log2_of(softmax_scale, head_dim);
  a.lse = lse;
  a.q_offsets = q_offsets;
  a.k_offsets = k_offsets;
  a.score_in = score_in;
  a.score_out = score_out;
  a.score_stride = score_stride;
  a.err_word = info.err_word;
  a.timeout_ns = info.timeout_ns;
  a.inject_skip_first_kv = info.inject_skip_first_kv;
  const cudaError_t e = quail::launch_attn_scores(a, q_map, k_map, head_dim, info.num_sms,
                                                  reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QUAIL_OK : QUAIL_ERR_CUDA;
}

size_t quail_paged_evict_workspace_size(const quail_paged_desc* desc, int32_t dst_num_pages) {
  if (check_desc(desc) != QUAIL_OK || dst_num_pages < 0) return 0;
  return (static_cast<size_t>(dst_num_pages) * 12 + 255) / 256 * 256 + 256;
}

quail_status quail_paged_kv_evict(const quail_paged_desc* desc, int32_t budget, int32_t recent,
                                  const void* k_pages, const void* v_pages,
                                  const int32_t* block_table, const int32_t* seq_lens,
                                  const float* score, int64_t score_stride,
                                  const int32_t* dst_table, int32_t dst_max_pages_per_seq,
                                  int32_t dst_num_pages, void* k_dst, void* v_dst, int32_t* kept,
                                  int32_t* new_lens, float* score_out, int64_t score_out_stride,
                                  void* workspace, size_t workspace_bytes,
                                  quail_stream_t stream) {
  const quail_status c = check_desc(desc);
  if (c != QUAIL_OK) return c;
  const quail_paged_desc& d = *desc;
  if (budget < 1 || recent < 0 || recent > budget || dst_max_pages_per_seq < 0 ||
      dst_num_pages < 0 || score_stride < d.max_seq_len)
    return QUAIL_ERR_INVALID_ARG;
  if (budget > (1 << 30)) return QUAIL_ERR_UNSUPPORTED;
  const int64_t most = budget < d.max_seq_len ? budget : d.max_seq_len;
  if (most > static_cast<int64_t>(dst_max_pages_per_seq) * d.page_size) return QUAIL_ERR_INVALID_ARG;
  if (score_out != nullptr && score_out_stride < budget) return QUAIL_ERR_INVALID_ARG;
  const int64_t pairs = static_cast<int64_t>(d.num_seqs) * d.num_kv_heads;
  if (static_cast<int64_t>(d.num_seqs) * dst_max_pages_per_seq > kInt32Max)
    return QUAIL_ERR_UNSUPPORTED;
  // blocks of 256 kept rows
  if (d.num_seqs > 0 &&
      (static_cast<int64_t>(budget) * d.num_kv_heads + 255) / 256 > kInt32Max / d.num_seqs)
    return QUAIL_ERR_UNSUPPORTED;
  const int row_bytes = d.head_dim * elem_bytes(d);
  const size_t page_bytes = static_cast<size_t>(d.page_size) * d.num_kv_heads * row_bytes;
  const size_t src_bytes = page_bytes * d.num_pages, dst_bytes = page_bytes * dst_num_pages;
  const bool same_pool = k_dst == k_pages;
  if (d.num_seqs > 0) {
    if (seq_lens == nullptr || kept == nullptr || new_lens == nullptr) return QUAIL_ERR_INVALID_ARG;
    if (d.max_seq_len > 0 && (k_pages == nullptr || v_pages == nullptr || block_table == nullptr ||
                              score == nullptr || dst_table == nullptr || k_dst == nullptr ||
                              v_dst == nullptr))
      return QUAIL_ERR_INVALID_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_dst, 16) ||
        !aligned(v_dst, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(score, 4) || !aligned(dst_table, 4) || !aligned(kept, 4) ||
        !aligned(new_lens, 4) || !aligned(score_out, 4))
      return QUAIL_ERR_INVALID_ARG;
    // one pool for both (the kernels tell its pages apart), or two that do not meet
    if (same_pool ? (v_dst != v_pages || dst_num_pages != d.num_pages)
                  : (overlap(k_dst, dst_bytes, k_pages, src_bytes) ||
                     overlap(v_dst, dst_bytes, v_pages, src_bytes)))
      return QUAIL_ERR_INVALID_ARG;
    if (overlap(k_dst, dst_bytes, v_pages, src_bytes) ||
        overlap(v_dst, dst_bytes, k_pages, src_bytes) || overlap(k_dst, dst_bytes, v_dst, dst_bytes))
      return QUAIL_ERR_INVALID_ARG;
    // read by some blocks while others write
    if (overlap(new_lens, 4 * static_cast<size_t>(d.num_seqs), seq_lens,
                4 * static_cast<size_t>(d.num_seqs)) ||
        (score_out != nullptr && overlap(score_out, 4 * pairs * static_cast<size_t>(score_out_stride),
                                         score, 4 * pairs * static_cast<size_t>(score_stride))))
      return QUAIL_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < quail_paged_evict_workspace_size(desc, dst_num_pages))
    return QUAIL_ERR_INVALID_ARG;
  quail::DeviceInfo info;
  const int ds = quail::current_device_info(&info);
  if (ds != QUAIL_OK) return static_cast<quail_status>(ds);
  if (d.num_seqs == 0) return QUAIL_OK;
  quail::PagedEvictArgs a{};
  a.num_seqs = d.num_seqs;
  a.hkv = d.num_kv_heads;
  a.row_bytes = row_bytes;
  a.max_len = d.max_seq_len;
  a.page_shift = log2_of(d.page_size);
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages;
  a.budget = budget;
  a.recent = recent;
  a.dst_max_pages = dst_max_pages_per_seq;
  a.dst_num_pages = dst_num_pages;
  a.same_pool = same_pool;
  a.k_pages = static_cast<const uint8_t*>(k_pages);
  a.v_pages = static_cast<const uint8_t*>(v_pages);
  a.table = block_table;
  a.lens = seq_lens;
  a.score = score;
  a.score_stride = score_stride;
  a.dst_table = dst_table;
  a.k_dst = static_cast<uint8_t*>(k_dst);
  a.v_dst = static_cast<uint8_t*>(v_dst);
  a.kept = kept;
  a.new_lens = new_lens;
  a.score_out = score_out;
  a.score_out_stride = score_out_stride;
  a.claim = static_cast<int32_t*>(workspace);
  a.dup = a.claim + dst_num_pages;
  a.hold = a.dup + dst_num_pages;
  a.err_word = info.err_word;
  const cudaError_t e =
      quail::launch_paged_evict(a, info.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QUAIL_OK : QUAIL_ERR_CUDA;
}

}  // extern "C"

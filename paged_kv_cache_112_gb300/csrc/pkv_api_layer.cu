// Host side of the layer operators around paged decode: norm + rotation +
// write, block summaries, block selection and sparse decode attention.
// Argument validation, descriptors and launches, as pkv_api.cu.
#include <cmath>

#include "pkv.h"
#include "pkv_internal.h"

namespace pkv {
pkv_status cuda_status(cudaError_t e);

namespace {

bool value_dtype_ok(pkv_dtype d) { return d == PKV_F16 || d == PKV_BF16; }

// Row stride in elements: 0 means dense; -1 when below a row or not whole 16-byte vectors.
int64_t row_stride(int64_t stride, int64_t row) {
  if (stride == 0) return row;
  return stride < row || stride % 8 != 0 ? -1 : stride;
}

// Validation shared by the two pool kinds; fills everything but the pools'
// strides and scales.
pkv_status prepare_norm_rope(NormRopeArgs* a, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                             const void* q, int64_t q_stride, const void* k, const void* v, int64_t new_row_stride,
                             const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                             const int32_t* positions, int max_positions, int rot_dim, int interleaved, void* k_pool,
                             void* v_pool, const int32_t* slot_mapping, int num_tokens, int num_q_heads,
                             int num_kv_heads, int head_dim, int block_size, int num_blocks, pkv_dtype dtype,
                             int32_t* dev_status) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || rot_dim < 0 ||
      rot_dim > head_dim || (interleaved != 0 && interleaved != 1) || !value_dtype_ok(dtype))
    return PKV_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && !(std::isfinite(eps) && eps > 0.f)) return PKV_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || rot_dim % 16 != 0 || block_shift_of(block_size) < 0)
    return PKV_ERR_UNSUPPORTED;
  // Tasks (at most one a token and head) are numbered in 32 bits.
  if (num_tokens * (num_q_heads + 2LL * num_kv_heads) > 0xfffffff0LL) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_q_heads) * head_dim > 0x7fffffff ||
      static_cast<int64_t>(num_kv_heads) * head_dim > 0x7fffffff)
    return PKV_ERR_UNSUPPORTED;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  const int64_t qs = row_stride(q_stride, q_row), qos = row_stride(q_out_stride, q_row);
  const int64_t kvs = row_stride(new_row_stride, kv_row), kos = row_stride(k_out_stride, kv_row);
  if (qs < 0 || qos < 0 || kvs < 0 || kos < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !k || !v || !k_pool || !v_pool || !slot_mapping) return PKV_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!cos_sin || !positions || max_positions <= 0)) return PKV_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(q_out), static_cast<const void*>(k_out), q, k, v, q_weight, k_weight,
                        static_cast<const void*>(cos_sin), static_cast<const void*>(k_pool),
                        static_cast<const void*>(v_pool)})
    if (!aligned(p, 16)) return PKV_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(slot_mapping, 4) || !aligned(dev_status, 4)) return PKV_ERR_INVALID_ARG;
  // Rows rewritten in place keep their places.
  if ((q_out == q && qos != qs) || (k_out == k && kos != kvs)) return PKV_ERR_INVALID_ARG;
  a->q = static_cast<const uint16_t*>(q);
  a->k = static_cast<const uint16_t*>(k);
  a->v = static_cast<const uint16_t*>(v);
  a->q_out = static_cast<uint16_t*>(q_out);
  a->k_out = static_cast<uint16_t*>(k_out);
  a->q_weight = static_cast<const uint16_t*>(q_weight);
  a->k_weight = static_cast<const uint16_t*>(k_weight);
  a->eps = eps;
  a->timeout_ns = kWaitTimeoutNs;
  a->cos_sin = cos_sin;
  a->positions = positions;
  a->slot_mapping = slot_mapping;
  a->k_pool = k_pool;
  a->v_pool = v_pool;
  a->dev_status = dev_status;
  a->q_stride = qs;
  a->q_out_stride = qos;
  a->kv_stride = kvs;
  a->k_out_stride = kos;
  a->num_tokens = num_tokens;
  a->num_q_heads = num_q_heads;
  a->num_kv_heads = num_kv_heads;
  a->rot_dim = rot_dim;
  a->interleaved = interleaved;
  a->max_positions = max_positions;
  a->block_shift = block_shift_of(block_size);
  a->num_slots = static_cast<int64_t>(num_blocks) << a->block_shift;
  return PKV_OK;
}

pkv_status prepare_summarize(SummarizeArgs* a, void* summary, float* summary_scale, const void* k_pool,
                             const int32_t* block_ids, int num_ids, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, int32_t* dev_status) {
  if (num_ids < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || block_shift_of(block_size) < 4) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_ids) * num_kv_heads > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
  if (num_ids == 0) return PKV_OK;
  if (!summary || !summary_scale || !k_pool || !block_ids) return PKV_ERR_INVALID_ARG;
  if (!aligned(summary, 16) || !aligned(summary_scale, 4) || !aligned(k_pool, 16) || !aligned(block_ids, 4) ||
      !aligned(dev_status, 4))
    return PKV_ERR_INVALID_ARG;
  a->summary = static_cast<int8_t*>(summary);
  a->summary_scale = summary_scale;
  a->k_pool = static_cast<const uint8_t*>(k_pool);
  a->block_ids = block_ids;
  a->dev_status = dev_status;
  a->num_ids = num_ids;
  a->num_kv_heads = num_kv_heads;
  a->num_blocks = num_blocks;
  a->block_size = block_size;
  return PKV_OK;
}

// Everything of a sparse decode call but the tensor maps and FP8 scales.
pkv_status prepare_sparse(DecodeArgs* a, SparseArgs* sp, void* out, const void* q, const void* k_pool,
                          const void* v_pool, const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* context_lens, const int32_t* selected, const int32_t* counts, int keep,
                          int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, float scale, int max_context_len, pkv_dtype kv_dtype, pkv_dtype out_dtype,
                          int32_t* dev_status) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq < 0 || num_blocks <= 0 ||
      max_context_len < 0 || keep <= 0 || !std::isfinite(scale))
    return PKV_ERR_INVALID_ARG;
  if (!value_dtype_ok(kv_dtype) || (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16))
    return PKV_ERR_INVALID_ARG;
  const int shift = block_shift_of(block_size);
  if (shift < 4 || (head_dim != 64 && head_dim != 128) || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > 8 || keep > kMaxKeep || static_cast<int64_t>(num_seqs) * num_kv_heads > kMaxUnits ||
      (static_cast<int64_t>(max_blocks_per_seq) << shift) > 0x7fffffff)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_pool || !v_pool || !context_lens || !selected || !counts || (!block_tables && max_blocks_per_seq))
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(q, 16) || !aligned(out, out_dtype == PKV_F32 ? 4 : 2) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(selected, 4) || !aligned(counts, 4) ||
      !aligned(dev_status, 4))
    return PKV_ERR_INVALID_ARG;
  a->out = out;
  a->q = static_cast<const uint16_t*>(q);
  a->block_tables = block_tables;
  a->context_lens = context_lens;
  a->dev_status = dev_status;
  a->num_seqs = num_seqs;
  a->num_q_heads = num_q_heads;
  a->num_kv_heads = num_kv_heads;
  a->group = num_q_heads / num_kv_heads;
  a->max_blocks_per_seq = max_blocks_per_seq;
  a->num_blocks = num_blocks;
  a->max_context_len = max_context_len;
  a->block_shift = shift;
  a->scale_log2 = scale * 1.4426950408889634f;
  a->out_dtype = static_cast<int>(out_dtype);
  a->heads_per_box = 1;
  a->timeout_ns = kWaitTimeoutNs;
  sp->selected = selected;
  sp->counts = counts;
  sp->keep = keep;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_norm_rope_write(void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, const void* q,
                               int64_t q_stride, const void* k, const void* v, int64_t new_row_stride,
                               const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                               const int32_t* positions, int max_positions, int rot_dim, int interleaved,
                               void* k_pool, void* v_pool, int64_t block_stride, const int32_t* slot_mapping,
                               int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, pkv_dtype kv_dtype, int32_t* dev_status, void* stream) {
  NormRopeArgs a{};
  const pkv_status st = prepare_norm_rope(
      &a, q_out, q_out_stride, k_out, k_out_stride, q, q_stride, k, v, new_row_stride, q_weight, k_weight, eps, cos_sin,
      positions, max_positions, rot_dim, interleaved, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads,
      num_kv_heads, head_dim, block_size, num_blocks, kv_dtype, dev_status);
  if (st != PKV_OK) return st;
  a.block_stride = resolve_block_stride(block_stride, block_size, num_kv_heads, head_dim);
  if (a.block_stride < 0) return PKV_ERR_INVALID_ARG;
  return cuda_status(
      launch_norm_rope_write(a, head_dim, kv_dtype == PKV_BF16, false, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_norm_rope_write_fp8(void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, const void* q,
                                   int64_t q_stride, const void* k, const void* v, int64_t new_row_stride,
                                   const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
                                   const int32_t* positions, int max_positions, int rot_dim, int interleaved,
                                   void* k_pool, void* v_pool, const float* k_scale, const float* v_scale,
                                   const int32_t* slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                                   int head_dim, int block_size, int num_blocks, int num_layers, pkv_dtype new_dtype,
                                   int32_t* dev_status, void* stream) {
  if (num_layers <= 0 || num_layers > kMaxLayers) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  NormRopeArgs a{};
  const pkv_status st = prepare_norm_rope(
      &a, q_out, q_out_stride, k_out, k_out_stride, q, q_stride, k, v, new_row_stride, q_weight, k_weight, eps, cos_sin,
      positions, max_positions, rot_dim, interleaved, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads,
      num_kv_heads, head_dim, block_size, num_blocks, new_dtype, dev_status);
  if (st != PKV_OK || num_tokens == 0) return st;
  if (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return PKV_ERR_INVALID_ARG;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_stride = static_cast<int64_t>(num_layers) * kBlockSize * num_kv_heads * head_dim;
  a.scale_stride = static_cast<int64_t>(num_layers) * num_kv_heads;
  return cuda_status(
      launch_norm_rope_write(a, head_dim, new_dtype == PKV_BF16, true, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_summarize_blocks(void* summary, float* summary_scale, const void* k_pool, int64_t block_stride,
                                const int32_t* block_ids, int num_ids, int num_kv_heads, int head_dim, int block_size,
                                int num_blocks, pkv_dtype kv_dtype, int32_t* dev_status, void* stream) {
  if (!value_dtype_ok(kv_dtype)) return PKV_ERR_INVALID_ARG;
  SummarizeArgs a{};
  const pkv_status st = prepare_summarize(&a, summary, summary_scale, k_pool, block_ids, num_ids, num_kv_heads,
                                          head_dim, block_size, num_blocks, dev_status);
  if (st != PKV_OK) return st;
  const int64_t bstride = resolve_block_stride(block_stride, block_size, num_kv_heads, head_dim);
  if (bstride < 0) return PKV_ERR_INVALID_ARG;
  a.block_bytes = bstride * 2;
  return cuda_status(
      launch_summarize_blocks(a, head_dim, kv_dtype == PKV_BF16, false, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_summarize_blocks_fp8(void* summary, float* summary_scale, const void* k_pool, const float* k_scale,
                                    const int32_t* block_ids, int num_ids, int num_kv_heads, int head_dim,
                                    int block_size, int num_blocks, int num_layers, int32_t* dev_status,
                                    void* stream) {
  if (num_layers <= 0 || num_layers > kMaxLayers) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  SummarizeArgs a{};
  const pkv_status st = prepare_summarize(&a, summary, summary_scale, k_pool, block_ids, num_ids, num_kv_heads,
                                          head_dim, block_size, num_blocks, dev_status);
  if (st != PKV_OK || num_ids == 0) return st;
  if (!k_scale || !aligned(k_scale, 4)) return PKV_ERR_INVALID_ARG;
  a.k_scale = k_scale;
  a.block_bytes = static_cast<int64_t>(num_layers) * kBlockSize * num_kv_heads * head_dim;
  a.scale_stride = static_cast<int64_t>(num_layers) * num_kv_heads;
  return cuda_status(launch_summarize_blocks(a, head_dim, false, true, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_select_blocks(int32_t* selected, int32_t* counts, const void* q, const void* summary,
                             const float* summary_scale, const int32_t* block_tables, int max_blocks_per_seq,
                             const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks, int keep, int first_blocks, int last_blocks,
                             int max_context_len, pkv_dtype q_dtype, int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq < 0 || num_blocks <= 0 ||
      max_context_len < 0 || keep <= 0 || first_blocks < 0 || last_blocks < 1 ||
      static_cast<int64_t>(first_blocks) + last_blocks > keep || !value_dtype_ok(q_dtype))
    return PKV_ERR_INVALID_ARG;
  const int shift = block_shift_of(block_size);
  if (shift < 4 || (head_dim != 64 && head_dim != 128) || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > 8 || keep > kMaxKeep || static_cast<int64_t>(num_seqs) * num_kv_heads > kMaxUnits ||
      (static_cast<int64_t>(max_blocks_per_seq) << shift) > 0x7fffffff)
    return PKV_ERR_UNSUPPORTED;
  const int64_t by_len = (static_cast<int64_t>(max_context_len) + block_size - 1) >> shift;
  if ((by_len < max_blocks_per_seq ? by_len : max_blocks_per_seq) > kSelectMaxBlocks) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!selected || !counts || !q || !summary || !summary_scale || !context_lens || (!block_tables && max_blocks_per_seq))
    return PKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(summary, 16) || !aligned(summary_scale, 4) || !aligned(selected, 4) ||
      !aligned(counts, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(dev_status, 4))
    return PKV_ERR_INVALID_ARG;
  SelectArgs a{};
  a.selected = selected;
  a.counts = counts;
  a.q = static_cast<const uint16_t*>(q);
  a.summary = static_cast<const int8_t*>(summary);
  a.summary_scale = summary_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.dev_status = dev_status;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = num_q_heads / num_kv_heads;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.block_shift = shift;
  a.max_context_len = max_context_len;
  a.keep = keep;
  a.first_blocks = first_blocks;
  a.last_blocks = last_blocks;
  return cuda_status(launch_select_blocks(a, head_dim, q_dtype == PKV_BF16, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_decode_sparse(void* out, const void* q, const void* k_pool, const void* v_pool, int64_t block_stride,
                             const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
                             const int32_t* selected, const int32_t* counts, int keep, int num_seqs, int num_q_heads,
                             int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                             int max_context_len, pkv_dtype kv_dtype, pkv_dtype out_dtype, int32_t* dev_status,
                             void* stream) {
  DecodeArgs a{};
  SparseArgs sp{};
  const pkv_status st =
      prepare_sparse(&a, &sp, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, context_lens, selected, counts,
                     keep, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, kv_dtype, out_dtype, dev_status);
  if (st != PKV_OK) return st;
  a.block_stride = resolve_block_stride(block_stride, block_size, num_kv_heads, head_dim);
  if (a.block_stride < 0) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  CUtensorMap tk, tv;
  if (!encode_pool_map(&tk, k_pool, num_blocks, block_size, num_kv_heads, head_dim, 2, a.block_stride) ||
      !encode_pool_map(&tv, v_pool, num_blocks, block_size, num_kv_heads, head_dim, 2, a.block_stride))
    return PKV_ERR_CUDA;
  return cuda_status(
      launch_decode_sparse(a, sp, tk, tv, head_dim, kv_dtype == PKV_BF16, false, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_decode_sparse_fp8(void* out, const void* q, const void* k_pool, const void* v_pool,
                                 const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                 int max_blocks_per_seq, const int32_t* context_lens, const int32_t* selected,
                                 const int32_t* counts, int keep, int num_seqs, int num_q_heads, int num_kv_heads,
                                 int head_dim, int block_size, int num_blocks, int num_layers, float scale,
                                 int max_context_len, pkv_dtype q_dtype, pkv_dtype out_dtype, int32_t* dev_status,
                                 void* stream) {
  if (num_layers <= 0 || num_layers > kMaxLayers) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || head_dim != 128) return PKV_ERR_UNSUPPORTED;
  DecodeArgs a{};
  SparseArgs sp{};
  const pkv_status st =
      prepare_sparse(&a, &sp, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, context_lens, selected, counts,
                     keep, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, q_dtype, out_dtype, dev_status);
  if (st != PKV_OK || num_seqs == 0) return st;
  if (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return PKV_ERR_INVALID_ARG;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.scale_stride = static_cast<int64_t>(num_layers) * num_kv_heads;
  a.block_stride = static_cast<int64_t>(num_layers) * kBlockSize * num_kv_heads * head_dim;
  CUtensorMap tk, tv;
  if (!encode_pool_map(&tk, k_pool, num_blocks, kBlockSize, num_kv_heads, head_dim, 1, a.block_stride) ||
      !encode_pool_map(&tv, v_pool, num_blocks, kBlockSize, num_kv_heads, head_dim, 1, a.block_stride))
    return PKV_ERR_CUDA;
  return cuda_status(
      launch_decode_sparse(a, sp, tk, tv, head_dim, q_dtype == PKV_BF16, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

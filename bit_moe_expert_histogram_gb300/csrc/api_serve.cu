// C ABI of the batch serving calls (declared in include/moe_w4.h): cache
// pages, shared-prompt attention and draft verification. Host checks and
// launches only; nothing here allocates device memory, synchronises, or
// throws.
#include <climits>

#include "attn_q4.cuh"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ints(const void* p) { return p && aligned(p, 4); }

moe_status_t done(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return MOE_OK;
  set_last_cuda_error(e, where);
  return MOE_ERR_CUDA;
}

moe_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

bool meta_ok(const moe_cache_meta_t* m) {
  return m && ints(m->table_dev) && ints(m->lens_dev) && ints(m->refs_dev);
}
// two states that share no array
bool metas_ok(const moe_cache_meta_t* a, const moe_cache_meta_t* b) {
  return meta_ok(a) && meta_ok(b) && a->table_dev != b->table_dev && a->lens_dev != b->lens_dev &&
         a->refs_dev != b->refs_dev;
}

bool pools_ok(void* const* host, int32_t n, CachePools* out) {
  if (n < 0 || n > kMaxPools || (n > 0 && !host)) return false;
  *out = CachePools{};
  out->n = n;
  for (int i = 0; i < n; ++i) {
    if (!host[i] || !aligned(host[i], 16)) return false;
    out->p[i] = host[i];
  }
  return true;
}
}  // namespace

#define MOE_TRY(x)                 \
  do {                             \
    const moe_status_t st_ = (x);  \
    if (st_ != MOE_OK) return st_; \
  } while (0)

extern "C" {

size_t moe_cache_workspace_bytes(const moe_cache_shape_t* shape) {
  return cache_supported(shape) ? cache_ws_bytes(shape) : 0;
}

moe_status_t moe_cache_fork(const moe_cache_shape_t* shape, const moe_cache_meta_t* in,
                            const int32_t* parent_dev, const int32_t* keep_dev,
                            const moe_cache_meta_t* out, void* ws_dev, size_t ws_bytes,
                            moe_stream_t stream) {
  if (!cache_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!metas_ok(in, out) || !ints(parent_dev) || !aligned(keep_dev, 4)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  return done(launch_cache_fork(shape, *in, *out, parent_dev, keep_dev,
                                static_cast<uint8_t*>(ws_dev), (cudaStream_t)stream),
              "cache fork launch");
}

moe_status_t moe_cache_reserve(const moe_cache_shape_t* shape, const moe_cache_meta_t* in,
                               const int32_t* n_new_dev, const moe_cache_meta_t* out,
                               int32_t* granted_dev, void* const* pools_host, int32_t n_pools,
                               void* ws_dev, size_t ws_bytes, moe_stream_t stream) {
  if (!cache_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  CachePools pools;
  if (!metas_ok(in, out) || !ints(n_new_dev) || !ints(granted_dev) ||
      !pools_ok(pools_host, n_pools, &pools))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  return done(launch_cache_reserve(shape, *in, *out, n_new_dev, granted_dev, pools,
                                   static_cast<uint8_t*>(ws_dev), nsm, (cudaStream_t)stream),
              "cache reserve launch");
}

moe_status_t moe_cache_write(const moe_cache_shape_t* shape, const moe_cache_meta_t* meta,
                             const int32_t* n_new_dev, int32_t T, const void* k_new_dev,
                             int64_t k_stride, const void* v_new_dev, int64_t v_stride,
                             void* k_cache_dev, void* v_cache_dev, void* ws_dev, size_t ws_bytes,
                             moe_stream_t stream) {
  if (!cache_supported(shape) || T < 1 || T > (1 << 18)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t row = (int64_t)shape->n_kv * shape->D;
  if (!meta_ok(meta) || !aligned(n_new_dev, 4) || !k_new_dev || !v_new_dev || !k_cache_dev ||
      !v_cache_dev || !aligned(k_new_dev, 16) || !aligned(v_new_dev, 16) ||
      !aligned(k_cache_dev, 16) || !aligned(v_cache_dev, 16) || k_stride < row || v_stride < row ||
      k_stride % 8 || v_stride % 8)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  return done(launch_cache_write(shape, *meta, n_new_dev, T,
                                 static_cast<const uint16_t*>(k_new_dev), k_stride,
                                 static_cast<const uint16_t*>(v_new_dev), v_stride, k_cache_dev,
                                 v_cache_dev, static_cast<uint8_t*>(ws_dev), (cudaStream_t)stream),
              "cache write launch");
}

moe_status_t moe_cache_compact(const moe_cache_shape_t* shape, const moe_cache_meta_t* in,
                               const moe_cache_meta_t* out, int32_t* n_live_dev,
                               void* const* pools_host, int32_t n_pools, void* ws_dev,
                               size_t ws_bytes, moe_stream_t stream) {
  return moe_cache_compact_map(shape, in, out, n_live_dev, nullptr, pools_host, n_pools, ws_dev,
                               ws_bytes, stream);
}

moe_status_t moe_cache_compact_map(const moe_cache_shape_t* shape, const moe_cache_meta_t* in,
                                   const moe_cache_meta_t* out, int32_t* n_live_dev,
                                   int32_t* moved_dev, void* const* pools_host, int32_t n_pools,
                                   void* ws_dev, size_t ws_bytes, moe_stream_t stream) {
  if (!cache_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  CachePools pools;
  if (!metas_ok(in, out) || !ints(n_live_dev) || !aligned(moved_dev, 4) ||
      !pools_ok(pools_host, n_pools, &pools))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  return done(launch_cache_compact(shape, *in, *out, n_live_dev, moved_dev, pools,
                                   static_cast<uint8_t*>(ws_dev), nsm, (cudaStream_t)stream),
              "cache compact launch");
}

moe_status_t moe_cache_copy_pages(const moe_cache_shape_t* shape, int32_t n,
                                  const int32_t* src_dev, const int32_t* dst_dev,
                                  void* const* from_host, void* const* to_host, int32_t n_pools,
                                  int32_t n_to, void* ws_dev, size_t ws_bytes,
                                  moe_stream_t stream) {
  if (!cache_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  CachePools from, to;
  if (n < 1 || n_to < 1 || n_pools < 1 || !ints(src_dev) || !ints(dst_dev) ||
      !pools_ok(from_host, n_pools, &from) || !pools_ok(to_host, n_pools, &to))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  return done(launch_cache_copy_pages(shape, n, src_dev, dst_dev, from, to, n_to,
                                      static_cast<uint8_t*>(ws_dev), nsm, (cudaStream_t)stream),
              "cache page copy launch");
}

size_t moe_attn_batch_workspace_bytes(const moe_attn_batch_shape_t* shape) {
  return attn_batch_supported(shape) ? attn_batch_ws_bytes(shape) : 0;
}

moe_status_t moe_attn_batch(const moe_attn_batch_shape_t* shape, const void* q_dev,
                            int64_t q_stride, const void* k_cache_dev, const void* v_cache_dev,
                            int32_t n_phys, const int32_t* table_dev, const int32_t* prefix_dev,
                            const int32_t* lens_dev, const int32_t* n_new_dev, void* o_dev,
                            void* ws_dev, size_t ws_bytes, moe_stream_t stream) {
  if (!attn_batch_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!q_dev || !k_cache_dev || !v_cache_dev || !o_dev || !aligned(q_dev, 16) ||
      !aligned(k_cache_dev, 16) || !aligned(v_cache_dev, 16) || !aligned(o_dev, 16) ||
      q_stride < (int64_t)shape->n_q * shape->D || q_stride % 8 || !ints(table_dev) ||
      !ints(lens_dev) || !aligned(n_new_dev, 4) || !aligned(prefix_dev, 4) ||
      (shape->prefix_blocks > 0 && !prefix_dev) || n_phys < 1 ||
      // rows of the pools, one page past the end too, are counted in 32 bits
      ((int64_t)n_phys + 1) * shape->n_kv * shape->block > INT32_MAX)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, attn_batch_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  const uint64_t rows = (uint64_t)n_phys * shape->n_kv * shape->block;
  const bool fp16 = shape->dtype == MOE_DTYPE_FP16;
  CUtensorMap tk, tv;
  MOE_TRY(encode_rows64(&tk, fp16, k_cache_dev, shape->D, rows));
  MOE_TRY(encode_rows64(&tv, fp16, v_cache_dev, shape->D, rows));
  AttnBatchArgs a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.q_stride = q_stride;
  a.table = table_dev;
  a.prefix = prefix_dev;
  a.lens = lens_dev;
  a.n_new = n_new_dev;
  a.n_phys = n_phys;
  a.o = static_cast<uint16_t*>(o_dev);
  return done(launch_attn_batch(shape, tk, tv, a, static_cast<uint8_t*>(ws_dev), nsm,
                                (cudaStream_t)stream),
              "batch attention launch");
}

size_t moe_verify_workspace_bytes(const moe_verify_shape_t* shape) {
  return verify_supported(shape) ? verify_ws_bytes(shape) : 0;
}

moe_status_t moe_verify_drafts(const moe_verify_shape_t* shape, const void* p_dev,
                               const void* q_dev, const int32_t* draft_dev,
                               const int32_t* n_draft_dev, const float* u_dev,
                               int32_t* tokens_dev, int32_t* n_acc_dev, void* ws_dev,
                               size_t ws_bytes, moe_stream_t stream) {
  if (!verify_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t e = shape->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!p_dev || !aligned(p_dev, e) || !aligned(q_dev, e) || !ints(draft_dev) ||
      !aligned(n_draft_dev, 4) || !ints(u_dev) || !ints(tokens_dev) || !ints(n_acc_dev))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, verify_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  return done(launch_verify(shape, p_dev, q_dev, draft_dev, n_draft_dev, u_dev, tokens_dev,
                            n_acc_dev, static_cast<uint8_t*>(ws_dev), nsm, (cudaStream_t)stream),
              "draft verification launch");
}

int32_t moe_cache_q4_units(int32_t D) { return q4_units(D); }

moe_status_t moe_cache_write_q4(const moe_cache_shape_t* shape, const moe_cache_meta_t* meta,
                                const int32_t* n_new_dev, int32_t T, int32_t dtype,
                                const void* k_new_dev, int64_t k_stride, const void* v_new_dev,
                                int64_t v_stride, void* k_cache_dev, void* v_cache_dev,
                                void* ws_dev, size_t ws_bytes, moe_stream_t stream) {
  if (!cache_q4_supported(shape) || T < 1 || T > (1 << 18)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t row = (int64_t)shape->n_kv * shape->D;
  if (!meta_ok(meta) || !aligned(n_new_dev, 4) || !k_new_dev || !v_new_dev || !k_cache_dev ||
      !v_cache_dev || !aligned(k_new_dev, 16) || !aligned(v_new_dev, 16) ||
      !aligned(k_cache_dev, 16) || !aligned(v_cache_dev, 16) || k_stride < row || v_stride < row ||
      k_stride % 8 || v_stride % 8)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  return done(launch_cache_write_q4(shape, *meta, n_new_dev, T,
                                    static_cast<const uint16_t*>(k_new_dev), k_stride,
                                    static_cast<const uint16_t*>(v_new_dev), v_stride,
                                    dtype == MOE_DTYPE_FP16, k_cache_dev, v_cache_dev,
                                    static_cast<uint8_t*>(ws_dev), (cudaStream_t)stream),
              "4-bit cache write launch");
}

moe_status_t moe_cache_read_q4(const moe_cache_shape_t* shape, const moe_cache_meta_t* meta,
                               const int32_t* first_dev, const int32_t* n_dev, int32_t T,
                               const void* k_cache_dev, const void* v_cache_dev, int32_t dtype,
                               void* k_out_dev, int64_t k_stride, void* v_out_dev,
                               int64_t v_stride, void* ws_dev, size_t ws_bytes,
                               moe_stream_t stream) {
  if (!cache_q4_supported(shape) || T < 1 || T > (1 << 18)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dtype < MOE_DTYPE_BF16 || dtype > MOE_DTYPE_FP32) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t row = (int64_t)shape->n_kv * shape->D;
  const int64_t per = dtype == MOE_DTYPE_FP32 ? 4 : 8;  // elements of 16 bytes
  if (!meta_ok(meta) || !aligned(first_dev, 4) || !aligned(n_dev, 4) || !k_cache_dev ||
      !v_cache_dev || !k_out_dev || !v_out_dev || !aligned(k_cache_dev, 16) ||
      !aligned(v_cache_dev, 16) || !aligned(k_out_dev, 16) || !aligned(v_out_dev, 16) ||
      k_stride < row || v_stride < row || k_stride % per || v_stride % per)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, cache_ws_bytes(shape)));
  return done(launch_cache_read_q4(shape, *meta, first_dev, n_dev, T, k_cache_dev, v_cache_dev,
                                   k_out_dev, k_stride, v_out_dev, v_stride, dtype,
                                   static_cast<uint8_t*>(ws_dev), (cudaStream_t)stream),
              "4-bit cache read launch");
}

size_t moe_attn_batch_q4_workspace_bytes(const moe_attn_batch_shape_t* shape) {
  return attn_q4_supported(shape) ? attn_q4_ws_bytes(shape) : 0;
}

moe_status_t moe_attn_batch_q4(const moe_attn_batch_shape_t* shape, const void* q_dev,
                               int64_t q_stride, const void* k_cache_dev, const void* v_cache_dev,
                               int32_t n_phys, const int32_t* table_dev, const int32_t* lens_dev,
                               const int32_t* n_new_dev, void* o_dev, void* ws_dev,
                               size_t ws_bytes, moe_stream_t stream) {
  if (!attn_q4_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!q_dev || !k_cache_dev || !v_cache_dev || !o_dev || !aligned(q_dev, 16) ||
      !aligned(k_cache_dev, 16) || !aligned(v_cache_dev, 16) || !aligned(o_dev, 16) ||
      q_stride < (int64_t)shape->n_q * shape->D || q_stride % 8 || !ints(table_dev) ||
      !ints(lens_dev) || !aligned(n_new_dev, 4) || n_phys < 1)
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, attn_q4_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  AttnQ4Args a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.q_stride = q_stride;
  a.k = static_cast<const char*>(k_cache_dev);
  a.v = static_cast<const char*>(v_cache_dev);
  a.table = table_dev;
  a.lens = lens_dev;
  a.n_new = n_new_dev;
  a.n_phys = n_phys;
  a.o = static_cast<uint16_t*>(o_dev);
  return done(launch_attn_q4(shape, a, static_cast<uint8_t*>(ws_dev), nsm, (cudaStream_t)stream),
              "4-bit batch attention launch");
}

size_t moe_logprobs_workspace_bytes(const moe_logprobs_shape_t* shape) {
  return logprobs_supported(shape) ? logprobs_ws_bytes(shape) : 0;
}

moe_status_t moe_token_logprobs(const moe_logprobs_shape_t* shape, const void* logits_dev,
                                int64_t stride, const int32_t* tokens_dev, float* logp_dev,
                                float* entropy_dev, int32_t* top_ids_dev, float* top_logp_dev,
                                void* ws_dev, size_t ws_bytes, moe_stream_t stream) {
  if (!logprobs_supported(shape)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t e = shape->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!logits_dev || !aligned(logits_dev, e) || stride < shape->V || !ints(tokens_dev) ||
      !ints(logp_dev) || !aligned(entropy_dev, 4) || !aligned(top_ids_dev, 4) ||
      !aligned(top_logp_dev, 4))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(ws_dev, ws_bytes, logprobs_ws_bytes(shape)));
  int nsm = 0;
  MOE_TRY(device_sm_count(&nsm));
  return done(launch_logprobs(shape, logits_dev, stride, tokens_dev, logp_dev, entropy_dev,
                              top_ids_dev, top_logp_dev, static_cast<uint8_t*>(ws_dev), nsm,
                              (cudaStream_t)stream),
              "log probabilities launch");
}

}  // extern "C"

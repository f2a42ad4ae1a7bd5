// Internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "moe_w4.h"

namespace moe {

struct Ctrl;

constexpr int kPlanChunk = 256;         // routed rows per plan block (workspace path)
constexpr int kPlanChunkNoalloc = 2048; // routed rows per plan block (moe_plan_noalloc)

// Arguments of one grouped W4A16 GEMM launch (gate_up or down).
struct FfnArgs {
  const int32_t* block_map;    // [max_blocks][3] (expert, row_start, nrows)
  const int32_t* num_blocks;   // device count of block-map entries
  const int32_t* sorted_rows;  // unused by the kernel (the operand rows come in plan order)
  int K;                       // experts per token
  int R;                       // routed rows (T*K)
  int E;                       // routed experts; entry expert E = shared
  int rows_per_expert;         // weight rows per expert (2I or H)
  int half_rows;               // gate_up: I (first up row); down: 0
  int mtiles;                  // unit tiles per entry (gate_up: 64 gate + 64 up rows; down: 128 rows)
  int kdim;                    // reduction length (H for gate_up, I for down)
  int kgroups;                 // 64-wide groups per weight row (Kdim / 64)
  const uint16_t* s_exp;       // [E][rows][kgroups] bf16 scales
  const uint16_t* b_exp;       // [E][rows][kgroups] bf16 biases
  const uint16_t* s_sh;        // shared expert [rows][kgroups]
  const uint16_t* b_sh;
  uint16_t* out;               // bf16 [S][out_ld]
  int out_ld;
  Ctrl* ctrl;
  int max_units;               // host bound on units
  int shared_blocks;           // block-map entries of the shared expert (the last ones)
};

// Arguments of the fused decode layer (decode.cu): every pointer device,
// ids / w / logits / h / part in the workspace or the caller's buffers.
constexpr int kDecodeMaxT = 4;  // moe_layer_w4 takes the decode kernels up to this T
struct DecodeArgs {
  const uint16_t* x;    // bf16 [T][H]
  const uint16_t* wr;   // bf16 [E][H]
  const float* bias;    // [E] or null
  int T, H, E, K, I, ns;
  moe_w4_weights_t ex;  // routed experts
  moe_w4_weights_t sh;  // shared expert (used when ns == 1)
  float* logits;        // [T][E]
  int32_t* ids;         // [T][K]
  float* w;             // [T][K]
  uint16_t* h;          // bf16 [T][K+ns][I]
  uint16_t* y;          // bf16 [T][H]
  uint16_t* x_next;     // bf16 [T][H] or null
  float* part;          // [decode_part_floats(T, H)]
  Ctrl* ctrl;
  // stacked layers (moe_decode_layers): with y_prev, the input is
  // bf16(y_prev * inv) with inv from part_prev (the previous layer's block
  // partials, nb_prev per token) instead of x; with has_next, dec_down writes
  // its block partials for the next layer
  const uint16_t* y_prev;
  const float* part_prev;
  int nb_prev;
  int has_next;
};
bool decode_supported(int T, int H, int E, int K, int I, int ns);
size_t decode_part_floats(int T, int H);
cudaError_t launch_decode_layer(const DecodeArgs& a, cudaStream_t stream);

// Persistent decode through stacked layers (decode_persist.cu): one
// cooperative launch runs up to kPersistMaxLayers layers.
constexpr int kPersistMaxLayers = 48;
struct PersistArgs {
  int T, H, E, K, I, ns, n_layers;
  const uint16_t* x;    // bf16 [T][H]: the first layer's input
  uint16_t* y;          // bf16 [T][H]: the last layer's output
  uint16_t* x_next;     // bf16 [T][H] or null: its unit-RMS normalisation
  int32_t* ids;         // [T][K]: routing of the last layer
  float* w;             // [T][K]
  // cross-block words (epoch << 32 | payload), laid out by persist_tags():
  // 16-word lines, each written by one warp
  uint64_t* logits_tag; // line t*E+e: word 0 = fp32 logit
  uint64_t* h_tag;      // line per gate_up tile: words 4 col + r = bf16 pair (h_r, h_r+4)
  uint64_t* y_tag;      // line t*(H/8)+g: words 0..3 = bf16 pairs (y_r, y_r+4), word 4 = y^2 partial
  Ctrl* ctrl;
  // decoder blocks (moe_decoder_blocks) when block != 0: layer l's input is
  // bf16(gain[l] * h_l / rms(h_l)) and its output h_{l+1} = bf16(h_l + y_l)
  // (y is then h, the residual stream; x_next must be null); h_0 is
  // embed[tok[t]] when tok is set (ids outside [0, vocab) are recorded and
  // read as zero rows), else x
  int block;
  const int32_t* tok;
  const uint16_t* embed;
  int vocab;
  const uint16_t* gain[kPersistMaxLayers];
  moe_layer_weights_t layer[kPersistMaxLayers];
};
bool persist_supported(int T, int H, int E, int K, int I, int ns);
// Word offsets of the three tagged buffers in one region, and its size.
struct PersistTags {
  size_t logits, h, y, total;
};
PersistTags persist_tags(int T, int H, int E, int K, int I, int ns);
// Grid and dynamic shared memory of a launch on the current device; false
// when the shape's blocks do not fit on it (the caller takes the per-layer
// kernels then).
// block: room for the residual stream too (decoder blocks)
bool persist_config(int T, int H, int E, int K, int I, int ns, int* grid, size_t* smem,
                    bool block = false);
cudaError_t launch_decode_persist(const PersistArgs& a, int grid, size_t smem,
                                  cudaStream_t stream);

// Tensor-core screened router (route_tc.cu), taken from this many tokens on.
constexpr int kRouteTcMinT = 64;
bool route_tc_supported(int T, int H, int E, int K);
size_t route_tc_partial_floats(int T, int H, int E);
cudaError_t launch_route_tc(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const uint16_t* x,
                            const uint16_t* wr, const float* bias, int T, int H, int E, int K,
                            float* part, int32_t* ids, float* w, Ctrl* ctrl, cudaStream_t stream,
                            int32_t* hist = nullptr, int chunk = 0);

cudaError_t launch_route(const uint16_t* x, const uint16_t* wr, const float* bias, int T, int H,
                         int E, int K, float* logits, int32_t* ids, float* w,
                         cudaStream_t stream);
cudaError_t launch_plan(const int32_t* ids, int T, int K, int E, int n_shared, int BM,
                        const moe_plan_t& plan, int32_t* hist, Ctrl* ctrl, int chunk,
                        cudaStream_t stream, bool hist_ready = false);
cudaError_t launch_ffn_gate_up(const CUtensorMap& tw, const CUtensorMap& twsh,
                               const CUtensorMap& tx, const FfnArgs& a, int grid,
                               cudaStream_t stream);
cudaError_t launch_ffn_down(const CUtensorMap& tw, const CUtensorMap& twsh, const CUtensorMap& th,
                            const FfnArgs& a, int grid, cudaStream_t stream);
// xs[p] = x row of plan row p (routed rows through sorted_rows, then the
// shared expert's rows in token order), S rows of H bf16
cudaError_t launch_gather_x(const uint16_t* x, const int32_t* sorted_rows, int K, int R, int S,
                            int T, int H, uint16_t* xs, Ctrl* ctrl, int nsm, cudaStream_t stream);
// h_out set: decoder blocks (h_out = bf16(h_in + y), x_next of h_out with
// gain); y may then be null
cudaError_t launch_combine(const uint16_t* y_slots, const int32_t* row_pos, const float* w, int T,
                           int H, int K, int n_shared, uint16_t* y, uint16_t* x_next,
                           cudaStream_t stream, const uint16_t* h_in = nullptr,
                           uint16_t* h_out = nullptr, const uint16_t* gain = nullptr);
// The first decoder block's h_0 (h_in, or the embedding rows of tok copied to
// h0_out) and its input x = bf16(gain * h_0 / rms(h_0)).
cudaError_t launch_block_input(const uint16_t* h_in, const int32_t* tok, const uint16_t* embed,
                               int vocab, const uint16_t* gain, int T, int H, uint16_t* h0_out,
                               uint16_t* x, Ctrl* ctrl, cudaStream_t stream);
// decode_routine: the decode kernels' dequant_word_i4 (pairs put back into
// natural order) instead of the grouped GEMMs' dequant_word
cudaError_t launch_dequant(const uint32_t* q, const uint16_t* s, const uint16_t* b, uint16_t* out,
                           int N, int Kd, bool decode_routine, cudaStream_t stream);
// Grouped-query decode attention over a block-paged cache (attn_decode.cu).
bool attn_supported(const moe_attn_shape_t* s);
size_t attn_part_floats(const moe_attn_shape_t* s);
// tm_k / tm_v: the caches as [n_phys * n_kv * 64 rows][D] bf16, boxes of
// 64 rows x 64 elements, 128-byte swizzle
cudaError_t launch_attn_decode(const moe_attn_shape_t* s, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const uint16_t* q, const int32_t* table,
                               int n_phys, uint16_t* o, float* part, Ctrl* ctrl, int nsm,
                               cudaStream_t stream);
// Gated delta rule scan (gdn_scan.cu).
bool gdn_supported(const moe_gdn_shape_t* s);
cudaError_t launch_gdn_scan(const moe_gdn_shape_t* s, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const float* alpha, const float* beta,
                            const float* s_in, float* s_out, uint16_t* o, cudaStream_t stream);
// Chunked form of the same rule (gdn_chunk.cu): workspace bytes, launch.
size_t gdn_chunk_ws_bytes(const moe_gdn_shape_t* s);
cudaError_t launch_gdn_chunked(const moe_gdn_shape_t* s, const uint16_t* q, const uint16_t* k,
                               const uint16_t* v, const float* alpha, const float* beta,
                               const float* s_in, float* s_out, uint16_t* o, float* ws,
                               cudaStream_t stream);
// Pages of a block-paged cache (cache.cu). Pools: device pointers of one
// launch's keys and values, [n_phys][n_kv][64][D] 16-bit each.
constexpr int kMaxPools = 128;
struct CachePools {
  void* p[kMaxPools];
  int n;
};
bool cache_supported(const moe_cache_shape_t* s);
size_t cache_ws_bytes(const moe_cache_shape_t* s);
cudaError_t launch_cache_fork(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                              const moe_cache_meta_t& out, const int32_t* parent,
                              const int32_t* keep, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_cache_reserve(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                                 const moe_cache_meta_t& out, const int32_t* n_new,
                                 int32_t* granted, const CachePools& pools, uint8_t* ws, int nsm,
                                 cudaStream_t stream);
cudaError_t launch_cache_write(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                               const int32_t* n_new, int T, const uint16_t* k_new,
                               int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                               void* k_cache, void* v_cache, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_cache_compact(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                                 const moe_cache_meta_t& out, int32_t* n_live, int32_t* moved,
                                 const CachePools& pools, uint8_t* ws, int nsm,
                                 cudaStream_t stream);
cudaError_t launch_cache_copy_pages(const moe_cache_shape_t* s, int n, const int32_t* src,
                                    const int32_t* dst, const CachePools& from,
                                    const CachePools& to, int n_to, uint8_t* ws, int nsm,
                                    cudaStream_t stream);
// The shared part's line (attn_prefix.cu): pairs of 256 rows and a head, each
// with `steps` steps of 128 prefix positions on `len` units; `per` units a CTA.
struct PrefixLine {
  int pairs, steps, len, per, grid;
};
// Attention of a batch of slots (attn_batch.cu).
struct AttnBatchArgs {
  const uint16_t* q;   // token (s, t) starts at q_stride * (s * T + t)
  int64_t q_stride;
  const int32_t* table;   // [n_slots][max_blocks]
  const int32_t* prefix;  // [prefix_blocks]: pages of the first blocks of every slot
  const int32_t* lens;    // [n_slots]
  const int32_t* n_new;   // [n_slots] or null: T
  int n_slots, T, n_q, n_kv, max_blocks, prefix_blocks, n_phys;
  int first;           // the first block that attn_own_kernel takes
  uint16_t* o;         // [n_slots][T][n_q][D]
  float* part;         // parts of pairs: per place m[R], l[R], O[D / 4][R][4]
  unsigned* count;     // [CTAs of the own line]: arrivals at the pair that the CTA's end cuts
  int pair_cost;       // units of the own line that a pair counts beside its blocks
  int32_t* pair_start; // [n_slots][n_kv]: where the pair starts on the own line
  int32_t* line;       // [3]: units per CTA of the own line and of the shared part's, and a
                       // pair's length on that
  int32_t* tok_start;  // [n_slots]: tokens (t < n_new) of the slots before
  // the shared part, when attn_prefix_kernel takes it (px_steps > 0): its
  // line of steps and its parts, per place m[256], l[256], O[D / 4][256][4]
  int px_steps;
  int sms;             // that the shared part and the own one divide between them
  int px_most;         // CTAs that the shared part was launched with
  int px_fixed;        // that is the size, whatever the lengths
  float unit_weight;   // a unit of the own line, against a step of the shared part's
  int join;            // attn_join_kernel follows
  int parts;           // about how many parts a row then has
  float* px_part;
  Ctrl* ctrl;
};
PrefixLine prefix_line(const moe_attn_batch_shape_t* s, int sms);
size_t prefix_part_floats(const moe_attn_batch_shape_t* s, int sms);
cudaError_t launch_attn_prefix(const moe_attn_batch_shape_t* s, const CUtensorMap& tk,
                               const CUtensorMap& tv, const AttnBatchArgs& a, int grid,
                               cudaStream_t stream);
bool attn_batch_supported(const moe_attn_batch_shape_t* s);
size_t attn_batch_ws_bytes(const moe_attn_batch_shape_t* s);
cudaError_t launch_attn_batch(const moe_attn_batch_shape_t* s, const CUtensorMap& tk,
                              const CUtensorMap& tv, AttnBatchArgs a, uint8_t* ws, int nsm,
                              cudaStream_t stream);
// Rows of a cache in 4 bits (cache_q4.cu) and attention over them (attn_q4.cu).
struct AttnQ4Args;
bool cache_q4_supported(const moe_cache_shape_t* s);
cudaError_t launch_cache_write_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                  const int32_t* n_new, int T, const uint16_t* k_new,
                                  int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                                  bool fp16, void* k, void* v, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_cache_read_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                 const int32_t* first, const int32_t* n, int T, const void* k,
                                 const void* v, void* k_out, int64_t k_stride, void* v_out,
                                 int64_t v_stride, int dtype, uint8_t* ws, cudaStream_t stream);
bool attn_q4_supported(const moe_attn_batch_shape_t* s);
size_t attn_q4_ws_bytes(const moe_attn_batch_shape_t* s);
cudaError_t launch_attn_q4(const moe_attn_batch_shape_t* s, AttnQ4Args a, uint8_t* ws, int nsm,
                           cudaStream_t stream);
// Log probabilities of given tokens (logprobs.cu).
bool logprobs_supported(const moe_logprobs_shape_t* s);
size_t logprobs_ws_bytes(const moe_logprobs_shape_t* s);
cudaError_t launch_logprobs(const moe_logprobs_shape_t* s, const void* logits, int64_t stride,
                            const int32_t* tokens, float* logp, float* entropy, int32_t* top_ids,
                            float* top_logp, uint8_t* ws, int nsm, cudaStream_t stream);
// Verification of drafted tokens (verify.cu).
bool verify_supported(const moe_verify_shape_t* s);
size_t verify_ws_bytes(const moe_verify_shape_t* s);
cudaError_t launch_verify(const moe_verify_shape_t* s, const void* p, const void* q,
                          const int32_t* draft, const int32_t* n_draft, const float* u,
                          int32_t* tokens, int32_t* n_acc, uint8_t* ws, int nsm,
                          cudaStream_t stream);
// Host helpers shared by the C-ABI translation units (api.cu keeps the state).
bool shape_supported(const moe_shape_t* shape);
void set_last_error(const char* text);
void set_last_cuda_error(cudaError_t e, const char* where);
// SMs of the current device, and the tensor map of `rows` dense rows of D
// 16-bit elements in boxes of 64 rows x 64 elements (128-byte swizzle)
moe_status_t device_sm_count(int* out);
moe_status_t encode_rows64(CUtensorMap* m, bool fp16, const void* base, int D, uint64_t rows);
int ffn_tile_m();
int ffn_max_tile_n();
int ffn_stage_k();
int ffn_b_box_rows();

}  // namespace moe

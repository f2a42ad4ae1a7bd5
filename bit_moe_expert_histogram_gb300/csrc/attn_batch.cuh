// What the kernels of the batch's attention share: the launch arguments, the
// slots' spans and the arithmetic of the two 16-bit types.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kBlk = 64;  // positions per page

// How `pairs` pairs of `steps` steps go over `ctas` CTAs. Cut evenly, most
// CTAs get the end of one pair and the start of the next, and a stretch costs
// about kStretch steps beside its own (queries in, O out); cut pair by pair
// every CTA has one stretch but some CTAs may be left over. The shorter way
// is taken; a stretch of fewer than two steps would be mostly cost.
__host__ __device__ inline PrefixLine prefix_cut(int pairs, int steps, int ctas) {
  constexpr int kStretch = 3;
  PrefixLine p;
  p.pairs = pairs;
  p.steps = steps;
  p.len = steps;
  // below 2^31: the calls' 2^30 blocks in all, and ctas
  p.per = (int)(((unsigned)pairs * (unsigned)steps + ctas - 1) / (unsigned)ctas);
  p.grid = ctas;
  if (pairs > 0 && pairs <= ctas) {
    const unsigned each = (unsigned)ctas / (unsigned)pairs;
    int per = (int)((steps + each - 1) / each);
    per = per < 2 ? 2 : per;
    if (per <= p.per + kStretch) {
      const int cuts = (int)((unsigned)(steps + per - 1) / (unsigned)per);
      p.per = per;
      p.len = cuts * per;
      p.grid = pairs * cuts;
    }
  }
  if (p.per < 1) p.per = 1;
  return p;
}

// New tokens of a slot, brought into range.
__device__ __forceinline__ int slot_tokens(const AttnBatchArgs& a, int s) {
  return a.n_new ? min(max(__ldg(a.n_new + s), 0), a.T) : a.T;
}

// What a slot brings: its length, new tokens and own blocks (at least one, a
// block of nothing where it has none, so that each slot's rows get written).
struct SlotSpan {
  int len, n_new, blocks;
};
__device__ __forceinline__ SlotSpan slot_span(const AttnBatchArgs& a, int s) {
  SlotSpan r;
  r.len = __ldg(a.lens + s);
  r.n_new = a.n_new ? __ldg(a.n_new + s) : a.T;
  const int most = a.max_blocks * kBlk;
  if (r.len < 0 || r.len > most || r.n_new < 0 || r.n_new > a.T) {
    set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, s);
    r.len = min(max(r.len, 0), most);
    r.n_new = min(max(r.n_new, 0), a.T);
  }
  const int nb = (r.len + kBlk - 1) / kBlk - a.first;
  r.blocks = r.n_new == 0 || nb < 1 ? 1 : nb;
  return r;
}

// 16 bytes to shared memory, past the first `bytes` (0 or 16) zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ float unpack_lo(uint32_t v) {
  return F16 ? half_bits_to_float(v & 0xFFFFu) : bf_lo(v);
}
template <bool F16>
__device__ __forceinline__ float unpack_hi(uint32_t v) {
  return F16 ? half_bits_to_float(v >> 16) : bf_hi(v);
}
// log2 of the weights' scale: fp16 weights are kept at up to 2^lift so that
// small ones stay above its smallest normal value (2^-14); bf16 needs none
template <bool F16>
__device__ __forceinline__ constexpr float lift() {
  return F16 ? 6.0f : 0.0f;
}

}  // namespace moe

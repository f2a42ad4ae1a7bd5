// What the kernels of the batch's attention share: the launch arguments, the
// slots' spans and the arithmetic of the two 16-bit types.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kBlk = 64;  // positions per page

__host__ __device__ inline int cut_up(unsigned n, unsigned d) {  // ceil(n / d)
#ifdef __CUDA_ARCH__
  // several of these in a row keep the shared part's kernel waiting, and a
  // float quotient put right takes a third of a division's time (below 2^22
  // it is off by two at most)
  unsigned q = __float2uint_rd(__fdividef((float)n, (float)d));
  if (q >= (1u << 22)) return (int)((n + d - 1) / d);
  while (q * d > n) --q;
  while (q * d < n) ++q;
  return (int)q;
#else
  return (int)((n + d - 1) / d);
#endif
}
// How `pairs` pairs of `steps` steps go over `ctas` CTAs. Cut evenly, most
// CTAs get the end of one pair and the start of the next, and a stretch costs
// about kStretch steps beside its own (queries in, O out); cut pair by pair
// every CTA has one stretch but some CTAs may be left over. The shorter way
// is taken; a stretch of fewer than two steps would be mostly cost.
constexpr int kStretch = 3;
__host__ __device__ inline PrefixLine prefix_cut(int pairs, int steps, int ctas) {
  PrefixLine p;
  p.pairs = pairs;
  p.steps = steps;
  p.len = steps;
  // below 2^31: the calls' 2^30 blocks in all, and ctas
  p.per = cut_up((unsigned)pairs * (unsigned)steps, ctas);
  p.grid = ctas;
  if (pairs > 0 && pairs <= ctas) {
    int each = cut_up(ctas, pairs);  // rounded down from here on
    each -= each * pairs > ctas;
    int per = cut_up(steps, each);
    per = per < 2 ? 2 : per;
    if (per <= p.per + kStretch) {
      const int cuts = cut_up(steps, per);
      p.per = per;
      p.len = cuts * per;
      p.grid = pairs * cuts;
    }
  }
  if (p.per < 1) p.per = 1;
  return p;
}

// How the SMs are divided between the shared part (one CTA each) and the slots'
// own line of `units`, which only the lengths tell: the i-th of 32 ways, and
// how long the longer of both then takes, in steps. The last way cuts evenly,
// the others pair by pair. weight: of a unit on one SM, against a step; most:
// CTAs that the shared part can have.
constexpr int kPRows = 256;  // rows of a tile pair of the shared part
constexpr int kWays = 32;
struct PrefixWay {
  PrefixLine line;
  float time;
};
__host__ __device__ inline PrefixWay prefix_way(int i, int pairs, int steps, int units,
                                                float weight, int sms, int most) {
  const bool even = i == kWays - 1;
  const float own = (float)units * weight, px = (float)pairs * (float)(steps + kStretch);
  int ctas = (int)((float)sms * px / (px + own) + 0.5f);
  ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
  int cuts = cut_up(most + 1, pairs) - 1;  // most / pairs
  cuts = (i + 1) * cuts / (kWays - 1);
  PrefixWay r;
  r.line.pairs = pairs;
  r.line.steps = steps;
  int per = cut_up(even ? (unsigned)pairs * (unsigned)steps : steps, even ? ctas : cuts > 0 ? cuts : 1);
  per = per < 2 ? 2 : per;
  cuts = cut_up(steps, per);
  r.line.per = per;
  r.line.len = even ? steps : cuts * per;
  r.line.grid = even ? ctas : pairs * cuts;
  // an even cut has the ends of per / steps pairs more in a CTA
  const float ends = even ? kStretch * (1.0f + (float)per / (float)steps) : 0.0f;
  const float t = own / (float)(sms - r.line.grid), p = (float)per + ends;
  r.time = r.line.grid > most ? INFINITY : t > p ? t : p;
  return r;
}
#ifdef __CUDACC__
// The best way, asked by a whole warp, a way a lane. (Both kernels ask, each
// for itself; did they not agree, the balance alone would suffer.)
__device__ __forceinline__ PrefixLine best_line(const AttnBatchArgs& a, int n_tok, int units) {
  const int pairs = (n_tok * (a.n_q / a.n_kv) + kPRows - 1) / kPRows * a.n_kv, lane = threadIdx.x & 31;
  if (a.px_fixed || pairs == 0) return prefix_cut(pairs, a.px_steps, a.px_most);
  const PrefixWay w = prefix_way(lane, pairs, a.px_steps, units, a.unit_weight, a.sms, a.px_most);
  const unsigned key = (__float_as_uint(w.time) & ~31u) | lane;
  const int best = (int)(__reduce_min_sync(0xFFFFFFFFu, key) & 31u);
  PrefixLine p;
  p.pairs = pairs;
  p.steps = a.px_steps;
  p.len = __shfl_sync(0xFFFFFFFFu, w.line.len, best);
  p.per = __shfl_sync(0xFFFFFFFFu, w.line.per, best);
  p.grid = __shfl_sync(0xFFFFFFFFu, w.line.grid, best);
  return p;
}
#endif

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

#ifdef __CUDACC__
// v / l to four 16-bit elements, 0 where l is (a row that sees nothing), even
// if what was summed for it is not finite; a NaN sum stays one
template <bool F16>
__device__ __forceinline__ void store4(uint16_t* to, const float4& v, float l) {
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(to) =
      l == 0.0f ? make_uint2(0u, 0u)
                : make_uint2(pack2<F16>(v.x * inv, v.y * inv), pack2<F16>(v.z * inv, v.w * inv));
}

// Joins parts 0 .. n - 1 in order, each batch of up to kBatch fetched as a
// whole: part k has m at p, l at p + l_at and O at p + o_at for its p.
struct Joined {
  float M, L;
  float4 o;
};
struct PartRef {
  const float* p;
  int l_at, o_at;
};
template <int kBatch, typename At>
__device__ __forceinline__ void join_parts(Joined& j, int n, At at) {
  for (int c0 = 0; c0 < n; c0 += kBatch) {
    float m[kBatch], l[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.0f;
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c0 + k < n) {
        const PartRef r = at(c0 + k);
        m[k] = __ldcg(r.p);
        l[k] = __ldcg(r.p + r.l_at);
        v[k] = __ldcg(reinterpret_cast<const float4*>(r.p + r.o_at));
      }
    }
    float nM = j.M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) nM = fmaxf(nM, m[k]);
    const float U = nM == -INFINITY ? 0.0f : nM;
    const float f = ex2(j.M - U);
    j.L *= f;
    j.o.x *= f;
    j.o.y *= f;
    j.o.z *= f;
    j.o.w *= f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = ex2(m[k] - U);
      j.L = fmaf(l[k], w, j.L);
      j.o.x = fmaf(v[k].x, w, j.o.x);
      j.o.y = fmaf(v[k].y, w, j.o.y);
      j.o.z = fmaf(v[k].z, w, j.o.z);
      j.o.w = fmaf(v[k].w, w, j.o.w);
    }
    j.M = nM;
  }
}
#endif

}  // namespace moe

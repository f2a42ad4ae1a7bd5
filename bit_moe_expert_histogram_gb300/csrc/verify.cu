// Verification of drafted tokens against the target's probabilities, from
// given random numbers (speculative sampling): per slot with n drafts
//   draft t is accepted while u_t q_t(x_t) < p_t(x_t), i = the first that is
//   not (i = n when all are);
//   w = max(p_i - q_i, 0) where i < n (p_i where that is zero everywhere),
//   w = p_n where i = n;
//   the new token is the least v with w_0 + .. + w_v > u_T (w_0 + .. + w_{V-1}).
// Accepting so, and drawing the replacement from the clipped difference,
// leaves every token distributed as p.
//
// The token is a whole number that a rounding must not change, so nothing
// here rounds where it could: u q is formed in 64 bits (two 24-bit factors,
// exact), p - q as an fp32 pair without error, and the sums as fp32 pairs
// (value and error term, 48 bits) that are joined in 64 bits. FP64 runs at a
// few operations a clock per SM here, so it only joins threads.
//
// What it has to read is one row of p and one of q per slot: HBM bounds large
// batches, a chain of dependent accesses small ones. The vocabulary is cut
// into segments of 4096; a slot's C CTAs (four per SM over the batch, at most
// one per segment) each find i by themselves (a warp, one draft a lane: two
// dependent loads), sum their segments and leave the sums in the workspace.
// The slot's last CTA scans the segments' sums, re-reads the one segment that
// the threshold falls into (it is in L2) and walks it. A thread's sixteen
// values come in 16-byte loads, or in single ones, a warp's neighbours each,
// where a row is not 16-byte aligned (an odd vocabulary).
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {
constexpr int kVThr = 256;
constexpr int kVPer = 16;             // elements per thread
constexpr int kVSeg = kVThr * kVPer;  // elements per segment
constexpr int kVWarps = kVThr / 32;
constexpr int kVCtas = 4;             // CTAs an SM

template <int DT>
__device__ __forceinline__ float elem(const void* p, int64_t i) {
  if (DT == MOE_DTYPE_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t h = __ldg(static_cast<const uint16_t*>(p) + i);
  return DT == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : half_bits_to_float(h);
}
// 16 values of a segment (of n <= 4096), those at or past n read as 0.
// Walk: elements 16 tid .. 16 tid + 15. Otherwise each load of the warp takes
// neighbours, in 16-byte pieces where the row allows (`vec`).
template <int DT, bool Walk>
__device__ __forceinline__ int place(int k, bool vec) {
  if (Walk) return threadIdx.x * kVPer + k;
  constexpr int kPiece = DT == MOE_DTYPE_FP32 ? 4 : 8;
  return vec ? ((k / kPiece) * kVThr + threadIdx.x) * kPiece + k % kPiece : k * kVThr + threadIdx.x;
}
template <int DT>
__device__ __forceinline__ void load_piece(const void* p, float* x) {
  if (DT == MOE_DTYPE_FP32) {
    const float4 v = __ldg(static_cast<const float4*>(p));
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const uint4 v = __ldg(static_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = DT == MOE_DTYPE_BF16 ? bf_lo(w[j]) : half_bits_to_float(w[j] & 0xFFFFu);
      x[2 * j + 1] = DT == MOE_DTYPE_BF16 ? bf_hi(w[j]) : half_bits_to_float(w[j] >> 16);
    }
  }
}
template <int DT, bool Walk>
__device__ __forceinline__ void load16(const char* seg, int n, bool vec, float (&x)[kVPer]) {
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2, kPiece = 16 / kE;
  if (vec) {
#pragma unroll
    for (int k = 0; k < kVPer; k += kPiece) {
      const int at = place<DT, Walk>(k, true);
      if (at + kPiece <= n) {
        load_piece<DT>(seg + (int64_t)at * kE, x + k);
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) x[k + j] = at + j < n ? elem<DT>(seg, at + j) : 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      const int at = place<DT, Walk>(k, false);
      x[k] = at < n ? elem<DT>(seg, at) : 0.0f;
    }
  }
}

// s + e += x without error but for e's own rounding
__device__ __forceinline__ void add_pair(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x);
  const float z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// the same of two pairs
__device__ __forceinline__ void join_pair(float& s, float& e, float s2, float e2) {
  e = __fadd_rn(e, e2);
  add_pair(s, e, s2);
}

// a weight as a pair (hi, lo): max(p - q, 0), 0 where p - q is not finite
__device__ __forceinline__ void weight(float p, float q, float& hi, float& lo) {
  const float d = __fsub_rn(p, q);
  const float z = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, z)), __fadd_rn(q, z));
  const bool ok = d > 0.0f && d < INFINITY;
  hi = ok ? d : 0.0f;
  lo = ok ? e : 0.0f;
}

// inclusive scan of one double per thread over the CTA (fixed order)
__device__ double block_scan(double v, double* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  double base = 0.0;
  for (int w = 0; w < warp; ++w) base += warp_tot[w];
  return base + v;
}
}  // namespace

struct VerifyArgs {
  const void* p;
  const void* q;  // or null: the draft is certain
  const int32_t* draft;
  const int32_t* n_draft;  // or null: T
  const float* u;
  int32_t* tokens;
  int32_t* n_acc;
  int T, V, S;     // S segments
  double* part;    // [slot][S]: sums of the segments' weights
  unsigned* done;  // [slot]: CTAs finished
  Ctrl* ctrl;
};

// the two rows that a slot's weights come from
struct Rows {
  const char* p;
  const char* q;  // or null
  int cut;        // the certain draft's token, which has no weight left; -1: none
  bool vp, vq;    // 16-byte aligned
};
// weights (value and error term) of this thread's 16 elements of segment sg
template <int DT, bool Walk>
__device__ __forceinline__ void seg_load(const Rows& r, int V, int sg, float (&p)[kVPer],
                                         float (&q)[kVPer]) {
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2;
  const int v0 = sg * kVSeg, n = min(kVSeg, V - v0);
  // one arrangement for both rows: pieces only where both allow them
  const bool vec = r.vp && r.vq;
  load16<DT, Walk>(r.p + (int64_t)v0 * kE, n, vec, p);
  if (r.q) {
    load16<DT, Walk>(r.q + (int64_t)v0 * kE, n, vec, q);
  } else {
#pragma unroll
    for (int k = 0; k < kVPer; ++k) q[k] = v0 + place<DT, Walk>(k, vec) == r.cut ? p[k] : 0.0f;
  }
}
__device__ __forceinline__ void seg_sum(const float (&p)[kVPer], const float (&q)[kVPer], float& s,
                                        float& e) {
  s = 0.0f;
  e = 0.0f;
#pragma unroll
  for (int k = 0; k < kVPer; ++k) {
    float hi, lo;
    weight(p[k], q[k], hi, lo);
    add_pair(s, e, hi);
    e = __fadd_rn(e, lo);
  }
}

template <int DT>
__global__ void __launch_bounds__(kVThr, kVCtas) verify_kernel(const VerifyArgs a) {
  extern __shared__ float2 s_seg[];  // [this CTA's segments][warps]: sums as pairs
  __shared__ int s_i, s_n, s_bad_x, s_last, s_first, s_lastpos;
  __shared__ double s_tot[kVWarps];
  __shared__ double s_thr, s_base;
  const int b = blockIdx.y, tid = threadIdx.x, C = gridDim.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int T = a.T, V = a.V, S = a.S;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int n = a.n_draft ? __ldg(a.n_draft + b) : T;
    // the draft is read beside its count, not after it
    const int x = lane < T ? __ldg(a.draft + (int64_t)b * T + lane) : 0;
    const float u = lane < T ? __ldg(a.u + (int64_t)b * (T + 1) + lane) : 0.0f;
    if (n < 0 || n > T) {
      if (lane == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_VERIFY, b);
      n = n < 0 ? 0 : T;
    }
    bool ok = false, bad = false;
    if (lane < n) {
      bad = x < 0 || x >= V;
      if (!bad) {
        const float px = elem<DT>(a.p, ((int64_t)b * (T + 1) + lane) * V + x);
        const float qx = a.q ? elem<DT>(a.q, ((int64_t)b * T + lane) * V + x) : 1.0f;
        ok = (double)u * (double)qx < (double)px;
      }
    }
    const unsigned no = __ballot_sync(0xFFFFFFFFu, lane < n && !ok);
    const unsigned badm = __ballot_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      const int i = no ? __ffs(no) - 1 : n;
      s_i = i;
      s_n = n;
      s_bad_x = i < n && ((badm >> i) & 1u);
      if (badm) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_VERIFY, b);
    }
  }
  __syncthreads();
  const int i = s_i;
  const bool rejected = i < s_n;
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2;
  Rows r;
  r.p = static_cast<const char*>(a.p) + ((int64_t)b * (T + 1) + i) * V * kE;
  r.q = rejected && a.q ? static_cast<const char*>(a.q) + ((int64_t)b * T + i) * V * kE : nullptr;
  r.cut = rejected && !a.q && !s_bad_x ? __ldg(a.draft + (int64_t)b * T + i) : -1;
  r.vp = (reinterpret_cast<uintptr_t>(r.p) & 15u) == 0;
  r.vq = (reinterpret_cast<uintptr_t>(r.q) & 15u) == 0;
  // ---- the sums of segments c, c + C, ...
  {
    int k = 0;
    for (int sg = blockIdx.x; sg < S; sg += C, ++k) {
      float p[kVPer], q[kVPer], s, e;
      seg_load<DT, false>(r, V, sg, p, q);
      seg_sum(p, q, s, e);
#pragma unroll
      for (int d = 16; d; d >>= 1)
        join_pair(s, e, __shfl_xor_sync(0xFFFFFFFFu, s, d), __shfl_xor_sync(0xFFFFFFFFu, e, d));
      if (lane == 0) s_seg[k * kVWarps + warp] = make_float2(s, e);
    }
    __syncthreads();
    for (int j = tid; j < k; j += kVThr) {
      double sum = 0.0;
      for (int w = 0; w < kVWarps; ++w) {
        const float2 v = s_seg[j * kVWarps + w];
        sum += (double)v.x + (double)v.y;
      }
      a.part[(int64_t)b * S + (int)blockIdx.x + j * C] = sum;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      s_last = atomicAdd(a.done + b, 1u) == (unsigned)C - 1u;
      if (s_last) a.done[b] = 0u;  // ready for the next call
      __threadfence();
    }
    __syncthreads();
  }
  if (!s_last) return;
  // ---- the slot's last CTA: first the segment (one a thread: S <= 256)
  double mine = tid < S ? __ldcg(a.part + (int64_t)b * S + tid) : 0.0;
  double inc = block_scan(mine, s_tot);
  if (tid == kVThr - 1) s_base = inc;
  __syncthreads();
  if (!(s_base > 0.0) && rejected) {
    // nothing left of the difference: the target's own row, summed here (a
    // case of roundings, where q is nowhere below p)
    r.q = nullptr;
    r.cut = -1;
    r.vq = true;
    mine = 0.0;
    for (int sg = 0; sg < S; ++sg) {
      float p[kVPer], q[kVPer], s, e;
      seg_load<DT, false>(r, V, sg, p, q);
      seg_sum(p, q, s, e);
      const double t = block_scan((double)s + (double)e, s_tot);
      if (tid == kVThr - 1) s_base = t;
      __syncthreads();
      if (tid == sg) mine = s_base;
      __syncthreads();
    }
    inc = block_scan(mine, s_tot);
  }
  if (tid == kVThr - 1) {
    s_thr = (double)__ldg(a.u + (int64_t)b * (T + 1) + T) * inc;
    s_base = inc;  // the total, for now
    s_first = kVThr;
    s_lastpos = -1;
  }
  __syncthreads();
  const double thr = s_thr, total = s_base;
  // the first segment whose running sum passes the threshold; where none
  // does (u_T not below 1, or a rounding), the last one that weighs anything
  if (mine > 0.0) {
    if (inc > thr) atomicMin(&s_first, tid);
    atomicMax(&s_lastpos, tid);
  }
  __syncthreads();
  int token = -1;
  if (total > 0.0) {
    const int sg = s_first < kVThr ? s_first : s_lastpos;
    __syncthreads();
    if (tid == sg) s_base = inc - mine;
    if (tid == 0) {
      s_first = kVThr;
      s_lastpos = -1;
    }
    float p[kVPer], q[kVPer], s, e;
    seg_load<DT, true>(r, V, sg, p, q);
    seg_sum(p, q, s, e);
    const double own = (double)s + (double)e;
    const double upto = block_scan(own, s_tot);  // synchronises: s_base is set
    const double incl = s_base + upto;
    // then the thread, in the same way
    if (own > 0.0) {
      if (incl > thr) atomicMin(&s_first, tid);
      atomicMax(&s_lastpos, tid);
    }
    __syncthreads();
    if (tid == (s_first < kVThr ? s_first : s_lastpos)) {
      // then the element: the first that passes, or the thread's last that
      // weighs anything
      double run = incl - own;
      int at = 0;
      bool passed = false;
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        float hi, lo;
        weight(p[k], q[k], hi, lo);
        if (hi > 0.0f && !passed) {
          run += (double)hi + (double)lo;
          at = k;
          passed = run > thr;
        }
      }
      s_i = sg * kVSeg + tid * kVPer + at;
    }
    __syncthreads();
    token = s_i;
  } else if (tid == 0) {
    set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_VERIFY, b);  // a row without any weight
  }
  if (tid <= T) {
    const int64_t at = (int64_t)b * (T + 1) + tid;
    a.tokens[at] = tid < i ? __ldg(a.draft + (int64_t)b * T + tid) : tid == i ? token : -1;
    if (tid == 0) a.n_acc[b] = i;
  }
}

bool verify_supported(const moe_verify_shape_t* s) {
  if (!s) return false;
  if (s->n_slots < 1 || s->n_slots > 4096 || s->T < 1 || s->T > 31) return false;
  if (s->V < 1 || s->V > kVSeg * kVThr) return false;
  return s->dtype == MOE_DTYPE_BF16 || s->dtype == MOE_DTYPE_FP16 || s->dtype == MOE_DTYPE_FP32;
}

// 256 bytes of status, the slots' counters, the segments' sums
size_t verify_ws_bytes(const moe_verify_shape_t* s) {
  const size_t S = (s->V + kVSeg - 1) / kVSeg;
  return 256 + (((size_t)s->n_slots * 4 + 255) & ~(size_t)255) + (size_t)s->n_slots * S * 8;
}

cudaError_t launch_verify(const moe_verify_shape_t* s, const void* p, const void* q,
                          const int32_t* draft, const int32_t* n_draft, const float* u,
                          int32_t* tokens, int32_t* n_acc, uint8_t* ws, int nsm, cudaStream_t stream) {
  VerifyArgs a{};
  a.p = p;
  a.q = q;
  a.draft = draft;
  a.n_draft = n_draft;
  a.u = u;
  a.tokens = tokens;
  a.n_acc = n_acc;
  a.T = s->T;
  a.V = s->V;
  a.S = (s->V + kVSeg - 1) / kVSeg;
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  a.done = reinterpret_cast<unsigned*>(ws + 256);
  a.part = reinterpret_cast<double*>(ws + 256 + (((size_t)s->n_slots * 4 + 255) & ~(size_t)255));
  // each CTA with as many segments as four CTAs an SM leave it
  const int per_slot = (kVCtas * nsm + s->n_slots - 1) / s->n_slots;
  const int C = per_slot < a.S ? per_slot : a.S;
  const dim3 grid(C, s->n_slots);
  const size_t smem = (size_t)((a.S + C - 1) / C) * kVWarps * sizeof(float2);
  auto kern = s->dtype == MOE_DTYPE_FP32   ? verify_kernel<MOE_DTYPE_FP32>
              : s->dtype == MOE_DTYPE_BF16 ? verify_kernel<MOE_DTYPE_BF16>
                                           : verify_kernel<MOE_DTYPE_FP16>;
  return launch_pdl(kern, grid, dim3(kVThr), smem, stream, a);
}

}  // namespace moe

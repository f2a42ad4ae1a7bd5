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
// What it has to read is one row of p and one of q per slot. The vocabulary
// is cut into segments of 4096: CTA (segment, slot) finds i by itself (a
// warp, one draft a lane: two dependent loads), sums its segment and leaves
// the sums in the workspace; the slot's last CTA scans the segments' sums,
// re-reads the one segment that the threshold falls into (it is in L2) and
// walks it.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {
constexpr int kVThr = 256;
constexpr int kVPer = 16;             // elements per thread
constexpr int kVSeg = kVThr * kVPer;  // elements per segment
constexpr int kVWarps = kVThr / 32;

template <int DT>
__device__ __forceinline__ float elem(const void* p, int64_t i) {
  if (DT == MOE_DTYPE_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t h = __ldg(static_cast<const uint16_t*>(p) + i);
  return DT == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : half_bits_to_float(h);
}
// elements i .. i + 15 of a row, those at or past i + n read as 0; `vec`:
// the row starts on a 16-byte boundary (i is a multiple of 16)
template <int DT>
__device__ __forceinline__ void load16(const void* row, int i, int n, bool vec, float (&x)[kVPer]) {
  if (n >= kVPer && vec) {
    if (DT == MOE_DTYPE_FP32) {
      const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = __ldg(r + k);
        x[4 * k] = v.x;
        x[4 * k + 1] = v.y;
        x[4 * k + 2] = v.z;
        x[4 * k + 3] = v.w;
      }
    } else {
      const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 v = __ldg(r + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * k + 2 * j] =
              DT == MOE_DTYPE_BF16 ? bf_lo(w[j]) : half_bits_to_float(w[j] & 0xFFFFu);
          x[8 * k + 2 * j + 1] = DT == MOE_DTYPE_BF16 ? bf_hi(w[j]) : half_bits_to_float(w[j] >> 16);
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kVPer; ++k) x[k] = k < n ? elem<DT>(row, i + k) : 0.0f;
  }
}

// s + e += x without error but for e's own rounding
__device__ __forceinline__ void add_pair(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x);
  const float z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
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
  double* part;    // [slot][S][2]: sums of the difference and of p
  unsigned* done;  // [slot]: CTAs finished
  Ctrl* ctrl;
};

template <int DT>
__global__ void __launch_bounds__(kVThr) verify_kernel(const VerifyArgs a) {
  __shared__ int s_i, s_n, s_bad_x, s_last, s_seg, s_first, s_lastpos;
  __shared__ double s_tot[kVWarps], s_r[kVWarps], s_p[kVWarps];
  __shared__ double s_thr, s_base;
  const int b = blockIdx.y, seg = blockIdx.x, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int T = a.T, V = a.V, S = a.S;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int n = a.n_draft ? __ldg(a.n_draft + b) : T;
    if (n < 0 || n > T) {
      if (lane == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_VERIFY, b);
      n = n < 0 ? 0 : T;
    }
    bool ok = false, bad = false;
    if (lane < n) {
      const int x = __ldg(a.draft + (int64_t)b * T + lane);
      bad = x < 0 || x >= V;
      if (!bad) {
        const float px = elem<DT>(a.p, ((int64_t)b * (T + 1) + lane) * V + x);
        const float qx = a.q ? elem<DT>(a.q, ((int64_t)b * T + lane) * V + x) : 1.0f;
        ok = (double)__ldg(a.u + (int64_t)b * (T + 1) + lane) * (double)qx < (double)px;
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
  const char* prow = static_cast<const char*>(a.p) + ((int64_t)b * (T + 1) + i) * V * kE;
  const char* qrow = rejected && a.q
                         ? static_cast<const char*>(a.q) + ((int64_t)b * T + i) * V * kE
                         : nullptr;
  // the certain draft's own token has no weight left
  const int cut = rejected && !a.q && !s_bad_x ? __ldg(a.draft + (int64_t)b * T + i) : -1;
  const bool vp = (reinterpret_cast<uintptr_t>(prow) & 15u) == 0;
  const bool vq = (reinterpret_cast<uintptr_t>(qrow) & 15u) == 0;
  // this thread's 16 elements of segment sg: weights, their error terms, p
  float w[kVPer], we[kVPer], pw[kVPer];
  auto load = [&](int sg) {
    const int v0 = sg * kVSeg + tid * kVPer, n = V - v0;
    float q[kVPer];
    load16<DT>(prow, v0, n, vp, pw);
    if (qrow) {
      load16<DT>(qrow, v0, n, vq, q);
    } else {
#pragma unroll
      for (int k = 0; k < kVPer; ++k) q[k] = v0 + k == cut ? pw[k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      weight(pw[k], q[k], w[k], we[k]);
      pw[k] = pw[k] > 0.0f && pw[k] < INFINITY ? pw[k] : 0.0f;
    }
  };
  load(seg);
  float rs = 0.0f, re = 0.0f, qs = 0.0f, qe = 0.0f;
#pragma unroll
  for (int k = 0; k < kVPer; ++k) {
    add_pair(rs, re, w[k]);
    re = __fadd_rn(re, we[k]);
    add_pair(qs, qe, pw[k]);
  }
  double dr = (double)rs + (double)re, dp = (double)qs + (double)qe;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    dr += __shfl_xor_sync(0xFFFFFFFFu, dr, d);
    dp += __shfl_xor_sync(0xFFFFFFFFu, dp, d);
  }
  if (lane == 0) {
    s_r[warp] = dr;
    s_p[warp] = dp;
  }
  __syncthreads();
  if (tid == 0) {
    double r = 0.0, p = 0.0;
    for (int k = 0; k < kVWarps; ++k) {
      r += s_r[k];
      p += s_p[k];
    }
    double* out = a.part + ((int64_t)b * S + seg) * 2;
    out[0] = r;
    out[1] = p;
    __threadfence();
    s_last = atomicAdd(a.done + b, 1u) == (unsigned)S - 1u;
    if (s_last) a.done[b] = 0u;  // ready for the next call
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  // ---- the slot's last CTA: first the segment (one a thread: S <= 256)
  const double pr = tid < S ? __ldcg(a.part + ((int64_t)b * S + tid) * 2) : 0.0;
  const double pp = tid < S ? __ldcg(a.part + ((int64_t)b * S + tid) * 2 + 1) : 0.0;
  const double inc_r = block_scan(pr, s_tot);
  if (tid == kVThr - 1) s_base = inc_r;
  __syncthreads();
  const bool use_p = !(s_base > 0.0);  // nothing left of the difference: p itself
  const double mine = use_p ? pp : pr;
  const double inc = use_p ? block_scan(pp, s_tot) : inc_r;
  __syncthreads();
  if (tid == kVThr - 1) {
    s_thr = (double)__ldg(a.u + (int64_t)b * (T + 1) + T) * inc;
    s_base = inc;  // the total, for now
    s_seg = kVThr;
    s_first = kVSeg;
    s_lastpos = -1;
  }
  __syncthreads();
  const double thr = s_thr, total = s_base;
  // the first segment whose running sum passes the threshold; where none
  // does (u_T not below 1, or a rounding), the last one that weighs anything
  if (mine > 0.0) {
    if (inc > thr) atomicMin(&s_seg, tid);
    atomicMax(&s_lastpos, tid);
  }
  __syncthreads();
  int token = -1;
  if (total > 0.0) {
    const int sg = s_seg < kVThr ? s_seg : s_lastpos;
    __syncthreads();
    if (tid == sg) s_base = inc - mine;
    if (tid == 0) s_lastpos = -1;
    load(sg);
    if (use_p) {
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        w[k] = pw[k];
        we[k] = 0.0f;
      }
    }
    float s = 0.0f, e = 0.0f;
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      add_pair(s, e, w[k]);
      e = __fadd_rn(e, we[k]);
    }
    const double own = (double)s + (double)e;
    const double incl = block_scan(own, s_tot);  // synchronises: s_base is set
    double run = s_base + (incl - own);
    int first = kVSeg, last = -1;
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      run += (double)w[k] + (double)we[k];
      if (w[k] > 0.0f) {
        last = tid * kVPer + k;
        if (run > thr && first == kVSeg) first = last;
      }
    }
    if (first < kVSeg) atomicMin(&s_first, first);
    if (last >= 0) atomicMax(&s_lastpos, last);
    __syncthreads();
    token = sg * kVSeg + (s_first < kVSeg ? s_first : s_lastpos);
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
  return 256 + (((size_t)s->n_slots * 4 + 255) & ~(size_t)255) + (size_t)s->n_slots * S * 16;
}

cudaError_t launch_verify(const moe_verify_shape_t* s, const void* p, const void* q,
                          const int32_t* draft, const int32_t* n_draft, const float* u,
                          int32_t* tokens, int32_t* n_acc, uint8_t* ws, cudaStream_t stream) {
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
  const dim3 grid(a.S, s->n_slots);
  auto kern = s->dtype == MOE_DTYPE_FP32   ? verify_kernel<MOE_DTYPE_FP32>
              : s->dtype == MOE_DTYPE_BF16 ? verify_kernel<MOE_DTYPE_BF16>
                                           : verify_kernel<MOE_DTYPE_FP16>;
  return launch_pdl(kern, grid, dim3(kVThr), 0, stream, a);
}

}  // namespace moe

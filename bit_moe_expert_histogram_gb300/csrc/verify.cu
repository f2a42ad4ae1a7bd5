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
// exact), p - q as an fp32 pair without error, and the sums, the threshold
// and the comparisons are fp32 pairs (value and error term). An addition adds
// at most 2^-24 of its sum to the error terms, so after k of them these hold
// (k + 1) 2^-24 of it, and their own two roundings an addition less than
// k (k + 2) 2^-48: 2^-37.9 for a total (32 additions deep), 2^-36.6 for a
// running sum (50), together below 2^-36 of the total on a threshold's way to
// a border. Restated on the host, totals of random rows were off by less than
// 2^-43 (vocabularies of 32000 to 2^20). FP64 does the same in fewer lines,
// but its rate here is a small fraction of fp32's: joining the threads in fp32
// pairs instead took 57.5 us to 28.2 (64 slots of 131072 in bf16), the search
// for the token too 26.6 to 22.5, and 11.9 to 7.1 for one slot of 32000.
//
// What it has to read is one row of p and one of q per slot: HBM bounds large
// batches, a chain of dependent accesses small ones. The vocabulary is cut
// into segments of 4096; a slot's C CTAs (one wave of four or five per SM over
// the batch, at most one per segment) each find i by themselves (a warp, one
// draft a lane: two dependent loads), sum their segments and leave the sums in
// the workspace. The slot's last CTA scans the segments' sums, re-reads the
// one segment that the threshold falls into (it is in L2) and walks it. A
// thread's sixteen values come in 16-byte loads, or in single ones, a warp's
// neighbours each, where a row is not 16-byte aligned (an odd vocabulary).
//
// 64 slots of 131072 in bf16: 17.5 us, 1.9 TB/s; 256 slots of 128001 in fp32
// with certain drafts: 38 us, 3.5 TB/s, 0.51 of a plain copy's rate. With the
// sums left out these take 11.6 and 31 us: the exact sums, some 20 to 29
// instructions an element, are what is left over the loads. (A ring in shared
// memory filled by bulk copies whatever a row's alignment read no faster: 19.9
// and 37.8 us.)
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {
constexpr int kVThr = 256;
constexpr int kVPer = 16;             // elements per thread
constexpr int kVSeg = kVThr * kVPer;  // elements per segment
constexpr int kVWarps = kVThr / 32;
// CTAs an SM: as many as the registers of a thread's values allow
template <int DT>
constexpr int kVCtas = DT == MOE_DTYPE_FP32 ? 4 : 5;

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
// They stay as they were read (a 16-bit word holds elements k, k + 1) until
// they are used.
template <int DT>
struct Raw {
  uint32_t w[DT == MOE_DTYPE_FP32 ? kVPer : kVPer / 2];
};
template <int DT>
__device__ __forceinline__ uint32_t bits(const char* seg, int i) {
  return DT == MOE_DTYPE_FP32 ? __ldg(reinterpret_cast<const uint32_t*>(seg) + i)
                              : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(seg) + i);
}
template <int DT, bool Walk>
__device__ __forceinline__ void load16(const char* seg, int n, bool vec, Raw<DT>& x) {
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2, kPiece = 16 / kE;
  const bool full = n >= kVSeg;  // the same for every thread
  if (vec) {
#pragma unroll
    for (int k = 0; k < kVPer / kPiece; ++k) {
      const int at = place<DT, Walk>(k * kPiece, true);
      if (full || at + kPiece <= n) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(seg + (int64_t)at * kE));
        x.w[4 * k] = v.x;
        x.w[4 * k + 1] = v.y;
        x.w[4 * k + 2] = v.z;
        x.w[4 * k + 3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (DT == MOE_DTYPE_FP32) {
            x.w[4 * k + j] = at + j < n ? bits<DT>(seg, at + j) : 0u;
          } else {
            const uint32_t lo = at + 2 * j < n ? bits<DT>(seg, at + 2 * j) : 0u;
            const uint32_t hi = at + 2 * j + 1 < n ? bits<DT>(seg, at + 2 * j + 1) : 0u;
            x.w[4 * k + j] = lo | hi << 16;
          }
        }
      }
    }
  } else {
    uint32_t e[kVPer];
    if (full) {
#pragma unroll
      for (int k = 0; k < kVPer; ++k) e[k] = bits<DT>(seg, place<DT, Walk>(k, false));
    } else {
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        const int at = place<DT, Walk>(k, false);
        e[k] = at < n ? bits<DT>(seg, at) : 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      if (DT == MOE_DTYPE_FP32)
        x.w[k] = e[k];
      else if (k & 1)
        x.w[k / 2] = e[k - 1] | e[k] << 16;
    }
  }
}
// elements k and k + 1 (k even) as fp32 numbers
template <int DT>
__device__ __forceinline__ uint64_t two(const Raw<DT>& x, int k) {
  if (DT == MOE_DTYPE_FP32) return pair2(x.w[k], x.w[k + 1]);
  const uint32_t w = x.w[k / 2];
  if (DT == MOE_DTYPE_BF16) return pair2(w << 16, w & 0xFFFF0000u);
  return pair2(__float_as_uint(half_bits_to_float(w & 0xFFFFu)),
               __float_as_uint(half_bits_to_float(w >> 16)));
}

// s + e += x without error but for e's own rounding
__device__ __forceinline__ void add_pair(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x);
  const float z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}
// A number as the sum of an fp32 value and an error term.
struct Pair {
  float s, e;
};
__device__ __forceinline__ void add(Pair& a, const Pair& b) {
  a.e = __fadd_rn(a.e, b.e);
  add_pair(a.s, a.e, b.s);
}
__device__ __forceinline__ Pair neg(const Pair& a) { return Pair{-a.s, -a.e}; }
// the error term brought below half a step of the value
__device__ __forceinline__ Pair tidy(const Pair& a) {
  const float s = __fadd_rn(a.s, a.e);
  return Pair{s, __fsub_rn(a.e, __fsub_rn(s, a.s))};
}
// a > b, both tidy: the values' difference is exact where it matters
__device__ __forceinline__ bool above(const Pair& a, const Pair& b) {
  return __fadd_rn(__fsub_rn(a.s, b.s), __fsub_rn(a.e, b.e)) > 0.0f;
}
__device__ __forceinline__ Pair times(float u, const Pair& t) {
  const float s = __fmul_rn(u, t.s);
  return tidy(Pair{s, fmaf(u, t.e, fmaf(u, t.s, -s))});
}
__device__ __forceinline__ Pair shfl_up(const Pair& a, int d) {
  return Pair{__shfl_up_sync(0xFFFFFFFFu, a.s, d), __shfl_up_sync(0xFFFFFFFFu, a.e, d)};
}
__device__ __forceinline__ Pair warp_scan(Pair v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Pair o = shfl_up(v, d);
    if (lane >= d) add(v, o);
  }
  return v;
}
// two elements at once, 0 where they are not positive finite numbers
__device__ __forceinline__ uint64_t clean2(uint64_t t) {
  const uint32_t t0 = (uint32_t)t, t1 = (uint32_t)(t >> 32);
  // 0 < bits < infinity's
  return pair2(t0 - 1u < 0x7F7FFFFFu ? t0 : 0u, t1 - 1u < 0x7F7FFFFFu ? t1 : 0u);
}
// p - q without error as d + e, 0 where the difference is not a positive
// finite number
__device__ __forceinline__ void weight2(uint64_t p, uint64_t q, uint64_t& d, uint64_t& e) {
  const uint64_t t = sub2(p, q), z = sub2(t, p);
  const uint64_t r = sub2(sub2(p, sub2(t, z)), add2(q, z));
  d = clean2(t);
  e = pair2((uint32_t)d ? (uint32_t)r : 0u, (uint32_t)(d >> 32) ? (uint32_t)(r >> 32) : 0u);
}

// inclusive scan of one pair per thread over the CTA (fixed order)
__device__ __forceinline__ Pair block_scan(Pair v, float2* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) warp_tot[warp] = make_float2(v.s, v.e);
  __syncthreads();
  Pair base{0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kVWarps; ++w)
    if (w < warp) add(base, Pair{warp_tot[w].x, warp_tot[w].y});
  add(v, base);
  return v;
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
  float2* part;    // [slot][S]: sums of the segments' weights
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
// this thread's 16 elements of segment sg
template <int DT, bool Walk>
__device__ __forceinline__ void seg_load(const Rows& r, int V, int sg, Raw<DT>& p, Raw<DT>& q) {
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2;
  const int v0 = sg * kVSeg, n = V - v0;
  // one arrangement for both rows: pieces only where both allow them
  const bool vec = r.vp && r.vq;
  load16<DT, Walk>(r.p + (int64_t)v0 * kE, n, vec, p);
  if (r.q) {
    load16<DT, Walk>(r.q + (int64_t)v0 * kE, n, vec, q);
  } else if (r.cut >= v0 && r.cut - v0 < kVSeg) {
#pragma unroll
    for (int k = 0; k < kVPer; ++k)
      if (v0 + place<DT, Walk>(k, vec) == r.cut) {
        if (DT == MOE_DTYPE_FP32)
          p.w[k] = 0u;
        else
          p.w[k / 2] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
      }
  }
}
// the sum of their weights
template <int DT>
__device__ __forceinline__ Pair seg_sum(bool has_q, const Raw<DT>& p, const Raw<DT>& q) {
  uint64_t s2 = 0, e2 = 0;  // even and odd elements
  if (has_q) {
#pragma unroll
    for (int k = 0; k < kVPer; k += 2) {
      uint64_t d, r;
      weight2(two<DT>(p, k), two<DT>(q, k), d, r);
      const uint64_t t = add2(s2, d), z = sub2(t, s2);
      e2 = add2(e2, add2(add2(sub2(s2, sub2(t, z)), sub2(d, z)), r));
      s2 = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kVPer; k += 2) {
      const uint64_t d = clean2(two<DT>(p, k));
      const uint64_t t = add2(s2, d), z = sub2(t, s2);
      e2 = add2(e2, add2(sub2(s2, sub2(t, z)), sub2(d, z)));
      s2 = t;
    }
  }
  Pair a, b;
  unpair2(s2, a.s, b.s);
  unpair2(e2, a.e, b.e);
  add(a, b);
  return a;
}

template <int DT>
__global__ void __launch_bounds__(kVThr, kVCtas<DT>) verify_kernel(const VerifyArgs a) {
  extern __shared__ float2 s_seg[];  // [this CTA's segments][warps]: sums as pairs
  __shared__ int s_i, s_n, s_bad_x, s_last, s_first, s_lastpos;
  __shared__ float2 s_tot[kVWarps];
  __shared__ Pair s_thr, s_base;
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
      Raw<DT> p, q;
      seg_load<DT, false>(r, V, sg, p, q);
      Pair v = seg_sum<DT>(r.q != nullptr, p, q);
#pragma unroll
      for (int d = 16; d; d >>= 1)
        add(v, Pair{__shfl_xor_sync(0xFFFFFFFFu, v.s, d), __shfl_xor_sync(0xFFFFFFFFu, v.e, d)});
      if (lane == 0) s_seg[k * kVWarps + warp] = make_float2(v.s, v.e);
    }
    __syncthreads();
    if (warp == 0) {
      for (int j = lane; j < k; j += 32) {
        Pair sum{0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kVWarps; ++w)
          add(sum, Pair{s_seg[j * kVWarps + w].x, s_seg[j * kVWarps + w].y});
        a.part[(int64_t)b * S + (int)blockIdx.x + j * C] = make_float2(sum.s, sum.e);
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        s_last = atomicAdd(a.done + b, 1u) == (unsigned)C - 1u;
        if (s_last) a.done[b] = 0u;  // ready for the next call
        __threadfence();
      }
    }
    __syncthreads();
  }
  if (!s_last) return;
  // ---- the slot's last CTA: first the segment, a warp with 8 a lane
  // (S <= 256). The first segment whose running sum passes the threshold;
  // where none does (u_T not below 1, or a rounding), the last that weighs
  // anything. s_first: the segment, -1 where nothing weighs anything, -2 where
  // the sum is past fp32's largest number (the thresholds mean nothing then).
  const float u_new = __ldg(a.u + (int64_t)b * (T + 1) + T);
  auto find_segment = [&](const float2* part) {
    Pair v[8], sum{0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int sg = lane * 8 + k;
      const float2 x = sg < S ? __ldcg(part + sg) : make_float2(0.0f, 0.0f);
      v[k] = Pair{x.x, x.y};
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) add(sum, v[k]);
    const Pair inc = warp_scan(sum, lane);
    const Pair total = tidy(Pair{__shfl_sync(0xFFFFFFFFu, inc.s, 31), __shfl_sync(0xFFFFFFFFu, inc.e, 31)});
    const Pair thr = times(u_new, total);
    const unsigned past = __ballot_sync(0xFFFFFFFFu, sum.s > 0.0f && above(tidy(inc), thr));
    const unsigned some = __ballot_sync(0xFFFFFFFFu, sum.s > 0.0f);
    const bool finite = fabsf(total.s) < INFINITY;  // a NaN is not
    if (lane == 0) s_first = finite ? -1 : -2;
    __syncwarp();
    if (finite && some && lane == (past ? __ffs(past) - 1 : 31 - __clz(some))) {
      Pair run = inc, base;
      add(run, neg(sum));
      base = run;
      int at = 0;
      bool passed = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (v[k].s > 0.0f && !passed) {
          base = run;
          add(run, v[k]);
          at = k;
          passed = above(tidy(run), thr);
        }
      }
      s_first = lane * 8 + at;
      s_base = base;
      s_thr = thr;
    }
    __syncwarp();
  };
  if (warp == 0) find_segment(a.part + (int64_t)b * S);
  __syncthreads();
  if (s_first == -1 && rejected) {
    // nothing left of the difference: the target's own row, summed here (a
    // case of roundings, where q is nowhere below p)
    r.q = nullptr;
    r.cut = -1;
    r.vq = true;
    for (int sg = 0; sg < S; ++sg) {
      Raw<DT> p, q;
      seg_load<DT, false>(r, V, sg, p, q);
      const Pair t = block_scan(seg_sum<DT>(false, p, q), s_tot);
      if (tid == kVThr - 1) a.part[(int64_t)b * S + sg] = make_float2(t.s, t.e);
    }
    __threadfence();
    __syncthreads();
    if (warp == 0) find_segment(a.part + (int64_t)b * S);
    __syncthreads();
  }
  const int sg = s_first;
  const Pair thr = s_thr;
  Pair incl = s_base;
  __syncthreads();
  int token = -1;
  if (sg >= 0) {
    if (tid == 0) {
      s_first = kVThr;
      s_lastpos = -1;
    }
    Raw<DT> p, q;
    seg_load<DT, true>(r, V, sg, p, q);
    const Pair own = seg_sum<DT>(r.q != nullptr, p, q);
    add(incl, block_scan(own, s_tot));  // synchronises
    // then the thread, in the same way
    if (own.s > 0.0f) {
      if (above(tidy(incl), thr)) atomicMin(&s_first, tid);
      atomicMax(&s_lastpos, tid);
    }
    __syncthreads();
    if (tid == (s_first < kVThr ? s_first : s_lastpos)) {
      // then the element: the first that passes, or the thread's last that
      // weighs anything
      Pair run = incl;
      add(run, neg(own));
      int at = 0;
      bool passed = false;
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        uint64_t d = two<DT>(p, k & ~1), e = 0;
        if (r.q)
          weight2(d, two<DT>(q, k & ~1), d, e);
        else
          d = clean2(d);
        const Pair w{__uint_as_float((uint32_t)(d >> (k & 1 ? 32 : 0))),
                     __uint_as_float((uint32_t)(e >> (k & 1 ? 32 : 0)))};
        if (w.s > 0.0f && !passed) {
          add(run, w);
          at = k;
          passed = above(tidy(run), thr);
        }
      }
      s_i = sg * kVSeg + tid * kVPer + at;
    }
    __syncthreads();
    token = s_i;
  } else if (tid == 0) {
    set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_VERIFY, b);  // no weight, or past all numbers
  }
  if (tid <= T) {
    const int64_t at = (int64_t)b * (T + 1) + tid;
    a.tokens[at] = tid < i ? __ldg(a.draft + (int64_t)b * T + tid) : tid == i ? token : -1;
    if (tid == 0) a.n_acc[b] = i;
  }
}

namespace {
constexpr int kMostSlots = 4096;
// The slots' counters (zeros between calls) lie at one place and have one
// extent, whatever the shape: a server's batch grows and shrinks in one
// workspace. The segments' sums follow, which no call leaves to the next.
constexpr size_t kDoneAt = 256, kPartAt = kDoneAt + kMostSlots * 4;
}  // namespace

bool verify_supported(const moe_verify_shape_t* s) {
  if (!s) return false;
  if (s->n_slots < 1 || s->n_slots > kMostSlots || s->T < 1 || s->T > 31) return false;
  if (s->V < 1 || s->V > kVSeg * kVThr) return false;
  return s->dtype == MOE_DTYPE_BF16 || s->dtype == MOE_DTYPE_FP16 || s->dtype == MOE_DTYPE_FP32;
}

size_t verify_ws_bytes(const moe_verify_shape_t* s) {
  const size_t S = (s->V + kVSeg - 1) / kVSeg;
  return kPartAt + (size_t)s->n_slots * S * 8;
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
  a.done = reinterpret_cast<unsigned*>(ws + kDoneAt);
  a.part = reinterpret_cast<float2*>(ws + kPartAt);
  // each CTA with as many segments as the CTAs that fit at once leave it
  const int ctas = s->dtype == MOE_DTYPE_FP32 ? kVCtas<MOE_DTYPE_FP32> : kVCtas<MOE_DTYPE_BF16>;
  const int per_slot = ctas * nsm / s->n_slots > 1 ? ctas * nsm / s->n_slots : 1;
  const int C = per_slot < a.S ? per_slot : a.S;
  const dim3 grid(C, s->n_slots);
  const size_t smem = (size_t)((a.S + C - 1) / C) * kVWarps * sizeof(float2);
  auto kern = s->dtype == MOE_DTYPE_FP32   ? verify_kernel<MOE_DTYPE_FP32>
              : s->dtype == MOE_DTYPE_BF16 ? verify_kernel<MOE_DTYPE_BF16>
                                           : verify_kernel<MOE_DTYPE_FP16>;
  return launch_pdl(kern, grid, dim3(kVThr), smem, stream, a);
}

}  // namespace moe

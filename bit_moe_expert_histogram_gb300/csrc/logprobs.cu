// Log probabilities of given tokens under rows of logits, the rows' entropies
// and their likeliest tokens.
//
// With m = max x, d = x - m: Z = sum e^d, A = sum d e^d, so that
//   log p(x) = d - ln Z,   entropy = ln Z - A / Z,
// and stretches of a row join as Z = sum Z_i e^(m_i - m), A = sum (A_i +
// (m_i - m) Z_i) e^(m_i - m). One pass over the logits: every thread keeps its
// own m, Z and A of what it reads (a new maximum comes a few times a thread),
// which are joined in a fixed order. d is taken before the exponential's
// factor log2(e), so nothing but its own rounding is in the exponent.
//
// The k likeliest, ties to the lower id. Of the first chunk that a CTA reads
// (16 bytes a thread and vector, held in registers) the k-th largest of the
// maxima of 64 groups of threads is a number that at least k elements reach,
// and few do (where fewer groups have anything, the k-th of the threads'): those
// are listed, ordered by counting, and the k-th of them is the bar for what
// follows, where only a larger number can still enter (an equal one has a higher
// id). Where more reach the first bar than the list holds (many equal logits),
// those above it are listed and then, in id order, as many of its equals as are
// missing. After 2, 4, 8 .. chunks the list is put in order and the bar raised,
// where more than one follows, so that some k elements enter in between and the
// CTA's warps need not meet at every chunk (meeting at each, with chunks of
// twice the size, took 203 us for 2048 rows of 128001). If more enter than the
// list holds (sorted or smooth rows), the CTA's stretch is read again, for every
// thread's maximum and for what reaches the k-th of these (2048 sorted rows of
// 128001, the first 32: 278 us); if that is still too much (a thousand equals of
// it), once for each of the k (5.3 ms). A stretch whose first chunk has fewer than
// k elements that are not -inf has no bar from it, what follows overfills the list,
// and the stretch is read again like those: 2048 rows of 128001 of which the first
// 16384 are -inf take 290 us.
//
// Many rows are bound by HBM: 2048 rows of 128001 bf16 logits, 524 MB, take 102
// us, 5.15 TB/s, 0.76 of a plain copy's rate (ten instructions a logit, one of
// them an exponential; pairs of fp32 numbers share what they can). Few rows are
// a chain of waits: 64 rows of 131072 with twenty alternatives, 17 MB, take 14.0
// us - logits 2, sums 0.5, the bar 1, the list 1.2, the second chunk 1.6, the
// part and the arrival 2, joining and ordering eight stretches' lists 3.
#include <cfloat>
#include <type_traits>

#include "attn_batch.cuh"

namespace moe {

namespace {
constexpr int kLThr = 256;
// CTAs an SM: many rows want loads in flight, a few want the shorter path that
// more registers give (64 rows of 131072, twenty alternatives: 14.5 us with 4,
// 16.4 with 5; 2048 rows of 128001: 107.5 and 102.7, although five leave 48
// registers and spill 36 to 40 bytes for 16-bit logits with alternatives).
constexpr int kLMany = 5, kLFew = 4;
constexpr int kLWarps = kLThr / 32;
constexpr int kVec = 4;         // 16-byte vectors a thread and chunk
constexpr int kCap = 1024;      // entries of the list, when stretches are joined
constexpr int kMost = 256;      // that one stretch may bring: ordering takes their square
constexpr int kMostTop = 32;
constexpr int kMostCuts = kCap / kMostTop;  // stretches of a row, whose entries one list holds
constexpr int kMostParts = 1024;            // (row, stretch) pairs where rows are cut
constexpr int kLGroups = kLThr / 4;
constexpr size_t kLCountAt = 256, kLPartAt = kLCountAt + kMostParts * 4;
constexpr int kLPart = 4 + 2 * kMostTop;  // floats of a part: m, Z, A, how many entries, those

struct LogpArgs {
  const char* x;
  int64_t stride;  // bytes
  const int32_t* tokens;
  float* logp;
  float* entropy;    // or null
  int32_t* top_ids;  // [rows][k]
  float* top_logp;
  int V, k, S, per;  // S stretches a row, of `per` chunks
  unsigned* count;
  float* part;
  Ctrl* ctrl;
};

template <int DT>
struct El {
  static constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2;  // bytes
  static constexpr int kN = 16 / kE;                       // of a vector
  static constexpr int kChunk = kLThr * kVec * kN;         // elements
  // -inf, and the least finite number, as a word
  static constexpr uint32_t kNone = DT == MOE_DTYPE_FP32   ? 0xFF800000u
                                    : DT == MOE_DTYPE_BF16 ? 0xFF80FF80u
                                                           : 0xFC00FC00u;
  static constexpr uint32_t kLeast = DT == MOE_DTYPE_FP32   ? 0xFF7FFFFFu
                                     : DT == MOE_DTYPE_BF16 ? 0xFF7FFF7Fu
                                                            : 0xFBFFFBFFu;
};
template <int DT>
__device__ __forceinline__ float el_at(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (DT == MOE_DTYPE_FP32) return __uint_as_float(w[i]);
  constexpr bool kF16 = DT == MOE_DTYPE_FP16;
  return i & 1 ? unpack_hi<kF16>(w[i / 2]) : unpack_lo<kF16>(w[i / 2]);
}
template <int DT>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {  // NaN if either is
  uint32_t r;
  if (DT == MOE_DTYPE_FP32)
    asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else if (DT == MOE_DTYPE_BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int DT>
__device__ __forceinline__ float max_of(const uint4 (&v)[kVec]) {
  uint32_t w = max_word<DT>(max_word<DT>(v[0].x, v[0].y), max_word<DT>(v[0].z, v[0].w));
#pragma unroll
  for (int j = 1; j < kVec; ++j)
    w = max_word<DT>(w, max_word<DT>(max_word<DT>(v[j].x, v[j].y), max_word<DT>(v[j].z, v[j].w)));
  if (DT == MOE_DTYPE_FP32) return __uint_as_float(w);
  constexpr bool kF16 = DT == MOE_DTYPE_FP16;
  return max_nan(unpack_lo<kF16>(w), unpack_hi<kF16>(w));
}
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float a) { return pair2(__float_as_uint(a), __float_as_uint(a)); }

struct Sums {
  float m, Z, A;
};
// the same sums from another maximum, M >= s.m
__device__ __forceinline__ Sums from(const Sums& s, float M) {
  const float d = s.m - M, f = ex2(d * 1.4426950408889634f);
  // nothing so far, or far below (the lowest number as a mask): no inf * 0
  return s.Z == 0.0f ? Sums{M, 0.0f, 0.0f} : Sums{M, s.Z * f, f == 0.0f ? 0.0f : fmaf(d, s.Z, s.A) * f};
}
// the sums of `n` lanes (a power of two), by each of them
__device__ __forceinline__ Sums join(const Sums& s, int n) {
  float M = s.m;
  for (int o = n / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  Sums r = from(s, M);
  for (int o = n / 2; o > 0; o >>= 1) {
    r.Z += __shfl_xor_sync(0xFFFFFFFFu, r.Z, o);
    r.A += __shfl_xor_sync(0xFFFFFFFFu, r.A, o);
  }
  return r;
}
// the least fp32 number above x (x is not NaN or +inf)
__device__ __forceinline__ float next_up(float x) {
  const int u = __float_as_int(x);
  return x == 0.0f ? __int_as_float(1) : __int_as_float(u + (u < 0 ? -1 : 1));
}
// adds a thread's vectors, whose largest element is `top`, to its sums
template <int DT>
__device__ __forceinline__ void add_chunk(Sums& s, const uint4 (&v)[kVec], float top) {
  if (top > s.m) s = from(s, top);
  if (top != top) s.Z = top;
  if (s.m < (DT == MOE_DTYPE_FP16 ? -65000.0f : -1e38f)) {
    // nothing but -inf, or what a mask of the least number leaves, which weighs
    // something beside nothing else: -inf is told from it
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int i = 0; i < El<DT>::kN; ++i) {
        const float x = el_at<DT>(v[j], i);
        if (x == -INFINITY) continue;
        const float d = fmaxf(x - s.m, -200.0f), e = ex2(d * 1.4426950408889634f);
        s.Z += e;
        s.A = fmaf(e, d, s.A);
      }
    return;
  }
  uint64_t Z = pair2(__float_as_uint(s.Z), 0u), A = pair2(__float_as_uint(s.A), 0u);
  const uint64_t nm = both(-s.m), l2 = both(1.4426950408889634f);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int i = 0; i < El<DT>::kN / 2; ++i) {
      // -inf as the least finite number: its weight is 0, and 0 times d, too
      uint64_t x;
      if (DT == MOE_DTYPE_FP32) {
        x = pair2(max_word<DT>(w[2 * (i & 1)], El<DT>::kLeast),
                  max_word<DT>(w[2 * (i & 1) + 1], El<DT>::kLeast));
      } else {
        const uint32_t c = max_word<DT>(w[i & 3], El<DT>::kLeast);
        x = pair2(__float_as_uint(unpack_lo<DT == MOE_DTYPE_FP16>(c)),
                  __float_as_uint(unpack_hi<DT == MOE_DTYPE_FP16>(c)));
      }
      const uint64_t d = add2(x, nm);
      float y0, y1;
      unpair2(mul2(d, l2), y0, y1);
      const uint64_t e = pair2(__float_as_uint(ex2(y0)), __float_as_uint(ex2(y1)));
      Z = add2(Z, e);
      A = fma2(e, d, A);
    }
  }
  float z0, z1, a0, a1;
  unpair2(Z, z0, z1);
  unpair2(A, a0, a1);
  s.Z = z0 + z1;
  s.A = a0 + a1;
}

// An entry as a whole number that is larger the earlier it comes: the logit in
// an order-keeping form (-0 is 0), below it the id, lower ones larger. 0: none.
// (Two comparisons with a branch between them took 42 ns an entry compared.)
__device__ __forceinline__ uint64_t entry(float x, int id) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (uint64_t)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ int entry_id(uint64_t e) { return (int)~(uint32_t)e; }
__device__ __forceinline__ float entry_x(uint64_t e) {
  const uint32_t u = (uint32_t)(e >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
// A maximum among `n` (a power of two): in an order-keeping form that ends in
// as many zeros as the number, whose last places are the index, lower ones
// larger; and the number back, or the one below it whose last places are zeros.
__device__ __forceinline__ uint32_t place(float x, int i, int n) {
  const uint32_t u = __float_as_uint(x + 0.0f), c = u & 0x80000000u ? 0u - u : u | 0x80000000u;
  return (c & (uint32_t)-n) | (uint32_t)(n - 1 - i);
}
__device__ __forceinline__ float placed(uint32_t p, int n) {
  const uint32_t c = p & (uint32_t)-n;
  return __uint_as_float(c & 0x80000000u ? c & 0x7FFFFFFFu : 0u - c);
}
// how many of t[from], four each `step`, below t[n], are before p
__device__ __forceinline__ int before(const uint32_t* t, int from, int step, int n, uint32_t p) {
  int r = 0;
#pragma unroll 4
  for (int j = from; j < n; j += step) {
    const uint4 o = *reinterpret_cast<const uint4*>(t + j);
    r += (o.x > p) + (o.y > p) + (o.z > p) + (o.w > p);
  }
  return r;
}
struct TopList {
  alignas(16) uint64_t e[kCap];
  uint64_t best[kMostTop];
  int n;
};
// how many of n entries are before this one
__device__ __forceinline__ int rank_of(const TopList& t, int n, uint64_t x) {
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) rank += t.e[j] > x;
  return rank;
}
// Puts the first k of the list's entries in order, in place. By the whole CTA,
// which has met since the last entry came; returns how many there are.
__device__ __forceinline__ int keep_best(TopList& t, int k) {
  const int n = t.n, m = n < k ? n : k;
  for (int i = threadIdx.x; i < n; i += kLThr) {
    const uint64_t x = t.e[i];
    const int rank = rank_of(t, n, x);
    if (rank < k) t.best[rank] = x;
  }
  __syncthreads();
  if ((int)threadIdx.x < m) t.e[threadIdx.x] = t.best[threadIdx.x];
  if (threadIdx.x == 0) t.n = m;
  __syncthreads();
  return m;
}
}  // namespace

template <int DT, bool TOP, int kCtas>
__global__ void __launch_bounds__(kLThr, kCtas) logprobs_kernel(const LogpArgs a) {
  using E = El<DT>;
  __shared__ TopList list;
  __shared__ uint4 s_vec[TOP ? kLThr : 1][kVec];
  __shared__ __align__(16) uint32_t s_group[kLGroups];
  __shared__ float s_bar, s_w[3][kLWarps];
  __shared__ int s_scan[kLWarps], s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.S, cut = blockIdx.x - row * a.S;
  if (TOP && tid == 0) list.n = 0;
  pdl_wait();
  pdl_trigger();
  const char* x0 = a.x + (int64_t)row * a.stride;
  const int tok = __ldg(a.tokens + row);
  uint32_t x_tok = 0;
  if (tid == 0 && tok >= 0 && tok < a.V)
    x_tok = DT == MOE_DTYPE_FP32 ? __ldg(reinterpret_cast<const uint32_t*>(x0) + tok)
                                 : __ldg(reinterpret_cast<const uint16_t*>(x0) + tok);
  // vectors lie on 16-byte borders; elements before the row's first and past
  // its last are left out
  const int shift = (int)(reinterpret_cast<uintptr_t>(x0) & 15u) / E::kE;
  const int n_vec = (a.V + shift + E::kN - 1) / E::kN;
  auto first_of = [&](int chunk, int j) { return ((chunk * kVec + j) * kLThr + tid) * E::kN - shift; };
  auto load = [&](int chunk, uint4 (&v)[kVec]) {
    const char* p = x0 + (int64_t)first_of(chunk, 0) * E::kE;
    if (chunk * E::kChunk >= shift && (chunk + 1) * E::kChunk - shift <= a.V) {  // all of it inside
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = load_stream(p + j * (kLThr * 16));
      return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int e0 = first_of(chunk, j);
      if (e0 >= 0 && e0 + E::kN <= a.V) {
        v[j] = load_stream(p + j * (kLThr * 16));
        continue;
      }
      uint32_t w[4] = {E::kNone, E::kNone, E::kNone, E::kNone};
      if (e0 + E::kN > 0 && e0 < a.V) {
#pragma unroll
        for (int i = 0; i < E::kN; ++i) {
          if (e0 + i < 0 || e0 + i >= a.V) continue;
          if (DT == MOE_DTYPE_FP32) {
            w[i & 3] = __ldg(reinterpret_cast<const uint32_t*>(x0) + e0 + i);
          } else {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(x0) + e0 + i);
            w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | h << 16 : (w[i / 2] & 0xFFFF0000u) | h;
          }
        }
      }
      v[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  auto own = [&](int b) {  // element b of the thread's vectors
    if (DT == MOE_DTYPE_FP32) return reinterpret_cast<const float*>(s_vec[tid])[b];
    return unpack_lo<DT == MOE_DTYPE_FP16>(reinterpret_cast<const uint16_t*>(s_vec[tid])[b]);
  };
  constexpr int kChunkVecs = kLThr * kVec;
  const int c0 = cut * a.per, c1 = min(c0 + a.per, (n_vec + kChunkVecs - 1) / kChunkVecs);
  Sums s{-INFINITY, 0.0f, 0.0f};
  float bar = -FLT_MAX;   // what a further element has to reach
  bool over = false;      // more came than the list holds
  bool spilled = false;   // an entry of this thread found it full
  uint4 v[kVec];
  if (c0 < c1) load(c0, v);
  for (int c = c0; c < c1; ++c) {
    const float top = max_of<DT>(v);
    add_chunk<DT>(s, v, top);
    if (!TOP) {
      if (c + 1 < c1) load(c + 1, v);
    } else {
      const bool begin = c == c0;
      float low = -INFINITY;
      if (begin) {
        // the number that at least k of this chunk reach, NaN aside: of the 64
        // groups' maxima the k-th, each group ranked by its four threads
        float g = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, 2));
        g = g != g ? -INFINITY : g;
        const int q = tid & 3;
        uint32_t mine = place(g, tid >> 2, kLGroups);
        if (q == 0) s_group[tid >> 2] = mine;
        if (tid == 0) s_bar = -INFINITY;
        __syncthreads();
        int rank = before(s_group, 4 * q, 16, kLGroups, mine);
        rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 1);
        rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 2);
        if (q == 0 && rank == a.k - 1) s_bar = placed(mine, kLGroups);
        __syncthreads();
        low = s_bar;
        if (low == -INFINITY) {
          // fewer groups have anything (a short row, or most of it masked): the
          // k-th of the threads' maxima (1160 rows of 952, the first 32: 244 us
          // without, as all of a row then overfills the list, 16.7 with)
          uint32_t* one = reinterpret_cast<uint32_t*>(list.e);
          g = top != top ? -INFINITY : top;
          mine = place(g, tid, kLThr);
          one[tid] = mine;
          __syncthreads();
          if (g > -INFINITY && before(one, 0, 4, kLThr, mine) == a.k - 1) s_bar = placed(mine, kLThr);
          __syncthreads();
          low = s_bar;
        }
        bar = fmaxf(low, -FLT_MAX);
      }
      const int seen = c - c0 + 1;
      const bool meet = begin || ((seen & (seen - 1)) == 0 && c + 1 < c1);
      bool equals = false;
#pragma unroll 1
      for (;;) {
        // which of the thread's elements reach the bar (few threads have one),
        // then the next chunk's loads, then those elements, through shared
        // memory (read again from L2 they took 1 us longer)
        uint32_t mask = 0;
        if (!(top < bar)) {
#pragma unroll
          for (int j = 0; j < kVec; ++j)
#pragma unroll
            for (int i = 0; i < E::kN; ++i) mask |= el_at<DT>(v[j], i) >= bar ? 1u << (j * E::kN + i) : 0u;
          if (mask) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) s_vec[tid][j] = v[j];
          }
        }
        if (c + 1 < c1) load(c + 1, v);
        {
#pragma unroll 1
          for (; mask; mask &= mask - 1) {
            const int b = __ffs(mask) - 1, id = first_of(c, b / E::kN) + b % E::kN;
            const int at = atomicAdd(&list.n, 1);
            if (at < kMost)
              list.e[at] = entry(own(b), id);
            else
              spilled = true;
          }
        }
        if (!meet || over) break;
        // the same answer for all: list.n may grow as soon as one thread goes on
        if (!__syncthreads_or(spilled)) break;
        spilled = false;
        // too many: of the first chunk those above the groups' bar and then the
        // first of its equals, once
        over = !begin || equals;
        equals = true;
        __syncthreads();
        if (over) break;
        if (tid == 0) list.n = 0;
        bar = next_up(low);
        load(c, v);
        __syncthreads();
      }
      if (equals && !over && low > -INFINITY) {
        load(c, v);
        int have = list.n, need = have < a.k ? a.k - have : 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (need == 0) break;  // the same for all
          int n = 0;
#pragma unroll
          for (int i = 0; i < E::kN; ++i) n += el_at<DT>(v[j], i) == low;
          int incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
          }
          __syncthreads();
          if (lane == 31) s_scan[warp] = incl;
          __syncthreads();
          int all = 0, start = incl - n;
          for (int w = 0; w < kLWarps; ++w) {
            if (w < warp) start += s_scan[w];
            all += s_scan[w];
          }
#pragma unroll
          for (int i = 0; i < E::kN; ++i)
            if (el_at<DT>(v[j], i) == low) {
              if (start < need) list.e[have + start] = entry(low, first_of(c, j) + i);
              ++start;
            }
          const int took = min(all, need);
          have += took;
          need -= took;
        }
        __syncthreads();
        if (tid == 0) list.n = have;
        __syncthreads();
        if (c + 1 < c1) load(c + 1, v);
      }
      if (over)
        bar = INFINITY;
      else if (meet && c + 2 < c1)
        // the list is put in order where more than a chunk follows; equals of
        // the k-th have higher ids from here on
        bar = keep_best(list, a.k) == a.k ? next_up(entry_x(list.e[a.k - 1])) : -FLT_MAX;
    }
  }
  if (TOP) {
    __syncthreads();
    over |= list.n > kMost;
    if (over) {
      // Large numbers that lie together, or came late. The stretch is read again,
      // for the threads' maxima, whose k-th is a bar (a thread has eight of what
      // lies together where a group has 32), and for what reaches it.
      uint32_t* one = reinterpret_cast<uint32_t*>(s_vec);
      float g = -INFINITY;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        load(c, v);
        const float top = max_of<DT>(v);
        g = fmaxf(g, top != top ? -INFINITY : top);
      }
      __syncthreads();
      const uint32_t mine = place(g, tid, kLThr);
      one[tid] = mine;
      if (tid == 0) {
        s_bar = -INFINITY;
        list.n = 0;
      }
      __syncthreads();
      if (g > -INFINITY && before(one, 0, 4, kLThr, mine) == a.k - 1) s_bar = placed(mine, kLThr);
      __syncthreads();
      bar = fmaxf(s_bar, -FLT_MAX);
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        load(c, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
#pragma unroll
          for (int i = 0; i < E::kN; ++i) {
            const float x = el_at<DT>(v[j], i);
            if (!(x >= bar)) continue;
            const int at = atomicAdd(&list.n, 1);
            if (at < kCap) list.e[at] = entry(x, first_of(c, j) + i);
          }
      }
      __syncthreads();
      over = list.n > kCap;
      __syncthreads();
      if (!over) keep_best(list, a.k);
    }
    if (over) {
      // the best k one after the other, each found by reading the stretch again
      if (tid == 0) list.n = 0;
      uint64_t last = ~0ull;
      for (int r = 0; r < a.k; ++r) {
        uint64_t mine = 0;
        for (int c = c0; c < c1; ++c) {
          load(c, v);
#pragma unroll
          for (int j = 0; j < kVec; ++j)
#pragma unroll
            for (int i = 0; i < E::kN; ++i) {
              const float x = el_at<DT>(v[j], i);
              const uint64_t e = x > -INFINITY ? entry(x, first_of(c, j) + i) : 0;
              if (e < last && e > mine) mine = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t y = __shfl_xor_sync(0xFFFFFFFFu, mine, o);
          mine = y > mine ? y : mine;
        }
        __syncthreads();
        if (lane == 0) list.best[warp] = mine;
        __syncthreads();
        last = 0;
        for (int w = 0; w < kLWarps; ++w) last = list.best[w] > last ? list.best[w] : last;
        if (tid == 0 && last != 0) list.e[list.n++] = last;
      }
    }
  }
  // ---- the CTA's sums, in a fixed order
  s = join(s, 32);
  if (lane == 0) {
    s_w[0][warp] = s.m;
    s_w[1][warp] = s.Z;
    s_w[2][warp] = s.A;
  }
  __syncthreads();
  s = Sums{s_w[0][lane % kLWarps], s_w[1][lane % kLWarps], s_w[2][lane % kLWarps]};
  s = join(s, kLWarps);
  if (a.S > 1) {
    float* part = a.part + (int64_t)blockIdx.x * kLPart;
    if (tid == 0) {
      part[0] = s.m;
      part[1] = s.Z;
      part[2] = s.A;
      part[3] = __int_as_float(TOP ? min(list.n, a.k) : 0);
    }
    if (TOP) {
      const int n = list.n;
      for (int i = tid; i < n; i += kLThr) {
        const uint64_t x = list.e[i];
        const int rank = rank_of(list, n, x);
        if (rank < a.k) reinterpret_cast<uint64_t*>(part + 4)[rank] = x;
      }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      s_last = atomicAdd(a.count + row, 1u) == (unsigned)(a.S - 1);
      if (s_last) a.count[row] = 0u;  // ready for the next call
      list.n = 0;
      __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    // the last of the row's CTAs joins them all, in the row's order
    const float* parts = a.part + (int64_t)row * a.S * kLPart;
    s = Sums{-INFINITY, 0.0f, 0.0f};
    if (lane < a.S) {  // at most 32
      const float* p = parts + lane * kLPart;
      s = Sums{__ldcg(p), __ldcg(p + 1), __ldcg(p + 2)};
    }
    if (TOP) {
      // nothing below a stretch's k-th can be among the first k
      uint64_t least = 0;
      if (lane < a.S && __float_as_int(__ldcg(parts + lane * kLPart + 3)) == a.k)
        least = __ldcg(reinterpret_cast<const unsigned long long*>(parts + lane * kLPart + 4) + a.k - 1);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xFFFFFFFFu, least, o);
        least = y > least ? y : least;
      }
      for (int i = tid; i < a.S * kMostTop; i += kLThr) {
        const float* p = parts + i / kMostTop * kLPart;
        const int j = i % kMostTop;
        const uint64_t x = __ldcg(reinterpret_cast<const unsigned long long*>(p + 4) + j);
        if (j < __float_as_int(__ldcg(p + 3)) && x >= least) list.e[atomicAdd(&list.n, 1)] = x;
      }
    }
    s = join(s, 32);
    __syncthreads();
  }
  // nothing but -inf, or a number that is none: no distribution
  const bool ok = s.m > -INFINITY && s.m < INFINITY && s.Z > 0.0f && s.Z < INFINITY;
  const float lz = logf(s.Z), nan = __int_as_float(0x7FC00000);
  if (tid == 0) {
    float r = 0.0f;
    if (tok >= 0 && tok < a.V) {
      const float x = DT == MOE_DTYPE_FP32 ? __uint_as_float(x_tok) : unpack_lo<DT == MOE_DTYPE_FP16>(x_tok);
      r = ok ? (x - s.m) - lz : nan;
    } else if (tok != -1) {
      r = nan;
    }
    if (!ok || (tok != -1 && (tok < 0 || tok >= a.V))) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_LOGP, row);
    a.logp[row] = r;
    if (a.entropy) a.entropy[row] = ok ? lz - s.A / s.Z : nan;
  }
  if (TOP) {
    const int n = list.n;
    auto put = [&](int rank, int id, float v) {
      const int64_t at = (int64_t)row * a.k + rank;
      if (a.top_ids) a.top_ids[at] = id;
      if (a.top_logp) a.top_logp[at] = v;
    };
    for (int i = tid; i < n; i += kLThr) {
      const uint64_t x = list.e[i];
      const int rank = rank_of(list, n, x);
      if (rank < a.k) put(rank, ok ? entry_id(x) : -1, ok ? (entry_x(x) - s.m) - lz : -INFINITY);
    }
    if (tid >= n && tid < a.k) put(tid, -1, -INFINITY);  // missing
  }
}

bool logprobs_supported(const moe_logprobs_shape_t* s) {
  if (!s || s->n_rows < 1 || s->n_rows > (1 << 20) || s->V < 1 || s->V > (1 << 20)) return false;
  if (s->k < 0 || s->k > kMostTop) return false;
  return s->dtype == MOE_DTYPE_BF16 || s->dtype == MOE_DTYPE_FP16 || s->dtype == MOE_DTYPE_FP32;
}

// status, the rows' counters, the stretches' parts: the same for every shape
size_t logprobs_ws_bytes(const moe_logprobs_shape_t*) { return kLPartAt + (size_t)kMostParts * kLPart * 4; }

cudaError_t launch_logprobs(const moe_logprobs_shape_t* s, const void* logits, int64_t stride,
                            const int32_t* tokens, float* logp, float* entropy, int32_t* top_ids,
                            float* top_logp, uint8_t* ws, int nsm, cudaStream_t stream) {
  const int e = s->dtype == MOE_DTYPE_FP32 ? 4 : 2;
  LogpArgs a;
  a.x = static_cast<const char*>(logits);
  a.stride = stride * e;
  a.tokens = tokens;
  a.logp = logp;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.V = s->V;
  a.k = s->k;
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  a.count = reinterpret_cast<unsigned*>(ws + kLCountAt);
  a.part = reinterpret_cast<float*>(ws + kLPartAt);
  // rows that do not start on 16 bytes may need a vector more
  const bool even = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && a.stride % 16 == 0;
  const int vecs = (s->V * e + 15) / 16 + (even ? 0 : 1), chunk = kLThr * kVec;
  const int chunks = (vecs + chunk - 1) / chunk;
  // rows are cut where there are fewer than CTAs that fit at once
  int most = kLFew * nsm < kMostParts ? kLFew * nsm : kMostParts;
  most /= s->n_rows;
  if (most > kMostCuts) most = kMostCuts;
  const int cuts = most < 1 ? 1 : most < chunks ? most : chunks;
  a.per = (chunks + cuts - 1) / cuts;
  a.S = (chunks + a.per - 1) / a.per;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((unsigned)s->n_rows * a.S), dim3(kLThr), 0, stream, a);
  };
  const bool top = s->k > 0 && (top_ids || top_logp);
  auto pick = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (a.S > 1) return top ? go(logprobs_kernel<DT, true, kLFew>) : go(logprobs_kernel<DT, false, kLFew>);
    return top ? go(logprobs_kernel<DT, true, kLMany>) : go(logprobs_kernel<DT, false, kLMany>);
  };
  if (s->dtype == MOE_DTYPE_FP32) return pick(std::integral_constant<int, MOE_DTYPE_FP32>());
  if (s->dtype == MOE_DTYPE_FP16) return pick(std::integral_constant<int, MOE_DTYPE_FP16>());
  return pick(std::integral_constant<int, MOE_DTYPE_BF16>());
}

}  // namespace moe

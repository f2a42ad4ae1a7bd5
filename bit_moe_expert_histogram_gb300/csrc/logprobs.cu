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
// maxima of 128 groups of threads is a number that at least k elements reach,
// and few do: those are listed, ordered by counting, and the k-th of them is
// the bar for what follows, where only a larger number can still enter (an
// equal one has a higher id). Chunks that bring more than the list holds
// (sorted logits, or many equal ones) are taken up again from the registers:
// first what is above the groups' bar, then, in id order, as many of its
// equals as are missing; and where even that is too much, one by one.
//
// Bound by HBM: a logit costs some five instructions and one exponential.
#include "attn_batch.cuh"

namespace moe {

namespace {
constexpr int kLThr = 512;
constexpr int kLWarps = kLThr / 32;
constexpr int kVec = 4;         // 16-byte vectors a thread and chunk
constexpr int kCap = 1024;      // entries of the list
constexpr int kMostTop = 32;
constexpr int kMostParts = 512; // (row, stretch) pairs where rows are cut
constexpr int kLGroups = kLThr / 4;
constexpr size_t kLCountAt = 256, kLPartAt = kLCountAt + kMostParts * 4;
constexpr int kLPart = 4 + 2 * kMostTop;  // floats of a part: m, Z, A, entries, values, ids

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
  static constexpr uint32_t kNone = DT == MOE_DTYPE_FP32 ? 0xFF800000u : DT == MOE_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
};
template <int DT>
__device__ __forceinline__ float el_at(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (DT == MOE_DTYPE_FP32) return __uint_as_float(w[i]);
  constexpr bool kF16 = DT == MOE_DTYPE_FP16;
  return i & 1 ? unpack_hi<kF16>(w[i / 2]) : unpack_lo<kF16>(w[i / 2]);
}
// the largest, of those that are numbers
template <int DT>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == MOE_DTYPE_FP32)
    r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  else if (DT == MOE_DTYPE_BF16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
  return fmaxf(unpack_lo<kF16>(w), unpack_hi<kF16>(w));
}
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Sums {
  float m, Z, A;
};
__device__ __forceinline__ void raise(Sums& s, float m) {  // m >= s.m
  if (m == s.m) return;
  if (s.Z != 0.0f) {
    const float d = s.m - m, f = expf(d);
    s.A = (s.A + d * s.Z) * f;
    s.Z *= f;
  }
  s.m = m;
}
__device__ __forceinline__ void join(Sums& a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  a.Z += b.Z;
  a.A += b.A;
}

struct Entry {
  float v;
  int id;
};
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {
  return a.v > b.v || (a.v == b.v && a.id < b.id);
}

// The first k of n entries (n <= kCap) in order, in place: each entry's rank
// is the number of those before it. Called by the whole CTA; returns how many
// there are.
struct TopList {
  Entry e[kCap];
  Entry best[kMostTop];
  int n;
};
__device__ __forceinline__ int keep_best(TopList& t, int n, int k) {
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kLThr) {
    const Entry x = t.e[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += before(t.e[j], x);
    if (rank < k) t.best[rank] = x;
  }
  __syncthreads();
  const int m = n < k ? n : k;
  if ((int)threadIdx.x < m) t.e[threadIdx.x] = t.best[threadIdx.x];
  if (threadIdx.x == 0) t.n = m;
  __syncthreads();
  return m;
}
}  // namespace

template <int DT, bool TOP>
__global__ void __launch_bounds__(kLThr, 2) logprobs_kernel(const LogpArgs a) {
  using E = El<DT>;
  __shared__ TopList list;
  __shared__ float s_group[kLGroups];
  __shared__ float s_bar, s_w[3][kLWarps];
  __shared__ int s_scan[kLWarps], s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.S, cut = blockIdx.x - row * a.S;
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
  const char* base = x0 - shift * E::kE;
  const int n_vec = (a.V + shift + E::kN - 1) / E::kN;
  auto first_of = [&](int chunk, int j) { return ((chunk * kVec + j) * kLThr + tid) * E::kN - shift; };
  auto load = [&](int chunk, uint4 (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int e0 = first_of(chunk, j);
      if (e0 >= 0 && e0 + E::kN <= a.V) {
        v[j] = load_stream(x0 + (int64_t)e0 * E::kE);
        continue;
      }
      uint32_t w[4] = {E::kNone, E::kNone, E::kNone, E::kNone};
      if (e0 + E::kN > 0 && e0 < a.V) {
#pragma unroll
        for (int i = 0; i < E::kN; ++i) {
          if (e0 + i < 0 || e0 + i >= a.V) continue;
          if (DT == MOE_DTYPE_FP32) {
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(x0) + e0 + i);
          } else {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(x0) + e0 + i);
            w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | h << 16 : (w[i / 2] & 0xFFFF0000u) | h;
          }
        }
      }
      v[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  const int c0 = cut * a.per, c1 = min(c0 + a.per, (n_vec + kLThr * kVec - 1) / (kLThr * kVec));
  Sums s{-INFINITY, 0.0f, 0.0f};
  float bar = -INFINITY;  // what a further element has to be above
  int n_list = 0;         // entries of the list at the last count
  bool full = false;      // k of them are known: the bar holds for what follows
  if (TOP && tid == 0) list.n = 0;
  if (TOP) __syncthreads();
  uint4 v[kVec], nv[kVec];
  if (c0 < c1) load(c0, v);
  for (int c = c0; c < c1; ++c) {
    if (c + 1 < c1) load(c + 1, nv);
    const float top = max_of<DT>(v);
    if (top > s.m) raise(s, top);
    if (s.m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int i = 0; i < E::kN; ++i) {
          // e^-200 is 0, and 0 times it, too, where x is -inf
          const float d = max_nan(el_at<DT>(v[j], i) - s.m, -200.0f);
          const float e = ex2(d * 1.4426950408889634f);
          s.Z += e;
          s.A = fmaf(e, d, s.A);
        }
    }
    if (TOP) {
      // lists what `want` takes; the place of this thread's last one, or -1
      auto push = [&](auto want) {
        int at = -1;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
#pragma unroll
          for (int i = 0; i < E::kN; ++i) {
            const float x = el_at<DT>(v[j], i);
            if (!want(x)) continue;
            at = atomicAdd(&list.n, 1);
            if (at < kCap) list.e[at] = Entry{x, first_of(c, j) + i};
          }
        return at;
      };
      bool over = !full;
      if (full) {
        int at = -1;
        if (top > bar) at = push([&](float x) { return x > bar; });
        if (__syncthreads_or(at >= kCap / 2)) {
          over = __syncthreads_or(at >= kCap);
          if (over) {  // only what was there before this chunk is whole
            const int begin = c * kVec * kLThr * E::kN - shift;
            for (int i = tid; i < kCap; i += kLThr)
              if (list.e[i].id >= begin) list.e[i].v = -INFINITY;
          }
          n_list = keep_best(list, over ? kCap : list.n, a.k);
          bar = list.e[a.k - 1].v;
        }
      }
      if (over) {
        // the bar that at least k of this chunk reach
        float g = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, 2));
        if ((tid & 3) == 0) s_group[tid >> 2] = g;
        if (tid == 0) {
          s_bar = -INFINITY;
          list.n = n_list;
        }
        __syncthreads();
        if (tid < kLGroups) {
          const float mine = s_group[tid];
          int rank = 0;
          for (int j = 0; j < kLGroups; ++j)
            rank += s_group[j] > mine || (s_group[j] == mine && j < tid);
          if (rank == a.k - 1) s_bar = mine;
        }
        __syncthreads();
        // equals of an earlier chunk's bar have lower ids
        const float low = fmaxf(s_bar, bar);
        const bool strict = full && low == bar;
        auto above = [&](float x) { return x > low; };
        auto reach = [&](float x) { return x >= low && x > -INFINITY; };
        int at = -1;
        if (strict ? top > low : top >= low) at = strict ? push(above) : push(reach);
        if (__syncthreads_or(at >= kCap)) {
          // too many: those above the bar, then the first of its equals
          if (tid == 0) list.n = n_list;
          __syncthreads();
          at = top > low ? push(above) : -1;
          if (__syncthreads_or(at >= kCap)) {
            // still too many: the best k one after the other
            if (tid == 0) list.n = n_list;
            Entry last{INFINITY, -1};
            for (int r = 0; r < a.k; ++r) {
              Entry mine{-INFINITY, 0x7FFFFFFF};
#pragma unroll
              for (int j = 0; j < kVec; ++j)
#pragma unroll
                for (int i = 0; i < E::kN; ++i) {
                  const Entry x{el_at<DT>(v[j], i), first_of(c, j) + i};
                  if (before(last, x) && before(x, mine)) mine = x;
                }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) {
                const Entry y{__shfl_xor_sync(0xFFFFFFFFu, mine.v, o), __shfl_xor_sync(0xFFFFFFFFu, mine.id, o)};
                if (before(y, mine)) mine = y;
              }
              __syncthreads();
              if (lane == 0) list.best[warp] = mine;
              __syncthreads();
              last = list.best[0];
              for (int w = 1; w < kLWarps; ++w)
                if (before(list.best[w], last)) last = list.best[w];
              if (tid == 0 && last.v > -INFINITY) list.e[list.n++] = last;
            }
          } else if (!strict && list.n - n_list < a.k && low > -INFINITY) {
            int need = a.k - (list.n - n_list), have = list.n;  // the same for all
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
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
                  if (start < need) list.e[have + start] = Entry{low, first_of(c, j) + i};
                  ++start;
                }
              const int took = min(all, need);
              have += took;
              need -= took;
            }
            __syncthreads();
            if (tid == 0) list.n = have;
          }
        }
        __syncthreads();
        n_list = keep_best(list, list.n, a.k);
        full = n_list == a.k;
        bar = full ? list.e[a.k - 1].v : -INFINITY;
      }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = nv[j];
  }
  if (TOP) {
    __syncthreads();
    n_list = keep_best(list, list.n, a.k);
  }
  // ---- the CTA's sums, in a fixed order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    join(s, Sums{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.Z, o),
                 __shfl_xor_sync(0xFFFFFFFFu, s.A, o)});
  if (lane == 0) {
    s_w[0][warp] = s.m;
    s_w[1][warp] = s.Z;
    s_w[2][warp] = s.A;
  }
  __syncthreads();
  s = Sums{s_w[0][0], s_w[1][0], s_w[2][0]};
  for (int w = 1; w < kLWarps; ++w) join(s, Sums{s_w[0][w], s_w[1][w], s_w[2][w]});
  if (a.S > 1) {
    float* part = a.part + (int64_t)blockIdx.x * kLPart;
    if (tid == 0) {
      part[0] = s.m;
      part[1] = s.Z;
      part[2] = s.A;
      part[3] = __int_as_float(n_list);
    }
    if (tid < n_list) {
      part[4 + tid] = list.e[tid].v;
      part[4 + kMostTop + tid] = __int_as_float(list.e[tid].id);
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
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      join(s, Sums{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.Z, o),
                   __shfl_xor_sync(0xFFFFFFFFu, s.A, o)});
    if (TOP) {
      for (int i = tid; i < a.S * kMostTop; i += kLThr) {
        const float* p = parts + i / kMostTop * kLPart;
        const int j = i % kMostTop;
        const float x = __ldcg(p + 4 + j), id = __ldcg(p + 4 + kMostTop + j);
        if (j < __float_as_int(__ldcg(p + 3)))
          list.e[atomicAdd(&list.n, 1)] = Entry{x, __float_as_int(id)};
      }
    }
    if (TOP) {
      __syncthreads();
      n_list = keep_best(list, list.n, a.k);
    }
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
  if (TOP && tid < a.k) {
    const bool here = ok && tid < n_list;
    const int64_t at = (int64_t)row * a.k + tid;
    if (a.top_ids) a.top_ids[at] = here ? list.e[tid].id : -1;
    if (a.top_logp) a.top_logp[at] = here ? (list.e[tid].v - s.m) - lz : -INFINITY;
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
  // rows are cut where there are fewer than CTAs that fit at once, two an SM
  int most = 2 * nsm < kMostParts ? 2 * nsm : kMostParts;
  most /= s->n_rows;
  if (most > kCap / kMostTop) most = kCap / kMostTop;  // whose entries one list holds
  const int cuts = most < 1 ? 1 : most < chunks ? most : chunks;
  a.per = (chunks + cuts - 1) / cuts;
  a.S = (chunks + a.per - 1) / a.per;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((unsigned)s->n_rows * a.S), dim3(kLThr), 0, stream, a);
  };
  const bool top = s->k > 0 && (top_ids || top_logp);
  if (s->dtype == MOE_DTYPE_FP32)
    return top ? go(logprobs_kernel<MOE_DTYPE_FP32, true>) : go(logprobs_kernel<MOE_DTYPE_FP32, false>);
  if (s->dtype == MOE_DTYPE_FP16)
    return top ? go(logprobs_kernel<MOE_DTYPE_FP16, true>) : go(logprobs_kernel<MOE_DTYPE_FP16, false>);
  return top ? go(logprobs_kernel<MOE_DTYPE_BF16, true>) : go(logprobs_kernel<MOE_DTYPE_BF16, false>);
}

}  // namespace moe

// Rows of a block-paged key/value cache held in 4 bits: written (quantised)
// and read back.
//
// A row is one position of one head, D elements in four groups of D / 4:
//   b = the largest bf16 number <= min, s = bf16((max - b) / 15), to nearest,
//   code = min(15, floor((x - b) / s + 1/2)), 0 where s = 0;
// a code stands for s * code + b. Rounding b down keeps every x - b >= 0, so
// that the 16 codes cover the whole group; it is exact for bf16 rows.
//
// Codes and scales are decided as the formulas say, not as roundings fall:
// fp32 finds the code, and where it comes within its own error of a border
// (2^-16 of a step, once in some ten thousand elements) the sign of
// x - b - (c + 1/2) s is taken without error. Two machines, or this kernel and
// a reference in 64 bits, so write the same cache.
//
// Layout of a row, 16-bit units: D / 4 units of codes, s[4], b[4]: 80 bytes
// for D = 128, 48 for D = 64. Element e's code is nibble e % 2 of byte e / 2;
// with D = 64 the bytes of groups 2 h and 2 h + 1 alternate, so that a group
// fills one half of every 16-bit unit: a 16-position step of the attention's
// matrix products then has one scale whatever D is. Rows of 80 and 48 bytes
// also spread over the shared-memory banks as they are (eight rows' 16-byte
// pieces never meet in one), so pages are copied as they lie.
#include "attn_q4.cuh"

namespace moe {

namespace {
constexpr int kPage = 64;  // positions per page
constexpr int kThr = 256;
constexpr int kRows = 4;   // rows a thread has a piece of

template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // NaN if either is
  uint32_t r;
  if (F16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ float lo_of(uint32_t v) {
  return F16 ? half_bits_to_float(v & 0xFFFFu) : bf_lo(v);
}
template <bool F16>
__device__ __forceinline__ float hi_of(uint32_t v) {
  return F16 ? half_bits_to_float(v >> 16) : bf_hi(v);
}
// what a - b leaves over, a - b = d + rest, d = fl(a - b)
__device__ __forceinline__ float sub_rest(float a, float b, float d) {
  const float z = __fsub_rn(d, a);
  return __fsub_rn(__fsub_rn(a, __fsub_rn(d, z)), __fadd_rn(b, z));
}
// bits of the largest bf16 number that is not above v
__device__ __forceinline__ uint32_t floor_bf16(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v != v) return 0x7FC0u;
  return (v < 0.0f ? u + 0xFFFFu : u) >> 16;
}
// bits of the bf16 number nearest to (hi - b) / 15, ties to even. The fp32
// quotient can only be wrong about the side of a midpoint by being one (a
// midpoint and its multiple by 15 are fp32 numbers, and rounding keeps order).
__device__ __forceinline__ uint32_t scale_bits(float hi, float b) {
  const float d = __fsub_rn(hi, b), q = __fdiv_rn(d, 15.0f);
  const uint32_t u = __float_as_uint(q), low = u & 0xFFFFu;
  if (q != q) return 0x7FC0u;
  bool up = low > 0x8000u;
  if (low == 0x8000u) {
    const float over = __fadd_rn(fmaf(-15.0f, q, d), sub_rest(hi, b, d));
    up = over > 0.0f || (over == 0.0f && (u & 0x10000u));
  }
  return (u >> 16) + up;
}

// the code of x where fp32 cannot tell: the border next to x is (c + 1/2) s
__device__ __noinline__ uint32_t code_exact(float x, float b, float s, float f) {
  const float c = floorf(f);
  if (!(c >= 0.0f) || c >= 15.0f) return c >= 15.0f ? 15u : 0u;
  const float d = __fsub_rn(x, b);
  // (c + 1/2) s has 13 bits, and d is next to it: both steps are exact
  const float over = __fadd_rn(__fsub_rn(d, __fmul_rn(c + 0.5f, s)), sub_rest(x, b, d));
  return (uint32_t)c + (over >= 0.0f);
}
// eight elements' codes, the first in the lowest bits
template <bool F16>
__device__ __forceinline__ uint32_t codes8(const uint4& v, float b, float s) {
  if (!(s > 0.0f)) return 0u;
  // 1 / s is a normal number from 2^-126 to 2^126; smaller scales (bf16 has
  // seven binades of them) go through 2^20 s
  const float up = s < 0x1p-120f ? 0x1p20f : 1.0f, inv = 1.0f / (s * up);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = i & 1 ? hi_of<F16>(w[i / 2]) : lo_of<F16>(w[i / 2]);
    const float f = fminf((x - b) * up * inv, 15.0f);
    const float t = f + 0x1.8p23f;  // the nearest whole number in the low bits
    uint32_t c = __float_as_uint(t) & 15u;
    // f is off by less than 2^-18 (three roundings of 2^-24 below 16)
    if (fabsf(f - (t - 0x1.8p23f)) > 0.5f - 0x1p-16f) c = code_exact(x, b, s, f);
    r |= c << (4 * i);
  }
  return r;
}
}  // namespace

// A thread has eight elements of kRows rows: of tokens one after the other, of
// one head and tensor (blockIdx.y), so that a CTA reads whole lines and writes
// a stretch of a page.
template <bool F16, int D>
__global__ void __launch_bounds__(kThr)
    cache_write_q4_kernel(const CacheQ4Args a, const uint16_t* __restrict__ k_new, int64_t k_stride,
                          const uint16_t* __restrict__ v_new, int64_t v_stride) {
  constexpr int kLanes = D / 8;          // threads of a row
  constexpr int kStep = kThr / kLanes;   // rows of a pass
  constexpr int kUnits = q4_units(D);
  const int part = threadIdx.x % kLanes, g = part * 8 / (D / 4);
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const uint16_t* from = (is_v ? v_new : k_new) + head * D + part * 8;
  const int64_t stride = is_v ? v_stride : k_stride;
  uint16_t* pool = static_cast<uint16_t*>(is_v ? a.v : a.k) + (int64_t)head * kPage * kUnits;
  pdl_wait();
  pdl_trigger();
  const int64_t all = (int64_t)a.n_slots * a.T;
  const int64_t tok0 = (int64_t)blockIdx.x * (kStep * kRows) + threadIdx.x / kLanes;
  uint4 x[kRows];
  int64_t at[kRows];  // the row's place in the pool, -1: nothing to write
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t tok = tok0 + k * kStep;
    at[k] = -1;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (tok >= all) continue;
    const int s = (int)(tok / a.T), t = (int)(tok - (int64_t)s * a.T);
    const int n = a.n ? __ldg(a.n + s) : a.T, len = __ldg(a.lens + s);
    if (n < 0 || n > a.T || len < n || len > a.max_blocks * kPage) {
      if (part == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
      continue;
    }
    if (t >= n) continue;
    const int pos = len - n + t;
    x[k] = __ldg(reinterpret_cast<const uint4*>(from + tok * stride));
    const int page = __ldg(a.table + (int64_t)s * a.max_blocks + pos / kPage);
    if (page < 0 || page >= a.n_phys) {
      if (part == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
      continue;
    }
    at[k] = ((int64_t)page * a.n_kv * kPage + pos % kPage) * kUnits;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    // all lanes take part in the exchanges, rows that are not there as zeros
    uint32_t lo = min2<F16>(min2<F16>(x[k].x, x[k].y), min2<F16>(x[k].z, x[k].w));
    uint32_t hi = max2<F16>(max2<F16>(x[k].x, x[k].y), max2<F16>(x[k].z, x[k].w));
#pragma unroll
    for (int d = 1; d < D / 32; d <<= 1) {
      lo = min2<F16>(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
      hi = max2<F16>(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
    }
    lo = min2<F16>(lo, lo >> 16 | lo << 16);
    hi = max2<F16>(hi, hi >> 16 | hi << 16);
    const uint32_t bb = floor_bf16(lo_of<F16>(lo));
    const float b = __uint_as_float(bb << 16);
    const uint32_t sb = scale_bits(lo_of<F16>(hi), b);
    uint32_t w = codes8<F16>(x[k], b, __uint_as_float(sb << 16));
    int word = part;
    if (D == 64) {  // bytes of groups 2 h and 2 h + 1 alternate
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 2);
      w = part & 2 ? __byte_perm(o, w, 0x7362) : __byte_perm(w, o, 0x5140);
      word = (part & 4) + (part & 1) * 2 + (part >> 1 & 1);
    }
    if (at[k] < 0) continue;
    uint16_t* row = pool + at[k];
    reinterpret_cast<uint32_t*>(row)[word] = w;
    if (part % (D / 32) == 0) {
      row[D / 4 + g] = (uint16_t)sb;
      row[D / 4 + 4 + g] = (uint16_t)bb;
    }
  }
}

// The same arrangement the other way. DT: moe_dtype_t of what comes out, each
// value rounded once.
template <int DT, int D>
__global__ void __launch_bounds__(kThr)
    cache_read_q4_kernel(const CacheQ4Args a, const int32_t* __restrict__ first,
                         void* __restrict__ k_out, int64_t k_stride, void* __restrict__ v_out,
                         int64_t v_stride) {
  constexpr int kLanes = D / 8, kStep = kThr / kLanes, kUnits = q4_units(D);
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2;
  const int part = threadIdx.x % kLanes;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  char* to = static_cast<char*>(is_v ? v_out : k_out) + (int64_t)head * D * kE;
  const int64_t stride = is_v ? v_stride : k_stride;
  const uint16_t* pool = static_cast<const uint16_t*>(is_v ? a.v : a.k) + (int64_t)head * kPage * kUnits;
  pdl_wait();
  pdl_trigger();
  const int64_t all = (int64_t)a.n_slots * a.T;
  const int64_t tok0 = (int64_t)blockIdx.x * (kStep * kRows) + threadIdx.x / kLanes;
  // D = 64: a word holds four elements of group 2 h and four of 2 h + 1
  const int ga = D == 128 ? part / 4 : part / 4 * 2, gb = D == 128 ? ga : ga + 1;
  uint32_t w[kRows], sb[kRows][2], bb[kRows][2];
  bool there[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t tok = tok0 + k * kStep;
    there[k] = false;
    if (tok >= all) continue;
    const int s = (int)(tok / a.T), t = (int)(tok - (int64_t)s * a.T);
    const int n = a.n ? __ldg(a.n + s) : a.T, len = __ldg(a.lens + s);
    const int f = first ? __ldg(first + s) : 0;
    if (n < 0 || n > a.T || len < 0 || len > a.max_blocks * kPage || (n > 0 && (f < 0 || f > len - n))) {
      if (part == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
      continue;
    }
    if (t >= n) continue;
    const int pos = f + t;
    const int page = __ldg(a.table + (int64_t)s * a.max_blocks + pos / kPage);
    if (page < 0 || page >= a.n_phys) {
      if (part == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
      continue;
    }
    const uint16_t* row = pool + ((int64_t)page * a.n_kv * kPage + pos % kPage) * kUnits;
    w[k] = __ldg(reinterpret_cast<const uint32_t*>(row) + part);
    sb[k][0] = __ldg(row + D / 4 + ga);
    bb[k][0] = __ldg(row + D / 4 + 4 + ga);
    if (D == 64) {
      sb[k][1] = __ldg(row + D / 4 + gb);
      bb[k][1] = __ldg(row + D / 4 + 4 + gb);
    }
    there[k] = true;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (!there[k]) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = D == 64 ? i >> 1 & 1 : 0;  // D = 64: nibbles 2, 3, 6, 7 are of the second group
      v[i] = fmaf((float)(w[k] >> (4 * i) & 15u), __uint_as_float(sb[k][p] << 16),
                  __uint_as_float(bb[k][p] << 16));
    }
    uint32_t o[8];
    if (DT == MOE_DTYPE_FP32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack2<DT == MOE_DTYPE_FP16>(v[2 * i], v[2 * i + 1]);
    }
    const int64_t tok = tok0 + k * kStep;
    if (D == 128) {
      uint4* p = reinterpret_cast<uint4*>(to + (tok * stride + part * 8) * kE);
      p[0] = make_uint4(o[0], o[1], o[2], o[3]);
      if (DT == MOE_DTYPE_FP32) p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
      char* p = to + (tok * stride + (part >> 2) * 32 + (part & 3) * 4) * kE;
      if (DT == MOE_DTYPE_FP32) {
        *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[4], o[5]);
        *reinterpret_cast<uint4*>(p + 16 * kE) = make_uint4(o[2], o[3], o[6], o[7]);
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[2]);
        *reinterpret_cast<uint2*>(p + 16 * kE) = make_uint2(o[1], o[3]);
      }
    }
  }
}

bool cache_q4_supported(const moe_cache_shape_t* s) {
  return cache_supported(s) && q4_units(s->D) > 0;
}

namespace {
CacheQ4Args args_of(const moe_cache_shape_t* s, const moe_cache_meta_t& meta, const int32_t* n,
                    int T, void* k, void* v, uint8_t* ws) {
  CacheQ4Args a;
  a.table = meta.table_dev;
  a.lens = meta.lens_dev;
  a.n = n;
  a.k = k;
  a.v = v;
  a.n_slots = s->n_slots;
  a.T = T;
  a.max_blocks = s->max_blocks;
  a.n_phys = s->n_phys;
  a.n_kv = s->n_kv;
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  return a;
}
// tokens of a CTA: kThr / (D / 8) * kRows
dim3 grid_of(const moe_cache_shape_t* s, int T) {
  const int64_t per = (int64_t)kThr / (s->D / 8) * kRows, n = (int64_t)s->n_slots * T;
  return dim3((unsigned)((n + per - 1) / per), 2 * s->n_kv);
}
}  // namespace

cudaError_t launch_cache_write_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                  const int32_t* n_new, int T, const uint16_t* k_new,
                                  int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                                  bool fp16, void* k, void* v, uint8_t* ws, cudaStream_t stream) {
  const CacheQ4Args a = args_of(s, meta, n_new, T, k, v, ws);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid_of(s, T), dim3(kThr), 0, stream, a, k_new, k_stride, v_new, v_stride);
  };
  if (s->D == 64) return fp16 ? go(cache_write_q4_kernel<true, 64>) : go(cache_write_q4_kernel<false, 64>);
  return fp16 ? go(cache_write_q4_kernel<true, 128>) : go(cache_write_q4_kernel<false, 128>);
}

cudaError_t launch_cache_read_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                 const int32_t* first, const int32_t* n, int T, const void* k,
                                 const void* v, void* k_out, int64_t k_stride, void* v_out,
                                 int64_t v_stride, int dtype, uint8_t* ws, cudaStream_t stream) {
  const CacheQ4Args a = args_of(s, meta, n, T, const_cast<void*>(k), const_cast<void*>(v), ws);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid_of(s, T), dim3(kThr), 0, stream, a, first, k_out, k_stride, v_out, v_stride);
  };
  if (s->D == 64) {
    if (dtype == MOE_DTYPE_FP32) return go(cache_read_q4_kernel<MOE_DTYPE_FP32, 64>);
    return dtype == MOE_DTYPE_FP16 ? go(cache_read_q4_kernel<MOE_DTYPE_FP16, 64>)
                                   : go(cache_read_q4_kernel<MOE_DTYPE_BF16, 64>);
  }
  if (dtype == MOE_DTYPE_FP32) return go(cache_read_q4_kernel<MOE_DTYPE_FP32, 128>);
  return dtype == MOE_DTYPE_FP16 ? go(cache_read_q4_kernel<MOE_DTYPE_FP16, 128>)
                                 : go(cache_read_q4_kernel<MOE_DTYPE_BF16, 128>);
}

}  // namespace moe

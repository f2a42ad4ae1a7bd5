// Rows of a block-paged key/value cache held in 4 bits: written (quantised)
// and read back.
//
// A row is one position of one head, D elements in four groups of D / 4:
//   b = the largest bf16 number <= min, s = bf16((max - b) / 15), to nearest,
//   code = min(15, floor((x - b) / s + 1/2)), 0 where s = 0;
// a code stands for s * code + b. Rounding b down keeps every x - b >= 0, so
// that the 16 codes cover the whole group; it is exact for bf16 rows.
//
// Codes and scales are decided as the formulas say, not as roundings fall, so
// two machines, or this kernel and a reference in 64 bits, write the same cache.
// (x - b) / s meets borders c + 1/2 exactly quite often, as 16-bit numbers have
// few digits. But what is not on a border is not near it either: x - b and
// (c + 1/2) s are multiples of q, the least of x's, b's and s / 2's last places,
// so that the quotient misses by q / s, which is 2^-16 or more unless x or b is
// tiny beside s. So fp32 with a factor of 1 + 2^-21 (+-2^-22, all roundings
// counted) takes every border upwards and nothing else: the quotient below 15.1
// moves by less than 2^-16.4. A tiny x lies next to -b / s; where that is next to
// a border, or b is tiny, or s so small that its reciprocal is not a normal
// number, each code is taken from the sign of x - b - (c + 1/2) s without error.
//
// Layout of a row, 16-bit units: D / 4 units of codes, s[4], b[4]: 80 bytes
// for D = 128, 48 for D = 64. Element e's code is nibble e % 2 of byte e / 2;
// with D = 64 the bytes of groups 2 h and 2 h + 1 alternate, so that a group
// fills one half of every 16-bit unit: a 16-position step of the attention's
// matrix products then has one scale whatever D is. Rows of 80 and 48 bytes
// also spread over the shared-memory banks as they are (eight rows' 16-byte
// pieces never meet in one), so pages are copied as they lie.
//
// Bound: both by HBM. A thread has sixteen elements of a row, whose group it
// shares with one other (D = 128) or has alone, so that a row's bookkeeping and
// a group's scale are paid once for as many; fp32 pairs share instructions, no
// element branches, and nothing divides. 111 thousand positions of 2 heads of
// 128 written, 148 MB, take 32 to 35 us, 4.2 to 4.7 TB/s (120 instructions a thread
// and row), and read back 26 to 28 us, 5.3 to 5.6 TB/s. Writing fills no pipe:
// instructions are issued in 70 cycles of a hundred, the integer pipe is busy in
// 57, 43 warps of a hundred are there, and every pass waits for its own rows. fp16
// rows take 54 us: what counts as tiny beside a scale is 2^-5 of it there, 2^-8 for
// bf16, and more groups have to be looked through for it. (Eight elements a thread,
// a division a group and each code checked for a border by itself took 78 and 50;
// borders checked by how near fp32 comes to them 61, as 16-bit numbers meet borders
// in most warps.)
#include <type_traits>

#include "attn_q4.cuh"

namespace moe {

namespace {
constexpr int kPage = 64;  // positions per page
constexpr int kThr = 256;
constexpr int kRows = 2;   // rows a thread has a piece of
constexpr int kMostCtas = 4096;  // where slots have more tokens than a pass, or a CTA a slot

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
__device__ __forceinline__ uint64_t both(float a) { return pair2(__float_as_uint(a), __float_as_uint(a)); }
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
// Bits of the bf16 number nearest to (hi - b) / 15, ties to even. An fp32
// product with 1/15 is off by less than two of its last places; near a midpoint
// of bf16 numbers the sign of hi - b - 15 midpoint says it without error.
__device__ __forceinline__ uint32_t scale_bits(float hi, float b) {
  const float d = __fsub_rn(hi, b), q = d * (1.0f / 15.0f);
  const uint32_t u = __float_as_uint(q), low = u & 0xFFFFu;
  if (q != q) return 0x7FC0u;
  uint32_t r = u + 0x8000u;  // no ties away from a midpoint
  if (low - 0x7FF8u <= 16u) {
    const uint32_t at = (u & 0xFFFF0000u) | 0x8000u;
    const float mid = __uint_as_float(at);
    // 15 mid has 13 bits; what it leaves of d is exact, as d is next to it
    const float over = __fadd_rn(fmaf(-15.0f, mid, d), sub_rest(hi, b, d));
    const bool up = over > 0.0f || (over == 0.0f && (at & 0x10000u));
    r = at + (up ? 0x8000u : 0u);
  }
  return r >> 16;
}

// the code of x: the borders around f are (c + 1/2) s
__device__ __forceinline__ uint32_t code_exact(float x, float b, float s, float f) {
  const float c = floorf(fminf(f, 15.0f));
  if (!(c >= 0.0f) || c >= 15.0f) return c >= 15.0f ? 15u : 0u;
  const float d = __fsub_rn(x, b);
  // (c + 1/2) s has 13 bits, and d is next to it: both steps are exact
  const float over = __fadd_rn(__fsub_rn(d, __fmul_rn(c + 0.5f, s)), sub_rest(x, b, d));
  return (uint32_t)c + (over >= 0.0f);
}
template <bool F16>
__device__ __noinline__ uint32_t codes_exact(uint4 v, float b, float s) {
  // 1 / s is a normal number down to 2^-126; smaller scales (bf16 has seven
  // binades of them) go through 2^20 s
  const float up = s < 0x1p-120f ? 0x1p20f : 1.0f, inv = 1.0f / (s * up);
  uint32_t r = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    const float x = i & 1 ? unpack_hi<F16>(w) : unpack_lo<F16>(w);
    r |= code_exact(x, b, s, (x - b) * up * inv) << (4 * i);
  }
  return r;
}
// Eight elements' codes, the first in the lowest bits; up = (1 + 2^-21) / s.
template <bool F16>
__device__ __forceinline__ uint32_t codes8(const uint4& v, float b, float up) {
  const uint64_t nb = both(-b), f2 = both(up), magic = both(0x1.8p23f);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // 1.5 2^23 + c is 0x4B400000 + c: of the sum of 16^i times that, the constant
  uint32_t r = 0u - 0x3F400000u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = pair2(__float_as_uint(unpack_lo<F16>(w[i])), __float_as_uint(unpack_hi<F16>(w[i])));
    const uint64_t c = fma2(add2(x, nb), f2, magic);
    r += (uint32_t)c << (8 * i);
    r += (uint32_t)(c >> 32) << (8 * i + 4);
  }
  return r;
}
// Whether the codes of these elements want codes_exact. tiny: below how many s
// an x has a last place below 2^-16 s.
template <bool F16>
__device__ __forceinline__ bool in_doubt(const uint4 (&v)[2], float b, float s, float up) {
  constexpr float kTiny = F16 ? 0x1p-5f : 0x1p-8f;
  const float fb = fabsf(b) * up + 0.5f;  // a whole number on a border
  const bool border = fabsf(fb - rintf(fb)) < kTiny + 0x1p-14f;
  if (!border && fabsf(b) >= s * kTiny && s >= 0x1p-120f) return false;
  if (s < 0x1p-120f || (b != 0.0f && fabsf(b) < s * kTiny)) return true;
  bool found = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = fabsf(unpack_lo<F16>(w[i])), x1 = fabsf(unpack_hi<F16>(w[i]));
      found |= (x0 > 0.0f && x0 < s * kTiny) || (x1 > 0.0f && x1 < s * kTiny);
    }
  }
  return border && found;
}

// Where a call's rows lie. LONG: a CTA has one slot's tokens, its passes go on
// along them, and where the slot has more than its n CTAs take at once the CTA
// goes on n times as far; else 2^n tokens of some slots a pass, and its passes go
// on along the slots.
template <int D, bool LONG>
struct Rows {
  static constexpr int kStep = kThr / (D / 16);  // rows of a pass
  int s0, t0, n;
  __device__ __forceinline__ explicit Rows(int n_) : n(n_) {
    const int r = threadIdx.x / (D / 16);
    if (LONG) {
      s0 = blockIdx.x / (unsigned)n;
      t0 = ((int)blockIdx.x - s0 * n) * (kStep * kRows) + r;
    } else {
      s0 = ((int)blockIdx.x * (kRows * kStep) + r) >> n;
      t0 = r & ((1 << n) - 1);
    }
  }
  __device__ __forceinline__ int slot(int k) const { return LONG ? s0 : s0 + (k * kStep >> n); }
  __device__ __forceinline__ int token(int k) const { return LONG ? t0 + k * kStep : t0; }
  // goes on along the slot, false (for the whole CTA) behind its last token
  __device__ __forceinline__ bool next(int tokens) {
    t0 += n * (kStep * kRows);
    return LONG && t0 - (int)threadIdx.x / (D / 16) < tokens;
  }
};
// A slot's new rows (write) or rows to read: the first one's position and how
// many, 0 where the numbers are out of range.
struct Span {
  int pos, n;
};
__device__ __forceinline__ Span span_of(const CacheQ4Args& a, const int32_t* first, bool read, int s) {
  const int n = a.n ? __ldg(a.n + s) : a.T, len = __ldg(a.lens + s);
  const int pos = read ? (first ? __ldg(first + s) : 0) : len - n;
  if (n < 0 || n > a.T || len < 0 || len > a.max_blocks * kPage || (n > 0 && (pos < 0 || pos > len - n))) {
    set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    return Span{0, 0};
  }
  return Span{pos, n};
}
// The page of a position, -1 where there is none.
__device__ __forceinline__ int page_of(const CacheQ4Args& a, int s, int pos) {
  const int page = __ldg(a.table + (int64_t)s * a.max_blocks + pos / kPage);
  if ((unsigned)page < (unsigned)a.n_phys) return page;
  set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
  return -1;
}
}  // namespace

// A thread has sixteen elements of kRows rows of one head and tensor
// (blockIdx.y), a CTA tokens one after the other: it reads whole lines and
// writes a stretch of a page.
template <bool F16, int D, bool LONG>
__global__ void __launch_bounds__(kThr)
    cache_write_q4_kernel(const CacheQ4Args a, int plan, const uint16_t* __restrict__ k_new,
                          int64_t k_stride, const uint16_t* __restrict__ v_new, int64_t v_stride) {
  constexpr int kLanes = D / 16;         // threads of a row
  constexpr int kUnits = q4_units(D);
  const int part = threadIdx.x % kLanes, head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const uint16_t* from = (is_v ? v_new : k_new) + head * D + part * 16;
  const int64_t stride = is_v ? v_stride : k_stride;
  uint16_t* pool = static_cast<uint16_t*>(is_v ? a.v : a.k) + (int64_t)head * kPage * kUnits;
  pdl_wait();
  pdl_trigger();
  Rows<D, LONG> rows(plan);
  Span sp{0, 0};
  if (LONG) {
    sp = span_of(a, nullptr, false, rows.s0);
    if (rows.t0 - (int)threadIdx.x / kLanes >= sp.n) return;  // the whole CTA
  }
  do {
    uint4 x[kRows][2];
    int64_t at[kRows];  // the row's place in the pool, -1: nothing to write
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int s = rows.slot(k), tok = rows.token(k);
      at[k] = -1;
      x[k][0] = x[k][1] = make_uint4(0u, 0u, 0u, 0u);
      if (!LONG) sp = s < a.n_slots ? span_of(a, nullptr, false, s) : Span{0, 0};
      if (tok >= sp.n) continue;
      const uint4* p = reinterpret_cast<const uint4*>(from + ((int64_t)s * a.T + tok) * stride);
      x[k][0] = __ldg(p);
      x[k][1] = __ldg(p + 1);
      const int pos = sp.pos + tok, page = page_of(a, s, pos);
      if (page >= 0) at[k] = ((int64_t)page * a.n_kv * kPage + pos % kPage) * kUnits;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      // all lanes take part in the exchanges, rows that are not there as zeros
      const uint4 &y = x[k][0], &z = x[k][1];
      uint32_t lo = min2<F16>(min2<F16>(min2<F16>(y.x, y.y), min2<F16>(y.z, y.w)),
                              min2<F16>(min2<F16>(z.x, z.y), min2<F16>(z.z, z.w)));
      uint32_t hi = max2<F16>(max2<F16>(max2<F16>(y.x, y.y), max2<F16>(y.z, y.w)),
                              max2<F16>(max2<F16>(z.x, z.y), max2<F16>(z.z, z.w)));
      if (D == 128) {  // two threads a group
        lo = min2<F16>(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, 1));
        hi = max2<F16>(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, 1));
      }
      lo = min2<F16>(lo, lo >> 16 | lo << 16);
      hi = max2<F16>(hi, hi >> 16 | hi << 16);
      const uint32_t bb = floor_bf16(unpack_lo<F16>(lo));
      const float b = __uint_as_float(bb << 16);
      const uint32_t sb = scale_bits(unpack_lo<F16>(hi), b);
      const float s = __uint_as_float(sb << 16);
      float up;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(up) : "f"(s));  // within 2^-23
      up *= 1.0f + 0x1p-21f;
      uint32_t w0 = codes8<F16>(y, b, up), w1 = codes8<F16>(z, b, up);
      if (in_doubt<F16>(x[k], b, s, up)) {
        w0 = s > 0.0f ? codes_exact<F16>(y, b, s) : 0u;
        w1 = s > 0.0f ? codes_exact<F16>(z, b, s) : 0u;
      }
      int word = 2 * part;
      if (D == 64) {
        // bytes of groups 2 h (this thread's or its neighbour's) and 2 h + 1 alternate
        const bool odd = part & 1;
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, odd ? w0 : w1, 1);
        const uint32_t p = odd ? o : w0, q = odd ? w1 : o;
        w0 = __byte_perm(p, q, 0x5140);
        w1 = __byte_perm(p, q, 0x7362);
      }
      if (at[k] < 0) continue;
      uint16_t* row = pool + at[k];
      *reinterpret_cast<uint2*>(row + 2 * word) = make_uint2(w0, w1);
      if (D == 64 || part % 2 == 0) {
        const int g = D == 64 ? part : part / 2;
        row[D / 4 + g] = (uint16_t)sb;
        row[D / 4 + 4 + g] = (uint16_t)bb;
      }
    }
  } while (rows.next(sp.n));
}

// s c + b in fp32, rounded to odd: rounded down and up it is the same number, or
// two neighbours of which one has an odd last place, and that one is taken. What
// is not exact then ends in a 1 below all of fp16's places, so that the rounding
// to fp16 is the only one that shows. (Rounded to nearest first, a product of
// twelve bits that is a tie of fp16 loses a bias below 2^-24 of it, and the tie
// may go to the wrong side.) Of an exact 0, the one rounded up counts: +0.
__device__ __forceinline__ float affine_odd(float c, float s, float b) {
  const float down = __fmaf_rd(c, s, b), up = __fmaf_ru(c, s, b);
  return __float_as_uint(down) & 1u ? down : up;
}
// Whether s c + b can want more than fp32's 24 places for a code c: a bf16 number
// with exponent e lies below 2^(e + 1) and on multiples of 2^(e - 7), so that the
// sum has at most eb - es + 9 places where b is the larger, es - eb + 13 where s
// is. (s, b: bits in the low half.) 16 times 4096 positions of 8 heads of 128 to
// fp16 take 61.1 us, of 64 39.0, a call a graph; with all rows rounded to odd
// 65.9 and 41.0, with none 62.3 and 35.0.
__device__ __forceinline__ bool past_fp32(uint32_t s, uint32_t b) {
  const int apart = (int)(b >> 7 & 0xFFu) - (int)(s >> 7 & 0xFFu);
  return (b & 0x7FFFu) != 0u && (apart > 15 || apart < -11);
}
// Eight codes of a word as numbers s c + b, each rounded once: to four words of
// 16-bit pairs or eight of fp32. D = 64: nibbles 2, 3, 6 and 7 are of the second
// group (s1, b1), and pairs come as 0 1, 4 5, 2 3, 6 7: each group's together.
template <int DT, int D>
__device__ __forceinline__ void values8(uint32_t w, uint32_t s0, uint32_t b0, uint32_t s1, uint32_t b1,
                                        uint32_t (&o)[DT == MOE_DTYPE_FP32 ? 8 : 4]) {
  if constexpr (DT == MOE_DTYPE_BF16) {
    uint32_t p[4];  // nibbles i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool second = D == 64 && i >= 2;
      p[i] = affine_pair(nibble_pair_128(w >> (4 * i)), second ? s1 : s0, second ? b1 : b0);
    }
    o[0] = __byte_perm(p[0], p[1], 0x5410);
    o[D == 64 ? 2 : 1] = __byte_perm(p[2], p[3], 0x5410);
    o[D == 64 ? 1 : 2] = __byte_perm(p[0], p[1], 0x7632);
    o[3] = __byte_perm(p[2], p[3], 0x7632);
  } else {
    float v[8];
    auto all = [&](auto one) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool second = D == 64 && (i & 2);
        // 2^23 + c, less 2^23
        const float c = __uint_as_float((w >> (4 * i) & 15u) | 0x4B000000u) - 0x1p23f;
        v[i] = one(c, bf_lo(second ? s1 : s0), bf_lo(second ? b1 : b0));
      }
    };
    if (DT == MOE_DTYPE_FP16 && (past_fp32(s0, b0) || (D == 64 && past_fp32(s1, b1))))
      all([](float c, float s, float b) { return affine_odd(c, s, b); });
    else
      all([](float c, float s, float b) { return fmaf(c, s, b); });
    constexpr int to[4] = {0, D == 64 ? 2 : 1, D == 64 ? 1 : 2, 3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MOE_DTYPE_FP32) {
        o[2 * to[i]] = __float_as_uint(v[2 * i]);
        o[2 * to[i] + 1] = __float_as_uint(v[2 * i + 1]);
      } else {
        o[to[i]] = pack2<true>(v[2 * i], v[2 * i + 1]);
      }
    }
  }
}

// The same arrangement the other way. DT: moe_dtype_t of what comes out.
template <int DT, int D, bool LONG>
__global__ void __launch_bounds__(kThr)
    cache_read_q4_kernel(const CacheQ4Args a, int plan, const int32_t* __restrict__ first,
                         void* __restrict__ k_out, int64_t k_stride, void* __restrict__ v_out,
                         int64_t v_stride) {
  constexpr int kLanes = D / 16, kUnits = q4_units(D);
  constexpr int kE = DT == MOE_DTYPE_FP32 ? 4 : 2, kW = DT == MOE_DTYPE_FP32 ? 8 : 4;
  const int part = threadIdx.x % kLanes, head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  char* to = static_cast<char*>(is_v ? v_out : k_out) + (int64_t)head * D * kE;
  const int64_t stride = is_v ? v_stride : k_stride;
  const uint16_t* pool = static_cast<const uint16_t*>(is_v ? a.v : a.k) + (int64_t)head * kPage * kUnits;
  pdl_wait();
  pdl_trigger();
  // D = 128: two words of a group; D = 64: two words of half a row, each with
  // four elements of group 2 h and four of 2 h + 1
  const int ga = D == 128 ? part / 2 : part / 2 * 2, gb = D == 128 ? ga : ga + 1;
  Rows<D, LONG> rows(plan);
  Span sp{0, 0};
  if (LONG) {
    sp = span_of(a, first, true, rows.s0);
    if (rows.t0 - (int)threadIdx.x / kLanes >= sp.n) return;  // the whole CTA
  }
  do {
    uint2 w[kRows];
    uint32_t sa[kRows], ba[kRows], sb[kRows], bb[kRows];
    int64_t at[kRows];  // the token, -1: not there
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int s = rows.slot(k), tok = rows.token(k);
      at[k] = -1;
      if (!LONG) sp = s < a.n_slots ? span_of(a, first, true, s) : Span{0, 0};
      if (tok >= sp.n) continue;
      const int pos = sp.pos + tok, page = page_of(a, s, pos);
      if (page < 0) continue;
      const uint16_t* q = pool + ((int64_t)page * a.n_kv * kPage + pos % kPage) * kUnits;
      w[k] = __ldg(reinterpret_cast<const uint2*>(q) + part);
      sa[k] = __ldg(q + D / 4 + ga);
      ba[k] = __ldg(q + D / 4 + 4 + ga);
      sb[k] = D == 64 ? __ldg(q + D / 4 + gb) : 0u;
      bb[k] = D == 64 ? __ldg(q + D / 4 + 4 + gb) : 0u;
      at[k] = (int64_t)s * a.T + tok;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (at[k] < 0) continue;
      const uint32_t s0 = dup_lo(sa[k]), b0 = dup_lo(ba[k]), s1 = dup_lo(sb[k]), b1 = dup_lo(bb[k]);
      uint32_t o[2][kW];
      values8<DT, D>(w[k].x, s0, b0, s1, b1, o[0]);
      values8<DT, D>(w[k].y, s0, b0, s1, b1, o[1]);
      if (D == 128) {
        uint4* p = reinterpret_cast<uint4*>(to + (at[k] * stride + part * 16) * kE);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < kW; i += 4)
            p[(j * kW + i) / 4] = make_uint4(o[j][i], o[j][i + 1], o[j][i + 2], o[j][i + 3]);
      } else {
        // elements 8 (part % 2) .. + 7 of group 2 h, then of the next
        char* p = to + (at[k] * stride + (part >> 1) * 32 + (part & 1) * 8) * kE;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < kW; i += 4) {
            const int j = g * (kW / 2);
            uint4* q = reinterpret_cast<uint4*>(p + g * 16 * kE + i * 4);
            if (DT == MOE_DTYPE_FP32)
              *q = make_uint4(o[i / 4][j], o[i / 4][j + 1], o[i / 4][j + 2], o[i / 4][j + 3]);
            else
              *q = make_uint4(o[0][j], o[0][j + 1], o[1][j], o[1][j + 1]);
          }
      }
    }
  } while (rows.next(sp.n));
}

bool cache_q4_supported(const moe_cache_shape_t* s) {
  return cache_supported(s) && q4_units(s->D) > 0;
}

namespace {
template <int N>
using Int = std::integral_constant<int, N>;

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
// Rows' n, and whether slots have more tokens than a pass (LONG).
int plan_of(const moe_cache_shape_t* s, int T, bool* along, dim3* grid) {
  const int step = kThr / (s->D / 16);
  *along = T > step;
  if (*along) {
    // T may be far above what most slots have, and CTAs without a token cost their
    // start: 39 slots of up to 1119 positions of 8 heads, T 8049, were read in 82
    // us with a CTA for each stretch of T, in 18.7 with 4096 in all (18.2 with
    // 8192, 21.5 with 2048); 16 prompts written and read back 62.3 and 63.7. The
    // price: slots get the same number whatever they have, so one long slot among
    // many is worked through by few. 8192 tokens beside 255 slots of one are written
    // in 39 us with 2 heads and 140 with 8 (alone 5.2 and 10.9), read back in 31 and 100.
    const int all = (T + step * kRows - 1) / (step * kRows), some = kMostCtas / (2 * s->n_slots * s->n_kv);
    const int ctas = some < 1 ? 1 : some < all ? some : all;
    *grid = dim3(s->n_slots * ctas, 2 * s->n_kv);
    return ctas;
  }
  int log_t = 0;
  while (1 << log_t < T) ++log_t;
  const int slots = (step >> log_t) * kRows;
  *grid = dim3((s->n_slots + slots - 1) / slots, 2 * s->n_kv);
  return log_t;
}
}  // namespace

cudaError_t launch_cache_write_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                  const int32_t* n_new, int T, const uint16_t* k_new,
                                  int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                                  bool fp16, void* k, void* v, uint8_t* ws, cudaStream_t stream) {
  const CacheQ4Args a = args_of(s, meta, n_new, T, k, v, ws);
  dim3 grid;
  bool along;
  const int plan = plan_of(s, T, &along, &grid);
  auto go = [&](auto d, auto f) {
    constexpr int D = decltype(d)::value;
    constexpr bool F16 = decltype(f)::value;
    auto* kern = along ? cache_write_q4_kernel<F16, D, true> : cache_write_q4_kernel<F16, D, false>;
    return launch_pdl(kern, grid, dim3(kThr), 0, stream, a, plan, k_new, k_stride, v_new, v_stride);
  };
  if (s->D == 64) return fp16 ? go(Int<64>(), std::true_type()) : go(Int<64>(), std::false_type());
  return fp16 ? go(Int<128>(), std::true_type()) : go(Int<128>(), std::false_type());
}

cudaError_t launch_cache_read_q4(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                                 const int32_t* first, const int32_t* n, int T, const void* k,
                                 const void* v, void* k_out, int64_t k_stride, void* v_out,
                                 int64_t v_stride, int dtype, uint8_t* ws, cudaStream_t stream) {
  const CacheQ4Args a = args_of(s, meta, n, T, const_cast<void*>(k), const_cast<void*>(v), ws);
  dim3 grid;
  bool along;
  const int plan = plan_of(s, T, &along, &grid);
  auto go = [&](auto d, auto dt) {
    constexpr int D = decltype(d)::value, DT = decltype(dt)::value;
    auto* kern = along ? cache_read_q4_kernel<DT, D, true> : cache_read_q4_kernel<DT, D, false>;
    return launch_pdl(kern, grid, dim3(kThr), 0, stream, a, plan, first, k_out, k_stride, v_out, v_stride);
  };
  auto type = [&](auto d) {
    if (dtype == MOE_DTYPE_FP32) return go(d, Int<MOE_DTYPE_FP32>());
    return dtype == MOE_DTYPE_FP16 ? go(d, Int<MOE_DTYPE_FP16>()) : go(d, Int<MOE_DTYPE_BF16>());
  };
  return s->D == 64 ? type(Int<64>()) : type(Int<128>());
}

}  // namespace moe

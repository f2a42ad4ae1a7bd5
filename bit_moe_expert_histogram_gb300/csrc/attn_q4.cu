// Grouped-query decode attention of a batch of slots over a cache in 4 bits
// (the rows of cache_q4.cu).
//
// The definition is the batch attention's, with k_j and v_j the numbers that
// the codes stand for. With code c, scale s and bias b of position j and group
// g of a row's elements,
//   q . k_j = sum_g s_jg (sum_{e in g} q_e c_je) + b_jg (sum_{e in g} q_e),
//   o_e     = sum_j (p_j s_jg) c_je + p_j b_jg,
// so the matrix products run over the codes as they are, and a position's
// scales and biases touch one number a query and group instead of every
// element:
//  - A code is an operand without arithmetic. Four bits in the low bits of a
//    16-bit half are the fp16 number c 2^-24 (a subnormal one, which the tensor
//    core takes exactly), in bits 4 to 7 c 2^-20: one AND makes two operands,
//    and eight elements take five instructions.
//  - The queries are fp16 with a power of two of their row that brings its
//    largest element to 2^14 .. 2^15, and divided by 16 where they meet codes
//    of bits 4 to 7. What is lost is below 2^-34 of the row's largest. The power
//    stays within 2^-100 and 2^100, so that its inverse and the codes' 2^24 are an
//    fp32 number: elements are of at most 2^100, and what is lost is 2^-121 at most
//    where the row's largest is below 2^-86.
//  - The biases' part of the scores is one bf16 product a position tile (the
//    queries' group sums split into three bf16 parts, 24 bits).
//  - The softmax weights are rounded to fp16 once (half a step: 2^-11 of
//    themselves), times a scale a second time; sums are fp32. The values'
//    scales and biases are fp16 under a power of two of their group, the
//    largest so far, which loses nothing but what is 2^-24 below that. The
//    biases' part of O and the sum of the weights are one more product: its
//    rows are the four groups' biases and a row of ones.
//  - Scales and biases are brought into those forms by one lane a position, and
//    exchanged through shared memory by position pairs, as the products' lanes
//    want them. (Each lane that needs them converting them for itself, eight
//    times over, took twice the instructions in all: 45 us at 48 slots of 8K.)
//
// Both products have the cache as the tile's 16 rows and the queries as its
// columns: S^T = K Q^T over positions, O^T = V^T P^T over elements. Eight rows
// (a pair's single token with eight heads to a key head) then waste nothing,
// and codes, which are made for each step anyway, are the operand of four
// registers in a row (the queries there, padded to sixteen rows, cost two moves
// a product). P goes from S^T's result to an operand by a transposition of two
// registers for sixteen positions. With queries as columns, a lane has two of
// them, and their maxima, factors and sums need no exchange between lanes.
//
// Every warp works by itself: the pages of the (slot, head, row tile) pairs lie
// on one line, warp w takes units (a page of one head) [w per, (w + 1) per), and
// fetches them through a ring of its own, one bulk copy of keys and one of
// values a unit: rows of a head lie together in a page. A pair that lies within
// a warp's share goes straight to the output; what a share's ends cut is left in
// shared memory, joined by the CTA, and where the CTA's ends cut it, left in
// the workspace and joined by the last of its CTAs to arrive, in CTA order. (A few
// short pairs have a CTA each instead.)
//
// Measured on one GB300, 16 query heads on 2 of 128, in us a call:
//  - 48 slots of some 8.4K, 123 MB: 29.0, of which the pages take 20 (6 TB/s,
//    0.9 of a plain copy's rate), the lengths, tables and first pages 4, joining
//    4; 8 slots of some 112K, 250 MB: 49.7, 5.0 TB/s. HBM bounds both. Twelve
//    warps with half a page a unit took 33.7 and 56.0: a unit's fixed work (two
//    copies, a wait, scales exchanged, maxima compared) then weighs twice.
//  - The 16-bit call over as many positions: 64.6 us for the first, 123 for the
//    second, 253 for the next; at 33 slots of up to 5000 with D = 64, where starting
//    and joining are most of it, 15.1 against 17.1 here. Slots that share a long
//    prompt's pages each walk them by themselves: 256 slots of up to 4 tokens under
//    32K shared positions take 862 us, the 16-bit call with its shared part 147.
//  - 256 slots of up to 16K and 4 tokens, 513 MB read for two tiles of 16 rows:
//    200, bound by instruction latency: two warps a scheduler (queries, O and
//    scores of 16 rows take all registers) issue in 45 cycles of a hundred, the
//    tensor pipe is busy in 44. Tiles of 32 rows (spills) took 330, 12 warps
//    of half pages 296.
#include "attn_q4.cuh"

namespace moe {

namespace {
constexpr int kMostCtas = 256;
constexpr int kMostRows = 16;    // of a tile, the others have 8
constexpr int kMostChunks = 16;  // of 32 items of a pair's output

constexpr int kWarps = 8;   // of a CTA
constexpr int kQThr = kWarps * 32;
constexpr int kS = 2;       // stages of a warp's ring
// Units a warp may have where every pair gets a CTA of its own, which saves the
// joining across CTAs, some 2 us: 2 slots of 300 positions 8.4 -> 6.1 us, 60 of
// up to 400 10.0 -> 6.6, of up to 1000 10.1 -> 8.6; with four, 8 of up to 2000
// took 11.7 against 9.6.
constexpr int kAloneMost = 2;
// A unit of work is a page of one head.
template <int D, int NT>
struct Q4 {
  static constexpr int kRow = q4_units(D) * 2;  // bytes of a row
  static constexpr int kTile = kBlk * kRow;     // of a unit's keys (or values)
  static constexpr int kCh = D / 32;            // 16-byte pieces of codes
  // sixteen rows' queries lie in shared memory, [D / 32][NT][lane][4]
  static constexpr int kQBytes = NT == 1 ? 0 : D / 32 * NT * 512;
  // whether a warp's first piece does, too (there is no room beside everything else)
  static constexpr bool kPieceHere = NT == 1 || D == 64;
};
// A warp's scratch for a unit's scales and biases: keys' scales fp32
// [position][4]; then, by position pairs, values' scales and biases fp16
// [pair][2][4][2].
constexpr int kVal = kBlk * 16, kScratch = kBlk * 32;
// A piece or part: R[kR], l[kR], O[kR][D + 4] (the pad spreads the banks)
template <int D, int NT>
__host__ __device__ constexpr int piece_floats() { return 2 * 8 * NT + 8 * NT * (D + 4); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// from zero
__device__ __forceinline__ void mma_f16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f), "f"(0.0f), "f"(0.0f), "f"(0.0f));
}
// eight steps of bf16
__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ void mma_bf16_k8_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%7, %8, %9, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f), "f"(0.0f), "f"(0.0f), "f"(0.0f));
}
// 8 x 8 of 16 bits, rows to columns
__device__ __forceinline__ uint32_t transpose(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 v = lds128(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ float elem4(const float4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_f(float a, float b) {
  return pair2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// A weight is 2^(x - m + kLift): the reference m lags the running maximum by up
// to kSlack (else nearly every unit of a pair's first hundreds moves it: of
// eight rows one has a new maximum), which leaves fp16's 2^15 as the largest
// weight; what is 2^-22 of it is still a normal number, 2^-32 not 0
constexpr float kSlack = 7.0f, kLift = 8.0f;
// biased exponents that a group's power of two can have: from 2^-100 on
constexpr int kSigLeast = 27, kSigMost = 253;
constexpr uint32_t kLoNib = 0x000F000Fu, kHiNib = 0x00F000F0u;

// What a slot brings: its length, new tokens, row tiles with a token in them,
// and the units of such a tile's pair (at least one, a unit of nothing where it
// has none, so that each slot's rows get written; a tile without a token has
// one, too).
struct Q4Span {
  int len, n_new, used, units;
};
__device__ __forceinline__ Q4Span q4_span(const AttnQ4Args& a, int s) {
  Q4Span r;
  r.len = __ldg(a.lens + s);
  r.n_new = a.n_new ? __ldg(a.n_new + s) : a.T;
  const int most = a.max_blocks * kBlk;
  if (r.len < 0 || r.len > most || r.n_new < 0 || r.n_new > a.T) {
    set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, s);
    r.len = min(max(r.len, 0), most);
    r.n_new = min(max(r.n_new, 0), a.T);
  }
  const int n = (r.len + kBlk - 1) / kBlk;
  r.used = (r.n_new * a.group + (1 << a.row_shift) - 1) >> a.row_shift;
  r.units = n < 1 ? 1 : n;
  return r;
}
// on the line: what a slot's heads take each
__device__ __forceinline__ int head_units(const AttnQ4Args& a, const Q4Span& sp) {
  return sp.used * (sp.units + a.pair_cost) + (a.tiles - sp.used) * (1 + a.pair_cost);
}

// A place on the line: the pair (slot, head, row tile) and its first unit pb.
struct Place {
  int s, head, tile, pb;
  Q4Span sp;
  __device__ __forceinline__ int units() const { return tile < sp.used ? sp.units : 1; }
  __device__ __forceinline__ void next(const AttnQ4Args& a) {
    pb += units() + a.pair_cost;
    if (++tile < a.tiles) return;
    tile = 0;
    if (++head < a.n_kv) return;
    head = 0;
    if (++s < a.n_slots) sp = q4_span(a, s);
  }
};

// a warp's piece of a pair
struct PieceInfo {
  int pair, pb, units;  // pair: (slot * n_kv + head) * tiles + tile, -1: none
  int s, head, tile;
  const float* at;      // in shared memory, or the warp's place in the workspace
};

// V floats of a row, to 16 bits or as they are
template <int V>
struct Elems {
  float v[V];
};
template <int V>
__device__ __forceinline__ void store_elems(float* p, const Elems<V>& x) {
  if (V == 4)
    *reinterpret_cast<float4*>(p) = make_float4(x.v[0], x.v[1], x.v[V - 2], x.v[V - 1]);
  else
    *reinterpret_cast<float2*>(p) = make_float2(x.v[0], x.v[1]);
}
// v / l, 0 where l is (a row that sees nothing), even if what was summed for it
// is not finite
template <bool F16, int V>
__device__ __forceinline__ void store_out(uint16_t* p, const Elems<V>& x, float l) {
  const float inv = 1.0f / l;
  const uint32_t lo = l == 0.0f ? 0u : pack2<F16>(x.v[0] * inv, x.v[1] * inv);
  if (V == 4)
    *reinterpret_cast<uint2*>(p) =
        make_uint2(lo, l == 0.0f ? 0u : pack2<F16>(x.v[V - 2] * inv, x.v[V - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(p) = lo;
}
// four more parts
__device__ __forceinline__ void join4(Joined& j, const float (&m)[4], const float (&l)[4],
                                      const float4 (&v)[4]) {
  const float M = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), j.M);
  const float U = M == -INFINITY ? 0.0f : M;
  const float f = ex2(j.M - U);
  j.L *= f;
  j.o = make_float4(j.o.x * f, j.o.y * f, j.o.z * f, j.o.w * f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float w = ex2(m[k] - U);
    j.L = fmaf(l[k], w, j.L);
    j.o = make_float4(fmaf(v[k].x, w, j.o.x), fmaf(v[k].y, w, j.o.y), fmaf(v[k].z, w, j.o.z),
                      fmaf(v[k].w, w, j.o.w));
  }
  j.M = M;
}
}  // namespace

template <bool F16, int D, int NT>
__global__ void __launch_bounds__(kQThr, 1) attn_q4_kernel(const AttnQ4Args a) {
  using C = Q4<D, NT>;
  constexpr int kR = 8 * NT;
  constexpr int kKS = D / 16;  // steps of the score product, and O's element tiles
  constexpr int kPiece = piece_floats<D, NT>();
  extern __shared__ __align__(128) uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[kWarps][kS];
  __shared__ int s_scan[kWarps], s_most[kWarps];
  __shared__ Place s_start[kWarps];  // where the warps' shares start
  __shared__ PieceInfo s_piece[2 * kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, cq = lane & 3;
  const uint32_t sbase = smem_u32(sm_raw);
  const uint32_t ring = sbase + warp * (kS * 2 * C::kTile);
  const uint32_t scratch = sbase + kWarps * (kS * 2 * C::kTile) + warp * kScratch;
  constexpr int kMore = C::kQBytes + (C::kPieceHere ? kPiece * 4 : 0);
  const uint32_t queries = sbase + kWarps * (kS * 2 * C::kTile + kScratch) + warp * kMore;
  const uint32_t bars = smem_u32(&full[warp][0]);
  if (lane < kS) mbar_init(bars + 8u * lane, 1);
  if (tid < 2 * kWarps) s_piece[tid].pair = -1;
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();
  // ---- this warp's part of the line of units
  int total = 0, per;
  bool alone = false;  // every CTA has a pair of its own
  {
    const int chunk = (a.n_slots + kQThr - 1) / kQThr;
    const int s0 = min(tid * chunk, a.n_slots), s1 = min(s0 + chunk, a.n_slots);
    int sum = 0, most = 0;
    Q4Span sp{0, 0, 0, 0};
    for (int s = s0; s < s1; ++s) {
      sp = q4_span(a, s);
      sum += head_units(a, sp);
      most = max(most, sp.units);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    sum *= a.n_kv;
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (lane == 0) s_most[warp] = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += s_scan[w];
      total += s_scan[w];
      most = max(most, s_most[w]);
    }
    if (a.pairs <= (int)gridDim.x && most <= kAloneMost * kWarps) {
      // a few short pairs: a CTA each, so that nothing is joined across CTAs
      per = (most + kWarps - 1) / kWarps;
      total = a.pairs * per * kWarps;
      alone = true;
    } else {
      per = cut_up((unsigned)total, gridDim.x * kWarps);
      // the slots that the CTA's warps start in: each is in one thread's part
      const int c0 = min((int)blockIdx.x * kWarps * per, total), run0 = incl - sum;
      for (int w = 0; w < kWarps; ++w) {
        const int f = c0 + w * per;
        if (f < run0 || f >= incl) continue;
        s_start[w].s = s0;
        s_start[w].pb = run0;
        s_start[w].sp = sp;  // of the part's last slot, its only one but in large batches
      }
      __syncthreads();
    }
  }
  const int F0 = min((int)blockIdx.x * kWarps * per, total);  // the CTA's share
  const int F1 = min(F0 + kWarps * per, total);
  const int f0 = min(F0 + warp * per, total);
  int f1 = min(f0 + per, total);
  const int G = a.group, rows = a.T * G;
  // row / G for row < 64: the product is off by less than 1 / (2 G)
  const float per_g = 1.0f / (float)G;
  auto token = [&](int r) { return (int)(((float)r + 0.5f) * per_g); };
  const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(D)
  if (f0 < f1) {
    Place at;
    if (alone) {
      const int head = (int)blockIdx.x / a.tiles;
      at.s = head / a.n_kv;
      at.head = head - at.s * a.n_kv;
      at.tile = (int)blockIdx.x - head * a.tiles;
      at.pb = F0;
      at.sp = q4_span(a, at.s);
      f1 = min(f1, F0 + at.units());
    } else {
      at = s_start[warp];
      if (a.n_slots > kQThr) {
        for (at.sp = q4_span(a, at.s); at.s < a.n_slots - 1; at.sp = q4_span(a, ++at.s)) {
          const int n = head_units(a, at.sp) * a.n_kv;
          if (f0 < at.pb + n) break;
          at.pb += n;
        }
      }
      {
        const int all = head_units(a, at.sp), each = at.sp.units + a.pair_cost, rest = 1 + a.pair_cost;
        at.head = a.n_kv == 1 ? 0 : cut_up((unsigned)(f0 - at.pb) + 1u, all) - 1;
        at.pb += at.head * all;
        int in = f0 - at.pb;  // of the head's units
        at.tile = min(a.tiles == 1 ? 0 : cut_up((unsigned)in + 1u, each) - 1, at.sp.used);
        at.pb += at.tile * each;
        in -= at.tile * each;
        if (at.tile == at.sp.used) {
          const int more = cut_up((unsigned)in + 1u, rest) - 1;
          at.tile += more;
          at.pb += more * rest;
        }
      }
    }
    // ---- the loader: kS units ahead on the line, all lanes follow, lane 0 issues
    Place ld = at;
    int lu = f0 - at.pb;                        // the pair's next unit
    int le = min(f1 - at.pb, at.units());      // and how many of them are the warp's
    int lst = 0, ln = 0, base = -1, pages = -1; // pages: of blocks base + lane
    unsigned absent = 0;                        // bit per stage: nothing was fetched for it
    bool dead = false;                          // a wait ran out: nothing more is fetched
    const uint64_t pol = policy_evict_first();
    const int page_bytes = a.n_kv * C::kTile;
    auto load_next = [&] {
      if (dead) return;
      while (lu >= le) {
        if (ld.pb + ld.units() + a.pair_cost >= f1) return;
        ld.next(a);
        lu = 0;
        le = min(f1 - ld.pb, ld.units());
        base = -1;
      }
      if ((lu & ~31) != base) {
        base = lu & ~31;
        const int64_t at = (int64_t)ld.s * a.max_blocks + base + lane;
        pages = base + lane < a.max_blocks ? __ldg(a.table + at) : -1;
      }
      const int page = __shfl_sync(0xFFFFFFFFu, pages, lu & 31);
      const int n = min(kBlk, ld.sp.len - lu * kBlk);
      const bool none = ld.tile >= ld.sp.used || n <= 0;
      const bool bad = !none && (unsigned)page >= (unsigned)a.n_phys;
      absent = (absent & ~(1u << lst)) | (none || bad ? 1u << lst : 0u);
      if (lane == 0) {
        const uint32_t bar = bars + 8u * lst;
        if (absent >> lst & 1u) {
          if (bad) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, ld.s);
          mbar_arrive(bar);
        } else {
          const int64_t from = (int64_t)page * page_bytes + ld.head * C::kTile;
          const uint32_t sk = ring + lst * 2 * C::kTile, bytes = n * C::kRow;
          mbar_arrive_expect_tx(bar, 2 * bytes);
          bulk_load(sk, a.k + from, bytes, bar, pol);
          bulk_load(sk + C::kTile, a.v + from, bytes, bar, pol);
        }
      }
      ++lu;
      ++ln;
      lst = lst + 1 == kS ? 0 : lst + 1;
    };
    // a row's 16-bit elements as this lane's products want them, per piece c:
    // D = 128: 32 c + 8 cq .. + 7; D = 64: 32 c + 4 cq .. + 3 and 16 on
    uint32_t raw[NT][C::kCh][4];
    auto fetch_q = [&] {
      const int first = at.sp.len - at.sp.n_new;  // may be negative
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int r = at.tile * kR + gq + 8 * i, t = r < rows ? token(r) : a.T;
        const bool sees = t < at.sp.n_new && first + t >= 0;
        const uint16_t* q = a.q + ((int64_t)at.s * a.T + t) * a.q_stride + (at.head * G + r - t * G) * D;
#pragma unroll
        for (int c = 0; c < C::kCh; ++c) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (sees) {
            if (D == 128) {
              w = __ldg(reinterpret_cast<const uint4*>(q + 32 * c + 8 * cq));
            } else {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 32 * c + 4 * cq));
              const uint2 y = __ldg(reinterpret_cast<const uint2*>(q + 32 * c + 16 + 4 * cq));
              w = make_uint4(x.x, x.y, y.x, y.y);
            }
          }
          raw[i][c][0] = w.x, raw[i][c][1] = w.y, raw[i][c][2] = w.z, raw[i][c][3] = w.w;
        }
      }
    };
    if (f0 - at.pb < at.units()) fetch_q();
    for (int i = 0; i < kS; ++i) load_next();

    int f = f0, st = 0, done = 0;
    uint32_t parity = 0;
    while (f < f1) {
      const int units = at.units();
      if (f - at.pb >= units) {  // this warp starts in a pair's cost
        at.next(a);
        f = at.pb;
        if (f < f1) fetch_q();
        continue;
      }
      const int fe = min(f1, at.pb + units);
      const bool whole = f == at.pb && fe == at.pb + units;
      const int basep = at.sp.len - at.sp.n_new;  // may be negative
      // ---- the rows: queries as fp16, their scale, their groups' sums
      // per query column 2 cq + e of eight: its last visible position (-1: none),
      // and scores = cf * (products of codes) + biases' part
      auto lim_of = [&](int i, int e) {  // little used, and registers are scarce
        const int r = at.tile * kR + 8 * i + 2 * cq + e, t = r < rows ? token(r) : a.T;
        return t < at.sp.n_new ? max(basep + t, -1) : -1;
      };
      float cf[NT][2];
      uint32_t qa[kKS][2 * NT], qs[2 * NT];  // with sixteen rows qa lies in shared memory
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        // steps 2 c and 2 c + 1 of piece c take elements 0 4 1 5 and 2 6 3 7 of
        // the lane's eight, with D = 64 0 2 1 3 of each four
        float v[kKS][4];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < C::kCh; ++c) {
          float e[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[2 * k] = unpack_lo<F16>(raw[i][c][k]);
            e[2 * k + 1] = unpack_hi<F16>(raw[i][c][k]);
            top = fmaxf(top, fmaxf(fabsf(e[2 * k]), fabsf(e[2 * k + 1])));
          }
          if (D == 128) {
            v[2 * c][0] = e[0], v[2 * c][1] = e[4], v[2 * c][2] = e[1], v[2 * c][3] = e[5];
            v[2 * c + 1][0] = e[2], v[2 * c + 1][1] = e[6], v[2 * c + 1][2] = e[3], v[2 * c + 1][3] = e[7];
          } else {
            v[2 * c][0] = e[0], v[2 * c][1] = e[2], v[2 * c][2] = e[1], v[2 * c][3] = e[3];
            v[2 * c + 1][0] = e[4], v[2 * c + 1][1] = e[6], v[2 * c + 1][2] = e[5], v[2 * c + 1][3] = e[7];
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^e with top 2^e in [2^14, 2^15)
        const int ex = min(max(127 + 14 - (int)(__float_as_uint(top) >> 23), -100), 100);
        const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
        const float back = sl2 * __uint_as_float((uint32_t)(127 + 24 - ex) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cf[i][e] = __shfl_sync(0xFFFFFFFFu, back, 8 * cq + 4 * e);
        }
        float sum[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) sum[g] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          sum[D == 128 ? ks >> 1 : ks] += (v[ks][0] + v[ks][1]) + (v[ks][2] + v[ks][3]);
          qa[ks][i] = pack2<true>(v[ks][0] * up, v[ks][1] * up);
          qa[ks][NT + i] = pack2<true>(v[ks][2] * up * 0.0625f, v[ks][3] * up * 0.0625f);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 1);
          sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 2);
          sum[g] *= sl2;
        }
        // columns 2 cq, 2 cq + 1 of the biases' product: groups 0 1 | 2 3 of
        // the first parts, of the second; then of the third, and nothing
        const uint32_t h01 = pack2<false>(sum[0], sum[1]), h23 = pack2<false>(sum[2], sum[3]);
        const float r0 = sum[0] - bf_lo(h01), r1 = sum[1] - bf_hi(h01);
        const float r2 = sum[2] - bf_lo(h23), r3 = sum[3] - bf_hi(h23);
        const uint32_t m01 = pack2<false>(r0, r1), m23 = pack2<false>(r2, r3);
        const uint32_t l01 = pack2<false>(r0 - bf_lo(m01), r1 - bf_hi(m01));
        const uint32_t l23 = pack2<false>(r2 - bf_lo(m23), r3 - bf_hi(m23));
        qs[i] = cq == 0 ? h01 : cq == 1 ? h23 : cq == 2 ? m01 : m23;
        qs[NT + i] = cq == 0 ? l01 : cq == 1 ? l23 : 0u;
      }
      // o: O^T, element tiles by rows; sb: rows 0 .. 3 the biases' part by
      // groups, row 4 the sum of the weights
      if (C::kQBytes > 0) {
#pragma unroll
        for (int c = 0; c < C::kCh; ++c)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            sts128(queries + (c * NT + i) * 512 + lane * 16, qa[2 * c][i], qa[2 * c][NT + i],
                   qa[2 * c + 1][i], qa[2 * c + 1][NT + i]);
      }
      float m[NT][2], sb[NT][4], o[kKS][NT][4];
      int sg[4];  // biased exponents of the groups' powers of two
#pragma unroll
      for (int g = 0; g < 4; ++g) sg[g] = kSigLeast;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        sb[i][0] = sb[i][1] = sb[i][2] = sb[i][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < kKS; ++j) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
      }
      for (; f < fe; ++f) {
        if (!dead) {
          volatile int never = 0;
          const bool ok = mbar_wait(bars + 8u * st, parity, &never);
          dead = !__all_sync(0xFFFFFFFFu, ok);
          if (dead) {
            if (lane == 0) set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, at.s);
          } else {
            ++done;
          }
        }
        if (!dead && !(absent >> st & 1u)) {
          const uint32_t sk = ring + st * 2 * C::kTile, sv = sk + C::kTile;
          const int pos0 = (f - at.pb) * kBlk, n_here = at.sp.len - pos0;
          // ---- keys' scales, a position a lane; rows past the slot's end hold
          // anything and are masked, values' count as nothing
          constexpr int kOf = kBlk / 32;  // positions of a lane
          uint4 wv[kOf];
#pragma unroll
          for (int v = 0; v < kOf; ++v) {
            const int pos = lane + 32 * v;
            const uint32_t at = D / 2 + pos * C::kRow;
            const uint2 wk = lds64(sk + at);
            wv[v] = lds128(sv + at);
            sts128(scratch + pos * 16, wk.x << 16, wk.x & 0xFFFF0000u, wk.y << 16, wk.y & 0xFFFF0000u);
          }
          __syncwarp();
          // ---- scores, in powers of two, of positions 16 h + gq and 8 on, and of
          // two queries a number pair
          uint64_t x[kBlk / 16][2][NT];
#pragma unroll
          for (int v = 0; v < kBlk / 32; ++v) {
            uint64_t t[2][NT][2];
#pragma unroll
            for (int c = 0; c < C::kCh; c += 2) {
              if (C::kQBytes > 0) {
#pragma unroll
                for (int k = c; k < c + 2; ++k)
#pragma unroll
                  for (int i = 0; i < NT; ++i) {
                    const uint4 q = lds128(queries + (k * NT + i) * 512 + lane * 16);
                    qa[2 * k][i] = q.x, qa[2 * k][NT + i] = q.y;
                    qa[2 * k + 1][i] = q.z, qa[2 * k + 1][NT + i] = q.w;
                  }
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t at = scratch + (16 * (2 * v + h) + gq) * 16;
                const float4 s[2] = {lds_f4(at), lds_f4(at + 128)};
                uint32_t kc[4];  // words of pieces c and c + 1 of positions gq, gq + 8
                ldsm4(sk + (16 * (2 * v + h) + (lane & 15)) * C::kRow + (c + (lane >> 4)) * 16, kc);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float acc[NT][4];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int ks = 2 * (c + k) + e, g = D == 128 ? ks >> 1 : ks;
                    const uint32_t w0 = e ? kc[2 * k] >> 8 : kc[2 * k];
                    const uint32_t w1 = e ? kc[2 * k + 1] >> 8 : kc[2 * k + 1];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                      if (D == 64 || e == 0)
                        mma_f16_0(acc[i], w0 & kLoNib, w1 & kLoNib, w0 & kHiNib, w1 & kHiNib, qa[ks][i],
                                  qa[ks][NT + i]);
                      else
                        mma_f16(acc[i], w0 & kLoNib, w1 & kLoNib, w0 & kHiNib, w1 & kHiNib, qa[ks][i],
                                qa[ks][NT + i]);
                      if (D == 64 || e == 1)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                          const float sy = elem4(s[y], g);
                          const uint64_t a2 = pair_f(acc[i][2 * y], acc[i][2 * y + 1]), s2 = pair_f(sy, sy);
                          t[h][i][y] = g == 0 ? mul2(s2, a2) : fma2(s2, a2, t[h][i][y]);
                        }
                    }
                  }
                }
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t r0 = sk + (16 * (2 * v + h) + gq) * C::kRow + D / 2 + 8 + 4 * (cq & 1);
              const uint32_t bw0 = lds32(r0), bw1 = lds32(r0 + 8 * C::kRow);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                float xb[4];
                mma_bf16_k8_0(xb, bw0, bw1, qs[i]);
                mma_bf16_k8(xb, bw0, bw1, qs[NT + i]);
                const uint64_t f2 = pair_f(cf[i][0], cf[i][1]);
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  x[2 * v + h][y][i] = fma2(t[h][i][y], f2,
                                            pair_f(xb[2 * y], xb[2 * y + 1]));
              }
            }
          }
          // every query that is in use sees positions up to basep
          if (pos0 + kBlk - 1 > basep) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const int lim0 = lim_of(i, 0), lim1 = lim_of(i, 1);
#pragma unroll
              for (int h = 0; h < kBlk / 8; ++h) {
                float x0, x1;
                unpair2(x[h >> 1][h & 1][i], x0, x1);
                if (pos0 + 8 * h + gq > lim0) x0 = -INFINITY;
                if (pos0 + 8 * h + gq > lim1) x1 = -INFINITY;
                x[h >> 1][h & 1][i] = pair_f(x0, x1);
              }
            }
          }
          // ---- values' scales and biases, while the products run
          {
            float s4[kOf][4], b4[kOf][4], big[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < kOf; ++v) {
              uint4 w = wv[v];
              if (lane + 32 * v >= n_here) w = make_uint4(0u, 0u, 0u, 0u);
              s4[v][0] = 16.0f * bf_lo(w.x), s4[v][1] = 16.0f * bf_hi(w.x);
              s4[v][2] = 16.0f * bf_lo(w.y), s4[v][3] = 16.0f * bf_hi(w.y);
              b4[v][0] = bf_lo(w.z), b4[v][1] = bf_hi(w.z), b4[v][2] = bf_lo(w.w), b4[v][3] = bf_hi(w.w);
#pragma unroll
              for (int g = 0; g < 4; ++g) big[g] = fmaxf(big[g], fmaxf(s4[v][g], fabsf(b4[v][g])));
            }
            bool grown = false;
            int was[4];
            float inv[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              // positive numbers order as whole numbers
              const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big[g]));
              was[g] = sg[g];
              sg[g] = min(max(sg[g], (int)(top >> 23) + 1), kSigMost);
              grown |= sg[g] != was[g];
              inv[g] = __uint_as_float((uint32_t)(254 - sg[g]) << 23);
            }
            if (grown) {  // the same for all lanes
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const float cut = sg[g] == was[g] ? 1.0f : ex2((float)(was[g] - sg[g]));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
#pragma unroll
                  for (int j = g * (kKS / 4); j < (g + 1) * (kKS / 4); ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][i][e] *= cut;
                  if (gq == g) {
                    sb[i][0] *= cut;
                    sb[i][1] *= cut;
                  }
                }
              }
            }
            // this lane's position as the low or high half of its pair: even
            // lanes take groups 0 and 1 of both, odd lanes 2 and 3
            const bool odd = lane & 1;
#pragma unroll
            for (int v = 0; v < kOf; ++v) {
              const uint32_t sa = pack2<true>(s4[v][0] * inv[0], s4[v][1] * inv[1]);
              const uint32_t sc = pack2<true>(s4[v][2] * inv[2], s4[v][3] * inv[3]);
              const uint32_t ba = pack2<true>(b4[v][0] * inv[0], b4[v][1] * inv[1]);
              const uint32_t bc = pack2<true>(b4[v][2] * inv[2], b4[v][3] * inv[3]);
              const uint32_t xs = __shfl_xor_sync(0xFFFFFFFFu, odd ? sa : sc, 1);
              const uint32_t xb = __shfl_xor_sync(0xFFFFFFFFu, odd ? ba : bc, 1);
              const uint32_t ls = odd ? xs : sa, hs = odd ? sc : xs;
              const uint32_t lb = odd ? xb : ba, hb = odd ? bc : xb;
              const uint32_t tv = scratch + kVal + ((lane >> 1) + 16 * v) * 32 + odd * 8;
              sts64(tv, __byte_perm(ls, hs, 0x5410), __byte_perm(ls, hs, 0x7632));
              sts64(tv + 16, __byte_perm(lb, hb, 0x5410), __byte_perm(lb, hb, 0x7632));
            }
          }
          // ---- the reference m follows the running maximum when that is kSlack
          // ahead of it; what was summed up to then follows
          float mx[NT][2];
          bool moved = false;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mx[i][0] = mx[i][1] = -INFINITY;
#pragma unroll
            for (int h = 0; h < kBlk / 8; ++h) {
              float x0, x1;
              unpair2(x[h >> 1][h & 1][i], x0, x1);
              mx[i][0] = fmaxf(mx[i][0], x0);
              mx[i][1] = fmaxf(mx[i][1], x1);
            }
            moved |= mx[i][0] > m[i][0] + kSlack || mx[i][1] > m[i][1] + kSlack;
          }
          if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float now = mx[i][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, d));
                now = fmaxf(now, m[i][e]);
                // nothing seen so far: everything stays 0 (no inf - inf)
                const float cut = ex2(m[i][e] - (now == -INFINITY ? 0.0f : now));
                m[i][e] = now;
                sb[i][e] *= cut;
#pragma unroll
                for (int j = 0; j < kKS; ++j) {
                  o[j][i][e] *= cut;
                  o[j][i][2 + e] *= cut;
                }
              }
          }
          uint64_t up[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
            up[i] = pair_f(kLift - (m[i][0] == -INFINITY ? 0.0f : m[i][0]),
                           kLift - (m[i][1] == -INFINITY ? 0.0f : m[i][1]));
          __syncwarp();
          // ---- weights and the second product, sixteen positions a step
#pragma unroll
          for (int kp = 0; kp < kBlk / 16; ++kp) {
            uint32_t p[NT][2];  // weights as an operand: two positions of query gq a register
            uint32_t s4[2][4];  // the values' scales of the same positions, by groups
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 w = lds128(scratch + kVal + (8 * kp + 4 * h + cq) * 32);
              s4[h][0] = w.x, s4[h][1] = w.y, s4[h][2] = w.z, s4[h][3] = w.w;
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                float x0, x1;
                unpair2(add2(x[kp][h][i], up[i]), x0, x1);
                p[i][h] = transpose(pack2<true>(ex2(x0), ex2(x1)));
              }
            }
            // rows 0 .. 3: the groups' biases, 4: ones; the others' results go nowhere
            const uint32_t ab = scratch + kVal + (8 * kp + cq) * 32 + 16 + (gq & 3) * 4;
            const uint32_t a0 = gq < 4 ? lds32(ab) : 0x3C003C00u, a2 = gq < 4 ? lds32(ab + 128) : 0x3C003C00u;
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma_f16(sb[i], a0, a0, a2, a2, p[i][0], p[i][1]);
#pragma unroll
            for (int c = 0; c < C::kCh; c += 2) {
              uint32_t vc[4];  // pieces c and c + 1 of positions 0..7, 8..15
              ldsm4_t(sv + (16 * kp + (lane & 15)) * C::kRow + (c + (lane >> 4)) * 16, vc);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t ps[NT][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = 2 * (c + k) + e, g = D == 128 ? j >> 1 : j;
                  const uint32_t x0 = e ? vc[2 * k] >> 8 : vc[2 * k];
                  const uint32_t x1 = e ? vc[2 * k + 1] >> 8 : vc[2 * k + 1];
#pragma unroll
                  for (int i = 0; i < NT; ++i) {
                    if (D == 64 || e == 0) {
                      ps[i][0] = mul_h2(p[i][0], s4[0][g]);
                      ps[i][1] = mul_h2(p[i][1], s4[1][g]);
                    }
                    mma_f16(o[j][i], x0 & kLoNib, x0 & kHiNib, x1 & kLoNib, x1 & kHiNib, ps[i][0], ps[i][1]);
                  }
                }
              }
            }
          }
          // the stage is the loader's again
          fence_proxy_async_smem();
          __syncwarp();
        }
        load_next();
        st = st + 1 == kS ? 0 : st + 1;
        parity ^= st == 0;
      }
      // ---- the pair's end
      // a cut pair's piece: the warp's last goes to the ring, which nothing is on
      // its way into any more; a first one before other pairs to a place of its own
      const int which = at.pb < f0 ? 0 : 1;
      const bool more = fe == at.pb + units && fe + a.pair_cost < f1;
      float sig[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) sig[g] = __uint_as_float((uint32_t)sg[g] << 23);
      float* pf = reinterpret_cast<float*>(sm_raw + (ring - sbase));
      if (more)
        pf = C::kPieceHere ? reinterpret_cast<float*>(sm_raw + (queries + C::kQBytes - sbase))
                           : a.pieces + ((int64_t)blockIdx.x * kWarps + warp) * kPiece;
      if (!whole && lane == 0)
        s_piece[2 * warp + which] = PieceInfo{(at.s * a.n_kv + at.head) * a.tiles + at.tile, at.pb, units,
                                              at.s, at.head, at.tile, pf};
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // row 2 cq + e of the eight: its sum and biases' part are with lanes
          // 16 + cq and 4 g + cq
          const int r = 8 * i + 2 * cq + e;
          const float sum = __shfl_sync(0xFFFFFFFFu, sb[i][e], 16 + cq);
          // rows that see nothing weigh nothing, whatever was summed for them
          const bool used = lim_of(i, e) >= 0;
          const float lr = used ? sum : 0.0f;
          if (!whole && gq == 0) {
            pf[r] = used ? m[i][e] : -INFINITY;
            pf[kR + r] = lr;
          }
          float b[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) b[g] = __shfl_sync(0xFFFFFFFFu, sb[i][e], 4 * g + cq) * sig[g];
          const int R = at.tile * kR + r, t = token(R);
          uint16_t* out = a.o + (((int64_t)at.s * a.T + t) * a.n_q + at.head * G + R - t * G) * D;
#pragma unroll
          for (int c = 0; c < C::kCh; ++c) {
            // D = 128: elements 32 c + 4 gq + {0, 1, 2, 3}; D = 64: 32 c + 2 gq +
            // {0, 1} and 16 on
            const int g0 = D == 128 ? c : 2 * c, g1 = D == 128 ? c : 2 * c + 1;
            float y[4] = {fmaf(o[2 * c][i][e] * 0x1p20f, sig[g0], b[g0]),
                          fmaf(o[2 * c][i][2 + e] * 0x1p16f, sig[g0], b[g0]),
                          fmaf(o[2 * c + 1][i][e] * 0x1p20f, sig[g1], b[g1]),
                          fmaf(o[2 * c + 1][i][2 + e] * 0x1p16f, sig[g1], b[g1])};
            const Elems<2> y0{y[0], y[1]}, y1{y[2], y[3]};
            const Elems<4> y4{y[0], y[1], y[2], y[3]};
            if (whole) {
              if (R < rows) {
                if (D == 128) {
                  store_out<F16>(out + 32 * c + 4 * gq, y4, lr);
                } else {
                  store_out<F16>(out + 32 * c + 2 * gq, y0, lr);
                  store_out<F16>(out + 32 * c + 16 + 2 * gq, y1, lr);
                }
              }
            } else {
              float* to = pf + 2 * kR + r * (D + 4);
              if (D == 128) {
                store_elems(to + 32 * c + 4 * gq, y4);
              } else {
                store_elems(to + 32 * c + 2 * gq, y0);
                store_elems(to + 32 * c + 16 + 2 * gq, y1);
              }
            }
          }
        }
      if (f < f1) {
        at.next(a);
        f = at.pb;
        if (f < f1) fetch_q();
      }
    }
    // after a wait that ran out, what is in flight lands before the CTA goes
    if (dead && lane == 0) {
      volatile int never = 0;
      for (; done < ln; ++done) mbar_wait(bars + 8u * (done % kS), (uint32_t)(done / kS) & 1u, &never);
    }
  }
  __syncthreads();
  // ---- the CTA's pieces, pair by pair in the line's order, a thread for four
  // elements of a row, a warp for 32 such items. What a pair that lies in the CTA
  // has goes to the output, what one that does not has to the workspace, place 0
  // of the CTA's two where it starts before the CTA. Then a warp counts itself
  // in at the cut pairs, for its items alone, and the last to arrive joins them.
  constexpr int kItems = kR * D / 4, kPasses = (kItems + kQThr - 1) / kQThr;
  const int pair_of = lane < 2 * kWarps ? s_piece[lane].pair : -1;
  const unsigned pieces = __ballot_sync(0xFFFFFFFFu, pair_of >= 0);
  const int share = kWarps * per;
  auto store = [&](const PieceInfo& p, int r, int d, const float4& y, float l) {
    const int R = p.tile * kR + r, t = token(R);
    uint16_t* to = a.o + (((int64_t)p.s * a.T + t) * a.n_q + p.head * G + R - t * G) * D + 4 * d;
    if (R < rows) store4<F16>(to, y, l);
  };
  bool cut = false;
  for (unsigned rest = pieces; rest;) {
    const int i = __ffs(rest) - 1;
    const PieceInfo p = s_piece[i];
    const unsigned mine = __ballot_sync(0xFFFFFFFFu, pair_of == p.pair);
    rest &= ~mine;
    const bool own = p.pb >= F0 && p.pb + p.units <= F1;
    cut |= !own;
#pragma unroll 1
    for (int item = tid; item < kItems; item += kQThr) {
      const int r = item / (D / 4), d = item % (D / 4);
      Joined j{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      unsigned left = mine;
#pragma unroll 1
      while (left) {  // four pieces at once
        float m[4], l[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* q = s_piece[left ? __ffs(left) - 1 : i].at;
          m[k] = left ? q[r] : -INFINITY;
          l[k] = q[kR + r];
          v[k] = *reinterpret_cast<const float4*>(q + 2 * kR + r * (D + 4) + 4 * d);
          left &= left - 1;
        }
        join4(j, m, l, v);
      }
      if (own) {
        store(p, r, d, j.o, j.L);
      } else {
        float* part = a.part + (int64_t)(2 * blockIdx.x + (p.pb < F0 ? 0 : 1)) * kPiece;
        *reinterpret_cast<float4*>(part + 2 * kR + r * (D + 4) + 4 * d) = j.o;
        if (d == 0) {
          part[r] = j.M;
          part[kR + r] = j.L;
        }
      }
    }
  }
  if (!cut) return;
  __syncwarp();
  // lane c + 2 k: the warp's k-th items of the pair that is cut at the CTA's
  // start (c = 0, the first piece's) or at its end (the last piece's)
  int c0 = 0, n = 0;
  bool last = false;
  if (lane < 2 * kPasses && warp * 32 + (lane >> 1) * kQThr < kItems) {
    const PieceInfo& p = s_piece[lane & 1 ? 31 - __clz(pieces) : __ffs(pieces) - 1];
    if (lane & 1 ? p.pb >= F0 && p.pb + p.units > F1 : p.pb < F0) {
      c0 = cut_up((unsigned)p.pb + 1u, share) - 1;
      n = cut_up((unsigned)(p.pb + p.units), share) - c0;
      // the counters are those of the pair's first CTA, whose end cuts this pair
      // and no other
      unsigned* cnt = a.count + c0 * kMostChunks + warp + (lane >> 1) * kWarps;
      __threadfence();
      last = atomicAdd(cnt, 1u) == (unsigned)(n - 1);
      if (last) *cnt = 0u;  // ready for the next call
      __threadfence();
    }
  }
  // single lanes counted and fenced, the whole warp reads the other CTAs' parts:
  // ordered by the barrier, as a vote orders no memory
  __syncwarp();
  for (unsigned todo = __ballot_sync(0xFFFFFFFFu, last); todo; todo &= todo - 1) {
    const int k = __ffs(todo) - 1, parts = __shfl_sync(0xFFFFFFFFu, n, k);
    const PieceInfo p = s_piece[k & 1 ? 31 - __clz(pieces) : __ffs(pieces) - 1];
    const int item = tid + (k >> 1) * kQThr, r = item / (D / 4), d = item % (D / 4);
    const float* from = a.part + (int64_t)(2 * __shfl_sync(0xFFFFFFFFu, c0, k)) * kPiece + r;
    Joined j{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    // part c of the pair: the first CTA's is its place 1, the others' place 0
    join_parts<6>(j, parts, [&](int c) {
      return PartRef{from + (int64_t)(2 * c + (c == 0)) * kPiece, kR, 2 * kR + r * (D + 3) + 4 * d};
    });
    store(p, r, d, j.o, j.L);
  }
}

namespace {
// Rows of a tile, as a power of two. Tiles of sixteen take every page of a pair
// half as often, but a unit of theirs takes 2.7 us from start to end, one of eight
// 1.7 (they spill, too, where D is 128): eight are better until the work is so much
// that there is always something to do. Units a warp has at most, as far as the
// shape says, against us with sixteen and eight rows:
//  D = 128: 0.1 12.0 8.4, 2 14.3 10.0, 14.7 33.4 27.5, 20 40.5 35.1, 30 43.2 42.3,
//   40 56.5 51.7, 54 73.8 70.6, 62 68.2 73.8, 107 133 141, 214 206 240
//  D = 64: 0.8 10.2 8.6, 2.4 10.7 10.5 and 12.7 10.7, 4.9 12.9 14.0 and 15.1 14.0,
//   10 16.9 17.8, 39 33.7 41.8, 47 49.5 53.9
// The shape's units are the table's width, not the lengths: 8 slots of 2800 with 4
// tokens take 14.0 us with a table of 44 blocks and 17.4 with one of 2048, 64 of 500
// 16.6 and 18.2 (64 of 6000 with 2 tokens 45.4 and 39.5).
int row_shift(const moe_attn_batch_shape_t* s, int ctas) {
  const int rows = s->T * (s->n_q / s->n_kv), warps = ctas * kWarps;
  if (rows <= 8) return 3;
  const int64_t units = (int64_t)s->n_slots * s->n_kv * ((rows + 15) / 16) * s->max_blocks;
  return units <= (int64_t)warps * (s->D == 128 ? 48 : 4) ? 3 : 4;
}
// the start and end of a pair against a unit: 31.6 us without, 29.5 with one and
// 31.7 with two for 48 slots of 8K, 27, 23.4 and 23.2 for 33 ragged ones
constexpr int kPairCost = 1;
constexpr size_t part_floats(int D) { return 2 * kMostRows + kMostRows * (D + 4); }
constexpr size_t kCountAt = 256, kPartAt = kCountAt + kMostCtas * kMostChunks * 4;

template <bool F16, int D, int NT>
cudaError_t launch(const AttnQ4Args& a, int ctas, cudaStream_t stream) {
  using C = Q4<D, NT>;
  const size_t smem = (size_t)kWarps * (kS * 2 * C::kTile + kScratch + C::kQBytes +
                                        (C::kPieceHere ? piece_floats<D, NT>() * 4 : 0));
  const cudaError_t e = cudaFuncSetAttribute(attn_q4_kernel<F16, D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q4_kernel<F16, D, NT>, dim3(ctas), dim3(kQThr), smem, stream, a);
}
template <bool F16, int D>
cudaError_t launch_rows(const AttnQ4Args& a, int ctas, cudaStream_t stream) {
  return a.row_shift == 3 ? launch<F16, D, 1>(a, ctas, stream) : launch<F16, D, 2>(a, ctas, stream);
}
}  // namespace

bool attn_q4_supported(const moe_attn_batch_shape_t* s) {
  if (!attn_batch_supported(s) || s->prefix_blocks != 0) return false;
  // the line of units is counted in 32 bits
  const int tiles = (s->T * (s->n_q / s->n_kv) + kMostRows - 1) / kMostRows;
  return (int64_t)s->n_slots * s->n_kv * tiles * (s->max_blocks + kPairCost) < (1 << 30);
}

// status, the CTAs' counters (one for 32 items), their two places for parts, the
// warps' places for pieces. The counters are all that one call leaves to the
// next (zeros), and their place and extent are the same for every shape.
size_t attn_q4_ws_bytes(const moe_attn_batch_shape_t* s) {
  return kPartAt + (2 + kWarps) * (size_t)kMostCtas * part_floats(s->D) * 4;
}

cudaError_t launch_attn_q4(const moe_attn_batch_shape_t* s, AttnQ4Args a, uint8_t* ws, int nsm,
                           cudaStream_t stream) {
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  a.count = reinterpret_cast<unsigned*>(ws + kCountAt);
  a.part = reinterpret_cast<float*>(ws + kPartAt);
  a.pieces = a.part + 2 * (size_t)kMostCtas * part_floats(s->D);
  a.n_slots = s->n_slots;
  a.T = s->T;
  a.n_q = s->n_q;
  a.n_kv = s->n_kv;
  a.group = s->n_q / s->n_kv;
  a.max_blocks = s->max_blocks;
  a.pair_cost = kPairCost;
  const int ctas = nsm < kMostCtas ? nsm : kMostCtas;
  a.row_shift = row_shift(s, ctas);
  a.tiles = (s->T * a.group + (1 << a.row_shift) - 1) >> a.row_shift;
  a.pairs = a.n_slots * a.n_kv * a.tiles;
  if (s->dtype == MOE_DTYPE_FP16)
    return s->D == 64 ? launch_rows<true, 64>(a, ctas, stream) : launch_rows<true, 128>(a, ctas, stream);
  return s->D == 64 ? launch_rows<false, 64>(a, ctas, stream) : launch_rows<false, 128>(a, ctas, stream);
}

}  // namespace moe

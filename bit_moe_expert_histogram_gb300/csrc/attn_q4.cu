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
//    of bits 4 to 7. What is lost is below 2^-34 of the row's largest.
//  - The biases' part of the scores is one bf16 product a position tile (the
//    queries' group sums split into three bf16 parts, 24 bits).
//  - p s is rounded to fp16 once (2^-11 of itself: half a step), after a power
//    of two that keeps it below 2^14 whatever the values' size: the rows'
//    largest scale so far, joined to the softmax's running maximum. p b and the
//    sum of p are fp32 throughout.
//
// Both products have their free dimension where it wastes least: S = Q K^T has
// the query rows as the tile's 16, and its result is, without any exchange,
// the second operand of O^T = V^T P^T, whose 16 are elements of V.
//
// Every warp works by itself: the (slot, head, row tile) pairs' units of 32
// positions lie on one line, warp w takes units [w per, (w + 1) per), and
// fetches them through a ring of its own (one bulk copy of keys, one of values
// a unit: rows of a head lie together in a page). A pair that lies within a
// warp's share goes straight to the output; what a share's ends cut is left in
// shared memory, joined by the CTA, and where the CTA's ends cut it, left in
// the workspace and joined by the last of its CTAs to arrive, in CTA order.
#include "attn_q4.cuh"

namespace moe {

namespace {
constexpr int kUnit = 32;   // positions of a unit
constexpr int kWarps = 8;
constexpr int kQThr = kWarps * 32;
constexpr int kMostCtas = 256;

template <int D>
struct Q4 {
  static constexpr int kRow = q4_units(D) * 2;      // bytes of a row
  static constexpr int kTile = kUnit * kRow;        // of a unit's keys (or values)
  static constexpr int kCh = D / 32;                // 16-byte pieces of codes
};
// stages of a warp's ring
template <int D, int NT>
__host__ __device__ constexpr int ring_stages() { return D == 64 ? 6 : NT == 1 ? 4 : 3; }
// A piece: rows R[kR], l[kR], O[kR][D + 4] (the pad spreads the banks)
template <int D, int NT>
__host__ __device__ constexpr int piece_floats() { return 2 * 8 * NT + 8 * NT * (D + 4); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

constexpr uint32_t kLoNib = 0x000F000Fu, kHiNib = 0x00F000F0u;

// What a slot brings: its length, new tokens and units (at least one, a unit
// of nothing where it has none, so that each slot's rows get written).
struct Q4Span {
  int len, n_new, units;
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
  const int n = (r.len + kUnit - 1) / kUnit;
  r.units = r.n_new == 0 || n < 1 ? 1 : n;
  return r;
}

// A place on the line: the pair that unit f belongs to, its first unit pb.
struct Place {
  int s, h, pb;  // h: head * row tiles + row tile
  Q4Span sp;
  __device__ __forceinline__ void next(const AttnQ4Args& a) {
    pb += sp.units + a.pair_cost;
    if (++h == a.n_kv * a.tiles) {
      h = 0;
      if (++s < a.n_slots) sp = q4_span(a, s);
    }
  }
};

// a warp's piece of a pair
struct PieceInfo {
  int pair, pb, units;  // pair: slot * n_kv * tiles + h, -1: none
  uint32_t at;          // shared-memory address
};
}  // namespace

template <bool F16, int D, int NT>
__global__ void __launch_bounds__(kQThr, 1) attn_q4_kernel(const AttnQ4Args a) {
  using C = Q4<D>;
  constexpr int kS = ring_stages<D, NT>(), kR = 8 * NT;
  constexpr int kKS = D / 16;  // steps of the score product, and O's element tiles
  constexpr int kNP = kUnit / 8;
  constexpr int kPiece = piece_floats<D, NT>();
  extern __shared__ __align__(128) uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[kWarps][kS];
  __shared__ int s_scan[kWarps];
  __shared__ int s_start[kWarps], s_off[kWarps];
  __shared__ PieceInfo s_piece[2 * kWarps];
  __shared__ int s_last[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, cq = lane & 3;
  const uint32_t sbase = smem_u32(sm_raw);
  const uint32_t ring = sbase + warp * (kS * 2 * C::kTile);
  const uint32_t extra = sbase + kWarps * (kS * 2 * C::kTile) + warp * (kPiece * 4);
  const uint32_t bars = smem_u32(&full[warp][0]);
  if (lane < kS) mbar_init(bars + 8u * lane, 1);
  if (tid < 2 * kWarps) s_piece[tid].pair = -1;
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();
  // ---- this warp's part of the line of units
  const int ht = a.n_kv * a.tiles;  // pairs of a slot
  int total = 0;
  {
    const int chunk = (a.n_slots + kQThr - 1) / kQThr;
    const int s0 = min(tid * chunk, a.n_slots), s1 = min(s0 + chunk, a.n_slots);
    int sum = 0;
    for (int s = s0; s < s1; ++s) sum += q4_span(a, s).units + a.pair_cost;
    sum *= ht;
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += s_scan[w];
      total += s_scan[w];
    }
    const unsigned warps = gridDim.x * kWarps;
    const int per = (int)(((unsigned)total + warps - 1) / warps);
    const int c0 = min((int)blockIdx.x * kWarps * per, total);
    // the slots that the CTA's warps start in: each is one thread's to find
    const int run0 = incl - sum;
    for (int w = 0; w < kWarps; ++w) {
      const int f = c0 + w * per;
      if (f < run0 || f >= incl) continue;
      int s = s0, run = run0;
      for (; s < s1 - 1; ++s) {
        const int n = (q4_span(a, s).units + a.pair_cost) * ht;
        if (f < run + n) break;
        run += n;
      }
      s_start[w] = s;
      s_off[w] = f - run;
    }
    __syncthreads();
  }
  const unsigned warps = gridDim.x * kWarps;
  const int per = (int)(((unsigned)total + warps - 1) / warps);
  const int F0 = min((int)blockIdx.x * kWarps * per, total);  // the CTA's share
  const int F1 = min(F0 + kWarps * per, total);
  const int f0 = min(F0 + warp * per, total), f1 = min(f0 + per, total);
  const int G = a.n_q / a.n_kv, rows = a.T * G;
  const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(D)
  if (f0 < f1) {
    Place at;
    at.s = s_start[warp];
    at.sp = q4_span(a, at.s);
    at.h = s_off[warp] / (at.sp.units + a.pair_cost);
    at.pb = f0 - (s_off[warp] - at.h * (at.sp.units + a.pair_cost));
    // ---- the loader's own place on the line, kS units ahead
    Place ld = at;
    int lf = f0, ln = 0, base = -1, pages = -1;
    unsigned absent = 0, phase = 0, pending = 0;  // bit per stage; pending: a copy not waited for
    bool dead = false;                            // a wait ran out: nothing more is fetched
    const uint64_t pol = policy_evict_first();
    auto load_next = [&] {
      while (lf < f1 && lf - ld.pb >= ld.sp.units) {
        ld.next(a);
        lf = ld.pb;
        base = -1;
      }
      if (lf >= f1) return;
      const int u = lf - ld.pb, block = u >> 1, st = ln % kS;
      if ((block & ~31) != base) {
        base = block & ~31;
        pages = base + lane < a.max_blocks ? __ldg(a.table + (int64_t)ld.s * a.max_blocks + base + lane) : -1;
      }
      const int page = __shfl_sync(0xFFFFFFFFu, pages, block & 31);
      const int n = ld.sp.n_new == 0 ? 0 : min(kUnit, ld.sp.len - u * kUnit);
      const bool bad = n > 0 && (page < 0 || page >= a.n_phys);
      if (bad && lane == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, ld.s);
      if (n <= 0 || bad || dead) {
        absent |= 1u << st;
      } else {
        absent &= ~(1u << st);
        pending |= 1u << st;
        if (lane == 0) {
          const int64_t row = ((int64_t)page * a.n_kv + ld.h / a.tiles) * kBlk + (u & 1) * kUnit;
          const uint32_t sk = ring + st * 2 * C::kTile, bytes = n * C::kRow;
          mbar_arrive_expect_tx(bars + 8u * st, 2 * bytes);
          bulk_load(sk, a.k + row * C::kRow, bytes, bars + 8u * st, pol);
          bulk_load(sk + C::kTile, a.v + row * C::kRow, bytes, bars + 8u * st, pol);
        }
      }
      ++lf;
      ++ln;
    };
    for (int i = 0; i < kS; ++i) load_next();

    int f = f0, it = 0;
    while (f < f1) {
      if (f - at.pb >= at.sp.units) {
        at.next(a);
        f = at.pb;
        continue;
      }
      const int fe = min(f1, at.pb + at.sp.units);
      const bool whole = f == at.pb && fe == at.pb + at.sp.units;
      const int head = at.h / a.tiles, mt = at.h - head * a.tiles;
      const int basep = at.sp.len - at.sp.n_new;  // may be negative
      // ---- the rows: queries as fp16, their scale, their groups' sums
      int lim[NT];        // last position that row gq + 8 i sees, -1: none
      float cq2[NT];      // scores = cq2 * (products of codes) + biases' part
      uint32_t qa[kKS][2 * NT], qs[2 * NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int r = mt * 16 + gq + 8 * i, t = r < rows ? r / G : a.T;
        lim[i] = t < at.sp.n_new ? max(basep + t, -1) : -1;
        float v[kKS][4];
        // step 2 c and 2 c + 1 of piece c take this lane's elements
        // D = 128: 32 c + 8 cq + {0, 4, 1, 5} and {2, 6, 3, 7}
        // D = 64: 32 c + 4 cq + {0, 2, 1, 3}, and those of the second group
        const uint16_t* q = a.q + ((int64_t)at.s * a.T + t) * a.q_stride + (head * G + r - t * G) * D;
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < C::kCh; ++c) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (lim[i] >= 0) {
            if (D == 128) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + 32 * c + 8 * cq));
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            } else {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 32 * c + 4 * cq));
              const uint2 y = __ldg(reinterpret_cast<const uint2*>(q + 32 * c + 16 + 4 * cq));
              w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
            }
          }
          float e[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[2 * k] = unpack_lo<F16>(w[k]);
            e[2 * k + 1] = unpack_hi<F16>(w[k]);
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
        cq2[i] = sl2 * __uint_as_float((uint32_t)(127 + 24 - ex) << 23);
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
      float m[NT], ref[NT], l[NT], ob[NT][4], o[kKS][NT][4];
      float ls = -80.0f;  // log2 of a power of two that no scale of the values is above
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        m[i] = ref[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int g = 0; g < 4; ++g) ob[i][g] = 0.0f;
#pragma unroll
        for (int j = 0; j < kKS; ++j) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
      }
      for (; f < fe; ++f, ++it) {
        const int st = it % kS;
        if (!(absent >> st & 1u) && !dead) {
          volatile int never = 0;
          const bool ok = mbar_wait(bars + 8u * st, phase >> st & 1u, &never);
          dead = !__all_sync(0xFFFFFFFFu, ok);
          if (dead && lane == 0) set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, at.s);
        }
        if (!(absent >> st & 1u) && !dead) {
          phase ^= 1u << st;
          pending &= ~(1u << st);
          const uint32_t sk = ring + st * 2 * C::kTile, sv = sk + C::kTile;
          const int pos0 = (f - at.pb) * kUnit, n_here = at.sp.len - pos0;
          // ---- scores, in powers of two
          float x[kNP][2 * NT];
          uint32_t kc[4];  // codes of a tile's rows; D = 64: of two tiles'
#pragma unroll
          for (int n = 0; n < kNP; ++n) {
            const uint32_t bw = lds32(sk + (8 * n + gq) * C::kRow + D / 2 + 8 + 4 * (cq & 1));
            float sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_bf16(sb, qs[0], NT > 1 ? qs[1] : 0u, qs[NT], NT > 1 ? qs[NT + 1] : 0u, bw, bw);
            if (D == 128)
              ldsm4(sk + (8 * n + (lane & 7)) * C::kRow + (lane >> 3) * 16, kc);
            else if (n % 2 == 0)
              ldsm4(sk + (8 * n + (lane & 7) + (lane >> 4) * 8) * C::kRow + (lane >> 3 & 1) * 16, kc);
            const uint2 s0 = lds64(sk + (8 * n + 2 * cq) * C::kRow + D / 2);
            const uint2 s1 = lds64(sk + (8 * n + 2 * cq + 1) * C::kRow + D / 2);
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float acc[4];
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
              const int g = D == 128 ? ks >> 1 : ks;
              const uint32_t word = D == 128 ? kc[ks >> 1] : kc[(n & 1) * 2 + (ks >> 1)];
              const uint32_t w = ks & 1 ? word >> 8 : word;
              if (D == 64 || (ks & 1) == 0) acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
              mma_f16(acc, qa[ks][0], NT > 1 ? qa[ks][1] : 0u, qa[ks][NT], NT > 1 ? qa[ks][NT + 1] : 0u,
                      w & kLoNib, w & kHiNib);
              if (D == 64 || (ks & 1)) {
                const uint32_t u0 = g < 2 ? s0.x : s0.y, u1 = g < 2 ? s1.x : s1.y;
                const float f0s = g & 1 ? bf_hi(u0) : bf_lo(u0), f1s = g & 1 ? bf_hi(u1) : bf_lo(u1);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                  t[2 * i] = fmaf(f0s, acc[2 * i], t[2 * i]);
                  t[2 * i + 1] = fmaf(f1s, acc[2 * i + 1], t[2 * i + 1]);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              x[n][2 * i] = fmaf(t[2 * i], cq2[i], sb[2 * i]);
              x[n][2 * i + 1] = fmaf(t[2 * i + 1], cq2[i], sb[2 * i + 1]);
            }
          }
          // every row that is in use sees positions up to basep
          if (pos0 + kUnit - 1 > basep) {
#pragma unroll
            for (int n = 0; n < kNP; ++n)
#pragma unroll
              for (int i = 0; i < 2 * NT; ++i)
                if (pos0 + 8 * n + 2 * cq + (i & 1) > lim[i >> 1]) x[n][i] = -INFINITY;
          } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (lim[i] < 0) {
#pragma unroll
                for (int n = 0; n < kNP; ++n) x[n][2 * i] = x[n][2 * i + 1] = -INFINITY;
              }
          }
          // ---- the values' largest scale: positive bf16 numbers order as whole numbers
          {
            uint32_t big = 0u;
            if (lane < n_here) {
              const uint2 w = lds64(sv + lane * C::kRow + D / 2);
              big = max(max(w.x >> 16, w.x & 0xFFFFu), max(w.y >> 16, w.y & 0xFFFFu));
            }
            big = __reduce_max_sync(0xFFFFFFFFu, big);
            ls = fmaxf(ls, (float)((int)(big >> 7 & 255u) - 126));
          }
          // ---- running maximum, and what was summed up to it
          bool moved = false;
          float cut[NT], u[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < kNP; ++n) mx = fmaxf(mx, fmaxf(x[n][2 * i], x[n][2 * i + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            m[i] = fmaxf(m[i], mx);
            // nothing seen so far: everything stays 0 (no inf - inf)
            const float now = m[i] == -INFINITY ? -INFINITY : m[i] + ls;
            u[i] = now == -INFINITY ? 0.0f : now;
            cut[i] = ex2(ref[i] - u[i]);
            moved |= now != ref[i];
            ref[i] = now;
          }
          if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              l[i] *= cut[i];
#pragma unroll
              for (int g = 0; g < 4; ++g) ob[i][g] *= cut[i];
              // O has the rows as columns: 2 cq and 2 cq + 1
              const float c0 = __shfl_sync(0xFFFFFFFFu, cut[i], 8 * cq);
              const float c1 = __shfl_sync(0xFFFFFFFFu, cut[i], 8 * cq + 4);
#pragma unroll
              for (int j = 0; j < kKS; ++j) {
                o[j][i][0] *= c0;
                o[j][i][1] *= c1;
                o[j][i][2] *= c0;
                o[j][i][3] *= c1;
              }
            }
          }
          // ---- weights and the second product, sixteen positions a step
#pragma unroll
          for (int kp = 0; kp < kUnit / 16; ++kp) {
            uint32_t pw[NT][4][2];  // p s as operands: [row half][group][position half]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = 2 * kp + h;
              uint4 w0 = lds128(sv + (8 * n + 2 * cq) * C::kRow + D / 2);
              uint4 w1 = lds128(sv + (8 * n + 2 * cq + 1) * C::kRow + D / 2);
              if (n_here < kUnit) {  // rows past the slot's end hold anything
                if (8 * n + 2 * cq >= n_here) w0 = make_uint4(0u, 0u, 0u, 0u);
                if (8 * n + 2 * cq + 1 >= n_here) w1 = make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const float p0 = ex2(x[n][2 * i] + (14.0f - u[i]));
                const float p1 = ex2(x[n][2 * i + 1] + (14.0f - u[i]));
                l[i] += p0 + p1;
                pw[i][0][h] = pack2<true>(p0 * bf_lo(w0.x), p1 * bf_lo(w1.x));
                pw[i][1][h] = pack2<true>(p0 * bf_hi(w0.x), p1 * bf_hi(w1.x));
                pw[i][2][h] = pack2<true>(p0 * bf_lo(w0.y), p1 * bf_lo(w1.y));
                pw[i][3][h] = pack2<true>(p0 * bf_hi(w0.y), p1 * bf_hi(w1.y));
                ob[i][0] = fmaf(p1, bf_lo(w1.z), fmaf(p0, bf_lo(w0.z), ob[i][0]));
                ob[i][1] = fmaf(p1, bf_hi(w1.z), fmaf(p0, bf_hi(w0.z), ob[i][1]));
                ob[i][2] = fmaf(p1, bf_lo(w1.w), fmaf(p0, bf_lo(w0.w), ob[i][2]));
                ob[i][3] = fmaf(p1, bf_hi(w1.w), fmaf(p0, bf_hi(w0.w), ob[i][3]));
              }
            }
#pragma unroll
            for (int c = 0; c < C::kCh; c += 2) {
              uint32_t vc[4];  // pieces c and c + 1 of positions 0..7, 8..15
              ldsm4_t(sv + (16 * kp + (lane & 15)) * C::kRow + (c + (lane >> 4)) * 16, vc);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = 2 * (c + k) + e, g = D == 128 ? j >> 1 : j;
                  const uint32_t x0 = e ? vc[2 * k] >> 8 : vc[2 * k];
                  const uint32_t x1 = e ? vc[2 * k + 1] >> 8 : vc[2 * k + 1];
#pragma unroll
                  for (int i = 0; i < NT; ++i)
                    mma_f16(o[j][i], x0 & kLoNib, x0 & kHiNib, x1 & kLoNib, x1 & kHiNib,
                            pw[i][g][0], pw[i][g][1]);
                }
            }
          }
          // the stage is the loader's again
          fence_proxy_async_smem();
          __syncwarp();
        }
        load_next();
      }
      // ---- the pair's end: sums over the lanes that share a row
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          ob[i][g] += __shfl_xor_sync(0xFFFFFFFFu, ob[i][g], 1);
          ob[i][g] += __shfl_xor_sync(0xFFFFFFFFu, ob[i][g], 2);
        }
      }
      // a cut pair's piece: the first goes to a place of its own, as units
      // after it are on their way into the ring; the last goes to the ring
      const int which = at.pb < f0 ? 0 : 1;
      const uint32_t piece = which == 0 ? extra : ring;
      if (!whole && lane == 0)
        s_piece[2 * warp + which] = PieceInfo{at.s * ht + at.h, at.pb, at.sp.units, piece};
      float* pf = reinterpret_cast<float*>(sm_raw + (piece - sbase));
      if (!whole && cq == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          pf[gq + 8 * i] = ref[i];
          pf[kR + gq + 8 * i] = l[i];
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // row 2 cq + e of the eight: its sums are with lane 4 (2 cq + e)
          const int src = 4 * (2 * cq + e), r = 8 * i + 2 * cq + e;
          const float lr = __shfl_sync(0xFFFFFFFFu, l[i], src);
          float b[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) b[g] = __shfl_sync(0xFFFFFFFFu, ob[i][g], src);
          const int R = mt * 16 + r, t = R / G;
          const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
          uint16_t* out = a.o + (((int64_t)at.s * a.T + t) * a.n_q + head * G + R - t * G) * D;
#pragma unroll
          for (int c = 0; c < C::kCh; ++c) {
            // D = 128: elements 32 c + 4 gq + {0, 1, 2, 3}; D = 64: 32 c + 2 gq +
            // {0, 1} and 16 on
            const int g0 = D == 128 ? c : 2 * c, g1 = D == 128 ? c : 2 * c + 1;
            float y[4] = {fmaf(o[2 * c][i][e], 0x1p24f, b[g0]), fmaf(o[2 * c][i][2 + e], 0x1p20f, b[g0]),
                          fmaf(o[2 * c + 1][i][e], 0x1p24f, b[g1]), fmaf(o[2 * c + 1][i][2 + e], 0x1p20f, b[g1])};
            if (whole) {
              if (R < rows) {
                // a row that sees nothing is 0, whatever was summed for it
                const uint32_t lo = lr == 0.0f ? 0u : pack2<F16>(y[0] * inv, y[1] * inv);
                const uint32_t hi = lr == 0.0f ? 0u : pack2<F16>(y[2] * inv, y[3] * inv);
                if (D == 128) {
                  *reinterpret_cast<uint2*>(out + 32 * c + 4 * gq) = make_uint2(lo, hi);
                } else {
                  *reinterpret_cast<uint32_t*>(out + 32 * c + 2 * gq) = lo;
                  *reinterpret_cast<uint32_t*>(out + 32 * c + 16 + 2 * gq) = hi;
                }
              }
            } else {
              float* to = pf + 2 * kR + r * (D + 4);
              if (D == 128) {
                *reinterpret_cast<float4*>(to + 32 * c + 4 * gq) = make_float4(y[0], y[1], y[2], y[3]);
              } else {
                *reinterpret_cast<float2*>(to + 32 * c + 2 * gq) = make_float2(y[0], y[1]);
                *reinterpret_cast<float2*>(to + 32 * c + 16 + 2 * gq) = make_float2(y[2], y[3]);
              }
            }
          }
        }
      if (f < f1) {
        at.next(a);
        f = at.pb;
      }
    }
    // after a wait that ran out, what is in flight lands before the CTA goes
    if (dead && lane == 0) {
      volatile int never = 0;
      for (int st = 0; st < kS; ++st)
        if (pending >> st & 1u) mbar_wait(bars + 8u * st, phase >> st & 1u, &never);
    }
  }
  __syncthreads();
  // ---- the CTA's pieces, pair by pair in the line's order; what its ends cut
  // goes to the workspace: place 0 for a pair that starts before, 1 for one
  // that starts here
  constexpr int kItems = kR * D / 4;
  int cut_pb[2] = {0, 0}, cut_units[2] = {0, 0}, cut_pair[2] = {-1, -1};
  for (int i = 0; i < 2 * kWarps;) {
    const PieceInfo p = s_piece[i];
    int n = i + 1;  // pieces i .. n - 1, those of no warp left out
    if (p.pair >= 0) {
      while (n < 2 * kWarps && (s_piece[n].pair < 0 || s_piece[n].pair == p.pair)) ++n;
      const bool own = p.pb >= F0 && p.pb + p.units <= F1;
      const int place = p.pb < F0 ? 0 : 1;
      if (!own) {
        cut_pb[place] = p.pb;
        cut_units[place] = p.units;
        cut_pair[place] = p.pair;
      }
      const int s = p.pair / ht, h = p.pair - s * ht, head = h / a.tiles, mt = h - head * a.tiles;
      float* part = a.part + (int64_t)(2 * blockIdx.x + place) * kPiece;
      for (int item = tid; item < kItems; item += kQThr) {
        const int r = item / (D / 4), d = item % (D / 4);
        float M = -INFINITY;
        for (int k = i; k < n; ++k)
          if (s_piece[k].pair >= 0)
            M = fmaxf(M, reinterpret_cast<const float*>(sm_raw + (s_piece[k].at - sbase))[r]);
        const float U = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = i; k < n; ++k) {
          if (s_piece[k].pair < 0) continue;
          const float* q = reinterpret_cast<const float*>(sm_raw + (s_piece[k].at - sbase));
          const float w = ex2(q[r] - U);
          const float4 v = *reinterpret_cast<const float4*>(q + 2 * kR + r * (D + 4) + 4 * d);
          L = fmaf(q[kR + r], w, L);
          y.x = fmaf(v.x, w, y.x);
          y.y = fmaf(v.y, w, y.y);
          y.z = fmaf(v.z, w, y.z);
          y.w = fmaf(v.w, w, y.w);
        }
        const int R = mt * 16 + r, t = R / G;
        if (own) {
          if (R < rows)
            store4<F16>(a.o + (((int64_t)s * a.T + t) * a.n_q + head * G + R - t * G) * D + 4 * d, y, L);
        } else {
          *reinterpret_cast<float4*>(part + 2 * kR + r * (D + 4) + 4 * d) = y;
          if (d == 0) {
            part[r] = M;
            part[kR + r] = L;
          }
        }
      }
    }
    i = n;
  }
  if (cut_pair[0] < 0 && cut_pair[1] < 0) return;
  __threadfence();
  __syncthreads();
  const int share = kWarps * per;
  if (tid < 2 && cut_pair[tid] >= 0) {
    // the pair's CTAs; the counter is the one of the first, whose end cuts this
    // pair and no other
    const int c0 = cut_pb[tid] / share, c1 = (cut_pb[tid] + cut_units[tid] - 1) / share;
    unsigned* cnt = a.count + c0;
    s_last[tid] = atomicAdd(cnt, 1u) == (unsigned)(c1 - c0);
    if (s_last[tid]) *cnt = 0u;  // ready for the next call
    __threadfence();
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (cut_pair[k] < 0 || !s_last[k]) continue;
    const int c0 = cut_pb[k] / share, c1 = (cut_pb[k] + cut_units[k] - 1) / share;
    const int s = cut_pair[k] / ht, h = cut_pair[k] - s * ht, head = h / a.tiles, mt = h - head * a.tiles;
    for (int item = tid; item < kItems; item += kQThr) {
      const int r = item / (D / 4), d = item % (D / 4);
      Joined j{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      join_parts<8>(j, c1 - c0 + 1, [&](int c) {
        const float* p = a.part + (int64_t)(2 * (c0 + c) + (c == 0)) * kPiece;
        return PartRef{p + r, kR, 2 * kR + r * (D + 4) + 4 * d - r};
      });
      const int R = mt * 16 + r, t = R / G;
      if (R < rows)
        store4<F16>(a.o + (((int64_t)s * a.T + t) * a.n_q + head * G + R - t * G) * D + 4 * d, j.o, j.L);
    }
  }
}

namespace {
int row_tiles(const moe_attn_batch_shape_t* s) { return (s->T * (s->n_q / s->n_kv) + 15) / 16; }
constexpr int kPairCost = 1;
constexpr size_t kCountAt = 256, kPartAt = kCountAt + kMostCtas * 4;

template <bool F16, int D, int NT>
cudaError_t launch(const AttnQ4Args& a, int ctas, cudaStream_t stream) {
  const size_t smem = (size_t)kWarps * (ring_stages<D, NT>() * 2 * Q4<D>::kTile + piece_floats<D, NT>() * 4);
  const cudaError_t e = cudaFuncSetAttribute(attn_q4_kernel<F16, D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q4_kernel<F16, D, NT>, dim3(ctas), dim3(kQThr), smem, stream, a);
}
}  // namespace

bool attn_q4_supported(const moe_attn_batch_shape_t* s) {
  if (!attn_batch_supported(s) || s->prefix_blocks != 0) return false;
  // the line of units is counted in 32 bits
  return (int64_t)s->n_slots * s->n_kv * row_tiles(s) * (2 * s->max_blocks + kPairCost) < (1 << 30);
}

// status, the CTAs' counters, their two places for parts. The counters are
// all that one call leaves to the next (zeros), and nothing lies elsewhere for
// another shape.
size_t attn_q4_ws_bytes(const moe_attn_batch_shape_t* s) {
  const size_t piece = 2 * 16 + 16 * (s->D + 4);
  return kPartAt + 2 * (size_t)kMostCtas * piece * 4;
}

cudaError_t launch_attn_q4(const moe_attn_batch_shape_t* s, AttnQ4Args a, uint8_t* ws, int nsm,
                           cudaStream_t stream) {
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  a.count = reinterpret_cast<unsigned*>(ws + kCountAt);
  a.part = reinterpret_cast<float*>(ws + kPartAt);
  a.n_slots = s->n_slots;
  a.T = s->T;
  a.n_q = s->n_q;
  a.n_kv = s->n_kv;
  a.max_blocks = s->max_blocks;
  a.tiles = row_tiles(s);
  a.pair_cost = kPairCost;
  const int ctas = nsm < kMostCtas ? nsm : kMostCtas;
  const bool one = s->T * (s->n_q / s->n_kv) <= 8;
  if (s->dtype == MOE_DTYPE_FP16) {
    if (s->D == 64) return one ? launch<true, 64, 1>(a, ctas, stream) : launch<true, 64, 2>(a, ctas, stream);
    return one ? launch<true, 128, 1>(a, ctas, stream) : launch<true, 128, 2>(a, ctas, stream);
  }
  if (s->D == 64) return one ? launch<false, 64, 1>(a, ctas, stream) : launch<false, 64, 2>(a, ctas, stream);
  return one ? launch<false, 128, 1>(a, ctas, stream) : launch<false, 128, 2>(a, ctas, stream);
}

}  // namespace moe

// Grouped-query decode attention for a batch of slots over one page pool,
// the leading pages of all slots being the same ones (a shared prompt).
//
// Row t of slot s sits at position p = lens[s] - n_new[s] + t:
//   o[s][t][h] = softmax_j(q . k_j / sqrt(D)) v_j over j <= p,
// head h reading key/value head h / (n_q / n_kv). A row with nothing to see
// (t >= n_new, an idle slot) is 0.
//
// Softmax of a row split over key ranges: each range keeps its reference
// maximum m, l = sum 2^(x - m) and O = sum 2^(x - m) v (x = log2(e) q.k /
// sqrt(D)); ranges join as O = sum O_i 2^(m_i - M) with M = max m_i, the same
// for l, in a fixed order.
//
// attn_own_kernel: each slot's own positions. The (slot, head) pairs' blocks
// lie on one line, and CTA c takes blocks [c per, (c + 1) per) of it whatever
// slots they belong to, so uneven lengths leave no CTA idle. (A pair counts
// pair_cost units more than its blocks: its start and end cost about that many
// blocks' time, so a CTA of many short slots gets fewer blocks. Measured with
// 1, 2, 3, 4, 6: 28.0, 25.4, 25.4, 25.4, 25.8 us for 64 slots of 8 + 5 pages
// and 8 heads, D = 128, 16 rows a pair; 26.8, 24.8, 23.7, 22.8, 22.9 for 64 of
// 16 + 5 and 2 heads, 32 rows; 12.5, 12.0, 11.5, 11.5, 11.2 for 16 of 16 + 5
// and 8 heads, D = 64.) The T * n_q / n_kv <= 64 query
// rows of a pair are the M rows of mma.sync tiles (16 rows; 1, 2 or 4 tiles),
// so each key and value is read once per slot: HBM bounds it, and the tensor
// core's own instructions, whose M is 128, would mostly multiply nothing. A
// warp of its own keeps a TMA ring of blocks full (64 rows x 64 elements per
// box, 128-byte swizzle) that runs on across pairs, knowing the next slot's
// pages before it gets there; the four others only meet at a pair's ends,
// where their results meet in the stage of its last block while the next
// pair's queries, span and blocks are on their way. A pair of one block takes
// 2.6 us (D = 128, 5 rows), no one wait of which is more than a seventh.
//  - where a pair has few parts, one inside a CTA goes straight to the output,
//    and one cut by a CTA border leaves (m, l, O) in the workspace and the
//    last of its CTAs to arrive joins them in CTA order;
//  - where it has many, or a shared part (attn_prefix.cu), every pair leaves
//    (m, l, O), and attn_join_kernel joins them all, a thread for four
//    elements of the output: few threads wait long for what many threads
//    fetch at once (one slot of 32768 positions: 28 us against 12.4).
// 33 slots of up to 5000 positions, D = 64, fp16, 65 MB: 14.5 us in a graph,
// 4.5 TB/s, 0.66 of a plain copy's rate (the next call's reads partly from L2;
// 17 us where the pages lie badly).
#include "attn_batch.cuh"

namespace moe {

namespace {
constexpr int kOThr = 128;         // the four warps that compute
constexpr int kOAll = kOThr + 32;  // and the one that loads

template <bool F16>
__device__ __forceinline__ void mma16816t(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// byte offset of 16-byte chunk ch of row p in a [64][D] tile stored as D/64
// TMA boxes of 64 rows x 128 bytes with the 128-byte swizzle
__device__ __forceinline__ uint32_t swz64(int p, int ch) {
  return (uint32_t)((ch >> 3) * (kBlk * 128) + p * 128 + (((ch & 7) ^ (p & 7)) << 4));
}
// v / l to four 16-bit elements, 0 where l is (a row that sees nothing), even
// if what was summed for it is not finite; a NaN sum stays one
template <bool F16>
__device__ __forceinline__ void store4(uint16_t* to, const float4& v, float l) {
  const float inv = 1.0f / l;
  *reinterpret_cast<uint2*>(to) =
      l == 0.0f ? make_uint2(0u, 0u)
                : make_uint2(pack2<F16>(v.x * inv, v.y * inv), pack2<F16>(v.z * inv, v.w * inv));
}
}  // namespace

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
// where row r, columns 4 d .. of a part of ld rows lie: m[ld], l[ld], O[d][ld][4]
__device__ __forceinline__ PartRef part_ref(const float* part, int ld, int r, int d) {
  return PartRef{part + r, ld, 2 * ld + 4 * (d * ld + r) - r};
}
template <int D>
struct OwnRing {
  static constexpr int kTile = kBlk * D * 2;       // bytes of a block's keys (or values)
  static constexpr int kStages = D == 64 ? 4 : 3;  // 64 and 96 KB
};
// Two places for a pair's queries, so that the next pair's come while one is
// computed (they took a seventh of a short pair); with more rows there is no
// room for them beside the ring.
template <int D, int MT>
constexpr int kQTile = MT * 16 * D * 2 <= 4096 ? MT * 16 * D * 2 : 0;
// CTAs an SM: two, or three where registers and stages allow (19.1 us instead
// of 20.2 for 33 slots of up to 5000 positions)
__host__ __device__ constexpr int own_ctas(int D, int MT) { return D == 64 && MT == 1 ? 3 : 2; }

template <bool F16, int D, int MT>
__global__ void __launch_bounds__(kOAll, own_ctas(D, MT))
    attn_own_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const AttnBatchArgs a) {
  constexpr int kTile = OwnRing<D>::kTile, kStages = OwnRing<D>::kStages;
  constexpr int kNS = 4 / MT;       // warps that share a row tile, each a slice of the block
  constexpr int kPos = kBlk / kNS;  // positions of a slice
  constexpr int kNT = kPos / 8;     // score n-tiles of a warp
  constexpr int kKS = D / 16, kDT = D / 8;
  constexpr int kR = MT * 16;       // rows of the tiles
  constexpr int kQB = kQTile<D, MT>;
  constexpr int kQPass = kQB / 16 / kOThr;     // 16-byte pieces of queries a thread fetches
  constexpr int kCols = kR * D / 4 / kOThr;    // float4 of the pair's output a thread has
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ int s_bad[kStages];
  __shared__ int s_abort, s_start, s_off, s_ctas, s_last;
  __shared__ int s_scan[kOAll / 32], s_tok[kOAll / 32];
  __shared__ float s_m[4][16], s_l[4][16];  // per warp: its rows' maximum and sum
  __shared__ float s_M[kR], s_L[kR];        // the segment's
  const uint32_t sbase = (smem_u32(sm_raw) + 1023u) & ~1023u;
  uint8_t* sm = sm_raw + (sbase - smem_u32(sm_raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t fb = smem_u32(&full[0]), eb = smem_u32(&empty[0]);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(fb + 8u * i, 1);
      mbar_init(eb + 8u * i, 4);
    }
    s_abort = 0;
    s_start = 0;
    s_off = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // With the shared part in the kernel before, everything that comes from
  // earlier work was complete before that kernel let this one start (it
  // triggers after its own wait), and nothing here reads its parts.
  const bool shared = a.px_steps > 0;
  if (!shared) {
    pdl_wait();
    pdl_trigger();
  }
  // ---- this CTA's part of the line of blocks
  const bool plan = shared && !a.px_fixed;
  int total = 0, ctas = (int)gridDim.x, per, f0;
  {
    const int chunk = (a.n_slots + kOAll - 1) / kOAll;
    const int s0 = min(tid * chunk, a.n_slots), s1 = min(s0 + chunk, a.n_slots);
    int sum = 0, tok = 0;
    for (int s = s0; s < s1; ++s) {
      const SlotSpan sp = slot_span(a, s);
      sum += sp.blocks + a.pair_cost;
      tok += sp.n_new;
    }
    sum *= a.n_kv;
    if (plan) tok = __reduce_add_sync(0xFFFFFFFFu, tok);
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) {
      s_scan[warp] = incl;
      s_tok[warp] = tok;
    }
    __syncthreads();
    for (int w = 0; w < kOAll / 32; ++w) {
      if (w < warp) incl += s_scan[w];
      total += s_scan[w];
    }
    if (plan) {  // as many CTAs as there is room for beside the shared part
      if (warp == kOAll / 32 - 1) {
        tok = __reduce_add_sync(0xFFFFFFFFu, lane < kOAll / 32 ? s_tok[lane] : 0);
        const int room = (a.sms - best_line(a, tok, total).grid) * own_ctas(D, MT);
        if (lane == 0) s_ctas = max(min(room, ctas), 1);
      }
      __syncthreads();
      ctas = s_ctas;
    }
    per = (int)((unsigned)(total + ctas - 1) / (unsigned)ctas);
    f0 = (int)blockIdx.x < ctas ? min((int)blockIdx.x * per, total) : total;
    int run = incl - sum;
    if (f0 >= run && f0 < incl) {  // one thread's slots hold the first block
      int s = s0;
      for (; s < s1 - 1; ++s) {
        const int n = (slot_span(a, s).blocks + a.pair_cost) * a.n_kv;
        if (f0 < run + n) break;
        run += n;
      }
      s_start = s;
      s_off = f0 - run;
    }
    __syncthreads();
  }
  const int f1 = min(f0 + per, total);
  int s = s_start;
  SlotSpan sp = slot_span(a, s);
  int g = s_off / (sp.blocks + a.pair_cost);
  // where the pair starts on the line; its blocks first, then its cost
  int pb = f0 - (s_off - g * (sp.blocks + a.pair_cost));
  volatile int* abort = &s_abort;

  if (warp == 4) {
    // ---- the loader: all lanes follow the line, lane 0 issues
    const uint64_t pol = policy_evict_first();  // own pages are read once
    // lane l: the pages of the slot's first 32 own blocks and of the next
    // slot's, with that slot's span: a short pair does not wait for them
    auto page_of = [&](int slot, int j) {
      const int jb = a.first + j + lane;
      if (slot >= a.n_slots || jb >= a.max_blocks) return -1;
      return jb < a.prefix_blocks ? __ldg(a.prefix + jb)
                                  : __ldg(a.table + (int64_t)slot * a.max_blocks + jb);
    };
    int first32 = page_of(s, 0), next32 = page_of(s + 1, 0);
    SlotSpan next_sp = s + 1 < a.n_slots ? slot_span(a, s + 1) : sp;
    int page = first32, base = 0;  // page: of blocks base + lane
    int n = 0;                     // blocks loaded
    for (int f = f0; f < f1;) {
      const int j = f - pb;  // block of the pair
      if (j >= sp.blocks) {
        pb += sp.blocks + a.pair_cost;
        f = pb;
        if (++g == a.n_kv) {
          g = 0;
          ++s;
          sp = next_sp;
          first32 = next32;
          next32 = page_of(s + 1, 0);
          if (s + 1 < a.n_slots) next_sp = slot_span(a, s + 1);
        }
        page = first32;
        base = 0;
        continue;
      }
      if ((j & ~31) != base) {
        base = j & ~31;
        page = page_of(s, base);
      }
      int phys = __shfl_sync(0xFFFFFFFFu, page, j & 31);
      if (sp.n_new == 0 || (a.first + j) * kBlk >= sp.len) {
        phys = -2;  // nothing there
      } else if (phys < 0 || phys >= a.n_phys) {
        if (lane == 0) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, s);
        phys = -1;
      }
      const int st = n % kStages;
      if (lane == 0) {
        if (!mbar_wait(eb + 8u * st, ((uint32_t)(n / kStages) & 1u) ^ 1u, abort) &&
            atomicCAS(&s_abort, 0, 1) == 0)
          set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, s);
      }
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, *abort != 0)) break;  // the others' waits end on it too
      if (lane == 0) {
        // a page that is not there reads past the pool's end: the copy fills zeros
        const int row0 = (phys < 0 ? a.n_phys * a.n_kv : phys * a.n_kv + g) * kBlk;
        s_bad[st] = phys == -1;
        const uint32_t sk = sbase + (uint32_t)(st * 2 * kTile), sv = sk + kTile;
        const uint32_t bar = fb + 8u * st;
        mbar_arrive_expect_tx(bar, 2u * kTile);
#pragma unroll
        for (int bx = 0; bx < D / 64; ++bx) {
          tma_load_2d(sk + bx * (kBlk * 128), &tm_k, bx * 64, row0, bar, pol);
          tma_load_2d(sv + bx * (kBlk * 128), &tm_v, bx * 64, row0, bar, pol);
        }
      }
      ++f;
      ++n;
    }
    if (lane == 0) {
      // what is still in flight lands before the CTA goes (bounded)
      volatile int never = 0;
      for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
        mbar_wait(fb + 8u * (i % kStages), (uint32_t)(i / kStages) & 1u, &never);
    }
    __syncwarp();
  } else {
    // ---- the pairs of this CTA. A wait that runs out is recorded and ends
    // all waits; the loops go on to their end over what is there.
    const int gq = lane >> 2, cq = lane & 3;
    const int mt = warp % MT, ps = warp / MT;
    const int G = a.n_q / a.n_kv, rows = a.T * G;
    const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(D)
    const int mi = lane >> 3, rr = lane & 7;
    auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    // rows r = t * G + head in group, of the products ...
    const int r0 = mt * 16 + gq, r1 = r0 + 8;
    const int t0 = r0 < rows ? r0 / G : a.T, t1 = r1 < rows ? r1 / G : a.T;
    // ... of the output: one a thread, every 128 / kR-th float4 of it ...
    const int ro = tid % kR, co = tid / kR, to = ro / G;
    const int64_t o_off = ((int64_t)to * a.n_q + ro - to * G) * D + 4 * co;
    // ... and of the queries to fetch
    const uint32_t sq = sbase + kStages * 2 * kTile;
    int64_t q_off[kQPass > 0 ? kQPass : 1];
#pragma unroll
    for (int k = 0; k < kQPass; ++k) {
      const int r = tid / (D / 8) + k * (kOThr * 8 / D), t = r / G;
      q_off[k] = r < rows ? t * a.q_stride + (r - t * G) * D + tid % (D / 8) * 8 : -1;
    }
    auto fetch_q = [&](int slot, int head, int place) {
      const uint16_t* q0 = a.q + (int64_t)slot * a.T * a.q_stride + head * G * D;
#pragma unroll
      for (int k = 0; k < kQPass; ++k) {
        const int r = tid / (D / 8) + k * (kOThr * 8 / D);
        if (q_off[k] >= 0)
          cp_async16(sq + place * kQB + r * (D * 2) + ((tid % (D / 8)) ^ (r & 7)) * 16,
                     q0 + q_off[k], 16);
      }
    };
    int place = -1;  // of the pair's queries, -1: not asked for yet
    int f = f0, it = 0;  // it: blocks done
    while (f < f1) {
      const int fe = min(f1, pb + sp.blocks);
      if (f >= fe) {  // this CTA starts in a pair's cost
        pb += sp.blocks + a.pair_cost;
        f = pb;
        if (++g == a.n_kv) {
          g = 0;
          if (++s < a.n_slots) sp = slot_span(a, s);
        }
        continue;
      }
      const bool whole = f == pb && fe == pb + sp.blocks;
      // where the pair after this one starts, whose span and queries are on
      // their way from here on
      const int next_pb = pb + sp.blocks + a.pair_cost;
      const int next_g = g + 1 == a.n_kv ? 0 : g + 1, next_s = next_g == 0 ? s + 1 : s;
      // a row's last position, -1: sees nothing
      const int base = sp.len - sp.n_new;  // may be negative
      const int lim0 = t0 < sp.n_new ? base + t0 : -1;
      const int lim1 = t1 < sp.n_new ? base + t1 : -1;
      uint32_t qa[kKS][4];
      if (kQB > 0) {
        if (place < 0) fetch_q(s, g, place = 0);
        cp_async_wait();
        meet();  // what warps share is this pair's from here
        // rows that see nothing hold anything, which reaches nothing but them
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
          ldm_x4(sq + place * kQB + (mt * 16 + (mi & 1) * 8 + rr) * (D * 2) +
                     ((ks * 2 + (mi >> 1)) ^ rr) * 16,
                 qa[ks]);
        place ^= 1;
        if (next_pb < f1) fetch_q(next_s, next_g, place);
      } else {
        const uint16_t* q0 = lim0 >= 0 ? a.q + ((int64_t)s * a.T + t0) * a.q_stride + (g * G + r0 - t0 * G) * D : nullptr;
        const uint16_t* q1 = lim1 >= 0 ? a.q + ((int64_t)s * a.T + t1) * a.q_stride + (g * G + r1 - t1 * G) * D : nullptr;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          const int d = ks * 16 + 2 * cq;
          qa[ks][0] = q0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + d)) : 0u;
          qa[ks][1] = q1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + d)) : 0u;
          qa[ks][2] = q0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + d + 8)) : 0u;
          qa[ks][3] = q1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + d + 8)) : 0u;
        }
      }
      SlotSpan next_sp = sp;
      if (next_pb < f1 && next_s != s) next_sp = slot_span(a, next_s);
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      float oacc[kDT][4];
#pragma unroll
      for (int j = 0; j < kDT; ++j) oacc[j][0] = oacc[j][1] = oacc[j][2] = oacc[j][3] = 0.0f;
      for (; f < fe; ++f, ++it) {
        const int st = it % kStages;
        if (!mbar_wait(fb + 8u * st, (uint32_t)(it / kStages) & 1u, abort) &&
            atomicCAS(&s_abort, 0, 1) == 0)
          set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, s);
        const uint32_t sk = sbase + (uint32_t)(st * 2 * kTile), sv = sk + kTile;
        const int pos0 = (a.first + f - pb) * kBlk;
        const bool bad = s_bad[st] != 0;
        if (pos0 + kBlk > sp.len) {
          // rows past the slot's end hold anything, NaN too: 0 x NaN in P V
          // would reach the output, so each warp sets those it reads to 0
#pragma unroll
          for (int k = 0; k < kPos * (D / 8) / 32; ++k) {
            const int z = kPos * ps + (k * 32 + lane) / (D / 8);
            if (pos0 + z >= sp.len)
              *reinterpret_cast<uint4*>(sm + st * 2 * kTile + kTile + swz64(z, lane % (D / 8))) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // S = Q K^T over this warp's positions
        float sc[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int n = 0; n < kNT; n += 2) {
            uint32_t kb[4];
            ldm_x4(sk + swz64(kPos * ps + 8 * n + ((mi & 2) ? 8 : 0) + rr, ks * 2 + (mi & 1)), kb);
            mma16816t<F16>(sc[n], qa[ks], kb[0], kb[1]);
            mma16816t<F16>(sc[n + 1], qa[ks], kb[2], kb[3]);
          }
        // every row that is in use sees positions up to base
        if (bad || pos0 + kBlk - 1 > base) {
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pos = pos0 + kPos * ps + 8 * n + 2 * cq + h;
              if (bad || pos > lim0) sc[n][h] = -INFINITY;
              if (bad || pos > lim1) sc[n][2 + h] = -INFINITY;
            }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          mx0 = fmaxf(mx0, fmaxf(sc[n][0], sc[n][1]));
          mx1 = fmaxf(mx1, fmaxf(sc[n][2], sc[n][3]));
        }
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, d));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, d));
        }
        const float n0 = fmaxf(m0, mx0 * sl2), n1 = fmaxf(m1, mx1 * sl2);
        // all masked so far: everything stays 0 (no inf - inf)
        const float u0 = n0 == -INFINITY ? 0.0f : n0, u1 = n1 == -INFINITY ? 0.0f : n1;
        const float c0 = ex2(m0 - u0), c1 = ex2(m1 - u1);
        m0 = n0;
        m1 = n1;
        l0 *= c0;
        l1 *= c1;
        const float x0 = lift<F16>() - u0, x1 = lift<F16>() - u1;
        uint32_t pa[kNT / 2][4];
        // the sums take the rounded weights, the ones that the product sees
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const uint32_t w0 = pack2<F16>(ex2(fmaf(sc[n][0], sl2, x0)), ex2(fmaf(sc[n][1], sl2, x0)));
          const uint32_t w1 = pack2<F16>(ex2(fmaf(sc[n][2], sl2, x1)), ex2(fmaf(sc[n][3], sl2, x1)));
          l0 += unpack_lo<F16>(w0) + unpack_hi<F16>(w0);
          l1 += unpack_lo<F16>(w1) + unpack_hi<F16>(w1);
          pa[n / 2][2 * (n & 1)] = w0;
          pa[n / 2][2 * (n & 1) + 1] = w1;
        }
#pragma unroll
        for (int j = 0; j < kDT; ++j) {
          oacc[j][0] *= c0;
          oacc[j][1] *= c0;
          oacc[j][2] *= c1;
          oacc[j][3] *= c1;
        }
#pragma unroll
        for (int kp = 0; kp < kPos / 16; ++kp)
#pragma unroll
          for (int j = 0; j < kDT; j += 2) {
            uint32_t vb[4];
            ldm_x4_t(sv + swz64(kPos * ps + 16 * kp + ((mi & 1) ? 8 : 0) + rr, j + (mi >> 1)), vb);
            mma16816t<F16>(oacc[j], pa[kp], vb[0], vb[1]);
            mma16816t<F16>(oacc[j + 1], pa[kp], vb[2], vb[3]);
          }
        if (f + 1 == fe) break;  // the last block's stage is kept for what follows
        // the stage goes back to the loader, after this warp's reads and writes
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(eb + 8u * st);
      }
      // ---- the slices' (m, l, O) become the segment's. Each warp's O, weighed,
      // goes to a quarter of the stage whose keys and values all are done with
      // ([16][D] floats, 16-byte pieces in an order that spreads the banks), and
      // a thread then adds up what the slices have for it. (One place of 8 KB
      // that the warps added to in turn, and rows by division, took three times
      // as long: 1.5 of a short pair's 3.6 us.)
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
        l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
      }
      // a row that sees nothing weighs nothing, whatever was summed for it
      if (lim0 < 0) {
        m0 = -INFINITY;
        l0 = 0.0f;
      }
      if (lim1 < 0) {
        m1 = -INFINITY;
        l1 = 0.0f;
      }
      if (cq == 0) {
        s_m[warp][gq] = m0;
        s_m[warp][gq + 8] = m1;
        s_l[warp][gq] = l0;
        s_l[warp][gq + 8] = l1;
      }
      meet();
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int k = 0; k < kNS; ++k) {
        M0 = fmaxf(M0, s_m[mt + k * MT][gq]);
        M1 = fmaxf(M1, s_m[mt + k * MT][gq + 8]);
      }
      const float U0 = M0 == -INFINITY ? 0.0f : M0, U1 = M1 == -INFINITY ? 0.0f : M1;
      if (ps == 0 && cq == 0) {
        float L0 = 0.0f, L1 = 0.0f;
#pragma unroll
        for (int k = 0; k < kNS; ++k) {
          L0 += s_l[mt + k * MT][gq] * ex2(s_m[mt + k * MT][gq] - U0);
          L1 += s_l[mt + k * MT][gq + 8] * ex2(s_m[mt + k * MT][gq + 8] - U1);
        }
        s_M[r0] = M0;
        s_M[r1] = M1;
        s_L[r0] = L0;
        s_L[r1] = L1;
      }
      const float w0 = ex2(m0 - U0), w1 = ex2(m1 - U1);
      const int st = it % kStages;
      float* area = reinterpret_cast<float*>(sm + st * 2 * kTile);
      auto piece = [](int r) { return ((r & 3) << 1) | ((r >> 2) & 1); };
      {
        float* mine = area + warp * (16 * D) + gq * D + 2 * (cq & 1);
        const int x = piece(gq);  // and of row gq + 8
#pragma unroll
        for (int j = 0; j < kDT; ++j) {
          float* p0 = mine + ((2 * j + (cq >> 1)) ^ x) * 4;
          *reinterpret_cast<float2*>(p0) = make_float2(oacc[j][0] * w0, oacc[j][1] * w0);
          *reinterpret_cast<float2*>(p0 + 8 * D) = make_float2(oacc[j][2] * w1, oacc[j][3] * w1);
        }
      }
      meet();
      // the pair's parts: one place per CTA and pair, both of which grow
      // along the line
      const int pair = s * a.n_kv + g;
      const bool direct = whole && !a.join;
      float* part = a.part + (int64_t)((int)blockIdx.x + pair) * kR * (D + 2);
      uint16_t* out = a.o + ((int64_t)s * a.T * a.n_q + g * G) * D + o_off;
      if (ro < rows) {
        const float* from = area + (ro >> 4) * (16 * D) + (ro & 15) * D;
        const int x = piece(ro);
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
          const int d = co + k * (kOThr / kR);
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < kNS; ++i) {
            const float4 u = *reinterpret_cast<const float4*>(from + i * MT * (16 * D) + (d ^ x) * 4);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          if (direct)
            store4<F16>(out + k * (kOThr / kR * 4), v, s_L[ro]);
          else
            *reinterpret_cast<float4*>(part + 2 * kR + (d * kR + ro) * 4) = v;
        }
      }
      // the stage goes back to the loader
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(eb + 8u * st);
      ++f;
      ++it;
      if (!direct) {
        if (tid < rows) {
          part[tid] = s_M[tid];
          part[kR + tid] = s_L[tid];
        }
        if (a.join) {
          if (tid == 0 && pb >= f0) a.pair_start[pair] = pb;  // the pair's first CTA
        } else {
          // the pair's CTAs: first and last to hold a block of it
          const int c0 = pb / per, c1 = (pb + sp.blocks - 1) / per;
          __threadfence();
          meet();
          if (tid == 0) {
            unsigned* cnt = a.count + c0;  // whose end cuts this pair and no other
            s_last = atomicAdd(cnt, 1u) == (unsigned)(c1 - c0);
            if (s_last) *cnt = 0u;  // ready for the next call
            __threadfence();
          }
          meet();
          if (s_last && ro < rows) {
#pragma unroll 1
            for (int k = 0; k < kCols; ++k) {
              Joined jn{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
              const PartRef own = part_ref(a.part + (int64_t)(c0 + pair) * kR * (D + 2), kR, ro,
                                           co + k * (kOThr / kR));
              join_parts<4>(jn, c1 - c0 + 1, [&](int c) {
                return PartRef{own.p + c * (kR * (D + 2)), own.l_at, own.o_at};
              });
              store4<F16>(out + k * (kOThr / kR * 4), jn.o, jn.L);
            }
          }
        }
      }
      if (kQB == 0) meet();  // what warps share is the next pair's from here
      // ---- the next pair
      pb = next_pb;
      f = pb;
      g = next_g;
      s = next_s;
      sp = next_sp;
    }
    if (a.join && blockIdx.x == 0 && tid == 0) a.line[0] = per;
  }
  if (shared) {
    // the join waits for this kernel, and this one for the shared part
    pdl_wait();
    pdl_trigger();
  }
}

// Joins the shared part's stretches and the own parts. kLanes threads for four
// elements of a row, each with every kLanes-th part, so that all of a row's
// parts are fetched at once; then the threads' results in their order. A CTA
// has items of one pair, rows (1 << row_bits of them, the pair's and none)
// fastest, of which it takes one batch after the other (a CTA a batch took 22
// us of 53 for 32000 rows, one after the other 19); divisions by what the
// kernel is given are done once a CTA. Latency bounds it: 14 us of 175 for 720
// tokens of 16 heads with about five parts a row, 34 MB from L2, and as long
// with batches of three to six parts.
template <bool F16, int D, int kLanes>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnBatchArgs a, int kR, int row_bits) {
  constexpr int kItems = 256 / kLanes;
  __shared__ float4 s_o[kLanes][kItems];
  __shared__ float2 s_ml[kLanes][kItems];
  __shared__ int s_cut[2][2];  // for the two tiles that a pair's rows can lie in: first stretch, how many
  __shared__ int s_own[2];     // first own part, how many
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, g = blockIdx.z, pair = s * a.n_kv + g;
  const int G = a.n_q / a.n_kv, rows = a.T * G;
  const bool shared = a.px_steps > 0;
  const SlotSpan sp = slot_span(a, s);
  const int row0 = shared ? __ldg(a.tok_start + s) * G : 0;
  if (threadIdx.x < 2 && shared) {
    const int per = __ldg(a.line + 1), len = __ldg(a.line + 2);
    const int u = ((row0 >> 8) + (int)threadIdx.x) * a.n_kv + g;
    const int x0 = u * len / per;
    s_cut[threadIdx.x][0] = x0;
    s_cut[threadIdx.x][1] = (u * len + a.px_steps - 1) / per - x0 + 1;
  } else if (threadIdx.x == 2) {
    const int per = __ldg(a.line), pb = __ldg(a.pair_start + pair);
    s_own[0] = pb / per;
    s_own[1] = (pb + sp.blocks - 1) / per - s_own[0] + 1;
  }
  __syncthreads();
  const int item = threadIdx.x % kItems, ln = threadIdx.x / kItems;
  for (int i0 = blockIdx.y * kItems; i0 < (D / 4) << row_bits; i0 += gridDim.y * kItems) {
    const int i = i0 + item;
    const int d = i >> row_bits, r = i & ((1 << row_bits) - 1);
    // r / G for r < 64: the product is off by less than 1/2 G steps of 2^-24
    const int t = (int)(((float)r + 0.5f) * (1.0f / (float)G));
    if (kLanes > 1) __syncthreads();  // the threads' results of the items before are read
    Joined jn{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    const bool here = r < rows && d < D / 4;
    if (here && t < sp.n_new && sp.len - sp.n_new + t >= 0) {
      const int row = row0 + r, tile = (row >> 8) - (row0 >> 8), u = (row >> 8) * a.n_kv + g;
      const int nx = shared ? s_cut[tile][1] : 0, n = nx + s_own[1];
      const PartRef px = part_ref(a.px_part + (int64_t)(shared ? s_cut[tile][0] + u : 0) * 256 * (D + 2),
                                  256, row & 255, d);
      const PartRef own = part_ref(a.part + (int64_t)(s_own[0] + pair) * kR * (D + 2), kR, r, d);
      join_parts<6>(jn, (n - ln + kLanes - 1) / kLanes, [&](int c) {
        const int k = c * kLanes + ln;
        return k < nx ? PartRef{px.p + k * (256 * (D + 2)), px.l_at, px.o_at}
                      : PartRef{own.p + (k - nx) * (kR * (D + 2)), own.l_at, own.o_at};
      });
    }
    if (kLanes > 1) {
      s_o[ln][item] = jn.o;
      s_ml[ln][item] = make_float2(jn.M, jn.L);
      __syncthreads();
      if (ln > 0) continue;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kLanes; ++k) M = fmaxf(M, s_ml[k][item].x);
      const float U = M == -INFINITY ? 0.0f : M;
      jn = Joined{M, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll
      for (int k = 0; k < kLanes; ++k) {
        const float w = ex2(s_ml[k][item].x - U);
        const float4 v = s_o[k][item];
        jn.L = fmaf(s_ml[k][item].y, w, jn.L);
        jn.o.x = fmaf(v.x, w, jn.o.x);
        jn.o.y = fmaf(v.y, w, jn.o.y);
        jn.o.z = fmaf(v.z, w, jn.o.z);
        jn.o.w = fmaf(v.w, w, jn.o.w);
      }
    }
    if (here)
      store4<F16>(a.o + (((int64_t)s * a.T + t) * a.n_q + g * G + r - t * G) * D + 4 * d, jn.o, jn.L);
  }
}

template <bool F16, int D, int kLanes>
cudaError_t launch_join(const AttnBatchArgs& a, int kR, cudaStream_t stream) {
  const int rows = a.T * (a.n_q / a.n_kv), per = 256 / kLanes;
  int bits = 0;
  while (1 << bits < rows) ++bits;
  // about as many CTAs as there is room for at once, four an SM
  const int items = (((D / 4) << bits) + per - 1) / per;
  const int64_t pairs = (int64_t)a.n_slots * a.n_kv, fit = (4 * a.sms + pairs - 1) / pairs;
  const int y = items < fit ? items : (int)fit;
  return launch_pdl(attn_join_kernel<F16, D, kLanes>, dim3(a.n_slots, y, a.n_kv), dim3(256), 0,
                    stream, a, kR, bits);
}

bool attn_batch_supported(const moe_attn_batch_shape_t* s) {
  if (!s) return false;
  if (s->n_slots < 1 || s->n_slots > 4096 || s->T < 1 || s->T > 64) return false;
  if (s->n_q < 1 || s->n_kv < 1 || s->n_kv > 64 || s->n_q % s->n_kv) return false;
  if ((int64_t)(s->n_q / s->n_kv) * s->T > 64) return false;
  if (s->D != 64 && s->D != 128) return false;
  if (s->block != kBlk || s->max_blocks < 1 || s->max_blocks > (1 << 18)) return false;
  if (s->prefix_blocks < 0 || s->prefix_blocks > s->max_blocks) return false;
  if (s->dtype != MOE_DTYPE_BF16 && s->dtype != MOE_DTYPE_FP16) return false;
  // the line of blocks is counted in 32 bits
  return (int64_t)s->n_slots * s->n_kv * s->max_blocks < (1 << 30);
}

namespace {
int own_tiles(const moe_attn_batch_shape_t* s) {  // row tiles: 1, 2 or 4
  const int rows = s->T * (s->n_q / s->n_kv);
  return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
constexpr int kMostSms = 256;
constexpr int kMostCtas = 3 * kMostSms;  // of attn_own_kernel
// Whether the prefix is read once for all slots. Otherwise each slot's own line
// reads it, in one or two launches instead of three, which is shorter while
// the slots' prefix blocks together are few. Measured, per slot against shared
// (blocks over all slots and heads, those of D = 64 as halves): rows of one
// tile 9.7 and 12.5 us at 512, 10.8 and 12.7, 13.4 and 13.4 at 1024, 16.1 and
// 15.2, 17.6 and 15.2 at 2048; of more tiles, blocks times tiles, 15.2 and
// 16.5, 19.1 and 17.0 at 2048 (13.3 and 15.2 with D = 64), 18.6 and 16.6, 25.8
// and 22.7 at 4096.
bool share(const moe_attn_batch_shape_t* s) {
  if (s->prefix_blocks == 0 || s->n_slots == 1) return false;
  const int64_t blocks = (int64_t)s->n_slots * s->n_kv * s->prefix_blocks;
  const int mt = own_tiles(s);
  return blocks * s->D / 128 * mt > (mt > 1 ? 2048 : 1024);
}
// a place per CTA and pair
size_t own_part_bytes(const moe_attn_batch_shape_t* s) {
  const size_t places = kMostCtas + (size_t)s->n_slots * s->n_kv;
  return round256(places * own_tiles(s) * 16 * (s->D + 2) * 4);
}

template <bool F16, int D, int MT>
cudaError_t launch_own(const CUtensorMap& tk, const CUtensorMap& tv, const AttnBatchArgs& a,
                       int grid, cudaStream_t stream) {
  const size_t smem =
      1024 + (size_t)OwnRing<D>::kStages * 2 * OwnRing<D>::kTile + 2 * kQTile<D, MT>;
  cudaError_t e = cudaFuncSetAttribute(attn_own_kernel<F16, D, MT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_own_kernel<F16, D, MT>, dim3(grid), dim3(kOAll), smem, stream, tk, tv, a);
  if (e != cudaSuccess || !a.join) return e;
  // A thread fetches six parts at once; with more of them several threads
  // share an output while all of them run at once (30 parts, 25000 outputs:
  // 18.8 us the call with four, 20.3 with one; 70000 outputs: 36.2 and 33.4).
  const int64_t outs = (int64_t)a.n_slots * a.T * a.n_q * (D / 4);
  if (a.parts <= 6 || outs > 32768) return launch_join<F16, D, 1>(a, MT * 16, stream);
  if (a.parts <= 48 || outs > 8192) return launch_join<F16, D, 4>(a, MT * 16, stream);
  return launch_join<F16, D, 16>(a, MT * 16, stream);
}
template <bool F16, int D>
cudaError_t launch_own_mt(int mt, const CUtensorMap& tk, const CUtensorMap& tv,
                          const AttnBatchArgs& a, int grid, cudaStream_t stream) {
  if (mt == 1) return launch_own<F16, D, 1>(tk, tv, a, grid, stream);
  if (mt == 2) return launch_own<F16, D, 2>(tk, tv, a, grid, stream);
  return launch_own<F16, D, 4>(tk, tv, a, grid, stream);
}
}  // namespace

// status and the lines' steps, the CTAs' counters, the pairs' starts, the
// slots' first tokens, the pairs' parts, the shared part's. The counters are
// all that one call leaves to the next (zeros), so their place and extent are
// the same for every shape: a server's batch grows and shrinks in one
// workspace.
constexpr size_t kCountAt = 512, kStartAt = kCountAt + kMostCtas * 4;
size_t attn_batch_ws_bytes(const moe_attn_batch_shape_t* s) {
  return kStartAt + round256((size_t)s->n_slots * s->n_kv * 4) +
         round256((size_t)s->n_slots * 4) + own_part_bytes(s) +
         (s->prefix_blocks > 0 ? prefix_part_floats(s, kMostSms) * 4 : 0);
}

cudaError_t launch_attn_batch(const moe_attn_batch_shape_t* s, const CUtensorMap& tk,
                              const CUtensorMap& tv, AttnBatchArgs a, uint8_t* ws, int nsm,
                              cudaStream_t stream) {
  a.ctrl = reinterpret_cast<Ctrl*>(ws);
  const size_t pairs = round256((size_t)s->n_slots * s->n_kv * 4);
  a.line = reinterpret_cast<int32_t*>(ws + 256);
  a.count = reinterpret_cast<unsigned*>(ws + kCountAt);
  a.pair_start = reinterpret_cast<int32_t*>(ws + kStartAt);
  a.tok_start = reinterpret_cast<int32_t*>(ws + kStartAt + pairs);
  a.part = reinterpret_cast<float*>(ws + kStartAt + pairs + round256((size_t)s->n_slots * 4));
  a.pair_cost = s->D == 64 || own_tiles(s) > 1 ? 4 : 2;
  a.n_slots = s->n_slots;
  a.T = s->T;
  a.n_q = s->n_q;
  a.n_kv = s->n_kv;
  a.max_blocks = s->max_blocks;
  a.prefix_blocks = s->prefix_blocks;
  const int sms = nsm < kMostSms ? nsm : kMostSms;
  const int mt = own_tiles(s);
  a.first = 0;
  a.px_steps = 0;
  int room = sms;  // SMs that the slots' own lines can have
  a.sms = sms;
  // fitted over twenty shapes; 0.15 more or less costs 2 to 8 us where the
  // next cut is another one, nothing elsewhere (a step takes 1.3 to 1.7 us, a
  // unit 0.15 to 0.4 us of an SM's two or three CTAs)
  a.unit_weight = s->D == 64 ? (mt == 1 ? 0.115f : 0.23f) : (mt == 1 ? 0.23f : 0.36f);
  a.parts = 0;
  if (share(s)) {
    // What the kernel gets of the SMs if every token is there and the slots'
    // own lines are as short as they can be, and as long: the most that it is
    // launched with, and what it leaves is the most for the own lines. (CTAs
    // for nothing cost 2 to 3 us where they stand in the way.) Where the own
    // lines are over in two steps anyway, nothing depends on the lengths.
    const PrefixLine whole = prefix_line(s, sms);
    const int64_t own_pairs = (int64_t)s->n_slots * s->n_kv;
    auto plan = [&](int64_t units) {
      PrefixWay best{};
      for (int i = 0; i < kWays; ++i) {
        const PrefixWay w =
            prefix_way(i, whole.pairs, whole.steps, (int)units, a.unit_weight, sms, sms - 1);
        if (i == 0 || w.time < best.time) best = w;
      }
      return best;
    };
    const int own_most = s->max_blocks - s->prefix_blocks > 1 ? s->max_blocks - s->prefix_blocks : 1;
    const PrefixLine line = plan(own_pairs * (1 + a.pair_cost)).line;
    const PrefixWay least = plan(own_pairs * (own_most + a.pair_cost));
    a.px_fixed = least.line.grid == line.grid && least.time <= 2.0f;
    room = sms - least.line.grid;
    a.first = s->prefix_blocks;
    a.px_steps = line.steps;
    a.px_most = line.grid;
    a.parts = (line.steps + line.per - 1) / line.per + 1;
    a.px_part = a.part + own_part_bytes(s) / 4;
    const cudaError_t e = launch_attn_prefix(s, tk, tv, a, line.grid, stream);
    if (e != cudaSuccess) return e;
  }
  // as many CTAs as fit there, and no more than there can be blocks
  const int64_t most = (int64_t)s->n_slots * s->n_kv * s->max_blocks;
  const int grid = (int)(most < own_ctas(s->D, mt) * room ? most : own_ctas(s->D, mt) * room);
  // the parts of a pair's own blocks, were all pairs as long as they can be
  const int64_t pairs_n = (int64_t)s->n_slots * s->n_kv;
  a.parts += (int)(grid / pairs_n < s->max_blocks - a.first ? grid / pairs_n : s->max_blocks - a.first);
  // Parts are joined by a pair's last CTA where few pairs are cut: 5.7 us
  // against 7.6 by a kernel of its own for pairs of two blocks (D = 128, 8 rows;
  // 9.6 and 12.1 for 512 such pairs, 67 and 70 for 1024 of up to 32), but 12.5
  // and 10.7 for 128 pairs of up to 16, 24.4 and 21.9 for 512, 11.9 and 8.6 for
  // 32 with nine parts each; with 64 rows 11.1 and 11.2 for two blocks, 16.6
  // and 12.2 for eight. In between, 8.2 and 7.5 for three to five blocks, the
  // second launch costs the host the 1.7 us that such a call cannot hide. A
  // pair of `longest` is cut if a border, `per` units apart, falls into it.
  const int longest = s->max_blocks - a.first;
  const int64_t per = (pairs_n * (longest + a.pair_cost) + grid - 1) / grid;
  const bool cut = longest >= (mt == 4 && s->D == 128 ? 2 : 3) && 2 * longest > per;
  a.join = a.px_steps > 0 || a.parts > 6 || (cut && (mt > 1 || per >= 6));
  if (s->dtype == MOE_DTYPE_FP16)
    return s->D == 64 ? launch_own_mt<true, 64>(mt, tk, tv, a, grid, stream)
                      : launch_own_mt<true, 128>(mt, tk, tv, a, grid, stream);
  return s->D == 64 ? launch_own_mt<false, 64>(mt, tk, tv, a, grid, stream)
                    : launch_own_mt<false, 128>(mt, tk, tv, a, grid, stream);
}

}  // namespace moe

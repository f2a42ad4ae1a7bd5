// The shared part of the batch's attention: every slot's rows against the
// prefix pages, which are read once for all of them.
//
// The tokens that are there (t < n_new[s]) are counted through, so a batch of
// uneven drafts has no empty rows: row tok G + head of key/value head g
// belongs to the tok-th of them, and attention over the prefix is one pair of
// large products per key/value head on the tensor cores (tcgen05): tiles of
// 256 rows (two of M = 128) against steps of 128 positions (two pages),
// S = Q K^T into TMEM, softmax weights P back into TMEM over S, O += P V.
// The (tile, head) pairs' steps lie on one line cut over CTAs, one an SM; each
// stretch leaves (m, l, O) of its 256 rows in the
// workspace, where attn_join_kernel joins them with the slots' own positions.
// Both parts run at once, on SMs of their own (best_line): a CTA without a
// stretch goes as soon as it has read the lengths, and leaves its SM to the
// slots' own line. One after the other on all SMs, 106 slots of up to 1726
// positions under 32 pages took 43.6 us, side by side 32.7; 48 of up to 777
// under 128 took 21.3 and 18.2.
//
// Warps: 0 loads K and V (TMA, two stages each of 128 positions), 1 and 2
// issue the products of the two row tiles, 4-11 and 12-19 do the softmax of
// the two row tiles, half a row a thread (the two warps of 32 rows exchange
// the halves' maxima through shared memory). While one tile's weights are
// formed the other's products run. The reference that a row's weights are
// relative to is only raised when the row grows past it by 2^8 (any reference
// near the maximum does): O in TMEM is rescaled a few times per stretch, not
// at every step.
//
// Measured at 256 slots of up to 4 tokens (12288 query rows a key/value head
// of 2 in all, D = 128, bf16) under 32768 positions, this kernel alone:
//   282 us  four warps a tile, a row a thread, one lane issuing with
//           descriptors built per product, rows of absent tokens computed
//   162 us  eight warps a tile, half a row a thread; absent tokens left out
//   141 us  one elected lane of a uniform warp issues, descriptors by
//           addition, a warp a tile, in turns
// and the whole call 181 us, 174 with the line cut pair by pair, 171 with the
// queries fetched by whole lines, 170 with the slots' own lines beside it.
// Leaving parts out for timing: without the exponentials the call takes as
// long as with them, without the maxima and their exchange 13 us less, without
// any softmax 23 us less, and then without the loads still as long: the rest
// is the products' own time and hand-over. 1.5 PFLOP/s, 0.78 of the burst rate
// of a plain bf16 product.
//
// Per step and two tiles (D = 128) the products take 32 MMAs of N = 128 at 64
// to 77 clocks, about 2256, and their operands, the TMA writes among them,
// about as much of shared memory's 128 bytes a clock; the exponentials 1024
// to 2048. A step's 64 KB come from HBM for the first tile, from L2 after.
#include "attn_batch.cuh"

namespace moe {

namespace {
constexpr int kPThr = 640;      // a warpgroup of single warps, 2 x 2 of softmax warps
constexpr int kPStep = 128;     // positions of a step
constexpr int kPStages = 2;
constexpr float kSlack = 8.0f;  // growth of a row (log2) that its reference may lag behind

// shared-memory descriptor of a 16-bit operand whose M or N index runs along
// the 128-byte swizzled rows (64 elements; lbo bytes to the next 64), the
// reduction index from row to row (8 rows = 1024 bytes)
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(lbo >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// kind::f16 instruction: fp32 D, A and B of one 16-bit type, A K-major, B
// K-major or (bmn) N-major
__device__ __forceinline__ constexpr uint32_t idesc16(bool f16, int M, int N, bool bmn) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (bmn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// true in one lane of the warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

struct PrefixBars {
  uint64_t k_full[kPStages], k_empty[kPStages], v_full[kPStages], v_empty[kPStages];
  uint64_t q_ready[2], s_full[2], p_ready[2], pv_done[2], turn[2], drain[2];
  uint64_t v_end;  // values of the step in which the longest slot ends
};
// The values of the step in which the longest slot ends, once they are there:
// rows from `end` to the end of its page become 0. Out of line: it is rare.
template <int D>
__device__ __noinline__ bool end_values(uint32_t sv, int end, uint32_t landed, uint32_t parity) {
  volatile int never = 0;  // bounded, and the copies land whatever the other roles do
  const bool ok = mbar_wait(landed, parity, &never);
#pragma unroll 1
  for (int r = end; r % kBlk != 0; ++r)
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                       sv + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16),
                   "r"(0)
                   : "memory");
  fence_proxy_async_smem();  // the tensor core reads it
  return ok;
}
}  // namespace

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;"
      : "=f"(r)
      : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}

template <bool F16, int D>
__global__ void __launch_bounds__(kPThr, 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const AttnBatchArgs a) {
  constexpr int kHalves = D / 64;              // 64-element column halves of a tile
  constexpr uint32_t kHalf = 128 * 128;        // bytes of 128 rows of one
  constexpr uint32_t kTile = kHalves * kHalf;  // a Q, K or V tile
  constexpr uint32_t kO = 0, kS = 256;         // TMEM columns: O tiles, then S tiles
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  __shared__ __align__(8) PrefixBars bars;
  __shared__ float s_mx[2][2][2][128];  // step parity, row tile, half, row
  __shared__ int s_scan[kPThr / 32], s_units[kPThr / 32], s_long[kPThr / 32], s_line[5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t sbase = (smem_u32(sm_raw) + 1023u) & ~1023u;
  uint8_t* sm = sm_raw + (sbase - smem_u32(sm_raw));
  const uint32_t sq = sbase, sk = sq + 2 * kTile, sv = sk + kPStages * kTile;
  // tokens before each slot
  int* s_tok = reinterpret_cast<int*>(sm + (2 + 2 * kPStages) * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.n_q / a.n_kv;
  auto bar = [&](const uint64_t& b) { return smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < kPStages; ++i) {
      mbar_init(bar(bars.k_full[i]), 1);
      mbar_init(bar(bars.k_empty[i]), 2);  // both tiles' products
      mbar_init(bar(bars.v_full[i]), 1);
      mbar_init(bar(bars.v_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.q_ready[i]), 8);  // the tile's warps
      mbar_init(bar(bars.s_full[i]), 1);
      mbar_init(bar(bars.p_ready[i]), 8);
      mbar_init(bar(bars.pv_done[i]), 1);
      mbar_init(bar(bars.turn[i]), 1);
      mbar_init(bar(bars.drain[i]), 1);
    }
    mbar_init(bar(bars.v_end), 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  pdl_trigger();
  // ---- the tokens that are there, counted through, and the units of the
  // slots' own line; one warp finds the shared part's
  {
    const int chunk = (a.n_slots + kPThr - 1) / kPThr;
    const int s0 = min(tid * chunk, a.n_slots), s1 = min(s0 + chunk, a.n_slots);
    int sum = 0, units = 0, longest = 0;
    // the whole span: its length is read again for the rows, out of L1 then
    for (int s = s0; s < s1; ++s) {
      const SlotSpan sp = slot_span(a, s);
      sum += sp.n_new;
      units += sp.blocks + a.pair_cost;
      longest = max(longest, sp.n_new > 0 ? sp.len : 0);
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    units = __reduce_add_sync(0xFFFFFFFFu, units);
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if (lane == 31) {
      s_scan[warp] = incl;
      s_units[warp] = units;
      s_long[warp] = longest;
    }
    __syncthreads();
    if (warp == 3) {
      constexpr int kWarps = kPThr / 32;
      const int all = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? s_scan[lane] : 0);
      units = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? s_units[lane] : 0) * a.n_kv;
      longest = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? s_long[lane] : 0);
      const PrefixLine line = best_line(a, all, units);
      if (lane == 0) {
        s_line[0] = line.per;
        s_line[1] = line.len;
        s_line[2] = line.pairs * line.len;
        s_line[3] = all;
        s_line[4] = longest;
      }
    }
    if (s0 < s1) {
      int run = incl - sum;
      for (int w = 0; w < warp; ++w) run += s_scan[w];
      for (int s = s0; s < s1; ++s) {
        s_tok[s] = run;
        if (blockIdx.x == 0) a.tok_start[s] = run;
        run += slot_tokens(a, s);
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int R = s_line[3] * G, steps = a.px_steps, plen = s_line[1];
  const int f0 = (int)min((int64_t)blockIdx.x * s_line[0], (int64_t)s_line[2]);
  const int f1 = min(f0 + s_line[0], s_line[2]);
  if (blockIdx.x == 0 && tid == 0) {
    a.line[1] = s_line[0];
    a.line[2] = plen;
  }
  volatile int* abort = &s_abort;
  // a bounded wait; one that runs out is recorded and ends every role
  auto wait = [&](const uint64_t& b, uint32_t parity) {
    if (mbar_wait(bar(b), parity, abort)) return true;
    if (atomicCAS(&s_abort, 0, 1) == 0) set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, -2);
    return false;
  };
  // the line's stretch f0 .. f1, pair u (tile u / n_kv, head u % n_kv) by
  // pair; a pair's units from `steps` on are nothing
  if (warp == 0) {
    // ---- the loader, one lane. Positions from `longest` on belong to no slot
    // and may hold anything, NaN too: 0 x NaN in P V would reach the output.
    // Pages past it are read as pages that are not there are; the page that it
    // ends in has the rest of its values set to 0 before the step goes on.
    if (lane == 0) {
      const int longest = s_line[4];
      volatile int never = 0;
      int n = 0, ends = 0;  // steps loaded, those among them in which longest lies
      for (int f = f0; f < f1; ++f) {
        const int u = f / plen, j = f - u * plen, g = u % a.n_kv;
        if (j >= steps) continue;
        const int st = n % kPStages;
        const uint32_t ph = (uint32_t)(n / kPStages) & 1u;
        int row[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int jb = 2 * j + i;
          const int phys = jb < a.prefix_blocks ? __ldg(a.prefix + jb) : -1;
          const bool bad = phys < 0 || phys >= a.n_phys;
          if (bad && jb < a.prefix_blocks) set_error(a.ctrl, MOE_ERR_BAD_INPUT, KID_ATTNB, -1);
          // a page that is not there reads past the pool's end: zeros
          row[i] = (bad || jb * kBlk >= longest ? a.n_phys * a.n_kv : phys * a.n_kv + g) * kBlk;
        }
        const int end = longest - j * kPStep;  // of what is anyone's, in the step
        const bool inside = end > 0 && end < kPStep && end % kBlk != 0;
        const uint32_t b_v = bar(inside ? bars.v_end : bars.v_full[st]);
        if (!wait(bars.k_empty[st], ph ^ 1u)) break;
        mbar_arrive_expect_tx(bar(bars.k_full[st]), kTile);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_rows(sk + st * kTile + h * kHalf + i * (kBlk * 128), &tm_k, h * 64, row[i],
                          bar(bars.k_full[st]));
        if (!wait(bars.v_empty[st], ph ^ 1u)) {
          // the keys just asked for must land before the CTA goes
          mbar_wait(bar(bars.k_full[st]), ph, &never);
          break;
        }
        mbar_arrive_expect_tx(b_v, kTile);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_rows(sv + st * kTile + h * kHalf + i * (kBlk * 128), &tm_v, h * 64, row[i],
                          b_v);
        if (inside) {
          if (!end_values<D>(sv + st * kTile, end, b_v, (uint32_t)ends++ & 1u) &&
              atomicCAS(&s_abort, 0, 1) == 0)
            set_error(a.ctrl, MOE_ERR_TIMEOUT, KID_ATTNB, -2);
          mbar_arrive(bar(bars.v_full[st]));
        }
        ++n;
      }
      // what is still in flight lands before the CTA goes (bounded)
      for (int i = n > kPStages ? n - kPStages : 0; i < n; ++i) {
        mbar_wait(bar(bars.k_full[i % kPStages]), (uint32_t)(i / kPStages) & 1u, &never);
        mbar_wait(bar(bars.v_full[i % kPStages]), (uint32_t)(i / kPStages) & 1u, &never);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // The products of row tile w. The whole warp follows the line and waits;
    // one elected lane issues. Its descriptors differ by constants, so an
    // instruction costs an addition. The two warps take turns: with the
    // tiles' products mixed both tiles would wait for all of them, then both
    // do their softmax at once. (One warp for both tiles adds its waits to the
    // tensor core's time.)
    const int w = warp - 1;
    constexpr uint32_t id_s = idesc16(F16, 128, kPStep, false), id_o = idesc16(F16, 128, D, true);
    constexpr uint32_t kTileD = kTile >> 4;  // in a descriptor's address units
    const uint64_t dq = smem_desc_sw128(sq + w * kTile), dk = smem_desc_sw128(sk);
    const uint64_t dv = desc_mn_sw128(sv, kHalf);
    const uint32_t tS = tmem + kS + w * 128, tO = tmem + kO + w * 128;
    const uint32_t b_k_empty = bar(bars.k_empty[0]), b_v_empty = bar(bars.v_empty[0]);
    auto qk = [&](int st) {
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
          mma_bf16_ss(tS, dq + off, dk + st * kTileD + off, id_s, ks > 0);
        }
        mma_commit(bar(bars.s_full[w]));
        mma_commit(b_k_empty + 8 * st);
      }
      __syncwarp();
    };
    auto pv = [&](int st, bool fresh) {
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kPStep / 16; ++ks)
          mma_bf16_ts(tO, tS + ks * 8, dv + st * kTileD + ks * (2048 >> 4), id_o,
                      ks > 0 || !fresh);
        mma_commit(bar(bars.pv_done[w]));
        mma_commit(b_v_empty + 8 * st);
      }
      __syncwarp();
    };
    auto wait_all = [&](const uint64_t& b, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0;
    };
    int n = 0, pn = 0, qn = 0, tn = 0;
    bool ok = true;
    for (int f = f0; ok && f < f1;) {
      const int u = f / plen, j0 = f - u * plen;
      const int cnt = min(steps - j0, f1 - f);
      f = cnt < 1 || j0 + cnt == steps ? (u + 1) * plen : f + cnt;
      if (cnt < 1) continue;
      const bool both = (u / a.n_kv) * kPRows + 128 < R;
      auto take = [&] {  // tile 0 has the first turn
        return !both || wait_all(bars.turn[w], (uint32_t)(tn++ & 1) ^ (w == 0 ? 1u : 0u));
      };
      auto pass = [&] {
        if (both && lane == 0) mbar_arrive(bar(bars.turn[1 - w]));
        __syncwarp();
      };
      if (w == 1 && !both) {
        // no such tile in the last pair: its stages go back as they come
        for (int j = 0; ok && j < cnt; ++j, ++n) {
          ok = wait_all(bars.k_full[n & 1], (uint32_t)(n >> 1) & 1u);
          if (ok && lane == 0) mbar_arrive(b_k_empty + 8 * (n & 1));
          ok = ok && wait_all(bars.v_full[n & 1], (uint32_t)(n >> 1) & 1u);
          if (ok && lane == 0) mbar_arrive(b_v_empty + 8 * (n & 1));
          __syncwarp();
        }
        continue;
      }
      ok = wait_all(bars.q_ready[w], qn++ & 1u) &&
           wait_all(bars.k_full[n & 1], (uint32_t)(n >> 1) & 1u) && take();
      if (!ok) break;
      tc_fence_after();
      qk(n & 1);
      pass();
      for (int j = 0; ok && j < cnt; ++j, ++n) {
        const int nx = n + 1;
        ok = wait_all(bars.v_full[n & 1], (uint32_t)(n >> 1) & 1u) &&
             (j + 1 == cnt || wait_all(bars.k_full[nx & 1], (uint32_t)(nx >> 1) & 1u)) &&
             wait_all(bars.p_ready[w], pn++ & 1u) && take();
        if (!ok) break;
        tc_fence_after();
        pv(n & 1, j == 0);
        if (j + 1 < cnt) qk(nx & 1);
        pass();
      }
    }
    // every product has finished before TMEM and shared memory go (bounded)
    if (elect_one()) {
      volatile int never = 0;
      mma_commit(bar(bars.drain[w]));
      mbar_wait(bar(bars.drain[w]), 0, &never);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int w = (warp - 4) >> 3;         // row tile
    const int hf = ((warp - 4) >> 2) & 1;  // half of the step's positions, of O's columns
    const int quarter = warp & 3;          // TMEM lanes 32 quarter ..
    const int r = quarter * 32 + lane;     // row in the tile
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + kS + w * 128 + lanes;
    const uint32_t tO = tmem + kO + w * 128 + hf * (D / 2) + lanes;
    const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(D)
    const uint64_t sl22 = pair2(__float_as_uint(sl2), __float_as_uint(sl2));
    // the two warps that share 32 rows; after a wait that ran out the loops go
    // on to their end over what is there, so that both keep meeting
    auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + w * 4 + quarter) : "memory"); };
    int n = 0;  // this tile's steps so far
    for (int f = f0; f < f1;) {
      const int u = f / plen, j0 = f - u * plen, g = u % a.n_kv;
      const int cnt = min(steps - j0, f1 - f);
      f = cnt < 1 || j0 + cnt == steps ? (u + 1) * plen : f + cnt;
      if (cnt < 1) continue;
      const int row0 = (u / a.n_kv) * kPRows + w * 128;
      if (row0 >= R) continue;  // the last tile pair has one tile only
      // ---- this row: its last position, its query's place
      const int row = row0 + r;
      int lim = -1;
      {
        int64_t src = -1;
        if (row < R) {
          const int tok = row / G, hh = row - tok * G;
          int s = 0;  // the last slot with s_tok <= tok: the one that holds it
          for (int step = 1 << (31 - __clz(a.n_slots)); step; step >>= 1)
            if (s + step < a.n_slots && s_tok[s + step] <= tok) s += step;
          const int t = tok - s_tok[s];
          const SlotSpan sp = slot_span(a, s);
          lim = sp.len - sp.n_new + t;
          if (lim >= 0) src = ((int64_t)s * a.T + t) * a.q_stride + (g * G + hh) * D;
        }
        // The warp's 32 half rows into shared memory, whole lines at a time
        // (a row a lane asks for 32 lines at once, 4700 clocks instead of 1400).
        constexpr int kL = D / 16;  // lanes a half row
        const int c = hf * kL + lane % kL;
#pragma unroll 4
        for (int i = 0; i < kL; ++i) {
          const int rw = i * (32 / kL) + lane / kL;
          const int64_t at = __shfl_sync(0xFFFFFFFFu, src, rw);
          cp_async16(sq + w * kTile + (c >> 3) * kHalf + (quarter * 32 + rw) * 128 + (((c & 7) ^ (rw & 7)) << 4),
                     a.q + (at >= 0 ? at : 0) + c * 8, at >= 0 ? 16 : 0);  // 0: zeros
        }
        cp_async_wait();
      }
      fence_proxy_async_smem();  // the tensor core reads it
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.q_ready[w]));
      float ref = -INFINITY, l = 0.0f;
      for (int j = j0; j < j0 + cnt; ++j, ++n) {
        // what of its half of the step this row sees
        const int jb = 2 * j + hf;
        const int page = jb < a.prefix_blocks ? __ldg(a.prefix + jb) : -1;
        const bool bad = page < 0 || page >= a.n_phys;
        const int left = bad ? -1 : lim - jb * kBlk;  // last position that is seen
        const bool plain = !__any_sync(0xFFFFFFFFu, left < kBlk - 1);
        wait(bars.s_full[w], (uint32_t)n & 1u);
        tc_fence_after();
        uint32_t x[kBlk];
        tmem_ld32(tS + hf * 64, x);
        tmem_ld32(tS + hf * 64 + 32, x + 32);
        tmem_wait_ld();
        if (!plain) {
#pragma unroll
          for (int c = 0; c < kBlk; ++c)
            if (c > left) x[c] = 0xFF800000u;  // -inf
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kBlk; c += 4) {
          mx[0] = max3(mx[0], x[c], x[c + 1]);
          mx[1] = max3(mx[1], x[c + 2], x[c + 3]);
        }
        mx[0] = fmaxf(mx[0], mx[1]);
        s_mx[n & 1][w][hf][r] = mx[0];
        meet();  // both halves have read S, too: P may overwrite it
        const float top = fmaxf(mx[0], s_mx[n & 1][w][hf ^ 1][r]) * sl2;
        if (j == j0) {
          ref = top;
        } else {
          const bool grow = top > ref + kSlack;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            // O of the steps before is complete, the next product waits for us
            wait(bars.pv_done[w], (uint32_t)(n - 1) & 1u);
            tc_fence_after();
            const float now = grow ? top : ref;
            const float fac = grow ? ex2(ref - now) : 1.0f;  // 0 where nothing was seen yet
            ref = now;
            l *= fac;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t y[16];
              tmem_ld16r(tO + c, y);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * fac);
              tmem_st16(tO + c, y);
            }
            tmem_wait_st();
          }
        }
        const float off = lift<F16>() - (ref == -INFINITY ? 0.0f : ref);
        const uint64_t off2 = pair2(__float_as_uint(off), __float_as_uint(off));
        uint64_t sum[2] = {0, 0};  // four sums
#pragma unroll
        for (int c = 0; c < kBlk; c += 2) {
          float e0, e1;
          unpair2(fma2(pair2(x[c], x[c + 1]), sl22, off2), e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pair2(__float_as_uint(e0), __float_as_uint(e1)));
          x[c >> 1] = pack2<F16>(e0, e1);
        }
        tmem_st32(tS + hf * 32, x);
        float t0, t1;
        unpair2(add2(sum[0], sum[1]), t0, t1);
        l += t0 + t1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bars.p_ready[w]));
      }
      // ---- the stretch's (m, l, O), rows fastest
      s_mx[n & 1][w][hf][r] = l;
      meet();
      float* part = a.px_part + (int64_t)((int)blockIdx.x + u) * kPRows * (D + 2);
      if (hf == 0) {
        part[w * 128 + r] = ref;
        part[kPRows + w * 128 + r] = l + s_mx[n & 1][w][1][r];
      }
      meet();  // read before the next stretch's maxima
      wait(bars.pv_done[w], (uint32_t)(n - 1) & 1u);
      tc_fence_after();
      float4* po = reinterpret_cast<float4*>(part + 2 * kPRows) + (hf * (D / 8)) * kPRows + w * 128 + r;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t y[32];
        tmem_ld32(tO + c, y);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          po[(int64_t)((c + k) / 4) * kPRows] =
              make_float4(__uint_as_float(y[k]), __uint_as_float(y[k + 1]),
                          __uint_as_float(y[k + 2]), __uint_as_float(y[k + 3]));
      }
      tc_fence_before();  // read before the next stretch's products write it
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

namespace {
template <bool F16, int D>
cudaError_t launch_px(const CUtensorMap& tk, const CUtensorMap& tv, const AttnBatchArgs& a, int grid,
                      cudaStream_t stream) {
  const size_t smem = 1024 + (size_t)(2 + 2 * kPStages) * 128 * D * 2 + (size_t)a.n_slots * 4;
  const cudaError_t e = cudaFuncSetAttribute(attn_prefix_kernel<F16, D>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_prefix_kernel<F16, D>, dim3(grid), dim3(kPThr), smem, stream, tk, tv, a);
}
}  // namespace

// the most that there can be: every slot with T tokens
PrefixLine prefix_line(const moe_attn_batch_shape_t* s, int sms) {
  const int64_t rows = (int64_t)s->n_slots * s->T * (s->n_q / s->n_kv);
  return prefix_cut((int)((rows + kPRows - 1) / kPRows) * s->n_kv, (s->prefix_blocks + 1) / 2, sms);
}
// one place per stretch: CTA + pair, both of which grow along the line
size_t prefix_part_floats(const moe_attn_batch_shape_t* s, int sms) {
  return (size_t)(sms + prefix_line(s, sms).pairs) * kPRows * (s->D + 2);
}

cudaError_t launch_attn_prefix(const moe_attn_batch_shape_t* s, const CUtensorMap& tk,
                               const CUtensorMap& tv, const AttnBatchArgs& a, int grid,
                               cudaStream_t stream) {
  if (s->dtype == MOE_DTYPE_FP16)
    return s->D == 64 ? launch_px<true, 64>(tk, tv, a, grid, stream)
                      : launch_px<true, 128>(tk, tv, a, grid, stream);
  return s->D == 64 ? launch_px<false, 64>(tk, tv, a, grid, stream)
                    : launch_px<false, 128>(tk, tv, a, grid, stream);
}

}  // namespace moe

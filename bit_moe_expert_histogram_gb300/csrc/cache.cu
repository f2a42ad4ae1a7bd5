// The pages of a block-paged key/value cache: fork (with reorder, cut and
// free), reserve (with copy-on-write), write, compact and copy.
//
// State: table [n_slots][max_blocks] (page of each 64-position block of a
// slot), lens [n_slots], refs [n_phys] (table entries that hold the page; 0 =
// free). Slot s holds the first ceil(lens[s] / 64) entries of its row. The
// pools (keys and values of every layer) share the page numbers, so one
// decision moves data in all of them.
//
// Everything is decided on the device, from the state as it was before the
// call, by rules that have one answer whatever order threads run in: counts
// change by integer atomics (any order gives the same sum), free pages are
// taken lowest first in slot order through prefix sums, and the result goes
// to a second state (the first stays whole: nothing is read after it was
// changed, and a caller can drop the result). Copies read only pages that
// are held and write only pages that are free, so none of them overlap.
//
// Bound: the copies by HBM (each byte once in, once out); fork and reserve by
// launch and L2 latency. A small state is one CTA's work, one launch; a large
// one takes two and three short kernels chained by programmatic dependent
// launch. (One cooperative launch whose CTAs meet in the workspace takes the
// host 1.3 us less than two, but the GPU 6.4 us instead of 4.1 for 1000 slots
// and 4.5 instead of 2.9 for 16.) Fork of 16 and of 1000 slots: 2.6 and 4.1 us
// in a graph, 5.3 and 6.9 from the host; 1740 pages of 4 pools of 8192 brought
// together: 75.3 us, 6.05 TB/s, 0.89 of a plain copy's rate.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {
constexpr int kPage = 64;         // positions per page
constexpr int kOneCta = 1024;     // threads of a CTA that plans alone
constexpr int kRankChunk = 1024;  // pages per CTA of the compaction's count and rank

__device__ __forceinline__ int blocks_of(int len) { return (len + kPage - 1) / kPage; }
// a slot's length, brought into what its row can hold
__device__ __forceinline__ int len_of(const int32_t* lens, int s, int max_blocks, Ctrl* ctrl) {
  const int l = __ldg(lens + s);
  const int most = max_blocks * kPage;
  if (l < 0 || l > most) {
    set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    return l < 0 ? 0 : most;
  }
  return l;
}

// inclusive scan of one int per thread over a CTA of up to 32 warps
__device__ __forceinline__ int block_scan_i(int v, int* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int t = lane < nw ? warp_tot[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
      if (lane >= d) t += o;
    }
    warp_tot[lane] = t;
  }
  __syncthreads();
  return v + (warp ? warp_tot[warp - 1] : 0);
}
}  // namespace

// ------------------------------------------------------------------ fork --
__global__ void __launch_bounds__(256)
    cache_copy_refs_kernel(const int32_t* __restrict__ in, int32_t* __restrict__ out, int n) {
  pdl_wait();
  pdl_trigger();
  const int i0 = blockIdx.x * 1024 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i0 + k * 256 < n) out[i0 + k * 256] = __ldg(in + i0 + k * 256);
}

// `per` threads per slot (a warp or four): the row of its parent cut to the new
// length, and the difference in the pages' counts (none where a page stays in
// its place). refs: the counts are not in the new state yet, and this CTA is
// the only one.
__global__ void __launch_bounds__(kOneCta)
    cache_fork_kernel(const moe_cache_meta_t in, const moe_cache_meta_t out,
                      const int32_t* __restrict__ parent, const int32_t* __restrict__ keep,
                      int n_slots, int max_blocks, int n_phys, int per, bool refs, Ctrl* ctrl) {
  pdl_wait();
  pdl_trigger();
  if (refs) {
    for (int i = threadIdx.x; i < n_phys; i += blockDim.x) out.refs_dev[i] = __ldg(in.refs_dev + i);
    __syncthreads();
  }
  const int j0 = threadIdx.x & (per - 1), slots = blockDim.x / per;
  for (int s = blockIdx.x * slots + threadIdx.x / per; s < n_slots; s += gridDim.x * slots) {
    const int a = __ldg(parent + s);
    const bool live = a >= 0 && a < n_slots;
    if (j0 == 0 && (a >= n_slots || a < -1)) set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    int len = 0;
    if (live) {
      len = len_of(in.lens_dev, a, max_blocks, ctrl);
      if (keep) len = min(len, max(0, __ldg(keep + s)));
    }
    const int nb_old = blocks_of(len_of(in.lens_dev, s, max_blocks, ctrl)), nb_new = blocks_of(len);
    const int32_t* row_old = in.table_dev + (int64_t)s * max_blocks;
    const int32_t* row_new = in.table_dev + (int64_t)(live ? a : s) * max_blocks;
    int32_t* row = out.table_dev + (int64_t)s * max_blocks;
    for (int j = j0; j < max_blocks; j += per) {
      int po = j < nb_old ? __ldg(row_old + j) : -1, pn = j < nb_new ? __ldg(row_new + j) : -1;
      if ((j < nb_old && (po < 0 || po >= n_phys)) || (j < nb_new && (pn < 0 || pn >= n_phys)))
        set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
      if (po < 0 || po >= n_phys) po = -1;
      if (pn < 0 || pn >= n_phys) pn = -1;
      row[j] = pn;
      if (po != pn) {
        if (pn >= 0) atomicAdd(out.refs_dev + pn, 1);
        if (po >= 0) atomicAdd(out.refs_dev + po, -1);
      }
    }
    if (j0 == 0) out.lens_dev[s] = len;
  }
}

// ---------------------------------------------------------------- copies --
// The first `rows` rows of every head of a page to another; row_u4: 16-byte
// words of a row, D * 2 / 16.
__device__ __forceinline__ void copy_page(const uint4* __restrict__ from, uint4* __restrict__ to,
                                          int n_kv, int rows, int row_u4) {
  const int per = rows * row_u4, page = kPage * row_u4;
  for (int h = 0; h < n_kv; ++h) {
    const uint4* f = from + (int64_t)h * page;
    uint4* t = to + (int64_t)h * page;
    for (int i0 = threadIdx.x; i0 < per; i0 += 256 * 4) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * 256 < per) v[k] = __ldcs(f + i0 + k * 256);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * 256 < per) __stcs(t + i0 + k * 256, v[k]);
    }
  }
}

// The listed copies, (source, destination, rows) each, in every pool: chunk q
// of head h of pool k of copy c, 4 KB a warp at a time, all of it in flight.
__device__ __forceinline__ void copy_list(const CachePools& pools, const int32_t* list, int copies,
                                          int n_kv, int row_u4) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int head = kPage * row_u4, chunks = (head + 255) / 256;
  // at most 4096 copies in 128 pools of 64 heads of 16 chunks: 32 bits
  const unsigned n = (unsigned)copies * pools.n * n_kv * chunks;
  for (unsigned w = blockIdx.x * warps + (threadIdx.x >> 5); w < n; w += gridDim.x * warps) {
    const unsigned hk = w / chunks, kc = hk / n_kv;
    const int q = w - hk * chunks, h = hk - kc * n_kv, c = kc / pools.n, k = kc - c * pools.n;
    const int32_t* it = list + 3 * c;
    const int end = min(__ldcg(it + 2) * row_u4, q * 256 + 256);
    uint4* pool = static_cast<uint4*>(pools.p[k]);
    const uint4* from = pool + ((int64_t)__ldcg(it) * n_kv + h) * head;
    uint4* to = pool + ((int64_t)__ldcg(it + 1) * n_kv + h) * head;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = q * 256 + i * 32 + lane;
      if (at < end) v[i] = __ldcs(from + at);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = q * 256 + i * 32 + lane;
      if (at < end) __stcs(to + at, v[i]);
    }
  }
}
__global__ void __launch_bounds__(256)
    cache_copy_list_kernel(const __grid_constant__ CachePools pools, const int32_t* list,
                           const int32_t* n_copies, int n_kv, int row_u4) {
  pdl_wait();
  pdl_trigger();
  copy_list(pools, list, __ldg(n_copies), n_kv, row_u4);
}

// --------------------------------------------------------------- reserve --
// Table and refs into the new state, rows s0, s0 + n, .. and pages likewise by
// CTA; a row's entries past its slot's blocks become -1.
__device__ __forceinline__ void bring_state(const moe_cache_meta_t& in, const moe_cache_meta_t& out,
                                            int n_slots, int max_blocks, int n_phys, Ctrl* ctrl) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_phys; i += gridDim.x * blockDim.x)
    out.refs_dev[i] = __ldg(in.refs_dev + i);
  for (int s = blockIdx.x * warps + (threadIdx.x >> 5); s < n_slots; s += gridDim.x * warps) {
    const int nb = blocks_of(len_of(in.lens_dev, s, max_blocks, ctrl));
    const int64_t r0 = (int64_t)s * max_blocks;
#pragma unroll 4
    for (int j = lane; j < max_blocks; j += 32)
      out.table_dev[r0 + j] = j < nb ? __ldg(in.table_dev + r0 + j) : -1;
  }
}
__global__ void __launch_bounds__(256)
    cache_state_kernel(const moe_cache_meta_t in, const moe_cache_meta_t out, int n_slots,
                       int max_blocks, int n_phys, Ctrl* ctrl) {
  pdl_wait();
  pdl_trigger();
  bring_state(in, out, n_slots, max_blocks, n_phys, ctrl);
}

// One CTA. The slots' needs and their running sum, the lowest free pages, as
// many as are needed; then each granted slot's entries, counts and page copy.
// all: the state is not in `out` yet, and no kernel for the copies follows.
__global__ void __launch_bounds__(kOneCta)
    cache_reserve_kernel(const __grid_constant__ CachePools pools, const moe_cache_meta_t in,
                         const moe_cache_meta_t out, const int32_t* __restrict__ n_new,
                         int32_t* __restrict__ granted, int n_slots, int max_blocks, int n_phys,
                         int n_kv, int row_u4, bool all, int32_t* before, int32_t* free_page,
                         int32_t* list, int32_t* n_copies, Ctrl* ctrl) {
  __shared__ int s_tot[32];
  __shared__ int s_sum;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (all) bring_state(in, out, n_slots, max_blocks, n_phys, ctrl);
  // what slot s asks for: its length, the new positions, its blocks, the
  // page to copy (-1: none); returns the pages that this takes. A request
  // that is wider than the row counts in full here, so that the slots after
  // it see the same running sum either way.
  auto ask = [&](int s, int& len, int& n, int& nb0, int& cow) {
    len = len_of(in.lens_dev, s, max_blocks, ctrl);
    n = __ldg(n_new + s);
    nb0 = blocks_of(len);
    cow = -1;
    if (n < 0) set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    if (n <= 0) {
      n = 0;
      return 0;
    }
    if (len % kPage) {
      const int last = __ldg(in.table_dev + (int64_t)s * max_blocks + nb0 - 1);
      if (last < 0 || last >= n_phys) {
        set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
        n = 0;  // no page to write to: nothing is granted
        return 0;
      }
      if (__ldg(in.refs_dev + last) > 1) cow = last;
    }
    const int64_t more = ((int64_t)len + n + kPage - 1) / kPage - nb0;
    return (int)min(more, (int64_t)1 << 20) + (cow >= 0 ? 1 : 0);
  };
  // running sum of the needs, in slot order, kept below 2^30
  int sum = 0;
  for (int s0 = 0; s0 < n_slots; s0 += kOneCta) {
    const int s = s0 + tid;
    int len, n, nb0, cow;
    const int need = s < n_slots ? ask(s, len, n, nb0, cow) : 0;
    const int incl = block_scan_i(need, s_tot);  // below 2^31: a need is at most 2^20 + 1
    if (s < n_slots) before[s] = (int)min((int64_t)sum + incl - need, (int64_t)1 << 30);
    if (tid == kOneCta - 1) s_sum = incl;
    __syncthreads();
    sum = (int)min((int64_t)sum + s_sum, (int64_t)1 << 30);
    __syncthreads();
  }
  // the lowest `sum` free pages (or all there are), in order
  int found = 0;
  for (int p0 = 0; p0 < n_phys && found < sum; p0 += kOneCta * 4) {
    int f[4], c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + tid * 4 + k;
      f[k] = p < n_phys && __ldg(in.refs_dev + p) == 0;
      c += f[k];
    }
    const int incl = block_scan_i(c, s_tot);
    int at = found + incl - c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) free_page[at++] = p0 + tid * 4 + k;
    if (tid == kOneCta - 1) s_sum = incl;
    __syncthreads();
    found += s_sum;
    __syncthreads();
  }
  // each slot's pages
  int copies = 0;
  for (int s0 = 0; s0 < n_slots; s0 += kOneCta) {
    const int s = s0 + tid;
    int len = 0, n = 0, nb0 = 0, cow = -1, at = 0;
    if (s < n_slots) {
      const int need = ask(s, len, n, nb0, cow);
      at = before[s];
      const int more = need - (cow >= 0 ? 1 : 0);
      if (need > 0 && (at + need > found || nb0 + more > max_blocks)) {
        n = 0;  // refused: the slot stays as it was
        cow = -1;
      }
      granted[s] = n;
      out.lens_dev[s] = len + n;
      int32_t* row = out.table_dev + (int64_t)s * max_blocks;
      int from = at;
      if (cow >= 0) {
        row[nb0 - 1] = free_page[from];
        atomicAdd(out.refs_dev + free_page[from], 1);
        atomicAdd(out.refs_dev + cow, -1);
        ++from;
      }
      for (int k = 0; n > 0 && k < more; ++k) {
        row[nb0 + k] = free_page[from + k];
        atomicAdd(out.refs_dev + free_page[from + k], 1);
      }
    }
    const int incl = block_scan_i(cow >= 0 ? 1 : 0, s_tot);
    if (cow >= 0) {
      int32_t* it = list + 3 * (copies + incl - 1);
      it[0] = cow;
      it[1] = free_page[at];
      it[2] = len % kPage;
    }
    if (tid == kOneCta - 1) s_sum = incl;
    __syncthreads();
    copies += s_sum;
    __syncthreads();
  }
  if (tid == 0) *n_copies = copies;
  if (all) copy_list(pools, list, copies, n_kv, row_u4);  // the list is complete: a scan ended it
}

// Whole pages from one set of pools to another by two caller-given lists.
__global__ void __launch_bounds__(256)
    cache_copy_pages_kernel(const __grid_constant__ CachePools from,
                            const __grid_constant__ CachePools to, const int32_t* __restrict__ src,
                            const int32_t* __restrict__ dst, int n, int n_from, int n_to, int n_kv,
                            int row_u4, Ctrl* ctrl) {
  pdl_wait();
  pdl_trigger();
  const int64_t page = (int64_t)n_kv * kPage * row_u4;
  for (int64_t w = blockIdx.x; w < (int64_t)n * from.n; w += gridDim.x) {
    const int c = (int)(w / from.n), k = (int)(w - (int64_t)c * from.n);
    const int a = __ldg(src + c), b = __ldg(dst + c);
    if (a < 0 || a >= n_from || b < 0 || b >= n_to) {
      if (threadIdx.x == 0) set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, c);
      continue;
    }
    copy_page(static_cast<const uint4*>(from.p[k]) + a * page,
              static_cast<uint4*>(to.p[k]) + b * page, n_kv, kPage, row_u4);
  }
}

// ----------------------------------------------------------------- write --
// One warp per (slot, token, key or value): a token's n_kv rows of D.
__global__ void __launch_bounds__(256)
    cache_write_kernel(const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                       const int32_t* __restrict__ n_new, const uint16_t* __restrict__ k_new,
                       int64_t k_stride, const uint16_t* __restrict__ v_new, int64_t v_stride,
                       uint4* __restrict__ k_cache, uint4* __restrict__ v_cache, int n_slots, int T,
                       int max_blocks, int n_phys, int n_kv, int row_u4, Ctrl* ctrl) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t tok = w >> 1;
  if (tok >= (int64_t)n_slots * T) return;
  const int s = (int)(tok / T), t = (int)(tok - (int64_t)s * T);
  const int n = n_new ? __ldg(n_new + s) : T;
  const int len = __ldg(lens + s);
  if (n < 0 || n > T || len < n || len > max_blocks * kPage) {
    if (lane == 0) set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    return;
  }
  if (t >= n) return;
  const int pos = len - n + t;
  const int page = __ldg(table + (int64_t)s * max_blocks + pos / kPage);
  if (page < 0 || page >= n_phys) {
    if (lane == 0) set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
    return;
  }
  const uint4* from = reinterpret_cast<const uint4*>((w & 1) ? v_new + tok * v_stride
                                                             : k_new + tok * k_stride);
  uint4* to = ((w & 1) ? v_cache : k_cache) + ((int64_t)page * n_kv * kPage + pos % kPage) * row_u4;
  for (int i = lane; i < n_kv * row_u4; i += 32)
    to[(int64_t)(i / row_u4) * kPage * row_u4 + i % row_u4] = __ldg(from + i);
}

// --------------------------------------------------------------- compact --
__global__ void __launch_bounds__(kRankChunk)
    cache_count_kernel(const int32_t* __restrict__ refs, int n_phys, int32_t* __restrict__ counts) {
  pdl_wait();
  pdl_trigger();
  const int p = blockIdx.x * kRankChunk + threadIdx.x;
  const int n = __syncthreads_count(p < n_phys && __ldg(refs + p) != 0);
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// L = live pages in all, B = live pages below L. A live page at or past L is
// the (live before it - B)-th to move; a free one below L the (free before
// it)-th to fill. rank[] holds that number for both; src / dst the pages.
__global__ void __launch_bounds__(kRankChunk)
    cache_rank_kernel(const int32_t* __restrict__ refs, int n_phys,
                      const int32_t* __restrict__ counts, int n_chunks, int32_t* __restrict__ rank,
                      int32_t* __restrict__ src, int32_t* __restrict__ dst,
                      int32_t* __restrict__ n_live, int32_t* __restrict__ n_moves) {
  __shared__ int s_tot[32];
  __shared__ int s_all, s_before, s_upto;
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  // n_chunks <= 1024: a chunk a thread
  const int c = tid < n_chunks ? __ldg(counts + tid) : 0;
  const int incl = block_scan_i(c, s_tot);
  if (tid == kRankChunk - 1) s_all = incl;
  if (tid == (int)blockIdx.x) s_before = incl - c;
  __syncthreads();
  const int L = s_all;
  // live pages below L: the chunks before the one that L falls into, and that
  // one's own up to L (a pool of 2^20 held pages has no such chunk)
  const int cl = L / kRankChunk;
  if (tid == cl) s_upto = incl - c;
  const int pl = cl * kRankChunk + tid;
  const int below = __syncthreads_count(pl < L && pl < n_phys && __ldg(refs + pl) != 0);
  const int B = cl >= kRankChunk ? L : s_upto + below;
  const int p = blockIdx.x * kRankChunk + tid;
  const int live = p < n_phys && __ldg(refs + p) != 0;
  const int before = s_before + block_scan_i(live, s_tot) - live;
  if (p < n_phys) {
    if (live && p >= L) {
      src[before - B] = p;
      rank[p] = before - B;
    } else if (!live && p < L) {
      dst[p - before] = p;
      rank[p] = p - before;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    *n_live = L;
    *n_moves = L - B;
  }
}

// The moves in every pool, the tables and the counts, and where each page went
// (moved, or null). The first meta_ctas CTAs take the state, the others the
// pages.
__global__ void __launch_bounds__(256)
    cache_move_kernel(const __grid_constant__ CachePools pools, const moe_cache_meta_t in,
                      const moe_cache_meta_t out, int n_slots, int max_blocks, int n_phys, int n_kv,
                      int row_u4, const int32_t* __restrict__ rank, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, const int32_t* __restrict__ n_live,
                      const int32_t* __restrict__ n_moves, int32_t* __restrict__ moved,
                      int meta_ctas, Ctrl* ctrl) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= meta_ctas) {
    const int64_t n = (int64_t)__ldg(n_moves) * pools.n;
    const int64_t page = (int64_t)n_kv * kPage * row_u4;
    for (int64_t w = (int)blockIdx.x - meta_ctas; w < n; w += (int)gridDim.x - meta_ctas) {
      const int m = (int)(w / pools.n), k = (int)(w - (int64_t)m * pools.n);
      uint4* pool = static_cast<uint4*>(pools.p[k]);
      copy_page(pool + __ldg(src + m) * page, pool + __ldg(dst + m) * page, n_kv, kPage, row_u4);
    }
    return;
  }
  const int L = __ldg(n_live);
  for (int s = blockIdx.x; s < n_slots; s += meta_ctas) {
    const int len = len_of(in.lens_dev, s, max_blocks, ctrl), nb = blocks_of(len);
    const int64_t r0 = (int64_t)s * max_blocks;
    for (int j = threadIdx.x; j < max_blocks; j += 256) {
      int p = -1;
      if (j < nb) {
        p = __ldg(in.table_dev + r0 + j);
        if (p < 0 || p >= n_phys || __ldg(in.refs_dev + p) == 0) {
          set_error(ctrl, MOE_ERR_BAD_INPUT, KID_CACHE, s);
          p = -1;
        } else if (p >= L) {
          p = __ldg(dst + __ldg(rank + p));
        }
      }
      out.table_dev[r0 + j] = p;
    }
    if (threadIdx.x == 0) out.lens_dev[s] = len;
  }
  for (int p = blockIdx.x * 256 + threadIdx.x; p < n_phys; p += meta_ctas * 256) {
    int r = 0;
    if (p < L) {
      r = __ldg(in.refs_dev + p);
      if (r == 0) r = __ldg(in.refs_dev + __ldg(src + __ldg(rank + p)));
    }
    out.refs_dev[p] = r;
    if (moved)
      moved[p] = __ldg(in.refs_dev + p) == 0 ? -1 : p < L ? p : __ldg(dst + __ldg(rank + p));
  }
}

// ------------------------------------------------------------------ host --
bool cache_supported(const moe_cache_shape_t* s) {
  if (!s) return false;
  if (s->n_slots < 1 || s->n_slots > 4096 || s->max_blocks < 1 || s->max_blocks > (1 << 18))
    return false;
  if (s->n_phys < 1 || s->n_phys > (1 << 20) || s->n_kv < 1 || s->n_kv > 64) return false;
  return s->D >= 8 && s->D <= 512 && s->D % 8 == 0 && s->block == kPage;
}

namespace {
struct CacheWs {
  size_t before, free_page, count, item, counts, rank, src, dst, moves, total;
};
CacheWs cache_ws(const moe_cache_shape_t* s) {
  CacheWs w{};
  size_t off = 256;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += (n * 4 + 255) & ~(size_t)255;
    return o;
  };
  w.before = take(s->n_slots);
  w.free_page = take(s->n_phys);
  w.count = take(1);
  w.item = take((size_t)s->n_slots * 3);
  w.counts = take(kRankChunk);
  w.rank = take(s->n_phys);
  w.src = take(s->n_phys);
  w.dst = take(s->n_phys);
  w.moves = take(1);
  w.total = off;
  return w;
}
int32_t* at(uint8_t* ws, size_t off) { return reinterpret_cast<int32_t*>(ws + off); }
int ceil_div(int64_t n, int d) { return (int)((n + d - 1) / d); }
// CTAs of a copy: a page of a pool each, eight CTAs of 256 threads an SM
int copy_ctas(int64_t pages, int nsm) { return (int)(pages < nsm * 8 ? pages : nsm * 8); }
}  // namespace

size_t cache_ws_bytes(const moe_cache_shape_t* s) { return cache_ws(s).total; }

// Few enough that one CTA, with four warps or one for a row, is done in the
// time of a launch: 2.6 us for a round or two of 32 rows x 32 entries, 4.7 for
// three, against 3.3 of a CTA a slot after a launch for the counts (one CTA
// that was given 461 slots took 40 us).
namespace {
int row_threads(const moe_cache_shape_t* s) { return s->n_slots <= kOneCta / 128 ? 128 : 32; }
bool small_fork(const moe_cache_shape_t* s) {
  const int per = row_threads(s);
  return (int64_t)ceil_div(s->n_slots, kOneCta / per) * ceil_div(s->max_blocks, per) <= 2 &&
         s->n_phys <= 8192;
}
}  // namespace

cudaError_t launch_cache_fork(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                              const moe_cache_meta_t& out, const int32_t* parent,
                              const int32_t* keep, uint8_t* ws, cudaStream_t stream) {
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(ws);
  if (small_fork(s))
    return launch_pdl(cache_fork_kernel, dim3(1), dim3(kOneCta), 0, stream, in, out, parent, keep,
                      s->n_slots, s->max_blocks, s->n_phys, row_threads(s), true, ctrl);
  const cudaError_t e = launch_pdl(cache_copy_refs_kernel, dim3(ceil_div(s->n_phys, 1024)),
                                   dim3(256), 0, stream, in.refs_dev, out.refs_dev, s->n_phys);
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_fork_kernel, dim3(s->n_slots), dim3(128), 0, stream, in, out, parent,
                    keep, s->n_slots, s->max_blocks, s->n_phys, 128, false, ctrl);
}

cudaError_t launch_cache_reserve(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                                 const moe_cache_meta_t& out, const int32_t* n_new,
                                 int32_t* granted, const CachePools& pools, uint8_t* ws, int nsm,
                                 cudaStream_t stream) {
  const CacheWs w = cache_ws(s);
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(ws);
  // one CTA brings a small state over, 4096 words at a time, and copies a few
  // pages, should every slot need it, in a few microseconds
  const int64_t copies = (int64_t)s->n_slots * pools.n;
  const bool all = (int64_t)s->n_slots * s->max_blocks + s->n_phys <= 16384 && copies * s->n_kv * s->D <= 8192;
  if (!all) {
    const int ctas = ceil_div((int64_t)s->n_slots * s->max_blocks + s->n_phys, 2048);
    const cudaError_t e =
        launch_pdl(cache_state_kernel, dim3(ctas < 8 * nsm ? ctas : 8 * nsm), dim3(256), 0, stream,
                   in, out, s->n_slots, s->max_blocks, s->n_phys, ctrl);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_pdl(
      cache_reserve_kernel, dim3(1), dim3(kOneCta), 0, stream, pools, in, out, n_new, granted,
      s->n_slots, s->max_blocks, s->n_phys, s->n_kv, s->D / 8, all, at(ws, w.before),
      at(ws, w.free_page), at(ws, w.item), at(ws, w.count), ctrl);
  if (e != cudaSuccess || all || pools.n == 0) return e;
  return launch_pdl(cache_copy_list_kernel, dim3(copy_ctas(copies, nsm)), dim3(256), 0, stream,
                    pools, at(ws, w.item), at(ws, w.count), s->n_kv, s->D / 8);
}

cudaError_t launch_cache_write(const moe_cache_shape_t* s, const moe_cache_meta_t& meta,
                               const int32_t* n_new, int T, const uint16_t* k_new,
                               int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                               void* k_cache, void* v_cache, uint8_t* ws, cudaStream_t stream) {
  return launch_pdl(cache_write_kernel, dim3(ceil_div((int64_t)s->n_slots * T * 2, 8)), dim3(256),
                    0, stream, meta.table_dev, meta.lens_dev, n_new, k_new, k_stride, v_new,
                    v_stride, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache),
                    s->n_slots, T, s->max_blocks, s->n_phys, s->n_kv, s->D / 8,
                    reinterpret_cast<Ctrl*>(ws));
}

cudaError_t launch_cache_compact(const moe_cache_shape_t* s, const moe_cache_meta_t& in,
                                 const moe_cache_meta_t& out, int32_t* n_live, int32_t* moved,
                                 const CachePools& pools, uint8_t* ws, int nsm,
                                 cudaStream_t stream) {
  const CacheWs w = cache_ws(s);
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(ws);
  const int chunks = ceil_div(s->n_phys, kRankChunk);
  cudaError_t e = launch_pdl(cache_count_kernel, dim3(chunks), dim3(kRankChunk), 0, stream,
                             in.refs_dev, s->n_phys, at(ws, w.counts));
  if (e != cudaSuccess) return e;
  e = launch_pdl(cache_rank_kernel, dim3(chunks), dim3(kRankChunk), 0, stream, in.refs_dev,
                 s->n_phys, at(ws, w.counts), chunks, at(ws, w.rank), at(ws, w.src),
                 at(ws, w.dst), n_live, at(ws, w.moves));
  if (e != cudaSuccess) return e;
  const int meta = s->n_slots < nsm ? s->n_slots : nsm;
  // at most half the pages move
  const int ctas = copy_ctas((int64_t)(s->n_phys / 2) * pools.n, nsm);
  return launch_pdl(cache_move_kernel, dim3(meta + ctas), dim3(256), 0, stream, pools, in, out,
                    s->n_slots, s->max_blocks, s->n_phys, s->n_kv, s->D / 8, at(ws, w.rank),
                    at(ws, w.src), at(ws, w.dst), n_live, at(ws, w.moves), moved, meta, ctrl);
}

cudaError_t launch_cache_copy_pages(const moe_cache_shape_t* s, int n, const int32_t* src,
                                    const int32_t* dst, const CachePools& from,
                                    const CachePools& to, int n_to, uint8_t* ws, int nsm,
                                    cudaStream_t stream) {
  return launch_pdl(cache_copy_pages_kernel, dim3(copy_ctas((int64_t)n * from.n, nsm)), dim3(256),
                    0, stream, from, to, src, dst, n, s->n_phys, n_to, s->n_kv, s->D / 8,
                    reinterpret_cast<Ctrl*>(ws));
}

}  // namespace moe

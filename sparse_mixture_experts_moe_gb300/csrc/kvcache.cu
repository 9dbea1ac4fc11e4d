// The paged key/value cache: growing and shrinking slots, forks that share pages, compaction, page copies
// and token writes (csdn/6a919c0d §3.3, a paged cache).
//
// Every operation has a table kernel, one CTA or (WIDE, for many entries or pages) a cluster of eight, that decides
// which pages go where; pages are then copied by
// a kernel over the whole GPU that reads the list's length on the device: no host round trip. (A resize copies
// in the table kernel itself: only a slot that grows again after a cut into a shared page needs it, and a second
// launch would cost every decode step more than it saves there.) A page is free exactly when its reference
// count is 0, and an allocation takes the lowest free pages in the order of the call's entries (a running
// count over the page numbers), so the tables come out the same every time, whatever the threads' order.
// The table kernels are bound by latency (L2 round trips of about 0.7 us between barriers), the copy and write
// kernels by HBM: 16-byte loads, four in flight a thread. Measured: a step's rollback, growth and write of 64 tokens
// 13 us, 16384 tokens of 8 heads of 128 (bf16) grown and written 31 us, 64 forks whose last pages of 2 x 128 KB are
// copied in 8 layers 38 us (7 TB/s), a compaction that moves about 900 pages of 2 x 128 KB 83 us (all in a graph).
//
// Values that other CTAs of the cluster wrote since the kernel began are read past L1 (__ldcg). A cluster barrier
// costs about 1 us against well under 0.1 us for a CTA's, which is why few entries stay in one CTA (16 forks: 9.5 us
// against 13).
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kTB = 1024;

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_cluster(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <bool WIDE> __device__ __forceinline__ void sync_all() {
  if (WIDE) cluster_sync_all();
  else __syncthreads();
}
template <bool WIDE> __device__ __forceinline__ int n_ctas() { return WIDE ? (int)cluster_size() : 1; }
template <bool WIDE> __device__ __forceinline__ int cta_rank() { return WIDE ? (int)cluster_ctarank() : 0; }

// Inclusive scan over the CTA; *total receives the sum. Two barriers.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // warp_sums may still be read from the scan before
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0);
}

// A value of each CTA of the cluster: their sum, and the sum of those of lower rank. `cell` is two words of shared
// memory that this and the next exchange alternate between (`turn`), so one barrier each is enough.
template <bool WIDE>
__device__ __forceinline__ void cluster_sums(int v, int* cell, int& turn, int* before, int* total) {
  if (!WIDE) {
    *before = 0;
    *total = v;
    return;
  }
  const int n = (int)cluster_size(), rank = (int)cluster_ctarank();
  if (threadIdx.x == 0) cell[turn] = v;
  cluster_sync_all();
  int b = 0, t = 0;
  for (int r = 0; r < n; ++r) {
    const int u = ld_cluster(map_to_cta(smem_u32(cell + turn), (uint32_t)r));
    t += u;
    if (r < rank) b += u;
  }
  turn ^= 1;
  *before = b;
  *total = t;
}

__device__ __forceinline__ int pages_for(int len, int shift) { return (int)(((long long)len + (1 << shift) - 1) >> shift); }

// Releases the pages of row `slot` in columns [from, to), one warp.
__device__ __forceinline__ void release_pages(const CacheView& c, int slot, int from, int to, int* status, int entry) {
  for (int p = from + (int)(threadIdx.x & 31); p < to; p += 32) {
    int32_t* t = c.table + (long long)slot * c.width + p;
    const int page = *t;
    if (page < 0 || page >= c.n_pages) record_error(status, MOE_ERR_DEVICE_CHECK, entry);
    else atomicSub(c.refs + page, 1);
    *t = -1;
  }
}

// The first `want` free pages, ascending, into w.freel; returns how many there are (at most want). Each round takes
// 4096 pages a CTA. Ends with a cluster barrier after the last write.
template <bool WIDE>
__device__ int find_free(const CacheView& c, const CacheWs& w, int want, int* warp_sums, int* cell, int& turn) {
  const int n = n_ctas<WIDE>(), rank = cta_rank<WIDE>();
  int found = 0;
  for (long long base = 0; base < c.n_pages && found < want; base += 4ll * kTB * n) {
    const long long p = base + 4ll * ((long long)rank * kTB + threadIdx.x);
    int fr[4], m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fr[i] = p + i < c.n_pages && __ldcg(c.refs + p + i) == 0;
      m += fr[i];
    }
    int mine, before, all;
    int at = block_scan(m, warp_sums, &mine) - m;
    cluster_sums<WIDE>(mine, cell, turn, &before, &all);
    at += found + before;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (fr[i]) {
        if (at < want) w.freel[at] = (int)(p + i);
        ++at;
      }
    found += all;
  }
  sync_all<WIDE>();
  return found < want ? found : want;
}

// One unit (16 KB) of a page copy, by 256 threads.
__device__ __forceinline__ void copy_unit(const CacheView& c, int a, int b, int kv, int layer, long long part,
                                          long long page_vec, int t) {
  uint4* base = reinterpret_cast<uint4*>(kv ? c.v : c.k) + (long long)layer * c.n_pages * page_vec;
  const uint4* from = base + (long long)a * page_vec;
  uint4* to = base + (long long)b * page_vec;
  const long long v0 = part * 1024 + t;
  uint4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (v0 + 256 * j < page_vec) x[j] = __ldcs(from + v0 + 256 * j);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (v0 + 256 * j < page_vec) __stcs(to + v0 + 256 * j, x[j]);
}

// Entries go to warps round-robin over the cluster: entry i to lane i / W of warp i mod W (of W). A lane keeps its
// entry's numbers in registers; its warp walks the table rows. entry[i] = {slot (-1: skipped), first new column,
// pages needed, their place in the free list}; bit 30 of the slot: the first one is a copy of the last page held.
constexpr int kCow = 1 << 30;

template <bool WIDE>
__global__ void __launch_bounds__(kTB)
cache_resize_kernel(const __grid_constant__ CacheView c, const __grid_constant__ CacheWs w,
                    const int32_t* __restrict__ slots, const int32_t* __restrict__ new_lens, int n, long long page_vec) {
  __shared__ int warp_sums[32], cell[2];
  griddep_launch_dependents();
  griddep_wait();
  // the copies of shared pages are the whole cluster's; unless WIDE, the tables are the first CTA's alone
  const int copier = (int)cluster_ctarank(), copiers = (int)cluster_size();
  const int rank = cta_rank<WIDE>(), nct = n_ctas<WIDE>();
  const int tid = threadIdx.x, lane = tid & 31, W = nct * (kTB / 32), gw = rank * (kTB / 32) + (tid >> 5);
  const long long most = (long long)c.width << c.page_shift;
  int turn = 0;
  int copies = 0;
  if (WIDE || copier == 0) {
    if (tid == 0 && rank == 0) w.counts[0] = 0;
    for (int i = rank * kTB + tid; i < n; i += nct * kTB) {
      const int s = slots[i], nl = new_lens[i];
      if (s < 0 || s >= c.n_slots || nl < 0 || nl > most)
        record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      else
        atomicMax(w.claim_d + s, n - i);  // the lowest entry that names the slot
    }
    sync_all<WIDE>();
    // shrinking slots give up their pages
    for (int base = 0; base < n; base += 32 * W) {
      const int i = base + lane * W + gw;
      int s = -1, po = 0, pn = 0, tail = -1;
      if (i < n) {
        s = slots[i];
        const int nl = new_lens[i];
        if (s < 0 || s >= c.n_slots || nl < 0 || nl > most) {
          s = -1;
        } else {
          const int old = c.lens[s];
          if (__ldcg(w.claim_d + s) != n - i || old < 0 || old > most) {
            record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
            s = -1;
          } else {
            po = pages_for(old, c.page_shift);
            pn = pages_for(nl, c.page_shift);
            if (nl > old && (old & (c.page_size - 1)) != 0) tail = c.table[(long long)s * c.width + po - 1];
            if (tail < -1 || tail >= c.n_pages) {
              record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
              tail = -1;
            }
          }
        }
        w.entry[i] = make_int4(s, po, pn, tail);
      }
      for (uint32_t shrink = __ballot_sync(0xffffffffu, pn < po); shrink != 0; shrink &= shrink - 1) {
        const int l = __ffs(shrink) - 1;
        release_pages(c, __shfl_sync(0xffffffffu, s, l), __shfl_sync(0xffffffffu, pn, l), __shfl_sync(0xffffffffu, po, l),
                      w.status, __shfl_sync(0xffffffffu, i, l));
      }
    }
    sync_all<WIDE>();
    // demand, in the entries' order: every CTA scans them all, the first one writes the places down
    int demand = 0;
    for (int base = 0; base < n; base += kTB) {
      const int i = base + tid;
      int4 e = make_int4(-1, 0, 0, -1);
      if (i < n) e = __ldcg(w.entry + i);
      const int cow = e.x >= 0 && e.w >= 0 && __ldcg(c.refs + e.w) > 1;
      const int need = e.x >= 0 && e.z > e.y - cow ? e.z - e.y + cow : 0;
      int total;
      const int incl = block_scan(need, warp_sums, &total);
      copies |= __syncthreads_or(cow);
      if (i < n && rank == 0) {
        const int s = slots[i];
        if (s >= 0 && s < c.n_slots) w.claim_d[s] = 0;  // zero again for the next call
        w.entry2[i] = make_int4(e.x | (cow ? kCow : 0), e.y - cow, need, demand + incl - need);
      }
      demand += total;
    }
    int have = 0;
    if (demand > 0) have = find_free<WIDE>(c, w, demand, warp_sums, cell, turn);
    else sync_all<WIDE>();
    for (int i = gw; i < n; i += W) {
      const int4 e = __ldcg(w.entry2 + i);
      if (e.x < 0) continue;
      const int s = e.x & ~kCow, cow = (e.x & kCow) != 0;
      if (e.z > 0 && e.w + e.z > have) {  // the pages ran out: the slot stays as it was
        if (lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        continue;
      }
      int32_t* row = c.table + (long long)s * c.width;
      for (int j = lane; j < e.z; j += 32) {
        const int page = __ldcg(w.freel + e.w + j);
        if (j == 0 && cow) {
          const int old = row[e.y];
          w.copies[atomicAdd(w.counts, 1)] = make_int2(old, page);
          atomicSub(c.refs + old, 1);
        }
        row[e.y + j] = page;
        c.refs[page] = 1;
      }
      if (lane == 0) c.lens[s] = new_lens[i];
    }
  }
  if (WIDE) {
    if (copies != 0) cluster_sync_all();
  } else {
    cluster_sync_all();
  }
  if (!WIDE || copies != 0) {
    const int count = __ldcg(w.counts);
    const long long per = (page_vec + 1023) / 1024, units = (long long)count * c.n_layers * 2 * per;
    for (long long u = (long long)copier * 4 + (tid >> 8); u < units; u += 4 * copiers) {
      const long long pl = u / per;
      const int2 m = __ldcg(w.copies + (pl >> 1) / c.n_layers);
      copy_unit(c, m.x, m.y, (int)(pl & 1), (int)((pl >> 1) % c.n_layers), u % per, page_vec, tid & 255);
    }
  }
  if (WIDE) cluster_sync_all();  // no CTA leaves while another may still read its shared memory
}

template <bool WIDE>
__global__ void __launch_bounds__(kTB)
cache_fork_kernel(const __grid_constant__ CacheView c, const __grid_constant__ CacheWs w, const int32_t* __restrict__ src,
                  const int32_t* __restrict__ dst, int n) {
  __shared__ int warp_sums[32], cell[2];
  griddep_launch_dependents();
  griddep_wait();
  const int rank = cta_rank<WIDE>(), nct = n_ctas<WIDE>();
  const int tid = threadIdx.x, lane = tid & 31, W = nct * (kTB / 32), gw = rank * (kTB / 32) + (tid >> 5);
  const long long most = (long long)c.width << c.page_shift;
  int turn = 0;
  if (tid == 0 && rank == 0) w.counts[0] = 0;
  for (int i = rank * kTB + tid; i < n; i += nct * kTB) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= c.n_slots || d < 0 || d >= c.n_slots) {
      record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
    } else {
      atomicMax(w.claim_d + d, n - i);
      w.claim_s[s] = 1;
    }
  }
  sync_all<WIDE>();
  for (int i = gw; i < n; i += W) {
    const int s = src[i], d = dst[i];
    bool ok = s >= 0 && s < c.n_slots && d >= 0 && d < c.n_slots;
    int ls = 0;
    if (ok) {
      ls = c.lens[s];
      const int ld = c.lens[d];
      ok = __ldcg(w.claim_d + d) == n - i && __ldcg(w.claim_s + d) == 0 && ls >= 0 && ls <= most && ld >= 0 && ld <= most;
      if (!ok && lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      if (ok) {
        release_pages(c, d, 0, pages_for(ld, c.page_shift), w.status, i);
        __syncwarp();
        if (lane == 0) c.lens[d] = 0;
      }
    }
    if (lane == 0) w.entry[i] = make_int4(ok ? s : -1, d, ls, 0);
  }
  sync_all<WIDE>();
  int demand = 0;
  for (int base = 0; base < n; base += kTB) {
    const int i = base + tid;
    int4 e = make_int4(-1, 0, 0, 0);
    if (i < n) e = __ldcg(w.entry + i);
    const int need = e.x >= 0 && (e.z & (c.page_size - 1)) != 0;
    int total;
    const int incl = block_scan(need, warp_sums, &total);
    if (i < n && rank == 0) {
      const int s = src[i], d = dst[i];
      if (s >= 0 && s < c.n_slots && d >= 0 && d < c.n_slots) {
        w.claim_d[d] = 0;
        w.claim_s[s] = 0;
      }
      w.entry2[i] = make_int4(e.x, e.y, e.z, demand + incl - need);
    }
    demand += total;
  }
  int have = 0;
  if (demand > 0) have = find_free<WIDE>(c, w, demand, warp_sums, cell, turn);
  else sync_all<WIDE>();
  for (int i = gw; i < n; i += W) {
    const int4 e = __ldcg(w.entry2 + i);
    if (e.x < 0) continue;
    const int len = e.z, full = len >> c.page_shift, part = (len & (c.page_size - 1)) != 0;
    if (part && e.w >= have) {
      if (lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      continue;
    }
    const int32_t* from = c.table + (long long)e.x * c.width;
    int32_t* to = c.table + (long long)e.y * c.width;
    if (lane == 0) {
      if (part) {
        const int page = __ldcg(w.freel + e.w), old = from[full];
        if (old >= 0 && old < c.n_pages) w.copies[atomicAdd(w.counts, 1)] = make_int2(old, page);
        else record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        to[full] = page;
        c.refs[page] = 1;
      }
      c.lens[e.y] = len;
    }
    for (int p = lane; p < full; p += 32) {
      int page = from[p];
      if (page < 0 || page >= c.n_pages) {
        record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        page = -1;
      } else {
        atomicAdd(c.refs + page, 1);
      }
      to[p] = page;
    }
  }
  sync_all<WIDE>();
}

// Which pages move: the j-th used page at or above the live count to the j-th free page below it. Each CTA of the
// cluster has a stretch of the pages; three walks over it (live pages; holes and movers; the lists).
template <bool WIDE>
__global__ void __launch_bounds__(kTB)
cache_compact_kernel(const __grid_constant__ CacheView c, const __grid_constant__ CacheWs w, int32_t* n_live) {
  __shared__ int warp_sums[32], cell[2];
  griddep_launch_dependents();
  griddep_wait();
  const int rank = cta_rank<WIDE>(), nct = n_ctas<WIDE>(), tid = threadIdx.x;
  const int per = ((c.n_pages + nct - 1) / nct + 3) & ~3;
  const int begin = (int)min((long long)c.n_pages, (long long)rank * per), end = (int)min((long long)c.n_pages, (long long)begin + per);
  int turn = 0, mine = 0, sum, before, live;
  for (int p = begin + tid; p < end; p += kTB) mine += c.refs[p] != 0;
  block_scan(mine, warp_sums, &sum);
  cluster_sums<WIDE>(sum, cell, turn, &before, &live);
  int nh = 0, nm = 0;
  for (int p = begin + tid; p < end; p += kTB) {
    const bool used = c.refs[p] != 0;
    nh += p < live && !used;
    nm += p >= live && used;
  }
  int holes, movers, total_h, total_m;
  block_scan(nh, warp_sums, &sum);
  cluster_sums<WIDE>(sum, cell, turn, &holes, &total_h);
  block_scan(nm, warp_sums, &sum);
  cluster_sums<WIDE>(sum, cell, turn, &movers, &total_m);
  for (int base = begin; base < end; base += 4 * kTB) {
    const int p0 = base + 4 * tid;
    int hole[4], move[4], th, tm;
    nh = nm = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + i;
      const bool used = p < end && c.refs[p] != 0;
      hole[i] = p < end && p < live && !used;
      move[i] = p >= live && used;
      nh += hole[i];
      nm += move[i];
    }
    int ah = holes + block_scan(nh, warp_sums, &th) - nh;
    int am = movers + block_scan(nm, warp_sums, &tm) - nm;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (hole[i]) w.copies[ah++].y = p0 + i;
      if (move[i]) w.copies[am++].x = p0 + i;
    }
    holes += th;
    movers += tm;
  }
  sync_all<WIDE>();
  for (int j = rank * kTB + tid; j < total_m; j += nct * kTB) {
    const int2 m = __ldcg(w.copies + j);
    w.map[m.x] = m.y;
    c.refs[m.y] = __ldcg(c.refs + m.x);
    c.refs[m.x] = 0;
  }
  if (tid == 0 && rank == 0) {
    w.counts[0] = total_m;
    w.counts[1] = live;
    if (n_live != nullptr) *n_live = live;
  }
}

// Copies pages by a list, on the device (list, count) or the caller's (src, dst): units of 16 KB, walked by the whole
// grid. With `retable`, table entries at or above the live count first follow their pages.
__global__ void __launch_bounds__(256)
cache_copy_kernel(const __grid_constant__ CacheView c, const __grid_constant__ CacheWs w,
                  const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n_given, int retable,
                  long long page_vec) {
  griddep_launch_dependents();
  griddep_wait();
  if (retable) {
    const int live = w.counts[1];
    const long long total = (long long)c.n_slots * c.width;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
      const int page = c.table[i];
      if (page >= live && page < c.n_pages) c.table[i] = w.map[page];
    }
  }
  const int n = src == nullptr ? w.counts[0] : n_given;
  const long long per = (page_vec + 1023) / 1024;  // units of a page
  const long long units = (long long)n * c.n_layers * 2 * per;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long pl = u / per;
    const int kv = (int)(pl & 1), layer = (int)((pl >> 1) % c.n_layers), i = (int)((pl >> 1) / c.n_layers);
    const int a = src == nullptr ? w.copies[i].x : src[i], b = src == nullptr ? w.copies[i].y : dst[i];
    if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
      if (threadIdx.x == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      continue;
    }
    if (a != b) copy_unit(c, a, b, kv, layer, u % per, page_vec, threadIdx.x);
  }
}

// One warp a token: its sequence by a 32-way search of the offsets, then 16 bytes a lane of K and of V, asked for
// before the token's place is known.
__global__ void __launch_bounds__(256)
cache_write_kernel(const __grid_constant__ CacheView c, uint4* __restrict__ kdst, uint4* __restrict__ vdst,
                   const int32_t* __restrict__ slots, const int32_t* __restrict__ offsets,
                   const int32_t* __restrict__ pos, int n, int total, const uint4* __restrict__ k,
                   const uint4* __restrict__ v, long long ks, long long vs, int head_vec, int* status) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= total) return;
  const int vec = c.Hkv * head_vec;
  uint4 a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 32 * j < vec) {
      a[j] = __ldcs(k + t * ks + lane + 32 * j);
      b[j] = __ldcs(v + t * vs + lane + 32 * j);
    }
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const bool at = lane * step < len && offsets[lo + lane * step] <= t;
    const int m = __popc(__ballot_sync(0xffffffffu, at)) - 1, skip = (m < 0 ? 0 : m) * step;
    lo += skip;
    len = len - skip < step ? len - skip : step;
  }
  const int s = slots[lo], o0 = offsets[lo], o1 = offsets[lo + 1], p0 = pos[lo];
  bool ok = s >= 0 && s < c.n_slots && t >= o0 && t < o1 && p0 >= 0;
  int page = 0;
  const long long p = (long long)p0 + (t - o0);
  if (ok && (p >> c.page_shift) < c.width) {
    const int held = c.lens[s];
    page = c.table[(long long)s * c.width + (p >> c.page_shift)];
    ok = p < held && page >= 0 && page < c.n_pages && c.refs[page] == 1;
  } else {
    ok = false;
  }
  if (!ok) {
    if (lane == 0) record_error(status, MOE_ERR_DEVICE_CHECK, (int)t);
    return;
  }
  const long long row = p & (c.page_size - 1);
  for (int i0 = 0; i0 < vec; i0 += 128) {
    if (i0 > 0)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + lane + 32 * j < vec) {
          a[j] = __ldcs(k + t * ks + i0 + lane + 32 * j);
          b[j] = __ldcs(v + t * vs + i0 + lane + 32 * j);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + lane + 32 * j;
      if (i < vec) {
        const int h = i / head_vec, x = i % head_vec;
        const long long at = (((long long)page * c.Hkv + h) * c.page_size + row) * head_vec + x;
        kdst[at] = a[j];
        vdst[at] = b[j];
      }
    }
  }
}

inline long long page_vectors(const CacheView& c) {
  return (long long)c.Hkv * c.page_size * c.D * (c.dt == MOE_DTYPE_BF16 ? 2 : 4) / 16;
}

constexpr int kCluster = 8;
// From here on a cluster works on the tables: entries of a resize, table cells of a fork (64 forks of 250 pages: 15
// to 21 against 17 to 24 us), pages of a pool.
constexpr int kWideEntries = 1024, kWideCells = 8192, kWidePages = 1 << 16;

cudaError_t copy_list(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n, int retable,
                      cudaStream_t s) {
  return launch_pdl(cache_copy_kernel, dim3(8 * device_sm_count()), dim3(256), 0, s, c, w, src, dst, n, retable,
                    page_vectors(c));
}

}  // namespace

cudaError_t launch_cache_resize(const CacheView& c, const CacheWs& w, const int32_t* slots, const int32_t* new_lens, int n,
                                cudaStream_t s) {
  return launch_clusters(n > kWideEntries ? cache_resize_kernel<true> : cache_resize_kernel<false>, dim3(kCluster),
                         dim3(kTB), dim3(kCluster), 0, s, c, w, slots, new_lens, n, page_vectors(c));
}

cudaError_t launch_cache_fork(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s) {
  const bool wide = (long long)n * c.width > kWideCells;
  const cudaError_t e = wide ? launch_clusters(cache_fork_kernel<true>, dim3(kCluster), dim3(kTB), dim3(kCluster), 0, s, c,
                                               w, src, dst, n)
                             : launch_pdl(cache_fork_kernel<false>, dim3(1), dim3(kTB), 0, s, c, w, src, dst, n);
  return e != cudaSuccess ? e : copy_list(c, w, nullptr, nullptr, 0, 0, s);
}

cudaError_t launch_cache_compact(const CacheView& c, const CacheWs& w, int32_t* n_live, cudaStream_t s) {
  const cudaError_t e = c.n_pages > kWidePages
                            ? launch_clusters(cache_compact_kernel<true>, dim3(kCluster), dim3(kTB), dim3(kCluster), 0, s,
                                              c, w, n_live)
                            : launch_pdl(cache_compact_kernel<false>, dim3(1), dim3(kTB), 0, s, c, w, n_live);
  return e != cudaSuccess ? e : copy_list(c, w, nullptr, nullptr, 0, 1, s);
}

cudaError_t launch_cache_copy(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s) {
  return copy_list(c, w, src, dst, n, 0, s);
}

cudaError_t launch_cache_write(const CacheView& c, const CacheWs& w, int layer, const int32_t* slots,
                               const int32_t* offsets, const int32_t* pos, int n, int total, const void* k, const void* v,
                               long long ks, long long vs, cudaStream_t s) {
  const int eb = c.dt == MOE_DTYPE_BF16 ? 2 : 4;
  const long long off = (long long)layer * c.n_pages * page_vectors(c);
  return launch_pdl(cache_write_kernel, dim3((unsigned)((total + 7LL) / 8)), dim3(256), 0, s, c, (uint4*)c.k + off,
                    (uint4*)c.v + off, slots, offsets, pos, n, total, (const uint4*)k, (const uint4*)v,
                    ks * eb / 16, vs * eb / 16, c.D * eb / 16, w.status);
}

}  // namespace moe

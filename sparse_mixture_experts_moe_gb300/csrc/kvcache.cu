// The paged key/value cache: growing and shrinking slots, forks that share pages, compaction, page copies
// and token writes (csdn/6a919c0d §3.3, a paged cache).
//
// Every operation is a table kernel (one CTA of 1024 threads: the tables are a few hundred kilobytes at
// most) that decides which pages go where and leaves a list of page copies in the workspace, then a copy
// kernel over the whole GPU that reads the list's length on the device: no host round trip. A page is
// free exactly when its reference count is 0, and an allocation takes the lowest free pages in the order
// of the call's entries (a running count over the page numbers), so the tables come out the same
// every time, whatever the threads' order.
// The table kernels are bound by latency (a chain of block-wide scans and L2 round trips), the copy and write
// kernels by HBM: 16-byte loads, four in flight a thread.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kTB = 1024;

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

// The first `want` free pages, ascending, into w.freel; returns how many there are (at most want).
__device__ int find_free(const CacheView& c, const CacheWs& w, int want, int* warp_sums) {
  int found = 0;
  for (int base = 0; base < c.n_pages && found < want; base += 4 * kTB) {
    const int p = base + 4 * (int)threadIdx.x;
    int fr[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fr[i] = p + i < c.n_pages && __ldcg(c.refs + p + i) == 0;
      n += fr[i];
    }
    int total;
    int at = found + block_scan(n, warp_sums, &total) - n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (fr[i]) {
        if (at < want) w.freel[at] = p + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return found < want ? found : want;
}

// entry[i] = {slot (-1: skipped), first new column, end column, bit 0: last page copied, start in the free list}
__global__ void __launch_bounds__(kTB)
cache_resize_kernel(const CacheView c, const CacheWs w, const int32_t* __restrict__ slots,
                    const int32_t* __restrict__ new_lens, int n) {
  __shared__ int warp_sums[32];
  __shared__ int n_copies;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) n_copies = 0;
  for (int i = tid; i < n; i += kTB) {
    const int s = slots[i], nl = new_lens[i];
    if (s < 0 || s >= c.n_slots || nl < 0 || (long long)nl > ((long long)c.width << c.page_shift))
      record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
    else
      atomicMax(w.claim_d + s, n - i);  // the lowest entry that names the slot
  }
  __syncthreads();
  // shrinking slots give up their pages
  for (int i = warp; i < n; i += kTB / 32) {
    const int s = slots[i], nl = new_lens[i];
    bool ok = s >= 0 && s < c.n_slots && nl >= 0 && (long long)nl <= ((long long)c.width << c.page_shift);
    int po = 0, pn = 0, old = 0;
    if (ok) {
      old = c.lens[s];
      if (__ldcg(w.claim_d + s) != n - i || old < 0 || (long long)old > ((long long)c.width << c.page_shift)) {
        if (lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        ok = false;
      } else {
        po = pages_for(old, c.page_shift);
        pn = pages_for(nl, c.page_shift);
        if (pn < po) release_pages(c, s, pn, po, w.status, i);
      }
    }
    if (lane == 0) w.entry[i] = make_int4(ok ? s : -1, po, pn, 0);
  }
  __syncthreads();
  // demand, in the entries' order
  int demand = 0;
  for (int base = 0; base < n; base += kTB) {
    const int i = base + tid;
    int need = 0, cow = 0;
    int4 e = make_int4(-1, 0, 0, 0);
    if (i < n) e = w.entry[i];
    if (e.x >= 0) {
      const int old = c.lens[e.x], nl = new_lens[i];
      if (nl > old && (old & (c.page_size - 1)) != 0) {
        const int page = c.table[(long long)e.x * c.width + e.y - 1];
        if (page < 0 || page >= c.n_pages) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        else cow = __ldcg(c.refs + page) > 1;
      }
      need = e.z - e.y + cow;
      if (need < 0) need = 0;
      e.y -= cow;
    }
    int total;
    const int incl = block_scan(need, warp_sums, &total);
    if (i < n) {
      // claims are zero again for the next call
      const int s = slots[i];
      if (s >= 0 && s < c.n_slots) w.claim_d[s] = 0;
      w.entry[i] = make_int4(e.x, e.y, e.z, ((demand + incl - need) << 1) | cow);
    }
    demand += total;
  }
  __syncthreads();
  const int have = demand > 0 ? find_free(c, w, demand, warp_sums) : 0;
  for (int i = warp; i < n; i += kTB / 32) {
    const int4 e = w.entry[i];
    if (e.x < 0) continue;
    const int cow = e.w & 1, start = e.w >> 1, need = e.z > e.y ? e.z - e.y : 0;
    if (need > 0 && start + need > have) {  // the pages ran out: the slot stays as it was
      if (lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      continue;
    }
    int32_t* row = c.table + (long long)e.x * c.width;
    for (int j = lane; j < need; j += 32) {
      const int page = w.freel[start + j];
      if (j == 0 && cow) {
        const int old = row[e.y];
        w.copies[atomicAdd(&n_copies, 1)] = make_int2(old, page);
        atomicSub(c.refs + old, 1);
      }
      row[e.y + j] = page;
      c.refs[page] = 1;
    }
    if (lane == 0) c.lens[e.x] = new_lens[i];
  }
  __syncthreads();
  if (tid == 0) w.counts[0] = n_copies;
}

__global__ void __launch_bounds__(kTB)
cache_fork_kernel(const CacheView c, const CacheWs w, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                  int n) {
  __shared__ int warp_sums[32];
  __shared__ int n_copies;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long most = (long long)c.width << c.page_shift;
  if (tid == 0) n_copies = 0;
  for (int i = tid; i < n; i += kTB) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= c.n_slots || d < 0 || d >= c.n_slots) {
      record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
    } else {
      atomicMax(w.claim_d + d, n - i);
      w.claim_s[s] = 1;
    }
  }
  __syncthreads();
  for (int i = warp; i < n; i += kTB / 32) {
    const int s = src[i], d = dst[i];
    bool ok = s >= 0 && s < c.n_slots && d >= 0 && d < c.n_slots;
    if (ok) {
      const int ls = c.lens[s], ld = c.lens[d];
      ok = __ldcg(w.claim_d + d) == n - i && __ldcg(w.claim_s + d) == 0 && ls >= 0 && ls <= most && ld >= 0 && ld <= most;
      if (!ok && lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      if (ok) {
        release_pages(c, d, 0, pages_for(ld, c.page_shift), w.status, i);
        __syncwarp();
        if (lane == 0) c.lens[d] = 0;
      }
    }
    if (lane == 0) w.entry[i] = make_int4(ok ? s : -1, d, 0, 0);
  }
  __syncthreads();
  int demand = 0;
  for (int base = 0; base < n; base += kTB) {
    const int i = base + tid;
    int4 e = make_int4(-1, 0, 0, 0);
    if (i < n) e = w.entry[i];
    const int need = e.x >= 0 && (c.lens[e.x] & (c.page_size - 1)) != 0;
    int total;
    const int incl = block_scan(need, warp_sums, &total);
    if (i < n) {
      const int s = src[i], d = dst[i];
      if (s >= 0 && s < c.n_slots && d >= 0 && d < c.n_slots) {
        w.claim_d[d] = 0;
        w.claim_s[s] = 0;
      }
      w.entry[i] = make_int4(e.x, e.y, demand + incl - need, need);
    }
    demand += total;
  }
  __syncthreads();
  const int have = demand > 0 ? find_free(c, w, demand, warp_sums) : 0;
  for (int i = warp; i < n; i += kTB / 32) {
    const int4 e = w.entry[i];
    if (e.x < 0) continue;
    if (e.w && e.z >= have) {
      if (lane == 0) record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
      continue;
    }
    const int len = c.lens[e.x], full = len >> c.page_shift;
    const int32_t* from = c.table + (long long)e.x * c.width;
    int32_t* to = c.table + (long long)e.y * c.width;
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
    if (lane == 0) {
      if (e.w) {
        const int page = w.freel[e.z], old = from[full];
        if (old >= 0 && old < c.n_pages) w.copies[atomicAdd(&n_copies, 1)] = make_int2(old, page);
        else record_error(w.status, MOE_ERR_DEVICE_CHECK, i);
        to[full] = page;
        c.refs[page] = 1;
      }
      c.lens[e.y] = len;
    }
  }
  __syncthreads();
  if (tid == 0) w.counts[0] = n_copies;
}

// Which pages move: the j-th used page at or above the live count to the j-th free page below it.
__global__ void __launch_bounds__(kTB)
cache_compact_kernel(const CacheView c, const CacheWs w, int32_t* n_live) {
  __shared__ int warp_sums[32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  int mine = 0, live;
  for (int p = tid; p < c.n_pages; p += kTB) mine += c.refs[p] != 0;
  block_scan(mine, warp_sums, &live);
  int holes = 0, movers = 0;
  for (int base = 0; base < c.n_pages; base += 4 * kTB) {
    const int p0 = base + 4 * tid;
    int hole[4], move[4], nh = 0, nm = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + i;
      const bool used = p < c.n_pages && c.refs[p] != 0;
      hole[i] = p < c.n_pages && p < live && !used;
      move[i] = p >= live && used;
      nh += hole[i];
      nm += move[i];
    }
    int th, tm;
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
  __syncthreads();
  for (int j = tid; j < movers; j += kTB) {
    const int2 m = w.copies[j];
    w.map[m.x] = m.y;
    c.refs[m.y] = c.refs[m.x];
    c.refs[m.x] = 0;
  }
  if (tid == 0) {
    w.counts[0] = movers;
    w.counts[1] = live;
    if (n_live != nullptr) *n_live = live;
  }
}

// Table entries at or above the live count follow their pages.
__global__ void __launch_bounds__(256) cache_retable_kernel(const CacheView c, const CacheWs w) {
  griddep_launch_dependents();
  griddep_wait();
  const int live = w.counts[1];
  const long long total = (long long)c.n_slots * c.width;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int page = c.table[i];
    if (page >= live && page < c.n_pages) c.table[i] = w.map[page];
  }
}

// Copies pages by a list on the device: units of 16 KB, walked by the whole grid.
__global__ void __launch_bounds__(256)
cache_copy_kernel(const CacheView c, const int2* __restrict__ list, const int32_t* __restrict__ count,
                  const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n_given, long long page_vec,
                  int* status) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = count != nullptr ? *count : n_given;
  const long long per = (page_vec + 1023) / 1024;  // units of a page
  const long long units = (long long)n * c.n_layers * 2 * per;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long part = u % per, pl = u / per;
    const int kv = (int)(pl & 1), layer = (int)((pl >> 1) % c.n_layers), i = (int)((pl >> 1) / c.n_layers);
    const int a = list != nullptr ? list[i].x : src[i], b = list != nullptr ? list[i].y : dst[i];
    if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
      if (threadIdx.x == 0) record_error(status, MOE_ERR_DEVICE_CHECK, i);
      continue;
    }
    if (a == b) continue;
    uint4* base = reinterpret_cast<uint4*>(kv ? c.v : c.k) + (long long)layer * c.n_pages * page_vec;
    const uint4* from = base + (long long)a * page_vec;
    uint4* to = base + (long long)b * page_vec;
    const long long v0 = part * 1024 + threadIdx.x;
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v0 + 256 * j < page_vec) x[j] = __ldcs(from + v0 + 256 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v0 + 256 * j < page_vec) __stcs(to + v0 + 256 * j, x[j]);
  }
}

// One warp a token: its sequence by bisection of the offsets, then 16 bytes a lane of K and of V.
__global__ void __launch_bounds__(256)
cache_write_kernel(const CacheView c, uint4* __restrict__ kdst, uint4* __restrict__ vdst,
                   const int32_t* __restrict__ slots, const int32_t* __restrict__ offsets,
                   const int32_t* __restrict__ pos, int n, int total, const uint4* __restrict__ k,
                   const uint4* __restrict__ v, long long ks, long long vs, int head_vec, int* status) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= total) return;
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int s = slots[lo];
  bool ok = s >= 0 && s < c.n_slots && t >= offsets[lo] && t < offsets[lo + 1] && pos[lo] >= 0;
  int page = 0;
  long long p = 0;
  if (ok) {
    p = (long long)pos[lo] + (t - offsets[lo]);
    ok = p < c.lens[s] && (p >> c.page_shift) < c.width;
    if (ok) {
      page = c.table[(long long)s * c.width + (p >> c.page_shift)];
      ok = page >= 0 && page < c.n_pages && c.refs[page] == 1;
    }
  }
  if (!ok) {
    if (lane == 0) record_error(status, MOE_ERR_DEVICE_CHECK, (int)t);
    return;
  }
  const long long row = p & (c.page_size - 1);
  for (int i = lane; i < c.Hkv * head_vec; i += 32) {
    const int h = i / head_vec, x = i % head_vec;
    const long long at = (((long long)page * c.Hkv + h) * c.page_size + row) * head_vec + x;
    const uint4 a = __ldcs(k + t * ks + i), b = __ldcs(v + t * vs + i);
    kdst[at] = a;
    vdst[at] = b;
  }
}

inline long long page_vectors(const CacheView& c) {
  return (long long)c.Hkv * c.page_size * c.D * (c.dt == MOE_DTYPE_BF16 ? 2 : 4) / 16;
}

cudaError_t copy_list(const CacheView& c, const CacheWs& w, cudaStream_t s) {
  return launch_pdl(cache_copy_kernel, dim3(8 * device_sm_count()), dim3(256), 0, s, c, (const int2*)w.copies,
                    (const int32_t*)w.counts, (const int32_t*)nullptr, (const int32_t*)nullptr, 0, page_vectors(c),
                    w.status);
}

}  // namespace

cudaError_t launch_cache_resize(const CacheView& c, const CacheWs& w, const int32_t* slots, const int32_t* new_lens, int n,
                                cudaStream_t s) {
  const cudaError_t e = launch_pdl(cache_resize_kernel, dim3(1), dim3(kTB), 0, s, c, w, slots, new_lens, n);
  return e != cudaSuccess ? e : copy_list(c, w, s);
}

cudaError_t launch_cache_fork(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s) {
  const cudaError_t e = launch_pdl(cache_fork_kernel, dim3(1), dim3(kTB), 0, s, c, w, src, dst, n);
  return e != cudaSuccess ? e : copy_list(c, w, s);
}

cudaError_t launch_cache_compact(const CacheView& c, const CacheWs& w, int32_t* n_live, cudaStream_t s) {
  cudaError_t e = launch_pdl(cache_compact_kernel, dim3(1), dim3(kTB), 0, s, c, w, n_live);
  if (e != cudaSuccess) return e;
  e = launch_pdl(cache_retable_kernel, dim3(device_sm_count()), dim3(256), 0, s, c, w);
  return e != cudaSuccess ? e : copy_list(c, w, s);
}

cudaError_t launch_cache_copy(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s) {
  return launch_pdl(cache_copy_kernel, dim3(8 * device_sm_count()), dim3(256), 0, s, c, (const int2*)nullptr,
                    (const int32_t*)nullptr, src, dst, n, page_vectors(c), w.status);
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

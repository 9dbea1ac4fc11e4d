// Shared declarations of the attention and cache kernels (internal to the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "attn_plan.cuh"
#include "common.cuh"

namespace moe {

// Words of the workspace's header (see kWsHeaderBytes) besides the status: [6] the decode kernel's counter of runs
// taken, [7] the prompt kernel's counter of items and [8] its count of finished CTAs. Zero between calls, like the
// others there.

// Packed rows: the G = H / H_kv query heads that share a key/value head are laid side by side, row
// r = token * G + g, so that one key/value tile serves all of them and short prompts or single tokens
// still fill a tile's rows.
struct PromptArgs {
  const void *q, *k, *v;
  const int32_t *qo, *ko;  // [n + 1] each
  int n, Tq, Tkv, H, Hkv, D;
  long long qs, ks, vs, os;  // token strides in elements
  float scale;
  int causal, dt;
  void* out;
  float* lse;
  int* status;
  uint64_t timeout_ns;
};

struct CacheView {
  void *k, *v;
  int32_t *table, *lens, *refs;
  int n_layers, n_pages, page_size, page_shift, n_slots, width, Hkv, D, dt;
  long long layer_elems() const { return (long long)n_pages * Hkv * page_size * D; }
};

// Copy descriptors of a bf16 cache's pages: a layer's page rows ((page H_kv + head) page_size + row) x D, the layer
// as the third coordinate; boxes of 64 elements x 16, min(page_size, 64) and min(page_size, 128) rows.
struct CacheMaps {
  CUtensorMap k16, v16, k64, v64, k128, v128;
};
bool encode_cache_maps(const CacheView& c, CacheMaps* m);

// Sets a kernel's dynamic shared memory limit, once a device: the last device it was set for is remembered (setting
// it again is harmless, so a race between threads is too).
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kern, size_t bytes, std::atomic<int>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || done.load(std::memory_order_relaxed) == dev + 1) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.store(dev + 1, std::memory_order_relaxed);
  return e;
}

// Launch in clusters, with programmatic stream serialisation (as launch_pdl).
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, dim3 cluster, size_t smem, cudaStream_t s,
                            Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = cluster.z;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct DecodeArgs {
  const void* q;
  long long qs, os;
  const int32_t* slots;
  const int32_t* lead;  // the call's first slot, whose pages hold the shared positions (slots may begin at a slice)
  int n, H, shared;
  int first;  // number in the call of row 0, for errors
  float scale;
  CacheView c;
  const void *k, *v;  // the layer's pages
  int layer;
  void* out;
  float* lse;
  float* part;  // partial results: attn_simt.cu has [row][piece][D + 2], attn_decode.cu arrays for o and ml apart
  int* status;
  uint64_t timeout_ns;
};

// The shared positions of a decode call that does not take the tcgen05 path, in tiles of 64 rows and 64 keys.
struct SharedPart {
  DecodeArgs d;
  int splits, per;  // pieces of a row over the shared positions; positions of a piece
  int pieces;       // of a row altogether
};

// A chunk call's run of items (attn_chunk.cu): the one that begins in it and goes on in others, up to run `end`. nrows =
// 0: none.
struct ChunkRun {
  int hk, q0, row0, nrows, end;
};

// What the other warps' waits allow a softmax warp of attn_tc.cu or attn_chunk.cu that replaces columns of its 32 rows
// (replace_unseen): 0.4 us a key and row, where 0.1 was measured, and 20 s at most.
constexpr uint64_t replace_time(long long keys) { return keys < 1562500 ? (uint64_t)keys * 32 * 400 : 20000000000ull; }

// Workspace of one decode call. A piece is the attention of one row over a part of its keys: the sum of
// the weighted values (D floats), the weights' sum l and the reference m (in log2 units) that the
// weights 2^(s - m) were taken against. A row's pieces join as out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// Pieces that a call may have: 4 a row, and enough for every SM to hold several pieces of many rows.
constexpr long long decode_pieces(long long rows) { return 4 * rows + 65536; }

cudaError_t launch_attn_prompt_simt(const PromptArgs& a, cudaStream_t s);  // fp32
cudaError_t launch_attn_prompt_mma(const PromptArgs& a, cudaStream_t s);   // bf16, any D
cudaError_t launch_attn_shared_mma(const SharedPart& sp, dim3 grid, cudaStream_t s);  // grid: (row tiles, H_kv, splits)
// bf16, D <= 128, at least one key.
// splits: attn_prompt_splits or 1; part: Tq H splits (D + 2) floats where there are several.
int attn_prompt_splits(int n, int Tq, int Tkv, int H, int Hkv);
cudaError_t launch_attn_prompt_tc(const PromptArgs& a, int splits, float* part, cudaStream_t s);
cudaError_t launch_attn_decode_tc(const DecodeArgs& a, const CacheMaps& m, cudaStream_t s);
// The shared keys of a decode batch: `splits` pieces of every row, part_o [(sequence, head)][splits][D] unnormalised.
int attn_shared_splits(const DecodeArgs& a);
cudaError_t launch_attn_shared_tc(const DecodeArgs& a, const CacheMaps& m, int splits, float* part_o, float2* part_ml,
                                  cudaStream_t s);
cudaError_t launch_attn_decode_simt(const DecodeArgs& a, cudaStream_t s);
// A chunk of new tokens over the cache: queries and offsets of a, the cache, slots and layer of d. bf16, D <= 128: scratch
// of chunk_tc_bytes.
size_t chunk_tc_bytes(int Tq, int G, int D);
cudaError_t launch_attn_chunk_tc(const PromptArgs& a, const DecodeArgs& d, const CacheMaps& m, void* scratch, cudaStream_t s);
// The other types and heads: rows in `pieces` parts, d.part [Tq H][pieces][D + 2] (none where clusters hold them).
int chunk_tile_pieces(const CacheView& c, int n, int Tq, int H);
bool chunk_tiles_in_clusters(const CacheView& c, int n, int Tq, int H, int pieces);
cudaError_t launch_attn_chunk_tiles(const PromptArgs& a, const DecodeArgs& d, int pieces, cudaStream_t s);
cudaError_t launch_attn_chunk_mma(const PromptArgs& a, const SharedPart& sp, dim3 grid, cudaStream_t s);

struct CacheWs {
  int* status;       // workspace header
  int32_t* claim_d;  // [n_slots] zero between calls: which entry names the slot (as dst)
  int32_t* claim_s;  // [n_slots] zero between calls: the slot is a source
  int4* entry;       // [n_slots]
  int4* entry2;      // [n_slots]
  int32_t* freel;    // [n_pages] pages found free, ascending
  int2* copies;      // [max(n_slots, n_pages)] (src, dst) pages
  int32_t* map;      // [n_pages] where a moved page went
  int32_t* counts;   // [0] number of copies, [1] pages in use
};
cudaError_t launch_cache_resize(const CacheView& c, const CacheWs& w, const int32_t* slots, const int32_t* new_lens, int n,
                                cudaStream_t s);
cudaError_t launch_cache_fork(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s);
cudaError_t launch_cache_compact(const CacheView& c, const CacheWs& w, int32_t* n_live, cudaStream_t s);
cudaError_t launch_cache_copy(const CacheView& c, const CacheWs& w, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t s);
cudaError_t launch_cache_write(const CacheView& c, const CacheWs& w, int layer, const int32_t* slots,
                               const int32_t* offsets, const int32_t* pos, int n, int total, const void* k, const void* v,
                               long long ks, long long vs, cudaStream_t s);

// Queries and keys turned by their positions (rotary.cu); append: keys and values into the cache's pages.
struct RotaryArgs {
  moe_rotary rot;
  const void *q, *k, *v;
  long long qs, ks, vs;  // token strides in elements
  const void *qw, *kw;   // norm weights (nullptr: no norm)
  float eps, inv_d;      // inv_d: 1 / D
  void *qo, *ko;
  long long qos, kos;
  const int32_t* positions;
  int T, H, Hkv, D;
  int lpr_shift, groups;  // log2 of the lanes of a row; units of a token (rotary.cu)
  // append: token t's place comes from the cache's tables
  CacheView c;
  void *kp, *vp;  // the layer's pages
  const int32_t *slots, *offsets, *pos;
  int n;
  int* status;
};

cudaError_t launch_rotary(RotaryArgs& a, int dt, cudaStream_t s);
cudaError_t launch_cache_append(RotaryArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ device helpers
// Positions that a slot holds: none if the slot or its length is out of range (recorded where the rows' own positions
// are read).
__device__ __forceinline__ int slot_len(const CacheView& c, int s) {
  if (s < 0 || s >= c.n_slots) return 0;
  const int len = c.lens[s];
  return len < 0 || (long long)len > (long long)c.width << c.page_shift ? 0 : len;
}
// That slot slots[i] holds the pages of the call's first slot at the shared positions, as far as it reaches, and that
// the first slot has them all; by threads `me` of `all`. A row that does not is recorded.
__device__ __forceinline__ void check_shared(const DecodeArgs& a, int i, int me, int all) {
  const CacheView& c = a.c;
  const int s0 = a.lead[0], s = a.slots[i], pages = a.shared >> c.page_shift;
  if (s0 < 0 || s0 >= c.n_slots) return;
  const int held = (slot_len(c, s0) + c.page_size - 1) >> c.page_shift;
  if (held < pages && a.first + i == 0 && me == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, 0);
  const int end = min(pages, min(held, (slot_len(c, s) + c.page_size - 1) >> c.page_shift));
  const int32_t *lead = c.table + (long long)s0 * c.width, *row = c.table + (long long)s * c.width;
  for (int p = me; p < end; p += all) {
    const int page = row[p];
    if (page < 0 || page >= c.n_pages || page != lead[p]) record_error(a.status, MOE_ERR_DEVICE_CHECK, a.first + i);
  }
}

inline long long prompt_tile_slots(int Tq, int n, int G, int R) { return (long long)Tq * G / R + n; }

// Sequence i of a prompt call, its offsets checked (a bad one is recorded and has no rows).
struct Seq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Seq load_seq(const PromptArgs& a, int i) {
  Seq s;
  s.q0 = a.qo[i];
  s.k0 = a.ko[i];
  const int q1 = a.qo[i + 1], k1 = a.ko[i + 1];
  s.nq = q1 - s.q0;
  s.nk = k1 - s.k0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.Tq || s.k0 < 0 || k1 < s.k0 || k1 > a.Tkv) {
    record_error(a.status, MOE_ERR_DEVICE_CHECK, i);
    s.nq = 0;
    s.nk = 0;
  }
  return s;
}
// Sequence i of a chunk call: its keys are the positions of its slot (k0). A slot or length out of range is recorded, and
// its rows see nothing.
__device__ __forceinline__ Seq load_chunk_seq(const PromptArgs& a, const DecodeArgs& d, int i) {
  Seq s;
  s.q0 = a.qo[i];
  const int q1 = a.qo[i + 1];
  s.nq = q1 - s.q0;
  s.k0 = d.slots[i];
  s.nk = slot_len(d.c, s.k0);
  if (bad_offsets(s.q0, q1, a.Tq)) {
    record_error(a.status, MOE_ERR_DEVICE_CHECK, i);
    s.nq = 0;
    s.nk = 0;
  } else if (s.nk == 0 && s.nq > 0 && (s.k0 < 0 || s.k0 >= d.c.n_slots || d.c.lens[s.k0] != 0)) {
    record_error(a.status, MOE_ERR_DEVICE_CHECK, i);
  }
  return s;
}
// The same by a warp: 32 places a step, and the four offsets in one load.
// (slot: 1 where every sequence has a slot of its own besides its tiles, 0 to find a token's sequence.)
__device__ __forceinline__ int find_tile_seq_warp(const int32_t* qo, int n, int G, int R, long long s, int slot = 1) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32, i = lo + lane * step;
    const bool at = lane * step < len && (long long)qo[i] * G / R + slot * i <= s;
    const int k = __popc(__ballot_sync(0xffffffffu, at)) - 1;  // (the first place always is, but for bad offsets)
    const int skip = (k < 0 ? 0 : k) * step;
    lo += skip;
    len = len - skip < step ? len - skip : step;
  }
  return lo;
}
__device__ __forceinline__ Seq load_seq_warp(const PromptArgs& a, int i) {
  const int lane = threadIdx.x & 31;
  const int v = (lane & 2 ? a.ko : a.qo)[i + (lane & 1)];
  Seq s;
  s.q0 = __shfl_sync(0xffffffffu, v, 0);
  s.k0 = __shfl_sync(0xffffffffu, v, 2);
  const int q1 = __shfl_sync(0xffffffffu, v, 1), k1 = __shfl_sync(0xffffffffu, v, 3);
  s.nq = q1 - s.q0;
  s.nk = k1 - s.k0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.Tq || s.k0 < 0 || k1 < s.k0 || k1 > a.Tkv) {
    if (lane == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, i);
    s.nq = 0;
    s.nk = 0;
  }
  return s;
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// try_wait that may sleep for up to 20 us. Without the hint it comes back after some tens of cycles, and warps that
// spin on it fill the queue that the MMA warp's own instructions pass through.
__device__ __forceinline__ bool mbar_try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// wait_or_abort for a whole converged warp: every branch is on a vote, so the warp never diverges, and what
// follows a wait of more than 20 us is laid out away from the loop that waits (an instruction cache miss costs
// the MMA warp more than the wait itself).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag,
                                          int* status, int role) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity)), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > timeout_ns)) {
      if ((threadIdx.x & 31) == 0) {
        record_error(status, MOE_ERR_DEVICE_TIMEOUT, role);
        *abort_flag = 1;
      }
      return false;
    }
  }
}
// A running reference rises with a score that is this much above it: 8 in log2 units (weights then stay below 2^8).
// Finite, as -inf plus it is to be -inf (c2, the scale times log2 e, may be next to 0).
__device__ __forceinline__ float rescale_above(float c2) { return fminf(8.0f / c2, 3.0e38f); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // the hardware 2^x, ~2 ulp; 2^-inf = 0
  return y;
}

// ------------------------------------------------------------------ rows that an unseen value made NaN
// A tile of the tensor cores multiplies the values of columns that a row does not see by a weight of 0, which makes NaN
// of a value that is not finite. The columns d of the head that this can touch are known: those with such a value in
// V[lim .. end) (the row sees lim keys, the tile's products took end). Their results are replaced, by a warp:
//   - where the row sees values that are not finite in d too, by what these add up to with weights above 0
//     (NaN, or an infinity),
//   - else by sum_j 2^(c q.k_j - c m) v_j[d] with the row's own m, every key computed again.
// Everything else the row already has is right. So the keys are only computed again for rows near the first such value
// of a column, and the two scans of V go on from row to row. (With every row that was not finite computed again over
// all its keys, one infinity made 8192 tokens of 32 heads of 128 take 200 ms instead of 0.4. One near the end takes 25
// ms now, 120 then.)
// A lane has columns 8 lane .. 8 lane + 7. at(j, ko, vo): the element offsets of key j.
struct Unseen {
  int from, upto;   // V has been looked through in [from, end) and in [0, upto)
  int last[8];      // the last key of the first stretch whose value is not finite
  uint32_t seen;    // of the second: a bit a column, 8 of NaN, 8 of +inf, 8 of -inf
  __device__ __forceinline__ explicit Unseen(int end) : from(end), upto(0), seen(0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) last[e] = -1;
  }
};
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
}
// found(e, bits, j) for every value in [a, b) that is not finite; more(): goes on
template <typename At, typename Found, typename More>
__device__ __forceinline__ int scan_values(const __nv_bfloat16* v, At at, int D, int a, int b, Found found, More more) {
  const int d = (int)(threadIdx.x & 31) * 8;
  int j = a;
  while (j < b && more()) {
    uint4 u[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      long long ko, vo;
      at(j + min(y, b - 1 - j), ko, vo);
      u[y] = d < D ? *reinterpret_cast<const uint4*>(v + vo + d) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      if (!not_finite2(u[y].x) && !not_finite2(u[y].y) && !not_finite2(u[y].z) && !not_finite2(u[y].w)) continue;
      const uint32_t w[4] = {u[y].x, u[y].y, u[y].z, u[y].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
        if ((h & 0x7F80u) == 0x7F80u) found(e, h, j + min(y, b - 1 - j));
      }
    }
    j += min(8, b - j);
  }
  return j;
}
// The columns of a row to replace (a bit each) and their sums, not yet divided. mc: m times scale * log2 e, 0 for -inf.
template <typename At>
__device__ __forceinline__ uint32_t replace_unseen(Unseen& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                   const __nv_bfloat16* v, At at, int D, int lim, float c2, float mc,
                                                   float (&o)[8]) {
  if (lim < s.from) {
    scan_values(v, at, D, lim, s.from, [&](int e, uint32_t, int j) { s.last[e] = max(s.last[e], j); }, [] { return true; });
    s.from = lim;
  }
  uint32_t cols = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) cols |= (s.last[e] >= lim ? 1u : 0u) << e;
  if (!__any_sync(0xffffffffu, cols != 0)) return 0;
  if (s.upto > lim) {  // (rows in another order than their limits)
    s.upto = 0;
    s.seen = 0;
  }
  s.upto = scan_values(
      v, at, D, s.upto, lim,
      [&](int e, uint32_t h, int) { s.seen |= (1u << e) << ((h & 0x7FFFu) > 0x7F80u ? 0 : (h & 0x8000u) ? 16 : 8); },
      [&] { return __any_sync(0xffffffffu, (cols & ~s.seen) != 0) != 0; });
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  const uint32_t odd = (s.seen | s.seen >> 8 | s.seen >> 16) & 0xFFu;
  if (__any_sync(0xffffffffu, (cols & ~odd) != 0)) {
    const int lane = (int)(threadIdx.x & 31), d = lane * 8;
    for (int j0 = 0; j0 < lim; j0 += min(32, lim - j0)) {
      long long ko, vo;
      at(j0 + min(lane, lim - 1 - j0), ko, vo);
      float x = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(q + c), b = *reinterpret_cast<const uint4*>(k + ko + c);
        x = fmaf(bf16lo(a.x), bf16lo(b.x), x); x = fmaf(bf16hi(a.x), bf16hi(b.x), x);
        x = fmaf(bf16lo(a.y), bf16lo(b.y), x); x = fmaf(bf16hi(a.y), bf16hi(b.y), x);
        x = fmaf(bf16lo(a.z), bf16lo(b.z), x); x = fmaf(bf16hi(a.z), bf16hi(b.z), x);
        x = fmaf(bf16lo(a.w), bf16lo(b.w), x); x = fmaf(bf16hi(a.w), bf16hi(b.w), x);
      }
      const float p = lane < lim - j0 ? ex2(fmaf(x, c2, -mc)) : 0.f;
#pragma unroll 8
      for (int y = 0; y < 32; ++y) {
        const float py = __shfl_sync(0xffffffffu, p, y);
        const long long vy = __shfl_sync(0xffffffffu, vo, y);
        const uint4 u = d < D ? *reinterpret_cast<const uint4*>(v + vy + d) : make_uint4(0u, 0u, 0u, 0u);
        o[0] = fmaf(py, bf16lo(u.x), o[0]); o[1] = fmaf(py, bf16hi(u.x), o[1]);
        o[2] = fmaf(py, bf16lo(u.y), o[2]); o[3] = fmaf(py, bf16hi(u.y), o[3]);
        o[4] = fmaf(py, bf16lo(u.z), o[4]); o[5] = fmaf(py, bf16hi(u.z), o[5]);
        o[6] = fmaf(py, bf16lo(u.w), o[6]); o[7] = fmaf(py, bf16hi(u.w), o[7]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if ((odd >> e & 1u) == 0) continue;
    const bool nan = s.seen >> e & 1u, up = s.seen >> (8 + e) & 1u, down = s.seen >> (16 + e) & 1u;
    o[e] = nan || (up && down) ? __int_as_float(0x7FFFFFFF) : up ? INFINITY : -INFINITY;
  }
  return cols;
}

}  // namespace moe

// Attention on the CUDA cores, fp32 arithmetic throughout: fp32 tensors, and the own positions of a decode batch of
// bf16 heads of more than 128 (whose prompts and shared positions attn_mma.cu takes).
//   out[r] = sum_{j < lim(r)} softmax_j(scale q[r] . k[j]) v[j]
// Scores are kept in log2 units (times scale * log2 e), so a weight is one 2^x. Keys past a row's limit are left
// out of both products by index, not by a zero weight, so that a non-finite value there stays there.
//
// attn_tile_kernel: 64 packed rows (see PromptArgs) of one key/value head against tiles of 64 keys, all in shared
// memory in fp32: packed prompts, and the shared positions of a decode batch (rows: every sequence's heads). 8
// threads share a row, each with 4 rows x 8 keys of the scores and 4 rows x D / 8 columns of the output in registers.
// Bound by reads of shared memory: a warp's 16-byte read takes four cycles whatever its lanes share, so an
// element of the scores costs (4 + 8) * 4 cycles for 32 of arithmetic, one of the output 20 for 16; with 2 rows a
// thread that was 40 for 16. Rows in shared memory have a length known to the compiler (D rounded up to 32, zeros
// past D): with D in the addresses and a test of each column the loops took 1.5 times as long. The weights take the
// place of the keys once the scores are done; two CTAs then fit on an SM and one computes while the other loads.
// Measured, fp32: 4096 tokens, 32 heads of 128 on 8: 3.04 ms, 45 TFLOP/s; heads of 64: 39 TFLOP/s.
//
// decode_rows_kernel: the positions that a sequence does not share, an HBM stream that meets up to 8 rows, far too
// few for tiles. Lanes lie along a head's elements; a warp takes 4 keys at a time straight from memory, its rows'
// products with them are summed over the lanes in one exchange (each step halves the values a lane holds: 31
// shuffles for 32 sums), which leaves each lane one score. Keys are split over warps and CTAs, whose pieces join in
// a fixed order. Bound by latency, each warp loading and computing in turn; the launch bounds are what measured
// best. fp32, heads of 128, 4096 positions: 32 sequences of 8 heads 187 us (5.7 TB/s), 8 of 32 heads on 8 61 us (4.4
// TB/s), 8 of 64 on 8 85 us; bf16, heads of 256, 16 on 4: 64 sequences 259 us (4.2 TB/s).
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float4 load4f(const T* p);
template <>
__device__ __forceinline__ float4 load4f<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4f<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
// 4 elements to shared memory, waited for with the group.
__device__ __forceinline__ void stage4(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <typename T> __device__ __forceinline__ void store_result(T* p, float x) { *p = from_f32<T>(x); }

// ------------------------------------------------------------------ tiles
constexpr int kRows = 64, KT = 64, kThreads = 128;
constexpr int TX = 8;               // threads of a row
constexpr int RPT = kRows * TX / kThreads, KPT = KT / TX;
constexpr int kLdP = KT + 4;
constexpr int kMaxCluster = 8;

// DP: D rounded up to a multiple of 32; the elements past D are zeros in shared memory.
constexpr int tile_keys(int DP) { return KT * (DP + 4) > kRows * kLdP ? KT * (DP + 4) : kRows * kLdP; }
constexpr size_t tile_smem(int DP) { return sizeof(float) * ((size_t)(kRows + KT) * (DP + 4) + tile_keys(DP)); }

// SHARED: rows and keys of a decode call, in pieces. SPLIT: a tile's keys over a cluster (in a kernel without it the
// code for it would cost registers and 3% of the time).
// PAGED: a chunk's rows over its slots' positions in the cache, in blockIdx.z pieces where there are several. A tile's
// rows are looked up in the table once. 256 tokens behind 2048, 16 heads of 128 on 4: 102 us, 26 TFLOP/s, bound like
// prompts by shared memory and issue.
template <int DP, bool SHARED, bool SPLIT, bool PAGED>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1)
attn_tile_kernel(const __grid_constant__ PromptArgs pa, const __grid_constant__ SharedPart sp) {
  constexpr int NC = DP / (4 * TX);  // groups of 4 columns of a thread
  extern __shared__ __align__(16) float sm[];
  __shared__ long long row_at[PAGED ? KT : 1];  // PAGED: where the tile's rows lie (found once, not for every 16 bytes)
  griddep_wait();
  griddep_launch_dependents();  // after the wait: the own positions' kernel relies on it
  const DecodeArgs& da = sp.d;
  const int H = SHARED ? da.H : pa.H, Hkv = SHARED ? da.c.Hkv : pa.Hkv, D = SHARED ? da.c.D : pa.D;
  const int G = H / Hkv, hk = blockIdx.y, tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
  constexpr int LD = DP + 4, d4 = DP / 4;
  float* Qs = sm;
  float* Ks = Qs + kRows * LD;
  float* Ps = Ks;  // [kRows][kLdP], once the scores are done
  float* Vs = Ks + tile_keys(DP);

  // ---- which rows, which keys
  int row0, nrows, j_begin, j_end, seq = 0;
  Seq sq{0, 0, 0, 0};
  const int32_t* pages = nullptr;
  if (SHARED) {
    row0 = blockIdx.x * kRows;
    nrows = min(kRows, da.n * G - row0);
    j_begin = min(da.shared, (int)blockIdx.z * sp.per);
    j_end = min(da.shared, j_begin + sp.per);
    const int s0 = da.lead[0];  // an out-of-range slot or page is recorded by the own part
    pages = da.c.table + (long long)(s0 < 0 || s0 >= da.c.n_slots ? 0 : s0) * da.c.width;
  } else {
    const int slot = gridDim.x - 1 - blockIdx.x;  // a prompt's last rows see the most keys: they start first
    // (Bad offsets' own slot may be found by nobody: CTA i looks at sequence i's, asked for here and looked at once the
    // slot's are there.)
    const int own = PAGED ? min((int)blockIdx.x, pa.n - 1) : 0;
    const int own0 = PAGED ? pa.qo[own] : 0, own1 = PAGED ? pa.qo[own + 1] : 0;
    seq = find_tile_seq(pa.qo, pa.n, G, kRows, slot);
    sq = PAGED ? load_chunk_seq(pa, da, seq) : load_seq(pa, seq);
    if (PAGED && bad_offsets(own0, own1, pa.Tq)) record_error(pa.status, MOE_ERR_DEVICE_CHECK, own);
    if (PAGED) pages = da.c.table + (long long)sq.k0 * da.c.width;
    const long long first = (long long)sq.q0 * G / kRows + seq;
    const long long r0 = ((long long)slot - first) * kRows;
    if (r0 < 0 || r0 >= (long long)sq.nq * G) return;
    row0 = (int)r0;
    nrows = min(kRows, sq.nq * G - row0);
    const int keys = visible_keys((row0 + nrows - 1) / G, sq.nq, sq.nk, pa.causal);
    const int per = ((keys - 1) / KT / (int)gridDim.z + 1) * KT;  // of each CTA of the cluster
    j_begin = (int)min((long long)keys, (long long)blockIdx.z * per);
    j_end = (int)min((long long)keys, (long long)j_begin + per);
  }
  const float c2 = (SHARED ? da.scale : pa.scale) * 1.4426950408889634f;
  const float* qsrc = (const float*)(SHARED ? da.q : pa.q);
  const long long qs = SHARED ? da.qs : pa.qs;
  for (int i = tid; i < kRows * d4; i += kThreads) {
    const int r = i / d4, c = (i % d4) * 4, R = row0 + min(r, nrows - 1);
    const float* row = qsrc + (long long)(sq.q0 + R / G) * qs + (long long)(hk * G + R % G) * D;
    stage4(Qs + r * LD + c, row + min(c, D - 4), r < nrows && c < D);
  }

  float m[RPT], l[RPT];
  int lim[RPT];
  uint64_t o[RPT][NC][2];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    const int R = ty * RPT + r;
    lim[r] = 0;
    if (R < nrows && SHARED) {  // a slot shorter than the shared positions sees its own length of them
      lim[r] = min(j_end, slot_len(da.c, da.slots[(row0 + R) / G]));
    } else if (R < nrows) {
      lim[r] = visible_keys((row0 + R) / G, sq.nq, sq.nk, pa.causal);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) o[r][c][0] = o[r][c][1] = 0ull;
  }

  const float* kb = (const float*)(SHARED || PAGED ? da.k : pa.k);
  const float* vb = (const float*)(SHARED || PAGED ? da.v : pa.v);
  // (what is left counts down: positions near 2^31 must not wrap)
  for (int j0 = j_begin, left = j_end - j_begin; left > 0; j0 += KT, left -= KT) {
    if (PAGED && tid < KT && tid < left) {  // (the tile before is past its loads)
      const int j = j0 + tid;
      int page = pages[j >> da.c.page_shift];
      if (page < 0 || page >= da.c.n_pages) {
        record_error(pa.status, MOE_ERR_DEVICE_CHECK, seq);
        page = 0;
      }
      row_at[tid] = (((long long)page * Hkv + hk) * da.c.page_size + (j & (da.c.page_size - 1))) * D;
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // K, then V
      float* dst = half ? Vs : Ks;
      const float* src = half ? vb : kb;
      const long long stride = SHARED || PAGED ? 0 : (half ? pa.vs : pa.ks);
      for (int i = tid; i < KT * d4; i += kThreads) {
        const int r = i / d4, c = (i % d4) * 4, j = j0 + min(r, left - 1), ce = min(c, D - 4);
        long long at;
        if (PAGED) {
          at = row_at[min(r, left - 1)] + ce;
        } else if (SHARED) {
          int page = pages[j >> da.c.page_shift];
          page = page < 0 || page >= da.c.n_pages ? 0 : page;
          at = (((long long)page * Hkv + hk) * da.c.page_size + (j & (da.c.page_size - 1))) * D + ce;
        } else {
          at = (long long)(sq.k0 + j) * stride + (long long)hk * D + ce;
        }
        stage4(dst + r * LD + c, src + at, r < left && c < D);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    // ---- scores of rows ty * RPT + r and keys tx + TX * k
    float sc[RPT][KPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int k = 0; k < KPT; ++k) sc[r][k] = 0.f;
#pragma unroll 2
    for (int d = 0; d < DP; d += 4) {
      float4 q[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) q[r] = *reinterpret_cast<const float4*>(Qs + (ty * RPT + r) * LD + d);
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const float4 kk = *reinterpret_cast<const float4*>(Ks + (tx + TX * k) * LD + d);
#pragma unroll
        for (int r = 0; r < RPT; ++r)
          sc[r][k] = fmaf(q[r].w, kk.w, fmaf(q[r].z, kk.z, fmaf(q[r].y, kk.y, fmaf(q[r].x, kk.x, sc[r][k]))));
      }
    }
    __syncthreads();  // the keys' place is free
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      float s[KPT], mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        s[k] = tx + TX * k < lim[r] - j0 ? sc[r][k] * c2 : -INFINITY;
        mx = fmaxf(mx, s[k]);
      }
#pragma unroll
      for (int w = TX / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[r], mx), ref = mn == -INFINITY ? 0.f : mn;  // no key yet: every weight is 0
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const float p = ex2(s[k] - ref);
        sum += p;
        Ps[(ty * RPT + r) * kLdP + tx + TX * k] = p;
      }
#pragma unroll
      for (int w = TX / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const float al = ex2(m[r] - ref);
      l[r] = l[r] * al + sum;
      m[r] = mn;
      const uint64_t al2 = f2_pack(al, al);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        o[r][c][0] = ffma2(o[r][c][0], al2, 0ull);
        o[r][c][1] = ffma2(o[r][c][1], al2, 0ull);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the values are there (a row's weights are written and read by the same warp)
    // ---- o += p v: columns 4 tx + 4 TX c
    int kmin = KT, kmax = 0;  // every row of the thread sees the keys below kmin, none those from kmax on
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int x = max(0, min(KT, lim[r] - j0));
      kmin = min(kmin, x);
      kmax = max(kmax, x);
    }
    kmin &= ~3;
    for (int kk = 0; kk < kmin; kk += 4) {
      float4 p[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) p[r] = *reinterpret_cast<const float4*>(Ps + (ty * RPT + r) * kLdP + kk);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint64_t pp[RPT];
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const float x = y == 0 ? p[r].x : y == 1 ? p[r].y : y == 2 ? p[r].z : p[r].w;
          pp[r] = f2_pack(x, x);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(Vs + (kk + y) * LD + tx * 4 + 4 * TX * c);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            o[r][c][0] = ffma2(pp[r], v.x, o[r][c][0]);
            o[r][c][1] = ffma2(pp[r], v.y, o[r][c][1]);
          }
        }
      }
    }
    for (int kk = kmin; kk < kmax; ++kk) {
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        if (kk >= lim[r] - j0) continue;
        const float x = Ps[(ty * RPT + r) * kLdP + kk];
        const uint64_t pp = f2_pack(x, x);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(Vs + kk * LD + tx * 4 + 4 * TX * c);
          o[r][c][0] = ffma2(pp, v.x, o[r][c][0]);
          o[r][c][1] = ffma2(pp, v.y, o[r][c][1]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  if (SPLIT) {
    // The cluster's CTAs hold parts of the same rows over different keys: they put them in shared memory, and each
    // adds up every C-th row from all of them, in order.
    const int C = gridDim.z, rank = (int)cluster_ctarank();
    __syncthreads();
    float* po = Qs;
    float2* ml = reinterpret_cast<float2*>(Vs);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int R = ty * RPT + r;
      if (tx == 0) ml[R] = make_float2(m[r], l[r]);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<ulonglong2*>(po + R * LD + tx * 4 + 4 * TX * c) = make_ulonglong2(o[r][c][0], o[r][c][1]);
    }
    cluster_sync_all();
    for (int i = tid; i < kRows / C * d4; i += kThreads) {
      const int R = rank + C * (i / d4), c = (i % d4) * 4;
      if (R >= nrows || c >= D) continue;
      float2 v[kMaxCluster];
      float4 u[kMaxCluster];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int y = 0; y < kMaxCluster; ++y) {
        if (y >= C) break;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[y].x), "=f"(v[y].y)
                     : "r"(map_to_cta(smem_u32(ml + R), (uint32_t)y)) : "memory");
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u[y].x), "=f"(u[y].y), "=f"(u[y].z), "=f"(u[y].w)
                     : "r"(map_to_cta(smem_u32(po + R * LD + c), (uint32_t)y)) : "memory");
        M = fmaxf(M, v[y].x);
      }
      const float ref = M == -INFINITY ? 0.f : M;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kMaxCluster; ++y) {
        if (y >= C) break;
        const float w = ex2(v[y].x - ref);  // (no key: 0, and the sums are 0)
        L = fmaf(w, v[y].y, L);
        t.x = fmaf(w, u[y].x, t.x);
        t.y = fmaf(w, u[y].y, t.y);
        t.z = fmaf(w, u[y].z, t.z);
        t.w = fmaf(w, u[y].w, t.w);
      }
      const float inv = L == 0.f ? 0.f : 1.0f / L;
      const int P = row0 + R, tok = sq.q0 + P / G, h = hk * G + P % G;
      float* dst = (float*)pa.out + (long long)tok * pa.os + (long long)h * D + c;
      store_result(dst, t.x * inv);
      store_result(dst + 1, t.y * inv);
      store_result(dst + 2, t.z * inv);
      store_result(dst + 3, t.w * inv);
      if (pa.lse != nullptr && c == 0)
        pa.lse[(long long)tok * H + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    cluster_sync_all();  // the others have read this CTA's part
    return;
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int R = ty * RPT + r;
    if (R >= nrows) continue;
    const int P = row0 + R, tok = sq.q0 + P / G, h = hk * G + P % G;
    if (SHARED || (PAGED && gridDim.z > 1)) {
      float* po = da.part + (((long long)tok * H + h) * sp.pieces + blockIdx.z) * (D + 2);
      if (tx == 0) *reinterpret_cast<float2*>(po + D) = make_float2(m[r], l[r]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (tx * 4 + 4 * TX * c >= D) continue;
        *reinterpret_cast<uint64_t*>(po + tx * 4 + 4 * TX * c) = o[r][c][0];
        *reinterpret_cast<uint64_t*>(po + tx * 4 + 4 * TX * c + 2) = o[r][c][1];
      }
      continue;
    }
    const float inv = l[r] == 0.f ? 0.f : 1.0f / l[r];
    float* dst = (float*)pa.out + (long long)tok * pa.os + (long long)h * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (tx * 4 + 4 * TX * c >= D) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        store_result(dst + tx * 4 + 4 * TX * c + e, (e & 1 ? f2_hi(o[r][c][e / 2]) : f2_lo(o[r][c][e / 2])) * inv);
    }
    if (pa.lse != nullptr && tx == 0)
      pa.lse[(long long)tok * H + h] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------ few rows
constexpr int kRowWarps = 4;
constexpr int NK = 4;  // keys of a warp's step
// From this many sequences on the shared positions are read once for all by tiles; fewer read them each. 4096 shared, 4
// key/value heads, in a graph: fp32 heads of 128, 4 sequences 21 us by tiles, 18 each, 8 sequences 21 and 26; bf16
// heads of 256, 2 sequences 16 and 15, 3 sequences 16 and 20.
constexpr int kSharedFromF32 = 6, kSharedFromBf16 = 3;

// V4: groups of 4 elements of a lane, 16 bytes side by side (fp32: elements 4 lane + 128 x, bf16: 8 lane + 4 x); GR:
// rows of a CTA.
template <typename T, int V4, int GR>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 2 ? 4 : V4 == 2 ? 3 : GR == 8 ? 4 : 5)
decode_rows_kernel(const __grid_constant__ DecodeArgs a, int groups, int first_piece, int splits, int pieces) {
  constexpr int NV = GR * NK;  // products of a step
  static_assert(NV == 32 || NV == 16, "one or two lanes a score");
  __shared__ __align__(16) float2 ps[kRowWarps][NV];  // each weight twice, a packed factor
  __shared__ float sml[2][kRowWarps][GR];
  __shared__ __align__(16) float buf[kRowWarps][GR][V4 * 128];
  // Behind the shared positions' kernel (first_piece > 0) this one need not wait for it: that kernel lets dependents
  // start only once it has itself waited for everything before it, and only the join reads what it writes.
  if (first_piece == 0) griddep_wait();
  griddep_launch_dependents();
  const CacheView& c = a.c;
  const int G = a.H / c.Hkv, D = c.D, hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.x / groups, row0 = (blockIdx.x % groups) * GR, nrows = min(GR, G - row0);
  const int from = first_piece > 0 ? a.shared : 0;
  const int slot = a.slots[seq], len = slot_len(c, slot);
  if (tid == 0 && len == 0 && (slot < 0 || slot >= c.n_slots || c.lens[slot] != 0))
    record_error(a.status, MOE_ERR_DEVICE_CHECK, seq);
  const int32_t* pages = c.table + (long long)slot * c.width;
  if (a.shared > 0 && blockIdx.y == 0 && blockIdx.z == 0 && row0 == 0)
    check_shared(a, seq, tid, 32 * kRowWarps);
  // this CTA's keys, then this warp's: NK at a time, the warps in turn
  const int own = max(0, len - from), step = NK * kRowWarps;
  const int per = (int)(((long long)own + splits - 1) / splits + step - 1) / step * step;
  const int j_begin = from + (int)min((long long)own, (long long)blockIdx.z * per), j_end = min(from + own, j_begin + per);

  constexpr bool kHalf = sizeof(T) == 2;
  static_assert(!kHalf || V4 == 2, "16 bytes a lane");
  auto col = [&](int x) { return kHalf ? 8 * lane + 4 * x : 4 * lane + 128 * x; };
  uint64_t q[GR][V4][2], o[GR][V4][2];
  const T* qp = (const T*)a.q + (long long)seq * a.qs + (long long)(hk * G + row0) * D;
#pragma unroll
  for (int r = 0; r < GR; ++r)
#pragma unroll
    for (int x = 0; x < V4; ++x) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows && col(x) < D) t = load4f<T>(qp + (long long)r * D + col(x));
      q[r][x][0] = f2_pack(t.x, t.y);
      q[r][x][1] = f2_pack(t.z, t.w);
      o[r][x][0] = o[r][x][1] = 0ull;
    }
  const float c2 = a.scale * 1.4426950408889634f;
  // this lane's score: row my_row, key my_key of the step
  const int idx = NV == 32 ? lane : lane >> 1, my_row = idx % GR, my_key = idx / GR;
  float m = -INFINITY, l = 0.f;  // of my_row
  const T* kb = (const T*)a.k;
  const T* vb = (const T*)a.v;
  int page[NK];
  auto look_up = [&](int j) {
#pragma unroll
    for (int k = 0; k < NK; ++k) page[k] = k < j_end - j ? pages[(j + k) >> c.page_shift] : 0;
  };
  int left = j_end - j_begin - warp * NK;
  int j = j_begin + warp * NK;
  if (left > 0) look_up(j);
  for (; left > 0; left -= step, j += step) {
    uint64_t kv[NK][V4][2], vv[NK][V4][2];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      int p = page[k];
      if (p < 0 || p >= c.n_pages) {
        if (lane == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, seq);
        p = 0;
      }
      const long long at = (((long long)p * c.Hkv + hk) * c.page_size + ((j + k) & (c.page_size - 1))) * D;
      if constexpr (kHalf) {
        const bool in = k < left && 8 * lane < D;
        const uint4 ke = in ? *reinterpret_cast<const uint4*>(kb + at + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 ve = in ? *reinterpret_cast<const uint4*>(vb + at + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
        kv[k][0][0] = f2_pack(bf16lo(ke.x), bf16hi(ke.x));
        kv[k][0][1] = f2_pack(bf16lo(ke.y), bf16hi(ke.y));
        kv[k][1][0] = f2_pack(bf16lo(ke.z), bf16hi(ke.z));
        kv[k][1][1] = f2_pack(bf16lo(ke.w), bf16hi(ke.w));
        vv[k][0][0] = f2_pack(bf16lo(ve.x), bf16hi(ve.x));
        vv[k][0][1] = f2_pack(bf16lo(ve.y), bf16hi(ve.y));
        vv[k][1][0] = f2_pack(bf16lo(ve.z), bf16hi(ve.z));
        vv[k][1][1] = f2_pack(bf16lo(ve.w), bf16hi(ve.w));
      } else {
#pragma unroll
        for (int x = 0; x < V4; ++x) {
          const bool in = k < left && col(x) < D;
          const float4 ke = in ? load4f<T>(kb + at + col(x)) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 ve = in ? load4f<T>(vb + at + col(x)) : make_float4(0.f, 0.f, 0.f, 0.f);
          kv[k][x][0] = f2_pack(ke.x, ke.y);
          kv[k][x][1] = f2_pack(ke.z, ke.w);
          vv[k][x][0] = f2_pack(ve.x, ve.y);
          vv[k][x][1] = f2_pack(ve.z, ve.w);
        }
      }
    }
    if (left > step) look_up(j + step);
    float v[NV];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int r = 0; r < GR; ++r) {
        uint64_t t = 0ull;
#pragma unroll
        for (int x = 0; x < V4; ++x) t = ffma2(q[r][x][1], kv[k][x][1], ffma2(q[r][x][0], kv[k][x][0], t));
        v[k * GR + r] = f2_lo(t) + f2_hi(t);
      }
#pragma unroll
    for (int half = NV / 2, w = 16; half > 0; half >>= 1, w >>= 1) {
      const bool up = lane & w;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
    }
    if (NV == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    const float s = my_key < left ? v[0] * c2 : -INFINITY;
    float mx = fmaxf(s, -INFINITY);  // (drops a NaN: the maximum is never NaN)
#pragma unroll
    for (int w = 32 / NK; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
    const float al = ex2(m - ref), p = ex2(s - ref);
    float sum = p;
#pragma unroll
    for (int w = 32 / NK; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * al + sum;
    if (__any_sync(0xffffffffu, mn > m))
#pragma unroll
      for (int r = 0; r < GR; ++r) {
        const float t = __shfl_sync(0xffffffffu, al, NV == 32 ? r : 2 * r);
#pragma unroll
        for (int x = 0; x < V4; ++x) {
          o[r][x][0] = ffma2(o[r][x][0], f2_pack(t, t), 0ull);
          o[r][x][1] = ffma2(o[r][x][1], f2_pack(t, t), 0ull);
        }
      }
    m = mn;
    __syncwarp();
    ps[warp][idx] = make_float2(p, p);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int r = 0; r < GR; r += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&ps[warp][k * GR + r]);
#pragma unroll
        for (int x = 0; x < V4; ++x) {
          o[r][x][0] = ffma2(w.x, vv[k][x][0], o[r][x][0]);
          o[r][x][1] = ffma2(w.x, vv[k][x][1], o[r][x][1]);
          o[r + 1][x][0] = ffma2(w.y, vv[k][x][0], o[r + 1][x][0]);
          o[r + 1][x][1] = ffma2(w.y, vv[k][x][1], o[r + 1][x][1]);
        }
      }
  }
  // ---- the warps' parts
  if (my_key == 0) {
    sml[0][warp][my_row] = m;
    sml[1][warp][my_row] = l;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < GR; ++r) {
    float M = -INFINITY;
#pragma unroll
    for (int y = 0; y < kRowWarps; ++y) M = fmaxf(M, sml[0][y][r]);
    const float w = M == -INFINITY ? 0.f : ex2(sml[0][warp][r] - M);
#pragma unroll
    for (int x = 0; x < V4; ++x)
      *reinterpret_cast<float4*>(&buf[warp][r][col(x)]) =
          sml[1][warp][r] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                 : make_float4(f2_lo(o[r][x][0]) * w, f2_hi(o[r][x][0]) * w, f2_lo(o[r][x][1]) * w,
                                               f2_hi(o[r][x][1]) * w);
  }
  __syncthreads();
  for (int i = tid; i < nrows * (D / 2); i += 32 * kRowWarps) {
    const int r = i / (D / 2), col = (i % (D / 2)) * 2, h = hk * G + row0 + r;
    float2 t = make_float2(0.f, 0.f);
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int y = 0; y < kRowWarps; ++y) {
      t.x += buf[y][r][col];
      t.y += buf[y][r][col + 1];
      M = fmaxf(M, sml[0][y][r]);
    }
#pragma unroll
    for (int y = 0; y < kRowWarps; ++y)
      if (M != -INFINITY) L += sml[1][y][r] * ex2(sml[0][y][r] - M);
    if (pieces > 1) {
      float* po = a.part + (((long long)seq * a.H + h) * pieces + first_piece + blockIdx.z) * (D + 2);
      *reinterpret_cast<float2*>(po + col) = t;
      if (col == 0) *reinterpret_cast<float2*>(po + D) = make_float2(M, L);
    } else {
      const float inv = L == 0.f ? 0.f : 1.0f / L;
      T* dst = (T*)a.out + (long long)seq * a.os + (long long)h * D + col;
      store_result<T>(dst, t.x * inv);
      store_result<T>(dst + 1, t.y * inv);
      if (a.lse != nullptr && col == 0)
        a.lse[(long long)seq * a.H + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  }
  if (first_piece > 0) griddep_wait();
}

// Joins a row's pieces in a fixed order, by WPR warps that take every WPR-th piece, eight on their way at a time: 4
// while there are few rows, 1 (four rows a CTA) when the rows alone fill the GPU. A lane holds elements 2 lane + 64
// x.
template <typename T, int WPR>
__global__ void __launch_bounds__(128)
decode_join_simt_kernel(const __grid_constant__ DecodeArgs a, int pieces) {
  __shared__ float2 part[WPR][4][32];
  __shared__ float part_l[WPR];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WPR, D = a.c.D;
  const long long row = (long long)blockIdx.x * (4 / WPR) + (threadIdx.x >> 5) / WPR;
  if (row >= (long long)a.n * a.H) return;  // (with WPR = 4 there is a CTA a row)
  const float* p = a.part + row * pieces * (D + 2);
  auto ml = [&](int i) { return *reinterpret_cast<const float2*>(p + (long long)i * (D + 2) + D); };
  float M = -INFINITY, l = 0.f;
  for (int i = lane; i < pieces; i += 32) M = fmaxf(M, ml(i).x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  float2 o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) o[x] = make_float2(0.f, 0.f);
  for (int i0 = warp; i0 < pieces; i0 += 32 * WPR) {  // lane: piece i0 + WPR lane
    const float2 v = i0 + WPR * lane < pieces ? ml(i0 + WPR * lane) : make_float2(-INFINITY, 0.f);
    const float wl = v.y == 0.f ? 0.f : ex2(v.x - ref);
    l += wl * v.y;
    for (int y0 = 0; y0 < 32 && i0 + WPR * y0 < pieces; y0 += 8) {
      float2 u[8][4];
#pragma unroll
      for (int y = 0; y < 8; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + WPR * (y0 + y);
          u[y][x] = i < pieces && 2 * lane + 64 * x < D
                        ? *reinterpret_cast<const float2*>(p + (long long)i * (D + 2) + 2 * lane + 64 * x) : make_float2(0.f, 0.f);
        }
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = __shfl_sync(0xffffffffu, wl, y0 + y);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[x].x = fmaf(w, u[y][x].x, o[x].x);
          o[x].y = fmaf(w, u[y][x].y, o[x].y);
        }
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  if (WPR > 1) {
#pragma unroll
    for (int x = 0; x < 4; ++x) part[warp][x][lane] = o[x];
    if (lane == 0) part_l[warp] = l;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int y = 1; y < WPR; ++y) {
      l += part_l[y];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        o[x].x += part[y][x][lane].x;
        o[x].y += part[y][x][lane].y;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  T* dst = (T*)a.out + (row / a.H) * a.os + (row % a.H) * D;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (2 * lane + 64 * x < D) {
      store_result<T>(dst + 2 * lane + 64 * x, o[x].x * inv);
      store_result<T>(dst + 2 * lane + 64 * x + 1, o[x].y * inv);
    }
  if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// A chunk's rows, whose keys were taken in `pieces` parts: a warp a row, the parts in their order. A lane holds elements
// 4 lane + 128 x. A row of no sequence (or of one with bad offsets) stays as it is. Tiles find a slot's sequence and the join a
// token's: over offsets out of order it may come to one whose tile nobody found, and whose pieces are another call's.
constexpr int kJoinThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
chunk_rows_join_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ DecodeArgs d, int pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, D = a.D;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  int i = min((int)threadIdx.x, a.n - 1);
  const int q0 = a.qo[i], q1 = a.qo[i + 1];  // (asked for ahead of the search)
  const int tok = (int)(row / a.H), h = (int)(row % a.H), seq = find_tile_seq_warp(a.qo, a.n, 1, 1, tok, 0);
  bool bad = bad_offsets(q0, q1, a.Tq);
#pragma unroll 1
  while ((i += kJoinThreads) < a.n) bad = bad || bad_offsets(a.qo[i], a.qo[i + 1], a.Tq);
  bad = __syncthreads_or(bad);
  if (row >= (long long)a.Tq * a.H) return;
  const Seq sq = load_chunk_seq(a, d, seq);
  if (tok < sq.q0 || tok >= sq.q0 + sq.nq) return;
  if (bad) {
    const int G = a.H / a.Hkv;
    const long long slot = (long long)sq.q0 * G / kRows + seq + ((long long)(tok - sq.q0) * G + h % G) / kRows;
    if (find_tile_seq(a.qo, a.n, G, kRows, slot) != seq) return;
  }
  const float* p = d.part + row * pieces * (D + 2);
  auto ml = [&](int i) { return *reinterpret_cast<const float2*>(p + (long long)i * (D + 2) + D); };
  float M = -INFINITY, l = 0.f;
  for (int i = lane; i < pieces; i += 32) M = fmaxf(M, ml(i).x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  float2 o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) o[x] = make_float2(0.f, 0.f);
  for (int i0 = 0; i0 < pieces; i0 += 32) {
    const float2 v = i0 + lane < pieces ? ml(i0 + lane) : make_float2(-INFINITY, 0.f);
    const float wl = v.y == 0.f ? 0.f : ex2(v.x - ref);
    l += wl * v.y;
    for (int y0 = 0; y0 < 32 && i0 + y0 < pieces; y0 += 4) {
      float2 u[4][4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          u[y][x] = i0 + y0 + y < pieces && 2 * lane + 64 * x < D
                        ? *reinterpret_cast<const float2*>(p + (long long)(i0 + y0 + y) * (D + 2) + 2 * lane + 64 * x)
                        : make_float2(0.f, 0.f);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float w = __shfl_sync(0xffffffffu, wl, y0 + y);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[x].x = fmaf(w, u[y][x].x, o[x].x);
          o[x].y = fmaf(w, u[y][x].y, o[x].y);
        }
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  T* dst = (T*)a.out + (long long)tok * a.os + (long long)h * D;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (2 * lane + 64 * x < D) {
      store_result<T>(dst + 2 * lane + 64 * x, o[x].x * inv);
      store_result<T>(dst + 2 * lane + 64 * x + 1, o[x].y * inv);
    }
  if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <int DP, bool SHARED, bool SPLIT, bool PAGED>
cudaError_t launch_tiles(const PromptArgs& pa, const SharedPart& sp, dim3 grid, cudaStream_t s) {
  auto kern = attn_tile_kernel<DP, SHARED, SPLIT, PAGED>;
  static std::atomic<int> done{0};
  const cudaError_t e = allow_smem(kern, tile_smem(DP), done);
  if (e != cudaSuccess) return e;
  if (!SPLIT) return launch_pdl(kern, grid, dim3(kThreads), tile_smem(DP), s, pa, sp);
  return launch_clusters(kern, grid, dim3(kThreads), dim3(1, 1, grid.z), tile_smem(DP), s, pa, sp);
}
template <bool SHARED, bool SPLIT, bool PAGED = false>
cudaError_t launch_tiles(const PromptArgs& pa, const SharedPart& sp, int D, dim3 grid, cudaStream_t s) {
  if (D <= 64) return launch_tiles<64, SHARED, SPLIT, PAGED>(pa, sp, grid, s);
  if (D <= 96) return launch_tiles<96, SHARED, SPLIT, PAGED>(pa, sp, grid, s);
  if (D <= 128) return launch_tiles<128, SHARED, SPLIT, PAGED>(pa, sp, grid, s);
  return D <= 192 ? launch_tiles<192, SHARED, SPLIT, PAGED>(pa, sp, grid, s)
                  : launch_tiles<256, SHARED, SPLIT, PAGED>(pa, sp, grid, s);
}

template <typename T, int V4, int GR>
cudaError_t launch_rows(const DecodeArgs& a, int first_piece, int splits, cudaStream_t s) {
  const int groups = (a.H / a.c.Hkv + GR - 1) / GR;
  const dim3 grid((unsigned)((long long)a.n * groups), (unsigned)a.c.Hkv, (unsigned)splits);
  return launch_pdl(decode_rows_kernel<T, V4, GR>, grid, dim3(32 * kRowWarps), 0, s, a, groups, first_piece, splits,
                    first_piece + splits);
}

template <typename T>
cudaError_t launch_join(const DecodeArgs& a, int pieces, cudaStream_t s) {
  const long long rows = (long long)a.n * a.H;
  if (rows <= 8 * device_sm_count())
    return launch_pdl(decode_join_simt_kernel<T, 4>, dim3((unsigned)rows), dim3(128), 0, s, a, pieces);
  return launch_pdl(decode_join_simt_kernel<T, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, pieces);
}

}  // namespace

cudaError_t launch_attn_prompt_simt(const PromptArgs& a, cudaStream_t s) {
  const long long slots = prompt_tile_slots(a.Tq, a.n, a.H / a.Hkv, kRows);
  const SharedPart none{};
  // Few tiles: a cluster of CTAs takes the keys of each, at least two tiles of them where the keys are one sequence's
  // (fp32, 1024 tokens of 8 heads of 128: 183 us without, 116 with two CTAs; 18 tokens of two sequences behind up to
  // 1100 keys: 98 without, 58 with eight).
  int C = 1;
  while (C < kMaxCluster && slots * a.Hkv * 2 * C <= 2LL * device_sm_count() && a.Tkv >= 4 * C * KT) C *= 2;
  const dim3 grid((unsigned)slots, (unsigned)a.Hkv, (unsigned)C);
  return C > 1 ? launch_tiles<false, true>(a, none, a.D, grid, s) : launch_tiles<false, false>(a, none, a.D, grid, s);
}

// Few tiles: a row's keys in pieces, about kPieceCtas CTAs an SM altogether, at least kPieceTiles tiles of keys each at the
// longest length that the cache may hold (lengths are only known on the device, and a piece behind its rows' last key
// ends at once). With longer pieces, and a row looked up for every 16 bytes of it, 2048 tokens behind 4096, 16 heads of
// 256 on 4, took 940 us, 446 so; 40 tokens of small fp32 heads 23 and 16.
constexpr int kPieceCtas = 8, kPieceTiles = 1;
int chunk_tile_pieces(const CacheView& c, int n, int Tq, int H) {
  const long long ctas = prompt_tile_slots(Tq, n, H / c.Hkv, kRows) * c.Hkv, rows = (long long)Tq * H;
  const long long most = ((long long)c.width * c.page_size + kPieceTiles * KT - 1) / (kPieceTiles * KT);
  const long long fit = rows > 0 ? decode_pieces(rows) / rows : 1;
  long long p = (long long)kPieceCtas * device_sm_count() / (ctas > 0 ? ctas : 1);
  p = p > most ? most : p;
  p = p > fit ? fit : p;
  return (int)(p < 1 ? 1 : p);
}
// fp32, up to 8 pieces of so few tiles that every CTA has an SM: a cluster of CTAs holds them in its shared memory, with no
// join behind. 40 tokens of 3 sequences, 4 heads of 32: 14.7 us so, 15.7 with a join; 24 of 6, 8 heads of 64, 10.4 and
// 12.1. (Clusters find no place in time where there are more: 64 tokens of 32 sequences, 16 heads of 128, 109 and 79.)
bool chunk_tiles_in_clusters(const CacheView& c, int n, int Tq, int H, int pieces) {
  return c.dt == MOE_DTYPE_F32 && pieces > 1 && pieces <= kMaxCluster &&
         prompt_tile_slots(Tq, n, H / c.Hkv, kRows) * c.Hkv * kMaxCluster <= device_sm_count();
}

cudaError_t launch_attn_chunk_tiles(const PromptArgs& a, const DecodeArgs& d, int pieces, cudaStream_t s) {
  SharedPart sp{};
  sp.d = d;
  sp.pieces = pieces;
  dim3 grid((unsigned)prompt_tile_slots(a.Tq, a.n, a.H / a.Hkv, kRows), (unsigned)a.Hkv, (unsigned)pieces);
  if (chunk_tiles_in_clusters(d.c, a.n, a.Tq, a.H, pieces)) {
    grid.z = pieces <= 2 ? 2 : pieces <= 4 ? 4 : 8;
    return launch_tiles<false, true, true>(a, sp, a.D, grid, s);
  }
  const cudaError_t e = a.dt == MOE_DTYPE_BF16 ? launch_attn_chunk_mma(a, sp, grid, s)
                                               : launch_tiles<false, false, true>(a, sp, a.D, grid, s);
  if (e != cudaSuccess || pieces == 1) return e;
  const dim3 rows((unsigned)(((long long)a.Tq * a.H + 3) / 4));
  return a.dt == MOE_DTYPE_BF16 ? launch_pdl(chunk_rows_join_kernel<__nv_bfloat16>, rows, dim3(kJoinThreads), 0, s, a, d, pieces)
                                : launch_pdl(chunk_rows_join_kernel<float>, rows, dim3(kJoinThreads), 0, s, a, d, pieces);
}

cudaError_t launch_attn_decode_simt(const DecodeArgs& a, cudaStream_t s) {
  const int G = a.H / a.c.Hkv, D = a.c.D, GR = D <= 128 && G > 4 ? 8 : 4, sms = device_sm_count();
  const long long rows = (long long)a.n * a.H, fit = decode_pieces(rows) / rows;
  const bool shared = a.shared > 0 && a.n >= (a.c.dt == MOE_DTYPE_BF16 ? kSharedFromBf16 : kSharedFromF32);
  // own positions: about 8 CTAs an SM, at least 64 positions each at the longest length
  const long long ctas = (long long)a.n * ((G + GR - 1) / GR) * a.c.Hkv;
  const long long most = (long long)a.c.width * a.c.page_size - (shared ? a.shared : 0);
  long long splits = (8LL * sms + ctas - 1) / ctas;
  const long long cap = (most + 63) / 64;
  splits = splits > cap ? cap : splits;
  splits = splits > fit / 2 ? fit / 2 : splits;
  splits = splits < 1 ? 1 : (splits > 65535 ? 65535 : splits);
  SharedPart sp{};
  cudaError_t e = cudaSuccess;
  if (shared) {
    const long long tiles = ((long long)a.n * G + kRows - 1) / kRows, tiles_kv = tiles * a.c.Hkv;
    const int blocks = (a.shared + KT - 1) / KT;
    long long n = (2LL * sms) / tiles_kv;
    n = n > fit / 2 ? fit / 2 : n;
    n = n < 1 ? 1 : (n > blocks ? blocks : n);
    const int per = (int)((blocks + n - 1) / n);
    sp.d = a;
    sp.per = per * KT;
    sp.splits = (blocks + per - 1) / per;
    sp.pieces = sp.splits + (int)splits;
    const PromptArgs none{};
    const dim3 grid((unsigned)tiles, (unsigned)a.c.Hkv, (unsigned)sp.splits);
    e = a.c.dt == MOE_DTYPE_BF16 ? launch_attn_shared_mma(sp, grid, s) : launch_tiles<true, false>(none, sp, D, grid, s);
    if (e != cudaSuccess) return e;
  }
  const int first = sp.splits, n = (int)splits;
  if (a.c.dt == MOE_DTYPE_BF16) e = launch_rows<__nv_bfloat16, 2, 4>(a, first, n, s);
  else if (D > 128) e = launch_rows<float, 2, 4>(a, first, n, s);
  else e = GR == 4 ? launch_rows<float, 1, 4>(a, first, n, s) : launch_rows<float, 1, 8>(a, first, n, s);
  if (e != cudaSuccess || first + n == 1) return e;
  return a.c.dt == MOE_DTYPE_BF16 ? launch_join<__nv_bfloat16>(a, first + n, s) : launch_join<float>(a, first + n, s);
}

}  // namespace moe

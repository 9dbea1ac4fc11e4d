// Attention for bf16 heads of 136 to 256 elements, whose output tile does not fit in TMEM beside two tiles of scores:
// warp-level MMAs (m16n8k16) with the output in registers. Packed prompts, and the shared positions of a decode batch.
//   S = Q K^T, P = 2^(c S - c m) (c = scale log2 e), O += P V, out = O / l
// with each row's running maximum m and sum l, in one pass over the keys.
//
// A CTA takes 64 packed rows (see PromptArgs) of one key/value head, 16 a warp, against tiles of 64 keys. Q, K and V
// are in shared memory, 16-byte pieces swizzled by their row so that no ldmatrix meets a bank twice; a tile's K is
// replaced while its softmax runs, its V while the next scores do, and two CTAs share an SM (96 KB and up to 255
// registers each). The scores' accumulators are the second product's A operand as they lie. Weights are rounded to
// bf16 (off by at most 2^-8 of each) as that operand; l takes them unrounded.
// Bound by the MMA's operands: each 16 x 16 piece of K or V read from shared memory meets only the warp's 16 rows. 4096
// tokens, 16 heads of 256 on 4: 471 us, 292 TFLOP/s (16384: 335; on the CUDA cores 4565 us); of 192: 398 us. Decode,
// 64 sequences behind 2048 shared positions with 2048 of their own: 157 us (340 with the shared ones on the CUDA
// cores). Columns of a row that a non-finite value at a position which it does not see can have touched are replaced,
// as in attn_tc.cu: 0 times that value must not reach it.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kRows = 64, KT = 64, kThreads = 128;
constexpr int kMaxCluster = 8;

template <int DP> constexpr size_t mma_smem() { return (size_t)(kRows + 2 * KT) * DP * 2; }

// Byte offset of 16-byte piece u of row r.
template <int DP> __device__ __forceinline__ uint32_t piece(int r, int u) { return (uint32_t)(r * DP * 2 + ((u ^ (r & 7)) << 4)); }

// (a call, as its registers would be the kernel's)
template <typename At>
__device__ __noinline__ uint32_t replace_row(Unseen& s, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                             At at, int D, int lim, float c2, float mc, float (&o)[8]) {
  return replace_unseen(s, q, k, v, at, D, lim, c2, mc, o);
}

// SPLIT: a tile's keys over the CTAs of a cluster. SHARED: the shared positions of a decode call, as in attn_simt.cu.
template <int DP, bool SPLIT, bool SHARED>
__global__ void __launch_bounds__(kThreads, 2)
attn_mma_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ SharedPart sp) {
  constexpr int NU = DP / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();  // after the wait: the own positions' kernel relies on it
  const uint32_t sQ = smem_u32(smem), sK = sQ + kRows * DP * 2, sV = sK + KT * DP * 2;
  const DecodeArgs& da = sp.d;
  const int H = SHARED ? da.H : a.H, Hkv = SHARED ? da.c.Hkv : a.Hkv, D = SHARED ? da.c.D : a.D;
  const int G = H / Hkv, hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int row0, nrows, j_begin, j_end, tile_end = 0;
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
    const int seq = find_tile_seq(a.qo, a.n, G, kRows, slot);
    sq = load_seq(a, seq);
    const long long r0 = ((long long)slot - ((long long)sq.q0 * G / kRows + seq)) * kRows;
    if (r0 < 0 || r0 >= (long long)sq.nq * G) return;
    row0 = (int)r0;
    nrows = min(kRows, sq.nq * G - row0);
    j_begin = 0;
    j_end = tile_end = visible_keys((row0 + nrows - 1) / G, sq.nq, sq.nk, a.causal);
    if (SPLIT) {
      const int keys = tile_end, per = ((keys - 1) / KT / (int)gridDim.z + 1) * KT;
      j_begin = (int)min((long long)keys, (long long)blockIdx.z * per);
      j_end = (int)min((long long)keys, (long long)j_begin + per);
    }
  }
  const __nv_bfloat16 *qb = (const __nv_bfloat16*)(SHARED ? da.q : a.q), *kb = (const __nv_bfloat16*)(SHARED ? da.k : a.k),
                      *vb = (const __nv_bfloat16*)(SHARED ? da.v : a.v);
  const long long qs = SHARED ? da.qs : a.qs;
  // where position j of the keys lies
  auto paged = [&](int j) {
    int page = pages[j >> da.c.page_shift];
    page = page < 0 || page >= da.c.n_pages ? 0 : page;
    return (((long long)page * Hkv + hk) * da.c.page_size + (j & (da.c.page_size - 1))) * D;
  };

  auto copy = [&](uint32_t dst, const __nv_bfloat16* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
  };
  // the tile of K or V at j0, `left` keys of it; what is past them and past D becomes zeros
  auto load = [&](uint32_t dst, const __nv_bfloat16* base, long long stride, int j0, int left) {
#pragma unroll 4
    for (int i = tid; i < KT * NU; i += kThreads) {
      const int r = i / NU, u = i % NU, j = j0 + min(r, left - 1);
      const long long at = SHARED ? paged(j) : (long long)(sq.k0 + j) * stride + (long long)hk * D;
      copy(dst + piece<DP>(r, u), base + at + min(u * 8, D - 8), r < left && u * 8 < D);
    }
  };
  if (j_end > j_begin) {
    for (int i = tid; i < kRows * NU; i += kThreads) {
      const int r = i / NU, u = i % NU, R = row0 + min(r, nrows - 1);
      const __nv_bfloat16* row = qb + (long long)(sq.q0 + R / G) * qs + (long long)(hk * G + R % G) * D;
      copy(sQ + piece<DP>(r, u), row + min(u * 8, D - 8), r < nrows && u * 8 < D);
    }
    load(sK, kb, a.ks, j_begin, j_end - j_begin);
    asm volatile("cp.async.commit_group;" ::: "memory");
    load(sV, vb, a.vs, j_begin, j_end - j_begin);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const float c2 = (SHARED ? da.scale : a.scale) * 1.4426950408889634f;
  const int g = lane >> 2, t4 = lane & 3, mi = lane >> 3, l8 = lane & 7;
  float o[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int lim[2];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = warp * 16 + g + 8 * y;
    lim[y] = 0;
    if (r < nrows && SHARED) {  // a slot shorter than the shared positions sees its own length of them
      lim[y] = min(j_end, slot_len(da.c, da.slots[(row0 + r) / G]));
    } else if (r < nrows) {
      lim[y] = visible_keys((row0 + r) / G, sq.nq, sq.nk, a.causal);
    }
  }
  for (int j0 = j_begin, left = j_end - j_begin; left > 0; j0 += KT, left -= KT) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // K is there
    float s[KT / 8][4];
#pragma unroll
    for (int n = 0; n < KT / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll 2
    for (int k = 0; k < DP / 16; ++k) {
      uint32_t q[4];
      ldsm4(sQ + piece<DP>(warp * 16 + (mi & 1) * 8 + l8, 2 * k + (mi >> 1)), q);
#pragma unroll
      for (int n = 0; n < KT / 16; ++n) {
        uint32_t b[4];
        ldsm4(sK + piece<DP>(n * 16 + (mi >> 1) * 8 + l8, 2 * k + (mi & 1)), b);
        mma16816(s[2 * n], q, b[0], b[1]);
        mma16816(s[2 * n + 1], q, b[2], b[3]);
      }
    }
    __syncthreads();  // K is read
    if (left > KT) load(sK, kb, a.ks, j0 + KT, left - KT);
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int see = lim[y] - j0;
      if (__any_sync(0xffffffffu, see < KT))
#pragma unroll
        for (int n = 0; n < KT / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (8 * n + 2 * t4 + e >= see) s[n][2 * y + e] = -INFINITY;
      float mx = -INFINITY;  // (max drops a NaN score)
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * y], s[n][2 * y + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[y], mx);
      if (__any_sync(0xffffffffu, mn > m[y])) {
        const float al = mn == m[y] ? 1.f : ex2((m[y] - mn) * c2);
        l[y] *= al;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[n][2 * y] *= al;
          o[n][2 * y + 1] *= al;
        }
        m[y] = mn;
      }
      const float mc = m[y] == -INFINITY ? 0.f : m[y] * c2;
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][2 * y + e] = ex2(fmaf(s[n][2 * y + e], c2, -mc));
          l[y] += s[n][2 * y + e];
        }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // V is there
#pragma unroll
    for (int k = 0; k < KT / 16; ++k) {
      const uint32_t p[4] = {pack_bf16x2(s[2 * k][0], s[2 * k][1]), pack_bf16x2(s[2 * k][2], s[2 * k][3]),
                             pack_bf16x2(s[2 * k + 1][0], s[2 * k + 1][1]), pack_bf16x2(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t b[4];
        ldsm4t(sV + piece<DP>(k * 16 + (mi & 1) * 8 + l8, 2 * n + (mi >> 1)), b);
        mma16816(o[2 * n], p, b[0], b[1]);
        mma16816(o[2 * n + 1], p, b[2], b[3]);
      }
    }
    __syncthreads();  // V is read
    if (left > KT) load(sV, vb, a.vs, j0 + KT, left - KT);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  Unseen unseen(SHARED || !SPLIT ? j_end : tile_end);
  auto replace = [&](int R, float mr, float lr) {  // in row R of the tile, by a warp
    const int P = row0 + R, tok = P / G, h = hk * G + P % G;
    float x[8];
    const uint32_t cols = replace_row(
        unseen, qb + (long long)(sq.q0 + tok) * qs + (long long)h * D, kb + (long long)sq.k0 * a.ks + (long long)hk * D,
        vb + (long long)sq.k0 * a.vs + (long long)hk * D,
        [&](int j, long long& ko, long long& vo) {
          ko = j * a.ks;
          vo = j * a.vs;
        },
        D, visible_keys(tok, sq.nq, sq.nk, a.causal), c2, mr == -INFINITY ? 0.f : mr * c2, x);
    const float inv = lr == 0.f ? 0.f : 1.0f / lr;
    __nv_bfloat16* dst = (__nv_bfloat16*)a.out + (long long)(sq.q0 + tok) * a.os + (long long)h * D + lane * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (cols >> e & 1u) dst[e] = __float2bfloat16_rn(x[e] * inv);
  };
  // m and l of row r of the warp's 16
  auto row_m = [&](int r) { return __shfl_sync(0xffffffffu, r < 8 ? m[0] : m[1], 4 * (r & 7)); };
  auto row_l = [&](int r) { return __shfl_sync(0xffffffffu, r < 8 ? l[0] : l[1], 4 * (r & 7)); };
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
  }
  if (SHARED) {
    uint32_t again[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int r = warp * 16 + g + 8 * y, P = row0 + min(r, nrows - 1);
      float* po = da.part + (((long long)(P / G) * H + hk * G + P % G) * sp.pieces + blockIdx.z) * (D + 2);
      bool fine = true;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        const int c = 8 * n + 2 * t4;
        const float x = lim[y] <= j_begin ? 0.f : o[n][2 * y], z = lim[y] <= j_begin ? 0.f : o[n][2 * y + 1];
        fine = fine && fabsf(x) <= 3.0e38f && fabsf(z) <= 3.0e38f;
        if (r < nrows && c < D) *reinterpret_cast<float2*>(po + c) = make_float2(x, z);
      }
      if (r < nrows && t4 == 0) *reinterpret_cast<float2*>(po + D) = make_float2(m[y] * c2, l[y]);
      again[y] = __ballot_sync(0xffffffffu, r < nrows && !fine && fabsf(l[y]) <= 3.0e38f);
    }
    __syncwarp();
    Unseen pieces_unseen(j_end - j_begin);
    for (int r = 0; r < 16; ++r) {
      if ((again[r >> 3] >> (4 * (r & 7)) & 15u) == 0) continue;
      const int P = row0 + warp * 16 + r, tok = P / G, h = hk * G + P % G;
      float x[8];
      const float mr = row_m(r);
      const int j0 = j_begin;  // (the keys counted from the piece's first)
      const uint32_t cols = replace_row(
          pieces_unseen, qb + (long long)tok * qs + (long long)h * D, kb, vb,
          [&](int j, long long& ko, long long& vo) { ko = vo = paged(j0 + j); }, D,
          max(0, min(j_end, slot_len(da.c, da.slots[tok])) - j0), c2, mr == -INFINITY ? 0.f : mr * c2, x);
      float* po = da.part + (((long long)tok * H + h) * sp.pieces + blockIdx.z) * (D + 2);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (cols >> e & 1u) po[lane * 8 + e] = x[e];
    }
    return;
  }
  if (SPLIT) {
    // The cluster's CTAs hold parts of the same rows: they put them in shared memory, and each adds up every C-th row
    // from all of them, in order.
    constexpr int LD = DP + 4;
    const int C = gridDim.z, rank = (int)cluster_ctarank();
    float* po = reinterpret_cast<float*>(smem);
    float2* ml = reinterpret_cast<float2*>(po + kRows * LD);
    float2* joined = ml + kRows;  // a row's m and l
    int* odd = reinterpret_cast<int*>(joined + kRows);
    static_assert(kRows * (LD * 4 + 8 + 8 + 4) <= mma_smem<DP>(), "the parts take the tiles' place");
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int R = warp * 16 + g + 8 * y;
      if (t4 == 0) ml[R] = make_float2(m[y], l[y]);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
        *reinterpret_cast<float2*>(po + R * LD + 8 * n + 2 * t4) = make_float2(o[n][2 * y], o[n][2 * y + 1]);
    }
    if (tid < kRows) odd[tid] = 0;
    cluster_sync_all();
    for (int i = tid; i < kRows / C * (DP / 4); i += kThreads) {
      const int R = rank + C * (i / (DP / 4)), c = (i % (DP / 4)) * 4;
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
        const float w = ex2((v[y].x - ref) * c2);
        L = fmaf(w, v[y].y, L);
        t.x = fmaf(w, u[y].x, t.x);
        t.y = fmaf(w, u[y].y, t.y);
        t.z = fmaf(w, u[y].z, t.z);
        t.w = fmaf(w, u[y].w, t.w);
      }
      const int P = row0 + R, tok = sq.q0 + P / G, h = hk * G + P % G;
      const bool none = visible_keys(P / G, sq.nq, sq.nk, a.causal) == 0;
      const float inv = none || L == 0.f ? 0.f : 1.0f / L;
      if (none) t = make_float4(0.f, 0.f, 0.f, 0.f);
      t.x *= inv; t.y *= inv; t.z *= inv; t.w *= inv;
      if (!(fabsf(t.x) <= 3.0e38f && fabsf(t.y) <= 3.0e38f && fabsf(t.z) <= 3.0e38f && fabsf(t.w) <= 3.0e38f)) odd[R] = 1;
      *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + (long long)tok * a.os + (long long)h * D + c) =
          make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
      if (c == 0) joined[R] = make_float2(M, L);
      if (a.lse != nullptr && c == 0)
        a.lse[(long long)tok * H + h] = none ? -INFINITY : (M * c2 + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();
    // (a row whose weights' sum is not finite sees a score that is not, and is NaN as a whole)
    for (int r = warp; r < kRows / C; r += kThreads / 32) {
      const int R = rank + C * r;
      if (odd[R] != 0 && fabsf(joined[R].y) <= 3.0e38f) replace(R, joined[R].x, joined[R].y);
    }
    cluster_sync_all();  // the others have read this CTA's part
    return;
  }
  uint32_t again[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = warp * 16 + g + 8 * y, R = row0 + r, tok = sq.q0 + R / G, h = hk * G + R % G;
    const float inv = l[y] == 0.f ? 0.f : 1.0f / l[y];
    __nv_bfloat16* dst = (__nv_bfloat16*)a.out + (long long)tok * a.os + (long long)h * D;
    bool fine = true;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const int c = 8 * n + 2 * t4;
      const float x = lim[y] == 0 ? 0.f : o[n][2 * y] * inv, z = lim[y] == 0 ? 0.f : o[n][2 * y + 1] * inv;
      fine = fine && fabsf(x) <= 3.0e38f && fabsf(z) <= 3.0e38f;
      if (r < nrows && c < D) *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(x, z);
    }
    if (a.lse != nullptr && r < nrows && t4 == 0)
      a.lse[(long long)tok * H + h] = lim[y] == 0 ? -INFINITY : (m[y] * c2 + log2f(l[y])) * 0.6931471805599453f;
    again[y] = __ballot_sync(0xffffffffu, r < nrows && !fine && fabsf(l[y]) <= 3.0e38f);
  }
  __syncwarp();
  for (int r = 0; r < 16; ++r) {
    if ((again[r >> 3] >> (4 * (r & 7)) & 15u) == 0) continue;
    const float mr = row_m(r), lr = row_l(r);
    replace(warp * 16 + r, mr, lr);
  }
}

template <int DP, bool SPLIT, bool SHARED>
cudaError_t launch(const PromptArgs& a, const SharedPart& sp, dim3 grid, cudaStream_t s) {
  auto kern = attn_mma_kernel<DP, SPLIT, SHARED>;
  static std::atomic<int> done{0};
  const cudaError_t e = allow_smem(kern, mma_smem<DP>(), done);
  if (e != cudaSuccess) return e;
  if (!SPLIT) return launch_pdl(kern, grid, dim3(kThreads), mma_smem<DP>(), s, a, sp);
  return launch_clusters(kern, grid, dim3(kThreads), dim3(1, 1, grid.z), mma_smem<DP>(), s, a, sp);
}

}  // namespace

cudaError_t launch_attn_prompt_mma(const PromptArgs& a, cudaStream_t s) {
  const long long slots = prompt_tile_slots(a.Tq, a.n, a.H / a.Hkv, kRows);
  // Few tiles: a cluster of CTAs takes the keys of each, at least two tiles of them where the keys are one sequence's
  // (heads of 256, 16 on 4: 16 tokens behind 8192 keys 64 us, 358 without; 1024 tokens of 4 heads on 4 31 and 53).
  int C = 1;
  while (C < kMaxCluster && slots * a.Hkv * 2 * C <= 2LL * device_sm_count() && a.Tkv >= 4 * C * KT) C *= 2;
  const dim3 grid((unsigned)slots, (unsigned)a.Hkv, (unsigned)C);
  const SharedPart none{};
  if (a.D <= 192) return C > 1 ? launch<192, true, false>(a, none, grid, s) : launch<192, false, false>(a, none, grid, s);
  return C > 1 ? launch<256, true, false>(a, none, grid, s) : launch<256, false, false>(a, none, grid, s);
}

cudaError_t launch_attn_shared_mma(const SharedPart& sp, dim3 grid, cudaStream_t s) {
  const PromptArgs none{};
  return sp.d.c.D <= 192 ? launch<192, false, true>(none, sp, grid, s) : launch<256, false, true>(none, sp, grid, s);
}

}  // namespace moe

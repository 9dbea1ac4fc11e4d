// Prompt attention for bf16 heads of 136 to 256 elements, whose output tile does not fit in TMEM beside two tiles of
// scores: warp-level MMAs (m16n8k16) with the output in registers.
//   S = Q K^T, P = 2^(c S - c m) (c = scale log2 e), O += P V, out = O / l
// with each row's running maximum m and sum l, in one pass over the keys.
//
// A CTA takes 64 packed rows (see PromptArgs) of one key/value head, 16 a warp, against tiles of 64 keys. Q, K and V are
// in shared memory, 16-byte pieces swizzled by their row so that no ldmatrix meets a bank twice; a tile's K is replaced
// while its softmax runs, its V while the next scores do, and two CTAs share an SM (96 KB and up to 255 registers each).
// The scores' accumulators are the second product's A operand as they lie. Weights are rounded to bf16 (off by at most
// 2^-8 of each) as that operand; l takes them unrounded.
// A row whose result is not finite is computed again over the keys that it sees, as in attn_tc.cu: 0 times a
// non-finite value that the row does not see must not reach it.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kRows = 64, KT = 64, kThreads = 128;

template <int DP> constexpr size_t mma_smem() { return (size_t)(kRows + 2 * KT) * DP * 2; }

// Byte offset of 16-byte piece u of row r.
template <int DP> __device__ __forceinline__ uint32_t piece(int r, int u) { return (uint32_t)(r * DP * 2 + ((u ^ (r & 7)) << 4)); }

// One row again, key by key (a warp; a lane owns 8 consecutive elements).
__device__ __noinline__ void exact_row256(const __nv_bfloat16* q, const __nv_bfloat16* k, long long ks, const __nv_bfloat16* v,
                                          long long vs, int D, int lim, float c2, __nv_bfloat16* out) {
  const int d = (threadIdx.x & 31) * 8;
  const bool on = d < D;
  float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < lim; ++j) {
    float s = 0.f;
    if (on)
      for (int e = 0; e < 8; ++e) s = fmaf(__bfloat162float(q[d + e]), __bfloat162float(k[j * ks + d + e]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= c2;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref), p = ex2(s - ref);
    l = fmaf(l, a, p);
    m = mn;
    if (on)
      for (int e = 0; e < 8; ++e) o[e] = fmaf(p, __bfloat162float(v[j * vs + d + e]), o[e] * a);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (on)
    for (int e = 0; e < 8; ++e) out[d + e] = __float2bfloat16_rn(o[e] * inv);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 2)
attn_mma_kernel(const __grid_constant__ PromptArgs a) {
  constexpr int NU = DP / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t sQ = smem_u32(smem), sK = sQ + kRows * DP * 2, sV = sK + KT * DP * 2;
  const int G = a.H / a.Hkv, D = a.D, hk = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = gridDim.x - 1 - blockIdx.x;  // a prompt's last rows see the most keys: they start first
  const int seq = find_tile_seq(a.qo, a.n, G, kRows, slot);
  const Seq sq = load_seq(a, seq);
  const long long r0 = ((long long)slot - ((long long)sq.q0 * G / kRows + seq)) * kRows;
  if (r0 < 0 || r0 >= (long long)sq.nq * G) return;
  const int row0 = (int)r0, nrows = min(kRows, sq.nq * G - row0);
  const int keys = visible_keys((row0 + nrows - 1) / G, sq.nq, sq.nk, a.causal);

  auto copy = [&](uint32_t dst, const __nv_bfloat16* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
  };
  // tile j0 of K or V; what is past the keys and past D becomes zeros
  auto load = [&](uint32_t dst, const void* base, long long stride, int j0) {
    const __nv_bfloat16* src = (const __nv_bfloat16*)base + (long long)(sq.k0 + j0) * stride + (long long)hk * D;
    const int left = keys - j0;
#pragma unroll 4
    for (int i = tid; i < KT * NU; i += kThreads) {
      const int r = i / NU, u = i % NU;
      copy(dst + piece<DP>(r, u), src + (long long)min(r, left - 1) * stride + min(u * 8, D - 8), r < left && u * 8 < D);
    }
  };
  if (keys > 0) {
    for (int i = tid; i < kRows * NU; i += kThreads) {
      const int r = i / NU, u = i % NU, R = row0 + min(r, nrows - 1);
      copy(sQ + piece<DP>(r, u), (const __nv_bfloat16*)a.q + (long long)(sq.q0 + R / G) * a.qs +
                                     (long long)(hk * G + R % G) * D + min(u * 8, D - 8), r < nrows && u * 8 < D);
    }
    load(sK, a.k, a.ks, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    load(sV, a.v, a.vs, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const float c2 = a.scale * 1.4426950408889634f;
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
    lim[y] = r < nrows ? visible_keys((row0 + r) / G, sq.nq, sq.nk, a.causal) : 0;
  }
  for (int j0 = 0, left = keys; left > 0; j0 += KT, left -= KT) {
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
    if (left > KT) load(sK, a.k, a.ks, j0 + KT);
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
    if (left > KT) load(sV, a.v, a.vs, j0 + KT);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  uint32_t again[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
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
      a.lse[(long long)tok * a.H + h] = lim[y] == 0 ? -INFINITY : (m[y] * c2 + log2f(l[y])) * 0.6931471805599453f;
    again[y] = __ballot_sync(0xffffffffu, r < nrows && !fine);
  }
  __syncwarp();
  for (int r = 0; r < 16; ++r) {
    if ((again[r >> 3] >> (4 * (r & 7)) & 15u) == 0) continue;
    const int R = row0 + warp * 16 + r, tok = R / G, h = hk * G + R % G;
    exact_row256((const __nv_bfloat16*)a.q + (long long)(sq.q0 + tok) * a.qs + (long long)h * D,
                 (const __nv_bfloat16*)a.k + (long long)sq.k0 * a.ks + (long long)hk * D, a.ks,
                 (const __nv_bfloat16*)a.v + (long long)sq.k0 * a.vs + (long long)hk * D, a.vs, D,
                 visible_keys(tok, sq.nq, sq.nk, a.causal), c2,
                 (__nv_bfloat16*)a.out + (long long)(sq.q0 + tok) * a.os + (long long)h * D);
  }
}

template <int DP>
cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
  auto kern = attn_mma_kernel<DP>;
  static std::atomic<int> done{0};
  const cudaError_t e = allow_smem(kern, mma_smem<DP>(), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)prompt_tile_slots(a.Tq, a.n, a.H / a.Hkv, kRows), (unsigned)a.Hkv);
  return launch_pdl(kern, grid, dim3(kThreads), mma_smem<DP>(), s, a);
}

}  // namespace

cudaError_t launch_attn_prompt_mma(const PromptArgs& a, cudaStream_t s) {
  return a.D <= 192 ? launch<192>(a, s) : launch<256>(a, s);
}

}  // namespace moe

// Attention on the CUDA cores, fp32 arithmetic throughout: fp32 tensors, and heads of more than 128.
//   out[r] = sum_{j < lim(r)} softmax_j(scale q[r] . k[j]) v[j]
// over packed prompts (PAGED = false) or, one token a sequence, over the paged cache (PAGED = true).
//
// One CTA takes ROWS packed rows (see PromptArgs) of one key/value head and walks the keys in tiles of KT,
// both in shared memory in fp32; the running maximum m and sum l of each row live in registers of the
// 16 threads that share the row, the output row in the registers of the same 16. Scores are kept in
// log2 units (times scale * log2 e), so a weight is one 2^x. Keys past a row's limit are left out of
// both products by index, not by a zero weight, so that a non-finite value there stays there.
// Bound by the CUDA cores' fp32 rate (prompts) and by their loads of shared memory; decode takes 16 rows
// instead of 64 and splits the keys over CTAs whose pieces decode_join_kernel adds in a fixed order.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int KT = 32;
constexpr int kThreads = 256;

__host__ __device__ constexpr size_t simt_smem(int rows, int D) {
  return sizeof(float) * ((size_t)(rows + 2 * KT) * (D + 4) + (size_t)rows * (KT + 1));
}

template <typename T>
__device__ __forceinline__ void load8f(const T* p, float* d);
template <>
__device__ __forceinline__ void load8f<float>(const float* p, float* d) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  reinterpret_cast<float4*>(d)[0] = a;
  reinterpret_cast<float4*>(d)[1] = b;
}
template <>
__device__ __forceinline__ void load8f<__nv_bfloat16>(const __nv_bfloat16* p, float* d) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  reinterpret_cast<float4*>(d)[0] = make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
  reinterpret_cast<float4*>(d)[1] = make_float4(bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w));
}

template <typename T, int ROWS, bool PAGED>
__global__ void __launch_bounds__(kThreads)
attn_simt_kernel(const __grid_constant__ PromptArgs pa, const __grid_constant__ DecodeArgs da, int n_tiles, int splits) {
  constexpr int RPT = ROWS / 16;  // rows per thread
  extern __shared__ __align__(16) float sm[];
  griddep_launch_dependents();
  griddep_wait();
  const int H = PAGED ? da.H : pa.H, Hkv = PAGED ? da.c.Hkv : pa.Hkv, D = PAGED ? da.c.D : pa.D;
  const int G = H / Hkv, hk = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int LD = D + 4;
  float* Qs = sm;
  float* Ks = Qs + ROWS * LD;
  float* Vs = Ks + KT * LD;
  float* Ps = Vs + KT * LD;

  // ---- which rows, which keys
  int row0, nrows, j_begin, j_end;  // packed rows row0 .. of the sequence; keys
  Seq sq{0, 0, 0, 0};
  int slot = 0, len = 0, seq;
  if (PAGED) {
    seq = blockIdx.x / n_tiles;
    row0 = (blockIdx.x % n_tiles) * ROWS;
    nrows = min(ROWS, G - row0);
    slot = da.slots[seq];
    if (slot < 0 || slot >= da.c.n_slots) {
      if (tid == 0) record_error(da.status, MOE_ERR_DEVICE_CHECK, seq);
      len = 0;
    } else {
      len = max(0, min(da.c.lens[slot], da.c.width << da.c.page_shift));
    }
    const int per = ((len + splits - 1) / splits + KT - 1) / KT * KT;
    j_begin = min(len, (int)blockIdx.z * per);
    j_end = min(len, j_begin + per);
  } else {
    seq = find_tile_seq(pa.qo, pa.n, G, ROWS, blockIdx.x);
    sq = load_seq(pa, seq);
    const long long first = (long long)sq.q0 * G / ROWS + seq;
    const long long r0 = ((long long)blockIdx.x - first) * ROWS;
    if (r0 < 0 || r0 >= (long long)sq.nq * G) return;
    row0 = (int)r0;
    nrows = min(ROWS, sq.nq * G - row0);
    j_begin = 0;
    j_end = visible_keys((row0 + nrows - 1) / G, sq.nq, sq.nk, pa.causal);
  }

  const float c2 = (PAGED ? da.scale : pa.scale) * 1.4426950408889634f;
  const int d8 = D / 8;
  for (int i = tid; i < ROWS * d8; i += kThreads) {
    const int r = i / d8, c = (i % d8) * 8;
    float t[8];
    if (r < nrows) {
      const int R = row0 + r, tok = PAGED ? seq : sq.q0 + R / G, h = hk * G + (PAGED ? R : R % G);
      const T* src = (const T*)(PAGED ? da.q : pa.q) + (long long)tok * (PAGED ? da.qs : pa.qs) + (long long)h * D + c;
      load8f<T>(src, t);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) Qs[r * LD + c + e] = t[e];
  }

  float m[RPT], l[RPT];
  int lim[RPT];
  float o[RPT][4][4];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    const int R = ty * RPT + r;
    lim[r] = R >= nrows ? 0 : (PAGED ? j_end : visible_keys((row0 + R) / G, sq.nq, sq.nk, pa.causal));
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][c][e] = 0.f;
  }

  for (int j0 = j_begin; j0 < j_end; j0 += KT) {
    __syncthreads();
    for (int i = tid; i < KT * d8; i += kThreads) {
      const int r = i / d8, c = (i % d8) * 8, j = j0 + r;
      float a[8], b[8];
      if (j < j_end) {
        long long ok, ov;
        if (PAGED) {
          int page = da.c.table[(long long)slot * da.c.width + (j >> da.c.page_shift)];
          if (page < 0 || page >= da.c.n_pages) {
            record_error(da.status, MOE_ERR_DEVICE_CHECK, seq);
            page = 0;
          }
          ok = ov = (((long long)page * Hkv + hk) * da.c.page_size + (j & (da.c.page_size - 1))) * D + c;
        } else {
          ok = (long long)(sq.k0 + j) * pa.ks + (long long)hk * D + c;
          ov = (long long)(sq.k0 + j) * pa.vs + (long long)hk * D + c;
        }
        load8f<T>((const T*)(PAGED ? da.k : pa.k) + ok, a);
        load8f<T>((const T*)(PAGED ? da.v : pa.v) + ov, b);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = b[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) { Ks[r * LD + c + e] = a[e]; Vs[r * LD + c + e] = b[e]; }
    }
    __syncthreads();
    // ---- scores of RPT rows x 2 keys (tx, tx + 16) per thread
    float s[RPT][2];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r][0] = s[r][1] = 0.f;
    for (int d = 0; d < D; d += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(Ks + tx * LD + d);
      const float4 k1 = *reinterpret_cast<const float4*>(Ks + (tx + 16) * LD + d);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(Qs + (ty * RPT + r) * LD + d);
        s[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[r][0]))));
        s[r][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[r][1]))));
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      float a = j0 + tx < lim[r] ? s[r][0] * c2 : -INFINITY, b = j0 + tx + 16 < lim[r] ? s[r][1] * c2 : -INFINITY;
      float mx = fmaxf(a, b);
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[r], mx), ref = mn == -INFINITY ? 0.f : mn;  // no key yet: every weight is 0
      a = ex2(a - ref);
      b = ex2(b - ref);
      float sum = a + b;
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const float al = ex2(m[r] - ref);
      l[r] = l[r] * al + sum;
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][c][e] *= al;
      Ps[(ty * RPT + r) * (KT + 1) + tx] = a;
      Ps[(ty * RPT + r) * (KT + 1) + tx + 16] = b;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    // ---- o += p v: each thread its RPT rows x columns tx * 4 + 64 c
    int kmax = 0;
#pragma unroll
    for (int r = 0; r < RPT; ++r) kmax = max(kmax, min(KT, lim[r] - j0));
    for (int kk = 0; kk < kmax; ++kk) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (tx * 4 + 64 * c < D) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + kk * LD + tx * 4 + 64 * c);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            if (j0 + kk < lim[r]) {
              const float p = Ps[(ty * RPT + r) * (KT + 1) + kk];
              o[r][c][0] = fmaf(p, v.x, o[r][c][0]);
              o[r][c][1] = fmaf(p, v.y, o[r][c][1]);
              o[r][c][2] = fmaf(p, v.z, o[r][c][2]);
              o[r][c][3] = fmaf(p, v.w, o[r][c][3]);
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int R = ty * RPT + r;
    if (R >= nrows) continue;
    const int P = row0 + R, tok = PAGED ? seq : sq.q0 + P / G, h = hk * G + (PAGED ? P : P % G);
    if (PAGED && splits > 1) {
      const long long row = (long long)seq * H + h, piece = row * splits + blockIdx.z;
      float* po = da.part + piece * (D + 2);
      if (tx == 0) { po[D] = m[r]; po[D + 1] = l[r]; }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tx * 4 + 64 * c < D) po[tx * 4 + 64 * c + e] = o[r][c][e];
      continue;
    }
    const float inv = l[r] == 0.f ? 0.f : 1.0f / l[r];
    T* dst = (T*)(PAGED ? da.out : pa.out) + (long long)tok * (PAGED ? da.os : pa.os) + (long long)h * D;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tx * 4 + 64 * c < D) dst[tx * 4 + 64 * c + e] = from_f32<T>(o[r][c][e] * inv);
    float* lse = PAGED ? da.lse : pa.lse;
    if (lse != nullptr && tx == 0)
      lse[(long long)tok * H + h] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * 0.6931471805599453f;
  }
}

// Joins a row's pieces (fixed order): one warp per (sequence, head).
template <typename T>
__global__ void __launch_bounds__(128)
decode_join_simt_kernel(const __grid_constant__ DecodeArgs a, int splits) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, D = a.c.D;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.n * a.H) return;
  const float* p = a.part + row * splits * (D + 2);
  float M = -INFINITY;
  for (int i = 0; i < splits; ++i) M = fmaxf(M, p[(long long)i * (D + 2) + D]);
  const float ref = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  for (int i = 0; i < splits; ++i) l += ex2(p[(long long)i * (D + 2) + D] - ref) * p[(long long)i * (D + 2) + D + 1];
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int tok = (int)(row / a.H), h = (int)(row % a.H);
  T* dst = (T*)a.out + (long long)tok * a.os + (long long)h * D;
  for (int d = lane; d < D; d += 32) {
    float o = 0.f;
    for (int i = 0; i < splits; ++i) {
      const float w = ex2(p[(long long)i * (D + 2) + D] - ref);
      if (p[(long long)i * (D + 2) + D + 1] != 0.f) o = fmaf(w, p[(long long)i * (D + 2) + d], o);
    }
    dst[d] = from_f32<T>(o * inv);
  }
  if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <typename T, int ROWS, bool PAGED>
cudaError_t launch(const PromptArgs& pa, const DecodeArgs& da, dim3 grid, int n_tiles, int splits, cudaStream_t s) {
  auto kern = attn_simt_kernel<T, ROWS, PAGED>;
  static std::atomic<int> done{0};
  const size_t smem = simt_smem(ROWS, PAGED ? da.c.D : pa.D);
  const cudaError_t e = allow_smem(kern, simt_smem(ROWS, 256), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, dim3(kThreads), smem, s, pa, da, n_tiles, splits);
}

}  // namespace

cudaError_t launch_attn_prompt_simt(const PromptArgs& a, cudaStream_t s) {
  const long long slots = prompt_tile_slots(a.Tq, a.n, a.H / a.Hkv, 64);
  const dim3 grid((unsigned)slots, (unsigned)a.Hkv);
  const DecodeArgs none{};
  return a.dt == MOE_DTYPE_BF16 ? launch<__nv_bfloat16, 64, false>(a, none, grid, 1, 1, s)
                                : launch<float, 64, false>(a, none, grid, 1, 1, s);
}

cudaError_t launch_attn_decode_simt(const DecodeArgs& a, cudaStream_t s) {
  const int G = a.H / a.c.Hkv, tiles = (G + 15) / 16;
  // enough CTAs to fill the GPU a few times over, at least 8 key tiles each at the longest length
  const long long ctas = (long long)a.n * tiles * a.c.Hkv, most = (long long)a.c.width * a.c.page_size;
  long long splits = (4LL * device_sm_count() + ctas - 1) / ctas;
  const long long cap = (most + 8 * KT - 1) / (8 * KT);
  splits = splits > cap ? cap : splits;
  const long long rows = (long long)a.n * a.H, fit = decode_pieces(rows) / rows;
  splits = splits > fit ? fit : (splits < 1 ? 1 : splits);
  splits = splits > 65535 ? 65535 : splits;
  const dim3 grid((unsigned)((long long)a.n * tiles), (unsigned)a.c.Hkv, (unsigned)splits);
  const PromptArgs none{};
  cudaError_t e = a.c.dt == MOE_DTYPE_BF16 ? launch<__nv_bfloat16, 16, true>(none, a, grid, tiles, (int)splits, s)
                                           : launch<float, 16, true>(none, a, grid, tiles, (int)splits, s);
  if (e != cudaSuccess || splits == 1) return e;
  const dim3 jg((unsigned)(((long long)a.n * a.H + 3) / 4));
  return a.c.dt == MOE_DTYPE_BF16
             ? launch_pdl(decode_join_simt_kernel<__nv_bfloat16>, jg, dim3(128), 0, s, a, (int)splits)
             : launch_pdl(decode_join_simt_kernel<float>, jg, dim3(128), 0, s, a, (int)splits);
}

}  // namespace moe

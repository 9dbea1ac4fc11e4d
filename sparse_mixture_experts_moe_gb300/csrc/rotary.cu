// Rotary positions of queries and keys, with a norm of each head in front, and the same on the way into a paged cache.
//   norm      y = x / sqrt(mean x^2 + eps) * w over a head's D elements (where there are weights w), fp32
//   rotation  (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for the pairs of the first R elements, c and s the cosine
//             and sine of position * f_p times the magnitude; the elements from R on stay as they are
// and one rounding to the heads' type at the end.
//
// An angle only matters modulo a circle, so f_p is held as a 64-bit fraction of a circle a position and multiplied by the
// position modulo 2^64: the product's upper bits are the angle, off by at most position * 2^-65 + 2^-32 of a circle
// however far the position (fp32 products lose all of it near 2^24). The two upper bits are the quadrant; sine and cosine
// of the rest, |x| <= pi / 4, are their Taylor sums to x^9 and x^10 (the first term left out is below 2.5e-9 of the value).
//
// LPR lanes share a row (a head of a token), so that a warp has 32 / LPR rows under way; a lane holds NC pairs of chunks
// of VEC elements. In the half layout those are elements p .. p + VEC - 1 and R/2 + p ..: both parts of its pairs, so no
// rotation crosses lanes. (VEC is 16 bytes, or what divides R / 2 where that is less.)
//
// The rows of all tokens lie in a row, kUnroll * 32 / LPR at a time (a unit), and each warp takes a run of them: it computes
// its lanes' sines and cosines once a token and looks for the token's place in the cache only where the sequence or the page
// changes. A lane copies its chunks of the next kStages units into shared memory while it works on the oldest, and reads
// back what it copied itself, so no barrier is needed.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 2, kStages = 4, kThreads = 256, kWarps = kThreads / 32, kBlocks = 2;

template <int BYTES> struct Raw;  // a chunk as it lies in memory
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<2> { using T = unsigned short; };

template <typename T, int VEC> struct Chunk {
  using R = typename Raw<VEC * sizeof(T)>::T;
  union U {
    R r;
    T e[VEC];
    __device__ U() {}
  };
};

// Cosine and sine of the angle `turn` / 2^64 of a circle.
__device__ __forceinline__ void cos_sin(uint64_t turn, float& c, float& s) {
  const uint32_t hi = (uint32_t)(turn >> 32), quad = (hi + 0x20000000u) >> 30;
  const float x = (float)(int)(hi - (quad << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float a = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(z, a, 1.f / 120.f);
  a = fmaf(z, a, -1.f / 6.f);
  const float sn = fmaf(x * z, a, x);
  float b = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  b = fmaf(z, b, -1.f / 720.f);
  b = fmaf(z, b, 1.f / 24.f);
  b = fmaf(z, b, -0.5f);
  const float cs = fmaf(z, b, 1.f);
  c = quad & 1u ? sn : cs;
  s = quad & 1u ? cs : sn;
  if ((quad + 1u) & 2u) c = -c;  // quadrants 1 and 2
  if (quad & 2u) s = -s;         // 2 and 3
}

// Where the tokens of a run go: the sequence and the page of the last one, and its position and page.
struct Place {
  int o0 = 0, o1 = 0, slot = 0, p0 = 0, held = 0;  // the sequence's tokens, slot, first position and the slot's length
  int col = -1, page = 0;                          // the table's column and what is there (-1: no page to write to)
  int position = 0;
  __device__ __forceinline__ bool find(const RotaryArgs& a, int t) {
    const CacheView& c = a.c;
    if (t < o0 || t >= o1) {  // (no sequence yet, or the next one)
      const int lane = threadIdx.x & 31;
      int lo = 0, len = a.n;
      while (len > 1) {
        const int step = (len + 31) / 32;
        const bool at = lane * step < len && a.offsets[lo + lane * step] <= t;
        const int m = __popc(__ballot_sync(0xffffffffu, at)) - 1, skip = (m < 0 ? 0 : m) * step;
        lo += skip;
        len = len - skip < step ? len - skip : step;
      }
      slot = a.slots[lo];
      o0 = a.offsets[lo];
      o1 = a.offsets[lo + 1];
      p0 = a.pos[lo];
      held = slot >= 0 && slot < c.n_slots && p0 >= 0 ? c.lens[slot] : 0;
      col = -1;
      if (t < o0 || t >= o1) return false;
    }
    const long long p = (long long)p0 + (t - o0);
    if (p < 0 || p >= held || (p >> c.page_shift) >= c.width) return false;
    position = (int)p;
    if (col != position >> c.page_shift) {
      col = position >> c.page_shift;
      page = c.table[(long long)slot * c.width + col];
      if (page < 0 || page >= c.n_pages || c.refs[page] != 1) page = -1;
    }
    return page >= 0;
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_chunk(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  } else if constexpr (BYTES >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
  } else {  // (copies have 4 bytes at least)
    const unsigned short x = *static_cast<const unsigned short*>(src);
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(x) : "memory");
  }
}

template <int CHUNK, int NC> constexpr int warp_smem() { return kStages * kUnroll * NC * 2 * 32 * CHUNK; }

template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kThreads, kBlocks)
rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using C = Chunk<T, VEC>;
  using R4 = typename C::R;
  constexpr int CB = VEC * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t smem[];
  uint64_t* turns = reinterpret_cast<uint64_t*>(smem);  // [R / 2]
  griddep_launch_dependents();
  griddep_wait();
  const int D = a.D, R = a.rot.R;
  for (int i = threadIdx.x; i < R / 2; i += kThreads) turns[i] = a.rot.turns[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, lpr = 1 << a.lpr_shift, me = lane & (lpr - 1), rpw = 32 >> a.lpr_shift;
  uint8_t* mine = smem + 1024 + (threadIdx.x >> 5) * warp_smem<CB, NC>() + lane * CB;  // chunk i of a stage: + i 32 CB
  // this lane's chunks: elements, whether they exist, and the first of their pairs
  int at[NC][2], pair[NC][2];
  bool in[NC][2];
#pragma unroll
  for (int y = 0; y < NC; ++y) {
    const int s = me + y * lpr, turning = R / (2 * VEC);
    if (INTERLEAVED) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        at[y][x] = (2 * s + x) * VEC;
        pair[y][x] = at[y][x] / 2;
      }
    } else if (s < turning) {
      at[y][0] = pair[y][0] = s * VEC;
      at[y][1] = R / 2 + s * VEC;
    } else {
      at[y][0] = R + 2 * (s - turning) * VEC;
      at[y][1] = at[y][0] + VEC;
      pair[y][0] = R;  // none
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) in[y][x] = at[y][x] < D;
  }
  typename C::U qw[NC][2], kw[NC][2];
#pragma unroll
  for (int y = 0; y < NC; ++y)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (a.qw != nullptr && in[y][x]) qw[y][x].r = *reinterpret_cast<const R4*>((const T*)a.qw + at[y][x]);
      if (a.kw != nullptr && in[y][x]) kw[y][x].r = *reinterpret_cast<const R4*>((const T*)a.kw + at[y][x]);
    }
  const int rows = a.H + (APPEND ? 2 : 1) * a.Hkv, groups = a.groups;
  const long long warps = (long long)gridDim.x * kWarps, w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long units = (long long)a.T * groups, u0 = units * w / warps, u1 = units * (w + 1) / warps;
  // the unit whose copies are asked for next
  long long next = u0;
  int nt = (int)(u0 / groups), ng = (int)(u0 - (long long)nt * groups);
  auto ask = [&](int stage) {
    if (next < u1) {
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int r = (ng * kUnroll + z) * rpw + (lane >> a.lpr_shift);
        const T* src = r < a.H ? (const T*)a.q + nt * a.qs + (long long)r * D
                     : r < a.H + a.Hkv ? (const T*)a.k + nt * a.ks + (long long)(r - a.H) * D
                                       : (const T*)a.v + nt * a.vs + (long long)(r - a.H - a.Hkv) * D;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (r < rows && in[y][x])
              copy_chunk<CB>(smem_u32(mine + (((stage * kUnroll + z) * NC + y) * 2 + x) * 32 * CB), src + at[y][x]);
      }
      ++next;
      if (++ng == groups) {
        ng = 0;
        ++nt;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st) ask(st);
  int t = (int)(u0 / groups), g = (int)(u0 - (long long)t * groups), position = 0, ahead = 0;
  if (!APPEND && u0 < u1) ahead = a.positions[t];
  bool fresh = true, ok = true;  // a token's first unit here; it has a place
  Place place;
  float c[NC][VEC], s[NC][VEC];
  int stage = 0;
  for (long long u = u0; u < u1; ++u) {
    if (fresh) {
      fresh = false;
      if (APPEND) {
        ok = place.find(a, t);
        position = place.position;
        if (!ok && g == 0 && lane == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, t);
      } else {
        position = ahead;
        if (t + 1 < a.T) ahead = a.positions[t + 1];
      }
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int p = INTERLEAVED ? pair[y][2 * i / VEC] + i % (VEC / 2 > 0 ? VEC / 2 : 1) : pair[y][0] + i;
          cos_sin((uint64_t)(long long)position * (p < R / 2 ? turns[p] : 0ull), c[y][i], s[y][i]);
          c[y][i] *= a.rot.magnitude;
          s[y][i] *= a.rot.magnitude;
        }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int z = 0; z < kUnroll; ++z) {
      const int r = (g * kUnroll + z) * rpw + (lane >> a.lpr_shift);
      const bool is_q = r < a.H, is_v = r >= a.H + a.Hkv;
      typename C::U u4[NC][2];
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          u4[y][x].r = *reinterpret_cast<const R4*>(mine + (((stage * kUnroll + z) * NC + y) * 2 + x) * 32 * CB);
      float f[NC][2][VEC];
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[y][x][i] = to_f32<T>(u4[y][x].e[i]);
      if (a.qw != nullptr || a.kw != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (r < rows && in[y][x])
#pragma unroll
              for (int i = 0; i < VEC; ++i) sum = fmaf(f[y][x][i], f[y][x][i], sum);
        for (int m = lpr >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float inv = rsqrtf(sum / (float)D + a.eps);
        if ((is_q ? a.qw : a.kw) != nullptr)
#pragma unroll
          for (int y = 0; y < NC; ++y)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int i = 0; i < VEC; ++i) f[y][x][i] = f[y][x][i] * inv * to_f32<T>(is_q ? qw[y][x].e[i] : kw[y][x].e[i]);
      }
      if (r >= rows || !ok) continue;
      T* dst;
      if (is_q) dst = (T*)a.qo + t * a.qos + (long long)r * D;
      else if (!APPEND) dst = (T*)a.ko + t * a.kos + (long long)(r - a.H) * D;
      else dst = (T*)(is_v ? a.vp : a.kp) +
                 (((long long)place.page * a.Hkv + (is_v ? r - a.H - a.Hkv : r - a.H)) * a.c.page_size + (position & (a.c.page_size - 1))) * D;
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        if (!APPEND || !is_v) {
          if (INTERLEAVED) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int i = 0; i < VEC / 2; ++i) {
                const float p = f[y][x][2 * i], q = f[y][x][2 * i + 1], cc = c[y][x * (VEC / 2) + i], ss = s[y][x * (VEC / 2) + i];
                const bool on = pair[y][x] + i < R / 2;
                u4[y][x].e[2 * i] = from_f32<T>(on ? fmaf(p, cc, -q * ss) : p);
                u4[y][x].e[2 * i + 1] = from_f32<T>(on ? fmaf(q, cc, p * ss) : q);
              }
          } else {
            const bool on = pair[y][0] < R / 2;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float p = f[y][0][i], q = f[y][1][i];
              u4[y][0].e[i] = from_f32<T>(on ? fmaf(p, c[y][i], -q * s[y][i]) : p);
              u4[y][1].e[i] = from_f32<T>(on ? fmaf(q, c[y][i], p * s[y][i]) : q);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (in[y][x]) *reinterpret_cast<R4*>(dst + at[y][x]) = u4[y][x].r;
      }
    }
    ask(stage);
    if (++stage == kStages) stage = 0;
    if (++g == groups) {
      g = 0;
      ++t;
      fresh = true;
    }
  }
}

template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND>
cudaError_t launch(RotaryArgs& a, cudaStream_t s) {
  const int R = a.rot.R, chunks = a.D / VEC;
  const int slots = INTERLEAVED ? (chunks + 1) / 2 : R / (2 * VEC) + ((a.D - R) / VEC + 1) / 2;
  a.lpr_shift = 0;
  while ((NC << a.lpr_shift) < slots) ++a.lpr_shift;
  const int rows = a.H + (APPEND ? 2 : 1) * a.Hkv, at_once = (32 >> a.lpr_shift) * kUnroll;
  a.groups = (rows + at_once - 1) / at_once;
  const long long units = (long long)a.T * a.groups, most = (long long)kBlocks * device_sm_count();
  const long long blocks = (units + kWarps - 1) / kWarps;
  auto kern = rotary_kernel<T, VEC, NC, INTERLEAVED, APPEND>;
  constexpr size_t bytes = 1024 + kWarps * warp_smem<VEC * (int)sizeof(T), NC>();
  static std::atomic<int> done{0};
  const cudaError_t e = allow_smem(kern, bytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), bytes, s, a);
}

template <bool APPEND>
cudaError_t launch(RotaryArgs& a, int dt, cudaStream_t s) {
  const int half = a.rot.R / 2;
  if (dt == MOE_DTYPE_BF16) {
    if (a.rot.layout == MOE_ROTARY_INTERLEAVED) return launch<__nv_bfloat16, 8, 1, true, APPEND>(a, s);
    if (half % 8 == 0) return launch<__nv_bfloat16, 8, 1, false, APPEND>(a, s);
    if (half % 4 == 0) return launch<__nv_bfloat16, 4, 1, false, APPEND>(a, s);
    if (half % 2 == 0) return launch<__nv_bfloat16, 2, 2, false, APPEND>(a, s);
    return launch<__nv_bfloat16, 1, 4, false, APPEND>(a, s);
  }
  if (a.rot.layout == MOE_ROTARY_INTERLEAVED) return launch<float, 4, 1, true, APPEND>(a, s);
  if (half % 4 == 0) return launch<float, 4, 1, false, APPEND>(a, s);
  if (half % 2 == 0) return launch<float, 2, 2, false, APPEND>(a, s);
  return launch<float, 1, 4, false, APPEND>(a, s);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs& a, int dt, cudaStream_t s) { return launch<false>(a, dt, s); }
cudaError_t launch_cache_append(RotaryArgs& a, cudaStream_t s) { return launch<true>(a, a.c.dt, s); }

}  // namespace moe

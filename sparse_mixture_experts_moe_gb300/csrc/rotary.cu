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
// rotation crosses lanes. (VEC is 16 bytes, or what divides R / 2 where that is less.) A warp takes a token, or with few
// tokens some of its rows, and computes its lanes' sines and cosines once for all of them; a group of kUnroll rows
// is loaded at once.
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 4, kThreads = 256;

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

// Where token t goes: its position, and the page and row (append). false: nowhere, which is recorded.
__device__ __forceinline__ bool find_place(const RotaryArgs& a, int t, bool first, int& position, int& page) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = a.n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const bool at = lane * step < len && a.offsets[lo + lane * step] <= t;
    const int m = __popc(__ballot_sync(0xffffffffu, at)) - 1, skip = (m < 0 ? 0 : m) * step;
    lo += skip;
    len = len - skip < step ? len - skip : step;
  }
  const CacheView& c = a.c;
  const int s = a.slots[lo], o0 = a.offsets[lo], o1 = a.offsets[lo + 1], p0 = a.pos[lo];
  bool ok = s >= 0 && s < c.n_slots && t >= o0 && t < o1 && p0 >= 0;
  const long long p = (long long)p0 + ((long long)t - o0);
  if (ok && (p >> c.page_shift) < c.width) {
    const int held = c.lens[s];
    page = c.table[(long long)s * c.width + (p >> c.page_shift)];
    ok = p < held && page >= 0 && page < c.n_pages && c.refs[page] == 1;
  } else {
    ok = false;
  }
  position = (int)p;
  if (!ok && first && lane == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, t);
  return ok;
}

template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kThreads, 2)
rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using C = Chunk<T, VEC>;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, lpr = 1 << a.lpr_shift, me = lane & (lpr - 1), rpw = 32 >> a.lpr_shift;
  const int D = a.D, R = a.rot.R;
  // this lane's chunks: elements, whether they exist, and the first of their pairs
  int at[NC][2], pair[NC][2];
  bool in[NC][2];
  uint64_t turn[NC][VEC];
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
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int p = INTERLEAVED ? pair[y][2 * i / VEC] + i % (VEC / 2 > 0 ? VEC / 2 : 1) : pair[y][0] + i;
      turn[y][i] = p < R / 2 ? a.rot.turns[p] : 0ull;
    }
  }
  typename C::U qw[NC][2], kw[NC][2];
#pragma unroll
  for (int y = 0; y < NC; ++y)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (a.qw != nullptr && in[y][x]) qw[y][x].r = *reinterpret_cast<const typename C::R*>((const T*)a.qw + at[y][x]);
      if (a.kw != nullptr && in[y][x]) kw[y][x].r = *reinterpret_cast<const typename C::R*>((const T*)a.kw + at[y][x]);
    }
  const int rows = a.H + (APPEND ? 2 : 1) * a.Hkv;
  const int groups = (rows + rpw * kUnroll - 1) / (rpw * kUnroll);  // of rows that are under way at once
  const long long warps = (long long)gridDim.x * (kThreads / 32), units = (long long)a.T * a.parts;
  for (long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < units; w += warps) {
    const int t = (int)(w / a.parts), part = (int)(w - (long long)t * a.parts);
    int position, page = 0;
    if (APPEND) {
      if (!find_place(a, t, part == 0, position, page)) continue;
    } else {
      position = a.positions[t];
    }
    float c[NC][VEC], s[NC][VEC];
#pragma unroll
    for (int y = 0; y < NC; ++y)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        cos_sin((uint64_t)(long long)position * turn[y][i], c[y][i], s[y][i]);
        c[y][i] *= a.rot.magnitude;
        s[y][i] *= a.rot.magnitude;
      }
    for (int g = part; g < groups; g += a.parts) {
      typename C::U u[kUnroll][NC][2];
      const int r0 = g * rpw * kUnroll + (lane >> a.lpr_shift);
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int r = r0 + z * rpw;
        const T* src = r < a.H ? (const T*)a.q + t * a.qs + (long long)r * D
                     : r < a.H + a.Hkv ? (const T*)a.k + t * a.ks + (long long)(r - a.H) * D
                                       : (const T*)a.v + t * a.vs + (long long)(r - a.H - a.Hkv) * D;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (r < rows && in[y][x]) u[z][y][x].r = __ldcs(reinterpret_cast<const typename C::R*>(src + at[y][x]));
      }
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int r = r0 + z * rpw;
        const bool is_q = r < a.H, is_v = r >= a.H + a.Hkv;
        float f[NC][2][VEC];
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[y][x][i] = to_f32<T>(u[z][y][x].e[i]);
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
                for (int i = 0; i < VEC; ++i)
                  f[y][x][i] *= inv * to_f32<T>(is_q ? qw[y][x].e[i] : kw[y][x].e[i]);
        }
        if (r >= rows) continue;
        T* dst;
        if (is_q) dst = (T*)a.qo + t * a.qos + (long long)r * D;
        else if (!APPEND) dst = (T*)a.ko + t * a.kos + (long long)(r - a.H) * D;
        else dst = (T*)(is_v ? a.vp : a.kp) +
                   (((long long)page * a.Hkv + (is_v ? r - a.H - a.Hkv : r - a.H)) * a.c.page_size + (position & (a.c.page_size - 1))) * D;
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
                  u[z][y][x].e[2 * i] = from_f32<T>(on ? fmaf(p, cc, -q * ss) : p);
                  u[z][y][x].e[2 * i + 1] = from_f32<T>(on ? fmaf(q, cc, p * ss) : q);
                }
            } else {
              const bool on = pair[y][0] < R / 2;
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                const float p = f[y][0][i], q = f[y][1][i];
                u[z][y][0].e[i] = from_f32<T>(on ? fmaf(p, c[y][i], -q * s[y][i]) : p);
                u[z][y][1].e[i] = from_f32<T>(on ? fmaf(q, c[y][i], p * s[y][i]) : q);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (in[y][x]) *reinterpret_cast<typename C::R*>(dst + at[y][x]) = u[z][y][x].r;
        }
      }
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
  const int groups = (rows + at_once - 1) / at_once, wpb = kThreads / 32;
  // Few tokens: their rows over several warps, up to 16 warps an SM.
  const long long fill = 16LL * device_sm_count();
  long long parts = (fill + a.T - 1) / a.T;
  a.parts = (int)(parts > groups ? groups : parts);
  long long blocks = ((long long)a.T * a.parts + wpb - 1) / wpb;
  const long long most = 8LL * device_sm_count();
  blocks = blocks > most ? most : blocks;
  return launch_pdl(rotary_kernel<T, VEC, NC, INTERLEAVED, APPEND>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
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

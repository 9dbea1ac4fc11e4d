// Rotary positions of queries and keys, with a norm of each head in front, and the same on the way into a paged cache.
//   norm      y = x / sqrt(mean x^2 + eps) * w over a head's D elements (where there are weights w), fp32
//   rotation  (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for the pairs of the first R elements, c and s the cosine
//             and sine of position * f_p times the magnitude; the elements from R on stay as they are
// and one rounding to the heads' type at the end.
//
// An angle only matters modulo a circle, so f_p is held as a 64-bit fraction of a circle a position and multiplied by the
// position modulo 2^64: the product's upper bits are the angle, however far the position (fp32 products lose all of it
// near 2^24). The fraction comes from doubles: pow, a scaling and the division by 2 pi leave less than 2^-52 of a circle a
// position for f_p <= 1 (2^-55 seen). The two upper bits of the product are the quadrant, the next 30 the rest, which
// fp32 holds to three roundings of 2^-24 of it, less than 2^-25 of a circle; sine and cosine of it, |x| <= pi / 4, are
// their Taylor sums to x^9 and x^10 (the first term left out is below 2.5e-9 of the value).
//
// LPR lanes share a row (a head of a token), so that a warp has 32 / LPR rows under way; a lane holds NC pairs of chunks
// of VEC elements. In the half layout those are elements p .. p + VEC - 1 and R/2 + p ..: both parts of its pairs, so no
// rotation crosses lanes. (VEC is 16 bytes, or what divides R / 2 where that is less.)
//
// The rows of all tokens lie in a row, kUnroll * 32 / LPR at a time (a unit), and each warp takes a run of them: it
// computes its lanes' sines and cosines once a token and looks for the token's place in the cache only where the
// sequence or the page changes. A lane copies its chunks of the next kStages units into shared memory while it works on
// the oldest, and reads back what it copied itself, so no barrier is needed. (Loads into registers, two rows ahead: 146
// us for 16384 tokens of 72 heads with a norm, 108 so; with 6 or 8 stages 110. One or three CTAs an SM: 112, and 83 us
// instead of 68 into pages.)
//
// Bound by memory: each element is read once and written once. Measured, bf16 heads of 128, 16384 tokens: 40 heads
// turned 58.8 us (5.7 TB/s, 84% of the copy rate); 72 heads normed and turned 108 us (5.6 TB/s, issue slots 60% busy:
// packed fp32 products and sums and weights in shared memory took 62 us to 58, 84 to 69 into pages); 32 heads' queries
// and 8 heads' keys normed and turned, with values, into pages 68 us (5.9 TB/s). A decode step's call takes 2.5 to 5 us
// on the GPU: the launch, the first row's latency and, into a cache, four loads that wait for one another (offsets, slot,
// length, table).
#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 1, kStages = 4, kThreads = 256, kWarps = kThreads / 32, kBlocks = 2;

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

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int CHUNK, int NC> constexpr int warp_smem() { return kStages * kUnroll * NC * 2 * 32 * CHUNK; }
constexpr int kTables = 128 * 8 + 2 * 256 * 4;  // the pairs' frequencies, and both norms' weights in fp32

// WHOLE: every element turns. NORM: there are weights.
template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND, bool WHOLE, bool NORM>
__global__ void __launch_bounds__(kThreads, kBlocks)
rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using C = Chunk<T, VEC>;
  using R4 = typename C::R;
  constexpr int CB = VEC * (int)sizeof(T), V2 = VEC / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  uint64_t* turns = reinterpret_cast<uint64_t*>(smem);           // [R / 2]
  float* weights = reinterpret_cast<float*>(smem + 128 * 8);      // of queries [D] and keys (256 on)
  griddep_launch_dependents();
  griddep_wait();
  const int D = a.D, R = a.rot.R;
  for (int i = threadIdx.x; i < R / 2; i += kThreads) turns[i] = a.rot.turns[i];
  if (NORM)
    for (int i = threadIdx.x; i < D; i += kThreads) {
      weights[i] = a.qw != nullptr ? to_f32<T>(((const T*)a.qw)[i]) : 1.f;
      weights[256 + i] = a.kw != nullptr ? to_f32<T>(((const T*)a.kw)[i]) : 1.f;
    }
  __syncthreads();
  const int lane = threadIdx.x & 31, lpr = 1 << a.lpr_shift, me = lane & (lpr - 1), rpw = 32 >> a.lpr_shift;
  uint8_t* mine = smem + kTables + (threadIdx.x >> 5) * warp_smem<CB, NC>() + lane * CB;  // chunk i of a stage: + i 32 CB
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
  const int H = a.H, Hk = H + a.Hkv, rows = H + (APPEND ? 2 : 1) * a.Hkv, groups = a.groups;
  const long long warps = (long long)gridDim.x * kWarps, w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long units = (long long)a.T * groups, u0 = units * w / warps, u1 = units * (w + 1) / warps;
  const int step = kUnroll * rpw, row_in = lane >> a.lpr_shift;
  // Row r of a token's queries, keys and values (and results) is at its array's base + r D, the bases moved back by the rows
  // before. The unit whose copies are asked for next: its first row, and the bases of its token.
  long long left = u1 - u0;
  int t = (int)(u0 / groups), g = (int)(u0 - (long long)t * groups);
  int ng = g;
  const T* nq = (const T*)a.q + t * a.qs;
  const T* nk = (const T*)a.k + t * a.ks - (long long)H * D;
  const T* nv = (const T*)a.v + t * a.vs - (long long)Hk * D;
  auto ask = [&](int stage) {
    if (left > 0) {
      --left;
#pragma unroll
      for (int z = 0; z < kUnroll; ++z) {
        const int r = ng * step + z * rpw + row_in;
        const T* src = (r < H ? nq : !APPEND || r < Hk ? nk : nv) + r * D;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (r < rows && in[y][x])
              copy_chunk<CB>(smem_u32(mine + (((stage * kUnroll + z) * NC + y) * 2 + x) * 32 * CB), src + at[y][x]);
      }
      if (++ng == groups) {
        ng = 0;
        nq += a.qs;
        nk += a.ks;
        if (APPEND) nv += a.vs;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st < kStages; ++st) ask(st);
  int position = 0, ahead = 0;
  if (!APPEND && u0 < u1) ahead = a.positions[t];
  bool fresh = true, ok = true;  // a token's first unit here; it has a place
  Place place;
  // cosines and sines: of pairs i, i + 1 side by side (half), or of pair i twice, the sine as (-s, s) (interleaved)
  uint64_t c2[NC][INTERLEAVED ? VEC : V2 > 0 ? V2 : 1], s2[NC][INTERLEAVED ? VEC : V2 > 0 ? V2 : 1];
  T *dq = nullptr, *dk = nullptr, *dv = nullptr;  // where the results' rows begin
  const int kv_row = APPEND ? a.c.page_size * D : D;
  int stage = 0;
  for (long long u = u0; u < u1; ++u) {
    if (fresh) {
      fresh = false;
      dq = (T*)a.qo + t * a.qos;
      if (APPEND) {
        ok = place.find(a, t);
        position = place.position;
        if (!ok && g == 0 && lane == 0) record_error(a.status, MOE_ERR_DEVICE_CHECK, t);
        const long long first = ((long long)place.page * a.Hkv * a.c.page_size + (position & (a.c.page_size - 1))) * D;
        dk = (T*)a.kp + first - (long long)H * kv_row;
        dv = (T*)a.vp + first - (long long)Hk * kv_row;
      } else {
        position = ahead;
        if (t + 1 < a.T) ahead = a.positions[t + 1];
        dk = (T*)a.ko + t * a.kos - (long long)H * D;
      }
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        float c[VEC], s[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int p = INTERLEAVED ? pair[y][2 * i / VEC] + i % (V2 > 0 ? V2 : 1) : pair[y][0] + i;
          cos_sin((uint64_t)(long long)position * (p < R / 2 ? turns[p] : 0ull), c[i], s[i]);
          c[i] *= a.rot.magnitude;
          s[i] *= a.rot.magnitude;
        }
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            c2[y][i] = f2_pack(c[i], c[i]);
            s2[y][i] = f2_pack(-s[i], s[i]);
          }
        } else if constexpr (VEC > 1) {
#pragma unroll
          for (int i = 0; i < V2; ++i) {
            c2[y][i] = f2_pack(c[2 * i], c[2 * i + 1]);
            s2[y][i] = f2_pack(s[2 * i], s[2 * i + 1]);
          }
        } else {
          c2[y][0] = f2_pack(c[0], c[0]);
          s2[y][0] = f2_pack(s[0], s[0]);
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int z = 0; z < kUnroll; ++z) {
      const int r = g * step + z * rpw + row_in;
      const bool is_q = r < H, is_v = APPEND && r >= Hk;
      typename C::U u4[NC][2];
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          u4[y][x].r = *reinterpret_cast<const R4*>(mine + (((stage * kUnroll + z) * NC + y) * 2 + x) * 32 * CB);
      // elements 2 i, 2 i + 1 of a chunk in one register pair (a chunk of one: twice)
      constexpr int N2 = V2 > 0 ? V2 : 1;
      uint64_t f[NC][2][N2];
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < N2; ++i)
            f[y][x][i] = f2_pack(to_f32<T>(u4[y][x].e[VEC > 1 ? 2 * i : 0]), to_f32<T>(u4[y][x].e[VEC > 1 ? 2 * i + 1 : 0]));
      if (NORM) {
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (r < rows && in[y][x])
#pragma unroll
              for (int i = 0; i < N2; ++i) sum2 = ffma2(f[y][x][i], f[y][x][i], sum2);
        float sum = VEC > 1 ? f2_lo(sum2) + f2_hi(sum2) : f2_lo(sum2);
        for (int m = lpr >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float inv = (is_q ? a.qw : a.kw) != nullptr ? rsqrtf(fmaf(sum, a.inv_d, a.eps)) : 1.f;
        const uint64_t inv2 = f2_pack(inv, inv);
        const float* wt = weights + (is_q ? 0 : 256);
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              // (past the head's end what is read is not used)
              const uint64_t w2 = VEC > 1 ? *reinterpret_cast<const uint64_t*>(wt + (in[y][x] ? at[y][x] : 0) + 2 * i)
                                          : f2_pack(wt[in[y][x] ? at[y][x] : 0], 0.f);
              f[y][x][i] = fmul2(fmul2(f[y][x][i], inv2), w2);
            }
      }
      if (r >= rows || !ok) continue;
      T* dst = is_q ? dq + r * D : (is_v ? dv : dk) + (APPEND ? (long long)r * kv_row : (long long)(r * D));
#pragma unroll
      for (int y = 0; y < NC; ++y) {
        if (!is_v) {
          uint64_t o[2][N2];
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int i = 0; i < N2; ++i) {
                const uint64_t v = f[y][x][i], swapped = f2_pack(f2_hi(v), f2_lo(v));
                const uint64_t turned = ffma2(v, c2[y][x * V2 + i], fmul2(swapped, s2[y][x * V2 + i]));
                o[x][i] = WHOLE || pair[y][x] + i < R / 2 ? turned : v;
              }
          } else {
            const bool on = WHOLE || pair[y][0] < R / 2;
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              const uint64_t p = f[y][0][i], q = f[y][1][i], qs = fmul2(q, s2[y][i]);
              const uint64_t minus = qs ^ 0x8000000080000000ull;
              o[0][i] = on ? ffma2(p, c2[y][i], minus) : p;
              o[1][i] = on ? ffma2(p, s2[y][i], fmul2(q, c2[y][i])) : q;
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              if constexpr (sizeof(T) == 2 && VEC > 1) {
                reinterpret_cast<uint32_t*>(&u4[y][x])[i] = pack_bf16x2(f2_lo(o[x][i]), f2_hi(o[x][i]));
              } else {
                u4[y][x].e[VEC > 1 ? 2 * i : 0] = from_f32<T>(f2_lo(o[x][i]));
                if (VEC > 1) u4[y][x].e[VEC > 1 ? 2 * i + 1 : 0] = from_f32<T>(f2_hi(o[x][i]));
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

template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND, bool WHOLE, bool NORM>
cudaError_t launch(RotaryArgs& a, cudaStream_t s) {
  const int R = a.rot.R, chunks = a.D / VEC;
  const int slots = INTERLEAVED ? (chunks + 1) / 2 : R / (2 * VEC) + ((a.D - R) / VEC + 1) / 2;
  a.lpr_shift = 0;
  while ((NC << a.lpr_shift) < slots) ++a.lpr_shift;
  const int rows = a.H + (APPEND ? 2 : 1) * a.Hkv, at_once = (32 >> a.lpr_shift) * kUnroll;
  a.groups = (rows + at_once - 1) / at_once;
  a.inv_d = 1.f / (float)a.D;
  const long long units = (long long)a.T * a.groups, most = (long long)kBlocks * device_sm_count();
  const long long blocks = (units + kWarps - 1) / kWarps;
  auto kern = rotary_kernel<T, VEC, NC, INTERLEAVED, APPEND, WHOLE, NORM>;
  constexpr size_t bytes = kTables + kWarps * warp_smem<VEC * (int)sizeof(T), NC>();
  static std::atomic<int> done{0};
  const cudaError_t e = allow_smem(kern, bytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), bytes, s, a);
}

template <typename T, int VEC, int NC, bool INTERLEAVED, bool APPEND, bool WHOLE = false>
cudaError_t launch_norm(RotaryArgs& a, cudaStream_t s) {
  return a.qw != nullptr || a.kw != nullptr ? launch<T, VEC, NC, INTERLEAVED, APPEND, WHOLE, true>(a, s)
                                            : launch<T, VEC, NC, INTERLEAVED, APPEND, WHOLE, false>(a, s);
}

template <bool APPEND, typename T>
cudaError_t launch_type(RotaryArgs& a, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int half = a.rot.R / 2;
  const bool whole = a.rot.R == a.D;
  if (a.rot.layout == MOE_ROTARY_INTERLEAVED)
    return whole ? launch_norm<T, V, 1, true, APPEND, true>(a, s) : launch_norm<T, V, 1, true, APPEND>(a, s);
  if (half % V == 0) return whole ? launch_norm<T, V, 1, false, APPEND, true>(a, s) : launch_norm<T, V, 1, false, APPEND>(a, s);
  if (V > 4 && half % 4 == 0) return launch_norm<T, 4, 1, false, APPEND>(a, s);
  if (half % 2 == 0) return launch_norm<T, 2, 2, false, APPEND>(a, s);
  return launch_norm<T, 1, 4, false, APPEND>(a, s);
}

template <bool APPEND>
cudaError_t launch(RotaryArgs& a, int dt, cudaStream_t s) {
  return dt == MOE_DTYPE_BF16 ? launch_type<APPEND, __nv_bfloat16>(a, s) : launch_type<APPEND, float>(a, s);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs& a, int dt, cudaStream_t s) { return launch<false>(a, dt, s); }
cudaError_t launch_cache_append(RotaryArgs& a, cudaStream_t s) { return launch<true>(a, a.c.dt, s); }

}  // namespace moe

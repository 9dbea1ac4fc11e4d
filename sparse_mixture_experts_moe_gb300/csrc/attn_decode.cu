// Decode attention over the paged cache (bf16, heads of up to 128 elements): one query token a sequence.
// Three launches: the shared prefix on the tensor cores (attn_tc.cu, all sequences' rows against each key block
// once), each sequence's own keys (here), and the join of the pieces.
//
// Own keys are an HBM stream: every key and value is read once and meets the G rows of its head group, far
// too few to fill a 128-row tile, so the products are m16n8k16 MMAs with the rows padded to 16.
//   work    a segment is (sequence, key/value head, group of 16 rows); its keys go in blocks of 64. All
//           segments' blocks laid end to end are cut into equal runs, one a CTA: lengths live on the device and
//           differ wildly, and equal runs keep every SM streaming whatever they are. A segment cut by a run's end
//           leaves pieces that the join adds up, in order.
//   warps   4, each with 16 keys of every block, its own ring of TMA copies (16 rows of K and V, swizzled: a box
//           never crosses a page) and its own running maximum: no barrier between warps until a segment
//           ends. Two CTAs an SM with 3 stages hold 2 x 4 x 2 x 8 KB = 128 KB in flight, more than the
//           latency of HBM times its rate (about 50 KB an SM).
// Piece (segment s, CTA c) has number s + c: going along the blocks, s or c grows by one from piece to piece.
#include <cuda.h>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kSlice = 2048;   // sequences a launch takes: their block counts are scanned in shared memory
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;      // keys of a warp's chunk
constexpr int kBlock = kWarps * kKeys;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;

template <int DP> constexpr int kHalf = DP * kKeys * 2;  // bytes of a chunk's K (or V)

template <int DP> __host__ __device__ constexpr size_t own_smem(int n) {
  return 1024 + (size_t)kWarps * kStages * 2 * kHalf<DP> + 16 * DP * 4 + 2 * kWarps * 16 * 4 + 8 * kWarps * kStages + 16 +
         4 * (size_t)(n + 1) + 4 * kThreads;
}

struct OwnArgs {
  DecodeArgs d;
  float* o;        // [piece][rows][D]
  float2* ml;      // [piece][rows]
  int32_t* prefix; // [n + 1] blocks of one head group before sequence i, then [n + 1] = blocks per CTA
  const float* sh_o;      // [(sequence, head)][splits][D]
  const float2* sh_ml;
  int splits;      // pieces of a row over the shared keys
  int first;       // sequence number of the slice's first row (for errors)
};

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

// A walk over the blocks of a run.
struct Cursor {
  int i, hr, b, nb;  // sequence, head group, block, blocks of the sequence
};
__device__ __forceinline__ void advance(Cursor& c, const int* P, int n, int HR) {
  if (++c.b < c.nb) return;
  c.b = 0;
  if (++c.hr < HR) return;
  c.hr = 0;
  do {
    if (++c.i >= n) return;
    c.nb = P[c.i + 1] - P[c.i];
  } while (c.nb == 0);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
decode_own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ OwnArgs a) {
  constexpr int KS = DP / 16;  // k-steps of the scores
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  float* buf = reinterpret_cast<float*>(gbase + kWarps * kStages * 2 * kHalf<DP>);  // [16][DP]
  float* sm_m = buf + 16 * DP;        // [warps][16]
  float* sm_l = sm_m + kWarps * 16;   // [warps][16]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm_l + kWarps * 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kStages);
  int* P = reinterpret_cast<int*>(bars + kWarps * kStages + 2);  // [n + 1]
  const int n = a.d.n, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* sums = P + n + 1;              // [kThreads]
  const CacheView& c = a.d.c;
  const int G = a.d.H / c.Hkv, RG = (G + 15) / 16, HR = c.Hkv * RG, R = G < 16 ? G : 16, D = c.D;

  if (tid == 0) {
    for (int s = 0; s < kWarps * kStages; ++s) mbar_init(smem_u32(bars + s), 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- blocks of every sequence, scanned
  const int chunk = (n + kThreads - 1) / kThreads, i0 = min(n, tid * chunk), i1 = min(n, i0 + chunk);
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    const int s = a.d.slots[i];
    int len = 0;
    if (s >= 0 && s < c.n_slots) len = c.lens[s];
    const bool bad = s < 0 || s >= c.n_slots || len < 0 || (long long)len > ((long long)c.width << c.page_shift);
    if (bad) {
      if (blockIdx.x == 0) record_error(a.d.status, MOE_ERR_DEVICE_CHECK, a.first + i);
      len = 0;
    }
    const int nb = len > a.d.shared ? (len - a.d.shared + kBlock - 1) / kBlock : 0;
    P[i + 1] = nb;
    mine += nb;
  }
  sums[tid] = mine;
  __syncthreads();
  if (warp == 0) {
    int v[kThreads / 32], t = 0;
#pragma unroll
    for (int j = 0; j < kThreads / 32; ++j) {
      v[j] = t;
      t += sums[lane * (kThreads / 32) + j];
    }
    int incl = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
#pragma unroll
    for (int j = 0; j < kThreads / 32; ++j) sums[lane * (kThreads / 32) + j] = incl - t + v[j];
  }
  __syncthreads();
  int run = sums[tid];
  for (int i = i0; i < i1; ++i) {
    run += P[i + 1];
    P[i + 1] = run;
  }
  if (tid == 0) P[0] = 0;
  __syncthreads();
  const long long total = (long long)P[n] * HR;
  const int per = (int)((total + gridDim.x - 1) / gridDim.x);
  if (blockIdx.x == 0) {
    for (int i = tid; i <= n; i += kThreads) a.prefix[i] = P[i];
    if (tid == 0) a.prefix[n + 1] = per;
  }
  // that the slots share what the caller says they share
  if (a.d.shared > 0) {
    const int s0 = a.d.slots[0], pages = a.d.shared >> c.page_shift;
    if (s0 >= 0 && s0 < c.n_slots)
      for (long long x = (long long)blockIdx.x * kThreads + tid; x < (long long)n * pages; x += (long long)gridDim.x * kThreads) {
        const int i = (int)(x / pages), p = (int)(x % pages), s = a.d.slots[i];
        if (s < 0 || s >= c.n_slots || (p << c.page_shift) >= c.lens[s]) continue;
        const int page = c.table[(long long)s * c.width + p];
        if (page < 0 || page >= c.n_pages || page != c.table[(long long)s0 * c.width + p])
          record_error(a.d.status, MOE_ERR_DEVICE_CHECK, a.first + i);
      }
  }
  const long long begin = (long long)blockIdx.x * per, end = min(total, begin + per);
  if (begin >= end) return;

  Cursor cu;
  {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)P[mid] * HR <= begin) lo = mid; else hi = mid - 1;
    }
    cu.i = lo;
    cu.nb = P[lo + 1] - P[lo];
    const int r = (int)(begin - (long long)P[lo] * HR);
    cu.hr = r / cu.nb;
    cu.b = r % cu.nb;
  }
  Cursor ld = cu;
  const int count = (int)(end - begin);
  const uint32_t ring = base + warp * kStages * 2 * kHalf<DP>;
  const uint32_t bar0 = smem_u32(bars + warp * kStages);

  // ---- this warp's copies, kStages chunks ahead
  int ld_slot_i = -1, ld_slot = 0;
  uint32_t issued = 0;
  auto issue = [&](int stage) {
    if (ld.i != ld_slot_i) { ld_slot_i = ld.i; ld_slot = a.d.slots[ld.i]; }
    const int key = a.d.shared + ld.b * kBlock + warp * kKeys, len = c.lens[ld_slot];
    if (key < len) {
      int page = c.table[(long long)ld_slot * c.width + (key >> c.page_shift)];
      if (page < 0 || page >= c.n_pages) {
        record_error(a.d.status, MOE_ERR_DEVICE_CHECK, a.first + ld.i);
        page = 0;
      }
      const int row = (page * c.Hkv + ld.hr / RG) * c.page_size + (key & (c.page_size - 1));
      const uint32_t dst = ring + stage * 2 * kHalf<DP>, b = bar0 + 8 * stage;
      mbar_arrive_expect_tx(b, 2 * kHalf<DP>);
#pragma unroll
      for (int h = 0; h < DP / 64; ++h) {
        tma_load_2d(dst + h * 2048, &tmK, 64 * h, row, b);
        tma_load_2d(dst + kHalf<DP> + h * 2048, &tmV, 64 * h, row, b);
      }
    } else {
      mbar_arrive(bar0 + 8 * stage);  // nothing of this block for this warp
    }
    issued |= 1u << stage;
    advance(ld, P, n, HR);
  };
  __syncwarp();
  if (lane == 0)
    for (int s = 0; s < kStages && s < count; ++s) issue(s);

  const float c2 = a.d.scale * 1.4426950408889634f, thr = 8.0f / c2;
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t q[KS][4];
  float o[DP / 8][4], m[2], l[2];
  int cur_i = -1, cur_hr = -1, len = 0, slot = 0;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;

  for (int x = 0; x < count; ++x) {
    if (cu.i != cur_i || cu.hr != cur_hr) {  // a new segment: its rows as A fragments
      if (cu.i != cur_i) {
        slot = a.d.slots[cu.i];
        len = c.lens[slot];
      }
      cur_i = cu.i;
      cur_hr = cu.hr;
      const int hk = cu.hr / RG, r0 = (cu.hr % RG) * 16, nr = min(R, G - r0);
      const __nv_bfloat16* qp = (const __nv_bfloat16*)a.d.q + (long long)cu.i * a.d.qs + (long long)(hk * G + r0) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = g + 8 * (e & 1), col = 16 * k + 2 * t4 + 8 * (e >> 1);
          q[k][e] = row < nr && col < D ? *reinterpret_cast<const uint32_t*>(qp + row * D + col) : 0u;
        }
#pragma unroll
      for (int j = 0; j < DP / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    if (ok) ok = warp_wait(bar0 + 8 * stage, phase, a.d.timeout_ns, abort_flag, a.d.status, 61);
    const int key = a.d.shared + cu.b * kBlock + warp * kKeys, left = len - key;
    if (ok && left > 0) {
      const uint32_t sk = ring + stage * 2 * kHalf<DP>, sv = sk + kHalf<DP>;
      if (left < kKeys) {  // positions past the end hold anything: zero their values
        for (int z = lane; z < (kKeys - left) * (DP / 64) * 8; z += 32) {
          const int rr = left + z / ((DP / 64) * 8), u = z % ((DP / 64) * 8);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sv + (u >> 3) * 2048 + rr * 128 + (u & 7) * 16), "r"(0)
                       : "memory");
        }
        __syncwarp();
      }
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kp = 0; kp < KS / 2; ++kp)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int row = 8 * nt + (lane & 7), u = 4 * kp + (lane >> 3);
          uint32_t b[4];
          ldsm4(sk + (u >> 3) * 2048 + row * 128 + (((u & 7) ^ (row & 7)) << 4), b);
          mma16816(s[nt], q[2 * kp], b[0], b[1]);
          mma16816(s[nt], q[2 * kp + 1], b[2], b[3]);
        }
      if (left < kKeys)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * nt + 2 * t4 + (e & 1) >= left) s[nt][e] = -INFINITY;
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      // rescaled only when a maximum rises by more than 2^8 (as in attn_tc.cu)
      if (__any_sync(0xffffffffu, mx[0] > m[0] + thr || mx[1] > m[1] + thr)) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (mx[r] > m[r] + thr) {
            const float al = ex2((m[r] - mx[r]) * c2);
            l[r] *= al;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) { o[j][2 * r] *= al; o[j][2 * r + 1] *= al; }
            m[r] = mx[r];
          }
      }
      uint32_t p[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mc = m[r] == -INFINITY ? 0.f : m[r] * c2;
        const float p0 = ex2(fmaf(s[0][2 * r], c2, -mc)), p1 = ex2(fmaf(s[0][2 * r + 1], c2, -mc));
        const float p2 = ex2(fmaf(s[1][2 * r], c2, -mc)), p3 = ex2(fmaf(s[1][2 * r + 1], c2, -mc));
        l[r] += (p0 + p1) + (p2 + p3);
        p[r] = pack_bf16x2(p0, p1);
        p[2 + r] = pack_bf16x2(p2, p3);
      }
#pragma unroll
      for (int np = 0; np < DP / 16; ++np) {
        const int mi = lane >> 3, row = (mi & 1) * 8 + (lane & 7), u = 2 * np + (mi >> 1);
        uint32_t b[4];
        ldsm4t(sv + (u >> 3) * 2048 + row * 128 + (((u & 7) ^ (row & 7)) << 4), b);
        mma16816(o[2 * np], p, b[0], b[1]);
        mma16816(o[2 * np + 1], p, b[2], b[3]);
      }
    }
    if (left < kKeys) fence_proxy_async_smem();  // the zeros above before the next copy into this stage
    __syncwarp();
    if (lane == 0 && x + kStages < count) issue(stage);
    if (++stage == kStages) { stage = 0; phase ^= 1u; }

    const Cursor was = cu;
    advance(cu, P, n, HR);
    if (x + 1 < count && cu.i == was.i && cu.hr == was.hr) continue;
    // ---- the segment (or the run) ends: the four warps' parts become one piece
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t4 == 0) {
        sm_m[warp * 16 + g + 8 * r] = m[r];
        sm_l[warp * 16 + g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float M = -INFINITY;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) M = fmaxf(M, sm_m[y * 16 + g + 8 * r]);
      w[r] = M == -INFINITY ? 0.f : ex2((m[r] - M) * c2);
    }
    for (int y = 0; y < kWarps; ++y) {
      if (warp == y)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (g + 8 * r < R)
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) {
              float2* d = reinterpret_cast<float2*>(buf + (g + 8 * r) * DP + 8 * j + 2 * t4);
              float2 v = make_float2(o[j][2 * r] * w[r], o[j][2 * r + 1] * w[r]);
              if (y > 0) { const float2 before = *d; v.x += before.x; v.y += before.y; }
              *d = v;
            }
      __syncthreads();
    }
    const int nr = min(R, G - (was.hr % RG) * 16);
    const long long piece = (long long)was.i * HR + was.hr + blockIdx.x;
    for (int z = tid; z < nr * (D / 4); z += kThreads) {
      const int row = z / (D / 4), col = (z % (D / 4)) * 4;
      *reinterpret_cast<float4*>(a.o + (piece * R + row) * D + col) = *reinterpret_cast<const float4*>(buf + row * DP + col);
    }
    if (tid < nr) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) M = fmaxf(M, sm_m[y * 16 + tid]);
#pragma unroll
      for (int y = 0; y < kWarps; ++y)
        if (M != -INFINITY) L += sm_l[y * 16 + tid] * ex2((sm_m[y * 16 + tid] - M) * c2);
      a.ml[piece * R + tid] = make_float2(M * c2, L);
    }
    __syncthreads();
  }
  // copies still in flight (after a wait that gave up) land before shared memory goes away
  if (!ok && lane == 0)
    for (int s = 0; s < kStages; ++s)
      if (issued & (1u << s)) {
        mbar_wait_bounded(bar0 + 8 * s, 0, a.d.timeout_ns);
        mbar_wait_bounded(bar0 + 8 * s, 1, a.d.timeout_ns);
      }
}

// One warp a (sequence, head): its pieces over the shared keys, then over its own, in order.
__global__ void __launch_bounds__(128)
decode_join_kernel(const __grid_constant__ OwnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const CacheView& c = a.d.c;
  const int H = a.d.H, G = H / c.Hkv, RG = (G + 15) / 16, HR = c.Hkv * RG, R = G < 16 ? G : 16, D = c.D;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.d.n * H) return;
  const int i = (int)(row / H), h = (int)(row % H), hr = (h / G) * RG + (h % G) / 16, r = (h % G) % 16;
  const int s = a.d.slots[i];
  const bool valid = s >= 0 && s < c.n_slots;
  const int b = a.prefix[i + 1] - a.prefix[i], per = a.prefix[a.d.n + 1];
  const int shared = valid ? a.splits : 0;
  int own = 0;
  long long p0 = 0;
  if (valid && b > 0) {
    const long long start = (long long)a.prefix[i] * HR + (long long)hr * b;
    const int c0 = (int)(start / per), c1 = (int)((start + b - 1) / per);
    own = c1 - c0 + 1;
    p0 = (long long)i * HR + hr + c0;
  }
  const int count = shared + own;
  auto ml = [&](int x) { return x < shared ? a.sh_ml[row * a.splits + x] : a.ml[(p0 + x - shared) * R + r]; };
  float M = -INFINITY;
  for (int x = lane; x < count; x += 32) M = fmaxf(M, ml(x).x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int x0 = 0; x0 < count; x0 += 32) {
    float2 v = make_float2(-INFINITY, 0.f);
    if (x0 + lane < count) v = ml(x0 + lane);
    const float wv = ex2(v.x - ref), lw = wv * v.y;
    const int m = min(32, count - x0);
#pragma unroll 4
    for (int y = 0; y < m; ++y) {
      const float w = __shfl_sync(0xffffffffu, wv, y);
      l += __shfl_sync(0xffffffffu, lw, y);
      const int x = x0 + y;
      const float* src = x < shared ? a.sh_o + (row * a.splits + x) * D : a.o + ((p0 + x - shared) * R + r) * D;
      if (lane * 4 < D) {
        const float4 u = *reinterpret_cast<const float4*>(src + lane * 4);
        o.x = fmaf(w, u.x, o.x);
        o.y = fmaf(w, u.y, o.y);
        o.z = fmaf(w, u.z, o.z);
        o.w = fmaf(w, u.w, o.w);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (lane * 4 < D) {
    uint2 u;
    u.x = pack_bf16x2(o.x * inv, o.y * inv);
    u.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.d.out + (long long)i * a.d.os + (long long)h * D + lane * 4) = u;
  }
  if (a.d.lse != nullptr && lane == 0) a.d.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

bool encode_pages(EncodeTiledFn enc, CUtensorMap* m, const void* p, const CacheView& c, int rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)c.D, (cuuint64_t)c.n_pages * c.Hkv * c.page_size};
  const cuuint64_t str[1] = {(cuuint64_t)c.D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)rows};
  return encode_tmap(enc, m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 2, dims, str, box);
}

template <int DP>
cudaError_t launch_own(const CUtensorMap& tk, const CUtensorMap& tv, const OwnArgs& o, int ctas, cudaStream_t s) {
  const size_t smem = own_smem<DP>(o.d.n);
  const cudaError_t e = cudaFuncSetAttribute(decode_own_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_own_kernel<DP>, dim3(ctas), dim3(kThreads), smem, s, tk, tv, o);
}

}  // namespace

cudaError_t launch_attn_decode_tc(const DecodeArgs& all, cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap ok{}, ov{};
  if (!encode_pages(enc, &ok, all.k, all.c, kKeys) || !encode_pages(enc, &ov, all.v, all.c, kKeys))
    return cudaErrorInvalidValue;
  const int G = all.H / all.c.Hkv, RG = (G + 15) / 16, HR = all.c.Hkv * RG, R = G < 16 ? G : 16, D = all.c.D;
  const int ctas = device_sm_count() * kCtasPerSm;
  for (int first = 0; first < all.n; first += kSlice) {
    DecodeArgs d = all;
    d.n = all.n - first < kSlice ? all.n - first : kSlice;
    d.q = (const __nv_bfloat16*)all.q + (long long)first * all.qs;
    d.out = (__nv_bfloat16*)all.out + (long long)first * all.os;
    d.slots = all.slots + first;
    if (all.lse != nullptr) d.lse = all.lse + (long long)first * all.H;
    OwnArgs o;
    o.d = d;
    o.first = first;
    o.splits = 0;
    // pieces: own ones [(n HR + ctas)][R], then the shared ones [n H][splits]; see decode_pieces
    const long long own_rows = ((long long)d.n * HR + ctas) * R;
    o.o = all.part;
    float* sh = all.part + own_rows * D;
    if (d.shared > 0) o.splits = attn_shared_splits(d);
    const long long sh_rows = (long long)d.n * d.H * o.splits;
    o.sh_o = sh;
    o.ml = reinterpret_cast<float2*>(sh + sh_rows * D);
    o.sh_ml = o.ml + own_rows;
    o.prefix = reinterpret_cast<int32_t*>(const_cast<float2*>(o.sh_ml) + sh_rows);
    if (own_rows + sh_rows + 2 * kSlice > decode_pieces((long long)all.n * all.H)) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (d.shared > 0) e = launch_attn_shared_tc(d, o.splits, sh, const_cast<float2*>(o.sh_ml), s);
    if (e == cudaSuccess)
      e = D <= 64 ? launch_own<64>(ok, ov, o, ctas, s) : launch_own<128>(ok, ov, o, ctas, s);
    if (e == cudaSuccess)
      e = launch_pdl(decode_join_kernel, dim3((unsigned)(((long long)d.n * d.H + 3) / 4)), dim3(128), 0, s, o);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe

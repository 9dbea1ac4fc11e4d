// Attention on the 5th-generation tensor cores (bf16, heads of up to 128 elements): packed prompts, and the
// shared prefix of a decode batch.
//   S = Q K^T (scores), P = 2^(c S - c m) (weights, c = scale log2 e), O += P V, out = O / l
// with m a running reference of each row and l the sum of its weights, in one pass over the keys: no score
// ever leaves the SM.
//
// One CTA per SM takes 256 packed rows (two tiles of 128) of one key/value head; the tiles share every
// key/value block (128 keys), which halves the reads of L2 against one tile a CTA.
//   warps 0..3, 4..7  softmax of tile 0 / 1: thread = row = TMEM lane. Reads S, takes the maximum, writes P
//                     (bf16) over S's own columns, sums the weights
//   warp 8            allocates TMEM; one thread issues every MMA: QK with both operands in shared memory, PV
//                     with P read from TMEM as the A operand
//   warp 9            one thread loads K and V blocks by TMA into a ring (K0 V0 K1 V1 ...)
// TMEM (512 columns): S0 S1 (128 fp32 columns each, P in the first 64), O0 O1.
// The MMAs go PV0(j) QK0(j+1) PV1(j) QK1(j+1): while one tile is in softmax the tensor cores work on the
// other. QK(j+1) may overwrite P(j) because MMAs of one thread run in issue order.
// O is only rescaled when a row's maximum rises by more than 8 in log2 units above the reference m (weights
// then stay below 2^8, exact enough for bf16 as only their relative precision counts); the softmax
// warp that sees it waits for the last PV and scales the 32 rows of O itself. After the first blocks
// that is rare, so no warps are kept for it.
// A weight is rounded to bf16 (half a step, 2^-9 of it) because the MMA takes both operands in one type; its
// sum l takes the unrounded value.
// Keys past a row's limit get weight 0 by index. 0 times a non-finite value in V would still be NaN: a row whose
// result is not finite is computed again, key by key over the keys it sees (exact_row), so that a
// non-finite value reaches only rows that see it. That costs nothing where everything is finite.
// All waits are bounded, as in ffn_tc.cu.
#include <cuda.h>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int BK = 128;       // keys per block
constexpr int TM = 128;       // rows per tile
// Registers: 12 warps of 168 at launch (64512); the softmax warps take 216 each (a row of 128 scores stays in
// registers), the other four keep 72: 8 * 32 * 216 + 4 * 32 * 72 = 64512.
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kMaxSmem = 232448;
constexpr float kRescale = 8.0f;  // log2 units

template <int DP> struct Cfg {
  static constexpr int kChunks = DP / 64;          // 64-element (128-byte) swizzle columns of a row
  static constexpr int kTileBytes = TM * DP * 2;   // a Q tile, and a K or V block
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr int kBars = 2 * kStages + 2 + 2 + 2 + 2 + 1;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kStages) * kTileBytes + 8 * kBars + 16;
};
static_assert(Cfg<128>::kSmem <= kMaxSmem && Cfg<64>::kSmem <= kMaxSmem, "shared memory");

// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem desc].
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// One row again, key by key (a warp; lane owns 4 consecutive elements): only keys below lim take part.
// at(j, k, v) gives key j's element offsets.
template <typename At>
__device__ __forceinline__ void exact_row(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v, At at,
                                          int D, int lim, float c2, float (&o)[4], float& m, float& l) {
  const int d = (int)(threadIdx.x & 31) * 4;
  const bool on = d < D;
  float qv[4] = {0.f, 0.f, 0.f, 0.f};
  if (on)
#pragma unroll
    for (int e = 0; e < 4; ++e) qv[e] = __bfloat162float(q[d + e]);
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = 0.f;
  for (int j = 0; j < lim; ++j) {
    float s = 0.f;
    long long ko, vo;
    at(j, ko, vo);
    if (on)
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(qv[e], __bfloat162float(k[ko + d + e]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= c2;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref), p = ex2(s - ref);
    l = fmaf(l, a, p);
    m = mn;
    if (on)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fmaf(p, __bfloat162float(v[vo + d + e]), o[e] * a);
  }
}

struct SharedArgs {
  DecodeArgs d;
  int per;        // keys of a split, a multiple of BK
  int splits;
  float* part_o;  // [piece][D]
  float2* part_ml;
};

// SHARED = false: blockIdx.x = tile-pair slot (descending, so that the longest rows of a sequence start first) and
// key/value head. SHARED = true: blockIdx = (key/value head, row pair, split of the shared keys); rows are
// (sequence, head) pairs, and each row's piece goes to the workspace unnormalised.
template <int DP, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ PromptArgs pa, const __grid_constant__ SharedArgs sa, int n_slots) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base, sKV = base + 2 * C::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + (2 + C::kStages) * C::kTileBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int FULL = 0, EMPTY = C::kStages, QFULL = 2 * C::kStages, SFULL = QFULL + 2, PFULL = SFULL + 2,
                ODONE = PFULL + 2, DONE = ODONE + 2;

  // (the shuffle tells the compiler that the warp number is the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(bar(FULL + s), 1); mbar_init(bar(EMPTY + s), 1); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(QFULL + t), 4);
      mbar_init(bar(SFULL + t), 1);
      mbar_init(bar(PFULL + t), 4);
      mbar_init(bar(ODONE + t), 1);
    }
    mbar_init(bar(DONE), 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kSoftWarps) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  // Only after TMEM is allocated: a dependent kernel that starts on this SM may allocate some before it waits for this
  // grid. And only after the wait: the decode's own-key kernel relies on everything before this grid being done.
  griddep_launch_dependents();

  // ---- the CTA's rows and keys
  const int H = SHARED ? sa.d.H : pa.H, Hkv = SHARED ? sa.d.c.Hkv : pa.Hkv, D = SHARED ? sa.d.c.D : pa.D;
  const int G = H / Hkv;
  int* status = SHARED ? sa.d.status : pa.status;
  const uint64_t timeout_ns = SHARED ? sa.d.timeout_ns : pa.timeout_ns;
  int hk, row0, nrows;        // packed rows row0 .. row0 + nrows - 1 of the sequence (or batch)
  int key0 = 0, n_keys;       // keys of this CTA
  int lim_t[2];               // keys that each tile's last row sees (relative to key0)
  Seq sq{0, 0, 0, 0};
  if (SHARED) {
    hk = blockIdx.x;
    row0 = blockIdx.y * 2 * TM;
    nrows = min(2 * TM, sa.d.n * G - row0);
    key0 = blockIdx.z * sa.per;
    n_keys = min(sa.per, sa.d.shared - key0);
    lim_t[0] = n_keys;
    lim_t[1] = nrows > TM ? n_keys : 0;
  } else {
    hk = blockIdx.x % Hkv;
    const int slot = n_slots - 1 - (int)(blockIdx.x / Hkv);
    const int i = find_tile_seq_warp(pa.qo, pa.n, G, 2 * TM, slot);
    sq = load_seq_warp(pa, i);
    const long long r0 = ((long long)slot - ((long long)sq.q0 * G / (2 * TM) + i)) * (2 * TM);
    const bool none = r0 < 0 || r0 >= (long long)sq.nq * G;  // a slot that no tile fills
    row0 = none ? 0 : (int)r0;
    nrows = none ? 0 : min(2 * TM, sq.nq * G - row0);
    key0 = 0;
    lim_t[0] = none ? 0 : visible_keys((row0 + min(nrows, TM) - 1) / G, sq.nq, sq.nk, pa.causal);
    lim_t[1] = nrows > TM ? visible_keys((row0 + nrows - 1) / G, sq.nq, sq.nk, pa.causal) : 0;
    n_keys = max(lim_t[0], lim_t[1]);
  }
  const int nb0 = (lim_t[0] + BK - 1) / BK, nb1 = (lim_t[1] + BK - 1) / BK, nb = max(nb0, nb1);

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");  // all four warps of the group, 10 and 11 idle
    if (warp == kSoftWarps + 1 && lane == 0) {
      // -------------------------------------------------------------- loads
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_phase = 0;
      const int32_t* table = nullptr;
      int pages = 0;
      if (SHARED) {
        int slot = sa.d.slots[0];  // an out-of-range slot or page is recorded by the own part
        slot = slot < 0 || slot >= sa.d.c.n_slots ? 0 : slot;
        table = sa.d.c.table + (long long)slot * sa.d.c.width;
        pages = sa.d.shared >> sa.d.c.page_shift;
      }
      for (int u = 0; u < 2 * nb; ++u) {
        const CUtensorMap* tm = (u & 1) ? &tmV : &tmK;
        const int j0 = key0 + (u >> 1) * BK;
        if (!wait_or_abort(bar(EMPTY + stage), phase ^ 1u, timeout_ns, abort_flag, status, 51)) break;
        const uint32_t dst = sKV + stage * C::kTileBytes;
        mbar_arrive_expect_tx(bar(FULL + stage), C::kTileBytes);
        if (SHARED) {
          const int rows = min(sa.d.c.page_size, BK);
          for (int r = 0; r < BK; r += rows) {
            // past the shared keys the last page again: those columns are masked, their values finite or seen anyway
            const int p = min((j0 + r) >> sa.d.c.page_shift, pages - 1);
            int page = table[p];
            page = page < 0 || page >= sa.d.c.n_pages ? 0 : page;
            const int g = (page * Hkv + hk) * sa.d.c.page_size + ((j0 + r) & (sa.d.c.page_size - 1));
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(dst + c * (BK * 128) + r * 128, tm, 64 * c, g, sa.d.layer, bar(FULL + stage));
          }
        } else {
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(dst + c * (BK * 128), tm, 64 * c, hk, sq.k0 + j0, bar(FULL + stage));
        }
        filled |= 1u << stage;
        fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
      for (int s = 0; s < C::kStages; ++s)
        if (filled & (1u << s)) mbar_wait_bounded(bar(FULL + s), (fill_phase >> s) & 1u, timeout_ns);
    }
    if (warp == kSoftWarps) {
      // -------------------------------------------------------------- MMAs
      // The whole warp walks the loop and one elected thread issues: descriptors and addresses then stay in uniform
      // registers. Inside a one-lane branch every MMA first moved its operands there, which took as long as
      // the MMA itself (about 70 of 64 cycles).
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int n0 = __shfl_sync(0xffffffffu, nb0, 0), n1 = __shfl_sync(0xffffffffu, nb1, 0), nn = max(n0, n1);
      constexpr uint32_t idesc_qk = make_idesc_bf16_f32(TM, BK, false);
      constexpr uint32_t idesc_pv = make_idesc_bf16_f32(TM, DP, true);
      int stage = 0;
      uint32_t phase = 0;
      auto wait = [&](int b, uint32_t ph) {
        const bool ok = warp_wait(bar(b), ph, timeout_ns, abort_flag, status, 52);
        tc_fence_after();
        return ok;
      };
      // three barriers at once: the tests go out together, as each takes about 100 cycles to answer (and waits in the
      // warp's queue behind the MMAs issued before it)
      auto wait3 = [&](int b0, uint32_t p0, int b1, uint32_t p1, int b2, uint32_t p2) {
        const bool r0 = mbar_try_wait_long(bar(b0), p0), r1 = mbar_try_wait_long(bar(b1), p1),
                   r2 = mbar_try_wait_long(bar(b2), p2);
        if (!__builtin_expect(__all_sync(0xffffffffu, r0 && r1 && r2), 1)) {
          if (!warp_wait(bar(b0), p0, timeout_ns, abort_flag, status, 52)) return false;
          if (!warp_wait(bar(b1), p1, timeout_ns, abort_flag, status, 52)) return false;
          if (!warp_wait(bar(b2), p2, timeout_ns, abort_flag, status, 52)) return false;
        }
        tc_fence_after();
        return true;
      };
      auto qk = [&](int t, int st) {
        const uint64_t a = make_smem_desc_sw128(sQ + t * C::kTileBytes, 16, 1024);
        const uint64_t b = make_smem_desc_sw128(sKV + st * C::kTileBytes, 16, 1024);
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * (TM * 128) + (kk % 4) * 32) >> 4);
          tc_mma_f16(tm + t * BK, a + off, b + off, idesc_qk, kk != 0);
        }
        tc_commit(bar(SFULL + t));
      };
      auto pv = [&](int t, int st, bool acc) {
        const uint64_t b = make_smem_desc_sw128(sKV + st * C::kTileBytes, BK * 128, 1024);
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_f16_ta(tm + 256 + t * DP, tm + t * BK + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                        acc || kk != 0);
        tc_commit(bar(ODONE + t));
      };
      auto next = [&]() { if (++stage == C::kStages) { stage = 0; phase ^= 1u; } };
      if (nn > 0) {
        bool ok = wait(FULL + stage, phase);
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t)
          if ((t ? n1 : n0) > 0) {
            ok = wait(QFULL + t, 0);
            if (ok) qk(t, stage);
          }
        if (leader) tc_commit(bar(EMPTY + stage));
        next();
        for (int j = 0; j < nn && ok; ++j) {
          const int vs = stage;
          const uint32_t vp = phase;
          next();
          const int ks = stage;
          const uint32_t kp = phase;
          if (j + 1 < nn) next();
          // V(j), K(j+1) and the first tile's P(j)
          const bool more = j + 1 < nn;
          const int pb = PFULL + (j < n0 ? 0 : 1);
          ok = wait3(FULL + vs, vp, more ? FULL + ks : FULL + vs, more ? kp : vp, pb, j & 1);
          if (!ok) break;
          if (j < n0) {
            pv(0, vs, j > 0);
            if (j + 1 < n0) qk(0, ks);
            if (j < n1) ok = wait(PFULL + 1, j & 1);
          }
          if (ok && j < n1) {
            pv(1, vs, j > 0);
            if (j + 1 < n1) qk(1, ks);
          }
          if (leader) {
            tc_commit(bar(EMPTY + vs));
            if (j + 1 < nn) tc_commit(bar(EMPTY + ks));
          }
        }
      }
      // every MMA has completed before TMEM and shared memory go away
      if (leader) tc_commit(bar(DONE));
      mbar_wait_bounded(bar(DONE), 0, timeout_ns);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2, r = tid & 127;      // tile, row of it
    const int q4 = warp & 3;                     // TMEM lanes 32 q4 ..
    const int nrow_t = min(TM, nrows - t * TM);  // rows of this tile (<= 0: none)
    const int n = t ? nb1 : nb0;
    const int R = row0 + t * TM + r;
    const bool valid = r < nrow_t;
    const int tok = valid ? R / G : 0, h = hk * G + (valid ? R % G : 0);
    // Q tile to shared memory as the swizzled K-major operand, zeros past the rows and past D: each warp its 32 rows,
    // kLanes lanes a row, every load in flight before the first store
    constexpr int kLanes = DP / 8, kIter = kLanes;  // 32 rows / (32 / kLanes) rows a step
    if (n > 0) {
      const __nv_bfloat16* qrow = (const __nv_bfloat16*)(SHARED ? sa.d.q : pa.q) +
                                  (long long)((SHARED ? 0 : sq.q0) + tok) * (SHARED ? sa.d.qs : pa.qs) + (long long)h * D;
      uint4 x[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int rr = i * (32 / kLanes) + lane / kLanes, u = lane % kLanes;
        const __nv_bfloat16* src = (const __nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)qrow, rr);
        x[i] = make_uint4(0, 0, 0, 0);
        if (32 * q4 + rr < nrow_t && u * 8 < D) x[i] = *reinterpret_cast<const uint4*>(src + u * 8);
      }
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int rr = 32 * q4 + i * (32 / kLanes) + lane / kLanes, u = lane % kLanes;
        const uint32_t dst = sQ + t * C::kTileBytes + (u / 8) * (TM * 128) + rr * 128 + (((u & 7) ^ (rr & 7)) * 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(x[i].x), "r"(x[i].y), "r"(x[i].z), "r"(x[i].w)
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(QFULL + t));
    }
    int lim = 0;
    if (valid && SHARED) {  // a slot shorter than the shared keys sees its own length of them
      const int slot = sa.d.slots[tok];
      lim = slot < 0 || slot >= sa.d.c.n_slots ? 0 : max(0, min(n_keys, sa.d.c.lens[slot] - key0));
    } else if (valid) {
      lim = visible_keys(tok, sq.nq, sq.nk, pa.causal);
    }
    const float c2 = (SHARED ? sa.d.scale : pa.scale) * 1.4426950408889634f;
    const float thr = kRescale / c2;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const uint32_t tS = tmem + lanes + t * BK, tO = tmem + lanes + 256 + t * DP;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = warp_wait(bar(SFULL + t), j & 1, timeout_ns, abort_flag, status, 53);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tS + 32 * c, s[c]);
      tmem_ld_wait();
      const int left = lim - j * BK;  // columns that this row sees
      if (__any_sync(0xffffffffu, left < BK)) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= left) s[c][i] = 0xff800000u;  // -inf
      }
      // four chains of three-input maxima (max drops a NaN score: the maximum is never NaN)
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 64; ++i)
        mx4[i & 3] = max3(mx4[i & 3], __uint_as_float(s[i >> 4][2 * (i & 15)]), __uint_as_float(s[i >> 4][2 * (i & 15) + 1]));
      const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
      if (__any_sync(0xffffffffu, mx > m + thr)) {
        const bool up = mx > m + thr;
        if (j > 0) {
          ok = warp_wait(bar(ODONE + t), (j - 1) & 1, timeout_ns, abort_flag, status, 53);
          if (!ok) break;
          tc_fence_after();
          const float a = up ? ex2((m - mx) * c2) : 1.0f;
          l *= a;
#pragma unroll
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st_32x32b_x32(tO + 32 * c, o);
          }
        }
        if (up) m = mx;
      }
      const float mc = m == -INFINITY ? 0.f : -m * c2;
      const uint64_t c2p = f2_pack(c2, c2), mcp = f2_pack(mc, mc);
      // in batches of 16: the arguments and powers of one batch are issued before the sums and packing of the one
      // before, so that nothing waits for a power of two just asked for
      uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[32];
#pragma unroll
        for (int b = 0; b < 5; ++b) {
          if (b < 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t* v = &s[2 * h + (b >> 1)][16 * (b & 1) + 2 * i];
              const uint64_t x = ffma2(((uint64_t)v[1] << 32) | v[0], c2p, mcp);
              v[0] = (uint32_t)x;
              v[1] = (uint32_t)(x >> 32);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t& v = s[2 * h + (b >> 1)][16 * (b & 1) + i];
              v = __float_as_uint(ex2(__uint_as_float(v)));
            }
          }
          if (b > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t* v = &s[2 * h + ((b - 1) >> 1)][16 * ((b - 1) & 1) + 2 * i];
              const uint64_t x = ((uint64_t)v[1] << 32) | v[0];
              if (i & 1) sum1 = fadd2(sum1, x); else sum0 = fadd2(sum0, x);
              p[8 * (b - 1) + i] = pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1]));
            }
          }
        }
        tmem_st_32x32b_x32(tS + 32 * h, p);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(PFULL + t));
      const uint64_t sum = fadd2(sum0, sum1);
      l += f2_lo(sum) + f2_hi(sum);
    }
    // ---- the rows' results
    if (ok && n > 0) {
      ok = warp_wait(bar(ODONE + t), (n - 1) & 1, timeout_ns, abort_flag, status, 53);
      tc_fence_after();
    }
    if (ok && nrow_t > 0 && __any_sync(0xffffffffu, valid)) {
      if (SHARED) {
        const long long piece = ((long long)tok * H + h) * sa.splits + blockIdx.z;
        bool fine = true;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld_32x32b_x32(tO + 32 * c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (lim == 0) o[i] = 0;
            fine = fine && fabsf(__uint_as_float(o[i])) <= 3.0e38f;
          }
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(sa.part_o + piece * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (32 * c + 4 * i < D)
                dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                     __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
        if (valid) sa.part_ml[piece] = make_float2(m * c2, l);
        uint32_t again = __ballot_sync(0xffffffffu, valid && !fine && lim < n_keys);
        while (again != 0) {
          const int w = __ffs(again) - 1;
          again &= again - 1;
          const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
          const int limw = __shfl_sync(0xffffffffu, lim, w);
          const CacheView& cv = sa.d.c;
          const int32_t* row = cv.table + (long long)sa.d.slots[tw] * cv.width;
          float o[4], mw, lw;
          exact_row((const __nv_bfloat16*)sa.d.q + (long long)tw * sa.d.qs + (long long)hw * D,
                    (const __nv_bfloat16*)sa.d.k, (const __nv_bfloat16*)sa.d.v,
                    [&](int j, long long& ko, long long& vo) {
                      const int p = key0 + j;
                      int page = row[p >> cv.page_shift];
                      page = page < 0 || page >= cv.n_pages ? 0 : page;
                      ko = vo = (((long long)page * Hkv + hk) * cv.page_size + (p & (cv.page_size - 1))) * D;
                    },
                    D, limw, c2, o, mw, lw);
          const long long pw = ((long long)tw * H + hw) * sa.splits + blockIdx.z;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (lane * 4 + e < D) sa.part_o[pw * D + lane * 4 + e] = o[e];
          if (lane == 0) sa.part_ml[pw] = make_float2(mw, lw);
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        // the rows go through this warp's part of the Q tile (its last QK is done), so that whole rows are stored at once
        __nv_bfloat16* orow = (__nv_bfloat16*)pa.out + (long long)(sq.q0 + tok) * pa.os + (long long)h * D;
        const uint32_t stg = sQ + t * C::kTileBytes + 32 * q4 * (DP * 2);
        bool fine = true;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld_32x32b_x32(tO + 32 * c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] = lim == 0 ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
            fine = fine && fabsf(__uint_as_float(o[i])) <= 3.0e38f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t dst = stg + lane * (DP * 2) + (((4 * c + i) ^ (lane & 7)) * 16);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst),
                         "r"(pack_bf16x2(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1]))),
                         "r"(pack_bf16x2(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]))),
                         "r"(pack_bf16x2(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]))),
                         "r"(pack_bf16x2(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])))
                         : "memory");
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int rr = i * (32 / kLanes) + lane / kLanes, u = lane % kLanes;
          __nv_bfloat16* dst = (__nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)orow, rr);
          uint4 x;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(stg + rr * (DP * 2) + ((u ^ (rr & 7)) * 16)) : "memory");
          if (32 * q4 + rr < nrow_t && u * 8 < D) *reinterpret_cast<uint4*>(dst + u * 8) = x;
        }
        if (valid && pa.lse != nullptr)
          pa.lse[(long long)(sq.q0 + tok) * H + h] = lim == 0 ? -INFINITY : (m * c2 + log2f(l)) * 0.6931471805599453f;
        uint32_t again = __ballot_sync(0xffffffffu, valid && !fine);
        while (again != 0) {
          const int w = __ffs(again) - 1;
          again &= again - 1;
          const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
          const int limw = __shfl_sync(0xffffffffu, lim, w);
          float o[4], mw, lw;
          exact_row((const __nv_bfloat16*)pa.q + (long long)(sq.q0 + tw) * pa.qs + (long long)hw * D,
                    (const __nv_bfloat16*)pa.k + (long long)sq.k0 * pa.ks + (long long)hk * D,
                    (const __nv_bfloat16*)pa.v + (long long)sq.k0 * pa.vs + (long long)hk * D,
                    [&](int j, long long& ko, long long& vo) {
                      ko = (long long)j * pa.ks;
                      vo = (long long)j * pa.vs;
                    },
                    D, limw, c2, o, mw, lw);
          const float iw = lw == 0.f ? 0.f : 1.0f / lw;
          __nv_bfloat16* dw = (__nv_bfloat16*)pa.out + (long long)(sq.q0 + tw) * pa.os + (long long)hw * D;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (lane * 4 + e < D) dw[lane * 4 + e] = __float2bfloat16_rn(o[e] * iw);
        }
      }
    }
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool encode3(EncodeTiledFn enc, CUtensorMap* m, const void* p, int D, int Hkv, int T, long long stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)T};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, BK};
  return encode_tmap(enc, m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, str, box);
}

template <int DP, bool SHARED>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PromptArgs& pa, const SharedArgs& sa, dim3 grid,
                   int n_slots, cudaStream_t s) {
  static std::atomic<int> done{0};
  auto kern = attn_tc_kernel<DP, SHARED>;
  const cudaError_t e = allow_smem(kern, Cfg<DP>::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, dim3(kThreads), Cfg<DP>::kSmem, s, tk, tv, pa, sa, n_slots);
}

}  // namespace

cudaError_t launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap tk{}, tv{};
  if (!encode3(enc, &tk, a.k, a.D, a.Hkv, a.Tkv, a.ks) || !encode3(enc, &tv, a.v, a.D, a.Hkv, a.Tkv, a.vs))
    return cudaErrorInvalidValue;
  const int G = a.H / a.Hkv;
  const long long slots = prompt_tile_slots(a.Tq, a.n, G, 2 * TM);
  const SharedArgs none{};
  const dim3 grid((unsigned)(slots * a.Hkv));
  return a.D <= 64 ? launch<64, false>(tk, tv, a, none, grid, (int)slots, s)
                   : launch<128, false>(tk, tv, a, none, grid, (int)slots, s);
}

// One CTA an SM takes 256 rows of one key/value head, the keys split over the SMs; about a sixth of those (where splits
// can be had) are left to the own keys, which run beside. 64 sequences behind 32768 positions, own keys up to 2048:
// see launch_attn_decode_tc.
int attn_shared_splits(const DecodeArgs& a) {
  const long long units = (long long)a.c.Hkv * ((a.n * (long long)(a.H / a.c.Hkv) + 2 * TM - 1) / (2 * TM));
  const int blocks = (a.shared + BK - 1) / BK;
  long long splits = (device_sm_count() - device_sm_count() / 6) / units;
  splits = splits < 1 ? 1 : (splits > blocks ? blocks : splits);
  const int per = (blocks + (int)splits - 1) / (int)splits;
  return (blocks + per - 1) / per;  // no empty split
}

cudaError_t launch_attn_shared_tc(const DecodeArgs& a, const CacheMaps& m, int splits, float* part_o, float2* part_ml,
                                  cudaStream_t s) {
  SharedArgs sa;
  sa.d = a;
  sa.splits = splits;
  const int blocks = (a.shared + BK - 1) / BK;
  sa.per = (blocks + splits - 1) / splits * BK;
  sa.part_o = part_o;
  sa.part_ml = part_ml;
  const PromptArgs none{};
  const long long pairs = (a.n * (long long)(a.H / a.c.Hkv) + 2 * TM - 1) / (2 * TM);
  const dim3 grid((unsigned)a.c.Hkv, (unsigned)pairs, (unsigned)splits);
  return a.c.D <= 64 ? launch<64, true>(m.k128, m.v128, none, sa, grid, 0, s)
                     : launch<128, true>(m.k128, m.v128, none, sa, grid, 0, s);
}

}  // namespace moe

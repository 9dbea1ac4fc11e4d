// Decode attention over the paged cache (bf16, heads of up to 128 elements): one query token a sequence.
// Three launches: the shared prefix on the tensor cores (attn_tc.cu, all sequences' rows against each key block
// once), each sequence's own keys (here), and the join of the pieces, which also checks that the prefix is shared.
//
// Own keys are an HBM stream: every key and value is read once and meets the G rows of its head group, far
// too few to fill a 128-row tile. The products are m16n8k16 MMAs with the keys on the long side,
//   S^T = K Q^T (16 keys x 8 rows),   O^T += V^T P^T (16 elements x 8 rows),
// so that a group of up to 8 rows wastes nothing (rows on the 16 side took twice the MMAs and accumulator
// registers); groups of more than 8 rows take two n-tiles for each load of K and V.
//   work    a segment is (sequence, key/value head, group of 8 or 16 rows); its keys go in units of 64. All
//           segments' units laid end to end are cut into equal runs, one a CTA: lengths live on the device and
//           differ wildly, and equal runs keep every SM streaming whatever they are. A segment cut by a run's end
//           leaves pieces that the join adds up, in order. A segment's end costs about as much as kEnd units (the
//           warps meet, a piece is written, new rows are fetched), so each segment is laid out with that many
//           empty units in front: without them runs of short segments took twice as long as the rest.
//           Beside a shared part there are four runs for each SM, taken from a counter: the SMs that the shared
//           part leaves free start at once, the others as its CTAs end. (64 sequences of up to 2048 own positions
//           behind 32768: 114 us with two runs, 108 with four, 109 with six; a sixth of the SMs left free against
//           none: 108 against 111 us, and 8 sequences behind 8192: 22.7 against 27.6.)
//   warps   two load units by TMA into a ring (boxes never cross a page), running ahead over segment ends; eight
//           take 16 keys each, four to a unit, with their own running maximum, and meet only where a segment ends.
//           Loaders and the two groups of four take every other unit: one loader could issue a unit only every
//           1350 cycles (barrier, page number and four copies in sequence).
// Piece (segment s, run c) has number s + c: going along the units, s or c grows by one from piece to piece.
#include <cuda.h>

#include <algorithm>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kSlice = 2048;   // sequences a launch takes: their unit counts are scanned in shared memory
constexpr int kWarps = 8, kLoaders = 2, kThreads = 32 * (kWarps + kLoaders);
constexpr int kKeys = 16;      // keys of a warp
constexpr int kUnit = 4 * kKeys;
constexpr int kScan = 256;     // threads that scan the lengths
constexpr int kEnd = 2;        // units that a segment's end is worth
constexpr int kQueue = 2;      // runs that the loading warp may be ahead

template <int DP, int NT> struct Cfg {
  static constexpr int kHalf = DP * kUnit * 2;  // bytes of a unit's K (or V)
  // Even: the units of a stage then all belong to one group of warps, which sees every phase of its barrier. (With an
  // odd ring a group meets a stage every other phase, whose parity cannot tell "loaded" from "not yet".)
  static constexpr int kStages = DP == 64 ? 8 : 4;
  static_assert(kStages % 2 == 0, "a stage belongs to one group of consumer warps");
  static constexpr int kRows = 8 * NT;
  static constexpr int kLd = DP + 4;            // floats of a row in the merge buffer: no bank conflicts
};

template <int DP, int NT> __host__ __device__ constexpr size_t own_smem(int n) {
  using C = Cfg<DP, NT>;
  return 1024 + (size_t)C::kStages * 2 * C::kHalf + (size_t)kWarps * C::kRows * C::kLd * 4 + 2 * kWarps * C::kRows * 4 +
         16 * C::kStages + 16 * kQueue + 4 * kQueue + 16 + 4 * (size_t)(2 * n + 1) + 4 * kScan;
}
static_assert(own_smem<128, 1>(kSlice) <= 232448 && own_smem<128, 2>(kSlice) <= 232448 &&
              own_smem<64, 2>(kSlice) <= 232448, "shared memory");

struct OwnArgs {
  DecodeArgs d;
  float* o;        // [piece][rows][D]
  float2* ml;      // [piece][rows]
  int32_t* prefix; // [n + 1] units of one head group before sequence i (kEnd a segment included), then [n + 1] =
                   // units per CTA
  const float* sh_o;      // [(sequence, head)][splits][D]
  const float2* sh_ml;
  int splits;      // pieces of a row over the shared keys
  int* next_run;   // nullable: runs are taken from this counter (zero before the call; the join sets it back)
  int n_runs;      // runs that the units are cut into (at most); without the counter one a CTA
  int min_run;     // units of a run, at least
  int R;           // rows of a piece: min(G, 8 NT)
  int RG;          // row groups of a key/value head
};

// The transpose of an 8 x 8 matrix of 16-bit values, one row a group of four lanes.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// A walk over the units of a run. b counts from 0 over the kEnd empty units and the nb - kEnd with keys.
struct Cursor {
  int i, hr, b, nb;  // sequence, head group, unit, units of the sequence
};
// To the next unit with keys: returns how many units it is away.
__device__ __forceinline__ int advance(Cursor& c, const int* P, int n, int HR) {
  if (++c.b < c.nb) return 1;
  c.b = kEnd;
  if (++c.hr < HR) return 1 + kEnd;
  c.hr = 0;
  do {
    if (++c.i >= n) return 1 << 30;
    c.nb = P[c.i + 1] - P[c.i];
  } while (c.nb == 0);
  return 1 + kEnd;
}

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, 1)
decode_own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16,
                  const __grid_constant__ OwnArgs a) {
  using C = Cfg<DP, NT>;
  constexpr int KS = DP / 16;  // k-steps of the scores, d-tiles of the output
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  float* buf = reinterpret_cast<float*>(gbase + C::kStages * 2 * C::kHalf);  // [warps][rows][kLd]
  float* sm_m = buf + kWarps * C::kRows * C::kLd;  // [warps][rows]
  float* sm_l = sm_m + kWarps * C::kRows;          // [warps][rows]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm_l + kWarps * C::kRows);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * C::kStages + 2 * kQueue);
  volatile int* queue = abort_flag + 4;                    // [kQueue]
  int* P = const_cast<int*>(abort_flag + 4 + kQueue);      // [n + 1]
  int* lens = P + a.d.n + 1;                               // [n] (0: nothing to read)
  const int n = a.d.n, tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  int* sums = lens + n;                            // [kScan]
  const CacheView& c = a.d.c;
  const int G = a.d.H / c.Hkv, HR = c.Hkv * a.RG, D = c.D;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int FULL = 0, EMPTY = C::kStages, RFULL = 2 * C::kStages, REMPTY = RFULL + kQueue;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(bar(FULL + s), 1); mbar_init(bar(EMPTY + s), 4); }
    for (int s = 0; s < kQueue; ++s) { mbar_init(bar(RFULL + s), 1); mbar_init(bar(REMPTY + s), kWarps + 1); }
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // After the shared part's kernel this one need not wait for it: that kernel lets dependents start only once it has
  // itself waited for everything before it, and what it writes is read by the join alone (for which this grid waits
  // at its end). Alone, it waits here.
  if (a.d.shared == 0) griddep_wait();
  griddep_launch_dependents();
  const int taken = tid == 0 && a.next_run != nullptr ? *reinterpret_cast<volatile int*>(a.next_run) : 0;

  // ---- units of every sequence, scanned
  const int chunk = (n + kScan - 1) / kScan, i0 = min(n, tid * chunk), i1 = tid < kScan ? min(n, i0 + chunk) : i0;
  int mine = 0;
  for (int i = i0; i < i1; ++i) {
    const int s = a.d.slots[i];
    int len = 0;
    if (s >= 0 && s < c.n_slots) len = c.lens[s];
    const bool bad = s < 0 || s >= c.n_slots || len < 0 || (long long)len > ((long long)c.width << c.page_shift);
    if (bad) {
      if (blockIdx.x == 0) record_error(a.d.status, MOE_ERR_DEVICE_CHECK, a.d.first + i);
      len = 0;
    }
    const int nb = len > a.d.shared ? (len - a.d.shared + kUnit - 1) / kUnit + kEnd : 0;
    P[i + 1] = nb;
    lens[i] = len;
    mine += nb;
  }
  if (n <= 32) {  // one warp's scan
    if (warp == 0) {
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      if (lane < n) P[lane + 1] = incl;
      if (lane == 0) P[0] = 0;
    }
  } else {
    if (tid < kScan) sums[tid] = mine;
    __syncthreads();
    if (warp == 0) {
      int v[kScan / 32], t = 0;
#pragma unroll
      for (int j = 0; j < kScan / 32; ++j) {
        v[j] = t;
        t += sums[lane * (kScan / 32) + j];
      }
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
#pragma unroll
      for (int j = 0; j < kScan / 32; ++j) sums[lane * (kScan / 32) + j] = incl - t + v[j];
    }
    __syncthreads();
    int run = tid < kScan ? sums[tid] : 0;
    for (int i = i0; i < i1; ++i) {
      run += P[i + 1];
      P[i + 1] = run;
    }
    if (tid == 0) P[0] = 0;
  }
  if (tid == 0) abort_flag[1] = taken;
  __syncthreads();
  // All runs were taken (see below) when this CTA started: it leaves, as the join waits for it (8 sequences behind
  // 8192 positions: 20.9 -> 18.7 us in a graph). The first CTA stays to write the prefix.
  if (a.next_run != nullptr && abort_flag[1] >= a.n_runs && blockIdx.x > 0) {
    griddep_wait();
    return;
  }
  const long long total = (long long)P[n] * HR;
  const int per = max((int)((total + a.n_runs - 1) / a.n_runs), a.min_run);
  auto past = [&](int run) { return run >= a.n_runs || (long long)run * per >= total; };  // no such run
  if (blockIdx.x == 0) {
    for (int i = tid; i <= n; i += kThreads) a.prefix[i] = P[i];
    if (tid == 0) a.prefix[n + 1] = per;
  }
  // Where a run begins; returns the units from there to its end, empty ones included (0 or less: nothing to do).
  auto start_run = [&](int run, Cursor& cu) {
    const long long begin = (long long)run * per, end = min(total, begin + per);
    if (end <= begin) return 0;
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
    int count = (int)(end - begin);
    if (cu.b < kEnd) {  // the run starts among a segment's empty units
      count -= kEnd - cu.b;
      cu.b = kEnd;
    }
    return count;
  };
  Cursor cu{0, 0, 0, 0};

  if (warp >= kWarps) {
    if (lane == 0) {
      // -------------------------------------------------------------- loads: the first loader takes the runs
      const int loader = warp - kWarps;
      int stage = 0, slot = 0, len = 0, cur = -1, rq = 0, x = 0;
      uint32_t phase = 0, filled = 0, fill_phase = 0, rphase = 0;
      const int box = min(c.page_size, kUnit);
      auto take = [&]() { return a.next_run != nullptr ? atomicAdd(a.next_run, 1) : a.n_runs; };
      int run = 0, next = 0;
      if (loader == 0) next = a.next_run != nullptr ? take() : (int)blockIdx.x;
      bool ok = true;
      while (ok) {
        if (loader == 0) {
          // the run's number to the other warps (one past the last ends them), and the next one asked for
          run = next;
          if (!wait_or_abort(bar(REMPTY + rq), rphase ^ 1u, a.d.timeout_ns, abort_flag, a.d.status, 63)) break;
          queue[rq] = run;
          mbar_arrive(bar(RFULL + rq));
          if (!past(run)) next = take();
        } else {
          if (!wait_or_abort(bar(RFULL + rq), rphase, a.d.timeout_ns, abort_flag, a.d.status, 63)) break;
          run = queue[rq];
          mbar_arrive(bar(REMPTY + rq));
        }
        if (++rq == kQueue) { rq = 0; rphase ^= 1u; }
        if (past(run)) {
          // tells CTAs that have not started yet; far from overflow, as each adds it once
          if (loader == 0 && a.next_run != nullptr) atomicAdd(a.next_run, a.n_runs);
          break;
        }
        for (int left = start_run(run, cu); left > 0; left -= advance(cu, P, n, HR), ++x) {
          if ((x & 1) == loader) {
            if (cu.i != cur) {
              cur = cu.i;
              slot = a.d.slots[cur];
              len = lens[cur];
            }
            const int key = a.d.shared + (cu.b - kEnd) * kUnit, rows = min(kUnit, (len - key + kKeys - 1) & ~(kKeys - 1));
            const int32_t* row_pages = c.table + (long long)slot * c.width;
            int page = row_pages[key >> c.page_shift];  // on its way during the wait
            if (!wait_or_abort(bar(EMPTY + stage), phase ^ 1u, a.d.timeout_ns, abort_flag, a.d.status, 62)) {
              ok = false;
              break;
            }
            const uint32_t dst = base + stage * 2 * C::kHalf, b = bar(FULL + stage);
            mbar_arrive_expect_tx(b, 2u * (uint32_t)(rows * DP * 2));
            for (int r = 0; r < rows;) {
              const int nr = rows - r >= box ? box : kKeys;  // whole boxes, then 16 rows at a time
              if (r > 0) page = row_pages[(key + r) >> c.page_shift];
              if (page < 0 || page >= c.n_pages) {
                record_error(a.d.status, MOE_ERR_DEVICE_CHECK, a.d.first + cur);
                page = 0;
              }
              const int row = (page * c.Hkv + cu.hr / a.RG) * c.page_size + ((key + r) & (c.page_size - 1));
              const CUtensorMap *mk = nr == box ? &tmK : &tmK16, *mv = nr == box ? &tmV : &tmV16;
#pragma unroll
              for (int h = 0; h < DP / 64; ++h) {
                tma_load_3d(dst + h * (kUnit * 128) + r * 128, mk, 64 * h, row, a.d.layer, b);
                tma_load_3d(dst + C::kHalf + h * (kUnit * 128) + r * 128, mv, 64 * h, row, a.d.layer, b);
              }
              r += nr;
            }
            filled |= 1u << stage;
            fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // copies in flight land before shared memory goes away
      for (int s = 0; s < C::kStages; ++s)
        if (filled & (1u << s)) mbar_wait_bounded(bar(FULL + s), (fill_phase >> s) & 1u, a.d.timeout_ns);
    }
    // The idle lanes stay here: one that went ahead into the wait for the shared part's grid below would hold up the
    // lane that loads.
    __syncwarp();
  } else {
    const float c2 = a.d.scale * 1.4426950408889634f, thr = rescale_above(c2);
    const int g = lane >> 2, t4 = lane & 3, quarter = warp & 3, group = warp >> 2;
    const int mi = lane >> 3, l8 = lane & 7;
    uint32_t q[KS][NT][2], qn[KS][NT][2];
    float o[KS][NT][4], m[NT][2], l[NT][2];
    int len = 0, len_n = 0;
    int stage = 0, x = 0;
    uint32_t phase = 0;
    bool ok = true;
    // the rows of the segment at `at`, as B fragments
    auto fetch = [&](const Cursor& at) {
      len_n = lens[at.i];
      const int hk = at.hr / a.RG, r0 = (at.hr % a.RG) * C::kRows, nr = min(a.R, G - r0);
      const __nv_bfloat16* qp = (const __nv_bfloat16*)a.d.q + (long long)at.i * a.d.qs + (long long)(hk * G + r0) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * t + g, col = 16 * k + 2 * t4 + 8 * e;
            qn[k][t][e] = row < nr && col < D ? *reinterpret_cast<const uint32_t*>(qp + row * D + col) : 0u;
          }
    };
    // A run's first unit goes to the group whose turn it is, which depends on the runs that the CTA had before: `flip`
    // says whether that is the second one. Parts are added up with the first unit's group first, so that the sums do not
    // depend on which CTA takes a run.
    int flip = 0;
    int rq = 0, run = 0, run_no = 0;
    uint32_t rphase = 0;
    // the next run with anything in it, at cu; false after the last
    auto next_run = [&]() {
      for (run = 0; run <= 0;) {
        if (!warp_wait(bar(RFULL + rq), rphase, a.d.timeout_ns, abort_flag, a.d.status, 64)) return false;
        run_no = queue[rq];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(REMPTY + rq));
        if (++rq == kQueue) { rq = 0; rphase ^= 1u; }
        if (past(run_no)) return false;
        run = start_run(run_no, cu);
      }
      return true;
    };
    bool fresh = true, more = next_run();
    if (more) fetch(cu);
    for (; more; ++x) {
      if (fresh) {
        fresh = false;
        len = len_n;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              q[k][t][e] = qn[k][t][e];
              o[k][t][2 * e] = o[k][t][2 * e + 1] = 0.f;
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          m[t][0] = m[t][1] = -INFINITY;
          l[t][0] = l[t][1] = 0.f;
        }
      }
      if ((x & 1) == group) {
        if (ok) ok = warp_wait(bar(FULL + stage), phase, a.d.timeout_ns, abort_flag, a.d.status, 61);
        const int left = len - (a.d.shared + (cu.b - kEnd) * kUnit + quarter * kKeys);  // keys of this warp's 16
        if (ok && left > 0) {
          const uint32_t sk = base + stage * 2 * C::kHalf + quarter * (kKeys * 128), sv = sk + C::kHalf;
          if (left < kKeys) {  // positions past the end hold anything: zero their values
            for (int z = lane; z < (kKeys - left) * (DP / 8); z += 32) {
              const int rr = left + z / (DP / 8), u = z % (DP / 8);
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sv + (u >> 3) * (kUnit * 128) + rr * 128 + (u & 7) * 16), "r"(0)
                           : "memory");
            }
            __syncwarp();
          }
          float s[NT][4], odd[NT][4];  // even and odd k-steps: two chains of dependent MMAs instead of one
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = odd[t][e] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int row = (mi & 1) * 8 + l8, u = 2 * k + (mi >> 1);
            uint32_t f[4];
            ldsm4(sk + (u >> 3) * (kUnit * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(k & 1 ? odd[t] : s[t], f, q[k][t][0], q[k][t][1]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] += odd[t][e];
          if (left < kKeys)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (g + 8 * (e >> 1) >= left) s[t][e] = -INFINITY;
          // the maxima are only reduced, and O rescaled, when one rises by more than 2^8 (as in attn_tc.cu)
          bool rise = false;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            rise = rise || fmaxf(s[t][0], s[t][2]) > m[t][0] + thr || fmaxf(s[t][1], s[t][3]) > m[t][1] + thr;
          if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(s[t][r], s[t][2 + r]), -INFINITY);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                if (mx > m[t][r] + thr) {
                  const float al = ex2((m[t][r] - mx) * c2);
                  l[t][r] *= al;
#pragma unroll
                  for (int k = 0; k < KS; ++k) { o[k][t][r] *= al; o[k][t][2 + r] *= al; }
                  m[t][r] = mx;
                }
              }
          }
          uint32_t p[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float mc0 = m[t][0] == -INFINITY ? 0.f : m[t][0] * c2, mc1 = m[t][1] == -INFINITY ? 0.f : m[t][1] * c2;
            const float p0 = ex2(fmaf(s[t][0], c2, -mc0)), p1 = ex2(fmaf(s[t][1], c2, -mc1));
            const float p2 = ex2(fmaf(s[t][2], c2, -mc0)), p3 = ex2(fmaf(s[t][3], c2, -mc1));
            l[t][0] += p0 + p2;
            l[t][1] += p1 + p3;
            p[t][0] = movm_t(pack_bf16x2(p0, p1));
            p[t][1] = movm_t(pack_bf16x2(p2, p3));
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int row = (mi >> 1) * 8 + l8, u = 2 * k + (mi & 1);
            uint32_t f[4];
            ldsm4t(sv + (u >> 3) * (kUnit * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(o[k][t], f, p[t][0], p[t][1]);
          }
          if (left < kKeys) fence_proxy_async_smem();  // the zeros above before the next copy into this stage
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(EMPTY + stage));
      }
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }

      const Cursor was = cu;
      const int was_run = run_no;
      const int part = quarter + 4 * (group ^ flip);  // this warp's place among the eight parts
      run -= advance(cu, P, n, HR);
      if (run > 0 && cu.i == was.i && cu.hr == was.hr) continue;
      // ---- the segment (or the run) ends: the eight warps' parts become one piece, while the next rows are on their way
      fresh = true;
      if (run <= 0) {
        more = next_run();
        flip = (x + 1) & 1;
      }
      if (more) fetch(cu);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], w);
          if (g == 0) {
            sm_m[part * C::kRows + 8 * t + 2 * t4 + r] = m[t][r];
            sm_l[part * C::kRows + 8 * t + 2 * t4 + r] = l[t][r];
          }
        }
      consumers_sync();
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 8 * t + 2 * t4 + r;
          float M = -INFINITY;
#pragma unroll
          for (int y = 0; y < kWarps; ++y) M = fmaxf(M, sm_m[y * C::kRows + row]);
          const float w = M == -INFINITY ? 0.f : ex2((m[t][r] - M) * c2);
          float* d = buf + (part * C::kRows + row) * C::kLd + g;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            d[16 * k] = o[k][t][r] * w;
            d[16 * k + 8] = o[k][t][2 + r] * w;
          }
        }
      consumers_sync();
      const int nr = min(a.R, G - (was.hr % a.RG) * C::kRows);
      const long long piece = (long long)was.i * HR + was.hr + was_run;
      for (int z = tid; z < nr * (D / 4); z += 32 * kWarps) {
        const int row = z / (D / 4), col = (z % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
          const float4 u = *reinterpret_cast<const float4*>(buf + (y * C::kRows + row) * C::kLd + col);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        *reinterpret_cast<float4*>(a.o + (piece * a.R + row) * D + col) = v;
      }
      if (tid < nr) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int y = 0; y < kWarps; ++y) M = fmaxf(M, sm_m[y * C::kRows + tid]);
#pragma unroll
        for (int y = 0; y < kWarps; ++y)
          if (M != -INFINITY) L += sm_l[y * C::kRows + tid] * ex2((sm_m[y * C::kRows + tid] - M) * c2);
        a.ml[piece * a.R + tid] = make_float2(M * c2, L);
      }
      consumers_sync();
    }
  }
  if (a.d.shared > 0) griddep_wait();
}

// A (sequence, head)'s pieces over the shared keys, then over its own, by WPR warps that take every WPR-th piece and
// add up in a fixed order: 4 while there are few rows, 1 (four rows a CTA) when the rows alone fill the GPU.
template <int WPR>
__global__ void __launch_bounds__(128)
decode_join_kernel(const __grid_constant__ OwnArgs a) {
  __shared__ float4 part[WPR == 1 ? 1 : WPR][32];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WPR;
  const CacheView& c = a.d.c;
  const int H = a.d.H, G = H / c.Hkv, HR = c.Hkv * a.RG, D = c.D;
  const int row = blockIdx.x * (4 / WPR) + (threadIdx.x >> 5) / WPR;
  const int i = row / H, h = row % H, hk = h / G, hg = h % G;
  // While the pieces are being computed: that the sequences share what the call says, a stretch of the pages for each
  // head. (The own positions' kernel lets this one start once everything before the call is done. In the shared
  // positions' kernel the check took registers from its loops: 64 sequences behind 32768 positions 109.2 -> 110.5 us.)
  if (a.d.shared > 0 && i < a.d.n) check_shared(a.d, i, h * 32 * WPR + threadIdx.x % (32 * WPR), H * 32 * WPR);
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.next_run != nullptr) *a.next_run = 0;
  if (i >= a.d.n) return;  // (with WPR = 4 there is a CTA a row)
  const int hr = hk * a.RG + hg / a.R, r = hg % a.R;
  const int s = a.d.slots[i], b0 = a.prefix[i], b1 = a.prefix[i + 1], per = a.prefix[a.d.n + 1];
  const bool valid = s >= 0 && s < c.n_slots;
  const int b = b1 - b0, shared = valid ? a.splits : 0;
  int own = 0;
  long long p0 = 0;
  if (valid && b > 0) {
    const long long start = (long long)b0 * HR + (long long)hr * b + kEnd, last = start + (b - kEnd) - 1;
    int c0, c1;
    if (last < (1ll << 31)) { c0 = (int)start / per; c1 = (int)last / per; }
    else { c0 = (int)(start / per); c1 = (int)(last / per); }
    own = c1 - c0 + 1;
    p0 = (long long)i * HR + hr + c0;
  }
  const int count = shared + own;
  auto ml = [&](int x) { return x < shared ? a.sh_ml[(long long)row * a.splits + x] : a.ml[(p0 + x - shared) * a.R + r]; };
  auto src = [&](int x) {
    return reinterpret_cast<const float4*>(x < shared ? a.sh_o + ((long long)row * a.splits + x) * D
                                                      : a.o + ((p0 + x - shared) * a.R + r) * D) + lane;
  };
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f, M = -INFINITY;
  const bool on = lane * 4 < D;
  if (count <= 32) {  // the usual case: one lane a piece, the weights computed once, the values on their way meanwhile
    const float2 v = lane < count ? ml(lane) : make_float2(-INFINITY, 0.f);
    float4 u[8];
#pragma unroll
    for (int y = 0; y < 8; ++y)
      u[y] = warp + WPR * y < count && on ? *src(warp + WPR * y) : make_float4(0.f, 0.f, 0.f, 0.f);
    M = fmaxf(v.x, -INFINITY);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    const float wv = ex2(v.x - (M == -INFINITY ? 0.f : M));
    l = wv * v.y;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    for (int y0 = 0; y0 * WPR < 32; y0 += 8) {
      if (y0 > 0) {
        if (warp + WPR * y0 >= count) break;
#pragma unroll
        for (int y = 0; y < 8; ++y)
          u[y] = warp + WPR * (y0 + y) < count && on ? *src(warp + WPR * (y0 + y)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = __shfl_sync(0xffffffffu, wv, (warp + WPR * (y0 + y)) & 31);
        o.x = fmaf(w, u[y].x, o.x);
        o.y = fmaf(w, u[y].y, o.y);
        o.z = fmaf(w, u[y].z, o.z);
        o.w = fmaf(w, u[y].w, o.w);
      }
    }
  } else {
    for (int x = lane; x < count; x += 32) M = fmaxf(M, ml(x).x);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    const float ref = M == -INFINITY ? 0.f : M;
    for (int x = lane; x < count; x += 32) {
      const float2 v = ml(x);
      l += ex2(v.x - ref) * v.y;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
#pragma unroll 4
    for (int x = warp; x < count; x += WPR) {
      const float w = ex2(ml(x).x - ref);
      if (on) {
        const float4 u = *src(x);
        o.x = fmaf(w, u.x, o.x);
        o.y = fmaf(w, u.y, o.y);
        o.z = fmaf(w, u.z, o.z);
        o.w = fmaf(w, u.w, o.w);
      }
    }
  }
  if (WPR > 1) {
    part[warp % WPR][lane] = o;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int y = 1; y < WPR; ++y) {
      const float4 u = part[y][lane];
      o.x += u.x; o.y += u.y; o.z += u.z; o.w += u.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (on) {
    uint2 u;
    u.x = pack_bf16x2(o.x * inv, o.y * inv);
    u.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.d.out + (long long)i * a.d.os + (long long)h * D + lane * 4) = u;
  }
  if (a.d.lse != nullptr && lane == 0) a.d.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <int DP, int NT>
cudaError_t launch_own(const CacheMaps& m, const OwnArgs& o, int ctas, cudaStream_t s) {
  static std::atomic<int> done{0};
  auto kern = decode_own_kernel<DP, NT>;
  const cudaError_t e = allow_smem(kern, own_smem<DP, NT>(kSlice), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kThreads), own_smem<DP, NT>(o.d.n), s, m.k64, m.v64, m.k16, m.v16, o);
}

}  // namespace

bool encode_cache_maps(const CacheView& c, CacheMaps* m) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t rows = (cuuint64_t)c.n_pages * c.Hkv * c.page_size;
  const cuuint64_t dims[3] = {(cuuint64_t)c.D, rows, (cuuint64_t)c.n_layers};
  const cuuint64_t str[2] = {(cuuint64_t)c.D * 2, rows * c.D * 2};
  auto one = [&](CUtensorMap* t, const void* p, int most) {
    const cuuint32_t box[3] = {64, (cuuint32_t)(c.page_size < most ? c.page_size : most), 1};
    return encode_tmap(enc, t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, str, box);
  };
  return one(&m->k16, c.k, kKeys) && one(&m->v16, c.v, kKeys) && one(&m->k64, c.k, kUnit) && one(&m->v64, c.v, kUnit) &&
         one(&m->k128, c.k, 128) && one(&m->v128, c.v, 128);
}

cudaError_t launch_attn_decode_tc(const DecodeArgs& all, const CacheMaps& m, cudaStream_t s) {
  const int G = all.H / all.c.Hkv, NT = G <= 8 ? 1 : 2, RG = (G + 8 * NT - 1) / (8 * NT), HR = all.c.Hkv * RG;
  const int R = G < 8 * NT ? G : 8 * NT, D = all.c.D;
  const int ctas = device_sm_count();
  // A slice's units are counted in 32 bits, and its shared part's row pairs are a grid's y.
  const long long longest = (long long)all.c.width * all.c.page_size;
  const long long fit = std::min((1ll << 36) / longest, 65535ll * 256 / G);
  const int slice = (int)std::max(1ll, std::min((long long)kSlice, fit));
  for (int first = 0; first < all.n; first += slice) {
    DecodeArgs d = all;
    d.n = std::min(slice, all.n - first);
    d.q = (const __nv_bfloat16*)all.q + (long long)first * all.qs;
    d.out = (__nv_bfloat16*)all.out + (long long)first * all.os;
    d.slots = all.slots + first;
    if (all.lse != nullptr) d.lse = all.lse + (long long)first * all.H;
    OwnArgs o;
    d.first = first;
    o.d = d;
    o.splits = 0;
    o.R = R;
    o.RG = RG;
    o.next_run = d.shared > 0 ? d.status + 6 : nullptr;
    o.n_runs = d.shared > 0 ? 4 * ctas : ctas;
    o.min_run = d.shared > 0 ? 6 : 1;
    // pieces: own ones [(n HR + runs)][R], then the shared ones [n H][splits]; see decode_pieces
    const long long own_rows = ((long long)d.n * HR + o.n_runs) * R;
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
    if (d.shared > 0) e = launch_attn_shared_tc(d, m, o.splits, sh, const_cast<float2*>(o.sh_ml), s);
    if (e == cudaSuccess) {
      if (D <= 64) e = NT == 1 ? launch_own<64, 1>(m, o, ctas, s) : launch_own<64, 2>(m, o, ctas, s);
      else e = NT == 1 ? launch_own<128, 1>(m, o, ctas, s) : launch_own<128, 2>(m, o, ctas, s);
    }
    const int rows = d.n * d.H;
    if (e == cudaSuccess)
      e = rows <= 8 * ctas ? launch_pdl(decode_join_kernel<4>, dim3((unsigned)rows), dim3(128), 0, s, o)
                           : launch_pdl(decode_join_kernel<1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, o);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe

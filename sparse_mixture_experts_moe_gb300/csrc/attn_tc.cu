// Attention on the 5th-generation tensor cores (bf16, heads of up to 128 elements): packed prompts, and the
// shared prefix of a decode batch.
//   S = Q K^T (scores), P = 2^(c S - c m) (weights, c = scale log2 e), O += P V, out = O / l
// with m a running reference of each row and l the sum of its weights, in one pass over the keys: no score
// ever leaves the SM.
//
// An item is 256 packed rows (two tiles of 128) of one key/value head; the tiles share every key/value block (128
// keys), which halves the reads of L2 against one tile an item. One CTA an SM takes items from a counter, the
// longest rows of a sequence first, and its warps walk the items one behind the other:
//   warps 0..3, 4..7  softmax of tile 0 / 1: thread = row = TMEM lane. Reads S, takes the maximum, writes P
//                     (bf16) over S's own columns, sums the weights; at the end divides and stores the rows
//   warp 8            allocates TMEM; one elected thread issues every MMA: QK with both operands in shared memory, PV
//                     with P read from TMEM as the A operand
//   warp 9            finds the items, one ahead, and loads K and V blocks by TMA into a ring (K0 V0 K1 V1 ...)
//   warps 10, 11      load the Q tiles of the next item as soon as the last QK of this one is done
// so an item's first loads, its search and its first scores overlap the end of the item before. (With a CTA for each
// item these cost 9 us an item, as much as six blocks of keys.)
// TMEM (512 columns): S0 S1 (128 fp32 columns each, P in the first 64), O0 O1.
// The MMAs go PV0(j) QK0(j+1) PV1(j) QK1(j+1): while one tile is in softmax the tensor cores work on the
// other. QK(j+1) may overwrite P(j) because MMAs of one thread run in issue order.
// O is only rescaled when a row's maximum rises by more than 8 in log2 units above the reference m (rescale_above;
// weights then stay below 2^8, exact enough for bf16 as only their relative precision counts); the softmax
// warp that sees it waits for the last PV and scales the 32 rows of O itself. After the first blocks
// that is rare, so no warps are kept for it.
// A weight is rounded to bf16 (off by at most 2^-8 of it) because the MMA takes both operands in one type; its
// sum l takes the unrounded value.
// Keys past a row's limit get weight 0 by index. 0 times a non-finite value in V would still be NaN: the columns of a
// row that such a value can have touched are replaced (replace_unseen), so that a non-finite value reaches only rows
// that see it. That costs nothing where everything is finite.
// All waits are bounded, as in ffn_tc.cu, with time for rows that are replaced (replace_time).
// Measured: one prompt of 16384 tokens, 32 heads of 128 on 8: 1.24 ms in a run of ten (1.77 PFLOP/s, 93% of the matrix
// rate measured in a burst), 1.37 ms in a loop of seconds (1.61, 93% of the sustained rate). Heads of 64: 1.00 ms,
// 1.10 PFLOP/s, bound by the powers of two: 256 warp instructions of 8 cycles a scheduler and block of a tile pair are
// 2048 of some 2200 cycles (scores computed one block ahead, so that no softmax waits for an MMA, gained nothing).
// 13 ragged prompts, 8192 tokens together, heads of 128: 104 us; the masked block of a row, its epilogue and the first
// scores cost about 3.5 us an item (taking the longest sequences first gains 1 us).
#include <cuda.h>

#include <type_traits>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int BK = 128;       // keys per block
constexpr int TM = 128;       // rows per tile
// Registers: 12 warps of 168 at launch (64512); the softmax warps take 232 each (a row of 128 scores stays in
// registers), the other four keep 40: 8 * 32 * 232 + 4 * 32 * 40 = 64512.
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kMaxSmem = 232448;

struct __align__(16) Item {
  int hk, row0, nrows;      // key/value head; packed rows row0 .. of the sequence (or batch)
  int q0, nq, k0, nk;       // the sequence
  int key0, n_keys;         // keys of the item
  int lim0, lim1;           // keys that each tile's last row sees (relative to key0)
  int last;                 // no item: the end
  int seq;                  // (of a chunk, for errors)
  int dual;                 // (of a chunk) one tile of rows: both softmax groups take it, with half of each block's keys
  int split;                // which part of the keys; of a chunk: the piece that takes the results (-1: the output)
};
constexpr int kItems = 3;   // items published: one worked on, one ahead, one being given back
constexpr int kItemReaders = 1 + 8 + 2;

template <int DP> struct Cfg {
  static constexpr int kChunks = DP / 64;          // 64-element (128-byte) swizzle columns of a row
  static constexpr int kTileBytes = TM * DP * 2;   // a Q tile, and a K or V block
  static constexpr int kStages = DP == 128 ? 4 : 8;
  static constexpr int kStage = 32 * 128;  // bytes of a softmax warp's output staging: 32 rows x 64 bf16 elements
  static constexpr int kBars = 2 * kStages + 7 * 2 + 1 + 2 * kItems + 1 + 8;
  static constexpr size_t kSmem =
      1024 + (size_t)(2 + kStages) * kTileBytes + 8 * kStage + 8 * kBars + 16 + (kItems + 1) * sizeof(Item) + 4 * 32 * 8;
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
// A TMA copy with an L2 eviction priority (a policy from createpolicy).
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(dst), "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_policy(bool first) {
  uint64_t a, b;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(a));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(b));
  return first ? a : b;
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

struct SharedArgs {
  DecodeArgs d;
  int per;        // keys of a split, a multiple of BK (decode)
  int splits;     // pieces of a row
  float* part_o;  // [piece][D]
  float2* part_ml;
  ChunkRun* runs;  // of a chunk call, one a CTA
  int piece_rows;  // and the rows of a piece
};

// ------------------------------------------------------------------ chunks over the paged cache
// How a chunk call is shared out. An item is, as for prompts, 256 packed rows of one key/value head; the items lie in a
// row (heads outside, tile slots inside), each as long as its cost: kBlock a block of keys, and kItem for Q, the first scores
// and the results. The row is cut into equally long runs, one a CTA, whatever items the
// cuts fall into: a decoding sequence of 100,000 keys beside a hundred short ones then takes as many CTAs as it needs.
// A block belongs to the run that its beginning lies in. An item inside one run goes to the output; of one that
// several runs share, each puts its part (a piece) into the workspace, and chunk_join_kernel adds them up in order. A
// run has at most two such items, its first and its last, so that 2 pieces a CTA are enough however long the keys.
constexpr int kBlock = 4, kItem = 16, kShortest = 16;

// Length of an item of so many keys.
__device__ __forceinline__ long long chunk_length(int keys) { return kItem + (long long)((keys + BK - 1) / BK) * kBlock; }
struct ChunkItem {
  int seq, row0, nrows, q0, nq, nk, slot;
  int lim0, lim1, n_blocks;
  __device__ __forceinline__ long long length() const { return nrows > 0 ? kItem + (long long)n_blocks * kBlock : 0; }
};
// What fills tile slot s (nrows = 0: nothing).
__device__ __forceinline__ ChunkItem chunk_item(const PromptArgs& pa, const SharedArgs& sa, int s, int i) {
  const int G = pa.H / pa.Hkv;
  ChunkItem it{};
  it.seq = i;
  const int q0 = pa.qo[i], q1 = pa.qo[i + 1];
  it.slot = sa.d.slots[i];
  if (q0 < 0 || q1 < q0 || q1 > pa.Tq) {
    record_error(pa.status, MOE_ERR_DEVICE_CHECK, i);
    return it;
  }
  it.q0 = q0;
  it.nq = q1 - q0;
  const long long r0 = ((long long)s - ((long long)q0 * G / (2 * TM) + i)) * (2 * TM);
  if (r0 < 0 || r0 >= (long long)it.nq * G) return it;
  it.nk = slot_len(sa.d.c, it.slot);
  if (it.nk == 0 && (it.slot < 0 || it.slot >= sa.d.c.n_slots || sa.d.c.lens[it.slot] != 0))
    record_error(pa.status, MOE_ERR_DEVICE_CHECK, i);
  it.row0 = (int)r0;
  it.nrows = min(2 * TM, it.nq * G - it.row0);
  it.lim0 = visible_keys((it.row0 + min(it.nrows, TM) - 1) / G, it.nq, it.nk, pa.causal);
  it.lim1 = it.nrows > TM ? visible_keys((it.row0 + it.nrows - 1) / G, it.nq, it.nk, pa.causal) : 0;
  it.n_blocks = (max(it.lim0, it.lim1) + BK - 1) / BK;
  return it;
}
// The runs: how many, their beginnings, and the run that place x lies in.
struct Runs {
  long long all;
  int n;
  __device__ __forceinline__ Runs(long long total, int ctas) : all(total) {
    const long long most = total / kShortest;
    n = (int)(most < 1 ? 1 : (most < ctas ? most : ctas));
  }
  __device__ __forceinline__ long long begin(int c) const { return all * c / n; }
  __device__ __forceinline__ int of(long long x) const { return (int)(((x + 1) * n - 1) / all); }
};

// SHARED = false: items are tile-pair slots (descending, so that the longest rows of a sequence start first) x
// key/value heads, n_items of them. SHARED = true: one item a CTA, blockIdx = (key/value head, row pair, split of
// the shared keys); rows are (sequence, head) pairs, and each row's piece goes to the workspace unnormalised. SPLIT
// (prompts of few rows): every item's keys in sa.splits parts, an item each, and the rows' pieces likewise. PAGED: the
// keys are a cache's, and each CTA takes a run of the items (above), n_items the number of tile slots.
template <int DP, bool SHARED, bool SPLIT, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptArgs pa,
               const __grid_constant__ SharedArgs sa, int n_items, int q_tma) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base, sKV = base + 2 * C::kTileBytes;
  const uint32_t sOut = sKV + C::kStages * C::kTileBytes;  // [softmax warp][32 rows][64]
  Item* items = reinterpret_cast<Item*>(gbase + (2 + C::kStages) * C::kTileBytes + 8 * C::kStage);  // [kItems]
  Item* late_item = items + kItems;  // (of a chunk)
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kItems + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int FULL = 0, EMPTY = C::kStages, QFULL = 2 * C::kStages, SFULL = QFULL + 2, PFULL = SFULL + 4,
                ODONE = PFULL + 4, QEMPTY = ODONE + 2, DONE = QEMPTY + 2, IFULL = DONE + 1, IEMPTY = IFULL + kItems,
                TAIL = IEMPTY + kItems, GIVEN = TAIL + 1, TAKEN = GIVEN + 4;
  float2* given_ml = reinterpret_cast<float2*>(gbase + C::kSmem - 1024 - 4 * 32 * 8);  // [warp of tile 1][row]

  // (the shuffle tells the compiler that the warp number is the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(bar(FULL + s), 1); mbar_init(bar(EMPTY + s), 1); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(QFULL + t), 1);
      for (int b = 0; b < 4; b += 2) {  // (the second of each is for halves of blocks)
        mbar_init(bar(SFULL + b + t), 1);
        mbar_init(bar(PFULL + b + t), 4);
      }
      mbar_init(bar(ODONE + t), 1);
      mbar_init(bar(QEMPTY + t), 1);
    }
    for (int i = 0; i < kItems; ++i) { mbar_init(bar(IFULL + i), 1); mbar_init(bar(IEMPTY + i), kItemReaders); }
    mbar_init(bar(DONE), 1);
    mbar_init(bar(TAIL), 1);
    for (int i = 0; i < 8; ++i) mbar_init(bar(GIVEN + i), 1);
    fence_mbar_init();
    *abort_flag = 0;
    if (q_tma) tma_prefetch_desc(&tmQ);
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
  // Only after TMEM is allocated: a dependent kernel that starts on this SM may allocate some before it waits for
  // this grid. And only after the wait: the decode's own-key kernel relies on everything before this grid being done.
  griddep_launch_dependents();

  const int H = SHARED ? sa.d.H : pa.H, Hkv = SHARED ? sa.d.c.Hkv : pa.Hkv, D = SHARED ? sa.d.c.D : pa.D;
  const int G = H / Hkv;
  int* status = SHARED ? sa.d.status : pa.status;
  const uint64_t timeout_ns = SHARED ? sa.d.timeout_ns : pa.timeout_ns;
  // The items, for every warp but the one that finds them: the next one (nullptr after the last), and giving it
  // back. The fields are read where they are needed, as the softmax warps have no registers to keep them in.
  int iq = 0;
  uint32_t iphase = 0;
  auto next_item = [&]() -> const Item* {
    if (!warp_wait(bar(IFULL + iq), iphase, timeout_ns, abort_flag, status, 54)) return nullptr;
    return items[iq].last ? nullptr : items + iq;
  };
  auto item_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(IEMPTY + iq));
    if (++iq == kItems) { iq = 0; iphase ^= 1u; }
  };
  auto blocks = [](int keys) { return (keys + BK - 1) / BK; };

  // This CTA's run: a scan over the lengths of all tile slots, each thread with some of them in a row. The results stay
  // in the output staging until the first item is published.
  long long* plan = reinterpret_cast<long long*>(gbase + (2 + C::kStages) * C::kTileBytes);
  if (PAGED) {
    const int per = (n_items + kThreads - 1) / kThreads, s0 = min(n_items, tid * per), s1 = min(n_items, s0 + per);
    // f(slot, length) for the slots of [s0, s1) that a tile fills, as long as it returns true. The sequences lie in the slots'
    // order, so what is read of them is read ahead, four at a time.
    auto walk = [&](auto f) {
      int s = s0, i = find_tile_seq(pa.qo, pa.n, G, 2 * TM, s0);
      while (s < s1 && i < pa.n) {
        int q[5], len[4];
#pragma unroll
        for (int k = 0; k < 5; ++k) q[k] = pa.qo[min(i + k, pa.n)];
#pragma unroll
        for (int k = 0; k < 4; ++k) len[k] = slot_len(sa.d.c, sa.d.slots[min(i + k, pa.n - 1)]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i + k >= pa.n || q[k] < 0 || q[k + 1] < q[k] || q[k + 1] > pa.Tq) continue;
          const long long first = (long long)q[k] * G / (2 * TM) + i + k, rows = (long long)(q[k + 1] - q[k]) * G;
          const long long end = min((long long)s1, first + (rows + 2 * TM - 1) / (2 * TM));
          for (s = max(s, (int)min(first, (long long)s1)); s < end; ++s) {
            const int row0 = (int)(s - first) * 2 * TM, nrows = min(2 * TM, (int)rows - row0), nq = q[k + 1] - q[k];
            const int lim0 = visible_keys((row0 + min(nrows, TM) - 1) / G, nq, len[k], pa.causal);
            const int lim1 = nrows > TM ? visible_keys((row0 + nrows - 1) / G, nq, len[k], pa.causal) : 0;
            if (!f(s, chunk_length(max(lim0, lim1)))) return;
          }
        }
        i += 4;
      }
    };
    long long sum = 0;
    if (s0 < s1) walk([&](int, long long len) { sum += len; return true; });
    long long upto = sum;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += x;
    }
    if (lane == 31) plan[4 + warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) upto += total;
      total += plan[4 + w];
    }
    if (total > 0) {
      const Runs runs(total * pa.Hkv, gridDim.x);
      if ((int)blockIdx.x < runs.n) {
        const long long begin = runs.begin(blockIdx.x), at = begin % total;
        if (at >= upto - sum && at < upto) {  // one thread
          long long x = upto - sum;
          walk([&](int s, long long len) {
            plan[1] = s;
            plan[2] = begin - at + x;  // where item (head, slot s) begins
            x += len;
            return x <= at;
          });
          plan[3] = begin / total;  // the head
        }
      }
    }
    if (tid == 0) {
      plan[0] = total;
      ChunkRun none;
      none.nrows = 0;
      sa.runs[blockIdx.x] = none;
    }
    __syncthreads();
  }

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (PAGED && warp == kSoftWarps + 1) {
      // -------------------------------------------------------------- K and V of a chunk's items (warp 10 finds them)
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_phase = 0;
      // the pages of 32 x page_size positions from table column 32 `window` on and of the next ones, a page a lane
      int window_slot = -1, window = 0, page_now = 0, page_next = 0;
      bool tail = false;  // the last block of values loaded needs its end cleared
      int tail_stage = 0, tail_keys = 0, behind = 0;
      uint32_t tail_phase = 0;
      // What pages hold past a sequence's end is anyone's: the last block's values there become zeros once they
      // have arrived, as 0 times a leftover that is not finite would be NaN. This is done when the two copies behind them
      // are on their way: their stages wait for nothing that comes after the block before.
      auto clear_tail = [&]() {
        if (!tail) return true;
        if (!warp_wait(bar(TAIL), tail_phase, timeout_ns, abort_flag, status, 51)) return false;
        tail = false;
        tail_phase ^= 1u;
        const uint32_t dst = sKV + tail_stage * C::kTileBytes;
        for (int i = lane; i < (BK - tail_keys) * 8; i += 32)
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + c * (BK * 128) + tail_keys * 128 + i * 16), "r"(0)
                         : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL + tail_stage));
        return true;
      };
      const CacheView& cv = sa.d.c;
      const int box = min(cv.page_size, BK), box_shift = min(cv.page_shift, 7);
      const bool leader = elect_one();
      bool ok = true;
      while (ok) {
        if (tail && !__all_sync(0xffffffffu, mbar_try_wait(bar(IFULL + iq), iphase)) && !clear_tail()) break;
        const Item* ip = next_item();
        if (ip == nullptr) break;
        const int slot = ip->k0, hk = ip->hk, n = blocks(ip->n_keys);
        int j0 = ip->key0, rest = ip->nk - j0;  // the block's first position, and what the sequence holds from there on
        const int seq = ip->seq;
        // Keys that one item alone reads leave L2 first: they would push out those that the tile pairs of a longer chunk share.
        const uint64_t policy = l2_policy((long long)ip->nq * G <= 2 * TM);
        item_done();
        const int32_t* row = cv.table + (long long)slot * cv.width;
        // The whole warp walks the copies and one elected thread issues them: what they are given stays in uniform registers.
        for (int j = 0; j < n && ok; ++j, j0 += BK, rest -= BK) {
          // the pages (the 32 of a window begin at a multiple of 32, so that no block lies in two)
          const int col = j0 >> cv.page_shift;
          if (window_slot != slot || window != col >> 5) {
            auto read = [&](int w) {
              int page = w * 32 + lane < cv.width ? row[w * 32 + lane] : 0;
              if (page < 0 || page >= cv.n_pages) page = -1;
              return page;
            };
            page_now = window_slot == slot && window + 1 == col >> 5 ? page_next : read(col >> 5);
            window_slot = slot;
            window = col >> 5;
            page_next = read(window + 1);
          }
          const int held = min(BK, rest), boxes = (held + box - 1) >> box_shift;
          if (__any_sync(0xffffffffu, page_now < 0 && ((lane - col) & 31) < boxes)) {
            if (lane == 0) record_error(status, MOE_ERR_DEVICE_CHECK, seq);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {  // K, then V
            const bool cut = v == 1 && held < BK;
            if (tail && (++behind > 2 || cut) && !(ok = clear_tail())) break;
            ok = warp_wait(bar(EMPTY + stage), phase ^ 1u, timeout_ns, abort_flag, status, 51);
            if (!ok) break;
            const uint32_t b = cut ? bar(TAIL) : bar(FULL + stage);
            uint32_t dst = sKV + stage * C::kTileBytes;
            if (leader) mbar_arrive_expect_tx(b, (uint32_t)((boxes << box_shift) * C::kChunks * 128));
            for (int i = 0; i < boxes; ++i, dst += 128 << box_shift) {
              const int page = max(0, __shfl_sync(0xffffffffu, page_now, (col + i) & 31));
              const int g = (page * Hkv + hk) * cv.page_size + (j0 & (cv.page_size - 1));
              if (leader) {
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) tma_load_3d_hint(dst + c * (BK * 128), v ? &tmV : &tmK, 64 * c, g, sa.d.layer, b, policy);
              }
            }
            if (cut) {
              tail = true;
              behind = 0;
              tail_stage = stage;
              tail_keys = held;
            }
            filled |= 1u << stage;
            fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (!clear_tail() && lane == 0) {  // (given up: the copies are waited for all the same)
        mbar_wait_bounded(bar(TAIL), tail_phase, timeout_ns);
        mbar_arrive(bar(FULL + tail_stage));
      }
      if (lane == 0)
        for (int s = 0; s < C::kStages; ++s)
          if (filled & (1u << s)) mbar_wait_bounded(bar(FULL + s), (fill_phase >> s) & 1u, timeout_ns);
      __syncwarp();
    } else if (warp == kSoftWarps + 1) {
      // -------------------------------------------------------------- items, K and V
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_phase = 0;
      const int32_t* table = nullptr;
      int pages = 0;
      if (SHARED) {
        int slot = sa.d.lead[0];  // an out-of-range slot or page is recorded by the own part
        slot = slot < 0 || slot >= sa.d.c.n_slots ? 0 : slot;
        table = sa.d.c.table + (long long)slot * sa.d.c.width;
        pages = sa.d.shared >> sa.d.c.page_shift;
      }
      int* counter = status + 7;  // items taken; status[8]: CTAs that are done with it
      auto take = [&]() { return lane == 0 ? atomicAdd(counter, 1) : 0; };
      int ahead = SHARED ? 0 : take();  // the next item's number (lane 0), asked for early
      // The next item with rows, by the whole warp (last: none).
      auto find = [&](Item& it) {
        it = Item{};
        it.last = 1;
        if (SHARED) {
          if (ahead++ == 0) {
            it.hk = blockIdx.x;
            it.row0 = blockIdx.y * 2 * TM;
            it.nrows = min(2 * TM, sa.d.n * G - it.row0);
            it.key0 = blockIdx.z * sa.per;
            it.n_keys = min(sa.per, sa.d.shared - it.key0);
            it.lim0 = it.n_keys;
            it.lim1 = it.nrows > TM ? it.n_keys : 0;
            it.last = 0;
          }
          return;
        }
        while (true) {
          const int w = __shfl_sync(0xffffffffu, ahead, 0);
          if (w >= n_items) return;
          ahead = take();
          const int parts = SPLIT ? sa.splits : 1, v = w / parts;
          const int slot = (n_items / parts - 1 - v) / Hkv;
          const int i = find_tile_seq_warp(pa.qo, pa.n, G, 2 * TM, slot);
          const Seq sq = load_seq_warp(pa, i);
          const long long r0 = ((long long)slot - ((long long)sq.q0 * G / (2 * TM) + i)) * (2 * TM);
          if (r0 < 0 || r0 >= (long long)sq.nq * G) continue;  // a slot that no tile fills
          it.hk = v % Hkv;
          it.row0 = (int)r0;
          it.nrows = min(2 * TM, sq.nq * G - it.row0);
          it.q0 = sq.q0; it.nq = sq.nq; it.k0 = sq.k0; it.nk = sq.nk;
          it.lim0 = visible_keys((it.row0 + min(it.nrows, TM) - 1) / G, sq.nq, sq.nk, pa.causal);
          it.lim1 = it.nrows > TM ? visible_keys((it.row0 + it.nrows - 1) / G, sq.nq, sq.nk, pa.causal) : 0;
          it.n_keys = max(it.lim0, it.lim1);
          if (SPLIT) {
            it.split = w % parts;
            const int per = (blocks(it.n_keys) + parts - 1) / parts * BK;
            it.key0 = (int)min((long long)it.split * per, (long long)it.n_keys);
            it.n_keys = min(it.n_keys - it.key0, per);
            it.lim0 = max(0, min(it.lim0 - it.key0, it.n_keys));
            it.lim1 = max(0, min(it.lim1 - it.key0, it.n_keys));
          }
          it.last = 0;
          return;
        }
      };
      auto publish = [&](const Item& it) {
        bool ok = true;
        if (lane == 0) {
          ok = wait_or_abort(bar(IEMPTY + iq), iphase ^ 1u, timeout_ns, abort_flag, status, 51);
          if (ok) {
            items[iq] = it;
            mbar_arrive(bar(IFULL + iq));
          }
        }
        if (++iq == kItems) { iq = 0; iphase ^= 1u; }
        return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      };
      // copies u = begin .. end - 1 of an item (K and V of block u / 2)
      auto load = [&](const Item& it, int begin, int end) {
        bool ok = true;
        if (lane == 0) {
          for (int u = begin; u < end; ++u) {
            const CUtensorMap* tm = (u & 1) ? &tmV : &tmK;
            const int j0 = it.key0 + (u >> 1) * BK;
            ok = wait_or_abort(bar(EMPTY + stage), phase ^ 1u, timeout_ns, abort_flag, status, 51);
            if (!ok) break;
            const uint32_t dst = sKV + stage * C::kTileBytes;
            mbar_arrive_expect_tx(bar(FULL + stage), C::kTileBytes);
            if (SHARED) {
              const int rows = min(sa.d.c.page_size, BK);
              for (int r = 0; r < BK; r += rows) {
                // past the shared keys the last page again: those columns are masked (and looked through for values
                // that are not finite like any that a row does not see)
                const int p = min((j0 + r) >> sa.d.c.page_shift, pages - 1);
                int page = table[p];
                page = page < 0 || page >= sa.d.c.n_pages ? 0 : page;
                const int g = (page * Hkv + it.hk) * sa.d.c.page_size + ((j0 + r) & (sa.d.c.page_size - 1));
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                  tma_load_3d(dst + c * (BK * 128) + r * 128, tm, 64 * c, g, sa.d.layer, bar(FULL + stage));
              }
            } else {
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(dst + c * (BK * 128), tm, 64 * c, it.hk, it.k0 + j0, bar(FULL + stage));
            }
            filled |= 1u << stage;
            fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
          }
        }
        return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      };
      // The next item is taken when this one's last ring of copies is due: early enough for its Q to be on its way
      // in time, and no earlier, as a long item would keep it from the CTAs that are idle by then.
      Item it, nx;
      find(it);
      bool ok = publish(it);
      while (ok && !it.last) {
        const int end = 2 * blocks(it.n_keys), first = end <= C::kStages ? end : end - C::kStages;
        ok = load(it, 0, first);
        find(nx);
        ok = ok && publish(nx) && load(it, first, end);
        it = nx;
      }
      if (lane == 0) {
        if (!SHARED) {  // the CTA that is done last sets the counters back: nobody takes items any more
          __threadfence();
          if (atomicAdd(counter + 1, 1) == (int)gridDim.x - 1) {
            atomicExch(counter, 0);
            atomicExch(counter + 1, 0);
          }
        }
        for (int s = 0; s < C::kStages; ++s)
          if (filled & (1u << s)) mbar_wait_bounded(bar(FULL + s), (fill_phase >> s) & 1u, timeout_ns);
      }
      __syncwarp();
    } else if (warp > kSoftWarps + 1) {
      // -------------------------------------------------------------- Q tiles, the swizzled K-major operand. Where the
      // group's heads divide a tile's rows one TMA box is 128 / G tokens of G heads, in the packed rows' order (rows
      // past the end hold whatever comes next: they see no key and are not stored). Else kLanes lanes copy a row,
      // with zeros past the rows and past D: 5 us a tile, against 1.5.
      constexpr int kLanes = DP / 8, kRowsPer = 32 / kLanes;
      const int t = warp - kSoftWarps - 2;
      uint32_t loads = 0;
      // PAGED: the first of these warps walks the CTA's run and publishes its items, one ahead of the Q tiles it loads. It
      // looks at 32 tile slots at once, one a lane (the next of an item after the other cost 9 us an item).
      const bool finder = PAGED && t == 0;
      const Runs runs(finder ? plan[0] * Hkv : 0, gridDim.x);
      const long long run_begin = finder && (int)blockIdx.x < runs.n ? runs.begin(blockIdx.x) : 0;
      const long long run_end = finder && (int)blockIdx.x < runs.n ? runs.begin(blockIdx.x + 1) : 0;
      ChunkItem ci{};
      int base = finder ? (int)plan[1] & ~31 : 0, head = finder ? (int)plan[3] : 0, loaded = -1;
      long long x = 0, before = 0, length = 0;  // the place of the 32 slots from `base` on in this head, of the lane's item among them, of all
      int b0 = 0, b1 = 0;
      uint32_t todo = 0;  // the lanes whose items have blocks in the run and are not published yet
      bool late = false;
      auto load_slots = [&]() {
        const int s = base + lane;
        ci = s < n_items ? chunk_item(pa, sa, s, find_tile_seq(pa.qo, pa.n, G, 2 * TM, s)) : ChunkItem{};
        loaded = base;
        const long long len = ci.length();
        before = len;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, before, w);
          if (lane >= w) before += y;
        }
        length = __shfl_sync(0xffffffffu, before, 31);
        before -= len;
      };
      auto my_item = [&]() {
        const int all = max(1, ci.n_blocks);  // (without a key: an item all the same, whose results are 0)
        Item it{};
        it.hk = head;
        it.seq = ci.seq;
        it.row0 = ci.row0;
        it.nrows = ci.nrows;
        it.q0 = ci.q0; it.nq = ci.nq; it.k0 = ci.slot; it.nk = ci.nk;
        it.key0 = b0 * BK;
        it.n_keys = min((b1 - b0) * BK, max(ci.lim0, ci.lim1) - it.key0);
        it.lim0 = max(0, min(ci.lim0 - it.key0, it.n_keys));
        it.lim1 = max(0, min(ci.lim1 - it.key0, it.n_keys));
        it.dual = ci.nrows <= TM;
        if (it.dual) it.lim1 = it.lim0;
        it.split = b0 == 0 && b1 == all ? -1 : 2 * (int)blockIdx.x + (b0 == 0 ? 1 : 0);
        if (b0 == 0 && b1 < all) {
          ChunkRun r;
          r.hk = head; r.q0 = ci.q0; r.row0 = ci.row0; r.nrows = ci.nrows;
          r.end = runs.of(x + before + (long long)(all - 1) * kBlock);
          sa.runs[blockIdx.x] = r;
        }
        return it;
      };
      // The blocks of the slots' items that lie in the run: block j begins at x + before + j kBlock.
      auto look = [&]() {
        if (loaded != base) load_slots();
        const int all = max(1, ci.n_blocks);
        auto first_from = [&](long long p) {
          p -= x + before;
          return p <= 0 ? 0 : (int)min((long long)all, (p + kBlock - 1) / kBlock);
        };
        b0 = first_from(run_begin);
        b1 = first_from(run_end);
        const bool in = ci.nrows > 0 && b0 < b1;
        // The end of an item that began in another run comes last: the whole items of all runs then begin with their first
        // keys at about the same time, and L2 serves those that share a head.
        const bool is_late = in && x + before < run_begin;
        if (is_late) *late_item = my_item();
        __syncwarp();
        late = late || __any_sync(0xffffffffu, is_late);
        todo = __ballot_sync(0xffffffffu, in && !is_late);
      };
      bool ended = run_begin == run_end;
      if (!ended) {
        load_slots();
        x = plan[2] - __shfl_sync(0xffffffffu, before, (int)plan[1] & 31);
        look();
      }
      // Publishes the run's next item, or its end.
      auto advance = [&]() {
        while (todo == 0 && !ended) {
          x += length;
          base += 32;
          if (base >= n_items) {
            base = 0;
            ++head;
          }
          if (x >= run_end) ended = true;
          else look();
        }
        if (!warp_wait(bar(IEMPTY + iq), iphase ^ 1u, timeout_ns, abort_flag, status, 51)) return false;
        int from = 0;
        if (todo != 0) {
          from = __ffs(todo) - 1;
          todo &= todo - 1;
          if (lane == from) items[iq] = my_item();
        } else if (late) {
          late = false;
          if (lane == 0) items[iq] = *late_item;
        } else if (lane == 0) {
          items[iq] = Item{};
          items[iq].last = 1;
        }
        __syncwarp();
        if (lane == from) mbar_arrive(bar(IFULL + iq));
        if (++iq == kItems) { iq = 0; iphase ^= 1u; }
        return true;
      };
      int mine = 0;  // the place of the finder's own next item
      if (finder && !advance()) ended = true;
      while (true) {
        Item it;
        if (finder) {
          it = items[mine];
          if (it.last || !advance()) break;
          if (++mine == kItems) mine = 0;
        } else {
          const Item* ip = next_item();
          if (ip == nullptr) break;
          it = *ip;
          item_done();
        }
        if ((t ? it.lim1 : it.lim0) == 0) continue;
        if (!warp_wait(bar(QEMPTY + t), (loads & 1u) ^ 1u, timeout_ns, abort_flag, status, 55)) break;
        ++loads;
        if (q_tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(QFULL + t), C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sQ + t * C::kTileBytes + c * (TM * 128), &tmQ, 64 * c, it.hk * G,
                          it.q0 + (it.row0 + (PAGED && it.dual ? 0 : t * TM)) / G, bar(QFULL + t));
          }
          continue;
        }
        const int first = PAGED && it.dual ? 0 : t * TM, nrow_t = min(TM, it.nrows - first);
        const __nv_bfloat16* q = (const __nv_bfloat16*)(SHARED ? sa.d.q : pa.q) + (long long)(SHARED ? 0 : it.q0) * (SHARED ? sa.d.qs : pa.qs);
#pragma unroll
        for (int k = 0; k < TM / 32; ++k) {
          const int R = it.row0 + first + 32 * k + lane, tok = R / G;  // (rows past the end are not read)
          const __nv_bfloat16* row = q + (long long)tok * (SHARED ? sa.d.qs : pa.qs) + (long long)(it.hk * G + R - tok * G) * D;
#pragma unroll 4
          for (int i = 0; i < 32 / kRowsPer; ++i) {
            const int rr = i * kRowsPer + lane / kLanes, u = lane % kLanes, rt = 32 * k + rr;
            const __nv_bfloat16* src = (const __nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)row, rr);
            const bool in = rt < nrow_t && u * 8 < D;
            const uint32_t dst = sQ + t * C::kTileBytes + (u / 8) * (TM * 128) + rt * 128 + (((u & 7) ^ (rt & 7)) * 16);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? src + u * 8 : q), "r"(in ? 16 : 0)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(QFULL + t));
      }
      if (loads > 0) mbar_wait_bounded(bar(QFULL + t), (loads - 1) & 1u, timeout_ns);  // copies in flight
    } else {
      // -------------------------------------------------------------- MMAs
      // The whole warp walks the loop and one elected thread issues: descriptors and addresses then stay in uniform
      // registers. Inside a one-lane branch every MMA first moved its operands there, which took as long as
      // the MMA itself (about 70 of 64 cycles).
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_qk = make_idesc_bf16_f32(TM, BK, false);
      constexpr uint32_t idesc_half = make_idesc_bf16_f32(TM, BK / 2, false);
      constexpr uint32_t idesc_pv = make_idesc_bf16_f32(TM, DP, true);
      bool dual = false;  // tile t has keys t BK / 2 .. of each block (the same rows)
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
      auto qk = [&](int t, int st, int b2 = 0) {  // (b2: which half of the tile's columns, by halves of blocks)
        const uint64_t a = make_smem_desc_sw128(sQ + t * C::kTileBytes, 16, 1024);
        const uint64_t b = make_smem_desc_sw128(sKV + st * C::kTileBytes + (PAGED && dual ? t * (BK / 2) * 128 : 0), 16, 1024);
        const uint32_t idesc = PAGED && dual ? idesc_half : idesc_qk;
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * (TM * 128) + (kk % 4) * 32) >> 4);
          tc_mma_f16(tm + t * BK + b2 * (BK / 2), a + off, b + off, idesc, kk != 0);
        }
        tc_commit(bar(SFULL + 2 * b2 + t));
      };
      auto pv = [&](int t, int st, bool acc, int b2 = 0) {
        const uint64_t b = make_smem_desc_sw128(sKV + st * C::kTileBytes + (PAGED && dual ? t * (BK / 2) * 128 : 0), BK * 128, 1024);
        if (!leader) return;
        if (PAGED && dual) {
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_f16_ta(tm + 256 + t * DP, tm + t * BK + b2 * (BK / 2) + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                          acc || kk != 0);
          tc_commit(bar(ODONE + t));
          return;
        }
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_f16_ta(tm + 256 + t * DP, tm + t * BK + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4), idesc_pv,
                        acc || kk != 0);
        tc_commit(bar(ODONE + t));
      };
      auto next = [&]() { if (++stage == C::kStages) { stage = 0; phase ^= 1u; } };
      uint32_t pp0 = 0, pp1 = 0, qp0 = 0, qp1 = 0;  // phases of the tiles' P and Q barriers
      uint32_t pp0b = 0, pp1b = 0;                  // and of the second P barriers
      bool ok = true;
      while (ok) {
        const Item* it = next_item();
        if (it == nullptr) break;
        const int n0 = __shfl_sync(0xffffffffu, blocks(it->lim0), 0), n1 = __shfl_sync(0xffffffffu, blocks(it->lim1), 0);
        const int nn = max(n0, n1);
        dual = PAGED && __shfl_sync(0xffffffffu, it->dual, 0) != 0;
        item_done();
        if (nn == 0) continue;
        if (dual) {
          // Both halves' scores are computed two blocks ahead: they take half of the tile's columns each time, so block
          // j + 1 need not wait for the softmax of block j. Copy i of the item (K0 V0 K1 V1 ..) is in this stage:
          auto copy_at = [&](int i, int& st, uint32_t& ph) {
            const int x = stage + i;
            st = x & (C::kStages - 1);
            ph = phase ^ ((uint32_t)(x / C::kStages) & 1u);
          };
          int st, ks;
          uint32_t ph, kp;
          for (int j = 0; j < 2 && j < nn && ok; ++j) {
            copy_at(2 * j, st, ph);
            ok = wait(FULL + st, ph);
            if (ok && j == 0) {
              ok = wait(QFULL, qp0) && wait(QFULL + 1, qp1);
              qp0 ^= 1u;
              qp1 ^= 1u;
            }
            if (!ok) break;
            qk(0, st, j);
            qk(1, st, j);
            if (leader) {
              tc_commit(bar(EMPTY + st));
              if (j + 1 == nn) {
                tc_commit(bar(QEMPTY));
                tc_commit(bar(QEMPTY + 1));
              }
            }
          }
          for (int j = 0; j < nn && ok; ++j) {
            const int b2 = j & 1;
            const bool more = j + 2 < nn;
            copy_at(2 * j + 1, st, ph);
            ok = wait3(FULL + st, ph, FULL + st, ph, PFULL + 2 * b2, b2 ? pp0b : pp0);
            if (!ok) break;
            pv(0, st, j > 0, b2);
            ok = wait(PFULL + 2 * b2 + 1, b2 ? pp1b : pp1);
            if (!ok) break;
            pv(1, st, j > 0, b2);
            if (leader) tc_commit(bar(EMPTY + st));
            if (more) {
              copy_at(2 * j + 4, ks, kp);
              ok = wait(FULL + ks, kp);
              if (!ok) break;
              qk(0, ks, b2);
              qk(1, ks, b2);
            }
            if (b2) { pp0b ^= 1u; pp1b ^= 1u; } else { pp0 ^= 1u; pp1 ^= 1u; }
            if (leader) {
              if (more) tc_commit(bar(EMPTY + ks));
              if (more && j + 3 == nn) {
                tc_commit(bar(QEMPTY));
                tc_commit(bar(QEMPTY + 1));
              }
            }
          }
          copy_at(2 * nn, st, ph);
          stage = st;
          phase = ph;
          continue;
        }
        ok = wait(FULL + stage, phase);
        if (ok && n0 > 0) {
          ok = wait(QFULL, qp0);
          qp0 ^= 1u;
          if (ok) qk(0, stage);
          if (leader && n0 == 1) tc_commit(bar(QEMPTY));
        }
        if (ok && n1 > 0) {
          ok = wait(QFULL + 1, qp1);
          qp1 ^= 1u;
          if (ok) qk(1, stage);
          if (leader && n1 == 1) tc_commit(bar(QEMPTY + 1));
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
          ok = wait3(FULL + vs, vp, more ? FULL + ks : FULL + vs, more ? kp : vp, pb, j < n0 ? pp0 : pp1);
          if (!ok) break;
          if (j < n0) {
            pp0 ^= 1u;
            pv(0, vs, j > 0);
            if (j + 1 < n0) qk(0, ks);
            if (leader && j + 2 == n0) tc_commit(bar(QEMPTY));
            if (j < n1) ok = wait(PFULL + 1, pp1);
          }
          if (ok && j < n1) {
            pp1 ^= 1u;
            pv(1, vs, j > 0);
            if (j + 1 < n1) qk(1, ks);
            if (leader && j + 2 == n1) tc_commit(bar(QEMPTY + 1));
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int t = warp >> 2, r = tid & 127;  // tile, row of it
    const int q4 = warp & 3;                 // TMEM lanes 32 q4 ..
    const float c2 = (SHARED ? sa.d.scale : pa.scale) * 1.4426950408889634f;
    const float thr = rescale_above(c2);
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const uint32_t tS = tmem + lanes + t * BK, tO = tmem + lanes + 256 + t * DP;
    uint32_t done = 0;  // blocks of all items so far: the phase of the last PV's barrier
    uint32_t seen = 0;  // phases of the scores' barriers, a bit each
    uint32_t given = 0;  // exchanges with the other tile's warp
    bool ok = true;
    while (ok) {
      const Item* it = next_item();
      if (it == nullptr) break;
      // Where the thread's row lies. (A chunk's is found again after the loop, which has no registers to keep it in.)
      bool dual, valid;
      int tile0, nrow_t, tok, h;
      auto place = [&]() {
        int g = G;
        if (PAGED) asm volatile("" : "+r"(g));
        dual = PAGED && it->dual;
        tile0 = dual ? 0 : t * TM;               // the tile's first row of the item's
        nrow_t = min(TM, it->nrows - tile0);     // rows of this tile (<= 0: none)
        const int R = it->row0 + tile0 + r;
        valid = r < nrow_t;
        tok = valid ? R / g : 0;
        h = it->hk * g + (valid ? R % g : 0);
      };
      place();
      const int n = blocks(t ? it->lim1 : it->lim0);
      // (What a row past the tile's end makes of whatever lies there is dropped, so a chunk's are not masked: a tile of a single
      // token's heads would go through the masking below in every block.)
      int lim = PAGED && !valid ? 0x7fffffff : 0;
      if (valid && SHARED) {  // a slot shorter than the shared keys sees its own length of them
        lim = max(0, min(it->n_keys, slot_len(sa.d.c, sa.d.slots[tok]) - it->key0));
      } else if (valid) {
        lim = visible_keys(tok, it->nq, it->nk, pa.causal);
        if (SPLIT || PAGED) lim = max(0, min(lim - it->key0, it->n_keys));
      }
      float m = -INFINITY, l = 0.f;
      // Block j, of which the tile has COLS keys: 128, or half of them.
      auto block = [&](auto cols, int j) {
        constexpr int NC = decltype(cols)::value / 32;
        const int b2 = NC < 4 ? j & 1 : 0;  // by halves, blocks alternate between the halves of the tile's columns
        const uint32_t tB = tS + b2 * (BK / 2);
        ok = warp_wait(bar(SFULL + 2 * b2 + t), seen >> b2 & 1u, timeout_ns, abort_flag, status, 53);
        if (!ok) return;
        seen ^= 1u << b2;
        tc_fence_after();
        uint32_t s[NC][32];
#pragma unroll
        for (int c = 0; c < NC; ++c) tmem_ld_32x32b_x32(tB + 32 * c, s[c]);
        tmem_ld_wait();
        const int left = lim - j * BK - (NC < 4 ? t * (BK / 2) : 0);  // columns that this row sees
        if (__any_sync(0xffffffffu, left < 32 * NC)) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= left) s[c][i] = 0xff800000u;  // -inf
        }
        // four chains of three-input maxima (max drops a NaN score: the maximum is never NaN)
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16 * NC; ++i)
          mx4[i & 3] = max3(mx4[i & 3], __uint_as_float(s[i >> 4][2 * (i & 15)]), __uint_as_float(s[i >> 4][2 * (i & 15) + 1]));
        const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
        if (__any_sync(0xffffffffu, mx > m + thr)) {
          const bool up = mx > m + thr;
          if (j > 0) {
            ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
            if (!ok) return;
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
        for (int h = 0; h < NC / 2; ++h) {
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
          tmem_st_32x32b_x32(tB + 32 * h, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (NC < 4 && j > 0 && j == n - 1) {
          // Once this block's weights are given the barrier may go on by two phases, whose parities would look alike, so the
          // PV before (in flight for one softmax by now) is waited for first.
          ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
          if (!ok) return;
        }
        if (lane == 0) mbar_arrive(bar(PFULL + 2 * b2 + t));
        const uint64_t sum = fadd2(sum0, sum1);
        l += f2_lo(sum) + f2_hi(sum);
      };
      const bool halves = dual;
      for (int j = 0; j < n && ok; ++j) {
        if (PAGED && halves) block(std::integral_constant<int, BK / 2>{}, j);
        else block(std::integral_constant<int, BK>{}, j);
        done += ok ? 1 : 0;
      }
      // ---- the rows' results
      if (ok && n > 0) {
        ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
        tc_fence_after();
      }
      if (PAGED) place();
      if (ok && nrow_t > 0 && __any_sync(0xffffffffu, valid)) {
        uint32_t again = 0;  // rows whose results are looked at again (replace_unseen)
        if (PAGED && dual && t == 1) {
          // the other half of the keys of tile 0's rows: m, l and the sums to the warp there, 32 elements a step
          const uint32_t stg = sOut + warp * C::kStage;
          given_ml[32 * q4 + lane] = make_float2(m, l);
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c, ++given) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + 32 * c, o);  // (not this item's where there was no block: not used then)
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = m == -INFINITY ? 0u : o[i];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + ((i ^ (lane & 7)) * 16)),
                           "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                           : "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(GIVEN + q4));
            ok = ok && warp_wait(bar(TAKEN + q4), given & 1, timeout_ns, abort_flag, status, 56);
          }
        } else if (PAGED) {
          // a piece: the sums in fp32; a whole item: the results in bf16. 32 elements a step through shared memory, as below
          const bool part = it->split >= 0;
          const long long at = part ? ((long long)it->split * sa.piece_rows + tile0 + r) * D : (long long)(it->q0 + tok) * pa.os + (long long)h * D;
          uint8_t* orow = part ? reinterpret_cast<uint8_t*>(sa.part_o + at) : (uint8_t*)pa.out + 2 * at;
          float f1 = 0.f, f0 = 1.f;  // factors of tile 1's sums and of this tile's
          if (dual) {
            ok = warp_wait(bar(GIVEN + q4), given & 1, timeout_ns, abort_flag, status, 56);
            const float2 x = given_ml[32 * q4 + lane];
            const float top = fmaxf(m, x.x);
            f0 = m == -INFINITY ? 0.f : ex2((m - top) * c2);
            f1 = x.x == -INFINITY ? 0.f : ex2((x.x - top) * c2);
            l = l * f0 + x.y * f1;
            m = top;
          }
          const float f = part ? 1.f : l == 0.f ? 0.f : 1.0f / l;
          f0 *= f;
          f1 *= f;
          const uint32_t stg = sOut + warp * C::kStage;
          const uint64_t f2 = f2_pack(f0, f0), g2 = f2_pack(f1, f1);
          uint64_t odd = 0ull;  // (times 0 and added up, only a value that is not finite leaves something else than 0)
          // A row's 128 bytes (32 sums or 64 results) from shared memory to `to`, of which the first `elems` exist
          auto store = [&](uint32_t to, int elems, int per) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int u = lane & 7, rr = 4 * i + (lane >> 3);
              uint8_t* dst = (uint8_t*)__shfl_sync(0xffffffffu, (unsigned long long)orow, rr) + to + 16 * u;
              uint4 x;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                           : "r"(stg + rr * 128 + ((u ^ (rr & 7)) * 16)) : "memory");
              if (32 * q4 + rr < nrow_t && per * u < elems) *reinterpret_cast<uint4*>(dst) = x;
            }
          };
#pragma unroll 1  // (run once an item: what is not in the instruction cache costs more than the loop)
          for (int c = 0; c < DP / 64; ++c) {
            uint32_t o2[2][32];
            tmem_ld_32x32b_x32(tO + 64 * c, o2[0]);  // (not this item's where there was no block: lim is 0 then)
            tmem_ld_32x32b_x32(tO + 64 * c + 32, o2[1]);
            tmem_ld_wait();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t(&o)[32] = o2[b];
              if (dual && c + b > 0) ok = ok && warp_wait(bar(GIVEN + q4), given & 1, timeout_ns, abort_flag, status, 56);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint64_t v0 = ffma2(((uint64_t)o[4 * i + 1] << 32) | o[4 * i], f2, 0ull);
                uint64_t v1 = ffma2(((uint64_t)o[4 * i + 3] << 32) | o[4 * i + 2], f2, 0ull);
                if (dual) {
                  uint64_t x0, x1;
                  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x0), "=l"(x1)
                               : "r"(stg + 4 * C::kStage + lane * 128 + ((i ^ (lane & 7)) * 16)) : "memory");
                  v0 = ffma2(x0, g2, v0);
                  v1 = ffma2(x1, g2, v1);
                }
                if (lim == 0) v0 = v1 = 0ull;
                odd = ffma2(v0, 0ull, odd);
                odd = ffma2(v1, 0ull, odd);
                o[4 * i] = (uint32_t)v0;
                o[4 * i + 1] = (uint32_t)(v0 >> 32);
                o[4 * i + 2] = (uint32_t)v1;
                o[4 * i + 3] = (uint32_t)(v1 >> 32);
              }
              if (dual) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(TAKEN + q4));
                ++given;
              }
              if (part) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + ((i ^ (lane & 7)) * 16)),
                               "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                               : "memory");
                __syncwarp();
                store((2 * c + b) * 128, D - 64 * c - 32 * b, 4);
                __syncwarp();
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + (((4 * b + i) ^ (lane & 7)) * 16)),
                               "r"(pack_bf16x2(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1]))),
                               "r"(pack_bf16x2(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]))),
                               "r"(pack_bf16x2(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]))),
                               "r"(pack_bf16x2(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])))
                               : "memory");
              }
            }
            if (!part) {
              __syncwarp();
              store(c * 128, D - 64 * c, 8);
              __syncwarp();
            }
          }
          if (valid && part) sa.part_ml[(long long)it->split * sa.piece_rows + tile0 + r] = make_float2(m * c2, l);
          if (valid && !part && pa.lse != nullptr)
            pa.lse[(long long)(it->q0 + tok) * H + h] = lim == 0 ? -INFINITY : (m * c2 + log2f(l)) * 0.6931471805599453f;
          // (a row whose weights' sum is not finite sees a score that is not, and is NaN as a whole)
          again = __ballot_sync(0xffffffffu, valid && !(f2_lo(odd) + f2_hi(odd) == 0.f) && fabsf(l) <= 3.0e38f);
        } else if (SHARED || SPLIT) {
          const long long piece = SHARED ? ((long long)tok * H + h) * sa.splits + blockIdx.z
                                          : ((long long)(it->q0 + tok) * H + h) * sa.splits + it->split;
          const float* orow = sa.part_o + piece * D;
          const uint32_t stg = sOut + warp * C::kStage;  // 32 elements a step through shared memory, as below
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
#pragma unroll
            for (int i = 0; i < 8; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + ((i ^ (lane & 7)) * 16)),
                           "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                           : "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3), u = lane & 7;
              float* dst = (float*)__shfl_sync(0xffffffffu, (unsigned long long)orow, rr) + 32 * c + 4 * u;
              uint4 x;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                           : "r"(stg + rr * 128 + ((u ^ (rr & 7)) * 16)) : "memory");
              if (32 * q4 + rr < nrow_t && 32 * c + 4 * u < D) *reinterpret_cast<uint4*>(dst) = x;
            }
            __syncwarp();
          }
          if (valid) sa.part_ml[piece] = make_float2(m * c2, l);
          // (a row whose weights' sum is not finite sees a score that is not, and is NaN as a whole)
          again = __ballot_sync(0xffffffffu, valid && !fine && fabsf(l) <= 3.0e38f);
          Unseen unseen(SHARED ? n * BK : min(n * BK, pa.Tkv - it->k0 - it->key0));
          while (again != 0) {
            const int w = __ffs(again) - 1;
            again &= again - 1;
            const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
            const int limw = __shfl_sync(0xffffffffu, lim, w);
            const float mw = __shfl_sync(0xffffffffu, m, w), mcw = mw == -INFINITY ? 0.f : mw * c2;
            float o[8];
            long long pw;
            uint32_t cols;
            if (SPLIT) {
              pw = ((long long)(it->q0 + tw) * H + hw) * sa.splits + it->split;
              cols = replace_unseen(unseen, (const __nv_bfloat16*)pa.q + (long long)(it->q0 + tw) * pa.qs + (long long)hw * D,
                                    (const __nv_bfloat16*)pa.k + (long long)(it->k0 + it->key0) * pa.ks + (long long)it->hk * D,
                                    (const __nv_bfloat16*)pa.v + (long long)(it->k0 + it->key0) * pa.vs + (long long)it->hk * D,
                                    [&](int j, long long& ko, long long& vo) {
                                      ko = (long long)j * pa.ks;
                                      vo = (long long)j * pa.vs;
                                    },
                                    D, limw, c2, mcw, o);
            } else {
              // (the pages are the first slot's, which the other slots share, and past them the last one, as loaded)
              const CacheView& cv = sa.d.c;
              const int s0 = sa.d.lead[0], last = (sa.d.shared >> cv.page_shift) - 1;
              const int32_t* row = cv.table + (long long)(s0 < 0 || s0 >= cv.n_slots ? 0 : s0) * cv.width;
              pw = ((long long)tw * H + hw) * sa.splits + blockIdx.z;
              cols = replace_unseen(unseen, (const __nv_bfloat16*)sa.d.q + (long long)tw * sa.d.qs + (long long)hw * D,
                                    (const __nv_bfloat16*)sa.d.k, (const __nv_bfloat16*)sa.d.v,
                                    [&](int j, long long& ko, long long& vo) {
                                      const int p = it->key0 + j;
                                      int page = row[min(p >> cv.page_shift, last)];
                                      page = page < 0 || page >= cv.n_pages ? 0 : page;
                                      ko = vo = (((long long)page * Hkv + it->hk) * cv.page_size + (p & (cv.page_size - 1))) * D;
                                    },
                                    D, limw, c2, mcw, o);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (cols >> e & 1u) sa.part_o[pw * D + lane * 8 + e] = o[e];
          }
        } else {
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          // 64 elements a step through shared memory, so that a store covers 4 rows and not 32 (2.2 -> 0.8 us an
          // item)
          __nv_bfloat16* orow = (__nv_bfloat16*)pa.out + (long long)(it->q0 + tok) * pa.os + (long long)h * D;
          const uint32_t stg = sOut + warp * C::kStage;
          const uint64_t inv2 = f2_pack(inv, inv);
          uint64_t odd = 0ull;
#pragma unroll
          for (int c = 0; c < DP / 64; ++c) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t o[32];
              if (n > 0) {
                tmem_ld_32x32b_x32(tO + 64 * c + 32 * b, o);
                tmem_ld_wait();
              }
              // times 0 and added up, only a value that is not finite leaves something else than 0
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                uint64_t v = ffma2(((uint64_t)o[i + 1] << 32) | o[i], inv2, 0ull);
                v = lim == 0 ? 0ull : v;
                odd = ffma2(v, 0ull, odd);
                o[i] = (uint32_t)v;
                o[i + 1] = (uint32_t)(v >> 32);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + (((4 * b + i) ^ (lane & 7)) * 16)),
                             "r"(pack_bf16x2(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1]))),
                             "r"(pack_bf16x2(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]))),
                             "r"(pack_bf16x2(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]))),
                             "r"(pack_bf16x2(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])))
                             : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3), u = lane & 7;
              __nv_bfloat16* dst = (__nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)orow, rr) + 64 * c + 8 * u;
              uint4 x;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                           : "r"(stg + rr * 128 + ((u ^ (rr & 7)) * 16)) : "memory");
              if (32 * q4 + rr < nrow_t && 64 * c + 8 * u < D) *reinterpret_cast<uint4*>(dst) = x;
            }
            __syncwarp();
          }
          if (valid && pa.lse != nullptr)
            pa.lse[(long long)(it->q0 + tok) * H + h] = lim == 0 ? -INFINITY : (m * c2 + log2f(l)) * 0.6931471805599453f;
          // (a row whose weights' sum is not finite sees a score that is not, and is NaN as a whole)
          again = __ballot_sync(0xffffffffu, valid && !(f2_lo(odd) + f2_hi(odd) == 0.f) && fabsf(l) <= 3.0e38f);
          Unseen unseen(min(n * BK, pa.Tkv - it->k0));
          while (again != 0) {
            const int w = __ffs(again) - 1;
            again &= again - 1;
            const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
            const int limw = __shfl_sync(0xffffffffu, lim, w);
            const float mw = __shfl_sync(0xffffffffu, m, w), iw = __shfl_sync(0xffffffffu, inv, w);
            float o[8];
            const uint32_t cols = replace_unseen(
                unseen, (const __nv_bfloat16*)pa.q + (long long)(it->q0 + tw) * pa.qs + (long long)hw * D,
                (const __nv_bfloat16*)pa.k + (long long)it->k0 * pa.ks + (long long)it->hk * D,
                (const __nv_bfloat16*)pa.v + (long long)it->k0 * pa.vs + (long long)it->hk * D,
                [&](int j, long long& ko, long long& vo) {
                  ko = (long long)j * pa.ks;
                  vo = (long long)j * pa.vs;
                },
                D, limw, c2, mw == -INFINITY ? 0.f : mw * c2, o);
            __nv_bfloat16* dw = (__nv_bfloat16*)pa.out + (long long)(it->q0 + tw) * pa.os + (long long)hw * D;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (cols >> e & 1u) dw[lane * 8 + e] = __float2bfloat16_rn(o[e] * iw);
          }
        }
        if (PAGED && again != 0) {
          Unseen unseen(min(n * BK, it->nk - it->key0));
          while (again != 0) {
            const int w = __ffs(again) - 1;
            again &= again - 1;
            const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
            const float mw = __shfl_sync(0xffffffffu, m, w), lw = __shfl_sync(0xffffffffu, l, w);
            float o[8];
            const uint32_t cols = replace_unseen(
                unseen, (const __nv_bfloat16*)pa.q + (long long)(it->q0 + tw) * pa.qs + (long long)hw * D,
                (const __nv_bfloat16*)sa.d.k, (const __nv_bfloat16*)sa.d.v,
                [&](int j, long long& ko, long long& vo) {  // where key j of the item lies
                  const CacheView& cv = sa.d.c;
                  const int p = it->key0 + j;
                  int page = cv.table[(long long)it->k0 * cv.width + (p >> cv.page_shift)];
                  page = page < 0 || page >= cv.n_pages ? 0 : page;
                  ko = vo = (((long long)page * Hkv + it->hk) * cv.page_size + (p & (cv.page_size - 1))) * D;
                },
                D, __shfl_sync(0xffffffffu, lim, w), c2, mw == -INFINITY ? 0.f : mw * c2, o);
            float* po = sa.part_o + ((long long)it->split * sa.piece_rows + tile0 + 32 * q4 + w) * D + lane * 8;
            __nv_bfloat16* dw = (__nv_bfloat16*)pa.out + (long long)(it->q0 + tw) * pa.os + (long long)hw * D + lane * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (cols >> e & 1u) {
                if (it->split >= 0) po[e] = o[e];
                else dw[e] = __float2bfloat16_rn(o[e] * (lw == 0.f ? 0.f : 1.0f / lw));
              }
          }
        }
      }
      tc_fence_before();
      item_done();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A row's pieces in their order, a warp each, eight pieces on their way at a time.
__global__ void __launch_bounds__(128)
prompt_join_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ SharedArgs sa) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.Tq * a.H) return;
  const int tok = (int)(row / a.H), h = (int)(row % a.H);
  const Seq sq = load_seq_warp(a, find_tile_seq_warp(a.qo, a.n, 1, 1, tok, 0));
  if (tok < sq.q0 || tok >= sq.q0 + sq.nq) return;  // not a row of a sequence (or of one with bad offsets)
  const long long p0 = row * sa.splits;
  float M = -INFINITY, l = 0.f;
  for (int i = lane; i < sa.splits; i += 32) M = fmaxf(M, sa.part_ml[p0 + i].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  const bool on = lane * 4 < a.D;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < sa.splits; i0 += 32) {
    const float2 v = i0 + lane < sa.splits ? sa.part_ml[p0 + i0 + lane] : make_float2(-INFINITY, 0.f);
    const float wl = ex2(v.x - ref);
    l += wl * v.y;
    for (int y0 = 0; y0 < 32 && i0 + y0 < sa.splits; y0 += 8) {
      float4 u[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        u[y] = on && i0 + y0 + y < sa.splits
                   ? reinterpret_cast<const float4*>(sa.part_o + (p0 + i0 + y0 + y) * a.D)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = __shfl_sync(0xffffffffu, wl, y0 + y);
        o.x = fmaf(w, u[y].x, o.x);
        o.y = fmaf(w, u[y].y, o.y);
        o.z = fmaf(w, u[y].z, o.z);
        o.w = fmaf(w, u[y].w, o.w);
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (on) {
    uint2 u;
    u.x = pack_bf16x2(o.x * inv, o.y * inv);
    u.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + (long long)tok * a.os + (long long)h * a.D + lane * 4) = u;
  }
  if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// The rows that several runs share, by the run that such an item begins in (blockIdx.x): a warp a row, its pieces in
// their order, eight on their way at a time.
__global__ void __launch_bounds__(256)
chunk_join_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ SharedArgs sa) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5), c0 = blockIdx.x;
  const ChunkRun run = sa.runs[c0];
  if (r >= run.nrows) return;
  const int G = a.H / a.Hkv, R = run.row0 + r, tok = run.q0 + R / G, h = run.hk * G + R % G, n = run.end - c0 + 1;
  // run c0 has its last item's piece, the others their first's
  auto row = [&](int i) { return (long long)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * sa.piece_rows + r; };
  float M = -INFINITY, l = 0.f;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, sa.part_ml[row(i)].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  const bool on = lane * 4 < a.D;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float2 v = i0 + lane < n ? sa.part_ml[row(i0 + lane)] : make_float2(-INFINITY, 0.f);
    const float wl = ex2(v.x - ref);
    l += wl * v.y;
    for (int y0 = 0; y0 < 32 && i0 + y0 < n; y0 += 8) {
      float4 u[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        u[y] = on && i0 + y0 + y < n ? reinterpret_cast<const float4*>(sa.part_o + row(i0 + y0 + y) * a.D)[lane]
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float w = __shfl_sync(0xffffffffu, wl, y0 + y);
        o.x = fmaf(w, u[y].x, o.x);
        o.y = fmaf(w, u[y].y, o.y);
        o.z = fmaf(w, u[y].z, o.z);
        o.w = fmaf(w, u[y].w, o.w);
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (on) {
    uint2 u;
    u.x = pack_bf16x2(o.x * inv, o.y * inv);
    u.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + (long long)tok * a.os + (long long)h * a.D + lane * 4) = u;
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[(long long)tok * a.H + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

bool encode3(EncodeTiledFn enc, CUtensorMap* m, const void* p, int D, int heads, int T, long long stride, int box_heads,
             int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  return encode_tmap(enc, m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, str, box);
}
// Q's descriptor, where a tile is a box of whole tokens; *ok says whether there is one.
bool encode_q(EncodeTiledFn enc, CUtensorMap* m, const void* p, int D, int H, int G, int T, long long stride, int* ok) {
  *ok = TM % G == 0;
  return !*ok || encode3(enc, m, p, D, H, T, stride, G, TM / G);
}

template <int DP, bool SHARED, bool SPLIT, bool PAGED = false>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PromptArgs& pa,
                   const SharedArgs& sa, dim3 grid, int n_items, int q_tma, cudaStream_t s) {
  static std::atomic<int> done{0};
  auto kern = attn_tc_kernel<DP, SHARED, SPLIT, PAGED>;
  const cudaError_t e = allow_smem(kern, Cfg<DP>::kSmem, done);
  if (e != cudaSuccess) return e;
  if (PAGED) {
    // Not as a programmatic dependent: its CTAs would then take the SMs in the order in which the kernel before leaves them,
    // and CTAs with neighbouring runs, which read the same keys, would lie anywhere on the two dies. 64 sequences of single
    // tokens and chunks back to back: 1045 us so, 865 us in the usual order.
    kern<<<grid, dim3(kThreads), Cfg<DP>::kSmem, s>>>(tq, tk, tv, pa, sa, n_items, q_tma);
    return cudaGetLastError();
  }
  return launch_pdl(kern, grid, dim3(kThreads), Cfg<DP>::kSmem, s, tq, tk, tv, pa, sa, n_items, q_tma);
}

}  // namespace

// Few items: each item's keys in as many parts as fill the SMs, four blocks a part at least where the keys are one
// sequence's. Heads of 128, 32 on 8: 16 tokens with 1024 keys 14 us in two parts, 17 in one; 4096 keys 17 and 52;
// 32768 44 and 392; 512 tokens behind 4096 41 and 54. 1024 tokens of their own (half the keys masked), 8 heads: 18
// and 17.
int attn_prompt_splits(int n, int Tq, int Tkv, int H, int Hkv) {
  const long long items = prompt_tile_slots(Tq, n, H / Hkv, 2 * TM) * Hkv;
  const long long most = Tkv / (4 * BK), fill = items > 0 ? device_sm_count() / items : 1;
  return (int)(fill < most ? (fill < 1 ? 1 : fill) : (most < 1 ? 1 : most));
}

cudaError_t launch_attn_prompt_tc(const PromptArgs& a, int splits, float* part, cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap tq{}, tk{}, tv{};
  const int G = a.H / a.Hkv;
  int q_tma = 0;
  if (!encode3(enc, &tk, a.k, a.D, a.Hkv, a.Tkv, a.ks, 1, BK) || !encode3(enc, &tv, a.v, a.D, a.Hkv, a.Tkv, a.vs, 1, BK) ||
      !encode_q(enc, &tq, a.q, a.D, a.H, G, a.Tq, a.qs, &q_tma))
    return cudaErrorInvalidValue;
  const long long slots = prompt_tile_slots(a.Tq, a.n, G, 2 * TM);
  SharedArgs sa{};
  sa.splits = splits;
  sa.part_o = part;
  sa.part_ml = reinterpret_cast<float2*>(part + (long long)a.Tq * a.H * splits * a.D);
  const long long items = slots * a.Hkv * splits;
  const dim3 grid((unsigned)(items < device_sm_count() ? items : device_sm_count()));
  if (splits == 1)
    return a.D <= 64 ? launch<64, false, false>(tq, tk, tv, a, sa, grid, (int)items, q_tma, s)
                     : launch<128, false, false>(tq, tk, tv, a, sa, grid, (int)items, q_tma, s);
  const cudaError_t e = a.D <= 64 ? launch<64, false, true>(tq, tk, tv, a, sa, grid, (int)items, q_tma, s)
                                  : launch<128, false, true>(tq, tk, tv, a, sa, grid, (int)items, q_tma, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_join_kernel, dim3((unsigned)(((long long)a.Tq * a.H + 3) / 4)), dim3(128), 0, s, a, sa);
}

// One CTA an SM takes 256 rows of one key/value head, the keys split over the SMs; about a sixth of those (where
// splits can be had) are left to the own keys, which run beside. 64 sequences behind 32768 positions, own keys up to
// 2048: see launch_attn_decode_tc.
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
  EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap tq{};
  int q_tma = 0;
  if (enc == nullptr || !encode_q(enc, &tq, a.q, a.c.D, a.H, a.H / a.c.Hkv, a.n, a.qs, &q_tma)) return cudaErrorInvalidValue;
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
  return a.c.D <= 64 ? launch<64, true, false>(tq, m.k128, m.v128, none, sa, grid, 0, q_tma, s)
                     : launch<128, true, false>(tq, m.k128, m.v128, none, sa, grid, 0, q_tma, s);
}

int chunk_piece_rows(int Tq, int G) {
  return (long long)Tq * G < 2 * TM ? Tq * G : 2 * TM;
}

cudaError_t launch_attn_chunk_tc(const PromptArgs& a, const DecodeArgs& d, const CacheMaps& m, ChunkRun* runs, float* part,
                                 cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap tq{};
  const int G = a.H / a.Hkv;
  int q_tma = 0;
  if (enc == nullptr || !encode_q(enc, &tq, a.q, a.D, a.H, G, a.Tq, a.qs, &q_tma)) return cudaErrorInvalidValue;
  const int slots = (int)prompt_tile_slots(a.Tq, a.n, G, 2 * TM);
  // one CTA an SM, as far as the longest sequences that the cache may hold make as many runs
  const long long runs_most = a.Hkv * (long long)slots * (kItem + ((long long)d.c.width * d.c.page_size + BK - 1) / BK * kBlock) / kShortest;
  const int ctas = (int)(runs_most < 1 ? 1 : (runs_most < device_sm_count() ? runs_most : device_sm_count()));
  SharedArgs sa{};
  sa.d = d;
  sa.runs = runs;
  sa.piece_rows = chunk_piece_rows(a.Tq, G);
  sa.part_o = part;
  sa.part_ml = reinterpret_cast<float2*>(part + 2LL * ctas * sa.piece_rows * a.D);
  const cudaError_t e = a.D <= 64 ? launch<64, false, false, true>(tq, m.k128, m.v128, a, sa, dim3(ctas), slots, q_tma, s)
                                  : launch<128, false, false, true>(tq, m.k128, m.v128, a, sa, dim3(ctas), slots, q_tma, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_join_kernel, dim3((unsigned)ctas, (unsigned)((sa.piece_rows + 7) / 8)), dim3(256), 0, s, a, sa);
}

}  // namespace moe

// Chunks: the new tokens of each sequence against everything that its slot of the paged cache holds, theirs included
// (bf16, heads of up to 128 elements, on the 5th-generation tensor cores). A prompt's piece, a draft of a few tokens
// and single tokens lie in one call.
//   S = Q K^T (scores), P = 2^(c S - c m) (weights, c = scale log2 e), O += P V, out = O / l
// in one pass over the keys, as for packed prompts (attn_tc.cu), whose item, MMA order and rescaling these are: 256
// packed rows (two tiles of 128) of one key/value head, with m only raised when a maximum exceeds it by 8 in log2 units.
// A weight is rounded to bf16 (off by at most 2^-8 of it) because the MMA takes both operands in one type; the weights' sum,
// O and the pieces of rows are fp32. That moves results by 5.4e-4 to 7.2e-4 of their norm (64 sequences with 8 chunks; 4096
// tokens behind 28672) and by up to 1.6e-3 where rows see few keys, beside the 1.7e-3 that their own rounding to bf16 is:
// from 64 bits they are 1.7e-3 with either weights, and 1.8e-3 over few keys. What is different here:
// - Work is shared out by keys, not by items (attn_plan.cuh): one sequence of 100,000 keys beside a hundred short ones takes
//   every SM.
// - Keys and values come from pages, by one TMA box a page and 64 elements (of pages of 128 positions and more a box a
//   block), and no page past a sequence's last is read. Values past its end become zeros in shared memory.
// - An item of one tile (a decoding sequence's heads, a short draft) would leave one softmax group idle, and the MMAs
//   waiting for the other: both groups take the same rows then, each half of every block's keys, with scores two blocks
//   ahead, and add up at the end. (64 single tokens behind up to 8192: 182 us, 6.2 TB/s.)
// - There is no output staging: rows are stored 32 bytes a lane, and the ring has a fifth stage in its place (a block
//   that misses L2 takes up to 2.6 us to come: 64 sequences with 8 chunks 811 us with four, 772 with five).
// Warps of a CTA (one an SM):
//   0..3, 4..7  softmax of tile 0 / 1 (or of the halves of the keys); thread = row = TMEM lane
//   8           allocates TMEM; one elected thread issues every MMA
//   9           pages, K and V by TMA into a ring
//   10          finds the items, one ahead, and loads tile 0's Q
//   11          loads tile 1's Q
// All waits are bounded; a wait that runs out records an error, and the CTA ends after its copies and MMAs have. So are
// the loops over sequences and slots, and the heads and runs that they name, whatever the offsets and lengths hold.
// Measured, heads of 128: 4096 tokens behind 28672, 32 heads on 8, 1.15 ms in a run of ten (1.79 PFLOP/s, 92% of the
// matrix rate measured in a burst), 1.25 in a loop of seconds: a block of a pair of tiles takes 1.31 to 1.36 us, of which
// its MMAs are 1.13 at the nominal rate, an item 5 to 6 us more. 64 sequences, 64 heads on 8, up to 16384 positions, 8
// with a piece of a prompt and 56 with 1 to 4 tokens: 0.69 ms; the chunks' MMAs alone would take 0.39, the reads 0.31.
// The pairs of tiles take 1.45 us a block there, as their keys come from memory beside the others' reads. Fetching them
// into L2 a few blocks ahead made it slower (772 -> 875 us: the lookups of L2 count). 64 drafts of 4 tokens behind up to
// 16384: 340 us, 6.7 TB/s, 98% of the copy rate. 40 tokens of 3 sequences behind 100: 14 us, the code and five waits on
// memory one behind the other (offsets, lengths, pages, keys, pieces).
#include "attn_tc.cuh"

namespace moe {
namespace {

struct __align__(16) Item {
  int hk, row0, nrows;      // key/value head; packed rows row0 .. of the sequence
  int q0, nq, k0, nk;       // the sequence: first token and tokens, slot and positions held
  int key0, n_keys;         // keys of the item
  int lim0, lim1;           // keys that each tile's last row sees (relative to key0)
  int last;                 // no item: the end
  int seq;                  // (for errors)
  int dual;                 // one tile of rows: both softmax groups take it, with half of each block's keys
  int piece;                // the first row of the piece that takes the results (-1: the output)
};
constexpr int kItems = 3;   // items published: one worked on, one ahead, one being given back
constexpr int kItemReaders = 1 + 8 + 2;

// What a CTA has of a kind: the length of all items of a head, its run's number, beginning and end, and the slot, place
// and head of the item that the run begins in.
struct Plan {
  long long all, begin, end, x;
  int run, slot, head, unused;
};

template <int DP> struct Cfg {
  static constexpr int kChunks = DP / 64;          // 64-element (128-byte) swizzle columns of a row
  static constexpr int kTileBytes = TM * DP * 2;   // a Q tile, and a K or V block
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr int kBars = 2 * kStages + 7 * 2 + 1 + 2 * kItems + 1 + 8;
  static constexpr int kPlan = 2 * (sizeof(Plan) / 8 + kThreads / 32);
  // tiles and ring, (m, l) of both tiles' rows, items, the plan, barriers, and the TMEM address beside the abort flag and
  // the first sequence of bad offsets
  static constexpr size_t kSmem = (size_t)(2 + kStages) * kTileBytes + 2 * TM * 8 + (kItems + 1) * sizeof(Item) +
                                  8 * kPlan + 8 * kBars + 16;
};
static_assert(Cfg<128>::kSmem <= kMaxSmem && Cfg<64>::kSmem <= kMaxSmem, "shared memory");

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

// Eight words to a multiple of 32 bytes.
__device__ __forceinline__ void store_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

struct ChunkArgs {
  DecodeArgs d;
  ChunkRun* runs;  // [kind][run] the item that begins in each run and goes on in the next ones
  int rows[2];     // rows of a piece, by kind
  int ctas;
  float* part_o;   // [kind][2 runs][rows][D]
  float2* part_ml;
  // The pieces' rows before run c's: of its first item, which began in another run, or of its last.
  __device__ __forceinline__ int piece(int kind, int c, bool last) const {
    return (kind ? 2 * ctas * rows[0] : 0) + (2 * c + (last ? 1 : 0)) * rows[kind];
  }
};

static_assert(chunk::kTile == TM && chunk::kKeys == BK, "tiles");

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptArgs pa,
               const __grid_constant__ ChunkArgs ca, int n_items, int q_tma) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (an address that the compiler does not know: it would keep dozens of sums with it in registers)
  uint32_t sQ = smem_u32(smem_raw);
  asm volatile("" : "+r"(sQ));
  uint8_t* smem = smem_raw + (sQ - smem_u32(smem_raw));
  const uint32_t sKV = sQ + 2 * C::kTileBytes;
  float2* given_ml = reinterpret_cast<float2*>(smem + (2 + C::kStages) * C::kTileBytes);  // [tile][row]
  Item* items = reinterpret_cast<Item*>(given_ml + 2 * TM);                                // [kItems]
  Item* late_item = items + kItems;
  Plan* plan = reinterpret_cast<Plan*>(items + kItems + 1);     // [kind]
  long long* warp_sums = reinterpret_cast<long long*>(plan + 2);  // [kind][warp]
  uint64_t* bars = reinterpret_cast<uint64_t*>(warp_sums + 2 * (kThreads / 32));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first_bad = reinterpret_cast<int*>(tmem_slot + 2);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int FULL = 0, EMPTY = C::kStages, QFULL = 2 * C::kStages, SFULL = QFULL + 2, PFULL = SFULL + 4,
                ODONE = PFULL + 4, QEMPTY = ODONE + 2, DONE = QEMPTY + 2, IFULL = DONE + 1, IEMPTY = IFULL + kItems,
                TAIL = IEMPTY + kItems, GIVEN = TAIL + 1, TAKEN = GIVEN + 4;

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
    for (int i = 0; i < 8; ++i) mbar_init(bar(GIVEN + i), 2);
    fence_mbar_init();
    *abort_flag = 0;
    *first_bad = pa.n;
    for (int kind = 0; kind < 2; ++kind) plan[kind].x = plan[kind].slot = plan[kind].head = 0;
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
  // Only after TMEM is allocated: a dependent kernel that starts on this SM may allocate some before it waits for this grid.
  griddep_launch_dependents();

  const int H = pa.H, Hkv = pa.Hkv, D = pa.D, G = H / Hkv;
  int* status = pa.status;
  const uint64_t timeout_ns = pa.timeout_ns;
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
  auto blocks = [](int keys) { return chunk::blocks_of(keys); };

  int seqs = pa.n;  // in front of the first bad offsets
  // This CTA's runs: a scan over the lengths of all tile slots, each thread with some of them in a row.
  {
    const int per = (n_items + kThreads - 1) / kThreads, s0 = min(n_items, tid * per), s1 = min(n_items, s0 + per);
    // The offsets are looked at beside the walk, and it is done again without the sequences from the first bad ones on:
    // in the usual case that costs no wait of its own.
    auto walk = [&](auto f) {
      chunk::walk_slots(pa.qo, seqs, pa.Tq, G, pa.causal, s0, s1,
                        [&](int i) { return slot_len(ca.d.c, ca.d.slots[i]); }, f);
    };
    long long sum[2], upto[2];
    while (true) {
      int bad = seqs;  // (from the last thread on: those of a short call have no slots to walk)
#pragma unroll 1
      for (int i = kThreads - 1 - tid; i < seqs && bad == seqs; i += kThreads)
        if (bad_offsets(pa.qo[i], pa.qo[i + 1], pa.Tq)) bad = i;
      sum[0] = sum[1] = 0;
      if (s0 < s1)
        walk([&](int, int kind, long long len) {
          sum[0] += kind ? 0 : len;
          sum[1] += kind ? len : 0;
          return true;
        });
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        upto[kind] = sum[kind];
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, upto[kind], w);
          if (lane >= w) upto[kind] += x;
        }
        if (lane == 31) warp_sums[kind * (kThreads / 32) + warp] = upto[kind];
      }
      if (!__syncthreads_or(bad < seqs)) break;
      if (bad < seqs) atomicMin(first_bad, bad);
      __syncthreads();
      seqs = *first_bad;
    }
    long long total[2] = {0, 0};
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) upto[kind] += total[kind];
        total[kind] += warp_sums[kind * (kThreads / 32) + w];
      }
    const chunk::Runs runs0(0, total[0] * Hkv, total[1] * Hkv, gridDim.x);
    long long at[2], x[2];  // the run's beginning in its head; the item's after the ones looked through
    bool here[2];           // it lies in one of this thread's slots
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const long long all = total[kind];
      const int c = chunk::run_of(kind, runs0, blockIdx.x, gridDim.x);
      long long begin = 0, end = 0;
      here[kind] = false;
      if (all > 0) {
        const chunk::Runs runs(kind, total[0] * Hkv, total[1] * Hkv, gridDim.x);
        if (c < runs.n) {
          begin = runs.begin(c);
          end = runs.begin(c + 1);
          const int head = (int)(begin / all);
          at[kind] = begin - head * all;
          x[kind] = upto[kind] - sum[kind];
          here[kind] = at[kind] >= x[kind] && at[kind] < upto[kind];
          if (here[kind]) plan[kind].head = head;
        }
      }
      if (tid == 0) {
        plan[kind].all = all;
        plan[kind].run = c;
        plan[kind].begin = begin;
        plan[kind].end = end;
        ChunkRun none;
        none.nrows = 0;
        ca.runs[kind * gridDim.x + c] = none;
      }
    }
    if (here[0] || here[1])
      walk([&](int s, int k, long long len) {
#pragma unroll
        for (int kind = 0; kind < 2; ++kind)
          if (k == kind && here[kind]) {
            plan[kind].slot = s;
            plan[kind].x = x[kind] - at[kind];  // where item (head, slot s) begins, from the run's beginning on
            x[kind] += len;
            here[kind] = x[kind] <= at[kind];
          }
        return here[0] || here[1];
      });
    __syncthreads();
  }

  if (warp >= kSoftWarps) {
    // 8 * 32 * 216 + 4 * 32 * 72 = 64512, as at the launch. (With 224 and 56 these warps spill twice as much: 4096 tokens
    // behind 28672 1167 us, 1150 so.)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kSoftWarps + 1) {
      // -------------------------------------------------------------- K and V (warp 10 finds the items)
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_phase = 0;
      // the pages of 32 x page_size positions from table column 32 `window` on and of the next ones, a page a lane
      int window_slot = -1, window = 0, page_now = 0, page_next = 0;
      bool tail = false;  // the last block of values loaded needs its end cleared
      int tail_stage = 0, tail_keys = 0, behind = 0;
      uint32_t tail_phase = 0;
      // What pages hold past a sequence's end is anyone's: the last block's values there become zeros once they have
      // arrived, as 0 times a leftover that is not finite would be NaN. This is done when the two copies behind them are
      // on their way: their stages wait for nothing that comes after the block before.
      auto clear_tail = [&]() {
        if (!tail) return true;
        if (!warp_wait(bar(TAIL), tail_phase, timeout_ns, abort_flag, status, 51)) return false;
        tail = false;
        tail_phase ^= 1u;
        const uint32_t dst = sKV + tail_stage * C::kTileBytes;
        for (int i = lane; i < (BK - tail_keys) * 8; i += 32)
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                         ::"r"(dst + c * (BK * 128) + tail_keys * 128 + i * 16), "r"(0) : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FULL + tail_stage));
        return true;
      };
      const CacheView& cv = ca.d.c;
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
        // Keys that one item alone reads leave L2 first: they would push out those that the items of a longer chunk
        // share (64 single tokens behind up to 8192: 194 us without, 183 so; 64 drafts behind 16384 shared positions, whose
        // items read the same pages: 475 and 469).
        const uint64_t policy = l2_policy((long long)ip->nq * G <= 2 * TM);
        // Copies lie in the ring in the order in which the MMAs take them: K0 V0 K1 V1 .., and where the scores are
        // computed two blocks ahead K0 K1 V0 K2 V1 .. (each copy then has two blocks' time to arrive).
        const int lag = ip->dual;
        item_done();
        const int32_t* row = cv.table + (long long)slot * cv.width;
        // The whole warp walks the copies and one elected thread issues them: what they are given stays in uniform
        // registers.
        for (int j = 0; j < n + lag && ok; ++j, j0 += BK, rest -= BK) {
          int page_v = page_now;
          if (j < n) {
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
            const int boxes = (min(BK, rest) + box - 1) >> box_shift;
            if (__any_sync(0xffffffffu, page_now < 0 && ((lane - col) & 31) < boxes)) {
              if (lane == 0) record_error(status, MOE_ERR_DEVICE_CHECK, seq);
            }
          }
          if (lag == 0) page_v = page_now;
#pragma unroll
          for (int v = 0; v < 2; ++v) {  // K of block j, then V of block j - lag
            if (v ? j < lag : j >= n) continue;
            const int back = v ? lag * BK : 0, p0 = j0 - back, held = min(BK, rest + back);
            const int col = p0 >> cv.page_shift, boxes = (held + box - 1) >> box_shift;
            const bool cut = v == 1 && held < BK;
            if (tail && (++behind > 2 || cut) && !(ok = clear_tail())) break;
            ok = warp_wait(bar(EMPTY + stage), phase ^ 1u, timeout_ns, abort_flag, status, 51);
            if (!ok) break;
            const uint32_t b = cut ? bar(TAIL) : bar(FULL + stage);
            uint32_t dst = sKV + stage * C::kTileBytes;
            if (leader) mbar_arrive_expect_tx(b, (uint32_t)((boxes << box_shift) * C::kChunks * 128));
            for (int i = 0; i < boxes; ++i, dst += 128 << box_shift) {
              const int page = max(0, __shfl_sync(0xffffffffu, v ? page_v : page_now, (col + i) & 31));
              const int g = (page * Hkv + hk) * cv.page_size + (p0 & (cv.page_size - 1));
              if (leader) {
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                  tma_load_3d_hint(dst + c * (BK * 128), v ? &tmV : &tmK, 64 * c, g, ca.d.layer, b, policy);
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
    } else if (warp > kSoftWarps + 1) {
      // -------------------------------------------------------------- Q tiles, the swizzled K-major operand. Where the
      // group's heads divide a tile's rows one TMA box is 128 / G tokens of G heads, in the packed rows' order (rows
      // past the end hold whatever comes next: they see no key and are not stored). Else kLanes lanes copy a row,
      // with zeros past the rows and past D: 5 us a tile, against 1.5.
      constexpr int kLanes = DP / 8, kRowsPer = 32 / kLanes;
      const int t = warp - kSoftWarps - 2;
      uint32_t loads = 0;
      // The first of these warps walks the CTA's runs and publishes their items, one ahead of the Q tiles it loads. It
      // looks at 32 tile slots at once, one a lane (the next of an item after the other cost 9 us an item).
      const bool finder = t == 0;
      int kind = 0;  // of the run at hand
      chunk::SlotItem ci{};
      // the 32 slots at hand, the place of the lane's item among them, the length of all
      chunk::Place at{0, 0, 0};
      int loaded = -1;
      long long before = 0, length = 0;
      int b0 = 0, b1 = 0;
      uint32_t todo = 0;  // the lanes whose items have blocks in the run and are not published yet
      bool late = false, ended = true;
      auto load_slots = [&]() {
        const int s = at.base + lane;
        ci = chunk::SlotItem{};
        if (s < n_items)
          ci = chunk::slot_item(pa.qo, ca.d.slots, pa.Tq, G, pa.causal, s,
                                find_tile_seq(pa.qo, seqs, G, chunk::kRows, s),
                                [&](int slot) { return slot_len(ca.d.c, slot); });
        if (chunk::item_kind(ci.nrows) != kind) ci.nrows = 0;
        loaded = at.base;
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
        it.hk = at.head;
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
        it.piece = b0 == 0 && b1 == all ? -1 : ca.piece(kind, plan[kind].run, b0 == 0);
        if (b0 == 0 && b1 < all) {
          ChunkRun r;
          r.hk = at.head; r.q0 = ci.q0; r.row0 = ci.row0; r.nrows = ci.nrows;
          r.end = chunk::Runs(kind, plan[0].all * Hkv, plan[1].all * Hkv, gridDim.x).of(
              plan[kind].begin + at.x + before + (long long)(all - 1) * chunk::kBlock);
          ca.runs[kind * gridDim.x + plan[kind].run] = r;
        }
        return it;
      };
      // The blocks of the slots' items that lie in the run: block j begins at at.x + before + j kBlock.
      auto look = [&]() {
        if (loaded != at.base) {
          const bool begins = loaded < 0;
          load_slots();
          if (begins) at.x -= __shfl_sync(0xffffffffu, before, plan[kind].slot & 31);
        }
        const int all = max(1, ci.n_blocks);
        b0 = chunk::first_block(0, at.x + before, all);
        b1 = chunk::first_block(plan[kind].end - plan[kind].begin, at.x + before, all);
        const bool in = ci.nrows > 0 && b0 < b1;
        // The end of an item that began in another run comes last: the whole items of all runs then begin with their
        // first keys at about the same time, and L2 serves those that share a head.
        const bool is_late = in && at.x + before < 0;
        if (is_late) *late_item = my_item();
        __syncwarp();
        late = late || __any_sync(0xffffffffu, is_late);
        todo = __ballot_sync(0xffffffffu, in && !is_late);
      };
      const int first_kind = 2 * blockIdx.x < gridDim.x ? 0 : 1;
      int begun = 0;  // kinds
      // Publishes the next item, or the end.
      auto advance = [&]() {
        while (todo == 0) {
          if (ended) {
            if (late || begun == 2) break;
            kind = begun++ ? 1 - first_kind : first_kind;
            if (plan[kind].begin == plan[kind].end) continue;
            ended = false;
            at.base = plan[kind].slot & ~31;
            at.head = plan[kind].head;
            loaded = -1;
            at.x = plan[kind].x;  // (of the run's first item: those before it are taken off below)
          } else if (!at.next(length, plan[kind].end - plan[kind].begin, n_items, Hkv)) {
            ended = true;
            continue;
          }
          look();
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
      int mine = -1;  // the place of the finder's own next item (none is published yet)
      while (true) {
        Item it;
        if (finder) {
          if (mine >= 0) it = items[mine];
          if ((mine >= 0 && it.last) || !advance()) break;
          if (mine++ < 0) continue;
          if (mine == kItems) mine = 0;
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
                          it.q0 + (it.row0 + (it.dual ? 0 : t * TM)) / G, bar(QFULL + t));
          }
          continue;
        }
        const int first = it.dual ? 0 : t * TM, nrow_t = min(TM, it.nrows - first);
        const __nv_bfloat16* q = (const __nv_bfloat16*)pa.q + (long long)it.q0 * pa.qs;
#pragma unroll
        for (int k = 0; k < TM / 32; ++k) {
          const int R = it.row0 + first + 32 * k + lane, tok = R / G;  // (rows past the end are not read)
          const __nv_bfloat16* row = q + (long long)tok * pa.qs + (long long)(it.hk * G + R - tok * G) * D;
#pragma unroll 4
          for (int i = 0; i < 32 / kRowsPer; ++i) {
            const int rr = i * kRowsPer + lane / kLanes, u = lane % kLanes, rt = 32 * k + rr;
            const __nv_bfloat16* src = (const __nv_bfloat16*)__shfl_sync(0xffffffffu, (unsigned long long)row, rr);
            const bool in = rt < nrow_t && u * 8 < D;
            const uint32_t dst = sQ + t * C::kTileBytes + (u / 8) * (TM * 128) + rt * 128 + (((u & 7) ^ (rt & 7)) * 16);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(dst), "l"(in ? src + u * 8 : q), "r"(in ? 16 : 0) : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(QFULL + t));
      }
      if (loads > 0) mbar_wait_bounded(bar(QFULL + t), (loads - 1) & 1u, timeout_ns);  // copies in flight
      if (t == 1)  // (records what is out of range)
        for (int i = blockIdx.x * 32 + lane; i < pa.n; i += gridDim.x * 32) load_chunk_seq(pa, ca.d, i);
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
      auto keys_of = [&](int t, int st) { return sKV + st * C::kTileBytes + (dual ? t * (BK / 2) * 128 : 0); };
      auto qk = [&](int t, int st, int b2 = 0) {  // (b2: which half of the tile's columns, by halves of blocks)
        const uint64_t a = make_smem_desc_sw128(sQ + t * C::kTileBytes, 16, 1024);
        const uint64_t b = make_smem_desc_sw128(keys_of(t, st), 16, 1024);
        const uint32_t idesc = dual ? idesc_half : idesc_qk;
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk / 4) * (TM * 128) + (kk % 4) * 32) >> 4);
          tc_mma_f16(tm + t * BK + b2 * (BK / 2), a + off, b + off, idesc, kk != 0);
        }
        tc_commit(bar(SFULL + 2 * b2 + t));
      };
      auto pv = [&](int t, int st, bool acc, int b2 = 0) {
        const uint64_t b = make_smem_desc_sw128(keys_of(t, st), BK * 128, 1024);
        if (!leader) return;
        if (dual) {
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_f16_ta(tm + 256 + t * DP, tm + t * BK + b2 * (BK / 2) + kk * 8, b + (uint64_t)((kk * 16 * 128) >> 4),
                          idesc_pv, acc || kk != 0);
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
        const int n0 = __shfl_sync(0xffffffffu, blocks(it->lim0), 0);
        const int n1 = __shfl_sync(0xffffffffu, blocks(it->lim1), 0);
        const int nn = max(n0, n1);
        dual = __shfl_sync(0xffffffffu, it->dual, 0) != 0;
        item_done();
        if (nn == 0) continue;
        if (dual) {
          // Both halves' scores are computed two blocks ahead: they take half of the tile's columns each time, so block
          // j + 1 need not wait for the softmax of block j.
          for (int j = 0; j < 2 && j < nn && ok; ++j) {
            ok = wait(FULL + stage, phase);
            if (ok && j == 0) {
              ok = wait(QFULL, qp0) && wait(QFULL + 1, qp1);
              qp0 ^= 1u;
              qp1 ^= 1u;
            }
            if (!ok) break;
            qk(0, stage, j);
            qk(1, stage, j);
            if (leader) {
              tc_commit(bar(EMPTY + stage));
              if (j + 1 == nn) {
                tc_commit(bar(QEMPTY));
                tc_commit(bar(QEMPTY + 1));
              }
            }
            next();
          }
          for (int j = 0; j < nn && ok; ++j) {
            const int b2 = j & 1;
            ok = wait3(FULL + stage, phase, FULL + stage, phase, PFULL + 2 * b2, b2 ? pp0b : pp0);
            if (!ok) break;
            pv(0, stage, j > 0, b2);
            ok = wait(PFULL + 2 * b2 + 1, b2 ? pp1b : pp1);
            if (!ok) break;
            pv(1, stage, j > 0, b2);
            if (leader) tc_commit(bar(EMPTY + stage));
            next();
            if (b2) { pp0b ^= 1u; pp1b ^= 1u; } else { pp0 ^= 1u; pp1 ^= 1u; }
            if (j + 2 < nn) {
              ok = wait(FULL + stage, phase);
              if (!ok) break;
              qk(0, stage, b2);
              qk(1, stage, b2);
              if (leader) {
                tc_commit(bar(EMPTY + stage));
                if (j + 3 == nn) {
                  tc_commit(bar(QEMPTY));
                  tc_commit(bar(QEMPTY + 1));
                }
              }
              next();
            }
          }
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
            if (leader) tc_commit(bar(EMPTY + vs));  // (before QK: the block that takes its place has longer to come)
            if (j + 1 < n1) qk(1, ks);
            if (leader && j + 2 == n1) tc_commit(bar(QEMPTY + 1));
          } else if (ok && leader) {
            tc_commit(bar(EMPTY + vs));
          }
          if (leader && j + 1 < nn) tc_commit(bar(EMPTY + ks));
        }
      }
      // every MMA has completed before TMEM and shared memory go away
      if (leader) tc_commit(bar(DONE));
      mbar_wait_bounded(bar(DONE), 0, timeout_ns);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2, r = tid & 127;  // tile, row of it
    const int q4 = warp & 3;                 // TMEM lanes 32 q4 ..
    const float c2 = pa.scale * 1.4426950408889634f;
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
      // Where the thread's row lies. (It is found again after the loop, which has no registers to keep it in.)
      bool dual, valid;
      int tile0, nrow_t, tok, h;
      auto place = [&]() {
        int g = G;
        asm volatile("" : "+r"(g));
        dual = it->dual;
        tile0 = dual ? 0 : t * TM;               // the tile's first row of the item's
        nrow_t = min(TM, it->nrows - tile0);     // rows of this tile (<= 0: none)
        const int R = it->row0 + tile0 + r;
        valid = r < nrow_t;
        tok = valid ? R / g : 0;
        h = it->hk * g + (valid ? R % g : 0);
      };
      place();
      const int n = blocks(t ? it->lim1 : it->lim0);
      // (What a row past the tile's end makes of whatever lies there is dropped, so these are not masked: a tile of a
      // single token's heads would go through the masking below in every block, 1.15 us a block against 0.95.)
      int lim = 0x7fffffff;
      if (valid) lim = max(0, min(visible_keys(tok, it->nq, it->nk, pa.causal) - it->key0, it->n_keys));
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
        for (int i = 0; i < 16 * NC; ++i) {
          const uint32_t* v = &s[i >> 4][2 * (i & 15)];
          mx4[i & 3] = max3(mx4[i & 3], __uint_as_float(v[0]), __uint_as_float(v[1]));
        }
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
          // Once this block's weights are given the barrier may go on by two phases, whose parities would look alike, so
          // the PV before (in flight for one softmax by now) is waited for first.
          ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
          if (!ok) return;
        }
        if (lane == 0) mbar_arrive(bar(PFULL + 2 * b2 + t));
        const uint64_t sum = fadd2(sum0, sum1);
        l += f2_lo(sum) + f2_hi(sum);
      };
      const bool halves = dual;
      for (int j = 0; j < n && ok; ++j) {
        if (halves) block(std::integral_constant<int, BK / 2>{}, j);
        else block(std::integral_constant<int, BK>{}, j);
        done += ok ? 1 : 0;
      }
      // ---- the rows' results
      if (ok && n > 0) {
        ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
        tc_fence_after();
      }
      place();
      if (ok && nrow_t > 0 && __any_sync(0xffffffffu, valid)) {
        const bool part = it->piece >= 0;  // a piece: the sums in fp32; a whole item: the results in bf16
        float f0 = 1.f, f1 = 0.f;          // factors of a tile's sums; of tile 0's and tile 1's
        if (dual) {
          // The tiles are the halves of the keys: of the two warps that share TMEM lanes each adds up half of the columns.
          given_ml[tid] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(GIVEN + q4));
          ok = warp_wait(bar(GIVEN + q4), given & 1, timeout_ns, abort_flag, status, 56);
          tc_fence_after();
          const float2 a = given_ml[r], b = given_ml[TM + r];
          m = fmaxf(a.x, b.x);
          f0 = a.x == -INFINITY ? 0.f : ex2((a.x - m) * c2);
          f1 = b.x == -INFINITY ? 0.f : ex2((b.x - m) * c2);
          l = a.y * f0 + b.y * f1;
        }
        const float f = part ? 1.f : l == 0.f ? 0.f : 1.0f / l;
        const uint64_t f0p = f2_pack(f0 * f, f0 * f), f1p = f2_pack(f1 * f, f1 * f);
        const long long at = part ? ((long long)it->piece + tile0 + r) * D
                                  : (long long)(it->q0 + tok) * pa.os + (long long)h * D;
        uint8_t* orow = part ? reinterpret_cast<uint8_t*>(ca.part_o + at) : (uint8_t*)pa.out + 2 * at;
        // 32 bytes a store: whole sectors, though each lane stores to a row of its own
        const bool wide = part || (((uint32_t)(uintptr_t)pa.out | (uint32_t)pa.os * 2 | (uint32_t)D * 2) & 31) == 0;
        uint64_t odd = 0ull;  // (times 0 and added up, only a value that is not finite leaves something else than 0)
        // 32 columns from `col` on
        auto emit = [&](uint32_t(&o)[32], int col) {
          if (part) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (valid && col + 8 * i < D) store_32(orow + 4 * (col + 8 * i), o + 8 * i);
            return;
          }
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          if (wide) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (valid && col + 16 * i < D) store_32(orow + 2 * (col + 16 * i), p + 8 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (valid && col + 8 * i < D)
                *reinterpret_cast<uint4*>(orow + 2 * (col + 8 * i)) =
                    make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
          }
        };
        // (64 columns of a tile or 32 of two a step; what is not in the instruction cache costs more than the loop)
        const uint32_t tA = tmem + lanes + 256 + (dual ? 0 : t * DP), tB = dual ? tA + DP : tA + 32;
        const int step = dual ? 32 : 64, col1 = dual ? (t + 1) * (DP / 2) : DP;
#pragma unroll 1
        for (int col = dual ? t * (DP / 2) : 0; col < col1; col += step) {
          uint32_t o[32], x[32];
          tmem_ld_32x32b_x32(tA + col, o);  // (not this item's where there was no block: lim is 0 then)
          tmem_ld_32x32b_x32(tB + col, x);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint64_t v = ffma2(((uint64_t)o[2 * i + 1] << 32) | o[2 * i], f0p, 0ull);
            uint64_t w = ((uint64_t)x[2 * i + 1] << 32) | x[2 * i];
            if (dual) {
              v = ffma2(w, f1p, v);
            } else {
              w = ffma2(w, f0p, 0ull);
            }
            if (lim == 0) v = w = 0ull;
            odd = ffma2(v, 0ull, odd);
            if (!dual) odd = ffma2(w, 0ull, odd);
            o[2 * i] = (uint32_t)v;
            o[2 * i + 1] = (uint32_t)(v >> 32);
            x[2 * i] = (uint32_t)w;
            x[2 * i + 1] = (uint32_t)(w >> 32);
          }
          emit(o, col);
          if (!dual) emit(x, col + 32);
        }
        if (dual) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(TAKEN + q4));
          ok = ok && warp_wait(bar(TAKEN + q4), given & 1, timeout_ns, abort_flag, status, 56);
          ++given;
        }
        const bool first = !dual || t == 0;
        if (valid && first && part) ca.part_ml[it->piece + tile0 + r] = make_float2(m * c2, l);
        if (valid && first && !part && pa.lse != nullptr)
          pa.lse[(long long)(it->q0 + tok) * H + h] =
              lim == 0 ? -INFINITY : (m * c2 + log2f(l)) * 0.6931471805599453f;
        // Rows whose results are looked at again. (One whose weights' sum is not finite sees a score that is not, and is
        // NaN as a whole.)
        uint32_t again = __ballot_sync(0xffffffffu, valid && !(f2_lo(odd) + f2_hi(odd) == 0.f) && fabsf(l) <= 3.0e38f);
        if (again != 0) {
          Unseen unseen(min(n * BK, it->nk - it->key0));
          while (again != 0) {
            const int w = __ffs(again) - 1;
            again &= again - 1;
            const int tw = __shfl_sync(0xffffffffu, tok, w), hw = __shfl_sync(0xffffffffu, h, w);
            const float mw = __shfl_sync(0xffffffffu, m, w), lw = __shfl_sync(0xffffffffu, l, w);
            float o[8];
            const uint32_t cols = replace_unseen(
                unseen, (const __nv_bfloat16*)pa.q + (long long)(it->q0 + tw) * pa.qs + (long long)hw * D,
                (const __nv_bfloat16*)ca.d.k, (const __nv_bfloat16*)ca.d.v,
                [&](int j, long long& ko, long long& vo) {  // where key j of the item lies
                  const CacheView& cv = ca.d.c;
                  const int p = it->key0 + j;
                  int page = cv.table[(long long)it->k0 * cv.width + (p >> cv.page_shift)];
                  page = page < 0 || page >= cv.n_pages ? 0 : page;
                  ko = vo = (((long long)page * Hkv + it->hk) * cv.page_size + (p & (cv.page_size - 1))) * D;
                },
                D, __shfl_sync(0xffffffffu, lim, w), c2, mw == -INFINITY ? 0.f : mw * c2, o);
            float* po = ca.part_o + ((long long)it->piece + tile0 + 32 * q4 + w) * D + lane * 8;
            __nv_bfloat16* dw =
                (__nv_bfloat16*)pa.out + (long long)(it->q0 + tw) * pa.os + (long long)hw * D + lane * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((cols >> e & 1u) && (!dual || lane / (DP / 16) == t)) {  // (its own columns)
                if (part) po[e] = o[e];
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

// Rows r0 .. r0 + ROWS - 1 of a shared item by a warp: n pieces each, in order, NP of them on their way at a time. Its
// lanes lie in ROWS parts, one a row, to weight the pieces.
template <int ROWS, int NP>
__device__ __forceinline__ void join_rows(const PromptArgs& a, const ChunkArgs& ca, const ChunkRun& run, int kind, int c0,
                                          int n, int r0) {
  constexpr int P = 32 / ROWS;
  const int lane = threadIdx.x & 31, k = lane / P, y0 = lane % P, rows = min(ROWS, run.nrows - r0);
  // run c0 has its last item's piece, the others their first's
  auto at = [&](int i, int r) { return (long long)ca.piece(kind, c0 + i, i == 0) + r0 + r; };
  auto ml = [&](int i) { return i < n && k < rows ? ca.part_ml[at(i, k)] : make_float2(-INFINITY, 0.f); };
  float M = -INFINITY, l = 0.f;
  for (int i = y0; i < n; i += P) M = fmaxf(M, ml(i).x);
#pragma unroll
  for (int w = P / 2; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const float ref = M == -INFINITY ? 0.f : M;
  const bool on = lane * 4 < a.D;
  float4 o[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += P) {
    const float2 v = ml(i0 + y0);
    const float wl = ex2(v.x - ref);
    l += wl * v.y;
    for (int y = 0; y < P && i0 + y < n; y += NP) {
      float4 u[NP][ROWS];
#pragma unroll
      for (int b = 0; b < NP; ++b)
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          u[b][r] = on && r < rows && i0 + y + b < n
                        ? reinterpret_cast<const float4*>(ca.part_o + at(i0 + y + b, r) * a.D)[lane]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int b = 0; b < NP; ++b)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float w = __shfl_sync(0xffffffffu, wl, P * r + y + b);
          o[r].x = fmaf(w, u[b][r].x, o[r].x);
          o[r].y = fmaf(w, u[b][r].y, o[r].y);
          o[r].z = fmaf(w, u[b][r].z, o[r].z);
          o[r].w = fmaf(w, u[b][r].w, o[r].w);
        }
    }
  }
#pragma unroll
  for (int w = P / 2; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int G = a.H / a.Hkv, R0 = run.row0 + r0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float f = __shfl_sync(0xffffffffu, inv, P * r);
    if (r >= rows || !on) continue;
    const int tok = run.q0 + (R0 + r) / G, h = run.hk * G + (R0 + r) % G;
    uint2 u;
    u.x = pack_bf16x2(o[r].x * f, o[r].y * f);
    u.y = pack_bf16x2(o[r].z * f, o[r].w * f);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + (long long)tok * a.os + (long long)h * a.D + lane * 4) = u;
  }
  if (a.lse != nullptr && y0 == 0 && k < rows) {
    const int tok = run.q0 + (R0 + k) / G, h = run.hk * G + (R0 + k) % G;
    a.lse[(long long)tok * a.H + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
  }
}

// The rows that several runs share, by the run that such an item begins in (blockIdx.x, either kind), 32 a CTA. Two or
// three pieces, as most have: a warp takes four rows, whose loads go out together (a warp a row: 130 us a call of 4
// sequences' 2048 tokens behind 8192, 122 so). Many, of a long sequence's few rows: a warp a row (one token behind 4096,
// 8 rows a head: 20 us a call, 29 with four rows a warp).
constexpr int kJoinRows = 32;

__global__ void __launch_bounds__(256, 4)
chunk_join_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ ChunkArgs ca) {
  griddep_wait();
  griddep_launch_dependents();
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, first = blockIdx.y * kJoinRows;
  const bool some[2] = {ca.runs[c0].nrows > 0, ca.runs[ca.ctas + c0].nrows > 0};
#pragma unroll 1  // (the code comes from memory: 1 us of a small call)
  for (int kind = some[0] ? 0 : 1; kind < (some[1] ? 2 : 1); ++kind) {
    const ChunkRun run = ca.runs[kind * ca.ctas + c0];
    const int n = run.end - c0 + 1, end = min(run.nrows, first + kJoinRows);
    if (n <= 4) {
      if (first + 4 * warp < end) join_rows<4, 2>(a, ca, run, kind, c0, n, first + 4 * warp);
    } else {
      for (int r = first + warp; r < end; r += 8) join_rows<1, 8>(a, ca, run, kind, c0, n, r);
    }
  }
}

template <int DP>
cudaError_t launch(const CUtensorMap& tq, const CacheMaps& m, const PromptArgs& pa, const ChunkArgs& ca, int ctas,
                   int slots, int q_tma, cudaStream_t s) {
  static std::atomic<int> done{0};
  auto kern = attn_chunk_kernel<DP>;
  const cudaError_t e = allow_smem(kern, Cfg<DP>::kSmem, done);
  if (e != cudaSuccess) return e;
  // Not as a programmatic dependent: its CTAs would then take the SMs in the order in which the kernel before leaves
  // them, and CTAs with neighbouring runs, which read the same keys, would lie anywhere on the two dies. 64 sequences of
  // single tokens and chunks back to back: 1045 us so, 865 us in the usual order.
  kern<<<dim3(ctas), dim3(kThreads), Cfg<DP>::kSmem, s>>>(tq, m.k128, m.v128, pa, ca, slots, q_tma);
  return cudaGetLastError();
}

}  // namespace

namespace {

// Rows of a piece of either kind: no more than a call's rows of a head.
int piece_rows(int kind, int Tq, int G) {
  const long long rows = (long long)Tq * G;
  return (int)(kind == 0 ? (rows <= TM ? 0 : rows < 2 * TM ? rows : 2 * TM) : (rows < TM ? rows : TM));
}
size_t runs_bytes(int ctas) { return ((sizeof(ChunkRun) * 2 * (size_t)ctas + 255) & ~(size_t)255); }

}  // namespace

size_t chunk_tc_bytes(int Tq, int G, int D) {
  const int ctas = device_sm_count();
  const size_t rows = 2 * (size_t)ctas * (piece_rows(0, Tq, G) + piece_rows(1, Tq, G));
  return 256 + runs_bytes(ctas) + rows * (D + 2) * 4;  // (256: the workspace begins at any multiple of 16)
}

cudaError_t launch_attn_chunk_tc(const PromptArgs& a, const DecodeArgs& d, const CacheMaps& m, void* scratch,
                                 cudaStream_t s) {
  EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap tq{};
  const int G = a.H / a.Hkv;
  int q_tma = 0;
  if (enc == nullptr || !encode_q(enc, &tq, a.q, a.D, a.H, G, a.Tq, a.qs, &q_tma)) return cudaErrorInvalidValue;
  const int slots = (int)prompt_tile_slots(a.Tq, a.n, G, 2 * TM);
  // one CTA an SM, as far as the longest sequences that the cache may hold make as many runs
  const long long longest = chunk::kItem + ((long long)d.c.width * d.c.page_size + BK - 1) / BK * chunk::kBlock;
  const long long runs_most = a.Hkv * (long long)slots * longest / chunk::kShortest;
  const int ctas = (int)(runs_most < 1 ? 1 : (runs_most < device_sm_count() ? runs_most : device_sm_count()));
  ChunkArgs ca{};
  ca.d = d;
  ca.ctas = ctas;
  uint8_t* at = reinterpret_cast<uint8_t*>(((uintptr_t)scratch + 255) & ~(uintptr_t)255);
  ca.runs = reinterpret_cast<ChunkRun*>(at);
  ca.part_o = reinterpret_cast<float*>(at + runs_bytes(ctas));
  long long rows = 0;
  for (int k = 0; k < 2; ++k) rows += 2LL * ctas * (ca.rows[k] = piece_rows(k, a.Tq, G));
  ca.part_ml = reinterpret_cast<float2*>(ca.part_o + rows * a.D);
  const cudaError_t e = a.D <= 64 ? launch<64>(tq, m, a, ca, ctas, slots, q_tma, s)
                                  : launch<128>(tq, m, a, ca, ctas, slots, q_tma, s);
  if (e != cudaSuccess) return e;
  const int most = ca.rows[0] > ca.rows[1] ? ca.rows[0] : ca.rows[1];
  return launch_pdl(chunk_join_kernel, dim3((unsigned)ctas, (unsigned)((most + kJoinRows - 1) / kJoinRows)), dim3(256),
                    0, s, a, ca);
}

}  // namespace moe

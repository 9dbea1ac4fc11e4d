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
#include "attn_tc.cuh"

namespace moe {
namespace {

struct __align__(16) Item {
  int hk, row0, nrows;      // key/value head; packed rows row0 .. of the sequence (or batch)
  int q0, nq, k0, nk;       // the sequence
  int key0, n_keys;         // keys of the item
  int lim0, lim1;           // keys that each tile's last row sees (relative to key0)
  int last;                 // no item: the end
  int split;                // which part of the keys
};
constexpr int kItems = 3;   // items published: one worked on, one ahead, one being given back
constexpr int kItemReaders = 1 + 8 + 2;

template <int DP> struct Cfg {
  static constexpr int kChunks = DP / 64;          // 64-element (128-byte) swizzle columns of a row
  static constexpr int kTileBytes = TM * DP * 2;   // a Q tile, and a K or V block
  static constexpr int kStages = DP == 128 ? 4 : 8;
  static constexpr int kStage = 32 * 128;  // bytes of a softmax warp's output staging: 32 rows x 64 bf16 elements
  static constexpr int kBars = 2 * kStages + 5 * 2 + 1 + 2 * kItems;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kStages) * kTileBytes + 8 * kStage + 8 * kBars + 16 + kItems * sizeof(Item);
};
static_assert(Cfg<128>::kSmem <= kMaxSmem && Cfg<64>::kSmem <= kMaxSmem, "shared memory");

struct SharedArgs {
  DecodeArgs d;
  int per;        // keys of a split, a multiple of BK (decode)
  int splits;     // pieces of a row
  float* part_o;  // [piece][D]
  float2* part_ml;
};

// SHARED = false: items are tile-pair slots (descending, so that the longest rows of a sequence start first) x
// key/value heads, n_items of them. SHARED = true: one item a CTA, blockIdx = (key/value head, row pair, split of
// the shared keys); rows are (sequence, head) pairs, and each row's piece goes to the workspace unnormalised. SPLIT
// (prompts of few rows): every item's keys in sa.splits parts, an item each, and the rows' pieces likewise.
template <int DP, bool SHARED, bool SPLIT>
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int FULL = 0, EMPTY = C::kStages, QFULL = 2 * C::kStages, SFULL = QFULL + 2, PFULL = SFULL + 2,
                ODONE = PFULL + 2, QEMPTY = ODONE + 2, DONE = QEMPTY + 2, IFULL = DONE + 1, IEMPTY = IFULL + kItems;

  // (the shuffle tells the compiler that the warp number is the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(bar(FULL + s), 1); mbar_init(bar(EMPTY + s), 1); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(QFULL + t), 1);
      mbar_init(bar(SFULL + t), 1);
      mbar_init(bar(PFULL + t), 4);
      mbar_init(bar(ODONE + t), 1);
      mbar_init(bar(QEMPTY + t), 1);
    }
    for (int i = 0; i < kItems; ++i) { mbar_init(bar(IFULL + i), 1); mbar_init(bar(IEMPTY + i), kItemReaders); }
    mbar_init(bar(DONE), 1);
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

  if (warp >= kSoftWarps) {
    // 8 * 32 * 232 + 4 * 32 * 40 = 64512, as at the launch.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kSoftWarps + 1) {
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
      while (const Item* ip = next_item()) {
        const Item it = *ip;
        item_done();
        if ((t ? it.lim1 : it.lim0) == 0) continue;
        if (!warp_wait(bar(QEMPTY + t), (loads & 1u) ^ 1u, timeout_ns, abort_flag, status, 55)) break;
        ++loads;
        if (q_tma) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(QFULL + t), C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(sQ + t * C::kTileBytes + c * (TM * 128), &tmQ, 64 * c, it.hk * G, it.q0 + (it.row0 + t * TM) / G,
                          bar(QFULL + t));
          }
          continue;
        }
        const int nrow_t = min(TM, it.nrows - t * TM);
        const __nv_bfloat16* q = (const __nv_bfloat16*)(SHARED ? sa.d.q : pa.q) + (long long)(SHARED ? 0 : it.q0) * (SHARED ? sa.d.qs : pa.qs);
#pragma unroll
        for (int k = 0; k < TM / 32; ++k) {
          const int R = it.row0 + t * TM + 32 * k + lane, tok = R / G;  // (rows past the end are not read)
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
      uint32_t pp0 = 0, pp1 = 0, qp0 = 0, qp1 = 0;  // phases of the tiles' P and Q barriers
      bool ok = true;
      while (ok) {
        const Item* it = next_item();
        if (it == nullptr) break;
        const int n0 = __shfl_sync(0xffffffffu, blocks(it->lim0), 0), n1 = __shfl_sync(0xffffffffu, blocks(it->lim1), 0);
        const int nn = max(n0, n1);
        item_done();
        if (nn == 0) continue;
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
    uint32_t done = 0;  // blocks of all items so far: their barriers' phases
    bool ok = true;
    while (ok) {
      const Item* it = next_item();
      if (it == nullptr) break;
      const int nrow_t = min(TM, it->nrows - t * TM);  // rows of this tile (<= 0: none)
      const int n = blocks(t ? it->lim1 : it->lim0);
      const int R = it->row0 + t * TM + r;
      const bool valid = r < nrow_t;
      const int tok = valid ? R / G : 0, h = it->hk * G + (valid ? R % G : 0);
      int lim = 0;
      if (valid && SHARED) {  // a slot shorter than the shared keys sees its own length of them
        lim = max(0, min(it->n_keys, slot_len(sa.d.c, sa.d.slots[tok]) - it->key0));
      } else if (valid) {
        lim = visible_keys(tok, it->nq, it->nk, pa.causal);
        if (SPLIT) lim = max(0, min(lim - it->key0, it->n_keys));
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++done) {
        ok = warp_wait(bar(SFULL + t), done & 1, timeout_ns, abort_flag, status, 53);
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
            ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
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
        ok = warp_wait(bar(ODONE + t), (done - 1) & 1, timeout_ns, abort_flag, status, 53);
        tc_fence_after();
      }
      if (ok && nrow_t > 0 && __any_sync(0xffffffffu, valid)) {
        if (SHARED || SPLIT) {
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
          uint32_t again = __ballot_sync(0xffffffffu, valid && !fine && fabsf(l) <= 3.0e38f);
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
          uint32_t again = __ballot_sync(0xffffffffu, valid && !(f2_lo(odd) + f2_hi(odd) == 0.f) && fabsf(l) <= 3.0e38f);
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

template <int DP, bool SHARED, bool SPLIT>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PromptArgs& pa,
                   const SharedArgs& sa, dim3 grid, int n_items, int q_tma, cudaStream_t s) {
  static std::atomic<int> done{0};
  auto kern = attn_tc_kernel<DP, SHARED, SPLIT>;
  const cudaError_t e = allow_smem(kern, Cfg<DP>::kSmem, done);
  if (e != cudaSuccess) return e;
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

}  // namespace moe

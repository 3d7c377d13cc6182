// Packed prompt attention, forward: softmax(scale Q K^T + mask) V on tcgen05.
//
// An item: up to two tiles of 128 packed query rows against the key blocks b1 - 1 ..
// b0 of one key head, the masked diagonal first. One pass with a running maximum and sum per row:
//   S = Q K_j^T (M = N = 128, K = d)          -> TMEM, one buffer per tile
//   m' = max(m, rowmax S), P = 2^(c S - c m'), l = l 2^(c m - c m') + rowsum P
//   O = O 2^(c m - c m') + P V_j (M = 128, N = d, K = 128; P bf16 in TMEM, over S)
// with c = scale log2 e. m is raised only when a row's maximum passed it by more
// than 8 in the exponent: P stays below 2^8, which costs no accuracy in bf16 or
// float32, and O is rescaled a few times per item instead of once per block.
// Statistics, sums and O are float32; P is rounded to bf16 for the product (the
// tensor cores take no wider A with a bf16 B), l adds the unrounded P.
//
// Roles: warps 0-3 own the rows of tile 0 (thread = row = TMEM lane), with two tiles
// warps 4-7 those of tile 1; the next warp loads (TMA), the one behind it issues the
// MMAs. The tensor cores run S and P V of one tile while the other tile's warps form
// its softmax; with one tile a second CTA on the SM fills the gaps.
// One CTA with two tiles fills an SM, so nothing would hide its start and its end (7.5
// us, four steps): it takes over the item of a block that has not started, and loads its
// queries and first keys while this one's last steps run. Measured: 6 sequences of 310 to
// 8191 tokens, 32 / 8 heads of 128, 604 us (with a block per item 670); 16 of 1000
// tokens, 16 / 4 heads of 64, 74 us (86).
// (Figures in this file: the same inputs call after call, 60 ms at a time, other GPUs up to
// 4 % off. In long runs on changing inputs the power limit sets a lower clock: 685 to 705 us
// for the first of these.)
// Every wait is bounded; the kernel drains its copies and MMAs before it ends.
//
// Bound: at d = 128 the tensor cores under the power limit (32768 causal tokens, 12
// heads: 2500 us at 1.49 GHz, 1.32 PFLOP/s, 80 % of cuBLAS's burst rate; in a long run 2840 us,
// 1.16 PFLOP/s, 83 % of its sustained one); at d = 64 no unit by itself (16384 causal
// tokens, 16 heads: 650 us; of 8192, special function units 55 %, issue slots 50 %, tensor pipe
// 35 %): a scheduler has two softmax warps, and each waits for its own S, maximum and
// exponentials in turn; with 32 rows or fewer the keys' bytes (single tokens over caches:
// 5.4 TB/s in the kernel).
#include <string.h>

#include "prompt_tc.cuh"

namespace sla {

using namespace tc;

struct PromptMaps {
  CUtensorMap q, k, v;
};

struct PromptDev {
  unsigned char* plan_dev;
  const PromptItem* items;
  const PromptJoin* joins;
  __nv_bfloat16* o;
  long long o_row, o_head;
  __nv_bfloat16* rest;
  float *lse, *part, *part_lse;
  int Hq, G, tpt, box, causal, tiles;  // box: tokens that a copy of Q brings
  long long Tq, Tk;
  int n_slots;
  float scale_log2;
};

namespace {


template <int D, int TILES, bool FEW>
struct FwdCfg {
  static constexpr int kSub = 128 * 128;             // 128 rows x 128 bytes (64 columns)
  static constexpr int kTileBytes = kSub * (D / 64);  // 128 x D bf16
  // Two tiles: one CTA per SM (8 softmax warps, loader, MMA issuer, two idle ones that
  // give up registers). One tile: two CTAs per SM, each with half the ring and TMEM.
  static constexpr int kSoft = 4 * TILES, kThreads = TILES == 2 ? 384 : 192;
  static constexpr int kCtas = TILES == 2 ? 1 : 2;
  // A CTA takes item after item, where it has the SM for itself. (In the other form the
  // softmax warps have no registers left for it: +6 % on 8192 tokens, 16 heads of 64.)
  static constexpr bool kAgain = TILES == 2;
  // FEW: no item has more than 32 rows (single tokens over caches): Q takes 32 rows of
  // shared memory and the ring one tile more, for the loads are what counts. The products
  // read 96 more rows from what follows, which reach only the TMEM lanes of rows that are not there.
  static constexpr int kQSub = FEW ? 32 * 128 : kSub;  // 64 columns of Q
  static constexpr int kStages = D == 128 ? (TILES == 2 ? 4 : FEW ? 3 : 2) : (TILES == 2 ? 8 : FEW ? 6 : 5);
  static constexpr int oQ = 0;
  static constexpr int oKV = TILES * kQSub * (D / 64);
  static constexpr int kBytes = oKV + kStages * kTileBytes;
  static constexpr int kSmem = kBytes + 1024;
  // Of every 8 pairs of exponents, this many are formed on the FMA units: the special
  // function units take 1024 clocks for a tile's exponentials, its products take 512
  // (d = 64) or 1024 (d = 128). Measured, 16384 causal tokens, 16 heads, d = 64: none
  // 711 us, one pair 675, two 650, three 665; 8192 full ones (one tile): 372, 377, 358, 358.
  // At d = 128 (32768 tokens, 12 heads) the power limit sets the clock: none 2530 us, two 2560.
  static constexpr int kFmaPairs = D == 64 ? 2 : 0;
  // In what way they treat NaN: one tile's warps feel the operation that keeping it costs
  // (8192 full tokens, 16 heads: 372 us, and 357 without), those of two do not (16384 causal
  // ones: 651, and 660). NaN scores make the row's maximum NaN and so the other columns; a row
  // with an infinite one alone is made NaN at its end.
  static constexpr bool kNan = TILES == 2;
  // TMEM columns: S of every tile (128 each), O of every tile (D each).
  // P takes the first 64 columns of its S at d = 128, where TMEM is full: the next S
  // waits for P V. At d = 64 it has columns of its own, so the next S is formed as soon
  // as the last one has been read, and the softmax warps never wait for products.
  static constexpr int kCols = 256 * TILES;
  static constexpr int cO = 128 * TILES;
  static constexpr bool kApart = D == 64;
  static constexpr int cP = kApart ? 192 * TILES : 0, kPStep = kApart ? 64 : 128;
};

// Per tile: Q loaded and released, S done, P's halves written, S read, P V done. Then
// the next item asked for, and two slots for it (filled, read), and the ring's stages.
enum {
  bQ0 = 0, bQ1, bE0, bE1, bS0, bS1, bO0, bO1, bDone, bNext, bJobF0, bJobF1,
  bP0, bP1, bR0, bR1, bX0, bX1,  // 128 arrivals
  bJobE0, bJobE1,
  bKV  // then full / empty of every stage
};

// What every role knows of an item.
struct Work {
  PromptItem it;
  int nb0, nb1, bmax, n;  // key blocks of tile t: [b0, nb_t); n: steps
};

}  // namespace

template <int D, int TILES, bool FEW>
__global__ void __launch_bounds__(FwdCfg<D, TILES, FEW>::kThreads, FwdCfg<D, TILES, FEW>::kCtas)
    prompt_fwd_kernel(const __grid_constant__ PromptMaps maps, const PromptDev a) {
  using C = FwdCfg<D, TILES, FEW>;
  constexpr int ST = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[bKV + 2 * ST];
  __shared__ __align__(16) uint4 next_sh;      // the hardware's answer: another block's index, or none
  __shared__ __align__(16) PromptItem first_sh, job_sh[2];  // the first item, those that follow (nq = 0: none)
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = reinterpret_cast<int*>(a.plan_dev);
  auto sound = [&](const PromptItem& it) {  // (heads fit 16 bits)
    return it.q0 >= 0 && it.nq >= 1 && it.k0 >= 0 && it.lk >= 0 && it.q0 + (long long)it.nq <= a.Tq &&
           it.k0 + (long long)it.lk <= a.Tk && it.nq <= TILES * a.tpt && (!FEW || it.nq <= a.box) && it.b0 >= 0 &&
           uint32_t(it.head) < 65536u && it.head * a.G < a.Hq && it.slot < a.n_slots;
  };
  auto work_of = [&](const PromptItem& it) {
    auto end_block = [&](int t) {
      const int last = min(it.nq, (t + 1) * a.tpt) - 1;
      if (last < t * a.tpt) return it.b0;
      const long long keys = a.causal ? min((long long)it.lk, (long long)it.pos0 + last + 1) : it.lk;
      return max(it.b0, min(it.b1, int((max(keys, 0LL) + 127) / 128)));
    };
    Work w{it, end_block(0), TILES == 2 ? end_block(1) : it.b0, 0, 0};
    w.bmax = max(w.nb0, w.nb1);
    w.n = w.bmax - it.b0;
    return w;
  };
  Work w{};
  w.it = a.items[blockIdx.x];
  if (!sound(w.it)) {
    if (threadIdx.x == 0) atomicExch(status, kDevBadIndex);
    return;
  }
  w = work_of(w.it);

  volatile int* abort_flag = &abort_sh;
  auto bar = [&](int b) { return smem_u32(&bars[b]); };
  auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, status); };
  auto wait_w = [&](int b, uint32_t parity) {
    const bool ok = wait(b, parity);
    __syncwarp();
    return ok;
  };
  int no_abort = 0;
  auto wait_drain = [&](int b, uint32_t parity) {
    return mbar_wait(bar(b), parity, reinterpret_cast<volatile int*>(&no_abort), status);
  };
  const uint32_t sb = smem_u32(smem);

  // Ring positions count on from item to item; in an item's own order they are K0, K1, V0,
  // K2, V1, ... - the next step's keys before this step's values.
  auto full = [&](uint32_t i) { return bKV + int(i % ST); };
  auto empty = [&](uint32_t i) { return bKV + ST + int(i % ST); };
  auto phase = [&](uint32_t i) { return (i / ST) & 1; };
  auto k_pos = [&](int s) { return s == 0 ? 0 : 2 * s - 1; };
  auto v_pos = [&](int s, int n) { return min(2 * s + 2, 2 * n - 1); };
  auto load = [&](const Work& w, uint32_t ring, int i) {
    const bool keys = i == 0 || ((i & 1) && i < 2 * w.n - 1);
    const int b = w.bmax - 1 - (keys ? (i + 1) / 2 : i == 2 * w.n - 1 ? w.n - 1 : i / 2 - 1);
    const CUtensorMap* m = keys ? &maps.k : &maps.v;
    mbar_expect_tx(bar(full(ring + i)), C::kTileBytes);
    for (int s = 0; s < D / 64; ++s)
      tma_load_3d(sb + C::oKV + ((ring + i) % ST) * C::kTileBytes + s * C::kSub, m, bar(full(ring + i)), s * 64,
                  w.it.k0 + b * 128, w.it.head);
  };
  auto load_q = [&](const Work& w, int t) {
    mbar_expect_tx(bar(bQ0 + t), a.G * a.box * D * 2);
    for (int s = 0; s < D / 64; ++s)
      tma_load_4d(sb + C::oQ + t * C::kTileBytes + s * C::kQSub, &maps.q, bar(bQ0 + t), s * 64, 0,
                  w.it.q0 + t * a.tpt, w.it.head);
  };
  auto active = [&](const Work& w, int t) { return (t == 0 ? w.nb0 : w.nb1) > w.it.b0; };
  // The item behind job number `job`: false when there is none.
  auto await_job = [&](int job, int n) {
    // (a tile without keys waits here for the other one's n steps: 16384 clocks more for each)
    const bool ok = mbar_wait_for(bar(bJobF0 + (job & 1)), (job >> 1) & 1, abort_flag, status,
                                  kWaitCycles + 16384LL * n);
    __syncwarp();
    return ok && job_sh[job & 1].nq != 0;
  };
  auto release_job = [&](int job) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bJobE0 + (job & 1)));
  };
  int issued = 0;  // ring positions of the first item that are on their way
  if (warp == C::kSoft) {
    // the loader sets the barriers up and starts the first copies before the block meets
    for (int i = lane; i < bKV + 2 * ST; i += 32)
      mbar_init(bar(i), i >= bP0 && i <= bX1 ? 128 : i == bJobE0 || i == bJobE1 ? C::kSoft + 1 : 1);
    fence_barrier_init();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      abort_sh = 0;
      if (C::kAgain) first_sh = w.it;
      for (int t = 0; t < TILES; ++t) {
        if (!active(w, t)) continue;
        load_q(w, t);
        if (issued == 0) load(w, 0, issued++);  // the first keys right behind the first queries
      }
      for (; issued < min(2 * w.n, ST); ++issued) load(w, 0, issued);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");  // the join's launch runs behind this kernel
  if (warp == C::kSoft + 1) tmem_alloc(smem_u32(&tmem_base_sh), C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base_sh;

  if (warp == C::kSoft) {
    if (TILES == 2) reg_dec<40>();
    if (lane == 0) {
      uint32_t ring = 0, last = 0;  // position of the item's first tile; positions on their way
      uint32_t nq[2] = {0, 0};      // queries loaded, per tile
      for (int job = 0;; ++job) {
        // Asks the hardware for the next block that has not started, when the item's last tile
        // is due: its answer comes while the ring's tiles are worked on. (Blocks are handed out
        // in order, the longest items first, so an early question would take them from an SM
        // that is done sooner; what nobody asks for starts as a block of its own.)
        auto ask = [&]() {
          if (!C::kAgain) return;
          if (job > 0) fence_async_smem();
          ask_block(&next_sh, bar(bNext));
        };
        bool asked = false, ok = true;
        for (int t = 0; t < TILES; ++t) {
          if (!active(w, t)) continue;
          if (job > 0) {
            ok = ok && (nq[t] == 0 || wait(bE0 + t, (nq[t] - 1) & 1));
            if (!ok) break;
            load_q(w, t);
          }
          ++nq[t];
        }
        for (int i = issued; ok && i < 2 * w.n; ++i) {
          if (i == 2 * w.n - 2) ask(), asked = true;
          ok = wait(empty(ring + i), phase(ring + i) ^ 1);
          if (!ok) break;
          issued = i + 1;
          load(w, ring, i);
        }
        last = ring + issued;
        ring += 2 * w.n;
        issued = 0;
        if (!asked) ask();
        if (!C::kAgain) break;
        // the answer, and the item, for everyone
        if (!wait_drain(bNext, job & 1)) break;
        const int block = answered_block(&next_sh);
        PromptItem it{};
        if (block >= 0 && ok) {
          it = a.items[block];
          if (!sound(it)) {
            atomicExch(status, kDevBadIndex);
            it.nq = 0;
          }
        }
        if (job > 1 && !wait(bJobE0 + (job & 1), ((job >> 1) - 1) & 1)) break;
        job_sh[job & 1] = it;
        mbar_arrive(bar(bJobF0 + (job & 1)));
        if (it.nq == 0 || !ok) break;
        w = work_of(it);
      }
      // every copy has landed before the CTA can end
      for (int t = 0; t < TILES; ++t)
        if (nq[t] > 0) wait_drain(bQ0 + t, (nq[t] - 1) & 1);
      for (uint32_t i = last > ST ? last - ST : 0; i < last; ++i) wait_drain(full(i), phase(i));
    }
    __syncwarp();
  } else if (warp == C::kSoft + 1) {
    if (TILES == 2) reg_dec<40>();
    constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
    uint32_t ring = 0;
    int done[2] = {0, 0}, items[2] = {0, 0};  // steps and items behind this one, per tile
    for (int job = 0;; ++job) {
      const int n = w.n;
      const int off[2] = {w.bmax - w.nb0, w.bmax - w.nb1};  // first step of each tile (n: none)
      auto issue_s = [&](int t, int s) {
        if (s == off[t]) wait_w(bQ0 + t, items[t] & 1);
        const uint32_t sq = sb + C::oQ + t * C::kTileBytes;
        const uint32_t sk = sb + C::oKV + ((ring + k_pos(s)) % ST) * C::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          mma_bf16(tb + t * 128, sdesc(sq + (k >> 2) * C::kQSub + (k & 3) * 32, 16, 1024),
                   sdesc(sk + (k >> 2) * C::kSub + (k & 3) * 32, 16, 1024), idS, k > 0);
        }
        mma_commit(bar(bS0 + t));
        if (s == n - 1) mma_commit(bar(bE0 + t));  // the item's last S: its queries may be replaced
      };
      auto have_k = [&](int s) {
        wait_w(full(ring + k_pos(s)), phase(ring + k_pos(s)));
        tc_fence_after();
      };
      if (n > 0) {
        have_k(0);
        for (int t = 0; t < TILES; ++t)
          if (off[t] == 0) issue_s(t, 0);
        mma_commit(bar(empty(ring)));
      }
      for (int s = 0; s < n; ++s) {
        const uint32_t iv = ring + v_pos(s, n);
        const uint32_t sv = sb + C::oKV + (iv % ST) * C::kTileBytes;
        auto have_v = [&]() {
          wait_w(full(iv), phase(iv));
          const int valid = w.it.lk - (w.bmax - 1 - s) * 128;
          if (valid < 128) {
            // the sequence ends inside this block: the rows behind it are another sequence's (0 x NaN is NaN)
            for (int x = valid * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
              for (int sub = 0; sub < D / 64; ++sub)
                *reinterpret_cast<uint4*>(smem + C::oKV + (iv % ST) * C::kTileBytes + sub * C::kSub + x * 16) =
                    make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
          }
        };
        auto issue_o = [&](int t) {
          const int i = s - off[t], at = done[t] + i;
          if (!C::kApart) {
            wait_w(bP0 + t, at & 1);
            tc_fence_after();
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k == (C::kApart ? 0 : 4)) {
              wait_w(bR0 + t, at & 1);
              tc_fence_after();
            }
            mma_bf16_ts(tb + C::cO + t * D, tb + C::cP + t * C::kPStep + k * 8, sdesc(sv + k * 2048, C::kSub, 1024),
                        idO, (i > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(bar(bO0 + t));
        };
        if (C::kApart) {
          if (s + 1 < n) {
            have_k(s + 1);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (s >= off[t]) {  // S of this step has been read
                wait_w(bX0 + t, (done[t] + s - off[t]) & 1);
                tc_fence_after();
              }
              if (s + 1 >= off[t]) issue_s(t, s + 1);
            }
            mma_commit(bar(empty(ring + k_pos(s + 1))));
          }
          have_v();
#pragma unroll
          for (int t = 0; t < TILES; ++t)
            if (s >= off[t]) issue_o(t);
        } else {
          have_v();
          bool have = false;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            if (s >= off[t]) issue_o(t);
            if (s + 1 < n && s + 1 >= off[t]) {
              if (!have) have_k(s + 1);
              have = true;
              issue_s(t, s + 1);
            }
          }
          if (s + 1 < n) mma_commit(bar(empty(ring + k_pos(s + 1))));
        }
        mma_commit(bar(empty(iv)));
      }
      ring += 2 * n;
#pragma unroll
      for (int t = 0; t < TILES; ++t)
        if (off[t] < n) {
          done[t] += n - off[t];
          ++items[t];
        }
      if (!C::kAgain || !await_job(job, n)) break;
      w = work_of(job_sh[job & 1]);
      release_job(job);
    }
    mma_commit(bar(bDone));
    wait_drain(bDone, 0);
    __syncwarp();
  } else if (warp < C::kSoft) {
    if (TILES == 2) reg_inc<232>();
    const int t = warp >> 2, r = threadIdx.x & 127;
    const uint32_t tq = tb + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t tS = tq + t * 128, tP = tq + C::cP + t * C::kPStep, tO = tq + C::cO + t * D;
    const float c = a.scale_log2;
    const float slack = 8.0f / c;
    const int tok = t * a.tpt + r / a.G, g = r - (r / a.G) * a.G;
    int done = 0;  // steps of the items before
    const PromptItem* cur = &first_sh;  // read again behind the steps, not held in registers over them
    for (int job = 0;; ++job) {
      if (C::kAgain) w = work_of(*cur);
      const PromptItem& it = w.it;
      const int nb = t == 0 ? w.nb0 : w.nb1, steps = nb - it.b0;
      const bool live = r < a.G * a.tpt && tok < it.nq;
      // keys 0 .. limit - 1 are seen
      const int limit = !live ? 0 : a.causal ? int(max(0LL, min((long long)it.lk, (long long)it.pos0 + tok + 1))) : it.lk;
      const int warp_limit = __reduce_min_sync(0xffffffffu, limit);
      float m = -INFINITY, l = 0.0f;
      const bool idle = !__any_sync(0xffffffffu, live);  // none of the warp's rows is there
      for (int i = 0; i < steps; ++i) {
        const int key0 = (nb - 1 - i) * 128;
        wait_w(bS0 + t, (done + i) & 1);
        tc_fence_after();
        if (idle) {  // whatever its P holds reaches no row that is
          if (C::kApart) {
            mbar_arrive(bar(bX0 + t));
            if (i > 0) wait_w(bO0 + t, (done + i - 1) & 1);  // not a block ahead of the other warps' P
          } else {
            mbar_arrive(bar(bP0 + t));
          }
          mbar_arrive(bar(bR0 + t));
          continue;
        }
        float s[128];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld32(tS + 32 * j, *reinterpret_cast<float(*)[32]>(&s[32 * j]));
        tmem_wait_ld();
        if (C::kApart) {
          tc_fence_before();
          mbar_arrive(bar(bX0 + t));
        }
        if (key0 + 128 > warp_limit) {
          const int seen = limit - key0;
#pragma unroll
          for (int j = 0; j < 128; ++j) s[j] = j < seen ? s[j] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < 124; j += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) mx[x] = max3_nan(mx[x], s[j + 2 * x], s[j + 2 * x + 1]);
        mx[0] = max3_nan(mx[0], s[124], s[125]);
        mx[1] = max3_nan(mx[1], s[126], s[127]);
        const float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        const bool raise = !(top <= m + slack);  // NaN raises: the row becomes NaN
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise && m != -INFINITY ? ex2((m - top) * c) : 1.0f;
          if (raise) m = top;
          l *= f;
          if (i > 0) {
            wait_w(bO0 + t, (done + i - 1) & 1);  // P V of the block before has been added
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
              float o[32];
              tmem_ld32(tO + j, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] *= f;
              tmem_st32(tO + j, o);
            }
            tmem_wait_st();
          }
        }
        if (C::kApart && i > 0) {  // P of the block before has been read
          wait_w(bO0 + t, (done + i - 1) & 1);
          tc_fence_after();
        }
        const float mc = m == -INFINITY ? 0.0f : -m * c;
        const uint64_t c2 = two(c, c), mc2 = two(mc, mc);
        uint64_t sum[4] = {two(l, 0.0f), 0, 0, 0};
        auto form = [&](int from, int to) {  // P = 2^(c s - c m), in place
#pragma unroll
          for (int j = from; j < to; j += 2) {
            const uint64_t x = fma2(two(s[j], s[j + 1]), c2, mc2);
            if ((j >> 1) % 8 >= 8 - C::kFmaPairs) {
              ex2_fma<C::kNan>(x, s[j], s[j + 1]);
            } else {
              untwo(x, s[j], s[j + 1]);
              s[j] = ex2(s[j]);
              s[j + 1] = ex2(s[j + 1]);
            }
            if (C::kApart) sum[(j >> 1) & 3] = add2(sum[(j >> 1) & 3], two(s[j], s[j + 1]));
          }
#pragma unroll
          for (int j = from; j < to; j += 32) {
            uint32_t p[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = pack_bf16(s[j + 2 * x], s[j + 2 * x + 1]);
            tmem_st16u(tP + j / 2, p);
          }
        };
        auto hand_over = [&](int b) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(b + t));
        };
        form(0, 64);
        if (!C::kApart) hand_over(bP0);  // half of P V runs while the other half of P is formed
        form(64, 128);
        hand_over(bR0);
        if (!C::kApart) {  // off the chain to the next product
#pragma unroll
          for (int j = 0; j < 128; j += 2) sum[(j >> 1) & 3] = add2(sum[(j >> 1) & 3], two(s[j], s[j + 1]));
        }
        float x, y;
        untwo(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
        l = x + y;
      }
      if (steps > 0) {
        wait_w(bO0 + t, (done + steps - 1) & 1);
        tc_fence_after();
      }
      if (!C::kNan && m == INFINITY) l = NAN;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const PromptItem& at = C::kAgain ? *cur : w.it;
      const int slot = at.slot;
      const long long token = (long long)at.q0 + tok;
      const int head = at.head * a.G + g;
      const size_t prow = size_t(max(slot, 0)) * (a.tiles * 128) + (t * 128 + r);
      __nv_bfloat16* orow = a.o + token * a.o_row + head * a.o_head;
      __nv_bfloat16* rest = a.rest ? a.rest + (token * a.Hq + head) * D : nullptr;
      float* part = a.part + prow * D;
#pragma unroll 1
      for (int j = 0; j < D; j += 32) {
        float o[32];
        if (steps > 0) {
          tmem_ld32(tO + j, o);
          tmem_wait_ld();
        }
        if (live) {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = l == 0.0f ? 0.0f : o[x] * inv;
          if (slot < 0) {
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              const uint4 v = make_uint4(pack_bf16(o[x], o[x + 1]), pack_bf16(o[x + 2], o[x + 3]),
                                         pack_bf16(o[x + 4], o[x + 5]), pack_bf16(o[x + 6], o[x + 7]));
              *reinterpret_cast<uint4*>(orow + j + x) = v;
              if (rest)
                *reinterpret_cast<uint4*>(rest + j + x) =
                    make_uint4(pack_rest(o[x], o[x + 1], v.x), pack_rest(o[x + 2], o[x + 3], v.y),
                               pack_rest(o[x + 4], o[x + 5], v.z), pack_rest(o[x + 6], o[x + 7], v.w));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; x += 4)
              *reinterpret_cast<float4*>(part + j + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
      }
      tc_fence_before();  // O has been read: the next item's first product waits for these threads' P
      if (live) {
        const float lse2 = l == 0.0f ? -INFINITY : m * c + log2f(l);
        if (slot >= 0)
          a.part_lse[prow] = lse2;
        else if (a.lse)
          a.lse[token * a.Hq + head] = lse2 * 0.6931471805599453f;
      }
      __syncwarp();
      done += steps;
      if (!C::kAgain) break;
      if (job > 0) release_job(job - 1);
      if (!await_job(job, w.n)) break;
      cur = &job_sh[job & 1];
    }
  } else {
    reg_dec<40>();  // two tiles only: the idle warps
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kSoft + 1) {
    tc_fence_after();
    tmem_dealloc(tb, C::kCols);
  }
}

// Joins the partial results of rows whose keys were split: with L_i the parts'
// log2-sums and M their maximum, O = sum 2^(L_i - M) O_i / sum 2^(L_i - M).
// W warps per row (four rows, or one, per block): each finds the weights 2^(L_i - M)
// and adds up every W-th part (a part's O row is one 16- or 8-byte load per lane); the
// W sums are added in order. Bound: latency. Four warps where rows have many parts: a
// single-token call over 100000 keys, 37 parts, takes 75 us, and 79 with one; one warp
// where many rows have a few: 3000 tokens, 8 heads of 64, two parts, take 35 us, and 44 with four.
template <int D, int W>
__global__ void __launch_bounds__(128) prompt_join_kernel(const PromptDev a) {
  constexpr int V = D / 32;
  __shared__ float sum_sh[4][D], den_sh[4];
  const PromptJoin jn = a.joins[blockIdx.x];  // the plan's, written before the forward kernel began
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y * (4 / W) + warp / W;
  const int t = r >> 7, rr = r & 127;
  const int tok = t * a.tpt + rr / a.G, g = rr - (rr / a.G) * a.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
  if (jn.q0 < 0 || jn.head < 0 || jn.head * (long long)a.G >= a.Hq || jn.first < 0 || jn.n < 0 || jn.first + (long long)jn.n > a.n_slots) {
    if (threadIdx.x == 0) atomicExch(reinterpret_cast<int*>(a.plan_dev), kDevBadIndex);
    return;
  }
  if (rr >= a.G * a.tpt || tok >= jn.nq || jn.q0 + (long long)tok >= a.Tq) return;  // all W warps of the row
  const size_t rows = size_t(a.tiles) * 128;
  const float* lse = a.part_lse + jn.first * rows + r;  // of part i: [i rows]
  float mx = -INFINITY;
  for (int i = lane; i < jn.n; i += 32) mx = max_nan(mx, lse[i * rows]);
  for (int s = 16; s > 0; s >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, s));
  float o[V], den = 0.0f;
#pragma unroll
  for (int x = 0; x < V; ++x) o[x] = 0.0f;
  for (int i0 = 0; i0 < jn.n && mx != -INFINITY; i0 += 32) {
    const float w = i0 + lane < jn.n ? exp2f(lse[(i0 + lane) * rows] - mx) : 0.0f;
    const int end = min(32, jn.n - i0);
#pragma unroll 8
    for (int i = warp % W; i < end; i += W) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* p = a.part + ((jn.first + i0 + i) * rows + r) * D + lane * V;
      float x[V];
      if (V == 4)
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(p);
      else
        *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(p);
      den += wi;
#pragma unroll
      for (int y = 0; y < V; ++y) o[y] += wi * x[y];
    }
  }
  if (W > 1) {  // one row per block: nobody has left
#pragma unroll
    for (int x = 0; x < V; ++x) sum_sh[warp][lane * V + x] = o[x];
    if (lane == 0) den_sh[warp] = den;
    __syncthreads();
    if (warp > 0) return;
    den = (den_sh[0] + den_sh[1]) + (den_sh[2] + den_sh[3]);
#pragma unroll
    for (int x = 0; x < V; ++x) {
      const int c = lane * V + x;
      o[x] = (sum_sh[0][c] + sum_sh[1][c]) + (sum_sh[2][c] + sum_sh[3][c]);
    }
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  const long long token = (long long)jn.q0 + tok;
  const int head = jn.head * a.G + g;
  __nv_bfloat16* orow = a.o + token * a.o_row + head * a.o_head + lane * V;
#pragma unroll
  for (int x = 0; x < V; x += 2) {
    const uint32_t w = pack_bf16(o[x] * inv, o[x + 1] * inv);
    *reinterpret_cast<uint32_t*>(orow + x) = w;
    if (a.rest)
      *reinterpret_cast<uint32_t*>(a.rest + (token * a.Hq + head) * D + lane * V + x) =
          pack_rest(o[x] * inv, o[x + 1] * inv, w);
  }
  if (lane == 0 && a.lse)
    a.lse[token * a.Hq + head] = den == 0.0f ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
}

namespace {

template <int D, int TILES, bool FEW>
cudaError_t set_up() {
  return cudaFuncSetAttribute(prompt_fwd_kernel<D, TILES, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              FwdCfg<D, TILES, FEW>::kSmem);
}

template <int D, int TILES, bool FEW>
cudaError_t launch_d(const PromptArgs& a, const PromptMaps& maps, const PromptDev& v, cudaStream_t s) {
  using C = FwdCfg<D, TILES, FEW>;
  prompt_fwd_kernel<D, TILES, FEW><<<a.plan->n_items, C::kThreads, C::kSmem, s>>>(maps, v);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.plan->n_joins == 0) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const bool many = a.plan->join_parts > 8;
  cfg.gridDim = dim3(a.plan->n_joins, many ? a.plan->join_rows : (a.plan->join_rows + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, prompt_join_kernel<D, 4>, v)
              : cudaLaunchKernelEx(&cfg, prompt_join_kernel<D, 1>, v);
}

}  // namespace

cudaError_t launch_prompt_forward(const PromptArgs& a, cudaStream_t s) {
  const PromptPlan& p = *a.plan;
  // first, for it makes the device's context current in this thread, which the tensor maps need
  const bool two = p.tiles == 2, few = p.few != 0;
  const cudaError_t e = p.d == 128 ? (two ? set_up<128, 2, false>() : few ? set_up<128, 1, true>() : set_up<128, 1, false>())
                                   : (two ? set_up<64, 2, false>() : few ? set_up<64, 1, true>() : set_up<64, 1, false>());
  if (e != cudaSuccess) return e;
  PromptMaps maps;
  memset(&maps, 0, sizeof(maps));
  PromptDev v{};
  v.plan_dev = a.plan_dev;
  v.items = reinterpret_cast<const PromptItem*>(a.plan_dev + p.items);
  v.joins = reinterpret_cast<const PromptJoin*>(a.plan_dev + p.joins);
  v.o = static_cast<__nv_bfloat16*>(a.o.base);
  v.o_row = a.o.row;
  v.o_head = a.o.head;
  v.rest = static_cast<__nv_bfloat16*>(a.rest);
  v.lse = a.lse;
  v.part = a.part;
  v.part_lse = a.part_lse;
  v.Hq = p.Hq;
  v.n_slots = p.n_slots;
  v.G = p.G;
  v.tpt = kPromptTile / p.G;
  v.box = p.few ? kPromptFew / p.G : v.tpt;
  v.causal = p.causal;
  v.tiles = p.tiles;
  v.Tq = p.Tq;
  v.Tk = p.Tk;
  v.scale_log2 = p.scale * kLog2e;
  if (!map_queries(&maps.q, a.q, p.d, p.G, p.Hkv, p.Tq, v.box)) return cudaErrorInvalidValue;
  if (p.Tk > 0 && (!map_keys(&maps.k, a.k, p.d, p.Hkv, p.Tk) || !map_keys(&maps.v, a.v, p.d, p.Hkv, p.Tk)))
    return cudaErrorInvalidValue;
  if (p.d == 128)
    return two   ? launch_d<128, 2, false>(a, maps, v, s)
           : few ? launch_d<128, 1, true>(a, maps, v, s)
                 : launch_d<128, 1, false>(a, maps, v, s);
  return two   ? launch_d<64, 2, false>(a, maps, v, s)
         : few ? launch_d<64, 1, true>(a, maps, v, s)
               : launch_d<64, 1, false>(a, maps, v, s);
}

}  // namespace sla

// Packed prompt attention, backward, for an upstream dO:
//   P = 2^(c S - lse2), D = rowsum(dO O), dP = dO V^T, dS = P (dP - D)
//   dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K.
// Two kernels, so that every sum has one owner and a fixed order (no atomics):
// one per key tile (S^T, dP^T, dV, dK) and one per pair of query tiles (S, dP,
// dQ) - seven products instead of five, against float32 traffic for dQ or an
// order of additions that changes from run to run.
//
// The G query heads of a group are rows of the same packed query tile, so the
// sums over them need no extra pass. P and dS stay in TMEM as the A operands of
// the products that read them (bf16, over the S and dP they came from); dV, dK,
// dQ and everything between S and dS are float32.
#include <string.h>

#include "prompt_tc.cuh"

namespace sla {

using namespace tc;

struct PromptGradMaps {
  CUtensorMap q, k, v, g;
};

struct PromptGradDev {
  unsigned char* plan_dev;
  const PromptItem* rows;
  const PromptKeys* keys;
  const PromptKeysJoin* kjoins;
  PromptTensor o, g, dq, dk, dv;
  const float* lse;
  const __nv_bfloat16* rest;
  float2* ld;
  float* part;
  int Hq, Hkv, G, tpt, causal, row_tiles, n_kslots;
  long long Tq, Tk;
  float scale, scale_log2;
};

namespace {

constexpr int kSub = 128 * 128;  // 128 rows x 128 bytes (64 columns)

}  // namespace

// (lse log2 e, D) of every query row, [key head][token G + g]. d / 8 lanes per row,
// 16 bytes each. Bound: reading O and dO (and O's rest): 8192 tokens, 16 heads of 128, with the
// rest, 21 us, 5.0 TB/s.
template <int D>
__global__ void __launch_bounds__(256) prompt_rowsum_kernel(const PromptGradDev a) {
  asm volatile("griddepcontrol.launch_dependents;");  // the key kernel's first copies run beside this one
  constexpr int kLanes = D / 8;
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  const bool live = row < a.Tq * a.Hq;
  const long long t = live ? row / a.Hq : 0;
  const int h = live ? int(row - t * a.Hq) : 0;
  float sum = 0.0f;
  if (live) {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o.base) + t * a.o.row +
                                                    h * a.o.head + lane * 8);
    const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.g.base) + t * a.g.row +
                                                    h * a.g.head + lane * 8);
    uint4 z = make_uint4(0, 0, 0, 0);  // O = x + z
    if (a.rest) z = *reinterpret_cast<const uint4*>(a.rest + row * D + lane * 8);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w}, w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += (bf16_lo(u[i]) + bf16_lo(w[i])) * bf16_lo(v[i]) + (bf16_hi(u[i]) + bf16_hi(w[i])) * bf16_hi(v[i]);
  }
  for (int s = kLanes / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (live && lane == 0) {
    const int hk = h / a.G;
    a.ld[hk * (a.Tq * a.G) + t * a.G + (h - hk * a.G)] = make_float2(a.lse[t * a.Hq + h] * kLog2e, sum);
  }
}

// ---------------------------------------------------------------------------
// dK, dV: one CTA per tile of 128 keys (TMEM lane = key), over the query tiles
// that see it. Per query tile i:
//   S^T = K Q_i^T, dP^T = V dO_i^T      (M = 128 keys, N = 128 query rows, K = d)
//   dV += P^T dO_i, dK += dS^T Q_i      (M = 128 keys, N = d, K = 128; A in TMEM)
// A query row's lse and D belong to a column here, which every thread would have to
// fetch from shared memory (64 vector loads per thread and tile, a quarter of the
// bandwidth that the products' operands need). They go into the products instead: one
// more K step of 16 whose A is (1, 1, 1, 0 ...) and whose B holds -lse / scale, or -D,
// as three bf16 that add up to its float32, gives S - lse / scale and dP - D.
// Warps 0-3 form columns 0-63 of P^T and dS^T, warps 4-7 columns 64-127; warp 8
// loads, warp 9 issues. While the tensor cores run dV_i and S^T_{i+1} the warps
// form dS_i, while they run dK_i and dP^T_{i+1} the warps form P_{i+1}. P is formed as the
// row kernel forms it, on the special function units alone: a share on the FMA units (the
// forward's at d = 64) made no difference (16384 causal tokens, 12 heads of 128: 2218 us, and
// 2220 with three of eight pairs; 1732 tokens: 51.3 and 50.8).
// Bound: the tensor cores at d = 128 (8192 causal tokens, 16 heads: 475 us, the tensor pipe
// 64 % busy); at d = 64 the chain S - P - dP - dS of one key tile, which waits for itself
// (344 us: tensor pipe 46 %, special function units 42 %, issue slots 33 %).
// ---------------------------------------------------------------------------
namespace {

template <int D>
struct KeyCfg {
  static constexpr int kTileBytes = kSub * (D / 64);
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int oK = 0, oV = kTileBytes, oQ = 2 * kTileBytes;
  static constexpr int oG = oQ + kStages * kTileBytes;
  // the extra K steps: [2 column octets][128 rows][8] bf16, not swizzled
  static constexpr int kStep = 4096;
  static constexpr int oOne = oG + kStages * kTileBytes;  // A, constant
  static constexpr int oL = oOne + kStep;                 // B of S and of dP, per stage
  static constexpr int kBytes = oL + kStages * 2 * kStep;
  static constexpr int kSmem = kBytes + 1024;
  // TMEM columns. At d = 64 there is room for a second S, so that the next tile's S is
  // formed while this one's P is in use (a tile takes 2280 clocks instead of 2620).
  static constexpr bool kTwoS = D == 64;
  static constexpr int cS = 0, cP = 128, cV = 256, cK = 256 + D, cS1 = kTwoS ? 384 : 0;
};
enum { kbKV = 0, kbS0, kbS1, kbP, kbPr, kbDr, kbDone, kbQ };  // then Q full / empty, dO full / empty, (lse, D) full of every stage

}  // namespace

template <int D>
__global__ void __launch_bounds__(320, 1)
    prompt_bwd_keys_kernel(const __grid_constant__ PromptGradMaps maps, const PromptGradDev a) {
  using C = KeyCfg<D>;
  constexpr int ST = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[kbQ + 5 * ST];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = reinterpret_cast<int*>(a.plan_dev);
  const PromptKeys it = a.keys[blockIdx.x];
  if (it.k0 < 0 || it.lk < 1 || it.q0 < 0 || it.lq < 0 || it.k0 + (long long)it.lk > a.Tk ||
      it.q0 + (long long)it.lq > a.Tq || it.block < 0 || it.block * 128LL >= it.lk || it.head < 0 ||
      it.head >= a.Hkv || it.slot >= a.n_kslots || it.t0 < 0 || (it.t1 > it.t0 && (it.t1 - 1LL) * a.tpt >= it.lq)) {
    if (threadIdx.x == 0) atomicExch(status, kDevBadIndex);
    return;
  }
  const int n = max(0, it.t1 - it.t0);
  const int rows = a.G * a.tpt;

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
  auto qfull = [&](int i) { return kbQ + i % ST; };
  auto qempty = [&](int i) { return kbQ + ST + i % ST; };
  auto gfull = [&](int i) { return kbQ + 2 * ST + i % ST; };
  auto gempty = [&](int i) { return kbQ + 3 * ST + i % ST; };
  auto lfull = [&](int i) { return kbQ + 4 * ST + i % ST; };
  // S of tile i: its barrier (with two S, one each), the phase of it, its columns
  auto s_bar = [&](int i) { return C::kTwoS ? kbS0 + (i & 1) : kbS0; };
  auto s_phase = [&](int i) { return uint32_t(C::kTwoS ? i >> 1 : i) & 1; };
  auto s_col = [&](int i) { return C::kTwoS && (i & 1) ? C::cS1 : C::cS; };
  auto phase = [&](int i) { return uint32_t(i / ST) & 1; };

  auto load_q = [&](int i) {
    mbar_expect_tx(bar(qfull(i)), rows * D * 2);
    for (int s = 0; s < D / 64; ++s)
      tma_load_4d(sb + C::oQ + (i % ST) * C::kTileBytes + s * kSub, &maps.q, bar(qfull(i)), s * 64, 0,
                  it.q0 + (it.t0 + i) * a.tpt, it.head);
  };
  auto load_g = [&](int i) {
    mbar_expect_tx(bar(gfull(i)), rows * D * 2);
    for (int s = 0; s < D / 64; ++s)
      tma_load_4d(sb + C::oG + (i % ST) * C::kTileBytes + s * kSub, &maps.g, bar(gfull(i)), s * 64, 0,
                  it.q0 + (it.t0 + i) * a.tpt, it.head);
  };
  if (warp == 8 && lane == 0) {
    // the loader sets the barriers up and starts the first copies before the block meets
    // (they are the caller's tensors: nothing here waits for the row sums yet)
    abort_sh = 0;
    for (int i = 0; i < kbQ + 5 * ST; ++i) mbar_init(bar(i), i == kbPr || i == kbDr ? 256 : i >= kbQ + 4 * ST ? 32 : 1);
    fence_barrier_init();
    fence_async_smem();
    if (n > 0) {
      mbar_expect_tx(bar(kbKV), 2 * C::kTileBytes);
      for (int s = 0; s < D / 64; ++s) {
        tma_load_3d(sb + C::oK + s * kSub, &maps.k, bar(kbKV), s * 64, it.k0 + it.block * 128, it.head);
        tma_load_3d(sb + C::oV + s * kSub, &maps.v, bar(kbKV), s * 64, it.k0 + it.block * 128, it.head);
      }
      for (int i = 0; i < min(n, ST); ++i) {
        load_q(i);
        load_g(i);
      }
    }
  }
  for (int x = threadIdx.x; x < (1 + 2 * ST) * (C::kStep / 16); x += 320) {
    const bool one = x < 128;  // 1.0 in bf16 is 0x3f80
    *reinterpret_cast<uint4*>(smem + C::oOne + x * 16) = make_uint4(one ? 0x3f803f80u : 0u, one ? 0x3f80u : 0u, 0, 0);
  }
  fence_async_smem();
  // rows that the query tiles' copies never write (128 is not a multiple of G): their products must add nothing
  if (rows < 128) {
    const int idle = (128 - rows) * 8;
    for (int x = threadIdx.x; x < idle * 2 * ST * (D / 64); x += 320) {
      const int tile = x / idle, y = x - tile * idle;
      *reinterpret_cast<uint4*>(smem + C::oQ + tile * kSub + rows * 128 + y * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
  }
  if (warp == 9) tmem_alloc(smem_u32(&tmem_base_sh), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base_sh;

  if (warp == 8) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the row sums are written
    // from here on the row kernel may start where this one leaves SMs idle: it reads the row
    // sums too, and nothing that this kernel writes
    asm volatile("griddepcontrol.launch_dependents;");
    if (n > 0) {
      const float2* ld = a.ld + it.head * (a.Tq * a.G);
      const float inv_c = 1.0f / a.scale_log2;
      // (lse2, D) of a tile, fetched a tile ahead: four rows per lane
      float2 next[4];
      auto fetch = [&](int i) {
        const int tok = (it.t0 + i) * a.tpt;
        const long long r0 = (it.q0 + (long long)tok) * a.G;
        const int have = i < n ? min(rows, (it.lq - tok) * a.G) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = j * 32 + lane;
          next[j] = r < have ? ld[r0 + r] : make_float2(0.0f, 0.0f);
        }
      };
      fetch(0);
      int qi = min(n, ST), gi = qi;  // copies on their way
      for (int i = 0; i < n; ++i) {
        if (!wait_w(qempty(i), phase(i) ^ 1)) break;
        if (lane == 0 && i >= ST) {
          qi = i + 1;
          load_q(i);
        }
        __syncwarp();
        // the stage's -lse / scale and -D: its last readers, S and dP, came before the dK that freed the stage
        unsigned char* to = smem + C::oL + (i % ST) * 2 * C::kStep;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = j * 32 + lane;
          // (a row that sees no key has lse = -inf; all its columns are masked)
          *reinterpret_cast<uint4*>(to + r * 16) = three_bf16(next[j].x == -INFINITY ? 0.0f : -next[j].x * inv_c);
          *reinterpret_cast<uint4*>(to + C::kStep + r * 16) = three_bf16(-next[j].y);
        }
        fence_async_smem();
        mbar_arrive(bar(lfull(i)));
        fetch(i + 1);
        if (!wait_w(gempty(i), phase(i) ^ 1)) break;
        if (lane == 0 && i >= ST) {
          gi = i + 1;
          load_g(i);
        }
      }
      if (lane == 0) {
        wait_drain(kbKV, 0);
        for (int i = max(0, qi - ST); i < qi; ++i) wait_drain(qfull(i), phase(i));
        for (int i = max(0, gi - ST); i < gi; ++i) wait_drain(gfull(i), phase(i));
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idD = idesc_bf16(128, D, 0, 1);
    // rows behind the sequence's last token (another sequence's, or none): 0 x NaN is NaN
    auto clear_tail = [&](int i, int at) {
      const int have = (it.lq - (it.t0 + i) * a.tpt) * a.G;
      if (have >= rows) return;
      for (int x = have * 8 + lane; x < rows * 8; x += 32)
#pragma unroll
        for (int s = 0; s < D / 64; ++s)
          *reinterpret_cast<uint4*>(smem + at + (i % ST) * C::kTileBytes + s * kSub + x * 16) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
      __syncwarp();
    };
    auto issue_wide = [&](int col, int a_off, int b_off, int ext) {  // [128 keys][d] x [128 rows][d]^T
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t o = (k >> 2) * kSub + (k & 3) * 32;
        mma_bf16(tb + col, sdesc(sb + a_off + o, 16, 1024), sdesc(sb + b_off + o, 16, 1024), idS, k > 0);
      }
      // no swizzle: 8 x 16-byte core matrices, 2048 bytes apart along K, 128 along the rows
      mma_bf16(tb + col, sdesc(sb + C::oOne, 2048, 128, 0), sdesc(sb + ext, 2048, 128, 0), idS, 1);
    };
    auto issue_s = [&](int i) {
      wait_w(lfull(i), phase(i));
      wait_w(qfull(i), phase(i));
      clear_tail(i, C::oQ);
      tc_fence_after();
      issue_wide(s_col(i), C::oK, C::oQ + (i % ST) * C::kTileBytes, C::oL + (i % ST) * 2 * C::kStep);
      mma_commit(bar(s_bar(i)));
    };
    auto issue_p = [&](int i) {
      wait_w(gfull(i), phase(i));
      clear_tail(i, C::oG);
      tc_fence_after();
      issue_wide(C::cP, C::oV, C::oG + (i % ST) * C::kTileBytes, C::oL + ((i % ST) * 2 + 1) * C::kStep);
      mma_commit(bar(kbP));
    };
    // A: packed columns 0-31 (rows 0-63 of the tile) and 64-95 (rows 64-127) of the region it overwrote
    auto issue_acc = [&](int col, int from, uint32_t b_at, bool first) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_bf16_ts(tb + col, tb + from + (k >> 2) * 64 + (k & 3) * 8, sdesc(b_at + k * 2048, kSub, 1024), idD,
                    (!first || k > 0) ? 1u : 0u);
    };
    if (n > 0) {
      wait_w(kbKV, 0);
      issue_s(0);
      issue_p(0);
    }
    for (int i = 0; i < n; ++i) {
      if (C::kTwoS && i + 1 < n) issue_s(i + 1);
      wait_w(kbPr, i & 1);
      tc_fence_after();
      issue_acc(C::cV, s_col(i), sb + C::oG + (i % ST) * C::kTileBytes, i == 0);
      mma_commit(bar(gempty(i)));
      if (!C::kTwoS && i + 1 < n) issue_s(i + 1);
      wait_w(kbDr, i & 1);
      tc_fence_after();
      issue_acc(C::cK, C::cP, sb + C::oQ + (i % ST) * C::kTileBytes, i == 0);
      mma_commit(bar(qempty(i)));
      if (i + 1 < n) issue_p(i + 1);
    }
    mma_commit(bar(kbDone));
    wait_drain(kbDone, 0);
    __syncwarp();
  } else {
    const int r = threadIdx.x & 127, half = warp >> 2;  // key row, column half
    const int key = it.block * 128 + r;                 // in the sequence
    const bool live = key < it.lk;
    const uint32_t tq = tb + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t tP = tq + C::cP + half * 64;
    const uint64_t c2 = two(a.scale_log2, a.scale_log2);
    for (int i = 0; i < n; ++i) {
      const int tok = (it.t0 + i) * a.tpt;
      // columns (packed query rows) lo .. hi - 1 of this half see the key
      const long long first = a.causal ? (long long)key - (it.lk - it.lq) - tok : 0;  // first token of the tile
      const int lo = int(max(0LL, min(128LL, first * a.G))) - half * 64;
      const int hi = min(rows, (it.lq - tok) * a.G) - half * 64;
      const bool masked = lo > 0 || hi < 64;
      const uint32_t tS = tq + s_col(i) + half * 64;
      wait_w(s_bar(i), s_phase(i));
      tc_fence_after();
      float p[64];
      tmem_ld32(tS, *reinterpret_cast<float(*)[32]>(&p[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<float(*)[32]>(&p[32]));
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 64; j += 2) {  // 2^(c S - lse2)
        untwo(mul2(two(p[j], p[j + 1]), c2), p[j], p[j + 1]);
        p[j] = ex2(p[j]);
        p[j + 1] = ex2(p[j + 1]);
      }
      if (__any_sync(0xffffffffu, masked)) {
#pragma unroll
        for (int j = 0; j < 64; ++j) p[j] = j >= lo && j < hi ? p[j] : 0.0f;
      }
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
      tmem_st32u(tS, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kbPr));
      wait_w(kbP, i & 1);
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float x[32];
        tmem_ld32(tP + 32 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          untwo(mul2(two(p[32 * q + j], p[32 * q + j + 1]), two(x[j], x[j + 1])), p[32 * q + j], p[32 * q + j + 1]);
      }
      if (__any_sync(0xffffffffu, masked)) {
#pragma unroll
        for (int j = 0; j < 64; ++j) p[j] = j >= lo && j < hi ? p[j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
      tmem_st32u(tP, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kbDr));
    }
    if (n > 0) {
      wait_w(kbDone, 0);
      tc_fence_after();
    }
    // half 0 writes dV, half 1 dK
    const int col = half == 0 ? C::cV : C::cK;
    const float f = half == 0 ? 1.0f : a.scale;
    const PromptTensor& t = half == 0 ? a.dv : a.dk;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t.base) + (it.k0 + (long long)key) * t.row + it.head * t.head;
    float* part = a.part + ((size_t(max(it.slot, 0)) * 2 + half) * 128 + r) * D;
#pragma unroll 1
    for (int j = 0; j < D; j += 32) {
      float x[32];
      if (n > 0) {
        tmem_ld32(tq + col + j, x);
        tmem_wait_ld();
      }
#pragma unroll
      for (int y = 0; y < 32; ++y) x[y] = n > 0 ? x[y] * f : 0.0f;
      if (!live) continue;
      if (it.slot < 0) {
#pragma unroll
        for (int y = 0; y < 32; y += 8)
          *reinterpret_cast<uint4*>(out + j + y) =
              make_uint4(pack_bf16(x[y], x[y + 1]), pack_bf16(x[y + 2], x[y + 3]), pack_bf16(x[y + 4], x[y + 5]),
                         pack_bf16(x[y + 6], x[y + 7]));
      } else {
#pragma unroll
        for (int y = 0; y < 32; y += 4)
          *reinterpret_cast<float4*>(part + j + y) = make_float4(x[y], x[y + 1], x[y + 2], x[y + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// Sums of the parts of split key tiles, in a fixed order; one warp per (key, dV or dK).
// Bound: latency and the parts' bytes, which the key kernel has just left in L2.
template <int D>
__global__ void __launch_bounds__(128) prompt_keys_join_kernel(const PromptGradDev a) {
  const PromptKeysJoin jn = a.kjoins[blockIdx.x];
  const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5), which = blockIdx.z;
  if (jn.row < 0 || jn.row + (long long)jn.nk > a.Tk || jn.head < 0 || jn.head >= a.Hkv || jn.first < 0 || jn.n < 0 ||
      jn.first + (long long)jn.n > a.n_kslots) {
    if (threadIdx.x == 0) atomicExch(reinterpret_cast<int*>(a.plan_dev), kDevBadIndex);
    return;
  }
  if (r >= jn.nk) return;
  float x[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = 0.0f;
  for (int s = 0; s < jn.n; ++s) {
    const float* part = a.part + ((size_t(jn.first + s) * 2 + which) * 128 + r) * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] += part[i];
  }
  const PromptTensor& t = which == 0 ? a.dv : a.dk;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t.base) + (jn.row + (long long)r) * t.row + jn.head * t.head +
                       lane * (D / 32);
#pragma unroll
  for (int i = 0; i < D / 32; i += 2) *reinterpret_cast<uint32_t*>(out + i) = pack_bf16(x[i], x[i + 1]);
}

// ---------------------------------------------------------------------------
// dQ: one CTA per item of up to two query tiles, as in the forward. Per key block:
//   X = Q K_j^T, X = dO V_j^T over it once S has been read, dS (bf16) over that,
//   dQ += dS K_j (M = 128, N = d, K = 128; A in TMEM).
// One 128-column region X per tile leaves TMEM room for two tiles' dQ: the chain
// S - dP - dS - dQ of one tile runs in the gaps of the other's. Measured, 8192 causal
// tokens, 16 heads: d = 128, 328 us, the tensor pipe 66 % busy (its bound); d = 64, 272 us, no
// unit at its limit (special function units 54 %, tensor pipe 39 %, issue slots 36 %): the chain.
// ---------------------------------------------------------------------------
namespace {

template <int D>
struct RowCfg {
  static constexpr int kTileBytes = kSub * (D / 64);
  // V is read early in a step (dP of both tiles), K from one step's S to the next
  // step's dQ: with shared memory for three tiles (d = 128), K takes two of them
  static constexpr int kK = D == 128 ? 2 : 3, kV = D == 128 ? 1 : 3;
  static constexpr int oQ = 0, oG = 2 * kTileBytes, oK = 4 * kTileBytes, oV = oK + kK * kTileBytes;
  static constexpr int kBytes = oV + kV * kTileBytes;
  static constexpr int kSmem = kBytes + 1024;
  static constexpr int cX = 0, cQ = 256;  // X0 X1 (128 columns each), dQ0 dQ1 (D each)
};
// per tile: Q and dO loaded, S done, S read, dP done, dS written
enum { rbIn0 = 0, rbIn1, rbS0, rbS1, rbR0, rbR1, rbP0, rbP1, rbD0, rbD1, rbDone, rbKV };  // then K full / empty, V full / empty of every stage

}  // namespace

template <int D>
__global__ void __launch_bounds__(384, 1)
    prompt_bwd_rows_kernel(const __grid_constant__ PromptGradMaps maps, const PromptGradDev a) {
  using C = RowCfg<D>;
  constexpr int KS = C::kK, VS = C::kV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[rbKV + 2 * (KS + VS)];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = reinterpret_cast<int*>(a.plan_dev);
  const PromptItem it = a.rows[blockIdx.x];
  if (it.q0 < 0 || it.nq < 1 || it.k0 < 0 || it.lk < 0 || it.q0 + (long long)it.nq > a.Tq ||
      it.k0 + (long long)it.lk > a.Tk || it.nq > a.row_tiles * a.tpt || it.head < 0 ||
      it.head >= a.Hkv) {
    if (threadIdx.x == 0) atomicExch(status, kDevBadIndex);
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  auto end_block = [&](int t) {
    const int last = min(it.nq, (t + 1) * a.tpt) - 1;
    if (last < t * a.tpt) return 0;
    const long long keys = a.causal ? min((long long)it.lk, (long long)it.pos0 + last + 1) : it.lk;
    return int((max(keys, 0LL) + 127) / 128);
  };
  const int nb0 = end_block(0), nb1 = end_block(1), n = max(nb0, nb1);

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
  auto kfull = [&](int s) { return rbKV + s % KS; };
  auto kempty = [&](int s) { return rbKV + KS + s % KS; };
  auto vfull = [&](int s) { return rbKV + 2 * KS + s % VS; };
  auto vempty = [&](int s) { return rbKV + 2 * KS + VS + s % VS; };
  auto kphase = [&](int s) { return uint32_t(s / KS) & 1; };
  auto vphase = [&](int s) { return uint32_t(s / VS) & 1; };

  auto load_k = [&](int s) {
    mbar_expect_tx(bar(kfull(s)), C::kTileBytes);
    for (int x = 0; x < D / 64; ++x)
      tma_load_3d(sb + C::oK + (s % KS) * C::kTileBytes + x * kSub, &maps.k, bar(kfull(s)), x * 64,
                  it.k0 + (n - 1 - s) * 128, it.head);
  };
  auto load_v = [&](int s) {
    mbar_expect_tx(bar(vfull(s)), C::kTileBytes);
    for (int x = 0; x < D / 64; ++x)
      tma_load_3d(sb + C::oV + (s % VS) * C::kTileBytes + x * kSub, &maps.v, bar(vfull(s)), x * 64,
                  it.k0 + (n - 1 - s) * 128, it.head);
  };
  if (warp == 8 && lane == 0) {  // the barriers and the first copies, before the block meets
    abort_sh = 0;
    for (int i = 0; i < rbKV + 2 * (KS + VS); ++i)
      mbar_init(bar(i), i == rbR0 || i == rbR1 || i == rbD0 || i == rbD1 ? 128 : 1);
    fence_barrier_init();
    fence_async_smem();
    const int rows = a.G * a.tpt;
    for (int t = 0; t < 2; ++t) {
      if ((t == 0 ? nb0 : nb1) == 0) continue;
      mbar_expect_tx(bar(rbIn0 + t), 2 * rows * D * 2);
      for (int s = 0; s < D / 64; ++s) {
        tma_load_4d(sb + C::oQ + t * C::kTileBytes + s * kSub, &maps.q, bar(rbIn0 + t), s * 64, 0,
                    it.q0 + t * a.tpt, it.head);
        tma_load_4d(sb + C::oG + t * C::kTileBytes + s * kSub, &maps.g, bar(rbIn0 + t), s * 64, 0,
                    it.q0 + t * a.tpt, it.head);
      }
    }
    if (n > 0) {
      load_k(0);
      load_v(0);
    }
  }
  if (warp == 9) tmem_alloc(smem_u32(&tmem_base_sh), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_base_sh;

  // A row's 128 P values stay in its thread's registers between S and dP: the
  // softmax warps take the registers that the other four leave (2 x 232 + 40 =
  // 3 x 168 per thread column, the launch's own share).
  if (warp == 8) {
    reg_dec<40>();
    if (lane == 0 && n > 0) {
      int ks = 1, vs = 1;  // tiles on their way
      for (int s = 1; s < n; ++s) {
        if (!wait(kempty(s), kphase(s) ^ 1)) break;
        ks = s + 1;
        load_k(s);
        if (!wait(vempty(s), vphase(s) ^ 1)) break;
        vs = s + 1;
        load_v(s);
      }
      if (nb0 > 0) wait_drain(rbIn0, 0);
      if (nb1 > 0) wait_drain(rbIn1, 0);
      for (int s = max(0, ks - KS); s < ks; ++s) wait_drain(kfull(s), kphase(s));
      for (int s = max(0, vs - VS); s < vs; ++s) wait_drain(vfull(s), vphase(s));
    }
    __syncwarp();
  } else if (warp == 9) {
    reg_dec<40>();
    constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idD = idesc_bf16(128, D, 0, 1);
    const int off[2] = {n - nb0, n - nb1};
    auto issue_wide = [&](int t, int a_off, int b_off) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t o = (k >> 2) * kSub + (k & 3) * 32;
        mma_bf16(tb + C::cX + t * 128, sdesc(sb + a_off + o, 16, 1024), sdesc(sb + b_off + o, 16, 1024), idS, k > 0);
      }
    };
    auto k_at = [&](int s) { return C::oK + (s % KS) * C::kTileBytes; };
    auto v_at = [&](int s) { return C::oV + (s % VS) * C::kTileBytes; };
    // K of step s is there, the rows behind the sequence's last key cleared (dS K adds them as 0 x value)
    auto have_k = [&](int s) {
      wait_w(kfull(s), kphase(s));
      const int valid = it.lk - (n - 1 - s) * 128;
      if (valid < 128) {
        for (int x = valid * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
          for (int sub = 0; sub < D / 64; ++sub)
            *reinterpret_cast<uint4*>(smem + k_at(s) + sub * kSub + x * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
      }
      tc_fence_after();
    };
    auto issue_s = [&](int t, int s) {
      if (s == off[t]) wait_w(rbIn0 + t, 0);
      issue_wide(t, C::oQ + t * C::kTileBytes, k_at(s));
      mma_commit(bar(rbS0 + t));
    };
    if (n > 0) {
      have_k(0);
      for (int t = 0; t < 2; ++t)
        if (off[t] == 0) issue_s(t, 0);
    }
    for (int s = 0; s < n; ++s) {
      wait_w(vfull(s), vphase(s));
      for (int t = 0; t < 2; ++t) {
        if (s < off[t]) continue;
        wait_w(rbR0 + t, (s - off[t]) & 1);
        tc_fence_after();
        issue_wide(t, C::oG + t * C::kTileBytes, v_at(s));
        mma_commit(bar(rbP0 + t));
      }
      mma_commit(bar(vempty(s)));
      bool have = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (s >= off[t]) {
          wait_w(rbD0 + t, (s - off[t]) & 1);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ts(tb + C::cQ + t * D, tb + C::cX + t * 128 + k * 8, sdesc(sb + k_at(s) + k * 2048, kSub, 1024),
                        idD, (s > off[t] || k > 0) ? 1u : 0u);
        }
        if (t == 1) mma_commit(bar(kempty(s)));
        if (s + 1 < n && s + 1 >= off[t]) {
          if (!have) have_k(s + 1);
          have = true;
          issue_s(t, s + 1);
        }
      }
    }
    mma_commit(bar(rbDone));
    wait_drain(rbDone, 0);
    __syncwarp();
  } else if (warp < 8) {
    reg_inc<232>();
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int nb = t == 0 ? nb0 : nb1;
    const int tok = t * a.tpt + r / a.G, g = r - (r / a.G) * a.G;
    const bool live = r < a.G * a.tpt && tok < it.nq;
    const int limit = !live ? 0 : a.causal ? int(max(0LL, min((long long)it.lk, (long long)it.pos0 + tok + 1))) : it.lk;
    const int warp_limit = __reduce_min_sync(0xffffffffu, limit);
    const uint32_t tq = tb + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t tX = tq + C::cX + t * 128, tO = tq + C::cQ + t * D;
    const float c = a.scale_log2;
    const long long token = (long long)it.q0 + tok;
    float2 w = make_float2(0.0f, 0.0f);
    if (live) w = a.ld[it.head * (a.Tq * a.G) + token * a.G + g];
    const uint64_t c2 = two(c, c), lse2 = two(-w.x, -w.x);
    for (int i = 0; i < nb; ++i) {
      const int seen = limit - (nb - 1 - i) * 128;
      const bool masked = (nb - i) * 128 > warp_limit;
      wait_w(rbS0 + t, i & 1);
      tc_fence_after();
      float p[128];
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_ld32(tX + 32 * j, *reinterpret_cast<float(*)[32]>(&p[32 * j]));
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(rbR0 + t));
#pragma unroll
      for (int j = 0; j < 128; j += 2) {
        untwo(fma2(two(p[j], p[j + 1]), c2, lse2), p[j], p[j + 1]);
        p[j] = ex2(p[j]);
        p[j + 1] = ex2(p[j + 1]);
      }
      wait_w(rbP0 + t, i & 1);
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[32];
        tmem_ld32(tX + 32 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = p[32 * q + j] * (x[j] - w.y);
        if (masked) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 32 * q + j < seen ? x[j] : 0.0f;
        }
        uint32_t y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
        tmem_st16u(tX + 16 * q, y);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(rbD0 + t));
    }
    if (nb > 0) {
      wait_w(rbDone, 0);
      tc_fence_after();
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq.base) + token * a.dq.row + (it.head * a.G + g) * a.dq.head;
#pragma unroll 1
    for (int j = 0; j < D; j += 32) {
      float x[32];
      if (nb > 0) {
        tmem_ld32(tO + j, x);
        tmem_wait_ld();
      }
#pragma unroll
      for (int y = 0; y < 32; ++y) x[y] = nb > 0 ? x[y] * a.scale : 0.0f;
      if (!live) continue;
#pragma unroll
      for (int y = 0; y < 32; y += 8)
        *reinterpret_cast<uint4*>(out + j + y) =
            make_uint4(pack_bf16(x[y], x[y + 1]), pack_bf16(x[y + 2], x[y + 3]), pack_bf16(x[y + 4], x[y + 5]),
                       pack_bf16(x[y + 6], x[y + 7]));
    }
  } else {
    reg_dec<40>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
  // This kernel may have started beside the key kernel and must not end before it: what
  // follows in the stream reads both. One block's wait is the grid's.
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

namespace {

template <int D>
cudaError_t set_up() {
  cudaError_t e = cudaFuncSetAttribute(prompt_bwd_keys_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       KeyCfg<D>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prompt_bwd_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowCfg<D>::kSmem);
  return e;
}

template <int D>
cudaError_t launch_d(const PromptGradArgs& a, const PromptGradMaps& maps, const PromptGradDev& v, cudaStream_t s) {
  const PromptPlan& p = *a.plan;
  const long long rows = p.Tq * p.Hq;
  prompt_rowsum_kernel<D><<<unsigned((rows * (D / 8) + 255) / 256), 256, 0, s>>>(v);
  // The key kernel starts beside the row sums and waits for them; the row kernel starts where
  // the key kernel's last blocks leave SMs idle (the key kernel's blocks have all seen the row
  // sums by then). Without key tiles the row kernel is an ordinary launch behind the row sums.
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cudaError_t e = cudaSuccess;
  if (p.n_keys > 0) {
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(p.n_keys);
    cfg.blockDim = dim3(320);
    cfg.dynamicSmemBytes = KeyCfg<D>::kSmem;
    e = cudaLaunchKernelEx(&cfg, prompt_bwd_keys_kernel<D>, maps, v);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(p.n_rows);
  cfg.blockDim = dim3(384);
  cfg.dynamicSmemBytes = RowCfg<D>::kSmem;
  e = cudaLaunchKernelEx(&cfg, prompt_bwd_rows_kernel<D>, maps, v);
  if (e != cudaSuccess) return e;
  if (p.n_kjoins > 0) prompt_keys_join_kernel<D><<<dim3(p.n_kjoins, 32, 2), 128, 0, s>>>(v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_backward(const PromptGradArgs& a, cudaStream_t s) {
  const PromptPlan& p = *a.plan;
  // first, for it makes the device's context current in this thread, which the tensor maps need
  // (autograd calls from a thread of its own)
  const cudaError_t e = p.d == 128 ? set_up<128>() : set_up<64>();
  if (e != cudaSuccess) return e;
  PromptGradMaps maps;
  memset(&maps, 0, sizeof(maps));
  PromptGradDev v{};
  v.plan_dev = a.plan_dev;
  v.rows = reinterpret_cast<const PromptItem*>(a.plan_dev + p.rows);
  v.keys = reinterpret_cast<const PromptKeys*>(a.plan_dev + p.keys);
  v.kjoins = reinterpret_cast<const PromptKeysJoin*>(a.plan_dev + p.kjoins);
  v.o = a.o;
  v.g = a.dO;
  v.dq = a.dq;
  v.dk = a.dk;
  v.dv = a.dv;
  v.lse = a.lse;
  v.rest = static_cast<const __nv_bfloat16*>(a.rest);
  v.ld = a.ld;
  v.part = a.part;
  v.Hq = p.Hq;
  v.Hkv = p.Hkv;
  v.G = p.G;
  v.tpt = kPromptTile / p.G;
  v.causal = p.causal;
  v.row_tiles = p.row_tiles;
  v.n_kslots = p.n_kslots;
  v.Tq = p.Tq;
  v.Tk = p.Tk;
  v.scale = p.scale;
  v.scale_log2 = p.scale * kLog2e;
  if (!map_queries(&maps.q, a.q, p.d, p.G, p.Hkv, p.Tq, v.tpt) ||
      !map_queries(&maps.g, a.dO, p.d, p.G, p.Hkv, p.Tq, v.tpt))
    return cudaErrorInvalidValue;
  if (p.Tk > 0 && (!map_keys(&maps.k, a.k, p.d, p.Hkv, p.Tk) || !map_keys(&maps.v, a.v, p.d, p.Hkv, p.Tk)))
    return cudaErrorInvalidValue;
  return p.d == 128 ? launch_d<128>(a, maps, v, s) : launch_d<64>(a, maps, v, s);
}

}  // namespace sla

// tcgen05 / TMA pieces that the packed prompt attention's kernels share.
#pragma once

#include "prompt.cuh"
#include "tc_util.cuh"

namespace sla {
namespace tc {

// D[tmem] (+)= A[tmem] * B[smem], warp-collective like mma_bf16
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// 32 lanes x 32 columns of packed bf16 pairs
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// What rounding (a, b) to the bf16 pair w left off, as a bf16 pair
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t w) {
  return pack_bf16(a - bf16_lo(w), b - bf16_hi(w));
}
// Registers per thread of this warpgroup, from here on (all four warps run it)
template <int n>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}
// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// two float32 values in one register pair, and the packed operations on them
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void untwo(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// x as three bf16 that add up to it, and zeros, as one 16-byte row piece (inf and NaN as they are)
__device__ __forceinline__ uint4 three_bf16(float x) {
  const float a = bf16_lo(pack_bf16(x, 0.0f));
  const float y = fabsf(a) < INFINITY ? x - a : 0.0f;
  const float b = bf16_lo(pack_bf16(y, 0.0f));
  return make_uint4(pack_bf16(a, b), pack_bf16(y - b, 0.0f), 0, 0);
}
// 2^x of two values on the FMA units, for x <= 127: x = i + f with i the nearest
// whole number (adding 1.5 2^23 rounds to it), 2^f by a cubic with p(0) = 1 fitted
// to the least relative error on [-1/2, 1/2] (1.0e-4, a twentieth of a bf16 step).
// x <= -127 gives 0. kNan: times 2^i (127 more on the way make i the exponent field
// of 2^i), which keeps NaN; else i is added to the exponent of 2^f, an operation
// less, and NaN comes out as a number near the largest.
template <bool kNan>
__device__ __forceinline__ void ex2_fma(uint64_t x2, float& lo, float& hi) {
  float x, y;
  untwo(x2, x, y);
  const uint64_t v = two(max_nan(x, -127.0f), max_nan(y, -127.0f));
  constexpr float kRound = 12582912.0f + (kNan ? 127.0f : 0.0f);
  const uint64_t t = add2(v, two(kRound, kRound));
  const uint64_t f = fma2(add2(t, two(-kRound, -kRound)), two(-1.0f, -1.0f), v);
  uint64_t p = fma2(f, two(0.05500893294811249f, 0.05500893294811249f), two(0.2422109693288803f, 0.2422109693288803f));
  p = fma2(p, f, two(0.6932829022407532f, 0.6932829022407532f));
  p = fma2(p, f, two(1.0f, 1.0f));
  float i, j;
  untwo(t, i, j);
  const int ei = __float_as_int(i) << 23, ej = __float_as_int(j) << 23;
  if (kNan) {
    untwo(mul2(p, two(__int_as_float(ei), __int_as_float(ej))), lo, hi);
  } else {
    float a, b;
    untwo(p, a, b);
    lo = __int_as_float(__float_as_int(a) + ei);
    hi = __int_as_float(__float_as_int(b) + ej);
  }
}

// Taking over a block of the grid that has not started (one thread asks; blocks are handed
// out in order). The answer arrives in `next`, 16 bytes in shared memory, on the barrier;
// after an answer without a block none may be asked for again.
__device__ __forceinline__ void ask_block(uint4* next, uint32_t bar) {
  mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(next)),
      "r"(bar)
      : "memory");
}
// Its index, or -1.
__device__ __forceinline__ int answered_block(uint4* next) {
  uint32_t block, have;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n .reg .b32 y, z, u;\n ld.shared.b128 h, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %1, 1, 0, p;\n mov.u32 %0, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, u}, h;\n}\n"
      : "=r"(block), "=r"(have)
      : "r"(smem_u32(next))
      : "memory");
  return have ? int(block) : -1;
}

// ---- host: tensor maps of packed tokens ----
// Packed query rows: (d, G, tokens, key heads), boxes of 64 values x G heads x tpt tokens.
inline bool map_queries(CUtensorMap* m, const PromptTensor& t, int d, int G, int Hkv, long long T, int tpt) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(G), cuuint64_t(T), cuuint64_t(Hkv)};
  cuuint64_t strides[3] = {cuuint64_t(t.head) * 2, cuuint64_t(t.row) * 2, cuuint64_t(t.head) * 2 * G};
  cuuint32_t box[4] = {64, cuuint32_t(G), cuuint32_t(tpt), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Keys or values: (d, tokens, key heads), boxes of 64 values x 128 tokens.
inline bool map_keys(CUtensorMap* m, const PromptTensor& t, int d, int Hkv, long long T) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(T), cuuint64_t(Hkv)};
  cuuint64_t strides[2] = {cuuint64_t(t.row) * 2, cuuint64_t(t.head) * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace sla

// Rotary positions, alone and behind the norm of every query and key head.
//
// Rotation: pair i of a head row, (u, v), becomes gain (u cos a - v sin a,
// v cos a + u sin a) with a = p f_i, p the token's position on the pair's axis.
// Norm: x -> x / sqrt(mean(x^2) + eps) * w over the head's d values.
//
// The angle. f_i / 2 pi is held as a 64-bit fixed-point fraction of a turn, so
// p f_i mod one turn is one 64-bit integer product mod 2^64: exact for every
// position (its error is p 2^-65 turns, from the table), where a float32
// product is off by p f_i 2^-24 radians - a whole turn at far positions. The
// signed top 32 bits, converted to float32, are the angle in turns within
// +-1/2, off by at most 2^-26 turns (4e-8 of a turn, 1e-7 rad).
//
// Bound: HBM (each value read and written once). Split: `tpr` lanes share a
// head row, each with one unit = two chunks of V values that hold V whole pairs
// (layout "half": chunks V apart by rot / 2; "interleaved": two neighbours), so
// no value crosses a lane; only the norm's sum does, by shuffles. A lane keeps
// its V cos / sin pairs in registers and walks over the heads of its token, so
// the sines (about 40 instructions each) are paid once per token and not per
// head. Neighbouring lane groups take neighbouring tokens: a head-major output
// is then written in runs of whole tiles.
#include "sla_internal.cuh"

#include <cuda_fp16.h>

#include "rope.cuh"

namespace sla {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// V values in one access of V * sizeof(T) bytes
template <typename T, int V>
struct alignas(V * sizeof(T)) Chunk {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_chunk(const T* p, float (&f)[V]) {
  const Chunk<T, V> c = *reinterpret_cast<const Chunk<T, V>*>(p);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = to_f(c.e[j]);
}
template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, const float (&f)[V]) {
  Chunk<T, V> c;
#pragma unroll
  for (int j = 0; j < V; ++j) c.e[j] = from_f<T>(f[j]);
  *reinterpret_cast<Chunk<T, V>*>(p) = c;
}

// The two chunks (element offsets) of unit u; unit u holds pairs u V .. u V + V - 1 while u V < rot / 2.
template <int V, bool HALF>
__device__ __forceinline__ void unit_offsets(int u, int rot, int& ea, int& eb) {
  if (HALF && u * V < rot / 2) {
    ea = u * V;
    eb = ea + rot / 2;
  } else {  // interleaved pairs, or values behind the rotated part
    ea = 2 * u * V;
    eb = ea + V;
  }
}

// (a, b) of one unit turned by (c, s): across the chunks, or (V > 1, interleaved) inside them
template <int V, bool HALF>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&s)[V]) {
  if (HALF || V == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = a[j], v = b[j];
      a[j] = u * c[j] - v * s[j];
      b[j] = v * c[j] + u * s[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float u = a[2 * j], v = a[2 * j + 1];
      a[2 * j] = u * c[j] - v * s[j];
      a[2 * j + 1] = v * c[j] + u * s[j];
      const float x = b[2 * j], y = b[2 * j + 1];
      b[2 * j] = x * c[V / 2 + j] - y * s[V / 2 + j];
      b[2 * j + 1] = y * c[V / 2 + j] + x * s[V / 2 + j];
    }
  }
}

template <int V>
__device__ __forceinline__ void angles(const RopeArgs& a, int b, int n, int u, float (&c)[V], float (&s)[V]) {
  long long p = n;
  auto position = [&](int axis) {
    if (a.pos == nullptr) return;
    const long long at = axis * a.pos_axis + b * a.pos_b + n * a.pos_n;
    p = a.pos64 ? static_cast<const long long*>(a.pos)[at] : static_cast<const int*>(a.pos)[at];
  };
  position(0);
  int now = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = u * V + j;
    if (a.axis != nullptr) {
      const int ax = min(int(a.axis[i]), a.n_axes - 1);
      if (ax != now) position(now = ax);
    }
    const unsigned long long turn = a.turns[i] * static_cast<unsigned long long>(p);
    const float half_turns = float(int(turn >> 32)) * 0x1p-31f;  // in [-1, 1]
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    c[j] = cs * a.gain;
    s[j] = a.inverse ? -sn * a.gain : sn * a.gain;
  }
}

__device__ __forceinline__ float group_sum(float x, int tpr) {
  for (int o = tpr >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int V>
__device__ __forceinline__ void load_weight(const RopeArgs& a, const void* w, int ea, int eb, float (&wa)[V],
                                            float (&wb)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (a.w_f32) {
      wa[j] = static_cast<const float*>(w)[ea + j];
      wb[j] = static_cast<const float*>(w)[eb + j];
    } else if (a.dtype == SLA_BF16) {
      wa[j] = to_f(static_cast<const __nv_bfloat16*>(w)[ea + j]);
      wb[j] = to_f(static_cast<const __nv_bfloat16*>(w)[eb + j]);
    } else {
      wa[j] = to_f(static_cast<const __half*>(w)[ea + j]);
      wb[j] = to_f(static_cast<const __half*>(w)[eb + j]);
    }
  }
}

}  // namespace

// grid: (token tiles, tensors, head ranges). NU units per lane (1 but for V = 1).
template <typename T, int V, int NU, bool HALF, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  const RopeTensor& t = a.t[blockIdx.y];
  const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr;
  const unsigned tok = blockIdx.x * unsigned(kThreads / a.tpr) + group;
  const int h0 = blockIdx.z * a.hpg, h1 = min(t.H, h0 + a.hpg);
  const bool live = tok < unsigned(a.B) * unsigned(a.N);
  const int b = live ? int(tok / unsigned(a.N)) : 0, n = live ? int(tok - unsigned(b) * unsigned(a.N)) : 0;
  float c[NU][V], s[NU][V];
  float wa[NORM ? NU : 1][V], wb[NORM ? NU : 1][V];
  int ea[NU], eb[NU];
  bool on[NU];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = lane + k * a.tpr;
    on[k] = live && 2 * u * V < a.d;
    unit_offsets<V, HALF>(u, a.rot, ea[k], eb[k]);
  }
  const T* x = static_cast<const T*>(t.x) + b * t.xb + n * t.xn;
  T* y = static_cast<T*>(t.y) + b * t.yb + n * t.yn;
  // the first heads' values are on their way while the sines are formed
  constexpr int U = NU == 1 ? 2 : 1;  // heads in flight
  float va[U][NU][V], vb[U][NU][V];
  auto fetch = [&](int h) {
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (on[k] && h + q < h1) {
          load_chunk<T, V>(x + (h + q) * t.xh + ea[k], va[q][k]);
          load_chunk<T, V>(x + (h + q) * t.xh + eb[k], vb[q][k]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) va[q][k][j] = vb[q][k][j] = 0.0f;
        }
  };
  fetch(h0);
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = lane + k * a.tpr;
    if (on[k] && 2 * u * V < a.rot) {
      angles<V>(a, b, n, u, c[k], s[k]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        c[k][j] = 1.0f;
        s[k][j] = 0.0f;
      }
    }
    if (NORM && on[k]) load_weight<V>(a, t.w, ea[k], eb[k], wa[k], wb[k]);
  }
  for (int h = h0; h < h1; h += U) {
    if (h != h0) fetch(h);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) sum += va[q][k][j] * va[q][k][j] + vb[q][k][j] * vb[q][k][j];
        sum = group_sum(sum, a.tpr);
        const float r = 1.0f / sqrtf(sum * a.inv_d + a.eps);
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (on[k]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              va[q][k][j] *= r * wa[k][j];
              vb[q][k][j] *= r * wb[k][j];
            }
          }
      }
      if (h + q < h1) {
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (on[k]) {
            if (2 * (lane + k * a.tpr) * V < a.rot) rotate<V, HALF>(va[q][k], vb[q][k], c[k], s[k]);
            store_chunk<T, V>(y + (h + q) * t.yh + ea[k], va[q][k]);
            store_chunk<T, V>(y + (h + q) * t.yh + eb[k], vb[q][k]);
          }
      }
    }
  }
}

// Gradients of the norm with the rotation behind it. With g = the rotation of
// dy backwards, xh = x r, r = 1 / sqrt(mean(x^2) + eps):
//   dw = sum over tokens and heads of g xh,
//   dx = r (g w - xh mean(g w xh)).
// Blocks walk over token tiles; each keeps its dw in registers and leaves one
// row of partial sums, which norm_dw_kernel adds in a fixed order.
template <typename T, int V, int NU, bool HALF>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const RopeArgs a) {
  extern __shared__ float dw_sh[];  // [groups][d]
  const RopeTensor& t = a.t[blockIdx.y];
  const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr, groups = kThreads / a.tpr;
  float wa[NU][V], wb[NU][V], da[NU][V], db[NU][V];
  int ea[NU], eb[NU];
  bool has[NU];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = lane + k * a.tpr;
    has[k] = 2 * u * V < a.d;
    unit_offsets<V, HALF>(u, a.rot, ea[k], eb[k]);
    if (has[k]) load_weight<V>(a, t.w, ea[k], eb[k], wa[k], wb[k]);
#pragma unroll
    for (int j = 0; j < V; ++j) da[k][j] = db[k][j] = 0.0f;
  }
  const unsigned total = unsigned(a.B) * unsigned(a.N), tiles = (total + groups - 1) / groups;
  const int ranges = (t.H + a.hpg - 1) / a.hpg;
  for (unsigned long long item = blockIdx.x; item < (unsigned long long)tiles * ranges; item += gridDim.x) {
    const unsigned tile = unsigned(item / ranges), range = unsigned(item - (unsigned long long)tile * ranges);
    const unsigned tok = tile * groups + group;
    const bool live = tok < total;
    const int b = live ? int(tok / unsigned(a.N)) : 0, n = live ? int(tok - unsigned(b) * unsigned(a.N)) : 0;
    const int h0 = range * a.hpg, h1 = min(t.H, h0 + a.hpg);
    float c[NU][V], s[NU][V];
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (live && has[k] && 2 * (lane + k * a.tpr) * V < a.rot) angles<V>(a, b, n, lane + k * a.tpr, c[k], s[k]);
    const T* x = static_cast<const T*>(t.x) + b * t.xb + n * t.xn;
    const T* dy = static_cast<const T*>(t.dy) + b * t.gb + n * t.gn;
    T* dx = static_cast<T*>(t.y) + b * t.yb + n * t.yn;
    for (int h = h0; h < h1; ++h) {
      float xa[NU][V], xb[NU][V], ga[NU][V], gb[NU][V];
      float sxx = 0.0f, sgx = 0.0f;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (live && has[k]) {
          load_chunk<T, V>(x + h * t.xh + ea[k], xa[k]);
          load_chunk<T, V>(x + h * t.xh + eb[k], xb[k]);
          load_chunk<T, V>(dy + h * t.gh + ea[k], ga[k]);
          load_chunk<T, V>(dy + h * t.gh + eb[k], gb[k]);
          if (2 * (lane + k * a.tpr) * V < a.rot) rotate<V, HALF>(ga[k], gb[k], c[k], s[k]);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            sxx += xa[k][j] * xa[k][j] + xb[k][j] * xb[k][j];
            sgx += ga[k][j] * wa[k][j] * xa[k][j] + gb[k][j] * wb[k][j] * xb[k][j];
          }
        }
      }
      sxx = group_sum(sxx, a.tpr);
      sgx = group_sum(sgx, a.tpr);
      const float r = 1.0f / sqrtf(sxx * a.inv_d + a.eps);
      const float m = sgx * r * a.inv_d;  // mean(g w xh)
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (live && has[k]) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float ha = xa[k][j] * r, hb = xb[k][j] * r;
            da[k][j] += ga[k][j] * ha;
            db[k][j] += gb[k][j] * hb;
            xa[k][j] = r * (ga[k][j] * wa[k][j] - ha * m);
            xb[k][j] = r * (gb[k][j] * wb[k][j] - hb * m);
          }
          store_chunk<T, V>(dx + h * t.yh + ea[k], xa[k]);
          store_chunk<T, V>(dx + h * t.yh + eb[k], xb[k]);
        }
    }
  }
  if (t.dw == nullptr) return;  // uniform over the block
#pragma unroll
  for (int k = 0; k < NU; ++k)
    if (has[k]) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dw_sh[group * a.d + ea[k] + j] = da[k][j];
        dw_sh[group * a.d + eb[k] + j] = db[k][j];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    float sum = 0.0f;
    for (int g = 0; g < groups; ++g) sum += dw_sh[g * a.d + i];
    a.partial[(size_t(blockIdx.y) * gridDim.x + blockIdx.x) * a.d + i] = sum;
  }
}

// dw[i] = sum of the blocks' partial rows, in a fixed order: 32 slices of rows per
// column, then the slices. One block per 32 columns of one tensor.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const RopeArgs a, int rows) {
  __shared__ float part[32][33];
  void* dw = a.t[blockIdx.y].dw;
  if (dw == nullptr) return;
  const int col = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  float sum = 0.0f;
  if (col < a.d)
    for (int r = slice; r < rows; r += 32) sum += a.partial[(size_t(blockIdx.y) * rows + r) * a.d + col];
  part[slice][threadIdx.x % 32] = sum;
  __syncthreads();
  if (slice == 0 && col < a.d) {
    float all = 0.0f;
    for (int k = 0; k < 32; ++k) all += part[k][threadIdx.x];
    if (a.w_f32)
      static_cast<float*>(dw)[col] = all;
    else if (a.dtype == SLA_BF16)
      static_cast<__nv_bfloat16*>(dw)[col] = __float2bfloat16_rn(all);
    else
      static_cast<__half*>(dw)[col] = __float2half_rn(all);
  }
}

namespace {

template <typename T, int V, int NU>
cudaError_t launch_fwd(const RopeArgs& a, dim3 grid, cudaStream_t s) {
  const bool norm = a.t[0].w != nullptr;
  if (a.half)
    norm ? rope_kernel<T, V, NU, true, true><<<grid, kThreads, 0, s>>>(a)
         : rope_kernel<T, V, NU, true, false><<<grid, kThreads, 0, s>>>(a);
  else
    norm ? rope_kernel<T, V, NU, false, true><<<grid, kThreads, 0, s>>>(a)
         : rope_kernel<T, V, NU, false, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int V, int NU>
cudaError_t launch_bwd(const RopeArgs& a, dim3 grid, cudaStream_t s) {
  const size_t sh = size_t(kThreads / a.tpr) * a.d * sizeof(float);  // at most 16 KB
  if (a.half)
    norm_rope_bwd_kernel<T, V, NU, true><<<grid, kThreads, sh, s>>>(a);
  else
    norm_rope_bwd_kernel<T, V, NU, false><<<grid, kThreads, sh, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.t[0].dw == nullptr && a.t[1].dw == nullptr)) return e;
  norm_dw_kernel<<<dim3((a.d + 31) / 32, grid.y), 1024, 0, s>>>(a, int(grid.x));
  return cudaGetLastError();
}

// Values per chunk: the widest of `widths` that the pair layout, the strides and the addresses allow.
int chunk_width(const RopeArgs& a, int tensors, bool bwd) {
  const int size = a.dtype == SLA_FP32 ? 4 : 2;
  for (int v : {8, 4}) {
    if (v * size > 16) continue;
    if (a.d % (2 * v) != 0 || a.rot % (2 * v) != 0) continue;
    bool ok = true;
    for (int i = 0; i < tensors; ++i) {
      const RopeTensor& t = a.t[i];
      auto fits = [&](const void* p, long long b, long long n, long long h) {
        return reinterpret_cast<uintptr_t>(p) % (size_t(v) * size) == 0 && b % v == 0 && n % v == 0 && h % v == 0;
      };
      ok = ok && fits(t.x, t.xb, t.xn, t.xh) && fits(t.y, t.yb, t.yn, t.yh) &&
           (!bwd || fits(t.dy, t.gb, t.gn, t.gh));
    }
    if (ok) return v;
  }
  return 1;
}

}  // namespace

// Blocks of the backward: what two waves of four blocks per SM hold; also the rows of partial sums.
int rope_bwd_blocks(long long tokens, int heads) {
  // tokens per block are at least 8 (32 lanes a row), head ranges of at least 1
  const long long most = ((tokens + 7) / 8) * heads;
  return int(std::max(1LL, std::min<long long>(most, kRopeBwdBlocks)));
}

cudaError_t launch_rope(RopeArgs a, int tensors, bool bwd, cudaStream_t s) {
  const int v = chunk_width(a, tensors, bwd);
  const int units = a.d / (2 * v);
  a.tpr = 1;
  while (a.tpr < units && a.tpr < 32) a.tpr *= 2;
  const int groups = kThreads / a.tpr;
  const long long tokens = (long long)a.B * a.N;
  const long long tiles = (tokens + groups - 1) / groups;
  const int heads = std::max(a.t[0].H, tensors > 1 ? a.t[1].H : 0);
  // Heads per lane group: all of them once the token tiles alone fill the GPU
  // (8 blocks of 256 threads per SM), fewer while they do not.
  const long long want = (148 * 8 + tiles * tensors - 1) / (tiles * tensors);
  a.hpg = std::max<long long>(1, heads / std::min<long long>(want, heads));
  dim3 grid(unsigned(tiles), tensors, unsigned((heads + a.hpg - 1) / a.hpg));
  if (bwd) grid = dim3(rope_bwd_blocks(tokens, heads), tensors, 1);
#define SLA_ROPE(T)                                                       \
  (v == 8   ? (bwd ? launch_bwd<T, 8, 1>(a, grid, s) : launch_fwd<T, 8, 1>(a, grid, s)) \
   : v == 4 ? (bwd ? launch_bwd<T, 4, 1>(a, grid, s) : launch_fwd<T, 4, 1>(a, grid, s)) \
            : (bwd ? launch_bwd<T, 1, 4>(a, grid, s) : launch_fwd<T, 1, 4>(a, grid, s)))
  if (a.dtype == SLA_BF16) return SLA_ROPE(__nv_bfloat16);
  if (a.dtype == SLA_FP16) return SLA_ROPE(__half);
  if (v == 4) return bwd ? launch_bwd<float, 4, 1>(a, grid, s) : launch_fwd<float, 4, 1>(a, grid, s);
  return bwd ? launch_bwd<float, 1, 4>(a, grid, s) : launch_fwd<float, 1, 4>(a, grid, s);
#undef SLA_ROPE
}

}  // namespace sla

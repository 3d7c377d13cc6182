// Rotary positions, alone and behind the norm of every query and key head.
//
// Rotation: pair i of a head row, (u, v), becomes gain (u cos a - v sin a,
// v cos a + u sin a) with a = p f_i, p the token's position on the pair's axis.
// Norm: x -> x / sqrt(mean(x^2) + eps) * w over the head's d values.
//
// The angle. f_i / 2 pi is held as a 64-bit fixed-point fraction of a turn, so
// p f_i mod one turn is one 64-bit integer product mod 2^64: exact for every
// position (its error is p 2^-65 turns, from the table's rounding), where a float32
// product is off by p f_i 2^-24 radians - a whole turn at far positions. The
// signed top 32 bits, converted to float32, are the angle in turns within
// +-1/2, off by at most 2^-26 turns (1.5e-8 of a turn, 1e-7 rad).
//
// Bound: HBM (each value read and written once). Split: `tpr` lanes share a
// head row, each with one unit = two chunks of V values that hold V whole pairs
// (layout "half": chunks rot / 2 apart; "interleaved": two neighbours), so no
// value crosses a lane; only the norm's sum does, by shuffles. A lane keeps its
// V cos / sin pairs in registers and walks over the heads of its token, so the
// sines are paid once per token and not per head.
// The next heads' chunks are on their way meanwhile, as they came from memory.
// Chunks of 8 (16-byte loads) hold twice the registers and run half the warps:
// 45.7 us against 35.3 (480p video queries), 570 against 481 (720p queries and keys).
// Neighbouring lane groups take neighbouring tokens: a
// head-major output is then written in runs of whole tiles.
#include "sla_internal.cuh"

#include <cuda_fp16.h>

#include "rope.cuh"

namespace sla {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half& y) { y = __float2half_rn(x); }

// V values in one access of V * sizeof(T) bytes
template <typename T, int V>
struct alignas(V * sizeof(T)) Chunk {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Chunk<T, V> fetch_chunk(const T* p) {
  return *reinterpret_cast<const Chunk<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Chunk<T, V>& c, float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = to_f(c.e[j]);
}
template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, const float (&f)[V]) {
  Chunk<T, V> c;
#pragma unroll
  for (int j = 0; j < V; ++j) from_f(f[j], c.e[j]);
  *reinterpret_cast<Chunk<T, V>*>(p) = c;
}
// four 16-bit values: two 32-bit words, converted in pairs
template <typename T>
struct alignas(8) Chunk4 {
  uint32_t w[2];
};
template <>
struct Chunk<__nv_bfloat16, 4> : Chunk4<__nv_bfloat16> {};
template <>
struct Chunk<__half, 4> : Chunk4<__half> {};
__device__ __forceinline__ void widen(const Chunk<__nv_bfloat16, 4>& c, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f[2 * j] = bf16_lo(c.w[j]);
    f[2 * j + 1] = bf16_hi(c.w[j]);
  }
}
__device__ __forceinline__ void widen(const Chunk<__half, 4>& c, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&c.w[j]));
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, const __nv_bfloat16*) { return pack_bf16(a, b); }
__device__ __forceinline__ uint32_t narrow2(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&f)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(narrow2(f[0], f[1], p), narrow2(f[2], f[3], p));
}
__device__ __forceinline__ void store_chunk(__half* p, const float (&f)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(narrow2(f[0], f[1], p), narrow2(f[2], f[3], p));
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

// The two values of pair j of a unit's chunks: across them, or (V > 1, interleaved) inside them
template <int V, bool HALF>
__device__ __forceinline__ float& first(float (&a)[V], float (&b)[V], int j) {
  return HALF || V == 1 ? a[j] : j < V / 2 ? a[2 * j] : b[2 * j - V];
}
template <int V, bool HALF>
__device__ __forceinline__ float& second(float (&a)[V], float (&b)[V], int j) {
  return HALF || V == 1 ? b[j] : j < V / 2 ? a[2 * j + 1] : b[2 * j - V + 1];
}
// (u, v) -> (u c - v s, v c + u s); the operations are spelled out, so that every chunk width rounds alike
template <int V, bool HALF>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&s)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float &u = first<V, HALF>(a, b, j), &v = second<V, HALF>(a, b, j);
    const float x = fmaf(u, c[j], -__fmul_rn(v, s[j]));
    v = fmaf(v, c[j], __fmul_rn(u, s[j]));
    u = x;
  }
}

template <typename T, int V>
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
    if (sizeof(T) == 2) {
      // off by 2^-20.5 at most within +-pi: a five-hundredth of an fp16 half-step, at a tenth of the instructions
      __sincosf(half_turns * 3.14159265358979f, &sn, &cs);
    } else {
      sincospif(half_turns, &sn, &cs);
    }
    c[j] = cs * a.gain;
    s[j] = a.inverse ? -sn * a.gain : sn * a.gain;
  }
}

__device__ __forceinline__ float group_sum(float x, int tpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ void group_sum2(float& x, float& y, int tpr) {  // two chains at once
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) {
      const float p = __shfl_xor_sync(0xffffffffu, x, o), q = __shfl_xor_sync(0xffffffffu, y, o);
      x += p;
      y += q;
    }
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
__global__ void __launch_bounds__(kThreads, NU == 1 ? 4 : 2) rope_kernel(const RopeArgs a) {
  const RopeTensor& t = a.t[blockIdx.y];
  const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr;
  const unsigned tok = blockIdx.x * unsigned(kThreads / a.tpr) + group;
  const int h0 = blockIdx.z * a.hpg, h1 = min(t.H, h0 + a.hpg);
  const bool live = tok < unsigned(a.B) * unsigned(a.N);
  const int b = live ? int(tok / unsigned(a.N)) : 0, n = live ? int(tok - unsigned(b) * unsigned(a.N)) : 0;
  int ea[NU], eb[NU];
  bool on[NU];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = lane + k * a.tpr;
    on[k] = live && 2 * u * V < a.d;
    unit_offsets<V, HALF>(u, a.rot, ea[k], eb[k]);
  }
  const T* x = static_cast<const T*>(t.x) + b * t.xb + n * t.xn + h0 * t.xh;  // of the next head to fetch
  T* y = static_cast<T*>(t.y) + b * t.yb + n * t.yn + h0 * t.yh;              // of the next head to store
  constexpr int kAhead = NU > 1 ? 1 : sizeof(T) == 2 ? 4 : 2;  // heads in flight
  Chunk<T, V> ra[kAhead][NU], rb[kAhead][NU];
  auto fetch = [&](int h, int q) {
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (on[k] && h < h1) {
        ra[q][k] = fetch_chunk<T, V>(x + ea[k]);
        rb[q][k] = fetch_chunk<T, V>(x + eb[k]);
      }
    x += t.xh;
  };
#pragma unroll
  for (int q = 0; q < kAhead; ++q) fetch(h0 + q, q);
  // the first heads' values are on their way while the sines are formed
  // NORM: the weights go into the pairs' factors, u (w_u c) - v (w_v s) and v (w_v c) + u (w_u s);
  // behind the rotated part, c and cv are the weights
  float c[NU][V], s[NU][V], cv[NORM ? NU : 1][V], sv[NORM ? NU : 1][V];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = lane + k * a.tpr;
    const bool turns = on[k] && 2 * u * V < a.rot;
    if (turns) angles<T, V>(a, b, n, u, c[k], s[k]);
    if (NORM && on[k]) {
      float wa[V], wb[V];
      load_weight<V>(a, t.w, ea[k], eb[k], wa, wb);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float wu = first<V, HALF>(wa, wb, j), wv = second<V, HALF>(wa, wb, j);
        const float cj = turns ? c[k][j] : 1.0f, sj = turns ? s[k][j] : 0.0f;
        c[k][j] = wu * cj;
        cv[k][j] = wv * cj;
        s[k][j] = wv * sj;
        sv[k][j] = wu * sj;
      }
    }
  }
  for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (h + q >= h1) break;  // uniform over the block
      float va[NU][V], vb[NU][V];
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (on[k]) {
          widen(ra[q][k], va[k]);
          widen(rb[q][k], vb[k]);
        }
      fetch(h + q + kAhead, q);
      float r = 1.0f;
      if (NORM) {
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (on[k]) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += va[k][j] * va[k][j] + vb[k][j] * vb[k][j];
          }
        sum = group_sum(sum, a.tpr);
        r = rsqrtf(sum * a.inv_d + a.eps);
      }
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (on[k]) {
          const bool turns = 2 * (lane + k * a.tpr) * V < a.rot;
          if (!NORM) {
            if (turns) rotate<V, HALF>(va[k], vb[k], c[k], s[k]);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              float &u = first<V, HALF>(va[k], vb[k], j), &v = second<V, HALF>(va[k], vb[k], j);
              float x = u * c[k][j], y = v * cv[k][j];
              if (turns) {  // no 0 x inf where nothing turns
                x -= v * s[k][j];
                y += u * sv[k][j];
              }
              u = x * r;
              v = y * r;
            }
          }
          store_chunk(y + ea[k], va[k]);
          store_chunk(y + eb[k], vb[k]);
        }
      y += t.yh;
    }
  }
}

// Gradients of the norm with the rotation behind it. With g = the rotation of
// dy backwards, xh = x r, r = 1 / sqrt(mean(x^2) + eps):
//   dw = sum over tokens and heads of g xh,
//   dx = r (g w - xh mean(g w xh)).
// One round of blocks, shared between q and k by their heads, walks over token
// tiles; each block keeps its dw in registers and leaves one row of partial sums,
// which norm_dw_kernel adds in a fixed order.
// Bound: latency, neither HBM nor issue by itself: of each head a block waits for its loads and
// for two chains of shuffles, with 24 warps to an SM. Measured, queries and keys of 32760 tokens,
// 12 heads of 128: 146 us, 4.1 TB/s (600 MB that it reads and writes; 63 % of a copy's rate), 58 %
// of the issue slots.
template <typename T, int V, int NU, bool HALF>
__global__ void __launch_bounds__(kThreads, NU == 1 ? 3 : 1) norm_rope_bwd_kernel(const RopeArgs a) {
  extern __shared__ float dw_sh[];  // [groups][d]
  asm volatile("griddepcontrol.launch_dependents;");  // the sum's launch runs behind this kernel
  const int tensor = int(blockIdx.x) < a.split ? 0 : 1;
  const unsigned block = tensor == 0 ? blockIdx.x : blockIdx.x - a.split;
  const unsigned blocks = tensor == 0 ? a.split : gridDim.x - a.split;
  const RopeTensor& t = a.t[tensor];
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
  const int h1 = t.H;
  for (unsigned tile = block; tile < tiles; tile += blocks) {
    const unsigned tok = tile * groups + group;
    const bool live = tok < total;
    const int b = live ? int(tok / unsigned(a.N)) : 0, n = live ? int(tok - unsigned(b) * unsigned(a.N)) : 0;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + n * t.xn;
    const T* dy = static_cast<const T*>(t.dy) + b * t.gb + n * t.gn;
    T* dx = static_cast<T*>(t.y) + b * t.yb + n * t.yn;
    constexpr int kAhead = NU == 1 && sizeof(T) == 2 ? 2 : 1;  // heads in flight
    Chunk<T, V> rx[kAhead][NU][2], rg[kAhead][NU][2];
    auto fetch = [&](int h, int q) {
#pragma unroll
      for (int k = 0; k < NU; ++k)
        if (live && has[k] && h < h1) {
          rx[q][k][0] = fetch_chunk<T, V>(x + ea[k]);
          rx[q][k][1] = fetch_chunk<T, V>(x + eb[k]);
          rg[q][k][0] = fetch_chunk<T, V>(dy + ea[k]);
          rg[q][k][1] = fetch_chunk<T, V>(dy + eb[k]);
        }
      x += t.xh;
      dy += t.gh;
    };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) fetch(q, q);
    float c[NU][V], s[NU][V];
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (live && has[k] && 2 * (lane + k * a.tpr) * V < a.rot) angles<T, V>(a, b, n, lane + k * a.tpr, c[k], s[k]);
    for (int h = 0; h < h1; h += kAhead) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (h + q >= h1) break;  // uniform over the block
        float xa[NU][V], xb[NU][V], ga[NU][V], gb[NU][V];
        float sxx = 0.0f, sgx = 0.0f;
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (live && has[k]) {
            widen(rx[q][k][0], xa[k]);
            widen(rx[q][k][1], xb[k]);
            widen(rg[q][k][0], ga[k]);
            widen(rg[q][k][1], gb[k]);
          }
        fetch(h + q + kAhead, q);
#pragma unroll
        for (int k = 0; k < NU; ++k)
          if (live && has[k]) {
            if (2 * (lane + k * a.tpr) * V < a.rot) rotate<V, HALF>(ga[k], gb[k], c[k], s[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              sxx += xa[k][j] * xa[k][j] + xb[k][j] * xb[k][j];
              sgx += wa[k][j] * (ga[k][j] * xa[k][j]) + wb[k][j] * (gb[k][j] * xb[k][j]);
            }
          }
        group_sum2(sxx, sgx, a.tpr);
        const float r = rsqrtf(sxx * a.inv_d + a.eps);
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
            store_chunk(dx + ea[k], xa[k]);
            store_chunk(dx + eb[k], xb[k]);
          }
        dx += t.yh;
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
    a.partial[size_t(blockIdx.x) * a.d + i] = sum;
  }
}

// dw[i] = sum of the blocks' partial rows, in a fixed order: 32 slices of rows per
// column, then the slices. One block per 32 columns of one tensor. Bound: latency
// (7.7 us by itself for 444 rows of 128; started beside the kernel before it).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const RopeArgs a, int rows) {
  __shared__ float part[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial rows are written
  void* dw = a.t[blockIdx.y].dw;
  const int from = blockIdx.y == 0 ? 0 : a.split, to = blockIdx.y == 0 ? a.split : rows;
  if (dw == nullptr) return;
  const int col = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  float sum = 0.0f;
  if (col < a.d)
#pragma unroll 8
    for (int r = from + slice; r < to; r += 32) sum += a.partial[size_t(r) * a.d + col];
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
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.d + 31) / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_dw_kernel, a, int(grid.x));
}

// Values per chunk: 4 where the pair layout, the strides and the addresses allow them, else 1.
int chunk_width(const RopeArgs& a, int tensors, bool bwd) {
  const int size = a.dtype == SLA_FP32 ? 4 : 2;
  constexpr int v = 4;
  bool ok = a.d % (2 * v) == 0 && a.rot % (2 * v) == 0;
  for (int i = 0; i < tensors; ++i) {
    const RopeTensor& t = a.t[i];
    auto fits = [&](const void* p, long long b, long long n, long long h) {
      return reinterpret_cast<uintptr_t>(p) % (size_t(v) * size) == 0 && b % v == 0 && n % v == 0 && h % v == 0;
    };
    ok = ok && fits(t.x, t.xb, t.xn, t.xh) && fits(t.y, t.yb, t.yn, t.yh) && (!bwd || fits(t.dy, t.gb, t.gn, t.gh));
  }
  return ok ? v : 1;
}

}  // namespace

// Blocks of the backward over both tensors: one round of three per SM; also the rows of partial sums.
int rope_bwd_blocks(long long tokens) {
  const long long most = 2 * ((tokens + 7) / 8);  // a block takes at least 8 tokens (32 lanes a row)
  return int(std::min<long long>(most, kRopeBwdBlocks));
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
  if (bwd) {
    const int blocks = rope_bwd_blocks(tokens);
    grid = dim3(blocks, 1, 1);
    a.split = std::max(1, std::min(blocks - 1, int((long long)blocks * a.t[0].H / (a.t[0].H + a.t[1].H))));
  }
#define SLA_ROPE(T)                                                                  \
  (v == 4 ? (bwd ? launch_bwd<T, 4, 1>(a, grid, s) : launch_fwd<T, 4, 1>(a, grid, s)) \
          : (bwd ? launch_bwd<T, 1, 4>(a, grid, s) : launch_fwd<T, 1, 4>(a, grid, s)))
  if (a.dtype == SLA_BF16) return SLA_ROPE(__nv_bfloat16);
  if (a.dtype == SLA_FP16) return SLA_ROPE(__half);
  return SLA_ROPE(float);
#undef SLA_ROPE
}

}  // namespace sla

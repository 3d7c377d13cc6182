// Arguments of the rotary-position kernels (rope_kernels.cu), filled by rope_api.cu.
#pragma once

#include "sla_internal.cuh"

namespace sla {

// One tensor of head rows: element (b, h, n, i) at base + b xb + h xh + n xn + i.
struct RopeTensor {
  const void *x, *dy, *w;  // input; upstream gradient (backward); norm weight (null: no norm)
  void* y;                 // output (backward: dx)
  void* dw;                // backward: [d] of the weights' type, or null
  long long xb, xn, xh, yb, yn, yh, gb, gn, gh;
  int H;
};

struct RopeArgs {
  RopeTensor t[2];
  int B, N, d, rot, dtype, half, inverse, w_f32;
  const unsigned long long* turns;  // [rot / 2] 2^64 f / 2 pi
  const unsigned char* axis;        // [rot / 2] or null (one axis)
  const void* pos;                  // int32 / int64 positions or null (0 .. N - 1)
  int pos64, n_axes;
  long long pos_axis, pos_b, pos_n;
  float gain, eps, inv_d;
  float* partial;  // backward: [blocks][d]
  // set by the launcher: lanes per head row, heads per lane group; backward: blocks of q, the rest are k's
  int tpr, hpg, split;
};

constexpr int kRopeBwdBlocks = 148 * 3;
int rope_bwd_blocks(long long tokens);
// Forward (rotation, or norm and rotation where t[i].w is set) or, with bwd, the norm's backward.
cudaError_t launch_rope(RopeArgs a, int tensors, bool bwd, cudaStream_t s);

}  // namespace sla

// Packed prompt attention: the plan (one block of bytes, the same on host and
// device) and the launchers.
#pragma once

#include "sla_internal.cuh"

namespace sla {

constexpr int kPromptTile = 128;  // packed query rows and keys per tile
constexpr int kPromptSms = 148;
constexpr int kPromptFew = 32;   // rows of an item that the single-token variant takes

// A packed query tile holds tpt = 128 / G whole tokens: row t G + g is token t,
// query head (key head) G + g. The G heads that share a key head so share its
// tiles, and single tokens fill a tile as far as they can.
struct PromptItem {
  int q0, nq;    // first query token (row of the packed tensor), tokens
  int k0, lk;    // first key row and number of keys of the sequence
  int pos0;      // causal: query token q0 + i sees keys 0 .. pos0 + i (full: unused)
  int head;      // key head
  int b0, b1;    // key blocks of 128 [b0, b1) that this item reads
  int slot;      // < 0: writes O itself; else the slot of its partial result
  int pad[3];
};
// Rows whose keys were split: slots first .. first + n - 1 are joined.
struct PromptJoin {
  int q0, nq, head, first, n, pad[3];
};
// A tile of 128 keys of one key head (dK, dV): the query tiles [t0, t1) of its sequence.
struct PromptKeys {
  int k0, lk;    // first key row of the sequence, its keys
  int q0, lq;    // first query token of the sequence, its tokens
  int block;     // key block
  int head;
  int t0, t1;
  int slot;      // < 0: writes dK and dV itself; else the slot of its partial sums
  int pad[3];
};
// A key tile whose query tiles were split: slots first .. first + n - 1 are added.
struct PromptKeysJoin {
  int row, nk;   // first key row, keys
  int head, first, n, pad[3];
};

struct PromptPlan {
  int status;  // device copy: the status word
  unsigned magic;
  int n_seq, Hq, Hkv, G, d, causal;
  float scale;
  int tiles;   // query tiles per forward item (1 or 2)
  int few;     // forward items have at most kPromptFew rows
  long long Tq, Tk;
  int n_items, n_joins, n_slots;
  int join_rows, join_parts;  // most rows of a joined item (up to its last live one), most parts
  // backward (all 0 in a plan without it)
  int n_keys, n_kjoins, n_kslots, n_rows, row_tiles;  // n_rows: dQ items, of row_tiles query tiles each
  unsigned long long items, joins, keys, kjoins, rows, total;  // byte offsets
};
constexpr unsigned kPromptMagic = 0x534c4131u;

struct PromptTensor {
  void* base;
  long long row, head;
};

struct PromptArgs {
  const PromptPlan* plan;     // host
  unsigned char* plan_dev;
  PromptTensor q, k, v, o;
  float* lse;                 // [Tq, Hq] or null
  void* rest;                 // [Tq, Hq, d] bf16 or null
  float* part;                // [slots][tiles 128][d] partial O
  float* part_lse;            // [slots][tiles 128], log2
};
struct PromptGradArgs {
  const PromptPlan* plan;
  unsigned char* plan_dev;
  PromptTensor q, k, v, o, dO, dq, dk, dv;
  const float* lse;   // [Tq, Hq]
  const void* rest;   // [Tq, Hq, d] bf16 or null
  float2* ld;         // [Hkv][Tq G]: (lse log2 e, rowsum dO O)
  float* part;        // [key slots][2][128][d] partial dK, dV
};
cudaError_t launch_prompt_backward(const PromptGradArgs& a, cudaStream_t s);
cudaError_t launch_prompt_forward(const PromptArgs& a, cudaStream_t s);

}  // namespace sla

// C ABI of the packed prompt attention (declared in include/sla.h): validation,
// the plan of work items, and the calls.
//
// The plan is made on the host because the lengths are known there: no kernel has
// to search for its sequence, the longest items start first (blocks are dispatched
// in order, so this is longest-processing-time scheduling over the SMs), and the
// keys of long caches are split where the rows alone would leave SMs idle.
#include <math.h>
#include <string.h>

#include <functional>
#include <queue>
#include <vector>

#include "prompt.cuh"

using namespace sla;

namespace {

constexpr long long kMostItems = 1LL << 22;

sla_status check_params(const sla_prompt_params* p) {
  if (p == nullptr || p->n_seq < 1 || p->len_q == nullptr) return SLA_ERR_INVALID_ARG;
  if (p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0) return SLA_ERR_INVALID_ARG;
  if ((p->causal != 0 && p->causal != 1) || (p->backward != 0 && p->backward != 1)) return SLA_ERR_INVALID_ARG;
  // 0: the default; tiny ones would make the backward's lse / scale overflow
  if (!(p->softmax_scale == 0.0f || p->softmax_scale >= 1e-30f) || isinf(p->softmax_scale)) return SLA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SLA_ERR_UNSUPPORTED;
  if (p->Hq / p->Hkv > 128 || p->Hq > 65535) return SLA_ERR_UNSUPPORTED;
  long long tq = 0, tk = 0;
  for (int i = 0; i < p->n_seq; ++i) {
    const int lq = p->len_q[i], lk = p->len_k ? p->len_k[i] : lq;
    if (lq < 0 || lk < 0) return SLA_ERR_INVALID_ARG;
    tq += lq;
    tk += lk;
  }
  if (tq < 1) return SLA_ERR_INVALID_ARG;
  // rows, positions and tile ends are 32-bit in the kernels
  if (tq > 0x7fffffffLL - 1024 || tk > 0x7fffffffLL - 1024) return SLA_ERR_UNSUPPORTED;
  // the plan's lists: at most 2^22 items each (200 MB)
  const int tpt = kPromptTile / (p->Hq / p->Hkv);
  long long rows = 0, keys = 0;
  for (int i = 0; i < p->n_seq; ++i) {
    rows += ((long long)p->len_q[i] + tpt - 1) / tpt;
    keys += ((long long)(p->len_k ? p->len_k[i] : p->len_q[i]) + kPromptTile - 1) / kPromptTile;
  }
  if (rows * p->Hkv > kMostItems || (p->backward && keys * p->Hkv > kMostItems)) return SLA_ERR_UNSUPPORTED;
  return SLA_OK;
}

struct Lists {
  std::vector<PromptItem> items, rows;
  std::vector<PromptJoin> joins;
  std::vector<PromptKeys> keys;
  std::vector<PromptKeysJoin> kjoins;
  int tiles = 2, slots = 0, row_tiles = 2, kslots = 0;
};

int key_blocks(const sla_prompt_params& p, int lq, int lk, int last_token) {
  const long long keys = p.causal ? std::min<long long>(lk, (long long)lk - lq + last_token + 1) : lk;
  return int((std::max(0LL, keys) + kPromptTile - 1) / kPromptTile);
}

long long row_item_count(const sla_prompt_params& p, int per) {
  long long n = 0;
  for (int s = 0; s < p.n_seq; ++s) n += ((long long)p.len_q[s] + per - 1) / per * p.Hkv;
  return n;
}

// Items of `per` tokens, all key blocks each.
std::vector<PromptItem> row_items(const sla_prompt_params& p, int per) {
  std::vector<PromptItem> out;
  out.reserve(size_t(row_item_count(p, per)));
  int q0 = 0, k0 = 0;
  for (int s = 0; s < p.n_seq; ++s) {
    const int lq = p.len_q[s], lk = p.len_k ? p.len_k[s] : lq;
    for (int t = 0; t < lq; t += per)
      for (int h = 0; h < p.Hkv; ++h) {
        PromptItem it{};
        it.q0 = q0 + t;
        it.nq = std::min(per, lq - t);
        it.k0 = k0;
        it.lk = lk;
        it.pos0 = lk - lq + t;
        it.head = h;
        it.b1 = key_blocks(p, lq, lk, t + it.nq - 1);
        it.slot = -1;
        out.push_back(it);
      }
    q0 += lq;
    k0 += lk;
  }
  return out;
}

// Longest first, equals in their order: a counting sort (plans are made per batch, and
// comparison sorts of their thousands of items were half of the time).
template <typename T, typename Length>
void longest_first(std::vector<T>& items, Length length) {
  int most = 0;
  for (const T& it : items) most = std::max(most, length(it));
  std::vector<int> at(size_t(most) + 2, 0);
  for (const T& it : items) ++at[size_t(most - length(it)) + 1];
  for (size_t i = 1; i < at.size(); ++i) at[i] += at[i - 1];
  std::vector<T> out(items.size());
  for (const T& it : items) out[size_t(at[size_t(most - length(it))]++)] = it;
  items.swap(out);
}

// Time at which the last of `places` ends, items dispatched longest first.
double makespan(std::vector<double> cost, int places) {
  std::sort(cost.begin(), cost.end(), std::greater<double>());
  if (int(cost.size()) <= places) return cost.empty() ? 0.0 : cost[0];
  std::priority_queue<double, std::vector<double>, std::greater<double>> sm;
  for (int i = 0; i < places; ++i) sm.push(0.0);
  double last = 0.0;
  for (double c : cost) {
    const double e = sm.top() + c;
    sm.pop();
    sm.push(e);
    last = std::max(last, e);
  }
  return last;
}

// Pieces that an item of n blocks is cut into for pieces of about `chunk` blocks.
int pieces(int n, int chunk) { return chunk <= 0 || n <= chunk ? 1 : (n + chunk - 1) / chunk; }

// The smallest chunk (of at least 4 blocks) that cuts items of these lengths into at most
// `most` pieces: pieces that fill whole rounds over the SMs' places and start no further one.
int chunk_for(const std::vector<int>& lengths, int most) {
  int lo = 4, hi = 4;
  for (int n : lengths) hi = std::max(hi, n);
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    long long parts = 0;
    for (int n : lengths) parts += pieces(n, mid);
    if (parts <= most)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Costs in units of one key block of a two-tile item, the only one on its SM.
constexpr double kItemCost = 3.0;  // start, first loads and the store
// The same for a two-tile item that the forward takes behind another one (measured, an item
// more of 1 to 16 blocks on every SM: 0.9 steps at d = 64, 1.5 at d = 128).
constexpr double kNextCost = 1.2;
constexpr double kJoinCost = 3.0;  // the second launch
// A step of a one-tile item, two of which share an SM, and of one that has its SM to
// itself. At d = 128 the second copy of the keys costs bandwidth to shared memory (4096
// causal tokens, 16 heads: 84 us as one-tile items, 60 as two-tile ones). At d = 64 the
// softmax bounds both, and the items' ends decide (8192 causal tokens, 16 heads: 188
// and 177 us; 4096: 63 and 52), or the last round (8192 full ones, whose two-tile items
// leave half of it idle, while the last one-tile items have an SM each: 357 and 417).
double one_tile_step(int d, bool shared) { return shared ? (d == 128 ? 1.4 : 1.02) : (d == 128 ? 0.9 : 0.7); }

// full_rows: how full of live rows the tiles are
// again: a CTA of two tiles takes item after item
double split_cost(const std::vector<PromptItem>& items, int chunk, int tiles, double full_rows, int d, bool again) {
  std::vector<double> cost;
  size_t parts = 0;
  for (const PromptItem& it : items) parts += pieces(it.b1, chunk);
  const bool shared = tiles == 1 && parts > size_t(kPromptSms);
  double joins = 0.0;  // rows of partial results, in tiles: written and read once more in float32
  for (const PromptItem& it : items) {
    const int n = pieces(it.b1, chunk);
    if (n > 1) joins += n * tiles;
    for (int i = 0; i < n; ++i) cost.push_back((it.b1 + n - 1) / n);
  }
  // the longest first, as they are handed out
  std::sort(cost.begin(), cost.end(), std::greater<double>());
  // one-tile items: of the last round's, those that share their SM
  const size_t left = cost.size() % (2 * kPromptSms);
  const double paired = left <= size_t(kPromptSms) ? 0.0 : 2.0 * (left - kPromptSms) / left;
  const double both = one_tile_step(d, true), last = paired * both + (1.0 - paired) * one_tile_step(d, false);
  for (size_t i = 0; i < cost.size(); ++i) {
    const double step = tiles == 2 ? 1.0 : i < cost.size() - left ? both : last;
    cost[i] = (again && tiles == 2 && i >= size_t(kPromptSms) ? kNextCost : kItemCost) + step * cost[i];
  }
  return makespan(cost, shared ? 2 * kPromptSms : kPromptSms) + (joins > 0.0 ? kJoinCost + full_rows * joins / kPromptSms : 0.0);
}

void add_backward(const sla_prompt_params& p, Lists& L);

Lists make_lists(const sla_prompt_params& p) {
  Lists L;
  const int G = p.Hq / p.Hkv, tpt = kPromptTile / G;
  int longest = 0;
  for (int s = 0; s < p.n_seq; ++s) longest = std::max(longest, p.len_q[s]);
  // Two tiles share every key tile and hide each other's softmax; one tile per
  // item spreads little work over more SMs. Few items may also split their keys.
  double best = 0.0;
  int best_chunk = 0;
  std::vector<PromptItem> base;
  for (int tiles = longest <= tpt ? 1 : 2; tiles >= 1; --tiles) {
    std::vector<PromptItem> items = row_items(p, tiles * tpt);
    if (base.empty() && items.size() >= 4 * kPromptSms && (tiles == 1 || items.size() >= 8 * kPromptSms)) {
      // rounds enough: neither splits nor smaller items can be better
      base = std::move(items);
      L.tiles = tiles;
      break;
    }
    std::vector<int> chunks = {0};
    if (items.size() < 4 * kPromptSms) {
      std::vector<int> lengths;
      for (const PromptItem& it : items) lengths.push_back(it.b1);
      for (int rounds = 1; rounds <= 3; ++rounds) chunks.push_back(chunk_for(lengths, rounds * kPromptSms * (3 - tiles)));
    }
    for (int chunk : chunks) {
      const double c = split_cost(items, chunk, tiles, std::min(1.0, double(longest) / tpt), p.d, true);
      if (base.empty() || c < best) {
        best = c;
        best_chunk = chunk;
        base = items;
        L.tiles = tiles;
      }
    }
    if (items.size() >= 4 * kPromptSms) break;  // enough two-tile items: one tile each cannot be better
  }
  for (const PromptItem& it : base) {
    const int n = pieces(it.b1, best_chunk);
    if (n == 1) {
      L.items.push_back(it);
      continue;
    }
    L.joins.push_back(PromptJoin{it.q0, it.nq, it.head, L.slots, n, {}});
    for (int i = 0; i < n; ++i) {
      PromptItem part = it;
      part.b0 = int((long long)it.b1 * i / n);
      part.b1 = int((long long)it.b1 * (i + 1) / n);
      part.slot = L.slots++;
      L.items.push_back(part);
    }
  }
  longest_first(L.items, [](const PromptItem& it) { return it.b1 - it.b0; });
  if (p.backward) add_backward(p, L);
  return L;
}

// Backward: dQ items like the forward's, and one item per key tile, whose query
// tiles are split where few key tiles see many of them.
void add_backward(const sla_prompt_params& p, Lists& L) {
  const int G = p.Hq / p.Hkv, tpt = kPromptTile / G;
  double best = 0.0;
  for (int tiles = 2; tiles >= 1; --tiles) {
    const long long count = row_item_count(p, tiles * tpt);
    if (tiles == 1 && count >= 8 * kPromptSms) break;
    std::vector<PromptItem> rows = row_items(p, tiles * tpt);
    if (tiles == 2 && count >= 4 * kPromptSms) {  // rounds enough for two tiles each
      L.rows = std::move(rows);
      L.row_tiles = 2;
      break;
    }
    const double c = split_cost(rows, 0, 2, 1.0, p.d, false) * (tiles == 2 ? 1.0 : 0.8);  // one CTA per SM either way
    if (tiles == 2 || c < best) {
      best = c;
      L.rows = std::move(rows);
      L.row_tiles = tiles;
    }
  }
  longest_first(L.rows, [](const PromptItem& it) { return it.b1; });

  std::vector<PromptKeys> base;
  int q0 = 0, k0 = 0;
  for (int s = 0; s < p.n_seq; ++s) {
    const int lq = p.len_q[s], lk = p.len_k ? p.len_k[s] : lq;
    const int tiles = (lq + tpt - 1) / tpt;
    for (int b = 0; b < (lk + kPromptTile - 1) / kPromptTile; ++b)
      for (int h = 0; h < p.Hkv; ++h) {
        // the first query that sees the block's first key
        const long long first = p.causal ? std::max(0LL, (long long)b * kPromptTile - (lk - lq)) : 0;
        PromptKeys it{};
        it.k0 = k0;
        it.lk = lk;
        it.q0 = q0;
        it.lq = lq;
        it.block = b;
        it.head = h;
        it.t0 = int(std::min<long long>(tiles, first / tpt));
        it.t1 = tiles;
        it.slot = -1;
        base.push_back(it);
      }
    q0 += lq;
    k0 += lk;
  }
  std::vector<int> chunks = {0};
  if (base.size() < 4 * kPromptSms) {
    std::vector<int> lengths;
    for (const PromptKeys& it : base) lengths.push_back(it.t1 - it.t0);
    for (int rounds = 1; rounds <= 3; ++rounds) chunks.push_back(chunk_for(lengths, rounds * kPromptSms));
  }
  int chunk = 0;
  best = -1.0;
  for (int c : chunks) {
    if (chunks.size() == 1) break;
    std::vector<double> cost;
    bool any = false;
    for (const PromptKeys& it : base) {
      const int n = pieces(it.t1 - it.t0, c);
      any = any || n > 1;
      for (int i = 0; i < n; ++i) cost.push_back(kItemCost + double((it.t1 - it.t0 + n - 1) / n));
    }
    const double m = makespan(cost, kPromptSms) + (any ? kJoinCost : 0.0);
    if (best < 0.0 || m < best) {
      best = m;
      chunk = c;
    }
  }
  for (const PromptKeys& it : base) {
    const int len = it.t1 - it.t0, n = pieces(len, chunk);
    if (n == 1) {
      L.keys.push_back(it);
      continue;
    }
    L.kjoins.push_back(PromptKeysJoin{it.k0 + it.block * kPromptTile, std::min(kPromptTile, it.lk - it.block * kPromptTile),
                                      it.head, L.kslots, n, {}});
    for (int i = 0; i < n; ++i) {
      PromptKeys part = it;
      part.t0 = it.t0 + int((long long)len * i / n);
      part.t1 = it.t0 + int((long long)len * (i + 1) / n);
      part.slot = L.kslots++;
      L.keys.push_back(part);
    }
  }
  longest_first(L.keys, [](const PromptKeys& it) { return it.t1 - it.t0; });
}

size_t layout(const sla_prompt_params& p, const Lists& L, PromptPlan* h) {
  memset(h, 0, sizeof(*h));
  h->magic = kPromptMagic;
  h->n_seq = p.n_seq;
  h->Hq = p.Hq;
  h->Hkv = p.Hkv;
  h->G = p.Hq / p.Hkv;
  h->d = p.d;
  h->causal = p.causal;
  h->scale = p.softmax_scale > 0.0f ? p.softmax_scale : 1.0f / sqrtf(float(p.d));
  h->tiles = L.tiles;
  int longest = 0;
  for (int i = 0; i < p.n_seq; ++i) longest = std::max(longest, p.len_q[i]);
  h->few = L.tiles == 1 && (long long)longest * h->G <= kPromptFew;
  for (int i = 0; i < p.n_seq; ++i) {
    h->Tq += p.len_q[i];
    h->Tk += p.len_k ? p.len_k[i] : p.len_q[i];
  }
  h->n_items = int(L.items.size());
  h->n_joins = int(L.joins.size());
  h->n_slots = L.slots;
  for (const PromptJoin& j : L.joins) {
    const int tpt = kPromptTile / h->G;
    h->join_parts = std::max(h->join_parts, j.n);
    h->join_rows = std::max(h->join_rows, j.nq > tpt ? kPromptTile + (j.nq - tpt) * h->G : j.nq * h->G);
  }
  h->n_keys = int(L.keys.size());
  h->n_kjoins = int(L.kjoins.size());
  h->n_kslots = L.kslots;
  h->n_rows = int(L.rows.size());
  h->row_tiles = L.row_tiles;
  size_t off = align256(sizeof(PromptPlan));
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  h->items = take(L.items.size() * sizeof(PromptItem));
  h->joins = take(L.joins.size() * sizeof(PromptJoin));
  h->keys = take(L.keys.size() * sizeof(PromptKeys));
  h->kjoins = take(L.kjoins.size() * sizeof(PromptKeysJoin));
  h->rows = take(L.rows.size() * sizeof(PromptItem));
  h->total = off;
  return off;
}

sla_status write_plan(const sla_prompt_params& p, unsigned char* out, size_t bytes) {
  const Lists L = make_lists(p);
  PromptPlan h;
  if (bytes < layout(p, L, &h)) return SLA_ERR_WORKSPACE;
  memset(out, 0, h.total);
  memcpy(out, &h, sizeof(h));
  auto put = [&](size_t at, const void* src, size_t size) {
    if (size) memcpy(out + at, src, size);
  };
  put(h.items, L.items.data(), L.items.size() * sizeof(PromptItem));
  put(h.joins, L.joins.data(), L.joins.size() * sizeof(PromptJoin));
  put(h.keys, L.keys.data(), L.keys.size() * sizeof(PromptKeys));
  put(h.kjoins, L.kjoins.data(), L.kjoins.size() * sizeof(PromptKeysJoin));
  put(h.rows, L.rows.data(), L.rows.size() * sizeof(PromptItem));
  return SLA_OK;
}

const PromptPlan* plan_of(const void* plan, size_t bytes) {
  if (plan == nullptr || reinterpret_cast<uintptr_t>(plan) % 8 != 0 || bytes < sizeof(PromptPlan)) return nullptr;
  const PromptPlan* p = static_cast<const PromptPlan*>(plan);
  return p->magic == kPromptMagic && p->total <= bytes ? p : nullptr;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Address, strides (TMA: multiples of 16 bytes, below 2^40) and, for outputs, distinct rows.
sla_status check_rows(const sla_rows* t, long long T, int H, int d, bool output, PromptTensor* out) {
  if (t == nullptr || t->base == nullptr) return SLA_ERR_INVALID_ARG;
  long long row = T > 1 ? t->row : (long long)d * H, head = H > 1 ? t->head : (long long)d;
  if (row <= 0 || head <= 0) return SLA_ERR_INVALID_ARG;
  if (row >= (1LL << 38) || head >= (1LL << 31)) return SLA_ERR_UNSUPPORTED;
  if (output) {
    const bool heads_inside = head >= d && (T == 1 || row >= head * (H - 1) + d);
    const bool rows_inside = row >= d && (H == 1 || head >= row * (T - 1) + d);
    if (!heads_inside && !rows_inside) return SLA_ERR_INVALID_ARG;
  }
  if (!aligned(t->base, 16) || row % 8 != 0 || head % 8 != 0) return SLA_ERR_ALIGNMENT;
  *out = PromptTensor{t->base, row, head};
  return SLA_OK;
}

size_t forward_workspace(const PromptPlan& p) {
  return p.n_slots == 0 ? 0 : align256(size_t(p.n_slots) * p.tiles * 128 * (size_t(p.d) + 1) * sizeof(float));
}

size_t backward_workspace(const PromptPlan& p) {
  return align256(size_t(p.Tq) * p.Hq * sizeof(float2)) + size_t(p.n_kslots) * 2 * 128 * p.d * sizeof(float);
}

sla_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SLA_OK;
  return ws == nullptr || !aligned(ws, 256) || have < need ? SLA_ERR_WORKSPACE : SLA_OK;
}

}  // namespace

extern "C" {

sla_status sla_prompt_validate(const sla_prompt_params* p) { return check_params(p); }

size_t sla_prompt_plan_size(const sla_prompt_params* p) {
  if (check_params(p) != SLA_OK) return 0;
  // an upper bound: every list at its longest (a split makes at most three rounds of pieces)
  const int tpt = kPromptTile / (p->Hq / p->Hkv);
  const size_t rows = size_t(row_item_count(*p, tpt)), parts = 6 * kPromptSms;
  size_t n = 6 * 256 + align256(sizeof(PromptPlan)) + std::max(rows, parts) * sizeof(PromptItem) +
             std::min(rows, parts) * sizeof(PromptJoin);
  if (p->backward) {
    size_t keys = 0;
    for (int i = 0; i < p->n_seq; ++i) {
      const size_t lk = size_t(p->len_k ? p->len_k[i] : p->len_q[i]);
      keys += (lk + kPromptTile - 1) / kPromptTile * p->Hkv;
    }
    n += std::max(keys, parts) * sizeof(PromptKeys) + std::min(keys, parts) * sizeof(PromptKeysJoin) +
         rows * sizeof(PromptItem);
  }
  return align256(n);
}

size_t sla_prompt_plan_used(const void* plan) {
  const PromptPlan* p = plan_of(plan, ~size_t(0));
  return p == nullptr ? 0 : size_t(p->total);
}

sla_status sla_prompt_plan(const sla_prompt_params* p, void* plan, size_t plan_bytes) {
  const sla_status st = check_params(p);
  if (st != SLA_OK) return st;
  if (plan == nullptr) return SLA_ERR_INVALID_ARG;
  if (!aligned(plan, 8)) return SLA_ERR_ALIGNMENT;
  try {  // the lists are host memory: running out of it must not pass this C boundary as an exception
    return write_plan(*p, static_cast<unsigned char*>(plan), plan_bytes);
  } catch (...) {
    return SLA_ERR_WORKSPACE;
  }
}

size_t sla_prompt_workspace_size(const void* plan) {
  const PromptPlan* p = plan_of(plan, ~size_t(0));
  return p == nullptr ? 0 : forward_workspace(*p);
}

sla_status sla_prompt_forward(const sla_rows* q, const sla_rows* k, const sla_rows* v, const sla_rows* o, float* lse,
                              void* rest, const void* plan, size_t plan_bytes, void* plan_device, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const PromptPlan* p = plan_of(plan, plan_bytes);
  if (p == nullptr || plan_device == nullptr) return SLA_ERR_INVALID_ARG;
  PromptArgs a{};
  sla_status st = check_rows(q, p->Tq, p->Hq, p->d, false, &a.q);
  if (st == SLA_OK) st = check_rows(o, p->Tq, p->Hq, p->d, true, &a.o);
  if (st == SLA_OK && p->Tk > 0) st = check_rows(k, p->Tk, p->Hkv, p->d, false, &a.k);
  if (st == SLA_OK && p->Tk > 0) st = check_rows(v, p->Tk, p->Hkv, p->d, false, &a.v);
  if (st != SLA_OK) return st;
  if (!aligned(plan_device, 256) || !aligned(lse, 4) || !aligned(rest, 16)) return SLA_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, forward_workspace(*p));
  if (st != SLA_OK) return st;
  a.plan = p;
  a.plan_dev = static_cast<unsigned char*>(plan_device);
  a.lse = lse;
  a.rest = rest;
  a.part = static_cast<float*>(workspace);
  a.part_lse = a.part + size_t(p->n_slots) * p->tiles * 128 * p->d;
  return launch_prompt_forward(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

size_t sla_prompt_backward_workspace_size(const void* plan) {
  const PromptPlan* p = plan_of(plan, ~size_t(0));
  return p == nullptr || p->n_rows == 0 ? 0 : backward_workspace(*p);
}

sla_status sla_prompt_backward(const sla_rows* q, const sla_rows* k, const sla_rows* v, const sla_rows* o,
                               const float* lse, const void* rest, const sla_rows* dO, const sla_rows* dq, const sla_rows* dk,
                               const sla_rows* dv, const void* plan, size_t plan_bytes, void* plan_device,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const PromptPlan* p = plan_of(plan, plan_bytes);
  if (p == nullptr || plan_device == nullptr || lse == nullptr) return SLA_ERR_INVALID_ARG;
  if (p->n_rows == 0) return SLA_ERR_UNSUPPORTED;  // planned without the backward
  PromptGradArgs a{};
  sla_status st = check_rows(q, p->Tq, p->Hq, p->d, false, &a.q);
  if (st == SLA_OK) st = check_rows(o, p->Tq, p->Hq, p->d, false, &a.o);
  if (st == SLA_OK) st = check_rows(dO, p->Tq, p->Hq, p->d, false, &a.dO);
  if (st == SLA_OK) st = check_rows(dq, p->Tq, p->Hq, p->d, true, &a.dq);
  if (p->Tk > 0) {
    if (st == SLA_OK) st = check_rows(k, p->Tk, p->Hkv, p->d, false, &a.k);
    if (st == SLA_OK) st = check_rows(v, p->Tk, p->Hkv, p->d, false, &a.v);
    if (st == SLA_OK) st = check_rows(dk, p->Tk, p->Hkv, p->d, true, &a.dk);
    if (st == SLA_OK) st = check_rows(dv, p->Tk, p->Hkv, p->d, true, &a.dv);
  }
  if (st != SLA_OK) return st;
  if (!aligned(plan_device, 256) || !aligned(lse, 4) || !aligned(rest, 16)) return SLA_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, backward_workspace(*p));
  if (st != SLA_OK) return st;
  a.plan = p;
  a.plan_dev = static_cast<unsigned char*>(plan_device);
  a.lse = lse;
  a.rest = rest;
  a.ld = static_cast<float2*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                    align256(size_t(p->Tq) * p->Hq * sizeof(float2)));
  return launch_prompt_backward(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SLA_OK : SLA_ERR_CUDA;
}

}  // extern "C"

// Shared parts of the prefill kernels: arguments, which tile a CTA works on,
// the keys a tile attends, and the checks of a sequence.
//
// Method: out = softmax(alpha * RoPE(q) K^T) V over a causal, optionally
// windowed range of keys, read from packed codes through a block table
// ([airllm] §2.2, §2.3, §3.4; [Shimmy] §2.3 for the rotation and the scale;
// [Fieldfare] "KV Cache 的双布局设计" for the ring and the window).
//
// A query tile is TQ consecutive query tokens of one sequence with all G heads
// of one kv head: TQ * G rows, row r = token r / G, head r % G, so the tile's
// keys are dequantized once for all of them.
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

struct PrefillArgs {
  const void* q;
  const int32_t* q_starts;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* rope_tab;
  void* out;
  float* ws_acc;     // [n_splits][n_rows][n_heads][head_dim] partial sums
  float2* ws_ml;     // [n_splits][n_rows][n_heads] partial (max, sum), base 2
  int32_t* status;
  int32_t batch, n_rows, n_heads, n_kv_heads, n_pool_pages, max_pages, rope_max_pos;
  int32_t ring_rows, pin_rows, window, sinks;
  int32_t act, rope;
  int32_t tq;          // query tokens per tile
  int32_t n_tiles;     // tiles of the grid: at least one for every tile of every sequence
  int32_t n_splits;    // key splits per tile
  float score_scale;   // alpha * log2(e)
  PoolLayout kl, vl;
};

// What a CTA works on: query tokens [t0, t0 + cnt) of sequence b, whose first
// has position p0; row0 is the row of q and out of token t0.
struct PrefillTile {
  int b, row0, cnt, p0;
  bool zero;   // a sequence with a bad length: its rows are zero
};

// The keys a tile attends, as tiles of TN tokens: n1 tiles of the sinks [0,
// end1), then tiles from lo2 (a page boundary) to end2.
struct KeyRange {
  int n1, n, end1, lo2, end2;
  template <int TN>
  __device__ __forceinline__ int base(int j) const { return j < n1 ? j * TN : lo2 + (j - n1) * TN; }
  __device__ __forceinline__ int end(int j) const { return j < n1 ? end1 : end2; }
};

// Finds tile x of the grid.  The tiles of sequence b start at x = q_starts[b]
// / TQ + b: floor((s + n) / TQ) + 1 - floor(s / TQ) >= ceil(n / TQ), so they
// never run into the next sequence's, and no prefix sum is needed.  False: no
// such tile, or a sequence that is left out (its bit set).
__device__ __forceinline__ bool find_tile(const PrefillArgs& a, int x, bool reporter, PrefillTile* t) {
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {   // the last b whose tiles start at or before x
    const int mid = (lo + hi + 1) / 2;
    if (a.q_starts[mid] / a.tq + mid <= x) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  const int s0 = a.q_starts[b], s1 = a.q_starts[b + 1], L = a.seq_lens[b];
  if (s0 < 0 || s1 < s0 || s1 > a.n_rows) {
    if (reporter) report(a.status, KVQ_DEV_BAD_SEQ);
    return false;
  }
  const int n = s1 - s0;
  const int i = x - (s0 / a.tq + b);
  if (i < 0 || (int64_t)i * a.tq >= n) return false;
  int bad = 0;
  // (a position past the last whole step of 2^31 tokens would overflow)
  if (L < n || L > INT_MAX - 1024 || (a.ring_rows == 0 && L > (int64_t)a.max_pages * 16)) {
    bad = KVQ_DEV_BAD_LEN;
  } else if (a.rope != KVQ_ROPE_NONE && L > a.rope_max_pos) {
    bad = KVQ_DEV_BAD_POS;
  } else if (a.ring_rows > 0) {   // every ring token the first query attends is still there
    const int first = max(L - n - a.window + 1, a.pin_rows);
    if (L - first > a.ring_rows) bad = KVQ_DEV_BAD_LEN;
  }
  if (bad && reporter) report(a.status, bad);
  t->b = b;
  t->zero = bad != 0;
  t->row0 = s0 + i * a.tq;
  t->cnt = min(a.tq, n - i * a.tq);
  t->p0 = L - n + i * a.tq;
  return true;
}

// q_starts out of order can hide a sequence from every tile: one thread block
// of the grid looks at them all.
__device__ __forceinline__ void check_starts(const PrefillArgs& a, int tid, int threads) {
  for (int b = tid; b < a.batch; b += threads) {
    const int s0 = a.q_starts[b], s1 = a.q_starts[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > a.n_rows) report(a.status, KVQ_DEV_BAD_SEQ);
  }
}

template <int TN>
__device__ __forceinline__ KeyRange key_range(const PrefillArgs& a, const PrefillTile& t) {
  KeyRange k;
  const int lo = a.window > 0 ? max(0, t.p0 - a.window + 1) : 0;
  const int sk = min(a.sinks, lo);
  k.end2 = t.p0 + t.cnt;
  k.lo2 = lo & ~15;
  k.end1 = sk;
  k.n1 = (sk + TN - 1) / TN;
  if (k.n1 > 0 && k.n1 * TN >= k.lo2) {   // the sinks' tiles reach the window: one run from 0
    k.n1 = 0;
    k.lo2 = 0;
  }
  k.n = k.n1 + (k.end2 - k.lo2 + TN - 1) / TN;
  return k;
}

// Whether the query at position p attends key t <= p.
__device__ __forceinline__ bool in_window(const PrefillArgs& a, int p, int t) {
  return a.window == 0 || t > p - a.window || t < a.sinks;
}

// 16 elements of a stored row, the kind known at run time only.
__device__ __forceinline__ void read16_any(const uint8_t* sub, const PoolLayout& L, int slot, int u, float (&x)[16]) {
  switch (L.kind) {
    case KVQ_SYM_INT4: return read16<KVQ_SYM_INT4>(sub, L, slot, u, x);
    case KVQ_SYM_INT8: return read16<KVQ_SYM_INT8>(sub, L, slot, u, x);
    case KVQ_AFFINE_INT4: return read16<KVQ_AFFINE_INT4>(sub, L, slot, u, x);
    case KVQ_SHIMMY_INT4: return read16<KVQ_SHIMMY_INT4>(sub, L, slot, u, x);
    default: return read16<KVQ_F16_KV>(sub, L, slot, u, x);
  }
}

}  // namespace kvq

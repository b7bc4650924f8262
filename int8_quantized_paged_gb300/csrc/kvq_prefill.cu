// Prefill attention: entry points, the plan of tiles and key splits, the fp32
// kernel and the combine of key splits.
//
// The fp32 kernel takes every config; the tensor-core kernel
// (kvq_prefill_tc.cu) takes f16 and bf16 activations.  When the query tiles
// alone do not fill the GPU, the keys of a tile are split over several CTAs,
// each of which leaves (m, l, acc) of its part in the workspace; the combine
// kernel merges them with log-sum-exp weights,
//   M = max_s m_s;  out = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s.
#include <cuda_runtime.h>

#include "kvq_prefill.cuh"
#include "kvq_prefill_tc.h"

namespace kvq {

// ---------------------------------------------------------------- fp32 kernel
// 64 rows x 32 keys a step, 256 threads: thread (ty, tx) holds rows 4 ty .. +3,
// the scores of keys tx and tx + 16, and the outputs 4 tx + 64 c .. +3.  K^ and
// V^ of the 32 keys are dequantized into shared memory once for the 64 rows.
// Bound by the fp32 multiply-adds and the shared-memory reads that feed them:
// 31 TFLOP/s of causal products for an 8K prompt of 32 heads of 128; a
// 100-token prompt of the smallest layer, 17 us, by the latency of its steps.
constexpr int kSimtRows = 64, kSimtKeys = 32, kSimtThreads = 256;

template <int HD>
constexpr size_t simt_smem() {
  return sizeof(float) * ((size_t)kSimtRows * (HD + 4) + 2 * (size_t)kSimtKeys * (HD + 4) +
                          (size_t)kSimtRows * (kSimtKeys + 1)) + kSimtKeys * sizeof(int);
}

template <int HD>
__global__ void __launch_bounds__(kSimtThreads) prefill_simt_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int P = 16, M = kSimtRows, N = kSimtKeys, LD = HD + 4, C = HD / 64;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                 // [M][LD]
  float* ks = qs + M * LD;        // [N][LD]
  float* vs = ks + N * LD;        // [N][LD]
  float* ps = vs + N * LD;        // [M][N + 1]
  int* state = reinterpret_cast<int*>(ps + M * (N + 1));   // [N]: 0 fine, 1 not finite, 2 left out

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int kvh = blockIdx.y, split = blockIdx.z;
  const int G = a.n_heads / a.n_kv_heads;
  if (blockIdx.x == 0 && kvh == 0 && split == 0) check_starts(a, tid, kSimtThreads);
  PrefillTile t;
  if (!find_tile(a, a.n_tiles - 1 - blockIdx.x, kvh == 0 && split == 0 && tid == 0, &t)) return;
  const int rows = t.cnt * G;
  auto out_row = [&](int r) -> int64_t {   // (query row, head) of tile row r, flattened
    return (int64_t)(t.row0 + r / G) * a.n_heads + kvh * G + r % G;
  };
  if (t.zero) {
    if (split == 0)
      for (int i = tid; i < rows * HD; i += kSimtThreads) store_act(a.out, a.act, out_row(i / HD) * HD + i % HD, 0.f);
    if (a.n_splits > 1)
      for (int r = tid; r < rows; r += kSimtThreads)
        a.ws_ml[(int64_t)split * a.n_rows * a.n_heads + out_row(r)] = make_float2(-INFINITY, 0.f);
    return;
  }

  // the queries, rotated and scaled; rows past the tile are zero
  for (int i = tid; i < M * (HD / 2); i += kSimtThreads) {
    const int r = i / (HD / 2), pi = i % (HD / 2);
    const int d0 = a.rope == KVQ_ROPE_NEOX ? pi : 2 * pi;
    const int d1 = a.rope == KVQ_ROPE_NEOX ? pi + HD / 2 : 2 * pi + 1;
    float x0 = 0.f, x1 = 0.f;
    if (r < rows) {
      const int64_t at = out_row(r) * HD;
      x0 = load_act(a.q, a.act, at + d0);
      x1 = load_act(a.q, a.act, at + d1);
      if (a.rope != KVQ_ROPE_NONE) {
        const float2 cs = reinterpret_cast<const float2*>(a.rope_tab)[(int64_t)(t.p0 + r / G) * (HD / 2) + pi];
        const float y0 = x0 * cs.x - x1 * cs.y;
        x1 = x0 * cs.y + x1 * cs.x;
        x0 = y0;
      }
    }
    qs[r * LD + d0] = x0 * a.score_scale;
    qs[r * LD + d1] = x1 * a.score_scale;
  }

  const KeyRange kr = key_range<N>(a, t);
  const int j0 = (int)((int64_t)split * kr.n / a.n_splits), j1 = (int)((int64_t)(split + 1) * kr.n / a.n_splits);
  const int32_t* bt = a.block_table + (int64_t)t.b * a.max_pages;
  float m[4], l[4], acc[4][4 * C];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < 4 * C; ++d) acc[i][d] = 0.f;
  }
  for (int j = j0; j < j1; ++j) {
    const int tb = kr.base<N>(j), end = kr.end(j);
    __syncthreads();   // every thread is done with the last step's tiles
    if (tid < N) state[tid] = 0;
    __syncthreads();
    for (int i = tid; i < N * (HD / 16) * 2; i += kSimtThreads) {
      const int which = i / (N * (HD / 16)), u = i % (HD / 16), k = i / (HD / 16) % N;
      float x[16];
      int st = 2;
      if (tb + k < end) {
        const int row = row_of(tb + k, a.ring_rows, a.pin_rows);
        const int page = bt[row / P];
        if (page < 0 || page >= a.n_pool_pages) {
          report(a.status, KVQ_DEV_BAD_PAGE);
        } else {
          const PoolLayout& L = which ? a.vl : a.kl;
          const uint8_t* pool = which ? a.v_pool : a.k_pool;
          read16_any(pool + page * L.page_bytes + (int64_t)kvh * L.sub_bytes, L, row % P, u, x);
          st = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) st |= !isfinite(x[e]);
        }
      }
      if (st) {
        state[k] = st;   // of several writers, all that is kept: left out, or not finite
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
      }
      float4* dst = reinterpret_cast<float4*>((which ? vs : ks) + k * LD + 16 * u);
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    }
    __syncthreads();
    // scores of rows 4 ty + i and keys tx + 16 c
    float s[4][2] = {};
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
      float4 kv[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) kv[c] = *reinterpret_cast<const float4*>(ks + (tx + 16 * c) * LD + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(qs + (4 * ty + i) * LD + d);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          s[i][c] = fmaf(qv.x, kv[c].x, fmaf(qv.y, kv[c].y, fmaf(qv.z, kv[c].z, fmaf(qv.w, kv[c].w, s[i][c]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = t.p0 + (4 * ty + i) / G;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = tx + 16 * c, key = tb + k, st = state[k];
        if (st == 2 || key > p || !in_window(a, p, key)) s[i][c] = -INFINITY;
        else if (st == 1) s[i][c] = NAN;
      }
      float mx = fmaxf(s[i][0], s[i][1]);
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - mu);
      const float p0 = exp2f(s[i][0] - mu), p1 = exp2f(s[i][1] - mu);
      float sum = p0 + p1;
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = l[i] * corr + sum;
      m[i] = mn;
#pragma unroll
      for (int d = 0; d < 4 * C; ++d) acc[i][d] *= corr;
      ps[(4 * ty + i) * (N + 1) + tx] = p0;
      ps[(4 * ty + i) * (N + 1) + tx + 16] = p1;
    }
    __syncwarp();   // a warp's 4 ty + i rows are its own
#pragma unroll 4
    for (int k = 0; k < N; ++k) {
      float4 v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = *reinterpret_cast<const float4*>(vs + k * LD + 4 * tx + 64 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = ps[(4 * ty + i) * (N + 1) + k];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          acc[i][4 * c] = fmaf(p, v[c].x, acc[i][4 * c]);
          acc[i][4 * c + 1] = fmaf(p, v[c].y, acc[i][4 * c + 1]);
          acc[i][4 * c + 2] = fmaf(p, v[c].z, acc[i][4 * c + 2]);
          acc[i][4 * c + 3] = fmaf(p, v[c].w, acc[i][4 * c + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
    const int64_t o = out_row(r);
    if (a.n_splits == 1) {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) store_act(a.out, a.act, o * HD + 4 * tx + 64 * c + e, acc[i][4 * c + e] * inv);
    } else {
      const int64_t w = (int64_t)split * a.n_rows * a.n_heads + o;
      if (tx == 0) a.ws_ml[w] = make_float2(m[i], l[i]);
      if (j1 > j0)
#pragma unroll
        for (int c = 0; c < C; ++c)
          *reinterpret_cast<float4*>(a.ws_acc + w * HD + 4 * tx + 64 * c) =
              make_float4(acc[i][4 * c], acc[i][4 * c + 1], acc[i][4 * c + 2], acc[i][4 * c + 3]);
    }
  }
}

// ---------------------------------------------------------------- combine
// One warp a row: its lanes hold the splits' weights, four outputs a lane (or
// twice four) the sums, eight splits in flight.  A split that saw no key has
// l = 0 and its sums are not read.  Latency: 8.5 us alone for 19 splits of 160
// rows, where a thread per four outputs that read its splits in turn took 17.
constexpr int kMaxSplits = 160;
template <int HD>
__global__ void __launch_bounds__(256) prefill_combine_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int NV = (HD + 127) / 128, NW = kMaxSplits / 32;   // float4s a lane, weights a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.y, G = a.n_heads / a.n_kv_heads, lane = threadIdx.x & 31;
  PrefillTile t;
  if (!find_tile(a, blockIdx.x, false, &t) || t.zero) return;
  const int64_t stride = (int64_t)a.n_rows * a.n_heads;
  for (int r = blockIdx.z * 8 + (threadIdx.x >> 5); r < t.cnt * G; r += gridDim.z * 8) {
    const int64_t o = (int64_t)(t.row0 + r / G) * a.n_heads + kvh * G + r % G;
    float2 ml[NW];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int s = lane + 32 * i;
      ml[i] = s < a.n_splits ? a.ws_ml[s * stride + o] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float w[NW], l = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      // a split whose only keys were not finite has m = -inf and l NaN, and keeps its weight
      w[i] = ml[i].y == 0.f ? 0.f : (ml[i].x == -INFINITY ? 1.f : exp2f(ml[i].x - M));
      l += ml[i].y == 0.f ? 0.f : w[i] * ml[i].y;
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    float4 y[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) y[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = HD >= 128 || lane < HD / 4;
    for (int s0 = 0; s0 < a.n_splits; s0 += 8) {
      float ws[8];
      float4 x[8][NV];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int s = s0 + k;
        float pick = w[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) pick = s0 / 32 == i ? w[i] : pick;
        ws[k] = __shfl_sync(0xffffffffu, pick, s & 31);
        if (s >= a.n_splits) ws[k] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          x[k][v] = on && !(ws[k] == 0.f)
                        ? *reinterpret_cast<const float4*>(a.ws_acc + (s * stride + o) * HD + 4 * (lane + 32 * v))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          y[v].x = fmaf(ws[k], x[k][v].x, y[v].x);
          y[v].y = fmaf(ws[k], x[k][v].y, y[v].y);
          y[v].z = fmaf(ws[k], x[k][v].z, y[v].z);
          y[v].w = fmaf(ws[k], x[k][v].w, y[v].w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (on)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t at = o * HD + 4 * (lane + 32 * v);
        store_act(a.out, a.act, at, y[v].x * inv);
        store_act(a.out, a.act, at + 1, y[v].y * inv);
        store_act(a.out, a.act, at + 2, y[v].z * inv);
        store_act(a.out, a.act, at + 3, y[v].w * inv);
      }
  }
}

// ---------------------------------------------------------------- host

struct PrefillPlan {
  bool tc;
  int tq, n_tiles, n_splits;
  size_t ml_offset, total;
};

// Tiles and key splits.  A sequence's tiles are at most n_b / tq + 1, so
// n_rows / tq + batch of them cover every case.  Keys are split while the
// tiles leave SMs idle, into parts of at least kMinSplitKeys keys of the
// longest range the table allows: two steps of the tensor-core kernel, one of
// the fp32 kernel.  Five tokens at 8K: 122 us in one part, 28 in 8, 22 in 16,
// 24 in 19; a 100-token fp32 prompt at 256: 38 us in one part, 19 in 4, 17 in 8.
constexpr int kMinSplitKeys = 256, kMinSplitKeysSimt = kSimtKeys;

// Whether the tensor-core kernel takes this config: 16-bit activations (its
// operands are fp16) and scale groups of whole 32-dim units (a lane's 16 bytes
// of codes then lie in one group).  The fp32 kernel takes 17.8 ms for the 8K
// prompt that takes 0.55 ms there.
static bool prefill_tc_takes(const kvq_config& c) {
  if (c.act_dtype == KVQ_F32) return false;
  return c.k_dtype == KVQ_F16_KV || (c.k_group % 32 == 0 && c.v_group % 32 == 0);
}

static PrefillPlan make_prefill_plan(const kvq_config& c, int32_t batch, int32_t n_rows, int32_t max_pages,
                                     int32_t sinks, int32_t window) {
  PrefillPlan p{};
  const int G = c.n_heads / c.n_kv_heads;
  p.tc = prefill_tc_takes(c);
  p.tq = (p.tc ? prefill_tc_rows(c.head_dim) : kSimtRows) / G;
  const int64_t tiles = (int64_t)n_rows / p.tq + batch;
  p.n_tiles = (int)(tiles > INT_MAX ? INT_MAX : tiles);
  int64_t keys = (int64_t)max_pages * c.page_size;
  if (window > 0) {
    const int64_t w = (int64_t)window + sinks + p.tq;
    if (w < keys) keys = w;
  }
  // about the tiles that have work: a batch of short chunks has one a sequence
  int64_t busy = ((int64_t)n_rows + p.tq - 1) / p.tq;
  if (busy < batch) busy = batch < n_rows ? batch : n_rows;
  busy *= c.n_kv_heads;
  int64_t s = busy > 0 ? num_sms() / busy : 1;
  const int64_t most = keys / (p.tc ? kMinSplitKeys : kMinSplitKeysSimt);
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  p.n_splits = (int)(s < 1 ? 1 : s);
  const size_t units = p.n_splits > 1 ? (size_t)p.n_splits * n_rows * c.n_heads : 0;
  p.ml_offset = (units * c.head_dim * sizeof(float) + 255) / 256 * 256;
  p.total = p.ml_offset + units * sizeof(float2) + 256;
  return p;
}

static kvq_status check_prefill(const kvq_config& c, int32_t batch, int32_t n_rows, int32_t max_pages,
                                int32_t ring_rows, int32_t sinks, int32_t window) {
  if (batch < 0 || n_rows < 0) return fail(KVQ_ERR_INVALID_ARG, "batch (%d) or n_rows (%d) < 0", batch, n_rows);
  if (max_pages < 1) return fail(KVQ_ERR_INVALID_ARG, "max_pages_per_seq must be >= 1");
  const kvq_status st = check_layout(c, max_pages, ring_rows, sinks);
  if (st != KVQ_OK) return st;
  if (window < 0 || (ring_rows > 0 && (window < 1 || window > ring_rows)))
    return fail(KVQ_ERR_INVALID_ARG, "window %d must be >= 0, and with a ring in [1, ring_rows=%d]", window, ring_rows);
  if (sinks > 0 && window == 0) return fail(KVQ_ERR_INVALID_ARG, "sinks (%d) need a window", sinks);
  return KVQ_OK;
}

template <int HD>
static cudaError_t launch_simt(cudaLaunchConfig_t& lc, const PrefillArgs& a) {
  lc.blockDim = dim3(kSimtThreads);
  lc.dynamicSmemBytes = simt_smem<HD>();
  const cudaError_t e = cudaFuncSetAttribute(prefill_simt_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)simt_smem<HD>());
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&lc, prefill_simt_kernel<HD>, a);
}

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_prefill_workspace_bytes(const kvq_config* cfg, int32_t batch, int32_t n_rows,
                                              int32_t max_pages_per_seq, int32_t ring_rows, int32_t sinks,
                                              int32_t window) {
  clear_error();
  if (check_kernel_config(cfg) != KVQ_OK) return 0;
  if (check_prefill(*cfg, batch, n_rows, max_pages_per_seq, ring_rows, sinks, window) != KVQ_OK) return 0;
  return make_prefill_plan(*cfg, batch, n_rows, max_pages_per_seq, sinks, window).total;
}

extern "C" kvq_status kvq_prefill_attention(const kvq_config* cfg, int32_t batch, int32_t n_rows, const void* q,
                                            const int32_t* q_starts, const void* k_pool, const void* v_pool,
                                            int32_t n_pool_pages, const int32_t* block_table,
                                            int32_t max_pages_per_seq, int32_t ring_rows, int32_t sinks,
                                            int32_t window, const int32_t* seq_lens, const float* rope_tab,
                                            int32_t rope_max_pos, void* out, void* workspace,
                                            size_t workspace_bytes, int32_t* dev_status, kvq_stream_t stream) {
  clear_error();
  kvq_status st = check_kernel_config(cfg);
  if (st != KVQ_OK) return st;
  st = check_prefill(*cfg, batch, n_rows, max_pages_per_seq, ring_rows, sinks, window);
  if (st != KVQ_OK) return st;
  if (batch == 0 || n_rows == 0) return KVQ_OK;
  if (!q || !q_starts || !k_pool || !v_pool || !block_table || !seq_lens || !out || !workspace || !dev_status)
    return fail(KVQ_ERR_INVALID_ARG, "a required device pointer is NULL");
  if (n_pool_pages < 1) return fail(KVQ_ERR_INVALID_ARG, "n_pool_pages must be >= 1");
  if (cfg->rope != KVQ_ROPE_NONE && (!rope_tab || rope_max_pos < 1))
    return fail(KVQ_ERR_INVALID_ARG, "RoPE config needs rope_tab and rope_max_pos >= 1");
  if ((reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool)) & 15)
    return fail(KVQ_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(KVQ_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (cfg->rope != KVQ_ROPE_NONE && (reinterpret_cast<uintptr_t>(rope_tab) & 15))
    return fail(KVQ_ERR_INVALID_ARG, "rope_tab must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(KVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const PrefillPlan p = make_prefill_plan(*cfg, batch, n_rows, max_pages_per_seq, sinks, window);
  if (workspace_bytes < p.total)
    return fail(KVQ_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes, p.total);
  if (cfg->n_kv_heads > 65535 || p.n_splits > 65535) return fail(KVQ_ERR_INVALID_ARG, "n_kv_heads too large");

  PrefillArgs a;
  a.q = q; a.q_starts = q_starts;
  a.k_pool = static_cast<const uint8_t*>(k_pool); a.v_pool = static_cast<const uint8_t*>(v_pool);
  a.block_table = block_table; a.seq_lens = seq_lens; a.rope_tab = rope_tab; a.out = out;
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.ml_offset);
  a.status = dev_status;
  a.batch = batch; a.n_rows = n_rows; a.n_heads = cfg->n_heads; a.n_kv_heads = cfg->n_kv_heads;
  a.n_pool_pages = n_pool_pages; a.max_pages = max_pages_per_seq; a.rope_max_pos = rope_max_pos;
  a.ring_rows = ring_rows; a.pin_rows = pinned_rows(*cfg, ring_rows, sinks);
  a.window = window; a.sinks = sinks; a.act = cfg->act_dtype; a.rope = cfg->rope;
  a.tq = p.tq; a.n_tiles = p.n_tiles; a.n_splits = p.n_splits;
  a.score_scale = score_scale_log2(*cfg);
  a.kl = pool_layout(*cfg, 0);
  a.vl = pool_layout(*cfg, 1);

  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)p.n_tiles, (unsigned)cfg->n_kv_heads, (unsigned)p.n_splits);
  lc.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  cudaError_t e;
  if (p.tc) {
    const int64_t blocks = (int64_t)p.n_tiles * cfg->n_kv_heads * p.n_splits;
    if (blocks > INT_MAX) return fail(KVQ_ERR_INVALID_ARG, "too many rows");
    lc.gridDim = dim3((unsigned)blocks);
    e = launch_prefill_tc(lc, cfg->head_dim, a);
  } else {
    switch (cfg->head_dim) {
      case 64: e = launch_simt<64>(lc, a); break;
      case 128: e = launch_simt<128>(lc, a); break;
      default: e = launch_simt<256>(lc, a); break;
    }
  }
  if (e == cudaSuccess && p.n_splits > 1) {
    lc.gridDim = dim3((unsigned)p.n_tiles, (unsigned)cfg->n_kv_heads, 8);
    lc.blockDim = dim3(256);
    lc.dynamicSmemBytes = 0;
    switch (cfg->head_dim) {
      case 64: e = cudaLaunchKernelEx(&lc, prefill_combine_kernel<64>, a); break;
      case 128: e = cudaLaunchKernelEx(&lc, prefill_combine_kernel<128>, a); break;
      default: e = cudaLaunchKernelEx(&lc, prefill_combine_kernel<256>, a); break;
    }
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

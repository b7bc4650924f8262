// Reading rows back: stored K and V rows of given tokens as numbers of the
// activation type.
//
//   K^ = s * code (+ bias), in fp32 (one product, or one fused multiply-add),
//   rounded once to act_dtype.
//
// Codec: [airllm] §4.2, [Shimmy] §3.2, [Fieldfare] "量化和精度" (as written by
// kvq_append.cu); pages: [airllm] §2.3.
//
// A thread owns 16 consecutive elements of one row of one kv head (every scale
// group is a multiple of 16, so they share one scale) of K, then of V.  Bound
// by the latency of four dependent steps (position, table, codes, store), so by
// the threads in flight: 32 registers, eight blocks an SM.  The outputs are
// most of the bytes (4 times the codes' at 4 bits and a 16-bit type), and 32
// bytes a store write whole sectors: four 64K contexts of 8-bit K and 4-bit V
// as fp16, 757 MB, 155 us, 4.9 TB/s or 73 % of the measured copy rate; 166 us
// in two stores of 16 bytes.  A block that looks its rows up first, 157 to 167.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

struct ReadArgs {
  const int32_t* seq_ids;
  const int32_t* pos;
  const int32_t* block_table;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  void* k_out;
  void* v_out;
  int32_t* status;
  int64_t n_units;   // n_rows * n_kv_heads * head_dim / 16
  int32_t wide;      // both outputs are 32-byte aligned
  int32_t n_kv_heads, n_seqs, max_pages, ring_rows, pin_rows, n_pool_pages;
  PoolLayout kl, vl;
};

// 32 bytes in one store where p is 32-byte aligned (WIDE), which writes whole
// sectors, else in two.
template <bool WIDE>
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int ACT, bool WIDE>
__device__ __forceinline__ void write16(void* out, int64_t i, const float (&x)[16]) {
  uint32_t w[8];
  if constexpr (ACT == KVQ_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[8 * h + j]);
      store32<WIDE>(static_cast<float*>(out) + i + 8 * h, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (ACT == KVQ_F16) {
        const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    store32<WIDE>(static_cast<unsigned short*>(out) + i, w);
  }
}

template <int KK, int VK, int HD, int ACT>
__global__ void __launch_bounds__(256, 8) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int P = 16, U = HD / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.n_units) return;
  const int u = (int)(i % U);
  const int64_t rh = i / U;
  const int row = (int)(rh / a.n_kv_heads), head = (int)(rh % a.n_kv_heads);
  const bool first = u == 0 && head == 0;
  const int seq = a.seq_ids ? a.seq_ids[row] : row;
  const int pos = a.pos[row];
  if (seq < 0 || seq >= a.n_seqs) {
    if (first) report(a.status, KVQ_DEV_BAD_SEQ);
    return;
  }
  const int r = pos >= 0 ? row_of(pos, a.ring_rows, a.pin_rows) : -1;
  if (r < 0 || r / P >= a.max_pages) {
    if (first) report(a.status, KVQ_DEV_BAD_POS);
    return;
  }
  const int page = a.block_table[(int64_t)seq * a.max_pages + r / P];
  if (page < 0 || page >= a.n_pool_pages) {
    if (first) report(a.status, KVQ_DEV_BAD_PAGE);
    return;
  }
  float x[16];
  if (a.k_out) {
    read16<KK>(a.k_pool + page * a.kl.page_bytes + (int64_t)head * a.kl.sub_bytes, a.kl, r % P, u, x);
    if (a.wide) write16<ACT, true>(a.k_out, i * 16, x);
    else write16<ACT, false>(a.k_out, i * 16, x);
  }
  if (a.v_out) {
    read16<VK>(a.v_pool + page * a.vl.page_bytes + (int64_t)head * a.vl.sub_bytes, a.vl, r % P, u, x);
    if (a.wide) write16<ACT, true>(a.v_out, i * 16, x);
    else write16<ACT, false>(a.v_out, i * 16, x);
  }
}

template <int KK, int VK, int HD>
static cudaError_t launch_read(const cudaLaunchConfig_t& lc, int act, const ReadArgs& a) {
  if (act == KVQ_F32) return cudaLaunchKernelEx(&lc, read_kernel<KK, VK, HD, KVQ_F32>, a);
  if (act == KVQ_F16) return cudaLaunchKernelEx(&lc, read_kernel<KK, VK, HD, KVQ_F16>, a);
  return cudaLaunchKernelEx(&lc, read_kernel<KK, VK, HD, KVQ_BF16>, a);
}
template <int KK, int VK>
static cudaError_t launch_read(const cudaLaunchConfig_t& lc, int hd, int act, const ReadArgs& a) {
  if (hd == 64) return launch_read<KK, VK, 64>(lc, act, a);
  if (hd == 128) return launch_read<KK, VK, 128>(lc, act, a);
  if constexpr (KK == KVQ_F16_KV) return cudaErrorInvalidValue;   // refused by the config check
  else return launch_read<KK, VK, 256>(lc, act, a);
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_read(const kvq_config* cfg, int32_t n_rows, const int32_t* seq_ids, const int32_t* pos,
                               const int32_t* block_table, int32_t n_seqs, int32_t max_pages_per_seq,
                               int32_t ring_rows, int32_t sinks, const void* k_pool, const void* v_pool,
                               int32_t n_pool_pages, void* k_out, void* v_out, int32_t* dev_status,
                               kvq_stream_t stream) {
  clear_error();
  kvq_status st = check_kernel_config(cfg);
  if (st != KVQ_OK) return st;
  if (n_rows < 0) return fail(KVQ_ERR_INVALID_ARG, "n_rows (%d) < 0", n_rows);
  if (n_rows == 0) return KVQ_OK;
  if (!pos || !block_table || !dev_status || (!k_out && !v_out) || (k_out && !k_pool) || (v_out && !v_pool))
    return fail(KVQ_ERR_INVALID_ARG, "a required device pointer is NULL");
  if (n_seqs < 1 || max_pages_per_seq < 1 || n_pool_pages < 1)
    return fail(KVQ_ERR_INVALID_ARG, "n_seqs, max_pages_per_seq and n_pool_pages must be >= 1");
  if (!seq_ids && n_rows > n_seqs)
    return fail(KVQ_ERR_INVALID_ARG, "without seq_ids, n_rows (%d) must be <= n_seqs (%d)", n_rows, n_seqs);
  st = check_layout(*cfg, max_pages_per_seq, ring_rows, sinks);
  if (st != KVQ_OK) return st;
  if ((reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool)) & 15)
    return fail(KVQ_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15)
    return fail(KVQ_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");

  ReadArgs a;
  a.seq_ids = seq_ids; a.pos = pos; a.block_table = block_table;
  a.k_pool = static_cast<const uint8_t*>(k_pool); a.v_pool = static_cast<const uint8_t*>(v_pool);
  a.k_out = k_out; a.v_out = v_out; a.status = dev_status;
  a.n_units = (int64_t)n_rows * cfg->n_kv_heads * (cfg->head_dim / 16);
  a.n_kv_heads = cfg->n_kv_heads; a.n_seqs = n_seqs; a.max_pages = max_pages_per_seq;
  a.ring_rows = ring_rows; a.pin_rows = pinned_rows(*cfg, ring_rows, sinks); a.n_pool_pages = n_pool_pages;
  a.wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  a.kl = pool_layout(*cfg, 0);
  a.vl = pool_layout(*cfg, 1);
  const int64_t blocks = (a.n_units + 255) / 256;
  if (blocks > 0x7fffffffLL) return fail(KVQ_ERR_INVALID_ARG, "too many rows");

  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)blocks);
  lc.blockDim = dim3(256);
  lc.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  const int k = cfg->k_dtype, v = cfg->v_dtype, hd = cfg->head_dim, act = cfg->act_dtype;
  cudaError_t e;
  if (k == KVQ_SYM_INT4) e = launch_read<KVQ_SYM_INT4, KVQ_SYM_INT4>(lc, hd, act, a);
  else if (k == KVQ_SYM_INT8 && v == KVQ_SYM_INT8) e = launch_read<KVQ_SYM_INT8, KVQ_SYM_INT8>(lc, hd, act, a);
  else if (k == KVQ_SYM_INT8) e = launch_read<KVQ_SYM_INT8, KVQ_SYM_INT4>(lc, hd, act, a);
  else if (k == KVQ_AFFINE_INT4) e = launch_read<KVQ_AFFINE_INT4, KVQ_AFFINE_INT4>(lc, hd, act, a);
  else if (k == KVQ_F16_KV) e = launch_read<KVQ_F16_KV, KVQ_F16_KV>(lc, hd, act, a);
  else e = launch_read<KVQ_SHIMMY_INT4, KVQ_SHIMMY_INT4>(lc, hd, act, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "read launch: %s", cudaGetErrorString(e));
  return KVQ_OK;
}

// Prefill attention on the fifth-generation tensor cores (tcgen05), for f16
// and bf16 activations.
//
// A CTA takes MT tiles of 128 query rows (a row is a query token and one of
// the G heads that share the kv head) over the keys they attend, 128 keys a
// step:
//   S = Q' K'^T   (fp16 operands in shared memory, fp32 in tensor memory)
//   P = 2^(S f - m + 7), rounded to fp16 and written back over S
//   O += P V'     (P from tensor memory, V' from shared memory)
// Roles, by warp: MT warpgroups of softmax (a thread owns a row: no shuffles),
// one warpgroup that dequantizes K and one that dequantizes V, and a warp per
// row tile that issues its products.  They meet at mbarriers only.  S comes in
// halves of 64 keys, two of them in flight per row tile, so that the products
// of one half run while the softmax works on the other; head_dim 256 has room
// for one row tile in tensor memory, the others for two.
//
// K' and V' sit in shared memory as blocks of 128 keys x 64 dims in the
// 128-byte swizzle, in two rings of four blocks.  Codes become fp16 values two
// nibbles (or bytes) of a word at a time, so the dims of every eight are stored
// in the order 0 4 1 5 2 6 3 7 (4-bit) or, of every four, 0 2 1 3 (8-bit); Q'
// is stored in the same order and the output is put back in order when it is
// written.
//
// fp16 range.  Operands are fp16 for every activation type: its 11 bits cost a
// bf16 result nothing, where bf16's 8 would add as much error as the result's
// own rounding.  A query row, the 128 keys of a step and the values seen so far
// are each held at a power-of-two scale (from the row's largest element, and
// from the scales of the step's keys) that keeps the largest magnitude in
// fp16's upper range: exact, and free, as the factors go into f, the one
// multiplier of a row's scores in a step, and into the last scaling of O.  When
// a step's values are larger than all before, O is rescaled, as it is when the
// running maximum rises by more than 2^8; P is held times 2^7, which keeps
// weights down to 2^-21 of the largest in fp16's normal range.  What is rounded
// to fp16 once: the rotated query, a 32-bit scale, each K^ and V^, each weight.
// Maxima, sums and O are fp32.
//
// Keys that no row may see (behind the last token, bad pages) are zero rows
// and masked; a key whose scale or element is not finite is a zero row and a
// bit that turns the scores of the rows that attend it into NaN, so it spoils
// no other row of the tile.
//
// Every wait is bounded (two seconds): when one runs out the CTA runs through
// its remaining steps without waiting, frees its tensor memory and reports
// KVQ_DEV_TIMEOUT.
//
// Measured, Llama-shaped layer (32 / 8 heads of 128, 4-bit K and V): an 8K
// prompt 0.537 ms, 1.02 PFLOP/s of causal products, 53 % of the measured
// matrix rate.  Tensor pipe active 43 %, issue slots 60 % with four to five
// warps a scheduler: bound by the instructions of softmax and dequantization
// (11,100 a step of 256 rows x 128 keys; the products alone would take 2500
// cycles of about 4000), and for a seventh of the time by a CTA's start and end,
// which nothing overlaps as a CTA fills its SM.  What was tried: a step's S in
// one buffer, 722 us where two halves took 640; products 128 keys wide, 653
// against 545; two threads a row or a warpgroup per half (more warps, more
// instructions), 777 and 610 against 722 and 555.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "kvq_prefill.cuh"
#include "kvq_prefill_tc.h"
#include "kvq_umma_ptx.cuh"

namespace kvq {
namespace {

using namespace um;

constexpr int kKeys = 128;               // keys a step, taken in two halves
constexpr int kHalf = kKeys / 2;
constexpr int kStages = 4;               // blocks of a ring
constexpr int kBlockBytes = kKeys * 128; // 128 keys x 64 dims of fp16
constexpr int kSlots = 8;                // steps whose metadata are kept
constexpr float kLazy = 8.0f;            // the running maximum rises past +2^8 only
constexpr float kShift = 7.0f;           // P is held times 2^7

__host__ __device__ constexpr int row_tiles(int hd) { return hd == 256 ? 1 : 2; }
// Tensor memory has 512 columns: S 128 and O head_dim a row tile.  Where the
// queries fit beside them (not at head_dim 128) the scores' products take them
// from there: from shared memory a product of 128 x 64 x 16 reads 6 KB in the
// time that moves 4 (window layer of head_dim 256: 209 -> 207 us).
template <int HD>
constexpr bool kQInTmem = HD != 128;
__host__ __device__ constexpr int tc_threads(int hd) { return 128 * row_tiles(hd) + 256 + 128; }
// Registers a thread: at launch (65536 over the threads, in eights), then by
// role.  A role may only take what the others gave back, so the shares must
// not exceed the launch's: (softmax * tiles + 2 producers + products) * 128.
// Eight fewer for the softmax and it spills (8K prompt 545 -> 582 us); eight
// fewer for the producers and they do (f16 rows 1.22 -> 1.30 ms).
__host__ __device__ constexpr int regs_launch(int hd) { return 65536 / tc_threads(hd) / 8 * 8; }
__host__ __device__ constexpr int regs_softmax(int hd) { return hd == 256 ? 184 : 136; }
__host__ __device__ constexpr int regs_produce(int hd) { return hd == 256 ? 128 : 88; }
constexpr int kRegsProducts = 32;
template <int HD>
constexpr bool split_fits() {
  return regs_softmax(HD) * row_tiles(HD) + 2 * regs_produce(HD) + kRegsProducts <=
         regs_launch(HD) * (tc_threads(HD) / 128);
}
static_assert(split_fits<64>() && split_fits<128>() && split_fits<256>(), "register split");

// What the softmax needs to know about the keys of a step, for K and for V.
struct StepMeta {
  int2 head[2];          // the exponent they are held at, and whether any key below is marked
  uint32_t skip[2][4];   // keys left out (bad pages), a bit each
  uint32_t bad[2][4];    // keys that are not finite
};

template <int HD>
struct Shared {
  static constexpr int MT = row_tiles(HD);
  static constexpr int HB = HD / 64;
  uint8_t q[MT * HB * kBlockBytes];
  uint8_t k[kStages * kBlockBytes];
  uint8_t v[kStages * kBlockBytes];
  StepMeta meta[kSlots];
  float qscale[MT * 128];   // f without the keys' part
  int2 red[2][2][4];
  // half a step's keys each
  uint64_t kfull[kStages][2], kempty[kStages][2], vfull[kStages][2], vempty[kStages][2];
  uint64_t ready[kSlots];   // a step's metadata are there
  uint64_t qfull;                        // the queries are there
  uint64_t sfull[MT][2], pfull[MT][2];   // scores and weights of a half step
  uint64_t ofull[MT][2];                 // O with it
  uint64_t qtmem[MT], drain[MT];
  uint32_t tmem;
  int stop;
};
template <int HD>
constexpr size_t shared_bytes() { return sizeof(Shared<HD>) + 1024; }   // the blocks want 1024-byte alignment

__device__ __forceinline__ float pow2i(int e) {   // 2^e, 0 below 2^-126
  return e < -126 ? 0.f : __int_as_float((e + 127) << 23);
}
// Exponents at which operands are held, as far as both factors stay normal
// floats: magnitudes up to x (finite, >= 0) in [2^14, 2^15) ...  For a query x is
// sqrt 2 times its largest element, the most that a rotated one can be.
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ int hold_exponent(float x) { return min(max(exponent_of(x) - 14, -100), 114); }
// ... and a key's scales up to s in [2^-10, 2^-9) and biases up to b below 2^15.
// dequant8 multiplies subnormals by 2^24 s, which stays finite even where s is
// rounded up to 2^-9 (a power of two more, and 2^16 would be infinite).
__device__ __forceinline__ int key_exponent(float s, float b) {
  return max(max(exponent_of(s) + 10, exponent_of(b) - 14), -100);
}
constexpr float kMostScale = 1.0e35f;   // held at 2^126 at most: a larger scale counts as not finite
__device__ __forceinline__ void group_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// How the dims of every eight are ordered in shared memory (see above).
__host__ __device__ constexpr int order_of(int kind) {
  return kind == KVQ_F16_KV ? 0 : (kind == KVQ_SYM_INT8 ? 1 : 2);
}
// The dim (0..7) at position i of an ordered group of eight.
__host__ __device__ constexpr int dim_at(int order, int i) {
  return order == 0 ? i : (order == 1 ? (i & 4) | ((i & 1) << 1) | ((i >> 1) & 1) : (i >> 1) | ((i & 1) << 2));
}

// A group's scale and bias for dequant8.
struct Scale {
  __half2 lo, hi, b;
};
template <int KIND>
__device__ __forceinline__ Scale make_scale(float s, float b) {   // s < 2^-9
  const __half2 h = __float2half2_rn(s);                           // the stored scale, to fp16
  Scale r;
  r.lo = __hmul2(h, __float2half2_rn(4096.f));                     // 2^24 s, exact
  r.lo = __hmul2(r.lo, __float2half2_rn(4096.f));
  r.hi = __hmul2(r.lo, __float2half2_rn(0.0625f));
  if (KIND == KVQ_AFFINE_INT4) r.b = __float2half2_rn(b);
  else r.b = __hmul2(h, __float2half2_rn(KIND == KVQ_SYM_INT8 ? -128.f : -8.f));
  return r;
}
// Eight codes (one word; two words for 8-bit kinds) to eight fp16 values
// s * code + b, in order_of(KIND).  An unsigned code n in the low bits of a
// half is the subnormal n 2^-24, and one multiply-add by 2^24 s makes it n s +
// b, rounded once; signed codes are n - 8 (n - 128).  The high nibble of a byte
// is 16 n.
template <int KIND>
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, const Scale& s) {
  uint32_t r[4];
  if constexpr (KIND == KVQ_SYM_INT8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = i ? w1 : w0;
      r[2 * i] = h2u(__hfma2(u2h((w & 0x00FF00FFu) ^ 0x00800080u), s.lo, s.b));
      r[2 * i + 1] = h2u(__hfma2(u2h(((w >> 8) & 0x00FF00FFu) ^ 0x00800080u), s.lo, s.b));
    }
  } else {
    constexpr uint32_t fl = KIND == KVQ_SYM_INT4 ? 0x00080008u : 0u, fh = KIND == KVQ_SYM_INT4 ? 0x00800080u : 0u;
    const uint32_t ws = w0 >> 8;
    r[0] = h2u(__hfma2(u2h((w0 & 0x000F000Fu) ^ fl), s.lo, s.b));
    r[1] = h2u(__hfma2(u2h((w0 & 0x00F000F0u) ^ fh), s.hi, s.b));
    r[2] = h2u(__hfma2(u2h((ws & 0x000F000Fu) ^ fl), s.lo, s.b));
    r[3] = h2u(__hfma2(u2h((ws & 0x00F000F0u) ^ fh), s.hi, s.b));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The dequantizing warpgroup of K or V.  A warp owns 32 keys of every step, two
// pages.  Its loads are whole: LPR lanes share a row, 16 bytes each, so a load
// covers KPL rows that lie one behind the other, and NL loads the 32 keys (a
// thread to a row had every 16-byte load of a warp touch 32 rows: four to
// eight times the passes through the L1, which the tensor cores read their
// operands through as well).  Loads run ahead of their use: a step's page ids
// two steps, its parameters and first codes one step.
template <int KIND, int HD>
__device__ void produce(const bool is_v, const PrefillArgs& a, const PrefillTile& t, const KeyRange& kr, int j0, int n,
                        int kvh, int pt, Shared<HD>& sh, volatile int* stop) {
  constexpr int P = 16, HB = HD / 64, RU = kStages / HB;   // blocks a step, steps a ring
  constexpr bool F16 = KIND == KVQ_F16_KV, AFF = KIND == KVQ_AFFINE_INT4;
  constexpr int BITS = F16 ? 16 : (KIND == KVQ_SYM_INT8 ? 8 : 4);
  constexpr int LPR = HD * BITS / 128, KPL = 32 / LPR, NL = LPR;
  constexpr int CPP = 16 / BITS, WPC = BITS / 4;           // eights of dims in 16 bytes, words of an eight
  constexpr int NLP = NL < 8 ? NL : 8, NP = NL / NLP;      // loads kept in registers, and how often a step
  constexpr int NS = F16 ? 1 : NL;
  const PoolLayout& L = is_v ? a.vl : a.kl;
  const uint8_t* pool = (is_v ? a.v_pool : a.k_pool) + (int64_t)kvh * L.sub_bytes;
  const int32_t* bt = a.block_table + (int64_t)t.b * a.max_pages;
  const int warp = pt >> 5, lane = pt & 31, kh = warp / 2;   // kh: its half of the step
  const int kq = lane / LPR, lp = lane % LPR;
  const int dim0 = lp * (CPP * 8), blk = dim0 / 64;
  // Where the lane's first eight dims of its key of load 0 are stored.  Lanes
  // of a row that meet the same chunk of different blocks store their eights in
  // another order (eight x in place of x ^ fl), so that they hit different banks.
  const int fl = BITS == 4 ? (HD == 128 ? 2 * blk : (HD == 256 ? blk : 0)) : (BITS == 8 ? blk & 1 : 0);
  const uint32_t dst0 = smem_u32(is_v ? sh.v : sh.k) + blk * kBlockBytes + (32 * warp + kq) * 128 +
                        (((dim0 % 64 / 8) ^ (kq & 7) ^ fl) << 4);
  uint64_t(*full)[2] = is_v ? sh.vfull : sh.kfull;
  uint64_t(*empty)[2] = is_v ? sh.vempty : sh.kempty;
  const int pb = param_bytes(L.param);
  const int par0 = F16 ? 0 : P * L.code_bytes + dim0 / L.group * (AFF ? 2 : 1) * pb;   // of slot 0
  const int page_bytes = (int)L.page_bytes;       // a page is far below 2 GB

  // The warp's two page ids in step i (-1: no token there).
  auto pages_at = [&](int i, int (&pg)[2]) {
    pg[0] = pg[1] = -1;
    if (i >= n) return;
    const int key = kr.base<kKeys>(j0 + i) + 32 * warp, end = kr.end(j0 + i);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (key + P * h < end) pg[h] = bt[row_of(key + P * h, a.ring_rows, a.pin_rows) / P];
  };
  uint32_t raw[NLP * 4];
  float nsc[NS], nbi[AFF ? NS : 1];
  const uint8_t *sub[2] = {pool, pool};   // the pages being loaded
  int keys[2] = {0, 0};                   // keys below which the pages hold tokens; a bad page holds none
  uint32_t nskip = 0;                     // keys of bad pages
  auto there = [&](int j) { return j * KPL + kq < keys[j * KPL / P]; };
  auto load_piece = [&](int p) {
#pragma unroll
    for (int x = 0; x < NLP; ++x) {
      const int j = p * NLP + x;
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(sub[j * KPL / P] + (j * KPL % P + kq) * (LPR * 16)) + lp);
      raw[4 * x] = y.x;
      raw[4 * x + 1] = y.y;
      raw[4 * x + 2] = y.z;
      raw[4 * x + 3] = y.w;
    }
  };
  auto open_step = [&](int i, const int (&pg)[2]) {   // the pages, and the parameters of the lane's keys
    const int tokens = i < n ? kr.end(j0 + i) - kr.base<kKeys>(j0 + i) - 32 * warp : 0;
    nskip = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool ok = (uint32_t)pg[h] < (uint32_t)a.n_pool_pages;
      keys[h] = ok ? tokens : 0;
      if (__builtin_expect(!ok && P * h < tokens, 0)) {
        nskip |= 0xFFFFu << (P * h);
        if (lane == 0) report(a.status, KVQ_DEV_BAD_PAGE);
      }
      sub[h] = pool + (int64_t)(ok ? pg[h] : 0) * page_bytes;   // some page: its codes meet a scale of 0
    }
    if constexpr (!F16) {
      const uint8_t* par[2] = {sub[0] + par0 + kq * L.param_row_bytes, sub[1] + par0 + kq * L.param_row_bytes};
      auto load = [&](auto type) {   // one branch on the type for all
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const uint8_t* p = par[j * KPL / P] + (j * KPL % P) * L.param_row_bytes;
          nsc[j] = load_param(p, type.value);
          if constexpr (AFF) nbi[j] = load_param(p + param_bytes(type.value), type.value);
        }
      };
      if (L.param == KVQ_F32) load(std::integral_constant<int, KVQ_F32>());
      else if (L.param == KVQ_F16) load(std::integral_constant<int, KVQ_F16>());
      else load(std::integral_constant<int, KVQ_BF16>());
    }
  };
  // One bit a key of 32 from a vote a load.
  auto key_bits = [&](int j, bool x) -> uint32_t {
    const uint32_t v = __ballot_sync(0xffffffffu, x);
    uint32_t r = 0;
    if (v != 0) {
#pragma unroll 1
      for (int k = 0; k < KPL; ++k)
        if ((v >> (k * LPR)) & ((1u << LPR) - 1u)) r |= 1u << (j * KPL + k);
    }
    return r;
  };

  int held = F16 ? 0 : -100;   // V: the exponent held so far
  int pg[2], pg1[2];
  pages_at(0, pg);
  open_step(0, pg);
  load_piece(0);
  pages_at(1, pg1);
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    int pg2[2];
    pages_at(i + 2, pg2);
    StepMeta& meta = sh.meta[i % kSlots];
    const uint32_t skip = nskip;
    uint32_t bad = 0;
    float sc[NS], bi[AFF ? NS : 1];
    // Joins the warps' exponents and marks and leaves them for the softmax;
    // returns the exponent the step is held at (V: the largest so far).
    auto publish = [&](int e) -> int {
      const int top = __reduce_max_sync(0xffffffffu, e);
      int2* r = sh.red[is_v][i & 1];
      if (lane == 0) {
        r[warp] = make_int2(top, skip | bad ? 1 : 0);
        meta.skip[is_v][warp] = skip;
        meta.bad[is_v][warp] = bad;
      }
      group_sync(is_v ? 2 : 1);
      const int2 r0 = r[0], r1 = r[1], r2 = r[2], r3 = r[3];
      const int all = max(max(r0.x, r1.x), max(r2.x, r3.x));
      const int now = is_v ? max(held, all) : all;
      if (pt == 0) {
        meta.head[is_v] = make_int2(now, r0.y | r1.y | r2.y | r3.y);
        mbar_arrive(smem_u32(&sh.ready[i % kSlots]));
      }
      return now;
    };
    if constexpr (!F16) {
      float ms = 0.f, mb = 0.f;   // the largest scale and bias of the lane's keys
      bool odd = false;           // parameters that are not finite, of a key or of what lies behind the keys
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const bool fine = nsc[j] < kMostScale && (!AFF || isfinite(nbi[AFF ? j : 0])), on = fine && there(j);
        odd |= !fine;
        sc[j] = on ? nsc[j] : 0.f;
        ms = fmaxf(ms, sc[j]);
        if constexpr (AFF) {
          bi[j] = on ? nbi[j] : 0.f;
          mb = fmaxf(mb, fabsf(bi[j]));
        }
      }
      if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
#pragma unroll
        for (int j = 0; j < NL; ++j)
          bad |= key_bits(j, !(nsc[j] < kMostScale && (!AFF || isfinite(nbi[AFF ? j : 0]))) && there(j));
      }
      held = publish(key_exponent(ms, mb));
      const float down = pow2i(-held);
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        sc[j] *= down;
        if constexpr (AFF) bi[j] *= down;
      }
    }
    const int us = i % RU;
    mbar_wait(smem_u32(&empty[us][kh]), (i / RU + 1) & 1, stop);
    const uint32_t dst = dst0 + us * (HB * kBlockBytes);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
      for (int x = 0; x < NLP; ++x) {
        const int j = p * NLP + x;
        uint32_t* w = raw + 4 * x;
        const uint32_t row = (dst + j * KPL * 128) ^ ((j * KPL & 7) << 4);
        if constexpr (F16) {
          // a half with all exponent bits set carries into its sign bit
          uint32_t inf = 0;
#pragma unroll
          for (int v = 0; v < 4; ++v) inf |= ((w[v] & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u;
          if (__builtin_expect(__any_sync(0xffffffffu, inf != 0), 0)) bad |= key_bits(j, inf != 0 && there(j));
          const bool z = inf != 0 || !there(j);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(z ? 0u : w[0]), "r"(z ? 0u : w[1]),
                       "r"(z ? 0u : w[2]), "r"(z ? 0u : w[3])
                       : "memory");
        } else {
          const Scale s = make_scale<KIND>(sc[j], bi[AFF ? j : 0]);
          auto swap = [&](int m, bool on) {   // eights x and x ^ m
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (!(v & m)) {
                const uint32_t lo = on ? w[v ^ m] : w[v], hi = on ? w[v] : w[v ^ m];
                w[v] = lo;
                w[v ^ m] = hi;
              }
          };
          if constexpr (BITS == 4 && HD == 128) swap(2, fl & 2);
          if constexpr (BITS == 4 && HD == 256) {
            swap(1, fl & 1);
            swap(2, fl & 2);
          }
          if constexpr (BITS == 8 && HD > 64) swap(2, fl & 1);   // an eight is two words
#pragma unroll
          for (int c = 0; c < CPP; ++c) {
            const uint4 y = dequant8<KIND>(w[c * WPC], w[c * WPC + WPC - 1], s);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row ^ (c << 4)), "r"(y.x), "r"(y.y),
                         "r"(y.z), "r"(y.w)
                         : "memory");
          }
        }
      }
      if (p < NP - 1) load_piece(p + 1);
    }
    if (F16) publish(0);   // known only now
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&full[us][kh]));
    // the next step is on its way while this warp waits for room for it
    open_step(i + 1, pg1);
    load_piece(0);
    pg1[0] = pg2[0];
    pg1[1] = pg2[1];
  }
}

template <int HD>
__device__ __forceinline__ void produce_kind(int kind, bool is_v, const PrefillArgs& a, const PrefillTile& t,
                                             const KeyRange& kr, int j0, int n, int kvh, int pt, Shared<HD>& sh,
                                             volatile int* stop) {
  switch (kind) {
    case KVQ_SYM_INT4: return produce<KVQ_SYM_INT4, HD>(is_v, a, t, kr, j0, n, kvh, pt, sh, stop);
    case KVQ_SYM_INT8: return produce<KVQ_SYM_INT8, HD>(is_v, a, t, kr, j0, n, kvh, pt, sh, stop);
    case KVQ_AFFINE_INT4: return produce<KVQ_AFFINE_INT4, HD>(is_v, a, t, kr, j0, n, kvh, pt, sh, stop);
    case KVQ_SHIMMY_INT4: return produce<KVQ_SHIMMY_INT4, HD>(is_v, a, t, kr, j0, n, kvh, pt, sh, stop);
    default:
      if constexpr (HD <= 128) return produce<KVQ_F16_KV, HD>(is_v, a, t, kr, j0, n, kvh, pt, sh, stop);
  }
}

// The queries of the CTA's rows, rotated, scaled into fp16 and stored as blocks
// of 64 dims.  HD / 8 lanes take a row, a 16-byte chunk of it each.  The rows
// are first copied as they are, all at once, while the CTA sets itself up, and
// then worked on in place, two of a lane's at once, or four where the launch
// has 128 registers (head_dim 256; with 96 four spill in the steps: 8K prompt
// 545 -> 564 us; window layer 202 us with two, 200 with four).  This runs once a
// CTA and costs the latency of its instructions: 13,000 cycles of 162,000 in an
// 8K prompt before a row's exponent was taken from its stored bits, two rows in
// a word (543 -> 537 us; window layer 207 -> 200).  Every warp but the producers'
// takes part, `warp` counted among those.
template <int HD>
struct Queries {
  static constexpr int HB = HD / 64, LANES = HD / 8, kRows = HD == 256 ? 4 : 2;
  static constexpr int WARP = 32 / LANES * kRows, STEP = (4 * row_tiles(HD) + 4) * WARP;   // rows of a warp, of all
  // The lane's eight dims: with NeoX pairing lanes 2 i and 2 i + 1 have the
  // i-th chunks of the two halves, the pairs of eight positions between them.
  static __device__ __forceinline__ int dim(int li, bool neox) {
    return neox ? 8 * (li >> 1) + (li & 1) * (HD / 2) : 8 * li;
  }
  // Where eight dims from d (a multiple of 8) of row R are.
  static __device__ __forceinline__ uint32_t chunk(uint32_t base, int R, int d) {
    return base + ((R >> 7) * HB + d / 64) * kBlockBytes + (R & 127) * 128 + (((d % 64 / 8) ^ (R & 7)) << 4);
  }
};
template <int HD>
__device__ void copy_queries(const PrefillArgs& a, const PrefillTile& t, int rows, int lg, int kvh, int warp, int lane,
                             Shared<HD>& sh) {
  using Q = Queries<HD>;
  const int d = Q::dim(lane % Q::LANES, a.rope == KVQ_ROPE_NEOX);
  const uint32_t base = smem_u32(sh.q);
  const unsigned short* q =
      static_cast<const unsigned short*>(a.q) + ((int64_t)t.row0 * a.n_heads + (kvh << lg)) * HD + d;
#pragma unroll 1
  for (int R0 = warp * Q::WARP + lane / Q::LANES * Q::kRows; R0 < rows; R0 += Q::STEP)
#pragma unroll
    for (int u = 0; u < Q::kRows; ++u) {
      const int R = R0 + u;
      if (R < rows)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(Q::chunk(base, R, d)),
                     "l"(q + ((int64_t)(R >> lg) * a.n_heads + (R & ((1 << lg) - 1))) * HD)
                     : "memory");
    }
}
template <int HD>
__device__ void load_queries(const PrefillArgs& a, const PrefillTile& t, int rows, int lg, int warp, int lane,
                             Shared<HD>& sh) {
  using Q = Queries<HD>;
  constexpr int U = Q::kRows;
  const int li = lane % Q::LANES;
  const bool neox = a.rope == KVQ_ROPE_NEOX, rope = a.rope != KVQ_ROPE_NONE, f16 = a.act == KVQ_F16;
  const bool odd = li & 1;
  const int d = Q::dim(li, neox), order = order_of(a.kl.kind);
  // Ordered words of dims 01 23 45 67: pairs of words, the low and the high halves.
  const bool swap = order != 2;
  const uint32_t lows = order == 0 ? 0x3210 : 0x5410, highs = order == 0 ? 0x7654 : 0x7632;
  const uint32_t base = smem_u32(sh.q);
  // both pairings meet pairs 4 li .. 4 li + 3
  const float4* rot = reinterpret_cast<const float4*>(a.rope_tab) + (int64_t)t.p0 * (HD / 4) + 2 * li;
  // The halves of two lanes' chunks change hands: NeoX positions 0..3 and 4..7 of their 16.
  auto exchange = [&](uint32_t (&w)[4]) {
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[2], 1);
    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, odd ? w[1] : w[3], 1);
    if (odd) w[0] = r0, w[1] = r1;
    else w[2] = r0, w[3] = r1;
  };
  bool copied = false;
#pragma unroll 1
  for (int Rw = warp * Q::WARP; Rw < rows; Rw += Q::STEP) {   // the same count for every lane of a warp
    const int R0 = Rw + lane / Q::LANES * U;
    float4 c[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c[u][0] = c[u][1] = make_float4(1.f, 0.f, 1.f, 0.f);
      if (rope && R0 + u < rows) {
        const float4* p = rot + (int64_t)((R0 + u) >> lg) * (HD / 4);
        c[u][0] = p[0];
        c[u][1] = p[1];
      }
    }
    if (!copied) asm volatile("cp.async.wait_all;" ::: "memory");   // a lane's own chunks
    copied = true;
    // (rows behind the last take part: nothing comes of them)
    // A row's largest element, as bits of the activation type (magnitudes are in
    // the order of their bits; a NaN is above all, and its row NaN whatever its
    // scale): two rows in a word.  A rotated element is at most sqrt 2 of it.
    uint32_t w[U][4], top[U / 2];
#pragma unroll
    for (int u = 0; u < U; ++u)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                   : "r"(Q::chunk(base, R0 + u, d))
                   : "memory");
#pragma unroll
    for (int v = 0; v < U / 2; ++v) {
      uint32_t m[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t(&y)[4] = w[2 * v + k];
        constexpr uint32_t mag = 0x7FFF7FFFu;
        m[k] = __vmaxu2(__vmaxu2(y[0] & mag, y[1] & mag), __vmaxu2(y[2] & mag, y[3] & mag));
      }
      top[v] = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
    }
#pragma unroll
    for (int o = Q::LANES / 2; o >= 1; o >>= 1)
#pragma unroll
      for (int v = 0; v < U / 2; ++v) top[v] = __vmaxu2(top[v], __shfl_xor_sync(0xffffffffu, top[v], o));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t bits = u & 1 ? top[u / 2] >> 16 : top[u / 2] & 0xFFFFu;
      const float most = f16 ? __half2float(__ushort_as_half((unsigned short)bits)) : __uint_as_float(bits << 16);
      const int e = hold_exponent(1.4142137f * most);
      const float down = pow2i(-e);
      if (neox) exchange(w[u]);
      float y[8], x[8];
      if (f16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = __half22float2(u2h(w[u][i]));
          y[2 * i] = z.x;
          y[2 * i + 1] = z.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = __uint_as_float(w[u][i] << 16);
          y[2 * i + 1] = __uint_as_float(w[u][i] & 0xFFFF0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= down;
      const float co[4] = {c[u][0].x, c[u][0].z, c[u][1].x, c[u][1].z};
      const float si[4] = {c[u][0].y, c[u][0].w, c[u][1].y, c[u][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = y[i];
      if (neox) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = y[i] * co[i] - y[4 + i] * si[i];
          x[4 + i] = y[i] * si[i] + y[4 + i] * co[i];
        }
      } else if (rope) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = y[2 * i] * co[i] - y[2 * i + 1] * si[i];
          x[2 * i + 1] = y[2 * i] * si[i] + y[2 * i + 1] * co[i];
        }
      }
      uint32_t n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = h2u(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
      if (neox) exchange(n);
      const uint32_t n1 = swap ? n[2] : n[1], n2 = swap ? n[1] : n[2];
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(Q::chunk(base, R0 + u, d)),
                   "r"(__byte_perm(n[0], n2, lows)), "r"(__byte_perm(n[0], n2, highs)),
                   "r"(__byte_perm(n1, n[3], lows)), "r"(__byte_perm(n1, n[3], highs))
                   : "memory");
      if (li == 0) sh.qscale[R0 + u] = a.score_scale * pow2i(e);
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Which of a step's 128 keys a row sees, and which of those are not finite.
struct RowMask {
  int hi, lo, sinks;   // columns c < hi with c >= lo or c < sinks
  const StepMeta* meta;
  __device__ __forceinline__ uint32_t visible(int c) const {   // columns 32 c .. 32 c + 31
    auto below = [&](int x) -> uint32_t {   // bits of columns < x
      const int k = min(max(x - 32 * c, 0), 32);
      return k == 32 ? ~0u : (1u << k) - 1u;
    };
    return below(hi) & (~below(lo) | below(sinks)) & ~(meta->skip[0][c] | meta->skip[1][c]);
  }
  __device__ __forceinline__ void apply(int c, float (&x)[32]) const {
    const uint32_t v = visible(c), b = v & (meta->bad[0][c] | meta->bad[1][c]);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = (v >> i) & 1u ? x[i] : -INFINITY;
    if (__any_sync(0xffffffffu, b != 0)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = (b >> i) & 1u ? NAN : x[i];
    }
  }
};

template <int HD>
__global__ void __launch_bounds__(tc_threads(HD), 1) prefill_tc_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int MT = row_tiles(HD), HB = HD / 64;
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ uint8_t raw_smem[];
  Shared<HD>& sh = *reinterpret_cast<Shared<HD>*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
  volatile int* stop = &sh.stop;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // block index: kv head fastest, then the split, then the tile, last tiles (the longest key ranges) first
  const int kvh = blockIdx.x % a.n_kv_heads, rest = blockIdx.x / a.n_kv_heads;
  const int split = rest % a.n_splits, x = a.n_tiles - 1 - rest / a.n_splits;
  const int G = a.n_heads / a.n_kv_heads;
  if (blockIdx.x == 0) check_starts(a, tid, tc_threads(HD));
  PrefillTile t;
  if (!find_tile(a, x, kvh == 0 && split == 0 && tid == 0, &t)) return;
  const int rows = t.cnt * G;
  const int lg = 31 - __clz(G);   // G is a power of two
  auto out_row = [&](int r) -> int64_t {
    return (int64_t)(t.row0 + (r >> lg)) * a.n_heads + kvh * G + (r & (G - 1));
  };
  const int64_t ws0 = (int64_t)split * a.n_rows * a.n_heads;
  KeyRange kr = key_range<kKeys>(a, t);
  const int j0 = (int)((int64_t)split * kr.n / a.n_splits), j1 = (int)((int64_t)(split + 1) * kr.n / a.n_splits);
  if (t.zero || j0 == j1) {   // no keys: zero rows, or an empty part
    if (t.zero && split == 0) {
      unsigned short* o = static_cast<unsigned short*>(a.out);
      for (int i = tid; i < rows * HD; i += tc_threads(HD)) o[out_row(i / HD) * HD + i % HD] = 0;
    }
    if (a.n_splits > 1)
      for (int r = tid; r < rows; r += tc_threads(HD)) a.ws_ml[ws0 + out_row(r)] = make_float2(-INFINITY, 0.f);
    return;
  }
  const int n = j1 - j0;
  const int na = MT == 1 || rows <= 128 ? 1 : 2;   // row tiles with rows
  // Half steps of row tile rt: the last ones may lie behind all of its queries.
  auto last_pos = [&](int rt) { return t.p0 + ((min(rows, rt * 128 + 128) - 1) >> lg); };
  auto half_steps = [&](int rt) {
    int k = 2 * n;
    while (k > 0 && kr.base<kKeys>(j0 + (k - 1) / 2) + (k - 1) % 2 * kHalf > last_pos(rt)) --k;
    return k;
  };

  constexpr int kMmaWarp = 4 * MT + 8;
  if (warp < 4 * MT || warp >= kMmaWarp)
    copy_queries<HD>(a, t, rows, lg, kvh, warp < 4 * MT ? warp : warp - 8, lane, sh);
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
  } else if (tid == 0) {
    for (int i = 0; i < kStages * 2; ++i) {
      mbar_init(smem_u32(&sh.kfull[0][0] + i), 2);
      mbar_init(smem_u32(&sh.vfull[0][0] + i), 2);
      mbar_init(smem_u32(&sh.kempty[0][0] + i), na);   // every row tile is done with it
      mbar_init(smem_u32(&sh.vempty[0][0] + i), na);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sh.ready[i]), 2);   // K's and V's
    }
    mbar_init(smem_u32(&sh.qfull), 4 * MT + 4);
    for (int i = 0; i < MT; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&sh.sfull[i][h]), 1);
        mbar_init(smem_u32(&sh.pfull[i][h]), 4);
        mbar_init(smem_u32(&sh.ofull[i][h]), 1);
      }
      mbar_init(smem_u32(&sh.qtmem[i]), 4);
      mbar_init(smem_u32(&sh.drain[i]), 1);
    }
    sh.stop = 0;
    mbar_init_fence();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t s_col = HD == 256 ? 256 : 0, o_col = HD == 256 ? 0 : 256;
  constexpr uint32_t q_col = 384;   // kQInTmem

  if (warp < 4 * MT || warp >= kMmaWarp) {
    load_queries<HD>(a, t, rows, lg, warp < 4 * MT ? warp : warp - 8, lane, sh);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.qfull));
    mbar_wait(smem_u32(&sh.qfull), 0, stop);
  }
  if (warp < 4 * MT) {
    // ------------------------------------------------------------ softmax
    regs_set<regs_softmax(HD), regs_launch(HD)>();
    const int rt = warp >> 2;
    if (rt < na) {
      const int R = rt * 128 + (tid & 127);
      const int pos = t.p0 + (min(R, rows - 1) >> lg);
      const int pmin = t.p0 + (rt * 128 >> lg), pmax = last_pos(rt);
      const float qs = R < rows ? sh.qscale[R] : 0.f;
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 lanes of tensor memory
      const uint32_t o_at = tmem + lanes + o_col + rt * HD;
      const int nh = half_steps(rt);
      float m = -INFINITY, l = 0.f, f = 0.f;
      int held = 0, tb = 0, end = 0, ve = 0;
      if constexpr (kQInTmem<HD>) {   // the row's queries, a dim pair a column
        const uint32_t q_at = smem_u32(sh.q) + rt * HB * kBlockBytes;
#pragma unroll 1
        for (int d = 0; d < HD; d += 32) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                         : "r"(q_at + (d / 64) * kBlockBytes + (R & 127) * 128 + (((d / 8 + c) % 8 ^ (R & 7)) << 4))
                         : "memory");
          tmem_st16(tmem + lanes + q_col + rt * (HD / 2) + d / 2, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.qtmem[rt]));
      }
      bool whole = false;
#pragma unroll 1
      for (int u = 0; u < nh; ++u) {
        const int i = u >> 1, hf = u & 1;
        const uint32_t s_at = tmem + lanes + s_col + rt * 128 + hf * 64;
        const StepMeta& meta = sh.meta[i % kSlots];
        if (hf == 0) {   // everything but the scores first
          tb = kr.base<kKeys>(j0 + i);
          end = kr.end(j0 + i);
          const bool inside = tb + kKeys <= min(end, pmin + 1) &&
                              (a.window == 0 || tb > pmax - a.window || tb + kKeys <= a.sinks);
          mbar_wait(smem_u32(&sh.ready[i % kSlots]), (i / kSlots) & 1, stop);
          const int4 head = *reinterpret_cast<const int4*>(meta.head);   // K's exponent and marks, V's
          f = fmaxf(qs * pow2i(head.x), 1.17549435e-38f);                // never 0: -inf stays -inf
          ve = head.z;
          whole = inside && (head.y | head.w) == 0;
        }
        mbar_wait(smem_u32(&sh.sfull[rt][hf]), i & 1, stop);
        tc_fence_after();

        // O of the steps before, times a power of two a row.
        auto scale_o = [&](float c) {
          // O is at rest once the last half step's product is done.  A barrier
          // for even and one for odd half steps: the phase before the awaited
          // one is product u - 3, done before scores u - 1 were, and the phase
          // behind it needs this row's weights, so the parity says which.
          mbar_wait(smem_u32(&sh.ofull[rt][hf ^ 1]), ((u - 1) >> 1) & 1, stop);
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < HD; d += 8) {   // few registers: the scores are live
            float o[8];
            tmem_ld8_wait(o_at + d, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= c;
            tmem_st8(o_at + d, o);
          }
        };
        // The row's 64 scores, all in registers; P then takes the place of S.
        float x[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(s_at + 32 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_wait(x[c]);
        if (__builtin_expect(!whole, 0)) {
          RowMask mask;
          mask.hi = min(end - tb, pos - tb + 1);
          mask.lo = a.window == 0 ? 0 : pos - a.window + 1 - tb;
          mask.sinks = a.window == 0 ? 0 : a.sinks - tb;
          mask.meta = &meta;
#pragma unroll
          for (int c = 0; c < 2; ++c) mask.apply(2 * hf + c, x[c]);
        }
        float mc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mc[e] = fmaxf(x[0][e], x[0][e + 4]);
#pragma unroll
        for (int k = 8; k < 64; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mc[e] = fmaxf(mc[e], fmaxf(x[k / 32][k % 32 + e], x[k / 32][k % 32 + 4 + e]));
        const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * f;
        const bool raise = mx > m + kLazy;
        if (__builtin_expect(__any_sync(0xffffffffu, raise || ve != held), 0)) {
          const float co = raise ? ex2(m - mx) : 1.f;   // 2^-inf = 0: no key so far
          if (raise) m = mx;
          l *= co;
          if (u > 0) scale_o(co * pow2i(held - ve));
          held = ve;
        }
        const float sub = m == -INFINITY ? 0.f : m - kShift;
        const uint64_t f2 = pack2(f, f), sub2 = pack2(-sub, -sub);
        uint64_t sum[2] = {pack2(l, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 y = unpack2(fma2(pack2(x[c][2 * k], x[c][2 * k + 1]), f2, sub2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            sum[k & 1] = add2(sum[k & 1], pack2(p0, p1));
            w[k] = h2u(__floats2half2_rn(p0, p1));
          }
          tmem_st16(s_at + 16 * c, w);
        }
        {
          const float2 s2 = unpack2(add2(sum[0], sum[1]));
          l = s2.x + s2.y;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.pfull[rt][hf]));
      }
      // ---- the result: O 2^held / l, dims back in order
      if (nh > 0) mbar_wait(smem_u32(&sh.ofull[rt][(nh - 1) & 1]), ((nh - 1) >> 1) & 1, stop);
      tc_fence_after();
      const bool mine = R < rows;
      const int64_t orow = out_row(mine ? R : 0);
      const float up = pow2i(held) * (a.n_splits > 1 ? 1.f : (l == 0.f ? 0.f : 1.f / l));
      const int order = order_of(a.vl.kind);
      const uint32_t q_at = smem_u32(sh.q) + rt * HB * kBlockBytes;
      if (mine && a.n_splits > 1) a.ws_ml[ws0 + orow] = make_float2(m == -INFINITY ? m : m - kShift, l);
#pragma unroll 1
      for (int d = 0; d < HD; d += 32) {
        float o[32], y[32];
        if (nh > 0) {
          tmem_ld32(o_at + d, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (order == 2) {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[(e & ~7) | dim_at(2, e & 7)] = o[e];
        } else if (order == 1) {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[(e & ~7) | dim_at(1, e & 7)] = o[e];
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o[e];
        }
        if (a.n_splits == 1) {   // to the row's place of the query tile, no longer needed
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = y[8 * c + 2 * e] * up, y1 = y[8 * c + 2 * e + 1] * up;
              if (a.act == KVQ_F16) {
                w[e] = h2u(__floats2half2_rn(y0, y1));
              } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
                w[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            const int k = (d / 8 + c) & 7;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             q_at + (d / 64) * kBlockBytes + (R & 127) * 128 + ((k ^ (R & 7)) << 4)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        } else if (mine) {
          float4* dst = reinterpret_cast<float4*>(a.ws_acc + (ws0 + orow) * HD + d);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(y[4 * e] * up, y[4 * e + 1] * up, y[4 * e + 2] * up, y[4 * e + 3] * up);
        }
      }
      if (a.n_splits == 1) {   // whole rows at a time: HD / 8 lanes write one
        constexpr int LANES = HD / 8, RPW = 32 / LANES;
        __syncwarp();
        const int c = lane % LANES;
#pragma unroll 4
        for (int k = 0; k < 32 / RPW; ++k) {
          const int r = (warp & 3) * 32 + k * RPW + lane / LANES, Rr = rt * 128 + r;
          uint4 y;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                       : "r"(q_at + (c / 8) * kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)));
          if (Rr < rows)
            *reinterpret_cast<uint4*>(static_cast<unsigned short*>(a.out) + out_row(Rr) * HD + 8 * c) = y;
        }
      }
      tc_fence_before();
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ K and V: one code, half the instructions to fetch
    regs_set<regs_produce(HD), regs_launch(HD)>();
    const bool is_v = warp >= 4 * MT + 4;
    produce_kind<HD>(is_v ? a.vl.kind : a.kl.kind, is_v, a, t, kr, j0, n, kvh, (tid - 128 * MT) & 127, sh, stop);
  } else {
    // ------------------------------------------------------------ products
    regs_set<kRegsProducts, regs_launch(HD)>();   // the whole warpgroup, one warp of which works
    const int rt = warp - kMmaWarp;
    if (rt < na) {
      // A warp issues the products of one row tile, so neither waits for the
      // other's softmax.  The whole warp walks the steps and one lane issues:
      // the operands then stay in uniform registers, where the instruction
      // takes them (a lone lane in a branch of its own spent 120 cycles on each
      // product, twice its length).
      constexpr int RU = kStages / HB;   // steps a ring
      constexpr uint32_t id_qk = idesc_f16(kHalf, false), id_pv = idesc_f16(HD, true);
      constexpr int kHalfBytes = kHalf * 128;   // half the keys of a block
      // descriptors count addresses in 16 bytes
      const uint64_t qd = smem_desc(smem_u32(sh.q) + rt * HB * kBlockBytes, 16), kd = smem_desc(smem_u32(sh.k), 16),
                     vd = smem_desc(smem_u32(sh.v), kBlockBytes);
      const bool leader = elect_one();
      const int nh = __shfl_sync(0xffffffffu, half_steps(rt), 0);
      const uint32_t s_at = __shfl_sync(0xffffffffu, tmem, 0) + s_col + rt * 128;
      const uint32_t o_at = __shfl_sync(0xffffffffu, tmem, 0) + o_col + rt * HD;
      const uint32_t q_at = __shfl_sync(0xffffffffu, tmem, 0) + q_col + rt * (HD / 2);
      auto qk = [&](int u) {   // scores of half step u
        const int i = u >> 1, hf = u & 1, us = i % RU;
        mbar_wait(smem_u32(&sh.kfull[us][hf]), (i / RU) & 1, stop);
        tc_fence_after();
        if (leader) {
          const uint64_t b = kd + (us * HB * kBlockBytes + hf * kHalfBytes) / 16;
#pragma unroll
          for (int k = 0; k < 4 * HB; ++k)
            if constexpr (kQInTmem<HD>)
              mma_ts(s_at + hf * 64, q_at + 8 * k, b + ((k / 4) * kBlockBytes + 32 * (k % 4)) / 16, id_qk, k > 0);
            else
              mma_ss(s_at + hf * 64, qd + ((k / 4) * kBlockBytes + 32 * (k % 4)) / 16,
                     b + ((k / 4) * kBlockBytes + 32 * (k % 4)) / 16, id_qk, k > 0);
          mma_commit(smem_u32(&sh.kempty[us][hf]));
          mma_commit(smem_u32(&sh.sfull[rt][hf]));
        }
        __syncwarp();
      };
      auto pv = [&](int u) {   // O of half step u
        const int i = u >> 1, hf = u & 1, us = i % RU;
        mbar_wait(smem_u32(&sh.vfull[us][hf]), (i / RU) & 1, stop);
        mbar_wait(smem_u32(&sh.pfull[rt][hf]), i & 1, stop);
        tc_fence_after();
        if (leader) {
          const uint64_t b = vd + (us * HB * kBlockBytes + hf * kHalfBytes) / 16;
#pragma unroll
          for (int k = 0; k < kHalf / 16; ++k)
            mma_ts(o_at, s_at + hf * 64 + 8 * k, b + 2048 * k / 16, id_pv, u > 0 || k > 0);
          mma_commit(smem_u32(&sh.vempty[us][hf]));
          mma_commit(smem_u32(&sh.ofull[rt][hf]));
        }
        __syncwarp();
      };
      // Scores run two half steps ahead of the weights, in two buffers.
      if constexpr (kQInTmem<HD>) mbar_wait(smem_u32(&sh.qtmem[rt]), 0, stop);   // (each wait has its fence behind it)
      if (nh > 0) qk(0);
      if (nh > 1) qk(1);
#pragma unroll 1
      for (int u = 0; u < nh; ++u) {
        pv(u);
        if (u + 2 < nh) qk(u + 2);
      }
      // blocks behind this row tile's queries are given back unread
#pragma unroll 1
      for (int u = nh; u < 2 * n; ++u) {
        const int i = u >> 1, hf = u & 1, us = i % RU;
        mbar_wait(smem_u32(&sh.kfull[us][hf]), (i / RU) & 1, stop);
        mbar_wait(smem_u32(&sh.vfull[us][hf]), (i / RU) & 1, stop);
        if (leader) {
          mma_commit(smem_u32(&sh.kempty[us][hf]));
          mma_commit(smem_u32(&sh.vempty[us][hf]));
        }
        __syncwarp();
      }
      if (leader) mma_commit(smem_u32(&sh.drain[rt]));
      __syncwarp();
      mbar_wait(smem_u32(&sh.drain[rt]), 0, stop);
      tc_fence_before();
    }
  }
  __syncthreads();
  if (tid == 0 && sh.stop) report(a.status, KVQ_DEV_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HD>
cudaError_t launch(cudaLaunchConfig_t& lc, const PrefillArgs& a) {
  lc.blockDim = dim3(tc_threads(HD));
  lc.dynamicSmemBytes = shared_bytes<HD>();
  static std::atomic<bool> ready[64];   // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    // the roles' register split counts on the launch's share
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, prefill_tc_kernel<HD>);
    if (e != cudaSuccess) return e;
    if (at.numRegs < regs_launch(HD)) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(prefill_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)shared_bytes<HD>());
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  return cudaLaunchKernelEx(&lc, prefill_tc_kernel<HD>, a);
}

}  // namespace

int prefill_tc_rows(int head_dim) { return 128 * row_tiles(head_dim); }

cudaError_t launch_prefill_tc(cudaLaunchConfig_t& lc, int head_dim, const PrefillArgs& a) {
  switch (head_dim) {
    case 64: return launch<64>(lc, a);
    case 128: return launch<128>(lc, a);
    default: return launch<256>(lc, a);
  }
}

}  // namespace kvq

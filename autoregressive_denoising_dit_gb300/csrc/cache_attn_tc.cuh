// Attention over a cache on the tensor cores (psv_cache_attention): shared
// heads, ragged lengths, causal / prefix / document masks, a tanh score cap
// and a distance bias.
//
//   s_ij = scale q_i.k_j;  s = cap tanh(s / cap);  s -= slope |qpos_i - kpos_j|
//   o_i  = sum_j exp(s_ij - m_i) v_j / l_i,  l_i = sum_j exp(s_ij - m_i)
//
// in one pass over the keys with a running maximum m and sum l (f32, in the
// log2 domain).  CTA pairs (clusters of two SMs) with 2-SM tcgen05 MMAs.  A
// work piece is 256 query rows of one (sequence, kv head), 128 per CTA, over
// its visible keys or one of nsplit equal shares of them, walked in tiles of
// 256 keys:
//   S_j = Q K_j^T   M=256, N=256, K=dh    (each CTA holds 128 of the keys)
//   O  += P_j V_j   M=256, N=dh,  K=256   (each CTA holds dh/2 columns of V)
// The query heads that share a kv head are rows of one tile (row = token * G +
// head), so a single token of G heads costs one tile's MMAs, not G.  V is read
// as users keep it, token-major: its tile is the MMA's MN-major B operand, no
// transposed copy is made.  Heads narrower than 64 or 128 are zero-filled by
// the tensor map's bounds.  S, P and O have TMEM columns of their own, so
// S_{j+1} runs while the softmax works on S_j.  Warp roles, 384 threads:
//   warp 0       TMA: Q tile of a piece, then this CTA's K halves (2 stages);
//                hands the pieces on to the softmax warps
//   warp 1       TMEM allocator (both CTAs) and MMA issuer (even CTA)
//   warp 2       TMA: this CTA's V halves (3 stages)
//   warp 3       even CTA: takes pieces from the work queue, publishes them
//   warps 4..11  softmax, two threads per query row (lanes l and l + 16), 128
//                keys each, through 16-lane TMEM accesses
// The weights are rounded to the operand type for P V: both operands of a product
// have 16 bits, and f32 weights would take two or three times the products.  That
// and the output's rounding are what o differs by from 32-bit arithmetic (bf16,
// relative to 64 bits: 1.8e-3 to 2.3e-3, with f32 weights 1.6e-3 to 1.7e-3; f16
// 2.9e-4, 2.1e-4); l is the sum of the weights before they are rounded.
// The softmax paces a tile, not the tensor cores: 2500 clocks against 2048 of
// products (of a tile's clocks, 570 go into the maximum, 1650 into the weights
// and their way to TMEM), and so does what a feature adds to it: the cap 1400
// clocks (four packed FMA-pipe operations a pair), masks seen key by key 1200.
// It is latency more than issue: two softmax warps a scheduler, each a chain of
// TMEM reads, the maximum, the weights and their way back, use 39% of the issue
// slots (with the cap 51%) and 33% of the exponential unit.
// Between pieces 3000 clocks are lost (the last P.V, O's way out, the next
// piece's notes); issuing the next piece's first S ahead of the last P.V was
// measured slower (short sequences 80 -> 84 us).
// Measured, calls on the same inputs one after another, 12 heads of 128, bf16:
// 12480 rows x 12480 keys 547 to 585 us (1640 to 1750 TFLOP/s, as the power cap
// allows), four sequences of 1560 rows x 7800 keys 211 us (1415; 13% of its row tiles
// are empty), with the distance bias 227 (243 where inputs change from call to
// call), with a cap of 50 285 (scores of deviation 8: 404); nine documents of 12480
// rows 132 us.
// Pieces are taken from a device counter (the first of a pair is its own
// index) that the last pair to finish rewinds.  Shares of a long cache leave
// O, m and l in a workspace and a second small kernel joins them in a fixed
// order; how many shares there are depends on the problem's heads, rows and
// key capacity but not on the batch, so a sequence's bits do not depend on it.
#pragma once

#include <cuda.h>

#include "../../include/psv.h"
#include "cache_cap.cuh"
#include "cache_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

namespace psv {

namespace cattn {

constexpr int QT = 128;  // query rows per CTA
constexpr int KT = 256;  // keys per tile
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_S = 0, COL_P = 256, COL_O = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 384;
constexpr int kStages = 3;
constexpr int kRegsLow = 64, kRegsHigh = 216;
constexpr int kRegsNeeded = 128 * kRegsLow + 256 * kRegsHigh;
// A step of 16 values for 128 rows: 8-row groups of 256 bytes, in each the rows'
// first 8 values (16 bytes a row), then their second 8 (no swizzle).
constexpr int kLinBytes = 128 * 32;
// Readers of a published piece: in both CTAs the Q/K loader (which hands it on
// to its CTA's softmax warps) and the V loader; the even CTA's MMA issuer.
constexpr int kPieceReaders = 5;
constexpr int kHanded = 4;  // pieces handed on at a time
constexpr int kOutRow = 144, kOutBytes = 16 * kOutRow;

// LIN: with the products that add the distance bias (see cache_attn_kernel).
template <int DH, bool LIN>
struct Cfg {
  static constexpr int KK = 2;                  // K stages (measured as fast as three)
  static constexpr int NA = DH / 64;            // 64-wide (128-byte) atoms along dh
  static constexpr int VR = DH / 2;             // V columns held per CTA
  static constexpr int Q_BYTES = QT * DH * 2;
  static constexpr int K_BYTES = 128 * DH * 2;  // this CTA's 128 keys of a tile
  static constexpr int V_BYTES = KT * VR * 2;   // 256 keys x this CTA's columns
  static constexpr int ATOM = 128 * 128;        // 128 rows of 128 bytes
  static constexpr int V_ROW = VR * 2;          // bytes of a V row: 128 or 64 (its swizzle width)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_BYTES;
  static constexpr int OFF_V = OFF_K + KK * K_BYTES;
  static constexpr int OFF_LIN = OFF_V + kStages * V_BYTES;  // Q's part, K's part, K's negative part
  // Per softmax warp 16 rows of 2 * 64 bytes, 16 apart (no bank twice): O on its way out.
  static constexpr int OFF_OUT = OFF_LIN + (LIN ? 3 * kLinBytes : 0);
  static constexpr int OFF_BAR = OFF_OUT + 8 * kOutBytes;
  static constexpr int N_BARS = 13 + 5 * kStages + 2 * kHanded;  // an even number
  // barriers, TMEM address, two published piece slots and the pieces handed on
  static constexpr size_t SMEM = OFF_BAR + N_BARS * 8 + 16 + (4 + 2 * kHanded) * 16;
  static constexpr int OH = DH / 2;             // O columns per thread
};

// By the whole warp: every lane polls (one access for all of them); a branch to
// one lane and a shuffle of its answer cost more than twice as much, and these
// waits are on the kernels' critical path even where they find the barrier done.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, ERR_ATTN_TIMEOUT));
}

__device__ __forceinline__ void mbar_arrive_local(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Instruction descriptor: f32 accumulate, A and B of the operand type, A
// K-major, B K-major or MN-major.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool b_mn) {
  return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// MN-major operand [k rows][row_bytes of the MN index]: 8-row groups along k
// are 8 * row_bytes apart; one row spans the whole MN extent (64 or 32
// values), so the offset between MN groups is not used.
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem_addr, uint32_t row_bytes) {
  return umma_desc_kmajor(smem_addr, row_bytes);
}

// K-major operand in the layout of kLinBytes.
__device__ __forceinline__ uint64_t desc_lin(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 16 |
         static_cast<uint64_t>(256 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

__device__ __forceinline__ void umma_pair_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_lin(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int z) {
  tma_load_3d_pair(dst, map, bar_cluster, 0, 0, z);
}

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster,
                                                 int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 16-lane TMEM accesses (shape 16x32bx2): threads 0-15 reach lanes [base,
// base + 16) at column c, threads 16-31 the same lanes at column c + SPLIT.
template <int SPLIT>
__device__ __forceinline__ void tmem_ld32x(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr), "n"(SPLIT));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
template <int SPLIT>
__device__ __forceinline__ void tmem_ld16x(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "n"(SPLIT));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16x(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, "
      "{%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17};" ::"r"(taddr),
      "n"(SPLIT), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
      "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (x0, x1) * s + (b, b) on the packed f32x2 path.
__device__ __forceinline__ void ffma2(float& x0, float& x1, float s, float b) {
  uint64_t x, sv, bv;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(sv) : "f"(s));
  asm("mov.b64 %0, {%1, %1};" : "=l"(bv) : "f"(b));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(sv), "l"(bv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}
__device__ __forceinline__ void fadd2(float& a0, float& a1, float b0, float b1) {
  uint64_t a, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("add.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// (x0, x1) = (x0, x1) * s + (c, c + 1) * bs + as, c a constant.
__device__ __forceinline__ void bias2(float& x0, float& x1, float s, float c, float bs, float as) {
  uint64_t x, y, sv, bv, av;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(c), "f"(c + 1.0f));
  asm("mov.b64 %0, {%1, %1};" : "=l"(sv) : "f"(s));
  asm("mov.b64 %0, {%1, %1};" : "=l"(bv) : "f"(bs));
  asm("mov.b64 %0, {%1, %1};" : "=l"(av) : "f"(as));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(y) : "l"(bv), "l"(av));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(sv), "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    return pack_bf16x2(lo, hi);
  } else {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int4 v) {
  asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ int4 ld_shared_v4(const void* ptr) {
  int4 v;
  asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(ptr))
               : "memory");
  return v;
}
__device__ __forceinline__ bool mbar_try_wait_acq_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_acq_cluster(uint64_t* bar, uint32_t parity, int* err,
                                                      uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait_acq_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait_acq_cluster(bar, parity)) return true;
    if ((i & 63) == 63) {
      if (error_raised(err)) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        raise_error(err, ERR_ATTN_TIMEOUT);
        return false;
      }
    }
  }
}

// The limit of the queue's wait for a slot: its readers release it at the end of
// their piece, which may be 2^20 key tiles (or 2^23 row tiles of the mass) long,
// over 2 s.  A tile takes 1 to 4 us.
constexpr uint64_t kTileLimitNs = 20000;
__device__ __forceinline__ uint64_t piece_limit_ns(int tiles0, int tiles1) {
  return kWaitLimitNs + (static_cast<uint64_t>(tiles0) + static_cast<uint64_t>(tiles1)) * kTileLimitNs;
}

// What a tile of 256 keys and a unit of rows hold, from a small kernel run
// before the attention where positions or documents are given: tiles that no
// row of a unit sees are not loaded, tiles that every row sees whole are not
// masked, and a tile of consecutive positions needs no position per key.
struct alignas(16) KeyTile {
  int pos_min, pos_max, doc_min, doc_max;  // over the keys in use (min > max: none)
  int base;                                // the first key's position
  int run;                                 // positions are base, base + 1, ..
  int sorted;                              // documents do not decrease
  int cut;  // the first `cut` keys are of doc_min, the others of doc_max; -1: not so
};
struct RowUnit {
  int pos_min, pos_max, doc_min, doc_max;
};

struct TcParams {
  CacheParams c;
  int rows_cta;     // packed rows of a CTA: a multiple of G
  int tok_cta;      // tokens of a CTA: rows_cta / G
  int units;        // units of 2 * tok_cta tokens per (sequence, kv head)
  int nsplit;       // shares of every unit's keys
  int tail_split;   // shares of the last unit's keys, where only those are shared; or 0
  int n_pieces;
  int part_rows;    // rows of a unit in the workspace
  int width;        // columns of a row there (the kernel's DH)
  int meta_vec;     // k_pos and k_doc rows are 16-byte aligned
  int meta_heads;   // kv heads with k_pos / k_doc rows of their own (1: shared)
  int tiles;        // key tiles of the buffer
  KeyTile* key_tiles;  // [B][meta_heads][tiles], with k_pos or k_doc only
  RowUnit* row_units;  // [B][units]
  // [B][units]: a sequence's units with most key tiles first (unit_order[0] < 0:
  // they have about as many), for order_heads kv heads at a time; or null.
  int* unit_order;
  int order_heads;
  // [Hkv]: whether a head group's slopes fit the operand type, and the rows'
  // slopes in three parts (kLinBytes).
  int* lin_ok;
  uint16_t* lin_q;
  CapForm cap;                    // where c.softcap > 0
  float cap_small, cap_mid;       // scores up to which cap2's polynomials hold (below 0: none)
  float2 cap_c3[3], cap_c7[7];    // their coefficients, each twice
  int* queue;       // next piece, pairs done (zero between launches)
  float* part_o;    // [piece][part_rows][DH], unnormalised
  float2* part_ml;  // [piece][part_rows]: m (log2), l
};

// Positions or documents of keys [j, j + 4), j a multiple of 4; behind the
// keys the last one's (those keys are masked by their number).
__device__ __forceinline__ int4 ld_meta4(const int32_t* m, int j, int k_len, int vec) {
  if (vec && j + 4 <= k_len) return __ldg(reinterpret_cast<const int4*>(m + j));
  const int last = k_len - 1;
  return make_int4(__ldg(m + min(j, last)), __ldg(m + min(j + 1, last)), __ldg(m + min(j + 2, last)),
                   __ldg(m + min(j + 3, last)));
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// First c in [lo, hi) with d[c] >= doc, else hi (d does not decrease).
__device__ __forceinline__ int first_doc(const int32_t* d, int lo, int hi, int doc) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(d + mid) < doc) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
// The n lowest bits (n below 0: none, over 31: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// {sequence * Hkv + kv head, unit, share (7 bits) and above it the number of
// key tiles from w on that every row sees whole, w (LIN: whether the tensor
// cores may add the bias)}, x = -1 past the end; and
// {k_len, q_len, first key tile, key tiles}.
struct Piece {
  int4 a, b;
};

__device__ __forceinline__ int4 piece_index(const TcParams& p, int k) {
  const int BH = p.c.B * p.c.Hkv;
  if (p.tail_split) {
    // The last units' shares come last.
    const int whole = p.units - 1, t = k - BH * whole;
    return t < 0 ? make_int4(k / whole, k % whole, 0, 0) : make_int4(t / p.tail_split, whole, t % p.tail_split, 0);
  }
  const int s = k % p.nsplit, r = k / p.nsplit;
  if (p.unit_order) {
    const int per_seq = p.c.Hkv * p.units, b = r / per_seq, q = r % per_seq;
    const int* order = p.unit_order + static_cast<int64_t>(b) * p.units;
    if (order[0] < 0) return make_int4(r / p.units, r % p.units, s, 0);
    const int h0 = q / (p.order_heads * p.units) * p.order_heads, at = q - h0 * p.units;
    const int heads = min(p.order_heads, p.c.Hkv - h0);
    return make_int4(b * p.c.Hkv + h0 + at % heads, order[at / heads], s, 0);
  }
  // Causal: the units with most keys first, so that the last pieces taken are
  // short.  Otherwise the units of one (sequence, kv head) run together and
  // share its keys in L2.
  if (p.c.causal) return make_int4(r % BH, p.units - 1 - r / BH, s, 0);
  return make_int4(r / p.units, r % p.units, s, 0);
}

// Into how many shares a unit's keys are divided.
__device__ __forceinline__ int unit_shares(const TcParams& p, int unit) {
  return p.tail_split && unit == p.units - 1 ? p.tail_split : p.nsplit;
}

// Keys [0, limit) hold every key that some row of the unit sees.
__device__ __forceinline__ int unit_limit(const TcParams& p, int b, int unit, int k_len, int q_len) {
  if (!p.c.causal || p.c.k_pos || p.c.q_pos) return k_len;
  const int last = min(q_len, (unit + 1) * 2 * p.tok_cta) - 1;
  const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
  return min(k_len, max(max(k_len - q_len + last + 1, prefix), 0));
}

// Narrows the key tiles [first, last) to those from the first to the last one
// with a key that some row of the unit sees, and finds a stretch of tiles that
// every row sees whole, [whole, whole + count) (by the whole warp).
__device__ __forceinline__ void seen_tiles(const TcParams& p, int b, int kvh, int unit, int& first, int& last,
                                           int& whole, int& count) {
  const KeyTile* tiles = p.key_tiles + (static_cast<int64_t>(b) * p.meta_heads + (p.meta_heads > 1 ? kvh : 0)) * p.tiles;
  const RowUnit u = p.row_units[static_cast<int64_t>(b) * p.units + unit];
  const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
  const bool ordered = p.c.causal && p.c.k_pos;
  const int most = max(u.pos_max + 1, prefix), least = max(u.pos_min + 1, prefix);
  auto is_whole = [&](const KeyTile& k) {
    return (!p.c.k_doc || (k.doc_min == k.doc_max && u.doc_min == k.doc_min && u.doc_max == k.doc_min)) &&
           (!ordered || k.pos_max < least);
  };
  int lo = 0x7fffffff, hi = 0, w0 = 0x7fffffff, w1 = 0x7fffffff;
  for (int t = static_cast<int>(lane_id()); t < last; t += 32) {
    const KeyTile k = tiles[t];
    const bool docs = !p.c.k_doc || (k.doc_min <= u.doc_max && k.doc_max >= u.doc_min);
    if (docs && (!p.c.causal || k.pos_min < most)) {
      lo = min(lo, t);
      hi = t + 1;
      if (is_whole(k)) w0 = min(w0, t);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  w0 = __reduce_min_sync(0xffffffffu, w0);
  for (int t = static_cast<int>(lane_id()); t < hi; t += 32)
    if (t > w0 && w1 > t && !is_whole(tiles[t])) w1 = t;
  w1 = min(__reduce_min_sync(0xffffffffu, w1), hi);
  first = min(lo, hi);
  last = hi;
  whole = min(w0, hi);
  count = max(w1 - whole, 0);
}

// LIN: the rows of the piece's unit lie at or behind all keys of tiles up to x,
// and at or before those of tiles from y on; the other tiles are done key by key
// (all of them if the slopes do not fit).
__device__ __forceinline__ int2 lin_tiles(const TcParams& p, const Piece& pc) {
  const int unit = 2 * p.tok_cta, first = pc.b.x - pc.b.y + pc.a.y * unit;
  const int last = pc.b.x - pc.b.y + min(pc.b.y, (pc.a.y + 1) * unit) - 1;
  static_assert(KT == 256, "the shifts");
  return pc.a.w ? make_int2((first - (KT - 1)) >> 8, (last + KT - 1) >> 8) : make_int2(-1, 0x7fffffff);
}
// Which of the two: 1, -1, or 0 for neither.
__device__ __forceinline__ int tile_side(int2 lin, int tile) { return tile <= lin.x ? 1 : tile >= lin.y ? -1 : 0; }

// The j-th key tile of a piece.  With a distance bias (and positions that are
// indexes) the walk starts at the unit's last row and goes down, then from the
// last tile down to there: the tiles towards the rows have the larger scores,
// and in ascending order nearly every one of them raised the running maximum
// and had O rescaled (wave with bias 257 us).
template <bool ROTATE>
__device__ __forceinline__ int tile_at(const TcParams& p, const Piece& pc, int j) {
  if constexpr (!ROTATE) return pc.b.z + j;
  const int row = pc.b.x - pc.b.y + min(pc.b.y, (pc.a.y + 1) * 2 * p.tok_cta) - 1;  // (may be negative)
  const int at = min(max(max(row, 0) / KT - pc.b.z, 0), pc.b.w - 1) - j;
  return at >= 0 ? pc.b.z + at : pc.b.z + pc.b.w + at;
}

// Whether a key tile ends behind the keys inside the buffer (rows behind the
// buffer are zero-filled by the tensor map).
__device__ __forceinline__ bool zero_tile(const TcParams& p, int key0, int k_len) {
  return key0 + KT > k_len && k_len < p.c.Lk;
}

// cap log2(e) tanh(s inv) of a pair of scores as s P(s^2), P of degree N - 1
// with coefficients c (scaled by the powers of inv = scale / cap and by cap
// log2 e), from interpolating tanh(sqrt z) / sqrt z at Chebyshev points: 3 of
// [0, 0.0324] for |s inv| <= 0.18, 7 of [0, 1] for |s inv| <= 1 (5.6e-8 and 5e-8 of
// the score).  The packed products are bound by the FMA pipe, which is why scores
// far below the cap have a short polynomial, and why the cap's powers are in the
// coefficients where f32 holds them (cap_within takes one product more: four
// sequences of 1560 rows, heads of 64, cap 20, deviation 4: 399 us, 421 with it).
template <int N>
__device__ __forceinline__ void cap2(float& x0, float& x1, const float2* c) {
  uint64_t x, z, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mul.rn.f32x2 %0, %1, %1;" : "=l"(z) : "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(z), "l"(pair_bits(c[N - 1])), "l"(pair_bits(c[N - 2])));
#pragma unroll
  for (int k = N - 3; k >= 0; --k) asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(y) : "l"(z), "l"(pair_bits(c[k])));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}

// F: what the scores need beside the row's key limit (lengths, causal, prefix),
// as bits, so that a kernel holds the registers of its own work only: the score
// cap, the distance bias, documents and explicit positions, and (with F_CAP) a cap
// over kCapLow, whose forms beside the usual caps' made both spill.
enum : int { F_CAP = 1, F_BIAS = 2, F_META = 4, F_WIDE = 8 };
//
// With the bias alone (LIN) the tensor cores add it, as its multiply-adds per
// score would lengthen the softmax, which paces the kernel: where all rows of a
// unit lie behind (before) a tile's keys, key c of the tile gets
// -slope (d0 -+ c) = -+slope d0 +- slope c; the row's slope / scale, in three
// parts of the operand type (24 bits), times c (0..255, exact) is one more
// step of 16 products, and -+slope d0 is the same for the whole row.  Only the
// tiles that a unit's rows lie in are done key by key.
template <int DH, bool BF16, int F>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmL,
                      const __grid_constant__ TcParams p) {
  // LATE: the next work item is taken once its slot is free, so that a pair holds
  // one item ahead, not two (two sequences of 1560 rows 119 -> 111 us).  Capped
  // kernels then spill in the softmax (prefix 696 -> 785).
  constexpr bool LATE = !(F & F_CAP);
  constexpr bool LIN = F == F_BIAS, ROT = (F & F_BIAS) && !(F & F_META);
  using C = Cfg<DH, LIN>;
  constexpr int KS = kStages, KK = C::KK;
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the same in both CTAs: swizzled tiles need it
    if (threadIdx.x == 0) raise_error(p.c.err, ERR_BOUNDS);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;      // even CTA: both Q tiles landed
  uint64_t* s_full = bars + 1;      // both: S of a tile in TMEM
  uint64_t* s_free = bars + 2;      // even: all 16 softmax warps read S
  uint64_t* p_full_a = bars + 3;    // even: ... wrote the first half of P
  uint64_t* o_done = bars + 4;      // both: P.V of a tile done
  uint64_t* p_full_b = bars + 5;    // even: ... and the second half
  uint64_t* q_empty = bars + 6;     // both: the last S MMA of a piece is done
  uint64_t* pc_full = bars + 8;     // [2] both: piece slot published
  uint64_t* pc_empty = bars + 10;   // [2] even: every reader took the slot
  uint64_t* k_full = bars + 12;     // [KS] even
  uint64_t* k_empty = k_full + KS;  // [KS] both
  uint64_t* v_full = k_empty + KS;  // [KS] even, one arrival per CTA
  uint64_t* v_empty = v_full + KS;  // [KS] both
  uint64_t* v_zero = v_empty + KS;  // [KS] own: a V tile to be zeroed behind the keys landed
  uint64_t* h_full = bars + 13 + 5 * KS;   // [kHanded] own: a piece handed on to the softmax warps
  uint64_t* h_empty = h_full + kHanded;    // [kHanded] own: all eight took it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  int4* pc_slot = reinterpret_cast<int4*>(smem + C::OFF_BAR + C::N_BARS * 8 + 16);  // [2][2]
  int4* sm_piece = pc_slot + 4;                                                            // [kHanded][2]
  static_assert((C::N_BARS * 8) % 16 == 0, "the piece slots are 16-byte aligned");

  pdl_trigger();
  const int warp = warp_id(), lane = lane_id();
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  int* err = p.c.err;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < C::N_BARS; ++i) {
      const bool all16 = i == 2 || i == 3 || i == 5;
      const bool readers = i == 10 || i == 11;
      const bool two = i >= 12 + 2 * KS && i < 12 + 3 * KS;  // v_full
      const bool taken = i >= 13 + 5 * KS + kHanded;
      mbar_init(&bars[i], all16 ? 16 : readers ? kPieceReaders : two ? 2 : taken ? 8 : 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if constexpr (LIN) {
    // Key c of a tile: c, c, c, 0, ..; and the same negative.
    for (int i = threadIdx.x; i < 256; i += kThreads) {
      const int n = i & 127;
      const float c = static_cast<float>(rank * 128 + n) * (i < 128 ? 1.0f : -1.0f);
      uint4* dst = reinterpret_cast<uint4*>(smem + C::OFF_LIN + (1 + i / 128) * kLinBytes + (n / 8) * 256 + (n % 8) * 16);
      dst[0] = make_uint4(pack2<BF16>(c, c), pack2<BF16>(c, 0.0f), 0, 0);
      dst[8] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const uint32_t pc_empty0 = mapa_shared(pc_empty, 0);
  auto take_piece = [&](int i, Piece& pc) -> bool {
    if (!mbar_wait_acq_cluster(&pc_full[i & 1], (i >> 1) & 1, err)) return false;
    pc.a = ld_shared_v4(&pc_slot[2 * (i & 1)]);
    pc.b = ld_shared_v4(&pc_slot[2 * (i & 1) + 1]);
    return pc.a.x >= 0;
  };
  // A slot may be rewritten once every reader has released it.  The reads must
  // be done by then, so the release is at cluster scope (a CTA-scope arrive on
  // the other CTA's barrier was seen to overtake them); as that waits for the
  // thread's other traffic, readers release late, at the end of their piece.
  auto release_piece = [&](int i) { mbar_arrive_cluster(pc_empty0 + (i & 1) * 8); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 3 && leader) {
      // ---------------- work queue (the whole warp scans the key tiles)
      const int pairs = static_cast<int>(gridDim.x >> 1);
      int k = static_cast<int>(blockIdx.x >> 1);
      int ahead[2] = {0, 0};  // key tiles of the last two pieces published
      for (int i = 0;;) {
        Piece pc;
        bool rows = true;
        pc.a = make_int4(-1, 0, 0, 0);
        pc.b = make_int4(0, 0, 0, 0);
        if (k < p.n_pieces) {
          pc.a = piece_index(p, k);
          const int b = pc.a.x / p.c.Hkv;
          const int nk = cache_k_len(p.c, b), nq = cache_q_len(p.c, b);
          rows = pc.a.y * 2 * p.tok_cta < nq;
          int first = 0, last = (unit_limit(p, b, pc.a.y, nk, nq) + KT - 1) / KT;
          int whole = 0, count = 0;
          if (rows && p.key_tiles) seen_tiles(p, b, pc.a.x % p.c.Hkv, pc.a.y, first, last, whole, count);
          // (At most 2^20 tiles and 76 shares.)
          const uint32_t nt = static_cast<uint32_t>(last - first), n = static_cast<uint32_t>(unit_shares(p, pc.a.y));
          const int t0 = static_cast<int>(nt * static_cast<uint32_t>(pc.a.z) / n);
          const int t1 = static_cast<int>(nt * static_cast<uint32_t>(pc.a.z + 1) / n);
          pc.b = make_int4(nk, nq, first + t0, t1 - t0);
          pc.a.z |= count << 7;
          pc.a.w = LIN ? p.lin_ok[pc.a.x % p.c.Hkv] : whole;
        }
        int next = 0;
        if (lane == 0) {
          bool ok = true;
          if (rows) {
            if constexpr (!LATE)
              ok = i < 2 || mbar_wait_acq_cluster(&pc_empty[i & 1], ((i >> 1) - 1) & 1, err, piece_limit_ns(ahead[0], ahead[1]));
            ahead[0] = ahead[1], ahead[1] = pc.b.w;
            if (ok) {
              for (uint32_t r = 0; r < 2; ++r) {
                st_cluster_v4(mapa_shared(&pc_slot[2 * (i & 1)], r), pc.a);
                st_cluster_v4(mapa_shared(&pc_slot[2 * (i & 1) + 1], r), pc.b);
              }
              for (uint32_t r = 0; r < 2; ++r) mbar_arrive_cluster(mapa_shared(&pc_full[i & 1], r));
              if (LATE && i >= 1 && pc.a.x >= 0)
                ok = mbar_wait_acq_cluster(&pc_empty[(i + 1) & 1], ((i - 1) >> 1) & 1, err, piece_limit_ns(ahead[0], ahead[1]));
            }
          }
          next = ok && pc.a.x >= 0 ? pairs + atomicAdd(p.queue, 1) : -1;
        }
        k = __shfl_sync(0xffffffffu, next, 0);
        if (k < 0) break;
        if (rows) ++i;
      }
    } else if (warp == 0) {
      if (lane == 0) {
        // ---------------- TMA: Q, then this CTA's 128 keys of every tile
        const uint32_t q_full0 = mapa_shared(q_full, 0);
        const uint32_t k_full0 = mapa_shared(k_full, 0);
        int gk = 0, gq = 0;
        Piece pc;
        for (int i = 0;; release_piece(i), ++i) {
          const bool more = take_piece(i, pc);
          // Handed on within the CTA: softmax warps that released slots of the pair
          // themselves would wait for their stores of O each time.
          const int s = i % kHanded;
          if (!mbar_wait(&h_empty[s], ((i / kHanded) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) break;
          sm_piece[2 * s] = more ? pc.a : make_int4(-1, 0, 0, 0);
          sm_piece[2 * s + 1] = pc.b;
          mbar_arrive_local(&h_full[s]);
          if (!more) break;
          const int nT = pc.b.w;
          if (nT == 0) continue;
          const int b = pc.a.x / p.c.Hkv, hk = pc.a.x % p.c.Hkv;
          if (gq > 0 && !mbar_wait(q_empty, (gq - 1) & 1, err, ERR_ATTN_TIMEOUT)) break;
          ++gq;
          if (leader) mbar_arrive_expect_tx(q_full, 2 * (p.rows_cta * DH * 2 + (LIN ? kLinBytes : 0)));
          if constexpr (LIN) tma_load_3d_lin(smem + C::OFF_LIN, &tmL, q_full0, hk);
#pragma unroll
          for (int a = 0; a < C::NA; ++a)
            tma_load_4d_pair(sQ + a * C::ATOM, &tmQ, q_full0, a * 64, hk * p.c.G,
                             (pc.a.y * 2 + rank) * p.tok_cta, b);
          bool ok = true;
          for (int j = 0; j < nT; ++j, ++gk) {
            const int st = gk % KK;
            if (!mbar_wait(&k_empty[st], ((gk / KK) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) {
              ok = false;
              break;
            }
            if (leader) mbar_arrive_expect_tx(&k_full[st], 2 * C::K_BYTES);
            uint8_t* dst = sK + st * C::K_BYTES;
#pragma unroll
            for (int a = 0; a < C::NA; ++a)
              tma_load_4d_pair(dst + a * C::ATOM, &tmK, k_full0 + st * 8, a * 64,
                               tile_at<ROT>(p, pc, j) * KT + rank * 128, hk, b);
          }
          if (!ok) break;
        }
        // No copy into or read of this CTA's shared memory may be left when it
        // exits: wait (bounded) until the MMAs released the last stages.
        const uint64_t t0 = global_timer_ns();
        for (int j = (gk > KK ? gk - KK : 0); j < gk; ++j) {
          while (!mbar_try_wait(&k_empty[j % KK], (j / KK) & 1) &&
                 global_timer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    } else if (warp == 2) {
      if (lane == 0) {
        // ---------------- TMA: this CTA's columns of V, 256 keys a tile.  A tile
        // that ends behind the keys completes on this CTA's own barrier: the
        // softmax warps zero those rows before they release the tile's P.
        const uint32_t v_full0 = mapa_shared(v_full, 0);
        const uint32_t v_zero0 = mapa_shared(v_zero, rank);
        int gv = 0;
        Piece pc;
        for (int i = 0; take_piece(i, pc); release_piece(i), ++i) {
          const int b = pc.a.x / p.c.Hkv, hk = pc.a.x % p.c.Hkv;
          bool ok = true;
          for (int j = 0; j < pc.b.w; ++j, ++gv) {
            const int st = gv % KS;
            const int key0 = tile_at<ROT>(p, pc, j) * KT;
            if (!mbar_wait(&v_empty[st], ((gv / KS) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) {
              ok = false;
              break;
            }
            const bool zero = zero_tile(p, key0, pc.b.x);
            if (zero) mbar_arrive_expect_tx(&v_zero[st], C::V_BYTES);
            if (leader && !zero) mbar_arrive_expect_tx(&v_full[st], 2 * C::V_BYTES);
            else mbar_arrive_remote(v_full0 + st * 8);
            tma_load_4d_pair(sV + st * C::V_BYTES, &tmV, (zero ? v_zero0 : v_full0) + st * 8, rank * C::VR, key0, hk, b);
          }
          if (!ok) break;
        }
        const uint64_t t0 = global_timer_ns();
        for (int j = (gv > KS ? gv - KS : 0); j < gv; ++j) {
          while (!mbar_try_wait(&v_empty[j % KS], (j / KS) & 1) &&
                 global_timer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    } else if (warp == 1 && lane == 0 && leader) {
      // ---------------- MMA issuer, in program order: S_0, then per tile j
      // S_{j+1} (once S_j was read), P_j V_j (once P_j was written).
      constexpr uint32_t IDESC_S = idesc_of<BF16>(2 * QT, KT, false);
      constexpr uint32_t IDESC_O = idesc_of<BF16>(2 * QT, DH, true);
      const uint64_t dq = umma_desc_kmajor(smem_u32(sQ), 128);
      const uint64_t dk = umma_desc_kmajor(smem_u32(sK), 128);
      const uint64_t dv = desc_mn(smem_u32(sV), C::V_ROW);
      const uint64_t dlq = desc_lin(smem_u32(smem + C::OFF_LIN));
      auto issue_s = [&](int t, int side) {
        const uint64_t b = dk + static_cast<uint64_t>(((t % KK) * C::K_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t o = ((kk / 4) * C::ATOM + (kk % 4) * 32) >> 4;
          umma_bf16_pair(tmem + COL_S, dq + o, b + o, IDESC_S, kk != 0);
        }
        if constexpr (LIN) {
          if (side != 0) umma_bf16_pair(tmem + COL_S, dlq, dlq + ((side > 0 ? 1 : 2) * kLinBytes >> 4), IDESC_S, 1);
        }
        umma_commit_pair_mc(s_full, 0x3);
        umma_commit_pair_mc(&k_empty[t % KK], 0x3);
      };
      int g = 0, gq = 0;
      bool ok = true;
      Piece pc;
      for (int i = 0; ok && take_piece(i, pc); ++i) {
        const int nT = pc.b.w;
        mbar_arrive_remote(pc_empty0 + (i & 1) * 8);  // this CTA's own slot: CTA scope
        if (nT == 0) continue;
        if (!mbar_wait(q_full, gq & 1, err, ERR_ATTN_TIMEOUT) ||
            !mbar_wait(&k_full[g % KK], (g / KK) & 1, err, ERR_ATTN_TIMEOUT) ||
            (g > 0 && !mbar_wait(s_free, (g - 1) & 1, err, ERR_ATTN_TIMEOUT)))
          break;
        ++gq;
        tc_fence_after();
        const int2 lin = LIN ? lin_tiles(p, pc) : int2{};
        issue_s(g, LIN ? tile_side(lin, tile_at<ROT>(p, pc, 0)) : 0);
        if (nT == 1) umma_commit_pair_mc(q_empty, 0x3);
        for (int j = 0; j < nT; ++j) {
          const int t = g + j;
          if (j + 1 < nT) {
            if (!mbar_wait(s_free, t & 1, err, ERR_ATTN_TIMEOUT) ||
                !mbar_wait(&k_full[(t + 1) % KK], ((t + 1) / KK) & 1, err, ERR_ATTN_TIMEOUT)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(t + 1, LIN ? tile_side(lin, tile_at<ROT>(p, pc, j + 1)) : 0);
            if (j + 2 == nT) umma_commit_pair_mc(q_empty, 0x3);
          }
          // The acquire at cluster scope pairs with the softmax warps' release after
          // they zeroed rows of V, in a piece's last tile at most (if not rotated).
          const bool plain = ROT ? !zero_tile(p, tile_at<ROT>(p, pc, j) * KT, pc.b.x) : j + 1 < nT;
          if (!(plain ? mbar_wait(p_full_a, t & 1, err, ERR_ATTN_TIMEOUT)
                      : mbar_wait_acq_cluster(p_full_a, t & 1, err)) ||
              !mbar_wait(&v_full[t % KS], (t / KS) & 1, err, ERR_ATTN_TIMEOUT)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b = dv + static_cast<uint64_t>(((t % KS) * C::V_BYTES) >> 4);
          auto issue_pv = [&](int kk) {  // keys [16 kk, 16 kk + 16)
            umma_pair_tmem_a(tmem + COL_O, tmem + COL_P + kk * 8, b + ((kk * 16 * C::V_ROW) >> 4), IDESC_O,
                             (j | kk) != 0);
          };
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) issue_pv(kk);
#pragma unroll
          for (int kk = 8; kk < 12; ++kk) issue_pv(kk);
          if (!mbar_wait(p_full_b, t & 1, err, ERR_ATTN_TIMEOUT)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk) issue_pv(kk);
#pragma unroll
          for (int kk = 12; kk < 16; ++kk) issue_pv(kk);
          umma_commit_pair_mc(o_done, 0x3);
          umma_commit_pair_mc(&v_empty[t % KS], 0x3);
        }
        g += nT;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // ---------------- softmax: warp 4 + 4 h + q serves rows 32 q + 16 h + [0, 16)
    const int hk16 = lane >> 4;  // which 128 keys of a tile, and which half of O's columns
    const int rb = (warp & 3) * 32 + ((warp - 4) >> 2) * 16;
    const int r = rb + (lane & 15);
    const uint32_t lane_off = static_cast<uint32_t>(rb) << 16;
    const uint32_t s_addr = tmem + COL_S + lane_off;
    const uint32_t p_addr = tmem + COL_P + lane_off;
    const uint32_t o_addr = tmem + COL_O + lane_off;
    const uint32_t s_free0 = mapa_shared(s_free, 0);
    const uint32_t p_full_a0 = mapa_shared(p_full_a, 0);
    const uint32_t p_full_b0 = mapa_shared(p_full_b, 0);
    const float scale2 = p.c.scale * kLog2e;
    int g = 0;
    uint32_t gz = 0;
    for (int i = 0;; ++i) {
      if (!warp_wait(&h_full[i % kHanded], (i / kHanded) & 1, err)) break;
      __syncwarp();
      const int4 pa = ld_shared_v4(sm_piece + 2 * (i % kHanded)), pb = ld_shared_v4(sm_piece + 2 * (i % kHanded) + 1);
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&h_empty[i % kHanded]);
      if (pa.x < 0) break;
      const int b = pa.x / p.c.Hkv, kvh = pa.x % p.c.Hkv;
      const int k_len = pb.x, q_len = pb.y, nT = pb.w;
      // This thread's row.
      const int tok = (pa.y * 2 + rank) * p.tok_cta + r / p.c.G;
      const int head = kvh * p.c.G + r % p.c.G;
      const bool valid = r < p.rows_cta && tok < q_len;
      const bool active = __any_sync(0xffffffffu, valid);  // a row of this warp counts
      int qp = k_len - q_len + tok, qd = 0;
      if ((F & F_META) && valid) {
        if (p.c.q_pos) qp = p.c.q_pos[b * p.c.qm_b + tok];
        if (p.c.q_doc) qd = p.c.q_doc[b * p.c.qm_b + tok];
      }
      const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
      // Keys at or behind klim are not seen (positions that are indexes).
      int klim = k_len;
      if (p.c.causal && !((F & F_META) && p.c.k_pos)) klim = min(klim, max(qp + 1, prefix));
      const float slope2 = (F & F_BIAS) && valid ? p.c.slopes[head] * kLog2e : 0.0f;
      const int64_t meta = (F & F_META) ? b * p.c.km_b + kvh * p.c.km_h : 0;
      const bool ordered = (F & F_META) && p.c.causal && p.c.k_pos;
      const KeyTile* tiles =
          p.key_tiles + (static_cast<int64_t>(b) * p.meta_heads + (p.meta_heads > 1 ? kvh : 0)) * p.tiles;
      const int plim = max(qp + 1, prefix);  // positions below it are seen
      // A tile's notes, and its keys' positions and documents, are brought to L1
      // one tile ahead (held in registers they were spilled, and waited for).
      auto fetch_meta = [&](int tile) {
        if (lane == 0) prefetch_l1(tiles + tile);
        const int j = min(tile * KT + 32 * lane, k_len - 1);
        if (lane < 8 && p.c.k_doc) prefetch_l1(p.c.k_doc + meta + j);
        if (lane < 8 && p.c.k_pos) prefetch_l1(p.c.k_pos + meta + j);
      };
      if ((F & F_META) && p.key_tiles && nT > 0 && active) fetch_meta(pb.z);
      const int2 lin = LIN ? lin_tiles(p, Piece{pa, pb}) : int2{};
      float m = -INFINITY, l = 0.0f;  // l: this thread's half of the row sum
      bool ok = true;
      // Releases the first half of a tile's P (and its V).  In a tile that ends
      // behind the keys the CTA's 256 softmax threads zero those rows of V
      // first: P is 0 there, but 0 times NaN is not.
      auto release_p = [&](int tile, int t) -> bool {
        const int key0 = tile * KT;
        if (!zero_tile(p, key0, k_len)) {
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(p_full_a0);
          __syncwarp();
          return true;
        }
        // A stage's barrier is armed again only after its tile's P.V, so each
        // warp sees every phase; gz holds the stages' phase parities.
        const int st = t % KS;
        if (!warp_wait(&v_zero[st], (gz >> st) & 1, err)) return false;
        gz ^= 1 << st;
        const int n0 = max(k_len - key0, 0);
        uint4* z = reinterpret_cast<uint4*>(sV + st * C::V_BYTES + n0 * C::V_ROW);
        const int n = (KT - n0) * (C::V_ROW / 16);
#pragma unroll 1
        for (int e = static_cast<int>(threadIdx.x) - 128; e < n; e += 256) z[e] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full_a0);
        __syncwarp();
        return true;
      };
      // Every softmax warp runs all nT iterations, also after a failed wait
      // (which only skips the work).
      for (int j = 0; j < nT; ++j) {
        const int t = g + j;
        const int tile = tile_at<ROT>(p, Piece{pa, pb}, j);
        const int key0 = tile * KT + hk16 * 128;
        // Which of the 128 keys this row sees, one bit each (while S is made),
        // if some row of the warp sees a part of the tile.
        uint32_t seen[4];
        bool masked = false, none = false;  // (none: no row of the warp sees a key of the tile)
        int d0 = qp - key0;  // distance of the first key, where positions run
        bool run = true;
        // (A stretch of tiles is known to be seen whole; only the distance bias
        // then needs the tile's notes.)
        const bool whole = static_cast<uint32_t>(tile - pa.w) < static_cast<uint32_t>(pa.z >> 7);
        if ((F & F_META) && p.key_tiles && active && j + 1 < nT) {
          const bool next_whole = static_cast<uint32_t>(tile + 1 - pa.w) < static_cast<uint32_t>(pa.z >> 7);
          if ((F & F_BIAS) || !next_whole) fetch_meta(tile + 1);
        }
        if ((F & F_META) && p.key_tiles && active && ((F & F_BIAS) || !whole)) {
          const KeyTile kt = tiles[tile];
          run = kt.run;
          if (p.c.k_pos) d0 = qp - kt.base - hk16 * 128;
          const bool doc_all = !p.c.k_doc || (kt.doc_min == qd && kt.doc_max == qd);
          const bool pos_all = !ordered || kt.pos_max < plim;
          none = __all_sync(0xffffffffu, !valid || (p.c.k_doc && (qd < kt.doc_min || qd > kt.doc_max)) ||
                                             (ordered && kt.pos_min >= plim));
          masked = !whole && !none && __any_sync(0xffffffffu, valid && !(doc_all && pos_all));
          if (masked && kt.sorted && (run || !ordered)) {
            // The row's document is one stretch of the tile, and positions that
            // run are seen up to a limit: keys [lo, hi).
            int lo = 0, hi = min(128, k_len - key0);
            if (p.c.k_doc && kt.cut >= 0) {
              const int cut = kt.cut - hk16 * 128;
              if (qd != kt.doc_min) lo = qd == kt.doc_max ? cut : 128;
              else if (qd != kt.doc_max) hi = min(hi, cut);
            } else if (p.c.k_doc) {
              const int end = hi;
              lo = first_doc(p.c.k_doc + meta + key0, 0, end, qd);
              hi = qd == 0x7fffffff ? end : first_doc(p.c.k_doc + meta + key0, lo, end, qd + 1);
            }
            if (ordered) hi = min(hi, plim - kt.base - hk16 * 128);
#pragma unroll
            for (int w = 0; w < 4; ++w) seen[w] = low_bits(hi - 32 * w) & ~low_bits(lo - 32 * w);
          } else if (masked) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t bits = 0;
#pragma unroll 2
              for (int c = 0; c < 32; c += 4) {
                const int k0 = key0 + 32 * w + c;
                uint32_t v = 15;
                if (p.c.k_doc) {
                  const int4 d = ld_meta4(p.c.k_doc + meta, k0, k_len, p.meta_vec);
                  v = (d.x == qd) | (d.y == qd) << 1 | (d.z == qd) << 2 | (d.w == qd) << 3;
                }
                if (ordered) {
                  const int4 x = ld_meta4(p.c.k_pos + meta, k0, k_len, p.meta_vec);
                  v &= (x.x < plim) | (x.y < plim) << 1 | (x.z < plim) << 2 | (x.w < plim) << 3;
                }
                bits |= v << c;
              }
              seen[w] = bits;
            }
          }
        }
        if (ok) ok = warp_wait(s_full, t & 1, err);
        if (!ok) continue;
        if (!active || ((F & F_META) && none)) {  // only keep the barriers' counts
          if (lane == 0) mbar_arrive_remote(s_free0);
          if (j > 0) ok = warp_wait(o_done, (t - 1) & 1, err);
          if ((F & F_META) && ok && active) {
            const uint32_t zero[16] = {};
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_st16x<64>(p_addr + 16 * c, zero);
            tmem_wait_st();
            tc_fence_before();
          }
          if (ok) ok = release_p(tile, t);
          if (ok && lane == 0) mbar_arrive_remote(p_full_b0);
          continue;
        }
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32x<128>(s_addr + c * 32, s + c * 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(s_free0);
        float sl2 = scale2, off = 0.0f;  // score = s * sl2 + off (log2)
        if constexpr ((F & F_CAP) != 0) {
          {
            // What lies behind the keys must not choose the branch.
            if (key0 + 128 > k_len) {
#pragma unroll
              for (int c = 0; c < 128; ++c)
                if (c >= k_len - key0) s[c] = 0.0f;
            }
            float big = 0.0f;
#pragma unroll
            for (int c = 0; c < 128; c += 2) big = max3(big, fabsf(s[c]), fabsf(s[c + 1]));
            if (__all_sync(0xffffffffu, !valid || big <= p.cap_small)) {
#pragma unroll
              for (int c = 0; c < 128; c += 2) cap2<3>(s[c], s[c + 1], p.cap_c3);
            } else if constexpr ((F & F_WIDE) != 0) {
              if (__all_sync(0xffffffffu, !valid || big * p.cap.inv <= 1.0f)) cap_within<128>(s, p.cap);
              else cap_any<128>(s, p.cap);
            } else if (__all_sync(0xffffffffu, !valid || big <= p.cap_mid)) {
#pragma unroll
              for (int c = 0; c < 128; c += 2) cap2<7>(s[c], s[c + 1], p.cap_c7);
            } else {
              cap_low<128>(s, p.cap);
            }
            sl2 = 1.0f;
          }
        }
        const int side = LIN ? tile_side(lin, tile) : 0;
        if constexpr (LIN) {
          if (side != 0) off = (side > 0 ? -slope2 : slope2) * static_cast<float>(qp - tile * KT);
        }
        if constexpr ((F & F_BIAS) != 0) {
          if (side == 0) {
            const float d = static_cast<float>(d0);
            if (run && __all_sync(0xffffffffu, d0 >= 127 || d0 <= 0)) {
              // The row lies on one side of all its keys: the bias is linear in c.
              const float bs = d0 > 0 ? slope2 : -slope2, as = -bs * d;
#pragma unroll
              for (int c = 0; c < 128; c += 2) bias2(s[c], s[c + 1], sl2, static_cast<float>(c), bs, as);
            } else if (!(F & F_META) || run) {
#pragma unroll
              for (int c = 0; c < 128; ++c) s[c] = fmaf(s[c], sl2, -slope2 * fabsf(d - static_cast<float>(c)));
            } else {
#pragma unroll
              for (int c = 0; c < 128; c += 4) {
                const int4 kp = ld_meta4(p.c.k_pos + meta, key0 + c, k_len, p.meta_vec);
                s[c] = fmaf(s[c], sl2, -slope2 * fabsf(static_cast<float>(qp - kp.x)));
                s[c + 1] = fmaf(s[c + 1], sl2, -slope2 * fabsf(static_cast<float>(qp - kp.y)));
                s[c + 2] = fmaf(s[c + 2], sl2, -slope2 * fabsf(static_cast<float>(qp - kp.z)));
                s[c + 3] = fmaf(s[c + 3], sl2, -slope2 * fabsf(static_cast<float>(qp - kp.w)));
              }
            }
            sl2 = 1.0f;
          }
        }
        if constexpr ((F & F_META) != 0) {
          if (masked) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!((seen[c >> 5] >> (c & 31)) & 1)) s[c] = -INFINITY;
          }
        }
        if (key0 + 128 > klim) {
          const int lim = klim - key0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= lim) s[c] = -INFINITY;
        }
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = max3(s[e], s[e + 8], s[e + 16]);
#pragma unroll
        for (int c = 24; c < 120; c += 16) {
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = max3(mx8[e], s[c + e], s[c + 8 + e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(mx8[e], s[120 + e]);
        const float mx = fmaxf(max3(mx8[0], mx8[1], mx8[2]),
                               fmaxf(max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const float m_tile = fmaf(fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)), sl2, off);
        const bool grow = m_tile > m + kRescaleThreshold;
        const bool any_grow = __any_sync(0xffffffffu, grow);
        const float m_new = grow ? m_tile : m;
        const float alpha = grow ? fast_exp2(m - m_new) : 1.0f;
        // A row that has seen no key keeps m = -inf; its weights are exp2(-inf).
        const float negm = m_new == -INFINITY ? 0.0f : off - m_new;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        auto exp_chunk = [&](int c, uint32_t* pk) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x = s[c * 32 + 2 * e], y = s[c * 32 + 2 * e + 1];
            ffma2(x, y, sl2, negm);
            x = fast_exp2(x);
            y = fast_exp2(y);
            fadd2(acc[2 * (e & 3)], acc[2 * (e & 3) + 1], x, y);
            pk[e] = pack2<BF16>(x, y);
          }
        };
        uint32_t pk0[16], pk1[16];
        exp_chunk(0, pk0);
        exp_chunk(1, pk1);
        m = m_new;
        if (j > 0) {
          ok = warp_wait(o_done, (t - 1) & 1, err);
          if (!ok) continue;
          tc_fence_after();
          if (any_grow) {
#pragma unroll 1
            for (int c = 0; c < C::OH / 16; ++c) {
              float o[16];
              tmem_ld16x<C::OH>(o_addr + c * 16, o);
              tmem_wait_ld();
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * alpha);
              tmem_st16x<C::OH>(o_addr + c * 16, u);
            }
          }
        }
        tmem_st16x<64>(p_addr, pk0);
        tmem_st16x<64>(p_addr + 16, pk1);
        tmem_wait_st();
        tc_fence_before();
        ok = release_p(tile, t);
        if (!ok) continue;
        exp_chunk(2, pk0);
        tmem_st16x<64>(p_addr + 32, pk0);
        exp_chunk(3, pk1);
        tmem_st16x<64>(p_addr + 48, pk1);
        l = l * alpha + (((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(p_full_b0);
      }
      // A thread's row leaves by way of shared memory, 64 bytes of either half of
      // its columns at a time, so that four lanes write 64 consecutive bytes
      // (lanes that wrote rows of their own took 4000 clocks a piece, this 1000).
      const float lo = __shfl_xor_sync(0xffffffffu, l, 16);
      l = hk16 == 0 ? l + lo : lo + l;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int shares = unit_shares(p, pa.y);
      const bool split = shares > 1;
      const int64_t piece =
          (p.tail_split ? static_cast<int64_t>(pa.x) : static_cast<int64_t>(pa.x) * p.units + pa.y) * shares + (pa.z & 127);
      const int64_t prow = piece * p.part_rows + rank * p.rows_cta + r;
      char* row = split ? reinterpret_cast<char*>(p.part_o + prow * DH)
                        : reinterpret_cast<char*>(static_cast<uint16_t*>(p.c.o) + b * p.c.os.b + tok * p.c.os.l + head * p.c.os.h);
      if (!valid) row = nullptr;
      char* out[4];  // of rows lane / 8 + 4 k
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[k] = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), 4 * k + (lane >> 3)));
      uint8_t* stage = smem + C::OFF_OUT + (warp - 4) * kOutBytes;
      uint4* mine = reinterpret_cast<uint4*>(stage + (lane & 15) * kOutRow + hk16 * 64);
      const int half = (lane >> 2) & 1, unit = lane & 3;  // what this lane writes of its four rows
      const uint4* theirs = reinterpret_cast<const uint4*>(stage + (lane >> 3) * kOutRow + half * 64 + unit * 16);
      const int width = split ? 2 * C::OH * 4 : p.c.dh * 2;  // bytes of a row (heads may be narrower than DH)
      auto put = [&](const uint32_t* w, int c) {  // 64 bytes c of this thread's half of its row
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        __syncwarp();
        const int at = half * (split ? C::OH * 4 : C::OH * 2) + c * 64 + unit * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (out[k] && at < width) *reinterpret_cast<uint4*>(out[k] + at) = theirs[k * (4 * kOutRow / 16)];
        __syncwarp();
      };
      // O is read before this thread writes any P of the next piece, whose
      // first P.V overwrites it.
      if (ok && nT > 0) {
        ok = warp_wait(o_done, (g + nT - 1) & 1, err);
        if (ok) tc_fence_after();
      }
      g += nT;
      if (!active || !ok) continue;
      float o[C::OH];
      if (nT > 0) {
#pragma unroll
        for (int c = 0; c < C::OH / 32; ++c) tmem_ld32x<C::OH>(o_addr + c * 32, o + c * 32);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < C::OH; ++e) o[e] = 0.0f;
      }
      uint32_t w[C::OH];
      if (split) {
#pragma unroll
        for (int e = 0; e < C::OH; ++e) w[e] = __float_as_uint(o[e]);
#pragma unroll
        for (int c = 0; c < C::OH / 16; ++c) put(w + 16 * c, c);
      } else {
#pragma unroll
        for (int e = 0; e < C::OH / 2; ++e) w[e] = pack2<BF16>(o[2 * e] * inv, o[2 * e + 1] * inv);
#pragma unroll
        for (int c = 0; c < C::OH / 32; ++c) put(w + 16 * c, c);
      }
      if (valid && hk16 == 0) {
        if (split) {
          p.part_ml[prow] = make_float2(m, l);
        } else if (p.c.lse) {
          p.c.lse[(static_cast<int64_t>(b) * p.c.Hq + head) * p.c.Lq + tok] =
              l == 0.0f ? -INFINITY : (m + fast_log2(l)) * kLn2;  // (NaN stays NaN)
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA leaves (nor frees the pair's TMEM) before both are done.
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
  if (leader && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.queue + 1, 1) == static_cast<int>(gridDim.x >> 1) - 1) {
      atomicExch(p.queue, 0);
      atomicExch(p.queue + 1, 0);
    }
  }
}

template <int DH, bool BF16, int F>
cudaError_t launch_one(const CUtensorMap* maps, const TcParams& p, int pairs, cudaStream_t st) {
  static uint64_t set_up = 0;
  // More than half an SM's shared memory: one CTA per SM, so its 512 TMEM
  // columns are free.
  using C = Cfg<DH, F == F_BIAS>;
  const size_t smem = C::SMEM > 120 * 1024 ? C::SMEM : 120 * 1024;
  static_assert(C::SMEM <= 232448, "over the per-block limit");
  cudaError_t e = once_per_device(&set_up, [&](int) {
    // The register split must fit the launch allocation, else the growing
    // warpgroups would wait for registers forever.
    cudaFuncAttributes fa;
    cudaError_t r = cudaFuncGetAttributes(&fa, cache_attn_kernel<DH, BF16, F>);
    if (r != cudaSuccess) return r;
    if (fa.numRegs * kThreads < kRegsNeeded || fa.numRegs < kRegsLow || fa.numRegs > kRegsHigh)
      return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(cache_attn_kernel<DH, BF16, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cache_attn_kernel<DH, BF16, F>, maps[0], maps[1], maps[2], maps[3], p);
}

template <int DH, bool BF16>
cudaError_t launch_features(const CUtensorMap* maps, const TcParams& p, int f, int pairs, cudaStream_t st) {
  switch (f) {
    case 0: return launch_one<DH, BF16, 0>(maps, p, pairs, st);
    case 1: return launch_one<DH, BF16, 1>(maps, p, pairs, st);
    case 2: return launch_one<DH, BF16, 2>(maps, p, pairs, st);
    case 3: return launch_one<DH, BF16, 3>(maps, p, pairs, st);
    case 4: return launch_one<DH, BF16, 4>(maps, p, pairs, st);
    case 5: return launch_one<DH, BF16, 5>(maps, p, pairs, st);
    case 6: return launch_one<DH, BF16, 6>(maps, p, pairs, st);
    case 7: return launch_one<DH, BF16, 7>(maps, p, pairs, st);
    case 9: return launch_one<DH, BF16, 9>(maps, p, pairs, st);
    case 11: return launch_one<DH, BF16, 11>(maps, p, pairs, st);
    case 13: return launch_one<DH, BF16, 13>(maps, p, pairs, st);
    case 15: return launch_one<DH, BF16, 15>(maps, p, pairs, st);
    default: return cudaErrorInvalidValue;
  }
}

// The description of a problem for these kernels, its maps (q, k and, with
// `values`, v), and the kernel that fills key_tiles and row_units where there
// are positions or documents.
TcParams plan(const CacheParams& c, char* scratch);
bool encode_maps(CUtensorMap* maps, const CacheParams& c, const TcParams& p, bool bf16, bool values);
cudaError_t launch_tiles(const TcParams& p, cudaStream_t st);
// And the one that fills unit_order from them.
cudaError_t launch_order(const TcParams& p, cudaStream_t st);

extern template cudaError_t launch_features<64, true>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);
extern template cudaError_t launch_features<64, false>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);
extern template cudaError_t launch_features<128, true>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);
extern template cudaError_t launch_features<128, false>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);

}  // namespace cattn

}  // namespace psv

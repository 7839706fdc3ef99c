// The attention mass on the tensor cores (psv_cache_mass, many rows):
//   mass[j] += sum over rows i and heads of the group of exp(s_ij - lse_i)
//
// The products are taken transposed, S^T = K Q^T, so that a key is a row of the
// accumulator: a thread adds up its key's weights in registers, and no sum
// crosses threads before the end.  CTA pairs with 2-SM tcgen05 MMAs: a piece is
// a tile of 256 keys (128 per CTA) of one (sequence, kv head), which stays in
// shared memory while the row tiles (256 rows: each CTA holds 128) stream past.
//   S^T_t = K Q_t^T   M=256, N=256, K=dh, double-buffered in TMEM
// Per score one multiply-add (scale and -lse), one exp2 and one add: the MMAs
// and the exponentials each take about 1050 clocks of a tile, and a tile takes
// 2200: each unit is half busy, as a warp's reads of TMEM, its waits and its
// weights follow one another and four warps a scheduler do not fill the gaps.
// (Measured no faster: -lse added by the products, the two halves of the warps
// on tiles of their own, the row notes read a tile ahead; slower: eight warps,
// S^T held double in registers.)  Four sequences of 1560 rows x 7800 keys, 12
// heads of 128: 162 us (925 TFLOP/s), causal 155, with a cap of 50 248 (scores of
// deviation 8: 330), with the distance bias 283.
// A row's -lse, position limit, document and slope are noted per tile in shared
// memory by a warp of their own.  Warp roles, 640 threads:
//   warp 0       TMA: the piece's K tile (2 buffers), the row tiles (4 stages);
//                hands the pieces on to the warps from 3 on
//   warp 1       TMEM allocator (both CTAs) and MMA issuer (even CTA)
//   warp 2       even CTA: takes pieces from the work queue, publishes them
//   warp 3       notes the columns of a row tile
//   warps 4..19  weights: four threads per key (lanes l and l + 16 of two warps),
//                64 rows each; with eight warps each unit stayed below 45% busy
#include "cache_attn_tc.cuh"

namespace psv {

using namespace cattn;

namespace {

constexpr int QS = 4;          // row-tile stages
constexpr int kMassThreads = 640, kWeightWarps = 16;
// Readers of a published piece: both loaders (which hand it on) and the MMA issuer.
constexpr int kMassReaders = 3;
constexpr int kHalf = 132;     // words between the halves of a column array: other banks
constexpr int kColWords = 2 * kHalf;

// Columns of a row tile: -lse (log2), -slope (log2), position, position limit, document.
enum : int { COL_NLSE, COL_NSLOPE, COL_QP, COL_PLIM, COL_DOC, COL_ARRAYS };

template <int DH>
struct MCfg {
  static constexpr int NA = DH / 64;
  static constexpr int TILE = 128 * DH * 2;  // this CTA's keys or rows of a tile
  static constexpr int ATOM = 128 * 128;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = OFF_K + 2 * TILE;
  static constexpr int OFF_COL = OFF_Q + QS * TILE;
  static constexpr int COL_BYTES = COL_ARRAYS * kColWords * 4 + 16;  // and {limit min, doc min, doc max, 0}
  static constexpr int OFF_BAR = OFF_COL + QS * ((COL_BYTES + 127) / 128 * 128);
  static constexpr int COL_STRIDE = (COL_BYTES + 127) / 128 * 128;
  static constexpr int N_BARS = 12 + 4 * QS + 2 * kHanded;
  static constexpr size_t SMEM = OFF_BAR + N_BARS * 8 + 16 + (4 + 2 * kHanded) * 16 + 2 * 128 * 4;
};

// (x0, x1) * s + (b0, b1).
__device__ __forceinline__ void ffma2v(float& x0, float& x1, float s, float b0, float b1) {
  uint64_t x, sv, bv;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(sv) : "f"(s));
  asm("mov.b64 %0, {%1, %2};" : "=l"(bv) : "f"(b0), "f"(b1));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(sv), "l"(bv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(x));
}

// mass_out = mass_in (or 0) for the keys in use.
__global__ void __launch_bounds__(256) mass_copy_kernel(const __grid_constant__ TcParams p) {
  pdl_trigger();
  const uint32_t per = (p.c.Lk + 1023) / 1024, bh = blockIdx.x / per;
  const int j = static_cast<int>(blockIdx.x - bh * per) * 1024 + threadIdx.x;
  const int64_t row = static_cast<int64_t>(bh) * p.c.Lk;
  pdl_wait();
  const int n = cache_k_len(p.c, bh / p.c.Hkv);
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = p.c.mass_in && j + 256 * i < n ? p.c.mass_in[row + j + 256 * i] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + 256 * i < n) p.c.mass_out[row + j + 256 * i] = x[i];
}

// F: F_CAP, F_BIAS (kernels of their own keep the loop within the instruction cache).
template <int DH, bool BF16, int F>
__global__ void __launch_bounds__(kMassThreads, 1)
    cache_mass_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ TcParams p) {
  using C = MCfg<DH>;
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) raise_error(p.c.err, ERR_BOUNDS);
    return;
  }
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sQ = smem + C::OFF_Q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars + 0;       // [2] even CTA: both K halves landed
  uint64_t* k_empty = bars + 2;      // [2] both: the piece's MMAs are done
  uint64_t* s_full = bars + 4;       // [2] both: S^T of a tile in TMEM
  uint64_t* s_free = bars + 6;       // [2] even: all 32 weight warps read it
  uint64_t* pc_full = bars + 8;      // [2] both
  uint64_t* pc_empty = bars + 10;    // [2] even
  uint64_t* q_full = bars + 12;      // [QS] even
  uint64_t* q_empty = q_full + QS;   // [QS] both
  uint64_t* c_full = q_empty + QS;   // [QS] own: columns noted
  uint64_t* c_empty = c_full + QS;   // [QS] own: all 16 weight warps used them
  uint64_t* h_full = c_empty + QS;       // [kHanded] own: a piece handed on to warps 3 and up
  uint64_t* h_empty = h_full + kHanded;  // [kHanded] own: all 17 took it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
  int4* pc_slot = reinterpret_cast<int4*>(smem + C::OFF_BAR + C::N_BARS * 8 + 16);  // [2][3]
  static_assert((C::N_BARS * 8) % 16 == 0, "the piece slots are 16-byte aligned");
  int4* sm_piece = pc_slot + 4;                                                      // [kHanded][2]
  float* part = reinterpret_cast<float*>(sm_piece + 2 * kHanded);                    // [2][128]

  pdl_trigger();
  const int warp = warp_id(), lane = lane_id();
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  int* err = p.c.err;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < C::N_BARS; ++i) {
      const bool free16 = i == 6 || i == 7;
      const bool readers = i == 10 || i == 11;
      const bool cols = i >= 12 + 3 * QS && i < 12 + 4 * QS, taken = i >= 12 + 4 * QS + kHanded;
      mbar_init(&bars[i], free16 ? 2 * kWeightWarps : readers ? kMassReaders : cols ? kWeightWarps : taken ? kWeightWarps + 1 : 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
  }
  // Rows of a row tile that no copy fills (128 is not a multiple of G) are zero.
  if (p.rows_cta < 128) {
    for (int a = 0; a < QS * C::NA; ++a) {
      uint4* z = reinterpret_cast<uint4*>(sQ + a * C::ATOM + p.rows_cta * 128);
      for (int e = threadIdx.x; e < (128 - p.rows_cta) * 8; e += kMassThreads) z[e] = make_uint4(0, 0, 0, 0);
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
  // {sequence * Hkv + kv head, key tile, first row tile, row tiles}, {k_len, q_len, 0, 0}
  auto take_piece = [&](int i, Piece& pc) -> bool {
    if (!mbar_wait_acq_cluster(&pc_full[i & 1], (i >> 1) & 1, err)) return false;
    pc.a = ld_shared_v4(&pc_slot[2 * (i & 1)]);
    pc.b = ld_shared_v4(&pc_slot[2 * (i & 1) + 1]);
    return pc.a.x >= 0;
  };
  auto release_piece = [&](int i) { mbar_arrive_cluster(pc_empty0 + (i & 1) * 8); };
  // By a whole warp: the piece handed on by the CTA's loader; false at the end.
  auto handed_piece = [&](int i, int4& a, int4& b) -> bool {
    const int s = i % kHanded;
    if (!warp_wait(&h_full[s], (i / kHanded) & 1, err)) return false;
    __syncwarp();
    a = ld_shared_v4(sm_piece + 2 * s);
    b = ld_shared_v4(sm_piece + 2 * s + 1);
    __syncwarp();
    if (lane == 0) mbar_arrive_local(&h_empty[s]);
    return a.x >= 0;
  };

  if (warp == 2) {
    if (leader) {
      // ---------------- work queue
      const int pairs = static_cast<int>(gridDim.x >> 1);
      int k = static_cast<int>(blockIdx.x >> 1);
      int ahead[2] = {0, 0};  // row tiles of the last two pieces published
      for (int i = 0;;) {
        Piece pc;
        bool keys = true;
        pc.a = make_int4(-1, 0, 0, 0);
        pc.b = make_int4(0, 0, 0, 0);
        if (k < p.n_pieces) {
          const int bh = k / p.tiles, tile = k % p.tiles, b = bh / p.c.Hkv, kvh = bh % p.c.Hkv;
          const int nk = cache_k_len(p.c, b), nq = cache_q_len(p.c, b);
          keys = tile * KT < nk;
          const int unit = 2 * p.tok_cta;
          const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
          int first = 0, last = (nq + unit - 1) / unit;
          if (keys && p.key_tiles) {
            const KeyTile kt =
                p.key_tiles[(static_cast<int64_t>(b) * p.meta_heads + (p.meta_heads > 1 ? kvh : 0)) * p.tiles + tile];
            int lo = 0x7fffffff, hi = 0;
            for (int t = lane; t < last; t += 32) {
              const RowUnit u = p.row_units[static_cast<int64_t>(b) * p.units + t];
              const bool docs = !p.c.k_doc || (kt.doc_min <= u.doc_max && kt.doc_max >= u.doc_min);
              if (docs && (!p.c.causal || kt.pos_min < max(u.pos_max + 1, prefix))) {
                lo = min(lo, t);
                hi = t + 1;
              }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            last = __reduce_max_sync(0xffffffffu, hi);
            first = min(lo, last);
          } else if (p.c.causal && !p.c.q_pos && prefix <= tile * KT) {
            // The first row that sees the tile's first key.
            first = min(last, max(tile * KT - (nk - nq), 0) / unit);
          }
          pc.a = make_int4(bh, tile, first, last - first);
          pc.b = make_int4(nk, nq, 0, 0);
        }
        int next = 0;
        if (lane == 0) {
          bool ok = true;
          if (keys) {
            ok = i < 2 || mbar_wait_acq_cluster(&pc_empty[i & 1], ((i >> 1) - 1) & 1, err, piece_limit_ns(ahead[0], ahead[1]));
            ahead[0] = ahead[1], ahead[1] = pc.a.w;
            if (ok) {
              for (uint32_t r = 0; r < 2; ++r) {
                st_cluster_v4(mapa_shared(&pc_slot[2 * (i & 1)], r), pc.a);
                st_cluster_v4(mapa_shared(&pc_slot[2 * (i & 1) + 1], r), pc.b);
              }
              for (uint32_t r = 0; r < 2; ++r) mbar_arrive_cluster(mapa_shared(&pc_full[i & 1], r));
            }
          }
          next = ok && pc.a.x >= 0 ? pairs + atomicAdd(p.queue, 1) : -1;
        }
        k = __shfl_sync(0xffffffffu, next, 0);
        if (k < 0) break;
        if (keys) ++i;
      }
    }
  } else if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA: the K tile of a piece, then its row tiles
      const uint32_t k_full0 = mapa_shared(k_full, 0);
      const uint32_t q_full0 = mapa_shared(q_full, 0);
      int gk = 0, g = 0;
      Piece pc;
      for (int i = 0;; release_piece(i), ++i) {
        const bool more = take_piece(i, pc);
        const int s = i % kHanded;
        if (!mbar_wait(&h_empty[s], ((i / kHanded) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) break;
        sm_piece[2 * s] = more ? pc.a : make_int4(-1, 0, 0, 0);
        sm_piece[2 * s + 1] = pc.b;
        mbar_arrive_local(&h_full[s]);
        if (!more) break;
        const int nT = pc.a.w;
        if (nT == 0) continue;
        const int b = pc.a.x / p.c.Hkv, kvh = pc.a.x % p.c.Hkv;
        const int kb = gk & 1;
        if (!mbar_wait(&k_empty[kb], ((gk >> 1) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) break;
        if (leader) mbar_arrive_expect_tx(&k_full[kb], 2 * C::TILE);
#pragma unroll
        for (int a = 0; a < C::NA; ++a)
          tma_load_4d_pair(sK + kb * C::TILE + a * C::ATOM, &tmK, k_full0 + kb * 8, a * 64, pc.a.y * KT + rank * 128,
                           kvh, b);
        ++gk;
        bool ok = true;
        for (int j = 0; j < nT; ++j, ++g) {
          const int st = g % QS;
          if (!mbar_wait(&q_empty[st], ((g / QS) & 1) ^ 1, err, ERR_ATTN_TIMEOUT)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&q_full[st], 2 * p.rows_cta * DH * 2);
#pragma unroll
          for (int a = 0; a < C::NA; ++a)
            tma_load_4d_pair(sQ + st * C::TILE + a * C::ATOM, &tmQ, q_full0 + st * 8, a * 64, kvh * p.c.G,
                             ((pc.a.z + j) * 2 + rank) * p.tok_cta, b);
        }
        if (!ok) break;
      }
      // No copy into or read of this CTA's shared memory may be left when it
      // exits: wait (bounded) until the MMAs released the last stages.
      const uint64_t t0 = global_timer_ns();
      for (int j = (g > QS ? g - QS : 0); j < g; ++j) {
        while (!mbar_try_wait(&q_empty[j % QS], (j / QS) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
      for (int j = (gk > 2 ? gk - 2 : 0); j < gk; ++j) {
        while (!mbar_try_wait(&k_empty[j & 1], (j >> 1) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- MMA issuer
      constexpr uint32_t IDESC = idesc_of<BF16>(256, 256, false);
      const uint64_t dk = umma_desc_kmajor(smem_u32(sK), 128);
      const uint64_t dq = umma_desc_kmajor(smem_u32(sQ), 128);
      int gk = 0, g = 0;
      bool ok = true;
      Piece pc;
      for (int i = 0; ok && take_piece(i, pc); ++i) {
        const int nT = pc.a.w;
        mbar_arrive_remote(pc_empty0 + (i & 1) * 8);  // this CTA's own slot: CTA scope
        if (nT == 0) continue;
        const int kb = gk & 1;
        if (!mbar_wait(&k_full[kb], (gk >> 1) & 1, err, ERR_ATTN_TIMEOUT)) break;
        const uint64_t a = dk + static_cast<uint64_t>((kb * C::TILE) >> 4);
        for (int j = 0; j < nT; ++j, ++g) {
          const int st = g % QS, sb = g & 1;
          if (!mbar_wait(&q_full[st], (g / QS) & 1, err, ERR_ATTN_TIMEOUT) ||
              (g >= 2 && !mbar_wait(&s_free[sb], ((g >> 1) - 1) & 1, err, ERR_ATTN_TIMEOUT))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b = dq + static_cast<uint64_t>((st * C::TILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t o = ((kk / 4) * C::ATOM + (kk % 4) * 32) >> 4;
            umma_bf16_pair(tmem + sb * 256, a + o, b + o, IDESC, kk != 0);
          }
          umma_commit_pair_mc(&s_full[sb], 0x3);
          umma_commit_pair_mc(&q_empty[st], 0x3);
        }
        if (!ok) break;
        umma_commit_pair_mc(&k_empty[kb], 0x3);
        ++gk;
      }
    }
  } else if (warp == 3) {
    // ---------------- columns of the row tiles.  A
    // lane notes columns 32 x + lane of both halves; their tokens and heads
    // within a tile are the same for every tile.
    int dtok[4], dhead[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = x * 32 + lane;
      dtok[x] = r < p.rows_cta ? r / p.c.G : 0x40000000;  // never below q_len
      dhead[x] = r % p.c.G;
    }
    const bool given = p.c.q_pos || p.c.q_doc || p.c.slopes;
    int g = 0;
    Piece pc;
    for (int i = 0;; ++i) {
      if (!handed_piece(i, pc.a, pc.b)) break;
      const int b = pc.a.x / p.c.Hkv, kvh = pc.a.x % p.c.Hkv, nk = pc.b.x, nq = pc.b.y;
      const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
      const float* lse = p.c.lse + (static_cast<int64_t>(b) * p.c.Hq + kvh * p.c.G) * p.c.Lq;
      bool ok = true;
      for (int j = 0; j < pc.a.w; ++j, ++g) {
        const int st = g % QS;
        // The reads of lse are on their way while the stage is waited for.
        const int tok0 = (pc.a.z + j) * 2 * p.tok_cta;
        float nl[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int tok = tok0 + (x >> 2) * p.tok_cta + dtok[x & 3];
          nl[x] = tok < nq ? __ldg(lse + static_cast<int64_t>(dhead[x & 3]) * p.c.Lq + tok) : -INFINITY;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&c_empty[st], ((g / QS) & 1) ^ 1, err, ERR_ATTN_TIMEOUT))) {
          ok = false;
          break;
        }
        float* col = reinterpret_cast<float*>(smem + C::OFF_COL + st * C::COL_STRIDE);
        int* icol = reinterpret_cast<int*>(col);
        int pl_min = 0x7fffffff, d_min = 0x7fffffff, d_max = -0x7fffffff - 1;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int tok = tok0 + (x >> 2) * p.tok_cta + dtok[x & 3];
          const int at = (x >> 2) * kHalf + (x & 3) * 32 + lane;
          const bool valid = tok < nq;
          int qp = nk - nq + tok, qd = 0;
          float ns = 0.0f;
          if (given && valid) {
            if (p.c.q_pos) qp = p.c.q_pos[b * p.c.qm_b + tok];
            if (p.c.q_doc) qd = p.c.q_doc[b * p.c.qm_b + tok];
            if (p.c.slopes) ns = -p.c.slopes[kvh * p.c.G + dhead[x & 3]] * kLog2e;
          }
          int pl = p.c.causal ? max(qp + 1, prefix) : 0x7fffffff;
          if (valid) {
            pl_min = min(pl_min, pl);
            d_min = min(d_min, qd), d_max = max(d_max, qd);
          } else {
            pl = -0x7fffffff - 1;
            // An unused row may hold NaN: its columns are masked one by one.
            if (tok < p.c.Lq) pl_min = pl;
          }
          col[COL_NLSE * kColWords + at] = nl[x] != -INFINITY ? -nl[x] * kLog2e : -INFINITY;
          icol[COL_PLIM * kColWords + at] = pl;
          if (p.c.slopes) {
            col[COL_NSLOPE * kColWords + at] = ns;
            icol[COL_QP * kColWords + at] = qp;
          }
          if (p.c.q_doc) icol[COL_DOC * kColWords + at] = qd;
        }
        pl_min = __reduce_min_sync(0xffffffffu, pl_min);
        if (p.c.q_doc) {
          d_min = __reduce_min_sync(0xffffffffu, d_min);
          d_max = __reduce_max_sync(0xffffffffu, d_max);
        }
        if (lane == 0) {
          int* stat = icol + COL_ARRAYS * kColWords;
          stat[0] = pl_min, stat[1] = d_min, stat[2] = d_max;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(&c_full[st], rank));
        __syncwarp();
      }
      if (!ok) break;
    }
  } else {
    // ---------------- weights: warps 4 + 4 h + q and 12 + 4 h + q serve keys
    // 32 q + 16 h + [0, 16), the first columns [0, 64) of each half of a tile,
    // the second columns [64, 128).
    const int half = lane >> 4, quarter = (warp - 4) >> 3;
    const int rb = (warp & 3) * 32 + (((warp - 4) >> 2) & 1) * 16;
    const int r = rb + (lane & 15);
    const uint32_t lane_off = static_cast<uint32_t>(rb) << 16;
    const uint32_t s_free0 = mapa_shared(s_free, 0);
    const float scale2 = p.c.scale * kLog2e;
    int g = 0;
    for (int i = 0;; ++i) {
      int4 pa, pb;
      if (!handed_piece(i, pa, pb)) break;
      const int b = pa.x / p.c.Hkv, kvh = pa.x % p.c.Hkv, nk = pb.x, nT = pa.w;
      const int key = pa.y * KT + rank * 128 + r;
      const bool valid = key < nk;
      const int64_t meta = b * p.c.km_b + kvh * p.c.km_h, kc = min(key, nk - 1);
      const int kp = p.c.k_pos ? p.c.k_pos[meta + kc] : key;
      const int kd = p.c.k_doc ? p.c.k_doc[meta + kc] : 0;
      const int64_t at = static_cast<int64_t>(pa.x) * p.c.Lk + key;
      const bool writes = valid && half == 0 && quarter == 0;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool ok = true;
      for (int j = 0; j < nT; ++j, ++g) {
        const int st = g % QS, sb = g & 1;
        if (ok) ok = warp_wait(&s_full[sb], (g >> 1) & 1, err);
        if (!ok) continue;
        tc_fence_after();
        const uint32_t s_addr = tmem + sb * 256 + lane_off;
        float s[32];
        tmem_ld32x<128>(s_addr + 64 * quarter, s);
        ok = warp_wait(&c_full[st], (g / QS) & 1, err);
        tmem_wait_ld();
        if (!ok) continue;
        const float* col = reinterpret_cast<const float*>(smem + C::OFF_COL + st * C::COL_STRIDE);
        const int4 stat = *reinterpret_cast<const int4*>(col + COL_ARRAYS * kColWords);
        const bool whole = kp < stat.x && (!p.c.k_doc || (stat.y == kd && stat.z == kd));
        const bool masked = __any_sync(0xffffffffu, valid && !whole);
        const bool unused = stat.x == -0x7fffffff - 1;
        // 32 columns at a time.
        auto add_chunk = [&](float* v, int ch) {
          const float* cc = col + half * kHalf + ch * 32;
          const int* ic = reinterpret_cast<const int*>(cc);
          float sc = scale2;
          if constexpr ((F & F_CAP) != 0) {
            // (What unused rows hold must not choose the branch.)
            if (unused) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (ic[COL_PLIM * kColWords + e] == -0x7fffffff - 1) v[e] = 0.0f;
            }
            float big = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; e += 2) big = max3(big, fabsf(v[e]), fabsf(v[e + 1]));
            if (__all_sync(0xffffffffu, !valid || big <= p.cap_small)) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) cap2<3>(v[e], v[e + 1], p.cap_c3);
            } else if (__all_sync(0xffffffffu, !valid || big * p.cap.inv <= 1.0f)) {
              cap_within<32>(v, p.cap);
            } else {
              // (A cap over kCapLow that scores pass is rare: its form goes over local
              // memory, eight scores at a time, which keeps the loop short.)
              if (p.cap.two > 0.0f) {
                cap_low<32>(v, p.cap);
              } else {
                float t[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) t[e] = v[e];
#pragma unroll 1
                for (int e = 0; e < 32; e += 8) cap_any<8>(t + e, p.cap);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = t[e];
              }
            }
            sc = 1.0f;
          }
          if constexpr ((F & F_BIAS) != 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 ns = *reinterpret_cast<const float4*>(cc + COL_NSLOPE * kColWords + e);
              const int4 qp = *reinterpret_cast<const int4*>(ic + COL_QP * kColWords + e);
              v[e] = fmaf(v[e], sc, ns.x * fabsf(static_cast<float>(qp.x - kp)));
              v[e + 1] = fmaf(v[e + 1], sc, ns.y * fabsf(static_cast<float>(qp.y - kp)));
              v[e + 2] = fmaf(v[e + 2], sc, ns.z * fabsf(static_cast<float>(qp.z - kp)));
              v[e + 3] = fmaf(v[e + 3], sc, ns.w * fabsf(static_cast<float>(qp.w - kp)));
            }
            sc = 1.0f;
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const int4 pl = *reinterpret_cast<const int4*>(ic + COL_PLIM * kColWords + e);
              int4 qd = make_int4(kd, kd, kd, kd);
              if (p.c.k_doc) qd = *reinterpret_cast<const int4*>(ic + COL_DOC * kColWords + e);
              if (kp >= pl.x || qd.x != kd) v[e] = -INFINITY;
              if (kp >= pl.y || qd.y != kd) v[e + 1] = -INFINITY;
              if (kp >= pl.z || qd.z != kd) v[e + 2] = -INFINITY;
              if (kp >= pl.w || qd.w != kd) v[e + 3] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 nl = *reinterpret_cast<const float4*>(cc + COL_NLSE * kColWords + e);
            ffma2v(v[e], v[e + 1], sc, nl.x, nl.y);
            ffma2v(v[e + 2], v[e + 3], sc, nl.z, nl.w);
            fadd2(acc[(e & 4)], acc[(e & 4) + 1], fast_exp2(v[e]), fast_exp2(v[e + 1]));
            fadd2(acc[(e & 4) + 2], acc[(e & 4) + 3], fast_exp2(v[e + 2]), fast_exp2(v[e + 3]));
          }
        };
#pragma unroll 1
        for (int ch = 2 * quarter;; ++ch) {
          add_chunk(s, ch);
          if (ch & 1) break;
          tmem_ld32x<128>(s_addr + (ch + 1) * 32, s);
          tmem_wait_ld();
          // S^T is read: the next but one tile's products wait for it, so it is
          // given back before the second half of the weights is computed.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(s_free0 + sb * 8);
          __syncwarp();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(&c_empty[st], rank));
        __syncwarp();
      }
      float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      // The two warps of a key: the second leaves its sum for the first.
      float* other = part + (i & 1) * 128;
      if (quarter == 1 && half == 0) other[r] = sum;
      __syncwarp();
      // (A buffer of sums is used again two pieces later, behind a barrier that its
      // reader has reached.)
      asm volatile("bar.sync %0, 64;" ::"r"(1 + ((warp - 4) & 7)) : "memory");
      // mass_out holds the old mass: one addition to each entry, whose order does
      // not matter, and which needs no answer.
      if (ok && writes) atomicAdd(p.c.mass_out + at, sum + other[r]);
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
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
cudaError_t launch(const CUtensorMap* maps, const TcParams& p, int pairs, cudaStream_t st) {
  static uint64_t set_up = 0;
  // More than half an SM's shared memory: one CTA per SM, so its TMEM is free.
  const size_t smem = MCfg<DH>::SMEM > 120 * 1024 ? MCfg<DH>::SMEM : 120 * 1024;
  static_assert(MCfg<DH>::SMEM <= 232448, "over the per-block limit");
  cudaError_t e = once_per_device(&set_up, [&](int) {
    return cudaFuncSetAttribute(cache_mass_kernel<DH, BF16, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  cfg.blockDim = dim3(kMassThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cache_mass_kernel<DH, BF16, F>, maps[0], maps[1], p);
}

template <int DH, bool BF16>
cudaError_t launch_any(const CUtensorMap* maps, const TcParams& p, int pairs, cudaStream_t st) {
  if (p.c.softcap > 0)
    return p.c.slopes ? launch<DH, BF16, F_CAP | F_BIAS>(maps, p, pairs, st) : launch<DH, BF16, F_CAP>(maps, p, pairs, st);
  return p.c.slopes ? launch<DH, BF16, F_BIAS>(maps, p, pairs, st) : launch<DH, BF16, 0>(maps, p, pairs, st);
}

}  // namespace

cudaError_t launch_cache_mass_tc(const CacheParams& c, bool bf16, char* scratch, int sms, cudaStream_t st) {
  if (static_cast<int64_t>(c.Lq) * c.G <= kFewRows) {
    // Keys are independent: about 8 pieces an SM, of 128 keys at least.
    const int64_t heads = static_cast<int64_t>(c.B) * c.Hkv, most = (c.Lk + 127) / 128;
    int64_t n = (8 * static_cast<int64_t>(sms) + heads - 1) / heads;
    if (n > most) n = most;
    if (n > 304) n = 304;
    CapForm cap{};
    if (c.softcap > 0) set_cap_form(cap, c.scale, c.softcap);
    const RowsParams r{c, cap, static_cast<int>(n), 0, static_cast<int>(heads * n), sms, nullptr, nullptr, nullptr};
    return launch_cache_rows(r, bf16, true, st);
  }
  TcParams p = plan(c, scratch);
  p.queue = reinterpret_cast<int*>(scratch) + 3;
  p.n_pieces = c.B * c.Hkv * p.tiles;
  CUtensorMap maps[3];
  if (!encode_maps(maps, c, p, bf16, false)) return cudaErrorInvalidValue;
  cudaError_t e = launch_tiles(p, st);
  if (e != cudaSuccess) return e;
  if (c.mass_in != c.mass_out) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(c.B) * c.Hkv * ((c.Lk + 1023) / 1024)));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, mass_copy_kernel, p)) != cudaSuccess) return e;
  }
  const int pairs = p.n_pieces < sms / 2 ? p.n_pieces : sms / 2;
  if (p.width == 64) return bf16 ? launch_any<64, true>(maps, p, pairs, st) : launch_any<64, false>(maps, p, pairs, st);
  return bf16 ? launch_any<128, true>(maps, p, pairs, st) : launch_any<128, false>(maps, p, pairs, st);
}

}  // namespace psv

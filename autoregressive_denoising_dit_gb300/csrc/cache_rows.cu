// Attention over a cache and the attention mass for few query rows (a token,
// a draft of tokens, shared heads: at most 16 rows per kv head).
//
// Bound by reading K (and V) once: a 16-row tile of mma.sync products costs
// less than the memory traffic of its keys and needs no TMEM and no cluster.
// Persistent CTAs, one an SM, take pieces (a sequence, a kv head and one of
// nsplit equal shares of its keys) in turn.  A producer warp brings tiles of 32
// keys by TMA into a ring of stages, across the ends of pieces; each of seven
// consumer warps keeps its own running maximum, sum and output over every
// seventh tile of a piece (the chain from a tile's scores to its weights takes
// about 1 us, so fewer warps would bound it, not the memory).  The seven are
// joined in shared memory at the end of a piece, the shares by the CTA that
// ends the last of them, or where there are many by cache_join_kernel.  The next piece's queries are read while the current one
// runs.  Measured, heads of 128: eight single tokens over 7800 keys of 12 heads
// 59.2 us with the join (5.4 TB/s; the pieces are 8% uneven over the SMs), one
// token over 65536 keys 61 us (6.6 TB/s), the mass of eight tokens 31.5 us.
#include <cuda.h>

#include "../../include/psv.h"
#include "cache_cap.cuh"
#include "cache_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

namespace psv {

namespace {

constexpr int kWarps = 7;  // consumers (with the producer eight: two an SM quarter, 255 registers each)
constexpr int kKeys = 32;  // keys of a tile
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int DH, bool MASS>
struct RCfg {
  static constexpr int NA = DH / 64;
  static constexpr int ATOM = kKeys * 128;                  // 32 rows of 128 bytes
  static constexpr int STAGE = NA * ATOM * (MASS ? 1 : 2);  // K, then V
  static constexpr int JOIN = MASS ? 0 : kWarps * 16 * (DH + 2) * 4;  // [warp][16][DH], then m and l
  static constexpr int STAGES = MASS ? 2 * kWarps : 10;
  static constexpr int OFF_JOIN = STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_JOIN + JOIN;
  static constexpr size_t SMEM = OFF_BAR + (2 * kWarps + STAGES) * 8;
  // A warp's tiles are kWarps apart, so that two of them at most are under way:
  // two barriers a warp tell it of its own tiles, one phase after the other.
  static_assert(STAGES <= 2 * kWarps, "two tiles of a warp in the ring at most");
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) return pack_bf16x2(lo, hi);
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row's scores need.
struct Row {
  int qp, qd, klim, plim;
  float slope2;
};

// Key tiles [t0, t1) of a share (at most 2^23 tiles and 304 shares: the
// product fits 32 bits, whose division is short).
__device__ __forceinline__ void share_tiles(const RowsParams& p, int k_len, int share, int& t0, int& t1) {
  const uint32_t nt = static_cast<uint32_t>(k_len + kKeys - 1) / kKeys, n = static_cast<uint32_t>(p.nsplit);
  t0 = static_cast<int>(nt * static_cast<uint32_t>(share) / n);
  t1 = static_cast<int>(nt * static_cast<uint32_t>(share + 1) / n);
}

// A piece and, for this thread's two rows, their queries as A fragments (rows
// lane / 4 and + 8; columns 2 (lane % 4) + {0, 1, 8, 9} of a step of 16).
// fetch() only issues the reads (none depends on another), while the piece
// before runs; settle() uses them.
template <int DH, bool MASS>
struct Work {
  int b, kvh, share, k_len, q_len, t0, t1, prefix;
  uint32_t qf[DH / 16][4];
  Row row[2];
  float lse2[2];

  __device__ __forceinline__ void fetch(const RowsParams& p, int piece, int lane) {
    const CacheParams& c = p.c;
    share = piece % p.nsplit;
    const int bh = piece / p.nsplit;
    b = bh / c.Hkv, kvh = bh % c.Hkv;
    k_len = c.k_lens ? c.k_lens[b] : c.Lk;
    q_len = c.q_lens ? c.q_lens[b] : c.Lq;
    prefix = c.prefix ? c.prefix[b] : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = lane / 4 + 8 * e, tok = r / c.G, head = kvh * c.G + r % c.G;
      const bool there = tok < c.Lq;
      const uint16_t* q = static_cast<const uint16_t*>(c.q) + b * c.qs.b + tok * c.qs.l + head * c.qs.h;
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int d = k * 16 + x * 8 + 2 * (lane % 4);
          qf[k][e + 2 * x] = there && d < c.dh ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
        }
      }
      row[e].qp = there && c.q_pos ? c.q_pos[b * c.qm_b + tok] : 0;
      row[e].qd = there && c.q_doc ? c.q_doc[b * c.qm_b + tok] : 0;
      row[e].slope2 = there && c.slopes ? c.slopes[head] : 0.0f;
      lse2[e] = MASS && there ? c.lse[(static_cast<int64_t>(b) * c.Hq + head) * c.Lq + tok] : -INFINITY;
    }
  }

  __device__ __forceinline__ void settle(const RowsParams& p, int lane) {
    const CacheParams& c = p.c;
    k_len = min(max(k_len, 0), c.Lk);
    q_len = min(max(q_len, 0), c.Lq);
    share_tiles(p, k_len, share, t0, t1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tok = (lane / 4 + 8 * e) / c.G;
      const bool valid = tok < q_len;
      if (!valid) {  // an unused row may hold anything
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) qf[k][e] = qf[k][e + 2] = 0u;
      }
      if (!c.q_pos) row[e].qp = k_len - q_len + tok;
      row[e].slope2 *= kLog2e;
      row[e].plim = c.causal ? max(row[e].qp + 1, prefix) : 0x7fffffff;  // positions below it are seen
      row[e].klim = c.k_pos ? k_len : min(k_len, max(row[e].plim, 0));
      lse2[e] = valid && lse2[e] != -INFINITY ? lse2[e] * kLog2e : INFINITY;
    }
  }
};

// Of a tile's 32 keys, the one whose summed weight ends up in this lane: the
// lane's upper three bits choose among the eight keys 8 n + 2 (lane % 4) + x.
__device__ __forceinline__ int mass_key(int lane) {
  const int k = lane >> 2;  // bit 2 (lane 16): n's upper bit, bit 1 (8): n's lower bit, bit 0 (4): x
  return 8 * (k >> 1) + 2 * (lane % 4) + (k & 1);
}

// Joins the shares of a (sequence, kv head) by all consumers: every fourth share
// added up in order, then the four sums, as cache_join_kernel does, so that the
// bits are the same.
template <int DH, bool BF16>
__device__ __forceinline__ void join_shares(const RowsParams& p, int b, int kvh, int rows) {
  const CacheParams& c = p.c;
  const int64_t first = (static_cast<int64_t>(b) * c.Hkv + kvh) * p.nsplit;
  for (int u = threadIdx.x; u < rows * (DH / 4); u += kWarps * 32) {
    const int r = u / (DH / 4), d = u % (DH / 4) * 4;
    const float2* ml = p.part_ml + first * p.part_rows + r;
    const float* part = p.part_o + (first * p.part_rows + r) * DH + d;
    float m = -INFINITY;
#pragma unroll 8
    for (int s = 0; s < p.nsplit; ++s) m = fmaxf(m, __ldcg(ml + s * p.part_rows).x);
    const float m0 = m == -INFINITY ? 0.0f : m;
    float4 acc[4];
    float l[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) acc[w] = make_float4(0.f, 0.f, 0.f, 0.f), l[w] = 0.0f;
#pragma unroll 2
    for (int s0 = 0; s0 < p.nsplit; s0 += 4) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int s = s0 + w;
        const float2 x = s < p.nsplit ? __ldcg(ml + s * p.part_rows) : make_float2(-INFINITY, 0.0f);
        const float4 y = s < p.nsplit ? __ldcg(reinterpret_cast<const float4*>(part + static_cast<int64_t>(s) * p.part_rows * DH))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        const float f = fast_exp2(x.x - m0);
        l[w] = fmaf(f, x.y, l[w]);
        acc[w].x = fmaf(f, y.x, acc[w].x);
        acc[w].y = fmaf(f, y.y, acc[w].y);
        acc[w].z = fmaf(f, y.z, acc[w].z);
        acc[w].w = fmaf(f, y.w, acc[w].w);
      }
    }
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      acc[0].x += acc[w].x, acc[0].y += acc[w].y, acc[0].z += acc[w].z, acc[0].w += acc[w].w;
      l[0] += l[w];
    }
    const float inv = l[0] > 0.0f ? 1.0f / l[0] : 0.0f;
    const int tok = r / c.G, head = kvh * c.G + r % c.G;
    if (d < c.dh)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.o) + b * c.os.b + tok * c.os.l + head * c.os.h + d) =
          make_uint2(pack2<BF16>(acc[0].x * inv, acc[0].y * inv), pack2<BF16>(acc[0].z * inv, acc[0].w * inv));
    if (d == 0 && c.lse)
      c.lse[(static_cast<int64_t>(b) * c.Hq + head) * c.Lq + tok] =
          l[0] == 0.0f ? -INFINITY : (m + fast_log2(l[0])) * kLn2;
  }
}

template <int DH, bool BF16, bool MASS>
__global__ void __launch_bounds__(kThreads, 1)
    cache_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ RowsParams p) {
  using C = RCfg<DH, MASS>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem[];
  const CacheParams& c = p.c;
  if (smem_u32(smem) & 1023) {  // swizzled tiles
    if (threadIdx.x == 0) raise_error(c.err, ERR_BOUNDS);
    return;
  }
  const int warp = warp_id(), lane = lane_id();
  // Tile g (counted over the CTA's pieces) goes to stage g % ST and to warp g %
  // kWarps, whose tiles are told by its two barriers in turn.
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [kWarps][2]
  uint64_t* empty = full + 2 * kWarps;                              // [ST]
  auto full_of = [&](uint32_t g) { return &full[2 * (g % kWarps) + (g / kWarps) % 2]; };
  auto full_parity = [](uint32_t g) { return (g / (2 * kWarps)) & 1; };
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kWarps + ST; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    if (!MASS) prefetch_tensormap(&tmV);
  }
  __syncthreads();
  pdl_wait();

  if (warp == kWarps) {
    // ---------------- producer: one lane
    if (lane == 0) {
      uint32_t g = 0;  // tiles so far
      bool ok = true;
      auto key_len = [&](int piece) {
        return c.k_lens && piece < p.n_pieces ? c.k_lens[piece / p.nsplit / c.Hkv] : c.Lk;
      };
      int len = key_len(blockIdx.x);
      for (int piece = blockIdx.x; piece < p.n_pieces && ok; piece += gridDim.x) {
        const int next_len = key_len(piece + gridDim.x);  // read while this piece is loaded
        const int share = piece % p.nsplit, bh = piece / p.nsplit, b = bh / c.Hkv, kvh = bh % c.Hkv;
        int t0, t1;
        share_tiles(p, min(max(len, 0), c.Lk), share, t0, t1);
        len = next_len;
        for (int t = t0; t < t1; ++t, ++g) {
          const uint32_t st = g % ST;
          if (!(ok = mbar_wait(&empty[st], ((g / ST) & 1) ^ 1, c.err, ERR_ATTN_TIMEOUT))) break;
          uint8_t* dst = smem + st * C::STAGE;
          uint64_t* bar = full_of(g);
          mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
          for (int a = 0; a < C::NA; ++a) tma_load_4d(dst + a * C::ATOM, &tmK, bar, a * 64, t * kKeys, kvh, b);
          if (!MASS) {
#pragma unroll
            for (int a = 0; a < C::NA; ++a)
              tma_load_4d(dst + (C::NA + a) * C::ATOM, &tmV, bar, a * 64, t * kKeys, kvh, b);
          }
        }
      }
      // No copy may be in flight when the CTA exits (bounded; the consumers have
      // waited for all of them unless one gave up).
      const uint64_t begin = global_timer_ns();
      for (uint32_t k = g > ST ? g - ST : 0; k < g; ++k)
        while (!mbar_try_wait(full_of(k), full_parity(k)) && global_timer_ns() - begin < kWaitLimitNs) {
        }
    }
    return;
  }

  // ---------------- consumers
  const float scale2 = c.scale * kLog2e;
  uint32_t g0 = 0;  // tiles of earlier pieces
  const bool two_areas = c.Lq * c.G <= 8;
  const int jrows = two_areas ? 8 : 16;
  int n_joined = 0;
  bool ok = true;
  int piece = blockIdx.x;
  Work<DH, MASS> w, next;
  if (piece < p.n_pieces) w.fetch(p, piece, lane);
  for (; piece < p.n_pieces; piece += gridDim.x) {
    w.settle(p, lane);
    if (piece + gridDim.x < p.n_pieces) next.fetch(p, piece + gridDim.x, lane);
    const int64_t meta = w.b * c.km_b + w.kvh * c.km_h;
    const int k_len = w.k_len;
    float o[MASS ? 1 : DH / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    if (!MASS) {
#pragma unroll
      for (int n = 0; n < DH / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    }
    for (uint32_t g = g0 + (warp + kWarps - g0 % kWarps) % kWarps; g < g0 + (w.t1 - w.t0); g += kWarps) {
      const uint32_t st = g % ST;
      const int t = w.t0 + static_cast<int>(g - g0);
      const int key0 = t * kKeys;
      float old = 0.0f;
      const int jm = key0 + mass_key(lane);  // MASS: the key that this lane writes
      const int64_t at = (static_cast<int64_t>(w.b) * c.Hkv + w.kvh) * c.Lk + jm;
      if (MASS && c.mass_in && jm < k_len) old = c.mass_in[at];
      // Every lane waits: it reads what the TMA wrote.  After a failed wait the
      // warp only keeps up the barriers below.
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full_of(g), full_parity(g), c.err, ERR_ATTN_TIMEOUT));
      if (!ok) continue;
      uint8_t* tile = smem + st * C::STAGE;
      float s[4][4];  // keys 8 n + 2 (lane % 4) + {0, 1}, rows lane / 4 and + 8
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < DH / 16; ++k) {
        const int chunk = k * 2 + (lane / 8) % 2;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int key = 16 * g + (lane / 16) * 8 + lane % 8;
          uint32_t bf[4];
          ldmatrix4(bf, smem_u32(tile) + key * 128 + (chunk / 8) * C::ATOM + (((chunk % 8) ^ (key & 7)) << 4));
          mma16<BF16>(s[2 * g], w.qf[k], bf[0], bf[1]);
          mma16<BF16>(s[2 * g + 1], w.qf[k], bf[2], bf[3]);
        }
      }
      // Scores in the log2 domain, -inf where the row does not see the key.
      if (c.softcap > 0) {
        float big = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(s[n][e]));
        if (__all_sync(0xffffffffu, big * p.cap.inv <= 1.0f)) cap_within<16>(&s[0][0], p.cap);
        else cap_any<16>(&s[0][0], p.cap);
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= scale2;
      }
      if (c.slopes || c.k_pos || c.k_doc) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = key0 + 8 * n + 2 * (lane % 4) + x, jc = min(j, k_len - 1);
            const int kp = c.k_pos ? c.k_pos[meta + jc] : j;
            const int kd = c.k_doc ? c.k_doc[meta + jc] : 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = s[n][2 * e + x];
              v -= w.row[e].slope2 * fabsf(static_cast<float>(w.row[e].qp - kp));
              if (kp >= w.row[e].plim || (c.k_doc && kd != w.row[e].qd)) v = -INFINITY;
            }
          }
        }
      }
      if (key0 + kKeys > min(w.row[0].klim, w.row[1].klim)) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 8 * n + 2 * (lane % 4) + e % 2 >= w.row[e / 2].klim) s[n][e] = -INFINITY;
      }
      if constexpr (MASS) {
        // Eight keys a lane (of four lanes), summed over the eight lanes that hold
        // their rows: each step halves the keys that a lane still carries.
        float v[8];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            v[2 * n + x] = fast_exp2(s[n][x] - w.lse2[0]) + fast_exp2(s[n][2 + x] - w.lse2[1]);
#pragma unroll
        for (int d = 16, cnt = 4; d >= 4; d >>= 1, cnt >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int k = 0; k < cnt; ++k) {
            const float give = up ? v[k] : v[k + cnt], keep = up ? v[k + cnt] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        }
        if (jm < k_len) c.mass_out[at] = old + v[0];
      } else {
        uint32_t pf[2][4];
        float a[2];
        bool grow = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          mx = fmaxf(mx, fmaxf(fmaxf(s[2][2 * e], s[2][2 * e + 1]), fmaxf(s[3][2 * e], s[3][2 * e + 1])));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          a[e] = 1.0f;
          if (mx > m[e] + kRescaleThreshold) {
            a[e] = fast_exp2(m[e] - mx);
            m[e] = mx;
            grow = true;
          }
          const float m0 = m[e] == -INFINITY ? 0.0f : m[e];
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float x = fast_exp2(s[n][2 * e] - m0), y = fast_exp2(s[n][2 * e + 1] - m0);
            sum += x + y;
            pf[n / 2][e + 2 * (n % 2)] = pack2<BF16>(x, y);
          }
          l[e] = l[e] * a[e] + sum;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < DH / 8; ++n) {
            o[n][0] *= a[0], o[n][1] *= a[0];
            o[n][2] *= a[1], o[n][3] *= a[1];
          }
        }
        if (key0 + kKeys > k_len) {
          // Values behind the keys may be NaN: their weight is 0, but 0 * NaN is not.
          for (int e = (k_len - key0) * 8 + lane; e < kKeys * 8; e += 32)
#pragma unroll
            for (int x = 0; x < C::NA; ++x)
              *reinterpret_cast<uint4*>(tile + (C::NA + x) * C::ATOM + e * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();  // the ring's next copy lands after these
          __syncwarp();
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int key = 16 * g + (lane / 8 % 2) * 8 + lane % 8;
          const uint32_t base = smem_u32(tile) + C::NA * C::ATOM + key * 128;
#pragma unroll
          for (int n = 0; n < DH / 16; ++n) {
            const int chunk = n * 2 + lane / 16;
            uint32_t bf[4];
            ldmatrix4_t(bf, base + (chunk / 8) * C::ATOM + (((chunk % 8) ^ (key & 7)) << 4));
            mma16<BF16>(o[2 * n], pf[g], bf[0], bf[1]);
            mma16<BF16>(o[2 * n + 1], pf[g], bf[2], bf[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(smem_u32(&empty[st]));
    }
    if constexpr (!MASS) {
      // Join the seven warps.  Up to 8 rows there are two join areas, taken in
      // turn, so that one barrier a piece is enough: an area is written again
      // two pieces later, behind a barrier that its readers have reached.
      const int area = two_areas ? n_joined & 1 : 0;
      ++n_joined;
      float* so = reinterpret_cast<float*>(smem + C::OFF_JOIN) + area * (C::JOIN / 8);
      float* sm = so + kWarps * jrows * DH;
      const int rows = w.q_len * c.G;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        const int r = lane / 4 + 8 * e;
        if (r < rows) {
#pragma unroll
          for (int n = 0; n < DH / 8; ++n)
            *reinterpret_cast<float2*>(so + (warp * jrows + r) * DH + n * 8 + 2 * (lane % 4)) =
                make_float2(o[n][2 * e], o[n][2 * e + 1]);
          if (lane % 4 == 0) {
            sm[(warp * jrows + r) * 2] = m[e];
            sm[(warp * jrows + r) * 2 + 1] = l[e];
          }
        }
      }
      __syncwarp();
      asm volatile("bar.sync 1, 224;" ::: "memory");
      for (int u = threadIdx.x; u < rows * (DH / 4); u += kWarps * 32) {
        const int r = u / (DH / 4), d = u % (DH / 4) * 4;
        float mm = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, sm[(x * jrows + r) * 2]);
        const float m0 = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float f = fast_exp2(sm[(x * jrows + r) * 2] - m0);
          const float4 y = *reinterpret_cast<const float4*>(so + (x * jrows + r) * DH + d);
          ll = fmaf(f, sm[(x * jrows + r) * 2 + 1], ll);
          acc.x = fmaf(f, y.x, acc.x);
          acc.y = fmaf(f, y.y, acc.y);
          acc.z = fmaf(f, y.z, acc.z);
          acc.w = fmaf(f, y.w, acc.w);
        }
        const int tok = r / c.G, head = w.kvh * c.G + r % c.G;
        if (p.nsplit > 1) {
          const int64_t prow = static_cast<int64_t>(piece) * p.part_rows + r;
          *reinterpret_cast<float4*>(p.part_o + prow * DH + d) = acc;
          if (d == 0) p.part_ml[prow] = make_float2(mm, ll);
        } else {
          const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
          if (d < c.dh)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.o) + w.b * c.os.b + tok * c.os.l + head * c.os.h + d) =
                make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
          if (d == 0 && c.lse)
            c.lse[(static_cast<int64_t>(w.b) * c.Hq + head) * c.Lq + tok] =
                ll == 0.0f ? -INFINITY : (mm + fast_log2(ll)) * kLn2;
        }
      }
      if (p.joined) {
        // The last share of a (sequence, kv head) to be done joins them all, in
        // their order.
        __threadfence();
        asm volatile("bar.sync 1, 224;" ::: "memory");
        const int bh = w.b * c.Hkv + w.kvh;
        int last = 0;
        if (threadIdx.x == 0) {
          last = atomicAdd(p.joined + bh, 1) == p.nsplit - 1;
          if (last) atomicExch(p.joined + bh, 0);
        }
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %0, 0;\n\t"
            "barrier.cta.red.or.pred q, 1, 224, p;\n\t"
            "selp.b32 %0, 1, 0, q;\n\t}"
            : "+r"(last)::"memory");
        if (last) {
          __threadfence();
          join_shares<DH, BF16>(p, w.b, w.kvh, rows);
        }
      }
      __syncwarp();
      if (!two_areas) asm volatile("bar.sync 1, 224;" ::: "memory");
    }
    g0 += w.t1 - w.t0;
    w = next;
  }
}

template <int DH, bool BF16, bool MASS>
cudaError_t launch_rows(const CUtensorMap* maps, const RowsParams& p, cudaStream_t st) {
  static uint64_t set_up = 0;
  using C = RCfg<DH, MASS>;
  static_assert(C::SMEM <= 232448, "over the per-block limit");
  cudaError_t e = once_per_device(&set_up, [&](int) {
    return cudaFuncSetAttribute(cache_rows_kernel<DH, BF16, MASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_pieces < p.ctas ? p.n_pieces : p.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_rows_kernel<DH, BF16, MASS>, maps[0], maps[1], p);
}

template <bool MASS>
cudaError_t launch_rows_any(const CUtensorMap* maps, const RowsParams& p, bool bf16, cudaStream_t st) {
  if (p.c.dh <= 64) return bf16 ? launch_rows<64, true, MASS>(maps, p, st) : launch_rows<64, false, MASS>(maps, p, st);
  return bf16 ? launch_rows<128, true, MASS>(maps, p, st) : launch_rows<128, false, MASS>(maps, p, st);
}

}  // namespace

cudaError_t launch_cache_rows(const RowsParams& p, bool bf16, bool mass, cudaStream_t st) {
  const CacheParams& c = p.c;
  CUtensorMap maps[2];
  for (int i = 0; i < (mass ? 1 : 2); ++i) {
    const Strides3& s = i ? c.vs : c.ks;
    const uint64_t dims[4] = {static_cast<uint64_t>(c.dh), static_cast<uint64_t>(c.Lk),
                              static_cast<uint64_t>(c.Hkv), static_cast<uint64_t>(c.B)};
    const uint64_t str[3] = {map_stride(s.l, c.Lk), map_stride(s.h, c.Hkv), map_stride(s.b, c.B)};
    const uint32_t box[4] = {64, kKeys, 1, 1};
    if (!encode_16bit_map(&maps[i], bf16, 4, const_cast<void*>(i ? c.v : c.k), dims, str, box,
                          CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if (mass) maps[1] = maps[0];
  return mass ? launch_rows_any<true>(maps, p, bf16, st) : launch_rows_any<false>(maps, p, bf16, st);
}

}  // namespace psv

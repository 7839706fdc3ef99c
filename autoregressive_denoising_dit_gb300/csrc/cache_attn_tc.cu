// psv_cache_attention on the tensor cores: the plan of a problem (units of
// rows, shares of the keys), the kernel that notes what the key tiles hold,
// the kernel that joins the shares, and the launch.
#include "cache_attn_tc.cuh"

#include <cfloat>
#include <cmath>

namespace psv {

using namespace cattn;

namespace {

// KeyTile of every key tile and RowUnit of every unit: one warp each.  Bound by
// its launch and the latency of two dependent reads.
__global__ void __launch_bounds__(256) cache_tiles_kernel(const __grid_constant__ TcParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = lane_id();
  int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + warp_id();
  const int64_t n_tiles = static_cast<int64_t>(p.c.B) * p.meta_heads * p.tiles;
  int pmin = 0x7fffffff, pmax = -0x7fffffff - 1, dmin = pmin, dmax = pmax;
  if (w < n_tiles) {
    const int tile = static_cast<int>(w % p.tiles);
    const int h = static_cast<int>(w / p.tiles % p.meta_heads), b = static_cast<int>(w / p.tiles / p.meta_heads);
    const int n = cache_k_len(p.c, b), key0 = tile * KT;
    const int64_t meta = b * p.c.km_b + h * p.c.km_h;
    const int base = key0 < n ? (p.c.k_pos ? p.c.k_pos[meta + key0] : key0) : 0;
    // Key c = 32 i + lane: all of a lane's reads are on their way at once.
    int pos[KT / 32], doc[KT / 32];
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      const int c = 32 * i + lane;
      const bool in = key0 + c < n;
      pos[i] = p.c.k_pos && in ? p.c.k_pos[meta + key0 + c] : key0 + c;
      doc[i] = p.c.k_doc && in ? p.c.k_doc[meta + key0 + c] : 0;
    }
    bool run = true, sorted = true;
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      const int c = 32 * i + lane;
      int before = __shfl_up_sync(0xffffffffu, doc[i], 1);  // the key before's document
      const int wrapped = __shfl_sync(0xffffffffu, doc[i ? i - 1 : 0], 31);
      if (lane == 0) before = wrapped;
      if (key0 + c < n) {
        pmin = min(pmin, pos[i]), pmax = max(pmax, pos[i]);
        dmin = min(dmin, doc[i]), dmax = max(dmax, doc[i]);
        run = run && pos[i] == base + c;
        sorted = sorted && (c == 0 || before <= doc[i]);
      }
    }
    run = __all_sync(0xffffffffu, run);
    sorted = __all_sync(0xffffffffu, sorted);
    pmin = __reduce_min_sync(0xffffffffu, pmin), pmax = __reduce_max_sync(0xffffffffu, pmax);
    dmin = __reduce_min_sync(0xffffffffu, dmin), dmax = __reduce_max_sync(0xffffffffu, dmax);
    int first = 0, other = 0;  // keys of doc_min, keys of neither end
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      const bool in = key0 + 32 * i + lane < n;
      first += in && doc[i] == dmin;
      other += in && doc[i] != dmin && doc[i] != dmax;
    }
    first = __reduce_add_sync(0xffffffffu, first);
    other = __reduce_add_sync(0xffffffffu, other);
    if (lane == 0) p.key_tiles[w] = KeyTile{pmin, pmax, dmin, dmax, base, run, sorted, sorted && !other ? first : -1};
    return;
  }
  w -= n_tiles;
  if (w >= static_cast<int64_t>(p.c.B) * p.units) return;
  const int unit = static_cast<int>(w % p.units), b = static_cast<int>(w / p.units);
  const int nk = cache_k_len(p.c, b), nq = cache_q_len(p.c, b);
#pragma unroll 8
  for (int i = unit * 2 * p.tok_cta + lane; i < min(nq, (unit + 1) * 2 * p.tok_cta); i += 32) {
    const int doc = p.c.q_doc ? p.c.q_doc[b * p.c.qm_b + i] : 0;
    const int pos = p.c.q_pos ? p.c.q_pos[b * p.c.qm_b + i] : nk - nq + i;
    pmin = min(pmin, pos), pmax = max(pmax, pos);
    dmin = min(dmin, doc), dmax = max(dmax, doc);
  }
  pmin = __reduce_min_sync(0xffffffffu, pmin);
  pmax = __reduce_max_sync(0xffffffffu, pmax);
  dmin = __reduce_min_sync(0xffffffffu, dmin), dmax = __reduce_max_sync(0xffffffffu, dmax);
  if (lane == 0) p.row_units[w] = RowUnit{pmin, pmax, dmin, dmax};
}

// Units that unit_order is made for: with more there are enough pieces after the
// longest ones to even out the pairs' times.
constexpr int kOrderUnits = 512;

// Sorts a sequence's units by the key tiles that they see: rows of two documents
// see the tiles of both, and such a unit taken last kept its pair at work while
// the others were done (nine documents of 12480 rows: 150 us, sorted 136).  One CTA per sequence.
__global__ void __launch_bounds__(1024) cache_order_kernel(const __grid_constant__ TcParams p) {
  __shared__ int s_w[kOrderUnits], s_most, s_least;
  pdl_trigger();
  const int b = blockIdx.x;
  if (threadIdx.x == 0) s_most = 0, s_least = 0x7fffffff;
  __syncthreads();
  pdl_wait();
  const int nk = cache_k_len(p.c, b), nq = cache_q_len(p.c, b), n = (nk + KT - 1) / KT;
  const int prefix = p.c.prefix ? p.c.prefix[b] : 0;
  const KeyTile* tiles = p.key_tiles + static_cast<int64_t>(b) * p.meta_heads * p.tiles;  // (of the first head)
  for (int u = warp_id(); u < p.units; u += 32) {
    const RowUnit ru = p.row_units[static_cast<int64_t>(b) * p.units + u];
    const int most = max(ru.pos_max + 1, prefix);
    int w = 0;
#pragma unroll 4
    for (int t = lane_id(); t < n; t += 32) {
      const KeyTile k = tiles[t];
      w += (!p.c.k_doc || (k.doc_min <= ru.doc_max && k.doc_max >= ru.doc_min)) && (!p.c.causal || k.pos_min < most);
    }
    w = __reduce_add_sync(0xffffffffu, w);
    if (lane_id() == 0) {
      const bool rows = u * 2 * p.tok_cta < nq;
      s_w[u] = rows ? w : 0;
      if (rows) {
        atomicMax(&s_most, w);
        atomicMin(&s_least, w);
      }
    }
  }
  __syncthreads();
  int* order = p.unit_order + static_cast<int64_t>(b) * p.units;
  if (s_most <= s_least || s_most - s_least <= s_least / 4) {
    if (threadIdx.x == 0) order[0] = -1;
    return;
  }
  for (int u = threadIdx.x; u < p.units; u += 1024) {
    const int w = s_w[u];
    int rank = 0;
#pragma unroll 8
    for (int v = 0; v < p.units; ++v) rank += s_w[v] > w || (s_w[v] == w && v < u);
    order[rank] = u;
  }
}

// A head group's rows' slopes / scale as three values of the operand type whose
// sum holds 24 bits, in the layout of kLinBytes; and whether they fit it.
template <bool BF16>
__global__ void __launch_bounds__(128) cache_lin_kernel(const __grid_constant__ TcParams p) {
  pdl_trigger();
  pdl_wait();
  const int r = threadIdx.x, kvh = blockIdx.x;
  const float v = r < p.rows_cta ? p.c.slopes[kvh * p.c.G + r % p.c.G] / p.c.scale : 0.0f;
  // (f16 ends at 65504; in bf16 255 times the value must stay finite.)
  const int ok = __syncthreads_and(fabsf(v) <= (BF16 ? 1e30f : 6e4f));
  auto part = [](float x) {
    if constexpr (BF16) return __bfloat162float(__float2bfloat16_rn(x));
    else return __half2float(__float2half_rn(x));
  };
  const float hi = part(v), mid = part(v - hi), lo = v - hi - mid;
  uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.lin_q) + kvh * kLinBytes + (r / 8) * 256 + (r % 8) * 16);
  dst[0] = ok ? make_uint4(pack2<BF16>(hi, mid), pack2<BF16>(lo, 0.0f), 0, 0) : make_uint4(0, 0, 0, 0);
  dst[8] = make_uint4(0, 0, 0, 0);
  if (r == 0) p.lin_ok[kvh] = ok;
}

// Joins the shares of a row: one CTA per (sequence, head, token).  Each of its
// four warps adds up every fourth share, lanes over the columns, four shares'
// rows on the way at once; the warps' sums are added in order.  Bound by its
// launch and the latency of two dependent reads (4 us for a token's 12 heads).
template <bool BF16>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ TcParams p) {
  __shared__ float4 s_acc[4][32];
  __shared__ float s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;  // (b, tok, head), of the last unit's tokens only if only that was shared
  const int tok0 = p.tail_split ? (p.units - 1) * 2 * p.tok_cta : 0, toks = p.c.Lq - tok0;
  const int head = static_cast<int>(row % p.c.Hq);
  const int tok = tok0 + static_cast<int>(row / p.c.Hq % toks);
  const int b = static_cast<int>(row / p.c.Hq / toks);
  const int kvh = head / p.c.G, unit = tok / (2 * p.tok_cta);
  const int in_unit = tok - unit * 2 * p.tok_cta;
  const int prow = in_unit * p.c.G + head % p.c.G;  // both CTAs' rows in a row
  const int nsplit = p.tail_split ? p.tail_split : p.nsplit;
  const int64_t bh = static_cast<int64_t>(b) * p.c.Hkv + kvh;
  const int64_t first = (p.tail_split ? bh : bh * p.units + unit) * nsplit;
  const float2* ml = p.part_ml + first * p.part_rows + prow;
  const float* part = p.part_o + (first * p.part_rows + prow) * p.width + lane * 4;
  const int64_t step = p.part_rows;  // rows from one share to the next
  pdl_wait();
  if (tok >= cache_q_len(p.c, b)) return;
  float m = -INFINITY;
  for (int s = lane; s < nsplit; s += 32) m = fmaxf(m, ml[s * step].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float m0 = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool in = lane * 4 < p.width;
  for (int s0 = warp; s0 < nsplit; s0 += 16) {
    float2 w[4];
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + 4 * k;
      w[k] = s < nsplit ? ml[s * step] : make_float2(-INFINITY, 0.0f);
      x[k] = s < nsplit && in ? *reinterpret_cast<const float4*>(part + s * step * p.width)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = fast_exp2(w[k].x - m0);  // 0 for a share that saw nothing (its O is 0)
      l = fmaf(f, w[k].y, l);
      acc.x = fmaf(f, x[k].x, acc.x);
      acc.y = fmaf(f, x[k].y, acc.y);
      acc.z = fmaf(f, x[k].z, acc.z);
      acc.w = fmaf(f, x[k].w, acc.w);
    }
  }
  s_acc[warp][lane] = acc;
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    const float4 x = s_acc[k][lane];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    l += s_l[k];
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if (lane * 4 < p.c.dh) {
    uint2 v = make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.c.o) + b * p.c.os.b + tok * p.c.os.l + head * p.c.os.h +
                              lane * 4) = v;
  }
  if (lane == 0 && p.c.lse)
    p.c.lse[(static_cast<int64_t>(b) * p.c.Hq + head) * p.c.Lq + tok] = l == 0.0f ? -INFINITY : (m + fast_log2(l)) * kLn2;
}

// Pairs of SMs that the shares of a sequence are planned for (half of this
// part's 152 SMs; a constant, so that the bits do not depend on the device).
constexpr int kPlanPairs = 76;

// Counters in the workspace's head: the ints from kJoinFirst on.
constexpr int kJoinFirst = 16, kJoinCounters = PSV_CACHE_SCRATCH_HEAD / 4 - kJoinFirst, kJoinShares = 32, kJoinRows = 4;

// Shares of a last unit of few rows.
constexpr int kTailShares = 4;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct TcLayout {
  bool few;  // at most kFewRows rows per kv head
  int width, rows_cta, tok_cta, units, nsplit, tail_split, part_rows;
  int64_t pieces;
  int tiles, meta_heads;  // of the buffer; 0: no positions or documents
  bool lin;  // the distance bias by products (no cap, no positions or documents given)
  size_t part_o, part_ml, key_tiles, row_units, unit_order, lin_ok, lin_q, total;
  int order_heads;  // 0: units in their own order
};

TcLayout tc_layout(const CacheParams& c) {
  TcLayout t{};
  t.width = c.dh <= 64 ? 64 : 128;
  t.tok_cta = QT / c.G;
  t.rows_cta = t.tok_cta * c.G;
  t.units = (c.Lq + 2 * t.tok_cta - 1) / (2 * t.tok_cta);
  const int64_t rows = static_cast<int64_t>(c.Lq) * c.G;
  t.part_rows = static_cast<int>(rows < 2 * t.rows_cta ? rows : 2 * t.rows_cta);
  t.few = rows <= kFewRows;
  // A share of n tiles reads n * 256 keys of K and V and leaves part_rows rows
  // of f32: at 256 rows as many bytes as one tile, hence five tiles at least.
  // Few rows: a share is a CTA of four warps that take 32 keys at a time.
  const int tiles = t.few ? (c.Lk + 127) / 128 : (c.Lk + KT - 1) / KT / (1 + t.part_rows / 64);
  const int64_t per_seq = static_cast<int64_t>(c.Hkv) * t.units;
  // One share an SM (a pair of SMs) of a sequence.
  const int64_t slots = t.few ? 2 * kPlanPairs : kPlanPairs;
  const int64_t want = per_seq >= slots ? 1 : slots / per_seq;
  t.nsplit = static_cast<int>(want < tiles ? want : tiles);
  if (t.nsplit < 1) t.nsplit = 1;
  t.pieces = static_cast<int64_t>(c.B) * per_seq * t.nsplit;
  int64_t parts = t.nsplit > 1 ? t.pieces : 0;
  // Units of equal length leave the pairs of SMs uneven, up to a whole unit's time.
  // A last unit of few rows takes as long as any other, and its shares leave little
  // to join: taken last they even the pairs out.  (Causal units and those of
  // documents differ in length, longest first.)  1560 rows x 7800 keys of 12 heads:
  // one sequence 94 -> 66 us, two 137 -> 111, four 225 -> 212; eight 422 -> 430, as
  // their keys come from memory again, but a sequence's shares must not depend on
  // the batch.  From two rounds of units a sequence on little is left to gain, and
  // more rows would leave as much to join.
  const int64_t tail_rows = rows - static_cast<int64_t>(t.units - 1) * 2 * t.rows_cta;
  if (t.nsplit == 1 && !t.few && t.units > 1 && per_seq <= 2 * kPlanPairs && !c.causal && !c.k_doc && tail_rows <= t.rows_cta / 2 &&
      (c.Lk + KT - 1) / KT >= 4 * kTailShares) {
    t.tail_split = kTailShares;
    parts = static_cast<int64_t>(c.B) * c.Hkv * kTailShares;
    t.pieces += parts - static_cast<int64_t>(c.B) * c.Hkv;
    t.part_rows = static_cast<int>(tail_rows);
  }
  size_t off = PSV_CACHE_SCRATCH_HEAD;
  if (parts > 0) {
    t.part_o = off;
    off += up256(static_cast<size_t>(parts) * t.part_rows * t.width * 4);
    t.part_ml = off;
    off += up256(static_cast<size_t>(parts) * t.part_rows * 8);
  }
  t.tiles = (c.Lk + KT - 1) / KT;
  t.meta_heads = !t.few && (c.k_pos || c.k_doc) ? (c.km_h == 0 ? 1 : c.Hkv) : 0;
  if (t.meta_heads) {
    t.key_tiles = off;
    off += up256(sizeof(KeyTile) * static_cast<size_t>(c.B) * t.meta_heads * t.tiles);
    t.row_units = off;
    off += up256(sizeof(RowUnit) * static_cast<size_t>(c.B) * t.units);
    if (t.units > 1 && t.units <= kOrderUnits && c.k_doc && !c.causal) {
      // Four rounds of the pairs at a time; the keys of more heads than that
      // would leave L2 before the next unit reads them.
      t.order_heads = (4 * kPlanPairs + t.units - 1) / t.units;
      if (t.order_heads > c.Hkv) t.order_heads = c.Hkv;
      t.unit_order = off;
      off += up256(sizeof(int) * static_cast<size_t>(c.B) * t.units);
    }
  }
  t.lin = !t.few && c.slopes && !(c.softcap > 0) && !c.k_pos && !c.k_doc && !c.q_pos;
  if (t.lin) {
    t.lin_ok = off;
    off += up256(sizeof(int) * static_cast<size_t>(c.Hkv));
    t.lin_q = off;
    off += static_cast<size_t>(c.Hkv) * kLinBytes;
  }
  t.total = off;
  return t;
}

bool map_strides_ok(const Strides3& s, int64_t nb, int64_t nl, int64_t nh) {
  const int64_t st[3] = {s.b, s.l, s.h}, n[3] = {nb, nl, nh};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] <= 0 || st[i] % 8 != 0 || st[i] >= (int64_t{1} << 38))) return false;
  return true;
}

}  // namespace

// Whether the tensor-core kernel takes the shapes (the workspace is sized by
// this) and, with the tensors, their alignment.
bool cache_attn_tc_shape(const CacheParams& c) {
  return c.dh <= 128 && c.dh % 8 == 0 && c.G <= QT && c.Lq > 0 && c.Lk > 0 && tc_layout(c).pieces < (1 << 30);
}

bool cache_attn_tc_aligned(const CacheParams& c) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(c.q) | reinterpret_cast<uintptr_t>(c.k) |
                       reinterpret_cast<uintptr_t>(c.v) | reinterpret_cast<uintptr_t>(c.o);
  return (at & 15) == 0 && map_strides_ok(c.qs, c.B, c.Lq, c.Hq) && map_strides_ok(c.ks, c.B, c.Lk, c.Hkv) &&
         map_strides_ok(c.vs, c.B, c.Lk, c.Hkv) && map_strides_ok(c.os, c.B, c.Lq, c.Hq);
}

size_t cache_attn_tc_scratch(const CacheParams& c) { return tc_layout(c).total; }

namespace {

// tanh(sqrt z) / sqrt z interpolated at the Chebyshev points of [0, 0.18^2] and [0, 1].
constexpr double kTanh3[3] = {0.9999999437513383, -0.33330206128320755, 0.13074870575291475};
constexpr double kTanh7[7] = {0.9999999486455696, -0.3333282797859907, 0.13325076146101278, -0.05345164636973283, 0.02027970828564412, -0.006194324833673898, 0.0010380250967268723};

// Coefficients of cap2 for scores s: cap log2(e) tanh(s inv) = s sum_k c_k s^(2k).
// A polynomial of which one leaves f32's normal range is not used (the short one
// from caps of about 1e8 on, the other from 60 at heads of 128).
bool set_cap_poly(float2* out, const double* c, int n, double inv, double cap2e) {
  double power = inv;
  for (int k = 0; k < n; ++k, power *= inv * inv) {
    const double v = c[k] * power * cap2e;
    if (std::fabs(v) < FLT_MIN || std::fabs(v) > FLT_MAX) return false;
    out[k].x = out[k].y = static_cast<float>(v);
  }
  return true;
}

void set_cap(TcParams& p) {
  p.cap_small = p.cap_mid = -1.0f;
  if (!(p.c.softcap > 0)) return;
  set_cap_form(p.cap, p.c.scale, p.c.softcap);
  const double inv = static_cast<double>(p.c.scale) / p.c.softcap, cap2e = p.c.softcap * 1.4426950408889634;
  if (set_cap_poly(p.cap_c3, kTanh3, 3, inv, cap2e)) p.cap_small = static_cast<float>(0.18 / inv);
  if (set_cap_poly(p.cap_c7, kTanh7, 7, inv, cap2e)) p.cap_mid = static_cast<float>(1.0 / inv);
}

cudaError_t launch_lin(const TcParams& p, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.c.Hkv);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, cache_lin_kernel<true>, p) : cudaLaunchKernelEx(&cfg, cache_lin_kernel<false>, p);
}

cudaError_t launch_join(const TcParams& p, bool bf16, cudaStream_t st) {
  const int toks = p.tail_split ? p.c.Lq - (p.units - 1) * 2 * p.tok_cta : p.c.Lq;
  const int64_t rows = static_cast<int64_t>(p.c.B) * toks * p.c.Hq;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, cache_join_kernel<true>, p) : cudaLaunchKernelEx(&cfg, cache_join_kernel<false>, p);
}

}  // namespace

void set_cap_form(CapForm& f, float scale, float cap) {
  const double inv = static_cast<double>(scale) / cap, c2 = cap * 1.4426950408889634, scale2 = scale * 1.4426950408889634;
  f.inv = static_cast<float>(inv < FLT_MAX ? inv : FLT_MAX);
  f.c2 = static_cast<float>(c2 < FLT_MAX ? c2 : FLT_MAX);
  const double two = 2.885390081777927 * inv;
  f.two = cap <= kCapLow ? static_cast<float>(two < FLT_MAX ? two : FLT_MAX) : 0.0f;
  for (int k = 0; k < 7; ++k) f.poly[k].x = f.poly[k].y = static_cast<float>(kTanh7[k] * scale2);
}

TcParams cattn::plan(const CacheParams& c, char* scratch) {
  const TcLayout t = tc_layout(c);
  TcParams p{};
  p.c = c;
  p.rows_cta = t.rows_cta, p.tok_cta = t.tok_cta, p.units = t.units, p.nsplit = t.nsplit;
  p.tail_split = t.tail_split;
  p.n_pieces = static_cast<int>(t.pieces), p.part_rows = t.part_rows, p.width = t.width;
  p.meta_vec = ((reinterpret_cast<uintptr_t>(c.k_pos) | reinterpret_cast<uintptr_t>(c.k_doc)) & 15) == 0 &&
               c.km_b % 4 == 0 && c.km_h % 4 == 0;
  p.tiles = t.tiles;
  p.meta_heads = t.meta_heads;
  if (t.meta_heads) {
    p.key_tiles = reinterpret_cast<KeyTile*>(scratch + t.key_tiles);
    p.row_units = reinterpret_cast<RowUnit*>(scratch + t.row_units);
    if (t.order_heads) p.unit_order = reinterpret_cast<int*>(scratch + t.unit_order);
    p.order_heads = t.order_heads;
  }
  if (t.lin) {
    p.lin_ok = reinterpret_cast<int*>(scratch + t.lin_ok);
    p.lin_q = reinterpret_cast<uint16_t*>(scratch + t.lin_q);
  }
  set_cap(p);
  p.queue = reinterpret_cast<int*>(scratch) + 1;
  p.part_o = reinterpret_cast<float*>(scratch + t.part_o);
  p.part_ml = reinterpret_cast<float2*>(scratch + t.part_ml);
  return p;
}

bool cattn::encode_maps(CUtensorMap* maps, const CacheParams& c, const TcParams& p, bool bf16, bool values) {
  bool ok = true;
  {
    const uint64_t dims[4] = {static_cast<uint64_t>(c.dh), static_cast<uint64_t>(c.Hq),
                              static_cast<uint64_t>(c.Lq), static_cast<uint64_t>(c.B)};
    const uint64_t str[3] = {map_stride(c.qs.h, c.Hq), map_stride(c.qs.l, c.Lq), map_stride(c.qs.b, c.B)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(c.G), static_cast<uint32_t>(p.tok_cta), 1};
    ok &= encode_16bit_map(&maps[0], bf16, 4, const_cast<void*>(c.q), dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  for (int i = 0; i < (values ? 2 : 1); ++i) {
    const Strides3& s = i ? c.vs : c.ks;
    const uint64_t dims[4] = {static_cast<uint64_t>(c.dh), static_cast<uint64_t>(c.Lk),
                              static_cast<uint64_t>(c.Hkv), static_cast<uint64_t>(c.B)};
    const uint64_t str[3] = {map_stride(s.l, c.Lk), map_stride(s.h, c.Hkv), map_stride(s.b, c.B)};
    const uint32_t vr = static_cast<uint32_t>(p.width / 2);
    const uint32_t box[4] = {i ? vr : 64u, i ? 256u : 128u, 1, 1};
    ok &= encode_16bit_map(&maps[1 + i], bf16, 4, const_cast<void*>(i ? c.v : c.k), dims, str, box,
                           i && vr == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  }
  return ok;
}

cudaError_t cattn::launch_tiles(const TcParams& p, cudaStream_t st) {
  if (!p.key_tiles) return cudaSuccess;
  const int64_t warps = static_cast<int64_t>(p.c.B) * (static_cast<int64_t>(p.meta_heads) * p.tiles + p.units);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tiles_kernel, p);
}

cudaError_t cattn::launch_order(const TcParams& p, cudaStream_t st) {
  if (!p.unit_order) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.c.B));
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_order_kernel, p);
}

namespace {

// Whether the few-row kernel joins the shares itself (to the same bits).  That
// saves a launch, which is what a short call costs: a token over 1560 keys of 12
// heads 8.4 us against 10.9, over 3120 9.1 against 10.5.  But one CTA joins a
// head's shares after the last of them: no gain from 24 MB of keys and values on
// (7800 keys 14.4 against 13.7), and a loss with more rows (16 rows 14.6 against
// 10.3) or several pieces a CTA (three tokens 19.1 against 13.0).
bool joins_within(const TcParams& p, int sms) {
  const int64_t bytes = static_cast<int64_t>(p.c.B) * p.c.Hkv * p.c.Lk * p.c.dh * 4;
  return p.nsplit > 1 && p.nsplit <= kJoinShares && p.c.B * p.c.Hkv <= kJoinCounters && p.n_pieces <= sms &&
         p.c.Lq * p.c.G <= kJoinRows && bytes <= (24 << 20);
}

}  // namespace

cudaError_t launch_cache_attention_tc(const CacheParams& c, bool bf16, char* scratch, int sms, cudaStream_t st) {
  const TcParams p = plan(c, scratch);
  cudaError_t e;
  if (static_cast<int64_t>(c.Lq) * c.G <= kFewRows) {
    const bool within = joins_within(p, sms);
    const RowsParams r{c, p.cap, p.nsplit, p.part_rows, p.n_pieces, sms, p.part_o, p.part_ml,
                       within ? reinterpret_cast<int*>(scratch) + kJoinFirst : nullptr};
    e = launch_cache_rows(r, bf16, false, st);
    return e != cudaSuccess || p.nsplit == 1 || within ? e : launch_join(p, bf16, st);
  }
  CUtensorMap maps[4];
  if (!encode_maps(maps, c, p, bf16, true)) return cudaErrorInvalidValue;
  maps[3] = maps[0];
  if (p.lin_q) {
    const uint64_t dims[3] = {64, kLinBytes / 128, static_cast<uint64_t>(c.Hkv)}, str[2] = {128, kLinBytes};
    const uint32_t box[3] = {64, kLinBytes / 128, 1};
    if (!encode_16bit_map(&maps[3], bf16, 3, p.lin_q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return cudaErrorInvalidValue;
    if ((e = launch_lin(p, bf16, st)) != cudaSuccess) return e;
  }
  if ((e = launch_tiles(p, st)) != cudaSuccess || (e = launch_order(p, st)) != cudaSuccess) return e;
  const int pairs = p.n_pieces < sms / 2 ? p.n_pieces : sms / 2;
  const int f = (c.softcap > 0 ? F_CAP : 0) | (c.softcap > kCapLow ? F_WIDE : 0) | (c.slopes ? F_BIAS : 0) | (c.k_doc || c.k_pos || c.q_pos ? F_META : 0);
  if (p.width == 64)
    e = bf16 ? launch_features<64, true>(maps, p, f, pairs, st) : launch_features<64, false>(maps, p, f, pairs, st);
  else
    e = bf16 ? launch_features<128, true>(maps, p, f, pairs, st) : launch_features<128, false>(maps, p, f, pairs, st);
  return e != cudaSuccess || (p.nsplit == 1 && !p.tail_split) ? e : launch_join(p, bf16, st);
}

bool cache_mass_tc(const CacheParams& c) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(c.q) | reinterpret_cast<uintptr_t>(c.k);
  return cache_attn_tc_shape(c) && static_cast<int64_t>(c.B) * c.Hkv * ((c.Lk + KT - 1) / KT) < (1 << 30) &&
         (at & 15) == 0 && map_strides_ok(c.qs, c.B, c.Lq, c.Hq) && map_strides_ok(c.ks, c.B, c.Lk, c.Hkv);
}

}  // namespace psv

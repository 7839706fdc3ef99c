// Attention of a token's rows, or a few tokens', over the pages of a cache.
//
// Bound by reading the codes of K and V once.  Each warp brings its own steps of 16 or
// 32 keys by 16-byte asynchronous copies, whole rows at a time, into a ring of its own in
// shared memory, and takes the products' operands from there as they are: the
// contraction over a head's values may run in any order, so that a thread holds 16
// bytes in a row of each key (and of its query rows), and the products are
// transposed, so that keys and values are the operand of 16 rows and 8 query rows
// fill a product:
//   S^T = K Q^T      a thread holds keys lane / 4 and + 8 of a step of 16
//   O^T += V^T P^T   a thread holds the keys 2 (lane % 4) + {0, 1, 8, 9}, whose
//                    bytes of one column are paired by a byte permutation
// No barrier and no alignment to a page's start stand between the pages and the
// products.  (A copy of a thread's own 16 bytes, half a row of 128 a copy, takes a
// quarter longer: 64-byte requests to L2.)
//
// Codes become f16 (exactly); bf16 queries become f16 with a power of two for each row
// that brings its largest to [2^14, 2^15), so that values down to 2^-31 of it keep their
// eight bits; a key's scale multiplies its scores.  A value's scale enters its weight as an
// exponent, exp2(s + log2 scale - m'), with a maximum m' of its own, so that
// weights fit f16 whatever the scales are.
//
// The m and m' that f16 weights are taken relative to are maxima less 7, and a new maximum
// is taken up where a weight passes 2^15: f16 ends at 2^16, and its fixed half step of
// 2^-25 below 2^-14 is 2^-32 of the largest weight then.  (Many small weights may be all that
// an output is made of: with m the maximum, a key 17.4 below it had no weight but counted in l.)
// bf16 weights, whose values may be as large as f32's, stay at 2^8 and below.
//
// The work (16-key steps of every sequence, kv head and tile of query rows) is
// one line that is cut into equal stretches, one a CTA, whatever the lengths.
// Where a cut falls into a group its shares go to the workspace, and a second kernel
// joins them in order.  (The last of a group's CTAs to be done took 5 to 12 us to
// notice that and to join them; all SMs take 3, launch included.)  Where the tables
// cover little, groups are not cut: a cluster of CTAs takes whole groups, and its CTAs
// read one another's sums; or, where there are many groups, a warp does by itself.
//
// Measured, heads of 128, 8 bits: eight tokens over 5203 to 7800 keys of 12 heads 34 us
// (165 MB; without any products 32), one over 131072 keys of 8 heads, five query heads
// each, 50 us (277 MB, 5.5 TB/s); 16-bit pages of the former 56 us (320 MB, 5.7 TB/s).
// Of a call about 8 us are its start (lengths, tables, first keys: three round trips
// after the kernel before), the join and the ends of SMs that get less of the memory.
// Two tiles of rows (9 to 16 a kv head) are bound by the chains of conversions, products
// and softmax of two warps a scheduler: 4 x 17600 keys of 8 heads, 12 rows, 42 us (149 MB).
// No pipe is over 25 %, 1.4 instructions issue a cycle and SM; waits of fixed length are
// the commonest stall, instructions that have to be fetched the next.
#pragma once

#include <algorithm>
#include <cfloat>

#include "page_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

namespace psv {

namespace {

// Who has a group: CTAs that share it by a cut line, a cluster, or a warp by itself.
enum Mode { kCut, kClusters, kAlone };

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// What a maximum's weight is when it is taken up (as an exponent), and beyond what weight
// a new one is.
__host__ __device__ constexpr float lift(int format) { return format == PSV_PAGE_BF16 ? 0.0f : 7.0f; }
__host__ __device__ constexpr float rescale(int format) { return format == PSV_PAGE_BF16 ? 256.0f : 32768.0f; }
constexpr float kNone = -FLT_MAX;   // a maximum of nothing: exp2(-inf - kNone) = 0, exp2(kNone - kNone) = 1

constexpr bool two_products(int dh, bool scaled, int nt) { return scaled && (dh == 64 || (dh == 128 && nt == 2)); }

template <int DH, int FMT, int NT>
struct ACfg {
  static constexpr bool kScaled = FMT == PSV_PAGE_E4M3 || FMT == PSV_PAGE_I8;
  static constexpr int ES = kScaled ? 1 : 2;
  static constexpr int ROWS = 8 * NT;
  static constexpr int KP = DH * ES / 64;   // 16-byte pieces of a key in a thread
  static constexpr int KS = kScaled ? 4 : 2;  // products (of 16 values) a piece
  static constexpr int VW = DH * ES / 32;   // 4-byte words of a value in a thread
  static constexpr bool QS = NT >= 2 || DH == 256;  // queries in shared memory, for want of registers
  static constexpr int Q_BYTES = QS ? NT * KP * KS * 256 + ROWS * 4 : 0;  // operands, a factor a row
  static constexpr int JSTRIDE = DH + 4;    // floats between a join area's rows
  static constexpr int RB = DH * ES;       // bytes of a row
  static constexpr int LPR = RB / 16;      // lanes that copy it
  static constexpr int RPC = 32 / LPR;     // rows of a copy
  // Keys of a warp's step: 16 a product, twice as many where that costs no step ahead.
  static constexpr int SUBS = two_products(DH, kScaled, NT) ? 2 : 1, STEP = 16 * SUBS;
  static constexpr int START = 8 / SUBS;   // steps on the line that a group's start counts for
  static constexpr int KV = STEP * RB;     // a step's keys, or values
  static constexpr int SLOT = 2 * KV + (kScaled ? STEP * 8 : 0);  // a warp's step: K, V, the scales
  // Two CTAs an SM (128, 168 or 255 registers a thread), or one of four tiles, whose shares
  // are twice as large.
  static constexpr int CTAS = NT == 4 ? 1 : 2, MAX_CTAS = kSms * CTAS;
  static constexpr int WARPS = NT == 4 ? 8 : DH == 256 ? (kScaled ? 3 : 2) : NT == 1 && DH == 64 && !kScaled ? 8 : (NT == 1 && kScaled) || DH == 64 ? 6 : 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int JOIN = WARPS * 8 * (JSTRIDE + 4) * 4;  // the warps' sums at the end of a group, a tile at a time
  static constexpr int STAGES = std::min(4, ((224 << 10) / CTAS - JOIN - Q_BYTES - ROWS * (DH + 4) * 4) / (WARPS * SLOT));
  static constexpr int RING = WARPS * STAGES * SLOT;
  static_assert(STAGES >= 2 && WARPS >= NT, "a step ahead, a warp a tile of queries");
  static constexpr int PART = ROWS * (DH + 4) * 4;  // a CTA's sums, which its cluster reads
  static constexpr int SMEM = RING + JOIN + Q_BYTES + PART;
  static_assert(CTAS * (SMEM + 1024 + 256) <= 233472, "an SM's shared memory");
  static_assert(NT == 4 || WARPS * Q_BYTES <= JOIN, "a warp's own queries, in the join's place");
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int FMT>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (FMT == PSV_PAGE_BF16) mma_bf16(c, a, b0, b1);
  else mma_f16(c, a, b0, b1);
}

// Four floats of another CTA's shared memory.
__device__ __forceinline__ float4 load_peer(const float* at, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(at, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes as two pairs of f16: bytes 0 and 1, bytes 2 and 3.
template <int FMT>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == PSV_PAGE_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  } else {
    // 1024 + (x + 128) is the f16 whose lower byte is x + 128: 1152 less is x.
    const uint32_t u = x ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __floats2half2_rn(-1152.0f, -1152.0f);
    const __half2 c = __hadd2(*reinterpret_cast<const __half2*>(&a), off), d = __hadd2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&c);
    hi = *reinterpret_cast<const uint32_t*>(&d);
  }
}

// Copies that do not wait; `bytes` 0 leaves zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where 16-byte piece `piece` of row `row` of a step lies: within 128 bytes pieces
// change places so that eight lanes that read two adjacent rows' four pieces (keys) or
// four even or odd rows' two (values) meet in no bank.
template <int RB>
__device__ __forceinline__ int placed(int row, int piece) {
  if constexpr (RB == 64) return row / 2 * 128 + ((row % 2 * 4 + piece) ^ (row / 2 % 4 * 2)) * 16;
  return row * RB + (piece ^ (((row / 4 ^ row) & 1) * 4 + (row & 2))) * 16;
}

// The row of the piece that lies in the 16 bytes number `at`.
template <int RB>
__device__ __forceinline__ int row_at(int at) {
  return RB == 64 ? at / 8 * 2 + ((at % 8) ^ (at / 8 % 4 * 2)) / 4 : at / (RB / 16);
}

// What a sequence's steps are: steps [0, head) from key 0 on (the sinks), the
// others from key `from` on.
struct Seq {
  int rows, n, keys;  // query rows, length, keys that may have a page
  int head, from, steps, tiles;
  int64_t total;  // on the line, of all its kv heads and row tiles
  int span;       // a group's
};

template <class C>
__device__ __forceinline__ Seq sequence(const PageAttnParams& p, int rows, int n) {
  constexpr int kStep = C::STEP;
  Seq s;
  s.rows = rows;
  s.n = n;
  s.keys = min(n, p.c.positions);
  const int first = p.window ? max(n - rows - p.window + 1, 0) : 0;  // of the first row
  const int end = (s.keys + kStep - 1) / kStep;
  s.head = min(p.window ? (min(p.sinks, s.keys) + kStep - 1) / kStep : 0, end);
  const int from = min(max(first / kStep, s.head), end);
  s.from = from * kStep;
  s.steps = max(s.head + end - from, 1);  // (a row without keys is written too)
  s.span = s.steps + C::START;
  s.tiles = (rows * p.G + C::ROWS - 1) / C::ROWS;
  s.total = static_cast<int64_t>(s.span) * s.tiles * p.Hkv;
  return s;
}

// a / b for 0 <= a, 0 < b, in 32 bits where they do.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The line of all groups (of `span` units: `start` of them, then a unit a step) in `ctas` equal
// stretches.
struct Cut {
  int64_t all, each;
  int ctas, more, start;
  __device__ __forceinline__ Cut(int64_t a, int n, int s) : all(a), each(0), ctas(n), more(0), start(s) {
    if (n) each = divide(a, n), more = static_cast<int>(a - each * n);
  }
  __device__ __forceinline__ int64_t begin(int cta) const {
    return each * cta + static_cast<int>(__fdiv_rn(static_cast<float>(more * cta), static_cast<float>(ctas)));  // (exact: < 2^23)
  }
  // A cut this near to an end of its group is moved there, so that fewer CTAs have
  // shares of two groups, and none has a start alone.
  __device__ __forceinline__ int near(int span) const {
    return max(static_cast<int>(min(each >> 3, static_cast<int64_t>(span >> 2))), start + 1);
  }
  // By how much, `within` units into a sequence of groups of `span`.
  __device__ __forceinline__ int moved(int64_t within, int span) const {
    const int rest = static_cast<int>(within - divide(within, span) * span), n = near(span);
    return rest < n ? -rest : span - rest < n ? span - rest : 0;
  }
  __device__ __forceinline__ int of(int64_t x) const { return static_cast<int>(divide((x + 1) * ctas - 1, all)); }
};

// The lse of a row with statistics m, l (without the lift l's logarithm is near 0 where few keys count).
__device__ __forceinline__ float row_lse(int format, float mm_l, float ll) {
  return ll == 0.0f ? -INFINITY : (mm_l + lift(format) + fast_log2(ll * (format == PSV_PAGE_BF16 ? 1.0f : 0x1p-7f))) * kLn2;
}

// What a row's sum of values times weights is multiplied by: it has statistics m', m, l.
__device__ __forceinline__ float finish(float mm_o, float mm_l, float ll) {
  return ll > 0.0f ? fast_exp2(mm_o - mm_l) / ll : ll;  // (0 or NaN)
}

// A row's finished value (four of it) and lse.
__device__ __forceinline__ void write_out(const PageAttnParams& p, int b, int kvh, int row, int d, float mm_o, float mm_l,
                                          float ll, float4 acc) {
  const int tok = p.by_group.div(row), head = kvh * p.G + row - tok * p.G;
  const float f = finish(mm_o, mm_l, ll);
  if (d < p.dh) {
    const uint2 y = p.bf16 ? make_uint2(pack2<true>(acc.x * f, acc.y * f), pack2<true>(acc.z * f, acc.w * f))
                           : make_uint2(pack2<false>(acc.x * f, acc.y * f), pack2<false>(acc.z * f, acc.w * f));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + b * p.os.b + tok * p.os.l + head * p.os.h + d) = y;
  }
  if (d == 0 && p.lse)
    p.lse[(static_cast<int64_t>(b) * p.Hq + head) * p.Lq + tok] = row_lse(p.c.format, mm_l, ll);
}

// Takes a share with statistics m', m, l into a sum.
__device__ __forceinline__ void add_share(float& mm_o, float& mm_l, float& ll, float4& acc, float4 st, float4 y) {
  const float m = fmaxf(mm_o, st.x), f = fast_exp2(mm_o - m), g = fast_exp2(st.x - m);
  acc.x = fmaf(g, y.x, acc.x * f), acc.y = fmaf(g, y.y, acc.y * f);
  acc.z = fmaf(g, y.z, acc.z * f), acc.w = fmaf(g, y.w, acc.w * f);
  mm_o = m;
  const float n = fmaxf(mm_l, st.y);
  ll = fmaf(st.z, fast_exp2(st.y - n), ll * fast_exp2(mm_l - n));
  mm_l = n;
}

template <int DH, int FMT, int NT, int MODE>
__global__ void __launch_bounds__(ACfg<DH, FMT, NT>::THREADS, ACfg<DH, FMT, NT>::CTAS)
    page_attn_kernel(const __grid_constant__ PageAttnParams p) {
  using C = ACfg<DH, FMT, NT>;
  constexpr bool CLUSTER = MODE == kClusters, WARP = MODE == kAlone, WHOLE = MODE != kCut;
  constexpr int ROWS = C::ROWS, kWarps = C::WARPS, kThreads = C::THREADS, kStages = C::STAGES;
  constexpr int SUBS = C::SUBS, kStep = C::STEP, kHalves = kStep / 8, kAhead = 32 / kHalves;
  constexpr bool kBf16Operands = FMT == PSV_PAGE_BF16;
  constexpr int kPart = share_floats(DH, ROWS);
  extern __shared__ __align__(128) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem + C::RING);  // [kWarps][8][JSTRIDE]
  float* sm = so + kWarps * 8 * C::JSTRIDE;              // [kWarps][8][4]: m', m, l
  // QS: [NT][KP * KS / 2][lane], of the CTA's group, or in the join's place of the warp's
  uint4* sq = reinterpret_cast<uint4*>(smem + C::RING + (WARP ? warp_id() * C::Q_BYTES : C::JOIN));
  float* sq_up = reinterpret_cast<float*>(sq + NT * C::KP * C::KS * 16);  // [ROWS]
  float* sp = reinterpret_cast<float*>(smem + C::RING + C::JOIN + C::Q_BYTES);  // CLUSTER: a share
  const PageCacheDev& c = p.c;
  const int warp = warp_id(), lane = lane_id(), quad = lane / 4, four = lane % 4;
  if (p.dh < DH) {  // pieces behind the head stay zeros
    for (int i = threadIdx.x; i < C::RING / 16; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();

  // The unit of the line: a step, or in clusters a group.
  const int peers = CLUSTER ? p.cluster : 1, rank = CLUSTER ? blockIdx.x % peers : 0;
  const int worker = WARP ? 0 : rank * kWarps + warp, workers = WARP ? 1 : peers * kWarps;
  auto units = [&](const Seq& x) { return WHOLE ? static_cast<int64_t>(x.tiles) * p.Hkv : x.total; };
  // The line's length, this CTA's stretch [lo, hi) of it, and the sequence that it begins in.
  const int place_of = WARP ? warp * gridDim.x + blockIdx.x : blockIdx.x / peers;
  const int places = WARP ? gridDim.x * kWarps : gridDim.x / peers;
  int64_t lo = 0, hi = 0;
  int b = 0;
  int64_t before = 0;  // steps of earlier sequences
  Seq s;
  Cut cut(0, 0, C::START);
  if (!WHOLE && threadIdx.x == 0) p.shared[blockIdx.x].rows = 0;
  auto sequence_at = [&](int k) {
    const int rows = page_rows(p, k);
    return sequence<C>(p, rows, page_length(p, k, rows));
  };
  if (p.quick) {  // up to 32 sequences a lane, 32 bits
    const int each = (p.B + 31) / 32;
    auto units32 = [&](const Seq& x) { return (WHOLE ? 1 : x.span) * x.tiles * p.Hkv; };
    int own = 0, rows_b = 0, n_b = 0;
    if (lane * each < p.B) {
      rows_b = page_rows(p, lane * each);
      n_b = page_length(p, lane * each, rows_b);
      own = units32(sequence<C>(p, rows_b, n_b));
    }
    if (each > 1) {
#pragma unroll 4
      for (int k = lane * each + 1; k < min((lane + 1) * each, p.B); ++k) own += units32(sequence_at(k));
      __syncwarp();
    }
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    cut = Cut(all, min(places, WHOLE ? all : (all + kWarps - 1) / kWarps), C::START);
    if (place_of >= cut.ctas) return;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int x = static_cast<int>(cut.begin(place_of + i));
      const unsigned hit = __ballot_sync(0xffffffffu, sum > x);
      lo = hi;
      hi = x;
      if (!hit) break;  // (behind all)
      const int at = __ffs(hit) - 1;
      int k = at * each, first = __shfl_sync(0xffffffffu, sum - own, at);
      Seq y;
      if (each == 1) {
        y = sequence<C>(p, __shfl_sync(0xffffffffu, rows_b, at), __shfl_sync(0xffffffffu, n_b, at));
      } else {
        // lane by lane the sequences of lane `at`
        int rows = 0, n = 0, mine = 0;
        if (lane < each && k + lane < p.B) {
          rows = page_rows(p, k + lane);
          n = page_length(p, k + lane, rows);
          mine = units32(sequence<C>(p, rows, n));
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += up;
        }
        const int in = __ffs(__ballot_sync(0xffffffffu, first + upto > x)) - 1;
        first += __shfl_sync(0xffffffffu, upto - mine, in);
        k += in;
        y = sequence<C>(p, __shfl_sync(0xffffffffu, rows, in), __shfl_sync(0xffffffffu, n, in));
      }
      if (!WHOLE) hi = x + cut.moved(x - first, y.span);
      if (i == 0) b = k, before = first, s = y;
    }
  } else {
    int64_t all = 0;
#pragma unroll 8
    for (int k = lane; k < p.B; k += 32) all += units(sequence_at(k));
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    cut = Cut(all, static_cast<int>(min(static_cast<int64_t>(places), WHOLE ? all : (all + kWarps - 1) / kWarps)), C::START);
    if (place_of >= cut.ctas) return;
    int64_t sum0 = 0, x = cut.begin(place_of);
    bool begun = false;
    auto units_at = [&](int k) { return k < p.B ? units(sequence_at(k)) : 0; };
    int64_t own = units_at(lane), ahead = units_at(32 + lane);
    for (int b0 = 0;;) {
      int64_t sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      // the cut at x lies in one of these sequences, or behind all
      const unsigned hit = __ballot_sync(0xffffffffu, sum0 + sum > x);
      if (hit || x >= all) {
        const int at = max(__ffs(hit) - 1, 0);
        const int64_t first = sum0 + __shfl_sync(0xffffffffu, sum - own, at);
        Seq y;
        int64_t moved = x;
        if (hit) {
          y = sequence_at(b0 + at);
          if (!WHOLE) moved += cut.moved(x - first, y.span);
        }
        if (begun) {
          hi = moved;
          break;
        }
        begun = true;
        b = b0 + at;
        before = first;
        s = y;
        lo = moved;
        x = cut.begin(place_of + 1);
        continue;  // (its end may lie in the same sequences)
      }
      sum0 += __shfl_sync(0xffffffffu, sum, 31);
      b0 += 32;
      own = ahead, ahead = units_at(b0 + 32 + lane);
    }
  }

  // Places within a step (128-byte aligned, so that a change of bits 4 to 6 changes places
  // of pieces): what this lane copies of rows [0, RPC), its pieces of key lane / 4 and of
  // value 2 (lane % 4).  Row i RPC + r is copied to (copied ^ flip(i)) + i 512, piece
  // four + 4 i of the key is at (key_at ^ 64 (i % 2)) + 128 (i / 2), the next row's value at
  // (value_at ^ 64) + RB (rows of 64 bytes: two to 128, value_at ^ 64).
  const uint32_t ring = smem_u32(smem), ring0 = warp * kStages * C::SLOT;
  const uint32_t copied = placed<C::RB>(lane / C::LPR, lane % C::LPR);
  const uint32_t key_at = placed<C::RB>(quad, four);
  const uint32_t value_at = C::RB == 64 ? placed<C::RB>(2 * four, quad / 2) + quad % 2 * 8 : placed<C::RB>(2 * four, quad);
  auto flip = [](int i) -> uint32_t {
    return C::RB == 512 ? ((i / 4 ^ i) % 2 * 4 + i / 2 % 2 * 2) * 16 : C::RB == 256 ? (i / 2 * 4 + i % 2 * 2) * 16 : i * 64;
  };
  const bool in_head = lane % C::LPR * 16 < p.dh * C::ES;  // the piece that this lane copies
  const bool eights = c.page_size % 8 == 0;  // eight keys lie in one page
  const int sinks = p.window ? p.sinks : 0;
  const char *k_mine = nullptr, *v_mine = nullptr, *s_mine[SUBS];  // (scales: of keys and values by lane, or one after the other)
  int kvh = 0, r0 = 0, n_rows = 0, step0 = 0, step1 = 0, taken = 0, slot = 0;
  int all_end = 0, any_end = 0, all_first = 0, any_first = 0;
  uint32_t found = 0;  // a bit for each step under way: whether key lane % 16 is there
  // Where the keys of the warp's next steps are: in lane kHalves i + h the eight keys h of
  // number i of kAhead steps, and of those behind them, or where eight keys may lie in
  // several pages of the next step key lane % kStep.
  PageRow place{-1, 0}, later{-1, 0};
  int issued = 0;  // steps of the group that the warp has asked for
  auto key_of = [&](int step) { return step < s.head ? step * kStep : s.from + (step - s.head) * kStep; };
  auto look = [&](int number) {  // of the warp's steps
    const int step = step0 + worker + (number + (eights ? lane / kHalves : 0)) * workers;
    return step < step1 ? page_row(c, b, key_of(step) + (eights ? lane % kHalves * 8 : lane % kStep)) : PageRow{-1, 0};
  };
  auto offset = [](uint32_t page_stride, uint32_t row_stride, int page, int row) {
    return static_cast<uint64_t>(page_stride) * static_cast<uint32_t>(page) +
           static_cast<uint64_t>(row_stride) * static_cast<uint32_t>(row);
  };
  auto issue = [&](int into) {
    const int step = step0 + worker + issued * workers, number = issued++;
    found <<= 1;
    if (step >= step1) return;
    const uint32_t dst = ring0 + into * C::SLOT;
    const int key0 = key_of(step);
    // Keys that some row of the tile sees are read.
    const bool every = key0 + kStep <= any_end && (key0 >= any_first || key0 + kStep <= sinks);
    PageRow at = place;  // of key lane % kStep
    int pages[kHalves], rows[kHalves], least = 0;
    if (eights) {
      const int first = number % kAhead * kHalves;
      if (first == 0 && number) place = later, later = look(number + kAhead);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        pages[h] = __shfl_sync(0xffffffffu, place.page, first + h);
        rows[h] = __shfl_sync(0xffffffffu, place.row, first + h);
        least = min(least, pages[h]);
      }
      at.page = __shfl_sync(0xffffffffu, place.page, first + lane % kStep / 8);
      at.row = __shfl_sync(0xffffffffu, place.row, first + lane % kStep / 8) + lane % 8;
    }
    if (eights && every && !p.halves && least >= 0) {
      found |= 1;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const char* k = k_mine + offset(p.kb, p.kl, pages[h], rows[h]);
        const char* v = v_mine + offset(p.vb, p.vl, pages[h], rows[h]);
        if (in_head) {
#pragma unroll
          for (int i = 0; i < 8 / C::RPC; ++i) {
            const uint32_t to = ring + ((dst + copied) ^ flip(i)) + (h * 8 / C::RPC + i) * 512;
            copy16(to, k + static_cast<uint64_t>(p.kl) * (i * C::RPC));
            copy16(to + C::KV, v + static_cast<uint64_t>(p.vl) * (i * C::RPC));
          }
        }
      }
      if constexpr (C::kScaled) {
        const uint64_t from = offset(p.sb, p.sl, at.page, at.row);
#pragma unroll
        for (int x = 0; x < SUBS; ++x) copy4(ring + dst + 2 * C::KV + x * 128 + lane * 4, s_mine[x] + from, 4);
      }
      return;
    }
    // Key by key; what is not wanted (keys, pieces behind the head) is zeros.
    if (!eights) place = look(issued);
    const int j = key0 + lane % kStep;
    if (at.page < 0 || j >= any_end || (j < any_first && j >= sinks)) at = PageRow{-1, 0};
    found |= at.page >= 0;
#pragma unroll 1
    for (int i = 0; i < kStep / C::RPC; ++i) {
      const int key = i * C::RPC + lane / C::LPR;
      const int page = __shfl_sync(0xffffffffu, at.page, key), row = __shfl_sync(0xffffffffu, at.row, key) - lane / C::LPR;
      const uint32_t to = ring + dst + placed<C::RB>(key, lane % C::LPR);
      const int bytes = page >= 0 && in_head ? 16 : 0;
      const char* from_k = bytes ? k_mine + offset(p.kb, 0, page, 0) + static_cast<int64_t>(p.kl) * row : static_cast<const char*>(c.k);
      const char* from_v = bytes ? v_mine + offset(p.vb, 0, page, 0) + static_cast<int64_t>(p.vl) * row : static_cast<const char*>(c.v);
      if (!C::kScaled || !p.halves) {
        copy16(to, from_k, bytes);
        copy16(to + C::KV, from_v, bytes);
      } else {
        const int more = bytes && lane % C::LPR * 16 + 8 < p.dh ? 8 : 0;  // bytes of the second half
        copy8(to, from_k, bytes / 2);
        copy8(to + 8, from_k + more, more);
        copy8(to + C::KV, from_v, bytes / 2);
        copy8(to + C::KV + 8, from_v + more, more);
      }
    }
    if constexpr (C::kScaled) {
      const uint64_t from = offset(p.sb, p.sl, max(at.page, 0), at.row);
#pragma unroll
      for (int x = 0; x < SUBS; ++x) copy4(ring + dst + 2 * C::KV + x * 128 + lane * 4, s_mine[x] + from, at.page >= 0 ? 4 : 0);
    }
  };
  // The column pair that this thread's products i belong to.
  auto column_of = [&](int i) {
    return C::VW == 2 ? quad * 8 + 2 * i : C::kScaled ? (quad + 8 * (i / 8)) * 16 + 2 * (i % 8) : (quad + 8 * (i / 4)) * 8 + 2 * (i % 4);
  };
  float o[NT][DH / 16][4], mo[NT][2], ml[NT][2], l[NT][2];
  bool joining = false, split = false;  // the group before, whose sums are still the warps'
  int was_b = 0, was_kvh = 0, was_r0 = 0, was_rows = 0, was_slot = 0;
  while (true) {
    const bool more = lo < hi;
    constexpr int kPer = 16 / C::ES;  // values of a piece
    constexpr bool kOneTile = C::QS && !WARP;  // a warp brings a tile of queries, or all
    constexpr int NQ = kOneTile ? 1 : NT;
    uint32_t raw[NQ][C::KP][kPer / 2];
    if (more) {
      // ---- the next group: its first keys and its queries are on their way before the last one is joined
      while (lo >= before + units(s)) {
        before += units(s);
        s = sequence_at(++b);
      }
      const int64_t within = lo - before;
      const int group = static_cast<int>(WHOLE ? within : divide(within, s.span));
      const int at = WHOLE ? 0 : static_cast<int>(within - static_cast<int64_t>(group) * s.span);
      taken = WHOLE ? 1 : static_cast<int>(min(static_cast<int64_t>(s.span - at), hi - lo));
      step0 = max(at - C::START, 0);
      step1 = WHOLE ? s.steps : at + taken - C::START;
      kvh = s.tiles == 1 ? group : group / s.tiles;
      r0 = (group - kvh * s.tiles) * ROWS;
      n_rows = min(s.rows * p.G - r0, ROWS);
      // what all rows see and what any of them sees, by their positions
      const int at0 = s.n - s.rows + static_cast<int>(p.by_group.div(r0));
      const int at1 = s.n - s.rows + static_cast<int>(p.by_group.div(r0 + n_rows - 1));
      all_end = p.causal ? min(at0 + 1, s.keys) : s.keys, any_end = p.causal ? min(at1 + 1, s.keys) : s.keys;
      all_first = p.window ? at1 - p.window + 1 : 0, any_first = p.window ? at0 - p.window + 1 : 0;
      // the piece that this lane copies of the first rows of page 0
      k_mine = static_cast<const char*>(c.k) + kvh * c.ks.h * C::ES + offset(0, p.kl, 0, lane / C::LPR) + lane % C::LPR * 16;
      v_mine = static_cast<const char*>(c.v) + kvh * c.vs.h * C::ES + offset(0, p.vl, 0, lane / C::LPR) + lane % C::LPR * 16;
#pragma unroll
      for (int x = 0; x < SUBS; ++x)
        s_mine[x] = reinterpret_cast<const char*>(((SUBS == 1 ? lane < 16 : x == 0) ? c.k_scale : c.v_scale) + kvh * c.ss.h);
      issued = 0;
      slot = 0;
      place = look(0);
      if (eights) later = look(kAhead);
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        // queries: row quad (+ 8) of the tile, values of this thread's pieces
        const int r_tile = 8 * (kOneTile ? warp : t) + quad;
        const bool there = r_tile < n_rows;
        const int r = r0 + r_tile, tok = p.by_group.div(r), head = kvh * p.G + r - tok * p.G;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.qs.b + tok * p.qs.l + head * p.qs.h;
#pragma unroll
        for (int i = 0; i < C::KP; ++i) {
          const int d = (four + 4 * i) * kPer;
#pragma unroll
          for (int x = 0; x < kPer / 8; ++x) {
            const uint4 y = there && d + 8 * x < p.dh ? *reinterpret_cast<const uint4*>(q + d + 8 * x) : make_uint4(0, 0, 0, 0);
            raw[t][i][4 * x] = y.x, raw[t][i][4 * x + 1] = y.y, raw[t][i][4 * x + 2] = y.z, raw[t][i][4 * x + 3] = y.w;
          }
        }
      }
      __syncwarp();  // (all lanes have read the slots that are filled again)
#pragma unroll 1
      for (int i = 0; i < kStages - 1; ++i) {
        issue(i);
        copies_commit();
      }
    }
    if (WARP && joining) {
      // ---- the warp's rows are whole
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], w);
          const int r = 8 * t + 2 * four + x;
          if (r >= was_rows) continue;
          const float ll = l[t][x], f = finish(C::kScaled ? mo[t][x] : ml[t][x], ml[t][x], ll);
          const int tok = p.by_group.div(was_r0 + r), head = was_kvh * p.G + was_r0 + r - tok * p.G;
          uint16_t* out = static_cast<uint16_t*>(p.o) + was_b * p.os.b + tok * p.os.l + head * p.os.h;
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            const int d = column_of(i);
            if (d < p.dh)
              *reinterpret_cast<uint32_t*>(out + d) = p.bf16 ? pack2<true>(o[t][i][x] * f, o[t][i][2 + x] * f)
                                                             : pack2<false>(o[t][i][x] * f, o[t][i][2 + x] * f);
          }
          if (quad == 0 && p.lse)
            p.lse[(static_cast<int64_t>(was_b) * p.Hq + head) * p.Lq + tok] = row_lse(FMT, ml[t][x], ll);
        }
      __syncwarp();
    } else if (joining) {
      // ---- join the warps
      float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + was_slot) * kPart;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (8 * t >= was_rows) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], w);
          const int r = 2 * four + x;
          if (8 * t + r < was_rows) {
            float* row = so + (warp * 8 + r) * C::JSTRIDE;
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
              const int d = column_of(i);
              *reinterpret_cast<float2*>(row + d) = make_float2(o[t][i][x], o[t][i][2 + x]);
            }
            if (quad == 0)
              *reinterpret_cast<float4*>(sm + (warp * 8 + r) * 4) = make_float4(C::kScaled ? mo[t][x] : ml[t][x], ml[t][x], l[t][x], 0.0f);
          }
        }
        __syncthreads();
#pragma unroll 1
        for (int x = threadIdx.x; x < min(was_rows - 8 * t, 8) * (DH / 4); x += kThreads) {
          const int r = x / (DH / 4), d = x % (DH / 4) * 4, row = 8 * t + r;
          float4 st[kWarps];
          float mm_o = kNone, mm_l = kNone;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            st[w] = *reinterpret_cast<const float4*>(sm + (w * 8 + r) * 4);
            mm_o = fmaxf(mm_o, st[w].x);
            mm_l = fmaxf(mm_l, st[w].y);
          }
          float ll = 0.0f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(so + (w * 8 + r) * C::JSTRIDE + d);
            const float f = fast_exp2(st[w].x - mm_o);
            ll = fmaf(fast_exp2(st[w].y - mm_l), st[w].z, ll);
            acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
            acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
          }
          if (split) {
            float* to = CLUSTER ? sp : part;
            *reinterpret_cast<float4*>(to + row * DH + d) = acc;
            if (d == 0) *reinterpret_cast<float4*>(to + ROWS * DH + row * 4) = make_float4(mm_o, mm_l, ll, 0.0f);
          } else {
            write_out(p, was_b, was_kvh, was_r0 + row, d, mm_o, mm_l, ll, acc);
          }
        }
        __syncthreads();
      }
      if (CLUSTER && split) {
        cluster_sync();
#pragma unroll 1
        for (int x = rank * kThreads + threadIdx.x; x < was_rows * (DH / 4); x += peers * kThreads) {
          const int r = x / (DH / 4), d = x % (DH / 4) * 4;
          float mm_o = kNone, mm_l = kNone, ll = 0.0f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < peers; ++k)
            add_share(mm_o, mm_l, ll, acc, load_peer(sp + ROWS * DH + r * 4, k), load_peer(sp + r * DH + d, k));
          write_out(p, was_b, was_kvh, was_r0 + r, d, mm_o, mm_l, ll, acc);
        }
        cluster_sync();  // (the sums are read; a CTA that ends takes its own along)
      }
    }
    if (!more) break;

    // ---- queries as operands: f16 with the row's largest value in [2^14, 2^15) where they are bf16 and codes f16
    uint32_t qf[C::QS ? 1 : NT][C::KP * C::KS][2];
    float up[NT][2];  // by row of the scores: what its power of two took
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (kOneTile && warp >= NT) continue;
      const int tile = kOneTile ? warp : t;
      float e = 1.0f;
      if (C::kScaled && p.bf16) {
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < C::KP; ++i)
#pragma unroll
          for (int x = 0; x < kPer / 2; ++x)
            big = max(big, max(raw[t][i][x] << 16 & 0x7fff0000u, raw[t][i][x] & 0x7fff0000u));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = big >= 0x7f800000u ? 0 : min(max(static_cast<int>(big >> 23) - 127, -112), 127);
        const float down = __int_as_float((127 + 14 - ex) << 23);
        e = __int_as_float((127 - 14 + ex) << 23);
#pragma unroll
        for (int i = 0; i < C::KP; ++i)
#pragma unroll
          for (int x = 0; x < kPer / 2; ++x)
            raw[t][i][x] = pack2<false>(__uint_as_float(raw[t][i][x] << 16) * down,
                                        __uint_as_float(raw[t][i][x] & 0xffff0000u) * down);
      }
      // (the cap takes raw products)
      if (!(p.softcap > 0)) e *= p.scale * kLog2e;
      if constexpr (C::QS) {
#pragma unroll
        for (int i = 0; i < C::KP * C::KS / 2; ++i) {
          const uint32_t* y = &raw[t][0][0] + 4 * i;
          sq[(tile * (C::KP * C::KS / 2) + i) * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (four == 0) sq_up[8 * tile + quad] = e;
      } else {
#pragma unroll
        for (int i = 0; i < C::KP * C::KS; ++i) qf[t][i][0] = (&raw[t][0][0])[2 * i], qf[t][i][1] = (&raw[t][0][0])[2 * i + 1];
        // (row quad's factor to the threads that hold its scores)
        up[t][0] = __shfl_sync(0xffffffffu, e, (2 * four) * 4);
        up[t][1] = __shfl_sync(0xffffffffu, e, (2 * four + 1) * 4);
      }
    }
    if constexpr (kOneTile) __syncthreads();
    else if constexpr (C::QS) __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (C::QS && NT < 4) up[t][0] = sq_up[8 * t + 2 * four], up[t][1] = sq_up[8 * t + 2 * four + 1];
#pragma unroll
      for (int i = 0; i < DH / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][i][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) mo[t][x] = ml[t][x] = kNone, l[t][x] = 0.0f;
    }

    [[maybe_unused]] const bool mixed = all_end < any_end || any_first < all_first;  // keys that some rows see and others do not
#pragma unroll 1
    for (int step = step0 + worker; step < step1; step += workers) {
      __syncwarp();  // (all lanes have read the step before, whose slot is filled again)
      issue(slot == 0 ? kStages - 1 : slot - 1);
      copies_commit();
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint32_t mine = ring0 + slot * C::SLOT;
      slot = slot == kStages - 1 ? 0 : slot + 1;
      const unsigned there = __ballot_sync(0xffffffffu, found >> (kStages - 1) & 1);
      if (!there) continue;
      // ---- scores
      float sc[SUBS][NT][4];
#pragma unroll
      for (int h = 0; h < SUBS; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[h][t][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::KP; ++i) {
        uint32_t qs[NT][2 * C::KS];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < C::KS / 2; ++x) {
            if constexpr (C::QS) {
              const uint4 y = sq[(t * (C::KP * C::KS / 2) + i * (C::KS / 2) + x) * 32 + lane];
              qs[t][4 * x] = y.x, qs[t][4 * x + 1] = y.y, qs[t][4 * x + 2] = y.z, qs[t][4 * x + 3] = y.w;
            } else {
#pragma unroll
              for (int z = 0; z < 4; ++z) qs[t][4 * x + z] = qf[t][i * C::KS + 2 * x + z / 2][z % 2];
            }
          }
#pragma unroll
        for (int h = 0; h < SUBS; ++h) {
          const uint8_t* key = smem + ((mine + key_at) ^ (i % 2 * 64)) + i / 2 * 128 + h * 16 * C::RB;
          const uint4 k0 = *reinterpret_cast<const uint4*>(key), k1 = *reinterpret_cast<const uint4*>(key + 8 * C::RB);
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int x = 0; x < C::KS; ++x) {
            uint32_t a[4];
            if constexpr (C::kScaled) {
              widen<FMT>(w0[x], a[0], a[2]);
              widen<FMT>(w1[x], a[1], a[3]);
            } else {
              a[0] = w0[2 * x], a[1] = w1[2 * x], a[2] = w0[2 * x + 1], a[3] = w1[2 * x + 1];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) mma<FMT>(sc[h][t], a, qs[t][2 * x], qs[t][2 * x + 1]);
          }
        }
      }
      // ---- scores and weights' exponents in the log2 domain
      const int key0 = key_of(step);
#pragma unroll
      for (int h = 0; h < SUBS; ++h) {
        float ks[2] = {1.0f, 1.0f};
        if constexpr (C::kScaled) {
          const float* scales = reinterpret_cast<const float*>(smem + mine + 2 * C::KV) + 16 * h;
          ks[0] = scales[quad], ks[1] = scales[quad + 8];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (NT == 4) up[t][0] = sq_up[8 * t + 2 * four], up[t][1] = sq_up[8 * t + 2 * four + 1];
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[h][t][e] *= C::kScaled ? ks[e >> 1] * up[t][e & 1] : up[t][e & 1];
        }
      }
      if (p.softcap > 0) {
        float big = 0.0f;
#pragma unroll
        for (int h = 0; h < SUBS; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(sc[h][t][e]));
        if (__all_sync(0xffffffffu, big * p.cap.inv <= 1.0f)) cap_within<4 * NT * SUBS>(&sc[0][0][0], p.cap);
        else cap_any<4 * NT * SUBS>(&sc[0][0][0], p.cap);
      }
      const bool whole = (key0 + kStep <= all_end && (key0 >= all_first || key0 + kStep <= sinks)) && there == 0xffffffffu;
      // whether row r of the tile sees the step's key
      auto sees = [&](int r, int key) {
        const int at_row = s.n - s.rows + static_cast<int>(p.by_group.div(r0 + r)), j = key0 + key;
        return r < n_rows && ((there >> key) & 1) && j < (p.causal ? min(at_row + 1, s.keys) : s.keys) &&
               (!p.window || j > at_row - p.window || j < sinks);
      };
      // ---- weights, two tiles at a time, and the second product's operand
      uint32_t pb[SUBS][NT][2];
      constexpr int kPair = NT < 2 ? NT : 2;
#pragma unroll
      for (int t0 = 0; t0 < NT; t0 += kPair) {
        if (t0 && 8 * t0 >= n_rows) {  // (no rows there)
#pragma unroll
          for (int h = 0; h < SUBS; ++h)
#pragma unroll
            for (int t = t0; t < t0 + kPair; ++t) pb[h][t][0] = pb[h][t][1] = 0;
          continue;
        }
        float u[SUBS][kPair][4];
#pragma unroll
        for (int h = 0; h < SUBS; ++h) {
          float lv[2] = {0.0f, 0.0f};
          if constexpr (C::kScaled) {
            const float* scales = reinterpret_cast<const float*>(smem + mine + 2 * C::KV) + kStep + 16 * h;
            lv[0] = fast_log2(scales[quad]), lv[1] = fast_log2(scales[quad + 8]);
          }
#pragma unroll
          for (int t = 0; t < kPair; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[h][t][e] = C::kScaled ? sc[h][t0 + t][e] + lv[e >> 1] : sc[h][t0 + t][e];
        }
        if (!whole) {
          if (FMT == PSV_PAGE_E4M3 && t0 == 0 && mixed) {
            // A value's code that is NaN, where some rows see its key and others do not: its
            // weight there will be 0, but 0 * NaN is not.  The code becomes a zero and the
            // value's scale NaN, and with it its weight in the rows that see the key.
            // (12 causal rows over 17600 keys 38.5 us without this and 38.8, single tokens
            // 38.3 and 38.5; handled before the scores 39.6 and 38.4.)
            __syncwarp();
            auto nans = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u) >> 7; };  // 1 a byte
            float* scales = reinterpret_cast<float*>(smem + mine + 2 * C::KV) + kStep;
#pragma unroll 1
            for (int i = lane; i < C::KV / 16; i += 32) {
              uint4* code = reinterpret_cast<uint4*>(smem + mine + C::KV) + i;
              const uint4 z = *code;
              if (nans(z.x) | nans(z.y) | nans(z.z) | nans(z.w)) {
                *code = make_uint4(z.x & ~(nans(z.x) * 0xff), z.y & ~(nans(z.y) * 0xff), z.z & ~(nans(z.z) * 0xff),
                                   z.w & ~(nans(z.w) * 0xff));
                scales[row_at<C::RB>(i)] = __int_as_float(0x7fc00000);
              }
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < SUBS; ++h)
#pragma unroll
              for (int t = 0; t < kPair; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float x = scales[16 * h + quad + 8 * (e >> 1)];
                  if (x != x) u[h][t][e] = x;
                }
          }
#pragma unroll
          for (int h = 0; h < SUBS; ++h)
#pragma unroll
            for (int t = 0; t < kPair; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!sees(8 * (t0 + t) + 2 * four + (e & 1), 16 * h + quad + 8 * (e >> 1)))
                  sc[h][t0 + t][e] = -INFINITY, u[h][t][e] = -INFINITY;
        }
        // a new maximum is taken up where one passes the old one by far
        float w[SUBS][kPair][4], y[SUBS][kPair][4];
        auto weigh = [&]() {
          float big = 0.0f;
#pragma unroll
          for (int h = 0; h < SUBS; ++h)
#pragma unroll
            for (int t = 0; t < kPair; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[h][t][e] = fast_exp2(sc[h][t0 + t][e] - ml[t0 + t][e & 1]);
                w[h][t][e] = C::kScaled ? fast_exp2(u[h][t][e] - mo[t0 + t][e & 1]) : y[h][t][e];
                big = fmaxf(big, fmaxf(y[h][t][e], w[h][t][e]));
              }
          return big;
        };
        if (__any_sync(0xffffffffu, weigh() > rescale(FMT))) {
#pragma unroll
          for (int t = 0; t < kPair; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float a = fmaxf(sc[0][t0 + t][x], sc[0][t0 + t][2 + x]), d = fmaxf(u[0][t][x], u[0][t][2 + x]);
              if (SUBS > 1) {
                a = fmaxf(a, fmaxf(sc[SUBS - 1][t0 + t][x], sc[SUBS - 1][t0 + t][2 + x]));
                d = fmaxf(d, fmaxf(u[SUBS - 1][t][x], u[SUBS - 1][t][2 + x]));
              }
#pragma unroll
              for (int i = 4; i < 32; i <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, i));
                if (C::kScaled) d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, i));
              }
              a = fmaxf(a - lift(FMT), ml[t0 + t][x]);
              if (C::kScaled) d = fmaxf(d - lift(FMT), mo[t0 + t][x]);
              const float g = fast_exp2(ml[t0 + t][x] - a), f = C::kScaled ? fast_exp2(mo[t0 + t][x] - d) : g;
              l[t0 + t][x] *= g;
              ml[t0 + t][x] = a;
              if (C::kScaled) mo[t0 + t][x] = d;
#pragma unroll
              for (int i = 0; i < DH / 16; ++i) o[t0 + t][i][x] *= f, o[t0 + t][i][2 + x] *= f;
            }
          weigh();
        }
#pragma unroll
        for (int h = 0; h < SUBS; ++h)
#pragma unroll
          for (int t = 0; t < kPair; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) l[t0 + t][e & 1] += y[h][t][e];
            pb[h][t0 + t][0] = movmatrix_t(pack2<kBf16Operands>(w[h][t][0], w[h][t][1]));
            pb[h][t0 + t][1] = movmatrix_t(pack2<kBf16Operands>(w[h][t][2], w[h][t][3]));
          }
      }
#pragma unroll
      for (int h = 0; h < SUBS; ++h) {
        uint32_t v[4][C::VW];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint8_t* from = smem + ((mine + value_at) ^ (x % 2 * 64)) + (C::RB == 64 ? 0 : x % 2 * C::RB) + C::KV +
                                (x / 2 * 8 + 16 * h) * C::RB;
          if constexpr (C::VW == 2) {
            const uint2 z = *reinterpret_cast<const uint2*>(from);
            v[x][0] = z.x, v[x][1] = z.y;
          } else {
#pragma unroll
            for (int i = 0; i < C::VW / 4; ++i) {
              const uint4 z = *reinterpret_cast<const uint4*>(from + i * 128);
              v[x][4 * i] = z.x, v[x][4 * i + 1] = z.y, v[x][4 * i + 2] = z.z, v[x][4 * i + 3] = z.w;
            }
          }
        }
        // ---- O^T += V^T P^T
        if constexpr (!C::kScaled) {
          // A value that is not finite, where some row does not see its key: its weight
          // there is 0, but 0 * NaN is not.  Row by row, with the values that it sees.
          bool odd = false;
          if (!whole) {
            constexpr uint32_t kExp = FMT == PSV_PAGE_BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int i = 0; i < C::VW; ++i)
                odd |= (v[x][i] & kExp) == kExp || (v[x][i] >> 16 & kExp) == kExp;
          }
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll 1
              for (int n = 0; n < 8; ++n) {
                uint32_t see[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  see[x] = sees(8 * t + n, 16 * h + 2 * four + (x & 1) + 8 * (x >> 1)) ? 0xffffffffu : 0u;
#pragma unroll
                for (int i = 0; i < DH / 16; ++i) {
                  const uint32_t z[4] = {v[0][i] & see[0], v[1][i] & see[1], v[2][i] & see[2], v[3][i] & see[3]};
                  const uint32_t a[4] = {__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[0], z[1], 0x7632),
                                         __byte_perm(z[2], z[3], 0x5410), __byte_perm(z[2], z[3], 0x7632)};
                  float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma<FMT>(add, a, pb[h][t][0], pb[h][t][1]);
                  if (n == 2 * four) o[t][i][0] += add[0], o[t][i][2] += add[2];
                  if (n == 2 * four + 1) o[t][i][1] += add[1], o[t][i][3] += add[3];
                }
              }
            continue;
          }
        }
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) {
          uint32_t a[4];
          if constexpr (C::kScaled) {
            const uint32_t sel = i % 2 ? 0x7362 : 0x5140;
            widen<FMT>(__byte_perm(v[0][i / 2], v[1][i / 2], sel), a[0], a[1]);
            widen<FMT>(__byte_perm(v[2][i / 2], v[3][i / 2], sel), a[2], a[3]);
          } else {
            a[0] = __byte_perm(v[0][i], v[1][i], 0x5410), a[1] = __byte_perm(v[0][i], v[1][i], 0x7632);
            a[2] = __byte_perm(v[2][i], v[3][i], 0x5410), a[3] = __byte_perm(v[2][i], v[3][i], 0x7632);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) mma<FMT>(o[t][i], a, pb[h][t][0], pb[h][t][1]);
        }
      }
    }

    // ---- what its join needs
    joining = true;
    split = WHOLE ? peers > 1 : step0 > 0 || step1 < s.steps;
    was_b = b, was_kvh = kvh, was_r0 = r0, was_rows = n_rows;
    was_slot = step0 == 0;
    if (!WHOLE && split && was_slot && threadIdx.x == 0) {
      // (the last cut that is not moved to the group's end)
      const int shares = cut.of(lo + s.span - cut.near(s.span)) - static_cast<int>(blockIdx.x) + 1;
      p.shared[blockIdx.x] = PageShared{n_rows, shares, b, kvh, r0};
    }
    lo += taken;
  }
}

constexpr int kJoinThreads = 128;

// Joins row blockIdx.y of the group that CTA blockIdx.x of the attention began.  A team of
// lanes, four values each, has every kTeams'th share; statistics and values are read at
// once, kReads shares at a time (a round trip to L2 takes 0.6 us), and the teams meet in
// shared memory.  (Small CTAs find room beside the attention's last ones, so that all
// wait for its end already: with 512 threads a CTA everything takes 1 to 2 us more.)
template <int DH>
__global__ void __launch_bounds__(kJoinThreads) page_join_kernel(const __grid_constant__ PageAttnParams p, int row_tile) {
  constexpr int kReads = 10, kLanes = DH / 4, kTeams = kJoinThreads / kLanes;
  __shared__ float4 sums[kJoinThreads];
  __shared__ float4 stats[kTeams];
  const int team = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4, r = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  const PageShared g = p.shared[blockIdx.x];
  if (r >= g.rows) return;
  const int floats = share_floats(DH, row_tile);
  const float* part = p.part + 2 * static_cast<int64_t>(blockIdx.x) * floats;
  float mm_o = kNone, mm_l = kNone, ll = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = team; k0 < g.shares; k0 += kReads * kTeams) {
    float4 z[kReads], st[kReads];
#pragma unroll
    for (int e = 0; e < kReads; ++e) {
      const int k = k0 + e * kTeams;
      if (k >= g.shares) break;
      // (a share that begins its group is its CTA's second, one that goes on with it its first)
      const float* share = part + static_cast<int64_t>(2 * k + (k == 0)) * floats;
      z[e] = __ldcg(reinterpret_cast<const float4*>(share + r * DH + d));
      st[e] = __ldcg(reinterpret_cast<const float4*>(share + row_tile * DH + r * 4));
    }
#pragma unroll
    for (int e = 0; e < kReads; ++e) {
      if (k0 + e * kTeams >= g.shares) break;
      add_share(mm_o, mm_l, ll, acc, st[e], z[e]);
    }
  }
  if (team) {
    sums[threadIdx.x] = acc;
    if (d == 0) stats[team] = make_float4(mm_o, mm_l, ll, 0.0f);
  }
  __syncthreads();
  if (team) return;
#pragma unroll
  for (int k = 1; k < kTeams; ++k) add_share(mm_o, mm_l, ll, acc, stats[k], sums[threadIdx.x + k * kLanes]);
  write_out(p, g.b, g.kvh, g.r0 + r, d, mm_o, mm_l, ll, acc);
}

template <int DH, int FMT, int NT, int MODE>
cudaError_t launch(const PageAttnParams& p, int sms, cudaStream_t st) {
  using C = ACfg<DH, FMT, NT>;
  static uint64_t set_up = 0;
  cudaError_t e = once_per_device(&set_up, [](int) {
    return cudaFuncSetAttribute(page_attn_kernel<DH, FMT, NT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  const int most = std::min(sms, kSms) * C::CTAS;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = MODE == kClusters ? p.cluster : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  const int64_t clusters = std::min<int64_t>(most / p.cluster, p.groups);
  cfg.gridDim = dim3(static_cast<unsigned>(MODE == kClusters ? clusters * p.cluster : most));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kClusters ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, page_attn_kernel<DH, FMT, NT, MODE>, p);
  if (e != cudaSuccess || MODE != kCut) return e;
  cfg.gridDim.y = static_cast<unsigned>(std::min(p.Lq * p.G, C::ROWS));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, page_join_kernel<DH>, p, C::ROWS);
}

// Whether 16-bit pages of heads of 128 are read once for 32 rows (2.1 us a step of all an
// SM's warps, two products of 16 rows each) instead of for 16 (1.4 us, which is what L2
// gives): where that is less in all, for groups of 4000 keys at least and 12 steps a warp,
// as these CTAs are an SM's only ones and their warps take no groups alone.  Measured, 8 x
// 7800 keys of 12 heads, 32 rows 94 and 128 us, 48 156 and 133, 64 166 and 237, 96 228 and
// 254; 64 groups of 4000 37 and 49, 256 of 1000 59 and 56; 8 of 17600 30 and 28.  (In 8 bits
// 32 rows take 93 us and 81: steps of 32 keys hide more of the conversions.)  The compiler
// spills 176 to 296 bytes a thread here, at 255 registers.
inline bool four_tiles(const PageAttnParams& p) {
  const int64_t rows = static_cast<int64_t>(p.Lq) * p.G, two = (rows + 15) / 16, four = (rows + 31) / 32;
  const int64_t steps = (p.window ? std::min<int64_t>(p.c.positions, static_cast<int64_t>(p.window) + p.sinks) : p.c.positions) / 16;
  return 21 * four < 14 * two && steps >= 240 && p.B * p.Hkv * four * steps >= 12 * 8 * kSms;
}

template <int DH, int FMT, int NT>
cudaError_t launch_tile(PageAttnParams p, int sms, cudaStream_t st) {
  using C = ACfg<DH, FMT, NT>;
  const int64_t tiles = (static_cast<int64_t>(p.Lq) * p.G + C::ROWS - 1) / C::ROWS;
  p.groups = p.B * p.Hkv * tiles;
  // At the greatest length that the tables allow:
  const int64_t steps = (p.window ? std::min<int64_t>(p.c.positions, static_cast<int64_t>(p.window) + p.Lq + p.sinks + 2 * C::STEP)
                                  : p.c.positions) / C::STEP + 1;
  p.quick = p.B <= 1024 && p.groups * (p.c.positions / C::STEP + 3 + C::START) < (int64_t{1} << 31);
  // As many CTAs a group as there is room for, at most 8.
  p.cluster = 1;
  while (p.cluster < 8 && p.groups * p.cluster * 2 <= C::MAX_CTAS && p.cluster * C::WARPS < steps) p.cluster *= 2;
  // What the modes would take, in us: rounds of groups, each with its steps (t: all warps'
  // in turn at 44 kB an SM and us) and its start and end.  Fitted on 8-bit heads of 128 and
  // taken as it is for other widths, formats and tiles.  Measured there:
  //   clusters against cuts: 12 groups of 1000 keys 7.4 and 12.1 us, 4000 10.8 and 12.5, 8000
  //   14.6 and 14.3; 96 of 2000 16.7 and 20.3, 7800 44 and 36; 384 of 500 18.8 and 21.1
  //   warps alone against cuts: 2048 groups of 250 keys 39 and 46 us, 8000 of 300 119 and 177,
  //   1000 of 300 22 and 40, 8198 of 100 78 and 178
  auto rounds = [](int64_t n, int64_t d) { return static_cast<double>((n + d - 1) / d); };
  const double t = 1.0 * C::CTAS * C::WARPS * C::SLOT / 44e3;
  const double alone = rounds(p.groups, C::MAX_CTAS * C::WARPS) * (steps * t + 3.3);
  // (Clusters of one do worse than this where lengths are uneven: 2048 groups of 235 to 1000
  // keys 91 us, cuts 83; all of 1000 97 and 101.)
  const double clusters = (p.cluster == 1 ? 1.1 : 1.0) * rounds(p.groups * p.cluster, C::MAX_CTAS) * (rounds(steps, p.cluster * C::WARPS) * t + 5.5);
  const double cut = static_cast<double>(p.groups) / C::MAX_CTAS * (steps * t / C::WARPS + 5.0) + 11.0;
  if constexpr (NT < 4) {  // (four tiles' queries do not fit a warp's registers beside their sums)
    if (alone < std::min(clusters, cut)) return launch<DH, FMT, NT, kAlone>(p, sms, st);
  }
  return clusters < cut ? launch<DH, FMT, NT, kClusters>(p, sms, st) : launch<DH, FMT, NT, kCut>(p, sms, st);
}

}  // namespace

template <int DH, int FMT>
cudaError_t launch_page_rows(const PageAttnParams& p, int sms, cudaStream_t st) {
  if constexpr (DH < 256) {  // (the sums of 16 rows of 256 values do not fit the registers)
    if constexpr (DH == 128 && (FMT == PSV_PAGE_BF16 || FMT == PSV_PAGE_F16)) {
      if (four_tiles(p)) return launch_tile<DH, FMT, 4>(p, sms, st);
    }
    if (p.Lq * p.G > 8) return launch_tile<DH, FMT, 2>(p, sms, st);
  }
  return launch_tile<DH, FMT, 1>(p, sms, st);
}

}  // namespace psv

// Attention of a token's rows, or a few tokens', over the pages of a cache.
//
// Bound by reading the codes of K and V once.  A thread brings the very bytes that
// its products take, by 16-byte asynchronous copies into a ring of its own in shared
// memory: the contraction over a head's values may run in any order, so that a
// thread holds 16 bytes in a row of each key (and of its query rows), and the
// products are transposed, so that keys and values are the operand of 16 rows and 8
// query rows fill a product:
//   S^T = K Q^T      a thread holds keys lane / 4 and + 8 of a step of 16
//   O^T += V^T P^T   a thread holds the keys 2 (lane % 4) + {0, 1, 8, 9}, whose
//                    bytes of one column are paired by a byte permutation
// No barrier and no alignment to a page's start stand between the pages and the
// products, and 100 to 200 kB an SM are on their way.
//
// Codes become f16 (exactly); queries become f16 with a power of two for each row;
// a key's scale multiplies its scores.  A value's scale enters its weight as an
// exponent, exp2(s + log2 scale - m'), with a maximum m' of its own, so that
// weights fit f16 whatever the scales are.
//
// The work (16-key steps of every sequence, kv head and tile of query rows) is
// one line that is cut into equal stretches, one a CTA, whatever the lengths.
// Where a cut falls into a group its shares go to the workspace and the last CTA
// to be done joins them in order.
#include <algorithm>
#include <cfloat>

#include "page_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

namespace psv {

namespace {

constexpr int kStep = 16;  // keys of a warp's step
constexpr int kCtasSm = 2;
constexpr int kMaxCtas = 152 * kCtasSm;  // shares in the workspace
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 256.0f;  // weights above it take up a new maximum
constexpr float kNone = -FLT_MAX;   // a maximum of nothing: exp2(-inf - kNone) = 0, exp2(kNone - kNone) = 1

template <int DH, int FMT, int NT>
struct ACfg {
  static constexpr bool kScaled = FMT == PSV_PAGE_E4M3 || FMT == PSV_PAGE_I8;
  static constexpr int ES = kScaled ? 1 : 2;
  static constexpr int ROWS = 8 * NT;
  static constexpr int KP = DH * ES / 64;   // 16-byte pieces of a key in a thread
  static constexpr int KS = kScaled ? 4 : 2;  // products (of 16 values) a piece
  static constexpr int VW = DH * ES / 32;   // 4-byte words of a value in a thread
  static constexpr int JSTRIDE = DH + 4;    // floats between a join area's rows
  static constexpr int K_BYTES = 2 * KP * 512, V_BYTES = 4 * VW * 128;
  static constexpr int SLOT = K_BYTES + V_BYTES + (kScaled ? 128 : 0);  // a warp's step: K, V, the scales
  // Two CTAs an SM: 128, 168 or 255 registers a thread.
  static constexpr int WARPS = NT == 1 && DH == 64 ? 8 : NT == 1 && kScaled ? 6 : DH == 64 ? 6 : 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int STAGES = std::min(4, (112 << 10) / (WARPS * SLOT));
  static constexpr int RING = WARPS * STAGES * SLOT;
  static constexpr int JOIN = WARPS * ROWS * (JSTRIDE + 4) * 4;  // in the ring's place
  static constexpr int SMEM = RING > JOIN ? RING : JOIN;
  static_assert(2 * (SMEM + 1024 + 64) <= 233472, "two CTAs an SM");
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
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

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
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
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffff), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x >> 16), __NV_E4M3);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
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

// Copies of 16 or 8 bytes that do not wait; `bytes` 0 leaves zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// What a sequence's steps are: steps [0, head) from key 0 on (the sinks), the
// others from key `from` on.
struct Seq {
  int rows, n, keys;  // query rows, length, keys that may have a page
  int head, from, steps, tiles;
  int64_t total;  // steps of all its kv heads and row tiles
};

template <int ROWS>
__device__ __forceinline__ Seq sequence(const PageAttnParams& p, int b) {
  Seq s;
  s.rows = page_rows(p, b);
  s.n = page_length(p, b, s.rows);
  s.keys = min(s.n, p.c.positions);
  const int first = p.window ? max(s.n - s.rows - p.window + 1, 0) : 0;  // of the first row
  const int end = (s.keys + kStep - 1) / kStep;
  s.head = min(p.window ? (min(p.sinks, s.keys) + kStep - 1) / kStep : 0, end);
  const int from = min(max(first / kStep, s.head), end);
  s.from = from * kStep;
  s.steps = max(s.head + end - from, 1);  // (a row without keys is written too)
  s.tiles = (s.rows * p.G + ROWS - 1) / ROWS;
  s.total = static_cast<int64_t>(s.steps) * s.tiles * p.Hkv;
  return s;
}

// The line of `all` steps in `ctas` stretches, the first ones a step longer.
struct Cut {
  int ctas, more;
  int64_t each;
  __device__ __forceinline__ Cut(int64_t all, int n) : ctas(n), more(0), each(0) {
    if (n) each = all / n, more = static_cast<int>(all - each * n);
  }
  __device__ __forceinline__ int64_t begin(int cta) const { return each * cta + min(cta, more); }
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t longer = (each + 1) * more;
    return static_cast<int>(x < longer ? x / (each + 1) : more + (x - longer) / each);
  }
};

template <int DH, int FMT, int NT>
__global__ void __launch_bounds__(ACfg<DH, FMT, NT>::THREADS, kCtasSm)
    page_attn_kernel(const __grid_constant__ PageAttnParams p) {
  using C = ACfg<DH, FMT, NT>;
  constexpr int ROWS = C::ROWS, kWarps = C::WARPS, kThreads = C::THREADS;
  constexpr bool kBf16Operands = FMT == PSV_PAGE_BF16;
  constexpr int kStages = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);      // [kWarps][ROWS][JSTRIDE]
  float* sm = so + kWarps * ROWS * C::JSTRIDE;     // [kWarps][ROWS][4]: m', m, l
  __shared__ int s_last;
  const PageCacheDev& c = p.c;
  const int warp = warp_id(), lane = lane_id(), quad = lane / 4, four = lane % 4;
  pdl_trigger();
  pdl_wait();

  // The line's length, and this CTA's stretch of it.
  static_assert(kMaxCtas * sizeof(int) <= PSV_PAGE_SCRATCH_HEAD, "counters in the workspace's head");
  int64_t all = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32)
    if (b0 + lane < p.B) all += sequence<ROWS>(p, b0 + lane).total;
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  const Cut cut(all, static_cast<int>(min(static_cast<int64_t>(gridDim.x), (all + kWarps - 1) / kWarps)));
  if (static_cast<int>(blockIdx.x) >= cut.ctas) return;
  int64_t lo = cut.begin(blockIdx.x);
  const int64_t hi = cut.begin(blockIdx.x + 1);
  // The sequence that it begins in.
  int b = 0;
  int64_t before = 0;  // steps of earlier sequences
  for (int b0 = 0;; b0 += 32) {
    const int64_t mine = b0 + lane < p.B ? sequence<ROWS>(p, b0 + lane).total : 0;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > lo);
    if (hit) {
      const int at = __ffs(hit) - 1;
      b = b0 + at;
      before += __shfl_sync(0xffffffffu, sum - mine, at);
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  Seq s = sequence<ROWS>(p, b);

  while (true) {
    const int64_t within = lo - before;
    const int group = static_cast<int>(within / s.steps), step0 = static_cast<int>(within - static_cast<int64_t>(group) * s.steps);
    const int step1 = static_cast<int>(min(static_cast<int64_t>(s.steps), step0 + (hi - lo)));
    const int kvh = group / s.tiles, r0 = group % s.tiles * ROWS;
    const int n_rows = min(s.rows * p.G - r0, ROWS);

    // ---- queries: row quad (+ 8) of the tile, values of this thread's pieces
    uint32_t qf[NT][C::KP * C::KS][2];
    float up[NT][2];  // by row of the scores: what its power of two took
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = r0 + 8 * t + quad, tok = r / p.G, head = kvh * p.G + r % p.G;
      const bool there = 8 * t + quad < n_rows;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.qs.b + tok * p.qs.l + head * p.qs.h;
      constexpr int kPer = 16 / C::ES;  // values of a piece
      uint32_t raw[C::KP][kPer / 2];
#pragma unroll
      for (int i = 0; i < C::KP; ++i) {
        const int d = (four + 4 * i) * kPer;
#pragma unroll
        for (int x = 0; x < kPer / 8; ++x) {
          const uint4 y = there && d + 8 * x < p.dh ? *reinterpret_cast<const uint4*>(q + d + 8 * x) : make_uint4(0, 0, 0, 0);
          raw[i][4 * x] = y.x, raw[i][4 * x + 1] = y.y, raw[i][4 * x + 2] = y.z, raw[i][4 * x + 3] = y.w;
        }
      }
      float e = 1.0f;
      if (C::kScaled && p.bf16) {
        // to f16, with the row's largest value in [1, 2)
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < C::KP; ++i)
#pragma unroll
          for (int x = 0; x < kPer / 2; ++x) big = max(big, max(raw[i][x] << 16 & 0x7fff0000u, raw[i][x] & 0x7fff0000u));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = big >= 0x7f800000u ? 0 : min(max(static_cast<int>(big >> 23) - 127, -120), 120);
        const float down = __int_as_float((127 - ex) << 23);
        e = __int_as_float((127 + ex) << 23);
#pragma unroll
        for (int i = 0; i < C::KP; ++i)
#pragma unroll
          for (int x = 0; x < kPer / 2; ++x)
            raw[i][x] = pack2<false>(__uint_as_float(raw[i][x] << 16) * down, __uint_as_float(raw[i][x] & 0xffff0000u) * down);
      }
#pragma unroll
      for (int i = 0; i < C::KP; ++i)
#pragma unroll
        for (int x = 0; x < C::KS; ++x) qf[t][i * C::KS + x][0] = raw[i][2 * x], qf[t][i * C::KS + x][1] = raw[i][2 * x + 1];
      // (row quad's factor to the threads that hold its scores; the cap takes raw products)
      if (!(p.softcap > 0)) e *= p.scale * kLog2e;
      up[t][0] = __shfl_sync(0xffffffffu, e, (2 * four) * 4);
      up[t][1] = __shfl_sync(0xffffffffu, e, (2 * four + 1) * 4);
    }
    // ---- what this thread's rows of scores, 8 t + 2 four + {0, 1}, see
    int end[NT][2], first[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * t + 2 * four + x, at = s.n - s.rows + (r0 + r) / p.G;
        end[t][x] = r < n_rows ? (p.causal ? min(at + 1, s.keys) : s.keys) : 0;
        first[t][x] = p.window ? at - p.window + 1 : 0;
      }
    const int sinks = p.window ? p.sinks : 0;
    // by all rows and by any of them
    const int at0 = s.n - s.rows + r0 / p.G, at1 = s.n - s.rows + (r0 + n_rows - 1) / p.G;
    const int all_end = p.causal ? min(at0 + 1, s.keys) : s.keys, any_end = p.causal ? min(at1 + 1, s.keys) : s.keys;
    const int all_first = p.window ? at1 - p.window + 1 : 0, any_first = p.window ? at0 - p.window + 1 : 0;

    float o[NT][DH / 16][4], mo[NT][2], ml[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < DH / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) mo[t][x] = ml[t][x] = kNone, l[t][x] = 0.0f;
    }

    // This thread's bytes of row 0 of page 0; pieces behind the head are left out.
    const char* k_mine = static_cast<const char*>(c.k) + kvh * c.ks.h * C::ES + four * 16;
    const char* v_mine = static_cast<const char*>(c.v) + kvh * c.vs.h * C::ES + quad * (C::VW == 2 ? 8 : 16);
    const char* s_mine = reinterpret_cast<const char*>((lane < 16 ? c.k_scale : c.v_scale) + kvh * c.ss.h);
    const bool aligned = c.page_size % kStep == 0;  // a step lies in one page
    auto key_of = [&](int step) { return step < s.head ? step * kStep : s.from + (step - s.head) * kStep; };
    // Where a step's key is: the first one, or where it may lie in several pages key lane % 16.
    auto locate = [&](int step) {
      return step < step1 ? page_row(c, b, key_of(step) + (aligned ? 0 : lane & 15)) : PageRow{-1, 0};
    };
    uint32_t found = 0;  // a bit for each step under way: whether the key is there
    auto issue = [&](int step, int slot, PageRow at) {
      found = found << 1 | (at.page >= 0);
      if (step >= step1) return;
      const int key0 = key_of(step);
      // Keys that some row of the tile sees are read.
      const bool every = key0 + kStep <= any_end && (key0 >= any_first || key0 + kStep <= sinks);
      const uint32_t dst = smem_u32(smem) + (warp * kStages + slot) * C::SLOT;
      auto wanted = [&](int key) {
        const int j = key0 + key;
        return every || (j < any_end && (j >= any_first || j < sinks));
      };
      const int page0 = max(at.page, 0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = quad + 8 * x;
        const int page = aligned ? at.page : __shfl_sync(0xffffffffu, at.page, key);
        const int row = aligned ? at.row + key : __shfl_sync(0xffffffffu, at.row, key);
        const char* src = k_mine + static_cast<uint64_t>(p.kb) * max(page, 0) + static_cast<uint64_t>(p.kl) * row;
        const bool want = page >= 0 && wanted(key);
#pragma unroll
        for (int i = 0; i < C::KP; ++i) {
          const bool in = (four + 4 * i) * 16 < p.dh * C::ES;
          copy16(dst + (x * C::KP + i) * 512 + lane * 16, in ? src + i * 64 : k_mine - four * 16, want && in ? 16 : 0);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = 2 * four + (x & 1) + 8 * (x >> 1);
        const int page = aligned ? at.page : __shfl_sync(0xffffffffu, at.page, key);
        const int row = aligned ? at.row + key : __shfl_sync(0xffffffffu, at.row, key);
        const char* src = v_mine + static_cast<uint64_t>(p.vb) * max(page, 0) + static_cast<uint64_t>(p.vl) * row;
        const bool want = page >= 0 && wanted(key);
        const uint32_t to = dst + C::K_BYTES + x * C::VW * 128;
        if constexpr (C::VW == 2) {
          const bool in = quad * 8 < p.dh * C::ES;
          copy8(to + lane * 8, in ? src : v_mine - quad * 8, want && in ? 8 : 0);
        } else {
#pragma unroll
          for (int i = 0; i < C::VW / 4; ++i) {
            const bool in = (quad + 8 * i) * 16 < p.dh * C::ES;
            copy16(to + i * 512 + lane * 16, in ? src + i * 128 : v_mine - quad * 16, want && in ? 16 : 0);
          }
        }
      }
      if constexpr (C::kScaled) {
        const int row = aligned ? at.row + (lane & 15) : at.row;
        copy4(dst + C::K_BYTES + C::V_BYTES + lane * 4,
              s_mine + static_cast<uint64_t>(p.sb) * page0 + static_cast<uint64_t>(p.sl) * row,
              at.page >= 0 && wanted(lane & 15) ? 4 : 0);
      }
    };

    int step = step0 + warp, slot = 0;
    {
      PageRow at[kStages - 1];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) at[i] = locate(step + i * kWarps);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        issue(step + i * kWarps, i, at[i]);
        copies_commit();
      }
    }
    PageRow next = locate(step + (kStages - 1) * kWarps);
    for (; step < step1; step += kWarps) {
      issue(step + (kStages - 1) * kWarps, slot == 0 ? kStages - 1 : slot - 1, next);
      copies_commit();
      next = locate(step + kStages * kWarps);
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* mine = smem + (warp * kStages + slot) * C::SLOT;
      slot = slot == kStages - 1 ? 0 : slot + 1;
      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::KP; ++i) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(mine + i * 512 + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(mine + (C::KP + i) * 512 + lane * 16);
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
          for (int t = 0; t < NT; ++t) mma<FMT>(sc[t], a, qf[t][i * C::KS + x][0], qf[t][i * C::KS + x][1]);
        }
      }
      float ks[2] = {1.0f, 1.0f}, lv[2] = {0.0f, 0.0f};
      if constexpr (C::kScaled) {
        const float* scales = reinterpret_cast<const float*>(mine + C::K_BYTES + C::V_BYTES);
        ks[0] = scales[quad], ks[1] = scales[quad + 8];
        lv[0] = fast_log2(scales[16 + quad]), lv[1] = fast_log2(scales[24 + quad]);
      }
      // ---- scores and weights' exponents in the log2 domain
      const int key0 = key_of(step);
      float u[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] = (C::kScaled ? sc[t][e] * ks[e >> 1] : sc[t][e]) * up[t][e & 1];
      if (p.softcap > 0) {
        float big = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(sc[t][e]));
        if (__all_sync(0xffffffffu, big * p.cap.inv <= 1.0f)) cap_within<4 * NT>(&sc[0][0], p.cap);
        else cap_any<4 * NT>(&sc[0][0], p.cap);
      }
      const bool whole = (key0 + kStep <= all_end && (key0 >= all_first || key0 + kStep <= sinks)) &&
                         __all_sync(0xffffffffu, found >> (kStages - 1) & 1);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[t][e] = C::kScaled ? sc[t][e] + lv[e >> 1] : sc[t][e];
      unsigned there = 0xffffu;
      if (!whole) {
        there = __ballot_sync(0xffffffffu, found >> (kStages - 1) & 1);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at_key = quad + 8 * (e >> 1), j = key0 + at_key, x = e & 1;
            if (!((there >> at_key) & 1) || j >= end[t][x] || (j < first[t][x] && j >= sinks))
              sc[t][e] = -INFINITY, u[t][e] = -INFINITY;
          }
      }
      // ---- weights; a new maximum is taken up where one passes the old one by far
      float w[NT][4], y[NT][4];
      auto weigh = [&]() {
        float big = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[t][e] = fast_exp2(sc[t][e] - ml[t][e & 1]);
            w[t][e] = C::kScaled ? fast_exp2(u[t][e] - mo[t][e & 1]) : y[t][e];
            big = fmaxf(big, fmaxf(y[t][e], w[t][e]));
          }
        return big;
      };
      if (__any_sync(0xffffffffu, weigh() > kRescale)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float a = fmaxf(sc[t][x], sc[t][2 + x]), d = fmaxf(u[t][x], u[t][2 + x]);
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, i));
              if (C::kScaled) d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, i));
            }
            a = fmaxf(a, ml[t][x]);
            d = C::kScaled ? fmaxf(d, mo[t][x]) : a;
            l[t][x] *= fast_exp2(ml[t][x] - a);
            const float f = fast_exp2(mo[t][x] - d);
            ml[t][x] = a, mo[t][x] = d;
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) o[t][i][x] *= f, o[t][i][2 + x] *= f;
          }
        weigh();
      }
      // ---- transposed into the second product's operand
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) l[t][e & 1] += y[t][e];
        pb[t][0] = movmatrix_t(pack2<kBf16Operands>(w[t][0], w[t][1]));
        pb[t][1] = movmatrix_t(pack2<kBf16Operands>(w[t][2], w[t][3]));
      }
      uint32_t v[4][C::VW];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint8_t* from = mine + C::K_BYTES + x * C::VW * 128;
        if constexpr (C::VW == 2) {
          const uint2 z = *reinterpret_cast<const uint2*>(from + lane * 8);
          v[x][0] = z.x, v[x][1] = z.y;
        } else {
#pragma unroll
          for (int i = 0; i < C::VW / 4; ++i) {
            const uint4 z = *reinterpret_cast<const uint4*>(from + i * 512 + lane * 16);
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
              const int at_row = s.n - s.rows + (r0 + 8 * t + n) / p.G;
              const int row_end = 8 * t + n < n_rows ? (p.causal ? min(at_row + 1, s.keys) : s.keys) : 0;
              const int row_first = p.window ? at_row - p.window + 1 : 0;
              uint32_t see[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int key = 2 * four + (x & 1) + 8 * (x >> 1), j = key0 + key;
                see[x] = ((there >> key) & 1) && j < row_end && (j >= row_first || j < sinks) ? 0xffffffffu : 0u;
              }
#pragma unroll
              for (int i = 0; i < DH / 16; ++i) {
                const uint32_t y[4] = {v[0][i] & see[0], v[1][i] & see[1], v[2][i] & see[2], v[3][i] & see[3]};
                const uint32_t a[4] = {__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                                       __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[2], y[3], 0x7632)};
                float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma<FMT>(z, a, pb[t][0], pb[t][1]);
                if (n == 2 * four) o[t][i][0] += z[0], o[t][i][2] += z[2];
                if (n == 2 * four + 1) o[t][i][1] += z[1], o[t][i][3] += z[3];
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
        for (int t = 0; t < NT; ++t) mma<FMT>(o[t][i], a, pb[t][0], pb[t][1]);
      }
    }

    // ---- join the warps, in the ring's place
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], w);
        const int r = 8 * t + 2 * four + x;
        if (r < n_rows) {
          float* row = so + (warp * ROWS + r) * C::JSTRIDE;
#pragma unroll
          for (int i = 0; i < DH / 16; ++i) {
            // the column pair that this thread's products i belong to
            const int d = C::kScaled ? quad * (DH / 8) + 2 * i : (quad + 8 * (i / 4)) * 8 + 2 * (i % 4);
            *reinterpret_cast<float2*>(row + d) = make_float2(o[t][i][x], o[t][i][2 + x]);
          }
          if (quad == 0) {
            float* st = sm + (warp * ROWS + r) * 4;
            st[0] = mo[t][x], st[1] = ml[t][x], st[2] = l[t][x];
          }
        }
      }
    __syncthreads();
    const bool split = step0 > 0 || step1 < s.steps;
    constexpr int kPart = ROWS * (DH + 4);  // floats of a share: O, then m', m, l of each row
    // a share that begins its group is a CTA's second, one that goes on with it its first
    float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (step0 == 0)) * kPart;
    // Scale, sum and value of a row's shares: finished and written, or left as a share.
    auto write_out = [&](int r, int d, float mm_o, float mm_l, float ll, float4 acc) {
      const int tok = (r0 + r) / p.G, head = kvh * p.G + (r0 + r) % p.G;
      const float f = ll > 0.0f ? fast_exp2(mm_o - mm_l) / ll : ll;  // (0 or NaN)
      if (d < p.dh) {
        const uint2 y = p.bf16 ? make_uint2(pack2<true>(acc.x * f, acc.y * f), pack2<true>(acc.z * f, acc.w * f))
                               : make_uint2(pack2<false>(acc.x * f, acc.y * f), pack2<false>(acc.z * f, acc.w * f));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + b * p.os.b + tok * p.os.l + head * p.os.h + d) = y;
      }
      if (d == 0 && p.lse)
        p.lse[(static_cast<int64_t>(b) * p.Hq + head) * p.Lq + tok] = ll == 0.0f ? -INFINITY : (mm_l + fast_log2(ll)) * kLn2;
    };
    for (int x = threadIdx.x; x < n_rows * (DH / 4); x += kThreads) {
      const int r = x / (DH / 4), d = x % (DH / 4) * 4;
      float mm_o = kNone, mm_l = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mm_o = fmaxf(mm_o, sm[(w * ROWS + r) * 4]);
        mm_l = fmaxf(mm_l, sm[(w * ROWS + r) * 4 + 1]);
      }
      float ll = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* st = sm + (w * ROWS + r) * 4;
        const float4 y = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * C::JSTRIDE + d);
        const float f = fast_exp2(st[0] - mm_o);
        ll = fmaf(fast_exp2(st[1] - mm_l), st[2], ll);
        acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
        acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
      }
      if (split) {
        *reinterpret_cast<float4*>(part + r * DH + d) = acc;
        if (d == 0) {
          float* st = part + ROWS * DH + r * 4;
          st[0] = mm_o, st[1] = mm_l, st[2] = ll;
        }
      } else {
        write_out(r, d, mm_o, mm_l, ll, acc);
      }
    }
    __syncthreads();
    if (split) {
      // The CTAs whose stretches hold the group's first and last step.
      const int64_t g0 = before + static_cast<int64_t>(group) * s.steps, g1 = g0 + s.steps - 1;
      const int c0 = cut.of(g0), c1 = cut.of(g1);
      if (threadIdx.x == 0) {
        __threadfence();
        const int last = atomicAdd(p.arrived + c0, 1) == c1 - c0;
        if (last) p.arrived[c0] = 0;
        __threadfence();
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        for (int x = threadIdx.x; x < n_rows * (DH / 4); x += kThreads) {
          const int r = x / (DH / 4), d = x % (DH / 4) * 4;
          auto share = [&](int cta) { return p.part + (2 * static_cast<int64_t>(cta) + (cta == c0)) * kPart; };
          float mm_o = kNone, mm_l = kNone;
#pragma unroll 4
          for (int cta = c0; cta <= c1; ++cta) {
            const float* st = share(cta) + ROWS * DH + r * 4;
            mm_o = fmaxf(mm_o, __ldcg(st));
            mm_l = fmaxf(mm_l, __ldcg(st + 1));
          }
              float ll = 0.0f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int cta = c0; cta <= c1; ++cta) {
            const float* at_share = share(cta);
            const float4 st = __ldcg(reinterpret_cast<const float4*>(at_share + ROWS * DH + r * 4));
            const float4 y = __ldcg(reinterpret_cast<const float4*>(at_share + r * DH + d));
            const float f = fast_exp2(st.x - mm_o);
            ll = fmaf(fast_exp2(st.y - mm_l), st.z, ll);
            acc.x = fmaf(f, y.x, acc.x), acc.y = fmaf(f, y.y, acc.y);
            acc.z = fmaf(f, y.z, acc.z), acc.w = fmaf(f, y.w, acc.w);
          }
          write_out(r, d, mm_o, mm_l, ll, acc);
        }
      }
    }
    // ---- the next stretch
    lo += step1 - step0;
    if (lo >= hi) break;
    while (lo >= before + s.total) {
      before += s.total;
      s = sequence<ROWS>(p, ++b);
    }
  }
}

template <int DH, int FMT, int NT>
cudaError_t launch(const PageAttnParams& p, int sms, cudaStream_t st) {
  using C = ACfg<DH, FMT, NT>;
  static uint64_t set_up = 0;
  cudaError_t e = once_per_device(&set_up, [](int) {
    return cudaFuncSetAttribute(page_attn_kernel<DH, FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(sms * kCtasSm, kMaxCtas)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_attn_kernel<DH, FMT, NT>, p);
}

template <int DH, int FMT>
cudaError_t launch_rows(const PageAttnParams& p, int sms, cudaStream_t st) {
  return p.Lq * p.G <= 8 ? launch<DH, FMT, 1>(p, sms, st) : launch<DH, FMT, 2>(p, sms, st);
}

template <int DH>
cudaError_t launch_format(const PageAttnParams& p, int sms, cudaStream_t st) {
  switch (p.c.format) {
    case PSV_PAGE_BF16: return launch_rows<DH, PSV_PAGE_BF16>(p, sms, st);
    case PSV_PAGE_F16: return launch_rows<DH, PSV_PAGE_F16>(p, sms, st);
    case PSV_PAGE_E4M3: return launch_rows<DH, PSV_PAGE_E4M3>(p, sms, st);
    default: return launch_rows<DH, PSV_PAGE_I8>(p, sms, st);
  }
}

}  // namespace

// At most two shares a CTA.
size_t page_attn_scratch(const PageAttnParams& p) {
  return PSV_PAGE_SCRATCH_HEAD +
         static_cast<size_t>(kMaxCtas) * 2 * (p.Lq * p.G <= 8 ? 8 : 16) * ((p.dh <= 64 ? 64 : 128) + 4) * sizeof(float);
}

cudaError_t launch_page_attention(const PageAttnParams& p, int sms, cudaStream_t st) {
  return p.dh <= 64 ? launch_format<64>(p, sms, st) : launch_format<128>(p, sms, st);
}

}  // namespace psv

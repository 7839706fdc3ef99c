// Entry points of the paged-cache operators (include/psv.h): argument checks,
// and the kernels that write rows into pages and read them back.  The attention
// over pages is launched from here.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <type_traits>

#include "cache_check.h"
#include "page_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

using namespace psv;

namespace {

bool scaled(int format) { return format == PSV_PAGE_E4M3 || format == PSV_PAGE_I8; }
int page_esize(int format) { return scaled(format) ? 1 : 2; }

// Rows of sequence b: number i of [0, L) at position starts[b] + i.
struct PageRowsParams {
  PageCacheDev c;
  int L, H, dh, lanes;  // lanes of a head's row (log2, at least 2): 8 values each
  int narrow;           // lanes of a row, not a power of two, where rows lie closer in a warp so; or 0
  FastDiv by_narrow;
  int heads, tokens;    // of a thread, at most kRows rows in all
  FastDiv by_groups;    // groups of heads a token (one where there are several tokens)
  Strides3 xs[2];
  void* x[2];  // k, v
  const int32_t *starts, *lens;
};

constexpr float kTiny = 0x1p-100f;  // a row whose largest size is below it is kept as zeros

template <int FMT>
struct PageFormat {
  static constexpr bool kScaled = FMT == PSV_PAGE_E4M3 || FMT == PSV_PAGE_I8;
  static constexpr float kMost = FMT == PSV_PAGE_E4M3 ? 448.0f : 127.0f;
  static constexpr int kSize = kScaled ? 1 : 2;
};

// Four values as they are stored in 8 bits, two in 16, from the lowest bits on.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float* f) {
  if constexpr (FMT == PSV_PAGE_E4M3) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3)) << 16;
  } else {
    // |f| < 2^22: the lowest byte of f + 1.5 2^23 is the nearest whole number, ties to even
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__fadd_rn(f[i], 12582912.0f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  }
}
template <int FMT>
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  if constexpr (FMT == PSV_PAGE_BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t u, float* f) {
  if constexpr (FMT == PSV_PAGE_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> 16 * i), __NV_E4M3);
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * i] = y.x, f[2 * i + 1] = y.y;
    }
  } else {
    // 2^23 + (code + 128) is the f32 whose lowest byte is code + 128
    u ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.0f;
  }
}
template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t u) {
  if constexpr (FMT == PSV_PAGE_BF16)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// The larger of two pairs' sizes (with some sign; NaN where either is one).
template <int FMT>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (FMT == PSV_PAGE_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Eight values of a program's row, as they are in memory.
template <class T>
struct Eight {
  static constexpr int kFmt = sizeof(T) == 2 ? (std::is_same<T, __half>::value ? PSV_PAGE_F16 : PSV_PAGE_BF16) : 0;
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (size_t i = 0; i < sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  __device__ __forceinline__ void load(const T* x, int n) {  // value by value
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) v[i] = x[i];
      else reinterpret_cast<uint16_t*>(&v[i])[0] = 0, reinterpret_cast<uint16_t*>(&v[i])[sizeof(T) / 2 - 1] = 0;
    memcpy(u, v, sizeof(v));
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(T) == 4) {
      memcpy(f, u, 32);
    } else {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = decode2<kFmt>(w[i]);
        f[2 * i] = y.x, f[2 * i + 1] = y.y;
      }
    }
  }
  // Bits of the largest |x| (NaN is above infinity), 16 of them for 16-bit types.
  __device__ __forceinline__ uint32_t size() const {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    if constexpr (sizeof(T) == 4) {
      const uint32_t y[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffffffu, y[i] & 0x7fffffffu));
      return m;
    } else {
      const uint32_t m = larger2<kFmt>(larger2<kFmt>(w[0], w[1]), larger2<kFmt>(w[2], w[3]));
      return max(m & 0x7fffu, m >> 16 & 0x7fffu);
    }
  }
  static __device__ __forceinline__ float size_value(uint32_t bits) {
    if constexpr (kFmt == PSV_PAGE_BF16) return __uint_as_float(bits << 16);
    if constexpr (kFmt == PSV_PAGE_F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    return __uint_as_float(bits);
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (sizeof(T) == 4) {
      memcpy(u, f, 32);
    } else {
      u[0] = make_uint4(encode2<kFmt>(f[0], f[1]), encode2<kFmt>(f[2], f[3]), encode2<kFmt>(f[4], f[5]),
                        encode2<kFmt>(f[6], f[7]));
    }
  }
  __device__ __forceinline__ void store(T* x) const {
#pragma unroll
    for (size_t i = 0; i < sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(x)[i] = u[i];
  }
  __device__ __forceinline__ void store(T* x, int n) const {
    T v[8];
    memcpy(v, u, sizeof(v));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) x[i] = v[i];
  }
};

constexpr int kRowThreads = 256;
constexpr int kRows = 4;

// Whose rows a thread has: up to four heads of a token (kHeads), or where there are one or two
// heads of four or two tokens `step` apart (kTokens).  A row (a head of a token) belongs to
// 2^lanes threads of a warp, eight values each, or (kNarrow) four heads of a token to
// `narrow` threads: three heads of 80 lie side by side in a warp then, not two (8 x 1560
// rows of 40 heads in bf16 to 8 bits 59 us and 47; heads of 128 so 72, and 63 by 2^n lanes).
enum Map { kHeads, kTokens, kNarrow };

template <int MAP>
struct RowMap {
  uint32_t i, step;  // first token
  int h0, heads, lane, first;  // (lane of the row, the row's first one)
  __device__ __forceinline__ explicit RowMap(const PageRowsParams& p) {
    if constexpr (MAP == kTokens) {
      const uint32_t each = kRowThreads >> p.lanes;
      lane = threadIdx.x & ((1 << p.lanes) - 1);
      i = blockIdx.x * each * p.tokens + (threadIdx.x >> p.lanes), step = each;
      h0 = 0, heads = p.H;
    } else {
      uint32_t r, in_warp = 0, row = 0;
      if constexpr (MAP == kNarrow) {
        in_warp = 32 / p.narrow, row = p.by_narrow.div(threadIdx.x % 32);
        first = static_cast<int>(row) * p.narrow;
        lane = static_cast<int>(threadIdx.x % 32) - first;
        r = (blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32) * in_warp + row;
      } else {
        lane = threadIdx.x & ((1 << p.lanes) - 1);
        r = blockIdx.x * (kRowThreads >> p.lanes) + (threadIdx.x >> p.lanes);
      }
      i = p.by_groups.div(r), step = 0;
      h0 = static_cast<int>(r - i * p.by_groups.d) * p.heads;
      heads = min(p.heads, p.H - h0);
      if (MAP == kNarrow && row >= in_warp) i = p.L;  // (lanes that are left over)
    }
  }
  // Token and head of the thread's row k (k < heads x tokens).
  __device__ __forceinline__ uint32_t token(int k) const { return MAP == kTokens ? i + (heads == 1 ? k : k / 2) * step : i; }
  __device__ __forceinline__ int head(int k) const { return MAP != kTokens ? k : heads == 1 ? 0 : k % 2; }
};

// Rows find their largest size by shuffles, and their divisions are made by a lane each.
// grid (tokens x groups of heads, sequence, key or value).  The first reads do not wait
// for the lengths: rows not in use are read too.
// Memory-bound where large: 12480 rows x 40 heads of 128 in f32 to 8 bits 91 us (7.1 TB/s),
// in bf16 63 us (6.2); four sequences of 1560 rows x 12 heads in bf16 13 us.
template <class T, int FMT, bool VEC, int MAP>
__global__ void __launch_bounds__(kRowThreads) page_write_kernel(const __grid_constant__ PageRowsParams p) {
  using F = PageFormat<FMT>;
  const int b = blockIdx.y, kv = blockIdx.z;
  constexpr bool MANY = MAP == kTokens;
  const RowMap<MAP> m(p);
  const int lane = m.lane, d = lane * 8, rows = MANY ? m.heads * p.tokens : m.heads;
  pdl_trigger();
  pdl_wait();
  const Strides3& xs = p.xs[kv];
  Eight<T> in[kRows];
  const T* x = static_cast<const T*>(p.x[kv]) + b * xs.b + m.h0 * xs.h + d;
  if (!MANY) x += m.i * xs.l;
#pragma unroll
  for (int k = 0; k < kRows; ++k, x += MANY ? 0 : xs.h)
    if (k < rows && m.token(k) < static_cast<uint32_t>(p.L) && d < p.dh) {
      const T* from = MANY ? x + m.token(k) * xs.l + m.head(k) * xs.h : x;
      if (VEC) in[k].load(from);
      else in[k].load(from, p.dh - d);
    }
  const int n = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int start = p.starts ? p.starts[b] : 0;
  PageRow at[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (k && (!MANY || m.token(k) == m.token(k - 1))) {
      at[k] = at[k - 1];
      continue;
    }
    at[k] = PageRow{-1, 0};
    if (k < rows && m.token(k) < static_cast<uint32_t>(n)) at[k] = page_row(p.c, b, static_cast<int64_t>(start) + m.token(k));
  }
  float turn[kRows];
  if constexpr (F::kScaled) {
    uint32_t size[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) size[k] = k < rows && m.token(k) < static_cast<uint32_t>(p.L) && d < p.dh ? in[k].size() : 0;
    // (after o = 1, 2, 4, .. a lane has the largest of the 2 o of its row from it on, around)
    auto around = [&](uint32_t x, int o) {
      return __shfl_sync(0xffffffffu, x, m.first + (lane + o < p.narrow ? lane + o : lane + o - p.narrow));
    };
    if constexpr (sizeof(T) == 2) {  // two rows a shuffle
#pragma unroll
      for (int k = 0; k < kRows; k += 2) {
        uint32_t two = size[k] | size[k + 1] << 16;
        if constexpr (MAP == kNarrow) {
          for (int o = 1; o < p.narrow; o *= 2) two = __vmaxu2(two, around(two, o));
        } else {
          for (int o = 1 << p.lanes >> 1; o; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
        }
        size[k] = two & 0xffffu, size[k + 1] = two >> 16;
      }
    } else {
      for (int o = MAP == kNarrow ? 1 : 1 << p.lanes >> 1; MAP == kNarrow ? o < p.narrow : o != 0; o = MAP == kNarrow ? o * 2 : o >> 1)
#pragma unroll
        for (int k = 0; k < kRows; ++k)
          size[k] = max(size[k], MAP == kNarrow ? around(size[k], o) : __shfl_xor_sync(0xffffffffu, size[k], o));
    }
    // Row lane % 4 is this lane's to divide for.
    const int mine = lane % 4;
    const float most = Eight<T>::size_value(mine & 2 ? (mine & 1 ? size[3] : size[2]) : (mine & 1 ? size[1] : size[0]));
    const PageRow to = mine & 2 ? (mine & 1 ? at[3] : at[2]) : (mine & 1 ? at[1] : at[0]);
    const bool finite = __float_as_uint(most) < 0x7f800000u, kept = finite && most >= kTiny;
    const float my_turn = kept ? __fdiv_rn(F::kMost, most) : 0.0f;
#pragma unroll
    for (int k = 0; k < kRows; ++k) turn[k] = MAP == kNarrow ? __shfl_sync(0xffffffffu, my_turn, m.first + k) : __shfl_sync(0xffffffffu, my_turn, k, 1 << p.lanes);
    if (lane < rows && lane < kRows && to.page >= 0)
      (kv ? p.c.v_scale : p.c.k_scale)[to.page * p.c.ss.b + to.row * p.c.ss.l + (m.h0 + m.head(mine)) * p.c.ss.h] =
          kept ? __fdiv_rn(most, F::kMost) : finite ? 0.0f : __int_as_float(0x7fc00000);
  }
  if (d >= p.dh || (!MANY && at[0].page < 0)) return;
  const Strides3& ps = kv ? p.c.vs : p.c.ks;
  char* pages = static_cast<char*>(kv ? p.c.v : p.c.k) + (m.h0 * ps.h + d) * F::kSize;
  if (!MANY) pages += (at[0].page * ps.b + at[0].row * ps.l) * F::kSize;
#pragma unroll
  for (int k = 0; k < kRows; ++k, pages += MANY ? 0 : ps.h * F::kSize) {
    if (k >= rows) break;
    if (MANY && at[k].page < 0) continue;
    char* out = MANY ? pages + (at[k].page * ps.b + at[k].row * ps.l + m.head(k) * ps.h) * F::kSize : pages;
    float f[8];
    in[k].get(f);
    if constexpr (F::kScaled) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= turn[k];
      uint2 y = make_uint2(encode4<FMT>(f), encode4<FMT>(f + 4));
      if (!(turn[k] > 0.0f)) y = make_uint2(0, 0);  // (not the code of 0 * NaN)
      if (VEC) *reinterpret_cast<uint2*>(out) = y;
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (d + j < p.dh) out[j] = static_cast<char>((j < 4 ? y.x : y.y) >> 8 * (j % 4));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = encode2<FMT>(f[2 * j], f[2 * j + 1]);
      if (VEC) *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (d + j < p.dh) reinterpret_cast<uint16_t*>(out)[j] = static_cast<uint16_t>(w[j / 2] >> 16 * (j % 2));
    }
  }
}

// The same threads read rows back; positions without a page read as zeros.  Memory-bound:
// eight sequences of 4836 rows x 40 heads of 128 from 8 bits 177 us (6.8 TB/s).
template <class T, int FMT, bool VEC, int MAP>
__global__ void __launch_bounds__(kRowThreads) page_read_kernel(const __grid_constant__ PageRowsParams p) {
  using F = PageFormat<FMT>;
  const int b = blockIdx.y, kv = blockIdx.z;
  constexpr bool MANY = MAP == kTokens;
  const RowMap<MAP> m(p);
  const int d = m.lane * 8, rows = MANY ? m.heads * p.tokens : m.heads;
  pdl_trigger();
  pdl_wait();
  const int n = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  if (d >= p.dh || m.i >= static_cast<uint32_t>(n)) return;
  const int start = p.starts ? p.starts[b] : 0;
  PageRow at[kRows];
#pragma unroll
  for (int k = 0; k < (MANY ? kRows : 1); ++k) {
    if (k && m.token(k) == m.token(k - 1)) {
      at[k] = at[k - 1];
      continue;
    }
    at[k] = PageRow{-1, 0};
    if (k < rows && m.token(k) < static_cast<uint32_t>(n)) at[k] = page_row(p.c, b, static_cast<int64_t>(start) + m.token(k));
  }
  const Strides3& ps = kv ? p.c.vs : p.c.ks;
  const char* pages = static_cast<const char*>(kv ? p.c.v : p.c.k) + (m.h0 * ps.h + d) * F::kSize;
  const float* scales = (kv ? p.c.v_scale : p.c.k_scale) + (F::kScaled ? m.h0 * p.c.ss.h : 0);
  uint32_t w[kRows][4] = {};
  float s[kRows] = {};
  if (!MANY && at[0].page >= 0) {
    pages += (at[0].page * ps.b + at[0].row * ps.l) * F::kSize;
    if (F::kScaled) scales += at[0].page * p.c.ss.b + at[0].row * p.c.ss.l;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k, pages += MANY ? 0 : ps.h * F::kSize) {
    if (k >= rows || (!MANY && at[0].page < 0)) break;
    if (MANY && at[k].page < 0) continue;
    const char* in = MANY ? pages + (at[k].page * ps.b + at[k].row * ps.l + m.head(k) * ps.h) * F::kSize : pages;
    if constexpr (F::kScaled) {
      s[k] = MANY ? scales[at[k].page * p.c.ss.b + at[k].row * p.c.ss.l + m.head(k) * p.c.ss.h] : scales[k * p.c.ss.h];
      if (VEC) {
        const uint2 y = *reinterpret_cast<const uint2*>(in);
        w[k][0] = y.x, w[k][1] = y.y;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (d + j < p.dh) w[k][j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(in[j])) << 8 * (j % 4);
      }
    } else if (VEC) {
      const uint4 y = *reinterpret_cast<const uint4*>(in);
      w[k][0] = y.x, w[k][1] = y.y, w[k][2] = y.z, w[k][3] = y.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (d + j < p.dh)
          w[k][j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(in)[j]) << 16 * (j % 2);
    }
  }
  T* x = static_cast<T*>(p.x[kv]) + b * p.xs[kv].b + m.h0 * p.xs[kv].h + d;
  if (!MANY) x += m.i * p.xs[kv].l;
#pragma unroll
  for (int k = 0; k < kRows; ++k, x += MANY ? 0 : p.xs[kv].h) {
    if (k >= rows || (MANY && m.token(k) >= static_cast<uint32_t>(n))) break;
    float f[8];
    if constexpr (F::kScaled) {
      decode4<FMT>(w[k][0], f);
      decode4<FMT>(w[k][1], f + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s[k];
      if (at[MANY ? k : 0].page < 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.0f;  // (not the codes' -128 * 0)
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = decode2<FMT>(w[k][j]);
        f[2 * j] = y.x, f[2 * j + 1] = y.y;
      }
    }
    Eight<T> out;
    out.set(f);
    T* to = MANY ? x + m.token(k) * p.xs[kv].l + m.head(k) * p.xs[kv].h : x;
    if (VEC) out.store(to);
    else out.store(to, p.dh - d);
  }
}

template <class T, int FMT>
cudaError_t launch_page_rows(const PageRowsParams& p, int B, bool vec, bool write, cudaStream_t st) {
  const uint32_t groups = static_cast<uint32_t>(p.L) * p.by_groups.d;
  const uint32_t each = p.narrow ? kRowThreads / 32 * (32 / p.narrow) : (kRowThreads >> p.lanes) * p.tokens;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((groups + each - 1) / each, B, 2), kRowThreads, 0, st, attr);
  if (write) {
    if (!vec) return cudaLaunchKernelEx(&cfg, page_write_kernel<T, FMT, false, kHeads>, p);
    return p.narrow       ? cudaLaunchKernelEx(&cfg, page_write_kernel<T, FMT, true, kNarrow>, p)
           : p.tokens > 1 ? cudaLaunchKernelEx(&cfg, page_write_kernel<T, FMT, true, kTokens>, p)
                          : cudaLaunchKernelEx(&cfg, page_write_kernel<T, FMT, true, kHeads>, p);
  }
  if (!vec) return cudaLaunchKernelEx(&cfg, page_read_kernel<T, FMT, false, kHeads>, p);
  return p.narrow       ? cudaLaunchKernelEx(&cfg, page_read_kernel<T, FMT, true, kNarrow>, p)
         : p.tokens > 1 ? cudaLaunchKernelEx(&cfg, page_read_kernel<T, FMT, true, kTokens>, p)
                        : cudaLaunchKernelEx(&cfg, page_read_kernel<T, FMT, true, kHeads>, p);
}

template <class T>
cudaError_t launch_page_rows_any(const PageRowsParams& p, int B, bool vec, bool write, cudaStream_t st) {
  switch (p.c.format) {
    case PSV_PAGE_E4M3: return launch_page_rows<T, PSV_PAGE_E4M3>(p, B, vec, write, st);
    case PSV_PAGE_I8: return launch_page_rows<T, PSV_PAGE_I8>(p, B, vec, write, st);
    case PSV_PAGE_BF16:
      if constexpr (!std::is_same<T, __half>::value) return launch_page_rows<T, PSV_PAGE_BF16>(p, B, vec, write, st);
      break;
    default:
      if constexpr (!std::is_same<T, __nv_bfloat16>::value) return launch_page_rows<T, PSV_PAGE_F16>(p, B, vec, write, st);
  }
  return cudaErrorInvalidValue;  // (refused before)
}

// ---------------------------------------------------------------- checks

// A tensor's reach in bytes, in a type that cannot overflow; false if it is none
// that an address space holds.
bool reach_ok(const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t width, int size) {
  const double reach = (static_cast<double>(s[0]) * (n0 - 1) + static_cast<double>(s[1]) * (n1 - 1) +
                        static_cast<double>(s[2]) * (n2 - 1) + width) * size;
  return reach < 0x1p56;
}

int check_page_cache(const psv_page_cache* c) {
  if (!c) return cache_fail(PSV_EINVAL, "null cache");
  if (c->format < PSV_PAGE_BF16 || c->format > PSV_PAGE_I8) return cache_fail(PSV_EINVAL, "unknown page format %d", c->format);
  if (c->B < 1 || c->B > 65535 || c->Hkv < 1) return cache_fail(PSV_EINVAL, "need B of 1 to 65535 and Hkv >= 1");
  if (c->dh < 1 || c->dh > 256) return cache_fail(PSV_EINVAL, "dh %d: 1 to 256", c->dh);
  if (c->n_pages < 1 || c->page_size < 1 || c->max_pages < 1)
    return cache_fail(PSV_EINVAL, "need n_pages, page_size, max_pages >= 1");
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (1 << 30))
    return cache_fail(PSV_EINVAL, "the table covers over 2^30 positions");
  if (static_cast<int64_t>(c->B) * c->Hkv > (1 << 24)) return cache_fail(PSV_EINVAL, "over 2^24 sequences x heads");
  if (!stride_ok(c->k_stride, 3) || !stride_ok(c->v_stride, 3) || !stride_ok(&c->table_stride, 1) ||
      (scaled(c->format) && !stride_ok(c->scale_stride, 3)))
    return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  const int size = page_esize(c->format);
  if (!reach_ok(c->k_stride, c->n_pages, c->page_size, c->Hkv, c->dh, size) ||
      !reach_ok(c->v_stride, c->n_pages, c->page_size, c->Hkv, c->dh, size) ||
      (scaled(c->format) && !reach_ok(c->scale_stride, c->n_pages, c->page_size, c->Hkv, 1, 4)))
    return cache_fail(PSV_EINVAL, "the pages reach over 2^56 bytes");
  if (!c->k_pages || !c->v_pages || !c->table || (scaled(c->format) && (!c->k_scales || !c->v_scales)))
    return cache_fail(PSV_EINVAL, "null pointer");
  if ((reinterpret_cast<uintptr_t>(c->k_pages) | reinterpret_cast<uintptr_t>(c->v_pages)) & (size - 1))
    return cache_fail(PSV_EINVAL, "pages must be aligned to their type");
  if (!on4({c->table, scaled(c->format) ? c->k_scales : nullptr, scaled(c->format) ? c->v_scales : nullptr}))
    return cache_fail(PSV_EINVAL, "tables and scales must be aligned to 4 bytes");
  return PSV_OK;
}

PageCacheDev page_cache_dev(const psv_page_cache* c) {
  PageCacheDev d{};
  d.format = c->format, d.n_pages = c->n_pages, d.page_size = c->page_size;
  d.positions = c->max_pages * c->page_size;
  d.by_page = FastDiv::of(static_cast<uint32_t>(c->page_size));
  d.ks = strides3(c->k_stride), d.vs = strides3(c->v_stride), d.ss = strides3(c->scale_stride);
  d.table = c->table, d.table_b = c->table_stride;
  d.k = c->k_pages, d.v = c->v_pages, d.k_scale = c->k_scales, d.v_scale = c->v_scales;
  return d;
}

// The bytes of a cache's parts.
struct PageAreas {
  Area k, v, ks, vs, table;
  explicit PageAreas(const psv_page_cache* c) {
    const int size = page_esize(c->format);
    k = tensor_area("k_pages", c->k_pages, c->k_stride, c->n_pages, c->page_size, c->Hkv, c->dh, size);
    v = tensor_area("v_pages", c->v_pages, c->v_stride, c->n_pages, c->page_size, c->Hkv, c->dh, size);
    auto scales = [&](const char* name, const void* at) {
      return scaled(c->format) ? tensor_area(name, at, c->scale_stride, c->n_pages, c->page_size, c->Hkv, 1, 4)
                               : plain_area(name, nullptr, 0);
    };
    ks = scales("k_scales", c->k_scales), vs = scales("v_scales", c->v_scales);
    const int64_t st[3] = {c->table_stride, 0, 0};
    table = tensor_area("table", c->table, st, c->B, 1, 1, c->max_pages, 4);
  }
};

int page_rows_call(const psv_page_cache* c, const psv_page_rows* r, const void* k, const void* v, bool write,
                   void* cuda_stream) {
  if (int e = check_page_cache(c)) return e;
  if (!r) return cache_fail(PSV_EINVAL, "null rows");
  const int size = dtype_size(r->dtype);
  if (!size) return cache_fail(PSV_EINVAL, "unknown dtype %d", r->dtype);
  if ((c->format == PSV_PAGE_BF16 && r->dtype == PSV_DTYPE_F16) || (c->format == PSV_PAGE_F16 && r->dtype == PSV_DTYPE_BF16))
    return cache_fail(PSV_EINVAL, "rows of one 16-bit type, pages of the other");
  if (r->L < 0 || static_cast<int64_t>(r->L) * c->Hkv > (1 << 30))
    return cache_fail(PSV_EINVAL, "L %d: not negative, L x Hkv at most 2^30", r->L);
  if (!stride_ok(r->k_stride, 3) || !stride_ok(r->v_stride, 3)) return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  if (r->L == 0) return PSV_OK;
  if (!reach_ok(r->k_stride, c->B, r->L, c->Hkv, c->dh, size) || !reach_ok(r->v_stride, c->B, r->L, c->Hkv, c->dh, size))
    return cache_fail(PSV_EINVAL, "the rows reach over 2^56 bytes");
  if (write) {
    const int pages[3] = {c->n_pages, c->page_size, c->Hkv};
    if (!rows_distinct(c->k_stride, pages[0], pages[1], pages[2], c->dh) ||
        !rows_distinct(c->v_stride, pages[0], pages[1], pages[2], c->dh) ||
        (scaled(c->format) && !rows_distinct(c->scale_stride, pages[0], pages[1], pages[2], 1)))
      return cache_fail(PSV_EINVAL, "the pages' rows overlap");
  } else if (!rows_distinct(r->k_stride, c->B, r->L, c->Hkv, c->dh) || !rows_distinct(r->v_stride, c->B, r->L, c->Hkv, c->dh)) {
    return cache_fail(PSV_EINVAL, "the rows of k or v overlap");
  }
  if (!k || !v) return cache_fail(PSV_EINVAL, "null pointer");
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & (size - 1))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  if (!on4({r->starts, r->lens})) return cache_fail(PSV_EINVAL, "starts and lengths must be aligned to 4 bytes");
  const PageAreas a(c);
  const Area ka = tensor_area("k", k, r->k_stride, c->B, r->L, c->Hkv, c->dh, size);
  const Area va = tensor_area("v", v, r->v_stride, c->B, r->L, c->Hkv, c->dh, size);
  const Area starts = plain_area("starts", r->starts, c->B * int64_t{4}), lens = plain_area("lens", r->lens, c->B * int64_t{4});
  if (int e = write ? check_areas({a.k, a.v, a.ks, a.vs}, {ka, va, a.table, starts, lens})
                    : check_areas({ka, va}, {a.k, a.v, a.ks, a.vs, a.table, starts, lens}))
    return e;
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return e;
  if (int e = check_device(dev, k, "k")) return e;
  if (int e = check_device(dev, c->k_pages, "k_pages")) return e;
  PageRowsParams p{};
  p.c = page_cache_dev(c);
  p.L = r->L, p.H = c->Hkv, p.dh = c->dh;
  p.lanes = 2;
  while (8 << p.lanes < c->dh) ++p.lanes;
  const int groups = (c->Hkv + kRows - 1) / kRows;
  p.heads = (c->Hkv + groups - 1) / groups;
  p.by_groups = FastDiv::of(static_cast<uint32_t>(groups));
  p.xs[0] = strides3(r->k_stride), p.xs[1] = strides3(r->v_stride);
  p.x[0] = const_cast<void*>(k), p.x[1] = const_cast<void*>(v);
  p.starts = r->starts, p.lens = r->lens;
  const int es = page_esize(c->format);
  auto eights = [&](const void* at, const int64_t* s) {  // eight stored values as one access
    return multiple_of(8 * es, at, s, c->n_pages, c->page_size, c->Hkv, es);
  };
  const bool vec = c->dh % 8 == 0 && multiple16(k, r->k_stride, c->B, r->L, c->Hkv, size) &&
                   multiple16(v, r->v_stride, c->B, r->L, c->Hkv, size) && eights(c->k_pages, c->k_stride) &&
                   eights(c->v_pages, c->v_stride);
  p.tokens = !vec ? 1 : c->Hkv == 1 ? 4 : c->Hkv == 2 ? 2 : 1;
  const int lanes = c->dh / 8;
  if (vec && p.tokens == 1 && lanes >= 4 && 32 / lanes > 32 >> p.lanes) {
    p.narrow = lanes;
    p.by_narrow = FastDiv::of(static_cast<uint32_t>(lanes));
  }
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = r->dtype == PSV_DTYPE_F32    ? launch_page_rows_any<float>(p, c->B, vec, write, st)
                        : r->dtype == PSV_DTYPE_BF16 ? launch_page_rows_any<__nv_bfloat16>(p, c->B, vec, write, st)
                                                     : launch_page_rows_any<__half>(p, c->B, vec, write, st);
  return cuda_status(e, write ? "page write launch" : "page read launch");
}

int check_page_query(const psv_page_cache* c, const psv_page_query* q) {
  if (int e = check_page_cache(c)) return e;
  if (!q) return cache_fail(PSV_EINVAL, "null query");
  if (q->dtype != PSV_DTYPE_BF16 && q->dtype != PSV_DTYPE_F16) return cache_fail(PSV_EINVAL, "dtype %d: bf16 or f16", q->dtype);
  if ((c->format == PSV_PAGE_BF16 && q->dtype == PSV_DTYPE_F16) || (c->format == PSV_PAGE_F16 && q->dtype == PSV_DTYPE_BF16))
    return cache_fail(PSV_EINVAL, "queries of one 16-bit type, pages of the other");
  if (q->Hq < 1 || q->Hq % c->Hkv) return cache_fail(PSV_EINVAL, "Hq (%d) must be a multiple of Hkv (%d)", q->Hq, c->Hkv);
  if (q->Lq < 0 || q->Lq > (1 << 20)) return cache_fail(PSV_EINVAL, "Lq %d: 0 to 2^20", q->Lq);
  if (static_cast<int64_t>(c->B) * q->Hq > (1 << 24)) return cache_fail(PSV_EINVAL, "over 2^24 sequences x heads");
  if (static_cast<double>(c->B) * q->Lq * q->Hq > 0x1p30) return cache_fail(PSV_EINVAL, "B x Lq x Hq over 2^30");
  if (q->window < 0 || q->sinks < 0) return cache_fail(PSV_EINVAL, "window and sinks must not be negative");
  if (q->sinks && !q->window) return cache_fail(PSV_EINVAL, "sinks need a window");
  if (!(std::isfinite(q->scale) && q->scale >= 0)) return cache_fail(PSV_EINVAL, "scale must be finite and not negative");
  if (!(std::isfinite(q->softcap) && q->softcap >= 0)) return cache_fail(PSV_EINVAL, "softcap must be finite and not negative");
  if (!stride_ok(q->q_stride, 3) || !stride_ok(q->o_stride, 3)) return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  if (q->Lq && (!reach_ok(q->q_stride, c->B, q->Lq, q->Hq, c->dh, 2) || !reach_ok(q->o_stride, c->B, q->Lq, q->Hq, c->dh, 2)))
    return cache_fail(PSV_EINVAL, "the rows reach over 2^56 bytes");
  if (!on4({q->q_lens, q->k_lens})) return cache_fail(PSV_EINVAL, "lengths must be aligned to 4 bytes");
  return PSV_OK;
}

PageAttnParams page_attn_params(const psv_page_cache* c, const psv_page_query* q) {
  PageAttnParams p{};
  p.c = page_cache_dev(c);
  p.B = c->B, p.Hq = q->Hq, p.Hkv = c->Hkv, p.G = q->Hq / c->Hkv, p.dh = c->dh, p.Lq = q->Lq;
  // (a window over every position that rows may stand at is none)
  const int most = (1 << 30) + (1 << 21);
  p.causal = q->causal != 0, p.append = q->append != 0;
  p.window = q->window < most ? q->window : most, p.sinks = q->sinks;
  p.bf16 = q->dtype == PSV_DTYPE_BF16;
  p.scale = q->scale > 0 ? q->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c->dh)));
  p.softcap = q->softcap;
  p.qs = strides3(q->q_stride), p.os = strides3(q->o_stride);
  p.q_lens = q->q_lens, p.k_lens = q->k_lens;
  return p;
}

// Whether heads are made of eight values each, for the tensor-core kernel.
bool page_attn_pieces(const psv_page_cache* c) { return c->dh % 8 == 0; }

size_t page_scratch(const psv_page_cache* c, const PageAttnParams& p) {
  return page_attn_pieces(c) ? page_attn_scratch(p) : 256;
}

}  // namespace

PSV_API int psv_page_write(const psv_page_cache* c, const psv_page_rows* r, const void* k, const void* v,
                           void* cuda_stream) {
  return page_rows_call(c, r, k, v, true, cuda_stream);
}

PSV_API int psv_page_read(const psv_page_cache* c, const psv_page_rows* r, void* k, void* v, void* cuda_stream) {
  return page_rows_call(c, r, k, v, false, cuda_stream);
}

PSV_API int psv_page_scratch_bytes(const psv_page_cache* c, const psv_page_query* q, size_t* bytes) {
  if (int e = check_page_query(c, q)) return e;
  if (!bytes) return cache_fail(PSV_EINVAL, "null pointer");
  *bytes = page_scratch(c, page_attn_params(c, q));
  return PSV_OK;
}

PSV_API int psv_page_attention(const psv_page_cache* c, const psv_page_query* q, const void* x, void* o, float* lse,
                               void* scratch, size_t scratch_bytes, void* cuda_stream) {
  if (int e = check_page_query(c, q)) return e;
  if (q->Lq == 0) return PSV_OK;
  if (!rows_distinct(q->o_stride, c->B, q->Lq, q->Hq, c->dh)) return cache_fail(PSV_EINVAL, "o's rows overlap");
  if (!x || !o || !scratch) return cache_fail(PSV_EINVAL, "null pointer");
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(o)) & 1) || (reinterpret_cast<uintptr_t>(lse) & 3))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  PageAttnParams p = page_attn_params(c, q);
  const size_t need = page_scratch(c, p);
  if (reinterpret_cast<uintptr_t>(scratch) & 255) return cache_fail(PSV_EINVAL, "scratch must be 256-byte aligned");
  if (scratch_bytes < need) return cache_fail(PSV_EINVAL, "scratch of %zu bytes, %zu needed", scratch_bytes, need);
  const bool in_place = x == o && same_rows(q->q_stride, q->o_stride, c->B, q->Lq, q->Hq);
  const PageAreas a(c);
  if (int e = check_areas(
          {tensor_area("o", o, q->o_stride, c->B, q->Lq, q->Hq, c->dh, 2),
           plain_area("lse", lse, static_cast<int64_t>(c->B) * q->Hq * q->Lq * 4), plain_area("scratch", scratch, need)},
          {in_place ? plain_area("", nullptr, 0) : tensor_area("q", x, q->q_stride, c->B, q->Lq, q->Hq, c->dh, 2), a.k, a.v,
           a.ks, a.vs, a.table, plain_area("q_lens", q->q_lens, c->B * int64_t{4}),
           plain_area("k_lens", q->k_lens, c->B * int64_t{4})}))
    return e;
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return e;
  if (int e = check_device(dev, x, "q")) return e;
  if (int e = check_device(dev, o, "o")) return e;
  p.q = x, p.o = o, p.lse = lse;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int es = page_esize(c->format);
  auto small = [](const int64_t* st, int size) { return st[0] * size < int64_t{1} << 32 && st[1] * size < int64_t{1} << 32; };
  if (page_attn_pieces(c) && small(c->k_stride, es) && small(c->v_stride, es) &&
      (es == 2 || small(c->scale_stride, 4)) && multiple16(x, q->q_stride, c->B, q->Lq, q->Hq, 2) &&
      multiple16(o, q->o_stride, c->B, q->Lq, q->Hq, 2) &&
      multiple_of(es * 8, c->k_pages, c->k_stride, c->n_pages, c->page_size, c->Hkv, es) &&
      multiple_of(es * 8, c->v_pages, c->v_stride, c->n_pages, c->page_size, c->Hkv, es)) {
    p.halves = !(c->dh * es % 16 == 0 && multiple16(c->k_pages, c->k_stride, c->n_pages, c->page_size, c->Hkv, es) &&
                 multiple16(c->v_pages, c->v_stride, c->n_pages, c->page_size, c->Hkv, es));
    int sms = 0;
    if (int e = cuda_status(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "device")) return e;
    if (p.softcap > 0) set_cap_form(p.cap, p.scale, p.softcap);
    p.by_group = FastDiv::of(static_cast<uint32_t>(p.G));
    p.kb = static_cast<uint32_t>(c->k_stride[0] * es), p.kl = static_cast<uint32_t>(c->k_stride[1] * es);
    p.vb = static_cast<uint32_t>(c->v_stride[0] * es), p.vl = static_cast<uint32_t>(c->v_stride[1] * es);
    p.sb = static_cast<uint32_t>(c->scale_stride[0] * 4), p.sl = static_cast<uint32_t>(c->scale_stride[1] * 4);
    page_attn_scratch(p, scratch);
    return cuda_status(launch_page_attention(p, sms, st), "page attention launch");
  }
  return cuda_status(launch_page_attention_general(p, st), "page attention launch");
}

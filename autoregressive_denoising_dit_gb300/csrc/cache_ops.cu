// Entry points of the rolling-cache operators (include/psv.h): argument
// checks, rotary positions with several axes, and eviction.  The attention
// over a cache and the attention mass are launched from here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/psv.h"
#include "cache_check.h"
#include "cache_kernels.h"
#include "psv_device.cuh"
#include "psv_kernels.h"

namespace psv {

static thread_local char t_cache_error[256];

int cache_fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_cache_error, sizeof(t_cache_error), fmt, ap);
  va_end(ap);
  return code;
}

}  // namespace psv

using namespace psv;

namespace {

// ------------------------------------------------------------------ rope

constexpr int kMaxPairs = 128;

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* pos;
  const int32_t* lens;
  Strides3 xs, os;
  int64_t pos_b, pos_l;
  uint32_t n;            // threads of a sequence: rows x units x head groups
  int B, L, H, dh, R;
  int units;             // units of a head: vectors (PAIRS) or vector pairs (HALVES), then copies
  int rot_units;         // HALVES: the units that rotate
  int hpt, hgroups;      // heads per thread
  int inverse;
  uint64_t turn[kMaxPairs];  // f_p / 2 pi in 64-bit fixed point: turns per position, mod 1
  uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }

// N values: 16 bytes as one access, fewer value by value (they need not be
// aligned to more than one value).
template <class T, int N>
struct Vec {
  static constexpr bool kWide = N * sizeof(T) == 16;
  alignas(kWide ? 16 : sizeof(T)) T v[N];
  __device__ __forceinline__ void load(const T* x) {
    if constexpr (kWide) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = x[i];
    }
  }
  __device__ __forceinline__ void store(T* x) const {
    if constexpr (kWide) {
      *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = v[i];
    }
  }
};

// (cos, sin) of pos * f_p.  pos * turn wraps modulo one turn in 64 bits, so
// the angle is off by at most |pos| 2^-53 f_p (and 2^-64 turns a position)
// whatever the position; of the signed fraction in [-1/2, 1/2) turns 24 bits are
// used (f32's: 9.4e-8 radians at half a turn, less towards zero).
__device__ __forceinline__ float2 pair_angle(const RopeParams& p, int pair, int b, int64_t l) {
  if (2 * pair >= p.R) return make_float2(1.0f, 0.0f);
  const int pos = p.pos[b * p.pos_b + l * p.pos_l + p.axis[pair]];
  const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turn[pair];
  const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, p.inverse ? -s : s);
}

// A thread holds one unit (VEC values of a head, or for HALVES VEC values and
// their partners R/2 further on) of a row, computes its angles once and
// applies them to hpt heads, kFlight at a time.  Memory-bound where large: one
// read and one write of x (12480 rows x 40 heads of 128 in f32 93 us, 5.5 TB/s).
// Four sequences of 1560 rows x 12 heads in bf16 (38 MB) take 12.1 us, of which the
// launch is 4: a thread's 12 heads are three rounds of loads, one after another.
template <class T, int VEC, bool HALVES>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams p) {
  using V = Vec<T, VEC>;
  // (32-bit divisions: 64-bit ones cost more than the rotation.)
  const uint32_t t = blockIdx.x * 256 + threadIdx.x;
  if (t >= p.n) return;
  const uint32_t units = p.units, hgroups = p.hgroups, rest = t / units;
  const int u = static_cast<int>(t - rest * units);
  const int hg = static_cast<int>(rest % hgroups);
  const int b = blockIdx.y;
  const int64_t l = rest / hgroups;
  pdl_trigger();
  pdl_wait();
  if (p.lens && l >= p.lens[b]) return;
  const bool rot = !HALVES || u < p.rot_units;
  // Values [d0, d0 + VEC); HALVES: partners at d0 + R/2.
  const int d0 = HALVES && !rot ? p.R + (u - p.rot_units) * VEC : u * VEC;
  const T* x = static_cast<const T*>(p.x) + b * p.xs.b + l * p.xs.l + d0;
  T* o = static_cast<T*>(p.out) + b * p.os.b + l * p.os.l + d0;
  // kFlight heads' loads are on their way at a time, the first ones while the
  // angles are computed.
  constexpr int kFlight = 4;
  const int h1 = min(p.H, (hg + 1) * p.hpt);
  V a[kFlight], c[HALVES ? kFlight : 1];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (h0 + k < h1) {
        a[k].load(x + (h0 + k) * p.xs.h);
        if constexpr (HALVES)
          if (rot) c[k].load(x + (h0 + k) * p.xs.h + p.R / 2);
      }
  };
  load(hg * p.hpt);
  constexpr int PR = HALVES ? VEC : (VEC + 1) / 2;  // pairs of a unit
  float2 cs[PR];
#pragma unroll
  for (int i = 0; i < PR; ++i)
    cs[i] = pair_angle(p, HALVES ? (rot ? d0 + i : p.R) : d0 / 2 + i, b, l);
  for (int h0 = hg * p.hpt; h0 < h1; h0 += kFlight) {
    if (h0 != hg * p.hpt) load(h0);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (h0 + k < h1) {
        if constexpr (HALVES) {
          if (rot) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const float f = to_f(a[k].v[i]), g = to_f(c[k].v[i]);
              from_f(a[k].v[i], f * cs[i].x - g * cs[i].y);
              from_f(c[k].v[i], f * cs[i].y + g * cs[i].x);
            }
            c[k].store(o + (h0 + k) * p.os.h + p.R / 2);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            if (2 * (d0 / 2 + i) < p.R) {  // values behind R are copied bit for bit
              const float f = to_f(a[k].v[2 * i]), g = to_f(a[k].v[2 * i + 1]);
              from_f(a[k].v[2 * i], f * cs[i].x - g * cs[i].y);
              from_f(a[k].v[2 * i + 1], f * cs[i].y + g * cs[i].x);
            }
          }
        }
        a[k].store(o + (h0 + k) * p.os.h);
      }
    }
  }
}

// f / 2 pi as 64-bit fixed-point turns modulo one turn.
uint64_t fixed_turns(double f) {
  // (Of a small negative t, t - floor(t) would keep 2^-54 only: 1e-6 radians at 2^31.)
  if (f < 0) return 0 - fixed_turns(-f);
  const double hi = 0.15915494309189535, lo = -9.839338337591997e-18;  // 1 / (2 pi)
  const double t = f * hi;
  const double e = std::fma(f, hi, -t) + f * lo;
  const double fr = t - std::floor(t);
  // fr < 1 holds 53 bits; the remainder e adds the bits behind them.
  const double scaled = fr * 0x1p64;
  const uint64_t base = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  return base + static_cast<uint64_t>(static_cast<int64_t>(e * 0x1p64));
}

template <class T, bool HALVES>
cudaError_t launch_rope_t(RopeParams& p, bool vec, cudaStream_t st) {
  constexpr int N = 16 / sizeof(T);
  const int V = vec ? N : (HALVES ? 1 : 2);
  if (HALVES) {
    p.rot_units = p.R / 2 / V;
    p.units = p.rot_units + (p.dh - p.R) / V;
  } else {
    p.units = p.dh / V;
  }
  p.n = static_cast<uint32_t>(p.L) * p.units * p.hgroups;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((p.n + 255) / 256, p.B), 256, 0, st, attr);
  return vec ? cudaLaunchKernelEx(&cfg, rope_kernel<T, N, HALVES>, p)
             : cudaLaunchKernelEx(&cfg, rope_kernel<T, HALVES ? 1 : 2, HALVES>, p);
}

}  // namespace

PSV_API const char* psv_cache_last_error(void) { return psv::t_cache_error; }

PSV_API int psv_rope(const psv_rope_problem* p, const void* x, const int32_t* pos, void* out,
                     void* cuda_stream) {
  if (!p) return cache_fail(PSV_EINVAL, "null problem");
  const int size = dtype_size(p->dtype);
  if (!size) return cache_fail(PSV_EINVAL, "unknown dtype %d", p->dtype);
  if (p->B < 1 || p->L < 1 || p->H < 1) return cache_fail(PSV_EINVAL, "need B, L, H >= 1");
  // (A thread takes at least one of a head's at most 256 values, and is numbered in 32 bits.)
  if (p->B > 65535 || static_cast<int64_t>(p->L) * p->H * 256 > 0xffffff00ll)
    return cache_fail(PSV_EINVAL, "B over 65535, or L x H not below 2^24");
  if (p->dh < 2 || p->dh > 256 || p->dh % 2) return cache_fail(PSV_EINVAL, "dh %d: even, 2 to 256", p->dh);
  if (p->n_axes < 1 || p->n_axes > 4) return cache_fail(PSV_EINVAL, "n_axes %d: 1 to 4", p->n_axes);
  if (p->layout != PSV_ROPE_PAIRS && p->layout != PSV_ROPE_HALVES)
    return cache_fail(PSV_EINVAL, "unknown layout %d", p->layout);
  int R = 0;
  for (int a = 0; a < p->n_axes; ++a) {
    if (p->axis_dims[a] < 2 || p->axis_dims[a] % 2 || p->axis_dims[a] > 256)
      return cache_fail(PSV_EINVAL, "axis_dims[%d] = %d: even and positive", a, p->axis_dims[a]);
    R += p->axis_dims[a];
  }
  if (R > p->dh) return cache_fail(PSV_EINVAL, "the axes rotate %d values of dh = %d", R, p->dh);
  if (!p->freqs && !(std::isfinite(p->theta) && p->theta > 0))
    return cache_fail(PSV_EINVAL, "theta must be positive and finite");
  if (!stride_ok(p->x_stride, 3) || !stride_ok(p->out_stride, 3) || !stride_ok(p->pos_stride, 2))
    return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  if (!rows_distinct(p->out_stride, p->B, p->L, p->H, p->dh))
    return cache_fail(PSV_EINVAL, "out's rows overlap");
  RopeParams k{};
  const double log_theta = p->freqs ? 0.0 : std::log2(p->theta);
  int pair = 0;
  for (int a = 0; a < p->n_axes; ++a)
    for (int j = 0; j < p->axis_dims[a] / 2; ++j, ++pair) {
      const double f = p->freqs ? p->freqs[pair] : std::exp2(log_theta * (-2.0 * j / p->axis_dims[a]));
      if (!std::isfinite(f)) return cache_fail(PSV_EINVAL, "frequency %d is not finite", pair);
      if (std::fabs(f) > 1e6) return cache_fail(PSV_EINVAL, "frequency %d is over 1e6 radians", pair);
      k.turn[pair] = fixed_turns(f);
      k.axis[pair] = static_cast<uint8_t>(a);
    }
  if (!x || !pos || !out) return cache_fail(PSV_EINVAL, "null pointer");
  const bool same = x == out && same_rows(p->x_stride, p->out_stride, p->B, p->L, p->H);
  if (!same && x == out) return cache_fail(PSV_EINVAL, "in place needs equal strides");
  const uintptr_t mask = static_cast<uintptr_t>(size - 1);
  if ((reinterpret_cast<uintptr_t>(x) & mask) || (reinterpret_cast<uintptr_t>(out) & mask) || !on4({pos, p->lens}))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  const Area out_area = tensor_area("out", out, p->out_stride, p->B, p->L, p->H, p->dh, size);
  const int64_t pos_st[3] = {p->pos_stride[0], p->pos_stride[1], 1};
  if (int r = check_areas({out_area}, {same ? plain_area("x", nullptr, 0)
                                            : tensor_area("x", x, p->x_stride, p->B, p->L, p->H, p->dh, size),
                                       tensor_area("pos", pos, pos_st, p->B, p->L, 1, p->n_axes, 4)}))
    return r;
  int dev = 0;
  if (int r = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return r;
  if (int r = check_device(dev, x, "x")) return r;
  if (out != x)
    if (int r = check_device(dev, out, "out")) return r;
  k.x = x;
  k.out = out;
  k.pos = pos;
  k.lens = p->lens;
  k.xs = strides3(p->x_stride);
  k.os = strides3(p->out_stride);
  k.pos_b = p->pos_stride[0];
  k.pos_l = p->pos_stride[1];
  k.B = p->B, k.L = p->L, k.H = p->H, k.dh = p->dh, k.R = R;
  k.inverse = p->inverse;
  const int N = 16 / size;
  const bool halves = p->layout == PSV_ROPE_HALVES;
  const bool vec = multiple16(x, p->x_stride, p->B, p->L, p->H, size) &&
                   multiple16(out, p->out_stride, p->B, p->L, p->H, size) && p->dh % N == 0 &&
                   (!halves || ((R / 2) % N == 0 && (p->dh - R) % N == 0));
  // A thread's angles serve as many heads as leave about 512 threads an SM.
  const int64_t all = static_cast<int64_t>(p->B) * p->L * p->H * (p->dh / (vec ? N : 2));
  const int64_t hpt = all / (152 * 512);
  k.hpt = static_cast<int>(hpt < 1 ? 1 : hpt > p->H ? p->H : hpt > 16 ? 16 : hpt);
  k.hgroups = (p->H + k.hpt - 1) / k.hpt;
  k.hpt = (p->H + k.hgroups - 1) / k.hgroups;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (p->dtype == PSV_DTYPE_F32)
    e = halves ? launch_rope_t<float, true>(k, vec, st) : launch_rope_t<float, false>(k, vec, st);
  else if (p->dtype == PSV_DTYPE_BF16)
    e = halves ? launch_rope_t<__nv_bfloat16, true>(k, vec, st) : launch_rope_t<__nv_bfloat16, false>(k, vec, st);
  else
    e = halves ? launch_rope_t<__half, true>(k, vec, st) : launch_rope_t<__half, false>(k, vec, st);
  return cuda_status(e, "rope launch");
}

// ---------------------------------------------------------------- eviction

namespace {

struct EvictParams {
  const void *k, *v;
  const float* mass;
  void *k_out, *v_out;
  float* mass_out;
  int32_t* idx;
  const int32_t *k_lens, *k_pos, *k_doc;
  int32_t *pos_out, *doc_out, *lens_out;
  Strides3 ks, vs, kos, vos;
  int64_t km_b, km_h;
  int B, H, dh, L, budget, sinks, recent;
};

constexpr int kSelThreads = 1024;
constexpr int kSelSmemKeys = 49152;  // keys held in shared memory (192 KB)

// Order of selection as an unsigned key: protected slots, then NaN, then by
// value (+0 and -0 are equal).
__device__ __forceinline__ uint32_t select_key(const EvictParams& p, float weight, int j, int n) {
  if (j < p.sinks || j >= n - p.recent) return 0xffffffffu;
  const float x = weight + 0.0f;
  if (x != x) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sums of a and b over the block's threads.
__device__ __forceinline__ void block_scan2(int& a, int& b, int* sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int xo = __shfl_up_sync(0xffffffffu, x, o), yo = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += xo, y += yo;
  }
  if (lane == 31) sm[w] = x, sm[32 + w] = y;
  __syncthreads();
  if (w == 0) {
    const bool there = lane < static_cast<int>(blockDim.x >> 5);
    int s = there ? sm[lane] : 0, t = there ? sm[32 + lane] : 0;
    const int s0 = s, t0 = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int so = __shfl_up_sync(0xffffffffu, s, o), to = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) s += so, t += to;
    }
    sm[lane] = s - s0, sm[32 + lane] = t - t0;
  }
  __syncthreads();
  a = x - a + sm[w];
  b = y - b + sm[32 + w];
}

// What the select kernels write for a kept slot j at place `at` of its row.
__device__ __forceinline__ void keep_slot(const EvictParams& p, float weight, int64_t row, int64_t meta, int at, int j) {
  p.idx[row + at] = j;
  p.mass_out[row + at] = weight;
  if (p.pos_out) p.pos_out[row + at] = p.k_pos ? p.k_pos[meta + j] : j;
  if (p.doc_out) p.doc_out[row + at] = p.k_doc[meta + j];
}

// One CTA per (sequence, kv head) with up to 512 KPT slots: every thread holds
// KPT consecutive slots' keys in registers.  The protected slots are set aside;
// of the others the greatest `left` are found by three histograms of 11 bits
// in shared memory (the value's sign, exponent and two bits first, so that
// weights over many octaves spread over the bins), and one scan gives the kept
// slots their places.  Bound by latency: about five barriers a pass, 11 us for
// 12 heads of 7800 slots (bins over the keys' own range were no faster).
constexpr int kRegThreads = 512;

template <int KPT>
__global__ void __launch_bounds__(kRegThreads) evict_select_kernel(const EvictParams p, int vec) {
  __shared__ int scan[64];
  __shared__ int hist[2048];
  __shared__ uint16_t kept[KPT * kRegThreads];
  static_assert(KPT * kRegThreads <= 65536, "slots fit 16 bits");
  __shared__ uint32_t s_thr;
  __shared__ int s_left;
  pdl_trigger();
  const int h = blockIdx.x % p.H, b = blockIdx.x / p.H, t = threadIdx.x;
  const float* mass = p.mass + (static_cast<int64_t>(b) * p.H + h) * p.L;
  for (int i = t; i < 2048; i += kRegThreads) hist[i] = 0;
  pdl_wait();
  const int n = p.k_lens ? min(max(p.k_lens[b], 0), p.L) : p.L;
  const int keep = min(n, p.budget);
  uint32_t key[KPT];
  float x[KPT];
#pragma unroll
  for (int i = 0; i < KPT; i += 4) {  // rows of L % 4 == 0 are read 16 bytes at a time
    const int j = t * KPT + i;
    if (vec && j + 4 <= p.L) {
      const float4 v = *reinterpret_cast<const float4*>(mass + j);
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i + e] = j + e < p.L ? mass[j + e] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < KPT; ++i) key[i] = t * KPT + i < n ? select_key(p, x[i], t * KPT + i, n) : 0u;
  // Keys over thr are kept, `left` of those equal to it.
  uint32_t thr = 0;
  int left = keep;
  if (keep < n) {
    // (sinks + recent <= budget = keep < n: they do not meet.)
    left = keep - min(p.sinks, n) - p.recent;
    __syncthreads();
    for (int shift = 21; left > 0; shift = shift == 21 ? 10 : 0) {
      const int bits = shift ? 11 : 10;
      const uint32_t hi = shift == 21 ? 0u : 0xffffffffu << (shift + bits);
#pragma unroll
      for (int i = 0; i < KPT; ++i) {
        const int j = t * KPT + i;
        const bool in = j < n && j >= p.sinks && j < n - p.recent && (key[i] & hi) == thr;
        if (in) atomicAdd(&hist[(key[i] >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // Thread t holds bins 2047 - 4 t .. 2044 - 4 t (from the top).
      int own[4], sum = 0, zero = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        own[k] = hist[2047 - 4 * t - k];
        sum += own[k];
        hist[2047 - 4 * t - k] = 0;
      }
      int before = sum;
      block_scan2(before, zero, scan);
      if (before < left && before + sum >= left) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (before < left && before + own[k] >= left) {
            s_thr = thr | static_cast<uint32_t>(2047 - 4 * t - k) << shift;
            s_left = left - before;
          }
          before += own[k];
        }
      }
      __syncthreads();
      thr = s_thr;
      left = s_left;
      if (shift == 0) break;
    }
    // With no place left but the protected slots', nothing else is kept.
    if (keep == min(p.sinks, n) + p.recent) thr = 0xffffffffu, left = keep;
  }
  int over = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const bool in = t * KPT + i < n;
    over += in && (keep == n || key[i] > thr);
    ties += in && keep < n && key[i] == thr;
  }
  __syncthreads();  // scan is used again
  block_scan2(over, ties, scan);
  const int64_t row = (static_cast<int64_t>(b) * p.H + h) * p.budget;
  const int64_t meta = b * p.km_b + h * p.km_h;
  // The kept slots are listed in shared memory and written from there, so that
  // consecutive threads write consecutive places.
  int at = over + min(ties, left);
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int j = t * KPT + i;
    if (j < n) {
      bool k = keep == n || key[i] > thr;
      if (!k && key[i] == thr) k = ties++ < left;
      if (k) kept[at++] = static_cast<uint16_t>(j);
    }
  }
  __syncthreads();
  for (int a0 = t; a0 < keep; a0 += 4 * kRegThreads) {  // four reads on their way at once
    int j[4], pos[4], doc[4];
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (a0 + k * kRegThreads >= keep) break;
      j[k] = kept[a0 + k * kRegThreads];
      w[k] = mass[j[k]];
      pos[k] = p.pos_out && p.k_pos ? p.k_pos[meta + j[k]] : j[k];
      doc[k] = p.doc_out ? p.k_doc[meta + j[k]] : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int a = a0 + k * kRegThreads;
      if (a >= keep) break;
      p.idx[row + a] = j[k];
      p.mass_out[row + a] = w[k];
      if (p.pos_out) p.pos_out[row + a] = pos[k];
      if (p.doc_out) p.doc_out[row + a] = doc[k];
    }
  }
  if (h == 0 && t == 0 && p.lens_out) p.lens_out[b] = keep;
}

// The same for any number of slots: radix selection, 8 bits a pass, over keys
// in shared memory (or read again), then the kept slots in order by one scan
// over contiguous shares of the slots.
__global__ void __launch_bounds__(kSelThreads) evict_select_long_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[256];
  __shared__ int scan[64];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x % p.H, b = blockIdx.x / p.H, t = threadIdx.x;
  const int n = p.k_lens ? min(max(p.k_lens[b], 0), p.L) : p.L;
  const int keep = min(n, p.budget);
  const float* mass = p.mass + (static_cast<int64_t>(b) * p.H + h) * p.L;
  const bool held = p.L <= kSelSmemKeys;
  if (held)
    for (int j = t; j < n; j += kSelThreads) keys[j] = select_key(p, mass[j], j, n);
  if (t == 0) s_prefix = 0, s_need = keep;
  __syncthreads();
  auto key_at = [&](int j) { return held ? keys[j] : select_key(p, mass[j], j, n); };
  // Keys over the threshold are kept, `need` of those equal to it.
  uint32_t thr = 0;
  int need = keep;
  if (keep < n) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = t; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t pre = s_prefix;
      const uint32_t hi = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const uint32_t u = j0 + t < n ? key_at(j0 + t) : 0u;
        const bool in = j0 + t < n && (u & hi) == pre;
        // One addition for the lanes of a warp that share a bin (weights crowd a few).
        const uint32_t bin = in ? (u >> shift) & 255 : 256u;
        const uint32_t same = __match_any_sync(0xffffffffu, bin);
        if (in && (t & 31) == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
      }
      __syncthreads();
      if (t < 32) {
        // Lane l holds bins 8 l .. 8 l + 7, counted from the top.
        int sum = 0, own[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += own[k] = hist[255 - (8 * t + k)];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (t >= o) before += x;
        }
        before -= sum;
        const int left = s_need;
        __syncwarp();
        if (before < left && before + sum >= left) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (before < left && before + own[k] >= left) {
              s_prefix = pre | static_cast<uint32_t>(255 - (8 * t + k)) << shift;
              s_need = left - before;
            }
            before += own[k];
          }
        }
      }
      __syncthreads();
    }
    thr = s_prefix;
    need = s_need;
  }
  const int per = (n + kSelThreads - 1) / kSelThreads;
  const int j0 = min(n, t * per), j1 = min(n, j0 + per);
  int over = 0, ties = 0;
  for (int j = j0; j < j1; ++j) {
    const uint32_t u = key_at(j);
    over += keep == n || u > thr;
    ties += keep < n && u == thr;
  }
  block_scan2(over, ties, scan);
  const int64_t row = (static_cast<int64_t>(b) * p.H + h) * p.budget;
  const int64_t meta = b * p.km_b + h * p.km_h;
  int at = over + min(ties, need);
  for (int j = j0; j < j1; ++j) {
    const uint32_t u = key_at(j);
    bool k = keep == n || u > thr;
    if (!k && u == thr) k = ties++ < need;
    if (k) keep_slot(p, mass[j], row, meta, at++, j);
  }
  if (h == 0 && t == 0 && p.lens_out) p.lens_out[b] = keep;
}

// Copies the kept rows.  Consecutive threads take consecutive units (16 bytes,
// or one value) of an out row and then the next head; a thread takes kRows such
// rows, a grid apart, with all their loads on the way at once.  Memory-bound:
// with the selection before it 23 us for 4680 of 7800 slots of 12 heads of 128
// (58 MB), 330 us for eight sequences of 40 heads (2 GB, 6.0 TB/s).
template <class U, int kRows>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p, uint32_t units, int esize, uint32_t step) {
  const uint32_t t = blockIdx.x * 256 + threadIdx.x, H = p.H;
  const uint32_t r = t / units;
  const int u = static_cast<int>(t - r * units);
  const int64_t row0 = r / H;
  const int h = static_cast<int>(r - static_cast<uint32_t>(row0) * H);
  const int b = blockIdx.y;
  pdl_wait();
  if (row0 >= step) return;
  const int n = p.k_lens ? min(max(p.k_lens[b], 0), p.L) : p.L;
  const int keep = min(n, p.budget);
  U kk[kRows], vv[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + i * static_cast<int64_t>(step);
    if (row >= keep) break;
    const int64_t j = p.idx[(static_cast<int64_t>(b) * p.H + h) * p.budget + row];
    kk[i] = reinterpret_cast<const U*>(static_cast<const char*>(p.k) + (b * p.ks.b + j * p.ks.l + h * p.ks.h) * esize)[u];
    vv[i] = reinterpret_cast<const U*>(static_cast<const char*>(p.v) + (b * p.vs.b + j * p.vs.l + h * p.vs.h) * esize)[u];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + i * static_cast<int64_t>(step);
    if (row >= keep) break;
    reinterpret_cast<U*>(static_cast<char*>(p.k_out) + (b * p.kos.b + row * p.kos.l + h * p.kos.h) * esize)[u] = kk[i];
    reinterpret_cast<U*>(static_cast<char*>(p.v_out) + (b * p.vos.b + row * p.vos.l + h * p.vos.h) * esize)[u] = vv[i];
  }
}

template <class U>
cudaError_t launch_gather(const EvictParams& p, int size, cudaStream_t st) {
  constexpr int kRows = 4;
  const int units = p.dh * size / static_cast<int>(sizeof(U));
  const uint32_t step = static_cast<uint32_t>((p.budget + kRows - 1) / kRows);
  const uint32_t threads = step * p.H * units;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((threads + 255) / 256, p.B), 256, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, evict_gather_kernel<U, kRows>, p, static_cast<uint32_t>(units), size, step);
}

template <int KPT>
cudaError_t launch_select(const EvictParams& p, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(p.B * p.H), kRegThreads, 0, st, attr);
  const int vec = p.L % 4 == 0 && (reinterpret_cast<uintptr_t>(p.mass) & 15) == 0;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<KPT>, p, vec);
}

cudaError_t launch_select_any(const EvictParams& p, cudaStream_t st) {
  if (p.L <= 4 * kRegThreads) return launch_select<4>(p, st);
  if (p.L <= 8 * kRegThreads) return launch_select<8>(p, st);
  if (p.L <= 16 * kRegThreads) return launch_select<16>(p, st);
  if (p.L <= 32 * kRegThreads) return launch_select<32>(p, st);
  static uint64_t set_up = 0;
  cudaError_t e = psv::once_per_device(&set_up, [](int) {
    return cudaFuncSetAttribute(evict_select_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemKeys * 4);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const size_t smem = p.L <= kSelSmemKeys ? static_cast<size_t>(p.L) * 4 : 0;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(p.B * p.H), kSelThreads, smem, st, attr);
  return cudaLaunchKernelEx(&cfg, evict_select_long_kernel, p);
}

}  // namespace

PSV_API int psv_cache_evict(const psv_evict_problem* p, const void* k, const void* v, const float* mass,
                            void* k_out, void* v_out, float* mass_out, int32_t* idx_out,
                            void* cuda_stream) {
  if (!p) return cache_fail(PSV_EINVAL, "null problem");
  const int size = dtype_size(p->dtype);
  if (!size) return cache_fail(PSV_EINVAL, "unknown dtype %d", p->dtype);
  if (p->B < 1 || p->Hkv < 1 || p->L < 1 || p->dh < 1)
    return cache_fail(PSV_EINVAL, "need B, Hkv, L, dh >= 1");
  if (p->B > 65535 || static_cast<int64_t>(p->B) * p->Hkv > 0x7fffffff)
    return cache_fail(PSV_EINVAL, "too many sequences and heads");
  // (The selection steps over the slots in 32 bits, by 1024 at a time and by shares.)
  if (p->L > (1 << 30)) return cache_fail(PSV_EINVAL, "L %d: at most 2^30 slots", p->L);
  if (p->budget < 1 || p->budget > p->L) return cache_fail(PSV_EINVAL, "budget %d: 1 to L = %d", p->budget, p->L);
  if (p->sinks < 0 || p->recent < 0 || static_cast<int64_t>(p->sinks) + p->recent > p->budget)
    return cache_fail(PSV_EINVAL, "sinks %d + recent %d do not fit the budget %d", p->sinks, p->recent, p->budget);
  if (!stride_ok(p->k_stride, 3) || !stride_ok(p->v_stride, 3) || !stride_ok(p->k_out_stride, 3) ||
      !stride_ok(p->v_out_stride, 3) || !stride_ok(p->k_meta_stride, 2))
    return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  if (!rows_distinct(p->k_out_stride, p->B, p->budget, p->Hkv, p->dh) ||
      !rows_distinct(p->v_out_stride, p->B, p->budget, p->Hkv, p->dh))
    return cache_fail(PSV_EINVAL, "the rows of k_out or v_out overlap");
  if (p->doc_out && !p->k_doc) return cache_fail(PSV_EINVAL, "doc_out needs k_doc");
  if (p->lens_out && p->lens_out == p->k_lens) return cache_fail(PSV_EINVAL, "lens_out must not be k_lens");
  if (static_cast<int64_t>(p->budget) * p->Hkv * p->dh > 0xffffff00ll)
    return cache_fail(PSV_EINVAL, "a sequence's kept keys are over 2^32 values");
  if (!k || !v || !mass || !k_out || !v_out || !mass_out || !idx_out)
    return cache_fail(PSV_EINVAL, "null pointer");
  const void* typed[4] = {k, v, k_out, v_out};
  for (const void* x : typed)
    if (reinterpret_cast<uintptr_t>(x) & (size - 1)) return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  if (!on4({mass, mass_out, idx_out, p->k_lens, p->k_pos, p->k_doc, p->pos_out, p->doc_out, p->lens_out}))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  if (k_out == v_out) return cache_fail(PSV_EINVAL, "k_out and v_out are the same buffer");
  const int64_t in_rows = static_cast<int64_t>(p->B) * p->Hkv, meta_st[3] = {p->k_meta_stride[0], p->k_meta_stride[1], 1};
  auto kept = [&](const char* name, const void* at) { return plain_area(name, at, in_rows * p->budget * 4); };
  auto meta = [&](const char* name, const void* at) {
    return at ? tensor_area(name, at, meta_st, p->B, p->Hkv, 1, p->L, 4) : plain_area(name, at, 0);
  };
  if (int r = check_areas({tensor_area("k_out", k_out, p->k_out_stride, p->B, p->budget, p->Hkv, p->dh, size),
                           tensor_area("v_out", v_out, p->v_out_stride, p->B, p->budget, p->Hkv, p->dh, size),
                           kept("mass_out", mass_out), kept("idx_out", idx_out), kept("pos_out", p->pos_out),
                           kept("doc_out", p->doc_out), plain_area("lens_out", p->lens_out, p->B * int64_t{4})},
                          {tensor_area("k", k, p->k_stride, p->B, p->L, p->Hkv, p->dh, size),
                           tensor_area("v", v, p->v_stride, p->B, p->L, p->Hkv, p->dh, size),
                           plain_area("mass", mass, in_rows * p->L * 4), plain_area("k_lens", p->k_lens, p->B * int64_t{4}),
                           meta("k_pos", p->k_pos), meta("k_doc", p->k_doc)}))
    return r;
  int dev = 0;
  if (int r = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return r;
  if (int r = check_device(dev, k, "k")) return r;
  if (int r = check_device(dev, k_out, "k_out")) return r;
  EvictParams e{};
  e.k = k, e.v = v, e.mass = mass, e.k_out = k_out, e.v_out = v_out, e.mass_out = mass_out, e.idx = idx_out;
  e.k_lens = p->k_lens, e.k_pos = p->k_pos, e.k_doc = p->k_doc;
  e.pos_out = p->pos_out, e.doc_out = p->doc_out, e.lens_out = p->lens_out;
  e.ks = strides3(p->k_stride), e.vs = strides3(p->v_stride);
  e.kos = strides3(p->k_out_stride), e.vos = strides3(p->v_out_stride);
  e.km_b = p->k_meta_stride[0], e.km_h = p->k_meta_stride[1];
  e.B = p->B, e.H = p->Hkv, e.dh = p->dh, e.L = p->L, e.budget = p->budget;
  e.sinks = p->sinks, e.recent = p->recent;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t r = launch_select_any(e, st);
  if (r != cudaSuccess) return cuda_status(r, "eviction launch");
  const bool vec = (static_cast<int64_t>(p->dh) * size) % 16 == 0 &&
                   multiple16(k, p->k_stride, p->B, p->L, p->Hkv, size) &&
                   multiple16(v, p->v_stride, p->B, p->L, p->Hkv, size) &&
                   multiple16(k_out, p->k_out_stride, p->B, p->budget, p->Hkv, size) &&
                   multiple16(v_out, p->v_out_stride, p->B, p->budget, p->Hkv, size);
  r = vec ? launch_gather<uint4>(e, size, st)
          : size == 4 ? launch_gather<uint32_t>(e, size, st) : launch_gather<uint16_t>(e, size, st);
  return cuda_status(r, "eviction launch");
}

// ------------------------------------------------- attention over a cache

namespace {

int check_cache(const psv_cache_problem* p) {
  if (!p) return cache_fail(PSV_EINVAL, "null problem");
  if (p->dtype != PSV_DTYPE_BF16 && p->dtype != PSV_DTYPE_F16)
    return cache_fail(PSV_EINVAL, "dtype %d: bf16 or f16", p->dtype);
  if (p->B < 1 || p->Hkv < 1 || p->Hq < 1 || p->Hq % p->Hkv)
    return cache_fail(PSV_EINVAL, "need B >= 1 and Hq (%d) a multiple of Hkv (%d)", p->Hq, p->Hkv);
  if (p->dh < 1 || p->dh > 256) return cache_fail(PSV_EINVAL, "dh %d: 1 to 256", p->dh);
  if (p->Lq < 0 || p->Lk < 0 || p->Lq > (1 << 24) || p->Lk > (1 << 28))
    return cache_fail(PSV_EINVAL, "Lq %d: 0 to 2^24, Lk %d: 0 to 2^28", p->Lq, p->Lk);
  if (static_cast<int64_t>(p->B) * p->Hq > (1 << 24)) return cache_fail(PSV_EINVAL, "over 2^24 sequences x heads");
  if (!(std::isfinite(p->scale) && p->scale >= 0)) return cache_fail(PSV_EINVAL, "scale must be finite and not negative");
  if (!(std::isfinite(p->softcap) && p->softcap >= 0))
    return cache_fail(PSV_EINVAL, "softcap must be finite and not negative");
  if (!stride_ok(p->q_stride, 3) || !stride_ok(p->k_stride, 3) || !stride_ok(p->v_stride, 3) ||
      !stride_ok(p->o_stride, 3) || !stride_ok(&p->q_meta_stride, 1) || !stride_ok(p->k_meta_stride, 2))
    return cache_fail(PSV_EINVAL, "strides must lie in [0, 2^40]");
  if (!on4({p->q_lens, p->k_lens, p->q_pos, p->q_doc, p->k_pos, p->k_doc, p->prefix, p->slopes}))
    return cache_fail(PSV_EINVAL, "lengths, positions, documents, prefixes and slopes must be aligned to 4 bytes");
  if (!p->k_doc != !p->q_doc) return cache_fail(PSV_EINVAL, "k_doc and q_doc come together");
  if (p->prefix && !p->causal) return cache_fail(PSV_EINVAL, "prefix needs causal");
  return PSV_OK;
}

int check_scratch(void* scratch, size_t bytes, size_t need) {
  if (reinterpret_cast<uintptr_t>(scratch) & 255) return cache_fail(PSV_EINVAL, "scratch must be 256-byte aligned");
  if (bytes < need) return cache_fail(PSV_EINVAL, "scratch of %zu bytes, %zu needed", bytes, need);
  return PSV_OK;
}

CacheParams cache_params(const psv_cache_problem* p, const void* q, const void* k, void* scratch) {
  CacheParams c{};
  c.B = p->B, c.Hq = p->Hq, c.Hkv = p->Hkv, c.G = p->Hq / p->Hkv, c.dh = p->dh;
  c.Lq = p->Lq, c.Lk = p->Lk, c.causal = p->causal != 0;
  c.scale = p->scale > 0 ? p->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(p->dh)));
  c.softcap = p->softcap;
  c.qs = strides3(p->q_stride), c.ks = strides3(p->k_stride);
  c.vs = strides3(p->v_stride), c.os = strides3(p->o_stride);
  c.q = q, c.k = k;
  c.q_lens = p->q_lens, c.k_lens = p->k_lens, c.q_pos = p->q_pos, c.q_doc = p->q_doc;
  c.k_pos = p->k_pos, c.k_doc = p->k_doc, c.prefix = p->prefix;
  c.qm_b = p->q_meta_stride, c.km_b = p->k_meta_stride[0], c.km_h = p->k_meta_stride[1];
  c.slopes = p->slopes;
  c.err = static_cast<int*>(scratch);
  return c;
}

size_t cache_scratch(const psv_cache_problem* p) {
  const CacheParams c = cache_params(p, nullptr, nullptr, nullptr);
  return psv::cache_attn_tc_shape(c) ? psv::cache_attn_tc_scratch(c) : PSV_CACHE_SCRATCH_HEAD;
}


}  // namespace

PSV_API int psv_cache_scratch_bytes(const psv_cache_problem* p, size_t* bytes) {
  if (int r = check_cache(p)) return r;
  if (!bytes) return cache_fail(PSV_EINVAL, "null pointer");
  *bytes = cache_scratch(p);
  return PSV_OK;
}

PSV_API int psv_cache_status(const void* scratch, int* status, void* cuda_stream) {
  if (!scratch || !status) return cache_fail(PSV_EINVAL, "null pointer");
  if (int r = check_scratch(const_cast<void*>(scratch), 0, 0)) return r;
  int dev = 0;
  if (int r = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return r;
  if (int r = check_device(dev, scratch, "scratch")) return r;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaStreamCaptureStatus capture;
  if (int r = cuda_status(cudaStreamIsCapturing(st, &capture), "status")) return r;
  if (capture != cudaStreamCaptureStatusNone) return cache_fail(PSV_EINVAL, "the stream is being captured");
  if (int r = cuda_status(cudaMemcpyAsync(status, scratch, sizeof(int), cudaMemcpyDeviceToHost, st), "status")) return r;
  return cuda_status(cudaStreamSynchronize(st), "status");
}

PSV_API int psv_cache_attention(const psv_cache_problem* p, const void* q, const void* k, const void* v,
                                void* o, float* lse, void* scratch, size_t scratch_bytes,
                                void* cuda_stream) {
  if (int r = check_cache(p)) return r;
  if (p->Lq == 0) return PSV_OK;
  if (!rows_distinct(p->o_stride, p->B, p->Lq, p->Hq, p->dh)) return cache_fail(PSV_EINVAL, "o's rows overlap");
  if (!q || !o || !scratch || (p->Lk && (!k || !v))) return cache_fail(PSV_EINVAL, "null pointer");
  const uintptr_t at = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                       reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o);
  if ((at & 1) || (reinterpret_cast<uintptr_t>(lse) & 3))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  // (Every row of q is read before the row of o is written.)
  const bool in_place = q == o && same_rows(p->q_stride, p->o_stride, p->B, p->Lq, p->Hq);
  const Area q_area = tensor_area("q", q, p->q_stride, p->B, p->Lq, p->Hq, p->dh, 2);
  const Area none = plain_area("", nullptr, 0);
  if (int r = check_areas(
          {tensor_area("o", o, p->o_stride, p->B, p->Lq, p->Hq, p->dh, 2),
           plain_area("lse", lse, static_cast<int64_t>(p->B) * p->Hq * p->Lq * 4)},
          {in_place ? none : q_area, p->Lk ? tensor_area("k", k, p->k_stride, p->B, p->Lk, p->Hkv, p->dh, 2) : none,
           p->Lk ? tensor_area("v", v, p->v_stride, p->B, p->Lk, p->Hkv, p->dh, 2) : none}))
    return r;
  int dev = 0;
  if (int r = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return r;
  if (int r = check_device(dev, q, "q")) return r;
  if (int r = check_device(dev, o, "o")) return r;
  if (int r = check_scratch(scratch, scratch_bytes, cache_scratch(p))) return r;
  CacheParams c = cache_params(p, q, k, scratch);
  c.v = v, c.o = o, c.lse = lse;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (psv::cache_attn_tc_shape(c) && psv::cache_attn_tc_aligned(c)) {
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = psv::launch_cache_attention_tc(c, p->dtype == PSV_DTYPE_BF16, static_cast<char*>(scratch), sms, st);
    return cuda_status(e, "attention launch");
  }
  return cuda_status(psv::launch_cache_attention_general(c, p->dtype == PSV_DTYPE_BF16, st), "attention launch");
}

PSV_API int psv_cache_mass(const psv_cache_problem* p, const void* q, const void* k, const float* lse,
                           const float* mass_in, float* mass_out, void* scratch, size_t scratch_bytes,
                           void* cuda_stream) {
  if (int r = check_cache(p)) return r;
  if (p->Lk == 0) return PSV_OK;
  if (!k || !mass_out || !scratch || (p->Lq && (!q || !lse))) return cache_fail(PSV_EINVAL, "null pointer");
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) & 1) ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(mass_in) | reinterpret_cast<uintptr_t>(mass_out)) & 3))
    return cache_fail(PSV_EINVAL, "pointers must be aligned to their type");
  const int64_t bytes = static_cast<int64_t>(p->B) * p->Hkv * p->Lk * 4;
  if (mass_in && mass_in != mass_out && overlap(mass_in, bytes, mass_out, bytes))
    return cache_fail(PSV_EINVAL, "mass_in overlaps mass_out in part");
  const Area none = plain_area("", nullptr, 0);
  if (int r = check_areas({plain_area("mass_out", mass_out, bytes)},
                          {p->Lq ? tensor_area("q", q, p->q_stride, p->B, p->Lq, p->Hq, p->dh, 2) : none,
                           tensor_area("k", k, p->k_stride, p->B, p->Lk, p->Hkv, p->dh, 2),
                           plain_area("lse", lse, static_cast<int64_t>(p->B) * p->Hq * p->Lq * 4)}))
    return r;
  int dev = 0;
  if (int r = cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return r;
  if (int r = check_device(dev, k, "k")) return r;
  if (int r = check_device(dev, mass_out, "mass_out")) return r;
  if (int r = check_scratch(scratch, scratch_bytes, cache_scratch(p))) return r;
  CacheParams c = cache_params(p, q, k, scratch);
  c.lse = const_cast<float*>(lse), c.mass_in = mass_in, c.mass_out = mass_out;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (psv::cache_mass_tc(c)) {
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = psv::launch_cache_mass_tc(c, p->dtype == PSV_DTYPE_BF16, static_cast<char*>(scratch), sms, st);
    return cuda_status(e, "mass launch");
  }
  return cuda_status(psv::launch_cache_mass_general(c, p->dtype == PSV_DTYPE_BF16, st), "mass launch");
}

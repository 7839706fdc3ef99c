// Attention over a cache and the attention mass for every layout, alignment
// and head width the calls accept: plain loads, one warp per row (or per
// key), 32-bit arithmetic throughout.  The tensor-core kernels take the
// aligned problems; these are bound by their uncoalesced 2-byte loads, which they
// repeat for every row, and are hundreds of times slower (a fallback for odd
// layouts, not tuned): eight tokens over 7800 keys of 12 heads of 256 8.5 ms, of
// 128 in the few-row kernel 67 us; 1560 rows x 1560 keys of 12 heads of 136 8.9 ms,
// their mass 6.9 ms, of 128 on the tensor cores 30 and 22 us.
#include "cache_kernels.h"

namespace psv {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float val(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float val(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(__nv_bfloat16* y, float x) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* y, float x) { *y = __float2half_rn(x); }

// Score of row (position qp, document qd) and key j, after the cap and the
// bias; false if the row does not see the key.
__device__ __forceinline__ bool finish_score(const CacheParams& p, float& s, int qp, int qd, int prefix,
                                             float slope, int64_t meta, int j) {
  if (p.k_doc && p.k_doc[meta + j] != qd) return false;
  const int kp = p.k_pos ? p.k_pos[meta + j] : j;
  if (p.causal && kp > qp && kp >= prefix) return false;
  s *= p.scale;
  if (p.softcap > 0) s = p.softcap * tanhf(s / p.softcap);
  if (p.slopes) s -= slope * fabsf(static_cast<float>(qp - kp));
  return true;
}

template <class T>
__global__ void __launch_bounds__(kWarps * 32) attention_general_kernel(const CacheParams p) {
  __shared__ float sq[kWarps][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int blocks = (p.Lq + kWarps - 1) / kWarps, pair = blockIdx.x / blocks;
  const int i = blockIdx.x % blocks * kWarps + w, h = pair % p.Hq, b = pair / p.Hq;
  if (i >= cache_q_len(p, b)) return;
  const int hk = h / p.G, n = cache_k_len(p, b);
  const T* q = static_cast<const T*>(p.q) + b * p.qs.b + i * p.qs.l + h * p.qs.h;
  for (int d = lane; d < p.dh; d += 32) sq[w][d] = val(q[d]);
  __syncwarp();
  const int qp = p.q_pos ? p.q_pos[b * p.qm_b + i] : n - cache_q_len(p, b) + i;
  const int qd = p.q_doc ? p.q_doc[b * p.qm_b + i] : 0;
  const int prefix = p.prefix ? p.prefix[b] : 0;
  const float slope = p.slopes ? p.slopes[h] : 0.0f;
  const int64_t meta = b * p.km_b + hk * p.km_h;
  const T* k = static_cast<const T*>(p.k) + b * p.ks.b + hk * p.ks.h;
  const T* v = static_cast<const T*>(p.v) + b * p.vs.b + hk * p.vs.h;
  float m = -INFINITY, l = 0.0f, acc[8] = {};
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    bool sees = false;
    if (j < n) {
      float dot = 0.0f;
      for (int d = 0; d < p.dh; ++d) dot = fmaf(sq[w][d], val(k[j * p.ks.l + d]), dot);
      sees = finish_score(p, dot, qp, qd, prefix, slope, meta, j);
      if (sees) s = dot;
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!__any_sync(0xffffffffu, sees)) continue;
    const float m_new = fmaxf(m, mx), m0 = m_new == -INFINITY ? 0.0f : m_new;  // (-inf: NaN at most so far)
    const float a = exp2f((m - m0) * kLog2e), e = sees ? exp2f((s - m0) * kLog2e) : 0.0f;
    float sum = e;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * a + sum;
    m = m_new;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= a;
    const unsigned seen = __ballot_sync(0xffffffffu, sees);
    for (int c = 0; c < 32; ++c) {
      const float pc = __shfl_sync(0xffffffffu, e, c);
      if (!((seen >> c) & 1)) continue;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (lane + 32 * x < p.dh) acc[x] = fmaf(pc, val(v[(j0 + c) * p.vs.l + lane + 32 * x]), acc[x]);
    }
  }
  T* o = static_cast<T*>(p.o) + b * p.os.b + i * p.os.l + h * p.os.h;
  const float inv = l > 0 ? 1.0f / l : 0.0f;
#pragma unroll
  for (int x = 0; x < 8; ++x)
    if (lane + 32 * x < p.dh) put(o + lane + 32 * x, acc[x] * inv);
  if (lane == 0 && p.lse) p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i] = l == 0 ? -INFINITY : m + logf(l);
}

// One warp per key: lanes take rows in turn, the lanes' sums are joined in a
// fixed order.
template <class T>
__global__ void __launch_bounds__(kWarps * 32) mass_general_kernel(const CacheParams p) {
  __shared__ float sk[kWarps][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int blocks = (p.Lk + kWarps - 1) / kWarps, pair = blockIdx.x / blocks;
  const int j = blockIdx.x % blocks * kWarps + w, hk = pair % p.Hkv, b = pair / p.Hkv;
  const int n = cache_k_len(p, b);
  if (j >= n) return;
  const int nq = cache_q_len(p, b);
  const T* k = static_cast<const T*>(p.k) + b * p.ks.b + j * p.ks.l + hk * p.ks.h;
  for (int d = lane; d < p.dh; d += 32) sk[w][d] = val(k[d]);
  __syncwarp();
  const int prefix = p.prefix ? p.prefix[b] : 0;
  const int64_t meta = b * p.km_b + hk * p.km_h;
  float sum = 0.0f;
  for (int g = 0; g < p.G; ++g) {
    const int h = hk * p.G + g;
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
    const T* q = static_cast<const T*>(p.q) + b * p.qs.b + h * p.qs.h;
    for (int i = lane; i < nq; i += 32) {
      const int qp = p.q_pos ? p.q_pos[b * p.qm_b + i] : n - nq + i;
      const int qd = p.q_doc ? p.q_doc[b * p.qm_b + i] : 0;
      float dot = 0.0f;
      for (int d = 0; d < p.dh; ++d) dot = fmaf(sk[w][d], val(q[i * p.qs.l + d]), dot);
      const float lse = p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i];
      if (finish_score(p, dot, qp, qd, prefix, slope, meta, j) && lse != -INFINITY)
        sum += exp2f((dot - lse) * kLog2e);
    }
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    const int64_t at = (static_cast<int64_t>(b) * p.Hkv + hk) * p.Lk + j;
    p.mass_out[at] = (p.mass_in ? p.mass_in[at] : 0.0f) + sum;
  }
}

template <class K>
cudaError_t launch_rows(K kernel, const CacheParams& p, int rows, int64_t pairs, cudaStream_t st) {
  const int64_t blocks = (rows + kWarps - 1) / kWarps * pairs;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  kernel<<<static_cast<unsigned>(blocks), kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_general(const CacheParams& p, bool bf16, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(p.B) * p.Hq;
  return bf16 ? launch_rows(attention_general_kernel<__nv_bfloat16>, p, p.Lq, n, st)
              : launch_rows(attention_general_kernel<__half>, p, p.Lq, n, st);
}

cudaError_t launch_cache_mass_general(const CacheParams& p, bool bf16, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(p.B) * p.Hkv;
  return bf16 ? launch_rows(mass_general_kernel<__nv_bfloat16>, p, p.Lk, n, st)
              : launch_rows(mass_general_kernel<__half>, p, p.Lk, n, st);
}

}  // namespace psv

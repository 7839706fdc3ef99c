// Attention of any number of rows over a paged cache for every layout, head
// width and alignment the call accepts: plain loads, one warp per row, 32-bit
// arithmetic throughout.  page_attn.cuh takes the aligned problems; this one is
// bound by its uncoalesced loads, which it repeats for every row (a fallback for
// odd layouts, not tuned): two tokens over 2000 keys of 12 heads of 100 750 us, of 256
// in the other kernel 13; one over 131072 keys of 8, five query heads each, 79 ms, as a
// warp walks all keys of its row by itself.
#include "page_kernels.h"

namespace psv {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int FMT>
__device__ __forceinline__ float stored(const void* base, int64_t i) {
  if constexpr (FMT == PSV_PAGE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  if constexpr (FMT == PSV_PAGE_F16) return __half2float(static_cast<const __half*>(base)[i]);
  if constexpr (FMT == PSV_PAGE_E4M3) return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[i]);
  if constexpr (FMT == PSV_PAGE_I8) return static_cast<float>(static_cast<const int8_t*>(base)[i]);
}

__device__ __forceinline__ float asked(const void* base, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i])
              : __half2float(static_cast<const __half*>(base)[i]);
}

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) page_attention_general_kernel(const PageAttnParams p) {
  constexpr bool kScaled = FMT == PSV_PAGE_E4M3 || FMT == PSV_PAGE_I8;
  __shared__ float sq[kWarps][256];
  const PageCacheDev& c = p.c;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int blocks = (p.Lq + kWarps - 1) / kWarps, pair = blockIdx.x / blocks;
  const int i = blockIdx.x % blocks * kWarps + w, h = pair % p.Hq, b = pair / p.Hq;
  const int rows = page_rows(p, b);
  if (i >= rows) return;
  const int hk = h / p.G, n = page_length(p, b, rows), qp = n - rows + i;
  const int64_t q_at = b * p.qs.b + i * p.qs.l + h * p.qs.h;
  for (int d = lane; d < p.dh; d += 32) sq[w][d] = asked(p.q, q_at + d, p.bf16);
  __syncwarp();
  // Keys [0, sinks) and [first, end).
  const int end = min(min(p.causal ? qp + 1 : n, n), c.positions);
  const int first = p.window ? max(qp - p.window + 1, 0) : 0, sinks = p.window ? min(p.sinks, end) : 0;
  float m = -INFINITY, l = 0.0f, acc[8] = {};
  for (int j0 = 0; j0 < end; j0 += 32) {
    if (j0 >= sinks && j0 + 32 <= first) continue;
    const int j = j0 + lane;
    float s = -INFINITY, vs = 1.0f;
    PageRow at{-1, 0};
    if (j < end && (j >= first || j < sinks)) at = page_row(c, b, j);
    const bool sees = at.page >= 0;
    if (sees) {
      const int64_t k_at = at.page * c.ks.b + at.row * c.ks.l + hk * c.ks.h;
      float dot = 0.0f;
      for (int d = 0; d < p.dh; ++d) dot = fmaf(sq[w][d], stored<FMT>(c.k, k_at + d), dot);
      if (kScaled) {
        const int64_t s_at = at.page * c.ss.b + at.row * c.ss.l + hk * c.ss.h;
        dot *= c.k_scale[s_at];
        vs = c.v_scale[s_at];
      }
      s = dot * p.scale;
      if (p.softcap > 0) s = p.softcap * tanhf(s / p.softcap);
    }
    const unsigned seen = __ballot_sync(0xffffffffu, sees);
    if (!seen) continue;
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_new = fmaxf(m, mx), m0 = m_new == -INFINITY ? 0.0f : m_new;  // (-inf: NaN at most so far)
    const float a = exp2f((m - m0) * kLog2e), e = sees ? exp2f((s - m0) * kLog2e) : 0.0f;
    float sum = e;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * a + sum;
    m = m_new;
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] *= a;
    for (int k = 0; k < 32; ++k) {
      const float pk = __shfl_sync(0xffffffffu, e, k) * __shfl_sync(0xffffffffu, vs, k);
      const int page = __shfl_sync(0xffffffffu, at.page, k), row = __shfl_sync(0xffffffffu, at.row, k);
      if (!((seen >> k) & 1)) continue;
      const int64_t v_at = page * c.vs.b + row * c.vs.l + hk * c.vs.h;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (lane + 32 * x < p.dh) acc[x] = fmaf(pk, stored<FMT>(c.v, v_at + lane + 32 * x), acc[x]);
    }
  }
  const float inv = l > 0 ? 1.0f / l : 0.0f;
  const int64_t o_at = b * p.os.b + i * p.os.l + h * p.os.h;
  const bool nan = l != l;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int d = lane + 32 * x;
    if (d >= p.dh) continue;
    const float y = nan ? l : acc[x] * inv;
    if (p.bf16) static_cast<__nv_bfloat16*>(p.o)[o_at + d] = __float2bfloat16_rn(y);
    else static_cast<__half*>(p.o)[o_at + d] = __float2half_rn(y);
  }
  if (lane == 0 && p.lse) p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i] = l == 0 ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_page_attention_general(const PageAttnParams& p, cudaStream_t st) {
  const int64_t blocks = static_cast<int64_t>((p.Lq + kWarps - 1) / kWarps) * p.B * p.Hq;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  switch (p.c.format) {
    case PSV_PAGE_BF16: page_attention_general_kernel<PSV_PAGE_BF16><<<grid, kWarps * 32, 0, st>>>(p); break;
    case PSV_PAGE_F16: page_attention_general_kernel<PSV_PAGE_F16><<<grid, kWarps * 32, 0, st>>>(p); break;
    case PSV_PAGE_E4M3: page_attention_general_kernel<PSV_PAGE_E4M3><<<grid, kWarps * 32, 0, st>>>(p); break;
    default: page_attention_general_kernel<PSV_PAGE_I8><<<grid, kWarps * 32, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace psv

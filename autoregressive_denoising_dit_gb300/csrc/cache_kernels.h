// Internal interface of the rolling-cache operators (public ABI:
// include/psv.h, "kernel-level operators of a rolling key/value cache").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_cap.cuh"

namespace psv {

// Stores `msg` (printf-style) as this thread's last error of the cache calls.
int cache_fail(int code, const char* fmt, ...);

struct Strides3 {
  int64_t b, l, h;  // batch, row, head; elements
};

// psv_cache_problem as the kernels see it, with the tensors of one call.
struct CacheParams {
  int B, Hq, Hkv, G, dh, Lq, Lk, causal;
  float scale, softcap;
  Strides3 qs, ks, vs, os;
  const void *q, *k, *v;
  void* o;
  float* lse;            // attention: written (or null); mass: read
  const float* mass_in;  // may be null
  float* mass_out;
  const int32_t *q_lens, *k_lens, *q_pos, *q_doc, *k_pos, *k_doc, *prefix;
  int64_t qm_b, km_b, km_h;
  const float* slopes;
  int* err;
};

__device__ __forceinline__ int cache_k_len(const CacheParams& p, int b) {
  return p.k_lens ? min(max(p.k_lens[b], 0), p.Lk) : p.Lk;
}
__device__ __forceinline__ int cache_q_len(const CacheParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.Lq) : p.Lq;
}

cudaError_t launch_cache_attention_general(const CacheParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_cache_mass_general(const CacheParams& p, bool bf16, cudaStream_t st);

// Byte stride of an index for a 16-bit tensor map (an index of extent one is never stepped).
inline uint64_t map_stride(int64_t s, int64_t n) { return n > 1 ? static_cast<uint64_t>(s) * 2 : 16; }

// The kernels for few rows (at most kFewRows per kv head): nsplit shares of
// the keys, left in part_o [sequence, kv head, share][part_rows][64 or 128]
// and part_ml (m in log2, l) where there is more than one.
constexpr int kFewRows = 16;
struct RowsParams {
  CacheParams c;
  CapForm cap;  // where c.softcap > 0
  int nsplit, part_rows;
  int n_pieces, ctas;  // pieces: sequences x kv heads x shares; CTAs at most
  float* part_o;
  float2* part_ml;
  int* joined;  // [sequences x kv heads] shares done, zero between calls; null: another kernel joins them
};
cudaError_t launch_cache_rows(const RowsParams& p, bool bf16, bool mass, cudaStream_t st);

// The tensor-core attention: which shapes it takes, which tensors, its
// workspace (head included), and the launch on `sms` SMs.
bool cache_attn_tc_shape(const CacheParams& p);
bool cache_attn_tc_aligned(const CacheParams& p);
size_t cache_attn_tc_scratch(const CacheParams& p);
cudaError_t launch_cache_attention_tc(const CacheParams& p, bool bf16, char* scratch, int sms, cudaStream_t st);
// The same for the mass (q and k only).
bool cache_mass_tc(const CacheParams& p);
cudaError_t launch_cache_mass_tc(const CacheParams& p, bool bf16, char* scratch, int sms, cudaStream_t st);

}  // namespace psv

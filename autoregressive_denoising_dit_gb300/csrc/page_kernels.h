// Internal interface of the paged-cache operators (public ABI: include/psv.h,
// "kernel-level operators of a paged key/value cache").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/psv.h"
#include "cache_cap.cuh"
#include "cache_kernels.h"

namespace psv {

// Division of 0 <= n < 2^31 by a divisor known to the host: n f / 2^32 + n shifted
// right, with s = ceil(log2 d) and f = 2^32 (2^s - d) / d + 1.
struct FastDiv {
  uint32_t d, f, s;
  static FastDiv of(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t{1} << s) < d) ++s;
    const uint64_t f = ((uint64_t{1} << 32) * ((uint64_t{1} << s) - d)) / d + 1;
    return FastDiv{d, static_cast<uint32_t>(f), s};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, f) + n) >> s; }
};

// psv_page_cache as the kernels see it (strides: page, row, head).
struct PageCacheDev {
  int format, n_pages, page_size, positions;  // positions that the table covers
  FastDiv by_page;
  Strides3 ks, vs, ss;
  const int32_t* table;
  int64_t table_b;
  void *k, *v;
  float *k_scale, *v_scale;
};

// Where a position's key and value lie: a page, or none (< 0), and a row of it.
struct PageRow {
  int page, row;
};
__device__ __forceinline__ PageRow page_row(const PageCacheDev& c, int b, int64_t pos) {
  if (pos < 0 || pos >= c.positions) return PageRow{-1, 0};
  const uint32_t at = c.by_page.div(static_cast<uint32_t>(pos));
  const int page = c.table[b * c.table_b + at];
  return PageRow{page < c.n_pages ? page : -1, static_cast<int>(static_cast<uint32_t>(pos) - at * c.by_page.d)};
}

// A group (a sequence's kv head and tile of query rows) that CTA `i` of the attention's grid
// begins and does not end: its rows (0: there is none) and how many CTAs have shares of it.
struct alignas(32) PageShared {
  int rows, shares, b, kvh, r0;
};
constexpr int kSms = 152;
constexpr int kMaxCtas = 2 * kSms;  // shares in the workspace (of 32 rows: half as many)
// Floats of a share: O, then m', m, l of each row.
constexpr int share_floats(int dh, int rows) { return rows * (dh + 4); }

// The attention's arguments.
struct PageAttnParams {
  PageCacheDev c;
  int B, Hq, Hkv, G, dh, Lq;
  int causal, window, sinks, append, bf16;
  float scale, softcap;
  FastDiv by_group;                 // by G
  int halves;                       // page_attn.cuh: 8-bit rows are aligned to 8 bytes only
  uint32_t kb, kl, vb, vl, sb, sl;  // page_attn.cuh: strides of a page and a row in bytes
  CapForm cap;
  Strides3 qs, os;
  const void* q;
  void* o;
  float* lse;  // or null
  const int32_t *q_lens, *k_lens;
  int cluster;            // page_attn.cuh: CTAs that share a group without cutting it
  int quick;              // at most 1024 sequences and 2^31 steps
  int64_t groups;         // kv heads and tiles of rows of all sequences, at most
  PageShared* shared;     // page_attn.cuh: the groups that several CTAs share
  float* part;            // their shares
};

__device__ __forceinline__ int page_rows(const PageAttnParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.Lq) : p.Lq;
}
// Length of sequence b, at whose end its rows are; keys behind the table's
// positions have no page.
__device__ __forceinline__ int page_length(const PageAttnParams& p, int b, int rows) {
  const int n = p.k_lens ? min(max(p.k_lens[b], 0), p.c.positions) : (p.append ? 0 : p.c.positions);
  return p.append ? n + rows : n;
}

cudaError_t launch_page_attention_general(const PageAttnParams& p, cudaStream_t st);

// For rows of 16-byte pieces and pages of 16-byte (or 8-bit ones of 8-byte) pieces: the workspace's size
// (Lq, G and dh count), its use, and the launch on `sms` SMs.
size_t page_attn_scratch(const PageAttnParams& p);
void page_attn_scratch(PageAttnParams& p, void* scratch);
cudaError_t launch_page_attention(const PageAttnParams& p, int sms, cudaStream_t st);
// Of heads of up to DH, in a translation unit for each width and size of values.
template <int DH, int FMT>
cudaError_t launch_page_rows(const PageAttnParams& p, int sms, cudaStream_t st);

}  // namespace psv

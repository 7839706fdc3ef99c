// The tensor-core attention over pages (page_attn.cuh): workspace, and the choice of
// the kernel's head width and page format.
#include "page_kernels.h"

namespace psv {

// At most two shares a CTA.
size_t page_attn_scratch(const PageAttnParams& p) {
  const int dh = p.dh <= 64 ? 64 : p.dh <= 128 ? 128 : 256, rows = p.Lq * p.G <= 8 || dh == 256 ? 8 : 16;
  return kMaxCtas * sizeof(PageShared) + static_cast<size_t>(kMaxCtas) * 2 * share_floats(dh, rows) * sizeof(float);
}

void page_attn_scratch(PageAttnParams& p, void* scratch) {
  p.shared = static_cast<PageShared*>(scratch);
  p.part = reinterpret_cast<float*>(p.shared + kMaxCtas);
}

namespace {

template <int DH>
cudaError_t launch_format(const PageAttnParams& p, int sms, cudaStream_t st) {
  switch (p.c.format) {
    case PSV_PAGE_BF16: return launch_page_rows<DH, PSV_PAGE_BF16>(p, sms, st);
    case PSV_PAGE_F16: return launch_page_rows<DH, PSV_PAGE_F16>(p, sms, st);
    case PSV_PAGE_E4M3: return launch_page_rows<DH, PSV_PAGE_E4M3>(p, sms, st);
    default: return launch_page_rows<DH, PSV_PAGE_I8>(p, sms, st);
  }
}

}  // namespace

cudaError_t launch_page_attention(const PageAttnParams& p, int sms, cudaStream_t st) {
  return p.dh <= 64 ? launch_format<64>(p, sms, st) : p.dh <= 128 ? launch_format<128>(p, sms, st) : launch_format<256>(p, sms, st);
}

}  // namespace psv

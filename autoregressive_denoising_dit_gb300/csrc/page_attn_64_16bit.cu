#include "page_attn.cuh"

namespace psv {
template cudaError_t launch_page_rows<64, PSV_PAGE_BF16>(const PageAttnParams&, int, cudaStream_t);
template cudaError_t launch_page_rows<64, PSV_PAGE_F16>(const PageAttnParams&, int, cudaStream_t);
}  // namespace psv

#include "page_attn.cuh"

namespace psv {
template cudaError_t launch_page_rows<128, PSV_PAGE_E4M3>(const PageAttnParams&, int, cudaStream_t);
template cudaError_t launch_page_rows<128, PSV_PAGE_I8>(const PageAttnParams&, int, cudaStream_t);
}  // namespace psv

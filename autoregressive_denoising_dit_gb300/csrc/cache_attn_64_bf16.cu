// Instances of the cache attention for heads of up to 64 values in bf16.
#include "cache_attn_tc.cuh"

template cudaError_t psv::cattn::launch_features<64, true>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);

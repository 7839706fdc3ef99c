// Instances of the cache attention for heads of up to 128 values in f16.
#include "cache_attn_tc.cuh"

template cudaError_t psv::cattn::launch_features<128, false>(const CUtensorMap*, const TcParams&, int, int, cudaStream_t);

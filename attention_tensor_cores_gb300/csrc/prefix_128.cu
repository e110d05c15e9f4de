// fmha_fwd_prefix at D = 128 (a translation unit for each D: their kernels take long to compile)
#include "prefix_kernel.cuh"

namespace atc_gb300 {

template int launch_prefix<128>(PrefixParams, const PagedArgs&, float*, float*, cudaStream_t);

}  // namespace atc_gb300

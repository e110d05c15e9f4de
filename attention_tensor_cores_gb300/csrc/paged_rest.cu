// The paged decode kernel over the keys of each request that are attended to nowhere else (see prefix.cu).  A
// translation unit of its own: its kernels take as long to compile as those of paged.cu.
#include "paged_run.cuh"

namespace atc_gb300 {

int launch_paged_rest(const PagedArgs& a, const PagedRest& rest, cudaStream_t st)
{
    const PagedWs none{};
    if (a.c->D == 64)
        return a.causal ? run_paged<64, true, true>(a, true, none, nullptr, st, &rest) : run_paged<64, false, true>(a, true, none, nullptr, st, &rest);
    return a.causal ? run_paged<128, true, true>(a, true, none, nullptr, st, &rest) : run_paged<128, false, true>(a, true, none, nullptr, st, &rest);
}

}  // namespace atc_gb300

// Launch of the attention over common and own keys (prefix_kernel.cuh), compiled for each D by itself.
#pragma once
#include "fastdiv.cuh"
#include "paged.h"

namespace atc_gb300 {

constexpr int kRows = 128;          // query rows of a tile
constexpr int kMaxGroups = 8192;

// Groups of requests whose first keys are in the same pages
struct Groups {
    const int32_t* cu = nullptr;       // [n + 1] first request of each
    const int32_t* prefix = nullptr;   // [n] tokens in the same pages
    int n = 0;
    int nb = 0;                        // requests in a row tile
    int R = 0, chunks = 0;             // of a request and key/value head: rows, and units of at most 16 of them
};

struct PrefixParams {
    int B;               // requests
    Groups gr;
    int Hkv, R, Sq;      // rows of a request and key/value head; row r is query r % Sq
    int causal;
    float c;             // scale * log2(e)
    const int32_t* seqlens;
    const int32_t* table;
    int max_pages, num_pages, page;
    FastDiv by_page;
    int box, box_log2, groups;   // as in DecodeParams
    int cap;             // max_pages * page: lengths are clamped to it
    float* part_o;       // [rows][D] partials of common keys
    float* part_lse;
    // for the merge
    int4* plan;          // [1 + B]: (cost, CTAs) of the common and of the own keys' line; of each request its group's place, tiles, requests and first one
    int2* own;           // [B]: each request's place on the own keys' line and its tiles there
    int32_t* rest_prefix;   // [B + 1]: tiles before each request's own, and their number, when there are too many for shared memory
    int rest_units;      // units of a request's own keys
    int weigh;           // the lines count costs, not tiles
    int* status;
    long long limit;
};

struct PagedArgs;
// own_o, own_lse: partials of own keys, [U + SMs][16][D] and [U + SMs][16]
template <int D>
int launch_prefix(PrefixParams p, const PagedArgs& a, float* own_o, float* own_lse, cudaStream_t st);
extern template int launch_prefix<64>(PrefixParams, const PagedArgs&, float*, float*, cudaStream_t);
extern template int launch_prefix<128>(PrefixParams, const PagedArgs&, float*, float*, cudaStream_t);

// pairs of row tiles of a group
__host__ __device__ inline int row_pairs(int members, int nb) { return (members + 2 * nb - 1) / (2 * nb); }

}  // namespace atc_gb300

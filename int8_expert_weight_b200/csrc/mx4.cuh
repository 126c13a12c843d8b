// Arguments and group table of the MX4 products grouped by expert.
#pragma once

#include "common.cuh"

namespace jmoe {
namespace mx4 {

constexpr int kMaxGroups = 256;

struct Args {
    WsHeader* hdr;         // device status word
    const int32_t* begin;  // first row of each expert
    const int32_t* count;  // rows of each expert, or NULL: begin has E + 1 entries and expert e ends at begin[e + 1]
    int E;                 // experts
    int reset_status;      // this call owns the status word: clear it, and report a bad group table there
    int64_t N;             // rows of x
    int64_t rows;          // of them at most in groups
    const uint8_t* xq;     // x codes [N][K / 2] and scales [N][K / 32]
    const uint8_t* xs;
    const uint8_t* qa;     // weights W (dual: W1) codes [E][M][K / 2] and scales [E][M][K / 32]
    const uint8_t* sa;
    const uint8_t* qb;     // dual: W3, else NULL
    const uint8_t* sb;
    const int32_t* perm;   // slot: assignment of each row, -1 = padding
    const float* wts;      // slot: routing weight of each assignment, else NULL
    uint16_t* y16;         // plain: y in bf16; dual: h
    float* y32;            // plain: y in fp32; slot: out [T*K][M]
    int K;                 // reduction length
    int M;                 // weight rows per expert and matrix
    int n_wt;              // weight tiles per expert (set by the launcher)
    int vec_scales;        // rows of scales are whole 32-byte pieces on 32-byte boundaries (set by the launcher)
    int band_max;          // token tiles per L2 band, at most (set by the launcher)
};

// Rows of expert e.  Returns whether its entries break the rule 0 <= begin, 0 <= count, begin + count <= N; as offsets
// (count NULL) that all keep it are in ascending order.
__device__ __forceinline__ bool group_at(const Args& p, int e, int64_t& row0, int& count) {
    const int64_t b = p.begin[e];
    const int64_t c = p.count ? p.count[e] : p.begin[e + 1] - b;
    const bool bad = b < 0 || c < 0 || b + c > p.N;
    row0 = bad ? 0 : b;
    count = bad ? 0 : (int)c;
    return bad;
}

}  // namespace mx4
}  // namespace jmoe

// MX4 rounding (see quantize_mx4.cu), and the arguments and group table of the products grouped by expert.
#pragma once

#include "common.cuh"

namespace jmoe {

// Largest magnitude (bf16 bits) of the 8 values of a chunk.
__device__ __forceinline__ uint32_t chunk_amax(const uint4& v) {
    const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m2 & 0xFFFFu, m2 >> 16);
}

// E8M0 scale byte of a block from its largest magnitude (bf16 bits).
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
    if (amax >= 0x7F80u) return 255u;
    if (amax == 0) return 127u;
    return (uint32_t)max((int)(amax >> 7) - 2, 0);
}

// Codes of the 8 values of a chunk, element i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t mx_codes(const uint4& v, uint32_t s) {
    if (s == 255u) return 0u;
    const float r = __uint_as_float((254u - s) << 23);  // 1 / scale = 2^(127 - s)
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16) * r;
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * r;
    }
    uint32_t out;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return out;
}

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
    uint8_t* hq;           // dual: h's codes [N][M / 2] and scales [N][M / 32], M a multiple of 32
    uint8_t* hs;
    uint16_t* y16;         // plain: y in bf16
    float* y32;            // plain: y in fp32; slot: out [T*K][M]
    int K;                 // reduction length
    int M;                 // weight rows per expert and matrix
    int n_wt;              // weight tiles per expert (set by the launcher)
    int skip_copy;         // test hook, heeded while it is on: CTA 0 skips the copies of its second stage
    uint32_t max_polls;    // bound of every mbarrier wait (set by the launcher)
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

// MX4 quantization and its inverse (OCP Microscaling Formats v1.0, MXFP4): 32 consecutive elements of
// a row share one E8M0 scale 2^(s - 127), each element is an E2M1 number (1 sign, 2 exponent bits with
// bias 1, 1 mantissa bit: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}), two codes to a byte, the even element low.
//
// The scale of a block with largest magnitude m > 0 is 2^(floor(log2 m) - 2), so that m / scale lies
// in [4, 8) and 4, the lower end of E2M1's last binade, is reached by every block; on bf16 bits that
// is s = max(E - 2, 0) with E the exponent field of m (subnormal m: E = 0; 2^-127 is the least
// E8M0 scale).  A block of zeros gets s = 127 (scale 1); a block holding a NaN or an infinity gets
// s = 255 (E8M0's NaN) and codes 0.  v / scale is a multiplication by a power of two, exact in fp32
// (the result is at most 8 in magnitude, and what falls below 2^-126 rounds to code 0 either way),
// so the hardware's conversion (nearest, ties to even, saturating at +-6) of that product is the
// correctly rounded code: no residual check as for the int8 and E4M3 codes is needed.
//
// HBM-bound: 2 bytes read and 17/32 written per element (and the reverse).  Blocks never straddle
// rows (cols is a multiple of 32), so both kernels walk the matrices as one flat run of 16-element
// chunks: two neighbouring lanes hold a block, a thread reads (quantization) or writes 32 bytes at a time.
#include <cuda_fp16.h>

#include "mx4.cuh"

namespace jmoe {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;  // chunks a thread has in flight

// 16 bf16 values; kWide: on a 32-byte boundary, else on a 16-byte one.  Each is read or written once.
struct Chunk {
    uint4 a, b;
};
template <bool kWide>
__device__ __forceinline__ Chunk ld_chunk(const uint16_t* p) {
    Chunk c;
    if constexpr (kWide)
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(c.a.x), "=r"(c.a.y), "=r"(c.a.z), "=r"(c.a.w), "=r"(c.b.x), "=r"(c.b.y), "=r"(c.b.z),
                       "=r"(c.b.w)
                     : "l"(p));
    else
        c = Chunk{ld_stream_v4(p), ld_stream_v4(p + 8)};
    return c;
}
template <bool kWide>
__device__ __forceinline__ void st_chunk(uint16_t* p, const uint32_t (&o)[8]) {
    if constexpr (kWide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

template <bool kWide>
__global__ void __launch_bounds__(kMxThreads) quantize_mx4_kernel(const uint16_t* __restrict__ W, int64_t chunks,
                                                                  uint8_t* __restrict__ Q, uint8_t* __restrict__ S) {
    pdl_wait();
    pdl_trigger();
    const int64_t step = (int64_t)gridDim.x * kMxThreads;
    // every lane of a warp takes part in the shuffles; chunks is a multiple of 2, so whole blocks are live
    for (int64_t c0 = (int64_t)blockIdx.x * kMxThreads; c0 < chunks; c0 += kMxUnroll * step) {
        Chunk v[kMxUnroll];
#pragma unroll
        for (int u = 0; u < kMxUnroll; ++u) {
            const int64_t c = c0 + u * step + threadIdx.x;
            v[u] = c < chunks ? ld_chunk<kWide>(W + c * 16) : Chunk{};
        }
#pragma unroll
        for (int u = 0; u < kMxUnroll; ++u) {
            const int64_t c = c0 + u * step + threadIdx.x;
            const uint32_t m = max(chunk_amax(v[u].a), chunk_amax(v[u].b));
            const uint32_t s = mx_scale(max(m, __shfl_xor_sync(0xffffffffu, m, 1)));
            if (c >= chunks) continue;
            *reinterpret_cast<uint2*>(Q + c * 8) = make_uint2(mx_codes(v[u].a, s), mx_codes(v[u].b, s));
            if ((c & 1) == 0) S[c >> 1] = (uint8_t)s;
        }
    }
}

// The layer's x in permuted order: the codes and scales of token t go to the rows inv[t * K + k] of its K assignments,
// so a token is read and rounded once.  An assignment that the permutation skipped (a routing id out of range: its
// row does not name it) is left out.  One CTA per token.
template <bool kWide>
__global__ void __launch_bounds__(kMxThreads)
    quantize_mx4_tokens_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ inv,
                               const int32_t* __restrict__ perm, int64_t T, int64_t cap_rows, int cols,
                               uint8_t* __restrict__ Q, uint8_t* __restrict__ S) {
    pdl_wait();
    pdl_trigger();
    const int chunks = cols / 16;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int64_t rows[kTopK];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            const int32_t r = inv[t * kTopK + k];
            rows[k] = r >= 0 && r < cap_rows && perm[r] == t * kTopK + k ? r : -1;
        }
        for (int c0 = 0; c0 < chunks; c0 += blockDim.x) {  // chunks is even and a block is two lanes of one warp
            const int c = c0 + threadIdx.x;
            const Chunk v = c < chunks ? ld_chunk<kWide>(x + t * cols + (int64_t)c * 16) : Chunk{};
            const uint32_t m = max(chunk_amax(v.a), chunk_amax(v.b));
            const uint32_t s = mx_scale(max(m, __shfl_xor_sync(0xffffffffu, m, 1)));
            if (c >= chunks) continue;
            const uint2 q = make_uint2(mx_codes(v.a, s), mx_codes(v.b, s));
#pragma unroll
            for (int k = 0; k < kTopK; ++k) {
                if (rows[k] < 0) continue;
                *reinterpret_cast<uint2*>(Q + rows[k] * (cols / 2) + c * 8) = q;
                if ((c & 1) == 0) S[rows[k] * (cols / 32) + (c >> 1)] = (uint8_t)s;
            }
        }
    }
}

// Values of 8 codes times `scale` as bf16 pairs.
__device__ __forceinline__ void mx_values(uint32_t q, float scale, uint32_t* o) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        o[i] = (uint32_t)f32_to_bf16_bits(f.x * scale) | ((uint32_t)f32_to_bf16_bits(f.y * scale) << 16);
    }
}

// The inverse: code x scale as bf16, exact (an E2M1 number has two significant bits, and the least
// magnitude, 2^-128, is a bf16 subnormal); products beyond bf16's range become infinities, a scale byte of 255 NaN.
template <bool kWide>
__global__ void __launch_bounds__(kMxThreads) dequantize_mx4_kernel(const uint8_t* __restrict__ Q,
                                                                    const uint8_t* __restrict__ S, int64_t chunks,
                                                                    uint16_t* __restrict__ W) {
    pdl_wait();
    pdl_trigger();
    const int64_t step = (int64_t)gridDim.x * kMxThreads;
    for (int64_t c0 = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; c0 < chunks; c0 += kMxUnroll * step) {
        uint2 q[kMxUnroll];
        uint32_t s[kMxUnroll];
#pragma unroll
        for (int u = 0; u < kMxUnroll; ++u) {
            const int64_t c = c0 + u * step;
            q[u] = c < chunks ? __ldg(reinterpret_cast<const uint2*>(Q + c * 8)) : make_uint2(0, 0);
            s[u] = c < chunks ? __ldg(S + (c >> 1)) : 127u;
        }
#pragma unroll
        for (int u = 0; u < kMxUnroll; ++u) {
            const int64_t c = c0 + u * step;
            if (c >= chunks) continue;
            const float sc = s[u] == 255u ? __uint_as_float(0x7FC00000u)
                                          : __uint_as_float(s[u] == 0 ? 0x00400000u : s[u] << 23);
            uint32_t o[8];
            mx_values(q[u].x, sc, o);
            mx_values(q[u].y, sc, o + 4);
            st_chunk<kWide>(W + c * 16, o);
        }
    }
}

// CTAs: one per 256 chunks, up to per_sm for each SM.  More than are resident at once (8): CTAs that end and start
// drift apart and keep reads and writes going together.  16 x 4096 x 14336, per_sm 8 / 64 / 256: quantization 356 /
// 343 / 362 us, inverse 431 / 371 / 359 us.
static unsigned mx_blocks(int64_t chunks, int num_sms, int per_sm) {
    int64_t blocks = (chunks + kMxThreads - 1) / kMxThreads;
    const int64_t cap = (int64_t)num_sms * per_sm;
    return (unsigned)(blocks > cap ? cap : (blocks < 1 ? 1 : blocks));
}

// elements % 32 == 0.
cudaError_t launch_quantize_mx4(const uint16_t* W, int64_t elements, uint8_t* Q, uint8_t* S, cudaStream_t st,
                                int num_sms) {
    const auto kernel =
        reinterpret_cast<uintptr_t>(W) % 32 == 0 ? quantize_mx4_kernel<true> : quantize_mx4_kernel<false>;
    return launch_pdl(kernel, dim3(mx_blocks(elements / 16, num_sms, 64)), dim3(kMxThreads), 0, st, W,
                      elements / 16, Q, S);
}

cudaError_t launch_quantize_mx4_tokens(const uint16_t* x, const int32_t* inv, const int32_t* perm, int64_t T,
                                       int64_t cap_rows, int64_t cols, uint8_t* Q, uint8_t* S, cudaStream_t st,
                                       int num_sms) {
    const int64_t cap = (int64_t)num_sms * 16;
    const int threads = cols / 16 >= kMxThreads ? kMxThreads : (int)(cols / 16 + 31) / 32 * 32;
    const auto kernel =
        reinterpret_cast<uintptr_t>(x) % 32 == 0 ? quantize_mx4_tokens_kernel<true> : quantize_mx4_tokens_kernel<false>;
    return launch_pdl(kernel, dim3((unsigned)(T > cap ? cap : T)), dim3(threads), 0, st, x, inv, perm, T, cap_rows,
                      (int)cols, Q, S);
}

cudaError_t launch_dequantize_mx4(const uint8_t* Q, const uint8_t* S, int64_t elements, uint16_t* W, cudaStream_t st,
                                  int num_sms) {
    const auto kernel =
        reinterpret_cast<uintptr_t>(W) % 32 == 0 ? dequantize_mx4_kernel<true> : dequantize_mx4_kernel<false>;
    return launch_pdl(kernel, dim3(mx_blocks(elements / 16, num_sms, 256)), dim3(kMxThreads), 0, st, Q, S,
                      elements / 16, W);
}

}  // namespace jmoe

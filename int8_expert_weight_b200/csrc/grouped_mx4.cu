// Matrix products grouped by expert on MX4 operands (see quantize_mx4.cu for the format): the rows of
// expert e, begin[e] .. begin[e] + count[e], are multiplied with that expert's weights,
//
//   plain   y[r][i]      = sum_k x^[r][k] W^_e[i][k]                   (bf16 or fp32)
//   slot    out[a][i]    = p_a * sum_k x^[r][k] W^_e[i][k]             (fp32; a = assignment of row r)
//   dual    h[r][j]      = bf16( SiLU(x^[r] . W1^_e[j]) * (x^[r] . W3^_e[j]) )
//
// with v^ the value of an MX4 code times its block's scale, fp32 sums.
//
// CTA = (64 weight rows, one expert), 64 token rows at a time; both operands' codes are expanded to
// fp32 in shared memory a block of 32 k at a time, and each of 256 threads keeps 4 x 4 sums.  A block's
// dot product of E2M1 numbers is exact (multiples of 1/4 below 32 * 36); it is added with the product of
// the two scales, so neither operand's scale alone can overflow or vanish.
#include "mx4.cuh"

namespace jmoe {
namespace mx4 {

constexpr int kTile = 64;
constexpr int kThreads = 256;

// Half of a block's 32 E2M1 numbers into column `col` of a [32][kTile + 4] array.
__device__ __forceinline__ void expand(float (*dst)[kTile + 4], int col, const uint8_t* q, int half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = q[8 * half + i];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint32_t c = (b >> (4 * n)) & 15u, m = c & 7u;
            const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
            dst[16 * half + 2 * i + n][col] = (c & 8u) ? -v : v;
        }
    }
}
__device__ __forceinline__ float scale_of(uint32_t s) {
    return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}

template <bool kDual>
__global__ void __launch_bounds__(kThreads) grouped_kernel(Args p) {
    __shared__ float sx[32][kTile + 4], sa[32][kTile + 4], sb[kDual ? 32 : 1][kTile + 4];
    __shared__ float scx[kTile], sca[kTile], scb[kTile];
    pdl_wait();
    const int e = blockIdx.y;
    if (p.reset_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) check_groups(p);
    int64_t row0;
    int count;
    group_at(p, e, row0, count);
    const int64_t j0 = (int64_t)blockIdx.x * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int lr = threadIdx.x & 63, lq = threadIdx.x >> 6;  // operand row and part this thread expands
    for (int n0 = 0; n0 < count; n0 += kTile) {
        float acc_a[4][4] = {}, acc_b[4][4] = {};
        for (int kb = 0; kb < p.K / 32; ++kb) {
            const int64_t xr = row0 + min(n0 + lr, count - 1);
            const int64_t wr = (int64_t)e * p.M + min(j0 + lr, (int64_t)p.M - 1);
            if (lq < 2) {
                expand(sx, lr, p.xq + xr * (p.K / 2) + kb * 16, lq);
                if (lq == 0) scx[lr] = scale_of(p.xs[xr * (p.K / 32) + kb]);
            } else {
                expand(sa, lr, p.qa + wr * (p.K / 2) + kb * 16, lq - 2);
                if (kDual) expand(sb, lr, p.qb + wr * (p.K / 2) + kb * 16, lq - 2);
                if (lq == 2) sca[lr] = scale_of(p.sa[wr * (p.K / 32) + kb]);
                if (kDual && lq == 3) scb[lr] = scale_of(p.sb[wr * (p.K / 32) + kb]);
            }
            __syncthreads();
            float blk_a[4][4] = {}, blk_b[4][4] = {};
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = sx[k][ty + 16 * i];
                        blk_a[i][j] = fmaf(x, sa[k][tx + 16 * j], blk_a[i][j]);
                        if (kDual) blk_b[i][j] = fmaf(x, sb[kDual ? k : 0][tx + 16 * j], blk_b[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float s = scx[ty + 16 * i];
                    acc_a[i][j] = fmaf(blk_a[i][j], s * sca[tx + 16 * j], acc_a[i][j]);
                    if (kDual) acc_b[i][j] = fmaf(blk_b[i][j], s * scb[tx + 16 * j], acc_b[i][j]);
                }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + ty + 16 * i;
            if (n >= count) continue;
            const int64_t r = row0 + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = j0 + tx + 16 * j;
                if (col >= p.M) continue;
                const float v = acc_a[i][j];
                if (kDual) {
                    p.y16[r * p.M + col] = f32_to_bf16_bits(silu(v) * acc_b[i][j]);
                } else if (p.wts) {
                    const int32_t a = p.perm[r];
                    if (a >= 0) p.y32[(int64_t)a * p.M + col] = p.wts[a] * v;
                } else if (p.y32) {
                    p.y32[r * p.M + col] = v;
                } else {
                    p.y16[r * p.M + col] = f32_to_bf16_bits(v);
                }
            }
        }
    }
}

}  // namespace mx4

cudaError_t launch_grouped_mx4(const mx4::Args& p, cudaStream_t st) {
    using namespace mx4;
    const dim3 grid((unsigned)((p.M + kTile - 1) / kTile), (unsigned)p.E);
    if (p.qb) return launch_pdl(grouped_kernel<true>, grid, dim3(kThreads), 0, st, p);
    return launch_pdl(grouped_kernel<false>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace jmoe

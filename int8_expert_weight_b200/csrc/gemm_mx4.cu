// Matrix products grouped by expert on MX4 operands (see quantize_mx4.cu for the format): the rows of
// expert e, begin[e] .. begin[e] + count[e], are multiplied with that expert's weights,
//
//   plain   y[r][i]      = sum_k x^[r][k] W^_e[i][k]                   (bf16 or fp32)
//   slot    out[a][i]    = p_a * sum_k x^[r][k] W^_e[i][k]             (fp32; a = assignment of row r)
//   dual    h[r][j]      = MX4( bf16( SiLU(x^[r] . W1^_e[j]) * (x^[r] . W3^_e[j]) ) )
//
// with v^ the value of an MX4 code times its block's scale, fp32 sums.  The tensor cores take the codes
// and the scales as they are (tcgen05.mma kind::mxf4.block_scale): nothing is expanded.
//
// One tile = 128 weight rows (the MMA's M, TMEM lanes) x up to kTok rows of one expert (N, TMEM
// columns).  Weights as M: their 128-row tiles are always full, while the rows of an expert, often few,
// only have to fill up a multiple of 16.  The rows of a group start anywhere: a copy of the tile reads past the
// group's end into the next one's rows, whose columns of the result are not stored.
//   dual: rows 32q .. 32q+15 of the tile are W1 rows j0+16q .., rows 32q+16 .. 32q+31 the W3 rows of the
//   same j (q = 0..3), so gate and up of one j sit in lanes l and l + 16 of a warp: the same place of two fragments.
//
// Many rows per expert: a pair of CTAs (cta_group::2) works on 256 weight rows x up to 208 rows of x; each
// holds the codes of its 128 weight rows and of half the rows of x, 29 instead of 43 KB per 256 of K, which is what
// bounds single CTAs (16384 x 14336 x 4096: 627 us single, 573 us in pairs, all else equal).  Few rows: single CTAs,
// tiles of 64 rows of x, the stages full of weights in flight.
//
// Persistent, one CTA per SM, warps in roles; a pipeline stage holds 256 of K (128 bytes of codes per row)
// or, where each tile has few tokens, 512:
//   warp 0      codes: TMA boxes of 128 bytes x 128 (dual: 16) weight rows and x 32 or a full tile's token rows
//   warp 1      TMEM allocator; per stage copies the scales to TMEM (tcgen05.cp) and issues the MMAs, 64 k each.
//   4-6 warps   scales: two sets, in turns, of one warp per 128 rows of weights or tokens.  The tensor core wants
//               512-byte blocks of 128 rows x 128 k with row r at 16 (r % 32) + 4 (r / 32); a lane reads 32 bytes (a
//               DRAM sector: 1024 of K) of rows lane, lane + 32, + 64, + 96 into registers, ahead of their use and
//               across tiles, and stores 16 bytes per block.  (One set, half as far ahead: 94 instead of 86 us on 128
//               rows.)
//   8 warps     epilogue: two warps per TMEM lane quarter, alternate 16-token units
// TMEM: two accumulators of kTok columns, so a tile's epilogue overlaps the next tile's MMAs, and sets of scale
// columns.  Every mbarrier wait is bounded: on timeout the kernel records JMOE_DEV_TIMEOUT in the workspace status
// word, the other roles stop at their next wait, in-flight copies and MMAs are waited for (bounded), TMEM is released
// and the CTA returns.
//
// Tile order: expert by expert; inside an expert, bands of token tiles whose codes stay in L2 while every
// weight tile streams past once per band; token tiles fastest, so the CTAs working at the same time share
// each weight tile.  CTA (or pair) i of n takes tiles i, i + n, ...: DRAM reads are the operands once (16384 x 14336 x
// 4096: 535 MB for 534).
//
// Measured (random codes; B200, 6.46 TB/s copy, 1.71 PFLOP/s bf16): 128 rows over 16 experts, 14336 x 4096: 80 us,
// 6.2 TB/s: HBM.  16384 rows: 421 us in short runs, 4.6 PFLOP/s, tensor pipe 70 % active; back to back for seconds 490 us
// at the 1290 MHz that the power limit leaves, and on constant codes 356 us at 1762 MHz: 630 thousand cycles with either,
// 321 us at the full 1965 MHz, where the operations need 282 at four times the bf16 rate.  (Constant codes in short runs:
// 324 us; an earlier build took 320, 265 of them without the epilogue and 245, the copies alone, without MMAs either.)
// So the power limit sets the pace of long runs, and the pipeline is 14 % from its own.  Tried and dropped: the stages of
// few tiles divided evenly among all CTAs with partial sums through memory (two rows x 4096 x 14336: 18.7 -> 21.1 us,
// the exchange costs what the balance gains), tiles of 64 weight rows (17.0 -> 19.0 us: the stages' pace, not their
// bytes, bounds 64 CTAs), a look at the next stage's barrier between a stage's MMAs (414 -> 427 us).

#include <atomic>

#include "mx4.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace jmoe {
namespace ts {
extern int g_skip_copy;  // set by jamba_moe_debug_skip_copy (tests only)
}
namespace mx4 {

constexpr int kWRows = 128;
constexpr int kSubBytes = 128;    // bytes of codes per row and sub-step: 256 of K
constexpr int kBoxRows = 32;      // token rows per copy
constexpr int kEpiWarps = 8;
constexpr int kOutPitch = 80;     // bytes per token of a warp's 16-token staging area (32 bf16, and no bank conflicts)
constexpr int kOutBytes = 16 * kOutPitch;
constexpr int kSfWords = 8;       // words of scales that a lane holds of each of its rows: 32 bytes
constexpr uint32_t kMaxPolls = 1u << 22;      // ~0.3 s of polling: far above any healthy wait
constexpr uint32_t kTestMaxPolls = 1u << 14;  // short bound used together with the test hook

// kPair: two CTAs work on one tile of 256 weight rows.
template <bool kPair, int kTok>
struct Cfg {
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kTokCta = kTok / kCtas;            // token rows whose codes a CTA holds
    // Sub-steps of 256 k in a stage.  With few tokens a sub-step's MMAs are short and the hand-over of a stage costs as
    // much, so two share one (two rows x 4096 x 14336: 17.5 or 17.0 us; the layer on one token: 67.5 or 63.6 us).
    static constexpr int kSub = kPair ? 1 : 2;
    static constexpr int kWords = 2 * kSub;                 // of 128 k: the scales' unit
    static constexpr int kSfBlocks = (kTok + 127) / 128;    // 512-byte blocks of token scales per word
    static constexpr int kASub = kWRows * kSubBytes, kBSub = kTokCta * kSubBytes;
    static constexpr int kA = kSub * kASub;
    static constexpr int kB = kSub * kBSub;
    static constexpr int kSfA = kWords * 512;
    static constexpr int kSfB = kWords * kSfBlocks * 512;
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = (227 * 1024 - 6 * 1024 - kEpiWarps * kOutBytes) / kStage;
    static constexpr int kSfCols = kWords * 4 * (1 + kSfBlocks);
    static constexpr int kSfCol0 = 2 * kTok;
    static constexpr int kSfSets = (512 - kSfCol0) / kSfCols < kStages ? (512 - kSfCol0) / kSfCols : kStages;
    static constexpr uint32_t kTmemCols = kSfCol0 + kSfSets * kSfCols <= 256 ? 256 : 512;
    static constexpr int kSfStages = kSfWords / kWords;     // stages whose scales a lane holds
    static constexpr int kSfWarps = 1 + kSfBlocks;          // of one set of scale warps
    static constexpr int kEpiWarp0 = 2 + 2 * kSfWarps;
    static constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
    static constexpr int kBars = 2 * kStages + 5;
    static constexpr int kSmem = kStages * kStage + kEpiWarps * kOutBytes + 1024 + 8 * kBars;
    static_assert(kThreads >= kMaxGroups, "one thread per group");
    static_assert(kTok % 16 == 0 && kB % 1024 == 0 && kSfSets >= 2, "tile");
    // A set of scale warps waits for stage g - kSfSets to be consumed and knows, from its last turn, that stage
    // g - kSfStages - 1 - kSfSets was: a barrier's parity says the right thing only if that is not before
    // g - kSfSets - kStages.
    static_assert(kStages > kSfStages, "scale warps would run a round ahead of the barrier they wait on");
};

struct Tile {
    int e = 0, n;  // expert, weight tile
    int64_t row0;  // first row of the token tile
    int ntok;      // its rows (1 .. kTok)
};

// The group table of a call, in shared memory.
struct Groups {
    int tile0[kMaxGroups + 1];  // tiles of the groups before each
    int count[kMaxGroups];
    int row0[kMaxGroups];
};

// Tile L.  t.e is where the search starts: the group of an earlier tile (the role's last one), or 0.
template <int kTok>
__device__ __forceinline__ void tile_at(const Groups& G, const Args& p, int L, Tile& t) {
    int e = t.e;  // to the last group whose first tile is <= L: groups without rows have no tile
    while (e + 1 < p.E && G.tile0[e + 1] <= L) ++e;
    const int count = G.count[e], nt = (count + kTok - 1) / kTok;
    int within = L - G.tile0[e], m_first = 0, bsz = nt;
    if (nt > p.band_max) {  // more token tiles than a band holds: bands as even as possible
        const int nb = (nt + p.band_max - 1) / p.band_max;
        const int bfull = (nt + nb - 1) / nb;
        const int band = within / (bfull * p.n_wt);
        within -= band * bfull * p.n_wt;
        m_first = band * bfull;
        bsz = min(bfull, nt - m_first);
    }
    const int n = within / bsz;
    const int m = m_first + within - n * bsz;
    t.e = e;
    t.n = n;
    t.row0 = (int64_t)G.row0[e] + m * kTok;
    t.ntok = min(kTok, count - m * kTok);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "r"(addr)
                 : "memory");
    return q;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {  // fp32 bits
    return pack_bf16(__uint_as_float(lo), __uint_as_float(hi));
}

__device__ __forceinline__ void fail(WsHeader* hdr, volatile int* abort) {
    *abort = 1;
    set_status(hdr, JMOE_DEV_TIMEOUT);
}

// 16 tokens (the first n of them live) of a warp's 32 TMEM lanes as bf16, y rows row0 .., columns j0 ..: the fragments
// v (see tmem_ld_16x16; lanes 0-15, then 16-31) go transposed through the warp's area `out` of shared memory and
// leave as 16-byte pieces of y rows, element by element where rows are no multiple of 8 long.  (Trading values
// between neighbouring lanes and storing 4 bytes each took 1200 cycles per 16 tokens.)
__device__ __forceinline__ void store_bf16(const Args& p, uint32_t out, const uint32_t (&v)[16], int64_t row0, int n,
                                           int j0, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i)  // 4 j blocks of 8, for each of two token blocks
        tc::stmatrix_x4_trans(out + (8 * i + (lane & 7)) * kOutPitch + 16 * (lane >> 3),
                              pack_bf16(v[4 * i], v[4 * i + 1]), pack_bf16(v[4 * i + 2], v[4 * i + 3]),
                              pack_bf16(v[8 + 4 * i], v[9 + 4 * i]), pack_bf16(v[10 + 4 * i], v[11 + 4 * i]));
    __syncwarp();
    uint16_t* y = p.y16 + row0 * p.M + j0;
    if (p.M % 8 == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = 8 * i + lane / 4, j = 8 * (lane % 4);
            const uint4 q = ld_shared_v4(out + tok * kOutPitch + 2 * j);
            if (tok < n && j0 + j < p.M) *reinterpret_cast<uint4*>(y + (int64_t)tok * p.M + j) = q;
        }
    } else {
        for (int tok = 0; tok < 16 && tok < n; ++tok) {
            uint16_t q;
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(q) : "r"(out + tok * kOutPitch + 2 * lane) : "memory");
            if (j0 + lane < p.M) y[(int64_t)tok * p.M + lane] = q;
        }
    }
    __syncwarp();  // the area is rewritten by the next 16 tokens
}

// dual: SwiGLU of 16 tokens and 16 columns j0 .. of h: gate and up of one j are in lanes l and l + 16, so in the same
// place of the two halves of v.  As bf16 transposed through `out`; returned: 8 values of h, of token lane / 2 and
// columns j0 + 8 (lane % 2) ...
__device__ __forceinline__ uint4 swiglu_bf16(uint32_t out, const uint32_t (&v)[16], int lane) {
    constexpr int kPitch = 48;
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // 2 j blocks x 2 token blocks of 8
        m[i] = pack_bf16(silu_fast(__uint_as_float(v[2 * i])) * __uint_as_float(v[8 + 2 * i]),
                         silu_fast(__uint_as_float(v[2 * i + 1])) * __uint_as_float(v[9 + 2 * i]));
    tc::stmatrix_x4_trans(out + (8 * (lane >> 4) + (lane & 7)) * kPitch + 16 * ((lane >> 3) & 1), m[0], m[1], m[2],
                          m[3]);
    __syncwarp();
    const uint4 q = ld_shared_v4(out + (lane >> 1) * kPitch + 16 * (lane & 1));
    __syncwarp();  // the area is rewritten by the next 16 tokens
    return q;
}

// 16 tokens (the first n of them live) of column j as fp32: y rows row0 .., or, times their routing weights, the slots
// of their assignments.
__device__ __forceinline__ void store_fp32(const Args& p, const uint32_t (&v)[16], int64_t row0, int n, int j,
                                           int lane) {
    if (p.wts) {
        const int32_t a_l = lane < min(n, 16) ? p.perm[row0 + lane] : -1;
        const float w_l = a_l >= 0 ? p.wts[a_l] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int32_t a = __shfl_sync(0xffffffffu, a_l, i);
            const float wt = __shfl_sync(0xffffffffu, w_l, i);
            if (a >= 0 && j < p.M) p.y32[(int64_t)a * p.M + j] = wt * __uint_as_float(v[i]);
        }
    } else {
        float* y = p.y32 + row0 * p.M + j;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n && j < p.M) y[(int64_t)i * p.M] = __uint_as_float(v[i]);
    }
}

// 32 bytes of scales; `vec`: 32-byte aligned and whole, else `words` 4-byte words of them are there.
__device__ __forceinline__ void ld_scales(const uint8_t* ptr, bool vec, int words, uint32_t (&v)[kSfWords]) {
    if (vec) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(ptr));
    } else {
#pragma unroll
        for (int i = 0; i < kSfWords; ++i)
            v[i] = i < words ? __ldg(reinterpret_cast<const uint32_t*>(ptr) + i) : 0u;
    }
}

template <bool kDual, bool kPair, int kTok>
__global__ void __launch_bounds__(Cfg<kPair, kTok>::kThreads, 1)
    gemm_mx4_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                    const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1, Args p) {
    using C = Cfg<kPair, kTok>;
    constexpr int kStages = C::kStages, kSfStages = C::kSfStages, kWords = C::kWords, kEpiWarp0 = C::kEpiWarp0;
    constexpr int kRowsCta = kDual ? kWRows / 2 : kWRows;  // weight rows (of each matrix) of a CTA's part of a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ Groups G;
    __shared__ int warp_sum[C::kThreads / 32];
    __shared__ uint32_t amax_sh[kDual ? kEpiWarps : 1][2][16];  // dual: largest |h| of 16 tokens over a warp's columns
    __shared__ uint32_t tmem_holder;
    __shared__ volatile int abort_flag;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    pdl_wait();
    pdl_trigger();  // the next kernel's CTAs may take their places beside this one's; they wait for its end
    // ---- group table: thread e takes group e
    {
        const int e = threadIdx.x;
        int64_t row0 = 0;
        int count = 0;
        bool bad = false;
        if (e < p.E) {
            bad = group_at(p, e, row0, count);
            G.count[e] = count;
            G.row0[e] = (int)row0;
        }
        bad = __syncthreads_or(bad);
        if (p.reset_status && blockIdx.x == 0 && e == 0) p.hdr->status = bad ? JMOE_DEV_BAD_INDEX : JMOE_OK;
        if (bad) return;  // from here on the groups are in order and apart
        const int tiles = (count + kTok - 1) / kTok * p.n_wt;
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += warp_sum[w];
        if (e < p.E) G.tile0[e] = sum - tiles;
        if (e == p.E - 1) G.tile0[p.E] = sum;
        __syncthreads();
    }
    const int total = G.tile0[p.E];
    const int rank = kPair ? (int)tc::cluster_rank() : 0;                      // 0: the CTA that issues the MMAs
    const int first = (int)blockIdx.x / C::kCtas, stride = (int)gridDim.x / C::kCtas;  // this CTA's tiles
    if (first >= total) return;  // no tile for this CTA (or pair): nothing was taken yet

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;                          // [kStages][kSub][128 rows][128 B]
    uint8_t* sB = sA + kStages * C::kA;          // [kStages][kSub][kTokCta rows][128 B]
    uint8_t* sSA = sB + kStages * C::kB;         // [kStages][kWords][512 B]
    uint8_t* sSB = sSA + kStages * C::kSfA;      // [kStages][kWords][kSfBlocks][512 B]
    uint8_t* sOut = sSB + kStages * C::kSfB;     // [kEpiWarps][16 tokens][kOutPitch]
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + kEpiWarps * kOutBytes);  // [kStages] codes and scales are there
    uint64_t* empty = full + kStages;            // [kStages] MMAs reading the stage are done
    uint64_t* acc_full = empty + kStages;        // [2] accumulator complete
    uint64_t* acc_empty = acc_full + 2;          // [2] accumulator read out by the epilogue
    uint64_t* mma_done = acc_empty + 2;          // every issued MMA complete (after an abort)

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1 + C::kCtas * C::kSfWarps);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], C::kCtas * kEpiWarps);
        }
        tc::mbar_init(mma_done, 1);
        abort_flag = 0;
        tc::mbar_fence_init();
    }
    if (warp == 0 && lane == 0) {
        tc::prefetch_tmap(&tmX);
        tc::prefetch_tmap(&tmXs);
        tc::prefetch_tmap(&tmW0);
        if (kDual) tc::prefetch_tmap(&tmW1);
    }
    if (warp == 1) {
        if constexpr (kPair)
            tc::tmem_alloc_pair(&tmem_holder, C::kTmemCols);
        else
            tc::tmem_alloc(&tmem_holder, C::kTmemCols);
    }
    tc::tc_fence_before();
    __syncthreads();
    if constexpr (kPair) tc::cluster_sync();  // the peer's barriers are there before anything arrives on them
    tc::tc_fence_after();
    const uint32_t tmem = tmem_holder;
    const int KW = p.K / 128;          // 4-byte words of scales per row
    const int KB = (KW + kWords - 1) / kWords;  // stages per tile; the last need not be whole
    int issued = 0;                    // codes: stages copied; MMA issuer: stages multiplied
    auto wait = [&](uint64_t* bar, int round) -> bool {
        if (tc::mbar_wait_bounded<kPair>(bar, round & 1, &abort_flag, p.max_polls)) return true;
        if (!abort_flag) fail(p.hdr, &abort_flag);
        return false;
    };
    // The same outcome for all lanes of a warp, where what follows needs them together.
    auto wait_warp = [&](uint64_t* bar, int round) -> bool { return __all_sync(0xffffffffu, wait(bar, round)); };
    // The two issuing warps: every lane walks the loop and waits, one elected lane issues.  Inside a tile nothing needs
    // the lanes together (one may give up alone); after each tile they agree whether to go on.  (Lane 0 as the issuer,
    // in place of an elected lane: 570 instead of 425 us for the large product; only the issuing lane in the loop:
    // 485; a vote on each wait: 450.)
    const bool lead = tc::elect_one();
    // Arrive on the barrier of the CTA that issues the MMAs.  Its copies and MMAs for the pair then read this CTA's
    // scales, or overwrite its accumulator.  Scales: each lane's fence into the async proxy, the warp's barrier, release
    // and acquire at cluster scope (kPair), the issuer's copies.  Accumulator: tcgen05 fences before the arrival and
    // after the issuer's wait.
    auto arrive = [&](uint64_t* bar) {
        if constexpr (kPair)
            tc::mbar_arrive_cluster(tc::map_to_cta(tc::smem_u32(bar), 0));
        else
            tc::mbar_arrive(bar);
    };

    if (warp == 0) {
        // ---------------- codes: this CTA's weight rows and its half (kPair) of the token rows; the first CTA's
        // barrier counts the bytes of both
        int g = 0;
        bool ok = true;
        Tile t;
        for (int L = first; L < total; L += stride) {
            tile_at<kTok>(G, p, L, t);
            const int w_row0 = t.e * p.M + (t.n * C::kCtas + rank) * kRowsCta;
            const int part = ((t.ntok + 15) & ~15) / C::kCtas;  // this CTA's token rows
            const int x_row0 = (int)t.row0 + rank * part;
            // one copy for a tile (nearly) full of tokens, else the 32-row boxes it needs
            const int n_box = part > C::kTokCta / kBoxRows * kBoxRows ? 0 : (part + kBoxRows - 1) / kBoxRows;
            const uint32_t sub_bytes = C::kCtas * (C::kASub + (n_box == 0 ? C::kTokCta : n_box * kBoxRows) * kSubBytes);
            for (int kb = 0; kb < KB; ++kb, ++g) {
                const int s = g % kStages, r = g / kStages;
                if (r > 0 && !(ok = wait(&empty[s], r - 1))) break;
                if (p.skip_copy && blockIdx.x == 0 && g == 1) continue;
                const int n_sub = min(C::kSub, (KW - kb * kWords + 1) / 2);
                if (lead) {
                    if (rank == 0) tc::mbar_arrive_expect_tx(&full[s], n_sub * sub_bytes);
                    for (int sub = 0; sub < n_sub; ++sub) {
                        const int x = (kb * C::kSub + sub) * kSubBytes;
                        auto load = [&](uint8_t* dst, const CUtensorMap* tm, int row) {
                            if constexpr (kPair)
                                tc::tma_load_2d_pair(dst, tm, tc::map_to_cta(tc::smem_u32(&full[s]), 0), x, row);
                            else
                                tc::tma_load_2d(dst, tm, &full[s], x, row);
                        };
                        uint8_t* da = sA + s * C::kA + sub * C::kASub;
                        uint8_t* db = sB + s * C::kB + sub * C::kBSub;
                        if (kDual) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                load(da + q * 32 * kSubBytes, &tmW0, w_row0 + 16 * q);
                                load(da + (q * 32 + 16) * kSubBytes, &tmW1, w_row0 + 16 * q);
                            }
                        } else {
                            load(da, &tmW0, w_row0);
                        }
                        if (n_box == 0) load(db, &tmX, x_row0);
                        for (int i = 0; i < n_box; ++i)
                            load(db + i * kBoxRows * kSubBytes, &tmXs, x_row0 + i * kBoxRows);
                    }
                }
                issued = g + 1;
            }
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        // the last stages' arrivals come from the other CTA: they have to be here before this one may end
        if (kPair)
            for (int s = 0; ok && s < kStages && s < g; ++s) ok = wait(&empty[s], (g - 1 - s) / kStages);
    } else if (warp < kEpiWarp0 && warp >= 2) {
        // ---------------- scales: two sets of warps take turns by kSfStages stages; the first warp of a set takes the
        // weights' scales, each other one those of 128 token rows
        const int set = (warp - 2) / C::kSfWarps, blk = (warp - 2) % C::kSfWarps - 1;
        const int64_t row_bytes = p.K / 32;
        const uint32_t dst0 = tc::smem_u32(blk < 0 ? sSA : sSB + 512 * blk) + 16 * lane;
        const uint32_t dst_stage = blk < 0 ? C::kSfA : C::kSfB;
        const uint32_t dst_word = blk < 0 ? 512 : 512 * C::kSfBlocks;
        // what is loaded next: rows 32 i + lane (i < live) of tile L, from the tile's stage kb on, which is this CTA's
        // stage g_load
        const uint8_t* ptr[4] = {};
        int L = first, kb = 0, g_load = 0, live = 0, opened = -1;
        Tile t;
        auto open_tile = [&]() {
            tile_at<kTok>(G, p, L, t);
            opened = L;
            const int n_mma = (t.ntok + 15) & ~15;
            live = blk < 0 ? 4 : max(0, min(4, (n_mma - 128 * blk + 31) / 32));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 32 * i + lane;
                // rows past the expert's (or the matrix's) last: any valid row, their results are not stored
                if (blk < 0) {
                    const int j = (t.n * C::kCtas + rank) * kRowsCta + (kDual ? 16 * i + (lane & 15) : r);
                    ptr[i] = (kDual && lane >= 16 ? p.sb : p.sa) + ((int64_t)t.e * p.M + min(j, p.M - 1)) * row_bytes;
                } else {
                    const int64_t row = t.row0 + 128 * blk + r;
                    ptr[i] = p.xs + (row < p.N ? row : p.N - 1) * row_bytes;
                }
            }
        };
        auto skip = [&]() {
            g_load += min(kSfStages, KB - kb);
            kb += kSfStages;
            if (kb >= KB) {
                kb = 0;
                L += stride;
            }
        };
        // Loads this set's next stages; returns how many (0: past the last tile), `at`: the first one.
        auto fetch = [&](uint32_t (&v)[4][kSfWords], int& at) -> int {
            if (L >= total) return 0;
            if (opened != L) open_tile();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < live) ld_scales(ptr[i] + 4 * kWords * kb, p.vec_scales, KW - kWords * kb, v[i]);
            at = g_load;
            const int n = min(kSfStages, KB - kb);
            skip();
            if (L < total) skip();
            return n;
        };
        uint32_t cur[4][kSfWords] = {}, nxt[4][kSfWords] = {};
        if (set == 1) skip();
        int g = 0, g_next = 0;
        bool ok = true;
        for (int n = fetch(cur, g); ok && n > 0;) {
            const int n_next = fetch(nxt, g_next);
#pragma unroll
            for (int st = 0; st < kSfStages; ++st) {
                if (st >= n) break;
                // the stage's place in shared memory is free, and so are its scale columns in TMEM, of which there may
                // be fewer sets than stages: the issuer need not look after those
                const int s = (g + st) % kStages, before = g + st - C::kSfSets;
                if (!(ok = before < 0 || wait_warp(&empty[before % kStages], before / kStages))) break;
#pragma unroll
                for (int w = 0; w < kWords; ++w)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst0 + s * dst_stage + w * dst_word),
                                 "r"(cur[0][kWords * st + w]), "r"(cur[1][kWords * st + w]),
                                 "r"(cur[2][kWords * st + w]), "r"(cur[3][kWords * st + w])
                                 : "memory");
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&full[s]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < kSfWords; ++j) cur[i][j] = nxt[i][j];
            n = n_next;
            g = g_next;
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer
        const uint64_t adesc0 = tc::sw128_kmajor_desc(tc::smem_u32(sA));
        const uint64_t bdesc0 = tc::sw128_kmajor_desc(tc::smem_u32(sB));
        const uint64_t sadesc0 = tc::linear_desc(tc::smem_u32(sSA)), sbdesc0 = tc::linear_desc(tc::smem_u32(sSB));
        auto commit = [](uint64_t* bar) {
            if constexpr (kPair)
                tc::mma_commit_pair(bar);
            else
                tc::mma_commit(bar);
        };
        int g = 0, it = 0;
        bool ok = true;
        Tile t;
        for (int L = first; L < total; L += stride, ++it) {
            tile_at<kTok>(G, p, L, t);
            const int n_mma = (t.ntok + 15) & ~15;
            const uint32_t idesc0 = tc::idesc_mx4_f32(C::kCtas * kWRows, n_mma, 0);
            const uint32_t idesc2 = tc::idesc_mx4_f32(C::kCtas * kWRows, n_mma, 2);
            const int buf = it & 1, u = it >> 1;
            if (u > 0 && !(ok = wait_warp(&acc_empty[buf], u - 1))) break;
            const uint32_t d_tmem = tmem + (uint32_t)(buf * kTok);
            for (int kb = 0; kb < KB; ++kb, ++g) {
                const int s = g % kStages, r = g / kStages;
                if (!(ok = wait(&full[s], r))) break;
                tc::tc_fence_after();
                if (lead) {
                    const uint32_t sf = tmem + C::kSfCol0 + (uint32_t)(g % C::kSfSets * C::kSfCols);
                    const uint64_t adesc = adesc0 + (uint32_t)(s * (C::kA >> 4));
                    const uint64_t bdesc = bdesc0 + (uint32_t)(s * (C::kB >> 4));
                    const uint64_t sadesc = sadesc0 + (uint32_t)(s * (C::kSfA >> 4));
                    const uint64_t sbdesc = sbdesc0 + (uint32_t)(s * (C::kSfB >> 4));
                    // 512 bytes = +32 in a descriptor's address field; a last stage need not hold all words
                    const int words = min(kWords, KW - kb * kWords);
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const uint32_t sfa = sf + 4 * w, sfb = sf + 4 * kWords + 4 * C::kSfBlocks * w;
                        tc::tmem_cp_32x16<kPair>(sfa, sadesc + 32 * w);
#pragma unroll
                        for (int i = 0; i < C::kSfBlocks; ++i)
                            tc::tmem_cp_32x16<kPair>(sfb + 4 * i, sbdesc + 32 * (C::kSfBlocks * w + i));
                    }
                    // 64 k = 32 bytes of the 128-byte row = +2 in the address field
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        if (w < words) {
                            const uint32_t sfa = sf + 4 * w, sfb = sf + 4 * kWords + 4 * C::kSfBlocks * w;
                            const uint64_t a = adesc + (w >> 1) * (C::kASub >> 4) + 4 * (w & 1);
                            const uint64_t b = bdesc + (w >> 1) * (C::kBSub >> 4) + 4 * (w & 1);
                            tc::mma_mx4_ss<kPair>(d_tmem, a, b, idesc0, sfa, sfb, (kb | w) != 0);
                            tc::mma_mx4_ss<kPair>(d_tmem, a + 2, b + 2, idesc2, sfa, sfb, 1);
                        }
                    }
                    commit(&empty[s]);
                    if (kb == KB - 1) commit(&acc_full[buf]);
                }
                issued = g + 1;
            }
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        if (!ok && lead) commit(mma_done);  // arrives once every MMA issued above has completed
        __syncwarp();
    } else if (warp >= kEpiWarp0) {
        // ---------------- epilogue, 16 tokens at a time
        const int qd = warp & 3, ew = warp - kEpiWarp0, part = ew >> 2;
        const bool bf16 = kDual || p.y16;
        int it = 0, swaps = 0;
        Tile t;
        for (int L = first; L < total; L += stride, ++it) {
            tile_at<kTok>(G, p, L, t);
            const int b = it & 1, u = it >> 1;
            bool ok = wait_warp(&acc_full[b], u);
            // the two warps that trade magnitudes stop together or not at all
            if constexpr (kDual) ok = !tc::named_sync_or(1 + (ew >> 1), 64, !ok);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16) + (uint32_t)(b * kTok);
            const uint32_t out = tc::smem_u32(sOut + ew * kOutBytes);
            const int n_unit = (t.ntok + 15) / 16;  // this warp's: part, part + 2, ...
            const int j0 = (t.n * C::kCtas + rank) * kRowsCta + (kDual ? 16 : 32) * qd;  // its first column of y (or h)
            auto release = [&]() {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&acc_empty[b]);
            };
            // bf16: two fragments (16 lanes x 8 tokens) of TMEM lanes 0-15 and two of lanes 16-31 of the quarter;
            // fp32: 16 tokens of this thread's lane
            auto load = [&](int unit, uint32_t (&v)[16]) {
                if (bf16) {
                    tc::tmem_ld_16x16(t_lane + (uint32_t)(16 * unit), v);
                    tc::tmem_ld_16x16(t_lane + (16u << 16) + (uint32_t)(16 * unit), v + 8);
                } else {
                    tc::tmem_ld16(t_lane + (uint32_t)(16 * unit), v);
                }
            };
            uint32_t next[16];
            if (part < n_unit) load(part, next);
            for (int unit = part; unit < n_unit; unit += 2) {
                tc::tmem_wait_ld();
                uint32_t v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = next[i];
                if (unit + 2 < n_unit)
                    load(unit + 2, next);
                else
                    release();
                const int64_t row0 = t.row0 + 16 * unit;
                const int n = t.ntok - 16 * unit;
                if constexpr (kDual) {
                    // h's blocks of 32 are the columns of two neighbouring warps: they trade each token's largest |h|
                    const uint4 h = swiglu_bf16(out, v, lane);
                    uint32_t amax = chunk_amax(h);
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    if ((lane & 1) == 0) amax_sh[ew][swaps & 1][lane >> 1] = amax;
                    tc::named_sync(1 + (ew >> 1), 64);
                    amax = max(amax, amax_sh[ew ^ 1][swaps & 1][lane >> 1]);
                    ++swaps;
                    const uint32_t s = mx_scale(amax);
                    const int tok = lane >> 1, j = j0 + 8 * (lane & 1);
                    if (tok < n && j < p.M) {
                        *reinterpret_cast<uint32_t*>(p.hq + (row0 + tok) * (p.M / 2) + j / 2) = mx_codes(h, s);
                        if (j % 32 == 0) p.hs[(row0 + tok) * (p.M / 32) + j / 32] = (uint8_t)s;
                    }
                } else if (bf16) {
                    store_bf16(p, out, v, row0, n, j0, lane);
                } else {
                    store_fp32(p, v, row0, n, j0 + lane, lane);
                }
            }
            if (part >= n_unit) release();  // a warp whose columns hold no tokens of this tile
        }
    }

    // ---- teardown: after an abort, let in-flight copies and MMAs finish (bounded) before TMEM goes
    tc::tc_fence_before();
    __syncthreads();
    if (abort_flag) {
        if (warp == 0 && lead && rank == 0) {
            for (int s = 0; s < kStages; ++s) {
                if (s >= issued) continue;
                const int last = (issued - 1 - s) / kStages;
                // a copy of round r completes phase `last` of full[s] once the scales are there too; else this wait
                // runs out, long after the copy has landed
                for (uint32_t i = 0; i < p.max_polls && !tc::mbar_try_wait(&full[s], last & 1); ++i) __nanosleep(64);
            }
        }
        // completes if the issuer gave up; if it did not, its last MMAs are long done after this
        if (warp == 1 && lead) {
            for (uint32_t i = 0; i < p.max_polls && !tc::mbar_try_wait(mma_done, 0); ++i) __nanosleep(64);
        }
        __syncthreads();
    }
    // nothing of the pair's is still on its way into the other CTA's shared or tensor memory
    if constexpr (kPair) tc::cluster_sync();
    if (warp == 1) {
        tc::tc_fence_after();
        if constexpr (kPair)
            tc::tmem_dealloc_pair(tmem, C::kTmemCols);
        else
            tc::tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ---------------------------------------------------------------- host side
// Codes [rows][K / 2], boxes of [box_rows][128 bytes].
bool codes_map(CUtensorMap* m, const uint8_t* ptr, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
    return make_map(m, ptr, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, row_bytes, box_rows, kSubBytes,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool kDual, bool kPair, int kTok>
cudaError_t launch(Args p, cudaStream_t st, int num_sms) {
    using C = Cfg<kPair, kTok>;
    CUtensorMap tx, txs, tw0, tw1;
    const uint64_t row_bytes = (uint64_t)p.K / 2, w_rows = (uint64_t)p.E * p.M;
    constexpr uint32_t kWBox = kDual ? 16 : kWRows;
    if (!codes_map(&tx, p.xq, (uint64_t)p.N, row_bytes, C::kTokCta) ||
        !codes_map(&txs, p.xq, (uint64_t)p.N, row_bytes, kBoxRows) || !codes_map(&tw0, p.qa, w_rows, row_bytes, kWBox))
        return cudaErrorInvalidValue;
    tw1 = tw0;
    if (kDual && !codes_map(&tw1, p.qb, w_rows, row_bytes, kWBox)) return cudaErrorInvalidValue;
    const auto kernel = gemm_mx4_kernel<kDual, kPair, kTok>;
    static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared-memory limit raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    constexpr int kRows = C::kCtas * (kDual ? kWRows / 2 : kWRows);
    p.n_wt = (p.M + kRows - 1) / kRows;
    const uintptr_t scales = reinterpret_cast<uintptr_t>(p.xs) | reinterpret_cast<uintptr_t>(p.sa) |
                             reinterpret_cast<uintptr_t>(kDual ? p.sb : p.sa);
    p.vec_scales = p.K % 1024 == 0 && scales % 32 == 0;
    p.max_polls = ts::g_skip_copy ? kTestMaxPolls : kMaxPolls;
    if (!ts::g_skip_copy) p.skip_copy = 0;
    // token tiles per band: the band's codes near 32 MB of L2
    const int64_t per_tile = (int64_t)kTok * (p.K / 2);
    p.band_max = (int)(per_tile >= (32ll << 20) ? 1 : (32ll << 20) / per_tile);
    // persistent: one CTA per SM, fewer when there cannot be that many tiles
    int64_t tiles = (p.rows / kTok + (p.rows < p.E ? p.rows : p.E)) * p.n_wt;
    if (tiles > num_sms / C::kCtas) tiles = num_sms / C::kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles * C::kCtas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::kCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tx, txs, tw0, tw1, p);
}

}  // namespace mx4

cudaError_t launch_grouped_mx4(const mx4::Args& p, cudaStream_t st, int num_sms) {
    using namespace mx4;
    // Few rows per expert: single CTAs with narrow token tiles, whose stages are the weights in flight; else pairs.
    // Single or pairs, us, 14336 x 4096 weights of 16 experts, by rows of each: 4: 79 / 84, 48: 85 / 89, 64: 86 / 90,
    // 96: 104 / 94, 128: 120 / 97.  A group over 64 rows takes two narrow tiles, and uneven groups reach that at a mean
    // of 48.  The host knows the mean alone, of all rows over all experts, so very uneven groups take the slower one:
    // 12288 rows all in one of 256 experts, 4096 x 4096 weights, 157 / 88 (single is taken); 768 in one of 16, 14336 x
    // 4096, 43 / 32 (single); 128 rows in groups of 8 and 16256 of no expert 82 / 86 (pairs).
    const bool few = p.rows <= (int64_t)48 * p.E;
    if (p.qb) return few ? launch<true, false, 64>(p, st, num_sms) : launch<true, true, 208>(p, st, num_sms);
    return few ? launch<false, false, 64>(p, st, num_sms) : launch<false, true, 208>(p, st, num_sms);
}

}  // namespace jmoe

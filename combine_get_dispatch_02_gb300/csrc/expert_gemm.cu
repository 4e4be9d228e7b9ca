// Expert products between dispatch and combine: matrix products grouped by
// expert, whose row groups are the receive rows base[e] .. base[e] + count[e]
// of a layout (counts and bases are read on the device, never on the host).
//   y[r]  = W[e] x[r]                        (bf16, or W stored transposed)
//   y[r]  = act(z[r]) + res[r], z[r] = W[e] x[r] + b[e]   (linear: bf16, all in fp32 with one rounding)
//   y[r]  = sum_b xs[r,b] ws[e,.,b] (Wq[e] xq[r])_b   (e4m3, 128-channel blocks b)
//   h[r]  = cast(silu(g) * u), (g, u) = the two halves of the e4m3 product
//   dW[e] = sum_r dy[r] x[r]^T
//
// One persistent kernel of CTA pairs (a cluster of 2, one CTA per SM).  Tiles:
//   bf16, wgrad      256 rows of the weights (the M side of the tensor cores, 128
//                    per CTA) by up to 256 rows of one expert (the N side, in
//                    steps of 32; wgrad: columns of x)
//   e4m3, column form  the same with two operands of weight rows (gate: 256
//                    channels of the gate and of the up product; else 512 rows) by
//                    up to 128 rows of an expert
//   e4m3, row form   256 rows of an expert on the M side by 256 weight rows
//                    (gate: 128 + 128)
// The weights have no remainders and the tokens are ragged, so with the tokens
// on the N side a group of 40 rows costs 64 columns of products, not a tile of
// 128 or 256 rows; few rows leave the kernel bound by the weights' bytes, many
// by the tensor cores.  The e4m3 products have a scale per row and 128
// channels, so their partial sums leave tensor memory every 128 channels and are
// scaled and added up in fp32 registers; that reading bounds them, and with many
// rows it is cheaper where a thread holds one row and needs one scale (row form,
// from kRowFormRows rows per expert on).  The tiles of an expert are numbered
// with its token tiles fastest and drawn in that order, so pairs that run at the
// same time share its weights in L2.
//
// Warps of a CTA: READ (8, e4m3 row form and linear 16) that read the accumulators out of
// tensor memory, then one that loads (tensor maps, 128-byte swizzle), one that
// issues the products (in the pair's first CTA), one that brings the e4m3
// scales or clears the rows past the end of an expert (wgrad), one that draws
// the tiles.  The accumulators are double buffered (2 x 256 columns).  A segment
// of products shares an accumulator:
//   bf16       the whole sum over k (the next tile's products run while this
//              tile is written out; linear: and while bias, activation and residual,
//              whose rows are asked for a step ahead, are done in the fp32 registers)
//   e4m3       one block of 128 channels
//   wgrad      the whole sum over rows; fp32 output: 256 rows, added up in
//              registers (the tensor cores truncate when they add, and a long
//              sum would drift: 8e-6 of the result over 7168 terms, measured);
//              stored, or added to what is there, by tensor map from shared
//              memory, which also leaves out what lies past the matrix
// Every wait for another role or CTA is bounded; one that gives up sets the status
// word and ends its role.  Not bounded are the hardware's own: for the kernel
// before this one, for tensor memory that another kernel on the SM still holds, for
// stores under way, and for the other CTA at the start and the end.
//
// Measured (one GB300, rows spread evenly unless said; of the 6.78 TB/s copy and
// the 1913 TFLOP/s bf16 peak, 1706 over seconds):
//   bf16   262144 rows x 2048 x 7168    5.0 ms, 1.53 PFLOP/s (power limit), 4.2 ms cold
//          256 experts x 16 rows x 7168 x 2048   1.10 ms, 6.9 TB/s
//   linear 262144 rows x 2048 x 7168, bias, SiLU, z kept   5.2 ms, 1.48 PFLOP/s (power limit), 4.3 ms
//          cold; 512 tokens, top-8 of 256, 7168 x 2048, bias and residual   1.10 ms, 7.0 TB/s
//   wgrad  16 x 1024 rows x 2048 x 7168   278 us, 1.73 PFLOP/s; fp32 output 356 us
//          (0.94 GB, which the tensor cores' work only partly covers), added 421 us
//   e4m3   8192^3   483 us, 2.28 PFLOP/s (row form: reading the partial sums takes
//          about 950 cycles a block, the products 512)
//          76 experts x 16 rows x 4096 x 7168   325 us, 6.9 TB/s; 256 experts x 16
//          rows x 7168 x 2048   545 us, 7.0 TB/s
//   gate   256 experts x 128 rows x 2 * 2048 x 7168   1.17 ms, 6.7 TB/s; 32768
//          entries drawn over 256 experts 1.56 to 1.59 ms (half the experts have more
//          than 128 rows and take two tiles, whose weights come through L2 twice)
//          256 experts x 1024 rows, the same weights   6.7 ms, 2.3 PFLOP/s
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "activation.cuh"
#include "ep_internal.cuh"
#include "umma.cuh"

namespace ep {

namespace {

using namespace umma;

constexpr int kTileRing = 2;      // tiles looked up ahead
constexpr int kNextRing = 4;      // tile numbers on their way to the second CTA
constexpr int kScaleGroup = 4;    // 128-channel blocks per fill of the scale buffer
constexpr int kMaxSmem = 232448;
// Mean rows per expert from which the e4m3 products take the row form.  Up to 128
// rows the column form needs one tile and the weights' bytes bound it; past that
// it takes two.  Of nine shapes (gate and plain product, n and k of 1024 to 7168, 16 to
// 128 experts) with the same rows in every expert, all had the column form ahead up to
// 128 rows (by 1.13 to 1.7 times) and the row form at 136 to 256 rows (by 1.1 to 1.3);
// at 320 and 384 they are within 11 %, at 512 the row form leads by 1.2 to 1.3.
// 64 experts, us, column / row form:
//   rows                      64        128        136        256        512
//   gate  4096 x 7168    285/428    305/437    501/438    554/445   1069/848
//         1024 x 1024    20/31      23/32      36/32      41/32      67/53
//   plain 7168 x 2048    151/217    162/232    261/232    300/244    586/465
//         1992 x 2176    56/72      63/78      89/78      99/81     190/150
// The mean is over the layout's entries and all experts: the host does not know
// which entries are masked or which experts get none, and such a call may take the
// slower form.
constexpr int kRowFormRows = 136;
constexpr int kSortExperts = 256;  // wgrad: most experts that are put in order
constexpr int kKeepExperts = 256;  // most experts whose counts and bases are kept in shared memory

// Tensor maps: [0] the M-side operand, [1..4] the token rows in boxes of 128,
// 64, 32 and 16 rows (wgrad: [1] x), [5] the output of the e4m3 row form
// and of wgrad.
struct Maps {
    CUtensorMap m[6];
};

// ALT: wgrad with fp32 output; e4m3 products in row form.
template <ExpertOp OP, bool ALT>
struct Shape {
    static constexpr bool FP8 = OP == ExpertOp::kFp8 || OP == ExpertOp::kGateFp8;
    static constexpr bool GATE = OP == ExpertOp::kGateFp8;
    static constexpr bool WG = OP == ExpertOp::kWgrad;
    static constexpr bool LIN = OP == ExpertOp::kLinear;  // bf16 with bias, activation and residual
    static constexpr bool F32 = WG && ALT;
    static constexpr bool ROW = FP8 && ALT;
    static constexpr bool COL = FP8 && !ALT;         // two M-side operands: gate and up product, or 2 x 256 weight rows
    static constexpr bool A_MN = OP == ExpertOp::kBf16T || WG;
    static constexpr bool B_MN = WG;
    // Warps that read the accumulators: 16 where there is work to do on them (linear, 32768 rows x 2048, SiLU and z
    // kept: k = 256 76 us, with 8 warps 92; k = 1024 107 and 111; k = 4096 332 and 333; 131072 rows x 4096 x 1024, GELU,
    // z and residual 1.01 ms and 1.13)
    static constexpr bool MANY = ROW || LIN;
    static constexpr int READ = MANY ? 16 : 8;
    static constexpr int THREADS = (READ + 4) * 32;
    // registers per thread: 384 x 168 at launch, split 256 x 216 + 128 x 72 (row form, linear: 640 x 96, split
    // 512 x 104 + 128 x 64)
    static constexpr int REGS_READ = MANY ? 104 : 216, REGS_REST = MANY ? 64 : 72;
    static constexpr int TOKENS = COL ? 128 : 256;            // most rows of a tile
    // weight rows (gate: channels of h) of a pair's tile
    static constexpr int WROWS = COL && !GATE ? 512 : GATE && ROW ? 128 : 256;
    static constexpr int A_BYTES = COL ? 32768 : 16384;       // per CTA and stage
    static constexpr int B_BYTES = ROW ? 16384 : TOKENS / 2 * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int OUT_BYTES = ROW ? (GATE ? 0 : 4096) : COL ? 512 : WG ? 4096 : LIN ? 1024 : 2048;  // per reading warp
    static constexpr int STAGES = ROW && !GATE ? 4 : COL ? 5 : 6;
    static constexpr int SCALES = FP8 ? 2 * kScaleGroup * 256 * 4 : 0;
    static constexpr int AMAX = GATE ? 2 * 4 * 128 * 4 + (COL ? READ * 64 * 4 : 0) : 0;
    // channels (bf16: 64, e4m3: 128) or rows (wgrad: 64) of one stage
    static constexpr int KSTEP = FP8 ? 128 : 64;
    // stages per segment; 0: all of them.  fp32 wgrad: 256 rows, 16 additions that truncate, whose drift
    // (2-norm of the error of equal-signed sums of 384 to 6000 rows: 3.1 to 3.8e-7) is what a plain fp32
    // product of the library is off by (1.8 to 4.3e-7).  384 rows drift by 5.6e-7, 128 by 1.9e-7.  16 x 1024
    // rows x 2048 x 7168: 339 / 356 / 404 us with 384 / 256 / 128 (the tensor cores run two segments ahead
    // and wait for the registers while those are stored), 64 x 256 rows 644 / 644 / 658.
    static constexpr int SEG = FP8 ? 1 : (F32 ? 4 : 0);
    static constexpr size_t fixed = 1024 + (size_t)STAGES * STAGE + READ * OUT_BYTES + SCALES + AMAX;
};

struct Tile {
    int64_t row0;   // first receive row (wgrad: of the expert)
    int e;
    int valid;      // rows (wgrad: all rows of the expert)
    int nt;         // columns of the products, a multiple of 32
    int w0;         // first weight row of the pair (gate: channel of h)
    int c0;         // wgrad: first column (channel of x)
};

struct Bars {
    uint64_t full[6], empty[6], land[6];
    uint64_t tfull[2], tempty[2], sfull[2], sempty[2], kfull[kTileRing], kempty[kTileRing];
    uint64_t nfull[kNextRing], nempty[kNextRing];
    uint64_t amax[4], want;
    Tile tiles[kTileRing];
    int next[kNextRing];
    uint32_t tmem;
};

// The layout's counts and bases in shared memory (nullptr: too many experts,
// they are read from global memory).
struct Kept {
    const int64_t *base;
    const int *count;
};

// Tile number t.  before[e]: token tiles of the experts before e (wgrad: the
// experts by falling row count).
template <ExpertOp OP, bool ALT>
__device__ __forceinline__ Tile tile_at(const ExpertGemmParams &p, const int *before, const Kept &kept, int t, int wtiles) {
    using S = Shape<OP, ALT>;
    Tile r;
    if constexpr (S::WG) {
        const int ctiles = (p.k + 255) / 256;
        const int per = wtiles * ctiles;
        const int i = t / per;
        const int local = t - i * per;
        r.e = p.E <= kSortExperts ? before[i] : i;
        r.w0 = local / ctiles * S::WROWS;
        r.c0 = local % ctiles * 256;
        r.row0 = kept.base != nullptr ? kept.base[r.e] : __ldg(p.base + r.e);
        r.valid = kept.base != nullptr ? kept.count[r.e] : __ldg(p.count + r.e);
        r.nt = p.k - r.c0 > 128 ? 256 : 128;
    } else {
        const int q = t / wtiles;
        int lo = 0, hi = p.E - 1;  // the last e with before[e] <= q
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= q)
                lo = mid;
            else
                hi = mid - 1;
        }
        r.e = lo;
        const int tt = before[lo + 1] - before[lo];
        const int local = t - before[lo] * wtiles;
        const int cnt = kept.base != nullptr ? kept.count[lo] : __ldg(p.count + lo);
        // equal token tiles, in steps of 32 rows (row form: whole ones and the rest)
        const int size = S::ROW ? S::TOKENS : ((cnt + tt - 1) / tt + 31) & ~31;
        const int r0 = local % tt * size;
        r.w0 = local / tt * S::WROWS;
        r.c0 = 0;
        r.row0 = (kept.base != nullptr ? kept.base[lo] : __ldg(p.base + lo)) + r0;
        r.valid = min(size, cnt - r0);
        r.nt = S::ROW ? 256 : (r.valid + 31) & ~31;
    }
    return r;
}

// Place of a column's scale in a block's 256 (column form): a thread T of the
// fragment layout needs the columns 4 j + T % 4 of 64, so they lie together (16
// floats), in 16-byte pieces swapped so that the four threads' reads of a piece
// fall into different banks.
__device__ __forceinline__ int scale_at(int col) {
    const int c = col & 3, j = (col & 63) >> 2;
    return (col & ~63) + c * 16 + (((j >> 2) ^ (c >> 1)) << 2) + (j & 3);
}

// g / (1 + exp(-g)) * u in fp32, from e = exp(-|g|): for g < 0 the quotient is
// g e / (1 + e).  e does not overflow, and the denominator lies in [1, 2], where
// the fast division is good to 2 ulp: 5 ulp in all, for every g.  (The fast
// exponential is off by 1.2 |g| ulp, and a fast division by 1 + exp(-g) is 0 below
// g = -87.3; with them 64 x 128 rows x 4096 x 512 took 48 instead of 53 us, 16 x 1024
// rows x 4096 x 7168 426 instead of 437, 32768 entries over 256 experts 1.58 ms instead
// of 1.59.)
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Write 32 tokens x 32 channels of a warp (lane = channel, v[i] = token i) as
// bf16 rows: neighbouring lanes swap halves so that each holds channel pairs,
// the pairs go through shared memory (64 bytes per token, free of bank conflicts), and
// 4 lanes store the 64 bytes of a token.
template <int T>
__device__ __forceinline__ void store_tokens(const float (&v)[T], uint32_t buf, int lane, __nv_bfloat16 *dst, int64_t ld,
                                             int tokens, int channels) {
    const bool odd = lane & 1;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < T / 4; ++j) {
        const uint32_t a = bf16x2(v[4 * j], v[4 * j + 2]), b = bf16x2(v[4 * j + 1], v[4 * j + 3]);
        const uint32_t keep = odd ? b : a;
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
        // even lanes: tokens 4j and 4j + 2; odd lanes: 4j + 1 and 4j + 3
        const uint32_t lo = __byte_perm(keep, got, odd ? 0x1054 : 0x5410);
        const uint32_t hi = __byte_perm(keep, got, odd ? 0x3276 : 0x7632);
        const uint32_t at = buf + (4 * j + (odd ? 1 : 0)) * 64 + (lane >> 1) * 4;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(lo) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 128), "r"(hi) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < T / 8; ++j) {
        const int tok = (lane >> 2) + 8 * j, c = (lane & 3) * 8;
        uint4 q;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(buf + tok * 64 + c * 2));
        if (tok < tokens && c < channels) *reinterpret_cast<uint4 *>(dst + tok * ld + c) = q;
    }
}

// linear: a step of a reading warp is 16 tokens x 32 channels.
constexpr int kStep = 16;

// A step's tokens the other way: loaded like the stores above, and, through the same
// 1 KB, added to v.
struct Residual {
    uint4 q[kStep / 8];
};
__device__ __forceinline__ void load_residual(Residual &r, int lane, const __nv_bfloat16 *src, int64_t ld, int tokens, int channels) {
#pragma unroll
    for (int j = 0; j < kStep / 8; ++j) {
        const int tok = (lane >> 2) + 8 * j, c = (lane & 3) * 8;
        r.q[j] = make_uint4(0, 0, 0, 0);
        if (tok < tokens && c < channels) r.q[j] = *reinterpret_cast<const uint4 *>(src + tok * ld + c);
    }
}
__device__ __forceinline__ void add_residual(float (&v)[kStep], const Residual &r, uint32_t buf, int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kStep / 8; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + ((lane >> 2) + 8 * j) * 64 + (lane & 3) * 16), "r"(r.q[j].x),
                     "r"(r.q[j].y), "r"(r.q[j].z), "r"(r.q[j].w)
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(buf + i * 64 + lane * 2));
        v[i] += __uint_as_float((uint32_t)h << 16);
    }
}

// Of the tokens that are there, 8 at a time: with few, most of the time is fetching the code (4 tokens, top-4 of 32,
// 1024 x 1024, GELU by erfcf: 10.8 us for all 32, 9.0).
template <Act ACT>
__device__ __forceinline__ void activate(float (&v)[kStep], int tokens) {
#pragma unroll
    for (int i = 0; i < kStep; i += 8) {
        if (i >= tokens) break;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t y = activate2<ACT>(two(v[i + j], v[i + j + 1]));
            v[i + j] = lo2(y);
            v[i + j + 1] = hi2(y);
        }
    }
}

// Two pieces of 16 bytes of one row, as one 32-byte store where `whole` (the
// rows are 32-byte aligned); pieces: how many of them lie in the row.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&v)[8], bool whole, int pieces) {
    if (whole && pieces >= 2) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
        return;
    }
    if (pieces >= 1) static_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if (pieces >= 2) static_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

// 32 lines of 128 bytes (lane = line) into a box of shared memory as a tensor
// map with such lines, swizzled over 128 bytes, has it.  Whole lines of 128
// bytes: the copy unit takes a line at a time, and with lines of 64 the fp32
// weights' gradient of 64 x 256 rows x 2048 x 7168 took 741 us instead of 664.
__device__ __forceinline__ void fill_box(const uint4 (&v)[8], uint32_t box, int lane) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((c ^ (lane & 7)) << 4)), "r"(v[c].x),
                     "r"(v[c].y), "r"(v[c].z), "r"(v[c].w)
                     : "memory");
    fence_async_shared();
    __syncwarp();
}

template <ExpertOp OP, bool ALT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<OP, ALT>::THREADS, 1)
    expert_gemm_kernel(const __grid_constant__ Maps maps, const ExpertGemmParams p) {
    using S = Shape<OP, ALT>;
    extern __shared__ uint8_t dyn[];
    __shared__ Bars bars;
    uint8_t *const smem = reinterpret_cast<uint8_t *>(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
    uint8_t *const outs = smem + S::STAGES * S::STAGE;
    float *const scales = reinterpret_cast<float *>(outs + S::READ * S::OUT_BYTES);
    float *const amaxs = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(scales) + S::SCALES);
    int *const before = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(amaxs) + S::AMAX);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarpLoad = S::READ, kWarpMma = S::READ + 1, kWarpAux = S::READ + 2, kWarpTiles = S::READ + 3;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const uint32_t b_full = saddr(bars.full), b_empty = saddr(bars.empty), b_land = saddr(bars.land);
    const uint32_t b_tfull = saddr(bars.tfull), b_tempty = saddr(bars.tempty);
    const uint32_t b_sfull = saddr(bars.sfull), b_sempty = saddr(bars.sempty);
    const uint32_t b_kfull = saddr(bars.kfull), b_kempty = saddr(bars.kempty);

    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(b_full + 8 * i, S::WG ? 2 : 1);
            bar_init(b_empty + 8 * i, 1);
            bar_init(b_land + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(b_tfull + 8 * i, 1);
            bar_init(b_tempty + 8 * i, 2 * S::READ);
            bar_init(b_sfull + 8 * i, 1);
            bar_init(b_sempty + 8 * i, S::READ);
        }
        for (int i = 0; i < kTileRing; ++i) {
            bar_init(b_kfull + 8 * i, 1);
            // readers: the reading warps, the loader, the first CTA's product warp, the auxiliary warp
            bar_init(b_kempty + 8 * i, S::READ + 1 + (rank == 0 ? 1 : 0) + (S::FP8 || S::WG ? 1 : 0));
        }
        for (int i = 0; i < kNextRing; ++i) {
            bar_init(saddr(&bars.nfull[i]), 1);
            bar_init(saddr(&bars.nempty[i]), 1);
        }
        for (int i = 0; i < 4; ++i) bar_init(saddr(&bars.amax[i]), 4);
        bar_init(saddr(&bars.want), 1);
        bar_init_fence();
        for (int i = 0; i < (S::WG ? 2 : 5); ++i) prefetch_map(&maps.m[i]);
    }
    __syncwarp();
    cluster_arrive();  // the barriers are initialised; waited for below
    if (warp == kWarpMma) tmem_alloc(saddr(&bars.tmem), 512);
    pdl_wait();  // the layout, the rows and possibly the weights come from kernels queued before
    // token tiles of the experts before each one, and behind them the counts and bases (wgrad: the
    // experts in order, and no room for those)
    Kept kept = {nullptr, nullptr};
    if (!S::WG && p.E <= kKeepExperts) {
        int64_t *kb = reinterpret_cast<int64_t *>(before + ((p.E + 2) & ~1));
        int *kc = reinterpret_cast<int *>(kb + p.E);
        kept.base = kb;
        kept.count = kc;
        if (tid < p.E) {
            kc[tid] = __ldg(p.count + tid);
            kb[tid] = __ldg(p.base + tid);
        }
        __syncthreads();
    }
    if constexpr (!S::WG) {
        for (int e = tid; e < p.E; e += S::THREADS)
            before[e + 1] = ((kept.base != nullptr ? kept.count[e] : __ldg(p.count + e)) + S::TOKENS - 1) / S::TOKENS;
        if (tid == 0) before[0] = 0;
        __syncthreads();
        if (warp == 0) {
            const int per = (p.E + 31) / 32;
            int sum = 0;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < p.E) sum += before[e + 1];
            }
            int run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, run, o);
                if (lane >= o) run += v;
            }
            run -= sum;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < p.E) {
                    run += before[e + 1];
                    before[e + 1] = run;
                }
            }
        }
    } else if (p.E <= kSortExperts) {
        // long sums first: tiles are handed out in this order, and a long one at the end would be
        // waited for alone
        const int c = tid < p.E ? __ldg(p.count + tid) : -1;
        if (tid < p.E) before[tid] = c;
        __syncthreads();
        int at = 0;
        if (tid < p.E)
            for (int e = 0; e < p.E; ++e) {
                const int o = before[e];
                at += o > c || (o == c && e < tid) ? 1 : 0;
            }
        __syncthreads();
        if (tid < p.E) before[at] = tid;
    }
    fence_before();
    __syncthreads();
    cluster_wait();
    fence_after();
    const uint32_t tmem = bars.tmem;

    const int width = S::GATE ? p.n / 2 : p.n;
    const int wtiles = (width + S::WROWS - 1) / S::WROWS;
    const int ctiles = (p.k + 255) / 256;
    const int total = S::WG ? p.E * wtiles * ctiles : before[p.E] * wtiles;
    const int kchan = (p.k + S::KSTEP - 1) / S::KSTEP;  // stages of a tile (wgrad: by the expert's rows)
    auto stages_of = [&](const Tile &ti) { return S::WG ? (ti.valid + 63) / 64 : kchan; };
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, p.wait_cycles); };
    // for a barrier behind which the other CTA has touched shared memory
    auto wait_cluster = [&](uint32_t bar, uint32_t parity) { return bar_wait<true>(bar, parity, p.wait_cycles); };
    // The i-th tile of this pair, for a whole warp; false after the last one.
    auto next_tile = [&](Tile &ti, int i) {
        const int s = i % kTileRing;
        ok = __all_sync(0xFFFFFFFFu, wait(b_kfull + 8 * s, (i / kTileRing) & 1));
        if (!ok) return false;
        ti = bars.tiles[s];
        __syncwarp();
        if (lane == 0) bar_arrive(b_kempty + 8 * s);
        return ti.e >= 0;
    };
    // The four warps that share a block's maximum (gate): all have written theirs.
    auto amax_ready = [&](int group, uint32_t turn) {
        __syncwarp();
        if (lane == 0) bar_arrive(saddr(&bars.amax[group]));
        ok = __all_sync(0xFFFFFFFFu, wait(saddr(&bars.amax[group]), turn & 1));
        return ok;
    };
    if (warp >= S::READ) {
        regs_dec<S::REGS_REST>();
        if (warp == kWarpTiles) {
            // Hands the pair's tiles out, looked up ahead of the others (a search, divisions and two
            // loads from L2).  The first tile is the pair's own number, the others come from a counter in
            // global memory, so that pairs with short tiles take more of them and the tiles of one
            // expert, which share its weights in L2, start together (every 76th tile instead: 262144 rows x
            // 2048 x 7168 5.8 instead of 4.9 ms, 32 x 128 tokens' FP8 gate 1.81 instead of 1.52).  The first
            // CTA draws the numbers and sends them to the second.
            if (lane == 0) {
                const bool drawn = p.next != nullptr && total > pairs;
                int t = pair;
                for (int i = 0; ok; ++i) {
                    const int n = i % kNextRing;
                    if (drawn && i > 0) {
                        const uint32_t full = saddr(&bars.nfull[n]), empty = saddr(&bars.nempty[n]);
                        if (rank == 0) {
                            // not before the loader is near the end of the tile before: a number drawn
                            // early starts late, and the tiles of one expert no longer together
                            if (!(ok = wait(saddr(&bars.want), (i - 1) & 1))) break;
                            t = pairs + (int)atomicAdd(p.next, 1u);
                            if (!(ok = wait_cluster(empty, ((i / kNextRing) & 1) ^ 1))) break;
                            send_u32(map_rank(saddr(&bars.next[n]), 1), (uint32_t)t, map_rank(full, 1));
                        } else {
                            bar_expect(full, 4);
                            if (!(ok = wait_cluster(full, (i / kNextRing) & 1))) break;
                            t = bars.next[n];
                            bar_arrive_cluster(map_rank(empty, 0));
                        }
                    } else if (drawn) {
                        // the first round of ring place 0 stands for the first tile, which nobody sends
                        if (rank == 1) {
                            bar_arrive(saddr(&bars.nfull[0]));
                            bar_arrive_cluster(map_rank(saddr(&bars.nempty[0]), 0));
                        }
                    } else if (i > 0) {
                        t += pairs;
                    }
                    const int s = i % kTileRing;
                    Tile ti;
                    ti.e = -1;
                    if (t < total) ti = tile_at<OP, ALT>(p, before, kept, t, wtiles);
                    if (!(ok = wait(b_kempty + 8 * s, ((i / kTileRing) & 1) ^ 1))) break;
                    bars.tiles[s] = ti;
                    bar_arrive(b_kfull + 8 * s);
                    if (t >= total) {
                        // the second CTA's arrivals are here before this CTA ends
                        if (drawn && rank == 0)
                            for (int j = max(0, i - kNextRing + 1); j <= i && ok; ++j)
                                ok = wait(saddr(&bars.nempty[j % kNextRing]), (j / kNextRing) & 1);
                        break;
                    }
                }
                // the last pair to stop drawing puts the counter back for the next launch
                if (drawn && rank == 0 && atomicAdd(p.next + 1, 1u) == (uint32_t)pairs - 1) {
                    p.next[0] = 0;
                    p.next[1] = 0;
                }
            }
        } else if (warp == kWarpLoad) {
            int st = 0;
            uint32_t ph = 0;
            int used = 0;
            Tile ti;
            for (int i = 0; ok; ++i) {
                if (!next_tile(ti, i)) break;
                const int nk = stages_of(ti);
                // rows that each CTA loads on the token side
                const int half = ti.nt >> 1;
                const int mine = S::ROW ? min(128, max(0, (ti.valid - (int)rank * 128 + 15) & ~15)) : half;
                const uint32_t bytes = (S::ROW ? S::B_BYTES : S::A_BYTES) + mine * 128;
                const uint32_t both = S::ROW ? 2 * S::B_BYTES + min(256, (ti.valid + 15) & ~15) * 128 : 2 * bytes;
                const int want = nk - S::STAGES - 2;  // stages loaded when the next tile is asked for
                if (want <= 0 && rank == 0 && lane == 0) bar_arrive(saddr(&bars.want));
                for (int kb = 0; kb < nk; ++kb) {
                    if (kb == want && kb > 0 && rank == 0 && lane == 0) bar_arrive(saddr(&bars.want));
                    ok = __all_sync(0xFFFFFFFFu, wait(b_empty + 8 * st, ph ^ 1));
                    if (!ok) break;
                    const uint32_t a = saddr(smem + st * S::STAGE), b = a + S::A_BYTES;
                    const uint32_t full0 = map_rank(b_full + 8 * st, 0);
                    if (ti.e == p.withhold) {  // test hook
                        ok = false;
                        break;
                    }
                    if (elect()) {
                        uint32_t bar = full0;
                        if constexpr (S::WG) {
                            const int part = ti.valid & 63;  // rows of the last 64 that are not full
                            if (kb == 0 && part != 0) {
                                // these come first: the rows past the end are cleared before the products
                                // see the stage, while they still work on the tile before
                                bar = map_rank(b_land + 8 * st, rank);
                                bar_expect(b_land + 8 * st, bytes);
                            } else if (rank == 0) {
                                bar_expect(b_full + 8 * st, 2 * bytes);
                                bar_arrive(b_full + 8 * st);  // for the other CTA
                            }
                            const int r = (int)(ti.row0 + (part == 0 ? kb : kb == 0 ? nk - 1 : kb - 1) * 64);
                            const int n0 = ti.w0 + (int)rank * 128, c0 = ti.c0 + (int)rank * half;
                            tma_2d(a, &maps.m[0], n0, r, bar);
                            tma_2d(a + 8192, &maps.m[0], n0 + 64, r, bar);
                            tma_2d(b, &maps.m[1], c0, r, bar);
                            if (half > 64) tma_2d(b + 8192, &maps.m[1], c0 + 64, r, bar);
                        } else {
                            if (rank == 0) bar_expect(b_full + 8 * st, both);
                            const int kc = kb * S::KSTEP, w = ti.w0 + (int)rank * 128;
                            if constexpr (S::ROW) {
                                // gate: the first CTA's half of the columns is the gate's, the second's the up product's
                                tma_3d(b, &maps.m[0], kc, S::GATE ? ti.w0 + (int)rank * width : w, ti.e, bar);
                            } else if constexpr (S::A_MN) {
                                tma_3d(a, &maps.m[0], w, kc, ti.e, bar);
                                tma_3d(a + 8192, &maps.m[0], w + 64, kc, ti.e, bar);
                            } else {
                                tma_3d(a, &maps.m[0], kc, w, ti.e, bar);
                                if constexpr (S::COL) tma_3d(a + 16384, &maps.m[0], kc, w + (S::GATE ? width : 256), ti.e, bar);
                            }
                            int r = (int)ti.row0 + (int)rank * (S::ROW ? 128 : half);
                            uint32_t d = S::ROW ? a : b;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int h = 128 >> j;
                                if (mine & h) {
                                    tma_2d(d, &maps.m[1 + j], kc, r, bar);
                                    r += h;
                                    d += h * 128;
                                }
                            }
                        }
                    }
                    __syncwarp();
                    used = min(used + 1, S::STAGES);
                    if (++st == S::STAGES) st = 0, ph ^= 1;
                }
            }
            // the stages in flight have been read (nothing lands or arrives here after the kernel's end)
            for (int i = 0; i < used; ++i) {
                if (--st < 0) st = S::STAGES - 1, ph ^= 1;
                if (!__all_sync(0xFFFFFFFFu, wait(b_empty + 8 * st, ph))) {
                    ok = false;
                    atomicOr(p.status, kStatusInFlight);
                    break;
                }
            }
        } else if (warp == kWarpMma) {
            if (rank == 0) {
                int st = 0;
                uint32_t ph = 0, seg = 0;
                Tile ti;
                for (int i = 0; ok; ++i) {
                    if (!next_tile(ti, i)) break;
                    const int nk = stages_of(ti);
                    const uint32_t id = idesc(S::FP8, S::A_MN, S::B_MN, ti.nt);
                    for (int kb = 0; kb < nk; ++kb) {
                        const int in_seg = S::SEG == 0 ? kb : kb % (S::SEG == 0 ? 1 : S::SEG);
                        const uint32_t buf = seg & 1;
                        // the operands first: they are there long before the accumulator is read out
                        const bool part = S::WG && kb == 0 && (ti.valid & 63) != 0;
                        ok = __all_sync(0xFFFFFFFFu, part ? wait_cluster(b_full + 8 * st, ph) : wait(b_full + 8 * st, ph));
                        if (!ok) break;
                        if (in_seg == 0) {
                            ok = __all_sync(0xFFFFFFFFu, wait(b_tempty + 8 * buf, ((seg >> 1) & 1) ^ 1));
                            if (!ok) break;
                        }
                        fence_after();
                        const uint32_t a = saddr(smem + st * S::STAGE), b = a + S::A_BYTES;
                        const uint32_t d = tmem + buf * 256;
                        const int steps = part ? ((ti.valid & 63) + 15) / 16 : 4;
                        const bool ends = kb == nk - 1 || (S::SEG != 0 && in_seg == S::SEG - 1);
                        if (elect()) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (S::WG && j >= steps) break;
                                const uint64_t da = desc(a + j * (S::A_MN ? 2048 : 32), S::A_MN ? 8192 : 16);
                                const uint64_t db = desc(b + j * (S::B_MN ? 2048 : 32), S::B_MN ? 8192 : 16);
                                mma<S::FP8>(d, da, db, id, in_seg != 0 || j != 0);
                                if constexpr (S::COL)
                                    mma<S::FP8>(d + 128, desc(a + 16384 + j * 32, 16), db, id, in_seg != 0 || j != 0);
                            }
                            commit_pair(b_empty + 8 * st);
                            if (ends) commit_pair(b_tfull + 8 * buf);
                        }
                        __syncwarp();
                        if (ends) ++seg;
                        if (++st == S::STAGES) st = 0, ph ^= 1;
                    }
                }
                // the last accumulators have been read: the second CTA's arrivals are here before this CTA ends
                for (uint32_t i = 1; i <= 2 && i <= seg && ok; ++i)
                    ok = __all_sync(0xFFFFFFFFu, wait(b_tempty + 8 * ((seg - i) & 1), ((seg - i) >> 1) & 1));
            }
        } else if (warp == kWarpAux) {
            if constexpr (S::FP8) {
                // Scales of 128 rows for kScaleGroup blocks at a time; the next group's (or tile's) loads
                // are in flight while one is stored.  Row form: of this CTA's rows, xs * ws with the two
                // blocks of weight rows.  Column form: xs, and apart from them the two ws, because each
                // thread needs 16 rows' and the reading warps' share of shared memory bounds them (products
                // of both operands read from here 334 instead of 327 us at 76 x 16 rows x 4096 x 7168).
                const int nb = (p.n + 127) / 128;
                struct Group {
                    float4 x[4];
                    float4 w, w2;  // row form
                    float wl;      // column form: lane j < 8 has that of block j / 2, operand j % 2
                } cur, nxt;
                uint32_t fill = 0;
                Tile ti = {};
                int i = 0, g = 0;
                auto fetch = [&](Group &o) {
                    const int r0 = S::ROW ? (int)rank * 128 : 0;
                    const int b0 = S::ROW ? ti.w0 / 128 : ti.w0 / 128 + (int)rank;
                    const int b1 = b0 + (S::GATE ? width / 128 : S::ROW ? 1 : 2);
                    auto four = [&](const float *q, bool vec) {
                        float4 v;
                        if (vec) {
                            v = __ldg(reinterpret_cast<const float4 *>(q));
                        } else {
                            v.x = __ldg(q);
                            v.y = g + 1 < kchan ? __ldg(q + 1) : 0.0f;
                            v.z = g + 2 < kchan ? __ldg(q + 2) : 0.0f;
                            v.w = g + 3 < kchan ? __ldg(q + 3) : 0.0f;
                        }
                        return v;
                    };
                    const float *ws = p.ws + (int64_t)ti.e * nb * kchan + g;
                    if constexpr (S::COL) {
                        o.wl = 0.0f;
                        if (lane < 8 && g + (lane >> 1) < kchan)
                            o.wl = __ldg(ws + (int64_t)min(lane & 1 ? b1 : b0, nb - 1) * kchan + (lane >> 1));
                    } else {
                        o.w = four(ws + (int64_t)min(b0, nb - 1) * kchan, p.ws_vec);
                        o.w2 = four(ws + (int64_t)min(b1, nb - 1) * kchan, p.ws_vec);
                    }
#pragma unroll
                    for (int j0 = 0; j0 < 128; j0 += 32) {
                        const int j = r0 + j0 + lane;
                        o.x[j0 / 32] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (j < ti.valid) o.x[j0 / 32] = four(p.xs + (ti.row0 + j) * kchan + g, p.xs_vec);
                    }
                };
                bool more = next_tile(ti, 0);
                if (more) fetch(cur);
                while (more) {
                    // on to the next group
                    g += kScaleGroup;
                    if (g >= kchan) {
                        g = 0;
                        more = next_tile(ti, ++i);
                        if (!ok) break;
                    }
                    if (more) fetch(nxt);
                    const uint32_t buf = fill & 1;
                    ok = __all_sync(0xFFFFFFFFu, wait(b_sempty + 8 * buf, ((fill >> 1) & 1) ^ 1));
                    if (!ok) break;
                    float *out = scales + buf * kScaleGroup * 256;
#pragma unroll
                    for (int j0 = 0; j0 < 128; j0 += 32) {
                        const int at = S::ROW ? j0 + lane : scale_at(j0 + lane);
                        const float4 v = cur.x[j0 / 32];
                        if constexpr (S::COL) {
                            out[at] = v.x;
                            out[256 + at] = v.y;
                            out[512 + at] = v.z;
                            out[768 + at] = v.w;
                            continue;
                        }
                        out[at] = v.x * cur.w.x;
                        out[256 + at] = v.y * cur.w.y;
                        out[512 + at] = v.z * cur.w.z;
                        out[768 + at] = v.w * cur.w.w;
                        out[128 + at] = v.x * cur.w2.x;
                        out[384 + at] = v.y * cur.w2.y;
                        out[640 + at] = v.z * cur.w2.z;
                        out[896 + at] = v.w * cur.w2.w;
                    }
                    if constexpr (S::COL) {
                        // behind each block's 128: those of its two blocks of weight rows
                        if (lane < 8) out[(lane >> 1) * 256 + 128 + (lane & 1)] = cur.wl;
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(b_sfull + 8 * buf);
                    ++fill;
                    cur = nxt;
                }
            } else if constexpr (S::WG) {
                // an expert's last rows, in its tile's first stage: clear the lines past its end
                // (both operands hold one 128-byte line per row and 64 channels), up to the 16 rows of a
                // product
                int st = 0;
                uint32_t landed = 0;  // parity of each stage's landing barrier
                Tile ti;
                for (int i = 0; ok; ++i) {
                    if (!next_tile(ti, i)) break;
                    const int nk = stages_of(ti);
                    if ((ti.valid & 63) != 0) {
                        ok = __all_sync(0xFFFFFFFFu, wait(b_land + 8 * st, (landed >> st) & 1));
                        if (!ok) break;
                        landed ^= 1u << st;
                        uint8_t *base = smem + st * S::STAGE;
                        const int r0 = ti.valid & 63, r1 = (r0 + 15) & ~15;
                        for (int i = lane; i < (r1 - r0) * 32; i += 32) {
                            const int row = r0 + (i >> 5), piece = i & 31;  // 4 chunks x 8 pieces of 16 bytes
                            *reinterpret_cast<uint4 *>(base + (piece >> 3) * 8192 + row * 128 + (piece & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        // The first CTA issues the products that read the lines of both: the zeros go before
                        // the tensor core's reads by the fence, and to that CTA's thread by a release at
                        // cluster scope.  Nothing waits for it: the loader is up to STAGES stages ahead of
                        // the products here (16 experts x 2048 x 7168: 280 us at 1000 rows each, 278 at 1024,
                        // where nothing is cleared; in a tile's last stage the release and its acquire took
                        // 2000 cycles a tile, 313 us).
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) bar_arrive_cluster(map_rank(b_full + 8 * st, 0));
                    }
                    st = (st + nk) % S::STAGES;
                }
            }
        }
    } else {
        regs_inc<S::REGS_READ>();
        const int sub = warp & 3, hw = warp >> 2;  // lanes 32 * sub .., every second chunk of 32 columns
        const uint32_t lanes = tmem + ((uint32_t)(sub * 32) << 16);
        const uint32_t out = saddr(outs + warp * S::OUT_BYTES);
        const uint32_t tempty0 = map_rank(b_tempty, 0);
        uint32_t seg = 0, fill = 0, turn = 0;
        Tile ti;
        for (int i = 0; ok; ++i) {
            if (!next_tile(ti, i)) break;
            const int nk = stages_of(ti);
            const int chunks = ti.nt >> 5;
            const int wc = ti.w0 + (int)rank * 128 + sub * 32;  // the warp's first weight row / channel of h
            if constexpr (S::WG && !S::F32) {
                // columns 128 hw on, as two boxes of 64 (128 bytes of bf16) that the tensor map stores
                // while the next one is read and the next tile is summed; what lies past n or k it
                // leaves out
                const uint32_t buf = seg & 1;
                if (nk > 0) {
                    ok = __all_sync(0xFFFFFFFFu, wait(b_tfull + 8 * buf, (seg >> 1) & 1));
                    if (!ok) break;
                    fence_after();
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = hw * 128 + q * 64;
                    uint4 line[8];
                    uint32_t *b4 = reinterpret_cast<uint32_t *>(line);
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        float v[32];
                        if (nk > 0) {
                            tmem_get32(v, lanes + buf * 256 + col + o * 32);  // past ti.nt: in the buffer, not stored
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) b4[o * 16 + j] = bf16x2(v[2 * j], v[2 * j + 1]);
                    }
                    if (q == 1 && nk > 0) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive_remote(tempty0 + 8 * buf);
                        ++seg;
                    }
                    if (wc >= p.n || ti.c0 + col >= p.k) continue;
                    if (lane == 0) store_read_wait();
                    __syncwarp();
                    fill_box(line, out, lane);
                    if (lane == 0) tma_store_3d(&maps.m[5], out, ti.c0 + col, wc, ti.e);
                }
            } else if constexpr (S::LIN) {
                const uint32_t buf = seg & 1;
                // asked for before the products are there: the bias of the lane's channel, the residual's first step
                // (the others into L2)
                float bias = 0.0f;
                Residual res;
                const int64_t at = ti.row0 * p.n + wc;
                const __nv_bfloat16 *const from = static_cast<const __nv_bfloat16 *>(p.residual) + at;
                if (p.bias != nullptr && wc + lane < p.n) {
                    const int64_t c = (int64_t)ti.e * p.n + wc + lane;
                    bias = p.bias_fp32 ? static_cast<const float *>(p.bias)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[c]);
                }
                if (p.residual != nullptr) {
                    load_residual(res, lane, from + (int64_t)hw * kStep * p.n, p.n, ti.valid - hw * kStep, p.n - wc);
                    for (int i = lane; i < 3 * kStep; i += 32) {
                        const int t = (hw + 4 + i / kStep * 4) * kStep + i % kStep;
                        if (t < ti.valid && wc < p.n) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + (int64_t)t * p.n));
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, wait(b_tfull + 8 * buf, (seg >> 1) & 1));
                if (!ok) break;
                fence_after();
                for (int c = hw; c * kStep < ti.valid; c += 4) {
                    const int tokens = ti.valid - c * kStep;
                    uint32_t raw[kStep];
                    float v[kStep];
                    tmem_get16(raw, lanes + buf * 256 + c * kStep);
#pragma unroll
                    for (int i = 0; i < kStep; ++i) v[i] = __uint_as_float(raw[i]) + bias;
                    if (p.z != nullptr)
                        store_tokens(v, out, lane, static_cast<__nv_bfloat16 *>(p.z) + at + (int64_t)c * kStep * p.n, p.n, tokens, p.n - wc);
                    switch (p.act) {
                        case Act::kRelu: activate<Act::kRelu>(v, tokens); break;
                        case Act::kGelu: activate<Act::kGelu>(v, tokens); break;
                        case Act::kGeluTanh: activate<Act::kGeluTanh>(v, tokens); break;
                        case Act::kSilu: activate<Act::kSilu>(v, tokens); break;
                        default: break;
                    }
                    if (p.residual != nullptr) {
                        add_residual(v, res, out, lane);
                        load_residual(res, lane, from + (int64_t)(c + 4) * kStep * p.n, p.n, tokens - 4 * kStep, p.n - wc);
                    }
                    store_tokens(v, out, lane, static_cast<__nv_bfloat16 *>(p.y) + at + (int64_t)c * kStep * p.n, p.n, tokens, p.n - wc);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_remote(tempty0 + 8 * buf);
                ++seg;
            } else if constexpr (S::SEG == 0) {
                __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y);
                const uint32_t buf = seg & 1;
                ok = __all_sync(0xFFFFFFFFu, wait(b_tfull + 8 * buf, (seg >> 1) & 1));
                if (!ok) break;
                fence_after();
                for (int c = hw; c < chunks; c += 2) {
                    float v[32];
                    tmem_get32(v, lanes + buf * 256 + c * 32);
                    store_tokens(v, out, lane, y + (ti.row0 + c * 32) * p.n + wc, p.n, ti.valid - c * 32, p.n - wc);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_remote(tempty0 + 8 * buf);
                ++seg;
            } else if constexpr (S::FP8) {
                // A block's products are scaled and added up here.
                //   row form: lane = row, one or two scales per thread and block; columns 64 hw on
                //     (gate: the gate's and the up product's 32 hw on) in 4 chunks of 16.  16 warps,
                //     because a read takes 200 cycles beside the products and nothing else hides it
                //     (8 warps: 572 instead of 492 us at 8192^3).
                //   column form: tokens 64 hw on of both operands, as fragments of 16 lanes: a thread has
                //     16 columns and needs their scales only (as whole lanes all 64: 4 times the reads of
                //     shared memory, 666 instead of 400 us at 76 x 128 rows x 4096 x 7168)
                //     acc[2 * operand + half][j]: column 4 j + lane % 4, weight rows 16 * half + lane / 4
                //     and + 8
                const int rows = ti.valid - (int)rank * 128 - sub * 32;  // row form: of this warp
                const int row = sub * 32 + lane;
                const int c4 = lane & 3;
                const int col0 = hw * (S::GATE && S::ROW ? 32 : 64);
                const bool live = S::ROW ? rows > 0 : col0 < ti.nt;
                constexpr int J = S::COL ? 16 : 8;
                uint64_t acc[4][J];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < J; ++j) acc[q][j] = 0;
                for (int k = 0; k < nk; ++k, ++seg) {
                    const uint32_t buf = seg & 1;
                    if (k % kScaleGroup == 0) {
                        ok = __all_sync(0xFFFFFFFFu, wait(b_sfull + 8 * (fill & 1), (fill >> 1) & 1));
                        if (!ok) break;
                    }
                    const float *sc = scales + ((fill & 1) * kScaleGroup + k % kScaleGroup) * 256;
                    uint64_t f0 = 0, f1 = 0;
                    if constexpr (S::ROW) {
                        const uint32_t s0 = __float_as_uint(sc[row + (S::GATE ? 0 : (hw >> 1) * 128)]);
                        const uint32_t s1 = S::GATE ? __float_as_uint(sc[row + 128]) : s0;
                        f0 = pair2(s0, s0);
                        f1 = pair2(s1, s1);
                    }
                    [[maybe_unused]] float xs[16];
                    [[maybe_unused]] float2 ws = {0.0f, 0.0f};
                    if constexpr (S::COL) {
                        if (live) {
                            ws = *reinterpret_cast<const float2 *>(sc + 128);
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                *reinterpret_cast<float4 *>(xs + 4 * m) =
                                    *reinterpret_cast<const float4 *>(sc + col0 + c4 * 16 + ((m ^ (c4 >> 1)) << 2));
                        }
                    }
                    ok = __all_sync(0xFFFFFFFFu, wait(b_tfull + 8 * buf, (seg >> 1) & 1));
                    if (!ok) break;
                    fence_after();
                    const uint32_t at = lanes + buf * 256 + col0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[2 * J];
                        if (live) {
                            if constexpr (S::COL) {
                                tmem_get_frag(v, at + (q >> 1) * 128 + ((q & 1) << 20));
                            } else {
                                tmem_get16(v, at + q * 16 + (S::GATE && q >= 2 ? 96 : 0));
                            }
                        }
                        if (q == 3) {  // all read: the buffer can be written again
                            fence_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive_remote(tempty0 + 8 * buf);
                        }
                        if (live) {
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                uint64_t f = q < 2 ? f0 : f1;
                                if constexpr (S::COL) {
                                    const uint32_t c = __float_as_uint(__fmul_rn(xs[j], q < 2 ? ws.x : ws.y));
                                    f = pair2(c, c);
                                }
                                acc[q][j] = fma2(pair2(v[2 * j], v[2 * j + 1]), f, acc[q][j]);
                            }
                        }
                    }
                    if (k % kScaleGroup == kScaleGroup - 1 || k == nk - 1) {
                        __syncwarp();
                        if (lane == 0) bar_arrive(b_sempty + 8 * (fill & 1));
                        ++fill;
                    }
                }
                if (!ok) break;
                if constexpr (S::COL) {
                    const int tokens = ti.valid - col0;
                    const int64_t first = ti.row0 + col0;
                    uint8_t *const own = outs + warp * S::OUT_BYTES;
                    if constexpr (S::GATE) {
                        if (live) {  // the same for the 4 warps of these tokens
                            // h in place of the gate's sums, and each column's maximum over the thread's 4
                            // channels; 16 tokens at a time, as many as there are
                            float top[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) top[j] = 0.0f;
#pragma unroll
                            for (int part = 0; part < 4; ++part) {
                                if (16 * part >= tokens) break;
#pragma unroll
                                for (int j = 4 * part; j < 4 * part + 4; ++j) {
#pragma unroll
                                    for (int r = 0; r < 2; ++r) {
                                        const float a0 = swiglu(lo2(acc[r][j]), lo2(acc[2 + r][j]));
                                        const float a1 = swiglu(hi2(acc[r][j]), hi2(acc[2 + r][j]));
                                        acc[r][j] = pair2(__float_as_uint(a0), __float_as_uint(a1));
                                        top[j] = fmaxf(top[j], fmaxf(fabsf(a0), fabsf(a1)));
                                    }
                                }
                            }
                            // over the warp's 32 channels: 8 lanes hold a column's; each step hands the half
                            // that the other lane will keep over, so that a lane ends with two columns
#pragma unroll
                            for (int o = 16, half = 8; o >= 4; o >>= 1, half >>= 1) {
                                const bool up = lane & o;
#pragma unroll
                                for (int j = 0; j < half; ++j) {
                                    const float give = up ? top[j] : top[j + half], keep = up ? top[j + half] : top[j];
                                    top[j] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
                                }
                            }
                            float *am = amaxs + ((turn & 1) * 2 + hw) * 256;
                            const int j0 = (lane >> 4 & 1) * 8 + (lane >> 3 & 1) * 4 + (lane >> 2 & 1) * 2;
                            am[sub * 64 + 4 * j0 + c4] = top[0];
                            am[sub * 64 + 4 * j0 + 4 + c4] = top[1];
                            // over the block's 128 channels: the four warps of these columns
                            if (!amax_ready(hw, turn++)) break;
                            const int h0 = ti.w0 + (int)rank * 128;
                            float *inv = amaxs + 1024 + warp * 64;  // [column % 4][column / 4]
#pragma unroll
                            for (int i2 = 0; i2 < 2; ++i2) {
                                const int col = lane + 32 * i2;
                                const float a = fmaxf(fmaxf(fmaxf(am[col], am[64 + col]), fmaxf(am[128 + col], am[192 + col])), 1e-4f);
                                inv[(col & 3) * 16 + (col >> 2)] = __fdiv_rn(448.0f, a);
                                if (sub == 0 && h0 < width && col < tokens)
                                    p.ys[(first + col) * (width / 128) + h0 / 128] = __fdiv_rn(a, 448.0f);
                            }
#pragma unroll
                            for (int part = 0; part < 4; ++part) {
                                if (16 * part >= tokens) break;
                                __syncwarp();
                                const float4 f4 = *reinterpret_cast<const float4 *>(inv + c4 * 16 + 4 * part);
                                const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint8_t *at = own + (4 * j + c4) * 32 + (lane >> 2);
#pragma unroll
                                    for (int r = 0; r < 2; ++r) {
                                        const uint64_t h = acc[r][4 * part + j];
                                        const uint32_t q = __nv_cvt_float2_to_fp8x2(
                                            make_float2(__fmul_rn(lo2(h), f[j]), __fmul_rn(hi2(h), f[j])), __NV_SATFINITE, __NV_E4M3);
                                        at[16 * r] = (uint8_t)q;
                                        at[16 * r + 8] = (uint8_t)(q >> 8);
                                    }
                                }
                                __syncwarp();
                                const int tok = 16 * part + (lane >> 1), off = (lane & 1) * 16;
                                const uint4 q = *reinterpret_cast<const uint4 *>(own + (lane >> 1) * 32 + off);
                                if (h0 < width && tok < tokens)
                                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.y) + (first + tok) * width + wc + off) = q;
                            }
                        }
                    } else if (live) {
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int c0 = wc + o * 256;
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.y) + first * p.n + c0;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                // 8 tokens x 32 channels as bf16, 64 bytes per token, 16-byte pieces swapped.
                                // Stored transposed: a thread's values are the tokens 8 j + lane % 4 and + 4, so
                                // row i of the store is token 8 j + i / 2 + 4 (i % 2)
                                uint32_t h[4];
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    const uint64_t a = acc[2 * o + r][2 * j], b = acc[2 * o + r][2 * j + 1];
                                    h[2 * r] = bf16x2(lo2(a), lo2(b));
                                    h[2 * r + 1] = bf16x2(hi2(a), hi2(b));
                                }
                                __syncwarp();
                                const int i8 = lane & 7, t8 = (i8 >> 1) + 4 * (i8 & 1);
                                stm_x4_trans(out + t8 * 64 + (((lane >> 3) ^ ((t8 >> 1) & 3)) << 4), h[0], h[1], h[2], h[3]);
                                __syncwarp();
                                const int t = lane >> 2, piece = lane & 3;
                                const uint4 q = *reinterpret_cast<const uint4 *>(own + t * 64 + ((piece ^ ((t >> 1) & 3)) << 4));
                                if (8 * j + t < tokens && piece * 8 < p.n - c0)
                                    *reinterpret_cast<uint4 *>(dst + (int64_t)(8 * j + t) * p.n + piece * 8) = q;
                            }
                        }
                    }
                    continue;
                }
                const int64_t row0 = ti.row0 + (int)rank * 128 + sub * 32;
                if constexpr (S::GATE) {
                    // 32 of the block's 128 channels here, the others in the three warps of the same rows
                    float top = 0.0f;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float a0 = swiglu(lo2(acc[q][j]), lo2(acc[2 + q][j]));
                            const float a1 = swiglu(hi2(acc[q][j]), hi2(acc[2 + q][j]));
                            acc[q][j] = pair2(__float_as_uint(a0), __float_as_uint(a1));
                            top = fmaxf(top, fmaxf(fabsf(a0), fabsf(a1)));
                        }
                    float *am = amaxs + (turn & 1) * 512;
                    am[hw * 128 + row] = top;
                    if (!amax_ready(sub, turn++)) break;
                    const float a = fmaxf(fmaxf(fmaxf(am[row], am[128 + row]), fmaxf(am[256 + row], am[384 + row])), 1e-4f);
                    const float inv = __fdiv_rn(448.0f, a);
                    if (hw == 0 && lane < rows) p.ys[(row0 + lane) * (width / 128) + ti.w0 / 128] = __fdiv_rn(a, 448.0f);
                    uint32_t b4[8];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const uint32_t b0 = __nv_cvt_float2_to_fp8x2(
                                make_float2(__fmul_rn(lo2(acc[q][j]), inv), __fmul_rn(hi2(acc[q][j]), inv)), __NV_SATFINITE, __NV_E4M3);
                            const uint32_t b1 = __nv_cvt_float2_to_fp8x2(
                                make_float2(__fmul_rn(lo2(acc[q][j + 1]), inv), __fmul_rn(hi2(acc[q][j + 1]), inv)), __NV_SATFINITE,
                                __NV_E4M3);
                            b4[q * 4 + j / 2] = b0 | b1 << 16;
                        }
                    if (lane < rows)
                        store32(static_cast<uint8_t *>(p.y) + (row0 + lane) * width + ti.w0 + hw * 32, b4, p.y_vec, 2);
                } else {
                    // 32 rows x 64 columns.  All rows in use: a box of shared memory (128 bytes per row,
                    // 16-byte pieces swizzled as the tensor map has it), stored while the next tile is
                    // added up; ordinary stores of 64 KB held the tile's end up for 3600 cycles.
                    const int c = ti.w0 + hw * 64;
                    if (rows >= 32) {
                        if (lane == 0) store_read_wait();
                        __syncwarp();
                        uint4 line[8];
                        uint32_t *b4 = reinterpret_cast<uint32_t *>(line);
#pragma unroll
                        for (int j = 0; j < 32; ++j) b4[j] = bf16x2(lo2(acc[j / 8][j % 8]), hi2(acc[j / 8][j % 8]));
                        fill_box(line, out, lane);
                        if (lane == 0 && c < p.n) tma_store_2d(&maps.m[5], out, c, (int)row0);
                    } else if (lane < rows) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t b4[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) b4[j] = bf16x2(lo2(acc[q][j]), hi2(acc[q][j]));
                            store32(static_cast<__nv_bfloat16 *>(p.y) + (row0 + lane) * p.n + c + q * 16, b4, p.y_vec,
                                    (p.n - c - q * 16) / 8);
                        }
                    }
                }
            } else {
                // wgrad in fp32: sums of 256 rows added up in registers, columns 128 hw on
                uint64_t acc[4][16];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[q][j] = 0;
                const int nseg = (nk + S::SEG - 1) / S::SEG;
                for (int k = 0; k < nseg; ++k, ++seg) {
                    const uint32_t buf = seg & 1;
                    ok = __all_sync(0xFFFFFFFFu, wait(b_tfull + 8 * buf, (seg >> 1) & 1));
                    if (!ok) break;
                    fence_after();
                    const uint32_t at = lanes + buf * 256 + hw * 128;
                    uint32_t v[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // columns past ti.nt are read (they lie in the buffer) and not written out
                        tmem_ld32(v, at + q * 32);
                        tmem_wait(v);
                        if (q == 3) {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive_remote(tempty0 + 8 * buf);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[q][j] = add2(pair2(v[2 * j], v[2 * j + 1]), acc[q][j]);
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = ti.c0 + hw * 128 + q * 32;
                    if (wc >= p.n || col >= p.k) continue;
                    uint4 line[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        line[j] = make_uint4((uint32_t)acc[q][2 * j], (uint32_t)(acc[q][2 * j] >> 32), (uint32_t)acc[q][2 * j + 1],
                                             (uint32_t)(acc[q][2 * j + 1] >> 32));
                    if (p.accumulate && nk == 0) continue;
                    if (lane == 0) store_read_wait();
                    __syncwarp();
                    fill_box(line, out, lane);
                    if (lane == 0) {
                        if (p.accumulate)
                            tma_add_3d(&maps.m[5], out, col, wc, ti.e);
                        else
                            tma_store_3d(&maps.m[5], out, col, wc, ti.e);
                    }
                }
            }
        }
    }
    if constexpr (S::WG || (S::ROW && !S::GATE)) {
        if (warp < S::READ && lane == 0) store_wait();
    }
    if (!ok) atomicOr(p.status, kStatusTimeout);
    __syncwarp();
    fence_before();
    cluster_arrive();
    cluster_wait();
    fence_after();
    if (warp == kWarpMma) tmem_free(tmem, 512);
}

// ------------------------------------------------------------ host side
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace

bool encode_rows(CUtensorMap *m, const void *base, int es, int64_t cols, int64_t rows, int64_t planes, int box_rows) {
    const EncodeTiled fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)(cols * es), (cuuint64_t)(cols * es * rows)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUtensorMapDataType type = es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    return fn(m, type, planes > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <ExpertOp OP, bool ALT>
size_t smem_bytes(int E) {
    if (Shape<OP, ALT>::WG) return Shape<OP, ALT>::fixed + (size_t)kSortExperts * 4;
    return Shape<OP, ALT>::fixed + (((size_t)E + 2) & ~(size_t)1) * 4 + (E <= kKeepExperts ? (size_t)E * 12 : 0);
}

template <ExpertOp OP, bool ALT>
cudaError_t launch(const ExpertGemmParams &p, cudaStream_t stream) {
    using S = Shape<OP, ALT>;
    ExpertGemmParams q = p;
    q.xs_vec = p.k % (4 * 128) == 0 && (uintptr_t)p.xs % 16 == 0;
    const int64_t ybytes = S::GATE ? p.n / 2 : (int64_t)p.n * 2;
    q.y_vec = ybytes % 32 == 0 && (uintptr_t)p.y % 32 == 0;
    q.ws_vec = p.k % (4 * 128) == 0 && (uintptr_t)p.ws % 16 == 0;
    Maps maps;
    bool ok;
    if constexpr (S::WG) {
        ok = encode_rows(&maps.m[0], p.dy, 2, p.n, p.rows, 0, 64) && encode_rows(&maps.m[1], p.x, 2, p.k, p.rows, 0, 64) &&
             encode_rows(&maps.m[5], p.y, S::F32 ? 4 : 2, p.k, p.n, p.E, 32);
    } else {
        constexpr int es = S::FP8 ? 1 : 2;
        ok = S::A_MN ? encode_rows(&maps.m[0], p.w, es, p.n, p.k, p.E, 64) : encode_rows(&maps.m[0], p.w, es, p.k, p.n, p.E, 128);
        for (int i = 0; i < 4 && ok; ++i) ok = encode_rows(&maps.m[1 + i], p.x, es, p.k, p.rows, 0, 128 >> i);
        if constexpr (S::ROW && !S::GATE) ok = ok && encode_rows(&maps.m[5], p.y, 2, p.n, p.rows, 0, 32);
    }
    if (!ok) return cudaErrorInvalidValue;
    int pairs = p.sms / 2;
    if (pairs < 1) pairs = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(S::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<OP, ALT>(p.E);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expert_gemm_kernel<OP, ALT>, maps, q);
}

}  // namespace

namespace {
template <ExpertOp OP, bool ALT>
void allow_smem() {
    // failing here means failing at the launch, which reports it
    if (cudaFuncSetAttribute(expert_gemm_kernel<OP, ALT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024) !=
        cudaSuccess)
        cudaGetLastError();
}
}  // namespace

void expert_gemm_init() {
    allow_smem<ExpertOp::kBf16, false>();
    allow_smem<ExpertOp::kBf16T, false>();
    allow_smem<ExpertOp::kLinear, false>();
    allow_smem<ExpertOp::kFp8, false>();
    allow_smem<ExpertOp::kFp8, true>();
    allow_smem<ExpertOp::kGateFp8, false>();
    allow_smem<ExpertOp::kGateFp8, true>();
    allow_smem<ExpertOp::kWgrad, false>();
    allow_smem<ExpertOp::kWgrad, true>();
}

cudaError_t launch_expert_gemm(ExpertOp op, const ExpertGemmParams &p, cudaStream_t stream) {
    const bool row = p.live > (int64_t)p.E * kRowFormRows;
    switch (op) {
        case ExpertOp::kBf16: return launch<ExpertOp::kBf16, false>(p, stream);
        case ExpertOp::kBf16T: return launch<ExpertOp::kBf16T, false>(p, stream);
        case ExpertOp::kLinear: return launch<ExpertOp::kLinear, false>(p, stream);
        case ExpertOp::kFp8: return row ? launch<ExpertOp::kFp8, true>(p, stream) : launch<ExpertOp::kFp8, false>(p, stream);
        case ExpertOp::kGateFp8:
            return row ? launch<ExpertOp::kGateFp8, true>(p, stream) : launch<ExpertOp::kGateFp8, false>(p, stream);
        default: return p.out_fp32 ? launch<ExpertOp::kWgrad, true>(p, stream) : launch<ExpertOp::kWgrad, false>(p, stream);
    }
}

}  // namespace ep

// The whole layer of gated experts for a few tokens (a decode step), in one
// kernel and without the receive layout between dispatch and combine:
//   gate   h[j] = silu(g) u, [g; u] = Wgu[e] x[t] + bgu[e]      for every entry j = (t, k), e = idx[t, k]
//   down   y[j] = Wd[e] h[j] + bd[e]
//          out[t] = bf16(res[t] + sum_k w[t, k] y[t, k])        k ascending, one rounding
// Weights are bf16, or e4m3 with a scale per 128 x 128 block.
//
// With few tokens the weights of the experts that are named are all that has to
// move, each used for a handful of tokens, so the kernel is one stream of weights per
// SM that never stops: a stage is 128 weight rows x 128 bytes, the M side of the tensor
// cores, whose N side are the tokens of one expert (16 to 64 columns).  All stages
// of a product, in the order expert, weight rows, tokens, channels, are cut into equal
// contiguous shares, one per SM, wherever that falls: a tile that begins in one SM's share
// and ends in another's leaves two partial sums (fp32, in the workspace), added in
// the order of the shares.  What needs all SMs' results is done between grid barriers
// (cooperative launch), and the weights' loader does not wait there:
//   entries sorted by expert (by every CTA) -- (tokens laid out as codes: kLaidStages) -- gate product -- SwiGLU, h
//   laid out -- down product -- sum over k
//
// Measured (one GB300), bytes of the named experts' weights over the time: 128 tokens, top-8 of 256, 7168 x 2048,
// FP8 1.8 ms, 6.2 TB/s; 32 tokens, top-6 of 64, 4096 x 1024, bf16 243 us, 6.2 TB/s; one token, top-8 of 256, 7168 x
// 2048, FP8 72 us, 4.9 TB/s: HBM bounds the products, which leave 10 us before the first stage, at the meetings (2
// us each, of which the ring covers 3 together) and behind the last.  Products on mma.sync with the codes
// converted on the way took 92 us and 2.4 ms there.
//
// Operands of e4m3 weights: a bf16 value has 8 significant bits, an e4m3 code 4, so x
// times a power of two per 128 channels (the largest to 128 .. 256) is the sum of two codes,
// the second worth 2^-4 of the first; exactly, down to 2^-13 of the largest, and to 2^-21
// of that below.  h, which has more bits, is the sum of four (2^-17 of it).  They are columns
// of the product, so nothing is converted on the weights' way.  The scales vary along the
// channels: a stage's sums leave tensor memory and are scaled and added in fp32
// registers.  bf16 weights: x as it is, h as the sum of two bf16 numbers.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "activation.cuh"
#include "ep_internal.cuh"
#include "umma.cuh"

namespace ep {

namespace {

using namespace umma;

// Warps: 0 .. 3 read the sums out of tensor memory, 4 loads weights, 6 issues the products, 8 .. 15 bring the
// tokens, a stage each in turn; 0 .. 3 and 8 .. 15 do what lies between the products ("workers").  Warp 7 goes through
// the latter's code once at the start, for nothing: the weights have washed the code out of L2, and the first
// run of 100 instructions takes 1300 cycles (one token, top-8 of 256, 7168 x 2048, FP8: 82 instead
// of 76 us).
constexpr int kWarpWeights = 4, kWarpMma = 6, kWarpSpare = 7, kWarpTokens = 8, kTokenWarps = 8;
constexpr int kThreads = 16 * 32, kWorkers = 12 * 32;
constexpr int kTile = 128;                   // weight rows of a job
constexpr int kMostColumns = 64;             // most columns of a job
constexpr int kWeightBytes = kTile * 128;
constexpr int kSums = 4;                     // accumulators
constexpr int kScales = 32;                  // stages whose tokens' scales are kept: the loaders are up to STAGES ahead
                                             // of the products, and those kSums + 1 ahead of the readers

// Columns of an entry (codes or numbers whose sum it is).
template <bool FP8, bool DOWN>
constexpr int kParts = FP8 ? (DOWN ? 4 : 2) : (DOWN ? 2 : 1);

// C: most columns of a job.  16 where no expert has more than 4 tokens of e4m3 (8 of bf16): what the ring does not
// hold of tokens it holds of weights, and is further ahead when the SMs meet.
template <bool FP8, int C>
struct Shape {
    static constexpr int STAGE = kWeightBytes + C * 128;
    static constexpr int STAGES = C == 16 ? 12 : 8;
    static constexpr bool LAID = FP8 && C != 16;  // has the form that lays the tokens out (p.laid)
    static constexpr size_t fixed = 1024 + (size_t)STAGES * STAGE;
    static_assert(STAGES + kSums + 1 <= kScales, "scales are overwritten before they are read");
};
// Entries of a job.
template <bool FP8, bool DOWN, int C>
constexpr int kTokens = C / kParts<FP8, DOWN>;
template <bool FP8>
constexpr int kLine = FP8 ? 128 : 64;        // channels of a stage

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Tensor memory and products of one CTA (umma.cuh has those of a pair).
__device__ __forceinline__ void tmem_alloc_one(uint32_t dst, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_one(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
template <bool FP8>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    if constexpr (FP8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(accumulate)
            : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory"); }

// The entries by expert, in shared memory: the D experts with entries, ascending,
// each with its list.
struct Route {
    int *first;           // [E + 1] first place in `list` of each expert
    uint16_t *live;       // [D] experts with entries
    uint16_t *list;       // [M] entries (token, k) by expert: token * 32 + k
    uint16_t *spot;       // [M] an entry's place in the list, 0xFFFF: none
    uint16_t *before[2];  // [D + 1] jobs of a tile (gate, down) before each live expert
    int D;
};
size_t route_bytes(int E, int M) {
    const int D = E < M ? E : M;
    return (size_t)(E + 2) * 4 + (size_t)D * 2 + (size_t)M * 4 + 2 * (size_t)(D + 1) * 2 + 16;
}

// `scratch`: 512 bytes for each warp, and 17 KB behind them.
template <bool FP8, int C>
__device__ __forceinline__ Route route(const ExpertLayerParams &p, uint8_t *at, uint32_t *scratch) {
    constexpr int kWarps = kThreads / 32, kGateTokens = kTokens<FP8, false, C>, kDownTokens = kTokens<FP8, true, C>;
    Route r;
    const int M = p.N * p.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    r.first = reinterpret_cast<int *>(at);
    r.list = reinterpret_cast<uint16_t *>(r.first + p.E + 1);
    r.spot = r.list + M;
    r.live = r.spot + M;
    r.before[0] = r.live + min(p.E, M);
    r.before[1] = r.before[0] + min(p.E, M) + 1;
    uint2 *const sums = reinterpret_cast<uint2 *>(scratch + kWarps * 128);       // [32] of 32 experts each
    uint16_t *const place = reinterpret_cast<uint16_t *>(sums + 32);            // [M] in its expert's list
    uint16_t *const owner = place + M;                                          // [M] expert, 0xFFFF: none
    for (int e = tid; e <= p.E; e += kThreads) r.first[e] = 0;
    __syncthreads();
    for (int j = tid; j < M; j += kThreads) {
        const int64_t e = p.idx[j];
        const bool ok = e >= 0 && e < p.E;
        if (!ok && e != -1 && blockIdx.x == 0) atomicOr(p.status, kStatusBadExpert);
        owner[j] = ok ? (uint16_t)e : 0xFFFFu;
        r.spot[j] = 0xFFFFu;
        if (ok) place[j] = (uint16_t)atomicAdd(&r.first[e], 1);
    }
    __syncthreads();
    // Prefix sums over the experts, 32 to a warp: entries and live experts, jobs of both products, two in
    // a word (4096 at most).
    const int chunks = (p.E + 31) / 32;
    constexpr int kTurns = (32 + kWarps - 1) / kWarps;  // 32 chunks at most
    uint2 own[kTurns], run[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int e = (warp + i * kWarps) * 32 + lane;
        const uint32_t c = warp + i * kWarps < chunks && e < p.E ? (uint32_t)r.first[e] : 0u;
        own[i] = make_uint2(c | (c > 0 ? 1u : 0u) << 16, (c + kGateTokens - 1) / kGateTokens | (c + kDownTokens - 1) / kDownTokens << 16);
        run[i] = own[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, run[i].x, o), y = __shfl_up_sync(0xFFFFFFFFu, run[i].y, o);
            if (lane >= o) run[i].x += x, run[i].y += y;
        }
        if (lane == 31 && warp + i * kWarps < 32) sums[warp + i * kWarps] = run[i];
    }
    __syncthreads();
    uint2 all = sums[lane];
    const uint2 mine = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, all.x, o), y = __shfl_up_sync(0xFFFFFFFFu, all.y, o);
        if (lane >= o) all.x += x, all.y += y;
    }
    const uint2 total = make_uint2(__shfl_sync(0xFFFFFFFFu, all.x, 31), __shfl_sync(0xFFFFFFFFu, all.y, 31));
    r.D = (int)(total.x >> 16);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int chunk = min(warp + i * kWarps, 31), e = chunk * 32 + lane;
        const uint32_t x = __shfl_sync(0xFFFFFFFFu, all.x - mine.x, chunk) + run[i].x - own[i].x;
        const uint32_t y = __shfl_sync(0xFFFFFFFFu, all.y - mine.y, chunk) + run[i].y - own[i].y;
        if (warp + i * kWarps >= chunks || e >= p.E) continue;
        r.first[e] = (int)(x & 0xFFFFu);
        if (own[i].x == 0) continue;
        r.live[x >> 16] = (uint16_t)e;
        r.before[0][x >> 16] = (uint16_t)(y & 0xFFFFu);
        r.before[1][x >> 16] = (uint16_t)(y >> 16);
    }
    if (tid == 0) {
        r.first[p.E] = (int)(total.x & 0xFFFFu);
        r.before[0][r.D] = (uint16_t)(total.y & 0xFFFFu);
        r.before[1][r.D] = (uint16_t)(total.y >> 16);
    }
    __syncthreads();
    for (int j = tid; j < M; j += kThreads)
        if (owner[j] != 0xFFFFu) r.list[r.first[owner[j]] + place[j]] = (uint16_t)(j / p.K * 32 + j % p.K);
    __syncthreads();
    // The order inside a list is the atomics', and has to be the same in every CTA: ascending, up to 32
    // entries by counting the smaller ones, else by a bit per entry.
    uint32_t *bits = scratch + warp * 128;
    for (int d = warp; d < r.D; d += kWarps) {
        const int e = r.live[d], a = r.first[e], b = r.first[e + 1];
        if (b - a <= 32) {
            const uint32_t v = a + lane < b ? r.list[a + lane] : 0xFFFFu;
            int rank = 0;
            for (int i = 0; i < b - a; ++i) rank += __shfl_sync(0xFFFFFFFFu, v, i) < v ? 1 : 0;
            if (a + lane < b) r.list[a + rank] = (uint16_t)v;
            continue;
        }
        for (int i = lane; i < 128; i += 32) bits[i] = 0;
        __syncwarp();
        for (int i = a + lane; i < b; i += 32) {
            const uint32_t v = r.list[i], j = (v >> 5) * p.K + (v & 31);
            atomicOr(bits + (j >> 5), 1u << (j & 31));
        }
        __syncwarp();
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += __popc(bits[lane * 4 + i]);
        int at0 = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, at0, o);
            if (lane >= o) at0 += v;
        }
        at0 += a - n;
        for (int i = 0; i < 4; ++i)
            for (uint32_t w = bits[lane * 4 + i]; w != 0; w &= w - 1) {
                const uint32_t j = (lane * 4 + i) * 32 + __ffs(w) - 1;
                r.list[at0++] = (uint16_t)(j / p.K * 32 + j % p.K);
            }
        __syncwarp();
    }
    __syncthreads();
    for (int i = tid; i < r.first[p.E]; i += kThreads) {
        const uint32_t v = r.list[i];
        r.spot[(v >> 5) * p.K + (v & 31)] = (uint16_t)i;
    }
    return r;
}

// The jobs of a product (0: gate, 1: down), in the order expert, tile of weight rows, tokens, and a CTA's share of
// their stages: pieces of jobs, stages l0 .. l1 - 1 of each.  (One code for both products: the second time it is
// there, see kWarpSpare.)
template <bool FP8, int C>
struct Walk {
    const uint16_t *before;
    int tokens;                        // most of a job
    int tiles, lines, d, part, parts;  // tiles of an expert, stages of a job, live expert, its tokens' part and parts
    int e, tile, first, count;         // the job: expert, tile, its tokens' places in the list
    int l0, l1;
    uint32_t left;                     // stages of the share from this piece on
    __device__ __forceinline__ void expert(const Route &r) {
        e = r.live[d];
        parts = before[d + 1] - before[d];
    }
    __device__ __forceinline__ void job(const Route &r) {
        first = r.first[e] + part * tokens;
        count = min(tokens, r.first[e + 1] - first);
        l1 = min(lines, l0 + (int)min(left, 0x7FFFFFFFu));
    }
    // To the first piece of the stages from .. to - 1; false: there are none.
    __device__ __forceinline__ bool start(const Route &r, int down, int tiles_, int lines_, uint32_t from, uint32_t to) {
        if (from == to) return false;
        before = down ? r.before[1] : r.before[0];
        tokens = down ? kTokens<FP8, true, C> : kTokens<FP8, false, C>;
        tiles = tiles_;
        lines = lines_;
        left = to - from;
        const uint32_t q = from / lines;
        l0 = (int)(from - q * lines);
        int lo = 0, hi = r.D - 1;  // the last d with before[d] * tiles <= q
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((uint32_t)before[mid] * tiles <= q)
                lo = mid;
            else
                hi = mid - 1;
        }
        d = lo;
        expert(r);
        const uint32_t rest = q - (uint32_t)before[lo] * tiles;
        tile = (int)(rest / parts);
        part = (int)(rest - tile * parts);
        job(r);
        return true;
    }
    __device__ __forceinline__ bool next(const Route &r) {
        left -= l1 - l0;
        if (left == 0) return false;
        l0 = 0;
        if (++part == parts) {
            part = 0;
            if (++tile == tiles) {
                tile = 0;
                ++d;
                expert(r);
            }
        }
        job(r);
        return true;
    }
};

struct Maps {
    CUtensorMap w[2];  // gate and up, down: [E, rows, channels] in boxes of 64 rows x 128 bytes, swizzled
    CUtensorMap h;     // h laid out by entry: [entries * R, channels] in boxes of 16 rows x 128 bytes
    CUtensorMap x;     // tokens laid out by entry, the same
};

template <int C>
struct Bars {
    uint64_t full[12], empty[12], tfull[kSums], tempty[kSums];
    uint32_t armed[1 + kTokenWarps];  // stages loaded (weights; by each token warp of its own)
    uint32_t failed, tmem;
    float scale[kScales][C / 2];  // what a code of an entry is worth
};

// The stages of a product in equal shares: CTA b has those from from(b) on, the first `more` CTAs one more.
struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ uint32_t from(uint32_t b) const { return each * b + min(b, more); }
    __device__ __forceinline__ int owner(uint32_t u) const {
        const uint32_t first = more * (each + 1);
        return (int)(u < first ? u / (each + 1) : more + (u - first) / each);
    }
};

// The power of two that brings top to 128 .. 256 (within fp32's own), and 1 over it.
__device__ __forceinline__ float2 scale_of(float top) {
    if (top == 0.0f) return make_float2(1.0f, 1.0f);
    const int ex = max((int)(__float_as_uint(top) >> 23), 1) - 127;        // top = 1.. * 2^ex
    const int k = min(7 - ex, 126);
    return make_float2(__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23));
}

// v times s as the sum of R e4m3 codes, code r worth 2^(-4 r): four bytes at a time to store(r, j, .).  What is
// not finite becomes NaN.
template <int R, int N, typename F>
__device__ __forceinline__ void codes(float (&v)[N], float s, F &&store) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = isfinite(v[i]) ? v[i] * s : __int_as_float(0x7FC00000);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            uint32_t w = 0;
#pragma unroll
            for (int i = j; i < j + 4; i += 2) {
                const __nv_fp8x2_storage_t q = __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, __NV_E4M3);
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(q, __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                v[i] = (v[i] - f.x) * 16.0f;
                v[i + 1] = (v[i + 1] - f.y) * 16.0f;
                w |= (uint32_t)q << (8 * (i - j));
            }
            store(r, j / 4, w);
        }
    }
}

// The scale of a block of 128 channels, N to a lane.
template <int N>
__device__ __forceinline__ float2 block_scale(const float (&v)[N]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, isfinite(v[i]) ? fabsf(v[i]) : 0.0f);
#pragma unroll
    for (int o = 64 / N; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return scale_of(top);
}

template <bool FP8, int C>
__global__ void __launch_bounds__(kThreads, 1) expert_layer_kernel(const __grid_constant__ Maps maps, const ExpertLayerParams p) {
    constexpr int kStages = Shape<FP8, C>::STAGES, kStage = Shape<FP8, C>::STAGE;
    const bool laid = Shape<FP8, C>::LAID && p.laid;
    const int at_gate = laid ? 2 : 1, at_h = at_gate + 1, at_down = at_gate + 2;  // meetings: gate done, h laid out, down done
    extern __shared__ uint8_t dyn[];
    __shared__ Bars<C> bars;
    uint8_t *const ring = reinterpret_cast<uint8_t *>(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = gridDim.x, cta = blockIdx.x;
    const uint32_t b_full = saddr(bars.full), b_empty = saddr(bars.empty), b_tfull = saddr(bars.tfull), b_tempty = saddr(bars.tempty);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(b_full + 8 * i, 2);  // the weights' loader and a token warp
            bar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < kSums; ++i) {
            bar_init(b_tfull + 8 * i, 1);
            bar_init(b_tempty + 8 * i, 4);
        }
        bar_init_fence();
        bars.failed = 0;
        for (int i = 0; i <= kTokenWarps; ++i) bars.armed[i] = 0;
        prefetch_map(&maps.w[0]);
        prefetch_map(&maps.w[1]);
        prefetch_map(&maps.h);
        if (laid) prefetch_map(&maps.x);
    }
    if (warp == kWarpMma) tmem_alloc_one(saddr(&bars.tmem), kSums * C);
    pdl_wait();
    const Route r = route<FP8, C>(p, ring + kStages * kStage, reinterpret_cast<uint32_t *>(ring));
    const bool worker = warp < 4 || warp >= 8;
    const int wid = warp < 4 ? tid : tid - 128;  // of a worker
    // tiles of an expert's weights, stages of a job, rows of the tiles
    const int tiles[2] = {(p.I + kTile / 2 - 1) / (kTile / 2), (p.H + kTile - 1) / kTile};
    const int lines[2] = {(p.H + kLine<FP8> - 1) / kLine<FP8>, (p.I + kLine<FP8> - 1) / kLine<FP8>};
    Shares shares[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t total = (uint32_t)tiles[d] * r.before[d][r.D] * lines[d];
        shares[d].each = total / ctas;
        shares[d].more = total - shares[d].each * ctas;
    }
    fence_async_shared();  // the scratch lies where the stages land
    fence_before();
    __syncthreads();
    fence_after();
    // A wait that has given up ends its warp's waits; one thread may know of it alone (`met`), so that every
    // wait of a warp is one of all its lanes.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool there = ok;
        if (there) there = bar_wait(bar, parity, p.wait_cycles);
        return __all_sync(0xFFFFFFFFu, there);
    };
    // All CTAs' workers have come to the i-th meeting; by one thread.
    auto met = [&](uint32_t i) {
        const long long t0 = clock64();
        uint32_t v;
        do {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.barrier) : "memory");
            if (v >= i * ctas) return true;
        } while (clock64() - t0 < p.wait_cycles);
        return false;
    };

    // this CTA's share of a product
    auto begin = [&](Walk<FP8, C> &w, int down) {
        return w.start(r, down, down ? tiles[1] : tiles[0], down ? lines[1] : lines[0], (down ? shares[1] : shares[0]).from(cta),
                       (down ? shares[1] : shares[0]).from(cta + 1));
    };

    if (r.D > 0 && warp == kWarpWeights) {
        uint32_t n = 0;
#pragma unroll 1
        for (int down = 0; down < 2; ++down) {
            Walk<FP8, C> w;
            if (!ok || !begin(w, down)) continue;
            const CUtensorMap *const map = &maps.w[down];
            do {
                if (w.e == p.withhold) ok = false;  // test hook
                const int row0 = w.tile * (down ? kTile : kTile / 2), row1 = row0 + (down ? kTile / 2 : p.I);
                for (int l = w.l0; l < w.l1 && ok; ++l) {
                    const uint32_t slot = n % kStages;
                    ok = wait(b_empty + 8 * slot, (n / kStages & 1) ^ 1);
                    if (!ok) break;
                    ++n;
                    if (elect()) {
                        const uint32_t bar = b_full + 8 * slot, at = saddr(ring + slot * kStage);
                        bar_expect(bar, kWeightBytes);
                        load_box(at, map, l * kLine<FP8>, row0, w.e, bar);
                        load_box(at + kWeightBytes / 2, map, l * kLine<FP8>, row1, w.e, bar);
                    }
                    __syncwarp();
                }
            } while (ok && w.next(r));
        }
        if (lane == 0) bars.armed[0] = n;
    } else if (r.D > 0 && warp == kWarpMma) {
        uint32_t n = 0, seg = 0;
#pragma unroll 1
        for (int down = 0; down < 2; ++down) {
            const int R = down ? kParts<FP8, true> : kParts<FP8, false>;
            Walk<FP8, C> w;
            if (!ok || !begin(w, down)) continue;
            do {
                // fp32 accumulator, both operands bf16 or both e4m3, 128 x columns
                const uint32_t columns = (w.count * R + 15) & ~15;
                const uint32_t id = (1u << 4) | (FP8 ? 0u : (1u << 7 | 1u << 10)) | (columns >> 3) << 17 | (kTile >> 4) << 24;
                for (int l = w.l0; l < w.l1 && ok; ++l) {
                    const uint32_t slot = n % kStages, buf = seg % kSums;
                    const bool begins = FP8 || l == w.l0, ends = FP8 || l == w.l1 - 1;
                    ok = wait(b_full + 8 * slot, n / kStages & 1);
                    if (ok && begins) ok = wait(b_tempty + 8 * buf, (seg / kSums & 1) ^ 1);
                    if (!ok) break;
                    fence_after();
                    ++n;
                    if (elect()) {
                        const uint32_t a = saddr(ring + slot * kStage), b = a + kWeightBytes;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_one<FP8>(bars.tmem + buf * C, desc(a + j * 32, 16), desc(b + j * 32, 16), id, !begins || j != 0);
                        commit_one(b_empty + 8 * slot);
                        if (ends) commit_one(b_tfull + 8 * buf);
                    }
                    __syncwarp();
                    if (ends) ++seg;
                }
            } while (ok && w.next(r));
        }
        // all products have been computed before tensor memory is given back
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
            if (!__all_sync(0xFFFFFFFFu, bar_wait(b_empty + 8 * (i % kStages), i / kStages & 1, p.wait_cycles))) ok = false;
    } else if (worker || (r.D > 0 && warp == kWarpSpare)) {
        const bool spare = warp == kWarpSpare;
        uint32_t seg = 0, stages = 0, brought = 0;  // accumulators read; stages gone by and brought (token warps)
        // Comes to the i-th meeting: what this CTA's workers wrote can be read behind it.  Not before all have
        // come to the one before, for which this CTA has not waited where only its tokens do: a CTA without a
        // share would be counted for a slow one.
        auto come = [&](uint32_t i) {
            workers_sync();
            if (wid == 0) {
                if ((i == at_down || (laid && i == at_gate)) && !met(i - 1)) ok = false;
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.barrier) : "memory");
            }
        };
        auto meet = [&](uint32_t i) {
            come(i);
            if (wid == 0 && ok && !met(i)) ok = false;
            workers_sync();
        };
        // Where the sums of entry `spot` for a tile are: in its row of p.sums, and in the pieces that other CTAs
        // than the one where the job begins had of it.
        struct Where {
            int d, part, at, parts;  // live expert, part of its tokens, place in the part, parts
        };
        auto where = [&](int down, int spot) {
            int lo = 0, hi = r.D - 1;  // the last live expert that begins at or before the entry
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (r.first[r.live[mid]] <= spot)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int tokens = down ? kTokens<FP8, true, C> : kTokens<FP8, false, C>;
            const int within = spot - r.first[r.live[lo]];
            return Where{lo, within / tokens, within % tokens, (down ? r.before[1] : r.before[0])[lo + 1] - (down ? r.before[1] : r.before[0])[lo]};
        };
        auto pieces = [&](int down, const Where &w, int tile) {
            const uint32_t u = ((uint32_t)r.before[down][w.d] * tiles[down] + tile * w.parts + w.part) * lines[down];
            return make_int2(shares[down].owner(u), shares[down].owner(u + lines[down] - 1));
        };
        // Tokens of every eighth stage, rows of 128 bytes, swizzled as the weights are.  Gate: x, by this warp; down (and
        // gate, laid): by tensor map, once all have laid theirs out.  (x not by read-only loads: `out` may be x.)
        auto bring = [&](auto down) {
            constexpr bool DOWN = decltype(down)::value;
            constexpr int R = kParts<FP8, DOWN>;
            Walk<FP8, C> w;
            if (!begin(w, DOWN)) return;
            if (DOWN || laid) {
                if (lane == 0 && !met(DOWN ? at_h : 1)) ok = false;
                asm volatile("fence.proxy.async;" ::: "memory");
                ok = __all_sync(0xFFFFFFFFu, ok);
            }
            do {
                for (int l = w.l0; l < w.l1; ++l, ++stages) {
                    if (stages % kTokenWarps != warp - kWarpTokens) continue;
                    const uint32_t slot = stages % kStages, bar = b_full + 8 * slot, at = saddr(ring + slot * kStage) + kWeightBytes;
                    if (DOWN || laid) {
                        const CUtensorMap *const map = DOWN ? &maps.h : &maps.x;
                        float s = 0.0f;
                        if (FP8 && lane < w.count) s = __ldcg((DOWN ? p.h_scale : p.x_scale) + (int64_t)(w.first + lane) * lines[DOWN] + l);
                        ok = wait(b_empty + 8 * slot, (stages / kStages & 1) ^ 1);
                        if (!ok) return;
                        if (elect()) {
                            // expected now, arrived for below
                            const int boxes = (w.count * R + 15) / 16;
                            asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(boxes * 2048) : "memory");
                            for (int i = 0; i < boxes; ++i) load_box(at + i * 2048, map, l * kLine<FP8>, w.first * R + i * 16, bar);
                        }
                        __syncwarp();
                        if (FP8 && lane < w.count) bars.scale[stages % kScales][lane] = s;
                    } else if constexpr (FP8) {
                        // four entries at a time, 16 channels to a lane
                        struct Two {
                            uint4 a, b;
                        };
                        auto get = [&](int i) {
                            const uint4 *src = reinterpret_cast<const uint4 *>(
                                static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)(r.list[w.first + min(i, w.count - 1)] >> 5) * p.H + l * 128 +
                                (lane & 7) * 16);
                            return Two{src[0], src[1]};
                        };
                        Two next = get(lane >> 3);
                        ok = wait(b_empty + 8 * slot, (stages / kStages & 1) ^ 1);
                        if (!ok) return;
                        for (int i0 = 0; i0 < w.count; i0 += 4) {
                            const Two q = next;
                            const int i = i0 + (lane >> 3);
                            if (i0 + 4 < w.count) next = get(i + 4);
                            const uint32_t q8[8] = {q.a.x, q.a.y, q.a.z, q.a.w, q.b.x, q.b.y, q.b.z, q.b.w};
                            float v[16];
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[2 * k] = bf16_lo(q8[k]), v[2 * k + 1] = bf16_hi(q8[k]);
                            const float2 s = block_scale(v);
                            uint32_t c[2][4];
                            codes<2>(v, s.x, [&](int k, int j, uint32_t x) { c[k][j] = x; });
                            if (i < w.count) {
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int row = i * 2 + k;
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + row * 128 + (((lane & 7) ^ (row & 7)) << 4)),
                                                 "r"(c[k][0]), "r"(c[k][1]), "r"(c[k][2]), "r"(c[k][3])
                                                 : "memory");
                                }
                                if ((lane & 7) == 0) bars.scale[stages % kScales][i] = s.y;
                            }
                        }
                    } else {
                        // four entries at a time, 8 channels to a lane; past the last channel zeros (the weights are
                        // zeros there, but times what was in the ring that may be NaN)
                        const int c = l * 64 + (lane & 7) * 8;
                        auto get = [&](int i) {
                            uint4 q = make_uint4(0, 0, 0, 0);
                            if (i < w.count && c < p.H)
                                q = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) +
                                                                     (int64_t)(r.list[w.first + i] >> 5) * p.H + c);
                            return q;
                        };
                        constexpr int U = C == 16 ? 2 : 8;  // loads in flight (128 tokens, top-2 of 8, 4096 x 4096: 1 227 us, 8 176)
                        uint4 next[U];
#pragma unroll
                        for (int u = 0; u < U; ++u) next[u] = get(u * 4 + (lane >> 3));
                        ok = wait(b_empty + 8 * slot, (stages / kStages & 1) ^ 1);
                        if (!ok) return;
                        const int rows = (w.count + 3) & ~3;
#pragma unroll 1
                        for (int i0 = lane >> 3; i0 < rows; i0 += 4 * U) {
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const int i = i0 + u * 4;
                                if (i >= rows) break;
                                const uint4 q = next[u];
                                next[u] = get(i + 4 * U);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + i * 128 + (((lane & 7) ^ (i & 7)) << 4)),
                                             "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                                             : "memory");
                            }
                        }
                    }
                    if (!DOWN && !laid) fence_async_shared();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar);
                    ++brought;
                }
            } while (w.next(r));
        };
        // Sums out of tensor memory: lane = weight row.
        auto product = [&](auto down) {
            constexpr bool DOWN = decltype(down)::value;
            constexpr int R = kParts<FP8, DOWN>, TOKENS = kTokens<FP8, DOWN, C>;
            if (warp >= kWarpTokens) {
                if (ok) bring(down);
                return;
            }
            Walk<FP8, C> w;
            if (!begin(w, DOWN)) return;
            const uint32_t lanes = bars.tmem + ((uint32_t)(warp * 32) << 16);
            const int kb = lines[DOWN], nb = ((DOWN ? p.H : 2 * p.I) + 127) / 128;
            do {
                const int columns = w.count * R;
                float acc[FP8 ? TOKENS : 1];
                float ws = 0.0f;
                // from tensor memory, 16 columns at a time: f(entry, sum of its columns)
                auto columns_of = [&](uint32_t buf, auto &&f) {
                    ok = wait(b_tfull + 8 * buf, seg / kSums & 1);
                    fence_after();
#pragma unroll
                    for (int q = 0; q < C / 16; ++q) {
                        if (q * 16 >= columns) break;
                        uint32_t v[16];
                        tmem_get16(v, lanes + buf * C + q * 16);
                        if ((q + 1) * 16 >= columns) {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive(b_tempty + 8 * buf);
                        }
#pragma unroll
                        for (int i = 0; i < 16 / R; ++i) {
                            float s = __uint_as_float(v[i * R + R - 1]);
#pragma unroll
                            for (int k = R - 2; k >= 0; --k) s = fmaf(s, FP8 ? 0.0625f : 1.0f, __uint_as_float(v[i * R + k]));
                            f(q * (16 / R) + i, s);
                        }
                    }
                    ++seg;
                };
                float *const to = w.l0 == 0 ? p.sums + (int64_t)w.first * (tiles[DOWN] * kTile) + w.tile * kTile + warp * 32 + lane
                                            : p.pieces + (int64_t)cta * C * kTile + warp * 32 + lane;
                const int64_t ld = w.l0 == 0 ? tiles[DOWN] * kTile : kTile;
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) acc[i] = 0.0f;
                    // the scales of 32 stages, one per lane; gate: the first two warps have gate rows, the others up rows
                    const int row = DOWN ? w.tile * kTile : w.tile * (kTile / 2) + (warp >> 1) * p.I;
                    const float *sc = (DOWN ? p.s_down : p.s_gate_up) + ((int64_t)w.e * nb + row / 128) * kb;
                    for (int l = w.l0; l < w.l1; ++l) {
                        if ((l - w.l0 & 31) == 0) ws = l + lane < w.l1 ? __ldg(sc + l + lane) : 0.0f;
                        const float f = __shfl_sync(0xFFFFFFFFu, ws, l - w.l0 & 31);
                        const float *xs = bars.scale[seg % kScales];  // a stage an accumulator
                        columns_of(seg % kSums, [&](int i, float s) { acc[i] = fmaf(s, f * xs[i], acc[i]); });
                    }
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i)
                        if (i < w.count) __stcg(to + i * ld, acc[i]);
                } else {
                    columns_of(seg % kSums, [&](int i, float s) {
                        if (i < w.count) __stcg(to + i * ld, s);
                    });
                }
            } while (w.next(r));
        };
        if (r.D > 0) {
            const int entries = r.first[p.E];
            // h: a warp takes 128 channels of an entry, 4 to a lane.  What does not hang on the sums is looked up before
            // they are there (the first item's; few tokens have no more).
            const int rows = tiles[0] * kTile, blocks = (p.I + 127) / 128, warps = ctas * (kWorkers / 32);
            struct Item {
                const float *own, *piece;  // sums: of the CTA where the job begins, of the first one behind it
                int others;                // CTAs behind it
                uint2 gate, up;            // biases
            };
            auto look = [&](int it) {
                Item q = {nullptr, nullptr, 0, make_uint2(0, 0), make_uint2(0, 0)};
                const int i = it / blocks, c = (it - i * blocks) * 128 + lane * 4;
                if (it >= entries * blocks || c >= p.I) return q;
                const Where w = where(0, i);
                const int tile = c / (kTile / 2), at = c % (kTile / 2);
                const int2 who = pieces(0, w, tile);
                q.own = p.sums + (int64_t)i * rows + tile * kTile + at;
                q.piece = p.pieces + ((int64_t)(who.x + 1) * C + w.at) * kTile + at;
                q.others = who.y - who.x;
                if (p.b_gate_up != nullptr) {
                    const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p.b_gate_up) + (int64_t)r.live[w.d] * 2 * p.I + c;
                    q.gate = __ldg(reinterpret_cast<const uint2 *>(b));
                    q.up = __ldg(reinterpret_cast<const uint2 *>(b + p.I));
                }
                return q;
            };
            const int it0 = spare ? 0 : cta * (kWorkers / 32) + (wid >> 5);
            if (laid) {
                // a warp takes 128 channels of a token, 4 to a lane, for all its entries
                for (int it = it0; it < p.N * lines[0] && !spare; it += warps) {
                    const int t = it / lines[0], l = it - t * lines[0];
                    const uint2 q = reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)t * p.H + l * 128)[lane];
                    float v[4] = {bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
                    const float2 s = block_scale(v);
                    uint32_t c[2];
                    codes<2>(v, s.x, [&](int k, int, uint32_t w) { c[k] = w; });
                    for (int k = 0; k < p.K; ++k) {
                        const uint32_t i = r.spot[t * p.K + k];
                        if (i == 0xFFFFu) continue;
                        uint8_t *const dst = static_cast<uint8_t *>(p.xq) + (int64_t)i * 2 * p.H + l * 128 + lane * 4;
                        *reinterpret_cast<uint32_t *>(dst) = c[0];
                        *reinterpret_cast<uint32_t *>(dst + p.H) = c[1];
                        if (lane == 0) p.x_scale[(int64_t)i * lines[0] + l] = s.y;
                    }
                }
                if (!spare) {
                    asm volatile("fence.proxy.async;" ::: "memory");  // read by copies
                    come(1);
                }
            }
            if (!spare) product(std::false_type{});
            Item item = look(it0);
            if (!spare) meet(at_gate);
            for (int it = it0; it < entries * blocks; it += warps) {
                if (it != it0) item = look(it);
                const int i = it / blocks, c = (it - i * blocks) * 128 + lane * 4;
                float h[4] = {};
                if (c < p.I) {
                    float4 g = __ldcg(reinterpret_cast<const float4 *>(item.own));
                    float4 u = __ldcg(reinterpret_cast<const float4 *>(item.own + kTile / 2));
                    for (int b0 = 0; b0 < item.others; b0 += 4) {
                        float4 x[4], y[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float *q = item.piece + (int64_t)min(b0 + b, item.others - 1) * C * kTile;
                            x[b] = __ldcg(reinterpret_cast<const float4 *>(q));
                            y[b] = __ldcg(reinterpret_cast<const float4 *>(q + kTile / 2));
                        }
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (b0 + b >= item.others) break;
                            g = make_float4(g.x + x[b].x, g.y + x[b].y, g.z + x[b].z, g.w + x[b].w);
                            u = make_float4(u.x + y[b].x, u.y + y[b].y, u.z + y[b].z, u.w + y[b].w);
                        }
                    }
                    const float g4[4] = {g.x + bf16_lo(item.gate.x), g.y + bf16_hi(item.gate.x), g.z + bf16_lo(item.gate.y),
                                         g.w + bf16_hi(item.gate.y)};
                    const float u4[4] = {u.x + bf16_lo(item.up.x), u.y + bf16_hi(item.up.x), u.z + bf16_lo(item.up.y),
                                         u.w + bf16_hi(item.up.y)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = silu(g4[k]) * u4[k];
                }
                if (spare) {
                    asm volatile("" ::"f"(h[0]), "f"(h[1]), "f"(h[2]), "f"(h[3]));
                    break;
                }
                if constexpr (FP8) {
                    const float2 s = block_scale(h);
                    uint8_t *const dst = static_cast<uint8_t *>(p.h) + (int64_t)i * 4 * p.I + c;
                    codes<4>(h, s.x, [&](int q, int, uint32_t w) { *reinterpret_cast<uint32_t *>(dst + (int64_t)q * p.I) = w; });
                    if (lane == 0) p.h_scale[it] = s.y;
                } else if (c < p.I) {
                    // the sum of two bf16 numbers, 2^-17 of the value off at most: rounded to one, h alone would put
                    // as much error into the result as its own rounding
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const __nv_bfloat162 a = __floats2bfloat162_rn(h[2 * k], h[2 * k + 1]);
                        const float2 f = __bfloat1622float2(a);
                        const __nv_bfloat162 b = __floats2bfloat162_rn(isfinite(f.x) ? h[2 * k] - f.x : 0.0f,
                                                                       isfinite(f.y) ? h[2 * k + 1] - f.y : 0.0f);
                        hi[k] = *reinterpret_cast<const uint32_t *>(&a);
                        lo[k] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.h) + (int64_t)i * 2 * p.I + c;
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(dst + p.I) = make_uint2(lo[0], lo[1]);
                }
            }
            if (!spare) {
                asm volatile("fence.proxy.async;" ::: "memory");  // h is read by copies
                come(at_h);
                product(std::true_type{});
            }
        }
        // out: a warp takes a token and the 128 channels of a tile; lane k looks entry k up, again before the sums
        // are there
        struct Item {
            int spot, at, e, b0, others;  // entry (-1: none), place in its job's tokens, expert, CTAs that have sums
            float weight;
            uint2 residual;               // of the lane's channels
        };
        auto look = [&](int it) {
            Item q = {-1, 0, 0, 0, 0, 0.0f, make_uint2(0, 0)};
            if (it >= p.N * tiles[1]) return q;
            const int t = it / tiles[1], tile = it - t * tiles[1], c = tile * kTile + lane * 4;
            if (p.residual != nullptr && c < p.H)
                q.residual = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.residual) + (int64_t)t * p.H + c);
            const uint32_t v = lane < p.K ? r.spot[t * p.K + lane] : 0xFFFFu;
            if (v == 0xFFFFu) return q;
            q.weight = p.wts != nullptr ? __ldg(p.wts + t * p.K + lane) : 1.0f;
            const Where w = where(1, (int)v);
            const int2 who = pieces(1, w, tile);
            q.spot = (int)v;
            q.at = w.at;
            q.e = r.live[w.d];
            q.b0 = who.x;
            q.others = who.y - who.x;
            return q;
        };
        const int it0 = spare ? 0 : cta * (kWorkers / 32) + (wid >> 5);
        Item item = look(it0);
        if (r.D > 0 && !spare) meet(at_down);
        for (int it = it0; it < p.N * tiles[1]; it += ctas * (kWorkers / 32)) {
            if (it != it0) item = look(it);
            const int t = it / tiles[1], c = (it - t * tiles[1]) * kTile + lane * 4;
            const bool in = c < p.H;
            float v[4] = {};
            constexpr int U = 4;  // entries whose loads are in flight together
            for (int k0 = 0; k0 < p.K; k0 += U) {
                float4 y[U], z[U];
                uint2 bias[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int k = k0 + j, s = __shfl_sync(0xFFFFFFFFu, item.spot, k), e = __shfl_sync(0xFFFFFFFFu, item.e, k);
                    const int b0 = __shfl_sync(0xFFFFFFFFu, item.b0, k), at = __shfl_sync(0xFFFFFFFFu, item.at, k);
                    const int others = __shfl_sync(0xFFFFFFFFu, item.others, k);
                    const bool there = k < p.K && s >= 0 && in;
                    y[j] = z[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    bias[j] = make_uint2(0, 0);
                    if (there) y[j] = __ldcg(reinterpret_cast<const float4 *>(p.sums + (int64_t)s * (tiles[1] * kTile) + c));
                    const float *piece = p.pieces + ((int64_t)(b0 + 1) * C + at) * kTile + lane * 4;
                    if (there && others > 0) z[j] = __ldcg(reinterpret_cast<const float4 *>(piece));
                    if (there && p.b_down != nullptr)
                        bias[j] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.b_down) + (int64_t)e * p.H + c));
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int k = k0 + j, s = __shfl_sync(0xFFFFFFFFu, item.spot, k), at = __shfl_sync(0xFFFFFFFFu, item.at, k);
                    const int b0 = __shfl_sync(0xFFFFFFFFu, item.b0, k), others = __shfl_sync(0xFFFFFFFFu, item.others, k);
                    const float w = __shfl_sync(0xFFFFFFFFu, item.weight, k);
                    if (k >= p.K || s < 0) continue;
                    y[j] = make_float4(y[j].x + z[j].x, y[j].y + z[j].y, y[j].z + z[j].z, y[j].w + z[j].w);
                    for (int b = 2; b <= others; b += 4) {
                        float4 q[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[i] = __ldcg(reinterpret_cast<const float4 *>(p.pieces +
                                                                           ((int64_t)(b0 + min(b + i, others)) * C + at) * kTile + lane * 4));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (b + i > others) break;
                            y[j] = make_float4(y[j].x + q[i].x, y[j].y + q[i].y, y[j].z + q[i].z, y[j].w + q[i].w);
                        }
                    }
                    v[0] = fmaf(w, y[j].x + bf16_lo(bias[j].x), v[0]);
                    v[1] = fmaf(w, y[j].y + bf16_hi(bias[j].x), v[1]);
                    v[2] = fmaf(w, y[j].z + bf16_lo(bias[j].y), v[2]);
                    v[3] = fmaf(w, y[j].w + bf16_hi(bias[j].y), v[3]);
                }
            }
            if (spare) {
                asm volatile("" ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
                break;
            }
            if (!in) continue;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0] + bf16_lo(item.residual.x), v[1] + bf16_hi(item.residual.x));
            const __nv_bfloat162 hi = __floats2bfloat162_rn(v[2] + bf16_lo(item.residual.y), v[3] + bf16_hi(item.residual.y));
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + (int64_t)t * p.H + c) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
        if (warp >= kWarpTokens && lane == 0) bars.armed[1 + warp - kWarpTokens] = brought;
    }
    if (!ok) {
        bars.failed = 1;
        atomicOr(p.status, kStatusTimeout);
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kWarpMma) tmem_free_one(bars.tmem, kSums * C);
    if (r.D == 0) return;
    if (tid == 0) {
        if (bars.failed) {
            // loads in flight land before the shared memory is given up: where only one side came, the other's
            // arrival is made up for
            uint32_t last = bars.armed[0];
            for (int i = 0; i < kTokenWarps; ++i)
                if (bars.armed[1 + i] > 0) last = max(last, (bars.armed[1 + i] - 1) * kTokenWarps + i + 1);
            for (uint32_t n = last > kStages ? last - kStages : 0; n < last; ++n) {
                const bool weights = n < bars.armed[0], tokens = n / kTokenWarps < bars.armed[1 + n % kTokenWarps];
                if (!weights && !tokens) continue;
                if (weights != tokens) bar_arrive(b_full + 8 * (n % kStages));
                if (!bar_wait(b_full + 8 * (n % kStages), n / kStages & 1, p.wait_cycles)) atomicOr(p.status, kStatusInFlight);
            }
        }
        // The last CTA puts the barrier back, behind all arrivals: one that came to its last meeting has seen them
        // all there; a CTA whose waits have given up has not, so its own are done before it is counted, and where
        // it is the last, it has those of the CTAs counted before it.
        if (bars.failed) __threadfence();
        if (atomicAdd(p.barrier + 1, 1u) == gridDim.x - 1) {
            if (bars.failed) __threadfence();
            p.barrier[0] = 0;
            p.barrier[1] = 0;
        }
    }
}

template <bool FP8, int C>
cudaError_t launch(const Maps &maps, const ExpertLayerParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.sms, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Shape<FP8, C>::fixed + route_bytes(p.E, p.N * p.K);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident: the grid barriers end
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, expert_layer_kernel<FP8, C>, maps, p);
}

// Most bytes of weights (of as many experts as there are entries) of the small form, for up to 4 entries per
// expert on average: past 8 it reads the weights again, where the large form has columns left.  The host knows the
// mean only: where one expert is named by all tokens, the CTAs that have its units are waited for (128 tokens, top-8
// of 256, 512 x 64, bf16: 101 us, even routing 57; 64 tokens, top-8 of 128, 1024 x 128: 40 and 34).  Us, small /
// large form, captured, the weights from HBM, even routing:
//   bf16  13 MB 11.6/18.6   25 MB 15.1/20.2   75 MB 25.7/27.9   83 MB 26.9/27.7   130 MB 36.5/35.7   151 MB 38.2/39.2
//         8 entries per expert: 104 MB 41/35   32: 25 MB 34/27
//   e4m3  38 MB 23.7/23.0   41 MB 23.2/22.9   50 MB 23.0/24.1   73 MB 32.7/29.0
//         8 entries per expert: 8 MB 20.6/19.4   12: 32 MB 40/25
constexpr double kSmallBytes[2] = {96e6, 32e6};  // bf16, e4m3

// Most tokens of a call whose jobs have 16 columns at most (one token, top-8 of 256, 7168 x 2048, FP8: 72 us with
// 12 stages, 74 with the 8 of the other form).
template <bool FP8>
constexpr int kFewTokens = kTokens<FP8, true, 16>;

template <bool FP8, int C>
void allow_smem() {
    // failing here means failing at the launch, which reports it
    const int tokens = C == 16 ? kFewTokens<FP8> : kLayerMaxTokens;
    if (cudaFuncSetAttribute(expert_layer_kernel<FP8, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(Shape<FP8, C>::fixed + route_bytes(1024, tokens * 32))) != cudaSuccess)
        cudaGetLastError();
}

// e4m3: from this many times on that an SM turns 128 channels of an entry into codes for a stage of the gate
// product, all SMs lay the tokens out as codes once, before, and meet once more.  Us, each tile its own / laid out
// (times; tokens, top-k of experts, channels):
//   65 (46, 2 of 7, 1152 x 768) 22.4/24.9   161 (8, 6 of 64, 4096 x 1024) 92/94   471 (5, 8 of 32, 7168 x 2048) 168.6/170.9
//   1160 (105, 8 of 14, 896 x 1920) 79.0/72.1   1725 (64, 2 of 8, 4096 x 4096) 114/103   3018 (32, 8 of 256, 7168 x 2048)
//   1096/1084   3449 (128, 2 of 8, 4096 x 4096) 198/161   12072 (128, 8 of 32, 7168 x 2048) 620/490
constexpr double kLaidStages = 800;

// The workspace's parts, each on a 256-byte boundary: sets their addresses from `base` on, returns the size.
size_t lay_out(ExpertLayerParams &p, uint8_t *base) {
    const size_t M = (size_t)p.N * p.K;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *const q = base + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    const size_t gate = (size_t)((p.I + kTile / 2 - 1) / (kTile / 2)) * kTile, down = (size_t)((p.H + kTile - 1) / kTile) * kTile;
    p.h = take(M * p.I * 4);
    p.sums = reinterpret_cast<float *>(take(M * (gate > down ? gate : down) * 4));
    p.pieces = reinterpret_cast<float *>(take((size_t)p.sms * kMostColumns * kTile * 4));
    p.h_scale = reinterpret_cast<float *>(take(M * ((p.I + 127) / 128) * 4));
    p.xq = take(M * p.H * 2);
    p.x_scale = reinterpret_cast<float *>(take(M * ((p.H + 127) / 128) * 4));
    uint32_t *const barrier = reinterpret_cast<uint32_t *>(take(8));
    if (p.barrier == nullptr) p.barrier = barrier;
    return at;
}

}  // namespace

void expert_layer_init() {
    allow_smem<false, 16>();
    allow_smem<false, 64>();
    allow_smem<true, 16>();
    allow_smem<true, 64>();
}

size_t expert_layer_workspace(ExpertLayerParams p) {
    const size_t large = lay_out(p, nullptr), small = expert_layer_small_workspace(p);
    return large > small ? large : small;
}

bool expert_layer_small(const ExpertLayerParams &p) {
    const double entries = (double)p.N * p.K, experts = entries < p.E ? entries : p.E;
    const double bytes = 3.0 * experts * p.H * p.I * (p.s_gate_up != nullptr ? 1 : 2);
    return entries <= 4.0 * p.E && bytes <= kSmallBytes[p.s_gate_up != nullptr];
}

cudaError_t launch_expert_layer(ExpertLayerParams p, void *workspace, cudaStream_t stream) {
    if (expert_layer_small(p)) return launch_expert_layer_small(p, workspace, stream);
    const bool fp8 = p.s_gate_up != nullptr, own = p.barrier != nullptr;
    lay_out(p, static_cast<uint8_t *>(workspace));
    if (!own) {
        // no counter of the context's left: the workspace's, cleared by a call of its own
        const cudaError_t e = cudaMemsetAsync(p.barrier, 0, 8, stream);
        if (e != cudaSuccess) return e;
    }
    const int es = fp8 ? 1 : 2;
    const int64_t M = (int64_t)p.N * p.K;
    Maps maps;
    if (!encode_rows(&maps.w[0], p.w_gate_up, es, p.H, 2 * (int64_t)p.I, p.E, kTile / 2) ||
        !encode_rows(&maps.w[1], p.w_down, es, p.I, p.H, p.E, kTile / 2) ||
        !encode_rows(&maps.h, p.h, es, p.I, M * (fp8 ? 4 : 2), 0, 16) || !encode_rows(&maps.x, p.xq, es, p.H, M * (fp8 ? 2 : 1), 0, 16))
        return cudaErrorInvalidValue;
    p.laid = (double)M * ((p.I + kTile / 2 - 1) / (kTile / 2)) * (p.H / 128) >= kLaidStages * p.sms;
    if (fp8) return p.N <= kFewTokens<true> ? launch<true, 16>(maps, p, stream) : launch<true, 64>(maps, p, stream);
    return p.N <= kFewTokens<false> ? launch<false, 16>(maps, p, stream) : launch<false, 64>(maps, p, stream);
}

}  // namespace ep

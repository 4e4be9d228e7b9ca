// Backward pass of the epilogue of a product grouped by expert (bias and
// activation; the products' own gradients are expert_gemm.cu's):
//   dz[r] = dy[r] act'(z[r]),   db[e] = sum over the rows r of e of dy[r] act'(z[r])
// One pass over dy and z: a CTA holds 256 (or 64) channels of one expert, 8 to a lane, its
// warps take the expert's rows in turn and add up in fp32 registers.  The rows of an
// expert are dealt out over a cluster of up to 8 CTAs, whose sums are sent to the first
// one and added in order: an expert may have all rows, and one CTA for its 256 channels
// would be waited for alone.  (Sent by st.async, counted on a barrier of the first CTA: a
// cluster barrier's release waits for dz's stores, 598 instead of 504 us below.)
//
// Measured (one GB300): 262144 rows over 256 experts x 2048 channels, none / ReLU / GELU /
// tanh GELU / SiLU 315 / 450 / 477 / 463 / 450 us (copying the bytes takes 316 / 474):
// HBM bounds it, with two numbers to an instruction and four CTAs to an SM (three: 504 us
// with tanh GELU).  27 K rows over 52 experts drawn by a Zipf law x 1416, GELU: 49 us (copying
// them takes 34): the end, when only the CTAs of the expert with a fifth of the rows are left.
#include <cuda_bf16.h>

#include "activation.cuh"
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kSortExperts = 256;  // most experts that are put in order

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// C: channels of a CTA, 8 to a lane, so that a warp takes 256 / C rows at a time.
template <Act ACT, int C>
__global__ void __launch_bounds__(kThreads, 4) linear_backward_kernel(const LinearBackwardParams p) {
    constexpr int LANES = C / 8, ROWS = 32 / LANES;
    __shared__ __align__(8) float part[kWarps * ROWS][C];
    __shared__ float others[kMaxCtas][C];
    __shared__ uint64_t sent;
    const int ctas = p.ctas, rank = blockIdx.x % ctas;
    const uint32_t bar = umma::saddr(&sent);
    if (ctas > 1) {
        if (rank == 0 && threadIdx.x == 0) {
            umma::bar_init(bar, 1);
            umma::bar_init_fence();
        }
        __syncwarp();
        umma::cluster_arrive();  // the first CTA can be sent to; waited for below
    }
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = (p.n + C - 1) / C, clusters = gridDim.x / ctas;
    // Uneven experts: those with the most rows first, because one that comes last is waited for alone (27 K rows over
    // 52 experts by a Zipf law x 1416: 78 us in their own order).
    __shared__ int counts[kSortExperts], most;
    __shared__ uint8_t order[kSortExperts];
    bool sorted = false;
    if (ctas == kMaxCtas && p.E <= kSortExperts) {
        const int own = threadIdx.x < p.E ? p.count[threadIdx.x] : 0;
        if (threadIdx.x == 0) most = 0;
        if (threadIdx.x < p.E) counts[threadIdx.x] = own;
        __syncthreads();
        const int top = __reduce_max_sync(0xFFFFFFFFu, own);
        if (lane == 0) atomicMax(&most, top);
        __syncthreads();
        sorted = most > 3 * (p.live / p.E);
        if (sorted) {
            if (threadIdx.x < p.E) {
                int at = 0;
                for (int e = 0; e < p.E; ++e) at += counts[e] > own || (counts[e] == own && e < (int)threadIdx.x) ? 1 : 0;
                order[at] = (uint8_t)threadIdx.x;
            }
            __syncthreads();
        }
    }
    uint32_t turn = 0;
    for (int it = blockIdx.x / ctas; it < p.E * tiles; it += clusters, ++turn) {
        const int place = it / tiles, e = sorted ? order[place] : place, c0 = (it - place * tiles) * C, c = c0 + lane % LANES * 8;
        const int64_t base = p.base[e];
        const int count = p.count[e];
        const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(p.dy) + base * p.n + c;
        const __nv_bfloat16 *z = static_cast<const __nv_bfloat16 *>(p.z) + base * p.n + c;
        __nv_bfloat16 *dz = p.dz != nullptr ? static_cast<__nv_bfloat16 *>(p.dz) + base * p.n + c : nullptr;
        uint64_t sum[4] = {};  // pairs of fp32
        if (c < p.n) {
            constexpr int U = 4;
            const int step = kWarps * ROWS * ctas;
            for (int r0 = (rank * kWarps + warp) * ROWS + lane / LANES; r0 < count; r0 += step * U) {
                uint4 vd[U], vz[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = (int64_t)(r0 + u * step) * p.n;
                    if (r0 + u * step >= count) continue;
                    vd[u] = *reinterpret_cast<const uint4 *>(dy + at);
                    if (ACT != Act::kNone) vz[u] = *reinterpret_cast<const uint4 *>(z + at);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (r0 + u * step >= count) continue;
                    const uint32_t d4[4] = {vd[u].x, vd[u].y, vd[u].z, vd[u].w};
                    uint32_t z4[4] = {}, o4[4];
                    if (ACT != Act::kNone) z4[0] = vz[u].x, z4[1] = vz[u].y, z4[2] = vz[u].z, z4[3] = vz[u].w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t d = mul2(two(bf16_lo(d4[j]), bf16_hi(d4[j])), slope2<ACT>(bf16_lo(z4[j]), bf16_hi(z4[j])));
                        sum[j] = umma::add2(sum[j], d);
                        o4[j] = pack_bf16(umma::lo2(d), umma::hi2(d));
                    }
                    if (dz != nullptr)
                        *reinterpret_cast<uint4 *>(dz + (int64_t)(r0 + u * step) * p.n) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                }
            }
        }
        if (p.db == nullptr) continue;
        if (turn > 0) __syncthreads();  // the sums before have been read
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint64_t *>(&part[warp * ROWS + lane / LANES][lane % LANES * 8 + 2 * j]) = sum[j];
        if (ctas > 1 && rank == 0 && threadIdx.x == 0) umma::bar_expect(bar, (ctas - 1) * C * 4);
        __syncthreads();
        if (ctas > 1) umma::cluster_wait();  // the first CTA has read what was sent before
        float s = 0.0f;
        if (threadIdx.x < C) {
#pragma unroll
            for (int w = 0; w < kWarps * ROWS; ++w) s += part[w][threadIdx.x];
            if (rank > 0) {
                umma::send_u32(umma::map_rank(umma::saddr(&others[rank][threadIdx.x]), 0), __float_as_uint(s), umma::map_rank(bar, 0));
            } else {
                if (ctas > 1 && !umma::bar_wait(bar, turn & 1, kExpertWaitCycles)) atomicOr(p.status, kStatusTimeout);
                for (int q = 1; q < ctas; ++q) s += others[q][threadIdx.x];
                const int ch = c0 + threadIdx.x;
                if (ch < p.n) {
                    float *to = p.db + (int64_t)e * p.n + ch;
                    *to = p.accumulate ? *to + s : s;
                }
            }
        }
        __syncwarp();
        if (ctas > 1) umma::cluster_arrive();
    }
    if (ctas > 1) umma::cluster_wait();
}

template <Act ACT, int C>
cudaError_t launch(LinearBackwardParams p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // CTAs of an expert's 256 channels, by the mean rows of an expert: one up to 16 rows (two for a warp).  More of
    // them than even experts need (64 x 384 rows x 2048, GELU: 61 us, with two CTAs 51), because the host does not
    // know the counts: drawn by a Zipf law eight take 70 us there and two 121 (256 x 128 rows: 92 and 190).
    const int64_t mean = p.live / p.E;
    const int ctas = mean > 128 ? kMaxCtas : mean > 48 ? 4 : mean > 16 ? 2 : 1;
    p.ctas = ctas;
    // every item its own cluster on all SMs (the hardware levels uneven experts out); fewer SMs: as many as they hold
    int64_t clusters = (int64_t)p.E * ((p.n + C - 1) / C);
    if (p.sms < p.all_sms && clusters > p.sms * 4 / ctas) clusters = p.sms * 4 / ctas > 1 ? p.sms * 4 / ctas : 1;
    cfg.gridDim = dim3((unsigned)(clusters * ctas), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, linear_backward_kernel<ACT, C>, p);
}

template <Act ACT>
cudaError_t launch(const LinearBackwardParams &p, cudaStream_t stream) {
    // 64 channels where CTAs of 256 would not be one for each SM (1 expert x 4096 rows x 1024, SiLU: 14 us instead
    // of 33); else whole lines of 512 bytes are faster (262144 rows over 256 experts x 2048: 451 us instead of 533)
    const bool narrow = (int64_t)p.E * ((p.n + 255) / 256) * kMaxCtas < p.all_sms;
    return narrow ? launch<ACT, 64>(p, stream) : launch<ACT, 256>(p, stream);
}

}  // namespace

cudaError_t launch_linear_backward(const LinearBackwardParams &p, cudaStream_t stream) {
    switch (p.act) {
        case Act::kRelu: return launch<Act::kRelu>(p, stream);
        case Act::kGelu: return launch<Act::kGelu>(p, stream);
        case Act::kGeluTanh: return launch<Act::kGeluTanh>(p, stream);
        case Act::kSilu: return launch<Act::kSilu>(p, stream);
        default: return launch<Act::kNone>(p, stream);
    }
}

}  // namespace ep

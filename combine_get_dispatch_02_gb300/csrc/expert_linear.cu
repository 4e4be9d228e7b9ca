// Backward pass of the epilogue of a product grouped by expert (bias and
// activation; the products' own gradients are expert_gemm.cu's):
//   dz[r] = dy[r] act'(z[r]),   db[e] = sum over the rows r of e of dy[r] act'(z[r])
// One pass over dy and z: a CTA holds 256 channels of one expert, 8 to a lane, its
// warps take the expert's rows in turn and add up in fp32 registers.
#include <cuda_bf16.h>

#include "activation.cuh"
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChannels = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <Act ACT>
__global__ void __launch_bounds__(kThreads) linear_backward_kernel(const LinearBackwardParams p) {
    __shared__ float part[kWarps][kChannels];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = (p.n + kChannels - 1) / kChannels;
    const int e = blockIdx.x / tiles, c = (blockIdx.x - e * tiles) * kChannels + lane * 8;
    const int64_t base = p.base[e];
    const int count = p.count[e];
    const __nv_bfloat16 *dy = static_cast<const __nv_bfloat16 *>(p.dy) + base * p.n + c;
    const __nv_bfloat16 *z = static_cast<const __nv_bfloat16 *>(p.z) + base * p.n + c;
    __nv_bfloat16 *dz = p.dz != nullptr ? static_cast<__nv_bfloat16 *>(p.dz) + base * p.n + c : nullptr;
    float sum[8] = {};
    if (c < p.n) {
        constexpr int U = 4;
        for (int r0 = warp; r0 < count; r0 += kWarps * U) {
            uint4 vd[U], vz[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = (int64_t)(r0 + u * kWarps) * p.n;
                if (r0 + u * kWarps >= count) continue;
                vd[u] = *reinterpret_cast<const uint4 *>(dy + at);
                if (ACT != Act::kNone) vz[u] = *reinterpret_cast<const uint4 *>(z + at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * kWarps >= count) continue;
                const uint32_t d4[4] = {vd[u].x, vd[u].y, vd[u].z, vd[u].w};
                uint32_t z4[4] = {}, o4[4];
                if (ACT != Act::kNone) z4[0] = vz[u].x, z4[1] = vz[u].y, z4[2] = vz[u].z, z4[3] = vz[u].w;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = bf16_lo(d4[j]) * slope<ACT>(bf16_lo(z4[j])), b = bf16_hi(d4[j]) * slope<ACT>(bf16_hi(z4[j]));
                    sum[2 * j] += a;
                    sum[2 * j + 1] += b;
                    o4[j] = pack_bf16(a, b);
                }
                if (dz != nullptr)
                    *reinterpret_cast<uint4 *>(dz + (int64_t)(r0 + u * kWarps) * p.n) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
            }
        }
    }
    if (p.db == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = sum[j];
    __syncthreads();
    const int ch = (blockIdx.x - e * tiles) * kChannels + threadIdx.x;
    if (ch < p.n) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
        float *to = p.db + (int64_t)e * p.n + ch;
        *to = p.accumulate ? *to + s : s;
    }
}

template <Act ACT>
cudaError_t launch(const LinearBackwardParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.E * ((p.n + kChannels - 1) / kChannels)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_backward_kernel<ACT>, p);
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

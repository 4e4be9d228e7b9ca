// The gated activation between the two expert products of a bf16 training
// step, its gradient, and the cast of expert weights to e4m3 blocks.
//   SwiGLU:    h = g s u, s = 1 / (1 + exp(-g)), gu = [g | u] in one row
//   gradient:  du = dh g s,  dg = dh u s (1 + g (1 - s))
//   cast:      per 128 x 128 block of W: a = max(amax |w|, 1e-4),
//              scale = a / 448, q = e4m3(w * (448 / a)), the dispatch's FP8
//              rule on blocks instead of rows
// Each is one pass over its data in fp32 with one rounding at the end.  HBM
// bounds the gradient: with h, of 14 K rows x 1416 channels, 43 us, 5.7 TB/s (two
// items in flight per warp: 48 us with one).  SwiGLU of 262144 rows x 1024 channels
// takes 273 us, 5.9 TB/s, with its instructions near the limit too: with the fast
// exponential, 1.2 |g| ulp off, 262 us, with two items in flight 282.  The cast of
// 256 x 4096 x 7168 weights, made once, takes 5.15 ms, 4.4 TB/s.
//
// Rows: the work item is (entry of the layout, chunk of channels) for one
// warp, as in the identity expert: entries without a row cost one slot load
// and no row outside the experts' ranges is touched, whatever the layout.
// 8 channels per lane and load are whole 16-byte accesses of 512 contiguous
// bytes per warp.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 256;  // channels of h per warp item

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// g s with s = 1 / (1 + exp(-g)), and s and its complement 1 - s, from
// e = exp(-|g|), which does not overflow: one of s and 1 - s is 1 / (1 + e), the
// other e / (1 + e), a few ulp each (the fast division is good to 2 where the
// denominator lies in [1, 2]) with no cancellation.  g s and g (1 - s) are NaN at
// the infinity where s or 1 - s is 0, as in the formula.
struct Gate {
    float gs, s, c;
};
__device__ __forceinline__ Gate gate(float g) {
    const float e = expf(-fabsf(g)), big = __fdividef(1.0f, 1.0f + e);
    Gate r;
    r.gs = (g < 0.0f ? g * e : g) * big;
    r.s = g < 0.0f ? e * big : big;
    r.c = g < 0.0f ? big : e * big;
    return r;
}

template <bool BWD>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams p) {
    pdl_wait();  // gu (and the slots) come from the kernels queued just before
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t nwarp = ((int64_t)gridDim.x * kThreads) >> 5;
    const int I = p.inner;
    const int nch = (I + kChunk - 1) / kChunk;
    const int64_t items = p.n * nch;
    const __nv_bfloat16 *gu = static_cast<const __nv_bfloat16 *>(p.gu);
    const __nv_bfloat16 *dh = static_cast<const __nv_bfloat16 *>(p.dh);
    __nv_bfloat16 *h = static_cast<__nv_bfloat16 *>(p.h);
    __nv_bfloat16 *dgu = static_cast<__nv_bfloat16 *>(p.dgu);
    constexpr int U = BWD ? 2 : 1;  // items at a time: all their loads before the first is computed
    for (int64_t it0 = warp; it0 < items; it0 += U * nwarp) {
        int64_t row[U];
        int ch[U];
        uint4 vg[U], vu[U], vd[U];
#pragma unroll
        for (int t = 0; t < U; ++t) {
            const int64_t it = it0 + t * nwarp;
            const int64_t i = it / nch;
            row[t] = it < items ? p.slot[i] : -1;
            ch[t] = (int)(it - i * nch) * kChunk + lane * 8;
            if (ch[t] >= I) row[t] = -1;
        }
#pragma unroll
        for (int t = 0; t < U; ++t) {
            if (row[t] < 0) continue;
            vg[t] = ld_nc_na_v4(gu + row[t] * 2 * I + ch[t]);
            vu[t] = ld_nc_na_v4(gu + row[t] * 2 * I + I + ch[t]);
            if constexpr (BWD) vd[t] = ld_nc_na_v4(dh + row[t] * I + ch[t]);
        }
#pragma unroll
        for (int t = 0; t < U; ++t) {
            if (row[t] < 0) continue;
            const int c = ch[t];
            const uint32_t g4[4] = {vg[t].x, vg[t].y, vg[t].z, vg[t].w}, u4[4] = {vu[t].x, vu[t].y, vu[t].z, vu[t].w};
            uint32_t d4[4] = {};
            if constexpr (BWD) d4[0] = vd[t].x, d4[1] = vd[t].y, d4[2] = vd[t].z, d4[3] = vd[t].w;
            uint32_t oh[4], og[4], ou[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ga = bf16_lo(g4[j]), gb = bf16_hi(g4[j]), ua = bf16_lo(u4[j]), ub = bf16_hi(u4[j]);
                const Gate a = gate(ga), b = gate(gb);
                oh[j] = pack_bf16(a.gs * ua, b.gs * ub);
                if constexpr (BWD) {
                    const float da = bf16_lo(d4[j]), db = bf16_hi(d4[j]);
                    ou[j] = pack_bf16(da * a.gs, db * b.gs);
                    // the slope (1.1 at most) first: dh u alone can overflow
                    og[j] = pack_bf16(da * (a.s * fmaf(ga, a.c, 1.0f)) * ua, db * (b.s * fmaf(gb, b.c, 1.0f)) * ub);
                }
            }
            if (!BWD || h != nullptr)
                *reinterpret_cast<uint4 *>(h + row[t] * I + c) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
            if constexpr (BWD) {
                *reinterpret_cast<uint4 *>(dgu + row[t] * 2 * I + c) = make_uint4(og[0], og[1], og[2], og[3]);
                *reinterpret_cast<uint4 *>(dgu + row[t] * 2 * I + I + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            }
        }
    }
}

// One CTA per 128 x 128 block: 256 threads, a thread holds 4 channels of 16
// rows in registers between the maximum and the cast.
__global__ void __launch_bounds__(kThreads) cast_weights_kernel(const CastWeightsParams p) {
    __shared__ float part[kThreads / 32];
    pdl_wait();
    const int nb = (p.n + 127) / 128, kb = p.k / 128;
    const int64_t blocks = (int64_t)p.E * nb * kb;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(p.w);
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t e = b / ((int64_t)nb * kb);
        const int rest = (int)(b - e * nb * kb);
        const int r0 = rest / kb * 128, c0 = rest % kb * 128 + lane * 4;
        uint2 v[16];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + wid + 8 * i;
            v[i] = make_uint2(0, 0);
            if (r < p.n) v[i] = ld_nc_na_v2(w + (e * p.n + r) * p.k + c0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[i].x)), fabsf(bf16_hi(v[i].x))));
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[i].y)), fabsf(bf16_hi(v[i].y))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        __syncthreads();  // part is free (the block before has been read)
        if (lane == 0) part[wid] = amax;
        __syncthreads();
        amax = part[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) amax = fmaxf(amax, part[i]);
        const float a = fmaxf(amax, 1e-4f), inv = __fdiv_rn(448.0f, a);
        if (tid == 0) p.scales[b] = __fdiv_rn(a, 448.0f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + wid + 8 * i;
            if (r >= p.n) continue;
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(bf16_lo(v[i].x), inv), __fmul_rn(bf16_hi(v[i].x), inv)), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(bf16_lo(v[i].y), inv), __fmul_rn(bf16_hi(v[i].y), inv)), __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint32_t *>(p.q + (e * p.n + r) * p.k + c0) = lo | hi << 16;
        }
    }
}

template <typename K, typename P>
cudaError_t launch_pdl(K kernel, const P &p, int64_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename K>
int occupancy(K kernel) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess) {
        cudaGetLastError();
        return 1;
    }
    return n > 0 ? n : 1;
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, bool backward, int sms, cudaStream_t stream) {
    const int64_t warps = p.n * ((p.inner + kChunk - 1) / kChunk);
    int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    static const int resident[2] = {occupancy(swiglu_kernel<false>), occupancy(swiglu_kernel<true>)};
    if (blocks > (int64_t)sms * resident[backward]) blocks = (int64_t)sms * resident[backward];
    return backward ? launch_pdl(swiglu_kernel<true>, p, blocks, stream)
                    : launch_pdl(swiglu_kernel<false>, p, blocks, stream);
}

cudaError_t launch_cast_weights(const CastWeightsParams &p, int sms, cudaStream_t stream) {
    int64_t blocks = (int64_t)p.E * ((p.n + 127) / 128) * (p.k / 128);
    if (blocks > (int64_t)sms * 8) blocks = (int64_t)sms * 8;
    return launch_pdl(cast_weights_kernel, p, blocks, stream);
}

}  // namespace ep

// Expert products between dispatch and combine: matrix products grouped by
// expert, whose row groups are the receive rows base[e] .. base[e] + count[e]
// of a layout (counts and bases are read on the device, never on the host).
//   y[r]  = W[e] x[r]                        (bf16, or W stored transposed)
//   y[r]  = sum_b xs[r,b] ws[e,.,b] (Wq[e] xq[r])_b   (e4m3, 128-channel blocks b)
//   h[r]  = cast(silu(g) * u), (g, u) = the two halves of the e4m3 product
//   dW[e] = sum_r dy[r] x[r]^T
// Plain form: one CTA per output tile of 32 x 128, fp32 accumulation on the
// CUDA cores.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kBM = 32, kBN = 128, kBK = 16, kT = 256;

__device__ __forceinline__ float e4m3_to_float(uint8_t q) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)q, __NV_E4M3)));
}
__device__ __forceinline__ float bf(const void *p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <ExpertOp OP>
__global__ void __launch_bounds__(kT) expert_gemm_plain(const ExpertGemmParams p) {
    constexpr bool DUAL = OP == ExpertOp::kGateFp8;
    constexpr int NB = DUAL ? 2 : 1;
    __shared__ float As[kBK][kBM + 1];
    __shared__ float Bs[NB][kBK][kBN + 1];
    const int tid = threadIdx.x, ty = tid >> 5, tx = tid & 31;
    const bool wg = OP == ExpertOp::kWgrad;
    const int e = blockIdx.z;
    const int64_t base = p.base[e];
    const int cnt = p.count[e];
    const int mdim = wg ? p.n : cnt;              // rows of this tile's output
    const int ndim = wg ? p.k : (DUAL ? p.n / 2 : p.n);
    const int kdim = wg ? cnt : p.k;
    const int n0 = blockIdx.x * kBN;
    const int kb = (p.k + 127) / 128;
    auto load_a = [&](int m, int kk) -> float {   // rows (wgrad: channels of dy)
        if (m >= mdim || kk >= kdim) return 0.0f;
        if constexpr (OP == ExpertOp::kWgrad) return bf(p.dy, (base + kk) * p.n + m);
        const int64_t r = base + m;
        if constexpr (OP == ExpertOp::kFp8 || OP == ExpertOp::kGateFp8)
            return e4m3_to_float(static_cast<const uint8_t *>(p.x)[r * p.k + kk]) * p.xs[r * kb + kk / 128];
        return bf(p.x, r * p.k + kk);
    };
    auto load_b = [&](int half, int c, int kk) -> float {
        if (c >= ndim || kk >= kdim) return 0.0f;
        if constexpr (OP == ExpertOp::kWgrad) return bf(p.x, (base + kk) * p.k + c);
        const int64_t w0 = (int64_t)e * p.n * p.k;
        const int ch = c + half * ndim;
        if constexpr (OP == ExpertOp::kFp8 || OP == ExpertOp::kGateFp8)
            return e4m3_to_float(static_cast<const uint8_t *>(p.w)[w0 + (int64_t)ch * p.k + kk]) *
                   p.ws[((int64_t)e * ((p.n + 127) / 128) + ch / 128) * kb + kk / 128];
        if constexpr (OP == ExpertOp::kBf16T) return bf(p.w, w0 + (int64_t)kk * p.n + ch);
        return bf(p.w, w0 + (int64_t)ch * p.k + kk);
    };
    for (int m0 = blockIdx.y * kBM; m0 < mdim; m0 += gridDim.y * kBM) {
        // partial sums of 256 terms, then sums of partial sums: a long fp32 sum
        // loses fewer bits
        float acc[NB][4][4] = {}, part[NB][4][4] = {};
        for (int k0 = 0; k0 < kdim; k0 += kBK) {
            for (int i = tid; i < kBM * kBK; i += kT) {
                const int m = wg ? i % kBM : i / kBK, kk = wg ? i / kBM : i % kBK;
                As[kk][m] = load_a(m0 + m, k0 + kk);
            }
            const bool nfast = wg || OP == ExpertOp::kBf16T;
            for (int h = 0; h < NB; ++h)
                for (int i = tid; i < kBN * kBK; i += kT) {
                    const int c = nfast ? i % kBN : i / kBK, kk = nfast ? i / kBN : i % kBK;
                    Bs[h][kk][c] = load_b(h, n0 + c, k0 + kk);
                }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kBK; ++kk)
#pragma unroll
                for (int h = 0; h < NB; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[h][i][j] = fmaf(As[kk][ty * 4 + i], Bs[h][kk][tx + 32 * j], part[h][i][j]);
            __syncthreads();
            if ((k0 + kBK) % 256 == 0 || k0 + kBK >= kdim)
#pragma unroll
                for (int h = 0; h < NB; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[h][i][j] += part[h][i][j];
                            part[h][i][j] = 0.0f;
                        }
        }
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty * 4 + i;
            if (m >= mdim) continue;
            if constexpr (DUAL) {
                float h[4], amax = 0.0f;
                for (int j = 0; j < 4; ++j) {
                    const float g = acc[0][i][j];
                    h[j] = g / (1.0f + expf(-g)) * acc[NB - 1][i][j];
                    amax = fmaxf(amax, fabsf(h[j]));
                }
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const float a = fmaxf(amax, 1e-4f), inv = __fdiv_rn(448.0f, a);
                const int64_t r = base + m;
                for (int j = 0; j < 4; ++j)
                    static_cast<uint8_t *>(p.y)[r * ndim + n0 + tx + 32 * j] =
                        __nv_cvt_float_to_fp8(__fmul_rn(h[j], inv), __NV_SATFINITE, __NV_E4M3);
                if (tx == 0) p.ys[r * (ndim / 128) + n0 / 128] = __fdiv_rn(a, 448.0f);
            } else {
                for (int j = 0; j < 4; ++j) {
                    const int c = n0 + tx + 32 * j;
                    if (c >= ndim) continue;
                    if constexpr (OP == ExpertOp::kWgrad) {
                        const int64_t o = ((int64_t)e * p.n + m) * p.k + c;
                        if (p.out_fp32) {
                            float *d = static_cast<float *>(p.y) + o;
                            *d = p.accumulate ? *d + acc[0][i][j] : acc[0][i][j];
                        } else {
                            static_cast<__nv_bfloat16 *>(p.y)[o] = __float2bfloat16_rn(acc[0][i][j]);
                        }
                    } else {
                        static_cast<__nv_bfloat16 *>(p.y)[(base + m) * p.n + c] = __float2bfloat16_rn(acc[0][i][j]);
                    }
                }
            }
        }
    }
}

template <ExpertOp OP>
cudaError_t launch(const ExpertGemmParams &p, cudaStream_t stream) {
    const int nd = OP == ExpertOp::kWgrad ? p.k : (OP == ExpertOp::kGateFp8 ? p.n / 2 : p.n);
    const int64_t md = OP == ExpertOp::kWgrad ? p.n : p.max_count;
    int64_t my = (md + kBM - 1) / kBM;
    if (my > 64) my = 64;
    if (my < 1) my = 1;
    expert_gemm_plain<OP><<<dim3((nd + kBN - 1) / kBN, (unsigned)my, p.E), kT, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_gemm(ExpertOp op, const ExpertGemmParams &p, cudaStream_t stream) {
    switch (op) {
        case ExpertOp::kBf16: return launch<ExpertOp::kBf16>(p, stream);
        case ExpertOp::kBf16T: return launch<ExpertOp::kBf16T>(p, stream);
        case ExpertOp::kFp8: return launch<ExpertOp::kFp8>(p, stream);
        case ExpertOp::kGateFp8: return launch<ExpertOp::kGateFp8>(p, stream);
        default: return launch<ExpertOp::kWgrad>(p, stream);
    }
}

}  // namespace ep

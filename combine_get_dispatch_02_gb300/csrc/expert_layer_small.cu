// The small form of the whole layer for a few tokens (expert_layer.cu has the formulas
// and the large form): two kernels, gate and down, without a grid barrier.  Where the
// weights are a few tens of MB the large form's three meetings of all SMs are most of
// its time (one token, top-4 of 32, 1024 x 512, bf16: 12 us here, 20 there).
//
// The unit of work is 32 weight rows of one expert (gate: 16 channels of h, their gate
// and up rows), over all tokens of that expert, 8 at a time, on the m16n8k16 product with
// the weights on the M side; a CTA of 8 warps, which share the channels, takes a
// contiguous share of all units.  Weights and tokens come straight into registers.  The
// second kernel starts behind the first (programmatic dependent launch) and sorts the
// entries meanwhile; whoever completes a tile of its output rows adds the entries up.
#include <cuda_bf16.h>

#include "activation.cuh"
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 codes times 2^-14 as a bf16 pair, exactly and with their NaN, through fp16 and fp32 (1.8 times as fast as
// moving the bits into place).  Times 2^-14: the sums before their scale, of codes up to 448, then overflow no
// sooner than the tokens.
constexpr float kCode = 0x1p-14f;
__device__ __forceinline__ uint32_t e4m3x2(uint16_t w) {
    uint32_t h, r;
    float a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    asm("{\n .reg .f16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}" : "=f"(a), "=f"(b) : "r"(h));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b * kCode), "f"(a * kCode));
    return r;
}

// 16 bytes of a token or of h.  (Not a read-only load: this kernel may have started before h was written.)
__device__ __forceinline__ uint4 load_token(const __nv_bfloat16 *src) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
    return v;
}

// The entries by expert, in shared memory: the D experts with entries, ascending,
// each with its list.  The order inside a list differs between CTAs; an entry's
// result does not depend on its place.
struct Route {
    int *first;        // [E + 1] count, then first place in list, of each expert
    uint16_t *live;    // [min(E, M)] experts with entries
    uint16_t *list;    // [M] entries by expert
    uint16_t *place;   // [M] place in its expert's list, 0xFFFF: no expert
    int D;
};

size_t route_bytes(int E, int M) { return (size_t)(E + 2) * 4 + (size_t)(E < M ? E : M) * 2 + (size_t)M * 4 + 16; }

__device__ __forceinline__ Route route(const ExpertLayerParams &p, uint8_t *smem) {
    __shared__ int live_experts;
    Route r;
    const int M = p.N * p.K, tid = threadIdx.x;
    r.first = reinterpret_cast<int *>(smem);
    r.list = reinterpret_cast<uint16_t *>(r.first + p.E + 1);
    r.place = r.list + M;
    r.live = r.place + M;
    for (int e = tid; e <= p.E; e += kThreads) r.first[e] = 0;
    __syncthreads();
    for (int j = tid; j < M; j += kThreads) {
        const int64_t e = p.idx[j];
        const bool ok = e >= 0 && e < p.E;
        if (!ok && e != -1 && blockIdx.x == 0) atomicOr(p.status, kStatusBadExpert);
        r.place[j] = ok ? (uint16_t)atomicAdd(&r.first[e], 1) : 0xFFFFu;
    }
    __syncthreads();
    if (tid < 32) {
        // first places and the live experts, both by prefix sums over the experts
        const int per = (p.E + 31) / 32, e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
        int n = 0, d = 0;
        for (int e = e0; e < e1; ++e) {
            n += r.first[e];
            d += r.first[e] > 0 ? 1 : 0;
        }
        int ns = n, ds = d;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xFFFFFFFFu, ns, o), b = __shfl_up_sync(0xFFFFFFFFu, ds, o);
            if (tid >= o) ns += a, ds += b;
        }
        if (tid == 31) live_experts = ds, r.first[p.E] = ns;
        ns -= n;
        ds -= d;
        for (int e = e0; e < e1; ++e) {
            const int c = r.first[e];
            r.first[e] = ns;
            ns += c;
            if (c > 0) r.live[ds++] = (uint16_t)e;
        }
    }
    __syncthreads();
    for (int j = tid; j < M; j += kThreads)
        if (r.place[j] != 0xFFFFu) r.list[r.first[p.idx[j]] + r.place[j]] = (uint16_t)j;
    __syncthreads();
    r.D = live_experts;
    return r;
}

// Products of two tiles of 16 weight rows (row(i, g): tile i, row g of 0 .. 15, as a
// pointer) with up to 8 columns, over this warp's share of K channels.  PLANES: a
// column is the sum of this many bf16 vectors, `plane` elements apart.
template <bool FP8, int PLANES>
__device__ __forceinline__ void products(float (&acc)[2][4], const uint8_t *const (&wr)[2][2], const float *const (&ws)[2][2],
                                         const __nv_bfloat16 *col, int64_t plane, int K, int warp, int t) {
    if constexpr (!FP8) {
        constexpr int U = 4;
        const int steps = (K + 31) / 32;
        for (int s0 = warp; s0 < steps; s0 += kWarps * U) {
            uint4 a[U][2][2], b[U][PLANES];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = (s0 + u * kWarps) * 32 + t * 8;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 2; ++q) a[u][i][q] = c < K ? ld_nc_na_v4(wr[i][q] + 2 * (int64_t)c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < PLANES; ++q)
                    b[u][q] = c < K ? load_token(col + q * plane + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < PLANES; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma_bf16(acc[i], a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y, b[u][q].x, b[u][q].y);
                        mma_bf16(acc[i], a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w, b[u][q].z, b[u][q].w);
                    }
        }
    } else {
        const int blocks = K / 128;
        for (int s = warp; s < blocks; s += kWarps) {
            uint4 a[2][2][2], b[2][PLANES][2];
            float sc[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = s * 128 + u * 64 + t * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 2; ++q) a[u][i][q] = ld_nc_na_v4(wr[i][q] + c);
#pragma unroll
                for (int q = 0; q < PLANES; ++q)
#pragma unroll
                    for (int v = 0; v < 2; ++v) b[u][q][v] = load_token(col + q * plane + c + 8 * v);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) sc[i][q] = __ldg(ws[i][q] + s);
            float part[2][4] = {};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w0[4] = {a[u][i][0].x, a[u][i][0].y, a[u][i][0].z, a[u][i][0].w};
                    const uint32_t w1[4] = {a[u][i][1].x, a[u][i][1].y, a[u][i][1].z, a[u][i][1].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a0 = e4m3x2((uint16_t)w0[j]), a1 = e4m3x2((uint16_t)w1[j]);
                        const uint32_t a2 = e4m3x2((uint16_t)(w0[j] >> 16)), a3 = e4m3x2((uint16_t)(w1[j] >> 16));
#pragma unroll
                        for (int q = 0; q < PLANES; ++q) {
                            const uint4 &v = b[u][q][j >> 1];
                            mma_bf16(part[i], a0, a1, a2, a3, j & 1 ? v.z : v.x, j & 1 ? v.w : v.y);
                        }
                    }
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(part[i][c] * sc[i][c >> 1], 1.0f / kCode, acc[i][c]);
        }
    }
}

// The 8 warps' sums of element c of tile i, lane l of the fragments.
__device__ __forceinline__ float summed(const float (*red)[2][4][32], int i, int c, int l) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][i][c][l];
    return v;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 2) small_gate_kernel(const ExpertLayerParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[kWarps][2][4][32];
    pdl_wait();
    pdl_launch_dependents();
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < (p.H + 31) / 32; i += gridDim.x * kThreads) p.done[i] = 0;
    const Route r = route(p, smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int tiles = (p.I + 15) / 16;
    const int64_t total = (int64_t)r.D * tiles;
    const int es = FP8 ? 1 : 2, nb = (2 * p.I + 127) / 128, kb = p.H / 128;
    const int64_t it1 = total * (blockIdx.x + 1) / gridDim.x;
    for (int64_t it = total * blockIdx.x / gridDim.x; it < it1; ++it) {
        const int d = (int)(it / tiles), c0 = (int)(it - (int64_t)d * tiles) * 16, e = r.live[d];
        const int j0 = r.first[e], j1 = r.first[e + 1];
        // tile i: channels c0 + 8 i .. of h, their gate rows above, their up rows below
        const uint8_t *wr[2][2];
        const float *ws[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int row = q * p.I + min(c0 + 8 * i, p.I - 8) + g;
                wr[i][q] = static_cast<const uint8_t *>(p.w_gate_up) + ((int64_t)e * 2 * p.I + row) * p.H * es;
                ws[i][q] = FP8 ? p.s_gate_up + ((int64_t)e * nb + row / 128) * kb : nullptr;
            }
        for (int j = j0; j < j1; j += 8) {
            float acc[2][4] = {};
            const int token = r.list[min(j + g, j1 - 1)] / p.K;
            products<FP8, 1>(acc, wr, ws, static_cast<const __nv_bfloat16 *>(p.x) + (int64_t)token * p.H, 0, p.H, warp, t);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) red[warp][i][c][lane] = acc[i][c];
            __syncthreads();
            if (tid < 128) {
                const int i = tid >> 6, c = tid >> 5 & 1, l = tid & 31;
                const int at = j + 2 * (l & 3) + c, ch = c0 + 8 * i + (l >> 2);
                if (at < j1 && ch < p.I) {
                    float gate = summed(red, i, c, l), up = summed(red, i, c + 2, l);
                    if (p.b_gate_up != nullptr) {
                        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(p.b_gate_up) + (int64_t)e * 2 * p.I;
                        gate += __bfloat162float(b[ch]);
                        up += __bfloat162float(b[p.I + ch]);
                    }
                    // kept as the sum of two bf16 numbers, 2^-17 of the value off at most: rounded to one, h alone
                    // would put as much error into the result as its own rounding
                    const float h = silu(gate) * up;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.h) + (int64_t)r.list[at] * 2 * p.I + ch;
                    const float top = __bfloat162float(hi);
                    to[0] = hi;
                    to[p.I] = __float2bfloat16_rn(isfinite(top) ? h - top : 0.0f);
                }
            }
        }
    }
}

// out[t, rows] from every entry's y, k ascending.
__device__ __forceinline__ void combine_rows(const ExpertLayerParams &p, const Route &r, int row0) {
    const int row = row0 + (threadIdx.x & 15) * 2;
    if (row >= p.H) return;
    for (int t = threadIdx.x >> 4; t < p.N; t += kThreads / 16) {
        float a = 0.0f, b = 0.0f;
        for (int k = 0; k < p.K; ++k) {
            const int j = t * p.K + k;
            if (r.place[j] == 0xFFFFu) continue;
            const float w = p.wts != nullptr ? __ldg(p.wts + j) : 1.0f;
            const float2 y = __ldcg(reinterpret_cast<const float2 *>(p.sums + (int64_t)j * p.H + row));
            a = fmaf(w, y.x, a);
            b = fmaf(w, y.y, b);
        }
        const int64_t at = (int64_t)t * p.H + row;
        if (p.residual != nullptr) {
            // (not a read-only load: `out` may be the residual)
            const uint32_t v = *reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.residual) + at);
            a += bf16_lo(v);
            b += bf16_hi(v);
        }
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + at) = __floats2bfloat162_rn(a, b);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 2) small_down_kernel(const ExpertLayerParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[kWarps][2][4][32];
    __shared__ int last;
    const Route r = route(p, smem);
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int tiles = (p.H + 31) / 32;
    if (r.D == 0) {
        for (int i = blockIdx.x; i < tiles; i += gridDim.x) combine_rows(p, r, i * 32);
        return;
    }
    const int64_t total = (int64_t)r.D * tiles;
    const int es = FP8 ? 1 : 2, nb = (p.H + 127) / 128, kb = p.I / 128;
    const int64_t it0 = total * blockIdx.x / gridDim.x, it1 = total * (blockIdx.x + 1) / gridDim.x;
    int mine = 0;  // units of this tile done here
    for (int64_t it = it0; it < it1; ++it) {
        const int tile = (int)(it / r.D), d = (int)(it - (int64_t)tile * r.D), e = r.live[d];
        const int j0 = r.first[e], j1 = r.first[e + 1], row0 = tile * 32;
        const uint8_t *wr[2][2];
        const float *ws[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int row = min(row0 + 16 * i + 8 * q, p.H - 8) + g;
                wr[i][q] = static_cast<const uint8_t *>(p.w_down) + ((int64_t)e * p.H + row) * p.I * es;
                ws[i][q] = FP8 ? p.s_down + ((int64_t)e * nb + row / 128) * kb : nullptr;
            }
        for (int j = j0; j < j1; j += 8) {
            float acc[2][4] = {};
            const int entry = r.list[min(j + g, j1 - 1)];
            products<FP8, 2>(acc, wr, ws, static_cast<const __nv_bfloat16 *>(p.h) + (int64_t)entry * 2 * p.I, p.I, p.I, warp, t);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) red[warp][i][c][lane] = acc[i][c];
            __syncthreads();
            const int i = tid >> 7, c = tid >> 5 & 3, l = tid & 31;
            const int at = j + 2 * (l & 3) + (c & 1), row = row0 + 16 * i + 8 * (c >> 1) + (l >> 2);
            if (at < j1 && row < p.H) {
                float y = summed(red, i, c, l);
                if (p.b_down != nullptr) y += __bfloat162float(static_cast<const __nv_bfloat16 *>(p.b_down)[(int64_t)e * p.H + row]);
                __stcg(p.sums + (int64_t)r.list[at] * p.H + row, y);
            }
        }
        ++mine;
        if (d == r.D - 1 || it == it1 - 1) {
            // whoever completes the tile's experts adds them up
            bool whole = mine == r.D;
            if (!whole) {
                __threadfence();
                __syncthreads();
                if (tid == 0) last = atomicAdd(p.done + tile, (uint32_t)mine) + mine == (uint32_t)r.D;
                __syncthreads();
                whole = last;
                __threadfence();
            } else {
                __syncthreads();
            }
            if (whole) combine_rows(p, r, row0);
            mine = 0;
        }
    }
}

template <typename K>
cudaError_t launch(K kernel, const ExpertLayerParams &p, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.sms, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

size_t expert_layer_small_workspace(const ExpertLayerParams &p) {
    const size_t M = (size_t)p.N * p.K;
    return M * p.H * 4 + M * p.I * 4 + (size_t)((p.H + 31) / 32) * 4;
}

cudaError_t launch_expert_layer_small(ExpertLayerParams p, void *workspace, cudaStream_t stream) {
    const size_t M = (size_t)p.N * p.K, smem = route_bytes(p.E, (int)M);
    p.sums = static_cast<float *>(workspace);
    p.h = p.sums + M * p.H;
    p.done = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.h) + M * p.I * 4);
    const bool fp8 = p.s_gate_up != nullptr;
    const cudaError_t e = fp8 ? launch(small_gate_kernel<true>, p, smem, stream) : launch(small_gate_kernel<false>, p, smem, stream);
    if (e != cudaSuccess) return e;
    return fp8 ? launch(small_down_kernel<true>, p, smem, stream) : launch(small_down_kernel<false>, p, smem, stream);
}

}  // namespace ep

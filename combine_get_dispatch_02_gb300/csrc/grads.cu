// The norm of many gradients together, and their clipping:
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / norm)
// Two kernels that only stream: the first leaves one partial sum per CTA, which
// every CTA of the second adds up in the same order, so nothing is kept between
// calls and a result repeats bit for bit.  The tensors are cut into pieces of 16 KB
// that start on 16-byte addresses, numbered through; their table travels in the
// kernel's parameters.
//
// Sums: the squares of a thread's 64 bytes in fp32, everything above in fp64, root and quotient too.  Where the
// largest of them could overflow or vanish when squared they are taken again in
// fp64 (which for all of them would bound the kernel: one fp64 operation for every
// 4 bytes is more than the device has).
//
// Measured (one GB300): 671M elements in fp32 and bf16, 2.7 GB: norm 389 us (6.90 TB/s, HBM), clipping into
// other tensors 786 us (6.83 TB/s, HBM), in place 858 us; 12 tensors of up to 1024 bf16 both together 13 us (two
// launches and fp64's latencies; the caller's host takes longer); 300 tensors of 0.48 GB, nothing to clip, 85 us.
#include <cuda_bf16.h>

#include "ep.h"
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                            // 16-byte vectors of a thread and piece
constexpr int kPiece = kThreads * kVecs * 16;       // bytes

template <int CAP>
struct Table {
    const uint8_t *src[CAP];
    uint8_t *dst[CAP];
    int64_t n[CAP];            // elements; ~n for fp32
    int32_t first[CAP + 1];    // first piece of each tensor
    int32_t count;
    int32_t in_place;          // every tensor is its own out
};

struct Piece {
    const uint8_t *src;
    uint8_t *dst;
    int64_t at, n;             // first element (may be negative: before the tensor) and elements of the tensor
    bool f32;
};

// Piece c, which lies in tensor t or one near it (kept from piece to piece).
template <int CAP>
__device__ __forceinline__ Piece piece_at(const Table<CAP> &tab, int c, int &t) {
    while (tab.first[t] > c) --t;
    while (tab.first[t + 1] <= c) ++t;
    Piece p;
    p.src = tab.src[t];
    p.dst = tab.dst[t];
    const int64_t n = tab.n[t];
    p.f32 = n < 0;
    p.n = n < 0 ? ~n : n;
    const int es = p.f32 ? 4 : 2;
    p.at = (int64_t)(c - tab.first[t]) * (kPiece / es) - ((uintptr_t)p.src & 15) / es;
    return p;
}

// The tensor of piece c.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP> &tab, int c) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Elements i .. i + ve - 1 of the tensor, zeros outside it.  (Not a read-only load:
// clipping in place writes them.)
__device__ __forceinline__ uint4 load_vec(const Piece &p, int64_t i, int ve) {
    const int es = p.f32 ? 4 : 2;
    if (i >= 0 && i + ve <= p.n) {
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p.src + i * es));
        return v;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= ve || i + j < 0 || i + j >= p.n) continue;
        if (p.f32)
            w[j & 3] = reinterpret_cast<const uint32_t *>(p.src)[i + j];
        else
            w[j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p.src)[i + j] << (16 * (j & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Over a warp, in every lane.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<CAP> tab, double *partials, int add) {
    pdl_wait();
    const int total = tab.first[tab.count];
    const int c0 = (int)((int64_t)total * blockIdx.x / gridDim.x), c1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    int t = c0 < c1 ? tensor_of(tab, c0) : 0;
    for (int c = c0; c < c1; ++c) {
        const Piece p = piece_at(tab, c, t);
        const int ve = p.f32 ? 4 : 8;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = load_vec(p, p.at + (int64_t)(i * kThreads + threadIdx.x) * ve, ve);
        float s = 0.0f, top = 0.0f;
        auto all = [&](auto &&f) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (p.f32) {
                        f(__uint_as_float(w[j]));
                    } else {
                        f(bf16_lo(w[j]));
                        f(bf16_hi(w[j]));
                    }
                }
            }
        };
        all([&](float g) {
            s = fmaf(g, g, s);
            top = fmaxf(top, fabsf(g));
        });
        if (top < 0x1p60f && (top > 0x1p-50f || top == 0.0f)) {
            sum += (double)s;
        } else {
            double wide = 0.0;
            all([&](float g) { wide = fma((double)g, (double)g, wide); });
            sum += wide;
        }
    }
    // by one warp: an fp64 instruction of a warp takes 16 cycles, and with all of them at it 12 small tensors
    // took 8 us here and 12 below
    __shared__ double part[kThreads];
    part[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        sum = part[threadIdx.x];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) sum += part[threadIdx.x + 32 * i];
        sum = warp_sum(sum);
        if (threadIdx.x == 0) partials[blockIdx.x] = add ? partials[blockIdx.x] + sum : sum;
    }
    if (!add && blockIdx.x == 0)
        for (int i = gridDim.x + threadIdx.x; i < kGradPartials; i += kThreads) partials[i] = 0.0;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_clip_kernel(const __grid_constant__ Table<CAP> tab, const double *partials,
                                                             float max_norm, float *norm_out) {
    pdl_wait();
    __shared__ double part[kGradPartials];
    __shared__ float factor;
#pragma unroll
    for (int i = 0; i < kGradPartials / kThreads; ++i) part[threadIdx.x + i * kThreads] = partials[threadIdx.x + i * kThreads];
    __syncthreads();
    if (threadIdx.x < 32) {
        double sum = part[threadIdx.x];
        for (int i = 1; i < kGradPartials / 32; ++i) sum += part[threadIdx.x + 32 * i];
        sum = warp_sum(sum);
        if (threadIdx.x == 0) {
            // the root and the quotient in fp64, each rounded once; a norm past fp32's range or an undefined one
            // scales nothing
            const double wide = sqrt(sum);
            const float norm = (float)wide;
            if (norm_out != nullptr && blockIdx.x == 0) *norm_out = norm;
            factor = isfinite(norm) && wide > (double)max_norm ? (float)((double)max_norm / wide) : 1.0f;
        }
    }
    __syncthreads();
    const float f = factor;
    if (f == 1.0f && tab.in_place) return;
    const int total = tab.first[tab.count];
    const int c0 = (int)((int64_t)total * blockIdx.x / gridDim.x), c1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    int t = c0 < c1 ? tensor_of(tab, c1 - 1) : 0;
    // backwards: what the norm read last is still in L2
    for (int c = c1 - 1; c >= c0; --c) {
        const Piece p = piece_at(tab, c, t);
        if (f == 1.0f && p.src == p.dst) continue;
        const int ve = p.f32 ? 4 : 8, es = p.f32 ? 4 : 2;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = load_vec(p, p.at + (int64_t)(i * kThreads + threadIdx.x) * ve, ve);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p.f32) {
                    w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
                    w[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            const int64_t at = p.at + (int64_t)(i * kThreads + threadIdx.x) * ve;
            uint8_t *to = p.dst + at * es;
            if (at >= 0 && at + ve <= p.n && ((uintptr_t)to & 15) == 0) {
                *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= ve || at + j < 0 || at + j >= p.n) continue;
                if (p.f32)
                    reinterpret_cast<uint32_t *>(p.dst)[at + j] = w[j & 3];
                else
                    reinterpret_cast<uint16_t *>(p.dst)[at + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

template <int CAP>
int fill(Table<CAP> &tab, const ep_grad *g, int count) {
    int pieces = 0;
    tab.count = count;
    tab.in_place = 1;
    for (int i = 0; i < count; ++i) {
        const int es = g[i].fp32 ? 4 : 2;
        const int64_t lead = ((uintptr_t)g[i].data & 15) / es;
        tab.src[i] = static_cast<const uint8_t *>(g[i].data);
        tab.dst[i] = static_cast<uint8_t *>(g[i].out);
        if (g[i].out != g[i].data) tab.in_place = 0;
        tab.n[i] = g[i].fp32 ? ~g[i].numel : g[i].numel;
        tab.first[i] = pieces;
        if (g[i].numel > 0) pieces += (int)((g[i].numel + lead + kPiece / es - 1) / (kPiece / es));
    }
    tab.first[count] = pieces;
    return pieces;
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int grid, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int grid_of(int pieces, int sms) {
    int grid = sms * 6;
    if (grid > kGradPartials) grid = kGradPartials;
    if (grid > pieces) grid = pieces;
    return grid < 1 ? 1 : grid;
}

template <int CAP, typename F>
cudaError_t in_groups_of(const ep_grad *g, int count, F &&f) {
    for (int i = 0, k = 0; i < count || k == 0; i += CAP, ++k) {
        Table<CAP> tab;
        const int pieces = fill(tab, g + i, count - i < CAP ? count - i : CAP);
        const cudaError_t e = f(tab, pieces, k);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Calls f(table, pieces, index) for the tensors in groups that a table holds: the smallest table that holds
// all, because a launch copies it whole (300 tensors, in place: 28 us for the clipping that has nothing to do
// with a table of 1024).
template <typename F>
cudaError_t in_groups(const ep_grad *g, int count, F &&f) {
    if (count <= 32) return in_groups_of<32>(g, count, f);
    if (count <= 128) return in_groups_of<128>(g, count, f);
    if (count <= 384) return in_groups_of<384>(g, count, f);
    return in_groups_of<1024>(g, count, f);
}

}  // namespace

cudaError_t launch_grad_norm(const ep_grad *g, int count, double *partials, int sms, cudaStream_t stream) {
    return in_groups(g, count, [&](const auto &tab, int pieces, int k) {
        return launch(grad_norm_kernel<(int)(sizeof(tab.src) / sizeof(tab.src[0]))>, grid_of(pieces, sms), stream, tab, partials,
                      k > 0 ? 1 : 0);
    });
}

cudaError_t launch_grad_clip(const ep_grad *g, int count, const double *partials, float max_norm, float *norm, int sms,
                             int all_sms, cudaStream_t stream) {
    return in_groups(g, count, [&](const auto &tab, int pieces, int k) {
        // Out of place short CTAs of 8 pieces take the stores at the copy rate (671M elements, 2.7 GB: 786 us, with
        // the resident CTAs each on a long way 854); in place, where there is mostly nothing to do, they would
        // only all add up the partial sums (61 instead of 8 us; where there is something to do 858 us).
        int grid = grid_of(pieces, sms);
        if (!tab.in_place && sms == all_sms && grid < pieces / 8) grid = pieces / 8;
        return launch(grad_clip_kernel<(int)(sizeof(tab.src) / sizeof(tab.src[0]))>, grid, stream, tab, partials, max_norm,
                      k == 0 ? norm : nullptr);
    });
}

}  // namespace ep

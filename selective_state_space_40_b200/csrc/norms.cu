// norms.cu -- the root-mean-square norms around a layer, fused with what sits
// beside them: the gate behind the layer, the residual add and its scales in
// front of the next one; and their gradients.
//
// Over a group of W columns of a row, with a the normed value and
// inv = 1 / sqrt(mean(a^2) + eps):
//   forward   y = a inv w                              one sum:  a^2
//   backward  da = inv (g - a inv^2 mean(g a)), g = dy w   two sums: a^2, g a
// Both passes hold their row in registers between the sum and the use of it,
// so every array crosses HBM once, which is what bounds them. A group is held
// by tpr threads, NV vectors of VEC neighbouring columns each (16 bytes of the
// inputs' type where every row allows it, else single columns); the sums go
// over the threads by shuffles, and over the warps through shared memory where
// a group has more than one. A block is a column block of gb groups times ty
// rows and walks down the rows, so a thread's columns, and the weights' sums
// over rows that it keeps for them in registers, stay the same. Those sums go
// to one row of partial sums per (block, ty), which a second kernel adds up in
// a fixed order: the results do not depend on the order in which blocks run.

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "mambascan.h"
#include "ms_device.cuh"
#include "ms_internal.h"

namespace ms {

namespace {

constexpr int kMaxThr = 512;  // threads of a block, at most

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = Elem<T>::load(p);
    } else if constexpr (sizeof(T) == 2) {
        static_assert(VEC % 8 == 0, "");
#pragma unroll
        for (int q = 0; q < VEC / 8; ++q) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p) + q);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[8 * q + 2 * i] = bf16_lo(u[i]);
                v[8 * q + 2 * i + 1] = bf16_hi(u[i]);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(p) + q);
            v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        Elem<T>::store(p, v[0]);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int q = 0; q < VEC / 8; ++q) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
            reinterpret_cast<uint4 *>(p)[q] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q)
            reinterpret_cast<float4 *>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
}

// How a launch lays threads over rows and columns.
struct NormPlan {
    int tpr;      // threads per group: a power of two up to 32, or a multiple of 32
    int gb;       // groups per block (1 when tpr > 32)
    int ty;       // rows per block
    int gblocks;  // column blocks
    int rblocks;  // row blocks
    int W;        // columns per group
};

// Sums of NS values over the tpr threads of a group, the same in every thread.
template <int NS>
__device__ __forceinline__ void group_sum(float (&s)[NS], int tpr, float *sm) {
    const int width = tpr < 32 ? tpr : 32;
    for (int off = width >> 1; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, wpg = tpr >> 5, w0 = warp / wpg * wpg;
        __syncthreads();  // the last row's sums have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) sm[NS * warp + i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] = 0.0f;
        for (int w = w0; w < w0 + wpg; ++w)
#pragma unroll
            for (int i = 0; i < NS; ++i) s[i] += sm[NS * w + i];
    }
}

// This thread's place: its row within the block, its group, and whether its
// vector j lies inside the group (columns [c0 + j * tpr * VEC, + VEC)).
struct Place {
    int ty;
    int64_t g;
    int c0;
    bool live;
};
template <int VEC>
__device__ __forceinline__ Place place_of(const NormPlan &pl, int64_t groups) {
    Place p;
    const int tx = pl.tpr * pl.gb, t = threadIdx.x;
    p.ty = t / tx;
    const int x = t % tx;
    p.g = (int64_t)blockIdx.y * pl.gb + x / pl.tpr;
    p.c0 = (x % pl.tpr) * VEC;
    p.live = p.g < groups;
    return p;
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThr) gated_norm_fwd_kernel(const GatedNormArgs a, const NormPlan pl) {
    __shared__ float sm[32];
    const Place p = place_of<VEC>(pl, a.groups);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.g * pl.W;
    float w[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = p.c0 + j * pl.tpr * VEC;
            w[j][i] = (a.w && p.live && c < pl.W) ? __ldg(a.w + col + c + i) : 1.0f;
        }
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += (int64_t)gridDim.x * pl.ty) {
        const int64_t r = r0 + p.ty;
        const bool on = p.live && r < a.rows;
        float x[NV][VEC], gt[NV][VEC], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = 0.0f, gt[j][i] = 1.0f;
            if (on && c < pl.W) {
                load_vec<T, VEC>(static_cast<const T *>(a.x) + r * a.x_sr + col + c, x[j]);
                if (a.z) {
                    load_vec<T, VEC>(static_cast<const T *>(a.z) + r * a.z_sr + col + c, gt[j]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        gt[j][i] = silu_f(gt[j][i]);
                        if (a.gate_first) x[j][i] *= gt[j][i];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(x[j][i], x[j][i], s[0]);
        }
        group_sum<1>(s, pl.tpr, sm);
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            if (on && c < pl.W) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] = x[j][i] * inv * w[j][i] * (a.gate_first ? 1.0f : gt[j][i]);
                store_vec<T, VEC>(static_cast<T *>(a.y) + r * a.y_sr + col + c, y);
            }
        }
    }
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThr) gated_norm_bwd_kernel(const GatedNormArgs a, const NormPlan pl) {
    __shared__ float sm[64];
    const Place p = place_of<VEC>(pl, a.groups);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.g * pl.W;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = p.c0 + j * pl.tpr * VEC;
            w[j][i] = (a.w && p.live && c < pl.W) ? __ldg(a.w + col + c + i) : 1.0f;
            dw[j][i] = 0.0f;
        }
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += (int64_t)gridDim.x * pl.ty) {
        const int64_t r = r0 + p.ty;
        const bool on = p.live && r < a.rows;
        float x[NV][VEC], z[NV][VEC], dy[NV][VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = z[j][i] = dy[j][i] = 0.0f;
            if (on && c < pl.W) {
                load_vec<T, VEC>(static_cast<const T *>(a.x) + r * a.x_sr + col + c, x[j]);
                load_vec<T, VEC>(static_cast<const T *>(a.dy) + r * a.y_sr + col + c, dy[j]);
                if (a.z) load_vec<T, VEC>(static_cast<const T *>(a.z) + r * a.z_sr + col + c, z[j]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                // u: the normed value; gr: the gradient of n(u) w
                const float gate = a.z ? silu_f(z[j][i]) : 1.0f;
                const float u = a.gate_first ? x[j][i] * gate : x[j][i];
                const float gr = a.gate_first ? dy[j][i] : dy[j][i] * gate;
                s[0] = fmaf(u, u, s[0]);
                s[1] = fmaf(gr * w[j][i], u, s[1]);
            }
        }
        group_sum<2>(s, pl.tpr, sm);
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
        const float k = inv * inv * s[1] * invW;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            if (on && c < pl.W) {
                float dx[VEC], dz[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    // silu = z sig, silu' = sig (1 + z (1 - sig))
                    const float sig = a.z ? rcp_mufu(1.0f + exp2_mufu(-z[j][i] * kLog2e)) : 1.0f;
                    const float gate = a.z ? z[j][i] * sig : 1.0f;
                    const float slope = sig * fmaf(z[j][i], 1.0f - sig, 1.0f);
                    const float u = a.gate_first ? x[j][i] * gate : x[j][i];
                    const float gr = a.gate_first ? dy[j][i] : dy[j][i] * gate;
                    const float du = inv * fmaf(-k, u, gr * w[j][i]);
                    const float hat = u * inv;
                    dw[j][i] = fmaf(gr, hat, dw[j][i]);
                    dx[i] = a.gate_first ? du * gate : du;
                    dz[i] = (a.gate_first ? du * x[j][i] : dy[j][i] * hat * w[j][i]) * slope;
                }
                store_vec<T, VEC>(static_cast<T *>(a.dx) + r * a.width + col + c, dx);
                if (a.z) store_vec<T, VEC>(static_cast<T *>(a.dz) + r * a.width + col + c, dz);
            }
        }
    }
    if (a.dw && p.live) {
        float *part = a.part + ((int64_t)blockIdx.x * pl.ty + p.ty) * a.width + col;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            if (c < pl.W) store_vec<float, VEC>(part + c, dw[j]);
        }
    }
}

template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThr) residual_norm_fwd_kernel(const ResidualNormArgs a, const NormPlan pl) {
    __shared__ float sm[32];
    const Place p = place_of<VEC>(pl, 1);
    const float invW = 1.0f / (float)pl.W;
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += (int64_t)gridDim.x * pl.ty) {
        const int64_t r = r0 + p.ty;
        const bool on = r < a.rows;
        float h[NV][VEC], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            float x[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] = x[i] = 0.0f;
            if (on && c < pl.W) {
                load_vec<T, VEC>(static_cast<const T *>(a.x) + r * a.x_sr + c, x);
                if (a.res) load_vec<R, VEC>(static_cast<const R *>(a.res) + r * a.res_sr + c, h[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    h[j][i] = fmaf(a.cs ? a.scale * __ldg(a.cs + c + i) : a.scale, x[i], h[j][i]);
                if (a.res_out) store_vec<R, VEC>(static_cast<R *>(a.res_out) + r * a.ro_sr + c, h[j]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(h[j][i], h[j][i], s[0]);
        }
        group_sum<1>(s, pl.tpr, sm);
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            if (on && c < pl.W) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] = h[j][i] * inv * (a.w ? __ldg(a.w + c + i) : 1.0f);
                store_vec<T, VEC>(static_cast<T *>(a.y) + r * a.y_sr + c, y);
            }
        }
    }
}

template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThr) residual_norm_bwd_kernel(const ResidualNormArgs a, const NormPlan pl) {
    __shared__ float sm[64];
    const Place p = place_of<VEC>(pl, 1);
    const float invW = 1.0f / (float)pl.W;
    float w[NV][VEC], dw[NV][VEC], dc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = p.c0 + j * pl.tpr * VEC;
            w[j][i] = (a.w && c < pl.W) ? __ldg(a.w + c + i) : 1.0f;
            dw[j][i] = dc[j][i] = 0.0f;
        }
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += (int64_t)gridDim.x * pl.ty) {
        const int64_t r = r0 + p.ty;
        const bool on = r < a.rows;
        float h[NV][VEC], dy[NV][VEC], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] = dy[j][i] = 0.0f;
            if (on && c < pl.W) {
                load_vec<R, VEC>(static_cast<const R *>(a.res_out) + r * a.ro_sr + c, h[j]);
                load_vec<T, VEC>(static_cast<const T *>(a.dy) + r * a.y_sr + c, dy[j]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[0] = fmaf(h[j][i], h[j][i], s[0]);
                s[1] = fmaf(dy[j][i] * w[j][i], h[j][i], s[1]);
            }
        }
        group_sum<2>(s, pl.tpr, sm);
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
        const float k = inv * inv * s[1] * invW;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = p.c0 + j * pl.tpr * VEC;
            if (on && c < pl.W) {
                float d[VEC], x[VEC];
                if (a.dres_out) {
                    load_vec<R, VEC>(static_cast<const R *>(a.dres_out) + r * a.res_sr + c, d);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) d[i] = 0.0f;
                }
                if (a.dcs) load_vec<T, VEC>(static_cast<const T *>(a.x) + r * a.x_sr + c, x);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    d[i] += inv * fmaf(-k, h[j][i], dy[j][i] * w[j][i]);
                    dw[j][i] = fmaf(dy[j][i], h[j][i] * inv, dw[j][i]);
                }
                if (a.dres) store_vec<R, VEC>(static_cast<R *>(a.dres) + r * a.width + c, d);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    d[i] *= a.scale;
                    if (a.dcs) dc[j][i] = fmaf(d[i], x[i], dc[j][i]);
                    if (a.cs) d[i] *= __ldg(a.cs + c + i);
                }
                if (a.dx) store_vec<T, VEC>(static_cast<T *>(a.dx) + r * a.width + c, d);
            }
        }
    }
    const int64_t prow = (int64_t)blockIdx.x * pl.ty + p.ty;
    float *part = a.part;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = p.c0 + j * pl.tpr * VEC;
        if (c < pl.W) {
            if (a.dw) store_vec<float, VEC>(part + prow * a.width + c, dw[j]);
            if (a.dcs) store_vec<float, VEC>(part + ((int64_t)gridDim.x * pl.ty + prow) * a.width + c, dc[j]);
        }
    }
}

// out[c] = sum over the rows of part, each thread its own rows in order and
// then the threads of a column in order.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float *part, float *out0, float *out1, int64_t parts,
                                                       int64_t width) {
    __shared__ float sm[8][32];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float *out = blockIdx.y ? out1 : out0;
    if (out == nullptr) return;
    const float *src = part + (int64_t)blockIdx.y * parts * width;
    float s = 0.0f;
    if (c < width)
        for (int64_t r = ty; r < parts; r += 8) s += src[r * width + c];
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < width) {
        for (int i = 1; i < 8; ++i) s += sm[i][tx];
        out[c] = s;
    }
}

// Threads per group for NV vectors each: a power of two up to a warp, else whole warps.
int threads_for(int64_t W, int vec, int nv) {
    const int64_t need = (W + (int64_t)vec * nv - 1) / ((int64_t)vec * nv);
    if (need > 32) return (int)((need + 31) / 32 * 32);
    int t = 1;
    while (t < need) t *= 2;
    return t;
}

// Vectors per thread: the fewest that keep a group within a block, and for
// groups of more than 256 vectors at least two, so that a block's sum over its
// warps is paid by more bytes.
int vectors_for(int64_t W, int vec) {
    for (int nv = W > 256 * vec ? 2 : 1; nv < 32; nv *= 2)
        if (threads_for(W, vec, nv) <= kMaxThr) return nv;
    return 32;
}

NormPlan plan_norm(int64_t rows, int64_t W, int64_t groups, int vec, int nv, int num_sms, bool bwd) {
    NormPlan pl{};
    pl.W = (int)W;
    pl.tpr = threads_for(W, vec, nv);
    pl.gb = 1;
    if (pl.tpr <= 32) {
        // as many whole groups as 256 threads hold, a multiple of a warp in all
        int64_t gb = std::min<int64_t>(groups, 256 / pl.tpr);
        pl.gb = (int)gb;
        pl.ty = 1;
        while (pl.tpr * pl.gb * pl.ty % 32 != 0) ++pl.ty;
        const int base = pl.ty;
        while (pl.tpr * pl.gb * (pl.ty + base) <= 256) pl.ty += base;
    } else {
        pl.ty = 1;
    }
    pl.gblocks = (int)((groups + pl.gb - 1) / pl.gb);
    const int64_t rb = (rows + pl.ty - 1) / pl.ty;
    // the backward's partial sums are one row per block and ty: few blocks, each down many rows
    const int64_t per_sm = std::max<int64_t>(1, (bwd ? 1024 : 2048) / ((int64_t)pl.tpr * pl.gb * pl.ty));
    const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms * per_sm / pl.gblocks);
    pl.rblocks = (int)std::max<int64_t>(1, std::min(rb, cap));
    return pl;
}

bool vec16(const void *p, int64_t sr, int es) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (sr * es) % 16 == 0);
}

template <int NV, typename T, int VEC>
cudaError_t run_gated(const GatedNormArgs &a, const NormPlan &pl, bool bwd, cudaStream_t st) {
    const dim3 grid((unsigned)pl.rblocks, (unsigned)pl.gblocks);
    const unsigned thr = (unsigned)(pl.tpr * pl.gb * pl.ty);
    if (bwd) gated_norm_bwd_kernel<T, VEC, NV><<<grid, thr, 0, st>>>(a, pl);
    else gated_norm_fwd_kernel<T, VEC, NV><<<grid, thr, 0, st>>>(a, pl);
    return cudaGetLastError();
}
template <int NV, typename T, typename R, int VEC>
cudaError_t run_residual(const ResidualNormArgs &a, const NormPlan &pl, bool bwd, cudaStream_t st) {
    const dim3 grid((unsigned)pl.rblocks, 1u);
    const unsigned thr = (unsigned)(pl.tpr * pl.gb * pl.ty);
    if (bwd) residual_norm_bwd_kernel<T, R, VEC, NV><<<grid, thr, 0, st>>>(a, pl);
    else residual_norm_fwd_kernel<T, R, VEC, NV><<<grid, thr, 0, st>>>(a, pl);
    return cudaGetLastError();
}

cudaError_t sum_parts(const float *part, float *o0, float *o1, const NormPlan &pl, int64_t width, cudaStream_t st) {
    if (!o0 && !o1) return cudaSuccess;
    const dim3 grid((unsigned)((width + 31) / 32), 2u);
    norm_sum_kernel<<<grid, 256, 0, st>>>(part, o0, o1, (int64_t)pl.rblocks * pl.ty, width);
    return cudaGetLastError();
}

// Vector widths: 8 columns where an array is bf16, 4 where all are fp32, 1 for rows that do not allow 16-byte accesses.
template <typename F>
cudaError_t with_nv(int nv, F f) {
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
        default: return f(std::integral_constant<int, 32>{});
    }
}

}  // namespace

// Rows of partial sums that a backward of these sizes can need, for any vector width.
size_t norm_parts(int64_t rows, int64_t width, int64_t groups, int num_sms) {
    size_t most = 0;
    for (int vec : {8, 4, 1}) {
        const int64_t W = width / groups;
        const NormPlan pl = plan_norm(rows, W, groups, vec, vectors_for(W, vec), num_sms, true);
        most = std::max(most, (size_t)pl.rblocks * (size_t)pl.ty);
    }
    return most;
}

cudaError_t launch_gated_norm(const GatedNormArgs &a, bool bf16, bool bwd, int num_sms, cudaStream_t stream) {
    const int64_t W = a.width / a.groups;
    const int es = bf16 ? 2 : 4, v = bf16 ? 8 : 4;
    const bool ok = W % v == 0 && vec16(a.x, a.x_sr, es) && vec16(a.z, a.z_sr, es) && vec16(a.y, a.y_sr, es) &&
                    vec16(a.dy, a.y_sr, es) && vec16(a.dx, a.width, es) && vec16(a.dz, a.width, es);
    const int vec = ok ? v : 1, nv = vectors_for(W, vec);
    const NormPlan pl = plan_norm(a.rows, W, a.groups, vec, nv, num_sms, bwd);
    cudaError_t e = with_nv(nv, [&](auto n) {
        constexpr int NV = decltype(n)::value;
        if (vec == 1)
            return bf16 ? run_gated<NV, __nv_bfloat16, 1>(a, pl, bwd, stream) : run_gated<NV, float, 1>(a, pl, bwd, stream);
        if constexpr (NV <= 8)
            return bf16 ? run_gated<NV, __nv_bfloat16, 8>(a, pl, bwd, stream) : run_gated<NV, float, 4>(a, pl, bwd, stream);
        else
            return cudaErrorInvalidConfiguration;
    });
    if (e == cudaSuccess && bwd) e = sum_parts(a.part, a.dw, nullptr, pl, a.width, stream);
    return e;
}

cudaError_t launch_residual_norm(const ResidualNormArgs &a, bool bf16, bool res_bf16, bool bwd, int num_sms,
                                 cudaStream_t stream) {
    const int64_t W = a.width;
    const int es = bf16 ? 2 : 4, rs = res_bf16 ? 2 : 4, v = bf16 || res_bf16 ? 8 : 4;
    const bool ok = W % v == 0 && vec16(a.x, a.x_sr, es) && vec16(a.res, a.res_sr, rs) && vec16(a.y, a.y_sr, es) &&
                    vec16(a.dy, a.y_sr, es) && vec16(a.res_out, a.ro_sr, rs) && vec16(a.dres_out, a.res_sr, rs) &&
                    vec16(a.dx, a.width, es) && vec16(a.dres, a.width, rs);
    const int vec = ok ? v : 1, nv = vectors_for(W, vec);
    const NormPlan pl = plan_norm(a.rows, W, 1, vec, nv, num_sms, bwd);
    cudaError_t e = with_nv(nv, [&](auto n) -> cudaError_t {
        constexpr int NV = decltype(n)::value;
        if (vec == 1) {
            if (bf16)
                return res_bf16 ? run_residual<NV, __nv_bfloat16, __nv_bfloat16, 1>(a, pl, bwd, stream)
                                : run_residual<NV, __nv_bfloat16, float, 1>(a, pl, bwd, stream);
            return res_bf16 ? run_residual<NV, float, __nv_bfloat16, 1>(a, pl, bwd, stream)
                            : run_residual<NV, float, float, 1>(a, pl, bwd, stream);
        }
        if constexpr (NV <= 8) {
            if (bf16)
                return res_bf16 ? run_residual<NV, __nv_bfloat16, __nv_bfloat16, 8>(a, pl, bwd, stream)
                                : run_residual<NV, __nv_bfloat16, float, 8>(a, pl, bwd, stream);
            return res_bf16 ? run_residual<NV, float, __nv_bfloat16, 8>(a, pl, bwd, stream)
                            : run_residual<NV, float, float, 4>(a, pl, bwd, stream);
        }
        return cudaErrorInvalidConfiguration;
    });
    if (e == cudaSuccess && bwd) e = sum_parts(a.part, a.dw, a.dcs, pl, a.width, stream);
    return e;
}

}  // namespace ms

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
// inputs' type where every row allows it, else loaded column by column); the sums go
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

constexpr int kMaxThr = 640;  // threads of a block, at most
// Registers of a thread. The backward keeps its columns' weights and their sums; its
// blocks of 640 threads (5120 bf16 columns) run one to an SM, of 320 two.
constexpr int regs_of(int nv, bool bwd) { return nv > 1 || bwd ? 96 : 56; }

// VEC neighbouring elements as they lie in memory: a row waits in this form.
template <typename T, int VEC, bool ODD>
struct Raw {
    uint4 v[VEC * sizeof(T) / 16];
    __device__ __forceinline__ void load(const T *p, int on) {
#pragma unroll
        for (int q = 0; q < (int)(VEC * sizeof(T) / 16); ++q)
            v[q] = on ? __ldg(reinterpret_cast<const uint4 *>(p) + q) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load_shared(uint32_t at, int on) {
#pragma unroll
        for (int q = 0; q < (int)(VEC * sizeof(T) / 16); ++q) {
            v[q] = make_uint4(0, 0, 0, 0);
            if (on)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[q].x), "=r"(v[q].y), "=r"(v[q].z), "=r"(v[q].w)
                             : "r"(at + 16u * q)
                             : "memory");
        }
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
        for (int q = 0; q < (int)(VEC * sizeof(T) / 16); ++q) {
            const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    f[8 * q + 2 * i] = bf16_lo(u[i]);
                    f[8 * q + 2 * i + 1] = bf16_hi(u[i]);
                } else {
                    f[4 * q + i] = __uint_as_float(u[i]);
                }
            }
        }
    }
};
// The same column by column, for rows of any alignment and width: `on` is how many there are.
template <typename T, int VEC>
struct Raw<T, VEC, true> {
    float v[VEC];
    __device__ __forceinline__ void load(const T *p, int on) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < on ? Elem<T>::load(p + i) : 0.0f;
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = v[i];
    }
};
// fp32 weights of VEC columns, 1 where there are none
template <int VEC, bool ODD>
__device__ __forceinline__ void weights(const float *w, int on, float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = 1.0f;
    if (w && on) {
        Raw<float, VEC, ODD> r;
        r.load(w, on);
        r.get(f);
    }
}
template <typename T, int VEC, bool ODD>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC], int on) {
    if constexpr (ODD) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < on) Elem<T>::store(p + i, v[i]);
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

// Rows on their way through shared memory: NA arrays' rows a stage, brought by bulk
// copies, so that several rows of a block are in flight without holding registers
// (the gated backward of 8192 x 5120 in bf16: 102 us, 109 us with rows straight to registers).
// For blocks of one group; row k of a block is in stage k % stages, phase k / stages.
template <int NA>
struct Ring {
    uint32_t data, bars, stage_bytes;
    uint32_t bytes[NA];  // of each array's row (0: not there)
    int stages;
    __device__ __forceinline__ uint32_t bar(int st) const { return bars + 8u * (uint32_t)st; }
    // by every thread, with a barrier behind it
    __device__ __forceinline__ void init(unsigned char *smem, int n) {
        stages = n;
        bars = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
        data = bars + 128u;
        stage_bytes = 0;
#pragma unroll
        for (int i = 0; i < NA; ++i) stage_bytes += bytes[i];
        if (threadIdx.x == 0) {
            for (int i = 0; i < n; ++i)
                asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar(i)) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    __device__ __forceinline__ void issue(int st, const void *const (&src)[NA]) const {
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar(st)), "r"(stage_bytes) : "memory");
        uint32_t at = data + (uint32_t)st * stage_bytes;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            if (bytes[i])
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(at),
                             "l"(src[i]), "r"(bytes[i]), "r"(bar(st))
                             : "memory");
            at += bytes[i];
        }
    }
    // bounded: on a timeout MS_ERR_TIMEOUT is recorded and the row is not valid
    __device__ __forceinline__ void wait(int st, uint32_t phase, int *status) const {
        for (uint32_t i = 0; i < (1u << 20); ++i) {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(bar(st)), "r"(phase & 1u)
                : "memory");
            if (done) return;
        }
        if (status) atomicOr(status, MS_ERR_TIMEOUT);
    }
    // shared address of array i's row in a stage
    __device__ __forceinline__ uint32_t row(int st, int i) const {
        uint32_t at = data + (uint32_t)st * stage_bytes;
#pragma unroll
        for (int k = 0; k < NA; ++k)
            if (k < i) at += bytes[k];
        return at;
    }
};

// How a launch lays threads over rows and columns.
struct NormPlan {
    int tpr;      // threads per group: a power of two up to 32, or a multiple of 32
    int gb;       // groups per block (1 when tpr > 32)
    int ty;       // rows per block
    int gblocks;  // column blocks
    int rblocks;  // row blocks
    int W;        // columns per group
    int stages;   // rows of a block's ring (0: rows go straight to registers)
};

// Sums of NS values over the tpr threads of a group, the same in every thread.
// `sm` holds two rows' sums of the warps, used in turn: one barrier a row.
constexpr int kMaxWarps = kMaxThr / 32;
template <int NS>
__device__ __forceinline__ void group_sum(float (&s)[NS], int tpr, float (*sm)[2 * kMaxWarps], int &turn) {
    const int width = tpr < 32 ? tpr : 32;
    for (int off = width >> 1; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, warps = tpr >> 5;  // (one group a block)
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) sm[turn][NS * warp + i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] = 0.0f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < NS; ++i) s[i] += sm[turn][NS * w + i];
        turn ^= 1;
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

// Weights of a thread's columns: read once where they fit into registers, else for every row (from L1).
template <int VEC, int NV>
constexpr bool kHold = VEC *NV <= 8;

// How the gate takes part: not at all, behind the norm, or in front of it.
enum { kNoGate = 0, kGateBehind = 1, kGateFirst = 2 };
__device__ __forceinline__ float sigmoid_f(float z) { return rcp_mufu(1.0f + exp2_mufu(-z * kLog2e)); }

// The rows of a block are read one ahead of the row in work where the registers
// allow it: a row's sums wait for all of its columns.
// How rows come: straight to registers, through a ring in shared memory, or straight and column by column
// (rows that 16-byte accesses do not fit).
enum { kStraight = 0, kRing = 1, kOdd = 2 };
template <int VEC>
__device__ __forceinline__ int columns(int left) {
    return left <= 0 ? 0 : left < VEC ? left : VEC;
}

template <int VEC, int NV, bool RING>
constexpr bool kAhead = !RING && VEC *NV <= 16;
template <int VEC, int NV, bool RING>
constexpr bool kAheadBwd = !RING && VEC *NV <= 4;

template <typename T, int VEC, int NV, int ROWS, int GATE>
__global__ void __maxnreg__(regs_of(NV, false)) gated_norm_fwd_kernel(const GatedNormArgs a, const NormPlan pl) {
    constexpr bool RING = ROWS == kRing, ODD = ROWS == kOdd;
    __shared__ float sm[2][2 * kMaxWarps];
    int turn = 0;
    const Place p = place_of<VEC>(pl, a.groups);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.g * pl.W + p.c0, dr = (int64_t)gridDim.x * pl.ty;
    const int dc = pl.tpr * VEC;
    int in[NV];  // columns of each vector that there are
    float w[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = p.live ? columns<VEC>(pl.W - p.c0 - j * dc) : 0;
        if (!MS_CHECK(a.status, in[j] == 0 || col + j * dc + in[j] <= a.width)) in[j] = 0;
        weights<VEC, ODD>(a.w ? a.w + col + j * dc : nullptr, in[j], w[j]);
    }
    Raw<T, VEC, ODD> rx[NV], rz[NV], nx[NV], nz[NV];
    const T *x = static_cast<const T *>(a.x) + col, *z = static_cast<const T *>(a.z) + col;
    auto fetch = [&](int64_t r, Raw<T, VEC, ODD> (&fx)[NV], Raw<T, VEC, ODD> (&fz)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int on = r < a.rows ? in[j] : 0;
            fx[j].load(x + r * a.x_sr + j * dc, on);
            if constexpr (GATE != kNoGate) fz[j].load(z + r * a.z_sr + j * dc, on);
        }
    };
    extern __shared__ __align__(128) unsigned char ring_smem[];
    Ring<2> ring;
    int st = 0;  // the row's stage, and its phase
    uint32_t phase = 0;
    auto refill = [&](int stage, int64_t row) {
        const void *const src[2] = {static_cast<const T *>(a.x) + row * a.x_sr + p.g * pl.W, static_cast<const T *>(a.z) + row * a.z_sr + p.g * pl.W};
        ring.issue(stage, src);
    };
    if constexpr (RING) {
        ring.bytes[0] = pl.W * (uint32_t)sizeof(T);
        ring.bytes[1] = GATE != kNoGate ? ring.bytes[0] : 0u;
        ring.init(ring_smem, pl.stages);
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < pl.stages; ++i)
                if (blockIdx.x + i * dr < a.rows) refill(i, blockIdx.x + i * dr);
    }
    int64_t r = (int64_t)blockIdx.x * pl.ty + p.ty;
    if (kAhead<VEC, NV, RING>) fetch(r, rx, rz);
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += dr, r += dr) {
        if (kAhead<VEC, NV, RING>) fetch(r + dr, nx, nz);
        else if constexpr (!RING) fetch(r, rx, rz);
        if constexpr (RING) {
            ring.wait(st, phase, a.status);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                rx[j].load_shared(ring.row(st, 0) + (p.c0 + j * dc) * (uint32_t)sizeof(T), in[j]);
                if constexpr (GATE != kNoGate) rz[j].load_shared(ring.row(st, 1) + (p.c0 + j * dc) * (uint32_t)sizeof(T), in[j]);
            }
        }
        float v[NV][VEC], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rx[j].get(v[j]);
            if constexpr (GATE == kGateFirst) {
                float g[VEC];
                rz[j].get(g);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j][i] *= silu_f(g[i]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(v[j][i], v[j][i], s[0]);
        }
        group_sum<1>(s, pl.tpr, sm, turn);
        if constexpr (RING) {
            // every thread has read the row: its place is the next one's
            if (threadIdx.x == 0 && r + pl.stages * dr < a.rows) refill(st, r + pl.stages * dr);
            if (++st == pl.stages) st = 0, ++phase;
        }
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] *= inv * w[j][i];
            if constexpr (GATE == kGateBehind) {
                float g[VEC];
                rz[j].get(g);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j][i] *= silu_f(g[i]);
            }
            if (in[j] && r < a.rows) store_vec<T, VEC, ODD>(static_cast<T *>(a.y) + r * a.y_sr + col + j * dc, v[j], in[j]);
            if (kAhead<VEC, NV, RING>) rx[j] = nx[j], rz[j] = nz[j];
        }
    }
}

template <typename T, int VEC, int NV, int ROWS, int GATE>
__global__ void __maxnreg__(regs_of(NV, true)) gated_norm_bwd_kernel(const GatedNormArgs a, const NormPlan pl) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr bool RING = ROWS == kRing, ODD = ROWS == kOdd;
    __shared__ float sm[2][2 * kMaxWarps];
    int turn = 0;
    const Place p = place_of<VEC>(pl, a.groups);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.g * pl.W + p.c0, dr = (int64_t)gridDim.x * pl.ty;
    const int dc = pl.tpr * VEC;
    int in[NV];  // columns of each vector that there are
    float dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = p.live ? columns<VEC>(pl.W - p.c0 - j * dc) : 0;
        if (!MS_CHECK(a.status, in[j] == 0 || col + j * dc + in[j] <= a.width)) in[j] = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = 0.0f;
    }
    constexpr bool kAh = kAheadBwd<VEC, NV, RING>;
    Raw<T, VEC, ODD> rx[NV], rz[NV], ry[NV], nx[kAh ? NV : 1], nz[kAh ? NV : 1], ny[kAh ? NV : 1];
    const T *x = static_cast<const T *>(a.x) + col, *z = static_cast<const T *>(a.z) + col;
    const T *dy = static_cast<const T *>(a.dy) + col;
    auto fetch = [&](int64_t r, int j, Raw<T, VEC, ODD> &fx, Raw<T, VEC, ODD> &fy, Raw<T, VEC, ODD> &fz) {
        const int on = r < a.rows ? in[j] : 0;
        fx.load(x + r * a.x_sr + j * dc, on);
        fy.load(dy + r * a.y_sr + j * dc, on);
        if constexpr (GATE != kNoGate) fz.load(z + r * a.z_sr + j * dc, on);
    };
    const float *wt = a.w ? a.w + col : nullptr;
    float hw[kHold<VEC, NV> ? NV : 1][VEC];
    if constexpr (kHold<VEC, NV>)
#pragma unroll
        for (int j = 0; j < NV; ++j) weights<VEC, ODD>(wt ? wt + j * dc : nullptr, in[j], hw[j]);
    auto weights_of = [&](int j, float (&w)[VEC]) {
        if constexpr (kHold<VEC, NV>) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = hw[j][i];
        } else {
            weights<VEC, ODD>(wt ? wt + j * dc : nullptr, in[j], w);
        }
    };
    extern __shared__ __align__(128) unsigned char ring_smem[];
    Ring<3> ring;
    int st = 0;  // the row's stage, and its phase
    uint32_t phase = 0;
    auto refill = [&](int stage, int64_t row) {
        const void *const src[3] = {static_cast<const T *>(a.x) + row * a.x_sr + p.g * pl.W, static_cast<const T *>(a.dy) + row * a.y_sr + p.g * pl.W,
                                     static_cast<const T *>(a.z) + row * a.z_sr + p.g * pl.W};
        ring.issue(stage, src);
    };
    if constexpr (RING) {
        ring.bytes[0] = ring.bytes[1] = pl.W * (uint32_t)sizeof(T);
        ring.bytes[2] = GATE != kNoGate ? ring.bytes[0] : 0u;
        ring.init(ring_smem, pl.stages);
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < pl.stages; ++i)
                if (blockIdx.x + i * dr < a.rows) refill(i, blockIdx.x + i * dr);
    }
    int64_t r = (int64_t)blockIdx.x * pl.ty + p.ty;
    if constexpr (kAh)
#pragma unroll
        for (int j = 0; j < NV; ++j) fetch(r, j, rx[j], ry[j], rz[j]);
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += dr, r += dr) {
        float s[2] = {0.0f, 0.0f};
        if constexpr (RING) ring.wait(st, phase, a.status);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (RING) {
                const int on = r < a.rows ? in[j] : 0;
                const uint32_t at = (p.c0 + j * dc) * (uint32_t)sizeof(T);
                rx[j].load_shared(ring.row(st, 0) + at, on);
                ry[j].load_shared(ring.row(st, 1) + at, on);
                if constexpr (GATE != kNoGate) rz[j].load_shared(ring.row(st, 2) + at, on);
            } else if constexpr (kAh) {
                fetch(r + dr, j, nx[j], ny[j], nz[j]);
            } else {
                fetch(r, j, rx[j], ry[j], rz[j]);
            }
        }
        // u: the normed value; gr: the gradient of n(u) w; sig: silu(z) = z sig, of which both
        // passes need, kept between them (the formulas' instructions, not HBM, bound this kernel)
        float sig[NV][GATE != kNoGate ? VEC : 1];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[VEC], gr[VEC], z_[VEC], w[VEC];
            rx[j].get(u);
            ry[j].get(gr);
            weights_of(j, w);
            if constexpr (GATE != kNoGate) {
                rz[j].get(z_);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    sig[j][i] = sigmoid_f(z_[i]);
                    if constexpr (GATE == kGateFirst) u[i] *= z_[i] * sig[j][i];
                    else gr[i] *= z_[i] * sig[j][i];
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[0] = fmaf(u[i], u[i], s[0]);
                s[1] = fmaf(gr[i] * w[i], u[i], s[1]);
            }
        }
        group_sum<2>(s, pl.tpr, sm, turn);
        if constexpr (RING) {
            // every thread has read the row: its place is the next one's
            if (threadIdx.x == 0 && r + pl.stages * dr < a.rows) refill(st, r + pl.stages * dr);
            if (++st == pl.stages) st = 0, ++phase;
        }
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
        const float k = inv * inv * s[1] * invW;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[VEC], gr[VEC], z_[VEC], w[VEC], dz[VEC];
            rx[j].get(u);
            ry[j].get(gr);
            weights_of(j, w);
            if constexpr (GATE != kNoGate) rz[j].get(z_);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (GATE == kNoGate) {
                    dw[j][i] = fmaf(gr[i], u[i] * inv, dw[j][i]);
                    u[i] = inv * fmaf(-k, u[i], gr[i] * w[i]);
                } else {
                    // silu' = sig (1 + z (1 - sig)) = sig + silu (1 - sig)
                    const float sg = sig[j][i], gate = z_[i] * sg, slope = fmaf(gate, 1.0f - sg, sg);
                    if constexpr (GATE == kGateFirst) {
                        const float n = u[i] * gate, du = inv * fmaf(-k, n, gr[i] * w[i]);
                        dw[j][i] = fmaf(gr[i], n * inv, dw[j][i]);
                        dz[i] = du * u[i] * slope;
                        u[i] = du * gate;
                    } else {
                        const float hat = u[i] * inv, gi = gr[i] * gate;
                        dw[j][i] = fmaf(gi, hat, dw[j][i]);
                        dz[i] = gr[i] * hat * w[i] * slope;
                        u[i] = inv * fmaf(-k, u[i], gi * w[i]);
                    }
                }
            }
            if (in[j] && r < a.rows) {
                store_vec<T, VEC, ODD>(static_cast<T *>(a.dx) + r * a.width + col + j * dc, u, in[j]);
                if constexpr (GATE != kNoGate) store_vec<T, VEC, ODD>(static_cast<T *>(a.dz) + r * a.width + col + j * dc, dz, in[j]);
            }
            if constexpr (kAh) rx[j] = nx[j], ry[j] = ny[j], rz[j] = nz[j];
        }
    }
    if (a.dw) {
        float *part = a.part + ((int64_t)blockIdx.x * pl.ty + p.ty) * a.width + col;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (in[j]) store_vec<float, VEC, ODD>(part + j * dc, dw[j], in[j]);
    }
}

template <typename T, typename R, int VEC, int NV, int ROWS>
__global__ void __maxnreg__(regs_of(NV, false)) residual_norm_fwd_kernel(const ResidualNormArgs a, const NormPlan pl) {
    constexpr bool RING = ROWS == kRing, ODD = ROWS == kOdd;
    __shared__ float sm[2][2 * kMaxWarps];
    int turn = 0;
    const Place p = place_of<VEC>(pl, 1);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.c0, dr = (int64_t)gridDim.x * pl.ty;
    const int dc = pl.tpr * VEC;
    int in[NV];  // columns of each vector that there are
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = columns<VEC>(pl.W - p.c0 - j * dc);
        if (!MS_CHECK(a.status, in[j] == 0 || col + j * dc + in[j] <= a.width)) in[j] = 0;
    }
    Raw<T, VEC, ODD> rx[NV], nx[NV];
    Raw<R, VEC, ODD> rr[NV], nr[NV];
    auto fetch = [&](int64_t r, Raw<T, VEC, ODD> (&fx)[NV], Raw<R, VEC, ODD> (&fr)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int on = r < a.rows ? in[j] : 0;
            fx[j].load(static_cast<const T *>(a.x) + r * a.x_sr + col + j * dc, on);
            fr[j].load(static_cast<const R *>(a.res) + r * a.res_sr + col + j * dc, a.res ? on : 0);
        }
    };
    extern __shared__ __align__(128) unsigned char ring_smem[];
    Ring<2> ring;
    int st = 0;  // the row's stage, and its phase
    uint32_t phase = 0;
    auto refill = [&](int stage, int64_t row) {
        const void *const src[2] = {static_cast<const T *>(a.x) + row * a.x_sr, static_cast<const R *>(a.res) + row * a.res_sr};
        ring.issue(stage, src);
    };
    if constexpr (RING) {
        ring.bytes[0] = pl.W * (uint32_t)sizeof(T);
        ring.bytes[1] = a.res ? pl.W * (uint32_t)sizeof(R) : 0u;
        ring.init(ring_smem, pl.stages);
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < pl.stages; ++i)
                if (blockIdx.x + i * dr < a.rows) refill(i, blockIdx.x + i * dr);
    }
    int64_t r = (int64_t)blockIdx.x * pl.ty + p.ty;
    if (kAhead<VEC, NV, RING>) fetch(r, rx, rr);
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += dr, r += dr) {
        if (kAhead<VEC, NV, RING>) fetch(r + dr, nx, nr);
        else if constexpr (!RING) fetch(r, rx, rr);
        if constexpr (RING) {
            ring.wait(st, phase, a.status);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                rx[j].load_shared(ring.row(st, 0) + (p.c0 + j * dc) * (uint32_t)sizeof(T), in[j]);
                rr[j].load_shared(ring.row(st, 1) + (p.c0 + j * dc) * (uint32_t)sizeof(R), a.res ? in[j] : 0);
            }
        }
        float h[NV][VEC], s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[VEC], c[VEC];
            rx[j].get(x);
            rr[j].get(h[j]);
            weights<VEC, ODD>(a.cs ? a.cs + col + j * dc : nullptr, in[j], c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[j][i] = fmaf(a.scale * c[i], x[i], h[j][i]);
                s[0] = fmaf(h[j][i], h[j][i], s[0]);
            }
            if (in[j] && r < a.rows && a.res_out)
                store_vec<R, VEC, ODD>(static_cast<R *>(a.res_out) + r * a.ro_sr + col + j * dc, h[j], in[j]);
        }
        group_sum<1>(s, pl.tpr, sm, turn);
        if constexpr (RING) {
            // every thread has read the row: its place is the next one's
            if (threadIdx.x == 0 && r + pl.stages * dr < a.rows) refill(st, r + pl.stages * dr);
            if (++st == pl.stages) st = 0, ++phase;
        }
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[VEC];
            weights<VEC, ODD>(a.w ? a.w + col + j * dc : nullptr, in[j], w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] *= inv * w[i];
            if (in[j] && r < a.rows) store_vec<T, VEC, ODD>(static_cast<T *>(a.y) + r * a.y_sr + col + j * dc, h[j], in[j]);
            if (kAhead<VEC, NV, RING>) rx[j] = nx[j], rr[j] = nr[j];
        }
    }
}

template <typename T, typename R, int VEC, int NV, int ROWS>
__global__ void __maxnreg__(regs_of(NV, true)) residual_norm_bwd_kernel(const ResidualNormArgs a, const NormPlan pl) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr bool RING = ROWS == kRing, ODD = ROWS == kOdd;
    __shared__ float sm[2][2 * kMaxWarps];
    int turn = 0;
    const Place p = place_of<VEC>(pl, 1);
    const float invW = 1.0f / (float)pl.W;
    const int64_t col = p.c0, dr = (int64_t)gridDim.x * pl.ty;
    const int dc = pl.tpr * VEC;
    int in[NV];  // columns of each vector that there are
    float dw[NV][VEC], dch[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = columns<VEC>(pl.W - p.c0 - j * dc);
        if (!MS_CHECK(a.status, in[j] == 0 || col + j * dc + in[j] <= a.width)) in[j] = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = dch[j][i] = 0.0f;
    }
    float hw[kHold<VEC, NV> ? NV : 1][VEC], hc[kHold<VEC, NV> ? NV : 1][VEC];
    if constexpr (kHold<VEC, NV>)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            weights<VEC, ODD>(a.w ? a.w + col + j * dc : nullptr, in[j], hw[j]);
            weights<VEC, ODD>(a.cs ? a.cs + col + j * dc : nullptr, in[j], hc[j]);
        }
    auto weights_of = [&](const float *from, const float (&held)[kHold<VEC, NV> ? NV : 1][VEC], int j, float (&w)[VEC]) {
        if constexpr (kHold<VEC, NV>) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = held[j][i];
        } else {
            weights<VEC, ODD>(from ? from + col + j * dc : nullptr, in[j], w);
        }
    };
    constexpr bool kAh = kAheadBwd<VEC, NV, RING>;
    Raw<R, VEC, ODD> rh[NV], rd[NV], nh[kAh ? NV : 1], nd[kAh ? NV : 1];
    Raw<T, VEC, ODD> ry[NV], rx[NV], ny[kAh ? NV : 1], nx[kAh ? NV : 1];
    auto fetch = [&](int64_t r, int j, Raw<R, VEC, ODD> &fh, Raw<T, VEC, ODD> &fy, Raw<R, VEC, ODD> &fd, Raw<T, VEC, ODD> &fx) {
        const int on = r < a.rows ? in[j] : 0;
        fh.load(static_cast<const R *>(a.res_out) + r * a.ro_sr + col + j * dc, on);
        fy.load(static_cast<const T *>(a.dy) + r * a.y_sr + col + j * dc, on);
        fd.load(static_cast<const R *>(a.dres_out) + r * a.res_sr + col + j * dc, a.dres_out ? on : 0);
        fx.load(static_cast<const T *>(a.x) + r * a.x_sr + col + j * dc, a.dcs ? on : 0);
    };
    extern __shared__ __align__(128) unsigned char ring_smem[];
    Ring<4> ring;
    int st = 0;  // the row's stage, and its phase
    uint32_t phase = 0;
    auto refill = [&](int stage, int64_t row) {
        const void *const src[4] = {static_cast<const R *>(a.res_out) + row * a.ro_sr, static_cast<const T *>(a.dy) + row * a.y_sr,
                                     static_cast<const R *>(a.dres_out) + row * a.res_sr, static_cast<const T *>(a.x) + row * a.x_sr};
        ring.issue(stage, src);
    };
    if constexpr (RING) {
        ring.bytes[0] = pl.W * (uint32_t)sizeof(R);
        ring.bytes[1] = pl.W * (uint32_t)sizeof(T);
        ring.bytes[2] = a.dres_out ? ring.bytes[0] : 0u;
        ring.bytes[3] = a.dcs ? ring.bytes[1] : 0u;
        ring.init(ring_smem, pl.stages);
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < pl.stages; ++i)
                if (blockIdx.x + i * dr < a.rows) refill(i, blockIdx.x + i * dr);
    }
    int64_t r = (int64_t)blockIdx.x * pl.ty + p.ty;
    if constexpr (kAh)
#pragma unroll
        for (int j = 0; j < NV; ++j) fetch(r, j, rh[j], ry[j], rd[j], rx[j]);
    for (int64_t r0 = (int64_t)blockIdx.x * pl.ty; r0 < a.rows; r0 += dr, r += dr) {
        float s[2] = {0.0f, 0.0f};
        if constexpr (RING) ring.wait(st, phase, a.status);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (RING) {
                const int on = r < a.rows ? in[j] : 0;
                const uint32_t at = (p.c0 + j * dc) * (uint32_t)sizeof(T), ar = (p.c0 + j * dc) * (uint32_t)sizeof(R);
                rh[j].load_shared(ring.row(st, 0) + ar, on);
                ry[j].load_shared(ring.row(st, 1) + at, on);
                rd[j].load_shared(ring.row(st, 2) + ar, a.dres_out ? on : 0);
                rx[j].load_shared(ring.row(st, 3) + at, a.dcs ? on : 0);
            } else if constexpr (kAh) {
                fetch(r + dr, j, nh[j], ny[j], nd[j], nx[j]);
            } else {
                fetch(r, j, rh[j], ry[j], rd[j], rx[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float h[VEC], y[VEC], w[VEC];
            rh[j].get(h);
            ry[j].get(y);
            weights_of(a.w, hw, j, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[0] = fmaf(h[i], h[i], s[0]);
                s[1] = fmaf(y[i] * w[i], h[i], s[1]);
            }
        }
        group_sum<2>(s, pl.tpr, sm, turn);
        if constexpr (RING) {
            // every thread has read the row: its place is the next one's
            if (threadIdx.x == 0 && r + pl.stages * dr < a.rows) refill(st, r + pl.stages * dr);
            if (++st == pl.stages) st = 0, ++phase;
        }
        const float inv = rsqrtf(fmaf(s[0], invW, a.eps));
        const float k = inv * inv * s[1] * invW;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float h[VEC], y[VEC], w[VEC], d[VEC], x[VEC], c[VEC];
            rh[j].get(h);
            ry[j].get(y);
            rd[j].get(d);
            rx[j].get(x);
            weights_of(a.w, hw, j, w);
            weights_of(a.cs, hc, j, c);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                d[i] += inv * fmaf(-k, h[i], y[i] * w[i]);
                dw[j][i] = fmaf(y[i], h[i] * inv, dw[j][i]);
                dch[j][i] = fmaf(a.scale * d[i], x[i], dch[j][i]);
            }
            if (in[j] && r < a.rows) {
                if (a.dres) store_vec<R, VEC, ODD>(static_cast<R *>(a.dres) + r * a.width + col + j * dc, d, in[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[i] *= a.scale * c[i];
                if (a.dx) store_vec<T, VEC, ODD>(static_cast<T *>(a.dx) + r * a.width + col + j * dc, d, in[j]);
            }
            if constexpr (kAh) rh[j] = nh[j], ry[j] = ny[j], rd[j] = nd[j], rx[j] = nx[j];
        }
    }
    const int64_t prow = (int64_t)blockIdx.x * pl.ty + p.ty, parts = (int64_t)gridDim.x * pl.ty;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        if (a.dw) store_vec<float, VEC, ODD>(a.part + prow * a.width + col + j * dc, dw[j], in[j]);
        if (a.dcs) store_vec<float, VEC, ODD>(a.part + (parts + prow) * a.width + col + j * dc, dch[j], in[j]);
    }
}

// out[c] = sum over the rows of part: each thread its own rows in order, then the threads
// of a column in order. Latency bounds it: 1024 threads share CW columns.
constexpr int kSumThr = 1024;
template <int CW>
__global__ void __launch_bounds__(kSumThr) norm_sum_kernel(const float *part, float *out0, float *out1, int64_t parts,
                                                           int64_t width) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
    constexpr int TY = kSumThr / CW, T2 = 16;
    __shared__ float sm[TY][CW + 1];
    const int tx = threadIdx.x % CW, ty = threadIdx.x / CW;
    const int64_t c = (int64_t)blockIdx.x * CW + tx;
    float *out = blockIdx.y ? out1 : out0;
    if (out == nullptr) return;
    const float *src = part + (int64_t)blockIdx.y * parts * width;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 8
        for (int64_t r = ty; r < parts; r += TY) s += src[r * width + c];
    }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty < T2) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < TY / T2; ++i) s += sm[ty * (TY / T2) + i][tx];
    }
    __syncthreads();
    if (ty < T2) sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < width) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < T2; ++i) s += sm[i][tx];
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

// Vectors per thread: the fewest that keep a group within a block (16384 columns in fours: 8). Rows that
// come column by column take smaller blocks, more of which have a row on its way, in the backward and where
// a thread has two vectors in any case (8000 rows, bf16: residual backward, 1503 columns 68 us, 119 us with
// 384 threads; gated forward, 4001 columns 114 and 135; but residual forward, 1503 columns 51 and 46).
int vectors_for(int64_t W, int vec, bool odd, bool bwd) {
    int nv = 1;
    while (nv < 8 && threads_for(W, vec, nv) > (odd && (bwd || nv > 1) ? kMaxThr / 2 : kMaxThr)) nv *= 2;
    return nv;
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
    // as many blocks as run at a time (the backward leaves a row of partial sums per block and ty)
    const int64_t thr = (int64_t)pl.tpr * pl.gb * pl.ty;
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(2048 / thr, 65536 / (regs_of(nv, bwd) * thr)));
    const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms * per_sm / pl.gblocks);
    pl.rblocks = (int)std::max<int64_t>(1, std::min(rb, cap));
    return pl;
}

// A ring of rows pays where a block works down several of them and a group fills more than
// a warp; its blocks share the SM's shared memory.
constexpr int kMaxSmem = 220 * 1024;
void add_ring(NormPlan &pl, int64_t rows, bool odd, size_t row_bytes, int num_sms) {
    if (odd || pl.tpr <= 32 || rows < 3 * (int64_t)pl.rblocks) return;
    const int64_t per_sm = std::max<int64_t>(1, ((int64_t)pl.rblocks * pl.gblocks + num_sms - 1) / num_sms);
    const int64_t n = (kMaxSmem / per_sm - 1024 - 128) / (int64_t)row_bytes;
    pl.stages = (int)std::min<int64_t>(n, 8);
    if (pl.stages < 2) pl.stages = 0;
}

bool vec16(const void *p, int64_t sr, int es) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (sr * es) % 16 == 0);
}

template <typename K, typename A>
cudaError_t launch(K kernel, const A &a, const NormPlan &pl, size_t row_bytes, SmemOptIn &opt_in, cudaStream_t st) {
    const size_t smem = pl.stages ? 128 + pl.stages * row_bytes : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = opt_in.ensure(reinterpret_cast<const void *>(kernel), kMaxSmem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<dim3((unsigned)pl.rblocks, (unsigned)pl.gblocks), (unsigned)(pl.tpr * pl.gb * pl.ty), smem, st>>>(a, pl);
    return cudaGetLastError();
}
template <int NV, typename T, int VEC, int GATE, bool ODD>
cudaError_t run_gate(const GatedNormArgs &a, const NormPlan &pl, size_t row_bytes, bool bwd, cudaStream_t st) {
    static SmemOptIn opt_in[2];
    if constexpr (!ODD)
        if (pl.stages)
            return bwd ? launch(gated_norm_bwd_kernel<T, VEC, NV, kRing, GATE>, a, pl, row_bytes, opt_in[1], st)
                       : launch(gated_norm_fwd_kernel<T, VEC, NV, kRing, GATE>, a, pl, row_bytes, opt_in[0], st);
    constexpr int ROWS = ODD ? kOdd : kStraight;
    return bwd ? launch(gated_norm_bwd_kernel<T, VEC, NV, ROWS, GATE>, a, pl, 0, opt_in[1], st)
               : launch(gated_norm_fwd_kernel<T, VEC, NV, ROWS, GATE>, a, pl, 0, opt_in[0], st);
}
template <int NV, typename T, int VEC, bool ODD>
cudaError_t run_gated(const GatedNormArgs &a, const NormPlan &pl, size_t row_bytes, bool bwd, cudaStream_t st) {
    if (!a.z) return run_gate<NV, T, VEC, kNoGate, ODD>(a, pl, row_bytes, bwd, st);
    return a.gate_first ? run_gate<NV, T, VEC, kGateFirst, ODD>(a, pl, row_bytes, bwd, st)
                        : run_gate<NV, T, VEC, kGateBehind, ODD>(a, pl, row_bytes, bwd, st);
}
template <int NV, typename T, typename R, int VEC, bool ODD>
cudaError_t run_residual(const ResidualNormArgs &a, const NormPlan &pl, size_t row_bytes, bool bwd, cudaStream_t st) {
    static SmemOptIn opt_in[2];
    if constexpr (!ODD)
        if (pl.stages)
            return bwd ? launch(residual_norm_bwd_kernel<T, R, VEC, NV, kRing>, a, pl, row_bytes, opt_in[1], st)
                       : launch(residual_norm_fwd_kernel<T, R, VEC, NV, kRing>, a, pl, row_bytes, opt_in[0], st);
    constexpr int ROWS = ODD ? kOdd : kStraight;
    return bwd ? launch(residual_norm_bwd_kernel<T, R, VEC, NV, ROWS>, a, pl, 0, opt_in[1], st)
               : launch(residual_norm_fwd_kernel<T, R, VEC, NV, ROWS>, a, pl, 0, opt_in[0], st);
}

cudaError_t sum_parts(const float *part, float *o0, float *o1, const NormPlan &pl, int64_t width, int num_sms, cudaStream_t st) {
    if (!o0 && !o1) return cudaSuccess;
    const int64_t parts = (int64_t)pl.rblocks * pl.ty;
    // 8 columns a block where blocks of 32 would leave SMs idle
    const int cw = (width + 31) / 32 * (o1 ? 2 : 1) < num_sms ? 8 : 32;
    // its blocks may take their places while the rows' last blocks run
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((width + cw - 1) / cw), o1 ? 2u : 1u);
    cfg.blockDim = dim3(kSumThr);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cw == 8 ? norm_sum_kernel<8> : norm_sum_kernel<32>, part, o0, o1, parts, width);
}

// Vector widths: 8 columns where an array is bf16, 4 where all are fp32, and 4 column by
// column for rows that do not allow 16-byte accesses (6190 rows of 398 columns, bf16 and
// fp32, backward: 21 us, 56 us with one column a thread, whose addresses were most of its work).
template <typename F>
cudaError_t with_nv(int nv, F f) {
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

}  // namespace

// Rows of partial sums that a backward of these sizes can need, for any vector width.
size_t norm_parts(int64_t rows, int64_t width, int64_t groups, int num_sms) {
    size_t most = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t W = width / groups;
        const int vec = i == 0 ? 8 : 4;
        const NormPlan pl = plan_norm(rows, W, groups, vec, vectors_for(W, vec, i == 2, true), num_sms, true);
        most = std::max(most, (size_t)pl.rblocks * (size_t)pl.ty);
    }
    return most;
}

cudaError_t launch_gated_norm(const GatedNormArgs &a, bool bf16, bool bwd, int num_sms, cudaStream_t stream) {
    const int64_t W = a.width / a.groups;
    const int es = bf16 ? 2 : 4, v = bf16 ? 8 : 4;
    const bool ok = W % v == 0 && vec16(a.x, a.x_sr, es) && vec16(a.z, a.z_sr, es) && vec16(a.y, a.y_sr, es) &&
                    vec16(a.dy, a.y_sr, es) && vec16(a.dx, a.width, es) && vec16(a.dz, a.width, es) && vec16(a.w, 0, 4);
    const int vec = ok ? v : 4, nv = vectors_for(W, vec, !ok, bwd);
    NormPlan pl = plan_norm(a.rows, W, a.groups, vec, nv, num_sms, bwd);
    const size_t rb = (size_t)W * es * ((bwd ? 2 : 1) + (a.z ? 1 : 0));
    add_ring(pl, a.rows, !ok, rb, num_sms);
    cudaError_t e = with_nv(nv, [&](auto n) -> cudaError_t {
        constexpr int NV = decltype(n)::value;
        if (!ok)
            return bf16 ? run_gated<NV, __nv_bfloat16, 4, true>(a, pl, rb, bwd, stream)
                        : run_gated<NV, float, 4, true>(a, pl, rb, bwd, stream);
        if (!bf16) return run_gated<NV, float, 4, false>(a, pl, rb, bwd, stream);
        if constexpr (NV <= 4) return run_gated<NV, __nv_bfloat16, 8, false>(a, pl, rb, bwd, stream);
        return cudaErrorInvalidConfiguration;
    });
    if (e == cudaSuccess && bwd) e = sum_parts(a.part, a.dw, nullptr, pl, a.width, num_sms, stream);
    return e;
}

cudaError_t launch_residual_norm(const ResidualNormArgs &a, bool bf16, bool res_bf16, bool bwd, int num_sms,
                                 cudaStream_t stream) {
    const int64_t W = a.width;
    const int es = bf16 ? 2 : 4, rs = res_bf16 ? 2 : 4, v = bf16 || res_bf16 ? 8 : 4;
    const bool ok = W % v == 0 && vec16(a.x, a.x_sr, es) && vec16(a.res, a.res_sr, rs) && vec16(a.y, a.y_sr, es) &&
                    vec16(a.dy, a.y_sr, es) && vec16(a.res_out, a.ro_sr, rs) && vec16(a.dres_out, a.res_sr, rs) &&
                    vec16(a.dx, a.width, es) && vec16(a.dres, a.width, rs) && vec16(a.w, 0, 4) && vec16(a.cs, 0, 4);
    const int vec = ok ? v : 4, nv = vectors_for(W, vec, !ok, bwd);
    NormPlan pl = plan_norm(a.rows, W, 1, vec, nv, num_sms, bwd);
    const size_t rb = (size_t)W * (bwd ? rs * (a.dres_out ? 2 : 1) + es * (a.dcs ? 2 : 1) : es + (a.res ? rs : 0));
    add_ring(pl, a.rows, !ok, rb, num_sms);
    cudaError_t e = with_nv(nv, [&](auto n) -> cudaError_t {
        constexpr int NV = decltype(n)::value;
        if (!ok) {
            if (bf16)
                return res_bf16 ? run_residual<NV, __nv_bfloat16, __nv_bfloat16, 4, true>(a, pl, rb, bwd, stream)
                                : run_residual<NV, __nv_bfloat16, float, 4, true>(a, pl, rb, bwd, stream);
            return res_bf16 ? run_residual<NV, float, __nv_bfloat16, 4, true>(a, pl, rb, bwd, stream)
                            : run_residual<NV, float, float, 4, true>(a, pl, rb, bwd, stream);
        }
        if (vec == 4) return run_residual<NV, float, float, 4, false>(a, pl, rb, bwd, stream);
        if constexpr (NV <= 4) {
            if (bf16)
                return res_bf16 ? run_residual<NV, __nv_bfloat16, __nv_bfloat16, 8, false>(a, pl, rb, bwd, stream)
                                : run_residual<NV, __nv_bfloat16, float, 8, false>(a, pl, rb, bwd, stream);
            return run_residual<NV, float, __nv_bfloat16, 8, false>(a, pl, rb, bwd, stream);
        }
        return cudaErrorInvalidConfiguration;
    });
    if (e == cudaSuccess && bwd) e = sum_parts(a.part, a.dw, a.dcs, pl, a.width, num_sms, stream);
    return e;
}

}  // namespace ms

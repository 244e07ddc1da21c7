// linattn_plain.cu -- linear attention with a decay per head as the plain
// recurrence, the sum of shared heads' gradients, and the one-token update.

#include <cstdint>

#include "mambascan.h"
#include "ms_device.cuh"
#include "ms_internal.h"

namespace ms {

namespace {

// lam S + c as keep S + (part S + c). For lam >= 1/2 keep = 1 and part = lam - 1, which
// keeps the bits of a slow decay: lam itself rounded to fp32 is up to 2^-25 off, which
// 4096 remembered tokens would make 2^-13 of the state. Below, keep = 0 and part = lam,
// so that what is forgotten leaves no rounding behind.
struct Decay {
    float keep, part;
};
__device__ __forceinline__ Decay decay_of(float log_decay) {
    const float m = expm1f(log_decay);
    return m >= -0.5f ? Decay{1.0f, m} : Decay{0.0f, expf(log_decay)};
}
__device__ __forceinline__ float decayed(float s, const Decay &d, float c) {
    return fmaf(d.keep, s, fmaf(d.part, s, c));
}

constexpr int kPT = 16;    // tokens staged at a time
constexpr int kPThr = 128; // one thread per column of the state

// The tokens of sequence i: offset of its first row inside the arrays (packed)
// and its length; false where the caller's offsets are not in order.
__device__ __forceinline__ bool seq_rows(const int32_t *seq_start, int64_t total, int64_t seqlen, int64_t i,
                                         int64_t &row0, int64_t &len) {
    if (seq_start == nullptr) {
        row0 = 0;
        len = seqlen;
        return true;
    }
    const int64_t s = seq_start[i], e = seq_start[i + 1];
    row0 = s;
    len = e - s;
    return s >= 0 && e >= s && e <= total;
}

// One CTA per (sequence, head, problem); thread e holds column e of the state,
// all dx rows of it, in registers. Per token 3 dx multiply-adds a thread: the
// FMA pipe bounds it. It serves the sizes, types and alignments that the
// tensor-core kernel does not take.
template <typename T, int DX>
__global__ void __launch_bounds__(kPThr) linattn_plain_kernel(const LaArgs a) {
    const LaProblem &p = a.p[blockIdx.y];
    const int64_t b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int e = threadIdx.x;
    __shared__ __align__(16) float xs[kPT][DX], ys[kPT][DX];
    int64_t row0, len;
    if (!seq_rows(a.seq_start, a.total, a.seqlen, b, row0, len)) {
        if (e == 0 && a.status) atomicOr(a.status, MS_ERR_SHAPE);
        return;
    }
    const int64_t bs = a.seq_start ? 0 : b;
    const T *x = static_cast<const T *>(p.x) + bs * p.x_sb + row0 * p.x_sl + (h / p.xg) * p.x_sh;
    const T *y = static_cast<const T *>(p.y) + bs * p.y_sb + row0 * p.y_sl + (h / p.yg) * p.y_sh;
    const T *z = static_cast<const T *>(p.z) + bs * p.z_sb + row0 * p.z_sl + (h / p.zg) * p.z_sh;
    const int64_t o0 = bs * p.o_sb + row0 * p.o_sl + h * p.o_sh;
    const Decay lam = decay_of(__ldg(a.log_decay + h));
    const bool live = e < p.dz;
    float S[DX];
    const float *s0 = p.s0 ? p.s0 + (b * a.H + h) * p.dx * p.dz : nullptr;
#pragma unroll
    for (int i = 0; i < DX; ++i) S[i] = (s0 && live && i < p.dx) ? s0[i * p.s0_sr + e * p.s0_sc] : 0.0f;
    for (int64_t c = 0; c < len; c += kPT) {
        const int n = (int)(len - c < kPT ? len - c : kPT);
        __syncthreads();
        for (int i = e; i < kPT * DX; i += kPThr) {
            const int t = i / DX, d = i % DX;
            const bool in = t < n && d < p.dx;
            const int64_t tok = p.rev ? len - 1 - c - t : c + t;
            xs[t][d] = in ? Elem<T>::load(x + tok * p.x_sl + d) : 0.0f;
            ys[t][d] = in ? Elem<T>::load(y + tok * p.y_sl + d) : 0.0f;
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            const int64_t tok = p.rev ? len - 1 - c - t : c + t;
            const float zt = live ? p.ws * Elem<T>::load(z + tok * p.z_sl + e) : 0.0f;
            // forward order decays before the token, reverse order after it (here: before the
            // next one, and once more at the end)
            const Decay pre = (p.rev && c + t == 0) ? Decay{1.0f, 0.0f} : lam;
            float acc = 0.0f;
#pragma unroll
            for (int i = 0; i < DX; ++i) {
                S[i] = decayed(S[i], pre, ys[t][i] * zt);
                acc = fmaf(xs[t][i], S[i], acc);
            }
            if (live && MS_CHECK(a.status, tok >= 0 && row0 + tok < (a.seq_start ? a.total : a.seqlen) && b < a.batch)) {
                const int64_t at = o0 + tok * p.o_sl + e;
                if (p.o_f32) static_cast<float *>(p.o)[at] = p.ro * acc;
                else Elem<T>::store(static_cast<T *>(p.o) + at, p.ro * acc);
            }
        }
    }
    if (p.fin && live) {
        float *f = p.fin + (b * a.H + h) * p.dx * p.dz + e;
        const Decay post = (p.rev && len > 0) ? lam : Decay{1.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < DX; ++i)
            if (i < p.dx) f[(int64_t)i * p.dz] = decayed(S[i], post, 0.0f);
    }
}

template <typename T>
cudaError_t launch_plain_t(const LaArgs &a, cudaStream_t stream) {
    int dx = 1;
    for (int i = 0; i < a.np; ++i) dx = a.p[i].dx > dx ? a.p[i].dx : dx;
    const int64_t blocks = a.batch * a.H;
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks, (unsigned)a.np);
    if (dx <= 32) linattn_plain_kernel<T, 32><<<grid, kPThr, 0, stream>>>(a);
    else if (dx <= 64) linattn_plain_kernel<T, 64><<<grid, kPThr, 0, stream>>>(a);
    else linattn_plain_kernel<T, 128><<<grid, kPThr, 0, stream>>>(a);
    return cudaGetLastError();
}

// out[row][g][i] = sum of part[row][h][i] over the heads h of g, in their order, for
// two arrays (blockIdx.y). HBM bounds it: a thread has VEC neighbouring columns of a
// row (16 bytes of part), a block whole rows, and all heads' loads are on their way
// together (4001 x 2 rows of 16 heads for 4, 128 and 96 columns: 28 us, 67 us with
// one column a thread and a launch for each array).
template <typename T, int VEC>
__global__ void __launch_bounds__(256) linattn_reduce_kernel(const LaReduceArgs a0, const LaReduceArgs a1) {
    const LaReduceArgs &a = blockIdx.y ? a1 : a0;
    const int per = (int)(a.kv * a.d) / VEC, n = (int)(a.H / a.kv), dv = (int)a.d / VEC;
    const int tpr = per < 256 ? per : 256, rpb = 256 / tpr;
    const int x = threadIdx.x % tpr, y = threadIdx.x / tpr;
    if (y >= rpb) return;
    int64_t first = 0, rows = a.batch * a.seqlen;
    if (a.seq_start) {
        // the rows of the sequences that lie in [0, total]: offsets do not decrease
        int64_t lo = 0, hi = a.batch;
        while (lo < hi && a.seq_start[lo] < 0) ++lo;
        while (hi > lo && a.seq_start[hi] > a.total) --hi;
        first = lo < hi ? a.seq_start[lo] : 0;
        rows = lo < hi ? a.seq_start[hi] - first : 0;
    }
    for (int64_t r = (int64_t)blockIdx.x * rpb + y; r < rows; r += (int64_t)gridDim.x * rpb) {
        const int64_t row = first + r;
        if (!MS_CHECK(a.status, row >= 0 && row < (a.seq_start ? a.total : a.batch * a.seqlen))) break;
        const int64_t b = a.seq_start ? 0 : row / a.seqlen, t = a.seq_start ? row : row - b * a.seqlen;
        T *out = static_cast<T *>(a.out) + b * a.o_sb + t * a.o_sl;
        const float *part = a.part + row * a.H * a.d;
        for (int i = x; i < per; i += tpr) {
            const int g = i / dv, c = (i - g * dv) * VEC;
            const float *src = part + (int64_t)g * n * a.d + c;
            float s[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[j] = 0.0f;
#pragma unroll 4
            for (int k = 0; k < n; ++k) {
                if constexpr (VEC == 4) {
                    const float4 v = __ldcs(reinterpret_cast<const float4 *>(src + k * a.d));
                    s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
                } else {
                    s[0] += src[k * a.d];
                }
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) Elem<T>::store(out + g * a.o_sh + c + j, s[j]);
        }
    }
}

// ------------------------------------------------------------ one token ----

constexpr int kUThr = 256;
constexpr int kURows = 8;   // rows of the state that a thread has on their way
constexpr int kUDk = 256;   // rows whose k and q wait in shared memory at a time

// S = lam S + k v^T and o = a q S for one (row, head): the state is read and
// written once, which bounds it (HBM). A thread owns VEC neighbouring columns
// and every rp-th row; its state is on its way before anything else is read,
// k and q go through shared memory, and the column sums of q S meet there.
// Back-to-back steps overlap through programmatic dependent launch. 64 x 80
// heads of 128 x 64: 62 us, 5.5 TB/s (107 us with k and q read beside the state).
template <typename T, int VEC>
__global__ void __launch_bounds__(kUThr) linattn_update_kernel(const LaUpdateArgs a, int cg) {
    // the next grid may be scheduled; what the previous one wrote is waited for before any read
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t b = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / (a.H / a.kv);
    const int col = threadIdx.x % cg, r0 = threadIdx.x / cg, rp = kUThr / cg;
    const int e0 = col * VEC;
    __shared__ __align__(16) float red[kUThr * VEC], ks[kUDk], qs[kUDk];
    const T *q = static_cast<const T *>(a.q) + b * a.q_sb + h * a.q_sh;
    const T *k = static_cast<const T *>(a.k) + b * a.k_sb + g * a.k_sh;
    const T *v = static_cast<const T *>(a.v) + b * a.v_sb + g * a.v_sh;
    float *st = a.state + b * a.st_sb + h * a.st_sh + e0;
    const bool live = e0 < a.dv && MS_CHECK(a.status, b < a.batch && e0 + VEC <= a.dv);
    float s[kURows][VEC], acc[VEC], vv[VEC];
    auto fetch = [&](int i0, int end) {
#pragma unroll
        for (int u = 0; u < kURows; ++u) {
            const int i = i0 + u * rp;
            if (live && i < end) {
                if constexpr (VEC == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(st + (int64_t)i * a.dv);
                    s[u][0] = t.x; s[u][1] = t.y; s[u][2] = t.z; s[u][3] = t.w;
                } else {
                    s[u][0] = st[(int64_t)i * a.dv];
                }
            }
        }
    };
    fetch(r0, a.dk < kUDk ? a.dk : kUDk);
    const Decay lam = decay_of(__ldg(a.log_decay + h));
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        acc[j] = 0.0f;
        vv[j] = live ? Elem<T>::load(v + e0 + j) : 0.0f;
    }
    for (int d0 = 0; d0 < a.dk; d0 += kUDk) {
        if (d0) __syncthreads();
        if (d0 + (int)threadIdx.x < a.dk) {
            ks[threadIdx.x] = Elem<T>::load(k + d0 + threadIdx.x);
            qs[threadIdx.x] = Elem<T>::load(q + d0 + threadIdx.x);
        }
        __syncthreads();
        const int end = a.dk < d0 + kUDk ? a.dk : d0 + kUDk;
        for (int i0 = d0 + r0; i0 < end; i0 += rp * kURows) {  // (rp divides kUDk)
            if (i0 != r0) fetch(i0, end);
#pragma unroll
            for (int u = 0; u < kURows; ++u) {
                const int i = i0 + u * rp;
                if (live && i < end) {
                    const float kk = ks[i - d0], qq = qs[i - d0];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        s[u][j] = decayed(s[u][j], lam, kk * vv[j]);
                        acc[j] = fmaf(qq, s[u][j], acc[j]);
                    }
                    if constexpr (VEC == 4)
                        *reinterpret_cast<float4 *>(st + (int64_t)i * a.dv) = make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
                    else
                        st[(int64_t)i * a.dv] = s[u][0];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[r0 * cg * VEC + e0 + j] = acc[j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.dv; e += kUThr) {
        float t = 0.0f;
        for (int r = 0; r < rp; ++r) t += red[r * cg * VEC + e];
        Elem<T>::store(static_cast<T *>(a.o) + b * a.o_sb + h * a.o_sh + e, a.scale * t);
    }
}

template <typename T>
cudaError_t launch_update_t(const LaUpdateArgs &a, cudaStream_t stream) {
    const int64_t blocks = a.batch * a.H;
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 && a.st_sb % 4 == 0 && a.st_sh % 4 == 0;
    const int cols = vec ? a.dv / 4 : a.dv;
    int cg = 1;
    while (cg < cols) cg *= 2;
    if (cg > kUThr) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kUThr);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&cfg, linattn_update_kernel<T, 4>, a, cg)
               : cudaLaunchKernelEx(&cfg, linattn_update_kernel<T, 1>, a, cg);
}

}  // namespace

cudaError_t launch_linattn_plain(const LaArgs &a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_plain_t<__nv_bfloat16>(a, stream) : launch_plain_t<float>(a, stream);
}

cudaError_t launch_linattn_reduce(const LaReduceArgs &a, const LaReduceArgs &b, bool bf16, cudaStream_t stream) {
    const int64_t rows = a.seq_start ? a.total : a.batch * a.seqlen;
    if (rows <= 0) return cudaSuccess;
    const dim3 grid((unsigned)(rows < 148 * 8 ? rows : 148 * 8), 2u);
    const bool vec = a.d % 4 == 0 && b.d % 4 == 0 && reinterpret_cast<uintptr_t>(a.part) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(b.part) % 16 == 0;
    if (bf16) {
        if (vec) linattn_reduce_kernel<__nv_bfloat16, 4><<<grid, 256, 0, stream>>>(a, b);
        else linattn_reduce_kernel<__nv_bfloat16, 1><<<grid, 256, 0, stream>>>(a, b);
    } else {
        if (vec) linattn_reduce_kernel<float, 4><<<grid, 256, 0, stream>>>(a, b);
        else linattn_reduce_kernel<float, 1><<<grid, 256, 0, stream>>>(a, b);
    }
    return cudaGetLastError();
}

cudaError_t launch_linattn_update(const LaUpdateArgs &a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_update_t<__nv_bfloat16>(a, stream) : launch_update_t<float>(a, stream);
}

}  // namespace ms

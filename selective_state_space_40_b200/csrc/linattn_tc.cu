// linattn_tc.cu -- linear attention with a decay per head on the sm_100a tensor
// cores (tcgen05, accumulators in tensor memory), in chunks of 128 tokens.
//
// Forward and gradients are one map of three token arrays (see LaProblem): with
// lam the decay, S the state entering a chunk of n tokens, t, s = 0..n-1,
//   o_t   = ro lam^(t+1) x_t S + ps sum_{s<=t} lam^(t-s) (x_t . y_s) z_s
//   S_out = lam^n S + ws sum_s lam^(n-1-s) y_s z_s^T
// and, for the gradients that run from the last token to the first,
//   o_t   = ro lam^(n-1-t) x_t R + ps sum_{s>=t} lam^(s-t) (x_t . y_s) z_s
//   R_out = lam^n R + ws sum_s lam^(s+1) y_s z_s^T.
// Four products per chunk, each M = 128 (bf16 operands, fp32 accumulators):
//   QK [128 x 128] = X Y^T              O_a [128 x 64] = P Z
//   KV [dx  x  64] = Y^T Z'             O_b [128 x 64] = X S
// P = QK weighted and rounded to bf16 (as its product's operand has to be: one
// rounding of each score, the size of the rounding of o itself); Z' = weighted
// rows of Z as the sum of three bf16 parts, all 24 bits of it, since the state
// is handed on for as long as lam remembers; S rounded to bf16 where X reads
// it, never where it is kept.
//
// A CTA owns one (segment of a sequence, head, 64 columns of z) and walks its
// chunks with the state in registers. What bounds it is shared memory: a chunk
// moves some 370 KB of it at dx = 128 (operands of the products 208, tensor
// copies 80, Z' 64, S 16), 2900 clocks at 128 bytes a clock, so KV takes the three
// parts of Z' as one product of N = 192 (24 products of N = 64 read Y three times,
// and took 1900 clocks a chunk against 800). The roles run on different chunks at
// the same time, each warp waiting for its own inputs only:
//   one warp loads (tensor copies, 128-byte swizzle, NS stages); one warp each
//   issues QK, KV, and O_a with O_b;
//   group P  weights QK into P (tensor memory, in place);
//   group E  adds up O_a and lam^.. O_b and writes o;
//   group V  forms Z', and clears the rows of a chunk's Y and Z that are behind
//            the sequence;
//   group S  keeps S (a thread: one row, or half of one), adds KV, and hands
//            its bf16 form to the next chunk's O_b.
//
// Where sequences times heads leave SMs idle, sequences are cut into segments:
// a first pass (kStates) forms each segment's own state from zero, a second
// chains them, and the main pass starts every segment from its true state.
// Every wait is bounded: a timeout sets MS_ERR_TIMEOUT and ends the CTA.

#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "mambascan.h"
#include "ms_device.cuh"
#include "ms_internal.h"

namespace ms {

namespace {

constexpr int kC = 128;   // tokens per chunk
constexpr int kZ = 64;    // columns of z per CTA
constexpr int kThreads = 640;
constexpr int kLoadWarp = 16, kQkWarp = 17, kKvWarp = 18, kOWarp = 19;  // groups P, V, S, E: warps 0-3, 4-7, 8-11, 12-15
constexpr uint32_t kSpinTries = 1u << 20;

// tensor memory: two buffers of QK (P takes its first 64 columns, O_a its last
// 64), O_b, and the three parts of KV
__host__ __device__ constexpr uint32_t col_qk(int b) { return 128u * b; }
__host__ __device__ constexpr uint32_t col_oa(int b) { return 128u * b + 64u; }
constexpr uint32_t kColOb = 256, kColKv = 320;

struct TcProblem {
    int mx, my, mz;  // tensor maps of x, y, z
    int xg, yg, zg, dx, dz, rev, o_f32;
    float ws, ps, ro;
    const float *s0;  // entering states: block (sequence or slot, head) of dx * dz, element (i, j) at i s0_sr + j s0_sc
    float *fin;       // leaving states [batch, H, dx, dz], or (kStates) [slots, H, dx, dz]
    int64_t s0_sr, s0_sc;
    int s0_slot;
    void *o;
    int64_t o_sb, o_sl, o_sh;
    int nzb;          // blocks of kZ columns of z
};
struct TcArgs {
    const float *log_decay;
    const int32_t *seq_start;
    int *status;
    int batch, seqlen, total, H;
    int seg;   // tokens per segment (a multiple of kC)
    int nseg;  // segments per sequence (dense); slots of the packed case are numbered below
    int segmented;
    int np, units;  // units: sum of nzb
    TcProblem p[kLaMaxProblems];
};
struct TcMaps {
    CUtensorMap m[4];
};

// shared memory (bytes)
template <int DX, bool kStates>
struct Smem {
    static constexpr int kX = kStates ? 0 : kC * DX * 2;
    static constexpr int kY = kC * DX * 2;
    static constexpr int kZb = kC * kZ * 2;
    static constexpr int kStage = kX + kY + kZb;
    static constexpr int kStages = DX == 64 ? 3 : 2;
    static constexpr int oZs = kStages * kStage;             // three parts of Z'
    static constexpr int oS = oZs + 3 * kZb;                 // S in bf16
    static constexpr int oPw = oS + (kStates ? 0 : DX * kZ * 2);  // lam^n, n = 0..128
    static constexpr int oPs = oPw + (132 + 32) * 4;         // ps lam^n, behind 32 zeros
    static constexpr int oCf = oPs + 132 * 4;                // lam^(31-c), in reverse lam^c, c < 32
    static constexpr int oBar = oCf + 32 * 4;
    static constexpr int kBytes = oBar + 8 * 26 + 16;
};
enum {
    kBarFull = 0,    // [3] a stage's tiles are in
    kBarFree = 3,    // [3] every product reading the stage is done
    kBarQK = 6,      // [2] QK is done
    kBarP = 8,       // [2] P is in tensor memory
    kBarO = 10,      // [2] O_a and O_b are done
    kBarOFree = 12,  // [2] group E has read O_a (and O_b)
    kBarZs = 14,     // [2] Z' of 64 tokens is in shared memory
    kBarZsFree = 16, // [2] KV has read it
    kBarKV = 18,     // KV is done
    kBarKVFree = 19, // group S has read it
    kBarS = 20,      // S is in shared memory
    kBarOB = 21,     // O_b is done (and S read)
    kBarClear = 22,  // the rows behind the sequence are cleared (once, in the chunk that has some)
    kBarEnd = 23,    // [3] nothing of an issuing warp is in flight
    kNumBars = 26
};

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Shared-memory descriptors, 128-byte swizzle. The tiles are rows of 128 bytes
// (64 columns), 8 rows to a 1024-byte atom. K-major (the row is M or N): atoms
// 1024 bytes apart along the rows. M/N-major (the row is K): the stride offset
// steps 8 rows of K, the leading offset 64 columns of M or N.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// kind::f16, fp32 accumulator, bf16 operands, M = 128
constexpr uint32_t idesc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :
        : "r"(d), "l"(da), "l"(db), "r"(id), "r"(acc ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint64_t db, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :
        : "r"(d), "r"(ta), "l"(db), "r"(id), "r"(acc ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for phase `k` of a barrier; false when the CTA is stopping or the wait
// ran out. Only the first try is inlined: the roles' loops have to share the
// SM's instruction cache (see the kernel).
__device__ __noinline__ bool bar_wait_on(uint32_t bar, uint32_t k, volatile uint32_t *abort_flag, int *status) {
    for (uint32_t i = 0; i < kSpinTries; ++i) {
        if (bar_try(bar, k & 1u)) return true;
        if ((i & 63u) == 63u && *abort_flag != 0u) return false;
    }
    *abort_flag = 1u;
    if (status) atomicOr(status, MS_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t k, volatile uint32_t *abort_flag, int *status) {
    return bar_try(bar, k & 1u) || bar_wait_on(bar, k, abort_flag, status);
}
__device__ __forceinline__ void tma_load4(const CUtensorMap *map, uint32_t dst, uint32_t bar, int c0, int c1, int c2,
                                          int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 columns from each of two places, and 8 from each of three, waited for in the same statement
__device__ __forceinline__ void tmem_ld2x16(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(a[8]), "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]), "=f"(a[14]), "=f"(a[15]), "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(b[8]), "=f"(b[9]), "=f"(b[10]), "=f"(b[11]), "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15])
        : "r"(ta), "r"(tb)
        : "memory");
}
__device__ __forceinline__ void tmem_ld3x8(uint32_t ta, uint32_t tb, uint32_t tc, float (&a)[8], float (&b)[8], float (&c)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%25];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%26];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]), "=f"(c[4]), "=f"(c[5]), "=f"(c[6]), "=f"(c[7])
        : "r"(ta), "r"(tb), "r"(tc)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// v = hi + mid + lo in bf16 parts (24 significant bits), a pair at a time
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = pack2(a, b);
    a -= bf16_lo(hi);
    b -= bf16_hi(hi);
    mid = pack2(a, b);
    lo = pack2(a - bf16_lo(mid), b - bf16_hi(mid));
}

// The sequence and segment of a slot. Slot numbers: dense, sequence * nseg +
// segment; packed, floor(first row / seg) + sequence + segment, which gives each
// sequence as many numbers as it has segments or more. Every lane returns the same.
struct Place {
    int seq, g, row0, len, ng;
    bool ok, bad;  // a segment of the sequence; offsets out of order
};
__device__ __forceinline__ Place place_of(const TcArgs &a, int slot, int lane) {
    Place p{};
    int64_t len = a.seqlen;
    if (a.seq_start == nullptr) {
        p.seq = slot / a.nseg;
        p.g = slot % a.nseg;
    } else {
        p.seq = slot;
        if (a.segmented) {
            // the last sequence whose first slot is not behind this one
            int base = 0;
            p.seq = 0;
            for (int i0 = 0; i0 < a.batch; i0 += 32) {
                const int i = i0 + lane;
                const int bi = i < a.batch ? a.seq_start[i] / a.seg + i : INT_MAX;
                const unsigned m = __ballot_sync(0xffffffffu, bi <= slot);
                if (m == 0u) break;
                const int last = 31 - __clz(m);
                p.seq = i0 + last;
                base = __shfl_sync(0xffffffffu, bi, last);
            }
            p.g = slot - base;
        }
        const int64_t s = a.seq_start[p.seq], e = a.seq_start[p.seq + 1];
        p.row0 = (int)s;
        len = e - s;
        p.bad = !(s >= 0 && e >= s && e <= a.total);
    }
    p.len = p.bad ? 0 : (int)len;
    p.ng = p.len > a.seg ? (p.len + a.seg - 1) / a.seg : 1;
    p.ok = !p.bad && p.g >= 0 && p.g < p.ng;
    return p;
}

template <int DX, bool kStates>
__global__ void __launch_bounds__(kThreads, 1) linattn_tc_kernel(const __grid_constant__ TcArgs a,
                                                                 const __grid_constant__ TcMaps maps) {
    using M = Smem<DX, kStates>;
    constexpr int NS = M::kStages;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = saddr(smem);
    auto bar = [&](int i) { return sbase + (uint32_t)(M::oBar + 8 * i); };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + M::oBar + 8 * 26);
    volatile uint32_t *abort_flag = misc + 1;
    float *pw = reinterpret_cast<float *>(smem + M::oPw), *pwp = reinterpret_cast<float *>(smem + M::oPs);
    float *cfw = reinterpret_cast<float *>(smem + M::oCf);

    int unit = (int)(blockIdx.x % (unsigned)a.units);
    const int hs = (int)(blockIdx.x / (unsigned)a.units), h = hs % a.H, slot = hs / a.H;
    int pi = 0;
    while (unit >= a.p[pi].nzb) unit -= a.p[pi++].nzb;
    const TcProblem &p = a.p[pi];
    const int zb = unit;
    const Place pl = place_of(a, slot, lane);
    if (pl.bad && tid == 0 && a.status) atomicOr(a.status, MS_ERR_SHAPE);
    if (!pl.ok || (kStates && (p.rev ? pl.g == 0 : pl.g == pl.ng - 1))) return;
    const int seg0 = pl.g * a.seg;
    const int ntok = pl.len - seg0 < a.seg ? pl.len - seg0 : a.seg;
    const int nc = (ntok + kC - 1) / kC;
    const bool rev = p.rev != 0;
    // chunk c in the order of work: its first token, and how many it has
    auto first_of = [&](int c) { return seg0 + (rev ? nc - 1 - c : c) * kC; };
    auto count_of = [&](int c) {
        const int left = ntok - (rev ? nc - 1 - c : c) * kC;
        return left < kC ? left : kC;
    };

    const float g = fmaxf(__ldg(a.log_decay + h), -1e30f);  // -inf: 0 * -inf must be 0
    if (tid <= kC) {
        const float w = expf((float)tid * g);
        pw[tid] = w;
        pwp[tid] = p.ps * w;
        if (tid < 32) pwp[tid - 32] = 0.0f;
        if (tid < 32) cfw[p.rev ? tid : 31 - tid] = w;
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const bool warps4 = (i >= kBarP && i < kBarP + 2) || (i >= kBarOFree && i < kBarOFree + 2) ||
                                (i >= kBarZs && i < kBarZs + 2) || i == kBarKVFree || i == kBarS || i == kBarClear;
            const bool stage = i >= kBarFree && i < kBarFree + 3;  // QK, KV, O: each commits once
            bar_init(bar(i), warps4 ? 4 : (stage && !kStates) ? 3 : 1);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kQkWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(misc)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = misc[0];
    auto wait = [&](int i, int k) { return bar_wait(bar(i), (uint32_t)k, abort_flag, a.status); };
    auto wait_all = [&](int i, int k) { return __all_sync(0xffffffffu, wait(i, k)) != 0; };  // whole warps: one answer

    // every product that an issuing thread has in flight completes before the tensor memory is freed
    auto drain = [&](int i) {
        mma_commit(bar(kBarEnd + i));
        for (uint32_t k = 0; k < kSpinTries && !bar_try(bar(kBarEnd + i), 0u); ++k) {}
    };

    if (warp == kLoadWarp) {
        if (lane == 0) {
            const CUtensorMap *mx = &maps.m[p.mx], *my = &maps.m[p.my], *mz = &maps.m[p.mz];
            const int b = a.seq_start ? 0 : (int)pl.seq;
            const int hx = (int)(h / p.xg), hy = (int)(h / p.yg), hz = (int)(h / p.zg);
            int c = 0;
            for (; c < nc; ++c) {
                const int st = c % NS;
                if (c >= NS && !wait(kBarFree + st, c / NS - 1)) break;
                const uint32_t dst = sbase + (uint32_t)(st * M::kStage), br = bar(kBarFull + st);
                const int t = pl.row0 + first_of(c);
                bar_arrive_tx(br, (uint32_t)M::kStage);
#pragma unroll
                for (int i = 0; i < DX / 64; ++i) tma_load4(my, dst + M::kX + i * 16384, br, 64 * i, hy, t, b);
                tma_load4(mz, dst + M::kX + M::kY, br, kZ * zb, hz, t, b);
                if constexpr (!kStates) {
#pragma unroll
                    for (int i = 0; i < DX / 64; ++i) tma_load4(mx, dst + i * 16384, br, 64 * i, hx, t, b);
                }
            }
            // when stopping, the copies issued have landed before the CTA ends
            if (c < nc)
                for (int i = c > NS ? c - NS : 0; i < c; ++i)
                    for (uint32_t k = 0; k < kSpinTries && !bar_try(bar(kBarFull + i % NS), (uint32_t)(i / NS) & 1u); ++k) {}
        }
    } else if (warp == kQkWarp) {
        if constexpr (!kStates) {
            if (lane == 0) {
                const int ksteps = (p.dx + 15) >> 4;
                for (int c = 0; c < nc; ++c) {
                    const int b = c & 1, st = c % NS;
                    const uint32_t x = sbase + (uint32_t)(st * M::kStage), y = x + M::kX;
                    if (!wait(kBarFull + st, c / NS) || (count_of(c) < kC && !wait(kBarClear, 0)) ||
                        (c >= 2 && !wait(kBarOFree + b, (c - 2) >> 1)))
                        break;
                    tc_after();
#pragma unroll 1
                    for (int k = 0; k < ksteps; ++k) {
                        const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32);
                        mma(tmem + col_qk(b), sdesc(x + off, 0), sdesc(y + off, 0), idesc(kC, false, false), k > 0);
                    }
                    mma_commit(bar(kBarQK + b));
                    mma_commit(bar(kBarFree + st));
                }
                drain(0);
            }
        }
    } else if (warp == kKvWarp) {
        if (lane == 0) {
            bool ok = true;
            for (int c = 0; c < nc && ok; ++c) {
                const int st = c % NS;
                const uint32_t y = sbase + (uint32_t)(st * M::kStage + M::kX);
                if (c > 0 && !(ok = wait(kBarKVFree, c - 1))) break;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    if (!(ok = wait(kBarZs + hf, c))) break;
                    tc_after();
#pragma unroll 1
                    for (int k = 4 * hf; k < 4 * hf + 4; ++k)
                        // dx <= 64: the second 64 rows of the product repeat the first
                        mma(tmem + kColKv, sdesc(y + 2048 * k, DX == 64 ? 0 : 16384), sdesc(sbase + M::oZs + 2048 * k, M::kZb),
                            idesc(3 * kZ, true, true), k > 0);
                    mma_commit(bar(kBarZsFree + hf));
                }
                mma_commit(bar(kBarKV));
                mma_commit(bar(kBarFree + st));
            }
            drain(1);
        }
    } else if (warp == kOWarp) {
        if constexpr (!kStates) {
            if (lane == 0) {
                const int ksteps = (p.dx + 15) >> 4;
                for (int c = 0; c < nc; ++c) {
                    const int b = c & 1, st = c % NS;
                    const uint32_t x = sbase + (uint32_t)(st * M::kStage), z = x + M::kX + M::kY;
                    if (!wait(kBarFull + st, c / NS) || !wait(kBarS, c) || (c > 0 && !wait(kBarOFree + (b ^ 1), (c - 1) >> 1))) break;
                    tc_after();
#pragma unroll 1
                    for (int k = 0; k < ksteps; ++k)
                        mma(tmem + kColOb, sdesc(x + (k >> 2) * 16384 + (k & 3) * 32, 0), sdesc(sbase + M::oS + 2048 * k, 0),
                            idesc(kZ, false, true), k > 0);
                    mma_commit(bar(kBarOB));
                    if (!wait(kBarP + b, c >> 1)) break;
                    tc_after();
#pragma unroll 1
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + col_oa(b), tmem + col_qk(b) + 8u * k, sdesc(z + 2048 * k, 0), idesc(kZ, false, true), k > 0);
                    mma_commit(bar(kBarO + b));
                    mma_commit(bar(kBarFree + st));
                }
                drain(2);
            }
        }
    } else if (warp < 4) {
        // ================================= group P =================================
        if constexpr (!kStates) {
            const int t = 32 * warp + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
            for (int c = 0; c < nc; ++c) {
                const uint32_t qk = lanes + col_qk(c & 1);
                if (!wait_all(kBarQK + (c & 1), c >> 1)) break;
                tc_after();
#pragma unroll 1
                for (int jb = 0; jb < 4; ++jb) {
                    uint32_t r[16];
                    const int past = rev ? jb - warp : warp - jb;  // blocks between this one and the diagonal
                    if (past < 0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = 0u;
                    } else {
                        float v[32];
                        tmem_ld32(qk + 32u * jb, v);
                        // lam^|t - s| from the row's distance to the block's edge and the column's; in
                        // the block on the diagonal from the table, whose other side is zeros
                        if (past > 0) {
                            const f2 rf = f2_splat(pwp[rev ? 32 * jb - t : t - 32 * jb - 31]);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                f2 w0, w1;
                                lds_f2x2(cfw + i, w0, w1);
                                f2_split(f2_mul(f2_make(v[i], v[i + 1]), f2_mul(rf, w0)), v[i], v[i + 1]);
                                f2_split(f2_mul(f2_make(v[i + 2], v[i + 3]), f2_mul(rf, w1)), v[i + 2], v[i + 3]);
                            }
                        } else {
                            const float *w = pwp + (rev ? -lane : lane);
                            if (rev) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= w[i];
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= w[-i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = pack2(v[2 * i], v[2 * i + 1]);
                    }
                    tmem_st16(qk + 16u * jb, r);
                }
                tmem_st_wait();
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarP + (c & 1)));
            }
        }
    } else if (warp >= 12 && warp < 16) {
        // ================================= group E =================================
        if constexpr (!kStates) {
            const int t = 32 * (warp - 12) + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp - 12)) << 16);
            const int64_t o0 = (a.seq_start ? 0 : (int64_t)pl.seq * p.o_sb) + (int64_t)h * p.o_sh + kZ * zb;
            const int cols = p.dz - kZ * zb < kZ ? p.dz - kZ * zb : kZ;
            for (int c = 0; c < nc; ++c) {
                const int b = c & 1, n = count_of(c);
                const float rf = t < n ? p.ro * pw[rev ? n - 1 - t : t + 1] : 0.0f;
                const int64_t at = o0 + (int64_t)(pl.row0 + first_of(c) + t) * p.o_sl;
                if (!wait_all(kBarO + b, c >> 1)) break;
                tc_after();
#pragma unroll 1
                for (int i = 0; i < kZ; i += 16) {
                    float v[16], ob[16];
                    tmem_ld2x16(lanes + col_oa(b) + (uint32_t)i, lanes + kColOb + (uint32_t)i, v, ob);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = fmaf(rf, ob[j], v[j]);
#pragma unroll
                    for (int j = 0; j < 16; j += 8)
                        if (t < n && i + j < cols) {
                            if (p.o_f32) {
                                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at + i + j);
                                o[0] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                                o[1] = make_float4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
                            } else {
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + at + i + j) =
                                    make_uint4(pack2(v[j], v[j + 1]), pack2(v[j + 2], v[j + 3]), pack2(v[j + 4], v[j + 5]),
                                               pack2(v[j + 6], v[j + 7]));
                            }
                        }
                }
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarOFree + b));
            }
        }
    } else if (warp < 8) {
        // ================================= group V =================================
        const int gt = tid - 128;
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            const int st = c % NS, n = count_of(c);
            if (!wait_all(kBarFull + st, c / NS)) break;
            unsigned char *y = smem + st * M::kStage + M::kX, *z = y + M::kY, *zs = smem + M::oZs;
            if (n < kC) {
                // the rows behind the sequence, before any product reads them
#pragma unroll 1
                for (int i = n * 8 + gt; i < kC * 8; i += 128) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(z + 16 * i) = zero;
#pragma unroll
                    for (int j = 0; j < DX / 64; ++j) *reinterpret_cast<uint4 *>(y + j * 16384 + 16 * i) = zero;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarClear));
            }
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                if (c > 0 && !(ok = wait_all(kBarZsFree + hf, c - 1))) break;
#pragma unroll 1
                for (int it = 0; it < 4; ++it) {
                    const int i = hf * 512 + it * 128 + gt, row = i >> 3;
                    uint4 hi, mid, lo;
                    float w = 0.0f;
                    uint4 q = make_uint4(0, 0, 0, 0);
                    if (row < n) {
                        w = p.ws * pw[rev ? row + 1 : n - 1 - row];
                        q = *reinterpret_cast<const uint4 *>(z + 16 * i);
                    }
                    split3(w * bf16_lo(q.x), w * bf16_hi(q.x), hi.x, mid.x, lo.x);
                    split3(w * bf16_lo(q.y), w * bf16_hi(q.y), hi.y, mid.y, lo.y);
                    split3(w * bf16_lo(q.z), w * bf16_hi(q.z), hi.z, mid.z, lo.z);
                    split3(w * bf16_lo(q.w), w * bf16_hi(q.w), hi.w, mid.w, lo.w);
                    *reinterpret_cast<uint4 *>(zs + 16 * i) = hi;
                    *reinterpret_cast<uint4 *>(zs + M::kZb + 16 * i) = mid;
                    *reinterpret_cast<uint4 *>(zs + 2 * M::kZb + 16 * i) = lo;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarZs + hf));
            }
        }
    } else if (warp < 12) {
        // ================================= group S =================================
        // dx <= 64: KV's second 64 rows repeat the first, so warps 2 and 3 take the
        // second 32 columns of rows 0..63
        constexpr int NCOL = DX == 64 ? 32 : 64;
        const int w = warp - 8, row = (DX == 64 ? 32 * (w & 1) : 32 * w) + lane, c0 = DX == 64 ? 32 * (w >> 1) : 0;
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
        float S[NCOL];
        const int64_t blk = p.dx * (int64_t)p.dz;
        {
            const float *s0 = p.s0 ? p.s0 + ((int64_t)(p.s0_slot ? slot : pl.seq) * a.H + h) * blk : nullptr;
#pragma unroll
            for (int i = 0; i < NCOL; ++i) {
                const int col = kZ * zb + c0 + i;
                S[i] = (s0 && !kStates && row < p.dx && col < p.dz) ? s0[row * p.s0_sr + col * p.s0_sc] : 0.0f;
            }
        }
        bool ok = true;
        const float m128 = expm1f((float)kC * g);
        for (int c = 0; c < nc; ++c) {
            if constexpr (!kStates) {
                if (c > 0 && !(ok = wait_all(kBarOB, c - 1))) break;
                unsigned char *dst = smem + M::oS + row * 128;
#pragma unroll
                for (int i = 0; i < NCOL; i += 8)
                    *reinterpret_cast<uint4 *>(dst + ((((c0 + i) >> 3) ^ (row & 7)) << 4)) =
                        make_uint4(pack2(S[i], S[i + 1]), pack2(S[i + 2], S[i + 3]), pack2(S[i + 4], S[i + 5]),
                                   pack2(S[i + 6], S[i + 7]));
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarS));
            }
            if (!(ok = wait_all(kBarKV, c))) break;
            tc_after();
            // lam^n S + KV as keep S + (part S + KV): with lam^n >= 1/2 part = lam^n - 1 keeps
            // the bits of a slow decay over many chunks
            const float m = count_of(c) == kC ? m128 : expm1f((float)count_of(c) * g);
            const float keep = m >= -0.5f ? 1.0f : 0.0f, part = m >= -0.5f ? m : pw[count_of(c)];
#pragma unroll
            for (int i = 0; i < NCOL; i += 8) {
                float hi[8], mid[8], lo[8];
                const uint32_t at = lanes + kColKv + (uint32_t)(c0 + i);
                tmem_ld3x8(at, at + kZ, at + 2 * kZ, hi, mid, lo);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    S[i + j] = fmaf(keep, S[i + j], fmaf(part, S[i + j], hi[j] + (mid[j] + lo[j])));
            }
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kBarKVFree));
        }
        const bool last = rev ? pl.g == 0 : pl.g == pl.ng - 1;
        if (ok && p.fin && (kStates || last) && row < p.dx) {
            float *f = p.fin + ((int64_t)(kStates ? slot : pl.seq) * a.H + h) * blk + row * (int64_t)p.dz + kZ * zb + c0;
#pragma unroll
            for (int i = 0; i < NCOL; i += 4)
                if (kZ * zb + c0 + i < p.dz) *reinterpret_cast<float4 *>(f + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
    }

    tc_before();
    __syncthreads();
    if (warp == kQkWarp) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// The states that segments start from, in place of what each contributes:
// st[j] <- lam^(tokens before it) s0 + the earlier segments' parts, in order.
struct ChainArgs {
    float *st[2];
    const float *s0[2];
    int64_t s0_sr[2], s0_sc[2];
    int dx[2], dz[2], rev[2];
};
__global__ void __launch_bounds__(256) linattn_chain_kernel(const __grid_constant__ TcArgs a, const ChainArgs ch) {
    const int k = blockIdx.z;
    const int64_t seq = (int)blockIdx.y / a.H, h = (int)blockIdx.y % a.H, blk = (int64_t)ch.dx[k] * ch.dz[k];
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t base = seq * a.nseg, len = a.seqlen;
    if (a.seq_start) {
        const int64_t s = a.seq_start[seq], t = a.seq_start[seq + 1];
        if (!(s >= 0 && t >= s && t <= a.total)) return;
        base = s / a.seg + seq;
        len = t - s;
    }
    if (e >= blk) return;
    const int64_t ng = len > a.seg ? (len + a.seg - 1) / a.seg : 1;
    const float g = fmaxf(__ldg(a.log_decay + h), -1e30f);
    const int64_t i = e / ch.dz[k], j = e % ch.dz[k];
    float S = ch.s0[k] ? ch.s0[k][(seq * a.H + h) * blk + i * ch.s0_sr[k] + j * ch.s0_sc[k]] : 0.0f;
    float *st = ch.st[k] + h * blk + e;
    for (int64_t c = 0; c < ng; ++c) {
        const int64_t q = ch.rev[k] ? ng - 1 - c : c;
        float *at = st + (base + q) * a.H * blk;
        const float own = c < ng - 1 ? *at : 0.0f;
        *at = S;
        const int64_t left = len - q * a.seg, n = left < a.seg ? left : a.seg;
        S = fmaf(expf((float)n * g), S, own);
    }
}

using PfnEncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                    const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
PfnEncodeTiled encode_fn() {
    static std::once_flag once;
    static PfnEncodeTiled fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PfnEncodeTiled>(f);
        cudaGetLastError();
    });
    return fn;
}

// A token array as a 4-D map {column, head, token, batch row}: box {64 columns,
// 1 head, 128 tokens, 1 row}, 128-byte swizzle; what lies outside reads as zero.
struct MapKey {
    const void *p;
    int64_t sb, sl, sh, heads;
    int d;
    bool operator==(const MapKey &o) const {
        return p == o.p && sb == o.sb && sl == o.sl && sh == o.sh && heads == o.heads && d == o.d;
    }
};
bool map_ok(const MapKey &k, int64_t batch) {
    auto st = [](int64_t s, bool used) { return !used || (s > 0 && (s * 2) % 16 == 0 && s * 2 < (1ll << 40)); };
    return reinterpret_cast<uintptr_t>(k.p) % 16 == 0 && st(k.sl, true) && st(k.sh, k.heads > 1) && st(k.sb, batch > 1);
}
bool encode(CUtensorMap *m, const MapKey &k, int64_t rows, int64_t batch) {
    PfnEncodeTiled fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)k.d, (cuuint64_t)k.heads, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)(k.heads > 1 ? k.sh * 2 : 16), (cuuint64_t)(k.sl * 2),
                                   (cuuint64_t)(batch > 1 ? k.sb * 2 : 16)};
    const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)kC, 1u};
    const cuuint32_t es[4] = {1u, 1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(k.p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

MapKey key_x(const LaArgs &a, const LaProblem &p) { return {p.x, p.x_sb, p.x_sl, p.x_sh, a.H / p.xg, p.dx}; }
MapKey key_y(const LaArgs &a, const LaProblem &p) { return {p.y, p.y_sb, p.y_sl, p.y_sh, a.H / p.yg, p.dx}; }
MapKey key_z(const LaArgs &a, const LaProblem &p) { return {p.z, p.z_sb, p.z_sl, p.z_sh, a.H / p.zg, p.dz}; }

int zblocks(int dz) { return (dz + kZ - 1) / kZ; }

// Segments: one block per SM is what runs at a time, so sequences are cut only
// where sequences, heads and column blocks are fewer than the SMs, into as many
// segments as fill them once, of at least 512 tokens.
struct SegPlan {
    int64_t seg, nseg, slots;
    bool segmented;
};
SegPlan seg_plan(int64_t batch, int64_t rows, bool packed, int64_t H, int units, int num_sms) {
    SegPlan s{};
    const int64_t base = std::max<int64_t>(1, batch * H * units);
    const int64_t longest = rows;  // packed: any one of the sequences may have them all
    const int64_t ways = num_sms / base;
    s.seg = std::max<int64_t>(512, ((longest + std::max<int64_t>(ways, 1) - 1) / std::max<int64_t>(ways, 1) + kC - 1) / kC * kC);
    s.segmented = ways >= 2 && s.seg < longest;
    if (!s.segmented) s.seg = std::max<int64_t>(kC, (longest + kC - 1) / kC * kC + (packed ? kC : 0));
    s.nseg = s.segmented && !packed ? (rows + s.seg - 1) / s.seg : 1;
    s.slots = !s.segmented ? batch : packed ? rows / s.seg + batch : batch * s.nseg;
    return s;
}

template <int DX, bool kStates>
cudaError_t launch_t(const TcArgs &a, const TcMaps &maps, int64_t slots, cudaStream_t stream) {
    static SmemOptIn opt_in;
    constexpr int bytes = Smem<DX, kStates>::kBytes;
    static_assert(bytes <= 232448, "shared memory of a block");
    cudaError_t e = opt_in.ensure(reinterpret_cast<const void *>(linattn_tc_kernel<DX, kStates>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = slots * a.H * a.units;
    if (grid > 0x7fffffffLL || a.seg <= 0) return cudaErrorInvalidConfiguration;
    linattn_tc_kernel<DX, kStates><<<(unsigned)grid, kThreads, bytes, stream>>>(a, maps);
    return cudaGetLastError();
}

}  // namespace

bool linattn_tc_applies(const LaArgs &a, bool bf16) {
    const int64_t rows = a.seq_start ? a.total : a.seqlen, batch = a.seq_start ? 1 : a.batch;
    if (!bf16 || rows <= 0) return false;
    for (int i = 0; i < a.np; ++i) {
        const LaProblem &p = a.p[i];
        const int eo = p.o_f32 ? 4 : 2;
        if (p.dx % 8 || p.dz % 8 || !map_ok(key_x(a, p), batch) || !map_ok(key_y(a, p), batch) ||
            !map_ok(key_z(a, p), batch) || reinterpret_cast<uintptr_t>(p.o) % 16 || (p.o_sb * eo) % 16 ||
            (p.o_sl * eo) % 16 || (p.o_sh * eo) % 16 || reinterpret_cast<uintptr_t>(p.fin) % 16)
            return false;
    }
    return true;
}

// Bytes of segment states: of one direction (forward), or two (gradients).
size_t linattn_tc_workspace(int64_t batch, int64_t rows, bool packed, int64_t H, int dk, int dv, bool bwd, int num_sms) {
    if (batch < 1 || rows < 1) return 0;
    const int units = bwd ? 2 * zblocks(dk) + zblocks(dv) : zblocks(dv);
    const SegPlan s = seg_plan(batch, rows, packed, H, units, num_sms);
    return s.segmented ? (size_t)(bwd ? 2 : 1) * (size_t)s.slots * H * dk * dv * sizeof(float) : 0;
}

cudaError_t launch_linattn_tc(const LaArgs &la, void *workspace, int num_sms, cudaStream_t stream) {
    const bool packed = la.seq_start != nullptr;
    const int64_t rows = packed ? la.total : la.seqlen, batch = packed ? 1 : la.batch;
    TcArgs a{};
    a.log_decay = la.log_decay;
    a.seq_start = la.seq_start;
    a.status = la.status;
    a.batch = (int)la.batch; a.seqlen = (int)la.seqlen; a.total = (int)la.total; a.H = (int)la.H;
    a.np = la.np;
    TcMaps maps;
    MapKey keys[4];
    int nk = 0, dxmax = 0;
    auto map_of = [&](const MapKey &k) {
        for (int i = 0; i < nk; ++i)
            if (keys[i] == k) return i;
        if (nk == 4 || !encode(&maps.m[nk], k, rows, batch)) return -1;
        keys[nk] = k;
        return nk++;
    };
    for (int i = 0; i < la.np; ++i) {
        const LaProblem &p = la.p[i];
        TcProblem &t = a.p[i];
        t.mx = map_of(key_x(la, p));
        t.my = map_of(key_y(la, p));
        t.mz = map_of(key_z(la, p));
        if (t.mx < 0 || t.my < 0 || t.mz < 0) return cudaErrorInvalidValue;
        t.xg = p.xg; t.yg = p.yg; t.zg = p.zg; t.dx = p.dx; t.dz = p.dz; t.rev = p.rev; t.o_f32 = p.o_f32;
        t.ws = p.ws; t.ro = p.ro; t.ps = p.ws * p.ro;
        t.s0 = p.s0; t.s0_sr = p.s0_sr; t.s0_sc = p.s0_sc; t.fin = p.fin;
        t.o = p.o; t.o_sb = p.o_sb; t.o_sl = p.o_sl; t.o_sh = p.o_sh;
        t.nzb = zblocks(p.dz);
        a.units += t.nzb;
        dxmax = std::max(dxmax, p.dx);
    }
    const SegPlan sp = seg_plan(la.batch, rows, packed, la.H, a.units, num_sms);
    a.seg = (int)sp.seg;
    a.nseg = (int)sp.nseg;
    a.segmented = sp.segmented ? 1 : 0;
    if (sp.segmented) {
        // the segments' own states: of the forward direction (problem 0), and of the reverse one
        // (problem 2; problem 1 reads it with rows and columns exchanged)
        TcArgs s = a;
        ChainArgs ch{};
        float *st = static_cast<float *>(workspace);
        const int own[2] = {0, 2};
        s.np = la.np == 1 ? 1 : 2;
        s.units = 0;
        for (int k = 0; k < s.np; ++k) {
            const TcProblem &p = a.p[own[k]];
            s.p[k] = p;
            s.p[k].fin = st + k * sp.slots * la.H * p.dx * p.dz;
            s.units += p.nzb;
            ch.st[k] = s.p[k].fin;
            ch.s0[k] = p.s0; ch.s0_sr[k] = p.s0_sr; ch.s0_sc[k] = p.s0_sc;
            ch.dx[k] = p.dx; ch.dz[k] = p.dz; ch.rev[k] = p.rev;
        }
        cudaError_t e = dxmax <= 64 ? launch_t<64, true>(s, maps, sp.slots, stream)
                                    : launch_t<128, true>(s, maps, sp.slots, stream);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)((ch.dx[0] * ch.dz[0] + 255) / 256), (unsigned)(la.batch * la.H), (unsigned)s.np);
        linattn_chain_kernel<<<grid, 256, 0, stream>>>(a, ch);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        for (int i = 0; i < la.np; ++i) {
            TcProblem &t = a.p[i];
            t.s0 = ch.st[i == 0 ? 0 : 1];
            t.s0_slot = 1;
            t.s0_sr = i == 1 ? 1 : t.dz;
            t.s0_sc = i == 1 ? t.dx : 1;
        }
    }
    return dxmax <= 64 ? launch_t<64, false>(a, maps, sp.slots, stream) : launch_t<128, false>(a, maps, sp.slots, stream);
}

}  // namespace ms

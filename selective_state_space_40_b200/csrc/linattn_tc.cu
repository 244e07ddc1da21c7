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
// a first pass (kStates) forms each segment's own state from zero, and the main
// pass starts every segment from the initial state and the earlier ones' own.
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
// The warps of a CTA: group P, group V, group S, group E, and one that loads and
// three that issue. Group V sets the pace at dx <= 64, so there it has eight warps
// (NNN); at dx = 128 the registers of S leave room for four.
template <int DX>
struct Roles {
    static constexpr int kV = DX == 64 ? 8 : 4;
    static constexpr int kV0 = 4, kS0 = kV0 + kV, kE0 = kS0 + 4;
    static constexpr int kLoad = kE0 + 4, kQk = kLoad + 1, kKv = kLoad + 2, kO = kLoad + 3;
    static constexpr int kThreads = 32 * (kO + 1);
};
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
    const float *s0;          // entering states: block (sequence, head) of dx * dz, element (i, j) at i s0_sr + j s0_sc
    const float *seg_states;  // segments' own states, blocks (slot, head), or null
    float *fin;               // leaving states [batch, H, dx, dz], or (kStates) [slots, H, dx, dz]
    int64_t s0_sr, s0_sc, seg_sr, seg_sc;  // seg_states' strides
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
    static constexpr int oTv = oS + (kStates ? 0 : DX * kZ * 2);  // weights of Z's rows
    static constexpr int oTe = oTv + 128 * 4;                // of O_b's rows
    static constexpr int oPs = oTe + 128 * 4;                // ps lam^n
    static constexpr int oDiag = oPs + 128 * 4;              // ps lam^|d| at 31 + d, d = t - s, 0 on the masked side
    static constexpr int oCf = oDiag + 64 * 4;               // lam^(31-c), in reverse lam^c, c < 32
    static constexpr int oBar = oCf + 32 * 4;
    static constexpr int kBytes = oBar + 8 * 38 + 16;
};
enum {
    kBarX = 0,        // [3] a stage's X, Y, Z tiles are in
    kBarY = 3,
    kBarZ = 6,
    kBarXFree = 9,    // [3] what uses the stage's X (QK, O_b), Y (QK, KV), Z (groups V, E) is done
    kBarYFree = 12,
    kBarZFree = 15,
    kBarQK = 18,      // [2] QK is done
    kBarP = 20,       // [2] P is in tensor memory
    kBarO = 22,       // [2] O_a and O_b are done
    kBarOFree = 24,   // [2] group E has read O_a (and O_b)
    kBarZs = 26,      // [2] Z' of 64 tokens is in shared memory
    kBarZsFree = 28,  // [2] KV has read it
    kBarKV = 30,      // KV is done
    kBarKVFree = 31,  // group S has read it
    kBarS = 32,       // S is in shared memory
    kBarOB = 33,      // O_b is done (and S read)
    kBarClear = 34,   // the rows behind the sequence are cleared (once, in the chunk that has some)
    kBarEnd = 35,     // [3] nothing of an issuing warp is in flight
    kNumBars = 38
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
__device__ __forceinline__ uint64_t dstep(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }  // (no carry out of the address)
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
// SM's instruction cache (see the kernel). (A warp's lanes all ask: one lane that
// asks for the others took 8 % more of the whole.)
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
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(f2 v) {
    float a, b;
    f2_split(v, a, b);
    return pack2(a, b);
}
__device__ __forceinline__ f2 unpack2(uint32_t v) { return f2_make(bf16_lo(v), bf16_hi(v)); }
// w q = hi + mid + lo in bf16 parts (24 significant bits) for a pair q of bf16
__device__ __forceinline__ void split3(f2 w, uint32_t q, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    f2 v = f2_mul(w, unpack2(q));
    hi = pack2(v);
    v = f2_sub(v, unpack2(hi));
    mid = pack2(v);
    lo = pack2(f2_sub(v, unpack2(mid)));
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

// The roles' code is what the SM's instruction cache has to hold at once (five
// groups of warps, each in a loop of its own): with the loops unrolled and the
// call's parameters read inside them, warps waited for instructions half of the
// time. So what a chunk needs is laid out before the loops (tables, addresses,
// steps), and the loops are short.
template <int DX, bool kStates>
__global__ void __launch_bounds__(Roles<DX>::kThreads, 1) linattn_tc_kernel(const __grid_constant__ TcArgs a,
                                                                 const __grid_constant__ TcMaps maps) {
    using M = Smem<DX, kStates>;
    using R = Roles<DX>;
    constexpr int NS = M::kStages, KX = DX / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = saddr(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + M::oBar + 8 * 38);
    volatile uint32_t *abort_flag = misc + 1;

    int unit = (int)(blockIdx.x % (unsigned)a.units);
    const int hs = (int)(blockIdx.x / (unsigned)a.units), h = hs % a.H, slot = hs / a.H;
    int pi = 0;
    while (unit >= a.p[pi].nzb) unit -= a.p[pi++].nzb;
    const TcProblem &p = a.p[pi];
    const int zb = unit;
    const Place pl = place_of(a, slot, lane);
    if (pl.bad && tid == 0 && a.status) atomicOr(a.status, MS_ERR_SHAPE);
    const bool rev = p.rev != 0;
    if (!pl.ok || (kStates && (rev ? pl.g == 0 : pl.g == pl.ng - 1))) return;
    const int seg0 = pl.g * a.seg;
    const int ntok = pl.len - seg0 < a.seg ? pl.len - seg0 : a.seg;
    const int nc = (ntok + kC - 1) / kC;
    // the chunk (in the order of work) that is not full, if one is not, and its tokens
    const int npart = ntok % kC == 0 ? kC : ntok % kC, cpart = npart == kC ? -1 : rev ? 0 : nc - 1;
    // the first row of chunk c is row0 + c * dt
    const int dt = rev ? -kC : kC, row0 = pl.row0 + seg0 + (rev ? (nc - 1) * kC : 0);

    const float g = fmaxf(__ldg(a.log_decay + h), -1e30f);  // -inf: 0 * -inf must be 0
    if (tid < kC) {
        float *tv = reinterpret_cast<float *>(smem + M::oTv), *te = reinterpret_cast<float *>(smem + M::oTe);
        float *ps = reinterpret_cast<float *>(smem + M::oPs), *dg = reinterpret_cast<float *>(smem + M::oDiag);
        float *cf = reinterpret_cast<float *>(smem + M::oCf);
        const float w = expf((float)tid * g), w1 = expf((float)(tid + 1) * g);
        if (rev) {
            tv[tid] = p.ws * w1;
            te[kC - 1 - tid] = p.ro * w;
        } else {
            tv[kC - 1 - tid] = p.ws * w;
            te[tid] = p.ro * w1;
        }
        ps[tid] = p.ps * w;
        if (tid < 32) {
            dg[31 + tid] = rev && tid > 0 ? 0.0f : p.ps * w;
            if (tid > 0) dg[31 - tid] = rev ? p.ps * w : 0.0f;
            cf[rev ? tid : 31 - tid] = w;
        }
    }
    const uint32_t bars = sbase + (uint32_t)M::oBar;
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const bool warps4 = (i >= kBarP && i < kBarP + 2) || (i >= kBarOFree && i < kBarOFree + 2) ||
                                i == kBarKVFree || i == kBarS;
            const bool warpsv = (i >= kBarZs && i < kBarZs + 2) || i == kBarClear;
            const bool two = (i >= kBarXFree && i < kBarYFree) || (i >= kBarYFree && i < kBarZFree && !kStates);
            const bool zfree = i >= kBarZFree && i < kBarZFree + 3;  // the warps of V and E
            bar_init(bars + 8 * i, warps4 ? 4 : warpsv ? R::kV : two ? 2 : zfree ? (kStates ? R::kV : R::kV + 4) : 1);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == R::kQk) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(misc)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = misc[0];
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](int i, int k) { return bar_wait(bar(i), (uint32_t)k, abort_flag, a.status); };
    auto wait_all = [&](int i, int k) { return __all_sync(0xffffffffu, wait(i, k)) != 0; };  // whole warps: one answer
    // every product that an issuing thread has in flight completes before the tensor memory is freed
    auto drain = [&](int i) {
        mma_commit(bar(kBarEnd + i));
        for (uint32_t k = 0; k < kSpinTries && !bar_try(bar(kBarEnd + i), 0u); ++k) {}
    };
    // stages go round: st = c % NS, and use = c / NS counts the rounds
    struct Ring {
        int st = 0, use = 0;
        __device__ __forceinline__ void next() {
            if (++st == NS) st = 0, ++use;
        }
    } ring;

    if (warp == R::kLoad) {
        if (lane == 0) {
            const CUtensorMap *mx = &maps.m[p.mx], *my = &maps.m[p.my], *mz = &maps.m[p.mz];
            const int b = a.seq_start ? 0 : pl.seq;
            const int hx = h / p.xg, hy = h / p.yg, hz = h / p.zg;
            int c = 0, t = row0, sent_of_last = 0;  // sent_of_last: of the chunk at which the loop stopped
            bool ok = true;
#pragma unroll 1
            for (; c < nc; ++c, t += dt, ring.next()) {
                const int st = ring.st, use = ring.use;
                const uint32_t dst = sbase + (uint32_t)(st * M::kStage);
                sent_of_last = 0;
                if (use > 0 && !(ok = wait(kBarYFree + st, use - 1))) break;
                bar_arrive_tx(bar(kBarY + st), (uint32_t)M::kY);
#pragma unroll
                for (int i = 0; i < DX / 64; ++i) tma_load4(my, dst + M::kX + i * 16384, bar(kBarY + st), 64 * i, hy, t, b);
                sent_of_last = 1;
                if (use > 0 && !(ok = wait(kBarZFree + st, use - 1))) break;
                bar_arrive_tx(bar(kBarZ + st), (uint32_t)M::kZb);
                tma_load4(mz, dst + M::kX + M::kY, bar(kBarZ + st), kZ * zb, hz, t, b);
                sent_of_last = 2;
                if constexpr (!kStates) {
                    if (use > 0 && !(ok = wait(kBarXFree + st, use - 1))) break;
                    bar_arrive_tx(bar(kBarX + st), (uint32_t)M::kX);
#pragma unroll
                    for (int i = 0; i < DX / 64; ++i) tma_load4(mx, dst + i * 16384, bar(kBarX + st), 64 * i, hx, t, b);
                }
            }
            // when stopping, the copies issued have landed before the CTA ends
            for (int q = 0; q < 3 && !ok; ++q) {
                const int at = q == 0 ? kBarY : q == 1 ? kBarZ : kBarX, last = q < sent_of_last ? c : c - 1;
                for (int i = last < NS ? 0 : last - NS + 1; i <= last && (q < 2 || !kStates); ++i)
                    for (uint32_t k = 0; k < kSpinTries && !bar_try(bar(at + i % NS), (uint32_t)(i / NS) & 1u); ++k) {}
            }
        }
    } else if (warp == R::kQk) {
        if constexpr (!kStates) {
            if (lane == 0) {
                const uint64_t dx0 = sdesc(sbase, 0), dy0 = sdesc(sbase + M::kX, 0);
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ring.next()) {
                    const int b = c & 1, st = ring.st;
                    if (!wait(kBarX + st, ring.use) || !wait(kBarY + st, ring.use) || (c == cpart && !wait(kBarClear, 0)) ||
                        (c >= 2 && !wait(kBarOFree + b, (c - 2) >> 1)))
                        break;
                    tc_after();
                    const uint64_t x = dstep(dx0, st * M::kStage), y = dstep(dy0, st * M::kStage);
#pragma unroll
                    for (int k = 0; k < KX; ++k) {
                        const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32);
                        mma(tmem + col_qk(b), dstep(x, off), dstep(y, off), idesc(kC, false, false), k > 0);
                    }
                    mma_commit(bar(kBarQK + b));
                    mma_commit(bar(kBarXFree + st));
                    mma_commit(bar(kBarYFree + st));
                }
                drain(0);
            }
        }
    } else if (warp == R::kKv) {
        if (lane == 0) {
            // dx <= 64: the second 64 rows of the product repeat the first
            const uint64_t dy0 = sdesc(sbase + M::kX, DX == 64 ? 0 : 16384), dz = sdesc(sbase + M::oZs, M::kZb);
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < nc && ok; ++c, ring.next()) {
                const int st = ring.st;
                const uint64_t y = dstep(dy0, st * M::kStage);
                if (!(ok = wait(kBarY + st, ring.use)) || (c > 0 && !(ok = wait(kBarKVFree, c - 1)))) break;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    if (!(ok = wait(kBarZs + hf, c))) break;
                    tc_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma(tmem + kColKv, dstep(y, 8192 * hf + 2048 * k), dstep(dz, 8192 * hf + 2048 * k),
                            idesc(3 * kZ, true, true), hf > 0 || k > 0);
                    mma_commit(bar(kBarZsFree + hf));
                }
                mma_commit(bar(kBarKV));
                mma_commit(bar(kBarYFree + st));
            }
            drain(1);
        }
    } else if (warp == R::kO) {
        if constexpr (!kStates) {
            if (lane == 0) {
                const uint64_t dx0 = sdesc(sbase, 0), dz0 = sdesc(sbase + M::kX + M::kY, 0), ds = sdesc(sbase + M::oS, 0);
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ring.next()) {
                    const int b = c & 1, st = ring.st;
                    if (!wait(kBarX + st, ring.use) || !wait(kBarZ + st, ring.use) || !wait(kBarS, c) ||
                        (c > 0 && !wait(kBarOFree + (b ^ 1), (c - 1) >> 1)))
                        break;
                    tc_after();
                    const uint64_t x = dstep(dx0, st * M::kStage), z = dstep(dz0, st * M::kStage);
#pragma unroll
                    for (int k = 0; k < KX; ++k)
                        mma(tmem + kColOb, dstep(x, (k >> 2) * 16384 + (k & 3) * 32), dstep(ds, 2048 * k),
                            idesc(kZ, false, true), k > 0);
                    mma_commit(bar(kBarOB));
                    mma_commit(bar(kBarXFree + st));
                    if (!wait(kBarP + b, c >> 1)) break;
                    tc_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + col_oa(b), tmem + col_qk(b) + 8u * k, dstep(z, 2048 * k), idesc(kZ, false, true), k > 0);
                    mma_commit(bar(kBarO + b));
                }
                drain(2);
            }
        }
    } else if (warp < 4) {
        // ================================= group P =================================
        if constexpr (!kStates) {
            const int t = 32 * warp + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
            // a block of 32 columns before the diagonal: lam^|t - s| from the row's distance to the
            // block's edge (rf, a step per block) and the column's (cf); the block on the diagonal
            // from a table by t - s, one side of which is zeros; behind it, zeros
            const float *cf = reinterpret_cast<const float *>(smem + M::oCf);
            const float *dg = reinterpret_cast<const float *>(smem + M::oDiag) + 31 + lane;
            const float *rf0 = reinterpret_cast<const float *>(smem + M::oPs) + (rev ? -t : t - 31);
            const int past0 = rev ? -warp : warp, dpast = rev ? 1 : -1, drf = rev ? 32 : -32;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
                const uint32_t qk = lanes + col_qk(c & 1);
                if (!wait_all(kBarQK + (c & 1), c >> 1)) break;
                tc_after();
                int past = past0;  // blocks between this one and the diagonal
                const float *rf = rf0;
#pragma unroll 1
                for (int jb = 0; jb < 4; ++jb, past += dpast, rf += drf) {
                    uint32_t r[16];
                    if (past < 0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = 0u;
                    } else {
                        float v[32];
                        tmem_ld32(qk + 32u * jb, v);
                        if (past > 0) {
                            const f2 w = f2_splat(*rf);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                f2 w0, w1;
                                lds_f2x2(cf + i, w0, w1);
                                r[i / 2] = pack2(f2_mul(f2_make(v[i], v[i + 1]), f2_mul(w, w0)));
                                r[i / 2 + 1] = pack2(f2_mul(f2_make(v[i + 2], v[i + 3]), f2_mul(w, w1)));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) r[i / 2] = pack2(v[i] * dg[-i], v[i + 1] * dg[-i - 1]);
                        }
                    }
                    tmem_st16(qk + 16u * jb, r);
                }
                tmem_st_wait();
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarP + (c & 1)));
            }
        }
    } else if (warp >= R::kE0) {
        // ================================= group E =================================
        if constexpr (!kStates) {
            const int t = 32 * (warp - R::kE0) + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp - R::kE0)) << 16);
            const int cols = p.dz - kZ * zb < kZ ? p.dz - kZ * zb : kZ;
            const int64_t at = (a.seq_start ? 0 : (int64_t)pl.seq * p.o_sb) + (int64_t)h * p.o_sh + kZ * zb +
                               (int64_t)(row0 + 32 * (warp - R::kE0) + (lane >> 3)) * p.o_sl;
            const int es = p.o_f32 ? 4 : 2;
            // A thread holds a row, but stores that touch 32 rows at once keep the load-store unit
            // from everybody else (2000 clocks a chunk): rows go through the chunk's Z tile, which
            // nothing reads any more, and leave 128 bytes of 4 rows at a time.
            const int q = lane & 7, r4 = lane >> 3;
            unsigned char *o = static_cast<unsigned char *>(p.o) + at * es + 16 * q;
            const int64_t step = (int64_t)dt * p.o_sl * es, row4 = 4 * p.o_sl * es;
            const float *te = reinterpret_cast<const float *>(smem + M::oTe) + t;
            const uint32_t zrow = (uint32_t)(M::kX + M::kY) + 128u * t;
            const uint32_t zcol = (uint32_t)(M::kX + M::kY) + 128u * (32 * (warp - R::kE0) + r4);
#pragma unroll 1
            for (int c = 0; c < nc; ++c, o += step, ring.next()) {
                const int b = c & 1, n = c == cpart ? npart : kC, nw = n - 32 * (warp - R::kE0) - r4;
                const f2 rf = f2_splat(t < n ? te[rev ? kC - n : 0] : 0.0f);
                const uint32_t oa = lanes + col_oa(b), ob = lanes + kColOb;
                const uint32_t tile = sbase + (uint32_t)(ring.st * M::kStage);
                // 128 bytes of every row from the tile to o, `off` bytes into the row; the tile is
                // free as soon as it is read
                auto copy_out = [&](int off, bool last) {
                    __syncwarp();
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = lds128(tile + zcol + 512u * i + (uint32_t)((q ^ ((4 * i + r4) & 7)) << 4));
                    if (last) fence_async_smem();  // (its next use is a copy's)
                    __syncwarp();
                    if (last && lane == 0) bar_arrive(bar(kBarZFree + ring.st));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (4 * i < nw && off + 16 * q < cols * es) *reinterpret_cast<uint4 *>(o + off + i * row4) = v[i];
                };
                if (!wait_all(kBarO + b, c >> 1)) break;
                tc_after();
                if (es == 2) {
                    uint32_t r[kZ / 2];
#pragma unroll
                    for (int i = 0; i < kZ; i += 16) {
                        float v[16], w[16];
                        tmem_ld2x16(oa + (uint32_t)i, ob + (uint32_t)i, v, w);
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
                            r[(i + j) >> 1] = pack2(f2_fma(rf, f2_make(w[j], w[j + 1]), f2_make(v[j], v[j + 1])));
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(kBarOFree + b));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sts128(tile + zrow + (uint32_t)((i ^ (t & 7)) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    copy_out(0, true);
                } else {
#pragma unroll 1
                    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            float v[16], w[16];
                            tmem_ld2x16(oa + (uint32_t)(32 * hf + i), ob + (uint32_t)(32 * hf + i), v, w);
#pragma unroll
                            for (int j = 0; j < 16; j += 2)
                                f2_split(f2_fma(rf, f2_make(w[j], w[j + 1]), f2_make(v[j], v[j + 1])), v[j], v[j + 1]);
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                sts128(tile + zrow + (uint32_t)((((i + j) >> 2) ^ (t & 7)) << 4), __float_as_uint(v[j]),
                                       __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]), __float_as_uint(v[j + 3]));
                        }
                        if (hf == 1) {
                            tc_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive(bar(kBarOFree + b));
                        }
                        copy_out(128 * hf, hf == 1);
                    }
                }
            }
        }
    } else if (warp < R::kS0) {
        // ================================= group V =================================
        constexpr int VT = 32 * R::kV, kItems = kC * 8 / VT / 2;  // 16-byte items a thread has in each half
        const int gt = tid - 32 * R::kV0;
        const uint32_t zs = sbase + M::oZs + 16u * gt;
        const float *tv0 = reinterpret_cast<const float *>(smem + M::oTv) + (gt >> 3);
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nc && ok; ++c, ring.next()) {
            const int st = ring.st, n = c == cpart ? npart : kC;
            const uint32_t y = sbase + (uint32_t)(st * M::kStage + M::kX), z = y + M::kY + 16u * gt;
            if (!wait_all(kBarZ + st, ring.use)) break;
            if (n < kC) {
                // the rows behind the sequence, before any product reads them
                if (!wait_all(kBarY + st, ring.use)) break;
#pragma unroll 1
                for (int i = n * 8 + gt; i < kC * 8; i += VT) {
                    sts128(y + M::kY + 16 * i, 0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < DX / 64; ++j) sts128(y + j * 16384 + 16 * i, 0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarClear));
            }
            const float *tv = tv0 + (rev ? 0 : kC - n);
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                if (c > 0 && !(ok = wait_all(kBarZsFree + hf, c - 1))) break;
#pragma unroll 1
                for (int it = kItems * hf; it < kItems * (hf + 1); ++it) {
                    // 8 columns of row VT / 8 it + gt / 8
                    uint4 q = make_uint4(0, 0, 0, 0), hi, mid, lo;
                    float w = 0.0f;
                    if (VT / 8 * it + (gt >> 3) < n) {
                        w = tv[VT / 8 * it];
                        q = lds128(z + 16u * VT * it);
                    }
                    const f2 w2 = f2_splat(w);
                    split3(w2, q.x, hi.x, mid.x, lo.x);
                    split3(w2, q.y, hi.y, mid.y, lo.y);
                    split3(w2, q.z, hi.z, mid.z, lo.z);
                    split3(w2, q.w, hi.w, mid.w, lo.w);
                    sts128(zs + 16u * VT * it, hi.x, hi.y, hi.z, hi.w);
                    sts128(zs + 16u * VT * it + M::kZb, mid.x, mid.y, mid.z, mid.w);
                    sts128(zs + 16u * VT * it + 2 * M::kZb, lo.x, lo.y, lo.z, lo.w);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(bar(kBarZs + hf));
                    if (hf == 1) bar_arrive(bar(kBarZFree + st));
                }
            }
        }
    } else {
        // ================================= group S =================================
        // dx <= 64: KV's second 64 rows repeat the first, so warps 2 and 3 take the
        // second 32 columns of rows 0..63
        constexpr int NCOL = DX == 64 ? 32 : 64;
        const int w = warp - R::kS0, row = (DX == 64 ? 32 * (w & 1) : 32 * w) + lane, c0 = DX == 64 ? 32 * (w >> 1) : 0;
        const uint32_t kv = tmem + ((uint32_t)(32 * w) << 16) + kColKv + (uint32_t)c0;
        f2 S[NCOL / 2];
        const int64_t blk = p.dx * (int64_t)p.dz;
        {
            const int64_t hb = (int64_t)h * blk, sb = a.H * blk;
            auto add = [&](const float *from, int64_t sr, int64_t sc, float decay) {
                const bool in = from && row < p.dx;
                const int64_t at = row * sr + (kZ * zb + c0) * sc;
#pragma unroll
                for (int i = 0; i < NCOL; i += 2) {
                    const bool use = in && kZ * zb + c0 + i < p.dz;  // (dz is a multiple of 8)
                    const float u = use ? from[at + i * sc] : 0.0f, v = use ? from[at + (i + 1) * sc] : 0.0f;
                    S[i / 2] = f2_fma(f2_splat(decay), S[i / 2], f2_make(u, v));
                }
            };
#pragma unroll
            for (int i = 0; i < NCOL / 2; ++i) S[i] = f2_splat(0.0f);
            if constexpr (!kStates) {
                add(p.s0 ? p.s0 + pl.seq * sb + hb : nullptr, p.s0_sr, p.s0_sc, 0.0f);
                // the earlier segments' own states, in the order of work
                if (p.seg_states)
#pragma unroll 1
                    for (int j = rev ? pl.ng - 1 : 0; j != pl.g; j += rev ? -1 : 1) {
                        const int n = pl.len - j * a.seg < a.seg ? pl.len - j * a.seg : a.seg;
                        add(p.seg_states + (int64_t)(slot - pl.g + j) * sb + hb, p.seg_sr, p.seg_sc, expf((float)n * g));
                    }
            }
        }
        // lam^n S as keep S + part S, rounded once: with lam^n >= 1/2 part = lam^n - 1 keeps the
        // bits of a slow decay over many chunks
        const float m = expm1f((float)kC * g), mp = expm1f((float)npart * g);
        const float keep = m >= -0.5f ? 1.0f : 0.0f, part = m >= -0.5f ? m : expf((float)kC * g);
        const float keepp = mp >= -0.5f ? 1.0f : 0.0f, partp = mp >= -0.5f ? mp : expf((float)npart * g);
        const uint32_t dst = sbase + M::oS + 128u * row;
        const int x8 = row & 7, j0 = c0 >> 3;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            if constexpr (!kStates) {
                if (c > 0 && !(ok = wait_all(kBarOB, c - 1))) break;
#pragma unroll
                for (int i = 0; i < NCOL; i += 8)
                    sts128(dst + (uint32_t)(((j0 + (i >> 3)) ^ x8) << 4), pack2(S[i / 2]), pack2(S[i / 2 + 1]),
                           pack2(S[i / 2 + 2]), pack2(S[i / 2 + 3]));
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(kBarS));
            }
            // lam^n S while KV is formed (before the wait: KV's columns are needed for the next chunk)
            const f2 k2 = f2_splat(c == cpart ? keepp : keep), p2 = f2_splat(c == cpart ? partp : part);
#pragma unroll
            for (int i = 0; i < NCOL / 2; ++i) S[i] = f2_fma(p2, S[i], f2_mul(k2, S[i]));
            if (!(ok = wait_all(kBarKV, c))) break;
            tc_after();
#pragma unroll
            for (int i = 0; i < NCOL; i += 8) {
                float hi[8], mid[8], lo[8];
                tmem_ld3x8(kv + i, kv + kZ + i, kv + 2 * kZ + i, hi, mid, lo);
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    S[(i + j) / 2] = f2_add(S[(i + j) / 2], f2_add(f2_make(hi[j], hi[j + 1]),
                                                                   f2_add(f2_make(mid[j], mid[j + 1]), f2_make(lo[j], lo[j + 1]))));
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
                if (kZ * zb + c0 + i < p.dz) *reinterpret_cast<ulonglong2 *>(f + i) = make_ulonglong2(S[i / 2], S[i / 2 + 1]);
        }
    }

    tc_before();
    __syncthreads();
    if (warp == R::kQk) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
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
    linattn_tc_kernel<DX, kStates><<<(unsigned)grid, Roles<DX>::kThreads, bytes, stream>>>(a, maps);
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
    // (forward: and a copy of the initial states, for a call that overwrites them)
    return s.segmented ? (size_t)(bwd ? 2 * s.slots : s.slots + batch) * H * dk * dv * sizeof(float) : 0;
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
        // (problem 2; problem 1 reads it with rows and columns exchanged, as it does dfinal)
        TcArgs s = a;
        float *st = static_cast<float *>(workspace);
        s.np = la.np == 1 ? 1 : 2;
        s.units = 0;
        for (int k = 0; k < s.np; ++k) {
            const TcProblem &p = a.p[2 * k];
            s.p[k] = p;
            s.p[k].fin = st + k * sp.slots * la.H * p.dx * p.dz;
            s.units += p.nzb;
        }
        const cudaError_t e = dxmax <= 64 ? launch_t<64, true>(s, maps, sp.slots, stream)
                                          : launch_t<128, true>(s, maps, sp.slots, stream);
        if (e != cudaSuccess) return e;
        for (int i = 0; i < la.np; ++i) {
            a.p[i].seg_states = s.p[i == 0 ? 0 : 1].fin;
            a.p[i].seg_sr = i == 1 ? 1 : a.p[i].dz;
            a.p[i].seg_sc = i == 1 ? a.p[i].dx : 1;
        }
        if (a.p[0].s0 && a.p[0].s0 == a.p[0].fin) {
            // a sequence's last segment may end before its others begin
            const size_t n = (size_t)la.batch * la.H * a.p[0].dx * a.p[0].dz;
            float *copy = st + (size_t)sp.slots * la.H * a.p[0].dx * a.p[0].dz;
            const cudaError_t ec = cudaMemcpyAsync(copy, a.p[0].s0, n * sizeof(float), cudaMemcpyDeviceToDevice, stream);
            if (ec != cudaSuccess) return ec;
            a.p[0].s0 = copy;
        }
    }
    return dxmax <= 64 ? launch_t<64, false>(a, maps, sp.slots, stream) : launch_t<128, false>(a, maps, sp.slots, stream);
}

}  // namespace ms

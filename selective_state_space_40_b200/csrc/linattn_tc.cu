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
// An item is one (segment of a sequence, head, 64 columns of z); a CTA walks its
// chunks with the state in registers. The kernel is persistent, one CTA per SM, and
// its roles run on from one item into the next, so a CTA's set-up and the filling
// of its pipeline are paid once. The roles, each waiting for its own inputs only:
//   one warp finds the items, lays out what they need and loads their tiles (tensor
//   copies, 128-byte swizzle, NS stages); one warp each issues QK, KV, and O_a with O_b;
//   group P  weights QK into P (tensor memory, in place);
//   group E  adds up O_a and lam^.. O_b and writes o;
//   group V  forms Z', and clears the rows of a chunk's Y and Z that are behind
//            the sequence;
//   group S  keeps S (a thread: one row, or half of one), adds KV, and hands
//            its bf16 form to the next chunk's O_b.
// KV takes the three parts of Z' as one product of N = 192 (24 products of N = 64
// read Y three times, and took 1900 clocks a chunk against 1200).
//
// Measured at one chain per SM (148 heads, 4096 tokens): a chunk takes 2.0 us at dk =
// dv = 64 (64 KB from and to HBM: 4.7 TB/s), 2.8 us at dk = 128, dv = 64 (96 KB, 5.1
// TB/s); 8 x 2048 tokens x 24 heads of 64 take 64 us. What bounds it is the roles'
// instructions, some 7000 a chunk, half of the issue slots, and the instruction cache
// they share: loops unrolled twice as far took 10 to 25 % more, a third and fourth stage
// with a ring of its own for Z nothing less.
//
// Three ways to cut the work, by the number of (sequence, head, column block)s, each
// of which is a chain of chunks (see plan_of):
//   kWhole    an item is a whole sequence;
//   kChained  a sequence is several items, and the state goes from one to the next
//             through the workspace: items are claimed in ticket order, all first
//             segments before all second ones, so an item's predecessor was claimed
//             before it and mostly has ended, and every wait ends. Evens out chains
//             that do not divide by the SMs.
//   kStates   too few chains to fill the SMs: a first pass forms each segment's own
//             state from zero, and the main pass starts every segment from the initial
//             state and the earlier ones' own.
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
// The warps of a CTA: group P, group V, group S, group E (four each), one that loads and three that issue.
struct R {
    static constexpr int kV0 = 4, kS0 = 8, kE0 = 12, kLoad = 16, kQk = 17, kKv = 18, kO = 19, kThreads = 640;
};
constexpr uint32_t kSpinTries = 1u << 20;   // tries of a barrier
constexpr uint32_t kFlagTries = 1u << 22;   // polls of a predecessor's flag

// tensor memory: two buffers of QK (P takes its first 64 columns, O_a its last
// 64), O_b, and the three parts of KV
__host__ __device__ constexpr uint32_t col_qk(int b) { return 128u * b; }
__host__ __device__ constexpr uint32_t col_oa(int b) { return 128u * b + 64u; }
constexpr uint32_t kColOb = 256, kColKv = 320;
// The first pass of kStates has no QK and O. So KV has two buffers, in the columns and with the barriers of QK and
// P, the warps of P form half of Z', those of E keep half of the state at dx = 128, and there are three stages
// (65536 tokens, 16 heads of 128: 190 -> 183, 150, 138 us of that pass with two buffers, P's and E's warps; two buffers
// of Z' at the cost of a stage: 178).
__host__ __device__ constexpr uint32_t col_kv(bool own, int cc) { return own ? 256u * (cc & 1) : kColKv; }

struct TcProblem {
    int mx, my, mz;  // tensor maps of x, y, z
    int xg, yg, zg, dx, dz, rev, o_f32;
    float ws, ps, ro;
    const float *s0;          // entering states: block (sequence, head) of dx * dz, element (i, j) at i s0_sr + j s0_sc
    const float *seg_states;  // segments' own states, blocks (slot, head), or null
    float *fin;               // leaving states [batch, H, dx, dz], or (first pass of kStates) [slots, H, dx, dz]
    int64_t s0_sr, s0_sc, seg_sr, seg_sc;  // seg_states' strides
    void *o;
    int64_t o_sb, o_sl, o_sh;
    int nzb;          // blocks of kZ columns of z
};
enum { kWhole = 0, kChained = 1, kStates = 2 };
struct TcArgs {
    const float *log_decay;
    const int32_t *seq_start;
    int *status;
    int batch, seqlen, total, H;
    int seg;    // tokens per segment (a multiple of kC)
    int nseg;   // segments per sequence (dense)
    int np, units;  // units: sum of nzb
    // kChained: the ticket, a flag per chain (warps of group S that have handed its state on), the states
    int *ticket, *flags;
    float *chain;
    TcProblem p[kLaMaxProblems];
};
struct TcMaps {
    CUtensorMap m[4];
};

// shared memory (bytes)
// what the roles need of an item
struct Item {
    int valid, seq, h, pi, zb;
    int row0, nc;      // the first row of chunk c is row0 + c * (rev ? -kC : kC)
    int cpart, npart;  // the chunk that is not full (-1: none), and its tokens
    int j, last;       // segment in the order of work, and whether it is the last of them
    int slot0;         // number of the sequence's first segment
    int ng, len;       // the sequence's segments and tokens
    int unit, pad;
};
template <int DX, bool kOwn>
struct Smem {
    static constexpr int kX = kOwn ? 0 : kC * DX * 2;
    static constexpr int kY = kC * DX * 2;
    static constexpr int kZb = kC * kZ * 2;
    static constexpr int kStage = kX + kY + kZb;
    static constexpr int kStages = DX == 64 || kOwn ? 3 : 2;
    static constexpr int oZs = kStages * kStage;               // three parts of Z'
    static constexpr int oS = oZs + 3 * kZb;                   // S in bf16
    // states on their way, a part per warp of group S: at dx = 128 the warp's own rows of the S tile
    static constexpr int oMove = DX == 64 ? oS + DX * kZ * 2 : oS;
    static constexpr bool kS2 = kOwn && DX == 128;             // eight warps keep the state: group S, and E's
    static constexpr int oItem = oMove + (kS2 ? 2 : 1) * DX * kZ * 2;  // two items
    // two items' tables: lam^n, n = 0..128; lam^|d| at 31 + d, d = t - s, 0 on the masked side;
    // lam^(31-c), in reverse lam^c, c < 32
    static constexpr int oTab = oItem + 2 * (int)sizeof(Item);
    static constexpr int kPw = 0, kDiag = 132, kCf = kDiag + 64, kTab = kCf + 32;  // floats
    static constexpr int oBar = oTab + 2 * kTab * 4;
    static constexpr int kBytes = oBar + 8 * 48 + 16;
};
enum {
    kBarX = 0,        // [3] a stage's X, Y, Z tiles are in
    kBarY = 3,
    kBarZ = 6,
    kBarXFree = 9,    // [3] what uses the stage's X (QK, O_b), Y (QK, KV), Z (group V, O_a, then group E) is done
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
    kBarClear = 34,   // [3] the rows behind the sequence are cleared (of a stage's chunk that has some)
    kBarItem = 37,    // [2] an item is laid out
    kBarItemFree = 39,  // [2] every role is done with it
    kBarZRead = 41,   // [3] group V has read the stage's Z
    kBarEnd = 44,     // [3] nothing of an issuing warp is in flight
    kNumBars = 47
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
// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0u;
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

__device__ __forceinline__ int ld_acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Segments of sequence i (0 where its offsets are out of order), its first row,
// length, and the number of its first segment's slot: dense, i * nseg; packed,
// floor(first row / seg) + i, which gives each sequence as many numbers as it has
// segments or more.
__device__ __forceinline__ int segments_of(const TcArgs &a, int i, int &row0, int &len, int &slot0) {
    row0 = 0;
    len = a.seqlen;
    slot0 = i * a.nseg;
    if (a.seq_start) {
        const int s = a.seq_start[i], e = a.seq_start[i + 1];
        if (s < 0 || e < s || e > a.total) return 0;
        row0 = s;
        len = e - s;
        slot0 = s / a.seg + i;
    }
    return len > a.seg ? (len - 1) / a.seg + 1 : 1;
}

// The items in their order: all sequences' first segments (in the order of work),
// then all second ones, and so on; within, sequence, head, unit. The first pass of
// kStates leaves out each sequence's last. A warp asks for increasing numbers, and
// gets the same answer in every lane.
template <bool kOwn>
struct Finder {
    // packed: the level, a block of 32 sequences, and the (sequence, segment)s before it and before the level
    int j = 0, i0 = 0, before = 0, level0 = 0;
    __device__ __forceinline__ bool find(const TcArgs &a, int n, int lane, Item &it) {
        it.unit = n % a.units;
        n /= a.units;
        it.h = n % a.H;
        n /= a.H;
        int row0, len, slot0, ng;
        if (a.seq_start == nullptr) {
            it.seq = n % a.batch;
            j = n / a.batch;
            if (j >= a.nseg - (kOwn ? 1 : 0)) return false;
        } else {
            for (;;) {
                const int i = i0 + lane;
                const unsigned m =
                    __ballot_sync(0xffffffffu, i < a.batch && segments_of(a, i, row0, len, slot0) - (kOwn ? 1 : 0) > j);
                if (n - before < __popc(m)) {
                    it.seq = i0 + (int)__fns(m, 0, n - before + 1);
                    break;
                }
                before += __popc(m);
                i0 += 32;
                if (i0 >= a.batch) {
                    if (before == level0) return false;  // no sequence has so many segments
                    level0 = before;
                    i0 = 0;
                    ++j;
                }
            }
        }
        ng = segments_of(a, it.seq, row0, len, slot0);
        int zb = it.unit, pi = 0;
        while (zb >= a.p[pi].nzb) zb -= a.p[pi++].nzb;
        const bool rev = a.p[pi].rev != 0;
        const int seg0 = (rev ? ng - 1 - j : j) * a.seg;
        const int ntok = len - seg0 < a.seg ? len - seg0 : a.seg;
        it.pi = pi;
        it.zb = zb;
        it.nc = (ntok + kC - 1) / kC;
        it.npart = ntok % kC == 0 ? kC : ntok % kC;
        it.cpart = it.npart == kC ? -1 : rev ? 0 : it.nc - 1;
        it.row0 = row0 + seg0 + (rev && it.nc > 0 ? (it.nc - 1) * kC : 0);
        it.j = j;
        it.last = j == ng - 1;
        it.slot0 = slot0;
        it.ng = ng;
        it.len = len;
        return true;
    }
};

// (0 * -inf must be 0; NaN stays)
__device__ __forceinline__ float log_decay_of(const TcArgs &a, int h) {
    const float g = __ldg(a.log_decay + h);
    return g < -1e30f ? -1e30f : g;
}

// What an item may touch lies inside the arrays: its rows, its place among them, its slot of states.
template <bool kOwn>
__device__ bool item_ok(const TcArgs &a, const Item &it) {
    if (it.pi < 0 || it.pi >= a.np || it.zb < 0 || it.zb >= a.p[it.pi].nzb || it.seq < 0 || it.seq >= a.batch || it.h < 0 ||
        it.h >= a.H || it.nc < 0 || it.j < 0 || it.j >= it.ng)
        return false;
    const int slots = a.seq_start ? a.total / a.seg + a.batch : a.batch * a.nseg;
    if (kOwn && (it.slot0 < 0 || it.slot0 + it.ng > slots)) return false;
    if (it.nc == 0) return true;
    const int part = it.cpart >= 0 ? it.npart : kC, steps = (it.nc - 1) * kC;
    const int lo = a.p[it.pi].rev ? it.row0 - steps : it.row0;
    const int hi = a.p[it.pi].rev ? it.row0 + part : it.row0 + steps + part;
    return lo >= 0 && hi <= (a.seq_start ? a.total : a.seqlen);
}

// The roles' code is what the SM's instruction cache has to hold at once (five
// groups of warps, each in a loop of its own): with the loops unrolled and the
// call's parameters read inside them, warps waited for instructions half of the
// time. So what a chunk needs is laid out before the loops (tables, addresses,
// steps), and the loops are short.
template <int DX, bool kOwn, int kMode, bool kF32>
__global__ void __launch_bounds__(R::kThreads, 1) linattn_tc_kernel(const __grid_constant__ TcArgs a,
                                                                 const __grid_constant__ TcMaps maps) {
    using M = Smem<DX, kOwn>;
    constexpr int NS = M::kStages, KX = DX / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be the same in all lanes)
    const uint32_t sbase = saddr(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + M::oBar + 8 * 48);
    volatile uint32_t *abort_flag = misc + 1;
    Item *items = reinterpret_cast<Item *>(smem + M::oItem);
    float *tabs = reinterpret_cast<float *>(smem + M::oTab);

    const uint32_t bars = sbase + (uint32_t)M::oBar;
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            int n = 1;
            if (i >= kBarXFree && i < kBarYFree) n = 2;
            else if (i >= kBarYFree && i < kBarZFree) n = kOwn ? 1 : 2;
            else if (i >= kBarZFree && i < kBarQK) n = kOwn ? 8 : 4;  // the warps of E, of V where there is no E
            else if (i >= kBarP && i < kBarO) n = M::kS2 ? 8 : 4;
            else if ((i >= kBarOFree && i < kBarZs) || i == kBarKVFree || i == kBarS) n = 4;
            else if ((i >= kBarZs && i < kBarZsFree) || (i >= kBarClear && i < kBarItem)) n = 4;
            else if (i >= kBarZRead && i < kBarEnd) n = 4;
            else if (i >= kBarItemFree && i < kBarZRead) n = M::kS2 ? 17 : kOwn ? 13 : 19;  // every role's warps
            bar_init(bars + 8 * i, n);
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
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](int i, int k) { return bar_wait(bar(i), (uint32_t)k, abort_flag, a.status); };
    auto wait_all = [&](int i, int k) { return __all_sync(0xffffffffu, wait(i, k)) != 0; };  // whole warps: one answer
    // every product that an issuing warp has in flight completes before the tensor memory is freed
    auto drain = [&](int i) {
        if (elect_one()) mma_commit(bar(kBarEnd + i));
        __syncwarp();
        for (uint32_t k = 0; k < kSpinTries && !bar_try(bar(kBarEnd + i), 0u); ++k) {}
    };
    // stages go round: st = c % NS, and use = c / NS counts the rounds
    struct Ring {
        int st = 0, use = 0;
        __device__ __forceinline__ void next() {
            if (++st == NS) st = 0, ++use;
        }
    } ring;

    // The items one after another: wait for one, read it, run `body`, let it go.
    // cc counts a role's chunks over all items: barriers go by it.
    int cc = 0;
    auto each_item = [&](auto body) {
#pragma unroll 1
        for (int i = 0;; ++i) {
            if (!wait_all(kBarItem + (i & 1), i >> 1)) return false;
            const Item &it = items[i & 1];
            if (!it.valid) return true;
            if (!body(it, tabs + (i & 1) * M::kTab)) return false;
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kBarItemFree + (i & 1)));
        }
    };

    if (warp == R::kLoad) {
        // ============================ items and loads ============================
        if (blockIdx.x == 0 && a.seq_start && a.status)
            for (int i = lane; i < a.batch; i += 32) {
                int row0, len, slot0;
                if (segments_of(a, i, row0, len, slot0) == 0) atomicOr(a.status, MS_ERR_SHAPE);
            }
        Finder<kOwn> finder;
        bool ok = true;
        int sent[3] = {0, 0, 0};  // copies of Y, Z, X issued
        int ticket = 0, next = 0;
        if (kMode == kChained && lane == 0) next = atomicAdd(a.ticket, 1);
#pragma unroll 1
        for (int i = 0; ok; ++i) {
            if (kMode == kChained) {
                ticket = __shfl_sync(0xffffffffu, next, 0);
                if (lane == 0) next = atomicAdd(a.ticket, 1);
            } else {
                ticket = (int)(blockIdx.x + (unsigned)i * gridDim.x);
            }
            Item it;
            const bool valid = finder.find(a, ticket, lane, it);
            it.valid = valid && MS_CHECK(a.status, item_ok<kOwn>(a, it)) ? 1 : 0;
            if (i >= 2) ok = __all_sync(0xffffffffu, wait(kBarItemFree + (i & 1), (i >> 1) - 1)) != 0;
            if (!ok) break;
            if (valid) {
                const TcProblem &p = a.p[it.pi];
                float *tab = tabs + (i & 1) * M::kTab;
                const float g = log_decay_of(a, it.h);
                for (int k = lane; k <= kC; k += 32) tab[M::kPw + k] = expf((float)k * g);
                const float w = p.ps * expf((float)lane * g);
                tab[M::kDiag + 31 + lane] = p.rev && lane > 0 ? 0.0f : w;
                if (lane > 0) tab[M::kDiag + 31 - lane] = p.rev ? w : 0.0f;
                tab[M::kCf + (p.rev ? lane : 31 - lane)] = expf((float)lane * g);
            }
            if (lane == 0) items[i & 1] = it;
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kBarItem + (i & 1)));
            if (!valid) break;
            if (lane == 0) {
                const TcProblem &p = a.p[it.pi];
                const CUtensorMap *mx = &maps.m[p.mx], *my = &maps.m[p.my], *mz = &maps.m[p.mz];
                const int b = a.seq_start ? 0 : it.seq, z0 = kZ * it.zb, dt = p.rev ? -kC : kC;
                const int hx = it.h / p.xg, hy = it.h / p.yg, hz = it.h / p.zg;
                int t = it.row0;
#pragma unroll 1
                for (int c = 0; c < it.nc; ++c, t += dt, ring.next()) {
                    const int st = ring.st, use = ring.use;
                    const uint32_t dst = sbase + (uint32_t)(st * M::kStage);
                    if (use > 0 && !(ok = wait(kBarYFree + st, use - 1))) break;
                    bar_arrive_tx(bar(kBarY + st), (uint32_t)M::kY);
#pragma unroll
                    for (int q = 0; q < DX / 64; ++q) tma_load4(my, dst + M::kX + q * 16384, bar(kBarY + st), 64 * q, hy, t, b);
                    ++sent[0];
                    if (use > 0 && !(ok = wait(kBarZFree + st, use - 1))) break;
                    bar_arrive_tx(bar(kBarZ + st), (uint32_t)M::kZb);
                    tma_load4(mz, dst + M::kX + M::kY, bar(kBarZ + st), z0, hz, t, b);
                    ++sent[1];
                    if constexpr (!kOwn) {
                        if (use > 0 && !(ok = wait(kBarXFree + st, use - 1))) break;
                        bar_arrive_tx(bar(kBarX + st), (uint32_t)M::kX);
#pragma unroll
                        for (int q = 0; q < DX / 64; ++q) tma_load4(mx, dst + q * 16384, bar(kBarX + st), 64 * q, hx, t, b);
                        ++sent[2];
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // when stopping, the copies issued have landed before the CTA ends
        for (int q = 0; q < 3 && !ok && lane == 0; ++q)
            for (int i = sent[q] < NS ? 0 : sent[q] - NS; i < sent[q]; ++i)
                for (uint32_t k = 0;
                     k < kSpinTries && !bar_try(bar((q == 0 ? kBarY : q == 1 ? kBarZ : kBarX) + i % NS), (uint32_t)(i / NS) & 1u); ++k) {}
    } else if (warp == R::kQk) {
        if constexpr (!kOwn) {
            const uint64_t dx0 = sdesc(sbase, 0), dy0 = sdesc(sbase + M::kX, 0);
            uint32_t cleared = 0;  // per stage, the parity of its cleared chunks
            each_item([&](const Item &it, const float *) {
                const int nc = it.nc, cpart = it.cpart;
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ++cc, ring.next()) {
                    const int b = cc & 1, st = ring.st;
                    if (!wait_all(kBarX + st, ring.use) || !wait_all(kBarY + st, ring.use)) return false;
                    if (c == cpart) {
                        if (!wait_all(kBarClear + st, (int)(cleared >> st) & 1)) return false;
                        cleared ^= 1u << st;
                    }
                    if (cc >= 2 && !wait_all(kBarOFree + b, (cc - 2) >> 1)) return false;
                    tc_after();
                    if (elect_one()) {
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
                    __syncwarp();
                }
                return true;
            });
            drain(0);
        }
    } else if (warp == R::kKv) {
        // dx <= 64: the second 64 rows of the product repeat the first
        const uint64_t dy0 = sdesc(sbase + M::kX, DX == 64 ? 0 : 16384), dz = sdesc(sbase + M::oZs, M::kZb);
        each_item([&](const Item &it, const float *) {
            const int nc = it.nc;
#pragma unroll 1
            for (int c = 0; c < nc; ++c, ++cc, ring.next()) {
                const int st = ring.st;
                if (!wait_all(kBarY + st, ring.use)) return false;
                if (kOwn ? cc >= 2 && !wait_all(kBarP + (cc & 1), (cc - 2) >> 1) : cc > 0 && !wait_all(kBarKVFree, cc - 1)) return false;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    if (!wait_all(kBarZs + hf, cc)) return false;
                    tc_after();
                    if (elect_one()) {
                        const uint64_t y = dstep(dy0, st * M::kStage + 8192 * hf), z = dstep(dz, 8192 * hf);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma(tmem + col_kv(kOwn, cc), dstep(y, 2048 * k), dstep(z, 2048 * k), idesc(3 * kZ, true, true), hf > 0 || k > 0);
                        mma_commit(bar(kBarZsFree + hf));
                        if (hf == 1) {
                            mma_commit(bar(kOwn ? kBarQK + (cc & 1) : kBarKV));
                            mma_commit(bar(kBarYFree + st));
                        }
                    }
                    __syncwarp();
                }
            }
            return true;
        });
        drain(1);
    } else if (warp == R::kO) {
        if constexpr (!kOwn) {
            const uint64_t dx0 = sdesc(sbase, 0), dz0 = sdesc(sbase + M::kX + M::kY, 0), ds = sdesc(sbase + M::oS, 0);
            each_item([&](const Item &it, const float *) {
                const int nc = it.nc;
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ++cc, ring.next()) {
                    const int b = cc & 1, st = ring.st;
                    if (!wait_all(kBarX + st, ring.use) || !wait_all(kBarZ + st, ring.use) || !wait_all(kBarS, cc) ||
                        (cc > 0 && !wait_all(kBarOFree + (b ^ 1), (cc - 1) >> 1)))
                        return false;
                    tc_after();
                    if (elect_one()) {
                        const uint64_t x = dstep(dx0, st * M::kStage);
#pragma unroll
                        for (int k = 0; k < KX; ++k)
                            mma(tmem + kColOb, dstep(x, (k >> 2) * 16384 + (k & 3) * 32), dstep(ds, 2048 * k),
                                idesc(kZ, false, true), k > 0);
                        mma_commit(bar(kBarOB));
                        mma_commit(bar(kBarXFree + st));
                    }
                    __syncwarp();
                    if (!wait_all(kBarP + b, cc >> 1)) return false;
                    tc_after();
                    if (elect_one()) {
                        const uint64_t z = dstep(dz0, st * M::kStage);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(tmem + col_oa(b), tmem + col_qk(b) + 8u * k, dstep(z, 2048 * k), idesc(kZ, false, true), k > 0);
                        mma_commit(bar(kBarO + b));
                    }
                    __syncwarp();
                }
                return true;
            });
            drain(2);
        }
    } else if (!kOwn && warp < 4) {
        // ================================= group P =================================
        if constexpr (!kOwn) {
            const int t = 32 * warp + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
            each_item([&](const Item &it, const float *tab) {
                // a block of 32 columns before the diagonal: lam^|t - s| from the row's distance to the
                // block's edge (rf, a step per block) and the column's (cf); the block on the diagonal
                // from a table by t - s, one side of which is zeros; behind it, zeros
                const TcProblem &p = a.p[it.pi];
                const bool rev = p.rev != 0;
                const float ps = p.ps;
                const float *cf = tab + M::kCf, *dg = tab + M::kDiag + 31 + lane, *rf0 = tab + M::kPw + (rev ? -t : t - 31);
                const int past0 = rev ? -warp : warp, dpast = rev ? 1 : -1, drf = rev ? 32 : -32, nc = it.nc;
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ++cc) {
                    const uint32_t qk = lanes + col_qk(cc & 1);
                    if (!wait_all(kBarQK + (cc & 1), cc >> 1)) return false;
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
                                const f2 w = f2_splat(ps * *rf);
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
                    if (lane == 0) bar_arrive(bar(kBarP + (cc & 1)));
                }
                return true;
            });
        }
    } else if (!M::kS2 && warp >= R::kE0) {
        // ================================= group E =================================
        if constexpr (!kOwn) {
            const int t0 = 32 * (warp - R::kE0), t = t0 + lane;
            const uint32_t lanes = tmem + ((uint32_t)t0 << 16);
            // A thread holds a row, but stores that touch 32 rows at once keep the load-store unit
            // from everybody else (2000 clocks a chunk, a quarter of the whole): rows go through the chunk's Z tile, which
            // nothing reads any more, and leave 128 bytes of 4 rows at a time.
            const int q = lane & 7, r4 = lane >> 3;
            const uint32_t zrow = (uint32_t)(M::kX + M::kY) + 128u * t;
            const uint32_t zcol = (uint32_t)(M::kX + M::kY) + 128u * (t0 + r4);
            each_item([&](const Item &it, const float *tab) {
                const TcProblem &p = a.p[it.pi];
                const bool rev = p.rev != 0;
                const int nc = it.nc, cpart = it.cpart, npart = it.npart;
                const bool f32 = kF32 && p.o_f32;
                const int es = f32 ? 4 : 2;
                const int bytes = (p.dz - kZ * it.zb < kZ ? p.dz - kZ * it.zb : kZ) * es;  // of a row
                const int64_t at = (a.seq_start ? 0 : (int64_t)it.seq * p.o_sb) + (int64_t)it.h * p.o_sh + kZ * it.zb +
                                   (int64_t)(it.row0 + t0 + r4) * p.o_sl;
                unsigned char *o = static_cast<unsigned char *>(p.o) + at * es + 16 * q;
                const int64_t step = (int64_t)(rev ? -kC : kC) * p.o_sl * es, row4 = 4 * p.o_sl * es;
                const float ro = p.ro, *pw = tab + M::kPw;
#pragma unroll 1
                for (int c = 0; c < nc; ++c, ++cc, o += step, ring.next()) {
                    const int b = cc & 1, n = c == cpart ? npart : kC, nw = n - t0 - r4;
                    const f2 rf = f2_splat(t < n ? ro * pw[rev ? n - 1 - t : t + 1] : 0.0f);
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
                            if (4 * i < nw && off + 16 * q < bytes) *reinterpret_cast<uint4 *>(o + off + i * row4) = v[i];
                    };
                    // (group V may be behind O_a)
                    if (!wait_all(kBarO + b, cc >> 1) || !wait_all(kBarZRead + ring.st, ring.use)) return false;
                    tc_after();
                    if (!f32) {
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
                return true;
            });
        }
    } else if (warp < R::kS0) {
        // ================================= group V =================================
        constexpr int VT = 128, kItems = kC * 8 / VT / 2;  // 16-byte pieces a thread has in each half
        // (the first pass of kStates has no P: its warps are a second group V, each has half of the tokens)
        const int gt = tid & (VT - 1), hf0 = kOwn && warp < R::kV0 ? 1 : 0, hf1 = kOwn ? hf0 + 1 : 2;
        const uint32_t zs = sbase + M::oZs + 16u * gt;
        each_item([&](const Item &it, const float *tab) {
            const TcProblem &p = a.p[it.pi];
            const bool rev = p.rev != 0;
            const int nc = it.nc, cpart = it.cpart, npart = it.npart, dpw = rev ? VT / 8 : -VT / 8;
            const float ws = p.ws;
#pragma unroll 1
            for (int c = 0; c < nc; ++c, ++cc, ring.next()) {
                const int st = ring.st, n = c == cpart ? npart : kC;
                const uint32_t y = sbase + (uint32_t)(st * M::kStage + M::kX), z = y + M::kY + 16u * gt;
                if (!wait_all(kBarZ + st, ring.use)) return false;
                if (n < kC) {
                    // the rows behind the sequence, before any product reads them
                    if (!wait_all(kBarY + st, ring.use)) return false;
#pragma unroll 1
                    for (int i = (n > 64 * hf0 ? n : 64 * hf0) * 8 + gt; i < 64 * 8 * hf1; i += VT) {
                        sts128(y + M::kY + 16 * i, 0, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < DX / 64; ++j) sts128(y + j * 16384 + 16 * i, 0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (!kOwn && lane == 0) bar_arrive(bar(kBarClear + st));
                }
                // the weight of row gt / 8 + VT / 8 k
                const float *pw = tab + M::kPw + (rev ? (gt >> 3) + 1 : n - 1 - (gt >> 3));
#pragma unroll 1
                for (int hf = hf0; hf < hf1; ++hf) {
                    if (cc > 0 && !wait_all(kBarZsFree + hf, cc - 1)) return false;
#pragma unroll 1
                    for (int k = kItems * hf; k < kItems * (hf + 1); ++k) {
                        uint4 q = make_uint4(0, 0, 0, 0), hi, mid, lo;
                        float w = 0.0f;
                        if (VT / 8 * k + (gt >> 3) < n) {
                            w = ws * pw[dpw * k];
                            q = lds128(z + 16u * VT * k);
                        }
                        const f2 w2 = f2_splat(w);
                        split3(w2, q.x, hi.x, mid.x, lo.x);
                        split3(w2, q.y, hi.y, mid.y, lo.y);
                        split3(w2, q.z, hi.z, mid.z, lo.z);
                        split3(w2, q.w, hi.w, mid.w, lo.w);
                        sts128(zs + 16u * VT * k, hi.x, hi.y, hi.z, hi.w);
                        sts128(zs + 16u * VT * k + M::kZb, mid.x, mid.y, mid.z, mid.w);
                        sts128(zs + 16u * VT * k + 2 * M::kZb, lo.x, lo.y, lo.z, lo.w);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(bar(kBarZs + hf));
                        if (kOwn) bar_arrive(bar(kBarZFree + st));
                        else if (hf == 1) bar_arrive(bar(kBarZRead + st));
                    }
                }
            }
            return true;
        });
    } else {
        // ================================= group S =================================
        // dx <= 64: KV's second 64 rows repeat the first, so warps 2 and 3 take the
        // second 32 columns of rows 0..63. In the first pass of kStates at dx = 128 group E's warps take the second 32
        constexpr int NCOL = DX == 64 || M::kS2 ? 32 : 64;
        const int w = warp - R::kS0, row = (DX == 64 ? 32 * (w & 1) : 32 * (w & 3)) + lane;
        const int c0 = DX == 64 ? 32 * (w >> 1) : M::kS2 ? 32 * (w >> 2) : 0;
        const uint32_t kv0 = tmem + ((uint32_t)(32 * (w & 3)) << 16) + (uint32_t)c0;
        const uint32_t dst = sbase + M::oS + 128u * row;
        const int x8 = row & 7, j0 = c0 >> 3;
        // A thread holds a row (or half of one); states come and go through a part of shared memory
        // that is the warp's own, kPc columns at a time, so that memory sees whole 64- or 128-byte pieces of kPr rows
        // (rows straight to and from memory took 30 % of the packed batch's time).
        constexpr int kPc = DX == 64 ? 16 : 32, kPr = 128 / kPc;
        const int row0 = row - lane, pq = lane % (kPc / 4), pr = lane / (kPc / 4);
        const uint32_t pbase = sbase + M::oMove + (uint32_t)(w * 32 * kPc * 4);
        auto piece = [&](int r, int q) {
            return pbase + (uint32_t)(r * kPc * 4 + ((q ^ (DX == 64 ? (r >> 1) & 3 : r & 7)) << 4));
        };
        each_item([&](const Item &it, const float *tab) {
            const TcProblem &p = a.p[it.pi];
            const bool rev = p.rev != 0;
            const int nc = it.nc, cpart = it.cpart, col0 = kZ * it.zb + c0;
            const int64_t blk = p.dx * (int64_t)p.dz, hb = (int64_t)it.h * blk, sb = a.H * blk;
            const float g = log_decay_of(a, it.h);
            const int chain = (it.seq * a.H + it.h) * a.units + it.unit;
            f2 S[NCOL / 2];
#pragma unroll
            for (int i = 0; i < NCOL / 2; ++i) S[i] = f2_splat(0.0f);
            if constexpr (!kOwn) {
                if (DX == 128 && cc > 0 && !wait_all(kBarOB, cc - 1)) return false;  // (the S tile is not read any more)
                if (kMode == kChained && it.j > 0) {
                    // from the previous segment's item, once its four warps have handed it on
                    bool there = true;
                    if (lane == 0) {
                        there = false;
                        for (uint32_t k = 0; k < kFlagTries && !there; ++k) {
                            there = ld_acquire(a.flags + chain) >= 4 * it.j;
                            if (!there && (k & 63u) == 63u && *abort_flag != 0u) break;
                        }
                        if (!there) {
                            if (a.status && *abort_flag == 0u) atomicOr(a.status, MS_ERR_TIMEOUT);
                            *abort_flag = 1u;
                        }
                    }
                    if (!__shfl_sync(0xffffffffu, there, 0)) return false;
                    // (laid out as the threads hold it: 4 columns of all rows)
                    const float4 *from = reinterpret_cast<const float4 *>(a.chain) + ((int64_t)chain * (kZ / 4) + c0 / 4) * DX + row;
#pragma unroll
                    for (int i = 0; i < NCOL; i += 4) {
                        const float4 v = __ldcg(from + (i / 4) * DX);
                        S[i / 2] = f2_make(v.x, v.y);
                        S[i / 2 + 1] = f2_make(v.z, v.w);
                    }
                } else {
                    // the initial state, and (kStates) the earlier segments' own in the order of work,
                    // each with what came before it decayed
#pragma unroll 1
                    for (int j = -1; j < (kMode == kStates ? it.j : 0); ++j) {
                        const float *from = p.s0 ? p.s0 + it.seq * sb + hb : nullptr;
                        int64_t sr = p.s0_sr, sc = p.s0_sc;
                        float decay = 0.0f;
                        if (kMode == kStates && j >= 0) {
                            const int i = rev ? it.ng - 1 - j : j, n = it.len - i * a.seg < a.seg ? it.len - i * a.seg : a.seg;
                            from = p.seg_states + (int64_t)(it.slot0 + i) * sb + hb;
                            sr = p.seg_sr;
                            sc = p.seg_sc;
                            decay = expf((float)n * g);
                        }
                        if (from == nullptr) continue;
                        if (kMode == kStates && sc == 1) {
                            // (few items: the way through shared memory below costs registers in the chunks' loop)
#pragma unroll
                            for (int i = 0; i < NCOL; i += 4) {
                                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                                if (row < p.dx && col0 + i < p.dz) u = *reinterpret_cast<const uint4 *>(from + row * sr + col0 + i);
                                S[i / 2] = f2_fma(f2_splat(decay), S[i / 2], f2_make(__uint_as_float(u.x), __uint_as_float(u.y)));
                                S[i / 2 + 1] = f2_fma(f2_splat(decay), S[i / 2 + 1], f2_make(__uint_as_float(u.z), __uint_as_float(u.w)));
                            }
                        } else if (sc == 1) {  // (and 16-byte aligned: dz is a multiple of 8)
#pragma unroll
                            for (int h0 = 0; h0 < NCOL; h0 += kPc) {
                                uint4 v[32 / kPr];
#pragma unroll
                                for (int i = 0; i < 32 / kPr; ++i) {
                                    const int r = pr + kPr * i;
                                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                                    if (row0 + r < p.dx && col0 + h0 + 4 * pq < p.dz)
                                        v[i] = *reinterpret_cast<const uint4 *>(from + (row0 + r) * sr + col0 + h0 + 4 * pq);
                                }
                                __syncwarp();
#pragma unroll
                                for (int i = 0; i < 32 / kPr; ++i) sts128(piece(pr + kPr * i, pq), v[i].x, v[i].y, v[i].z, v[i].w);
                                __syncwarp();
#pragma unroll
                                for (int i = 0; i < kPc; i += 4) {
                                    const uint4 u = lds128(piece(lane, i / 4));
                                    f2 &a0 = S[(h0 + i) / 2], &a1 = S[(h0 + i) / 2 + 1];
                                    a0 = f2_fma(f2_splat(decay), a0, f2_make(__uint_as_float(u.x), __uint_as_float(u.y)));
                                    a1 = f2_fma(f2_splat(decay), a1, f2_make(__uint_as_float(u.z), __uint_as_float(u.w)));
                                }
                            }
                        } else {
                            const int64_t at = row * sr + col0 * sc;  // (rows are neighbours)
#pragma unroll
                            for (int i = 0; i < NCOL; i += 2) {
                                const bool use = row < p.dx && col0 + i < p.dz;
                                const float u = use ? from[at + i * sc] : 0.0f, v = use ? from[at + (i + 1) * sc] : 0.0f;
                                S[i / 2] = f2_fma(f2_splat(decay), S[i / 2], f2_make(u, v));
                            }
                        }
                    }
                }
            }
            // lam^n S as keep S + part S, rounded once: with lam^n >= 1/2 part = lam^n - 1 keeps the
            // bits of a slow decay over many chunks
            const float m = expm1f((float)kC * g), mp = expm1f((float)it.npart * g);
            const float keep = m >= -0.5f ? 1.0f : 0.0f, part = m >= -0.5f ? m : tab[M::kPw + kC];
            const float keepp = mp >= -0.5f ? 1.0f : 0.0f, partp = mp >= -0.5f ? mp : tab[M::kPw + it.npart];
#pragma unroll 1
            for (int c = 0; c < nc; ++c, ++cc) {
                if constexpr (!kOwn) {
                    if (cc > 0 && !wait_all(kBarOB, cc - 1)) return false;
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
                if (!(kOwn ? wait_all(kBarQK + (cc & 1), cc >> 1) : wait_all(kBarKV, cc))) return false;
                tc_after();
                const uint32_t kv = kv0 + col_kv(kOwn, cc);
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
                if (lane == 0) bar_arrive(bar(kOwn ? kBarP + (cc & 1) : kBarKVFree));
            }
            if (kMode == kChained && !kOwn && !it.last) {
                float4 *to = reinterpret_cast<float4 *>(a.chain) + ((int64_t)chain * (kZ / 4) + c0 / 4) * DX + row;
#pragma unroll
                for (int i = 0; i < NCOL; i += 4)
                    *reinterpret_cast<ulonglong2 *>(to + (i / 4) * DX) = make_ulonglong2(S[i / 2], S[i / 2 + 1]);
                __threadfence();
                __syncwarp();
                if (lane == 0) atomicAdd(a.flags + chain, 1);
            } else if (p.fin && (kOwn || it.last)) {
                const int64_t to = kOwn ? it.slot0 + (rev ? it.ng - 1 - it.j : it.j) : it.seq;
                float *f = p.fin + to * sb + hb + col0 + 4 * pq;
                if (DX == 128 && !kOwn && cc > 0 && !wait_all(kBarOB, cc - 1)) return false;
#pragma unroll
                for (int h0 = 0; h0 < NCOL; h0 += kPc) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kPc; i += 4) {
                        float x, y, z, u;
                        f2_split(S[(h0 + i) / 2], x, y);
                        f2_split(S[(h0 + i) / 2 + 1], z, u);
                        sts128(piece(lane, i / 4), __float_as_uint(x), __float_as_uint(y), __float_as_uint(z), __float_as_uint(u));
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32 / kPr; ++i) {
                        const int r = pr + kPr * i;
                        if (row0 + r < p.dx && col0 + h0 + 4 * pq < p.dz)
                            *reinterpret_cast<uint4 *>(f + (row0 + r) * (int64_t)p.dz + h0) = lds128(piece(r, pq));
                    }
                }
                __syncwarp();
            }
            return true;
        });
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

// How the work is cut (see the top). `chains` runs of chunks over num_sms SMs; a
// round of items takes as long as their chunks, and half a chunk to change over.
struct Plan {
    int mode;
    int64_t seg, nseg, slots;  // tokens per segment, segments per sequence (dense), slots of segments
};
Plan plan_of(int64_t batch, int64_t rows, bool packed, int64_t H, int units, int num_sms) {
    const int64_t chains = std::max<int64_t>(1, batch * H * units);
    // packed: the longest sequence is not known here. kStates goes by the case that one has most rows,
    // kChained by their mean
    const int64_t most = (rows + kC - 1) / kC, mean = packed ? (rows / std::max<int64_t>(1, batch) + kC - 1) / kC : most;
    Plan p{kWhole, 0, 1, batch};
    int64_t chunks = 0;  // per segment
    if (2 * chains <= num_sms) {
        // as many segments as fill the SMs once, twice or three times, of at least four chunks
        double best = (double)most;
        for (int r = 1; r <= 3; ++r) {
            const int64_t n = r * num_sms / chains, len = std::max<int64_t>(4, (most + n - 1) / n);
            const double t = r * (double)(len + 1) * 1.45;  // the first pass takes 0.45 of the main one
            if (len < most && t < best) best = t, chunks = len, p.mode = kStates;
        }
    } else if (chains > num_sms && mean >= 4) {
        // equal chains: the segments per chain that leave the least idle at the end
        auto rounds = [&](int64_t n) { return (n + num_sms - 1) / num_sms; };
        double best = 0.97 * rounds(chains) * (mean + 0.5);
        for (int64_t k = 2; 2 * k <= mean; ++k) {
            const int64_t len = (mean + k - 1) / k;
            const double t = rounds(chains * k) * (len + 0.5);
            if (t < best) best = t, chunks = len, p.mode = kChained;
        }
    }
    if (p.mode == kWhole) {
        p.seg = std::max<int64_t>(1, most + (packed ? 1 : 0)) * kC;
        return p;
    }
    p.seg = chunks * kC;
    p.nseg = packed ? 1 : (rows + p.seg - 1) / p.seg;
    p.slots = packed ? rows / p.seg + batch : batch * p.nseg;
    return p;
}
// Workspace: kStates, the segments' states of one direction (forward; and a copy of the
// initial states, for a call that overwrites them) or two; kChained, ticket and flags, and
// the chains' states.
size_t flag_bytes(int64_t chains) { return ((size_t)(chains + 1) * sizeof(int) + 255) / 256 * 256; }

template <int DX, bool kOwn, int kMode, bool kF32>
cudaError_t launch_t(const TcArgs &a, const TcMaps &maps, int64_t slots, int num_sms, cudaStream_t stream) {
    static SmemOptIn opt_in;
    constexpr int bytes = Smem<DX, kOwn>::kBytes;
    static_assert(bytes <= 232448, "shared memory of a block");
    cudaError_t e = opt_in.ensure(reinterpret_cast<const void *>(linattn_tc_kernel<DX, kOwn, kMode, kF32>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = slots * a.H * a.units;
    if (items > 0x3fffffffLL || a.seg <= 0) return cudaErrorInvalidConfiguration;
    linattn_tc_kernel<DX, kOwn, kMode, kF32>
        <<<(unsigned)std::min<int64_t>(items, num_sms), R::kThreads, bytes, stream>>>(a, maps);
    return cudaGetLastError();
}
template <bool kOwn, int kMode>
cudaError_t launch_dx(int dx, const TcArgs &a, const TcMaps &maps, int64_t slots, int num_sms, cudaStream_t stream) {
    bool f32 = false;  // (some of the outputs)
    for (int i = 0; i < a.np; ++i) f32 = f32 || a.p[i].o_f32;
    if constexpr (!kOwn) {
        if (f32)
            return dx <= 64 ? launch_t<64, false, kMode, true>(a, maps, slots, num_sms, stream)
                            : launch_t<128, false, kMode, true>(a, maps, slots, num_sms, stream);
    }
    return dx <= 64 ? launch_t<64, kOwn, kMode, false>(a, maps, slots, num_sms, stream)
                    : launch_t<128, kOwn, kMode, false>(a, maps, slots, num_sms, stream);
}

}  // namespace

// A chunk costs the same however few of its tokens there are: sequences that have at most
// kFew (packed ones: in all, as the longest is not known here) are left to the recurrence,
// in us at 1, 8, 12 tokens: 64 sequences x 24 heads of 64, forward 21, 39, 51, here 50;
// backward 59, 110, 142, here 145; one sequence of 24 heads 6, 10, 13, here 11; backward of
// 16 x 32 heads of 128 64, 108, 134, here 109.
constexpr int64_t kFew = 8;

bool linattn_tc_applies(const LaArgs &a, bool bf16) {
    const int64_t rows = a.seq_start ? a.total : a.seqlen, batch = a.seq_start ? 1 : a.batch;
    if (!bf16 || rows <= kFew) return false;
    for (int i = 0; i < a.np; ++i) {
        const LaProblem &p = a.p[i];
        const int eo = p.o_f32 ? 4 : 2;
        if (p.dx % 8 || p.dz % 8 || !map_ok(key_x(a, p), batch) || !map_ok(key_y(a, p), batch) ||
            !map_ok(key_z(a, p), batch) || reinterpret_cast<uintptr_t>(p.o) % 16 || (p.o_sb * eo) % 16 ||
            (p.o_sl * eo) % 16 || (p.o_sh * eo) % 16 || reinterpret_cast<uintptr_t>(p.fin) % 16 || reinterpret_cast<uintptr_t>(p.s0) % 16)
            return false;
    }
    return true;
}

size_t linattn_tc_workspace(int64_t batch, int64_t rows, bool packed, int64_t H, int dk, int dv, bool bwd, int num_sms) {
    if (batch < 1 || rows < 1) return 0;
    const int units = bwd ? 2 * zblocks(dk) + zblocks(dv) : zblocks(dv);
    const Plan p = plan_of(batch, rows, packed, H, units, num_sms);
    if (p.mode == kStates) return (size_t)(bwd ? 2 * p.slots : p.slots + batch) * H * dk * dv * sizeof(float);
    if (p.mode == kWhole) return 0;
    const int64_t chains = batch * H * units;
    const int dx = (bwd ? std::max(dk, dv) : dk) <= 64 ? 64 : 128;
    return flag_bytes(chains) + (size_t)chains * dx * kZ * sizeof(float);
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
    const Plan sp = plan_of(la.batch, rows, packed, la.H, a.units, num_sms);
    a.seg = (int)sp.seg;
    a.nseg = (int)sp.nseg;
    if (sp.mode == kWhole) return launch_dx<false, kWhole>(dxmax, a, maps, sp.slots, num_sms, stream);
    if (sp.mode == kChained) {
        const int64_t chains = la.batch * la.H * a.units;
        const size_t fb = flag_bytes(chains);
        a.ticket = static_cast<int *>(workspace);
        a.flags = a.ticket + 1;
        a.chain = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + fb);
        const cudaError_t e = cudaMemsetAsync(workspace, 0, fb, stream);
        if (e != cudaSuccess) return e;
        return launch_dx<false, kChained>(dxmax, a, maps, sp.slots, num_sms, stream);
    }
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
    const cudaError_t e = launch_dx<true, kStates>(dxmax, s, maps, sp.slots, num_sms, stream);
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
    return launch_dx<false, kStates>(dxmax, a, maps, sp.slots, num_sms, stream);
}

}  // namespace ms

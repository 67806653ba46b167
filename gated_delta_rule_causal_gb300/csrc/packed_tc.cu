// The gated delta rule over packed requests on the tcgen05 tensor cores: bf16
// q, k and v, value heads of 128, blocks of 64 tokens. The algebra is that of
// packed_chunk.cu (value heads of 64 and 128, warp-level MMAs), with b's columns in T:
//   T' = (I + A)^-1 diag(b),   U = T' (V - diag(G) K X^T)
//   O = diag(G) Q X^T + P U,   X <- G_63 X + U^T diag(D_63,.) K
// and so is the precision: q, k, v exact; X, G Z, T' and U in two bf16 parts
// wherever the state depends on them; X in Q X^T and P in one.
//
// Work split. A CTA takes one (request, value head) after another, longest
// requests first: the grid has one CTA for each, and a running one takes over
// the next that has not been started (cluster launch control), so that its
// prep and load warps are already at the next request while the chain finishes
// one. The state's 128 rows lie on the 128 tensor-memory lanes, fp32, for the
// whole request, so that every product of the chain is an M = 128 MMA with its
// A operand (X, R = -G Z, U: bf16 parts) in tensor memory too and its B operand
// (K, Q, T', P) in shared memory:
//   Z = X K^T, O = X Q^T  [dv][token],  U = V^T T'^T + R T'^T,
//   X += U' K,  O += U P^T
// Sixteen warps convert between them: thread (row r, part cp) takes a quarter
// of the columns of each product in row r. Two groups of four prep warps
// compute T' and P of the blocks that follow; of the others one issues the
// chain's MMAs, one loads K and Q and issues the prep warps' [K;Q] K^T, one
// copies the outputs out, and one fetches the work, loads V and clears its rows
// behind a request. (Prep warps that did so waited for V, which comes only after
// the outputs of the block before the last: 65536 tokens 457 us for 452, 128
// requests of 100 tokens 160 for 144, of 130 206 for 196; 256 of 40 190 for 195.)
//
// The chain's steps depend on one another, so what bounds a request is their
// latency: three products (Z, R T'^T, U' K) with a conversion after each. High
// parts are published first, so that a product starts while the low ones are
// still formed. V^T T'^T, Q X^T, the scaling of X by G_63 and of O by G, and the
// outputs run in the gaps.
//
// Measured, bf16, d 128: two requests of 8192 tokens, 16 heads (32 CTAs, where the
// blocks of 32 are faster): 430 us, 3.3 us or 6400 clocks a block; 96 requests of
// 65536 tokens together, 16 heads: 452 us; 16 of 8191, 32 heads: 129 us. Of a
// block's clocks MMAs take 2700 (the tensor pipe is 34 % busy), the chain's
// conversions 2500; the prep of a block takes 10000 to 12000, half of which two
// groups make good. Issue slots are 53 % busy, and 8 % of the warps' waiting is
// for instructions: 84 KB of code in which every role has its own loop, where
// code beyond 32 KB was measured to come at 3 clocks an instruction when all of
// it is walked in turn. Smaller was slower all the same, for the two requests of
// 8192: waits as a function (73 KB) 507 us, conversions too 518, MMAs by one
// rolled loop 909.
#include <cuda.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "launch.cuh"
#include "packed.h"
#include "prefill_impl.cuh"
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace la {
namespace packed {
namespace {

using chunk::kmaj;
using chunk::ld_shared_bf16;
using chunk::ld_shared_v4;
using chunk::mnmaj;
using chunk::st_shared_v4;

constexpr int C = 64;                 // tokens per block
constexpr int DV = 128;
constexpr int kConvWarps = 16, kPrepWarps = 4, kGroups = 2;     // two groups of prep warps, every other block each
constexpr int kThreads = 32 * (kConvWarps + kGroups * kPrepWarps + 4);   // + MMA issue, loads, output copies, work
constexpr int kPrepThreads = 32 * kPrepWarps;
constexpr int kOther = kConvWarps + kGroups * kPrepWarps;      // first of the four other warps
constexpr uint32_t kBarPrep = 1;      // named barriers of the prep groups: 1, 2
constexpr int kTiles = 3;             // ring of K and Q tiles (V's has two: its loads are awaited later)
constexpr int kItems = 4;             // ring of work items (the loads run at most three blocks ahead)
constexpr int kAStride = 68;          // floats per row of A
constexpr int kMStride = 80;          // bytes per row of the 32x32 bf16 product between the two merges
constexpr int kVec = 6 * C;           // floats of a block's gate vectors: g, b, G, D_63, and G inside 16 and 32 tokens

template <int DK>
struct TcLayout {
    static constexpr int KA = DK / 64;
    // K and Q of a block: per 64-channel atom K rows 0-63, then Q rows 0-63
    static constexpr uint32_t KQ_BYTES = KA * 16384;
    static constexpr uint32_t V_BYTES = 16384;                  // two atoms [64 t][64]; later the output tile [64 t][128]
    static constexpr uint32_t KQ = 0;                           // [kTiles]
    static constexpr uint32_t V = kTiles * KQ_BYTES;            // [2]
    static constexpr uint32_t TP = V + 2 * V_BYTES;        // [2]: T high, T low, P, each [64 t][64 j]
    static constexpr uint32_t TP_BYTES = 3 * 8192;
    static constexpr uint32_t A = TP + 2 * TP_BYTES;            // per prep group: fp32 [64][kAStride]
    static constexpr uint32_t M = A + kGroups * C * kAStride * 4;   // per prep group: bf16 high, low [32][kMStride bytes]
    static constexpr uint32_t VEC = M + kGroups * 2 * 32 * kMStride;      // [kTiles][kVec] fp32
    static constexpr uint32_t BAR = VEC + kTiles * kVec * 4;
    static constexpr uint32_t BYTES = BAR + 1024;
    // Tensor memory columns. Operands in two bf16 parts lie by steps of 16 along their columns: 8 columns
    // of high parts, then 8 of low ones.
    static constexpr uint32_t COL_X = 0;       // X, fp32 [DK]
    static constexpr uint32_t COL_XP = 128;    // parts of X; of U' once Z and Q X^T are done
    static constexpr uint32_t COL_Z = 256;     // Z; parts of R over it
    static constexpr uint32_t COL_U = 320;     // U; its parts over it
    static constexpr uint32_t COL_O = 384;
    static constexpr uint32_t COL_G = 448;     // [K;Q] K^T
    static constexpr uint32_t TMEM_COLS = 512;
};

// A (request, value head); blocks 0: there is no more.
struct __align__(16) Work {
    int row0, len, slot, fresh;
    int head, khead, blocks, pad;
};

// Barriers, in shared memory.
struct Bars {
    // (A wait for a turn takes the turn two before for it while the one before is not complete, so whoever waits has to
    // know that one complete. A prep group looks at K's arrival only where a block has rows past the request's end:
    // six of them, block nb's at nb % 6, whose turn before, block nb - 6's, the group's T' of block nb - 4 came after.)
    uint64_t kq_full[6], kq_free[kTiles];        // TMA; MMA: every product of the block is done
    uint64_t v_full[2], v_free[2];               // TMA; copier: the output tile over V has left
    uint64_t v_clear[2];                         // work warp: V's rows past the request's end are zero
    uint64_t vec_free[6];                        // converters: the block's vectors are read (16)
    uint64_t ot_full[2];                         // converters: the output tile is written (16)
    uint64_t ready[2], t_free[2], p_free[2];     // prep warps: T', P and vectors (4); MMA: T', P is read
    uint64_t g[2], g_free;                       // MMA: [K;Q] K^T, per prep group; prep warps: it is read (4)
    uint64_t xh, xl, rh, rl, dh, dl, uo;         // converters: parts of X, R, U' and both of U published (16 each)
    uint64_t z, u, o1, dx, o;                    // MMA: Z, U, Q X^T, dX, O done
    uint64_t drain[2];                           // after a failure: MMAs of either issuer are done
    uint64_t item_full[kItems], item_free[kItems];   // work warp; every other warp has read the item (27)
    uint64_t stolen;                             // the answer to a request for more work is here
    uint32_t tmem;
    int abort;
    uint4 answer;
    Work item[kItems];
};

// One lane of a converged warp; MMAs issued under it keep their descriptors in
// uniform registers (a single thread's branch takes 45 clocks per MMA to issue,
// more than the 32 that an M = 128, N = 64 one runs).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

static_assert(sizeof(Bars) <= 1024, "barrier space");

// A block's place among N, stepped instead of divided, and the parity of its turn.
template <int N>
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            phase ^= 1;
        }
    }
};

// 16 lanes x 2 N columns of tensor memory between a warp's registers, by quads: with g = lane / 4,
// c = lane % 4, x[4 i], x[4 i + 1] are columns 8 i + 2 c, + 1 of lane g, x[4 i + 2], x[4 i + 3] of lane g + 8.
template <int N>
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const float* x) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
    static_assert(N == 16 || N == 8, "32 or 16 columns");
    if constexpr (N == 16)
        asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                     ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]) : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float* x) {
    uint32_t* u = reinterpret_cast<uint32_t*>(x);
    static_assert(N == 16 || N == 8, "32 or 16 columns");
    if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]) : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]) : "r"(taddr));
}
// Each thread of the warp writes 8 consecutive columns of its lane.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&u)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}

// Bounded wait of a whole warp on phase `parity` of `bar`: the same answer in every
// lane; false after a failure here or elsewhere (*abort). One try (which waits a while
// itself) in line, the loop out of line: the warps' code, dozens of waits among it,
// has to stay in the instruction cache.
__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, const volatile int* abort) {
    const uint64_t t0 = globaltimer_ns();
    bool ok;
    do {
        ok = mbar_try_wait(bar, parity);
    } while (!ok && !*abort && globaltimer_ns() - t0 <= kWaitLimitNs);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int* abort) {
    bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
    if (!ok) ok = warp_wait_on(bar, parity, abort);
    tc_fence_after();
    return ok;
}

// Whether phase `parity` of `bar` is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// The k-th item of this CTA, for a whole warp; false when there is none (blocks
// 0) or after a failure.
__device__ __forceinline__ bool next_item(Bars* B, int k, Work& w, bool& fail) {
    const int i = k % kItems;
    if (!warp_wait(smem_u32(&B->item_full[i]), (k / kItems) & 1, &B->abort)) {
        fail = true;
        return false;
    }
    w = B->item[i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&B->item_free[i]);
    return w.blocks > 0;
}

// Ask for a CTA of this grid that has not been started to be taken over; the
// answer (16 bytes) completes on `bar`.
__device__ __forceinline__ void steal_request(uint4* answer, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(smem_u32(answer)), "r"(smem_u32(bar)) : "memory");
}
// The block index of the CTA taken over, or -1.
__device__ __forceinline__ int stolen_index(const uint4* answer) {
    int idx;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 x;\n\t"
        "ld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "mov.b32 x, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, r;\n\t"
        "mov.b32 %0, x;\n\t}"
        : "=r"(idx) : "r"(smem_u32(answer)) : "memory");
    return idx;
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z) : "memory");
}

// ---------------------------------------------------------------- prep warps

// Gate vectors of a block from the gates and betas of tokens 2 lane, 2 lane + 1: g, b, the product of
// the gates up to a token, from behind it, and up to it inside its 16 and its 32 tokens.
__device__ __noinline__ void write_gates(float* vec, float2 gn, float2 bn) {
    const int lane = threadIdx.x & 31;
    float pre = gn.x * gn.y, suf = pre, g16 = pre;   // up to / from this lane's pair
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, pre, o), z = __shfl_down_sync(0xffffffffu, suf, o);
        const float x = __shfl_up_sync(0xffffffffu, g16, o);
        if (lane >= o) pre *= y;
        if (lane + o < 32) suf *= z;
        if (o < 8 && (lane & 7) >= o) g16 *= x;
    }
    const float first = __shfl_sync(0xffffffffu, g16, (lane & 16) + 7);   // all of the 32's first 16
    const float g32 = lane & 8 ? first * g16 : g16;
    float b16 = __shfl_up_sync(0xffffffffu, g16, 1), b32 = __shfl_up_sync(0xffffffffu, g32, 1);
    if ((lane & 7) == 0) b16 = 1.f;
    if ((lane & 15) == 0) b32 = 1.f;
    float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
    if (lane == 0) before = 1.f;
    if (lane == 31) after = 1.f;
    float2* v = reinterpret_cast<float2*>(vec) + lane;
    v[0] = gn;
    v[C / 2] = bn;
    v[2 * C / 2] = make_float2(before * gn.x, pre);
    v[3 * C / 2] = make_float2(gn.y * after, after);
    v[4 * C / 2] = make_float2(b16 * gn.x, g16);
    v[5 * C / 2] = make_float2(b32 * gn.x, g32);
}

// A fragment of rows r0.., columns c0.. of an fp32 matrix in shared memory, in two bf16 parts.
__device__ __forceinline__ void load_split(const float* m, int r0, int c0, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const int lane = threadIdx.x & 31;
    const float* p = m + (r0 + (lane >> 2)) * kAStride + c0 + 2 * (lane & 3);
    const float2 y0 = *reinterpret_cast<const float2*>(p), y1 = *reinterpret_cast<const float2*>(p + 8 * kAStride);
    const float2 y2 = *reinterpret_cast<const float2*>(p + 8), y3 = *reinterpret_cast<const float2*>(p + 8 * kAStride + 8);
    split2(y0.x, y0.y, hi[0], lo[0]);
    split2(y1.x, y1.y, hi[1], lo[1]);
    split2(y2.x, y2.y, hi[2], lo[2]);
    split2(y3.x, y3.y, hi[3], lo[3]);
}
// d[2] (16x16) += A B, A and B (two n-tiles) in two parts, the product of the low ones dropped.
__device__ __forceinline__ void mma_split(float (&d)[2][4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
    mma_16816(d[0], ah, bh[0], bh[1]);
    mma_16816(d[1], ah, bh[2], bh[3]);
    mma_16816(d[0], al, bh[0], bh[1]);
    mma_16816(d[1], al, bh[2], bh[3]);
    mma_16816(d[0], ah, bl[0], bl[1]);
    mma_16816(d[1], ah, bl[2], bl[3]);
}
// -d as rows r0.., columns c0.. of T' (swizzled tiles of high and low parts).
__device__ __forceinline__ void store_negated(uint32_t aTH, uint32_t aTL, int r0, int c0, const float (&d)[2][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi, lo;
            split2(-d[i][2 * h], -d[i][2 * h + 1], hi, lo);
            const uint32_t o = sw128_off(r0 + 8 * h + (lane >> 2), c0 / 8 + i) + 4 * (lane & 3);
            st_shared_b32(aTH + o, hi);
            st_shared_b32(aTL + o, lo);
        }
}

// A group of four warps takes every other block: [K;Q] K^T on the tensor cores;
// E_tj = D_tj k_t.k_j (j < t; warps 0, 1) and P_tj = D_tj q_t.k_j (j <= t;
// warps 2, 3) row by row (lane = tensor-memory lane = row; D_tj is a running
// product from the diagonal leftwards); then T' (A = diag(b) E): 16x16 diagonal
// blocks by forward substitution in fp32 (warps 0 and 1, a half-warp each),
// merged twice by T'_21 = -T'_22 (E_21 T'_11) on warp-level MMAs with two bf16
// parts. Two groups because a block's steps wait for one another longer than
// the chain takes for a block.
template <int DK>
__device__ __forceinline__ bool prep_warps(const StepArgs& a, uint8_t* sm, uint32_t sbase, Bars* B, uint32_t tmem) {
    using L = TcLayout<DK>;
    const int lane = threadIdx.x & 31, group = ((threadIdx.x >> 5) - kConvWarps) / kPrepWarps;
    const int pw = (threadIdx.x >> 5) & 3, ptid = threadIdx.x & (kPrepThreads - 1);
    const int gq = lane >> 2, cq = lane & 3;
    const int fr = (lane & 7) + ((lane >> 3) & 1) * 8, fc = lane >> 4;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * pw) << 16);
    const uint32_t bar = kBarPrep + group;
    volatile int* abort = &B->abort;
    auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(smem_u32(b), parity, abort); };
    float* E = reinterpret_cast<float*>(sm + L::A) + group * C * kAStride;
    const uint32_t aM = sbase + L::M + group * 2 * 32 * kMStride;
    const uint32_t aTH = sbase + L::TP + group * L::TP_BYTES, aTL = aTH + 8192, aP = aTH + 16384;

    // gates and betas of tokens 2 lane, 2 lane + 1 of block c (past the end: gate 1, beta 0)
    float2 gn = make_float2(1.f, 1.f), bn = make_float2(0.f, 0.f);
    auto load_gates = [&](const Work& w, int c) {
        const int t = c * C + 2 * lane;
        const size_t i = static_cast<size_t>(w.row0 + t) * a.Hv + w.head;
        gn = make_float2(1.f, 1.f);
        bn = make_float2(0.f, 0.f);
        if (t < w.len) {
            gn.x = __ldg(a.gate + i);
            bn.x = __ldg(a.beta + i);
        }
        if (t + 1 < w.len) {
            gn.y = __ldg(a.gate + i + a.Hv);
            bn.y = __ldg(a.beta + i + a.Hv);
        }
    };
    // T' and P above their diagonal blocks stay zero: the MMAs read whole tiles
    for (int i = ptid; i < static_cast<int>(L::TP_BYTES) / 16; i += kPrepThreads) st_shared_v4(aTH + i * 16, 0, 0, 0, 0);
    named_sync(bar, kPrepThreads);

    Work w = {};
    int items = 0, c = -1;
    bool lost = false;
    auto step = [&]() {   // on to the next block; false when there is none
        if (++c < w.blocks) return true;
        c = 0;
        return next_item(B, items++, w, lost);
    };
    Ring<kTiles> at;   // of block nb of the CTA
    Ring<6> six;
    int nb = 0;
    bool more = step();
    if (group == 1 && more) {
        more = step();
        at.next();
        six.next();
        ++nb;
    }
    if (more && pw == 3) load_gates(w, c);
    // Warps that fail say so at the next barrier of the group and all leave together: a barrier has no limit.
    bool ok = true;
    while (true) {
        const uint32_t kq = sbase + L::KQ + at.s * L::KQ_BYTES;
        float* vec = reinterpret_cast<float*>(sm + L::VEC) + at.s * kVec;
        const int n = w.len - c * C;   // tokens of the block
        if (pw == 3 && more && ok) {   // the slot's vectors of block nb - 3 are read
            const int b3 = six.s < 3 ? six.s + 3 : six.s - 3;   // block nb - 3's place; its turn is the one before from 0 .. 2
            ok = nb < kTiles || wait(&B->vec_free[b3], six.phase ^ (six.s < 3 ? 1 : 0));
            if (ok) write_gates(vec, gn, bn);
        }
        if (more && n < C) {   // rows of the next request (or past the tensor): K (and V) zero, so that they leave the state alone
            ok = ok && wait(&B->kq_full[six.s], six.phase);
            if (ok) {
                for (int i = ptid; i < (C - n) * 8; i += kPrepThreads) {
                    const uint32_t o = sw128_off(n + i / 8, i % 8);
#pragma unroll
                    for (int x = 0; x < L::KA; ++x) st_shared_v4(kq + x * 16384 + o, 0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
        }
        if (named_sync_or(bar, kPrepThreads, !ok || lost)) return false;
        if (!more) return true;
        // The block after next, its gates loaded meanwhile. (Only within the request: the next one may wait for
        // this one's loads, and those for this very block.)
        const bool same = c + 2 < w.blocks;
        if (same) {
            c += 2;
            if (pw == 3) load_gates(w, c);
        }
        ok = ok && wait(&B->g[group], (nb >> 1) & 1);
        // ---- E and P by rows, 16 columns at a time from the right. D at a group's right edge: zero in the
        //      group of the diagonal and right of it, else the row's gates from the edge on -----------
        if (ok) {
            const bool isP = pw >= 2;
            const int hd = pw & 1;   // the half of the columns with this warp's diagonal
            const int t = 32 * hd + lane;
            const float g16 = vec[4 * C + t], g32 = vec[5 * C + t], mid = vec[4 * C + 31];
            // P waits in scratch until the one of block nb - 2 is read: rows 0..31 where the merges' product
            // comes later, rows 32..63 in E's columns 32.. of rows 0..31, which nothing else uses
            const uint32_t ps = hd ? smem_u32(E) + lane * (kAStride * 4) + 128 : aM + lane * 64;
#pragma unroll 1
            for (int c16 = 2 * hd + 1; c16 >= 0; --c16) {
                const int u = 2 * hd + 1 - c16;   // 0, 1: the half of the diagonal; 2, 3: columns 16..31, 0..15 of rows 32..
                float d = u == 0 ? 0.f : u == 1 ? (lane >= 16 ? g16 : 0.f) : u == 2 ? g32 : g32 * mid;
                const int diag = u < 2 ? lane - (16 - 16 * u) : 99;   // the column of the row's diagonal element
                // the last column that counts: what lies right of it, or in rows past the request's end, may be anything
                const int lim = isP ? diag : t < n ? diag - 1 : -1;
                float x[16];
                tmem_ld16(tlane + L::COL_G + 16 * c16, x);
                tmem_ld_wait();
                if (u < 2 || n < C) {
#pragma unroll
                    for (int q4 = 3; q4 >= 0; --q4) {
                        const float4 g4 = *reinterpret_cast<const float4*>(vec + 16 * c16 + 4 * q4);
                        const float gl[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                        for (int i = 3; i >= 0; --i) {
                            const int j = 4 * q4 + i;
                            d = j == diag ? 1.f : d;
                            x[j] = j <= lim ? d * x[j] : 0.f;
                            d *= gl[i];   // the gate of column j itself comes before the columns left of it
                        }
                    }
                } else {   // whole columns left of every diagonal element
#pragma unroll
                    for (int q4 = 3; q4 >= 0; --q4) {
                        const float4 g4 = *reinterpret_cast<const float4*>(vec + 16 * c16 + 4 * q4);
                        const float gl[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                        for (int i = 3; i >= 0; --i) {
                            x[4 * q4 + i] *= d;
                            d *= gl[i];
                        }
                    }
                }
                if (isP) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        st_shared_v4(ps + (2 * c16 + m) * 16, pack_bf16(x[8 * m], x[8 * m + 1]), pack_bf16(x[8 * m + 2], x[8 * m + 3]),
                                     pack_bf16(x[8 * m + 4], x[8 * m + 5]), pack_bf16(x[8 * m + 6], x[8 * m + 7]));
                } else {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        *reinterpret_cast<float4*>(E + t * kAStride + 16 * c16 + 4 * q4) =
                            make_float4(x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->g_free);
            if (isP) {
                if (nb >= 2) ok = wait(&B->p_free[group], ((nb - 2) >> 1) & 1);
#pragma unroll 1
                for (int i = lane; i < 128 << hd && ok; i += 32) {   // this warp's 32 rows of 4 (8) chunks
                    const int row = i >> (2 + hd), ch = i & (3 + 4 * hd);
                    const uint4 y = ld_shared_v4((hd ? smem_u32(E) + row * (kAStride * 4) + 128 : aM + row * 64) + ch * 16);
                    st_shared_v4(aP + sw128_off(32 * hd + row, ch), y.x, y.y, y.z, y.w);
                }
            }
        }
        if (pw < 2 && ok) {
            // ---- diagonal blocks 2 pw and 2 pw + 1 (rows of this warp), lane = (block, column):
            //      x_i = b_i (1_ij - sum E_is x_s), column by column of E, two at a time -------------
            const int blk = 2 * pw + (lane >> 4), col = lane & 15;
            const float* eb = E + 16 * blk * kAStride + 16 * blk;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
            for (int s2 = 0; s2 < 16; s2 += 2) {
                const float2 b2 = *reinterpret_cast<const float2*>(vec + C + 16 * blk + s2);
                float2 e[16];
#pragma unroll
                for (int i = s2 + 1; i < 16; ++i) e[i] = *reinterpret_cast<const float2*>(eb + i * kAStride + s2);
                x[s2] *= b2.x;
                x[s2 + 1] = b2.y * (x[s2 + 1] - e[s2 + 1].x * x[s2]);
#pragma unroll
                for (int i = s2 + 2; i < 16; ++i) x[i] = x[i] - e[i].x * x[s2] - e[i].y * x[s2 + 1];
            }
            if (nb >= 2) ok = wait(&B->t_free[group], ((nb - 2) >> 1) & 1);
            if (ok) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t o = sw128_off(16 * blk + i, 2 * blk + (col >> 3)) + 2 * (col & 7);
                    const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                    st_shared_u16(aTH + o, hi);
                    st_shared_u16(aTL + o, __float2bfloat16_rn(x[i] - __bfloat162float(hi)));
                }
            }
        }
        if (named_sync_or(bar, kPrepThreads, !ok)) {
            *abort = 1;
            return false;
        }
        // ---- the blocks below: 16x16 ones (warps 0, 1), then the 32x32 one, a 16x16 tile per warp:
        //      -T'(r0.., tk..) (E(r0.., ck..) T'(ck.., c0..)), the product in brackets through shared memory
#pragma unroll 1
        for (int level = 0; level < 2; ++level) {
            const bool on = level == 1 || pw < 2;
            const int r0 = level ? 32 + 16 * (pw >> 1) : 32 * pw + 16, c0 = level ? 16 * (pw & 1) : 32 * pw;
            const int ck = level ? 0 : 32 * pw, tk = level ? 32 : r0;
            const int mr = level ? 16 * (pw >> 1) : 16 * pw, mc = level ? 16 * (pw & 1) : 0, mk = level ? 0 : mr;
            uint32_t ah[4], al[4], th[4], tl[4];
            if (on) {
                float Mx[2][4] = {};
#pragma unroll 1
                for (int kk = 0; kk <= 16 * level; kk += 16) {
                    load_split(E, r0, ck + kk, ah, al);
                    const uint32_t o = sw128_off(ck + kk + fr, c0 / 8 + fc);
                    ldsm4t(th, aTH + o);
                    ldsm4t(tl, aTL + o);
                    mma_split(Mx, ah, al, th, tl);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi, lo;
                        split2(Mx[i][2 * h], Mx[i][2 * h + 1], hi, lo);
                        const uint32_t o = (mr + 8 * h + gq) * kMStride + (mc + 8 * i) * 2 + 4 * cq;
                        st_shared_b32(aM + o, hi);
                        st_shared_b32(aM + 32 * kMStride + o, lo);
                    }
            }
            named_sync(bar, kPrepThreads);
            if (on) {
                float N[2][4] = {};
#pragma unroll 1
                for (int kk = 0; kk <= 16 * level; kk += 16) {
                    const uint32_t o = sw128_off(r0 + fr, (tk + kk) / 8 + fc), m = (mk + kk + fr) * kMStride + mc * 2 + fc * 16;
                    ldsm4(ah, aTH + o);
                    ldsm4(al, aTL + o);
                    ldsm4t(th, aM + m);
                    ldsm4t(tl, aM + 32 * kMStride + m);
                    mma_split(N, ah, al, th, tl);
                }
                store_negated(aTH, aTL, r0, c0, N);
            }
            if (level == 0) named_sync(bar, kPrepThreads);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->ready[group]);
        if (!same) {
            more = step() && step();
            if (more && pw == 3) load_gates(w, c);
        }
        nb += 2;
        at.next();
        at.next();
        six.next();
        six.next();
    }
}

// ---------------------------------------------------------------- the kernel

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
          const __grid_constant__ CUtensorMap tmv, const StepArgs a) {
    using L = TcLayout<DK>;
    constexpr int KA = L::KA, XC = DK / 4;   // channels of X of a converting thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Bars* B = reinterpret_cast<Bars*>(sm + L::BAR);
    volatile int* abort = &B->abort;

    if (tid == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&B->kq_free[i], 1);
        }
        for (int i = 0; i < 6; ++i) {
            mbar_init(&B->kq_full[i], 1);
            mbar_init(&B->vec_free[i], kConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B->g[i], 1);
            mbar_init(&B->v_full[i], 1);
            mbar_init(&B->v_free[i], 1);
            mbar_init(&B->v_clear[i], 1);
            mbar_init(&B->ot_full[i], kConvWarps);
            mbar_init(&B->ready[i], kPrepWarps);
            mbar_init(&B->t_free[i], 1);
            mbar_init(&B->p_free[i], 1);
            mbar_init(&B->drain[i], 1);
        }
        mbar_init(&B->g_free, kPrepWarps);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&B->item_full[i], 1);
            mbar_init(&B->item_free[i], kThreads / 32 - 1);
        }
        mbar_init(&B->stolen, 1);
        for (uint64_t* b : {&B->xh, &B->xl, &B->rh, &B->rl, &B->dh, &B->dl, &B->uo}) mbar_init(b, kConvWarps);
        for (uint64_t* b : {&B->z, &B->u, &B->o1, &B->dx, &B->o}) mbar_init(b, 1);
        B->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    griddep_wait();
    {   // This CTA's request has no part, or is short and left to the launch that follows: others of the grid may have work
        // all the same, which is theirs or whoever's takes it over.
        Request rq;
        if (a.above) griddep_launch_dependents();   // a launch for the shorter requests follows, which may run beside this one
        if (!read_request(a, blockIdx.x / a.Hv, rq)) return;
    }
    if (warp == 0) tmem_alloc(&B->tmem, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B->tmem;

    int status = 0;
    bool fail = false;
    if (warp < kConvWarps) {
        // ======================= converting warps ==================================
        const int r = 32 * (warp & 3) + lane, cp = warp >> 2, t0 = 16 * cp;   // row; part: tokens t0 .., channels XC cp ..
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t colx = tl + L::COL_X + cp * XC, colxp = tl + L::COL_XP + cp * XC;
        const uint32_t colz = tl + L::COL_Z + t0, colu = tl + L::COL_U + t0, colo = tl + L::COL_O + t0, cold = tl + L::COL_XP + t0;
        auto signal = [&](uint64_t* b) {   // this warp's tensor-memory stores (and loads) are done
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        // 16 values: their high parts to 8 columns, kept in h for the low ones' turn
        auto store_high = [&](uint32_t col, const float* x, uint32_t (&h)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            tmem_st8(col, h);
        };
        auto store_low = [&](uint32_t col, const float* x, const uint32_t (&h)[8]) {
            uint32_t l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = low_parts(x[2 * i], x[2 * i + 1], h[i]);
            tmem_st8(col, l);
        };
        auto load_x = [&](float (&x)[XC]) {
            if constexpr (XC == 32) tmem_ld32(colx, x);
            else tmem_ld16(colx, x);
            tmem_ld_wait();
        };
        auto publish_x = [&]() {
            float x[XC];
            uint32_t h[XC / 16][8];
            load_x(x);
#pragma unroll
            for (int p = 0; p < XC / 16; ++p) store_high(colxp + 16 * p, x + 16 * p, h[p]);
            signal(&B->xh);
#pragma unroll
            for (int p = 0; p < XC / 16; ++p) store_low(colxp + 16 * p + 8, x + 16 * p, h[p]);
            signal(&B->xl);
        };
        // warp-uniform before the warp-collective tensor-memory accesses
        auto wait_all = [&](uint64_t* b, uint32_t parity) {
            fail = fail || !warp_wait(smem_u32(b), parity, abort);
        };
        Ring<kTiles> at;
        Ring<6> six;
        // outputs of block nb through the tile over its V, [64 t][128], 16-byte chunks of odd tokens
        // shifted by half a bank row
        auto outputs = [&](int nb) {
            wait_all(&B->o, nb & 1);
            if (fail) return;
            const bool odd = lane & 1;
            const int ch = (r & ~1) / 8;
            const uint32_t ot = sbase + L::V + (nb & 1) * L::V_BYTES + (r & 6) * 2 + (t0 + (odd ? 1 : 0)) * 256 + ((ch ^ (odd ? 4 : 0)) << 4);
            float o[16];
            tmem_ld16(colo, o);
            tmem_ld_wait();
#pragma unroll
            for (int m = 0; m < 8; ++m) {   // lane pairs trade values: two adjacent rows of one token per lane
                const float send = odd ? o[2 * m] : o[2 * m + 1], keep = odd ? o[2 * m + 1] : o[2 * m];
                const float recv = __shfl_xor_sync(0xffffffffu, send, 1);
                st_shared_b32(ot + 512 * m, odd ? pack_bf16(recv, keep) : pack_bf16(keep, recv));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->ot_full[nb & 1]);
        };
        // The state in global memory: a warp moves its 32 rows by quads of lanes, 32 contiguous bytes of a row
        // each (rows lane / 4 + 8 i of its 32).
        auto state_row = [&](const Work& w) {
            return a.states + ((static_cast<size_t>(w.slot) * a.Hv + w.head) * DV + 32 * (warp & 3) + (lane >> 2)) * DK + cp * XC + 2 * (lane & 3);
        };
        Work w;
        int nb = 0;   // blocks of the CTA so far
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k) {
            {
                float x[XC];
                const float* sp = state_row(w);
#pragma unroll
                for (int i = 0; i < XC; i += 2) {   // 16 rows at a time: rows lane / 4, then + 8, of 8 columns
                    const int h16 = i / (XC / 2), e = i % (XC / 2);
                    float2 u = make_float2(0.f, 0.f);
                    if (!w.fresh) u = __ldcs(reinterpret_cast<const float2*>(sp + (16 * h16 + 8 * ((e / 2) & 1)) * DK + 8 * (e / 4)));
                    x[i] = u.x;
                    x[i + 1] = u.y;
                }
                tmem_st_rows<XC / 2>(colx, x);
                tmem_st_rows<XC / 2>(colx + (16u << 16), x + XC / 2);
                tmem_st_wait();
                __syncwarp();
            }
            for (int c = 0; c < w.blocks && !fail; ++c, ++nb) {
                const uint32_t p = nb & 1;
                const float* vec = reinterpret_cast<const float*>(sm + L::VEC) + at.s * kVec;
                uint32_t h[8];
                publish_x();
                // ---- while Z is computed: the outputs of the block before; X scaled by G_63 --------------
                if (nb > 0) outputs(nb - 1);
                wait_all(&B->ready[p], (nb >> 1) & 1);
                if (fail) break;
                {
                    float x[XC];
                    const float gc = vec[2 * C + C - 1];
                    load_x(x);
#pragma unroll
                    for (int i = 0; i < XC; ++i) x[i] *= gc;
                    if constexpr (XC == 32) tmem_st32(colx, reinterpret_cast<const uint32_t(&)[32]>(x));
                    else tmem_st16(colx, reinterpret_cast<const uint32_t(&)[16]>(x));
                }
                // ---- R = -G Z, tokens t0 .. ----------------------------------------------------------
                wait_all(&B->z, p);
                if (fail) break;
                float y[16], g[16];
                tmem_ld16(colz, y);
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(&g[i]) = *reinterpret_cast<const float4*>(vec + 2 * C + t0 + i);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] *= -g[i];
                store_high(colz, y, h);
                signal(&B->rh);
                store_low(colz + 8, y, h);
                signal(&B->rl);
                // ---- O = G (Q X^T), in place, while U is computed ---------------------------------------
                wait_all(&B->o1, p);
                if (fail) break;
                tmem_ld16(colo, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] *= g[i];
                tmem_st16(colo, reinterpret_cast<const uint32_t(&)[16]>(y));
                // ---- U' = U D_63 for the state, then U for the outputs -----------------------------------
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(&g[i]) = *reinterpret_cast<const float4*>(vec + 3 * C + t0 + i);
                wait_all(&B->u, p);
                if (fail) break;
                tmem_ld16(colu, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] *= y[i];
                store_high(cold, g, h);
                signal(&B->dh);
                store_low(cold + 8, g, h);
                signal(&B->dl);
                store_high(colu, y, h);
                store_low(colu + 8, y, h);
                signal(&B->uo);
                if (lane == 0) mbar_arrive(&B->vec_free[six.s]);
                // ---- X is whole ----------------------------------------------------------------------------
                wait_all(&B->dx, p);
                at.next();
                six.next();
            }
            if (fail) break;
            float x[XC];
            tmem_ld_rows<XC / 2>(colx, x);
            tmem_ld_rows<XC / 2>(colx + (16u << 16), x + XC / 2);
            tmem_ld_wait();
            float* sp = state_row(w);
#pragma unroll
            for (int i = 0; i < XC; i += 2) {
                const int h16 = i / (XC / 2), e = i % (XC / 2);
                __stcs(reinterpret_cast<float2*>(sp + (16 * h16 + 8 * ((e / 2) & 1)) * DK + 8 * (e / 4)), make_float2(x[i], x[i + 1]));
            }
            __syncwarp();
        }
        if (!fail && nb > 0) outputs(nb - 1);
        if (fail) status = kStatusMmaWait;
    } else if (warp < kConvWarps + kGroups * kPrepWarps) {
        if (!prep_warps<DK>(a, sm, sbase, B, tmem)) {
            fail = true;
            status = kStatusMmaWait;
        }
    } else if (warp == kOther) {
        // ======================= MMA issue ==========================================
        {
            const bool el = elect_one();
            constexpr uint32_t ID_64 = idesc_bf16(128, 64, false, false);
            constexpr uint32_t ID_V = idesc_bf16(128, 64, true, false);    // V^T T'^T
            constexpr uint32_t ID_K = idesc_bf16(128, DK, false, true);    // U' K
            // the A operand of k-step kk: 16 kk columns on, 8 more for the low parts
            auto kstep = [](int kk) { return static_cast<uint64_t>((kk / 4) * 1024 + (kk % 4) * 2); };
            // operand descriptors of stage 0; offsets in 16-byte units are added to them
            const uint64_t dK0 = kmaj(sbase + L::KQ), dKm0 = mnmaj(sbase + L::KQ, 16384), dV0 = mnmaj(sbase + L::V, 8192);
            const uint64_t dT0 = kmaj(sbase + L::TP);
            const uint32_t cx = tmem + L::COL_X, cxp = tmem + L::COL_XP, cz = tmem + L::COL_Z, cu = tmem + L::COL_U, co = tmem + L::COL_O;
            auto wait_w = [&](uint64_t* b, uint32_t parity) {   // the whole warp goes on, or gives up, together
                fail = fail || !warp_wait(smem_u32(b), parity, abort);
            };
            Ring<kTiles> at;
            Ring<6> six;
            Work w;
            int nb = 0;   // blocks of the CTA so far
            uint32_t clear = 0;   // the turn of each v_clear, a bit each
            for (int k = 0; !fail && next_item(B, k, w, fail); ++k)
            for (int c = 0; c < w.blocks && !fail; ++c, ++nb, at.next(), six.next()) {
                const uint32_t p = nb & 1;
                const uint64_t dK = dK0 + at.s * (L::KQ_BYTES / 16), dKm = dKm0 + at.s * (L::KQ_BYTES / 16);
                const uint64_t dV = dV0 + p * (L::V_BYTES / 16);
                const uint64_t dT = dT0 + p * (L::TP_BYTES / 16);
                const bool part = w.len - c * C < C;
                auto start_u = [&]() {   // U = V^T T'^T, both parts of T'; the parts of the U before are read by now
                    wait_w(&B->v_full[p], (nb >> 1) & 1);
                    if (part) {
                        wait_w(&B->v_clear[p], (clear >> p) & 1);
                        clear ^= 1u << p;
                    }
                    if (nb >= 1) wait_w(&B->o, p ^ 1);
                    if (!fail && el) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_bf16_ss(cu, dV + kk * 128, dT + kk * 2, ID_V, kk > 0);
                            mma_bf16_ss(cu, dV + kk * 128, dT + 512 + kk * 2, ID_V, true);
                        }
                    }
                };
                // before X is published if T' and V are there already and the block before's products are done
                const bool u_early = __all_sync(0xffffffffu, mbar_test(smem_u32(&B->ready[p]), (nb >> 1) & 1) &&
                                                                 mbar_test(smem_u32(&B->v_full[p]), (nb >> 1) & 1) &&
                                                                 (!part || mbar_test(smem_u32(&B->v_clear[p]), (clear >> p) & 1)) &&
                                                                 (nb == 0 || mbar_test(smem_u32(&B->o), p ^ 1)));
                if (u_early) start_u();
                wait_w(&B->kq_full[six.s], six.phase);
                if (part) wait_w(&B->ready[p], (nb >> 1) & 1);   // K's rows past the end are zeroed
                wait_w(&B->xh, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) mma_bf16_ts(cz, cxp + 16 * kk, dK + kstep(kk), ID_64, kk > 0);
                }
                wait_w(&B->xl, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) mma_bf16_ts(cz, cxp + 16 * kk + 8, dK + kstep(kk), ID_64, true);
                    mma_commit(&B->z);
                }
                if (!u_early) {
                    wait_w(&B->ready[p], (nb >> 1) & 1);
                    start_u();
                }
                if (nb >= 1) wait_w(&B->ot_full[p ^ 1], ((nb - 1) >> 1) & 1);   // the outputs of the block before are read
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) mma_bf16_ts(co, cxp + 16 * kk, dK + 512 + kstep(kk), ID_64, kk > 0);
                    mma_commit(&B->o1);
                }
                wait_w(&B->rh, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_bf16_ts(cu, cz + 16 * kk, dT + kk * 2, ID_64, true);
                        mma_bf16_ts(cu, cz + 16 * kk, dT + 512 + kk * 2, ID_64, true);
                    }
                }
                wait_w(&B->rl, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(cu, cz + 16 * kk + 8, dT + kk * 2, ID_64, true);
                    mma_commit(&B->u);
                    mma_commit(&B->t_free[p]);
                }
                wait_w(&B->dh, p);   // (after Q X^T was waited for: U' lies where the parts of X were)
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(cx, cxp + 16 * kk, dKm + kk * 128, ID_K, true);
                }
                wait_w(&B->dl, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(cx, cxp + 16 * kk + 8, dKm + kk * 128, ID_K, true);
                    mma_commit(&B->dx);
                }
                wait_w(&B->uo, p);
                if (fail) break;
                if (el) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_bf16_ts(co, cu + 16 * kk, dT + 1024 + kk * 2, ID_64, true);
                        mma_bf16_ts(co, cu + 16 * kk + 8, dT + 1024 + kk * 2, ID_64, true);
                    }
                    mma_commit(&B->o);
                    mma_commit(&B->kq_free[at.s]);
                    mma_commit(&B->p_free[p]);
                }
            }
            // the last arrivals that nobody else waits for: after the CTA has left they would hit another's memory
            for (int m = nb < kTiles ? 0 : nb - kTiles; m < nb && !fail; ++m) wait_w(&B->kq_free[m % kTiles], (m / kTiles) & 1);
            for (int m = nb < 2 ? 0 : nb - 2; m < nb && !fail; ++m) {
                wait_w(&B->t_free[m & 1], (m >> 1) & 1);
                wait_w(&B->p_free[m & 1], (m >> 1) & 1);
            }
            if (fail) {   // every MMA issued completes before the CTA leaves (bounded)
                status = kStatusMmaWait;
                if (el) {
                    mma_commit(&B->drain[0]);
                    mbar_wait(&B->drain[0], 0, 100000000ull);
                }
                __syncwarp();
            }
        }
    } else if (warp == kOther + 1) {
        // ======================= K and Q loads, [K;Q] K^T ============================
        Ring<kTiles> at, pt;   // of the loads; of the products
        Ring<6> six, psix;
        const bool el = elect_one();
        const uint64_t dK0 = kmaj(sbase + L::KQ);
        Work w;
        int nb = 0, np = 0;
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k) {
            const int first = nb;
            while (!fail && np < first + w.blocks) {
                // the loads of block np, and of those after it whose slots are free already
                while (nb < first + w.blocks && nb < np + kTiles) {
                    const uint32_t slot = smem_u32(&B->kq_free[at.s]);
                    if (nb >= kTiles) {
                        if (nb == np)
                            fail = !warp_wait(slot, at.phase ^ 1, abort);
                        else if (!__all_sync(0xffffffffu, mbar_test(slot, at.phase ^ 1)))
                            break;
                        if (fail) break;
                    }
                    if (lane == 0) {
                        uint8_t* kq = sm + L::KQ + at.s * L::KQ_BYTES;
                        const int row = w.row0 + (nb - first) * C;
                        mbar_arrive_expect_tx(&B->kq_full[six.s], L::KQ_BYTES);
#pragma unroll 1
                        for (int x = 0; x < KA; ++x) {
                            tma_load_3d(&tmk, &B->kq_full[six.s], kq + x * 16384, x * 64, w.khead, row);
                            tma_load_3d(&tmq, &B->kq_full[six.s], kq + x * 16384 + 8192, x * 64, w.khead, row);
                        }
                    }
                    __syncwarp();
                    ++nb;
                    at.next();
                    six.next();
                }
                if (fail) break;
                // its product, once the tile is here and the product before is read
                fail = !warp_wait(smem_u32(&B->kq_full[psix.s]), psix.phase, abort) ||
                       (np > 0 && !warp_wait(smem_u32(&B->g_free), (np - 1) & 1, abort));
                if (el && !fail) {
                    constexpr uint32_t ID_G = idesc_bf16(128, 64, false, false);
                    const uint64_t d0 = dK0 + pt.s * (L::KQ_BYTES / 16);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t d = d0 + (kk / 4) * 1024 + (kk % 4) * 2;
                        mma_bf16_ss(tmem + L::COL_G, d, d, ID_G, kk > 0);
                    }
                    mma_commit(&B->g[np & 1]);
                }
                __syncwarp();
                ++np;
                pt.next();
                psix.next();
            }
        }
        if (fail || *abort) {
            status = kStatusTmaWait;
            if (el) {   // the products in flight
                mma_commit(&B->drain[1]);
                mbar_wait(&B->drain[1], 0, 100000000ull);
            }
            // After a failure loads may be in flight: let them land (bounded; a
            // phase that no load began runs into the limit).
            if (lane == 0)
                for (int i = 0; i < 6; ++i)
                    for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(&B->kq_full[i], ph, 10000000ull);
            __syncwarp();
        }
    } else if (warp == kOther + 2) {
        // ======================= output copies =======================================
        Work w;
        int nb = 0;
        const size_t ostep = static_cast<size_t>(a.Hv) * DV;
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k) {
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(w.row0) * a.Hv + w.head) * DV;
            for (int c = 0; c < w.blocks; ++c, ++nb) {
                const int vs = nb & 1;
                fail = !warp_wait(smem_u32(&B->ot_full[vs]), (nb >> 1) & 1, abort);
                if (fail) break;
                const uint32_t ot = sbase + L::V + vs * L::V_BYTES;
                const int n = min(C, w.len - c * C);
                const int ch = lane & 15;
#pragma unroll 4
                for (int t = lane >> 4; t < n; t += 2) {
                    const uint4 y = ld_shared_v4(ot + t * 256 + ((ch ^ ((t & 1) << 2)) << 4));
                    *reinterpret_cast<uint4*>(op + static_cast<size_t>(c * C + t) * ostep + ch * 8) = y;
                }
                fence_proxy_async_smem();   // the tile's generic accesses come before the load that overwrites it
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->v_free[vs]);
            }
        }
        if (fail) status = kStatusMmaWait;
    } else {
        // ======================= work, V loads =======================================
        int idx = blockIdx.x, nb = 0;
        int keep = C;   // tokens of the block before, if it has rows past its request's end
        for (int k = 0;; ++k) {
            Request rq;
            // (a CTA that takes over a request without a part, or a short one, ends; those not yet started start by themselves)
            const bool have = idx >= 0 && read_request(a, idx / a.Hv, rq);
            const int i = k % kItems;
            if (k >= kItems) fail = !warp_wait(smem_u32(&B->item_free[i]), ((k / kItems) & 1) ^ 1, abort);
            if (fail) break;
            Work w = {};
            if (have) {
                w.row0 = rq.row0;
                w.len = rq.len;
                w.slot = rq.slot;
                w.fresh = rq.fresh;
                w.head = idx % a.Hv;
                w.khead = w.head / (a.Hv / a.Hk);
                w.blocks = (rq.len + C - 1) / C;
            }
            if (lane == 0) {
                B->item[i] = w;
                mbar_arrive(&B->item_full[i]);
            }
            if (have && !w.fresh) {   // the state, into L2
                const float* st = a.states + (static_cast<size_t>(w.slot) * a.Hv + w.head) * DV * DK;
                for (int x = lane; x < DV * DK / 32; x += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(st + 32 * x));
            }
            if (keep < C) {   // those rows of V, zero (once the next item is out: the prep of its first blocks starts with it)
                const int m = nb - 1;
                // (the turn before is complete: V of block m was loaded after block m - 2's outputs had left)
                if (!warp_wait(smem_u32(&B->v_full[m & 1]), (m >> 1) & 1, abort)) {
                    fail = true;
                    break;
                }
                const uint32_t v = sbase + L::V + (m & 1) * L::V_BYTES;
                for (int x = lane; x < (C - keep) * 8; x += 32) {
                    const uint32_t o = sw128_off(keep + x / 8, x % 8);
                    st_shared_v4(v + o, 0, 0, 0, 0);
                    st_shared_v4(v + 8192 + o, 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->v_clear[m & 1]);
            }
            if (!have) break;
            keep = w.len - (w.blocks - 1) * C;
            for (int c = 0; c < w.blocks && !fail; ++c, ++nb) {
                const int vs = nb & 1, row = w.row0 + c * C;
                // more work only once this item's last loads are at hand: what waits here could run elsewhere
                if (c + 1 == w.blocks && lane == 0) steal_request(&B->answer, &B->stolen);
                if (nb >= 2) fail = !warp_wait(smem_u32(&B->v_free[vs]), ((nb - 2) >> 1) & 1, abort);
                if (lane == 0 && !fail) {
                    uint8_t* v = sm + L::V + vs * L::V_BYTES;
                    mbar_arrive_expect_tx(&B->v_full[vs], L::V_BYTES);
#pragma unroll 1
                    for (int x = 0; x < DV / 64; ++x) tma_load_3d(&tmv, &B->v_full[vs], v + x * 8192, x * 64, w.head, row);
                }
                // the block after next, into L2 (K, Q and V; lanes 0 ..)
                if (c + kTiles < w.blocks && lane < 2 * KA + DV / 64) {
                    const CUtensorMap* m = lane < KA ? &tmk : lane < 2 * KA ? &tmq : &tmv;
                    const int x = lane < KA ? lane : lane < 2 * KA ? lane - KA : lane - 2 * KA;
                    prefetch_3d(m, x * 64, lane < 2 * KA ? w.khead : w.head, row + kTiles * C);
                }
                __syncwarp();
            }
            if (!fail) fail = !warp_wait(smem_u32(&B->stolen), k & 1, abort);
            if (fail) break;
            idx = stolen_index(&B->answer);
            fence_proxy_async_smem();   // this read comes before the next answer's write
            __syncwarp();
        }
        if (fail) {
            status = kStatusFlagWait;
            if (lane == 0)
                for (int i = 0; i < 2; ++i)
                    for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait(&B->v_full[i], ph, 10000000ull);
            __syncwarp();
        }
    }
    if (fail) *abort = 1;
    if (status && lane == 0) atomicOr(a.status, status);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, L::TMEM_COLS);
}

template <int DK>
cudaError_t run(const StepArgs& a, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v) {
    constexpr uint32_t smem = TcLayout<DK>::BYTES + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    const cudaError_t e = cudaFuncSetAttribute(tc_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long grid = static_cast<long long>(a.requests) * a.Hv;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(tc_kernel<DK>, static_cast<unsigned>(grid), kThreads, smem, s, q, k, v, a);
}

}  // namespace

cudaError_t launch_tc(const StepArgs& a, cudaStream_t s, PFN_cuTensorMapEncodeTiled_v12000 enc) {
    CUtensorMap q, k, v;
    if (a.dv != DV || !make_map(enc, &q, a.q, a.dk, a.Hk, a.rows, a.q_stride, C) ||
        !make_map(enc, &k, a.k, a.dk, a.Hk, a.rows, a.k_stride, C) || !make_map(enc, &v, a.v, a.dv, a.Hv, a.rows, a.v_stride, C))
        return cudaErrorInvalidValue;
    if (a.dk == 64) return run<64>(a, s, q, k, v);
    if (a.dk == 128) return run<128>(a, s, q, k, v);
    return cudaErrorInvalidValue;
}

}  // namespace packed
}  // namespace la

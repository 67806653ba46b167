// The gated delta rule over packed requests on the tcgen05 tensor cores: bf16
// q, k and v, value heads of 128, blocks of 64 tokens. The algebra is that of
// packed_chunk.cu (value heads of 64, warp-level MMAs), with b's columns in T:
//   T' = (I + A)^-1 diag(b),   U = T' (V - diag(G) K X^T)
//   O = diag(G) Q X^T + P U,   X <- G_63 X + U^T diag(D_63,.) K
// and so is the precision: q, k, v exact; X, G Z, T' and U in two bf16 parts
// wherever the state depends on them; X in Q X^T and P in one.
//
// Work split. A CTA takes one (request, value head) after another, longest
// requests first: the grid has one CTA for each, and a running one takes over
// the next that has not been started (cluster launch control), so that its
// prep and load warps are already at the next request while the chain finishes
// one. The state's 128 rows lie on the 128 tensor-memory lanes, so that every product of the chain is an M = 128
// MMA with its A operand (X, R = -G Z, U: bf16 parts) in tensor memory and its
// B operand (K, Q, T', P) in shared memory:
//   Z = X K^T, O1 = X Q^T  [dv][token],  U = V^T T'^T + R T'^T,
//   dX = U' K,  O2 = U P^T
// Eight warps convert between them: thread (row r, half hh) holds half of row
// r of X in fp32 registers and takes half the columns of each product. Four
// prep warps compute T' and P of the next block meanwhile; of the others one
// issues the chain's MMAs, one the loads, one copies the outputs out, and one
// fetches the work.
//
// The chain's steps depend on one another, so what bounds a long request is
// their latency: three products (Z, R T'^T, dX) with a conversion after each.
// High parts are published first, so that a product starts while the low ones
// are still formed. V^T T'^T, Q X^T and the outputs run in the gaps: the
// outputs of a block are read while the next one's Z and U run.
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
constexpr int kConvWarps = 8, kPrepWarps = 4;
constexpr int kThreads = 32 * (kConvWarps + kPrepWarps + 4);   // + MMA issue, loads, output copies, work
constexpr int kPrepThreads = 32 * kPrepWarps;
constexpr uint32_t kBarPrep = 1;      // named barrier of the prep warps
constexpr int kTiles = 3;             // ring of K, Q and V tiles
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
    static constexpr uint32_t V = kTiles * KQ_BYTES;            // [kTiles]
    static constexpr uint32_t TP = V + kTiles * V_BYTES;        // [2]: T high, T low, P, each [64 t][64 j]
    static constexpr uint32_t TP_BYTES = 3 * 8192;
    static constexpr uint32_t A = TP + 2 * TP_BYTES;            // fp32 [64][kAStride]
    static constexpr uint32_t M = A + C * kAStride * 4;         // bf16 high, low [32][kMStride bytes]
    static constexpr uint32_t VEC = M + 2 * 32 * kMStride;      // [kTiles][kVec] fp32
    static constexpr uint32_t BAR = VEC + kTiles * kVec * 4;
    static constexpr uint32_t BYTES = BAR + 1024;
    // Tensor memory columns. X: per half hh of the channels DK/4 columns of
    // high parts, then DK/4 of low ones; dX (fp32, DK columns) takes the same
    // columns once Z and Q X^T are done, each half over its own.
    static constexpr uint32_t COL_X = 0;
    // Z; R over it, per half of the tokens 16 columns of high parts, then 16 of low ones
    static constexpr uint32_t COL_Z = 128;
    static constexpr uint32_t COL_U = 192;     // U; its parts over it, like R
    static constexpr uint32_t COL_UD = 256;    // parts of U'
    static constexpr uint32_t COL_O1 = 320;
    static constexpr uint32_t COL_O2 = 384;
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
    uint64_t kq_full[kTiles], kq_free[kTiles];   // TMA; MMA: every product of the block is done
    uint64_t v_full[kTiles], v_free[kTiles];     // TMA; copier: the output tile over V has left
    uint64_t vec_free[kTiles];                   // converters: the block's vectors are read (8)
    uint64_t ot_full[kTiles];                    // converters: the output tile is written (8)
    uint64_t ready[2], tp_free[2];               // prep warps: T, P and vectors (4); MMA: T and P are read
    uint64_t g;                                  // MMA: [K;Q] K^T
    uint64_t xh, xl, rh, rl, dh, dl, uo;         // converters: parts of X, R, U' and both of U published (8 each)
    uint64_t z, u, o1, dx, o;                    // MMA: Z, U, Q X^T, dX, O done
    uint64_t drain[2];                           // after a failure: MMAs of either issuer are done
    uint64_t item_full[kItems], item_free[kItems];   // work warp; every other warp has read the item (15)
    uint64_t want, stolen;                       // loads: all of the item is issued; the answer to a request for more work
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

struct Ring3 {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == kTiles) {
            s = 0;
            phase ^= 1;
        }
    }
};

// mbar_wait_or_abort with the loop out of line: the warps' code, dozens of waits
// among it, has to stay in the instruction cache (148 KB with the loops inline
// ran a third slower once every SM fetched it). One try waits for a while itself.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, const volatile int* abort) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const volatile int* abort) {
    const uint32_t b = smem_u32(bar);
    return mbar_try_wait(b, parity) || wait_on(b, parity, abort);
}

// 16 lanes x 64 (32) columns of tensor memory between a warp's registers, by quads: with g = lane / 4,
// c = lane % 4, x[4 i], x[4 i + 1] are columns 8 i + 2 c, + 1 of lane g, x[4 i + 2], x[4 i + 3] of lane g + 8.
template <int N>
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const float* x) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
    if constexpr (N == 32) {
        asm volatile(
            "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
            "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
            "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
            ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
              "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
              "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]),
              "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
            : "memory");
    } else {
        static_assert(N == 16, "64 or 32 columns");
        asm volatile(
            "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
            "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
            ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
              "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
            : "memory");
    }
}
template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float* x) {
    uint32_t* u = reinterpret_cast<uint32_t*>(x);
    if constexpr (N == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
              "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
              "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
              "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
              "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
            : "r"(taddr));
    } else {
        static_assert(N == 16, "64 or 32 columns");
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
              "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
              "=r"(u[14]), "=r"(u[15])
            : "r"(taddr));
    }
}

// The k-th item of this CTA, for a whole warp; false when there is none (blocks
// 0) or after a failure.
__device__ __forceinline__ bool next_item(Bars* B, int k, Work& w, bool& fail) {
    const int i = k % kItems;
    const bool ok = wait_bar(&B->item_full[i], (k / kItems) & 1, &B->abort);
    if (!__all_sync(0xffffffffu, ok)) {
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

// Four warps, block by block: [K;Q] K^T on the tensor cores; E_tj = D_tj
// k_t.k_j (j < t; warps 0, 1) and P_tj = D_tj q_t.k_j (j <= t; warps 2, 3) row
// by row (lane = tensor-memory lane = row; D_tj is a running product from the
// diagonal leftwards); then T' (A = diag(b) E): 16x16 diagonal blocks by
// forward substitution in fp32 (warps 0 and 1, a half-warp each), merged twice
// by T'_21 = -T'_22 (E_21 T'_11) on warp-level MMAs with two bf16 parts.
// Meanwhile warp 2 issues the next block's [K;Q] K^T and warp 3 computes its
// gate vectors.
template <int DK>
__device__ __forceinline__ bool prep_warps(const StepArgs& a, uint8_t* sm, uint32_t sbase, Bars* B, uint32_t tmem) {
    using L = TcLayout<DK>;
    const int lane = threadIdx.x & 31, pw = (threadIdx.x >> 5) - kConvWarps, ptid = threadIdx.x - 32 * kConvWarps;
    const int gq = lane >> 2, cq = lane & 3;
    const int fr = (lane & 7) + ((lane >> 3) & 1) * 8, fc = lane >> 4;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * pw) << 16);
    const bool issuer = pw == 2;
    const bool el = elect_one();
    volatile int* abort = &B->abort;
    float* E = reinterpret_cast<float*>(sm + L::A);
    const uint32_t aM = sbase + L::M;

    // gate vectors of block c from tokens 2 lane, 2 lane + 1 (past the end: gate 1, beta 0)
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
    auto vec_of = [&](int s) { return reinterpret_cast<float*>(sm + L::VEC) + s * kVec; };
    auto issue_products = [&](int s) {   // [K;Q] K^T of the block in stage s
        constexpr uint32_t ID_G = idesc_bf16(128, 64, false, false);
        const uint64_t d0 = kmaj(sbase + L::KQ + s * L::KQ_BYTES);
        if (el) {
#pragma unroll 1
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint64_t d = d0 + (kk / 4) * 1024 + (kk % 4) * 2;
                mma_bf16_ss(tmem + L::COL_G, d, d, ID_G, kk > 0);
            }
            mma_commit(&B->g);
        }
        __syncwarp();
    };
    Work w, wn;       // of the current and the next block
    int items = 1;
    bool lost = false;
    if (!next_item(B, 0, w, lost)) return !lost;
    if (pw == 3) {
        load_gates(w, 0);
        write_gates(vec_of(0), gn, bn);
    }
    // T' and P above their diagonal blocks stay zero: the MMAs read whole tiles
    for (int i = ptid; i < 2 * static_cast<int>(L::TP_BYTES) / 16; i += kPrepThreads)
        st_shared_v4(sbase + L::TP + i * 16, 0, 0, 0, 0);
    named_sync(kBarPrep, kPrepThreads);

    bool early = false;   // (issuer) this block's products were issued during the block before
    Ring3 at;
    // block c of the item, block nb of the CTA
    for (int c = 0, nb = 0; w.blocks > 0; ++nb, at.next()) {
        const uint32_t kq = sbase + L::KQ + at.s * L::KQ_BYTES;
        const uint32_t aTH = sbase + L::TP + (nb & 1) * L::TP_BYTES, aTL = aTH + 8192, aP = aTH + 16384;
        const float* vec = reinterpret_cast<const float*>(sm + L::VEC) + at.s * kVec;
        Ring3 nx = at;
        nx.next();
        int cn = c + 1;
        wn = w;
        if (cn == w.blocks) {
            cn = 0;
            next_item(B, items++, wn, lost);   // (blocks 0: this block is the last)
            if (lost) wn.blocks = 0;
        }
        const bool more = wn.blocks > 0;
        if (pw == 3 && more) load_gates(wn, cn);
        bool ok = !lost;
        const int n = w.len - c * C;
        if (n < C) {   // rows of the next request (or past the tensor): K and V zero, so that they leave the state alone
            ok = ok && wait_bar(&B->kq_full[at.s], at.phase, abort) && wait_bar(&B->v_full[at.s], at.phase, abort);
            if (ok) {
                const uint32_t v = sbase + L::V + at.s * L::V_BYTES;
                for (int i = ptid; i < (C - n) * 8; i += kPrepThreads) {
                    const uint32_t o = sw128_off(n + i / 8, i % 8);
#pragma unroll
                    for (int x = 0; x < L::KA; ++x) st_shared_v4(kq + x * 16384 + o, 0, 0, 0, 0);
                    st_shared_v4(v + o, 0, 0, 0, 0);
                    st_shared_v4(v + 8192 + o, 0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        }
        if (issuer && !early) {
            ok = __all_sync(0xffffffffu, ok && wait_bar(&B->kq_full[at.s], at.phase, abort));
            if (ok) issue_products(at.s);
        }
        early = false;
        ok = ok && wait_bar(&B->g, nb & 1, abort);
        if (ok && nb >= 2) ok = wait_bar(&B->tp_free[nb & 1], ((nb - 2) >> 1) & 1, abort);
        tc_fence_after();
        ok = __all_sync(0xffffffffu, ok);
        // ---- E and P by rows, 16 columns at a time from the right. D at a group's right edge: zero in the
        //      group of the diagonal and right of it, else the row's gates from the edge on -----------
        if (ok) {
            const bool isP = pw >= 2;
            const int hd = pw & 1;   // the half of the columns with this warp's diagonal
            const int t = 32 * hd + lane;
            const float g16 = vec[4 * C + t], g32 = vec[5 * C + t], mid = vec[4 * C + 31];
#pragma unroll 1
            for (int c16 = 2 * hd + 1; c16 >= 0; --c16) {
                const int u = 2 * hd + 1 - c16;   // 0, 1: the half of the diagonal; 2, 3: columns 16..31, 0..15 of rows 32..
                float d = u == 0 ? 0.f : u == 1 ? (lane >= 16 ? g16 : 0.f) : u == 2 ? g32 : g32 * mid;
                const int diag = u < 2 ? lane - (16 - 16 * u) : -1;   // the column of the row's diagonal element
                float x[16];
                tmem_ld16(tlane + L::COL_G + 16 * c16, x);
                tmem_ld_wait();
#pragma unroll
                for (int q4 = 3; q4 >= 0; --q4) {
                    const float4 g4 = *reinterpret_cast<const float4*>(vec + 16 * c16 + 4 * q4);
                    const float gl[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const int j = 4 * q4 + i;
                        if (j == diag) d = 1.f;
                        x[j] *= (j == diag && !isP) ? 0.f : d;
                        d *= gl[i];   // the gate of column j itself comes before the columns left of it
                    }
                }
                if (isP) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        st_shared_v4(aP + sw128_off(t, 2 * c16 + m), pack_bf16(x[8 * m], x[8 * m + 1]), pack_bf16(x[8 * m + 2], x[8 * m + 3]),
                                     pack_bf16(x[8 * m + 4], x[8 * m + 5]), pack_bf16(x[8 * m + 6], x[8 * m + 7]));
                } else {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        *reinterpret_cast<float4*>(E + t * kAStride + 16 * c16 + 4 * q4) =
                            make_float4(x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]);
                }
            }
        }
        tc_fence_before();
        if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        if (pw < 2) {
            // ---- diagonal blocks 2 pw and 2 pw + 1, lane = (block, column): x_i = b_i (1_ij - sum E_is x_s),
            //      column by column of E, four at a time ----------------------------------------
            const int blk = 2 * pw + (lane >> 4), col = lane & 15;
            const float* eb = E + 16 * blk * kAStride + 16 * blk;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
            for (int s4 = 0; s4 < 16; s4 += 4) {
                const float4 b4 = *reinterpret_cast<const float4*>(vec + C + 16 * blk + s4);
                float4 e[16];
#pragma unroll
                for (int i = s4 + 1; i < 16; ++i) e[i] = *reinterpret_cast<const float4*>(eb + i * kAStride + s4);
                x[s4] *= b4.x;
                x[s4 + 1] = b4.y * (x[s4 + 1] - e[s4 + 1].x * x[s4]);
                x[s4 + 2] = b4.z * (x[s4 + 2] - e[s4 + 2].x * x[s4] - e[s4 + 2].y * x[s4 + 1]);
                x[s4 + 3] = b4.w * (x[s4 + 3] - e[s4 + 3].x * x[s4] - e[s4 + 3].y * x[s4 + 1] - e[s4 + 3].z * x[s4 + 2]);
#pragma unroll
                for (int i = s4 + 4; i < 16; ++i)
                    x[i] = x[i] - e[i].x * x[s4] - e[i].y * x[s4 + 1] - e[i].z * x[s4 + 2] - e[i].w * x[s4 + 3];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t o = sw128_off(16 * blk + i, 2 * blk + (col >> 3)) + 2 * (col & 7);
                const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                st_shared_u16(aTH + o, hi);
                st_shared_u16(aTL + o, __float2bfloat16_rn(x[i] - __bfloat162float(hi)));
            }
            __syncwarp();
            // ---- the 16x16 block below: -T'_22 (E_21 T'_11) ----------------------------------
            const int rb = 32 * pw + 16, cb = 32 * pw;   // its first row and column
            uint32_t ah[4], al[4], th[4], tl[4], mh[4], ml[4];
            load_split(E, rb, cb, ah, al);
            ldsm4t(th, aTH + sw128_off(cb + fr, cb / 8 + fc));
            ldsm4t(tl, aTL + sw128_off(cb + fr, cb / 8 + fc));
            float Mx[2][4] = {}, N[2][4] = {};
            mma_split(Mx, ah, al, th, tl);
            split_tiles(Mx[0], Mx[1], mh, ml);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mh[i] = transpose8x8(mh[i]);
                ml[i] = transpose8x8(ml[i]);
            }
            ldsm4(th, aTH + sw128_off(rb + fr, rb / 8 + fc));
            ldsm4(tl, aTL + sw128_off(rb + fr, rb / 8 + fc));
            mma_split(N, th, tl, mh, ml);
            store_negated(aTH, aTL, rb, cb, N);
        } else if (pw == 3) {
            if (more) {
                // the slot's vectors of block nb - 2 are read (its phase is the one before block nb + 1's)
                if (nb + 1 < kTiles || __all_sync(0xffffffffu, wait_bar(&B->vec_free[nx.s], nx.phase ^ 1, abort)))
                    write_gates(vec_of(nx.s), gn, bn);
                else
                    ok = false;
            }
        } else if (issuer && more && wn.len - cn * C >= C) {
            // the next block is whole: its products now (this one's are read). Its loads wait for the
            // chain alone, which has all it needs for the blocks before.
            ok = __all_sync(0xffffffffu, wait_bar(&B->kq_full[nx.s], nx.phase, abort));
            tc_fence_after();
            if (ok) issue_products(nx.s);
            early = true;
        }
        if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        // ---- rows 32..63, columns 0..31: -T'_B (E_BA T'_A), a 16x16 tile per warp -----------
        {
            const int mi = pw >> 1, ni = pw & 1;
            float Mx[2][4] = {}, N[2][4] = {};
            uint32_t ah[4], al[4], th[4], tl[4];
#pragma unroll 1
            for (int kk = 0; kk < 2; ++kk) {
                load_split(E, 32 + 16 * mi, 16 * kk, ah, al);
                ldsm4t(th, aTH + sw128_off(16 * kk + fr, 2 * ni + fc));
                ldsm4t(tl, aTL + sw128_off(16 * kk + fr, 2 * ni + fc));
                mma_split(Mx, ah, al, th, tl);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi, lo;
                    split2(Mx[i][2 * h], Mx[i][2 * h + 1], hi, lo);
                    const uint32_t o = (16 * mi + 8 * h + gq) * kMStride + (16 * ni + 8 * i) * 2 + 4 * cq;
                    st_shared_b32(aM + o, hi);
                    st_shared_b32(aM + 32 * kMStride + o, lo);
                }
            named_sync(kBarPrep, kPrepThreads);
#pragma unroll 1
            for (int kk = 0; kk < 2; ++kk) {
                ldsm4(ah, aTH + sw128_off(32 + 16 * mi + fr, 4 + 2 * kk + fc));
                ldsm4(al, aTL + sw128_off(32 + 16 * mi + fr, 4 + 2 * kk + fc));
                ldsm4t(th, aM + (16 * kk + fr) * kMStride + (2 * ni + fc) * 16);
                ldsm4t(tl, aM + 32 * kMStride + (16 * kk + fr) * kMStride + (2 * ni + fc) * 16);
                mma_split(N, ah, al, th, tl);
            }
            store_negated(aTH, aTL, 32 + 16 * mi, 16 * ni, N);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->ready[nb & 1]);
        w = wn;
        c = cn;
    }
    return true;
}

// ---------------------------------------------------------------- the kernel

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
          const __grid_constant__ CUtensorMap tmv, const StepArgs a) {
    using L = TcLayout<DK>;
    constexpr int KA = L::KA, XH = DK / 2;   // channels of X a converting thread holds
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Bars* B = reinterpret_cast<Bars*>(sm + L::BAR);
    volatile int* abort = &B->abort;

    if (tid == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&B->kq_full[i], 1);
            mbar_init(&B->kq_free[i], 1);
            mbar_init(&B->v_full[i], 1);
            mbar_init(&B->v_free[i], 1);
            mbar_init(&B->vec_free[i], kConvWarps);
            mbar_init(&B->ot_full[i], kConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B->ready[i], kPrepWarps);
            mbar_init(&B->tp_free[i], 1);
            mbar_init(&B->drain[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&B->item_full[i], 1);
            mbar_init(&B->item_free[i], kThreads / 32 - 1);
        }
        mbar_init(&B->want, 1);
        mbar_init(&B->stolen, 1);
        for (uint64_t* b : {&B->xh, &B->xl, &B->rh, &B->rl, &B->dh, &B->dl, &B->uo}) mbar_init(b, kConvWarps);
        for (uint64_t* b : {&B->g, &B->z, &B->u, &B->o1, &B->dx, &B->o}) mbar_init(b, 1);
        B->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    griddep_wait();
    {   // requests without a part come last: where this CTA's has none, nobody's after it has
        Request rq;
        if (!read_request(a, blockIdx.x / a.Hv, rq)) return;
    }
    if (warp == 0) tmem_alloc(&B->tmem, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B->tmem;

    int status = 0;
    bool fail = false;
    auto wait = [&](uint64_t* b, uint32_t parity) { fail = fail || !wait_bar(b, parity, abort); };
    if (warp < kConvWarps) {
        // ======================= converting warps ==================================
        const int r = 32 * (warp & 3) + lane, hh = warp >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t colx = tl + L::COL_X + hh * XH;
        float X[XH];
        // The state in global memory: a warp moves its 32 rows by quads of lanes, 32 contiguous bytes of a row
        // each (rows lane / 4 + 8 i), and turns them to a row a lane through the columns of dX.
        auto state_row = [&](const Work& w) {
            return a.states + ((static_cast<size_t>(w.slot) * a.Hv + w.head) * DV + 32 * (warp & 3) + (lane >> 2)) * DK + hh * XH + 2 * (lane & 3);
        };
        auto signal = [&](uint64_t* b) {   // this warp's tensor-memory stores (and loads) are done
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        // 32 values: their high parts to 16 columns, kept in h for the low ones' turn
        auto pack_high = [&](const float* x, uint32_t (&h)[16]) {
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        };
        auto store_high = [&](uint32_t col, const float* x, uint32_t (&h)[16]) {
            pack_high(x, h);
            tmem_st16(col, h);
        };
        auto store_low = [&](uint32_t col, const float* x, const uint32_t (&h)[16]) {
            uint32_t l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) l[i] = low_parts(x[2 * i], x[2 * i + 1], h[i]);
            tmem_st16(col, l);
        };
        auto publish_x = [&]() {
            uint32_t h[16];
#pragma unroll
            for (int p = 0; p < XH / 32; ++p) store_high(colx + 16 * p, X + 32 * p, h);
            signal(&B->xh);
#pragma unroll
            for (int p = 0; p < XH / 32; ++p) {   // (the high parts again: fewer registers than keeping them)
                if (XH > 32) pack_high(X + 32 * p, h);
                store_low(colx + XH / 2 + 16 * p, X + 32 * p, h);
            }
            signal(&B->xl);
        };
        // warp-uniform before the warp-collective tensor-memory accesses
        auto wait_all = [&](uint64_t* b, uint32_t parity) {
            const bool ok = !fail && wait_bar(b, parity, abort);
            fail = !__all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        Ring3 at, last;
        // outputs of block nb, o = G O1 + O2, 16 tokens a half (q) at a time, through the tile over its V,
        // [64 t][128], 16-byte chunks of odd tokens shifted by half a bank row
        auto outputs = [&](int nb, int s, int q) {
            if (q == 0) wait_all(&B->o, nb & 1);
            if (fail) return;
            const bool odd = lane & 1;
            const int ch = (r & ~1) / 8, t0 = 32 * hh + 16 * q;
            const uint32_t ot = sbase + L::V + s * L::V_BYTES + (r & 6) * 2 + (t0 + (odd ? 1 : 0)) * 256 + ((ch ^ (odd ? 4 : 0)) << 4);
            const float* G = reinterpret_cast<const float*>(sm + L::VEC) + s * kVec + 2 * C + t0;
            float o[16], o2[16];
            tmem_ld16(tl + L::COL_O1 + t0, o);
            tmem_ld16(tl + L::COL_O2 + t0, o2);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(G + i);
                o[i] = g4.x * o[i] + o2[i];
                o[i + 1] = g4.y * o[i + 1] + o2[i + 1];
                o[i + 2] = g4.z * o[i + 2] + o2[i + 2];
                o[i + 3] = g4.w * o[i + 3] + o2[i + 3];
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) {   // lane pairs trade values: two adjacent rows of one token per lane
                const float send = odd ? o[2 * m] : o[2 * m + 1], keep = odd ? o[2 * m + 1] : o[2 * m];
                const float recv = __shfl_xor_sync(0xffffffffu, send, 1);
                st_shared_b32(ot + 512 * m, odd ? pack_bf16(recv, keep) : pack_bf16(keep, recv));
            }
            if (q == 0) return;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B->ot_full[s]);
                mbar_arrive(&B->vec_free[s]);
            }
        };
        Work w;
        int nb = 0;   // blocks of the CTA so far
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k) {
        for (int c = 0; c < w.blocks && !fail; ++c, ++nb) {
            const int s = at.s;
            const uint32_t p = nb & 1;
            if (c == 0) {
                const float* sp = state_row(w);
#pragma unroll
                for (int i = 0; i < XH; i += 2) {   // 16 rows at a time: x[(column / 8) * 4 + ..]: rows lane / 4, then + 8
                    const int h16 = i / (XH / 2), e = i % (XH / 2);
                    float2 u = make_float2(0.f, 0.f);
                    if (!w.fresh) u = __ldcs(reinterpret_cast<const float2*>(sp + (16 * h16 + 8 * ((e / 2) & 1)) * DK + 8 * (e / 4)));
                    X[i] = u.x;
                    X[i + 1] = u.y;
                }
            }
            if (nb > 0) outputs(nb - 1, last.s, 0);   // while Z is computed, or the state arrives
            if (c == 0) {
                tmem_st_rows<XH / 2>(colx, X);
                tmem_st_rows<XH / 2>(colx + (16u << 16), X + XH / 2);
                tmem_st_wait();
                __syncwarp();
#pragma unroll
                for (int q = 0; q < XH / 32; ++q) tmem_ld32(colx + 32 * q, reinterpret_cast<float(&)[32]>(X[32 * q]));
                tmem_ld_wait();
                publish_x();
            }
            const float* vec = reinterpret_cast<const float*>(sm + L::VEC) + s * kVec;
            float y[32];
            uint32_t h[16];
            // ---- R = -G Z, tokens 32 hh .. --------------------------------------------
            wait_all(&B->ready[p], (nb >> 1) & 1);
            wait_all(&B->z, p);
            if (fail) break;
            const uint32_t colz = tl + L::COL_Z + 32 * hh, colu = tl + L::COL_U + 32 * hh, cold = tl + L::COL_UD + 32 * hh;
            tmem_ld32(colz, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(vec + 2 * C + 32 * hh + i);
                y[i] *= -g4.x;
                y[i + 1] *= -g4.y;
                y[i + 2] *= -g4.z;
                y[i + 3] *= -g4.w;
            }
            store_high(colz, y, h);
            signal(&B->rh);
            store_low(colz + 16, y, h);
            signal(&B->rl);
            if (nb > 0) outputs(nb - 1, last.s, 1);   // while U is computed
            // ---- U' = U D_63 for the state, then U for the outputs ------------------------
            wait_all(&B->u, p);
            if (fail) break;
            tmem_ld32(colu, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 d4 = *reinterpret_cast<const float4*>(vec + 3 * C + 32 * hh + i);
                y[i] *= d4.x;
                y[i + 1] *= d4.y;
                y[i + 2] *= d4.z;
                y[i + 3] *= d4.w;
            }
            store_high(cold, y, h);
            signal(&B->dh);
            store_low(cold + 16, y, h);
            signal(&B->dl);
            tmem_ld32(colu, y);
            tmem_ld_wait();
            store_high(colu, y, h);
            store_low(colu + 16, y, h);
            signal(&B->uo);
            // ---- X = G_63 X + dX ----------------------------------------------------------
            const float gc = vec[2 * C + C - 1];
            wait_all(&B->dx, p);
            if (fail) break;
#pragma unroll
            for (int q = 0; q < XH / 32; ++q) {
                tmem_ld32(colx + 32 * q, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) X[32 * q + i] = gc * X[32 * q + i] + y[i];
            }
            if (c + 1 < w.blocks) publish_x();
            last = at;
            at.next();
        }
        if (fail) break;
#pragma unroll
        for (int q = 0; q < XH / 32; ++q) tmem_st32(colx + 32 * q, reinterpret_cast<const uint32_t(&)[32]>(X[32 * q]));
        tmem_st_wait();
        __syncwarp();
        tmem_ld_rows<XH / 2>(colx, X);
        tmem_ld_rows<XH / 2>(colx + (16u << 16), X + XH / 2);
        tmem_ld_wait();
        float* sp = state_row(w);
#pragma unroll
        for (int i = 0; i < XH; i += 2) {
            const int h16 = i / (XH / 2), e = i % (XH / 2);
            __stcs(reinterpret_cast<float2*>(sp + (16 * h16 + 8 * ((e / 2) & 1)) * DK + 8 * (e / 4)), make_float2(X[i], X[i + 1]));
        }
        }
        if (!fail && nb > 0) {
            outputs(nb - 1, last.s, 0);
            outputs(nb - 1, last.s, 1);
        }
        if (fail) status = kStatusMmaWait;
    } else if (warp < kConvWarps + kPrepWarps) {
        if (!prep_warps<DK>(a, sm, sbase, B, tmem)) {
            fail = true;
            status = kStatusMmaWait;
            *abort = 1;
            if (warp == kConvWarps + 2 && elect_one()) {   // the lane that issued this role's MMAs
                mma_commit(&B->drain[1]);
                mbar_wait(&B->drain[1], 0, 100000000ull);
            }
            __syncwarp();
        }
    } else if (warp == kConvWarps + kPrepWarps) {
        // ======================= MMA issue ==========================================
        {
            const bool el = elect_one();
            constexpr uint32_t ID_64 = idesc_bf16(128, 64, false, false);
            constexpr uint32_t ID_V = idesc_bf16(128, 64, true, false);    // V^T T'^T
            constexpr uint32_t ID_K = idesc_bf16(128, DK, false, true);    // U' K
            // the A operands of k-step kk: channels 16 kk .., tokens 16 kk ..
            auto colx = [&](int kk) { return tmem + L::COL_X + (kk / (XH / 16)) * XH + (kk % (XH / 16)) * 8; };
            auto colt = [](uint32_t col, int kk) { return col + (kk / 2) * 32 + (kk % 2) * 8; };
            auto kstep = [](int kk) { return static_cast<uint64_t>((kk / 4) * 1024 + (kk % 4) * 2); };
            // operand descriptors of stage 0; offsets in 16-byte units are added to them
            const uint64_t dK0 = kmaj(sbase + L::KQ), dKm0 = mnmaj(sbase + L::KQ, 16384), dV0 = mnmaj(sbase + L::V, 8192);
            const uint64_t dT0 = kmaj(sbase + L::TP);
            const uint32_t cz = tmem + L::COL_Z, cu = tmem + L::COL_U, cd = tmem + L::COL_UD;
            auto wait_w = [&](uint64_t* b, uint32_t parity) {   // the whole warp goes on, or gives up, together
                const bool ok = !fail && wait_bar(b, parity, abort);
                fail = !__all_sync(0xffffffffu, ok);
                tc_fence_after();
            };
            Ring3 at;
            Work w;
            int nb = 0;   // blocks of the CTA so far
            for (int k = 0; !fail && next_item(B, k, w, fail); ++k)
            for (int c = 0; c < w.blocks && !fail; ++c, ++nb, at.next()) {
                const uint32_t p = nb & 1;
                const uint64_t dK = dK0 + at.s * (L::KQ_BYTES / 16), dKm = dKm0 + at.s * (L::KQ_BYTES / 16);
                const uint64_t dV = dV0 + at.s * (L::V_BYTES / 16);
                const uint64_t dT = dT0 + p * (L::TP_BYTES / 16);
                auto start_u = [&]() {   // U = V^T T'^T, both parts of T'; the parts of the U before are read by now
                    wait_w(&B->v_full[at.s], at.phase);
                    if (nb >= 1) wait_w(&B->o, p ^ 1);
                    if (!fail && el) {
#pragma unroll 1
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_bf16_ss(cu, dV + kk * 128, dT + kk * 2, ID_V, kk > 0);
                            mma_bf16_ss(cu, dV + kk * 128, dT + 512 + kk * 2, ID_V, true);
                        }
                    }
                };
                // before X is published if T' is there already
                const bool u_early = __all_sync(0xffffffffu, mbar_try_wait(smem_u32(&B->ready[p]), (nb >> 1) & 1));
                if (u_early) start_u();
                wait_w(&B->kq_full[at.s], at.phase);
                if (w.len - c * C < C) wait_w(&B->ready[p], (nb >> 1) & 1);   // K's rows past the end are zeroed
                wait_w(&B->xh, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < DK / 16; ++kk) mma_bf16_ts(cz, colx(kk), dK + kstep(kk), ID_64, kk > 0);
                }
                wait_w(&B->xl, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < DK / 16; ++kk) mma_bf16_ts(cz, colx(kk) + XH / 2, dK + kstep(kk), ID_64, true);
                    mma_commit(&B->z);
                }
                if (!u_early) {
                    wait_w(&B->ready[p], (nb >> 1) & 1);
                    start_u();
                }
                wait_w(&B->rh, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_bf16_ts(cu, colt(cz, kk), dT + kk * 2, ID_64, true);
                        mma_bf16_ts(cu, colt(cz, kk), dT + 512 + kk * 2, ID_64, true);
                    }
                }
                wait_w(&B->rl, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(cu, colt(cz, kk) + 16, dT + kk * 2, ID_64, true);
                    mma_commit(&B->u);
                }
                if (nb >= 1) {   // the outputs of the block before are read
                    Ring3 before = at;
                    before.next();
                    before.next();   // the stage of block nb + 2, and of block nb - 1 a round earlier
                    wait_w(&B->ot_full[before.s], before.phase ^ 1);
                    if (fail) break;
                }
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_bf16_ts(tmem + L::COL_O1, colx(kk), dK + 512 + kstep(kk), ID_64, kk > 0);
                    mma_commit(&B->o1);
                }
                wait_w(&B->dh, p);
                wait_w(&B->o1, p);   // X is read: dX may take its columns
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(tmem + L::COL_X, colt(cd, kk), dKm + kk * 128, ID_K, kk > 0);
                }
                wait_w(&B->dl, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(tmem + L::COL_X, colt(cd, kk) + 16, dKm + kk * 128, ID_K, true);
                    mma_commit(&B->dx);
                }
                wait_w(&B->uo, p);
                if (fail) break;
                if (el) {
#pragma unroll 1
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_bf16_ts(tmem + L::COL_O2, colt(cu, kk), dT + 1024 + kk * 2, ID_64, kk > 0);
                        mma_bf16_ts(tmem + L::COL_O2, colt(cu, kk) + 16, dT + 1024 + kk * 2, ID_64, true);
                    }
                    mma_commit(&B->o);
                    mma_commit(&B->kq_free[at.s]);
                    mma_commit(&B->tp_free[p]);
                }
            }
            // the last arrivals that nobody else waits for: after the CTA has left they would hit another's memory
            for (int m = nb < kTiles ? 0 : nb - kTiles; m < nb && !fail; ++m) wait_w(&B->kq_free[m % kTiles], (m / kTiles) & 1);
            for (int m = nb < 2 ? 0 : nb - 2; m < nb && !fail; ++m) wait_w(&B->tp_free[m & 1], (m >> 1) & 1);
            if (fail) {   // every MMA issued completes before the CTA leaves (bounded)
                status = kStatusMmaWait;
                if (el) {
                    mma_commit(&B->drain[0]);
                    mbar_wait(&B->drain[0], 0, 100000000ull);
                }
                __syncwarp();
            }
        }
    } else if (warp == kConvWarps + kPrepWarps + 1) {
        // ======================= loads ===============================================
        Ring3 at;
        Work w;
        int nb = 0;
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k)
            for (int c = 0; c < w.blocks && !fail; ++c, ++nb, at.next()) {
                const int s = at.s, row = w.row0 + c * C;
                if (lane == 0) {
                    if (c + kTiles < w.blocks) {   // into L2, three blocks ahead
#pragma unroll
                        for (int x = 0; x < KA; ++x) {
                            prefetch_3d(&tmk, x * 64, w.khead, row + kTiles * C);
                            prefetch_3d(&tmq, x * 64, w.khead, row + kTiles * C);
                        }
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x) prefetch_3d(&tmv, x * 64, w.head, row + kTiles * C);
                    }
                    if (nb >= kTiles) wait(&B->kq_free[s], at.phase ^ 1);
                    if (!fail) {
                        uint8_t* kq = sm + L::KQ + s * L::KQ_BYTES;
                        mbar_arrive_expect_tx(&B->kq_full[s], L::KQ_BYTES);
#pragma unroll
                        for (int x = 0; x < KA; ++x) {
                            tma_load_3d(&tmk, &B->kq_full[s], kq + x * 16384, x * 64, w.khead, row);
                            tma_load_3d(&tmq, &B->kq_full[s], kq + x * 16384 + 8192, x * 64, w.khead, row);
                        }
                    }
                    if (nb >= kTiles) wait(&B->v_free[s], at.phase ^ 1);
                    if (!fail) {
                        uint8_t* v = sm + L::V + s * L::V_BYTES;
                        mbar_arrive_expect_tx(&B->v_full[s], L::V_BYTES);
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x) tma_load_3d(&tmv, &B->v_full[s], v + x * 8192, x * 64, w.head, row);
                        if (c + 1 == w.blocks) mbar_arrive(&B->want);
                    }
                }
                fail = __any_sync(0xffffffffu, fail);
            }
        if (lane == 0) {
            // After a failure loads may be in flight: let them land (bounded; a
            // phase that no load began runs into the limit).
            if (fail || *abort) {
                status = kStatusTmaWait;
                for (int i = 0; i < kTiles; ++i)
                    for (uint32_t ph = 0; ph < 2; ++ph) {
                        mbar_wait(&B->kq_full[i], ph, 10000000ull);
                        mbar_wait(&B->v_full[i], ph, 10000000ull);
                    }
            }
        }
    } else if (warp == kConvWarps + kPrepWarps + 2) {
        // ======================= output copies =======================================
        Ring3 at;
        Work w;
        const size_t ostep = static_cast<size_t>(a.Hv) * DV;
        for (int k = 0; !fail && next_item(B, k, w, fail); ++k) {
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(w.row0) * a.Hv + w.head) * DV;
            for (int c = 0; c < w.blocks; ++c, at.next()) {
                wait(&B->ot_full[at.s], at.phase);
                fail = !__all_sync(0xffffffffu, !fail);
                if (fail) break;
                const uint32_t ot = sbase + L::V + at.s * L::V_BYTES;
                const int n = min(C, w.len - c * C);
                const int ch = lane & 15;
#pragma unroll 8
                for (int t = lane >> 4; t < n; t += 2) {
                    const uint4 y = ld_shared_v4(ot + t * 256 + ((ch ^ ((t & 1) << 2)) << 4));
                    *reinterpret_cast<uint4*>(op + static_cast<size_t>(c * C + t) * ostep + ch * 8) = y;
                }
                fence_proxy_async_smem();   // the tile's generic accesses come before the load that overwrites it
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->v_free[at.s]);
            }
        }
        if (fail) status = kStatusMmaWait;
    } else {
        // ======================= work ================================================
        int idx = blockIdx.x;
        for (int k = 0;; ++k) {
            Request rq;
            const bool have = idx >= 0 && read_request(a, idx / a.Hv, rq);
            const int i = k % kItems;
            if (k >= kItems) wait(&B->item_free[i], ((k / kItems) & 1) ^ 1);
            fail = __any_sync(0xffffffffu, fail);
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
            if (!have) break;
            // what the item begins with, into L2
            if (!w.fresh) {
                const float* st = a.states + (static_cast<size_t>(w.slot) * a.Hv + w.head) * DV * DK;
                for (int x = lane; x < DV * DK / 32; x += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(st + 32 * x));
            }
            if (lane < min(w.blocks, kTiles)) {
                const int row = w.row0 + lane * C;
#pragma unroll
                for (int x = 0; x < KA; ++x) {
                    prefetch_3d(&tmk, x * 64, w.khead, row);
                    prefetch_3d(&tmq, x * 64, w.khead, row);
                }
#pragma unroll
                for (int x = 0; x < DV / 64; ++x) prefetch_3d(&tmv, x * 64, w.head, row);
            }
            // more work only once this item's loads are under way: what waits here could run elsewhere
            wait(&B->want, k & 1);
            fail = __any_sync(0xffffffffu, fail);
            if (fail) break;
            if (lane == 0) steal_request(&B->answer, &B->stolen);
            wait(&B->stolen, k & 1);
            fail = __any_sync(0xffffffffu, fail);
            if (fail) break;
            idx = stolen_index(&B->answer);
            fence_proxy_async_smem();   // this read comes before the next answer's write
            __syncwarp();
        }
        if (fail) status = kStatusFlagWait;
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

// The gated delta rule over packed requests in blocks of 32 tokens: bf16 q, k
// and v, fp32 states in a pool.
//
// Per value head (key head h * Hk / Hv), state X [dv][dk] at a block's start,
// tokens t, j of the block, g and b the gates:
//   D_tj = prod_{j < s <= t} g_s,  G_t = prod_{s <= t} g_s
//   A_tj = b_t D_tj k_t.k_j  (j < t),   T = (I + A)^-1,   P_tj = D_tj q_t.k_j  (j <= t)
//   R = diag(b) (V - diag(G) K X^T),   U = T R             [token][dv]
//   O = diag(G) Q X^T + P U,           X <- G_31 X + U^T diag(D_31,.) K
// The decays are running products, never quotients or logarithms, so a gate may
// be zero or negative. (Gates above 1 whose product over a block overflows give
// infinity times zero where the recurrence may stay finite.)
//
// Work split. One CTA per (request, value head, 64 or 32 rows of the state),
// longest requests first: rows of the state are independent. Four chain warps
// own 16 rows each, for the whole request. With X^T's products written as
// [dv][token], a warp's accumulators (X, Z = X K^T, R, U) turn into the next
// product's A operand inside its own registers, so from the state's load to
// its store the chain exchanges nothing between warps. K, Q, V tiles come by
// TMA into a ring of three stages; two prep warps compute T and P of a block
// each, ahead of the chain. The last chain warp to leave a stage issues the
// loads that reuse it.
// Where there are no more CTAs of 32 rows than SMs, each has an SM to itself:
// more stages, two chain warps to 16 rows, half of the channels each, who add
// up Z through shared memory, and an output warp to 16 rows, to which they hand
// X (high parts) and U.
//
// Precision. q, k, v are bf16 and enter the MMAs as they are. What the state
// depends on (X in K X^T, R and T in T R, U in U^T K) is split into two bf16
// parts, high and low, whose sum is off by at most 2^-16 of the value;
// products of two low parts (2^-16 again) are dropped. Measured: states off by
// 3.6e-6 of themselves against float64 (one part alone: about 2e-3). What only
// an output depends on, rounded to bf16 itself, keeps one part where the other
// factor is exact: X in Q X^T, P in P U.
// Accumulators, gates, A and the inverse are fp32.
//
// Bound by latency: a block's products follow one another inside a warp, some
// 2000 to 2700 clocks at d_k 64 for 66 to 110 MMAs of 8 each and their operands'
// splits. Measured, 16 heads: one request at d 64 of 130 tokens 8.4 us, of 2048
// 66 us (1.0 us a block); at d_k 128, d_v 64 82 us; two of 8192 at d 128 363 us.
// By CTAs of 64 rows: 9.7, 92, 131 and 511 us; without the output warps 8.3, 82,
// 100 and 399. Nine of 2048 at d_k 128, d_v 64 (64 rows): 136 us, and 201 us with
// prep warps that took T and P of every block instead of alternate blocks.
// Fragments loaded ahead of the exchange of Z: no gain (74 us for 71).
//
// Rows past a request's end belong to the next request: they are zeroed in the
// tiles before anything reads them, with gate 1 and beta 0, and are not
// written.
#include <cuda.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "launch.cuh"
#include "packed.h"
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace la {
namespace packed {
namespace {

constexpr int C = 32;                      // tokens per block
constexpr int kTStride = 80;               // bytes per row of a 32x32 bf16 tile: 16-byte chunks of 8 rows hit all banks
// prep warps' fp32 scratch: two 16x16 sub-blocks each of K K^T and Q K^T, rows and blocks so far apart that the MMA
// fragments' stores and the column reads of both halves of the warp hit all banks; then the gates
constexpr int kSStride = 24;
constexpr int kSBlock = 16 * kSStride + 16;
constexpr int kScratch = 4 * kSBlock + C;

constexpr int lcm(int a, int b) {
    int x = a;
    while (x % b) x += a;
    return x;
}

// A CTA's shape: ROWS state rows, the channels of each split over SPLIT warps, PREP prep warps, STAGES blocks in flight.
template <int DK_, int ROWS_, int SPLIT_, int PREP_, int STAGES_>
struct Layout {
    static constexpr int DK = DK_, ROWS = ROWS_, SPLIT = SPLIT_, PREP = PREP_, STAGES = STAGES_;
    static constexpr int GROUPS = ROWS / 16;                 // of 16 state rows
    static constexpr int CHAIN = GROUPS * SPLIT;             // chain warps
    static constexpr int OUT = SPLIT > 1 ? GROUPS : 0;       // warps that compute the outputs (else the chain does)
    static constexpr int THREADS = 32 * (CHAIN + OUT + PREP);
    // barriers of arrived tiles: so many that a prep warp waits for every turn of those it waits for at all (one that
    // sees every other turn of a barrier could take the turn before for its own)
    static constexpr int FULL = lcm(PREP, STAGES);
    static constexpr int KA = DK / 64;                       // 64-channel atoms of [32][64] bf16, 4 KB, 128-byte swizzle
    static constexpr uint32_t K = 0;
    static constexpr uint32_t Q = K + KA * 4096;
    static constexpr uint32_t V = Q + KA * 4096;             // [32][64]: the CTA's own rows of the state among them
    static constexpr uint32_t TX = V + 4096;                 // bytes a stage's loads bring
    static constexpr uint32_t TH = TX;                       // T, high and low parts, [t][j]
    static constexpr uint32_t TL = TH + C * kTStride;
    static constexpr uint32_t P = TL + C * kTStride;
    static constexpr uint32_t VEC = P + C * kTStride;        // fp32: b, b G, G, D_31 [32 each]
    static constexpr uint32_t STAGE = (VEC + 4 * C * 4 + 1023) / 1024 * 1024;
    static constexpr uint32_t SCRATCH = STAGES * STAGE;      // kScratch floats per prep warp
    static constexpr uint32_t ZX = SCRATCH + PREP * kScratch * 4;             // SPLIT 2: [2][CHAIN] partial Z, 2 KB
    static constexpr uint32_t XO = ZX + (SPLIT > 1 ? 2 * CHAIN * 2048 : 0);        // [2][OUT] X, high parts: 512 a step of 16
    static constexpr uint32_t UO = XO + 2 * OUT * (DK / 16) * 512;                 // [2][OUT] U, both parts: 2 KB
    static constexpr uint32_t BAR = UO + 2 * OUT * 2048;
    static constexpr uint32_t BYTES = BAR + 512;
    static_assert(SPLIT <= 2 && (FULL + STAGES + 5 * GROUPS) * 8 + STAGES * 4 + 8 <= 512, "barrier space");
};

__device__ __forceinline__ void st_shared_4(uint32_t addr, const uint32_t (&x)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
__device__ __forceinline__ void ld_shared_4(uint32_t (&x)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0) : "memory");
}

struct Item {
    int head, khead, split;
    Request rq;
    int blocks;
};

// ---------------------------------------------------------------- prep warps
// T (two bf16 parts), P and the gate vectors of blocks pw, pw + PREP, ...
//
// By 16x16 sub-blocks: the diagonal ones by forward substitution in fp32, lane
// l one column of sub-block l / 16; the one below them as T21 = -T22 (A21 T11)
// on the tensor cores, operands in two bf16 parts. Between the halves the
// decay factors: D_tj = (g_16 .. g_t)(g_{j+1} .. g_15) for j < 16 <= t.
template <class L>
__device__ __forceinline__ void prep_warp(const StepArgs& a, const Item& it, uint8_t* sm, uint32_t sbase, int pw,
                                          uint64_t* full, uint64_t* ready, volatile int* abort_flag) {
    constexpr int DK = L::DK;
    const int lane = threadIdx.x & 31, gq = lane >> 2, cq = lane & 3;
    const int blk = lane >> 4, col = lane & 15;
    float* kk = reinterpret_cast<float*>(sm + L::SCRATCH) + pw * kScratch;   // diagonal sub-blocks of K K^T, then A
    float* qk = kk + 2 * kSBlock;                                            // and of Q K^T
    float* gs = qk + 2 * kSBlock;                                            // gates [32]
    // A fragment of an m16 x k16 tile by ldmatrix: lane -> row, 16-byte chunk
    // (the same addresses, transposed, give the B fragments of a k16 x n16 tile)
    const int fr = (lane & 7) + ((lane >> 3) & 1) * 8, fc = lane >> 4;
    auto gates = [&](int c, float& g, float& b) {   // token `lane` of block c; gate 1, beta 0 past the end
        const int t = c * C + lane;
        g = 1.f;
        b = 0.f;
        if (t < it.rq.len) {
            const size_t i = static_cast<size_t>(it.rq.row0 + t) * a.Hv + it.head;
            g = __ldg(a.gate + i);
            b = __ldg(a.beta + i);
        }
    };
    float gn, bn;
    gates(pw, gn, bn);
    for (int c = pw; c < it.blocks; c += L::PREP) {
        const int s = c % L::STAGES;
        const uint32_t st = sbase + s * L::STAGE;
        const float g = gn, b = bn;
        gates(c + L::PREP, gn, bn);
        // ---- gate vectors: products inside each half, then over the block ----------------
        float G = g;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, G, o);
            if (col >= o) G *= y;
        }
        const float Gq = G;   // (second half) the gates from 16 up to this token
        const float G15 = __shfl_sync(0xffffffffu, G, 15), G31 = __shfl_sync(0xffffffffu, G, 31);
        if (blk) G *= G15;
        gs[lane] = g;
        bool ok = mbar_wait_or_abort(&full[c % L::FULL], (c / L::FULL) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return;
        float* vec = reinterpret_cast<float*>(sm + s * L::STAGE + L::VEC);
        vec[lane] = b;
        vec[C + lane] = b * G;
        vec[2 * C + lane] = G;
        const int n = it.rq.len - c * C;   // tokens of the block
        if (n < C) {                       // rows of the next request (or past the tensor): zero
            for (int i = lane; i < (C - n) * 8; i += 32) {
                const uint32_t o = sw128_off(n + i / 8, i % 8);
#pragma unroll
                for (int at = 0; at < L::KA; ++at) {
                    st_shared_zero16(st + L::K + at * 4096 + o);
                    st_shared_zero16(st + L::Q + at * 4096 + o);
                }
                st_shared_zero16(st + L::V + o);
            }
            __syncwarp();
        }
        // ---- K K^T and Q K^T, lower tiles only; a key fragment serves as A and as B ----
        float dk[6][4] = {}, dq[6][4] = {};   // tiles (m, n): (0,0) (0,1) (1,0) (1,1) (1,2) (1,3)
        uint32_t f[2][4][4];                  // fragments k rows 0-15, 16-31, q rows 0-15, 16-31; one step ahead
        auto load = [&](int x, uint32_t (&w)[4][4]) {
            const uint32_t at = (x / 4) * 4096, ch = (x % 4) * 2 + fc;
            ldsm4(w[0], st + L::K + at + sw128_off(fr, ch));
            ldsm4(w[1], st + L::K + at + sw128_off(16 + fr, ch));
            ldsm4(w[2], st + L::Q + at + sw128_off(fr, ch));
            ldsm4(w[3], st + L::Q + at + sw128_off(16 + fr, ch));
        };
        load(0, f[0]);
#pragma unroll
        for (int x = 0; x < DK / 16; ++x) {
            if (x + 1 < DK / 16) load(x + 1, f[(x + 1) & 1]);
            const auto& w = f[x & 1];
            mma_16816(dk[0], w[0], w[0][0], w[0][2]);
            mma_16816(dk[1], w[0], w[0][1], w[0][3]);
            mma_16816(dk[2], w[1], w[0][0], w[0][2]);
            mma_16816(dk[3], w[1], w[0][1], w[0][3]);
            mma_16816(dk[4], w[1], w[1][0], w[1][2]);
            mma_16816(dk[5], w[1], w[1][1], w[1][3]);
            mma_16816(dq[0], w[2], w[0][0], w[0][2]);
            mma_16816(dq[1], w[2], w[0][1], w[0][3]);
            mma_16816(dq[2], w[3], w[0][0], w[0][2]);
            mma_16816(dq[3], w[3], w[0][1], w[0][3]);
            mma_16816(dq[4], w[3], w[1][0], w[1][2]);
            mma_16816(dq[5], w[3], w[1][1], w[1][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* k0 = kk + h * kSBlock + gq * kSStride + 8 * i + 2 * cq;
                float* q0 = qk + h * kSBlock + gq * kSStride + 8 * i + 2 * cq;
                const float(&x)[4] = dk[4 * h + i];
                const float(&y)[4] = dq[4 * h + i];
                *reinterpret_cast<float2*>(k0) = make_float2(x[0], x[1]);
                *reinterpret_cast<float2*>(k0 + 8 * kSStride) = make_float2(x[2], x[3]);
                *reinterpret_cast<float2*>(q0) = make_float2(y[0], y[1]);
                *reinterpret_cast<float2*>(q0 + 8 * kSStride) = make_float2(y[2], y[3]);
            }
        __syncwarp();
        // ---- A and P of the diagonal sub-blocks: D_tj is the lane's running product -------
        float* ak = kk + blk * kSBlock;
        const float* aq = qk + blk * kSBlock;
        float kc[16], qc[16], gt[16], bt[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            kc[t] = ak[t * kSStride + col];
            qc[t] = aq[t * kSStride + col];
        }
#pragma unroll
        for (int t = 0; t < 16; t += 4) {
            *reinterpret_cast<float4*>(&gt[t]) = *reinterpret_cast<const float4*>(gs + 16 * blk + t);
            *reinterpret_cast<float4*>(&bt[t]) = *reinterpret_cast<const float4*>(vec + 16 * blk + t);
        }
        float d = 0.f;   // zero above the diagonal
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            d = t == col ? 1.f : d * gt[t];
            kc[t] = t > col ? bt[t] * d * kc[t] : 0.f;
            qc[t] = t >= col ? d * qc[t] : 0.f;
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            ak[t * kSStride + col] = kc[t];
            st_shared_u16(st + L::P + (16 * blk + t) * kTStride + 2 * lane, __float2bfloat16_rn(qc[t]));
        }
        vec[3 * C + lane] = blk ? d : d * G31;
        __syncwarp();
        // ---- their inverses by forward substitution ----------------------------------------
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float s0 = t == col ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int i = 0; i < t; i += 4) {
                const float4 r = *reinterpret_cast<const float4*>(ak + t * kSStride + i);
                s0 -= r.x * x[i];
                if (i + 1 < t) s1 -= r.y * x[i + 1];
                if (i + 2 < t) s2 -= r.z * x[i + 2];
                if (i + 3 < t) s3 -= r.w * x[i + 3];
            }
            x[t] = (s0 + s1) + (s2 + s3);
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(x[t]);
            st_shared_u16(st + L::TH + (16 * blk + t) * kTStride + 2 * lane, hi);
            st_shared_u16(st + L::TL + (16 * blk + t) * kTStride + 2 * lane, __float2bfloat16_rn(x[t] - __bfloat162float(hi)));
        }
        // ---- the sub-block below: P21 = Q S qk, A21 = b Q S kk (Q by token, S by column) --------
        const float Q0 = __shfl_sync(0xffffffffu, Gq, 16 + gq), Q1 = __shfl_sync(0xffffffffu, Gq, 24 + gq);
        const float b0 = __shfl_sync(0xffffffffu, b, 16 + gq), b1 = __shfl_sync(0xffffffffu, b, 24 + gq);
        uint32_t ah[4], al[4];
        {
            float S[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                S[i][0] = __shfl_sync(0xffffffffu, d, 8 * i + 2 * cq);
                S[i][1] = __shfl_sync(0xffffffffu, d, 8 * i + 2 * cq + 1);
                float(&y)[4] = dq[2 + i];
                st_shared_b32(st + L::P + (16 + gq) * kTStride + 16 * i + 4 * cq, pack_bf16(Q0 * S[i][0] * y[0], Q0 * S[i][1] * y[1]));
                st_shared_b32(st + L::P + (24 + gq) * kTStride + 16 * i + 4 * cq, pack_bf16(Q1 * S[i][0] * y[2], Q1 * S[i][1] * y[3]));
                float(&z)[4] = dk[2 + i];
                z[0] *= b0 * Q0 * S[i][0];
                z[1] *= b0 * Q0 * S[i][1];
                z[2] *= b1 * Q1 * S[i][0];
                z[3] *= b1 * Q1 * S[i][1];
            }
            split_tiles(dk[2], dk[3], ah, al);
        }
        __syncwarp();
        float M[2][4] = {}, N[2][4] = {};
        {
            uint32_t th[4], tl[4];   // T11 [k = s][n = j]
            ldsm4t(th, st + L::TH + fr * kTStride + 16 * fc);
            ldsm4t(tl, st + L::TL + fr * kTStride + 16 * fc);
            mma_16816(M[0], ah, th[0], th[1]);
            mma_16816(M[1], ah, th[2], th[3]);
            mma_16816(M[0], al, th[0], th[1]);
            mma_16816(M[1], al, th[2], th[3]);
            mma_16816(M[0], ah, tl[0], tl[1]);
            mma_16816(M[1], ah, tl[2], tl[3]);
        }
        {
            uint32_t th[4], tl[4], mh[4], ml[4];   // T22 [t][s]; M [k = s][n = j], transposed between lanes
            ldsm4(th, st + L::TH + (16 + fr) * kTStride + 32 + 16 * fc);
            ldsm4(tl, st + L::TL + (16 + fr) * kTStride + 32 + 16 * fc);
            split_tiles(M[0], M[1], mh, ml);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mh[i] = transpose8x8(mh[i]);
                ml[i] = transpose8x8(ml[i]);
            }
            mma_16816(N[0], th, mh[0], mh[1]);
            mma_16816(N[1], th, mh[2], mh[3]);
            mma_16816(N[0], tl, mh[0], mh[1]);
            mma_16816(N[1], tl, mh[2], mh[3]);
            mma_16816(N[0], th, ml[0], ml[1]);
            mma_16816(N[1], th, ml[2], ml[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi, lo;
                split2(-N[i][2 * h], -N[i][2 * h + 1], hi, lo);
                st_shared_b32(st + L::TH + (16 + 8 * h + gq) * kTStride + 16 * i + 4 * cq, hi);
                st_shared_b32(st + L::TL + (16 + 8 * h + gq) * kTStride + 16 * i + 4 * cq, lo);
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[s]);
    }
}

// ---------------------------------------------------------------- the kernel

template <class L, int RESIDENT>
__global__ void __launch_bounds__(L::THREADS, RESIDENT)
chunk_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
             const __grid_constant__ CUtensorMap tmv, const StepArgs a) {
    constexpr int DK = L::DK, SPLIT = L::SPLIT, STAGES = L::STAGES;
    constexpr int NT = DK / 8 / SPLIT;   // n-tiles of a warp's part of its state rows
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR);   // [FULL] TMA: a block's tiles have arrived
    uint64_t* ready = full + L::FULL;                            // [STAGES] prep: T, P and vectors are written
    uint64_t* swap = ready + STAGES;                             // [GROUPS] both warps of 16 rows have written their parts
    uint64_t* given = swap + L::GROUPS;                          // [2][GROUPS] chain: X and U are there for the outputs
    uint64_t* taken = given + 2 * L::GROUPS;                     // [2][GROUPS] output warp: they are read
    int* left = reinterpret_cast<int*>(taken + 2 * L::GROUPS);   // [STAGES] warps that have left the stage
    volatile int* issued = left + STAGES;                        // blocks whose loads were issued
    volatile int* abort_flag = left + STAGES + 1;

    if (tid == 0) {
        for (int i = 0; i < L::FULL; ++i) mbar_init(&full[i], 1);
        for (int i = 0; i < L::GROUPS; ++i) {
            mbar_init(&swap[i], SPLIT);
            for (int b = i; b < 2 * L::GROUPS; b += L::GROUPS) {   // one for each buffer: the sides may be two blocks apart
                mbar_init(&given[b], SPLIT);
                mbar_init(&taken[b], 1);
            }
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&ready[i], 1);
            left[i] = 0;
        }
        *issued = 0;
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    griddep_wait();
    Item it;
    {
        const int splits = a.dv / L::ROWS;
        const int per_req = a.Hv * splits;
        const int rank = blockIdx.x / per_req, hs = blockIdx.x % per_req;
        if (a.above) griddep_launch_dependents();   // a launch for the shorter requests follows, which may run beside this one
        if (!read_request(a, rank, it.rq)) return;
        it.head = hs / splits;
        it.split = hs % splits;
        it.khead = it.head / (a.Hv / a.Hk);
        it.blocks = (it.rq.len + C - 1) / C;
    }
    __syncthreads();

    auto issue = [&](int c) {   // loads of block c (one thread); rows past the tensor read as zeros
        const int row = it.rq.row0 + c * C;
        uint8_t* st = sm + c % STAGES * L::STAGE;
        uint64_t* bar = &full[c % L::FULL];
        mbar_arrive_expect_tx(bar, L::TX);
#pragma unroll
        for (int x = 0; x < L::KA; ++x) {
            tma_load_3d(&tmk, bar, st + L::K + x * 4096, x * 64, it.khead, row);
            tma_load_3d(&tmq, bar, st + L::Q + x * 4096, x * 64, it.khead, row);
        }
        tma_load_3d(&tmv, bar, st + L::V, it.split * L::ROWS / 64 * 64, it.head, row);
        *issued = c + 1;
    };
    if (tid == 0)
        for (int c = 0; c < STAGES && c < it.blocks; ++c) issue(c);

    // a warp has read stage c % STAGES: the last one to say so reloads it
    auto leave = [&](int c) {
        __syncwarp();
        if (lane == 0) {
            const int s = c % STAGES;
            int before;
            asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(smem_u32(&left[s])) : "memory");
            if (before == L::CHAIN + L::OUT - 1 && c + STAGES < it.blocks) {
                left[s] = 0;
                issue(c + STAGES);
            }
        }
    };
    auto here = [&](int c) {   // block c's tiles, T, P and vectors
        const bool ok = mbar_wait_or_abort(&full[c % L::FULL], (c / L::FULL) & 1, abort_flag) &&
                        mbar_wait_or_abort(&ready[c % STAGES], (c / STAGES) & 1, abort_flag);
        return __all_sync(0xffffffffu, ok);
    };
    const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;   // ldmatrix: B fragments of two n-tiles (rows = n, 16-byte chunks along k)
    const size_t ostep = static_cast<size_t>(a.Hv) * a.dv;
    // outputs, rounded: [dv][token] fragments y of tokens 8n .. of block c, turned to [token][dv] pairs
    auto store_out = [&](__nv_bfloat16* op, int n, int c, const uint32_t (&y)[2]) {
        const uint32_t y0 = transpose8x8(y[0]);   // token 8n + g, rows 2c, 2c + 1
        const uint32_t y1 = transpose8x8(y[1]);   // rows 8 + 2c, ..
        const int t = c * C + 8 * n + (lane >> 2);
        if (c >= 0 && t < it.rq.len) {
            __nv_bfloat16* o = op + static_cast<size_t>(t) * ostep;
            *reinterpret_cast<uint32_t*>(o) = y0;
            *reinterpret_cast<uint32_t*>(o + 8) = y1;
        }
    };
    auto out_rows = [&](int r0) {
        return static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(it.rq.row0) * a.Hv + it.head) * a.dv + r0 + 2 * (lane & 3);
    };
    // O = X Q^T (channels 16 x ..), high parts of X
    auto read_step = [&](uint32_t st, int x, const uint32_t (&hi)[4], float (&O)[4][4]) {
        uint32_t b0[4], b1[4];
        const uint32_t at = st + L::Q + (x / 4) * 4096, ch = (x % 4) * 2 + bc;
        ldsm4(b0, at + sw128_off(br, ch));
        ldsm4(b1, at + sw128_off(16 + br, ch));
        mma_16816(O[0], hi, b0[0], b0[1]);
        mma_16816(O[1], hi, b0[2], b0[3]);
        mma_16816(O[2], hi, b1[0], b1[1]);
        mma_16816(O[3], hi, b1[2], b1[3]);
    };
    // O = G O + P U
    auto load_p = [&](uint32_t st, uint32_t (&t0)[4], uint32_t (&t1)[4], uint32_t (&t2)[4]) {
        const uint32_t tp = st + L::P + br * kTStride + bc * 16;
        ldsm4(t0, tp);
        ldsm4(t1, tp + 16 * kTStride);
        ldsm4(t2, tp + 16 * kTStride + 32);
    };
    auto finish_out = [&](const float* vec, const uint32_t (&t0)[4], const uint32_t (&t1)[4], const uint32_t (&t2)[4],
                          const uint32_t (&h0)[4], const uint32_t (&l0)[4], const uint32_t (&h1)[4], const uint32_t (&l1)[4],
                          float (&O)[4][4]) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 g = *reinterpret_cast<const float2*>(vec + 2 * C + 8 * n + 2 * (lane & 3));
            O[n][0] *= g.x;
            O[n][1] *= g.y;
            O[n][2] *= g.x;
            O[n][3] *= g.y;
        }
        mma_16816(O[0], h0, t0[0], t0[1]);
        mma_16816(O[1], h0, t0[2], t0[3]);
        mma_16816(O[2], h0, t1[0], t1[1]);
        mma_16816(O[3], h0, t1[2], t1[3]);
        mma_16816(O[0], l0, t0[0], t0[1]);
        mma_16816(O[1], l0, t0[2], t0[3]);
        mma_16816(O[2], l0, t1[0], t1[1]);
        mma_16816(O[3], l0, t1[2], t1[3]);
        mma_16816(O[2], h1, t2[0], t2[1]);
        mma_16816(O[3], h1, t2[2], t2[3]);
        mma_16816(O[2], l1, t2[0], t2[1]);
        mma_16816(O[3], l1, t2[2], t2[3]);
    };

    bool failed = false;
    if (warp >= L::CHAIN + L::OUT) {
        prep_warp<L>(a, it, sm, sbase, warp - L::CHAIN - L::OUT, full, ready, abort_flag);
    } else if (warp >= L::CHAIN) {
        // ======================= output warp: 16 rows =======================================
        const int grp = warp - L::CHAIN;
        __nv_bfloat16* op = out_rows(it.split * L::ROWS + 16 * grp);
        for (int c = 0; c < it.blocks; ++c) {
            const uint32_t st = sbase + c % STAGES * L::STAGE;
            bool ok = here(c);
            ok = ok && __all_sync(0xffffffffu, mbar_wait_or_abort(&given[(c & 1) * L::GROUPS + grp], (c >> 1) & 1, abort_flag));
            if (!ok) {
                failed = true;
                break;
            }
            const uint32_t buf = ((c & 1) * L::OUT + grp), xo = sbase + L::XO + buf * (DK / 16) * 512 + lane * 16;
            const uint32_t uo = sbase + L::UO + buf * 2048 + lane * 16;
            float O[4][4] = {};
#pragma unroll
            for (int x = 0; x < DK / 16; ++x) {
                uint32_t hi[4];
                ld_shared_4(hi, xo + 512 * x);
                read_step(st, x, hi, O);
            }
            uint32_t h0[4], l0[4], h1[4], l1[4], t0[4], t1[4], t2[4];
            load_p(st, t0, t1, t2);
            ld_shared_4(h0, uo);
            ld_shared_4(l0, uo + 512);
            ld_shared_4(h1, uo + 1024);
            ld_shared_4(l1, uo + 1536);
            finish_out(reinterpret_cast<const float*>(sm + c % STAGES * L::STAGE + L::VEC), t0, t1, t2, h0, l0, h1, l1, O);
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[(c & 1) * L::GROUPS + grp]);
            leave(c);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t y[2] = {pack_bf16(O[n][0], O[n][1]), pack_bf16(O[n][2], O[n][3])};
                store_out(op, n, c, y);
            }
        }
        if (failed && lane == 0) {
            *abort_flag = 1;
            atomicOr(a.status, kStatusTmaWait);
        }
    } else {
        // ======================= chain warp: rows r0 + g and r0 + g + 8, 8 NT channels ======
        const int gq = lane >> 2, cq = lane & 3;
        const int grp = warp % L::GROUPS, part = SPLIT > 1 ? warp / L::GROUPS : 0;
        const int r0 = it.split * L::ROWS + 16 * grp;
        float* sp = a.states + ((static_cast<size_t>(it.rq.slot) * a.Hv + it.head) * a.dv + r0 + gq) * DK + 8 * NT * part + 2 * cq;
        float X[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 u = make_float2(0.f, 0.f), w = u;
            if (!it.rq.fresh) {
                u = *reinterpret_cast<const float2*>(sp + 8 * n);
                w = *reinterpret_cast<const float2*>(sp + 8 * DK + 8 * n);
            }
            X[n][0] = u.x;
            X[n][1] = u.y;
            X[n][2] = w.x;
            X[n][3] = w.y;
        }
        const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, tc = lane >> 4;   // transposed, of K as [k = token][n = channel]
        __nv_bfloat16* op = out_rows(r0);
        uint32_t Y[4][2] = {};   // (SPLIT 1) outputs of the block before

        // SPLIT 2: Z is a sum over the channels of both warps of a row group, each of which hands its part over, in two
        // buffers taken in turn: what is written for block c + 2 comes after a turn of the barrier that follows the
        // other's reads for block c.
        auto zx = [&](int c, int of) {
            return sm + L::ZX + ((c & 1) * L::CHAIN + grp + L::GROUPS * of) * 2048 + lane * 16;
        };
        for (int c = 0; c < it.blocks; ++c) {
            const int s = c % STAGES;
            const uint32_t st = sbase + s * L::STAGE;
            bool ok = here(c);
            if (SPLIT > 1 && c >= 2) ok = ok && __all_sync(0xffffffffu, mbar_wait_or_abort(&taken[(c & 1) * L::GROUPS + grp], ((c >> 1) - 1) & 1, abort_flag));
            if (!ok) {
                failed = true;
                break;
            }
            const uint32_t buf = (c & 1) * L::OUT + grp, xo = sbase + L::XO + buf * (DK / 16) * 512 + lane * 16;
            // ---- Z = X K^T, both parts of X; the block before's outputs leave meanwhile ----
            float Z[4][4] = {}, O[4][4] = {};
#pragma unroll
            for (int x = 0; x < NT / 2; ++x) {
                uint32_t hi[4], lo[4], b0[4], b1[4];
                const int xk = NT / 2 * part + x;   // 16 channels
                const uint32_t at = st + L::K + (xk / 4) * 4096, ch = (xk % 4) * 2 + bc;
                ldsm4(b0, at + sw128_off(br, ch));
                ldsm4(b1, at + sw128_off(16 + br, ch));
                split_tiles(X[2 * x], X[2 * x + 1], hi, lo);
                mma_16816(Z[0], hi, b0[0], b0[1]);
                mma_16816(Z[1], hi, b0[2], b0[3]);
                mma_16816(Z[2], hi, b1[0], b1[1]);
                mma_16816(Z[3], hi, b1[2], b1[3]);
                if (SPLIT == 1 && x < 4) store_out(op, x, c - 1, Y[x]);
                if (SPLIT > 1) st_shared_4(xo + 512 * xk, hi);
                mma_16816(Z[0], lo, b0[0], b0[1]);
                mma_16816(Z[1], lo, b0[2], b0[3]);
                mma_16816(Z[2], lo, b1[0], b1[1]);
                mma_16816(Z[3], lo, b1[2], b1[3]);
            }
            // ---- (SPLIT 1) O = X Q^T, the high part, in two runs between the steps of U --------
            auto read_out = [&](int x0, int x1) {
#pragma unroll
                for (int x = x0; x < x1; ++x) {
                    const uint32_t hi[4] = {pack_bf16(X[2 * x][0], X[2 * x][1]), pack_bf16(X[2 * x][2], X[2 * x][3]),
                                            pack_bf16(X[2 * x + 1][0], X[2 * x + 1][1]), pack_bf16(X[2 * x + 1][2], X[2 * x + 1][3])};
                    read_step(st, x, hi, O);
                }
            };
            if constexpr (SPLIT > 1) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    *reinterpret_cast<float4*>(zx(c, part) + 512 * n) = make_float4(Z[n][0], Z[n][1], Z[n][2], Z[n][3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&swap[grp]);
                ok = mbar_wait_or_abort(&swap[grp], c & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    failed = true;
                    break;
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float4 z = *reinterpret_cast<const float4*>(zx(c, 1 - part) + 512 * n);
                    Z[n][0] += z.x;
                    Z[n][1] += z.y;
                    Z[n][2] += z.z;
                    Z[n][3] += z.w;
                }
            } else {
                read_out(0, NT / 4);
            }
            // ---- R = b (V - G Z), in Z --------------------------------------------------------
            const float* vec = reinterpret_cast<const float*>(sm + s * L::STAGE + L::VEC);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                uint32_t v4[4];   // (token 8n, row g) (.., row g + 8) (token 8n + 8, ..) (..)
                ldsm4t(v4, st + L::V + sw128_off(8 * n + (lane & 7) + (lane >> 4) * 8, r0 % 64 / 8 + ((lane >> 3) & 1)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = 8 * (n + i) + 2 * cq;
                    const float2 b = *reinterpret_cast<const float2*>(vec + t);
                    const float2 bg = *reinterpret_cast<const float2*>(vec + C + t);
                    const float2 vl = unpack_bf16(v4[2 * i]), vh = unpack_bf16(v4[2 * i + 1]);
                    float(&z)[4] = Z[n + i];
                    z[0] = b.x * vl.x - bg.x * z[0];
                    z[1] = b.y * vl.y - bg.y * z[1];
                    z[2] = b.x * vh.x - bg.x * z[2];
                    z[3] = b.y * vh.y - bg.y * z[3];
                }
            }
            // ---- U = R T^T: lower triangular, columns j < 16 reach every t, j >= 16 only t >= 16
            float U[4][4] = {};
            {
                uint32_t h0[4], l0[4], h1[4], l1[4], t0[4], t1[4], t2[4];
                const uint32_t th = st + L::TH + br * kTStride + bc * 16, tl = st + L::TL + br * kTStride + bc * 16;
                ldsm4(t0, th);                         // t 0..15, j 0..15
                ldsm4(t1, th + 16 * kTStride);         // t 16..31, j 0..15
                ldsm4(t2, th + 16 * kTStride + 32);    // t 16..31, j 16..31
                split_tiles(Z[0], Z[1], h0, l0);
                split_tiles(Z[2], Z[3], h1, l1);
                mma_16816(U[0], h0, t0[0], t0[1]);
                mma_16816(U[1], h0, t0[2], t0[3]);
                mma_16816(U[2], h0, t1[0], t1[1]);
                mma_16816(U[3], h0, t1[2], t1[3]);
                mma_16816(U[0], l0, t0[0], t0[1]);
                mma_16816(U[1], l0, t0[2], t0[3]);
                mma_16816(U[2], l0, t1[0], t1[1]);
                mma_16816(U[3], l0, t1[2], t1[3]);
                mma_16816(U[2], h1, t2[0], t2[1]);
                mma_16816(U[3], h1, t2[2], t2[3]);
                mma_16816(U[2], l1, t2[0], t2[1]);
                mma_16816(U[3], l1, t2[2], t2[3]);
                ldsm4(t0, tl);
                ldsm4(t1, tl + 16 * kTStride);
                ldsm4(t2, tl + 16 * kTStride + 32);
                mma_16816(U[0], h0, t0[0], t0[1]);
                mma_16816(U[1], h0, t0[2], t0[3]);
                mma_16816(U[2], h0, t1[0], t1[1]);
                mma_16816(U[3], h0, t1[2], t1[3]);
                mma_16816(U[2], h1, t2[0], t2[1]);
                mma_16816(U[3], h1, t2[2], t2[3]);
            }
            if constexpr (SPLIT == 1) read_out(NT / 4, NT / 2);
            // ---- O = G O + U P^T; X = G_31 X + (U D_31) K --------------------------------------
            uint32_t h0[4], l0[4], h1[4], l1[4];
            const float gc = vec[2 * C + C - 1];
            if constexpr (SPLIT > 1) {   // half of U by each warp
                if (part == 0) split_tiles(U[0], U[1], h0, l0);
                else split_tiles(U[2], U[3], h0, l0);
                const uint32_t uo = sbase + L::UO + buf * 2048 + part * 1024 + lane * 16;
                st_shared_4(uo, h0);
                st_shared_4(uo + 512, l0);
                __syncwarp();
                if (lane == 0) mbar_arrive(&given[(c & 1) * L::GROUPS + grp]);
            } else {
                uint32_t t0[4], t1[4], t2[4];
                load_p(st, t0, t1, t2);
                split_tiles(U[0], U[1], h0, l0);
                split_tiles(U[2], U[3], h1, l1);
                finish_out(vec, t0, t1, t2, h0, l0, h1, l1, O);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 dc = *reinterpret_cast<const float2*>(vec + 3 * C + 8 * n + 2 * cq);
                U[n][0] *= dc.x;
                U[n][1] *= dc.y;
                U[n][2] *= dc.x;
                U[n][3] *= dc.y;
            }
            split_tiles(U[0], U[1], h0, l0);
            split_tiles(U[2], U[3], h1, l1);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b0[4], b1[4];
                const int nk = NT * part + n;
                const uint32_t at = st + L::K + (nk / 8) * 4096, ch = nk % 8 + tc;
                ldsm4t(b0, at + sw128_off(tr, ch));
                ldsm4t(b1, at + sw128_off(16 + tr, ch));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    X[n][i] *= gc;
                    X[n + 1][i] *= gc;
                }
                mma_16816(X[n], h0, b0[0], b0[1]);
                mma_16816(X[n + 1], h0, b0[2], b0[3]);
                mma_16816(X[n], h1, b1[0], b1[1]);
                mma_16816(X[n + 1], h1, b1[2], b1[3]);
                mma_16816(X[n], l0, b0[0], b0[1]);
                mma_16816(X[n + 1], l0, b0[2], b0[3]);
                mma_16816(X[n], l1, b1[0], b1[1]);
                mma_16816(X[n + 1], l1, b1[2], b1[3]);
            }
            leave(c);
            if constexpr (SPLIT == 1) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    Y[n][0] = pack_bf16(O[n][0], O[n][1]);
                    Y[n][1] = pack_bf16(O[n][2], O[n][3]);
                }
            }
        }
        if (SPLIT == 1 && !failed) {
#pragma unroll
            for (int n = 0; n < 4; ++n) store_out(op, n, it.blocks - 1, Y[n]);
        }
        if (!failed) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(sp + 8 * n) = make_float2(X[n][0], X[n][1]);
                *reinterpret_cast<float2*>(sp + 8 * DK + 8 * n) = make_float2(X[n][2], X[n][3]);
            }
        } else if (lane == 0) {
            *abort_flag = 1;
            atomicOr(a.status, kStatusTmaWait);
        }
    }
    if (failed) {   // let the loads in flight land before the CTA leaves (bounded)
        if (lane == 0)
            for (int c = max(0, *issued - STAGES); c < *issued; ++c)
                mbar_wait(&full[c % L::FULL], (c / L::FULL) & 1, 100000000ull);
    }
}

template <class L, int RESIDENT>
cudaError_t run_shape(const StepArgs& a, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v) {
    constexpr uint32_t smem = L::BYTES + 1024;
    static_assert(RESIDENT * (smem + 1024) <= 228 * 1024 && smem <= 232448, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<L, RESIDENT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long grid = static_cast<long long>(a.requests) * a.Hv * (a.dv / L::ROWS);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(chunk_kernel<L, RESIDENT>, static_cast<unsigned>(grid), L::THREADS, smem, s, q, k, v, a);
}

template <int DK>
cudaError_t run(const StepArgs& a, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v) {
    // Rows of 32 while every CTA has an SM: one request of 2048 tokens, 16 heads, d 64 (d_k 128, d_v 64) 66 (82) us, with
    // 64 rows 92 (131). With 64 rows two CTAs share an SM and half of the prep, which counts where SMs are short.
    // Two prep warps are enough and disturb the chain less (three: 74 and 93 us), but with more CTAs than half of the
    // SMs three did better: 32 sequence-heads of 8192 tokens at d 128 363 us, by two prep warps 378.
    const long long rows32 = static_cast<long long>(a.requests) * a.Hv * (a.dv / 32);
    if (2 * rows32 <= a.sm_count) return run_shape<Layout<DK, 32, 2, 2, 4>, 1>(a, s, q, k, v);
    if (chunk_is_alone(a.requests, a.Hv, a.dv, a.sm_count)) return run_shape<Layout<DK, 32, 2, 3, 5>, 1>(a, s, q, k, v);
    return run_shape<Layout<DK, 64, 1, 2, 3>, 2>(a, s, q, k, v);
}

}  // namespace

cudaError_t launch_chunk(const StepArgs& a, cudaStream_t s, PFN_cuTensorMapEncodeTiled_v12000 enc) {
    CUtensorMap q, k, v;
    if (!make_map(enc, &q, a.q, a.dk, a.Hk, a.rows, a.q_stride, C) || !make_map(enc, &k, a.k, a.dk, a.Hk, a.rows, a.k_stride, C) ||
        !make_map(enc, &v, a.v, a.dv, a.Hv, a.rows, a.v_stride, C))
        return cudaErrorInvalidValue;
    if (a.dk == 64) return run<64>(a, s, q, k, v);
    if (a.dk == 128) return run<128>(a, s, q, k, v);
    return cudaErrorInvalidValue;
}

}  // namespace packed
}  // namespace la

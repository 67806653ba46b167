// The gated delta rule over packed requests in blocks of 32 tokens: bf16 q, k
// and v, fp32 states in a pool.
//
// Per value head (key head h * Hk / Hv), state X [dv][dk] at a block's start,
// tokens t, j of the block, g and b the gates:
//   D_tj = prod_{j < s <= t} g_s,  G_t = prod_{s <= t} g_s
//   A_tj = b_t D_tj k_t.k_j  (j < t),   T = (I + A)^-1,   P_tj = D_tj q_t.k_j  (j <= t)
//   R = diag(b) (V - diag(G) K X^T),   U = T R             [token][dv]
//   O = diag(G) Q X^T + P U,           X <- G_31 X + U^T diag(D_31,.) K
// The decays are running products, never quotients or logarithms: any gate,
// zero among them, gives what the recurrence gives.
//
// Work split. One CTA per (request, value head, 64 rows of the state), longest
// requests first: rows of the state are independent. Four chain warps own 16
// rows each, for the whole request. With X^T's products written as
// [dv][token], a warp's accumulators (X, Z = X K^T, R, U) turn into the next
// product's A operand inside its own registers, so from the state's load to
// its store the chain exchanges nothing between warps. K, Q, V tiles come by
// TMA into a ring of three stages; ahead of the chain one prep warp computes T
// of every block, another P, which also issues the loads.
//
// Precision. q, k, v are bf16 and enter the MMAs as they are. What the state
// depends on (X in K X^T, R and T in T R, U in U^T K) is split into two bf16
// parts, high and low, whose sum is off by at most 2^-16 of the value;
// products of two low parts (2^-16 again) are dropped. Measured: states off by
// 3.6e-6 of themselves against float64 (one part alone: about 2e-3). What only an output depends on, rounded to bf16 itself,
// keeps one part where the other factor is exact: X in Q X^T, P in P U.
// Accumulators, gates, A and the inverse are fp32.
//
// Rows past a request's end belong to the next request: K and V are zeroed there
// before the chain reads them, with gate 1 and beta 0, so that they leave the
// state alone; Q's reach only outputs that are not written.
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

constexpr int C = kBlock;
constexpr int kChain = 4;                  // chain warps: 16 state rows each
constexpr int kRows = 16 * kChain;         // state rows of a CTA
constexpr int kPrep = 2;                   // prep warps: T, and P with the loads
constexpr int kThreads = 32 * (kChain + kPrep);
constexpr int kStages = 3;
constexpr int kTStride = 80;               // bytes per row of a 32x32 bf16 tile: 16-byte chunks of 8 rows hit all banks
// a prep warp's fp32 scratch: two 16x16 sub-blocks of K K^T or Q K^T, rows and blocks so far apart that the MMA
// fragments' stores and the column reads of both halves of the warp hit all banks; then the gates
constexpr int kSStride = 24;
constexpr int kSBlock = 16 * kSStride + 16;
constexpr int kScratch = 2 * kSBlock + C;

template <int DK>
struct Layout {
    static constexpr int KA = DK / 64;                       // 64-channel atoms of [32][64] bf16, 4 KB, 128-byte swizzle
    static constexpr uint32_t K = 0;
    static constexpr uint32_t Q = K + KA * 4096;
    static constexpr uint32_t V = Q + KA * 4096;             // [32][64]: the CTA's own rows of the state
    static constexpr uint32_t TX = V + 4096;                 // bytes a stage's loads bring
    static constexpr uint32_t TH = TX;                       // T, high and low parts, [t][j]
    static constexpr uint32_t TL = TH + C * kTStride;
    static constexpr uint32_t P = TL + C * kTStride;
    static constexpr uint32_t VEC = P + C * kTStride;        // fp32: b, b G, G, D_31 [32 each]
    static constexpr uint32_t STAGE = (VEC + 4 * C * 4 + 1023) / 1024 * 1024;
    static constexpr uint32_t SCRATCH = kStages * STAGE;     // kScratch floats per prep warp
    static constexpr uint32_t BAR = SCRATCH + kPrep * kScratch * 4;
    static constexpr uint32_t BYTES = BAR + 128;
};

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0) : "memory");
}

struct Item {
    int head, khead, split;
    Request rq;
    int blocks;
};

// ---------------------------------------------------------------- prep warps

// Ring position of a block, stepped instead of divided.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == kStages) {
            s = 0;
            phase ^= 1;
        }
    }
};

// Loads of the request's next block into stage s (one thread); rows past the
// tensor read as zeros.
template <int DK>
__device__ __forceinline__ void issue_loads(const CUtensorMap* tmq, const CUtensorMap* tmk, const CUtensorMap* tmv,
                                            const Item& it, uint8_t* sm, uint64_t* full, int c, int s) {
    using L = Layout<DK>;
    const int row = it.rq.row0 + c * C;
    uint8_t* st = sm + s * L::STAGE;
    mbar_arrive_expect_tx(&full[s], L::TX);
#pragma unroll
    for (int x = 0; x < L::KA; ++x) {
        tma_load_3d(tmk, &full[s], st + L::K + x * 4096, x * 64, it.khead, row);
        tma_load_3d(tmq, &full[s], st + L::Q + x * 4096, x * 64, it.khead, row);
    }
    tma_load_3d(tmv, &full[s], st + L::V, it.split * kRows, it.head, row);
}

// The lower 16x16 tiles of M K^T, M = K or Q: tiles (m, n) of 16x8
// (0,0) (0,1) (1,0) (1,1) (1,2) (1,3). Fragments are loaded a step ahead; a
// key fragment serves as A and as B.
template <int DK, bool QK>
__device__ __forceinline__ void lower_products(uint32_t aM, uint32_t aK, int fr, int fc, float (&d)[6][4]) {
    uint32_t k0[2][4], k1[2][4], m0[2][4], m1[2][4];
    auto load = [&](int x) {
        const uint32_t at = (x / 4) * 4096, ch = (x % 4) * 2 + fc;
        const uint32_t lo = at + sw128_off(fr, ch), hi = at + sw128_off(16 + fr, ch);
        ldsm4(k0[x & 1], aK + lo);
        ldsm4(k1[x & 1], aK + hi);
        if (QK) {
            ldsm4(m0[x & 1], aM + lo);
            ldsm4(m1[x & 1], aM + hi);
        }
    };
    load(0);
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) {
        if (x + 1 < DK / 16) load(x + 1);
        const auto& u0 = k0[x & 1];
        const auto& u1 = k1[x & 1];
        const auto& w0 = QK ? m0[x & 1] : k0[x & 1];
        const auto& w1 = QK ? m1[x & 1] : k1[x & 1];
        mma_16816(d[0], w0, u0[0], u0[2]);
        mma_16816(d[1], w0, u0[1], u0[3]);
        mma_16816(d[2], w1, u0[0], u0[2]);
        mma_16816(d[3], w1, u0[1], u0[3]);
        mma_16816(d[4], w1, u1[0], u1[2]);
        mma_16816(d[5], w1, u1[1], u1[3]);
    }
}

// One prep warp: T (two bf16 parts) and the gate vectors of every block, or
// (QK) P of every block, as the loads' issuer besides.
//
// By 16x16 sub-blocks: on the diagonal lane l takes one column of sub-block
// l / 16, D_tj being its running product, and inverts by forward substitution
// in fp32; the sub-block below is T21 = -T22 (A21 T11) on the tensor cores,
// operands in two bf16 parts, with D_tj = (g_16 .. g_t)(g_{j+1} .. g_15).
template <int DK, bool QK>
__device__ __forceinline__ void prep_warp(const CUtensorMap* tmq, const CUtensorMap* tmk, const CUtensorMap* tmv,
                                          const StepArgs& a, const Item& it, uint8_t* sm, uint32_t sbase,
                                          uint64_t* full, uint64_t* ready, uint64_t* empty, volatile int* abort_flag) {
    using L = Layout<DK>;
    const int lane = threadIdx.x & 31, gq = lane >> 2, cq = lane & 3;
    const int blk = lane >> 4, col = lane & 15;
    float* raw = reinterpret_cast<float*>(sm + L::SCRATCH) + (QK ? kScratch : 0);   // diagonal sub-blocks, then A
    float* gs = raw + 2 * kSBlock;                                                  // gates [32]
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
            if (!QK) b = __ldg(a.beta + i);
        }
    };
    if (QK && lane == 0)
        for (int c = 0; c < kStages && c < it.blocks; ++c) issue_loads<DK>(tmq, tmk, tmv, it, sm, full, c, c);
    float gn, bn;
    gates(0, gn, bn);
    Ring at;   // block c
    Ring old;  // block c - kStages + 1, whose stage block c + 1 takes
    for (int c = 0; c < it.blocks; ++c, at.next()) {
        const int s = at.s;
        const uint32_t st = sbase + s * L::STAGE;
        float* vec = reinterpret_cast<float*>(sm + s * L::STAGE + L::VEC);
        const float g = gn, b = bn;
        gates(c + 1, gn, bn);
        float Gh = g;   // product of the gates from the half's start up to this token
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, Gh, o);
            if (col >= o) Gh *= y;
        }
        const float G15 = __shfl_sync(0xffffffffu, Gh, 15), G31 = __shfl_sync(0xffffffffu, Gh, 31);
        gs[lane] = g;
        const bool ok = mbar_wait_or_abort(&full[s], at.phase, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return;
        const int n = it.rq.len - c * C;   // tokens of the block
        if (!QK && n < C) {                // rows of the next request (or past the tensor): zero
            for (int i = lane; i < (C - n) * 8; i += 32) {
                const uint32_t o = sw128_off(n + i / 8, i % 8);
#pragma unroll
                for (int x = 0; x < L::KA; ++x) st_shared_zero16(st + L::K + x * 4096 + o);
                st_shared_zero16(st + L::V + o);
            }
        }
        if (!QK) {
            const float G = blk ? Gh * G15 : Gh;
            vec[lane] = b;
            vec[C + lane] = b * G;
            vec[2 * C + lane] = G;
        }
        __syncwarp();
        float d[6][4] = {};
        lower_products<DK, QK>(st + (QK ? L::Q : L::K), st + L::K, fr, fc, d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* r0 = raw + h * kSBlock + gq * kSStride + 8 * i + 2 * cq;
                const float(&x)[4] = d[4 * h + i];
                *reinterpret_cast<float2*>(r0) = make_float2(x[0], x[1]);
                *reinterpret_cast<float2*>(r0 + 8 * kSStride) = make_float2(x[2], x[3]);
            }
        __syncwarp();
        float* rb = raw + blk * kSBlock;
        float m[16], gt[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) m[t] = rb[t * kSStride + col];
#pragma unroll
        for (int t = 0; t < 16; t += 4)
            *reinterpret_cast<float4*>(&gt[t]) = *reinterpret_cast<const float4*>(gs + 16 * blk + t);
        float D = 0.f;   // zero above the diagonal; at the end the gates behind this column in its half
        const float Q0 = __shfl_sync(0xffffffffu, Gh, 16 + gq), Q1 = __shfl_sync(0xffffffffu, Gh, 24 + gq);
        if constexpr (QK) {
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                D = t == col ? 1.f : D * gt[t];
                st_shared_u16(st + L::P + (16 * blk + t) * kTStride + 2 * lane, __float2bfloat16_rn(t >= col ? D * m[t] : 0.f));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // the sub-block below the diagonal
                const float S0 = __shfl_sync(0xffffffffu, D, 8 * i + 2 * cq), S1 = __shfl_sync(0xffffffffu, D, 8 * i + 2 * cq + 1);
                const float(&y)[4] = d[2 + i];
                st_shared_b32(st + L::P + (16 + gq) * kTStride + 16 * i + 4 * cq, pack_bf16(Q0 * S0 * y[0], Q0 * S1 * y[1]));
                st_shared_b32(st + L::P + (24 + gq) * kTStride + 16 * i + 4 * cq, pack_bf16(Q1 * S0 * y[2], Q1 * S1 * y[3]));
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ready[s]);
                // the block after next but one goes where block c - kStages + 1 was, once the chain has left it
                if (c + 1 >= kStages && c + 1 < it.blocks) {
                    if (mbar_wait_or_abort(&empty[old.s], old.phase, abort_flag))
                        issue_loads<DK>(tmq, tmk, tmv, it, sm, full, c + 1, old.s);
                }
            }
            if (c + 1 >= kStages) old.next();
            __syncwarp();
        } else {
            float bt[16];
#pragma unroll
            for (int t = 0; t < 16; t += 4)
                *reinterpret_cast<float4*>(&bt[t]) = *reinterpret_cast<const float4*>(vec + 16 * blk + t);
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                D = t == col ? 1.f : D * gt[t];
                rb[t * kSStride + col] = t > col ? bt[t] * D * m[t] : 0.f;
            }
            vec[3 * C + lane] = blk ? D : D * G31;
            __syncwarp();
            // forward substitution: x = column `col` of the sub-block's inverse
            float x[16];
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                float s0 = t == col ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int i = 0; i < t; i += 4) {
                    const float4 r = *reinterpret_cast<const float4*>(rb + t * kSStride + i);
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
            // the sub-block below: A21 from its product tiles
            const float b0 = Q0 * __shfl_sync(0xffffffffu, b, 16 + gq), b1 = Q1 * __shfl_sync(0xffffffffu, b, 24 + gq);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float S0 = __shfl_sync(0xffffffffu, D, 8 * i + 2 * cq), S1 = __shfl_sync(0xffffffffu, D, 8 * i + 2 * cq + 1);
                float(&z)[4] = d[2 + i];
                z[0] *= b0 * S0;
                z[1] *= b0 * S1;
                z[2] *= b1 * S0;
                z[3] *= b1 * S1;
            }
            uint32_t ah[4], al[4];
            split_tiles(d[2], d[3], ah, al);
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
}

// ---------------------------------------------------------------- the kernel

template <int DK>
__global__ void __launch_bounds__(kThreads, 2)
chunk_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
             const __grid_constant__ CUtensorMap tmv, const StepArgs a) {
    using L = Layout<DK>;
    constexpr int NT = DK / 8;   // n-tiles of a warp's state rows
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR);   // [kStages] TMA: a block's tiles have arrived
    uint64_t* ready = full + kStages;                            // [kStages] prep warps: T, P and vectors are written
    uint64_t* empty = ready + kStages;                           // [kStages] chain warps: the stage is read
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kStages);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&ready[i], kPrep);
            mbar_init(&empty[i], kChain);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    griddep_wait();
    Item it;
    {
        const int splits = a.dv / kRows;
        const int per_req = a.Hv * splits;
        const int rank = blockIdx.x / per_req, hs = blockIdx.x % per_req;
        if (!read_request(a, rank, it.rq)) return;
        it.head = hs / splits;
        it.split = hs % splits;
        it.khead = it.head / (a.Hv / a.Hk);
        it.blocks = (it.rq.len + C - 1) / C;
    }
    __syncthreads();

    bool failed = false;
    if (warp == kChain) {
        prep_warp<DK, false>(&tmq, &tmk, &tmv, a, it, sm, sbase, full, ready, empty, abort_flag);
    } else if (warp > kChain) {
        prep_warp<DK, true>(&tmq, &tmk, &tmv, a, it, sm, sbase, full, ready, empty, abort_flag);
    } else {
        // ======================= chain warp: rows r0 + g and r0 + g + 8 ====================
        const int gq = lane >> 2, cq = lane & 3;
        const int r0 = it.split * kRows + 16 * warp;
        float* sp = a.states + ((static_cast<size_t>(it.rq.slot) * a.Hv + it.head) * a.dv + r0 + gq) * DK + 2 * cq;
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
        // ldmatrix lane addresses: B fragments of two n-tiles (rows = n, 16-byte
        // chunks along k) and, transposed, of K as [k = token][n = channel]
        const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;
        const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, tc = lane >> 4;
        __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) +
                            (static_cast<size_t>(it.rq.row0) * a.Hv + it.head) * a.dv + r0 + 2 * cq;
        const size_t ostep = static_cast<size_t>(a.Hv) * a.dv;
        // outputs of the block before, rounded: [dv][token] fragments, turned
        // to [token][dv] pairs when they leave
        uint32_t Y[4][2] = {};
        auto store_out = [&](int n, int c) {   // tokens 8n .. 8n + 7 of block c
            const uint32_t y0 = transpose8x8(Y[n][0]);   // token 8n + g, rows 2c, 2c + 1
            const uint32_t y1 = transpose8x8(Y[n][1]);   // rows 8 + 2c, ..
            const int t = c * C + 8 * n + gq;
            if (c >= 0 && t < it.rq.len) {
                __nv_bfloat16* o = op + static_cast<size_t>(t) * ostep;
                *reinterpret_cast<uint32_t*>(o) = y0;
                *reinterpret_cast<uint32_t*>(o + 8) = y1;
            }
        };

        Ring at;
        for (int c = 0; c < it.blocks; ++c, at.next()) {
            const int s = at.s;
            const uint32_t st = sbase + s * L::STAGE;
            const bool ok = mbar_wait_or_abort(&full[s], at.phase, abort_flag) && mbar_wait_or_abort(&ready[s], at.phase, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                failed = true;
                break;
            }
            // ---- Z = X K^T, both parts of X; the block before's outputs leave meanwhile ----
            float Z[4][4] = {}, O[4][4] = {};
#pragma unroll
            for (int x = 0; x < DK / 16; ++x) {
                uint32_t hi[4], lo[4], b0[4], b1[4];
                const uint32_t at = st + L::K + (x / 4) * 4096, ch = (x % 4) * 2 + bc;
                ldsm4(b0, at + sw128_off(br, ch));
                ldsm4(b1, at + sw128_off(16 + br, ch));
                split_tiles(X[2 * x], X[2 * x + 1], hi, lo);
                mma_16816(Z[0], hi, b0[0], b0[1]);
                mma_16816(Z[1], hi, b0[2], b0[3]);
                mma_16816(Z[2], hi, b1[0], b1[1]);
                mma_16816(Z[3], hi, b1[2], b1[3]);
                if (x < 4) store_out(x, c - 1);
                mma_16816(Z[0], lo, b0[0], b0[1]);
                mma_16816(Z[1], lo, b0[2], b0[3]);
                mma_16816(Z[2], lo, b1[0], b1[1]);
                mma_16816(Z[3], lo, b1[2], b1[3]);
            }
            // ---- O = X Q^T, the high part, in two runs between the steps of U --------------
            auto read_out = [&](int x0, int x1) {
#pragma unroll
                for (int x = x0; x < x1; ++x) {
                    uint32_t hi[4], b0[4], b1[4];
                    const uint32_t at = st + L::Q + (x / 4) * 4096, ch = (x % 4) * 2 + bc;
                    ldsm4(b0, at + sw128_off(br, ch));
                    ldsm4(b1, at + sw128_off(16 + br, ch));
                    hi[0] = pack_bf16(X[2 * x][0], X[2 * x][1]);
                    hi[1] = pack_bf16(X[2 * x][2], X[2 * x][3]);
                    hi[2] = pack_bf16(X[2 * x + 1][0], X[2 * x + 1][1]);
                    hi[3] = pack_bf16(X[2 * x + 1][2], X[2 * x + 1][3]);
                    mma_16816(O[0], hi, b0[0], b0[1]);
                    mma_16816(O[1], hi, b0[2], b0[3]);
                    mma_16816(O[2], hi, b1[0], b1[1]);
                    mma_16816(O[3], hi, b1[2], b1[3]);
                }
            };
            read_out(0, DK / 32);
            // ---- R = b (V - G Z), in Z --------------------------------------------------------
            const float* vec = reinterpret_cast<const float*>(sm + s * L::STAGE + L::VEC);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                uint32_t v4[4];   // (token 8n, row g) (.., row g + 8) (token 8n + 8, ..) (..)
                ldsm4t(v4, st + L::V + sw128_off(8 * n + (lane & 7) + (lane >> 4) * 8, 2 * warp + ((lane >> 3) & 1)));
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
            read_out(DK / 32, DK / 16);
            // ---- O = G O + U P^T; X = G_31 X + (U D_31) K --------------------------------------
            uint32_t h0[4], l0[4], h1[4], l1[4];
            const float gc = vec[2 * C + C - 1];
            {
                uint32_t t0[4], t1[4], t2[4];
                const uint32_t tp = st + L::P + br * kTStride + bc * 16;
                ldsm4(t0, tp);
                ldsm4(t1, tp + 16 * kTStride);
                ldsm4(t2, tp + 16 * kTStride + 32);
                split_tiles(U[0], U[1], h0, l0);
                split_tiles(U[2], U[3], h1, l1);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 g = *reinterpret_cast<const float2*>(vec + 2 * C + 8 * n + 2 * cq);
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
                const uint32_t at = st + L::K + (n / 8) * 4096, ch = n % 8 + tc;
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);   // this warp has read the stage
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                Y[n][0] = pack_bf16(O[n][0], O[n][1]);
                Y[n][1] = pack_bf16(O[n][2], O[n][3]);
            }
        }
        if (!failed) {
#pragma unroll
            for (int n = 0; n < 4; ++n) store_out(n, it.blocks - 1);
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
    // After a failure loads may be in flight: let them land before the CTA
    // leaves (bounded: a phase that was never begun runs into the limit).
    if (__syncthreads_or(failed) && tid == 0)
        for (int i = 0; i < kStages; ++i) {
            mbar_wait(&full[i], 0, 20000000ull);
            mbar_wait(&full[i], 1, 20000000ull);
        }
}

template <int DK>
cudaError_t run(const StepArgs& a, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v) {
    constexpr uint32_t smem = Layout<DK>::BYTES + 1024;
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
    const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long grid = static_cast<long long>(a.requests) * a.Hv * (a.dv / kRows);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(chunk_kernel<DK>, static_cast<unsigned>(grid), kThreads, smem, s, q, k, v, a);
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

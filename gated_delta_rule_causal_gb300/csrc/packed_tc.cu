// The gated delta rule over packed requests on the tcgen05 tensor cores: bf16
// q, k and v, value heads of 128, blocks of 64 tokens. The algebra and the
// precision are those of packed_chunk.cu (value heads of 64, warp-level MMAs):
//   R = diag(b) (V - diag(G) K X^T),   U = T R,   T = (I + A)^-1
//   O = diag(G) Q X^T + P U,           X <- G_63 X + U^T diag(D_63,.) K
// with q, k, v exact, X, R, T and U in two bf16 parts wherever the state
// depends on them, X in Q X^T and P in one.
//
// Work split. One CTA per (request, value head), the state's 128 rows on the
// 128 tensor-memory lanes, so that every product of the chain is an M = 128
// MMA with its A operand (X, R, U: bf16 parts) in tensor memory and its B
// operand (K, Q, T, P) in shared memory:
//   Z = X K^T, O = X Q^T  [dv][token],  U = R T^T,  dX = U' K,  O += U P^T
// Eight warps convert between them: thread (row r, half hh) holds half of row
// r of X in fp32 registers and takes half the columns of each product. Four
// prep warps compute T and P of the next block meanwhile; of the others one
// issues the chain's MMAs, one the loads, and one copies the outputs out.
//
// The chain's steps depend on one another, so what bounds a long request is
// their latency: four products (Z 512 clocks at the rate of the tensor cores,
// U 384, dX 512) with a conversion after each. Outputs are kept off that path:
// Q X^T runs while R is formed, is scaled by G while U is computed, and the
// block's outputs are read while the next block's Z runs.
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
constexpr int kThreads = 32 * (kConvWarps + kPrepWarps + 3);   // + MMA issue, loads, output copies
constexpr int kPrepThreads = 32 * kPrepWarps;
constexpr uint32_t kBarPrep = 1;      // named barrier of the prep warps
constexpr int kTiles = 3;             // ring of K, Q and V tiles
constexpr int kAStride = 68;          // floats per row of A
constexpr int kMStride = 80;          // bytes per row of the 32x32 bf16 product between the two merges
constexpr int kVec = 5 * C;           // floats of a block's gate vectors: g, b, b G, G, D_63

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
    static constexpr uint32_t BYTES = BAR + 40 * 8;
    // Tensor memory columns. X: per half hh of the channels DK/4 columns of
    // high parts, then DK/4 of low ones; dX (fp32, DK columns) takes the same
    // columns once Z and Q X^T are done, each half over its own.
    static constexpr uint32_t COL_X = 0;
    static constexpr uint32_t COL_Z = 128;     // Z, then U
    static constexpr uint32_t COL_R = 192;     // R high, low (32 columns each); then U high, low
    static constexpr uint32_t COL_UD = 256;    // U' high, low
    static constexpr uint32_t COL_O = 320;     // two buffers of 64
    static constexpr uint32_t COL_G = 448;     // [K;Q] K^T
    static constexpr uint32_t TMEM_COLS = 512;
};

struct Work {
    Request rq;
    int head, khead, blocks;
};

// Barriers, in shared memory.
struct Bars {
    uint64_t kq_full[kTiles], kq_free[kTiles];   // TMA; MMA: every product of the block is done
    uint64_t v_full[kTiles], v_free[kTiles];     // TMA; copier: the output tile over V has left
    uint64_t vec_free[kTiles];                   // converters: the block's vectors are read (8)
    uint64_t ot_full[kTiles];                    // converters: the output tile is written (8)
    uint64_t ready[2], tp_free[2];               // prep warps: T, P and vectors (4); MMA: T and P are read
    uint64_t g;                                  // MMA: [K;Q] K^T
    uint64_t x, r, up, uo;                       // converters: X, R, U', (U and O scaled) published (8 each)
    uint64_t z, o1, u, dx, o;                    // MMA: Z, Q X^T, U, dX, O done
    uint64_t drain[2];                           // after a failure: MMAs of either issuer are done
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Bars) <= 40 * 8, "barrier space");

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

// ---------------------------------------------------------------- prep warps
// Four warps, block by block: [K;Q] K^T on the tensor cores, A and P row by
// row (lane = tensor-memory lane = row; D_tj is a running product from the
// diagonal leftwards), then T: 16x16 diagonal blocks by forward substitution
// in fp32 (warps 0 and 1, a half-warp each), merged twice by
// T21 = -T22 (A21 T11) on warp-level MMAs with two bf16 parts. Warp 3 computes
// the next block's gate vectors while warps 0 and 1 solve.
template <int DK>
__device__ __forceinline__ bool prep_warps(const StepArgs& a, const Work& w, uint8_t* sm, uint32_t sbase, Bars* B,
                                           uint32_t tmem) {
    using L = TcLayout<DK>;
    const int lane = threadIdx.x & 31, pw = (threadIdx.x >> 5) - kConvWarps, ptid = threadIdx.x - 32 * kConvWarps;
    const int gq = lane >> 2, cq = lane & 3;
    const int fr = (lane & 7) + ((lane >> 3) & 1) * 8, fc = lane >> 4;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * pw) << 16);
    volatile int* abort = &B->abort;
    float* As = reinterpret_cast<float*>(sm + L::A);
    const uint32_t aM = sbase + L::M;
    constexpr uint32_t ID_G = idesc_bf16(128, 64, false, false);

    // gate vectors of block c from tokens 2 lane, 2 lane + 1 (past the end: gate 1, beta 0)
    float2 gn = make_float2(1.f, 1.f), bn = make_float2(0.f, 0.f);
    auto load_gates = [&](int c) {
        const int t = c * C + 2 * lane;
        const size_t i = static_cast<size_t>(w.rq.row0 + t) * a.Hv + w.head;
        gn = make_float2(1.f, 1.f);
        bn = make_float2(0.f, 0.f);
        if (t < w.rq.len) {
            gn.x = __ldg(a.gate + i);
            bn.x = __ldg(a.beta + i);
        }
        if (t + 1 < w.rq.len) {
            gn.y = __ldg(a.gate + i + a.Hv);
            bn.y = __ldg(a.beta + i + a.Hv);
        }
    };
    auto write_gates = [&](int s) {
        float* vec = reinterpret_cast<float*>(sm + L::VEC) + s * kVec;
        float pre = gn.x * gn.y, suf = pre;   // products up to / from this lane's pair
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, pre, o), z = __shfl_down_sync(0xffffffffu, suf, o);
            if (lane >= o) pre *= y;
            if (lane + o < 32) suf *= z;
        }
        float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
        if (lane == 0) before = 1.f;
        if (lane == 31) after = 1.f;
        const float G0 = before * gn.x;
        reinterpret_cast<float2*>(vec)[lane] = gn;
        reinterpret_cast<float2*>(vec + C)[lane] = bn;
        reinterpret_cast<float2*>(vec + 2 * C)[lane] = make_float2(bn.x * G0, bn.y * pre);
        reinterpret_cast<float2*>(vec + 3 * C)[lane] = make_float2(G0, pre);
        reinterpret_cast<float2*>(vec + 4 * C)[lane] = make_float2(gn.y * after, after);
    };
    if (pw == 3) {
        load_gates(0);
        write_gates(0);
    }
    // T's sub-blocks above the diagonal stay zero: the MMAs read whole tiles
    for (int i = ptid; i < 2 * 2 * 8192 / 16; i += kPrepThreads) {
        const int b = i / 1024, o = i % 1024;   // buffer, 16-byte chunk of T high and low
        st_shared_v4(sbase + L::TP + b * L::TP_BYTES + o * 16, 0, 0, 0, 0);
    }
    named_sync(kBarPrep, kPrepThreads);

    Ring3 at;
    for (int c = 0; c < w.blocks; ++c, at.next()) {
        const uint32_t kq = sbase + L::KQ + at.s * L::KQ_BYTES;
        const uint32_t tp = sbase + L::TP + (c & 1) * L::TP_BYTES;
        const uint32_t aTH = tp, aTL = tp + 8192, aP = tp + 16384;
        const float* vec = reinterpret_cast<const float*>(sm + L::VEC) + at.s * kVec;
        if (pw == 3 && c + 1 < w.blocks) load_gates(c + 1);
        bool ok = mbar_wait_or_abort(&B->kq_full[at.s], at.phase, abort);
        const int n = w.rq.len - c * C;
        if (n < C) {   // rows of the next request (or past the tensor): K and V zero, so that they leave the state alone
            ok = ok && mbar_wait_or_abort(&B->v_full[at.s], at.phase, abort);
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
        }
        // the products of the block before are read, this one's tiles are whole
        tc_fence_before();
        if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        tc_fence_after();
        if (ptid == 0) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint64_t d = kmaj(kq + (kk / 4) * 16384 + (kk % 4) * 32);
                mma_bf16_ss(tmem + L::COL_G, d, d, ID_G, kk > 0);
            }
            mma_commit(&B->g);
        }
        ok = mbar_wait_or_abort(&B->g, c & 1, abort);
        if (ok && c >= 2) ok = mbar_wait_or_abort(&B->tp_free[c & 1], ((c - 2) >> 1) & 1, abort);
        tc_fence_after();
        if (!__all_sync(0xffffffffu, ok)) ok = false;
        // ---- A (warps 0, 1) and P (warps 2, 3): row t, columns from the right ----------
        const int t = 32 * (pw & 1) + lane;
        if (ok) {
            const float bt = vec[C + t];
            float d = 0.f;
#pragma unroll
            for (int h = 1; h >= 0; --h) {
                float x[32];
                tmem_ld32(tlane + L::COL_G + 32 * h, x);
                tmem_ld_wait();
                float carry = 0.f;   // gate of the column to the right
                if (h == 0) carry = vec[32];
#pragma unroll
                for (int q4 = 7; q4 >= 0; --q4) {
                    const float4 g4 = *reinterpret_cast<const float4*>(vec + 32 * h + 4 * q4);
                    const float gr[4] = {g4.y, g4.z, g4.w, carry};
                    carry = g4.x;
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const int j = 32 * h + 4 * q4 + i;
                        d = j == t ? 1.f : d * gr[i];
                        const bool in = pw < 2 ? j < t : j <= t;
                        x[4 * q4 + i] = in ? (pw < 2 ? bt * d : d) * x[4 * q4 + i] : 0.f;
                    }
                }
                if (pw < 2) {
#pragma unroll
                    for (int q4 = 0; q4 < 8; ++q4)
                        *reinterpret_cast<float4*>(As + t * kAStride + 32 * h + 4 * q4) =
                            make_float4(x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]);
                } else {
                    chunk::store_row32_bf16(aP, t, 4 * h, x);
                }
            }
        }
        if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        if (pw < 2) {
            // ---- diagonal blocks 2 pw and 2 pw + 1, lane = (block, column) -----------------
            const int blk = 2 * pw + (lane >> 4), col = lane & 15;
            const float* ab = As + 16 * blk * kAStride + 16 * blk;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == col ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 r = *reinterpret_cast<const float4*>(ab + i * kAStride + j);
                    s0 -= r.x * x[j];
                    if (j + 1 < i) s1 -= r.y * x[j + 1];
                    if (j + 2 < i) s2 -= r.z * x[j + 2];
                    if (j + 3 < i) s3 -= r.w * x[j + 3];
                }
                x[i] = (s0 + s1) + (s2 + s3);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t o = sw128_off(16 * blk + i, 2 * blk + (col >> 3)) + 2 * (col & 7);
                const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                st_shared_u16(aTH + o, hi);
                st_shared_u16(aTL + o, __float2bfloat16_rn(x[i] - __bfloat162float(hi)));
            }
            __syncwarp();
            // ---- the 16x16 block below: -T22 (A21 T11) -------------------------------------
            const int rb = 32 * pw + 16, cb = 32 * pw;   // its first row and column
            uint32_t ah[4], al[4], th[4], tl[4];
            {
                const float* p = As + (rb + gq) * kAStride + cb + 2 * cq;
                const float2 y0 = *reinterpret_cast<const float2*>(p), y1 = *reinterpret_cast<const float2*>(p + 8 * kAStride);
                const float2 y2 = *reinterpret_cast<const float2*>(p + 8), y3 = *reinterpret_cast<const float2*>(p + 8 * kAStride + 8);
                split2(y0.x, y0.y, ah[0], al[0]);
                split2(y1.x, y1.y, ah[1], al[1]);
                split2(y2.x, y2.y, ah[2], al[2]);
                split2(y3.x, y3.y, ah[3], al[3]);
            }
            float Mx[2][4] = {}, N[2][4] = {};
            ldsm4t(th, aTH + sw128_off(cb + fr, cb / 8 + fc));
            ldsm4t(tl, aTL + sw128_off(cb + fr, cb / 8 + fc));
            mma_16816(Mx[0], ah, th[0], th[1]);
            mma_16816(Mx[1], ah, th[2], th[3]);
            mma_16816(Mx[0], al, th[0], th[1]);
            mma_16816(Mx[1], al, th[2], th[3]);
            mma_16816(Mx[0], ah, tl[0], tl[1]);
            mma_16816(Mx[1], ah, tl[2], tl[3]);
            uint32_t mh[4], ml[4];
            split_tiles(Mx[0], Mx[1], mh, ml);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mh[i] = transpose8x8(mh[i]);
                ml[i] = transpose8x8(ml[i]);
            }
            ldsm4(th, aTH + sw128_off(rb + fr, rb / 8 + fc));
            ldsm4(tl, aTL + sw128_off(rb + fr, rb / 8 + fc));
            mma_16816(N[0], th, mh[0], mh[1]);
            mma_16816(N[1], th, mh[2], mh[3]);
            mma_16816(N[0], tl, mh[0], mh[1]);
            mma_16816(N[1], tl, mh[2], mh[3]);
            mma_16816(N[0], th, ml[0], ml[1]);
            mma_16816(N[1], th, ml[2], ml[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi, lo;
                    split2(-N[i][2 * h], -N[i][2 * h + 1], hi, lo);
                    const uint32_t o = sw128_off(rb + 8 * h + gq, cb / 8 + i) + 4 * cq;
                    st_shared_b32(aTH + o, hi);
                    st_shared_b32(aTL + o, lo);
                }
        } else if (pw == 3 && c + 1 < w.blocks) {
            Ring3 nx = at;
            nx.next();
            // the slot's vectors of block c - 2 are read (its phase is the one before block c + 1's)
            if (c + 1 < kTiles || __all_sync(0xffffffffu, mbar_wait_or_abort(&B->vec_free[nx.s], nx.phase ^ 1, abort)))
                write_gates(nx.s);
            else
                ok = false;
        }
        if (named_sync_or(kBarPrep, kPrepThreads, !ok)) return false;
        // ---- rows 32..63, columns 0..31: -T_B (A_BA T_A), a 16x16 tile per warp -----------
        {
            const int mi = pw >> 1, ni = pw & 1;
            float Mx[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t ah[4], al[4], th[4], tl[4];
                const float* p = As + (32 + 16 * mi + gq) * kAStride + 16 * kk + 2 * cq;
                const float2 y0 = *reinterpret_cast<const float2*>(p), y1 = *reinterpret_cast<const float2*>(p + 8 * kAStride);
                const float2 y2 = *reinterpret_cast<const float2*>(p + 8), y3 = *reinterpret_cast<const float2*>(p + 8 * kAStride + 8);
                split2(y0.x, y0.y, ah[0], al[0]);
                split2(y1.x, y1.y, ah[1], al[1]);
                split2(y2.x, y2.y, ah[2], al[2]);
                split2(y3.x, y3.y, ah[3], al[3]);
                ldsm4t(th, aTH + sw128_off(16 * kk + fr, 2 * ni + fc));
                ldsm4t(tl, aTL + sw128_off(16 * kk + fr, 2 * ni + fc));
                mma_16816(Mx[0], ah, th[0], th[1]);
                mma_16816(Mx[1], ah, th[2], th[3]);
                mma_16816(Mx[0], al, th[0], th[1]);
                mma_16816(Mx[1], al, th[2], th[3]);
                mma_16816(Mx[0], ah, tl[0], tl[1]);
                mma_16816(Mx[1], ah, tl[2], tl[3]);
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
            float N[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t th[4], tl[4], mh[4], ml[4];
                ldsm4(th, aTH + sw128_off(32 + 16 * mi + fr, 4 + 2 * kk + fc));
                ldsm4(tl, aTL + sw128_off(32 + 16 * mi + fr, 4 + 2 * kk + fc));
                ldsm4t(mh, aM + (16 * kk + fr) * kMStride + (2 * ni + fc) * 16);
                ldsm4t(ml, aM + 32 * kMStride + (16 * kk + fr) * kMStride + (2 * ni + fc) * 16);
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
                    const uint32_t o = sw128_off(32 + 16 * mi + 8 * h + gq, 2 * ni + i) + 4 * cq;
                    st_shared_b32(aTH + o, hi);
                    st_shared_b32(aTL + o, lo);
                }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->ready[c & 1]);
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
        for (uint64_t* b : {&B->x, &B->r, &B->up, &B->uo}) mbar_init(b, kConvWarps);
        for (uint64_t* b : {&B->g, &B->z, &B->o1, &B->u, &B->dx, &B->o}) mbar_init(b, 1);
        B->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    griddep_wait();
    Work w;
    if (!read_request(a, blockIdx.x / a.Hv, w.rq)) return;
    w.head = blockIdx.x % a.Hv;
    w.khead = w.head / (a.Hv / a.Hk);
    w.blocks = (w.rq.len + C - 1) / C;
    if (warp == 0) tmem_alloc(&B->tmem, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B->tmem;

    int status = 0;
    bool fail = false;
    auto wait = [&](uint64_t* b, uint32_t parity) { fail = fail || !mbar_wait_or_abort(b, parity, abort); };
    if (warp < kConvWarps) {
        // ======================= converting warps ==================================
        const int r = 32 * (warp & 3) + lane, hh = warp >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t colx = tl + L::COL_X + hh * XH;
        float* sp = a.states + ((static_cast<size_t>(w.rq.slot) * a.Hv + w.head) * DV + r) * DK + hh * XH;
        float X[XH];
#pragma unroll
        for (int i = 0; i < XH; i += 4) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!w.rq.fresh) y = *reinterpret_cast<const float4*>(sp + i);
            X[i] = y.x;
            X[i + 1] = y.y;
            X[i + 2] = y.z;
            X[i + 3] = y.w;
        }
        auto signal = [&](uint64_t* b) {   // this warp's tensor-memory stores (and loads) are done
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        auto store_split = [&](uint32_t hi_col, uint32_t lo_col, const float* x) {   // 32 values: 16 columns each
            uint32_t h[16], l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
            tmem_st16(hi_col, h);
            tmem_st16(lo_col, l);
        };
        auto publish_x = [&]() {
#pragma unroll
            for (int p = 0; p < XH / 32; ++p) store_split(colx + 16 * p, colx + XH / 2 + 16 * p, X + 32 * p);
            signal(&B->x);
        };
        // warp-uniform before the warp-collective tensor-memory accesses
        auto wait_all = [&](uint64_t* b, uint32_t parity) {
            const bool ok = !fail && mbar_wait_or_abort(b, parity, abort);
            fail = !__all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        publish_x();
        Ring3 at, last;
        // outputs of block c: O through the tile over its V, [64 t][128], 16-byte
        // chunks of odd tokens shifted by half a bank row
        auto outputs = [&](int c, int s) {
            wait_all(&B->o, c & 1);
            if (fail) return;
            const bool odd = lane & 1;
            const int ch = (r & ~1) / 8;
            const uint32_t ot = sbase + L::V + s * L::V_BYTES + (r & 6) * 2;
            float o[32];
            tmem_ld32(tl + L::COL_O + 64 * (c & 1) + 32 * hh, o);
            tmem_ld_wait();
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const float send = odd ? o[2 * m] : o[2 * m + 1];
                const float recv = __shfl_xor_sync(0xffffffffu, send, 1);
                const int t = 32 * hh + 2 * m + (odd ? 1 : 0);
                st_shared_b32(ot + t * 256 + ((ch ^ (odd ? 4 : 0)) << 4), odd ? pack_bf16(recv, o[2 * m + 1]) : pack_bf16(o[2 * m], recv));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->ot_full[s]);
        };
        for (int c = 0; c < w.blocks && !fail; ++c) {
            const int s = at.s;
            const uint32_t p = c & 1;
            if (c > 0) outputs(c - 1, last.s);
            const float* vec = reinterpret_cast<const float*>(sm + L::VEC) + s * kVec;
            float y[32];
            // ---- R = b V - b G Z, tokens 32 hh .. ------------------------------------
            wait_all(&B->ready[p], (c >> 1) & 1);
            wait_all(&B->v_full[s], at.phase);
            wait_all(&B->z, p);
            if (fail) break;
            tmem_ld32(tl + L::COL_Z + 32 * hh, y);
            {
                const uint32_t av = sbase + L::V + s * L::V_BYTES + (r / 64) * 8192 + (r % 8) * 2;
                const uint32_t c8 = (r % 64) / 8;
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = ld_shared_bf16(av + sw128_off(32 * hh + i, c8));
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 b4 = *reinterpret_cast<const float4*>(vec + C + 32 * hh + i);
                    const float4 g4 = *reinterpret_cast<const float4*>(vec + 2 * C + 32 * hh + i);
                    y[i] = b4.x * v[i] - g4.x * y[i];
                    y[i + 1] = b4.y * v[i + 1] - g4.y * y[i + 1];
                    y[i + 2] = b4.z * v[i + 2] - g4.z * y[i + 2];
                    y[i + 3] = b4.w * v[i + 3] - g4.w * y[i + 3];
                }
            }
            store_split(tl + L::COL_R + 16 * hh, tl + L::COL_R + 32 + 16 * hh, y);
            signal(&B->r);
            // ---- O = G (Q X^T), in place, while U is computed ---------------------------
            wait_all(&B->o1, p);
            if (fail) break;
            tmem_ld32(tl + L::COL_O + 64 * p + 32 * hh, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(vec + 3 * C + 32 * hh + i);
                y[i] *= g4.x;
                y[i + 1] *= g4.y;
                y[i + 2] *= g4.z;
                y[i + 3] *= g4.w;
            }
            tmem_st32(tl + L::COL_O + 64 * p + 32 * hh, reinterpret_cast<const uint32_t(&)[32]>(y));
            // ---- U' = U D_63 for the state, then U for the outputs ------------------------
            wait_all(&B->u, p);
            if (fail) break;
            tmem_ld32(tl + L::COL_Z + 32 * hh, y);
            tmem_ld_wait();
            {
                float d[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 d4 = *reinterpret_cast<const float4*>(vec + 4 * C + 32 * hh + i);
                    d[i] = y[i] * d4.x;
                    d[i + 1] = y[i + 1] * d4.y;
                    d[i + 2] = y[i + 2] * d4.z;
                    d[i + 3] = y[i + 3] * d4.w;
                }
                store_split(tl + L::COL_UD + 16 * hh, tl + L::COL_UD + 32 + 16 * hh, d);
            }
            signal(&B->up);
            store_split(tl + L::COL_R + 16 * hh, tl + L::COL_R + 32 + 16 * hh, y);
            signal(&B->uo);
            // ---- X = G_63 X + dX ----------------------------------------------------------
            const float gc = vec[3 * C + C - 1];
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&B->vec_free[s]);
            last = at;
            at.next();
        }
        if (!fail) {
#pragma unroll
            for (int i = 0; i < XH; i += 4)
                *reinterpret_cast<float4*>(sp + i) = make_float4(X[i], X[i + 1], X[i + 2], X[i + 3]);
            outputs(w.blocks - 1, last.s);
        }
        if (fail) status = kStatusMmaWait;
    } else if (warp < kConvWarps + kPrepWarps) {
        if (!prep_warps<DK>(a, w, sm, sbase, B, tmem)) {
            fail = true;
            status = kStatusMmaWait;
            if (tid == 32 * kConvWarps) {
                *abort = 1;
                mma_commit(&B->drain[1]);
                mbar_wait(&B->drain[1], 0, 100000000ull);
            }
        }
    } else if (warp == kConvWarps + kPrepWarps) {
        // ======================= MMA issue ==========================================
        if (lane == 0) {
            constexpr uint32_t ID_64 = idesc_bf16(128, 64, false, false);
            constexpr uint32_t ID_K = idesc_bf16(128, DK, false, true);
            // the A operand of k-step kk: channels 16 kk ..
            auto colx = [&](int kk) { return tmem + L::COL_X + (kk / (XH / 16)) * XH + (kk % (XH / 16)) * 8; };
            Ring3 at;
            for (int c = 0; c < w.blocks && !fail; ++c, at.next()) {
                const uint32_t p = c & 1;
                const uint32_t kq = sbase + L::KQ + at.s * L::KQ_BYTES;
                const uint32_t tp = sbase + L::TP + p * L::TP_BYTES;
                wait(&B->kq_full[at.s], at.phase);
                wait(&B->ready[p], (c >> 1) & 1);
                wait(&B->x, p);
                if (fail) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_bf16_ts(tmem + L::COL_Z, colx(kk), kmaj(kq + (kk / 4) * 16384 + (kk % 4) * 32), ID_64, kk > 0);
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_bf16_ts(tmem + L::COL_Z, colx(kk) + XH / 2, kmaj(kq + (kk / 4) * 16384 + (kk % 4) * 32), ID_64, true);
                mma_commit(&B->z);
                if (c >= 2) {   // the outputs of block c - 2 have left this buffer
                    Ring3 two = at;   // c - 2 is the next stage's block before
                    two.next();
                    wait(&B->ot_full[two.s], two.phase ^ 1);
                    if (fail) break;
                    tc_fence_after();
                }
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_bf16_ts(tmem + L::COL_O + 64 * p, colx(kk), kmaj(kq + 8192 + (kk / 4) * 16384 + (kk % 4) * 32), ID_64,
                                kk > 0);
                mma_commit(&B->o1);
                wait(&B->r, p);
                if (fail) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ts(tmem + L::COL_Z, tmem + L::COL_R + 8 * kk, kmaj(tp + kk * 32), ID_64, kk > 0);
                    mma_bf16_ts(tmem + L::COL_Z, tmem + L::COL_R + 32 + 8 * kk, kmaj(tp + kk * 32), ID_64, true);
                    mma_bf16_ts(tmem + L::COL_Z, tmem + L::COL_R + 8 * kk, kmaj(tp + 8192 + kk * 32), ID_64, true);
                }
                mma_commit(&B->u);
                wait(&B->up, p);
                if (fail) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ts(tmem + L::COL_X, tmem + L::COL_UD + 8 * kk, mnmaj(kq + kk * 2048, 16384), ID_K, kk > 0);
                    mma_bf16_ts(tmem + L::COL_X, tmem + L::COL_UD + 32 + 8 * kk, mnmaj(kq + kk * 2048, 16384), ID_K, true);
                }
                mma_commit(&B->dx);
                wait(&B->uo, p);
                if (fail) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ts(tmem + L::COL_O + 64 * p, tmem + L::COL_R + 8 * kk, kmaj(tp + 16384 + kk * 32), ID_64, true);
                    mma_bf16_ts(tmem + L::COL_O + 64 * p, tmem + L::COL_R + 32 + 8 * kk, kmaj(tp + 16384 + kk * 32), ID_64, true);
                }
                mma_commit(&B->o);
                // only where somebody will wait: an arrival after the CTA has left would hit another's memory
                if (c + kTiles < w.blocks) mma_commit(&B->kq_free[at.s]);
                if (c + 2 < w.blocks) mma_commit(&B->tp_free[p]);
            }
            if (fail) {   // every MMA issued completes before the CTA leaves (bounded)
                status = kStatusMmaWait;
                mma_commit(&B->drain[0]);
                mbar_wait(&B->drain[0], 0, 100000000ull);
            }
        }
    } else if (warp == kConvWarps + kPrepWarps + 1) {
        // ======================= loads ===============================================
        if (lane == 0) {
            Ring3 at;
            int c = 0;
            for (; c < w.blocks; ++c, at.next()) {
                const int s = at.s, row = w.rq.row0 + c * C;
                if (c >= kTiles) wait(&B->kq_free[s], at.phase ^ 1);
                if (fail) break;
                uint8_t* kq = sm + L::KQ + s * L::KQ_BYTES;
                mbar_arrive_expect_tx(&B->kq_full[s], L::KQ_BYTES);
#pragma unroll
                for (int x = 0; x < KA; ++x) {
                    tma_load_3d(&tmk, &B->kq_full[s], kq + x * 16384, x * 64, w.khead, row);
                    tma_load_3d(&tmq, &B->kq_full[s], kq + x * 16384 + 8192, x * 64, w.khead, row);
                }
                if (c >= kTiles) wait(&B->v_free[s], at.phase ^ 1);
                if (fail) break;
                uint8_t* v = sm + L::V + s * L::V_BYTES;
                mbar_arrive_expect_tx(&B->v_full[s], L::V_BYTES);
#pragma unroll
                for (int x = 0; x < DV / 64; ++x) tma_load_3d(&tmv, &B->v_full[s], v + x * 8192, x * 64, w.head, row);
            }
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
    } else {
        // ======================= output copies =======================================
        Ring3 at;
        __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(w.rq.row0) * a.Hv + w.head) * DV;
        const size_t ostep = static_cast<size_t>(a.Hv) * DV;
        for (int c = 0; c < w.blocks; ++c, at.next()) {
            wait(&B->ot_full[at.s], at.phase);
            fail = !__all_sync(0xffffffffu, !fail);
            if (fail) break;
            const uint32_t ot = sbase + L::V + at.s * L::V_BYTES;
            const int n = min(C, w.rq.len - c * C);
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
        if (fail) status = kStatusMmaWait;
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

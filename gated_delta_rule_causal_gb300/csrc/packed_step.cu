// The gated delta rule token by token over packed requests, states in a pool
// of slots: decode steps, a few drafted tokens, and every type and head size
// that the blockwise kernel does not take. Per value head and state row i
// (key head h * Hk / Hv), for each token
//
//   u_i = beta (v_i - g S_i . k),   S_i = g S_i + u_i k,
//   o_i = S_i . q = g (old S_i . q) + u_i (k . q)
//
// A warp owns a unit of state rows of one request's head: the rows are read
// once, stay in registers over all the request's tokens and are written once,
// so a one-token step moves each state once in and once out and HBM bounds
// it; a request without tokens seen starts from zeros and reads nothing.
// Each lane holds four consecutive columns of a row, as a 16-byte vector. The
// two products S k and S q of the unit's eight row passes are summed over the
// lanes together, by halving: each exchange sends the half of the partial sums
// that the partner keeps, 17 shuffles for 16 sums where one by one would take
// 80; the lane that ends up with S_i . k computes u_i. The next token's
// vectors are loaded before the current one is used.
#include <cuda_bf16.h>

#include "kernels.h"
#include "launch.cuh"
#include "packed.h"
#include "ptx.cuh"

namespace la {
namespace packed {
namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 8;   // row passes of a unit: 16-byte loads in flight per lane

template <typename IO> __device__ __forceinline__ float4 ld4(const IO* p);
template <> __device__ __forceinline__ float4 ld4<float>(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
template <> __device__ __forceinline__ float4 ld4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = unpack_bf16(u.x), b = unpack_bf16(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float ld1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }

// Sum of x over the W consecutive lanes of a group, in every lane.
template <int W>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// x[i] summed over the W lanes of a group, i < 16. By halving while there is
// more than one value: lane l ends with the sum of value l * 16 / W (W 16 or 32).
template <int W>
__device__ __forceinline__ float sums_by_halving(float (&x)[16], int lane) {
    int o = W / 2;
#pragma unroll
    for (int n = 8; n > 0; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? x[i + n] : x[i], send = up ? x[i] : x[i + n];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    if (W == 32) x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
    return x[0];
}

template <int DK, typename IO>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepArgs a) {
    constexpr int LPR = DK / 4;          // lanes per row
    constexpr int RPP = 32 / LPR;        // rows per pass
    constexpr int R = RPP * kPasses;     // rows per unit
    constexpr bool HALVING = LPR >= 16;
    const int dv = a.dv;
    const int uph = (dv + R - 1) / R;    // units per head
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, cl = lane % LPR;
    // by halving: the row pass whose sums this lane holds, and whether it
    // holds S k (lower half of the group) or S q
    const int myp = (cl * 16 / LPR) & 7;
    const bool upper = cl >= LPR / 2;
    const long long warp0 = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const long long nwarps = (static_cast<long long>(gridDim.x) * kThreads) >> 5;
    const IO* q = static_cast<const IO*>(a.q);
    const IO* k = static_cast<const IO*>(a.k);
    const IO* v = static_cast<const IO*>(a.v);
    IO* out = static_cast<IO*>(a.out);

    griddep_launch_dependents();
    griddep_wait();   // the plan and the states of the step before are complete
    const int per_req = a.Hv * uph;
    const long long units = static_cast<long long>(a.requests) * per_req;
    for (long long u = warp0; u < units; u += nwarps) {
        const int r = static_cast<int>(u / per_req);
        const int hu = static_cast<int>(u % per_req);
        const int h = hu / uph, r0 = (hu % uph) * R;
        const int hk = h / (a.Hv / a.Hk);
        Request x;
        if (!read_request(a, r, x)) continue;
        float* st = a.states + (static_cast<size_t>(x.slot) * a.Hv + h) * dv * DK;
        float4 S[kPasses];
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int row = r0 + p * RPP + sub;
            S[p] = (!x.fresh && row < dv) ? __ldcs(reinterpret_cast<const float4*>(st + static_cast<size_t>(row) * DK) + cl)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const IO* qp = q + static_cast<size_t>(x.row0) * a.q_stride + hk * DK + 4 * cl;
        const IO* kp = k + static_cast<size_t>(x.row0) * a.k_stride + hk * DK + 4 * cl;
        const IO* vp = v + static_cast<size_t>(x.row0) * a.v_stride + static_cast<size_t>(h) * dv + r0;
        const float* gp = a.gate + static_cast<size_t>(x.row0) * a.Hv + h;
        const float* bp = a.beta + static_cast<size_t>(x.row0) * a.Hv + h;
        IO* op = out + (static_cast<size_t>(x.row0) * a.Hv + h) * dv + r0;
        const int myrow = myp * RPP + sub;   // row of the unit whose u this lane computes
        const bool mine = r0 + myrow < dv;
        auto load_v = [&](const IO* p, float (&w)[HALVING ? 1 : kPasses]) {
            if (HALVING) {
                w[0] = mine ? ld1(p + myrow) : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < (HALVING ? 1 : kPasses); ++i)
                    w[i] = r0 + i * RPP + sub < dv ? ld1(p + i * RPP + sub) : 0.f;
            }
        };
        float4 kn = ld4(kp), qn = ld4(qp);
        float vn[HALVING ? 1 : kPasses];
        load_v(vp, vn);
        float gn = __ldg(gp), bn = __ldg(bp);
        for (int t = 0; t < x.len; ++t) {
            const float4 k4 = kn, q4 = qn;
            float vr[HALVING ? 1 : kPasses];
#pragma unroll
            for (int i = 0; i < (HALVING ? 1 : kPasses); ++i) vr[i] = vn[i];
            const float g = gn, b = bn;
            if (t + 1 < x.len) {
                kp += a.k_stride;
                qp += a.q_stride;
                vp += a.v_stride;
                gp += a.Hv;
                bp += a.Hv;
                kn = ld4(kp);
                qn = ld4(qp);
                load_v(vp, vn);
                gn = __ldg(gp);
                bn = __ldg(bp);
            }
            const float kq = group_sum<LPR>(dot4(k4, q4));
            if constexpr (HALVING) {
                float d[16];
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    d[p] = dot4(S[p], k4);
                    d[8 + p] = dot4(S[p], q4);
                }
                const float s0 = sums_by_halving<LPR>(d, cl);
                const float s1 = __shfl_xor_sync(0xffffffffu, s0, LPR / 2);
                const float sk = upper ? s1 : s0, sq = upper ? s0 : s1;
                const float ui = b * (vr[0] - g * sk);
                if (!upper && mine && (LPR == 16 || !(cl & 1))) st1(op + myrow, g * sq + ui * kq);
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    const float w = __shfl_sync(0xffffffffu, ui, sub * LPR + p * (LPR / 16));
                    S[p].x = g * S[p].x + w * k4.x;
                    S[p].y = g * S[p].y + w * k4.y;
                    S[p].z = g * S[p].z + w * k4.z;
                    S[p].w = g * S[p].w + w * k4.w;
                }
            } else {
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    const float sk = group_sum<LPR>(dot4(S[p], k4));
                    const float sq = group_sum<LPR>(dot4(S[p], q4));
                    const float w = b * (vr[HALVING ? 0 : p] - g * sk);
                    S[p].x = g * S[p].x + w * k4.x;
                    S[p].y = g * S[p].y + w * k4.y;
                    S[p].z = g * S[p].z + w * k4.z;
                    S[p].w = g * S[p].w + w * k4.w;
                    if (cl == 0 && r0 + p * RPP + sub < dv) st1(op + p * RPP + sub, g * sq + w * kq);
                }
            }
            op += static_cast<size_t>(a.Hv) * dv;
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int row = r0 + p * RPP + sub;
            if (row < dv) __stcs(reinterpret_cast<float4*>(st + static_cast<size_t>(row) * DK) + cl, S[p]);
        }
    }
}

template <int DK, typename IO>
cudaError_t run(const StepArgs& a, cudaStream_t s) {
    // persistent: as many CTAs as are resident at once, no more than there are units
    static int per_sm = 0;
    if (per_sm == 0) {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, step_kernel<DK, IO>, kThreads, 0) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        per_sm = n;
    }
    constexpr int rows = 32 / (DK / 4) * kPasses;
    const long long units = static_cast<long long>(a.requests) * a.Hv * ((a.dv + rows - 1) / rows);
    long long grid = (units + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > static_cast<long long>(a.sm_count) * per_sm) grid = static_cast<long long>(a.sm_count) * per_sm;
    return launch_pdl(step_kernel<DK, IO>, static_cast<unsigned>(grid), kThreads, 0, s, a);
}

template <typename IO>
cudaError_t run_dk(const StepArgs& a, cudaStream_t s) {
    switch (a.dk) {
        case 16: return run<16, IO>(a, s);
        case 32: return run<32, IO>(a, s);
        case 64: return run<64, IO>(a, s);
        case 128: return run<128, IO>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, cudaStream_t s) {
    return a.io == kFp32 ? run_dk<float>(a, s) : run_dk<__nv_bfloat16>(a, s);
}

}  // namespace packed
}  // namespace la

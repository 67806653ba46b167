// The gated delta rule token by token over packed requests, states in a pool
// of slots: decode steps, a few tokens a request, and every type and head size
// that the blockwise kernel does not take. Per value head and state row i
// (key head h * Hk / Hv), for each token
//
//   u_i = beta (v_i - g S_i . k),   S_i = g S_i + u_i k,
//   o_i = S_i . q = g (old S_i . q) + u_i (k . q)
//
// A warp owns a unit of state rows (4 KB, less where there are few) of one
// request's head: the rows are read once, stay in registers over all the
// request's tokens and are written once, so a one-token step moves each state
// once in and once out and HBM bounds it; a request without tokens seen starts
// from zeros and reads nothing.
// Eight lanes share a row (four at d_k 16), each with every eighth 16-byte
// vector of it, so that a few tokens cost little besides: at d_k 128 four sums
// over eight lanes where 32 lanes to a row would have sixteen over 32. The two
// products S k and S q of a unit's row passes are summed over the lanes
// together, by halving: each exchange sends the half of the partial sums that
// the partner keeps; the lane that ends up with S_i . k computes u_i. The next
// token's vectors are loaded before the current one is used.
//
// Measured, d 128, 16 heads, bf16: one token of 256 requests 83 us, 0.96 of the
// measured copy bandwidth; of 4 requests 3.5 us, the launch and two trips to
// memory; 400 tokens of 128 requests 53 us, 0.75 of it: there the tokens'
// arithmetic, about 9 us a token, is in part beside the traffic and in part
// before it. Tried and slower: the next unit's state into
// shared memory (256 requests 90 us) or L2 (98 us) while one is computed; three
// CTAs per SM at 80 registers (89 us).
#include <cuda_bf16.h>

#include "kernels.h"
#include "launch.cuh"
#include "packed.h"
#include "ptx.cuh"

namespace la {
namespace packed {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 8;   // 16-byte vectors of the state per lane: loads in flight

// Loads of what other launches write; PAST: past the SM's own cache, for a launch that does not begin with a wait for the
// one before it.
template <bool PAST, typename T>
__device__ __forceinline__ T fetch(const T* p) {
    return PAST ? __ldcg(p) : __ldg(p);
}
// Four elements as they are loaded, and as numbers.
template <typename IO, bool PAST> struct Raw;
template <bool PAST> struct Raw<float, PAST> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = fetch<PAST>(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ float4 get() const { return u; }
};
template <bool PAST> struct Raw<__nv_bfloat16, PAST> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = fetch<PAST>(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ float4 get() const {
        const float2 a = unpack_bf16(u.x), b = unpack_bf16(u.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
template <bool PAST> __device__ __forceinline__ float ld1(const float* p) { return fetch<PAST>(p); }
template <bool PAST> __device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(fetch<PAST>(p)); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
// Two fp32 values in one register pair: one instruction for two multiply-adds.
using Pair = unsigned long long;
struct __align__(16) Pairs {   // four consecutive columns
    Pair a, b;
};
__device__ __forceinline__ Pairs pairs(float4 x) {
    Pairs y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y.a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y.b) : "f"(x.z), "f"(x.w));
    return y;
}
__device__ __forceinline__ Pair both(float x) {
    Pair y;
    asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Pair fma2(Pair x, Pair y, Pair z) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair x, Pair y) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float sum(Pair x) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
    return lo + hi;
}

// x[i] summed over the W lanes of a group, i < N. By halving while there is
// more than one value: lane l ends with the sums of values l N / W ..
template <int N, int W>
__device__ __forceinline__ void sums_by_halving(float (&x)[N], int lane) {
    int n = N / 2;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        if (n > 0) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = up ? x[i + n] : x[i], send = up ? x[i] : x[i + n];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            n /= 2;
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
        }
    }
}

// How a warp holds a unit: lane (sub, cl) has vectors cl, cl + LPR, ... of rows p RPP + sub.
template <int DK>
struct Lanes {
    static constexpr int LPR = DK >= 32 ? 8 : 4;      // lanes per row
    static constexpr int V = DK / (4 * LPR);          // vectors of a row per lane
};
template <int DK, int P_>
struct Unit {
    static constexpr int LPR = Lanes<DK>::LPR, V = Lanes<DK>::V;
    static constexpr int P = P_;                      // row passes
    static constexpr int RPP = 32 / LPR;              // rows per pass
    static constexpr int R = RPP * P;                 // rows
    static constexpr int Q = LPR / 2;                 // lanes that end with S k (the lower half of a row's), with S q
    static constexpr int M = P >= Q ? P / Q : 1;      // passes whose sums a lane ends with,
    static constexpr int DUP = P >= Q ? 1 : Q / P;    // or lanes that end with the same
    Pairs S[P][V];
    int sub, cl, pass0;
    bool upper;

    __device__ __forceinline__ explicit Unit(int lane)
        : sub(lane / LPR), cl(lane % LPR), pass0(lane % LPR % Q / DUP * M), upper(lane % LPR >= Q) {}
    // row of the unit whose u (i < M) this lane computes
    __device__ __forceinline__ int own_row(int i) const { return (pass0 + i) * RPP + sub; }

    // One token: the state's update and the outputs of the unit's `rows` rows.
    template <typename IO>
    __device__ __forceinline__ void step(const Pairs (&k4)[V], const Pairs (&q4)[V], const float (&v)[M], float g, float b,
                                         IO* out, int rows) {
        Pair kq2 = mul2(k4[0].a, q4[0].a);
        kq2 = fma2(k4[0].b, q4[0].b, kq2);
#pragma unroll
        for (int w = 1; w < V; ++w) kq2 = fma2(k4[w].b, q4[w].b, fma2(k4[w].a, q4[w].a, kq2));
        float kq = sum(kq2), d[2 * P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            Pair x = fma2(S[p][0].b, k4[0].b, mul2(S[p][0].a, k4[0].a)), y = fma2(S[p][0].b, q4[0].b, mul2(S[p][0].a, q4[0].a));
#pragma unroll
            for (int w = 1; w < V; ++w) {
                x = fma2(S[p][w].b, k4[w].b, fma2(S[p][w].a, k4[w].a, x));
                y = fma2(S[p][w].b, q4[w].b, fma2(S[p][w].a, q4[w].a, y));
            }
            d[p] = sum(x);
            d[P + p] = sum(y);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        sums_by_halving<2 * P, LPR>(d, cl);
        float u[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, d[i], Q);
            const float sk = upper ? other : d[i], sq = upper ? d[i] : other;
            u[i] = b * (v[i] - g * sk);
            if (!upper && cl % DUP == 0 && own_row(i) < rows) st1(out + own_row(i), g * sq + u[i] * kq);
        }
        const Pair g2 = both(g);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const Pair c = both(__shfl_sync(0xffffffffu, u[p % M], sub * LPR + p / M * DUP));
#pragma unroll
            for (int w = 0; w < V; ++w) {
                S[p][w].a = fma2(c, k4[w].a, mul2(g2, S[p][w].a));
                S[p][w].b = fma2(c, k4[w].b, mul2(g2, S[p][w].b));
            }
        }
    }
    // The unit's rows to or from memory (vectors cl + LPR w of row p RPP + sub of `st`)
    __device__ __forceinline__ size_t at(int p, int w) const { return static_cast<size_t>(p * RPP + sub) * DK + 4 * (cl + LPR * w); }
    template <bool PAST>
    __device__ __forceinline__ void load(const float* st, int rows) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int w = 0; w < V; ++w) {
                const float4* from = reinterpret_cast<const float4*>(st + at(p, w));
                S[p][w] = pairs(p * RPP + sub < rows ? (PAST ? __ldcg(from) : __ldcs(from)) : make_float4(0.f, 0.f, 0.f, 0.f));
            }
    }
    __device__ __forceinline__ void store(float* st, int rows) const {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int w = 0; w < V; ++w)
                if (p * RPP + sub < rows) __stcs(reinterpret_cast<ulonglong2*>(st + at(p, w)), make_ulonglong2(S[p][w].a, S[p][w].b));
    }
};

// What a unit reads and writes.
template <typename IO>
struct Where {
    const IO *q, *k, *v;
    const float *gate, *beta;
    float* st;
    IO* out;
    int len, rows;   // tokens; rows of the unit
    bool fresh;
};
// Unit u; false if its request has no part.
template <class U, int DK, bool PAST, typename IO>
__device__ __forceinline__ bool find(const StepArgs& a, int u, Where<IO>& x) {
    constexpr int R = U::R;
    const int uph = (a.dv + R - 1) / R, per_req = a.Hv * uph;   // units per head, per request
    const int hu = u % per_req, h = hu / uph, r0 = hu % uph * R, hk = h / (a.Hv / a.Hk);
    Request rq;
    if (!read_request<PAST>(a, u / per_req, rq)) return false;
    const size_t row = static_cast<size_t>(rq.row0);
    x.q = static_cast<const IO*>(a.q) + row * a.q_stride + hk * DK;
    x.k = static_cast<const IO*>(a.k) + row * a.k_stride + hk * DK;
    x.v = static_cast<const IO*>(a.v) + row * a.v_stride + static_cast<size_t>(h) * a.dv + r0;
    x.gate = a.gate + row * a.Hv + h;
    x.beta = a.beta + row * a.Hv + h;
    x.st = a.states + ((static_cast<size_t>(rq.slot) * a.Hv + h) * a.dv + r0) * DK;
    x.out = static_cast<IO*>(a.out) + (row * a.Hv + h) * a.dv + r0;
    x.len = rq.len;
    x.rows = min(R, a.dv - r0);
    x.fresh = rq.fresh;
    return true;
}
template <class U>
__host__ __device__ inline long long unit_count(const StepArgs& a) {
    return static_cast<long long>(a.requests) * a.Hv * ((a.dv + U::R - 1) / U::R);
}

// BESIDE: the launch before this one runs other requests of the same step, and lets this one start once it has waited
// for what came before it; no row or slot is in both. So whatever wrote the plan, the tensors and the states is complete
// when a CTA of this launch starts, without a wait of its own. That holds even if another thread's launch came in
// between on the stream: it starts no earlier than every CTA of the blockwise launch has let it, which is after its wait.
template <int DK, typename IO, int P, bool BESIDE>
__global__ void __launch_bounds__(kThreads, 2) step_kernel(const StepArgs a) {
    using U = Unit<DK, P>;
    U s(threadIdx.x & 31);
    if constexpr (!BESIDE) {   // (beside, the next launch would only wait on the same SMs)
        griddep_launch_dependents();
        griddep_wait();   // the plan and the states of the step before are complete
    }
    const int units = static_cast<int>(unit_count<U>(a)), stride = (gridDim.x * kThreads) >> 5;
    for (int u = (blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += stride) {
        Where<IO> x;
        if (!find<U, DK, BESIDE>(a, u, x)) continue;
        s.template load<BESIDE>(x.st, x.fresh ? 0 : x.rows);
        Raw<IO, BESIDE> kn[U::V], qn[U::V];   // of the next token
        float vn[U::M], gn, bn;
        auto load = [&]() {
#pragma unroll
            for (int w = 0; w < U::V; ++w) {
                kn[w].load(x.k + 4 * (s.cl + U::LPR * w));
                qn[w].load(x.q + 4 * (s.cl + U::LPR * w));
            }
#pragma unroll
            for (int i = 0; i < U::M; ++i) vn[i] = s.own_row(i) < x.rows ? ld1<BESIDE>(x.v + s.own_row(i)) : 0.f;
            gn = fetch<BESIDE>(x.gate);
            bn = fetch<BESIDE>(x.beta);
        };
        load();
        for (int t = 0; t < x.len; ++t) {
            Pairs k4[U::V], q4[U::V];
            float v[U::M];
#pragma unroll
            for (int w = 0; w < U::V; ++w) {
                k4[w] = pairs(kn[w].get());
                q4[w] = pairs(qn[w].get());
            }
#pragma unroll
            for (int i = 0; i < U::M; ++i) v[i] = vn[i];
            const float g = gn, b = bn;
            if (t + 1 < x.len) {
                x.k += a.k_stride;
                x.q += a.q_stride;
                x.v += a.v_stride;
                x.gate += a.Hv;
                x.beta += a.Hv;
                load();
            }
            s.step(k4, q4, v, g, b, x.out, x.rows);
            x.out += static_cast<size_t>(a.Hv) * a.dv;
        }
        s.store(x.st, x.rows);
    }
    // Whoever waits for this launch waits for both: one warp stays until the other is complete. (All of them, 304 CTAs,
    // slow what runs beside them down.)
    if (BESIDE && blockIdx.x == 0 && threadIdx.x < 32) griddep_wait();
}

template <int DK, typename IO, int P, bool BESIDE>
cudaError_t run_units(const StepArgs& a, cudaStream_t s) {
    // two CTAs per SM, each warp one unit after another (at most 2^14 requests x 2^12 heads x 2^4 units of 4 KB)
    const long long grid = (unit_count<Unit<DK, P>>(a) + kThreads / 32 - 1) / (kThreads / 32), most = 2ll * a.sm_count;
    return launch_pdl(step_kernel<DK, IO, P, BESIDE>, static_cast<unsigned>(grid < most ? grid : most), kThreads, 0, s, a);
}
template <int DK, typename IO>
cudaError_t run(const StepArgs& a, cudaStream_t s) {
    // Units of one pass (4 or 8 rows) while no SM gets more than a CTA of them: a token takes a warp less time. Measured
    // against units of 4 KB, fp32, four requests of 64 tokens, 8 heads: d 64 25.0 us (27.6), d 128 32.3 (37.5), d_k 16
    // and d_v 128 20.9 (51.7); six requests of 611 tokens, 8 heads of 64: 75 us (96).
    if (unit_count<Unit<DK, 1>>(a) <= a.sm_count * (kThreads / 32)) return run_units<DK, IO, 1, false>(a, s);
    return run_units<DK, IO, kVectors / Lanes<DK>::V, false>(a, s);
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

cudaError_t launch_step_beside(const StepArgs& a, cudaStream_t s) {
    if (a.io == kBf16 && a.dk == 64) return run_units<64, __nv_bfloat16, kVectors / Lanes<64>::V, true>(a, s);
    if (a.io == kBf16 && a.dk == 128) return run_units<128, __nv_bfloat16, kVectors / Lanes<128>::V, true>(a, s);
    return cudaErrorInvalidValue;
}
cudaError_t launch_step(const StepArgs& a, cudaStream_t s) {
    return a.io == kFp32 ? run_dk<float>(a, s) : run_dk<__nv_bfloat16>(a, s);
}

}  // namespace packed
}  // namespace la

// The plan of one step over packed requests, built on the GPU from the
// requests' lengths: row offsets, the state slot of every request (slots of
// ended requests go back to the free stack, new requests take from it), the
// order in which the prefill walks the requests, and for every row its
// request and position.
//
//   offsets[r] = min(sum_{i<r} max(lengths[i], 0), rows + 1)
//   request r takes part if lengths[r] > 0, its rows end by `rows` and it has
//   a slot of its own (claimed twice: the lowest request keeps it)
//
// Everything is whole numbers and every result is independent of the order in
// which threads run: prefix sums, a minimum over claims, a stable counting
// sort. One launch: CTA 0 does the requests, the other CTAs the row maps, each
// from its own prefix sum over the lengths (a few microseconds of redundant
// work instead of a second launch that waits for the first).
//
// Bound by latency: 8192 requests and 262144 rows are 2.3 MB to read and write,
// 0.3 us at the memory's rate; the dependent steps of CTA 0 (loads, claims, two
// block-wide sums, the sort) take the time, some 13000 clocks for a few requests
// and 40000 for 8192, whose steps one SM works through by 32 warps. Measured
// where no slot is given or taken back: 8 requests 6.3 us, 512 7.0 us, 8192
// 20.2 us; 8192 of which 2570 take one and 482 give theirs back 23.1 us.
#include <climits>

#include "kernels.h"
#include "launch.cuh"
#include "packed.h"
#include "ptx.cuh"

namespace la {
namespace packed {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerCta = 4 * kThreads;   // row maps: four consecutive rows a thread
constexpr int kKeys = 26;                   // bit lengths of a request's blocks (0: no part)
constexpr int kPopped = 1 << 30;            // claims from the free stack come after claims by requests
constexpr int kBatch = 4;                   // requests whose loads a thread has in flight together

// What is known of a request, a byte each in shared memory; behind the claims its sort key takes the place.
enum : int { kNegative = 1, kPositive = 2, kUnseen = 4, kEnds = 8, kNeeds = 16, kKeeps = 32, kPops = 64 };

// Exclusive prefix sum of one value per thread; `total` is the sum of all.
// Op saturates where it has to (x + y capped is associative on x, y >= 0).
template <typename T, typename Op>
__device__ __forceinline__ T block_scan(T x, T* warp_sum, T& total, Op op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = op(inc, y);
    }
    __syncthreads();   // warp_sum may still be read by the scan before
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w = op(w, y);
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    T ex = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) ex = 0;
    total = warp_sum[kWarps - 1];
    return warp > 0 ? op(ex, warp_sum[warp - 1]) : ex;
}

// Who claims a slot (scratch of CTA 0): in shared memory where it fits, else in
// the plan. One SM reaches scattered words of global memory at a few clocks
// each: 8192 requests took 33 us with the claims there.
template <bool SHARED>
__device__ __forceinline__ int claim_of(const int* owner, int x) {
    return SHARED ? owner[x] : __ldcg(owner + x);
}

template <bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanArgs a) {
    extern __shared__ int smem[];
    __shared__ unsigned long long warp_sum[kWarps];
    __shared__ int hist[kWarps * 32];
    __shared__ int found[3];   // faults, requests taking part, slots taken
    const int R = a.requests, rows = a.rows, S = a.lay.S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = (R + kThreads - 1) / kThreads;   // consecutive requests of a thread
    int* off = smem;                                                         // [R + 1]
    int* slot = smem + PlanLayout::pad(static_cast<size_t>(R) + 1);          // [R], CTA 0
    uint8_t* know = reinterpret_cast<uint8_t*>(slot + PlanLayout::pad(R));   // [R], CTA 0
    int* owner = SHARED ? reinterpret_cast<int*>(know + PlanLayout::pad(R)) : a.plan + a.lay.owner();   // [S]
    const int r0 = min(tid * E, R), r1 = min(r0 + E, R);

    griddep_wait();
    // ---- offsets (every CTA) ---------------------------------------------------
    if (tid < 3) found[tid] = 0;
    const int cap = rows + 1;
    int c0 = 0;
    if (blockIdx.x > 0) {
        for (int b = tid; b < R; b += kBatch * kThreads) {
            int n[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) n[i] = b + i * kThreads < R ? __ldg(a.lengths + b + i * kThreads) : 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (b + i * kThreads < R) off[b + i * kThreads] = min(max(n[i], 0), cap);
        }
    } else {   // CTA 0: slots too; the owners that may be claimed are cleared
        c0 = min(max(*a.free_count, 0), S);
        if (SHARED)
            for (int x = tid; x < S; x += kThreads) owner[x] = INT_MAX;
        for (int b = tid; b < R; b += kBatch * kThreads) {
            int n[kBatch], x[kBatch], sn[kBatch], f[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = b + i * kThreads;
                n[i] = r < R ? __ldg(a.lengths + r) : 0;
                sn[i] = r < R ? __ldg(a.seen + r) : 0;
                x[i] = r < R ? a.slots[r] : -1;
                f[i] = !SHARED && r < min(R, c0) ? a.free_slots[c0 - 1 - r] : -1;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = b + i * kThreads;
                if (r < R) {
                    off[r] = min(max(n[i], 0), cap);
                    slot[r] = x[i];
                    know[r] = (n[i] < 0 ? kNegative : 0) | (n[i] > 0 ? kPositive : 0) | (sn[i] == 0 ? kUnseen : 0);
                    if (!SHARED && x[i] >= 0 && x[i] < S) owner[x[i]] = INT_MAX;
                    if (!SHARED && f[i] >= 0 && f[i] < S) owner[f[i]] = INT_MAX;
                }
            }
        }
    }
    __syncthreads();
    // Sums inside a warp's consecutive requests first, then the warps' own over the block. (A thread's consecutive
    // requests would lie in the same few banks.)
    auto capped = [cap](int x, int y) { return min(x + y, cap); };
    const int per_warp = (R + kThreads - 1) / kThreads * 32;   // consecutive requests of a warp
    const int w0 = min(warp * per_warp, R), w1 = min(w0 + per_warp, R);
    {
        int carry = 0;
        for (int t0 = w0; t0 < w1; t0 += 32) {
            int x = t0 + lane < w1 ? off[t0 + lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x = capped(x, y);
            }
            const int before = __shfl_up_sync(0xffffffffu, x, 1);
            if (t0 + lane < w1) off[t0 + lane] = lane > 0 ? capped(carry, before) : carry;
            carry = capped(carry, __shfl_sync(0xffffffffu, x, 31));
        }
        int* sums = reinterpret_cast<int*>(warp_sum);
        if (lane == 0) sums[warp] = carry;
        __syncthreads();
        int x = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = capped(x, y);
        }
        const int base = __shfl_sync(0xffffffffu, x, (warp - 1) & 31);
        if (warp > 0)
            for (int t0 = w0 + lane; t0 < w1; t0 += 32) off[t0] = capped(base, off[t0]);
        if (tid == kThreads - 1) off[R] = x;
    }
    __syncthreads();

    if (blockIdx.x > 0) {
        // ---- row maps: the last request that starts at or before the row ----------
        const int row = (blockIdx.x - 1) * kRowsPerCta + 4 * tid;
        if (row >= rows) return;
        int lo = 0, hi = R;   // off[lo] <= row < off[hi] where the row is used
        const bool used = row < off[R];
        if (used) {
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (off[m] <= row) lo = m; else hi = m;
            }
        }
        int req[4], pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = row + i;
            req[i] = pos[i] = -1;
            if (used && x < off[R]) {
                while (off[lo + 1] <= x) ++lo;
                if (off[lo + 1] <= rows) {   // a request that ends past the rows given has no part
                    req[i] = lo;
                    pos[i] = a.seen[lo] + x - off[lo];
                }
            }
        }
        int* tr = a.plan + a.lay.token_request() + row;
        int* tp = a.plan + a.lay.token_position() + row;
        if (row + 4 <= rows) {
            *reinterpret_cast<int4*>(tr) = make_int4(req[0], req[1], req[2], req[3]);
            *reinterpret_cast<int4*>(tp) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int i = 0; row + i < rows; ++i) {
                tr[i] = req[i];
                tp[i] = pos[i];
            }
        }
        return;
    }

    // ---- CTA 0: the requests ------------------------------------------------------
    // (what waits for memory runs over requests tid, tid + 1024, ..., several loads
    // in flight; what needs an order over a thread's consecutive requests, in
    // shared memory)
    int* p_off = a.plan + a.lay.offsets();
    // claims: the lowest request that names a slot
    for (int r = tid; r < R; r += kThreads) {
        const int x = slot[r];
        if (x >= 0 && x < S) atomicMin(&owner[x], r);
        p_off[r] = off[r];
    }
    if (tid == 0) p_off[R] = off[R];
    __syncthreads();
    // per request: ends (gives its slot back), needs one, keeps its own, or none of these
    int bad = 0, part = 0, taken = 0;
    int sn[kBatch];   // tokens seen, of the warp's first requests: wanted at the end
#pragma unroll
    for (int i = 0; i < kBatch; ++i) sn[i] = w0 + 32 * i + lane < w1 ? __ldg(a.seen + w0 + 32 * i + lane) : 0;
    for (int b = tid; b < R; b += kBatch * kThreads) {
        int o[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads, x = r < R ? slot[r] : -1;
            o[i] = x >= 0 && x < S ? claim_of<SHARED>(owner, x) : -1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads;
            if (r < R) {
                const int x = slot[r], k = know[r];
                const bool mine = o[i] == r, fits = off[r + 1] <= rows, pos = k & kPositive;
                if (pos && !fits) bad |= kFaultRows;
                if (x >= S || x < -1) bad |= kFaultSlot;
                if (x >= 0 && x < S && !mine) bad |= kFaultOwner;
                if (pos && x == -1 && !(k & kUnseen)) bad |= kFaultState;
                know[r] = ((k & kNegative) && mine ? kEnds : 0) | (pos && x == -1 && (k & kUnseen) && fits ? kNeeds : 0) |
                          (pos && mine && fits ? kKeeps : 0);
            }
        }
    }
    __syncthreads();
    unsigned long long cnt = 0;   // needs << 32 | ends
    for (int r = r0; r < r1; ++r) cnt += (know[r] & kEnds ? 1ull : 0ull) + (know[r] & kNeeds ? 1ull << 32 : 0ull);
    unsigned long long total;
    const unsigned long long at =
        block_scan(cnt, warp_sum, total, [](unsigned long long x, unsigned long long y) { return x + y; });
    const int n_ends = static_cast<int>(total & 0xffffffffu);
    const int c1 = min(c0 + n_ends, S);
    if (tid == 0 && c0 + n_ends > S) bad |= kFaultOverflow;
    {
        int e = static_cast<int>(at & 0xffffffffu), w = static_cast<int>(at >> 32);
        for (int r = r0; r < r1; ++r) {
            if (know[r] & kEnds) {
                if (c0 + e < S) a.free_slots[c0 + e] = slot[r];
                ++e;
                owner[slot[r]] = INT_MAX;   // it may be taken again below
                slot[r] = -1;
            } else if (know[r] & kNeeds) {
                slot[r] = w++;              // the place on the stack
            }
        }
    }
    __syncthreads();
    for (int b = tid; b < R; b += kBatch * kThreads) {
        int f[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads;
            const bool needs = r < R && (know[r] & kNeeds);
            const int w = needs ? c1 - 1 - slot[r] : -1;
            f[i] = w >= 0 ? a.free_slots[w] : -1;
            if (w >= 0) ++taken;
            else if (needs) bad |= kFaultFree;
            if (w >= 0 && (f[i] < 0 || f[i] >= S)) {
                bad |= kFaultSlot;
                f[i] = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads;
            if (r < R && (know[r] & kNeeds)) {
                slot[r] = f[i];
                if (f[i] >= 0) {
                    atomicMin(&owner[f[i]], kPopped + r);
                    know[r] = kPops;
                }
            }
        }
    }
    for (int i = tid; i < kWarps * 32; i += kThreads) hist[i] = 0;
    __syncthreads();
    // ---- slots out, who takes part, the sort's keys -----------------------------------
    for (int b = tid; b < R; b += kBatch * kThreads) {
        int o[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads;
            o[i] = r < R && (know[r] & kPops) ? claim_of<SHARED>(owner, slot[r]) : -1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = b + i * kThreads;
            if (r < R) {
                bool ok = know[r] & kKeeps;
                if (know[r] & kPops) {
                    ok = o[i] == kPopped + r;
                    if (!ok) {   // the stack held a slot that has an owner, or held it twice
                        bad |= kFaultOwner;
                        slot[r] = -1;
                    }
                }
                a.slots[r] = slot[r];
                if (!ok) slot[r] = -1;
                a.plan[a.lay.slots() + r] = slot[r];
                know[r] = ok ? 32 - __clz((off[r + 1] - off[r] + kBlock - 1) / kBlock) : 0;
                part += ok;
            }
        }
    }
    __syncthreads();
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int r = t0 + lane, key = r < w1 ? know[r] : kKeys + 1;
        const unsigned peers = __match_any_sync(0xffffffffu, key);
        if (r < w1 && __popc(peers & ((1u << lane) - 1)) == 0) hist[warp * 32 + key] += __popc(peers);
        __syncwarp();
    }
    const unsigned any = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad));
    part = __reduce_add_sync(0xffffffffu, part);
    taken = __reduce_add_sync(0xffffffffu, taken);
    if (lane == 0) {
        if (any) atomicOr(&found[0], static_cast<int>(any));
        if (part) atomicAdd(&found[1], part);
        if (taken) atomicAdd(&found[2], taken);
    }
    __syncthreads();   // the histogram
    if (tid == 0) {
        a.plan[0] = min(off[R], rows);
        a.plan[1] = found[1];
        a.plan[2] = c1 - found[2];
        a.plan[3] = found[0];
        a.plan[4] = R;
        a.plan[5] = rows;
        *a.free_count = c1 - found[2];
    }
    // ---- stable counting sort, most blocks first: position of (key, warp) ------------
    {
        const int key = kKeys - 1 - (tid >> 5), w = tid & 31;   // thread order = position order
        const int x = key >= 0 ? hist[w * 32 + key] : 0;
        int all;
        const int pos = block_scan(x, reinterpret_cast<int*>(warp_sum), all, [](int u, int v) { return u + v; });
        __syncthreads();
        if (key >= 0) hist[w * 32 + key] = pos;
    }
    __syncthreads();
    for (int t1 = w0; t1 < w1; t1 += 32 * kBatch) {
        if (t1 > w0)
#pragma unroll
            for (int i = 0; i < kBatch; ++i) sn[i] = t1 + 32 * i + lane < w1 ? __ldg(a.seen + t1 + 32 * i + lane) : 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = t1 + 32 * i + lane;
            const int key = r < w1 ? know[r] : kKeys + 1;
            const unsigned peers = __match_any_sync(0xffffffffu, key);
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int base = r < w1 ? hist[warp * 32 + key] : 0;
            __syncwarp();
            if (r < w1) {
                a.plan[a.lay.order() + base + rank] = r;
                reinterpret_cast<int4*>(a.plan + a.lay.items())[base + rank] =
                    make_int4(off[r], slot[r] >= 0 ? off[r + 1] - off[r] : 0, slot[r], sn[i]);
                if (rank == 0) hist[warp * 32 + key] = base + __popc(peers);
            }
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
    constexpr size_t most = 220 * 1024;   // of a CTA's 227 KB; static arrays take 4
    const size_t base = (PlanLayout::pad(static_cast<size_t>(a.requests) + 1) + PlanLayout::pad(a.requests)) * sizeof(int) +
                        PlanLayout::pad(a.requests);
    const size_t claims = a.lay.S * sizeof(int);
    const unsigned grid = 1 + (a.rows + kRowsPerCta - 1) / kRowsPerCta;
    const bool shared = base + claims <= most;
    const size_t smem = shared ? base + claims : base;
    const auto kernel = shared ? plan_kernel<true> : plan_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, kThreads, smem, s, a);
}

}  // namespace packed
}  // namespace la

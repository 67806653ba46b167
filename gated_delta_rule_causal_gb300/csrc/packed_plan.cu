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
// Bound by latency: the longest case (8192 requests, 262144 rows) reads and
// writes 2.3 MB, 0.3 us at the memory's rate; the dependent steps of CTA 0
// (loads, three block-wide sums, claims, the sort) take the time.
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
constexpr int kEnded = INT_MIN;             // mark of a request whose slot went back

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

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanArgs a) {
    extern __shared__ int smem[];
    __shared__ unsigned long long warp_sum[kWarps];
    __shared__ int hist[kWarps * 32];
    __shared__ int faults;
    const int R = a.requests, rows = a.rows, S = a.lay.S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = (R + kThreads - 1) / kThreads;   // consecutive requests of a thread
    int* off = smem;   // [R + 1]
    const int r0 = min(tid * E, R), r1 = min(r0 + E, R);

    griddep_wait();
    // ---- offsets (every CTA) ---------------------------------------------------
    if (tid == 0) faults = 0;
    const int cap = rows + 1;
    for (int r = tid; r < R; r += kThreads) off[r] = min(max(a.lengths[r], 0), cap);
    __syncthreads();
    auto capped = [cap](int x, int y) { return min(x + y, cap); };
    {
        int sum = 0;
        for (int r = r0; r < r1; ++r) sum = capped(sum, off[r]);
        int total;
        int at = block_scan(sum, reinterpret_cast<int*>(warp_sum), total, capped);
        for (int r = r0; r < r1; ++r) {
            const int n = off[r];
            off[r] = at;
            at = capped(at, n);
        }
        if (tid == 0) off[R] = total;
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
    int* slot = smem + PlanLayout::pad(static_cast<size_t>(R) + 1);   // [R]
    int* owner = a.plan + a.lay.owner();
    int* p_off = a.plan + a.lay.offsets();
    const int c0 = min(max(*a.free_count, 0), S);
    // claims: clear what may be claimed, then the lowest request that names a slot
    for (int r = tid; r < R; r += kThreads) {
        const int s = a.slots[r];
        slot[r] = s;
        p_off[r] = off[r];
        if (s >= 0 && s < S) owner[s] = INT_MAX;
        if (r < c0) {
            const int f = a.free_slots[c0 - 1 - r];
            if (f >= 0 && f < S) owner[f] = INT_MAX;
        }
    }
    if (tid == 0) p_off[R] = off[R];
    __syncthreads();
    for (int r = tid; r < R; r += kThreads) {
        const int s = slot[r];
        if (s >= 0 && s < S) atomicMin(&owner[s], r);
    }
    __syncthreads();
    // per request: ends (gives its slot back), needs one, or neither
    auto fits = [&](int r) { return off[r + 1] <= rows; };
    auto mine = [&](int r) { return slot[r] >= 0 && slot[r] < S && __ldcg(&owner[slot[r]]) == r; };
    auto ends = [&](int r) { return a.lengths[r] < 0 && mine(r); };
    auto needs = [&](int r) { return a.lengths[r] > 0 && slot[r] == -1 && a.seen[r] == 0 && fits(r); };
    unsigned long long cnt = 0;   // needs << 32 | ends
    int bad = 0;
    for (int r = r0; r < r1; ++r) {
        const int s = slot[r], n = a.lengths[r];
        if (ends(r)) cnt += 1;
        if (needs(r)) cnt += 1ull << 32;
        if (n > 0 && !fits(r)) bad |= kFaultRows;
        if (s >= S || s < -1) bad |= kFaultSlot;
        if (s >= 0 && s < S && !mine(r)) bad |= kFaultOwner;
        if (n > 0 && s == -1 && a.seen[r] != 0) bad |= kFaultState;
    }
    unsigned long long total;
    unsigned long long at = block_scan(cnt, warp_sum, total, [](unsigned long long x, unsigned long long y) { return x + y; });
    const int n_ends = static_cast<int>(total & 0xffffffffu);
    const int c1 = min(c0 + n_ends, S);
    if (tid == 0 && c0 + n_ends > S) bad |= kFaultOverflow;
    {
        int e = static_cast<int>(at & 0xffffffffu);
        for (int r = r0; r < r1; ++r)
            if (ends(r)) {
                const int s = slot[r];
                if (c0 + e < S) a.free_slots[c0 + e] = s;
                ++e;
                slot[r] = kEnded;
            }
    }
    __syncthreads();   // every mine() above has read the claims
    for (int r = r0; r < r1; ++r)   // slots given back may be taken again below
        if (slot[r] == kEnded && a.slots[r] >= 0) owner[a.slots[r]] = INT_MAX;
    __syncthreads();
    int taken = 0;
    {
        int w = static_cast<int>(at >> 32);
        for (int r = r0; r < r1; ++r)
            if (needs(r)) {
                const int i = c1 - 1 - w++;
                if (i >= 0) {
                    const int s = a.free_slots[i];
                    ++taken;
                    if (s >= 0 && s < S) {
                        atomicMin(&owner[s], kPopped + r);
                        slot[r] = s;
                    } else {
                        bad |= kFaultSlot;
                    }
                } else {
                    bad |= kFaultFree;
                }
            }
    }
    __syncthreads();
    // ---- slots out, who takes part, the sort's histogram ----------------------------
    int part = 0;
    for (int i = tid; i < kWarps * 32; i += kThreads) hist[i] = 0;
    __syncthreads();
    const int per_warp = (R + kThreads - 1) / kThreads * 32;   // consecutive requests of a warp
    const int w0 = min(warp * per_warp, R), w1 = min(w0 + per_warp, R);
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int r = t0 + lane;
        int key = 0;
        if (r < w1) {
            const int given = a.slots[r], n = a.lengths[r];
            int now = slot[r];
            bool ok = false;
            if (now == kEnded && given >= 0) {
                now = -1;
            } else if (now != given) {               // taken from the free stack
                ok = __ldcg(&owner[now]) == kPopped + r;
                if (!ok) {
                    bad |= kFaultOwner;
                    now = -1;
                }
            } else if (n > 0 && now >= 0 && now < S) {
                ok = __ldcg(&owner[now]) == r && fits(r);
            }
            a.slots[r] = now;
            a.plan[a.lay.slots() + r] = ok ? now : -1;
            if (ok) {
                key = 32 - __clz((n + kBlock - 1) / kBlock);
                ++part;
            }
            slot[r] = key;   // the slot numbers are written: the keys take their place
        }
        const unsigned peers = __match_any_sync(0xffffffffu, r < w1 ? key : kKeys + 1);
        if (r < w1 && __popc(peers & ((1u << lane) - 1)) == 0) hist[warp * 32 + key] += __popc(peers);
        __syncwarp();
    }
    const int any = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad));
    if (lane == 0 && any) atomicOr(&faults, any);
    unsigned long long sums = block_scan(
        (static_cast<unsigned long long>(part) << 32) | static_cast<unsigned>(taken), warp_sum, total,
        [](unsigned long long x, unsigned long long y) { return x + y; });
    (void)sums;
    if (tid == 0) {
        a.plan[0] = min(off[R], rows);
        a.plan[1] = static_cast<int>(total >> 32);
        a.plan[2] = c1 - static_cast<int>(total & 0xffffffffu);
        a.plan[3] = faults;
        a.plan[4] = R;
        a.plan[5] = rows;
        *a.free_count = c1 - static_cast<int>(total & 0xffffffffu);
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
    for (int t0 = w0; t0 < w1; t0 += 32) {
        const int r = t0 + lane;
        const int key = r < w1 ? slot[r] : kKeys + 1;
        const unsigned peers = __match_any_sync(0xffffffffu, key);
        const int rank = __popc(peers & ((1u << lane) - 1));
        const int base = r < w1 ? hist[warp * 32 + key] : 0;
        __syncwarp();
        if (r < w1) {
            const int use = a.plan[a.lay.slots() + r];   // this thread's own, from above
            a.plan[a.lay.order() + base + rank] = r;
            reinterpret_cast<int4*>(a.plan + a.lay.items())[base + rank] =
                make_int4(off[r], use >= 0 ? a.lengths[r] : 0, use, a.seen[r]);
            if (rank == 0) hist[warp * 32 + key] = base + __popc(peers);
        }
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
    const size_t smem = (PlanLayout::pad(static_cast<size_t>(a.requests) + 1) + PlanLayout::pad(a.requests)) * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((2 * (kMaxRequests + 8)) * sizeof(int)));
    if (e != cudaSuccess) return e;
    const unsigned grid = 1 + (a.rows + kRowsPerCta - 1) / kRowsPerCta;
    return launch_pdl(plan_kernel, grid, kThreads, smem, s, a);
}

}  // namespace packed
}  // namespace la

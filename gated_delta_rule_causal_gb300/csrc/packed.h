// Internal interface of the packed gated delta rule: requests of different
// lengths behind each other in token-major tensors, states in a pool of slots
// (C ABI in packed_api.cu, kernels in packed_plan.cu, packed_chunk.cu and
// packed_step.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace la {
namespace packed {

constexpr int kBlock = 32;            // tokens per block of the chunkwise form
constexpr int kMaxRequests = 16384;   // the plan kernel keeps the offsets of all requests in shared memory
constexpr int kMaxTokens = 1 << 24;

// Words (int32) of a plan, each section padded to four words:
//   counts[8]            0 rows used, 1 requests taking part, 2 free slots left, 3 faults,
//                        4 requests, 5 rows given (the last two for the kernels that read the plan)
//   offsets[R + 1]       first row of every request (rows + 1 where it lies past the rows given)
//   slots[R]             state slot of a request that takes part, else -1
//   order[R]             requests, most blocks first (to a power of two), those without a part last
//   seen[R]              tokens a request had absorbed before
//   token_request[N], token_position[N]
//   owner[S]             scratch: which request claims a slot
struct PlanLayout {
    int R, N, S;
    __host__ __device__ static size_t pad(size_t n) { return (n + 3) / 4 * 4; }
    __host__ __device__ size_t offsets() const { return 8; }
    __host__ __device__ size_t slots() const { return offsets() + pad(static_cast<size_t>(R) + 1); }
    __host__ __device__ size_t order() const { return slots() + pad(R); }
    __host__ __device__ size_t seen() const { return order() + pad(R); }
    __host__ __device__ size_t token_request() const { return seen() + pad(R); }
    __host__ __device__ size_t token_position() const { return token_request() + pad(N); }
    __host__ __device__ size_t owner() const { return token_position() + pad(N); }
    __host__ __device__ size_t words() const { return owner() + pad(S); }
};

// Faults a plan reports (counts[3]); the requests concerned take no part.
enum : int {
    kFaultRows = 1,      // rows past the rows given
    kFaultFree = 2,      // no free slot for a new request
    kFaultSlot = 4,      // a slot number outside the pool
    kFaultOwner = 8,     // a slot claimed twice
    kFaultState = 16,    // a request that has seen tokens but has no slot
    kFaultOverflow = 32, // more slots given back than the pool has
};

struct PlanArgs {
    const int* lengths;   // [R] tokens of this step; negative: ended, gives its slot back
    const int* seen;      // [R]
    int* slots;           // [R] in and out
    int* free_slots;      // [S] stack of free slots, in and out
    int* free_count;      // [1] in and out
    int* plan;
    PlanLayout lay;       // of the handle's maxima
    int requests, rows;   // of this step
};
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s);

struct StepArgs {
    const int* plan;
    PlanLayout lay;
    const void* q;        // [rows][Hk][dk], rows q_stride elements apart
    const void* k;
    const void* v;        // [rows][Hv][dv]
    const float* gate;    // [rows][Hv]
    const float* beta;    // [rows][Hv]
    float* states;        // [S][Hv][dv][dk]
    void* out;            // [rows][Hv][dv], contiguous
    long long q_stride, k_stride, v_stride;   // elements
    int requests, rows;
    int Hk, Hv, dk, dv;
    int io;               // Io
    int sm_count;
    int* status;
};
// Token by token, CUDA cores: any supported head size and type.
cudaError_t launch_step(const StepArgs& a, cudaStream_t s);
// In blocks of 32 tokens, warp-level MMAs: bf16, dk and dv in {64, 128}.
cudaError_t launch_chunk(const StepArgs& a, cudaStream_t s, PFN_cuTensorMapEncodeTiled_v12000 enc);

// The requests of a plan as the kernels read them, every word checked against
// what the tensors hold, so that a plan of other sizes or a buffer that no
// plan was made in reaches no memory outside them.
struct Request {
    int row0, len, slot;
    bool fresh;   // no token seen: the state starts at zero
};
__device__ __forceinline__ bool read_request(const StepArgs& a, int r, Request& x) {
    const int* p = a.plan;
    const int lo = p[a.lay.offsets() + r], hi = p[a.lay.offsets() + r + 1];
    x.slot = p[a.lay.slots() + r];
    x.fresh = p[a.lay.seen() + r] <= 0;
    x.row0 = lo;
    x.len = hi - lo;
    return x.slot >= 0 && x.slot < a.lay.S && lo >= 0 && hi > lo && hi <= a.rows;
}
// Requests of the plan that this call may walk.
__device__ __forceinline__ int plan_requests(const StepArgs& a) {
    const int n = a.plan[4];
    return n < a.requests ? n : a.requests;
}

}  // namespace packed
}  // namespace la

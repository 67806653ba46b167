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

constexpr int kBlock = 32;            // tokens per block that a plan orders its requests by
constexpr int kMaxRequests = 16384;   // the plan kernel keeps the offsets of all requests in shared memory
constexpr int kMaxTokens = 1 << 24;

// Words (int32) of a plan, each section padded to four words:
//   counts[8]            0 rows used, 1 requests taking part, 2 free slots left, 3 faults,
//                        4 requests, 5 rows given (the last two for the kernels that read the plan)
//   offsets[R + 1]       first row of every request (rows + 1 where it lies past the rows given)
//   slots[R]             state slot of a request that takes part, else -1
//   order[R]             requests, most blocks first (to a power of two), those without a part last
//   items[R][4]          the requests in that order: first row, length, slot (-1: no part), tokens seen before
//   token_request[N], token_position[N]
//   owner[S]             scratch: which request claims a slot
struct PlanLayout {
    int R, N, S;
    __host__ __device__ static size_t pad(size_t n) { return (n + 3) / 4 * 4; }
    __host__ __device__ size_t offsets() const { return 8; }
    __host__ __device__ size_t slots() const { return offsets() + pad(static_cast<size_t>(R) + 1); }
    __host__ __device__ size_t order() const { return slots() + pad(R); }
    __host__ __device__ size_t items() const { return order() + pad(R); }
    __host__ __device__ size_t token_request() const { return items() + 4 * static_cast<size_t>(R); }
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
    int above, upto;      // only requests of above < tokens <= upto
};
// Token by token, CUDA cores: any supported head size and type.
cudaError_t launch_step(const StepArgs& a, cudaStream_t s);
// The same beside the blockwise launch before it on the stream, which takes the step's other requests (bf16, dk in
// {64, 128}).
cudaError_t launch_step_beside(const StepArgs& a, cudaStream_t s);
// Whether every CTA of 32 state rows would have an SM to itself.
inline bool chunk_is_alone(int requests, int Hv, int dv, int sm_count) {
    return static_cast<long long>(requests) * Hv * (dv / 32) <= sm_count;
}
// In blocks of 32 tokens, warp-level MMAs: bf16, dk and dv in {64, 128}.
cudaError_t launch_chunk(const StepArgs& a, cudaStream_t s, PFN_cuTensorMapEncodeTiled_v12000 enc);
// In blocks of 64 tokens on the tcgen05 tensor cores: bf16, dk in {64, 128}, dv 128.
cudaError_t launch_tc(const StepArgs& a, cudaStream_t s, PFN_cuTensorMapEncodeTiled_v12000 enc);

// 3-D map over a packed tensor [rows][H][d], rows `stride` elements apart:
// boxes of `block` rows of one head's 64 channels, 128-byte swizzle. Rows past
// the tensor read as zeros.
inline bool make_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* base, int d, int H, int rows,
              long long stride, int block) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(block)};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


// The rank-th request of a plan as the kernels read it, every word checked
// against what the tensors hold, so that a plan of other sizes or a buffer
// that no plan was made in reaches no memory outside them.
struct Request {
    int row0, len, slot;
    bool fresh;   // no token seen: the state starts at zero
};
template <bool PAST = false>   // past the SM's own cache
__device__ __forceinline__ bool read_request(const StepArgs& a, int rank, Request& x) {
    const int* count = a.plan + 4;
    const int4* item = reinterpret_cast<const int4*>(a.plan + a.lay.items()) + rank;
    const int n = PAST ? __ldcg(count) : *count;
    const int4 w = PAST ? __ldcg(item) : *item;
    x.row0 = w.x;
    x.len = w.y;
    x.slot = w.z;
    x.fresh = w.w == 0;
    return rank < n && x.slot >= 0 && x.slot < a.lay.S && x.len > 0 && x.len <= a.rows && x.row0 >= 0 &&
           x.row0 <= a.rows - x.len && x.len > a.above && x.len <= a.upto;
}

}  // namespace packed
}  // namespace la

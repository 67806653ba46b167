// C ABI of the packed gated delta rule (declared in include/la.h): argument
// validation and kernel selection. The handle holds the configuration and one
// device status word; plans, states and tensors are the caller's.
#include <cstdint>
#include <cstdio>
#include <new>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/la.h"
#include "host.h"
#include "kernels.h"
#include "packed.h"

struct la_packed {
    la_packed_config cfg;
    la::packed::PlanLayout lay;
    int sm_count;
    int* d_status;
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    char last_error[256];
    int last_launches;
};

namespace {

using la::aligned16;
using la::DeviceGuard;
using la::supported_d;
using la::packed::PlanLayout;
using la::packed::StepArgs;

int fail(la_packed* h, int code, const char* msg) {
    std::snprintf(h->last_error, sizeof(h->last_error), "%s", msg);
    return code;
}
int fail_for(la_packed* h, int code, const char* name, const char* msg) {
    std::snprintf(h->last_error, sizeof(h->last_error), "%s %s", name, msg);
    return code;
}
int cuda_fail(la_packed* h, cudaError_t e, const char* what) {
    std::snprintf(h->last_error, sizeof(h->last_error), "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return LA_ERR_CUDA;
}

// What a configuration has to satisfy; LA_OK or the error.
int check_config(const la_packed_config* c) {
    if (!c) return LA_ERR_INVALID_ARG;
    if (c->max_requests < 1 || c->max_tokens < 1 || c->slots < 1 || c->H_k < 1 || c->H_v < 1) return LA_ERR_INVALID_ARG;
    if (c->H_v % c->H_k) return LA_ERR_INVALID_ARG;
    if (c->io != LA_BF16 && c->io != LA_FP32) return LA_ERR_INVALID_ARG;
    if (c->flags) return LA_ERR_INVALID_ARG;
    if (!supported_d(c->d_k) || !supported_d(c->d_v)) return LA_ERR_UNSUPPORTED;
    if (c->max_requests > la::packed::kMaxRequests || c->max_tokens > la::packed::kMaxTokens) return LA_ERR_UNSUPPORTED;
    if (c->slots > (1 << 28) || c->H_v > 4096) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Whether a step at d_v 128 takes blocks of 64 tokens on the tcgen05 tensor cores (packed_tc.cu, one CTA per SM)
// instead of blocks of 32 by warp-level MMAs (packed_chunk.cu, two or four CTAs per head). The former starts later and
// has the higher throughput; the latter waits less between the steps of one request. Measured, 32 / 64:
//   few heads (every CTA of 32 state rows has an SM), d_k 128: 16 of 64 rows 6.5 / 10.6 us, of 8192 320 / 422; 32 of
//            16384 (two requests) 363 / 426; d_k 64: 16 of 64 5.5 / 9.3, of 8192 256 / 383
//   d_k 128, 32 requests, 16 heads: 256 rows 29.0 / 31.2, 512 33.2 / 31.5, 4096 120 / 100
//   d_k 64, 64 requests, 16 heads: 4096 rows 53 / 56, 8192 78 / 77, 32768 235 / 208; 16 requests of one length,
//           16 heads: 8192 67 / 61, 32768 258 / 211
bool blocks_of_64(const la_packed* h, int requests, int tokens) {
    if (h->cfg.d_v != 128 || la::packed::chunk_is_alone(requests, h->cfg.H_v, 128, h->sm_count)) return false;
    if (h->cfg.d_k == 128) return tokens > 256;
    return static_cast<long long>(tokens) * h->cfg.H_v >= 1 << 17 && static_cast<long long>(requests) * h->cfg.H_v >= h->sm_count;
}

// Requests of up to so many tokens run token by token beside the others' blocks. Measured, us, 16 heads of 128, every
// third request new, beside / all in blocks: 64 requests of one token 21 / 52, of four 35 / 52; 256 of one 87 / 198, of
// four 151 / 198; one prompt of 1800 and 255 single tokens 130 / 206, and 63 single tokens 107 / 106, eight of 500 and 56
// single tokens 57 / 73; 64 prompts of 600: 287 / 287, the second launch finds nothing to do.
constexpr int kShort = 4;

int run_step(la_packed* h, const int* plan, const void* q, const void* k, const void* v, const float* gate,
             const float* beta, float* states, void* out, int requests, int tokens, long long q_stride,
             long long k_stride, long long v_stride, int chunk, void* cuda_stream) {
    if (!h) return LA_ERR_INVALID_ARG;
    h->last_error[0] = 0;
    h->last_launches = 0;
    const la_packed_config& c = h->cfg;
    if (requests < 0 || tokens < 0) return fail(h, LA_ERR_INVALID_ARG, "requests and tokens must be >= 0");
    if (requests > c.max_requests || tokens > c.max_tokens)
        return fail(h, LA_ERR_INVALID_ARG, "requests or tokens above the handle's maxima");
    if (chunk != 0 && chunk != 1 && chunk != 32 && chunk != 64)
        return fail(h, LA_ERR_UNSUPPORTED, "chunk must be 0 (default), 1 (recurrent), 32 or 64");
    const bool blocks_ok = c.io == LA_BF16 && c.d_k >= 64 && c.d_v >= 64;
    if (chunk >= 32 && !blocks_ok)
        return fail(h, LA_ERR_UNSUPPORTED, "chunk 32 and 64 need bf16 io and d_k, d_v in {64, 128}");
    if (chunk == 64 && c.d_v != 128) return fail(h, LA_ERR_UNSUPPORTED, "chunk 64 needs d_v 128");
    const int form = chunk ? chunk : !blocks_ok ? 1 : blocks_of_64(h, requests, tokens) ? 64 : 32;
    if (requests == 0 || tokens == 0) return LA_OK;
    const void* ptrs[] = {plan, q, k, v, gate, beta, states, out};
    const char* names[] = {"plan", "q", "k", "v", "gate", "beta", "states", "out"};
    for (int i = 0; i < 8; ++i) {
        if (!ptrs[i]) return fail_for(h, LA_ERR_INVALID_ARG, names[i], "is required");
        const bool scalars = i == 4 || i == 5;   // gate, beta: read one by one, so any row of them may come first
        if (scalars ? (reinterpret_cast<uintptr_t>(ptrs[i]) & 3u) != 0 : !aligned16(ptrs[i]))
            return fail_for(h, LA_ERR_MISALIGNED, names[i], scalars ? "is not 4-byte aligned" : "is not 16-byte aligned");
    }
    const long long es = c.io == LA_BF16 ? 2 : 4;
    const long long strides[] = {q_stride, k_stride, v_stride};
    const long long least[] = {static_cast<long long>(c.H_k) * c.d_k, static_cast<long long>(c.H_k) * c.d_k,
                               static_cast<long long>(c.H_v) * c.d_v};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < least[i]) return fail_for(h, LA_ERR_INVALID_ARG, names[1 + i], "has rows that overlap");
        if (strides[i] > (1LL << 32)) return fail_for(h, LA_ERR_UNSUPPORTED, names[1 + i], "has rows too far apart");
        if (strides[i] * es % 16) return fail_for(h, LA_ERR_MISALIGNED, names[1 + i], "has rows that are not 16-byte aligned");
    }
    StepArgs a;
    a.plan = plan;
    a.lay = h->lay;
    a.q = q;
    a.k = k;
    a.v = v;
    a.gate = gate;
    a.beta = beta;
    a.states = states;
    a.out = out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.requests = requests;
    a.rows = tokens;
    a.Hk = c.H_k;
    a.Hv = c.H_v;
    a.dk = c.d_k;
    a.dv = c.d_v;
    a.io = c.io == LA_FP32 ? la::kFp32 : la::kBf16;
    a.sm_count = h->sm_count;
    a.status = h->d_status;
    DeviceGuard g(c.device);
    if (!g.ok) return fail(h, LA_ERR_CUDA, "cannot select the handle's device");
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    // By default the requests of a few tokens run token by token in a launch of their own beside the others' blocks,
    // where there are more (request, head) pairs than SMs (else each pair has an SM at once, and a launch costs more).
    const bool split = chunk == 0 && form != 1 && requests > 1 && static_cast<long long>(requests) * c.H_v > h->sm_count;
    a.above = split ? kShort : 0;
    a.upto = 0x7fffffff;
    cudaError_t e = form == 1    ? la::packed::launch_step(a, s)
                    : form == 32 ? la::packed::launch_chunk(a, s, h->encode)
                                 : la::packed::launch_tc(a, s, h->encode);
    if (e != cudaSuccess) return cuda_fail(h, e, form == 1 ? "packed step launch" : "packed prefill launch");
    h->last_launches = 1;
    if (split) {
        a.above = 0;
        a.upto = kShort;
        e = la::packed::launch_step_beside(a, s);
        if (e != cudaSuccess) return cuda_fail(h, e, "packed step launch");
        h->last_launches = 2;
    }
    return LA_OK;
}

}  // namespace

extern "C" {

long long la_packed_plan_words(const la_packed_config* cfg) {
    if (check_config(cfg) != LA_OK) return 0;
    return static_cast<long long>(PlanLayout{cfg->max_requests, cfg->max_tokens, cfg->slots}.words());
}

int la_packed_create(const la_packed_config* cfg, la_packed** out) {
    if (!out) return LA_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = check_config(cfg);
    if (rc != LA_OK) return rc;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    if (cfg->device < 0 || cfg->device >= ndev) return LA_ERR_INVALID_ARG;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, cfg->device) != cudaSuccess) return LA_ERR_CUDA;
    if (!(prop.major == 10 && prop.minor == 3)) return LA_ERR_UNSUPPORTED;   // built for sm_103a only
    la_packed* h = new (std::nothrow) la_packed();
    if (!h) return LA_ERR_CUDA;
    h->cfg = *cfg;
    h->lay = PlanLayout{cfg->max_requests, cfg->max_tokens, cfg->slots};
    h->sm_count = prop.multiProcessorCount;
    h->d_status = nullptr;
    h->last_launches = 0;
    h->last_error[0] = 0;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    DeviceGuard g(cfg->device);
    if (!g.ok || cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn || cudaMalloc(&h->d_status, sizeof(int)) != cudaSuccess ||
        cudaMemset(h->d_status, 0, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        if (h->d_status) cudaFree(h->d_status);
        delete h;
        return LA_ERR_CUDA;
    }
    h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    *out = h;
    return LA_OK;
}

void la_packed_destroy(la_packed* h) {
    if (!h) return;
    {
        DeviceGuard g(h->cfg.device);
        if (h->d_status) cudaFree(h->d_status);
    }
    delete h;
}

int la_packed_plan(la_packed* h, const int* lengths, const int* seen, int* slots, int* free_slots, int* free_count,
                   int* plan, int requests, int tokens, void* cuda_stream) {
    if (!h) return LA_ERR_INVALID_ARG;
    h->last_error[0] = 0;
    h->last_launches = 0;
    const la_packed_config& c = h->cfg;
    if (requests < 0 || tokens < 0) return fail(h, LA_ERR_INVALID_ARG, "requests and tokens must be >= 0");
    if (requests > c.max_requests || tokens > c.max_tokens)
        return fail(h, LA_ERR_INVALID_ARG, "requests or tokens above the handle's maxima");
    const void* ptrs[] = {lengths, seen, slots, free_slots, free_count, plan};
    const char* names[] = {"lengths", "seen", "slots", "free_slots", "free_count", "plan"};
    for (int i = 0; i < 6; ++i) {
        if (!ptrs[i] && (i >= 3 || requests > 0)) return fail_for(h, LA_ERR_INVALID_ARG, names[i], "is required");
        if (reinterpret_cast<uintptr_t>(ptrs[i]) & 3u) return fail_for(h, LA_ERR_MISALIGNED, names[i], "is not 4-byte aligned");
    }
    if (!aligned16(plan)) return fail(h, LA_ERR_MISALIGNED, "plan is not 16-byte aligned");
    la::packed::PlanArgs a;
    a.lengths = lengths;
    a.seen = seen;
    a.slots = slots;
    a.free_slots = free_slots;
    a.free_count = free_count;
    a.plan = plan;
    a.lay = h->lay;
    a.requests = requests;
    a.rows = tokens;
    DeviceGuard g(c.device);
    if (!g.ok) return fail(h, LA_ERR_CUDA, "cannot select the handle's device");
    const cudaError_t e = la::packed::launch_plan(a, static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return cuda_fail(h, e, "plan launch");
    h->last_launches = 1;
    return LA_OK;
}

int la_packed_forward(la_packed* h, const int* plan, const void* q, const void* k, const void* v, const float* gate,
                      const float* beta, float* states, void* out, int requests, int tokens, long long q_stride,
                      long long k_stride, long long v_stride, int chunk, void* cuda_stream) {
    return run_step(h, plan, q, k, v, gate, beta, states, out, requests, tokens, q_stride, k_stride, v_stride, chunk,
                    cuda_stream);
}

int la_packed_decode_step(la_packed* h, const int* plan, const void* q, const void* k, const void* v,
                          const float* gate, const float* beta, float* states, void* out, int requests, int tokens,
                          long long q_stride, long long k_stride, long long v_stride, void* cuda_stream) {
    return run_step(h, plan, q, k, v, gate, beta, states, out, requests, tokens, q_stride, k_stride, v_stride, 1,
                    cuda_stream);
}

int la_packed_status(la_packed* h, void* cuda_stream) {
    if (!h) return LA_ERR_INVALID_ARG;
    DeviceGuard g(h->cfg.device);
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return cuda_fail(h, e, "stream synchronize");
    int word = 0;
    e = cudaMemcpy(&word, h->d_status, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(h, e, "status read");
    if (word != 0) {
        e = cudaMemset(h->d_status, 0, sizeof(int));
        if (e != cudaSuccess) return cuda_fail(h, e, "status clear");
        std::snprintf(h->last_error, sizeof(h->last_error),
                      "a bounded device wait expired (status bits 0x%x: 1=TMA, 2=MMA, 8=work items and V)", word);
        return LA_ERR_TIMEOUT;
    }
    return LA_OK;
}

const char* la_packed_last_error(const la_packed* h) { return h ? h->last_error : "null handle"; }

int la_packed_last_launches(const la_packed* h) { return h ? h->last_launches : 0; }

}  // extern "C"

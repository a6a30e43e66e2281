// internal.h -- what the translation units of libspecverify share on the host
// side: error text, launch counting, argument checks of strided tensors.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "spec_verify.h"

#define SV_HIDDEN __attribute__((visibility("hidden")))

namespace sv_host {

// Sets the calling thread's error detail and returns `st`.
SV_HIDDEN spec_status fail(spec_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// After a launch: the runtime's verdict, and one more in spec_launch_count().
SV_HIDDEN spec_status launched(const char* what);
SV_HIDDEN int num_sms();
// Polls of the first wait for copied bytes (spec_debug_wait_budget of the calling thread).
SV_HIDDEN unsigned wait_tries();
// NVTX range of one C-ABI call.
SV_HIDDEN void range_push(const char* name);
SV_HIDDEN void range_pop();

struct Range {
    explicit Range(const char* name) { range_push(name); }
    ~Range() { range_pop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

// Dynamic shared memory for a kernel on the current device, set once per device: `done` is a
// static of the caller, one for each kernel.
inline spec_status allow_smem(const void* kernel, const char* what, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (done.load(std::memory_order_acquire) & bit) != 0) return SPEC_OK;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return fail(SPEC_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    done.fetch_or(bit, std::memory_order_release);
    return SPEC_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// A [B, N, H, D] tensor with unit stride in D: byte strides of the other axes.
struct Rows {
    char* p;
    int64_t b, n, h;
};

inline spec_status make_rows(const char* what, const void* p, const int64_t* strides, int B, int N, int H, int esz,
                             Rows* out) {
    if (!p) return fail(SPEC_ERR_INVALID_ARG, "%s is NULL", what);
    if (!strides) return fail(SPEC_ERR_INVALID_ARG, "%s: strides are NULL", what);
    if (((uintptr_t)p & 15u) != 0) return fail(SPEC_ERR_INVALID_ARG, "%s: base pointer not 16-byte aligned", what);
    const int dims[3] = {B, N, H};
    int64_t s[3];
    for (int i = 0; i < 3; ++i) {           // the stride of an axis of size 1 is never used
        s[i] = dims[i] > 1 ? strides[i] * esz : 0;
        if (s[i] % 16 != 0)
            return fail(SPEC_ERR_INVALID_ARG, "%s: stride %d * element size (%lld bytes) not a multiple of 16", what,
                        i, (long long)s[i]);
    }
    *out = Rows{static_cast<char*>(const_cast<void*>(p)), s[0], s[1], s[2]};
    return SPEC_OK;
}

// The workspace of the cache calls: the status word (the word that
// spec_read_device_status reads), an append's arrival counters (one per
// sequence; zero between calls), the attention's records of items that several CTAs
// share and their partial results (both written by every call before it reads them).  The counters lie at the same place for
// every shape, so that a workspace can serve calls of different sizes.
constexpr int ATT_MAX_CTAS = 1024;
constexpr int CACHE_MAX_B = 16384;
constexpr size_t CACHE_WS_STATUS = 0, CACHE_WS_SEQ = 256, CACHE_WS_CUT = CACHE_WS_SEQ + 4 * CACHE_MAX_B,
                 CACHE_WS_PARTIAL = CACHE_WS_CUT + 32 * ATT_MAX_CTAS;
static_assert(CACHE_WS_CUT == SPEC_CACHE_STATE_BYTES, "what has to be zero comes first");
SV_HIDDEN spec_status check_cache_ws(void* ws, size_t bytes, size_t need);
SV_HIDDEN spec_status check_cache(const spec_kv_cache* c, int B);

}  // namespace sv_host

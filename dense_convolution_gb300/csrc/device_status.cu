// The device status words and wait limits of the kernels' translation units, read
// and set as a whole.  One kernel fetches and clears all words, so a call makes one
// launch, one copy and one synchronisation however many units there are.
#include <atomic>

#include "internal.h"

namespace conv2d_gb300 {

namespace {

constexpr int kUnits = 7, kSlots = 64;
struct Words { uint32_t* at[kUnits]; };
__device__ uint32_t g_gathered[kSlots];    // a slot per call in flight

__global__ void gather_status_kernel(const Words w, int slot) {
    uint32_t all = 0;
    for (int i = 0; i < kUnits; ++i) all |= atomicExch(w.at[i], 0u);
    g_gathered[slot] = all;
}

}  // namespace

cudaError_t status_read_clear(cudaStream_t st, uint32_t* out) {
    static std::atomic<unsigned> calls{0};
    cudaError_t (*const word[])(void**) = {status_word_tc, status_word_fp32, status_word_wg,
                                                 status_word_ce, status_word_ln,   status_word_lp,
                                                 status_word_ffn};
    static_assert(sizeof(word) / sizeof(*word) == kUnits, "a unit is missing");
    Words w;
    for (int i = 0; i < kUnits; ++i) {
        void* p = nullptr;
        const cudaError_t e = word[i](&p);
        if (e != cudaSuccess) return e;
        w.at[i] = static_cast<uint32_t*>(p);
    }
    const int slot = (int)(calls.fetch_add(1, std::memory_order_relaxed) % kSlots);
    gather_status_kernel<<<1, 1, 0, st>>>(w, slot);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbolAsync(out, g_gathered, sizeof(*out), slot * sizeof(*out), cudaMemcpyDeviceToHost, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

cudaError_t wait_limit_set(cudaStream_t st, uint64_t ns) {
    cudaError_t (*const set[])(cudaStream_t, uint64_t) = {wait_limit_set_tc, wait_limit_set_fp32, wait_limit_set_wg,
                                                                wait_limit_set_ce, wait_limit_set_ln,   wait_limit_set_lp,
                                                                wait_limit_set_ffn};
    static_assert(sizeof(set) / sizeof(*set) == kUnits, "a unit is missing");
    for (int i = 0; i < kUnits; ++i) {
        const cudaError_t e = set[i](st, ns);
        if (e != cudaSuccess) return e;
    }
    return cudaStreamSynchronize(st);
}

}  // namespace conv2d_gb300

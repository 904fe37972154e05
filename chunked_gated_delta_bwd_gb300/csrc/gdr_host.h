// Host helpers shared by the translation units that define the C ABI: the error string,
// argument checks and the optional event timing (gdr_profile_begin / gdr_profile_end).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {

// Record the message of gdr_last_error (thread-local) and return the status.
gdr_status fail(gdr_status s, const char* fmt, const char* what = "");
gdr_status cuda_fail(cudaError_t e, const char* where);
gdr_status ok();  // clears the message

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

#define NEED(ptr)                                                                    \
    do {                                                                             \
        if (!(ptr)) return fail(GDR_ERR_INVALID, "required pointer %s is NULL", #ptr); \
        if (!aligned16(ptr)) return fail(GDR_ERR_INVALID, "pointer %s is not 16-byte aligned", #ptr); \
    } while (0)
#define OPT(ptr)                                                                     \
    do {                                                                             \
        if ((ptr) && !aligned16(ptr)) return fail(GDR_ERR_INVALID, "pointer %s is not 16-byte aligned", #ptr); \
    } while (0)

// Event timing of the launches (off unless gdr_profile_begin was called).
struct Prof {
    bool on = false;
    int max_launches = 0, n = 0;
    cudaEvent_t* ev = nullptr;  // 2 per timed section
    int* kind = nullptr;
    int* kernels = nullptr;     // kernels launched in each timed section
};
extern Prof g_prof;

// Launches `f` (which launches `kernels` kernels) between two recorded events when
// profiling is on.
template <class F>
cudaError_t timed(int kind, cudaStream_t s, F&& f, int kernels = 1) {
    if (!g_prof.on || g_prof.n >= g_prof.max_launches) return f();
    const int i = g_prof.n++;
    g_prof.kind[i] = kind;
    g_prof.kernels[i] = kernels;
    cudaEventRecord(g_prof.ev[2 * i], s);
    cudaError_t e = f();
    cudaEventRecord(g_prof.ev[2 * i + 1], s);
    return e;
}

}  // namespace gdr

// launch.hpp -- host-side launch, timing and argument helpers that every
// translation unit of the library shares.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <mutex>
#include <vector>

#include "rs.h"
#include "rs_prof.h"

namespace rs_host {

// ---------------------------------------------------------------------------
// Per-kernel event timing (rs_prof.h).
// ---------------------------------------------------------------------------
struct ProfRecord {
    int kind;
    int sub;  // pass index of a pass launch, else -1
    hipEvent_t start;
    hipEvent_t stop;
};

struct ProfSample {
    int sub;
    double ms;
};

struct Prof {
    bool on = false;
    std::mutex mu;
    std::vector<ProfRecord> pending;
    std::vector<hipEvent_t> spare;
    uint64_t launches[RS_KERNEL_KINDS] = {};
    double ms[RS_KERNEL_KINDS] = {};
    std::vector<ProfSample> samples[RS_KERNEL_KINDS];
};

inline Prof &prof() {
    static Prof p;
    return p;
}

inline hipEvent_t take_event(Prof &p) {
    if (!p.spare.empty()) {
        hipEvent_t e = p.spare.back();
        p.spare.pop_back();
        return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
}

// Timing events of the launch under way (set by launch_kernel while timing
// is on, else null).
inline thread_local hipEvent_t t_launch_start = nullptr;
inline thread_local hipEvent_t t_launch_stop = nullptr;

// Enqueues kernel<<<grid, block, 0, stream>>>(args...); while a launch is
// timed, the timing events are attached to the dispatch itself.
template <class... KArgs, class... Args>
void run_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t stream, Args... args) {
    if (t_launch_start != nullptr) {
        hipExtLaunchKernelGGL(kernel, grid, block, 0, stream, t_launch_start, t_launch_stop, 0,
                              static_cast<KArgs>(args)...);
    } else {
        kernel<<<grid, block, 0, stream>>>(static_cast<KArgs>(args)...);
    }
}

// Runs `launch` (which enqueues one kernel on `stream` with run_kernel) and
// reports whether the launch succeeded; times it while timing is on.  `sub`
// tags the record (the pass index of a pass launch).
template <class F>
bool launch_kernel(int kind, hipStream_t stream, F &&launch, int sub = -1) {
    Prof &p = prof();
    if (!p.on) {
        launch();
        return hipGetLastError() == hipSuccess;
    }
    std::lock_guard<std::mutex> lock(p.mu);
    hipEvent_t a = take_event(p);
    hipEvent_t b = take_event(p);
    // The launch attaches the pair to the kernel's dispatch (run_kernel):
    // they stamp the kernel's own start and end, as a profiler's trace does.
    // (A pair recorded around the launch added ~3.5 us per launch at 2^28.)
    if (a && b) {
        t_launch_start = a;
        t_launch_stop = b;
    }
    launch();
    t_launch_start = nullptr;
    t_launch_stop = nullptr;
    const bool ok = hipGetLastError() == hipSuccess;
    if (a && b) {
        p.pending.push_back({kind, sub, a, b});
    } else {
        if (a) p.spare.push_back(a);
        if (b) p.spare.push_back(b);
    }
    return ok;
}

inline unsigned grid_for(size_t work, unsigned per_block, unsigned max_grid) {
    size_t g = (work + per_block - 1) / per_block;
    if (g < 1) g = 1;
    if (g > max_grid) g = max_grid;
    return static_cast<unsigned>(g);
}

// ---------------------------------------------------------------------------
// Byte ranges of arguments.
// ---------------------------------------------------------------------------
struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Span span_of(const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + bytes};
}

inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// In/out pair: identical start (in place) or disjoint.
inline bool same_or_disjoint(Span a, Span b) { return a.lo == b.lo || !overlap(a, b); }

}  // namespace rs_host

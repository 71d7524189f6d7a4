// launch.hpp -- what the C ABI's source files share: kernel launches with their
// timing (rs_prof.h), and argument checks.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <mutex>
#include <type_traits>
#include <vector>

#include "elements.hpp"
#include "rs.h"
#include "rs_prof.h"

namespace rs {

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

}  // namespace rs

namespace {

using rs::Prof;
using rs::ProfSample;
using rs::prof;
using rs::take_event;

// Timing events of the launch under way (set by launch_kernel while timing
// is on, else null).
thread_local hipEvent_t t_launch_start = nullptr;
thread_local hipEvent_t t_launch_stop = nullptr;

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

[[maybe_unused]] unsigned grid_for(size_t work, unsigned per_block, unsigned max_grid) {
    size_t g = (work + per_block - 1) / per_block;
    if (g < 1) g = 1;
    if (g > max_grid) g = max_grid;
    return static_cast<unsigned>(g);
}

// ---------------------------------------------------------------------------
// Argument checks (host only, before any HIP call), and calls by type.
// ---------------------------------------------------------------------------
struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

[[maybe_unused]] Span span_of(const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + bytes};
}

[[maybe_unused]] bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

constexpr unsigned kMaxGrid = 1u << 20;  // workgroups; the kernels stride over the rest

[[maybe_unused]] int dtype_bytes(int dtype) {
    switch (dtype) {
        case RS_F32: return 4;
        case RS_F16:
        case RS_BF16: return 2;
        default: return 0;
    }
}

[[maybe_unused]] bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes that `count` rows of `width` elements span.
[[maybe_unused]] size_t span_bytes(size_t count, size_t width, size_t stride, size_t elem) {
    return count == 0 ? 0 : ((count - 1) * stride + width) * elem;
}

// A present, aligned array; or any pointer for an empty one.
[[maybe_unused]] bool good(const void *p, size_t count, size_t align) { return count == 0 || (p != nullptr && aligned(p, align)); }

constexpr size_t kMaxStride = size_t{1} << 40;

// Whether the rows of an array are addressable and, for an output, disjoint.
[[maybe_unused]] bool good_rows(const void *p, size_t count, int width, size_t stride, size_t elem, bool output) {
    if (!good(p, count, elem)) return false;
    if (count <= 1) return true;
    if (stride > kMaxStride || (count - 1) > (size_t{1} << 62) / ((stride + 1) * elem)) return false;
    return !output || stride >= static_cast<size_t>(width);
}

[[maybe_unused]] bool disjoint(const Span *spans, int outputs, int all) {
    for (int o = 0; o < outputs; ++o) {
        for (int i = o + 1; i < all; ++i) {
            if (spans[o].lo != spans[o].hi && spans[i].lo != spans[i].hi && overlap(spans[o], spans[i])) return false;
        }
    }
    return true;
}

template <int N>
using IntC = std::integral_constant<int, N>;

template <class F>
bool with_dtype(int dtype, F &&f) {
    switch (dtype) {
        case RS_F32: return f(float{});
        case RS_F16: return f(rs::f16{});
        default: return f(rs::bf16{});
    }
}

}  // namespace

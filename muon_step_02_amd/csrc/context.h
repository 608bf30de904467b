// The handle and the small host helpers that the entry points share
// (api.hip, api_inputs.hip).  Nothing here is part of the public ABI.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <vector>

#include "muon_internal.h"

struct TimedLaunch {
    int phase;
    hipEvent_t start, stop;
};

struct muon_context {
    int device = 0;
    float* scratch = nullptr;  // this device's copy of `scratch` (api.hip), device address
    int cus_per_xcd = 32;  // compute units per XCD (tile rounds)
    // second stream (default priority) for the Newton-Schulz launches of the
    // size classes other than the large one, forked from and joined back into
    // the caller's stream with two events
    hipStream_t side = nullptr;
    hipEvent_t fork = nullptr, join = nullptr;
    std::vector<char> table;  // host image of the descriptor table (reused)
    bool profiling = false;
    std::vector<TimedLaunch> timed;     // recorded since the last collect
    std::vector<hipEvent_t> event_pool;  // timing events ready for reuse
};

namespace muon {

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) == hipSuccess && prev != dev) {
            changed = hipSetDevice(dev) == hipSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) (void)hipSetDevice(prev);
    }
};

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool finite(float v) { return isfinite(v) != 0; }

inline size_t elem_bytes(int32_t dt) { return dt == MUON_BF16 ? 2 : 4; }
inline bool valid_dtype(int32_t dt) { return dt == MUON_F32 || dt == MUON_BF16; }

inline muon_status hip_status(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }

// `rows` rows of `width` bytes, `stride` bytes apart: what a call reads or
// writes of one tensor (owner: whose it is).
struct Rect {
    uintptr_t lo, hi;
    size_t width, stride;
    bool write;
    int owner;
};

inline Rect rect_of(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es, bool write, int owner) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Rect{b, b + (size_t)((rows - 1) * ld + cols) * es, (size_t)cols * es,
                (size_t)(rows > 1 ? ld : cols) * es, write, owner};
}

// Whether two ranges share bytes.  Column blocks of one buffer (the same row
// stride, disjoint columns) interleave without sharing any, and so does what
// lies between a tensor's rows.
inline bool collide(const Rect& a, const Rect& b) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    if (a.stride == b.stride) {
        const Rect& f = a.lo <= b.lo ? a : b;
        const Rect& s = a.lo <= b.lo ? b : a;
        const size_t d = (s.lo - f.lo) % f.stride;
        return d < f.width || d + s.width > f.stride;
    }
    if (a.width != a.stride && b.width != b.stride) return true;
    // one of them is one run of bytes: against the other's rows
    const Rect& run = a.width == a.stride ? a : b;
    const Rect& r = a.width == a.stride ? b : a;
    if (run.lo <= r.lo) return true;
    const size_t d = (run.lo - r.lo) % r.stride;
    const uintptr_t next = run.lo + (r.stride - d);  // the row behind run.lo
    return d < r.width || (next < run.hi && next < r.hi);
}

inline Rect run_of(const void* p, size_t bytes, bool write, int owner) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Rect{b, b + bytes, bytes, bytes, write, owner};
}

inline hipEvent_t take_event(muon_context* h) {
    if (!h->event_pool.empty()) {
        hipEvent_t e = h->event_pool.back();
        h->event_pool.pop_back();
        return e;
    }
    // timing only: no system-scope fence (its cache writeback would slow the
    // launches being timed); the host reads nothing but the timestamps
    hipEvent_t e = nullptr;
    if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
    return e;
}

// Runs `launch` (a callable returning hipError_t); when profiling, brackets it
// with two timing events on stream s.
template <class F>
hipError_t timed(muon_context* h, int phase, hipStream_t s, F&& launch) {
    if (!h->profiling) return launch();
    TimedLaunch t{phase, take_event(h), take_event(h)};
    if (!t.start || !t.stop) return hipErrorOutOfMemory;
    hipError_t e = hipEventRecord(t.start, s);
    if (e == hipSuccess) e = launch();
    if (e == hipSuccess) e = hipEventRecord(t.stop, s);
    h->timed.push_back(t);
    return e;
}

}  // namespace muon

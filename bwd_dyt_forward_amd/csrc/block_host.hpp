// block_host.hpp - argument checks shared by the block operators' entries.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "dyt.h"

namespace dytb {

inline bool dtype_ok(int d) { return d == DYT_F32 || d == DYT_BF16 || d == DYT_F16; }
inline int64_t dtype_size(int d) { return d == DYT_F32 ? 4 : 2; }

inline bool aligned(std::initializer_list<const void*> ps, int64_t a) {
    for (const void* p : ps)
        if ((uintptr_t)p % (uintptr_t)a) return false;
    return true;
}

// A row pitch of at least N whose last element's byte offset fits 63 bits.
inline bool pitch_ok(int64_t M, int64_t N, int64_t ld) {
    return ld >= N && (M <= 1 || ld <= (INT64_MAX / 8 - N) / (M - 1));
}

struct Range {
    const void* p;
    int64_t bytes;
};

inline bool meet(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// No output overlaps an input or another output.
inline bool disjoint(const Range* in, int n_in, const Range* out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return false;
    }
    return true;
}

inline int hip_status() { return hipGetLastError() == hipSuccess ? DYT_OK : DYT_ERR_HIP; }

}  // namespace dytb

// What the C-ABI checks of the pointers it is given, before anything is launched.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/wtconv.h"

namespace wtc {

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline size_t elem_bytes(int dtype) { return dtype == WTCONV_BF16 ? 2 : 4; }

struct Buf {
    const void* p;
    size_t bytes, align;
};

// No output overlaps an input or another output; everything is aligned to
// its element type. Absent buffers are null.
template <int NI, int NO>
bool buffers_ok(const Buf (&in)[NI], const Buf (&out)[NO]) {
    auto hit = [](const Buf& a, const Buf& b) {
        const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
        return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
    };
    for (const Buf& b : in)
        if (!aligned(b.p, b.align)) return false;
    for (int i = 0; i < NO; ++i) {
        if (!aligned(out[i].p, out[i].align)) return false;
        for (const Buf& b : in)
            if (hit(out[i], b)) return false;
        for (int j = 0; j < i; ++j)
            if (hit(out[i], out[j])) return false;
    }
    return true;
}

inline wtconv_status_t done(hipError_t err) { return err == hipSuccess ? WTCONV_OK : WTCONV_ERR_LAUNCH; }

}  // namespace wtc

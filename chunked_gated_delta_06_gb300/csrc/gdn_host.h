// gdn_host.h -- host helpers of the entry points: sub-allocation, alignment and overlap checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

constexpr size_t kAlign = 256;

// Sequential sub-allocator over a caller buffer; with base == nullptr it only counts.
struct Carver {
    char *base;
    size_t off = 0;
    explicit Carver(void *b) : base(static_cast<char *>(b)) {}
    template <typename T>
    T *take(size_t count) {
        off = (off + kAlign - 1) / kAlign * kAlign;
        T *p = base ? reinterpret_cast<T *>(base + off) : nullptr;
        off += count * sizeof(T);
        return p;
    }
    size_t used() const { return (off + kAlign - 1) / kAlign * kAlign; }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Bytes of a call's buffer.
struct Span {
    const void *at;
    size_t bytes;
    bool meets(const Span &x) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(x.at);
        return at && x.at && bytes && x.bytes && a < b + x.bytes && b < a + bytes;
    }
    bool same(const Span &x) const { return at == x.at && bytes == x.bytes; }
};

}  // namespace gdn

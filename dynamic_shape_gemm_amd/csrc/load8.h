// Reading eight bf16 values from rows of any alignment (device code).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace mkp {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Up to 8 consecutive bf16 values element by element (any alignment);
// missing elements read as zero; nothing is read when nvalid <= 0.
__device__ __forceinline__ u32x4 load8_elems(const uint16_t* p, int nvalid) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t lo = (2 * e < nvalid) ? (uint32_t)p[2 * e] : 0u;
        uint32_t hi = (2 * e + 1 < nvalid) ? (uint32_t)p[2 * e + 1] : 0u;
        w[e] = lo | (hi << 16);
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

// 8 consecutive bf16 values that are all inside the operand, from rows of
// any alignment: 4-byte words, shifted by 16 bits when the first value sits
// in the upper half of a word.  The words read never leave those holding
// the 8 values (so never a page beyond them).
__device__ __forceinline__ u32x4 load8_words(const uint16_t* p) {
    const uintptr_t a = (uintptr_t)p;
    const uint32_t* q = (const uint32_t*)(a & ~uintptr_t(3));
    if ((a & 2) == 0) return u32x4{q[0], q[1], q[2], q[3]};
    const uint32_t w0 = q[0], w1 = q[1], w2 = q[2], w3 = q[3], w4 = q[4];
    return u32x4{__builtin_amdgcn_alignbit(w1, w0, 16), __builtin_amdgcn_alignbit(w2, w1, 16),
                 __builtin_amdgcn_alignbit(w3, w2, 16), __builtin_amdgcn_alignbit(w4, w3, 16)};
}

// Up to 8 values: whole chunks by words, partial ones element by element.
__device__ __forceinline__ u32x4 load8_any(const uint16_t* p, int nvalid) {
    return nvalid >= 8 ? load8_words(p) : load8_elems(p, nvalid);
}

}  // namespace
}  // namespace mkp

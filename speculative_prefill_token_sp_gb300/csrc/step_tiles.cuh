// What the kernels for few query rows share (attend_step.cu, weights_step.cu): mma.sync, copies to a ring in shared memory, and codes
// as operands.
#pragma once

#include "attend_split.cuh"

#include <cuda_fp16.h>

namespace sp {
namespace {

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kBytes>
struct Chunk {
    uint32_t w[kBytes / 4];
};
template <int kBytes>
__device__ __forceinline__ Chunk<kBytes> read_chunk(const uint8_t* p) {
    Chunk<kBytes> c;
    if constexpr (kBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        c.w[0] = v.x; c.w[1] = v.y;
    }
    return c;
}

// Copies kBytes (16 or 4) to shared memory in the background; zeros where `there` is false.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
    const int size = there ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// The same with fp16 operands.
__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four codes as two pairs of fp16 (their values before the scale, exactly).
template <int kKind>
__device__ __forceinline__ void half_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (kKind == SP_CACHE_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    } else {
        // 0x6400 + (8 bits) is 1024 + those bits; with the sign bit flipped they are the code + 128
        const uint32_t u = w ^ 0x80808080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
    }
}

// A pair of bf16, times a power of two, as a pair of fp16.
__device__ __forceinline__ uint32_t half_of(uint32_t w, float scale) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xffff0000u) * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace
}  // namespace sp

// attn_common.cuh -- device helpers shared by the tensor-core attention kernels
// (prefill over a cached prefix, attention over a whole prompt): tensor copies,
// a non-blocking barrier test, packed binary32 arithmetic, 16-bit packing.
#pragma once

#include <cuda.h>

#include <cstring>
#include <type_traits>

#include "common.cuh"

namespace pa {

// Tensor copies without an L2 hint: a K/V tile is read again by the other
// query tiles of its sequence and, for a shared prefix, by other sequences.
__device__ inline void tma_load_2d_plain(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ inline void tma_load_3d_plain(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Non-blocking test of an mbarrier phase (the MMA issuer polls two
// conditions and must not sleep on either).
__device__ inline bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Packed pairs of binary32 (Blackwell f32x2 arithmetic): each half is
// rounded to nearest like the scalar instruction, two results per issue.
// (x0, x1) = (x0 * a0 + b0, x1 * a1 + b1)
__device__ __forceinline__ void fma2_rn(float& x0, float& x1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, a, b;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "fma.rn.f32x2 x, x, a, b;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// (x0, x1) += (y0, y1)
__device__ __forceinline__ void add2_rn(float& x0, float& x1, float y0, float y1) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}
// (x0, x1) -= (y0, y1)
__device__ __forceinline__ void sub2_rn(float& x0, float& x1, float y0, float y1) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "sub.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}

// Two 16-bit values in one 32-bit word, the first in the low half.
__device__ inline uint32_t pack_hi_halves(float a, float b) {
    // the high 16 bits of each binary32: bfloat16 truncation
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

template <typename T>
__device__ inline uint32_t pack_rn(float a, float b) {
    uint32_t w;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&w, &h, 4);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        memcpy(&w, &h, 4);
    }
    return w;
}

}  // namespace pa

// Building blocks shared by the layer operators' kernels (norm, convolution,
// selective scan): rows of up to four elements a lane through buffer descriptors,
// wave and workgroup sums, and the checks of their entry points.
//
// Every store is at most 8 bytes a lane, and no lane stores two adjacent
// 8-byte words in a row (the compiler would join them into a wider store).
#pragma once

#include "../../include/libgdn_layer.h"
#include "gdn_buffer.h"
#include "gdn_internal.h"

namespace gdn {

bool tracing();

inline bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline int dtype_bytes(int dt) { return dt == GDN_F32 ? 4 : dt == GDN_BF16 ? 2 : 1; }
// A launch has fewer than 2^32 threads (threads > 0; the product itself may pass 64 bits).
inline bool grid_ok(int64_t wgs, int64_t threads) { return wgs <= (((int64_t)1 << 32) - 1) / threads; }
inline bool io_dtype_ok(int dt) { return dt == GDN_F32 || dt == GDN_BF16; }

// ---------------------------------------------------------------------------
// VEC consecutive elements of a row, as floats.  Offsets are in elements from
// the descriptor's base; what lies behind the row reads as zero and is not
// stored.
// ---------------------------------------------------------------------------
template <typename T, int VEC>
__device__ __forceinline__ void row_load(rsrc_t r, uint32_t e, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = BufElem<T>::load(r, e * io_traits<T>::bytes, 0);
    } else if constexpr (VEC == 2 && sizeof(T) == 2) {
        const uint32_t v = bload32(r, e * 2, 0);
        x[0] = __uint_as_float(v << 16);
        x[1] = __uint_as_float(v & 0xffff0000u);
    } else if constexpr (VEC == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, e * 4, 0, 0);
        x[0] = __uint_as_float(v[0]);
        x[1] = __uint_as_float(v[1]);
    } else if constexpr (sizeof(T) == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, e * 2, 0, 0);
        x[0] = __uint_as_float(v[0] << 16);
        x[1] = __uint_as_float(v[0] & 0xffff0000u);
        x[2] = __uint_as_float(v[1] << 16);
        x[3] = __uint_as_float(v[1] & 0xffff0000u);
    } else {
        const u32x4 v = bload128(r, e * 4, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
    }
}

// two floats as bf16, in one instruction
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float float2v __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2v{a, b}, bf16x2));
}

__device__ __forceinline__ float swap_pair(float x) {      // the value of lane ^ 1
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xf, 0xf, false));
}

// All lanes of a pair (l, l ^ 1) take part, with adjacent offsets e.  Four
// fp32 values go out as two 8-byte stores that are 16 bytes apart: the lanes
// of a pair first swap halves.
template <typename T, int VEC>
__device__ __forceinline__ void row_store(rsrc_t r, uint32_t e, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        BufElem<T>::store(x[0], r, e * io_traits<T>::bytes, 0);
    } else if constexpr (VEC == 2 && sizeof(T) == 2) {
        bstore32(pack_bf16(x[0], x[1]), r, e * 2, 0);
    } else if constexpr (VEC == 2) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(x[0]), __float_as_uint(x[1])}, r, e * 4, 0, 0);
    } else if constexpr (sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, r, e * 2, 0, 0);
    } else {
        const bool odd = lane_id() & 1;
        const float r0 = swap_pair(odd ? x[0] : x[2]), r1 = swap_pair(odd ? x[1] : x[3]);
        const uint32_t at = odd ? e * 4 - 8 : e * 4;
        const float a0 = odd ? r0 : x[0], a1 = odd ? r1 : x[1];
        const float b0 = odd ? x[2] : r0, b1 = odd ? x[3] : r1;
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(a0), __float_as_uint(a1)}, r, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(b0), __float_as_uint(b1)}, r, at + 16, 0, 0);
    }
}

// A row whose element type is known at run time (weights: io type or fp32).
template <typename T, int VEC>
__device__ __forceinline__ void row_load_either(rsrc_t r, bool f32, uint32_t e, float (&x)[VEC]) {
    if (sizeof(T) == 4 || f32)
        row_load<float, VEC>(r, e, x);
    else
        row_load<T, VEC>(r, e, x);
}

// A workgroup barrier that orders LDS only: global loads in flight (the next
// chunk's rows) and stores stay in flight, which __syncthreads would wait for.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Sums and maxima over the lanes of a wave; every lane gets the result.  The
// order of the additions does not depend on anything but the lane numbers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
    return x;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) x = fmaxf(x, __shfl_xor(x, m, 64));
    return x;
}

}  // namespace gdn

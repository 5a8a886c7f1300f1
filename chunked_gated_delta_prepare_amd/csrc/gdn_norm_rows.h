// What the norms' kernels share: sums over the threads of a row, and a row's
// output in 8 bits with its scales, the reduction of the weights' gradients, and
// the checks of a problem.
#pragma once

#include "gdn_layer.h"

namespace gdn {

constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;      // 2^-126

// Sum over the TPR threads of a row, in every one of them.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *red) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TPR > 64) {
        constexpr int kW = TPR / 64;
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave_id() * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < kW; ++k) t += red[k * N + i];
            v[i] = t;
        }
    }
}

__device__ __forceinline__ uint32_t clamp_e4m3(float x) {
    // (a NaN passes)
    return __float_as_uint(x > kE4m3Max ? kE4m3Max : x < -kE4m3Max ? -kE4m3Max : x);
}

// v / scale as a division rounds it: the product with the reciprocal, and what that
// leaves over of v once more.  (bf16 rows and weights put many quotients at e4m3's
// halfway points exactly, where the product alone goes to either side; a division
// costs ten instructions.)  A scale of infinity leaves nothing over.
template <int VEC>
__device__ __forceinline__ void store_e4m3(rsrc_t r, uint32_t e, const float (&v)[VEC], float scale) {
    const float inv = 1.f / scale, back = scale <= 3.40282347e38f ? scale : 0.f;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float q = v[i] * inv;
        c[i] = __uint_as_float(clamp_e4m3(fmaf(fmaf(-q, back, v[i]), inv, q)));
    }
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    if constexpr (VEC == 4) {
        q = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], q, true);
        bstore32((uint32_t)q, r, e, 0);
    } else if constexpr (VEC == 2) {
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)q, r, e, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)q, r, e, 0, 0);
    }
}

// Weights and biases of a row's K vectors, `step` elements apart from e on, in the io
// type or fp32: all loads first, then their conversions (a choice of type at every
// vector would wait for each of them).
template <typename T, int VEC, int K>
__device__ __forceinline__ void load_affine_as(rsrc_t rw, rsrc_t rb, uint32_t e, uint32_t step, float (&w)[K][VEC], float (&b)[K][VEC]) {
    RawRow<T, VEC> x[K], y[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k].load(rw, e * sizeof(T), k * step * sizeof(T));
        y[k].load(rb, e * sizeof(T), k * step * sizeof(T));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k].get(w[k]);
        y[k].get(b[k]);
    }
}
template <typename IO, int VEC, int K>
__device__ __forceinline__ void load_affine(rsrc_t rw, rsrc_t rb, bool f32, uint32_t e, uint32_t step, float (&w)[K][VEC], float (&b)[K][VEC]) {
    if (sizeof(IO) == 4 || f32)
        load_affine_as<float, VEC, K>(rw, rb, e, step, w, b);
    else
        load_affine_as<IO, VEC, K>(rw, rb, e, step, w, b);
}

// Scales that a row of K vectors of VEC elements for each of TPR threads may have.
template <int VEC, int TPR, int K>
constexpr int kRowGroups = (TPR * VEC * K + 127) / 128;

// A row's values in e4m3 with one scale (group 0; amax is this thread's largest
// size) or one per 128 columns.  scales: the row's, written where live.  red
// has TPR / 64 places and gmax the row's groups, both free when this is called
// (all threads of the workgroup take part).
template <int VEC, int TPR, int K>
__device__ __forceinline__ void store_row_e4m3(rsrc_t ry, float *scales, bool live, int D, int group, float amax,
                                               const float (&y)[K][VEC], int tid, float *red, uint32_t *gmax) {
    constexpr int kMaxG = kRowGroups<VEC, TPR, K>;
    if (group == 0) {
        amax = lanes_max<64>(amax);
        if constexpr (TPR > 64) {
            __syncthreads();
            if (lane_id() == 0) red[wave_id()] = amax;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < TPR / 64; ++k) amax = fmaxf(amax, red[k]);
        }
        const float scale = fmaxf(amax / kE4m3Max, kTinyScale);
#pragma unroll
        for (int k = 0; k < K; ++k) store_e4m3<VEC>(ry, (k * TPR + tid) * VEC, y[k], scale);
        if (tid == 0 && live) scales[0] = scale;
        return;
    }
    const int ng = (D + 127) >> 7;
    if constexpr (VEC > 1) {
        // 128 columns are 32 (64) lanes of one vector index
        constexpr int kL = 128 / VEC;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(y[k][i]));
            m = lanes_max<kL>(m);
            const float scale = fmaxf(m / kE4m3Max, kTinyScale);
            store_e4m3<VEC>(ry, (k * TPR + tid) * VEC, y[k], scale);
            const int gi = ((k * TPR + tid) * VEC) >> 7;
            if ((tid & (kL - 1)) == 0 && gi < ng && live) scales[gi] = scale;
        }
    } else {
        // 128 columns are two waves of one element: their maxima meet in LDS
        for (int i = tid; i < kMaxG; i += TPR) gmax[i] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            // (the larger with zero: a wave of NaN alone has none to leave out)
            const float m = fmaxf(lanes_max<64>(fabsf(y[k][0])), 0.f);
            const int gi = (k * TPR + tid) >> 7;
            if (lane_id() == 0) atomicMax(&gmax[gi], __float_as_uint(m));
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int gi = (k * TPR + tid) >> 7;
            const float scale = fmaxf(__uint_as_float(gmax[gi]) / kE4m3Max, kTinyScale);
            store_e4m3<VEC>(ry, k * TPR + tid, y[k], scale);
            if (((k * TPR + tid) & 127) == 0 && gi < ng && live) scales[gi] = scale;
        }
    }
}

inline gdn_status check_norm(const gdn_norm_problem *pr) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->rows < 0 || pr->D < 1 || !(pr->eps >= 0.f)) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->x_dtype)) return GDN_ERR_UNSUPPORTED;
    if (pr->s_dtype != pr->x_dtype && pr->s_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    if (pr->w_dtype != pr->x_dtype && pr->w_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    if (pr->out_dtype != pr->x_dtype && pr->out_dtype != GDN_E4M3) return GDN_ERR_UNSUPPORTED;
    if (pr->group != 0 && pr->group != 128) return GDN_ERR_UNSUPPORTED;
    if (pr->D > 16384 || pr->rows >= ((int64_t)1 << 31)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// dw[c][j] and db[c][j] (either may be NULL) = the sums over the rows i of part [classes][rows][2][D], in
// a fixed order.  One launch (for every 2^22 workgroups: D columns in sixteens, of each class and of dw and db).
gdn_status enqueue_norm_sums(const float *part, float *dw, float *db, int64_t D, int64_t rows, int64_t classes, hipStream_t s);

}  // namespace gdn

// Root-mean-square norm of x plus a residual, forward and backward.
//
//   s = x + residual,  r = (mean s^2 + eps)^(-1/2),  y = s r w
//   ds = dres + r (dy w - s r^2 mean(dy w s)),  dw = sum over rows dy s r
//
// Both directions are bound by memory: every tensor is read or written once
// and nothing is read twice.  A row stays in registers between its loads and
// its stores (TPR threads hold it, K vectors of VEC elements each), so the
// statistics cost one reduction and no second pass.
//   D <= 256      one wave per row, four rows per workgroup
//   D <= 8192     one workgroup of 256 threads per row
//   D <= 16384    one workgroup of 512 threads per row
// VEC is 4 (8 bytes of bf16) where every row starts at four aligned elements,
// else 2 or 1 (1003 rows of 2050, bf16 with fp32 sums, at VEC 2 and 1: 7.7 and
// 10.6 us forward, 12.1 and 24.2 us backward, when VEC 2 was added).
// Measured: 16384 rows of 8192 in bf16 with a residual to e4m3 190 us, 4.9 TB/s;
// 16384 rows of 4096 in bf16 with a residual forward 85 us (6.3 TB/s, part of
// it out of the last cache), backward 120 us (4.5 TB/s); 32 rows 5 us, a
// launch's own time and one reduction's.
#include "gdn_norm_rows.h"

namespace gdn {

struct NormParams {
    const void *x, *res, *w, *dy, *dres;
    void *y, *s, *ds, *dx;
    float *scales, *dw, *part;
    int64_t rows, x_stride;
    int D, nwg, w_f32, fp8, group;
    float eps, inv_d;
};

template <typename IO, typename RS, int VEC, int TPR, int K>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_forward_kernel(NormParams p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[TPR / 64];
    __shared__ uint32_t gmax[kRows][kRowGroups<VEC, TPR, K>];
    const int sub = TPR < 256 ? wave_id() : 0;
    const int tid = TPR < 256 ? lane_id() : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * kRows + sub;
    const bool live = row < p.rows;
    const uint32_t D = p.D, dm = live ? D : 0;       // a row past the end reads and stores nothing
    const int64_t at = live ? row : 0;
    const rsrc_t rx = make_rsrc((const IO *)p.x + at * p.x_stride, dm * sizeof(IO));
    const rsrc_t rw = make_rsrc(p.w, D * (p.w_f32 ? 4 : (uint32_t)sizeof(IO)));
    float s[K][VEC], ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) row_load<IO, VEC>(rx, (k * TPR + tid) * VEC, s[k]);
    if (p.res) {
        const rsrc_t rr = make_rsrc((const RS *)p.res + at * D, dm * sizeof(RS));
        const rsrc_t ro = make_rsrc((RS *)p.s + at * D, dm * sizeof(RS));
        float t[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) row_load<RS, VEC>(rr, (k * TPR + tid) * VEC, t[k]);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[k][i] += t[k][i];
                // the norm is taken of the row as it is kept, which the
                // backward pass reads
                if constexpr (sizeof(RS) == 2) s[k][i] = bf16_bits_to_f32(f32_to_bf16_bits(s[k][i]));
            }
            row_store<RS, VEC>(ro, (k * TPR + tid) * VEC, s[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss[0] += s[k][i] * s[k][i];
    row_sum<TPR>(ss, red);
    const float r = 1.f / sqrtf(ss[0] * p.inv_d + p.eps);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float w[VEC];
        row_load_either<IO, VEC>(rw, p.w_f32, (k * TPR + tid) * VEC, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s[k][i] = s[k][i] * r * w[i];
            amax = fmaxf(amax, fabsf(s[k][i]));
        }
    }
    if (!p.fp8) {
        const rsrc_t ry = make_rsrc((IO *)p.y + at * D, dm * sizeof(IO));
#pragma unroll
        for (int k = 0; k < K; ++k) row_store<IO, VEC>(ry, (k * TPR + tid) * VEC, s[k]);
        return;
    }
    store_row_e4m3<VEC, TPR, K>(make_rsrc((uint8_t *)p.y + at * D, dm), p.scales + at * (p.group ? (D + 127) >> 7 : 1), live, D, p.group,
                                amax, s, tid, red, gmax[sub]);
}

// Rows go to the workgroups in turn; each keeps its share of dw in registers
// and leaves it in the workspace, one row of D sums per row it holds at a
// time, for norm_dw_kernel to add up in a fixed order.
template <typename IO, typename RS, int VEC, int TPR, int K>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_backward_kernel(NormParams p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[2][2 * (TPR / 64)];
    const int sub = TPR < 256 ? wave_id() : 0;
    const int tid = TPR < 256 ? lane_id() : threadIdx.x;
    const uint32_t D = p.D;
    const rsrc_t rw = make_rsrc(p.w, D * (p.w_f32 ? 4 : (uint32_t)sizeof(IO)));
    float w[K][VEC], dw[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        row_load_either<IO, VEC>(rw, p.w_f32, (k * TPR + tid) * VEC, w[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = 0.f;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + sub; row < p.rows; row += (int64_t)p.nwg * kRows) {
        const rsrc_t rs = make_rsrc((const RS *)p.s + row * D, D * sizeof(RS));
        const rsrc_t rd = make_rsrc((const IO *)p.dy + row * D, D * sizeof(IO));
        float s[K][VEC], d[K][VEC], sums[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            row_load<RS, VEC>(rs, (k * TPR + tid) * VEC, s[k]);
            row_load<IO, VEC>(rd, (k * TPR + tid) * VEC, d[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sums[0] += s[k][i] * s[k][i];
                sums[1] += d[k][i] * w[k][i] * s[k][i];
            }
        // the other half of red: a wave may still read the last row's sums
        row_sum<TPR>(sums, red[turn]);
        turn ^= 1;
        const float r = 1.f / sqrtf(sums[0] * p.inv_d + p.eps);
        const float c = r * r * (sums[1] * p.inv_d);
        const rsrc_t ro = make_rsrc((RS *)p.ds + row * D, D * sizeof(RS));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            float g[VEC];
            if (p.dres) {
                row_load<RS, VEC>(make_rsrc((const RS *)p.dres + row * D, D * sizeof(RS)), e, g);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) g[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                dw[k][i] += d[k][i] * (s[k][i] * r);
                g[i] += r * (d[k][i] * w[k][i] - s[k][i] * c);
            }
            row_store<RS, VEC>(ro, e, g);
            if (p.dx) row_store<IO, VEC>(make_rsrc((IO *)p.dx + row * D, D * sizeof(IO)), e, g);
        }
    }
    const rsrc_t rp = make_rsrc(p.part + ((int64_t)blockIdx.x * kRows + sub) * D, D * 4);
#pragma unroll
    for (int k = 0; k < K; ++k) row_store<float, VEC>(rp, (k * TPR + tid) * VEC, dw[k]);
}

// dw[c] = the sum of column c of n rows: kDwCols columns a workgroup, and
// 1024 / kDwCols rows at a time (768 rows of 2050 columns: 4.0 us; with 64
// columns a workgroup only 33 have work, 15.4 us).
constexpr int kDwCols = 16, kDwRows = 1024 / kDwCols;
__global__ void __launch_bounds__(1024) norm_dw_kernel(NormParams p) {
    __shared__ float red[kDwRows][kDwCols];
    const int j = threadIdx.x % kDwCols, w = threadIdx.x / kDwCols, c = blockIdx.x * kDwCols + j;
    float a = 0.f;
    if (c < p.D) {
        const float *q = p.part + c;
#pragma unroll 4
        for (int64_t i = w; i < p.nwg; i += kDwRows) a += q[i * p.D];
    }
    red[w][j] = a;
    __syncthreads();
    if (w < 4) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kDwRows / 4; ++i) a += red[4 * i + w][j];
    }
    __syncthreads();
    if (w < 4) red[w][j] = a;
    __syncthreads();
    if (w == 0 && c < p.D) p.dw[c] = (red[0][j] + red[1][j]) + (red[2][j] + red[3][j]);
}

namespace {

constexpr int64_t kNormRows = 1 << 22;      // a forward launch's: a multiple of 4, under 2^32 threads
constexpr int kNormWgs = 768;      // workgroups of the backward pass, at most

int rows_per_wg(int64_t D) { return D <= 256 ? 4 : 1; }
int64_t norm_wgs(const gdn_norm_problem *pr) {
    const int64_t k = rows_per_wg(pr->D), n = (pr->rows + k - 1) / k;
    return n < kNormWgs ? n : kNormWgs;
}

template <bool BWD, typename IO, typename RS, int VEC, int TPR, int K>
gdn_status run_norm(NormParams &np, int64_t grid, hipStream_t s) {
    const void *fn = BWD ? (const void *)&norm_backward_kernel<IO, RS, VEC, TPR, K>
                         : (const void *)&norm_forward_kernel<IO, RS, VEC, TPR, K>;
    return launch_kernel(fn, (int)grid, &np, s, TPR < 256 ? 256 : TPR);
}

template <bool BWD, typename IO, typename RS, int VEC>
gdn_status norm_d(NormParams &np, int64_t grid, hipStream_t s) {
    const int D = np.D;
    if (D <= 256) return run_norm<BWD, IO, RS, VEC, 64, 4 / VEC>(np, grid, s);
    if (D <= 1024) return run_norm<BWD, IO, RS, VEC, 256, 4 / VEC>(np, grid, s);
    if (D <= 2048) return run_norm<BWD, IO, RS, VEC, 256, 8 / VEC>(np, grid, s);
    if (D <= 4096) return run_norm<BWD, IO, RS, VEC, 256, 16 / VEC>(np, grid, s);
    if (D <= 8192) return run_norm<BWD, IO, RS, VEC, 256, 32 / VEC>(np, grid, s);
    return run_norm<BWD, IO, RS, VEC, 512, 32 / VEC>(np, grid, s);
}

template <bool BWD, typename IO, typename RS>
gdn_status norm_vec(NormParams &np, int vec, int64_t grid, hipStream_t s) {
    if (vec == 4) return norm_d<BWD, IO, RS, 4>(np, grid, s);
    if (vec == 2) return norm_d<BWD, IO, RS, 2>(np, grid, s);
    return norm_d<BWD, IO, RS, 1>(np, grid, s);
}

template <bool BWD>
gdn_status norm_types(const gdn_norm_problem *pr, NormParams &np, int vec, int64_t grid, hipStream_t s) {
    if (pr->x_dtype == GDN_F32) return norm_vec<BWD, float, float>(np, vec, grid, s);
    if (pr->s_dtype == GDN_F32) return norm_vec<BWD, bf16_t, float>(np, vec, grid, s);
    return norm_vec<BWD, bf16_t, bf16_t>(np, vec, grid, s);
}

void fill_norm(const gdn_norm_problem *pr, NormParams &np) {
    np = NormParams{};
    np.rows = pr->rows;
    np.x_stride = pr->x_stride;
    np.D = (int)pr->D;
    np.w_f32 = pr->w_dtype == GDN_F32;
    np.fp8 = pr->out_dtype == GDN_E4M3;
    np.group = pr->group;
    np.eps = pr->eps;
    np.inv_d = 1.f / (float)pr->D;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_norm_forward(const gdn_norm_problem *pr, const void *x, const void *residual,
                            const void *weight, void *y, void *s, float *scales, void *stream) {
    const gdn_status st = check_norm(pr);
    if (st != GDN_OK) return st;
    if (pr->rows == 0) return GDN_OK;
    if (!x || !weight || !y || (residual && !s)) return GDN_ERR_NULL_ARG;
    if (pr->out_dtype == GDN_E4M3 && !scales) return GDN_ERR_NULL_ARG;
    if (!residual && pr->s_dtype != pr->x_dtype) return GDN_ERR_UNSUPPORTED;
    const size_t eb = dtype_bytes(pr->x_dtype), sb = dtype_bytes(pr->s_dtype), wb = dtype_bytes(pr->w_dtype),
                 ob = dtype_bytes(pr->out_dtype);
    if (!aligned_to(x, eb) || !aligned_to(weight, wb) || !aligned_to(y, ob) || !aligned_to(residual, sb) ||
        !aligned_to(s, sb) || !aligned_to(scales, 4))
        return GDN_ERR_ALIGNMENT;
    NormParams np;
    fill_norm(pr, np);
    np.w = weight;
    int vec = 4;
    while (vec > 1 && !(pr->D % vec == 0 && pr->x_stride % vec == 0 && aligned_to(x, vec * eb) && aligned_to(weight, vec * wb) &&
                        aligned_to(y, vec * ob) && aligned_to(residual, vec * sb) && (!residual || aligned_to(s, vec * sb))))
        vec /= 2;
    // (as many launches as rows need; one up to kNormRows)
    const int k = rows_per_wg(pr->D);
    const int64_t ng = pr->group ? (pr->D + pr->group - 1) / pr->group : 1;
    for (int64_t r = 0; r < pr->rows; r += kNormRows) {
        np.rows = pr->rows - r < kNormRows ? pr->rows - r : kNormRows;
        np.x = (const char *)x + r * pr->x_stride * (int64_t)eb;
        np.res = residual ? (const char *)residual + r * pr->D * (int64_t)sb : nullptr;
        np.y = (char *)y + r * pr->D * (int64_t)ob;
        np.s = s ? (char *)s + r * pr->D * (int64_t)sb : nullptr;
        np.scales = scales ? scales + r * ng : nullptr;
        const gdn_status at = norm_types<false>(pr, np, vec, (np.rows + k - 1) / k, (hipStream_t)stream);
        if (at != GDN_OK) return at;
    }
    return GDN_OK;
}

size_t gdn_workspace_bytes_norm_backward(const gdn_norm_problem *pr) {
    if (check_norm(pr) != GDN_OK) return 0;
    return (size_t)norm_wgs(pr) * rows_per_wg(pr->D) * pr->D * 4;
}

gdn_status gdn_norm_backward(const gdn_norm_problem *pr, const void *dy, const void *s, const void *weight,
                             const void *dres, void *ds, void *dx, float *dweight, void *workspace,
                             size_t workspace_bytes, void *stream) {
    gdn_status st = check_norm(pr);
    if (st != GDN_OK) return st;
    if (!weight || !dweight) return GDN_ERR_NULL_ARG;
    if (pr->rows > 0 && (!dy || !s || !ds)) return GDN_ERR_NULL_ARG;
    const size_t eb = dtype_bytes(pr->x_dtype), sb = dtype_bytes(pr->s_dtype), wb = dtype_bytes(pr->w_dtype);
    if (!aligned_to(dy, eb) || !aligned_to(s, sb) || !aligned_to(weight, wb) || !aligned_to(dres, sb) ||
        !aligned_to(ds, sb) || !aligned_to(dx, eb) || !aligned_to(dweight, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_workspace_bytes_norm_backward(pr);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    NormParams np;
    fill_norm(pr, np);
    np.dy = dy;
    np.s = const_cast<void *>(s);
    np.w = weight;
    np.dres = dres;
    np.ds = ds;
    np.dx = dx;
    np.dw = dweight;
    np.part = (float *)workspace;
    np.nwg = (int)norm_wgs(pr);
    int vec = 4;
    while (vec > 1 && !(pr->D % vec == 0 && aligned_to(dy, vec * eb) && aligned_to(s, vec * sb) && aligned_to(weight, vec * wb) &&
                        aligned_to(dres, vec * sb) && aligned_to(ds, vec * sb) && aligned_to(dx, vec * eb)))
        vec /= 2;
    st = norm_types<true>(pr, np, vec, np.nwg, (hipStream_t)stream);
    if (st != GDN_OK) return st;
    np.nwg *= rows_per_wg(pr->D);
    return launch_kernel((const void *)&norm_dw_kernel, (int)((pr->D + kDwCols - 1) / kDwCols), &np, (hipStream_t)stream, 1024);
}

}  // extern "C"

// Layer norm of x plus a residual, forward and backward.
//
//   s = x + residual,  m = mean s,  r = (mean (s - m)^2 + eps)^(-1/2),  h = (s - m) r
//   y = h w + b
//   u = dy w,  ds = dres + r (u - mean u - h mean(u h)),  dw = sum over rows dy h,  db = sum dy
//
// Bound by memory: every tensor is read or written once.  A row stays in
// registers between its loads and its stores (TPR threads hold it, K vectors of
// VEC elements each): the mean is taken first and the squares of what is left
// after it, so rows far from zero keep their digits; what rounding left of the
// mean (the mean of s - m) is taken out in the same sums.
// Measured (the kernels alone): 16384 rows of 8192 in bf16 with a residual to e4m3 200 us, 4.7 TB/s (249 with a
// row a workgroup, 242 with 256 threads a row); 16384 rows of 4096 in bf16 with a residual
// forward 90 us (6.0 TB/s, part of it out of the last cache), backward 114 to 118 us (4.6 TB/s), the
// sums 7; 1003 rows of 2050 with an fp32 residual 9, 12 and 6 us, three launches that wait for each
// other, the sums' rows of two rows each 8.2 MB written and read again beside 33 MB of data;
// 32 rows 4 us, a launch's own time and two reductions.
#include "gdn_norm_rows.h"

namespace gdn {

struct LayerNormParams {
    const void *x, *res, *w, *b, *dy, *dres;
    void *y, *s, *ds, *dx;
    float *scales, *dw, *db, *part;
    int64_t rows, x_stride;
    int D, nwg, turns, w_f32, fp8, group;
    float eps, inv_d;
};

// Sums over the TPR threads of a row (a wave, or a workgroup), in every one of them.
template <int TPR, int N>
__device__ __forceinline__ void row_total(float (&v)[N], float *red) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<64>(v[i]);
    if constexpr (TPR > 64) {
        constexpr int kW = TPR / 64;
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[i * kW + wave_id()] = v[i];
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < kW; ++k) t += red[i * kW + k];
            v[i] = t;
        }
    }
}

// (var + eps)^(-1/2); rounding may leave the variance of equal elements below zero.
__device__ __forceinline__ float inverse_deviation(float var, float eps) { return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps); }

// s - mean s, where the row has elements (behind it s stays zero).
template <int VEC, int TPR, int K>
__device__ __forceinline__ void take_mean(float (&s)[K][VEC], uint32_t D, int tid, float inv_d, float *red) {
    float t[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[0] += s[k][i];
    row_total<TPR>(t, red);
    const float m = t[0] * inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[k][i] = (uint32_t)((k * TPR + tid) * VEC) < D ? s[k][i] - m : 0.f;
}

// A workgroup takes `turns` rows (or four times as many, one a wave), with the
// weights in registers and the next row in flight (not where a thread holds 32
// elements of a row): the weights of one row after the other would be half of
// what comes through the second cache.
template <typename IO, typename RS, int VEC, int TPR, int K>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) layer_norm_forward_kernel(LayerNormParams p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    constexpr bool kAhead = K * VEC <= 16;
    __shared__ float red[4][TPR / 64];
    __shared__ uint32_t gmax[kRows][kRowGroups<VEC, TPR, K>];
    const int sub = TPR < 256 ? wave_id() : 0;
    const int tid = TPR < 256 ? lane_id() : threadIdx.x;
    const uint32_t D = p.D;
    RawRow<IO, VEC> xn[kAhead ? K : 1];
    RawRow<RS, VEC> rn[kAhead ? K : 1];
    // (a row past the end reads zeros and stores nothing)
    auto fetch = [&](int64_t row) {
        if constexpr (!kAhead) return;
        const bool live = row < p.rows;
        const int64_t at = live ? row : 0;
        const rsrc_t rx = make_rsrc((const IO *)p.x + at * p.x_stride, live ? D * sizeof(IO) : 0);
        const rsrc_t rr = make_rsrc((const RS *)p.res + (p.res ? at * D : 0), live && p.res ? D * sizeof(RS) : 0);
#pragma unroll
        for (int k = 0; k < (kAhead ? K : 1); ++k) {
            xn[k].load(rx, tid * VEC * sizeof(IO), k * TPR * VEC * sizeof(IO));
            rn[k].load(rr, tid * VEC * sizeof(RS), k * TPR * VEC * sizeof(RS));
        }
    };
    const int turns = kAhead ? p.turns : 1;
    int64_t row = (int64_t)blockIdx.x * turns * kRows + sub;
    if (kAhead) fetch(row);
    const uint32_t wb = p.w_f32 ? 4 : (uint32_t)sizeof(IO);
    const rsrc_t rw = make_rsrc(p.w, D * wb), rb = make_rsrc(p.b, p.b ? D * wb : 0);
    float w[kAhead ? K : 1][VEC], b[kAhead ? K : 1][VEC];
    if constexpr (kAhead) load_affine<IO, VEC, K>(rw, rb, p.w_f32, tid * VEC, TPR * VEC, w, b);
    for (int turn = 0; turn < turns; ++turn, row += kRows) {
        const bool live = row < p.rows;
        const uint32_t dm = live ? D : 0;
        const int64_t at = live ? row : 0;
        float s[K][VEC];
        auto keep = [&](int k, const float (&r)[VEC]) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[k][i] += r[i];
                // the norm is taken of the row as it is kept, which the
                // backward pass reads
                if constexpr (sizeof(RS) == 2) s[k][i] = bf16_bits_to_f32(f32_to_bf16_bits(s[k][i]));
            }
        };
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[VEC];
                xn[k].get(s[k]);
                rn[k].get(r);
                if (p.res) keep(k, r);
            }
        } else {
            const rsrc_t rx = make_rsrc((const IO *)p.x + at * p.x_stride, dm * sizeof(IO));
#pragma unroll
            for (int k = 0; k < K; ++k) row_load<IO, VEC>(rx, (k * TPR + tid) * VEC, s[k]);
            if (p.res) {
                const rsrc_t rr = make_rsrc((const RS *)p.res + at * D, dm * sizeof(RS));
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float r[VEC];
                    row_load<RS, VEC>(rr, (k * TPR + tid) * VEC, r);
                    keep(k, r);
                }
            }
        }
        if (kAhead && turn + 1 < turns) fetch(row + kRows);
        if (p.res) {
            const rsrc_t ro = make_rsrc((RS *)p.s + at * D, dm * sizeof(RS));
#pragma unroll
            for (int k = 0; k < K; ++k) row_store<RS, VEC>(ro, (k * TPR + tid) * VEC, s[k]);
        }
        take_mean<VEC, TPR, K>(s, D, tid, p.inv_d, red[0]);
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                t[0] += s[k][i];
                t[1] += s[k][i] * s[k][i];
            }
        row_total<TPR>(t, red[1]);
        const float m = t[0] * p.inv_d;
        const float r = inverse_deviation(t[1] * p.inv_d - m * m, p.eps);
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (!kAhead) load_affine<IO, VEC, 1>(rw, rb, p.w_f32, (k * TPR + tid) * VEC, 0, w, b);
            const int at = kAhead ? k : 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[k][i] = fmaf((s[k][i] - m) * r, w[at][i], b[at][i]);
                amax = fmaxf(amax, fabsf(s[k][i]));
            }
        }
        if (!p.fp8) {
            const rsrc_t ry = make_rsrc((IO *)p.y + at * D, dm * sizeof(IO));
#pragma unroll
            for (int k = 0; k < K; ++k) row_store<IO, VEC>(ry, (k * TPR + tid) * VEC, s[k]);
        } else {
            store_row_e4m3<VEC, TPR, K>(make_rsrc((uint8_t *)p.y + at * D, dm), p.scales + at * (p.group ? (D + 127) >> 7 : 1), live, D,
                                        p.group, amax, s, tid, red[3], gmax[sub]);
        }
    }
}

// Rows go to the workgroups in turn; each keeps its shares of dw and db in
// registers and leaves them in the workspace, two rows of D sums per row it
// holds at a time, for norm_sums_kernel to add up in a fixed order.  The next
// row's s and dy are in flight while a row is worked on.
template <typename IO, typename RS, int VEC, int TPR, int K>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) layer_norm_backward_kernel(LayerNormParams p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    constexpr bool kAhead = K * VEC <= 16;
    __shared__ float red[2][5][TPR / 64];
    const int sub = TPR < 256 ? wave_id() : 0;
    const int tid = TPR < 256 ? lane_id() : threadIdx.x;
    const uint32_t D = p.D;
    const rsrc_t rw = make_rsrc(p.w, D * (p.w_f32 ? 4 : (uint32_t)sizeof(IO)));
    // a vector of the weights: kept, or loaded again where it is used
    float kept[kAhead ? K : 1][VEC], dw[K][VEC], db[K][VEC];
    auto weights = [&](int k, float (&w)[VEC]) {
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = kept[k][i];
        } else {
            row_load_either<IO, VEC>(rw, p.w_f32, (k * TPR + tid) * VEC, w);
        }
    };
    if constexpr (kAhead) load_affine<IO, VEC, K>(rw, make_rsrc(nullptr, 0), p.w_f32, tid * VEC, TPR * VEC, kept, dw);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.f;
    RawRow<RS, VEC> sn[K];
    RawRow<IO, VEC> dn[K];
    auto fetch = [&](int64_t row) {
        // (a row past the end reads zeros)
        const uint32_t dm = row < p.rows ? D : 0;
        const int64_t at = row < p.rows ? row : 0;
        const rsrc_t rs = make_rsrc((const RS *)p.s + at * D, dm * sizeof(RS)), rd = make_rsrc((const IO *)p.dy + at * D, dm * sizeof(IO));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            sn[k].load(rs, tid * VEC * sizeof(RS), k * TPR * VEC * sizeof(RS));
            dn[k].load(rd, tid * VEC * sizeof(IO), k * TPR * VEC * sizeof(IO));
        }
    };
    const int64_t step = (int64_t)p.nwg * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + sub;
    if (kAhead) fetch(row);
    int turn = 0;
    for (; row < p.rows; row += step) {
        if (!kAhead) fetch(row);
        float s[K][VEC], d[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            sn[k].get(s[k]);
            dn[k].get(d[k]);
        }
        // (without dres the descriptor is empty, and reads zeros)
        const rsrc_t rg = make_rsrc((const RS *)p.dres + (p.dres ? row * D : 0), p.dres ? D * sizeof(RS) : 0);
        RawRow<RS, VEC> gn[kAhead ? K : 1];
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < K; ++k) gn[k].load(rg, tid * VEC * sizeof(RS), k * TPR * VEC * sizeof(RS));
        }
        if (kAhead) fetch(row + step);
        // (the other half of red: a wave may still read the last row's sums)
        take_mean<VEC, TPR, K>(s, D, tid, p.inv_d, red[turn][0]);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[VEC];
            if constexpr (!kAhead) __builtin_amdgcn_sched_barrier(0);      // no loads ahead
            weights(k, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = d[k][i] * w[i];
                t[0] += s[k][i];
                t[1] += s[k][i] * s[k][i];
                t[2] += u;
                t[3] += u * s[k][i];
            }
        }
        row_total<TPR>(t, red[turn][1]);
        turn ^= 1;
        const float m = t[0] * p.inv_d;
        const float r = inverse_deviation(t[1] * p.inv_d - m * m, p.eps);
        const float mu = t[2] * p.inv_d, c = r * (t[3] * p.inv_d - m * mu);       // mean u, mean(u h)
        const rsrc_t ro = make_rsrc((RS *)p.ds + row * D, D * sizeof(RS)), rx = make_rsrc((IO *)p.dx + row * D, p.dx ? D * sizeof(IO) : 0);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            float g[VEC], w[VEC];
            if constexpr (!kAhead) __builtin_amdgcn_sched_barrier(0);
            if constexpr (!kAhead) gn[0].load(rg, tid * VEC * sizeof(RS), k * TPR * VEC * sizeof(RS));
            gn[kAhead ? k : 0].get(g);
            weights(k, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = (s[k][i] - m) * r;
                dw[k][i] += d[k][i] * h;
                db[k][i] += d[k][i];
                g[i] += r * (d[k][i] * w[i] - mu - h * c);
            }
            row_store<RS, VEC>(ro, e, g);
            if (p.dx) row_store<IO, VEC>(rx, e, g);
        }
    }
    float *part = p.part + ((int64_t)blockIdx.x * kRows + sub) * 2 * D;
    const rsrc_t rp = make_rsrc(part, D * 4), rq = make_rsrc(part + D, D * 4);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        row_store<float, VEC>(rp, (k * TPR + tid) * VEC, dw[k]);
        row_store<float, VEC>(rq, (k * TPR + tid) * VEC, db[k]);
    }
}

// 16 columns a workgroup and 64 rows at a time.
struct SumsParams {
    const float *part;
    float *dw, *db;
    int64_t D, rows, cols;
};
constexpr int kSumCols = 16, kSumRows = 1024 / kSumCols;
__global__ void __launch_bounds__(1024) norm_sums_kernel(SumsParams p) {
    __shared__ float red[kSumRows][kSumCols];
    const int j = threadIdx.x % kSumCols, w = threadIdx.x / kSumCols, n = p.dw && p.db ? 2 : 1;
    const int which = p.dw ? blockIdx.x % n : 1;
    const int64_t at = blockIdx.x / n, cls = at / p.cols, c = at % p.cols * kSumCols + j;
    float a = 0.f;
    if (c < p.D) {
        const float *q = p.part + (cls * p.rows * 2 + which) * p.D + c;
#pragma unroll 4
        for (int64_t i = w; i < p.rows; i += kSumRows) a += q[i * 2 * p.D];
    }
    red[w][j] = a;
    __syncthreads();
    if (w < 4) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kSumRows / 4; ++i) a += red[4 * i + w][j];
    }
    __syncthreads();
    if (w < 4) red[w][j] = a;
    __syncthreads();
    if (w == 0 && c < p.D) (which ? p.db : p.dw)[cls * p.D + c] = (red[0][j] + red[1][j]) + (red[2][j] + red[3][j]);
}

gdn_status enqueue_norm_sums(const float *part, float *dw, float *db, int64_t D, int64_t rows, int64_t classes, hipStream_t s) {
    const int64_t cols = (D + kSumCols - 1) / kSumCols, both = (dw != nullptr) + (db != nullptr);
    if (!both) return GDN_OK;
    // (as many launches as classes need, of under 2^32 threads)
    const int64_t step = (((int64_t)1 << 32) - 1) / 1024 / (cols * both);
    for (int64_t c = 0; c < classes; c += step) {
        const int64_t n = classes - c < step ? classes - c : step;
        SumsParams sp{part + c * rows * 2 * D, dw ? dw + c * D : nullptr, db ? db + c * D : nullptr, D, rows, cols};
        const gdn_status st = launch_kernel((const void *)&norm_sums_kernel, (int)(n * cols * both), &sp, s, 1024);
        if (st != GDN_OK) return st;
    }
    return GDN_OK;
}

namespace {

constexpr int64_t kLnRows = 1 << 22;      // a forward launch's: a multiple of 4, under 2^32 threads
constexpr int kLnWgs = 512;               // workgroups of the backward pass, at most

constexpr int kLnTurns = 4, kLnMany = 1024;      // rows of a forward workgroup, where that leaves kLnMany of them

int ln_rows_per_wg(int64_t D) { return D <= 256 ? 4 : 1; }

// Workgroups of the backward pass: as many as need the same number of turns as kLnWgs.
int64_t ln_wgs(const gdn_norm_problem *pr) {
    const int64_t k = ln_rows_per_wg(pr->D), n = (pr->rows + k - 1) / k;
    const int64_t turns = (n + kLnWgs - 1) / kLnWgs;
    return turns ? (n + turns - 1) / turns : 0;
}

template <bool BWD, typename IO, typename RS, int VEC, int TPR, int K>
gdn_status run_ln(LayerNormParams &np, int64_t grid, hipStream_t s) {
    const void *fn = BWD ? (const void *)&layer_norm_backward_kernel<IO, RS, VEC, TPR, K>
                         : (const void *)&layer_norm_forward_kernel<IO, RS, VEC, TPR, K>;
    return launch_kernel(fn, (int)grid, &np, s, TPR < 256 ? 256 : TPR);
}

template <bool BWD, typename IO, typename RS, int VEC>
gdn_status ln_d(LayerNormParams &np, int64_t grid, hipStream_t s) {
    const int D = np.D;
    if (D <= 256) return run_ln<BWD, IO, RS, VEC, 64, 4 / VEC>(np, grid, s);
    if (D <= 1024) return run_ln<BWD, IO, RS, VEC, 256, 4 / VEC>(np, grid, s);
    if (D <= 2048) return run_ln<BWD, IO, RS, VEC, 256, 8 / VEC>(np, grid, s);
    if (D <= 4096) return run_ln<BWD, IO, RS, VEC, 256, 16 / VEC>(np, grid, s);
    if (D <= 8192) return run_ln<BWD, IO, RS, VEC, 512, 16 / VEC>(np, grid, s);
    return run_ln<BWD, IO, RS, VEC, 512, 32 / VEC>(np, grid, s);
}

template <bool BWD, typename IO, typename RS>
gdn_status ln_vec(LayerNormParams &np, int vec, int64_t grid, hipStream_t s) {
    if (vec == 4) return ln_d<BWD, IO, RS, 4>(np, grid, s);
    if (vec == 2) return ln_d<BWD, IO, RS, 2>(np, grid, s);
    return ln_d<BWD, IO, RS, 1>(np, grid, s);
}

template <bool BWD>
gdn_status ln_types(const gdn_norm_problem *pr, LayerNormParams &np, int vec, int64_t grid, hipStream_t s) {
    if (pr->x_dtype == GDN_F32) return ln_vec<BWD, float, float>(np, vec, grid, s);
    if (pr->s_dtype == GDN_F32) return ln_vec<BWD, bf16_t, float>(np, vec, grid, s);
    return ln_vec<BWD, bf16_t, bf16_t>(np, vec, grid, s);
}

void fill_ln(const gdn_norm_problem *pr, LayerNormParams &np) {
    np = LayerNormParams{};
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

gdn_status gdn_layer_norm_forward(const gdn_norm_problem *pr, const void *x, const void *residual,
                                  const void *weight, const void *bias, void *y, void *s, float *scales, void *stream) {
    const gdn_status st = check_norm(pr);
    if (st != GDN_OK) return st;
    if (pr->rows == 0) return GDN_OK;
    if (!x || !weight || !y || (residual && !s)) return GDN_ERR_NULL_ARG;
    if (pr->out_dtype == GDN_E4M3 && !scales) return GDN_ERR_NULL_ARG;
    if (!residual && pr->s_dtype != pr->x_dtype) return GDN_ERR_UNSUPPORTED;
    const size_t eb = dtype_bytes(pr->x_dtype), sb = dtype_bytes(pr->s_dtype), wb = dtype_bytes(pr->w_dtype),
                 ob = dtype_bytes(pr->out_dtype);
    if (!aligned_to(x, eb) || !aligned_to(weight, wb) || !aligned_to(bias, wb) || !aligned_to(y, ob) ||
        !aligned_to(residual, sb) || !aligned_to(s, sb) || !aligned_to(scales, 4))
        return GDN_ERR_ALIGNMENT;
    LayerNormParams np;
    fill_ln(pr, np);
    np.w = weight;
    np.b = bias;
    int vec = 4;
    while (vec > 1 && !(pr->D % vec == 0 && pr->x_stride % vec == 0 && aligned_to(x, vec * eb) && aligned_to(weight, vec * wb) &&
                        aligned_to(bias, vec * wb) && aligned_to(y, vec * ob) && aligned_to(residual, vec * sb) &&
                        (!residual || aligned_to(s, vec * sb))))
        vec /= 2;
    // (as many launches as rows need; one up to kLnRows)
    const int k = ln_rows_per_wg(pr->D);
    const int64_t ng = pr->group ? (pr->D + pr->group - 1) / pr->group : 1;
    for (int64_t r = 0; r < pr->rows; r += kLnRows) {
        np.rows = pr->rows - r < kLnRows ? pr->rows - r : kLnRows;
        np.x = (const char *)x + r * pr->x_stride * (int64_t)eb;
        np.res = residual ? (const char *)residual + r * pr->D * (int64_t)sb : nullptr;
        np.y = (char *)y + r * pr->D * (int64_t)ob;
        np.s = s ? (char *)s + r * pr->D * (int64_t)sb : nullptr;
        np.scales = scales ? scales + r * ng : nullptr;
        const int64_t groups = (np.rows + k - 1) / k;
        np.turns = np.D <= 8192 && groups >= kLnTurns * kLnMany ? kLnTurns : 1;
        const gdn_status at = ln_types<false>(pr, np, vec, (groups + np.turns - 1) / np.turns, (hipStream_t)stream);
        if (at != GDN_OK) return at;
    }
    return GDN_OK;
}

size_t gdn_workspace_bytes_layer_norm_backward(const gdn_norm_problem *pr) {
    if (check_norm(pr) != GDN_OK) return 0;
    return (size_t)ln_wgs(pr) * ln_rows_per_wg(pr->D) * pr->D * 8;
}

gdn_status gdn_layer_norm_backward(const gdn_norm_problem *pr, const void *dy, const void *s, const void *weight,
                                   const void *dres, void *ds, void *dx, float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    gdn_status st = check_norm(pr);
    if (st != GDN_OK) return st;
    if (!weight || !dweight) return GDN_ERR_NULL_ARG;
    if (pr->rows > 0 && (!dy || !s || !ds)) return GDN_ERR_NULL_ARG;
    const size_t eb = dtype_bytes(pr->x_dtype), sb = dtype_bytes(pr->s_dtype), wb = dtype_bytes(pr->w_dtype);
    if (!aligned_to(dy, eb) || !aligned_to(s, sb) || !aligned_to(weight, wb) || !aligned_to(dres, sb) ||
        !aligned_to(ds, sb) || !aligned_to(dx, eb) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_workspace_bytes_layer_norm_backward(pr);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    LayerNormParams np;
    fill_ln(pr, np);
    np.dy = dy;
    np.s = const_cast<void *>(s);
    np.w = weight;
    np.dres = dres;
    np.ds = ds;
    np.dx = dx;
    np.part = (float *)workspace;
    np.nwg = (int)ln_wgs(pr);
    int vec = 4;
    while (vec > 1 && !(pr->D % vec == 0 && aligned_to(dy, vec * eb) && aligned_to(s, vec * sb) && aligned_to(weight, vec * wb) &&
                        aligned_to(dres, vec * sb) && aligned_to(ds, vec * sb) && aligned_to(dx, vec * eb)))
        vec /= 2;
    st = ln_types<true>(pr, np, vec, np.nwg, (hipStream_t)stream);
    if (st != GDN_OK) return st;
    return enqueue_norm_sums(np.part, dweight, dbias, pr->D, np.nwg * ln_rows_per_wg(pr->D), 1, (hipStream_t)stream);
}

}  // extern "C"

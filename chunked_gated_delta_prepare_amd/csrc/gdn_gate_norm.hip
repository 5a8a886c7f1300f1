// Gated norm: rows of D elements x with a gate z of their own.
//
//   n(v) = (v - m) r w + b,  m = mean v (or 0),  r = (mean (v - m)^2 + eps)^(-1/2)
//   gate first:  y = n(x act(z));   else  y = n(x) act(z)
// Backward, with h = (v - m) r, dn = dy (gate first) or dy act(z), u = dn w:
//   dv = r (u - mean u - h mean(u h))     (mean u only where m is taken)
//   dx, dz = dv act(z), dv x act'(z)      or  dv, dy (h w + b) act'(z)
//   dw = sum dn h,  db = sum dn over the rows that share w
//
// Bound by memory: every tensor is read or written once.  TPR threads hold a
// row (K vectors of VEC elements each), from 16 lanes for the 64 elements of a
// small head to a workgroup; rows of one wave or less need no barrier.  Where
// a head's rows lie is a stride between tokens and one between heads, so the
// gate may be a part of a projection's rows.
#include "gdn_norm_rows.h"

namespace gdn {

struct GateNormParams {
    const void *x, *z, *w, *b, *dy;
    void *y, *dx, *dz;
    float *part;
    int64_t rows;                                    // of one class: rows that share their weights
    int64_t xt, xh, zt, zh, dzt, dzh;
    uint32_t H, classes;
    int D, parts, w_f32, first, center, silu;
    int64_t row0;                                    // of this launch (forward)
    float eps, inv_d;
};

// VEC elements of a row at its element e, zero where the row has none.
template <typename T, int VEC>
__device__ __forceinline__ void fetch_row(RawRow<T, VEC> &r, const T *row, uint32_t e, bool ok) {
#pragma unroll
    for (auto &v : r.u) v = 0;
    if (!ok) return;
    if constexpr (VEC * sizeof(T) == 2) {
        r.u[0] = *(const uint16_t *)(row + e);
    } else if constexpr (VEC * sizeof(T) == 4) {
        r.u[0] = *(const uint32_t *)(row + e);
    } else if constexpr (VEC * sizeof(T) == 8) {
        const u32x2 v = *(const u32x2 *)(row + e);
        r.u[0] = v[0];
        r.u[1] = v[1];
    } else {
        const u32x4 v = *(const u32x4 *)(row + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.u[i] = v[i];
    }
}

// VEC values to a row's element e, where e < end (the row's length, or 0).  All
// lanes of a pair take part, with adjacent e of one row (see row_store).
template <typename T, int VEC>
__device__ __forceinline__ void put_row(T *row, uint32_t e, uint32_t end, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        if (e < end) io_traits<T>::store(row + e, x[0]);
    } else if constexpr (sizeof(T) == 2) {
        if (e < end) *(u32x2 *)(row + e) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    } else {
        const bool odd = lane_id() & 1;
        const float r0 = swap_pair(odd ? x[0] : x[2]), r1 = swap_pair(odd ? x[1] : x[3]);
        const uint32_t at = odd ? e - 2 : e;
        if (at < end) *(u32x2 *)(row + at) = u32x2{__float_as_uint(odd ? r0 : x[0]), __float_as_uint(odd ? r1 : x[1])};
        if (at + 4 < end) *(u32x2 *)(row + at + 4) = u32x2{__float_as_uint(odd ? x[2] : r0), __float_as_uint(odd ? x[3] : r1)};
    }
}

// act(z) and act'(z)
struct Act {
    float a, d;
    __device__ __forceinline__ Act(float z, int silu) {
        const Sigmoid g(z);
        a = silu ? z * g.s : g.s;
        d = silu ? fmaf(z * g.s, g.o, g.s) : g.s * g.o;
    }
};

template <int TPR, int N>
__device__ __forceinline__ void slot_total(float (&v)[N], float *red) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<(TPR < 64 ? TPR : 64)>(v[i]);
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

template <int TPR>
constexpr int kGateThreads = TPR < 256 ? 256 : TPR;

// v -> v - mean v where the row has elements
template <int VEC, int TPR, int K>
__device__ __forceinline__ void slot_mean(float (&v)[K][VEC], uint32_t D, int tid, float inv_d, float *red) {
    float t[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[0] += v[k][i];
    slot_total<TPR>(t, red);
    const float m = t[0] * inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[k][i] = (uint32_t)((k * TPR + tid) * VEC) < D ? v[k][i] - m : 0.f;
}

__device__ __forceinline__ float inverse_root(float ms, float eps) { return 1.f / sqrtf((ms < 0.f ? 0.f : ms) + eps); }

// R rows of a slot's are loaded before the first is worked on.
template <typename IO, int VEC, int TPR, int K, int R>
__global__ void __launch_bounds__(kGateThreads<TPR>) gate_norm_forward_kernel(GateNormParams p) {
    constexpr int kSlots = kGateThreads<TPR> / TPR;
    __shared__ float red[2][2][TPR < 64 ? 1 : TPR / 64];
    const int slot = threadIdx.x / TPR, tid = threadIdx.x % TPR;
    const uint32_t D = p.D;
    RawRow<IO, VEC> xr[R][K], zr[R][K];
    uint32_t head[R];
    const int64_t row0 = p.row0 + (int64_t)blockIdx.x * (kSlots * R) + slot;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int64_t row = row0 + j * kSlots;
        const bool live = row < p.rows;
        const uint32_t at = live ? (uint32_t)row : 0, t = at / p.H;
        head[j] = at - t * p.H;
        const IO *xp = (const IO *)p.x + t * p.xt + head[j] * p.xh, *zp = (const IO *)p.z + t * p.zt + head[j] * p.zh;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            fetch_row(xr[j][k], xp, e, live && e < D);
            fetch_row(zr[j][k], zp, e, live && e < D);
        }
    }
    const uint32_t wb = p.w_f32 ? 4 : (uint32_t)sizeof(IO), nw = D * (p.classes > 1 ? p.H : 1);
    const rsrc_t rw = make_rsrc(p.w, nw * wb), rb = make_rsrc(p.b, p.b ? nw * wb : 0);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int64_t row = row0 + j * kSlots;
        float v[K][VEC], g[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xr[j][k].get(v[k]);
            zr[j][k].get(g[k]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float a = Act(g[k][i], p.silu).a;
                if (p.first) v[k][i] *= a;
                g[k][i] = p.first ? 1.f : a;
            }
        }
        if (p.center) slot_mean<VEC, TPR, K>(v, D, tid, p.inv_d, red[0][0]);
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                t[0] += v[k][i] * v[k][i];
                t[1] += v[k][i];
            }
        slot_total<TPR>(t, red[1][0]);
        const float m = p.center ? t[1] * p.inv_d : 0.f;
        const float r = inverse_root(t[0] * p.inv_d - m * m, p.eps);
        const uint32_t own = p.classes > 1 ? head[j] * D : 0, end = row < p.rows ? D : 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            // (a row's end is not the weights': what lies behind it is not stored)
            float w[VEC], b[VEC];
            row_load_either<IO, VEC>(rw, p.w_f32, own + e, w);
            row_load_either<IO, VEC>(rb, p.w_f32, own + e, b);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[k][i] = fmaf((v[k][i] - m) * r, w[i], b[i]) * g[k][i];
            put_row<IO, VEC>((IO *)p.y + row * D, e, end, v[k]);
        }
    }
}

// A class is the rows that share their weights: all, or one head's.  Its rows
// go to its workgroups' slots in turn; the slots' shares of dw and db stay in
// registers and meet in LDS, and every workgroup leaves one row of D sums of
// each in the workspace.  The next row is in flight while one is worked on (not
// in the workgroups of 1024 threads, which have 128 registers each).
template <typename IO, int VEC, int TPR, int K>
__global__ void __launch_bounds__(kGateThreads<TPR>) gate_norm_backward_kernel(GateNormParams p) {
    constexpr int kSlots = kGateThreads<TPR> / TPR;
    constexpr int kW = TPR < 64 ? 1 : TPR / 64;
    constexpr bool kAhead = TPR < 1024;
    __shared__ float red[2][5][kW];
    __shared__ float sums[TPR < 256 ? 4 : 1][TPR < 256 ? 2 : 1][TPR < 256 ? TPR * K * VEC : 1];
    const int slot = threadIdx.x / TPR, tid = threadIdx.x % TPR;
    const uint32_t D = p.D, cls = blockIdx.x % p.classes, part = blockIdx.x / p.classes;
    const uint32_t wb = p.w_f32 ? 4 : (uint32_t)sizeof(IO);
    const rsrc_t rw = make_rsrc((const char *)p.w + (int64_t)cls * D * wb, D * wb),
                 rb = make_rsrc((const char *)p.b + (p.b ? (int64_t)cls * D * wb : 0), p.b ? D * wb : 0);
    float w[K][VEC], b[K][VEC], dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        row_load_either<IO, VEC>(rw, p.w_f32, (k * TPR + tid) * VEC, w[k]);
        row_load_either<IO, VEC>(rb, p.w_f32, (k * TPR + tid) * VEC, b[k]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.f;
    }
    RawRow<IO, VEC> xn[K], zn[K], dn[K];
    // row i of this class: row i classes + cls of all
    auto fetch = [&](int64_t i) {
        const bool live = i < p.rows;
        const uint32_t at = live ? (uint32_t)(i * p.classes + cls) : 0, t = at / p.H, h = at - t * p.H;
        const IO *xp = (const IO *)p.x + t * p.xt + h * p.xh, *zp = (const IO *)p.z + t * p.zt + h * p.zh,
                 *dp = (const IO *)p.dy + (int64_t)at * D;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            fetch_row(xn[k], xp, e, live && e < D);
            fetch_row(zn[k], zp, e, live && e < D);
            fetch_row(dn[k], dp, e, live && e < D);
        }
    };
    // (all slots of a workgroup make the same number of turns: rows of several waves meet at barriers)
    const int64_t step = (int64_t)p.parts * kSlots;
    int64_t i0 = (int64_t)part * kSlots;
    if (kAhead) fetch(i0 + slot);
    int turn = 0;
    for (; i0 < p.rows; i0 += step) {
        if (!kAhead) fetch(i0 + slot);
        const bool live = i0 + slot < p.rows;
        const uint32_t at = live ? (uint32_t)((i0 + slot) * p.classes + cls) : 0, t0 = at / p.H, hd = at - t0 * p.H;
        float x[K][VEC], z[K][VEC], d[K][VEC], v[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k].get(x[k]);
            zn[k].get(z[k]);
            dn[k].get(d[k]);
        }
        if (kAhead) fetch(i0 + step + slot);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[k][i] = p.first ? x[k][i] * Act(z[k][i], p.silu).a : x[k][i];
        if (p.center) slot_mean<VEC, TPR, K>(v, D, tid, p.inv_d, red[turn][0]);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = (p.first ? d[k][i] : d[k][i] * Act(z[k][i], p.silu).a) * w[k][i];
                t[0] += v[k][i] * v[k][i];
                t[1] += u * v[k][i];
                t[2] += v[k][i];
                t[3] += u;
            }
        slot_total<TPR>(t, red[turn][1]);
        turn ^= 1;
        const float m = p.center ? t[2] * p.inv_d : 0.f, mu = p.center ? t[3] * p.inv_d : 0.f;
        const float r = inverse_root(t[0] * p.inv_d - m * m, p.eps);
        const float c = r * (t[1] * p.inv_d - m * (t[3] * p.inv_d));
        IO *xo = (IO *)p.dx + (int64_t)at * D, *zo = (IO *)p.dz + t0 * p.dzt + hd * p.dzh;
        const uint32_t end = live ? D : 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            float dx[VEC], dz[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Act g(z[k][i], p.silu);
                const float h = (v[k][i] - m) * r, dd = p.first ? d[k][i] : d[k][i] * g.a;
                const float dv = r * (dd * w[k][i] - mu - h * c);
                dw[k][i] += dd * h;
                db[k][i] += dd;
                dx[i] = p.first ? dv * g.a : dv;
                dz[i] = (p.first ? dv * x[k][i] : d[k][i] * fmaf(h, w[k][i], b[k][i])) * g.d;
            }
            put_row<IO, VEC>(xo, e, end, dx);
            put_row<IO, VEC>(zo, e, end, dz);
        }
    }
    float *out = p.part + ((int64_t)cls * p.parts + part) * 2 * D;
    const rsrc_t rp = make_rsrc(out, D * 4), rq = make_rsrc(out + D, D * 4);
    if constexpr (TPR < 256) {
        // the slots of a wave, then the waves
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma unroll
                for (int s = TPR; s < 64; s <<= 1) {
                    dw[k][i] += __shfl_xor(dw[k][i], s, 64);
                    db[k][i] += __shfl_xor(db[k][i], s, 64);
                }
                if (lane_id() < TPR) {
                    sums[wave_id()][0][(k * TPR + tid) * VEC + i] = dw[k][i];
                    sums[wave_id()][1][(k * TPR + tid) * VEC + i] = db[k][i];
                }
            }
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < D; e += 256) {
            float a[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) a[q] = (sums[0][q][e] + sums[1][q][e]) + (sums[2][q][e] + sums[3][q][e]);
            bstore32(__float_as_uint(a[0]), rp, e * 4, 0);
            bstore32(__float_as_uint(a[1]), rq, e * 4, 0);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            row_store<float, VEC>(rp, (k * TPR + tid) * VEC, dw[k]);
            row_store<float, VEC>(rq, (k * TPR + tid) * VEC, db[k]);
        }
    }
}

namespace {

constexpr int64_t kGateRows = 1 << 22;     // a forward launch's, under 2^32 threads
constexpr int kGateWgs = 1024;             // workgroups of the backward pass, about

gdn_status check_gate_norm(const gdn_gate_norm_problem *pr) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->T < 0 || pr->H < 1 || pr->D < 1 || !(pr->eps >= 0.f)) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->io_dtype) || (pr->w_dtype != pr->io_dtype && pr->w_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (pr->act != GDN_ACT_SILU && pr->act != GDN_ACT_SIGMOID) return GDN_ERR_UNSUPPORTED;
    const int64_t most = ((int64_t)1 << 31) - 1;
    if (pr->D > 8192 || pr->H > most || pr->T > most / pr->H) return GDN_ERR_UNSUPPORTED;
    // a class's workgroups; weights are reached with 32-bit byte offsets
    if (pr->each && (pr->H > 65536 || pr->H * pr->D > (1 << 28))) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int64_t gate_classes(const gdn_gate_norm_problem *pr) { return pr->each ? pr->H : 1; }
int gate_tpr(int64_t D) { return D <= 64 ? 16 : D <= 128 ? 32 : D <= 512 ? 64 : D <= 2048 ? 256 : D <= 4096 ? 512 : 1024; }
int gate_slots(int64_t D) { return gate_tpr(D) < 256 ? 256 / gate_tpr(D) : 1; }

// Workgroups of a class in the backward pass.
int64_t gate_parts(const gdn_gate_norm_problem *pr) {
    const int64_t c = gate_classes(pr), rows = pr->T * pr->H / c, n = (rows + gate_slots(pr->D) - 1) / gate_slots(pr->D);
    int64_t most = kGateWgs / c;
    most = most < 1 ? 1 : most;
    const int64_t turns = (n + most - 1) / most;
    return turns ? (n + turns - 1) / turns : 0;
}

template <bool BWD, typename IO, int VEC, int TPR, int K, int R>
gdn_status run_gate(GateNormParams &np, int64_t rows, hipStream_t s) {
    if constexpr (BWD) {
        return launch_kernel((const void *)&gate_norm_backward_kernel<IO, VEC, TPR, K>, (int)rows, &np, s, kGateThreads<TPR>);
    } else {
        constexpr int kPer = kGateThreads<TPR> / TPR * R;
        return launch_kernel((const void *)&gate_norm_forward_kernel<IO, VEC, TPR, K, R>, (int)((rows + kPer - 1) / kPer), &np, s,
                             kGateThreads<TPR>);
    }
}

template <bool BWD, typename IO, int VEC>
gdn_status gate_d(GateNormParams &np, int64_t rows, hipStream_t s) {
    const int D = np.D;
    constexpr int M = 4 / VEC;
    if (D <= 64) return run_gate<BWD, IO, VEC, 16, M, 4>(np, rows, s);
    if (D <= 128) return run_gate<BWD, IO, VEC, 32, M, 4>(np, rows, s);
    if (D <= 256) return run_gate<BWD, IO, VEC, 64, M, 4>(np, rows, s);
    if (D <= 512) return run_gate<BWD, IO, VEC, 64, 2 * M, 2>(np, rows, s);
    if (D <= 1024) return run_gate<BWD, IO, VEC, 256, M, 1>(np, rows, s);
    if (D <= 2048) return run_gate<BWD, IO, VEC, 256, 2 * M, 1>(np, rows, s);
    if (D <= 4096) return run_gate<BWD, IO, VEC, 512, 2 * M, 1>(np, rows, s);
    return run_gate<BWD, IO, VEC, 1024, 2 * M, 1>(np, rows, s);
}

template <bool BWD>
gdn_status gate_types(const gdn_gate_norm_problem *pr, GateNormParams &np, bool vec, int64_t rows, hipStream_t s) {
    if (pr->io_dtype == GDN_F32) return vec ? gate_d<BWD, float, 4>(np, rows, s) : gate_d<BWD, float, 1>(np, rows, s);
    return vec ? gate_d<BWD, bf16_t, 4>(np, rows, s) : gate_d<BWD, bf16_t, 1>(np, rows, s);
}

void fill_gate(const gdn_gate_norm_problem *pr, GateNormParams &np) {
    np = GateNormParams{};
    np.xt = pr->x_stride_t;
    np.xh = pr->x_stride_h;
    np.zt = pr->z_stride_t;
    np.zh = pr->z_stride_h;
    np.dzt = pr->dz_stride_t;
    np.dzh = pr->dz_stride_h;
    np.H = (uint32_t)pr->H;
    np.classes = (uint32_t)gate_classes(pr);
    np.D = (int)pr->D;
    np.w_f32 = pr->w_dtype == GDN_F32;
    np.first = pr->gate_first != 0;
    np.center = pr->center != 0;
    np.silu = pr->act == GDN_ACT_SILU;
    np.eps = pr->eps;
    np.inv_d = 1.f / (float)pr->D;
}

// Whether every row begins at four aligned elements.
bool gate_vec(const gdn_gate_norm_problem *pr, std::initializer_list<const void *> io, const void *weight, const void *bias) {
    const size_t eb = dtype_bytes(pr->io_dtype), wb = dtype_bytes(pr->w_dtype);
    if (pr->D % 4 != 0 || !aligned_to(weight, 4 * wb) || !aligned_to(bias, 4 * wb)) return false;
    for (int64_t v : {pr->x_stride_t, pr->x_stride_h, pr->z_stride_t, pr->z_stride_h, pr->dz_stride_t, pr->dz_stride_h})
        if (v % 4 != 0) return false;
    for (const void *q : io)
        if (!aligned_to(q, 4 * eb)) return false;
    return true;
}

bool gate_aligned(const gdn_gate_norm_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> w) {
    for (const void *q : io)
        if (!aligned_to(q, dtype_bytes(pr->io_dtype))) return false;
    for (const void *q : w)
        if (!aligned_to(q, dtype_bytes(pr->w_dtype))) return false;
    return true;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_gate_norm_forward(const gdn_gate_norm_problem *pr, const void *x, const void *z, const void *weight,
                                 const void *bias, void *y, void *stream) {
    gdn_status st = check_gate_norm(pr);
    if (st != GDN_OK) return st;
    if (!pr->center && bias) return GDN_ERR_UNSUPPORTED;
    const int64_t rows = pr->T * pr->H;
    if (rows == 0) return GDN_OK;
    if (!x || !z || !weight || !y) return GDN_ERR_NULL_ARG;
    if (!gate_aligned(pr, {x, z, y}, {weight, bias})) return GDN_ERR_ALIGNMENT;
    GateNormParams np;
    fill_gate(pr, np);
    np.x = x;
    np.z = z;
    np.w = weight;
    np.b = bias;
    np.y = y;
    np.dzt = np.dzh = 0;
    gdn_gate_norm_problem own = *pr;
    own.dz_stride_t = own.dz_stride_h = 0;
    const bool vec = gate_vec(&own, {x, z, y}, weight, bias);
    // (as many launches as rows need; one up to kGateRows)
    for (int64_t r = 0; r < rows; r += kGateRows) {
        np.row0 = r;
        np.rows = rows - r < kGateRows ? rows : r + kGateRows;
        st = gate_types<false>(pr, np, vec, np.rows - r, (hipStream_t)stream);
        if (st != GDN_OK) return st;
    }
    return GDN_OK;
}

size_t gdn_workspace_bytes_gate_norm_backward(const gdn_gate_norm_problem *pr) {
    if (check_gate_norm(pr) != GDN_OK) return 0;
    return (size_t)(gate_parts(pr) * gate_classes(pr)) * pr->D * 8;
}

gdn_status gdn_gate_norm_backward(const gdn_gate_norm_problem *pr, const void *dy, const void *x, const void *z,
                                  const void *weight, const void *bias, void *dx, void *dz, float *dweight, float *dbias,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_gate_norm(pr);
    if (st != GDN_OK) return st;
    if (!pr->center && (bias || dbias)) return GDN_ERR_UNSUPPORTED;
    if (!weight || !dweight) return GDN_ERR_NULL_ARG;
    if (pr->T > 0 && (!dy || !x || !z || !dx || !dz)) return GDN_ERR_NULL_ARG;
    if (!gate_aligned(pr, {dy, x, z, dx, dz}, {weight, bias}) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_workspace_bytes_gate_norm_backward(pr);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    GateNormParams np;
    fill_gate(pr, np);
    np.dy = dy;
    np.x = x;
    np.z = z;
    np.w = weight;
    np.b = bias;
    np.dx = dx;
    np.dz = dz;
    np.part = (float *)workspace;
    const int64_t classes = gate_classes(pr);
    np.rows = pr->T * pr->H / classes;
    np.parts = (int)gate_parts(pr);
    st = gate_types<true>(pr, np, gate_vec(pr, {dy, x, z, dx, dz}, weight, bias), np.parts * classes, (hipStream_t)stream);
    if (st != GDN_OK) return st;
    return enqueue_norm_sums(np.part, dweight, dbias, pr->D, np.parts, classes, (hipStream_t)stream);
}

}  // extern "C"

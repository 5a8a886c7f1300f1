// Gated norm: rows of D elements x with a gate z of their own.
//
//   n(v) = (v - m) r w + b,  m = mean v (or 0),  r = (mean (v - m)^2 + eps)^(-1/2)
//   gate first:  y = n(x act(z));   else  y = n(x) act(z)
// Backward, with h = (v - m) r, dn = dy (gate first) or dy act(z), u = dn w:
//   dv = r (u - mean u - h mean(u h))     (mean u only where m is taken)
//   dx, dz = dv act(z), dv x act'(z)      or  dv, dy (h w + b) act'(z)
//   dw = sum dn h,  db = sum dn over the rows that share w
//
// Bound by memory: every tensor is read or written once (16384 tokens of 64 rows of 128 in
// bf16 forward 160 us, 5.0 TB/s; 16384 of 4 rows of 1024, gate first, forward 91 us, 4.4
// TB/s, backward 152 us, 4.4 TB/s, and 4.8 us the sums; 4096 rows of 128 4 us, a launch's own time; rows of
// single elements as fast as of four: 16384 of 1030 26.0 us forward, of 1028 26.5).  TPR threads hold a
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
    uint32_t H, inv_h, classes;                      // inv_h: 2^32 / H, rounded down
    int D, parts, w_f32, silu;
    int64_t row0;                                    // first row of each class in this launch (forward)
    float eps, inv_d;
};

// VEC elements of a row at its element e, or at its first where it has none there
// (so that no branch stands around a load): keep() makes those zero.
template <typename T, int VEC>
__device__ __forceinline__ void fetch_row(RawRow<T, VEC> &r, const T *row, uint32_t e, uint32_t D) {
    row += e < D ? e : 0;
    if constexpr (VEC * sizeof(T) == 2) {
        r.u[0] = *(const uint16_t *)row;
    } else if constexpr (VEC * sizeof(T) == 4) {
        r.u[0] = *(const uint32_t *)row;
    } else if constexpr (VEC * sizeof(T) == 8) {
        const u32x2 v = *(const u32x2 *)row;
        r.u[0] = v[0];
        r.u[1] = v[1];
    } else {
        const u32x4 v = *(const u32x4 *)row;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.u[i] = v[i];
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void keep(RawRow<T, VEC> &r, bool ok) {
#pragma unroll
    for (auto &v : r.u) v = ok ? v : 0;
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

// Row `at` of all as token t and head h.
__device__ __forceinline__ void token_head(const GateNormParams &p, uint32_t at, uint32_t &t, uint32_t &h) {
    // (the product falls short of the quotient by less than 2)
    t = __umulhi(at, p.inv_h);
    h = at - t * p.H;
    if (h >= p.H) {
        ++t;
        h -= p.H;
    }
}

// act(z) and act'(z); for bf16 the exponential's last digits do not matter.
template <typename IO>
struct Act {
    float a, d;
    __device__ __forceinline__ Act(float z, int silu) {
        const Sigmoid<sizeof(IO) == 4> g(z);
        a = silu ? z * g.s : g.s;
        d = silu ? fmaf(z * g.s, g.o, g.s) : g.s * g.o;
    }
};

// Sums over the TPR threads of a slot, in every one of them; red has N TPR / 64 places.
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

// v -> v - mean v of each of R rows, where it has elements
template <int VEC, int TPR, int K, int R>
__device__ __forceinline__ void slot_mean(float (&v)[R][K][VEC], uint32_t D, int tid, float inv_d, float *red) {
    float t[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        t[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) t[j] += v[j][k][i];
    }
    slot_total<TPR>(t, red);
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][k][i] = (uint32_t)((k * TPR + tid) * VEC) < D ? v[j][k][i] - t[j] * inv_d : 0.f;
}

__device__ __forceinline__ float inverse_root(float ms, float eps) { return 1.f / sqrtf((ms < 0.f ? 0.f : ms) + eps); }

// A slot (TPR threads) has R rows in flight, of one class (rows that share their weights:
// all, or one head's), and works on them together.
template <typename IO, int VEC, int TPR, int K, int R, bool FIRST, bool CENTER>
__global__ void __launch_bounds__(kGateThreads<TPR>) gate_norm_forward_kernel(GateNormParams p) {
    constexpr int kSlots = kGateThreads<TPR> / TPR;
    __shared__ float red[3 * R * (TPR < 64 ? 1 : TPR / 64)];
    const int slot = threadIdx.x / TPR, tid = threadIdx.x % TPR;
    const uint32_t D = p.D;
    const uint32_t cls = blockIdx.x % p.classes, block = blockIdx.x / p.classes;
    RawRow<IO, VEC> xr[R][K], zr[R][K];
    // rows i0 + j kSlots of this class: row i classes + cls of all
    const int64_t i0 = p.row0 + (int64_t)block * (kSlots * R) + slot;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int64_t i = i0 + j * kSlots;
        uint32_t t, h;
        token_head(p, i < p.rows ? (uint32_t)(i * p.classes + cls) : 0, t, h);
        const IO *xp = (const IO *)p.x + t * p.xt + h * p.xh, *zp = (const IO *)p.z + t * p.zt + h * p.zh;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t e = (k * TPR + tid) * VEC;
            fetch_row(xr[j][k], xp, e, D);
            fetch_row(zr[j][k], zp, e, D);
        }
    }
    const uint32_t wb = p.w_f32 ? 4 : (uint32_t)sizeof(IO);
    const rsrc_t rw = make_rsrc((const char *)p.w + (int64_t)cls * D * wb, D * wb),
                 rb = make_rsrc((const char *)p.b + (p.b ? (int64_t)cls * D * wb : 0), p.b ? D * wb : 0);
    float w[K][VEC], b[K][VEC];
    load_affine<IO, VEC, K>(rw, rb, p.w_f32, tid * VEC, TPR * VEC, w, b);
    float v[R][K][VEC], g[R][K][VEC], t[2 * R];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            // (a row past the end is the first one again, and is not stored)
            keep(xr[j][k], (uint32_t)((k * TPR + tid) * VEC) < D);
            keep(zr[j][k], (uint32_t)((k * TPR + tid) * VEC) < D);
            xr[j][k].get(v[j][k]);
            zr[j][k].get(g[j][k]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float a = Act<IO>(g[j][k][i], p.silu).a;
                if (FIRST) v[j][k][i] *= a;
                g[j][k][i] = FIRST ? 1.f : a;
            }
        }
    if (CENTER) slot_mean<VEC, TPR, K, R>(v, D, tid, p.inv_d, red);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        t[2 * j] = t[2 * j + 1] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                t[2 * j] += v[j][k][i] * v[j][k][i];
                t[2 * j + 1] += v[j][k][i];
            }
    }
    slot_total<TPR>(t, red + R * (TPR < 64 ? 1 : TPR / 64));
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int64_t i1 = i0 + j * kSlots;
        const float m = CENTER ? t[2 * j + 1] * p.inv_d : 0.f;
        const float r = inverse_root(t[2 * j] * p.inv_d - m * m, p.eps);
        const uint32_t end = i1 < p.rows ? D : 0;
        IO *y = (IO *)p.y + (i1 * p.classes + cls) * D;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][k][i] = fmaf((v[j][k][i] - m) * r, w[k][i], b[k][i]) * g[j][k][i];
            put_row<IO, VEC>(y, (k * TPR + tid) * VEC, end, v[j][k]);
        }
    }
}

// A class's rows go to its workgroups' slots in turn; the slots' shares of dw and db stay in
// registers and meet in LDS, and every workgroup leaves one row of D sums of
// each in the workspace.  The next R rows are in flight while R are worked on
// (not where rows of more than 4096 elements fill the registers).
template <typename IO, int VEC, int TPR, int K, int R, bool FIRST, bool CENTER>
__global__ void __launch_bounds__(kGateThreads<TPR>) gate_norm_backward_kernel(GateNormParams p) {
    constexpr int kSlots = kGateThreads<TPR> / TPR;
    constexpr int kW = TPR < 64 ? 1 : TPR / 64;
    constexpr bool kAhead = K * VEC * R <= 8;
    __shared__ float red[2][5 * R * kW];
    __shared__ float sums[TPR < 256 ? 4 : 1][TPR < 256 ? 2 : 1][TPR < 256 ? TPR * K * VEC : 1];
    const int slot = threadIdx.x / TPR, tid0 = threadIdx.x % TPR;
    int tid = tid0;
    const uint32_t D = p.D, cls = blockIdx.x % p.classes, part = blockIdx.x / p.classes;
    const uint32_t wb = p.w_f32 ? 4 : (uint32_t)sizeof(IO);
    const rsrc_t rw = make_rsrc((const char *)p.w + (int64_t)cls * D * wb, D * wb),
                 rb = make_rsrc((const char *)p.b + (p.b ? (int64_t)cls * D * wb : 0), p.b ? D * wb : 0);
    // a vector of the weights: kept, or loaded again where it is used
    float kw[kAhead ? K : 1][VEC], kb[kAhead ? K : 1][VEC], dw[K][VEC], db[K][VEC];
    // (without a branch: of the two types' descriptors one is empty, and reads zeros)
    const rsrc_t rw4 = make_rsrc((const char *)p.w + (int64_t)cls * D * wb, wb == 4 ? D * 4 : 0),
                 rw2 = make_rsrc((const char *)p.w + (int64_t)cls * D * wb, wb == 2 ? D * 2 : 0),
                 rb4 = make_rsrc((const char *)p.b + (p.b ? (int64_t)cls * D * wb : 0), p.b && wb == 4 ? D * 4 : 0),
                 rb2 = make_rsrc((const char *)p.b + (p.b ? (int64_t)cls * D * wb : 0), p.b && wb == 2 ? D * 2 : 0);
    auto load_both = [&](rsrc_t r4, rsrc_t r2, int k, float (&w)[VEC]) {
        RawRow<float, VEC> a4;
        RawRow<bf16_t, VEC> a2;
        float w2[VEC];
        a4.load(r4, tid0 * VEC * 4, k * TPR * VEC * 4);
        a2.load(r2, tid0 * VEC * 2, k * TPR * VEC * 2);
        a4.get(w);
        a2.get(w2);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = __uint_as_float(__float_as_uint(w[i]) | __float_as_uint(w2[i]));
    };
    auto weights = [&](int k, float (&w)[VEC], float (&b)[VEC]) {
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                w[i] = kw[k][i];
                b[i] = kb[k][i];
            }
        } else {
            __builtin_amdgcn_sched_barrier(0);      // no loads ahead
            load_both(rw4, rw2, k, w);
            load_both(rb4, rb2, k, b);
        }
    };
    if constexpr (kAhead) load_affine<IO, VEC, K>(rw, rb, p.w_f32, tid * VEC, TPR * VEC, kw, kb);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.f;
    RawRow<IO, VEC> xn[R][K], zn[R][K], dn[R][K];
    // rows i + j kSlots of this class: row i classes + cls of all
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool live = i + j * kSlots < p.rows;
            const uint32_t at = live ? (uint32_t)((i + j * kSlots) * p.classes + cls) : 0;
            uint32_t t, h;
            token_head(p, at, t, h);
            const IO *xp = (const IO *)p.x + t * p.xt + h * p.xh, *zp = (const IO *)p.z + t * p.zt + h * p.zh,
                     *dp = (const IO *)p.dy + (int64_t)at * D;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const uint32_t e = (k * TPR + tid) * VEC;
                fetch_row(xn[j][k], xp, e, D);
                fetch_row(zn[j][k], zp, e, D);
                fetch_row(dn[j][k], dp, e, D);
            }
        }
    };
    // (all slots of a workgroup make the same number of turns: rows of several waves meet at barriers)
    const int64_t step = (int64_t)p.parts * (kSlots * R);
    int64_t i0 = (int64_t)part * (kSlots * R);
    if (kAhead) fetch(i0 + slot);
    int turn = 0;
    for (; i0 < p.rows; i0 += step) {
        if constexpr (!kAhead) {
            // (offsets formed in the loop: kept, they would fill the registers)
            asm volatile("" : "+v"(tid));
            fetch(i0 + slot);
        }
        // v: the row that is normed; d: dy; act(z) and act'(z)
        float x[R][K][VEC], v[R][K][VEC], d[R][K][VEC], ga[R][K][VEC], gd[R][K][VEC], t[4 * R];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float z[VEC];
                // (nor does a row past the end enter the sums)
                const bool ok = i0 + slot + j * kSlots < p.rows && (uint32_t)((k * TPR + tid) * VEC) < D;
                keep(xn[j][k], ok);
                keep(zn[j][k], ok);
                keep(dn[j][k], ok);
                xn[j][k].get(x[j][k]);
                zn[j][k].get(z);
                dn[j][k].get(d[j][k]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const Act<IO> g(z[i], p.silu);
                    ga[j][k][i] = g.a;
                    gd[j][k][i] = g.d;
                    v[j][k][i] = FIRST ? x[j][k][i] * g.a : x[j][k][i];
                }
            }
        if (kAhead) fetch(i0 + step + slot);
        if (CENTER) slot_mean<VEC, TPR, K, R>(v, D, tid, p.inv_d, red[turn]);
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q) t[4 * j + q] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float w[VEC], b[VEC];
                weights(k, w, b);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = (FIRST ? d[j][k][i] : d[j][k][i] * ga[j][k][i]) * w[i];
                    t[4 * j] += v[j][k][i] * v[j][k][i];
                    t[4 * j + 1] += u * v[j][k][i];
                    t[4 * j + 2] += v[j][k][i];
                    t[4 * j + 3] += u;
                }
            }
        }
        slot_total<TPR>(t, red[turn] + R * kW);
        turn ^= 1;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t i1 = i0 + slot + j * kSlots;
            const bool live = i1 < p.rows;
            const uint32_t at = live ? (uint32_t)(i1 * p.classes + cls) : 0;
            uint32_t t0, hd;
            token_head(p, at, t0, hd);
            const float m = CENTER ? t[4 * j + 2] * p.inv_d : 0.f, mu = CENTER ? t[4 * j + 3] * p.inv_d : 0.f;
            const float r = inverse_root(t[4 * j] * p.inv_d - m * m, p.eps);
            const float c = r * (t[4 * j + 1] * p.inv_d - m * (t[4 * j + 3] * p.inv_d));
            IO *xo = (IO *)p.dx + (int64_t)at * D, *zo = (IO *)p.dz + t0 * p.dzt + hd * p.dzh;
            const uint32_t end = live ? D : 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const uint32_t e = (k * TPR + tid) * VEC;
                float dx[VEC], dz[VEC], w[VEC], b[VEC];
                weights(k, w, b);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float h = (v[j][k][i] - m) * r, dd = FIRST ? d[j][k][i] : d[j][k][i] * ga[j][k][i];
                    const float dv = r * (dd * w[i] - mu - h * c);
                    dw[k][i] += dd * h;
                    db[k][i] += dd;
                    dx[i] = FIRST ? dv * ga[j][k][i] : dv;
                    dz[i] = (FIRST ? dv * x[j][k][i] : d[j][k][i] * fmaf(h, w[i], b[i])) * gd[j][k][i];
                }
                put_row<IO, VEC>(xo, e, end, dx);
                put_row<IO, VEC>(zo, e, end, dz);
            }
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

constexpr int64_t kGateRows = 1 << 21;     // a forward launch's, under 2^32 threads
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
int gate_tpr(int64_t D) { return D <= 64 ? 16 : D <= 128 ? 32 : D <= 512 ? 64 : D <= 2048 ? 256 : 512; }
// rows that a workgroup of the backward pass works on at a time (see gate_d)
int gate_slots(int64_t D) {
    return (gate_tpr(D) < 256 ? 256 / gate_tpr(D) : 1) * (D <= 256 || (D > 512 && D <= 1024) ? 2 : 1);
}

// Workgroups of a class in the backward pass.
int64_t gate_parts(const gdn_gate_norm_problem *pr) {
    const int64_t c = gate_classes(pr), rows = pr->T * pr->H / c, n = (rows + gate_slots(pr->D) - 1) / gate_slots(pr->D);
    int64_t most = kGateWgs / c;
    most = most < 1 ? 1 : most;
    const int64_t turns = (n + most - 1) / most;
    return turns ? (n + turns - 1) / turns : 0;
}

struct GateForm {
    bool first, center;
};

template <bool BWD, typename IO, int VEC, int TPR, int K, int R, bool FIRST, bool CENTER>
gdn_status run_gate(GateNormParams &np, int64_t rows, hipStream_t s) {
    if constexpr (BWD) {
        return launch_kernel((const void *)&gate_norm_backward_kernel<IO, VEC, TPR, K, R, FIRST, CENTER>, (int)rows, &np, s, kGateThreads<TPR>);
    } else {
        constexpr int kPer = kGateThreads<TPR> / TPR * R;
        return launch_kernel((const void *)&gate_norm_forward_kernel<IO, VEC, TPR, K, R, FIRST, CENTER>, (int)((rows + kPer - 1) / kPer * np.classes), &np, s,
                             kGateThreads<TPR>);
    }
}

template <bool BWD, typename IO, int VEC, int TPR, int K, int R>
gdn_status gate_form(GateNormParams &np, GateForm f, int64_t rows, hipStream_t s) {
    if (f.first) return f.center ? run_gate<BWD, IO, VEC, TPR, K, R, true, true>(np, rows, s) : run_gate<BWD, IO, VEC, TPR, K, R, true, false>(np, rows, s);
    return f.center ? run_gate<BWD, IO, VEC, TPR, K, R, false, true>(np, rows, s) : run_gate<BWD, IO, VEC, TPR, K, R, false, false>(np, rows, s);
}

// Rows of a slot at a time: forward 16 elements a thread in flight, backward 8 (of three
// tensors; 16 take 280 registers).
template <bool BWD, typename IO, int VEC>
gdn_status gate_d(GateNormParams &np, GateForm f, int64_t rows, hipStream_t s) {
    const int D = np.D;
    constexpr int M = 4 / VEC, R = BWD ? 2 : 4;
    if (D <= 64) return gate_form<BWD, IO, VEC, 16, M, R>(np, f, rows, s);
    if (D <= 128) return gate_form<BWD, IO, VEC, 32, M, R>(np, f, rows, s);
    if (D <= 256) return gate_form<BWD, IO, VEC, 64, M, R>(np, f, rows, s);
    if (D <= 512) return gate_form<BWD, IO, VEC, 64, 2 * M, R / 2>(np, f, rows, s);
    if (D <= 1024) return gate_form<BWD, IO, VEC, 256, M, R>(np, f, rows, s);
    if (D <= 2048) return gate_form<BWD, IO, VEC, 256, 2 * M, R / 2>(np, f, rows, s);
    if (D <= 4096) return gate_form<BWD, IO, VEC, 512, 2 * M, R / 2>(np, f, rows, s);
    if constexpr (BWD)
        return gate_form<BWD, IO, VEC, 512, 4 * M, 1>(np, f, rows, s);
    else
        return gate_form<BWD, IO, VEC, 1024, 2 * M, 1>(np, f, rows, s);
}

template <bool BWD>
gdn_status gate_types(const gdn_gate_norm_problem *pr, GateNormParams &np, bool vec, int64_t rows, hipStream_t s) {
    const GateForm f{pr->gate_first != 0, pr->center != 0};
    if (pr->io_dtype == GDN_F32) return vec ? gate_d<BWD, float, 4>(np, f, rows, s) : gate_d<BWD, float, 1>(np, f, rows, s);
    return vec ? gate_d<BWD, bf16_t, 4>(np, f, rows, s) : gate_d<BWD, bf16_t, 1>(np, f, rows, s);
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
    np.inv_h = pr->H == 1 ? 0xffffffffu : (uint32_t)(((uint64_t)1 << 32) / pr->H);
    np.classes = (uint32_t)gate_classes(pr);
    np.D = (int)pr->D;
    np.w_f32 = pr->w_dtype == GDN_F32;
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
    const int64_t classes = gate_classes(pr), each = rows / classes, step = kGateRows / classes;
    for (int64_t r = 0; r < each; r += step) {
        np.row0 = r;
        np.rows = each - r < step ? each : r + step;
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

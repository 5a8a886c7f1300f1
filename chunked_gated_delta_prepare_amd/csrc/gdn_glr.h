// Gated linear recurrence of single channels: what its passes share.
//
//   h_t = a_t h_{t-1} + u_t,  u_t = c_t x_t
//
// A run of tokens moves a state h to A h + H with A the product of its a's and
// H its end from zero; two runs behind each other are (A1 A2, H2 + A2 H1).  So
// every thread takes a few consecutive tokens of VEC channels, the threads'
// runs are put together in a wave (shuffles) and in a workgroup (LDS), and a
// long sequence is cut into segments whose runs meet in the workspace.
//
// Memories of thousands of tokens: A is kept as the product P and as the lack
// C = 1 - A, C12 = C1 + C2 - C1 C2, from 1 - a of log a itself.  Where C < 1/2 the
// state moves as h - C h: a product of a's rounded near 1 would lose a digit
// for every hundred tokens.
//
// Layout of a wave: 64 channels innermost, 4 bytes a lane where rows allow it
// (VEC = 2 channels of bf16 in CL = 32 lanes; else VEC = 1, CL = 64), and TG =
// 64 / CL groups of lanes behind each other that take runs of L consecutive
// tokens.  (8 bytes a lane would make four groups, and twice the joining.)
#pragma once

#include <initializer_list>

#include "gdn_layer.h"

namespace gdn {

constexpr int kGlrCols = 64;                   // channels of a workgroup

struct GlrParams {
    const void *x, *g, *dy;
    const float *bias, *rate, *h0, *dhT;
    const int32_t *cu, *slots;
    void *y, *dx, *dg;
    float *state, *hT, *dh0, *ws, *part;
    int64_t xb, xt, gb, gt, yb, yt, dxb, dxt, dgb, dgt;      // strides (y: dy)
    int64_t n_slots, n_states;                               // states: B or n_seqs
    int B, T, D, n_seqs, scale;
    int groups, segs, seg_len;                               // channels / 64; segments (backward: tiles)
    int grads;                                               // whether dbias or drate is wanted
};

// ---------------------------------------------------------------------------
// gates
// ---------------------------------------------------------------------------

// 1 - e^z, and e^z.  |z| < 1/2: the series -z (1 + z/2 + ... + z^7/8!), whose next term is
// below 2^-26 of it; else 1 - e^z is at least 0.39 and loses a bit.
__device__ __forceinline__ void decay_of_log(float z, float &a, float &c) {
    float s = fmaf(z, 1.f / 40320.f, 1.f / 5040.f);
    s = fmaf(z, s, 1.f / 720.f);
    s = fmaf(z, s, 1.f / 120.f);
    s = fmaf(z, s, 1.f / 24.f);
    s = fmaf(z, s, 1.f / 6.f);
    s = fmaf(z, s, 0.5f);
    s = fmaf(z, s, 1.f) * -z;
    const float e = exact_exp(z);
    const bool small = fabsf(z) < 0.5f;
    c = small ? s : 1.f - e;
    a = small ? 1.f - s : e;
}

// A token's decay a, c = 1 - a, and for the gradients d(log a)/d(gate) (slope) and the
// gate's sigmoid (GDN_GLR_RATE).
template <int FORM>
__device__ __forceinline__ void gate_of(float v, float rate, float &a, float &c, float &slope, float &sig) {
    if constexpr (FORM == GDN_GLR_LOG) {
        decay_of_log(v, a, c);
        slope = 1.f;
        sig = 0.f;
    } else {
        const Sigmoid g(v);
        if constexpr (FORM == GDN_GLR_SIGMOID) {
            a = g.s;
            c = g.o;
            slope = g.o;
            sig = 0.f;
        } else {
            const float la = -rate * g.s;
            decay_of_log(la, a, c);
            slope = la * g.o;
            sig = g.s;
        }
    }
}

// The input's factor.
__device__ __forceinline__ float input_scale(int scale, float a, float c) {
    return scale == GDN_GLR_PLAIN ? 1.f : scale == GDN_GLR_COMPLEMENT ? c : __builtin_amdgcn_sqrtf(c * (1.f + a));
}
// Its derivative by log a, for the factor k.
__device__ __forceinline__ float input_slope(int scale, float a, float k) {
    if (scale == GDN_GLR_PLAIN) return 0.f;
    if (scale == GDN_GLR_COMPLEMENT) return -a;
    return k > 0.f ? -a * a * __builtin_amdgcn_rcpf(k) : k == 0.f ? 0.f : k;      // (a NaN stays one)
}

// ---------------------------------------------------------------------------
// runs
// ---------------------------------------------------------------------------

// The moves of VEC channels over a run.  P < 0 marks a run in which a sequence
// begins (packed): what comes before it does not pass.
template <int VEC>
struct Moves {
    float P[VEC], C[VEC];
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            P[i] = 1.f;
            C[i] = 0.f;
        }
    }
};

// A h + H
template <bool PK>
__device__ __forceinline__ float move(float P, float C, float h, float H) {
    const bool near = C >= 0.f && C < 0.5f;
    const float m = near ? fmaf(-C, h, h) + H : fmaf(P, h, H);
    return PK && P < 0.f ? H : m;
}
// run 1, then run 2
template <bool PK>
__device__ __forceinline__ void join(float P1, float C1, float P2, float C2, float &P, float &C) {
    C = C1 + fmaf(-C1, C2, C2);
    P = PK && (P1 < 0.f || P2 < 0.f) ? -1.f : P1 * P2;
}

// The same in one number, for LDS and the workspace: C where it is in [0, 1/2), else -P (its
// sign bit set); -inf for a run in which a sequence begins.
template <bool PK>
__device__ __forceinline__ float pack_move(float P, float C) {
    if (PK && P < 0.f) return -__builtin_inff();
    return C >= 0.f && C < 0.5f ? fabsf(C) : -P;
}
template <bool PK>
__device__ __forceinline__ float packed_move(float q, float h, float H) {
    const bool far = __float_as_int(q) < 0;
    const float m = fmaf(-q, h, far ? H : h), r = far ? m : m + H;
    return PK && q == -__builtin_inff() ? H : r;
}

// The value of the lane with the other token of lane bit 5 (lane ^ 32).
__device__ __forceinline__ float other_half(float x) {
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(lane_id() & 32 ? h[0] : h[1]);
}

// ---------------------------------------------------------------------------
// sequences
// ---------------------------------------------------------------------------

__device__ __forceinline__ int cu_at(const GlrParams &p, int n) {
    const int v = p.cu[n];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

// The last packed sequence that begins at or before token t.
__device__ __forceinline__ int seq_of(const GlrParams &p, int t) {
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu_at(p, mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Of a thread's L tokens from t0: which exist and are in a sequence, which are the
// first and the last of one.
struct Marks {
    uint32_t valid, first, last;
};
// A packed sequence's rows, kept from run to run.
struct Span {
    int n = 0, begin = 0, end = 0;
    __device__ __forceinline__ void at(const GlrParams &p, int t) {
        if (t >= begin && t < end) return;
        n = seq_of(p, t);
        begin = cu_at(p, n);
        end = cu_at(p, n + 1);
    }
};
template <bool PK, int L>
__device__ __forceinline__ Marks marks_of(const GlrParams &p, int t0, Span &s) {
    constexpr uint32_t kAll = (1u << L) - 1;
    const int n = p.T - t0;
    const uint32_t exist = n >= L ? kAll : n <= 0 ? 0 : (1u << n) - 1;
    Marks m{exist, 0, 0};
    if constexpr (!PK) {
        m.first = t0 == 0 ? 1 & exist : 0;
        m.last = n >= 1 && n <= L ? 1u << (n - 1) : 0;
    } else if (exist) {
        s.at(p, t0);
        if (!(s.begin < t0 && t0 + L < s.end)) {
            m.valid = 0;
#pragma unroll 1
            for (int i = 0; i < L && t0 + i < p.T; ++i) {
                const int t = t0 + i;
                s.at(p, t);
                const uint32_t in = t >= s.begin && t < s.end ? 1u << i : 0;
                m.valid |= in;
                if (t == s.begin) m.first |= in;
                if (t == s.end - 1) m.last |= in;
            }
        }
    }
    return m;
}
// The sequence of token t: its number (packed), else the batch.
template <bool PK>
__device__ __forceinline__ int state_of(const GlrParams &p, int b, int t) {
    return PK ? seq_of(p, t) : b;
}

// Sequences without a token hand their state through: out[n] = in[n] (or zero).
__device__ __forceinline__ void pass_empty(const GlrParams &p, bool packed, int b, int c0, const float *in, float *out) {
    if (!out) return;
    const int n0 = packed ? 0 : b, n1 = packed ? p.n_seqs : b + 1;
    const int c = c0 + (int)(threadIdx.x & 63);
    for (int n = n0 + (int)(threadIdx.x >> 6); n < n1; n += (int)(blockDim.x >> 6)) {
        const bool empty = packed ? cu_at(p, n) >= cu_at(p, n + 1) : p.T == 0;
        if (empty && c < p.D) out[(int64_t)n * p.D + c] = in ? in[(int64_t)n * p.D + c] : 0.f;
    }
}

// A lane's place: VEC channels from c, in token group tg of its wave.
template <int VEC>
struct GlrLane {
    static constexpr int kCL = kGlrCols / VEC, kTG = 64 / kCL;
    int c, tg;
    __device__ __forceinline__ explicit GlrLane(int group) {
        c = group * kGlrCols + (lane_id() % kCL) * VEC;
        tg = lane_id() / kCL;
    }
    __device__ __forceinline__ int local() const { return (lane_id() % kCL) * VEC; }      // among the workgroup's channels
};

// An offset past every descriptor here (rows' offsets are below 2^30 bytes).
constexpr uint32_t kNowhere = 0x80000000u;

// A lane's VEC (1, or 2 of bf16) columns in rows at one stride, from its own first
// row on; rows that are not ok, and columns behind the last, read as zero and are
// not stored.
template <typename T, int VEC>
struct TileRows {
    static_assert(VEC * sizeof(T) <= 4, "a lane's columns are 4 bytes");
    rsrc_t r;
    uint32_t off, pitch;
    __device__ __forceinline__ TileRows(const void *base, int64_t elems, int64_t stride, int row, int c, int D) {
        r = make_rsrc((const T *)base + elems, kNowhere);
        pitch = (uint32_t)stride * sizeof(T);
        off = c < D ? (uint32_t)c * sizeof(T) + (uint32_t)row * pitch : kNowhere;
    }
    __device__ __forceinline__ void load(RawRow<T, VEC> &x, int i, bool ok) const { x.load(r, ok ? off : kNowhere, i * pitch); }
    __device__ __forceinline__ void store(const float (&x)[VEC], int i, bool ok) const {
        if constexpr (VEC == 2)
            bstore32(pack_bf16(x[0], x[1]), r, ok ? off : kNowhere, i * pitch);
        else
            BufElem<T>::store(x[0], r, ok ? off : kNowhere, i * pitch);
    }
};

// A lane's VEC values of a state [n_states][D] fp32.
template <int VEC>
__device__ __forceinline__ void state_load(const GlrParams &p, const float *s, int n, int c, float (&x)[VEC]) {
    const rsrc_t r = make_rsrc(s, s ? (uint32_t)(p.n_states * p.D) * 4 : 0);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        x[i] = __uint_as_float(bload32(r, c + i < p.D ? ((uint32_t)n * p.D + c + i) * 4 : kNowhere, 0));
}
template <int VEC>
__device__ __forceinline__ void state_store(const GlrParams &p, float *s, int n, int c, bool ok, const float (&x)[VEC]) {
    const rsrc_t r = make_rsrc(s, s ? (uint32_t)(p.n_states * p.D) * 4 : 0);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        bstore32(__float_as_uint(x[i]), r, ok && c + i < p.D ? ((uint32_t)n * p.D + c + i) * 4 : kNowhere, 0);
}

// A lane's VEC channel weights (fp32), zero without any.
template <int VEC>
__device__ __forceinline__ void channel_load(const float *w, int c, int D, float (&x)[VEC]) {
    row_load<float, VEC>(make_rsrc(w, w ? (uint32_t)D * 4 : 0), c, x);
}

// A thread's run: a and u = c x of its L tokens, and where they move a state.
template <typename IO, typename GT, int VEC, int FORM, int L>
struct Run {
    RawRow<IO, VEC> x[L];
    RawRow<GT, VEC> g[L];
    float a[L][VEC], u[L][VEC], H[VEC];
    Moves<VEC> m;

    // rows of the run's first token on; `exist` of them do
    __device__ __forceinline__ void fetch(const GlrParams &p, int b, int t_base, int row, int c) {
        const TileRows<IO, VEC> rx(p.x, b * p.xb + (int64_t)t_base * p.xt, p.xt, row, c, p.D);
        const TileRows<GT, VEC> rg(p.g, b * p.gb + (int64_t)t_base * p.gt, p.gt, row, c, p.D);
        const int n = p.T - t_base - row;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            rx.load(x[i], i, i < n);
            rg.load(g[i], i, i < n);
        }
    }
    template <int SCALE>
    __device__ __forceinline__ void form_as(const float (&bias)[VEC], const float (&rate)[VEC]) {
        m.none();
#pragma unroll
        for (int e = 0; e < VEC; ++e) H[e] = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC], gv[VEC];
            x[i].get(xv);
            g[i].get(gv);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float c, slope, sig;
                gate_of<FORM>(gv[e] + bias[e], rate[e], a[i][e], c, slope, sig);
                u[i][e] = xv[e] * input_scale(SCALE, a[i][e], c);
                H[e] = fmaf(a[i][e], H[e], u[i][e]);
                m.P[e] *= a[i][e];
                m.C[e] = fmaf(c, 1.f - m.C[e], m.C[e]);
            }
        }
    }
    __device__ __forceinline__ void form(int scale, const float (&bias)[VEC], const float (&rate)[VEC]) {
        if (scale == GDN_GLR_PLAIN)
            form_as<GDN_GLR_PLAIN>(bias, rate);
        else if (scale == GDN_GLR_COMPLEMENT)
            form_as<GDN_GLR_COMPLEMENT>(bias, rate);
        else
            form_as<GDN_GLR_NORM>(bias, rate);
    }
    // The first tokens of sequences take their initial state; in packed rows
    // nothing passes them.
    template <bool PK>
    __device__ __forceinline__ void begin(const GlrParams &p, int b, int t0, int c, uint32_t first) {
        if (__ballot(first != 0) == 0) return;
        float h[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const bool f = first >> i & 1;
            if (f && p.h0) {
                float h0[VEC];
                state_load<VEC>(p, p.h0, state_of<PK>(p, b, t0 + i), c, h0);
#pragma unroll
                for (int e = 0; e < VEC; ++e) u[i][e] = fmaf(a[i][e], h0[e], u[i][e]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[e] = f ? u[i][e] : fmaf(a[i][e], h[e], u[i][e]);
        }
        if (first) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                H[e] = h[e];
                if (PK) m.P[e] = -1.f;
            }
        }
    }
};

// The move of a wave's whole run into (P, C, H), of what lies in it before this lane's
// into `before` and E.
template <bool PK, int VEC>
__device__ __forceinline__ void join_wave(Moves<VEC> &m, float (&H)[VEC], Moves<VEC> &before, float (&E)[VEC]) {
    before.none();
#pragma unroll
    for (int e = 0; e < VEC; ++e) E[e] = 0.f;
    if constexpr (GlrLane<VEC>::kTG == 2) {
        const bool second = lane_id() & 32;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float oP = other_half(m.P[e]), oC = other_half(m.C[e]), oH = other_half(H[e]);
            if (second) {
                before.P[e] = oP;
                before.C[e] = oC;
                E[e] = oH;
            }
            const float P2 = second ? m.P[e] : oP, C2 = second ? m.C[e] : oC;
            H[e] = move<PK>(P2, C2, second ? oH : H[e], second ? H[e] : oH);
            join<PK>(second ? oP : m.P[e], second ? oC : m.C[e], P2, C2, m.P[e], m.C[e]);
        }
    }
}

// Host side, shared by the passes (gdn_glr.hip).
gdn_status check_glr(const gdn_glr_problem *pr, bool packed);
void fill_glr(const gdn_glr_problem *pr, GlrParams &gp, const int32_t *cu);
bool glr_pairs(const gdn_glr_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> gates,
               std::initializer_list<int64_t> strides);
bool glr_aligned(const gdn_glr_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> gates,
                 std::initializer_list<const void *> f32);

}  // namespace gdn

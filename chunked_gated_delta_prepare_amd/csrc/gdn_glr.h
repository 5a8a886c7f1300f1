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
// tokens.  (8 bytes a lane would make four groups, and twice the joining.)  Runs are put
// together with one channel a lane: a swap of the wave's halves brings both groups'
// runs of one channel into a lane, and the states at their fronts back (both channels of
// both lanes: 402 us for 2 x 8192 tokens of 4096 channels forward and backward, so 368).
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
    int groups, segs, seg_len, pieces;                       // channels / 64; segments (backward: tiles) and their pieces
    int grads;                                               // whether dbias or drate is wanted
};

// A lane's VEC channel weights (fp32), zero without any.
template <int VEC>
__device__ __forceinline__ void channel_load(const float *w, int c, int D, float (&x)[VEC]) {
    row_load<float, VEC>(make_rsrc(w, w ? (uint32_t)D * 4 : 0), c, x);
}

// ---------------------------------------------------------------------------
// gates
// ---------------------------------------------------------------------------

// 1 - e^-y, and e^-y.  |y| < 1/2: the series y (1 - y/2 + ... - y^7/8!), whose next term is
// below 2^-26 of it; else 1 - e^-y is at least 0.39 and loses a bit.  NEAR: |y| < 1/8
// is known, where five terms do (y^5/720 < 2^-24).
template <bool NEAR>
__device__ __forceinline__ void decay_of(float y, float &a, float &c) {
    float s = 1.f / 120.f;
    if constexpr (!NEAR) {
        s = fmaf(y, -1.f / 40320.f, 1.f / 5040.f);
        s = fmaf(y, s, -1.f / 720.f);
        s = fmaf(y, s, 1.f / 120.f);
    }
    s = fmaf(y, s, -1.f / 24.f);
    s = fmaf(y, s, 1.f / 6.f);
    s = fmaf(y, s, -0.5f);
    s = fmaf(y, s, 1.f) * y;
    if constexpr (NEAR) {
        c = s;
        a = 1.f - s;
    } else {
        const float e = fast_exp2(y * -kLog2e);
        const bool small = fabsf(y) < 0.5f;
        c = small ? s : 1.f - e;
        a = small ? 1.f - s : e;
    }
}

// How a gate becomes a decay: its form, and whether |log a| < 1/8 is known (a rate
// below 1/8 in all channels of a wave, as gates of long memories have it).
enum { kLog = GDN_GLR_LOG, kSigmoid = GDN_GLR_SIGMOID, kRate = GDN_GLR_RATE };

// A channel's bias, for a sigmoid as its exponent takes it: in units of it, rounded, and 2 to
// the power of what the rounding left out.  Without that the sigmoid would be off by |bias| units
// where gate and bias cancel.
struct GateBias {
    float b, fix;
};
template <int FORM, int VEC>
__device__ __forceinline__ void load_bias(const float *w, int c, int D, GateBias (&bias)[VEC]) {
    float b[VEC];
    channel_load<VEC>(w, c, D, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float t = b[e] * -kLog2e;
        bias[e].b = FORM == kLog ? b[e] : t;
        // (a larger one leaves gate + bias nothing behind the point; an infinite one has nothing left out)
        bias[e].fix = fabsf(t) < 0x1p26f ? fast_exp2(fmaf(b[e], -kLog2e, -t)) : 1.f;
    }
}

// A token's decay a, c = 1 - a, and for the gradients d(log a)/d(gate) (slope) and the
// gate's sigmoid (kRate).  The sigmoid s = 1 / (1 + e^-v), v = gate + bias, and o = 1 - s are good to their
// own last digits and |v| units of 2^-24 more, o as e^-v s where e^-v is below 1.
template <int FORM, bool NEAR = false>
__device__ __forceinline__ void gate_of(float g, GateBias bias, float rate, float &a, float &c, float &slope, float &sig) {
    if constexpr (FORM == kLog) {
        decay_of<false>(-(g + bias.b), a, c);
        slope = 1.f;
        sig = 0.f;
    } else {
        const float x = fast_exp2(fmaf(g, -kLog2e, bias.b)), e = x * bias.fix, s = __builtin_amdgcn_rcpf(fmaf(x, bias.fix, 1.f));
        const float o = e < 1.f ? e * s : 1.f - s;
        if constexpr (FORM == kSigmoid) {
            a = s;
            c = o;
            slope = o;
            sig = 0.f;
        } else {
            const float y = rate * s;
            decay_of<NEAR>(y, a, c);
            slope = -y * o;
            sig = s;
        }
    }
}

// Whether a wave's rates are all below 1/8.
template <int FORM, int VEC>
__device__ __forceinline__ bool near_rates(const float (&rate)[VEC]) {
    if constexpr (FORM != kRate) return false;
    bool far = false;
#pragma unroll
    for (int e = 0; e < VEC; ++e) far |= !(fabsf(rate[e]) < 0.125f);
    return __ballot(far) == 0;
}

// The input's factor.
template <int SCALE>
__device__ __forceinline__ float input_scale(float a, float c) {
    return SCALE == GDN_GLR_PLAIN ? 1.f : SCALE == GDN_GLR_COMPLEMENT ? c : __builtin_amdgcn_sqrtf(fmaf(c, a, c));
}
// The factor k and its derivative by log a.  Both are 0 where 1 - a^2 is below fp32's
// normal numbers: the root's instruction, and its reciprocal's, take those for zero, and the
// reciprocal would be infinite.  (Scaled by 2^64 and back they are right down to the
// least denormal number, for 3 % of the time of the packed rows' forward pass.)
template <int SCALE>
__device__ __forceinline__ void input_slope(float a, float c, float &k, float &dk) {
    k = 1.f;
    dk = 0.f;
    if constexpr (SCALE == GDN_GLR_COMPLEMENT) {
        k = c;
        dk = -a;
    }
    if constexpr (SCALE == GDN_GLR_NORM) {
        const float q = fmaf(c, a, c), r = fabsf(q) < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q);
        k = q * r;
        dk = -a * a * r;
    }
}

// f(scale, near) with both as constants.
template <int FORM, typename F>
__device__ __forceinline__ void with_scale(int scale, bool near, F f) {
    auto by_scale = [&](auto n) {
        if (scale == GDN_GLR_PLAIN)
            f(std::integral_constant<int, GDN_GLR_PLAIN>(), n);
        else if (scale == GDN_GLR_COMPLEMENT)
            f(std::integral_constant<int, GDN_GLR_COMPLEMENT>(), n);
        else
            f(std::integral_constant<int, GDN_GLR_NORM>(), n);
    };
    if constexpr (FORM == kRate) {
        if (near) {
            by_scale(std::true_type());
            return;
        }
    }
    by_scale(std::false_type());
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

// Two groups of lanes with two channels each, or, after a swap of halves, both groups'
// values of one channel: {x[0], x[1]} of a lane to {the first group's, the second's}, and back.
__device__ __forceinline__ void swap_halves(float &x, float &y) {
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    x = __uint_as_float(h[0]);
    y = __uint_as_float(h[1]);
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

// A packed sequence's rows, kept from run to run.
struct Span {
    int n = 0, begin = 0, end = 0;
    __device__ __forceinline__ void set(const GlrParams &p, int seq) {
        n = seq;
        begin = cu_at(p, n);
        end = cu_at(p, n + 1);
    }
    __device__ __forceinline__ void at(const GlrParams &p, int t) {
        if (t >= begin && t < end) return;
        // mostly the next one
        if (n + 2 <= p.n_seqs) set(p, n + 1);
        if (t < begin || t >= end) set(p, seq_of(p, t));
    }
    // The same for a token that the wave has in common: 64 offsets at a time.
    __device__ __forceinline__ void at_wave(const GlrParams &p, int t) {
        if (t >= begin && t < end) return;
        int lo = 0, hi = p.n_seqs;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64, i = lo + lane_id() * step;
            const int k = __popcll(__ballot(i < hi && cu_at(p, i < hi ? i : lo) <= t));
            lo += (k ? k - 1 : 0) * step;
            hi = hi < lo + step ? hi : lo + step;
        }
        set(p, lo);
    }
};
// Of a thread's L tokens from t0: which exist and are in a sequence, which are the
// first and the last of one; and, in packed rows with a first or a last, the
// sequence of the first of them.
struct Marks {
    uint32_t valid, first, last;
    Span start;
};
// t_wave: the first token of the wave's runs, `tokens` in all; s: the wave's.
template <bool PK, int L>
__device__ __forceinline__ Marks marks_of(const GlrParams &p, int t_wave, int tokens, int t0, Span &s) {
    constexpr uint32_t kAll = (1u << L) - 1;
    const int n = p.T - t0;
    const uint32_t exist = n >= L ? kAll : n <= 0 ? 0 : (1u << n) - 1;
    Marks m{exist, 0, 0, {}};
    if constexpr (!PK) {
        m.first = t0 == 0 ? 1 & exist : 0;
        m.last = n >= 1 && n <= L ? 1u << (n - 1) : 0;
    } else if (t_wave < p.T) {
        s.at_wave(p, t_wave);
        if (s.begin < t_wave && t_wave + tokens < s.end) return m;
        // a sequence begins or ends here, or there is none
        Span own = s;
        m.valid = 0;
#pragma unroll 1
        for (int i = 0; i < L && t0 + i < p.T; ++i) {
            const int t = t0 + i;
            own.at(p, t);
            if (i == 0) m.start = own;
            const uint32_t in = t >= own.begin && t < own.end ? 1u << i : 0;
            m.valid |= in;
            if (t == own.begin) m.first |= in;
            if (t == own.end - 1) m.last |= in;
        }
    }
    return m;
}
// Sequences without a token hand their state through: out[n] = in[n] (or zero).  A wave
// looks at 64 of them at a time.
__device__ __forceinline__ void pass_empty(const GlrParams &p, bool packed, int b, int c0, const float *in, float *out) {
    if (!out) return;
    const int c = c0 + lane_id();
    auto pass = [&](int n) {
        if (c < p.D) out[(int64_t)n * p.D + c] = in ? in[(int64_t)n * p.D + c] : 0.f;
    };
    if (!packed) {
        if (p.T == 0 && wave_id() == 0) pass(b);
        return;
    }
    for (int n0 = wave_id() * 64; n0 < p.n_seqs; n0 += (int)blockDim.x) {
        const int n = n0 + lane_id();
        uint64_t empty = __ballot(n < p.n_seqs && cu_at(p, n < p.n_seqs ? n : 0) >= cu_at(p, n < p.n_seqs ? n + 1 : 0));
        for (; empty; empty &= empty - 1) pass(n0 + __builtin_ctzll(empty));
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
    // the lane's one channel, among the workgroup's, behind swap_halves
    __device__ __forceinline__ int one() const { return VEC == 2 ? (lane_id() & 31) * 2 + (lane_id() >> 5) : lane_id(); }
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

// A thread's rows of L tokens.
template <typename IO, typename GT, int VEC, int L>
struct RunRows {
    RawRow<IO, VEC> x[L];
    RawRow<GT, VEC> g[L];
    // full: all rows of the workgroup exist
    __device__ __forceinline__ void fetch(const GlrParams &p, int b, int t_base, int row, int c, bool full) {
        const TileRows<IO, VEC> rx(p.x, b * p.xb + (int64_t)t_base * p.xt, p.xt, row, c, p.D);
        const TileRows<GT, VEC> rg(p.g, b * p.gb + (int64_t)t_base * p.gt, p.gt, row, c, p.D);
        if (full) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                rx.load(x[i], i, true);
                rg.load(g[i], i, true);
            }
            return;
        }
        const int n = p.T - t_base - row;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            rx.load(x[i], i, i < n);
            rg.load(g[i], i, i < n);
        }
    }
};

// One channel of a state, by lane.
__device__ __forceinline__ float state_at(const GlrParams &p, const float *s, int n, int c) {
    float x[1];
    state_load<1>(p, s, n, c, x);
    return x[0];
}

// Where a run moves a state: H from zero, and its P and C, a token at a time.  In packed
// rows (ODD: some lane's run has one) a first token takes its sequence's initial
// state, and nothing passes it.
template <bool ODD>
__device__ __forceinline__ void move_on(bool first, float h0, float a, float c, float u, float &H, float &P, float &C) {
    if constexpr (ODD) {
        H = first ? fmaf(a, h0, u) : fmaf(a, H, u);
        P = first || P < 0.f ? -1.f : P * a;
    } else {
        H = fmaf(a, H, u);
        P *= a;
    }
    C = fmaf(c, 1.f - C, C);
}

// A wave's run, of one channel a lane: its move, its H and (backward) E, and those of its
// two groups of lanes, whose runs lie behind each other.
struct WaveRun {
    float P, C, H, E, P0, C0, H0, E0, P1, C1, H1, E1;
};
template <bool PK, int VEC, bool BOTH>
__device__ __forceinline__ WaveRun join_wave(const Moves<VEC> &m, const float (&H)[VEC], const float (&E)[VEC]) {
    WaveRun r;
    r.P = r.P0 = m.P[0];
    r.C = r.C0 = m.C[0];
    r.H = r.H0 = H[0];
    r.E = r.E0 = E[0];
    if constexpr (VEC == 2) {
        r.P1 = m.P[1];
        r.C1 = m.C[1];
        r.H1 = H[1];
        swap_halves(r.P0, r.P1);
        swap_halves(r.C0, r.C1);
        swap_halves(r.H0, r.H1);
        r.H = move<PK>(r.P1, r.C1, r.H0, r.H1);
        if constexpr (BOTH) {
            r.E1 = E[1];
            swap_halves(r.E0, r.E1);
            r.E = move<PK>(r.P0, r.C0, r.E1, r.E0);
        }
        join<PK>(r.P0, r.C0, r.P1, r.C1, r.P, r.C);
    }
    return r;
}
// The state in front of the wave's run -> in front of the lane's, of its VEC channels.
template <bool PK, int VEC>
__device__ __forceinline__ void spread_state(const WaveRun &r, float h, float (&x)[VEC]) {
    x[0] = h;
    if constexpr (VEC == 2) {
        x[1] = move<PK>(r.P0, r.C0, h, r.H0);
        swap_halves(x[0], x[1]);
    }
}
// The same backwards, with what lies behind.
template <bool PK, int VEC>
__device__ __forceinline__ void spread_behind(const WaveRun &r, float d, float (&x)[VEC]) {
    x[0] = d;
    if constexpr (VEC == 2) {
        x[1] = d;
        x[0] = move<PK>(r.P1, r.C1, d, r.E1);
        swap_halves(x[0], x[1]);
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

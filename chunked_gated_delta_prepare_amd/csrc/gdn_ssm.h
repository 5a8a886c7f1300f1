// Selective state space scan: what its forward and backward kernels share.
//
// A head's state h [N, P] follows h_t = e^(g_t) h_{t-1} + dt_t B_t x_t^T with
// g = dt A, and y_t = h_t^T C_t + D x_t.  Over a chunk of 64 tokens, with
// cum_t the sum of g up to t inside the chunk and h the state before it,
//
//   y_t = sum_{s<=t} (C_t . B_s) e^(cum_t - cum_s) dt_s x_s + e^(cum_t) h^T C_t
//   h' = e^(cum_63) h + sum_s e^(cum_63 - cum_s) dt_s B_s x_s^T
//
// so that all of it is matrix products over 64 x 64, 64 x N and N x P tiles.
//
// Streams are cut into segments that run side by side: a first launch forms
// every segment's end state from a zero start, a second one starts each
// segment from the sum of those before it, each times the decays between,
// and h0.
//
// Decays.  cum is summed in 64 bits and kept as two floats, so that a
// difference of two of them has the relative accuracy of its own size, not of
// cum's: weak gates late in a chunk stay exact behind strong ones.  Every
// exponent is a sum of g over tokens between two others, so no factor
// exceeds 1 while A <= 0.
#pragma once

#include "gdn_layer.h"

namespace gdn {

constexpr int kSsmChunk = 64;

struct SsmParams {
    const void *x, *dt, *Bm, *Cm, *dy;
    const float *A, *D, *bias, *h0, *dhT;
    void *y, *dx, *dB, *dC, *ddt;
    float *hT, *dA, *dD, *dbias, *dh0, *state, *ws;
    const int32_t *cu, *slots;
    int64_t xb, xt, bb, bt, db, dt_, gb, gt, n_slots;
    int T, H, P, N, G, n_seqs, heads_per_group;
    int seg_tokens, n_items, n_hb;    // tokens of a segment, segments in all, blocks of columns
    int softplus, swizzle, dt_f32;
};

// Operands of the matrix cores by io type: bf16 products for bf16 io, fp32
// products for fp32 io.  Both take eight k slots a lane.
template <typename IO> struct SOp;

template <> struct SOp<bf16_t> {
    typedef uint16_t elem;
    typedef bf16x8 frag;
    static constexpr int kPad = 8;
    static constexpr bool kSplit = true;      // an fp32 operand takes two products
    __device__ static frag bits(u32x2 a, u32x2 b) { return __builtin_bit_cast(frag, u32x4{a[0], a[1], b[0], b[1]}); }
    __device__ static void mma(float4v &acc, const frag &a, const frag &b) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }
    // S[row][k0 + 8 q ..] of a row-major S
    __device__ static frag row(const elem *S, int ld, int m0, int k0) {
        const int l = lane_id();
        return __builtin_bit_cast(frag, *(const u32x4 *)(S + (m0 + (l & 15)) * ld + k0 + 8 * (l >> 4)));
    }
    // S[k0 + 8 q + e][m0 + j] of a row-major S (its transpose's rows)
    __device__ static frag col(const elem *S, int ld, int m0, int k0) {
        const int l = lane_id(), q = l >> 4;
        // (read_T4 takes rows 4 q ..; slots 8 q .. need rows 8 q ..)
        return bits(read_T4(S + (k0 + 4 * q) * ld, ld, m0), read_T4(S + (k0 + 4 * q + 4) * ld, ld, m0));
    }
    // split slots: S[m0 + j][k0 + 4 q ..] and S[..][k0 + 16 + 4 q ..]
    __device__ static frag row_split(const elem *S, int ld, int m0, int k0) {
        const int l = lane_id();
        const elem *p = S + (m0 + (l & 15)) * ld + k0 + 4 * (l >> 4);
        return bits(*(const u32x2 *)p, *(const u32x2 *)(p + 16));
    }
    __device__ static frag acc_split(const float4v &lo, const float4v &hi) {
        frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = (__bf16)lo[e];
            f[4 + e] = (__bf16)hi[e];
        }
        return f;
    }
    // what a rounding to bf16 leaves over, itself in bf16: with both parts an
    // fp32 operand enters a product with a relative error of 2^-18 at most
    __device__ static frag acc_split_rest(const float4v &lo, const float4v &hi, const frag &f) {
        frag r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[e] = (__bf16)(lo[e] - (float)f[e]);
            r[4 + e] = (__bf16)(hi[e] - (float)f[4 + e]);
        }
        return r;
    }
    // w .* f in two parts
    __device__ static void scaled(const frag &f, const float (&w)[8], frag &hi, frag &lo) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = (float)f[e] * w[e];
            hi[e] = (__bf16)v;
            lo[e] = (__bf16)(v - (float)hi[e]);
        }
    }
    __device__ static void put4(elem *p, const float4v &v) {
        *(u32x2 *)p = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
    __device__ static void get4(const elem *p, float (&v)[4]) {
        const u32x2 u = *(const u32x2 *)p;
        v[0] = __uint_as_float(u[0] << 16);
        v[1] = __uint_as_float(u[0] & 0xffff0000u);
        v[2] = __uint_as_float(u[1] << 16);
        v[3] = __uint_as_float(u[1] & 0xffff0000u);
    }
};

template <> struct SOp<float> {
    typedef float elem;
    typedef Mma<float>::frag frag;
    static constexpr int kPad = 4;
    static constexpr bool kSplit = false;
    __device__ static void mma(float4v &acc, const frag &a, const frag &b) { Mma<float>::mma(acc, a, b); }
    __device__ static frag row(const elem *S, int ld, int m0, int k0) { return Mma<float>::load(frag_ptr(S + m0 * ld, ld, k0)); }
    __device__ static frag col(const elem *S, int ld, int m0, int k0) { return frag_T(S, ld, m0, k0); }
    __device__ static frag row_split(const elem *S, int ld, int m0, int k0) { return fragA_split(S, ld, m0, k0); }
    __device__ static frag acc_split(const float4v &lo, const float4v &hi) { return frag{lo, hi}; }
    __device__ static frag acc_split_rest(const float4v &, const float4v &, const frag &f) { return f; }
    __device__ static void scaled(const frag &f, const float (&w)[8], frag &hi, frag &lo) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi.lo[e] = f.lo[e] * w[e];
            hi.hi[e] = f.hi[e] * w[4 + e];
        }
        lo = hi;
    }
    __device__ static void put4(elem *p, const float4v &v) { *(float4v *)p = v; }
    __device__ static void get4(const elem *p, float (&v)[4]) {
        const float4v u = *(const float4v *)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = u[e];
    }
};

// softplus(v) = log(1 + e^v), to fp32's accuracy for every v
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ double wave_scan(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double u = __shfl_up(v, m, 64);
        if (lane_id() >= m) v += u;
    }
    return v;
}

// A chunk's gates of one head, a lane a token.
struct Gates {
    float2 cum[kSsmChunk];      // log2 of the decay from the chunk's start through the token
    float ecum[kSsmChunk];      // that decay
    float end[kSsmChunk];       // dt times the decay from behind the token to the chunk's end
    float dt[kSsmChunk];
    double total;               // log2 of the whole chunk's decay
};

__device__ __forceinline__ float decay_between(const float2 &t, const float2 &s) {
    return fast_exp2((t.x - s.x) + (t.y - s.y));
}

// dt of a token from its raw value (0 where there is no token).
__device__ __forceinline__ float dt_of(const SsmParams &p, float raw, float bias, bool live) {
    const float v = raw + bias;
    return live ? (p.softplus ? softplus(v) : v) : 0.f;
}

__device__ __forceinline__ void make_gates(Gates &g, float dt, float A) {
    const int l = lane_id();
    const double cum = wave_scan((double)dt * (double)A * 1.4426950408889634074);
    const double total = __shfl(cum, 63, 64);
    const float hi = (float)cum;
    g.cum[l] = make_float2(hi, (float)(cum - (double)hi));
    g.ecum[l] = fast_exp2(hi);
    g.end[l] = dt * fast_exp2((float)(total - cum));
    g.dt[l] = dt;
    if (l == 63) g.total = total;
}

// A segment of a sequence: its place in the workspace, its tokens, and the
// sequence it belongs to.
struct Segment {
    int item, first;            // this segment and the first of its sequence
    int seq, batch;             // number of the sequence; batch its rows lie in
    int begin, end;             // tokens of the segment
    int seq_begin, seq_end;
    bool live;
};

__device__ __forceinline__ int ssm_cu(const SsmParams &p, int n) {
    const int v = p.cu[n];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

__device__ __forceinline__ Segment find_segment(const SsmParams &p, int item) {
    Segment s;
    s.item = item;
    s.live = true;
    if (!p.cu) {
        const int per = p.n_items / p.n_seqs;
        s.seq = s.batch = item / per;
        s.first = s.seq * per;
        s.seq_begin = 0;
        s.seq_end = p.T;
    } else {
        // every sequence has at least one segment; 64 sequences a step
        int base = 0;
        s.live = false;
        s.batch = 0;
        for (int n0 = 0; n0 < p.n_seqs && !s.live; n0 += 64) {
            const int n = n0 + lane_id();
            int b = 0, e = 0, cnt = 0;
            if (n < p.n_seqs) {
                b = ssm_cu(p, n);
                e = ssm_cu(p, n + 1);
                e = e < b ? b : e;
                cnt = e > b ? (e - b + p.seg_tokens - 1) / p.seg_tokens : 1;
            }
            int upto = cnt;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int u = __shfl_up(upto, m, 64);
                if (lane_id() >= m) upto += u;
            }
            const uint64_t hit = __ballot(cnt > 0 && item >= base + upto - cnt && item < base + upto);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                s.live = true;
                s.seq = __builtin_amdgcn_readfirstlane(n0 + l);
                s.first = __builtin_amdgcn_readfirstlane(base + __shfl(upto - cnt, l, 64));
                s.seq_begin = __builtin_amdgcn_readfirstlane(__shfl(b, l, 64));
                s.seq_end = __builtin_amdgcn_readfirstlane(__shfl(e, l, 64));
            }
            base += __builtin_amdgcn_readfirstlane(__shfl(upto, 63, 64));
        }
        if (!s.live) return s;
    }
    s.begin = s.seq_begin + (item - s.first) * p.seg_tokens;
    s.end = s.begin + p.seg_tokens < s.seq_end ? s.begin + p.seg_tokens : s.seq_end;
    return s;
}

// blockIdx -> (segment, block of columns).  The blocks of one segment share
// its B and C: with swizzle they go to one XCD (workgroups are dealt to the
// eight XCDs in turn), else they are neighbours.
__device__ __forceinline__ void place(const SsmParams &p, int &item, int &hb) {
    const int i = blockIdx.x;
    if (p.swizzle) {
        const int j = i >> 3;
        hb = j % p.n_hb;
        item = (j / p.n_hb) * 8 + (i & 7);
    } else {
        hb = i % p.n_hb;
        item = i / p.n_hb;
    }
}

// ROWS x COLS of a row-major operand from HBM through registers into LDS:
// 16 bytes a lane and step, rows at or past `rows` as zeros.
template <typename IO, int ROWS, int COLS>
struct TileRegs {
    static constexpr int kPer = 16 / sizeof(IO), kLine = COLS / kPer, kN = ROWS * kLine / 256;
    u32x4 v[kN];
    __device__ __forceinline__ void load(const void *base, int64_t elems, uint32_t stride, int rows) {
        const rsrc_t r = make_rsrc((const IO *)base + elems, rows > 0 ? 0x7fffffffu : 0u);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int k = i * 256 + threadIdx.x, t = k / kLine, c = k % kLine * kPer;
            const uint32_t off = (t * stride + c) * (uint32_t)sizeof(IO);
            v[i] = bload128(r, t < rows ? off : 0xfffffff0u, 0);
        }
    }
    __device__ __forceinline__ void put(typename SOp<IO>::elem *S, int ld) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int k = i * 256 + threadIdx.x, t = k / kLine, c = k % kLine * kPer;
            *(u32x4 *)(S + t * ld + c) = v[i];
        }
    }
};

int64_t ssm_state_bytes(const gdn_ssm_problem *pr);

}  // namespace gdn

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
// The gradients are scans of the same form.  With du_s the gradient of
// dt_s x_s and dh that of the state,
//
//   du_s = sum_{t>=s} (B_s . C_t) e^(cum_t - cum_s) dy_t + e^(cum_63 - cum_s) dh^T B_s
//   dC_t = sum_{s<=t} (dy_t . x_s) e^(cum_t - cum_s) dt_s B_s + e^(cum_t) h dy_t
//   dB_s = dt_s (sum_{t>=s} (x_s . dy_t) e^(cum_t - cum_s) C_t + e^(cum_63 - cum_s) dh x_s)
//
// so that one description serves all: rows q [N], q2 [P], k [N], v [P] and
// weights w in scan order i, cum_i the sum of gates that lie between the
// chunk's start and row i, and the state S before the chunk,
//
//   out1_i = sum_{j<=i} (q_i . k_j) e^(cum_i - cum_j) w_j v_j + e^(cum_i) S^T q_i
//   out2_i = sum_{j<=i} (q2_i . v_j) e^(cum_i - cum_j) w_j k_j + e^(cum_i) S q2_i
//   S'     = e^(total) S + sum_j e^(total - cum_j) w_j k_j v_j^T
//
//            q   q2  k   v   w    out1  out2
//   forward  C   dy  B   x   dt   y     dC
//   reverse  B   x   C   dy  1    du    dB / dt    rows from the last to the first
//
// Forward, cum_i holds row i's own gate (it acts before the row is added);
// in reverse it holds those of the rows before it.
//
// dt's and A's gradients.  A pair of tokens s <= t adds
//   W_ts = (C_t . B_s) (dy_t . x_s) e^(cum_t - cum_s) dt_s
// to the loss's derivative along y; the gate g_u takes part where s < u <= t.
// Rows leave q_i . out2_i, split into the pairs inside the chunk (without
// s = t) and those across its border: r_t = sum over s of W_ts from the
// forward scan and c_s = sum over t of W_ts / dt_s from the reverse one.  With
// X the sum of W over all pairs across the end of a chunk,
//   dg_u = sum_{t>=u} (r_t - dt_t c_t)_inside + sum_{t>=u} r_t,across
//        + sum_{s<u} dt_s c_s,across + Q,      Q = X - sum_s dt_s c_s,across
// where Q is what crosses the whole chunk, and Q + sum_t r_t,across is X of
// the chunk before.  Every difference is one of terms inside one chunk: the
// sum of r - dt c over a long stream, which is the same number, would drown
// short memories in the rounding of far tokens.  For the same reason X is formed
// anew every four chunks as <h, dh>: the forward scan leaves h there, and the
// reverse one meets it with dh.  Behind a sequence's last chunk dh is the final
// state's own gradient, so the forward scan forms X there itself and leaves no
// state.  (dA of 2 x 8192 tokens, 32 heads: 1.2e-5 off with X passed on over 16
// chunks.)
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

#include <type_traits>

#include "gdn_layer.h"

namespace gdn {

constexpr int kSsmChunk = 64;

struct SsmParams {
    // the scan's rows and results (see above)
    const void *q, *q2, *k, *v, *dt;
    const float *A, *D, *bias, *s0;         // s0: the state behind the first segment (h0; dhT)
    void *out;                              // out1's rows (y; dx) or out2's (dC; dB)
    float *sT;                              // the state behind the last one (hT; dh0)
    const int32_t *cu;
    int64_t qkb, qkt, vb, vt, q2b, q2t, db, dt_, ob, ot;   // strides: batch, token
    // workspace
    double *total;                          // [end][n_hb][NH]: log2 of a segment's decay
    float *ends;                            // [end][n_hb][N][64 NCB]: end states from zero
    float *part;                            // out2 by block of columns, for ssm_sum_kernel
    float *inside, *across;                 // [n_hb][NH][B T]: q . out2 in two parts
    float *dyx, *wtt;                       // the same: dy_t . x_t, and W_tt / dt_t
    const float *dT;                        // the final states' gradient
    float *marks;                           // [mark][n_hb][N][64 NCB]: h every four chunks
    double *X;                              // [place][n_hb][NH]: <h, dh> there, and behind sequences
    int64_t rows;                           // B T
    int n_slots, n_marks, n_x;              // places for chunks in part, for marks and in X
    int T, H, P, n_seqs, heads_per_group;
    int seg_tokens, n_items, n_hb;          // tokens of a segment, segments in all, blocks of columns
    int n_ends, n_units;                    // places for end states; segments or ends that this launch works on
    int softplus, swizzle, dt_f32;
    int all_ends;                           // the last segments' end states are in the workspace too
};

// x, unknown to the compiler: what is computed from it inside a loop stays
// there.  Addresses of swizzled tiles, taken out of the chunk loop, would hold
// some forty registers a lane.
__device__ __forceinline__ int again(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Element (row, col) of a row-major tile of LD elements in LDS: 16-byte chunk c
// of row r sits at chunk c ^ s(r), s linear over r mod 16's bits.  Of the 2^16
// such maps, timed with eight waves reading at once, these cost a fragment
// read of 16 bytes a lane and transposed reads of two and of four chunks the
// least there is (4.3, 4.3 and 3.4 cycles a wave's read; r's bits in order
// cost 4.3, 8.2 and 4.3, and no map at all 32, 16 and 16).
template <int CHUNKS>
__device__ __forceinline__ constexpr int swizzle(int r) {
    if (CHUNKS == 8) return ((r & 1) ? 7 : 0) ^ ((r & 2) ? 6 : 0) ^ ((r & 8) ? 2 : 0);
    return ((r & 1) ? 4 : 0) ^ ((r & 2) ? 2 : 0) ^ ((r & 4) ? 9 : 0) ^ ((r & 8) ? 8 : 0);
}
template <typename E, int LD>
__device__ __forceinline__ int at(int row, int col) {
    constexpr int kPer = 16 / sizeof(E);
    return row * LD + (((col / kPer) ^ swizzle<LD / kPer>(row)) * kPer) + col % kPer;
}

// A lane's byte offsets into tiles of LD elements, from which a fragment's
// are an xor with its first column and an addition of its first row (see at:
// rows come in multiples of 16, and a column's high bits do not meet the
// lane's low ones).  Kept out of the compiler's sight once a chunk, so that it
// does not keep every fragment's offset in a register of its own.
template <typename E, int LD> struct Lane {
    int row, tr2, tr4;
};
template <int LD> struct Lane<uint16_t, LD> {
    static constexpr int kFour = swizzle<LD / 8>(4) << 4;      // what four rows on changes
    int row, tr2, tr4;         // fragments of rows; transposed reads of two and of four chunks
    __device__ explicit Lane(int l) {
        const int q = l >> 4, j = l & 15, r = 8 * q + (j >> 2), s = swizzle<LD / 8>(r), c = j & 3;
        row = again(j * LD * 2 + ((q ^ swizzle<LD / 8>(j)) << 4));
        tr2 = again(r * LD * 2 + (((c >> 1) ^ s) << 4) + (c & 1) * 8);
        tr4 = again(r * LD * 2 + ((c ^ s) << 4));
    }
};
template <int LD> struct Lane<float, LD> {
    int l;
    __device__ explicit Lane(int lane) : l(again(lane)) {}
};

// Operands of the matrix cores by io type: bf16 products for bf16 io, fp32
// products for fp32 io.  Both take eight k slots a lane.
//
// row: lane (q, j) gets S[m0 + j][k0 + 8 q .. +7].
// col: S[k0 + 8 q + e][m0 + j], e = 0..7: rows of the transpose.
// pair: as col, but for the 16 columns that half `hf` of a block of 32 takes
// in accumulators: lane j gets column m0 + 8 (j / 4) + 4 hf + j % 4, so that
// accumulators of both halves hold, in lane group q, rows m0 + 8 q .. +7 of
// their product, which are the slots of a row fragment.
template <typename IO> struct SOp;

template <> struct SOp<bf16_t> {
    typedef uint16_t elem;
    typedef bf16x8 frag;
    template <int PARTS> static constexpr int kParts = PARTS;
    __device__ static void mma(float4v &acc, const frag &a, const frag &b) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }
    template <int LD>
    __device__ static frag row(const elem *S, const Lane<elem, LD> &a, int m0, int k0) {
        return __builtin_bit_cast(frag, *(const u32x4 *)((const char *)S + (a.row ^ (k0 * 2)) + m0 * LD * 2));
    }
    // two transposed reads of four rows each; lane L of a group of 16 fetches
    // row L / 4, and columns c(L % 4) .. +3, which lanes 4 (L % 4) .. +3 get
    template <int LD>
    __device__ static frag tr(const elem *S, int off, int plus) {
        typedef __fp16 v4fp16 __attribute__((vector_size(8)));
        typedef __attribute__((address_space(3))) v4fp16 lds_v4fp16;
        const char *p = (const char *)S + off + plus, *r = (const char *)S + (off ^ Lane<elem, LD>::kFour) + plus + 4 * LD * 2;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_v4fp16 *)p));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_v4fp16 *)r));
        return __builtin_bit_cast(frag, u32x4{a[0], a[1], b[0], b[1]});
    }
    template <int LD>
    __device__ static frag col(const elem *S, const Lane<elem, LD> &a, int m0, int k0) {
        return tr<LD>(S, a.tr2 ^ (m0 * 2), k0 * LD * 2);
    }
    template <int LD>
    __device__ static frag pair(const elem *S, const Lane<elem, LD> &a, int m0, int hf, int k0) {
        return tr<LD>(S, a.tr4 ^ (m0 * 2), k0 * LD * 2 + 8 * hf);
    }
    // an fp32 operand in PARTS bf16 ones, each holding what rounding left over
    // of those before: a relative error of 2^-9, 2^-18 or 2^-27 at most
    template <int PARTS>
    __device__ static void parts_of(const float (&v)[8], frag (&f)[PARTS]) {
        u32x4 u[PARTS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                u[k][i] = pack_bf16(a, b);
                a -= __uint_as_float(u[k][i] << 16);
                b -= __uint_as_float(u[k][i] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int k = 0; k < PARTS; ++k) f[k] = __builtin_bit_cast(frag, u[k]);
    }
    // the accumulators of both halves of a block
    template <int PARTS>
    __device__ static void acc(const float4v &lo, const float4v &hi, frag (&f)[PARTS]) {
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        parts_of(v, f);
    }
    // w .* a
    template <int PARTS>
    __device__ static void scaled(const frag &a, const float (&w)[8], frag (&f)[PARTS]) {
        const u32x4 u = __builtin_bit_cast(u32x4, a);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16) * w[2 * i];
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u) * w[2 * i + 1];
        }
        parts_of(v, f);
    }
    // z stays zero while a's values are numbers
    __device__ static void times_zero(float4v &z, const frag &a) { mma(z, a, __builtin_bit_cast(frag, u32x4{0, 0, 0, 0})); }
    __device__ static float get(elem x) { return __uint_as_float((uint32_t)x << 16); }
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
    template <int PARTS> static constexpr int kParts = 1;
    __device__ static void mma(float4v &acc, const frag &a, const frag &b) { Mma<float>::mma(acc, a, b); }
    template <int LD>
    __device__ static frag row(const elem *S, const Lane<elem, LD> &a, int m0, int k0) {
        const int l = a.l, r = m0 + (l & 15), c = k0 + 8 * (l >> 4);
        return frag{*(const float4v *)(S + at<elem, LD>(r, c)), *(const float4v *)(S + at<elem, LD>(r, c + 4))};
    }
    template <int LD>
    __device__ static frag col_at(const elem *S, int c, int r) {
        frag f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f.lo[e] = S[at<elem, LD>(r + e, c)];
            f.hi[e] = S[at<elem, LD>(r + 4 + e, c)];
        }
        return f;
    }
    template <int LD>
    __device__ static frag col(const elem *S, const Lane<elem, LD> &a, int m0, int k0) {
        return col_at<LD>(S, m0 + (a.l & 15), k0 + 8 * (a.l >> 4));
    }
    template <int LD>
    __device__ static frag pair(const elem *S, const Lane<elem, LD> &a, int m0, int hf, int k0) {
        const int j = a.l & 15;
        return col_at<LD>(S, m0 + 8 * (j >> 2) + 4 * hf + (j & 3), k0 + 8 * (a.l >> 4));
    }
    template <int PARTS>
    __device__ static void acc(const float4v &lo, const float4v &hi, frag (&f)[PARTS]) { f[0] = frag{lo, hi}; }
    template <int PARTS>
    __device__ static void scaled(const frag &a, const float (&w)[8], frag (&f)[PARTS]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[0].lo[e] = a.lo[e] * w[e];
            f[0].hi[e] = a.hi[e] * w[4 + e];
        }
    }
    __device__ static void times_zero(float4v &z, const frag &a) { z += a.lo * 0.f + a.hi * 0.f; }
    __device__ static float get(elem x) { return x; }
    __device__ static void put4(elem *p, const float4v &v) { *(float4v *)p = v; }
    __device__ static void get4(const elem *p, float (&v)[4]) {
        const float4v u = *(const float4v *)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = u[e];
    }
};

// Four columns of a row at byte offset off: 8 bytes of bf16, or two times 8 of
// fp32, of which the second goes out with an immediate wait in between (two
// adjacent stores in a row would be joined into one of 16 bytes).
template <typename IO>
__device__ __forceinline__ void store_row4(rsrc_t r, uint32_t off, const float4v &o) {
    if constexpr (sizeof(IO) == 2) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])}, r, off, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(o[0]), __float_as_uint(o[1])}, r, off, 0, 0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(o[2]), __float_as_uint(o[3])}, r, off + 8, 0, 0);
    }
}

// softplus(v) = log(1 + e^v), to fp32's accuracy for every v
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// Inclusive sum over the lanes of a wave: within rows of 16 lanes, then the
// rows' sums handed on (lanes that take nothing add 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double v) {
    v = dpp_add<0x111, 0xf>(v);      // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);      // lane 15 of rows 0 and 2 to rows 1 and 3
    return dpp_add<0x143, 0xc>(v);   // lane 31 to rows 2 and 3
}
// lane 63's value
__device__ __forceinline__ double last_lane(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A chunk's gates of one head, a lane a row.  (w is dt forward, 1 in reverse.)
struct __align__(16) Gates {
    float2 cum[kSsmChunk];      // log2 of the decay from the chunk's start to the row
    float ecum[kSsmChunk];      // that decay
    float end[kSsmChunk];       // w times the decay from the row to the chunk's end
    float dt[kSsmChunk];
    double total;               // log2 of the whole chunk's decay
};

// The decays from rows k .. k + 3 (k a multiple of 4) to row i, times the
// weights w.  Those of rows behind i mean nothing and may be no numbers: what is
// made of them is cut off by until().
template <bool REV>
__device__ __forceinline__ float4v decays(const Gates &g, int i, int k) {
    const float2 ci = g.cum[i];
    const float4v a = *(const float4v *)&g.cum[k], b = *(const float4v *)&g.cum[k + 2];
    float4v d = {(ci.x - a[0]) + (ci.y - a[1]), (ci.x - a[2]) + (ci.y - a[3]), (ci.x - b[0]) + (ci.y - b[1]), (ci.x - b[2]) + (ci.y - b[3])};
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = fast_exp2(d[e]);
    if constexpr (!REV) d *= *(const float4v *)&g.dt[k];
    return d;
}

// x of rows k .. k + 3 up to row i, 0 behind it
__device__ __forceinline__ float4v until(int i, int k, float4v x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = k + e <= i ? x[e] : 0.f;
    return x;
}

// dt of a token from its raw value (0 where there is no token).
__device__ __forceinline__ float dt_of(const SsmParams &p, float raw, float bias, bool live) {
    const float v = raw + bias;
    return live ? (p.softplus ? softplus(v) : v) : 0.f;
}

// `before` and `behind` are the signs that the state is held with before and
// behind the chunk.  A row without a token has gate 0 by `live`, not by its dt of
// 0: A may be -inf, and 0 times that is no number.
template <bool REV>
__device__ __forceinline__ void make_gates(Gates &g, float dt, float A, bool live, float before, float behind) {
    const int l = again(lane_id());
    asm volatile("" : "+s"(A));                // (its double is not kept in registers either)
    // a gate below e^-1000 is 0 to all that follows; without the bound one of
    // -1e20 would take the digits of the sums behind it, one of -inf all of them
    // (a NaN stays one)
    const double raw = (double)dt * (double)A, own = live ? (raw < -1000.0 ? -1000.0 : raw) * 1.4426950408889634074 : 0.0, upto = wave_scan(own);
    const double total = last_lane(upto), cum = REV ? upto - own : upto;
    const float hi = (float)cum, w = REV ? 1.f : dt;
    g.cum[l] = make_float2(hi, (float)(cum - (double)hi));
    g.ecum[l] = before * fast_exp2(hi);
    g.end[l] = behind * w * fast_exp2((float)(total - cum));
    g.dt[l] = dt;
    if (l == 63) g.total = total;
}

// A segment of a sequence, its tokens, and the sequence it belongs to.  Segments
// of sequences that have several are counted apart too: those have a place for
// an end state (see SsmPlan), one behind the other.
struct Segment {
    int end_at, first_end;      // that place and the one of the sequence's first segment; -1 without
    int seq, batch;             // number of the sequence; batch its rows lie in
    int begin, end;             // tokens of the segment
    int seq_begin, seq_end;
    bool live;
};

__device__ __forceinline__ int ssm_cu(const SsmParams &p, int n) {
    const int v = p.cu[n];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

// The segment of number `unit`, or (BY_END) the one whose end state's place that is.
template <bool BY_END>
__device__ __forceinline__ Segment find_segment(const SsmParams &p, int unit) {
    Segment s;
    s.live = true;
    int in;                     // its number within the sequence
    if (!p.cu) {
        const int per = p.n_items / p.n_seqs;
        s.seq = s.batch = unit / per;
        in = unit - s.seq * per;
        s.seq_begin = 0;
        s.seq_end = p.T;
        s.first_end = per > 1 ? s.seq * per : -1;
    } else {
        // every sequence has at least one segment; 64 sequences a step
        int items = 0, ends = 0;
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
            // segments of sequences with several, up to this one, and lone segments before it
            const int several = cnt > 1 ? cnt : 0;
            int upto = several;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int u = __shfl_up(upto, m, 64);
                if (lane_id() >= m) upto += u;
            }
            const uint64_t lone = __ballot(cnt == 1);
            const int before = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(lone >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lone, 0));
            const int first_end = ends + upto - several, first = BY_END ? first_end : items + upto - several + before;
            const uint64_t hit = __ballot((BY_END ? several : cnt) > 0 && unit >= first && unit < first + cnt);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                s.live = true;
                s.seq = __builtin_amdgcn_readfirstlane(n0 + l);
                in = unit - __builtin_amdgcn_readfirstlane(__shfl(first, l, 64));
                s.first_end = __builtin_amdgcn_readfirstlane(__shfl(several ? first_end : -1, l, 64));
                s.seq_begin = __builtin_amdgcn_readfirstlane(__shfl(b, l, 64));
                s.seq_end = __builtin_amdgcn_readfirstlane(__shfl(e, l, 64));
            }
            const int sum = __builtin_amdgcn_readfirstlane(__shfl(upto, 63, 64));
            ends += sum;
            items += sum + (int)__builtin_popcountll(lone);
        }
        if (!s.live) return s;
    }
    s.end_at = s.first_end < 0 ? -1 : s.first_end + in;
    s.begin = s.seq_begin + in * p.seg_tokens;
    s.end = s.begin + p.seg_tokens < s.seq_end ? s.begin + p.seg_tokens : s.seq_end;
    return s;
}

// blockIdx -> (segment or end, block of columns).  The blocks of one segment and
// group share its B and C: with swizzle they go to one XCD (workgroups are
// dealt to the eight XCDs in turn), else they are neighbours.
__device__ __forceinline__ void place(const SsmParams &p, int &unit, int &hb) {
    const int i = blockIdx.x;
    if (p.swizzle) {
        const int groups = p.H / p.heads_per_group, per = p.n_hb / groups, j = i >> 3, at = (j / per) * 8 + (i & 7);
        unit = at / groups;
        hb = (at % groups) * per + j % per;
    } else {
        hb = i % p.n_hb;
        unit = i / p.n_hb;
    }
}

__device__ __forceinline__ float uniform(float x) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// 64 rows of COLS elements from HBM through registers into LDS, 16 bytes a
// lane and step: rows at or past `rows` as zeros (they lie behind the
// descriptor's end).  LDS has them in scan order (REV: the last row first).
template <typename IO, int COLS, bool REV, int THREADS>
struct TileRegs {
    typedef typename SOp<IO>::elem E;
    static constexpr int kPer = 16 / sizeof(IO), kLine = COLS / kPer, kN = kSsmChunk * kLine / THREADS, kStep = THREADS / kLine;
    u32x4 v[kN];
    __device__ __forceinline__ void load(int tid, const void *base, int64_t elems, uint32_t stride, int rows) {
        const rsrc_t r = make_rsrc((const IO *)base + elems, ((uint32_t)(rows - 1) * stride + COLS) * (uint32_t)sizeof(IO));
        const uint32_t off = ((uint32_t)(tid / kLine) * stride + tid % kLine * kPer) * (uint32_t)sizeof(IO);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = bload128(r, off + i * (kStep * stride * (uint32_t)sizeof(IO)), 0);
    }
    __device__ __forceinline__ void put(int tid, E *S, int rows) const {
        // a step of 16 rows or more keeps the swizzle
        const int t = tid / kLine, c = tid % kLine * kPer;
        if (kStep % 16 == 0 && (!REV || rows == kSsmChunk)) {
            E *p = S + at<E, COLS>(REV ? kSsmChunk - 1 - t : t, c);
#pragma unroll
            for (int i = 0; i < kN; ++i) *(u32x4 *)(p + (REV ? -i : i) * kStep * COLS) = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int k = t + i * kStep;
                *(u32x4 *)(S + at<E, COLS>(REV && k < rows ? rows - 1 - k : k, c)) = v[i];
            }
        }
    }
};

__device__ __forceinline__ int chunks_of(const Segment &s) { return (s.end - s.begin + kSsmChunk - 1) / kSsmChunk; }

// The chunks of a segment in scan order: tokens [lo, lo + rows).
template <bool REV>
__device__ __forceinline__ int chunk_of(const Segment &s, int c, int &lo) {
    lo = s.begin + (REV ? chunks_of(s) - 1 - c : c) * kSsmChunk;
    return s.end - lo < kSsmChunk ? s.end - lo : kSsmChunk;
}

// The place of a segment's chunk among all: sequences begin at their first
// token's 64th plus their number, so that no two share one.
__device__ __forceinline__ int chunk_slot(const SsmParams &p, const Segment &s, int c) {
    const int in = (s.begin - s.seq_begin) / kSsmChunk + c;
    return p.cu ? s.seq_begin / kSsmChunk + s.seq + in : s.seq * ((p.T + kSsmChunk - 1) / kSsmChunk) + in;
}
// The places of the state behind a chunk and of its X, -1 where none is kept.  States
// are kept behind every fourth chunk of a sequence but its last one; a sequence's
// begin at its first token's 256th, since its places end before the next one's.
// (With one for its last chunk too, places would be numbered by sequences, a
// state each: 256 sequences of 64 tokens, 64 heads of 128 x 128, 1.3 GB and not
// 0.3.)  X is a number, and has a place there too.
struct Mark {
    int state, x;
};
__device__ __forceinline__ Mark mark_of(const SsmParams &p, const Segment &s, int c) {
    const int in = (s.begin - s.seq_begin) / kSsmChunk + c, chunks = (s.seq_end - s.seq_begin + kSsmChunk - 1) / kSsmChunk;
    const bool last = in == chunks - 1;
    Mark m{-1, -1};
    if ((in & 3) != 3 && !last) return m;
    const int per = 4 * kSsmChunk;
    m.x = (p.cu ? s.seq_begin / per + s.seq : s.seq * ((p.T + per - 1) / per)) + in / 4;
    if (m.x >= p.n_x) m.x = -1;
    if (!last) m.state = (p.cu ? s.seq_begin / per : s.seq * ((p.T - 1) / per)) + in / 4;
    if (m.state >= p.n_marks) m.state = -1;
    return m;
}

// The raw dt of row l of a chunk, as its bits: turned into a number only where
// it is used, since a conversion here would wait for every load in flight.
template <typename IO, bool REV>
__device__ __forceinline__ uint32_t raw_dt(const SsmParams &p, int batch, int head, int lo, int rows) {
    const int l = again(lane_id());
    const int64_t at = batch * p.db + lo * p.dt_ + head;
    const uint32_t e = (uint32_t)((REV ? rows - 1 - l : l) * (int)p.dt_);
    if (sizeof(IO) == 4 || p.dt_f32) return bload32(make_rsrc((const float *)p.dt + at, 0x7fffffffu), l < rows ? e * 4 : 0xfffffff0u, 0);
    return bload16(make_rsrc((const uint16_t *)p.dt + at, 0x7fffffffu), l < rows ? e * 2 : 0xfffffff0u, 0);
}
template <typename IO>
__device__ __forceinline__ float raw_value(const SsmParams &p, uint32_t bits) {
    return __uint_as_float(sizeof(IO) == 4 || p.dt_f32 ? bits : bits << 16);
}

// For every segment that the scan passes before this one, nearest first:
// f(its place in the workspace, the decay between it and this one); returns
// the decay since the scan's very start.
template <bool REV, typename F>
__device__ __forceinline__ float segments_before(const SsmParams &p, const Segment &s, int hb, int nh, int hh, F f) {
    double d = 0.0;
    if (s.first_end < 0) return 1.f;
    const int per = (s.seq_end - s.seq_begin + p.seg_tokens - 1) / p.seg_tokens;
    // (overlapping sequences have more segments than there are places)
    const int top = s.first_end + per < p.n_ends ? s.first_end + per : p.n_ends;
    const int stop = REV ? top : s.first_end - 1;
    for (int i = REV ? s.end_at + 1 : (s.end_at < top ? s.end_at : top) - 1; REV ? i < stop : i > stop; i += REV ? 1 : -1) {
        const int64_t at = (int64_t)i * p.n_hb + hb;
        f(at, fast_exp2((float)d));
        d += p.total[at * nh + hh];
    }
    return fast_exp2((float)d);
}

// ---------------------------------------------------------------------------
// out1, the state, or both, for COLS columns of one head or (NH = 2) of two.
// Wave w keeps the state of columns 16 w .. +15, all N rows of them, in
// accumulators, and uses them as operands without a trip through LDS.  Per
// chunk:
//   1  the lower triangle of q k^T, times decays and weights, to LDS (16 x 16
//      blocks, dealt to the waves); S^T q on the way
//   2  out1 = M v + e^cum S^T q, transposed, so that a lane stores four columns
//   3  S' = e^total S + k^T (w v)
// The products of a state that is an output or another segment's start take
// w v in three bf16 parts (relative error 2^-27): with two the final state was
// 2.4e-6 off, against 1e-7 of fp32 arithmetic throughout, and dA, a sum over
// all tokens of both signs, 5e-5.  So do those of a sequence's only segment,
// whose state is the final one, whether or not it is asked for: out1 has the
// same bits either way.  In the segments of longer sequences only out1 is read
// from the main pass's state (an output state comes from the segments' end
// states), and w v is rounded once to bf16, as out1's other operands are and
// out1 itself, and S too before it is multiplied.  The next chunk's rows are in
// flight while one is worked on, and the gates of several chunks are formed at a
// time, one a wave.
// ENDS: only the state, from a zero start, to the workspace.
//
// Sixteen columns a wave, eight waves for 128 columns, two workgroups a CU: with
// 32 columns a wave and four waves the kernel read a third less from LDS but
// held 375 registers a lane, one wave per SIMD (65536 tokens, 64 heads of 128 x
// 128: 1.8 ms when tried; now 1.31 ms for both launches, of 2.4 GB of rows and
// 774 GFLOP on the matrix cores).  What bounds it: no unit is full.  In the main
// pass the matrix cores are busy 0.21 of the time, vector issue 0.53 (some 390
// instructions a wave and chunk: decays, roundings, the state's scaling) and LDS
// 0.46, and 0.43 of the waves' time is waiting: three barriers a chunk, between
// them one chain of loads, products and stores for all waves, and ten blocks of
// M for eight waves, so that six wait for two.
// ---------------------------------------------------------------------------
template <typename IO, int N, int COLS, int NH, bool ENDS, bool REV>
__global__ void __launch_bounds__(4 * COLS, sizeof(IO) == 4 ? 1 : COLS == 64 && N == 128 ? 3 : 4) ssm_scan_kernel(SsmParams p) {
    typedef SOp<IO> O;
    typedef typename O::elem E;
    constexpr int C = kSsmChunk, NW = COLS / 16, NB = N / 16, kThreads = 4 * COLS, P = COLS / NH;
    constexpr int kP = O::template kParts<3>;
    __shared__ __align__(16) E sv[C * COLS], sk[C * N], sq[ENDS ? 8 : C * N], sm[ENDS ? 1 : NH][ENDS ? 8 : C * C];
    // chunks whose gates are formed at once, one chunk and head a wave
    constexpr int GC = NW / NH;
    __shared__ Gates gates[GC][NH];
    int unit, hb;
    place(p, unit, hb);
    if (unit >= p.n_units) return;
    const Segment seg = find_segment<ENDS>(p, unit);
    if (!seg.live) return;
    const bool last = REV ? seg.begin == seg.seq_begin : seg.end == seg.seq_end;      // of the scan
    // an output state comes from the end states, but for a sequence's only segment
    const bool only = seg.begin == seg.seq_begin && seg.end == seg.seq_end, via_ends = last && p.all_ends && !only && seg.end_at < p.n_ends;
    if (ENDS && last && !via_ends) return;
    const int w = wave_id(), l = lane_id(), q = l >> 4, j = l & 15;
    const int col0 = hb * COLS, head0 = col0 / p.P, mine = w * 16 / P, head = head0 + mine, grp = head0 / p.heads_per_group;
    const int wc = w * 16;                        // this wave's first column
    const int gh = w % NH, gc = w / NH;           // the head and the chunk of a group whose gates it forms
    const bool gater = gc < GC;
    const float A = uniform(p.A[head0 + gh]), bias = p.bias ? uniform(p.bias[head0 + gh]) : 0.f;
    const float Dh = p.D ? uniform(p.D[head]) : 0.f;

    // h[nb][e] = S[row_of(nb, e)][column wc + j]
    float4v h[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) h[i] = float4v{0.f, 0.f, 0.f, 0.f};
    auto row_of = [&](int nb, int e) { return 32 * (nb >> 1) + 8 * q + 4 * (nb & 1) + e; };
    auto state_at = [&](const int l) {            // of h[0][0] in s0 and sT, less 8 q rows
        const int col = col0 + wc + (l & 15);
        return ((int64_t)seg.seq * p.H + col / p.P) * N * p.P + col % p.P;
    };
    if constexpr (!ENDS) {
        const float d = segments_before<REV>(p, seg, hb, NH, mine, [&](int64_t at, float f) {
            const float *e0 = p.ends + at * (N * COLS) + wc + j;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) h[nb][e] += f * e0[row_of(nb, e) * COLS];
        });
        if (p.s0) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) h[nb][e] += d * p.s0[state_at(l) + row_of(nb, e) * p.P];
        }
        if (p.sT && via_ends) {
            // the state behind the last segment, from that segment's own
            const int64_t mark = (int64_t)seg.end_at * p.n_hb + hb;
            const float *e0 = p.ends + mark * (N * COLS) + wc + j;
            const float f = fast_exp2((float)p.total[mark * NH + mine]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p.sT[state_at(l) + row_of(nb, e) * p.P] = f * h[nb][e] + e0[row_of(nb, e) * COLS];
        }
        // the blocks of M right of the diagonal that a 32-wide step touches
        for (int i = threadIdx.x; i < NH * 2 * 16 * 16; i += kThreads) {
            const int hh = i >> 9, blk = (i >> 8) & 1, r = (i >> 4) & 15, c = i & 15;
            sm[hh][at<E, C>(32 * blk + r, 32 * blk + 16 + c)] = E(0);
        }
    }

    TileRegs<IO, COLS, REV, kThreads> tv;
    TileRegs<IO, N, REV, kThreads> tk, tq;
    const int64_t voff = seg.batch * p.vb + col0, koff = seg.batch * p.qkb + (int64_t)grp * N;
    const int nc = chunks_of(seg);
    auto fetch = [&](int c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo), tid = again(threadIdx.x);
        tv.load(tid, p.v, voff + lo * p.vt, (uint32_t)p.vt, rows);
        tk.load(tid, p.k, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
        if constexpr (!ENDS) tq.load(tid, p.q, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
    };
    uint32_t raw = 0;
    auto fetch_dt = [&](int c) {                  // of this wave's chunk of the group at c
        if (gater && c + gc < nc) {
            int lo;
            const int rows = chunk_of<REV>(seg, c + gc, lo);
            raw = raw_dt<IO, REV>(p, seg.batch, head0 + gh, lo, rows);
        }
    };
    auto form_gates = [&](int c) {
        if (gater && c + gc < nc) {
            int lo;
            const int rows = chunk_of<REV>(seg, c + gc, lo);
            const bool live = again(lane_id()) < rows;
            make_gates<REV>(gates[gc][gh], dt_of(p, raw_value<IO>(p, raw), bias, live), A, live, 1.f, 1.f);
        }
    };
    double total = 0.0;
    if (nc > 0) {
        fetch_dt(0);
        fetch(0);
    }
    for (int c = 0; c < nc; ++c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo), tid = again(threadIdx.x), l = tid & 63, q = l >> 4, j = l & 15;
        const Lane<E, N> aN(l);
        const Lane<E, COLS> aP(l);
        const Lane<E, C> aM(l);
        lds_barrier();                            // the last chunk's tiles are done with
        if (c % GC == 0) form_gates(c);
        tv.put(tid, sv, rows);
        tk.put(tid, sk, rows);
        if constexpr (!ENDS) tq.put(tid, sq, rows);
        if (c + 1 < nc) fetch(c + 1);
        if (c % GC == 0) fetch_dt(c + GC);
        lds_barrier();
        const Gates *gs = gates[c % GC], &g = gs[mine];
        float4v y[ENDS ? 1 : 4];
        bool plain = true;
        if constexpr (!ENDS && !REV) {
            // is every value of this wave's columns a number?
            float4v z = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s0 = 0; s0 < C; s0 += 32) O::times_zero(z, O::template col<COLS>(sv, aP, wc, s0));
            plain = __ballot((z[0] + z[1]) + (z[2] + z[3]) != 0.f) == 0;
        }
        if constexpr (!ENDS) {
            // 1: M[i][k] = (q_i . k_k) e^(cum_i - cum_k) w_k, k <= i
#pragma unroll
            for (int r = 0; r < (10 + NW - 1) / NW; ++r) {
                const int idx = w + NW * r;
                if (idx < 10) {
                    const int bi = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bk = idx - bi * (bi + 1) / 2;
                    float4v s = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += 32)
                        O::mma(s, O::template row<N>(sk, aN, 16 * bk, n0), O::template row<N>(sq, aN, 16 * bi, n0));
                    const int ii = 16 * bi + j;
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        const int k = 16 * bk + 4 * q;
                        O::put4(&sm[hh][at<E, C>(ii, k)], until(ii, k, s * decays<REV>(gs[hh], ii, k)));
                    }
                }
            }
            // out1^T = S^T q^T, then times e^cum
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 32) {
                typename O::frag hf[1];
                O::acc(h[n0 / 16], h[n0 / 16 + 1], hf);
#pragma unroll
                for (int bi = 0; bi < 4; ++bi) O::mma(y[bi], hf[0], O::template row<N>(sq, aN, 16 * bi, n0));
            }
#pragma unroll
            for (int bi = 0; bi < 4; ++bi) y[bi] *= g.ecum[16 * bi + j];
        }
        if constexpr (!ENDS) lds_barrier();       // M is whole
        // 2; its stores go out before the state's part, which they have time
        // to end behind (the next tiles wait for everything in flight)
        if constexpr (!ENDS) {
            if (plain) {
#pragma unroll
                for (int s0 = 0; s0 < C; s0 += 32) {
                    const typename O::frag vf = O::template col<COLS>(sv, aP, wc, s0);
#pragma unroll
                    for (int bi = s0 / 16; bi < 4; ++bi) O::mma(y[bi], vf, O::template row<C>(sm[mine], aM, 16 * bi, s0));
                }
            } else {
                // M's zeros times what is none would reach the rows before it: row by row
                // instead (to ask costs 0.5 to 0.8 % of 65536 tokens, 64 heads)
#pragma unroll
                for (int bi = 0; bi < 4; ++bi) {
                    const int ii = 16 * bi + j;
                    for (int k = 0; k <= ii; ++k) {
                        float x[4];
                        O::get4(&sv[at<E, COLS>(k, wc + 4 * q)], x);
                        const float m = O::get(sm[mine][at<E, C>(ii, k)]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[bi][e] += m * x[e];
                    }
                }
            }
            // y = out1 + D x, dx = dt out1 + D dy
            const rsrc_t ry = make_rsrc((IO *)p.out + seg.batch * p.ob + lo * p.ot + col0, 0x7fffffffu);
#pragma unroll
            for (int bi = 0; bi < 4; ++bi) {
                const int ii = 16 * bi + j, t = REV ? rows - 1 - ii : ii, cc = wc + 4 * q;
                const float post = REV ? g.dt[ii] : 1.f;
                float x[4];
                O::get4(&sv[at<E, COLS>(ii, cc)], x);
                float4v o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = post * y[bi][e] + Dh * x[e];
                store_row4<IO>(ry, ii < rows ? (uint32_t)(t * (uint32_t)p.ot + cc) * (uint32_t)sizeof(IO) : 0xfffffff0u, o);
            }
        }
        // 3
        const double tot = g.total;
        if constexpr (ENDS) total += tot;
        const float et = fast_exp2((float)tot);
#pragma unroll
        for (int i = 0; i < NB; ++i) h[i] *= et;
        // parts [from, to) of w v
        auto add_parts = [&](auto from, auto to) {
            constexpr int k0 = decltype(from)::value, k1 = decltype(to)::value;
#pragma unroll
            for (int s0 = 0; s0 < C; s0 += 32) {
                float wt[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) wt[e] = g.end[s0 + 8 * q + e];
                typename O::frag vw[k1];
                O::scaled(O::template col<COLS>(sv, aP, wc, s0), wt, vw);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const typename O::frag kf = O::template pair<N>(sk, aN, 32 * (nb >> 1), nb & 1, s0);
#pragma unroll
                    for (int k = k0; k < k1; ++k) O::mma(h[nb], kf, vw[k]);
                }
            }
        };
        typedef std::integral_constant<int, 0> I0;
        typedef std::integral_constant<int, 1> I1;
        typedef std::integral_constant<int, kP> IP;
        if constexpr (ENDS) {
            add_parts(I0(), IP());
        } else {
            add_parts(I0(), I1());
            if constexpr (kP > 1) {
                if (only) add_parts(I1(), IP());
            }
        }
    }
    if constexpr (ENDS) {
        const int64_t place_at = (int64_t)unit * p.n_hb + hb;
        float *e0 = p.ends + place_at * (N * COLS) + wc + j;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) e0[row_of(nb, e) * COLS] = h[nb][e];
        if (!REV && l == 0 && w == mine * (NW / NH)) p.total[place_at * NH + mine] = total;
    } else if (p.sT && only) {
        const int l = again(lane_id()), q = l >> 4;
        float *sT = p.sT + state_at(l) + 8 * q * p.P;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) sT[(32 * (nb >> 1) + 4 * (nb & 1) + e) * p.P] = h[nb][e];
    }
}

// n_ends: places for the end states of sequences with several segments
struct SsmPlan {
    int ncb, nh, n_hb, n_items, n_ends, seg_tokens, seqs;
};

gdn_status check_ssm(const gdn_ssm_problem *pr, bool packed);
gdn_status check_ssm_pointers(const gdn_ssm_problem *pr, const void *x, const void *dt, const float *A, const void *Bm,
                              const void *Cm, const float *D, const float *bias, bool rows);
void fill_ssm(const gdn_ssm_problem *pr, SsmParams &sp);
SsmPlan ssm_plan(const gdn_ssm_problem *pr, bool packed);
int ssm_grid(const gdn_ssm_problem *pr, SsmParams &sp, const SsmPlan &s, bool ends);

}  // namespace gdn

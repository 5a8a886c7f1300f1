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
// anew every four chunks, and at a segment's end, as <h, dh>: the forward scan
// leaves h there, and the reverse one meets it with dh.  (dA of 2 x 8192
// tokens, 32 heads: 1.2e-5 off with X passed on over 16 chunks.)
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
    // the scan's rows and results (see above)
    const void *q, *q2, *k, *v, *dt;
    const float *A, *D, *bias, *s0;         // s0: the state behind the first segment (h0; dhT)
    void *out;                              // out1's rows (y; dx) or out2's (dC; dB)
    float *sT;                              // the state behind the last one (hT; dh0)
    const int32_t *cu;
    int64_t qkb, qkt, vb, vt, q2b, q2t, db, dt_, ob, ot;   // strides: batch, token
    // workspace
    double *total;                          // [item][n_hb][NH]: log2 of a segment's decay
    float *ends;                            // [item][n_hb][N][64 NCB]: end states from zero
    float *part;                            // out2 by block of columns, for ssm_sum_kernel
    float *inside, *across;                 // [n_hb][NH][B T]: q . out2 in two parts
    float *dyx, *wtt;                       // the same: dy_t . x_t, and W_tt / dt_t
    float *marks;                           // [place][n_hb][N][64 NCB]: h every four chunks
    double *X;                              // [place][n_hb][NH]: <h, dh> there
    int64_t rows;                           // B T
    int n_slots, n_marks;                   // places for chunks in part, and for marks
    int T, H, P, n_seqs, heads_per_group;
    int seg_tokens, n_items, n_hb;          // tokens of a segment, segments in all, blocks of columns
    int softplus, swizzle, dt_f32;
};

// Operands of the matrix cores by io type: bf16 products for bf16 io, fp32
// products for fp32 io.  Both take eight k slots a lane.
template <typename IO> struct SOp;

template <> struct SOp<bf16_t> {
    typedef uint16_t elem;
    typedef bf16x8 frag;
    static constexpr int kPad = 8;
    template <int PARTS> static constexpr int kParts = PARTS;
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
    // an fp32 operand in PARTS bf16 ones, each holding what rounding left over
    // of those before: a relative error of 2^-9, 2^-18 or 2^-27 at most
    template <int PARTS>
    __device__ static void parts_of(const float (&v)[8], frag (&f)[PARTS]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x = v[e];
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                f[k][e] = (__bf16)x;
                x -= (float)f[k][e];
            }
        }
    }
    template <int PARTS>
    __device__ static void acc_split(const float4v &lo, const float4v &hi, frag (&f)[PARTS]) {
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        parts_of(v, f);
    }
    // w .* a
    template <int PARTS>
    __device__ static void scaled(const frag &a, const float (&w)[8], frag (&f)[PARTS]) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)a[e] * w[e];
        parts_of(v, f);
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
    template <int PARTS> static constexpr int kParts = 1;
    __device__ static void mma(float4v &acc, const frag &a, const frag &b) { Mma<float>::mma(acc, a, b); }
    __device__ static frag row(const elem *S, int ld, int m0, int k0) { return Mma<float>::load(frag_ptr(S + m0 * ld, ld, k0)); }
    __device__ static frag col(const elem *S, int ld, int m0, int k0) { return frag_T(S, ld, m0, k0); }
    __device__ static frag row_split(const elem *S, int ld, int m0, int k0) { return fragA_split(S, ld, m0, k0); }
    template <int PARTS>
    __device__ static void acc_split(const float4v &lo, const float4v &hi, frag (&f)[PARTS]) { f[0] = frag{lo, hi}; }
    template <int PARTS>
    __device__ static void scaled(const frag &a, const float (&w)[8], frag (&f)[PARTS]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[0].lo[e] = a.lo[e] * w[e];
            f[0].hi[e] = a.hi[e] * w[4 + e];
        }
    }
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

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ double wave_scan(double v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double u = __shfl_up(v, m, 64);
        if (lane_id() >= m) v += u;
    }
    return v;
}

// A chunk's gates of one head, a lane a row.
struct Gates {
    float2 cum[kSsmChunk];      // log2 of the decay from the chunk's start to the row
    float ecum[kSsmChunk];      // that decay
    float end[kSsmChunk];       // w times the decay from the row to the chunk's end
    float w[kSsmChunk];
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

template <bool REV>
__device__ __forceinline__ void make_gates(Gates &g, float dt, float A) {
    const int l = lane_id();
    const double own = (double)dt * (double)A * 1.4426950408889634074, upto = wave_scan(own);
    const double total = __shfl(upto, 63, 64), cum = REV ? upto - own : upto;
    const float hi = (float)cum, w = REV ? 1.f : dt;
    g.cum[l] = make_float2(hi, (float)(cum - (double)hi));
    g.ecum[l] = fast_exp2(hi);
    g.end[l] = w * fast_exp2((float)(total - cum));
    g.w[l] = w;
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

// 64 rows of COLS elements from HBM through registers into LDS, 16 bytes a
// lane and step, in scan order (REV: from the last of `rows` to the first);
// rows at or past `rows` as zeros.
template <typename IO, int COLS, bool REV>
struct TileRegs {
    static constexpr int kPer = 16 / sizeof(IO), kLine = COLS / kPer, kN = kSsmChunk * kLine / 256;
    u32x4 v[kN];
    __device__ __forceinline__ void load(const void *base, int64_t elems, uint32_t stride, int rows) {
        const rsrc_t r = make_rsrc((const IO *)base + elems, 0x7fffffffu);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int k = i * 256 + threadIdx.x, t = k / kLine, c = k % kLine * kPer;
            const uint32_t off = ((REV ? rows - 1 - t : t) * stride + c) * (uint32_t)sizeof(IO);
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
// The place of the state behind a chunk, or -1 where none is kept: behind
// every fourth chunk of a sequence and behind a segment's last (a segment is a
// multiple of four chunks, unless it is a sequence's last).
__device__ __forceinline__ int mark_slot(const SsmParams &p, const Segment &s, int c) {
    const int in = (s.begin - s.seq_begin) / kSsmChunk + c;
    if ((in & 3) != 3 && c != chunks_of(s) - 1) return -1;
    const int per = 4 * kSsmChunk;
    const int m = (p.cu ? s.seq_begin / per + s.seq : s.seq * ((p.T + per - 1) / per)) + in / 4;
    return m < p.n_marks ? m : -1;
}

// The raw dt of row l of a chunk.
template <typename IO, bool REV>
__device__ __forceinline__ float raw_dt(const SsmParams &p, int batch, int head, int lo, int rows) {
    const int l = lane_id();
    if (l >= rows) return 0.f;
    const int64_t at = batch * p.db + (lo + (REV ? rows - 1 - l : l)) * p.dt_ + head;
    return p.dt_f32 ? ((const float *)p.dt)[at] : io_traits<IO>::load((const IO *)p.dt + at);
}

// For every segment that the scan passes before this one, nearest first:
// f(its place in the workspace, the decay between it and this one); returns
// the decay since the scan's very start.
template <bool REV, typename F>
__device__ __forceinline__ float segments_before(const SsmParams &p, const Segment &s, int hb, int nh, int hh, F f) {
    double d = 0.0;
    const int per = (s.seq_end - s.seq_begin + p.seg_tokens - 1) / p.seg_tokens;
    const int stop = REV ? s.first + per : s.first - 1;
    for (int i = REV ? s.item + 1 : s.item - 1; i != stop && (REV ? i < stop : i > stop); i += REV ? 1 : -1) {
        const int64_t at = (int64_t)i * p.n_hb + hb;
        f(at, fast_exp2((float)d));
        d += p.total[at * nh + hh];
    }
    return fast_exp2((float)d);
}

// ---------------------------------------------------------------------------
// out1, the state, or both.  A wave keeps the state of its columns, all N
// rows of them, in accumulators, and uses them as operands without a trip
// through LDS.  Per chunk:
//   1  the lower triangle of q k^T, times decays and weights, to LDS (16 x 16
//      blocks, dealt to the waves); S^T q on the way
//   2  out1 = M v + e^cum S^T q, transposed, so that a lane stores four columns
//   3  S' = e^total S + k^T (w v)
// The state's products take w v in PARTS bf16 parts: two (relative error 2^-18)
// for a state that is an output and is read on by every later chunk, three
// where it goes into dA, a sum over all tokens of both signs in which two
// left errors of up to 5e-5.  out1's operands are rounded once to bf16,
// its own type.  The next chunk's rows are in flight while one is worked on.
// ENDS: only the state, from a zero start, to the workspace.
// ---------------------------------------------------------------------------
template <typename IO, int N, int NCB, bool ENDS, bool REV, int PARTS>
__global__ void __launch_bounds__(256) ssm_scan_kernel(SsmParams p) {
    typedef SOp<IO> O;
    typedef typename O::elem E;
    constexpr int C = kSsmChunk, COLS = 64 * NCB, LX = COLS + O::kPad, LN = N + O::kPad, LM = C + O::kPad;
    constexpr int NH = NCB, NB = N / 16;          // heads at most; row blocks of the state
    constexpr int kP = O::template kParts<PARTS>;
    __shared__ E sv[C * LX], sk[C * LN], sq[ENDS ? 1 : C * LN], sm[ENDS ? 1 : NH][ENDS ? 1 : C * LM];
    __shared__ Gates gates[NH];
    int item, hb;
    place(p, item, hb);
    if (item >= p.n_items) return;
    const Segment seg = find_segment(p, item);
    if (!seg.live) return;
    if (ENDS && (REV ? seg.begin == seg.seq_begin : seg.end == seg.seq_end)) return;
    const int w = wave_id(), l = lane_id(), q = l >> 4, j = l & 15;
    const int col0 = hb * COLS, head0 = col0 / p.P, nh = p.P == 64 ? NCB : 1;
    const int mine = nh == 2 ? w >> 1 : 0, head = head0 + mine, grp = head0 / p.heads_per_group;
    const int wc = w * 16 * NCB;                  // this wave's first column
    const bool gater = w < nh;                    // waves that form the gates of head0 + w
    const float A = gater ? p.A[head0 + w] : 0.f, bias = gater && p.bias ? p.bias[head0 + w] : 0.f;
    const float Dh = p.D ? p.D[head] : 0.f;

    // h[cb * NB + nb][e] = S[16 nb + 4 q + e][column wc + 16 cb + j]
    float4v h[NCB * NB];
#pragma unroll
    for (int i = 0; i < NCB * NB; ++i) h[i] = float4v{0.f, 0.f, 0.f, 0.f};
    const int64_t hoff = ((int64_t)seg.seq * p.H * N) * p.P;
    auto hidx = [&](int cb, int nb, int e) {
        const int col = col0 + wc + 16 * cb + j;
        return hoff + ((int64_t)(col / p.P) * N + 16 * nb + 4 * q + e) * p.P + col % p.P;
    };
    const int ends_at = 4 * q * COLS + wc + j;    // of h[0][0] in a segment's [N][COLS]
    if constexpr (!ENDS) {
        const float d = segments_before<REV>(p, seg, hb, NH, mine, [&](int64_t at, float f) {
            const float *e0 = p.ends + at * (N * COLS) + ends_at;
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[cb * NB + nb][e] += f * e0[(16 * nb + e) * COLS + 16 * cb];
        });
        if (p.s0) {
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[cb * NB + nb][e] += d * p.s0[hidx(cb, nb, e)];
        }
        // the blocks of M right of the diagonal that a 32-wide step touches
        for (int i = threadIdx.x; i < NH * 2 * 16 * 16; i += 256) {
            const int hh = i >> 9, blk = (i >> 8) & 1, r = (i >> 4) & 15, c = i & 15;
            sm[hh][(32 * blk + r) * LM + 32 * blk + 16 + c] = E(0);
        }
    }

    TileRegs<IO, COLS, REV> tv;
    TileRegs<IO, N, REV> tk, tq;
    float raw = 0.f;
    const int64_t voff = seg.batch * p.vb + col0, koff = seg.batch * p.qkb + (int64_t)grp * N;
    auto fetch = [&](int c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo);
        tv.load(p.v, voff + lo * p.vt, (uint32_t)p.vt, rows);
        tk.load(p.k, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
        if constexpr (!ENDS) tq.load(p.q, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
        if (gater) raw = raw_dt<IO, REV>(p, seg.batch, head0 + w, lo, rows);
    };
    double total = 0.0;
    const int nc = chunks_of(seg);
    if (nc > 0) fetch(0);
    for (int c = 0; c < nc; ++c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo);
        __syncthreads();                          // the last chunk's tiles are done with
        tv.put(sv, LX);
        tk.put(sk, LN);
        if constexpr (!ENDS) tq.put(sq, LN);
        if (gater) make_gates<REV>(gates[w], dt_of(p, raw, bias, l < rows), A);
        if (c + 1 < nc) fetch(c + 1);
        __syncthreads();
        const Gates &g = gates[mine];
        float4v y[ENDS ? 1 : NCB * 4];
        if constexpr (!ENDS) {
            // 1: M[i][k] = (q_i . k_k) e^(cum_i - cum_k) w_k, k <= i
#pragma unroll
            for (int r = 0; r < 3; ++r) {
                const int idx = w + 4 * r;
                if (idx < 10) {
                    const int bi = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bk = idx - bi * (bi + 1) / 2;
                    float4v s = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += 32)
                        O::mma(s, O::row(sk, LN, 16 * bk, n0), O::row(sq, LN, 16 * bi, n0));
                    const int ii = 16 * bi + j;
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh)
                        if (hh < nh) {
                            float4v m;
                            const float2 ci = gates[hh].cum[ii];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kk = 16 * bk + 4 * q + e;
                                m[e] = kk <= ii ? s[e] * decay_between(ci, gates[hh].cum[kk]) * gates[hh].w[kk] : 0.f;
                            }
                            O::put4(&sm[hh][ii * LM + 16 * bk + 4 * q], m);
                        }
                }
            }
            // out1^T = S^T q^T, then times e^cum
#pragma unroll
            for (int i = 0; i < NCB * 4; ++i) y[i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 32) {
                typename O::frag hf[NCB][1];
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) O::acc_split(h[cb * NB + n0 / 16], h[cb * NB + n0 / 16 + 1], hf[cb]);
#pragma unroll
                for (int bi = 0; bi < 4; ++bi) {
                    const typename O::frag qf = O::row_split(sq, LN, 16 * bi, n0);
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) O::mma(y[cb * 4 + bi], hf[cb][0], qf);
                }
            }
#pragma unroll
            for (int bi = 0; bi < 4; ++bi) {
                const float ec = g.ecum[16 * bi + j];
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) y[cb * 4 + bi] *= ec;
            }
            __syncthreads();                      // M is whole
        }
        // 2 and 3: both take v by columns
        const double tot = g.total;
        total += tot;
        const float et = fast_exp2((float)tot);
#pragma unroll
        for (int i = 0; i < NCB * NB; ++i) h[i] *= et;
#pragma unroll
        for (int s0 = 0; s0 < C; s0 += 32) {
            float wt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wt[e] = g.end[s0 + 8 * q + e];
            typename O::frag vf[NCB], vw[NCB][kP];
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                vf[cb] = O::col(sv, LX, wc + 16 * cb, s0);
                O::scaled(vf[cb], wt, vw[cb]);
            }
            if constexpr (!ENDS) {
#pragma unroll
                for (int bi = s0 / 16; bi < 4; ++bi) {
                    const typename O::frag mf = O::row(sm[mine], LM, 16 * bi, s0);
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) O::mma(y[cb * 4 + bi], vf[cb], mf);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const typename O::frag kf = O::col(sk, LN, 16 * nb, s0);
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                    for (int k = 0; k < kP; ++k) O::mma(h[cb * NB + nb], kf, vw[cb][k]);
            }
        }
        if constexpr (!ENDS) {
            // y = out1 + D x, dx = dt out1 + D dy
            const rsrc_t ry = make_rsrc((IO *)p.out + seg.batch * p.ob + lo * p.ot + col0, 0x7fffffffu);
#pragma unroll
            for (int bi = 0; bi < 4; ++bi) {
                const int ii = 16 * bi + j, t = REV ? rows - 1 - ii : ii;
                const float post = REV ? g.dt[ii] : 1.f;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) {
                    const int cc = wc + 16 * cb + 4 * q;
                    float x[4];
                    O::get4(&sv[ii * LX + cc], x);
                    float4v o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = post * y[cb * 4 + bi][e] + Dh * x[e];
                    const uint32_t off = ii < rows ? (uint32_t)(t * (uint32_t)p.ot + cc) * (uint32_t)sizeof(IO) : 0xfffffff0u;
                    store_row4<IO>(ry, off, o);
                }
            }
        }
    }
    if constexpr (ENDS) {
        const int64_t at = (int64_t)item * p.n_hb + hb;
        float *e0 = p.ends + at * (N * COLS) + ends_at;
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) e0[(16 * nb + e) * COLS + 16 * cb] = h[cb * NB + nb][e];
        if (!REV && l == 0 && (nh == 1 ? w == 0 : (w & 1) == 0)) p.total[at * NH + mine] = total;
    } else if (p.sT && (REV ? seg.begin == seg.seq_begin : seg.end == seg.seq_end)) {
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) p.sT[hidx(cb, nb, e)] = h[cb * NB + nb][e];
    }
}

struct SsmPlan {
    int ncb, n_hb, n_items, seg_tokens, seqs;
};

gdn_status check_ssm(const gdn_ssm_problem *pr, bool packed);
gdn_status check_ssm_pointers(const gdn_ssm_problem *pr, const void *x, const void *dt, const float *A, const void *Bm,
                              const void *Cm, const float *D, const float *bias, bool rows);
void fill_ssm(const gdn_ssm_problem *pr, SsmParams &sp);
SsmPlan ssm_plan(const gdn_ssm_problem *pr, bool packed);
int ssm_grid(SsmParams &sp, const SsmPlan &s);

}  // namespace gdn

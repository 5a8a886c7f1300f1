// Selective state space scan, backward: dx by the reverse scan of
// ssm_scan_kernel, dC and dB by ssm_key_kernel in either direction, and the
// gates' gradients from the sums the two leave (see gdn_ssm.h).
#include "gdn_ssm.h"

namespace gdn {

// ---------------------------------------------------------------------------
// out2 (dC forward, dB in reverse), and per head and row the sum
// q_i . out2_i.  Here wave w keeps rows 16 w .. +15 of the state, all columns of
// them: S q2 sums over columns.  Per chunk:
//   1  the lower triangles of q k^T and q2 v^T; the products of both, times
//      decays and weights, sum up to the rows' part inside the chunk; those
//      of q2 v^T alone, summed over the heads here, go to LDS as M
//   2  out2 = e^cum S q2 + M k, transposed, so that a lane holds four of the
//      N values of a row
//   3  S' = e^total S + (w k)^T v
// S enters its product in three bf16 parts and (w k) in three (relative error
// 2^-27): the sums feed dt's and A's gradients, which are fp32.  M is rounded
// once to out2's own type.
//
// S changes its sign from chunk to chunk (its weights and decays bring that
// about).  The matrix cores' sums lean to one side by some 2.5e-10 of their
// terms, which inputs of one sign (x, B and C behind a silu) add up over N x P
// products to 3e-8 of X a chunk, always the same way: over 16384 tokens dA was
// 2.6e-6 and d(dt_bias) 4.9e-6 off.  With the sign alternating the chunks'
// shares cancel (4.7e-7 and 1.9e-6 at the same inputs).  What is left varies with
// the inputs: over ten seeds, with the gate kernel's part below, dA is 0.2 to
// 5e-6 of its norm off and d(dt_bias) 1 to 3.3e-6.
//
// 2 x 8192 tokens, 32 heads of 128 x 128: 246 and 267 us in the two directions, of
// which the products are 100 us at a large product's rate and the 268 MB that
// the heads leave for ssm_sum_kernel 55 us at a copy's.  A group's heads do not
// fit one workgroup (a state is 64 KB of registers), and atomic sums would
// depend on their order.
// ---------------------------------------------------------------------------
template <typename IO, int N, int COLS, int NH, bool REV>
__global__ void __launch_bounds__(4 * N, sizeof(IO) == 4 ? 1 : NH == 1 && N == 128 ? 4 : 2) ssm_key_kernel(SsmParams p) {
    typedef SOp<IO> O;
    typedef typename O::elem E;
    constexpr int C = kSsmChunk, NW = N / 16, PB = COLS / 16, kThreads = 4 * N;      // PB: blocks of columns
    constexpr int kP = O::template kParts<3>;
    __shared__ __align__(16) E sv[C * COLS], sz[C * COLS], sk[C * N], sq[C * N], sm[C * C];
    // chunks whose gates are formed at once, one chunk and head a wave
    constexpr int GC = 2;
    __shared__ Gates gates[GC][NH];
    __shared__ float inner[NH][4][C], outer[NH][NW][C], dots[NH][NW];
    int unit, hb;
    place(p, unit, hb);
    if (unit >= p.n_units) return;
    const Segment seg = find_segment<false>(p, unit);
    if (!seg.live) return;
    const int w = wave_id(), l = lane_id(), q = l >> 4, j = l & 15;
    const int col0 = hb * COLS, head0 = col0 / p.P, grp = head0 / p.heads_per_group;
    const int wn = 16 * w;                        // this wave's first row of the state
    const int gh = w % NH, gc = w / NH;           // the head and the chunk of a group whose gates it forms
    const bool gater = gc < GC;
    const float A = uniform(p.A[head0 + gh]), bias = p.bias ? uniform(p.bias[head0 + gh]) : 0.f;

    // h[pb][e] = S[n = wn + j][column col_of(pb, e)]
    float4v h[PB];
#pragma unroll
    for (int i = 0; i < PB; ++i) h[i] = float4v{0.f, 0.f, 0.f, 0.f};
    auto col_of = [&](int pb) { return 32 * (pb >> 1) + 8 * q + 4 * (pb & 1); };      // of e = 0
#pragma unroll
    for (int hh = 0; hh < NH; ++hh) {
        const float d = segments_before<REV>(p, seg, hb, NH, hh, [&](int64_t at, float f) {
            const float *e0 = p.ends + at * (N * COLS) + (wn + j) * COLS;
#pragma unroll
            for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) h[pb] += f * *(const float4v *)(e0 + col_of(pb));
        });
        if (p.s0) {
#pragma unroll
            for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) {
                const int col = col0 + col_of(pb);
                const float *s = p.s0 + (((int64_t)seg.seq * p.H + col / p.P) * N + wn + j) * p.P + col % p.P;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[pb][e] += d * s[e];
            }
        }
    }
    for (int i = threadIdx.x; i < 2 * 16 * 16; i += kThreads) {
        const int blk = i >> 8, r = (i >> 4) & 15, c = i & 15;
        sm[at<E, C>(32 * blk + r, 32 * blk + 16 + c)] = E(0);
    }

    TileRegs<IO, COLS, REV, kThreads> tv, tz;
    TileRegs<IO, N, REV, kThreads> tk, tq;
    const int64_t voff = seg.batch * p.vb + col0, zoff = seg.batch * p.q2b + col0, koff = seg.batch * p.qkb + (int64_t)grp * N;
    const int nc = chunks_of(seg);
    auto fetch = [&](int c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo), tid = again(threadIdx.x);
        tv.load(tid, p.v, voff + lo * p.vt, (uint32_t)p.vt, rows);
        tz.load(tid, p.q2, zoff + lo * p.q2t, (uint32_t)p.q2t, rows);
        tk.load(tid, p.k, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
        tq.load(tid, p.q, koff + lo * p.qkt, (uint32_t)p.qkt, rows);
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
            make_gates<REV>(gates[gc][gh], dt_of(p, raw_value<IO>(p, raw), bias, live), A, live,
                             (c + gc) & 1 ? -1.f : 1.f, (c + gc) & 1 ? 1.f : -1.f);
        }
    };
    if (nc > 0) {
        fetch_dt(0);
    }
    for (int c = 0; c < nc; ++c) {
        int lo;
        const int rows = chunk_of<REV>(seg, c, lo), tid = again(threadIdx.x), l = tid & 63, q = l >> 4, j = l & 15;
        const Lane<E, N> aN(l);
        const Lane<E, COLS> aP(l);
        const Lane<E, C> aM(l);
        // (not a chunk ahead: the registers that would take leave one workgroup a
        // CU; the other one's work covers the wait)
        fetch(c);
        lds_barrier();                            // the last chunk's tiles and sums are done with
        if (c % GC == 0) {
            form_gates(c);
            fetch_dt(c + GC);
        }
        tv.put(tid, sv, rows);
        tz.put(tid, sz, rows);
        tk.put(tid, sk, rows);
        tq.put(tid, sq, rows);
        const Mark mark = mark_of(p, seg, REV ? nc - 1 - c : c);
        if constexpr (REV) {
            // behind this chunk h meets the state's gradient
            if (mark.state >= 0) {
                const float2 *m = (const float2 *)p.marks + ((int64_t)mark.state * p.n_hb + hb) * (N * COLS / 2) + tid;
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float d = 0.f;
#pragma unroll
                    for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) {
                        const float2 a = m[(2 * pb) * kThreads], b = m[(2 * pb + 1) * kThreads];
                        d += a.x * h[pb][0] + a.y * h[pb][1] + b.x * h[pb][2] + b.y * h[pb][3];
                    }
                    d = wave_sum(d);
                    if (l == 0) dots[hh][w] = d;
                }
            }
        }
        lds_barrier();
        const Gates *gs = gates[c % GC];
        if constexpr (REV) {
            if (mark.state >= 0 && mark.x >= 0 && w < NH && l == 0) {
                double d = 0.0;
#pragma unroll
                for (int k = 0; k < NW; ++k) d += (double)dots[w][k];
                // h behind chunk nc - 1 - c has that one's sign turned, dh chunk c's
                p.X[((int64_t)mark.x * p.n_hb + hb) * NH + w] = nc & 1 ? -d : d;
            }
        }
        // 1
        const int64_t row0 = (int64_t)seg.batch * p.T + lo;
#pragma unroll
        for (int r = 0; r < (10 + NW - 1) / NW; ++r) {
            const int idx = w + NW * r;
            if (idx < 10) {
                const int bi = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bk = idx - bi * (bi + 1) / 2;
                const int ii = 16 * bi + j, k0 = 16 * bk + 4 * q;
                float4v s = float4v{0.f, 0.f, 0.f, 0.f}, m = s;
#pragma unroll
                for (int n0 = 0; n0 < N; n0 += 32) O::mma(s, O::template row<N>(sk, aN, 16 * bk, n0), O::template row<N>(sq, aN, 16 * bi, n0));
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float4v x = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = hh * (COLS / NH); k < (hh + 1) * (COLS / NH); k += 32)
                        O::mma(x, O::template row<COLS>(sv, aP, 16 * bk, k), O::template row<COLS>(sz, aP, 16 * bi, k));
                    const float4v d = until(ii, k0, x * decays<REV>(gs[hh], ii, k0));
                    m += d * (REV ? gs[hh].dt[ii] : 1.f);
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum += k0 + e < ii ? d[e] * s[e] : 0.f;
                        if (!REV && k0 + e == ii && ii < rows) {
                            const int64_t to = ((int64_t)hb * NH + hh) * p.rows + row0 + ii;
                            p.dyx[to] = x[e];
                            p.wtt[to] = x[e] * s[e];
                        }
                    }
                    sum += __shfl_xor(sum, 16, 64);
                    sum += __shfl_xor(sum, 32, 64);
                    if (q == 0) inner[hh][bk][ii] = sum;
                }
                O::put4(&sm[at<E, C>(ii, k0)], m);
            }
        }
        // 2, the state's part: z = S q2 of every head, its sum with q, and
        // times e^cum the start of out2
        float4v z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            float4v a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); pb += 2) {
                typename O::frag hf[kP];
                O::acc(h[pb], h[pb + 1], hf);
#pragma unroll
                for (int bi = 0; bi < 4; ++bi) {
                    const typename O::frag zf = O::template row<COLS>(sz, aP, 16 * bi, 16 * pb);
#pragma unroll
                    for (int k = 0; k < kP; ++k) O::mma(a[bi], hf[k], zf);
                }
            }
#pragma unroll
            for (int bi = 0; bi < 4; ++bi) {
                const int ii = 16 * bi + j;
                float x[4], sum = 0.f;
                O::get4(&sq[at<E, N>(ii, wn + 4 * q)], x);
                a[bi] *= gs[hh].ecum[ii];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += a[bi][e] * x[e];
                z[bi] += a[bi] * (REV ? gs[hh].dt[ii] : 1.f);
                sum += __shfl_xor(sum, 16, 64);
                sum += __shfl_xor(sum, 32, 64);
                if (q == 0) outer[hh][w][ii] = sum;
            }
        }
        lds_barrier();                            // M and the sums are whole
        if (w < NH && l < rows) {
            // row l's sums, to the token's place
            const int64_t to = ((int64_t)hb * NH + w) * p.rows + row0 + (REV ? rows - 1 - l : l);
            float sum = 0.f, out = 0.f;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b <= l >> 4) sum += inner[w][b][l];
#pragma unroll
            for (int b = 0; b < NW; ++b) out += outer[w][b][l];
            p.inside[to] = sum;
            p.across[to] = out;
        }
        // 2; z goes out before the state's part
#pragma unroll
        for (int s0 = 0; s0 < C; s0 += 32) {
            const typename O::frag kf = O::template col<N>(sk, aN, wn, s0);
#pragma unroll
            for (int bi = s0 / 16; bi < 4; ++bi) O::mma(z[bi], kf, O::template row<C>(sm, aM, 16 * bi, s0));
        }
        // (the sum over the blocks of columns of a group follows in ssm_sum_kernel)
        const int slot = chunk_slot(p, seg, REV ? nc - 1 - c : c);
        if (slot < p.n_slots) {
            float2 *part = (float2 *)p.part + ((int64_t)slot * p.n_hb + hb) * (8 * kThreads) + tid;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part[(2 * i) * kThreads] = make_float2(z[i][0], z[i][1]);
                part[(2 * i + 1) * kThreads] = make_float2(z[i][2], z[i][3]);
            }
        }
        // 3
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            const float et = -fast_exp2((float)gs[hh].total);
#pragma unroll
            for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) h[pb] *= et;
        }
#pragma unroll
        for (int s0 = 0; s0 < C; s0 += 32) {
            const typename O::frag kf = O::template col<N>(sk, aN, wn, s0);
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                typename O::frag kw[kP];
                float wt[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) wt[e] = gs[hh].end[s0 + 8 * q + e];
                O::scaled(kf, wt, kw);
#pragma unroll
                for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) {
                    const typename O::frag vf = O::template pair<COLS>(sv, aP, 32 * (pb >> 1), pb & 1, s0);
#pragma unroll
                    for (int k = 0; k < kP; ++k) O::mma(h[pb], vf, kw[k]);
                }
            }
        }
        if constexpr (!REV) {
            if (mark.state >= 0) {
                float2 *m = (float2 *)p.marks + ((int64_t)mark.state * p.n_hb + hb) * (N * COLS / 2) + tid;
#pragma unroll
                for (int pb = 0; pb < PB; ++pb) {
                    m[(2 * pb) * kThreads] = make_float2(h[pb][0], h[pb][1]);
                    m[(2 * pb + 1) * kThreads] = make_float2(h[pb][2], h[pb][3]);
                }
            }
        }
    }
    if constexpr (!REV) {
        // behind a sequence: h, as the last chunk left its sign, and the final state's gradient
        if (nc == 0 || seg.end != seg.seq_end) return;
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
            float d = 0.f;
            if (p.dT) {
#pragma unroll
                for (int pb = hh * (PB / NH); pb < (hh + 1) * (PB / NH); ++pb) {
                    const int col = col0 + col_of(pb);
                    const float *s = p.dT + (((int64_t)seg.seq * p.H + col / p.P) * N + wn + j) * p.P + col % p.P;
#pragma unroll
                    for (int e = 0; e < 4; ++e) d += h[pb][e] * s[e];
                }
            }
            d = wave_sum(d);
            if (l == 0) dots[hh][w] = d;
        }
        lds_barrier();
        const Mark mark = mark_of(p, seg, nc - 1);
        if (mark.x >= 0 && w < NH && l == 0) {
            double d = 0.0;
#pragma unroll
            for (int k = 0; k < NW; ++k) d += (double)dots[w][k];
            p.X[((int64_t)mark.x * p.n_hb + hb) * NH + w] = nc & 1 ? -d : d;
        }
    }
}

// out2 of a chunk and group: the sum over the group's blocks of columns, in
// the lanes' own layout.  A workgroup for every place that a chunk can have (see
// chunk_slot), so that the launch grows with the tokens and the sequences, not
// with segments of which most are not there.
template <typename IO, int N, bool REV>
__global__ void __launch_bounds__(4 * N) ssm_sum_kernel(SsmParams p) {
    constexpr int kThreads = 4 * N;
    const int G = p.H / p.heads_per_group, g = blockIdx.x % G, slot = blockIdx.x / G;
    int batch = 0, lo = 0, rows = 0;
    if (!p.cu) {
        const int per = (p.T + kSsmChunk - 1) / kSsmChunk;
        batch = slot / per;
        lo = slot % per * kSsmChunk;
        rows = p.T - lo;
    } else {
        // the last sequence whose places begin at or before this one
        int n = 0, hi = p.n_seqs - 1;
        while (n < hi) {
            const int mid = (n + hi + 1) >> 1;
            if (ssm_cu(p, mid) / kSsmChunk + mid <= slot)
                n = mid;
            else
                hi = mid - 1;
        }
        const int begin = ssm_cu(p, n), in = slot - (begin / kSsmChunk + n);
        if (in < 0) return;
        lo = begin + in * kSsmChunk;
        rows = ssm_cu(p, n + 1) - lo;
    }
    if (rows <= 0) return;
    rows = rows < kSsmChunk ? rows : kSsmChunk;
    const int w = wave_id(), l = lane_id(), q = l >> 4, j = l & 15, per = p.n_hb / G;
    float4v z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = float4v{0.f, 0.f, 0.f, 0.f};
    const float2 *part = (const float2 *)p.part + ((int64_t)slot * p.n_hb + g * per) * (8 * kThreads) + threadIdx.x;
    for (int k = 0; k < per; ++k, part += 8 * kThreads) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = part[(2 * i) * kThreads], b = part[(2 * i + 1) * kThreads];
            z[i] += float4v{a.x, a.y, b.x, b.y};
        }
    }
    const rsrc_t r = make_rsrc((IO *)p.out + batch * p.ob + lo * p.ot + (int64_t)g * N, 0x7fffffffu);
#pragma unroll
    for (int bi = 0; bi < 4; ++bi) {
        const int ii = 16 * bi + j, t = REV ? rows - 1 - ii : ii;
        const uint32_t e = (uint32_t)t * (uint32_t)p.ot + 16 * w + 4 * q;
        store_row4<IO>(r, ii < rows ? e * (uint32_t)sizeof(IO) : 0xfffffff0u, z[bi]);
    }
}

// The gradients of a segment's gates, one head a workgroup, a chunk a wave
// (see gdn_ssm.h): ddt_t = c_t + A dg_t, through softplus; dA += dt_t dg_t.
// 21 us at 2 x 8192 tokens, 32 heads: six rows of floats a head and two barriers
// for every four chunks.
struct GateParams {
    SsmParams s;                          // the forward scan's
    const float *c_inside, *c_across;     // the reverse scan's sums
    void *ddt;
    double *grads;                        // [3][item][H]: dA, d(dt_bias), dD
    float *dA, *dD, *dbias;
    int ncb;
};

__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (lane_id() == 0) red[wave_id()] = v;
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];
}

template <typename IO>
__global__ void __launch_bounds__(256) ssm_gate_kernel(GateParams gp) {
    const SsmParams &p = gp.s;
    __shared__ double red[4], wsum[4][5];
    const int head = blockIdx.x % p.H, item = blockIdx.x / p.H, tid = threadIdx.x;
    const Segment seg = find_segment<false>(p, item);
    if (!seg.live) {
        // a place that no segment has
        if (tid < 3) gp.grads[((int64_t)tid * p.n_items + item) * p.H + head] = 0.0;
        return;
    }
    const int cols = 64 * gp.ncb, per_hb = cols / p.P;          // heads of a block of columns (0: a part of one)
    const int nh = per_hb > 1 ? per_hb : 1;
    const int hb0 = head * p.P / cols, tiles = per_hb ? 1 : p.P / cols, hh = per_hb ? head % per_hb : 0;
    const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.f;
    double dA = 0.0, dD = 0.0, db = 0.0;
    double x = 0.0;                           // X at the end of the chunk at hand
    const int w = wave_id(), l = lane_id();
    for (int c0 = chunks_of(seg) - 1; c0 >= 0; c0 -= 4) {
        // wave w takes chunk c0 - w
        const int t = seg.begin + (c0 - w) * kSsmChunk + l;
        const bool on = c0 >= w && t < seg.end;
        float ri = 0.f, ra = 0.f, ci = 0.f, ca = 0.f, dd = 0.f, wtt = 0.f, raw = 0.f;
        if (on) {
            for (int k = 0; k < tiles; ++k) {
                const int64_t at = ((int64_t)(hb0 + k) * nh + hh) * p.rows + (int64_t)seg.batch * p.T + t;
                ri += p.inside[at];
                ra += p.across[at];
                ci += gp.c_inside[at];
                ca += gp.c_across[at];
                dd += p.dyx[at];
                wtt += p.wtt[at];
            }
            const int64_t at = seg.batch * p.db + t * p.dt_ + head;
            raw = (p.dt_f32 ? ((const float *)p.dt)[at] : io_traits<IO>::load((const IO *)p.dt + at)) + bias;
        }
        const float dt = on ? (p.softplus ? softplus(raw) : raw) : 0.f;
        const double dca = (double)dt * (double)ca, in = (double)ri - (double)dt * (double)ci;
        const double pre_in = wave_scan(in), pre_ca = wave_scan(dca), pre_ra = wave_scan((double)ra);
        const double all_in = last_lane(pre_in), all_ca = last_lane(pre_ca), all_ra = last_lane(pre_ra);
        // nothing of weight crosses a chunk whose decay is below fp32's step
        const bool cut = (float)last_lane(wave_scan(on ? (double)dt * (double)A : 0.0)) < -16.6f;
        __syncthreads();
        if (l == 0) {
            const int mark = c0 >= w ? mark_of(p, seg, c0 - w).x : -1;
            wsum[w][0] = all_ca;
            wsum[w][1] = all_ra;
            wsum[w][2] = cut ? 0.0 : 1.0;
            wsum[w][3] = mark >= 0 ? 1.0 : 0.0;
            double m = 0.0;
            for (int k = 0; mark >= 0 && k < tiles; ++k) m += p.X[((int64_t)mark * p.n_hb + hb0 + k) * nh + hh];
            wsum[w][4] = m;
        }
        __syncthreads();
        double Q = 0.0;
        for (int k = 0; k < 4; ++k) {
            if (wsum[k][3] != 0.0) x = wsum[k][4];
            const double qk = wsum[k][2] * (x - wsum[k][0]);
            if (k == w) Q = qk;
            x = qk + wsum[k][1];
        }
        if (on) {
            const int n = seg.end - (t - l) < kSsmChunk ? seg.end - (t - l) : kSsmChunk;
            // The pairs inside sum to zero over the chunk; what they sum to
            // instead is the roundings of the n rows' sums, taken back evenly
            // (d(dt_bias) of one seed's 2 x 8192 tokens 1.9e-6 -> 1.2e-6 off, dA 4.7e-7 -> 2.3e-7)
            const double pairs = all_in - pre_in + in - all_in * (double)(n - l) / (double)n;
            const double dg = pairs + (all_ra - pre_ra + (double)ra) + (pre_ca - dca) + Q;
            double g = (double)ci + (double)ca + (double)wtt + (double)A * dg;
            if (p.softplus) g /= 1.0 + (double)expf(-raw);
            const int64_t at = ((int64_t)seg.batch * p.T + t) * p.H + head;
            if (p.dt_f32)
                ((float *)gp.ddt)[at] = (float)g;
            else
                io_traits<IO>::store((IO *)gp.ddt + at, (float)g);
            dA += (double)dt * dg;
            db += g;
            dD += (double)dd;
        }
    }
    dA = block_sum(dA, red);
    db = block_sum(db, red);
    dD = block_sum(dD, red);
    if (tid == 0) {
        const int64_t plane = (int64_t)p.n_items * p.H;
        double *o = gp.grads + (int64_t)item * p.H + head;
        o[0] = dA;
        o[plane] = db;
        o[2 * plane] = dD;
    }
}

// dA, d(dt_bias) and dD of a head: the sums over the segments, a head a wave.
__global__ void __launch_bounds__(64) ssm_head_kernel(GateParams gp) {
    const SsmParams &p = gp.s;
    const int head = blockIdx.x;
    double a[3] = {0.0, 0.0, 0.0};
    for (int i0 = 0; i0 < p.n_items; i0 += 64) {
        const int i = i0 + lane_id();
        if (i < p.n_items)
            for (int k = 0; k < 3; ++k) a[k] += gp.grads[((int64_t)k * p.n_items + i) * p.H + head];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) a[k] += __shfl_xor(a[k], m, 64);
    if (lane_id() == 0) {
        gp.dA[head] = (float)a[0];
        if (gp.dbias) gp.dbias[head] = (float)a[1];
        if (gp.dD) gp.dD[head] = (float)a[2];
    }
}

namespace {

struct BwdPlan {
    SsmPlan s;
    int64_t slots, marks, xs, rows;
    size_t total, ends, ends_rev, sums[6], mark, X, part, grads, bytes;      // offsets
};

BwdPlan bwd_plan(const gdn_ssm_problem *pr, bool packed) {
    BwdPlan b;
    b.s = ssm_plan(pr, packed);
    b.rows = pr->B * pr->T;
    b.slots = packed ? pr->T / kSsmChunk + pr->n_seqs + 1 : pr->B * ((pr->T + kSsmChunk - 1) / kSsmChunk);
    const int64_t per = 4 * kSsmChunk;
    b.marks = packed ? pr->T / per : pr->T > 0 ? pr->B * ((pr->T - 1) / per) : 0;
    b.xs = packed ? pr->T / per + pr->n_seqs + 1 : pr->B * ((pr->T + per - 1) / per);
    const size_t blocks = (size_t)b.s.n_ends * b.s.n_hb;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 15) / 16 * 16;
        return was;
    };
    b.total = take(blocks * b.s.nh * 8);
    b.ends = take(blocks * pr->N * 64 * b.s.ncb * 4);
    b.ends_rev = take(blocks * pr->N * 64 * b.s.ncb * 4);
    for (size_t &o : b.sums) o = take((size_t)b.s.n_hb * b.s.nh * b.rows * 4);
    b.mark = take((size_t)b.marks * b.s.n_hb * pr->N * 64 * b.s.ncb * 4);
    b.X = take((size_t)b.xs * b.s.n_hb * b.s.nh * 8);
    b.part = take((size_t)b.slots * b.s.n_hb * kSsmChunk * pr->N * 4);
    b.grads = take((size_t)b.s.n_items * pr->H * 3 * 8);
    b.bytes = at;
    return b;
}

gdn_status check_ssm_backward(const gdn_ssm_problem *pr, bool packed) {
    const gdn_status st = check_ssm(pr, packed);
    if (st != GDN_OK) return st;
    // the sums' workgroups
    return grid_ok(bwd_plan(pr, packed).slots * pr->G, 4 * pr->N) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

template <typename IO, int N, int COLS, int NH>
struct BwdFns {
    static constexpr int kScanThreads = 4 * COLS, kKeyThreads = 4 * N;
    static const void *ends(bool rev) {
        return rev ? (const void *)&ssm_scan_kernel<IO, N, COLS, NH, true, true> : (const void *)&ssm_scan_kernel<IO, N, COLS, NH, true, false>;
    }
    static const void *dx() { return (const void *)&ssm_scan_kernel<IO, N, COLS, NH, false, true>; }
    static const void *key(bool rev) {
        return rev ? (const void *)&ssm_key_kernel<IO, N, COLS, NH, true> : (const void *)&ssm_key_kernel<IO, N, COLS, NH, false>;
    }
    static const void *sum(bool rev) {
        return rev ? (const void *)&ssm_sum_kernel<IO, N, true> : (const void *)&ssm_sum_kernel<IO, N, false>;
    }
};

template <typename F>
gdn_status bwd_launches(const gdn_ssm_problem *pr, const BwdPlan &b, const SsmParams &fwd, const SsmParams &rev, GateParams &gp,
                        void *dx, void *dB, void *dC, float *dh0, hipStream_t s) {
    SsmParams f = fwd, r = rev;
    gdn_status st = GDN_OK;
    auto go = [&](const void *fn, int g, SsmParams &sp, int threads) {
        if (st == GDN_OK) st = launch_kernel(fn, g, &sp, s, threads);
    };
    if (b.s.n_ends > 0) {
        // (the last segments' decays stand between dhT and the others)
        r.all_ends = dh0 != nullptr;
        f.all_ends = r.all_ends || r.s0;
        const int ends = ssm_grid(pr, f, b.s, true);
        ssm_grid(pr, r, b.s, true);
        go(F::ends(false), ends, f, F::kScanThreads);
        go(F::ends(true), ends, r, F::kScanThreads);
    }
    const int grid = ssm_grid(pr, f, b.s, false);
    ssm_grid(pr, r, b.s, false);
    SsmParams d = r;
    d.out = dx;
    d.sT = dh0;
    go(F::dx(), grid, d, F::kScanThreads);
    const int sgrid = (int)(b.slots * pr->G);
    f.out = dC;
    go(F::key(false), grid, f, F::kKeyThreads);
    go(F::sum(false), sgrid, f, F::kKeyThreads);
    r.out = dB;
    go(F::key(true), grid, r, F::kKeyThreads);
    go(F::sum(true), sgrid, r, F::kKeyThreads);
    if (st != GDN_OK) return st;
    gp.s = f;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_workspace_bytes_ssm_backward(const gdn_ssm_problem *pr) {
    const bool packed = pr && pr->n_seqs > 0;
    if (check_ssm_backward(pr, packed) != GDN_OK) return 0;
    return bwd_plan(pr, packed).bytes;
}

gdn_status gdn_ssm_backward(const gdn_ssm_problem *pr, const void *dy, const void *x, const void *dt, const float *A,
                            const void *Bm, const void *Cm, const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const float *dhT, void *dx, void *ddt, float *dA, void *dB,
                            void *dC, float *dD, float *ddt_bias, float *dh0, void *workspace, size_t workspace_bytes,
                            void *stream) {
    gdn_status st = check_ssm_backward(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (pr->T > 1 && (pr->dxbc_stride_t < pr->H * pr->P || pr->dxbc_stride_t < pr->G * pr->N)) return GDN_ERR_UNSUPPORTED;
    if (!A || !dA) return GDN_ERR_NULL_ARG;
    const int64_t eb = dtype_bytes(pr->io_dtype);
    if (pr->T > 0) {
        st = check_ssm_pointers(pr, x, dt, A, Bm, Cm, D, dt_bias, true);
        if (st != GDN_OK) return st;
        if (!dy || !dx || !ddt || !dB || !dC) return GDN_ERR_NULL_ARG;
        if (pr->dxbc_stride_b * eb % 16 || pr->dxbc_stride_t * eb % 16) return GDN_ERR_ALIGNMENT;
    }
    for (const void *q : {dy, (const void *)dx, (const void *)dB, (const void *)dC, (const void *)workspace})
        if (!aligned_to(q, 16)) return GDN_ERR_ALIGNMENT;
    for (const void *q : {(const void *)A, (const void *)D, (const void *)dt_bias, (const void *)h0, (const void *)dhT, (const void *)dA,
                          (const void *)dD, (const void *)ddt_bias, (const void *)dh0, (const void *)cu_seqlens})
        if (!aligned_to(q, 4)) return GDN_ERR_ALIGNMENT;
    if (!aligned_to(ddt, dtype_bytes(pr->dt_dtype))) return GDN_ERR_ALIGNMENT;
    const BwdPlan b = bwd_plan(pr, cu_seqlens != nullptr);
    if (!workspace || workspace_bytes < b.bytes) return GDN_ERR_WORKSPACE;
    char *ws = (char *)workspace;
    SsmParams f;
    fill_ssm(pr, f);
    f.dt = dt;
    f.A = A;
    f.D = D;
    f.bias = dt_bias;
    f.cu = cu_seqlens;
    f.total = (double *)(ws + b.total);
    f.part = (float *)(ws + b.part);
    f.n_slots = (int)b.slots;
    f.marks = (float *)(ws + b.mark);
    f.X = (double *)(ws + b.X);
    f.n_marks = (int)b.marks;
    f.n_x = (int)b.xs;
    f.rows = b.rows;
    f.ob = pr->dxbc_stride_b;
    f.ot = pr->dxbc_stride_t;
    SsmParams r = f;
    const int64_t yt = pr->H * pr->P, yb = yt * pr->T;
    f.q = Cm;
    f.k = Bm;
    f.v = x;
    f.vb = pr->x_stride_b;
    f.vt = pr->x_stride_t;
    f.q2 = dy;
    f.q2b = yb;
    f.q2t = yt;
    f.s0 = h0;
    f.dT = dhT;
    f.ends = (float *)(ws + b.ends);
    f.inside = (float *)(ws + b.sums[0]);
    f.across = (float *)(ws + b.sums[1]);
    f.dyx = (float *)(ws + b.sums[2]);
    f.wtt = (float *)(ws + b.sums[3]);
    r.q = Bm;
    r.k = Cm;
    r.v = dy;
    r.vb = yb;
    r.vt = yt;
    r.q2 = x;
    r.q2b = pr->x_stride_b;
    r.q2t = pr->x_stride_t;
    r.s0 = dhT;
    r.ends = (float *)(ws + b.ends_rev);
    r.inside = (float *)(ws + b.sums[4]);
    r.across = (float *)(ws + b.sums[5]);
    GateParams gp{};
    gp.c_inside = r.inside;
    gp.c_across = r.across;
    gp.ddt = ddt;
    gp.grads = (double *)(ws + b.grads);
    gp.dA = dA;
    gp.dD = dD;
    gp.dbias = ddt_bias;
    gp.ncb = b.s.ncb;
    hipStream_t s = (hipStream_t)stream;
    auto run = [&](auto n64, auto n128) {
        return pr->N == 64 ? bwd_launches<decltype(n64)>(pr, b, f, r, gp, dx, dB, dC, dh0, s)
                           : bwd_launches<decltype(n128)>(pr, b, f, r, gp, dx, dB, dC, dh0, s);
    };
    if (pr->io_dtype == GDN_F32)
        st = run(BwdFns<float, 64, 64, 1>(), BwdFns<float, 128, 64, 1>());
    else if (b.s.ncb == 1)
        st = run(BwdFns<bf16_t, 64, 64, 1>(), BwdFns<bf16_t, 128, 64, 1>());
    else if (b.s.nh == 2)
        st = run(BwdFns<bf16_t, 64, 128, 2>(), BwdFns<bf16_t, 128, 128, 2>());
    else
        st = run(BwdFns<bf16_t, 64, 128, 1>(), BwdFns<bf16_t, 128, 128, 1>());
    if (st != GDN_OK) return st;
    const void *fn = pr->io_dtype == GDN_F32 ? (const void *)&ssm_gate_kernel<float> : (const void *)&ssm_gate_kernel<bf16_t>;
    st = launch_kernel(fn, b.s.n_items * (int)pr->H, &gp, s);
    if (st != GDN_OK) return st;
    return launch_kernel((const void *)&ssm_head_kernel, (int)pr->H, &gp, s, 64);
}

}  // extern "C"

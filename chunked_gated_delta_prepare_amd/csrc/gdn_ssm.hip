// Selective state space scan, forward (see gdn_ssm.h for the mathematics).
//
// A workgroup of four waves walks one segment of one stream, a stream being
// 64 NCB columns of the state: one head's, or with P = 64 and NCB = 2 two
// heads' of a group, which then share B, C and the products C . B.  Each wave
// keeps its columns' state in accumulators (N rows, 16 NCB columns) and uses
// them as operands without a trip through LDS.  Per chunk:
//   1  the lower triangle of C B^T, times decays and dt, to LDS (16 x 16
//      blocks, dealt to the waves); C h on the way
//   2  y = M x + e^cum C h, transposed, so that a lane stores four columns
//   3  h' = e^cum h + B^T (w x)
// The state's products take w x in two bf16 parts (relative error 2^-18): the
// final state is fp32 and read on by every later chunk.  y's operands are
// rounded once to bf16, the type of y.
// The next chunk's rows are in flight while one is worked on.
#include "gdn_ssm.h"

namespace gdn {

// State segments' accumulators in the workspace: two planes of float2 per
// 16 x 16 block, so that a lane's stores are 8 bytes and a wave's are whole
// lines.
template <int NB>
__device__ __forceinline__ void put_state(float *ws, const float4v (&h)[NB]) {
    float2 *p = (float2 *)ws + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        p[(2 * i) * 256] = make_float2(h[i][0], h[i][1]);
        p[(2 * i + 1) * 256] = make_float2(h[i][2], h[i][3]);
    }
}
template <int NB>
__device__ __forceinline__ void add_state(const float *ws, float f, float4v (&h)[NB]) {
    const float2 *p = (const float2 *)ws + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const float2 a = p[(2 * i) * 256], b = p[(2 * i + 1) * 256];
        h[i][0] += f * a.x;
        h[i][1] += f * a.y;
        h[i][2] += f * b.x;
        h[i][3] += f * b.y;
    }
}

// ENDS: only the end state from a zero start, to the workspace.
template <typename IO, int N, int NCB, bool ENDS>
__global__ void __launch_bounds__(256) ssm_forward_kernel(SsmParams p) {
    typedef SOp<IO> O;
    typedef typename O::elem E;
    constexpr int C = kSsmChunk, COLS = 64 * NCB, LX = COLS + O::kPad, LN = N + O::kPad, LM = C + O::kPad;
    constexpr int NH = NCB, NB = N / 16;          // heads at most; row blocks of the state
    __shared__ E sx[C * LX], sb[C * LN], sc[ENDS ? 1 : C * LN], sm[ENDS ? 1 : NH][ENDS ? 1 : C * LM];
    __shared__ Gates gates[NH];
    int item, hb;
    place(p, item, hb);
    if (item >= p.n_items) return;
    const Segment seg = find_segment(p, item);
    if (!seg.live || (ENDS && seg.end == seg.seq_end)) return;
    const int w = wave_id(), l = lane_id(), q = l >> 4, j = l & 15;
    const int col0 = hb * COLS, head0 = col0 / p.P, nh = p.P == 64 ? NCB : 1;
    const int mine = nh == 2 ? w >> 1 : 0, head = head0 + mine, grp = head0 / p.heads_per_group;
    const int wc = w * 16 * NCB;                  // this wave's first column
    const bool gater = w < nh;                    // waves that form the gates of head0 + w
    const float A = gater ? p.A[head0 + w] : 0.f, bias = gater && p.bias ? p.bias[head0 + w] : 0.f;
    const float Dh = p.D ? p.D[head] : 0.f;
    constexpr int kState = N * COLS;
    const int64_t ws_doubles = (int64_t)p.n_items * p.n_hb;     // totals, before the states
    double *ws_total = (double *)p.ws;
    float *ws_state = p.ws + ws_doubles * 2 * NH;

    float4v h[NCB * NB];
#pragma unroll
    for (int i = 0; i < NCB * NB; ++i) h[i] = float4v{0.f, 0.f, 0.f, 0.f};
    // h[cb * NB + nb][e] = state[n = 16 nb + 4 q + e][column wc + 16 cb + j]
    const int64_t hoff = ((int64_t)seg.seq * p.H * N) * p.P;
    auto hidx = [&](int cb, int nb, int e) {
        const int col = col0 + wc + 16 * cb + j;
        return hoff + ((int64_t)(col / p.P) * N + 16 * nb + 4 * q + e) * p.P + col % p.P;
    };
    if constexpr (!ENDS) {
        double f = 0.0;                           // log2 of the decay since segment i's end
        for (int i = item - 1; i >= seg.first; --i) {
            const int64_t at = (int64_t)i * p.n_hb + hb;
            add_state<NCB * NB>(ws_state + at * kState, fast_exp2((float)f), h);
            f += ws_total[at * NH + mine];
        }
        if (p.h0) {
            const float d = fast_exp2((float)f);
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[cb * NB + nb][e] += d * p.h0[hidx(cb, nb, e)];
        }
        // the blocks of M right of the diagonal that a 32-wide step touches
        for (int i = threadIdx.x; i < NH * 2 * 16 * 16; i += 256) {
            const int hh = i >> 9, blk = (i >> 8) & 1, r = (i >> 4) & 15, c = i & 15;
            sm[hh][(32 * blk + r) * LM + 32 * blk + 16 + c] = E(0);
        }
    }

    TileRegs<IO, C, COLS> tx;
    TileRegs<IO, C, N> tb, tc;
    float raw = 0.f;
    const int64_t xoff = seg.batch * p.xb + col0, boff = seg.batch * p.bb + (int64_t)grp * N;
    auto fetch = [&](int t) {
        const int rows = seg.end - t;
        tx.load(p.x, xoff + t * p.xt, (uint32_t)p.xt, rows);
        tb.load(p.Bm, boff + t * p.bt, (uint32_t)p.bt, rows);
        if constexpr (!ENDS) tc.load(p.Cm, boff + t * p.bt, (uint32_t)p.bt, rows);
        if (gater && l < rows) {
            const int64_t at = seg.batch * p.db + (t + l) * p.dt_ + head0 + w;
            raw = p.dt_f32 ? ((const float *)p.dt)[at] : io_traits<IO>::load((const IO *)p.dt + at);
        }
    };
    double total = 0.0;
    if (seg.begin < seg.end) fetch(seg.begin);
    for (int t = seg.begin; t < seg.end; t += C) {
        const int rows = seg.end - t < C ? seg.end - t : C;
        __syncthreads();                          // the last chunk's tiles are done with
        tx.put(sx, LX);
        tb.put(sb, LN);
        if constexpr (!ENDS) tc.put(sc, LN);
        if (gater) make_gates(gates[w], dt_of(p, raw, bias, l < rows), A);
        if (t + C < seg.end) fetch(t + C);
        __syncthreads();
        const Gates &g = gates[mine];
        float4v y[ENDS ? 1 : NCB * 4];
        if constexpr (!ENDS) {
            // 1: M[t][s] = (C_t . B_s) e^(cum_t - cum_s) dt_s, s <= t
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int idx = w + 4 * k;
                if (idx < 10) {
                    const int bt = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, bs = idx - bt * (bt + 1) / 2;
                    float4v s = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += 32)
                        O::mma(s, O::row(sb, LN, 16 * bs, n0), O::row(sc, LN, 16 * bt, n0));
                    const int tt = 16 * bt + j;
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh)
                        if (hh < nh) {
                            float4v m;
                            const float2 ct = gates[hh].cum[tt];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int ss = 16 * bs + 4 * q + e;
                                m[e] = ss <= tt ? s[e] * decay_between(ct, gates[hh].cum[ss]) * gates[hh].dt[ss] : 0.f;
                            }
                            O::put4(&sm[hh][tt * LM + 16 * bs + 4 * q], m);
                        }
                }
            }
            // y^T = h^T C^T, then times e^cum
#pragma unroll
            for (int i = 0; i < NCB * 4; ++i) y[i] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 32) {
                typename O::frag hf[NCB];
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) hf[cb] = O::acc_split(h[cb * NB + n0 / 16], h[cb * NB + n0 / 16 + 1]);
#pragma unroll
                for (int bt = 0; bt < 4; ++bt) {
                    const typename O::frag cf = O::row_split(sc, LN, 16 * bt, n0);
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) O::mma(y[cb * 4 + bt], hf[cb], cf);
                }
            }
#pragma unroll
            for (int bt = 0; bt < 4; ++bt) {
                const float ec = g.ecum[16 * bt + j];
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) y[cb * 4 + bt] *= ec;
            }
            __syncthreads();                      // M is whole
        }
        // 3 (and 2): both take x by columns
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
            typename O::frag xf[NCB], xh[NCB], xl[NCB];
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                xf[cb] = O::col(sx, LX, wc + 16 * cb, s0);
                O::scaled(xf[cb], wt, xh[cb], xl[cb]);
            }
            if constexpr (!ENDS) {
#pragma unroll
                for (int bt = s0 / 16; bt < 4; ++bt) {
                    const typename O::frag mf = O::row(sm[mine], LM, 16 * bt, s0);
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) O::mma(y[cb * 4 + bt], xf[cb], mf);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const typename O::frag bf = O::col(sb, LN, 16 * nb, s0);
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) {
                    O::mma(h[cb * NB + nb], bf, xh[cb]);
                    if constexpr (O::kSplit) O::mma(h[cb * NB + nb], bf, xl[cb]);
                }
            }
        }
        if constexpr (!ENDS) {
            const rsrc_t ry = make_rsrc((IO *)p.y + ((int64_t)seg.batch * p.T + t) * p.H * p.P + col0, 0x7fffffffu);
#pragma unroll
            for (int bt = 0; bt < 4; ++bt) {
                const int tt = 16 * bt + j;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) {
                    const int c = wc + 16 * cb + 4 * q;
                    float x[4];
                    O::get4(&sx[tt * LX + c], x);
                    float o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = y[cb * 4 + bt][e] + Dh * x[e];
                    const uint32_t off = tt < rows ? (uint32_t)(tt * p.H * p.P + c) * (uint32_t)sizeof(IO) : 0xfffffff0u;
                    if constexpr (sizeof(IO) == 2) {
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])}, ry, off, 0, 0);
                    } else {
                        // (two stores of 8 bytes that the compiler does not
                        // join: the first halves of all blocks come first)
                        y[cb * 4 + bt] = float4v{o[0], o[1], o[2], o[3]};
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(o[0]), __float_as_uint(o[1])}, ry, off, 0, 0);
                    }
                }
            }
            if constexpr (sizeof(IO) == 4) {
                asm volatile("" ::: "memory");
#pragma unroll
                for (int bt = 0; bt < 4; ++bt) {
                    const int tt = 16 * bt + j;
#pragma unroll
                    for (int cb = 0; cb < NCB; ++cb) {
                        const uint32_t off = tt < rows ? (uint32_t)(tt * p.H * p.P + wc + 16 * cb + 4 * q) * 4u + 8u : 0xfffffff0u;
                        const float4v o = y[cb * 4 + bt];
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(o[2]), __float_as_uint(o[3])}, ry, off, 0, 0);
                    }
                }
            }
        }
    }
    if constexpr (ENDS) {
        const int64_t at = (int64_t)item * p.n_hb + hb;
        put_state<NCB * NB>(ws_state + at * kState, h);
        if (l == 0 && (nh == 1 ? w == 0 : (w & 1) == 0)) ws_total[at * NH + mine] = total;
    } else if (p.hT && seg.end == seg.seq_end) {
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) p.hT[hidx(cb, nb, e)] = h[cb * NB + nb][e];
    }
}

// One token: h' = e^(dt A) h + dt B x^T, y = h'^T C + D x.  A workgroup moves
// one head's state on, once through registers; its rows of P columns are dealt
// to the waves, a lane two columns.  Bound by reading and writing the state.
template <typename IO, int P, int N>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmParams p) {
    constexpr int kLanes = P / 2, kRows = 64 / kLanes, kIter = N / 4 / kRows;
    __shared__ float2 red[4][64];
    const int head = blockIdx.x % p.H, b = blockIdx.x / p.H, w = wave_id(), l = lane_id();
    const int64_t s = p.slots ? p.slots[b] : b;
    bool ok = s >= 0 && s < p.n_slots;
    if (ok && p.slots) {
        // a row behind another one with its slot is padding
        bool seen = false;
        for (int i = 0; i < b; i += 64) {
            const int k = i + l;
            seen |= k < b && p.slots[k] == (int)s;
        }
        ok = __ballot(seen) == 0;
    }
    const int c = l % kLanes * 2, n0 = w * (N / 4) + l / kLanes;
    IO *y = (IO *)p.y + ((int64_t)b * p.H + head) * P;
    if (!ok) {
        if (threadIdx.x < P) io_traits<IO>::store(y + threadIdx.x, 0.f);
        return;
    }
    float2 *h = (float2 *)(p.state + ((s * p.H + head) * N + n0) * P + c);
    float2 v[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) v[i] = h[i * kRows * P / 2];
    const int grp = head / p.heads_per_group;
    const int64_t dat = b * p.db + head;
    const float raw = p.dt_f32 ? ((const float *)p.dt)[dat] : io_traits<IO>::load((const IO *)p.dt + dat);
    const float dt = dt_of(p, raw, p.bias ? p.bias[head] : 0.f, true);
    const float a = fast_exp2(dt * p.A[head] * kLog2e);
    const IO *xp = (const IO *)p.x + b * p.xb + head * P + c;
    const float x0 = io_traits<IO>::load(xp), x1 = io_traits<IO>::load(xp + 1);
    const IO *bp = (const IO *)p.Bm + b * p.bb + grp * N + n0, *cp = (const IO *)p.Cm + b * p.bb + grp * N + n0;
    const float u0 = dt * x0, u1 = dt * x1;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const float bn = io_traits<IO>::load(bp + i * kRows), cn = io_traits<IO>::load(cp + i * kRows);
        v[i].x = a * v[i].x + bn * u0;
        v[i].y = a * v[i].y + bn * u1;
        o.x += cn * v[i].x;
        o.y += cn * v[i].y;
        h[i * kRows * P / 2] = v[i];
    }
    red[w][l] = o;
    __syncthreads();
    if (threadIdx.x >= kLanes) return;
    o = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            o.x += red[i][l + k * kLanes].x;
            o.y += red[i][l + k * kLanes].y;
        }
    const float D = p.D ? p.D[head] : 0.f;
    io_traits<IO>::store(y + c, o.x + D * x0);
    io_traits<IO>::store(y + c + 1, o.y + D * x1);
}

namespace {

struct SsmPlan {
    int ncb, n_hb, n_items, seg_tokens, seqs;
};

// Two blocks of 16 columns a wave where the columns of a head, or of two
// heads of one group, fill them: every fragment of B, C and M then feeds two
// products.  fp32 io has one (its tiles fill LDS).
int columns(const gdn_ssm_problem *pr) {
    if (pr->io_dtype == GDN_F32) return 1;
    return pr->P == 128 || (pr->H / pr->G) % 2 == 0 ? 2 : 1;
}

SsmPlan plan(const gdn_ssm_problem *pr, bool packed) {
    SsmPlan s;
    s.ncb = columns(pr);
    s.n_hb = (int)(pr->H * pr->P / (64 * s.ncb));
    s.seqs = (int)(packed ? pr->n_seqs : pr->B);
    const int64_t chunks = (pr->T + kSsmChunk - 1) / kSsmChunk;
    // segments for about 512 workgroups, of four chunks at least
    const int64_t streams = (int64_t)s.n_hb * (packed ? 1 : pr->B);
    int64_t per = (512 + streams - 1) / streams;
    int64_t seg = (chunks + per - 1) / per;
    seg = seg < 4 ? 4 : seg;
    s.seg_tokens = (int)(seg * kSsmChunk);
    const int64_t cut = (pr->T + s.seg_tokens - 1) / s.seg_tokens;
    s.n_items = (int)(packed ? cut + pr->n_seqs : pr->B * (cut > 0 ? cut : 1));
    return s;
}

size_t ws_bytes(const gdn_ssm_problem *pr, const SsmPlan &s) {
    if (s.n_items == s.seqs) return 0;            // one segment each
    return (size_t)s.n_items * s.n_hb * (8 * s.ncb + 4 * pr->N * 64 * s.ncb);
}

}  // namespace

gdn_status check_ssm(const gdn_ssm_problem *pr, bool packed) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->B < 1 || pr->T < 0 || pr->H < 1 || pr->P < 1 || pr->N < 1 || pr->G < 1 || pr->H % pr->G != 0)
        return GDN_ERR_BAD_SHAPE;
    if (packed && (pr->B != 1 || pr->n_seqs < 1 || pr->n_seqs > (1 << 24))) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->io_dtype) || (pr->dt_dtype != pr->io_dtype && pr->dt_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if ((pr->P != 64 && pr->P != 128) || (pr->N != 64 && pr->N != 128)) return GDN_ERR_UNSUPPORTED;
    // a chunk's rows are addressed with 32-bit byte offsets, workgroups are
    // numbered in 31 bits
    if (pr->T > (1 << 30) || pr->B > (1 << 20) || pr->H > (1 << 14)) return GDN_ERR_UNSUPPORTED;
    for (int64_t v : {pr->x_stride_t, pr->bc_stride_t, pr->dt_stride_t, pr->dxbc_stride_t})
        if (v < 0 || v > (1 << 22)) return GDN_ERR_UNSUPPORTED;
    const int64_t items = (packed ? pr->n_seqs : pr->B) + (pr->T + 255) / 256 * pr->B;
    if (items * pr->H * 2 > ((int64_t)1 << 30)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_ssm_pointers(const gdn_ssm_problem *pr, const void *x, const void *dt, const float *A, const void *Bm,
                              const void *Cm, const float *D, const float *bias, bool rows) {
    if (!x || !dt || !A || !Bm || !Cm) return GDN_ERR_NULL_ARG;
    const size_t eb = dtype_bytes(pr->io_dtype);
    if (!aligned_to(x, 16) || !aligned_to(Bm, 16) || !aligned_to(Cm, 16) || !aligned_to(dt, dtype_bytes(pr->dt_dtype)) ||
        !aligned_to(A, 4) || !aligned_to(D, 4) || !aligned_to(bias, 4))
        return GDN_ERR_ALIGNMENT;
    for (int64_t v : {pr->x_stride_b, pr->bc_stride_b})
        if (v * (int64_t)eb % 16) return GDN_ERR_ALIGNMENT;
    if (rows)
        for (int64_t v : {pr->x_stride_t, pr->bc_stride_t})
            if (v * (int64_t)eb % 16) return GDN_ERR_ALIGNMENT;
    return GDN_OK;
}

void fill_ssm(const gdn_ssm_problem *pr, SsmParams &sp) {
    sp = SsmParams{};
    sp.xb = pr->x_stride_b;
    sp.xt = pr->x_stride_t;
    sp.bb = pr->bc_stride_b;
    sp.bt = pr->bc_stride_t;
    sp.db = pr->dt_stride_b;
    sp.dt_ = pr->dt_stride_t;
    sp.gb = pr->dxbc_stride_b;
    sp.gt = pr->dxbc_stride_t;
    sp.T = (int)pr->T;
    sp.H = (int)pr->H;
    sp.P = (int)pr->P;
    sp.N = (int)pr->N;
    sp.G = (int)pr->G;
    sp.heads_per_group = (int)(pr->H / pr->G);
    sp.softplus = pr->softplus != 0;
    sp.dt_f32 = pr->dt_dtype == GDN_F32;
}

namespace {

template <typename IO, int NCB>
const void *ssm_fn(int N, bool ends) {
    if (N == 64) return ends ? (const void *)&ssm_forward_kernel<IO, 64, NCB, true> : (const void *)&ssm_forward_kernel<IO, 64, NCB, false>;
    return ends ? (const void *)&ssm_forward_kernel<IO, 128, NCB, true> : (const void *)&ssm_forward_kernel<IO, 128, NCB, false>;
}

const void *ssm_pick(const gdn_ssm_problem *pr, int ncb, bool ends) {
    const int N = (int)pr->N;
    if (pr->io_dtype == GDN_F32) return ssm_fn<float, 1>(N, ends);
    return ncb == 2 ? ssm_fn<bf16_t, 2>(N, ends) : ssm_fn<bf16_t, 1>(N, ends);
}

template <typename IO>
const void *step_fn(int64_t P, int64_t N) {
    if (P == 64) return N == 64 ? (const void *)&ssm_step_kernel<IO, 64, 64> : (const void *)&ssm_step_kernel<IO, 64, 128>;
    return N == 64 ? (const void *)&ssm_step_kernel<IO, 128, 64> : (const void *)&ssm_step_kernel<IO, 128, 128>;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_workspace_bytes_ssm(const gdn_ssm_problem *pr) {
    const bool packed = pr && pr->n_seqs > 0;
    if (check_ssm(pr, packed) != GDN_OK) return 0;
    return ws_bytes(pr, plan(pr, packed));
}

gdn_status gdn_ssm_forward(const gdn_ssm_problem *pr, const void *x, const void *dt, const float *A, const void *Bm,
                           const void *Cm, const float *D, const float *dt_bias, const float *h0,
                           const int32_t *cu_seqlens, void *y, float *hT, void *workspace, size_t workspace_bytes,
                           void *stream) {
    gdn_status st = check_ssm(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (pr->T > 0) {
        st = check_ssm_pointers(pr, x, dt, A, Bm, Cm, D, dt_bias, true);
        if (st != GDN_OK) return st;
        if (!y) return GDN_ERR_NULL_ARG;
    }
    if (!aligned_to(y, 16) || !aligned_to(h0, 4) || !aligned_to(hT, 4) || !aligned_to(cu_seqlens, 4)) return GDN_ERR_ALIGNMENT;
    if (pr->T == 0 && !hT) return GDN_OK;
    const SsmPlan s = plan(pr, cu_seqlens != nullptr);
    const size_t need = ws_bytes(pr, s);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    SsmParams sp;
    fill_ssm(pr, sp);
    sp.x = x;
    sp.dt = dt;
    sp.A = A;
    sp.Bm = Bm;
    sp.Cm = Cm;
    sp.D = D;
    sp.bias = dt_bias;
    sp.h0 = h0;
    sp.cu = cu_seqlens;
    sp.y = y;
    sp.hT = hT;
    sp.ws = (float *)workspace;
    sp.seg_tokens = s.seg_tokens;
    sp.n_items = s.n_items;
    sp.n_hb = s.n_hb;
    sp.n_seqs = s.seqs;
    sp.swizzle = s.n_items >= 16;
    const int grid = (sp.swizzle ? (s.n_items + 7) / 8 * 8 : s.n_items) * s.n_hb;
    if (need) {
        st = launch_kernel(ssm_pick(pr, s.ncb, true), grid, &sp, (hipStream_t)stream);
        if (st != GDN_OK) return st;
    }
    return launch_kernel(ssm_pick(pr, s.ncb, false), grid, &sp, (hipStream_t)stream);
}

gdn_status gdn_ssm_step(const gdn_ssm_problem *pr, const void *x, const void *dt, const float *A, const void *Bm,
                        const void *Cm, const float *D, const float *dt_bias, float *state, const int32_t *slots,
                        int64_t n_slots, void *y, void *stream) {
    gdn_status st = check_ssm(pr, false);
    if (st != GDN_OK) return st;
    if (pr->T != 1 || n_slots < 0 || n_slots >= ((int64_t)1 << 31) || (!slots && n_slots < pr->B)) return GDN_ERR_BAD_SHAPE;
    st = check_ssm_pointers(pr, x, dt, A, Bm, Cm, D, dt_bias, false);
    if (st != GDN_OK) return st;
    if (!y || (!state && n_slots > 0)) return GDN_ERR_NULL_ARG;
    if (!aligned_to(state, 16) || !aligned_to(slots, 4) || !aligned_to(y, 16)) return GDN_ERR_ALIGNMENT;
    SsmParams sp;
    fill_ssm(pr, sp);
    sp.x = x;
    sp.dt = dt;
    sp.A = A;
    sp.Bm = Bm;
    sp.Cm = Cm;
    sp.D = D;
    sp.bias = dt_bias;
    sp.state = state;
    sp.slots = slots;
    sp.n_slots = n_slots;
    sp.y = y;
    const void *fn = pr->io_dtype == GDN_F32 ? step_fn<float>(pr->P, pr->N) : step_fn<bf16_t>(pr->P, pr->N);
    return launch_kernel(fn, (int)(pr->B * pr->H), &sp, (hipStream_t)stream);
}

}  // extern "C"

// Gated linear recurrence, forward and step (see gdn_glr.h for the mathematics).
//
// Bound by memory where channels and sequences fill the chip (8 sequences of 8192
// tokens, 4096 channels of bf16: 343 us, 4.7 TB/s, near a copy's rate); a single long
// sequence is cut into segments and its rows are read once more for their moves
// (65536 tokens: 167 us, 4.8 TB/s, then 325, 5.0 TB/s).  Vector instructions come next: with the
// gate's exponential, reciprocal, series and square root some 24 an element (rate, norm) or
// 20 (sigmoid, complement), which keep the units busy for half of the time (long moves,
// two workgroups a CU: 0.74).  16384 packed tokens of 4096 channels, rate and norm, are short of
// waves, with one workgroup a CU (165 to 191 registers): 64 us the moves (3.1 TB/s), 94 us y (4.3 TB/s),
// vector instructions for half of either.  Prompts of some thousand tokens fill few CUs: 2048 of
// 1024 channels 7 us the moves and 20 us y, of 32 workgroups.  Eight waves of 16
// tokens a thread and one workgroup a CU for y (before the moves had pieces: four waves and 512
// workgroups 556 against 536 us for 65536 tokens, 8 tokens a thread 580, 16 waves 619).
#include <algorithm>

#include "gdn_glr.h"

namespace gdn {

constexpr int kGlrWaves = 8;
constexpr int kGlrRun = 16;            // tokens of a thread at a time
constexpr int kGlrAhead = 4;           // moves that a workgroup of the forward pass reads at a time

template <int VEC, int NW = kGlrWaves>
constexpr int kGlrTile = NW * GlrLane<VEC>::kTG * kGlrRun;      // tokens of a workgroup at a time

// y and the final states: a workgroup walks one segment of 64 channels, tile by
// tile; the state at a segment's start comes from the segments' moves in the
// workspace.  One read of x and the gate and one write of y; the next tile's
// rows are in flight while one is worked on.  NW waves: eight, or four or one for
// many short sequences.
template <typename IO, typename GT, int VEC, bool PK, int FORM, int NW>
__global__ void __launch_bounds__(64 * NW, 2) glr_forward_kernel(GlrParams p) {
    constexpr int L = kGlrRun, kTile = kGlrTile<VEC, NW>;
    __shared__ float lds_q[2][NW][kGlrCols], lds_h[2][NW][kGlrCols];
    const int group = blockIdx.x % p.groups, rest = blockIdx.x / p.groups, seg = rest % p.segs, b = rest / p.segs;
    const GlrLane<VEC> ln(group);
    const int w = wave_id(), row = (w * ln.kTG + ln.tg) * L;
    const int t_begin = seg * p.seg_len, t_end = t_begin + p.seg_len < p.T ? t_begin + p.seg_len : p.T;
    RunRows<IO, GT, VEC, L> rows;
    if (t_begin < t_end) rows.fetch(p, b, t_begin, row, ln.c, t_begin + kTile <= p.T);
    // (states and moves between runs are of one channel a lane)
    const int l = lane_id(), c1 = group * kGlrCols + ln.one();
    GateBias bias[VEC];
    float rate[VEC];
    load_bias<FORM, VEC>(p.bias, ln.c, p.D, bias);
    channel_load<VEC>(p.rate, ln.c, p.D, rate);
    const bool near = near_rates<FORM, VEC>(rate);
    // (packed rows take initial states at their sequences' first tokens)
    float h = state_at(p, PK ? nullptr : p.h0, b, c1);
    // the moves of what lies in front, whose loads go out kGlrAhead at a time
    const int moves = seg * p.pieces;
    const float *ws = p.ws + (int64_t)b * (p.segs - 1) * p.pieces * 2 * p.D;
    for (int j0 = 0; j0 < moves; j0 += kGlrAhead) {
        float q[kGlrAhead][1], H[kGlrAhead][1];
#pragma unroll
        for (int j = 0; j < kGlrAhead; ++j) {
            const float *s = ws + (int64_t)(j0 + j < moves ? j0 + j : j0) * 2 * p.D;
            channel_load<1>(s, c1, p.D, q[j]);
            channel_load<1>(s + p.D, c1, p.D, H[j]);
        }
#pragma unroll
        for (int j = 0; j < kGlrAhead; ++j)
            if (j0 + j < moves) h = packed_move<PK>(q[j][0], h, H[j][0]);
    }
    if (seg == 0) pass_empty(p, PK, b, group * kGlrCols, p.h0, p.hT);
    Span span;
    int turn = 0;
    for (int t = t_begin; t < t_end; t += kTile, turn ^= 1) {
        const int t0 = t + row;
        const Marks marks = marks_of<PK, L>(p, t + w * ln.kTG * L, ln.kTG * L, t0, span);
        const bool odd = PK && __ballot(marks.first != 0) != 0;
        float a[L][VEC], u[L][VEC], H[VEC];
        Moves<VEC> m;
        m.none();
#pragma unroll
        for (int e = 0; e < VEC; ++e) H[e] = 0.f;
        with_scale<FORM>(p.scale, near, [&](auto sc, auto nr) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                float xv[VEC], gv[VEC];
                rows.x[i].get(xv);
                rows.g[i].get(gv);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float c, slope, sig;
                    gate_of<FORM, nr.value>(gv[e], bias[e], rate[e], a[i][e], c, slope, sig);
                    u[i][e] = xv[e] * input_scale<sc.value>(a[i][e], c);
                    move_on<false>(false, 0.f, a[i][e], c, u[i][e], H[e], m.P[e], m.C[e]);
                }
            }
        });
        if (t + kTile < t_end) rows.fetch(p, b, t + kTile, row, ln.c, t + 2 * kTile <= p.T);
        if (odd) {
            // u of a first token holds its sequence's initial state
            float n[VEC];
            Span q = marks.start;
#pragma unroll
            for (int e = 0; e < VEC; ++e) n[e] = 0.f;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool f = marks.first >> i & 1;
                if (f) {
                    float h0[VEC];
                    q.at(p, t0 + i);
                    state_load<VEC>(p, p.h0, q.n, ln.c, h0);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) u[i][e] = fmaf(a[i][e], h0[e], u[i][e]);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) n[e] = f ? u[i][e] : fmaf(a[i][e], n[e], u[i][e]);
            }
            if (marks.first) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    H[e] = n[e];
                    m.P[e] = -1.f;
                }
            }
        }
        const WaveRun run = join_wave<PK, VEC, false>(m, H, H);
        lds_q[turn][w][l] = pack_move<PK>(run.P, run.C);
        lds_h[turn][w][l] = run.H;
        // (one barrier a tile: the other half of LDS is next, and its readers are behind the next barrier)
        lds_barrier();
        float front, mine[VEC];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            if (j == w) front = h;
            h = packed_move<PK>(lds_q[turn][j][l], h, lds_h[turn][j][l]);
        }
        spread_state<PK, VEC>(run, front, mine);
        const TileRows<IO, VEC> ry(p.y, ((int64_t)b * p.T + t) * p.D, p.D, row, ln.c, p.D);
        if (!odd && __ballot(marks.valid != (1u << L) - 1 || marks.last != 0) == 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) mine[e] = fmaf(a[i][e], mine[e], u[i][e]);
                ry.store(mine, i, true);
            }
        } else {
            Span q = marks.start;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool f = PK && (marks.first >> i & 1);
#pragma unroll
                for (int e = 0; e < VEC; ++e) mine[e] = f ? u[i][e] : fmaf(a[i][e], mine[e], u[i][e]);
                ry.store(mine, i, marks.valid >> i & 1);
                if (p.hT && (marks.last >> i & 1)) {
                    if (PK) q.at(p, t0 + i);
                    state_store<VEC>(p, p.hT, PK ? q.n : b, ln.c, true, mine);
                }
            }
        }
    }
}

// The moves of all segments but the last, each in pieces of its tiles so that there
// are workgroups for the whole chip.  A wave walks its share of a piece backwards,
// and a segment's first pieces come last, so that what is read last is what the
// next launch reads first.
template <typename IO, typename GT, int VEC, bool PK, int FORM>
__global__ void __launch_bounds__(64 * kGlrWaves, 2) glr_moves_kernel(GlrParams p) {
    constexpr int L = kGlrRun, NW = kGlrWaves, kStep = GlrLane<VEC>::kTG * L;
    __shared__ float lds_p[NW][kGlrCols], lds_c[NW][kGlrCols], lds_h[NW][kGlrCols];
    const int segs = p.segs - 1, K = p.pieces, tiles = p.seg_len / kGlrTile<2>;
    const int group = blockIdx.x % p.groups, rest = blockIdx.x / p.groups, seg = rest % segs, b = rest / segs % p.B;
    const int piece = K - 1 - rest / segs / p.B, tile = piece * tiles / K, share = ((piece + 1) * tiles / K - tile) * (kGlrTile<2> / NW);
    const GlrLane<VEC> ln(group);
    const int w = wave_id(), row = ln.tg * L;
    const int t_first = seg * p.seg_len + tile * kGlrTile<2> + w * share;
    GateBias bias[VEC];
    float rate[VEC];
    load_bias<FORM, VEC>(p.bias, ln.c, p.D, bias);
    channel_load<VEC>(p.rate, ln.c, p.D, rate);
    const bool near = near_rates<FORM, VEC>(rate);
    float P = 1.f, C = 0.f, S = 0.f;      // of one channel a lane
    RunRows<IO, GT, VEC, L> rows;
    rows.fetch(p, b, t_first + share - kStep, row, ln.c, true);
    Span span;
    for (int t = t_first + share - kStep; t >= t_first; t -= kStep) {
        const int t0 = t + row;
        const Marks marks = PK ? marks_of<PK, L>(p, t, kStep, t0, span) : Marks{};
        Moves<VEC> m;
        float H[VEC];
        m.none();
#pragma unroll
        for (int e = 0; e < VEC; ++e) H[e] = 0.f;
        auto walk = [&](auto odd) {
            with_scale<FORM>(p.scale, near, [&](auto sc, auto nr) {
                Span q = marks.start;
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    float xv[VEC], gv[VEC];
                    rows.x[i].get(xv);
                    rows.g[i].get(gv);
                    const bool f = odd.value && (marks.first >> i & 1);
                    if (f) q.at(p, t0 + i);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float a, c, slope, sig;
                        gate_of<FORM, nr.value>(gv[e], bias[e], rate[e], a, c, slope, sig);
                        move_on<odd.value>(f, f ? state_at(p, p.h0, q.n, ln.c + e) : 0.f, a, c, xv[e] * input_scale<sc.value>(a, c), H[e], m.P[e], m.C[e]);
                    }
                }
            });
        };
        if (PK && __ballot(marks.first != 0) != 0)
            walk(std::bool_constant<PK>());
        else
            walk(std::false_type());
        if (t > t_first) rows.fetch(p, b, t - kStep, row, ln.c, true);
        const WaveRun run = join_wave<PK, VEC, false>(m, H, H);
        S = move<PK>(P, C, run.H, S);
        join<PK>(run.P, run.C, P, C, P, C);
    }
    const int l = lane_id(), c = group * kGlrCols + ln.one();
    lds_p[w][l] = P;
    lds_c[w][l] = C;
    lds_h[w][l] = S;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    P = lds_p[0][l];
    C = lds_c[0][l];
    float H = lds_h[0][l];
#pragma unroll
    for (int j = 1; j < NW; ++j) {
        H = move<PK>(lds_p[j][l], lds_c[j][l], H, lds_h[j][l]);
        join<PK>(P, C, lds_p[j][l], lds_c[j][l], P, C);
    }
    float *out = p.ws + (((int64_t)b * segs + seg) * K + piece) * 2 * p.D + c;
    out[0] = pack_move<PK>(P, C);
    out[p.D] = H;
}

// One token for each of B rows, 256 channels a workgroup.
template <typename IO, typename GT, int FORM>
__global__ void __launch_bounds__(256) glr_step_kernel(GlrParams p) {
    const int col = blockIdx.x % p.groups, b = blockIdx.x / p.groups, c = col * 256 + threadIdx.x;
    const int64_t s = p.slots ? p.slots[b] : b;
    IO *y = (IO *)p.y + (int64_t)b * p.D + c;
    if (s < 0 || s >= p.n_slots || (p.slots && !first_with_slot(p.slots, b, (int)s))) {
        if (c < p.D) io_traits<IO>::store(y, 0.f);
        return;
    }
    if (c >= p.D) return;
    float *h = p.state + s * p.D + c;
    const float x = io_traits<IO>::load((const IO *)p.x + b * p.xb + c), g = io_traits<GT>::load((const GT *)p.g + b * p.gb + c);
    float a, k, slope, sig;
    GateBias bias[1];
    load_bias<FORM, 1>(p.bias, c, p.D, bias);
    gate_of<FORM>(g, bias[0], p.rate ? p.rate[c] : 0.f, a, k, slope, sig);
    const float v = fmaf(a, *h, x * (p.scale == GDN_GLR_PLAIN ? 1.f : p.scale == GDN_GLR_COMPLEMENT ? k : input_scale<GDN_GLR_NORM>(a, k)));
    *h = v;
    io_traits<IO>::store(y, v);
}

gdn_status check_glr(const gdn_glr_problem *pr, bool packed) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->B < 1 || pr->T < 0 || pr->D < 1) return GDN_ERR_BAD_SHAPE;
    if (packed && (pr->B != 1 || pr->n_seqs < 1 || pr->n_seqs > (1 << 24))) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->io_dtype) || (pr->g_dtype != pr->io_dtype && pr->g_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (pr->form < GDN_GLR_LOG || pr->form > GDN_GLR_RATE || pr->scale < GDN_GLR_PLAIN || pr->scale > GDN_GLR_NORM)
        return GDN_ERR_UNSUPPORTED;
    if (pr->T > (1 << 30) || pr->B > (1 << 24) || pr->D > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    // a tile's rows and the states are addressed with 32-bit byte offsets
    for (int64_t v : {pr->x_stride_t, pr->g_stride_t, pr->dy_stride_t, pr->dx_stride_t, pr->dg_stride_t})
        if (v < 0 || v > (1 << 20)) return GDN_ERR_UNSUPPORTED;
    if ((packed ? pr->n_seqs : pr->B) * pr->D >= (1 << 29)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Channels two at a time (bf16): every row of every tensor at an even element.
bool glr_pairs(const gdn_glr_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> gates,
               std::initializer_list<int64_t> strides) {
    if (pr->io_dtype != GDN_BF16 || pr->g_dtype != GDN_BF16 || pr->D % 2 != 0) return false;
    for (int64_t v : strides)
        if (v % 2 != 0) return false;
    for (const void *q : io)
        if (!aligned_to(q, 4)) return false;
    for (const void *q : gates)
        if (!aligned_to(q, 4)) return false;
    return true;
}

void fill_glr(const gdn_glr_problem *pr, GlrParams &gp, const int32_t *cu) {
    gp = GlrParams{};
    gp.cu = cu;
    gp.xb = pr->x_stride_b;
    gp.xt = pr->x_stride_t;
    gp.gb = pr->g_stride_b;
    gp.gt = pr->g_stride_t;
    gp.yb = pr->dy_stride_b;
    gp.yt = pr->dy_stride_t;
    gp.dxb = pr->dx_stride_b;
    gp.dxt = pr->dx_stride_t;
    gp.dgb = pr->dg_stride_b;
    gp.dgt = pr->dg_stride_t;
    gp.B = (int)pr->B;
    gp.T = (int)pr->T;
    gp.D = (int)pr->D;
    gp.n_seqs = cu ? (int)pr->n_seqs : 0;
    gp.n_states = cu ? pr->n_seqs : pr->B;
    gp.scale = pr->scale;
    gp.groups = (int)((pr->D + kGlrCols - 1) / kGlrCols);
}

namespace {

struct GlrPlan {
    int64_t segs, seg_len, pieces;
};

// Segments for about 256 workgroups of 64 channels, one a CU, of four tiles at least
// (a segment's rows are read once more for its move).  Their pieces for the moves: for 256
// workgroups however short, for 1024 if they keep four tiles (fp32: and are four at least, or
// the moves are of one segment, for half of the chip), for 2048, as two run on a CU, if they keep eight
// (packed rows, of which one does: not).
// Whole segments against pieces, forward: 65536 tokens of 4096 channels of bf16 530 and 492 us, 2048 of 1024
// 33.5 and 25.5; two pieces, 4096 of 8192 65.8 and 55.9 (a gate of fp32 80.8 and 69.5), 8192 of 4096 66.2 and
// 64.5; fp32, 2 x 8192 of 4096 (four pieces) 219 and 205, 4096 of 8192 (two, of one segment) 105.4 and 103.5,
// but two of each of three segments, 8192 of 4096, 104.7 and 111.3, and three, 12288 of 4096, 173 and 179.
// Pieces of one tile, for 1024 workgroups, 76 against 69 us (16384 tokens of 1030 channels); for 512 or 768
// workgroups 544 and 530 us (65536 tokens), for 1024 504; for 2048 of four tiles 251 against 247 (32768
// tokens), and packed, 65536 tokens, 551 against 539.
GlrPlan glr_plan(const gdn_glr_problem *pr) {
    constexpr int64_t kTile = kGlrTile<2>;         // (a multiple of the tile of single channels)
    const int64_t streams = pr->B * ((pr->D + kGlrCols - 1) / kGlrCols), tiles = (pr->T + kTile - 1) / kTile;
    int64_t segs = (256 + streams - 1) / streams;
    segs = segs < tiles / 4 ? segs : tiles / 4;
    segs = segs < 1 ? 1 : segs;
    GlrPlan s;
    s.seg_len = (tiles + segs - 1) / segs * kTile;
    s.seg_len = s.seg_len < kTile ? kTile : s.seg_len;
    s.segs = (pr->T + s.seg_len - 1) / s.seg_len;
    s.segs = s.segs < 1 ? 1 : s.segs;
    const int64_t wgs = streams * s.segs, n = s.seg_len / kTile;
    const int64_t fill = std::min((255 + wgs) / wgs, n), many = pr->n_seqs > 0 ? 0 : std::min((2047 + wgs) / wgs, n / 8);
    const int64_t more = std::max(std::min((1023 + wgs) / wgs, n / 4), many);
    s.pieces = std::max(fill, pr->io_dtype == GDN_F32 && s.segs > 2 && more < 4 ? 1 : more);
    return s;
}

int64_t glr_bytes(const gdn_glr_problem *pr, const GlrPlan &s) { return pr->B * (s.segs - 1) * s.pieces * 2 * pr->D * 4; }

enum { kMoves, kForward, kMany, kShort };
template <typename IO, typename GT, int VEC, bool PK, int FORM>
const void *glr_form_fn(int which) {
    if constexpr (!PK) {
        if (which == kShort) return (const void *)&glr_forward_kernel<IO, GT, VEC, PK, FORM, 1>;
        if (which == kMany) return (const void *)&glr_forward_kernel<IO, GT, VEC, PK, FORM, 4>;
    }
    return which == kMoves ? (const void *)&glr_moves_kernel<IO, GT, VEC, PK, FORM> : (const void *)&glr_forward_kernel<IO, GT, VEC, PK, FORM, kGlrWaves>;
}
template <typename IO, typename GT, int VEC, bool PK>
const void *glr_fn(int form, int which) {
    return form == GDN_GLR_LOG ? glr_form_fn<IO, GT, VEC, PK, 0>(which)
           : form == GDN_GLR_SIGMOID ? glr_form_fn<IO, GT, VEC, PK, 1>(which) : glr_form_fn<IO, GT, VEC, PK, 2>(which);
}
template <bool PK>
const void *glr_pick(const gdn_glr_problem *pr, bool pairs, int which) {
    if (pairs) return glr_fn<bf16_t, bf16_t, 2, PK>(pr->form, which);
    if (pr->io_dtype == GDN_F32) return glr_fn<float, float, 1, PK>(pr->form, which);
    return pr->g_dtype == GDN_F32 ? glr_fn<bf16_t, float, 1, PK>(pr->form, which) : glr_fn<bf16_t, bf16_t, 1, PK>(pr->form, which);
}

template <typename IO, typename GT>
const void *glr_step_fn(int form) {
    return form == GDN_GLR_LOG ? (const void *)&glr_step_kernel<IO, GT, 0>
           : form == GDN_GLR_SIGMOID ? (const void *)&glr_step_kernel<IO, GT, 1> : (const void *)&glr_step_kernel<IO, GT, 2>;
}

}  // namespace

bool glr_aligned(const gdn_glr_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> gates,
                 std::initializer_list<const void *> f32) {
    for (const void *q : io)
        if (!aligned_to(q, dtype_bytes(pr->io_dtype))) return false;
    for (const void *q : gates)
        if (!aligned_to(q, dtype_bytes(pr->g_dtype))) return false;
    for (const void *q : f32)
        if (!aligned_to(q, 4)) return false;
    return true;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_workspace_bytes_glr(const gdn_glr_problem *pr) {
    if (check_glr(pr, pr && pr->n_seqs > 0) != GDN_OK) return 0;
    return (size_t)glr_bytes(pr, glr_plan(pr));
}

gdn_status gdn_glr_forward(const gdn_glr_problem *pr, const void *x, const void *gate, const float *bias, const float *rate,
                           const float *h0, const int32_t *cu_seqlens, void *y, float *hT, void *workspace,
                           size_t workspace_bytes, void *stream) {
    gdn_status st = check_glr(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if ((pr->form == GDN_GLR_RATE) != (rate != nullptr)) return rate ? GDN_ERR_UNSUPPORTED : GDN_ERR_NULL_ARG;
    if (pr->T > 0 && (!x || !gate || !y)) return GDN_ERR_NULL_ARG;
    if (!glr_aligned(pr, {x, y}, {gate}, {bias, rate, h0, cu_seqlens, hT})) return GDN_ERR_ALIGNMENT;
    if (pr->T == 0 && !hT) return GDN_OK;
    const GlrPlan s = glr_plan(pr);
    GlrParams gp;
    fill_glr(pr, gp, cu_seqlens);
    const bool pairs = glr_pairs(pr, {x, y}, {gate}, {pr->x_stride_b, pr->x_stride_t, pr->g_stride_b, pr->g_stride_t});
    const int64_t wgs = pr->B * gp.groups;
    // A workgroup of eight waves fills a CU, so sequences that do not fill its tile are waited
    // for one after the other: one wave for up to 64 tokens (or a single run of each thread), four
    // for up to 512, where there are workgroups enough.  4096 channels of bf16: 256 sequences of 16 tokens
    // 338 us with eight waves, 35 with one; 64 of 4 tokens 85 and 11; 64 of 100 tokens 90 with eight, 35 with
    // four, of 512 tokens (32 sequences) 95 and 90.
    const int which = cu_seqlens                                                         ? kForward
                      : pr->T <= (pairs ? kGlrTile<2, 1> : kGlrTile<1, 1>) || (pr->T <= 64 && wgs >= 512) ? kShort
                      : pr->T <= 512 && wgs >= 1024                                      ? kMany
                                                                                         : kForward;
    const int waves = which == kShort ? 1 : which == kMany ? 4 : kGlrWaves;
    if (!grid_ok(s.segs * s.pieces * pr->B, (int64_t)gp.groups * 64 * waves)) return GDN_ERR_UNSUPPORTED;
    const size_t need = (size_t)glr_bytes(pr, s);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    gp.x = x;
    gp.g = gate;
    gp.bias = bias;
    gp.rate = rate;
    gp.h0 = h0;
    gp.y = y;
    gp.hT = hT;
    gp.ws = (float *)workspace;
    gp.segs = (int)s.segs;
    gp.seg_len = (int)s.seg_len;
    gp.pieces = (int)s.pieces;
    if (s.segs > 1) {
        st = launch_kernel(cu_seqlens ? glr_pick<true>(pr, pairs, kMoves) : glr_pick<false>(pr, pairs, kMoves), (int)(wgs * (s.segs - 1) * s.pieces), &gp,
                           (hipStream_t)stream, 64 * kGlrWaves);
        if (st != GDN_OK) return st;
    }
    return launch_kernel(cu_seqlens ? glr_pick<true>(pr, pairs, which) : glr_pick<false>(pr, pairs, which), (int)(wgs * s.segs), &gp,
                         (hipStream_t)stream, 64 * waves);
}

gdn_status gdn_glr_step(const gdn_glr_problem *pr, const void *x, const void *gate, const float *bias, const float *rate,
                        float *state, const int32_t *slots, int64_t n_slots, void *y, void *stream) {
    const gdn_status st = check_glr(pr, false);
    if (st != GDN_OK) return st;
    if ((pr->form == GDN_GLR_RATE) != (rate != nullptr)) return rate ? GDN_ERR_UNSUPPORTED : GDN_ERR_NULL_ARG;
    if (pr->T != 1 || n_slots < 0 || n_slots >= ((int64_t)1 << 31) || (!slots && n_slots < pr->B)) return GDN_ERR_BAD_SHAPE;
    if (!x || !gate || !y || (!state && n_slots > 0)) return GDN_ERR_NULL_ARG;
    if (!glr_aligned(pr, {x, y}, {gate}, {bias, rate, state, slots})) return GDN_ERR_ALIGNMENT;
    GlrParams gp;
    fill_glr(pr, gp, nullptr);
    gp.x = x;
    gp.g = gate;
    gp.bias = bias;
    gp.rate = rate;
    gp.state = state;
    gp.slots = slots;
    gp.n_slots = n_slots;
    gp.y = y;
    gp.groups = (int)((pr->D + 255) / 256);
    if (!grid_ok(pr->B, (int64_t)gp.groups * 256)) return GDN_ERR_UNSUPPORTED;
    const void *fn = pr->io_dtype == GDN_F32   ? glr_step_fn<float, float>(pr->form)
                     : pr->g_dtype == GDN_F32 ? glr_step_fn<bf16_t, float>(pr->form)
                                              : glr_step_fn<bf16_t, bf16_t>(pr->form);
    return launch_kernel(fn, (int)(pr->B * gp.groups), &gp, (hipStream_t)stream);
}

}  // extern "C"

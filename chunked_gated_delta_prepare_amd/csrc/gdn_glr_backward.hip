// Gated linear recurrence, backward (see gdn_glr.h).  With h_t formed again,
//
//   dh_t = dy_t + e_{t+1},  e_t = a_t dh_t        (e behind the last token: dhT)
//   dx_t = c_t dh_t,  d(log a_t) = e_t h_{t-1} + dh_t x_t dc/d(log a)
//
// so two recurrences with the same decays, h forwards and e backwards, whose
// runs join alike.  A workgroup has one tile of tokens and 64 channels and needs
// the h in front of it and the e behind it: a first launch leaves every tile's
// moves in the workspace, a second turns them into those states, and the third
// reads its tile again and writes the gradients.  It takes the tiles in the
// other order, so that the last ones come out of the last cache.
// 2 x 8192 tokens of 4096 channels, rate and norm: 87 us the moves (403 MB, 4.6 TB/s), 13 the
// states, 156 the gradients (700 MB, 4.5 TB/s; some 60 vector instructions an element keep the
// units busy for 0.77 of it), 8 the sums.  Tiles of 32 tokens, 4 a thread, in 104
// registers: 8 a thread do not fit the 128 of four waves a SIMD.
#include "gdn_glr.h"
#include "gdn_norm_rows.h"

namespace gdn {

constexpr int kGbWaves = 4;
template <int VEC>
constexpr int kGbRun = VEC == 2 ? 4 : 8;      // tokens of a thread
template <int VEC>
constexpr int kGbTile = kGbWaves * GlrLane<VEC>::kTG * kGbRun<VEC>;
static_assert(kGbTile<1> == 32 && kGbTile<2> == 32, "whether channels go in pairs depends on pointers, a workspace's size does not");

template <typename IO, int VEC, int L>
__device__ __forceinline__ void fetch_dy(const GlrParams &p, RawRow<IO, VEC> (&dy)[L], int b, int t_base, int row, int c, bool full) {
    const TileRows<IO, VEC> rd(p.dy, b * p.yb + (int64_t)t_base * p.yt, p.yt, row, c, p.D);
    const int n = p.T - t_base - row;
#pragma unroll
    for (int i = 0; i < L; ++i) rd.load(dy[i], i, full || i < n);
}

// A tile's place in the workspace: [3][D], its packed move, then H and E, which the
// second launch replaces by the states at its borders.
__device__ __forceinline__ float *tile_at(const GlrParams &p, int b, int tile) { return p.ws + ((int64_t)b * p.segs + tile) * 3 * p.D; }

template <typename IO, typename GT, int VEC, bool PK, int FORM>
__global__ void __launch_bounds__(64 * kGbWaves) glr_tiles_kernel(GlrParams p) {
    constexpr int L = kGbRun<VEC>, NW = kGbWaves;
    __shared__ float lds[4][NW][kGlrCols];
    const int group = blockIdx.x % p.groups, rest = blockIdx.x / p.groups, tile = rest % p.segs, b = rest / p.segs;
    const GlrLane<VEC> ln(group);
    const int w = wave_id(), row = (w * ln.kTG + ln.tg) * L, t = tile * kGbTile<VEC>, t0 = t + row;
    RunRows<IO, GT, VEC, L> rows;
    RawRow<IO, VEC> dyr[L];
    const bool full = t + kGbTile<VEC> <= p.T;
    rows.fetch(p, b, t, row, ln.c, full);
    fetch_dy<IO, VEC, L>(p, dyr, b, t, row, ln.c, full);
    GateBias bias[VEC];
    float rate[VEC];
    load_bias<FORM, VEC>(p.bias, ln.c, p.D, bias);
    channel_load<VEC>(p.rate, ln.c, p.D, rate);
    const bool near = near_rates<FORM, VEC>(rate);
    Span span;
    const Marks marks = marks_of<PK, L>(p, t + w * ln.kTG * L, ln.kTG * L, t0, span);
    Moves<VEC> m;
    float H[VEC], E[VEC];
    m.none();
#pragma unroll
    for (int e = 0; e < VEC; ++e) H[e] = E[e] = 0.f;
    // E as a sum over the run: what its tokens' dy leave behind the run's front
    auto walk = [&](auto odd) {
        with_scale<FORM>(p.scale, near, [&](auto sc, auto nr) {
            Span q = marks.start;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                float xv[VEC], gv[VEC], dv[VEC];
                rows.x[i].get(xv);
                rows.g[i].get(gv);
                dyr[i].get(dv);
                const bool ok = !odd.value || (marks.valid >> i & 1), f = PK && odd.value && (marks.first >> i & 1);
                const bool end = PK && odd.value && (marks.last >> i & 1);
                if (f || end) q.at(p, t0 + i);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float a, c, slope, sig;
                    gate_of<FORM, nr.value>(gv[e], bias[e], rate[e], a, c, slope, sig);
                    float u = xv[e] * input_scale<sc.value>(a, c);
                    if (odd.value && !ok) {
                        // a token of no sequence moves nothing
                        a = 1.f;
                        c = u = dv[e] = 0.f;
                    }
                    if (end) dv[e] += state_at(p, p.dhT, q.n, ln.c + e);
                    move_on<PK && odd.value>(f, f ? state_at(p, p.h0, q.n, ln.c + e) : 0.f, a, c, u, H[e], m.P[e], m.C[e]);
                    // (behind a first token P is marked, and e does not pass it)
                    E[e] = PK && m.P[e] < 0.f ? E[e] : fmaf(m.P[e], dv[e], E[e]);
                }
            }
        });
    };
    if (__ballot(marks.valid != (1u << L) - 1 || (PK && (marks.first | marks.last) != 0)) != 0)
        walk(std::true_type());
    else
        walk(std::false_type());
    const WaveRun run = join_wave<PK, VEC, true>(m, H, E);
    const int l = lane_id(), c = group * kGlrCols + ln.one();
    lds[0][w][l] = run.P;
    lds[1][w][l] = run.C;
    lds[2][w][l] = run.H;
    lds[3][w][l] = run.E;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
    float P = lds[0][0][l], C = lds[1][0][l], hh = lds[2][0][l], ee = lds[3][0][l];
#pragma unroll
    for (int j = 1; j < NW; ++j) {
        const float P2 = lds[0][j][l], C2 = lds[1][j][l];
        hh = move<PK>(P2, C2, hh, lds[2][j][l]);
        ee = move<PK>(P, C, lds[3][j][l], ee);
        join<PK>(P, C, P2, C2, P, C);
    }
    float *out = tile_at(p, b, tile) + c;
    out[0] = pack_move<PK>(P, C);
    out[p.D] = hh;
    out[2 * (int64_t)p.D] = ee;
}

// H -> the h in front of a tile, E -> the e behind it: 64 channels and one
// direction a workgroup.  Each of its waves (16, or one a tile if they are fewer: many short
// sequences need many workgroups) has a share of the tiles: its move first, then, from the
// state at its border, its tiles'.
constexpr int kGsWaves = 16;
template <bool PK>
__global__ void __launch_bounds__(64 * kGsWaves) glr_states_kernel(GlrParams p) {
    __shared__ float lds_p[kGsWaves][kGlrCols], lds_c[kGsWaves][kGlrCols], lds_h[kGsWaves][kGlrCols];
    const int back = blockIdx.x & 1, rest = blockIdx.x >> 1, group = rest % p.groups, b = rest / p.groups;
    const int w = wave_id(), l = lane_id(), c = group * kGlrCols + l;
    const bool live = c < p.D;
    const int waves = blockDim.x / 64, share = (p.segs + waves - 1) / waves, n0 = w * share, n1 = n0 + share < p.segs ? n0 + share : p.segs;
    // tile i of this direction's order
    auto at = [&](int i) { return tile_at(p, b, back ? p.segs - 1 - i : i) + (live ? c : 0); };
    const int64_t from = (int64_t)(1 + back) * p.D;
    float P = 1.f, C = 0.f, S = 0.f;
#pragma unroll 4
    for (int i = n0; i < n1; ++i) {
        const float q = at(i)[0], H = at(i)[from];
        const bool far = __float_as_int(q) < 0;
        const bool cut = PK && q == -__builtin_inff();
        S = packed_move<PK>(q, S, H);
        join<PK>(P, C, cut ? -1.f : far ? -q : 1.f - q, cut ? 1.f : far ? 1.f + q : q, P, C);
    }
    lds_p[w][l] = P;
    lds_c[w][l] = C;
    lds_h[w][l] = S;
    __syncthreads();
    if (!live) return;
    // (packed rows take them at their sequences' first and last tokens)
    const float *s0 = PK ? nullptr : back ? p.dhT : p.h0;
    S = s0 ? s0[(int64_t)b * p.D + c] : 0.f;
    for (int j = 0; j < w; ++j) S = move<PK>(lds_p[j][l], lds_c[j][l], S, lds_h[j][l]);
#pragma unroll 4
    for (int i = n0; i < n1; ++i) {
        float *s = at(i);
        const float q = s[0], H = s[from];
        s[from] = S;
        S = packed_move<PK>(q, S, H);
    }
}

template <typename IO, typename GT, int VEC, bool PK, int FORM>
__global__ void __launch_bounds__(64 * kGbWaves, 4) glr_backward_kernel(GlrParams p) {
    constexpr int L = kGbRun<VEC>, NW = kGbWaves;
    __shared__ float lds[3][NW][kGlrCols];
    const int group = blockIdx.x % p.groups, rest = blockIdx.x / p.groups, tile = p.segs - 1 - rest % p.segs, b = rest / p.segs;
    const GlrLane<VEC> ln(group);
    const int w = wave_id(), row = (w * ln.kTG + ln.tg) * L, t = tile * kGbTile<VEC>, t0 = t + row;
    RunRows<IO, GT, VEC, L> rows;
    RawRow<IO, VEC> dyr[L];
    const bool full = t + kGbTile<VEC> <= p.T;
    rows.fetch(p, b, t, row, ln.c, full);
    fetch_dy<IO, VEC, L>(p, dyr, b, t, row, ln.c, full);
    // (states and moves between runs are of one channel a lane)
    const int l = lane_id(), c1 = group * kGlrCols + ln.one();
    GateBias bias[VEC];
    float rate[VEC], h1[1], d1[1];
    load_bias<FORM, VEC>(p.bias, ln.c, p.D, bias);
    channel_load<VEC>(p.rate, ln.c, p.D, rate);
    const bool near = near_rates<FORM, VEC>(rate);
    if (p.segs > 1) {
        channel_load<1>(tile_at(p, b, tile) + p.D, c1, p.D, h1);
        channel_load<1>(tile_at(p, b, tile) + 2 * (int64_t)p.D, c1, p.D, d1);
    } else {
        state_load<1>(p, PK ? nullptr : p.h0, b, c1, h1);
        state_load<1>(p, PK ? nullptr : p.dhT, b, c1, d1);
    }
    if (tile == 0) pass_empty(p, PK, b, group * kGlrCols, p.dhT, p.dh0);
    Span span;
    const Marks marks = marks_of<PK, L>(p, t + w * ln.kTG * L, ln.kTG * L, t0, span);
    const bool odd = __ballot(marks.valid != (1u << L) - 1 || marks.first != 0 || (PK && marks.last != 0)) != 0;
    // what the walk back needs of a token: a, the input's factor k and its slope, the gate's slope and sigmoid
    float a[L][VEC], k[L][VEC], dk[L][VEC], slope[L][VEC], sig[L][VEC], x[L][VEC], dy[L][VEC], H[VEC], E[VEC];
    Moves<VEC> m;
    m.none();
#pragma unroll
    for (int e = 0; e < VEC; ++e) H[e] = E[e] = 0.f;
    with_scale<FORM>(p.scale, near, [&](auto sc, auto nr) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float gv[VEC];
            rows.x[i].get(x[i]);
            rows.g[i].get(gv);
            dyr[i].get(dy[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float c;
                gate_of<FORM, nr.value>(gv[e], bias[e], rate[e], a[i][e], c, slope[i][e], sig[i][e]);
                input_slope<sc.value>(a[i][e], c, k[i][e], dk[i][e]);
                move_on<false>(false, 0.f, a[i][e], c, k[i][e] * x[i][e], H[e], m.P[e], m.C[e]);
                E[e] = fmaf(m.P[e], dy[i][e], E[e]);
            }
        }
    });
    int seq[L];                    // of first tokens
#pragma unroll
    for (int i = 0; i < L; ++i) seq[i] = b;
    if (odd) {
        // the run again, token by token
        float n[VEC];
        Span q = marks.start;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            n[e] = E[e] = 0.f;
            m.P[e] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const bool ok = marks.valid >> i & 1, f = PK && (marks.first >> i & 1), end = PK && (marks.last >> i & 1);
            if (f || end) {
                q.at(p, t0 + i);
                seq[i] = q.n;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (!ok) {
                    // a token of no sequence moves nothing, and may hold anything
                    a[i][e] = 1.f;
                    k[i][e] = dk[i][e] = slope[i][e] = sig[i][e] = x[i][e] = dy[i][e] = 0.f;
                }
                if (end) dy[i][e] += state_at(p, p.dhT, seq[i], ln.c + e);
                const float h0 = f ? state_at(p, p.h0, seq[i], ln.c + e) : n[e];
                n[e] = fmaf(a[i][e], h0, k[i][e] * x[i][e]);
                m.P[e] = f || m.P[e] < 0.f ? -1.f : m.P[e] * a[i][e];
                E[e] = m.P[e] < 0.f ? E[e] : fmaf(m.P[e], dy[i][e], E[e]);
            }
        }
        if (marks.valid != (1u << L) - 1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) m.C[e] = 1.f - m.P[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) H[e] = n[e];
    }
    const WaveRun run = join_wave<PK, VEC, true>(m, H, E);
    lds[0][w][l] = pack_move<PK>(run.P, run.C);
    lds[1][w][l] = run.H;
    lds[2][w][l] = run.E;
    lds_barrier();
#pragma unroll
    for (int j = 0; j < NW - 1; ++j) {
        const int q = NW - 1 - j;
        if (j < w) h1[0] = packed_move<PK>(lds[0][j][l], h1[0], lds[1][j][l]);
        if (q > w) d1[0] = packed_move<PK>(lds[0][q][l], d1[0], lds[2][q][l]);
    }
    float h[VEC], d[VEC];
    spread_state<PK, VEC>(run, h1[0], h);
    spread_behind<PK, VEC>(run, d1[0], d);
    // the state in front of every token
    float prev[L][VEC];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if (PK && odd && (marks.first >> i & 1)) state_load<VEC>(p, p.h0, seq[i], ln.c, h);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            prev[i][e] = h[e];
            h[e] = fmaf(a[i][e], h[e], k[i][e] * x[i][e]);
        }
    }
    const TileRows<IO, VEC> rx(p.dx, b * p.dxb + (int64_t)t * p.dxt, p.dxt, row, ln.c, p.D);
    const TileRows<GT, VEC> rg(p.dg, b * p.dgb + (int64_t)t * p.dgt, p.dgt, row, ln.c, p.D);
    float sb[VEC], sr[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sb[e] = sr[e] = 0.f;
    auto walk = [&](auto some) {
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            float dx[VEC], dg[VEC];
            const bool ok = !some.value || (marks.valid >> i & 1);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float dh = dy[i][e] + d[e], out = a[i][e] * dh;
                const float da = fmaf(out, prev[i][e], dh * x[i][e] * dk[i][e]);
                dx[e] = dh * k[i][e];
                dg[e] = da * slope[i][e];
                // (what a token of no sequence has in front of it may be no number)
                sb[e] += ok ? dg[e] : 0.f;
                sr[e] -= ok ? da * sig[i][e] : 0.f;
                d[e] = out;
            }
            rx.store(dx, i, ok);
            rg.store(dg, i, ok);
            if (some.value && (marks.first >> i & 1)) {
                if (p.dh0) state_store<VEC>(p, p.dh0, seq[i], ln.c, true, d);
                if (PK) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = 0.f;
                }
            }
        }
    };
    if (odd)
        walk(std::true_type());
    else
        walk(std::false_type());
    if (!p.grads) return;
    // the tile's sums, in a fixed order
    __syncthreads();
    if constexpr (VEC == 2) {
        swap_halves(sb[0], sb[1]);
        swap_halves(sr[0], sr[1]);
        sb[0] += sb[1];
        sr[0] += sr[1];
    }
    lds[0][w][l] = sb[0];
    lds[1][w][l] = sr[0];
    __syncthreads();
    if (w > 1 || c1 >= p.D) return;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NW; ++j) s += lds[w][j][l];
    p.part[(((int64_t)b * p.segs + tile) * 2 + w) * p.D + c1] = s;
}

namespace {

int64_t glr_tiles(const gdn_glr_problem *pr) {
    const int64_t n = (pr->T + kGbTile<2> - 1) / kGbTile<2>;
    return n < 1 ? 1 : n;
}

// Two sums a tile and channel, and where tiles meet its move, H and E.
int64_t glr_backward_bytes(const gdn_glr_problem *pr) {
    const int64_t n = glr_tiles(pr);
    return pr->B * n * (n > 1 ? 5 : 2) * pr->D * 4;
}

template <typename IO, typename GT, int VEC, bool PK>
const void *glr_back_fn(int form, bool tiles) {
    switch (form) {
        case GDN_GLR_LOG:
            return tiles ? (const void *)&glr_tiles_kernel<IO, GT, VEC, PK, 0> : (const void *)&glr_backward_kernel<IO, GT, VEC, PK, 0>;
        case GDN_GLR_SIGMOID:
            return tiles ? (const void *)&glr_tiles_kernel<IO, GT, VEC, PK, 1> : (const void *)&glr_backward_kernel<IO, GT, VEC, PK, 1>;
        default:
            return tiles ? (const void *)&glr_tiles_kernel<IO, GT, VEC, PK, 2> : (const void *)&glr_backward_kernel<IO, GT, VEC, PK, 2>;
    }
}
template <bool PK>
const void *glr_back_pick(const gdn_glr_problem *pr, bool pairs, bool tiles) {
    if (pairs) return glr_back_fn<bf16_t, bf16_t, 2, PK>(pr->form, tiles);
    if (pr->io_dtype == GDN_F32) return glr_back_fn<float, float, 1, PK>(pr->form, tiles);
    return pr->g_dtype == GDN_F32 ? glr_back_fn<bf16_t, float, 1, PK>(pr->form, tiles) : glr_back_fn<bf16_t, bf16_t, 1, PK>(pr->form, tiles);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_workspace_bytes_glr_backward(const gdn_glr_problem *pr) {
    if (check_glr(pr, pr && pr->n_seqs > 0) != GDN_OK) return 0;
    return (size_t)glr_backward_bytes(pr);
}

gdn_status gdn_glr_backward(const gdn_glr_problem *pr, const void *dy, const void *x, const void *gate, const float *bias,
                            const float *rate, const float *h0, const int32_t *cu_seqlens, const float *dhT, void *dx,
                            void *dgate, float *dbias, float *drate, float *dh0, void *workspace, size_t workspace_bytes,
                            void *stream) {
    gdn_status st = check_glr(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if ((pr->form == GDN_GLR_RATE) != (rate != nullptr)) return rate ? GDN_ERR_UNSUPPORTED : GDN_ERR_NULL_ARG;
    if (drate && !rate) return GDN_ERR_UNSUPPORTED;
    if (pr->T > 0 && (!dy || !x || !gate || !dx || !dgate)) return GDN_ERR_NULL_ARG;
    if (!glr_aligned(pr, {dy, x, dx}, {gate, dgate}, {bias, rate, h0, cu_seqlens, dhT, dbias, drate, dh0})) return GDN_ERR_ALIGNMENT;
    const size_t need = (size_t)glr_backward_bytes(pr);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    GlrParams gp;
    fill_glr(pr, gp, cu_seqlens);
    const bool pairs = glr_pairs(pr, {dy, x, dx}, {gate, dgate},
                                 {pr->x_stride_b, pr->x_stride_t, pr->g_stride_b, pr->g_stride_t, pr->dy_stride_b, pr->dy_stride_t,
                                  pr->dx_stride_b, pr->dx_stride_t, pr->dg_stride_b, pr->dg_stride_t});
    const int64_t tiles = glr_tiles(pr);
    // (the states' launch, of two waves or fewer for every tile, is the smaller one)
    if (!grid_ok(tiles * pr->B, (int64_t)gp.groups * 64 * kGbWaves)) return GDN_ERR_UNSUPPORTED;
    gp.dy = dy;
    gp.x = x;
    gp.g = gate;
    gp.bias = bias;
    gp.rate = rate;
    gp.h0 = h0;
    gp.dhT = dhT;
    gp.dx = dx;
    gp.dg = dgate;
    gp.dh0 = dh0;
    gp.segs = (int)tiles;
    gp.grads = dbias || drate;
    gp.part = (float *)workspace;
    gp.ws = gp.part + pr->B * tiles * 2 * pr->D;
    const int grid = (int)(pr->B * tiles * gp.groups);
    hipStream_t s = (hipStream_t)stream;
    if (tiles > 1) {
        st = launch_kernel(cu_seqlens ? glr_back_pick<true>(pr, pairs, true) : glr_back_pick<false>(pr, pairs, true), grid, &gp, s, 64 * kGbWaves);
        if (st != GDN_OK) return st;
        st = launch_kernel(cu_seqlens ? (const void *)&glr_states_kernel<true> : (const void *)&glr_states_kernel<false>,
                           (int)(2 * pr->B * gp.groups), &gp, s, 64 * (int)(tiles < kGsWaves ? tiles : kGsWaves));
        if (st != GDN_OK) return st;
    }
    st = launch_kernel(cu_seqlens ? glr_back_pick<true>(pr, pairs, false) : glr_back_pick<false>(pr, pairs, false), grid, &gp, s, 64 * kGbWaves);
    if (st != GDN_OK || !gp.grads) return st;
    return enqueue_norm_sums(gp.part, dbias, drate, pr->D, pr->B * tiles, 1, s);
}

}  // extern "C"

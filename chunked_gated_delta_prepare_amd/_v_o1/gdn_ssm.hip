// Selective state space scan, forward (see gdn_ssm.h for the mathematics).
//
// A workgroup walks one segment of one stream, a stream being 64 or 128
// columns of the state: one head's, or two heads' of a group, which then share
// B, C and the products C . B.
#include "gdn_ssm.h"

namespace gdn {

struct StepParams {
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *bias;
    float *state;
    void *y;
    const int32_t *slots;
    int64_t xb, bb, db, n_slots;
    int H, heads_per_group, softplus, dt_f32;
};

// One token: h' = e^(dt A) h + dt B x^T, y = h'^T C + D x.  A workgroup moves
// one head's state on, once through registers; its rows of P columns are dealt
// to the waves, a lane two columns.  Bound by reading and writing the state: 64
// rows of 64 heads of 128 x 128 take 109 us (4.8 TB/s, the rate of a copy).
template <typename IO, int P, int N>
__global__ void __launch_bounds__(256) ssm_step_kernel(StepParams p) {
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
    const float dv = raw + (p.bias ? p.bias[head] : 0.f), dt = p.softplus ? softplus(dv) : dv;
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

// 128 columns a workgroup where a head, or two heads of one group, fill them
// (every row of B and C then serves twice the columns), else 64.  fp32 io has
// 64 (its tiles fill LDS).
static int columns(const gdn_ssm_problem *pr) {
    if (pr->io_dtype == GDN_F32) return 1;
    return pr->P == 128 || (pr->H / pr->G) % 2 == 0 ? 2 : 1;
}

SsmPlan ssm_plan(const gdn_ssm_problem *pr, bool packed) {
    SsmPlan s;
    s.ncb = columns(pr);
    s.nh = s.ncb == 2 && pr->P == 64 ? 2 : 1;
    s.n_hb = (int)(pr->H * pr->P / (64 * s.ncb));
    s.seqs = (int)(packed ? pr->n_seqs : pr->B);
    const int64_t chunks = (pr->T + kSsmChunk - 1) / kSsmChunk;
    // segments for about 512 workgroups, two a CU, of four chunks or a multiple,
    // and 32 a stream at most (each reads the end states of those before it).
    // For 256, 512 and 1024 workgroups 65536 tokens of 64 heads take 1.52, 1.31
    // and 1.35 ms, 16384 tokens 404, 350 and 383 us.  Packed sequences end
    // inside a segment, so a quarter more (16384 tokens for 512 and 640: 80 heads
    // of 64 columns, 9 sequences 269 and 266 us, 3 sequences 291 and 262; but 64
    // heads of 128, 8 sequences 378 and 386).
    const int64_t streams = (int64_t)s.n_hb * (packed ? 1 : pr->B);
    const int64_t wgs = packed ? 640 : 512;
    int64_t per = (wgs + streams - 1) / streams;
    per = per > 32 ? 32 : per;
    int64_t seg = (chunks + per - 1) / per;
    seg = (seg < 4 ? 4 : seg + 3) / 4 * 4;
    s.seg_tokens = (int)(seg * kSsmChunk);
    const int64_t cut = (pr->T + s.seg_tokens - 1) / s.seg_tokens;
    s.n_items = (int)(packed ? cut + pr->n_seqs : pr->B * (cut > 0 ? cut : 1));
    // A sequence of L tokens with several segments has (L - 1) / seg + 1 of them; of
    // m such ones, T tokens in all, the segments are at most (T - m) / seg + m,
    // which grows with m.  (A lone segment has no end state to hand on: with a place
    // for every segment 16384 tokens of 64 heads of 128 x 128 took 46 MB as one
    // sequence and 1.1 GB as 256, now 42 and 76 MB.)
    const int64_t m = packed ? (pr->n_seqs < pr->T / (s.seg_tokens + 1) ? pr->n_seqs : pr->T / (s.seg_tokens + 1)) : 0;
    s.n_ends = (int)(packed ? (m > 0 ? (pr->T - m) / s.seg_tokens + m : 0) : cut > 1 ? s.n_items : 0);
    return s;
}

// Blocks that share B and C go to one XCD where the (segment, group) pairs come
// out even over the eight: B and C are then read from HBM once, not once per
// XCD (64 heads of 128 columns, 8 groups, with and without: 65536 tokens 1.31
// and 1.36 ms, 16384 tokens 350 and 365 us, 16384 tokens in 8 packed sequences
// 386 and 400 us).
int ssm_grid(const gdn_ssm_problem *pr, SsmParams &sp, const SsmPlan &s, bool ends) {
    sp.seg_tokens = s.seg_tokens;
    sp.n_items = s.n_items;
    sp.n_ends = s.n_ends;
    sp.n_units = ends ? s.n_ends : s.n_items;
    sp.n_hb = s.n_hb;
    sp.n_seqs = s.seqs;
    sp.swizzle = (int64_t)sp.n_units * pr->G % 8 == 0 && s.n_hb % pr->G == 0;
    return sp.n_units * s.n_hb;
}

static size_t forward_ws(const gdn_ssm_problem *pr, const SsmPlan &s) {
    return (size_t)s.n_ends * s.n_hb * (8 * 2 + 4 * pr->N * 64 * s.ncb);
}

gdn_status check_ssm(const gdn_ssm_problem *pr, bool packed) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->B < 1 || pr->T < 0 || pr->H < 1 || pr->P < 1 || pr->N < 1 || pr->G < 1 || pr->H % pr->G != 0)
        return GDN_ERR_BAD_SHAPE;
    if (packed && (pr->B != 1 || pr->n_seqs < 1 || pr->n_seqs > (1 << 24))) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->io_dtype) || (pr->dt_dtype != pr->io_dtype && pr->dt_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if ((pr->P != 64 && pr->P != 128) || (pr->N != 64 && pr->N != 128)) return GDN_ERR_UNSUPPORTED;
    // a chunk's rows are addressed with 32-bit byte offsets
    if (pr->T > (1 << 30) || pr->B > (1 << 20) || pr->H > (1 << 14)) return GDN_ERR_UNSUPPORTED;
    for (int64_t v : {pr->x_stride_t, pr->bc_stride_t, pr->dt_stride_t, pr->dxbc_stride_t})
        if (v < 0 || v > (1 << 22)) return GDN_ERR_UNSUPPORTED;
    // what lies behind a chunk's last row is told by its place: rows do not overlap
    if (pr->T > 1 && (pr->x_stride_t < pr->H * pr->P || pr->bc_stride_t < pr->G * pr->N)) return GDN_ERR_UNSUPPORTED;
    // the scans' and the gates' workgroups
    const SsmPlan s = ssm_plan(pr, packed);
    const int64_t n = s.n_items;
    if (!grid_ok(n * s.n_hb, 512) || !grid_ok(n * pr->H, 256)) return GDN_ERR_UNSUPPORTED;
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
    sp.qkb = pr->bc_stride_b;
    sp.qkt = pr->bc_stride_t;
    sp.db = pr->dt_stride_b;
    sp.dt_ = pr->dt_stride_t;
    sp.T = (int)pr->T;
    sp.H = (int)pr->H;
    sp.P = (int)pr->P;
    sp.heads_per_group = (int)(pr->H / pr->G);
    sp.softplus = pr->softplus != 0;
    sp.dt_f32 = pr->dt_dtype == GDN_F32;
}

namespace {

// The main pass, or the one for the end states.
template <typename IO, int N, int COLS, int NH>
const void *ssm_fn(bool ends) {
    return ends ? (const void *)&ssm_scan_kernel<IO, N, COLS, NH, true, false> : (const void *)&ssm_scan_kernel<IO, N, COLS, NH, false, false>;
}

template <int N>
const void *ssm_pick(const gdn_ssm_problem *pr, const SsmPlan &s, bool ends) {
    if (pr->io_dtype == GDN_F32) return ssm_fn<float, N, 64, 1>(ends);
    if (s.ncb == 1) return ssm_fn<bf16_t, N, 64, 1>(ends);
    return s.nh == 2 ? ssm_fn<bf16_t, N, 128, 2>(ends) : ssm_fn<bf16_t, N, 128, 1>(ends);
}
const void *ssm_pick(const gdn_ssm_problem *pr, const SsmPlan &s, bool ends) {
    return pr->N == 64 ? ssm_pick<64>(pr, s, ends) : ssm_pick<128>(pr, s, ends);
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
    return forward_ws(pr, ssm_plan(pr, packed));
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
    } else if (hT) {
        // (the scan reads its heads' A, D and bias before it knows of no token)
        if (!A) return GDN_ERR_NULL_ARG;
        if (!aligned_to(A, 4) || !aligned_to(D, 4) || !aligned_to(dt_bias, 4)) return GDN_ERR_ALIGNMENT;
    }
    if (!aligned_to(y, 16) || !aligned_to(h0, 4) || !aligned_to(hT, 4) || !aligned_to(cu_seqlens, 4)) return GDN_ERR_ALIGNMENT;
    if (pr->T == 0 && !hT) return GDN_OK;
    const SsmPlan s = ssm_plan(pr, cu_seqlens != nullptr);
    const size_t need = forward_ws(pr, s);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    SsmParams sp;
    fill_ssm(pr, sp);
    sp.q = Cm;
    sp.k = Bm;
    sp.v = x;
    sp.vb = pr->x_stride_b;
    sp.vt = pr->x_stride_t;
    sp.dt = dt;
    sp.A = A;
    sp.D = D;
    sp.bias = dt_bias;
    sp.s0 = h0;
    sp.cu = cu_seqlens;
    sp.out = y;
    sp.ot = pr->H * pr->P;
    sp.ob = sp.ot * pr->T;
    sp.sT = hT;
    sp.total = (double *)workspace;
    sp.ends = (float *)workspace + (int64_t)s.n_ends * s.n_hb * 4;
    sp.all_ends = hT != nullptr && s.n_ends > 0;
    if (s.n_ends > 0) {
        const int grid = ssm_grid(pr, sp, s, true);
        st = launch_kernel(ssm_pick(pr, s, true), grid, &sp, (hipStream_t)stream, 256 * s.ncb);
        if (st != GDN_OK) return st;
    }
    const int grid = ssm_grid(pr, sp, s, false);
    return launch_kernel(ssm_pick(pr, s, false), grid, &sp, (hipStream_t)stream, 256 * s.ncb);
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
    StepParams sp{};
    sp.x = x;
    sp.dt = dt;
    sp.Bm = Bm;
    sp.Cm = Cm;
    sp.A = A;
    sp.D = D;
    sp.bias = dt_bias;
    sp.state = state;
    sp.slots = slots;
    sp.n_slots = n_slots;
    sp.y = y;
    sp.xb = pr->x_stride_b;
    sp.bb = pr->bc_stride_b;
    sp.db = pr->dt_stride_b;
    sp.H = (int)pr->H;
    sp.heads_per_group = (int)(pr->H / pr->G);
    sp.softplus = pr->softplus != 0;
    sp.dt_f32 = pr->dt_dtype == GDN_F32;
    const void *fn = pr->io_dtype == GDN_F32 ? step_fn<float>(pr->P, pr->N) : step_fn<bf16_t>(pr->P, pr->N);
    return launch_kernel(fn, (int)(pr->B * pr->H), &sp, (hipStream_t)stream);
}

}  // extern "C"

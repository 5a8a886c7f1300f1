// Short causal convolution, one filter of W taps (2, 3 or 4) per channel:
//
//   v_t = b + sum_j w_j x_{t-(W-1)+j},  y_t = act(v_t)
//   dv_t = dy_t act'(v_t),  dx_t = sum_j w_j dv_{t+(W-1)-j},
//   dw_j = sum_t dv_t x_{t-(W-1)+j},  db = sum_t dv_t
//
// Bound by memory.  Channels lie innermost, so a lane takes VEC of them (8
// bytes of bf16) and walks down a run of tokens with the last W inputs in
// registers: an input is read once, and W - 1 times in W..run more at a run's
// border, from cache.  A run never crosses a batch; in packed sequences the
// window is loaded anew from the next sequence's state where one begins.
// States are a copy of W - 1 rows, done by workgroups of their own behind the
// runs.
// Runs of 32 tokens, rows eight ahead in flight: 16384 packed tokens of 10240
// channels in bf16 133 us (5.1 TB/s; 211 us without rows in flight); 2 x 8192
// tokens of 6144 channels 73 us forward (5.5 TB/s, part of it out of the last
// cache) and 139 us backward (4.4 TB/s); a token for 64 rows of 10240 channels
// 4.7 us, a launch's own time.
#include "gdn_layer.h"

namespace gdn {

struct ConvParams {
    const void *x, *w, *bias, *init, *dy, *dfinal;
    void *y, *final_, *dx, *dinit, *state;
    float *dw, *db, *part;
    const int32_t *cu, *slots;
    int64_t xb, xt, db_, dt_;          // strides of x and dy
    int64_t n_slots;
    int B, T, D, n_seqs, runs, cols, w_f32, silu, nparts;
};

// The sequence that row b * T + t belongs to: its number and its rows
// [begin, end) within batch b.
struct Seq {
    int n, begin, end;
};

__device__ __forceinline__ int cu_at(const ConvParams &p, int n) {
    const int v = p.cu[n];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

// The last sequence that begins at or before token t (packed), or batch b.
__device__ __forceinline__ Seq find_seq(const ConvParams &p, int b, int t) {
    if (!p.cu) return Seq{b, 0, p.T};
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu_at(p, mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return Seq{lo, cu_at(p, lo), cu_at(p, lo + 1)};
}

__device__ __forceinline__ Seq seq_at(const ConvParams &p, int n) {
    return p.cu ? Seq{n, cu_at(p, n), cu_at(p, n + 1)} : Seq{n, 0, p.T};
}

template <typename IO, int VEC, int W>
struct Filter {
    float w[W][VEC], b[VEC];
    __device__ __forceinline__ void load(const ConvParams &p, int c) {
        const uint32_t wb = p.w_f32 ? 4 : sizeof(IO);
        const rsrc_t rw = make_rsrc(p.w, (uint32_t)p.D * W * wb);
        if constexpr (VEC == 4) {
            // VEC W consecutive weights
            float flat[W][4];
#pragma unroll
            for (int i = 0; i < W; ++i) row_load_either<IO, 4>(rw, p.w_f32, (uint32_t)c * W + 4 * i, flat[i]);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][i] = flat[(i * W + j) / 4][(i * W + j) % 4];
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float one[1];
                row_load_either<IO, 1>(rw, p.w_f32, (uint32_t)c * W + j, one);
                w[j][0] = one[0];
            }
        }
        if (p.bias) {
            row_load_either<IO, VEC>(make_rsrc(p.bias, (uint32_t)p.D * wb), p.w_f32, c, b);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[i] = 0.f;
        }
    }
};

template <typename IO>
__device__ __forceinline__ rsrc_t row_of(const void *base, int64_t elems, int D) {
    return make_rsrc((const IO *)base + elems, (uint32_t)D * sizeof(IO));
}

// (the reciprocal is good to one unit in the last place; a division proper
// costs ten instructions: with it and a descriptor per row the forward pass of
// 16384 tokens, 10240 channels took 249 us, without 211)
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + fast_exp2(v * -kLog2e)); }

// A lane's VEC columns in rows at one stride: a descriptor at the first row,
// the lane's byte offset, and a uniform offset for the row.  Columns at or past
// D read as zero and are not stored.
template <typename IO, int VEC>
struct Cols {
    static constexpr uint32_t kNone = 0x80000000u;      // (and past it with any row's offset)
    static constexpr int kB = sizeof(IO);
    uint32_t off, lo, hi;             // of loads (and 8-byte stores); of fp32's two stores
    __device__ __forceinline__ Cols(int c, int D) {
        off = c < D ? (uint32_t)c * kB : kNone;
        if constexpr (VEC == 4 && kB == 4) {
            // the lanes of a pair swap halves (see row_store)
            const uint32_t at = lane_id() & 1 ? c * 4 - 8 : c * 4;
            lo = at < (uint32_t)D * 4 ? at : kNone;
            hi = at + 16 < (uint32_t)D * 4 ? at + 16 : kNone;
        }
    }
    // as loaded; turned into floats where they are used
    struct Raw {
        uint32_t u[VEC == 1 ? 1 : kB];
        __device__ __forceinline__ void get(float (&x)[VEC]) const {
            if constexpr (VEC == 1) {
                x[0] = __uint_as_float(kB == 2 ? u[0] << 16 : u[0]);
            } else if constexpr (kB == 2) {
                x[0] = __uint_as_float(u[0] << 16);
                x[1] = __uint_as_float(u[0] & 0xffff0000u);
                x[2] = __uint_as_float(u[1] << 16);
                x[3] = __uint_as_float(u[1] & 0xffff0000u);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
            }
        }
    };
    __device__ __forceinline__ Raw load(rsrc_t r, uint32_t soff) const {
        Raw x;
        if constexpr (VEC == 1 && kB == 2) {
            x.u[0] = bload16(r, off, soff);
        } else if constexpr (VEC == 1) {
            x.u[0] = bload32(r, off, soff);
        } else if constexpr (kB == 2) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, off, soff, 0);
            x.u[0] = v[0];
            x.u[1] = v[1];
        } else {
            const u32x4 v = bload128(r, off, soff);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.u[i] = v[i];
        }
        return x;
    }
    __device__ __forceinline__ void store(rsrc_t r, uint32_t soff, const float (&x)[VEC]) const {
        if constexpr (VEC == 1) {
            BufElem<IO>::store(x[0], r, off, soff);
        } else if constexpr (kB == 2) {
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, r, off, soff, 0);
        } else {
            const bool odd = lane_id() & 1;
            const float r0 = swap_pair(odd ? x[0] : x[2]), r1 = swap_pair(odd ? x[1] : x[3]);
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(odd ? r0 : x[0]), __float_as_uint(odd ? r1 : x[1])}, r, lo, soff, 0);
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(odd ? x[2] : r0), __float_as_uint(odd ? x[3] : r1)}, r, hi, soff, 0);
        }
    }
};

template <typename IO>
__device__ __forceinline__ rsrc_t rows_at(const void *base, int64_t elems) {
    return make_rsrc((const IO *)base + elems, 0x80000000u);
}

// Position p of a sequence (p < 0: its initial state) into x.
template <typename IO, int VEC, int W>
__device__ __forceinline__ void load_pos(const ConvParams &p, int b, const Seq &q, int pos, int c, float (&x)[VEC]) {
    if (pos >= 0) {
        row_load<IO, VEC>(row_of<IO>(p.x, b * p.xb + (q.begin + pos) * p.xt, p.D), c, x);
    } else if (p.init) {
        row_load<IO, VEC>(row_of<IO>(p.init, ((int64_t)q.n * (W - 1) + W - 1 + pos) * p.D, p.D), c, x);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = 0.f;
    }
}

template <int VEC, int W>
__device__ __forceinline__ void taps(const float (&w)[W][VEC], const float (&b)[VEC], const float (&win)[W][VEC],
                                     float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        v[i] = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) v[i] += w[j][i] * win[j][i];
    }
}

constexpr int kConvRun = 32;         // tokens of a wave's run, forward
constexpr int kConvAhead = 8;        // rows loaded before the first is used
constexpr int kConvBwdRun = 32;      // tokens of a wave's run, backward

template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(256) conv_forward_kernel(ConvParams p) {
    const int wave = blockIdx.x * 4 + wave_id();
    const int col = wave % p.cols, job = wave / p.cols;
    const int c = (col * 64 + lane_id()) * VEC;
    if (job >= p.B * p.runs) {
        // the final state of one sequence
        const int n = job - p.B * p.runs;
        if (!p.final_ || n >= (p.cu ? p.n_seqs : p.B)) return;
        const Seq q = seq_at(p, n);
        const int len = q.end > q.begin ? q.end - q.begin : 0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float x[VEC];
            load_pos<IO, VEC, W>(p, p.cu ? 0 : n, q, len + i - (W - 1), c, x);
            row_store<IO, VEC>(row_of<IO>(p.final_, ((int64_t)n * (W - 1) + i) * p.D, p.D), c, x);
        }
        return;
    }
    const int b = job / p.runs, t0 = (job % p.runs) * kConvRun;
    const int t1 = t0 + kConvRun < p.T ? t0 + kConvRun : p.T;
    Filter<IO, VEC, W> f;
    f.load(p, c);
    Seq q = find_seq(p, b, t0);
    float win[W][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (t0 >= q.begin && t0 < q.end) load_pos<IO, VEC, W>(p, b, q, t0 - q.begin - (W - 1) + j, c, win[j + 1]);
        else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[j + 1][i] = 0.f;
        }
    }
    const Cols<IO, VEC> cols(c, p.D);
    const rsrc_t rx = rows_at<IO>(p.x, b * p.xb + t0 * p.xt), ry = rows_at<IO>(p.y, ((int64_t)b * p.T + t0) * p.D);
    const uint32_t sx = (uint32_t)p.xt * sizeof(IO), sy = (uint32_t)p.D * sizeof(IO);
    // (rows past the run's last are loaded again: no branch around a load)
    typename Cols<IO, VEC>::Raw in[kConvAhead], next[kConvAhead];
    auto fetch = [&](int ta) {
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) next[k] = cols.load(rx, ((ta + k < t1 ? ta + k : t1 - 1) - t0) * sx);
    };
    fetch(t0);
    for (int ta = t0; ta < t1; ta += kConvAhead) {
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) in[k] = next[k];
        if (ta + kConvAhead < t1) fetch(ta + kConvAhead);
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) {
            const int t = ta + k;
            if (t < t1) {
                if (p.cu && ((t >= q.end && q.n < p.n_seqs - 1) || (t == q.begin && t > t0))) {
                    q = find_seq(p, b, t);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        load_pos<IO, VEC, W>(p, b, q, t - q.begin - (W - 1) + j, c, win[j + 1]);
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) win[j][i] = win[j + 1][i];
                in[k].get(win[W - 1]);
                if (t >= q.begin && t < q.end) {
                    float v[VEC];
                    taps<VEC, W>(f.w, f.b, win, v);
                    if (p.silu) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[i] *= sigmoid(v[i]);
                    }
                    cols.store(ry, (t - t0) * sy, v);
                }
            }
        }
    }
}

template <int VEC, int W>
__device__ __forceinline__ void grad_of_v(const ConvParams &p, const float (&v)[VEC], float (&d)[VEC]) {
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float g = sigmoid(v[i]);
            d[i] *= g * (1.f + v[i] * (1.f - g));
        }
    }
}

// A run needs dv of its own tokens and of the W - 1 behind them; the sums
// over tokens take its own.  The sums of a workgroup's four runs meet in LDS.
template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(256) conv_backward_kernel(ConvParams p) {
    __shared__ float red[4][64][VEC * (W + 1) + 1];
    const int wave = wave_id();
    const int col = blockIdx.x % p.cols, part = blockIdx.x / p.cols;
    const int c = (col * 64 + lane_id()) * VEC;
    Filter<IO, VEC, W> f;
    f.load(p, c);
    if (part >= p.nparts) {
        // the initial state's gradient: one sequence a wave
        const int n = (part - p.nparts) * 4 + wave;
        if (!p.dinit || n >= (p.cu ? p.n_seqs : p.B)) return;
        const Seq q = seq_at(p, n);
        const int len = q.end > q.begin ? q.end - q.begin : 0, b = p.cu ? 0 : n;
        float di[W - 1][VEC];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) di[i][e] = 0.f;
            // a row that no token pushes out of the window is still there at the end
            if (p.dfinal && i >= len)
                row_load<IO, VEC>(row_of<IO>(p.dfinal, ((int64_t)n * (W - 1) + i - len) * p.D, p.D), c, di[i]);
        }
#pragma unroll
        for (int t = 0; t < W - 1; ++t)
            if (t < len) {
                float win[W][VEC], v[VEC], d[VEC];
#pragma unroll
                for (int j = 0; j < W; ++j) load_pos<IO, VEC, W>(p, b, q, t - (W - 1) + j, c, win[j]);
                taps<VEC, W>(f.w, f.b, win, v);
                row_load<IO, VEC>(row_of<IO>(p.dy, b * p.db_ + (q.begin + t) * p.dt_, p.D), c, d);
                grad_of_v<VEC, W>(p, v, d);
#pragma unroll
                for (int i = t; i < W - 1; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) di[i][e] += f.w[i - t][e] * d[e];
            }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            row_store<IO, VEC>(row_of<IO>(p.dinit, ((int64_t)n * (W - 1) + i) * p.D, p.D), c, di[i]);
        return;
    }
    float dw[W][VEC], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    const Cols<IO, VEC> cols(c, p.D);
    // runs go to the workgroups' waves in turn
    for (int64_t job = part * 4 + wave; job < (int64_t)p.B * p.runs; job += p.nparts * 4) {
        const int b = (int)(job / p.runs), t0 = (int)(job % p.runs) * kConvBwdRun;
        const int t1 = t0 + kConvBwdRun < p.T ? t0 + kConvBwdRun : p.T;
        Seq q = find_seq(p, b, t0);
        float win[W][VEC], acc[W][VEC];       // acc[k]: the gradient so far of x at token t - k
        auto start = [&](int t) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                if (t >= q.begin && t < q.end) load_pos<IO, VEC, W>(p, b, q, t - q.begin - (W - 1) + j, c, win[j + 1]);
                else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) win[j + 1][i] = 0.f;
                }
            }
        };
        start(t0);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[k][i] = 0.f;
        const rsrc_t rx = rows_at<IO>(p.x, b * p.xb + t0 * p.xt), rd = rows_at<IO>(p.dy, b * p.db_ + t0 * p.dt_),
                     ro = rows_at<IO>(p.dx, ((int64_t)b * p.T + t0) * p.D);
        const uint32_t sx = (uint32_t)p.xt * sizeof(IO), sd = (uint32_t)p.dt_ * sizeof(IO), so = (uint32_t)p.D * sizeof(IO);
        const int te = t1 + W - 1;            // dx of token t - (W - 1) goes out at step t
        constexpr int kAhead = 4;
        typename Cols<IO, VEC>::Raw xin[kAhead], din[kAhead], xnext[kAhead], dnext[kAhead];
        auto fetch = [&](int ta) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int row = (ta + k < p.T ? ta + k : p.T - 1) - t0;
                xnext[k] = cols.load(rx, row * sx);
                dnext[k] = cols.load(rd, row * sd);
            }
        };
        fetch(t0);
        for (int ta = t0; ta < te; ta += kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                xin[k] = xnext[k];
                din[k] = dnext[k];
            }
            if (ta + kAhead < te) fetch(ta + kAhead);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int t = ta + k;
                if (t < te) {
                    // gradients move one place back
#pragma unroll
                    for (int m = W - 1; m > 0; --m)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) acc[m][i] = acc[m - 1][i];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[0][i] = 0.f;
                    if (t < p.T) {
                        if (p.cu && ((t >= q.end && q.n < p.n_seqs - 1) || (t == q.begin && t > t0))) {
                            q = find_seq(p, b, t);
                            start(t);
                        }
#pragma unroll
                        for (int j = 0; j < W - 1; ++j)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) win[j][i] = win[j + 1][i];
                        xin[k].get(win[W - 1]);
                        if (t >= q.begin && t < q.end) {
                            float v[VEC], d[VEC];
                            taps<VEC, W>(f.w, f.b, win, v);
                            din[k].get(d);
                            grad_of_v<VEC, W>(p, v, d);
                            // token t - m takes it through tap W - 1 - m, if it
                            // is of this sequence
#pragma unroll
                            for (int m = 0; m < W; ++m)
                                if (t - m >= q.begin) {
#pragma unroll
                                    for (int i = 0; i < VEC; ++i) acc[m][i] += f.w[W - 1 - m][i] * d[i];
                                }
                            if (t < t1) {
#pragma unroll
                                for (int i = 0; i < VEC; ++i) {
                                    db[i] += d[i];
#pragma unroll
                                    for (int j = 0; j < W; ++j) dw[j][i] += d[i] * win[j][i];
                                }
                            }
                            // the final state holds the last W - 1 inputs
                            if (p.dfinal && t + W - 1 >= q.end) {
                                float g[VEC];
                                row_load<IO, VEC>(row_of<IO>(p.dfinal, ((int64_t)q.n * (W - 1) + t - q.end + W - 1) * p.D, p.D), c, g);
#pragma unroll
                                for (int i = 0; i < VEC; ++i) acc[0][i] += g[i];
                            }
                        }
                    }
                    if (t - (W - 1) >= t0)
                        cols.store(ro, (t - (W - 1) - t0) * so, acc[W - 1]);
                }
            }
        }
    }
    // [W + 1][D] sums of this workgroup: wave 0 adds the four runs up
    float *mine = red[wave][lane_id()];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        mine[W * VEC + i] = db[i];
#pragma unroll
        for (int j = 0; j < W; ++j) mine[j * VEC + i] = dw[j][i];
    }
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float a[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            a[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) a[i] += red[k][lane_id()][j * VEC + i];
        }
        row_store<float, VEC>(make_rsrc(p.part + ((int64_t)part * (W + 1) + j) * p.D, (uint32_t)p.D * 4), c, a);
    }
}

// dw[c][j] and db[c] (j = W) from the workgroups' sums: 64 channels and one j
// a workgroup.
template <int W>
__global__ void __launch_bounds__(1024) conv_dw_kernel(ConvParams p) {
    __shared__ float red[16][64];
    const int nc = (p.D + 63) / 64, j = blockIdx.x / nc, c = (blockIdx.x % nc) * 64 + lane_id(), w = wave_id();
    float a = 0.f;
    if (c < p.D)
        for (int i = w; i < p.nparts; i += 16) a += p.part[((int64_t)i * (W + 1) + j) * p.D + c];
    red[w][lane_id()] = a;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) a += red[i][lane_id()];
    if (j < W)
        p.dw[(int64_t)c * W + j] = a;
    else if (p.db)
        p.db[c] = a;
}

// Whether row b has slot s to itself or is the first to name it.
__device__ __forceinline__ bool first_with_slot(const int32_t *slots, int b, int s) {
    bool seen = false;
    for (int i = 0; i < b; i += 64) {
        const int k = i + lane_id();
        seen |= k < b && slots[k] == s;
    }
    return __ballot(seen) == 0;
}

template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(64) conv_step_kernel(ConvParams p) {
    const int col = blockIdx.x % p.cols, b = blockIdx.x / p.cols;
    const int c = (col * 64 + lane_id()) * VEC;
    const int64_t s = p.slots ? p.slots[b] : b;
    const rsrc_t ry = row_of<IO>(p.y, (int64_t)b * p.D, p.D);
    float v[VEC];
    if (s < 0 || s >= p.n_slots || (p.slots && !first_with_slot(p.slots, b, (int)s))) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
        row_store<IO, VEC>(ry, c, v);
        return;
    }
    Filter<IO, VEC, W> f;
    f.load(p, c);
    float win[W][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row_load<IO, VEC>(row_of<IO>(p.state, (s * (W - 1) + j) * p.D, p.D), c, win[j]);
    row_load<IO, VEC>(row_of<IO>(p.x, b * p.xb, p.D), c, win[W - 1]);
    taps<VEC, W>(f.w, f.b, win, v);
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] *= sigmoid(v[i]);
    }
    row_store<IO, VEC>(ry, c, v);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        row_store<IO, VEC>(row_of<IO>(p.state, (s * (W - 1) + j) * p.D, p.D), c, win[j + 1]);
}

namespace {

gdn_status check_conv(const gdn_conv_problem *pr, bool packed) {
    if (!pr) return GDN_ERR_NULL_ARG;
    if (pr->B < 1 || pr->T < 0 || pr->D < 1 || pr->W < 1) return GDN_ERR_BAD_SHAPE;
    if (packed && (pr->B != 1 || pr->n_seqs < 1 || pr->n_seqs > (1 << 24))) return GDN_ERR_BAD_SHAPE;
    if (!io_dtype_ok(pr->io_dtype) || (pr->w_dtype != pr->io_dtype && pr->w_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (pr->W < 2 || pr->W > 4) return GDN_ERR_UNSUPPORTED;
    // wave numbers and byte offsets within a row stay in 32 bits
    if (pr->T > (1 << 30) || pr->B > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    // a run's rows are addressed with 32-bit byte offsets
    for (int64_t v : {pr->x_stride_t, pr->dy_stride_t})
        if (v < 0 || v > (1 << 23)) return GDN_ERR_UNSUPPORTED;
    if (pr->D > (1 << 23)) return GDN_ERR_UNSUPPORTED;
    const int64_t jobs = pr->B * ((pr->T + 31) / 32) + (packed ? pr->n_seqs : pr->B);
    if (!grid_ok(jobs, (pr->D + 63) / 64 * 64)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

void fill_conv(const gdn_conv_problem *pr, ConvParams &cp, const int32_t *cu) {
    cp = ConvParams{};
    cp.cu = cu;
    cp.xb = pr->x_stride_b;
    cp.xt = pr->x_stride_t;
    cp.db_ = pr->dy_stride_b;
    cp.dt_ = pr->dy_stride_t;
    cp.B = (int)pr->B;
    cp.T = (int)pr->T;
    cp.D = (int)pr->D;
    cp.n_seqs = cu ? (int)pr->n_seqs : 0;
    cp.w_f32 = pr->w_dtype == GDN_F32;
    cp.silu = pr->silu != 0;
}

int conv_cols(int D, bool vec) { return (D + (vec ? 256 : 64) - 1) / (vec ? 256 : 64); }

// Workgroups of the backward pass that share a column of 64 lanes: up to
// four waves of runs each, about 2048 workgroups in all.
int conv_parts(const gdn_conv_problem *pr) {
    const int64_t runs = pr->B * ((pr->T + kConvBwdRun - 1) / kConvBwdRun), most = (runs + 3) / 4;
    int64_t n = 2048 / ((pr->D + 255) / 256);
    n = n < 8 ? 8 : n;
    return (int)(n < most ? n : most);
}

template <typename IO, int VEC, int W>
struct ConvFns {
    static const void *get(int which) {
        return which == 0   ? (const void *)&conv_forward_kernel<IO, VEC, W>
               : which == 1 ? (const void *)&conv_backward_kernel<IO, VEC, W>
                            : (const void *)&conv_step_kernel<IO, VEC, W>;
    }
};
template <typename IO, int VEC>
const void *conv_w(int which, int W) {
    return W == 2 ? ConvFns<IO, VEC, 2>::get(which) : W == 3 ? ConvFns<IO, VEC, 3>::get(which) : ConvFns<IO, VEC, 4>::get(which);
}
const void *conv_fn(const gdn_conv_problem *pr, int which, bool vec) {
    if (pr->io_dtype == GDN_F32) return vec ? conv_w<float, 4>(which, (int)pr->W) : conv_w<float, 1>(which, (int)pr->W);
    return vec ? conv_w<bf16_t, 4>(which, (int)pr->W) : conv_w<bf16_t, 1>(which, (int)pr->W);
}

// Whether every row and vector begins at four aligned elements.
bool conv_vec(const gdn_conv_problem *pr, std::initializer_list<const void *> io, const void *weight, const void *bias) {
    const size_t eb = dtype_bytes(pr->io_dtype), wb = dtype_bytes(pr->w_dtype);
    if (pr->D % 4 != 0 || !aligned_to(weight, 4 * wb) || !aligned_to(bias, 4 * wb)) return false;
    for (const void *q : io)
        if (!aligned_to(q, 4 * eb)) return false;
    return true;
}

bool conv_aligned(const gdn_conv_problem *pr, std::initializer_list<const void *> io, std::initializer_list<const void *> w) {
    for (const void *q : io)
        if (!aligned_to(q, dtype_bytes(pr->io_dtype))) return false;
    for (const void *q : w)
        if (!aligned_to(q, dtype_bytes(pr->w_dtype))) return false;
    return true;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_conv_forward(const gdn_conv_problem *pr, const void *x, const void *weight, const void *bias,
                            const void *initial_state, const int32_t *cu_seqlens, void *y, void *final_state,
                            void *stream) {
    const gdn_status st = check_conv(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!weight || (pr->T > 0 && (!x || !y))) return GDN_ERR_NULL_ARG;
    if (!conv_aligned(pr, {x, y, initial_state, final_state}, {weight, bias}) || !aligned_to(cu_seqlens, 4))
        return GDN_ERR_ALIGNMENT;
    ConvParams cp;
    fill_conv(pr, cp, cu_seqlens);
    cp.x = x;
    cp.w = weight;
    cp.bias = bias;
    cp.init = initial_state;
    cp.y = y;
    cp.final_ = final_state;
    cp.runs = (int)((pr->T + kConvRun - 1) / kConvRun);
    const bool vec = conv_vec(pr, {x, y, initial_state, final_state}, weight, bias) && pr->x_stride_b % 4 == 0 && pr->x_stride_t % 4 == 0;
    cp.cols = conv_cols(cp.D, vec);
    const int64_t jobs = (int64_t)cp.B * cp.runs + (final_state ? (cu_seqlens ? pr->n_seqs : pr->B) : 0);
    return launch_kernel(conv_fn(pr, 0, vec), (int)((jobs * cp.cols + 3) / 4), &cp, (hipStream_t)stream);
}

size_t gdn_workspace_bytes_conv_backward(const gdn_conv_problem *pr) {
    if (check_conv(pr, pr && pr->n_seqs > 0) != GDN_OK) return 0;
    return (size_t)conv_parts(pr) * (pr->W + 1) * pr->D * 4;
}

gdn_status gdn_conv_backward(const gdn_conv_problem *pr, const void *dy, const void *x, const void *weight,
                             const void *bias, const void *initial_state, const int32_t *cu_seqlens,
                             const void *dfinal, void *dx, float *dweight, float *dbias, void *dinitial,
                             void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_conv(pr, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!weight || !dweight || (pr->T > 0 && (!dy || !x || !dx))) return GDN_ERR_NULL_ARG;
    if (!conv_aligned(pr, {dy, x, initial_state, dfinal, dx, dinitial}, {weight, bias}) || !aligned_to(cu_seqlens, 4) ||
        !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return GDN_ERR_ALIGNMENT;
    ConvParams cp;
    fill_conv(pr, cp, cu_seqlens);
    cp.nparts = conv_parts(pr);
    const size_t need = (size_t)cp.nparts * (pr->W + 1) * pr->D * 4;
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GDN_ERR_ALIGNMENT;
    cp.dy = dy;
    cp.x = x;
    cp.w = weight;
    cp.bias = bias;
    cp.init = initial_state;
    cp.dfinal = dfinal;
    cp.dx = dx;
    cp.dw = dweight;
    cp.db = dbias;
    cp.dinit = dinitial;
    cp.part = (float *)workspace;
    cp.runs = (int)((pr->T + kConvBwdRun - 1) / kConvBwdRun);
    const bool vec = conv_vec(pr, {dy, x, initial_state, dfinal, dx, dinitial}, weight, bias) && pr->x_stride_b % 4 == 0 &&
                     pr->x_stride_t % 4 == 0 && pr->dy_stride_b % 4 == 0 && pr->dy_stride_t % 4 == 0;
    cp.cols = conv_cols(cp.D, vec);
    const int64_t extra = dinitial ? ((cu_seqlens ? pr->n_seqs : pr->B) + 3) / 4 : 0;
    st = launch_kernel(conv_fn(pr, 1, vec), (int)((cp.nparts + extra) * cp.cols), &cp, (hipStream_t)stream);
    if (st != GDN_OK) return st;
    const void *fn = pr->W == 2   ? (const void *)&conv_dw_kernel<2>
                     : pr->W == 3 ? (const void *)&conv_dw_kernel<3>
                                  : (const void *)&conv_dw_kernel<4>;
    return launch_kernel(fn, (int)((pr->D + 63) / 64 * (pr->W + 1)), &cp, (hipStream_t)stream, 1024);
}

gdn_status gdn_conv_step(const gdn_conv_problem *pr, const void *x, const void *weight, const void *bias, void *state,
                         const int32_t *slots, int64_t n_slots, void *y, void *stream) {
    const gdn_status st = check_conv(pr, false);
    if (st != GDN_OK) return st;
    if (pr->T != 1 || n_slots < 0 || n_slots >= ((int64_t)1 << 31) || (!slots && n_slots < pr->B)) return GDN_ERR_BAD_SHAPE;
    if (!x || !weight || !y || (!state && n_slots > 0)) return GDN_ERR_NULL_ARG;
    if (!conv_aligned(pr, {x, y, state}, {weight, bias}) || !aligned_to(slots, 4)) return GDN_ERR_ALIGNMENT;
    ConvParams cp;
    fill_conv(pr, cp, nullptr);
    cp.x = x;
    cp.w = weight;
    cp.bias = bias;
    cp.state = state;
    cp.slots = slots;
    cp.n_slots = n_slots;
    cp.y = y;
    const bool vec = conv_vec(pr, {x, y, state}, weight, bias) && pr->x_stride_b % 4 == 0;
    cp.cols = conv_cols(cp.D, vec);
    return launch_kernel(conv_fn(pr, 2, vec), (int)(pr->B * cp.cols), &cp, (hipStream_t)stream, 64);
}

}  // extern "C"

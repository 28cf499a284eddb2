// norm.cu — the norms around a block: before it (moe_norm_forward) and after it,
// fused with the block's gate, the residual add and its scales and with the next
// block's norm (moe_norm_residual_forward), and their gradients.
//
//   xhat = (x - mean) rstd (layer norm) or x rstd (RMS),  N(x) = xhat (w + o) + b
//   before:  y = N(x)
//   after:   out = alpha r + beta gate N(y);   x_next = N2(out), out as it is stored
//
// Backward, with G the gradient of xhat, c(G) = mean(G) for layer norm, else 0:
//   d x = rstd (G - c(G) - xhat mean(G xhat))   [+ the residual stream's gradient]
//   d w = sum_t D xhat, d b = sum_t D, with D the gradient of N's result
//   after: D = beta gate dout, d r = alpha dout, d gate = beta sum dout N(y)
//
// All of it is bound by HBM: each row is read once into registers, the sums are
// taken there (fp32; the variance in a second pass over the registers, so a large
// mean costs no digits) and the results are written once. A row belongs to 1 to 8
// warps, so that a thread holds as few of its elements as the length allows: the
// loads of a block's rows are then spread over many threads and several blocks
// share an SM, which hides the two reductions of a row behind the others' loads.
// The weights' gradients are sums over rows: each group of warps keeps its
// columns' partial sums in registers over all its rows and writes them once;
// a second kernel adds the groups' sums in a fixed order, so that a call's result
// does not change from run to run (no atomics).
#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct NormArgs {
    const void* x;       // pre: x (stream dtype); post: the block's output (block dtype)
    const void* resid;   // post
    const void* weight;
    const void* bias;
    const void* gate;
    const void* next_weight;
    const void* next_bias;
    void* y;             // pre: y; post: x_next (block dtype)
    void* out;           // post: stream dtype
    uint8_t* q8;         // y (pre) or x_next (post) in e4m3
    float* s8;           // [ceil(d/128), T]
    float* mean;
    float* rstd;
    float* next_mean;
    float* next_rstd;
    int64_t ld_stream, ld_block;
    int T, d, kind, next_kind, stream_dt, block_dt, param_dt, gate_kind;
    float eps, offset, alpha, beta;
};

// Sum of a value over the wpr warps of a row; every thread of the block calls it.
MOE_DEV float row_sum(float v, int wpr, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (wpr == 1) return v;
    const int warp = threadIdx.x >> 5, g0 = warp / wpr * wpr;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < wpr; ++i) s += buf[g0 + i];
    return s;
}

// Mean and 1/sqrt(var + eps) of the row in v; buf: 16 floats of the block.
template <int NV, bool VEC>
MOE_DEV void row_stats(const float (&v)[NV][8], int kind, int d, float eps, int wpr, int th, int t, float* buf,
                       float& mean, float& rstd) {
    mean = 0.f;
    if (kind == MOE_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        mean = row_sum(s, wpr, buf) / float(d);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = in_row<VEC>(i, j, d, th, t) ? v[i][j] - mean : 0.f;
            s = fmaf(c, c, s);
        }
    rstd = 1.0f / sqrtf(row_sum(s, wpr, buf + 8) / float(d) + eps);
}

// v <- (v - mean) rstd (w + o) + b
template <int NV, bool VEC>
MOE_DEV void apply_norm(float (&v)[NV][8], float mean, float rstd, const void* w, const void* b, float offset,
                        int param_dt, int d, int th, int t) {
    float p[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] - mean) * rstd;
    if (w) {
        load_row<NV, VEC>(p, w, d, param_dt, th, t);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= p[i][j] + offset;
    }
    if (b) {
        load_row<NV, VEC>(p, b, d, param_dt, th, t);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += p[i][j];
    }
}

MOE_DEV char* at_row(const void* p, int64_t row, int64_t ld, int dt) {
    return static_cast<char*>(const_cast<void*>(p)) + row * ld * (dt == MOE_DT_F32 ? 4 : 2);
}

template <int NV, bool VEC, bool POST>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormArgs a, int wpr) {
    __shared__ float buf[2][16];
    griddep_wait();
    griddep_launch();
    const int th = wpr * 32, t = threadIdx.x % th, rpb = kThreads / th;
    const int d = a.d;
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < a.T; r0 += int64_t(gridDim.x) * rpb) {
        // rows past T take part in the block's reductions and store nothing
        const int64_t r = r0 + threadIdx.x / th;
        const bool live = r < a.T;
        const int dl = live ? d : 0;
        float v[NV][8];
        load_row<NV, VEC>(v, at_row(a.x, live ? r : 0, POST ? a.ld_block : a.ld_stream, POST ? a.block_dt : a.stream_dt),
                          dl, POST ? a.block_dt : a.stream_dt, th, t);
        float res[POST ? NV : 1][8];
        if constexpr (POST)
            load_row<NV, VEC>(res, at_row(a.resid, live ? r : 0, a.ld_stream, a.stream_dt), dl, a.stream_dt, th, t);
        if (a.kind != MOE_NORM_NONE) {
            float mean, rstd;
            row_stats<NV, VEC>(v, a.kind, d, a.eps, wpr, th, t, buf[0], mean, rstd);
            if (live && t == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
            apply_norm<NV, VEC>(v, mean, rstd, a.weight, a.bias, a.offset, a.param_dt, d, th, t);
        }
        if constexpr (POST) {
            float gt = a.beta;
            if (a.gate_kind == MOE_GATE_TOKEN) gt *= live ? load_elem(a.gate, r, a.param_dt) : 0.f;
            if (a.gate_kind == MOE_GATE_CHANNEL) {
                float p[NV][8];
                load_row<NV, VEC>(p, a.gate, d, a.param_dt, th, t);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] *= p[i][j];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = round_to(fmaf(a.alpha, res[i][j], gt * v[i][j]), a.stream_dt);
            if (live) store_row<NV, VEC>(v, at_row(a.out, r, a.ld_stream, a.stream_dt), d, a.stream_dt, th, t);
            if (a.next_kind != MOE_NORM_NONE) {
                float mean, rstd;
                row_stats<NV, VEC>(v, a.next_kind, d, a.eps, wpr, th, t, buf[1], mean, rstd);
                if (live && t == 0) {
                    if (a.next_mean) a.next_mean[r] = mean;
                    if (a.next_rstd) a.next_rstd[r] = rstd;
                }
                apply_norm<NV, VEC>(v, mean, rstd, a.next_weight, a.next_bias, a.offset, a.param_dt, d, th, t);
            }
        }
        if (a.y && live) store_row<NV, VEC>(v, at_row(a.y, r, a.ld_block, a.block_dt), d, a.block_dt, th, t);
        if constexpr (VEC) {
            if (a.q8) store_row_e4m3<NV>(v, a.q8 + (live ? r : 0) * d, a.s8 + (live ? r : 0), a.T, dl, th, t);
        }
        if (wpr > 1) __syncthreads();  // the block's sums are read before the next rows write theirs
    }
}

struct NormBwdArgs {
    const void* x;      // pre: x (stream dtype); post: the block's output (block dtype)
    const void* dy;     // pre: dy (block dtype); post: dout (stream dtype)
    const void* dres;   // pre: the residual stream's gradient to add (stream dtype), or null
    const void* weight;
    const void* bias;
    const void* gate;
    const float* mean;
    const float* rstd;
    void* dx;           // as x
    void* dresid;       // post: alpha dout (stream dtype), or null
    float* dgate_tok;   // post, gate per token: [T], or null
    float* s1;          // [groups, d] sums of rs D xhat, or null
    float* s0;          // [groups, d] sums of rs D, or null
    int64_t ld_x, ld_dy;
    int T, d, kind, x_dt, dy_dt, param_dt, gate_kind;
    float offset, alpha, beta;
};

template <int NV, bool VEC, bool POST>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormBwdArgs a, int wpr) {
    __shared__ float buf[24];
    griddep_wait();
    griddep_launch();
    const int th = wpr * 32, t = threadIdx.x % th, rpb = kThreads / th;
    const int d = a.d;
    const float inv_d = 1.0f / float(d);
    float s1[NV][8], s0[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[i][j] = s0[i][j] = 0.f;
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < a.T; r0 += int64_t(gridDim.x) * rpb) {
        const int64_t r = r0 + threadIdx.x / th;
        const bool live = r < a.T;
        const int dl = live ? d : 0;
        float x[NV][8], g[NV][8], p[NV][8];
        load_row<NV, VEC>(x, at_row(a.x, live ? r : 0, a.ld_x, a.x_dt), dl, a.x_dt, th, t);
        load_row<NV, VEC>(g, at_row(a.dy, live ? r : 0, a.ld_dy, a.dy_dt), dl, a.dy_dt, th, t);
        const float mean = live && a.kind == MOE_NORM_LAYER ? a.mean[r] : 0.f;
        const float rstd = live && a.kind != MOE_NORM_NONE ? a.rstd[r] : 1.f;
        float rs = 1.f;
        if (POST) {
            rs = a.beta;
            if (a.gate_kind == MOE_GATE_TOKEN) rs *= live ? load_elem(a.gate, r, a.param_dt) : 0.f;
            if (a.dresid && live) {
                float q[NV][8];
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[i][j] = a.alpha * g[i][j];
                store_row<NV, VEC>(q, at_row(a.dresid, r, a.ld_dy, a.dy_dt), d, a.dy_dt, th, t);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = in_row<VEC>(i, j, dl, th, t) ? (x[i][j] - mean) * rstd : 0.f;
                s1[i][j] = fmaf(rs * g[i][j], x[i][j], s1[i][j]);
                s0[i][j] = fmaf(rs, g[i][j], s0[i][j]);
            }
        // g <- the gradient of xhat without the row's factor rs; the token gate's gradient on the way
        float dot_n = 0.f;
        if (a.weight) {
            load_row<NV, VEC>(p, a.weight, d, a.param_dt, th, t);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) p[i][j] = in_row<VEC>(i, j, d, th, t) ? p[i][j] + a.offset : 0.f;
        }
        if (POST && a.dgate_tok) {
            if (a.bias) {
                float q[NV][8];
                load_row<NV, VEC>(q, a.bias, d, a.param_dt, th, t);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot_n = fmaf(g[i][j], q[i][j], dot_n);
            }
        }
        if (a.weight) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] *= p[i][j];
        }
        if (POST && a.dgate_tok) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) dot_n = fmaf(g[i][j], x[i][j], dot_n);
            dot_n = row_sum(dot_n, wpr, buf + 16);
            if (live && t == 0) a.dgate_tok[r] = a.beta * dot_n;
        }
        if (POST && a.gate_kind == MOE_GATE_CHANNEL) {
            load_row<NV, VEC>(p, a.gate, d, a.param_dt, th, t);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] *= p[i][j];
        }
        if (a.kind != MOE_NORM_NONE) {
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sa = fmaf(g[i][j], x[i][j], sa);
                    sb += g[i][j];
                }
            sa = row_sum(sa, wpr, buf) * inv_d;
            sb = a.kind == MOE_NORM_LAYER ? row_sum(sb, wpr, buf + 8) * inv_d : 0.f;
            const float f = rs * rstd;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] = f * (g[i][j] - sb - x[i][j] * sa);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] *= rs;
        }
        if (!POST && a.dres) {
            load_row<NV, VEC>(p, at_row(a.dres, live ? r : 0, a.ld_x, a.x_dt), dl, a.x_dt, th, t);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] += p[i][j];
        }
        if (live) store_row<NV, VEC>(g, at_row(a.dx, r, a.ld_x, a.x_dt), d, a.x_dt, th, t);
        if (wpr > 1) __syncthreads();
    }
    const int64_t grp = int64_t(blockIdx.x) * rpb + threadIdx.x / th;
    if (a.s1) store_row<NV, VEC>(s1, a.s1 + grp * d, d, MOE_DT_F32, th, t);
    if (a.s0) store_row<NV, VEC>(s0, a.s0 + grp * d, d, MOE_DT_F32, th, t);
}

// The groups' partial sums added in order: block of 32 columns x 32 strips of groups,
// then the strips. dw = gate S1, db = gate S0, dgate = (w + o) S1 + b S0 (gate per
// channel; else gate = 1 here, the token's gate and beta being in the sums).
struct NormSumArgs {
    const float* s1;
    const float* s0;
    const void* weight;
    const void* bias;
    const void* gate;  // per channel, or null
    float* dw;
    float* db;
    float* dgate;
    int groups, d, param_dt;
    float offset;
};

__global__ void __launch_bounds__(1024) norm_sum_kernel(const NormSumArgs a) {
    __shared__ float sm[2][32][33];
    griddep_wait();
    griddep_launch();
    const int cx = threadIdx.x & 31, sy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float v1 = 0.f, v0 = 0.f;
    if (c < a.d) {
#pragma unroll 4
        for (int g = sy; g < a.groups; g += 32) {
            if (a.s1) v1 += a.s1[int64_t(g) * a.d + c];
            if (a.s0) v0 += a.s0[int64_t(g) * a.d + c];
        }
    }
    sm[0][sy][cx] = v1;
    sm[1][sy][cx] = v0;
    __syncthreads();
    // warp y adds the 32 strips of column y
    float w1 = sm[0][cx][sy], w0 = sm[1][cx][sy];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        w1 += __shfl_xor_sync(0xFFFFFFFFu, w1, o);
        w0 += __shfl_xor_sync(0xFFFFFFFFu, w0, o);
    }
    const int col = blockIdx.x * 32 + sy;
    if (cx == 0 && col < a.d) {
        const float gate = a.gate ? load_elem(a.gate, col, a.param_dt) : 1.f;
        if (a.dw) a.dw[col] = gate * w1;
        if (a.db) a.db[col] = gate * w0;
        if (a.dgate) {
            const float w = a.weight ? load_elem(a.weight, col, a.param_dt) + a.offset : 1.f;
            a.dgate[col] = w * w1 + (a.bias ? load_elem(a.bias, col, a.param_dt) * w0 : 0.f);
        }
    }
}

// Warps per row and groups of 8 per thread: as many warps as give each thread one
// group, up to the block's 8.
void shape_of(int d, int* wpr, int* nv) {
    const int v = (d + 7) / 8;
    int w = 1;
    while (w < kThreads / 32 && w * 32 < v) w *= 2;
    *wpr = w;
    int n = 1;
    while (n * w * 32 < v) n *= 2;
    *nv = n;
}
static_assert(MOE_NORM_MAX_D <= 4 * 8 * kThreads, "a row fits four groups of 8 a thread");

constexpr int kFwdBlocksPerSm = 8;
// Backward blocks: the groups' partial sums are written and read once more, so few
// enough that they stay small beside the rows.
constexpr int kBwdBlocksPerSm = 4;

int grid_of(int T, int wpr, int per_sm) {
    const int rpb = kThreads / (32 * wpr);
    const int64_t blocks = (int64_t(T) + rpb - 1) / rpb;
    return int(std::min<int64_t>(blocks, int64_t(num_sms()) * per_sm));
}

size_t esize(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// 16-byte vectors on every row: the row's length and stride and the base.
bool rows_vec(const void* p, int d, int64_t ld, int dt) {
    return !p || (d % 8 == 0 && (ld * int64_t(esize(dt))) % 16 == 0 && aligned(p, 16));
}

int check_params(const moe_norm_params* p) {
    if (!p) return MOE_ERR_INVALID_ARG;
    if (p->T < 0 || p->d < 1) return MOE_ERR_INVALID_ARG;
    if (p->d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
    for (int k : {p->kind, p->next_kind})
        if (k < MOE_NORM_NONE || k > MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
    for (int dt : {p->stream_dtype, p->block_dtype, p->param_dtype})
        if (dt < MOE_DT_F32 || dt > MOE_DT_F16) return MOE_ERR_INVALID_ARG;
    if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !(p->eps <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    for (float f : {p->weight_offset, p->alpha, p->beta})
        if (!(f >= -3.4e38f && f <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if ((p->ld_stream != 0 && p->ld_stream < p->d) || (p->ld_block != 0 && p->ld_block < p->d))
        return MOE_ERR_INVALID_ARG;
    if (p->ld_stream > (int64_t(1) << 31) || p->ld_block > (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int64_t ld_of(int64_t ld, int d) { return ld ? ld : d; }

bool elem_aligned(const void* p, int dt) { return aligned(p, esize(dt)); }

template <bool POST, bool VEC>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    int wpr, nv;
    shape_of(a.d, &wpr, &nv);
    const int grid = grid_of(a.T, wpr, kFwdBlocksPerSm);
    ProfScope prof_(MOE_K_NORM, s);
    const bool pdl = use_pdl(a.T);
    switch (nv) {
        case 1: return launch_pdl(pdl, norm_forward_kernel<1, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
        case 2: return launch_pdl(pdl, norm_forward_kernel<2, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
        default: return launch_pdl(pdl, norm_forward_kernel<4, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
    }
}

template <bool POST, bool VEC>
cudaError_t launch_bwd(const NormBwdArgs& a, int grid, int wpr, int nv, cudaStream_t s) {
    ProfScope prof_(MOE_K_NORM_BWD, s);
    const bool pdl = use_pdl(a.T);
    switch (nv) {
        case 1: return launch_pdl(pdl, norm_backward_kernel<1, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
        case 2: return launch_pdl(pdl, norm_backward_kernel<2, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
        default: return launch_pdl(pdl, norm_backward_kernel<4, VEC, POST>, dim3(grid), dim3(kThreads), 0, s, a, wpr);
    }
}

size_t norm_ws_bytes(const moe_norm_params* p) {
    int wpr, nv;
    shape_of(p->d, &wpr, &nv);
    const int64_t groups = int64_t(grid_of(std::max(1, p->T), wpr, kBwdBlocksPerSm)) * (kThreads / (32 * wpr));
    const size_t one = (size_t(groups) * p->d * 4 + 255) & ~size_t(255);
    return 256 + 2 * one;
}

int check_f8_rows(const uint8_t* q8, const float* s8, int d, bool vec) {
    if (!q8 != !s8) return MOE_ERR_INVALID_ARG;
    if (!q8) return MOE_OK;
    if (d % 16) return MOE_ERR_INVALID_ARG;
    return vec && aligned(q8, 16) && aligned(s8, 4) ? MOE_OK : MOE_ERR_MISALIGNED;
}

template <bool POST>
int run_backward(const moe_norm_params* p, NormBwdArgs a, const moe_norm_grads& g, void* ws, size_t ws_bytes,
                 cudaStream_t stream, bool vec) {
    int wpr, nv;
    shape_of(p->d, &wpr, &nv);
    const int grid = grid_of(p->T, wpr, kBwdBlocksPerSm);
    const int groups = grid * (kThreads / (32 * wpr));
    const bool gate_c = POST && p->gate_kind == MOE_GATE_CHANNEL;
    const bool need1 = g.dweight || (gate_c && g.dgate);
    const bool need0 = g.dbias || (gate_c && g.dgate && a.bias);
    if (need1 || need0) {
        if (!ws) return MOE_ERR_INVALID_ARG;
        if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
        if (ws_bytes < norm_ws_bytes(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        const size_t one = (size_t(groups) * p->d * 4 + 255) & ~size_t(255);
        uint8_t* w = static_cast<uint8_t*>(ws) + 256;
        if (need1) a.s1 = reinterpret_cast<float*>(w);
        if (need0) a.s0 = reinterpret_cast<float*>(w + one);
    }
    a.dgate_tok = POST && p->gate_kind == MOE_GATE_TOKEN ? g.dgate : nullptr;
    if ((vec ? launch_bwd<POST, true>(a, grid, wpr, nv, stream) : launch_bwd<POST, false>(a, grid, wpr, nv, stream)) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    if (need1 || need0) {
        const NormSumArgs sa{a.s1, a.s0, a.weight, a.bias, gate_c ? a.gate : nullptr, g.dweight, g.dbias,
                             gate_c ? g.dgate : nullptr, groups, p->d, p->param_dtype, p->weight_offset};
        ProfScope prof_(MOE_K_NORM_BWD, stream);
        if (launch_pdl(use_pdl(p->T), norm_sum_kernel, dim3((p->d + 31) / 32), dim3(1024), 0, stream, sa) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// An empty batch's sums over tokens are zero.
int zero_sums(const moe_norm_params* p, const moe_norm_grads& g, cudaStream_t stream) {
    for (float* v : {g.dweight, g.dbias, p->gate_kind == MOE_GATE_CHANNEL ? g.dgate : nullptr})
        if (v && cudaMemsetAsync(v, 0, size_t(p->d) * 4, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_size(const moe_norm_params* p) {
    return check_params(p) == MOE_OK ? norm_ws_bytes(p) : 0;
}

int moe_norm_forward(const moe_norm_params* p, const void* x, const void* weight, const void* bias, void* y,
                     uint8_t* q8, float* s8, float* mean, float* rstd, moe_stream_t stream) {
    int st = check_params(p);
    if (st != MOE_OK) return st;
    if (p->kind == MOE_NORM_NONE || p->next_kind != MOE_NORM_NONE || p->gate_kind != MOE_GATE_NONE)
        return MOE_ERR_INVALID_ARG;
    if (p->T == 0) return MOE_OK;
    if (!x || (!y && !q8)) return MOE_ERR_INVALID_ARG;
    const int64_t lds = ld_of(p->ld_stream, p->d), ldb = ld_of(p->ld_block, p->d);
    if (!elem_aligned(x, p->stream_dtype) || !elem_aligned(y, p->block_dtype) || !elem_aligned(weight, p->param_dtype) ||
        !elem_aligned(bias, p->param_dtype) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    const bool vec = rows_vec(x, p->d, lds, p->stream_dtype) && rows_vec(y, p->d, ldb, p->block_dtype) &&
                     rows_vec(weight, p->d, p->d, p->param_dtype) && rows_vec(bias, p->d, p->d, p->param_dtype);
    if ((st = check_f8_rows(q8, s8, p->d, vec)) != MOE_OK) return st;
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.q8 = q8; a.s8 = s8; a.mean = mean; a.rstd = rstd;
    a.ld_stream = lds; a.ld_block = ldb; a.T = p->T; a.d = p->d; a.kind = p->kind;
    a.stream_dt = p->stream_dtype; a.block_dt = p->block_dtype; a.param_dt = p->param_dtype;
    a.eps = p->eps; a.offset = p->weight_offset; a.alpha = 1.f; a.beta = 1.f;
    return (vec ? launch_fwd<false, true>(a, stream) : launch_fwd<false, false>(a, stream)) == cudaSuccess ? MOE_OK
                                                                                                           : MOE_ERR_CUDA;
}

int moe_norm_backward(const moe_norm_params* p, const void* x, const void* weight, const void* dy, const void* dres,
                      const float* mean, const float* rstd, void* dx, const moe_norm_grads* g, void* ws,
                      size_t ws_bytes, moe_stream_t stream) {
    int st = check_params(p);
    if (st != MOE_OK) return st;
    if (p->kind == MOE_NORM_NONE || p->next_kind != MOE_NORM_NONE || p->gate_kind != MOE_GATE_NONE)
        return MOE_ERR_INVALID_ARG;
    const moe_norm_grads none{};
    if (!g) g = &none;
    if (g->dgate) return MOE_ERR_INVALID_ARG;
    if (!aligned(g->dweight, 4) || !aligned(g->dbias, 4)) return MOE_ERR_MISALIGNED;
    if (p->T == 0) return zero_sums(p, *g, stream);
    if (!x || !dy || !dx || !rstd || (p->kind == MOE_NORM_LAYER && !mean) || (g->dweight && !weight))
        return MOE_ERR_INVALID_ARG;
    const int64_t lds = ld_of(p->ld_stream, p->d), ldb = ld_of(p->ld_block, p->d);
    if (!elem_aligned(x, p->stream_dtype) || !elem_aligned(dy, p->block_dtype) ||
        !elem_aligned(weight, p->param_dtype) || !elem_aligned(dres, p->stream_dtype) ||
        !elem_aligned(dx, p->stream_dtype) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    const bool vec = rows_vec(x, p->d, lds, p->stream_dtype) && rows_vec(dy, p->d, ldb, p->block_dtype) &&
                     rows_vec(weight, p->d, p->d, p->param_dtype) && rows_vec(dres, p->d, lds, p->stream_dtype) &&
                     rows_vec(dx, p->d, lds, p->stream_dtype);
    NormBwdArgs a{};
    a.x = x; a.dy = dy; a.dres = dres; a.weight = weight; a.mean = mean; a.rstd = rstd; a.dx = dx;
    a.ld_x = lds; a.ld_dy = ldb; a.T = p->T; a.d = p->d; a.kind = p->kind;
    a.x_dt = p->stream_dtype; a.dy_dt = p->block_dtype; a.param_dt = p->param_dtype;
    a.offset = p->weight_offset; a.alpha = 1.f; a.beta = 1.f;
    return run_backward<false>(p, a, *g, ws, ws_bytes, stream, vec);
}

int moe_norm_residual_forward(const moe_norm_params* p, const void* resid, const void* y, const void* weight,
                              const void* bias, const void* gate, void* out, float* mean, float* rstd,
                              const void* next_weight, const void* next_bias, void* x_next, uint8_t* q8, float* s8,
                              float* next_mean, float* next_rstd, moe_stream_t stream) {
    int st = check_params(p);
    if (st != MOE_OK) return st;
    const bool next = p->next_kind != MOE_NORM_NONE;
    if (p->kind == MOE_NORM_NONE && (weight || bias || mean || rstd)) return MOE_ERR_INVALID_ARG;
    if (!next && (next_weight || next_bias || x_next || q8 || s8 || next_mean || next_rstd)) return MOE_ERR_INVALID_ARG;
    if (!gate != (p->gate_kind == MOE_GATE_NONE) && p->T > 0) return MOE_ERR_INVALID_ARG;
    if (p->T == 0) return MOE_OK;
    if (!resid || !y || !out || (next && !x_next && !q8)) return MOE_ERR_INVALID_ARG;
    const int64_t lds = ld_of(p->ld_stream, p->d), ldb = ld_of(p->ld_block, p->d);
    for (const void* v : {resid, static_cast<const void*>(out)})
        if (!elem_aligned(v, p->stream_dtype)) return MOE_ERR_MISALIGNED;
    for (const void* v : {y, static_cast<const void*>(x_next)})
        if (!elem_aligned(v, p->block_dtype)) return MOE_ERR_MISALIGNED;
    for (const void* v : {weight, bias, gate, next_weight, next_bias})
        if (!elem_aligned(v, p->param_dtype)) return MOE_ERR_MISALIGNED;
    for (const float* v : {mean, rstd, next_mean, next_rstd})
        if (!aligned(v, 4)) return MOE_ERR_MISALIGNED;
    bool vec = rows_vec(resid, p->d, lds, p->stream_dtype) && rows_vec(out, p->d, lds, p->stream_dtype) &&
               rows_vec(y, p->d, ldb, p->block_dtype) && rows_vec(x_next, p->d, ldb, p->block_dtype);
    for (const void* v : {weight, bias, p->gate_kind == MOE_GATE_CHANNEL ? gate : nullptr, next_weight, next_bias})
        vec = vec && rows_vec(v, p->d, p->d, p->param_dtype);
    if ((st = check_f8_rows(q8, s8, p->d, vec)) != MOE_OK) return st;
    NormArgs a{};
    a.x = y; a.resid = resid; a.weight = weight; a.bias = bias; a.gate = gate; a.next_weight = next_weight;
    a.next_bias = next_bias; a.y = x_next; a.out = out; a.q8 = q8; a.s8 = s8; a.mean = mean; a.rstd = rstd;
    a.next_mean = next_mean; a.next_rstd = next_rstd; a.ld_stream = lds; a.ld_block = ldb; a.T = p->T; a.d = p->d;
    a.kind = p->kind; a.next_kind = p->next_kind; a.stream_dt = p->stream_dtype; a.block_dt = p->block_dtype;
    a.param_dt = p->param_dtype; a.gate_kind = p->gate_kind; a.eps = p->eps; a.offset = p->weight_offset;
    a.alpha = p->alpha; a.beta = p->beta;
    return (vec ? launch_fwd<true, true>(a, stream) : launch_fwd<true, false>(a, stream)) == cudaSuccess ? MOE_OK
                                                                                                         : MOE_ERR_CUDA;
}

int moe_norm_residual_backward(const moe_norm_params* p, const void* y, const void* weight, const void* bias,
                               const void* gate, const void* dout, const float* mean, const float* rstd, void* dresid,
                               void* dy, const moe_norm_grads* g, void* ws, size_t ws_bytes, moe_stream_t stream) {
    int st = check_params(p);
    if (st != MOE_OK) return st;
    const moe_norm_grads none{};
    if (!g) g = &none;
    const bool norm = p->kind != MOE_NORM_NONE;
    if (!norm && (weight || bias || g->dweight || g->dbias)) return MOE_ERR_INVALID_ARG;
    if (p->gate_kind == MOE_GATE_NONE && (gate || g->dgate)) return MOE_ERR_INVALID_ARG;
    if (!aligned(g->dweight, 4) || !aligned(g->dbias, 4) || !aligned(g->dgate, 4)) return MOE_ERR_MISALIGNED;
    if (p->T == 0) return zero_sums(p, *g, stream);
    if (!y || !dout || !dy || (norm && !rstd) || (p->kind == MOE_NORM_LAYER && !mean) || (g->dweight && !weight) ||
        (g->dbias && !bias) || (p->gate_kind != MOE_GATE_NONE && !gate))
        return MOE_ERR_INVALID_ARG;
    const int64_t lds = ld_of(p->ld_stream, p->d), ldb = ld_of(p->ld_block, p->d);
    for (const void* v : {dout, static_cast<const void*>(dresid)})
        if (!elem_aligned(v, p->stream_dtype)) return MOE_ERR_MISALIGNED;
    for (const void* v : {y, static_cast<const void*>(dy)})
        if (!elem_aligned(v, p->block_dtype)) return MOE_ERR_MISALIGNED;
    for (const void* v : {weight, bias, gate})
        if (!elem_aligned(v, p->param_dtype)) return MOE_ERR_MISALIGNED;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_MISALIGNED;
    bool vec = rows_vec(y, p->d, ldb, p->block_dtype) && rows_vec(dy, p->d, ldb, p->block_dtype) &&
               rows_vec(dout, p->d, lds, p->stream_dtype) && rows_vec(dresid, p->d, lds, p->stream_dtype);
    for (const void* v : {weight, bias, p->gate_kind == MOE_GATE_CHANNEL ? gate : nullptr})
        vec = vec && rows_vec(v, p->d, p->d, p->param_dtype);
    NormBwdArgs a{};
    a.x = y; a.dy = dout; a.weight = weight; a.bias = bias; a.gate = gate; a.mean = mean; a.rstd = rstd; a.dx = dy;
    a.dresid = dresid; a.ld_x = ldb; a.ld_dy = lds; a.T = p->T; a.d = p->d; a.kind = p->kind;
    a.x_dt = p->block_dtype; a.dy_dt = p->stream_dtype; a.param_dt = p->param_dtype; a.gate_kind = p->gate_kind;
    a.offset = p->weight_offset; a.alpha = p->alpha; a.beta = p->beta;
    return run_backward<true>(p, a, *g, ws, ws_bytes, stream, vec);
}

}  // extern "C"

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
//
// B200, replayed graphs, bytes of each row read and written once: before a block 8192 rows of 4096
// bf16 26.9 us, 4.99 TB/s, 4096 of 2048 9.7 us; backward with the weight's gradient 67 us, 4.0 TB/s
// (its sums' kernel 4.8). After it, 8192 rows of 1024, fp32 stream, with the next norm 25.3 us, 3.98 TB/s,
// backward 29.7, 3.4 TB/s. Neither the issue slots (36%) nor HBM are full: a row's chain of sums at two to
// three blocks an SM, and a grid whose last rows leave warps without any, take the rest. One row of 4096:
// 2.1 us, backward 5.6 (two launches).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// How a row gets into registers: element by element (any alignment), by loads of 4 elements (8 bytes of
// 16 bits, 16 of fp32: few rows, where the way is shortest, and any number of rows that lie on 4 elements'
// bytes but not on 16), or by 16-byte asynchronous copies of the next rows into shared memory (many rows:
// HBM stays busy while a row is summed). kStagedFull: rows of exactly 8 * NV * 32 W.
enum Mode { kScalar = 0, kVec = 1, kStaged = 2, kStagedFull = 3 };
__host__ __device__ constexpr int layout_of(int mode) { return mode == kScalar ? kScalarRow : mode == kStagedFull ? kFullRow : kVecRow; }

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

// Sums of N values over the W warps of a row, together; every thread of the block calls it.
// buf: 8 floats a value.
template <int W, int N>
MOE_DEV void row_sums(float (&v)[N], float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], o);
    if (W == 1) return;
    const int warp = threadIdx.x >> 5, g0 = warp / W * W;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) buf[n * 8 + warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) v[n] += buf[n * 8 + g0 + i];
    }
}
template <int W>
MOE_DEV float row_sum(float v, float* buf) {
    float a[1] = {v};
    row_sums<W>(a, buf);
    return a[0];
}

// Mean and 1/sqrt(var + eps) of the row in v, which becomes v - mean; buf: 16 floats of the block.
template <int W, int NV, int L>
MOE_DEV void row_stats(float (&v)[NV][8], int kind, int d, float eps, int t, float* buf, float& mean, float& rstd) {
    mean = 0.f;
    if (kind == MOE_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i][j];
        mean = row_sum<W>(s, buf) / float(d);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = in_row<L>(i, j, d, 32 * W, t) ? v[i][j] - mean : 0.f;
    }
    float s = 0.f;  // elements past the row are zero
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
    rstd = 1.0f / sqrtf(row_sum<W>(s, buf + 8) / float(d) + eps);
}

// v <- v rstd (w + o) + b; the weights, from L1 after the first rows, 8 at a time
template <int W, int NV, int L>
MOE_DEV void apply_norm(float (&v)[NV][8], float rstd, const void* w, const void* b, float offset, int param_dt, int d,
                        int t) {
    if (w) {
        by_dtype(param_dt, [&](auto DT) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float p[8];
                load_group<L, decltype(DT)::value>(p, w, i, d, 32 * W, t);
                if (offset != 0.f) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] += offset;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * p[j];
            }
        });
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    }
    if (b) {
        by_dtype(param_dt, [&](auto DT) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float p[8];
                load_group<L, decltype(DT)::value>(p, b, i, d, 32 * W, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += p[j];
            }
        });
    }
}

MOE_DEV char* at_row(const void* p, int64_t row, int64_t ld, int dt) {
    return static_cast<char*>(const_cast<void*>(p)) + row * ld * (dt == MOE_DT_F32 ? 4 : 2);
}

// Blocks an SM (their registers): before a block three, after it two, as the row's residual is held too
// (8192 rows of 1024, fp32 stream, with the next norm: 25.3 us with two, 30.9 with three).
template <int W, int NV, int MODE, bool POST>
__global__ void __launch_bounds__(kThreads, POST ? 2 : 3) norm_forward_kernel(const NormArgs a, const int depth) {
    constexpr int L = layout_of(MODE);
    constexpr bool STAGED = MODE >= kStaged;
    extern __shared__ uint4 stage[];  // STAGED: depth rows of every tensor
    __shared__ float buf[2][16];
    griddep_wait();
    griddep_launch();
    constexpr int th = 32 * W, rpb = kThreads / th;
    const int t = threadIdx.x % th;
    const int d = a.d;
    const int x_dt = POST ? a.block_dt : a.stream_dt;
    const int64_t ld_x = POST ? a.ld_block : a.ld_stream, step = int64_t(gridDim.x) * rpb;
    const int px = stage_pieces(NV, x_dt), pieces = px + (POST ? stage_pieces(NV, a.stream_dt) : 0);
    auto fetch = [&](int slot, int64_t r) {  // the row's copies, in a group of their own
        if (r < a.T) {
            const uint32_t dst = smem_u32(stage + slot * pieces * kThreads);
            copy_row<NV, L, kThreads>(dst, at_row(a.x, r, ld_x, x_dt), d, x_dt, th, t);
            if (POST)
                copy_row<NV, L, kThreads>(dst + px * kThreads * 16, at_row(a.resid, r, a.ld_stream, a.stream_dt), d,
                             a.stream_dt, th, t);
        }
        cp_async_commit();
    };
    const int64_t first = int64_t(blockIdx.x) * rpb + threadIdx.x / th;
    int slot = 0;
    if (STAGED)
        for (int i = 0; i < depth; ++i) fetch(i, first + i * step);
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < a.T; r0 += step) {
        // rows past T take part in the block's reductions and store nothing
        const int64_t r = r0 + threadIdx.x / th;
        const bool live = r < a.T;
        const int dl = live ? d : 0;
        float v[NV][8];
        float res[POST ? NV : 1][8];
        if constexpr (STAGED) {
            cp_async_wait_most(depth - 1);
            __syncwarp();  // a lane's quads may be another lane's copies
            const uint4* src = stage + slot * pieces * kThreads;
            read_row<NV, L, kThreads>(v, src, dl, x_dt, th, t);
            if constexpr (POST) read_row<NV, L, kThreads>(res, src + px * kThreads, dl, a.stream_dt, th, t);
        } else {
            load_row<NV, L>(v, at_row(a.x, live ? r : 0, ld_x, x_dt), dl, x_dt, th, t);
            if constexpr (POST)
                load_row<NV, L>(res, at_row(a.resid, live ? r : 0, a.ld_stream, a.stream_dt), dl, a.stream_dt, th, t);
        }
        if (a.kind != MOE_NORM_NONE) {
            float mean, rstd;
            row_stats<W, NV, L>(v, a.kind, d, a.eps, t, buf[0], mean, rstd);
            if (live && t == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
            apply_norm<W, NV, L>(v, rstd, a.weight, a.bias, a.offset, a.param_dt, d, t);
        }
        if constexpr (POST) {
            float gt = a.beta;
            if (a.gate_kind == MOE_GATE_TOKEN) gt *= live ? load_elem(a.gate, r, a.param_dt) : 0.f;
            if (a.gate_kind == MOE_GATE_CHANNEL) {
                by_dtype(a.param_dt, [&](auto DT) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        float p[8];
                        load_group<L, decltype(DT)::value>(p, a.gate, i, d, th, t);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] *= p[j];
                    }
                });
            }
            by_dtype(a.stream_dt, [&](auto DT) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = round_to(fmaf(a.alpha, res[i][j], gt * v[i][j]), decltype(DT)::value);
            });
            if (live) store_row<NV, L>(v, at_row(a.out, r, a.ld_stream, a.stream_dt), d, a.stream_dt, th, t);
            if (a.next_kind != MOE_NORM_NONE) {
                float mean, rstd;
                row_stats<W, NV, L>(v, a.next_kind, d, a.eps, t, buf[1], mean, rstd);
                if (live && t == 0) {
                    if (a.next_mean) a.next_mean[r] = mean;
                    if (a.next_rstd) a.next_rstd[r] = rstd;
                }
                apply_norm<W, NV, L>(v, rstd, a.next_weight, a.next_bias, a.offset, a.param_dt, d, t);
            }
        }
        if (a.y && live) store_row<NV, L>(v, at_row(a.y, r, a.ld_block, a.block_dt), d, a.block_dt, th, t);
        if constexpr (L != kScalarRow) {
            // `live` is one value a warp; a full row's stores have no bound of their own that could keep a row past T back
            if (a.q8 && live) store_row_e4m3<NV, L>(v, a.q8 + r * d, a.s8 + r, a.T, d, th, t);
        }
        if constexpr (STAGED) {  // the row is in registers: its place takes the row `depth` on
            __syncwarp();
            fetch(slot, r + depth * step);
            slot = slot + 1 == depth ? 0 : slot + 1;
        }
        if (W > 1) __syncthreads();  // the block's sums are read before the next rows write theirs
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
    float* s1;          // [blocks, d] sums of rs D xhat, or null: no sums over tokens
    float* s0;          // [blocks, d] sums of rs D (S0)
    int64_t ld_x, ld_dy;
    int T, d, kind, x_dt, dy_dt, param_dt, gate_kind;
    float offset, alpha, beta;
};

// Backward blocks an SM (their registers): also the grid, whose partial sums are written and read once
// more, so few enough that they stay small beside the rows. In vectors the copies ahead keep HBM busy
// (4096 rows of 2048 bf16: 18.2 us with 2 blocks and 96 registers, 21.2 with 3, 27.5 with 4, whose
// registers do not hold a row); element by element the warps do (rows of 2047: 67.8, 56.0, 47.9 us, although
// the 64 registers that four blocks leave a thread spill 300 to 1300 bytes). Rows of more than 4096 (NV of 4)
// spill up to 1200 bytes at 128 registers too: 2048 rows of 8192 bf16 60 us, 2.2 TB/s.
__host__ __device__ constexpr int bwd_blocks(int nv, int mode) { return mode == kScalar && nv <= 2 ? 4 : 2; }
constexpr int kBwdBlocksMost = 4;

// S0: whether sums without xhat are wanted (a bias).
template <int W, int NV, int MODE, bool POST, bool S0>
__global__ void __launch_bounds__(kThreads, bwd_blocks(NV, MODE)) norm_backward_kernel(const NormBwdArgs a, const int depth) {
    constexpr int L = layout_of(MODE);
    constexpr bool STAGED = MODE >= kStaged;
    constexpr int th = 32 * W, rpb = kThreads / th;
    __shared__ float buf[24];
    extern __shared__ uint4 stage[];  // STAGED: depth rows of every tensor; at the end, rpb > 1: sums [1 + S0][d]
    float* sums = reinterpret_cast<float*>(stage);
    griddep_wait();
    const int t = threadIdx.x % th;
    const int d = a.d;
    const float inv_d = 1.0f / float(d);
    float s1[NV][8], s0[S0 ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s1[i][j] = 0.f;
            if (S0) s0[i][j] = 0.f;
        }
    const int64_t step = int64_t(gridDim.x) * rpb;
    const int px = stage_pieces(NV, a.x_dt), pg = px + stage_pieces(NV, a.dy_dt), pieces = pg + (!POST && a.dres ? px : 0);
    auto fetch = [&](int slot, int64_t r) {
        if (r < a.T) {
            const uint32_t dst = smem_u32(stage + slot * pieces * kThreads);
            copy_row<NV, L, kThreads>(dst, at_row(a.x, r, a.ld_x, a.x_dt), d, a.x_dt, th, t);
            copy_row<NV, L, kThreads>(dst + px * kThreads * 16, at_row(a.dy, r, a.ld_dy, a.dy_dt), d, a.dy_dt, th, t);
            if (!POST && a.dres)
                copy_row<NV, L, kThreads>(dst + pg * kThreads * 16, at_row(a.dres, r, a.ld_x, a.x_dt), d, a.x_dt, th, t);
        }
        cp_async_commit();
    };
    const int64_t first = int64_t(blockIdx.x) * rpb + threadIdx.x / th;
    int slot = 0;
    if (STAGED)
        for (int i = 0; i < depth; ++i) fetch(i, first + i * step);
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < a.T; r0 += step) {
        const int64_t r = r0 + threadIdx.x / th;
        const bool live = r < a.T;
        const int dl = live ? d : 0;
        float x[NV][8], g[NV][8];
        const uint4* src = stage + slot * pieces * kThreads;
        if constexpr (STAGED) {
            cp_async_wait_most(depth - 1);
            __syncwarp();  // a lane's quads may be another lane's copies
            read_row<NV, L, kThreads>(x, src, dl, a.x_dt, th, t);
            read_row<NV, L, kThreads>(g, src + px * kThreads, dl, a.dy_dt, th, t);
            if (L == kFullRow && !live) {  // nothing was copied for a row past T
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] = g[i][j] = 0.f;
            }
        } else {
            load_row<NV, L>(x, at_row(a.x, live ? r : 0, a.ld_x, a.x_dt), dl, a.x_dt, th, t);
            load_row<NV, L>(g, at_row(a.dy, live ? r : 0, a.ld_dy, a.dy_dt), dl, a.dy_dt, th, t);
        }
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
                store_row<NV, L>(q, at_row(a.dresid, r, a.ld_dy, a.dy_dt), d, a.dy_dt, th, t);
            }
        }
        // g becomes the gradient of xhat without the row's factor rs; on the way the sums over
        // tokens (s1, s0), the row's two sums and a token gate's gradient
        float dot_n = 0.f, sa = 0.f, sb = 0.f;
        by_dtype(a.param_dt, [&](auto DT) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[i][j] = (x[i][j] - mean) * rstd;  // past the row: any number, its g is zero
                    const float e = rs * g[i][j];
                    s1[i][j] = fmaf(e, x[i][j], s1[i][j]);
                    if (S0) s0[i][j] += e;
                }
                if (POST && a.dgate_tok && a.bias) {
                    load_group<L, decltype(DT)::value>(p, a.bias, i, d, th, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot_n = fmaf(g[i][j], p[j], dot_n);
                }
                if (a.weight) {
                    load_group<L, decltype(DT)::value>(p, a.weight, i, d, th, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[i][j] *= p[j] + a.offset;
                }
                if (POST && a.dgate_tok) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot_n = fmaf(g[i][j], x[i][j], dot_n);
                }
                if (POST && a.gate_kind == MOE_GATE_CHANNEL) {
                    load_group<L, decltype(DT)::value>(p, a.gate, i, d, th, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[i][j] *= p[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sa = fmaf(g[i][j], x[i][j], sa);
                    sb += g[i][j];
                }
            }
        });
        float sums3[3] = {sa, sb, dot_n};
        row_sums<W>(sums3, buf);
        if (POST && a.dgate_tok && live && t == 0) a.dgate_tok[r] = a.beta * sums3[2];
        if (a.kind != MOE_NORM_NONE) {
            sa = sums3[0] * inv_d;
            sb = a.kind == MOE_NORM_LAYER ? sums3[1] * inv_d : 0.f;
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
            if constexpr (STAGED) read_row<NV, L, kThreads>(x, src + pg * kThreads, dl, a.x_dt, th, t);
            else load_row<NV, L>(x, at_row(a.dres, live ? r : 0, a.ld_x, a.x_dt), dl, a.x_dt, th, t);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] += x[i][j];
        }
        if (live) store_row<NV, L>(g, at_row(a.dx, r, a.ld_x, a.x_dt), d, a.x_dt, th, t);
        if constexpr (STAGED) {
            __syncwarp();
            fetch(slot, r + depth * step);
            slot = slot + 1 == depth ? 0 : slot + 1;
        }
        if (W > 1) __syncthreads();
    }
    if constexpr (STAGED) {
        cp_async_wait<0>();  // (groups without copies)
        __syncthreads();     // the stages become the sums' place
    }
    griddep_launch();
    if (!a.s1) return;
    // the block's rows added in the order of its groups of warps, then one row of sums a block
    if (rpb > 1) {
        const int grp = threadIdx.x / th;
        for (int k = 1; k < rpb; ++k) {
            if (grp == k) {
                store_row<NV, L>(s1, sums, d, MOE_DT_F32, th, t);
                if constexpr (S0) store_row<NV, L>(s0, sums + d, d, MOE_DT_F32, th, t);
            }
            __syncthreads();
            if (grp == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float p[8];
                    load_group<L, MOE_DT_F32>(p, sums, i, d, th, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s1[i][j] += p[j];
                    if constexpr (S0) {
                        load_group<L, MOE_DT_F32>(p, sums + d, i, d, th, t);
#pragma unroll
                        for (int j = 0; j < 8; ++j) s0[i][j] += p[j];
                    }
                }
            }
            __syncthreads();
        }
        if (grp != 0) return;
    }
    store_row<NV, L>(s1, a.s1 + int64_t(blockIdx.x) * d, d, MOE_DT_F32, th, t);
    if constexpr (S0) store_row<NV, L>(s0, a.s0 + int64_t(blockIdx.x) * d, d, MOE_DT_F32, th, t);
}

// The blocks' partial sums added in a fixed order: 8 columns x 128 strips of blocks, then the
// strips. dw = gate S1, db = gate S0, dgate = (w + o) S1 + b S0 (gate per channel; else gate = 1
// here, the token's gate and beta being in the sums).
struct NormSumArgs {
    const float* s1;
    const float* s0;
    const void* weight;
    const void* bias;
    const void* gate;  // per channel, or null
    float* dw;
    float* db;
    float* dgate;
    int blocks, d, param_dt;
    float offset;
};

constexpr int kSumCols = 8, kSumStrips = 128;

__global__ void __launch_bounds__(kSumCols* kSumStrips) norm_sum_kernel(const NormSumArgs a) {
    __shared__ float sm[2][kSumStrips][kSumCols + 1];
    griddep_wait();
    griddep_launch();
    const int cx = threadIdx.x % kSumCols, sy = threadIdx.x / kSumCols;
    const int c = blockIdx.x * kSumCols + cx;
    float v1 = 0.f, v0 = 0.f;
    if (c < a.d) {
#pragma unroll 4
        for (int g = sy; g < a.blocks; g += kSumStrips) {
            v1 += a.s1[int64_t(g) * a.d + c];
            if (a.s0) v0 += a.s0[int64_t(g) * a.d + c];
        }
    }
    sm[0][sy][cx] = v1;
    sm[1][sy][cx] = v0;
    __syncthreads();
    // warp w adds column w's strips, four a lane
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (w >= kSumCols) return;
    float w1 = 0.f, w0 = 0.f;
#pragma unroll
    for (int i = 0; i < kSumStrips / 32; ++i) {
        w1 += sm[0][lane + 32 * i][w];
        w0 += sm[1][lane + 32 * i][w];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        w1 += __shfl_xor_sync(0xFFFFFFFFu, w1, o);
        w0 += __shfl_xor_sync(0xFFFFFFFFu, w0, o);
    }
    const int col = blockIdx.x * kSumCols + w;
    if (lane == 0 && col < a.d) {
        const float gate = a.gate ? load_elem(a.gate, col, a.param_dt) : 1.f;
        if (a.dw) a.dw[col] = gate * w1;
        if (a.db) a.db[col] = gate * w0;
        if (a.dgate) {
            const float w = a.weight ? load_elem(a.weight, col, a.param_dt) + a.offset : 1.f;
            a.dgate[col] = w * w1 + (a.bias ? load_elem(a.bias, col, a.param_dt) * w0 : 0.f);
        }
    }
}

// Warps per row, groups of 8 a thread, and the way in. Few rows (less than two warps for each of
// the SMs' four schedulers): 8 warps a row, the shortest chain. Many: as few warps a row as hold it
// with `most` groups a thread, so that a row's sums meet few warps; the copies ahead, not the warps,
// keep HBM busy.
struct Shape {
    int w, nv, mode;
};
Shape shape_of(int T, int d, int vec, int most) {  // vec: rows_vec of every tensor
    const int v = (d + 7) / 8;
    Shape s{1, 1, vec == 2 ? kStaged : kScalar};
    while (s.w < 8 && s.w * 32 * most < v) s.w *= 2;
    if (vec == 1 || int64_t(T) * s.w < int64_t(num_sms()) * 8) {
        s.w = 8;
        if (vec) s.mode = kVec;
    }
    while (s.w * 32 * s.nv < v) s.nv *= 2;
    if (s.mode == kStaged && s.w * 32 * s.nv * 8 == d) s.mode = kStagedFull;
    return s;
}
// The backward kernel also holds the sums over tokens. Forward: before a block 2 (4096 rows of 2047: 21.9 us
// with 4, 17.9 with 2; 8192 rows of 4096: 27.6 and 26.9), after it 4 (its three sums a row then mostly
// need no other warp; 8192 rows of 1024 with the next norm: 25.3 us, with 2 28.2).
template <bool POST>
constexpr int kMostFwd = POST ? 4 : 2;
constexpr int kMostBwd = 2;
static_assert(MOE_NORM_MAX_D <= 8 * 32 * 8 * 4, "a row fits a block");

// f with the shape as compile-time constants.
template <int MOST, typename F>
cudaError_t with_shape(const Shape& s, F f) {
    using std::integral_constant;
#define MOE_SHAPE(W_, NV_, M_)                    \
    if (s.w == W_ && s.nv == NV_ && s.mode == M_) \
        return f(integral_constant<int, W_>{}, integral_constant<int, NV_>{}, integral_constant<int, M_>{});
#define MOE_SHAPES(W_, NV_) MOE_SHAPE(W_, NV_, kScalar) MOE_SHAPE(W_, NV_, kStaged) MOE_SHAPE(W_, NV_, kStagedFull)
    MOE_SHAPE(8, 1, kVec) MOE_SHAPE(8, 2, kVec) MOE_SHAPE(8, 4, kVec)
    MOE_SHAPE(8, 1, kScalar)
    MOE_SHAPES(1, 1) MOE_SHAPES(1, 2) MOE_SHAPES(8, 4)
    if constexpr (MOST == 4) {
        MOE_SHAPES(1, 4) MOE_SHAPES(2, 4) MOE_SHAPES(4, 4)
        MOE_SHAPE(8, 2, kScalar)
    } else {
        MOE_SHAPES(2, 2) MOE_SHAPES(4, 2) MOE_SHAPES(8, 2)
    }
#undef MOE_SHAPES
#undef MOE_SHAPE
    return cudaErrorInvalidValue;
}

// Rows ahead: as many as a third of an SM's shared memory takes, two to four (three blocks an SM
// where the registers allow).
int depth_of(const Shape& s, size_t slot_bytes) {
    return s.mode >= kStaged ? int(std::max<size_t>(2, std::min<size_t>(4, 72 * 1024 / slot_bytes))) : 0;
}
size_t pieces_bytes(int nv, int dt) { return size_t(nv) * (dt == MOE_DT_F32 ? 2 : 1) * 16 * kThreads; }

constexpr int kMaxSmem = 200 * 1024;  // two rows of three fp32 tensors and the sums' place; a block may opt into 227 KB

// The kernel may use more than 48 KB of shared memory (set once a device).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load() & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// Blocks of a kernel that share an SM: a grid of just as many leaves no part of a second wave behind
// (592 blocks where 444 fit took 34.7 us for 8192 rows of 4096 bf16, 444 blocks 28.7 us).
template <typename K>
int blocks_per_sm(K kernel, size_t smem, std::atomic<uint64_t>& fit) {
    const uint64_t known = fit.load();
    if ((known >> 8) == smem + 1) return int(known & 255);
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = 1;
    }
    fit.store((uint64_t(smem + 1) << 8) | uint64_t(n));
    return n;
}
int grid_of(int T, int w, int per_sm) {
    const int rpb = kThreads / (32 * w);
    const int64_t blocks = (int64_t(T) + rpb - 1) / rpb;
    return int(std::min<int64_t>(blocks, int64_t(num_sms()) * per_sm));
}

size_t esize(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// How far rows can be read in vectors: 1 quads on every row (its length and stride and the base), 2
// also every row on 16 bytes, 0 neither.
int rows_vec(const void* p, int d, int64_t ld, int dt) {
    if (!p) return 2;
    if (d % 4 || ld % 4 || !aligned(p, 4 * esize(dt))) return 0;
    return (ld * int64_t(esize(dt))) % 16 == 0 && aligned(p, 16) ? 2 : 1;
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

template <bool POST>
cudaError_t launch_fwd(const NormArgs& a, int vec, cudaStream_t s) {
    const Shape sh = shape_of(a.T, a.d, vec, kMostFwd<POST>);
    const size_t slot = POST ? pieces_bytes(sh.nv, a.block_dt) + pieces_bytes(sh.nv, a.stream_dt) : pieces_bytes(sh.nv, a.stream_dt);
    const int depth = depth_of(sh, slot);
    const size_t smem = depth * slot;
    ProfScope prof_(MOE_K_NORM, s);
    return with_shape<kMostFwd<POST>>(sh, [&](auto W, auto NV, auto MODE) {
        static std::atomic<uint64_t> done{0};
        auto kernel = norm_forward_kernel<W(), NV(), MODE(), POST>;
        const cudaError_t e = allow_smem(kernel, smem, done);
        if (e != cudaSuccess) return e;
        static std::atomic<uint64_t> fit{0};  // (shared memory, blocks an SM) of the last call
        return launch_pdl(use_pdl(a.T), kernel, dim3(grid_of(a.T, sh.w, blocks_per_sm(kernel, smem, fit))), dim3(kThreads), smem, s,
                          a, depth);
    });
}

template <bool POST, bool S0>
cudaError_t launch_bwd(const NormBwdArgs& a, const Shape& sh, int grid, cudaStream_t s) {
    const size_t px = pieces_bytes(sh.nv, a.x_dt), slot = px + pieces_bytes(sh.nv, a.dy_dt) + (!POST && a.dres ? px : 0);
    const int depth = depth_of(sh, slot);
    const size_t sums = a.s1 && sh.w < kThreads / 32 ? size_t(a.d) * 4 * (S0 ? 2 : 1) : 0;
    const size_t smem = std::max(depth * slot, sums);
    ProfScope prof_(MOE_K_NORM_BWD, s);
    return with_shape<kMostBwd>(sh, [&](auto W, auto NV, auto MODE) {
        static std::atomic<uint64_t> done{0};
        auto kernel = norm_backward_kernel<W(), NV(), MODE(), POST, S0>;
        const cudaError_t e = allow_smem(kernel, smem, done);
        if (e != cudaSuccess) return e;
        return launch_pdl(use_pdl(a.T), kernel, dim3(grid), dim3(kThreads), smem, s, a, depth);
    });
}

// Room for the partial sums of either way in: the larger grid.
size_t sums_bytes(const moe_norm_params* p) {
    int grid = 0;
    for (int vec : {0, 1, 2})
        grid = std::max(grid, grid_of(std::max(1, p->T), shape_of(std::max(1, p->T), p->d, vec, kMostBwd).w, kBwdBlocksMost));
    return (size_t(grid) * p->d * 4 + 255) & ~size_t(255);
}
size_t norm_ws_bytes(const moe_norm_params* p) { return 256 + 2 * sums_bytes(p); }

int check_f8_rows(const uint8_t* q8, const float* s8, int d, int vec) {
    if (!q8 != !s8) return MOE_ERR_INVALID_ARG;
    if (!q8) return MOE_OK;
    if (d % 16) return MOE_ERR_INVALID_ARG;
    return vec && aligned(q8, 16) && aligned(s8, 4) ? MOE_OK : MOE_ERR_MISALIGNED;
}

template <bool POST>
int run_backward(const moe_norm_params* p, NormBwdArgs a, const moe_norm_grads& g, void* ws, size_t ws_bytes,
                 cudaStream_t stream, int vec) {
    const Shape sh = shape_of(p->T, p->d, vec, kMostBwd);
    const bool gate_c = POST && p->gate_kind == MOE_GATE_CHANNEL;
    const bool need1 = g.dweight || (gate_c && g.dgate);
    const bool need0 = g.dbias || (gate_c && g.dgate && a.bias);
    const int grid = grid_of(p->T, sh.w, bwd_blocks(sh.nv, sh.mode));
    if (need1 || need0) {
        if (!ws) return MOE_ERR_INVALID_ARG;
        if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
        if (ws_bytes < norm_ws_bytes(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        uint8_t* w = static_cast<uint8_t*>(ws) + 256;
        a.s1 = reinterpret_cast<float*>(w);
        if (need0) a.s0 = reinterpret_cast<float*>(w + sums_bytes(p));
    }
    a.dgate_tok = POST && p->gate_kind == MOE_GATE_TOKEN ? g.dgate : nullptr;
    const cudaError_t e = need0 ? launch_bwd<POST, true>(a, sh, grid, stream) : launch_bwd<POST, false>(a, sh, grid, stream);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (need1 || need0) {
        const NormSumArgs sa{a.s1, a.s0, a.weight, a.bias, gate_c ? a.gate : nullptr, g.dweight, g.dbias,
                             gate_c ? g.dgate : nullptr, grid, p->d, p->param_dtype, p->weight_offset};
        ProfScope prof_(MOE_K_NORM_BWD, stream);
        // its blocks may start as the rows' blocks end
        if (launch_pdl(true, norm_sum_kernel, dim3((p->d + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumStrips), 0,
                       stream, sa) != cudaSuccess)
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
    int vec = std::min(rows_vec(x, p->d, lds, p->stream_dtype), rows_vec(y, p->d, ldb, p->block_dtype));
    for (const void* v : {weight, bias})
        if (!rows_vec(v, p->d, p->d, p->param_dtype)) vec = 0;
    if ((st = check_f8_rows(q8, s8, p->d, vec)) != MOE_OK) return st;
    if (x == y && (p->stream_dtype != p->block_dtype || lds != ldb)) return MOE_ERR_INVALID_ARG;  // rows over others
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.q8 = q8; a.s8 = s8; a.mean = mean; a.rstd = rstd;
    a.ld_stream = lds; a.ld_block = ldb; a.T = p->T; a.d = p->d; a.kind = p->kind;
    a.stream_dt = p->stream_dtype; a.block_dt = p->block_dtype; a.param_dt = p->param_dtype;
    a.eps = p->eps; a.offset = p->weight_offset; a.alpha = 1.f; a.beta = 1.f;
    return launch_fwd<false>(a, vec, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    int vec = rows_vec(dy, p->d, ldb, p->block_dtype);
    for (const void* v : {x, dres, static_cast<const void*>(dx)}) vec = std::min(vec, rows_vec(v, p->d, lds, p->stream_dtype));
    if (!rows_vec(weight, p->d, p->d, p->param_dtype)) vec = 0;
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
    int vec = std::min({rows_vec(resid, p->d, lds, p->stream_dtype), rows_vec(out, p->d, lds, p->stream_dtype),
                        rows_vec(y, p->d, ldb, p->block_dtype), rows_vec(x_next, p->d, ldb, p->block_dtype)});
    for (const void* v : {weight, bias, p->gate_kind == MOE_GATE_CHANNEL ? gate : nullptr, next_weight, next_bias})
        if (!rows_vec(v, p->d, p->d, p->param_dtype)) vec = 0;
    if ((st = check_f8_rows(q8, s8, p->d, vec)) != MOE_OK) return st;
    NormArgs a{};
    a.x = y; a.resid = resid; a.weight = weight; a.bias = bias; a.gate = gate; a.next_weight = next_weight;
    a.next_bias = next_bias; a.y = x_next; a.out = out; a.q8 = q8; a.s8 = s8; a.mean = mean; a.rstd = rstd;
    a.next_mean = next_mean; a.next_rstd = next_rstd; a.ld_stream = lds; a.ld_block = ldb; a.T = p->T; a.d = p->d;
    a.kind = p->kind; a.next_kind = p->next_kind; a.stream_dt = p->stream_dtype; a.block_dt = p->block_dtype;
    a.param_dt = p->param_dtype; a.gate_kind = p->gate_kind; a.eps = p->eps; a.offset = p->weight_offset;
    a.alpha = p->alpha; a.beta = p->beta;
    return launch_fwd<true>(a, vec, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    int vec = std::min({rows_vec(y, p->d, ldb, p->block_dtype), rows_vec(dy, p->d, ldb, p->block_dtype),
                        rows_vec(dout, p->d, lds, p->stream_dtype), rows_vec(dresid, p->d, lds, p->stream_dtype)});
    for (const void* v : {weight, bias, p->gate_kind == MOE_GATE_CHANNEL ? gate : nullptr})
        if (!rows_vec(v, p->d, p->d, p->param_dtype)) vec = 0;
    NormBwdArgs a{};
    a.x = y; a.dy = dout; a.weight = weight; a.bias = bias; a.gate = gate; a.mean = mean; a.rstd = rstd; a.dx = dy;
    a.dresid = dresid; a.ld_x = ldb; a.ld_dy = lds; a.T = p->T; a.d = p->d; a.kind = p->kind;
    a.x_dt = p->block_dtype; a.dy_dt = p->stream_dtype; a.param_dt = p->param_dtype; a.gate_kind = p->gate_kind;
    a.offset = p->weight_offset; a.alpha = p->alpha; a.beta = p->beta;
    return run_backward<true>(p, a, *g, ws, ws_bytes, stream, vec);
}

}  // extern "C"

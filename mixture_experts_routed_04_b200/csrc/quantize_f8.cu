// quantize_f8.cu — rows and weights to e4m3 with a scale for each block of 128:
// moe_quantize_f8 (rows, gathered by token for the experts' products) and
// moe_quantize_f8_weights (once, at load time).
//
// Rows: a warp takes up to 1024 columns of a row, a block of 128 at 4 columns a lane, with
// all of its loads in flight first; one warp maximum finds a block's largest magnitude
// (rows.cuh). Bytes: 2 to 4 a value in, 1 out; a gathered
// row is read k times, from L2 for a prompt's x. Weights: a block of threads takes
// one 128 x 128 block into registers; given [K, N] it turns it in shared memory.
#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kRowNV = 4;  // groups of 8 columns a lane: 1024 columns a warp

template <bool VEC>
MOE_DEV void load8(float (&v)[8], const void* p, int64_t i, int dt) {
    if (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load_elem(p, i + j, dt);
    } else if (dt == MOE_DT_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), dt == MOE_DT_BF16, v);
    }
}

template <bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* x, int x_dt, int64_t ld, int64_t src_rows,
                                                            const int32_t* row_index, const int32_t* n_rows,
                                                            int64_t rows, int K, uint8_t* q, float* s, uint32_t* err) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    const int chunks = (K + 32 * 8 * kRowNV - 1) / (32 * 8 * kRowNV);
    const int64_t n = n_rows ? min(rows, int64_t(max(0, *n_rows))) : rows;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    bool bad = false;
    for (int64_t u = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < n * chunks; u += warps) {
        const int64_t r = u / chunks;
        const int c0 = int(u - r * chunks) * (32 * 8 * kRowNV);
        int64_t src = r;
        if (row_index) {
            src = row_index[r];
            if (src < 0 || src >= src_rows) {
                bad = true;
                continue;
            }
        }
        float v[kRowNV][8];
        const int dc = min(K - c0, 32 * 8 * kRowNV);
        const char* row = static_cast<const char*>(x) + (src * ld + c0) * (x_dt == MOE_DT_F32 ? 4 : 2);
        if (VEC) {
            load_row<kRowNV, kVecRow>(v, row, dc, x_dt, 32, lane);
        } else {
#pragma unroll
            for (int i = 0; i < kRowNV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = quad_at(i, j >> 2, 32, lane);
                    v[i][j] = c < dc ? load_elem(row, c + (j & 3), x_dt) : 0.f;  // K is a multiple of 16
                }
        }
        store_row_e4m3<kRowNV, kVecRow>(v, q + r * K + c0, s + int64_t(c0 >> 7) * rows + r, rows, dc, 32, lane);
    }
    if (bad) set_error(err, MOE_DEVERR_BOUNDS);
}

constexpr int kTurnPitch = 132;  // bytes of a turned row in shared memory: neighbouring rows 33 banks apart

// One 128 x 128 block of a matrix of `rows` x `cols` (row-major): thread t holds
// the 8 columns (t & 15) * 8 of rows (t >> 4) + 16 i. TURN: the matrix is [K, N]
// and the result its transpose.
template <bool VEC, bool TURN>
__global__ void __launch_bounds__(256) quantize_weights_kernel(const void* w, int w_dt, int N, int K, uint8_t* q,
                                                               float* s) {
    __shared__ uint32_t wmax[8];
    __shared__ __align__(16) uint8_t turn[TURN ? 128 * kTurnPitch : 16];
    griddep_wait();
    griddep_launch();
    const int e = blockIdx.z, nb = blockIdx.y, kb = blockIdx.x;
    const int rows = TURN ? K : N, cols = TURN ? N : K;
    const int r0 = (TURN ? kb : nb) * 128, c0 = (TURN ? nb : kb) * 128;
    const int cx = (threadIdx.x & 15) * 8, ry = threadIdx.x >> 4;
    const int64_t base = int64_t(e) * N * K;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + ry + 16 * i, c = c0 + cx;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (r < rows && c < cols) load8<VEC>(v[i], w, base + int64_t(r) * cols + c, w_dt);  // cols: a multiple of 8
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, wmax[i]);
    const float sc = f8_scale(m);
    const F8Div div(sc);
    if (threadIdx.x == 0) s[(int64_t(e) * gridDim.y + nb) * gridDim.x + kb] = sc;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint2 b = make_uint2(pack4_e4m3(v[i], div), pack4_e4m3(v[i] + 4, div));
        if (!TURN) {
            const int r = r0 + ry + 16 * i, c = c0 + cx;
            if (r < rows && c < cols) *reinterpret_cast<uint2*>(q + base + int64_t(r) * K + c) = b;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                turn[(cx + j) * kTurnPitch + ry + 16 * i] = uint8_t((j < 4 ? b.x >> (8 * j) : b.y >> (8 * (j - 4))) & 0xFFu);
        }
    }
    if (TURN) {
        __syncthreads();
        // 16 bytes of K of one column of N a thread and step
        for (int i = threadIdx.x; i < 128 * 8; i += 256) {
            const int n = i >> 3, k = (i & 7) * 16;
            if (c0 + n >= N || r0 + k >= K) continue;  // K is a multiple of 16
            const uint32_t* p = reinterpret_cast<const uint32_t*>(turn + n * kTurnPitch + k);
            *reinterpret_cast<uint4*>(q + base + int64_t(c0 + n) * K + r0 + k) = make_uint4(p[0], p[1], p[2], p[3]);
        }
    }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize_f8(int64_t rows, int32_t K, const void* x, int32_t x_dtype, int64_t ld_x, int64_t src_rows,
                    const int32_t* row_index, const int32_t* n_rows, uint8_t* q, float* s, void* ws, size_t ws_bytes,
                    moe_stream_t stream) {
    if (rows < 0 || rows >= (int64_t(1) << 31) || K < 16 || K % 16 || src_rows < 0) return MOE_ERR_INVALID_ARG;
    if (x_dtype < MOE_DT_F32 || x_dtype > MOE_DT_F16) return MOE_ERR_INVALID_ARG;
    if (ld_x != 0 && (ld_x < K || ld_x > (int64_t(1) << 31))) return MOE_ERR_INVALID_ARG;
    if (!row_index && src_rows < rows) return MOE_ERR_INVALID_ARG;
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < 256) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !s) return MOE_ERR_INVALID_ARG;
    const int64_t ld = ld_x ? ld_x : K;
    const size_t es = x_dtype == MOE_DT_F32 ? 4 : 2;
    if (!aligned(q, 16) || !aligned(s, 4) || !aligned(x, es) || !aligned(row_index, 4) || !aligned(n_rows, 4))
        return MOE_ERR_MISALIGNED;
    const bool vec = aligned(x, 4 * es) && ld % 4 == 0;
    const int64_t chunks = (K + 32 * 8 * kRowNV - 1) / (32 * 8 * kRowNV);
    const int64_t blocks = std::min<int64_t>((rows * chunks + 7) / 8, int64_t(num_sms()) * 8);
    ProfScope prof_(MOE_K_QUANT_F8, stream);
    const cudaError_t e =
        vec ? launch_pdl(use_pdl(rows), quantize_rows_kernel<true>, dim3(int(blocks)), dim3(256), 0, stream, x, x_dtype,
                         ld, src_rows, row_index, n_rows, rows, K, q, s, static_cast<uint32_t*>(ws))
            : launch_pdl(use_pdl(rows), quantize_rows_kernel<false>, dim3(int(blocks)), dim3(256), 0, stream, x,
                         x_dtype, ld, src_rows, row_index, n_rows, rows, K, q, s, static_cast<uint32_t*>(ws));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_quantize_f8_weights(int32_t E, int32_t N, int32_t K, const void* w, int32_t w_dtype, int32_t transposed,
                            uint8_t* q, float* s, moe_stream_t stream) {
    if (E < 1 || E > 65535 || N < 8 || N % 8 || K < 16 || K % 16 || (transposed != 0 && transposed != 1))
        return MOE_ERR_INVALID_ARG;
    if (w_dtype < MOE_DT_F32 || w_dtype > MOE_DT_F16) return MOE_ERR_INVALID_ARG;
    if ((N + 127) / 128 > 65535 || int64_t(N) * K >= (int64_t(1) << 40)) return MOE_ERR_INVALID_ARG;
    if (!w || !q || !s) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(s, 4) || !aligned(w, w_dtype == MOE_DT_F32 ? 4 : 2)) return MOE_ERR_MISALIGNED;
    // rows of [N, K] are 16-byte multiples (K: a multiple of 16), of [K, N] too (N: of 8)
    const bool vec = aligned(w, 16);
    const dim3 grid((K + 127) / 128, (N + 127) / 128, E);
    ProfScope prof_(MOE_K_QUANT_F8, stream);
    auto go = [&](auto kernel) {
        return launch_pdl(false, kernel, grid, dim3(256), 0, stream, w, w_dtype, N, K, q, s);
    };
    const cudaError_t e = transposed ? (vec ? go(quantize_weights_kernel<true, true>) : go(quantize_weights_kernel<false, true>))
                                     : (vec ? go(quantize_weights_kernel<true, false>) : go(quantize_weights_kernel<false, false>));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

// quantize_f8.cu — rows and weights to e4m3 with a scale for each block of 128:
// moe_quantize_f8 (rows, gathered by token for the experts' products) and
// moe_quantize_f8_weights (once, at load time).
//
// Rows: a warp takes up to 1024 columns of a row in 16-byte pieces, with all of its
// loads in flight first. The largest magnitudes of the 8 blocks of 128 in them are found
// together: halves of the lanes swap the partial maxima of half of the blocks, so that 5 exchanges
// (9 for fp32) do for all, and at the end every four lanes hold one block's and divide for it.
// 16-bit values are compared two at a time as they were read (bit patterns of magnitudes sort
// like the magnitudes, NaN above infinity), and widened only to be rounded.
// Bytes: 2 to 4 a value in, 1 out; a gathered row is read k times, from L2 for a prompt's x.
// Weights: a block of threads takes one 128 x 128 block into registers; given [K, N] it turns it
// in shared memory.
#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kChunk = 1024;             // columns a warp holds at once
constexpr int kSpan = 32 * 128;          // columns whose scales a warp gathers, one a lane

MOE_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Rounds columns c0 .. c0 + dc (<= kChunk) of a row; scales[g]: of the g-th 128 of them.
// FULL: dc is kChunk. DT: the values' type; PER of them are one piece of 16 bytes, and piece k of the
// lane holds columns (k * 32 + lane) * PER on. VEC: rows start on 16 bytes.
template <bool VEC, int DT, bool FULL>
MOE_DEV void round_chunk(const char* p, int dc, uint8_t* q, float* scales, int lane) {
    constexpr bool F32 = DT == MOE_DT_F32;
    constexpr int PER = F32 ? 4 : 8, N = kChunk / (32 * PER);  // pieces a lane
    uint4 raw[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int c = (k * 32 + lane) * PER;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (FULL || c < dc) {  // K is a multiple of 16
            if (VEC) {
                raw[k] = reinterpret_cast<const uint4*>(p)[k * 32 + lane];
            } else if (F32) {
                const uint32_t* x = reinterpret_cast<const uint32_t*>(p) + c;
                raw[k] = make_uint4(x[0], x[1], x[2], x[3]);
            } else {
                const uint16_t* x = reinterpret_cast<const uint16_t*>(p) + c;
                raw[k] = make_uint4(x[0] | uint32_t(x[1]) << 16, x[2] | uint32_t(x[3]) << 16,
                                    x[4] | uint32_t(x[5]) << 16, x[6] | uint32_t(x[7]) << 16);
            }
        }
    }
    // magnitudes: fp32 one a word, 16 bits two
    auto larger = [](uint32_t a, uint32_t b) { return F32 ? max(a, b) : max_u16x2(a, b); };
    constexpr uint32_t kMagnitude = F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    uint32_t m[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        m[k] = larger(larger(raw[k].x & kMagnitude, raw[k].y & kMagnitude),
                      larger(raw[k].z & kMagnitude, raw[k].w & kMagnitude));
    // a block of 128 columns: piece k of 32 lanes (fp32) or of 16. Lanes `o` apart keep the maxima of
    // half of the pieces each, until one is left: that of piece (lane >> 2) % N.
    int o = F32 ? 16 : 8;
#pragma unroll
    for (int h = N / 2; h >= 1; h >>= 1, o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const uint32_t keep = upper ? m[i + h] : m[i], give = upper ? m[i] : m[i + h];
            m[i] = larger(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
        }
    }
#pragma unroll
    for (; o >= 1; o >>= 1) m[0] = larger(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], o));
    uint32_t top = m[0];
    if (!F32) {
        top = max(top & 0xFFFFu, top >> 16);
        top = DT == MOE_DT_BF16 ? top << 16 : abs_bits(f16_lo(top));
    }
    const float scale = f8_scale(top);
    const F8Div mine(f8_divisor(top, scale));
    if ((lane & 3) == 0) scales[F32 ? lane >> 2 : (lane >> 2) % 4 * 2 + (lane >> 4)] = scale;
    const bool fast = __all_sync(0xFFFFFFFFu, mine.fast);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int from = F32 ? k * 4 : (lane & 16) | k * 4, c = (k * 32 + lane) * PER;
        F8Div div;
        div.s = __shfl_sync(0xFFFFFFFFu, mine.s, from);
        div.rs = __shfl_sync(0xFFFFFFFFu, mine.rs, from);
        div.fast = fast;  // not with a tiny, infinite or NaN scale among them
        if (!FULL && c >= dc) continue;
        if constexpr (F32) {
            const float v[4] = {__uint_as_float(raw[k].x), __uint_as_float(raw[k].y), __uint_as_float(raw[k].z),
                                __uint_as_float(raw[k].w)};
            *reinterpret_cast<uint32_t*>(q + c) = pack4_e4m3(v, div);
        } else {
            float v[8];
            unpack8(raw[k], DT == MOE_DT_BF16, v);
            *reinterpret_cast<uint2*>(q + c) = make_uint2(pack4_e4m3(v, div), pack4_e4m3(v + 4, div));
        }
    }
}

// RPW: rows a warp. 4 (many rows): their scales of a block of columns lie next to each other and
// leave 16 bytes at a time, where one row a warp writes 4 bytes of a sector at a time, as many of
// those as there are 128-byte pieces of q (8 rows a warp, whole sectors, leave a grid that does not
// fill the last SMs: 28.7 us where 4 take 26.3). 1 (few rows): a warp takes 1024 columns of a row (the
// grid's second dimension).
// 32768 rows of 2048 gathered from 4096 of bf16: 26.3 us, 2.55 TB/s of results; bound by the
// instructions' issue (8 a value: unpacking, three packed FMAs for two quotients, the conversion), a
// third of which are the ALU's.
template <bool VEC, int DT, int RPW>
__global__ void __launch_bounds__(256, DT == MOE_DT_F32 ? 3 : 4) quantize_rows_kernel(const void* x, int64_t ld, int64_t src_rows,
                                                            const int32_t* row_index, const int32_t* n_rows, int rows,
                                                            int K, uint8_t* q, float* s, uint32_t* err) {
    __shared__ float held[8][RPW][32 + 1];  // a warp's scales of a span: [row][group]
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    float(*mine)[33] = held[threadIdx.x >> 5];
    const int n = n_rows ? min(rows, max(0, *n_rows)) : rows;
    const bool wide = (reinterpret_cast<uintptr_t>(s) & 15) == 0 && rows % 4 == 0;
    const int units = int((uint32_t(n) + RPW - 1) / RPW), warps = gridDim.x * (blockDim.x >> 5);
    const int first = RPW > 1 ? 0 : int(blockIdx.y) * kChunk, last = RPW > 1 ? K : min(K, first + kChunk);
    bool bad = false;
    for (int64_t u = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < units; u += warps) {
        const int r0 = int(u) * RPW, nr = min(RPW, n - r0);
        int src = -1;
        if (lane < nr) {
            src = r0 + lane;
            if (row_index) {
                src = row_index[r0 + lane];
                if (src < 0 || src >= src_rows) {
                    bad = true;
                    src = -1;
                }
            }
        }
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, src >= 0);  // rows to write
        for (int c0 = first; c0 < last; c0 += kSpan) {
            const int end = min(last, c0 + kSpan);
#pragma unroll 1
            for (int i = 0; i < RPW; ++i) {
                const int row = __shfl_sync(0xFFFFFFFFu, src, i);
                if (row < 0) continue;
#pragma unroll 1
                for (int c = c0; c < end; c += kChunk) {
                    const char* p = static_cast<const char*>(x) + (row * ld + c) * (DT == MOE_DT_F32 ? 4 : 2);
                    uint8_t* qp = q + int64_t(r0 + i) * K + c;
                    float* sc = mine[i] + ((c - c0) >> 7);
                    if (end - c >= kChunk) round_chunk<VEC, DT, true>(p, kChunk, qp, sc, lane);
                    else round_chunk<VEC, DT, false>(p, end - c, qp, sc, lane);
                }
            }
            __syncwarp();
            const int g = c0 / 128 + lane;
            if (g * 128 < last) {
                float* sp = s + int64_t(g) * rows + r0;
                if (RPW == 4 && ok == 0xFu && wide) {
                    *reinterpret_cast<float4*>(sp) = make_float4(mine[0][lane], mine[1 % RPW][lane], mine[2 % RPW][lane], mine[3 % RPW][lane]);
                } else {
#pragma unroll
                    for (int i = 0; i < RPW; ++i)
                        if (ok >> i & 1u) sp[i] = mine[i][lane];
                }
            }
            __syncwarp();
        }
    }
    if (bad) set_error(err, MOE_DEVERR_BOUNDS);
}

// One 128 x 128 block of a matrix of `rows` x `cols` (row-major): thread t holds the 8 columns
// (t & 15) * 8 of the 8 rows (t >> 4) * 8 on. TURN: the matrix is [K, N] and the result its transpose;
// a thread's 8 values along K of a column are 8 neighbouring bytes of it, rounded two at a time along
// K, and pass through shared memory: chunk c of column n's 128 bytes at n*128 + 8 (c ^ n/8 % 16), so
// that a half warp's writes, eight columns apart, fall in all the banks.
// The values stay in registers as they were read (F32: 8 words a row, else 4) between the block's
// largest magnitude and their rounding.
template <bool F32>
MOE_DEV void widen(const uint4 (&r)[F32 ? 2 : 1], bool bf16, float (&v)[8]) {
    if (F32) {
        const uint4 a = r[0], b = r[F32 ? 1 : 0];
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        unpack8(r[0], bf16, v);
    }
}

template <bool VEC, bool TURN, bool F32>
__global__ void __launch_bounds__(256, F32 ? 2 : 4) quantize_weights_kernel(const void* w, int w_dt, int N, int K,
                                                                            uint8_t* q, float* s) {
    __shared__ uint32_t wmax[8];
    __shared__ __align__(16) uint8_t turn[TURN ? 128 * 128 : 16];
    griddep_wait();
    griddep_launch();
    const int e = blockIdx.z, nb = blockIdx.y, kb = blockIdx.x;
    const int rows = TURN ? K : N, cols = TURN ? N : K;
    const int r0 = (TURN ? kb : nb) * 128, c0 = (TURN ? nb : kb) * 128;
    const int cx = (threadIdx.x & 15) * 8, ry = (threadIdx.x >> 4) * 8;
    const int64_t base = int64_t(e) * N * K;
    const bool bf16 = w_dt == MOE_DT_BF16;
    uint4 raw[8][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + ry + i, c = c0 + cx;
        const int64_t at = base + int64_t(r) * cols + c;
        const bool in = r < rows && c < cols;  // cols: a multiple of 8
#pragma unroll
        for (int h = 0; h < (F32 ? 2 : 1); ++h) {
            raw[i][h] = make_uint4(0, 0, 0, 0);
            if (!in) continue;
            if (VEC) {
                raw[i][h] = F32 ? *reinterpret_cast<const uint4*>(static_cast<const float*>(w) + at + 4 * h)
                                : *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at);
            } else if (F32) {
                const uint32_t* p = static_cast<const uint32_t*>(w) + at + 4 * h;
                raw[i][h] = make_uint4(p[0], p[1], p[2], p[3]);
            } else {
                const uint16_t* p = static_cast<const uint16_t*>(w) + at;
                raw[i][h] = make_uint4(p[0] | uint32_t(p[1]) << 16, p[2] | uint32_t(p[3]) << 16, p[4] | uint32_t(p[5]) << 16,
                                       p[6] | uint32_t(p[7]) << 16);
            }
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        widen<F32>(raw[i], bf16, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, wmax[i]);
    const float scale = f8_scale(m);
    const F8Div div(f8_divisor(m, scale));
    if (threadIdx.x == 0) s[(int64_t(e) * gridDim.y + nb) * gridDim.x + kb] = scale;
    if (!TURN) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + ry + i, c = c0 + cx;
            float v[8];
            widen<F32>(raw[i], bf16, v);
            if (r < rows && c < cols)
                *reinterpret_cast<uint2*>(q + base + int64_t(r) * K + c) = make_uint2(pack4_e4m3(v, div), pack4_e4m3(v + 4, div));
        }
    } else {
        // two rows' bytes of each column at a time, then 8 rows' bytes of a column
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) lo[j] = hi[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float a[8], b[8];
            widen<F32>(raw[i], bf16, a);
            widen<F32>(raw[i + 1], bf16, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t two = div.fast ? pack_e4m3x2(div(a[j]), div(b[j])) : pack_e4m3x2(__fdiv_rn(a[j], div.s), __fdiv_rn(b[j], div.s));
                if (i < 4) lo[j] |= two << (8 * i);
                else hi[j] |= two << (8 * (i - 4));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = cx + j;
            *reinterpret_cast<uint2*>(turn + n * 128 + (((ry >> 3) ^ ((n >> 3) & 15)) << 3)) = make_uint2(lo[j], hi[j]);
        }
        __syncthreads();
        // 16 bytes of K of one column of N a thread and step
        for (int i = threadIdx.x; i < 128 * 8; i += 256) {
            const int n = i >> 3, k = (i & 7) * 16, x = (n >> 3) & 15;
            if (c0 + n >= N || r0 + k >= K) continue;  // K is a multiple of 16
            const uint2 p = *reinterpret_cast<const uint2*>(turn + n * 128 + (((k >> 3) ^ x) << 3));
            const uint2 p2 = *reinterpret_cast<const uint2*>(turn + n * 128 + ((((k >> 3) + 1) ^ x) << 3));
            *reinterpret_cast<uint4*>(q + base + int64_t(c0 + n) * K + r0 + k) = make_uint4(p.x, p.y, p2.x, p2.y);
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
    if (rows < 0 || rows >= (int64_t(1) << 31) || K < 16 || K % 16 || src_rows < 0 || K > MOE_F8_MAX_K)
        return MOE_ERR_INVALID_ARG;
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
    const bool vec = aligned(x, 16) && ld * int64_t(es) % 16 == 0;
    // 4 rows a warp once that gives every scheduler of every SM eight warps
    const bool many = rows >= int64_t(num_sms()) * 32 * 4;
    const int64_t units = many ? (rows + 3) / 4 : rows;
    const dim3 grid(int(std::min<int64_t>((units + 7) / 8, int64_t(num_sms()) * 8)), many ? 1 : (K + kChunk - 1) / kChunk);
    ProfScope prof_(MOE_K_QUANT_F8, stream);
    auto go = [&](auto kernel) {
        return launch_pdl(use_pdl(rows), kernel, grid, dim3(256), 0, stream, x, ld, src_rows, row_index, n_rows,
                          int(rows), K, q, s, static_cast<uint32_t*>(ws));
    };
    auto pick = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return many ? (vec ? go(quantize_rows_kernel<true, DT, 4>) : go(quantize_rows_kernel<false, DT, 4>))
                    : (vec ? go(quantize_rows_kernel<true, DT, 1>) : go(quantize_rows_kernel<false, DT, 1>));
    };
    const cudaError_t e = x_dtype == MOE_DT_F32    ? pick(std::integral_constant<int, MOE_DT_F32>{})
                          : x_dtype == MOE_DT_BF16 ? pick(std::integral_constant<int, MOE_DT_BF16>{})
                                                   : pick(std::integral_constant<int, MOE_DT_F16>{});
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_quantize_f8_weights(int32_t E, int32_t N, int32_t K, const void* w, int32_t w_dtype, int32_t transposed,
                            uint8_t* q, float* s, moe_stream_t stream) {
    if (E < 1 || E > 65535 || N < 8 || N % 8 || K < 16 || K % 16 || K > MOE_F8_MAX_K || (transposed != 0 && transposed != 1))
        return MOE_ERR_INVALID_ARG;
    if (w_dtype < MOE_DT_F32 || w_dtype > MOE_DT_F16) return MOE_ERR_INVALID_ARG;
    if ((int64_t(N) + 127) / 128 > 65535 || int64_t(N) * K >= (int64_t(1) << 40)) return MOE_ERR_INVALID_ARG;
    if (!w || !q || !s) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(s, 4) || !aligned(w, w_dtype == MOE_DT_F32 ? 4 : 2)) return MOE_ERR_MISALIGNED;
    // rows of [N, K] are 16-byte multiples (K: a multiple of 16), of [K, N] too (N: of 8)
    const bool vec = aligned(w, 16);
    const dim3 grid((K + 127) / 128, (N + 127) / 128, E);
    ProfScope prof_(MOE_K_QUANT_F8, stream);
    auto go = [&](auto kernel) {
        return launch_pdl(false, kernel, grid, dim3(256), 0, stream, w, w_dtype, N, K, q, s);
    };
    cudaError_t e;
    if (w_dtype == MOE_DT_F32)
        e = transposed ? (vec ? go(quantize_weights_kernel<true, true, true>) : go(quantize_weights_kernel<false, true, true>))
                       : (vec ? go(quantize_weights_kernel<true, false, true>) : go(quantize_weights_kernel<false, false, true>));
    else
        e = transposed ? (vec ? go(quantize_weights_kernel<true, true, false>) : go(quantize_weights_kernel<false, true, false>))
                       : (vec ? go(quantize_weights_kernel<true, false, false>) : go(quantize_weights_kernel<false, false, false>));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

// f8_stream.cu — the 8-bit products for a few rows (single tokens): every weight
// byte is read once, straight into registers, and the time is HBM's.
//
// A block takes one or two strips of 16 columns of the result (16 rows of the K-major
// weights, of both projections when gated) and up to 8 rows of one expert; its 8 warps take every
// eighth block of 128 along K. A lane loads 16 bytes of weights at a time; they
// are the A operand of mma.sync m16n8k32 (e4m3) as they come: the fragment wants
// 4 bytes of K at tig*4 and at 16 + tig*4, but a sum over K may take K in any order,
// so lane tig holds bytes 16 tig.. of a 64-byte piece and feeds them to two products,
// with the same bytes of the 8 rows as the B operand. Nothing passes through shared
// memory. A block of 128 is summed from zero, multiplied by its two scales and added
// in fp32; the 8 warps' sums are added in order at the end (no atomics).
//
// A block is small (8 warps of 64 to 85 registers), so that three or four of them share
// an SM and one's start and joint hide behind the others' loads. One row of 8 experts,
// gate and up of 1536 x 4096 (100 MB): 23.0 us with 16-bit results, 4.4 TB/s (two blocks of 128
// registers 26.1; one persistent block with copies ahead through shared memory 40), 26.2 with e4m3
// ones; down of 4096 x 1536 15.4 us (three blocks an SM, one strip each, 22.5). One dense row, 4096 ->
// 1536: 3.7 us. Pieces of 128 bytes of rows 4 KB apart, as here, are read at 5.2 TB/s by a kernel
// that does nothing else.
// Gated with e4m3 results needs the largest of 128 columns: the blocks that hold them are one
// cluster and exchange their maxima through its shared memory.
#include <algorithm>

#include "f8.cuh"

namespace moe {

namespace f8 {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCols = 16;   // columns of the result per block
constexpr int kRows = 8;    // rows per block
MOE_DEV void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

MOE_DEV uint4 ld_weights(const uint8_t* p, bool in) {
    // read once: past L1
    return in ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// Blocks of `chunk` rows of the experts, in the experts' order: block `u` is rows
// [row0, row0 + n) of expert e; false past the last one. Every thread of a block of
// at least 256 threads calls it (E <= 256: one expert a thread, one pass of scans;
// a search by row would be a chain of dependent loads). sm: 12 ints.
MOE_DEV bool find_rows(const Args& p, int u, int chunk, int* sm, int& e, int64_t& row0, int& n) {
    if (!p.offsets) {
        e = 0;
        row0 = int64_t(u) * chunk;
        n = int(min(int64_t(chunk), p.rows - row0));
        return n > 0;
    }
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int off = 0, cnt = 0;
    if (t < p.E) {
        off = __ldg(p.offsets + t);
        cnt = __ldg(p.offsets + t + 1) - off;
        // offsets outside the buffers (never from moe_permute) are not followed
        if (off < 0 || cnt < 0 || int64_t(off) + cnt > p.rows) {
            set_error(p.err, MOE_DEVERR_BOUNDS);
            cnt = 0;
        }
    }
    const int c = int((uint32_t(cnt) + chunk - 1) / chunk);
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += v;
    }
    if (warp < 8 && lane == 31) sm[warp] = s;
    if (t == 0) sm[8] = -1;
    __syncthreads();
    if (warp < 8) {
        for (int w = 0; w < warp; ++w) s += sm[w];
        const int first = s - c;
        if (u >= first && u < s) {
            const int m = u - first;
            sm[8] = t;
            sm[9] = off + m * chunk;
            sm[10] = min(chunk, cnt - m * chunk);
        }
    }
    __syncthreads();
    e = sm[8];
    row0 = sm[9];
    n = sm[10];
    return e >= 0;
}

// S: strips of 16 columns a block, one after the other; G blocks have 128 columns (the cluster of the
// e4m3 form).
template <bool GATED, bool E4M3, int S>
__global__ void __launch_bounds__(kThreads, GATED ? 3 : 4) f8_stream_kernel(const Args p) {
    constexpr int M = GATED ? 2 : 1;
    __shared__ int found[12];
    constexpr int G = 128 / (S * kCols);
    __shared__ float part[S][kWarps][M][kRows][kCols + 1];
    __shared__ uint32_t amax[S][kRows];
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    int e, nr;
    int64_t row0;
    // the same chunks of rows for every block of a cluster: they leave together
    for (int u = blockIdx.y; find_rows(p, u, kRows, found, e, row0, nr); u += gridDim.y) {
#pragma unroll 1
        for (int strip = 0; strip < S; ++strip) {
            const int n0 = (blockIdx.x * S + strip) * kCols;
            float acc[M][4];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
            const bool in0 = n0 + gid < p.N, in1 = n0 + 8 + gid < p.N, inr = gid < nr;
            const int64_t w0 = (int64_t(e) * p.N + n0 + gid) * p.K + tig * 16;
            const int64_t w8 = w0 + int64_t(8) * p.K;
            const uint8_t* arow = p.a + (row0 + gid) * p.K + tig * 16;
            const int r0 = min(2 * tig, nr - 1), r1 = min(2 * tig + 1, nr - 1);  // columns of the product past nr are not kept
            const int sb0 = (e * p.NB + n0 / 128) * p.KB;
#pragma unroll 1
            for (int kb = warp; kb < p.KB; kb += kWarps) {
                const int k = kb * 128;
                const bool ka = k + tig * 16 < p.K, kc = k + 64 + tig * 16 < p.K;
                uint4 w[M][4], x[2];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    w[m][0] = ld_weights(p.b[m] + w0 + k, in0 && ka);
                    w[m][1] = ld_weights(p.b[m] + w8 + k, in1 && ka);
                    w[m][2] = ld_weights(p.b[m] + w0 + k + 64, in0 && kc);
                    w[m][3] = ld_weights(p.b[m] + w8 + k + 64, in1 && kc);
                }
                x[0] = inr && ka ? __ldg(reinterpret_cast<const uint4*>(arow + k)) : make_uint4(0, 0, 0, 0);
                x[1] = inr && kc ? __ldg(reinterpret_cast<const uint4*>(arow + k + 64)) : make_uint4(0, 0, 0, 0);
                const float* as = p.a_scale + int64_t(kb) * p.rows + row0;
                const float s0 = __ldg(as + r0), s1 = __ldg(as + r1);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float sb = __ldg(p.b_scale[m] + sb0 + kb);
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma_e4m3(c, w[m][2 * h].x, w[m][2 * h + 1].x, w[m][2 * h].y, w[m][2 * h + 1].y, x[h].x, x[h].y);
                        mma_e4m3(c, w[m][2 * h].z, w[m][2 * h + 1].z, w[m][2 * h].w, w[m][2 * h + 1].w, x[h].z, x[h].w);
                    }
                    acc[m][0] = fmaf(c[0], sb * s0, acc[m][0]);
                    acc[m][1] = fmaf(c[1], sb * s1, acc[m][1]);
                    acc[m][2] = fmaf(c[2], sb * s0, acc[m][2]);
                    acc[m][3] = fmaf(c[3], sb * s1, acc[m][3]);
                }
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                part[strip][warp][m][2 * tig][gid] = acc[m][0];
                part[strip][warp][m][2 * tig + 1][gid] = acc[m][1];
                part[strip][warp][m][2 * tig][gid + 8] = acc[m][2];
                part[strip][warp][m][2 * tig + 1][gid + 8] = acc[m][3];
            }
        }
        __syncthreads();
        // one value a thread: strip i / 128, row i / 16 % 8, column i % 16
        const int i = threadIdx.x, strip = i / (kRows * kCols), r = i / kCols % kRows, c = i % kCols;
        const int col = (blockIdx.x * S + strip) * kCols + c;
        const bool mine = strip < S, keep = mine && r < nr && col < p.N;
        float v = 0.f;
        if (mine) {
            float s[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                s[m] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s[m] += part[strip][w][m][r][c];
            }
            if constexpr (GATED) v = gated(s[0], s[1], p.limit);
            else v = s[0];
        }
        if constexpr (!E4M3) {
            if (keep) {
                if constexpr (!GATED) v *= row_weight(p, row0 + r);
                store_out(p, row0 + r, col, v);
            }
        } else {
            // the row's largest of these 16 columns, then of the cluster's 128
            uint32_t m = keep ? abs_bits(v) : 0u;
#pragma unroll
            for (int o = 1; o < kCols; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (mine && c == 0) amax[strip][r] = m;  // one strip: half of the threads have none
            cluster_sync_all();
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const uint32_t place = smem_u32(&amax[k][r]);
#pragma unroll
                for (int b = 0; b < G; ++b) {
                    uint32_t o;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(o) : "r"(mapa_shared(place, b)));
                    m = max(m, o);
                }
            }
            cluster_sync_all();  // no block leaves while another reads its maxima
            if (keep) {
                const float sc = f8_scale(m);
                const F8Div div(f8_divisor(m, sc));
                static_cast<uint8_t*>(p.out)[(row0 + r) * p.N + col] =
                    uint8_t(pack_e4m3x2(div.fast ? div(v) : __fdiv_rn(v, sc), 0.f) & 0xFFu);
                if (col % 128 == 0) p.h_scale[int64_t(col / 128) * p.rows + row0 + r] = sc;
            }
        }
        __syncthreads();  // found, part and amax are written anew
    }
}

}  // namespace

cudaError_t launch_stream(const Args& p, bool gated, cudaStream_t s) {
    const bool e4m3 = p.out_dt == MOE_DT_E4M3;
    // at most one partial chunk an expert beside the full ones
    const int64_t chunks = p.offsets ? std::min<int64_t>(p.rows, p.E) + p.rows / kRows : (p.rows + kRows - 1) / kRows;
    // Two strips a block once one would give more blocks than run at once: fewer waves, starts and joints.
    // One row of 8 experts: down of 4096 x 1536 17.8 us with one, 15.4 with two; gate and up of 1536 x 4096
    // with e4m3 results 30.7 and 26.2, with bf16 ones 23.6 and 23.0. One dense row, 4096 -> 1536: 3.7 and 5.1.
    const int64_t ones = e4m3 ? p.NB * 8 : (p.N + kCols - 1) / kCols;
    const int S = ones * chunks > int64_t(num_sms()) * (gated ? 3 : 4) ? 2 : 1;
    const int strips = int((ones + S - 1) / S);
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = use_pdl(p.rows) ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 8 / S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = e4m3 ? 2 : 1;
    cfg.gridDim = dim3(strips, unsigned(std::min<int64_t>(chunks, 65535)));
    ProfScope prof_(MOE_K_STREAM_F8, s);
    auto go = [&](auto one, auto two) { return cudaLaunchKernelEx(&cfg, S == 1 ? one : two, p); };
    return !gated ? go(f8_stream_kernel<false, false, 1>, f8_stream_kernel<false, false, 2>)
           : e4m3 ? go(f8_stream_kernel<true, true, 1>, f8_stream_kernel<true, true, 2>)
                  : go(f8_stream_kernel<true, false, 1>, f8_stream_kernel<true, false, 2>);
}

}  // namespace f8

}  // namespace moe

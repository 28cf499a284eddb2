// f8.cuh — what the 8-bit products' kernels share (f8_stream.cu: a few rows;
// f8_tile.cu: tcgen05 tiles; f8.cu: the entry points).
#pragma once

#include "rows.cuh"

namespace moe {

namespace f8 {

struct Args {
    const uint8_t* a;         // [rows, K]
    const float* a_scale;     // [KB, rows]
    const int32_t* offsets;   // [E+1], or null: one dense product of all rows
    const uint8_t* b[2];      // [E, N, K]; gated: gate, up
    const float* b_scale[2];  // [E, NB, KB]
    const int32_t* sorted_pair;
    const float* topk_w;
    void* out;                // [rows, N] out_dt
    float* h_scale;           // out_dt e4m3: [NB, rows]
    int64_t rows;
    int K, N, E, KB, NB;      // KB, NB: blocks of 128
    int out_dt;
    float limit;              // of the gated form; infinity: none
    uint32_t* err;
    uint64_t wait_ns;
};

// min and max that keep a NaN
MOE_DEV float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
MOE_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// silu(clamp(g)) clamp(u); L: the limit, infinity without one. The exponential and the
// reciprocal are the hardware's approximate ones: relative error about 1e-6 (as in the bf16
// kernels), far below the rounding of the results to 16 or 8 bits.
MOE_DEV float gated(float g, float u, float L) {
    g = max_nan(min_nan(g, L), -L);
    u = max_nan(min_nan(u, L), -L);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-g)));
    return g * u * r;
}

// The gate weight of a row (1 without).
MOE_DEV float row_weight(const Args& p, int64_t row) {
    if (!p.sorted_pair) return 1.0f;
    const int sp = __ldg(p.sorted_pair + row);
    return sp >= 0 ? __ldg(p.topk_w + sp) : 1.0f;
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
    const int c = (cnt + chunk - 1) / chunk;
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

// One output value.
MOE_DEV void store_out(const Args& p, int64_t row, int col, float v) {
    const int64_t i = row * p.N + col;
    if (p.out_dt == MOE_DT_F16 && !f16_range_ok(v)) set_error(p.err, MOE_DEVERR_RANGE);
    store_elem(p.out, i, v, p.out_dt);
}

cudaError_t launch_stream(const Args& p, bool gated, cudaStream_t s);
cudaError_t launch_tile(const Args& p, bool gated, cudaStream_t s);

}  // namespace f8

}  // namespace moe

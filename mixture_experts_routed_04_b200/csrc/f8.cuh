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
    int copies;               // tiles: blocks along K a CTA's producer brings; -1: all (else moe_f8_wait_selftest)
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
// kernels), far below the rounding of the results to 16 or 8 bits. silu(g) first: g u alone may pass
// the largest fp32 value where the result does not (g = -50, u = 1e38).
MOE_DEV float gated(float g, float u, float L) {
    g = max_nan(min_nan(g, L), -L);
    u = max_nan(min_nan(u, L), -L);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-g)));
    return g * r * u;
}

// The gate weight of a row (1 without).
MOE_DEV float row_weight(const Args& p, int64_t row) {
    if (!p.sorted_pair) return 1.0f;
    const int sp = __ldg(p.sorted_pair + row);
    return sp >= 0 ? __ldg(p.topk_w + sp) : 1.0f;
}

// The experts' blocks of `chunk` rows: exclusive prefix of their numbers and the experts' row offsets.
struct Chunks {
    int base[kMaxE + 1];
    int off[kMaxE + 1];
    int warp_sum[32];
};
// Fills c; every thread of a block of at least 256 threads calls it (E <= 256: one expert a thread,
// one pass of scans). Offsets outside the buffers (never from moe_permute) are reported and not
// followed. The caller synchronises the block before it reads c.
MOE_DEV void count_chunks(const Args& p, int chunk, Chunks& c) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int cnt = 0;
    if (!p.offsets) {
        if (t == 0) {
            cnt = int((p.rows + chunk - 1) / chunk);
            c.off[0] = 0;
            c.off[1] = int(p.rows);
        }
    } else if (t < p.E) {
        const int off = __ldg(p.offsets + t), end = __ldg(p.offsets + t + 1);
        c.off[t] = off;
        if (t == p.E - 1) c.off[t + 1] = end;
        if (off < 0 || end < off || end > p.rows) set_error(p.err, MOE_DEVERR_BOUNDS);
        else cnt = int((uint32_t(end - off) + chunk - 1) / chunk);
    }
    int s = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += v;
    }
    if (lane == 31) c.warp_sum[warp] = s;
    __syncthreads();
    for (int w = 0; w < warp; ++w) s += c.warp_sum[w];
    if (t < p.E) c.base[t + 1] = s;
    if (t == 0) c.base[0] = 0;
}
// The expert of chunk u < base[E].
MOE_DEV int expert_of(const Chunks& c, int u, int E) {
    int lo = 0, hi = E;  // base[lo] <= u < base[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c.base[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
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

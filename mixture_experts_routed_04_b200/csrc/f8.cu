// f8.cu — entry points of the products in 8-bit floating point: argument checks and
// the choice between the streaming kernels (f8_stream.cu) and the tiles (f8_tile.cu).
#include <algorithm>
#include <cmath>
#include <limits>

#include "f8.cuh"

namespace moe {

namespace f8 {

namespace {

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_params(const moe_f8_params* p) {
    if (!p || p->rows < 0 || p->rows >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
    if (p->K < 16 || p->K % 16 || p->K > MOE_F8_MAX_K || p->N < 8 || p->N % 8 || p->E < 1 || p->E > kMaxE)
        return MOE_ERR_INVALID_ARG;
    if (p->out_dtype < MOE_DT_F32 || p->out_dtype > MOE_DT_E4M3) return MOE_ERR_INVALID_ARG;
    if (p->variant < MOE_VARIANT_AUTO || p->variant > MOE_VARIANT_STREAM) return MOE_ERR_INVALID_ARG;
    if (!(p->swiglu_limit >= -3.4e38f && p->swiglu_limit <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    // weight rows, rounded up to tiles of 256, and scale blocks are counted in 32 bits
    if (int64_t(p->N) * p->E > (int64_t(1) << 31) - 256) return MOE_ERR_INVALID_ARG;
    if ((int64_t(p->N) + 127) / 128 * ((p->K + 127) / 128) * p->E >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_call(const moe_f8_params* p, const uint8_t* a, const float* a_scale, const int32_t* offsets, const void* out,
               const void* ws, size_t ws_bytes) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!al(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < moe_f8_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (p->rows == 0) return MOE_OK;
    if (!a || !a_scale || !out || (p->E > 1 && !offsets)) return MOE_ERR_INVALID_ARG;
    if (!al(a, 16) || !al(a_scale, 4) || !al(offsets, 4) || !al(out, 16)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

int check_weights(const uint8_t* b, const float* s) {
    if (!b || !s) return MOE_ERR_INVALID_ARG;
    return al(b, 16) && al(s, 4) ? MOE_OK : MOE_ERR_MISALIGNED;
}

Args args_of(const moe_f8_params* p, const uint8_t* a, const float* a_scale, const int32_t* offsets, void* out,
             void* ws) {
    Args x{};
    x.a = a;
    x.a_scale = a_scale;
    x.offsets = offsets;
    x.out = out;
    x.rows = p->rows;
    x.K = p->K;
    x.N = p->N;
    x.E = p->E;
    x.KB = (p->K + 127) / 128;
    x.NB = (p->N + 127) / 128;
    x.out_dt = p->out_dtype;
    x.limit = p->swiglu_limit > 0.f ? p->swiglu_limit : std::numeric_limits<float>::infinity();
    x.err = static_cast<uint32_t*>(ws);
    x.wait_ns = wait_limit_ns();
    x.copies = -1;
    return x;
}

// The streaming kernel reads an expert's weights once a chunk of 8 rows; the tiles walk K block by
// block, each tile's blocks one after the other, however few its rows are. Estimates in us of B200
// runs (stream / tiles): one dense product of 4096 x 4096, 8 rows 5.2 / 21.6, 32 rows 12.0 / 21.6,
// 128 rows 39 / 24; 1024 x 1024, 128 rows 5.8 / 10.2; 768 -> 8192, 32 rows 7.7 / 7.4; 8 experts' gate
// and up of 1536 x 4096, one row each 26.3 / 34 to 39, 64 experts with two rows each 189 / 150; down of
// 4096 x 1536, 8 experts 15.5 / 15.4 to 17.7.
bool takes_stream(const Args& x, bool gated) {
    const double touched = double(std::min<int64_t>(x.rows, x.E));
    const double chunks = x.offsets ? std::max(touched, x.rows / 8.0) : std::ceil(x.rows / 8.0);
    const double bytes = double(x.N) * x.K * (gated ? 2 : 1), sms = num_sms();
    const bool dense = !x.offsets;  // its chunks find the weights in L2 after the first
    const double stream_us = 2.0 + chunks * bytes / (dense ? 6.0e6 : 3.6e6);
    const double tiles = std::max(touched, x.rows / 128.0) * std::ceil(x.N / (gated ? 128.0 : 256.0));
    const double tile_us = 3.0 + (dense ? 0.6 : 1.0) * x.KB * std::ceil(tiles / sms);
    return stream_us < tile_us;
}

int launch(const moe_f8_params* p, const Args& x, bool gated, cudaStream_t s) {
    const bool stream = p->variant == MOE_VARIANT_STREAM || (p->variant == MOE_VARIANT_AUTO && takes_stream(x, gated));
    return (stream ? launch_stream(x, gated, s) : launch_tile(x, gated, s)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

}  // namespace f8

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_f8_workspace_size(const moe_f8_params* p) { return f8::check_params(p) == MOE_OK ? 256 : 0; }

int moe_matmul_f8(const moe_f8_params* p, const uint8_t* a, const float* a_scale, const int32_t* offsets,
                  const uint8_t* b, const float* b_scale, const int32_t* sorted_pair, const float* topk_w, void* out,
                  void* ws, size_t ws_bytes, moe_stream_t stream) {
    int st = f8::check_params(p);
    if (st != MOE_OK) return st;
    if (p->out_dtype == MOE_DT_E4M3) return MOE_ERR_UNSUPPORTED;  // its 128 columns' scale is the gated form's
    if ((st = f8::check_call(p, a, a_scale, offsets, out, ws, ws_bytes)) != MOE_OK || p->rows == 0) return st;
    if ((st = f8::check_weights(b, b_scale)) != MOE_OK) return st;
    if (!sorted_pair != !topk_w) return MOE_ERR_INVALID_ARG;
    if (!f8::al(sorted_pair, 4) || !f8::al(topk_w, 4)) return MOE_ERR_MISALIGNED;
    f8::Args x = f8::args_of(p, a, a_scale, offsets, out, ws);
    x.b[0] = x.b[1] = b;
    x.b_scale[0] = x.b_scale[1] = b_scale;
    x.sorted_pair = sorted_pair;
    x.topk_w = topk_w;
    return f8::launch(p, x, false, stream);
}

int moe_gated_f8(const moe_f8_params* p, const uint8_t* a, const float* a_scale, const int32_t* offsets,
                 const uint8_t* w_gate, const float* s_gate, const uint8_t* w_up, const float* s_up, void* h,
                 float* h_scale, void* ws, size_t ws_bytes, moe_stream_t stream) {
    int st = f8::check_params(p);
    if (st != MOE_OK) return st;
    const bool e4m3 = p->out_dtype == MOE_DT_E4M3;
    if (e4m3 && p->N % 16) return MOE_ERR_INVALID_ARG;
    if ((st = f8::check_call(p, a, a_scale, offsets, h, ws, ws_bytes)) != MOE_OK || p->rows == 0) return st;
    if ((st = f8::check_weights(w_gate, s_gate)) != MOE_OK || (st = f8::check_weights(w_up, s_up)) != MOE_OK) return st;
    if (e4m3 != (h_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!f8::al(h_scale, 4)) return MOE_ERR_MISALIGNED;
    f8::Args x = f8::args_of(p, a, a_scale, offsets, h, ws);
    x.b[0] = w_gate;
    x.b[1] = w_up;
    x.b_scale[0] = s_gate;
    x.b_scale[1] = s_up;
    x.h_scale = h_scale;
    return f8::launch(p, x, true, stream);
}

int moe_f8_wait_selftest(int32_t gated, int32_t blocks, uint64_t limit_ns, void* ws, size_t ws_bytes,
                         moe_stream_t stream) {
    // three M-tiles and two n-tiles, the last M-tile partial, 8 blocks along K, all in the workspace
    constexpr int R = 300, K = 1024, N = 256, KB = K / 128, NB = N / 128;
    if (!ws || blocks < 0 || blocks >= KB || limit_ns == 0 || limit_ns > 10000000000ull) return MOE_ERR_INVALID_ARG;
    if (!f8::al(ws, 256)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < MOE_F8_SELFTEST_BYTES) return MOE_ERR_WORKSPACE_TOO_SMALL;
    uint8_t* at = static_cast<uint8_t*>(ws) + 256;
    auto take = [&](size_t n) {
        uint8_t* r = at;
        at += (n + 255) & ~size_t(255);
        return r;
    };
    const uint8_t* a = take(size_t(R) * K);
    const uint8_t* b = take(size_t(N) * K);
    const float* a_scale = reinterpret_cast<float*>(take(size_t(KB) * R * 4));
    const float* b_scale = reinterpret_cast<float*>(take(size_t(NB) * KB * 4));
    float* h_scale = reinterpret_cast<float*>(take(size_t(NB) * R * 4));
    void* out = take(size_t(R) * N * 4);
    static_assert(256 + R * K + N * K + KB * R * 4 + NB * KB * 4 + NB * R * 4 + R * N * 4 + 6 * 255 <= MOE_F8_SELFTEST_BYTES,
                  "the workspace holds every tensor");
    moe_f8_params p{};
    p.rows = R; p.K = K; p.N = N; p.E = 1;
    p.out_dtype = gated ? MOE_DT_E4M3 : MOE_DT_F32;
    f8::Args x = f8::args_of(&p, a, a_scale, nullptr, out, ws);
    x.b[0] = x.b[1] = b;
    x.b_scale[0] = x.b_scale[1] = b_scale;
    x.h_scale = gated ? h_scale : nullptr;
    x.wait_ns = limit_ns;
    x.copies = blocks;
    return f8::launch_tile(x, gated != 0, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

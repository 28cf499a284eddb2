// f8_tile.cu — the 8-bit products on the tcgen05 tensor cores: 128 rows of an
// expert x 256 weight rows a tile (gated: 128 of gate and 128 of up), persistent,
// one CTA an SM.
//
//   warp 0     TMA producer: per block of 128 along K, the 128 x 128 bytes of the
//              rows and the 256 x 128 bytes of the weights (128-byte swizzle; past
//              K and N zeros come in), 4 stages of 48 KB.
//   warp 1     TMEM and the MMAs: tcgen05.mma kind::f8f6f4, M=128 N=256 K=32, four
//              a block. Every block of 128 is summed from zero into one of two
//              256-column accumulators, because its scales are its own.
//   warps 2-9  the sums: each block's accumulator leaves TMEM as soon as it is done,
//              is multiplied by its two scales and added in fp32 registers (128
//              columns of one row a thread), while the MMAs fill the other one. The
//              scaled sum takes about as many issue slots (128 packed fp32 FMAs and 4
//              loads of 32 columns a warp and block) as half the MMAs' time (512 cycles
//              a block), so the tensor pipe stays the longer one.
//              After the last block: the gate weight or the clamped SwiGLU, the
//              rounding, and the store, turned through 2 KB of shared memory a warp so
//              that a store writes 64-byte pieces of 8 rows (32 rows of 16 bytes each
//              would take 32 passes of the load/store unit).
//
// Gated with e4m3 results: a row's 128 columns lie in two threads (two warps of a
// lane quadrant), which exchange their maxima over a barrier of those two warps.
// Units (expert, n-tile, M-tile; M fastest, so that neighbours share the weights in
// L2) are all alike in length and dealt out by index: no counter, no workspace.
#include <algorithm>

#include "f8.cuh"
#include "tmap.h"

namespace moe {

namespace f8 {

namespace {

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int EPI = 8, THREADS = 32 * (2 + EPI);
constexpr int PIECE = 32 * 64;  // a warp's turn buffer: 32 rows of 64 bytes
constexpr int OFF_TURN = STAGES * STAGE;
constexpr int OFF_MISC = OFF_TURN + EPI * PIECE;
constexpr int MISC = 4096;
constexpr int SMEM = 1024 + OFF_MISC + MISC;
static_assert(SMEM <= 232448, "dynamic shared memory a block may opt into");

// kind::f8f6f4, e4m3 x e4m3 -> f32, both operands K-major.
constexpr uint32_t kIdesc = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);

MOE_DEV void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
        : "memory");
}

struct Misc {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t tfull[2], tempty[2];
    uint64_t xch[4];      // the two warps of a lane quadrant
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int found[12];
    int base[kMaxE + 1];          // exclusive prefix of the experts' M-tiles
    uint32_t amax[2][2][BM];      // [unit parity][column half][row]
};
static_assert(sizeof(Misc) <= MISC, "barriers, tile prefix and maxima fit their place");

struct Unit {
    int e, n, rows;
    int64_t row0;
};

MOE_DEV Unit unit_of(int u, int nt, const Args& p, const int* base) {
    Unit U;
    const int g = u / nt;  // as if every M-tile had its n-tiles next to each other: the expert is the same
    int lo = 0, hi = p.E;  // base[lo] <= g < base[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= g) lo = mid;
        else hi = mid;
    }
    U.e = lo;
    const int mt = base[lo + 1] - base[lo], local = u - base[lo] * nt;
    U.n = local / mt;
    const int m = local - U.n * mt;
    const int64_t off = p.offsets ? __ldg(p.offsets + lo) : 0;
    const int64_t end = p.offsets ? __ldg(p.offsets + lo + 1) : p.rows;
    U.row0 = off + int64_t(m) * BM;
    U.rows = int(min(int64_t(BM), end - U.row0));
    return U;
}

// Every lane waits; warp-uniform result.
MOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, Misc* m, const Args& p) {
    const bool ok = mbar_wait_bounded(bar, parity, &m->abort, p.err, p.wait_ns);
    return __all_sync(0xFFFFFFFFu, ok);
}

template <bool GATED>
__global__ void __launch_bounds__(THREADS, 1)
    f8_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                   const __grid_constant__ CUtensorMap tmB1, const Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc* ms = reinterpret_cast<Misc*>(smem + OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(ms->full + s, 1);
            mbar_init(ms->empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(ms->tfull + a, 1);
            mbar_init(ms->tempty + a, EPI);
        }
        for (int q = 0; q < 4; ++q) mbar_init(ms->xch + q, 2);
        mbar_init(&ms->drain, 1);
        ms->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB0);
        if (GATED) tma_prefetch_desc(&tmB1);
    }
    if (warp == 1) {
        tmem_alloc(&ms->tmem, 512);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch();
    // the experts' M-tiles, one expert a thread
    {
        const int t = threadIdx.x;
        int cnt = 0;
        if (!p.offsets) {
            if (t == 0) cnt = int((p.rows + BM - 1) / BM);
        } else if (t < p.E) {
            const int off = __ldg(p.offsets + t), end = __ldg(p.offsets + t + 1);
            if (off < 0 || end < off || end > p.rows) set_error(p.err, MOE_DEVERR_BOUNDS);  // not followed
            else cnt = (end - off + BM - 1) / BM;
        }
        int s = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += v;
        }
        if (lane == 31) ms->found[warp] = s;
        __syncthreads();
        for (int w = 0; w < warp; ++w) s += ms->found[w];
        if (t < p.E) ms->base[t + 1] = s;
        if (t == 0) ms->base[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ms->tmem;
    const int cols = GATED ? 128 : BN;  // columns of the result a tile
    const int nt = (p.N + cols - 1) / cols;
    const int total = ms->base[p.E] * nt;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
            const Unit U = unit_of(u, nt, p, ms->base);
            for (int kb = 0; kb < p.KB; ++kb) {
                int okl = 1;
                if (lane == 0) okl = mbar_wait_bounded(ms->empty + stage, phase ^ 1u, &ms->abort, p.err, p.wait_ns);
                okl = __shfl_sync(0xFFFFFFFFu, okl, 0);
                if (!okl) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t* sa = smem + stage * STAGE;
                    mbar_arrive_expect_tx(ms->full + stage, STAGE);
                    tma_load_2d(sa, &tmA, ms->full + stage, kb * BK, int(U.row0));
                    if (GATED) {
                        tma_load_3d(sa + A_BYTES, &tmB0, ms->full + stage, kb * BK, U.n * 128, U.e);
                        tma_load_3d(sa + A_BYTES + B_BYTES / 2, &tmB1, ms->full + stage, kb * BK, U.n * 128, U.e);
                    } else {
                        tma_load_3d(sa + A_BYTES, &tmB0, ms->full + stage, kb * BK, U.n * BN, U.e);
                    }
                    issued |= 1u << stage;
                    issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // on abort, every copy already issued lands before the CTA can exit
        if (!ok && lane == 0) {
            for (int s = 0; s < STAGES; ++s)
                if (issued >> s & 1u) mbar_wait_bounded(ms->full + s, (issued_par >> s) & 1u, nullptr, p.err, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
            for (int kb = 0; kb < p.KB; ++kb) {
                int okl = 1;
                if (lane == 0) {
                    okl = mbar_wait_bounded(ms->tempty + acc, acc_phase ^ 1u, &ms->abort, p.err, p.wait_ns) &&
                          mbar_wait_bounded(ms->full + stage, phase, &ms->abort, p.err, p.wait_ns);
                    if (okl) {
                        tc_fence_after();
                        const uint32_t a0 = smem_u32(smem + stage * STAGE), b0 = a0 + A_BYTES;
#pragma unroll
                        for (int j = 0; j < BK / 32; ++j)  // 32 bytes of K inside the swizzled rows
                            umma_f8(tmem_base + uint32_t(acc * BN), sdesc_sw128(a0 + j * 32, 16, 1024),
                                    sdesc_sw128(b0 + j * 32, 16, 1024), j != 0);
                        umma_commit(ms->empty + stage);
                        umma_commit(ms->tfull + acc);
                    }
                }
                okl = __shfl_sync(0xFFFFFFFFu, okl, 0);
                if (!okl) {
                    ok = false;
                    break;
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
        // every MMA this thread issued has completed before TMEM is freed
        if (lane == 0) {
            umma_commit(&ms->drain);
            mbar_wait_bounded(&ms->drain, 0, nullptr, p.err, kDrainLimitNs);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ scaled sums and results
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = uint32_t(q * 32) << 16;
        // columns of the accumulator: matmul 128 in a row; gated 64 of gate, 64 of up
        const uint32_t c0 = GATED ? half * 64 : half * 128, c1 = GATED ? 128 + half * 64 : half * 128 + 64;
        uint8_t* turn = smem + OFF_TURN + (warp - 2) * PIECE;
        int acc = 0, par = 0;
        uint32_t acc_phase = 0, xph = 0;
        bool ok = true, range_bad = false;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
            const Unit U = unit_of(u, nt, p, ms->base);
            const int rt = q * 32 + lane;  // row of the tile
            const bool live = rt < U.rows;
            const int64_t row = U.row0 + rt;
            float2 s[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = make_float2(0.f, 0.f);
            const float* as = p.a_scale + (live ? row : U.row0);
            const int nb = GATED ? U.n : min(U.n * 2 + half, p.NB - 1);
            const float* b0 = p.b_scale[0] + (int64_t(U.e) * p.NB + nb) * p.KB;
            const float* b1 = GATED ? p.b_scale[1] + (int64_t(U.e) * p.NB + nb) * p.KB : b0;
            // the scales of a block are loaded a block ahead
            float sa = __ldg(as), sb0 = __ldg(b0), sb1 = __ldg(b1);
            for (int kb = 0; kb < p.KB; ++kb) {
                const float f0 = sa * sb0, f1 = sa * sb1;
                if (kb + 1 < p.KB) {
                    sa = __ldg(as + int64_t(kb + 1) * p.rows);
                    sb0 = __ldg(b0 + kb + 1);
                    if (GATED) sb1 = __ldg(b1 + kb + 1);
                    else sb1 = sb0;
                }
                if (!warp_wait(ms->tfull + acc, acc_phase, ms, p)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tb = tmem_base + lanes + uint32_t(acc * BN);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t t[32];
                    tmem_ld_32x32b_x32(tb + (c < 2 ? c0 + c * 32 : c1 + (c - 2) * 32), t);
                    tmem_ld_wait();
                    const float f = c < 2 ? f0 : f1;
                    const float2 ff = make_float2(f, f);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[c * 16 + i] = __ffma2_rn(make_float2(__uint_as_float(t[2 * i]), __uint_as_float(t[2 * i + 1])),
                                                   ff, s[c * 16 + i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ms->tempty + acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if (!ok) break;
            // ---- the row's values of this thread: n of them from column col0
            constexpr int NV = GATED ? 64 : 128;
            const int col0 = GATED ? U.n * 128 + half * 64 : U.n * BN + half * 128;
            float* v = reinterpret_cast<float*>(s);
            if (GATED) {
#pragma unroll
                for (int i = 0; i < 64; ++i) v[i] = gated(v[i], v[64 + i], p.limit);
            } else {
                const float w = live ? row_weight(p, row) : 0.f;
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] *= w;
            }
            const int es = p.out_dt == MOE_DT_F32 ? 4 : p.out_dt == MOE_DT_E4M3 ? 1 : 2;
            float sc = 1.f;
            if (GATED && p.out_dt == MOE_DT_E4M3) {
                uint32_t m = 0;  // columns past N are zeros of zero weights
#pragma unroll
                for (int i = 0; i < 64; ++i) m = max(m, abs_bits(v[i]));
                ms->amax[par][half][rt] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(ms->xch + q);
                if (!warp_wait(ms->xch + q, xph, ms, p)) {
                    ok = false;
                    break;
                }
                xph ^= 1u;
                m = max(m, ms->amax[par][half ^ 1][rt]);
                par ^= 1;
                sc = f8_scale(m);
                if (half == 0 && live) p.h_scale[int64_t(U.n) * p.rows + row] = sc;
            }
            // pieces of 32 rows x 64 bytes: 16-byte chunk c of row r at r*64 + ((c ^ (r/2)%4) * 16)
            char* obase = static_cast<char*>(p.out);
            auto put = [&](int ch, uint4 x) {
                *reinterpret_cast<uint4*>(turn + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) = x;
            };
            auto flush = [&](int piece) {
                __syncwarp();
                const int rr = lane >> 2, ch = lane & 3;
                const int col = col0 + (piece * 64 + ch * 16) / es;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + rr;
                    if (q * 32 + r < U.rows && col < p.N)  // rows of the result are multiples of 16 bytes
                        *reinterpret_cast<uint4*>(obase + ((U.row0 + q * 32 + r) * p.N + col) * es) =
                            *reinterpret_cast<const uint4*>(turn + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
                }
                __syncwarp();
            };
            if (es == 4) {
#pragma unroll
                for (int pc = 0; pc < NV / 16; ++pc) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        const float* x = v + pc * 16 + ch * 4;
                        put(ch, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                           __float_as_uint(x[3])));
                    }
                    flush(pc);
                }
            } else if (es == 2) {
                const bool bf = p.out_dt == MOE_DT_BF16;
                if (!bf && live) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) range_bad |= !f16_range_ok(v[i]) && col0 + i < p.N;
                }
#pragma unroll
                for (int pc = 0; pc < NV / 32; ++pc) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = v[pc * 32 + ch * 8 + i];
                        put(ch, pack8(x, bf));
                    }
                    flush(pc);
                }
            } else if (GATED) {
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float x[8], y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = v[ch * 16 + i];
                        y[i] = v[ch * 16 + 8 + i];
                    }
                    const uint2 lo = pack8_e4m3(x, sc), hi = pack8_e4m3(y, sc);
                    put(ch, make_uint4(lo.x, lo.y, hi.x, hi.y));
                }
                flush(0);
            }
        }
        if (range_bad) set_error(p.err, MOE_DEVERR_RANGE);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <bool GATED>
cudaError_t go(const CUtensorMap& A, const CUtensorMap& B0, const CUtensorMap& B1, const Args& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(f8_tile_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    const int64_t mt = p.offsets ? std::min<int64_t>(p.rows, p.E) + p.rows / BM : (p.rows + BM - 1) / BM;
    const int64_t units = mt * ((p.N + (GATED ? 127 : BN - 1)) / (GATED ? 128 : BN));
    ProfScope prof_(MOE_K_TC_F8, s);
    return launch_pdl(use_pdl(p.rows), f8_tile_kernel<GATED>, dim3(int(std::min<int64_t>(units, num_sms()))),
                      dim3(THREADS), SMEM, s, A, B0, B1, p);
}

// Bytes, innermost dimension K; box 128 (K) x `box_rows`, 128-byte swizzle.
bool map_bytes(CUtensorMap* m, const void* base, int K, int64_t rows, int n, int box_rows) {
    const uint64_t dims[3] = {uint64_t(K), uint64_t(rows), uint64_t(n)};
    const uint64_t str[2] = {uint64_t(K), uint64_t(K) * uint64_t(rows)};
    const uint32_t box[3] = {128, uint32_t(box_rows), 1};
    return tc::make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, n ? 3 : 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_tile(const Args& p, bool gated, cudaStream_t s) {
    CUtensorMap A, B0, B1;
    const int box = gated ? 128 : BN;
    if (!map_bytes(&A, p.a, p.K, p.rows, 0, BM) || !map_bytes(&B0, p.b[0], p.K, p.N, p.E, box) ||
        !map_bytes(&B1, p.b[1], p.K, p.N, p.E, box))
        return cudaErrorInvalidValue;
    return gated ? go<true>(A, B0, B1, p, s) : go<false>(A, B0, B1, p, s);
}

}  // namespace f8

}  // namespace moe

// f8_tile.cu — the 8-bit products on the tcgen05 tensor cores: 128 rows of an
// expert x 256 weight rows a tile (gated: 128 of gate and 128 of up), persistent,
// one CTA an SM.
//
//   c[r, n] = sum over blocks b of 128 along K of  sa[b, r] sb[n / 128, b] sum_{k in b} a[r, k] w[n, k]
//
//   warp 0      TMA producer: per block along K, the 128 x 128 bytes of the rows and
//               the 256 x 128 bytes of the weights (128-byte swizzle; past K and N
//               zeros come in), 4 stages of 48 KB.
//   warp 1      TMEM and the MMAs: tcgen05.mma kind::f8f6f4, M=128 N=256 K=32, four a
//               block. Every block of 128 is summed from zero into one of two
//               256-column accumulators, because its scales are its own.
//   warp 2      the blocks' scales, 8 blocks ahead, and what a tile's results need.
//   warps 4-11  the sums: a block's accumulator is read from TMEM as soon as it is
//               done, 64 columns a load, multiplied by its two scales and added in fp32
//               registers (128 columns of a row a thread), while the MMAs fill the other
//               one. After the last block: the gate weight or the clamped SwiGLU, the
//               rounding, and stores of 32 bytes a lane.
//
// What bounds it. Every block brings 48 KB into shared memory and the MMAs read as much: 768 cycles
// at 128 bytes a cycle, against 512 of the MMAs, so that the feed and the MMAs alone, no sums, take
// 56 us for 4096 x 4096 x 4096. The tiles' ends, where every CTA writes its 64 KB at once, add 12, the
// accumulators' loads 2 and the sums' FMAs 16, which the accumulators' way round (MMA, load, sum, hand
// back) does not hide: 85 us with bf16 results, 1.62 PFLOP/s. 32768 rows of 128 experts:
// 768 -> 2048 (fp16) 122 us; gate and up 2048 -> 2 x 768, e4m3 results 172 us (1.2 PFLOP/s).
// No faster when tried: three loads of 32 columns in turn with their sums. Slower: the next block's
// scales read behind a load (101), four accumulators of 128 columns (99: the rows' bytes are read
// twice), 16 warps of sums, pairs of SMs on 256-row tiles (89 for this product, the peer's hand-back
// without a release: half the traffic, but every block's accumulator waits for two SMs).
//
// Gated with e4m3 results: a row's 128 columns lie in two threads (two warps of a
// lane quadrant), which exchange their maxima over a barrier of those two warps.
// Units (expert, n-tile, M-tile; M fastest, so that neighbours share the weights in
// L2) are all alike in length and dealt out by index: no counter, no workspace.
#include <algorithm>
#include <atomic>

#include "f8.cuh"

namespace moe {

namespace f8 {

namespace {

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int EPI = 8, FIRST = 4, THREADS = 32 * (FIRST + EPI);
constexpr int PARTS = EPI / 4;      // column parts of a tile; the warps of a lane quadrant
constexpr int CW = BN / PARTS;      // columns of the accumulator a thread
constexpr int OFF_MISC = STAGES * STAGE;
constexpr int SLOTS = 8;         // blocks whose scales are on their way
constexpr int MISC = 11 * 1024;
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

// Registers of a warpgroup from here on. The launch gives 12 warps 168 each; the split's sum,
// 4 x 40 + 8 x 232 a lane, is the same.
template <int N>
MOE_DEV void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
MOE_DEV void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Waits for the loads from TMEM, tied to the registers that one of them fills: no use of them moves
// before the wait.
MOE_DEV void tmem_ld_wait_for(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

struct Misc {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t tfull[2], tempty[2];
    uint64_t sfull[SLOTS], sempty[SLOTS];
    uint64_t ufull[2], uempty[2];
    uint64_t xch[4];      // the two warps of a lane quadrant
    uint64_t drain;
    uint32_t tmem;
    int abort;
    Chunks tiles;                 // the experts' M-tiles
    float sa[SLOTS][BM];          // the rows' scales of a block
    float sb[SLOTS][2];           // the weights': of the tile's two 128-column halves, or gate and up
    int64_t urow0[2];             // by unit parity: what the tile's results need
    int urows[2], un[2];
    float uw[2][BM];              // the rows' gate weights
    uint32_t amax[2][PARTS][BM];  // [unit parity][column part][row]
};
static_assert(sizeof(Misc) <= MISC, "barriers, tile prefix and maxima fit their place");

struct Unit {
    int e, n, rows;
    int64_t row0;
};

MOE_DEV Unit unit_of(int u, int nt, const Args& p, const Misc* ms) {
    Unit U;
    const int* base = ms->tiles.base;
    const int lo = expert_of(ms->tiles, u / nt, p.E);  // as if every M-tile had its n-tiles next to each other
    U.e = lo;
    const int mt = base[lo + 1] - base[lo], local = u - base[lo] * nt;
    U.n = local / mt;
    const int m = local - U.n * mt;
    U.row0 = ms->tiles.off[lo] + int64_t(m) * BM;
    U.rows = int(min(int64_t(BM), ms->tiles.off[lo + 1] - U.row0));
    return U;
}

MOE_DEV void st_global_32(void* p, const uint4& lo, const uint4& hi) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
                 "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
}
// Eight values to 16 bits; sixteen in units of a scale to e4m3.
MOE_DEV uint4 pack8_at(const float* x, bool bf16) {
    return bf16 ? make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7]))
                : make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]), pack_f16x2(x[6], x[7]));
}
MOE_DEV uint4 pack16_e4m3(const float* x, const F8Div& div) {
    uint32_t w[4];
    if (div.fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_e4m3x2(div(x[4 * i]), div(x[4 * i + 1])) | pack_e4m3x2(div(x[4 * i + 2]), div(x[4 * i + 3])) << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_e4m3x2(__fdiv_rn(x[4 * i], div.s), __fdiv_rn(x[4 * i + 1], div.s)) |
                   pack_e4m3x2(__fdiv_rn(x[4 * i + 2], div.s), __fdiv_rn(x[4 * i + 3], div.s)) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 4 bytes global -> shared, asynchronous; the thread's arrival on bar once its copies have landed.
MOE_DEV void cp_async_4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
MOE_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Every lane waits; warp-uniform result.
MOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, Misc* m, const Args& p) {
    const bool ok = mbar_wait_bounded(bar, parity, &m->abort, p.err, p.wait_ns);
    return __all_sync(0xFFFFFFFFu, ok);
}

template <bool GATED, int OUT>
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
        for (int q = 0; q < 4; ++q) mbar_init(ms->xch + q, PARTS);
        for (int a = 0; a < 2; ++a) {
            mbar_init(ms->ufull + a, 32);
            mbar_init(ms->uempty + a, EPI);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(ms->sfull + i, 32);
            mbar_init(ms->sempty + i, EPI);
        }
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
    count_chunks(p, BM, ms->tiles);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ms->tmem;
    const int cols = GATED ? 128 : BN;  // columns of the result a tile
    const int nt = (p.N + cols - 1) / cols;
    const int total = ms->tiles.base[p.E] * nt;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_bounded(bar, parity, &ms->abort, p.err, p.wait_ns);
    };

    if (warp < FIRST) {
        reg_dec<40>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (one thread)
            if (lane == 0) {
                int stage = 0, left = p.copies;
                uint32_t phase = 0, issued = 0, issued_par = 0;
                bool ok = true;
                for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
                    const Unit U = unit_of(u, nt, p, ms);
                    for (int kb = 0; kb < p.KB; ++kb) {
                        if (left-- == 0 || !wait(ms->empty + stage, phase ^ 1u)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = smem + stage * STAGE;
                        mbar_arrive_expect_tx(ms->full + stage, STAGE);
                        tma_load_3d(sa, &tmA, ms->full + stage, kb * BK, int(U.row0), 0);
                        if (GATED) {
                            tma_load_3d(sa + A_BYTES, &tmB0, ms->full + stage, kb * BK, U.n * 128, U.e);
                            tma_load_3d(sa + A_BYTES + B_BYTES / 2, &tmB1, ms->full + stage, kb * BK, U.n * 128, U.e);
                        } else {
                            tma_load_3d(sa + A_BYTES, &tmB0, ms->full + stage, kb * BK, U.n * BN, U.e);
                        }
                        issued |= 1u << stage;
                        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                // on abort, every copy already issued lands before the CTA can exit
                if (!ok)
                    for (int s = 0; s < STAGES; ++s)
                        if (issued >> s & 1u)
                            mbar_wait_bounded(ms->full + s, (issued_par >> s) & 1u, nullptr, p.err, kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer (one thread)
            if (lane == 0) {
                const uint64_t da = sdesc_sw128(smem_u32(smem), 16, 1024), db = sdesc_sw128(smem_u32(smem) + A_BYTES, 16, 1024);
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true;
                for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
                    for (int kb = 0; kb < p.KB; ++kb) {
                        if (!wait(ms->full + stage, phase) || !wait(ms->tempty + acc, acc_phase ^ 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        // addresses in the descriptors are in units of 16 bytes, below 2^14
                        const uint64_t so = uint64_t(stage * (STAGE / 16));
#pragma unroll
                        for (int j = 0; j < BK / 32; ++j)  // 32 bytes of K inside the swizzled rows
                            umma_f8(tmem_base + uint32_t(acc * BN), da + so + j * 2, db + so + j * 2, j != 0);
                        umma_commit(ms->tfull + acc);
                        umma_commit(ms->empty + stage);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        acc ^= 1;
                        if (acc == 0) acc_phase ^= 1u;
                    }
                }
                // every MMA this thread issued has completed before TMEM is freed
                umma_commit(&ms->drain);
                mbar_wait_bounded(&ms->drain, 0, nullptr, p.err, kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------ scales
            // A block's 128 row scales and 2 weight scales: loaded by the warps that use them, a block
            // ahead, their latency under load was longer than a block.
            int slot = 0, par = 0;
            uint32_t phase = 0, uphase = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
                const Unit U = unit_of(u, nt, p, ms);
                const float* as[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) as[i] = p.a_scale + U.row0 + min(i * 32 + lane, U.rows - 1);
                if (!warp_wait(ms->uempty + par, uphase ^ 1u, ms, p)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    ms->urow0[par] = U.row0;
                    ms->urows[par] = U.rows;
                    ms->un[par] = U.n;
                }
                if (p.sorted_pair) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ms->uw[par][i * 32 + lane] = row_weight(p, U.row0 + min(i * 32 + lane, U.rows - 1));
                }
                mbar_arrive(ms->ufull + par);
                par ^= 1;
                if (par == 0) uphase ^= 1u;
                const int nb = GATED ? U.n : min(U.n * 2 + (lane & 1), p.NB - 1);
                const float* bs = p.b_scale[GATED ? lane & 1 : 0] + (int64_t(U.e) * p.NB + nb) * p.KB;
                for (int kb = 0; kb < p.KB; ++kb) {
                    if (!warp_wait(ms->sempty + slot, phase ^ 1u, ms, p)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        cp_async_4(smem_u32(&ms->sa[slot][i * 32 + lane]), as[i] + int64_t(kb) * p.rows);
                    if (lane < 2) cp_async_4(smem_u32(&ms->sb[slot][lane]), bs + kb);
                    cp_async_arrive(ms->sfull + slot);
                    if (++slot == SLOTS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait_all();
            __syncwarp();
        }
    } else {
        reg_inc<232>();
        // ------------------------------------------------ scaled sums and results
        const int q = warp & 3, part = (warp - FIRST) >> 2;
        const uint32_t lanes = uint32_t(q * 32) << 16;
        // columns of the accumulator: matmul CW in a row; gated CW/2 of gate, CW/2 of up
        const uint32_t c0 = GATED ? part * (CW / 2) : part * CW, c1 = GATED ? 128 + c0 : c0 + CW / 2;
        int acc = 0, par = 0, slot = 0;
        uint32_t acc_phase = 0, xph = 0, sph = 0, uphase = 0;
        bool ok = true, range_bad = false;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
            float2 s[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) s[i] = make_float2(0.f, 0.f);
            for (int kb = 0; kb < p.KB; ++kb) {
                if (!warp_wait(ms->sfull + slot, sph, ms, p)) {
                    ok = false;
                    break;
                }
                const float sa = ms->sa[slot][q * 32 + lane];
                const float f0 = sa * ms->sb[slot][GATED ? 0 : part * CW / 128], f1 = GATED ? sa * ms->sb[slot][1] : f0;
                __syncwarp();
                if (lane == 0) mbar_arrive(ms->sempty + slot);
                if (++slot == SLOTS) {
                    slot = 0;
                    sph ^= 1u;
                }
                if (!warp_wait(ms->tfull + acc, acc_phase, ms, p)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tb = tmem_base + lanes + uint32_t(acc * BN);
                // 64 columns at a time: one latency for four loads; the accumulator is handed back
                // as soon as the last have come
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t t[2][32];
                    const uint32_t ch = tb + (h ? c1 : c0);
                    tmem_ld_32x32b_x32(ch, t[0]);
                    tmem_ld_32x32b_x32(ch + 32, t[1]);
                    tmem_ld_wait_for(t[0]);
                    tmem_ld_wait_for(t[1]);
                    if (h == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ms->tempty + acc);
                    }
                    const float f = h ? f1 : f0;
                    const float2 ff = make_float2(f, f);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        s[h * 32 + i] = __ffma2_rn(make_float2(__uint_as_float(t[i >> 4][2 * (i & 15)]),
                                                               __uint_as_float(t[i >> 4][2 * (i & 15) + 1])),
                                                   ff, s[h * 32 + i]);
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if (!ok) break;
            // ---- the row's values of this thread: NV columns from col0 on
            if (!warp_wait(ms->ufull + par, uphase, ms, p)) {
                ok = false;
                break;
            }
            const int rt = q * 32 + lane;  // row of the tile
            const bool live = rt < ms->urows[par];
            const int64_t row = ms->urow0[par] + rt;
            const int un = ms->un[par];
            const float w = !GATED && p.sorted_pair ? ms->uw[par][rt] : 1.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(ms->uempty + par);
            constexpr int NV = GATED ? CW / 2 : CW;
            const int col0 = GATED ? un * 128 + part * (CW / 2) : un * BN + part * CW;
            float* v = reinterpret_cast<float*>(s);
            if constexpr (GATED) {
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] = gated(v[i], v[NV + i], p.limit);
            } else if (p.sorted_pair) {
#pragma unroll
                for (int i = 0; i < NV; ++i) v[i] *= w;
            }
            constexpr int es = OUT == MOE_DT_F32 ? 4 : OUT == MOE_DT_E4M3 ? 1 : 2;
            float divisor = 1.f;
            if constexpr (OUT == MOE_DT_E4M3) {
                uint32_t m = 0;  // columns past N are zeros of zero weights
#pragma unroll
                for (int i = 0; i < NV; ++i) m = max(m, abs_bits(v[i]));
                ms->amax[par][part][rt] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(ms->xch + q);
                if (!warp_wait(ms->xch + q, xph, ms, p)) {
                    ok = false;
                    break;
                }
                xph ^= 1u;
#pragma unroll
                for (int i = 0; i < PARTS; ++i) m = max(m, ms->amax[par][i][rt]);
                const float sc = f8_scale(m);
                if (part == 0 && live) p.h_scale[int64_t(un) * p.rows + row] = sc;
                if (live) divisor = f8_divisor(m, sc);  // rows past the expert's may hold anything
            }
            const F8Div div(divisor);
            if constexpr (OUT == MOE_DT_F16) {
                if (live) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) range_bad |= !f16_range_ok(v[i]) && col0 + i < p.N;
                }
            }
            // 32 bytes a store: a whole sector of the row, and nothing to wait for (turning the
            // rows through shared memory for longer pieces kept the warps from the next tile)
            char* orow = static_cast<char*>(p.out) + (row * p.N + col0) * es;
            constexpr int per = 32 / es;  // columns of 32 bytes
            const bool wide = (int64_t(p.N) * es) % 32 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll
            for (int c = 0; c < NV / per; ++c) {
                const float* x = v + c * per;
                uint4 lo, hi;
                if constexpr (es == 4) {
                    lo = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                    hi = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
                } else if constexpr (es == 2) {
                    lo = pack8_at(x, OUT == MOE_DT_BF16);
                    hi = pack8_at(x + 8, OUT == MOE_DT_BF16);
                } else {
                    lo = pack16_e4m3(x, div);
                    hi = pack16_e4m3(x + 16, div);
                }
                const int col = col0 + c * per;
                if (!live || col >= p.N) continue;
                if (wide) {
                    st_global_32(orow + c * 32, lo, hi);
                } else {  // rows of the result are multiples of 16 bytes
                    *reinterpret_cast<uint4*>(orow + c * 32) = lo;
                    if (col + per / 2 < p.N) *reinterpret_cast<uint4*>(orow + c * 32 + 16) = hi;
                }
            }
            par ^= 1;
            if (par == 0) uphase ^= 1u;
        }
        if (range_bad) set_error(p.err, MOE_DEVERR_RANGE);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <bool GATED, int OUT>
cudaError_t go(const CUtensorMap& A, const CUtensorMap& B0, const CUtensorMap& B1, const Args& p, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};  // one bit a device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev >= 64 || !(configured.load() & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(f8_tile_kernel<GATED, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    const int64_t mt = p.offsets ? std::min<int64_t>(p.rows, p.E) + p.rows / BM : (p.rows + BM - 1) / BM;
    const int64_t units = mt * ((p.N + (GATED ? 127 : BN - 1)) / (GATED ? 128 : BN));
    ProfScope prof_(MOE_K_TC_F8, s);
    return launch_pdl(use_pdl(p.rows), f8_tile_kernel<GATED, OUT>, dim3(int(std::min<int64_t>(units, num_sms()))),
                      dim3(THREADS), SMEM, s, A, B0, B1, p);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    return fn;
}

// Bytes [n, rows, K]; box 128 (K) x `box_rows` x 1, 128-byte swizzle.
bool map_bytes(CUtensorMap* m, const void* base, int K, int64_t rows, int n, int box_rows) {
    const EncodeTiledFn enc = encode_fn();
    const cuuint64_t dims[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(n)};
    const cuuint64_t str[2] = {cuuint64_t(K), cuuint64_t(K) * cuuint64_t(rows)};
    const cuuint32_t box[3] = {BK, cuuint32_t(box_rows), 1}, step[3] = {1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, str, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_tile(const Args& p, bool gated, cudaStream_t s) {
    CUtensorMap A, B0, B1;
    const int box = gated ? 128 : BN;
    if (!map_bytes(&A, p.a, p.K, p.rows, 1, BM) || !map_bytes(&B0, p.b[0], p.K, p.N, p.E, box) ||
        !map_bytes(&B1, p.b[1], p.K, p.N, p.E, box))
        return cudaErrorInvalidValue;
    switch (p.out_dt) {
        case MOE_DT_F32: return gated ? go<true, MOE_DT_F32>(A, B0, B1, p, s) : go<false, MOE_DT_F32>(A, B0, B1, p, s);
        case MOE_DT_BF16: return gated ? go<true, MOE_DT_BF16>(A, B0, B1, p, s) : go<false, MOE_DT_BF16>(A, B0, B1, p, s);
        case MOE_DT_F16: return gated ? go<true, MOE_DT_F16>(A, B0, B1, p, s) : go<false, MOE_DT_F16>(A, B0, B1, p, s);
        default: return gated ? go<true, MOE_DT_E4M3>(A, B0, B1, p, s) : cudaErrorInvalidValue;
    }
}

}  // namespace f8

}  // namespace moe

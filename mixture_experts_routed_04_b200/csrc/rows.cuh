// rows.cuh — rows of fp32, bf16 or fp16 in registers, and their rounding to e4m3
// with one scale for each 128 columns: shared by the norms (norm.cu) and the
// 8-bit kernels (quantize_f8.cu, gated products).
#pragma once

#include <type_traits>

#include "internal.h"

namespace moe {

MOE_DEV float f16_bits_to_f32(uint16_t v) { return f16_lo(uint32_t(v)); }

// Two values to bf16, nearest even, in one instruction (NaN becomes the canonical NaN).
MOE_DEV uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One element of a row of dtype dt (MOE_DT_F32 / BF16 / F16).
MOE_DEV float load_elem(const void* p, int64_t i, int dt) {
    if (dt == MOE_DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return dt == MOE_DT_BF16 ? bf16_to_f32(v) : f16_bits_to_f32(v);
}
MOE_DEV void store_elem(void* p, int64_t i, float v, int dt) {
    if (dt == MOE_DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = uint16_t((dt == MOE_DT_BF16 ? cvt_bf16x2(v, 0.f) : pack_f16x2(v, 0.f)) & 0xFFFFu);
}
// v as the dtype holds it.
MOE_DEV float round_to(float v, int dt) {
    if (dt == MOE_DT_F32) return v;
    return dt == MOE_DT_BF16 ? bf16_lo(cvt_bf16x2(v, 0.f)) : f16_lo(pack_f16x2(v, 0.f));
}

MOE_DEV void unpack8(const uint4& r, bool bf16, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16 ? bf16_lo(w[i]) : f16_lo(w[i]);
        v[2 * i + 1] = bf16 ? bf16_hi(w[i]) : f16_hi(w[i]);
    }
}
MOE_DEV void unpack4(const uint2& r, bool bf16, float* v) {
    v[0] = bf16 ? bf16_lo(r.x) : f16_lo(r.x);
    v[1] = bf16 ? bf16_hi(r.x) : f16_hi(r.x);
    v[2] = bf16 ? bf16_lo(r.y) : f16_lo(r.y);
    v[3] = bf16 ? bf16_hi(r.y) : f16_hi(r.y);
}
MOE_DEV uint2 pack4(const float* v, bool bf16) {
    return bf16 ? make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]))
                : make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
}

// A row spread over `th` threads, NV groups of 8 elements each: two quads of 4.
//   kScalarRow: element j of group v sits at (v*8 + j)*th + t, so that any length, stride and
//        alignment is read with neighbouring threads on neighbouring elements.
//   kVecRow: quad q = 2v, 2v + 1 of thread t holds the 4 consecutive elements at (q*th + t)*4, so
//        that a warp's access is 128 elements in a row whatever the dtype: 16 bytes a lane of fp32, 8
//        of 16 bits (with 8 elements a lane, fp32 rows and weights took two accesses of every
//        other 16 bytes each: half sectors). The row's length is a multiple of 4 and every row
//        starts on 4 elements.
//   kFullRow: the same for a row of exactly NV*th*8 elements: no quad needs its place checked.
// Elements past the row's end are zero and are not stored. The dtype is looked at once a row, not
// in the loops: with a branch a group these took more instructions than the arithmetic.
enum RowLayout { kScalarRow = 0, kVecRow = 1, kFullRow = 2 };

// The first column of quad h of group i, and whether it is inside the row.
MOE_DEV int quad_at(int i, int h, int th, int t) { return ((2 * i + h) * th + t) * 4; }
template <int L>
MOE_DEV bool quad_in(int c, int d) {
    return L == kFullRow || c < d;
}
template <int L, bool F32>
MOE_DEV void load_group_as(float (&v)[8], const void* row, int i, int d, bool bf16, int th, int t) {
    if (L != kScalarRow) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = quad_at(i, h, th, t);
            const bool in = quad_in<L>(c, d);
            if (F32) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in) a = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
                v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
            } else {
                uint2 a = make_uint2(0, 0);
                if (in) a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + c);
                unpack4(a, bf16, v + 4 * h);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (i * 8 + j) * th + t;
            if (F32) {
                v[j] = c < d ? static_cast<const float*>(row)[c] : 0.f;
            } else {
                const uint16_t u = c < d ? static_cast<const uint16_t*>(row)[c] : uint16_t(0);
                v[j] = bf16 ? bf16_to_f32(u) : f16_bits_to_f32(u);
            }
        }
    }
}

template <int NV, int L>
MOE_DEV void load_row(float (&v)[NV][8], const void* row, int d, int dt, int th, int t) {
    if (dt == MOE_DT_F32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_group_as<L, true>(v[i], row, i, d, false, th, t);
    } else if (dt == MOE_DT_BF16) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_group_as<L, false>(v[i], row, i, d, true, th, t);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_group_as<L, false>(v[i], row, i, d, false, th, t);
    }
}

template <int NV, int L, bool F32>
MOE_DEV void store_row_as(const float (&v)[NV][8], void* row, int d, bool bf16, int th, int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (L != kScalarRow) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = quad_at(i, h, th, t);
                if (!quad_in<L>(c, d)) continue;
                if (F32)
                    *reinterpret_cast<float4*>(static_cast<float*>(row) + c) =
                        make_float4(v[i][4 * h], v[i][4 * h + 1], v[i][4 * h + 2], v[i][4 * h + 3]);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + c) = pack4(v[i] + 4 * h, bf16);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (i * 8 + j) * th + t;
                if (c < d) {
                    if (F32) static_cast<float*>(row)[c] = v[i][j];
                    else store_elem(row, c, v[i][j], bf16 ? MOE_DT_BF16 : MOE_DT_F16);
                }
            }
        }
    }
}
template <int NV, int L>
MOE_DEV void store_row(const float (&v)[NV][8], void* row, int d, int dt, int th, int t) {
    if (dt == MOE_DT_F32) store_row_as<NV, L, true>(v, row, d, false, th, t);
    else if (dt == MOE_DT_BF16) store_row_as<NV, L, false>(v, row, d, true, th, t);
    else store_row_as<NV, L, false>(v, row, d, false, th, t);
}

// f with the dtype as a compile-time constant (0 fp32, 1 bf16, 2 fp16): one branch around a loop.
template <typename F>
MOE_DEV void by_dtype(int dt, F f) {
    if (dt == MOE_DT_F32) f(std::integral_constant<int, 0>{});
    else if (dt == MOE_DT_BF16) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 2>{});
}
template <int L, int DT>
MOE_DEV void load_group(float (&v)[8], const void* row, int i, int d, int th, int t) {
    load_group_as<L, DT == MOE_DT_F32>(v, row, i, d, DT == MOE_DT_BF16, th, t);
}

// Whether element (group i, place j) of thread t lies inside a row of d elements.
template <int L>
MOE_DEV bool in_row(int i, int j, int d, int th, int t) {
    if (L == kScalarRow) return (i * 8 + j) * th + t < d;
    return quad_in<L>(quad_at(i, j >> 2, th, t), d);
}

// ---- rows on their way through shared memory (vector layouts, every row on 16 bytes). Quad q of
// the block's thread t sits at q * threads + t. A warp copies its own quads in 16-byte pieces: of
// fp32 a quad a lane, of 16 bits two quads of neighbouring lanes (8-byte copies of the lane's own
// took a third longer). So a warp's copies are its own affair: each lane waits for its pieces, the
// warp meets, and meets again before the place is copied to anew. Room for a row of a tensor:
// stage_pieces() * 16 bytes a thread.
__host__ __device__ inline int stage_pieces(int nv, int dt) { return nv * (dt == MOE_DT_F32 ? 2 : 1); }

// base: the tensor's place in the stage (thread 0's).
template <int NV, int L, int THREADS>
MOE_DEV void copy_row(uint32_t base, const char* row, int d, int dt, int th, int t) {
    if (dt == MOE_DT_F32) {
#pragma unroll
        for (int q = 0; q < 2 * NV; ++q) {
            const int c = (q * th + t) * 4;
            if (quad_in<L>(c, d)) cp_async_16(base + (q * THREADS + threadIdx.x) * 16, row + c * 4, 16);
        }
    } else {
        const int lane = t & 31;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int q = 2 * i + (lane >> 4);  // half a warp a quad row: 16 pieces of 8 elements
            const int c = (q * th + (t & ~31)) * 4 + (lane & 15) * 8;
            if (quad_in<L>(c, d))
                cp_async_16(base + (q * THREADS + (threadIdx.x & ~31)) * 8 + (lane & 15) * 16, row + c * 2,
                            L == kFullRow || c + 8 <= d ? 16 : 8);  // d may end after half a piece
        }
    }
}
template <int NV, int L, int THREADS>
MOE_DEV void read_row(float (&v)[NV][8], const uint4* base, int d, int dt, int th, int t) {
    by_dtype(dt, [&](auto DT) {
#pragma unroll
        for (int q = 0; q < 2 * NV; ++q) {
            const bool in = quad_in<L>((q * th + t) * 4, d);
            float* w = v[q >> 1] + 4 * (q & 1);
            if (decltype(DT)::value == MOE_DT_F32) {
                uint4 a = make_uint4(0, 0, 0, 0);
                if (in) a = base[q * THREADS + threadIdx.x];
                w[0] = __uint_as_float(a.x); w[1] = __uint_as_float(a.y);
                w[2] = __uint_as_float(a.z); w[3] = __uint_as_float(a.w);
            } else {
                uint2 a = make_uint2(0, 0);
                if (in) a = reinterpret_cast<const uint2*>(base)[q * THREADS + threadIdx.x];
                unpack4(a, decltype(DT)::value == MOE_DT_BF16, w);
            }
        }
    });
}
// At most n of this thread's committed groups of copies still on their way (n < 4).
MOE_DEV void cp_async_wait_most(int n) {
    switch (n) {
        case 0: cp_async_wait<0>(); break;
        case 1: cp_async_wait<1>(); break;
        case 2: cp_async_wait<2>(); break;
        default: cp_async_wait<3>(); break;
    }
}

// ------------------------------------------------------------------ e4m3 with a scale
// A group of 128 values x is held as q = e4m3(x / s) (round to nearest even) and
// s = max(amax / 448, 2^-126), both divisions in fp32: 448 is e4m3's largest value,
// and the floor keeps x / s finite for a group of zeros or denormals. The largest
// magnitude is found on the absolute values' bit patterns, where NaN sorts above
// infinity: a NaN or an infinity anywhere makes the scale NaN or infinite, so the
// whole group reads back as NaN and never as plausible numbers.
MOE_DEV uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// The larger of two magnitudes; a NaN wins.
MOE_DEV float amax2(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
    return m;
}
MOE_DEV uint32_t amax4_bits(const float* v) { return abs_bits(amax2(amax2(v[0], v[1]), amax2(v[2], v[3]))); }
MOE_DEV float f8_scale(uint32_t amax_bits) {
    const float s = __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // a NaN passes
}
// Two values in units of the scale -> two e4m3 bytes (lo in the low byte); beyond
// +-448 they saturate (x / s may round up to just above it), NaN stays NaN.
MOE_DEV uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// x / s rounded once, for a group's scale s and rs = 1/s rounded once. With a
// correctly rounded reciprocal, one Newton step on the quotient (its remainder is
// exact in an fma) gives the correctly rounded quotient (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): three
// instructions a value instead of a whole division, which bounds the rounding of
// rows that sit in L2. The remainder must not underflow: quotients that do not
// round to zero have x >= 2^-10 s, so from s >= 2^-90 on it does not.
struct F8Div {
    float s, rs;
    bool fast;
    F8Div() = default;
    MOE_DEV explicit F8Div(float scale) {
        s = scale;
        rs = __fdiv_rn(1.0f, scale);
        fast = scale >= 0x1p-90f && scale <= 3.4e38f;
    }
    MOE_DEV float operator()(float x) const {
        const float q = x * rs;
        return fmaf(-fmaf(q, s, -x), rs, q);  // the remainder with this sign keeps -0
    }
};
// Four values of a group whose scale is s, nrs = -1/s; two quotients an instruction. The quotient comes
// out negative, which takes a sign off no operand of the packed fmas (they have no negation), and the
// four signs are turned at once at the end; a zero keeps its sign.
MOE_DEV uint32_t pack4_e4m3_fast(const float* v, float s, float nrs) {
    const float2 s2 = make_float2(s, s), n2 = make_float2(nrs, nrs);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
        const float2 q = __fmul2_rn(x, n2);                       // -x / s
        const float2 y = __ffma2_rn(__ffma2_rn(q, s2, x), n2, q);  // less its remainder's quotient
        w[i] = pack_e4m3x2(y.x, y.y);
    }
    return (w[0] | w[1] << 16) ^ 0x80808080u;
}
MOE_DEV uint32_t pack4_e4m3(const float* v, const F8Div& div) {
    return div.fast ? pack4_e4m3_fast(v, div.s, -div.rs)
                    : pack_e4m3x2(__fdiv_rn(v[0], div.s), __fdiv_rn(v[1], div.s)) |
                          pack_e4m3x2(__fdiv_rn(v[2], div.s), __fdiv_rn(v[3], div.s)) << 16;
}

// What a group whose largest magnitude is m divides by: its scale, or 1 for a group of zeros, whose
// scale of 2^-126 would take the long way to the same zeros.
MOE_DEV float f8_divisor(uint32_t m, float scale) { return m ? scale : 1.0f; }

// The scales of a warp's N <= 32 groups of 128 columns from their largest magnitudes m[k], which the
// warp agrees on: lane k divides for group k, so that the two divisions are done once a warp and not
// once a lane and group. Warp-uniform result: whether every group's quotients may take the short way.
template <int N>
MOE_DEV bool warp_scales(const uint32_t (&m)[N], float& scale, float& divisor, float& recip) {
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((threadIdx.x & 31) == k) mine = m[k];
    scale = f8_scale(mine);
    const F8Div div(f8_divisor(mine, scale));
    divisor = div.s;
    recip = div.rs;
    return __all_sync(0xFFFFFFFFu, div.fast);
}

// A row in a vector layout to e4m3: a warp's quads are a group of 128 columns. q: the row's bytes;
// s: scale of column group 0, the next ones `lds` on. Every thread of the warp takes part; a warp whose
// row is not to be written does not call it (kFullRow stores all of the row, whatever d says).
template <int NV, int L>
MOE_DEV void store_row_e4m3(const float (&v)[NV][8], uint8_t* q, float* s, int64_t lds, int d, int th, int t) {
    uint32_t m[2 * NV];
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
        const float* x = v[k >> 1] + 4 * (k & 1);
        m[k] = __reduce_max_sync(0xFFFFFFFFu, amax4_bits(x));
    }
    float scale, divisor, recip;
    const bool fast = warp_scales(m, scale, divisor, recip);
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
        F8Div div;
        div.s = __shfl_sync(0xFFFFFFFFu, divisor, k);
        div.rs = __shfl_sync(0xFFFFFFFFu, recip, k);
        div.fast = fast;
        const int c = (k * th + t) * 4;
        if (quad_in<L>(c, d)) *reinterpret_cast<uint32_t*>(q + c) = pack4_e4m3(v[k >> 1] + 4 * (k & 1), div);
    }
    const int lane = t & 31, c = (lane * th + (t & ~31)) * 4;  // lane k: the first column of the warp's k-th quad row
    if (lane < 2 * NV && quad_in<L>(c, d)) s[int64_t(c >> 7) * lds] = scale;
}

}  // namespace moe

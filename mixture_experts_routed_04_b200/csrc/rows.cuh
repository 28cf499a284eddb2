// rows.cuh — rows of fp32, bf16 or fp16 in registers, and their rounding to e4m3
// with one scale for each 128 columns: shared by the norms (norm.cu) and the
// 8-bit kernels (quantize_f8.cu, gated products).
#pragma once

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
MOE_DEV uint4 pack8(const float (&v)[8], bool bf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = bf16 ? cvt_bf16x2(v[2 * i], v[2 * i + 1]) : pack_f16x2(v[2 * i], v[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row spread over `th` threads, NV groups of 8 elements each.
//   VEC: group v of thread t holds the 8 consecutive elements at (v*th + t)*8
//        (16-byte loads; the row's length is a multiple of 8 and every row
//        starts on 16 bytes).
//   else element j of group v sits at (v*8 + j)*th + t, so that any length,
//        stride and alignment is read with neighbouring threads on
//        neighbouring elements.
// Elements past the row's end are zero and are not stored.
template <int NV, bool VEC>
MOE_DEV void load_row(float (&v)[NV][8], const void* row, int d, int dt, int th, int t) {
    if (VEC) {
        if (dt == MOE_DT_F32) {
            float4 a[NV], b[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * th + t) * 8;
                a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < d) {
                    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
                    a[i] = p[0];
                    b[i] = p[1];
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i][0] = a[i].x; v[i][1] = a[i].y; v[i][2] = a[i].z; v[i][3] = a[i].w;
                v[i][4] = b[i].x; v[i][5] = b[i].y; v[i][6] = b[i].z; v[i][7] = b[i].w;
            }
        } else {
            uint4 r[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * th + t) * 8;
                r[i] = make_uint4(0, 0, 0, 0);
                if (c < d) r[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c);
            }
            if (dt == MOE_DT_BF16) {
#pragma unroll
                for (int i = 0; i < NV; ++i) unpack8(r[i], true, v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) unpack8(r[i], false, v[i]);
            }
        }
    } else if (dt == MOE_DT_F32) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (i * 8 + j) * th + t;
                v[i][j] = c < d ? static_cast<const float*>(row)[c] : 0.f;
            }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (i * 8 + j) * th + t;
                const uint16_t u = c < d ? static_cast<const uint16_t*>(row)[c] : uint16_t(0);
                v[i][j] = dt == MOE_DT_BF16 ? bf16_to_f32(u) : f16_bits_to_f32(u);
            }
    }
}

template <int NV, bool VEC>
MOE_DEV void store_row(const float (&v)[NV][8], void* row, int d, int dt, int th, int t) {
    if (VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * th + t) * 8;
            if (c >= d) continue;
            if (dt == MOE_DT_F32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + c);
                p[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                p[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + c) = pack8(v[i], dt == MOE_DT_BF16);
            }
        }
    } else if (dt == MOE_DT_F32) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (i * 8 + j) * th + t;
                if (c < d) static_cast<float*>(row)[c] = v[i][j];
            }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (i * 8 + j) * th + t;
                if (c < d) store_elem(row, c, v[i][j], dt);
            }
    }
}

// Whether element (group i, place j) of thread t lies inside a row of d elements.
template <bool VEC>
MOE_DEV bool in_row(int i, int j, int d, int th, int t) {
    return (VEC ? (i * th + t) * 8 + j : (i * 8 + j) * th + t) < d;
}

// ------------------------------------------------------------------ e4m3 with a scale
// A group of 128 values x is held as q = e4m3(x / s) (round to nearest even) and
// s = max(amax / 448, 2^-126), both divisions in fp32: 448 is e4m3's largest value,
// and the floor keeps x / s finite for a group of zeros or denormals. The largest
// magnitude is found on the absolute values' bit patterns, where NaN sorts above
// infinity: a NaN or an infinity anywhere makes the scale NaN or infinite, so the
// whole group reads back as NaN and never as plausible numbers.
MOE_DEV uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
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
// Eight values of a group whose scale is s.
MOE_DEV uint2 pack8_e4m3(const float (&v)[8], float s) {
    const F8Div div(s);
    uint32_t h[4];
    if (div.fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = pack_e4m3x2(div(v[2 * i]), div(v[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = pack_e4m3x2(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// A row in the VEC layout to e4m3: 16 neighbouring threads hold a group of 128
// columns. q: the row's bytes; s: scale of column group 0, the next ones `lds` on.
// Every thread of the warp takes part.
template <int NV>
MOE_DEV void store_row_e4m3(const float (&v)[NV][8], uint8_t* q, float* s, int64_t lds, int d, int th, int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * th + t) * 8;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float sc = f8_scale(m);
        if (c < d) {
            *reinterpret_cast<uint2*>(q + c) = pack8_e4m3(v[i], sc);
            if ((t & 15) == 0) s[int64_t(c >> 7) * lds] = sc;
        }
    }
}

}  // namespace moe

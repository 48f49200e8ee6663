// Activations kept in 8 bits: blocks of 32 columns of a row under one power of two.
//
// A block's scale byte b stands for 2^(b - 127) (255: not a number), its codes are int8 or e4m3 values. The
// writer takes the smallest power of two with max |x| <= 127 2^e (int8) or 448 2^e (e4m3), e >= -126, and
// rounds x / 2^e to the nearest code, ties to even. Scaling by a power of two is exact, so a code does not
// depend on the precision it is computed in, and no division is needed. A block that holds an infinity or a
// NaN gets b = 255 and reads back as NaN throughout.
#pragma once

#include "post.cuh"

namespace rlk {

constexpr int kAct8Block = 32;

// Eight neighbouring columns of a thread; a block is four neighbouring lanes.
constexpr int kVec = 8;

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Eight neighbouring columns as four pairs.
struct V8 {
    f32x2 p[4];
};
__device__ __forceinline__ V8 pairs_of(const float (&v)[kVec]) {
    V8 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.p[k] = pack2(v[2 * k], v[2 * k + 1]);
    return r;
}
__device__ __forceinline__ void floats_of(const V8 &a, float (&v)[kVec]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2(a.p[k], v[2 * k], v[2 * k + 1]);
}
__device__ __forceinline__ V8 bf16_pairs(uint4 a) {
    V8 r;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) r.p[k] = pack2(bf16_lo(w[k]), bf16_hi(w[k]));
    return r;
}
__device__ __forceinline__ V8 f32_pairs(uint4 a, uint4 b) {
    V8 r;
    r.p[0] = pack2(__uint_as_float(a.x), __uint_as_float(a.y));
    r.p[1] = pack2(__uint_as_float(a.z), __uint_as_float(a.w));
    r.p[2] = pack2(__uint_as_float(b.x), __uint_as_float(b.y));
    r.p[3] = pack2(__uint_as_float(b.z), __uint_as_float(b.w));
    return r;
}
// The scale byte of a block from the bits of its largest |x| (as integers, so that NaN is above infinity).
// For 127 = 1.984375 2^6 and 448 = 1.75 2^8 the test is one on the mantissa.
__device__ __forceinline__ uint32_t act8_scale(uint32_t amax, bool e4m3) {
    const int man = (int)(amax & 0x7fffffu);
    const int b = (int)(amax >> 23) - (e4m3 ? 8 : 6) + (man > (e4m3 ? 0x600000 : 0x7e0000) ? 1 : 0);
    return amax >= 0x7f800000u ? 255u : (uint32_t)max(b, 1);
}

// The bits of the largest |v|; a NaN wins.
__device__ __forceinline__ uint32_t act8_amax(const float (&v)[kVec]) {
    float a = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < kVec; ++j) asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(fabsf(v[j])));
    return __float_as_uint(a);
}

// The largest of the four lanes that share a block (every lane of the warp takes part).
__device__ __forceinline__ uint32_t act8_block_max(uint32_t a) {
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// Codes of eight values under scale byte b. int8: adding 1.5 2^23 rounds to a whole number (to nearest even)
// and leaves it in the low byte.
__device__ __forceinline__ uint2 act8_encode(const float (&v)[kVec], uint32_t b, bool e4m3) {
    if (b == 255u) return make_uint2(0u, 0u);
    const float inv = __uint_as_float((254u - b) << 23);
    uint32_t w[2];
    if (e4m3) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * k + 1] * inv), "f"(v[4 * k] * inv));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * k + 3] * inv), "f"(v[4 * k + 2] * inv));
            w[k] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
    } else {
        uint32_t t[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) t[j] = __float_as_uint(fmaf(v[j], inv, 12582912.f));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = __byte_perm(__byte_perm(t[4 * k], t[4 * k + 1], 0x0040), __byte_perm(t[4 * k + 2], t[4 * k + 3], 0x0040), 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

// What eight codes stand for, as pairs. An int8 code plus 128 in the low byte of 2^23 is 2^23 + 128 + code, and
// times s the difference is exact. An e4m3 code's 7 low bits, put where fp32 has its exponent and mantissa, are the
// value times 2^-120 (subnormal codes included). Where products may pass fp32's range (a code can stand for a
// value that was rounded up to 2^128), they end at +-`most`, the largest finite value of the type that is read back.
__device__ __forceinline__ V8 act8_decode(uint2 c, uint32_t b, bool e4m3, float most) {
    const float s = __uint_as_float(b == 255u ? 0x7fc00000u : (b ? b << 23 : 0x00400000u));
    const bool plain = b <= (e4m3 ? 134u : 230u);
    V8 r;
    if (e4m3) {
        const float k = plain ? s * 0x1p120f : 0x1p120f;
        const f32x2 mul = pack2(k, k);
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[j] = (uint32_t)((int32_t)__byte_perm(w[i >> 1], 0u, 0x0444u | (uint32_t)((2 * i + j) & 3) << 12) >> 4) & 0x87f00000u;
            r.p[i] = mul2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), mul);
        }
    } else {
        const float m = plain ? s : 1.f;
        const f32x2 mul = pack2(m, m), off = pack2(-8388736.f * m, -8388736.f * m);
        const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.p[i] = fma2(pack2(__uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7440u | (2 * i & 3))),
                                __uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7440u | ((2 * i + 1) & 3)))), mul, off);
    }
    if (!plain) {
        float v[kVec];
        floats_of(r, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            v[j] *= s;
            if (fabsf(v[j]) > most) v[j] = copysignf(most, v[j]);  // (NaN stays)
        }
        r = pairs_of(v);
    }
    return r;
}

// The factor of scale byte b: 2^(b - 127), NaN for 255. (Bit 22 is both 2^-127, for 0, and what makes an infinity NaN.)
__device__ __forceinline__ float act8_factor(uint32_t b) { return __uint_as_float(b << 23 | (((b + 1u) & 255u) <= 1u ? 1u << 22 : 0u)); }

// What eight codes stand for in fp32, plus `add` (ADD), without branches; a value past fp32's range is infinite. `s` is the
// block's act8_factor: a code's own value is exact and its product with a power of two is too, so that the sum is rounded once.
template <bool E4M3, bool ADD>
__device__ __forceinline__ V8 act8_decode_plus(uint2 c, float s, f32x2 add) {
    const f32x2 mul = pack2(s, s);
    V8 r;
    if (E4M3) {
        const f32x2 up = pack2(0x1p120f, 0x1p120f);
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[j] = (uint32_t)((int32_t)__byte_perm(w[i >> 1], 0u, 0x0444u | (uint32_t)((2 * i + j) & 3) << 12) >> 4) & 0x87f00000u;
            r.p[i] = mul2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), up);
        }
    } else {
        const f32x2 off = pack2(-8388736.f, -8388736.f);
        const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.p[i] = add2(pack2(__uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7440u | (2 * i & 3))),
                                __uint_as_float(__byte_perm(w[i >> 1], 0x4b000000u, 0x7440u | ((2 * i + 1) & 3)))), off);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = ADD ? fma2(r.p[i], mul, add) : mul2(r.p[i], mul);
    return r;
}

// ---------------------------------------------------------------- eight columns of a row in memory
//
// `fast` (one flag per matrix, from its address and row stride): rows start on 16-byte boundaries (2: 32-byte ones)
// and are read up to their length rounded up to those; otherwise single columns are read and written.

__device__ __forceinline__ void ld32(const void *p, uint4 &a, uint4 &b) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}

struct Raw16 { uint4 a; };
struct Raw32 { uint4 a, b; };

__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ void load_raw(Raw16 &r, const __nv_bfloat16 *row, int col, int) { r.a = ld16(row + col); }
__device__ __forceinline__ void load_raw(Raw32 &r, const float *row, int col, int cols) {
    r.a = *reinterpret_cast<const uint4 *>(row + col);
    r.b = col + 4 < cols ? *reinterpret_cast<const uint4 *>(row + col + 4) : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ void to_float(const Raw16 &r, float (&v)[kVec]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
}
__device__ __forceinline__ void to_float(const Raw32 &r, float (&v)[kVec]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
}

// Sets what lies past the row's end to 0.
__device__ __forceinline__ void clip_row(float (&v)[kVec], int col, int cols) {
    if (col + kVec > cols) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (col + j >= cols) v[j] = 0.f;
    }
}

// Eight values rounded once to the matrix's type; nothing past the row's end is written.
__device__ __forceinline__ void store_vec(__nv_bfloat16 *row, int col, int cols, bool fast, const float (&v)[kVec]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    if (fast && col + kVec <= cols) {
        *reinterpret_cast<uint4 *>(row + col) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    uint16_t *p = reinterpret_cast<uint16_t *>(row) + col;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (col + j < cols) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}
__device__ __forceinline__ void store_vec(float *row, int col, int cols, bool fast, const float (&v)[kVec]) {
    if (fast && col + kVec <= cols) {
        *reinterpret_cast<float4 *>(row + col) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(row + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (col + j < cols) row[col + j] = v[j];
}
// The same in one store of 32 bytes (rows on 32-byte boundaries): two stores of 16 write every second half of a warp's
// 32-byte pieces of memory, and each write of half a piece costs as much as a whole one (unpacking to fp32 67% of the
// copy rate so, 94% in one store).
__device__ __forceinline__ void st32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                 "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void store_vec32(float *row, int col, const float (&v)[kVec]) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = __float_as_uint(v[j]);
    st32(row + col, w);
}
__device__ __forceinline__ void store_codes(uint8_t *row, int col, int cols, bool fast, uint2 c) {
    if (fast && col + kVec <= cols) {
        *reinterpret_cast<uint2 *>(row + col) = c;
        return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (col + j < cols) row[col + j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
}

// ---------------------------------------------------------------- parameters

// A matrix: its first element, the row stride in elements, and whether vector accesses are allowed (2: of 32 bytes).
struct RowMat {
    void *p;
    int64_t ld;
    int32_t bf16;
    int32_t fast;
};

struct Act8Mat {
    uint8_t *codes, *scales;
    int64_t ld_codes, ld_scales;
    int32_t e4m3;
    int32_t fast;
};

struct Act8Params {
    RowMat x;
    Act8Mat a;
    int64_t rows;
    int32_t cols;
    int32_t row_parts;      // parts of a row, one thread each
    int64_t step_rows;      // rows and parts that the grid's threads step over
    int32_t step_parts;
};

cudaError_t launch_act8_pack(Act8Params p, cudaStream_t stream);
cudaError_t launch_act8_unpack(Act8Params p, cudaStream_t stream);

// A row of a matrix of either type.
__device__ __forceinline__ void store_row(const RowMat &m, int64_t row, int col, int cols, const float (&v)[kVec]) {
    if (m.bf16)
        store_vec(static_cast<__nv_bfloat16 *>(m.p) + row * m.ld, col, cols, m.fast, v);
    else if (m.fast == 2 && col + kVec <= cols)
        store_vec32(static_cast<float *>(m.p) + row * m.ld, col, v);
    else
        store_vec(static_cast<float *>(m.p) + row * m.ld, col, cols, m.fast, v);
}

}  // namespace rlk

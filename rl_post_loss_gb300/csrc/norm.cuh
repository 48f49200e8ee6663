// Layer norm and RMS norm over rows of activations, forward and backward (internal).
//
//   forward   h = x (+ residual, rounded to the type of x);  y = (h - mean) rstd w + b
//             mean = sum h / C,  rstd = (sum (h - mean)^2 / C + eps)^-1/2;  RMS: mean = 0
//   backward  xh = (h - mean) rstd,  g = dy w
//             dx = rstd (g - mean(g) - xh mean(g xh)) + dsummed     (RMS: without mean(g))
//             dw = sum over rows of dy xh,  db = sum over rows of dy
//
// All arithmetic is fp32. A row's columns lie over `lanes` threads in vectors of eight; thread t has vectors
// t, t + lanes, ... . Rows of up to 256 columns share a warp or take one, longer ones take the 1 to 16 warps
// of a block.
#pragma once

#include "act8.cuh"
#include "post.cuh"

namespace rlk {

constexpr int kNormMaxCols = 16384;
constexpr int kNormSMs = 152;

struct NormForwardParams {
    RowMat x, residual, y, h;  // p = nullptr where there is none
    Act8Mat ckpt;              // codes = nullptr: none
    const void *w, *b;         // [cols] or nullptr
    int32_t params_bf16, params_fast;
    const uint8_t *mask;
    float *mean, *rstd;        // or nullptr
    int32_t rows, cols, rms, lanes;
    float eps, inv_cols;
    uint32_t *status;
};

struct NormBackwardParams {
    RowMat dy, x, dsummed, dx, y;  // x.p = nullptr: from ckpt
    Act8Mat ckpt;
    const void *w, *b;
    int32_t params_bf16, params_fast;
    const uint8_t *mask;
    const float *mean, *rstd;
    int32_t rows, cols, rms, lanes;
    float inv_cols;
    float *partials;   // [parts][1 or 2][ld_part]: dw, then db
    int64_t ld_part;
    int32_t want_dw, want_db;
    float *dw, *db;
    int32_t accumulate;  // dw and db are added to
    uint32_t *status;
};

// How a norm's rows are laid over threads.
struct NormShape {
    int lanes;    // threads of a row
    int vecs;     // vectors of a thread
    int threads;  // of a block
    int groups;   // rows that a block works on at a time
};
NormShape norm_shape(int cols);

// Blocks of the backward pass, which is also the number of partial sums of dw and db.
int norm_backward_parts(int rows, int cols);

cudaError_t launch_norm_forward(const NormForwardParams &p, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormBackwardParams &p, cudaStream_t stream);
cudaError_t launch_norm_ring_bf16(const NormBackwardParams &p, const struct NormRing &r, int parts, cudaStream_t stream);
cudaError_t launch_norm_ring_f32(const NormBackwardParams &p, const struct NormRing &r, int parts, cudaStream_t stream);
cudaError_t launch_norm_ring_act8(const NormBackwardParams &p, const struct NormRing &r, int parts, cudaStream_t stream);

constexpr size_t kNormRingSmem = 226 * 1024;  // of a block

// The backward pass of rows that bulk copies can take (16-byte aligned ones): how many blocks of how many warps,
// and how many rows' room each block has in shared memory. depth = 0: the rows do not fit.
struct NormRing {
    int warps, vecs, blocks_per_sm, depth;
    size_t h_bytes, dy_bytes, ds_bytes, w_bytes, smem;  // of a row, of the weight, of a block
};

// ---------------------------------------------------------------- device helpers

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
__device__ __forceinline__ V8 clipped(const V8 &a, int col, int cols) {
    float v[kVec];
    floats_of(a, v);
    clip_row(v, col, cols);
    return pairs_of(v);
}
// act8_decode for fp32, as pairs.
__device__ __forceinline__ V8 act8_pairs(uint2 c, uint32_t b, bool e4m3) {
    float v[kVec];
    if (!e4m3 && b <= 230u) {
        const float s = __uint_as_float(b ? b << 23 : 0x00400000u);
        const f32x2 mul = pack2(s, s), off = pack2(-8388736.f * s, -8388736.f * s);
        const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
        V8 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = w[k >> 1];
            r.p[k] = fma2(pack2(__uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440u | (2 * k & 3))),
                                __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440u | ((2 * k + 1) & 3)))), mul, off);
        }
        return r;
    }
    act8_decode(c, b, e4m3, __uint_as_float(0x7f7fffffu), v);
    return pairs_of(v);
}
__device__ __forceinline__ float sum_of(f32x2 a) {
    float x, y;
    unpack2(a, x, y);
    return x + y;
}

// Sums over the threads of a row. Inside a warp a butterfly, so that every lane has the same bits; over a
// block's warps one exchange through shared memory (two buffers in turn: a thread may still read the last
// one while another writes the next), added in the order of the warps.
template <int LANES>
struct RowSum {
    float (*buf)[2][16];
    int turn;
    __device__ __forceinline__ RowSum(float (*b)[2][16]) : buf(b), turn(0) {}

    template <int N>
    __device__ __forceinline__ void run(float (&v)[N]) {
        static_assert(N <= 2, "two sums at most");
#pragma unroll
        for (int off = (LANES < 32 ? LANES : 32) / 2; off > 0; off >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = __fadd_rn(v[n], __shfl_xor_sync(0xffffffffu, v[n], off));
        if (LANES <= 32) return;
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) buf[turn][n][threadIdx.x >> 5] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = buf[turn][n][0];
            for (int w = 1; w < warps; ++w) s = __fadd_rn(s, buf[turn][n][w]);
            v[n] = s;
        }
        turn ^= 1;
    }
};

__device__ __forceinline__ void load_params(const void *p, int bf16, int fast, int col, int cols, float (&v)[kVec]) {
    if (bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(p) + col;
        if (fast && col + kVec <= cols) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(q));
            to_float(Raw16{a}, v);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = col + j < cols ? __uint_as_float((uint32_t)__ldg(q + j) << 16) : 0.f;
        }
    } else {
        const float *q = static_cast<const float *>(p) + col;
        if (fast && col + kVec <= cols) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(q)), b = __ldg(reinterpret_cast<const float4 *>(q) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = col + j < cols ? __ldg(q + j) : 0.f;
        }
    }
}

}  // namespace rlk

// Layer norm and RMS norm over rows of activations, forward and backward (internal).
//
//   forward   h = x (+ residual, rounded to the type of x);  y = (h - mean) rstd w + b
//             mean = sum h / C,  rstd = (sum (h - mean)^2 / C + eps)^-1/2;  RMS: mean = 0
//   backward  xh = (h - mean) rstd,  g = dy w
//             dx = rstd (g - mean(g) - xh mean(g xh)) + dsummed     (RMS: without mean(g))
//             dw = sum over rows of dy xh,  db = sum over rows of dy
//
// All arithmetic is fp32. The backward pass works with r = dy rstd, u = r w, d = h - mean, so that dw += r d,
// rstd mean(g) = mean(u), mean(g xh) = mean(u d), dx = u - mean(u) - d k + dsummed with k = rstd^2 mean(u d).
// A block of the backward pass keeps the sums of dw and db over its rows and leaves them as one partial sum
// of a column; a second launch adds the partial sums.
#pragma once

#include <atomic>

#include "act8.cuh"
#include "norm_layout.cuh"

namespace rlk {

static_assert(kNormVec == kVec, "");

struct NormForwardParams {
    RowMat x, residual, y, h;  // p = nullptr where there is none
    Act8Mat ckpt;              // codes = nullptr: none
    const void *w, *b;         // [cols] or nullptr
    int32_t params_bf16, params_fast;
    const uint8_t *mask;
    float *mean, *rstd;        // or nullptr
    int32_t rows, cols, rms;
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
    int32_t rows, cols, rms;
    float inv_cols;
    float *partials;   // [parts][2][ld_part]: dw, then db
    int64_t ld_part;
    int32_t want_dw, want_db;
    float *dw, *db;
    int32_t accumulate;  // dw and db are added to
    uint32_t *status;
};

cudaError_t launch_norm_forward(const NormForwardParams &p, cudaStream_t stream);
cudaError_t launch_norm_forward_any(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream);
cudaError_t launch_norm_forward_shift(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormBackwardParams &p, cudaStream_t stream);
// The backward pass's kernels by the types of h and dy.
#define RLK_NORM_ROWS(H, DY) cudaError_t launch_norm_rows_##H##_##DY(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream)
RLK_NORM_ROWS(bf16, bf16);
RLK_NORM_ROWS(bf16, f32);
RLK_NORM_ROWS(f32, bf16);
RLK_NORM_ROWS(f32, f32);
RLK_NORM_ROWS(int8, bf16);
RLK_NORM_ROWS(int8, f32);
RLK_NORM_ROWS(e4m3, bf16);
RLK_NORM_ROWS(e4m3, f32);
#undef RLK_NORM_ROWS

// Launches a kernel that may take `most` bytes of shared memory, which the driver is told once on a device (some 0.5 us of
// host time).
template <auto Kernel, typename... Args>
cudaError_t run_kernel(int blocks, int threads, size_t smem, size_t most, cudaStream_t stream, Args... args) {
    static std::atomic<uint64_t> told{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(told.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        told.fetch_or(bit, std::memory_order_relaxed);
    }
    Kernel<<<blocks, threads, smem, stream>>>(args...);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- device helpers

// The next launch, if it is one that waits for this one (grid_dependency_wait), may begin.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ V8 clipped(const V8 &a, int col, int cols) {
    float v[kVec];
    floats_of(a, v);
    clip_row(v, col, cols);
    return pairs_of(v);
}
__device__ __forceinline__ float sum_of(f32x2 a) {
    float x, y;
    unpack2(a, x, y);
    return x + y;
}
// A thread's sum, kept as two chains of pairs, as one would be waited for.
__device__ __forceinline__ float sum_of(const f32x2 (&a)[2]) { return sum_of(add2(a[0], a[1])); }
__device__ __forceinline__ V8 zeros() {
    V8 r;
    r.p[0] = r.p[1] = r.p[2] = r.p[3] = 0ull;
    return r;
}

// The sums over a block's warps (or, with WARP, over the warp) of two values (BOTH) or of the second one: a
// butterfly in each warp, which for two values first gives each half of the warp one of them; then another
// over the warps' sums from shared memory (`buf`: 16 places, the unused ones 0; two buffers in turn, as a thread may
// still read the last one while another writes the next). Every thread gets the same bits.
template <bool BOTH>
__device__ __forceinline__ float warp_sums(float a, float b) {  // BOTH: a's sum in lanes 0 to 15, b's in the others
    const int lane = threadIdx.x & 31;
    float v = b;
    if (BOTH) {
        const float give = lane < 16 ? b : a, keep = lane < 16 ? a : b;
        v = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, 16));
    }
#pragma unroll
    for (int off = BOTH ? 8 : 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
template <bool BOTH, bool WARP>
__device__ __forceinline__ void team_sums(float &a, float &b, float2 *buf, int warps) {
    const int lane = threadIdx.x & 31;
    const float v = warp_sums<BOTH>(a, b);
    if (WARP) {
        if (BOTH) a = __shfl_sync(0xffffffffu, v, 0);
        b = BOTH ? __shfl_sync(0xffffffffu, v, 16) : v;
        return;
    }
    if (BOTH ? (lane & 15) == 0 : lane == 0) reinterpret_cast<float *>(buf + (threadIdx.x >> 5))[BOTH ? lane >> 4 : 1] = v;
    __syncthreads();
    float2 x = buf[lane & (warps > 8 ? 15 : 7)];
    if (warps > 8) {
        if (BOTH) x.x = __fadd_rn(x.x, __shfl_xor_sync(0xffffffffu, x.x, 8));
        x.y = __fadd_rn(x.y, __shfl_xor_sync(0xffffffffu, x.y, 8));
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
        if (BOTH) x.x = __fadd_rn(x.x, __shfl_xor_sync(0xffffffffu, x.x, off));
        x.y = __fadd_rn(x.y, __shfl_xor_sync(0xffffffffu, x.y, off));
    }
    if (BOTH) a = x.x;
    b = x.y;
}

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
__device__ __forceinline__ float load_param(const void *p, int bf16, int col) {
    return bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(p) + col) << 16) : __ldg(static_cast<const float *>(p) + col);
}

// A block's partial sum of dw or db: the teams' sums, which they left in shared memory, added in their order.
__device__ __forceinline__ void join_teams(const float *sums, int teams, int ld, int cols, float *part) {
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < teams; ++k) s += sums[k * ld + c];
        part[c] = s;
    }
}

}  // namespace rlk

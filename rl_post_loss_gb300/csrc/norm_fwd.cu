// The forward pass of the norms (mathematics and layout: norm.cuh).
#include "norm.cuh"

namespace rlk {

namespace {

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

template <typename T>
struct RawOf;
template <>
struct RawOf<__nv_bfloat16> { using type = Raw16; };
template <>
struct RawOf<float> { using type = Raw32; };

// One row at a time per group of threads, held in registers between the statistics and the output. The
// variance is a second sum over the registers, of squares of differences from the mean, together with the
// sum of these differences: what rounding left of the mean is taken off both.
template <typename T, int VPT, int LANES>
__global__ void __launch_bounds__(512) norm_forward_kernel(NormForwardParams p) {
    using Raw = typename RawOf<T>::type;
    __shared__ float s_buf[2][2][16];
    RowSum<LANES> sums(s_buf);
    const int lanes = p.lanes, groups = blockDim.x / lanes, group = threadIdx.x / lanes, t = threadIdx.x - group * lanes;
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += (int64_t)gridDim.x * groups) {
        const int64_t row = r0 + group;
        const bool mine = row < p.rows;
        const bool on = mine && (!p.mask || p.mask[row]);
        float v[VPT][kVec];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[i][j] = 0.f;
            if (on && col < p.cols) {
                Raw r;
                load_raw(r, static_cast<const T *>(p.x.p) + row * p.x.ld, col, p.cols, p.x.fast);
                to_float(r, v[i]);
            }
        }
        if (p.residual.p) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (on && col < p.cols) {
                    Raw r;
                    float u[kVec];
                    load_raw(r, static_cast<const T *>(p.residual.p) + row * p.residual.ld, col, p.cols, p.residual.fast);
                    to_float(r, u);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        v[i][j] += u[j];
                        if (sizeof(T) == 2) v[i][j] = __bfloat162float(__float2bfloat16_rn(v[i][j]));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) clip_row(v[i], (t + i * lanes) * kVec, p.cols);
        if (mine && p.h.p)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (col < p.cols) store_vec(static_cast<T *>(p.h.p) + row * p.h.ld, col, p.cols, p.h.fast, v[i]);
            }
        if (p.ckpt.codes) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                const uint32_t b = act8_scale(act8_block_max(act8_amax(v[i])), p.ckpt.e4m3);
                if (mine && col < p.cols) {
                    store_codes(p.ckpt.codes + row * p.ckpt.ld_codes, col, p.cols, p.ckpt.fast, act8_encode(v[i], b, p.ckpt.e4m3));
                    if ((vec & 3) == 0) p.ckpt.scales[row * p.ckpt.ld_scales + (vec >> 2)] = (uint8_t)b;
                }
            }
        }

        float mean = 0.f, var;
        if (p.rms) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) s[0] = fmaf(v[i][j], v[i][j], s[0]);
            sums.run(s);
            var = s[0] * p.inv_cols;
        } else {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) s[0] += v[i][j];
            sums.run(s);
            mean = s[0] * p.inv_cols;
            float d[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] -= mean;
                if (col + kVec > p.cols) clip_row(v[i], col, p.cols);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    d[0] += v[i][j];
                    d[1] = fmaf(v[i][j], v[i][j], d[1]);
                }
            }
            sums.run(d);
            const float rest = d[0] * p.inv_cols;
            var = fmaxf(fmaf(-rest, rest, d[1] * p.inv_cols), 0.f) + (d[1] - d[1]);  // (NaN stays)
            mean += rest;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] -= rest;
        }
        const float rstd = __frsqrt_rn(var + p.eps);
        if (!mine) continue;
        if (t == 0) {
            if (on && !(var < INFINITY) && p.status) raise_status(p.status, RL_ERR_NONFINITE);
            if (p.mean) p.mean[row] = on ? mean : 0.f;
            if (p.rstd) p.rstd[row] = on ? rstd : 0.f;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (col >= p.cols) continue;
            float w[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[i][j] *= rstd;
            if (p.w) {
                load_params(p.w, p.params_bf16, p.params_fast, col, p.cols, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] *= w[j];
            }
            if (p.b) {
                load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] += w[j];
            }
            if (!on)
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] = 0.f;
            store_row(p.y, row, col, p.cols, v[i]);
        }
    }
}

template <typename T, int VPT, int LANES>
cudaError_t launch(const NormForwardParams &p, const NormShape &s, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)p.rows + s.groups - 1) / s.groups;
    const int most = kNormSMs * (2048 / s.threads);
    norm_forward_kernel<T, VPT, LANES><<<(int)(blocks < most ? blocks : most), s.threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_shape(const NormForwardParams &p, const NormShape &s, cudaStream_t stream) {
    switch (s.lanes) {
        case 8: return launch<T, 1, 8>(p, s, stream);
        case 16: return launch<T, 1, 16>(p, s, stream);
        case 32: return launch<T, 1, 32>(p, s, stream);
    }
    switch (s.vecs) {
        case 1: return launch<T, 1, 64>(p, s, stream);
        case 2: return launch<T, 2, 64>(p, s, stream);
        case 3: return launch<T, 3, 64>(p, s, stream);
        default: return launch<T, 4, 64>(p, s, stream);
    }
}

}  // namespace

// Rows of up to 256 columns: 8, 16 or 32 lanes, a vector each. Longer rows: the fewest warps that hold them in
// three vectors a thread, in four beyond 12288 columns (16 warps at most).
NormShape norm_shape(int cols) {
    const int vecs = (cols + kVec - 1) / kVec;
    NormShape s;
    if (vecs <= 32) {
        s.lanes = vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
        s.vecs = 1;
        s.threads = 128;
        s.groups = s.threads / s.lanes;
        return s;
    }
    int warps = (vecs + 95) / 96;
    if (warps > 16) warps = 16;
    if (warps < 2) warps = 2;
    s.lanes = s.threads = warps * 32;
    s.vecs = (vecs + s.lanes - 1) / s.lanes;
    s.groups = 1;
    return s;
}

cudaError_t launch_norm_forward(const NormForwardParams &q, cudaStream_t stream) {
    NormForwardParams p = q;
    const NormShape s = norm_shape(p.cols);
    p.lanes = s.lanes;
    return p.x.bf16 ? launch_shape<__nv_bfloat16>(p, s, stream) : launch_shape<float>(p, s, stream);
}

}  // namespace rlk

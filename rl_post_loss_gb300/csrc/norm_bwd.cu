// The backward pass of the norms (mathematics and layout: norm.cuh).
#include <algorithm>

#include "norm.cuh"

namespace rlk {

namespace {

constexpr int kJoinCols = 32, kJoinRows = 8;

struct Bf16Rows {
    using Raw = Raw16;
    static __device__ __forceinline__ void load(Raw &r, const RowMat &m, int64_t row, int col, int cols) {
        load_raw(r, static_cast<const __nv_bfloat16 *>(m.p) + row * m.ld, col, cols, m.fast);
    }
};
struct F32Rows {
    using Raw = Raw32;
    static __device__ __forceinline__ void load(Raw &r, const RowMat &m, int64_t row, int col, int cols) {
        load_raw(r, static_cast<const float *>(m.p) + row * m.ld, col, cols, m.fast);
    }
};

// h from where the forward pass left it.
struct FromBf16 {
    Raw16 r;
    __device__ __forceinline__ void load(const NormBackwardParams &p, int64_t row, int col) { Bf16Rows::load(r, p.x, row, col, p.cols); }
    __device__ __forceinline__ void get(const NormBackwardParams &, float (&v)[kVec]) const { to_float(r, v); }
};
struct FromF32 {
    Raw32 r;
    __device__ __forceinline__ void load(const NormBackwardParams &p, int64_t row, int col) { F32Rows::load(r, p.x, row, col, p.cols); }
    __device__ __forceinline__ void get(const NormBackwardParams &, float (&v)[kVec]) const { to_float(r, v); }
};
struct FromAct8 {
    Raw8 r;
    uint32_t b;
    __device__ __forceinline__ void load(const NormBackwardParams &p, int64_t row, int col) {
        load_raw(r, p.ckpt.codes + row * p.ckpt.ld_codes, col, p.cols, p.ckpt.fast);
        b = p.ckpt.scales[row * p.ckpt.ld_scales + col / kAct8Block];
    }
    __device__ __forceinline__ void get(const NormBackwardParams &p, float (&v)[kVec]) const {
        act8_decode(r.a, b, p.ckpt.e4m3, __uint_as_float(0x7f7fffffu), v);
    }
};

// A block takes rows in turn and keeps, in every thread, the sums of dw (and db) over them for that thread's
// columns; it leaves them as one of the partial sums that norm_join_kernel adds.
template <typename From, typename Dy, int VPT, int LANES, bool DB>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormBackwardParams p) {
    __shared__ float s_buf[2][2][16];
    RowSum<LANES> sums(s_buf);
    const int lanes = p.lanes, groups = blockDim.x / lanes, group = threadIdx.x / lanes, t = threadIdx.x - group * lanes;
    float dw[VPT][kVec], db[DB ? VPT : 1][kVec];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            dw[i][j] = 0.f;
            if (DB) db[i][j] = 0.f;
        }
    for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < p.rows; r0 += (int64_t)gridDim.x * groups) {
        const int64_t row = r0 + group;
        const bool mine = row < p.rows;
        const bool on = mine && (!p.mask || p.mask[row]);
        From h[VPT];
        typename Dy::Raw dy[VPT];
        float mean = 0.f, rstd = 0.f;
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (col < p.cols) {
                    h[i].load(p, row, col);
                    Dy::load(dy[i], p.dy, row, col, p.cols);
                }
            }
            rstd = p.rstd[row];
            if (!p.rms) mean = p.mean[row];
        }
        float s[2] = {0.f, 0.f};
        float xh[VPT][kVec], g[VPT][kVec];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
#pragma unroll
            for (int j = 0; j < kVec; ++j) xh[i][j] = g[i][j] = 0.f;
            if (!on || col >= p.cols) continue;
            h[i].get(p, xh[i]);
            to_float(dy[i], g[i]);
#pragma unroll
            for (int j = 0; j < kVec; ++j) xh[i][j] = (xh[i][j] - mean) * rstd;
            if (col + kVec > p.cols) {
                clip_row(xh[i], col, p.cols);
                clip_row(g[i], col, p.cols);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                if (DB) db[i][j] += g[i][j];
            }
            if (p.w) {
                float w[kVec];
                load_params(p.w, p.params_bf16, p.params_fast, col, p.cols, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) g[i][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                s[0] += g[i][j];
                s[1] = fmaf(g[i][j], xh[i][j], s[1]);
            }
        }
        sums.run(s);
        const float c1 = p.rms ? 0.f : s[0] * p.inv_cols, c2 = s[1] * p.inv_cols;
        if (!mine) continue;
        if (t == 0 && on && p.status && !(fabsf(s[0]) < INFINITY && fabsf(s[1]) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (col >= p.cols) continue;
            float o[kVec];
            if (p.y.p) {
                float w[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) o[j] = xh[i][j];
                if (p.w) {
                    load_params(p.w, p.params_bf16, p.params_fast, col, p.cols, w);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) o[j] *= w[j];
                }
                if (p.b && on) {
                    load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, w);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) o[j] += w[j];
                }
                store_row(p.y, row, col, p.cols, o);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) o[j] = on ? rstd * (g[i][j] - c1 - xh[i][j] * c2) : 0.f;
            if (on && p.dsummed.p) {
                float u[kVec];
                if (p.dsummed.bf16) {
                    Raw16 r;
                    Bf16Rows::load(r, p.dsummed, row, col, p.cols);
                    to_float(r, u);
                } else {
                    Raw32 r;
                    F32Rows::load(r, p.dsummed, row, col, p.cols);
                    to_float(r, u);
                }
#pragma unroll
                for (int j = 0; j < kVec; ++j) o[j] += u[j];
            }
            store_row(p.dx, row, col, p.cols, o);
        }
    }

    if (!p.want_dw && !p.want_db) return;
    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part;
    if (LANES > 32) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (col < p.cols) {
                store_vec(part, col, (int)p.ld_part, true, dw[i]);
                if (DB) store_vec(part + p.ld_part, col, (int)p.ld_part, true, db[i]);
            }
        }
        return;
    }
    // several rows at a time: the groups' sums added in their order
    __shared__ float s_join[LANES <= 32 ? 128 * kVec : 1];
#pragma unroll
    for (int which = 0; which < (DB ? 2 : 1); ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kVec; ++j) s_join[threadIdx.x * kVec + j] = which ? db[0][j] : dw[0][j];
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < groups; ++k) s += s_join[k * lanes * kVec + c];
            part[which * p.ld_part + c] = s;
        }
    }
}

// Adds the partial sums of a column in a fixed order: eight threads take every eighth, their sums are added in turn.
__global__ void __launch_bounds__(kJoinCols * kJoinRows) norm_join_kernel(const float *partials, int64_t ld, int parts, int cols, float *dw, float *db, int accumulate) {
    __shared__ float s[kJoinRows][kJoinCols];
    const int c = blockIdx.x * kJoinCols + threadIdx.x, k = threadIdx.y;
    const int which = dw ? (int)blockIdx.y : 1;
    float *out = which ? db : dw;
    float v = 0.f;
    if (c < cols)
        for (int i = k; i < parts; i += kJoinRows) v += partials[((int64_t)i * 2 + which) * ld + c];
    s[k][threadIdx.x] = v;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < kJoinRows; ++i) v += s[i][threadIdx.x];
        out[c] = accumulate ? out[c] + v : v;
    }
}

cudaError_t launch_join(const NormBackwardParams &p, int parts, cudaStream_t stream) {
    if (!p.want_dw && !p.want_db) return cudaSuccess;
    const dim3 grid((p.cols + kJoinCols - 1) / kJoinCols, p.want_dw && p.want_db ? 2 : 1);
    norm_join_kernel<<<grid, dim3(kJoinCols, kJoinRows), 0, stream>>>(p.partials, p.ld_part, parts, p.cols, p.want_dw ? p.dw : nullptr, p.want_db ? p.db : nullptr, p.accumulate);
    return cudaGetLastError();
}

// The fewest warps of a block that leave a thread three vectors, 16 at most.
int fewest_warps(int cols) {
    const int vecs = (cols + kVec - 1) / kVec;
    return std::min(16, std::max(1, (vecs + 95) / 96));
}

constexpr size_t kSmemOfSM = 228 * 1024;

// Blocks of up to 16 warps on an SM, 128 registers a thread; the fewest warps a block that leave a thread three
// vectors (four beyond 12288 columns), and stages of the whole SM's shared memory.
NormRing ring_of(const NormBackwardParams &p) {
    NormRing r{};
    const auto row_bytes = [&](size_t es) { return (p.cols * es + 15) / 16 * 16; };
    r.h_bytes = row_bytes(!p.x.p ? 1 : p.x.bf16 ? 2 : 4);
    r.dy_bytes = row_bytes(p.dy.bf16 ? 2 : 4);
    r.ds_bytes = p.dsummed.p ? row_bytes(p.dsummed.bf16 ? 2 : 4) : 0;
    const int vecs = (p.cols + kVec - 1) / kVec;
    r.w_bytes = (size_t)vecs * kVec * 4;
    const size_t stage = r.h_bytes + r.dy_bytes + r.ds_bytes, fixed = r.w_bytes + 32 + 2048;  // (32: an fp32 vector past the row's end)
    int blocks = 16 / fewest_warps(p.cols);
    while (blocks > 1 && blocks * (2 * stage + fixed) > kSmemOfSM) --blocks;
    r.warps = std::min(16 / blocks, (vecs + 31) / 32);
    r.vecs = (vecs + r.warps * 32 - 1) / (r.warps * 32);
    r.warps = (vecs + r.vecs * 32 - 1) / (r.vecs * 32);
    r.blocks_per_sm = blocks;
    const size_t room = std::min(kNormRingSmem, kSmemOfSM / blocks);
    if (room < fixed + 2 * stage) return r;
    r.depth = (int)std::min<size_t>(8, (room - fixed) / stage);
    r.smem = r.depth * stage + r.w_bytes + 32;
    return r;
}

template <typename From, typename Dy, int VPT, int LANES>
cudaError_t launch(const NormBackwardParams &p, const NormShape &s, cudaStream_t stream) {
    const int parts = norm_backward_parts(p.rows, p.cols);
    if (p.want_db)
        norm_backward_kernel<From, Dy, VPT, LANES, true><<<parts, s.threads, 0, stream>>>(p);
    else
        norm_backward_kernel<From, Dy, VPT, LANES, false><<<parts, s.threads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(p, parts, stream) : e;
}

template <typename From, typename Dy>
cudaError_t launch_shape(const NormBackwardParams &p, const NormShape &s, cudaStream_t stream) {
    switch (s.lanes) {
        case 8: return launch<From, Dy, 1, 8>(p, s, stream);
        case 16: return launch<From, Dy, 1, 16>(p, s, stream);
        case 32: return launch<From, Dy, 1, 32>(p, s, stream);
    }
    switch (s.vecs) {
        case 1: return launch<From, Dy, 1, 64>(p, s, stream);
        case 2: return launch<From, Dy, 2, 64>(p, s, stream);
        case 3: return launch<From, Dy, 3, 64>(p, s, stream);
        default: return launch<From, Dy, 4, 64>(p, s, stream);
    }
}

}  // namespace

int norm_backward_parts(int rows, int cols) {
    const NormShape s = norm_shape(cols);
    const int64_t blocks = ((int64_t)rows + s.groups - 1) / s.groups;
    const int ring = s.groups == 1 ? 16 / fewest_warps(cols) : 0;  // blocks on an SM, of either kernel
    const int most = kNormSMs * std::max({ring, 512 / s.threads, 1});
    return (int)(blocks < most ? blocks : most);
}

cudaError_t launch_norm_backward(const NormBackwardParams &q, cudaStream_t stream) {
    NormBackwardParams p = q;
    const NormShape s = norm_shape(p.cols);
    p.lanes = s.lanes;
    const bool act8 = !p.x.p;
    if (p.cols > 256 && (p.dx.bf16 <= p.dy.bf16) && p.dy.fast && (act8 ? p.ckpt.fast : p.x.fast) && (!p.dsummed.p || p.dsummed.fast)) {
        const NormRing r = ring_of(p);
        if (r.depth >= 2) {
            const int parts = std::min(p.rows, kNormSMs * r.blocks_per_sm);
            const cudaError_t e = !act8 ? p.x.bf16 ? launch_norm_ring_bf16(p, r, parts, stream) : launch_norm_ring_f32(p, r, parts, stream)
                                        : launch_norm_ring_act8(p, r, parts, stream);
            return e == cudaSuccess ? launch_join(p, parts, stream) : e;
        }
    }
    if (!p.x.p) return p.dy.bf16 ? launch_shape<FromAct8, Bf16Rows>(p, s, stream) : launch_shape<FromAct8, F32Rows>(p, s, stream);
    if (p.x.bf16) return p.dy.bf16 ? launch_shape<FromBf16, Bf16Rows>(p, s, stream) : launch_shape<FromBf16, F32Rows>(p, s, stream);
    return p.dy.bf16 ? launch_shape<FromF32, Bf16Rows>(p, s, stream) : launch_shape<FromF32, F32Rows>(p, s, stream);
}

}  // namespace rlk

// The forward pass of the norms: rows on 16-byte boundaries (norm_fwd.cuh), short ones among them, and which kernel takes a call.
#include "norm_fwd.cuh"

namespace rlk {

namespace {

// ---------------------------------------------------------------- short rows
//
// Rows on 16-byte boundaries of up to 512 columns: `lanes` threads of a warp (4 to 32) with VPT vectors each, so that
// a warp works on several rows and a row's sums take few steps. The loads of a row go out together.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(256, 4) norm_forward_short_kernel(NormForwardParams p, int lanes) {
    using Raw = typename RawMat<BF16>::type;
    const int lane = threadIdx.x & 31, t = lane & (lanes - 1), per_warp = 32 / lanes;
    const int64_t warp = blockIdx.x + (int64_t)(threadIdx.x >> 5) * gridDim.x, step = (int64_t)gridDim.x * (blockDim.x >> 5) * per_warp;
    for (int64_t base = warp * per_warp; base < p.rows; base += step) {
        const int64_t row = base + lane / lanes;
        const bool mine = row < p.rows, on = mine && (!p.mask || p.mask[row]);
        Raw x[VPT], r[VPT];
        V8 v[VPT];
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (col < p.cols) {
                    load_mat<BF16>(x[i], p.x, row, col, p.cols);
                    if (p.residual.p) load_mat<BF16>(r[i], p.residual, row, col, p.cols);
                }
            }
        }
        f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int vec = t + i * lanes, col = vec * kVec;
            v[i] = zeros();
            if (on && col < p.cols) {
                v[i] = pairs(x[i]);
                if (p.residual.p) v[i] = add_residual<BF16>(v[i], pairs(r[i]));
                if (col + kVec > p.cols) v[i] = clipped(v[i], col, p.cols);
            }
            if (mine && col < p.cols && p.h.p) {
                float f[kVec];
                floats_of(v[i], f);
                store_row(p.h, row, col, p.cols, f);
            }
            if (p.ckpt.codes) {
                float f[kVec];
                floats_of(v[i], f);
                const uint32_t b = act8_scale(act8_block_max(act8_amax(f)), p.ckpt.e4m3);
                if (mine && col < p.cols) {
                    store_codes(p.ckpt.codes + row * p.ckpt.ld_codes, col, p.cols, p.ckpt.fast, act8_encode(f, b, p.ckpt.e4m3));
                    if ((vec & 3) == 0) p.ckpt.scales[row * p.ckpt.ld_scales + (vec >> 2)] = (uint8_t)b;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (p.rms)
                    s1 = fma2(v[i].p[k], v[i].p[k], s1);
                else
                    s0 = add2(s0, v[i].p[k]);
            }
        }
        float b = sum_of(p.rms ? s1 : s0), mean = 0.f, var;
        for (int off = lanes >> 1; off > 0; off >>= 1) b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
        if (p.rms) {
            var = b * p.inv_cols;
        } else {
            mean = b * p.inv_cols;
            const f32x2 nm = pack2(-mean, -mean);
            s0 = s1 = 0ull;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (col >= p.cols) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].p[k] = add2(v[i].p[k], nm);
                if (col + kVec > p.cols) v[i] = clipped(v[i], col, p.cols);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s0 = add2(s0, v[i].p[k]);
                    s1 = fma2(v[i].p[k], v[i].p[k], s1);
                }
            }
            float a = sum_of(s0);
            b = sum_of(s1);
            for (int off = lanes >> 1; off > 0; off >>= 1) {
                a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, off));
                b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
            }
            float rest;
            var = variance(a, b, p.inv_cols, rest);
            mean += rest;
            const f32x2 nr = pack2(-rest, -rest);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].p[k] = add2(v[i].p[k], nr);
        }
        if (!mine) continue;
        const float rstd = finish_stats(p, row, t == 0 && on, mean, var);
        if (t == 0 && !on) {
            if (p.mean) p.mean[row] = 0.f;
            if (p.rstd) p.rstd[row] = 0.f;
        }
        const f32x2 rs = pack2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (col >= p.cols) continue;
            float f[kVec] = {};
            if (on) {
                float u[kVec];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].p[k] = mul2(v[i].p[k], rs);
                if (p.w) {
                    load_params(p.w, p.params_bf16, p.params_fast, col, p.cols, u);
                    const V8 w = pairs_of(u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i].p[k] = mul2(v[i].p[k], w.p[k]);
                }
                if (p.b) {
                    load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, u);
                    const V8 c = pairs_of(u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i].p[k] = add2(v[i].p[k], c.p[k]);
                }
                floats_of(v[i], f);
            }
            store_row(p.y, row, col, p.cols, f);
        }
    }
}

constexpr int kShortCols = 512;
constexpr size_t kSmemOfSM = 228 * 1024, kBlockExtra = 1024 + 1024;  // what a block takes beside its rows

template <bool BF16>
cudaError_t launch_short(const NormForwardParams &p, cudaStream_t stream) {
    constexpr int kVecs = 2;
    int lanes = 4;
    while (lanes * kVecs * kVec < p.cols) lanes *= 2;
    const int64_t blocks = ((int64_t)p.rows * lanes + 255) / 256;
    norm_forward_short_kernel<BF16, kVecs><<<(int)std::min<int64_t>(blocks, kNormSMs * 4), 256, 0, stream>>>(p, lanes);
    return cudaGetLastError();
}

// A block per row, 24 warps on an SM: of the numbers of vectors a thread, the one whose blocks take all rows soonest, by
// a row's time of its vectors and two more for each exchange of sums.
NormTeams teams_of(const NormForwardParams &p, int mode) {
    const int vecs = (p.cols + kVec - 1) / kVec, pad = mode == kAnyRow ? 16 : 0;
    NormTeams n{};
    n.mode = mode;
    n.at_dy = (p.cols * (p.x.bf16 ? 2 : 4) + 15) / 16 * 16 + pad;
    n.stage_bytes = n.at_dy * (p.residual.p ? 2 : 1);
    if (mode == kWarpRow) {
        n.warps = 1;
        n.vecs = vecs > 96 ? 4 : 3;
        n.blocks_per_sm = 2;
        n.depth = (int)std::min<size_t>(kNormDepth, (kSmemOfSM / 2 - kBlockExtra) / (forward_threads(mode) / 32 * n.stage_bytes));
        n.smem = (size_t)(forward_threads(mode) / 32) * n.depth * n.stage_bytes;
        return n;
    }
    double best = 0;
    for (const int v : {1, 2, 3, 4, 6}) {
        if (mode == kAnyRow && v > 4) break;
        const int warps = (vecs + 32 * v - 1) / (32 * v);
        if (warps > forward_threads(mode) / 32 || (v - 1) * warps * 32 >= vecs) continue;
        if (mode == kAnyRow && v > 2 && n.warps) continue;  // (single columns take more registers)
        int blocks = forward_warps(mode) / warps;
        while (blocks > 1 && blocks * (kBlockExtra + 2 * n.stage_bytes) > kSmemOfSM) --blocks;
        const double time = (double)((p.rows + blocks * kNormSMs - 1) / (blocks * kNormSMs)) * (v + (p.rms ? 2 : 4));
        if (n.warps && time >= best) continue;
        best = time;
        n.warps = warps, n.vecs = v, n.blocks_per_sm = blocks;
        n.depth = (int)std::min<size_t>(kNormDepth, std::min(kNormRingSmem, kSmemOfSM / blocks - kBlockExtra) / n.stage_bytes);
        n.smem = (size_t)n.depth * n.stage_bytes;
    }
    return n;
}

}  // namespace

cudaError_t launch_norm_forward(const NormForwardParams &p, cudaStream_t stream) {
    const bool fast = p.x.fast && (!p.residual.p || p.residual.fast);
    if (fast && p.cols <= kShortCols) return p.x.bf16 ? launch_short<true>(p, stream) : launch_short<false>(p, stream);
    if (!fast) {
        const NormTeams n = teams_of(p, kAnyRow);
        return launch_norm_forward_any(p, n, stream);
    }
    if (p.cols <= 1024 && p.rows >= kNormSMs * forward_warps(kWarpRow)) {
        const NormTeams n = teams_of(p, kWarpRow);
        if (n.vecs == 3) return p.x.bf16 ? launch_forward_rows<true, 3, kWarpRow>(p, n, stream) : launch_forward_rows<false, 3, kWarpRow>(p, n, stream);
        return p.x.bf16 ? launch_forward_rows<true, 4, kWarpRow>(p, n, stream) : launch_forward_rows<false, 4, kWarpRow>(p, n, stream);
    }
    const NormTeams n = teams_of(p, kBlockRow);
    return p.x.bf16 ? launch_forward_vecs<true, kBlockRow>(p, n, stream) : launch_forward_vecs<false, kBlockRow>(p, n, stream);
}

}  // namespace rlk

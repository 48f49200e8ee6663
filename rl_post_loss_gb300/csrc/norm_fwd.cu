// The forward pass of the norms: rows on 16-byte boundaries (norm_fwd.cuh), short ones among them, and which kernel takes a call.
#include "norm_fwd.cuh"
#include "norm_short.cuh"

namespace rlk {

namespace {

// ---------------------------------------------------------------- short rows (norm_short.cuh)

// EXACT: the threads' vectors are the row's columns to the last one, no mask, and rows of y on 16-byte boundaries.
template <bool BF16, int VPT, bool FULL, bool EXACT>
__global__ void __launch_bounds__(kShortWarps * 32, 1) norm_forward_short_kernel(NormForwardParams p, NormShort n) {
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(8) uint64_t s_full[kShortWarps * kNormDepth];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = n.lanes, t = lane & (lanes - 1), slot = lane / lanes, S = n.depth;
    const int width = lanes * VPT * kVec;
    float *w_smem = reinterpret_cast<float *>(smem + n.smem) - 2 * width, *b_smem = w_smem + width;
    for (int c = threadIdx.x; c < width; c += kShortWarps * 32) {
        const int to = plane_of(c, width / kVec);
        w_smem[to] = c < p.cols ? (p.w ? load_param(p.w, p.params_bf16, c) : 1.f) : 0.f;
        b_smem[to] = c < p.cols && p.b ? load_param(p.b, p.params_bf16, c) : 0.f;
    }
    if (threadIdx.x == 0) {
        for (int k = 0; k < kShortWarps * S; ++k) ptx::mbar_init(ptx::smem_u32(&s_full[k]), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ShortRing ring(n);
    ring.mask = p.mask;
    ring.base[0] = static_cast<const char *>(p.x.p);
    ring.pitch[0] = p.x.ld * (BF16 ? 2 : 4);
    ring.base[1] = static_cast<const char *>(p.residual.p);
    ring.pitch[1] = p.residual.ld * (BF16 ? 2 : 4);
    ring.base[2] = nullptr;
    ring.pitch[2] = 0;
    ring.rows = p.rows;
    char *stages = smem + warp * S * n.stage_bytes;
    ring.stages = ptx::smem_u32(stages);
    ring.full = ptx::smem_u32(&s_full[warp * S]);
    ring.lane = lane;
    ring.per = 32 / lanes;
    const int64_t first = blockIdx.x + (int64_t)warp * gridDim.x, step = (int64_t)gridDim.x * kShortWarps;
    const int64_t batches = ((int64_t)p.rows + ring.per - 1) / ring.per;
    for (int s = 0; s < S; ++s)
        if (first + s * step < batches) ring.fetch(first + s * step, s);
    const auto live = [&](int64_t batch) { return batch * ring.per + slot < p.rows && (EXACT || !p.mask || p.mask[batch * ring.per + slot]); };
    bool dead = false, on = live(first);
    uint32_t phases = 0;
    int s = 0;
    for (int64_t batch = first; batch < batches; batch += step) {
        const bool on_next = live(batch + step);
        const int64_t row = batch * ring.per + slot;
        const bool mine = row < p.rows;
        if (__any_sync(0xffffffffu, on)) {
            if (!dead && !ptx::mbar_wait(ring.full + s * 8, (phases >> s) & 1u, kNormWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
        }
        const char *sx = stages + s * n.stage_bytes + slot * n.row_bytes[0], *sr = stages + s * n.stage_bytes + n.at[1] + slot * n.row_bytes[1];
        V8 v[VPT];
        f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = zeros();
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                if (!EXACT && col >= p.cols) continue;
                v[i] = read_vec<BF16>(sx, vec);
                if (p.residual.p) v[i] = add_residual<BF16>(v[i], read_vec<BF16>(sr, vec));
                if (!EXACT && col + kVec > p.cols) v[i] = clipped(v[i], col, p.cols);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (!FULL || p.rms)
                        s1 = fma2(v[i].p[k], v[i].p[k], s1);
                    else
                        s0 = add2(s0, v[i].p[k]);
                }
            }
        }
        __syncwarp();  // the stage is read
        if (batch + S * step < batches && !__any_sync(0xffffffffu, dead)) ring.fetch(batch + S * step, s);
        if (p.h.p || p.ckpt.codes)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                float f[kVec];
                floats_of(v[i], f);
                if (mine && col < p.cols && p.h.p) store_row(p.h, row, col, p.cols, f);
                if (!p.ckpt.codes) continue;
                const uint32_t b = act8_scale(act8_block_max(act8_amax(f)), p.ckpt.e4m3);
                if (mine && col < p.cols) {
                    store_codes(p.ckpt.codes + row * p.ckpt.ld_codes, col, p.cols, p.ckpt.fast, act8_encode(f, b, p.ckpt.e4m3));
                    if ((vec & 3) == 0) p.ckpt.scales[row * p.ckpt.ld_scales + (vec >> 2)] = (uint8_t)b;
                }
            }
        float b = !FULL || p.rms ? sum_of(s1) : sum_of(s0), mean = 0.f, var;
        for (int off = lanes >> 1; off > 0; off >>= 1) b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
        if (!FULL || p.rms) {
            var = b * p.inv_cols;
        } else {
            mean = b * p.inv_cols;
            const f32x2 nm = pack2(-mean, -mean);
            s0 = s1 = 0ull;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * lanes) * kVec;
                if (!EXACT && col >= p.cols) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].p[k] = add2(v[i].p[k], nm);
                if (!EXACT && col + kVec > p.cols) v[i] = clipped(v[i], col, p.cols);
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
        if (on) {
            const float rstd = finish_stats(p, row, t == 0, mean, var);
            const f32x2 rs = pack2(rstd, rstd);
            const int64_t out = row * p.y.ld;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                if (!EXACT && col >= p.cols) continue;
                const V8 w = read_planes(w_smem, vec, width / kVec);
                V8 c;
                if (FULL) c = read_planes(b_smem, vec, width / kVec);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 x = mul2(v[i].p[k], rs);
                    v[i].p[k] = FULL ? fma2(x, w.p[k], c.p[k]) : mul2(x, w.p[k]);
                }
                float f[kVec];
                floats_of(v[i], f);
                const int end = EXACT ? col + kVec : p.cols;  // (EXACT: no part of a vector)
                if (p.y.bf16)
                    store_vec(static_cast<__nv_bfloat16 *>(p.y.p) + out, col, end, EXACT || p.y.fast, f);
                else if (p.y.fast == 2 && col + kVec <= end)
                    store_vec32(static_cast<float *>(p.y.p) + out, col, f);
                else
                    store_vec(static_cast<float *>(p.y.p) + out, col, end, EXACT || p.y.fast, f);
            }
        } else if (!EXACT && mine) {
            if (t == 0) {
                if (p.mean) p.mean[row] = 0.f;
                if (p.rstd) p.rstd[row] = 0.f;
            }
            const float f[kVec] = {};
            for (int vec = t; vec * kVec < p.cols; vec += lanes) store_row(p.y, row, vec * kVec, p.cols, f);
        }
        on = on_next;
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead && lane == 0)  // (copies in flight end before the block does, or do not within another wait)
        for (int k = 0; k < S; ++k) ptx::mbar_wait(ring.full + k * 8, (phases >> k) & 1u, kNormWaitNs);
}

template <bool BF16>
cudaError_t launch_short(const NormForwardParams &p, cudaStream_t stream) {
    const int es[2] = {BF16 ? 2 : 4, !p.residual.p ? 0 : BF16 ? 2 : 4};
    const int64_t ld[2] = {p.x.ld, p.residual.ld};
    const int width = norm_short_width(p.cols);
    const NormShort n = norm_short(p.cols, es, ld, 2, p.mask != nullptr, kShortWarps, (size_t)width * 8, 0);
    const bool full = !p.rms || p.b;
    const bool exact = p.cols == width && !p.mask && p.y.fast;
#define RLK_RUN(V, F, E) run_kernel<norm_forward_short_kernel<BF16, V, F, E>>(std::min(p.rows, kNormSMs), kShortWarps * 32, n.smem, kNormRingSmem, stream, p, n)
#define RLK_SHORT(V, F) (exact ? RLK_RUN(V, F, true) : RLK_RUN(V, F, false))
    return n.vecs == 2 ? full ? RLK_SHORT(2, true) : RLK_SHORT(2, false) : full ? RLK_SHORT(4, true) : RLK_SHORT(4, false);
#undef RLK_SHORT
#undef RLK_RUN
}

NormForwardShape shape_of(const NormForwardParams &p) {
    const int es = p.x.bf16 ? 2 : 4;
    return NormForwardShape{p.rows, p.cols, es, p.residual.p ? es : 0, p.rms != 0, p.b != nullptr, p.mask != nullptr, p.ckpt.codes != nullptr};
}

}  // namespace

cudaError_t launch_norm_forward(const NormForwardParams &p, cudaStream_t stream) {
    // (with rows that start anywhere on any side: vectors cut up at the store, a warp's stores 16 bytes apart, took 515 us for
    // 8920 x 9118 bf16 with a residual, which takes 182 so, and 112 between rows on 16-byte boundaries)
    const bool fast = p.x.fast && (!p.residual.p || p.residual.fast) && p.y.fast && (!p.h.p || p.h.fast) && (!p.ckpt.codes || p.ckpt.fast);
    if (fast && p.cols <= kShortCols) return p.x.bf16 ? launch_short<true>(p, stream) : launch_short<false>(p, stream);
    const NormForwardShape shape = shape_of(p);
    const RowMode mode = norm_forward_mode(shape, fast);
    const NormTeams n = norm_forward_teams(shape, mode);
    if (!fast) return mode == kShiftRow ? launch_norm_forward_shift(p, n, stream) : launch_norm_forward_any(p, n, stream);
    const bool full = forward_full(shape, mode), warp = mode == kWarpRow;
#define RLK_ROWS(BF16) (warp ? full ? launch_forward_rows<BF16, 3, true, kWarpRow>(p, n, stream) : n.vecs == 3 ? launch_forward_rows<BF16, 3, false, kWarpRow>(p, n, stream) : launch_forward_rows<BF16, 4, false, kWarpRow>(p, n, stream) \
                             : full ? launch_forward_vecs<BF16, true, kBlockRow>(p, n, stream) : launch_forward_vecs<BF16, false, kBlockRow>(p, n, stream))
    return p.x.bf16 ? RLK_ROWS(true) : RLK_ROWS(false);
#undef RLK_ROWS
}

}  // namespace rlk

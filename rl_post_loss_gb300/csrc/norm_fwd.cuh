// The forward pass of the norms (mathematics: norm.cuh; how rows are held and brought: norm_rows.cuh).
//
// A row is read from shared memory once and held in registers between the statistics and the output; its
// stage is filled again as soon as the first exchange of sums shows that every thread has read it. The
// variance is a second sum over the registers, of squares of differences from the mean, together with the sum
// of these differences: what rounding left of the mean is taken off both.
//
// Bound by memory where a row has one exchange of sums or is short enough for three blocks on an SM (65536 x 6144 bf16, RMS with a
// residual: 464 us, 102% of the measured copy rate; with an int8 checkpoint 523, 103%); layer norm without a residual waits
// for its two exchanges (16384 x 6144: 79 us, 75%; 16384 x 8192: 122 us, 65%; 65536 x 1024: 66 us, 60%).
#pragma once

#include <algorithm>

#include "norm_rows.cuh"

namespace rlk {


// h's 8-bit codes; a block of 32 columns is four lanes' vectors.
template <int MODE, int VPT>
__device__ __forceinline__ void store_act8(const Columns<MODE, VPT> &at, const Act8Mat &a, int64_t row, int i, const V8 &h) {
    float v[kVec];
    floats_of(h, v);
    const int vec = at.vec(i), col = vec * kVec;
    const uint32_t b = act8_scale(act8_block_max(act8_amax(v)), a.e4m3);
    if (at.none(i)) return;
    store_codes(a.codes + row * a.ld_codes, col, at.cols, a.fast, act8_encode(v, b, a.e4m3));
    if ((vec & 3) == 0) a.scales[row * a.ld_scales + (vec >> 2)] = (uint8_t)b;
}

template <bool BF16>
__device__ __forceinline__ V8 add_residual(V8 x, const V8 &r) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x.p[k] = add2(x.p[k], r.p[k]);
        if (BF16) {  // h is what the type of x holds
            float a, b;
            unpack2(x.p[k], a, b);
            const uint32_t w = pack_bf16x2(a, b);
            x.p[k] = pack2(bf16_lo(w), bf16_hi(w));
        }
    }
    return x;
}

// What follows from a row's sums: the statistics are written by one thread.
__device__ __forceinline__ float finish_stats(const NormForwardParams &p, int64_t row, bool one, float mean, float var) {
    const float rstd = rsqrtf(var + p.eps);  // within 2 units in the last place
    if (one) {
        if (!(var < INFINITY) && p.status) raise_status(p.status, RL_ERR_NONFINITE);
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    return rstd;
}
__device__ __forceinline__ float variance(float sum, float squares, float inv_cols, float &rest) {
    rest = sum * inv_cols;
    const float var = fmaf(-rest, rest, squares * inv_cols);
    return var < 0.f ? 0.f : var;  // (NaN stays)
}

// FULL = false is the RMS form without a bias. A thread's weights and biases stay in registers where there is room.
template <bool BF16, int VPT, bool FULL, int MODE>
__global__ void __launch_bounds__(kForwardWarps * 32, 1) norm_forward_kernel(NormForwardParams p, NormTeams n) {
    constexpr int kTeams = MODE == kWarpRow ? kForwardWarps : 1;
    constexpr bool kHeld = VPT <= (MODE == kAnyRow ? 2 : FULL ? 3 : 4);
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) float2 s_sums[2][16];
    __shared__ __align__(8) uint64_t s_full[kTeams * kNormDepth];
    const int T = MODE == kWarpRow ? 32 : (int)blockDim.x, team = MODE == kWarpRow ? (int)threadIdx.x >> 5 : 0;
    const int t = MODE == kWarpRow ? (int)threadIdx.x & 31 : (int)threadIdx.x, S = n.depth;
    Columns<MODE, VPT> at(t, T, p.cols);
    char *stages = smem + team * S * n.stage_bytes;
    if (threadIdx.x < 32) (&s_sums[0][0])[threadIdx.x] = make_float2(0.f, 0.f);
    if (threadIdx.x == 0) {
        for (int k = 0; k < kTeams * S; ++k) ptx::mbar_init(ptx::smem_u32(&s_full[k]), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const uint32_t full0 = ptx::smem_u32(&s_full[team * S]);
    const int64_t first = blockIdx.x + (int64_t)team * gridDim.x, step = (int64_t)kTeams * gridDim.x;
    const auto x_row = [&](int64_t row) -> const char * { return static_cast<const char *>(p.x.p) + row * p.x.ld * (BF16 ? 2 : 4); };
    const auto r_row = [&](int64_t row) -> const char * { return static_cast<const char *>(p.residual.p) + row * p.residual.ld * (BF16 ? 2 : 4); };
    const auto copy_row = [&](int64_t row, int s) {  // by the team's thread 0
        const uint32_t full = full0 + s * 8, to = ptx::smem_u32(stages + s * n.stage_bytes);
        if (!starts_anywhere(MODE)) {
            ptx::mbar_arrive_expect_tx(full, (uint32_t)(n.copy_bytes[0] + n.copy_bytes[1]));
            ptx::bulk_g2s(to, x_row(row), (uint32_t)n.copy_bytes[0], full);
            if (p.residual.p) ptx::bulk_g2s(to + n.at_dy, r_row(row), (uint32_t)n.copy_bytes[1], full);
            return;
        }
        const int bytes = p.cols * (BF16 ? 2 : 4);
        const uint32_t bx = window(x_row(row), bytes), br = p.residual.p ? window(r_row(row), bytes) : 0u;
        ptx::mbar_arrive_expect_tx(full, bx + br);
        ptx::bulk_g2s(to, x_row(row) - row_shift<MODE>(x_row(row)), bx, full);
        if (br) ptx::bulk_g2s(to + n.at_dy, r_row(row) - row_shift<MODE>(r_row(row)), br, full);
    };
    if (t == 0)
        for (int s = 0; s < S; ++s) {
            const int64_t row = first + s * step;
            if (row < p.rows && (!p.mask || p.mask[row])) copy_row(row, s);
        }

    V8 w_held[kHeld ? VPT : 1], b_held[kHeld && FULL ? VPT : 1];
    if (kHeld)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            w_held[kHeld ? i : 0] = at.none(i) ? zeros() : at.params(p.w, p.params_bf16, p.params_fast, i, 1.f);
            if (FULL) b_held[kHeld && FULL ? i : 0] = at.none(i) ? zeros() : at.params(p.b, p.params_bf16, p.params_fast, i, 0.f);
        }
    // else in shared memory as fp32, a thread's own beside one another, where that fits
    float *w_smem = reinterpret_cast<float *>(smem + kTeams * S * n.stage_bytes), *b_smem = w_smem + VPT * T * kVec;
    if (!kHeld && MODE != kAnyRow && n.w_in_smem)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (at.none(i)) continue;
            write_planes(w_smem, at.vec(i), VPT * T, at.params(p.w, p.params_bf16, p.params_fast, i, 1.f));
            write_planes(b_smem, at.vec(i), VPT * T, at.params(p.b, p.params_bf16, p.params_fast, i, 0.f));
        }
    const auto param = [&](const V8 &held, const void *q, const float *q_smem, int i, float missing) -> V8 {
        if (kHeld) return held;
        if (MODE != kAnyRow && n.w_in_smem) return read_planes(q_smem, at.vec(i), VPT * T);
        return at.params(q, p.params_bf16, p.params_fast, i, missing);
    };
    const bool plain = p.y.fast && (p.y.bf16 != 0) == BF16;
    uint32_t phases = 0;  // of the stages' barriers
    bool dead = false, on = first < p.rows && (!p.mask || p.mask[first]);
    int s = 0, turn = 0;
    for (int64_t row = first; row < p.rows; row += step) {
        at.next_row();
        const bool on_next = !p.mask || row + step >= p.rows || p.mask[row + step];
        const int64_t row_more = row + S * step;  // takes this row's stage
        const bool more = t == 0 && row_more < p.rows && (!p.mask || p.mask[row_more]);
        V8 v[VPT];
        if (on) {
            if (!dead && !ptx::mbar_wait(full0 + s * 8, (phases >> s) & 1u, kNormWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
            const char *sx = stages + s * n.stage_bytes, *sr = sx + n.at_dy;
            const int x_shift = row_shift<MODE>(x_row(row)), r_shift = row_shift<MODE>(r_row(row));
            f32x2 s0[2] = {}, s1[2] = {};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                v[i] = zeros();
                if (at.none(i)) continue;
                v[i] = at.template read<BF16>(sx, x_shift, i);
                if (p.residual.p) v[i] = add_residual<BF16>(v[i], at.template read<BF16>(sr, r_shift, i));
                if (MODE != kAnyRow && i == VPT - 1 && at.cut) v[i] = at.cut_off(v[i], i);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (!FULL || p.rms)
                        s1[k & 1] = fma2(v[i].p[k], v[i].p[k], s1[k & 1]);
                    else
                        s0[k & 1] = add2(s0[k & 1], v[i].p[k]);
                }
            }
            float a = 0.f, b = !FULL || p.rms ? sum_of(s1) : sum_of(s0), mean = 0.f, rest = 0.f, var;
            team_sums<false, MODE == kWarpRow>(a, b, s_sums[turn], T >> 5);
            turn ^= 1;
            if (MODE == kWarpRow) __syncwarp();
            if (more && !dead) copy_row(row_more, s);
            if (p.h.p)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (!at.none(i)) at.store(p.h, row, i, v[i]);
            if (MODE != kAnyRow && p.ckpt.codes)
#pragma unroll
                for (int i = 0; i < VPT; ++i) store_act8(at, p.ckpt, row, i, v[i]);
            if (!FULL || p.rms) {
                var = b * p.inv_cols;
            } else {
                mean = b * p.inv_cols;
                const f32x2 nm = pack2(-mean, -mean);
                s0[0] = s0[1] = s1[0] = s1[1] = 0ull;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    if (at.none(i)) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i].p[k] = add2(v[i].p[k], nm);
                    if (i == VPT - 1 && at.cut) v[i] = at.cut_off(v[i], i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s0[k & 1] = add2(s0[k & 1], v[i].p[k]);
                        s1[k & 1] = fma2(v[i].p[k], v[i].p[k], s1[k & 1]);
                    }
                }
                a = sum_of(s0), b = sum_of(s1);
                team_sums<true, MODE == kWarpRow>(a, b, s_sums[turn], T >> 5);
                turn ^= 1;
                var = variance(a, b, p.inv_cols, rest);
                mean += rest;
            }
            const float rstd = finish_stats(p, row, t == 0, mean, var);
            char *y_row = static_cast<char *>(p.y.p) + row * p.y.ld * (BF16 ? 2 : 4);
            const f32x2 rs = pack2(rstd, rstd), off = pack2(-rest * rstd, -rest * rstd);  // (v - rest) rstd in one step
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (at.none(i)) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i].p[k] = FULL ? fma2(v[i].p[k], rs, off) : mul2(v[i].p[k], rs);
                const V8 w = param(w_held[kHeld ? i : 0], p.w, w_smem, i, 1.f);
                if (FULL) {
                    const V8 c = param(b_held[kHeld && FULL ? i : 0], p.b, b_smem, i, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i].p[k] = fma2(v[i].p[k], w.p[k], c.p[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i].p[k] = mul2(v[i].p[k], w.p[k]);
                }
                if (!starts_anywhere(MODE) && plain)
                    at.template store_plain<BF16>(y_row, p.y.fast, i, v[i]);
                else
                    at.store(p.y, row, i, v[i]);
            }
        } else {
            if (more && !dead) copy_row(row_more, s);
            if (t == 0) {
                if (p.mean) p.mean[row] = 0.f;
                if (p.rstd) p.rstd[row] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!at.none(i)) {
                    at.store(p.y, row, i, zeros());
                    if (p.h.p) at.store(p.h, row, i, zeros());
                }
                if (MODE != kAnyRow && p.ckpt.codes) store_act8(at, p.ckpt, row, i, zeros());
            }
        }
        on = on_next;
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead && t == 0)  // (copies in flight end before the block does, or do not within another wait)
        for (int k = 0; k < S; ++k) ptx::mbar_wait(full0 + k * 8, (phases >> k) & 1u, kNormWaitNs);
}

template <bool BF16, int VPT, bool FULL, int MODE>
cudaError_t launch_forward_rows(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream) {
    return run_kernel<norm_forward_kernel<BF16, VPT, FULL, MODE>>(n.blocks, MODE == kWarpRow ? kForwardWarps * 32 : n.warps * 32, n.smem, kNormRingSmem, stream, p, n);
}

template <bool BF16, bool FULL, int MODE>
cudaError_t launch_forward_vecs(const NormForwardParams &p, const NormTeams &n, cudaStream_t stream) {
    switch (n.vecs) {
        case 1: return launch_forward_rows<BF16, 1, FULL, MODE>(p, n, stream);
        case 2: return launch_forward_rows<BF16, 2, FULL, MODE>(p, n, stream);
        case 3: return launch_forward_rows<BF16, 3, FULL, MODE>(p, n, stream);
        default: return launch_forward_rows<BF16, 4, FULL, MODE>(p, n, stream);
    }
}

}  // namespace rlk

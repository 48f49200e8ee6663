// The backward pass of the norms with rows brought into shared memory by bulk copies (mathematics: norm.cuh).
//
// While a team of warps works on a row, the copies of its next rows are under way. The row is read twice from
// shared memory (the sums, then dx), so that a thread holds little more than its sums of dw and db in
// registers. A row's stage is filled again after the next row's exchange of sums, when every thread of the
// team has left it: no barrier but that exchange's (with room for one row only, one more after each row).
//
// A team is a block (kBlockRow: two or more on an SM cover each other's exchanges) or, for rows of 1024
// columns and less, one warp of a block of 16 (kWarpRow: no barriers, and one partial sum for 16 rows at a
// time); of rows that start anywhere a block takes each, in one of two ways (kShiftRow, kAnyRow: norm_rows.cuh).
//
// Bound by memory with one exchange a row (65536 x 6144 bf16, RMS with the residual's gradient: 471 us, 101% of the measured copy rate; from
// int8 427, 98%); reading e4m3 codes costs instructions (65536 x 5120 layer norm 519 us, 67%), rows of 8192
// columns leave a block alone on its SM with its exchange (164 us for 16384, 72%), and for the longest fp32 rows with a
// residual's gradient the weight has room neither in registers nor beside the ring (8192 x 16384 layer norm 468 us, 68%; RMS 341, 93%).
//
// FULL = false is the RMS form without db, in which mean = 0 and sum(u) is not needed.
#pragma once

#include "norm_rows.cuh"

namespace rlk {

enum HSource { kHBf16, kHF32, kHInt8, kHE4M3 };
constexpr bool from_act8(int src) { return src >= kHInt8; }
// A vector of h, or, from codes, of d = h - mean (FULL = false: h), which takes no more steps than h; `nm` is -mean twice.
template <int SRC, bool FULL>
__device__ __forceinline__ V8 read_h(const char *row, int vec, float scale, f32x2 nm) {
    if (!from_act8(SRC)) return read_vec<SRC == kHBf16>(row, vec);
    return act8_decode_plus<SRC == kHE4M3, FULL>(*reinterpret_cast<const uint2 *>(row + vec * 8), scale, nm);
}
template <int SRC, bool FULL>
__device__ __forceinline__ V8 read_h_shifted(const char *row, int shift, int vec, float scale, f32x2 nm) {
    if (!from_act8(SRC)) return read_shifted<SRC == kHBf16>(row, shift, vec);
    return act8_decode_plus<SRC == kHE4M3, FULL>(codes_shifted(row, shift, vec), scale, nm);
}
template <int SRC, bool FULL>
__device__ __forceinline__ f32x2 less_mean(f32x2 h, f32x2 nm) { return FULL && !from_act8(SRC) ? add2(h, nm) : h; }

template <int SRC, bool DYBF16, int VPT, bool FULL, int MODE>
__global__ void __launch_bounds__(kNormWarps * 32, 1) norm_backward_ring_kernel(NormBackwardParams p, NormTeams n) {
    constexpr bool kAct8 = from_act8(SRC), kWInRegs = MODE == kAnyRow ? VPT == 1 : VPT <= (MODE == kShiftRow ? 2 : 3) || !FULL;  // (else no room is left)
    constexpr int kTeams = MODE == kWarpRow ? kNormWarps : 1;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) float2 s_sums[2][16];
    __shared__ __align__(8) uint64_t s_full[kTeams * kNormDepth];
    const int T = MODE == kWarpRow ? 32 : (int)blockDim.x, team = MODE == kWarpRow ? (int)threadIdx.x >> 5 : 0;
    const int t = MODE == kWarpRow ? (int)threadIdx.x & 31 : (int)threadIdx.x, S = n.depth;
    Columns<MODE, VPT> at(t, T, p.cols);
    const bool plain = p.dx.fast;
    const bool x_bf16 = kAct8 ? p.dx.bf16 : SRC == kHBf16;
    char *stages = smem + team * S * n.stage_bytes;
    if (threadIdx.x < 32) (&s_sums[0][0])[threadIdx.x] = make_float2(0.f, 0.f);
    if (threadIdx.x == 0) {
        for (int k = 0; k < kTeams * S; ++k) ptx::mbar_init(ptx::smem_u32(&s_full[k]), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    grid_launch_dependents();
    const uint32_t full0 = ptx::smem_u32(&s_full[team * S]);

    const int64_t first = blockIdx.x + (int64_t)team * gridDim.x, step = (int64_t)kTeams * gridDim.x;
    const auto h_row = [&](int64_t row) -> const char * {
        return kAct8 ? reinterpret_cast<const char *>(p.ckpt.codes) + row * p.ckpt.ld_codes : static_cast<const char *>(p.x.p) + row * p.x.ld * (SRC == kHBf16 ? 2 : 4);
    };
    const auto dy_row = [&](int64_t row) -> const char * { return static_cast<const char *>(p.dy.p) + row * p.dy.ld * (DYBF16 ? 2 : 4); };
    const auto ds_row = [&](int64_t row) -> const char * { return static_cast<const char *>(p.dsummed.p) + row * p.dsummed.ld * (x_bf16 ? 2 : 4); };
    const auto copy_row = [&](int64_t row, int s) {  // by the team's thread 0
        char *stage = stages + s * n.stage_bytes;
        const uint32_t full = full0 + s * 8, to = ptx::smem_u32(stage);
        if (!starts_anywhere(MODE)) {
            ptx::mbar_arrive_expect_tx(full, (uint32_t)(n.copy_bytes[0] + n.copy_bytes[1] + n.copy_bytes[2]));
            ptx::bulk_g2s(to, h_row(row), (uint32_t)n.copy_bytes[0], full);
            ptx::bulk_g2s(to + n.at_dy, dy_row(row), (uint32_t)n.copy_bytes[1], full);
            if (p.dsummed.p) ptx::bulk_g2s(to + n.at_ds, ds_row(row), (uint32_t)n.copy_bytes[2], full);
            return;
        }
        const uint32_t bytes[3] = {window(h_row(row), p.cols * (kAct8 ? 1 : SRC == kHBf16 ? 2 : 4)), window(dy_row(row), p.cols * (DYBF16 ? 2 : 4)),
                                   p.dsummed.p ? window(ds_row(row), p.cols * (x_bf16 ? 2 : 4)) : 0u};
        ptx::mbar_arrive_expect_tx(full, bytes[0] + bytes[1] + bytes[2]);
        ptx::bulk_g2s(to, h_row(row) - row_shift<MODE>(h_row(row)), bytes[0], full);
        ptx::bulk_g2s(to + n.at_dy, dy_row(row) - row_shift<MODE>(dy_row(row)), bytes[1], full);
        if (p.dsummed.p) ptx::bulk_g2s(to + n.at_ds, ds_row(row) - row_shift<MODE>(ds_row(row)), bytes[2], full);
    };
    if (t == 0)
        for (int s = 0; s < S; ++s) {
            const int64_t row = first + s * step;
            if (row < p.rows && (!p.mask || p.mask[row])) copy_row(row, s);
        }

    float *w_smem = reinterpret_cast<float *>(smem + kTeams * S * n.stage_bytes);  // [VPT T 8], a thread reads its own
    V8 w[kWInRegs ? VPT : 1], dw[VPT], db[FULL ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const V8 v = at.none(i) ? zeros() : at.params(p.w, p.params_bf16, p.params_fast, i, 1.f);
        if (kWInRegs) {
            w[i] = v;
        } else if (n.w_in_smem) {
            write_planes(w_smem, at.vec(i), VPT * T, v);
        }
        dw[i] = zeros();
        if (FULL) db[i] = zeros();
    }
    const auto weight = [&](int i) -> V8 {
        if constexpr (kWInRegs) return w[i];
        if (!n.w_in_smem) return at.params(p.w, p.params_bf16, p.params_fast, i, 1.f);
        return read_planes(w_smem, at.vec(i), VPT * T);
    };

    // of the row at hand, loaded a row ahead
    constexpr int kScales = kAct8 ? VPT : 1;
    bool dead = false, on = true;
    float mean = 0.f, rstd = 0.f;
    float scale[kScales];
    uint32_t scale_first[kScales] = {};
    const auto row_data = [&](int64_t row, bool &o, float &m, float &r, uint32_t (&sc)[kScales]) {
        if (row >= p.rows) return;
        o = !p.mask || p.mask[row];
        r = p.rstd[row];
        if (FULL && !p.rms) m = p.mean[row];
        if (kAct8) {
            const uint8_t *q = p.ckpt.scales + row * p.ckpt.ld_scales;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (!at.none(i)) sc[i] = q[at.vec(i) >> 2];
        }
    };
    row_data(first, on, mean, rstd, scale_first);
#pragma unroll
    for (int i = 0; i < kScales; ++i) scale[i] = act8_factor(scale_first[i]);
    uint32_t phases = 0;  // of the stages' barriers
    int s = 0, last = 0, turn = 0;
    for (int64_t row = first; row < p.rows; row += step) {
        at.next_row();
        bool on_next = true;
        float mean_next = 0.f, rstd_next = 0.f;
        uint32_t scale_next[kScales] = {};
        row_data(row + step, on_next, mean_next, rstd_next, scale_next);
        const int64_t row_more = row + (S - 1) * step;  // takes the last row's stage (the only stage: the next row takes it)
        const bool more = t == 0 && S > 1 && row != first && row_more < p.rows && (!p.mask || p.mask[row_more]);

        const char *stage = stages + s * n.stage_bytes, *sh = stage, *sdy = stage + n.at_dy, *sds = stage + n.at_ds;
        const int h_shift = row_shift<MODE>(h_row(row)), dy_shift = row_shift<MODE>(dy_row(row)), ds_shift = row_shift<MODE>(ds_row(row));
        const f32x2 nm = pack2(-mean, -mean), rs = pack2(rstd, rstd);
        const auto get_h = [&](int i) -> V8 {
            if constexpr (MODE == kAnyRow) return at.template read<SRC == kHBf16>(sh, h_shift, i);  // (no codes)
            if constexpr (MODE == kShiftRow) return read_h_shifted<SRC, FULL>(sh, h_shift, at.vec(i), scale[kScales > 1 ? i : 0], nm);
            return read_h<SRC, FULL>(sh, at.vec(i), scale[kScales > 1 ? i : 0], nm);
        };
        float c1 = 0.f, c2 = 0.f;
        if (on) {
            if (!dead && !ptx::mbar_wait(full0 + s * 8, (phases >> s) & 1u, kNormWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
            f32x2 s0[2] = {}, s1[2] = {};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (at.none(i)) continue;
                V8 h = get_h(i), g = at.template read<DYBF16>(sdy, dy_shift, i);
                if (MODE != kAnyRow && i == VPT - 1 && at.cut) h = at.cut_off(h, i), g = at.cut_off(g, i);
                const V8 ww = weight(i);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 d = less_mean<SRC, FULL>(h.p[k], nm), r = mul2(g.p[k], rs), u = mul2(r, ww.p[k]);
                    dw[i].p[k] = fma2(r, d, dw[i].p[k]);
                    if (FULL) {
                        db[i].p[k] = add2(db[i].p[k], g.p[k]);
                        s0[k & 1] = add2(s0[k & 1], u);
                    }
                    s1[k & 1] = fma2(u, d, s1[k & 1]);
                }
            }
            c1 = sum_of(s0), c2 = sum_of(s1);
            team_sums<FULL, MODE == kWarpRow>(c1, c2, s_sums[turn], T >> 5);
            turn ^= 1;
            if (t == 0 && p.status && !(fabsf(c1) < INFINITY && fabsf(c2) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
            c1 = FULL && !p.rms ? c1 * p.inv_cols : 0.f;
            c2 = c2 * p.inv_cols * rstd * rstd;
        } else if (MODE != kWarpRow) {
            __syncthreads();
        }
        if (MODE == kWarpRow) __syncwarp();
        if (more && !dead) copy_row(row_more, last);
        const f32x2 o1 = pack2(-c1, -c1), nk = pack2(-c2, -c2);
        char *dx_row = static_cast<char *>(p.dx.p) + row * p.dx.ld * (x_bf16 ? 2 : 4);
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (at.none(i)) continue;
                const V8 h = get_h(i), g = at.template read<DYBF16>(sdy, dy_shift, i), ww = weight(i);
                V8 r;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 rr = mul2(g.p[k], rs), u = FULL ? fma2(rr, ww.p[k], o1) : mul2(rr, ww.p[k]);
                    r.p[k] = fma2(less_mean<SRC, FULL>(h.p[k], nm), nk, u);
                }
                if (p.dsummed.p) {
                    const V8 d = x_bf16 ? at.template read<true>(sds, ds_shift, i) : at.template read<false>(sds, ds_shift, i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r.p[k] = add2(r.p[k], d.p[k]);
                }
                if (p.y.p) {
                    V8 u = at.params(p.b, p.params_bf16, p.params_fast, i, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) u.p[k] = fma2(mul2(less_mean<SRC, FULL>(h.p[k], nm), rs), ww.p[k], u.p[k]);
                    at.store(p.y, row, i, u);
                }
                if (starts_anywhere(MODE) || !plain)
                    at.store(p.dx, row, i, r);
                else if (x_bf16)
                    at.template store_plain<true>(dx_row, 1, i, r);
                else
                    at.template store_plain<false>(dx_row, p.dx.fast, i, r);
            }
        } else {
            for (int i = 0; i < VPT; ++i) {
                if (at.none(i)) continue;
                at.store(p.dx, row, i, zeros());
                if (p.y.p) at.store(p.y, row, i, zeros());
            }
        }
        if (S == 1) {
            if (MODE == kWarpRow) __syncwarp(); else __syncthreads();
            if (t == 0 && row + step < p.rows && on_next && !dead) copy_row(row + step, 0);
        }
        on = on_next, mean = mean_next, rstd = rstd_next;
#pragma unroll
        for (int i = 0; i < kScales; ++i) scale[i] = act8_factor(scale_next[i]);
        last = s;
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead && t == 0)  // (copies in flight end before the block does, or do not within another wait)
        for (int k = 0; k < S; ++k) ptx::mbar_wait(full0 + k * 8, (phases >> k) & 1u, kNormWaitNs);
    if (!p.want_dw && !p.want_db) return;

    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part;
    if (MODE != kWarpRow) {
        const RowMat out{part, p.ld_part, 0, 1};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (at.none(i)) continue;
            at.store(out, 0, i, dw[i]);
            if (FULL) at.store(out, 1, i, db[i]);
        }
        return;
    }
    // the warps' sums, over the rows' room
    float *sums = reinterpret_cast<float *>(smem);
    constexpr int kWidth = VPT * 32 * kVec;
#pragma unroll
    for (int which = 0; which < (FULL ? 2 : 1); ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float v[kVec];
            floats_of(which ? db[FULL ? i : 0] : dw[i], v);
            store_vec(sums + team * kWidth, at.vec(i) * kVec, kWidth, true, v);
        }
        __syncthreads();
        join_teams(sums, kTeams, kWidth, p.cols, part + which * p.ld_part);
    }
}

template <int SRC, bool DYBF16, int VPT, bool FULL, int MODE>
cudaError_t launch_norm_ring(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream) {
    return run_kernel<norm_backward_ring_kernel<SRC, DYBF16, VPT, FULL, MODE>>(blocks, MODE == kWarpRow ? kNormWarps * 32 : n.warps * 32, n.smem, kNormRingSmem, stream, p, n);
}

template <int SRC, bool DYBF16>
cudaError_t launch_norm_rows(const NormBackwardParams &p, const NormTeams &n, int blocks, cudaStream_t stream) {
#define RLK_RING(V, FULL, MODE) launch_norm_ring<SRC, DYBF16, V, FULL, MODE>(p, n, blocks, stream)
    constexpr int kAnywhere = from_act8(SRC) ? kShiftRow : kAnyRow;
    if (starts_anywhere(n.mode)) {
        switch (n.vecs) {
            case 1: return RLK_RING(1, true, kAnywhere);
            case 2: return RLK_RING(2, true, kAnywhere);
            case 3: return RLK_RING(3, true, kAnywhere);
            default: return RLK_RING(4, true, kAnywhere);
        }
    }
    if constexpr (SRC != kHBf16 || DYBF16) {
        const bool full = !p.rms || p.want_db;
        if (n.mode == kWarpRow) return full ? RLK_RING(3, true, kWarpRow) : n.vecs == 3 ? RLK_RING(3, false, kWarpRow) : RLK_RING(4, false, kWarpRow);
        switch (n.vecs) {
            case 1: return full ? RLK_RING(1, true, kBlockRow) : RLK_RING(1, false, kBlockRow);
            case 2: return full ? RLK_RING(2, true, kBlockRow) : RLK_RING(2, false, kBlockRow);
            case 3: return full ? RLK_RING(3, true, kBlockRow) : RLK_RING(3, false, kBlockRow);
            default: return full ? RLK_RING(4, true, kBlockRow) : RLK_RING(4, false, kBlockRow);
        }
    }
#undef RLK_RING
    return cudaErrorInvalidValue;
}

}  // namespace rlk

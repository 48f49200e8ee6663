// The backward pass of the norms (mathematics: norm.cuh): the kernel for short rows, the sum of the blocks' partial sums, and
// which kernel takes a call (those of longer rows and of rows that start anywhere: norm_ring.cuh).
#include <algorithm>

#include "norm_ring.cuh"
#include "norm_short.cuh"

namespace rlk {

namespace {

constexpr int kThreads = kNormWarps * 32;
constexpr int kJoin = 32;  // columns and warps of a block that adds partial sums

// ---------------------------------------------------------------- short rows (norm_short.cuh)

// EXACT: the threads' vectors are the row's columns to the last one, no mask and no output made again.
template <int SRC, bool DYBF16, int VPT, bool FULL, bool EXACT>
__global__ void __launch_bounds__(kThreads, 1) norm_backward_short_kernel(NormBackwardParams p, NormShort n) {
    constexpr bool kAct8 = from_act8(SRC);
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(8) uint64_t s_full[kNormWarps * kNormDepth];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = n.lanes, t = lane & (lanes - 1), slot = lane / lanes, S = n.depth;
    const int width = lanes * VPT * kVec;
    const bool x_bf16 = kAct8 ? p.dx.bf16 : SRC == kHBf16;
    float *w_smem = reinterpret_cast<float *>(smem + n.smem) - width;
    for (int c = threadIdx.x; c < width; c += kThreads) w_smem[plane_of(c, width / kVec)] = c < p.cols ? (p.w ? load_param(p.w, p.params_bf16, c) : 1.f) : 0.f;
    if (threadIdx.x == 0) {
        for (int k = 0; k < kNormWarps * S; ++k) ptx::mbar_init(ptx::smem_u32(&s_full[k]), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    grid_launch_dependents();
    ShortRing ring(n);
    ring.mask = p.mask;
    ring.base[0] = kAct8 ? reinterpret_cast<const char *>(p.ckpt.codes) : static_cast<const char *>(p.x.p);
    ring.pitch[0] = kAct8 ? p.ckpt.ld_codes : p.x.ld * (SRC == kHBf16 ? 2 : 4);
    ring.base[1] = static_cast<const char *>(p.dy.p);
    ring.pitch[1] = p.dy.ld * (DYBF16 ? 2 : 4);
    ring.base[2] = static_cast<const char *>(p.dsummed.p);
    ring.pitch[2] = p.dsummed.ld * (x_bf16 ? 2 : 4);
    ring.rows = p.rows;
    char *stages = smem + warp * S * n.stage_bytes;
    ring.stages = ptx::smem_u32(stages);
    ring.full = ptx::smem_u32(&s_full[warp * S]);
    ring.lane = lane;
    ring.per = 32 / lanes;
    const int64_t first = blockIdx.x + (int64_t)warp * gridDim.x, step = (int64_t)gridDim.x * kNormWarps;
    const int64_t batches = ((int64_t)p.rows + ring.per - 1) / ring.per;
    for (int s = 0; s < S; ++s)
        if (first + s * step < batches) ring.fetch(first + s * step, s);

    V8 dw[VPT], db[FULL ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        dw[i] = zeros();
        if (FULL) db[i] = zeros();
    }
    constexpr int kScales = kAct8 ? VPT : 1;
    bool dead = false, mine = false, on = false;  // of the thread's row, loaded a batch ahead
    float mean = 0.f, rstd = 0.f;
    uint32_t scale[kScales];
    const auto row_data = [&](int64_t batch, bool &m, bool &o, float &mu, float &r, uint32_t (&sc)[kScales]) {
        const int64_t row = batch * ring.per + slot;
        m = row < p.rows;
        o = m && (EXACT || !p.mask || p.mask[row]);
        mu = r = 0.f;
        if (!o) return;
        r = p.rstd[row];
        if (FULL && !p.rms) mu = p.mean[row];
        if (kAct8)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes;
                sc[kAct8 ? i : 0] = vec * kVec < p.cols ? p.ckpt.scales[row * p.ckpt.ld_scales + (vec >> 2)] : 0;
            }
    };
    if (first < batches) row_data(first, mine, on, mean, rstd, scale);
    uint32_t phases = 0;
    int s = 0;
    for (int64_t batch = first; batch < batches; batch += step) {
        bool mine_next = false, on_next = false;
        float mean_next = 0.f, rstd_next = 0.f;
        uint32_t scale_next[kScales] = {};
        if (batch + step < batches) row_data(batch + step, mine_next, on_next, mean_next, rstd_next, scale_next);
        const int64_t row = batch * ring.per + slot;
        if (kAct8)
#pragma unroll
            for (int i = 0; i < kScales; ++i) scale[i] = __float_as_uint(act8_factor(scale[i]));  // the factors
        if (__any_sync(0xffffffffu, on)) {
            if (!dead && !ptx::mbar_wait(ring.full + s * 8, (phases >> s) & 1u, kNormWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
        }
        const char *sh = stages + s * n.stage_bytes + n.at[0] + slot * n.row_bytes[0], *sdy = stages + s * n.stage_bytes + n.at[1] + slot * n.row_bytes[1];
        const char *sds = stages + s * n.stage_bytes + n.at[2] + slot * n.row_bytes[2];
        const f32x2 nm = pack2(-mean, -mean), rs = pack2(rstd, rstd);
        f32x2 s0[2] = {}, s1[2] = {};
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                if (!EXACT && col >= p.cols) continue;
                V8 h = read_h<SRC, FULL>(sh, vec, __uint_as_float(scale[kAct8 ? i : 0]), nm), g = read_vec<DYBF16>(sdy, vec);
                if (!EXACT && col + kVec > p.cols) h = clipped(h, col, p.cols), g = clipped(g, col, p.cols);
                const V8 w = read_planes(w_smem, vec, width / kVec);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 d = less_mean<SRC, FULL>(h.p[k], nm), r = mul2(g.p[k], rs), u = mul2(r, w.p[k]);
                    dw[i].p[k] = fma2(r, d, dw[i].p[k]);
                    if (FULL) {
                        db[i].p[k] = add2(db[i].p[k], g.p[k]);
                        s0[k & 1] = add2(s0[k & 1], u);
                    }
                    s1[k & 1] = fma2(u, d, s1[k & 1]);
                }
            }
        }
        float c1 = sum_of(s0), c2 = sum_of(s1);
        for (int off = lanes >> 1; off > 0; off >>= 1) {
            if (FULL) c1 = __fadd_rn(c1, __shfl_xor_sync(0xffffffffu, c1, off));
            c2 = __fadd_rn(c2, __shfl_xor_sync(0xffffffffu, c2, off));
        }
        if (t == 0 && p.status && !(fabsf(c1) < INFINITY && fabsf(c2) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
        c1 = FULL && !p.rms ? c1 * p.inv_cols : 0.f;
        c2 = c2 * p.inv_cols * rstd * rstd;
        const f32x2 o1 = pack2(-c1, -c1), nk = pack2(-c2, -c2);
        if (kAct8)
#pragma unroll
            for (int i = 0; i < kScales; ++i) asm volatile("" : "+r"(scale[i]));  // (pairs of it made again, not kept: registers)
        if (on) {
            const int64_t out = row * p.dx.ld;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                if (!EXACT && col >= p.cols) continue;
                const V8 h = read_h<SRC, FULL>(sh, vec, __uint_as_float(scale[kAct8 ? i : 0]), nm), g = read_vec<DYBF16>(sdy, vec), w = read_planes(w_smem, vec, width / kVec);
                V8 r;
                float o[kVec];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 rr = mul2(g.p[k], rs), u = FULL ? fma2(rr, w.p[k], o1) : mul2(rr, w.p[k]);
                    r.p[k] = fma2(less_mean<SRC, FULL>(h.p[k], nm), nk, u);
                }
                if (p.dsummed.p) {
                    const V8 q = x_bf16 ? read_vec<true>(sds, vec) : read_vec<false>(sds, vec);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r.p[k] = add2(r.p[k], q.p[k]);
                }
                if (!EXACT && p.y.p) {
                    float b[kVec] = {};
                    if (p.b) load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, b);
                    V8 v = pairs_of(b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v.p[k] = fma2(mul2(less_mean<SRC, FULL>(h.p[k], nm), rs), w.p[k], v.p[k]);
                    floats_of(v, o);
                    store_row(p.y, row, col, p.cols, o);
                }
                floats_of(r, o);
                const int end = EXACT ? col + kVec : p.cols;  // (EXACT: no part of a vector)
                if (x_bf16)
                    store_vec(static_cast<__nv_bfloat16 *>(p.dx.p) + out, col, end, EXACT || p.dx.fast, o);
                else if (p.dx.fast == 2 && col + kVec <= end)
                    store_vec32(static_cast<float *>(p.dx.p) + out, col, o);
                else
                    store_vec(static_cast<float *>(p.dx.p) + out, col, end, EXACT || p.dx.fast, o);
            }
        } else if (!EXACT && mine) {
            const float o[kVec] = {};
            for (int vec = t; vec * kVec < p.cols; vec += lanes) {
                store_row(p.dx, row, vec * kVec, p.cols, o);
                if (p.y.p) store_row(p.y, row, vec * kVec, p.cols, o);
            }
        }
        __syncwarp();
        if (batch + S * step < batches && !__any_sync(0xffffffffu, dead)) ring.fetch(batch + S * step, s);
        mine = mine_next, on = on_next, mean = mean_next, rstd = rstd_next;
#pragma unroll
        for (int i = 0; i < kScales; ++i) scale[i] = scale_next[i];
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead && lane == 0)  // (copies in flight end before the block does, or do not within another wait)
        for (int k = 0; k < S; ++k) ptx::mbar_wait(ring.full + k * 8, (phases >> k) & 1u, kNormWaitNs);
    if (!p.want_dw && !p.want_db) return;
    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part, *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int which = 0; which < (FULL ? 2 : 1); ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float v[kVec];
            floats_of(which ? db[FULL ? i : 0] : dw[i], v);
            for (int off = lanes; off < 32; off <<= 1)  // the warp's rows
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], __shfl_xor_sync(0xffffffffu, v[j], off));
            if (lane < lanes) store_vec(sums + warp * width, (t + i * lanes) * kVec, width, true, v);
        }
        __syncthreads();
        join_teams(sums, kNormWarps, width, p.cols, part + which * p.ld_part);
    }
}

// ---------------------------------------------------------------- the sum of the partial sums

// A block adds 32 columns' partial sums: warp k takes every 32nd one, a lane a column, ten loads under way at a time;
// then warp c adds column c's 32 sums by a butterfly. (Eight warps, each thread a long chain of loads: 4096 x 6144 41.8 us,
// against 41.2.)
// The launch begins while the blocks before it still work, and waits for them.
__global__ void __launch_bounds__(kJoin * kJoin) norm_join_kernel(const float *partials, int64_t ld, int parts, int cols, float *dw, float *db, int accumulate) {
    __shared__ float s[kJoin][kJoin + 1];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * kJoin + lane;
    const int which = dw ? (int)blockIdx.y : 1;
    float *out = which ? db : dw;
    grid_dependency_wait();
    float v = 0.f;
    if (c < cols) {
        const float *q = partials + which * ld + c;
#pragma unroll 10
        for (int i = k; i < parts; i += kJoin) v += q[(int64_t)i * 2 * ld];
    }
    s[k][lane] = v;
    __syncthreads();
    v = s[lane][k];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    const int mine = blockIdx.x * kJoin + k;
    if (lane == 0 && mine < cols) out[mine] = accumulate ? out[mine] + v : v;
}

cudaError_t launch_join(const NormBackwardParams &p, int parts, cudaStream_t stream) {
    if (!p.want_dw && !p.want_db) return cudaSuccess;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.cols + kJoin - 1) / kJoin, p.want_dw && p.want_db ? 2 : 1);
    cfg.blockDim = dim3(kJoin * kJoin);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_join_kernel, (const float *)p.partials, p.ld_part, parts, (int)p.cols,
                              p.want_dw ? p.dw : nullptr, p.want_db ? p.db : nullptr, (int)p.accumulate);
}

// ---------------------------------------------------------------- which kernel

template <int SRC, bool DYBF16>
cudaError_t launch_short(const NormBackwardParams &p, int blocks, cudaStream_t stream) {
    const int es[3] = {from_act8(SRC) ? 1 : SRC == kHBf16 ? 2 : 4, DYBF16 ? 2 : 4, !p.dsummed.p ? 0 : p.dx.bf16 ? 2 : 4};
    const int64_t ld[3] = {from_act8(SRC) ? p.ckpt.ld_codes : p.x.ld, p.dy.ld, p.dsummed.ld};
    const int width = norm_short_width(p.cols);
    const NormShort n = norm_short(p.cols, es, ld, 3, p.mask != nullptr, kNormWarps, (size_t)width * 4, (size_t)kNormWarps * width * 4);
    const bool full = !p.rms || p.want_db;
    const bool exact = p.cols == width && !p.mask && !p.y.p && p.dx.fast;
#define RLK_RUN(V, F, E) run_kernel<norm_backward_short_kernel<SRC, DYBF16, V, F, E>>(blocks, kThreads, n.smem, kNormRingSmem, stream, p, n)
#define RLK_SHORT(V, F) (exact ? RLK_RUN(V, F, true) : RLK_RUN(V, F, false))
    return n.vecs == 2 ? full ? RLK_SHORT(2, true) : RLK_SHORT(2, false) : full ? RLK_SHORT(4, true) : RLK_SHORT(4, false);
#undef RLK_SHORT
#undef RLK_RUN
}

}  // namespace

cudaError_t launch_norm_backward(const NormBackwardParams &p, cudaStream_t stream) {
    const bool act8 = !p.x.p;
    const bool fast = p.dy.fast && (act8 ? p.ckpt.fast : p.x.fast) && (!p.dsummed.p || p.dsummed.fast) && p.dx.fast && (!p.y.p || p.y.fast);
    cudaError_t e = cudaErrorUnknown;
    int blocks;
    if (fast && p.cols <= kShortCols) {
        blocks = std::min(p.rows, kNormSMs);
#define RLK_SHORT(SRC) (p.dy.bf16 ? launch_short<SRC, true>(p, blocks, stream) : launch_short<SRC, false>(p, blocks, stream))
        e = act8 ? p.ckpt.e4m3 ? RLK_SHORT(kHE4M3) : RLK_SHORT(kHInt8) : p.x.bf16 ? RLK_SHORT(kHBf16) : RLK_SHORT(kHF32);
#undef RLK_SHORT
    } else {
        const int es[3] = {act8 ? 1 : p.x.bf16 ? 2 : 4, p.dy.bf16 ? 2 : 4, !p.dsummed.p ? 0 : p.dx.bf16 ? 2 : 4};
        const NormBackwardShape shape{p.rows, p.cols, es[0], es[1], es[2], p.rms != 0, p.want_db != 0};
        const NormTeams n = norm_backward_teams(shape, norm_backward_mode(shape, fast));
        blocks = norm_backward_blocks(shape, n);
#define RLK_ROWS(H) (p.dy.bf16 ? launch_norm_rows_##H##_bf16(p, n, blocks, stream) : launch_norm_rows_##H##_f32(p, n, blocks, stream))
        e = act8 ? p.ckpt.e4m3 ? RLK_ROWS(e4m3) : RLK_ROWS(int8) : p.x.bf16 ? RLK_ROWS(bf16) : RLK_ROWS(f32);
#undef RLK_ROWS
    }
    return e == cudaSuccess ? launch_join(p, blocks, stream) : e;
}

}  // namespace rlk

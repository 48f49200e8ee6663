// The backward pass of the norms (mathematics: norm.cuh): the kernels for short rows and for rows that start
// anywhere, the sum of the blocks' partial sums, and which kernel takes a call.
#include <algorithm>

#include "norm.cuh"
#include "norm_ring.cuh"

namespace rlk {

namespace {

constexpr int kThreads = kNormWarps * 32;
constexpr int kJoinCols = 32, kJoinRows = 8;

// ---------------------------------------------------------------- short rows
//
// Rows on 16-byte boundaries that fit `lanes` threads of a warp (4 to 32) with VPT vectors each, so that a warp
// works on several rows and a row's sums take few steps; rows are held in registers from one load to the store.

template <int SRC, bool XBF16, bool DYBF16, int VPT, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) norm_backward_short_kernel(NormBackwardParams p, int lanes) {
    extern __shared__ __align__(16) float smem_short[];
    float *w_smem = smem_short;  // [lanes VPT 8]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & (lanes - 1), per_warp = 32 / lanes;
    const int width = lanes * VPT * kVec;
    for (int c = threadIdx.x; c < width; c += kThreads) w_smem[c] = c < p.cols ? (p.w ? load_param(p.w, p.params_bf16, c) : 1.f) : 0.f;
    __syncthreads();
    V8 dw[VPT], db[FULL ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        dw[i] = zeros();
        if (FULL) db[i] = zeros();
    }
    const int64_t step = (int64_t)gridDim.x * kNormWarps * per_warp;
    for (int64_t base = (blockIdx.x + (int64_t)warp * gridDim.x) * per_warp; base < p.rows; base += step) {
        const int64_t row = base + lane / lanes;
        const bool mine = row < p.rows, on = mine && (!p.mask || p.mask[row]);
        typename RawMat<DYBF16>::type dy[VPT];
        typename RawMat<XBF16>::type hx[VPT], ds[VPT];
        Raw8 h8[VPT];
        uint32_t scale[VPT];
        float mean = 0.f, rstd = 0.f;
        if (on) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int vec = t + i * lanes, col = vec * kVec;
                if (col < p.cols) {
                    if (from_act8(SRC)) {
                        load_raw(h8[i], p.ckpt.codes + row * p.ckpt.ld_codes, col, p.cols, true);
                        scale[i] = p.ckpt.scales[row * p.ckpt.ld_scales + (vec >> 2)];
                    } else {
                        load_mat<XBF16>(hx[i], p.x, row, col, p.cols);
                    }
                    load_mat<DYBF16>(dy[i], p.dy, row, col, p.cols);
                    if (p.dsummed.p) load_mat<XBF16>(ds[i], p.dsummed, row, col, p.cols);
                }
            }
            rstd = p.rstd[row];
            if (FULL && !p.rms) mean = p.mean[row];
        }
        const f32x2 nm = pack2(-mean, -mean), rs = pack2(rstd, rstd);
        const auto get_h = [&](int i) -> V8 {
            if constexpr (from_act8(SRC))
                return act8_decode_norm<SRC == kHE4M3>(h8[i].a, scale[i]);
            else
                return pairs(hx[i]);
        };
        f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (!on || col >= p.cols) continue;
            V8 g = pairs(dy[i]), h = get_h(i);
            if (col + kVec > p.cols) h = clipped(h, col, p.cols), g = clipped(g, col, p.cols);
            const V8 w = read_vec<false>(reinterpret_cast<const char *>(w_smem), t + i * lanes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 d = FULL ? add2(h.p[k], nm) : h.p[k], r = mul2(g.p[k], rs), u = mul2(r, w.p[k]);
                dw[i].p[k] = fma2(r, d, dw[i].p[k]);
                if (FULL) {
                    db[i].p[k] = add2(db[i].p[k], g.p[k]);
                    s0 = add2(s0, u);
                }
                s1 = fma2(u, d, s1);
            }
        }
        float c1 = sum_of(s0), c2 = sum_of(s1);
        for (int off = lanes >> 1; off > 0; off >>= 1) {
            if (FULL) c1 = __fadd_rn(c1, __shfl_xor_sync(0xffffffffu, c1, off));
            c2 = __fadd_rn(c2, __shfl_xor_sync(0xffffffffu, c2, off));
        }
        if (!mine) continue;
        if (t == 0 && p.status && !(fabsf(c1) < INFINITY && fabsf(c2) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
        c1 = FULL && !p.rms ? c1 * p.inv_cols : 0.f;
        c2 = c2 * p.inv_cols * rstd * rstd;
        const f32x2 o1 = pack2(-c1, -c1), nk = pack2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * lanes) * kVec;
            if (col >= p.cols) continue;
            float o[kVec] = {};
            if (on) {
                const V8 g = pairs(dy[i]), h = get_h(i), w = read_vec<false>(reinterpret_cast<const char *>(w_smem), t + i * lanes);
                V8 r;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 rr = mul2(g.p[k], rs), u = FULL ? fma2(rr, w.p[k], o1) : mul2(rr, w.p[k]);
                    r.p[k] = fma2(FULL ? add2(h.p[k], nm) : h.p[k], nk, u);
                }
                if (p.dsummed.p) {
                    const V8 q = pairs(ds[i]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r.p[k] = add2(r.p[k], q.p[k]);
                }
                if (p.y.p) {
                    float b[kVec] = {};
                    if (p.b) load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, b);
                    V8 v = pairs_of(b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v.p[k] = fma2(mul2(add2(h.p[k], nm), rs), w.p[k], v.p[k]);
                    floats_of(v, o);
                    store_row(p.y, row, col, p.cols, o);
                }
                floats_of(r, o);
            } else if (p.y.p) {
                store_row(p.y, row, col, p.cols, o);
            }
            if (XBF16)
                store_vec(static_cast<__nv_bfloat16 *>(p.dx.p) + row * p.dx.ld, col, p.cols, p.dx.fast, o);
            else
                store_vec(static_cast<float *>(p.dx.p) + row * p.dx.ld, col, p.cols, p.dx.fast, o);
        }
    }
    if (!p.want_dw && !p.want_db) return;
    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part;
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
            if (lane < lanes) store_vec(smem_short + warp * width, (t + i * lanes) * kVec, width, true, v);
        }
        __syncthreads();
        join_teams(smem_short, kNormWarps, width, p.cols, part + which * p.ld_part);
    }
}

// ---------------------------------------------------------------- the sum of the partial sums

// Eight threads take every eighth partial sum of a column, their sums are added in turn.
__global__ void __launch_bounds__(kJoinCols * kJoinRows) norm_join_kernel(const float *partials, int64_t ld, int parts, int cols, float *dw, float *db, int accumulate) {
    __shared__ float s[kJoinRows][kJoinCols];
    const int c = blockIdx.x * kJoinCols + threadIdx.x, k = threadIdx.y;
    const int which = dw ? (int)blockIdx.y : 1;
    float *out = which ? db : dw;
    grid_dependency_wait();
    float v = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int i = k; i < parts; i += kJoinRows) v += partials[((int64_t)i * 2 + which) * ld + c];
    }
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
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.cols + kJoinCols - 1) / kJoinCols, p.want_dw && p.want_db ? 2 : 1);
    cfg.blockDim = dim3(kJoinCols, kJoinRows);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_join_kernel, (const float *)p.partials, p.ld_part, parts, (int)p.cols,
                              p.want_dw ? p.dw : nullptr, p.want_db ? p.db : nullptr, (int)p.accumulate);
}

// ---------------------------------------------------------------- which kernel

int vectors(int cols) { return (cols + kVec - 1) / kVec; }

// Four vectors a thread where registers hold them (16-bit rows, one sum), two otherwise.
template <int SRC, bool XBF16, bool DYBF16, bool FULL>
cudaError_t launch_short(const NormBackwardParams &p, int blocks, cudaStream_t stream) {
    constexpr int kVecs = DYBF16 && XBF16 && !FULL ? 4 : 2;
    int lanes = 4;
    while (lanes * kVecs * kVec < p.cols) lanes *= 2;
    const size_t smem = (size_t)kNormWarps * lanes * kVecs * kVec * sizeof(float);  // (the sums; the weight before them)
    norm_backward_short_kernel<SRC, XBF16, DYBF16, kVecs, FULL><<<blocks, kThreads, smem, stream>>>(p, lanes);
    return cudaGetLastError();
}

constexpr int kShortCols = 512;  // at most a warp of two vectors, 32 KB of sums

constexpr size_t kSmemOfSM = 228 * 1024, kBlockExtra = 1024 + 512;  // what a block takes beside its rows

// A block per row, 128 registers a thread, so 16 warps on an SM: of the numbers of vectors a thread, the one whose
// blocks take all rows soonest, by a row's time of its vectors and two more for the exchange of sums. Both sums with
// four vectors a thread (rows that start anywhere: with three) do not fit the registers, and are taken for the
// longest rows alone.
NormTeams teams_of(const NormBackwardParams &p, int mode) {
    const bool act8 = !p.x.p, full = !p.rms || p.want_db || mode == kAnyRow;
    const int vecs = vectors(p.cols), pad = mode == kAnyRow ? 16 : 0;
    const auto bytes = [&](int es) { return (p.cols * es + 15) / 16 * 16 + pad; };
    NormTeams n{};
    n.mode = mode;
    n.at_dy = bytes(act8 ? 1 : p.x.bf16 ? 2 : 4);
    n.at_ds = n.at_dy + bytes(p.dy.bf16 ? 2 : 4);
    n.at_scales = n.at_ds + (p.dsummed.p ? bytes(p.dx.bf16 ? 2 : 4) : 0);
    n.stage_bytes = n.at_scales + (mode == kAnyRow && act8 ? (p.cols / kAct8Block + 1 + 15) / 16 * 16 + pad : 0);
    if (mode == kWarpRow) {
        n.warps = 1;
        n.vecs = vecs > 96 ? 4 : 3;
        n.blocks_per_sm = 1;
        n.depth = (int)std::min<size_t>(kNormDepth, kNormRingSmem / (kNormWarps * n.stage_bytes));
        n.smem = std::max((size_t)kNormWarps * n.depth * n.stage_bytes, (size_t)kNormWarps * n.vecs * 32 * kVec * 4);
        return n;
    }
    double best = 0;
    for (int v = 1; v <= 4; ++v) {
        const int warps = (vecs + 32 * v - 1) / (32 * v);
        if ((v - 1) * warps * 32 >= vecs) continue;  // fewer vectors a thread do
        if (warps > kNormWarps || (v >= (mode == kAnyRow ? 3 : 4) && full && n.warps)) continue;
        const bool regs = mode == kAnyRow ? v == 1 : v <= 3 || !full;
        size_t w_bytes = regs ? 0 : (size_t)v * warps * 32 * kVec * 4;
        int blocks = kNormWarps / warps;
        while (blocks > 1 && blocks * (kBlockExtra + w_bytes + 2 * n.stage_bytes) > kSmemOfSM) --blocks;
        const double time = (double)((p.rows + blocks * kNormSMs - 1) / (blocks * kNormSMs)) * (v + (v == 4 ? 3.5 : 2));
        if (n.warps && time >= best) continue;
        best = time;
        const size_t room = std::min(kNormRingSmem, kSmemOfSM / blocks - kBlockExtra);
        n.w_in_smem = w_bytes + n.stage_bytes <= room;
        if (!n.w_in_smem) w_bytes = 0;
        n.warps = warps, n.vecs = v, n.blocks_per_sm = blocks;
        n.depth = (int)std::min<size_t>(kNormDepth, (room - w_bytes) / n.stage_bytes);
        n.smem = (size_t)n.depth * n.stage_bytes + w_bytes;
    }
    return n;
}

}  // namespace

// As many blocks as run at once: one of 16 warps on an SM for rows that warps take, else of the warps that four
// vectors a thread need.
int norm_backward_parts(int rows, int cols) {
    const int warps = (vectors(cols) + 127) / 128;
    return (int)std::min<int64_t>(rows, kNormSMs * (kNormWarps / warps));
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, cudaStream_t stream) {
    const bool act8 = !p.x.p, full = !p.rms || p.want_db;
    const bool fast = p.dy.fast && (act8 ? p.ckpt.fast : p.x.fast) && (!p.dsummed.p || p.dsummed.fast);
    cudaError_t e = cudaErrorUnknown;
    int blocks;
    if (fast && p.cols <= kShortCols && p.dx.bf16 <= p.dy.bf16) {
        blocks = std::min(p.rows, kNormSMs);
#define RLK_SHORT(SRC, X, DY) (full ? launch_short<SRC, X, DY, true>(p, blocks, stream) : launch_short<SRC, X, DY, false>(p, blocks, stream))
        if (act8)
            e = p.ckpt.e4m3 ? p.dx.bf16 ? RLK_SHORT(kHE4M3, true, true) : p.dy.bf16 ? RLK_SHORT(kHE4M3, false, true) : RLK_SHORT(kHE4M3, false, false)
                            : p.dx.bf16 ? RLK_SHORT(kHInt8, true, true) : p.dy.bf16 ? RLK_SHORT(kHInt8, false, true) : RLK_SHORT(kHInt8, false, false);
        else
            e = p.x.bf16 ? RLK_SHORT(kHBf16, true, true) : p.dy.bf16 ? RLK_SHORT(kHF32, false, true) : RLK_SHORT(kHF32, false, false);
#undef RLK_SHORT
    } else {
        const bool any = !fast || (!act8 && p.x.bf16 && !p.dy.bf16);
        // a warp per row where there are rows for all warps
        const bool warp = !any && p.cols > 512 && p.cols <= (full ? 768 : 1024) && p.rows >= kNormSMs * kNormWarps;
        const NormTeams n = teams_of(p, any ? kAnyRow : warp ? kWarpRow : kBlockRow);
        blocks = std::min(p.rows, kNormSMs * n.blocks_per_sm);
#define RLK_ROWS(H) (p.dy.bf16 ? launch_norm_rows_##H##_bf16(p, n, blocks, stream) : launch_norm_rows_##H##_f32(p, n, blocks, stream))
        e = act8 ? p.ckpt.e4m3 ? RLK_ROWS(e4m3) : RLK_ROWS(int8) : p.x.bf16 ? RLK_ROWS(bf16) : RLK_ROWS(f32);
#undef RLK_ROWS
    }
    return e == cudaSuccess ? launch_join(p, blocks, stream) : e;
}

}  // namespace rlk

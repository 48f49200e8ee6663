// The forward pass of the norms: rows on 16-byte boundaries (norm_fwd.cuh), short ones among them, and which kernel takes a call.
#include "norm_fwd.cuh"
#include "norm_short.cuh"

namespace rlk {

namespace {

constexpr int kShortWarps = 24;  // 80 registers a thread

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

constexpr size_t kSmemOfSM = 228 * 1024, kBlockExtra = 1024 + 1024;  // what a block takes beside its rows

template <bool BF16>
cudaError_t launch_short(const NormForwardParams &p, cudaStream_t stream) {
    const int es[2] = {BF16 ? 2 : 4, !p.residual.p ? 0 : BF16 ? 2 : 4};
    const int64_t ld[2] = {p.x.ld, p.residual.ld};
    const int width = (p.cols <= 64 ? 2 : 4) * kVec * (p.cols <= 128 ? 4 : p.cols <= 256 ? 8 : 16);
    const NormShort n = norm_short(p.cols, es, ld, 2, p.mask != nullptr, kShortWarps, (size_t)width * 8, 0);
    const bool full = !p.rms || p.b;
    const bool exact = p.cols == width && !p.mask && p.y.fast;
#define RLK_RUN(V, F, E) run_kernel<norm_forward_short_kernel<BF16, V, F, E>>(std::min(p.rows, kNormSMs), kShortWarps * 32, n.smem, kNormRingSmem, stream, p, n)
#define RLK_SHORT(V, F) (exact ? RLK_RUN(V, F, true) : RLK_RUN(V, F, false))
    return n.vecs == 2 ? full ? RLK_SHORT(2, true) : RLK_SHORT(2, false) : full ? RLK_SHORT(4, true) : RLK_SHORT(4, false);
#undef RLK_SHORT
#undef RLK_RUN
}

// Two rows of a block in its ring: with as many as fit, reads far ahead of the writes cost the memory's rate. (65536 x 6144
// bf16, RMS: 246 us, with eight 281; 32768 x 16384: 317, 367.)
constexpr int kForwardDepth = 2;

// The blocks that run at once, or, for as many bytes to write as to read, blocks of eight rows for a warp or block, which
// start when others end: they do not read and write all in step, and a slow SM takes fewer. Where the weights' way into shared memory
// or arithmetic is what a block waits for, their starts cost more, and masked rows break the step too. (RMS with a
// residual, us: 65536 x 6144 bf16 with an int8 checkpoint 599 -> 525, 32768 x 6144 fp32 527 -> 471, 8192 x 6144 bf16 72 -> 65; layer norm
// so 534 -> 466; but with an e4m3 checkpoint 65536 x 5120 489 -> 576, without a residual 16384 x 6144 79 -> 88, with a mask 125 -> 132.)
int blocks_of(const NormForwardParams &p, int mode, const NormTeams &n, int teams) {
    const bool full = starts_anywhere(mode) || !p.rms || p.b;
    const int at_once = std::min(p.rows, kNormSMs * n.blocks_per_sm), short_ones = p.rows / (8 * teams);
    const bool apart = p.residual.p && !p.mask && !starts_anywhere(mode) && (!full || (mode == kBlockRow && n.vecs < 4 && !p.ckpt.codes));
    return apart && short_ones >= 3 * at_once ? short_ones : at_once;
}

// A block per row, 16 warps on an SM: of the numbers of vectors a thread, the one whose blocks take all rows soonest, by a
// row's time of its vectors and two or three more for its exchanges of sums and what else is done once a row. (16384 x
// 8192 bf16: layer norm with two, three, four vectors 141, 147, 125 us, RMS with a residual 180, 174, 181 (without blocks of eight rows); 20000 x 5120: 156, 92,
// 102 us; so layer norm with four, whose weights are read from shared memory, counts as 9.8.)
NormTeams teams_of(const NormForwardParams &p, int mode) {
    const int vecs = (p.cols + kVec - 1) / kVec, pad = starts_anywhere(mode) ? 32 : 0;
    const bool full = starts_anywhere(mode) || !p.rms || p.b;
    NormTeams n{};
    n.mode = mode;
    n.at_dy = (p.cols * (p.x.bf16 ? 2 : 4) + 15) / 16 * 16 + pad;
    n.stage_bytes = n.at_dy * (p.residual.p ? 2 : 1);
    if (mode == kWarpRow) {
        n.warps = 1;
        n.vecs = vecs > 96 ? 4 : 3;
        n.blocks_per_sm = 1;
        n.depth = (int)std::min<size_t>(kNormDepth, kNormRingSmem / (kForwardWarps * n.stage_bytes));
        n.smem = (size_t)(kForwardWarps) * n.depth * n.stage_bytes;
        n.blocks = blocks_of(p, mode, n, kForwardWarps);
        return n;
    }
    double best = 0;
    for (int v = 1; v <= 4; ++v) {
        const int warps = (vecs + 32 * v - 1) / (32 * v);
        if (warps > kForwardWarps || (v - 1) * warps * 32 >= vecs) continue;
        if (n.warps && mode == kAnyRow && v > 2) continue;  // (registers)
        // layer norm with four vectors a thread: weight and bias in shared memory, as registers have no room
        size_t params = mode != kAnyRow && full && v == 4 ? (size_t)2 * v * warps * 32 * kVec * 4 : 0;
        int blocks = kForwardWarps / warps;
        while (blocks > 1 && blocks * (kBlockExtra + params + 2 * n.stage_bytes) > kSmemOfSM) --blocks;
        const double time = (double)((p.rows + blocks * kNormSMs - 1) / (blocks * kNormSMs)) * (v + (p.rms ? 2 : v == 4 ? 5.8 : 3));
        if (n.warps && time >= best) continue;
        best = time;
        const size_t room = std::min(kNormRingSmem, kSmemOfSM / blocks - kBlockExtra);
        n.w_in_smem = params + n.stage_bytes <= room;
        if (!n.w_in_smem) params = 0;
        n.warps = warps, n.vecs = v, n.blocks_per_sm = blocks;
        n.depth = (int)std::min<size_t>(kForwardDepth, (room - params) / n.stage_bytes);
        n.smem = (size_t)n.depth * n.stage_bytes + params;
    }
    n.blocks = blocks_of(p, mode, n, 1);
    return n;
}

}  // namespace

cudaError_t launch_norm_forward(const NormForwardParams &p, cudaStream_t stream) {
    // (with rows that start anywhere on any side: vectors cut up at the store, a warp's stores 16 bytes apart, took 515 us for
    // 8920 x 9118 bf16 with a residual, which takes 182 so, and 112 between rows on 16-byte boundaries)
    const bool fast = p.x.fast && (!p.residual.p || p.residual.fast) && p.y.fast && (!p.h.p || p.h.fast) && (!p.ckpt.codes || p.ckpt.fast);
    if (fast && p.cols <= kShortCols) return p.x.bf16 ? launch_short<true>(p, stream) : launch_short<false>(p, stream);
    if (!fast) {
        // The pieces shifted into place, where 8-bit codes are made or a thread would hold more than two vectors' single columns,
        // whose weights have no room in registers: 16000 x 3001 bf16 layer norm to int8 94 us (single columns 199), 8920 x 9118 bf16
        // with a residual 182 (270), 8192 x 6145 layer norm 95 (99); but 8192 x 4095 61 (52), 30000 x 1031 fp32 with a residual 115 (88).
        const bool shift = p.ckpt.codes || p.cols > 4096;
        const NormTeams n = teams_of(p, shift ? kShiftRow : kAnyRow);
        return shift ? launch_norm_forward_shift(p, n, stream) : launch_norm_forward_any(p, n, stream);
    }
    const bool full = !p.rms || p.b, warp = p.cols <= (full ? 768 : 1024) && p.rows >= kNormSMs * kForwardWarps;  // a warp per row where there are rows for all
    const NormTeams n = teams_of(p, warp ? kWarpRow : kBlockRow);
#define RLK_ROWS(BF16) (warp ? full ? launch_forward_rows<BF16, 3, true, kWarpRow>(p, n, stream) : n.vecs == 3 ? launch_forward_rows<BF16, 3, false, kWarpRow>(p, n, stream) : launch_forward_rows<BF16, 4, false, kWarpRow>(p, n, stream) \
                             : full ? launch_forward_vecs<BF16, true, kBlockRow>(p, n, stream) : launch_forward_vecs<BF16, false, kBlockRow>(p, n, stream))
    return p.x.bf16 ? RLK_ROWS(true) : RLK_ROWS(false);
#undef RLK_ROWS
}

}  // namespace rlk

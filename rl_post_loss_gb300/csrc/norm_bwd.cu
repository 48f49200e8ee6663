// The backward pass of the norms (mathematics and layout: norm.cuh).
#include <algorithm>

#include "norm.cuh"
#include "ptx.cuh"

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

// ---------------------------------------------------------------- rows through shared memory
//
// Rows that start on 16-byte boundaries: bulk copies bring the next rows into shared memory while the block
// works on one, which it reads twice from there (the sums, then dx), so that a thread holds little more than
// its sums of dw and db in registers. A row's stage is filled again after the next row's exchange of sums,
// when every thread has left it: no barrier but that exchange's.

enum HSource { kHBf16, kHF32, kHAct8 };

template <int SRC>
__device__ __forceinline__ V8 read_h(const char *stage, int col, uint32_t scale, const NormBackwardParams &p) {
    if (SRC == kHBf16) return bf16_pairs(*reinterpret_cast<const uint4 *>(stage + (size_t)col * 2));
    if (SRC == kHF32) {
        const uint4 *q = reinterpret_cast<const uint4 *>(stage + (size_t)col * 4);
        return f32_pairs(q[0], q[1]);
    }
    float v[kVec];
    act8_decode(*reinterpret_cast<const uint2 *>(stage + col), scale, p.ckpt.e4m3, __uint_as_float(0x7f7fffffu), v);
    return pairs_of(v);
}
__device__ __forceinline__ V8 read_mat(const char *stage, int col, bool bf16) {
    if (bf16) return bf16_pairs(*reinterpret_cast<const uint4 *>(stage + (size_t)col * 2));
    const uint4 *q = reinterpret_cast<const uint4 *>(stage + (size_t)col * 4);
    return f32_pairs(q[0], q[1]);
}

constexpr uint64_t kCopyWaitNs = 1000000000ull;

template <int SRC, bool DYBF16, int VPT, bool DB>
__global__ void __launch_bounds__(512) norm_backward_ring_kernel(NormBackwardParams p, NormRing ring) {
    extern __shared__ __align__(128) char smem[];
    __shared__ float s_buf[2][2][16];
    __shared__ __align__(8) uint64_t s_full[16];
    RowSum<64> sums(s_buf);
    const int T = blockDim.x, t = threadIdx.x, S = ring.depth, stage_bytes = (int)(ring.h_bytes + ring.dy_bytes + ring.ds_bytes);
    char *w_smem = smem + (size_t)S * stage_bytes;
    const int off_dy = (int)ring.h_bytes, off_ds = off_dy + (int)ring.dy_bytes;
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(ptx::smem_u32(&s_full[s]), 1);
        ptx::fence_mbar_init();
    }
    // a thread's part of the weight, which nobody else reads, stays beside the rows
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = (t + i * T) * kVec;
        if (col < p.cols) {
            float w[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) w[j] = 1.f;
            if (p.w) load_params(p.w, p.params_bf16, p.params_fast, col, p.cols, w);
            if (p.params_bf16)
                store_vec(reinterpret_cast<__nv_bfloat16 *>(w_smem), col, col + kVec, true, w);
            else
                store_vec(reinterpret_cast<float *>(w_smem), col, col + kVec, true, w);
        }
    }
    V8 dw[VPT], db[DB ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            dw[i].p[k] = 0ull;
            if (DB) db[i].p[k] = 0ull;
        }
    __syncthreads();

    const int64_t step = gridDim.x;
    const auto copy_row = [&](int64_t row, int s) {  // by thread 0
        char *stage = smem + (size_t)s * stage_bytes;
        const uint32_t full = ptx::smem_u32(&s_full[s]);
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive_expect_tx(full, (uint32_t)stage_bytes);
        const char *h = SRC == kHAct8 ? reinterpret_cast<const char *>(p.ckpt.codes) + row * p.ckpt.ld_codes
                                      : static_cast<const char *>(p.x.p) + row * p.x.ld * (SRC == kHBf16 ? 2 : 4);
        ptx::bulk_g2s(ptx::smem_u32(stage), h, (uint32_t)ring.h_bytes, full);
        ptx::bulk_g2s(ptx::smem_u32(stage + off_dy), static_cast<const char *>(p.dy.p) + row * p.dy.ld * (DYBF16 ? 2 : 4), (uint32_t)ring.dy_bytes, full);
        if (ring.ds_bytes)
            ptx::bulk_g2s(ptx::smem_u32(stage + off_ds), static_cast<const char *>(p.dsummed.p) + row * p.dsummed.ld * (p.dsummed.bf16 ? 2 : 4), (uint32_t)ring.ds_bytes, full);
    };
    if (t == 0)
        for (int s = 0; s < S; ++s) {
            const int64_t row = blockIdx.x + s * step;
            if (row < p.rows && (!p.mask || p.mask[row])) copy_row(row, s);
        }

    bool dead = false, on = true;  // on, mean, rstd, scales: of the row at hand, loaded a row ahead
    float mean = 0.f, rstd = 0.f;
    uint32_t scale[SRC == kHAct8 ? VPT : 1];
    const auto row_data = [&](int64_t row, bool &o, float &m, float &r, uint32_t (&sc)[SRC == kHAct8 ? VPT : 1]) {
        if (row >= p.rows) return;
        o = !p.mask || p.mask[row];
        r = p.rstd[row];
        if (!p.rms) m = p.mean[row];
        if (SRC == kHAct8) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * T) * kVec;
                sc[i] = col < p.cols ? p.ckpt.scales[row * p.ckpt.ld_scales + col / kAct8Block] : 0;
            }
        }
    };
    row_data(blockIdx.x, on, mean, rstd, scale);
    uint32_t phases = 0;  // of the stages' barriers
    int s = 0, last = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += step) {
        bool on_next = true;
        float mean_next = 0.f, rstd_next = 0.f;
        uint32_t scale_next[SRC == kHAct8 ? VPT : 1] = {};
        row_data(row + step, on_next, mean_next, rstd_next, scale_next);
        bool more = false;  // the row that takes the last row's stage
        const int64_t row_more = row + (S - 1) * step;
        if (t == 0 && row != blockIdx.x && row_more < p.rows) more = !p.mask || p.mask[row_more];

        const char *stage = smem + (size_t)s * stage_bytes;
        float c1 = 0.f, c2 = 0.f;
        const f32x2 nm = pack2(-mean, -mean), rs = pack2(rstd, rstd);
        if (on) {
            if (!dead && !ptx::mbar_wait(ptx::smem_u32(&s_full[s]), (phases >> s) & 1u, kCopyWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
            f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int col = (t + i * T) * kVec;
                if (col >= p.cols) continue;
                V8 h = read_h<SRC>(stage, col, scale[SRC == kHAct8 ? i : 0], p), g = read_mat(stage + off_dy, col, DYBF16);
                if (col + kVec > p.cols) h = clipped(h, col, p.cols), g = clipped(g, col, p.cols);
                const V8 w = read_mat(w_smem, col, p.params_bf16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 xh = mul2(add2(h.p[k], nm), rs);
                    dw[i].p[k] = fma2(g.p[k], xh, dw[i].p[k]);
                    if (DB) db[i].p[k] = add2(db[i].p[k], g.p[k]);
                    const f32x2 gw = mul2(g.p[k], w.p[k]);
                    s0 = add2(s0, gw);
                    s1 = fma2(gw, xh, s1);
                }
            }
            float two[2] = {sum_of(s0), sum_of(s1)};
            sums.run(two);
            c1 = p.rms ? 0.f : two[0] * p.inv_cols;
            c2 = two[1] * p.inv_cols;
            if (t == 0 && p.status && !(fabsf(two[0]) < INFINITY && fabsf(two[1]) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
        } else {
            __syncthreads();
        }
        if (more && !dead) copy_row(row_more, last);
        const f32x2 m1 = pack2(-c1, -c1), m2 = pack2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (t + i * T) * kVec;
            if (col >= p.cols) continue;
            float o[kVec] = {};
            if (on) {
                const V8 h = read_h<SRC>(stage, col, scale[SRC == kHAct8 ? i : 0], p), g = read_mat(stage + off_dy, col, DYBF16);
                const V8 w = read_mat(w_smem, col, p.params_bf16);
                V8 d = {}, r;
                if (ring.ds_bytes) d = read_mat(stage + off_ds, col, p.dsummed.bf16);
                V8 xh;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xh.p[k] = mul2(add2(h.p[k], nm), rs);
                    r.p[k] = fma2(fma2(xh.p[k], m2, add2(mul2(g.p[k], w.p[k]), m1)), rs, d.p[k]);
                }
                if (p.y.p) {
                    float b[kVec] = {};
                    if (p.b) load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, b);
                    const V8 bb = pairs_of(b);
                    V8 u;
#pragma unroll
                    for (int k = 0; k < 4; ++k) u.p[k] = add2(mul2(xh.p[k], w.p[k]), bb.p[k]);
                    floats_of(u, o);
                    store_row(p.y, row, col, p.cols, o);
                }
                floats_of(r, o);
            } else if (p.y.p) {
                store_row(p.y, row, col, p.cols, o);
            }
            store_row(p.dx, row, col, p.cols, o);
        }
        on = on_next, mean = mean_next, rstd = rstd_next;
#pragma unroll
        for (int i = 0; i < (SRC == kHAct8 ? VPT : 1); ++i) scale[i] = scale_next[i];
        last = s;
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead) {  // (copies in flight end before the block does, or do not within another wait)
        if (t == 0)
            for (int k = 0; k < S; ++k) ptx::mbar_wait(ptx::smem_u32(&s_full[k]), (phases >> k) & 1u, kCopyWaitNs);
        __syncthreads();
    }
    if (!p.want_dw && !p.want_db) return;
    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = (t + i * T) * kVec;
        if (col >= p.cols) continue;
        float v[kVec];
        floats_of(dw[i], v);
        store_vec(part, col, (int)p.ld_part, true, v);
        if (DB) {
            floats_of(db[i], v);
            store_vec(part + p.ld_part, col, (int)p.ld_part, true, v);
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

constexpr size_t kSmemOfSM = 228 * 1024, kSmemOfBlock = 227 * 1024;

// Blocks of up to 16 warps on an SM, 128 registers a thread; the fewest warps a block that leave a thread three
// vectors (four beyond 12288 columns), and stages of the whole SM's shared memory.
NormRing ring_of(const NormBackwardParams &p) {
    NormRing r{};
    const auto row_bytes = [&](size_t es) { return (p.cols * es + 15) / 16 * 16; };
    r.h_bytes = row_bytes(!p.x.p ? 1 : p.x.bf16 ? 2 : 4);
    r.dy_bytes = row_bytes(p.dy.bf16 ? 2 : 4);
    r.ds_bytes = p.dsummed.p ? row_bytes(p.dsummed.bf16 ? 2 : 4) : 0;
    const int vecs = (p.cols + kVec - 1) / kVec;
    r.w_bytes = (size_t)vecs * kVec * (p.params_bf16 ? 2 : 4);
    const size_t stage = r.h_bytes + r.dy_bytes + r.ds_bytes, fixed = r.w_bytes + 32 + 2048;  // (32: an fp32 vector past the row's end)
    int blocks = 16 / fewest_warps(p.cols);
    while (blocks > 1 && blocks * (2 * stage + fixed) > kSmemOfSM) --blocks;
    r.warps = std::min(16 / blocks, (vecs + 31) / 32);
    r.vecs = (vecs + r.warps * 32 - 1) / (r.warps * 32);
    r.warps = (vecs + r.vecs * 32 - 1) / (r.vecs * 32);
    r.blocks_per_sm = blocks;
    const size_t room = std::min(kSmemOfBlock, kSmemOfSM / blocks);
    if (room < fixed + 2 * stage) return r;
    r.depth = (int)std::min<size_t>(8, (room - fixed) / stage);
    r.smem = r.depth * stage + r.w_bytes + 32;
    return r;
}

template <int SRC, bool DYBF16, int VPT, bool DB>
cudaError_t launch_ring(const NormBackwardParams &p, const NormRing &r, cudaStream_t stream) {
    auto kernel = norm_backward_ring_kernel<SRC, DYBF16, VPT, DB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmemOfBlock - 2048));
    if (e != cudaSuccess) return e;
    const int parts = std::min(p.rows, kNormSMs * r.blocks_per_sm);
    kernel<<<parts, r.warps * 32, r.smem, stream>>>(p, r);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(p, parts, stream) : e;
}

template <int SRC, bool DYBF16>
cudaError_t launch_ring_shape(const NormBackwardParams &p, const NormRing &r, cudaStream_t stream) {
    switch (r.vecs * 2 + (p.want_db ? 1 : 0)) {
        case 2: return launch_ring<SRC, DYBF16, 1, false>(p, r, stream);
        case 3: return launch_ring<SRC, DYBF16, 1, true>(p, r, stream);
        case 4: return launch_ring<SRC, DYBF16, 2, false>(p, r, stream);
        case 5: return launch_ring<SRC, DYBF16, 2, true>(p, r, stream);
        case 6: return launch_ring<SRC, DYBF16, 3, false>(p, r, stream);
        case 7: return launch_ring<SRC, DYBF16, 3, true>(p, r, stream);
        case 8: return launch_ring<SRC, DYBF16, 4, false>(p, r, stream);
        default: return launch_ring<SRC, DYBF16, 4, true>(p, r, stream);
    }
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
    if (p.cols > 256 && p.dy.fast && (act8 ? p.ckpt.fast : p.x.fast) && (!p.dsummed.p || p.dsummed.fast)) {
        const NormRing r = ring_of(p);
        if (r.depth >= 2) {
            if (act8) return p.dy.bf16 ? launch_ring_shape<kHAct8, true>(p, r, stream) : launch_ring_shape<kHAct8, false>(p, r, stream);
            if (p.x.bf16) return p.dy.bf16 ? launch_ring_shape<kHBf16, true>(p, r, stream) : launch_ring_shape<kHBf16, false>(p, r, stream);
            return p.dy.bf16 ? launch_ring_shape<kHF32, true>(p, r, stream) : launch_ring_shape<kHF32, false>(p, r, stream);
        }
    }
    if (!p.x.p) return p.dy.bf16 ? launch_shape<FromAct8, Bf16Rows>(p, s, stream) : launch_shape<FromAct8, F32Rows>(p, s, stream);
    if (p.x.bf16) return p.dy.bf16 ? launch_shape<FromBf16, Bf16Rows>(p, s, stream) : launch_shape<FromBf16, F32Rows>(p, s, stream);
    return p.dy.bf16 ? launch_shape<FromF32, Bf16Rows>(p, s, stream) : launch_shape<FromF32, F32Rows>(p, s, stream);
}

}  // namespace rlk

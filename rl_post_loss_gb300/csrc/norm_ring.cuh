// The backward pass of the norms on rows that start on 16-byte boundaries (mathematics: norm.cuh).
//
// Bulk copies bring the next rows into shared memory while the block works on one, which it reads twice from
// there (the sums, then dx), so that a thread holds little more than its sums of dw and db in registers. A
// row's stage is filled again after the next row's exchange of sums, when every thread has left it: no
// barrier but that exchange's.
//
// Written with r = dy rstd, u = r w, d = h - mean: xh = d rstd, g = dy w, so dw += r d, mean(g) rstd =
// mean(u), mean(g xh) = mean(u d), and dx = u - mean(u) - d k + dsummed with k = rstd^2 mean(u d). FULL = false
// is the RMS form without db, in which mean = 0 and sum(u) is not needed.
#pragma once

#include "norm.cuh"
#include "ptx.cuh"

namespace rlk {

enum HSource { kHBf16, kHF32, kHAct8 };

constexpr uint64_t kNormWaitNs = 1000000000ull;

template <bool BF16>
__device__ __forceinline__ V8 read_vec(const char *row, int vec) {
    if (BF16) return bf16_pairs(*reinterpret_cast<const uint4 *>(row + vec * 16));
    const uint4 *q = reinterpret_cast<const uint4 *>(row + vec * 32);
    return f32_pairs(q[0], q[1]);
}
template <int SRC>
__device__ __forceinline__ V8 read_h(const char *row, int vec, uint32_t scale, bool e4m3) {
    if (SRC != kHAct8) return read_vec<SRC == kHBf16>(row, vec);
    return act8_pairs(*reinterpret_cast<const uint2 *>(row + vec * 8), scale, e4m3);
}

// The block's sums of two values (FULL) or of the second one: a butterfly in each warp, which for two values
// first gives each half of the warp one of them; then the warps' sums, in their order, from shared memory.
// Two buffers in turn; unused places hold 0.
template <bool FULL>
__device__ __forceinline__ void block_sums(float &a, float &b, float2 *buf, int warps) {
    const int lane = threadIdx.x & 31;
    if (FULL) {
        const float give = lane < 16 ? b : a, keep = lane < 16 ? a : b;
        float v = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, 16));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
        if ((lane & 15) == 0) reinterpret_cast<float *>(buf + (threadIdx.x >> 5))[lane >> 4] = v;
    } else {
        float v = b;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
        if (lane == 0) buf[threadIdx.x >> 5].y = v;
    }
    __syncthreads();
    const float4 *q = reinterpret_cast<const float4 *>(buf);
    a = b = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 x = q[k];
        a += x.x + x.z;
        b += x.y + x.w;
    }
    if (warps > 8) {
#pragma unroll
        for (int k = 4; k < 8; ++k) {
            const float4 x = q[k];
            a += x.x + x.z;
            b += x.y + x.w;
        }
    }
}

template <int SRC, bool XBF16, bool DYBF16, int VPT, bool FULL>
__global__ void __launch_bounds__(512) norm_backward_ring_kernel(NormBackwardParams p, NormRing ring) {
    constexpr bool kWInRegs = VPT <= 3 || !FULL;  // (four vectors with both sums leave no room for it)
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) float2 s_sums[2][16];
    __shared__ __align__(8) uint64_t s_full[8];
    const int T = blockDim.x, t = threadIdx.x, S = ring.depth;
    const int off_dy = (int)ring.h_bytes, off_ds = off_dy + (int)ring.dy_bytes, stage_bytes = off_ds + (int)ring.ds_bytes;
    const int last_vec = t + (VPT - 1) * T;  // the one vector of a thread that may be short or missing
    const bool has_last = last_vec * kVec < p.cols, cut = has_last && (last_vec + 1) * kVec > p.cols;
    if (t < 32) reinterpret_cast<float2 *>(s_sums)[t] = make_float2(0.f, 0.f);
    if (t == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(ptx::smem_u32(&s_full[s]), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();

    const int64_t step = gridDim.x;
    const auto copy_row = [&](int64_t row, int s) {  // by thread 0
        char *stage = smem + s * stage_bytes;
        const uint32_t full = ptx::smem_u32(&s_full[s]);
        ptx::mbar_arrive_expect_tx(full, (uint32_t)stage_bytes);
        const char *h = SRC == kHAct8 ? reinterpret_cast<const char *>(p.ckpt.codes) + row * p.ckpt.ld_codes
                                      : static_cast<const char *>(p.x.p) + row * p.x.ld * (XBF16 ? 2 : 4);
        ptx::bulk_g2s(ptx::smem_u32(stage), h, (uint32_t)ring.h_bytes, full);
        ptx::bulk_g2s(ptx::smem_u32(stage + off_dy), static_cast<const char *>(p.dy.p) + row * p.dy.ld * (DYBF16 ? 2 : 4), (uint32_t)ring.dy_bytes, full);
        if (ring.ds_bytes)
            ptx::bulk_g2s(ptx::smem_u32(stage + off_ds), static_cast<const char *>(p.dsummed.p) + row * p.dsummed.ld * (XBF16 ? 2 : 4), (uint32_t)ring.ds_bytes, full);
    };
    if (t == 0)
        for (int s = 0; s < S; ++s) {
            const int64_t row = blockIdx.x + s * step;
            if (row < p.rows && (!p.mask || p.mask[row])) copy_row(row, s);
        }

    float *w_smem = reinterpret_cast<float *>(smem + S * stage_bytes);  // a thread's own part, read by nobody else
    V8 w[kWInRegs ? VPT : 1], dw[VPT], db[FULL ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = 1.f;
        if (p.w && (i < VPT - 1 || has_last)) load_params(p.w, p.params_bf16, p.params_fast, (t + i * T) * kVec, p.cols, v);
        if (kWInRegs)
            w[i] = pairs_of(v);
        else if (i < VPT - 1 || has_last)
            store_vec(w_smem, (t + i * T) * kVec, (t + i * T) * kVec + kVec, true, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            dw[i].p[k] = 0ull;
            if (FULL) db[i].p[k] = 0ull;
        }
    }

    // of the row at hand, loaded a row ahead
    constexpr int kScales = SRC == kHAct8 ? VPT : 1;
    bool dead = false, on = true;
    float mean = 0.f, rstd = 0.f;
    uint32_t scale[kScales];
    const auto row_data = [&](int64_t row, bool &o, float &m, float &r, uint32_t (&sc)[kScales]) {
        if (row >= p.rows) return;
        o = !p.mask || p.mask[row];
        r = p.rstd[row];
        if (FULL && !p.rms) m = p.mean[row];
        if (SRC == kHAct8) {
            const uint8_t *q = p.ckpt.scales + row * p.ckpt.ld_scales;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (i < VPT - 1 || has_last) sc[i] = q[(t + i * T) >> 2];
        }
    };
    row_data(blockIdx.x, on, mean, rstd, scale);
    uint32_t phases = 0;  // of the stages' barriers
    int s = 0, last = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += step) {
        bool on_next = true;
        float mean_next = 0.f, rstd_next = 0.f;
        uint32_t scale_next[kScales] = {};
        row_data(row + step, on_next, mean_next, rstd_next, scale_next);
        const int64_t row_more = row + (S - 1) * step;  // takes the last row's stage
        const bool more = t == 0 && row != blockIdx.x && row_more < p.rows && (!p.mask || p.mask[row_more]);

        const char *stage = smem + s * stage_bytes;
        float c1 = 0.f, c2 = 0.f;
        const f32x2 nm = pack2(-mean, -mean), rs = pack2(rstd, rstd);
        if (on) {
            if (!dead && !ptx::mbar_wait(ptx::smem_u32(&s_full[s]), (phases >> s) & 1u, kNormWaitNs)) {
                dead = true;
                if (p.status) raise_status(p.status, RL_ERR_TIMEOUT);
            }
            phases ^= 1u << s;
            f32x2 s0 = 0ull, s1 = 0ull;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (i == VPT - 1 && !has_last) continue;
                const int vec = t + i * T;
                V8 h = read_h<SRC>(stage, vec, scale[SRC == kHAct8 ? i : 0], p.ckpt.e4m3), g = read_vec<DYBF16>(stage + off_dy, vec);
                if (i == VPT - 1 && cut) h = clipped(h, vec * kVec, p.cols), g = clipped(g, vec * kVec, p.cols);
                const V8 ww = kWInRegs ? w[kWInRegs ? i : 0] : read_vec<false>(reinterpret_cast<const char *>(w_smem), vec);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 d = FULL ? add2(h.p[k], nm) : h.p[k], r = mul2(g.p[k], rs), u = mul2(r, ww.p[k]);
                    dw[i].p[k] = fma2(r, d, dw[i].p[k]);
                    if (FULL) {
                        db[i].p[k] = add2(db[i].p[k], g.p[k]);
                        s0 = add2(s0, u);
                    }
                    s1 = fma2(u, d, s1);
                }
            }
            c1 = sum_of(s0), c2 = sum_of(s1);
            block_sums<FULL>(c1, c2, s_sums[turn], T >> 5);
            turn ^= 1;
            if (t == 0 && p.status && !(fabsf(c1) < INFINITY && fabsf(c2) < INFINITY)) raise_status(p.status, RL_ERR_NONFINITE);
            c1 = FULL && !p.rms ? c1 * p.inv_cols : 0.f;
            c2 = c2 * p.inv_cols * rstd * rstd;
        } else {
            __syncthreads();
        }
        if (more && !dead) copy_row(row_more, last);
        const f32x2 o1 = pack2(-c1, -c1), nk = pack2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i == VPT - 1 && !has_last) continue;
            const int vec = t + i * T, col = vec * kVec;
            float o[kVec] = {};
            if (on) {
                const V8 h = read_h<SRC>(stage, vec, scale[SRC == kHAct8 ? i : 0], p.ckpt.e4m3), g = read_vec<DYBF16>(stage + off_dy, vec);
                const V8 ww = kWInRegs ? w[kWInRegs ? i : 0] : read_vec<false>(reinterpret_cast<const char *>(w_smem), vec);
                V8 r;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 rr = mul2(g.p[k], rs), u = FULL ? fma2(rr, ww.p[k], o1) : mul2(rr, ww.p[k]);
                    r.p[k] = fma2(FULL ? add2(h.p[k], nm) : h.p[k], nk, u);
                }
                if (ring.ds_bytes) {
                    const V8 d = read_vec<XBF16>(stage + off_ds, vec);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r.p[k] = add2(r.p[k], d.p[k]);
                }
                if (p.y.p) {
                    float b[kVec] = {};
                    if (p.b) load_params(p.b, p.params_bf16, p.params_fast, col, p.cols, b);
                    V8 u = pairs_of(b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) u.p[k] = fma2(mul2(add2(h.p[k], nm), rs), ww.p[k], u.p[k]);
                    floats_of(u, o);
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
        on = on_next, mean = mean_next, rstd = rstd_next;
#pragma unroll
        for (int i = 0; i < kScales; ++i) scale[i] = scale_next[i];
        last = s;
        s = s + 1 == S ? 0 : s + 1;
    }
    if (dead) {  // (copies in flight end before the block does, or do not within another wait)
        if (t == 0)
            for (int k = 0; k < S; ++k) ptx::mbar_wait(ptx::smem_u32(&s_full[k]), (phases >> k) & 1u, kNormWaitNs);
        __syncthreads();
    }
    if (!p.want_dw && !p.want_db) return;
    float *part = p.partials + (int64_t)blockIdx.x * 2 * p.ld_part;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (i == VPT - 1 && !has_last) continue;
        float v[kVec];
        floats_of(dw[i], v);
        store_vec(part, (t + i * T) * kVec, (int)p.ld_part, true, v);
        if (FULL) {
            floats_of(db[i], v);
            store_vec(part + p.ld_part, (t + i * T) * kVec, (int)p.ld_part, true, v);
        }
    }
}

template <int SRC, bool XBF16, bool DYBF16, int VPT, bool FULL>
cudaError_t launch_norm_ring(const NormBackwardParams &p, const NormRing &r, int parts, cudaStream_t stream) {
    auto kernel = norm_backward_ring_kernel<SRC, XBF16, DYBF16, VPT, FULL>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormRingSmem);
    if (e != cudaSuccess) return e;
    kernel<<<parts, r.warps * 32, r.smem, stream>>>(p, r);
    return cudaGetLastError();
}

template <int SRC, bool XBF16, bool DYBF16>
cudaError_t launch_norm_ring_shape(const NormBackwardParams &p, const NormRing &r, int parts, cudaStream_t stream) {
    const bool full = !p.rms || p.want_db;
    switch (r.vecs) {
        case 1: return full ? launch_norm_ring<SRC, XBF16, DYBF16, 1, true>(p, r, parts, stream) : launch_norm_ring<SRC, XBF16, DYBF16, 1, false>(p, r, parts, stream);
        case 2: return full ? launch_norm_ring<SRC, XBF16, DYBF16, 2, true>(p, r, parts, stream) : launch_norm_ring<SRC, XBF16, DYBF16, 2, false>(p, r, parts, stream);
        case 3: return full ? launch_norm_ring<SRC, XBF16, DYBF16, 3, true>(p, r, parts, stream) : launch_norm_ring<SRC, XBF16, DYBF16, 3, false>(p, r, parts, stream);
        default: return full ? launch_norm_ring<SRC, XBF16, DYBF16, 4, true>(p, r, parts, stream) : launch_norm_ring<SRC, XBF16, DYBF16, 4, false>(p, r, parts, stream);
    }
}

}  // namespace rlk

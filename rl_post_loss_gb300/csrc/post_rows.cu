// Row kernels of the vocabulary-wide post-training operators (post.cuh has their mathematics): one
// block walks a row twice, first for its softmax statistics, then for its gradient.
#include <algorithm>

#include "post.cuh"
#include "ptx.cuh"

namespace rlk {

namespace {

enum PostOp { kLogp, kPolicy, kDistill };

constexpr int kThreads = 512;
constexpr int kMarkBits = 1 << 16;  // vocabulary entries whose marks are held at once (distill)

// Fixed-order sums of the blocks' partials by the last block to finish; it leaves the count at 0.
template <typename Finish>
__device__ __forceinline__ void finish_sums(const PostRows &r, const PostPartial &mine, int nblocks, Finish finish) {
    __shared__ int s_last;
    __shared__ double s_d[32];
    __shared__ int s_i[32];
    if (threadIdx.x == 0) {
        r.partials[blockIdx.x] = mine;
        __threadfence();
        s_last = atomicAdd(r.blocks_done, 1u) == (uint32_t)nblocks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    PostPartial a{};
    for (int b = threadIdx.x; b < nblocks; b += blockDim.x) {
        const PostPartial q = r.partials[b];
        a.loss += q.loss;
        a.ent += q.ent;
        a.kl += q.kl;
        a.n += q.n;
        a.popped += q.popped;
        a.clipped += q.clipped;
        a.masked += q.masked;
    }
    a.loss = block_sum_f64(a.loss, s_d);
    a.ent = block_sum_f64(a.ent, s_d);
    a.kl = block_sum_f64(a.kl, s_d);
    a.n = block_sum_i32(a.n, s_i);
    a.popped = block_sum_i32(a.popped, s_i);
    a.clipped = block_sum_i32(a.clipped, s_i);
    a.masked = block_sum_i32(a.masked, s_i);
    finish(a, s_i);
    if (threadIdx.x == 0) {
        *r.blocks_done = 0;
        r.loss[0] = (float)a.loss;
        if (r.loss_f64) r.loss_f64[0] = a.loss;
        if (!isfinite(a.loss)) post_raise(r.status, RL_ERR_NONFINITE);
    }
}

template <typename T>
__device__ __forceinline__ const char *row_in(const PostRows &r, int t) {
    return reinterpret_cast<const char *>(r.logits) + (size_t)t * r.ld * sizeof(T);
}
template <typename T>
__device__ __forceinline__ char *row_out(const PostRows &r, int t) {
    return reinterpret_cast<char *>(r.dlogits) + (size_t)t * r.ldd * sizeof(T);
}

template <bool kEnt>
__device__ __forceinline__ PostStats block_merge(PostStats st, PostStats *s_warp, float c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    st = post_warp_merge<kEnt>(st, c);
    __syncthreads();
    if (lane == 0) s_warp[warp] = st;
    __syncthreads();
    st = lane < kThreads / 32 ? s_warp[lane] : kPostStart;
    return post_warp_merge<kEnt>(st, c);
}

// Statistics of a row without its entry y (y < 0: of the whole row).
template <typename T, bool kEnt>
__device__ __forceinline__ PostStats row_stats(const char *z, int V, float c, int y) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    const int nvec = V / VEC;
    PostStats st = kPostStart;
#pragma unroll 4
    for (int k = threadIdx.x; k < nvec; k += kThreads) {
        float x[VEC];
        VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
        if (y >= 0 && k == y / VEC) {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (j == y % VEC) x[j] = -INFINITY;
        }
        post_fold<kEnt>(st, x, c);
    }
    const int v = nvec * VEC + threadIdx.x;
    if (v < V && v != y) {
        float x[1] = {VT::load1(z, v)};
        post_fold<kEnt>(st, x, c);
    }
    return st;
}

// dz_v = a 2^{c (z_v - m)}, except dz_y = gy (y < 0: no such entry). a == 0 writes zeros without reading.
template <typename T>
__device__ __forceinline__ void write_row(const char *z, char *dz, int V, float c, RowGrad gr) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    const int nvec = V / VEC;
    const bool zero = gr.a == 0.f && gr.y < 0;
#pragma unroll 4
    for (int k = threadIdx.x; k < nvec; k += kThreads) {
        float x[VEC];
        if (zero) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = 0.f;
        } else {
            VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = gr.a * ex2_approx((x[j] - gr.m) * c);
            if (k == gr.y / VEC && gr.y >= 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (j == gr.y % VEC) x[j] = gr.gy;
            }
        }
        __stcs(reinterpret_cast<uint4 *>(dz + (size_t)k * 16), VT::encode(x));
    }
    const int v = nvec * VEC + threadIdx.x;
    if (v < V) VT::store1(dz, v, zero ? 0.f : v == gr.y ? gr.gy : gr.a * ex2_approx((VT::load1(z, v) - gr.m) * c));
}

template <typename T, bool kEnt>
__global__ void __launch_bounds__(kThreads) logp_rows_kernel(LogpParams p) {
    __shared__ PostStats s_warp[kThreads / 32];
    if (p.zero && blockIdx.x == 0 && threadIdx.x == 0) *p.zero = 0;
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        if (p.r.mask && !__ldg(p.r.mask + t)) {
            if (threadIdx.x == 0) {
                p.r.logp[t] = 0.f;
                if (kEnt) p.r.entropy[t] = 0.f;
                if (p.stats) p.stats[t] = make_float2(0.f, 1.f);
            }
            continue;
        }
        const char *z = row_in<T>(p.r, t);
        const int y = __ldg(p.r.targets + t);
        const bool ok = y >= 0 && y < p.r.V;
        PostStats st = block_merge<kEnt>(row_stats<T, kEnt>(z, p.r.V, kLog2e, ok ? y : -1), s_warp, kLog2e);
        if (threadIdx.x == 0) {
            float logp = __int_as_float(0x7fc00000);
            if (ok) logp = post_target<kEnt>(st, PostVec<T>::load1(z, y), st);
            if (!ok) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
            if (!post_finite(st)) post_raise(p.r.status, RL_ERR_NONFINITE);
            p.r.logp[t] = logp;
            if (kEnt) p.r.entropy[t] = post_entropy(st);
            if (p.stats) p.stats[t] = make_float2(st.m, st.s);
        }
    }
}

template <typename T, bool kEnt>
__global__ void __launch_bounds__(kThreads) policy_rows_kernel(PolicyParams p) {
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ RowGrad s_grad;
    PostPartial sum{};
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        const char *z = row_in<T>(p.r, t);
        const bool read = p.read_masked || __ldg(p.r.mask + t);
        const int y = __ldg(p.r.targets + t);
        const bool ok = y >= 0 && y < p.r.V;
        PostStats st{0.f, 1.f, 0.f};
        if (read) st = block_merge<kEnt>(row_stats<T, kEnt>(z, p.r.V, kLog2e, ok ? y : -1), s_warp, kLog2e);
        if (threadIdx.x == 0) {
            const float logp = ok && read ? post_target<kEnt>(st, PostVec<T>::load1(z, y), st) : 0.f;
            s_grad = policy_row(p, t, policy_load(p, t, find_seq(p.r.cu_seqlens, p.r.S, t)), st, logp, true, sum);
        }
        __syncthreads();
        const RowGrad gr = s_grad;
        write_row<T>(z, row_out<T>(p.r, t), p.r.V, kLog2e, gr);
        __syncthreads();
    }
    finish_sums(p.r, sum, gridDim.x, [&](const PostPartial &a, int *s_i) {
        int empty = 0;
        for (int i = threadIdx.x; i < p.r.S; i += blockDim.x) empty += p.seq_n[i] == 0;
        empty = block_sum_i32(empty, s_i);
        if (threadIdx.x != 0) return;
        if (p.counts) {
            p.counts[0] = a.popped;
            p.counts[1] = a.clipped;
            p.counts[2] = a.masked;
            p.counts[3] = empty;
        }
        if (p.mean_entropy) p.mean_entropy[0] = a.n > 0 ? (float)(a.ent / a.n) : 0.f;
        if (p.kl.mean_kl) p.kl.mean_kl[0] = a.n > 0 ? (float)(a.kl / a.n) : 0.f;
    });
}

// pref: dz_v = g (1[v == y] - p_v) with g the response's coefficient, from the statistics of the
// log-prob pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) scale_rows_kernel(ScaleParams p) {
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        const int i = find_seq(p.r.cu_seqlens, p.r.S, t);
        const int y = __ldg(p.r.targets + t);
        RowGrad gr{0.f, 0.f, 0.f, -1};
        if (i >= 0 && __ldg(p.r.mask + t) && y >= 0 && y < p.r.V) {
            const float2 st = p.stats[t];
            const float g = p.coef[i];
            if (g != 0.f) gr = post_row_grad(g, PostStats{st.x, st.y, 0.f}, p.r.logp[t], y);
        }
        write_row<T>(row_in<T>(p.r, t), row_out<T>(p.r, t), p.r.V, kLog2e, gr);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_rows_kernel(DistillParams p) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    extern __shared__ float s_dyn[];
    float *s_z = s_dyn, *s_lq = s_dyn + p.K;
    int *s_id = reinterpret_cast<int *>(s_dyn + 2 * p.K);
    __shared__ uint32_t s_mark[kMarkBits / 32];
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ DistillRow s_row;
    __shared__ int s_int[32];
    const int V = p.r.V, nvec = V / VEC;
    PostPartial sum{};
    int N = 0;
    if (p.per_token) {
        for (int i = threadIdx.x; i < p.r.S; i += kThreads) N += p.seq_n[i];
        N = block_sum_i32(N, s_int);
    }
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        const char *z = row_in<T>(p.r, t);
        char *dz = row_out<T>(p.r, t);
        const int i = find_seq(p.r.cu_seqlens, p.r.S, t);
        const bool on = i >= 0 && __ldg(p.r.mask + t);
        if (!on) {
            if (threadIdx.x == 0 && p.kl) p.kl[t] = 0.f;
            write_row<T>(z, dz, V, p.c, RowGrad{0.f, 0.f, 0.f, -1});
            continue;
        }
        const float4 rec = p.rec[t];
        // the teacher's entries
        int bad = 0, have = 0;
        for (int k = threadIdx.x; k < p.K; k += kThreads) {
            const int id = __ldg(p.ids + (int64_t)t * p.ldk + k);
            const bool real = id >= 0 && id < V;
            bad |= id < -1 || id >= V;
            have += real;
            s_id[k] = real ? id : -1;
            s_z[k] = real ? VT::load1(z, id) : -INFINITY;
            s_lq[k] = real ? (__ldg(p.vals + (int64_t)t * p.ldk + k) - rec.x) - rec.y : -INFINITY;
        }
        have = block_sum_i32(have, s_int);
        // the statistics outside them: marked entries count as -inf
        PostStats st = kPostStart;
        for (int64_t base = 0; base < V; base += kMarkBits) {
            for (int w = threadIdx.x; w < kMarkBits / 32; w += kThreads) s_mark[w] = 0;
            __syncthreads();
            for (int k = threadIdx.x; k < p.K; k += kThreads) {
                const int64_t at = (int64_t)s_id[k] - base;
                if (s_id[k] >= 0 && at >= 0 && at < kMarkBits)
                    bad |= (atomicOr(&s_mark[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1;  // listed twice
            }
            __syncthreads();
            const int k1 = (int)min((int64_t)nvec, (base + kMarkBits) / VEC);
            for (int k = (int)(base / VEC) + threadIdx.x; k < k1; k += kThreads) {
                float x[VEC];
                VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
                const int at = (int)((int64_t)k * VEC - base);
                const uint32_t mark = s_mark[at >> 5] >> (at & 31);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if ((mark >> j) & 1) x[j] = -INFINITY;
                post_fold<false>(st, x, p.c);
            }
            if (base + kMarkBits >= V && nvec * VEC + (int)threadIdx.x < V) {
                const int v = nvec * VEC + threadIdx.x, at = (int)(v - base);
                if (at >= 0) {  // the last entries lie in the last chunk
                    float x[1] = {(s_mark[at >> 5] >> (at & 31)) & 1 ? -INFINITY : VT::load1(z, v)};
                    post_fold<false>(st, x, p.c);
                }
            }
            __syncthreads();
        }
        bad = __syncthreads_or(bad);
        st = block_merge<false>(st, s_warp, p.c);
        const int n_i = p.seq_n[i];
        const double w = p.per_token ? 1.0 / (double)N : 1.0 / ((double)p.r.S * (double)n_i);
        const bool none = have == 0 || !(rec.w > 0.f || isnan(rec.w));  // the teacher gives the row no mass
        if (bad || none) {  // excluded: contributes nothing
            if (threadIdx.x == 0) {
                if (bad) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
                if (p.kl) p.kl[t] = bad ? __int_as_float(0x7fc00000) : 0.f;
            }
            write_row<T>(z, dz, V, p.c, RowGrad{0.f, 0.f, 0.f, -1});
            __syncthreads();
            continue;
        }
        if (threadIdx.x < 32) {
            float Mk, Sk;
            distill_entry_stats(s_z, p.K, p.c, Mk, Sk);
            const DistillRow r = distill_finish(p, st, Mk, Sk, s_z, s_lq, rec, (float)w * p.scale * p.inv_tau, V - have);
            if (threadIdx.x == 0) {
                s_row = r;
                if (!isfinite(r.ls)) post_raise(p.r.status, RL_ERR_NONFINITE);
                if (p.kl) p.kl[t] = r.kl;
                sum.loss += w * (double)p.scale * (double)r.kl;
            }
        }
        __syncthreads();
        const DistillRow r = s_row;
        // the teacher's entries are written after the rest of the row, whose value they replace
        write_row<T>(z, dz, V, p.c, RowGrad{r.ct, r.m, 0.f, -1});
        __syncthreads();
        for (int k = threadIdx.x; k < p.K; k += kThreads)
            if (s_id[k] >= 0) VT::store1(dz, s_id[k], distill_entry(p, r, s_z[k], s_lq[k]));
        __syncthreads();
    }
    finish_sums(p.r, sum, gridDim.x, [](const PostPartial &, int *) {});
}

int grid_rows(int T) { return std::max(1, std::min(T, 608)); }

}  // namespace

cudaError_t launch_post_logp(const LogpParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0 && !p.zero) return cudaSuccess;
    const int grid = grid_rows(p.r.T);
    const bool ent = p.r.entropy != nullptr;
    if (dtype == RL_F32) {
        if (ent) logp_rows_kernel<float, true><<<grid, kThreads, 0, stream>>>(p);
        else logp_rows_kernel<float, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (ent) logp_rows_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(p);
        else logp_rows_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_post_policy(const PolicyParams &p, int dtype, cudaStream_t stream) {
    const int grid = grid_rows(p.r.T);
    const bool ent = p.r.entropy || p.mean_entropy;
    if (dtype == RL_F32) {
        if (ent) policy_rows_kernel<float, true><<<grid, kThreads, 0, stream>>>(p);
        else policy_rows_kernel<float, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (ent) policy_rows_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(p);
        else policy_rows_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_post_distill(const DistillParams &p, int dtype, cudaStream_t stream) {
    const int grid = grid_rows(p.r.T);
    const size_t smem = (size_t)p.K * 12;
    if (dtype == RL_F32) distill_rows_kernel<float><<<grid, kThreads, smem, stream>>>(p);
    else distill_rows_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_post_scale(const ScaleParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0) return cudaSuccess;
    const int grid = grid_rows(p.r.T);
    if (dtype == RL_F32) scale_rows_kernel<float><<<grid, kThreads, 0, stream>>>(p);
    else scale_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace rlk

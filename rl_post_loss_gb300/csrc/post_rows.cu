// Row kernels of the vocabulary-wide post-training operators (post.cuh has their mathematics).
//
// A row is cut over the CTAs of a cluster (one to eight). In each CTA a producer warp copies its
// slice of the next rows into a ring of shared-memory tiles (bulk copies completing on mbarriers)
// and gathers what the row needs besides its logits (the token's record, or the teacher's entries);
// the consumer warps fold the tiles into softmax statistics as they land. The CTAs exchange their
// statistics through distributed shared memory, every CTA finishes the row for itself, and the
// consumers walk the tiles, still in shared memory, a second time for the gradient: each logit is
// read from memory once. A tile is refilled with the next row's as soon as its second walk is done,
// so copies, folds and stores of consecutive rows overlap, and two or three CTAs on an SM fill each
// other's exchanges.
//
// Rows too long for the rings of a cluster (above about 1.8 MB with eight CTAs) take the block-per-row
// kernels at the end, which read a row twice.
#include <algorithm>
#include <mutex>

#include "post.cuh"
#include "ptx.cuh"

namespace rlk {

namespace {

// ---------------------------------------------------------------- sums of the batch

// Fixed-order sums of the slots' partials by the last of `nslots` blocks to fill its slot; it leaves
// the count at 0. Called by every thread of the block, with 512 bytes of shared memory.
template <typename Finish>
__device__ __forceinline__ void finish_sums(const PostRows &r, const PostPartial &mine, int slot, int nslots, void *scratch,
                                            Finish finish) {
    double *s_d = static_cast<double *>(scratch);      // [32]
    int *s_i = reinterpret_cast<int *>(s_d + 32);      // [32]
    int &s_last = s_i[32];
    __syncthreads();  // the scratch may be the ring's memory
    if (threadIdx.x == 0) {
        r.partials[slot] = mine;
        __threadfence();
        s_last = atomicAdd(r.blocks_done, 1u) == (uint32_t)nslots - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    PostPartial a{};
    for (int b = threadIdx.x; b < nslots; b += blockDim.x) {
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

__device__ __forceinline__ void policy_finish(const PolicyParams &p, const PostPartial &a, int *s_i) {
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
}

template <typename T>
__device__ __forceinline__ const char *row_in(const PostRows &r, int t) {
    return reinterpret_cast<const char *>(r.logits) + (size_t)t * r.ld * sizeof(T);
}
template <typename T>
__device__ __forceinline__ char *row_out(const PostRows &r, int t) {
    return reinterpret_cast<char *>(r.dlogits) + (size_t)t * r.ldd * sizeof(T);
}

// ---------------------------------------------------------------- the ring kernel

enum RowOp { kOpLogp, kOpPolicy, kOpDistill, kOpScale };

constexpr int kWarps = 8;                      // consumer warps
constexpr int kCons = 32 * kWarps;             // consumer threads
constexpr int kRowThreads = kCons + 32;        // and the producer warp
constexpr int kMaxCluster = 8;
constexpr int kMaxSlots = 8;
constexpr int kMeta = 2;                       // rows whose records are held

// How a launch cuts its rows.
struct RowPlan {
    int32_t cluster;    // CTAs per row
    int32_t slice;      // 16-byte groups per CTA
    int32_t tile;       // 16-byte groups per tile
    int32_t slots;      // tiles in the ring
};

template <int OP>
struct RowMeta;
template <>
struct RowMeta<kOpLogp> {
    int32_t copied, read;  // the row's logits are in the ring; they are needed
    int32_t y;             // the sampled entry, -1: none
    float zy;
};
template <>
struct RowMeta<kOpPolicy> {
    int32_t copied, read, y;
    float zy;
    PolicyTok tok;
};
template <>
struct RowMeta<kOpDistill> {
    int32_t copied, read;
    int32_t bad, have;     // an id outside the vocabulary; entries that are not padding
    float4 rec;
    double w;              // the row's weight
};
template <>
struct RowMeta<kOpScale> {
    int32_t copied, read;
    RowGrad grad;
};

struct RowMsg {
    float m, s, u;
    int32_t bad;
};

template <int OP>
struct RowShared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t mfull[kMeta], mempty[kMeta];
    uint64_t xbar[2];
    RowMsg xmsg[2][kMaxCluster];
    RowMsg warp[2][kWarps];
    RowMeta<OP> meta[kMeta];
    RowGrad grad[2];    // of the last two rows: a row without logits passes one barrier only
    DistillRow drow[2];
    int32_t dead;       // a wait ran out: nothing waits any more
    int32_t dup;        // distill: an entry is listed twice
    uint32_t tail_mark; // distill: marks of the last V mod VEC entries
};

// A bounded wait that gives up for good once any wait of the block has.
template <int OP>
__device__ __forceinline__ void row_wait(RowShared<OP> &sh, uint64_t *bar, uint32_t parity, uint32_t *status) {
    const uint32_t b = ptx::smem_u32(bar);
    if (ptx::mbar_try_wait(b, parity)) return;
    if (*reinterpret_cast<volatile int32_t *>(&sh.dead)) return;
    if (!ptx::mbar_wait(b, parity)) {
        *reinterpret_cast<volatile int32_t *>(&sh.dead) = 1;
        post_raise(status, RL_ERR_TIMEOUT);
    }
}

// A barrier of the consumer warps.
__device__ __forceinline__ void cons_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kCons) : "memory");
}

// 16 bytes into the shared memory of a CTA of the cluster, counted on its mbarrier.
__device__ __forceinline__ void st_async16(uint32_t dst, uint32_t bar, const RowMsg &v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(__float_as_uint(v.u)), "r"(v.bad), "r"(bar)
                 : "memory");
}

// find_seq by a warp: each step narrows 32-fold.
__device__ __forceinline__ int warp_find_seq(const int32_t *__restrict__ cu, int S, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane == 0 || (at < hi && __ldg(cu + at) <= t);
        const int l = 31 - __clz(__ballot_sync(0xffffffffu, le));
        lo += l * step;
        hi = min(hi, lo + step);
    }
    return (__ldg(cu + lo) <= t && t < __ldg(cu + lo + 1)) ? lo : -1;
}

template <int OP>
struct OpParams;
template <>
struct OpParams<kOpLogp> { using type = LogpParams; };
template <>
struct OpParams<kOpPolicy> { using type = PolicyParams; };
template <>
struct OpParams<kOpDistill> { using type = DistillParams; };
template <>
struct OpParams<kOpScale> { using type = ScaleParams; };

// Whether row t is copied into the ring.
template <int OP>
__device__ __forceinline__ bool row_wanted(const typename OpParams<OP>::type &p, int t) {
    if constexpr (OP == kOpLogp) return !p.r.mask || __ldg(p.r.mask + t);
    if constexpr (OP == kOpPolicy) return p.read_masked || __ldg(p.r.mask + t);
    return __ldg(p.r.mask + t) != 0;
}

// The record of row t, by the producer warp.
template <typename T, int OP>
__device__ __forceinline__ void load_meta(const typename OpParams<OP>::type &p, int t, int N, RowMeta<OP> &m, float *s_z,
                                          float *s_lq, int *s_id) {
    using VT = PostVec<T>;
    const int lane = threadIdx.x & 31;
    const char *z = row_in<T>(p.r, t);
    const bool copied = row_wanted<OP>(p, t);
    if constexpr (OP == kOpLogp) {
        if (lane == 0) {
            const int y = __ldg(p.r.targets + t);
            m.copied = m.read = copied;
            m.y = y >= 0 && y < p.r.V ? y : -1;
            m.zy = copied && m.y >= 0 ? VT::load1(z, y) : 0.f;
        }
    } else if constexpr (OP == kOpPolicy) {
        const int i = warp_find_seq(p.r.cu_seqlens, p.r.S, t);
        if (lane == 0) {
            m.tok = policy_load(p, t, i);
            m.copied = copied;
            m.read = m.tok.m || p.read_masked;
            m.y = m.tok.ok ? m.tok.y : -1;
            m.zy = copied && m.tok.ok ? VT::load1(z, m.tok.y) : 0.f;
        }
    } else if constexpr (OP == kOpScale) {
        const int i = warp_find_seq(p.r.cu_seqlens, p.r.S, t);
        if (lane == 0) {
            const int y = __ldg(p.r.targets + t);
            RowGrad gr{0.f, 0.f, 0.f, -1};
            if (i >= 0 && copied && y >= 0 && y < p.r.V) {
                const float2 st = p.stats[t];
                const float g = p.coef[i];
                if (g != 0.f) gr = post_row_grad(g, PostStats{st.x, st.y, 0.f}, p.r.logp[t], y);
            }
            m.copied = copied;
            m.read = gr.y >= 0;
            m.grad = gr;
        }
    } else {
        const int i = warp_find_seq(p.r.cu_seqlens, p.r.S, t);
        const bool on = i >= 0 && copied;
        int bad = 0, have = 0;
        float4 rec = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll 4
            for (int k = lane; k < p.K; k += 32) {
                const int id = __ldg(p.ids + (int64_t)t * p.ldk + k);
                const float val = __ldg(p.vals + (int64_t)t * p.ldk + k);
                const bool real = id >= 0 && id < p.r.V;
                bad |= id < -1 || id >= p.r.V;
                have += real;
                s_id[k] = real ? id : -1;
                s_z[k] = real ? VT::load1(z, id) : -INFINITY;
                s_lq[k] = val;
            }
            rec = p.rec[t];
            for (int k = lane; k < p.K; k += 32) s_lq[k] = s_id[k] >= 0 ? (s_lq[k] - rec.x) - rec.y : -INFINITY;
            have = warp_sum_i32(have);
            bad = __any_sync(0xffffffffu, bad);
        }
        if (lane == 0) {
            // a teacher that gives the row no mass contributes nothing; nor does a bad row
            const bool none = have == 0 || !(rec.w > 0.f || isnan(rec.w));
            m.copied = copied;
            m.read = on && !bad && !none;
            m.bad = bad;
            m.have = have;
            m.rec = rec;
            m.w = !on ? 0.0 : p.per_token ? 1.0 / (double)N : 1.0 / ((double)p.r.S * (double)p.seq_n[i]);
        }
    }
}

template <typename T, int OP, bool kEnt>
__global__ void __launch_bounds__(kRowThreads, 3)
ring_rows_kernel(const __grid_constant__ typename OpParams<OP>::type p, const __grid_constant__ RowPlan plan, int nclusters) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    constexpr bool kStats = OP != kOpScale;   // a row is folded first
    constexpr bool kGrad = OP != kOpLogp;     // a row is written
    extern __shared__ __align__(128) uint4 s_ring[];
    __shared__ RowShared<OP> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = plan.cluster;
    const int rank = (int)blockIdx.x % C, q = (int)blockIdx.x / C;
    const int T_ = p.r.T, V = p.r.V, nvec = V / VEC;
    const int v0 = min(nvec, rank * plan.slice), v1 = min(nvec, v0 + plan.slice);  // this CTA's 16-byte groups
    const int n_tiles = (v1 - v0 + plan.tile - 1) / plan.tile;
    const bool last_rank = rank == C - 1;    // has the last V mod VEC entries too
    const int tail_v = nvec * VEC + tid;     // a consumer's entry of those
    const bool has_tail = last_rank && tail_v < V;
    float c = kLog2e;
    int K = 0, N = 0;
    if constexpr (OP == kOpDistill) {
        c = p.c;
        K = p.K;
    }
    float *s_meta = reinterpret_cast<float *>(s_ring + (size_t)plan.slots * plan.tile);  // [kMeta][3][K]

    if (tid == 0) {
        for (int s = 0; s < plan.slots; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kWarps);
        }
        for (int s = 0; s < kMeta; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.mfull[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.mempty[s]), kWarps);
        }
        for (int s = 0; s < 2; ++s) ptx::mbar_init(ptx::smem_u32(&sh.xbar[s]), 1);
        ptx::fence_mbar_init();
        sh.dead = 0;
        sh.dup = 0;
        sh.tail_mark = 0;
    }
    if constexpr (OP == kOpLogp)
        if (p.zero && blockIdx.x == 0 && tid == 0) *p.zero = 0;
    if constexpr (OP == kOpDistill) {
        if (p.per_token) {
            for (int i = tid; i < p.r.S; i += kRowThreads) N += p.seq_n[i];
            N = block_sum_i32(N, reinterpret_cast<int *>(s_ring));
            ptx::fence_proxy_async_smem();  // the ring's first copies come after this use of its memory
        }
    }
    __syncthreads();
    if (kStats && C > 1) ptx::cluster_sync();  // every CTA's mbarriers are ready
    PostPartial sum{};

    if (warp == kWarps) {
        // ------------------------------------------------ producer
        int n = 0;  // tiles issued
        int slot = 0;
        uint32_t phase = 0;
        const uint64_t pol = ptx::l2_evict_first_policy();
        int r = 0;
        for (int qt = q; qt < T_; qt += nclusters, ++r) {
            const int t = OP == kOpScale ? T_ - 1 - qt : qt;  // scale: the rows read last are the likeliest in L2
            const int tiles = row_wanted<OP>(p, t) ? n_tiles : 0;
            const char *src = row_in<T>(p.r, t) + (size_t)v0 * 16;
            auto record = [&] {
                const int ms = r % kMeta;
                if (r >= kMeta) row_wait(sh, &sh.mempty[ms], ((r / kMeta) & 1) ^ 1, p.r.status);
                float *mz = s_meta + (size_t)ms * 3 * K;
                load_meta<T, OP>(p, t, N, sh.meta[ms], mz, mz + K, reinterpret_cast<int *>(mz + 2 * K));
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.mfull[ms]));
            };
            if (tiles == 0) record();
            for (int j = 0; j < tiles; ++j) {
                const int g = min(plan.tile, v1 - v0 - j * plan.tile);
                if (n >= plan.slots) row_wait(sh, &sh.empty[slot], phase ^ 1, p.r.status);
                if (lane == 0 && !*reinterpret_cast<volatile int32_t *>(&sh.dead)) {
                    const uint32_t bar = ptx::smem_u32(&sh.full[slot]);
                    ptx::mbar_arrive_expect_tx(bar, (uint32_t)g * 16);
                    const uint32_t dst = ptx::smem_u32(s_ring + (size_t)slot * plan.tile);
                    const char *from = src + (size_t)j * plan.tile * 16;
                    if (OP == kOpLogp && p.r.dlogits) ptx::bulk_g2s(dst, from, (uint32_t)g * 16, bar);  // read again
                    else ptx::bulk_g2s_hint(dst, from, (uint32_t)g * 16, bar, pol);
                }
                __syncwarp();
                ++n;
                if (++slot == plan.slots) slot = 0, phase ^= 1;
                // the record goes between the row's first copies and those that wait for tiles of the
                // same row (a row longer than the ring): the consumers free none before they have it
                if (j == min(tiles, plan.slots) - 1) record();
            }
        }
        if (*reinterpret_cast<volatile int32_t *>(&sh.dead) && lane == 0) {
            // a wait ran out: no copy may be in flight when the block exits
            for (int k = max(0, n - plan.slots); k < n; ++k)
                ptx::mbar_wait(ptx::smem_u32(&sh.full[k % plan.slots]), (k / plan.slots) & 1, 100000000ull);
        }
    } else {
        // ------------------------------------------------ consumers
        int slot = 0;
        uint32_t phase = 0;
        int r = 0, nr = 0;  // rows; rows folded
        for (int qt = q; qt < T_; qt += nclusters, ++r) {
            const int t = OP == kOpScale ? T_ - 1 - qt : qt;
            const int ms = r % kMeta;
            row_wait(sh, &sh.mfull[ms], (r / kMeta) & 1, p.r.status);
            const RowMeta<OP> &meta = sh.meta[ms];
            const bool copied = meta.copied, read = meta.read;
            const char *z = row_in<T>(p.r, t);
            const float *s_z = s_meta + (size_t)ms * 3 * K, *s_lq = s_z + K;
            const int *s_id = reinterpret_cast<const int *>(s_z + 2 * K);
            int y = -1;
            if constexpr (OP == kOpLogp || OP == kOpPolicy) y = meta.y;
            PostStats st{0.f, 1.f, 0.f};
            int dup = 0;

            if (kStats && read) {
                if constexpr (OP == kOpDistill) {
                    // marks: the teacher's entries of this slice become -inf in the ring, so that the
                    // fold leaves them out. Each first gets its index as a tag: an entry listed twice
                    // finds another's tag (or -inf) in its place.
                    int sl = slot;
                    uint32_t ph = phase;
                    for (int j = 0; j < n_tiles; ++j) {
                        row_wait(sh, &sh.full[sl], ph, p.r.status);
                        if (++sl == plan.slots) sl = 0, ph ^= 1;
                    }
                    using Tag = typename VT::Tag;
                    auto place = [&](int id) -> volatile Tag * {
                        const int g = id / VEC - v0;
                        int s = slot + g / plan.tile;
                        if (s >= plan.slots) s -= plan.slots;
                        return reinterpret_cast<volatile Tag *>(s_ring + (size_t)s * plan.tile + g % plan.tile) + id % VEC;
                    };
                    for (int k = tid; k < K; k += kCons) {
                        const int id = s_id[k];
                        if (id >= v0 * VEC && id < v1 * VEC) {
                            *place(id) = (Tag)k;
                        } else if (last_rank && id >= nvec * VEC) {
                            const uint32_t bit = 1u << (id - nvec * VEC);
                            if (atomicOr(&sh.tail_mark, bit) & bit) sh.dup = 1;
                        }
                    }
                    cons_sync();
                    for (int k = tid; k < K; k += kCons) {
                        const int id = s_id[k];
                        if (id < v0 * VEC || id >= v1 * VEC) continue;
                        if (*place(id) == (Tag)k) *place(id) = VT::kNegInf;
                        else sh.dup = 1;
                    }
                    ptx::fence_proxy_async_smem();  // the next copy into these tiles comes after the marks
                    cons_sync();
                }
                st = kPostStart;
                const int ky = y >= 0 ? y / VEC - v0 : -1;
                int sl = slot;
                uint32_t ph = phase;
                for (int j = 0; j < n_tiles; ++j) {
                    if (OP != kOpDistill) row_wait(sh, &sh.full[sl], ph, p.r.status);
                    uint4 *tile = s_ring + (size_t)sl * plan.tile;
                    const int g = min(plan.tile, v1 - v0 - j * plan.tile);
                    if constexpr (OP != kOpDistill) {
                        // the thread that folds the sampled entry's group takes the entry out of it
                        const int kyt = ky - j * plan.tile;
                        if (kyt >= 0 && kyt < g && kyt % kCons == tid) {
                            reinterpret_cast<volatile typename VT::Tag *>(tile + kyt)[y % VEC] = VT::kNegInf;
                            ptx::fence_proxy_async_smem();  // the next copy into the tile comes after this
                        }
                    }
                    int k = tid;
                    for (; k + 3 * kCons < g; k += 4 * kCons) {
                        const uint4 v[4] = {tile[k], tile[k + kCons], tile[k + 2 * kCons], tile[k + 3 * kCons]};
                        post_fold_groups<T, kEnt>(st, v, c);
                    }
                    for (; k < g; k += kCons) {
                        const uint4 v[1] = {tile[k]};
                        post_fold_groups<T, kEnt>(st, v, c);
                    }
                    if (!kGrad) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[sl]));
                    }
                    if (++sl == plan.slots) sl = 0, ph ^= 1;
                }
                if (!kGrad) slot = sl, phase = ph;
                if (has_tail && tail_v != y && !(OP == kOpDistill && (sh.tail_mark >> tid) & 1)) {
                    const float x[1] = {VT::load1(z, tail_v)};
                    post_fold<kEnt>(st, x, c);
                }
                st = post_warp_merge<kEnt>(st, c);
                const int x = nr & 1;
                if (lane == 0) sh.warp[x][warp] = RowMsg{st.m, st.s, st.u, 0};
                cons_sync();
                if (warp == 0) {
                    RowMsg w = sh.warp[x][lane < kWarps ? lane : 0];
                    st = lane < kWarps ? PostStats{w.m, w.s, w.u} : kPostStart;
                    st = post_warp_merge<kEnt>(st, c);
                    if constexpr (OP == kOpDistill) {
                        dup = *reinterpret_cast<volatile int32_t *>(&sh.dup);
                        __syncwarp();
                        if (lane == 0) sh.dup = 0, sh.tail_mark = 0;
                    }
                    if (C > 1) {
                        const uint32_t bar = ptx::smem_u32(&sh.xbar[x]);
                        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(C * sizeof(RowMsg)));
                        __syncwarp();
                        if (lane < C)
                            st_async16(ptx::mapa_shared(ptx::smem_u32(&sh.xmsg[x][rank]), lane), ptx::mapa_shared(bar, lane),
                                       RowMsg{st.m, st.s, st.u, dup});
                        row_wait(sh, &sh.xbar[x], (nr >> 1) & 1, p.r.status);
                        w = sh.xmsg[x][lane < C ? lane : 0];
                        st = lane < C ? PostStats{w.m, w.s, w.u} : kPostStart;
                        dup = __any_sync(0xffffffffu, lane < C && w.bad);
                        st = post_warp_merge<kEnt>(st, c);
                    }
                }
                ++nr;
            }

            // the row's results, by warp 0 of every CTA (rank 0 writes them)
            if constexpr (OP == kOpLogp) {
                if (tid == 0 && rank == 0) {
                    float logp = 0.f, ent = 0.f;
                    if (read) {
                        logp = __int_as_float(0x7fc00000);
                        if (y >= 0) logp = post_target<kEnt>(st, meta.zy, st);
                        else post_raise(p.r.status, RL_ERR_TARGET_RANGE);
                        if (!post_finite(st)) post_raise(p.r.status, RL_ERR_NONFINITE);
                        if (kEnt) ent = post_entropy(st);
                    }
                    p.r.logp[t] = logp;
                    if (kEnt) p.r.entropy[t] = ent;
                    if (p.stats) p.stats[t] = make_float2(st.m, st.s);
                }
            } else if constexpr (OP == kOpPolicy) {
                if (tid == 0) {
                    const float logp = read && y >= 0 ? post_target<kEnt>(st, meta.zy, st) : 0.f;
                    sh.grad[r & 1] = policy_row(p, t, meta.tok, st, logp, rank == 0, sum);
                }
                cons_sync();
            } else if constexpr (OP == kOpDistill) {
                if (warp == 0) {
                    const bool live = read && !dup;
                    DistillRow d{};
                    if (live) {
                        float Mk, Sk;
                        distill_entry_stats(s_z, K, c, Mk, Sk);
                        d = distill_finish(p, st, Mk, Sk, s_z, s_lq, meta.rec, (float)meta.w * p.scale * p.inv_tau, V - meta.have);
                    }
                    if (lane == 0) {
                        sh.drow[r & 1] = d;
                        sh.grad[r & 1] = RowGrad{live ? d.ct : 0.f, d.m, 0.f, live ? 0 : -1};
                        if (rank == 0) {
                            const bool bad = meta.bad || dup;
                            if (bad) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
                            if (live && !isfinite(d.ls)) post_raise(p.r.status, RL_ERR_NONFINITE);
                            if (p.kl) p.kl[t] = bad ? __int_as_float(0x7fc00000) : d.kl;
                            sum.loss += meta.w * (double)p.scale * (double)d.kl;
                        }
                    }
                }
                cons_sync();
            }

            if constexpr (kGrad) {
                RowGrad gr;
                if constexpr (OP == kOpScale) gr = meta.grad;
                else gr = sh.grad[r & 1];
                char *dz = row_out<T>(p.r, t);
                const bool zero = gr.y < 0;
                const int ky = OP == kOpDistill || zero ? -1 : gr.y / VEC - v0;
                for (int j = 0; j < n_tiles; ++j) {
                    const int g = min(plan.tile, v1 - v0 - j * plan.tile);
                    char *to = dz + ((size_t)v0 + (size_t)j * plan.tile) * 16;
                    const uint4 *tile = s_ring + (size_t)slot * plan.tile;
                    if (copied && !(kStats && read)) row_wait(sh, &sh.full[slot], phase, p.r.status);
                    if (zero) {
                        for (int k = tid; k < g; k += kCons) __stcs(reinterpret_cast<uint4 *>(to) + k, make_uint4(0, 0, 0, 0));
                    } else {
                        const int kyt = ky - j * plan.tile;
#pragma unroll 4
                        for (int k = tid; k < g; k += kCons) {
                            float x[VEC];
                            VT::decode(tile[k], x);
#pragma unroll
                            for (int i = 0; i < VEC; ++i) x[i] = gr.a * ex2_approx((x[i] - gr.m) * c);
                            __stcs(reinterpret_cast<uint4 *>(to) + k, VT::encode(x));
                        }
                        // by the thread that wrote the group, after it
                        if (OP != kOpDistill && kyt >= 0 && kyt < g && kyt % kCons == tid) VT::store1(dz, gr.y, gr.gy);
                    }
                    if (copied) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[slot]));
                        if (++slot == plan.slots) slot = 0, phase ^= 1;
                    }
                }
                if (has_tail) {
                    const float e = zero ? 0.f : gr.a * ex2_approx((VT::load1(z, tail_v) - gr.m) * c);
                    VT::store1(dz, tail_v, OP != kOpDistill && !zero && tail_v == gr.y ? gr.gy : e);
                }
                if constexpr (OP == kOpDistill) {
                    if (!zero) {
                        cons_sync();  // the entries are written after the rest of the row, whose value they replace
                        const DistillRow d = sh.drow[r & 1];
                        for (int k = tid; k < K; k += kCons) {
                            const int id = s_id[k];
                            if ((id >= v0 * VEC && id < v1 * VEC) || (last_rank && id >= nvec * VEC))
                                VT::store1(dz, id, distill_entry(p, d, s_z[k], s_lq[k]));
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.mempty[ms]));
        }
    }
    if constexpr (OP == kOpPolicy || OP == kOpDistill) {
        if (rank == 0) {
            finish_sums(p.r, sum, q, nclusters, s_ring, [&](const PostPartial &a, int *s_i) {
                if constexpr (OP == kOpPolicy) policy_finish(p, a, s_i);
            });
        }
    }
    if (kStats && C > 1) ptx::cluster_sync();  // no CTA leaves while another may still write to it
}

// ---------------------------------------------------------------- rows too long for the rings

constexpr int kThreads = 512;
constexpr int kMarkBits = 1 << 16;  // vocabulary entries whose marks are held at once (distill)

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
__global__ void __launch_bounds__(kThreads) long_policy_kernel(PolicyParams p) {
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ RowGrad s_grad;
    __shared__ double s_scratch[64];
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
    finish_sums(p.r, sum, blockIdx.x, gridDim.x, s_scratch, [&](const PostPartial &a, int *s_i) { policy_finish(p, a, s_i); });
}

template <typename T>
__global__ void __launch_bounds__(kThreads) long_distill_kernel(DistillParams p) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    extern __shared__ float s_dyn[];
    float *s_z = s_dyn, *s_lq = s_dyn + p.K;
    int *s_id = reinterpret_cast<int *>(s_dyn + 2 * p.K);
    __shared__ uint32_t s_mark[kMarkBits / 32];
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ DistillRow s_row;
    __shared__ int s_int[32];
    __shared__ double s_scratch[64];
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
    finish_sums(p.r, sum, blockIdx.x, gridDim.x, s_scratch, [](const PostPartial &, int *) {});
}

// ---------------------------------------------------------------- launches

// The ring of one CTA: what three (two, one) CTAs on an SM leave each of its 228 KB, less the 1 KB the
// system takes per CTA and the static state.
constexpr size_t kRingBytes[3] = {76800, 115712, 231424};

// How many clusters of this launch are resident at once; sets the kernel's shared-memory limit on its
// first use on a device and size. Remembered for the last sizes asked for.
cudaError_t resident_clusters(const void *kernel, const cudaLaunchConfig_t &cfg, int C, int max_dynamic, int *out) {
    struct Entry {
        const void *kernel = nullptr;
        int dev = -1, C = 0;
        size_t smem = 0;
        int resident = 0;
    };
    constexpr int kEntries = 64;
    static std::mutex mu;
    static Entry known[kEntries];
    static int next = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry &k : known)
        if (k.kernel == kernel && k.dev == dev && k.C == C && k.smem == cfg.dynamicSmemBytes) {
            *out = k.resident;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_dynamic);
    int resident = 0;
    if (e == cudaSuccess && cfg.numAttrs) {
        e = cudaOccupancyMaxActiveClusters(&resident, kernel, &cfg);
    } else if (e == cudaSuccess) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kRowThreads, cfg.dynamicSmemBytes);
        resident = sms * per / C;
    }
    if (e != cudaSuccess) return e;
    *out = std::max(1, std::min(resident, kPostMaxBlocks));
    known[next] = Entry{kernel, dev, C, cfg.dynamicSmemBytes, *out};
    next = (next + 1) % kEntries;
    return cudaSuccess;
}

template <typename T, int OP, bool kEnt>
cudaError_t launch_ring(const typename OpParams<OP>::type &p, int K, cudaStream_t stream, bool &fits) {
    auto kernel = ring_rows_kernel<T, OP, kEnt>;
    constexpr bool kStats = OP != kOpScale, kKeep = OP == kOpPolicy || OP == kOpDistill;
    const int nvec = p.r.V / PostVec<T>::kElems;
    constexpr size_t kMaxDynamic = kRingBytes[2] - sizeof(RowShared<OP>);
    const size_t fixed = sizeof(RowShared<OP>) + (size_t)kMeta * 12 * K + 16;
    RowPlan plan{};
    size_t smem = 0;
    fits = false;
    // the fewest CTAs per row whose slice stays in the ring of one of three CTAs on an SM; with eight,
    // of one of two, or of one
    int C = 1;
    for (int want = 456 / std::max(1, p.r.T); C < kMaxCluster && C * 2 <= want && nvec >= C * 2 * 256;) C *= 2;
    for (int occ = 0; occ < 3 && !fits;) {
        plan.cluster = C;
        plan.slice = std::max(1, (nvec + C - 1) / C);
        plan.tile = std::max(1, (plan.slice + 3) / 4);
        const size_t room = kRingBytes[occ] - fixed;
        if (!kKeep) plan.tile = std::min<int>(plan.tile, (int)(room / 16 / 4));
        plan.slots = (int)std::min<size_t>(kMaxSlots, room / ((size_t)plan.tile * 16));
        fits = kKeep ? (size_t)plan.slots * plan.tile >= (size_t)plan.slice : plan.slots >= 2;
        if (fits) break;
        if (C < kMaxCluster) C *= 2;
        else ++occ;
    }
    if (!fits) return cudaSuccess;
    smem = (size_t)plan.slots * plan.tile * 16 + (size_t)kMeta * 12 * K;
    smem = std::max<size_t>(smem, 1024);

    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = kStats && C > 1 ? 1 : 0;
    int resident = 0;
    const cudaError_t e = resident_clusters(reinterpret_cast<const void *>(kernel), cfg, C, (int)kMaxDynamic, &resident);
    if (e != cudaSuccess) return e;
    const int nclusters = std::max(1, std::min(p.r.T, resident));
    cfg.gridDim = dim3((unsigned)(nclusters * C));
    return cudaLaunchKernelEx(&cfg, kernel, p, plan, nclusters);
}

template <typename T>
cudaError_t launch_logp(const LogpParams &p, cudaStream_t stream) {
    bool fits;
    return p.r.entropy ? launch_ring<T, kOpLogp, true>(p, 0, stream, fits) : launch_ring<T, kOpLogp, false>(p, 0, stream, fits);
}

int long_grid(int T) { return std::max(1, std::min(T, 608)); }

template <typename T>
cudaError_t launch_policy(const PolicyParams &p, cudaStream_t stream) {
    const bool ent = p.r.entropy || p.mean_entropy;
    bool fits;
    const cudaError_t e = ent ? launch_ring<T, kOpPolicy, true>(p, 0, stream, fits) : launch_ring<T, kOpPolicy, false>(p, 0, stream, fits);
    if (fits) return e;
    if (ent) long_policy_kernel<T, true><<<long_grid(p.r.T), kThreads, 0, stream>>>(p);
    else long_policy_kernel<T, false><<<long_grid(p.r.T), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_distill(const DistillParams &p, cudaStream_t stream) {
    bool fits;
    const cudaError_t e = launch_ring<T, kOpDistill, false>(p, p.K, stream, fits);
    if (fits) return e;
    long_distill_kernel<T><<<long_grid(p.r.T), kThreads, (size_t)p.K * 12, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scale(const ScaleParams &p, cudaStream_t stream) {
    bool fits;
    return launch_ring<T, kOpScale, false>(p, 0, stream, fits);
}

}  // namespace

cudaError_t launch_post_logp(const LogpParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0 && !p.zero) return cudaSuccess;
    return dtype == RL_F32 ? launch_logp<float>(p, stream) : launch_logp<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_policy(const PolicyParams &p, int dtype, cudaStream_t stream) {
    return dtype == RL_F32 ? launch_policy<float>(p, stream) : launch_policy<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_distill(const DistillParams &p, int dtype, cudaStream_t stream) {
    return dtype == RL_F32 ? launch_distill<float>(p, stream) : launch_distill<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_scale(const ScaleParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0) return cudaSuccess;
    return dtype == RL_F32 ? launch_scale<float>(p, stream) : launch_scale<__nv_bfloat16>(p, stream);
}

}  // namespace rlk

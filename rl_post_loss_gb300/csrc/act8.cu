// Activations packed into 8 bits and read back (the format: act8.cuh).
#include "act8.cuh"

namespace rlk {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 8;

// A row's whole blocks are numbered in vectors of eight columns, so that four neighbouring lanes always hold
// one block; the threads of the grid step through all rows' vectors together.
struct Place {
    int64_t row;
    int vec;
    __device__ Place(const Act8Params &p) {
        const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        row = i / p.row_vecs;
        vec = (int)(i - row * p.row_vecs);
    }
    __device__ void step(const Act8Params &p) {
        row += p.step_rows;
        vec += p.step_vecs;
        if (vec >= p.row_vecs) {
            vec -= p.row_vecs;
            ++row;
        }
    }
};

template <typename T, typename Raw>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(Act8Params p) {
    for (Place at(p);; at.step(p)) {
        const bool live = at.row < p.rows;
        if (!__any_sync(0xffffffffu, live)) break;
        const int col = at.vec * kVec;
        float v[kVec] = {};
        if (live && col < p.cols) {
            Raw r;
            load_raw(r, static_cast<const T *>(p.x.p) + at.row * p.x.ld, col, p.cols, p.x.fast);
            to_float(r, v);
            clip_row(v, col, p.cols);
        }
        const uint32_t b = act8_scale(act8_block_max(act8_amax(v)), p.a.e4m3);
        if (live && col < p.cols) {
            store_codes(p.a.codes + at.row * p.a.ld_codes, col, p.cols, p.a.fast, act8_encode(v, b, p.a.e4m3));
            if ((at.vec & 3) == 0) p.a.scales[at.row * p.a.ld_scales + (at.vec >> 2)] = (uint8_t)b;
        }
    }
}

__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(Act8Params p) {
    const float most = p.x.bf16 ? __uint_as_float(0x7f7f0000u) : __uint_as_float(0x7f7fffffu);
    for (Place at(p); at.row < p.rows; at.step(p)) {
        const int col = at.vec * kVec;
        if (col >= p.cols) continue;
        Raw8 r;
        load_raw(r, p.a.codes + at.row * p.a.ld_codes, col, p.cols, p.a.fast);
        const uint32_t b = p.a.scales[at.row * p.a.ld_scales + (at.vec >> 2)];
        float v[kVec];
        floats_of(act8_decode(r.a, b, p.a.e4m3, most), v);
        store_row(p.x, at.row, col, p.cols, v);
    }
}

int grid_of(Act8Params &p) {
    p.row_vecs = (p.cols + kAct8Block - 1) / kAct8Block * (kAct8Block / kVec);
    const int64_t blocks = (p.rows * p.row_vecs + kThreads - 1) / kThreads;
    const int grid = (int)(blocks < kBlocks ? blocks : kBlocks);
    const int64_t all = (int64_t)grid * kThreads;
    p.step_rows = all / p.row_vecs;
    p.step_vecs = (int32_t)(all % p.row_vecs);
    return grid;
}

}  // namespace

cudaError_t launch_act8_pack(Act8Params p, cudaStream_t stream) {
    const int grid = grid_of(p);
    if (p.x.bf16)
        act8_pack_kernel<__nv_bfloat16, Raw16><<<grid, kThreads, 0, stream>>>(p);
    else
        act8_pack_kernel<float, Raw32><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(Act8Params p, cudaStream_t stream) {
    const int grid = grid_of(p);
    act8_unpack_kernel<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace rlk

// Short rows of the norms (512 columns and less, on 16-byte boundaries): 4, 8 or 16 threads of a warp take a row,
// with two or four vectors of eight columns each, so that a warp works on 8, 4 or 2 rows at a time and a row's
// sums take few steps. Every warp has a ring of its own in shared memory; the copies of its next rows are under
// way while it works on one batch. Rows that follow one another without a gap come in one copy.
//
// Bound by what a row costs beside its bytes, its shuffles and accesses to shared memory: 202752 x 128 bf16 layer norm 25 us forward
// (62% of the measured copy rate), 39 us backward (59%); 200000 x 512 78 us (77%) and 107 us (85%). With a mask every row is a copy of
// its own and the columns are checked (202752 x 128, a fifth masked: 34 us, 40%, and 58 us, 34%; backward from int8 78 us, 22%), and
// widths between powers of two leave lanes idle (100000 x 384: 49 us, 47%, and 70 us, 48%). (Two vectors a thread with the weights
// in registers, twice the lanes a row: 202752 x 128 forward 31 us. Weights that lie as in memory instead of in planes: 26 and 39 us, 93
// and 114 us; from int8 with a mask, 202752 x 128 backward, 72 against 76; 78 since every scale byte is read.)
#pragma once

#include "norm_rows.cuh"

namespace rlk {

// A warp's ring. Batch b is rows b (32 / lanes), ...; `base` and `pitch` are the matrices in memory, in bytes.
struct ShortRing {
    const NormShort &n;
    const uint8_t *mask;
    const char *base[3];
    int64_t pitch[3];
    int64_t rows;
    uint32_t stages, full;  // in shared memory
    int lane, per;
    __device__ __forceinline__ ShortRing(const NormShort &n) : n(n) {}
    // By the whole warp, which has read the stage.
    __device__ __forceinline__ void fetch(int64_t batch, int s) const {
        const int64_t row = batch * per + lane;
        const bool on = lane < per && row < rows && (!mask || mask[row]);
        const int count = __popc(__ballot_sync(0xffffffffu, on));
        if (count == 0) return;
        const uint32_t bar = full + s * 8, to = stages + s * n.stage_bytes;
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(count * (n.row_bytes[0] + n.row_bytes[1] + n.row_bytes[2])));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (!n.row_bytes[k]) continue;
            if (n.whole[k]) {
                if (lane == 0) ptx::bulk_g2s(to + n.at[k], base[k] + row * pitch[k], (uint32_t)(count * n.row_bytes[k]), bar);
            } else if (on) {
                ptx::bulk_g2s(to + n.at[k] + lane * n.row_bytes[k], base[k] + row * pitch[k], (uint32_t)n.row_bytes[k], bar);
            }
        }
    }
};

}  // namespace rlk

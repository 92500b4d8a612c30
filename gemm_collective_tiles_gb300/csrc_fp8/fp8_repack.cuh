// The copies that bring operands into the layout that the tensor memory
// accelerator reads.
#pragma once
#include "fp8_ptx.cuh"

namespace gct {
namespace fp8 {

// Copy of `rows` rows of unit-stride bytes, any distance apart, into rows of
// `pitch` bytes (a multiple of 16) on a 16-byte base; the last granule's bytes
// past a row's end are whatever follows there.  Bound by memory: a lane reads
// the two granules of 16 bytes around its source (the second is a neighbour's
// first, so it comes from the L1 cache), shifts and writes one; four rows are
// under way per thread.  Near the matrix's ends, byte by byte.
constexpr int COPY_ROWS = 32;  // rows of a CTA's tile: 8 warps x 4; columns: 32 granules
static __global__ void __launch_bounds__(256) repack_rows_kernel(const uint8_t* src, long long rs, uint8_t* dst, long long pitch,
                                                          long long rows, long long bytes) {
    constexpr int PER = COPY_ROWS / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tiles_c = (pitch + 511) / 512, tiles = tiles_c * ((rows + COPY_ROWS - 1) / COPY_ROWS);
    const uint8_t* const end = src + (rows - 1) * rs + bytes;
    grid_wait();
    grid_release();
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        const long long r0 = t / tiles_c * COPY_ROWS + warp, c = t % tiles_c * 512 + lane * 16;
        if (c >= pitch) continue;
        uint32_t g[PER][8], off[PER];
        bool whole[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const long long r = r0 + 8 * i;
            const uint8_t* at = src + r * rs + c;
            off[i] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
            at -= off[i];
            whole[i] = r < rows && at >= src && at + (off[i] ? 32 : 16) <= end;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint4 q = load16_if(at + 16 * w, whole[i] && (w == 0 || off[i]));
                g[i][4 * w] = q.x;
                g[i][4 * w + 1] = q.y;
                g[i][4 * w + 2] = q.z;
                g[i][4 * w + 3] = q.w;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const long long r = r0 + 8 * i;
            if (whole[i]) {
                uint32_t o[4];
                shift_granules<1>(g[i], off[i], o);
                *reinterpret_cast<uint4*>(dst + r * pitch + c) = make_uint4(o[0], o[1], o[2], o[3]);
            } else if (r < rows) {
                for (int e = 0; e < 16 && c + e < bytes; ++e) dst[r * pitch + c + e] = src[r * rs + c + e];
            }
        }
    }
}

// The same from any strides, in elements E.
template <typename E>
__global__ void __launch_bounds__(256) repack_kernel(const E* src, long long rs, long long cs, E* dst, long long pitch,
                                                     long long rows, long long cols) {
    // 32 x 32 tiles through shared memory: reads run along the source's
    // unit-stride dimension, writes along the destination's rows
    __shared__ E tile[32][33];
    const long long tiles_c = (cols + 31) / 32, tiles = tiles_c * ((rows + 31) / 32);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const bool by_col = rs == 1 && cs != 1;  // the source's rows are its unit-stride dimension
    grid_wait();
    grid_release();
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        const long long r0 = t / tiles_c * 32, c0 = t % tiles_c * 32;
        for (int i = ty; i < 32; i += 8) {
            const int a = by_col ? tx : i, b = by_col ? i : tx;
            if (r0 + a < rows && c0 + b < cols) tile[a][b] = src[(r0 + a) * rs + (c0 + b) * cs];
        }
        __syncthreads();
        for (int i = ty; i < 32; i += 8)
            if (r0 + i < rows && c0 + tx < cols) dst[(r0 + i) * pitch + c0 + tx] = tile[i][tx];
        __syncthreads();
    }
}

}  // namespace fp8
}  // namespace gct

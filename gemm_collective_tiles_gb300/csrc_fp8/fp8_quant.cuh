// Block quantiser to 8-bit floats, and the copies that bring operands into the
// layout the tensor memory accelerator reads.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_ptx.cuh"

namespace gct {
namespace fp8 {

enum : int { T_F16 = 0, T_BF16 = 1, T_F32 = 2 };

struct QuantParams {
    const void* x;
    uint8_t* codes;
    float* scales;
    long long x_rs, x_cs;      // elements
    long long c_rs, c_cs;      // codes (bytes)
    long long s_rs, s_cs;      // scales (elements), per block row and block column
    long long M, K;
    unsigned kblocks;          // blocks along K
    int e5m2, pow2;
    float fmax;                // largest code: 448 or 57344
    int pmin;                  // exponent of the smallest scale
};

template <int T>
__device__ __forceinline__ float load_elem(const void* p, long long i) {
    if (T == T_F32) return static_cast<const float*>(p)[i];
    if (T == T_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int T>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
    if (T == T_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
}

// largest finite magnitude so far and |v|
__device__ __forceinline__ float amax_finite(float m, float v) {
    const float a = fabsf(v);
    return a < __int_as_float(0x7F800000) ? fmaxf(m, a) : m;
}
// an infinity has no code of its own: it becomes NaN, like a NaN
__device__ __forceinline__ float finite_or_nan(float v) {
    return fabsf(v) < __int_as_float(0x7F800000) ? v : __int_as_float(0x7FFFFFFF);
}

// Scale and reciprocal of a block.  Power of two: FMAX is 1.75 * 2^n, so the
// smallest 2^p with amax <= 2^p * FMAX follows from amax's exponent and from
// whether its mantissa is above 1.75; both factors are exact.  Otherwise
// scale = amax / FMAX and the codes are x * (FMAX / amax), both rounded to
// nearest (true divisions, not approximations).
__device__ __forceinline__ void block_scale(const QuantParams& p, float amax, float& scale, float& inv) {
    amax = fmaxf(amax, p.fmax * __int_as_float((p.pmin + 127) << 23));
    if (p.pow2) {
        const uint32_t b = __float_as_uint(amax);
        const int e = static_cast<int>(b >> 23) - 127 - (p.e5m2 ? 15 : 8) + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        scale = __int_as_float((e + 127) << 23);
        inv = __int_as_float((127 - e) << 23);
    } else {
        scale = __fdiv_rn(amax, p.fmax);
        inv = __fdiv_rn(p.fmax, amax);
    }
}

constexpr int Q_THREADS = 256;
constexpr int Q_ROWS = 128;  // rows per CTA
constexpr int Q_PER = Q_ROWS / (Q_THREADS / 16);  // rows per thread

// largest value over the CTA (every thread gets it)
__device__ __forceinline__ float cta_max(float v) {
    __shared__ float part[Q_THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < Q_THREADS / 32; ++i) v = fmaxf(v, part[i]);
    return v;
}

// One CTA quantises 128 rows x one 128-column block; 16 lanes share a row,
// 8 consecutive elements each, and a thread holds its 8 rows in registers, so
// x is read once and every load is in flight before the first reduction.
// TILE: one scale for the whole 128 x 128 block, else one per row.
// Needs x rows on 16 bytes and code rows on 8 bytes, both with unit stride.
template <int T, bool TILE>
__global__ void __launch_bounds__(Q_THREADS) quantize_vec_kernel(const QuantParams p) {
    const int lane16 = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const long long kb = blockIdx.x % p.kblocks, rb = blockIdx.x / p.kblocks;
    const long long col = kb * 128 + lane16 * 8, row0 = rb * Q_ROWS;
    const int left = static_cast<int>(max(0ll, min(8ll, p.K - col)));  // elements of this lane that exist
    constexpr int W = T == T_F32 ? 2 : 1;                               // 16-byte words per 8 elements
    uint4 raw[Q_PER][W];
    float m[Q_PER];
#pragma unroll
    for (int i = 0; i < Q_PER; ++i) {
        const long long r = row0 + grp + i * (Q_THREADS / 16);
#pragma unroll
        for (int w = 0; w < W; ++w) raw[i][w] = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.M && left > 0) {
            const char* src = static_cast<const char*>(p.x) + (r * p.x_rs + col) * (T == T_F32 ? 4 : 2);
            if (left == 8) {
#pragma unroll
                for (int w = 0; w < W; ++w) raw[i][w] = __ldg(reinterpret_cast<const uint4*>(src) + w);
            } else {  // ragged last block: element by element
                uint32_t tmp[4 * W];
#pragma unroll
                for (int w = 0; w < 4 * W; ++w) tmp[w] = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) {
                        if (T == T_F32)
                            tmp[e] = reinterpret_cast<const uint32_t*>(src)[e];
                        else
                            tmp[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[e]) << (16 * (e & 1));
                    }
#pragma unroll
                for (int w = 0; w < W; ++w) raw[i][w] = make_uint4(tmp[4 * w], tmp[4 * w + 1], tmp[4 * w + 2], tmp[4 * w + 3]);
            }
        }
    }
    auto values = [&](int i, float (&v)[8]) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t q[4] = {raw[i][w].x, raw[i][w].y, raw[i][w].z, raw[i][w].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (T == T_F32)
                    v[4 * w + e] = __uint_as_float(q[e]);
                else
                    unpack16<T>(q[e], v[2 * e], v[2 * e + 1]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < Q_PER; ++i) {
        float v[8];
        values(i, v);
        m[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[i] = amax_finite(m[i], v[e]);
    }
    if (TILE) {
#pragma unroll
        for (int i = 1; i < Q_PER; ++i) m[0] = fmaxf(m[0], m[i]);
        m[0] = cta_max(m[0]);
#pragma unroll
        for (int i = 1; i < Q_PER; ++i) m[i] = m[0];
    } else {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < Q_PER; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    }
    float scale, inv;
    if (TILE) {
        block_scale(p, m[0], scale, inv);
        if (threadIdx.x == 0) p.scales[rb * p.s_rs + kb * p.s_cs] = scale;
    }
#pragma unroll
    for (int i = 0; i < Q_PER; ++i) {
        const long long r = row0 + grp + i * (Q_THREADS / 16);
        if (r >= p.M) continue;
        if (!TILE) {
            block_scale(p, m[i], scale, inv);
            if (lane16 == 0) p.scales[r * p.s_rs + kb * p.s_cs] = scale;
        }
        if (left <= 0) continue;
        float v[8];
        values(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = finite_or_nan(v[e]) * inv;
        const uint32_t lo = cvt_f8x2(v[0], v[1], p.e5m2) | cvt_f8x2(v[2], v[3], p.e5m2) << 16;
        const uint32_t hi = cvt_f8x2(v[4], v[5], p.e5m2) | cvt_f8x2(v[6], v[7], p.e5m2) << 16;
        uint8_t* dst = p.codes + r * p.c_rs + col;
        if (left == 8) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) dst[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
    }
}

// Any strides and alignment: a warp takes a row's 128 columns, four elements
// 32 apart per lane, so unit-stride rows are still read and written in whole
// sectors.  TILE: the CTA's 8 warps walk the tile's 128 rows twice (largest
// value, then codes; the second read comes from the caches).
template <int T, bool TILE>
__global__ void __launch_bounds__(Q_THREADS) quantize_any_kernel(const QuantParams p) {
    constexpr int WARPS = Q_THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const long long kb = blockIdx.x % p.kblocks, rb = blockIdx.x / p.kblocks;
    const long long col0 = kb * 128 + lane, row0 = rb * Q_ROWS;
    float scale = 0.f, inv = 0.f;
    if (TILE) {
        float m = 0.f;
        for (int i = warp; i < Q_ROWS; i += WARPS) {
            const long long r = row0 + i;
            if (r >= p.M) break;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col0 + 32 * e < p.K) m = amax_finite(m, load_elem<T>(p.x, r * p.x_rs + (col0 + 32 * e) * p.x_cs));
        }
        m = cta_max(m);
        block_scale(p, m, scale, inv);
        if (threadIdx.x == 0) p.scales[rb * p.s_rs + kb * p.s_cs] = scale;
    }
#pragma unroll 4
    for (int i = warp; i < Q_ROWS; i += WARPS) {
        const long long r = row0 + i;
        if (r >= p.M) break;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = col0 + 32 * e < p.K ? load_elem<T>(p.x, r * p.x_rs + (col0 + 32 * e) * p.x_cs) : 0.f;
        if (!TILE) {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = amax_finite(m, v[e]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            block_scale(p, m, scale, inv);
            if (lane == 0) p.scales[r * p.s_rs + kb * p.s_cs] = scale;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col0 + 32 * e < p.K)
                p.codes[r * p.c_rs + (col0 + 32 * e) * p.c_cs] =
                    static_cast<uint8_t>(cvt_f8x2(finite_or_nan(v[e]) * inv, 0.f, p.e5m2));
    }
}

// Copy of a rows x cols matrix of E-byte elements with any strides into rows
// of `pitch` elements (a multiple of 16 bytes) on a 16-byte base.
template <typename E>
__global__ void __launch_bounds__(256) repack_kernel(const E* __restrict__ src, long long rs, long long cs,
                                                     E* __restrict__ dst, long long pitch, long long rows,
                                                     long long cols) {
    // 32 x 32 tiles through shared memory: reads run along the source's
    // unit-stride dimension, writes along the destination's rows
    __shared__ E tile[32][33];
    const long long tiles_c = (cols + 31) / 32, tiles = tiles_c * ((rows + 31) / 32);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const bool by_col = rs == 1 && cs != 1;  // the source's rows are its unit-stride dimension
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

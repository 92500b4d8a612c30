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
    float fmax, rfmax;         // largest code (448 or 57344) and its reciprocal in fp32
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

constexpr float INF = __builtin_huge_valf();
// the larger of m and |v|, over finite v
__device__ __forceinline__ float amax_finite(float m, float v) {
    return fabsf(v) < INF ? fmaxf(m, fabsf(v)) : m;
}
// an infinity has no code of its own: it becomes NaN, like a NaN
__device__ __forceinline__ float finite_or_nan(float v) {
    return fabsf(v) < INF ? v : __int_as_float(0x7FFFFFFF);
}

// Scale and reciprocal of a block.  Power of two: FMAX is 1.75 * 2^n, so the
// smallest 2^p with amax <= 2^p * FMAX follows from amax's exponent and from
// whether its mantissa is above 1.75; both factors are exact.  Otherwise
// scale = amax * (1 / FMAX) and the codes are x * (FMAX * (1 / amax)), every
// operation in fp32, rounded to nearest.
__device__ __forceinline__ void block_scale(const QuantParams& p, float amax, float& scale, float& inv) {
    amax = fmaxf(amax, p.fmax * __int_as_float((p.pmin + 127) << 23));
    if (p.pow2) {
        const uint32_t b = __float_as_uint(amax);
        const int e = static_cast<int>(b >> 23) - 127 - (p.e5m2 ? 15 : 8) + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        scale = __int_as_float((e + 127) << 23);
        inv = __int_as_float((127 - e) << 23);
    } else {
        scale = amax * p.rfmax;
        inv = __frcp_rn(amax) * p.fmax;
    }
}

constexpr int Q_THREADS = 256;
constexpr int Q_TILE = 128;  // rows of a tile of scales
constexpr int Q_ROWS = 64;   // rows per CTA with a scale per row

// largest value over the CTA (every thread gets it)
__device__ __forceinline__ float cta_max(float v) {
    __shared__ float part[Q_THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();  // the last round's values have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < Q_THREADS / 32; ++i) v = fmaxf(v, part[i]);
    return v;
}

// One CTA quantises R rows x one 128-column block; 8 lanes share a row, 16
// consecutive elements each, and a thread holds its rows in registers, so x is
// read once and every load is in flight before the first reduction.  Bound by
// memory, with instructions close behind: 16-bit maxima are taken on pairs, as
// integers (magnitudes order like their bits), which keeps them to about six
// per element.
// TILE: one scale for the whole 128 x 128 block, else one per row.
// Needs x and codes of unit stride, with code rows on 16 bytes.
// SHIFT: rows of x start anywhere; a lane reads the 16-byte granules around its
// elements, as far as they lie within x, and shifts them into place.
// Shifted f32 tiles hold 144 words of x for a moment: two CTAs per SM (three
// spill: 16384 x 4096 70 us against 73, 1537 x 5003 13.2 against 10.9).
template <int T, bool TILE, bool SHIFT>
__global__ void __launch_bounds__(Q_THREADS, !TILE ? 4 : SHIFT && T == T_F32 ? 2 : 3)
    quantize_vec_kernel(const __grid_constant__ QuantParams p) {
    constexpr int GROUPS = Q_THREADS / 8, R = TILE ? Q_TILE : Q_ROWS, PER = R / GROUPS;
    constexpr int E = T == T_F32 ? 4 : 2, W = E;  // bytes per element; granules of 16 bytes per 16 elements
    const int lane8 = threadIdx.x & 7, grp = threadIdx.x >> 3;
    const unsigned kb = blockIdx.x % p.kblocks, rb = blockIdx.x / p.kblocks;
    const long long col = static_cast<long long>(kb) * 128 + lane8 * 16;
    const long long row = static_cast<long long>(rb) * R + grp;         // this thread's first row
    const int left = static_cast<int>(max(0ll, min(16ll, p.K - col)));  // elements of this lane that exist
    const int rows = static_cast<int>(max(0ll, min(static_cast<long long>(PER), (p.M - row + GROUPS - 1) / GROUPS)));
    const char* src = static_cast<const char*>(p.x) + (row * p.x_rs + col) * E;
    const long long step = GROUPS * p.x_rs * E;
    grid_wait();
    grid_release();
    uint32_t raw[PER][4 * W];
    auto by_element = [&](int i) {
#pragma unroll
        for (int w = 0; w < 4 * W; ++w) raw[i][w] = 0u;
        const char* at = src + i * step;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < left) {
                if constexpr (T == T_F32)
                    raw[i][e] = reinterpret_cast<const uint32_t*>(at)[e];
                else
                    raw[i][e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[e]) << (16 * (e & 1));
            }
    };
    if constexpr (SHIFT) {
        uint32_t g[PER][4 * W + 4];
        uint32_t off[PER];
        bool whole[PER];
        const char* const x = static_cast<const char*>(p.x);
        const char* const end = x + ((p.M - 1) * p.x_rs + p.K) * E;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const char* at = src + i * step;
            off[i] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
            at -= off[i];
            whole[i] = i < rows && left == 16 && at >= x && at + 16 * W + (off[i] ? 16 : 0) <= end;
#pragma unroll
            for (int w = 0; w <= W; ++w) {
                const uint4 q = load16_if(at + 16 * w, whole[i] && (w < W || off[i]));
                g[i][4 * w] = q.x;
                g[i][4 * w + 1] = q.y;
                g[i][4 * w + 2] = q.z;
                g[i][4 * w + 3] = q.w;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            shift_granules<W>(g[i], off[i], raw[i]);
            if (!whole[i] && i < rows) by_element(i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
#pragma unroll
            for (int w = 0; w < 4 * W; ++w) raw[i][w] = 0u;
            if (i < rows && left > 0) {
                if (left == 16) {
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint4 q = reinterpret_cast<const uint4*>(src + i * step)[w];
                        raw[i][4 * w] = q.x;
                        raw[i][4 * w + 1] = q.y;
                        raw[i][4 * w + 2] = q.z;
                        raw[i][4 * w + 3] = q.w;
                    }
                } else {  // ragged last block
                    by_element(i);
                }
            }
        }
    }
    auto value = [&](int i, int e) {
        if constexpr (T == T_F32) {
            return __uint_as_float(raw[i][e]);
        } else {
            float lo, hi;
            unpack16<T>(raw[i][e / 2], lo, hi);
            return (e & 1) ? hi : lo;
        }
    };
    // largest magnitudes.  f32: the hardware maximum passes over NaN.  16-bit:
    // as integers, infinity and NaN are the largest; either way a block that
    // is not all finite shows as one at least INF or NaN, and is done again.
    float m[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (T == T_F32) {
            m[i] = fabsf(value(i, 0));
#pragma unroll
            for (int e = 1; e < 16; ++e) m[i] = fmaxf(m[i], fabsf(value(i, e)));
        } else {
            uint32_t two = raw[i][0] & 0x7FFF7FFFu;
#pragma unroll
            for (int w = 1; w < 8; ++w) two = max_u16x2(two, raw[i][w] & 0x7FFF7FFFu);
            two = max(two & 0xFFFFu, two >> 16);
            m[i] = T == T_F16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(two))) : __uint_as_float(two << 16);
        }
    }
    auto reduce = [&]() {
        if (TILE) {
#pragma unroll
            for (int i = 1; i < PER; ++i) m[0] = fmaxf(m[0], m[i]);
            m[0] = cta_max(m[0]);
        } else {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < PER; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
        }
    };
    bool odd = false;  // something is not finite
#pragma unroll
    for (int i = 0; i < PER; ++i) odd = odd || !(m[i] < INF);
    odd = TILE ? __syncthreads_or(odd) : __any_sync(0xFFFFFFFFu, odd);
    if (odd) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            m[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) m[i] = amax_finite(m[i], value(i, e));
        }
    }
    reduce();
    float scale, inv;
    if (TILE) {
        block_scale(p, m[0], scale, inv);
        if (threadIdx.x == 0) p.scales[rb * p.s_rs + kb * p.s_cs] = scale;
    }
    uint8_t* dst = p.codes + row * p.c_rs + col;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i >= rows) break;
        if (!TILE) {
            block_scale(p, m[i], scale, inv);
            if (lane8 == 0) p.scales[(row + GROUPS * i) * p.s_rs + kb * p.s_cs] = scale;
        }
        if (left <= 0) continue;
        uint32_t out[4];
        auto encode = [&](auto fix, int e5m2) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                out[w] = cvt_f8x2(fix(value(i, 4 * w)) * inv, fix(value(i, 4 * w + 1)) * inv, e5m2) |
                         cvt_f8x2(fix(value(i, 4 * w + 2)) * inv, fix(value(i, 4 * w + 3)) * inv, e5m2) << 16;
        };
        if (odd)
            encode([](float v) { return finite_or_nan(v); }, p.e5m2);
        else if (p.e5m2)
            encode([](float v) { return v; }, 1);
        else
            encode([](float v) { return v; }, 0);
        uint8_t* to = dst + GROUPS * i * p.c_rs;
        if (left == 16) {
            *reinterpret_cast<uint4*>(to) = make_uint4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < left) to[e] = static_cast<uint8_t>(out[e / 4] >> (8 * (e & 3)));
        }
    }
}

// Any strides and alignment: a warp takes rows of 128 columns, four elements 32
// apart per lane, so unit-stride rows are still read and written in whole
// sectors; four rows at a time, so that 16 loads per lane are in flight.
// TILE: the CTA's warps walk the tile's rows twice (largest value, then codes;
// the second read comes from the caches).
template <int T, bool TILE>
__global__ void __launch_bounds__(Q_THREADS) quantize_any_kernel(const __grid_constant__ QuantParams p) {
    constexpr int R = TILE ? Q_TILE : Q_ROWS, WARPS = Q_THREADS / 32, PER = R / WARPS, U = 4;
    constexpr int E = T == T_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const unsigned kb = blockIdx.x % p.kblocks, rb = blockIdx.x / p.kblocks;
    const long long col = static_cast<long long>(kb) * 128 + lane, row = static_cast<long long>(rb) * R + warp;
    const char* const x0 = static_cast<const char*>(p.x) + (row * p.x_rs + col * p.x_cs) * E;
    uint8_t* const c0 = p.codes + row * p.c_rs + col * p.c_cs;
    const long long x_row = p.x_rs * WARPS * E, x_col = p.x_cs * 32 * E, c_row = p.c_rs * WARPS, c_col = p.c_cs * 32;
    const int rows = static_cast<int>(max(0ll, min(static_cast<long long>(PER), (p.M - row + WARPS - 1) / WARPS)));
    grid_wait();
    grid_release();
    bool there[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) there[e] = col + 32 * e < p.K;
    auto load = [&](int i, float (&v)[U][4]) {  // rows i .. i + U - 1 of this warp
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const char* at = x0 + (i + j) * x_row;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[j][e] = i + j < rows && there[e] ? load_elem<T>(at, 0) : 0.f;
                at += x_col;
            }
        }
    };
    float scale = 0.f, inv = 0.f;
    if (TILE) {
        float m = 0.f;
#pragma unroll 1
        for (int i = 0; i < PER; i += U) {
            float v[U][4];
            load(i, v);
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = amax_finite(m, v[j][e]);
        }
        m = cta_max(m);
        block_scale(p, m, scale, inv);
        if (threadIdx.x == 0) p.scales[rb * p.s_rs + kb * p.s_cs] = scale;
    }
#pragma unroll 1
    for (int i = 0; i < rows; i += U) {
        float v[U][4];
        load(i, v);
        float m[U];
        if (!TILE) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                m[j] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) m[j] = amax_finite(m[j], v[j][e]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < U; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (i + j >= rows) break;
            if (!TILE) {
                block_scale(p, m[j], scale, inv);
                if (lane == 0) p.scales[(row + (i + j) * WARPS) * p.s_rs + kb * p.s_cs] = scale;
            }
            uint8_t* to = c0 + (i + j) * c_row;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const uint32_t two = cvt_f8x2(finite_or_nan(v[j][e]) * inv, finite_or_nan(v[j][e + 1]) * inv, p.e5m2);
                if (there[e]) to[0] = static_cast<uint8_t>(two);
                if (there[e + 1]) to[c_col] = static_cast<uint8_t>(two >> 8);
                to += 2 * c_col;
            }
        }
    }
}

// Copy of `rows` rows of unit-stride bytes, any distance apart, into rows of
// `pitch` bytes (a multiple of 16) on a 16-byte base; the last granule's bytes
// past a row's end are whatever follows there.  Bound by memory: a lane reads
// the two granules of 16 bytes around its source (the second is a neighbour's
// first, so it comes from the L1 cache), shifts and writes one; four rows are
// under way per thread.  Near the matrix's ends, byte by byte.
constexpr int COPY_ROWS = 32;  // rows of a CTA's tile: 8 warps x 4; columns: 32 granules
__global__ void __launch_bounds__(256) repack_rows_kernel(const uint8_t* src, long long rs, uint8_t* dst, long long pitch,
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

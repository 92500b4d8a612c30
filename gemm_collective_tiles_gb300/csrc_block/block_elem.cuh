// Dropout with its residual, and the gradient of an epilogue: the activation's
// derivative, the dropped gradients and the bias gradient in one pass.
//
// Both are bound by memory.  A warp takes 256 columns of a row, in one of two
// layouts: 8 neighbouring columns a lane where rows lie on 16 bytes (one or two
// 16-byte accesses), else column lane + 32 e, so that any strides serve and
// elements of unit stride still make whole sectors.  Either way a lane computes
// the random bits of its own 8 columns once; in the second layout the warp hands
// them round as bytes of keep bits.  Measured: dropout of 16384 x 4096 bf16 with its
// residual 57.6 us (7.0 TB/s, with what stays in L2), without 45; 1537 x 5003 f32
// (second layout) 17; act_grad of 4096 x 14336 bf16 with gelu and bias 72 us (4.9
// TB/s: loads of two rows under way a warp, 78 registers).
#pragma once
#include "act.cuh"

namespace gct {
namespace block {

using namespace gct::fp8;

constexpr int SEG = 256;  // columns of a warp's piece of a row

struct Mat {
    const void* data;
    long long rs, cs;
};
struct DropParams {
    Mat x, residual, out;
    long long M;
    int N, type;
    unsigned segs;         // pieces of a row
    long long row_step;    // rows that the grid takes at once
    Drop drop;
};
struct ActGradParams {
    Mat dy, z, dz;
    long long M;
    int N, type, dz_type, act;
    unsigned segs;
    int rows;        // of a CTA
    float* sums;     // (row block, N): column sums of dz, or null
    Drop drop;
};
struct ColumnSumParams {
    const float* sums;
    int blocks, N;
    void* out;
    int type;
};

template <int T>
struct Raw {
    uint4 q[T == T_F32 ? 2 : 1];
};
// 8 neighbouring elements on 16 bytes
template <int T>
__device__ __forceinline__ Raw<T> load8(const void* p, long long i) {
    Raw<T> r;
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (T == T_F32 ? 4 : 2));
    r.q[0] = at[0];
    if (T == T_F32) r.q[T == T_F32 ? 1 : 0] = at[1];
    return r;
}
template <int T>
__device__ __forceinline__ void spread8(const Raw<T>& r, float (&v)[8]) {
    if (T == T_F32) {
        const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
        const uint4 s = r.q[T == T_F32 ? 1 : 0];
        const uint32_t x[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(w[e]);
            v[4 + e] = __uint_as_float(x[e]);
        }
    } else {
        const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack16<T>(w[e], v[2 * e], v[2 * e + 1]);
    }
}
__device__ __forceinline__ void store8(void* p, int type, long long i, const float (&v)[8]) {
    if (type == T_F32) {
        float4* at = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        at[0] = make_float4(v[0], v[1], v[2], v[3]);
        at[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    const int bf = type == T_BF16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack16(v[0], v[1], bf), pack16(v[2], v[3], bf), pack16(v[4], v[5], bf), pack16(v[6], v[7], bf));
}

// column of element e of a lane
template <bool VEC>
__device__ __forceinline__ int column(unsigned seg, int lane, int e) {
    return seg * SEG + (VEC ? lane * 8 + e : e * 32 + lane);
}
// 8 elements of a row's piece as they were loaded, zeros past its end
template <int T, bool VEC>
struct Piece {
    Raw<T> raw;
    float v[VEC ? 1 : 8];
    __device__ __forceinline__ void load(const Mat& m, long long row, unsigned seg, int lane, int N) {
        if constexpr (VEC) {
            const int c = column<true>(seg, lane, 0);
            if (c < N) {
                raw = load8<T>(m.data, row * m.rs + c);
            } else {
#pragma unroll
                for (uint4& q : raw.q) q = make_uint4(0u, 0u, 0u, 0u);
            }
        } else {
            const long long o = row * m.rs;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = column<false>(seg, lane, e);
                v[e] = c < N ? load_elem<T>(m.data, o + c * m.cs) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void spread(float (&x)[8]) const {
        if constexpr (VEC) {
            spread8<T>(raw, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = v[e];
        }
    }
};
template <bool VEC>
__device__ __forceinline__ void store_piece(const Mat& m, int type, long long row, unsigned seg, int lane, int N, const float (&v)[8]) {
    void* const to = const_cast<void*>(m.data);
    if constexpr (VEC) {
        const int c = column<true>(seg, lane, 0);
        if (c < N) store8(to, type, row * m.rs + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false>(seg, lane, e);
            if (c < N) store_any(to, type, row * m.rs + c * m.cs, v[e]);
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void drop_piece(float (&v)[8], const Drop& d, const DropKey& key, long long row, unsigned seg, int lane) {
    const uint32_t group = seg * (SEG / 8) + lane;
    if constexpr (VEC) {
        drop8(v, d, key, group, static_cast<uint32_t>(row));
    } else {
        uint32_t w[4], keep = 0;
        philox8(key, group, static_cast<uint32_t>(row), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) keep |= static_cast<uint32_t>(kept(w, e, d)) << e;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t bits = __shfl_sync(0xFFFFFFFFu, keep, e * 4 + (lane >> 3));
            v[e] = (bits >> (lane & 7) & 1u) ? v[e] * d.scale : 0.f;
        }
    }
}

template <int T, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropParams p) {
    const int lane = threadIdx.x & 31;
    grid_wait();
    grid_release();
    const DropKey key = drop_key(p.drop);
    const unsigned seg = blockIdx.x % p.segs;
    for (long long row = blockIdx.x / p.segs * 8 + (threadIdx.x >> 5); row < p.M; row += p.row_step) {
        Piece<T, VEC> x, res;
        x.load(p.x, row, seg, lane, p.N);
        if (p.residual.data) res.load(p.residual, row, seg, lane, p.N);
        float v[8];
        x.spread(v);
        if (p.drop.least) drop_piece<VEC>(v, p.drop, key, row, seg, lane);
        if (p.residual.data) {
            float r[8];
            res.spread(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
        store_piece<VEC>(p.out, T, row, seg, lane, p.N, v);
    }
}

template <int T, bool VEC>
__global__ void __launch_bounds__(256) act_grad_kernel(const __grid_constant__ ActGradParams p) {
    __shared__ float part[8][SEG];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_wait();
    grid_release();
    const DropKey key = drop_key(p.drop);
    const unsigned seg = blockIdx.x % p.segs, block = blockIdx.x / p.segs;
    const long long first = static_cast<long long>(block) * p.rows, end = min(p.M, first + p.rows);
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    // the loads of U rows are under way at once
    constexpr int U = 2;
    const bool act = p.act != ACT_NONE;
    for (long long row = first + warp; row < end; row += 8 * U) {
        Piece<T, VEC> g[U], z[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (row + 8 * k < end) {
                g[k].load(p.dy, row + 8 * k, seg, lane, p.N);
                if (act) z[k].load(p.z, row + 8 * k, seg, lane, p.N);
            }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (row + 8 * k >= end) break;
            float v[8];
            g[k].spread(v);
            if (p.drop.least) drop_piece<VEC>(v, p.drop, key, row + 8 * k, seg, lane);
            if (act) {
                float w[8];
                z[k].spread(w);
                apply_act_grad(v, w, p.act);
            }
            if (p.dz.data) store_piece<VEC>(p.dz, p.dz_type, row + 8 * k, seg, lane, p.N, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[e];
        }
    }
    if (!p.sums) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][column<VEC>(0, lane, e)] = sum[e];
    __syncthreads();
    const int c = threadIdx.x;
    float s = part[0][c];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += part[w][c];
    if (seg * SEG + c < p.N) p.sums[static_cast<long long>(block) * p.N + seg * SEG + c] = s;
}

// Columns of (blocks, N) added up in a fixed order: 32 columns a CTA, 8 warps
// take every 8th block.
template <int DUMMY>
__global__ void __launch_bounds__(256) column_sum_kernel(const __grid_constant__ ColumnSumParams p) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_wait();
    grid_release();
    float s = 0.f;
    if (c < p.N) {
#pragma unroll 4
        for (int b = warp; b < p.blocks; b += 8) s += p.sums[static_cast<long long>(b) * p.N + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.N) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += part[w][lane];
        store_any(p.out, p.type, c, s);
    }
}

}  // namespace block
}  // namespace gct

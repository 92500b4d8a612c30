// The norms around a block's end, its gate and its residual, and their gradient.
//
//   u = N_post(y) or y,   h = x + scale * gate * u,   n = N_pre(h)
//   N(v) = w (v - m) r + b,  r = 1 / sqrt(mean((v - m)^2) + eps),  m = mean(v) ("layer") or 0 ("rms")
//
// Gradient, with g = dn w and a hat for a normalised value:
//   dH = dh + r (g - hhat mean(g hhat) - [layer] mean(g));   dx = dH
//   du = dH scale gate;  dy = the same of N_post, of du;   dgate = sum dH scale u
//   dw = sum dn hhat, db = sum dn over the rows, of both norms
//
// Bound by memory: a row's pieces stay in registers between the reductions (two
// passes over them for a variance), so every tensor is read and written once; h
// enters the second norm unrounded, and the gradient computes it again from x
// and y instead of reading it back rounded.
//
// T threads take a row, 8 C elements a thread: neighbouring ones where all rows
// lie on 16 bytes (VEC), else one in T, so that any strides serve and elements
// of unit stride still make whole sectors.  Rows longer than that are gone over
// once per reduction.
#pragma once
#include "block_elem.cuh"

namespace gct {
namespace block {

enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
constexpr int NORM_MAX_T = 512, NORM_MAX_C = 4;
constexpr int NORM_LONGEST = NORM_MAX_T * NORM_MAX_C * 8;  // elements of a row in registers
constexpr int NORM_GRAD_C = 2;                             // of the gradient, whose long rows are shared by a cluster

struct Vec {
    const void* data;
    int type;
};
struct NormParams {
    Mat y, x, gate, h, n;
    Vec post_w, post_b, pre_w, pre_b;
    int gate_type;
    long long M, group_rows;  // rows of y per row of gate
    int D, post, pre;
    float scale, eps;
    float4* stats;            // per row: mean and r of y, mean and r of h; may be absent
    // shared memory of a row's threads: the places of post_w, post_b, pre_w, pre_b and
    // gate there (-1: not kept), their bytes, the bytes of a row, rows ahead
    int vec_at[5];
    unsigned vec_bytes, row_bytes;
    int depth;
};
struct NormGradParams {
    NormParams f;             // h and n unused; stats read
    Mat dh, dn, dy, dx, dgate;
    // Sums over the rows that a CTA keeps for itself: which of dpre_w, dpre_b,
    // dpost_w, dpost_b are wanted, by slot (-1: not)
    int slot[4], slots;
    int gate_sums;            // dgate is a sum over rows
    int parts;                // CTAs of a cluster that share a row
    float* part;              // (CTA, slot, D)
    float* gate_part;         // (CTA, 2, D): a group begun before, a group that goes on
    long long ctas;
};
struct NormFinishParams {
    const float* part;
    int ctas, slots, D;
    void* out[4];
    int type[4];
    const float* gate_part;
    Mat dgate;
    int gate_type;
    long long M, group_rows, groups;
};

// first row of CTA c
__host__ __device__ __forceinline__ long long norm_row(long long M, long long ctas, long long c) { return M * c / ctas; }

// column of a thread's element i, in the CTA's part of the row
template <bool VEC>
__device__ __forceinline__ int norm_column(int T, int t, int i) {
    return VEC ? ((i >> 3) * T + t) * 8 + (i & 7) : i * T + t;
}
template <int TYPE, bool VEC, int C>
__device__ __forceinline__ void load_row(const Mat& m, long long row, int T, int t, int base, int D, float (&v)[8 * C]) {
    const long long o = row * m.rs;
    if constexpr (VEC) {
        Raw<TYPE> raw[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (base + norm_column<true>(T, t, 8 * c) < D) raw[c] = load8<TYPE>(m.data, o + base + norm_column<true>(T, t, 8 * c));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            if (base + norm_column<true>(T, t, 8 * c) < D) {
                spread8<TYPE>(raw[c], w);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * c + e] = w[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            const int c = base + norm_column<false>(T, t, i);
            v[i] = c < D ? load_elem<TYPE>(m.data, o + c * m.cs) : 0.f;
        }
    }
}
template <bool VEC, int C>
__device__ __forceinline__ void store_row(const Mat& m, int type, long long row, int T, int t, int base, int D,
                                          const float (&v)[8 * C]) {
    void* const to = const_cast<void*>(m.data);
    const long long o = row * m.rs;
    if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = base + norm_column<true>(T, t, 8 * c);
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = v[8 * c + e];
            if (at < D) store8(to, type, o + at, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            const int c = base + norm_column<false>(T, t, i);
            if (c < D) store_any(to, type, o + c * m.cs, v[i]);
        }
    }
}
// f(i, value) for this thread's elements of a vector or of a row of gate
template <bool VEC, int C, typename F>
__device__ __forceinline__ void with_vector(const void* data, int type, long long o, long long cs, int T, int t, int base, int D, F f) {
    if (!data) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (VEC) {
            const int at = base + norm_column<true>(T, t, 8 * c);
            if (at >= D) continue;
            float w[8];
            if (type == T_F32)
                spread8<T_F32>(load8<T_F32>(data, o + at), w);
            else if (type == T_F16)
                spread8<T_F16>(load8<T_F16>(data, o + at), w);
            else
                spread8<T_BF16>(load8<T_BF16>(data, o + at), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(8 * c + e, w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = base + norm_column<false>(T, t, 8 * c + e);
                if (at < D) f(8 * c + e, load_any(data, type, o + at * cs));
            }
        }
    }
}
// Sums of one or two values over a row's T threads (a whole number of warps, 16
// at most).  `turn` alternates between two buffers, so that one barrier a
// reduction is enough; every warp adds the warps' sums up for itself.
template <bool TWO>
__device__ __forceinline__ float2 row_sum(float a, float b, int T, int t, float2 (*buffer)[16], int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (TWO) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (T == 32) return make_float2(a, b);
    if ((t & 31) == 0) buffer[turn][t >> 5] = make_float2(a, b);
    __syncthreads();
    const int w = t & 15;
    float2 s = buffer[turn][w];
    if (w * 32 >= T) s = make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
        if (TWO) s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
    }
    turn ^= 1;
    return s;
}
// Mean and r of the values; those past the row's end are 0 and left out.
template <bool VEC, int C>
__device__ __forceinline__ float2 row_stats(const float (&v)[8 * C], int kind, float eps, float over_d, int T, int t, int D,
                                            float2 (*buffer)[16], int& turn) {
    float s = 0.f;
    if (kind == NORM_RMS) {
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) s = fmaf(v[i], v[i], s);
        return make_float2(0.f, rsqrtf(fmaf(row_sum<false>(s, 0.f, T, t, buffer, turn).x, over_d, eps)));
    }
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) s += v[i];
    const float mean = row_sum<false>(s, 0.f, T, t, buffer, turn).x * over_d;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) {
        const float d = norm_column<VEC>(T, t, VEC ? i & ~7 : i) < D ? v[i] - mean : 0.f;
        s = fmaf(d, d, s);
    }
    return make_float2(mean, rsqrtf(fmaf(row_sum<false>(s, 0.f, T, t, buffer, turn).x, over_d, eps)));
}

__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest `left` groups of this thread have landed
__device__ __forceinline__ void copies_wait(int left) {
    if (left <= 0)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (left == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 3;" ::: "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ void shared16(uint32_t at, const uint4& q) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
// 8 elements of a piece in shared memory, whose second 16 bytes (f32) lie `apart` further on
template <int TYPE>
__device__ __forceinline__ void shared8(uint32_t at, uint32_t apart, float (&w)[8]) {
    Raw<TYPE> raw;
    raw.q[0] = shared16(at);
    if (TYPE == T_F32) raw.q[TYPE == T_F32 ? 1 : 0] = shared16(at + apart);
    spread8<TYPE>(raw, w);
}

// One of the tensors whose rows come ahead: where this thread's next piece lies,
// and the bytes to the row after.  `type` decides the pieces' size.
struct Ahead {
    const char* at;
    long long step;
    int pieces;  // of 16 bytes per 8 elements; 0: not there
    __device__ __forceinline__ void start(const Mat& m, int type, long long row, int col) {
        const int elem = type == T_F32 ? 4 : 2;
        pieces = m.data ? elem / 2 : 0;
        at = static_cast<const char*>(m.data) + (row * m.rs + col) * elem;
        step = m.rs * elem;
    }
};

// The threads of a row, and the shared memory that each of them has to itself:
// its elements of the vectors, in fp32, and its pieces of the next rows, which it
// copies asynchronously.  No barrier stands between a copy and its use, and the
// copies run under the reductions of the rows before.
template <bool VEC, int C>
struct RowThreads {
    int T, t, base, D;     // base: first column of the CTA's part of the row
    uint32_t cache, ring;  // this thread's
    uint32_t bytes;        // of a row ahead
    int depth, slot, left; // rows ahead (0: none), the next one's place, rows not yet copied

    __device__ __forceinline__ uint32_t apart() const { return T * 16; }
    __device__ __forceinline__ bool chunk_there(int c) const { return base + norm_column<true>(T, t, 8 * c) < D; }
    __device__ __forceinline__ bool there(int i) const { return base + norm_column<VEC>(T, t, VEC ? i & ~7 : i) < D; }
    // a vector, or a gate's row, into shared memory; zeros past its end
    __device__ __forceinline__ void keep(int slot, const void* data, int type, long long o, long long cs) const {
        if (!data || slot < 0) return;
        const uint32_t to = cache + slot * (2 * C) * apart();
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = base + norm_column<VEC>(T, t, 4 * j + e);
                w[e] = at < D ? load_any(data, type, o + at * cs) : 0.f;
            }
            shared16(to + j * apart(), make_uint4(__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]), __float_as_uint(w[3])));
        }
    }
    // f(i, value) for this thread's elements of a vector or a gate's row
    template <typename F>
    __device__ __forceinline__ void each(int slot, const void* data, int type, long long o, long long cs, F f) const {
        if (!data) return;
        if (slot < 0) {
            with_vector<VEC, C>(data, type, o, cs, T, t, base, D, f);
            return;
        }
        const uint32_t from = cache + slot * (2 * C) * apart();
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
            const uint4 q = shared16(from + j * apart());
            f(4 * j, __uint_as_float(q.x));
            f(4 * j + 1, __uint_as_float(q.y));
            f(4 * j + 2, __uint_as_float(q.z));
            f(4 * j + 3, __uint_as_float(q.w));
        }
    }
    // threads past a row's end find zeros
    __device__ __forceinline__ void clear() const {
        if constexpr (VEC) {
            bool all = true;
#pragma unroll
            for (int c = 0; c < C; ++c) all = all && chunk_there(c);
            if (!all)
                for (uint32_t at = 0; at < depth * bytes; at += apart()) shared16(ring + at, make_uint4(0u, 0u, 0u, 0u));
        }
    }
    // a row of N tensors on its way
    template <int N>
    __device__ __forceinline__ void issue(Ahead (&a)[N]) {
        if (left > 0) {
            uint32_t to = ring + slot * bytes;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (a[k].pieces) {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if (chunk_there(c)) {
                            const char* from = a[k].at + static_cast<long long>(c) * T * 16 * a[k].pieces;
                            copy16_async(to, from);
                            if (a[k].pieces == 2) copy16_async(to + apart(), from + 16);
                        }
                        to += a[k].pieces * apart();
                    }
                    a[k].at += a[k].step;
                }
            }
        }
        --left;
        copies_commit();
        slot = slot + 1 == depth ? 0 : slot + 1;
    }
    template <int TYPE>
    __device__ __forceinline__ void take(uint32_t& from, const Mat& m, float (&v)[8 * C]) const {
        if (!m.data) return;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            shared8<TYPE>(from, apart(), w);
            from += (TYPE == T_F32 ? 2 : 1) * apart();
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * c + e] = w[e];
        }
    }
};
// the gate's row for a row of y, kept up row by row
struct GateRow {
    long long row, left, rows;
    __device__ __forceinline__ GateRow(long long first, long long group_rows) : row(first / group_rows), rows(group_rows) {
        left = (row + 1) * group_rows - first;
    }
    __device__ __forceinline__ void next() {
        if (--left == 0) {
            ++row;
            left = rows;
        }
    }
};
// this thread's pieces of a row: a pointer that moves on by rows, or any strides
template <bool VEC, int C>
struct Output {
    char* at;
    long long step;
    __device__ __forceinline__ Output(const Mat& m, int type, long long row, int col) {
        const int elem = type == T_F32 ? 4 : 2;
        at = const_cast<char*>(static_cast<const char*>(m.data)) + (row * m.rs + col) * elem;
        step = m.rs * elem;
    }
    template <int TYPE>
    __device__ __forceinline__ void store(const RowThreads<VEC, C>& rt, const Mat& m, long long row, const float (&v)[8 * C]) {
        if constexpr (VEC) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = v[8 * c + e];
                if (rt.chunk_there(c)) store8(at, TYPE, static_cast<long long>(c) * rt.T * 8, w);
            }
            at += step;
        } else {
            store_row<false, C>(m, TYPE, row, rt.T, rt.t, rt.base, rt.D, v);
        }
    }
};

// A unit of T threads (blockDim.y of them in a CTA where T is a warp) takes
// consecutive rows.
template <int TY, int TX, bool VEC, int C>
__global__ void __launch_bounds__(NORM_MAX_T) norm_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ float4 dynamic[];
    __shared__ float2 buffer[2][16];
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    const long long units = static_cast<long long>(gridDim.x) * blockDim.y, unit = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const long long begin = norm_row(p.M, units, unit), end = norm_row(p.M, units, unit + 1);
    if (begin == end) return;
    int turn = 0;
    RowThreads<VEC, C> rt{T, t, 0, D, 0u, 0u, p.row_bytes, p.depth, 0, static_cast<int>(end - begin)};
    rt.cache = smem_u32(dynamic) + threadIdx.y * (p.vec_bytes + p.depth * p.row_bytes) + t * 16;
    rt.ring = rt.cache + p.vec_bytes;
    rt.clear();
    const bool row_gate = p.gate.data && p.group_rows == 1;
    const int col = norm_column<VEC>(T, t, 0);
    Ahead ahead[3];
    ahead[0].start(p.y, TY, begin, col);
    ahead[1].start(p.x, TX, begin, col);
    ahead[2].start(row_gate ? p.gate : Mat{nullptr, 0, 0}, p.gate_type, begin, col);
    Output<VEC, C> out_h(p.h, TX, begin, col), out_n(p.n, TY, begin, col);
    GateRow gate(begin, p.group_rows);
    float4* to_stats = p.stats + begin;
    grid_wait();
    grid_release();
    if (VEC)
        for (int i = 0; i < p.depth; ++i) rt.issue(ahead);
    rt.keep(p.vec_at[0], p.post_w.data, p.post_w.type, 0, 1);
    rt.keep(p.vec_at[1], p.post_b.data, p.post_b.type, 0, 1);
    rt.keep(p.vec_at[2], p.pre_w.data, p.pre_w.type, 0, 1);
    rt.keep(p.vec_at[3], p.pre_b.data, p.pre_b.type, 0, 1);
    long long kept_gate = -1;
    const float over_d = 1.f / D;
    for (long long row = begin; row < end; ++row) {
        float v[8 * C], x[8 * C], gv[8 * C];
        if (p.gate.data && !row_gate && gate.row != kept_gate) {
            rt.keep(p.vec_at[4], p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs);
            kept_gate = gate.row;
        }
        auto get = [&](int i, float w) { gv[i] = w; };
        if (VEC && p.depth > 0) {
            copies_wait(p.depth - 1);
            uint32_t from = rt.ring + rt.slot * rt.bytes;
            rt.template take<TY>(from, p.y, v);
            rt.template take<TX>(from, p.x, x);
            if (row_gate) {
                if (p.gate_type == T_F32)
                    rt.template take<T_F32>(from, p.gate, gv);
                else if (p.gate_type == T_F16)
                    rt.template take<T_F16>(from, p.gate, gv);
                else
                    rt.template take<T_BF16>(from, p.gate, gv);
            }
            rt.issue(ahead);
        } else {
            load_row<TY, VEC, C>(p.y, row, T, t, 0, D, v);
            if (p.x.data) load_row<TX, VEC, C>(p.x, row, T, t, 0, D, x);
            if (row_gate) with_vector<VEC, C>(p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs, T, t, 0, D, get);
        }
        float4 stats = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.post) {
            const float2 s = row_stats<VEC, C>(v, p.post, p.eps, over_d, T, t, D, buffer, turn);
            stats.x = s.x;
            stats.y = s.y;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = (v[i] - s.x) * (rt.there(i) ? s.y : 0.f);
            rt.each(p.vec_at[0], p.post_w.data, p.post_w.type, 0, 1, [&](int i, float w) { v[i] *= w; });
            rt.each(p.vec_at[1], p.post_b.data, p.post_b.type, 0, 1, [&](int i, float w) { v[i] += w; });
        }
        if (p.gate.data) {
            if (!row_gate) rt.each(p.vec_at[4], p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs, get);
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = rt.there(i) ? v[i] * gv[i] : 0.f;
        }
        if (p.x.data) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = fmaf(p.scale, v[i], x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] *= p.scale;
        }
        if (p.h.data) out_h.template store<TX>(rt, p.h, row, v);
        if (p.pre) {
            const float2 s = row_stats<VEC, C>(v, p.pre, p.eps, over_d, T, t, D, buffer, turn);
            stats.z = s.x;
            stats.w = s.y;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = (v[i] - s.x) * s.y;
            rt.each(p.vec_at[2], p.pre_w.data, p.pre_w.type, 0, 1, [&](int i, float w) { v[i] *= w; });
            rt.each(p.vec_at[3], p.pre_b.data, p.pre_b.type, 0, 1, [&](int i, float w) { v[i] += w; });
            out_n.template store<TY>(rt, p.n, row, v);
        }
        if (p.stats) {
            if (t == 0) *to_stats = stats;
            ++to_stats;
        }
        gate.next();
    }
    if (VEC) copies_wait(0);
}

// Rows of any length, read anew for each reduction: one CTA per row.
template <int TY, int TX>
__global__ void __launch_bounds__(NORM_MAX_T) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 buffer[2][16];
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    int turn = 0;
    grid_wait();
    grid_release();
    const long long row = blockIdx.x;
    float4 stats = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load_y = [&](int c) { return load_elem<TY>(p.y.data, row * p.y.rs + c * p.y.cs); };
    const long long gate_row = p.gate.data ? row / p.group_rows * p.gate.rs : 0;
    auto load_h = [&](int c) {
        float u = load_y(c);
        if (p.post) {
            u = (u - stats.x) * stats.y;
            if (p.post_w.data) u *= load_any(p.post_w.data, p.post_w.type, c);
            if (p.post_b.data) u += load_any(p.post_b.data, p.post_b.type, c);
        }
        if (p.gate.data) u *= load_any(p.gate.data, p.gate_type, gate_row + c * p.gate.cs);
        return p.x.data ? fmaf(p.scale, u, load_elem<TX>(p.x.data, row * p.x.rs + c * p.x.cs)) : p.scale * u;
    };
    auto row_stats = [&](int kind, auto value, float& mean, float& r) {
        float m = 0.f, s = 0.f;
        if (kind == NORM_LAYER) {
            for (int c = t; c < D; c += T) s += value(c);
            m = row_sum<false>(s, 0.f, T, t, buffer, turn).x / D;
        }
        s = 0.f;
        for (int c = t; c < D; c += T) {
            const float d = value(c) - m;
            s = fmaf(d, d, s);
        }
        r = rsqrtf(row_sum<false>(s, 0.f, T, t, buffer, turn).x / D + p.eps);
        mean = m;
    };
    if (p.post) {
        float m, r;
        row_stats(p.post, load_y, m, r);
        stats.x = m;
        stats.y = r;
    }
    if (p.pre) row_stats(p.pre, load_h, stats.z, stats.w);
    // h may be y or x: each element is read before it is written, by one thread
    for (int c = t; c < D; c += T) {
        const float h = load_h(c);
        if (p.h.data) store_any(const_cast<void*>(p.h.data), TX, row * p.h.rs + c * p.h.cs, h);
        if (!p.pre) continue;
        float n = (h - stats.z) * stats.w;
        if (p.pre_w.data) n *= load_any(p.pre_w.data, p.pre_w.type, c);
        if (p.pre_b.data) n += load_any(p.pre_b.data, p.pre_b.type, c);
        store_any(const_cast<void*>(p.n.data), TY, row * p.n.rs + c * p.n.cs, n);
    }
    if (p.stats && t == 0) p.stats[row] = stats;
}

// A row's sums over the CTAs of a cluster that share it, in their order.
struct Shared {
    float2 (*buffer)[16];
    float2 (*meet)[8];
    int T, t, parts, rank, turn;
    template <bool TWO>
    __device__ __forceinline__ float2 sum(float a, float b) {
        const int now = turn;
        float2 s = row_sum<TWO>(a, b, T, t, buffer, turn);
        if (parts == 1) return s;
        if (T == 32) turn ^= 1;
        if (t < parts) {
            const uint32_t to = map_to(smem_u32(&meet[now][rank]), t);
            st_shared_cluster_u32(to, __float_as_uint(s.x));
            st_shared_cluster_u32(to + 4, __float_as_uint(s.y));
        }
        cluster_sync();
        s = make_float2(0.f, 0.f);
        for (int k = 0; k < parts; ++k) {
            s.x += meet[now][k].x;
            s.y += meet[now][k].y;
        }
        return s;
    }
};

// Sums over rows: element i of a thread, in registers (8 elements a thread: 40
// numbers) or, two float4 per 8 elements, in shared memory that only it uses.
template <int C>
struct RowSums {
    float v[C == 1 ? 5 : 1][C == 1 ? 8 : 1];
    float4* at;
    int T;
    __device__ __forceinline__ void clear(int slots) {
        if constexpr (C == 1) {
#pragma unroll
            for (int s = 0; s < 5; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[s][i] = 0.f;
        } else {
            for (int s = 0; s < slots; ++s) zero(s, s);
        }
    }
    __device__ __forceinline__ void zero(int which, int slot) {
        if constexpr (C == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[which][i] = 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) at[(slot * 2 * C + j) * T] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    // `which` names the sum (a constant), `slot` its place
    __device__ __forceinline__ void add(int which, int slot, const float (&x)[8 * C]) {
        if constexpr (C == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[which][i] += x[i];
        } else {
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) {
                float4 f = at[(slot * 2 * C + j) * T];
                f.x += x[4 * j];
                f.y += x[4 * j + 1];
                f.z += x[4 * j + 2];
                f.w += x[4 * j + 3];
                at[(slot * 2 * C + j) * T] = f;
            }
        }
    }
    // of products, by fused multiply-adds
    __device__ __forceinline__ void add(int which, int slot, const float (&x)[8 * C], const float (&y)[8 * C]) {
        if constexpr (C == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[which][i] = fmaf(x[i], y[i], v[which][i]);
        } else {
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) {
                float4 f = at[(slot * 2 * C + j) * T];
                f.x = fmaf(x[4 * j], y[4 * j], f.x);
                f.y = fmaf(x[4 * j + 1], y[4 * j + 1], f.y);
                f.z = fmaf(x[4 * j + 2], y[4 * j + 2], f.z);
                f.w = fmaf(x[4 * j + 3], y[4 * j + 3], f.w);
                at[(slot * 2 * C + j) * T] = f;
            }
        }
    }
    __device__ __forceinline__ void get(int which, int slot, float (&x)[8 * C]) const {
        if constexpr (C == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = v[which][i];
        } else {
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) {
                const float4 f = at[(slot * 2 * C + j) * T];
                x[4 * j] = f.x;
                x[4 * j + 1] = f.y;
                x[4 * j + 2] = f.z;
                x[4 * j + 3] = f.w;
            }
        }
    }
};

// The rows of a CTA, or of a cluster of `parts` CTAs that each take a part of a
// row, are consecutive; the sums over them are left in `part`.  A gate row's sum
// is done where all of its rows are the CTA's, else its share goes to gate_part.
template <int TY, int TX, bool VEC, int C>
__global__ void __launch_bounds__(NORM_MAX_T) norm_grad_kernel(const __grid_constant__ NormGradParams g) {
    extern __shared__ float4 dynamic[];  // sums (C > 1), vectors, the rows ahead
    __shared__ float2 buffer[2][16], meet[2][8];
    const NormParams& p = g.f;
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    const int rank = g.parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int base = rank * T * 8 * C;
    const long long cta = blockIdx.x / g.parts;
    const long long begin = norm_row(p.M, g.ctas, cta), end = norm_row(p.M, g.ctas, cta + 1);
    Shared shared{buffer, meet, T, t, g.parts, rank, 0};
    const int all = g.slots + g.gate_sums;
    RowSums<C> sums;
    sums.at = dynamic + t;
    sums.T = T;
    sums.clear(all);
    RowThreads<VEC, C> rt{T, t, base, D, 0u, 0u, p.row_bytes, p.depth, 0, static_cast<int>(end - begin)};
    rt.cache = smem_u32(dynamic + (C == 1 ? 0 : all * 2 * C * T) + t);
    rt.ring = rt.cache + p.vec_bytes;
    rt.clear();
    const bool row_gate = p.gate.data && p.group_rows == 1;
    const Mat none{nullptr, 0, 0};
    const int col = base + norm_column<VEC>(T, t, 0);
    Ahead ahead[5];
    ahead[0].start(p.y, TY, begin, col);
    ahead[1].start(p.x, TX, begin, col);
    ahead[2].start(g.dh, TX, begin, col);
    ahead[3].start(g.dn, TY, begin, col);
    ahead[4].start(row_gate ? p.gate : none, p.gate_type, begin, col);
    Output<VEC, C> out_x(g.dx, TX, begin, col), out_y(g.dy, TY, begin, col);
    GateRow gate(begin, p.group_rows);
    const float4* stats_at = p.stats + begin;
    // every CTA of the cluster is there before another writes its shared memory
    if (g.parts > 1) cluster_sync();
    grid_wait();
    grid_release();
    if (VEC)
        for (int i = 0; i < p.depth; ++i) rt.issue(ahead);
    rt.keep(p.vec_at[0], p.post_w.data, p.post_w.type, 0, 1);
    rt.keep(p.vec_at[1], p.post_b.data, p.post_b.type, 0, 1);
    rt.keep(p.vec_at[2], p.pre_w.data, p.pre_w.type, 0, 1);
    long long kept_gate = -1;
    float4 next = *stats_at;
    const float over_d = 1.f / D;
    for (long long row = begin; row < end; ++row) {
        float y[8 * C], h[8 * C], d[8 * C], e[8 * C], u[8 * C], gv[8 * C];
        const float4 stats = next;
        if (row + 1 < end) next = *++stats_at;
        if (p.gate.data && !row_gate && gate.row != kept_gate) {
            rt.keep(p.vec_at[4], p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs);
            kept_gate = gate.row;
        }
        auto get = [&](int i, float w) { gv[i] = w; };
        if (VEC && p.depth > 0) {
            copies_wait(p.depth - 1);
            uint32_t from = rt.ring + rt.slot * rt.bytes;
            rt.template take<TY>(from, p.y, y);
            rt.template take<TX>(from, p.x, h);
            rt.template take<TX>(from, g.dh, d);
            rt.template take<TY>(from, g.dn, e);
            if (row_gate) {
                if (p.gate_type == T_F32)
                    rt.template take<T_F32>(from, p.gate, gv);
                else if (p.gate_type == T_F16)
                    rt.template take<T_F16>(from, p.gate, gv);
                else
                    rt.template take<T_BF16>(from, p.gate, gv);
            }
            rt.issue(ahead);
        } else {
            load_row<TY, VEC, C>(p.y, row, T, t, base, D, y);
            if (p.x.data) load_row<TX, VEC, C>(p.x, row, T, t, base, D, h);
            if (g.dh.data) load_row<TX, VEC, C>(g.dh, row, T, t, base, D, d);
            if (g.dn.data) load_row<TY, VEC, C>(g.dn, row, T, t, base, D, e);
            if (row_gate) with_vector<VEC, C>(p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs, T, t, base, D, get);
        }
        if (p.gate.data && !row_gate) rt.each(p.vec_at[4], p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs, get);
        // y becomes yhat, u what the gate multiplies, h the sum and then hhat
        if (p.post) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) y[i] = (y[i] - stats.x) * (rt.there(i) ? stats.y : 0.f);
        }
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) u[i] = y[i];
        if (p.post) {
            rt.each(p.vec_at[0], p.post_w.data, p.post_w.type, 0, 1, [&](int i, float w) { u[i] *= w; });
            rt.each(p.vec_at[1], p.post_b.data, p.post_b.type, 0, 1, [&](int i, float w) { u[i] += w; });
        }
        if (g.dn.data) {
            if (p.gate.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) h[i] = fmaf(p.scale, gv[i] * u[i], p.x.data ? h[i] : 0.f);
            } else {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) h[i] = fmaf(p.scale, u[i], p.x.data ? h[i] : 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) h[i] = rt.there(i) ? (h[i] - stats.z) * stats.w : 0.f;
            if (g.slot[0] >= 0) sums.add(0, g.slot[0], e, h);
            if (g.slot[1] >= 0) sums.add(1, g.slot[1], e);
            rt.each(p.vec_at[2], p.pre_w.data, p.pre_w.type, 0, 1, [&](int i, float w) { e[i] *= w; });
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) a = fmaf(e[i], h[i], a);
            float m0 = 0.f, m1;
            if (p.pre == NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) b += e[i];
                const float2 s = shared.template sum<true>(a, b);
                m1 = s.x * over_d;
                m0 = s.y * over_d;
            } else {
                m1 = shared.template sum<false>(a, 0.f).x * over_d;
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) e[i] = fmaf(-m1, h[i], e[i] - m0);
            if (g.dh.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) d[i] = fmaf(stats.w, e[i], d[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) d[i] = stats.w * e[i];
            }
        }
        if (g.dx.data) out_x.template store<TX>(rt, g.dx, row, d);
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) d[i] *= p.scale;
        if (p.gate.data) {
            if (g.gate_sums) {
                sums.add(4, g.slots, d, u);
            } else if (g.dgate.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) u[i] *= d[i];
                store_row<VEC, C>(g.dgate, p.gate_type, gate.row, T, t, base, D, u);
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] *= gv[i];
        }
        if (p.post) {
            if (g.slot[2] >= 0) sums.add(2, g.slot[2], d, y);
            if (g.slot[3] >= 0) sums.add(3, g.slot[3], d);
            rt.each(p.vec_at[0], p.post_w.data, p.post_w.type, 0, 1, [&](int i, float w) { d[i] *= w; });
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) a = fmaf(rt.there(i) ? d[i] : 0.f, y[i], a);
            float m0 = 0.f, m1;
            if (p.post == NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) b += rt.there(i) ? d[i] : 0.f;
                const float2 s = shared.template sum<true>(a, b);
                m1 = s.x * over_d;
                m0 = s.y * over_d;
            } else {
                m1 = shared.template sum<false>(a, 0.f).x * over_d;
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] = stats.y * fmaf(-m1, y[i], d[i] - m0);
        }
        if (g.dy.data) out_y.template store<TY>(rt, g.dy, row, d);
        // the last row of a gate row, or of this CTA
        if (g.gate_sums && (row + 1 == end || gate.left == 1)) {
            const bool begins = gate.row * p.group_rows >= begin, ends = (gate.row + 1) * p.group_rows <= end;
            float* const to = g.gate_part + (cta * 2 + begins) * D;
            sums.get(4, g.slots, u);
            sums.zero(4, g.slots);
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                const int c = base + norm_column<VEC>(T, t, i);
                if (c >= D) continue;
                if (begins && ends)
                    store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate.row * g.dgate.rs + c * g.dgate.cs, u[i]);
                else
                    to[c] = u[i];
            }
        }
        gate.next();
    }
    if (VEC) copies_wait(0);
#pragma unroll
    for (int which = 0; which < 4; ++which) {
        if (g.slot[which] < 0) continue;
        float* const to = g.part + (cta * g.slots + g.slot[which]) * D;
        float u[8 * C];
        sums.get(which, g.slot[which], u);
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            const int c = base + norm_column<VEC>(T, t, i);
            if (c < D) to[c] = u[i];
        }
    }
    // no CTA leaves while another may write its shared memory
    if (g.parts > 1) cluster_sync();
}

// Rows of any length; the sums are kept in `part` and gate_part themselves.
template <int TY, int TX>
__global__ void __launch_bounds__(NORM_MAX_T) norm_grad_long_kernel(const __grid_constant__ NormGradParams g) {
    __shared__ float2 buffer[2][16];
    const NormParams& p = g.f;
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    int turn = 0;
    grid_wait();
    grid_release();
    const float over_d = 1.f / D;
    const long long begin = norm_row(p.M, g.ctas, blockIdx.x), end = norm_row(p.M, g.ctas, blockIdx.x + 1);
    float* const part = g.part + static_cast<long long>(blockIdx.x) * g.slots * D;
    for (int s = 0; s < g.slots; ++s)
        for (int c = t; c < D; c += T) part[static_cast<long long>(s) * D + c] = 0.f;
    auto add = [&](int which, int c, float v) {
        if (g.slot[which] >= 0) part[static_cast<long long>(g.slot[which]) * D + c] += v;
    };
    auto vec = [&](const Vec& w, int c, float none) { return w.data ? load_any(w.data, w.type, c) : none; };
    for (long long row = begin; row < end; ++row) {
        const float4 stats = p.stats[row];
        const long long gate_row = p.gate.data ? row / p.group_rows : 0;
        const bool begins = gate_row * p.group_rows >= begin, ends = (gate_row + 1) * p.group_rows <= end;
        const bool fresh = row == begin || row % p.group_rows == 0, last = row + 1 == end || (row + 1) % p.group_rows == 0;
        float* const gate_part = g.gate_part + (static_cast<long long>(blockIdx.x) * 2 + begins) * D;
        auto load_yhat = [&](int c) {
            const float y = load_elem<TY>(p.y.data, row * p.y.rs + c * p.y.cs);
            return p.post ? (y - stats.x) * stats.y : y;
        };
        auto load_gate = [&](int c) { return p.gate.data ? load_any(p.gate.data, p.gate_type, gate_row * p.gate.rs + c * p.gate.cs) : 1.f; };
        auto u_of = [&](int c, float yhat) { return p.post ? fmaf(yhat, vec(p.post_w, c, 1.f), vec(p.post_b, c, 0.f)) : yhat; };
        auto load_hhat = [&](int c) {
            const float v = load_gate(c) * u_of(c, load_yhat(c));
            const float h = p.x.data ? fmaf(p.scale, v, load_elem<TX>(p.x.data, row * p.x.rs + c * p.x.cs)) : p.scale * v;
            return (h - stats.z) * stats.w;
        };
        auto load_dn = [&](int c) { return load_elem<TY>(g.dn.data, row * g.dn.rs + c * g.dn.cs); };
        float h1 = 0.f, h0 = 0.f;
        if (g.dn.data) {
            float a = 0.f, b = 0.f;
            for (int c = t; c < D; c += T) {
                const float e = load_dn(c) * vec(p.pre_w, c, 1.f);
                a = fmaf(e, load_hhat(c), a);
                b += e;
            }
            const float2 s = row_sum<true>(a, b, T, t, buffer, turn);
            h1 = s.x * over_d;
            h0 = p.pre == NORM_LAYER ? s.y * over_d : 0.f;
        }
        auto load_dH = [&](int c) {
            float d = g.dh.data ? load_elem<TX>(g.dh.data, row * g.dh.rs + c * g.dh.cs) : 0.f;
            if (g.dn.data) d += stats.w * (load_dn(c) * vec(p.pre_w, c, 1.f) - load_hhat(c) * h1 - h0);
            return d;
        };
        float y1 = 0.f, y0 = 0.f;
        if (p.post) {
            float a = 0.f, b = 0.f;
            for (int c = t; c < D; c += T) {
                const float d = load_dH(c) * p.scale * load_gate(c) * vec(p.post_w, c, 1.f);
                a = fmaf(d, load_yhat(c), a);
                b += d;
            }
            const float2 s = row_sum<true>(a, b, T, t, buffer, turn);
            y1 = s.x * over_d;
            y0 = p.post == NORM_LAYER ? s.y * over_d : 0.f;
        }
        for (int c = t; c < D; c += T) {
            const float dH = load_dH(c), yhat = load_yhat(c);
            if (g.dn.data) {
                const float e = load_dn(c);
                add(0, c, e * load_hhat(c));
                add(1, c, e);
            }
            float d = dH * p.scale;
            if (p.gate.data) {
                const float dg = d * u_of(c, yhat);
                if (!g.gate_sums) {
                    if (g.dgate.data) store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate_row * g.dgate.rs + c * g.dgate.cs, dg);
                } else {
                    const float s = (fresh ? 0.f : gate_part[c]) + dg;
                    if (last && begins && ends)
                        store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate_row * g.dgate.rs + c * g.dgate.cs, s);
                    else
                        gate_part[c] = s;
                }
                d *= load_gate(c);
            }
            if (g.dx.data) store_any(const_cast<void*>(g.dx.data), TX, row * g.dx.rs + c * g.dx.cs, dH);
            if (p.post) {
                add(2, c, d * yhat);
                add(3, c, d);
                d = stats.y * (d * vec(p.post_w, c, 1.f) - yhat * y1 - y0);
            }
            if (g.dy.data) store_any(const_cast<void*>(g.dy.data), TY, row * g.dy.rs + c * g.dy.cs, d);
        }
    }
}

// The CTAs' sums, in the order of the CTAs: blockIdx.y names a sum over all rows,
// or a gate row past those; 32 columns a CTA, 8 warps take every 8th part.
template <int DUMMY>
__global__ void __launch_bounds__(256) norm_finish_kernel(const __grid_constant__ NormFinishParams p) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_wait();
    grid_release();
    for (long long what = blockIdx.y; what < p.slots + p.groups; what += gridDim.y) {
        const bool gate = what >= p.slots;
        const long long group = what - p.slots;
        long long first = 0, last = p.ctas - 1;
        if (gate) {
            // the CTAs that hold the group's first and last row
            const long long r0 = group * p.group_rows, r1 = r0 + p.group_rows - 1;
            first = r0 * p.ctas / p.M;
            while (norm_row(p.M, p.ctas, first + 1) <= r0) ++first;
            last = r1 * p.ctas / p.M;
            while (norm_row(p.M, p.ctas, last + 1) <= r1) ++last;
            if (first == last) continue;  // that CTA has written it
        }
        float s = 0.f;
        if (c < p.D) {
#pragma unroll 4
            for (long long k = first + warp; k <= last; k += 8) {
                const long long at = gate ? k * 2 + (k == first) : k * p.slots + what;
                s += (gate ? p.gate_part : p.part)[at * p.D + c];
            }
        }
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < p.D) {
#pragma unroll
            for (int w = 1; w < 8; ++w) s += part[w][lane];
            if (gate)
                store_any(const_cast<void*>(p.dgate.data), p.gate_type, group * p.dgate.rs + c * p.dgate.cs, s);
            else
                store_any(p.out[what], p.type[what], c, s);
        }
    }
}

}  // namespace block
}  // namespace gct

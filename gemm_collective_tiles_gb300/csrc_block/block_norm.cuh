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
};
struct NormGradParams {
    NormParams f;             // h and n unused; stats read
    Mat dh, dn, dy, dx, dgate;
    // Sums over the rows that a CTA keeps for itself: which of dpre_w, dpre_b,
    // dpost_w, dpost_b are wanted, by slot (-1: not)
    int slot[4], slots;
    int gate_sums;            // dgate is a sum over rows
    int parts;                // CTAs of a cluster that share a row
    int depth;                // rows ahead in shared memory
    unsigned row_bytes;       // of them each
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
// Sums of two values over a row's T threads (a whole number of warps).  `turn`
// alternates between two buffers, so that one barrier a reduction is enough.
__device__ __forceinline__ float2 row_sum(float a, float b, int T, int t, float2 (*buffer)[32], int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (T == 32) return make_float2(a, b);
    if ((t & 31) == 0) buffer[turn][t >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
    for (int w = 0; w < T / 32; ++w) {
        const float2 x = buffer[turn][w];
        s.x += x.x;
        s.y += x.y;
    }
    turn ^= 1;
    return s;
}
// mean and r of the values, those past the row's end left out
template <bool VEC, int C>
__device__ __forceinline__ float2 row_stats(const float (&v)[8 * C], int kind, float eps, int T, int t, int D, float2 (*buffer)[32],
                                            int& turn) {
    float mean = 0.f;
    if (kind == NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) s += v[i];  // zeros past the end
        mean = row_sum(s, 0.f, T, t, buffer, turn).x / D;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) {
        const float d = norm_column<VEC>(T, t, i) < D ? v[i] - mean : 0.f;
        s = fmaf(d, d, s);
    }
    return make_float2(mean, rsqrtf(row_sum(s, 0.f, T, t, buffer, turn).x / D + eps));
}

template <int TY, int TX, bool VEC, int C>
__global__ void __launch_bounds__(NORM_MAX_T) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 buffer[2][32];
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    int turn = 0;
    grid_wait();
    grid_release();
    // a row per CTA, or per warp
    const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.M) return;
    float v[8 * C], x[8 * C];
    load_row<TY, VEC, C>(p.y, row, T, t, 0, D, v);
    if (p.x.data) load_row<TX, VEC, C>(p.x, row, T, t, 0, D, x);
    float4 stats = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.post) {
        const float2 s = row_stats<VEC, C>(v, p.post, p.eps, T, t, D, buffer, turn);
        stats.x = s.x;
        stats.y = s.y;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) v[i] = norm_column<VEC>(T, t, i) < D ? (v[i] - s.x) * s.y : 0.f;
        with_vector<VEC, C>(p.post_w.data, p.post_w.type, 0, 1, T, t, 0, D, [&](int i, float w) { v[i] *= w; });
        with_vector<VEC, C>(p.post_b.data, p.post_b.type, 0, 1, T, t, 0, D, [&](int i, float w) { v[i] += w; });
    }
    with_vector<VEC, C>(p.gate.data, p.gate_type, p.gate.data ? row / p.group_rows * p.gate.rs : 0, p.gate.cs, T, t, 0, D,
                        [&](int i, float w) { v[i] *= w; });
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) v[i] = p.x.data ? fmaf(p.scale, v[i], x[i]) : p.scale * v[i];
    if (p.h.data) store_row<VEC, C>(p.h, TX, row, T, t, 0, D, v);
    if (p.pre) {
        const float2 s = row_stats<VEC, C>(v, p.pre, p.eps, T, t, D, buffer, turn);
        stats.z = s.x;
        stats.w = s.y;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) v[i] = (v[i] - s.x) * s.y;
        with_vector<VEC, C>(p.pre_w.data, p.pre_w.type, 0, 1, T, t, 0, D, [&](int i, float w) { v[i] *= w; });
        with_vector<VEC, C>(p.pre_b.data, p.pre_b.type, 0, 1, T, t, 0, D, [&](int i, float w) { v[i] += w; });
        store_row<VEC, C>(p.n, TY, row, T, t, 0, D, v);
    }
    if (p.stats && t == 0) p.stats[row] = stats;
}

// Rows of any length, read anew for each reduction: one CTA per row.
template <int TY, int TX>
__global__ void __launch_bounds__(NORM_MAX_T) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 buffer[2][32];
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
            m = row_sum(s, 0.f, T, t, buffer, turn).x / D;
        }
        s = 0.f;
        for (int c = t; c < D; c += T) {
            const float d = value(c) - m;
            s = fmaf(d, d, s);
        }
        r = rsqrtf(row_sum(s, 0.f, T, t, buffer, turn).x / D + p.eps);
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

// Rows come to a thread through shared memory that only it uses: it copies its
// own pieces of the next `depth` rows asynchronously, so that no barrier stands
// between a copy and its use, and the copies of rows ahead run under the
// reductions of this one.
template <int TY, int TX, bool VEC, int C>
struct RowQueue {
    static constexpr int GY = TY == T_F32 ? 2 : 1, GX = TX == T_F32 ? 2 : 1;  // 16-byte pieces of 8 elements
    const NormGradParams& g;
    int T, t, base, depth, slot = 0;
    uint32_t ring, unit;  // address of this thread's first piece; a row's bytes
    long long next, end;

    __device__ __forceinline__ void issue() {
        uint32_t to = ring + slot * unit;
        if (next < end) {
            auto copy = [&](const Mat& m, int elem, int pieces) {
                if (!m.data) return;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = base + norm_column<true>(T, t, 8 * c);
                    if (col < g.f.D) {
                        const char* from = static_cast<const char*>(m.data) + (next * m.rs + col) * elem;
                        for (int k = 0; k < pieces; ++k) copy16_async(to + (c * pieces + k) * T * 16, from + 16 * k);
                    }
                }
                to += C * pieces * T * 16;
            };
            copy(g.f.y, TY == T_F32 ? 4 : 2, GY);
            copy(g.f.x, TX == T_F32 ? 4 : 2, GX);
            copy(g.dh, TX == T_F32 ? 4 : 2, GX);
            copy(g.dn, TY == T_F32 ? 4 : 2, GY);
        }
        ++next;
        copies_commit();
        slot = slot + 1 == depth ? 0 : slot + 1;
    }
    template <int TYPE>
    __device__ __forceinline__ void take(const Mat& m, uint32_t& from, float (&v)[8 * C]) const {
        constexpr int G = TYPE == T_F32 ? 2 : 1;
        if (!m.data) return;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            Raw<TYPE> raw;
#pragma unroll
            for (int k = 0; k < G; ++k)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(raw.q[k].x), "=r"(raw.q[k].y), "=r"(raw.q[k].z), "=r"(raw.q[k].w)
                             : "r"(from + (c * G + k) * T * 16)
                             : "memory");
            float w[8];
            spread8<TYPE>(raw, w);
            const bool there = base + norm_column<true>(T, t, 8 * c) < g.f.D;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * c + e] = there ? w[e] : 0.f;
        }
        from += C * G * T * 16;
    }
    // the row's pieces into registers, and the copies of a row ahead on their way
    __device__ __forceinline__ void row(long long r, float (&y)[8 * C], float (&x)[8 * C], float (&dh)[8 * C], float (&dn)[8 * C]) {
        if (VEC && depth > 0) {
            copies_wait(depth - 1);
            uint32_t from = ring + slot * unit;
            take<TY>(g.f.y, from, y);
            take<TX>(g.f.x, from, x);
            take<TX>(g.dh, from, dh);
            take<TY>(g.dn, from, dn);
            issue();
            return;
        }
        load_row<TY, VEC, C>(g.f.y, r, T, t, base, g.f.D, y);
        if (g.f.x.data) load_row<TX, VEC, C>(g.f.x, r, T, t, base, g.f.D, x);
        if (g.dh.data) load_row<TX, VEC, C>(g.dh, r, T, t, base, g.f.D, dh);
        if (g.dn.data) load_row<TY, VEC, C>(g.dn, r, T, t, base, g.f.D, dn);
    }
};

// A row's sums over the CTAs of a cluster that share it, in their order.
struct Shared {
    float2 (*buffer)[32];
    float2 (*meet)[8];
    int T, t, parts, rank, turn;
    __device__ __forceinline__ float2 sum(float a, float b) {
        const int now = turn;
        float2 s = row_sum(a, b, T, t, buffer, turn);
        if (parts == 1) {
            return s;
        }
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
    extern __shared__ float4 dynamic[];  // sums (C > 1), then the rows ahead
    __shared__ float2 buffer[2][32], meet[2][8];
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
    RowQueue<TY, TX, VEC, C> queue{g, T, t, base, g.depth, 0, 0u, g.row_bytes, begin, end};
    queue.ring = smem_u32(dynamic + (C == 1 ? 0 : all * 2 * C * T) + t);
    // every CTA of the cluster is there before another writes its shared memory
    if (g.parts > 1) cluster_sync();
    grid_wait();
    grid_release();
    if (VEC)
        for (int i = 0; i < g.depth; ++i) queue.issue();
    auto add = [&](int which, const float (&v)[8 * C]) {
        if (g.slot[which] >= 0) sums.add(which, g.slot[which], v);
    };
    auto there = [&](int i) { return base + norm_column<VEC>(T, t, i) < D; };
    const float over_d = 1.f / D;
    for (long long row = begin; row < end; ++row) {
        float y[8 * C], h[8 * C], d[8 * C], e[8 * C];
        const float4 stats = p.stats[row];
        queue.row(row, y, h, d, e);
        const long long gate_row = p.gate.data ? row / p.group_rows : 0;
        // y becomes yhat, u what the gate multiplies, h the sum
        float u[8 * C];
        if (p.post) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) y[i] = there(i) ? (y[i] - stats.x) * stats.y : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) u[i] = y[i];
        if (p.post) {
            with_vector<VEC, C>(p.post_w.data, p.post_w.type, 0, 1, T, t, base, D, [&](int i, float w) { u[i] *= w; });
            with_vector<VEC, C>(p.post_b.data, p.post_b.type, 0, 1, T, t, base, D, [&](int i, float w) { u[i] += w; });
        }
        if (g.dn.data) {
            float v[8 * C];
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = u[i];
            with_vector<VEC, C>(p.gate.data, p.gate_type, gate_row * p.gate.rs, p.gate.cs, T, t, base, D, [&](int i, float w) { v[i] *= w; });
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                h[i] = p.x.data ? fmaf(p.scale, v[i], h[i]) : p.scale * v[i];
                h[i] = there(i) ? (h[i] - stats.z) * stats.w : 0.f;  // hhat
                v[i] = e[i] * h[i];
            }
            add(0, v);
            add(1, e);
            with_vector<VEC, C>(p.pre_w.data, p.pre_w.type, 0, 1, T, t, base, D, [&](int i, float w) { e[i] *= w; });
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                a = fmaf(e[i], h[i], a);
                b += e[i];
            }
            const float2 s = shared.sum(a, b);
            const float m1 = s.x * over_d, m0 = p.pre == NORM_LAYER ? s.y * over_d : 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                const float v = stats.w * (e[i] - h[i] * m1 - m0);
                d[i] = g.dh.data ? d[i] + v : v;
            }
        }
        if (g.dx.data) store_row<VEC, C>(g.dx, TX, row, T, t, base, D, d);
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) d[i] *= p.scale;
        if (p.gate.data) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) u[i] *= d[i];
            if (g.gate_sums)
                sums.add(4, g.slots, u);
            else if (g.dgate.data)
                store_row<VEC, C>(g.dgate, p.gate_type, gate_row, T, t, base, D, u);
            with_vector<VEC, C>(p.gate.data, p.gate_type, gate_row * p.gate.rs, p.gate.cs, T, t, base, D, [&](int i, float w) { d[i] *= w; });
        }
        if (p.post) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                d[i] = there(i) ? d[i] : 0.f;
                u[i] = d[i] * y[i];
            }
            add(2, u);
            add(3, d);
            with_vector<VEC, C>(p.post_w.data, p.post_w.type, 0, 1, T, t, base, D, [&](int i, float w) { d[i] *= w; });
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                a = fmaf(d[i], y[i], a);
                b += d[i];
            }
            const float2 s = shared.sum(a, b);
            const float m1 = s.x * over_d, m0 = p.post == NORM_LAYER ? s.y * over_d : 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] = stats.y * (d[i] - y[i] * m1 - m0);
        }
        if (g.dy.data) store_row<VEC, C>(g.dy, TY, row, T, t, base, D, d);
        // the last row of a gate row, or of this CTA
        if (g.gate_sums && (row + 1 == end || (row + 1) % p.group_rows == 0)) {
            const bool begins = gate_row * p.group_rows >= begin, ends = (gate_row + 1) * p.group_rows <= end;
            float* const to = g.gate_part + (cta * 2 + begins) * D;
            sums.get(4, g.slots, u);
            sums.zero(4, g.slots);
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                const int c = base + norm_column<VEC>(T, t, i);
                if (c >= D) continue;
                if (begins && ends)
                    store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate_row * g.dgate.rs + c * g.dgate.cs, u[i]);
                else
                    to[c] = u[i];
            }
        }
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
    __shared__ float2 buffer[2][32];
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
            const float2 s = row_sum(a, b, T, t, buffer, turn);
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
            const float2 s = row_sum(a, b, T, t, buffer, turn);
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

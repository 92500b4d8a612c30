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
// Every tensor is read and written once: a row's elements stay in registers
// between the reductions (two passes over them for a variance); h enters the second
// norm unrounded, and the gradient computes it again from x and y instead of
// reading it back rounded.
//
// T threads take a row, 8 C elements each, and one group of threads many rows; rows
// come ahead of their use by asynchronous copies.  The forward pass is bound by
// memory (16384 x 4096 bf16, f32 stream, both norms and a gate: 129 us, 6.2 TB/s),
// the gradient by its reductions, whose latency 16 warps an SM (128 registers) hide
// in part, and by instructions (16384 x 4096 bf16, layer norm and gate: 165 us, 4.9
// TB/s; rms alone 128, 6.3).  Rows that start anywhere come as single elements (1537 x 5003
// f16, both norms: 38 and 117 us).  Rows that are too long
// for a group's registers are shared by a cluster (gradient), or gone over once per
// reduction.
#pragma once
#include "block_elem.cuh"

namespace gct {
namespace block {

enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
constexpr int NORM_MAX_T = 512;                          // threads of a row, in the gradient
constexpr int NORM_CTA = 1024;                           // of a CTA, and of a row
constexpr int NORM_LONGEST = NORM_CTA * 2 * 8, NORM_GRAD_LONGEST = NORM_MAX_T * 2 * 8;  // elements of a row in registers

struct Vec {
    const void* data;
    int type;
};
// Threads T of a row at 8 C elements each.
struct RowShape {
    int T, C;
};
struct NormParams {
    Mat y, x, gate, h, n;
    Vec post_w, post_b, pre_w, pre_b;
    int gate_type;
    long long M, group_rows, gate_rows;  // rows of y per row of gate
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

// The layout of a row over its T threads, 8 C elements each: W > 0: pieces of W
// neighbouring elements, one piece of every thread after another (8 where all
// tensors are of 16 bits, 4 beside f32: 16 bytes of the wider type, so that a
// warp's access is one run of memory); W = 0: one element in T, any strides.
template <int W>
__device__ __forceinline__ int norm_column(int T, int t, int i) {
    return W ? (i / (W ? W : 1) * T + t) * W + i % (W ? W : 1) : i * T + t;
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ uint2 shared_8(uint32_t at) {
    uint2 q;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ void shared16(uint32_t at, const uint4& q) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
// W elements of a type, as they lie in memory
template <int TYPE, int W>
struct Bits {
    static constexpr int WORDS = W * (TYPE == T_F32 ? 4 : 2) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const void* p) {
        if constexpr (WORDS == 2) {
            const uint2 q = *static_cast<const uint2*>(p);
            w[0] = q.x;
            w[1] = q.y;
        } else {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) put(k, static_cast<const uint4*>(p)[k]);
        }
    }
    // from shared memory, 16 bytes `apart`
    __device__ __forceinline__ void load_shared(uint32_t at, uint32_t apart) {
        if constexpr (WORDS == 2) {
            const uint2 q = shared_8(at);
            w[0] = q.x;
            w[1] = q.y;
        } else {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) put(k, shared16(at + k * apart));
        }
    }
    __device__ __forceinline__ void put(int k, const uint4& q) {
        w[4 * k] = q.x;
        w[4 * k + 1] = q.y;
        w[4 * k + 2] = q.z;
        w[4 * k + 3] = q.w;
    }
    __device__ __forceinline__ void spread(float* v) const {
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            if (TYPE == T_F32)
                v[k] = __uint_as_float(w[k]);
            else
                unpack16<TYPE>(w[k], v[2 * k], v[2 * k + 1]);
        }
    }
};
template <int TYPE, int W>
__device__ __forceinline__ void store_bits(char* to, const float* v) {
    if constexpr (TYPE == T_F32) {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) reinterpret_cast<float4*>(to)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack16(v[0], v[1], TYPE == T_BF16), pack16(v[2], v[3], TYPE == T_BF16));
    } else {
        constexpr int bf = TYPE == T_BF16;
        *reinterpret_cast<uint4*>(to) = make_uint4(pack16(v[0], v[1], bf), pack16(v[2], v[3], bf), pack16(v[4], v[5], bf), pack16(v[6], v[7], bf));
    }
}
template <int TYPE, int W, int C>
__device__ __forceinline__ void load_row(const Mat& m, long long row, int T, int t, int base, int D, float (&v)[8 * C]) {
    const long long o = row * m.rs;
    if constexpr (W > 0) {
        constexpr int P = 8 * C / W, E = TYPE == T_F32 ? 4 : 2;
        Bits<TYPE, W> raw[P];
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const int c = base + norm_column<W>(T, t, W * k);
            if (c < D) {
                raw[k].load(static_cast<const char*>(m.data) + (o + c) * E);
            } else {
#pragma unroll
                for (int j = 0; j < Bits<TYPE, W>::WORDS; ++j) raw[k].w[j] = 0u;
            }
        }
#pragma unroll
        for (int k = 0; k < P; ++k) raw[k].spread(v + W * k);
    } else {
        constexpr int E = TYPE == T_F32 ? 4 : 2;
        const char* at = static_cast<const char*>(m.data) + (o + (base + t) * m.cs) * E;
        const long long step = T * m.cs * E;
        int left = D - base - t;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i, at += step, left -= T) v[i] = left > 0 ? load_elem<TYPE>(at, 0) : 0.f;
    }
}
// f(i, value) for this thread's elements of a vector or of a row of gate
template <int W, int C, typename F>
__device__ __forceinline__ void with_vector(const void* data, int type, long long o, long long cs, int T, int t, int base, int D, F f) {
    if (!data) return;
    auto typed = [&](auto tag) {
        constexpr int TYPE = decltype(tag)::value, E = TYPE == T_F32 ? 4 : 2;
        if constexpr (W > 0) {
#pragma unroll
            for (int k = 0; k < 8 * C / W; ++k) {
                const int at = base + norm_column<W>(T, t, W * k);
                if (at >= D) continue;
                Bits<TYPE, W> raw;
                raw.load(static_cast<const char*>(data) + (o + at) * E);
                float w[W];
                raw.spread(w);
#pragma unroll
                for (int e = 0; e < W; ++e) f(W * k + e, w[e]);
            }
        } else {
            const char* at = static_cast<const char*>(data) + (o + (base + t) * cs) * E;
            const long long step = T * cs * E;
            int left = D - base - t;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i, at += step, left -= T)
                if (left > 0) f(i, load_elem<TYPE>(at, 0));
        }
    };
    if (type == T_F32)
        typed(std::integral_constant<int, T_F32>());
    else if (type == T_F16)
        typed(std::integral_constant<int, T_F16>());
    else
        typed(std::integral_constant<int, T_BF16>());
}
// Sums of one or two values over a row's T threads (a whole number of warps, 32
// at most), which are group `id` of the CTA.  `turn` alternates between two
// buffers, so that one barrier a reduction is enough; every warp adds the warps'
// sums up for itself.
struct RowGroup {
    int T, t, id, turn;
    float2 (*buffer)[32];  // by warp of the CTA
    __device__ __forceinline__ void sync() const {
        if (T == 32)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(T) : "memory");
    }
    template <bool TWO>
    __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (TWO) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (T == 32) return make_float2(a, b);
        float2* const mine = buffer[turn] + id * (T >> 5);
        if ((t & 31) == 0) mine[t >> 5] = make_float2(a, b);
        sync();
        const int w = t & 31;
        float2 s = make_float2(0.f, 0.f);
        if (w * 32 < T) s = mine[w];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
            if (TWO) s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
        }
        turn ^= 1;
        return s;
    }
};
// Mean and r of the values; those past the row's end are 0 and left out.
template <int W, int C>
__device__ __forceinline__ float2 row_stats(const float (&v)[8 * C], int kind, float eps, float over_d, int D, RowGroup& group) {
    float s = 0.f;
    if (kind == NORM_RMS) {
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) s = fmaf(v[i], v[i], s);
        return make_float2(0.f, rsqrtf(fmaf(group.sum<false>(s, 0.f).x, over_d, eps)));
    }
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) s += v[i];
    const float mean = group.sum<false>(s, 0.f).x * over_d;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) {
        const float d = norm_column<W>(group.T, group.t, W ? i / (W ? W : 1) * W : i) < D ? v[i] - mean : 0.f;
        s = fmaf(d, d, s);
    }
    return make_float2(mean, rsqrtf(fmaf(group.sum<false>(s, 0.f).x, over_d, eps)));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
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

// The gate's row for a row of y, kept up row by row.
struct GateRow {
    long long row, left, rows;
    __device__ __forceinline__ GateRow(long long first, long long group_rows) : row(first / group_rows), rows(group_rows) {
        left = (row + 1) * group_rows - first;
    }
    __device__ __forceinline__ bool next() {  // whether the gate's row is another one now
        if (--left) return false;
        ++row;
        left = rows;
        return true;
    }
};

// What a row's threads have of shared memory.  The vectors (post_w, post_b,
// pre_w, pre_b, and a gate of one row) lie there in fp32, for all of a CTA's rows.
// Each thread has its pieces of the next rows to itself, which it copies
// asynchronously: no barrier stands between a copy and its use, and the copies
// run under the reductions of the rows before.  A gate of several rows comes
// with the rows.
template <int W, int C>
struct RowMemory {
    int T, t, base, D;     // base: first column of the CTA's part of the row
    uint32_t cache, ring;  // this thread's
    uint32_t bytes;        // of a row ahead
    int depth, slot, left; // rows ahead (0: none), the next one's place, rows not yet copied
    uint32_t to;           // where the row under copy goes on
    int used;              // the place of the row that is used next
    __device__ __forceinline__ uint32_t here() const { return ring + used * bytes; }
    // the row that is used next is there
    __device__ __forceinline__ void arrived(const RowGroup& group) {
        if (W > 0) {
            copies_wait(depth - 1);
        } else {
            copies_wait(depth - 2);
            group.sync();  // all of its threads' copies
        }
        used = used + 1 == depth ? 0 : used + 1;
    }

    __device__ __forceinline__ uint32_t apart() const { return T * 16; }
    __device__ __forceinline__ int column(int i) const { return base + norm_column<W>(T, t, i); }
    __device__ __forceinline__ bool there(int i) const { return column(W ? i / (W ? W : 1) * W : i) < D; }
    // a vector into shared memory; zeros past its end
    __device__ __forceinline__ void keep(int at, const Vec& v, long long cs) const {
        if (!v.data || at < 0) return;
        float w[8 * C];
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) w[i] = 0.f;
        with_vector<W, C>(v.data, v.type, 0, cs, T, t, base, D, [&](int i, float x) { w[i] = x; });
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
            shared16(cache + (at * 2 * C + j) * apart(), make_uint4(__float_as_uint(w[4 * j]), __float_as_uint(w[4 * j + 1]),
                                                                    __float_as_uint(w[4 * j + 2]), __float_as_uint(w[4 * j + 3])));
    }
    // f(i, value) for this thread's elements of a vector.  KEPT: it lies in shared
    // memory, if there is one
    template <bool KEPT = false, typename F>
    __device__ __forceinline__ void each(int at, const Vec& v, F f, long long cs = 1) const {
        if (KEPT ? at < 0 : !v.data) return;
        if (!KEPT && at < 0) {
            with_vector<W, C>(v.data, v.type, 0, cs, T, t, base, D, f);
            return;
        }
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
            const uint4 q = shared16(cache + (at * 2 * C + j) * apart());
            f(4 * j, __uint_as_float(q.x));
            f(4 * j + 1, __uint_as_float(q.y));
            f(4 * j + 2, __uint_as_float(q.z));
            f(4 * j + 3, __uint_as_float(q.w));
        }
    }
    // threads past a row's end find zeros
    __device__ __forceinline__ void clear() const {
        if constexpr (W > 0) {
            if (!there(8 * C - 1))
                for (uint32_t at = 0; at < depth * bytes; at += apart()) shared16(ring + at, make_uint4(0u, 0u, 0u, 0u));
        }
    }
    // Pieces lie T * 16 bytes apart, whatever their size.
    template <int TYPE>
    __device__ __forceinline__ void copy(const char* from) {
        constexpr int B = W * (TYPE == T_F32 ? 4 : 2);
#pragma unroll
        for (int k = 0; k < 8 * C / (W ? W : 1); ++k) {
            if (there(W * k)) {
                const char* at = from + static_cast<long long>(k) * T * B;
#pragma unroll
                for (int j = 0; j < (B + 15) / 16; ++j) copy_async<(B < 16 ? 8 : 16)>(to + j * apart(), at + 16 * j);
            }
            to += (B + 15) / 16 * apart();
        }
    }
    // W = 0, elements of unit stride: a row's threads copy it together, in the pieces
    // of 16 bytes that it lies in, and its elements begin `shift` bytes into the
    // first.  Pieces that reach past the tensor's ends are filled by elements.
    static __device__ __forceinline__ uint32_t shift(const char* row) {
        return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u;
    }
    __device__ __forceinline__ uint32_t room(int elem) const { return 8 * C * T * elem + 32; }
    template <int TYPE>
    __device__ __forceinline__ void copy_pieces(const char* row, const char* lo, const char* hi) {
        constexpr int E = TYPE == T_F32 ? 4 : 2;
        const uint32_t s = shift(row);
        const int bytes_here = min(D - base, 8 * C * T) * E + static_cast<int>(s);  // from the first piece on
        const char* const first = row - s;
        const int from_lo = static_cast<int>(min(static_cast<long long>(s), max(0ll, static_cast<long long>(lo - first))));
        const long long to_hi = hi - first;
#pragma unroll
        for (int k = 0; k < C * E / 2 + 1; ++k) {
            const int at = (t + k * T) * 16;
            if (at >= bytes_here) break;
            if (at >= from_lo && at + 16 <= to_hi) {
                copy_async<16>(to + at, first + at);
            } else {
                for (int b = 0; b < 16; b += E) {
                    if (at + b < from_lo || at + b >= bytes_here) continue;
                    if (TYPE == T_F32)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + at + b), "f"(*reinterpret_cast<const float*>(first + at + b)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + at + b), "h"(*reinterpret_cast<const uint16_t*>(first + at + b)) : "memory");
                }
            }
        }
        to += room(E);
    }
    // an element past the row's end is read as well, and left out
    template <int TYPE, typename F>
    __device__ __forceinline__ void take_pieces(uint32_t& from, const char* row, F f) const {
        constexpr int E = TYPE == T_F32 ? 4 : 2;
        uint32_t at = from + shift(row) + t * E;
        const int n = D - base - t;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i, at += T * E) {
            float v;
            if (TYPE == T_F32) {
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            } else {
                uint32_t h;
                asm volatile("{\n\t.reg .b16 x;\n\tld.shared.b16 x, [%1];\n\tmov.b32 %0, {x, x};\n\t}" : "=r"(h) : "r"(at) : "memory");
                v = TYPE == T_BF16 ? __uint_as_float(h & 0xFFFF0000u) : __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
            }
            f(i, i * T < n ? v : 0.f);
        }
        from += room(E);
    }
    __device__ __forceinline__ void copy_typed(int type, const char* from) {
        if (type == T_F32)
            copy<T_F32>(from);
        else
            copy<T_F16>(from);
    }
    __device__ __forceinline__ bool begin_copy() {
        to = ring + slot * bytes;
        return left > 0;
    }
    __device__ __forceinline__ void end_copy() {
        --left;
        copies_commit();
        slot = slot + 1 == depth ? 0 : slot + 1;
    }
    template <int TYPE, typename F>
    __device__ __forceinline__ void take(uint32_t& from, F f) const {
        constexpr int N = (W * (TYPE == T_F32 ? 4 : 2) + 15) / 16;
#pragma unroll
        for (int k = 0; k < 8 * C / (W ? W : 1); ++k) {
            Bits<TYPE, W ? W : 8> raw;
            raw.load_shared(from, apart());
            from += N * apart();
            float w[W ? W : 8];
            raw.spread(w);
#pragma unroll
            for (int e = 0; e < W; ++e) f(W * k + e, w[e]);
        }
    }
    template <typename F>
    __device__ __forceinline__ void take_typed(int type, uint32_t& from, F f) const {
        if (type == T_F32)
            take<T_F32>(from, f);
        else if (type == T_F16)
            take<T_F16>(from, f);
        else
            take<T_BF16>(from, f);
    }
};
// One of the tensors whose rows come ahead: where this thread's first piece of the
// next one lies.
struct Ahead {
    const char *at, *hi;  // hi: the tensor's end
    long long step;
    __device__ __forceinline__ Ahead(const Mat& m, int type, long long row, int col, long long rows, int D) {
        const int elem = type == T_F32 ? 4 : 2;
        at = m.data ? static_cast<const char*>(m.data) + (row * m.rs + col) * elem : nullptr;
        hi = static_cast<const char*>(m.data) + ((rows - 1) * m.rs + D) * elem;
        step = m.rs * elem;
    }
};
// A tensor's rows under way, and where the one that is used now lies (W = 0: its
// address says how its pieces hold it).
template <int TYPE, int W, int C>
struct Stream {
    Ahead a;
    const char *lo, *now;
    __device__ __forceinline__ Stream(const Mat& m, long long row, int base, int col, long long rows, int D)
        : a(m, TYPE, row, W ? col : base, rows, D), lo(static_cast<const char*>(m.data)), now(a.at) {}
    // THERE: known not to be absent
    template <bool THERE = false>
    __device__ __forceinline__ void copy(RowMemory<W, C>& rm) {
        if (!THERE && !a.at) return;
        if constexpr (W > 0)
            rm.template copy<TYPE>(a.at);
        else
            rm.template copy_pieces<TYPE>(a.at, lo, a.hi);
        a.at += a.step;
    }
    template <bool THERE = false, typename F>
    __device__ __forceinline__ void take(const RowMemory<W, C>& rm, uint32_t& from, F f) {
        if (!THERE && !a.at) return;
        if constexpr (W > 0) {
            rm.template take<TYPE>(from, f);
        } else {
            rm.template take_pieces<TYPE>(from, now, f);
            now += a.step;
        }
    }
};
// The same of a gate of several rows, whose type is one of three.
template <int W, int C>
struct GateStream {
    Ahead a;
    const char *lo, *now;
    GateRow under_way, used;
    int type;
    __device__ __forceinline__ GateStream(const NormParams& p, bool there, long long row, int base, int col)
        : a(there ? p.gate : Mat{nullptr, 0, 0}, p.gate_type, row / p.group_rows, W ? col : base, p.gate_rows, p.D),
          lo(static_cast<const char*>(p.gate.data)), now(a.at), under_way(row, p.group_rows), used(under_way), type(p.gate_type) {}
    __device__ __forceinline__ void copy(RowMemory<W, C>& rm) {
        if (!a.at) return;
        if constexpr (W > 0) {
            rm.copy_typed(type, a.at);
        } else if (type == T_F32) {
            rm.template copy_pieces<T_F32>(a.at, lo, a.hi);
        } else {
            rm.template copy_pieces<T_F16>(a.at, lo, a.hi);
        }
        if (under_way.next()) a.at += a.step;
    }
    template <typename F>
    __device__ __forceinline__ void take(const RowMemory<W, C>& rm, uint32_t& from, F f) {
        if (!a.at) return;
        if constexpr (W > 0) {
            rm.take_typed(type, from, f);
        } else {
            if (type == T_F32)
                rm.template take_pieces<T_F32>(from, now, f);
            else if (type == T_F16)
                rm.template take_pieces<T_F16>(from, now, f);
            else
                rm.template take_pieces<T_BF16>(from, now, f);
        }
    }
    __device__ __forceinline__ void next() {
        if (used.next()) now += a.step;
    }
};
// this thread's part of an output, a row after the other
template <int TYPE, int W, int C>
struct Output {
    char* at;
    long long step;
    __device__ __forceinline__ Output(const Mat& m, long long row, int col) {
        constexpr int E = TYPE == T_F32 ? 4 : 2;
        at = m.data ? const_cast<char*>(static_cast<const char*>(m.data)) + (row * m.rs + col * (W ? 1 : m.cs)) * E : nullptr;
        step = m.rs * E;
    }
    __device__ __forceinline__ void store(const RowMemory<W, C>& rm, const Mat& m, const float (&v)[8 * C]) {
        if (!at) return;
        if constexpr (W > 0) {
#pragma unroll
            for (int k = 0; k < 8 * C / W; ++k)
                if (rm.there(W * k)) store_bits<TYPE, W>(at + static_cast<long long>(k) * rm.T * W * (TYPE == T_F32 ? 4 : 2), v + W * k);
        } else {
            const long long apart = rm.T * m.cs * (TYPE == T_F32 ? 4 : 2);
            char* to = at;
            int left = rm.D - rm.column(0);
#pragma unroll
            for (int i = 0; i < 8 * C; ++i, to += apart, left -= rm.T)
                if (left > 0) store_any(to, TYPE, 0, v[i]);
        }
        at += step;
    }
};

// blockDim.y groups of T threads, each with rows of its own one after another, so
// that one group's reductions pass under the others' work.
// QUEUED, for single elements: rows come ahead through shared memory; else they are
// read where they lie (a group has one, or no unit stride), by a kernel of its own,
// because those loads cost the other registers (6148 x 5003 f16: 130 us with, 121
// without).  Pieces do both in one (16384 x 4096 bf16: 107 us, 132 apart).
template <int TY, int TX, int W, int C, int CTA, bool QUEUED>
__global__ void __launch_bounds__(CTA) norm_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ float4 dynamic[];
    __shared__ float2 buffer[2][32];
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    const long long units = static_cast<long long>(gridDim.x) * blockDim.y, unit = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const long long begin = norm_row(p.M, units, unit), end = norm_row(p.M, units, unit + 1);
    RowGroup group{T, t, static_cast<int>(threadIdx.y), 0, buffer};
    RowMemory<W, C> rm{T, t, 0, D, 0u, 0u, p.row_bytes, p.depth, 0, static_cast<int>(end - begin), 0u, 0};
    rm.cache = smem_u32(dynamic) + t * 16;
    rm.ring = rm.cache + p.vec_bytes + threadIdx.y * p.depth * p.row_bytes - (W ? 0 : t * 16);
    rm.clear();
    const bool row_gate = p.gate.data && p.gate_rows > 1;
    const int col = norm_column<W>(T, t, 0);
    Stream<TY, W, C> in_y(p.y, begin, 0, col, p.M, D);
    Stream<TX, W, C> in_x(p.x, begin, 0, col, p.M, D);
    GateStream<W, C> in_gate(p, row_gate, begin, 0, col);
    Output<TX, W, C> out_h(p.h, begin, col);
    Output<TY, W, C> out_n(p.n, begin, col);
    float4* to_stats = p.stats ? p.stats + begin : nullptr;
    auto issue = [&]() {
        if (rm.begin_copy()) {
            in_y.copy(rm);
            in_gate.copy(rm);
            in_x.copy(rm);
        }
        rm.end_copy();
    };
    grid_wait();
    grid_release();
    // W = 0: a row's place is free again once all its threads have passed the next
    // row's barrier, so one row less is under way
    for (int i = 0; i < (W ? p.depth : p.depth - 1); ++i) issue();
    const Vec one_gate{row_gate ? nullptr : p.gate.data, p.gate_type};
    if (p.vec_bytes) {
        if (threadIdx.y == 0) {
            rm.keep(p.vec_at[0], p.post_w, 1);
            rm.keep(p.vec_at[1], p.post_b, 1);
            rm.keep(p.vec_at[2], p.pre_w, 1);
            rm.keep(p.vec_at[3], p.pre_b, 1);
            rm.keep(p.vec_at[4], one_gate, p.gate.cs);
        }
        __syncthreads();
    }
    const float over_d = 1.f / D;
    for (long long row = begin; row < end; ++row) {
        float v[8 * C], x[8 * C];
        const bool queued = W > 0 ? p.depth > 0 : QUEUED;
        uint32_t from = rm.here();
        auto get = [&](int i, float w) { v[i] = w; };
        auto times = [&](int i, float w) { v[i] *= w; };
        auto plus = [&](int i, float w) { v[i] += w; };
        if (queued) {
            rm.arrived(group);
            if constexpr (W == 0) issue();
            in_y.take(rm, from, get);
        } else {
            load_row<TY, W, C>(p.y, row, T, t, 0, D, v);
            if (p.x.data) load_row<TX, W, C>(p.x, row, T, t, 0, D, x);
        }
        float4 stats = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.post) {
            const float2 s = row_stats<W, C>(v, p.post, p.eps, over_d, D, group);
            stats.x = s.x;
            stats.y = s.y;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = (v[i] - s.x) * (rm.there(i) ? s.y : 0.f);
            rm.each(p.vec_at[0], p.post_w, times);
            rm.each(p.vec_at[1], p.post_b, plus);
        }
        // what lies past a row's end of x and of the gate in shared memory is 0
        auto add_x = [&](int i, float w) { v[i] = fmaf(p.scale, v[i], w); };
        if (queued)
            in_gate.take(rm, from, times);
        else if (row_gate)
            with_vector<W, C>(p.gate.data, p.gate_type, in_gate.used.row * p.gate.rs, p.gate.cs, T, t, 0, D, times);
        rm.each(p.vec_at[4], one_gate, times, p.gate.cs);
        if (!p.x.data) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] *= p.scale;
        } else if (queued) {
            in_x.take(rm, from, add_x);
        } else {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) add_x(i, x[i]);
        }
        if constexpr (W > 0) {
            if (queued) issue();
        }
        out_h.store(rm, p.h, v);
        if (p.pre) {
            const float2 s = row_stats<W, C>(v, p.pre, p.eps, over_d, D, group);
            stats.z = s.x;
            stats.w = s.y;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) v[i] = (v[i] - s.x) * s.y;
            rm.each(p.vec_at[2], p.pre_w, times);
            rm.each(p.vec_at[3], p.pre_b, plus);
            out_n.store(rm, p.n, v);
        }
        if (to_stats) {
            if (t == 0) *to_stats = stats;
            ++to_stats;
        }
        in_gate.next();
    }
    copies_wait(0);
}

// Rows of any length, read anew for each reduction: one CTA per row.
template <int TY, int TX>
__global__ void __launch_bounds__(NORM_MAX_T) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float2 buffer[2][32];
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    RowGroup group{T, t, 0, 0, buffer};
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
            m = group.sum<false>(s, 0.f).x / D;
        }
        s = 0.f;
        for (int c = t; c < D; c += T) {
            const float d = value(c) - m;
            s = fmaf(d, d, s);
        }
        r = rsqrtf(group.sum<false>(s, 0.f).x / D + p.eps);
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
    RowGroup group;
    float2 (*meet)[8];
    int parts, rank, turn;
    template <bool TWO>
    __device__ __forceinline__ float2 sum(float a, float b) {
        float2 s = group.sum<TWO>(a, b);
        if (parts == 1) return s;
        if (group.t < parts) {
            const uint32_t to = map_to(smem_u32(&meet[turn][rank]), group.t);
            st_shared_cluster_u32(to, __float_as_uint(s.x));
            st_shared_cluster_u32(to + 4, __float_as_uint(s.y));
        }
        cluster_sync();
        s = make_float2(0.f, 0.f);
        for (int k = 0; k < parts; ++k) {
            s.x += meet[turn][k].x;
            s.y += meet[turn][k].y;
        }
        turn ^= 1;
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

// POST: with a post-norm.  ALL: rows of x, dh and dn come ahead, and the vectors lie in
// shared memory.  Both are known beforehand so that the way through a row has few
// branches: loads wait at one (16384 x 4096 bf16, layer norm and gate: 208 us with
// neither, 198 with POST, 165 with both; 16384 x 2048, both norms: 150, 148, 121).
//
// The rows of a CTA, or of a cluster of `parts` CTAs that each take a part of a
// row, are consecutive; the sums over them are left in `part`.  A gate row's sum
// is done where all of its rows are the CTA's, else its share goes to gate_part.
template <int TY, int TX, int W, int C, bool POST, bool ALL>
__global__ void __launch_bounds__(NORM_MAX_T) norm_grad_kernel(const __grid_constant__ NormGradParams g) {
    extern __shared__ float4 dynamic[];  // sums (C > 1), vectors, the rows ahead
    __shared__ float2 buffer[2][32], meet[2][8];
    const NormParams& p = g.f;
    const int T = blockDim.x, t = threadIdx.x, D = p.D;
    const int rank = g.parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int base = rank * T * 8 * C;
    const long long cta = blockIdx.x / g.parts;
    const long long begin = norm_row(p.M, g.ctas, cta), end = norm_row(p.M, g.ctas, cta + 1);
    Shared shared{RowGroup{T, t, 0, 0, buffer}, meet, g.parts, rank, 0};
    const int all = g.slots + g.gate_sums;
    RowSums<C> sums;
    sums.at = dynamic + t;
    sums.T = T;
    sums.clear(all);
    RowMemory<W, C> rm{T, t, base, D, 0u, 0u, p.row_bytes, p.depth, 0, static_cast<int>(end - begin), 0u, 0};
    rm.cache = smem_u32(dynamic + (C == 1 ? 0 : all * 2 * C * T) + t);
    rm.ring = rm.cache + p.vec_bytes - (W ? 0 : t * 16);
    rm.clear();
    const bool row_gate = p.gate.data && p.gate_rows > 1;
    const Vec one_gate{row_gate ? nullptr : p.gate.data, p.gate_type};
    const int col = base + norm_column<W>(T, t, 0);
    Stream<TY, W, C> in_y(p.y, begin, base, col, p.M, D), in_n(g.dn, begin, base, col, p.M, D);
    Stream<TX, W, C> in_x(p.x, begin, base, col, p.M, D), in_h(g.dh, begin, base, col, p.M, D);
    GateStream<W, C> in_gate(p, row_gate, begin, base, col);
    Output<TX, W, C> out_x(g.dx, begin, col);
    Output<TY, W, C> out_y(g.dy, begin, col);
    GateRow gate(begin, p.group_rows);
    const float4* stats_at = p.stats + begin;
    auto issue = [&]() {
        if (rm.begin_copy()) {
            in_y.template copy<true>(rm);
            in_x.template copy<ALL>(rm);
            in_h.template copy<ALL>(rm);
            in_n.template copy<ALL>(rm);
            in_gate.copy(rm);
        }
        rm.end_copy();
    };
    // every CTA of the cluster is there before another writes its shared memory
    if (g.parts > 1) cluster_sync();
    grid_wait();
    grid_release();
    for (int i = 0; i < (W ? p.depth : p.depth - 1); ++i) issue();  // as in norm_kernel
    rm.keep(p.vec_at[0], p.post_w, 1);
    rm.keep(p.vec_at[1], p.post_b, 1);
    rm.keep(p.vec_at[2], p.pre_w, 1);
    rm.keep(p.vec_at[4], one_gate, p.gate.cs);
    // a gate row per row of y: its gradient
    auto store_gate = [&](const float (&u)[8 * C]) {
        if constexpr (W > 0) {
            auto typed = [&](auto tag) {
                constexpr int TYPE = decltype(tag)::value, E = TYPE == T_F32 ? 4 : 2;
                char* const to = const_cast<char*>(static_cast<const char*>(g.dgate.data)) + (gate.row * g.dgate.rs + col) * E;
#pragma unroll
                for (int k = 0; k < 8 * C / W; ++k)
                    if (rm.there(W * k)) store_bits<TYPE, W>(to + k * T * W * E, u + W * k);
            };
            if (p.gate_type == T_F32)
                typed(std::integral_constant<int, T_F32>());
            else if (p.gate_type == T_F16)
                typed(std::integral_constant<int, T_F16>());
            else
                typed(std::integral_constant<int, T_BF16>());
        } else {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i)
                if (rm.column(i) < D)
                    store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate.row * g.dgate.rs + rm.column(i) * g.dgate.cs, u[i]);
        }
    };
    float4 next = *stats_at;
    const float over_d = 1.f / D;
    for (long long row = begin; row < end; ++row) {
        float y[8 * C], h[8 * C], d[8 * C], e[8 * C], u[8 * C], gv[8 * C];
        const float4 stats = next;
        if (row + 1 < end) next = *++stats_at;
        auto get = [&](int i, float w) { gv[i] = w; };
        if (!ALL && p.gate.data && (p.depth == 0 || p.vec_bytes == 0)) {  // read where it lies, which leaves out what is past the end
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) gv[i] = 0.f;
        }
        if (ALL || p.depth > 0) {
            uint32_t from = rm.here();
            rm.arrived(shared.group);
            if constexpr (W == 0) issue();
            in_y.template take<true>(rm, from, [&](int i, float w) { y[i] = w; });
            in_x.template take<ALL>(rm, from, [&](int i, float w) { h[i] = w; });
            in_h.template take<ALL>(rm, from, [&](int i, float w) { d[i] = w; });
            in_n.template take<ALL>(rm, from, [&](int i, float w) { e[i] = w; });
            in_gate.take(rm, from, get);
            if constexpr (W > 0) issue();
        } else {
            load_row<TY, W, C>(p.y, row, T, t, base, D, y);
            if (p.x.data) load_row<TX, W, C>(p.x, row, T, t, base, D, h);
            if (g.dh.data) load_row<TX, W, C>(g.dh, row, T, t, base, D, d);
            if (g.dn.data) load_row<TY, W, C>(g.dn, row, T, t, base, D, e);
            if (row_gate) with_vector<W, C>(p.gate.data, p.gate_type, gate.row * p.gate.rs, p.gate.cs, T, t, base, D, get);
        }
        rm.template each<ALL>(p.vec_at[4], one_gate, get, p.gate.cs);
        // y becomes yhat, u what the gate multiplies, h the sum and then hhat.  What
        // they are past the row's end meets zeros of dn, or of d below.
        if constexpr (POST) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) y[i] = (y[i] - stats.x) * stats.y;
        }
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) u[i] = y[i];
        if constexpr (POST) {
            rm.template each<ALL>(p.vec_at[0], p.post_w, [&](int i, float w) { u[i] *= w; });
            rm.template each<ALL>(p.vec_at[1], p.post_b, [&](int i, float w) { u[i] += w; });
        }
        if (ALL || g.dn.data) {
            if (!ALL && !p.x.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) h[i] = 0.f;
            }
            if (p.gate.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) h[i] = fmaf(p.scale, gv[i] * u[i], h[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) h[i] = fmaf(p.scale, u[i], h[i]);
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) h[i] = (h[i] - stats.z) * stats.w;
            if (g.slot[0] >= 0) sums.add(0, g.slot[0], e, h);
            if (g.slot[1] >= 0) sums.add(1, g.slot[1], e);
            rm.template each<ALL>(p.vec_at[2], p.pre_w, [&](int i, float w) { e[i] *= w; });
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
            if (ALL || g.dh.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) d[i] = fmaf(stats.w, e[i], d[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) d[i] = stats.w * e[i];
            }
        }
        out_x.store(rm, g.dx, d);
        if (p.scale != 1.f) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] *= p.scale;
        }
        if (p.gate.data) {
            if (g.gate_sums) {
                sums.add(4, g.slots, d, u);
            } else if (g.dgate.data) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) u[i] *= d[i];
                store_gate(u);
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] *= gv[i];
        }
        if constexpr (POST) {
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] = rm.there(i) ? d[i] : 0.f;
            if (g.slot[2] >= 0) sums.add(2, g.slot[2], d, y);
            if (g.slot[3] >= 0) sums.add(3, g.slot[3], d);
            rm.template each<ALL>(p.vec_at[0], p.post_w, [&](int i, float w) { d[i] *= w; });
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) a = fmaf(d[i], y[i], a);
            float m0 = 0.f, m1;
            if (p.post == NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) b += d[i];
                const float2 s = shared.template sum<true>(a, b);
                m1 = s.x * over_d;
                m0 = s.y * over_d;
            } else {
                m1 = shared.template sum<false>(a, 0.f).x * over_d;
            }
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) d[i] = stats.y * fmaf(-m1, y[i], d[i] - m0);
        }
        out_y.store(rm, g.dy, d);
        // the last row of a gate row, or of this CTA
        if (g.gate_sums && (row + 1 == end || gate.left == 1)) {
            const bool begins = gate.row * p.group_rows >= begin, ends = (gate.row + 1) * p.group_rows <= end;
            float* const to = g.gate_part + (cta * 2 + begins) * D;
            sums.get(4, g.slots, u);
            sums.zero(4, g.slots);
#pragma unroll
            for (int i = 0; i < 8 * C; ++i) {
                const int c = rm.column(i);
                if (c >= D) continue;
                if (begins && ends)
                    store_any(const_cast<void*>(g.dgate.data), p.gate_type, gate.row * g.dgate.rs + c * g.dgate.cs, u[i]);
                else
                    to[c] = u[i];
            }
        }
        gate.next();
        in_gate.next();
    }
    copies_wait(0);
#pragma unroll
    for (int which = 0; which < 4; ++which) {
        if (g.slot[which] < 0) continue;
        float* const to = g.part + (cta * g.slots + g.slot[which]) * D;
        float u[8 * C];
        sums.get(which, g.slot[which], u);
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            const int c = rm.column(i);
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
    RowGroup group{T, t, 0, 0, buffer};
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
            const float2 s = group.sum<true>(a, b);
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
            const float2 s = group.sum<true>(a, b);
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
// or a gate row past those; 32 columns a CTA, 8 warps take every 8th part, with
// 20 loads of a thread under way.
template <int DUMMY>
__global__ void __launch_bounds__(256) norm_finish_kernel(const __grid_constant__ NormFinishParams p) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_wait();
    grid_release();
    for (int what = blockIdx.y; what < p.slots + p.groups; what += gridDim.y) {
        const bool gate = what >= p.slots;
        const int group = what - p.slots;
        int first = 0, last = p.ctas - 1;
        if (gate && p.M > 0) {
            // the CTAs that hold the group's first and last row
            const long long r0 = group * p.group_rows, r1 = r0 + p.group_rows - 1;
            first = static_cast<int>(r0 * p.ctas / p.M);
            while (norm_row(p.M, p.ctas, first + 1) <= r0) ++first;
            last = static_cast<int>(r1 * p.ctas / p.M);
            while (norm_row(p.M, p.ctas, last + 1) <= r1) ++last;
            if (first == last) continue;  // that CTA has written it
        }
        float s = 0.f;
        if (c < p.D) {
            // a gate row begins in its first CTA, whose share lies in the second half
            const float* at = (gate ? p.gate_part : p.part + static_cast<long long>(what) * p.D) + c;
            const long long step = static_cast<long long>(gate ? 2 : p.slots) * p.D;
            if (gate && warp == 0 && p.M > 0) s = at[first * step + p.D];
            at += (first + warp) * step;
            for (int k = first + warp; k <= last; k += 160) {
                float v[20];
#pragma unroll
                for (int j = 0; j < 20; ++j, at += 8 * step) v[j] = k + 8 * j <= last && !(gate && k + 8 * j == first) ? *at : 0.f;
#pragma unroll
                for (int j = 0; j < 20; ++j) s += v[j];
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

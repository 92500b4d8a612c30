// Activations, their derivatives, and dropout's random numbers.
#pragma once
#include "../csrc_fp8/fp8_elem.cuh"

namespace gct {
namespace block {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two values at once: packed fp32 arithmetic issues once for both, each rounded to
// nearest as by itself; the special functions take one after the other.
struct Two {
    unsigned long long v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
    __device__ __forceinline__ void get(float& a, float& b) const { fp8::unpack_f32x2(v, a, b); }
    template <typename F>
    __device__ __forceinline__ Two map(F f) const {
        float a, b;
        get(a, b);
        return Two(f(a), f(b));
    }
};
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    Two d;
    d.v = fp8::fma_f32x2(a.v, b.v, c.v);
    return d;
}

constexpr float LOG2E = 1.44269504088896f;
constexpr float GELU_ROOT = 1.59576912160573f;  // 2 sqrt(2 / pi)
constexpr float GELU_CUBE = 0.044715f;

// 1 / (1 + 2^t)
__device__ __forceinline__ Two falling(Two t) {
    return (t.map([](float x) { return exp2_approx(x); }) + Two(1.f)).map([](float x) { return rcp_approx(x); });
}
// Half of 1 + tanh of gelu's argument is a sigmoid of twice that
__device__ __forceinline__ Two gelu_tanh_sigmoid(Two z, Two z2) {
    return falling(z * fma(z2, Two(-LOG2E * GELU_ROOT * GELU_CUBE), Two(-LOG2E * GELU_ROOT)));
}

// The upper tail of the normal distribution at |z|: half of erfc(x), x = |z| /
// sqrt(2), as exp(-x^2) times a polynomial in t = 1 / (1 + 0.37 x) (the form of
// Hastings' approximations; these coefficients are a least-maximum fit to
// exp(x^2) erfc(x) / 2, relative error 7e-7).  `e` is exp(-z^2 / 2).  Small tails
// keep their relative precision, which 1 + erf(x) of a negative x loses.
__device__ __forceinline__ Two normal_tail(Two z, Two& e) {
    const Two size = z.map([](float x) { return fabsf(x); });
    const Two t = fma(Two(0.37f * 0.70710678118655f), size, Two(1.f)).map([](float x) { return rcp_approx(x); });
    e = (z * z * Two(-0.5f * LOG2E)).map([](float x) { return exp2_approx(x); });
    Two g = fma(Two(0.5f * -0.14294943f), t, Two(0.5f * 0.43710686f));
    g = fma(g, t, Two(0.5f * -0.18854363f));
    g = fma(g, t, Two(0.5f * 0.31898374f));
    g = fma(g, t, Two(0.5f * 0.15202124f));
    g = fma(g, t, Two(0.5f * 0.21501255f));
    g = fma(g, t, Two(0.5f * 0.20836934f));
    return g * t * e;
}
// Phi(z) from the tail at |z|
__device__ __forceinline__ Two normal_below(Two z, Two tail) {
    float z0, z1, t0, t1;
    z.get(z0, z1);
    tail.get(t0, t1);
    return Two(z0 < 0.f ? t0 : 1.f - t0, z1 < 0.f ? t1 : 1.f - t1);
}

template <int ACT>
__device__ __forceinline__ Two act_of(Two z) {
    if (ACT == ACT_RELU) return z.map([](float x) { return x < 0.f ? 0.f : x; });  // NaN stays
    if (ACT == ACT_GELU) {
        Two e;
        return z * normal_below(z, normal_tail(z, e));
    }
    if (ACT == ACT_GELU_TANH) return z * gelu_tanh_sigmoid(z, z * z);
    if (ACT == ACT_SILU) return z * falling(z * Two(-LOG2E));
    return z;
}
template <int ACT>
__device__ __forceinline__ Two act_grad_of(Two z) {
    if (ACT == ACT_RELU) return z.map([](float x) { return x > 0.f ? 1.f : x == x ? 0.f : x; });
    if (ACT == ACT_GELU) {
        Two e;
        const Two below = normal_below(z, normal_tail(z, e));
        return fma(Two(0.398942280401433f) * z, e, below);
    }
    if (ACT == ACT_GELU_TANH) {
        const Two z2 = z * z, s = gelu_tanh_sigmoid(z, z2);
        const Two rest = fma(s * Two(-1.f), s, s);  // s (1 - s): 0 past 16, where its factor must not overflow
        const Two q = z2.map([](float x) { return fminf(x, 256.f); });
        return fma(z * rest, fma(q, Two(3.f * GELU_CUBE * GELU_ROOT), Two(GELU_ROOT)), s);
    }
    if (ACT == ACT_SILU) {
        const Two s = falling(z * Two(-LOG2E));
        return fma(z, fma(s * Two(-1.f), s, s), s);
    }
    return Two(1.f);
}
// one of them for N values, chosen once
template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], int act) {
    auto all = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; i += 2) f(Two(v[i], v[i + 1])).get(v[i], v[i + 1]);
    };
    switch (act) {
        case ACT_RELU: all([](Two z) { return act_of<ACT_RELU>(z); }); break;
        case ACT_GELU: all([](Two z) { return act_of<ACT_GELU>(z); }); break;
        case ACT_GELU_TANH: all([](Two z) { return act_of<ACT_GELU_TANH>(z); }); break;
        case ACT_SILU: all([](Two z) { return act_of<ACT_SILU>(z); }); break;
        default: break;
    }
}
// g times the derivative at z
template <int N>
__device__ __forceinline__ void apply_act_grad(float (&g)[N], const float (&z)[N], int act) {
    auto all = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; i += 2) (Two(g[i], g[i + 1]) * f(Two(z[i], z[i + 1]))).get(g[i], g[i + 1]);
    };
    switch (act) {
        case ACT_RELU: all([](Two v) { return act_grad_of<ACT_RELU>(v); }); break;
        case ACT_GELU: all([](Two v) { return act_grad_of<ACT_GELU>(v); }); break;
        case ACT_GELU_TANH: all([](Two v) { return act_grad_of<ACT_GELU_TANH>(v); }); break;
        default: all([](Two v) { return act_grad_of<ACT_SILU>(v); }); break;
    }
}

// Dropout.  Element (i, j) has 16 random bits: lane j % 8 of Philox4x32-10
// (Salmon, Moraes, Dror and Shaw, 2011) under the seed as key, with counter
// (j / 8, i, offset).  It is kept where they are at least `least` =
// rint(65536 p), so the mask is a function of the element's place and never
// stored.  16 bits an element halve the rounds that 32 would need: ten rounds
// are 20 wide multiplications for 8 elements.
struct Drop {
    const long long* rng;  // seed, offset
    uint32_t least;        // 0: nothing is dropped
    uint32_t limit;        // (least << 16) - 1: upper 16 bits are at least `least` where a word is above it
    float scale;           // 1 / (1 - least / 65536), or 0
};
struct DropKey {
    uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const Drop& d) {
    DropKey k{0u, 0u, 0u, 0u};
    if (d.least) {
        const unsigned long long s = static_cast<unsigned long long>(d.rng[0]), o = static_cast<unsigned long long>(d.rng[1]);
        k = DropKey{static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(o), static_cast<uint32_t>(o >> 32)};
    }
    return k;
}
// the random bits of elements (row, 8 group .. 8 group + 7), two to a word
__device__ __forceinline__ void philox8(const DropKey& key, uint32_t group, uint32_t row, uint32_t (&w)[4]) {
    uint32_t c0 = group, c1 = row, c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}
// by element 0 .. 7 of a group: even ones have the lower half of a word
__device__ __forceinline__ bool kept(const uint32_t (&w)[4], int e, const Drop& d) {
    return ((e & 1) ? w[e >> 1] : w[e >> 1] << 16) > d.limit;
}
// v[0..7] are the elements of one group; dropped ones become 0 whatever they were
__device__ __forceinline__ void drop8(float* v, const Drop& d, const DropKey& key, uint32_t group, uint32_t row) {
    uint32_t w[4];
    philox8(key, group, row, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = kept(w, e, d) ? v[e] * d.scale : 0.f;
}
__device__ __forceinline__ float load_any(const void* p, int type, long long i) {
    if (type == fp8::T_F32) return fp8::load_elem<fp8::T_F32>(p, i);
    return type == fp8::T_F16 ? fp8::load_elem<fp8::T_F16>(p, i) : fp8::load_elem<fp8::T_BF16>(p, i);
}
__device__ __forceinline__ void store_any(void* p, int type, long long i, float v) {
    if (type == fp8::T_F32)
        static_cast<float*>(p)[i] = v;
    else if (type == fp8::T_F16)
        static_cast<__half*>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace block
}  // namespace gct

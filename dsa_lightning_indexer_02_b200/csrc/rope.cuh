// Rotary positions: y[t,h] = x[t,h] with R = 2n dims of each head turned pairwise by the angles
// pos[t] * inv_freq[i], i < n, and scaled by mscale; the gradient is the same with the angle's sign
// changed (the rotation's transpose).
//   half layout         pairs (off + i, off + n + i)
//   interleaved layout  pairs (off + 2i, off + 2i + 1)
//
// The angle is held in turns as a 64-bit binary fraction: with f = frac(inv_freq / 2 pi) * 2^64, the
// product pos * f modulo 2^64 is the position's turn exactly up to f's own rounding (a double's 53
// bits), whatever the position; a far position costs no precision, no table and no wide reduction.
//
// Bound by memory: every element is read once and written once, 16 bytes per access.  A thread owns
// 8 pairs (bf16; 4 in fp32) of one token and applies their 8 sines and cosines to several heads, so
// that the turns cost a few instructions per element.
//
// Measured: 131072 tokens of 32 heads x 128, bf16, out of a fused projection 336-339 us, 98 % of the copy rate; the
// gradient for 32768 tokens of 32 heads x 64 with 32 dims turned 43 us (97 %); 4095 tokens of 4 heads x 128 in fp32
// 4.7 us and 16 of 32 x 128 in bf16 2.5 us, of which an empty kernel takes 2.2.
#pragma once

#include "ptx.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;      // heads whose loads a thread has in flight together
constexpr int kRopeMostHeads = 8;  // heads that share a thread's sines, where there are many tokens

struct RopeParams {
    const void* x;
    void* out;
    const int* pos;          // [T], or null: pos0 + t
    const double* inv_freq;  // [n]
    long long pos0;
    long long T;
    long long x_ts, x_hs, out_ts, out_hs;  // elements between tokens and between heads
    int H, n, off;
    float mscale;
    int inverse;
    int rot_units;   // units of a head that turn (two vectors of 16 bytes each)
    int copy_vecs;   // vectors of 16 bytes of a head that are copied (0 when x and out are the same)
    int units;       // rot_units + the copied vectors in pairs
    int head_slots;  // heads that a block works on at a time
    int tokens;      // tokens that a block works on at a time
};

// f = frac(inv_freq / 2 pi) * 2^64, rounded down.
__device__ __forceinline__ unsigned long long rope_turn(double inv_freq) {
    const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of the angle phase / 2^32 turns.  The quadrant is taken off the integer, so that the
// remainder r, |r| <= pi / 4, keeps fp32's relative precision; Taylor's series to r^9 and r^10 then leave
// 2^-28, and with fp32's roundings each result is off by 2^-23 at most.
__device__ __forceinline__ void rope_sincos(uint32_t phase, float& c, float& s) {
    const uint32_t quad = (phase + 0x20000000u) >> 30;
    const float r = static_cast<float>(static_cast<int>(phase - (quad << 30))) * 1.4629180792671596e-9f;  // pi / 2^31
    const float q = r * r;
    const float ps = fmaf(q, fmaf(q, fmaf(q, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    const float pc = fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f);
    const float sr = fmaf(r * q, ps, r), cr = fmaf(q, pc, 1.f);
    const bool odd = quad & 1;
    c = __uint_as_float(__float_as_uint(odd ? sr : cr) ^ (((quad + 1) & 2) << 30));
    s = __uint_as_float(__float_as_uint(odd ? cr : sr) ^ ((quad & 2) << 30));
}

// The same by the hardware's sine and cosine, whose absolute error on [-pi, pi] stays below 2^-21: for
// results that are rounded to bf16 (half a step is 2^-9 of the value at least).
__device__ __forceinline__ void rope_sincos_fast(uint32_t phase, float& c, float& s) {
    __sincosf(static_cast<float>(static_cast<int>(phase)) * 1.4629180792671596e-9f, &s, &c);  // pi / 2^31
}

template <typename T>
struct RopeElem;
template <>
struct RopeElem<__nv_bfloat16> {
    static constexpr int V = 8;  // elements per 16 bytes
    static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ void sincos(uint32_t ph, float& c, float& s) { rope_sincos_fast(ph, c, s); }
};
template <>
struct RopeElem<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ void sincos(uint32_t ph, float& c, float& s) { rope_sincos(ph, c, s); }
};

// A unit is two vectors a, b of 16 bytes (V elements each) of one head.  Turned units: in the half
// layout a holds the first members of V pairs and b the second; interleaved, a and b are adjacent and
// hold V / 2 pairs each.  Copied units: two of the vectors outside [off, off + 2n), bits as they are.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const RopeParams P) {
    using E = RopeElem<T>;
    constexpr int V = E::V;
    const int per_token = P.units * P.head_slots;
    const int u = threadIdx.x % P.units;
    const int h0 = threadIdx.x / P.units % P.head_slots;
    const int tl = threadIdx.x / per_token;
    if (tl >= P.tokens) return;

    const bool turned = u < P.rot_units;
    int a, b;  // element offsets of the two vectors in a head; b < 0: none
    if (turned) {
        a = P.off + (INTER ? 2 * u * V : u * V);
        b = INTER ? a + V : a + P.n;
    } else {
        const int half = P.units - P.rot_units, v0 = u - P.rot_units, v1 = v0 + half, lead = P.off / V;
        a = v0 < lead ? v0 * V : v0 * V + 2 * P.n;
        b = v1 < P.copy_vecs ? (v1 < lead ? v1 * V : v1 * V + 2 * P.n) : -1;
    }
    unsigned long long f[V];
    if (turned) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = rope_turn(P.inv_freq[u * V + i]);
    }
    const T* x = static_cast<const T*>(P.x);
    T* out = static_cast<T*>(P.out);
    const long long t0 = (long long)blockIdx.x * P.tokens + tl, dt = (long long)gridDim.x * P.tokens;
    long long pos = t0 < P.T ? (P.pos ? (long long)P.pos[t0] : P.pos0 + t0) : 0;
    for (long long t = t0; t < P.T; t += dt) {
        const T* xt = x + t * P.x_ts;
        T* ot = out + t * P.out_ts;
        uint4 va[kRopeBatch], vb[kRopeBatch];
        auto load = [&](int hb) {
#pragma unroll
            for (int i = 0; i < kRopeBatch; ++i) {
                const int h = hb + i * P.head_slots;
                if (h >= P.H) break;
                va[i] = *reinterpret_cast<const uint4*>(xt + h * P.x_hs + a);
                if (b >= 0) vb[i] = *reinterpret_cast<const uint4*>(xt + h * P.x_hs + b);
            }
        };
        load(h0);  // in flight while the sines are made
        float c[V], s[V];
        if (turned) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                E::sincos(static_cast<uint32_t>((static_cast<unsigned long long>(pos) * f[i]) >> 32), c[i], s[i]);
                c[i] *= P.mscale;
                s[i] *= P.inverse ? -P.mscale : P.mscale;
            }
        }
        if (t + dt < P.T) pos = P.pos ? (long long)P.pos[t + dt] : P.pos0 + t + dt;
        for (int hb = h0; hb < P.H; hb += P.head_slots * kRopeBatch) {
            if (hb != h0) load(hb);
#pragma unroll
            for (int i = 0; i < kRopeBatch; ++i) {
                const int h = hb + i * P.head_slots;
                if (h >= P.H) break;
                if (turned) {
                    float p[V], q[V], y[V], z[V];
                    E::unpack(va[i], p);
                    E::unpack(vb[i], q);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (INTER) {  // pair j: the adjacent elements 2j, 2j + 1 of a|b
                            const float e0 = j < V / 2 ? p[2 * j % V] : q[2 * j % V];
                            const float e1 = j < V / 2 ? p[(2 * j + 1) % V] : q[(2 * j + 1) % V];
                            const float r0 = e0 * c[j] - e1 * s[j], r1 = e0 * s[j] + e1 * c[j];
                            if (j < V / 2) y[2 * j % V] = r0, y[(2 * j + 1) % V] = r1;
                            else z[2 * j % V] = r0, z[(2 * j + 1) % V] = r1;
                        } else {
                            y[j] = p[j] * c[j] - q[j] * s[j];
                            z[j] = p[j] * s[j] + q[j] * c[j];
                        }
                    }
                    va[i] = E::pack(y);
                    vb[i] = E::pack(z);
                }
                *reinterpret_cast<uint4*>(ot + h * P.out_hs + a) = va[i];
                if (b >= 0) *reinterpret_cast<uint4*>(ot + h * P.out_hs + b) = vb[i];
            }
        }
    }
}

}  // namespace dsa

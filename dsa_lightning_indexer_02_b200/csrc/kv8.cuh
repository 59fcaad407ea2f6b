// The paged 8-bit KV cache: its formats, and the kernel that appends tokens to it.
//
// A page holds `page` tokens of one sequence, [page][Hkv][128] bytes for K and as many for V; token
// pos of sequence b lies in page page_table[b][pos / page], slot pos mod page.  Every (page, KV head)
// has one scale for K and one for V, a power of two 2^e: a stored byte stands for 2^e times its e4m3
// or int8 value.  e is the least with amax <= 448 * 2^e (e4m3) or 127 * 2^e (int8), so that nothing
// saturates; a page's slot 0 sets its scale, later tokens may only raise it, and the tokens that the
// page holds already are then rounded again.  Powers of two make that second rounding exact in e4m3
// (down to its subnormals), cost e4m3 no precision, and make every stored value exact in bf16 and,
// unscaled, in fp16.
//
// Append: one block per touched page for K and one for V; the page's new rows stay in registers
// (packed bf16) between the pass that finds each head's largest magnitude and the pass that rounds,
// so every input is read once and every byte written once.  The block's sines and cosines are made
// once per (token, pair) in shared memory and serve all its KV heads.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rope.cuh"

namespace dsa {

constexpr int kKvD = 128;
constexpr int kKvEMin = -64;       // least scale exponent (an all-zero block gets it)
constexpr int kKvUnits = 16;       // 8-dim units of a token and head
constexpr int kAppendPasses = 16;  // units per thread of the append kernel

enum { KV_E4M3 = 0, KV_INT8 = 1 };

struct AppendParams {
    const __nv_bfloat16 *k_new, *v_new;  // [N, Hkv, 128]
    long long k_ts, k_hs, v_ts, v_hs;    // elements between tokens and heads
    uint8_t *k_pages, *v_pages;          // [num_pages, page, Hkv, 128]
    float *k_scale, *v_scale;            // [num_pages, Hkv]
    const int* table;                    // [B, max_pages]
    const int* ctx_len;                  // [B]
    const int* cu_new;                   // [B + 1], or null: one token each
    const int* rope_pos;                 // [N], or null: the cache position
    const double* inv_freq;              // [n], null when n == 0
    int B, N, Hkv, page_shift, max_pages, num_pages;
    int n, off, inter;
    float mscale;
};

// The power of two of a block whose largest magnitude is amax: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6,
// compared on the bits, hence exactly.
template <int FMT>
__device__ __forceinline__ int kv_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int x = static_cast<int>(bits >> 23) - 127;
    const uint32_t most = FMT == KV_E4M3 ? 0x600000u : 0x7e0000u;
    const int e = x - (FMT == KV_E4M3 ? 8 : 6) + ((bits & 0x7fffffu) > most ? 1 : 0);
    return max(e, kKvEMin);
}
__device__ __forceinline__ float kv_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Four values, already divided by the scale, to four bytes; nearest, ties to even, saturating.
// int8 has no NaN: it becomes 0 (the caller reports it).
template <int FMT>
__device__ __forceinline__ uint32_t kv_round4(float a, float b, float c, float d) {
    if constexpr (FMT == KV_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    } else {
        auto r = [](float v) { return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(v == v ? v : 0.f, -127.f), 127.f))) & 255u; };
        return r(a) | r(b) << 8 | r(c) << 16 | r(d) << 24;
    }
}
// Four stored bytes as floats.
template <int FMT>
__device__ __forceinline__ void kv_value4(uint32_t w, float (&f)[4]) {
    if constexpr (FMT == KV_E4M3) {
        const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3));
        const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3));
        const float2 a = __half22float2(lo), b = __half22float2(hi);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    }
}

// Which page a block fills: sequence b, its page number pj, tokens [i0, i1) of the input at cache
// positions starting with p0.  Sequence b owns the blocks cu[b] / page + 2 b and on, which are as many
// as n new tokens can touch: at most n / page + 2 pages.
struct AppendSpan {
    int b, pj, i0, i1, p0;
    bool any;
};
__device__ __forceinline__ AppendSpan append_span(const AppendParams& P, int unit, int lane) {
    AppendSpan S{};
    int i0, n, j;
    if (!P.cu_new) {
        S.b = unit, i0 = unit, n = 1, j = 0;
    } else {
        // the last sequence whose first block is not behind this one, 32 candidates a step
        int lo = 0, hi = P.B;  // the answer lies in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) >> 5;
            const int b = lo + lane * step;
            const bool ok = b < hi && (P.cu_new[b] >> P.page_shift) + 2 * b <= unit;
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            const int last = m ? 31 - __clz(m) : 0;
            lo += last * step;
            hi = min(hi, lo + step);
        }
        S.b = lo;
        i0 = P.cu_new[lo];
        const int i1 = P.cu_new[lo + 1];
        if (i0 < 0 || i1 < i0 || i1 > P.N) {
            record_error(DSA_DEV_ERR_BOUNDS, 0xa01);
            return S;
        }
        n = i1 - i0;
        j = unit - (i0 >> P.page_shift) - 2 * lo;
    }
    if (n <= 0 || j < 0) return S;
    const int ctx = P.ctx_len[S.b];
    const long long cap = (long long)P.max_pages << P.page_shift;
    if (ctx < 0 || (long long)ctx + n > cap) {
        record_error(DSA_DEV_ERR_BOUNDS, 0xa02);
        return S;
    }
    const int pj = (ctx >> P.page_shift) + j;
    const long long first = (long long)pj << P.page_shift;
    const int p0 = (int)max((long long)ctx, first);
    const int p1 = (int)min((long long)ctx + n, first + (1ll << P.page_shift));
    if (p1 <= p0) return S;
    S.pj = pj, S.p0 = p0, S.i0 = i0 + (p0 - ctx), S.i1 = i0 + (p1 - ctx), S.any = true;
    return S;
}

template <int FMT>
__global__ void __launch_bounds__(512) kv_append_kernel(const AppendParams P) {
    extern __shared__ __align__(16) float2 s_turn[];  // [tokens][n]: cos, sin (K blocks)
    __shared__ unsigned s_amax[4];
    __shared__ float s_old[4], s_new[4];
    const int lane = threadIdx.x & 31;
    const AppendSpan S = append_span(P, blockIdx.x, lane);
    if (!S.any) return;
    const bool is_k = blockIdx.y == 0;
    const int Hkv = P.Hkv, page = 1 << P.page_shift;
    const int pid = P.table[(long long)S.b * P.max_pages + S.pj];
    if (pid < 0 || pid >= P.num_pages) {
        if (threadIdx.x == 0) record_error(DSA_DEV_ERR_BOUNDS, 0xa03);
        return;
    }
    uint8_t* pages = (is_k ? P.k_pages : P.v_pages) + (long long)pid * page * Hkv * kKvD;
    float* scale = (is_k ? P.k_scale : P.v_scale) + (long long)pid * Hkv;
    const __nv_bfloat16* x = is_k ? P.k_new : P.v_new;
    const long long ts = is_k ? P.k_ts : P.v_ts, hs = is_k ? P.k_hs : P.v_hs;
    const int tokens = S.i1 - S.i0, slot0 = S.p0 & (page - 1);
    const int n = is_k ? P.n : 0;
    if (threadIdx.x < Hkv) {
        s_amax[threadIdx.x] = 0u;
        s_old[threadIdx.x] = slot0 ? scale[threadIdx.x] : 0.f;
    }

    // unit i of this thread: row (token, head) of the page, dims 8 d8 .. 8 d8 + 7
    const int d8 = threadIdx.x & (kKvUnits - 1);
    const int row0 = threadIdx.x / kKvUnits, rows = tokens * Hkv, step = blockDim.x / kKvUnits;
    uint4 raw[kAppendPasses];
#pragma unroll
    for (int i = 0; i < kAppendPasses; ++i) {
        const int r = row0 + i * step;
        if (r < rows)
            raw[i] = *reinterpret_cast<const uint4*>(x + (long long)(S.i0 + r / Hkv) * ts + (r % Hkv) * hs + d8 * 8);
    }
    if (n) {
        for (int e = threadIdx.x; e < tokens * n; e += blockDim.x) {
            const int t = e / n, p = e % n;
            const long long pos = P.rope_pos ? P.rope_pos[S.i0 + t] : S.p0 + t;
            float c, s;
            rope_sincos((uint32_t)((static_cast<unsigned long long>(pos) * rope_turn(P.inv_freq[p])) >> 32), c, s);
            s_turn[e] = make_float2(c * P.mscale, s * P.mscale);
        }
    }
    __syncthreads();

    // the row's 8 values in fp32, turned (all lanes of the warp take part)
    const int a8 = P.off / 8, n8 = n / 8;
    const bool turned = n && d8 >= a8 && d8 < a8 + 2 * n8;
    const bool second = turned && !P.inter && d8 >= a8 + n8;
    const int src = (lane & 16) | (turned && !P.inter ? (second ? d8 - n8 : d8 + n8) : d8);
    auto values = [&](const uint4& v, int r, float (&f)[8]) {
        RopeElem<__nv_bfloat16>::unpack(v, f);
        if (!n) return;
        if (P.inter) {
            if (!turned) return;
            const float2* cs = s_turn + (r / Hkv) * n + (d8 - a8) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 t = cs[j];
                const float e0 = f[2 * j], e1 = f[2 * j + 1];
                f[2 * j] = e0 * t.x - e1 * t.y;
                f[2 * j + 1] = e0 * t.y + e1 * t.x;
            }
        } else {
            uint4 w;
            w.x = __shfl_sync(0xffffffffu, v.x, src), w.y = __shfl_sync(0xffffffffu, v.y, src);
            w.z = __shfl_sync(0xffffffffu, v.z, src), w.w = __shfl_sync(0xffffffffu, v.w, src);
            if (!turned) return;
            float g[8];
            RopeElem<__nv_bfloat16>::unpack(w, g);
            const float2* cs = s_turn + (r / Hkv) * n + (second ? d8 - a8 - n8 : d8 - a8) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 t = cs[j];
                f[j] = second ? g[j] * t.y + f[j] * t.x : f[j] * t.x - g[j] * t.y;
            }
        }
    };

    // pass 1: the largest finite magnitude of each head
    const int passes = (rows + step - 1) / step;  // uniform over the block
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kAppendPasses; ++i) {
        if (i >= passes) break;
        const int r = row0 + i * step;
        const bool in = r < rows;
        float f[8];
        values(in ? raw[i] : make_uint4(0, 0, 0, 0), in ? r : 0, f);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fabsf(f[j]);
            if (v < INFINITY) m = fmaxf(m, v);
            nan |= in && !(f[j] == f[j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (in && d8 == 0) atomicMax(&s_amax[r % Hkv], __float_as_uint(m));  // m >= 0: bits keep the order
    }
    if (FMT == KV_INT8 && nan) record_error(DSA_DEV_ERR_BOUNDS, 0xa04);
    __syncthreads();
    if (threadIdx.x < Hkv) {
        const float s = fmaxf(s_old[threadIdx.x], kv_pow2(kv_exponent<FMT>(__uint_as_float(s_amax[threadIdx.x]))));
        s_new[threadIdx.x] = s;
        scale[threadIdx.x] = s;
    }
    __syncthreads();

    // pass 2: round and store the new rows
#pragma unroll
    for (int i = 0; i < kAppendPasses; ++i) {
        if (i >= passes) break;
        const int r = row0 + i * step;
        const bool in = r < rows;
        float f[8];
        values(in ? raw[i] : make_uint4(0, 0, 0, 0), in ? r : 0, f);
        if (!in) continue;
        const float s = s_new[r % Hkv];
        const float inv = 1.f / s;  // a power of two
        uint2 w;
        w.x = kv_round4<FMT>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        w.y = kv_round4<FMT>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        *reinterpret_cast<uint2*>(pages + ((long long)slot0 * Hkv + r) * kKvD + d8 * 8) = w;
    }

    // tokens that the page held before: rounded again where their head's scale grew
    if (!slot0) return;
    for (int e = threadIdx.x; e < slot0 * Hkv * 8; e += blockDim.x) {
        const int h = (e >> 3) % Hkv;
        if (s_old[h] == s_new[h]) continue;
        const float ratio = s_old[h] / s_new[h];
        uint4* at = reinterpret_cast<uint4*>(pages + (long long)(e >> 3) * kKvD) + (e & 7);
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[4];
            kv_value4<FMT>(w[i], f);
            w[i] = kv_round4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace dsa

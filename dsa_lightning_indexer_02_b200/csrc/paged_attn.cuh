// Attention over the paged 8-bit KV cache (kv8.cuh): row t reads keys of sequence seq[t],
//   z_s = scale * 2^ek(s) * sum_d q[t,h,d] k8[s,d],  out = sum_s softmax(z)_s 2^ev(s) v8[s,:]
// over all its n_keys[t] cached keys, or over those that idx names.
#pragma once

#include "kv8.cuh"

namespace dsa {

constexpr int kPagedMaxG = 16;
constexpr int kPagedPartCtas = 296;  // split partials in the workspace: two for each of so many CTAs
constexpr int kPagedPartStride = kKvD + 4;

struct PagedParams {
    const __nv_bfloat16* q;            // [T, Hq, 128]
    const uint8_t *k_pages, *v_pages;  // [num_pages, page, Hkv, 128]
    const float *k_scale, *v_scale;    // [num_pages, Hkv]
    const int* table;                  // [B, max_pages]
    const int* seq;                    // [T], or null: row t is of sequence t
    const int* n_keys;                 // [T]
    const int* idx;                    // [T, topk], or null
    int T, B, num_pages, page_shift, max_pages, Hq, Hkv, topk;
    float scale_log2;
    __nv_bfloat16* out;                // [T, Hq, 128]
    float* lse;                        // [T, Hq], may be null
    float* part;
};

// Sequence and key count of row t; a bad one is reported and leaves the row empty.
__device__ __forceinline__ void paged_row(const PagedParams& P, int t, int& b, int& n) {
    b = P.seq ? P.seq[t] : t;
    n = P.n_keys[t];
    const long long cap = (long long)P.max_pages << P.page_shift;
    if (b < 0 || b >= P.B || n < 0 || n > cap) {
        record_error(DSA_DEV_ERR_BOUNDS, 0xb01);
        b = 0, n = 0;
    }
}

// One block per (row, KV head); each warp takes every fourth key, a lane 4 dims of it.
template <int FMT>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedParams P) {
    __shared__ float sm[4][kPagedMaxG], sl[4][kPagedMaxG], so[4][kPagedMaxG][kKvD];
    const int t = blockIdx.x, g = blockIdx.y, G = P.Hq / P.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int b, n;
    paged_row(P, t, b, n);
    const int count = P.idx ? min(P.topk, n) : n;
    float q[kPagedMaxG][4], o[kPagedMaxG][4], m[kPagedMaxG], l[kPagedMaxG];
#pragma unroll
    for (int h = 0; h < kPagedMaxG; ++h) {
        m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[h][i] = 0.f;
            q[h][i] = h < G ? __bfloat162float(P.q[((long long)t * P.Hq + g * G + h) * kKvD + lane * 4 + i]) : 0.f;
        }
    }
    for (int e = warp; e < count; e += 4) {
        const int key = P.idx ? P.idx[(long long)t * P.topk + e] : e;
        if (key < 0 || key >= n) continue;
        const int pid = P.table[(long long)b * P.max_pages + (key >> P.page_shift)];
        if (pid < 0 || pid >= P.num_pages) {
            record_error(DSA_DEV_ERR_BOUNDS, 0xb02);
            continue;
        }
        const long long slot = ((long long)pid << P.page_shift) + (key & ((1 << P.page_shift) - 1));
        const long long at = (slot * P.Hkv + g) * kKvD + lane * 4;
        float k[4], v[4];
        kv_value4<FMT>(*reinterpret_cast<const uint32_t*>(P.k_pages + at), k);
        kv_value4<FMT>(*reinterpret_cast<const uint32_t*>(P.v_pages + at), v);
        const float ks = P.k_scale[(long long)pid * P.Hkv + g] * P.scale_log2;
        const float vs = P.v_scale[(long long)pid * P.Hkv + g];
#pragma unroll
        for (int h = 0; h < kPagedMaxG; ++h) {
            if (h >= G) break;
            float z = q[h][0] * k[0] + q[h][1] * k[1] + q[h][2] * k[2] + q[h][3] * k[3];
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
            z *= ks;
            const float mn = fmaxf(m[h], z), a = exp2f(m[h] - mn), p = exp2f(z - mn);
            m[h] = mn, l[h] = l[h] * a + p;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[h][i] = o[h][i] * a + p * v[i] * vs;
        }
    }
#pragma unroll
    for (int h = 0; h < kPagedMaxG; ++h) {
        if (h >= G) break;
        if (lane == 0) sm[warp][h] = m[h], sl[warp][h] = l[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) so[warp][h][lane * 4 + i] = o[h][i];
    }
    __syncthreads();
    for (int h = warp; h < G; h += 4) {
        float mx = -INFINITY, sum = 0.f, acc[4] = {};
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, sm[w][h]);
        for (int w = 0; w < 4; ++w) {
            const float a = sm[w][h] == -INFINITY ? 0.f : exp2f(sm[w][h] - mx);
            sum += sl[w][h] * a;
            for (int i = 0; i < 4; ++i) acc[i] += so[w][h][lane * 4 + i] * a;
        }
        const long long row = (long long)t * P.Hq + g * G + h;
        for (int i = 0; i < 4; ++i)
            P.out[row * kKvD + lane * 4 + i] = __float2bfloat16_rn(count && mx != -INFINITY ? acc[i] / sum : 0.f);
        if (P.lse && lane == 0) P.lse[row] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
}

}  // namespace dsa

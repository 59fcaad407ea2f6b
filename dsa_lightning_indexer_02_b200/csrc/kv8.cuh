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
// Append: one block per touched page (of up to 128 rows of a token and head) for K and one for V.  A thread
// owns 16 dims of one, two or four rows, both members of the pairs that it turns; they stay in registers
// between finding each head's largest magnitude and rounding, so every input is read once and every byte
// written once.  The sines and cosines are made once per (token, pair) in shared memory for all heads.
//
// Rounding of turned keys: fp32's own error moves one value in some 10^5 across a border between two 8-bit
// values.  Where the interval of twice that error around a value rounds to two different bytes, the pair is
// computed again in fp64, so the stored byte is the exact product's.  Where a head's largest lies within that error of
// a border between two scales (one in some 2^18, but one in 128 where a slow pair leaves a bf16 value almost as it
// was), the block settles the scale in fp64 when all else is done, and rounds that head's rows again if fp32 had it
// wrong.  Done out of line, this costs a prefill 0.1 us of 23.5; decided before the rows are rounded, 1.9.
//
// Measured: 16 single tokens, 4 KV heads 4.1 us, a launch and two dependent loads more than an empty kernel's 2.2; 61
// chunks of up to 37 tokens, int8 3.4 us; 23 K tokens of 8 sequences 23.6 us, where the bytes alone take 11: bound by
// instructions (issue slots 55 % busy, two blocks of 256 threads an SM): by count of operations a third of a key
// block's make sines, which its two heads share, and a fifth round twice.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rope.cuh"

namespace dsa {

constexpr int kKvD = 128;
constexpr int kKvEMin = -64;       // least scale exponent (an all-zero block gets it)
constexpr int kKvUnits = 8;        // 16-dim units of a row (a token and head)
constexpr int kAppendRows = 128;   // most rows of a block

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
    int n, off, hg_shift;  // hg_shift: log2 of the heads of a block
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
// Whether fp32's error may have put a largest turned magnitude on the wrong side of a border between two scales:
// it is off by 2^-20.9 at most (where bytes are rounded, below), which is less than 16 steps next to a border.
template <int FMT>
__device__ __forceinline__ bool kv_near_border(uint32_t bits) {
    return (bits & 0x7fffffu) - ((FMT == KV_E4M3 ? 0x600000u : 0x7e0000u) - 16u) <= 32u;
}
__device__ __forceinline__ float kv_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Four values, already divided by the scale, to four bytes; nearest, ties to even, saturating.
// int8 has no NaN: it becomes 0 (the caller reports it).
template <int FMT>
__device__ __forceinline__ uint32_t kv_round4(float a, float b, float c, float d) {
    if constexpr (FMT == KV_E4M3) {
        uint32_t w;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
            : "=r"(w)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return w;
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
    int i0, n, j = 0, ctx;
    if (!P.cu_new) {
        S.b = unit, i0 = unit, n = 1, ctx = P.ctx_len[unit];
    } else {
        // the last sequence whose first block is not behind this one: 32 candidates a step, the last step's
        // with what the block needs to know of each
        int lo = 0, hi = P.B;  // the answer lies in [lo, hi)
        while (hi - lo > 32) {
            const int step = (hi - lo + 31) >> 5;
            const int b = lo + lane * step;
            const bool ok = b < hi && (P.cu_new[b] >> P.page_shift) + 2 * b <= unit;
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            const int last = m ? 31 - __clz(m) : 0;
            lo += last * step;
            hi = min(hi, lo + step);
        }
        const int b = min(lo + lane, hi - 1);
        const int c0 = P.cu_new[b], c1 = P.cu_new[b + 1], cx = P.ctx_len[b];
        const unsigned m = __ballot_sync(0xffffffffu, lo + lane < hi && (c0 >> P.page_shift) + 2 * b <= unit);
        const int last = m ? 31 - __clz(m) : 0;
        S.b = lo + last;
        i0 = __shfl_sync(0xffffffffu, c0, last);
        const int i1 = __shfl_sync(0xffffffffu, c1, last);
        ctx = __shfl_sync(0xffffffffu, cx, last);
        if (i0 < 0 || i1 < i0 || i1 > P.N) {
            record_error(DSA_DEV_ERR_BOUNDS, 0xa01);
            return S;
        }
        n = i1 - i0;
        j = unit - (i0 >> P.page_shift) - 2 * S.b;
    }
    if (n <= 0 || j < 0) return S;
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

// Largest of 16 magnitudes; infinities, which it tells of, and NaN do not count.
__device__ __forceinline__ float kv_amax(const float (&f)[16], bool& infinite) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(f[j]));  // passes NaN over
    infinite = m == INFINITY;
    if (infinite) {
        m = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (fabsf(f[j]) < INFINITY) m = fmaxf(m, fabsf(f[j]));
    }
    return m;
}

// y to fp32 so that rounding the result again, to fewer bits, gives what rounding y itself gives: towards
// zero, with the last bit set where anything was cut off.
__device__ __forceinline__ float round_odd(double y) {
    const float r = __double2float_rz(y);
    return static_cast<double>(r) == y || !(y == y) ? r : __uint_as_float(__float_as_uint(r) | 1u);
}

// The bytes of a pair turned by ph / 2^64 turns, in fp64.  Out of line: rarely taken, and long.
template <int FMT>
__device__ __noinline__ uint32_t kv_turn_exact(float e0, float e1, unsigned long long ph, float mscale, float inv) {
    double s, c;
    sincospi(static_cast<double>(static_cast<long long>(ph)) * 1.0842021724855044e-19, &s, &c);  // 2^-63
    const double a = e0, b = e1, m = mscale;
    return kv_round4<FMT>(round_odd(m * (a * c - b * s)) * inv, round_odd(m * (a * s + b * c)) * inv, 0.f, 0.f);
}

// What a block's threads share: per head the largest magnitude's bits, the page's scale before and after, and whether
// an exact product lies above the border that the largest is next to.
struct AppendShared {
    unsigned amax[4];
    float old[4], now[4];
    int over[4];
};

// Settles the scales of heads whose largest magnitude is next to a border, once the rows are rounded: pairs long enough
// to reach the border are turned in fp64, and a head's rows rounded again, every pair in fp64, where its scale changes.
// All threads of a key block call it, each for its own rows (their first token is i0 at position p0); out of line, so
// that the rows' registers are not kept for it.
template <int FMT, bool INTER>
__device__ __noinline__ void kv_settle_scale(const AppendParams& P, AppendShared& sh, const __nv_bfloat16* in, uint8_t* to, float* scale,
                                             int a, int b, int i0, int p0, int rows) {
    const int tid = threadIdx.x, u = tid & (kKvUnits - 1), row0 = tid / kKvUnits, step = blockDim.x / kKvUnits;
    const int hshift = P.hg_shift, hmask = (1 << hshift) - 1, my_h = row0 & hmask;
    const bool turned = u < P.n / 8;
    const float most_of = FMT == KV_E4M3 ? 448.f : 127.f;
    auto lower = [&](int h) { return kv_exponent<FMT>(__uint_as_float(sh.amax[h]) * (1.f - 1.9073486328125e-6f)); };  // 2^-19
    // pair y of row r: where its members stand in the row, and its turn
    auto pair = [&](int y, int& lo, int& hi) {
        lo = INTER ? 2 * y : y, hi = INTER ? 2 * y + 1 : 8 + y;
        lo = lo < 8 ? a + lo : b + lo - 8, hi = hi < 8 ? a + hi : b + hi - 8;
    };
    auto turn = [&](int r, int y) {
        const int t = r >> hshift;
        const long long pos = P.rope_pos ? (long long)P.rope_pos[i0 + t] : (long long)(p0 + t);
        return static_cast<unsigned long long>(pos) * rope_turn(P.inv_freq[u * 8 + y]);
    };
    const float most = most_of * kv_pow2(lower(my_h));
    if (turned && kv_near_border<FMT>(sh.amax[my_h])) {
#pragma unroll 1
        for (int r = row0; r < rows; r += step) {
            const __nv_bfloat16* at = in + (long long)(r >> hshift) * P.k_ts + my_h * P.k_hs;
#pragma unroll 1
            for (int y = 0; y < 8; ++y) {
                int lo, hi;
                pair(y, lo, hi);
                const float e0 = __bfloat162float(at[lo]), e1 = __bfloat162float(at[hi]);
                if (!((e0 * e0 + e1 * e1) * (P.mscale * P.mscale) >= most * most * 0.9999f)) continue;  // a turn keeps its length
                double sn, cs;
                sincospi(static_cast<double>(static_cast<long long>(turn(r, y))) * 1.0842021724855044e-19, &sn, &cs);  // 2^-63
                const double x0 = e0, x1 = e1, m = P.mscale;
                const double y0 = fabs(m * (x0 * cs - x1 * sn)), y1 = fabs(m * (x0 * sn + x1 * cs));
                if ((y0 > most && y0 < INFINITY) || (y1 > most && y1 < INFINITY)) sh.over[my_h] = 1;
            }
        }
    }
    const float before = sh.now[my_h];
    __syncthreads();
    if (tid <= hmask && kv_near_border<FMT>(sh.amax[tid]))
        scale[tid] = sh.now[tid] = fmaxf(sh.old[tid], kv_pow2(max(lower(tid) + sh.over[tid], kKvEMin)));
    __syncthreads();
    const float now = sh.now[my_h];
    if (now == before) return;
#pragma unroll 1
    for (int r = row0; r < rows; r += step) {
        const __nv_bfloat16* at = in + (long long)(r >> hshift) * P.k_ts + my_h * P.k_hs;
        uint8_t* dst = to + (long long)(r >> hshift) * P.Hkv * kKvD;
#pragma unroll 1
        for (int y = 0; y < 8; ++y) {
            int lo, hi;
            pair(y, lo, hi);
            const float e0 = __bfloat162float(at[lo]), e1 = __bfloat162float(at[hi]);
            const uint32_t both = turned ? kv_turn_exact<FMT>(e0, e1, turn(r, y), P.mscale, 1.f / now)
                                         : kv_round4<FMT>(e0 / now, e1 / now, 0.f, 0.f);
            dst[lo] = both & 255u, dst[hi] = both >> 8 & 255u;
        }
    }
}

// PASSES: units of a thread, 1, 2 or 4.
template <int FMT, bool INTER, int PASSES>
__global__ void __launch_bounds__(PASSES == 2 ? 512 : 256, PASSES == 2 ? 1 : 2) kv_append_kernel(const __grid_constant__ AppendParams P) {
    // cos, sin times mscale (K blocks), [tokens][4][n / 8][2]: pairs 2 k, 2 k + 1 of unit u at [k][u], so that the
    // units' 16-byte reads lie side by side
    extern __shared__ __align__(16) float2 s_turn[];
    __shared__ __align__(16) AppendShared sh;
    const int tid = threadIdx.x, lane = tid & 31;
    const bool is_k = (blockIdx.y & 1) == 0;
    const int n = is_k ? P.n : 0, hshift = P.hg_shift, hmask = (1 << hshift) - 1, h0 = (blockIdx.y >> 1) << hshift;
    // the pair whose sines this thread makes, for every tstep-th token, in the order of s_turn
    const int entry = n ? tid % n : 0, tstep = n ? blockDim.x / n : 1, tfirst = n ? tid / n : 0;
    const int pair = n ? (entry / 2 % (n / 8)) * 8 + entry / (n / 4) * 2 + (entry & 1) : 0;
    const double freq = n ? P.inv_freq[pair] : 0.0;

    const AppendSpan S = append_span(P, blockIdx.x, lane);
    if (!S.any) return;
    const int page = 1 << P.page_shift, tokens = S.i1 - S.i0, slot0 = S.p0 & (page - 1);

    // unit u of a row: two vectors of 8 dims, a and b.  Turned: in the half layout the first and the second
    // members of 8 pairs, interleaved 4 adjacent pairs each; otherwise two of the vectors left over.
    const int u = tid & (kKvUnits - 1), turned_units = n / 8;
    const bool turned = u < turned_units;
    int a, b;
    if (turned) {
        a = P.off + (INTER ? 16 * u : 8 * u);
        b = INTER ? a + 8 : a + n;
    } else {
        const int v0 = u - turned_units, v1 = v0 + kKvUnits - turned_units, lead = is_k ? P.off / 8 : 0;
        a = v0 < lead || !n ? v0 * 8 : v0 * 8 + 2 * n;
        b = v1 < lead || !n ? v1 * 8 : v1 * 8 + 2 * n;
    }
    const int row0 = tid / kKvUnits, rows = tokens << hshift, step = blockDim.x / kKvUnits;  // step: whole tokens
    const __nv_bfloat16* in = (is_k ? P.k_new : P.v_new) + (long long)S.i0 * (is_k ? P.k_ts : P.v_ts) +
                             (long long)h0 * (is_k ? P.k_hs : P.v_hs);
    const long long ts = is_k ? P.k_ts : P.v_ts, hs = is_k ? P.k_hs : P.v_hs;
    const int my_h = row0 & hmask;  // the same for all rows of this thread
    uint4 ra[PASSES], rb[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = row0 + i * step;
        if (r < rows) {
            const __nv_bfloat16* at = in + (long long)(r >> hshift) * ts + my_h * hs;
            ra[i] = *reinterpret_cast<const uint4*>(at + a);
            rb[i] = *reinterpret_cast<const uint4*>(at + b);
        }
    }
    const int pid = P.table[(long long)S.b * P.max_pages + S.pj];
    const unsigned long long turn = rope_turn(freq);
    auto position = [&](int t) {
        return static_cast<unsigned long long>(P.rope_pos ? (long long)P.rope_pos[S.i0 + t] : (long long)(S.p0 + t));
    };
    if (n && tfirst < tstep) {
        for (int t = tfirst; t < tokens; t += tstep) {
            float c, s;
            rope_sincos(static_cast<uint32_t>((position(t) * turn) >> 32), c, s);
            s_turn[t * n + entry] = make_float2(c * P.mscale, s * P.mscale);
        }
    }
    if (pid < 0 || pid >= P.num_pages) {
        if (tid == 0) record_error(DSA_DEV_ERR_BOUNDS, 0xa03);
        return;
    }
    uint8_t* pages = (is_k ? P.k_pages : P.v_pages) + (long long)pid * page * P.Hkv * kKvD;
    float* scale = (is_k ? P.k_scale : P.v_scale) + (long long)pid * P.Hkv + h0;
    float old = 0.f;
    if (tid < 4) {
        sh.amax[tid] = 0u;
        sh.over[tid] = 0;
        if (tid <= hmask) old = slot0 ? scale[tid] : 0.f;  // consumed after the pass over the rows
    }
    __syncthreads();

    // the largest finite magnitude of this thread's rows, which are of one head.  Turned keys stay in fp32 from
    // here on (f[0..8) of vector a, f[8..16) of vector b); values, and keys stored as they come, in bf16.
    float f[PASSES][16];
    float m = 0.f;
    bool nan = false;
    unsigned infinite = 0;  // bit i: turned row i has an infinity
    if (n) {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (row0 + i * step >= rows) break;
            float p[8], q[8];
            RopeElem<__nv_bfloat16>::unpack(ra[i], p);
            RopeElem<__nv_bfloat16>::unpack(rb[i], q);
            if (turned) {
                const float4* cs = reinterpret_cast<const float4*>(s_turn + ((row0 + i * step) >> hshift) * n) + u;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float4 t = cs[(x / 2) * turned_units];
                    const float c = x & 1 ? t.z : t.x, s = x & 1 ? t.w : t.y;
                    const float e0 = INTER ? (x < 4 ? p[2 * x % 8] : q[2 * x % 8]) : p[x];
                    const float e1 = INTER ? (x < 4 ? p[(2 * x + 1) % 8] : q[(2 * x + 1) % 8]) : q[x];
                    f[i][INTER ? 2 * x : x] = e0 * c - e1 * s, f[i][INTER ? 2 * x + 1 : 8 + x] = e0 * s + e1 * c;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = p[j], f[i][8 + j] = q[j];
            }
            bool inf;
            m = fmaxf(m, kv_amax(f[i], inf));
            if (inf) infinite |= 1u << i;
            if (FMT == KV_INT8) {
#pragma unroll
                for (int j = 0; j < 16; ++j) nan |= !(f[i][j] == f[i][j]);
            }
        }
    } else {
        __nv_bfloat162 most = __float2bfloat162_rn(0.f), seen = most;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            if (row0 + i * step >= rows) break;
            const uint32_t w[8] = {ra[i].x, ra[i].y, ra[i].z, ra[i].w, rb[i].x, rb[i].y, rb[i].z, rb[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const __nv_bfloat162 v = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
                most = __hmax2(most, v);  // passes NaN over
                if (FMT == KV_INT8) seen = __hmax2_nan(seen, v);
            }
        }
        m = fmaxf(__low2float(most), __high2float(most));
        if (m == INFINITY) {
            m = 0.f;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (row0 + i * step >= rows) break;
                float v[16];
                RopeElem<__nv_bfloat16>::unpack(ra[i], *reinterpret_cast<float(*)[8]>(v));
                RopeElem<__nv_bfloat16>::unpack(rb[i], *reinterpret_cast<float(*)[8]>(v + 8));
                bool inf;
                m = fmaxf(m, kv_amax(v, inf));
            }
        }
        nan = FMT == KV_INT8 && (__hisnan(__low2bfloat16(seen)) || __hisnan(__high2bfloat16(seen)));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (u == 0 && row0 < rows) atomicMax(&sh.amax[my_h], __float_as_uint(m));  // m >= 0: bits keep the order
    if (FMT == KV_INT8 && nan) record_error(DSA_DEV_ERR_BOUNDS, 0xa04);
    __syncthreads();
    if (tid <= hmask) {
        const float s = fmaxf(old, kv_pow2(kv_exponent<FMT>(__uint_as_float(sh.amax[tid]))));
        sh.old[tid] = old;
        sh.now[tid] = s;
        scale[tid] = s;
    }
    bool open = false;  // the same in all threads
    if (n) {
        const uint4 top = *reinterpret_cast<const uint4*>(sh.amax);
        open = kv_near_border<FMT>(top.x) || kv_near_border<FMT>(top.y) || kv_near_border<FMT>(top.z) || kv_near_border<FMT>(top.w);
    }
    __syncthreads();

    // round and store the new rows
    const float s = sh.now[my_h], inv = 1.f / s;  // powers of two
    uint8_t* to = pages + (long long)slot0 * P.Hkv * kKvD + (h0 + my_h) * kKvD;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = row0 + i * step;
        if (r >= rows) break;
        uint32_t w[4];
        if (!n) {
            float v[16];
            RopeElem<__nv_bfloat16>::unpack(ra[i], *reinterpret_cast<float(*)[8]>(v));
            RopeElem<__nv_bfloat16>::unpack(rb[i], *reinterpret_cast<float(*)[8]>(v + 8));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = kv_round4<FMT>(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
        } else if (!turned) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = kv_round4<FMT>(f[i][4 * k] * inv, f[i][4 * k + 1] * inv, f[i][4 * k + 2] * inv, f[i][4 * k + 3] * inv);
        } else {
            // pair x lies in bytes lo(x), hi(x); both ends of its error's interval are rounded.  The sine and
            // cosine are off by 2^-23 of 1 at most (their own ulp, the angle's rounding, mscale's), products and
            // sum by 2^-24, in all 2^-22.4 (|a| + |b|) <= 2^-21.9 (|y0| + |y1|).
            const float eps = inv * 4.76837158203125e-7f;  // 2^-21
            unsigned differ[4], any = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[4], x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int e = 4 * k + y;
                    const float d = (fabsf(f[i][e]) + fabsf(f[i][INTER ? e ^ 1 : e ^ 8])) * eps;
                    v[y] = fmaf(f[i][e], inv, -d);
                    x[y] = fmaf(f[i][e], inv, d);
                }
                w[k] = kv_round4<FMT>(v[0], v[1], v[2], v[3]);
                differ[k] = w[k] ^ kv_round4<FMT>(x[0], x[1], x[2], x[3]);
                any |= differ[k];
            }
            // an infinite member's interval is NaN, and so is its partner's: their bytes come from the formula too
            if (any || infinite >> i & 1) {
                const __nv_bfloat16* at = in + (long long)(r >> hshift) * ts + my_h * hs;
                const unsigned long long p = position(r >> hshift);
                unsigned todo = infinite >> i & 1 ? 255u : 0u;  // pairs of which a byte differs
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const int lo = INTER ? 2 * y : y, hi = INTER ? 2 * y + 1 : 8 + y;
                    if ((differ[lo >> 2] >> (8 * (lo & 3)) | differ[hi >> 2] >> (8 * (hi & 3))) & 255u) todo |= 1u << y;
                }
#pragma unroll 1
                for (; todo; todo &= todo - 1) {
                    const int y = __ffs(todo) - 1;
                    const int lo = INTER ? 2 * y : y, hi = INTER ? 2 * y + 1 : 8 + y;
                    const unsigned at_lo = 255u << (8 * (lo & 3)), at_hi = 255u << (8 * (hi & 3));
                    const uint32_t both = kv_turn_exact<FMT>(__bfloat162float(at[lo < 8 ? a + lo : b + lo - 8]),
                                                             __bfloat162float(at[hi < 8 ? a + hi : b + hi - 8]),
                                                             p * rope_turn(P.inv_freq[u * 8 + y]), P.mscale, inv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (lo >> 2 == k) w[k] = (w[k] & ~at_lo) | ((both & 255u) << (8 * (lo & 3)));
                        if (hi >> 2 == k) w[k] = (w[k] & ~at_hi) | ((both >> 8 & 255u) << (8 * (hi & 3)));
                    }
                }
            }
        }
        uint8_t* dst = to + (long long)(r >> hshift) * P.Hkv * kKvD;
        *reinterpret_cast<uint2*>(dst + a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + b) = make_uint2(w[2], w[3]);
    }

    if (open) kv_settle_scale<FMT, INTER>(P, sh, in, to, scale, a, b, S.i0, S.p0, rows);

    // tokens that the page held before: rounded again where their head's scale grew
    if (!slot0) return;
    for (int e = tid; e < slot0 << (hshift + 3); e += blockDim.x) {
        const int h = (e >> 3) & hmask;
        if (sh.old[h] == sh.now[h]) continue;
        const float ratio = sh.old[h] / sh.now[h];
        uint4* at = reinterpret_cast<uint4*>(pages + ((long long)(e >> (hshift + 3)) * P.Hkv + h0 + h) * kKvD) + (e & 7);
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
            kv_value4<FMT>(w[i], x);
            w[i] = kv_round4<FMT>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace dsa

// Attention over the paged 8-bit KV cache (kv8.cuh): row t reads keys of sequence seq[t],
//   z_s = scale * ks(s) * sum_d q[t,h,d] k8[s,d],  out = sum_s softmax(z)_s vs(s) v8[s,:]
// over all its n_keys[t] cached keys, or over those that idx names; ks, vs are the scales of the key's page.
//
// Bound by the cache's bytes: at 32 query and 4 KV heads a key is 1 KB against 16 Kflop.
//   - A warp works alone: it owns one KV head and 32 keys of every tile, copies their K and V rows
//     (32 x 128 bytes each) and scales into a ring of its own with cp.async and multiplies them, so
//     that no barrier stands between copies and products and every SM keeps 12 rings in flight.
//     Dense rows and selected keys differ only in where a lane's key number comes from.
//   - Both products run on fp16 matrix instructions, where e4m3 and int8 values are exact:
//     S^T[keys x heads] = K Q^T and O^T += V^T P^T, the G query heads of the KV head as columns.  The rows of
//     K's fragments stand for whichever dims make a thread's bytes adjacent, so K goes from shared memory by
//     16-byte loads; V's fragments come transposed as bytes, their columns keys 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of
//     a tile, as S leaves them.  K's 16-byte chunks are exchanged by key parity, V's by f(key) = key mod 4 +
//     4 (key / 8 mod 2), which keeps these reads free of bank conflicts.
//   - q goes to fp16 after its head is scaled by a power of two to at most 2^14: no bit of bf16's is lost
//     within 2^-28 of the head's largest.
//   - V's scale 2^e * m, 1 <= m < 2, enters through the exponent: the softmax's reference is the running
//     maximum of z + e (less 7), so that P = 2^(z + e - ref) * m, rounded to fp16, keeps its bits however far the
//     scales of a row's pages lie apart; the row sum adds P's 2^-e part in fp32.  Keys whose V scale lies 2^64 below
//     that of the reference's, for which P alone may underflow, add theirs by an exponential of their own (all scales
//     that an append makes are safe so; the test for it costs 1 to 2 % of the times below).
//   - Rows are dealt to blocks by units, a row's units being its tiles and two more for its end: block c of
//     C takes units [c, c + 1) * ceil(U / C) of all rows' U, in order, whatever the rows' lengths.  A row that
//     one block holds whole is finished there; of the others each block writes its unnormalised part, and
//     paged_combine_kernel joins them.
//   - Where that second kernel would cost more than even shares save (few keys, or rows enough to fill the
//     GPU), a row gets a cluster of 1 to 8 blocks, which split its tiles evenly and join their outputs
//     through each other's shared memory.
//
// Measured (32 query heads):
//   16 x 131328 keys, 4 KV heads, e4m3   328-341 us, 6.3-6.5 TB/s, 97-101 % of the copy rate: bound by memory
//   122 rows of 1 to 16000 keys, 2 KV heads, int8   75 us, 2.2 TB/s: bound by instructions and their latencies (16 heads a
//                                        KV head; issue slots 55 % busy with 3 warps a scheduler)
//   1024 rows x 2048 of 32768 keys       257 us, 8.4 TB/s of gathered rows, from L2: the same (57 %, 570 instructions
//                                        for a warp's 32 keys; leaving out V's conversions alone saves 3 %)
//   16 rows x 2048 of 131328 keys        13.5 us (5.3 for the bytes): latency of launch, look-up, four tiles, join
//   1 row of 777 keys                    9.2 us: latency of launch, look-up, two tiles, join
#pragma once

#include <type_traits>

#include "kv8.cuh"

namespace dsa {

constexpr int kPagedPartCtas = 296;     // most blocks that share rows; each has two partial slots
constexpr int kPagedSharedRows = 1184;  // most rows that are dealt by units
constexpr int kPagedMostCluster = 8;    // most blocks of a cluster (the portable limit)
constexpr int kPagedPartStride = kKvD + 4;  // floats of a partial: O[128], max, sum, 2 pad
constexpr int kPagedRowTiles = 2;       // what the end of a row costs a block, in tiles, when rows are dealt

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
    int cluster;                       // blocks of a row; 0: rows are dealt by units (and joined)
    float* part;                       // [2 * gridDim.x, Hq, kPagedPartStride]
    long long* row_start;              // [T + 1]: where the rows start, in units dealt; behind them a block's units
};

// NT: groups of 8 query heads of a KV head.  KT: 16-key tiles of a warp's step (a transposed load of V takes two).
template <int NT>
struct PagedCfg {
    static constexpr int KT = 2;
    static constexpr int NW = 12;
    static constexpr int S = 2;  // ring stages of a warp
    static constexpr int CTAS = 1;
    static constexpr int THREADS = NW * 32;
    static constexpr int STAGE = KT * 2 * 16 * kKvD;  // K rows, V rows
    static constexpr int META = 68;                   // floats of a stage: K's and V's scales, mask
    static constexpr int RING_BYTES = NW * S * STAGE;
    static constexpr int META_BYTES = NW * S * META * 4;
    static constexpr int XCH_BYTES = NW * NT * 16 * 4;  // maxima and sums of a warp's heads
    static_assert(NT * 8 * 4 * 32 * 4 <= STAGE, "a warp's outputs are exchanged through one of its stages");
    // two groups' queries would not leave registers for 12 warps: they are read from shared memory, [KV head][k][lane]
    static constexpr int Q_BYTES = NT == 2 ? 4 * 8 * 32 * 16 : 0;
    static constexpr int SMEM = RING_BYTES + META_BYTES + XCH_BYTES + Q_BYTES;
};
constexpr float kPagedNone = -1e30f;  // the reference before any key
// The reference is taken kPagedBelow below the step's maximum, and moves when a logit exceeds it by kPagedMost (both in
// log2): P * m stays below 2^15, under fp16's 2^16, and is right to 2^-11 of itself down to 2^-21 of the largest, below
// to 2^-32 of the largest.  (Taken at the maximum, P is lost below 2^-25 of it: 16384 such keys of a warp beside one
// large one were missing from the output altogether.)
constexpr float kPagedBelow = 7.f, kPagedMost = 14.f;

// 2^(d / 2), d <= 0.  References differ by V's exponents too, up to 200 between pages, but the row sums behind them hold
// that much: what is brought from one reference to another is multiplied by this twice, since 2^d alone may be 0.
__device__ __forceinline__ float paged_root(float d) { return exp2f(0.5f * d); }

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
__device__ __forceinline__ int paged_count(const PagedParams& P, int n) { return P.idx ? min(P.topk, n) : n; }

__device__ __forceinline__ void cp_async_4(void* dst, const void* src, bool valid) {
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
// The address of block `rank`'s counterpart of this block's shared-memory address, and reads of it.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 16 x 16 byte matrices (lane i gives row i's address), transposed: thread (g, j) gets column g's and g + 8's
// bytes of rows 4 j .. 4 j + 3 of the first, then of the second.
__device__ __forceinline__ void ldmatrix_b8_x2_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Four stored bytes as fp16 values, two to a register.
template <int FMT>
__device__ __forceinline__ void kv_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == KV_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // byte + 128 in the low bits of the fp16 number 1024 is 1152 + byte
        const uint32_t u = w ^ 0x80808080u, m0 = __byte_perm(u, 0x64646464u, 0x4140), m1 = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 c = __half2half2(__ushort_as_half(0x6480));
        const __half2 r0 = __hsub2(*reinterpret_cast<const __half2*>(&m0), c);
        const __half2 r1 = __hsub2(*reinterpret_cast<const __half2*>(&m1), c);
        lo = *reinterpret_cast<const uint32_t*>(&r0), hi = *reinterpret_cast<const uint32_t*>(&r1);
    }
}

// A key whose logit plus e lies z above the reference adds P 2^-e, with P = 2^z and d = 2^-e, to the row sum: what of it
// is missing from the product where P is below fp32's range.
__device__ __forceinline__ float paged_missed(float z, float d) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(z + static_cast<float>(static_cast<int>(__float_as_uint(d) >> 23) - 127)));
    return r - ex2_approx(z) * d;
}

// Where token `slot` of the pool starts: a product and sum in one step on the multipliers' side.
template <int ROWB>
__device__ __forceinline__ const uint8_t* paged_token(const uint8_t* base, uint32_t slot) {
    const uint8_t* at;
    asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(at) : "r"(slot), "n"(ROWB), "l"(base));
    return at;
}

// IDX: keys named by idx; otherwise the 16 keys of a step's tile lie side by side in one page.  CLU: P.cluster blocks a row.
template <int FMT, int NT, int HKV, bool IDX, bool CLU>
__global__ void __launch_bounds__(PagedCfg<NT>::THREADS, PagedCfg<NT>::CTAS) paged_attn_kernel(const PagedParams P) {
    using C = PagedCfg<NT>;
    constexpr int NW = C::NW, S = C::S, KT = C::KT;
    constexpr int NSUB = NW / HKV;        // warps of a KV head
    constexpr int TK = NSUB * KT * 16;    // keys of a tile
    constexpr int ROWB = HKV * kKvD;      // bytes between a page's tokens
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = P.Hq / HKV;
    const int head = warp % HKV, sub = warp / HKV;
    const int g = lane >> 2, j = lane & 3;

    // ---- this block's units [w0, w1); its first tile is `tile0` of row `row0`, which is unit `at`
    long long w0 = 0, w1, at = 0;
    int row0 = blockIdx.x, tile0 = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto row_tiles = [&](int r) {
        int b, n;
        paged_row(P, r, b, n);
        return (paged_count(P, n) + TK - 1) / TK;
    };
    if (!CLU && P.T <= 32) {
        // every warp for itself, a row to a lane
        const int nt = lane < P.T ? row_tiles(lane) : 0, mine = nt ? nt + kPagedRowTiles : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31), chunk = max(1, (total + (int)gridDim.x - 1) / (int)gridDim.x);
        const int start = incl - mine;
        w0 = (long long)blockIdx.x * chunk;
        w1 = min((long long)total, w0 + chunk);
        if (blockIdx.x == 0 && warp == 0) {
            if (lane < P.T) P.row_start[lane] = start;
            if (lane == 0) P.row_start[P.T] = chunk;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, nt && w0 < start + nt && start < w1);
        if (!hit) return;
        row0 = __ffs(hit) - 1;
        const int s0 = __shfl_sync(0xffffffffu, start, row0);
        tile0 = (int)max(0ll, w0 - s0);
        at = s0 + tile0;
    } else if (!CLU) {
        __shared__ long long s_sum[NW], s_total, s_start;
        __shared__ int s_row0;
        const int per = (P.T + C::THREADS - 1) / C::THREADS;
        const int r0 = min(P.T, (int)threadIdx.x * per), r1 = min(P.T, r0 + per);
        long long mine = 0;
        for (int r = r0; r < r1; ++r) {
            const int nt = row_tiles(r);
            mine += nt ? nt + kPagedRowTiles : 0;
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        if (threadIdx.x == 0) {
            long long run = 0;
            for (int w = 0; w < NW; ++w) {
                const long long x = s_sum[w];
                s_sum[w] = run;
                run += x;
            }
            s_total = run;
            s_row0 = P.T;
        }
        __syncthreads();
        const long long total = s_total;
        const long long chunk = max(1ll, (total + gridDim.x - 1) / gridDim.x);
        w0 = blockIdx.x * chunk;
        w1 = min(total, w0 + chunk);
        long long start = s_sum[warp] + incl - mine, found_start = 0;
        int found = P.T;
        if (blockIdx.x == 0 || (start < w1 && w0 < start + mine)) {
            for (int r = r0; r < r1; ++r) {
                const int nt = row_tiles(r);
                if (found == P.T && nt && w0 < start + nt && start < w1) found = r, found_start = start;
                if (blockIdx.x == 0) P.row_start[r] = start;
                start += nt ? nt + kPagedRowTiles : 0;
            }
            if (found < P.T) atomicMin(&s_row0, found);
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) P.row_start[P.T] = chunk;
        __syncthreads();
        row0 = s_row0;
        if (row0 == P.T) return;
        if (found == row0) s_start = found_start;
        __syncthreads();
        tile0 = (int)max(0ll, w0 - s_start);
        at = s_start + tile0;
    } else {
        row0 = blockIdx.x / P.cluster;
        const int nt = row_tiles(row0), per = (nt + P.cluster - 1) / P.cluster;
        tile0 = min(nt, (int)(blockIdx.x % P.cluster) * per);
        w1 = min(nt, tile0 + per);
        at = tile0;
    }

    // from here on units count from w0: the block's are [0, units), the next one `now`
    const int units = (int)(w1 - w0);
    int now = (int)(at - w0);

    uint8_t* ring = smem + warp * (S * C::STAGE);
    float* meta = reinterpret_cast<float*>(smem + C::RING_BYTES) + warp * (S * C::META);
    float* xch = reinterpret_cast<float*>(smem + C::RING_BYTES + C::META_BYTES);
    uint4* q_sh = reinterpret_cast<uint4*>(smem + C::RING_BYTES + C::META_BYTES + C::XCH_BYTES) + head * (8 * 32) + lane;

    // ---- copies.  A step's keys pass three stages, one iteration apart: their numbers are loaded, their
    // pages looked up, their rows copied.  With IDX lane i has key i of the step;
    // otherwise lane i has the first key of 16-key tile i mod 16, for i mod 16 < KT.
    int f_row = row0, f_tile = tile0, f_b, f_n;  // front cursor: the next tile whose keys are loaded
    int f_at = now;
    paged_row(P, f_row, f_b, f_n);
    int f_nt = (paged_count(P, f_n) + TK - 1) / TK;
    const int my_key = IDX ? lane : (lane & 15) * 16;
    const bool has_key = IDX || (lane & 15) < KT;
    int a_key = -1, a_n = 0, a_b = 0;   // numbers loaded
    int b_key = -1, b_n = 0, b_pid = 0; // pages looked up; nothing waits for the page number before the copy
    auto load_keys = [&]() {
        a_key = -1;
        if (f_at >= units) return;
        const int e = f_tile * TK + sub * (KT * 16) + my_key;
        a_n = f_n, a_b = f_b;
        if (has_key && e < paged_count(P, f_n)) a_key = IDX ? P.idx[(long long)f_row * P.topk + e] : e;
        ++f_at;
        if (++f_tile == f_nt) {
            f_at += kPagedRowTiles;
            f_tile = 0;
            if (f_at < units) {  // some later row has units of this block
                do {
                    paged_row(P, ++f_row, f_b, f_n);
                    f_nt = (paged_count(P, f_n) + TK - 1) / TK;
                } while (f_nt == 0);
            }
        }
    };
    auto look_up = [&]() {
        b_key = a_key < a_n ? a_key : -1, b_n = a_n;
        if (b_key >= 0) b_pid = P.table[(long long)a_b * P.max_pages + (b_key >> P.page_shift)];
    };
    // lane's part of every row copy: row lane / 8 of four, 16-byte chunk lane % 8
    const uint8_t* k_lane = P.k_pages + head * kKvD + (lane & 7) * 16 + (IDX ? 0 : (lane >> 3) * ROWB);
    const uint8_t* v_lane = P.v_pages + head * kKvD + (lane & 7) * 16 + (IDX ? 0 : (lane >> 3) * ROWB);
    const int lr = lane >> 3, lc = lane & 7;
    auto copy_rows = [&](int st) {
        float* sc = meta + st * C::META;
        uint8_t* dst = ring + st * C::STAGE + lr * kKvD;
        // row r = 4 i + lr of a tile: K's chunk c goes to c ^ 4 (r & 1), V's to c ^ f(r)
        const int k_at = (lc ^ ((lr & 1) << 2)) << 4;
        // the token's slot in the pool (-1: none) and the keys from it on
        int b_slot = -1, b_valid = 0;
        if (b_key >= 0) {
            if (b_pid < 0 || b_pid >= P.num_pages) {
                record_error(DSA_DEV_ERR_BOUNDS, 0xb02);
            } else {
                b_slot = (b_pid << P.page_shift) + (b_key & ((1 << P.page_shift) - 1));
                b_valid = min(16, b_n - b_key);
            }
        }
        if constexpr (IDX) {
            const unsigned mask = __ballot_sync(0xffffffffu, b_slot >= 0);
            if (lane == 0) reinterpret_cast<unsigned*>(sc)[C::META - 1] = mask;
            if (mask) {
                if (mask == 0xffffffffu) {  // the usual step: nothing to fill (258 -> 253 us for 1024 rows of 2048 keys)
#pragma unroll
                    for (int i = 0; i < 4 * KT; ++i) {
                        const uint32_t s = __shfl_sync(0xffffffffu, b_slot, i * 4 + lr);
                        const int v_at = (lc ^ (lr | (i & 2) << 1)) << 4;
                        cp_async_16(dst + (i >> 2) * 4096 + (i & 3) * 512 + k_at, paged_token<ROWB>(k_lane, s), true);
                        cp_async_16(dst + (i >> 2) * 4096 + 2048 + (i & 3) * 512 + v_at, paged_token<ROWB>(v_lane, s), true);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4 * KT; ++i) {
                        const int s = __shfl_sync(0xffffffffu, b_slot, i * 4 + lr);
                        const bool ok = s >= 0;
                        const uint32_t at = ok ? s : 0;
                        const int v_at = (lc ^ (lr | (i & 2) << 1)) << 4;
                        cp_async_16(dst + (i >> 2) * 4096 + (i & 3) * 512 + k_at, paged_token<ROWB>(k_lane, at), ok);
                        cp_async_16(dst + (i >> 2) * 4096 + 2048 + (i & 3) * 512 + v_at, paged_token<ROWB>(v_lane, at), ok);
                    }
                }
                const bool ok = b_slot >= 0;
                const long long at = ok ? (long long)(b_slot >> P.page_shift) * HKV + head : 0;
                cp_async_4(sc + lane, P.k_scale + at, ok);
                cp_async_4(sc + 32 + lane, P.v_scale + at, ok);
            }
        } else {
            int s[KT], n[KT], all = 0;
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                s[t] = __shfl_sync(0xffffffffu, b_slot, t), n[t] = __shfl_sync(0xffffffffu, b_valid, t);
                if (lane == 0) reinterpret_cast<int*>(sc)[C::META - 1 - t] = n[t];
                all |= n[t];
            }
            if (all) {  // a tile without keys is filled with zeros if the step's other one has some
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const long long at = n[t] ? (long long)s[t] * ROWB : 0;  // a tile's 16 slots are in the pool, filled or not
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool ok = i * 4 + lr < n[t];
                        const int v_at = (lc ^ (lr | (i & 2) << 1)) << 4;
                        cp_async_16(dst + t * 4096 + i * 512 + k_at, k_lane + at + i * 4 * ROWB, ok);
                        cp_async_16(dst + t * 4096 + 2048 + i * 512 + v_at, v_lane + at + i * 4 * ROWB, ok);
                    }
                }
            }
            if (has_key && b_valid)
                cp_async_4(sc + (lane & 15) * 2 + (lane >> 4),
                           (lane < 16 ? P.k_scale : P.v_scale) + (long long)(b_slot >> P.page_shift) * HKV + head, true);
        }
        cp_async_commit();
    };
    // ---- per row: queries, running maximum, sums, outputs
    uint32_t qf[NT == 1 ? 8 : 1][2];
    float qfac[NT][2];     // of heads nt * 8 + 2 j + {0, 1}: logits in log2 per unit of the product
    bool started = false;  // this warp has seen a key of the row: m_run holds maxima
    float v_far;           // 2^-64 times the largest 2^e of the keys that the references were taken from
    float o[NT][8][4], m_run[NT][2], l_run[NT][2];
    int row = row0, left;  // left: tiles of the row still to come in this block
    bool whole;            // the block holds the row from its first tile to its last
    int slot;              // where its part goes if not: 0 where the row reaches back to the block's first unit
    uint2 q_raw[NT][8];
    auto load_q = [&]() {
#pragma unroll
        for (int nt8 = 0; nt8 < NT; ++nt8) {
            const int hl = nt8 * 8 + g;
            const __nv_bfloat16* qrow = P.q + ((long long)row * P.Hq + head * G + (hl < G ? hl : 0)) * kKvD;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                q_raw[nt8][kk] = *reinterpret_cast<const uint2*>(qrow + (kk < 4 ? j * 16 + kk * 4 : 64 + j * 16 + (kk - 4) * 4));
        }
    };
    auto begin_row = [&](int tile, int n) {  // after load_q
        const int nt = (paged_count(P, n) + TK - 1) / TK;
        left = min(nt - tile, units - now);
        whole = tile == 0 && left == nt;
        slot = now <= tile ? 0 : 1;
        started = false;
        v_far = 0.f;
#pragma unroll
        for (int nt8 = 0; nt8 < NT; ++nt8) {
            float f[8][4], top = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint2 w = q_raw[nt8][kk];
                f[kk][0] = __uint_as_float(w.x << 16), f[kk][1] = __uint_as_float(w.x & 0xffff0000u);
                f[kk][2] = __uint_as_float(w.y << 16), f[kk][3] = __uint_as_float(w.y & 0xffff0000u);
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(f[kk][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^s brings the head's largest below 2^14
            int s = 13 - ((int)(__float_as_uint(top) >> 23) - 127);
            s = max(-114, min(100, s));
            const float up = nt8 * 8 + g < G ? kv_pow2(s) : 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint2 w = make_uint2(pack_f16x2(f[kk][0] * up, f[kk][1] * up), pack_f16x2(f[kk][2] * up, f[kk][3] * up));
                if constexpr (NT == 1) qf[kk][0] = w.x, qf[kk][1] = w.y;
                else if (sub == 0) reinterpret_cast<uint2*>(q_sh + kk * 32)[nt8] = w;
            }
            const float fac = P.scale_log2 * kv_pow2(-s);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                qfac[nt8][jj] = __shfl_sync(0xffffffffu, fac, (2 * j + jj) * 4);
                m_run[nt8][jj] = 0.f, l_run[nt8][jj] = 0.f;
            }
#pragma unroll
            for (int dt = 0; dt < 8; ++dt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt8][dt][i] = 0.f;
        }
    };
    {
        const int n0 = f_n;  // of row0
        load_keys();
        look_up();
        load_q();
        load_keys();
#pragma unroll
        for (int s = 0; s < S - 1; ++s) {
            copy_rows(s);
            look_up();
            load_keys();
        }
        begin_row(tile0, n0);
        if (NT == 2) __syncthreads();  // the queries are in shared memory
    }

    // This warp's outputs, maxima and sums to shared memory: fragments [nt * 8 + dt][lane][4] in ring stage st,
    // (two maxima, two sums) as [nt][j] in xch.
    auto leave = [&](int st) {
        float4* frag = reinterpret_cast<float4*>(ring + st * C::STAGE) + lane;
        float4* ml = reinterpret_cast<float4*>(xch) + warp * (NT * 4) + j;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = l_run[nt][x];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                l_run[nt][x] = l;
            }
            if (g == 0)
                ml[nt * 4] = make_float4(started ? m_run[nt][0] : kPagedNone, started ? m_run[nt][1] : kPagedNone, l_run[nt][0], l_run[nt][1]);
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) frag[(nt * 8 + dt) * 32] = make_float4(o[nt][dt][0], o[nt][dt][1], o[nt][dt][2], o[nt][dt][3]);
        }
    };
    // A fragment of the row's output: weights and adds what `parts` of at most MOST warps (or blocks) left, and
    // writes dims 16 dt + g, + 8 of heads nt * 8 + 2 j, + 1 (a lane and the next one pair theirs to adjacent dims).  max_sum(p) gives part p's maxima and sums of the
    // two heads, value(p) its fragment.
    auto join = [&](auto most, int nt, int dt, int parts, auto max_sum, auto value) {
        constexpr int MOST = decltype(most)::value;
        float2 m = make_float2(kPagedNone, kPagedNone), l = make_float2(0.f, 0.f);
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        float4 t[MOST], v[MOST];
#pragma unroll
        for (int p = 0; p < MOST; ++p)
            if (p < parts) t[p] = max_sum(p), v[p] = value(p);
#pragma unroll
        for (int p = 0; p < MOST; ++p)
            if (p < parts) m.x = fmaxf(m.x, t[p].x), m.y = fmaxf(m.y, t[p].y);
#pragma unroll
        for (int p = 0; p < MOST; ++p) {
            if (p >= parts) continue;
            const float hx = paged_root(t[p].x - m.x), hy = paged_root(t[p].y - m.y), wx = hx * hx, wy = hy * hy;
            l.x += t[p].z * hx * hx, l.y += t[p].w * hy * hy;
            a[0] += v[p].x * wx, a[1] += v[p].y * wy, a[2] += v[p].z * wx, a[3] += v[p].w * wy;
        }
        const bool odd = g & 1;
        const int dim = 16 * dt + (g & 6) + (odd ? 8 : 0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int hl = nt * 8 + 2 * j + x;
            const float other = __shfl_xor_sync(0xffffffffu, odd ? a[x] : a[2 + x], 4);
            const float v0 = odd ? other : a[x], v1 = odd ? a[2 + x] : other;  // dims dim, dim + 1
            if (hl >= G) continue;
            const long long h = (long long)row * P.Hq + head * G + hl;
            const float mx = x ? m.y : m.x, lx = x ? l.y : l.x;
            if (whole) {
                const float inv = lx == 0.f ? 0.f : 1.f / lx;
                *reinterpret_cast<uint32_t*>(P.out + h * kKvD + dim) = pack_bf16x2(v0 * inv, v1 * inv);
                if (P.lse && g == 0 && dt == 0) P.lse[h] = lx == 0.f ? -INFINITY : (mx + log2f(lx)) * 0.69314718055994531f;
            } else {
                float* part = P.part + ((2ll * blockIdx.x + slot) * P.Hq + head * G + hl) * kPagedPartStride;
                *reinterpret_cast<float2*>(part + dim) = make_float2(v0, v1);
                if (g == 0 && dt == 0) *reinterpret_cast<float2*>(part + kKvD) = make_float2(mx, lx);
            }
        }
    };

    // V's row of this lane in a transposed load: lane 16 t + 4 a + b gives key 2 a + (b & 1) + 8 (b >> 1) of tile t
    const int v_row = (lane >> 4) * 4096 + 2048 + (((lane >> 2) & 3) * 2 + (lane & 1) + (lane & 2) * 4) * kKvD;
    const int v_swz = (lane & 1) | ((lane >> 2) & 1) << 1 | (lane & 2) << 1;
    int used = 0;
    for (int st = 0; now < units;) {
        // The next copies go into the stage that the last iteration used up.  Dense rows dealt to blocks run at the
        // memory's rate, and have them in flight before they wait; elsewhere their instructions are worth more
        // between those of the products (16 x 128K dense keys: 324 us, in flight first 317; 1024 x 2048 selected
        // keys: 265, in flight first 282; 777 dense keys 11.3, in flight first 12.2).
        constexpr bool kCopyFirst = !IDX && !CLU;
        if constexpr (kCopyFirst) {
            __syncwarp();
            copy_rows(st == 0 ? S - 1 : st - 1);
            look_up();
            load_keys();
        }
        cp_async_wait<kCopyFirst ? S - 1 : S - 2>();
        __syncwarp();
        if constexpr (!kCopyFirst) {
            copy_rows(st == 0 ? S - 1 : st - 1);
            look_up();
            load_keys();
        }
        const float* sc = meta + st * C::META;
        int valid[KT];      // dense: keys of each tile;  IDX: the tile's bits of the mask
        bool some = false;  // any key at all
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            if constexpr (IDX) valid[t] = reinterpret_cast<const unsigned*>(sc)[C::META - 1] >> (16 * t) & 0xffffu;
            else valid[t] = reinterpret_cast<const int*>(sc)[C::META - 1 - t];
            some |= valid[t] != 0;
        }
        if (some) {
            const uint8_t* stage = ring + st * C::STAGE;
            // S^T: rows are keys g and g + 8; the dims of step kk are word kk of the thread's two chunks
            float z[KT][NT][4];
            const uint8_t* k0 = stage + g * kKvD + ((j ^ ((g & 1) << 2)) << 4);
            const uint8_t* k1 = stage + g * kKvD + ((j ^ ((g & 1) << 2) ^ 4) << 4);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) z[t][nt][x] = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t xw[KT][4], yw[KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const uint8_t* p = (half ? k1 : k0) + t * 4096;
                    const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 8 * kKvD);
                    xw[t][0] = x.x, xw[t][1] = x.y, xw[t][2] = x.z, xw[t][3] = x.w;
                    yw[t][0] = y.x, yw[t][1] = y.y, yw[t][2] = y.z, yw[t][3] = y.w;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t q[NT][2];
                    if constexpr (NT == 1) {
                        q[0][0] = qf[half * 4 + w][0], q[0][1] = qf[half * 4 + w][1];
                    } else {
                        const uint4 v = q_sh[(half * 4 + w) * 32];
                        q[0][0] = v.x, q[0][1] = v.y, q[NT - 1][0] = v.z, q[NT - 1][1] = v.w;
                    }
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        uint32_t a[4];
                        kv_f16x4<FMT>(xw[t][w], a[0], a[2]);
                        kv_f16x4<FMT>(yw[t][w], a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816_f16(z[t][nt], a, q[nt][0], q[nt][1]);
                    }
                }
            }
            // logits in log2 plus V's exponent, less the reference; d = 2^-e, vm = V's scale * d
            float d[KT][2], vm[KT][2];
            float v_least;  // the least V scale of the tiles, or this lane's of the step's 32 keys (0 where there is none)
            if constexpr (IDX) v_least = fabsf(sc[32 + lane]);
            else v_least = fminf(fabsf(sc[1]), fabsf(sc[3]));
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                float ks[2], vs[2];
                if constexpr (IDX) {
                    ks[0] = sc[16 * t + g], ks[1] = sc[16 * t + 8 + g];
                    vs[0] = sc[32 + 16 * t + g], vs[1] = sc[32 + 16 * t + 8 + g];
                } else {
                    const float2 kv = *reinterpret_cast<const float2*>(sc + 2 * t);
                    ks[0] = ks[1] = kv.x, vs[0] = vs[1] = kv.y;
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int e = min(120, max(-80, (int)(__float_as_uint(vs[y]) >> 23 & 255u) - 127));
                    d[t][y] = kv_pow2(-e);
                    vm[t][y] = vs[y] * d[t][y];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            z[t][nt][2 * y + x] = fmaf(z[t][nt][2 * y + x], ks[y] * qfac[nt][x], (float)e - m_run[nt][x]);
                }
                if (valid[t] != (IDX ? 0xffff : 16)) {
                    const bool v0 = IDX ? valid[t] >> g & 1 : g < valid[t], v1 = IDX ? valid[t] >> (g + 8) & 1 : g + 8 < valid[t];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (!v0) z[t][nt][x] = -INFINITY;
                            if (!v1) z[t][nt][2 + x] = -INFINITY;
                        }
                    if (!v0) d[t][0] = 0.f, vm[t][0] = 0.f;  // whatever an uncopied scale holds
                    if (!v1) d[t][1] = 0.f, vm[t][1] = 0.f;
                }
            }
            uint32_t pb[KT][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mx[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mx[x] = fmaxf(z[0][nt][x], z[0][nt][2 + x]);
#pragma unroll
                    for (int t = 1; t < KT; ++t) mx[x] = fmaxf(mx[x], fmaxf(z[t][nt][x], z[t][nt][2 + x]));
                }
                // the reference moves only when a logit exceeds it by more than kPagedMost (and keys far below it are seen to)
                if (!started || __any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > kPagedMost || v_least < v_far)) {
                    float root[2], alpha[2];
                    // the largest V scale of the step's keys, from one of which the reference may be taken (its power of two)
                    float v_most, d_top = 0.f;
                    if constexpr (IDX) {
                        v_most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v_least)));
                    } else {
                        unsigned least = 0x7f800000u;
#pragma unroll
                        for (int t = 0; t < KT; ++t)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                d_top = fmaxf(d_top, d[t][y]);
                                if (d[t][y] > 0.f) least = min(least, __float_as_uint(d[t][y]));
                            }
                        v_most = kv_pow2(127 - (int)(__reduce_min_sync(0xffffffffu, least) >> 23));
                    }
                    v_far = fmaxf(v_far, v_most * 5.421010862427522e-20f);  // 2^-64
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 4));
                        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 8));
                        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 16));
                        const float up = !started || mx[x] > kPagedMost ? fmaxf(mx[x] - kPagedBelow, kPagedNone) : 0.f;
                        root[x] = started ? ex2_approx(-0.5f * up) : 1.f;  // at the start there is nothing to scale
                        alpha[x] = root[x] * root[x];
                        m_run[nt][x] += up;
                        l_run[nt][x] = l_run[nt][x] * root[x] * root[x];
#pragma unroll
                        for (int t = 0; t < KT; ++t) z[t][nt][x] -= up, z[t][nt][2 + x] -= up;
                    }
                    // P may be 0 for keys whose V scale is below v_far, though their weight is not: what the sum below misses
                    if (IDX ? __any_sync(0xffffffffu, v_least < v_far) : d_top * v_far > 1.f) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int t = 0; t < KT; ++t)
                                l_run[nt][x] += paged_missed(z[t][nt][x], d[t][0]) + paged_missed(z[t][nt][2 + x], d[t][1]);
                    }
#pragma unroll
                    for (int dt = 0; dt < 8; ++dt) {
                        o[nt][dt][0] *= alpha[0];
                        o[nt][dt][1] *= alpha[1];
                        o[nt][dt][2] *= alpha[0];
                        o[nt][dt][3] *= alpha[1];
                    }
                }
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    float p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) p[x] = ex2_approx(z[t][nt][x]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) l_run[nt][x] = fmaf(p[2 + x], d[t][1], fmaf(p[x], d[t][0], l_run[nt][x]));
                    // P^T (keys x heads) -> B operand (keys as K, heads as N)
                    pb[t][nt][0] = movmatrix_trans(pack_f16x2(p[0] * vm[t][0], p[1] * vm[t][0]));
                    pb[t][nt][1] = movmatrix_trans(pack_f16x2(p[2] * vm[t][1], p[3] * vm[t][1]));
                }
            }
            started = true;
            // O^T += V^T P^T: fragment dt's rows are dims 16 dt + g and 16 dt + g + 8; its columns the tile's keys 2 j,
            // 2 j + 1, 2 j + 8, 2 j + 9
            static_assert(KT == 2, "a transposed load takes the step's two tiles");
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) {
                uint32_t w[4];
                ldmatrix_b8_x2_trans(w, smem_u32(stage) + v_row + ((dt ^ v_swz) << 4));
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    uint32_t a[4];
                    kv_f16x4<FMT>(w[2 * t], a[0], a[2]);
                    kv_f16x4<FMT>(w[2 * t + 1], a[1], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][dt], a, pb[t][nt][0], pb[t][nt][1]);
                }
            }
        }
        used = st;
        st = st + 1 == S ? 0 : st + 1;
        ++now;
        if (--left) continue;

        // ---- the row's last tile in this block: the warps of a KV head exchange their outputs through the
        // stages that they have just used up, and each joins and writes every NSUB-th fragment
        if (CLU && P.cluster > 1) break;
        leave(used);
        __syncthreads();
#pragma unroll 1
        for (int i = sub; i < NT * 8; i += NSUB) {
            const float4* ml = reinterpret_cast<const float4*>(xch) + head * (NT * 4) + (i >> 3) * 4 + j;
            const float4* src = reinterpret_cast<const float4*>(smem + head * (S * C::STAGE) + used * C::STAGE) + i * 32 + lane;
            join(
                std::integral_constant<int, NSUB>(), i >> 3, i & 7, NSUB, [&](int p) { return ml[p * HKV * (NT * 4)]; },
                [&](int p) { return src[p * HKV * (S * C::STAGE / 16)]; });
        }
        if (CLU) break;
        now += kPagedRowTiles;
        if (now >= units) break;
        int b, n;
        do paged_row(P, ++row, b, n);
        while (paged_count(P, n) == 0);
        load_q();
        begin_row(0, n);
        __syncthreads();  // the stages are read: the next copies may take them
    }
    if (CLU && P.cluster == 1 && units == 0) {  // a row without keys
        uint4* o = reinterpret_cast<uint4*>(P.out + (long long)row0 * P.Hq * kKvD);
        for (int i = threadIdx.x; i < P.Hq * kKvD / 8; i += C::THREADS) o[i] = make_uint4(0, 0, 0, 0);
        if (P.lse)
            for (int h = threadIdx.x; h < P.Hq; h += C::THREADS) P.lse[(long long)row0 * P.Hq + h] = -INFINITY;
    }
    if (CLU && P.cluster > 1) {
        // ---- the blocks of a cluster join the row: first each the fragments of its own warps, into the stages of
        // its first warps, then one warp of one block each fragment from all blocks
        __syncwarp();
        leave(0);
        __syncthreads();
        float4 all[NT];  // maxima and sums over this block's warps of the head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4* ml = reinterpret_cast<const float4*>(xch) + head * (NT * 4) + nt * 4 + j;
            float4 w[NSUB];
            all[nt] = make_float4(kPagedNone, kPagedNone, 0.f, 0.f);
#pragma unroll
            for (int p = 0; p < NSUB; ++p) {
                w[p] = ml[p * HKV * (NT * 4)];
                all[nt].x = fmaxf(all[nt].x, w[p].x), all[nt].y = fmaxf(all[nt].y, w[p].y);
            }
#pragma unroll
            for (int p = 0; p < NSUB; ++p) {
                const float hx = paged_root(w[p].x - all[nt].x), hy = paged_root(w[p].y - all[nt].y);
                all[nt].z += w[p].z * hx * hx, all[nt].w += w[p].w * hy * hy;
                w[p].x = hx * hx, w[p].y = hy * hy;
            }
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) {
                if ((nt * 8 + dt) % NSUB != sub) continue;  // each fragment by one warp
                float4* at = reinterpret_cast<float4*>(smem + head * (S * C::STAGE)) + (nt * 8 + dt) * 32 + lane;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int p = 0; p < NSUB; ++p) {
                    const float4 v = at[p * HKV * (S * C::STAGE / 16)];
                    a.x += v.x * w[p].x, a.y += v.y * w[p].y, a.z += v.z * w[p].x, a.w += v.w * w[p].y;
                }
                *at = a;
            }
        }
        __syncthreads();  // the warps' maxima are read
        if (sub == 0 && g == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) reinterpret_cast<float4*>(xch)[head * (NT * 4) + nt * 4 + j] = all[nt];
        }
        cluster_sync();
        whole = true;
        const int rank = blockIdx.x % P.cluster;
#pragma unroll 1
        for (int i = sub * P.cluster + rank; i < NT * 8; i += NSUB * P.cluster) {
            const uint32_t ml = smem_u32(reinterpret_cast<const float4*>(xch) + head * (NT * 4) + (i >> 3) * 4 + j);
            const uint32_t src = smem_u32(reinterpret_cast<const float4*>(smem + head * (S * C::STAGE)) + i * 32 + lane);
            join(
                std::integral_constant<int, kPagedMostCluster>(), i >> 3, i & 7, P.cluster, [&](int p) { return ld_cluster(cluster_addr(ml, p)); },
                [&](int p) { return ld_cluster(cluster_addr(src, p)); });
        }
        cluster_sync();  // no block leaves while another reads its shared memory
    }
}

constexpr int kCombineThreads = 256;

// Joins the parts of the rows that several blocks shared, and writes the rows without keys.  A block has
// 8 / WPH heads of a row at a time, WPH warps on each, which take the parts in turn.
template <int WPH>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedParams P, int TK) {
    constexpr int HB = 8 / WPH;
    __shared__ float s_l[8];
    __shared__ float4 s_o[8][32];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hs = warp / WPH, pw = warp % WPH;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int b, n;
    paged_row(P, t, b, n);
    const int nt = (paged_count(P, n) + TK - 1) / TK;
    const long long start = P.row_start[t], chunk = P.row_start[P.T];
    const long long c0 = start / chunk, c1 = nt ? (start + nt - 1) / chunk : c0;
    if (nt && c0 == c1) return;  // one block held the row and wrote it
    const int parts = nt ? (int)(c1 - c0) + 1 : 0;
    for (int h0 = blockIdx.y * HB; h0 < P.Hq; h0 += gridDim.y * HB) {
        const int h = h0 + hs;
        const bool any = h < P.Hq;
        // part p: of block c0 + p, its slot 0 where the row reaches back to or before the block's first tile
        auto at = [&](int p) {
            const long long c = c0 + p;
            return P.part + ((2 * c + (start <= c * chunk ? 0 : 1)) * P.Hq + h) * kPagedPartStride;
        };
        float mx = kPagedNone;
        if (any)
            for (int p = lane; p < parts; p += 32) mx = fmaxf(mx, at(p)[kKvD]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (any) {
#pragma unroll 8
            for (int p = pw; p < parts; p += WPH) {
                const float* src = at(p);
                const float2 ml = *reinterpret_cast<const float2*>(src + kKvD);
                const float4 v = *reinterpret_cast<const float4*>(src + lane * 4);
                const float root = paged_root(ml.x - mx), w = root * root;
                l += ml.y * root * root;
                acc.x += v.x * w, acc.y += v.y * w, acc.z += v.z * w, acc.w += v.w * w;
            }
        }
        if (WPH > 1) {
            __syncthreads();
            s_o[warp][lane] = acc;
            if (lane == 0) s_l[warp] = l;
            __syncthreads();
            if (pw == 0) {
#pragma unroll
                for (int w = 1; w < WPH; ++w) {
                    const float4 v = s_o[warp + w][lane];
                    l += s_l[warp + w];
                    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
                }
            }
        }
        if (pw == 0 && any) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint2 w;
            w.x = pack_bf16x2(acc.x * inv, acc.y * inv), w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(P.out + ((long long)t * P.Hq + h) * kKvD + lane * 4) = w;
            if (P.lse && lane == 0)
                P.lse[(long long)t * P.Hq + h] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.69314718055994531f;
        }
    }
}

}  // namespace dsa

// Rows of a key/value cache held in 4 bits: writing them from bf16 and reading them back.
//
// A row of D values is D/2 + 4 bytes: element 2i in the low nibble of byte i and element
// 2i + 1 in its high one, then two bf16 values, the step s and the minimum m. It stands for
// s * code + m, where m is the row's smallest value (exact: the input is bf16 too),
// s = bf16((max - min) / 15) and code = round_half_even((x - m) * r), x - m and r = 1 / s each
// rounded to 32 bits. s is off by at most 2^-8 of the exact step, so the largest code is
// round(15 / (1 - 2^-8)) = round(15.06) = 15; the codes are those of s itself, so every value is off by at
// most (1/2 + 2^-18) s before the bf16 rounding of the read.
// A row with a NaN or an infinity, or whose max - min exceeds fp32's range, is stored with
// s = m = NaN: all of it reads as NaN. A step below 2^-126 is stored as 0: the row is m.
//
// The code needs no division and no conversion: fma(x - m, r, 1.5 * 2^23) rounds the
// product once, half to even, and leaves the code in the low bits of the float.
//
// D/8 lanes take a row, 16 bytes of bf16 and one word of codes each; a team takes heads of one
// token, four rows at a time, and neighbouring teams neighbouring tokens, whose packed rows lie side
// by side. The rows' extremes are exchanged together, each step halving the rows that a lane still
// compares, and a row's step and its inverse are computed by a quarter of the lanes. Bound by
// HBM: 2.53 bytes an element at D = 128. 35197 tokens of 8 heads: written in 35 us and read back in
// 30, 86 % of the measured copy rate together (140 us with a row a team).
#pragma once

#include "sm100_ptx.cuh"

namespace gqa {

constexpr int kKv4Threads = 256;

template <int D>
struct Kv4Row {
    static constexpr int kBytes = D / 2 + 4;
};

struct Kv4Side {
    __nv_bfloat16* rows;      // bf16 rows, element (n, h, d) at n*st + h*sh + d
    uint8_t* pool;            // 4-bit rows, row r of page p of head h at p*pool_sb + h*pool_sh + r*(D/2+4) bytes
    long long sh, st, pool_sb, pool_sh;
};

constexpr int kKv4Unroll = 4;  // rows a team takes at a time

struct Kv4RowsParams {
    Kv4Side x[2];      // keys, values
    const int* slots;  // [N]
    int N, H, page_size, num_pages;
    int heads_per_team, blocks;  // heads a team takes in turn; such blocks of H. gridDim.y is twice that
    uint32_t* err;
};

__device__ __forceinline__ __nv_bfloat162 bf162_of(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Where a team of D/8 lanes stands.
struct Kv4At {
    bool live;    // there is such a token
    bool stored;  // its slot is a row of the pool
    int h0, h1;
    __nv_bfloat16* row;  // this lane's eight elements of head h0's row
    uint8_t* packed;     // that row in the pool
    long long row_step, packed_step;  // to the next head's: elements, bytes
};
template <int D>
__device__ __forceinline__ Kv4At kv4_at(const Kv4RowsParams& p) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    const unsigned token = blockIdx.x * (kKv4Threads / kLanes) + threadIdx.x / kLanes;
    const bool second = (int)blockIdx.y >= p.blocks;
    const Kv4Side& x = second ? p.x[1] : p.x[0];
    Kv4At a;
    a.live = token < (unsigned)p.N;
    const int n = a.live ? (int)token : 0;
    a.h0 = ((int)blockIdx.y - (second ? p.blocks : 0)) * p.heads_per_team;
    a.h1 = min(a.h0 + p.heads_per_team, p.H);
    const int slot = __ldg(p.slots + n);
    const int page = slot / p.page_size;
    a.stored = a.live && slot >= 0 && page < p.num_pages;
    if (a.live && slot >= 0 && page >= p.num_pages && j == 0) atomicOr(p.err, kDevErrBadSeqlens);
    a.row_step = x.sh;
    a.packed_step = x.pool_sh;
    a.row = x.rows + n * x.st + a.h0 * x.sh + 8 * j;
    a.packed = x.pool + a.h0 * x.pool_sh +
               (a.stored ? page * x.pool_sb + (long long)(slot - page * p.page_size) * Kv4Row<D>::kBytes : 0);
    return a;
}

// Pack eight elements' codes: x in bf16 pairs.
__device__ __forceinline__ uint32_t kv4_codes(const uint4& x, float m, float r) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    uint32_t word = 0;
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: the sum's last bit is worth 1
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xffff0000u);
        word = (word << 4) + __float_as_uint(__fmaf_rn(__fsub_rn(hi, m), r, kRound));
        word = (word << 4) + __float_as_uint(__fmaf_rn(__fsub_rn(lo, m), r, kRound));
    }
    // the eight copies of kRound's bits, shifted and added up (mod 2^32)
    constexpr uint32_t kB = 0x4B400000u;
    constexpr uint32_t kAll = kB + (kB << 4) + (kB << 8) + (kB << 12) + (kB << 16) + (kB << 20) + (kB << 24) + (kB << 28);
    return word - kAll;
}

// The larger (max, -min) of two; NaN wins.
__device__ __forceinline__ uint32_t kv4_wider(uint32_t a, uint32_t b) { return u32_of(__hmax2_nan(bf162_of(a), bf162_of(b))); }
// Four rows' extremes over the team's lanes: lane j ends with those of row (j & kLanes/2 ? 1 : 0) +
// (j & kLanes/4 ? 2 : 0).
template <int kLanes>
__device__ __forceinline__ uint32_t kv4_extremes(const uint32_t (&v)[4], int j) {
    const bool h = j & (kLanes / 2), q = j & (kLanes / 4);
    const uint32_t t0 = kv4_wider(h ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, h ? v[0] : v[1], kLanes / 2));
    const uint32_t t1 = kv4_wider(h ? v[3] : v[2], __shfl_xor_sync(0xffffffffu, h ? v[2] : v[3], kLanes / 2));
    uint32_t s = kv4_wider(q ? t1 : t0, __shfl_xor_sync(0xffffffffu, q ? t0 : t1, kLanes / 4));
#pragma unroll
    for (int d = kLanes / 8; d > 0; d >>= 1) s = kv4_wider(s, __shfl_xor_sync(0xffffffffu, s, d));
    return s;
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads, 4) gqa_kv4_append_kernel(const __grid_constant__ Kv4RowsParams p) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    Kv4At a = kv4_at<D>(p);
    const int mine = (j & (kLanes / 2) ? 1 : 0) + (j & (kLanes / 4) ? 2 : 0);  // the row whose extremes this lane gets
    const bool heads = (j & (kLanes / 4 - 1)) == 0;                            // it stores that row's last word
    for (int h = a.h0; h < a.h1; h += kKv4Unroll) {
        uint4 u[kKv4Unroll];
        uint32_t mm[kKv4Unroll];
#pragma unroll
        for (int i = 0; i < kKv4Unroll; ++i) {
            u[i] = make_uint4(0u, 0u, 0u, 0u);
            if (a.stored && h + i < a.h1) u[i] = __ldcs(reinterpret_cast<const uint4*>(a.row));
            a.row += a.row_step;
        }
#pragma unroll
        for (int i = 0; i < kKv4Unroll; ++i) {
            // (max, -min) of the lane's eight as one bf16 pair; NaN wins
            const __nv_bfloat162 x = bf162_of(u[i].x), y = bf162_of(u[i].y), z = bf162_of(u[i].z), w = bf162_of(u[i].w);
            const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(x, y), __hmax2_nan(z, w));
            const __nv_bfloat162 lo = __hneg2(__hmin2_nan(__hmin2_nan(x, y), __hmin2_nan(z, w)));
            mm[i] = kv4_wider(__byte_perm(u32_of(hi), u32_of(lo), 0x5410), __byte_perm(u32_of(hi), u32_of(lo), 0x7632));
        }
        const __nv_bfloat162 e = bf162_of(kv4_extremes<kLanes>(mm, j));
        const float top = __low2float(e), m = -__high2float(e);
        const float range = top - m;
        __nv_bfloat16 step = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
        __nv_bfloat16 least = __float2bfloat16_rn(m);
        if (!(range < __uint_as_float(0x7f800000u))) step = least = __ushort_as_bfloat16((unsigned short)0x7fc0u);  // NaN
        const float s = __bfloat162float(step);
        if (s < 1.17549435e-38f) step = __ushort_as_bfloat16((unsigned short)0u);
        const float r = s < 1.17549435e-38f ? 0.f : __frcp_rn(s);
        if (heads && a.stored && h + mine < a.h1)
            *reinterpret_cast<uint32_t*>(a.packed + mine * a.packed_step + 4 * kLanes) =
                (uint32_t)__bfloat16_as_ushort(step) | (uint32_t)__bfloat16_as_ushort(least) << 16;
#pragma unroll
        for (int i = 0; i < kKv4Unroll; ++i) {
            const int from = (i & 1 ? kLanes / 2 : 0) + (i & 2 ? kLanes / 4 : 0);
            const float mi = __shfl_sync(0xffffffffu, m, from, kLanes), ri = __shfl_sync(0xffffffffu, r, from, kLanes);
            const uint32_t word = kv4_codes(u[i], mi, ri);
            if (a.stored && h + i < a.h1) reinterpret_cast<uint32_t*>(a.packed)[j] = word;
            a.packed += a.packed_step;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads, 4) gqa_kv4_gather_kernel(const __grid_constant__ Kv4RowsParams p) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    Kv4At a = kv4_at<D>(p);
    if (!a.live) return;
    for (int h = a.h0; h < a.h1; h += kKv4Unroll) {
        uint32_t word[kKv4Unroll], head[kKv4Unroll];
#pragma unroll
        for (int i = 0; i < kKv4Unroll; ++i) {
            word[i] = head[i] = 0u;  // a slot outside the pool reads as zeros
            if (a.stored && h + i < a.h1) {
                word[i] = reinterpret_cast<const uint32_t*>(a.packed)[j];
                head[i] = reinterpret_cast<const uint32_t*>(a.packed)[kLanes];
            }
            a.packed += a.packed_step;
        }
#pragma unroll
        for (int i = 0; i < kKv4Unroll; ++i) {
            const float s = __uint_as_float(head[i] << 16), m = __uint_as_float(head[i] & 0xffff0000u);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // 2^23 + code as float bits; the difference is the code, exactly
                const float code = __uint_as_float(0x4B000000u | ((word[i] >> (4 * e)) & 15u)) - 8388608.f;
                f[e] = fmaf(code, s, m);
            }
            if (h + i < a.h1)
                *reinterpret_cast<uint4*>(a.row) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            a.row += a.row_step;
        }
    }
}

}  // namespace gqa

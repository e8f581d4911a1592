// Rows of a key/value cache held in 4 bits: writing them from bf16 and reading them back.
//
// A row of D values is D/2 + 4 bytes: element 2i in the low nibble of byte i and element
// 2i + 1 in its high one, then two bf16 values, the step s and the minimum m. It stands for
// s * code + m, where m is the row's smallest value (exact: the input is bf16 too),
// s = bf16((max - min) / 15) and code = round_half_even((x - m) * r), x - m and r = 1 / s each
// rounded to 32 bits. s is off by at most 2^-9 of itself, so the largest code is round(15 (1 + 2^-9)) = 15
// and every value is off by at most (1/2 + 15 * 2^-9) s before the bf16 rounding of the read.
// A row with a NaN or an infinity, or whose max - min exceeds fp32's range, is stored with
// s = m = NaN: all of it reads as NaN. A step below 2^-126 is stored as 0: the row is m.
//
// The code needs no division and no conversion: fma(x - m, r, 1.5 * 2^23) rounds the
// product once, half to even, and leaves the code in the low bits of the float.
//
// D/8 lanes take a row, 16 bytes of bf16 and one word of codes each. Bound by HBM: 2.53 bytes
// an element at D = 128.
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

struct Kv4RowsParams {
    Kv4Side x[2];      // keys, values
    const int* slots;  // [N]
    int N, H, page_size, num_pages;
    uint32_t* err;
};

__device__ __forceinline__ __nv_bfloat162 bf162_of(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Which row a team of D/8 lanes has: neighbouring teams take neighbouring heads of a token.
struct Kv4At {
    bool live;    // there is such a row
    bool stored;  // its slot is a row of the pool
    __nv_bfloat16* row;  // this lane's eight elements
    uint32_t* packed;    // the row in the pool, as words
};

template <int D>
__device__ __forceinline__ Kv4At kv4_at(const Kv4RowsParams& p) {
    constexpr int kLanes = D / 8;
    const long long team = (long long)blockIdx.x * (kKv4Threads / kLanes) + threadIdx.x / kLanes;
    Kv4At a;
    a.live = team < 2LL * p.N * p.H;
    const long long r = a.live ? team / p.H : 0;
    const int h = a.live ? (int)(team - r * p.H) : 0;
    const bool second = r >= p.N;
    const int n = (int)(second ? r - p.N : r);
    const int slot = p.slots[n];
    const int page = slot / p.page_size;
    a.stored = a.live && slot >= 0 && page < p.num_pages;
    if (a.live && slot >= 0 && page >= p.num_pages && threadIdx.x % kLanes == 0) atomicOr(p.err, kDevErrBadSeqlens);
    // field by field: an index into the parameters would copy them to the stack
    const long long st = second ? p.x[1].st : p.x[0].st, sh = second ? p.x[1].sh : p.x[0].sh;
    const long long pool_sb = second ? p.x[1].pool_sb : p.x[0].pool_sb;
    const long long pool_sh = second ? p.x[1].pool_sh : p.x[0].pool_sh;
    a.row = (second ? p.x[1].rows : p.x[0].rows) + n * st + h * sh + 8 * (threadIdx.x % kLanes);
    a.packed = reinterpret_cast<uint32_t*>(
        (second ? p.x[1].pool : p.x[0].pool) +
        (a.stored ? page * pool_sb + h * pool_sh + (long long)(slot - page * p.page_size) * Kv4Row<D>::kBytes : 0));
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

template <int D>
__global__ void __launch_bounds__(kKv4Threads) gqa_kv4_append_kernel(const Kv4RowsParams p) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    const Kv4At a = kv4_at<D>(p);
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (a.stored) u = __ldcs(reinterpret_cast<const uint4*>(a.row));
    // (max, -min) of the row as one bf16 pair; NaN wins
    __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(bf162_of(u.x), bf162_of(u.y)), __hmax2_nan(bf162_of(u.z), bf162_of(u.w)));
    __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(bf162_of(u.x), bf162_of(u.y)), __hmin2_nan(bf162_of(u.z), bf162_of(u.w)));
    __nv_bfloat162 mm = __halves2bfloat162(__hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi)),
                                           __hneg(__hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo))));
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
        mm = __hmax2_nan(mm, bf162_of(__shfl_xor_sync(0xffffffffu, u32_of(mm), d, kLanes)));
    const float top = __low2float(mm), m = -__high2float(mm);
    const float range = top - m;
    __nv_bfloat16 step = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
    __nv_bfloat16 least = __float2bfloat16_rn(m);
    if (!(range < __uint_as_float(0x7f800000u))) step = least = __ushort_as_bfloat16((unsigned short)0x7fc0u);  // NaN
    const float s = __bfloat162float(step);
    if (s < 1.17549435e-38f) step = __ushort_as_bfloat16((unsigned short)0u);
    const float r = s < 1.17549435e-38f ? 0.f : __frcp_rn(s);
    const uint32_t word = kv4_codes(u, m, r);
    if (!a.stored) return;
    a.packed[j] = word;
    if (j == 0) a.packed[kLanes] = (uint32_t)__bfloat16_as_ushort(step) | (uint32_t)__bfloat16_as_ushort(least) << 16;
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads) gqa_kv4_gather_kernel(const Kv4RowsParams p) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    const Kv4At a = kv4_at<D>(p);
    if (!a.live) return;
    uint4 out = make_uint4(0u, 0u, 0u, 0u);  // a slot outside the pool reads as zeros
    if (a.stored) {
        const uint32_t word = a.packed[j], head = a.packed[kLanes];
        const float s = __uint_as_float(head << 16), m = __uint_as_float(head & 0xffff0000u);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // 2^23 + code as float bits; the difference is the code, exactly
            const float code = __uint_as_float(0x4B000000u | ((word >> (4 * i)) & 15u)) - 8388608.f;
            f[i] = fmaf(code, s, m);
        }
        out = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7]));
    }
    *reinterpret_cast<uint4*>(a.row) = out;
}

}  // namespace gqa

// RMS norm of each query and key head with the position rotation in the same pass, its
// backward pass, and the serving form that writes keys and values into their cache pages.
//
//   n = x * rsqrt(mean(x^2) + eps),  y = n * w,  z = R(pos) y
//
// R(pos) turns each pair (a, b) of the first `rot` elements by its angle:
// (a c - b s, b c + a s); pairs are (i, i + rot/2), or (2i, 2i + 1) when interleaved. cos and
// sin come from the caller's fp32 table, so the angles of far positions are as exact as the
// caller made them. Without a weight x is not normalised; without a table it is not rotated.
//
// Backward, with g = R(pos)^T dz and e = g * w:
//   dw = sum over rows of g * n,   dx = rsqrt(...) * (e - n * mean(e * n)).
// n is computed again from x, which costs a read that the pass makes anyway.
//
// All of it is bound by HBM: a row is read once and written once (backward: two reads). What has to
// be kept small beside it is instructions. D/8 lanes take a row, each lane eight elements in two
// groups of four that hold whole pairs, so the rotation needs no exchange, and packed pairs of
// fp32 do the arithmetic. A lane keeps its angles and weights in registers over the heads of a
// token, four rows at a time: their sums over the lanes are formed together, each step of the
// exchange halving the rows that a lane still adds up, so four rows cost five exchanges and one
// reciprocal root instead of sixteen and four. Everything between the loads and the one rounding
// to bf16 at the end is fp32.
//
// 4 x 4096 tokens, 32 + 8 heads of 128: forward 57 us, 5.9 TB/s, 90 % of the measured copy rate
// (77 us with every row summed by itself); backward 98 us, 78 % (16 warps an SM, whose loads do
// not all overlap; 106 us once the power limit holds the SMs at 1850 of their 1965 MHz). 35197 tokens appended:
// 148 us, 91 %. 64 tokens appended: 3.5 us, a launch.
#pragma once

#include "sm100_ptx.cuh"

namespace gqa {

constexpr int kRopeThreads = 256;

// One operand's rows: element (b, h, t, d) at p + b*sb + h*sh + t*st + d.
struct RopeRows {
    const __nv_bfloat16* in;
    __nv_bfloat16* out;
    const __nv_bfloat16* grad;  // backward: the output gradient
    long long in_sb, in_sh, in_st;
    long long out_sb, out_sh, out_st;
    long long grad_sb, grad_sh, grad_st;
    const void* weight;  // [D] bf16 or fp32, or null: no norm
    int H;
};

constexpr int kRopeUnroll = 4;  // rows a team takes at a time

struct RopeParams {
    RopeRows x[3];       // queries, keys, values (values only when appending; copied)
    const float* cos;    // [n_positions, rot/2] or null
    const float* sin;
    const int* positions;  // element (b, t) at b*pos_sb + t, or null: t
    long long pos_sb;
    int n_positions;
    int B, T, rot;
    int weight_fp32;
    float eps;
    // appending: rows of x[1], x[2] go to row slot % page_size of pool page slot / page_size
    // (out_sb: page stride, out_st: row stride)
    const int* slots;  // [T], or null: not appending
    int page_size, num_pages;
    int heads_per_team;  // rows of one token that a team takes in turn
    int blocks[3];       // head blocks of each operand; forward: gridDim.y is their sum
    float* partial;      // backward: [gridDim.x, D] sums of dw
    int q_ctas;          // backward: CTAs that take queries, the first ones
    uint32_t* err;
};

struct RopeLane {
    int e0, e1;  // this lane's two groups of four elements
    int angle;   // index of the first of its four angles, -1: not rotated
};

template <int D, bool kInterleaved>
__device__ __forceinline__ RopeLane rope_lane(int j, int rot) {
    RopeLane l;
    if (kInterleaved) {
        l.e0 = 8 * j;
        l.e1 = 8 * j + 4;
        l.angle = 8 * j < rot ? 4 * j : -1;
    } else {
        const int i = 4 * j, half = rot >> 1;
        if (i < half) {
            l.e0 = i;
            l.e1 = i + half;
            l.angle = i;
        } else {  // the rest of the row, in two halves of its own
            l.e0 = rot + (i - half);
            l.e1 = l.e0 + ((D - rot) >> 1);
            l.angle = -1;
        }
    }
    return l;
}

// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t rope2(float lo, float hi) { return f2_pack(lo, hi); }
__device__ __forceinline__ uint64_t rope2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t rope2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float rope2_sum(uint64_t a) {
    float lo, hi;
    f2_unpack(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ uint64_t rope2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }

// A lane's eight elements as the first and second elements of its four pairs, two pairs a register.
struct RopePairs {
    uint64_t a[2], b[2];
};
__device__ __forceinline__ uint64_t rope_lows(uint32_t u, uint32_t v) {
    return rope2(__uint_as_float(u << 16), __uint_as_float(v << 16));
}
__device__ __forceinline__ uint64_t rope_highs(uint32_t u, uint32_t v) {
    return rope2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint64_t rope_both(uint32_t u) {
    return rope2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t rope_round(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return pack_bf16x2(lo, hi);
}
template <bool kInterleaved>
__device__ __forceinline__ RopePairs rope_unpack(uint2 u0, uint2 u1) {
    RopePairs p;
    if (kInterleaved) {
        p.a[0] = rope_lows(u0.x, u0.y), p.b[0] = rope_highs(u0.x, u0.y);
        p.a[1] = rope_lows(u1.x, u1.y), p.b[1] = rope_highs(u1.x, u1.y);
    } else {
        p.a[0] = rope_both(u0.x), p.a[1] = rope_both(u0.y);
        p.b[0] = rope_both(u1.x), p.b[1] = rope_both(u1.y);
    }
    return p;
}
template <bool kInterleaved>
__device__ __forceinline__ void rope_pack(const RopePairs& p, uint2& u0, uint2& u1) {
    if (kInterleaved) {
        float a0, a1, b0, b1;
        f2_unpack(p.a[0], a0, a1);
        f2_unpack(p.b[0], b0, b1);
        u0 = make_uint2(pack_bf16x2(a0, b0), pack_bf16x2(a1, b1));
        f2_unpack(p.a[1], a0, a1);
        f2_unpack(p.b[1], b0, b1);
        u1 = make_uint2(pack_bf16x2(a0, b0), pack_bf16x2(a1, b1));
    } else {
        u0 = make_uint2(rope_round(p.a[0]), rope_round(p.a[1]));
        u1 = make_uint2(rope_round(p.b[0]), rope_round(p.b[1]));
    }
}
__device__ __forceinline__ uint2 rope_load(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint2*>(p)); }

// A lane's weights in the order of its pairs (without a weight: ones).
template <bool kInterleaved>
__device__ __forceinline__ RopePairs rope_weights(const void* w, int fp32, const RopeLane& l) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
    if (w != nullptr && fp32) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + l.e0));
        const float4 y = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + l.e1));
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    } else if (w != nullptr) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + l.e0));
        const uint2 y = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + l.e1));
        const uint32_t u[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    RopePairs p;
    if (kInterleaved) {
        p.a[0] = rope2(f[0], f[2]), p.b[0] = rope2(f[1], f[3]);
        p.a[1] = rope2(f[4], f[6]), p.b[1] = rope2(f[5], f[7]);
    } else {
        p.a[0] = rope2(f[0], f[1]), p.a[1] = rope2(f[2], f[3]);
        p.b[0] = rope2(f[4], f[5]), p.b[1] = rope2(f[6], f[7]);
    }
    return p;
}

// Sums of four rows' values over the team's lanes: lane j ends with the sum of row rope_row(j).
template <int kLanes>
__device__ __forceinline__ int rope_row(int j) {
    return (j & (kLanes / 2) ? 1 : 0) + (j & (kLanes / 4) ? 2 : 0);
}
template <int kLanes>
__device__ __forceinline__ float rope_sums(const float (&v)[4], int j) {
    const bool h = j & (kLanes / 2), q = j & (kLanes / 4);
    const float t0 = (h ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, h ? v[0] : v[1], kLanes / 2);
    const float t1 = (h ? v[3] : v[2]) + __shfl_xor_sync(0xffffffffu, h ? v[2] : v[3], kLanes / 2);
    float s = (q ? t1 : t0) + __shfl_xor_sync(0xffffffffu, q ? t0 : t1, kLanes / 4);
#pragma unroll
    for (int d = kLanes / 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}
// Row i's value from a lane that has it.
template <int kLanes>
__device__ __forceinline__ float rope_of_row(float v, int i) {
    return __shfl_sync(0xffffffffu, v, (i & 1 ? kLanes / 2 : 0) + (i & 2 ? kLanes / 4 : 0), kLanes);
}

// Where a team stands: its token, and its operand's heads.
struct RopeAt {
    bool live;
    int b, t, which, h0, h1;
};
__device__ __forceinline__ RopeAt rope_at(const RopeParams& p, unsigned tok, int which, int hb) {
    RopeAt a;
    a.which = which;
    a.live = tok < (unsigned)p.B * (unsigned)p.T;  // every lane stays for the exchanges
    if (!a.live) tok = 0;
    a.b = p.B == 1 ? 0 : (int)(tok / (unsigned)p.T);
    a.t = (int)(tok - (unsigned)a.b * (unsigned)p.T);
    a.h0 = hb * p.heads_per_team;
    a.h1 = min(a.h0 + p.heads_per_team, p.x[which].H);
    return a;
}
// The angles of a team's token in the lane's four pairs (1, 0 where nothing turns, as in values);
// false, with an error set, if its position is outside the tables: then a token's value row is left
// out with its key row.
__device__ __forceinline__ bool rope_angles(const RopeParams& p, const RopeAt& a, const RopeLane& l, uint64_t (&c)[2],
                                            uint64_t (&s)[2]) {
    c[0] = c[1] = rope2(1.f, 1.f);
    s[0] = s[1] = rope2(0.f, 0.f);
    if (p.cos == nullptr) return true;
    const int pos = p.positions ? __ldg(p.positions + a.b * p.pos_sb + a.t) : a.t;
    if ((unsigned)pos >= (unsigned)p.n_positions) {
        if (a.live) atomicOr(p.err, kDevErrBadSeqlens);
        return false;
    }
    if (l.angle >= 0 && a.which != 2) {
        const long long at = (long long)pos * (p.rot >> 1) + l.angle;
        const float4 x = __ldg(reinterpret_cast<const float4*>(p.cos + at)), y = __ldg(reinterpret_cast<const float4*>(p.sin + at));
        c[0] = rope2(x.x, x.y), c[1] = rope2(x.z, x.w);
        s[0] = rope2(y.x, y.y), s[1] = rope2(y.z, y.w);
    }
    return true;
}

// Forward and appending form. A team of D/8 lanes takes up to heads_per_team heads of one
// operand of one token.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) gqa_rope_fwd_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kUnroll = kRopeUnroll;
    const int j = threadIdx.x % kLanes;
    int hb = blockIdx.y;
    const int which = hb < p.blocks[0] ? 0 : hb < p.blocks[0] + p.blocks[1] ? 1 : 2;
    hb -= which == 0 ? 0 : which == 1 ? p.blocks[0] : p.blocks[0] + p.blocks[1];
    const RopeAt a = rope_at(p, blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes, which, hb);
    const RopeRows& x = p.x[a.which];
    const RopeLane l = rope_lane<D, kInterleaved>(j, p.rot);

    bool write = a.live;
    long long out = a.b * x.out_sb + a.t * x.out_st;
    if (p.slots != nullptr && a.which > 0) {
        const int slot = __ldg(p.slots + a.t);
        const int page = slot / p.page_size;
        if (slot < 0 || page >= p.num_pages) {
            if (slot >= 0 && a.live) atomicOr(p.err, kDevErrBadSeqlens);
            write = false;
            out = 0;
        } else {
            out = page * x.out_sb + (slot - page * p.page_size) * x.out_st;
        }
    }
    const bool norm = x.weight != nullptr;
    // z_a = (r x_a)(w_a c) - (r x_b)(w_b s), z_b = (r x_b)(w_b c) + (r x_a)(w_a s)
    uint64_t c[2], s[2];
    if (!rope_angles(p, a, l, c, s)) write = false;
    const RopePairs w = rope_weights<kInterleaved>(x.weight, p.weight_fp32, l);
    uint64_t ac[2], as[2], bc[2], bs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ac[i] = rope2_mul(w.a[i], c[i]);
        as[i] = rope2_mul(w.a[i], s[i]);
        bc[i] = rope2_mul(w.b[i], c[i]);
        bs[i] = rope2_neg(rope2_mul(w.b[i], s[i]));
    }
    const bool copy = !norm && (p.cos == nullptr || a.which == 2 || l.angle < 0);  // these elements stay as they are
    // the lane's first group of the next head's row; its second is `gap` elements on
    const __nv_bfloat16* in = x.in + a.b * x.in_sb + a.t * x.in_st + a.h0 * x.in_sh + l.e0;
    __nv_bfloat16* dst = x.out + out + a.h0 * x.out_sh + l.e0;
    const int gap = l.e1 - l.e0;
    for (int h = a.h0; h < a.h1; h += kUnroll) {
        uint2 u0[kUnroll], u1[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            u0[i] = u1[i] = make_uint2(0u, 0u);
            if (a.live && h + i < a.h1) {
                u0[i] = rope_load(in);
                u1[i] = rope_load(in + gap);
            }
            in += x.in_sh;
        }
        float r = 1.f;
        if (norm) {
            float sq[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const RopePairs f = rope_unpack<kInterleaved>(u0[i], u1[i]);
                uint64_t v = rope2_mul(f.a[0], f.a[0]);
                v = rope2_fma(f.a[1], f.a[1], v);
                v = rope2_fma(f.b[0], f.b[0], v);
                sq[i] = rope2_sum(rope2_fma(f.b[1], f.b[1], v));
            }
            r = rsqrtf(rope_sums<kLanes>(sq, j) * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (!copy) {
                RopePairs f = rope_unpack<kInterleaved>(u0[i], u1[i]);
                RopePairs z;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    z.a[e] = rope2_fma(f.b[e], bs[e], rope2_mul(f.a[e], ac[e]));
                    z.b[e] = rope2_fma(f.a[e], as[e], rope2_mul(f.b[e], bc[e]));
                }
                if (norm) {
                    const float ri = rope_of_row<kLanes>(r, i);
                    const uint64_t rr = rope2(ri, ri);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        z.a[e] = rope2_mul(z.a[e], rr);
                        z.b[e] = rope2_mul(z.b[e], rr);
                    }
                }
                rope_pack<kInterleaved>(z, u0[i], u1[i]);
            }
            if (write && h + i < a.h1) {
                *reinterpret_cast<uint2*>(dst) = u0[i];
                *reinterpret_cast<uint2*>(dst + gap) = u1[i];
            }
            dst += x.out_sh;
        }
    }
}

// Backward. A CTA takes one operand's rows, a strided share of its (token group, head block)s, and
// leaves one row of dw sums; gqa_rope_dw_kernel adds those up in a fixed order, so the gradients do
// not change from run to run. The operands get CTAs in proportion to their heads.
//   g = R^T dz,  dw += (g x) r,  dx = (r g) w - x (r^3 sum(g w x) / D)
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 2) gqa_rope_bwd_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kTeams = kRopeThreads / kLanes;
    constexpr int kUnroll = kRopeUnroll;
    __shared__ float sums[kTeams][D];
    const int j = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
    const RopeLane l = rope_lane<D, kInterleaved>(j, p.rot);
    const int which = (int)blockIdx.x < p.q_ctas ? 0 : 1;
    const RopeRows& x = p.x[which];
    const bool norm = x.weight != nullptr;
    const RopePairs w = rope_weights<kInterleaved>(x.weight, p.weight_fp32, l);
    RopePairs dw;
    dw.a[0] = dw.a[1] = dw.b[0] = dw.b[1] = rope2(0.f, 0.f);
    const unsigned blocks = p.blocks[which], units = ((unsigned)p.B * (unsigned)p.T + kTeams - 1) / kTeams * blocks;
    const unsigned stride = which ? gridDim.x - p.q_ctas : p.q_ctas;
    const auto place = [&](unsigned u) {  // of this team in unit u
        const unsigned group = u / blocks;
        return rope_at(p, group * kTeams + team, which, (int)(u - group * blocks));
    };
    for (unsigned u = which ? blockIdx.x - p.q_ctas : blockIdx.x; u < units; u += stride) {  // the same for every lane
        const RopeAt a = place(u);
        uint64_t c[2], s[2];
        const bool use = rope_angles(p, a, l, c, s) && a.live;
        const uint64_t ns[2] = {rope2_neg(s[0]), rope2_neg(s[1])};
        const __nv_bfloat16* in = x.in + a.b * x.in_sb + a.t * x.in_st + a.h0 * x.in_sh + l.e0;
        const __nv_bfloat16* gr = x.grad + a.b * x.grad_sb + a.t * x.grad_st + a.h0 * x.grad_sh + l.e0;
        __nv_bfloat16* out = x.out + a.b * x.out_sb + a.t * x.out_st + a.h0 * x.out_sh + l.e0;
        const int gap = l.e1 - l.e0;
        const bool copy = !norm && l.angle < 0;
        if (u + stride < units) {  // bring the next unit's rows to L2
            const RopeAt next = place(u + stride);
            constexpr int kLines = D / 64;  // of 128 bytes in a row
            const int n = next.live ? (next.h1 - next.h0) * kLines : 0;
            const __nv_bfloat16* xs = x.in + next.b * x.in_sb + next.t * x.in_st;
            const __nv_bfloat16* gs = x.grad + next.b * x.grad_sb + next.t * x.grad_st;
            for (int i = j; i < n; i += kLanes) {
                const long long h = next.h0 + i / kLines, at = i % kLines * 64;
                if (norm) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(xs + h * x.in_sh + at)));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(gs + h * x.grad_sh + at)));
            }
        }
        for (int h = a.h0; h < a.h1; h += kUnroll) {
            uint2 x0[kUnroll], x1[kUnroll], g0[kUnroll], g1[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                x0[i] = x1[i] = g0[i] = g1[i] = make_uint2(0u, 0u);
                if (a.live && h + i < a.h1) {  // whether the position is good does not hold the loads up
                    g0[i] = rope_load(gr);
                    g1[i] = rope_load(gr + gap);
                    if (norm) {
                        x0[i] = rope_load(in);
                        x1[i] = rope_load(in + gap);
                    }
                }
                gr += x.grad_sh;
                in += x.in_sh;
            }
            if (!use) {  // a bad position's rows may hold a NaN
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) x0[i] = x1[i] = g0[i] = g1[i] = make_uint2(0u, 0u);
            }
            RopePairs gs[kUnroll];  // g
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const RopePairs d = rope_unpack<kInterleaved>(g0[i], g1[i]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    gs[i].a[e] = rope2_fma(d.b[e], s[e], rope2_mul(d.a[e], c[e]));
                    gs[i].b[e] = rope2_fma(d.a[e], ns[e], rope2_mul(d.b[e], c[e]));
                }
            }
            float r = 1.f, k = 0.f;  // of the lane's row of the four
            if (norm) {
                float sq[kUnroll], dot[kUnroll];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    const RopePairs f = rope_unpack<kInterleaved>(x0[i], x1[i]);
                    const RopePairs& g = gs[i];
                    uint64_t u = rope2(0.f, 0.f), v = u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u = rope2_fma(f.a[e], f.a[e], u);
                        u = rope2_fma(f.b[e], f.b[e], u);
                        v = rope2_fma(rope2_mul(g.a[e], f.a[e]), w.a[e], v);
                        v = rope2_fma(rope2_mul(g.b[e], f.b[e]), w.b[e], v);
                    }
                    sq[i] = rope2_sum(u);
                    dot[i] = rope2_sum(v);
                }
                r = rsqrtf(rope_sums<kLanes>(sq, j) * (1.f / D) + p.eps);
                k = -rope_sums<kLanes>(dot, j) * (1.f / D) * r * r * r;
                // rows that are not there add nothing to dw, whatever eps is
                if (!use || h + rope_row<kLanes>(j) >= a.h1) r = k = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                uint2 u0 = g0[i], u1 = g1[i];
                if (!copy) {
                    RopePairs& g = gs[i];
                    if (norm) {
                        const RopePairs f = rope_unpack<kInterleaved>(x0[i], x1[i]);
                        const float ri = rope_of_row<kLanes>(r, i), ki = rope_of_row<kLanes>(k, i);
                        const uint64_t rr = rope2(ri, ri), kk = rope2(ki, ki);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint64_t ga = rope2_mul(g.a[e], rr), gb = rope2_mul(g.b[e], rr);
                            dw.a[e] = rope2_fma(ga, f.a[e], dw.a[e]);
                            dw.b[e] = rope2_fma(gb, f.b[e], dw.b[e]);
                            g.a[e] = rope2_fma(ga, w.a[e], rope2_mul(f.a[e], kk));
                            g.b[e] = rope2_fma(gb, w.b[e], rope2_mul(f.b[e], kk));
                        }
                    }
                    rope_pack<kInterleaved>(g, u0, u1);
                }
                if (use && h + i < a.h1) {
                    *reinterpret_cast<uint2*>(out) = u0;
                    *reinterpret_cast<uint2*>(out + gap) = u1;
                }
                out += x.out_sh;
            }
        }
    }
    if (!norm) return;  // uniform over the CTA
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float a0, a1, b0, b1;
        f2_unpack(dw.a[e], a0, a1);
        f2_unpack(dw.b[e], b0, b1);
        if (kInterleaved) {
            float* at = sums[team] + (e ? l.e1 : l.e0);
            at[0] = a0, at[1] = b0, at[2] = a1, at[3] = b1;
        } else {
            sums[team][l.e0 + 2 * e] = a0, sums[team][l.e0 + 2 * e + 1] = a1;
            sums[team][l.e1 + 2 * e] = b0, sums[team][l.e1 + 2 * e + 1] = b1;
        }
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kTeams; ++i) v += sums[i][threadIdx.x];
        p.partial[(long long)blockIdx.x * D + threadIdx.x] = v;
    }
}

// dw[d] = sum of the CTAs' partial sums; blockIdx.x 0: queries, 1: keys; eight columns a CTA, so
// that a thread has few rows to wait for.
constexpr int kRopeDwColumns = 8;
template <int D>
__global__ void __launch_bounds__(1024) gqa_rope_dw_kernel(const float* partial, int q_rows, int rows, float* dq_w, float* dk_w) {
    constexpr int kGroups = 1024 / kRopeDwColumns;
    __shared__ float sums[kGroups][kRopeDwColumns + 1];
    float* out = blockIdx.x ? dk_w : dq_w;
    if (out == nullptr) return;
    const int lo = blockIdx.x ? q_rows : 0, hi = blockIdx.x ? rows : q_rows;
    const int c = threadIdx.x % kRopeDwColumns, g = threadIdx.x / kRopeDwColumns, d = blockIdx.y * kRopeDwColumns + c;
    float v = 0.f;
#pragma unroll 8
    for (int i = lo + g; i < hi; i += kGroups) v += partial[(long long)i * D + d];
    sums[g][c] = v;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= kRopeDwColumns) return;
    v = 0.f;
#pragma unroll
    for (int i = lane; i < kGroups; i += 32) v += sums[i][warp];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    if (lane == 0) out[blockIdx.y * kRopeDwColumns + warp] = v;
}

}  // namespace gqa

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
// All of it is bound by HBM: a row is read once and written once (backward: two reads). D/8
// lanes take a row, each lane eight elements in two groups of four that hold whole pairs, so
// the rotation needs no exchange and the row's sum is D/8-lane shuffles. A lane keeps its cos,
// sin and weights in registers over the heads of one token. Everything between the loads and
// the one rounding to bf16 at the end is fp32.
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
    int blocks[3];       // head blocks of each operand
    float* partial;      // backward: [gridDim.x, D] sums of dw, queries' blocks first
    int q_blocks;        // backward: CTAs that take queries
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

__device__ __forceinline__ void rope_unpack(uint2 u, float* f) {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 rope_pack(const float* f) {
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ uint2 rope_load(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint2*>(p)); }

__device__ __forceinline__ void rope_weight(const void* w, int fp32, int e, float* f) {
    if (fp32) {
        for (int i = 0; i < 4; ++i) f[i] = static_cast<const float*>(w)[e + i];
    } else {
        for (int i = 0; i < 4; ++i) f[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[e + i]);
    }
}

// Turn the eight elements' pairs by +angle (dir = 1) or -angle (dir = -1).
template <bool kInterleaved>
__device__ __forceinline__ void rope_turn(float* a, float* b, const float4& c, const float4& s, float dir) {
    const float cs[4] = {c.x, c.y, c.z, c.w};
    const float sn[4] = {s.x * dir, s.y * dir, s.z * dir, s.w * dir};
    if (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            a[2 * i] = a0 * cs[i] - a1 * sn[i];
            a[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
            b[2 * i] = b0 * cs[2 + i] - b1 * sn[2 + i];
            b[2 * i + 1] = b1 * cs[2 + i] + b0 * sn[2 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = y * cs[i] + x * sn[i];
        }
    }
}

template <int kLanes>
__device__ __forceinline__ float rope_team_sum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d, kLanes);
    return v;
}

// Forward and appending form. A team of D/8 lanes takes up to heads_per_team heads of one
// operand of one token; kUnroll rows are loaded before the first is used.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) gqa_rope_fwd_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kUnroll = 4;
    const int j = threadIdx.x % kLanes;
    const long long team = (long long)blockIdx.x * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
    const int per_token = p.blocks[0] + p.blocks[1] + p.blocks[2];
    long long tok = team / per_token;
    int hb = (int)(team - tok * per_token);
    const bool live = tok < (long long)p.B * p.T;  // every lane stays for the shuffles
    if (!live) tok = hb = 0;
    const int b = (int)(tok / p.T), t = (int)(tok - (long long)b * p.T);
    int which = 0;
    while (hb >= p.blocks[which]) hb -= p.blocks[which++];
    const RopeRows& x = p.x[which];
    const RopeLane l = rope_lane<D, kInterleaved>(j, p.rot);

    bool write = live;
    long long out = (long long)b * x.out_sb + (long long)t * x.out_st;
    if (p.slots != nullptr && which > 0) {
        const int slot = p.slots[t];
        const int page = slot / p.page_size;
        if (slot < 0 || page >= p.num_pages) {
            if (slot >= 0 && live && j == 0) atomicOr(p.err, kDevErrBadSeqlens);
            write = false;
            out = 0;
        } else {
            out = (long long)page * x.out_sb + (long long)(slot - page * p.page_size) * x.out_st;
        }
    }
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool turn = p.cos != nullptr && which < 2;
    if (turn) {
        const int pos = p.positions ? p.positions[(long long)b * p.pos_sb + t] : t;
        if (pos < 0 || pos >= p.n_positions) {
            if (live && j == 0) atomicOr(p.err, kDevErrBadSeqlens);
            write = false;
        } else if (l.angle >= 0) {
            c = *reinterpret_cast<const float4*>(p.cos + (long long)pos * (p.rot >> 1) + l.angle);
            s = *reinterpret_cast<const float4*>(p.sin + (long long)pos * (p.rot >> 1) + l.angle);
        }
    }
    float w0[4], w1[4];
    const bool norm = x.weight != nullptr;
    if (norm) {
        rope_weight(x.weight, p.weight_fp32, l.e0, w0);
        rope_weight(x.weight, p.weight_fp32, l.e1, w1);
    }
    const int h0 = hb * p.heads_per_team, h1 = min(h0 + p.heads_per_team, x.H);
    const __nv_bfloat16* in = x.in + (long long)b * x.in_sb + (long long)t * x.in_st;
    for (int h = 0; h < p.heads_per_team; h += kUnroll) {
        uint2 u0[kUnroll], u1[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int hh = h0 + h + i;
            u0[i] = u1[i] = make_uint2(0u, 0u);
            if (live && h + i < p.heads_per_team && hh < h1) {
                u0[i] = rope_load(in + hh * x.in_sh + l.e0);
                u1[i] = rope_load(in + hh * x.in_sh + l.e1);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (h + i >= p.heads_per_team) break;  // the same for every lane
            const int hh = h0 + h + i;
            float f0[4], f1[4];
            rope_unpack(u0[i], f0);
            rope_unpack(u1[i], f1);
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sq += f0[e] * f0[e] + f1[e] * f1[e];
            sq = rope_team_sum<kLanes>(sq);
            if (norm) {
                const float r = rsqrtf(sq * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f0[e] *= r * w0[e];
                    f1[e] *= r * w1[e];
                }
            }
            if (turn && l.angle >= 0) rope_turn<kInterleaved>(f0, f1, c, s, 1.f);
            if (norm || turn) {
                u0[i] = rope_pack(f0);
                u1[i] = rope_pack(f1);
            }
            if (write && hh < h1) {
                __nv_bfloat16* o = x.out + out + hh * x.out_sh;
                *reinterpret_cast<uint2*>(o + l.e0) = u0[i];
                *reinterpret_cast<uint2*>(o + l.e1) = u1[i];
            }
        }
    }
}

// Backward. A CTA takes rows of one operand only, a strided share of its (token, head block)s,
// and leaves one row of dw sums; gqa_rope_dw_kernel adds those up in a fixed order, so the
// gradients do not change from run to run.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) gqa_rope_bwd_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kTeams = kRopeThreads / kLanes;
    constexpr int kUnroll = 2;
    __shared__ float sums[kTeams][D];
    const int j = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
    const int which = (int)blockIdx.x < p.q_blocks ? 0 : 1;
    const RopeRows& x = p.x[which];
    const int cta = which ? blockIdx.x - p.q_blocks : blockIdx.x;
    const int ctas = which ? gridDim.x - p.q_blocks : p.q_blocks;
    const RopeLane l = rope_lane<D, kInterleaved>(j, p.rot);
    const bool norm = x.weight != nullptr, turn = p.cos != nullptr;
    float w0[4], w1[4], d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
    if (norm) {
        rope_weight(x.weight, p.weight_fp32, l.e0, w0);
        rope_weight(x.weight, p.weight_fp32, l.e1, w1);
    }
    const long long units = (long long)p.B * p.T * p.blocks[which];
    for (long long u0 = (long long)cta * kTeams; u0 < units; u0 += (long long)ctas * kTeams) {
        long long u = u0 + team;
        const bool live = u < units;
        if (!live) u = 0;
        const long long tok = u / p.blocks[which];
        const int hb = (int)(u - tok * p.blocks[which]);
        const int b = (int)(tok / p.T), t = (int)(tok - (long long)b * p.T);
        bool use = live;
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turn) {
            const int pos = p.positions ? p.positions[(long long)b * p.pos_sb + t] : t;
            if (pos < 0 || pos >= p.n_positions) {
                if (live && j == 0) atomicOr(p.err, kDevErrBadSeqlens);
                use = false;
            } else if (l.angle >= 0) {
                c = *reinterpret_cast<const float4*>(p.cos + (long long)pos * (p.rot >> 1) + l.angle);
                s = *reinterpret_cast<const float4*>(p.sin + (long long)pos * (p.rot >> 1) + l.angle);
            }
        }
        const int h0 = hb * p.heads_per_team, h1 = min(h0 + p.heads_per_team, x.H);
        const __nv_bfloat16* in = x.in + (long long)b * x.in_sb + (long long)t * x.in_st;
        const __nv_bfloat16* gr = x.grad + (long long)b * x.grad_sb + (long long)t * x.grad_st;
        __nv_bfloat16* out = x.out + (long long)b * x.out_sb + (long long)t * x.out_st;
        for (int h = 0; h < p.heads_per_team; h += kUnroll) {
            uint2 a0[kUnroll], a1[kUnroll], g0[kUnroll], g1[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int hh = h0 + h + i;
                a0[i] = a1[i] = g0[i] = g1[i] = make_uint2(0u, 0u);
                if (use && h + i < p.heads_per_team && hh < h1) {
                    g0[i] = rope_load(gr + hh * x.grad_sh + l.e0);
                    g1[i] = rope_load(gr + hh * x.grad_sh + l.e1);
                    if (norm) {
                        a0[i] = rope_load(in + hh * x.in_sh + l.e0);
                        a1[i] = rope_load(in + hh * x.in_sh + l.e1);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (h + i >= p.heads_per_team) break;  // the same for every lane
                const int hh = h0 + h + i;
                const bool row = use && hh < h1;
                float f0[4], f1[4], n0[4], n1[4];
                rope_unpack(g0[i], f0);
                rope_unpack(g1[i], f1);
                if (turn && l.angle >= 0) rope_turn<kInterleaved>(f0, f1, c, s, -1.f);
                if (norm) {
                    rope_unpack(a0[i], n0);
                    rope_unpack(a1[i], n1);
                    float sq = 0.f, dot = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sq += n0[e] * n0[e] + n1[e] * n1[e];
                        dot += f0[e] * w0[e] * n0[e] + f1[e] * w1[e] * n1[e];
                    }
                    sq = rope_team_sum<kLanes>(sq);
                    dot = rope_team_sum<kLanes>(dot);
                    // rows that are not there add nothing to dw, whatever eps is
                    const float r = row ? rsqrtf(sq * (1.f / D) + p.eps) : 0.f;
                    const float m = dot * r * (1.f / D);  // mean(e * n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        n0[e] *= r;
                        n1[e] *= r;
                        d0[e] += f0[e] * n0[e];
                        d1[e] += f1[e] * n1[e];
                        f0[e] = r * (f0[e] * w0[e] - n0[e] * m);
                        f1[e] = r * (f1[e] * w1[e] - n1[e] * m);
                    }
                }
                if (row) {
                    *reinterpret_cast<uint2*>(out + hh * x.out_sh + l.e0) = rope_pack(f0);
                    *reinterpret_cast<uint2*>(out + hh * x.out_sh + l.e1) = rope_pack(f1);
                }
            }
        }
    }
    if (!norm) return;  // uniform over the CTA
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sums[team][l.e0 + e] = d0[e];
        sums[team][l.e1 + e] = d1[e];
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float v = 0.f;
        for (int i = 0; i < kTeams; ++i) v += sums[i][threadIdx.x];
        p.partial[(long long)blockIdx.x * D + threadIdx.x] = v;
    }
}

// dw[d] = sum of the CTAs' partial sums; CTA 0: queries, CTA 1: keys.
template <int D>
__global__ void __launch_bounds__(1024) gqa_rope_dw_kernel(const float* partial, int q_blocks, int blocks, float* dq_w,
                                                           float* dk_w) {
    constexpr int kGroups = 1024 / D;
    __shared__ float sums[kGroups][D];
    float* out = blockIdx.x ? dk_w : dq_w;
    if (out == nullptr) return;
    const int lo = blockIdx.x ? q_blocks : 0, hi = blockIdx.x ? blocks : q_blocks;
    const int d = threadIdx.x % D, g = threadIdx.x / D;
    float v = 0.f;
#pragma unroll 8
    for (int i = lo + g; i < hi; i += kGroups) v += partial[(long long)i * D + d];
    sums[g][d] = v;
    __syncthreads();
    if (g == 0) {
        v = 0.f;
        for (int i = 0; i < kGroups; ++i) v += sums[i][d];
        out[d] = v;
    }
}

}  // namespace gqa

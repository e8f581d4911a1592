// Decode over a paged cache held in 4 bits (rows as kv4_rows_sm100.cuh writes them): up to 16
// new queries a sequence, any group size, optional sliding window.
//
// A stored row is k_j = s_j c_j + m_j with codes c in 0..15, so
//   q . k_j = s_j (q . c_j) + m_j sum(q),
//   sum_j p_j v_j = sum_j w_j (c_j - 8) + sum_j p_j (m_j + 8 s_j),   w_j = fp16(p_j s_j):
// the scales stay out of the products, which run on tensor cores in fp16 with fp32 sums. A code
// needs no conversion: its bits, masked out of the word, are the fp16 subnormal c * 2^-24 (16 c four
// bits up), so eight codes cost four logic operations and one shift. q is exact in fp16 after a
// scaling by a power of two a row (see below). w is the only operand that is rounded; it is
// scaled by the largest step seen, since a probability times a step can be of any size, and summed
// about the middle of the code range (sum_j 8 w_j is one more product). Over long sequences the fp32 sums'
// own rounding shows too, since the two differ by little then: 64 sequences of 4096 to 32768 keys are off by 0.0020 of
// the output where sums in 32 bits of unpacked rows are by 0.0017, both mostly the rounding to bf16; one of 4099 keys by 0.0017. A row's NaN can only reach
// the queries that see the key: the codes themselves are always finite.
//
// Keys are the M dimension of the products and query rows their N (8 a tile), so that one
// unpacked fragment serves every query row of the KV head. mma m16n8k16 takes any order of the
// contracted index as long as both operands agree; the orders here are chosen so that every
// fragment is whole 32-bit words of the packed rows: a row is D/8 + 1 words, which makes the
// lanes' words (keys 4g + c, words t + 4i) fall on 32 different banks without padding or swizzle.
// Values and probabilities go to their operand layouts with 8x8 transposes (movmatrix, which leaves
// the logic pipe alone). The unpacked operands are born in registers, which warp-level products
// take as they are; tensor memory would take a store and a wait a tile more, and the tensor pipe is
// at 30 %.
//
// Work, two forms. Few tiles: a cluster takes each (sequence, KV head, row chunk), its warps equal
// parts of the tiles, and merges through shared memory: one launch (4099 keys, 8 KV heads of 4
// queries, D = 128: 8.4 us; with runs and a merge 12.5). Many: the tiles of all units laid end
// to end are cut into equal runs, one per warp, so all warps finish together whatever the lengths;
// a unit cut between warps leaves fp32 partials that a second kernel merges in a fixed order. A warp
// has a ring of its own that its own lanes fill with bulk copies (a page's rows of one head are
// contiguous): no warp waits for another.
//
// The bytes are D + 8 a key and KV head; what bounds it is instructions. 64 sequences of 4096 to
// 32768 keys, 8 KV heads of 4 queries, D = 128: 224 us, 5.9 TB/s, 90 % of the measured copy rate, as long as the
// SMs run at 1965 MHz; after half a second of such calls the power limit holds them near 1700 MHz and it is
// 264 to 275 us, 4.9 to 5.0 TB/s, 74 to 77 %. 449 instructions a 32 keys, 54 % of the issue slots and 55 % of the
// logic pipe (12 warps an SM; 16 with smaller rings were no faster). 64-key tiles where the
// scores fit the registers: 32-key tiles took 8 % longer, by what is done once a tile.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "sm100_ptx.cuh"

namespace gqa {

constexpr int kD4MergeWarps = 8;
constexpr int kD4MinRun = 2;  // tiles: shorter runs would leave more pieces to merge than they save

struct Dec4Params {
    const __nv_bfloat16* q;  // [B, Hq, Tq, D]
    __nv_bfloat16* o;
    const uint8_t* k;
    const uint8_t* v;
    long long k_sb, k_sh, v_sb, v_sh;  // bytes
    const int* seqlens;
    const int* table;
    int B, Hq, Hkv, G, Tq;
    int n_rc;  // chunks of query rows a group
    int page_size, num_pages, max_pages, capacity, window;
    float scale_log2;
    float* part;      // [2 * warps, rows, D] partial outputs
    float* part_lse;  // [2 * warps, rows] log2-domain log-sum-exp
    int2* ends;       // [B * Hkv * n_rc] first and last run of each unit's pieces
    int runs;         // that the workspace has room for
    uint32_t* err;
    unsigned long long timeout_ns;
};

template <int D, int NT>
struct Dec4Cfg {
    static constexpr int kRows = 8 * NT;                // query rows a warp takes
    static constexpr int kRow = D / 2 + 4;              // bytes of a stored row
    // groups of 32 keys (two m16 tiles) in a tile: two, where the registers hold their scores
    static constexpr int kGroups = NT * D <= 128 ? 2 : 1;
    static constexpr int kKeys = 32 * kGroups;
    static constexpr int kTile = kKeys * kRow;          // K or V rows of a tile
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStages = NT * D <= 128 ? 2 : NT == 4 ? 4 : 3;
    static constexpr int kWarps = NT == 4 ? 8 : 6;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtasPerSm = NT == 4 ? 1 : 2;
    static constexpr int kQBytes = NT == 1 ? 0 : (D / 32) * NT * 32 * 16;  // Q fragments, in registers for one tile
    static constexpr int kWarpBytes = kStages * kStage + kQBytes;
    static constexpr int kMergeOff = kWarps * kWarpBytes;  // a CTA's state, for its cluster to read
    static constexpr int kMergeBytes = (kRows * D + 2 * kRows) * 4;
    static constexpr int kCtlOff = kMergeOff + kMergeBytes;
    struct Ctl {
        uint64_t full[kWarps][kStages];
        unsigned long long sums[kWarps];
        unsigned long long first[kWarps];  // tiles before the sequence that holds a warp's first one
        int b[kWarps];                     // that sequence
        uint32_t abort;
    };
    static constexpr int kBytes = kCtlOff + (int)sizeof(Ctl);
    static_assert(kTile % 16 == 0 && kWarpBytes % 16 == 0, "bulk copies need 16 bytes");
    static_assert(kCtasPerSm * (kBytes + 1024) <= 233472, "shared memory of an SM");
    static_assert(kMergeBytes <= kWarpBytes, "a warp hands its state over in its ring");
};

// Tiles of one sequence: [first, first + n). A valid sequence has at least one, so that the
// rows of an empty one are written too; one outside [0, capacity] has none.
struct Dec4Seq {
    int len, first, n;
};
template <int kKeys>
__device__ __forceinline__ Dec4Seq dec4_seq(const Dec4Params& p, int b) {
    Dec4Seq s;
    s.len = __ldg(p.seqlens + b);
    s.first = s.n = 0;
    if (s.len < 0 || s.len > p.capacity) return s;
    const long long lo = p.window > 0 ? (long long)s.len - p.Tq - p.window + 1 : 0;
    s.first = lo > 0 ? (int)(lo / kKeys) : 0;
    s.n = max(1, (s.len + kKeys - 1) / kKeys - s.first);
    return s;
}

// Runs that `total` tiles are cut into, of at most `places`, and the start of run i; total is below
// 2^52 (checked on the host) and runs at most a few thousand.
__host__ __device__ __forceinline__ unsigned dec4_runs(unsigned long long total, unsigned places) {
    const unsigned long long most = (total + kD4MinRun - 1) / kD4MinRun;
    return most < places ? (unsigned)most : places;
}
__host__ __device__ __forceinline__ unsigned long long dec4_cut(unsigned long long total, unsigned i, unsigned runs) {
    if (total < 1u << 19 && runs <= 1u << 13) return (unsigned)total * i / runs;  // i <= runs: 32 bits do
    return total * i / runs;
}

// Codes as fp16 numbers without a conversion: below 2^-14 the format is linear, so the bits of a
// code are the number c * 2^-24, and four bits up 16 c * 2^-24. Pairs of nibbles e of a word's low
// half and of its high half: e = 0, 2 at factor 1, e = 1, 3 at factor 16.
__device__ __forceinline__ void dec4_codes(uint32_t w, uint32_t (&d)[4]) {
    const uint32_t up = w >> 8;
    d[0] = w & 0x000F000Fu;
    d[1] = w & 0x00F000F0u;
    d[2] = up & 0x000F000Fu;
    d[3] = up & 0x00F000F0u;
}
// The step and the minimum of a row from its last word.
__device__ __forceinline__ float dec4_step(uint32_t head) { return __uint_as_float(head << 16); }
__device__ __forceinline__ float dec4_least(uint32_t head) { return __uint_as_float(head & 0xffff0000u); }
__device__ __forceinline__ uint32_t dec4_halves(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Exponent field e of |x| for scaling x to [2^kTo, 2^(kTo + 1)), by dec4_up, and for taking products
// with the codes back, by dec4_down (2^24 times the inverse); kept where both are normal numbers
// (|x| from 2^-112 to 2^113).
__device__ __forceinline__ int dec4_exponent(float x) { return min(max((int)(__float_as_uint(x) >> 23), 15), 240); }
__device__ __forceinline__ float dec4_pow2(int field) { return __uint_as_float((uint32_t)field << 23); }
template <int kTo>
__device__ __forceinline__ float dec4_up(int e) { return dec4_pow2(254 + kTo - e); }
template <int kTo>
__device__ __forceinline__ float dec4_down(int e) { return dec4_pow2(e + 24 - kTo); }
// The running maximum of a row's scores (log2 units) is raised once they pass it by more than kD4Slack:
// a probability is then below 2^kD4Slack, and few tiles have to rescale what they add to (of 16
// rows, one nearly always has a new maximum). w = p * step stays below 2^15.
constexpr float kD4Slack = 4.f;
constexpr int kD4StepTo = 10;  // the largest step yet is scaled to [2^10, 2^11)
constexpr float kD4Lowest = -3.402823466e38f;  // the maximum of no scores

// Two fp32 values in one instruction, denormals kept.
__device__ __forceinline__ void dec4_fma2(float (&d)[2], const float (&a)[2], const float (&b)[2], const float (&c)[2]) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_pack(a[0], a[1])), "l"(f2_pack(b[0], b[1])), "l"(f2_pack(c[0], c[1])));
    f2_unpack(r, d[0], d[1]);
}
__device__ __forceinline__ void dec4_mul2(float (&d)[2], const float (&a)[2], const float (&b)[2]) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_pack(a[0], a[1])), "l"(f2_pack(b[0], b[1])));
    f2_unpack(r, d[0], d[1]);
}
__device__ __forceinline__ void dec4_add2(float (&d)[2], const float (&a)[2]) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_pack(d[0], d[1])), "l"(f2_pack(a[0], a[1])));
    f2_unpack(r, d[0], d[1]);
}

// D = A(16x16 fp16, row) * B(16x8 fp16, col) + C, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// kCluster: the form for few tiles; the states are merged in the CTA, then over the cluster.
template <int D, int NT, bool kCluster>
__global__ void __launch_bounds__(Dec4Cfg<D, NT>::kThreads, Dec4Cfg<D, NT>::kCtasPerSm) gqa_decode_kv4_kernel(const Dec4Params p) {
    namespace cg = cooperative_groups;
    using C = Dec4Cfg<D, NT>;
    constexpr int kStages = C::kStages;
    constexpr int kWarps = C::kWarps;
    constexpr int U = C::kGroups;
    constexpr int kKeys = C::kKeys;
    constexpr int RW = C::kRow / 4;  // words of a stored row
    constexpr int kKI = D / 32;      // word groups of a key row: four words, one a lane of a quad
    constexpr int kVI = D / 64;      // word groups of a value row: eight words, one a quad
    constexpr int kMT = D / 16;      // m16 tiles of the output's d
    extern __shared__ __align__(16) uint8_t dec4_smem[];
    typename C::Ctl* ctl = reinterpret_cast<typename C::Ctl*>(dec4_smem + C::kCtlOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = dec4_smem + warp * C::kWarpBytes;
    const uint32_t ring_addr = smem_u32(ring);
    const uint32_t bars = smem_u32(&ctl->full[warp][0]);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
        if (warp == 0) ctl->abort = 0;
        fence_mbar_init();
    }

    // ---- this warp's run of tiles and the sequence it starts in. Neighbouring runs go to
    // different CTAs, so that few tiles spread over all SMs.
    const int units = p.Hkv * p.n_rc;  // units of a sequence
    const auto work_of = [&](int b) { return b < p.B ? (unsigned long long)dec4_seq<kKeys>(p, b).n * units : 0ull; };
    const unsigned run = warp * gridDim.x + blockIdx.x;
    unsigned long long at, end;  // this warp's tiles
    unsigned long long seq0;     // tiles before sequence b
    int b;
    Dec4Seq s;
    if constexpr (kCluster) {
        const unsigned ctas = cg::this_cluster().num_blocks(), unit = blockIdx.x / ctas;
        b = (int)(unit / (unsigned)units);
        s = dec4_seq<kKeys>(p, b);
        if (s.n == 0) {  // the whole cluster leaves
            if (threadIdx.x == 0) atomicOr(p.err, kDevErrBadSeqlens);
            return;
        }
        const unsigned i = cg::this_cluster().block_rank() * kWarps + warp;
        seq0 = 0;
        at = (unsigned long long)(unit - b * units) * s.n;
        end = at + dec4_cut(s.n, i + 1, ctas * kWarps);
        at += dec4_cut(s.n, i, ctas * kWarps);
        __syncthreads();  // the barriers and the flag are set up
    } else {
        const bool one_pass = p.B <= C::kThreads;
        unsigned long long total = 0;
        if (!one_pass) {
            for (int b = threadIdx.x; b < p.B; b += C::kThreads) total += work_of(b);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
            if (lane == 0) ctl->sums[warp] = total;
            __syncthreads();
            total = 0;
            for (int w = 0; w < kWarps; ++w) total += ctl->sums[w];
            __syncthreads();
        }
        unsigned runs = 0;
        unsigned long long before = 0;  // tiles of the rounds of sequences already seen
        for (int b0 = 0; b0 < p.B; b0 += C::kThreads) {
            const int b = b0 + threadIdx.x;
            const unsigned long long x = work_of(b);
            unsigned long long inc = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += y;
            }
            if (lane == 31) ctl->sums[warp] = inc;
            __syncthreads();
            unsigned long long lo = before + inc - x;
            for (int w = 0; w < warp; ++w) lo += ctl->sums[w];
            for (int w = 0; w < kWarps; ++w) before += ctl->sums[w];
            if (one_pass) total = before;
            runs = dec4_runs(total, gridDim.x * kWarps);
            for (int w = 0; w < kWarps; ++w) {
                const unsigned r = w * gridDim.x + blockIdx.x;
                const unsigned long long first = r < runs ? dec4_cut(total, r, runs) : total;
                if (lo <= first && first < lo + x) {
                    ctl->b[w] = b;
                    ctl->first[w] = lo;
                }
            }
            if (blockIdx.x == 0 && b < p.B && x == 0) atomicOr(p.err, kDevErrBadSeqlens);
            __syncthreads();
        }
        if (run >= runs) return;
        at = dec4_cut(total, run, runs);
        end = dec4_cut(total, run + 1, runs);
        b = ctl->b[warp];
        seq0 = ctl->first[warp];
        s = dec4_seq<kKeys>(p, b);
    }

    const int box = min(p.page_size, kKeys);  // rows of one bulk copy
    const int boxes = kKeys / box;
    const unsigned all_boxes = (1u << boxes) - 1;
    const int page_step = kKeys / p.page_size, row_step = kKeys - page_step * p.page_size;
    volatile uint32_t* abort_flag = &ctl->abort;
    int stage = 0;
    uint32_t phase = 0;

    do {  // a warp of a cluster without a tile still joins the merge
        while (!kCluster && at >= seq0 + (unsigned long long)s.n * units) {  // sequences without work have n = 0
            seq0 += (unsigned long long)s.n * units;
            s = dec4_seq<kKeys>(p, ++b);
        }
        // ---- the piece: tiles [t0, t1) of unit u of sequence b
        const unsigned long long in_seq = at - seq0;
        const int u = kCluster ? (int)(blockIdx.x / cg::this_cluster().num_blocks()) - b * units : (int)(in_seq / (unsigned)s.n);
        const int t0 = (int)(in_seq - (unsigned long long)u * s.n);
        const int t1 = (int)min((unsigned long long)s.n, t0 + (end - at));
        at += t1 - t0;
        const int h = u / p.n_rc, rc = u - h * p.n_rc;
        const int rbase = rc * C::kRows;
        const int nrows = min(C::kRows, p.G * p.Tq - rbase);
        const size_t row0 = ((size_t)b * p.Hq + (size_t)h * p.G) * p.Tq + rbase;
        const int key_base = (s.first + t0) * kKeys;
        const int n_tiles = t1 - t0;
        const uint8_t* k_head = p.k + h * p.k_sh;
        const uint8_t* v_head = p.v + h * p.v_sh;

        // The next tile to fetch: this lane's box starts at key next_key, row next_row of pool page
        // next_page (-1: outside the pool, -2: no box), which is looked up one tile ahead of its copy.
        int next_key = key_base + lane * box;
        int ord = next_key / p.page_size, next_row = next_key - ord * p.page_size;
        const int* table = p.table + (size_t)b * p.max_pages;
        const auto look_up = [&]() {
            if (lane >= boxes || next_key >= s.len) return -2;
            const int pg = __ldg(table + ord);
            return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
        };
        int next_page = look_up();
        // Copy the next tile into ring stage st. Boxes past the sequence are left out (their keys
        // are masked); a page number outside the pool reads as rows of zeros.
        const auto fetch = [&](int st) {
            const unsigned oks = __ballot_sync(0xffffffffu, next_page >= 0);
            const uint32_t bar = bars + 8 * st;
            const int dst = st * C::kStage + lane * box * C::kRow;
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(oks) * 2 * box * C::kRow);
            __syncwarp();
            if (next_page >= 0) {
                const long long row = (long long)next_row * C::kRow;
                bulk_load(ring_addr + dst, k_head + next_page * p.k_sb + row, box * C::kRow, bar);
                bulk_load(ring_addr + dst + C::kTile, v_head + next_page * p.v_sb + row, box * C::kRow, bar);
            }
            if (oks != all_boxes) {
                if (next_page == -1) {
                    uint32_t* z = reinterpret_cast<uint32_t*>(ring + dst);
                    for (int e = 0; e < box * RW; ++e) z[e] = z[C::kTile / 4 + e] = 0u;
                    fence_proxy_async_smem();  // before a later copy into these bytes
                }
                __syncwarp();
            }
            next_key += kKeys;
            ord += page_step;
            next_row += row_step;
            if (next_row >= p.page_size) {
                next_row -= p.page_size;
                ++ord;
            }
            next_page = look_up();
        };
        for (int i = 0, st = stage; i < kStages && i < n_tiles; ++i) {
            fetch(st);
            st = st + 1 == kStages ? 0 : st + 1;
        }

        // ---- Q fragments: lane (g, t) holds words t + 4i of row g's elements, as pairs (e, e + 4), the
        // odd ones divided by their codes' 16. Each row is taken times the power of two that brings
        // its largest element to [2^14, 2^15): its fp16 form is then exact (fp16 has three bits more)
        // down to 2^-27 of the largest, and off by at most 2^-35 of it below. A row with an infinity
        // or a NaN keeps it.
        uint4 qf[NT == 1 ? kKI : 1];
        uint4* q_frags = reinterpret_cast<uint4*>(ring + kStages * C::kStage);
        // of the rows 2t, 2t + 1 of each tile: the sum, in the products' units, and the factor from
        // these to log2 units
        float sumq[NT][2], unit[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[kKI][8], top = 0.f, sum = 0.f;
            const bool row_ok = 8 * nt + g < nrows;
#pragma unroll
            for (int i = 0; i < kKI; ++i) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (row_ok) x = *reinterpret_cast<const uint4*>(p.q + (row0 + 8 * nt + g) * D + 8 * (t + 4 * i));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[i][2 * e] = __uint_as_float(w[e] << 16);
                    f[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[i][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = dec4_exponent(top);
            const float up = dec4_up<14>(ex);
#pragma unroll
            for (int i = 0; i < kKI; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[i][e] *= up;
                    sum += f[i][e];
                }
                const uint4 v = make_uint4(dec4_halves(f[i][0], f[i][4]), dec4_halves(f[i][1] * 0.0625f, f[i][5] * 0.0625f),
                                           dec4_halves(f[i][2], f[i][6]), dec4_halves(f[i][3] * 0.0625f, f[i][7] * 0.0625f));
                if constexpr (NT == 1)
                    qf[i] = v;
                else
                    q_frags[(i * NT + nt) * 32 + lane] = v;
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sumq[nt][x] = __shfl_sync(0xffffffffu, sum, 8 * t + 4 * x) * 0x1p-24f;
                unit[nt][x] = __shfl_sync(0xffffffffu, dec4_down<14>(ex), 8 * t + 4 * x) * p.scale_log2;
            }
        }
        if constexpr (NT > 1) __syncwarp();

        float less_m[NT][2], l[NT][2], beta[NT][2];
        float oacc[kMT][NT][4], eights[NT][4];
        int step_ex = dec4_exponent(0.f);  // of the largest step yet
        float up_step = dec4_up<kD4StepTo>(step_ex), step_limit = dec4_pow2(step_ex + 1);  // w's factor; the next exponent
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            less_m[nt][0] = less_m[nt][1] = -kD4Lowest;
            l[nt][0] = l[nt][1] = beta[nt][0] = beta[nt][1] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                eights[nt][e] = 0.f;
#pragma unroll
                for (int i = 0; i < kMT; ++i) oacc[i][nt][e] = 0.f;
            }
        }
        const int pos_min = s.len - p.Tq;                                          // position of row 0
        const int lo_min = p.window > 0 ? s.len - min(p.window + p.Tq - 1, s.len) : 0;  // first key of the first row
        const int lo_max = p.window > 0 ? s.len - min(p.window, s.len) : -1;  // first key of the last row

        for (int it = 0; it < n_tiles; ++it) {
            const bool ready = mbar_wait_bounded(bars + 8 * stage, phase, abort_flag, p.err, p.timeout_ns);
            if (!__all_sync(0xffffffffu, ready)) {
                // let the copies that are under way land, oldest first
                for (int i = it; i < n_tiles && i < it + kStages; ++i) {
                    mbar_wait_drain(bars + 8 * stage, phase, p.timeout_ns);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if constexpr (kCluster) break;  // the others wait in the merge
                return;                         // no other warp waits for this one
            }
            const uint32_t* K = reinterpret_cast<const uint32_t*>(ring + stage * C::kStage);
            const uint32_t* V = K + C::kTile / 4;
            const int key0 = key_base + it * kKeys;
            // ---- S^T = K Q^T: of each group of 32 keys, accumulator rows g, g + 8 of m16 tile mt are
            // keys 4g + 2mt, 4g + 2mt + 1
            float sacc[U][2][NT][4];
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sacc[j][mt][nt][e] = 0.f;
            const uint32_t* kr = K + 4 * g * RW + t;
#pragma unroll
            for (int i = 0; i < kKI; ++i) {
                uint4 f[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (NT == 1)
                        f[nt] = qf[i];
                    else
                        f[nt] = q_frags[(i * NT + nt) * 32 + lane];
                }
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t* w = kr + (32 * j + 2 * mt) * RW + 4 * i;
                        uint32_t a0[4], a1[4];
                        dec4_codes(w[0], a0);
                        dec4_codes(w[RW], a1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(sacc[j][mt][nt], a0[0], a1[0], a0[1], a1[1], f[nt].x, f[nt].y);
                            mma_f16_16816(sacc[j][mt][nt], a0[2], a1[2], a0[3], a1[3], f[nt].z, f[nt].w);
                        }
                    }
            }
            // ---- scores, in units of the row; score(j, c, nt, x) is of key 32j + 4g + c, row 8nt + 2t + x
            const auto score = [&](int j, int c, int nt, int x) -> float& { return sacc[j][c >> 1][nt][(c & 1) * 2 + x]; };
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t head = K[(32 * j + 4 * g + c) * RW + D / 8];
                    const float step = dec4_step(head), least = dec4_least(head);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float steps[2] = {step, step}, leasts[2] = {least, least};
                        float sc[2] = {score(j, c, nt, 0), score(j, c, nt, 1)}, part[2];
                        dec4_mul2(part, leasts, sumq[nt]);
                        dec4_fma2(sc, sc, steps, part);
                        score(j, c, nt, 0) = sc[0], score(j, c, nt, 1) = sc[1];
                    }
                }
            const bool masked = key0 + kKeys > pos_min + 1 || key0 < lo_max;
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // keys this row sees, counted from 4g of the tile
                        const int hi = pos_min + (rbase + 8 * nt + 2 * t + x) % p.Tq - key0 - 4 * g;
                        const int lo = p.window > 0 ? hi - p.window + 1 : -0x40000000;
#pragma unroll
                        for (int j = 0; j < U; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (32 * j + c > hi || 32 * j + c < lo) score(j, c, nt, x) = -INFINITY;
                    }
            }
            // steps and middles of this lane's value rows; of a row that no query sees they may be anything
            float vstep[U][4], vmid[U][4], top = 0.f;
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t head = V[(32 * j + 4 * g + c) * RW + D / 8];
                    if (masked) {
                        const int key = key0 + 32 * j + 4 * g + c;
                        if (key >= s.len || key < lo_min) head = 0u;
                    }
                    vstep[j][c] = dec4_step(head);
                    vmid[j][c] = fmaf(8.f, vstep[j][c], dec4_least(head));
                    top = fmaxf(top, fabsf(vstep[j][c]));
                }
            bool raise = top >= step_limit;
            float mx[NT][2];  // of this lane's keys
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mx[nt][x] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < U; ++j)
#pragma unroll
                        for (int c = 0; c < 4; c += 2) mx[nt][x] = max3f(mx[nt][x], score(j, c, nt, x), score(j, c + 1, nt, x));
                    raise |= fmaf(mx[nt][x], unit[nt][x], less_m[nt][x]) > kD4Slack;
                }
            if (__any_sync(0xffffffffu, raise)) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                step_ex = max(step_ex, dec4_exponent(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16))));
                const float down = dec4_up<kD4StepTo>(step_ex) / up_step;  // a power of two, or 0 past fp32's range
                up_step = dec4_up<kD4StepTo>(step_ex);
                step_limit = step_ex < 240 ? dec4_pow2(step_ex + 1) : INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[nt][x] = fmaxf(mx[nt][x], __shfl_xor_sync(0xffffffffu, mx[nt][x], d));
                        const float m_new = fmaxf(mx[nt][x] * unit[nt][x], -less_m[nt][x]);
                        const float alpha = ex2_approx(-less_m[nt][x] - m_new);
                        less_m[nt][x] = -m_new;
                        l[nt][x] *= alpha;
                        beta[nt][x] *= alpha;
                        const float both = alpha * down;
                        eights[nt][x] *= both;  // its rows are alike: only the first is used
#pragma unroll
                        for (int i = 0; i < kMT; ++i) {
                            oacc[i][nt][x] *= both;
                            oacc[i][nt][x + 2] *= both;
                        }
                    }
            }
            uint32_t pb[U][NT][4];  // B operand: keys 8t + c and 8t + 4 + c of query row g
            const auto weigh = [&](auto masked_keys) {
                constexpr bool kMasked = decltype(masked_keys)::value;
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float sc[2] = {score(j, c, nt, 0), score(j, c, nt, 1)};
                            float e[2], w[2];
                            dec4_fma2(e, sc, unit[nt], less_m[nt]);
                            e[0] = ex2_approx(e[0]);
                            e[1] = ex2_approx(e[1]);
                            dec4_add2(l[nt], e);
                            const float vs = vstep[j][c] * up_step, vss[2] = {vs, vs}, mids[2] = {vmid[j][c], vmid[j][c]};
                            if constexpr (kMasked) {  // such a key's step may be NaN
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    w[x] = sc[x] == -INFINITY ? 0.f : e[x] * vs;
                                    if (sc[x] != -INFINITY) beta[nt][x] = fmaf(e[x], vmid[j][c], beta[nt][x]);
                                }
                            } else {
                                dec4_mul2(w, e, vss);
                                dec4_fma2(beta[nt], e, mids, beta[nt]);
                            }
                            pb[j][nt][c] = movmatrix_trans(dec4_halves(w[0], w[1]));
                        }
                    }
            };
            if (masked)
                weigh(std::true_type{});
            else
                weigh(std::false_type{});
            // ---- O^T += V^T P^T
            const uint32_t* vr = V + 4 * g * RW + t;
#pragma unroll
            for (int ks = 0; ks < 2 * U; ++ks) {  // 16 keys: sets c0, c0 + 1 of group ks / 2
                const int c0 = ks % 2 * 2;
                const auto product = [&](float (&acc)[NT][4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(acc[nt], a0, a1, a2, a3, pb[ks / 2][nt][c0], pb[ks / 2][nt][c0 + 1]);
                };
                product(eights, 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u);
#pragma unroll
                for (int i = 0; i < kVI; ++i) {
                    // transposed, a word's halves (four codes each) of keys 4g + c become those of keys
                    // 8t + c and 8t + 4 + c; rows g, g + 8 of tile 4i + e: d = 64i + 4g + e, 64i + 32 + 4g + e
                    uint32_t v[2][2][4];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            dec4_codes(movmatrix_trans(vr[(32 * (ks / 2) + c0 + c) * RW + 8 * i + 4 * r]), v[c][r]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) product(oacc[4 * i + e], v[0][0][e], v[0][1][e], v[1][0][e], v[1][1][e]);
                }
            }
            __syncwarp();  // every lane has read the stage
            if (it + kStages < n_tiles) fetch(stage);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if constexpr (NT > 1) __syncwarp();  // every lane has read the Q fragments

        if constexpr (kCluster) {
            // ---- merge: the warp's state through its ring, the CTA's through its own place
            const float down = dec4_down<kD4StepTo>(step_ex);
            const auto state = [&](uint8_t* base) { return reinterpret_cast<float*>(base); };  // m, l of each row, then O
            float* mine = state(ring);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
                        beta[nt][x] += __shfl_xor_sync(0xffffffffu, beta[nt][x], d);
                    }
                    const int n = 8 * nt + 2 * t + x;
                    if (g == 0) mine[n] = -less_m[nt][x], mine[C::kRows + n] = l[nt][x];
#pragma unroll
                    for (int i = 0; i < kMT; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float o = oacc[i][nt][2 * r + x] * (i % 2 ? 0.0625f : 1.f);  // odd codes count 16 times
                            mine[2 * C::kRows + n * D + 64 * (i / 4) + 32 * r + 4 * g + i % 4] =
                                fmaf(o - eights[nt][x], down, beta[nt][x]);
                        }
                }
            __syncthreads();
            cg::cluster_group cluster = cg::this_cluster();
            float* ours = state(dec4_smem + C::kMergeOff);
            // element (row, d) of the sum of `n` states at `at(i)`
            const auto merged = [&](int n, auto at, int row, int d, float& top, float& sum) {
                top = -INFINITY;
                for (int i = 0; i < n; ++i) top = fmaxf(top, at(i)[row]);
                const float mu = top == -INFINITY ? 0.f : top;
                float acc = 0.f;
                sum = 0.f;
#pragma unroll 8
                for (int i = 0; i < n; ++i) {
                    const float f = ex2_approx(at(i)[row] - mu);
                    sum += at(i)[C::kRows + row] * f;
                    acc += at(i)[2 * C::kRows + row * D + d] * f;
                }
                return acc;
            };
            for (int idx = threadIdx.x; idx < nrows * D; idx += C::kThreads) {
                const int row = idx / D, d = idx % D;
                float top, sum;
                const float acc = merged(kWarps, [&](int i) { return state(dec4_smem + i * C::kWarpBytes); }, row, d, top, sum);
                ours[2 * C::kRows + idx] = acc;
                if (d == 0) ours[row] = top, ours[C::kRows + row] = sum;
            }
            cluster.sync();
            for (int idx = cluster.block_rank() * C::kThreads + threadIdx.x; idx < nrows * D; idx += cluster.num_blocks() * C::kThreads) {
                const int row = idx / D, d = idx % D;
                float top, sum;
                const float acc = merged(cluster.num_blocks(), [&](int i) { return cluster.map_shared_rank(ours, i); }, row, d, top, sum);
                p.o[(row0 + row) * D + d] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);  // a row that sees no key: 0
            }
            cluster.sync();  // the states are read
            return;
        }
        // ---- the piece's rows: final if it is a whole unit, else partial. A row that sees no key of
        // the piece: 0, and weight 0 in the merge (NaN stays NaN).
        const bool whole = t0 == 0 && t1 == s.n;
        const size_t part = (2 * (size_t)run + (t0 > 0 ? 0 : 1)) * C::kRows;
        if (lane == 0 && p.ends != nullptr) {
            int2* e = p.ends + (size_t)b * units + u;
            if (t0 == 0) e->x = (int)run;
            if (t1 == s.n) e->y = (int)run;
        }
        const float down = dec4_down<kD4StepTo>(step_ex);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
                    beta[nt][x] += __shfl_xor_sync(0xffffffffu, beta[nt][x], d);
                }
                const int n = 8 * nt + 2 * t + x;
                if (n >= nrows) continue;
                const float inv = l[nt][x] == 0.f ? 0.f : 1.f / l[nt][x];
                if (!whole && g == 0)
                    p.part_lse[part + n] = l[nt][x] == 0.f ? -INFINITY : __log2f(l[nt][x]) - less_m[nt][x];
#pragma unroll
                for (int i = 0; i < kMT / 4; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {  // four elements from d = 64i + 32r + 4g
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float o = oacc[4 * i + e][nt][2 * r + x] * (e % 2 ? 0.0625f : 1.f);  // odd codes count 16 times
                            v[e] = fmaf(o - eights[nt][x], down, beta[nt][x]) * inv;
                        }
                        const int d = 64 * i + 32 * r + 4 * g;
                        if (whole)
                            *reinterpret_cast<uint2*>(p.o + (row0 + n) * D + d) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                        else
                            *reinterpret_cast<float4*>(p.part + (part + n) * D + d) = make_float4(v[0], v[1], v[2], v[3]);
                    }
            }
    } while (at < end);
}

// Merge the pieces of the units that were cut between warps, in run order: one block a row, of
// sequence blockIdx.x. Which runs they are the first kernel has left; a warp of it whose wait ran
// out has not, so `ends` may be anything the workspace held, and is only followed inside it.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kD4MergeWarps) gqa_decode_kv4_merge_kernel(const Dec4Params p) {
    constexpr int kRows = 8 * NT;
    constexpr int E = D / 32;
    __shared__ float accs[kD4MergeWarps][D];
    __shared__ float weights[kD4MergeWarps];
    const int rows = p.G * p.Tq;  // of a KV head
    const int h = (int)blockIdx.y / rows, in_group = (int)blockIdx.y - h * rows;
    const int rc = in_group / kRows;
    const int2 ends = p.ends[((size_t)blockIdx.x * p.Hkv + h) * p.n_rc + rc];
    const int len = __ldg(p.seqlens + blockIdx.x);
    if (len < 0 || len > p.capacity || ends.x == ends.y) return;  // no output, or whole
    if (ends.x < 0 || ends.x > ends.y || ends.y >= p.runs) return;  // a wait ran out, which is reported
    const size_t row = (size_t)blockIdx.x * gridDim.y + blockIdx.y;
    const int c0 = ends.x, c1 = ends.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first piece starts the unit (slot 1 of its run), the others do not (slot 0)
    const auto at = [&](int c) { return (2 * (size_t)c + (c == c0 ? 1 : 0)) * kRows + (in_group - rc * kRows); };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.part_lse[at(c)]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if (M == -INFINITY) M = 0.f;
    float sum = 0.f, acc[E] = {};
#pragma unroll 8
    for (int c = c0 + warp; c <= c1; c += kD4MergeWarps) {
        const float f = ex2_approx(p.part_lse[at(c)] - M);
        const float* src = p.part + at(c) * D + lane * E;
        float v[E];
        if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[0] = x.x, v[1] = x.y;
        }
        sum += f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) accs[warp][lane * E + e] = acc[e];
    if (lane == 0) weights[warp] = sum;
    __syncthreads();
    for (int d = 2 * threadIdx.x; d < D; d += 64 * kD4MergeWarps) {
        float total_weight = 0.f, v[2] = {};
#pragma unroll
        for (int w = 0; w < kD4MergeWarps; ++w) {
            total_weight += weights[w];
            v[0] += accs[w][d];
            v[1] += accs[w][d + 1];
        }
        const float inv = total_weight == 0.f ? 0.f : 1.f / total_weight;
        *reinterpret_cast<uint32_t*>(p.o + row * D + d) = pack_bf16x2(v[0] * inv, v[1] * inv);
    }
}

}  // namespace gqa

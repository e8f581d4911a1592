// The operators around a paged key/value cache (declared in include/gqa.h): the plan of a step,
// the norm and rotation of queries and keys with its gradients and its cache-writing form, the
// rows of a cache held in 4 bits, and decode over that cache. Argument checks and launches; the
// kernels are in paged_plan.cuh, rope_sm100.cuh, kv4_rows_sm100.cuh and decode_kv4_sm100.cuh.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/gqa.h"
#include "../../include/gqa_testing.h"
#include "decode_kv4_sm100.cuh"
#include "gqa_internal.h"
#include "kv4_rows_sm100.cuh"
#include "paged_plan.cuh"
#include "rope_sm100.cuh"

namespace {

using bf16 = __nv_bfloat16;

bool aligned(const void* p, uintptr_t n) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned_or_null(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Pages the attention calls read, and rows that fit the 32-bit slot numbers.
gqa_status check_pages(int page_size, int num_pages) {
    const bool ok = page_size >= 16 && page_size % 16 == 0 &&
                    (page_size % gqa::kTileKeys == 0 || gqa::kTileKeys % page_size == 0);
    if (!ok || num_pages <= 0) return GQA_ERR_INVALID_ARGUMENT;
    return (long long)page_size * num_pages <= 0x7fffffffLL ? GQA_OK : GQA_ERR_UNSUPPORTED;
}

// Element strides of rows that are read or written 8 or 16 bytes at a time. A stride along an
// axis of extent 1 is not used.
gqa_status check_rows(const gqa_layout* l, int B, int H, int T, int D, long long* sb, long long* sh, long long* st) {
    if (l == nullptr) return GQA_ERR_INVALID_ARGUMENT;
    *sb = B > 1 ? l->sb : 0;
    *sh = H > 1 ? l->sh : 0;
    *st = T > 1 ? l->st : 0;
    if ((B > 1 && *sb <= 0) || (H > 1 && *sh <= 0) || (T > 1 && *st < D)) return GQA_ERR_INVALID_ARGUMENT;
    if ((*sb | *sh | *st) & 7) return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

gqa_status check_heads(int Hq, int Hkv, int D) {
    if (Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARGUMENT;
    return D == 64 || D == 128 ? GQA_OK : GQA_ERR_UNSUPPORTED;
}

gqa_status launched(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        sms = 148;
    return sms;
}

// ---------------------------------------------------------------- plan
// Threads that a step keeps busy once: four tokens each, or one page that it may take or give back.
long long paged_work(const gqa::PagedPlanParams& p) {
    return ((long long)p.max_tokens + 3) / 4 + p.max_tokens / p.page_size + p.S;
}
// Blocks of 256 threads for few requests, whose scans then cost less, while at most two rounds of
// them do the work; else of 1024. us with 256 / 1024: 64 requests with 1024 tokens 3.6 / 4.5, 262 144
// tokens 5.1 / 5.5, 524 288 tokens 7.8 / 5.5, in place 16 384 tokens 5.5 / 6.0, 32 768 tokens 8.1 / 6.1;
// 256 requests with 65 536 tokens 4.2 / 5.5; 768 requests with 768 tokens 7.5 / 7.0.
bool paged_few(const gqa::PagedPlanParams& p, int ctas) {
    return p.S <= gqa::kPagedFewSeqs && paged_work(p) <= 2LL * gqa::kPagedFewThreads * ctas;
}

template <int kThreads, bool kCluster>
gqa_status paged_plan(const gqa::PagedPlanParams& p, cudaStream_t stream) {
    const auto kernel = gqa::gqa_paged_plan_kernel<kThreads, kCluster>;
    const size_t smem = gqa::paged_plan_smem(p.S);
    if (smem > 48 * 1024 - 1024 &&  // beside the kernel's static shared memory
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)gqa::paged_plan_smem(gqa::kPagedMaxSeqs)) != cudaSuccess)
        return GQA_ERR_CUDA;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    if (kCluster)
        cfg.gridDim.x = attr.val.clusterDim.x = gqa::kPagedCluster;
    else
        cfg.gridDim.x = (unsigned)std::min<long long>((paged_work(p) + kThreads - 1) / kThreads, sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = kCluster ? 1 : 0;
    return launched(cudaLaunchKernelEx(&cfg, kernel, p));
}

// ---------------------------------------------------------------- norm and rotation
gqa_status rope_params(gqa::RopeParams& p, const gqa_rope* r, int B, int T, int Hq, int Hkv, int D) {
    gqa_status st = check_heads(Hq, Hkv, D);
    if (st != GQA_OK) return st;
    if (r == nullptr || B <= 0 || T <= 0) return GQA_ERR_INVALID_ARGUMENT;
    if ((long long)B * T > 0x7fffffffLL) return GQA_ERR_UNSUPPORTED;
    p.x[0].weight = r->q_weight;
    p.x[1].weight = r->k_weight;
    p.weight_fp32 = r->weight_fp32 != 0;
    if (!aligned_or_null(r->q_weight, 16) || !aligned_or_null(r->k_weight, 16)) return GQA_ERR_INVALID_ARGUMENT;
    if (!(r->eps >= 0.f) || std::isinf(r->eps)) return GQA_ERR_INVALID_ARGUMENT;
    p.eps = r->eps;
    if ((r->cos == nullptr) != (r->sin == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
    if (r->cos != nullptr) {
        if (!aligned(r->cos, 16) || !aligned(r->sin, 16) || !aligned_or_null(r->positions, 4)) return GQA_ERR_INVALID_ARGUMENT;
        if (r->rot < 8 || r->rot > D || r->rot % 8 != 0 || r->n_positions <= 0) return GQA_ERR_INVALID_ARGUMENT;
        if (r->positions == nullptr && T > r->n_positions) return GQA_ERR_INVALID_ARGUMENT;
        if (r->positions != nullptr && B > 1 && r->positions_sb < 0) return GQA_ERR_INVALID_ARGUMENT;
        p.cos = r->cos;
        p.sin = r->sin;
        p.rot = r->rot;
        p.n_positions = r->n_positions;
        p.positions = r->positions;
        p.pos_sb = B > 1 ? r->positions_sb : 0;
    } else {
        p.rot = D;  // lanes take the halves of the row; nothing turns
    }
    p.B = B;
    p.T = T;
    p.x[0].H = Hq;
    p.x[1].H = Hkv;
    return GQA_OK;
}

// Heads of a token that one team of D/8 lanes takes in turn: its loads of the angles and weights
// serve that many rows, so a large launch takes `many`; a small one takes the four it has in
// flight at a time, to spread over the SMs. The sides meet near 512 lanes an SM. Forward, us with 4 / 16:
// 32 + 8 heads of 128, 256 tokens 3.2 / 5.5, 1536 tokens 6.9 / 7.1, 2048 tokens 8.8 / 8.2, 6144 tokens 23.9 / 20.1;
// 6 + 2 heads of 64, 4096 tokens 3.9 / 4.0, 12 288 tokens 7.2 / 6.9. Backward, with 4 / 8: 32 + 8 heads of
// 128, 256 tokens 6.6 / 7.0, 1024 tokens 11.4 / 11.5, 3584 tokens 25.6 / 22.7; 32 + 1 heads, 1024 tokens 9.7 / 8.9.
int rope_heads_per_team(long long tokens, int heads, int D, int many, int sms) {
    const long long lanes = tokens * ((heads + many - 1) / many) * (D / 8);
    return lanes >= (long long)sms * 512 ? many : gqa::kRopeUnroll;
}
// Heads, split into blocks; false if there are more blocks than a grid's y extent.
bool rope_blocks(gqa::RopeParams& p, int heads_per_team) {
    p.heads_per_team = heads_per_team;
    int all = 0;
    for (int i = 0; i < 3; ++i) all += p.blocks[i] = (p.x[i].H + heads_per_team - 1) / heads_per_team;
    return all <= 65535;
}

template <int D>
gqa_status rope_fwd(gqa::RopeParams p, bool interleaved, cudaStream_t stream) {
    int heads = 0;
    for (int i = 0; i < 3; ++i) heads += p.x[i].H;
    if (!rope_blocks(p, rope_heads_per_team((long long)p.B * p.T, heads, D, 16, sm_count()))) return GQA_ERR_UNSUPPORTED;
    if ((p.err = gqa::device_error_ptr()) == nullptr) return GQA_ERR_CUDA;
    constexpr int kPer = gqa::kRopeThreads / (D / 8);
    const dim3 grid((unsigned)(((long long)p.B * p.T + kPer - 1) / kPer), (unsigned)(p.blocks[0] + p.blocks[1] + p.blocks[2]));
    if (interleaved)
        gqa::gqa_rope_fwd_kernel<D, true><<<grid, gqa::kRopeThreads, 0, stream>>>(p);
    else
        gqa::gqa_rope_fwd_kernel<D, false><<<grid, gqa::kRopeThreads, 0, stream>>>(p);
    return launched(cudaGetLastError());
}

// The backward pass's CTAs: as many as run at once (two a SM), or as there is work for, dealt to the
// operands in proportion to their heads in fours. Each leaves one row of weight sums.
struct RopeBwdPlan {
    int heads_per_team, q_ctas, ctas;
};
RopeBwdPlan rope_bwd_plan(int B, int T, int Hq, int Hkv, int D) {
    const int sms = sm_count(), per_cta = gqa::kRopeThreads / (D / 8);
    const long long groups = ((long long)B * T + per_cta - 1) / per_cta;
    RopeBwdPlan r;
    r.heads_per_team = rope_heads_per_team((long long)B * T, Hq + Hkv, D, 8, sms);
    const auto fours = [](int H) { return (H + gqa::kRopeUnroll - 1) / gqa::kRopeUnroll; };  // a lane's steps
    const auto ctas = [&](int H) {
        const long long units = groups * ((H + r.heads_per_team - 1) / r.heads_per_team);
        return (int)std::min<long long>(units, std::max<long long>(1, 2LL * sms * fours(H) / (fours(Hq) + fours(Hkv))));
    };
    r.q_ctas = ctas(Hq);
    r.ctas = r.q_ctas + ctas(Hkv);
    return r;
}

template <int D>
gqa_status rope_bwd(gqa::RopeParams p, const RopeBwdPlan& r, bool interleaved, float* dq_weight, float* dk_weight,
                    cudaStream_t stream) {
    if (!rope_blocks(p, r.heads_per_team)) return GQA_ERR_UNSUPPORTED;
    if ((long long)p.B * p.T * p.blocks[0] > 0x7fffffffLL) return GQA_ERR_UNSUPPORTED;  // units in 32 bits
    if ((p.err = gqa::device_error_ptr()) == nullptr) return GQA_ERR_CUDA;
    p.q_ctas = r.q_ctas;
    const unsigned grid = (unsigned)r.ctas;
    if (interleaved)
        gqa::gqa_rope_bwd_kernel<D, true><<<grid, gqa::kRopeThreads, 0, stream>>>(p);
    else
        gqa::gqa_rope_bwd_kernel<D, false><<<grid, gqa::kRopeThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (dq_weight == nullptr && dk_weight == nullptr)) return launched(e);
    gqa::gqa_rope_dw_kernel<D><<<dim3(2, D / gqa::kRopeDwColumns), 1024, 0, stream>>>(p.partial, r.q_ctas, r.ctas, dq_weight,
                                                                     dk_weight);
    return launched(cudaGetLastError());
}

// ---------------------------------------------------------------- 4-bit rows
gqa_status check_kv4_pool(const void* pool, const gqa_kv4_layout* l, int num_pages, int Hkv, int page_size, int D,
                          long long* sb, long long* sh) {
    if (l == nullptr || !aligned(pool, 16)) return GQA_ERR_INVALID_ARGUMENT;
    *sb = num_pages > 1 ? l->sb : 0;
    *sh = Hkv > 1 ? l->sh : 0;
    const long long rows = (long long)page_size * (D / 2 + 4);
    if ((num_pages > 1 && *sb < rows) || (Hkv > 1 && *sh < rows)) return GQA_ERR_INVALID_ARGUMENT;
    return ((*sb | *sh) & 15) ? GQA_ERR_INVALID_ARGUMENT : GQA_OK;
}

gqa_status kv4_rows(bool append, const void* k, const void* v, const void* k_pool, const void* v_pool, const int* slots,
                    int N, int Hkv, int D, int page_size, int num_pages, const gqa_layout* k_layout,
                    const gqa_layout* v_layout, const gqa_kv4_layout* k_pool_layout, const gqa_kv4_layout* v_pool_layout,
                    void* stream) {
    gqa_status st = check_heads(Hkv, Hkv, D);
    if (st != GQA_OK) return st;
    if (N < 0) return GQA_ERR_INVALID_ARGUMENT;
    if ((st = check_pages(page_size, num_pages)) != GQA_OK) return st;
    gqa::Kv4RowsParams p{};
    if ((st = check_kv4_pool(k_pool, k_pool_layout, num_pages, Hkv, page_size, D, &p.x[0].pool_sb, &p.x[0].pool_sh)) != GQA_OK)
        return st;
    if ((st = check_kv4_pool(v_pool, v_pool_layout, num_pages, Hkv, page_size, D, &p.x[1].pool_sb, &p.x[1].pool_sh)) != GQA_OK)
        return st;
    if (N == 0) return GQA_OK;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return GQA_ERR_INVALID_ARGUMENT;
    long long unused;
    if ((st = check_rows(k_layout, 1, Hkv, N, D, &unused, &p.x[0].sh, &p.x[0].st)) != GQA_OK) return st;
    if ((st = check_rows(v_layout, 1, Hkv, N, D, &unused, &p.x[1].sh, &p.x[1].st)) != GQA_OK) return st;
    p.x[0].rows = static_cast<bf16*>(const_cast<void*>(k));
    p.x[1].rows = static_cast<bf16*>(const_cast<void*>(v));
    p.x[0].pool = static_cast<uint8_t*>(const_cast<void*>(k_pool));
    p.x[1].pool = static_cast<uint8_t*>(const_cast<void*>(v_pool));
    p.slots = slots;
    p.N = N;
    p.H = Hkv;
    p.page_size = page_size;
    p.num_pages = num_pages;
    if ((p.err = gqa::device_error_ptr()) == nullptr) return GQA_ERR_CUDA;
    const int per = gqa::kKv4Threads / (D / 8);
    // Many rows: eight heads a team, to spread its set-up; few: the four it has in flight at a time. us with 4 / 8,
    // written and read, 8 heads of 128: 256 tokens 4.2 / 5.6, 4096 tokens 10.2 / 10.3, 6144 tokens 14.0 / 13.7, 16 384
    // tokens 33.0 / 30.1; 8 heads of 64, 10 240 tokens 12.2 / 12.0.
    p.heads_per_team = 2LL * N * ((Hkv + 7) / 8) * (D / 8) >= (long long)sm_count() * 1024 ? 8 : gqa::kKv4Unroll;
    p.blocks = (Hkv + p.heads_per_team - 1) / p.heads_per_team;
    if (2LL * p.blocks > 65535) return GQA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((N + (long long)per - 1) / per), (unsigned)(2 * p.blocks));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (append) {
        if (D == 128)
            gqa::gqa_kv4_append_kernel<128><<<grid, gqa::kKv4Threads, 0, s>>>(p);
        else
            gqa::gqa_kv4_append_kernel<64><<<grid, gqa::kKv4Threads, 0, s>>>(p);
    } else {
        if (D == 128)
            gqa::gqa_kv4_gather_kernel<128><<<grid, gqa::kKv4Threads, 0, s>>>(p);
        else
            gqa::gqa_kv4_gather_kernel<64><<<grid, gqa::kKv4Threads, 0, s>>>(p);
    }
    return launched(cudaGetLastError());
}

// ---------------------------------------------------------------- decode over 4-bit rows
constexpr int kMaxDecodeRows = 16;           // new queries a sequence
constexpr int kDec4MaxKeys = 1 << 30;        // key numbers plus a tile stay below 2^31

gqa_status check_dec4(int B, int Hq, int Hkv, int Tq, int max_seqlen_k, int D, int window) {
    const gqa_status st = check_heads(Hq, Hkv, D);
    if (st != GQA_OK) return st;
    if (B <= 0 || Tq <= 0 || max_seqlen_k <= 0 || window < 0) return GQA_ERR_INVALID_ARGUMENT;
    if (Tq > kMaxDecodeRows || max_seqlen_k > kDec4MaxKeys) return GQA_ERR_UNSUPPORTED;
    // the merge's grid; tiles of all units in 52 bits, times the warps in 64
    const long long rows = (long long)B * Hq * Tq;
    if ((long long)Hq * Tq > 65535 || rows > 0x7fffffffLL || rows * (max_seqlen_k / 32 + 2) >= 1LL << 52) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

// N tiles of 8 query rows a CTA takes: as few as hold a group's rows, four at most (more would not fit
// the registers). us with one / two / four, 18 x 20000 keys, D = 128: 8 rows 48.9 / 67.2 / -, 16 rows 45.9 / 45.9 / 75.9;
// 64 x 8192 keys of 4 KV heads, D = 64, 16 rows 80.2 / 64.9 / 111. Of 32 rows two passes of two tiles or one of four
// come out either way: 18 x 20000 keys 44.2 / 51.8, with D = 64 39.4 / 34.3; 16 x 4096 keys of 4 KV heads 37.2 / 34.4.
int dec4_nt(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

struct Dec4Plan {
    int nt, n_rc, ctas, warps;  // warps: of a CTA
    int cluster;                // CTAs of a unit's cluster, 0: runs of tiles and a merge
    size_t part, lse, ends, bytes;  // the workspace's parts and size
};
constexpr int kDec4MergeRounds = 4;  // rounds of tiles that take as long as the merge's launch
constexpr int kDec4MostRounds = 8;   // of a cluster: lengths may differ, and only even runs balance that
template <int D, int NT>
Dec4Plan dec4_plan_for(int B, int Hkv, int rows, int Tq, int max_seqlen_k, int window) {
    using C = gqa::Dec4Cfg<D, NT>;
    Dec4Plan r;
    r.nt = NT;
    r.n_rc = (rows + C::kRows - 1) / C::kRows;
    r.warps = C::kWarps;
    // no more CTAs than the longest lengths have tiles
    const long long keys = window > 0 ? std::min<long long>(max_seqlen_k, (long long)window + Tq + C::kKeys) : max_seqlen_k;
    const long long tiles = (long long)B * Hkv * r.n_rc * ((keys + C::kKeys - 1) / C::kKeys);
    r.ctas = (int)std::min<long long>((long long)sm_count() * C::kCtasPerSm, tiles);
    // A cluster a unit, if they all run at once (16 CTAs have to fit a GPC together: half the places)
    // and have little more to do than the even runs, which pay for their merge with a second launch. us with
    // clusters / runs, 8 KV heads of 4 queries, D = 128: 1 x 4099 keys 7.6 / 13.2, 1 x 32768 19.3 / 24.0, 16 x 4096
    // 19.9 / 23.6, 16 x 16384 60.4 / 59.4, 1 x 131072 57.7 / 43.9. Where the rounds are about to tip it the rule takes the runs a
    // little early: one KV head of 32 queries over 32768 keys 31.7 / 34.6.
    const long long units = (long long)B * Hkv * r.n_rc, of_unit = tiles / units;
    const long long places = (long long)sm_count() * C::kCtasPerSm;
    int cluster = 1;
    while (cluster < 16 && cluster * C::kWarps < of_unit && units * 2 * cluster <= (cluster < 8 ? places : places / 2)) cluster *= 2;
    const long long rounds = (of_unit + cluster * C::kWarps - 1) / (cluster * C::kWarps);
    const long long even = (tiles + (long long)r.ctas * r.warps - 1) / ((long long)r.ctas * r.warps);
    r.cluster = units * cluster <= places && rounds <= kDec4MostRounds && rounds <= even + kDec4MergeRounds ? cluster : 0;
    if (r.cluster) r.ctas = (int)(units * cluster);
    const size_t slots = !r.cluster ? (size_t)2 * r.ctas * r.warps * C::kRows : 0;
    r.part = 0;
    r.lse = gqa::round256(slots * D * sizeof(float));
    r.ends = r.lse + gqa::round256(slots * sizeof(float));
    r.bytes = !r.cluster ? r.ends + (size_t)B * Hkv * r.n_rc * sizeof(int2) : 0;
    return r;
}
Dec4Plan dec4_plan(int B, int Hq, int Hkv, int Tq, int max_seqlen_k, int D, int window) {
    const int rows = Hq / Hkv * Tq, nt = dec4_nt(rows);
    if (D == 128)
        return nt == 1   ? dec4_plan_for<128, 1>(B, Hkv, rows, Tq, max_seqlen_k, window)
               : nt == 2 ? dec4_plan_for<128, 2>(B, Hkv, rows, Tq, max_seqlen_k, window)
                         : dec4_plan_for<128, 4>(B, Hkv, rows, Tq, max_seqlen_k, window);
    return nt == 1   ? dec4_plan_for<64, 1>(B, Hkv, rows, Tq, max_seqlen_k, window)
           : nt == 2 ? dec4_plan_for<64, 2>(B, Hkv, rows, Tq, max_seqlen_k, window)
                     : dec4_plan_for<64, 4>(B, Hkv, rows, Tq, max_seqlen_k, window);
}

// The workspace of a plan that has one.
gqa_status dec4_workspace(gqa::Dec4Params& p, const Dec4Plan& r, void* workspace, size_t workspace_bytes) {
    if (r.bytes == 0) return GQA_OK;
    if (!aligned(workspace, 256) || workspace_bytes < r.bytes) return GQA_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    p.part = reinterpret_cast<float*>(ws + r.part);
    p.part_lse = reinterpret_cast<float*>(ws + r.lse);
    p.ends = reinterpret_cast<int2*>(ws + r.ends);
    p.runs = r.ctas * r.warps;
    return GQA_OK;
}

std::atomic<int> g_dec4_largest{16};  // CTAs of a cluster, for tests of the smaller forms

// Clusters above the portable eight CTAs need a GPC with that many SMs free to the process, which a
// partitioned device may not have: 16 or 8, asked once a device. The kernel takes any size. One sequence,
// us with 8 / 16: 4099 keys of 8 KV heads 8.1 / 7.8, 32768 keys 24.3 / 19.4, 16384 keys of 2 heads 15.1 / 10.9.
template <int D, int NT>
int dec4_largest_cluster(cudaLaunchConfig_t cfg) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3(16);
        cfg.attrs = nullptr;
        cfg.numAttrs = 0;
        if (cudaOccupancyMaxPotentialClusterSize(&n, gqa::gqa_decode_kv4_kernel<D, NT, true>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        n = n >= 16 ? 16 : 8;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int D, int NT>
gqa_status launch_dec4_merge(const gqa::Dec4Params& p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.B, (unsigned)(p.Hq * p.Tq));
    gqa::gqa_decode_kv4_merge_kernel<D, NT><<<grid, 32 * gqa::kD4MergeWarps, 0, stream>>>(p);
    return launched(cudaGetLastError());
}

template <int D, int NT>
gqa_status launch_dec4(const gqa::Dec4Params& p, const Dec4Plan& r, cudaStream_t stream) {
    using C = gqa::Dec4Cfg<D, NT>;
    const auto kernel = r.cluster ? gqa::gqa_decode_kv4_kernel<D, NT, true> : gqa::gqa_decode_kv4_kernel<D, NT, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    if (e == cudaSuccess && r.cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return GQA_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)r.ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = r.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    if (r.cluster > 1) {
        int most = g_dec4_largest.load(std::memory_order_relaxed);
        if (r.cluster > 8) most = std::min(most, dec4_largest_cluster<D, NT>(cfg));
        if (r.cluster > most) {
            attr.val.clusterDim.x = most;
            cfg.gridDim = dim3((unsigned)(r.ctas / r.cluster * most));
        }
    }
    cfg.attrs = &attr;
    cfg.numAttrs = r.cluster ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess || r.cluster) return launched(e);
    return launch_dec4_merge<D, NT>(p, stream);
}

// f with D and the N tiles as constants.
template <class F>
gqa_status dec4_dispatch(int D, int nt, F f) {
    const auto of = [&](auto d) {
        return nt == 1   ? f(d, std::integral_constant<int, 1>{})
               : nt == 2 ? f(d, std::integral_constant<int, 2>{})
                         : f(d, std::integral_constant<int, 4>{});
    };
    return D == 128 ? of(std::integral_constant<int, 128>{}) : of(std::integral_constant<int, 64>{});
}

}  // namespace

extern "C" {

gqa_status gqa_paged_plan(const int* seqlens, const int* keep, const int* new_tokens, int* block_table, int* free_list,
                          const int* free_count, int* seqlens_out, int* cu_seqlens, int* positions, int* slots,
                          int* free_count_out, int S, int max_pages, int page_size, int num_pages, int free_capacity,
                          int max_tokens, void* stream) {
    if (S <= 0 || max_pages <= 0 || free_capacity <= 0 || max_tokens <= 0) return GQA_ERR_INVALID_ARGUMENT;
    gqa_status st = check_pages(page_size, num_pages);
    if (st != GQA_OK) return st;
    if (S > gqa::kPagedMaxSeqs || (long long)max_pages * page_size > 0x7fffffffLL) return GQA_ERR_UNSUPPORTED;
    if ((long long)S * max_pages > 0x7fffffffLL) return GQA_ERR_UNSUPPORTED;  // pages of a step are counted in 32 bits
    if (!aligned(seqlens, 4) || !aligned_or_null(keep, 4) || !aligned(new_tokens, 4) || !aligned(block_table, 4) ||
        !aligned(free_list, 4) || !aligned(free_count, 4) || !aligned(seqlens_out, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(positions, 16) || !aligned(slots, 16) || !aligned(free_count_out, 4))
        return GQA_ERR_INVALID_ARGUMENT;
    gqa::PagedPlanParams p{seqlens, keep,      new_tokens, block_table, free_list,  free_count, seqlens_out, cu_seqlens,
                           positions, slots,   free_count_out, S,       max_pages,  page_size,  num_pages,   free_capacity,
                           max_tokens, gqa::device_error_ptr()};
    if (p.err == nullptr) return GQA_ERR_CUDA;
    const bool in_place =
        seqlens_out == seqlens || seqlens_out == keep || seqlens_out == new_tokens || free_count_out == free_count;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (paged_few(p, in_place ? gqa::kPagedCluster : sm_count()))
        return in_place ? paged_plan<gqa::kPagedFewThreads, true>(p, s) : paged_plan<gqa::kPagedFewThreads, false>(p, s);
    return in_place ? paged_plan<1024, true>(p, s) : paged_plan<1024, false>(p, s);
}

gqa_status gqa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int T, int Hq, int Hkv, int D,
                            const gqa_layout* q_layout, const gqa_layout* k_layout, const gqa_layout* q_out_layout,
                            const gqa_layout* k_out_layout, const gqa_rope* rope, void* stream) {
    gqa::RopeParams p{};
    gqa_status st = rope_params(p, rope, B, T, Hq, Hkv, D);
    if (st != GQA_OK) return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16)) return GQA_ERR_INVALID_ARGUMENT;
    gqa::RopeRows &x = p.x[0], &y = p.x[1];
    if ((st = check_rows(q_layout, B, Hq, T, D, &x.in_sb, &x.in_sh, &x.in_st)) != GQA_OK) return st;
    if ((st = check_rows(k_layout, B, Hkv, T, D, &y.in_sb, &y.in_sh, &y.in_st)) != GQA_OK) return st;
    if ((st = check_rows(q_out_layout, B, Hq, T, D, &x.out_sb, &x.out_sh, &x.out_st)) != GQA_OK) return st;
    if ((st = check_rows(k_out_layout, B, Hkv, T, D, &y.out_sb, &y.out_sh, &y.out_st)) != GQA_OK) return st;
    x.in = static_cast<const bf16*>(q);
    y.in = static_cast<const bf16*>(k);
    x.out = static_cast<bf16*>(q_out);
    y.out = static_cast<bf16*>(k_out);
    const bool inter = rope->interleaved != 0;
    return D == 128 ? rope_fwd<128>(p, inter, static_cast<cudaStream_t>(stream))
                    : rope_fwd<64>(p, inter, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out, void* k_pool, void* v_pool,
                                   const int* slots, int N, int Hq, int Hkv, int D, int page_size, int num_pages,
                                   const gqa_layout* q_layout, const gqa_layout* k_layout, const gqa_layout* v_layout,
                                   const gqa_layout* q_out_layout, const gqa_layout* k_pool_layout,
                                   const gqa_layout* v_pool_layout, const gqa_rope* rope, void* stream) {
    if (N < 0) return GQA_ERR_INVALID_ARGUMENT;
    gqa::RopeParams p{};
    gqa_status st = rope_params(p, rope, 1, N > 0 ? N : 1, Hq, Hkv, D);
    if (st != GQA_OK) return st;
    if ((st = check_pages(page_size, num_pages)) != GQA_OK) return st;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return GQA_ERR_INVALID_ARGUMENT;
    gqa::RopeRows &x = p.x[0], &y = p.x[1], &z = p.x[2];
    z.H = Hkv;
    if ((st = check_rows(k_pool_layout, num_pages, Hkv, page_size, D, &y.out_sb, &y.out_sh, &y.out_st)) != GQA_OK) return st;
    if ((st = check_rows(v_pool_layout, num_pages, Hkv, page_size, D, &z.out_sb, &z.out_sh, &z.out_st)) != GQA_OK) return st;
    if (N == 0) return GQA_OK;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(slots, 4))
        return GQA_ERR_INVALID_ARGUMENT;
    if ((st = check_rows(q_layout, 1, Hq, N, D, &x.in_sb, &x.in_sh, &x.in_st)) != GQA_OK) return st;
    if ((st = check_rows(k_layout, 1, Hkv, N, D, &y.in_sb, &y.in_sh, &y.in_st)) != GQA_OK) return st;
    if ((st = check_rows(v_layout, 1, Hkv, N, D, &z.in_sb, &z.in_sh, &z.in_st)) != GQA_OK) return st;
    if ((st = check_rows(q_out_layout, 1, Hq, N, D, &x.out_sb, &x.out_sh, &x.out_st)) != GQA_OK) return st;
    x.in = static_cast<const bf16*>(q);
    y.in = static_cast<const bf16*>(k);
    z.in = static_cast<const bf16*>(v);
    x.out = static_cast<bf16*>(q_out);
    y.out = static_cast<bf16*>(k_pool);
    z.out = static_cast<bf16*>(v_pool);
    p.slots = slots;
    p.page_size = page_size;
    p.num_pages = num_pages;
    const bool inter = rope->interleaved != 0;
    return D == 128 ? rope_fwd<128>(p, inter, static_cast<cudaStream_t>(stream))
                    : rope_fwd<64>(p, inter, static_cast<cudaStream_t>(stream));
}

size_t gqa_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    if (check_heads(Hq, Hkv, D) != GQA_OK || B <= 0 || T <= 0) return 0;
    const RopeBwdPlan r = rope_bwd_plan(B, T, Hq, Hkv, D);
    return gqa::round256((size_t)r.ctas * D * sizeof(float));
}

gqa_status gqa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, void* dq, void* dk,
                                float* dq_weight, float* dk_weight, int B, int T, int Hq, int Hkv, int D,
                                const gqa_layout* dq_out_layout, const gqa_layout* dk_out_layout,
                                const gqa_layout* q_layout, const gqa_layout* k_layout, const gqa_layout* dq_layout,
                                const gqa_layout* dk_layout, const gqa_rope* rope, void* workspace, size_t workspace_bytes,
                                void* stream) {
    gqa::RopeParams p{};
    gqa_status st = rope_params(p, rope, B, T, Hq, Hkv, D);
    if (st != GQA_OK) return st;
    if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq, 16) || !aligned(dk, 16))
        return GQA_ERR_INVALID_ARGUMENT;
    gqa::RopeRows &x = p.x[0], &y = p.x[1];
    // without a weight the inputs are not read, and there is no weight gradient
    if ((x.weight != nullptr) != (dq_weight != nullptr) || (y.weight != nullptr) != (dk_weight != nullptr))
        return GQA_ERR_INVALID_ARGUMENT;
    if (!aligned_or_null(dq_weight, 4) || !aligned_or_null(dk_weight, 4)) return GQA_ERR_INVALID_ARGUMENT;
    if ((x.weight && !aligned(q, 16)) || (y.weight && !aligned(k, 16))) return GQA_ERR_INVALID_ARGUMENT;
    if ((st = check_rows(dq_out_layout, B, Hq, T, D, &x.grad_sb, &x.grad_sh, &x.grad_st)) != GQA_OK) return st;
    if ((st = check_rows(dk_out_layout, B, Hkv, T, D, &y.grad_sb, &y.grad_sh, &y.grad_st)) != GQA_OK) return st;
    if (x.weight && (st = check_rows(q_layout, B, Hq, T, D, &x.in_sb, &x.in_sh, &x.in_st)) != GQA_OK) return st;
    if (y.weight && (st = check_rows(k_layout, B, Hkv, T, D, &y.in_sb, &y.in_sh, &y.in_st)) != GQA_OK) return st;
    if ((st = check_rows(dq_layout, B, Hq, T, D, &x.out_sb, &x.out_sh, &x.out_st)) != GQA_OK) return st;
    if ((st = check_rows(dk_layout, B, Hkv, T, D, &y.out_sb, &y.out_sh, &y.out_st)) != GQA_OK) return st;
    const RopeBwdPlan r = rope_bwd_plan(B, T, Hq, Hkv, D);
    if (x.weight || y.weight) {
        if (!aligned(workspace, 256) || workspace_bytes < gqa_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hkv, D))
            return GQA_ERR_WORKSPACE;
        p.partial = static_cast<float*>(workspace);
    }
    x.grad = static_cast<const bf16*>(dq_out);
    y.grad = static_cast<const bf16*>(dk_out);
    x.in = static_cast<const bf16*>(q);
    y.in = static_cast<const bf16*>(k);
    x.out = static_cast<bf16*>(dq);
    y.out = static_cast<bf16*>(dk);
    const bool inter = rope->interleaved != 0;
    return D == 128 ? rope_bwd<128>(p, r, inter, dq_weight, dk_weight, static_cast<cudaStream_t>(stream))
                    : rope_bwd<64>(p, r, inter, dq_weight, dk_weight, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv4_append(const void* k, const void* v, void* k_pool, void* v_pool, const int* slots, int N, int Hkv,
                          int D, int page_size, int num_pages, const gqa_layout* k_layout, const gqa_layout* v_layout,
                          const gqa_kv4_layout* k_pool_layout, const gqa_kv4_layout* v_pool_layout, void* stream) {
    return kv4_rows(true, k, v, k_pool, v_pool, slots, N, Hkv, D, page_size, num_pages, k_layout, v_layout, k_pool_layout,
                    v_pool_layout, stream);
}

gqa_status gqa_kv4_gather(const void* k_pool, const void* v_pool, void* k, void* v, const int* slots, int N, int Hkv,
                          int D, int page_size, int num_pages, const gqa_kv4_layout* k_pool_layout,
                          const gqa_kv4_layout* v_pool_layout, const gqa_layout* k_layout, const gqa_layout* v_layout,
                          void* stream) {
    return kv4_rows(false, k, v, k_pool, v_pool, slots, N, Hkv, D, page_size, num_pages, k_layout, v_layout, k_pool_layout,
                    v_pool_layout, stream);
}

size_t gqa_attn_decode_kv4_workspace_bytes(int B, int Hq, int Hkv, int Tq, int max_seqlen_k, int D, int window) {
    if (check_dec4(B, Hq, Hkv, Tq, max_seqlen_k, D, window) != GQA_OK) return 0;
    return dec4_plan(B, Hq, Hkv, Tq, max_seqlen_k, D, window).bytes;
}

gqa_status gqa_attn_decode_kv4(const void* q, const void* k_pool, const void* v_pool, void* o, const int* seqlens_k,
                               const int* block_table, int page_size, int num_pages, int max_pages, int B, int Hq,
                               int Hkv, int Tq, int max_seqlen_k, int D, const gqa_kv4_layout* k_layout,
                               const gqa_kv4_layout* v_layout, float softmax_scale, int window, void* workspace,
                               size_t workspace_bytes, void* stream) {
    gqa_status st = check_dec4(B, Hq, Hkv, Tq, max_seqlen_k, D, window);
    if (st != GQA_OK) return st;
    if ((st = check_pages(page_size, num_pages)) != GQA_OK) return st;
    if (max_pages <= 0 || !aligned(q, 16) || !aligned(o, 16) || !aligned(seqlens_k, 4) || !aligned(block_table, 4))
        return GQA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(softmax_scale)) return GQA_ERR_INVALID_ARGUMENT;
    gqa::Dec4Params p{};
    if ((st = check_kv4_pool(k_pool, k_layout, num_pages, Hkv, page_size, D, &p.k_sb, &p.k_sh)) != GQA_OK) return st;
    if ((st = check_kv4_pool(v_pool, v_layout, num_pages, Hkv, page_size, D, &p.v_sb, &p.v_sh)) != GQA_OK) return st;
    const Dec4Plan r = dec4_plan(B, Hq, Hkv, Tq, max_seqlen_k, D, window);
    if ((st = dec4_workspace(p, r, workspace, workspace_bytes)) != GQA_OK) return st;
    p.q = static_cast<const bf16*>(q);
    p.o = static_cast<bf16*>(o);
    p.k = static_cast<const uint8_t*>(k_pool);
    p.v = static_cast<const uint8_t*>(v_pool);
    p.seqlens = seqlens_k;
    p.table = block_table;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.Tq = Tq;
    p.n_rc = r.n_rc;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.capacity = (int)std::min<long long>(max_seqlen_k, (long long)max_pages * page_size);
    p.window = window >= max_seqlen_k ? 0 : window;  // a window covering every key is plain causal
    p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)D)) * 1.4426950408889634f;
    p.timeout_ns = gqa::kWaitTimeoutNs;
    if ((p.err = gqa::device_error_ptr()) == nullptr) return GQA_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dec4_dispatch(D, r.nt, [&](auto d, auto nt) { return launch_dec4<d, nt>(p, r, s); });
}

gqa_status gqa_testing_decode_kv4_cut(unsigned long long total, int places, int i, int* out_runs,
                                      unsigned long long* out_start) {
    if (total == 0 || total >= 1ULL << 52 || places <= 0 || places > 1 << 12 || i < 0 || out_runs == nullptr || out_start == nullptr)
        return GQA_ERR_INVALID_ARGUMENT;
    *out_runs = (int)gqa::dec4_runs(total, (unsigned)places);
    if (i > *out_runs) return GQA_ERR_INVALID_ARGUMENT;
    *out_start = gqa::dec4_cut(total, (unsigned)i, (unsigned)*out_runs);
    return GQA_OK;
}

gqa_status gqa_testing_decode_kv4_largest_cluster(int ctas) {
    if (ctas < 1 || ctas > 16 || (ctas & (ctas - 1))) return GQA_ERR_INVALID_ARGUMENT;
    g_dec4_largest.store(ctas, std::memory_order_relaxed);
    return GQA_OK;
}

gqa_status gqa_testing_decode_kv4_merge(void* o, const int* seqlens_k, int B, int Hq, int Hkv, int Tq, int max_seqlen_k,
                                        int D, void* workspace, size_t workspace_bytes, int* out_runs, void* stream) {
    gqa_status st = check_dec4(B, Hq, Hkv, Tq, max_seqlen_k, D, 0);
    if (st != GQA_OK) return st;
    if (!aligned(o, 16) || !aligned(seqlens_k, 4) || out_runs == nullptr) return GQA_ERR_INVALID_ARGUMENT;
    const Dec4Plan r = dec4_plan(B, Hq, Hkv, Tq, max_seqlen_k, D, 0);
    if (r.bytes == 0) return GQA_ERR_UNSUPPORTED;  // merged without the workspace
    gqa::Dec4Params p{};
    if ((st = dec4_workspace(p, r, workspace, workspace_bytes)) != GQA_OK) return st;
    *out_runs = p.runs;
    p.o = static_cast<bf16*>(o);
    p.seqlens = seqlens_k;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.Tq = Tq;
    p.n_rc = r.n_rc;
    p.capacity = max_seqlen_k;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dec4_dispatch(D, r.nt, [&](auto d, auto nt) { return launch_dec4_merge<d, nt>(p, s); });
}

}  // extern "C"

// The whole routed layer for a few tokens (m <= 32) in two kernels.
//
//   logits = x . W_router^T   (f64 sums, rounded once to f32)
//   s = sigmoid(logits), ids = top_k of s + bias, w_j = s_j / sum_j s_j
//   a = silu(W_gate[e] x) * (W_up[e] x);  d = W_down[e] a
//   y = sum_j w_j d_j (slot order) [+ sigmoid(w_sh . x) d_shared]
// [cortiq-engine 0.7.7, src/mimo_moe.rs: routing of Dynamic::run and
// tests::exact_moe; hf2q qwen35/dense_ffn_arena.rs MoeFfnArena's shared
// expert], the definitions of moe_router_topk and moe_ffn_forward_shared.
//
// Kernel 1 (router): a block computes the logits of a few experts for a few
//   tokens, its warps splitting K.  The sum is kept in f64, in an order that
//   does not depend on the batch: the rounded logits are those of the exact sum
//   unless it lies within the f64 error of a border between two f32 values.
// Kernel 2 (experts): a cooperative grid of one block per SM.  Every block
//   repeats the routing of the few tokens (cheaper than a launch), takes an
//   equal share of all active experts' gate/up rows, then, after a grid
//   barrier, a share of the down rows.  For m <= 8 that share is the block's
//   own hidden rows of every active expert, so the weighted combine happens in
//   its shared memory, in slot order.  Larger batches may crowd many tokens on
//   one expert; re-reading all their activations in every block would then
//   cost more L2 traffic than the weights, so a block takes consecutive rows
//   of few experts instead, and the outputs d meet in global memory behind a
//   second grid barrier (same sums, same slot order, no atomics).
//
// The bound is reading the distinct chosen experts' weights once; every warp
// streams its own rows (stream_mma.cuh).  gate/up multiplies the bf16 x as it
// is; the f32 activation enters the down projection as three bf16 parts, so
// nothing is rounded below f32.  A row's K order is the same wherever it
// lands, so its bits depend on its own token alone.
//
// Measured (graph replays; 256 experts, hidden 4096, inter 1536, top-8): 1
// token 64 us (4.7 TB/s over the call, 5.6 while it streams), 8 tokens of 53
// experts 348 (5.8), 32 tokens of 126 experts 797 (6.0), 32 tokens on 16 experts
// 227 (2.7: their token rows, through L1 and L2).  Before the first expert byte: 9 us
// at 1 token, 21 at 32 (router 2.5 and 9, launch gap 2.6, routing 3.5 and 9).
#include <climits>
#include <math.h>

#include <type_traits>

#include "launch.h"
#include "stream_mma.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTileI = 16;   // intermediate rows of a gate/up tile (gate and up rows each)
constexpr int kTileH = 32;   // hidden rows of a down tile
constexpr int kMaxRows = kLayerDecodeMaxRows;

__device__ __forceinline__ double sigmoid_f64(float v) {
    return 1.0 / (1.0 + exp(-static_cast<double>(v)));
}

// ------------------------------------------------------------------ router
// A block takes ROWS experts (or the shared expert's gate) and TOK tokens; its
// warps split K.  Converting to f64 costs four times a multiply-add, so each
// converted weight serves TOK tokens and each converted x ROWS experts.  Few
// tokens take 2 x 4 or 2 x 8, so that many blocks read the weights, more take 4
// x 8, two blocks per SM.  (256 experts of 4096, against 2 x 4 with the tokens in
// passes: 8 tokens 4.2 us and 5.0, 32 tokens 9.7 and 13.0; 64 experts of 1024, 32
// tokens 4.0 and 8.2.)
// f64 additions round too, so their order is the same in every form: kSlices
// interleaved slices of K (8 columns each), each summed in the order of K, the
// slices of a warp in a tree over the lane's bits from the highest, the warps
// in order.  A block of fewer threads takes its slices in passes.
constexpr int kSlices = 512;

template <int ROWS, int TOK, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) layer_router_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ W_router,
    const __nv_bfloat16* __restrict__ w_sh, int m, int hidden, int n_experts,
    float* __restrict__ logits, float* __restrict__ scores, float* __restrict__ gate,
    unsigned* __restrict__ barrier, int* __restrict__ status) {
    constexpr int kSums = ROWS * TOK, kLanes = 32 / kSums;  // lanes that end with the same sum
    static_assert(kSums * kLanes == 32, "sums of a warp");
    __shared__ double part[kSlices / 32][kSums];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        *barrier = 0;  // of the kernel that follows
        *status = kDevOk;
    }
    const int n_rows = n_experts + (w_sh ? 1 : 0);
    const int r0 = blockIdx.x * ROWS, t0 = blockIdx.y * TOK;
    const __nv_bfloat16* wrow[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        const int r = min(r0 + j, n_rows - 1);
        wrow[j] = r < n_experts ? W_router + static_cast<size_t>(r) * hidden : w_sh;
    }
#pragma unroll 1
    for (int pass = 0; pass < kSlices / THREADS; ++pass) {
        double acc[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) acc[i] = 0.0;
        for (int k = (pass * THREADS + threadIdx.x) * 8; k < hidden; k += kSlices * 8) {
            float wf[ROWS][8];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) bf16x8_to_f32(*reinterpret_cast<const uint4*>(wrow[j] + k), wf[j]);
            uint4 xv[TOK];
#pragma unroll
            for (int q = 0; q < TOK; ++q)
                xv[q] = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(min(t0 + q, m - 1)) * hidden + k);
#pragma unroll
            for (int q = 0; q < TOK; ++q) {
                float xf[8];
                bf16x8_to_f32(xv[q], xf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double xd = xf[e];
#pragma unroll
                    for (int j = 0; j < ROWS; ++j)
                        acc[j * TOK + q] = fma(static_cast<double>(wf[j][e]), xd, acc[j * TOK + q]);
                }
            }
        }
        // the sums over 32 lanes: steps that halve the sums a lane holds (it ends
        // with sum number lane / kLanes), then the rest
#pragma unroll
        for (int h = kSums / 2; h >= 1; h >>= 1) {
            const bool upper = lane & (h * kLanes);
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const double give = upper ? acc[i] : acc[i + h];
                const double keep = upper ? acc[i + h] : acc[i];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, h * kLanes);
            }
        }
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        if (lane % kLanes == 0) part[pass * (THREADS / 32) + warp][lane / kLanes] = acc[0];
    }
    __syncthreads();
    const int r = r0 + threadIdx.x / TOK, t = t0 + threadIdx.x % TOK;
    if (threadIdx.x < kSums && r < n_rows && t < m) {
        double sum = 0.0;
#pragma unroll
        for (int w = 0; w < kSlices / 32; ++w) sum += part[w][threadIdx.x];
        const float l = static_cast<float>(sum);
        const float s = static_cast<float>(sigmoid_f64(l));
        if (r < n_experts) {
            logits[static_cast<size_t>(t) * n_experts + r] = l;
            scores[static_cast<size_t>(t) * n_experts + r] = s;
        } else {
            gate[t] = s;
        }
    }
}

// ----------------------------------------------------------------- experts
// Ring slots per warp: one holds the step that is used, the others are in
// flight.  With several groups of 8 tokens the L1 that a third slot takes is
// worth more for the token rows (32 tokens of 126 experts: 768 us with two, 790
// with three; on 16 experts 237 and 246), with one the bytes in flight are (8
// tokens of 53 experts: 360 and 348 us).
__host__ __device__ constexpr int ring_slots(int nt) { return nt == 1 ? 3 : 2; }

template <int SLOTS>
struct ExpertsSmem {
    unsigned char ring[kWarps][SLOTS][kRingBytes];  // first the routing keys, then weights
    int key[kMaxRows], sorted[kMaxRows], perm[kMaxRows];
    int gexp[kMaxRows], gfirst[kMaxRows + 1];
    int slot_id[kMaxRows];
    float weight[kMaxRows];
    int warp_n[kWarps], flag;
};
// The block-combining variant keeps the down outputs of its 32 hidden rows in
// shared memory, [routed rows, then shared rows][hidden row], behind ExpertsSmem;
// this many rows fit.
constexpr int kCombineRows = (232448 - static_cast<int>(sizeof(ExpertsSmem<ring_slots(1)>))) / ((kTileH + 1) * 4);

// Top-k of one token by (score + bias descending, expert ascending), by one
// warp.  key: the warp's scratch of n_experts floats.  Each lane keeps the
// best of its own experts; after a round only the winner's lane looks for its
// next one.
__device__ __forceinline__ void route_token(const float* __restrict__ scores,
                                            const float* __restrict__ bias, int n_experts, int top_k,
                                            float* key, int* out_id, float* out_w, int lane) {
    const auto ordered = [](float k) -> unsigned {  // NaN ranks as -inf, -0 as +0
        if (isnan(k)) k = -INFINITY;
        if (k == 0.0f) k = 0.0f;
        const unsigned b = __float_as_uint(k);
        return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    };
    unsigned* k = reinterpret_cast<unsigned*>(key);
    unsigned best = 0;  // 0: nothing left (every real key is above it)
    int best_e = INT_MAX;
    for (int e0 = lane; e0 < n_experts; e0 += 8 * 32) {  // eight loads at a time
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + 32 * i;
            s[i] = e < n_experts ? scores[e] + (bias ? bias[e] : 0.0f) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + 32 * i;
            const unsigned u = ordered(s[i]);
            if (e < n_experts) {
                k[e] = u;
                if (u > best) {
                    best = u;
                    best_e = e;
                }
            }
        }
    }
    int my_e = 0;
    for (int j = 0; j < top_k; ++j) {
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        const int win = static_cast<int>(
            __reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(best_e) : 0xffffffffu));
        if (lane == j) my_e = win;
        if (best_e == win) {
            k[win] = 0;
            best = 0;
            best_e = INT_MAX;
#pragma unroll 8
            for (int e = lane; e < n_experts; e += 32) {
                const unsigned u = k[e];
                if (u > best) {
                    best = u;
                    best_e = e;
                }
            }
        }
    }
    const float s = lane < top_k ? scores[my_e] : 0.0f;
    double wsum = 0.0;
    for (int j = 0; j < top_k; ++j) wsum += static_cast<double>(__shfl_sync(0xffffffffu, s, j));
    if (lane < top_k) {
        out_id[lane] = my_e;
        out_w[lane] = static_cast<float>(static_cast<double>(s) / wsum);
    }
    __syncwarp();
}

// One warp's share of a phase.  The rows of all groups (`wid` rows for each
// routed group, then wid_sh of the shared expert) are cut into tiles of `n`
// rows, the last of a group with fewer.  All warps take one tile each per
// round, so the grid reads one moving window of the weights (with a contiguous
// range of tiles per warp the slowest SM took 1.5 times the fastest's time at
// 6 GB of weights).  Within a round a block's warps take neighbouring tiles,
// mostly of one expert, whose tokens they share in the L1.
struct Share {
    int pos;    // this warp's tile of the round, or past the end
    int round;  // first tile of the round
    int end;    // tiles
    int n, per_group, wid, wid_sh;
};

struct Tile {
    int q, r, n;       // group, first row within it, rows
    int first, cnt;    // the group's tokens: sorted rows [first, first + cnt)
    int expert;        // -1: the shared expert
    const __nv_bfloat16 *w0, *w1;  // row r of gate and up (phase 1) or of down (w0)
    int k;             // row length
};

// Expert map of the routed rows (rows <= kMaxRows): sm.perm lists them by
// (expert, routed row); group q holds the rows of expert sm.gexp[q] at sorted
// positions sm.gfirst[q] up to sm.gfirst[q + 1].  Returns the number of groups.
template <class Smem>
__device__ __forceinline__ int map_rows(Smem& sm, int rows) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    static_assert(MOE_MAX_EXPERTS * kMaxRows <= INT_MAX, "sort keys");
    const int mine = tid < rows ? sm.slot_id[tid] * kMaxRows + tid : INT_MAX;  // keys are distinct
    if (tid < kMaxRows) sm.key[tid] = mine;
    __syncthreads();
    if (tid < rows) {
        int rank = 0;
        const int4* keys = reinterpret_cast<const int4*>(sm.key);
#pragma unroll 4
        for (int i = 0; i < (rows + 3) / 4; ++i) {
            const int4 v = keys[i];
            rank += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
        }
        sm.sorted[rank] = mine;
        sm.perm[rank] = tid;
    }
    __syncthreads();
    const int e = tid < rows ? sm.sorted[tid] / kMaxRows : -1;
    const bool opens = tid < rows && (tid == 0 || sm.sorted[tid - 1] / kMaxRows != e);
    const unsigned ballot = __ballot_sync(0xffffffffu, opens);
    if (lane == 0) sm.warp_n[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm.warp_n[w];
        total += sm.warp_n[w];
    }
    if (opens) {
        const int q = before + __popc(ballot & ((1u << lane) - 1u));
        sm.gexp[q] = e;
        sm.gfirst[q] = tid;
    }
    if (tid == 0) sm.gfirst[total] = rows;
    __syncthreads();
    return total;
}

template <int NT, bool COMBINE>
__global__ void __launch_bounds__(kThreads, 1) layer_experts_kernel(const LayerDecodeArgs a) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    constexpr int kStages = ring_slots(NT);
    using Smem = ExpertsSmem<kStages>;
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    float(*sm_d)[kTileH + 1] = reinterpret_cast<float(*)[kTileH + 1]>(smem_raw + sizeof(Smem));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int rows = a.m * a.top_k;
    const int n_shared = a.inter_sh > 0 ? 1 : 0;

    // routing and expert map of the few tokens, in every block
    {
        float* keys = reinterpret_cast<float*>(&sm.ring[warp][0][0]);
        static_assert(kStages * kRingBytes >= 4 * MOE_MAX_EXPERTS, "routing keys");
        for (int t = warp; t < a.m; t += kWarps)
            route_token(a.scores + static_cast<size_t>(t) * a.n_experts, a.bias, a.n_experts, a.top_k,
                        keys, sm.slot_id + t * a.top_k, sm.weight + t * a.top_k, lane);
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int r = tid; r < rows; r += kThreads) {
            a.ids[r] = sm.slot_id[r];
            a.weights[r] = sm.weight[r];
        }
    const int n_groups = map_rows(sm, rows);

    // Rows of the down phase: with COMBINE this block's own hidden rows
    // [h_lo, h_hi) of every group, otherwise all hidden rows.
    const int h_lo = COMBINE ? static_cast<int>(static_cast<long long>(a.hidden) * blockIdx.x / gridDim.x) : 0;
    const int h_hi = COMBINE ? static_cast<int>(static_cast<long long>(a.hidden) * (blockIdx.x + 1) / gridDim.x)
                             : a.hidden;

    // h0: hidden row of row 0 (down)
    const auto find_tile = [&](bool down, const Share& s, int h0) -> Tile {
        Tile t;
        t.q = min(s.pos / s.per_group, n_groups);
        t.r = (s.pos - t.q * s.per_group) * s.n;
        t.n = min(s.n, (t.q < n_groups ? s.wid : s.wid_sh) - t.r);
        if (t.q < n_groups) {
            t.first = sm.gfirst[t.q];
            t.cnt = sm.gfirst[t.q + 1] - t.first;
            t.expert = sm.gexp[t.q];
        } else {
            t.first = 0;
            t.cnt = a.m;
            t.expert = -1;
        }
        const int inter = t.expert < 0 ? a.inter_sh : a.inter;
        const size_t e = t.expert < 0 ? 0 : t.expert;
        if (!down) {
            const size_t at = (e * inter + t.r) * a.hidden;
            t.w0 = (t.expert < 0 ? a.S_gate : a.W_gate) + at;
            t.w1 = (t.expert < 0 ? a.S_up : a.W_up) + at;
            t.k = a.hidden;
        } else {
            t.w0 = (t.expert < 0 ? a.S_down : a.W_down) + (e * a.hidden + h0 + t.r) * inter;
            t.w1 = nullptr;
            t.k = inter;
        }
        return t;
    };
    // The warp's next tile (pos >= end when there is none).
    const auto next_round = [&](Share& s, bool of_grid) {
        const int blocks = of_grid ? gridDim.x : 1, b = of_grid ? blockIdx.x : 0;
        s.round += blocks * kWarps;
        const int tiles = min(blocks * kWarps, s.end - s.round);
        if (tiles <= 0) {
            s.pos = s.end;
            return;
        }
        // Large batches: a round is four runs of tiles, and a block takes a part
        // of each for four of its warps (one on each of the SM's schedulers), so
        // that no block gets crowded experts alone.  (32 tokens on 16 experts: 258
        // us instead of 271 with one run; on 126 experts 853 and 861.)  The warps
        // of a block then share fewer token rows in the L1, which costs a single
        // token 3%: it takes one run.
        constexpr int kRuns = NT == 1 ? 1 : 4, kW = kWarps / kRuns;
        const int run = warp / kW, first = tiles * run / kRuns, n = tiles * (run + 1) / kRuns - first;
        const int lo = n * b / blocks, hi = n * (b + 1) / blocks;
        s.pos = lo + warp % kW < hi ? s.round + first + lo + warp % kW : s.end;
    };
    // Tiles of at most `cap` rows whose rounds over the warps leave the least
    // of the last one idle.
    const auto share = [&](int wid, int wid_sh, int cap, bool of_grid) -> Share {
        Share s;
        const int workers = of_grid ? gridDim.x * kWarps : kWarps;
        // lane n - 1 weighs tiles of n rows
        const int n = lane + 1;
        const int per = (wid + n - 1) / n, tiles = n_groups * per + (wid_sh + n - 1) / n;
        const unsigned cost = n <= cap ? static_cast<unsigned>((tiles + workers - 1) / workers * (n + 3)) : UINT_MAX;
        const unsigned best = __reduce_min_sync(0xffffffffu, cost);
        const int pick = 31 - __clz(__ballot_sync(0xffffffffu, cost == best));  // the tallest of the best
        s.n = pick + 1;
        s.per_group = __shfl_sync(0xffffffffu, per, pick);
        s.end = __shfl_sync(0xffffffffu, tiles, pick);
        s.wid = wid;
        s.wid_sh = wid_sh;
        s.round = -workers;
        next_round(s, of_grid);
        return s;
    };

    // The producer side of the warp's stream: the tile and column that the
    // next ring fill takes.
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0]);
    Share ps{};
    Tile pt{};
    int pk = 0, fill_slot = 0, use_slot = 0;
    const auto fill = [&](bool down, int h0) {
        if (ps.pos < ps.end) {
            const uint32_t slot = ring + fill_slot * kRingBytes;
            const Tile& t = pt;
            const bool wide = t.n <= (down ? 16 : 8);
            const auto row = [&](int r) -> const __nv_bfloat16* {
                if (down) return r < t.n ? t.w0 + static_cast<size_t>(r) * t.k : nullptr;
                const int i = (r >> 4) * 8 + (r & 7);  // ring rows: 8 of gate, 8 of up, again
                return i < t.n ? (r & 8 ? t.w1 : t.w0) + static_cast<size_t>(i) * t.k : nullptr;
            };
            if (wide)
                ring_fill<true>(slot, row, pk, t.k, lane);
            else
                ring_fill<false>(slot, row, pk, t.k, lane);
            pk += wide ? 128 : 64;
            if (pk >= t.k) {
                next_round(ps, !(COMBINE && down));
                pk = 0;
                if (ps.pos < ps.end) pt = find_tile(down, ps, h0);
            }
        }
        cp_async_commit();  // an empty group once the share is used up, so that waits still count
        fill_slot = fill_slot + 1 == kStages ? 0 : fill_slot + 1;
    };

    // Issues the first fills of a share; the fills that the share before it
    // left over are empty.
    const auto begin = [&](bool down, const Share& s, int h0) {
        ps = s;
        pk = 0;
        if (ps.pos < ps.end) pt = find_tile(down, ps, h0);
        use_slot = fill_slot;
        for (int i = 0; i < kStages - 1; ++i) fill(down, h0);
    };

    // 32 rows per tile read the tokens half as often; with several token groups
    // the down phase's three parts leave no registers for it (32 tokens of 126
    // experts: 795 us with 32 rows, 768 with 16; 13 tokens 140 and 131; only on
    // 16 experts 227 and 237).
    constexpr int kDownCap = NT == 1 ? kTileH : 16;
    float acc[2][NT][4];
    const __nv_bfloat16* tok[NT];
    // Runs the warp's share after begin().
    const auto stream = [&](auto down_tag, Share s, int h0, auto finish) {
        constexpr bool kDown = decltype(down_tag)::value;
        constexpr int kParts = kDown ? 3 : 1;
        for (; s.pos < s.end; next_round(s, !(COMBINE && kDown))) {
            const Tile t = find_tile(kDown, s, h0);
            const int nt = (t.cnt + 7) >> 3;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int p = min(n * 8 + g, t.cnt - 1);
                if (kDown)
                    tok[n] = (t.expert < 0 ? a.act_sh : a.act) + static_cast<size_t>(t.first + p) * 3 * t.k;
                else
                    tok[n] = a.x + static_cast<size_t>(t.expert < 0 ? p : sm.perm[t.first + p] / a.top_k) * t.k;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
            }
            const bool wide = t.n <= (kDown ? 16 : 8);
            const auto ready = [&] {
                cp_async_wait_group<kStages - 2>();
                __syncwarp();
                // every lane has read the slot of the step before: it is free
                fill(kDown, h0);
            };
            const auto steps = [&](auto wide_tag) {
                constexpr bool kWide = decltype(wide_tag)::value;
                constexpr int kStep = kWide ? 128 : 64;
                if (NT == 1 || nt == 1) {
                    TokenPieces<kParts> ahead[2];
                    first_tokens<kWide>(ahead, tok[0], 0, t.k, kStep, lane);
                    for (int k0 = 0; k0 < t.k; k0 += kStep) {
                        ready();
                        ring_multiply_one<kWide>(acc, ring + use_slot * kRingBytes, ahead, tok[0], k0, t.k, kStep,
                                                 lane);
                        use_slot = use_slot + 1 == kStages ? 0 : use_slot + 1;
                    }
                } else {
                    for (int k0 = 0; k0 < t.k; k0 += kStep) {
                        ring_multiply<kWide, NT, kParts>(acc, ring + use_slot * kRingBytes, tok, nt, k0, t.k, lane,
                                                         ready);
                        use_slot = use_slot + 1 == kStages ? 0 : use_slot + 1;
                    }
                }
            };
            if (wide || (kDown && kDownCap == 16))
                steps(std::true_type{});
            else
                steps(std::false_type{});
            finish(t, nt);
        }
    };

    // ------------------------------------------------ gate / up -> activation
    {
        const Share s = share(a.inter, a.inter_sh, kTileI, true);
        begin(false, s, 0);
        stream(std::false_type{}, s, 0, [&](const Tile& t, int nt) {
            // element (h, n, e): gate (e < 2) or up (e >= 2) of row h * 8 + g, token n * 8 + 2 c + e % 2
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt) break;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = h * 8 + g, p = n * 8 + c * 2 + e;
                        if (row >= t.n || p >= t.cnt) continue;
                        const float gate = acc[h][n][e];
                        __nv_bfloat16 part[3];
                        split_bf16x3(gate / (1.0f + expf(-gate)) * acc[h][n][2 + e], part);
                        const int width = t.expert < 0 ? a.inter_sh : a.inter;
                        __nv_bfloat16* dst = (t.expert < 0 ? a.act_sh : a.act) +
                                             static_cast<size_t>(t.first + p) * 3 * width + t.r + row;
#pragma unroll
                        for (int z = 0; z < 3; ++z) dst[static_cast<size_t>(z) * width] = part[z];
                    }
            }
        });
    }

    // The down weights do not depend on the activation: their first steps are
    // on their way while the grid meets.
    grid_arrive(a.barrier);
    int h0 = h_lo;
    int nh = COMBINE ? min(kTileH, h_hi - h0) : a.hidden;
    Share s = share(max(nh, 0), n_shared ? max(nh, 0) : 0, kDownCap, !COMBINE);
    begin(true, s, h0);
    if (!grid_wait(a.barrier, gridDim.x, &sm.flag, a.status, a.wait_limit_ns)) return;

    // ------------------------------------------------ down + combine
    // element (h, n, e): hidden row h * 16 + (e / 2) * 8 + g, token n * 8 + 2 c + e % 2
    const auto each_output = [&](const Tile& t, int nt, auto store) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = h * 16 + (e >> 1) * 8 + g, p = n * 8 + c * 2 + (e & 1);
                    if (row < t.n && p < t.cnt)
                        store(t.expert < 0 ? rows + p : sm.perm[t.first + p], t.r + row, acc[h][n][e]);
                }
        }
    };
    if (COMBINE) {
        while (h0 < h_hi) {
            stream(std::true_type{}, s, h0, [&](const Tile& t, int nt) {
                each_output(t, nt, [&](int r, int h, float v) { sm_d[r][h] = v; });
            });
            __syncthreads();
            for (int u = tid; u < a.m * kTileH; u += kThreads) {
                const int t = u / kTileH, h = u % kTileH;
                if (h >= nh) continue;
                float y = 0.0f;
                for (int j = 0; j < a.top_k; ++j) y += sm.weight[t * a.top_k + j] * sm_d[t * a.top_k + j][h];
                if (n_shared) y += a.gate[t] * sm_d[rows + t][h];
                a.y[static_cast<size_t>(t) * a.hidden + h0 + h] = y;
            }
            __syncthreads();
            h0 += kTileH;
            nh = min(kTileH, h_hi - h0);
            if (h0 >= h_hi) break;
            s = share(nh, n_shared ? nh : 0, kDownCap, false);
            begin(true, s, h0);
        }
    } else {
        stream(std::true_type{}, s, 0, [&](const Tile& t, int nt) {
            each_output(t, nt, [&](int r, int h, float v) { a.d[static_cast<size_t>(r) * a.hidden + h] = v; });
        });
        grid_arrive(a.barrier);
        if (!grid_wait(a.barrier, 2 * gridDim.x, &sm.flag, a.status, a.wait_limit_ns)) return;
        const int total = a.m * (a.hidden / 4);
        for (int u = blockIdx.x * kThreads + tid; u < total; u += gridDim.x * kThreads) {
            const int t = u / (a.hidden / 4), h = (u % (a.hidden / 4)) * 4;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            const auto add = [&](float w, size_t r) {
                const float4 v = *reinterpret_cast<const float4*>(a.d + r * a.hidden + h);
                y.x += w * v.x;
                y.y += w * v.y;
                y.z += w * v.z;
                y.w += w * v.w;
            };
            for (int j = 0; j < a.top_k; ++j) add(sm.weight[t * a.top_k + j], t * a.top_k + j);
            if (n_shared) add(a.gate[t], rows + t);
            *reinterpret_cast<float4*>(a.y + static_cast<size_t>(t) * a.hidden + h) = y;
        }
    }
}

template <int NT, bool COMBINE>
cudaError_t launch_experts(const LayerDecodeArgs& args, int num_sms, cudaStream_t stream) {
    const int d_rows = COMBINE ? args.m * (args.top_k + (args.inter_sh > 0 ? 1 : 0)) : 0;
    using Smem = ExpertsSmem<ring_slots(NT)>;
    const int smem = static_cast<int>(sizeof(Smem)) + d_rows * (kTileH + 1) * 4;
    static PerDeviceOnce once;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(layer_experts_kernel<NT, COMBINE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_experts_kernel<NT, COMBINE>, args);
}

}  // namespace

cudaError_t launch_layer_decode(const LayerDecodeArgs& args, const __nv_bfloat16* W_router,
                                const __nv_bfloat16* w_sh, float* logits, int num_sms,
                                cudaStream_t stream) {
    const int n_rows = args.n_experts + (args.inter_sh > 0 ? 1 : 0);
    float *scores = const_cast<float*>(args.scores), *gate = const_cast<float*>(args.gate);
    const auto router = [&](auto kernel, int rows, int tokens, int threads) {
        kernel<<<dim3((n_rows + rows - 1) / rows, (args.m + tokens - 1) / tokens), threads, 0, stream>>>(
            args.x, W_router, w_sh, args.m, args.hidden, args.n_experts, logits, scores, gate, args.barrier,
            args.status);
    };
    if (args.m <= 4)
        router(layer_router_kernel<2, 4, 512>, 2, 4, 512);
    else if (args.m <= 8)
        router(layer_router_kernel<2, 8, 512>, 2, 8, 512);
    else
        router(layer_router_kernel<4, 8, 256>, 4, 8, 256);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int d_rows = args.m * (args.top_k + (args.inter_sh > 0 ? 1 : 0));
    if (args.m <= 8 && d_rows <= kCombineRows) return launch_experts<1, true>(args, num_sms, stream);
    if (args.m <= 8) return launch_experts<1, false>(args, num_sms, stream);
    if (args.m <= 16) return launch_experts<2, false>(args, num_sms, stream);
    return launch_experts<4, false>(args, num_sms, stream);
}

}  // namespace moe

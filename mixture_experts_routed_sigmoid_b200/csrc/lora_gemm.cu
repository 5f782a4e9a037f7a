// The projection with adapters for larger batches, in one tcgen05 GEMM:
//   y[t] = W x[t] + B[a] (scales[a] h[t]),  a = adapter_ids[t],
// with h = A x and its scaling from the shrink kernel, as bf16 parts that add up
// to it: three for an f32 y, which keep its 24 bits (two leave an error of 2.5e-6
// of the adapter's term, ten times that of f32 arithmetic), two for a bf16 y
// (2^-17, below its own 2^-8).
//
// A CTA pair owns a tile of 256 tokens x `bn` output columns (M = 256, N = bn
// MMAs over both CTAs; each CTA loads its 128 tokens and its half of W's rows,
// 128 bytes of K per stage).  The adapters enter as more columns of K beside the
// projection's: for every adapter that occurs among the tile's tokens, its
// rank columns (rounded up to 16) once for each part of h, which is zero for the
// tokens of other adapters.  So they cost parts * rank / k of the projection's
// MMAs per adapter of a tile, and no pass over y.
//
// Where tiles are few (SPLIT), a cluster of 1, 2 or 4 pairs takes one tile: each
// pair a part of K and of the adapters' stages.  The partial tiles meet in
// distributed shared memory, and all warps of every CTA add and store their
// share of the columns, pairs in order.
//
// The adapters' stages have two buffers of their own beside the ring, so they
// are copied while the projection of the same tile runs (in the ring's order
// they came six stages ahead at most, and the tensor core waited 1.7 us a tile).
//
// A zero times NaN or infinity is NaN, so a piece of B that is not finite never
// reaches the tensor core: its writer replaces it by zeros and marks the tile,
// and the epilogue adds the piece's products for the tokens that do use it.
//
// Warps per CTA: 0 copies the tiles (TMA), 1 issues the MMAs (leader CTA only),
// 2 and 3 check the adapters' stages and announce them to the leader, 8-11 copy
// those stages (cp.async: 16-byte pieces of h and B picked by adapter), 4-7 and
// 12-15 are the epilogue.  A fence or a release waits for its thread's copies in
// flight, so the threads that copy never fence (a stage took 3100 cycles when
// they did).  Two accumulators let the epilogue of one overlap the next one's
// MMAs.  Every wait is bounded.
//
// Bound by the tensor core: 4096 tokens of 4096 x 4096, 8 adapters of rank 16,
// bf16 out: 122.5 us with the shrink kernel (1.12 PFLOP/s); 16384 tokens of 2048 x
// 4096, 16 adapters of rank 64, f32 out: 254 us (1.08).
#include <algorithm>

#include "launch.h"
#include "pair_mma.cuh"

namespace moe {
namespace {

constexpr int kMaxStages = 8;         // ring of the projection's stages
constexpr int kExt = 2;               // stages of the adapters' columns, beside the ring
constexpr int kHalf = 128 * 128;      // bytes of 128 rows x 64 columns
constexpr int kThreads = 512;
constexpr int kChunk = 12;            // stages per accumulator, at most (f32 output, first product)
constexpr int kChunkBf16 = 16;        // and of the projection for a bf16 output
constexpr int kTmemCols = 512;
constexpr int kFixSlots = 4;
constexpr int kPartPitch = 36;        // words of a partial tile's row of 32 columns
constexpr int kPitch = 33;            // words of a staged epilogue row
constexpr int kEpiBytes = 8 * 16 * kPitch * 4;  // 16 rows of 32 columns per epilogue warp
constexpr int kTail = kEpiBytes + 512 + kLoraTileRows * 4 + 1024;  // behind the stages, and alignment
constexpr int kSmemLimit = 232448;
// Bytes of a stage and the ring's stages for tiles of bn columns: 4 at 256, 5
// at 192 (430 -> 385 cycles a stage against 4 there), 8 at 64.
__host__ __device__ inline int stage_bytes(int bn) { return kHalf + bn / 2 * 128; }
__host__ __device__ inline int ring_stages(int bn) {
    const int fit = (kSmemLimit - kTail) / stage_bytes(bn) - kExt;
    return fit < kMaxStages ? fit : kMaxStages;
}

__device__ __forceinline__ bool not_finite_bf16x8(const uint4& v) {
    bool bad = false;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// The conjunction over the four warps that write the adapters' stages, so that
// they go on or stop together.
__device__ __forceinline__ bool all_of_four_warps(bool v) {
    int r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, 128, q;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<int>(v))
        : "memory");
    return r != 0;
}

// Barriers 2 to 5: the warps of one warpgroup (1 is the copying warps').
__device__ __forceinline__ void warpgroup_sync(int warpgroup) {
    asm volatile("bar.sync %0, 128;" ::"r"(2 + warpgroup) : "memory");
}

// Products of the pieces of B[adapter] row `col` that are not finite.
__device__ __forceinline__ float fix_up(const LoraArgs& a, long long t, int id, int col) {
    const __nv_bfloat16* b = a.B + (static_cast<size_t>(id) * a.n + col) * a.rank;
    const __nv_bfloat16* h = a.h_split + static_cast<size_t>(t) * a.h_parts * a.r16;
    float s = 0.0f;
    for (int r = 0; r < a.rank; r += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(b + r);
        if (!not_finite_bf16x8(v)) continue;
        float bf[8];
        bf16x8_to_f32(v, bf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float hv = 0.0f;
            for (int z = a.h_parts - 1; z >= 0; --z) hv += __bfloat162float(h[z * a.r16 + r + e]);
            s += bf[e] * hv;
        }
    }
    return s;
}

// Stores ROWS rows x 32 columns from shared memory (rows of kPitch words).
template <int ROWS>
__device__ __forceinline__ void store_chunk(const LoraArgs& a, const float* buf, long long t0, int col0,
                                            int lane) {
    if (a.y_dtype == MOE_DTYPE_BF16) {
        // 8 columns per lane: 8 rows x 64 bytes per instruction
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
        const int cc = (lane & 3) * 8, col = col0 + cc;
#pragma unroll
        for (int i = 0; i < ROWS / 8; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (t0 + r >= a.m || col >= a.n) continue;
            const float* s = buf + r * kPitch + cc;
            __nv_bfloat16* dst = y + (t0 + r) * a.n + col;
            if ((a.n & 7) == 0) {
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(s[2 * q], s[2 * q + 1]);
                    o[q] = *reinterpret_cast<const uint32_t*>(&b);
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                for (int q = 0; q < 8; ++q)
                    if (col + q < a.n) dst[q] = __float2bfloat16_rn(s[q]);
            }
        }
    } else {
        float* y = static_cast<float*>(a.y);
        const int cc = (lane & 7) * 4, col = col0 + cc;
#pragma unroll
        for (int i = 0; i < ROWS / 4; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (t0 + r >= a.m || col >= a.n) continue;
            const float* s = buf + r * kPitch + cc;
            float* dst = y + (t0 + r) * a.n + col;
            if ((a.n & 3) == 0) {
                *reinterpret_cast<float4*>(dst) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                for (int q = 0; q < 4; ++q)
                    if (col + q < a.n) dst[q] = s[q];
            }
        }
    }
}

// An adapter id out of range anywhere in the call: nothing is written.
__device__ __forceinline__ bool any_bad_tile(const LoraArgs& a, int row_tiles, int lane) {
    bool bad = false;
    for (int i = lane; i < row_tiles; i += 32) bad |= a.tile_count[i] < 0;
    return __any_sync(0xffffffffu, bad);
}

// SPLIT tiles with many adapters add them token by token while the pairs' sums
// are joined: the stages' time grows with the adapters, the rank and the parts, a
// token's rows of B are read once either way.  (128 tokens of 4096 x 4096, us with
// stages and by token: rank 16, two parts, 20 adapters 34.2 and 34.9, 40 39.1 and
// 35.3, three parts, 16 34.8 and 35.5, 20 36.9 and 35.6; rank 32, two, 24 39.8 and
// 41.9, 40 47.4 and 43.8, three, 16 39.5 and 41.7, 24 44.7 and 42.5; rank 128,
// two, 24 84.8 and 137, 64 195 and 198, three, 24 108 and 138, 64 255 and 199.)
__device__ __forceinline__ bool gathers(const LoraArgs& a, int tile_count) {
    return tile_count * a.h_parts > 36 + 12 * (a.r16 / 16);
}

// more[r] = B[id of token t0 + r] row `col` . h[t0 + r] for 8 tokens (my_id: the
// ids in lanes 0 to 7); the lanes' columns are neighbours.  Sixteen loads of B
// are in flight at a time; four lanes hold a token's h (32 columns of the rank)
// and pass the values around.
__device__ __forceinline__ void gather_rows(const LoraArgs& a, float (&more)[8], long long t0, int my_id,
                                            int col, int lane) {
    int id[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        more[r] = 0.0f;
        id[r] = __shfl_sync(0xffffffffu, my_id, r);
    }
    const bool in = col < a.n;
    const int h_token = lane >> 2, h_id = __shfl_sync(0xffffffffu, my_id, h_token);
    const __nv_bfloat16* h_row = a.h_split + (t0 + (h_id >= 0 ? h_token : 0)) * a.h_parts * a.r16 + (lane & 3) * 8;
    for (int k0 = 0; k0 < a.rank; k0 += 32) {
        float h[8];
        const bool h_in = h_id >= 0 && k0 + (lane & 3) * 8 < a.rank;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = 0.0f;
        for (int z = a.h_parts - 1; z >= 0; --z) {
            float part[8];
            bf16x8_to_f32(h_in ? *reinterpret_cast<const uint4*>(h_row + z * a.r16 + k0) : make_uint4(0u, 0u, 0u, 0u),
                          part);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] += part[e];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (k0 + half * 16 >= a.rank) break;
            uint4 b[2][8];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int k = k0 + half * 16 + s * 8;
                    b[s][r] = in && id[r] >= 0 && k < a.rank
                        ? *reinterpret_cast<const uint4*>(
                              a.B + (static_cast<size_t>(id[r]) * a.n + col) * a.rank + k)
                        : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float bf[8];
                    bf16x8_to_f32(b[s][r], bf);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        more[r] = fmaf(bf[e], __shfl_sync(0xffffffffu, h[e], r * 4 + half * 2 + s), more[r]);
                }
        }
    }
}

// grid: CTA pairs as clusters of 2 that walk the tiles, or with SPLIT a cluster
// of `split` pairs per tile.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const LoraArgs a, int bn, int n_col_tiles, int n_tiles, int split) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int stage_size = stage_bytes(bn), n_stages = ring_stages(bn);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + (n_stages + kExt) * stage_size + kEpiBytes);  // leader's
    uint64_t* empty = full + kMaxStages;
    uint64_t* acc_full = empty + kMaxStages;   // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2], leader's are used
    uint64_t* ext_full = acc_empty + 2;     // [kExt], leader's are used
    uint64_t* ext_empty = ext_full + kExt;
    uint64_t* landed = ext_empty + kExt;    // [kExt] an adapters' stage whose copies have landed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(landed + kExt);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* bad_ext = reinterpret_cast<volatile int*>(tmem_slot + 2);  // [kExt], leader's are used
    // Tiles (1 + index) that hold a piece of B which is not finite, at the
    // tile's place in this pair's sequence modulo kFixSlots.  The MMA issuer
    // writes them, at most two accumulators ahead of the epilogue.
    volatile int* fix = bad_ext + kExt;
    int* list = const_cast<int*>(fix) + kFixSlots;  // [kLoraTileRows] the tile's adapters
    float* epi = reinterpret_cast<float*>(smem + (n_stages + kExt) * stage_size);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this CTA of its pair, the pair's leader, and the pair's part of a split tile
    const uint32_t rank = cluster_rank() & 1u, lead = cluster_rank() & ~1u;
    const int part = SPLIT ? static_cast<int>(cluster_rank() >> 1) : 0, parts = SPLIT ? split : 1;
    if (tid == 0) {
        for (int s = 0; s < n_stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kExt; ++s) {
            mbar_init(&ext_full[s], 2);   // one arrival from each CTA
            mbar_init(&ext_empty[s], 1);
            mbar_init(&landed[s], 128);   // the copying threads
            bad_ext[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);  // the epilogue warps of both CTAs
        }
        for (int i = 0; i < kFixSlots; ++i) fix[i] = 0;
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&map_x);
        prefetch_tensormap(&map_w);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.status, a.wait_limit_ns};

    const int cluster = blockIdx.x / (2 * parts), n_clusters = gridDim.x / (2 * parts);
    const int nk_all = (a.k + 63) / 64, kb_lo = nk_all * part / parts;
    const int nk = nk_all * (part + 1) / parts - kb_lo;  // this pair's stages of the projection
    const int half = bn / 2;
    // The tensor core's accumulator truncates: its sums over K are off by 1e-9 K of
    // their size (2.1e-6 at 2048, 1.9e-5 at 16384), where additions that round are
    // off by 5e-7.  So they are taken from it every 768 columns of K for an f32
    // output (6.5e-7 at every K), every 1024 for a bf16 one, and added in registers.
    // (16384 tokens of 2048 x 4096, f32: 242 us without, 250 with 768 columns, 261
    // with 512: the two accumulators then hold too little work to cover the stores
    // of a tile.  4096 tokens of 4096 x 4096, bf16: 120.5 us without, 122.5 with
    // 1024 columns, 126 with 768; 2.4, 0.7 and 0.5 of 1000 values are then not the
    // rounding of the exact one, of sums in f32 arithmetic 0.4.)
    const int chunk = a.y_dtype == MOE_DTYPE_F32 ? kChunk : kChunkBf16, n_chunks = (nk + chunk - 1) / chunk;
    // MMA steps (16 columns of K) of the adapters of a tile.  The shrink kernel
    // must have finished: waited for behind the first tile's projection, and
    // from the second tile on the count is loaded ahead of the tile.
    const auto ext_steps = [&](int tile, int& first) {
        const int count = max(a.tile_count[tile / n_col_tiles], 0);
        const int all = SPLIT && gathers(a, count) ? 0 : count * a.h_parts * (a.r16 / 16);
        if (!SPLIT) {
            first = 0;
            return all;
        }
        const int stages = (all + 3) / 4;  // whole stages to each pair
        first = stages * part / parts * 4;
        return min(stages * (part + 1) / parts * 4, all) - first;
    };
    const auto advance = [&](int& stage, uint32_t& phase) {
        if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
        }
    };

    // SPLIT: the pair's partial tile [bn / 32][128 rows][kPartPitch], over the
    // stages once they are used up
    float* partial = reinterpret_cast<float*>(smem);

    // The epilogue's sums are 128 registers a thread: 4 warpgroups of 128 at
    // launch become 72 + 184 + 72 + 184.
    constexpr int kFewRegisters = 72, kManyRegisters = 184;
    static_assert(2 * (kFewRegisters + kManyRegisters) <= 4 * 65536 / kThreads, "of those at launch");
    if (((warp >> 2) & 1) == 0) {
        registers_down<kFewRegisters>();
        if (warp == 0) {
            // ------------------------------------------------------ tile copies
            if (lane == 0) {
                int stage = 0;
                uint32_t phase = 0;
                bool good = true;
                for (int tile = cluster; tile < n_tiles && good; tile += n_clusters) {
                    const int mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
                    for (int kb = 0; kb < nk; ++kb) {
                        if (!(good = mbar_wait_cluster(&empty[stage], phase ^ 1, ctl))) break;
                        const uint32_t bar = cluster_addr(smem_u32(&full[stage]), lead);
                        uint8_t* sa = smem + stage * stage_size;
                        // the leader expects both CTAs' bytes (an arrival from the other CTA
                        // would need a release at cluster scope, 0.5 us a stage)
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kHalf + half * 128));
                        tma_load_2d_pair(sa, &map_x, bar, (kb_lo + kb) * 64, mt * 256 + static_cast<int>(rank) * 128);
                        tma_load_2d_pair(sa + kHalf, &map_w, bar, (kb_lo + kb) * 64,
                                         nt * bn + static_cast<int>(rank) * half);
                        advance(stage, phase);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            // The whole warp walks the loop and one elected lane issues: in a branch
            // that only one lane enters, the compiler does not know the operands to
            // be uniform, and the four MMAs of a stage took 489 cycles to issue.
            if (rank == 0) {
                int stage = 0, acc = 0, n = 0, seq = 0;
                uint32_t phase = 0, acc_phase = 0;
                const bool leader = elect_one();
                // instruction descriptor: M = 256, N = bn
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                       (static_cast<uint32_t>(bn >> 3) << 17) | ((256u >> 4) << 24);
                // the start address is the descriptor's low 14 bits (in 16 bytes); all
                // of the ring lies below 2^18, so additions never carry out of it
                const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
                bool good = true;
                const auto finish_chunk = [&] {
                    if (leader) umma_commit_pair(&acc_full[acc], lead);
                    __syncwarp();
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1;
                };
                for (int tile = cluster; tile < n_tiles && good; tile += n_clusters, ++seq) {
                    uint32_t d = 0;
                    int first, steps = tile == cluster ? 0 : ext_steps(tile, first);
                    // The adapters' stages are spread evenly over the projection's, so
                    // that the copies of those beyond the two buffers have their time
                    // (16384 tokens of rank 64, three stages a tile: 286 us, 319 with all
                    // at the end); those of the first tile follow it.
                    int ext = 0, ext_all = (steps + 3) / 4;
                    const auto adapter_stage = [&]() -> bool {
                        const int e = n % kExt, left = steps - 4 * ext;
                        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&ext_full[e], n / kExt & 1u, ctl))) return false;
                        tc_fence_after_sync();
                        const uint64_t da = desc0 + static_cast<uint64_t>((n_stages + e) * (stage_size >> 4));
                        if (bad_ext[e] && lane == 0) {
                            bad_ext[e] = 0;
                            const uint32_t at = smem_u32(const_cast<int*>(&fix[seq % kFixSlots]));
                            for (int q = 0; q < 2 * parts; ++q) st_shared_cluster(cluster_addr(at, q), tile + 1);
                            fence_cluster();
                        }
                        __syncwarp();
                        if (leader) {
                            for (int k4 = 0; k4 < min(4, left); ++k4)
                                umma_bf16_pair(d, da + k4 * 2, da + (kHalf >> 4) + k4 * 2, idesc, 1);
                            umma_commit_pair(&ext_empty[e], lead);
                        }
                        __syncwarp();
                        ++ext, ++n;
                        return true;
                    };
                    bool ready = false;
                    int in_chunk = chunk;  // stages that the accumulator has
                    int kb = 0;
                    bool waited = tile != cluster;
                    for (;;) {
                        const int stop = ext < ext_all ? ((ext + 1) * nk + ext_all - 1) / ext_all : nk;
                        for (; kb < stop; ++kb, ++in_chunk) {
                            if (in_chunk == chunk) {
                                if (kb > 0) finish_chunk();
                                in_chunk = 0;
                                good = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[acc], acc_phase ^ 1, ctl));
                                if (!good) break;
                                tc_fence_after_sync();
                                d = tmem + static_cast<uint32_t>(acc * 256);
                            }
                            good = __all_sync(0xffffffffu, ready || mbar_wait(&full[stage], phase, ctl));
                            if (!good) break;
                            tc_fence_after_sync();
                            const uint64_t da = desc0 + static_cast<uint64_t>(stage * (stage_size >> 4));
                            uint64_t* done = &empty[stage];
                            advance(stage, phase);
                            // the next stage's barrier is asked while these MMAs are issued
                            if (kb + 1 < nk) ready = mbar_test(&full[stage], phase);
                            if (leader) {
#pragma unroll
                                for (int k4 = 0; k4 < 4; ++k4)
                                    umma_bf16_pair(d, da + k4 * 2, da + (kHalf >> 4) + k4 * 2, idesc,
                                                   (in_chunk | k4) != 0);
                                umma_commit_pair(done, lead);
                            }
                            __syncwarp();
                        }
                        if (good && kb == nk && !waited) {
                            wait_for_previous_kernel();
                            steps = ext_steps(tile, first);
                            ext_all = (steps + 3) / 4;
                            waited = true;
                        }
                        if (!good || ext == ext_all) break;
                        if (!(good = adapter_stage())) break;
                    }
                    if (!good) break;
                    finish_chunk();
                }
            }
            __syncwarp();
        } else if (warp < 4) {
            // ------------------------------------------------------ checking them
            // a stage each
            wait_for_previous_kernel();
            const int e = warp - 2;
            static_assert(kExt == 2, "one checking warp per stage");
            uint8_t* sa = smem + (n_stages + e) * stage_size;
            int n = 0;
            bool good = true;
            for (int tile = cluster; tile < n_tiles && good; tile += n_clusters) {
                int first;
                for (int left = ext_steps(tile, first); left > 0; left -= 4, ++n) {
                    if (n % kExt == e) {
                        good = __all_sync(0xffffffffu, mbar_wait(&landed[e], n / kExt & 1u, ctl));
                        if (!good) break;
                        // pieces of B that are not finite become zeros (the epilogue
                        // adds their products)
                        uint4* b = reinterpret_cast<uint4*>(sa + kHalf) + lane;
                        bool bad = false;
#pragma unroll 8
                        for (int i = 0; i < half * 8 / 32; ++i) {
                            if (not_finite_bf16x8(b[i * 32])) {
                                b[i * 32] = make_uint4(0u, 0u, 0u, 0u);
                                bad = true;
                            }
                        }
                        if (bad) st_shared_cluster(cluster_addr(smem_u32(const_cast<int*>(&bad_ext[e])), lead), 1);
                        fence_proxy_async_smem();  // the copies and the zeros, for the tensor core
                        __syncwarp();
                        if (lane == 0) {
                            if (rank == 0)
                                mbar_arrive(&ext_full[e]);
                            else
                                mbar_arrive_cluster(cluster_addr(smem_u32(&ext_full[e]), lead));
                        }
                    }
                }
            }
        } else {
            // ------------------------------------------------------ adapters' stages
            wait_for_previous_kernel();
            // A thread copies piece tid % 8 of rows tid / 8 + 16 i: eight lanes take
            // 128 contiguous bytes of a row (a row per lane would cost 32 memory
            // transactions per instruction, 2000 cycles a stage).
            const int pt = tid - 256, piece = pt & 7, row0 = pt >> 3;
            const uint32_t ext = smem_u32(smem) + static_cast<uint32_t>(row0 * 128 + ((piece ^ (row0 & 7)) << 4));
            const size_t b_adapter = static_cast<size_t>(a.n) * a.rank;
            const int h_pitch = a.h_parts * a.r16;
            int n = 0;
            bool good = true;
            for (int tile = cluster; tile < n_tiles; tile += n_clusters) {
                const int mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
                const int count = max(a.tile_count[mt], 0);
                // the warps go on or stop together; the last tile's list is read
                if (!all_of_four_warps(good)) break;
                for (int i = pt; i < count; i += 128)
                    list[i] = a.tile_list[static_cast<size_t>(mt) * kLoraTileRows + i];
                all_of_four_warps(true);
                const long long t0 = static_cast<long long>(mt) * 256 + rank * 128 + row0;
                const int col0 = nt * bn + static_cast<int>(rank) * half + row0;
                int id[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) id[i] = t0 + 16 * i < a.m ? a.adapter_ids[t0 + 16 * i] : -1;
                // this thread's column among the adapters': adapter of the list and
                // column within its parts
                int first;
                const int steps = ext_steps(tile, first);
                int ad = (first * 16 + piece * 8) / h_pitch, rem = first * 16 + piece * 8 - ad * h_pitch;
                for (int left = steps; left > 0; left -= 4, ++n) {
                    const int e = n % kExt;
                    if (!(good = mbar_wait_cluster(&ext_empty[e], (n / kExt & 1u) ^ 1u, ctl))) break;
                    const uint32_t sa = ext + static_cast<uint32_t>((n_stages + e) * stage_size);
                    const bool in = ad < count;
                    const int adapter = in ? list[ad] : 0;
                    int r = rem;  // column of the rank
                    while (r >= a.r16) r -= a.r16;
                    const bool b_in = in && r < a.rank;
                    const __nv_bfloat16* h = a.h_split + t0 * h_pitch + rem;
                    const __nv_bfloat16* b = a.B + adapter * b_adapter + static_cast<size_t>(col0) * a.rank + r;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool use = in && id[i] == adapter;
                        cp_async_16(sa + i * 16 * 128, use ? h + i * 16 * h_pitch : a.h_split, use ? 16u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (row0 + 16 * i >= half) break;
                        const bool use = b_in && col0 + 16 * i < a.n;
                        cp_async_16(sa + kHalf + i * 16 * 128, use ? b + i * 16 * a.rank : a.B, use ? 16u : 0u);
                    }
                    cp_async_arrive_noinc(&landed[e]);
                    for (rem += 64; rem >= h_pitch; rem -= h_pitch) ++ad;
                }
            }
            cp_async_wait_all();
        }
        __syncwarp();
        if (SPLIT) {
            warpgroup_sync(warp >> 2);  // between two register changes
            registers_up<65536 / kThreads>();
        }
    } else {
        registers_up<kManyRegisters>();
        // ------------------------------------------------------ epilogue
        // Two warps per 32 rows, each half of the tile's columns (32 at a time).
        wait_for_previous_kernel();
        const bool write = !any_bad_tile(a, n_tiles / n_col_tiles, lane);
        if (!write && blockIdx.x == 0 && tid == 128) set_status(a.status, kDevBadId);
        const int quarter = warp & 3, blocks = bn / 32;
        const int c_lo = warp < 8 ? 0 : (blocks + 1) / 2, n_c = warp < 8 ? (blocks + 1) / 2 : blocks / 2;
        float* buf = epi + (quarter + (warp < 8 ? 0 : 4)) * 16 * kPitch;
        int acc = 0, seq = 0;
        uint32_t acc_phase = 0;
        for (int tile = cluster; tile < n_tiles; tile += n_clusters, ++seq) {
            const int mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
            const long long t0 = static_cast<long long>(mt) * 256 + rank * 128 + quarter * 32;
            float sum[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
            bool good = true;
            for (int ch = 0; ch < n_chunks; ++ch) {
                good = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[acc], acc_phase, ctl));
                if (!good) break;
                tc_fence_after_sync();
                const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(acc * 256 + c_lo * 32);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= n_c) break;  // warp-uniform
                    uint32_t v[32];
                    tmem_load_32cols(taddr + c * 32, v);
                    tmem_load_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(v[j]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[acc]), lead));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
            if (!good) break;
            if (SPLIT) {  // this pair's partial tile, for the whole cluster
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= n_c) break;
                    float4* dst = reinterpret_cast<float4*>(
                        partial + ((c_lo + c) * 128 + quarter * 32 + lane) * kPartPitch);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        dst[j] = make_float4(sum[c][4 * j], sum[c][4 * j + 1], sum[c][4 * j + 2], sum[c][4 * j + 3]);
                }
                break;
            }
            if (!write) continue;
            const bool mend = fix[seq % kFixSlots] == tile + 1;
            const int id = mend && t0 + lane < a.m ? a.adapter_ids[t0 + lane] : -1;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int col0 = nt * bn + (c_lo + c) * 32;
                if (c >= n_c || col0 >= a.n) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // 16 rows at a time
                    if (lane >> 4 == half) {
                        float* row = buf + (lane & 15) * kPitch;
#pragma unroll
                        for (int j = 0; j < 32; ++j) row[j] = sum[c][j];
                        if (id >= 0)
                            for (int j = 0; j < 32; ++j)
                                if (col0 + j < a.n) row[j] += fix_up(a, t0 + lane, id, col0 + j);
                    }
                    __syncwarp();
                    store_chunk<16>(a, buf, t0 + half * 16, col0, lane);
                    __syncwarp();
                }
            }
        }
        __syncwarp();
        if (SPLIT) {
            warpgroup_sync(warp >> 2);
            registers_down<65536 / kThreads>();
        }
    }
    if (SPLIT) {
        __syncwarp();
        tc_fence_before_sync();
        __syncthreads();
        cluster_sync();
        wait_for_previous_kernel();
        const int tile = cluster, mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
        // columns 32 c of the tile, c = part, part + parts, ...: all pairs' partial
        // sums, in their order, 8 rows x 32 columns to a warp at a time
        const bool mend = fix[0] == tile + 1;
        const bool by_token = gathers(a, a.tile_count[mt]);
        float* buf = epi + warp * 8 * kPitch;
        static_assert(kEpiBytes >= kThreads / 32 * 8 * kPitch * 4, "a buffer per warp");
        if (!any_bad_tile(a, n_tiles / n_col_tiles, lane)) {
            const int mine = (bn / 32 - part + parts - 1) / parts;
#pragma unroll 1
            for (int u = warp; u < mine * 16; u += kThreads / 32) {
                const int c = part + (u >> 4) * parts, r0 = (u & 15) * 8, col0 = nt * bn + c * 32;
                const long long t0 = static_cast<long long>(mt) * 256 + rank * 128 + r0;
                if (col0 >= a.n || t0 >= a.m) continue;  // warp-uniform
                const int my_id = lane < 8 && t0 + lane < a.m ? a.adapter_ids[t0 + lane] : -1;
                float more[8];  // the adapters' part of column `lane` of the 8 rows
                if (by_token) gather_rows(a, more, t0, my_id, col0 + lane, lane);
                const uint32_t at = smem_u32(partial + (c * 128 + r0 + (lane >> 3)) * kPartPitch + (lane & 7) * 4);
                float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
                for (int q = 0; q < parts; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 x = ld_shared_cluster_f4(cluster_addr(at + i * 16 * kPartPitch, 2 * q + rank));
                        v[i].x += x.x;
                        v[i].y += x.y;
                        v[i].z += x.z;
                        v[i].w += x.w;
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float* dst = buf + (i * 4 + (lane >> 3)) * kPitch + (lane & 7) * 4;
                    dst[0] = v[i].x;
                    dst[1] = v[i].y;
                    dst[2] = v[i].z;
                    dst[3] = v[i].w;
                }
                __syncwarp();
                if (by_token) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) buf[r * kPitch + lane] += more[r];
                } else if (mend) {
                    for (int r = 0; r < 8; ++r) {
                        const int id = __shfl_sync(0xffffffffu, my_id, r);
                        if (id >= 0 && col0 + lane < a.n)
                            buf[r * kPitch + lane] += fix_up(a, t0 + r, id, col0 + lane);
                    }
                }
                __syncwarp();
                store_chunk<8>(a, buf, t0, col0, lane);
                __syncwarp();
            }
        }
    }
    // A CTA that gave up may have copies or MMAs in flight: let them land.
    if (*abort_flag && tid == 0) {
        const uint64_t start = global_timer_ns();
        while (global_timer_ns() - start < 1000000ull) {
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ shrink
// h[t] = scales[a] * (A[a] x[t]) for 128 tokens and `group` adapters at a time:
// M = 128 tokens, N = group x the rank rounded up to 16 (at most 128), one
// tcgen05 accumulator.  A token takes its own adapter's columns, the others are
// computed along and dropped.  grid: (token tiles x cluster, adapter lanes):
// lane j of L takes every L-th group of its tokens' adapters, the CTAs of a
// cluster split K and add their sums in rank order over
// distributed shared memory.  Reads x once from HBM (16384 tokens of 2048: 11
// us), where the projection then finds it in the L2.  Also writes the adapters
// of every 256-token row tile (their number is -1 where an id is out of range).
constexpr int kShrinkMaxStages = 10;
constexpr int kShrinkThreads = 256;
// Shared memory for `cols` columns (a multiple of 16): as many stages (16 KB of
// x, 128 bytes per adapter row) as fit beside the partial sums [128][cols + 1].
struct ShrinkSmem {
    int stage, stages, sums, total;  // bytes, except `stages`
};
__host__ __device__ inline ShrinkSmem shrink_smem(int cols) {
    ShrinkSmem s;
    s.stage = kHalf + cols * 128;
    s.sums = 128 * (cols + 1) * 4;
    s.stages = (225280 - s.sums) / s.stage;
    if (s.stages > kShrinkMaxStages) s.stages = kShrinkMaxStages;
    s.total = s.stages * s.stage + s.sums + 256 + 1024;
    return s;
}

// Distinct ids >= 0 of the first n threads' `id` (n a multiple of 32), in the
// order of their first thread, into list; returns their number in every thread.
// The block's threads all call it; ids: scratch of n ints, counts: of n / 32.
__device__ __forceinline__ int distinct_ids(int id, int n, int* ids, int* counts, int* list) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < n) ids[tid] = id;
    __syncthreads();
    const unsigned twins = __match_any_sync(0xffffffffu, id);  // every lane takes part
    bool opens = tid < n && id >= 0 && __ffs(twins) - 1 == lane;
    if (tid < n)
#pragma unroll 8
        for (int j = 0; j < warp * 8; ++j) {
            const int4 v = reinterpret_cast<const int4*>(ids)[j];
            opens = opens && v.x != id && v.y != id && v.z != id && v.w != id;
        }
    const unsigned ballot = __ballot_sync(0xffffffffu, opens);
    if (tid < n && lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < n / 32; ++w) {
        if (w < warp) before += counts[w];
        total += counts[w];
    }
    if (opens) list[before + __popc(ballot & lanemask_lt())] = id;
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kShrinkThreads, 1)
    lora_shrink_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                            const __grid_constant__ CUtensorMap map_a, const LoraArgs a, int split, int group) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int cols = group * a.r16, pitch = cols + 1;
    const ShrinkSmem lay = shrink_smem(cols);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.stages * lay.stage);
    uint64_t* empty = full + kShrinkMaxStages;
    uint64_t* acc_full = empty + kShrinkMaxStages;
    uint64_t* acc_empty = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* sums = reinterpret_cast<float*>(smem + lay.stages * lay.stage + 256);  // [128][pitch]
    __shared__ __align__(16) int s_id[kLoraTileRows];
    __shared__ int s_list[kLoraTileRows], s_count[kLoraTileRows / 32], s_bad;

    allow_next_kernel();  // it waits for this one's writes before it reads them
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % split, mt = static_cast<int>(blockIdx.x) / split;
    const long long t0 = static_cast<long long>(mt) * 128;
    if (tid == 0) {
        for (int s = 0; s < lay.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 4);  // the warps that read the accumulators
        *abort_flag = 0;
        s_bad = 0;
        fence_barrier_init();
        prefetch_tensormap(&map_x);
        prefetch_tensormap(&map_a);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, nullptr, a.wait_limit_ns};

    const auto id_of = [&](long long t) {
        const int id = t < a.m ? a.adapter_ids[t] : -1;
        if (id < -1 || id >= a.n_adapters) s_bad = 1;  // of the 256 tokens from t0 on
        return id < a.n_adapters ? id : -1;            // no adapter is read for it
    };
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *a.status = kDevOk;
    if (blockIdx.y == 0 && rank == 0 && mt % 2 == 0) {
        const int n = distinct_ids(id_of(t0 + tid), kLoraTileRows, s_id, s_count,
                                   a.tile_list + static_cast<size_t>(mt / 2) * kLoraTileRows);
        if (tid == 0) a.tile_count[mt / 2] = s_bad ? -1 : n;  // an id out of range in the tile
    }
    const int my_id = tid < 128 ? id_of(t0 + tid) : -1;
    const int n_list = distinct_ids(my_id, 128, s_id, s_count, s_list);  // s_id: the tile's ids

    const int nkb = (a.k + 63) / 64;
    const int kb_lo = nkb * rank / split, kb_hi = nkb * (rank + 1) / split;
    // Against the tensor core's truncation (see the projection), a round of up to
    // four accumulators of at most kChunk stages, and as many rounds as K takes.
    const int n_kb = kb_hi - kb_lo, rounds = (n_kb + 4 * kChunk - 1) / (4 * kChunk);
    const auto round_begin = [&](int round) { return kb_lo + n_kb * round / rounds; };
    const auto accumulators = [](int n) { return min((n + 7) / 8, 4); };
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    const auto advance = [&] {
        if (++stage == lay.stages) {
            stage = 0;
            phase ^= 1;
        }
    };
    // A CTA that gave up goes through the same cluster barriers as the others.
    for (int j = blockIdx.y * group; j < n_list; j += gridDim.y * group) {
        const int here = min(group, n_list - j);  // adapters of this pass
        const int* ads = s_list + j;
        if (warp == 0) {
            if (lane == 0)
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, ctl)) break;
                    uint8_t* sa = smem + stage * lay.stage;
                    mbar_arrive_expect_tx(&full[stage], kHalf + static_cast<uint32_t>(here * a.rank) * 128);
                    tma_load_2d(sa, &map_x, &full[stage], kb * 64, static_cast<int>(t0));
                    for (int g = 0; g < here; ++g)
                        tma_load_2d(sa + kHalf + g * a.r16 * 128, &map_a, &full[stage], kb * 64, ads[g] * a.rank);
                    advance();
                }
        } else if (warp == 1) {
            const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
            const uint32_t idesc = umma_idesc_bf16_f32(128, here * a.r16);
            const bool leader = elect_one();
            bool good = true;
            for (int round = 0; round < rounds && good; ++round) {
                const int lo = round_begin(round), n = round_begin(round + 1) - lo, n_sums = accumulators(n);
                good = __all_sync(0xffffffffu, mbar_wait(acc_empty, acc_phase ^ 1, ctl));
                if (!good) break;
                tc_fence_after_sync();
                int q = 0, next_q = 0;  // this stage's accumulator; the stage where it is the next one's turn
                for (int i = 0; i < n; ++i) {
                    good = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, ctl));
                    if (!good) break;
                    tc_fence_after_sync();
                    const uint64_t da = desc0 + static_cast<uint64_t>(stage * (lay.stage >> 4));
                    const bool first = i == next_q;
                    if (first) {
                        q = i * n_sums / n;
                        next_q = ((q + 1) * n + n_sums - 1) / n_sums;
                    }
                    if (leader) {
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4)
                            umma_bf16(tmem + q * MOE_MAX_LORA_RANK, da + k4 * 2, da + (kHalf >> 4) + k4 * 2, idesc,
                                      !first || k4 > 0);
                        umma_commit(&empty[stage]);
                    }
                    __syncwarp();
                    advance();
                }
                if (good && leader) umma_commit(acc_full);
                __syncwarp();
                acc_phase ^= 1;
            }
        } else if (warp >= 4) {
            for (int round = 0; round < rounds; ++round) {
                if (!__all_sync(0xffffffffu, mbar_wait(acc_full, acc_phase, ctl))) break;
                tc_fence_after_sync();
                const int n_sums = accumulators(round_begin(round + 1) - round_begin(round));
                for (int c = 0; c < (here * a.r16 + 31) / 32; ++c) {
                    float* row = sums + ((warp & 3) * 32 + lane) * pitch + c * 32;
                    float sum[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[i] = round > 0 && c * 32 + i < cols ? row[i] : 0.0f;
                    for (int q = 0; q < n_sums; ++q) {
                        uint32_t v[32];
                        tmem_load_32cols(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                                             q * MOE_MAX_LORA_RANK + c * 32, v);
                        tmem_load_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[i] += __uint_as_float(v[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + i < cols) row[i] = sum[i];
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
                acc_phase ^= 1;
            }
        }
        __syncwarp();
        if (split > 1)
            cluster_sync();
        else
            __syncthreads();
        // this CTA's rows of the tile: the partial sums of all CTAs, in rank order
        const int r_lo = 128 * rank / split, r_hi = 128 * (rank + 1) / split;
        for (int row = r_lo + warp; row < r_hi; row += kShrinkThreads / 32) {
            const int ad = s_id[row];
            int g = 0;
            while (g < here && ads[g] != ad) ++g;
            if (g == here) continue;
            const float scale = a.scales ? a.scales[ad] : 1.0f;
            for (int r = 2 * lane; r < a.r16; r += 64) {  // a pair of columns per lane
                float v[2] = {0.0f, 0.0f};
                if (r < a.rank) {  // even, as the rank is
                    const float* own = sums + row * pitch + g * a.r16 + r;
                    if (split > 1) {
                        const uint32_t at = smem_u32(own);
                        for (int q = 0; q < split; ++q) {
                            const uint32_t there = cluster_addr(at, q);
                            v[0] += ld_shared_cluster(there);
                            v[1] += ld_shared_cluster(there + 4);
                        }
                    } else {
                        v[0] = own[0];
                        v[1] = own[1];
                    }
                }
                __nv_bfloat16 p0[3], p1[3];
                split_bf16x3(v[0] * scale, p0);
                split_bf16x3(v[1] * scale, p1);
                __nv_bfloat16* dst = a.h_split + (t0 + row) * a.h_parts * a.r16 + r;
#pragma unroll
                for (int z = 0; z < 3; ++z)
                    if (z < a.h_parts)
                        *reinterpret_cast<__nv_bfloat162*>(dst + z * a.r16) = __nv_bfloat162(p0[z], p1[z]);
            }
        }
        // the sums are read (the lanes took different shares of the columns: a
        // cluster barrier wants the warp together again)
        __syncwarp();
        if (split > 1)
            cluster_sync();
        else
            __syncthreads();
        tc_fence_after_sync();
    }
    if (*abort_flag && tid == 0) {
        set_status(a.status, kDevTimeout);
        const uint64_t start = global_timer_ns();  // copies in flight land
        while (global_timer_ns() - start < 1000000ull) {
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_lora_shrink_gemm(const LoraArgs& a, const CUtensorMap& map_x, const CUtensorMap& map_a,
                                    cudaStream_t stream) {
    static PerDeviceOnce once;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_shrink_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    225280 + 256 + 1024);
    });
    if (err != cudaSuccess) return err;
    // K split over as many CTAs (1 to 8, at least four stages each) as 148 SMs
    // hold once, then adapter lanes for what is left of them; a second lane in
    // any case, for the tiles in which one request ends and another begins
    const long long tiles = (a.m + 127) / 128;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 148 && (a.k + 63) / 64 >= split * 8) split *= 2;
    const long long rest = 148 / (tiles * split);
    // Adapters of a pass: up to 128 columns for small batches, whose tokens may
    // all have adapters of their own, up to 64 for large ones, whose ring then
    // is deeper.  (4096 x 4096, rank 16, 256 requests: 2048 tokens 172 us with one
    // adapter a pass, 117 with eight; 8192 tokens 294, 258 with four, 270 with
    // eight; with 4 requests 202, 205 and 209.)
    const int group = std::max(1, (tiles <= 16 ? 128 : 64) / a.r16);
    const unsigned lanes = static_cast<unsigned>(rest < 2 ? 2 : rest > 128 ? 128 : rest);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), lanes);
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = shrink_smem(group * a.r16).total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_shrink_gemm_kernel, map_x, map_a, a, split, group);
}

template <bool SPLIT>
static cudaError_t launch_gemm(const LoraArgs& a, const CUtensorMap& map_x, const CUtensorMap& map_w, int bn,
                               int split, int num_sms, cudaStream_t stream) {
    static PerDeviceOnce once;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_gemm_kernel<SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemLimit);
    });
    if (err != cudaSuccess) return err;
    const long long n_col = (a.n + bn - 1) / bn, tiles = (a.m + 255) / 256 * n_col;
    const long long clusters = SPLIT || tiles < num_sms / 2 ? tiles : num_sms / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * split * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (ring_stages(bn) + kExt) * stage_bytes(bn) + kTail;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_gemm_kernel<SPLIT>, map_x, map_w, a, bn, static_cast<int>(n_col),
                              static_cast<int>(tiles), split);
}

cudaError_t launch_lora_gemm(const LoraArgs& a, const CUtensorMap& map_x, const CUtensorMap& map_w, int bn,
                             int split, int num_sms, cudaStream_t stream) {
    // one row tile: a decode batch, whose tokens may all have adapters of their
    // own (100 tokens of 512 x 512 with 64 adapters of rank 128: 217 -> 127 us;
    // without adapters 12.4 -> 14.4)
    const bool join = split > 1 || (a.m <= kLoraTileRows && (a.n + bn - 1) / bn <= num_sms / 2);
    return join ? launch_gemm<true>(a, map_x, map_w, bn, split, num_sms, stream)
                : launch_gemm<false>(a, map_x, map_w, bn, 1, num_sms, stream);
}

}  // namespace moe

// The projection with adapters for larger batches, in one tcgen05 GEMM:
//   y[t] = W x[t] + B[a] (scales[a] h[t]),  a = adapter_ids[t],
// with h = A x and its scaling from the shrink kernel, as two bf16 parts (hi,
// lo: 16 significant bits).
//
// A CTA pair owns a tile of 256 tokens x `bn` output columns (M = 256, N = bn
// MMAs over both CTAs; each CTA loads its 128 tokens and its half of W's rows,
// 128 bytes of K per stage).  The adapters enter as more columns of K behind
// the projection's: for every adapter that occurs among the tile's tokens, its
// rank columns (rounded up to 16) twice, against the hi and the lo part of h,
// which are zero for the tokens of other adapters.  So they cost 2 * rank / k of
// the projection's MMAs per adapter of a tile, and no pass over y.
//
// A zero times NaN or infinity is NaN, so a piece of B that is not finite never
// reaches the tensor core: its writer replaces it by zeros and marks the tile,
// and the epilogue adds the piece's products for the tokens that do use it.
//
// Warps per CTA: 0 copies the tiles (TMA), 1 issues the MMAs (leader CTA only),
// 4-7 epilogue, 8-11 write the adapters' stages.  Two accumulators let the
// epilogue of a tile overlap the next tile's MMAs.  Every wait is bounded.
#include "launch.h"
#include "pair_mma.cuh"

namespace moe {
namespace {

constexpr int kStages = 6;
constexpr int kHalf = 128 * 128;      // bytes of 128 rows x 64 columns
constexpr int kStage = 2 * kHalf;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kFixSlots = 16;
constexpr int kPitch = 33;            // words of a staged epilogue row
constexpr int kEpiBytes = 4 * 32 * kPitch * 4;
constexpr int kSmem = kStages * kStage + kEpiBytes + 512 + kLoraTileRows * 4 + 1024;

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

// Products of the pieces of B[adapter] row `col` that are not finite.
__device__ __noinline__ float fix_up(const LoraArgs& a, long long t, int id, int col) {
    const __nv_bfloat16* b = a.B + (static_cast<size_t>(id) * a.n + col) * a.rank;
    const __nv_bfloat16* h = a.h_split + static_cast<size_t>(t) * 2 * a.r16;
    float s = 0.0f;
    for (int r = 0; r < a.rank; r += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(b + r);
        if (!not_finite_bf16x8(v)) continue;
        float bf[8];
        bf16x8_to_f32(v, bf);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s += bf[e] * (__bfloat162float(h[r + e]) + __bfloat162float(h[a.r16 + r + e]));
    }
    return s;
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    lora_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const LoraArgs a, int bn, int n_col_tiles, int n_tiles) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStage + kEpiBytes);  // leader's are used
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;   // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2], leader's are used
    uint64_t* grant = acc_empty + 2;        // [kStages] an empty stage handed to the adapters' writers
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(grant + kStages);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // Tiles (1 + index) that hold a piece of B which is not finite, at the
    // tile's place in this pair's sequence modulo kFixSlots.  The writers are
    // at most kStages stages and two accumulators ahead of the epilogue.
    volatile int* fix = reinterpret_cast<volatile int*>(tmem_slot + 2);
    int* list = const_cast<int*>(fix) + kFixSlots;  // [kLoraTileRows] the tile's adapters
    float* epi = reinterpret_cast<float*>(smem + kStages * kStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);   // both by the leader's copies, or one by each CTA's adapter writers
            mbar_init(&empty[s], 1);
            mbar_init(&grant[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);  // the epilogue warps of both CTAs
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

    const int cluster = blockIdx.x / 2, n_clusters = gridDim.x / 2;
    const int nk = (a.k + 63) / 64;
    const int half = bn / 2;
    // stages of the adapters' columns of row tile mt (the shrink kernel has run)
    const auto ext_steps = [&](int mt) { return a.tile_count[mt] * 2 * (a.r16 / 16); };  // MMA steps of 16
    const auto advance = [](int& stage, uint32_t& phase, int by) {
        stage += by;
        phase ^= static_cast<uint32_t>(stage / kStages) & 1u;
        stage %= kStages;
    };

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
                    const uint32_t bar = cluster_addr(smem_u32(&full[stage]), 0);
                    uint8_t* sa = smem + stage * kStage;
                    if (rank == 0) {  // for both CTAs' copies; the stage's second arrival too
                        mbar_arrive_expect_tx(&full[stage], 2 * (kHalf + half * 128));
                        mbar_arrive(&full[stage]);
                    }
                    tma_load_2d_pair(sa, &map_x, bar, kb * 64, mt * 256 + static_cast<int>(rank) * 128);
                    tma_load_2d_pair(sa + kHalf, &map_w, bar, kb * 64, nt * bn + static_cast<int>(rank) * half);
                    advance(stage, phase, 1);
                }
                if (!good) break;
                // This thread alone follows every phase of `empty` (a parity
                // names a phase only to a waiter that is at most one behind);
                // it hands the adapters' stages to their writers.
                wait_for_previous_kernel();
                for (int e = (ext_steps(mt) + 3) / 4; e > 0; --e) {
                    if (!(good = mbar_wait_cluster(&empty[stage], phase ^ 1, ctl))) break;
                    mbar_arrive(&grant[stage]);
                    advance(stage, phase, 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (rank == 0 && lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            // instruction descriptor: M = 256, N = bn
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                   (static_cast<uint32_t>(bn >> 3) << 17) | ((256u >> 4) << 24);
            bool good = true;
            for (int tile = cluster; tile < n_tiles && good; tile += n_clusters) {
                if (!(good = mbar_wait_cluster(&acc_empty[acc], acc_phase ^ 1, ctl))) break;
                tc_fence_after_sync();
                const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
                int steps = nk * 4, ext = -1;
                for (int done = 0; done < steps || ext < 0;) {
                    if (done == steps) {  // the projection is issued; now the adapters
                        wait_for_previous_kernel();
                        ext = ext_steps(tile / n_col_tiles);
                        steps += ext;
                        continue;
                    }
                    if (!(good = mbar_wait_cluster(&full[stage], phase, ctl))) break;
                    tc_fence_after_sync();
                    const uint32_t sa = smem_u32(smem + stage * kStage);
                    const int here = min(4, steps - done);
                    for (int k4 = 0; k4 < here; ++k4)
                        umma_bf16_pair(d, sw128_kmajor_desc(sa + k4 * 32),
                                       sw128_kmajor_desc(sa + kHalf + k4 * 32), idesc, (done + k4) != 0);
                    umma_commit_pair(&empty[stage]);
                    done += here;
                    advance(stage, phase, 1);
                }
                if (!good) break;
                umma_commit_pair(&acc_full[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ------------------------------------------------------ adapters' stages
        wait_for_previous_kernel();
        // Two stages of copies are in flight before the first is handed on, so a
        // tile with many adapters does not wait for each copy's latency.
        const int row = tid - 256;  // 0..127: this CTA's token row and its W row of the tile
        const uint32_t ext = smem_u32(smem) + static_cast<uint32_t>(row * 128);
        const auto piece_at = [&](int p) { return static_cast<uint32_t>((p ^ (row & 7)) << 4); };
        int stage = 0, seq = 0;
        uint32_t granted = 0;  // bit s: parity of grant[s]'s next phase
        bool good = true;
        for (int tile = cluster; tile < n_tiles && good; tile += n_clusters, ++seq) {
            const int mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
            stage = (stage + nk) % kStages;
            const int count = a.tile_count[mt];
            all_of_four_warps(true);  // the last tile's list is read
            for (int i = row; i < count; i += 128)
                list[i] = a.tile_list[static_cast<size_t>(mt) * kLoraTileRows + i];
            all_of_four_warps(true);
            const long long t = static_cast<long long>(mt) * 256 + rank * 128 + row;
            const int id = t < a.m ? a.adapter_ids[t] : -1;
            const int col = nt * bn + static_cast<int>(rank) * half + row;
            const bool col_in = row < half && col < a.n;
            const __nv_bfloat16* h_row = a.h_split + (t < a.m ? t : 0) * 2 * a.r16;
            const __nv_bfloat16* b_row = a.B + static_cast<size_t>(col_in ? col : 0) * a.rank;
            const size_t b_adapter = static_cast<size_t>(a.n) * a.rank;
            const int cols = count * 2 * a.r16;

            // Hands stage `st` on: its copies have landed; pieces of B that are
            // not finite become zeros (the epilogue adds their products).
            const auto hand_on = [&](int st) {
                bool bad = false;
                if (row < half) {
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        uint4* at = reinterpret_cast<uint4*>(smem + st * kStage + kHalf + row * 128 + piece_at(p));
                        if (not_finite_bf16x8(*at)) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            bad = true;
                        }
                    }
                }
                if (bad) {
                    const uint32_t at = smem_u32(const_cast<int*>(&fix[seq % kFixSlots]));
                    st_shared_cluster(cluster_addr(at, 0), tile + 1);
                    st_shared_cluster(cluster_addr(at, 1), tile + 1);
                }
                fence_proxy_async_smem();
                all_of_four_warps(true);
                if (row == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&full[st]), 0));
            };
            int ad = 0, rem = 0;       // adapter of the list and column within its 2 * r16
            int older = -1, newer = -1;  // stages whose copies are in flight
            for (int c0 = 0; c0 < cols; c0 += 64) {
                good = all_of_four_warps(mbar_wait(&grant[stage], granted >> stage & 1u, ctl));
                if (!good) break;
                granted ^= 1u << stage;
                const uint32_t sa = ext + static_cast<uint32_t>(stage * kStage);
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const bool in = ad < count;
                    const int adapter = in ? list[ad] : 0;
                    const int r = rem < a.r16 ? rem : rem - a.r16;
                    const bool use_a = in && adapter == id, use_b = in && col_in && r < a.rank;
                    cp_async_16(sa + piece_at(p), use_a ? h_row + rem : a.h_split, use_a ? 16u : 0u);
                    if (row < half)
                        cp_async_16(sa + kHalf + piece_at(p), use_b ? b_row + adapter * b_adapter + r : a.B,
                                    use_b ? 16u : 0u);
                    rem += 8;
                    if (rem == 2 * a.r16) {
                        rem = 0;
                        ++ad;
                    }
                }
                cp_async_commit();
                if (older >= 0) {
                    cp_async_wait_group<2>();
                    hand_on(older);
                }
                older = newer;
                newer = stage;
                stage = (stage + 1) % kStages;
            }
            if (good && older >= 0) {
                cp_async_wait_group<1>();
                hand_on(older);
            }
            if (good && newer >= 0) {
                cp_async_wait_group<0>();
                hand_on(newer);
            }
        }
        cp_async_wait_all();
    } else if (warp >= 4) {
        // ------------------------------------------------------ epilogue
        wait_for_previous_kernel();
        const bool write = *a.status == kDevOk;
        const int quarter = warp & 3;
        float* buf = epi + quarter * 32 * kPitch;
        int acc = 0, seq = 0;
        uint32_t acc_phase = 0;
        for (int tile = cluster; tile < n_tiles; tile += n_clusters, ++seq) {
            const int mt = tile / n_col_tiles, nt = tile - mt * n_col_tiles;
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[acc], acc_phase, ctl))) break;
            tc_fence_after_sync();
            const long long t0 = static_cast<long long>(mt) * 256 + rank * 128 + quarter * 32;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * 256);
            const bool mend = write && fix[seq % kFixSlots] == tile + 1;
            const int id = mend && t0 + lane < a.m ? a.adapter_ids[t0 + lane] : -1;
#pragma unroll 1
            for (int c = 0; c < bn / 32; ++c) {
                const int col0 = nt * bn + c * 32;
                if (col0 >= a.n) break;
                uint32_t v[32];
                tmem_load_32cols(taddr + c * 32, v);
                tmem_load_wait();
                if (mend && id >= 0)
                    for (int j = 0; j < 32; ++j)
                        if (col0 + j < a.n)
                            v[j] = __float_as_uint(__uint_as_float(v[j]) + fix_up(a, t0 + lane, id, col0 + j));
#pragma unroll
                for (int j = 0; j < 32; ++j) buf[lane * kPitch + j] = __uint_as_float(v[j]);
                __syncwarp();
                if (a.y_dtype == MOE_DTYPE_BF16) {
                    // 8 columns per lane: 8 rows x 64 bytes per instruction
                    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
                    const int cc = (lane & 3) * 8, col = col0 + cc;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = i * 8 + (lane >> 2);
                        if (!write || t0 + r >= a.m || col >= a.n) continue;
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
                    for (int i = 0; i < 8; ++i) {
                        const int r = i * 4 + (lane >> 3);
                        if (!write || t0 + r >= a.m || col >= a.n) continue;
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
                __syncwarp();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[acc]), 0));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
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

}  // namespace

cudaError_t launch_lora_gemm(const LoraArgs& a, const CUtensorMap& map_x, const CUtensorMap& map_w, int bn,
                             int num_sms, cudaStream_t stream) {
    static PerDeviceOnce once;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (err != cudaSuccess) return err;
    const long long n_col = (a.n + bn - 1) / bn, tiles = (a.m + 255) / 256 * n_col;
    const long long pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_gemm_kernel, map_x, map_w, a, bn, static_cast<int>(n_col),
                              static_cast<int>(tiles));
}

}  // namespace moe

// A projection that all tokens share, with the low-rank adapter of each
// token's own request beside it:
//   y[t] = W x[t] + scales[a] * B[a] (A[a] x[t]),   a = adapter_ids[t]
// (a = -1: the projection alone).
//
// m <= 32, here:
// Kernel 1 (shrink): h[t] = A[a] x[t], one adapter of the call's at a time;
//   only its own tokens' rows of x are read.  The tokens are the rows of the
//   MMA (stream_mma.cuh, with x in the place of the weights), the adapter's
//   rank its columns; rows of other tokens are dropped by selection, never by a
//   multiplication with zero, so an adapter that holds NaN or infinities
//   reaches its own requests only.
// Kernel 2 streams W once through mma.sync (stream_mma.cuh) and adds scales[a]
//   * B[a] h in its epilogue.  It starts beside kernel 1 and waits for it only
//   before that epilogue.
// Bound: reading W (4096 x 4096: 5.2 us at the copy rate) and the launches of
// two kernels; 1 token of 8 adapters of rank 16 takes 15 us, 32 tokens of 64
// adapters 21.5 us (graph replays).
// Larger m: the two tcgen05 kernels of lora_gemm.cu.
#include <algorithm>

#include "launch.h"
#include "stream_mma.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKb = 64;       // K columns of one warp step
constexpr int kTileN = 32;    // output columns of a streaming tile

// ------------------------------------------------------------------ shrink
// grid: (rank tiles x adapter lanes, K ranges).  A block's warps split its K
// range of an adapter and add their sums in the order of K.  Adapter lane j of
// L takes every L-th adapter of the tokens.  The f32 sums of K range z go to h
// + z * m * rank; the reader adds the ranges in order.
constexpr int kShrinkStages = 3;

template <int NT>  // NT: groups of 8 rank rows per block
__global__ void __launch_bounds__(kThreads, 1)
    lora_shrink_kernel(const LoraArgs a, int rank_tiles) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    allow_next_kernel();  // it waits for this one's writes before it reads them
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2;
    int my_id = lane < a.m ? a.adapter_ids[lane] : -1;
    if (my_id >= a.n_adapters) my_id = -1;  // the next kernel reports it; no adapter is read for it
    // lanes that open an adapter: the first token of each distinct id
    const unsigned same = __match_any_sync(0xffffffffu, my_id);
    unsigned leaders = __ballot_sync(0xffffffffu, my_id >= 0 && (__ffs(same) - 1) == lane);
    const int adapter_lanes = gridDim.x / rank_tiles, my_lane = blockIdx.x / rank_tiles;
    const int r0 = static_cast<int>(blockIdx.x % rank_tiles) * NT * 8;
    const int nr = min(NT * 8, a.rank - r0), nt = (nr + 7) >> 3;
    const int nkb = (a.k + kKb - 1) / kKb, shares = kWarps * gridDim.y, share = blockIdx.y * kWarps + warp;
    const int k_lo = static_cast<int>(static_cast<long long>(nkb) * share / shares) * kKb;
    const int k_hi = min(a.k, static_cast<int>(static_cast<long long>(nkb) * (share + 1) / shares) * kKb);
    unsigned char* ring_mem = smem_raw + warp * kShrinkStages * kRingBytes;
    const uint32_t ring = smem_u32(ring_mem);
    static_assert(kShrinkStages * kRingBytes >= 2 * NT * 4 * 32 * 4, "partial sums lie in the ring");
    for (int j = 0; leaders; ++j) {
        const int lead = __ffs(leaders) - 1;
        leaders &= leaders - 1;
        if (j % adapter_lanes != my_lane) continue;
        const int ad = __shfl_sync(0xffffffffu, my_id, lead);
        const unsigned mine = __ballot_sync(0xffffffffu, my_id == ad);  // tokens of this adapter
        const __nv_bfloat16* A = a.A + (static_cast<size_t>(ad) * a.rank + r0) * a.k;
        const __nv_bfloat16* tok[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) tok[n] = A + static_cast<size_t>(min(n * 8 + g, nr - 1)) * a.k;
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
        const auto row = [&](int r) -> const __nv_bfloat16* {
            return mine >> r & 1u ? a.x + static_cast<size_t>(r) * a.k : nullptr;
        };
        int fill_k = k_lo, fill_slot = 0, use_slot = 0;
        const auto fill = [&] {
            if (fill_k < k_hi) ring_fill<false>(ring + fill_slot * kRingBytes, row, fill_k, a.k, lane);
            fill_k += kKb;
            cp_async_commit();
            fill_slot = fill_slot + 1 == kShrinkStages ? 0 : fill_slot + 1;
        };
        for (int i = 0; i < kShrinkStages - 1; ++i) fill();
        for (int k0 = k_lo; k0 < k_hi; k0 += kKb) {
            const uint32_t slot = ring + use_slot * kRingBytes;
            ring_multiply<false, NT, 1>(acc, slot, tok, nt, k0, a.k, lane, [&] {
                cp_async_wait_group<kShrinkStages - 2>();
                __syncwarp();
                fill();
            });
            use_slot = use_slot + 1 == kShrinkStages ? 0 : use_slot + 1;
        }
        // the block's warps add their partial sums, in the order of K; element
        // (h, n, e): token h * 16 + (e / 2) * 8 + g, rank row n * 8 + 2 c + e % 2
        cp_async_wait_group<0>();
        __syncwarp();
        float* own = reinterpret_cast<float*>(ring_mem);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) own[((h * NT + n) * 4 + e) * 32 + lane] = acc[h][n][e];
        __syncthreads();
        const float* parts = reinterpret_cast<const float*>(smem_raw);
        constexpr int kPart = kShrinkStages * kRingBytes / 4;
        for (int u = tid; u < 2 * NT * 4 * 32; u += kThreads) {
            const int l = u & 31, hne = u >> 5, e = hne & 3, n = (hne >> 2) % NT, h = (hne >> 2) / NT;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += parts[w * kPart + u];
            const int token = h * 16 + (e >> 1) * 8 + (l >> 2), r = n * 8 + (l & 3) * 2 + (e & 1);
            if ((mine >> token & 1u) && r < nr) a.h[(blockIdx.y * a.m + token) * a.rank + r0 + r] = v;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void store_y(void* y, int y_dtype, size_t at, float v) {
    if (y_dtype == MOE_DTYPE_BF16)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[at] = v;
}

// scale * (B row . h row) for one (token, output column); h in shared or
// global memory (f32), B row of `rank` bf16.
__device__ __forceinline__ float expand_dot(const __nv_bfloat16* __restrict__ b_row, const float* h,
                                            int rank) {
    float s = 0.0f;
    for (int r = 0; r < rank; r += 8) {
        float bf[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(b_row + r), bf);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(bf[e], h[r + e], s);
    }
    return s;
}

// ------------------------------------------------------- streaming (m <= 32)
// Every block takes an equal share of the output columns, 32 rows of W at a
// time; its 16 warps split K, each through its own ring (stream_mma.cuh), and
// add their sums in shared memory.  Only the adapters' part waits for the shrink
// kernel, so W is on its way while that one runs.  Bound by reading W.
constexpr int kStreamStages = 3;

template <int NT>
struct StreamSmem {
    unsigned char ring[kWarps][kStreamStages][kRingBytes];  // then the warps' sums
    float h[8 * NT][MOE_MAX_LORA_RANK + 1];
    int id[32], bad;
    float scale[32];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) lora_stream_kernel(const LoraArgs a) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    StreamSmem<NT>& sm = *reinterpret_cast<StreamSmem<NT>*>(smem_raw);
    static_assert(sizeof(sm.ring) >= sizeof(float) * kWarps * 2 * NT * 4 * 32, "sums lie in the ring");
    float(*red)[2 * NT * 4][32] = reinterpret_cast<float(*)[2 * NT * 4][32]>(&sm.ring[0][0][0]);  // [kWarps]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2;
    const int m = static_cast<int>(a.m), nt = (m + 7) >> 3;
    const int lo = static_cast<int>(static_cast<long long>(a.n) * blockIdx.x / gridDim.x);
    const int hi = static_cast<int>(static_cast<long long>(a.n) * (blockIdx.x + 1) / gridDim.x);
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0]);
    const __nv_bfloat16* tok[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) tok[n] = a.x + static_cast<size_t>(min(n * 8 + g, m - 1)) * a.k;

    int fill_k = 0, fill_slot = 0, use_slot = 0;
    for (int n0 = lo; n0 < hi; n0 += kTileN) {
        const int nn = min(kTileN, hi - n0);
        const __nv_bfloat16* w = a.W + static_cast<size_t>(n0) * a.k;
        const bool wide = nn <= 16;
        const int step = wide ? 128 : 64;
        const auto row = [&](int r) { return r < nn ? w + static_cast<size_t>(r) * a.k : nullptr; };
        const auto fill = [&] {
            if (fill_k < a.k) {
                if (wide)
                    ring_fill<true>(ring + fill_slot * kRingBytes, row, fill_k, a.k, lane);
                else
                    ring_fill<false>(ring + fill_slot * kRingBytes, row, fill_k, a.k, lane);
            }
            fill_k += kWarps * step;
            cp_async_commit();
            fill_slot = fill_slot + 1 == kStreamStages ? 0 : fill_slot + 1;
        };
        fill_k = warp * step;
        fill_slot = use_slot = 0;
        for (int i = 0; i < kStreamStages - 1; ++i) fill();
        if (n0 == lo) {
            // the ids, while the first weights are on their way: any outside
            // [-1, n_adapters) and the call does nothing
            if (warp == 0) {
                const int id = lane < m ? a.adapter_ids[lane] : -1;
                const bool bad = __any_sync(0xffffffffu, id < -1 || id >= a.n_adapters);
                sm.id[lane] = id;
                sm.scale[lane] = !bad && id >= 0 && a.scales ? a.scales[id] : 1.0f;
                if (lane == 0) {
                    sm.bad = bad;
                    if (blockIdx.x == 0) *a.status = bad ? kDevBadId : kDevOk;
                }
            }
            __syncthreads();
            if (sm.bad) break;
        }
        // the adapters' rows of this tile, into the L2
        for (int u = tid; u < m * kTileN; u += kThreads) {
            const int r = u % kTileN, id = sm.id[u / kTileN];
            if (r < nn && id >= 0)
                prefetch_l2(a.B + (static_cast<size_t>(id) * a.n + n0 + r) * a.rank);
        }
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
        for (int k0 = warp * step; k0 < a.k; k0 += kWarps * step) {
            const uint32_t slot = ring + use_slot * kRingBytes;
            const auto ready = [&] {
                cp_async_wait_group<kStreamStages - 2>();
                __syncwarp();
                fill();
            };
            if (wide)
                ring_multiply<true, NT, 1>(acc, slot, tok, nt, k0, a.k, lane, ready);
            else
                ring_multiply<false, NT, 1>(acc, slot, tok, nt, k0, a.k, lane, ready);
            use_slot = use_slot + 1 == kStreamStages ? 0 : use_slot + 1;
        }
        if (n0 == lo) {
            wait_for_previous_kernel();
            for (int u = tid; u < m * a.rank; u += kThreads) {
                float s = a.h[u];
                for (int z = 1; z < a.k_splits; ++z) s += a.h[static_cast<size_t>(z) * m * a.rank + u];
                sm.h[u / a.rank][u % a.rank] = s;
            }
        }
        cp_async_wait_group<0>();
        __syncthreads();  // the ring is used up
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) red[warp][(h * NT + n) * 4 + e][lane] = acc[h][n][e];
        __syncthreads();
        // lane = output column of the tile, so that stores are contiguous
        for (int u = tid; u < m * kTileN; u += kThreads) {
            const int r = u % kTileN, t = u / kTileN;
            if (r >= nn) continue;
            const int hne = ((r >> 4) * NT + (t >> 3)) * 4 + ((r >> 3) & 1) * 2 + (t & 1);
            const int l = (r & 7) * 4 + ((t & 7) >> 1);
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += red[q][hne][l];
            const int id = sm.id[t];
            if (id >= 0)
                v += sm.scale[t] * expand_dot(a.B + (static_cast<size_t>(id) * a.n + n0 + r) * a.rank,
                                              sm.h[t], a.rank);
            store_y(a.y, a.y_dtype, static_cast<size_t>(t) * a.n + n0 + r, v);
        }
        __syncthreads();
    }
    // after a bad id: copies in flight, and this kernel must not end before the
    // one whose memory the stream's next kernel may write
    cp_async_wait_all();
    wait_for_previous_kernel();
}

template <int NT>
cudaError_t launch_stream(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    static PerDeviceOnce once;
    constexpr int smem = sizeof(StreamSmem<NT>);
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_stream_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.n < num_sms ? a.n : num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_stream_kernel<NT>, a);
}

}  // namespace

template <int NT>
static cudaError_t launch_shrink(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    static PerDeviceOnce once;
    constexpr int smem = kWarps * kShrinkStages * kRingBytes;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_shrink_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err != cudaSuccess) return err;
    const int rank_tiles = (a.rank + NT * 8 - 1) / (NT * 8);
    // a block per adapter and K range while that fills the SMs once
    const int fit = num_sms / (rank_tiles * a.k_splits), lanes = std::max(1, std::min(fit, static_cast<int>(a.m)));
    lora_shrink_kernel<NT><<<dim3(rank_tiles * lanes, a.k_splits), kThreads, smem, stream>>>(a, rank_tiles);
    return cudaGetLastError();
}

cudaError_t launch_lora_shrink(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    // 16 rank rows per block: a request's adapter then reaches several SMs (whole
    // call, k = n = 4096, rank 128, 1 token: 14.4 us, 14.6 with 32 rows and 22.7
    // with 64; 32 tokens of one adapter 30.8, 32.9 and 49; of 32 adapters 42.5,
    // 40.3 and 61.6)
    return a.rank <= 8 ? launch_shrink<1>(a, num_sms, stream) : launch_shrink<2>(a, num_sms, stream);
}

cudaError_t launch_lora_stream(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    if (a.m <= 8) return launch_stream<1>(a, num_sms, stream);
    if (a.m <= 16) return launch_stream<2>(a, num_sms, stream);
    return launch_stream<4>(a, num_sms, stream);
}

}  // namespace moe

// A projection that all tokens share, with the low-rank adapter of each
// token's own request beside it:
//   y[t] = W x[t] + scales[a] * B[a] (A[a] x[t]),   a = adapter_ids[t]
// (a = -1: the projection alone).
//
// Kernel 1 (shrink): h[t] = A[a] x[t], f32 [m, rank].  A block takes 32
//   consecutive tokens and walks the adapters that occur among them; the
//   tokens of another adapter ride along in the MMA's unused columns and are
//   dropped by selection, never by a multiplication with zero, so an adapter
//   that holds NaN or infinities reaches its own requests only.
// Kernel 2, m <= 64: streams W once through mma.sync (stream_mma.cuh) and
//   adds scales[a] * B[a] h in its epilogue.
// Kernel 2, larger m: the tcgen05 GEMM of lora_gemm.cu.
#include "launch.h"
#include "stream_mma.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKb = 64;       // K columns of one warp step
constexpr int kGroup = 32;    // tokens per shrink block
constexpr int kRankTile = 32; // adapter rows per shrink block
constexpr int kTileN = 32;    // output columns of a streaming tile

// ------------------------------------------------------------------ shrink
// grid: (token groups, rank tiles x adapter lanes, K ranges).  Adapter lane j
// of L takes every L-th adapter of its tokens.  The streaming kernel gets the
// f32 sums, K range z at h + z * m * rank (it adds the ranges in order); the
// GEMM gets them scaled and split into two bf16 parts, with the list of the
// adapters that occur in each of its row tiles.
template <bool GEMM>
__global__ void __launch_bounds__(kThreads, 1) lora_shrink_kernel(const LoraArgs a, int rank_tiles) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float(*red)[2 * 4 * 4][32] = reinterpret_cast<float(*)[2 * 4 * 4][32]>(smem_raw);  // [kWarps]
    __shared__ __align__(16) int s_id[kGroup];
    __shared__ __align__(16) int s_tile[kLoraTileRows];
    __shared__ int s_count[kLoraTileRows / 32];
    __shared__ int s_bad;
    allow_next_kernel();  // it waits for this one's writes before it reads them
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c8 = (lane & 3) * 8;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        // the call's status word: any adapter id outside [-1, n_adapters)
        if (tid == 0) s_bad = 0;
        __syncthreads();
        bool bad = false;
        for (long long t = tid; t < a.m; t += kThreads) {
            const int id = a.adapter_ids[t];
            bad |= id < -1 || id >= a.n_adapters;
        }
        if (bad) s_bad = 1;
        __syncthreads();
        if (tid == 0) *a.status = s_bad ? kDevBadId : kDevOk;
    }
    if (GEMM && blockIdx.y == 0 && blockIdx.x % (kLoraTileRows / kGroup) == 0) {
        // the adapters of this block's row tile, in order of their first token
        const long long first = static_cast<long long>(blockIdx.x) * kGroup;
        int id = -1;
        if (tid < kLoraTileRows) {
            if (first + tid < a.m) id = a.adapter_ids[first + tid];
            if (id >= a.n_adapters) id = -1;
            s_tile[tid] = id;
        }
        __syncthreads();
        bool opens = false;
        unsigned ballot = 0;
        if (tid < kLoraTileRows) {
            const unsigned twins = __match_any_sync(0xffffffffu, id);  // every lane takes part
            opens = id >= 0 && __ffs(twins) - 1 == lane;
            for (int j = 0; j < warp * 8; ++j) {
                const int4 v = reinterpret_cast<const int4*>(s_tile)[j];
                opens = opens && v.x != id && v.y != id && v.z != id && v.w != id;
            }
            ballot = __ballot_sync(0xffffffffu, opens);
            if (lane == 0) s_count[warp] = __popc(ballot);
        }
        __syncthreads();
        const int mt = static_cast<int>(first / kLoraTileRows);
        if (tid < kLoraTileRows) {
            int before = 0, total = 0;
            for (int w = 0; w < kLoraTileRows / 32; ++w) {
                if (w < warp) before += s_count[w];
                total += s_count[w];
            }
            if (opens)
                a.tile_list[static_cast<size_t>(mt) * kLoraTileRows + before + __popc(ballot & lanemask_lt())] = id;
            if (tid == 0) a.tile_count[mt] = total;
        }
    }
    const long long t0 = static_cast<long long>(blockIdx.x) * kGroup;
    const int nt_here = static_cast<int>(min(static_cast<long long>(kGroup), a.m - t0));
    if (tid < kGroup) {
        int id = tid < nt_here ? a.adapter_ids[t0 + tid] : -1;
        if (id >= a.n_adapters) id = -1;  // reported above; no adapter is read for it
        s_id[tid] = id;
    }
    __syncthreads();
    const int my_id = s_id[lane];
    // lanes that open an adapter: the first token of each distinct id
    const unsigned same = __match_any_sync(0xffffffffu, my_id);
    unsigned leaders = __ballot_sync(0xffffffffu, my_id >= 0 && (__ffs(same) - 1) == lane);
    const int adapter_lanes = gridDim.y / rank_tiles, my_lane = blockIdx.y / rank_tiles;
    const int r0 = static_cast<int>(blockIdx.y % rank_tiles) * kRankTile;
    const int nr = min(kRankTile, a.rank - r0);
    const int nkb_all = (a.k + kKb - 1) / kKb;
    const int kb_lo = static_cast<int>(static_cast<long long>(nkb_all) * blockIdx.z / gridDim.z);
    const int kb_hi = static_cast<int>(static_cast<long long>(nkb_all) * (blockIdx.z + 1) / gridDim.z);
    float* h_out = a.h + static_cast<size_t>(blockIdx.z) * a.m * a.rank;
    for (int j = 0; leaders; ++j) {
        const int lead = __ffs(leaders) - 1;
        leaders &= leaders - 1;
        if (j % adapter_lanes != my_lane) continue;
        const int ad = s_id[lead];
        const unsigned mine = __ballot_sync(0xffffffffu, my_id == ad);  // tokens of this adapter
        const __nv_bfloat16* A = a.A + (static_cast<size_t>(ad) * a.rank + r0) * a.k;
        float acc[2][4][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
        for (int kb = kb_lo + warp; kb < kb_hi; kb += kWarps) {
            uint4 wv[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = h * 8 + g;
                    wv[s][h] = r < nr && k < a.k
                        ? *reinterpret_cast<const uint4*>(A + static_cast<size_t>(r) * a.k + k) : zero_u4();
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (!(mine >> (8 * n) & 0xffu)) continue;  // warp-uniform
                    const long long t = t0 + min(n * 8 + g, nt_here - 1);
                    const uint4 xv = k < a.k ? *reinterpret_cast<const uint4*>(a.x + t * a.k + k) : zero_u4();
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma_pieces(acc[h][n], wv[s][2 * h], wv[s][2 * h + 1], xv);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) red[warp][(h * 4 + n) * 4 + e][lane] = acc[h][n][e];
        __syncthreads();
        for (int u = tid; u < 2 * 4 * 4 * 32; u += kThreads) {
            const int l = u & 31, hne = u >> 5, e = hne & 3, n = (hne >> 2) & 3, h = hne >> 4;
            const int p = n * 8 + (l & 3) * 2 + (e & 1), r = h * 16 + (e >> 1) * 8 + (l >> 2);
            if (!(mine >> p & 1u) || (GEMM ? r0 + r >= a.r16 : r >= nr)) continue;
            float s = 0.0f;
            if (r < nr) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += red[w][hne][l];
            }
            if (GEMM) {
                if (a.scales) s *= a.scales[ad];
                __nv_bfloat16 part[3];
                split_bf16x3(s, part);
                __nv_bfloat16* dst = a.h_split + static_cast<size_t>(t0 + p) * 2 * a.r16 + r0 + r;
                dst[0] = part[0];
                dst[a.r16] = part[1];
            } else {
                h_out[(t0 + p) * a.rank + r0 + r] = s;
            }
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

// ------------------------------------------------------- streaming (m <= 64)
template <int NT>
struct StreamSmem {
    // double buffered where two fit into shared memory
    static constexpr int kBufs = NT < 8 ? 2 : 1;
    float red[kBufs][kWarps][2 * NT * 4][32];
    float h[8 * NT][MOE_MAX_LORA_RANK + 1];
    int id[8 * NT];
    float scale[8 * NT];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) lora_stream_kernel(const LoraArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    StreamSmem<NT>& sm = *reinterpret_cast<StreamSmem<NT>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c8 = (lane & 3) * 8;
    if (*a.status != kDevOk) return;
    const int m = static_cast<int>(a.m);
    if (tid < m) {
        const int id = a.adapter_ids[tid];
        sm.id[tid] = id;
        sm.scale[tid] = id >= 0 && a.scales ? a.scales[id] : 1.0f;
    }
    for (int u = tid; u < m * a.rank; u += kThreads) {
        float s = a.h[u];
        for (int z = 1; z < a.k_splits; ++z) s += a.h[static_cast<size_t>(z) * m * a.rank + u];
        sm.h[u / a.rank][u % a.rank] = s;
    }
    const int lo = static_cast<int>(static_cast<long long>(a.n) * blockIdx.x / gridDim.x);
    const int hi = static_cast<int>(static_cast<long long>(a.n) * (blockIdx.x + 1) / gridDim.x);
    const int nkb = (a.k + kKb - 1) / kKb;
    const int nt = (m + 7) >> 3;
    // steps go round robin over the warps; `rot` is the warp of a tile's first
    // step, from which the partial sums are added (the order is K's alone)
    int kb = warp, buf = 0, rot = 0;
    for (int n0 = lo; n0 < hi; n0 += kTileN) {
        const int nn = min(kTileN, hi - n0);
        const __nv_bfloat16* w = a.W + static_cast<size_t>(n0) * a.k;
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
        for (; kb < nkb; kb += kWarps) {
            uint4 wv[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = h * 8 + g;
                    wv[s][h] = r < nn && k < a.k ? ld_stream_u4(w + static_cast<size_t>(r) * a.k + k) : zero_u4();
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n >= nt) break;
                    const int t = min(n * 8 + g, m - 1);
                    const uint4 xv = k < a.k
                        ? *reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.k + k) : zero_u4();
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma_pieces(acc[h][n], wv[s][2 * h], wv[s][2 * h + 1], xv);
                }
            }
        }
        kb -= nkb;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sm.red[buf][warp][(h * NT + n) * 4 + e][lane] = acc[h][n][e];
        __syncthreads();
        // lane = output column of the tile, so that stores are contiguous
        for (int u = tid; u < m * kTileN; u += kThreads) {
            const int row = u % kTileN, t = u / kTileN;
            if (row >= nn) continue;
            const int hne = ((row >> 4) * NT + (t >> 3)) * 4 + ((row >> 3) & 1) * 2 + (t & 1);
            const int l = (row & 7) * 4 + ((t & 7) >> 1);
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) v += sm.red[buf][(q + rot) % kWarps][hne][l];
            const int id = sm.id[t];
            if (id >= 0)
                v += sm.scale[t] * expand_dot(a.B + (static_cast<size_t>(id) * a.n + n0 + row) * a.rank,
                                              sm.h[t], a.rank);
            store_y(a.y, a.y_dtype, static_cast<size_t>(t) * a.n + n0 + row, v);
        }
        rot = (rot + nkb) % kWarps;
        if (StreamSmem<NT>::kBufs == 2)
            buf ^= 1;
        else
            __syncthreads();
    }
}

template <int NT>
cudaError_t launch_stream(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    static PerDeviceOnce once;
    constexpr int smem = sizeof(StreamSmem<NT>);
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_stream_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err != cudaSuccess) return err;
    lora_stream_kernel<NT><<<num_sms, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

template <bool GEMM>
static cudaError_t launch_shrink(const LoraArgs& a, cudaStream_t stream) {
    static PerDeviceOnce once;
    constexpr int smem = kWarps * 2 * 4 * 4 * 32 * sizeof(float);
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(lora_shrink_kernel<GEMM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err != cudaSuccess) return err;
    const unsigned groups = static_cast<unsigned>((a.m + kGroup - 1) / kGroup);
    const unsigned rank_tiles = (a.rank + kRankTile - 1) / kRankTile;
    // a block per adapter for a few tokens, one for all of them when the
    // token groups fill the SMs by themselves
    const unsigned most = static_cast<unsigned>(a.m < kGroup ? a.m : kGroup);
    unsigned lanes = 296 / (groups * rank_tiles * a.k_splits);
    lanes = lanes < 1 ? 1 : lanes > most ? most : lanes;
    lora_shrink_kernel<GEMM><<<dim3(groups, rank_tiles * lanes, a.k_splits), kThreads, smem, stream>>>(
        a, static_cast<int>(rank_tiles));
    return cudaGetLastError();
}

cudaError_t launch_lora_shrink(const LoraArgs& a, cudaStream_t stream) {
    return a.h_split ? launch_shrink<true>(a, stream) : launch_shrink<false>(a, stream);
}

cudaError_t launch_lora_stream(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    if (a.m <= 8) return launch_stream<1>(a, num_sms, stream);
    if (a.m <= 16) return launch_stream<2>(a, num_sms, stream);
    if (a.m <= 32) return launch_stream<4>(a, num_sms, stream);
    return launch_stream<8>(a, num_sms, stream);
}

}  // namespace moe

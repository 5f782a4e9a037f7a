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
// Kernel 1 (router): a block computes the logits of two experts for all
//   tokens, its 16 warps splitting K.  The sum is kept in f64 so that the
//   choice of experts does not depend on the order of the additions: the
//   rounded logits are those of the exact sum but for ties of the rounding.
// Kernel 2 (experts): a cooperative grid of one block per SM.  Every block
//   repeats the routing of the few tokens (cheaper than a launch), takes an
//   equal share of all active experts' gate/up rows, and after a grid barrier
//   an equal share of the output's hidden rows over all active experts, so
//   the weighted combine happens in its own shared memory, in slot order,
//   with no atomics and no per-slot rows in global memory.
//
// The bound is reading the distinct chosen experts' weights once.  Weight
// rows go from global memory straight into mma.sync fragments
// (stream_mma.cuh); the 16 warps of a block split K, and partial sums meet in
// shared memory once per tile.  gate/up multiplies the bf16 x as it is; the
// f32 activation enters the down projection as three bf16 parts, so nothing
// is rounded below f32.
#include <climits>
#include <math.h>

#include "launch.h"
#include "stream_mma.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKb = 64;      // K columns of one warp step: 128 bytes of each weight row
constexpr int kTileI = 16;   // intermediate rows of a gate/up tile (gate and up rows each)
constexpr int kTileH = 32;   // hidden rows of a down tile
constexpr int kMaxTokens = kLayerDecodeMaxTokens;
constexpr int kMaxRows = kLayerDecodeMaxRows;

__device__ __forceinline__ double sigmoid_f64(float v) {
    return 1.0 / (1.0 + exp(-static_cast<double>(v)));
}

// ------------------------------------------------------------------ router
constexpr int kRouterRows = 2;    // experts per block
constexpr int kRouterTokens = 4;  // tokens per pass over a warp's weights

__global__ void __launch_bounds__(kThreads) layer_router_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ W_router,
    const __nv_bfloat16* __restrict__ w_sh, int m, int hidden, int n_experts,
    float* __restrict__ logits, float* __restrict__ scores, float* __restrict__ gate,
    unsigned* __restrict__ barrier, int* __restrict__ status) {
    __shared__ double part[kWarps][kRouterRows * kMaxTokens];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *barrier = 0;  // of the kernel that follows
        *status = kDevOk;
    }
    const int n_rows = n_experts + (w_sh ? 1 : 0);
    const int r0 = blockIdx.x * kRouterRows;
    const __nv_bfloat16* wrow[kRouterRows];
#pragma unroll
    for (int j = 0; j < kRouterRows; ++j) {
        const int r = min(r0 + j, n_rows - 1);
        wrow[j] = r < n_experts ? W_router + static_cast<size_t>(r) * hidden : w_sh;
    }
    for (int t0 = 0; t0 < m; t0 += kRouterTokens) {
        double acc[kRouterRows * kRouterTokens];
#pragma unroll
        for (int i = 0; i < kRouterRows * kRouterTokens; ++i) acc[i] = 0.0;
        for (int k = (warp * 32 + lane) * 8; k < hidden; k += kThreads * 8) {
            float wf[kRouterRows][8];
#pragma unroll
            for (int j = 0; j < kRouterRows; ++j)
                bf16x8_to_f32(*reinterpret_cast<const uint4*>(wrow[j] + k), wf[j]);
#pragma unroll
            for (int q = 0; q < kRouterTokens; ++q) {
                const int t = min(t0 + q, m - 1);
                float xf[8];
                bf16x8_to_f32(*reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * hidden + k), xf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double xd = xf[e];
#pragma unroll
                    for (int j = 0; j < kRouterRows; ++j)
                        acc[j * kRouterTokens + q] = fma(static_cast<double>(wf[j][e]), xd,
                                                         acc[j * kRouterTokens + q]);
                }
            }
        }
        // 8 sums over 32 lanes: three steps that halve the sums a lane holds
        // (it ends with sum number lane / 4), then two over the quad
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1) {
            const bool upper = lane & (h * 4);
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const double give = upper ? acc[i] : acc[i + h];
                const double keep = upper ? acc[i + h] : acc[i];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, h * 4);
            }
        }
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 2);
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
        if ((lane & 3) == 0) {
            const int i = lane >> 2;
            const int t = t0 + i % kRouterTokens;
            if (t < m) part[warp][(i / kRouterTokens) * kMaxTokens + t] = acc[0];
        }
    }
    __syncthreads();
    const int j = threadIdx.x / kMaxTokens, t = threadIdx.x % kMaxTokens;
    if (j < kRouterRows && r0 + j < n_rows && t < m) {
        double sum = 0.0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += part[w][j * kMaxTokens + t];
        const float l = static_cast<float>(sum);
        const float s = static_cast<float>(sigmoid_f64(l));
        const int r = r0 + j;
        if (r < n_experts) {
            logits[static_cast<size_t>(t) * n_experts + r] = l;
            scores[static_cast<size_t>(t) * n_experts + r] = s;
        } else {
            gate[t] = s;
        }
    }
}

// ----------------------------------------------------------------- experts
// Dynamic shared memory of the experts kernel for NT token groups of 8.
template <int NT>
struct ExpertsSmem {
    float red[2][kWarps][2 * NT * 4][32];  // partial sums of one tile, double buffered
    float d[kMaxRows + kMaxTokens][kTileH + 1];  // d[routed row or shared token][hidden row]
    int id[kMaxRows], perm[kMaxRows], gexp[kMaxRows], gfirst[kMaxRows], gcnt[kMaxRows];
    int slot_id[kMaxRows];
    float weight[kMaxRows];
    int warp_n[kWarps], flag;
};

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
    unsigned best = 0;  // 0: nothing left (every real key is above it)
    int best_e = INT_MAX;
    for (int e = lane; e < n_experts; e += 32) {
        const unsigned u = ordered(scores[e] + (bias ? bias[e] : 0.0f));
        reinterpret_cast<unsigned*>(key)[e] = u;
        if (u > best) {
            best = u;
            best_e = e;
        }
    }
    int my_e = 0;
    for (int j = 0; j < top_k; ++j) {
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        const int win = static_cast<int>(
            __reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(best_e) : 0xffffffffu));
        if (lane == j) my_e = win;
        if (best_e == win) {
            unsigned* k = reinterpret_cast<unsigned*>(key);
            k[win] = 0;
            best = 0;
            best_e = INT_MAX;
            for (int e = lane; e < n_experts; e += 32)
                if (k[e] > best) {
                    best = k[e];
                    best_e = e;
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

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) layer_experts_kernel(const LayerDecodeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    ExpertsSmem<NT>& sm = *reinterpret_cast<ExpertsSmem<NT>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c8 = (lane & 3) * 8;
    const int rows = a.m * a.top_k;
    const int n_shared = a.inter_sh > 0 ? 1 : 0;

    // routing and expert map of the few tokens, in every block
    {
        float* keys = &sm.red[0][0][0][0] + warp * a.n_experts;  // of the warps that have tokens
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
    int n_groups = 0;
    block_small_map(sm.slot_id, rows, a.n_experts, sm.id, sm.perm, sm.gexp, sm.gfirst, sm.gcnt,
                    sm.warp_n, &sm.flag, &n_groups);

    // Group q: expert sm.gexp[q] with the sorted rows [first, first + cnt);
    // group n_groups: the shared expert with every token.
    const auto group = [&](int q, int& first, int& cnt, int& expert) {
        if (q < n_groups) {
            first = sm.gfirst[q];
            cnt = sm.gcnt[q];
            expert = sm.gexp[q];
        } else {
            first = 0;
            cnt = a.m;
            expert = -1;
        }
    };

    // A tile's K steps go round robin over the warps, on from where the last
    // tile's ended: `rot` is the warp of a tile's first step.  Partial sums are
    // added from that warp on, so a row's bits depend on K alone and not on
    // the tiles that came before.
    int buf = 0, rot = 0;
    // ------------------------------------------------ gate / up -> activation
    {
        const long long routed = static_cast<long long>(n_groups) * a.inter;
        const long long total = routed + (n_shared ? a.inter_sh : 0);
        const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
        const int nkb = (a.hidden + kKb - 1) / kKb;
        int kb = warp;  // this warp's step of the current tile; steps go round robin over all tiles
        for (long long pos = lo; pos < hi;) {
            const int q = pos < routed ? static_cast<int>(pos / a.inter) : n_groups;
            int first, cnt, expert;
            group(q, first, cnt, expert);
            const int width = expert < 0 ? a.inter_sh : a.inter;
            const int i0 = static_cast<int>(pos - static_cast<long long>(q) * a.inter);
            int ni = min(kTileI, width - i0);
            if (ni > hi - pos) ni = static_cast<int>(hi - pos);
            pos += ni;
            const size_t row0 = (expert < 0 ? 0 : static_cast<size_t>(expert) * a.inter) + i0;
            const __nv_bfloat16* wg = (expert < 0 ? a.S_gate : a.W_gate) + row0 * a.hidden;
            const __nv_bfloat16* wu = (expert < 0 ? a.S_up : a.W_up) + row0 * a.hidden;
            const int nt = (cnt + 7) >> 3;
            const __nv_bfloat16* xr[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int p = min(n * 8 + g, cnt - 1);
                const int t = expert < 0 ? p : sm.perm[first + p] / a.top_k;
                xr[n] = a.x + static_cast<size_t>(t) * a.hidden;
            }
            float acc[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
            for (; kb < nkb; kb += kWarps) {
                uint4 wv[2][2][2];  // [32-column piece][row half][gate / up]
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = h * 8 + g;
                        const bool in = r < ni && k < a.hidden;
                        wv[s][h][0] = in ? ld_stream_u4(wg + static_cast<size_t>(r) * a.hidden + k) : zero_u4();
                        wv[s][h][1] = in ? ld_stream_u4(wu + static_cast<size_t>(r) * a.hidden + k) : zero_u4();
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (n >= nt) break;
                        const uint4 xv = k < a.hidden ? *reinterpret_cast<const uint4*>(xr[n] + k) : zero_u4();
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma_pieces(acc[h][n], wv[s][h][0], wv[s][h][1], xv);
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
            // element (h, n, e) holds gate (e < 2) or up (e >= 2) of row h * 8 + g, token n * 8 + 2 c + (e & 1)
            for (int u = tid; u < 2 * NT * 64; u += kThreads) {
                const int l = u & 31, par = (u >> 5) & 1, hn = u >> 6;
                const int row = (hn / NT) * 8 + (l >> 2), p = (hn % NT) * 8 + (l & 3) * 2 + par;
                if (row >= ni || p >= cnt) continue;
                float gs = 0.0f, us = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    gs += sm.red[buf][(w + rot) % kWarps][hn * 4 + par][l];
                    us += sm.red[buf][(w + rot) % kWarps][hn * 4 + 2 + par][l];
                }
                __nv_bfloat16 part[3];
                split_bf16x3(gs / (1.0f + expf(-gs)) * us, part);
                __nv_bfloat16* dst = expert < 0
                    ? a.act_sh + static_cast<size_t>(p) * 3 * a.inter_sh
                    : a.act + static_cast<size_t>(first + p) * 3 * a.inter;
#pragma unroll
                for (int s = 0; s < 3; ++s) dst[static_cast<size_t>(s) * width + i0 + row] = part[s];
            }
            buf ^= 1;
            rot = (rot + nkb) % kWarps;
        }
    }
    if (!grid_barrier(a.barrier, gridDim.x, &sm.flag, a.status, a.wait_limit_ns)) return;

    // ------------------------------------------------ down + combine
    const int lo = static_cast<int>(static_cast<long long>(a.hidden) * blockIdx.x / gridDim.x);
    const int hi = static_cast<int>(static_cast<long long>(a.hidden) * (blockIdx.x + 1) / gridDim.x);
    int kb = warp;
    rot = 0;
    for (int h0 = lo; h0 < hi; h0 += kTileH) {
        const int nh = min(kTileH, hi - h0);
        for (int q = 0; q < n_groups + n_shared; ++q) {
            int first, cnt, expert;
            group(q, first, cnt, expert);
            const int width = expert < 0 ? a.inter_sh : a.inter;
            const int nkb = (width + kKb - 1) / kKb;
            const __nv_bfloat16* wd =
                expert < 0 ? a.S_down + static_cast<size_t>(h0) * width
                           : a.W_down + (static_cast<size_t>(expert) * a.hidden + h0) * width;
            const __nv_bfloat16* act = expert < 0 ? a.act_sh : a.act;
            const int nt = (cnt + 7) >> 3;
            float acc[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.0f;
            for (; kb < nkb; kb += kWarps) {
                uint4 wv[2][4];  // [32-column piece][group of 8 rows]
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int r = h * 8 + g;
                        wv[s][h] = r < nh && k < width ? ld_stream_u4(wd + static_cast<size_t>(r) * width + k)
                                                       : zero_u4();
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = kb * kKb + s * 32 + c8;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (n >= nt) break;
                        const __nv_bfloat16* ar =
                            act + static_cast<size_t>(first + min(n * 8 + g, cnt - 1)) * 3 * width + k;
#pragma unroll
                        for (int z = 2; z >= 0; --z) {
                            const uint4 av = k < width
                                ? *reinterpret_cast<const uint4*>(ar + static_cast<size_t>(z) * width)
                                : zero_u4();
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma_pieces(acc[h][n], wv[s][2 * h], wv[s][2 * h + 1], av);
                        }
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
            // element (h, n, e): hidden row h * 16 + (e / 2) * 8 + g, token n * 8 + 2 c + (e & 1)
            for (int u = tid; u < 2 * NT * 4 * 32; u += kThreads) {
                const int l = u & 31, hne = u >> 5, e = hne & 3, n = (hne >> 2) % NT, h = (hne >> 2) / NT;
                const int p = n * 8 + (l & 3) * 2 + (e & 1);
                if (p >= cnt) continue;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sm.red[buf][(w + rot) % kWarps][hne][l];
                sm.d[expert < 0 ? rows + p : sm.perm[first + p]][h * 16 + (e >> 1) * 8 + (l >> 2)] = s;
            }
            buf ^= 1;
            rot = (rot + nkb) % kWarps;
        }
        __syncthreads();
        for (int u = tid; u < a.m * kTileH; u += kThreads) {
            const int t = u / kTileH, h = u % kTileH;
            if (h >= nh) continue;
            float y = 0.0f;
            for (int j = 0; j < a.top_k; ++j) {
                const int r = t * a.top_k + j;
                y += sm.weight[r] * sm.d[r][h];
            }
            if (n_shared) y += a.gate[t] * sm.d[rows + t][h];
            a.y[static_cast<size_t>(t) * a.hidden + h0 + h] = y;
        }
        __syncthreads();
    }
}

template <int NT>
cudaError_t launch_experts(const LayerDecodeArgs& args, int num_sms, cudaStream_t stream) {
    // the routing keys of the min(16, 8 NT) warps that route lie in the partial-sum buffers
    static_assert(sizeof(ExpertsSmem<NT>::red) >= sizeof(float) * MOE_MAX_EXPERTS * (NT < 2 ? 8 : kWarps),
                  "routing scratch");
    constexpr int smem = sizeof(ExpertsSmem<NT>);
    static PerDeviceOnce once;
    cudaError_t err = once.run([] {
        return cudaFuncSetAttribute(layer_experts_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
    return cudaLaunchKernelEx(&cfg, layer_experts_kernel<NT>, args);
}

}  // namespace

cudaError_t launch_layer_decode(const LayerDecodeArgs& args, const __nv_bfloat16* W_router,
                                const __nv_bfloat16* w_sh, float* logits, int num_sms,
                                cudaStream_t stream) {
    const int n_rows = args.n_experts + (args.inter_sh > 0 ? 1 : 0);
    layer_router_kernel<<<(n_rows + kRouterRows - 1) / kRouterRows, kThreads, 0, stream>>>(
        args.x, W_router, w_sh, args.m, args.hidden, args.n_experts, logits,
        const_cast<float*>(args.scores), const_cast<float*>(args.gate), args.barrier, args.status);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    if (args.m <= 8) return launch_experts<1>(args, num_sms, stream);
    if (args.m <= 16) return launch_experts<2>(args, num_sms, stream);
    return launch_experts<4>(args, num_sms, stream);
}

}  // namespace moe

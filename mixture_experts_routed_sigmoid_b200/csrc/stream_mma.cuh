// Weight streaming through mma.sync: building blocks of the decode-size
// kernels that read every weight row once and multiply it with a few tokens.
//
// A warp multiplies 16 weight rows (the MMA's M) with up to 8 token rows (its
// N) over 32 columns of K with two m16n8k16 instructions.  Which K columns an
// instruction's k index means is free as long as both operands agree, so lane
// (g = lane / 4, c = lane % 4) simply loads 16 contiguous bytes, columns
// [8c, 8c + 8) of the 32, of weight rows g and g + 8 and of token row g: the
// fragments come straight from global memory in 16-byte pieces, with no
// shared memory and no shuffles.  (tcgen05 would want the weights staged in
// shared memory; at one MMA per 512 weight bytes the tensor pipe idles either
// way, and the loads are all that counts.)
#pragma once

#include "device_common.cuh"

namespace moe {

// d += A (16 x 16, rows) * B (16 x 8, columns), bf16 operands, f32 accumulator.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d += 16 weight rows x 8 token rows over the lane quad's 32 columns: `lo` and
// `hi` are the lane's pieces of weight rows g and g + 8, `t` of token row g.
// Result element d[2 * r + p] belongs to weight row g + 8 r, token 2 c + p.
__device__ __forceinline__ void mma_pieces(float (&d)[4], const uint4& lo, const uint4& hi,
                                           const uint4& t) {
    mma_16x8x16(d, lo.x, hi.x, lo.y, hi.y, t.x, t.y);
    mma_16x8x16(d, lo.z, hi.z, lo.w, hi.w, t.z, t.w);
}

__device__ __forceinline__ uint4 zero_u4() { return make_uint4(0u, 0u, 0u, 0u); }

// v as the sum of three bf16 values (24 significant bits): hi = bf16(v), mid =
// bf16(v - hi), lo = bf16(v - hi - mid).  The MMA operands of an f32 value:
// one bf16 keeps 8 bits and two keep 16, both short of the f32 product that
// the value stands for.  A value that is not finite is its own hi part.
__device__ __forceinline__ void split_bf16x3(float v, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(v);
    const float h = __bfloat162float(p[0]);
    const bool finite = fabsf(h) <= 3.4e38f;
    const float r1 = finite ? v - h : 0.0f;
    p[1] = __float2bfloat16_rn(r1);
    p[2] = __float2bfloat16_rn(r1 - __bfloat162float(p[1]));
}

// Grid-wide barrier of a cooperative launch: every block's earlier writes are
// visible to every block after it.  `counter` is zero before the launch; the
// n-th barrier of a kernel passes target = n * gridDim.x.  Returns false in
// every thread of the block when the wait ran out (status set).
__device__ __forceinline__ bool grid_barrier(unsigned* counter, unsigned target, int* s_flag,
                                             int* status, uint64_t limit_ns) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
        int good = 1;
        unsigned seen;
        uint64_t start = 0;
        for (uint64_t polls = 0;; ++polls) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(counter) : "memory");
            if (seen >= target) break;
            if ((polls & 255) == 255) {
                const uint64_t now = global_timer_ns();
                if (!start) start = now;
                if (now - start > limit_ns || polls > kMaxWaitPolls) {
                    set_status(status, kDevTimeout);
                    good = 0;
                    break;
                }
            }
        }
        *s_flag = good;
    }
    __syncthreads();
    return *s_flag != 0;
}

}  // namespace moe

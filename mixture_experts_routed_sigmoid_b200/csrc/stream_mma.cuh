// Weight streaming through mma.sync: building blocks of the decode-size
// kernels that read every weight row once and multiply it with a few tokens.
//
// A warp owns a tile of 16 or 32 weight rows (the MMA's M) and walks their
// whole K on its own, so no partial sums cross warps and no block-wide barrier
// stands in the stream.  Its weights arrive through a ring in shared memory
// that only this warp fills and reads (cp.async, 16 bytes per lane and copy):
// 4 KB per step, as 32 rows x 64 columns or 16 rows x 128.  The ring keeps 4 or
// 8 KB per warp in flight without holding registers, across tile ends
// and grid barriers.
//
// Which K columns an instruction's k index means is free as long as both
// operands agree, so lane (g = lane / 4, c = lane % 4) takes 16 contiguous
// bytes, columns [8 c, 8 c + 8) of 32, of weight rows g and g + 8 (from the
// ring) and of token row g (from global memory): two m16n8k16 instructions
// per 32 columns, no shuffles.  The tokens are the MMA's N: up to 8 each.
// (tcgen05 would idle just the same: at one instruction per 512 weight bytes
// the loads are all that counts.)
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

// 16-byte copy that reads 256 bytes into the L2 at once: a ring step takes 128
// or 256 contiguous bytes of each of many rows, and the next step takes the
// next ones.  (Without it 8 tokens of 55 experts took 379 us, with it 350.)
__device__ __forceinline__ void cp_async_16_l2(uint32_t dst_smem, const void* src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src),
                 "r"(src_bytes)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

constexpr int kRingBytes = 4096;  // one step of one warp

// Byte offset of 16-byte piece j of ring row r.  Odd rows swap the 64-byte
// halves of each 128 bytes, so the eight lanes of a fragment read (two rows,
// four pieces each) touch all banks once.
template <bool WIDE>  // 16 rows x 128 columns, else 32 rows x 64
__device__ __forceinline__ uint32_t ring_offset(int r, int j) {
    return static_cast<uint32_t>(r * (WIDE ? 256 : 128) + ((j ^ ((r & 1) << 2)) << 4));
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

// Copies one step into the ring slot at `slot`: columns [k0, k0 + 64 or 128)
// of the tile's rows.  row(r) gives the global address of ring row r, or null
// for a row that the tile does not have (its slot keeps what it held: rows
// never mix in an MMA, and the results of such rows are dropped).  Columns
// past k are zeros.
template <bool WIDE, class Row>
__device__ __forceinline__ void ring_fill(uint32_t slot, Row row, int k0, int k, int lane) {
    constexpr int kPieces = WIDE ? 16 : 8, kRowsPerCopy = 32 / kPieces;
    const int j = lane % kPieces, kk = k0 + j * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = lane / kPieces + i * kRowsPerCopy;
        const __nv_bfloat16* src = row(r);
        if (src) cp_async_16_l2(slot + ring_offset<WIDE>(r, j), src + (kk < k ? kk : 0), kk < k ? 16u : 0u);
    }
}

// One unit of token operands: the lane's pieces of 64 columns from k0 on of one
// group of 8 tokens, for PARTS consecutive rows of length k.
template <int PARTS>
struct TokenPieces {
    uint4 v[2][PARTS];
    __device__ __forceinline__ void load(const __nv_bfloat16* tok, int k0, int k, int lane) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int kk = k0 + s * 32 + (lane & 3) * 8;
#pragma unroll
            for (int z = 0; z < PARTS; ++z)
                v[s][z] = kk < k ? *reinterpret_cast<const uint4*>(tok + static_cast<size_t>(z) * k + kk)
                                 : make_uint4(0u, 0u, 0u, 0u);
        }
    }
};

// acc[h][n] += the step's weights times the tokens, for a step whose weights
// are being copied: `ready` waits for them.  The token operands are loaded one
// unit ahead, the first before the wait.  A unit's products are summed in the
// tensor core's accumulator and added to acc by one f32 addition: its
// accumulation truncates, and a chain of K / 16 instructions would lose several
// times what rounding does.
// tok[n]: the lane's token row (row n * 8 + g); with PARTS > 1 an f32 value as
// bf16 parts in consecutive rows of length k, whose products are all summed.
template <bool WIDE, int NT, int PARTS, class Ready>
__device__ __forceinline__ void ring_multiply(float (&acc)[2][NT][4], uint32_t slot,
                                              const __nv_bfloat16* const (&tok)[NT], int nt, int k0,
                                              int k, int lane, Ready ready) {
    constexpr int kHalves = WIDE ? 2 : 1, kTiles = WIDE ? 1 : 2;
    const int g = lane >> 2, c = lane & 3;
    TokenPieces<PARTS> t[2];
    t[0].load(tok[0], k0, k, lane);
    ready();
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
        uint4 w[kTiles][2][2];  // [16 rows][32 columns][rows g, g + 8]
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    w[h][s][r] = ld_shared_u4(slot + ring_offset<WIDE>(h * 16 + r * 8 + g, half * 8 + s * 4 + c));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt) break;  // warp-uniform
            const int u = half * NT + n;  // which buffer: units alternate where NT is 1 or even
            if (n + 1 < NT && n + 1 < nt)
                t[(u + 1) & 1].load(tok[n + 1 < NT ? n + 1 : 0], k0 + half * 64, k, lane);
            else if (half + 1 < kHalves && NT == 1)
                t[(u + 1) & 1].load(tok[0], k0 + (half + 1) * 64, k, lane);
            float d[kTiles][4];
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) d[h][e] = 0.0f;
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int z = PARTS - 1; z >= 0; --z) mma_pieces(d[h], w[h][s][0], w[h][s][1], t[u & 1].v[s][z]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] += d[h][e];
            }
        }
        // (the number of groups is not known at compile time, so the second
        // half's first unit has a buffer of its own parity)
        if (half + 1 < kHalves && NT > 1) t[0].load(tok[0], k0 + (half + 1) * 64, k, lane);
    }
}

// The same for one group of tokens, whose operands are loaded a step ahead:
// t holds those of this step's two halves (WIDE), or of this step and the next.
// `stride` columns lie between the warp's steps.
template <bool WIDE, int PARTS>
__device__ __forceinline__ void first_tokens(TokenPieces<PARTS> (&t)[2], const __nv_bfloat16* tok, int k0, int k,
                                             int stride, int lane) {
    t[0].load(tok, k0, k, lane);
    t[1].load(tok, k0 + (WIDE ? 64 : stride), k, lane);
}
template <bool WIDE, int PARTS, int NT>
__device__ __forceinline__ void ring_multiply_one(float (&acc)[2][NT][4], uint32_t slot, TokenPieces<PARTS> (&t)[2],
                                                  const __nv_bfloat16* tok, int k0, int k, int stride, int lane) {
    constexpr int kHalves = WIDE ? 2 : 1, kTiles = WIDE ? 1 : 2;
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint4 lo = ld_shared_u4(slot + ring_offset<WIDE>(h * 16 + g, half * 8 + s * 4 + c));
                const uint4 hi = ld_shared_u4(slot + ring_offset<WIDE>(h * 16 + 8 + g, half * 8 + s * 4 + c));
#pragma unroll
                for (int z = PARTS - 1; z >= 0; --z) mma_pieces(d, lo, hi, t[half].v[s][z]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[h][0][e] += d[e];
        }
        if (WIDE) t[half].load(tok, k0 + stride + half * 64, k, lane);
    }
    if (!WIDE) {
        t[0] = t[1];
        t[1].load(tok, k0 + 2 * stride, k, lane);
    }
}

// Grid-wide barrier of a cooperative launch: every block's writes before
// grid_arrive are visible to every block after its grid_wait.  `counter` is
// zero before the launch; the n-th barrier of a kernel waits for target = n *
// gridDim.x.  What a block issues between the two calls is on its way while the
// grid meets.
__device__ __forceinline__ void grid_arrive(unsigned* counter) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(counter, 1u);
    }
}

// False in every thread of the block when the wait ran out (status set); the
// thread's copies in flight have then landed, so that the block can leave.
__device__ __forceinline__ bool grid_wait(unsigned* counter, unsigned target, int* s_flag, int* status,
                                          uint64_t limit_ns) {
    if (threadIdx.x == 0) {
        int good = 1;
        uint64_t start = 0;
        // relaxed polls and one fence at the end: an acquire per poll would
        // drop the L1 each time
        for (uint64_t polls = 0; *reinterpret_cast<volatile unsigned*>(counter) < target; ++polls) {
            if ((polls & 63) == 63) {
                const uint64_t now = global_timer_ns();
                if (!start) start = now;
                if (now - start > limit_ns || polls > kMaxWaitPolls) {
                    set_status(status, kDevTimeout);
                    good = 0;
                    break;
                }
            }
        }
        __threadfence();
        *s_flag = good;
    }
    __syncthreads();
    if (*s_flag) return true;
    cp_async_wait_all();
    return false;
}

}  // namespace moe

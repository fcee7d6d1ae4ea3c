// int8_tiles.cuh -- INT8 codes to f16 tiles for the tcgen05 kernels over an INT8 cache (prefill_int8.cu,
// decode_int8_wide.cu): K = sk c and V = sv c enter the products as (s / W) c in f16, W a power of two at or above
// every scale that the CTA meets -- exact for powers of two down to 2^-17 of the largest, else within 2^-25 of W or
// half a step of f16 --, and W goes into the softmax's scale or the output's.
#pragma once

#include "pkv_device.cuh"
#include "warp_mma.cuh"

namespace pkv {

constexpr uint32_t kTileHalf = 128 * 128;  // 128 rows x 128 bytes: a 128-byte swizzle atom along head_dim

// Smallest power of two >= x, for finite x >= 0 (0 for 0; at most 2^127).
__device__ __forceinline__ float pow2_at_least(float x) {
    uint32_t b = __float_as_uint(x);
    if (b & 0x7fffffu) b = (b & 0x7f800000u) + 0x800000u;
    return b >= 0x7f800000u ? 1.7014118e38f : __uint_as_float(b);
}

// Four codes (one word) times the f16 pair kk. 1024 + (c + 128) less 1152 is c exactly; kk a power of two: (1024 + c + 128)
// kk - 1152 kk in one rounding, the exact product's (n = -1152 kk); else the product of c and kk, rounded.
template <bool POW2>
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t kk, uint32_t n, uint32_t &lo, uint32_t &hi) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    if (POW2) {
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(lo) : "r"(a), "r"(kk), "r"(n));
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(hi) : "r"(b), "r"(kk), "r"(n));
    } else {
        asm("{\n\t.reg .b32 c;\n\tadd.rn.f16x2 c, %1, %2;\n\tmul.rn.f16x2 %0, c, %3;\n\t}" : "=r"(lo) : "r"(a), "r"(0xe480e480u), "r"(kk));
        asm("{\n\t.reg .b32 c;\n\tadd.rn.f16x2 c, %1, %2;\n\tmul.rn.f16x2 %0, c, %3;\n\t}" : "=r"(hi) : "r"(b), "r"(0xe480e480u), "r"(kk));
    }
}

// 32 rows r0 .. r0 + 31 of a tile by a warp: codes (rows of D bytes, 128-byte swizzle or, head_dim 64, 64-byte) to the f16
// layout that TMA writes for a 16-bit cache (64-column halves of 128-byte rows, 128-byte swizzle), times the factor of
// their page, which lane i holds for page i. Groups of 8 rows lie in one page.
template <int D, bool POW2>
__device__ __forceinline__ void convert_rows(const uint8_t *codes, uint8_t *f16, int r0, uint32_t kk, int log2_bs, int lane) {
    constexpr int kLanes = D / 16;             // lanes a row: 16 codes each
    constexpr int kRowsLoad = 32 / kLanes;     // rows a load of the warp: 4 (head_dim 128) or 8
    constexpr int kLoads = 4;                  // loads in flight
    const int c = lane % kLanes, rr = lane / kLanes;
    // f16 chunks 2c and 2c + 1 (16 bytes each) of the row, in half c / 4; the lanes of the two halves store opposite chunks
    // first: the stores of a row in one instruction then fill all 32 banks once
    const int hf = c >> 2, k0 = 2 * (c & 3), ka = k0 + hf, kb = k0 + 1 - hf;
#pragma unroll
    for (int b0 = 0; b0 < 32; b0 += kLoads * kRowsLoad) {
        uint4 raw[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = r0 + b0 + i * kRowsLoad + rr;
            const int cc = D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
            raw[i] = *reinterpret_cast<const uint4 *>(codes + r * D + (cc << 4));
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int g = r0 + b0 + i * kRowsLoad, r = g + rr;
            const uint32_t f = __shfl_sync(0xffffffffu, kk, (g >> log2_bs) & 31);
            uint32_t nf;
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(nf) : "r"(f), "r"(0xe480e480u));
            uint4 v0, v1;
            codes4_f16<POW2>(raw[i].x, f, nf, v0.x, v0.y);
            codes4_f16<POW2>(raw[i].y, f, nf, v0.z, v0.w);
            codes4_f16<POW2>(raw[i].z, f, nf, v1.x, v1.y);
            codes4_f16<POW2>(raw[i].w, f, nf, v1.z, v1.w);
            uint8_t *row = f16 + hf * kTileHalf + r * 128;
            *reinterpret_cast<uint4 *>(row + ((ka ^ (r & 7)) << 4)) = hf ? v1 : v0;
            *reinterpret_cast<uint4 *>(row + ((kb ^ (r & 7)) << 4)) = hf ? v0 : v1;
        }
    }
}

// q tiles (n16 16-byte vectors) from bf16 to f16 in place by 128 threads, exactly for |q| within f16's range.
__device__ __forceinline__ void q_tiles_to_f16(uint8_t *sq, int n16, int t) {
    uint4 *q4 = reinterpret_cast<uint4 *>(sq);
    for (int i = t; i < n16; i += 128) {
        const uint4 v = q4[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = pack_pair<false>(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
        q4[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Scales of the pages that hold keys [from, to) of a block-table row, by 128 threads (t): the largest finite K and V
// scale (their bits, in max[2]) and the first position of a page whose scale is not finite (nan[2]). A page id outside
// the pool counts as page 0, which is read in its place.
__device__ __forceinline__ void page_scales(const float *scales, const int *bt, int num_blocks, int num_kv_heads, int head,
                                            int log2_bs, int from, int to, int t, uint32_t *max, int *nan) {
    float mk = 0.f, mv = 0.f;
    int nk = 0x7fffffff, nv = 0x7fffffff;
    for (int i = (from >> log2_bs) + t; i <= (to - 1) >> log2_bs; i += 128) {
        int pb = __ldg(bt + i);
        if (pb < 0 || pb >= num_blocks) pb = 0;
        const float *sc = scales + (size_t)pb * 2 * num_kv_heads + head;
        const float k = __ldg(sc), v = __ldg(sc + num_kv_heads);
        if (k < INFINITY) mk = fmaxf(mk, k); else nk = min(nk, i << log2_bs);
        if (v < INFINITY) mv = fmaxf(mv, v); else nv = min(nv, i << log2_bs);
    }
    const uint32_t bk = __reduce_max_sync(0xffffffffu, __float_as_uint(mk));  // (bits of numbers >= 0 are in order)
    const uint32_t bv = __reduce_max_sync(0xffffffffu, __float_as_uint(mv));
    nk = __reduce_min_sync(0xffffffffu, nk);
    nv = __reduce_min_sync(0xffffffffu, nv);
    if ((t & 31) == 0) {
        atomicMax(&max[0], bk);
        atomicMax(&max[1], bv);
        atomicMin(&nan[0], nk);
        atomicMin(&nan[1], nv);
        __threadfence_block();
    }
}

}  // namespace pkv

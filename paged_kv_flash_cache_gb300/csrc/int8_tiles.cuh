// int8_tiles.cuh -- INT8 codes to f16 tiles for the tcgen05 kernels over an INT8 cache (prefill_int8.cu,
// decode_int8_wide.cu): K = sk c and V = sv c enter the products as (s / W) c in f16, W a power of two at or above
// every scale that the CTA meets, and W goes into the softmax's scale or the output's. Exact for powers of two down to
// 2^-24 of W (f16's smallest step), below which they count as 0; else within two half steps of f16 and 2^-24 W times the code.
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

// 32 rows r0 .. r0 + 31 (r0 a multiple of 32) of a tile by a warp: codes (rows of D bytes, 128-byte swizzle or, head_dim 64,
// 64-byte) to the f16 layout that TMA writes for a 16-bit cache (64-column halves of 128-byte rows, 128-byte swizzle), times the
// factor of their page, which lane i holds for page i. Groups of 8 rows lie in one page.
template <int D, bool POW2>
__device__ __forceinline__ void convert_rows(const uint8_t *codes, uint8_t *f16, int r0, uint32_t kk, int log2_bs, int lane) {
    constexpr int kLanes = D / 16;             // lanes a row: 16 codes each
    constexpr int kRowsLoad = 32 / kLanes;     // rows a load of the warp: 4 (head_dim 128) or 8
    constexpr int kLoads = 32 / kRowsLoad;
    constexpr int kAhead = 4;                  // loads in flight
    const int c = lane % kLanes, rr = lane / kLanes;
    uint32_t f[4], n[4];  // of the groups of 8 rows
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[q] = __shfl_sync(0xffffffffu, kk, ((r0 + 8 * q) >> log2_bs) & 31);
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(n[q]) : "r"(f[q]), "r"(0xe480e480u));
    }
    // f16 chunks 2c and 2c + 1 (16 bytes each) of the row, in half c / 4; the lanes of the two halves store opposite chunks
    // first: the stores of a row in one instruction then fill all 32 banks once
    const int hf = c >> 2, ka = 2 * (c & 3) + hf, kb = ka ^ 1;
    const uint8_t *src = codes + (r0 + rr) * D;
    uint8_t *dst = f16 + hf * kTileHalf + (r0 + rr) * 128;
    auto load = [&](int i) {
        const int r = i * kRowsLoad + rr;  // (its low bits: the row's)
        return *reinterpret_cast<const uint4 *>(src + i * kRowsLoad * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
    };
    uint4 raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) raw[i] = load(i);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint4 x = raw[i % kAhead];
        if (i + kAhead < kLoads) raw[i % kAhead] = load(i + kAhead);
        const int q = i * kRowsLoad / 8, s = (i * kRowsLoad + rr) & 7;
        uint4 va, vb;
        codes4_f16<POW2>(hf ? x.z : x.x, f[q], n[q], va.x, va.y);
        codes4_f16<POW2>(hf ? x.w : x.y, f[q], n[q], va.z, va.w);
        codes4_f16<POW2>(hf ? x.x : x.z, f[q], n[q], vb.x, vb.y);
        codes4_f16<POW2>(hf ? x.y : x.w, f[q], n[q], vb.z, vb.w);
        uint8_t *row = dst + i * kRowsLoad * 128;
        *reinterpret_cast<uint4 *>(row + ((ka ^ s) << 4)) = va;
        *reinterpret_cast<uint4 *>(row + ((kb ^ s) << 4)) = vb;
    }
}

// The scales of a tile's pages, lane i those of page i, on their way while the tile before is converted: the page ids are
// loaded a tile further ahead, so that no load waits for another one.
struct TileScales {
    const float *scales;
    const int *bt;  // the sequence's pages
    int num_blocks, num_kv_heads, head, log2_bs, from, to, lane;  // keys [from, to), tiles of 128 keys
    int pb;
    float k, v;  // 0: no page there
    __device__ __forceinline__ bool has(int j) const {
        const int key = from + j * 128 + (lane << log2_bs);
        return (lane << log2_bs) < 128 && key < to;
    }
    __device__ __forceinline__ void page(int j) {
        pb = has(j) ? __ldg(bt + ((from + j * 128) >> log2_bs) + lane) : 0;
    }
    __device__ __forceinline__ void load(int j) {  // of tile j, whose page ids are here; then the ids of tile j + 1
        k = v = 0.f;
        if (has(j)) {
            const int p = pb < 0 || pb >= num_blocks ? 0 : pb;
            const float *sc = scales + (size_t)p * 2 * num_kv_heads + head;
            k = __ldg(sc);
            v = __ldg(sc + num_kv_heads);
        }
        page(j + 1);
    }
};

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

// decode_int8.cu -- paged_attn_decode over an INT8 cache (one scale per page, K or V, and KV head), head_dim 64 or 128,
// any head grouping, with both contractions on tensor cores.
//
// out = sum_t p_t sv_t c^v_t / sum_t p_t, p_t = 2^(scale log2(e) sk_t (q . c^k_t) - m): sk, sv the scales of the
// token's page, c the codes, m a running maximum per query head (online softmax), the context split over CTAs and merged
// by log-sum-exp.
//
// What it costs. A token and KV head is 2 D bytes of codes (scales: 8 bytes a page), so at the copy rate an SM takes 23.5
// codes a clock, each of which has to become a 16-bit operand. 16 tokens x 8 head slots x 16 dims are one mma.sync
// m16n8k16 in f16. A code becomes f16 by two instructions a pair: c + 128 placed as the low byte of a half of exponent
// 1024 (a byte permute, after one exclusive-or for four codes), then 1152 subtracted: exact. The K scale multiplies the
// FP32 scores. The V scales enter the weights, which go into the product relative to their tile's largest, as an f16
// part and its remainder: the output's rounding is the only 16-bit one on the path, however small weights and scales are.
//
// Structure (persistent, two CTAs an SM, 6 warps each). A unit is (sequence, KV head's query group, split). Warp 4
// streams the unit's tiles of 32 tokens into a ring: page slices of min(bs, 32) rows, each one 5-D TMA box of its K
// rows and its V rows; a slice lies in one page, so its scales are two floats beside it. Tile j is warp j % 4's alone:
// it waits for no other warp, and its two blocks of 16 tokens are two independent chains of ldmatrix, conversion
// and mma. Warp 5 merges the four warps' rows and writes the output or the split's partial.
//
// Operand layouts. ldmatrix (.b16) hands lane (gid, tig) the codes of dims 4 tig .. 4 tig + 3 of a 16-dim chunk: the
// k slots of the A fragment are the permutation {2tig, 2tig+1, 2tig+8, 2tig+9} -> {4tig .. 4tig+3}, and q's B fragment
// is built alike. For P.V, ldmatrix.trans hands a lane (token 2tig: dims 2gid, 2gid+1; token 2tig+1: the same): the
// permute that widens the codes also pairs them by dim, M slot gid holding dim 2gid and slot gid + 8 dim 2gid + 1.
#include <cuda.h>

#include "decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;  // consumer warps
constexpr int kProducerWarp = kWarps;
constexpr int kMergeWarp = kWarps + 1;
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kTile = 32;  // tokens a stage
constexpr int kCtasPerSm = 2;
constexpr float kRescale = 8.0f;  // lazy rescale threshold (log2 units)

template <int D, int G>
struct Int8Layout {
    // ring slots: what two CTAs an SM leave room for beside their merge buffers and unit tables
    static constexpr int kStages = D == 64 ? (G > 4 ? 20 : 22) : (G > 4 ? 10 : 11);
    static constexpr int kMergeBufs = G > 2 ? 1 : 2;
    static constexpr uint32_t kStageBytes = 2 * kTile * D;  // per slice: br K rows, br V rows of D bytes
    static constexpr uint32_t kQBytes = G * D * 2;
    static constexpr uint32_t kQOffset = kStages * kStageBytes;                          // [2]
    static constexpr uint32_t kScaleOffset = kQOffset + 2 * kQBytes;                     // [kStages][4] (K, V) of a slice
    static constexpr uint32_t kBarOffset = kScaleOffset + kStages * 32;
    // full / empty per stage, q full / empty [2], merge full / empty, then the abort flag and the merge buffers' units
    static constexpr uint32_t kMergeOffset = (kBarOffset + (2 * kStages + 4 + 2 * kMergeBufs) * 8 + 32 + 15) / 16 * 16;
    static constexpr uint32_t kMergeFloats = kWarps * G * kMergeRow<D>;
    static constexpr uint32_t kIntsOffset = kMergeOffset + kMergeBufs * kMergeFloats * 4;
    static size_t smem_bytes(int batch, int s_max) {
        return kIntsOffset + unit_table_ints(batch, s_max) * 4 + 1024;  // + 1024-byte alignment slack
    }
};

// Shared-memory address of row t, 16-byte chunk c of rows of D bytes in the swizzled layout that TMA writes (128-byte
// swizzle for rows of 128 bytes, 64-byte for rows of 64).
template <int D>
__device__ __forceinline__ uint32_t swz(uint32_t tile, int t, int c) {
    if (D == 128) return tile + (uint32_t)t * 128u + ((uint32_t)(c ^ (t & 7)) << 4);
    return tile + (uint32_t)t * 64u + ((uint32_t)(c ^ ((t >> 1) & 3)) << 4);
}

// Bytes (codes + 128) a, b of x as two halves 1024 + byte, less 1152: the two codes, exactly.
template <int SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(x, 0x64646464u, SEL)), "r"(0xe480e480u));
    return r;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_int8_kernel(const __grid_constant__ CUtensorMap tm, DecodeArgs a) {
    using L = Int8Layout<D, G>;
    constexpr int S = L::kStages, NB = L::kMergeBufs;
    constexpr int kChunks = D / 16;  // 16-dim chunks: k-steps of q.K^T, m-tiles of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBarOffset);
    uint64_t *empty = full + S;
    uint64_t *qfull = empty + S;     // [2]
    uint64_t *qempty = qfull + 2;    // [2]
    uint64_t *mfull = qempty + 2;    // [NB] the warps' rows of a unit are in buffer i
    uint64_t *mempty = mfull + NB;   // [NB] the merge warp has read buffer i
    volatile int *abort_flag = reinterpret_cast<volatile int *>(mempty + NB);
    int *merge_unit = reinterpret_cast<int *>(mempty + NB) + 4;  // [NB] unit of each merge buffer, -1: end
    float *scales = reinterpret_cast<float *>(smem + L::kScaleOffset);  // [S][4][2]
    float *merge = reinterpret_cast<float *>(smem + L::kMergeOffset);
    const UnitTable ut = unit_table(reinterpret_cast<int *>(smem + L::kIntsOffset), a.batch, a.s_max);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hkv = a.cache.num_kv_heads, bs = a.cache.block_size;
    const int hu = hkv * a.head_groups;  // unit heads
    const int br = bs < kTile ? bs : kTile;  // rows of a slice: splits and tiles start at multiples of 32 tokens

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 2);  // the copies' bytes; the scales
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], kWarps);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&mfull[i], kWarps);
            mbar_init(&mempty[i], 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait();  // lengths, tables, q and the cache may come from the previous kernel
    const int num_units = decode_scan_units<kThreads>(a, ut);
    const int chunk = ut.misc[0];  // the launch's split size

    if (warp == kProducerWarp) {
        // ===================================== producer warp =====================================
        const uint64_t pol = l2_policy_evict_first();
        const uint16_t *qg = static_cast<const uint16_t *>(a.q);
        if (lane == 0) tc::prefetch_tensormap(&tm);
        uint32_t it = 0;  // tiles issued
        uint32_t qn = 0;  // units issued
        bool ok = true;
        UnitCursor c = {};
        PageWindow win = {};
        float k0 = 0.f, v0 = 0.f, k1 = 0.f, v1 = 0.f;  // scales of the window's pages (lane j: pages j and 32 + j)
        auto load_scales = [&](const PageWindow &w, int head) {
            const size_t at0 = (size_t)(unsigned)w.p0 * 2 * hkv + head, at1 = (size_t)(unsigned)w.p1 * 2 * hkv + head;
            if (lane < w.count && (unsigned)w.p0 < (unsigned)a.cache.num_blocks) {
                k0 = __ldg(a.cache.scales + at0);
                v0 = __ldg(a.cache.scales + at0 + hkv);
            } else if (lane < w.count) {  // (flagged and read from page 0)
                k0 = __ldg(a.cache.scales + head);
                v0 = __ldg(a.cache.scales + head + hkv);
            }
            if (lane + 32 < w.count && (unsigned)w.p1 < (unsigned)a.cache.num_blocks) {
                k1 = __ldg(a.cache.scales + at1);
                v1 = __ldg(a.cache.scales + at1 + hkv);
            } else if (lane + 32 < w.count) {
                k1 = __ldg(a.cache.scales + head);
                v1 = __ldg(a.cache.scales + head + hkv);
            }
        };
        if ((int)blockIdx.x < num_units) {
            c = unit_of(blockIdx.x, ut, a.s_max, hu, chunk);
            win = unit_pages(a, c, lane);
            load_scales(win, c.kvh / a.head_groups);
        }
        for (int u = blockIdx.x; ok && u < num_units; u += gridDim.x) {
            // the next unit's cursor and page ids, loading while this unit's copies go out
            UnitCursor cn = c;
            PageWindow wn = win;
            if (u + (int)gridDim.x < num_units) {
                cn = unit_of(u + gridDim.x, ut, a.s_max, hu, chunk);
                wn = unit_pages(a, cn, lane);
            }
            const int kvr = c.kvh / a.head_groups;  // the KV head of this unit
            const int *bt = a.block_tables + (size_t)c.b * a.max_blocks_per_seq;
            const int unit_last_page = (c.t1 - 1) >> a.cache.log2_block_size;
            // q into its slot
            if (!(ok = mbar_wait(&qempty[qn & 1], ((qn >> 1) & 1u) ^ 1u, abort_flag, a.err))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&qfull[qn & 1], L::kQBytes);
                bulk_g2s(smem + L::kQOffset + (qn & 1) * L::kQBytes,
                         qg + ((size_t)ut.qrow[c.b] * a.num_q_heads + (size_t)c.kvh * G) * D, L::kQBytes,
                         &qfull[qn & 1], pol);
            }
            ++qn;
            for (int ts = c.t0; ts < c.t1; ts += kTile, ++it) {
                const int n = min(kTile, c.t1 - ts);
                const int nslices = (n + br - 1) / br;  // <= 4
                const int page0 = ts >> a.cache.log2_block_size;
                const int page_last = (ts + n - 1) >> a.cache.log2_block_size;
                if (page_last >= win.first + win.count) {  // units of more than 64 pages
                    win = load_pages(bt, page0, unit_last_page - page0 + 1, lane);
                    load_scales(win, kvr);
                }
                const int tok0 = ts + lane * br;  // this lane's slice
                const int off = tok0 & (bs - 1);
                const int lp = tok0 >> a.cache.log2_block_size;
                int pb = window_page(win, lp);
                const PageWindow wk = {win.first, win.count, __float_as_int(k0), __float_as_int(k1)};
                const PageWindow wv = {win.first, win.count, __float_as_int(v0), __float_as_int(v1)};
                const int stage = it % S;
                if (lane < nslices && (pb < 0 || pb >= a.cache.num_blocks)) {
                    set_error(a.err, kErrDeviceRange);
                    pb = 0;
                }
                if (!(ok = mbar_wait(&empty[stage], ((it / S) & 1u) ^ 1u, abort_flag, a.err))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], (uint32_t)nslices * br * 2u * D);
                __syncwarp();
                if (lane < nslices)  // one box: the slice's K rows, then its V rows
                    tc::tma_load_5d_hint(smem + (size_t)stage * L::kStageBytes + (size_t)lane * 2 * br * D, &tm, 0, off, kvr, 0,
                                         pb, &full[stage], pol);
                const float sk = __int_as_float(window_page(wk, lp)), sv = __int_as_float(window_page(wv, lp));
                if (lane < nslices) *reinterpret_cast<float2 *>(scales + stage * 8 + lane * 2) = make_float2(sk, sv);
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);
            }
            if (ok && u + (int)gridDim.x < num_units) load_scales(wn, cn.kvh / a.head_groups);
            c = cn;
            win = wn;
        }
        if (!ok) {
            // let copies in flight land before the CTA exits (bounded)
            volatile int no_abort = 0;
            for (uint32_t i = it > (uint32_t)S ? it - S : 0u; i < it; ++i)
                mbar_wait(&full[i % S], (i / S) & 1u, &no_abort, nullptr);
            for (uint32_t i = qn > 2u ? qn - 2 : 0u; i < qn; ++i) mbar_wait(&qfull[i & 1], (i >> 1) & 1u, &no_abort, nullptr);
        }
        return;
    }

    if (warp == kMergeWarp) {
        // ====================================== merge warp ======================================
        merge_warp_loop<D, G, kWarps, NB, true>(a, ut, merge, L::kMergeFloats, mfull, mempty, merge_unit, abort_flag, lane);
        pdl_launch_dependents();
        return;
    }

    // ===================================== consumer warps =====================================
    const int gid = lane >> 2, tig = lane & 3;
    const int mi = lane >> 3;
    const float sl = a.scale * kLog2e;
    const bool bf16 = a.cache.dtype == 1;
    uint32_t bq[kChunks][2];  // q as f16 B fragments, k slots permuted as the K codes
    uint32_t base = 0;        // tiles of the units before this one
    uint32_t qn = 0;
    int mbuf = 0;  // merge buffer of the next unit
    uint32_t mphase = 0;
    // rows of the warp's ldmatrix in the slice layout (slice j starts at row 2 j br): 16 tokens a block
    int trow[2];
#pragma unroll
    for (int bl = 0; bl < 2; ++bl) {
        const int t = bl * 16 + (lane & 7) + 8 * (mi & 1);
        trow[bl] = t + (t & -br);
    }
    for (int u = blockIdx.x; u < num_units; u += gridDim.x) {
        const UnitCursor c = unit_of(u, ut, a.s_max, hu, chunk);
        const int ntiles = (c.t1 - c.t0 + kTile - 1) / kTile;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[kChunks][4];
#pragma unroll
        for (int mt = 0; mt < kChunks; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        if (!mbar_wait(&qfull[qn & 1], (qn >> 1) & 1u, abort_flag, a.err)) return;
        {
            const uint16_t *sq = reinterpret_cast<const uint16_t *>(smem + L::kQOffset + (qn & 1) * L::kQBytes);
#pragma unroll
            for (int kk = 0; kk < kChunks; ++kk) {
                uint2 raw = make_uint2(0u, 0u);
                if (gid < G) raw = *reinterpret_cast<const uint2 *>(sq + gid * D + kk * 16 + 4 * tig);
                if (bf16) {
                    raw = make_uint2(pack_pair<false>(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u)),
                                     pack_pair<false>(__uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)));
                }
                bq[kk][0] = raw.x;
                bq[kk][1] = raw.y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&qempty[qn & 1]);
            ++qn;
        }
        for (int j = warp; j < ntiles; j += kWarps) {
            const uint32_t it = base + j;
            const int stage = it % S;
            const int n = min(kTile, c.t1 - c.t0 - j * kTile);
            if (!mbar_wait(&full[stage], (it / S) & 1u, abort_flag, a.err)) return;
            const uint32_t aK = smem_addr(smem + (size_t)stage * L::kStageBytes), aV = aK + br * D;
            // scales of the four groups of 8 tokens (a group lies in one page)
            float sk[4], sv[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float2 x = *reinterpret_cast<const float2 *>(scales + stage * 8 + (g * 8 / br) * 2);
                sk[g] = x.x * sl;
                sv[g] = x.y;
            }
            // ---- S^T = K q^T: two blocks of 16 tokens x 8 head slots ----
            float s[2][4];
#pragma unroll
            for (int bl = 0; bl < 2; ++bl) {
                s[bl][0] = s[bl][1] = s[bl][2] = s[bl][3] = 0.f;
            }
#pragma unroll
            for (int cp = 0; cp < kChunks; cp += 2) {
                uint32_t r[2][4];
#pragma unroll
                for (int bl = 0; bl < 2; ++bl) ldsm_x4(swz<D>(aK, trow[bl], cp + (mi >> 1)), r[bl]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int bl = 0; bl < 2; ++bl) {
                        const uint32_t x = r[bl][2 * h] ^ 0x80808080u, y = r[bl][2 * h + 1] ^ 0x80808080u;
                        const uint32_t af[4] = {codes_f16<0x4140>(x), codes_f16<0x4140>(y), codes_f16<0x4342>(x),
                                                codes_f16<0x4342>(y)};
                        mma16816<false>(s[bl], af, bq[cp + h][0], bq[cp + h][1]);
                    }
            }
            // token of s[bl][i]: bl * 16 + gid + 8 * (i >> 1); head slot 2 tig + (i & 1)
            bool seen[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) seen[g] = g * 8 + gid < n;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int bl = 0; bl < 2; ++bl)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int g = bl * 2 + (i >> 1);
                    s[bl][i] = seen[g] ? s[bl][i] * sk[g] : -INFINITY;
                    mx[i & 1] = fmaxf(mx[i & 1], s[bl][i]);
                }
#pragma unroll
            for (int ofs = 4; ofs < 32; ofs <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], ofs));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], ofs));
            }
            // The tile's weights are relative to its own maximum and its largest V scale: P' = 2^14 p / 2^mx * sv / w, as
            // an f16 part and its remainder, holds weights down to 2^-38 of the tile's largest. The tile's product
            // then enters O in FP32 times f = 2^(mx - m) w / 2^14; the running max m of a head moves only when a
            // tile's exceeds it by more than 2^8.
            float w = sv[0];
#pragma unroll
            for (int g = 1; g < 4; ++g) w = fmaxf(w, g * 8 < n ? sv[g] : 0.f);
            const float rw = w >= 1.17549435e-38f ? 1.f / w : 0.f;  // (scales below 2^-126 count as 0)
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (mx[i] > m[i] + kRescale) {
                    const float al = ex2f(m[i] - mx[i]);  // 0 when m = -inf
                    l[i] *= al;
#pragma unroll
                    for (int mt = 0; mt < kChunks; ++mt) {
                        o[mt][i] *= al;
                        o[mt][i + 2] *= al;
                    }
                    m[i] = mx[i];
                }
                f[i] = ex2f(mx[i] - m[i]);
            }
            float lt[2] = {0.f, 0.f};
            uint32_t ph[2][2], pe[2][2];
#pragma unroll
            for (int bl = 0; bl < 2; ++bl)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int g = bl * 2 + hf;
                    const float p0 = seen[g] ? ex2f(s[bl][2 * hf] - mx[0]) : 0.f;
                    const float p1 = seen[g] ? ex2f(s[bl][2 * hf + 1] - mx[1]) : 0.f;
                    lt[0] += p0;
                    lt[1] += p1;
                    const float r = seen[g] ? sv[g] * rw * 16384.f : 0.f;
                    uint32_t hi, lo;
                    split_pair<false>(p0 * r, p1 * r, hi, lo);
                    ph[bl][hf] = movmatrix_t(hi);
                    pe[bl][hf] = movmatrix_t(lo);
                }
            l[0] = fmaf(lt[0], f[0], l[0]);
            l[1] = fmaf(lt[1], f[1], l[1]);
            f[0] *= w * (1.f / 16384.f);
            f[1] *= w * (1.f / 16384.f);
            // ---- O^T += f V^T P'^T: D dims (permuted within each 16-dim chunk) x 8 slots ----
#pragma unroll
            for (int cp = 0; cp < kChunks; cp += 2) {
                uint32_t r[2][4];
#pragma unroll
                for (int bl = 0; bl < 2; ++bl) ldsm_x4_t(swz<D>(aV, trow[bl], cp + (mi >> 1)), r[bl]);
                float ot[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) ot[h][0] = ot[h][1] = ot[h][2] = ot[h][3] = 0.f;
#pragma unroll
                for (int bl = 0; bl < 2; ++bl)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = r[bl][2 * h] ^ 0x80808080u, y = r[bl][2 * h + 1] ^ 0x80808080u;
                        const uint32_t af[4] = {codes_f16<0x4240>(x), codes_f16<0x4341>(x), codes_f16<0x4240>(y),
                                                codes_f16<0x4341>(y)};
                        mma16816<false>(ot[h], af, pe[bl][0], pe[bl][1]);
                        mma16816<false>(ot[h], af, ph[bl][0], ph[bl][1]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[cp + h][i] = fmaf(ot[h][i], f[i & 1], o[cp + h][i]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
        }
        base += ntiles;
        // ---- l summed over the lanes of each head slot; rows to the merge warp ----
#pragma unroll
        for (int ofs = 4; ofs < 32; ofs <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], ofs);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], ofs);
        }
        if (!mbar_wait(&mempty[mbuf], mphase ^ 1u, abort_flag, a.err)) return;
        float *rows = merge + (size_t)mbuf * L::kMergeFloats;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int g = 2 * tig + jj;
            if (g < G) {
                float *row = rows + ((size_t)warp * G + g) * kMergeRow<D>;
#pragma unroll
                for (int mt = 0; mt < kChunks; ++mt)  // M slot gid: dim 2gid of the chunk; gid + 8: dim 2gid + 1
                    *reinterpret_cast<float2 *>(row + mt * 16 + 2 * gid) = make_float2(o[mt][jj], o[mt][jj + 2]);
                if (gid == 0) {
                    // (every score NaN: the maximum passed over them; 0 lets the NaN sum through the merge)
                    row[D] = m[jj] == -INFINITY && l[jj] != l[jj] ? 0.f : m[jj];
                    row[D + 1] = l[jj];
                }
            }
        }
        if (warp == 0 && lane == 0) merge_unit[mbuf] = u;
        __syncwarp();
        if (lane == 0) mbar_arrive(&mfull[mbuf]);
        if (++mbuf == NB) {
            mbuf = 0;
            mphase ^= 1u;
        }
    }
    // end marker for the merge warp
    if (mbar_wait(&mempty[mbuf], mphase ^ 1u, abort_flag, a.err)) {
        if (warp == 0 && lane == 0) merge_unit[mbuf] = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&mfull[mbuf]);
    }
    pdl_launch_dependents();
}

template <int D, int G>
cudaError_t launch_g(const DecodeArgs &a, int grid, cudaStream_t s) {
    CUtensorMap tm;
    cudaError_t e = encode_int8_map(a.cache, a.cache.block_size < kTile ? a.cache.block_size : kTile, 2, &tm);
    if (e != cudaSuccess) return e;
    auto kern = decode_int8_kernel<D, G>;
    static DeviceFlags configured;
    const int dev = device_info().device;
    if (!configured.test(dev)) {
        e = set_smem_attributes(kern, device_info().max_smem);
        if (e != cudaSuccess) return e;
        configured.set(dev);
    }
    // two CTAs an SM when both fit in its shared memory (one CTA's maximum plus its 1 KB reserve, each less the
    // reserve); a batch with large unit tables runs one
    const size_t smem = Int8Layout<D, G>::smem_bytes(a.batch, a.s_max);
    const size_t cta_smem = ((size_t)device_info().max_smem + 1024) / kCtasPerSm - 1024;
    const int ctas = smem <= cta_smem ? kCtasPerSm : 1;
    return launch_pdl(kern, dim3(grid * ctas), dim3(kThreads), smem, s, tm, a);
}

template <int D>
cudaError_t launch_d(const DecodeArgs &a, int grid, cudaStream_t s) {
    switch (a.num_q_heads / (a.cache.num_kv_heads * a.head_groups)) {  // query heads per unit
        case 1: return launch_g<D, 1>(a, grid, s);
        case 2: return launch_g<D, 2>(a, grid, s);
        case 3: return launch_g<D, 3>(a, grid, s);
        case 4: return launch_g<D, 4>(a, grid, s);
        case 5: return launch_g<D, 5>(a, grid, s);
        case 6: return launch_g<D, 6>(a, grid, s);
        case 7: return launch_g<D, 7>(a, grid, s);
        case 8: return launch_g<D, 8>(a, grid, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_decode_int8(const DecodeArgs &a, int grid, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    return a.cache.head_dim == 128 ? launch_d<128>(a, grid, s) : launch_d<64>(a, grid, s);
}

}  // namespace pkv

// decode_int8_wide.cu -- paged_attn_decode over an INT8 cache with more than 8 query heads per KV head, head_dim 64 or 128,
// on the 5th-generation tensor cores.
//
// decode_int8.cu's warps convert a tile's codes for 8 heads; 16 or 128 heads would convert (and fetch from L2) the same
// codes again and again. Here a unit's heads, up to 128 of one KV head, are the rows of a tcgen05 product, the codes become
// f16 once, and a key tile costs the same for any number of heads: 32 KB of codes for a product of 1040 clocks.
//
// One CTA (512 threads) a unit (sequence, group of heads, split), two lanes A and B that take the even and the odd 128-key
// tiles, so that one lane's softmax overlaps the other's MMAs:
//   warp 0     TMA producer: the q rows; then each key tile's codes of K and V into one of 4 code buffers;
//   warp 1     TMEM owner and MMA issuer (one thread). S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [384,384+D); P_x
//              over the first 64 columns of S_x. Per tile j of lane x: O_x += P_x V_j, S_x = Q K_{j+2}^T;
//   WG 1, 2    softmax of lane A / B, one head a thread (warps without heads have nothing to do); then B's sums go to A
//              through shared memory, and A writes the output or the split's partial;
//   WG 3       converters, as in prefill_int8.cu: 4 f16 tiles, K and V of each lane.
// Weights are rounded once to f16 in the product with V (half a step, 2^-11 of a weight; 2^7 times themselves, so that
// small ones count), sums are FP32.
//
// 64 sequences x 8192 tokens, 1 KV head (134 MB): 47.5 us with 32 query heads, 56 with 128 (a bf16 cache: 56 and 109). A tile
// takes 2300 cycles, of which the tensor cores work 1040: the four converter warps bound it (1275 of a tile's cycles converting,
// 420 waiting for a tile whose products are not done). K two tiles ahead of V in their order: 54 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include "int8_tiles.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kBM = 128;       // rows of the product: heads of a unit at most
constexpr int kBN = 128;       // keys per tile
constexpr int kRing = 4;       // f16 tiles: K and V of lane A, of lane B
constexpr int kCodes = 4;      // tiles of codes
constexpr int kThreads = 512;
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the max grows by more than 2^8
constexpr float kWeightLog2 = 7.0f;
constexpr uint32_t kColS = 0, kColO = 256;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kTileBytes = kHalves * kTileHalf;  // q, or one f16 K or V tile
    static constexpr uint32_t kCodeBytes = 128 * D;
    static constexpr uint32_t kRingOff = kTileBytes;
    static constexpr uint32_t kCodeOff = kRingOff + kRing * kTileBytes;
    static constexpr uint32_t kBarOff = kCodeOff + kCodes * kCodeBytes;
    static constexpr uint32_t kSmemBytes = kBarOff + 512 + 1024;  // + alignment slack
    static constexpr int kRowFloats = D + 3;  // lane B's rows at the end: O, m, l (over the f16 tiles; odd, so that the
                                              // rows of a warp's threads start in different banks)
    static_assert(kBM * kRowFloats * 4 <= kRing * kTileBytes + kCodes * kCodeBytes, "B's rows fit over tiles and codes");
    static constexpr uint32_t kTmemCols = 512;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    decode_int8_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, DecodeArgs a) {
    using Lay = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem;
    uint8_t *sRing = smem + Lay::kRingOff;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff);
    uint64_t *kv_full = bars;          // [kRing] an f16 tile is ready
    uint64_t *kv_empty = bars + 4;     // [kRing] its MMAs are done
    uint64_t *code_full = bars + 8;    // [kCodes] a tile's codes have landed
    uint64_t *code_empty = bars + 12;  // [kCodes] and have been converted
    uint64_t *s_full = bars + 16;      // [2]
    uint64_t *p_full = bars + 18;      // [2]
    uint64_t *o_done = bars + 20;      // [2]
    uint64_t *q_full = bars + 22;
    uint64_t *q_ready = bars + 23;
    uint64_t *w_ready = bars + 24;
    uint64_t *b_done = bars + 25;      // lane B's rows are in shared memory
    uint64_t *drain = bars + 26;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 27);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 28);
    uint32_t *sMax = reinterpret_cast<uint32_t *>(bars + 29);  // [2] bits of the largest finite K / V scale
    int *sNan = reinterpret_cast<int *>(bars + 30);            // [2] below 2^31 - 1: some page's K / V scale is not finite

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bs = a.cache.block_size, log2_bs = a.cache.log2_block_size, hkv = a.cache.num_kv_heads;
    const int hu = hkv * a.head_groups, G = a.num_q_heads / hu;
    pdl_wait();  // lengths, tables, q and the cache may come from the previous kernel
    // unit: split-major, then sequence, then head group (the groups of a KV head read the same codes at one time)
    const int per_split = a.batch * hu;
    const int split = blockIdx.x / per_split, rest = blockIdx.x - split * per_split;
    const int b = rest / hu, unit = rest - b * hu;
    const int head0 = unit * G, kvr = unit / a.head_groups;
    const int cap = a.max_blocks_per_seq * bs;
    int len = __ldg(a.context_lens + b), qrow = b;
    if (len < 0 || len > cap) {
        if (threadIdx.x == 0) set_error(a.err, kErrDeviceRange);
        len = len < 0 ? 0 : cap;
    }
    if (a.cu_q_lens) {  // mixed batch: only single-row sequences are decoded here
        qrow = __ldg(a.cu_q_lens + b);
        if (__ldg(a.cu_q_lens + b + 1) - qrow != 1) return;
    }
    const int t0 = split * a.chunk;
    if (t0 >= len) return;  // uniform: nothing allocated yet
    const int t1 = min(t0 + a.chunk, len);
    const int n_tiles = (t1 - t0 + kBN - 1) / kBN;
    const int active = (G + 31) / 32;  // softmax warps of a lane that have heads
    const int *bt = a.block_tables + (size_t)b * a.max_blocks_per_seq;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&kv_full[s], 4);
            mbar_init(&kv_empty[s], 1);
            mbar_init(&code_full[s], 1);
            mbar_init(&code_empty[s], 4);
        }
        mbar_init(q_full, 1);
        mbar_init(q_ready, 4);
        mbar_init(w_ready, 4);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], active);
            mbar_init(&o_done[x], 1);
        }
        mbar_init(b_done, active);
        mbar_init(drain, 1);
        *abort_flag = 0;
        sMax[0] = sMax[1] = 0u;
        sNan[0] = sNan[1] = 0x7fffffff;
        fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, Lay::kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        tc::regs_dec<80>();
        if (warp == 0) {
            // ==================================== TMA producer ====================================
            const int box_rows = bs < kBN ? bs : kBN;
            const uint64_t pol = l2_policy_evict_first();
            uint32_t issued = 0;  // items issued (for the abort drain)
            if (lane == 0) {
                tc::prefetch_tensormap(&tm_q);
                tc::prefetch_tensormap(&tm_kv);
                mbar_arrive_expect_tx(q_full, Lay::kTileBytes);
#pragma unroll
                for (int hf = 0; hf < Lay::kHalves; ++hf)  // (rows behind the unit's heads: other heads', or zeros)
                    tc::tma_load_2d(sQ + hf * kTileHalf, &tm_q, hf * 64, qrow * a.num_q_heads + head0, q_full);
            }
            bool ok = true;
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int kv_start = t0 + j * kBN;
                const int n_valid = min(kBN, t1 - kv_start);
                const int npages = bs < kBN ? (n_valid + bs - 1) >> log2_bs : 1;
                const int off = bs < kBN ? 0 : (kv_start & (bs - 1));
                int pb = 0;
                if (lane < npages) {
                    pb = __ldg(bt + (kv_start >> log2_bs) + lane);
                    if (pb < 0 || pb >= a.cache.num_blocks) {
                        set_error(a.err, kErrDeviceRange);
                        pb = 0;
                    }
                }
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t u = 2u * j + kv, slot = u % kCodes, ph = (u / kCodes) & 1u;
                    if (!mbar_wait(&code_empty[slot], ph ^ 1u, abort_flag, a.err)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_expect_tx(&code_full[slot], (uint32_t)npages * box_rows * D);
                    __syncwarp();
                    if (lane < npages)
                        tc::tma_load_5d_hint(smem + Lay::kCodeOff + slot * Lay::kCodeBytes + (uint32_t)lane * box_rows * D, &tm_kv,
                                             0, off, kvr, kv, pb, &code_full[slot], pol);
                    ++issued;
                }
            }
            if (!ok) {
                // let copies in flight land before the CTA exits (bounded)
                volatile int no_abort = 0;
                mbar_wait(q_full, 0, &no_abort, nullptr);
                for (uint32_t u = issued > (uint32_t)kCodes ? issued - kCodes : 0u; u < issued; ++u)
                    mbar_wait(&code_full[u % kCodes], (u / kCodes) & 1u, &no_abort, nullptr);
            }
        } else if (warp == 1) {
            // ===================================== MMA issuer =====================================
            if (tc::elect_one()) {
                const uint32_t id_qk = tc::idesc_f16(false, kBM, kBN, false);
                const uint32_t id_pv = tc::idesc_f16(false, kBM, D, true);
                const uint32_t aQ = smem_addr(sQ), aRing = smem_addr(sRing);
                auto qk = [&](int j) {  // S of lane j & 1 = Q K_j^T
                    const int x = j & 1;
                    const uint32_t aK = aRing + ((2u * j) % kRing) * Lay::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = (uint32_t)(kk >> 2) * kTileHalf + (uint32_t)(kk & 3) * 32u;
                        tc::mma_f16_ss(tmem + kColS + 128u * x, tc::smem_desc(aQ + o, 16, 1024), tc::smem_desc(aK + o, 16, 1024),
                                       id_qk, kk > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(&s_full[x]);
                    tc::mma_commit(&kv_empty[(2u * j) % kRing]);
                };
                auto ring_wait = [&](uint32_t u) {
                    return mbar_wait(&kv_full[u % kRing], (u / kRing) & 1u, abort_flag, a.err);
                };
                bool ok = mbar_wait(q_ready, 0, abort_flag, a.err);
                for (int j = 0; ok && j < 2 && j < n_tiles; ++j) {
                    if (!(ok = ring_wait(2u * j))) break;
                    tc::fence_after_sync();
                    qk(j);
                }
                for (int j = 0; ok && j < n_tiles; ++j) {
                    const int x = j & 1;
                    const uint32_t uV = 2u * j + 1;
                    if (!(ok = ring_wait(uV) && mbar_wait(&p_full[x], (uint32_t)(j >> 1) & 1u, abort_flag, a.err))) break;
                    tc::fence_after_sync();
                    const uint32_t tP = tmem + kColS + 128u * x, tO = tmem + kColO + 128u * x;
                    const uint32_t aV = aRing + (uV % kRing) * Lay::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        // V is [keys x D], D contiguous: MN-major B; 8-key groups 1024 B apart, 64-column halves kTileHalf
                        // apart. P: 16 keys = 8 TMEM columns.
                        tc::mma_f16_ts(tO, tP + 8u * kk, tc::smem_desc(aV + (uint32_t)kk * 2048u, kTileHalf, 1024), id_pv,
                                       (j > 1 || kk > 0) ? 1u : 0u);
                    tc::mma_commit(&o_done[x]);
                    tc::mma_commit(&kv_empty[uV % kRing]);
                    if (j + 2 < n_tiles) {
                        // (the tensor pipe runs the MMAs of this thread in issue order: S_x(j + 2) is written only after
                        // P_x(j) V_j has read P_x(j))
                        if (!(ok = ring_wait(2u * (j + 2)))) break;
                        tc::fence_after_sync();
                        qk(j + 2);
                    }
                }
                tc::mma_commit(drain);
                volatile int no_abort = 0;
                mbar_wait(drain, 0, &no_abort, a.err);
            }
            __syncwarp();
        }
    } else if (warp >= 12) {
        tc::regs_dec<64>();
        // ===================================== converters =====================================
        const int cw = warp - 12;
        page_scales(a.cache.scales, bt, a.cache.num_blocks, hkv, kvr, log2_bs, t0, t1, cw * 32 + lane, sMax, sNan);
        if (lane == 0) mbar_arrive(w_ready);
        __syncwarp();
        bool ok = mbar_wait(q_full, 0, abort_flag, a.err);
        if (BF16 && ok) {
            q_tiles_to_f16(sQ, (int)Lay::kTileBytes / 16, cw * 32 + lane);
            tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(q_ready);
        ok = ok && mbar_wait(w_ready, 0, abort_flag, a.err);
        const float wk = pow2_at_least(__uint_as_float(sMax[0])), wv = pow2_at_least(__uint_as_float(sMax[1]));
        const float ik = wk >= 1.17549435e-38f ? copysignf(1.f / wk, a.scale) : 0.f, iv = wv >= 1.17549435e-38f ? 1.f / wv : 0.f;
        TileScales sc = {a.cache.scales, bt, a.cache.num_blocks, hkv, kvr, log2_bs, t0, t1, lane, 0, 0.f, 0.f};
        sc.page(0);
        sc.load(0);
        for (int j = 0; ok && j < n_tiles; ++j) {
            // f16 factors of the tile's pages; what is not finite counts as 0 here (the rows are made NaN at the end)
            const float fk = sc.k < INFINITY ? sc.k * ik : 0.f, fv = sc.v < INFINITY ? sc.v * iv : 0.f;
            const uint32_t kk = pack_pair<false>(fk, fk), kv2 = pack_pair<false>(fv, fv);
            const bool pow2 = __all_sync(0xffffffffu, ((__float_as_uint(fk) | __float_as_uint(fv)) & 0x7fffffu) == 0u);
            sc.load(j + 1);
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t u = 2u * j + kv, slot = u % kRing, cs = u % kCodes;
                if (!(ok = mbar_wait(&code_full[cs], (u / kCodes) & 1u, abort_flag, a.err))) break;
                if (!(ok = mbar_wait(&kv_empty[slot], ((u / kRing) & 1u) ^ 1u, abort_flag, a.err))) break;
                const uint8_t *codes = smem + Lay::kCodeOff + cs * Lay::kCodeBytes;
                uint8_t *f16 = sRing + slot * Lay::kTileBytes;
                if (pow2) convert_rows<D, true>(codes, f16, cw * 32, kv ? kv2 : kk, log2_bs, lane);
                else convert_rows<D, false>(codes, f16, cw * 32, kv ? kv2 : kk, log2_bs, lane);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&kv_full[slot]);
                    mbar_arrive(&code_empty[cs]);
                }
            }
        }
    } else {
        tc::regs_inc<184>();
        // ================================= softmax + epilogue =================================
        const int x = (warp >> 2) - 1;                 // lane A or B
        const int quarter = warp & 3;                  // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;             // head of the unit
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + kColS + 128u * x + lane_base;
        const uint32_t tO = tmem + kColO + 128u * x + lane_base;
        const int mine = n_tiles > x ? (n_tiles - x + 1) >> 1 : 0;  // tiles of this lane
        if (quarter < active) {
            float m_use = -INFINITY, l = 0.f;
            bool ok = mbar_wait(w_ready, 0, abort_flag, a.err);
            // (never 0, which times a masked score's -inf would be NaN; a negative scale has its sign in K)
            const float wk = pow2_at_least(__uint_as_float(sMax[0]));
            const float c = fmaxf(fabsf(a.scale * kLog2e * (wk > 0.f ? wk : 1.f)), 1.17549435e-38f);
            for (int i = 0; ok && i < mine; ++i) {
                const int kv_start = t0 + (2 * i + x) * kBN;
                if (!(ok = mbar_wait(&s_full[x], (uint32_t)i & 1u, abort_flag, a.err))) break;
                tc::fence_after_sync();
                float s[kBN];
#pragma unroll
                for (int cc = 0; cc < kBN / 32; ++cc)
                    tc::tmem_ld32(tS + cc * 32, *reinterpret_cast<float(*)[32]>(&s[cc * 32]));
                tc::tmem_wait_ld();
                const int lim = t1 - 1 - kv_start;  // last key of this tile
                if (lim < kBN - 1) {
#pragma unroll
                    for (int k = 0; k < kBN; ++k) s[k] = (k <= lim) ? s[k] : -INFINITY;
                }
                float m8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) m8[k] = fmax3(s[k], s[k + 8], s[k + 16]);
#pragma unroll
                for (int q = 24; q < kBN; q += 16)
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], s[q + k], (q + 8 + k < kBN) ? s[q + 8 + k] : -INFINITY);
                const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
                const float m_new = fmaxf(m_use, mx * c);
                const bool grow = m_new > m_use + kRescaleLog2;   // false when m_new = -inf
                const float alpha = grow ? ex2f(m_use - m_new) : 1.f;  // 0 when m_use = -inf
                if (grow) {
                    m_use = m_new;
                    l *= alpha;
                }
                const float neg_m = kWeightLog2 - ((m_use == -INFINITY) ? 0.f : m_use);
                uint32_t pk[kBN / 2];
                float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 c2 = make_float2(c, c), nm2 = make_float2(neg_m, neg_m);
#pragma unroll
                for (int q = 0; q < kBN / 2; ++q) {
                    const float2 xq = ffma2(make_float2(s[2 * q], s[2 * q + 1]), c2, nm2);
                    const float2 e = make_float2(ex2f(xq.x), ex2f(xq.y));
                    l4[q & 3] = fadd2(l4[q & 3], e);
                    pk[q] = pack_pair<false>(e.x, e.y);
                }
                const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
                l += l2.x + l2.y;
                // P_x and O_x are touched only after the lane's last P V is done
                if (i > 0) {
                    if (!(ok = mbar_wait(&o_done[x], (uint32_t)(i - 1) & 1u, abort_flag, a.err))) break;
                    tc::fence_after_sync();
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int cc = 0; cc < D / 32; ++cc) {
                            float o[32];
                            tc::tmem_ld32(tO + cc * 32, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= alpha;
                            tc::tmem_st32(tO + cc * 32, o);
                        }
                    }
                }
#pragma unroll
                for (int cc = 0; cc < kBN / 32; ++cc)
                    tc::tmem_st16(tS + cc * 16, *reinterpret_cast<uint32_t(*)[16]>(&pk[cc * 16]));
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
            // ---- B's rows over the f16 tiles and codes, which every product has read by then; A joins them with its own ----
            float *rowB = reinterpret_cast<float *>(sRing) + (size_t)r * Lay::kRowFloats;
            if (ok && mine > 0) {
                ok = mbar_wait(&o_done[x], (uint32_t)(mine - 1) & 1u, abort_flag, a.err);
                tc::fence_after_sync();
            }
            // (the last product is lane (n_tiles - 1) & 1's: B waits for A's too)
            if (x == 1) {
                const int other = (n_tiles + 1) >> 1;
                ok = ok && mbar_wait(&o_done[0], (uint32_t)(other - 1) & 1u, abort_flag, a.err);
                if (ok) {
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        float o[32];
                        if (mine > 0) {
                            tc::tmem_ld32(tO + cc * 32, o);
                            tc::tmem_wait_ld();
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) rowB[cc * 32 + k] = mine > 0 ? o[k] : 0.f;
                    }
                    rowB[D] = m_use;
                    rowB[D + 1] = l;
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(b_done);
            } else if (ok && mbar_wait(b_done, 0, abort_flag, a.err)) {
                const float mB = rowB[D], lB = rowB[D + 1];
                const float M = fmaxf(m_use, mB);
                const float fa = m_use == -INFINITY ? 0.f : ex2f(m_use - M), fb = mB == -INFINITY ? 0.f : ex2f(mB - M);
                const float sum = l * fa + lB * fb;
                const float nan = __uint_as_float(0x7fc00000u);
                const bool nan_k = sNan[0] != 0x7fffffff, nan_v = sNan[1] != 0x7fffffff;
                const float wv = pow2_at_least(__uint_as_float(sMax[1]));
                // (a split has a key, so the sum is above 0, or NaN; O / sum first, then times Wv: Wv / sum has no normal
                // number where the scales are near 2^-126)
                const float inv = nan_k || nan_v ? nan : 1.f / sum;
                const float lse = nan_k ? nan : (M + (__log2f(sum) - kWeightLog2)) * kLn2;
                const int splits = (len - 1) / a.chunk + 1;
                const size_t head = (size_t)head0 + r;
                const size_t row_o = (size_t)qrow * a.num_q_heads + head;
                const size_t row_p = ((size_t)b * a.num_q_heads + head) * a.s_max + split;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    float o[32];
                    tc::tmem_ld32(tO + cc * 32, o);
                    tc::tmem_wait_ld();
                    if (r < G) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float v[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[k] = (o[8 * q + k] * fa + rowB[cc * 32 + 8 * q + k] * fb) * inv * wv;
                            if (splits == 1) store_out_vec<8>(a.out, row_o * D + cc * 32 + 8 * q, v, a.out_dtype);
                            else store_out_vec<8>(a.part_o, row_p * D + cc * 32 + 8 * q, v, 2);
                        }
                    }
                }
                if (r < G) {
                    if (splits > 1) a.part_lse[row_p] = lse;
                    else if (a.lse) a.lse[row_o] = lse;
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    pdl_launch_dependents();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, Lay::kTmemCols);
    }
}

template <int D, bool BF16>
cudaError_t launch_t(const DecodeArgs &a, cudaStream_t s) {
    using Lay = Layout<D>;
    CUtensorMap tm_q, tm_kv;
    cudaError_t e = encode_rows_map(a.q, BF16 ? 1 : 0, (long long)a.q_rows * a.num_q_heads, D, 64, kBM, &tm_q);
    if (e != cudaSuccess) return e;
    e = encode_int8_map(a.cache, a.cache.block_size < kBN ? a.cache.block_size : kBN, 1, &tm_kv);
    if (e != cudaSuccess) return e;
    auto kern = decode_int8_wide_kernel<D, BF16>;
    static DeviceFlags configured;
    const int dev = device_info().device;
    if (!configured.test(dev)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::kSmemBytes);
        if (e != cudaSuccess) return e;
        configured.set(dev);
    }
    const long long ctas = (long long)a.s_max * a.batch * a.cache.num_kv_heads * a.head_groups;
    if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
    return launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), Lay::kSmemBytes, s, tm_q, tm_kv, a);
}

}  // namespace

cudaError_t launch_decode_int8_wide(const DecodeArgs &a, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    const bool bf16 = a.cache.dtype == 1;
    if (a.cache.head_dim == 128) return bf16 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
    return bf16 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace pkv

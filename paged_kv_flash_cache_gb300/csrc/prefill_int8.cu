// prefill_int8.cu -- paged_attn_prefill over an INT8 cache (one scale per page, K or V, and KV head), head_dim 64 or
// 128: a chunk of queries per sequence against its paged context, causal (bottom-right aligned) or not, on the
// 5th-generation tensor cores.
//
// out = softmax(Q K^T * scale) V with K = sk c^k, V = sv c^v per page. The CTA first finds Wk and Wv, powers of two at or
// above every scale of its pages; the converters then write (sk / Wk) c^k and (sv / Wv) c^v in f16 -- exact for powers of
// two down to 2^-24 of W, else within two half steps of f16 and 2^-24 W times the code --, and Wk goes into the softmax's
// scale, Wv onto the epilogue's O / l. So the softmax and the MMAs are those of a 16-bit cache, and a scale costs one
// packed multiplication per pair of codes, in warps that have time for it.
//
// CTA = 256 query rows of one sequence, as two 128-row tiles A and B that share every K/V tile: 256 tokens of one query head,
// or, for short chunks, of P heads of a KV head's group (a divisor of it; 128 / P tokens a tile, row = token x P + head), whose
// keys are then fetched and converted once. Few blocks over long contexts: a cluster of 2 to 8 CTAs takes a block, a run of its keys
// each, and joins the rows (max, sum, output) over shared memory. A CTA's warps (512 threads, four warpgroups):
//   warp 0     TMA producer: both Q tiles once; then for each 128-key tile the codes of K and of V, each into one of 4
//              code buffers: a lane looks up a page in the block table and issues its box;
//   warp 1     TMEM owner and MMA issuer (one thread). TMEM columns: S_A [0,128), S_B [128,256), O_A [256,256+D),
//              O_B [384,384+D); P_x over the first 64 columns of S_x. Per key tile j: O_A += P_A V_j, S_A = Q_A K_{j+1}^T,
//              O_B += P_B V_j, S_B = Q_B K_{j+1}^T, so one tile's softmax overlaps the other tile's MMAs;
//   WG 1, 2    softmax of tile A / tile B, one query row per thread; epilogue O / l -> out, lse;
//   WG 3       converters: Q to f16 once (a bf16 one), then the code buffers to one of 3 f16 tiles each, 32 rows a warp.
// Conversion in a warpgroup of its own keeps it off the softmax, and code buffers apart from the f16 tiles let four loads
// run ahead of the conversions. The issuing thread is chosen by elect.sync and has 80 registers: whatever delays the next
// MMA delays everything. 4 x 512 queries of 32 heads over 8192 keys: 225 us (1.18 PFLOP/s, 60% of the dense rate); 290 with
// codes converted in place and 48 registers for the issuing warp. The 256 CTAs are 1.7 rounds of the 152 SMs; a pair of tiles
// takes 3080 cycles, 2048 of them in the tensor cores: the issuing thread waits 1150 for the weights (softmax), 210 for
// conversions. P handed over in two halves, the second's exponentials under the first's product: 238 us.
// Short chunks, one sequence of 32 / 8 heads: 16 queries over 16000 keys 35 us (272 with a CTA for each head and 256 rows),
// 256 queries over 16000 keys 73 (207), 16 over 1000 10 (23); 256 queries of 16 heads over 1000 keys 18 (22).
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "cluster.cuh"
#include "int8_tiles.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "prefill_common.cuh"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kBM = 128;       // query rows per tile
constexpr int kRows = 256;     // query rows per CTA (tiles A and B)
constexpr int kBN = 128;       // keys per KV tile
constexpr int kRing = 3;       // f16 K/V tiles
constexpr int kCodes = 4;      // tiles of codes
constexpr int kThreads = 512;  // 4 warpgroups
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the max grows by more than 2^8
// Weights are 2^7 times themselves in the product with V (at most 2^15): f16 has no step below 2^-24, and many small
// weights add up.
constexpr float kWeightLog2 = 7.0f;
constexpr uint32_t kColS = 0, kColO = 256;

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                    // 128-byte swizzle atoms along D
    static constexpr uint32_t kQBytes = kHalves * kTileHalf;  // one 128-row Q tile
    static constexpr uint32_t kKVBytes = kHalves * kTileHalf; // one f16 K or V tile
    static constexpr uint32_t kCodeBytes = 128 * D;           // its codes
    static constexpr uint32_t kRingOff = 2 * kQBytes;
    static constexpr uint32_t kCodeOff = kRingOff + kRing * kKVBytes;
    static constexpr uint32_t kBarOff = kCodeOff + kCodes * kCodeBytes;
    static constexpr uint32_t kSmemBytes = kBarOff + 512 + 1024;  // + alignment slack
    static constexpr uint32_t kTmemCols = 512;
    // a cluster's CTA: its rows at the end, over everything before the barriers: O, max, sum, what is not a number (16-byte
    // stores of 8 threads, a row each, fill all 32 banks)
    static constexpr int kRowFloats = D + 4;
    static_assert(kRows * kRowFloats * 4 <= kBarOff, "the rows fit over tiles and codes");
};

struct Params {
    const int *cu_q_lens, *context_lens, *block_tables;
    int batch, mb, num_q_heads, num_kv_heads, group, bs, log2_bs, num_blocks;
    float scale_log2;
    int causal;
    int pack, tile_tokens;  // heads of a row block, tokens of a tile of it
    int cluster;          // CTAs that share a row block's keys
    int skip_single;      // mixed batch: leave sequences with one query row to the decode kernels
    const float *scales;  // [NB, 2, Hkv]
    void *out;
    int out_dtype;
    float *lse;
    int *err;
};

// BF16: type of q and the default output; the products run in f16. SHORT: blocks of packed heads, of one tile only, or shared
// by a cluster (the other kernel knows that there is none of it: 225 us for the chunks above, 240 with SHORT).
template <int D, bool BF16, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_int8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, Params p) {
    using Lay = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte alignment: the 128-byte swizzle pattern is a function of address bits 4-9.
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem;
    uint8_t *sRing = smem + Lay::kRingOff;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff);
    uint64_t *kv_full = bars;         // [kRing] an f16 tile is ready
    uint64_t *kv_empty = bars + 3;    // [kRing] its MMAs are done
    uint64_t *code_full = bars + 26;  // [kCodes] a tile's codes have landed
    uint64_t *code_empty = bars + 30; // [kCodes] and have been converted
    uint64_t *s_full = bars + 12;   // [2] S_A / S_B computed
    uint64_t *p_full = bars + 14;   // [2] P_A / P_B in TMEM (and O rescaled)
    uint64_t *o_done = bars + 16;   // [2] P V accumulated into O_A / O_B
    uint64_t *q_full = bars + 18;
    uint64_t *q_ready = bars + 19;  // Q converted to f16 (or left as it is)
    uint64_t *w_ready = bars + 20;  // Wk, Wv and the first pages that are not numbers
    uint64_t *drain = bars + 21;    // every MMA issued has completed
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 22);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 23);
    uint32_t *sMax = reinterpret_cast<uint32_t *>(bars + 24);  // [2] bits of the largest finite K / V scale
    int *sNan = reinterpret_cast<int *>(bars + 25);            // [2] first position of a page whose K / V scale is not finite

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // grid (heads, batch, row blocks) with the row blocks last-first: CTAs start in linear order, so
    // the row blocks that see the most keys (causal) start in the first wave and the short ones
    // fill in behind them. A mixed batch: (heads, row blocks last-first, sequences by their rank
    // among those with several query rows), so that no CTA without work precedes one with work.
    const int n_cta = SHORT ? p.cluster : 1, pack = SHORT ? p.pack : 1, tile_tokens = SHORT ? p.tile_tokens : kBM;
    const int rank = n_cta > 1 ? cluster_rank() : 0;
    const int h = (int)blockIdx.x / n_cta * pack;  // the block's first head
    const int mt = p.skip_single ? (int)gridDim.y - 1 - (int)blockIdx.y : (int)gridDim.z - 1 - (int)blockIdx.z;
    pdl_wait();  // lengths, tables, q and the chunk's own K/V may come from the previous kernel
    const int b = p.skip_single ? nth_multi_row_sequence(p.cu_q_lens, p.batch, blockIdx.z) : (int)blockIdx.y;
    if (b < 0) return;  // uniform: past the mixed batch's last chunk
    const int q0 = __ldg(p.cu_q_lens + b);
    const int q_len = __ldg(p.cu_q_lens + b + 1) - q0;
    const int m_start = mt * 2 * tile_tokens;
    if (m_start >= q_len || (p.skip_single && q_len == 1)) return;  // uniform: nothing allocated yet
    const int L = __ldg(p.context_lens + b);
    if (L > p.mb * p.bs || q_len > L || L < 0) {
        if (threadIdx.x == 0) set_error(p.err, kErrDeviceRange);
        return;
    }
    const int tokens = min(2 * tile_tokens, q_len - m_start);
    const bool two = !SHORT || tokens > tile_tokens;    // tile B has rows (or takes part without)
    const int qpos0 = L - q_len + m_start;             // absolute position of row 0
    const int all_end = p.causal ? qpos0 + tokens : L;  // keys [0, all_end) are needed,
    const int per = ((all_end + kBN - 1) / kBN + n_cta - 1) / n_cta * kBN;
    // [kv0, kv_end) by this CTA (maybe none)
    const int kv0 = SHORT ? min(rank * per, all_end) : 0, kv_end = SHORT ? min(kv0 + per, all_end) : all_end;
    const int n_tiles = (kv_end - kv0 + kBN - 1) / kBN;
    const int g = h / p.group;
    const int *bt = p.block_tables + (size_t)b * p.mb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&kv_full[s], 4);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < kCodes; ++s) {
            mbar_init(&code_full[s], 1);
            mbar_init(&code_empty[s], 4);
        }
        mbar_init(q_full, 1);
        mbar_init(q_ready, 4);
        mbar_init(w_ready, 4);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_done[x], 1);
        }
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

    // (a cluster's two barriers, at the end of each role: its registers differ)
    if (warp < 4) {
        tc::regs_dec<80>();
        if (warp == 0) {
            // ==================================== TMA producer ====================================
            const int box_rows = p.bs < kBN ? p.bs : kBN;
            uint32_t issued = 0;  // ring items issued (for the abort drain)
            if (lane == 0) {
                tc::prefetch_tensormap(&tm_q);
                tc::prefetch_tensormap(&tm_kv);
                mbar_arrive_expect_tx(q_full, (uint32_t)((two ? 2 : 1) * tile_tokens * pack) * 128u * Lay::kHalves);
                for (int x = 0; x < (two ? 2 : 1); ++x)
#pragma unroll
                    for (int hf = 0; hf < Lay::kHalves; ++hf)
                        tc::tma_load_3d(sQ + x * Lay::kQBytes + hf * kTileHalf, &tm_q, hf * 64, h,
                                        q0 + m_start + x * tile_tokens, q_full);
            }
            bool ok = true;
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int kv_start = kv0 + j * kBN;
                const int n_valid = min(kBN, L - kv_start);
                const int npages = p.bs < kBN ? (n_valid + p.bs - 1) >> p.log2_bs : 1;
                const int off = p.bs < kBN ? 0 : (kv_start & (p.bs - 1));
                int pb = 0;
                if (lane < npages) {
                    pb = __ldg(bt + (kv_start >> p.log2_bs) + lane);
                    if (pb < 0 || pb >= p.num_blocks) {
                        set_error(p.err, kErrDeviceRange);
                        pb = 0;
                    }
                }
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t u = 2u * j + kv, slot = u % kCodes, ph = (u / kCodes) & 1u;
                    if (!mbar_wait(&code_empty[slot], ph ^ 1u, abort_flag, p.err)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_expect_tx(&code_full[slot], (uint32_t)npages * box_rows * D);
                    __syncwarp();
                    if (lane < npages)
                        tc::tma_load_5d(smem + Lay::kCodeOff + slot * Lay::kCodeBytes + (uint32_t)lane * box_rows * D, &tm_kv, 0,
                                        off, g, kv, pb, &code_full[slot]);
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
            if ((!SHORT || n_tiles > 0) && tc::elect_one()) {
                const uint32_t id_qk = tc::idesc_f16(false, kBM, kBN, false);
                const uint32_t id_pv = tc::idesc_f16(false, kBM, D, true);
                const uint32_t aQ = smem_addr(sQ), aRing = smem_addr(sRing);
                auto ring_wait = [&](uint32_t u) {
                    return mbar_wait(&kv_full[u % kRing], (u / kRing) & 1u, abort_flag, p.err);
                };
                auto qk = [&](int x, uint32_t aK) {
                    const uint32_t aQx = aQ + (uint32_t)x * Lay::kQBytes;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = (uint32_t)(kk >> 2) * kTileHalf + (uint32_t)(kk & 3) * 32u;
                        tc::mma_f16_ss(tmem + kColS + 128u * x, tc::smem_desc(aQx + o, 16, 1024), tc::smem_desc(aK + o, 16, 1024),
                                       id_qk, kk > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(&s_full[x]);
                };
                auto pv = [&](int x, uint32_t aV, int j) {
                    const uint32_t tP = tmem + kColS + 128u * x, tO = tmem + kColO + 128u * x;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk) {
                        // V is [keys x D], D contiguous: MN-major B; 8-key groups 1024 B apart,
                        // 64-column halves kTileHalf apart. P: 16 keys = 8 TMEM columns.
                        tc::mma_f16_ts(tO, tP + 8u * kk, tc::smem_desc(aV + (uint32_t)kk * 2048u, kTileHalf, 1024),
                                       id_pv, (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc::mma_commit(&o_done[x]);
                };
                bool ok = mbar_wait(q_ready, 0, abort_flag, p.err) && ring_wait(0);
                if (ok) {
                    tc::fence_after_sync();
                    qk(0, aRing);  // S_A = Q_A K_0^T
                    if (two) qk(1, aRing);  // S_B = Q_B K_0^T
                    tc::mma_commit(&kv_empty[0]);
                }
                // Ping-pong: tile A's P V_j then its next S, then tile B's. P_x sits in S_x's columns;
                // the tensor pipe runs the MMAs of this thread in issue order, so S_x(j+1) is
                // written only after P_x(j) V_j has read P_x(j).
                for (int j = 0; ok && j < n_tiles; ++j) {
                    const uint32_t uK = 2u * j, uV = uK + 1, uKn = uK + 2;
                    const uint32_t aV = aRing + (uV % kRing) * Lay::kKVBytes;
                    const uint32_t aKn = aRing + (uKn % kRing) * Lay::kKVBytes;
                    const uint32_t ph = (uint32_t)j & 1u;
                    const bool more = j + 1 < n_tiles;
                    if (!(ok = ring_wait(uV) && mbar_wait(&p_full[0], ph, abort_flag, p.err))) break;
                    tc::fence_after_sync();
                    pv(0, aV, j);
                    if (more) {
                        if (!(ok = ring_wait(uKn))) break;
                        qk(0, aKn);
                    }
                    if (two) {
                        if (!(ok = mbar_wait(&p_full[1], ph, abort_flag, p.err))) break;
                        tc::fence_after_sync();
                        pv(1, aV, j);
                    }
                    tc::mma_commit(&kv_empty[uV % kRing]);
                    if (more) {
                        if (two) qk(1, aKn);
                        tc::mma_commit(&kv_empty[uKn % kRing]);
                    }
                }
                tc::mma_commit(drain);
                volatile int no_abort = 0;
                mbar_wait(drain, 0, &no_abort, p.err);
            }
            __syncwarp();
        }
        if (n_cta > 1) {
            cluster_barrier();
            cluster_barrier();
        }
    } else if (warp >= 12) {
        tc::regs_dec<64>();
        // ===================================== converters =====================================
        const int cw = warp - 12;
        // ---- Wk, Wv over the pages of keys [0, kv_end); a page id outside the pool: page 0, as the producer reads it ----
        {
            page_scales(p.scales, bt, p.num_blocks, p.num_kv_heads, g, p.log2_bs, kv0, kv_end, cw * 32 + lane, sMax, sNan);
            if (lane == 0) mbar_arrive(w_ready);
            __syncwarp();
        }
        bool ok = true;
        if (BF16) {
            // q to f16 in place (exact for |q| within f16's range)
            ok = mbar_wait(q_full, 0, abort_flag, p.err);
            if (ok) {
                q_tiles_to_f16(sQ, (two ? 2 : 1) * (int)Lay::kQBytes / 16, cw * 32 + lane);
                tc::fence_proxy_async_smem();
            }
        } else {
            ok = mbar_wait(q_full, 0, abort_flag, p.err);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(q_ready);
        ok = ok && mbar_wait(w_ready, 0, abort_flag, p.err);
        const float wk = pow2_at_least(__uint_as_float(sMax[0])), wv = pow2_at_least(__uint_as_float(sMax[1]));
        const float ik = wk >= 1.17549435e-38f ? copysignf(1.f / wk, p.scale_log2) : 0.f, iv = wv >= 1.17549435e-38f ? 1.f / wv : 0.f;
        // (pages behind kv_end: no row's weight is above 0, and W does not know them: 0, lest a factor overflow f16)
        TileScales sc = {p.scales, bt, p.num_blocks, p.num_kv_heads, g, p.log2_bs, kv0, kv_end, lane, 0, 0.f, 0.f};
        sc.page(0);
        sc.load(0);
        for (int j = 0; ok && j < n_tiles; ++j) {
            // f16 factors of the tile's pages; what is not finite counts as 0 here (its rows are made NaN at the end)
            const float fk = sc.k < INFINITY ? sc.k * ik : 0.f, fv = sc.v < INFINITY ? sc.v * iv : 0.f;
            const uint32_t kk = pack_pair<false>(fk, fk), kv2 = pack_pair<false>(fv, fv);
            // (every factor of the tile a power of two, as kv_cache_append makes them)
            const bool pow2 = __all_sync(0xffffffffu, ((__float_as_uint(fk) | __float_as_uint(fv)) & 0x7fffffu) == 0u);
            sc.load(j + 1);
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t u = 2u * j + kv, slot = u % kRing, cs = u % kCodes;
                if (!(ok = mbar_wait(&code_full[cs], (u / kCodes) & 1u, abort_flag, p.err))) break;
                if (!(ok = mbar_wait(&kv_empty[slot], ((u / kRing) & 1u) ^ 1u, abort_flag, p.err))) break;
                const uint8_t *codes = smem + Lay::kCodeOff + cs * Lay::kCodeBytes;
                uint8_t *f16 = sRing + slot * Lay::kKVBytes;
                if (pow2) convert_rows<D, true>(codes, f16, cw * 32, kv ? kv2 : kk, p.log2_bs, lane);
                else convert_rows<D, false>(codes, f16, cw * 32, kv ? kv2 : kk, p.log2_bs, lane);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&kv_full[slot]);
                    mbar_arrive(&code_empty[cs]);
                }
            }
        }
        if (n_cta > 1) {
            cluster_barrier();
            cluster_barrier();
        }
    } else {
        tc::regs_inc<184>();
        // ================================= softmax + epilogue =================================
        const int x = (warp >> 2) - 1;                 // 0: tile A, 1: tile B
        const int quarter = warp & 3;                  // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;             // row within the tile
        const int tile_rows = (x == 0 ? min(tokens, tile_tokens) : tokens - tile_tokens) * pack;
        const bool row_ok = r < tile_rows;
        const bool warp_ok = !SHORT || quarter * 32 < tile_rows;  // (uniform)
        const int token = x * tile_tokens + r / pack;  // of the block
        const int qpos = qpos0 + token;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + kColS + 128u * x + lane_base;   // S_x, and P_x over its first 64 columns
        const uint32_t tO = tmem + kColO + 128u * x + lane_base;
        float m_use = -INFINITY, l = 0.f;
        bool ok = mbar_wait(w_ready, 0, abort_flag, p.err);
        // (never 0, which times a masked score's -inf would be NaN; a negative scale has its sign in K)
        const float wk = pow2_at_least(__uint_as_float(sMax[0]));
        const float c = fmaxf(fabsf(p.scale_log2 * (wk > 0.f ? wk : 1.f)), 1.17549435e-38f);
        for (int j = 0; ok && j < n_tiles && (x == 0 || two); ++j) {
            const int kv_start = kv0 + j * kBN;
            const uint32_t ph = (uint32_t)j & 1u;
            if (!(ok = mbar_wait(&s_full[x], ph, abort_flag, p.err))) break;
            tc::fence_after_sync();
            if (!warp_ok) {  // (a product's row touches no other row: what these hold does not matter)
                tc::fence_before_sync();
                if (lane == 0) mbar_arrive(&p_full[x]);
                continue;
            }
            float s[kBN];
#pragma unroll
            for (int cc = 0; cc < kBN / 32; ++cc)
                tc::tmem_ld32(tS + cc * 32, *reinterpret_cast<float(*)[32]>(&s[cc * 32]));
            tc::tmem_wait_ld();
            // last key index this row may see in this tile (below 0: none; a row behind the last one: as the last)
            int lim = L - 1 - kv_start;
            if (p.causal) lim = min(lim, qpos - kv_start);
            if (lim < kBN - 1) {
#pragma unroll
                for (int i = 0; i < kBN; ++i) s[i] = (i <= lim) ? s[i] : -INFINITY;
            }
            // row max as 8 independent chains (two warps per scheduler cannot hide a 64-deep chain)
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = fmax3(s[k], s[k + 8], s[k + 16]);
#pragma unroll
            for (int i = 24; i < kBN; i += 16)
#pragma unroll
                for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], s[i + k], (i + 8 + k < kBN) ? s[i + 8 + k] : -INFINITY);
            const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
            const float m_new = fmaxf(m_use, mx * c);
            const bool grow = m_new > m_use + kRescaleLog2;   // false when m_new = -inf
            const float alpha = grow ? ex2f(m_use - m_new) : 1.f;  // 0 when m_use = -inf
            if (grow) {
                m_use = m_new;
                l *= alpha;
            }
            // masked entries are -inf; m_use is finite for a row with a visible key, and a row
            // without one (padding row) uses 0 so that exp2(-inf) = 0 instead of a NaN
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
            // P_x and O_x are touched only after P_x V_{j-1} is done
            if (j > 0) {
                if (!(ok = mbar_wait(&o_done[x], (uint32_t)(j - 1) & 1u, abort_flag, p.err))) break;
                tc::fence_after_sync();
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        float o[32];
                        tc::tmem_ld32(tO + cc * 32, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= alpha;
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
        // ---- epilogue: O / l; of a cluster's CTA: O, max and sum to its shared memory, once every product is done ----
        const int last = p.causal ? qpos : L - 1;
        const float nan = __uint_as_float(0x7fc00000u);
        // a row that sees a key of a page whose scale is not finite is NaN
        const bool nan_k = last >= sNan[0], nan_v = last >= sNan[1];
        // (O / l first, then times Wv: Wv / l has no normal number where the scales are near 2^-126)
        const float wv = pow2_at_least(__uint_as_float(sMax[1])), over_l = l == 0.f ? 0.f : 1.f / l;  // (a NaN sum stays one)
        if (n_cta > 1) {
            float *out_row = reinterpret_cast<float *>(smem) + (size_t)(x * kBM + r) * Lay::kRowFloats;
            if (ok && n_tiles > 0)
                ok = mbar_wait(&o_done[0], (uint32_t)(n_tiles - 1) & 1u, abort_flag, p.err) &&
                     (!two || mbar_wait(&o_done[1], (uint32_t)(n_tiles - 1) & 1u, abort_flag, p.err));
            else if (ok)
                ok = mbar_wait(q_ready, 0, abort_flag, p.err);  // (no keys: q is still on its way to where the rows go)
            tc::fence_after_sync();
            if (ok && warp_ok) {
                if (n_tiles > 0) {
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        float o[32];
                        tc::tmem_ld32(tO + cc * 32, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(out_row + cc * 32 + i) =
                                make_float4(o[i] * over_l * wv, o[i + 1] * over_l * wv, o[i + 2] * over_l * wv, o[i + 3] * over_l * wv);
                    }
                }
                *reinterpret_cast<float4 *>(out_row + D) = make_float4(m_use, l, nan_k ? 2.f : nan_v ? 1.f : 0.f, 0.f);
            }
        } else if (ok && warp_ok && mbar_wait(&o_done[x], (uint32_t)(n_tiles - 1) & 1u, abort_flag, p.err)) {
            tc::fence_after_sync();
            const float inv = nan_k || nan_v ? nan : over_l;
            const size_t orow = (size_t)(q0 + m_start + token) * p.num_q_heads + h + r % pack;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                tc::tmem_ld32(tO + cc * 32, o);
                tc::tmem_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = o[8 * i + k] * inv * wv;
                        store_out_vec<8>(p.out, orow * D + cc * 32 + 8 * i, v, p.out_dtype);
                    }
                }
            }
            if (row_ok && p.lse)
                p.lse[orow] = nan_k ? nan : l == 0.f ? -INFINITY : (m_use + (__log2f(l) - kWeightLog2)) * kLn2;
        }
        if (n_cta > 1) {
            // ---- the cluster's rows: row i by a softmax warp of CTA i % cluster; every CTA comes here, whatever its waits did ----
            cluster_barrier();
            if (!*abort_flag) {
                // as many rows at a time as make 8 (row, CTA) pairs, whose loads are in flight together; lanes 8 r + i: the
                // max and sum of the batch's row r in CTA i
                const int batch = 8 / n_cta, step = 8 * n_cta;
                const int rows = two ? kBM + (tokens - tile_tokens) * pack : tokens * pack;
                auto has = [&](int row) { return row < rows && (row & (kBM - 1)) < tile_tokens * pack; };
                for (int r0 = (warp - 4) * n_cta + rank; r0 < rows; r0 += batch * step) {
                    const float *first = reinterpret_cast<const float *>(smem);
                    const int lr = r0 + (lane >> 3) * step, li = lane & 7;
                    float m = -INFINITY, l = 0.f, bad = 0.f;
                    if ((lane >> 3) < batch && has(lr) && li < n_cta) {
                        float x4[4];
                        ld_cluster(smem_of(first + (size_t)lr * Lay::kRowFloats + D, li), x4);
                        m = x4[0], l = x4[1], bad = x4[2];
                    }
                    float v[8][D / 32];
#pragma unroll
                    for (int k = 0, r = 0, i = 0; k < 8; ++k) {
                        const int at_row = r0 + r * step;
                        if (r < batch && has(at_row)) {
                            ld_cluster(smem_of(first + (size_t)at_row * Lay::kRowFloats + lane * (D / 32), i), v[k]);
                        }
                        if (++i == n_cta) i = 0, ++r;
                    }
                    float M = m;
#pragma unroll
                    for (int i = 4; i > 0; i >>= 1) {
                        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
                        bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, i));
                    }
                    float w = m == -INFINITY ? 0.f * l : ex2f(m - M) * l, sum = w;  // (0 times a NaN sum: NaN)
#pragma unroll
                    for (int i = 4; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
                    w = sum != 0.f ? w / sum : 0.f;  // shares of the row: nothing is above the largest value
                    float acc[D / 32];
#pragma unroll
                    for (int k = 0, r = 0, i = 0; k < 8; ++k) {
                        const int at_row = r0 + r * step;
                        const float wk = __shfl_sync(0xffffffffu, w, (8 * r + i) & 31);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            if (i == 0) acc[c] = 0.f;
                            if (wk != 0.f) acc[c] = fmaf(wk, v[k][c], acc[c]);  // (0: nothing there, or nothing of it left)
                        }
                        if (++i == n_cta) {
                            const float s = __shfl_sync(0xffffffffu, sum, (8 * r) & 31), b8 = __shfl_sync(0xffffffffu, bad, (8 * r) & 31);
                            const float top = __shfl_sync(0xffffffffu, M, (8 * r) & 31);
                            if (r < batch && has(at_row)) {
                                const int tr = at_row & (kBM - 1), tok = (at_row / kBM) * tile_tokens + tr / pack;
                                const size_t orow = (size_t)(q0 + m_start + tok) * p.num_q_heads + h + tr % pack;
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) acc[c] = b8 > 0.f ? nan : acc[c];
                                store_out_vec<D / 32>(p.out, orow * D + lane * (D / 32), acc, p.out_dtype);
                                if (lane == 0 && p.lse) p.lse[orow] = b8 > 1.f ? nan : (top + (__log2f(s) - kWeightLog2)) * kLn2;
                            }
                            i = 0, ++r;
                        }
                    }
                }
            }
            cluster_barrier();  // (no CTA leaves before its rows have been read)
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

// Heads of a row block: the largest divisor of a group with which chunks of max_q_len tokens fit one block.
int pack_heads(int group, int max_q_len) {
    int n = 1;
    for (int d = 2; d <= group && d <= kBM; ++d)
        if (group % d == 0 && 2 * (kBM / d) >= max_q_len) n = d;
    return n;
}

template <int D, bool BF16, bool SHORT>
auto configured_kernel(cudaError_t &e) {
    auto kern = prefill_int8_kernel<D, BF16, SHORT>;
    static DeviceFlags configured;
    const int dev = device_info().device;
    e = cudaSuccess;
    if (!configured.test(dev)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::kSmemBytes);
        if (e == cudaSuccess) configured.set(dev);
    }
    return kern;
}

// Clusters of 1 to 8 CTAs, an SM each, that the device runs at once (a cluster lies in one GPC, so that a few SMs stay out):
// asked once a device.
template <int D, bool BF16>
cudaError_t clusters_at_once(int (&out)[9]) {
    static int table[64][9];
    static DeviceFlags known;
    static std::mutex filling;
    cudaError_t e;
    auto kern = configured_kernel<D, BF16, true>(e);
    if (e != cudaSuccess) return e;
    const int dev = device_info().device;
    if (!known.test(dev)) {
        out[0] = 0;
        out[1] = device_info().num_sms;
        for (int n = 2; n <= 8; ++n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)n);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = Layout<D>::kSmemBytes;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)n;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if ((e = cudaOccupancyMaxActiveClusters(&out[n], kern, &cfg)) != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) {
            std::lock_guard<std::mutex> lock(filling);
            for (int n = 0; n <= 8; ++n) table[dev][n] = out[n];
            known.set(dev);
        }
        return cudaSuccess;
    }
    for (int n = 0; n <= 8; ++n) out[n] = table[dev][n];
    return cudaSuccess;
}

// CTAs of a cluster that share a row block's keys, by the time that the launch takes for full tables: rounds of clusters, each a
// share of the key tiles and what a CTA costs besides (kStart tiles' time; kJoin more for a cluster: 100 queries over 500 keys
// take 14.8 us in clusters or not).
int cluster_of(long long blocks, long long capacity, const int (&at_once)[9]) {
    constexpr long long kStart = 5, kJoin = 4;
    const long long tiles = (capacity + kBN - 1) / kBN;
    int best = 1;
    long long best_cost = -1;
    for (int n = 1; n <= 8; ++n) {
        if (at_once[n] <= 0) continue;
        const long long cost = (blocks + at_once[n] - 1) / at_once[n] * ((tiles + n - 1) / n + kStart + (n > 1 ? kJoin : 0));
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = n;
        }
    }
    return best;
}

template <int D, bool BF16>
cudaError_t launch_t(const PrefillArgs &a, cudaStream_t stream) {
    Params p;
    p.group = a.num_q_heads / a.cache.num_kv_heads;
    p.pack = pack_heads(p.group, a.max_q_len);
    p.tile_tokens = kBM / p.pack;
    const int block = 2 * p.tile_tokens;  // tokens of a row block
    const unsigned row_blocks = (unsigned)((a.max_q_len + block - 1) / block), heads = (unsigned)(a.num_q_heads / p.pack);
    const long long by_grid = (long long)a.batch * row_blocks, by_rows = (long long)a.total_q / block + a.batch;
    int at_once[9];
    cudaError_t e = clusters_at_once<D, BF16>(at_once);
    if (e != cudaSuccess) return e;
    p.cluster = cluster_of(heads * (by_grid < by_rows ? by_grid : by_rows), (long long)a.max_blocks_per_seq * a.cache.block_size,
                           at_once);
    CUtensorMap tm_q, tm_kv;
    e = encode_q_group_map(a.q, BF16 ? 1 : 0, a.total_q, a.num_q_heads, D, p.pack, p.tile_tokens, &tm_q);
    if (e != cudaSuccess) return e;
    e = encode_int8_map(a.cache, a.cache.block_size < kBN ? a.cache.block_size : kBN, 1, &tm_kv);
    if (e != cudaSuccess) return e;
    p.cu_q_lens = a.cu_q_lens;
    p.context_lens = a.context_lens;
    p.block_tables = a.block_tables;
    p.batch = a.batch;
    p.mb = a.max_blocks_per_seq;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.cache.num_kv_heads;
    p.bs = a.cache.block_size;
    p.log2_bs = a.cache.log2_block_size;
    p.num_blocks = a.cache.num_blocks;
    p.scale_log2 = a.scale * kLog2e;
    p.causal = a.causal;
    p.skip_single = a.skip_single;
    p.scales = a.cache.scales;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.lse = a.lse;
    p.err = a.err;
    const bool is_short = p.cluster > 1 || p.pack > 1 || a.max_q_len <= kBM;
    auto kern = is_short ? configured_kernel<D, BF16, true>(e) : configured_kernel<D, BF16, false>(e);
    if (e != cudaSuccess) return e;
    const unsigned x = heads * (unsigned)p.cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = a.skip_single ? dim3(x, row_blocks, a.batch) : dim3(x, a.batch, row_blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tm_q, tm_kv, p);
}

}  // namespace

cudaError_t launch_prefill_int8(const PrefillArgs &a, cudaStream_t s) {
    const bool bf16 = a.cache.dtype == 1;
    if (a.cache.head_dim == 128) return bf16 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
    return bf16 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace pkv

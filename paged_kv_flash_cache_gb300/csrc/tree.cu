// tree.cu -- paged_attn_tree: the drafted tokens of each sequence, a tree (or any set) of n_b nodes whose
// keys and values are the sequence's last n_b cached tokens, attend to the paged context before them and,
// among themselves, to the nodes that a bit mask gives each (its ancestors and itself).
//
// Mathematics: node i of sequence b sees position p when p < L_b - n_b, or when bit p - (L_b - n_b) of its
// mask row is set; out = softmax over what it sees of (q . k * scale), times V ("为什么Attention是O(n²)",
// mathematics section), keys read through the block table ("企业官网建设流程全解析", section 2.1; layout of
// "Flash Attention与Paged Attention如何共同优化大模型推理？", section 3) in one pass with that page's
// section 2 running max and sum.
//
// Rows: the query heads of a KV head read the same keys, so the rows of a product are (node, head of the
// group): 128 of them a tile, whole nodes. S = Q K^T and O += P V are tcgen05.mma with M = 128.
//
// Two lanes, each with an output and two score buffers of 64 keys in TMEM (head_dim up to 128) and a warpgroup
// for its softmax; K and V come in tiles of 128 keys, once for both:
//   wide    a block of more than 128 rows: lane A its first 128 rows, lane B the others, both over every key;
//   narrow  up to 128 rows: both lanes the same rows, lane A the first 64 keys of each tile, lane B the other
//           64, their (max, sum, output) joined at the end.
// At head_dim 256 the output takes half of TMEM: one lane, 64-key tiles. While a lane's softmax works on one
// score buffer its next 64 keys' Q K^T fills the other: Q K(u + 1) is issued before P V(u). (With one buffer of
// 128 keys a lane the chain softmax - P V - Q K - softmax, 5100 cycles a tile of a wide block, bounded the kernel.)
//
// Work: the (sequence, KV head, row block) items, laid end to end in key tiles (an item weighs kItemCost tiles more for
// its set-up and output), are cut into equal runs, one a CTA (one CTA an SM): any mix of lengths fills the GPU
// evenly, an item is split only where a run ends, and a CTA leaves at most two partial items, so the workspace does
// not grow with the batch. A merge kernel joins the partials of each split item in the order of the keys (no atomics:
// the same result every time).
//
// Warps: 0 loads Q and the K tiles, 3 the V tiles by TMA into a ring, 1 issues the MMAs and owns TMEM, 2 walks the run
// and hands its segments to the others, the warpgroups of lanes A and B do softmax and output.
//
// P goes to the tensor cores as its 16-bit rounding plus the rounding's remainder (two products), so that it is not a
// rounding to 16 bits. Two exceptions round it once, by half a step of the 16-bit type: wide blocks with a 16-bit output,
// which the chain of products and softmax bounds (a 63-node batch: 90 us with two parts, 75 with one; the prefill's choice
// too), and FP8 caches, whose codes are far coarser.
//
// An FP8 cache: the codes land where the tile's second half goes (head_dim 64: apart) and become 16-bit values in place,
// exactly: the keys' by a warpgroup of their own, with their row scales on the scores in FP32; the values' by the softmax
// warps, times their scales' powers of two, what the scales are above those going to the weights before P's one rounding.
// Bound by the chain of conversion and softmax in the same warps.
//
// Measured, main kernel and merge, back to back (of the copy rate):
//   16 sequences x 64 nodes, 32 KV heads x 128, contexts 1k-8k in pages of 16 (1.02 GB): 165 us, 91%, bound by HBM;
//     over an FP8 cache (0.54 GB) 209 us
//   25 nodes of 32 / 8 heads over 131k tokens in pages of 64 (0.54 GB): 98 us, 81%, the merge 8 us of it; FP8 117 us
//   32 sequences x 63 nodes of 32 / 8 heads, contexts to 8k (0.27 GB, 252 rows a KV head): 75 us, 53%, bound by the wide
//     chain (about 3800 cycles a tile, of them 2560 in the tensor cores) and the merge, 13 us; FP8 117 us
//   8 sequences x 31 nodes at head_dim 256 (0.16 GB): 38 us, 62%: its 64-key tiles at the copy rate (2400 cycles each), the
//     rest set-up, output and merge of short runs
// A partial's rows go out at 29 to 53 bytes a cycle and SM, all SMs at once (L2's write rate): 5000 to 10000 cycles a run.
//
// Rows that see nothing (a padded node): 0 and -inf. Masked keys: their scores are replaced, never
// multiplied, so that K may hold anything; V rows beyond the context are zeroed in shared memory, and a
// drafted token's V is swept for infinities and NaN, since 0 * inf would reach rows that do not see it:
// they are zeroed for the product and, for the rows that do see them, put back in the output.
#include <cuda.h>

#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kBM = 128;              // rows of a tile
constexpr float kRescaleLog2 = 8.0f;  // O is rescaled when the running max grows by more than 2^8
// f16 weights (and with them the sum and the output, which the quotient takes out again) are 2^kUp times themselves: f16 has no
// step below 2^-24, and of a long context keys that far below the largest weight can be as much as the rest together. Up to
// 2^8 (kRescaleLog2) times that they stay within 2^15; over FP8 the V scales' rests, below 2^3 for scales below 2^10, do too.
template <bool BF16, bool FP8>
constexpr float kUp = BF16 ? 0.f : FP8 ? 4.f : 7.f;
constexpr int kSegs = 4;              // segments handed out ahead
// An item's set-up and output, in key tiles: about 11000 cycles against the 3800 of a wide block's tile at head_dim 128, where it
// was measured. The other kernels use it too, though it fits them less well (head_dim 256: 64-key tiles of 2400 cycles), so
// that their runs are less evenly cut.
constexpr int kItemCost = 3;
constexpr int kMinTiles = 2;          // work of a run at least, in key tiles (4: 16.2 us for 15.6, 16 nodes over 4k tokens)

// One run's part of an item: key tiles [t0, t1) of nodes [node0, node0 + nodes) of one sequence and KV
// head (or share of its group). nodes = 0 ends the run.
struct Segment {
    int b, q0, n, len;       // sequence, its first row of q, nodes, cached tokens (drafted ones included)
    int unit, node0, nodes;  // unit head, first node, nodes of this row block
    int t0, t1;
    int slot;  // -1: the whole item (the output is final); else the CTA's partial 0 or 1
    int pad[2];
};

template <int D, bool FP8>
struct TreeLayout {
    static constexpr int kLanes = D <= 128 ? 2 : 1;
    static constexpr int kBN = D <= 128 ? 128 : 64;  // keys a tile
    static constexpr int kSub = 64;                  // keys of a score buffer
    static constexpr int kHalves = D / 64;           // 128-byte swizzle atoms along D
    static constexpr uint32_t kQHalf = kBM * 128;
    static constexpr uint32_t kQBytes = kHalves * kQHalf;
    static constexpr uint32_t kTileHalf = kBN * 128;
    static constexpr uint32_t kTileBytes = kHalves * kTileHalf;  // a K or a V tile
    // ring slots; a launch whose blocks are all narrow has one more in the place of lane B's Q tile
    static constexpr int kRing = D == 64 && !FP8 ? 8 : 4;
    static constexpr int kRingMax = kRing + (kLanes == 2 ? 1 : 0);
    static_assert(kLanes == 1 || kQBytes == kTileBytes, "a Q tile's place is a ring slot's");
    // output rows on their way out, kStageRow bytes of each: 4 (FP8: 2) KB a softmax warp
    static constexpr uint32_t kStageRow = FP8 ? 64 : 128;
    static constexpr uint32_t kStageOff = kLanes * kQBytes + kRing * kTileBytes;
    static constexpr uint32_t kStageEnd = kStageOff + 4 * kLanes * 32 * kStageRow;
    static_assert(32 * kStageRow >= 2 * 32 * 8, "two (max, sum) of a warp's rows fit in its stage");
    // FP8: the row scales of the ring's tiles, and of the last four K tiles (a ring slot may be refilled while its scores
    // are still in the softmax); head_dim 64: the codes of the ring's tiles (head_dim 128: in the tile's second half)
    static constexpr uint32_t kScaleOff = kStageEnd;
    static constexpr uint32_t kKScaleOff = kScaleOff + (FP8 ? kRingMax * 512u : 0u);
    static constexpr uint32_t kCodeOff = kKScaleOff + (FP8 ? 4 * 512u : 0u);
    static constexpr uint32_t kBarOff = kCodeOff + (FP8 && D == 64 ? kRingMax * kBN * 64u : 0u);
    static constexpr uint32_t kSegOff = kBarOff + 640;
    static constexpr uint32_t kSmem = kSegOff + kSegs * sizeof(Segment) + 1024;  // + alignment slack
    static constexpr int kThreads = 128 * (1 + kLanes + (FP8 ? 1 : 0));  // FP8: a warpgroup for the keys' codes
    // TMEM: score buffer i of lane x at 128 i + 64 x (P in its place), O of lane x at 256 + 128 x
    static constexpr uint32_t kColO = 256;
};

// What a run works on, from the lengths on the device; false (flagged) if they are out of range.
struct SeqWork {
    int q0, n, len;
    int tiles, blocks;  // key tiles, row blocks
};

// Work of one unit (KV head) of a sequence, in key tiles: an item costs its tiles and kItemCost for its set-up,
// refill of the pipeline and output.
__device__ __forceinline__ long long seq_cost(const SeqWork &w) {
    return w.blocks > 0 ? (long long)(w.tiles + kItemCost) * w.blocks : 0;
}

__device__ __forceinline__ SeqWork seq_work(const TreeArgs &a, int b, int bn, bool flag) {
    SeqWork w;
    const int q1 = __ldg(a.cu_q_lens + b + 1);
    w.q0 = __ldg(a.cu_q_lens + b);
    w.len = __ldg(a.context_lens + b);
    w.n = q1 - w.q0;
    w.tiles = w.blocks = 0;
    const bool ok = w.q0 >= 0 && q1 >= w.q0 && q1 <= a.total_q && w.n <= a.max_q_len && w.len >= w.n &&
                    w.len <= (a.max_blocks_per_seq << a.cache.log2_block_size);
    if (!ok) {
        if (flag) set_error(a.err, kErrDeviceRange);
        w.n = 0;
    }
    if (w.n > 0) {
        w.tiles = (w.len + bn - 1) / bn;
        w.blocks = (w.n + a.block_nodes - 1) / a.block_nodes;
    }
    return w;
}

// 32 mask bits of a row for keys j .. j + 31 of the tree (j may be negative: context, seen by all; bits at
// or behind n are not set).
__device__ __forceinline__ uint32_t mask_word(const uint32_t *row, int w, int n) {
    if (w < 0) return 0xffffffffu;
    const int left = n - 32 * w;
    if (left <= 0) return 0u;
    const uint32_t x = __ldg(row + w);
    return left < 32 ? x & ((1u << left) - 1u) : x;
}

template <bool BF16>
__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
    constexpr uint32_t m = BF16 ? 0x7f80u : 0x7c00u;
    return (w & m) == m || ((w >> 16) & m) == m;
}

template <bool BF16>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
    constexpr uint32_t m = BF16 ? 0x7f80u : 0x7c00u;
    if ((w & m) == m) w &= 0xffff0000u;
    if (((w >> 16) & m) == m) w &= 0x0000ffffu;
    return w;
}

// What rounding to 16 bits left of a pair (hi: the rounded pair), itself rounded to 16 bits.
template <bool BF16>
__device__ __forceinline__ uint32_t remainder_pair(float a, float b, uint32_t hi) {
    if constexpr (BF16) return pack_pair<true>(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_pair<false>(a - f.x, b - f.y);
}

// E4M3 codes as 16-bit values, exactly: cvt to f16, for bf16 on through FP32 (16 x 64 nodes: 209 us; 279 with the codes' bits
// moved into place by integer instructions, which read a NaN as 480). A NaN code (0x7f, 0xff) is a NaN. V: times a power of
// two, a pair of it in `factor` (see split_scale).
template <bool BF16, bool V>
__device__ __forceinline__ uint32_t code_pair(uint32_t codes, uint32_t factor) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)codes));
    if constexpr (BF16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        r = pack_pair<true>(f.x, f.y);
        if constexpr (V) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(factor));
    } else {
        if constexpr (V) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(factor));
    }
    return r;
}

// Eight codes (8 bytes) as 16-bit values: K as they are, V times `factor`.
template <bool BF16, bool V>
__device__ __forceinline__ uint4 values_of(const uint2 &codes, uint32_t factor) {
    return make_uint4(code_pair<BF16, V>(codes.x & 0xffffu, factor), code_pair<BF16, V>(codes.x >> 16, factor),
                      code_pair<BF16, V>(codes.y & 0xffffu, factor), code_pair<BF16, V>(codes.y >> 16, factor));
}

// A V row's scale as 2^e times the rest: the power of two goes to the values (`factor` for code_pair), the rest to the
// weights. e is held to where factor and values are numbers of the 16-bit type: [-22, 7] (f16), [-100, 7] (bf16). The rest is
// in [1, 2) for scales there, above 2 for scales from 2^8 on: bf16's exponents have room for it, f16's up to scales of 2^10
// (f16 values have scales up to 147). Values are exact but for f16 and e < -15, where they round as subnormals do, by 2^-25 at
// most: 2^-11.8 of the row's largest, 448 x 2^e. A scale that is not finite: values that are not.
template <bool BF16>
__device__ __forceinline__ uint32_t split_scale(float scale, float &rest) {
    const uint32_t bits = __float_as_uint(scale);
    const int biased = (int)(bits >> 23) & 255;
    if (biased == 255) {
        rest = 1.f;
        return pack_pair<BF16>(scale, scale);
    }
    const int e = min(max(biased - 127, BF16 ? -100 : -22), 7);
    rest = scale * __uint_as_float((uint32_t)(127 - e) << 23);
    const float power = __uint_as_float((uint32_t)(127 + e) << 23);
    return pack_pair<BF16>(power, power);
}

template <bool BF16>
__device__ __forceinline__ bool nonfinite8(const uint4 &v) {
    return nonfinite_pair<BF16>(v.x) || nonfinite_pair<BF16>(v.y) || nonfinite_pair<BF16>(v.z) || nonfinite_pair<BF16>(v.w);
}

template <bool BF16>
__device__ __forceinline__ uint4 drop_nonfinite8(const uint4 &v) {
    return make_uint4(drop_nonfinite<BF16>(v.x), drop_nonfinite<BF16>(v.y), drop_nonfinite<BF16>(v.z), drop_nonfinite<BF16>(v.w));
}

// FP8: a warp's kRows rows of a ring tile, rows `first` on, codes to 16-bit values in the layout that TMA writes for a
// 16-bit cache. Both exactly: K the codes' own values (the row scales multiply the scores), V times their scales' powers
// of two (the scales' rests, left in the scales' place, multiply the weights). Rows from n_valid on (beyond the context)
// become 0; what is not finite in a V row from `drafted` on becomes 0. Returns whether there was any of that.
template <int D, bool BF16, bool V, int kRows>
__device__ __forceinline__ bool convert_rows(uint8_t *tile, const uint8_t *codes64, float *sc, int first, int n_valid,
                                             int drafted, int lane) {
    using L = TreeLayout<D, true>;
    // head_dim 128: 8 lanes a row of codes, which lie where the second half of the row's values goes (the warp reads its
    // rows before it writes any); of 8 lanes, lanes 4-7 take row r ^ 5 of the chunks that lanes 0-3 take of row r: neither
    // their reads nor their writes meet in a bank then. head_dim 64: 4 lanes a row, the codes in a place of their own.
    constexpr int kSteps = kRows * D / 512;
    const int c = D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3, hf = c >> 2, k0 = 2 * (c & 3);
    const int r8 = D == 128 ? (lane >> 4) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    auto row_of = [&](int i) { return first + (D == 128 ? 8 * (i >> 1) + (r8 ^ (2 * (i & 1))) : 8 * i + r8); };
    uint4 raw[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int row = row_of(i);
        raw[i] = *reinterpret_cast<const uint4 *>(D == 128 ? tile + L::kTileHalf + row * 128 + ((c ^ (row & 7)) << 4)
                                                           : codes64 + row * 64 + c * 16);
    }
    uint32_t factor[kSteps];
    float rest = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) factor[i] = V ? split_scale<BF16>(sc[row_of(i)], rest) : 0u;
    if (V && lane < kRows) split_scale<BF16>(sc[first + lane], rest);
    __syncwarp();
    if (V && lane < kRows) sc[first + lane] = rest;
    bool bad = false;
    auto run = [&](auto has_tail) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int row = row_of(i);
            uint4 v0 = values_of<BF16, V>(make_uint2(raw[i].x, raw[i].y), factor[i]);
            uint4 v1 = values_of<BF16, V>(make_uint2(raw[i].z, raw[i].w), factor[i]);
            if constexpr (decltype(has_tail)::value) {
                if (row >= n_valid) {
                    v0 = v1 = make_uint4(0, 0, 0, 0);
                } else if (V && row >= drafted && (nonfinite8<BF16>(v0) || nonfinite8<BF16>(v1))) {
                    v0 = drop_nonfinite8<BF16>(v0);
                    v1 = drop_nonfinite8<BF16>(v1);
                    bad = true;
                }
            }
            uint8_t *dst = tile + hf * L::kTileHalf + row * 128;
            *reinterpret_cast<uint4 *>(dst + ((k0 ^ (row & 7)) << 4)) = v0;
            *reinterpret_cast<uint4 *>(dst + (((k0 + 1) ^ (row & 7)) << 4)) = v1;
        }
    };
    if (n_valid < L::kBN || (V && drafted < L::kBN)) run(std::true_type{});
    else run(std::false_type{});
    return bad;
}

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(TreeLayout<D, FP8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, TreeArgs a) {
    using L = TreeLayout<D, FP8>;
    static_assert(!FP8 || D <= 128, "an FP8 cache has head_dim 64 or 128");
    constexpr int kBN = L::kBN, kSub = L::kSub, kLanes = L::kLanes, kRingMax = L::kRingMax;
    const bool all_narrow = kLanes == 2 && a.max_q_len <= a.tile_nodes;
    const uint32_t ring = all_narrow ? kRingMax : L::kRing;
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte alignment: the 128-byte swizzle pattern is a function of address bits 4-9.
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem;
    uint8_t *sRing = smem + (all_narrow ? 1 : kLanes) * L::kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *kv_full = bars;                 // [kRingMax]
    uint64_t *kv_empty = kv_full + kRingMax;  // [kRingMax]
    uint64_t *q_full = kv_empty + kRingMax;   // a segment's Q tiles have landed
    uint64_t *q_empty = q_full + 1;        // its QK products are done
    uint64_t *s_full = q_empty + 1;        // [2] score buffer i of the lanes computed
    uint64_t *p_full = s_full + 2;         // [2] P written over it
    uint64_t *pv_late = p_full + 2;        // the segment's last P V but one is done
    uint64_t *o_done = pv_late + 1;        // every P V of the segment is done
    uint64_t *o_empty = o_done + 1;        // its outputs are read
    uint64_t *ml_full = o_empty + 1;       // narrow: (max, sum) handed over
    uint64_t *seg_full = ml_full + 1;      // [kSegs]
    uint64_t *seg_empty = seg_full + kSegs;
    uint64_t *drain = seg_empty + kSegs;   // every MMA issued has completed
    uint64_t *conv_full = drain + 1;       // FP8: [kRingMax] a tile's codes are 16-bit values
    unsigned long long *s_total = reinterpret_cast<unsigned long long *>(conv_full + kRingMax);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_total + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *s_poison = abort_flag + 1;  // [4] by segment: V of a drafted token was not finite
    Segment *segs = reinterpret_cast<Segment *>(smem + L::kSegOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gu = a.unit_heads;  // query heads of a unit
    constexpr int kSoftmaxWarps = 4 * kLanes;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRingMax; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
            mbar_init(&conv_full[i], kSoftmaxWarps);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kSoftmaxWarps);
        }
        mbar_init(pv_late, 1);
        mbar_init(o_done, 1);
        mbar_init(o_empty, kSoftmaxWarps);
        mbar_init(ml_full, kSoftmaxWarps);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 3 + kSoftmaxWarps + (FP8 ? 4 : 0));  // producers, MMA, softmax, conversion
        }
        mbar_init(drain, 1);
        *s_total = 0;
        *abort_flag = 0;
        s_poison[0] = s_poison[1] = s_poison[2] = s_poison[3] = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // lengths, tables, masks, q and the drafted K / V may come from the previous kernel

    // the whole batch's key tiles, and this CTA's run of them
    {
        long long mine = 0;
        for (int b = threadIdx.x; b < a.batch; b += L::kThreads) {
            const SeqWork w = seq_work(a, b, kBN, blockIdx.x == 0);
            mine += seq_cost(w);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0 && mine) atomicAdd(s_total, (unsigned long long)mine);
    }
    __syncthreads();
    const long long total = (long long)*s_total * a.units;
    long long run = (total + gridDim.x - 1) / gridDim.x;
    if (run < kMinTiles) run = kMinTiles;

    // segment seg_i of the run; it stays in shared memory until every role has arrived on seg_empty
    uint32_t seg_i = 0;
    auto next_segment = [&]() -> bool {
        return mbar_wait(&seg_full[seg_i % kSegs], (seg_i / kSegs) & 1u, abort_flag, a.err) &&
               segs[seg_i % kSegs].nodes > 0;
    };

    if (warp < 4) {
        if constexpr (kLanes == 2) tc::regs_dec<72>();
        if (warp == 0 || warp == 3) {
            // ======================= TMA producers: Q and the K tiles (warp 0), the V tiles (warp 3) =======================
            // Two warps, since issuing the boxes of a tile's pages takes about 50 cycles a box: at 16 tokens a page one
            // warp spent 1300 cycles an item, which bounded the kernel. Page ids are read 32 at a time, one window ahead.
            const int kv = warp == 0 ? 0 : 1;
            const int bs = a.cache.block_size, lbs = a.cache.log2_block_size;
            const int box_rows = bs < kBN ? bs : kBN;
            const uint64_t pol = l2_policy_evict_first();
            if (tc::elect_one()) {
                if (kv == 0) tc::prefetch_tensormap(&tm_q);
                tc::prefetch_tensormap(&tm_kv);
            }
            uint32_t qn = 0;
            uint32_t base = 0, base_ph = 1;  // ring slot of the segment's first item, and the parity to find on kv_empty
            uint32_t slot = 0, ph = 1;
            uint32_t used = 0, par = 0;  // slots this warp has loaded into, and the parity of each one's last load
            uint32_t items = 0;          // items of the run, up to ring
            bool ok = true;
            for (; (ok = next_segment()); ++seg_i) {
                const Segment s = segs[seg_i % kSegs];
                const bool wide = kLanes == 2 && s.nodes > a.tile_nodes;
                const int T = s.t1 - s.t0, ahead = wide ? 1 : min(2, T);
                const int kvh = s.unit / a.head_groups;
                const int *bt = a.block_tables + (size_t)s.b * a.max_blocks_per_seq;
                const int last_page = (min(s.t1 * kBN, s.len) - 1) >> lbs;
                // ids of pages first + lane (a tile's pages never straddle two windows)
                auto window = [&](int first) -> int {
                    int pb = 0;
                    if (first + lane <= last_page) {
                        pb = __ldg(bt + first + lane);
                        if (pb < 0 || pb >= a.cache.num_blocks) {
                            set_error(a.err, kErrDeviceRange);
                            pb = 0;
                        }
                    }
                    return pb;
                };
                int first = (s.t0 * kBN) >> lbs;
                int w0 = window(first), w1 = first + 32 <= last_page ? window(first + 32) : 0;
                if (kv == 0) {
                    // Q: the block's nodes, gu heads each, one box per tile and 64 columns
                    if (!(ok = mbar_wait(q_empty, (qn & 1u) ^ 1u, abort_flag, a.err))) break;
                    if (tc::elect_one()) {
                        const int tiles = wide ? 2 : 1;
                        mbar_arrive_expect_tx(q_full, (uint32_t)tiles * a.tile_nodes * gu * 128u * L::kHalves);
                        for (int x = 0; x < tiles; ++x)
#pragma unroll
                            for (int hf = 0; hf < L::kHalves; ++hf)
                                tc::tma_load_3d(sQ + x * L::kQBytes + hf * L::kQHalf, &tm_q, hf * 64, s.unit * gu,
                                                s.q0 + s.node0 + x * a.tile_nodes, q_full);
                    }
                    ++qn;
                }
                // ring order = the order of use: K of the first `ahead` tiles, then V_j, K_{j + ahead}, and the last V
                slot = base;
                ph = base_ph;
                auto step = [&](uint32_t n) {
                    slot += n;
                    if (slot >= ring) {
                        slot -= ring;
                        ph ^= 1u;
                    }
                };
                if (kv) step((uint32_t)ahead);
                for (int j = 0; j < T; ++j) {
                    if (j > 0) step(kv ? (ahead + j <= T ? 2u : 1u) : (j < ahead ? 1u : 2u));
                    const int start = (s.t0 + j) * kBN, page0 = start >> lbs;
                    const int npages = bs < kBN ? (min(kBN, s.len - start) + bs - 1) >> lbs : 1;
                    const int off = bs < kBN ? 0 : (start & (bs - 1));
                    if (page0 >= first + 32) {
                        first += 32;
                        w0 = w1;
                        if (first + 32 <= last_page) w1 = window(first + 32);
                    }
                    if (!(ok = mbar_wait(&kv_empty[slot], ph, abort_flag, a.err))) break;
                    uint8_t *dst = sRing + slot * L::kTileBytes;
                    if constexpr (FP8) {
                        // one box row of codes and a scale a token
                        dst = D == 128 ? dst + L::kTileHalf : smem + L::kCodeOff + slot * (kBN * 64u);
                        float *dst_sc = reinterpret_cast<float *>(smem + L::kScaleOff) + slot * 128u;
                        if (tc::elect_one()) mbar_arrive_expect_tx(&kv_full[slot], (uint32_t)npages * box_rows * (D + 4u));
                        for (int pg = 0; pg < npages; ++pg, dst += (uint32_t)box_rows * D, dst_sc += box_rows) {
                            const int pb = __shfl_sync(0xffffffffu, w0, page0 - first + pg);
                            const int row = ((pb * 2 + kv) * a.cache.num_kv_heads + kvh) * bs + off;
                            if (tc::elect_one()) {
                                tc::tma_load_2d_hint(dst, &tm_kv, 0, row, &kv_full[slot], pol);
                                bulk_g2s(dst_sc, a.cache.scales + row, (uint32_t)box_rows * 4u, &kv_full[slot], pol);
                            }
                        }
                    } else {
                        if (tc::elect_one())
                            mbar_arrive_expect_tx(&kv_full[slot], (uint32_t)npages * box_rows * 128u * L::kHalves);
                        for (int pg = 0; pg < npages; ++pg, dst += (uint32_t)box_rows * 128u) {
                            const int pb = __shfl_sync(0xffffffffu, w0, page0 - first + pg);
                            const int row = ((pb * 2 + kv) * a.cache.num_kv_heads + kvh) * bs + off;
                            if (tc::elect_one()) {
#pragma unroll
                                for (int hf = 0; hf < L::kHalves; ++hf)
                                    tc::tma_load_2d_hint(dst + hf * L::kTileHalf, &tm_kv, hf * 64, row, &kv_full[slot], pol);
                            }
                        }
                    }
                    used |= 1u << slot;
                    par = (par & ~(1u << slot)) | ((ph ^ 1u) << slot);
                }
                if (!ok) break;
                items = min(ring, items + 2u * (uint32_t)T);
                base += 2u * (uint32_t)T;
                if ((base / ring) & 1u) base_ph ^= 1u;
                base %= ring;
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[seg_i % kSegs]);
            }
            // Every copy lands before the CTA exits. At the end of the run warp 3, whose item is the last, waits for
            // the last item of every slot; a warp that gave up in between waits for its own (a slot that the other
            // one has loaded since shows another parity: a short limit).
            volatile int no_abort = 0;
            if (*abort_flag) {
                for (uint32_t i = 0; i < ring; ++i)
                    if ((used >> i) & 1u) mbar_wait(&kv_full[i], (par >> i) & 1u, &no_abort, nullptr, 10000000ull);
            } else if (kv == 1) {
                for (; items > 0; --items) {
                    if (base == 0) {
                        base = ring;
                        base_ph ^= 1u;
                    }
                    --base;
                    mbar_wait(&kv_full[base], base_ph ^ 1u, &no_abort, nullptr);
                }
            }
            if (qn > 0) mbar_wait(q_full, (qn - 1) & 1u, &no_abort, nullptr);
        } else if (warp == 1) {
            // ====================================== MMA issuer ======================================
            if (tc::elect_one()) {
                const uint32_t id_sub = tc::idesc_f16(BF16, kBM, kSub, false), id_tile = tc::idesc_f16(BF16, kBM, kBN, false);
                const uint32_t id_pv = tc::idesc_f16(BF16, kBM, D, true);
                const uint32_t aQ = smem_addr(sQ), aRing = smem_addr(sRing);
                // (a descriptor's address field counts 16 bytes and has room for all of shared memory: the steps
                // along it are additions)
                const uint64_t dK0 = tc::smem_desc(aRing, 16, 1024), dQ0 = tc::smem_desc(aQ, 16, 1024);
                const uint64_t dV0 = tc::smem_desc(aRing, L::kTileHalf, 1024);
                uint32_t slot = 0, ph = 0;  // ring position
                uint32_t g = 0;             // score buffers that each lane has used
                uint64_t *const tile_full = FP8 ? conv_full : kv_full;  // the ring's tiles as the products read them
                auto advance = [&]() {
                    if (++slot == ring) {
                        slot = 0;
                        ph ^= 1u;
                    }
                };
                // score buffer i: the lanes' Q K of the K tile in ring slot sl. Wide: 64 of its keys (`half`) for each
                // lane's rows; else the tile's keys for the one set of rows, the halves of 128 landing in the lanes'
                // (neighbouring) buffers.
                auto qk = [&](bool wide, uint32_t sl, uint32_t half, uint32_t i) {
                    uint64_t dK = dK0 + sl * (L::kTileBytes >> 4) + half * (kSub * 128 >> 4), dQ = dQ0;
                    const uint32_t idesc = wide ? id_sub : id_tile;
                    uint32_t tS = tmem + 128u * i;
#pragma unroll 1
                    for (int x = 0; x < (wide ? 2 : 1); ++x, dQ += L::kQBytes >> 4, tS += 64u)
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc::mma_f16_ss(tS, dQ + (((kk >> 2) * L::kQHalf + (kk & 3) * 32u) >> 4),
                                           dK + (((kk >> 2) * L::kTileHalf + (kk & 3) * 32u) >> 4), idesc, kk > 0 ? 1u : 0u);
                    tc::mma_commit(&s_full[i]);
                };
                // O (+)= P V of score buffer i: the V tile in ring slot sl, wide: its 64 keys `half` for both lanes, else
                // a half for each lane. 16 keys a step: 8 columns of P in their 32-column chunk, the remainders 16 behind.
                auto pv = [&](bool wide, bool two_parts, uint32_t sl, uint32_t half, uint32_t i, bool first) {
                    uint64_t dV = dV0 + sl * (L::kTileBytes >> 4) + half * (kSub * 128 >> 4);
                    uint32_t tO = tmem + L::kColO, tP = tmem + 128u * i;
#pragma unroll 1
                    for (int x = 0; x < kLanes; ++x, tO += 128u, tP += 64u) {
                        if (two_parts) {
#pragma unroll
                            for (int kk = 0; kk < kSub / 16; ++kk) {
                                const uint32_t tPk = tP + 32u * (kk >> 1) + 8u * (kk & 1);
                                const uint64_t dVk = dV + (uint32_t)(kk * 2048 >> 4);
                                tc::mma_f16_ts(tO, tPk, dVk, id_pv, (first && kk == 0) ? 0u : 1u);
                                tc::mma_f16_ts(tO, tPk + 16u, dVk, id_pv, 1u);
                            }
                        } else {
#pragma unroll
                            for (int kk = 0; kk < kSub / 16; ++kk)
                                tc::mma_f16_ts(tO, tP + 32u * (kk >> 1) + 8u * (kk & 1), dV + (uint32_t)(kk * 2048 >> 4), id_pv,
                                               (first && kk == 0) ? 0u : 1u);
                        }
                        if (!wide) dV += kSub * 128 >> 4;
                    }
                };
                auto wait = [&](uint64_t *bar, uint32_t par) { return mbar_wait(bar, par, abort_flag, a.err); };
                bool ok = true;
                for (; (ok = next_segment()); ++seg_i) {
                    const Segment &s = segs[seg_i % kSegs];
                    const int T = s.t1 - s.t0;
                    // A lane's work is U score buffers: wide, both halves of every tile; else a tile each. Step u: Q K of
                    // buffer u + 1, then P V of buffer u. (A buffer's Q K follows its last P V in issue order.) The ring
                    // holds the tiles in this order of use: wide K_0, V_0, K_1, V_1 ..., else K_0, K_1, V_0, K_2, V_1 ...
                    const bool wide = kLanes == 2 && s.nodes > a.tile_nodes;
                    if (!(ok = wait(q_full, seg_i & 1u))) break;
                    tc::fence_after_sync();
                    if (wide) {
                        const bool two_parts = !FP8 && a.out_dtype == 2;
                        if (!(ok = wait(&tile_full[slot], ph))) break;
                        qk(true, slot, 0, g & 1u);
                        for (int j = 0; j < T; ++j) {
                            // buffers 2 j (the tile's first half), 2 j + 1
                            qk(true, slot, 1, (g + 1u) & 1u);
                            tc::mma_commit(&kv_empty[slot]);
                            if (j == T - 1) tc::mma_commit(q_empty);  // the segment's last Q K
                            advance();
                            if (!(ok = wait(&tile_full[slot], ph) && wait(&p_full[g & 1u], (g >> 1) & 1u))) break;
                            // a segment's first P V overwrites an output: the last segment's must be read
                            if (j == 0 && !(ok = wait(o_empty, (seg_i & 1u) ^ 1u))) break;
                            tc::fence_after_sync();
                            pv(true, two_parts, slot, 0, g & 1u, j == 0);
                            const uint32_t v_slot = slot;
                            advance();
                            if (j + 1 < T) {
                                if (!(ok = wait(&tile_full[slot], ph))) break;
                                qk(true, slot, 0, g & 1u);
                            } else {
                                tc::mma_commit(pv_late);
                            }
                            ++g;
                            if (!(ok = wait(&p_full[g & 1u], (g >> 1) & 1u))) break;
                            tc::fence_after_sync();
                            pv(true, two_parts, v_slot, 1, g & 1u, false);
                            tc::mma_commit(&kv_empty[v_slot]);
                            ++g;
                        }
                    } else {
                        if (!(ok = wait(&tile_full[slot], ph))) break;
                        qk(false, slot, 0, g & 1u);
                        tc::mma_commit(&kv_empty[slot]);
                        if (T == 1) tc::mma_commit(q_empty);
                        advance();
                        for (int j = 0; j < T; ++j, ++g) {
                            if (j + 1 < T) {
                                if (!(ok = wait(&tile_full[slot], ph))) break;
                                qk(false, slot, 0, (g + 1u) & 1u);
                                tc::mma_commit(&kv_empty[slot]);
                                if (j + 2 == T) tc::mma_commit(q_empty);
                                advance();
                            }
                            if (!(ok = wait(&tile_full[slot], ph) && wait(&p_full[g & 1u], (g >> 1) & 1u))) break;
                            if (j == 0 && !(ok = wait(o_empty, (seg_i & 1u) ^ 1u))) break;
                            tc::fence_after_sync();
                            pv(false, !FP8, slot, 0, g & 1u, j == 0);
                            tc::mma_commit(&kv_empty[slot]);
                            if (j + 2 == T) tc::mma_commit(pv_late);
                            advance();
                        }
                    }
                    if (!ok) break;
                    tc::mma_commit(o_done);
                    mbar_arrive(&seg_empty[seg_i % kSegs]);
                }
                tc::mma_commit(drain);
                volatile int no_abort = 0;
                mbar_wait(drain, 0, &no_abort, a.err);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ================================== walk of the run ==================================
            const long long begin = run * blockIdx.x, end = min(total, begin + run);
            uint32_t n = 0;
            bool ok = true;
            MergeItem left = {};  // the item that begins in this run and goes on in the next ones
            auto publish = [&](const Segment &s) -> bool {
                if (!mbar_wait(&seg_empty[n % kSegs], ((n / kSegs) & 1u) ^ 1u, abort_flag, a.err)) return false;
                if (lane == 0) {
                    segs[n % kSegs] = s;
                    mbar_arrive(&seg_full[n % kSegs]);
                }
                ++n;
                return true;
            };
            long long before = 0;  // work of the sequences passed
            for (int b0 = 0; ok && b0 < a.batch && before < end; b0 += 32) {
                SeqWork w = {0, 0, 0, 0, 0};
                if (b0 + lane < a.batch) w = seq_work(a, b0 + lane, kBN, false);
                const long long mine = seq_cost(w) * a.units;
                long long scan = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, scan, o);
                    if (lane >= o) scan += y;
                }
                const long long first = before + scan - mine, last = before + scan;
                unsigned hit = __ballot_sync(0xffffffffu, mine > 0 && first < end && last > begin);
                before += __shfl_sync(0xffffffffu, scan, 31);
                while (ok && hit) {
                    const int src = __ffs(hit) - 1;
                    hit &= hit - 1;
                    Segment s = {};
                    s.b = b0 + src;
                    s.q0 = __shfl_sync(0xffffffffu, w.q0, src);
                    s.n = __shfl_sync(0xffffffffu, w.n, src);
                    s.len = __shfl_sync(0xffffffffu, w.len, src);
                    const long long s0 = __shfl_sync(0xffffffffu, first, src), s1 = __shfl_sync(0xffffffffu, last, src);
                    const int tiles = __shfl_sync(0xffffffffu, w.tiles, src);
                    const int blocks = __shfl_sync(0xffffffffu, w.blocks, src);
                    const int cost = tiles + kItemCost;
                    // the sequence's items (a unit's row blocks one after the other: the second finds the keys in
                    // L2) that this run meets, from the one that `begin` falls into
                    const int it0 = begin > s0 ? (int)((begin - s0) / cost) : 0;
                    s.unit = it0 / blocks;
                    int blk = it0 - s.unit * blocks;
                    for (long long at = s0 + (long long)it0 * cost; ok && at < min(end, s1); at += cost) {
                        // an item's first kItemCost units of work stand for its set-up and output
                        s.t0 = (int)max(0ll, begin - at - kItemCost);
                        s.t1 = (int)min((long long)tiles, end - at - kItemCost);
                        if (s.t1 > s.t0) {
                            s.node0 = blk * a.block_nodes;
                            s.nodes = min(a.block_nodes, s.n - s.node0);
                            s.slot = s.t0 > 0 ? 0 : (s.t1 < tiles ? 1 : -1);
                            if (s.slot == 1) {
                                left.q0 = s.q0;
                                left.node0 = s.node0;
                                left.nodes = s.nodes;
                                left.unit = s.unit;
                                left.parts = (int)((at + cost - 1) / run - blockIdx.x) + 1;  // to its last tile's run
                            }
                            ok = publish(s);
                        }
                        if (++blk == blocks) {
                            blk = 0;
                            ++s.unit;
                        }
                    }
                }
            }
            if (lane == 0) a.merge[blockIdx.x] = left;
            if (ok) publish(Segment{});
        }
    } else if (FP8 && warp >= 12) {
        // ============================ FP8: the K tiles' codes to 16-bit values ============================
        if constexpr (FP8) {
            tc::regs_dec<96>();
            uint32_t slot = 0, par = 0;  // ring slot and parity of the K tile in work
            uint32_t tiles = 0;          // key tiles so far
            auto step = [&](uint32_t n) {
                slot += n;
                if (slot >= ring) {
                    slot -= ring;
                    par ^= 1u;
                }
            };
            for (; next_segment(); ++seg_i) {
                const Segment &s = segs[seg_i % kSegs];
                const bool wide = s.nodes > a.tile_nodes;
                const int T = s.t1 - s.t0, ahead = wide ? 1 : min(2, T), first = (warp - 12) * 32;
                bool ok = true;
                for (int j = 0; j < T; ++j, ++tiles) {
                    if (j > 0) step(j < ahead ? 1u : 2u);
                    if (!(ok = mbar_wait(&kv_full[slot], par, abort_flag, a.err))) break;
                    float *const sc = reinterpret_cast<float *>(smem + L::kScaleOff) + slot * 128u;
                    convert_rows<D, BF16, false, 32>(sRing + slot * L::kTileBytes, smem + L::kCodeOff + slot * (kBN * 64u),
                                                     sc, first, s.len - (s.t0 + j) * kBN, 0, lane);
                    float *const ks = reinterpret_cast<float *>(smem + L::kKScaleOff) + (tiles & 3u) * 128u;
                    ks[first + lane] = sc[first + lane];
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&conv_full[slot], 2);  // (a V tile has 8 warps' arrivals)
                }
                if (!ok) break;
                step((uint32_t)ahead + 1u);  // (behind the segment's last V)
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[seg_i % kSegs]);
            }
        }
    } else {
        // ================================ softmax + output: lane x ================================
        if constexpr (kLanes == 2) tc::regs_inc<FP8 ? 168 : 208>();
        const int x = (warp - 4) >> 2, w4 = warp & 3;
        const int r = w4 * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
        const float c2 = a.scale * kLog2e;
        const uint32_t tO = tmem + L::kColO + 128u * x + lane_base;
        uint32_t g0 = 0;    // score buffers of this lane before this segment
        uint32_t item = 0;  // ring items before this segment (the V of its tile j: see the sweep)
        uint32_t tiles0 = 0;  // FP8: key tiles before this segment
        uint32_t c_slot = 0, c_par = 0;  // FP8: ring slot and parity of the V tile in work
        auto c_step = [&](uint32_t n) {
            c_slot += n;
            if (c_slot >= ring) {
                c_slot -= ring;
                c_par ^= 1u;
            }
        };
        uint32_t nml = 0;     // narrow segments so far
        uint32_t n_late = 0;  // segments of two buffers or more so far
        for (; next_segment(); ++seg_i) {
            const Segment &s = segs[seg_i % kSegs];
            const bool wide = kLanes == 2 && s.nodes > a.tile_nodes;
            const bool split = kLanes == 2 && !wide;  // the lanes share the rows
            const bool two_parts = !FP8 && (!wide || a.out_dtype == 2);
            const int T = s.t1 - s.t0, ahead = wide ? 1 : min(2, T);
            const int U = wide ? 2 * T : T;  // score buffers
            // wide: lane A's tile is full, lane B has the rest
            const int rows = (!wide ? s.nodes : x == 0 ? a.tile_nodes : s.nodes - a.tile_nodes) * gu;
            const bool row_ok = r < rows, warp_ok = w4 * 32 < rows;  // warp_ok: uniform
            // (recomputed from the segment where they are needed)
            auto row_node = [&]() -> int { return s.node0 + (s.nodes > a.tile_nodes ? x * a.tile_nodes : 0) + r / gu; };
            auto mask_row = [&]() -> const uint32_t * {
                return a.tree_mask + (size_t)(s.q0 + row_node()) * a.mask_words;
            };
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            // FP8: this warp's 16 rows of V_j, in the order of the tiles, V_0 now and V_{j + 1} after the last P over V_j
            // is handed over. The keys' codes are the conversion warps', a tile and more ahead. (With conversions by
            // integer instructions, 16 x 64 nodes and the long context: 279 and 122 us; all conversions there 288 and 138;
            // all of them here, before the values were exact, 336 and 169 against 319 and 138 then.)
            const int seg_len = s.len, seg_t0 = s.t0, seg_n = s.n;
            auto convert_v = [&](int j) -> bool {
                c_step(j == 0 ? (uint32_t)ahead : ahead + j <= T ? 2u : 1u);
                if (!mbar_wait(&kv_full[c_slot], c_par, abort_flag, a.err)) return false;
                const int n_valid = seg_len - (seg_t0 + j) * kBN;
                if (convert_rows<D, BF16, true, 16>(sRing + c_slot * L::kTileBytes, smem + L::kCodeOff + c_slot * (kBN * 64u),
                                                    reinterpret_cast<float *>(smem + L::kScaleOff) + c_slot * 128u,
                                                    (warp - 4) * 16, n_valid, n_valid - seg_n, lane))
                    s_poison[seg_i & 3u] = 1;
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&conv_full[c_slot]);
                return true;
            };
            if constexpr (FP8) {
                if (!convert_v(0)) break;
            }
            for (int u = 0; u < U; ++u) {
                const uint32_t g = g0 + (uint32_t)u, i = g & 1u;
                const int half = kLanes == 1 ? 0 : wide ? u & 1 : x, j = wide ? u >> 1 : u;
                const int start = (s.t0 + j) * kBN + half * kSub;
                const int j0 = start - (s.len - s.n);  // tree index of the buffer's first key (negative: context)
                const bool tail = j0 + kSub > 0;       // drafted tokens (or the end) among its keys
                const uint32_t tS = tmem + 128u * i + 64u * x + lane_base;
                uint32_t vis[2] = {0u, 0u};
                if (tail && row_ok) {
                    const uint32_t *mrow = mask_row();
                    const int w0 = j0 >> 5;
                    const uint32_t a0 = mask_word(mrow, w0, s.n), a1 = mask_word(mrow, w0 + 1, s.n),
                                   a2 = mask_word(mrow, w0 + 2, s.n);
                    vis[0] = __funnelshift_r(a0, a1, j0 & 31);
                    vis[1] = __funnelshift_r(a1, a2, j0 & 31);
                }
                if (!(ok = mbar_wait(&s_full[i], (g >> 1) & 1u, abort_flag, a.err))) break;
                tc::fence_after_sync();
                if (warp_ok) {
                    float v[kSub];
                    tc::tmem_ld32(tS, *reinterpret_cast<float(*)[32]>(&v[0]));
                    tc::tmem_ld32(tS + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
                    tc::tmem_wait_ld();
                    if constexpr (FP8) {
                        // the K row scales (the warps wrote them before conv_full, which the scores' products waited for)
                        const float4 *ks = reinterpret_cast<const float4 *>(smem + L::kKScaleOff) +
                                           ((tiles0 + (uint32_t)j) & 3u) * 32u + half * (kSub / 4);
#pragma unroll
                        for (int k = 0; k < kSub / 4; ++k) {
                            const float4 f = ks[k];
                            const float2 p = fmul2(make_float2(v[4 * k], v[4 * k + 1]), make_float2(f.x, f.y));
                            const float2 q = fmul2(make_float2(v[4 * k + 2], v[4 * k + 3]), make_float2(f.z, f.w));
                            v[4 * k] = p.x, v[4 * k + 1] = p.y, v[4 * k + 2] = q.x, v[4 * k + 3] = q.y;
                        }
                    }
                    if (tail) {
#pragma unroll
                        for (int k = 0; k < kSub; ++k) v[k] = (vis[k / 32] >> (k % 32)) & 1u ? v[k] : -INFINITY;
                    }
                    float m8[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) m8[q] = fmax3(v[q], v[q + 8], v[q + 16]);
#pragma unroll
                    for (int k = 24; k < kSub; k += 16)
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            m8[q] = fmax3(m8[q], v[k + q], (k + 8 + q < kSub) ? v[k + 8 + q] : -INFINITY);
                    const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
                    const float m_new = fmaxf(m, mx * c2);
                    const bool grow = m_new > m + kRescaleLog2;  // false while the row has seen nothing
                    const float alpha = grow ? ex2f(m - m_new) : 1.f;  // 0 when m = -inf
                    if (grow) {
                        m = m_new;
                        l *= alpha;
                    }
                    // (a row that has seen nothing: ex2(-inf - 0) = 0)
                    const float base = m == -INFINITY ? 0.f : m - kUp<BF16, FP8>;
                    const float2 cc2 = make_float2(c2, c2), nm2 = make_float2(-base, -base);
                    float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                    make_float2(0.f, 0.f)};
                    // FP8: the V scales' rests, once every warp has converted its rows of the tile
                    const float4 *vs = reinterpret_cast<const float4 *>(smem + L::kScaleOff) + c_slot * 32u +
                                       half * (kSub / 4);
                    if (FP8 && !(ok = mbar_wait(&conv_full[c_slot], c_par, abort_flag, a.err))) break;
#pragma unroll
                    for (int cc = 0; cc < kSub / 32; ++cc) {
                        // P over the chunk's own scores: 16 columns of roundings, 16 of remainders
                        uint32_t ph[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float2 xq = ffma2(make_float2(v[cc * 32 + 2 * q], v[cc * 32 + 2 * q + 1]), cc2, nm2);
                            const float2 e = make_float2(ex2f(xq.x), ex2f(xq.y));
                            l4[q & 3] = fadd2(l4[q & 3], e);
                            if constexpr (FP8) {
                                const float4 r4 = vs[cc * 8 + q / 2];
                                const float2 f = fmul2(e, q & 1 ? make_float2(r4.z, r4.w) : make_float2(r4.x, r4.y));
                                ph[q] = pack_pair<BF16>(f.x, f.y);
                                continue;
                            }
                            ph[q] = pack_pair<BF16>(e.x, e.y);
                            v[cc * 32 + 2 * q] = e.x;
                            v[cc * 32 + 2 * q + 1] = e.y;
                        }
                        tc::tmem_st16(tS + cc * 32, ph);
                        if (two_parts) {
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                ph[q] = remainder_pair<BF16>(v[cc * 32 + 2 * q], v[cc * 32 + 2 * q + 1], ph[q]);
                            tc::tmem_st16(tS + cc * 32 + 16, ph);
                        }
                    }
                    const float2 ls = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
                    l += ls.x + ls.y;
                    // O of the lane's earlier keys, once their last P V is done: it was issued before the next
                    // buffer's Q K, so that buffer's barrier says so (it waits for no P of this one)
                    if (u > 0 && __any_sync(0xffffffffu, grow)) {
                        uint64_t *bar = u + 1 < U ? &s_full[i ^ 1u] : pv_late;
                        if (!(ok = mbar_wait(bar, u + 1 < U ? ((g + 1u) >> 1) & 1u : n_late & 1u, abort_flag, a.err))) break;
                        tc::fence_after_sync();
#pragma unroll 1
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
                // V of drafted tokens and beyond the end: zero what is past the end, sweep the drafted rows. A
                // narrow lane does its half of the tile, lane A of a wide block all of it with the first half
                // (its products come before lane B's).
                const int tile_j0 = j0 - half * kSub;  // tree index of the tile's first key
                if (!FP8 && (wide ? x == 0 && half == 0 && tile_j0 + kBN > 0 : tail)) {
                    const uint32_t vi = item + j + min(T, ahead + j);
                    if (!(ok = mbar_wait(&kv_full[vi % ring], (vi / ring) & 1u, abort_flag, a.err))) break;
                    uint8_t *const sV = sRing + (vi % ring) * L::kTileBytes;
                    const int n_valid = min(kBN, s.len - (s.t0 + j) * kBN);
                    const int row0 = wide ? 0 : half * kSub, row1 = wide ? kBN : row0 + kSub;
                    bool bad = false;
                    // 8 lanes a row (128 bytes of a 64-column half), 4 rows a warp and step
                    for (int row = max(row0, -tile_j0 / 16 * 16) + w4 * 4 + (lane >> 3); row < row1; row += 16)
#pragma unroll
                        for (int hf = 0; hf < L::kHalves; ++hf) {
                            uint4 *p = reinterpret_cast<uint4 *>(sV + hf * L::kTileHalf + (uint32_t)row * 128u + (lane & 7) * 16);
                            if (row >= n_valid) {
                                *p = make_uint4(0, 0, 0, 0);
                            } else if (row >= -tile_j0) {
                                uint4 q = *p;
                                if (nonfinite_pair<BF16>(q.x) || nonfinite_pair<BF16>(q.y) || nonfinite_pair<BF16>(q.z) ||
                                    nonfinite_pair<BF16>(q.w)) {
                                    q = make_uint4(drop_nonfinite<BF16>(q.x), drop_nonfinite<BF16>(q.y),
                                                   drop_nonfinite<BF16>(q.z), drop_nonfinite<BF16>(q.w));
                                    *p = q;
                                    bad = true;
                                }
                            }
                        }
                    if (bad) s_poison[seg_i & 3u] = 1;
                    tc::fence_proxy_async_smem();
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
                if constexpr (FP8) {
                    if ((!wide || (u & 1)) && j + 1 < T && !(ok = convert_v(j + 1))) break;
                }
            }
            if (!ok) break;
            g0 += (uint32_t)U;
            if (U > 1) ++n_late;
            // ---- output of the segment ----
            // rows shared by the lanes: rows 0-63 are finished by lane A, 64-127 by lane B
            const bool mine = !split || (w4 >> 1) == x;
            float fa = 1.f, fb = 0.f, lse2 = m, lt = l;  // out = fa O_A + fb O_B (or f O of this lane)
            if (split) {
                // (max, sum) through the stage of the warp that hands them over, which puts out no rows of a split segment:
                // two places in turn. A place is written again two split segments later, behind a phase of ml_full that
                // takes its reader's arrival; or by a wide segment's rows, behind an o_done that takes its reader's P.
                float2 *const ml = reinterpret_cast<float2 *>(smem + L::kStageOff + ((warp - 4) ^ (mine ? 4 : 0)) * 32 *
                                                              L::kStageRow) + (nml & 1u) * 32u + lane;
                if (!mine) *ml = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
                if (!mbar_wait(ml_full, nml & 1u, abort_flag, a.err)) break;
                ++nml;
                if (mine) {
                    const float2 o = *ml;
                    const float M = fmaxf(m, o.x);
                    const float w_me = m == -INFINITY ? 0.f : ex2f(m - M), w_o = o.x == -INFINITY ? 0.f : ex2f(o.x - M);
                    lt = w_me * l + w_o * o.y;
                    lse2 = M;
                    fa = x == 0 ? w_me : w_o;
                    fb = x == 0 ? w_o : w_me;
                }
            }
            const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);  // (a NaN sum stays NaN)
            lse2 = lt == 0.f ? -INFINITY : lse2 + __log2f(lt) - kUp<BF16, FP8>;
            fa *= inv;
            fb *= inv;
            if (!mbar_wait(o_done, seg_i & 1u, abort_flag, a.err)) break;
            tc::fence_after_sync();
            if (mine && warp_ok) {
                const bool poison = s_poison[seg_i & 3u] != 0;
                const int node = row_node(), tree0 = s.len - s.n;  // position of node 0
                const uint32_t *mrow = mask_row();
                const bool part = s.slot >= 0;
                const size_t prow = ((size_t)blockIdx.x * 2 + (s.slot > 0)) * a.part_rows + (wide ? x * kBM : 0) + r;
                const size_t orow = part ? prow : (size_t)(s.q0 + node) * a.num_q_heads + (size_t)s.unit * gu + r % gu;
                if (row_ok) {
                    if (part) a.part_lse[prow] = lse2;
                    else if (a.lse) a.lse[orow] = lse2 * kLn2;
                }
                const uint32_t tOa = tmem + L::kColO + lane_base + (wide ? 128u * x : 0u);
                // rows go out through shared memory, 128 bytes of each at a time: 8 lanes a row instead of
                // 32 rows a store
                const bool f32 = part || a.out_dtype == 2;
                uint8_t *out = static_cast<uint8_t *>(part ? static_cast<void *>(a.part_o) : a.out);
                const long long row_bytes = D * (f32 ? 4 : 2);
                const long long dst_row = row_ok ? (long long)orow * row_bytes : -1;
                constexpr int kStageRow = L::kStageRow, kPieces = kStageRow / 16;  // 16-byte pieces of a row at a time
                uint8_t *stage = smem + L::kStageOff + (warp - 4) * 32 * kStageRow;
                auto place = [&](int rr, int c) { return stage + rr * kStageRow + ((c ^ (rr & (kPieces - 1))) << 4); };
                long long dst[kPieces];  // where this lane's pieces go
#pragma unroll
                for (int i = 0; i < kPieces; ++i) dst[i] = __shfl_sync(0xffffffffu, dst_row, i * (32 / kPieces) + lane / kPieces);
                auto flush = [&](int col_bytes) {
                    __syncwarp();
                    uint4 v[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        v[i] = *reinterpret_cast<const uint4 *>(place(i * (32 / kPieces) + lane / kPieces, lane % kPieces));
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        if (dst[i] >= 0) *reinterpret_cast<uint4 *>(out + dst[i] + col_bytes + lane % kPieces * 16) = v[i];
                    __syncwarp();
                };
                auto stage16 = [&](int piece, const uint4 &v) {  // 16-byte piece of this lane's output row
                    *reinterpret_cast<uint4 *>(place(lane, piece % kPieces)) = v;
                    if (piece % kPieces == kPieces - 1) flush((piece + 1 - kPieces) * 16);
                };
                // a weight of 0 (a lane that saw nothing) takes nothing, whatever the output holds
                const bool use_a = fa != 0.f, use_b = split && fb != 0.f;
                float nxt[32], nxt_b[32];  // the chunk read ahead
                tc::tmem_ld32(tOa, nxt);
                if (split) tc::tmem_ld32(tOa + 128u, nxt_b);
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    float o[32];
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = use_a ? nxt[i] * fa : 0.f;
                    if (split) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = use_b ? fmaf(nxt_b[i], fb, o[i]) : o[i];
                    }
                    if (cc + 1 < D / 32) {
                        tc::tmem_ld32(tOa + (cc + 1) * 32, nxt);
                        if (split) tc::tmem_ld32(tOa + 128u + (cc + 1) * 32, nxt_b);
                    }
                    if (poison && row_ok) {
                        // infinities and NaN of the drafted V rows that this row sees
                        const int k0 = max(0, s.t0 * kBN - tree0), k1 = min(s.n, s.t1 * kBN - tree0);
                        for (int k = k0; k < k1; ++k) {
                            if (!((mask_word(mrow, k >> 5, s.n) >> (k & 31)) & 1u)) continue;
                            const int pos = tree0 + k;
                            int pb = __ldg(a.block_tables + (size_t)s.b * a.max_blocks_per_seq +
                                           (pos >> a.cache.log2_block_size));
                            if (pb < 0 || pb >= a.cache.num_blocks) pb = 0;
                            const size_t row = (((size_t)pb * 2 + 1) * a.cache.num_kv_heads + s.unit / a.head_groups) *
                                                   a.cache.block_size + (pos & (a.cache.block_size - 1));
#pragma unroll 1
                            for (int i = 0; i < 4; ++i) {
                                uint4 raw;  // 8 values as the products would read them
                                if constexpr (FP8) {
                                    float rest;
                                    const uint2 *codes = static_cast<const uint2 *>(a.cache.ptr) + row * (D / 8);
                                    raw = values_of<BF16, true>(__ldg(codes + cc * 4 + i),
                                                                split_scale<BF16>(__ldg(a.cache.scales + row), rest));
                                } else {
                                    raw = __ldg(static_cast<const uint4 *>(a.cache.ptr) + row * (D / 8) + cc * 4 + i);
                                }
                                if (!nonfinite8<BF16>(raw)) continue;
                                float f[8];
                                if constexpr (BF16) unpack8(raw, f, BF16Tag());
                                else unpack8(raw, f, F16Tag());
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (c == i)
#pragma unroll
                                        for (int q = 0; q < 8; ++q)
                                            if (!isfinite(f[q])) o[8 * c + q] += f[q];
                            }
                        }
                    }
                    if (f32) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            stage16(cc * 8 + q, make_uint4(__float_as_uint(o[4 * q]), __float_as_uint(o[4 * q + 1]),
                                                           __float_as_uint(o[4 * q + 2]), __float_as_uint(o[4 * q + 3])));
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            stage16(cc * 4 + q,
                                    make_uint4(pack_pair<BF16>(o[8 * q], o[8 * q + 1]), pack_pair<BF16>(o[8 * q + 2], o[8 * q + 3]),
                                               pack_pair<BF16>(o[8 * q + 4], o[8 * q + 5]),
                                               pack_pair<BF16>(o[8 * q + 6], o[8 * q + 7])));
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                // the flag of the segment after next: its last readers, two segments back, arrived on
                // o_empty before the last segment's products; its next setters follow products that
                // wait for the arrival below
                if (warp == 4) s_poison[(seg_i + 2u) & 3u] = 0;
                mbar_arrive(o_empty);
                mbar_arrive(&seg_empty[seg_i % kSegs]);
            }
            item += 2 * T;
            tiles0 += (uint32_t)T;
            if constexpr (FP8) c_step(1u);  // (the last V was the segment's last item)
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    pdl_launch_dependents();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// The partials of the item that begins in run blockIdx.x and is split: run c0's partial 1, then partial 0
// of the runs behind it. A warp per row: weights 2^(lse_i - max), out = sum w o / sum w, in the order of the keys. Bound:
// latency (three dependent reads), so that a row's first partials are read along with their lse.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(TreeArgs a) {
    constexpr int V = D / 32;
    constexpr int kFlight = D == 256 ? 4 : 8;  // rows in flight
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const MergeItem it = a.merge[blockIdx.x];
    const int rows = it.nodes * a.unit_heads;
    const int r = blockIdx.y * 8 + warp;
    if (r < rows) {
        // rows of a wide block: lane B's start at row 128 of the partial
        const int node = r / a.unit_heads, head = r - node * a.unit_heads;
        const int pr = node < a.tile_nodes ? r : kBM + r - a.tile_nodes * a.unit_heads;
        auto prow = [&](int i) { return ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * a.part_rows + pr; };
        float y[kFlight][V];
        auto read = [&](int k0, int n) {
#pragma unroll
            for (int f = 0; f < kFlight; ++f)
                if (f < n) {
                    const float *p = a.part_o + prow(k0 + f) * D + V * lane;
                    if constexpr (V == 2) {
                        const float2 q = __ldcg(reinterpret_cast<const float2 *>(p));
                        y[f][0] = q.x, y[f][1] = q.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < V / 4; ++c) {
                            const float4 q = __ldcg(reinterpret_cast<const float4 *>(p) + c);
                            y[f][4 * c] = q.x, y[f][4 * c + 1] = q.y, y[f][4 * c + 2] = q.z, y[f][4 * c + 3] = q.w;
                        }
                    }
                }
        };
        read(0, it.parts);
        float x = lane < it.parts ? __ldcg(a.part_lse + prow(lane)) : -INFINITY;
        float M = x;
        bool nan = x != x;
        for (int i = lane + 32; i < it.parts; i += 32) {
            const float z = __ldcg(a.part_lse + prow(i));
            nan |= z != z;
            M = fmaxf(M, z);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (__any_sync(0xffffffffu, nan)) M = NAN;
        float acc[V], sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
        // 32 partials at a time: lane i holds the weight of partial i
        for (int i0 = 0; i0 < it.parts; i0 += 32) {
            const int n = min(32, it.parts - i0);
            if (i0 > 0) x = lane < n ? __ldcg(a.part_lse + prow(i0 + lane)) : -INFINITY;
            const float w_l = x == -INFINITY ? 0.f : ex2f(x - M);
            sum += w_l;
            for (int k = 0; k < n; k += kFlight) {
                if (i0 + k > 0) read(i0 + k, n - k);
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    if (k + f >= n) break;
                    const float w = __shfl_sync(0xffffffffu, w_l, k + f);
                    if (w == 0.f) continue;  // saw nothing
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, y[f][v], acc[v]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= inv;
        const size_t orow = (size_t)(it.q0 + it.node0 + node) * a.num_q_heads + (size_t)it.unit * a.unit_heads + head;
        store_out_vec<V>(a.out, orow * D + V * lane, acc, a.out_dtype);
        if (lane == 0 && a.lse) a.lse[orow] = sum == 0.f ? -INFINITY : (M + __log2f(sum)) * kLn2;
    }
    pdl_launch_dependents();
}

template <int D, bool BF16, bool FP8 = false>
cudaError_t launch_tree_t(const TreeArgs &a, int grid, cudaStream_t s) {
    using L = TreeLayout<D, FP8>;
    CUtensorMap tm_q, tm_kv;
    cudaError_t e = encode_q_group_map(a.q, BF16 ? 1 : 0, a.total_q, a.num_q_heads, D, a.unit_heads, a.tile_nodes, &tm_q);
    if (e != cudaSuccess) return e;
    e = encode_cache_map(a.cache, a.cache.block_size < L::kBN ? a.cache.block_size : L::kBN, &tm_kv);
    if (e != cudaSuccess) return e;
    const DeviceInfo &info = device_info();
    if ((int)L::kSmem > info.max_smem) return cudaErrorNotSupported;
    auto kern = tree_kernel<D, BF16, FP8>;
    static DeviceFlags configured;
    if (!configured.test(info.device)) {
        e = set_smem_attributes(kern, info.max_smem);
        if (e != cudaSuccess) return e;
        configured.set(info.device);
    }
    e = launch_pdl(kern, dim3(grid), dim3(L::kThreads), L::kSmem, s, tm_q, tm_kv, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(tree_merge_kernel<D>, dim3(grid, (a.block_nodes * a.unit_heads + 7) / 8), dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, int grid, cudaStream_t s) {
    const bool bf16 = a.cache.dtype == 1;
    if (a.cache.fp8) {
        if (a.cache.head_dim == 128)
            return bf16 ? launch_tree_t<128, true, true>(a, grid, s) : launch_tree_t<128, false, true>(a, grid, s);
        return bf16 ? launch_tree_t<64, true, true>(a, grid, s) : launch_tree_t<64, false, true>(a, grid, s);
    }
    switch (a.cache.head_dim) {
        case 256: return bf16 ? launch_tree_t<256, true>(a, grid, s) : launch_tree_t<256, false>(a, grid, s);
        case 128: return bf16 ? launch_tree_t<128, true>(a, grid, s) : launch_tree_t<128, false>(a, grid, s);
        case 64: return bf16 ? launch_tree_t<64, true>(a, grid, s) : launch_tree_t<64, false>(a, grid, s);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pkv

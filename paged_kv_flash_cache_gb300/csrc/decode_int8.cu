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
// FP32 scores. The V scales enter the weights, which go into the product relative to the power of two at or above their
// tile's largest, as an f16 part and its remainder: the output's rounding is the only 16-bit one on the path
// (weights times scales below 2^-35 of the row's largest weight and the tile's largest scale are lost).
//
// Structure (persistent, three CTAs an SM of four warps). A unit is (sequence, KV head's query group, split); tile j (8 KB of
// codes) of a unit is warp j % W's. Every warp feeds itself: it has a ring of its own and sends for the tile that goes into a slot as
// soon as it has read the slot's last one, so no warp waits for another one and there is no producer to fall behind
// (with one, 0.131 ms on the 7B-like batch, 0.111 with three quarters of the arithmetic left out). A tile arrives in page
// slices of min(bs, tile) rows, each one 5-D TMA box of its K rows and its V rows; a slice lies in one page, whose scales
// come beside it by 4-byte asynchronous copies on the same mbarrier. The page ids of the tile after are loaded a tile
// ahead. The blocks of 16 tokens of a tile are independent chains of ldmatrix, conversion and mma. At the
// end of a unit the warps merge their rows, a head each, and write the output or the split's partial.
//
// Measured with the merge, back to back: 16 sequences of 1024 to 8192 tokens, 32 heads (505 MB) 80.7 us, 92% of the copy rate,
// issue slots half used; 64 of 16 to 8192, 32 / 8 heads (179 MB) 37.4 us, 70%: ten of them are set-up, uneven units and the
// merge; one request of 4096 tokens 8.0 us, latency. 64 x 4096 tokens over 8 KV heads: 86 us with 1 query head each, 89 with 4,
// 100 with 8 (92, 89 and 79%); at head_dim 64 54, 57 and 65 (73, 70 and 61%), bound by the conversions.
//
// Operand layouts. ldmatrix (.b16) hands lane (gid, tig) the codes of dims 4 tig .. 4 tig + 3 of a 16-dim chunk: the
// k slots of the A fragment are the permutation {2tig, 2tig+1, 2tig+8, 2tig+9} -> {4tig .. 4tig+3}, and q's B fragment
// is built alike. For P.V, ldmatrix.trans hands a lane (token 2tig: dims 2gid, 2gid+1; token 2tig+1: the same): the
// permute that widens the codes also pairs them by dim, M slot gid holding dim 2gid and slot gid + 8 dim 2gid + 1.
// Up to four heads take head slots 0-3 and, once more, 4-7: the first four carry the weights' f16 parts into the
// product with V and the others the remainders, in one mma; with more heads the remainders are a second mma.
#include <cuda.h>

#include <atomic>

#include "cluster.cuh"
#include "decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Tokens of a tile: 8 KB of codes. (head_dim 64 with 32 tokens a tile: what a tile costs besides its codes bounded it, 64
// sequences of 4096 tokens, 8 KV heads 61 us.)
template <int D>
constexpr int kTile = D == 64 ? 64 : 32;
constexpr int kCtasPerSm = kInt8CtasPerSm;
constexpr float kRescale = 4.0f;  // lazy rescale threshold (log2 units)
constexpr float kWeight = 2048.0f;  // weights, at most 2^kRescale, go into the product times this: below f16's 65504

template <int D, int G>
struct Int8Layout {
    static constexpr int kStages = 2;  // slots of a warp's ring
    static constexpr int kSlices = kTile<D> / 8;                  // page slices of a tile at most
    static constexpr uint32_t kStageBytes = 2 * kTile<D> * D;     // per slice: br K rows, br V rows of D bytes
    static constexpr uint32_t kScaleOffset = kWarps * kStages * kStageBytes;  // [kWarps][kStages][kSlices] (K, V)
    static constexpr uint32_t kBarOffset = kScaleOffset + kWarps * kStages * kSlices * 8;
    // full per slot, rows written, rows read, then the abort flag
    static constexpr uint32_t kMergeOffset = (kBarOffset + (kWarps * kStages + 2) * 8 + 16 + 15) / 16 * 16;
    // the warps' rows of up to four heads at a time (eight at once would leave room for two CTAs an SM only), and, in a
    // cluster, the CTA's row of each head
    static constexpr int kMergeHeads = G < 4 ? G : 4;
    static constexpr uint32_t kMergeFloats = kWarps * kMergeHeads * kMergeRow<D>;
    static constexpr uint32_t kIntsOffset = kMergeOffset + kMergeFloats * 4;
    static size_t smem_bytes(int batch, int s_max) {
        return kIntsOffset + unit_table_ints(batch, s_max) * 4 + 1024;  // + 1024-byte alignment slack
    }
    static size_t smem_bytes_one() { return kIntsOffset + G * kMergeRow<D> * 4 + 1024; }
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

// A wait that gave up for one lane has for the warp: what follows needs its lanes together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *err) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}

// Four bytes global -> shared, asynchronously; and an arrival on `bar` once this thread's copies so far have landed
// (one of the arrivals that the barrier expects).
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// The unit tables. For small batches straight from their definitions, a thread an entry: first[s] = sum of min(splits, s)
// over the sequences, ord by counting the sequences in front (2 us less a launch than decode_scan_units' scans, whose
// latency a single request waits for).
template <int kThreads>
__device__ __forceinline__ int scan_units(const DecodeArgs &a, const UnitTable &t) {
    const int S = a.s_max, cap = a.max_blocks_per_seq * a.cache.block_size;
    if (a.auto_chunk || a.batch > kThreads || (long long)a.batch * (S / kThreads + 1) > 128)
        return decode_scan_units<kThreads>(a, t);
    const int tid = threadIdx.x;
    int len = 0, k = 0;
    if (tid < a.batch) {
        len = __ldg(a.context_lens + tid);
        int qrow = tid;
        bool mine = true;
        if (a.cu_q_lens) {  // mixed batch: only single-row sequences are decoded here
            qrow = __ldg(a.cu_q_lens + tid);
            mine = __ldg(a.cu_q_lens + tid + 1) - qrow == 1;
        }
        if (len < 0 || len > cap) {
            set_error(a.err, kErrDeviceRange);
            len = len < 0 ? 0 : cap;
        }
        if (!mine) len = 0;
        k = (len + a.chunk - 1) / a.chunk;
        t.lens[tid] = len;
        t.qrow[tid] = qrow;
        t.ord[tid] = k;
    }
    if (tid == 0) t.misc[0] = a.chunk;
    __syncthreads();
    int rank = 0;
    if (tid < a.batch)
        for (int j = 0; j < a.batch; ++j) rank += t.ord[j] > k || (t.ord[j] == k && j < tid) ? 1 : 0;
    for (int s = tid; s <= S; s += kThreads) {
        int f = 0;
        for (int j = 0; j < a.batch; ++j) f += min(t.ord[j], s);
        t.first[s] = f;
    }
    __syncthreads();
    if (tid < a.batch) t.ord[rank] = tid;
    __syncthreads();
    return t.first[S] * a.cache.num_kv_heads * a.head_groups;
}

// ONE: a cluster takes the whole context of one (sequence, KV head's query group), a run of keys a CTA, and merges it
// over shared memory: no unit tables, partials or second launch. For launches that leave most CTAs with a unit or less
// (decode_int8_cluster).
template <int D, int G, bool ONE>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_int8_kernel(const __grid_constant__ CUtensorMap tm, DecodeArgs a) {
    using L = Int8Layout<D, G>;
    constexpr int S = L::kStages;
    constexpr int kChunks = D / 16;    // 16-dim chunks: k-steps of q.K^T, m-tiles of O^T
    constexpr bool kPacked = G <= 4;   // weights and their remainders side by side in one mma
    constexpr int T = kTile<D>, kBlocks = T / 16;
    constexpr int kLanesFull = L::kSlices;  // lanes that copy scales
    constexpr int kMH = L::kMergeHeads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBarOffset);  // [kWarps][S]
    uint64_t *written = full + kWarps * S;  // the warps' rows of a unit are in the merge buffer
    uint64_t *read = written + 1;           // and have been merged
    volatile int *abort_flag = reinterpret_cast<volatile int *>(read + 1);
    float *merge = reinterpret_cast<float *>(smem + L::kMergeOffset);
    float *cta_rows = reinterpret_cast<float *>(smem + L::kIntsOffset);  // ONE: in the tables' place
    const UnitTable ut = unit_table(reinterpret_cast<int *>(smem + L::kIntsOffset), a.batch, a.s_max);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hkv = a.cache.num_kv_heads, bs = a.cache.block_size;
    const int hu = hkv * a.head_groups;  // unit heads
    // rows of a slice (a power of two): splits and tiles start at multiples of the tile
    const int log2_br = min(a.cache.log2_block_size, T == 64 ? 6 : 5), br = 1 << log2_br;

    if (tid == 0) {
        for (int i = 0; i < kWarps * S; ++i) mbar_init(&full[i], 1 + kLanesFull);  // the boxes' bytes; the scales
        mbar_init(written, kWarps);
        mbar_init(read, kWarps);
        *abort_flag = 0;
        fence_barrier_init();
        tc::prefetch_tensormap(&tm);
    }
    pdl_wait();  // lengths, tables, q and the cache may come from the previous kernel
    UnitCursor one = {};
    int num_units = 1, chunk = 0, first_unit = 0, one_row = 0;
    bool one_mine = true;
    if constexpr (ONE) {
        const int n = cluster_size(), rank = cluster_rank(), id = blockIdx.x / n;
        one.b = id / hu;
        one.kvh = id - one.b * hu;
        int len = __ldg(a.context_lens + one.b);
        one_row = one.b;
        if (a.cu_q_lens) {  // mixed batch: only single-row sequences are decoded here
            one_row = __ldg(a.cu_q_lens + one.b);
            one_mine = __ldg(a.cu_q_lens + one.b + 1) - one_row == 1;
        }
        const int cap = a.max_blocks_per_seq * bs;
        if (len < 0 || len > cap) {
            if (tid == 0) set_error(a.err, kErrDeviceRange);
            len = len < 0 ? 0 : cap;
        }
        if (!one_mine) len = 0;
        const int per = ((len + n - 1) / n + T - 1) / T * T;
        one.t0 = min(rank * per, len);
        one.t1 = min(one.t0 + per, len);
        __syncthreads();  // (the barriers are initialised)
    } else {
        num_units = scan_units<kThreads>(a, ut);
        chunk = ut.misc[0];  // the launch's split size
        first_unit = blockIdx.x;
    }

    uint8_t *ring = smem + (size_t)warp * S * L::kStageBytes;
    float *scales = reinterpret_cast<float *>(smem + L::kScaleOffset) + warp * S * L::kSlices * 2;
    full += warp * S;
    // ---- what is sent for: the next tile, its unit and the page ids of its slices (lane j: slice j) ----
    const uint64_t pol = l2_policy_evict_first();
    int iu = first_unit, its = 0, ipb = 0, ikv = 0;
    uint32_t issued = 0;
    UnitCursor ic = {};
    auto seek = [&]() {  // from unit iu on, the first one with a tile of this warp; its page ids
        for (; iu < num_units; iu += gridDim.x) {
            ic = ONE ? one : unit_of(iu, ut, a.s_max, hu, chunk);
            its = ic.t0 + warp * T;
            ikv = a.head_groups == 1 ? ic.kvh : ic.kvh / a.head_groups;  // the KV head of the unit
            if (its < ic.t1) break;
        }
    };
    auto page_ids = [&]() {
        const int tok = its + lane * br;
        ipb = 0;
        if (iu < num_units && lane < kLanesFull && tok < ic.t1 && lane * br < T)
            ipb = __ldg(a.block_tables + (size_t)ic.b * a.max_blocks_per_seq + (tok >> a.cache.log2_block_size));
    };
    auto send = [&](int slot) {
        if (iu >= num_units) return;
        const int n = min(T, ic.t1 - its);
        const int nslices = (n + br - 1) >> log2_br;  // <= kSlices
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)nslices * br * 2u * D);
        __syncwarp();
        if (lane < nslices) {
            int pb = ipb;
            if (pb < 0 || pb >= a.cache.num_blocks) {
                set_error(a.err, kErrDeviceRange);
                pb = 0;
            }
            tc::tma_load_5d_hint(ring + (size_t)slot * L::kStageBytes + (size_t)lane * 2 * br * D, &tm, 0,
                                 (its + lane * br) & (bs - 1), ikv, 0, pb, &full[slot], pol);
            const float *sc = a.cache.scales + (size_t)pb * 2 * hkv + ikv;
            cp_async4(scales + slot * L::kSlices * 2 + lane * 2, sc);
            cp_async4(scales + slot * L::kSlices * 2 + lane * 2 + 1, sc + hkv);
        }
        if (lane < kLanesFull) cp_async_arrive(&full[slot]);
        ++issued;
        its += kWarps * T;
        if (its >= ic.t1) {
            iu += gridDim.x;
            seek();
        }
        page_ids();
    };
    seek();
    page_ids();
    for (int i = 0; i < S; ++i) send(i);

    const int gid = lane >> 2, tig = lane & 3;
    const int mi = lane >> 3;
    const float sl = a.scale * kLog2e;
    const bool bf16 = a.cache.dtype == 1;
    const uint16_t *qg = static_cast<const uint16_t *>(a.q);
    uint32_t bq[kChunks][2];  // q as f16 B fragments, k slots permuted as the K codes
    uint32_t taken = 0;       // tiles read
    int slot = 0;
    uint32_t phase = 0;
    uint32_t mphase = 0;  // of the merge buffer
    bool ok = true;
    // rows of the warp's ldmatrix in the slice layout (slice j starts at row 2 j br): 16 tokens a block
    int trow[kBlocks];
#pragma unroll
    for (int bl = 0; bl < kBlocks; ++bl) {
        const int t = bl * 16 + (lane & 7) + 8 * (mi & 1);
        trow[bl] = t + (t & -br);
    }
    for (int u = first_unit; u < num_units; u += gridDim.x) {
        const UnitCursor c = ONE ? one : unit_of(u, ut, a.s_max, hu, chunk);
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float2 o[kChunks][2];
#pragma unroll
        for (int mt = 0; mt < kChunks; ++mt) o[mt][0] = o[mt][1] = make_float2(0.f, 0.f);
        const int first = c.t0 + warp * T;
        if (first < c.t1) {
            const int hq = kPacked ? gid & 3 : gid;  // head of this lane's column of the B fragment
            const uint16_t *qr = qg + ((size_t)(ONE ? one_row : ut.qrow[c.b]) * a.num_q_heads + (size_t)c.kvh * G + hq) * D + 4 * tig;
#pragma unroll
            for (int kk = 0; kk < kChunks; ++kk) {
                uint2 raw = make_uint2(0u, 0u);
                if (hq < G) raw = __ldg(reinterpret_cast<const uint2 *>(qr + kk * 16));
                bq[kk][0] = raw.x;
                bq[kk][1] = raw.y;
            }
            if (bf16) {
#pragma unroll
                for (int kk = 0; kk < kChunks; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        bq[kk][i] = pack_pair<false>(__uint_as_float(bq[kk][i] << 16), __uint_as_float(bq[kk][i] & 0xffff0000u));
            }
        }
        for (int ts = first; ts < c.t1; ts += kWarps * T) {
            const int n = min(T, c.t1 - ts);
            if (!(ok = warp_wait(&full[slot], phase, abort_flag, a.err))) break;
            const uint32_t aK = smem_addr(ring + (size_t)slot * L::kStageBytes), aV = aK + br * D;
            // scales of the groups of 8 tokens (a group lies in one page)
            float sk[2 * kBlocks], sv[2 * kBlocks];
#pragma unroll
            for (int g = 0; g < 2 * kBlocks; ++g) {
                const float2 x = *reinterpret_cast<const float2 *>(scales + slot * L::kSlices * 2 + ((g * 8) >> log2_br) * 2);
                sk[g] = x.x * sl;
                sv[g] = x.y;
            }
            // ---- S^T = K q^T: blocks of 16 tokens x 8 head slots ----
            float s[kBlocks][4];
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl) s[bl][0] = s[bl][1] = s[bl][2] = s[bl][3] = 0.f;
#pragma unroll
            for (int cp = 0; cp < kChunks; cp += 2)
#pragma unroll
                for (int b0 = 0; b0 < kBlocks; b0 += 2) {
                    uint32_t r[2][4];
#pragma unroll
                    for (int bl = 0; bl < 2; ++bl) ldsm_x4(swz<D>(aK, trow[b0 + bl], cp + (mi >> 1)), r[bl]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int bl = 0; bl < 2; ++bl) {
                            const uint32_t x = r[bl][2 * h] ^ 0x80808080u, y = r[bl][2 * h + 1] ^ 0x80808080u;
                            const uint32_t af[4] = {codes_f16<0x4140>(x), codes_f16<0x4140>(y), codes_f16<0x4342>(x),
                                                    codes_f16<0x4342>(y)};
                            mma16816<false>(s[b0 + bl], af, bq[cp + h][0], bq[cp + h][1]);
                        }
                }
            // token of s[bl][i]: bl * 16 + gid + 8 * (i >> 1); head slot 2 tig + (i & 1)
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[bl][i] *= sk[bl * 2 + (i >> 1)];
            if (n < T) {  // behind the context's end (and maybe beyond the last slice): no weight, and no scale
#pragma unroll
                for (int g = 0; g < 2 * kBlocks; ++g) {
                    if (g * 8 >= n) sv[g] = 0.f;
                    if (g * 8 + gid >= n) s[g >> 1][(g & 1) * 2] = s[g >> 1][(g & 1) * 2 + 1] = -INFINITY;
                }
            }
            // The running max m of a head is a past maximum: it moves only when a score exceeds it by more than 2^4, so
            // the lanes need one vote a tile and rarely each other's maxima.
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int i = 0; i < 2; ++i) mx[i] = fmax3(mx[i], s[bl][i], s[bl][i + 2]);
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale)) {
#pragma unroll
                for (int ofs = 4; ofs < 32; ofs <<= 1) {
                    mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], ofs));
                    mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], ofs));
                }
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mn = fmaxf(m[i], mx[i]);
                    al[i] = mn > m[i] ? ex2f(m[i] - mn) : 1.f;  // 0 when m = -inf
                    m[i] = mn;
                    l[i] *= al[i];
                }
#pragma unroll
                for (int mt = 0; mt < kChunks; ++mt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) o[mt][k] = fmul2(o[mt][k], make_float2(al[0], al[1]));
            }
            // The tile's weights enter the product relative to W, the power of two at or above its largest V scale, and times
            // 2^11: P' = 2^11 (p sv / W) (at most 2^15), as an f16 part and its remainder, holds weights down to 2^-35. The
            // tile's product enters O in FP32 times W / 2^11. A power of two: 1 / W is one at both ends of the scales'
            // range, W / 2^11 has no bits to lose below 2^-126, and neither rounds (2^11 / W would pass FP32's range for
            // scales up to 2^-117).
            float w = sv[0];
#pragma unroll
            for (int g = 1; g < 2 * kBlocks; ++g) w = fmaxf(w, sv[g]);
            const uint32_t wb = (__float_as_uint(w) + 0x7fffffu) & 0xff800000u;
            const float rw = w >= 1.17549435e-38f ? __uint_as_float(0x7f000000u - wb) : 0.f;  // (scales below 2^-126 count as 0)
            uint32_t ph[kBlocks][2], pe[kBlocks][2];
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float p0 = ex2f(s[bl][2 * hf] - m[0]), p1 = ex2f(s[bl][2 * hf + 1] - m[1]);
                    l[0] += p0;
                    l[1] += p1;
                    const float r = sv[bl * 2 + hf] * rw * kWeight;
                    uint32_t hi, lo;
                    split_pair<false>(p0 * r, p1 * r, hi, lo);
                    if (kPacked) {
                        ph[bl][hf] = movmatrix_t(tig < 2 ? hi : lo);
                    } else {
                        ph[bl][hf] = movmatrix_t(hi);
                        pe[bl][hf] = movmatrix_t(lo);
                    }
                }
            const float f = __uint_as_float(wb) * (1.f / kWeight);
            const float2 f2 = make_float2(f, f);
            // ---- O^T += f V^T P'^T: D dims (permuted within each 16-dim chunk) x 8 slots ----
#pragma unroll
            for (int cp = 0; cp < kChunks; cp += 2) {
                float ot[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) ot[h][0] = ot[h][1] = ot[h][2] = ot[h][3] = 0.f;
#pragma unroll
                for (int b0 = 0; b0 < kBlocks; b0 += 2) {
                    uint32_t r[2][4];
#pragma unroll
                    for (int bl = 0; bl < 2; ++bl) ldsm_x4_t(swz<D>(aV, trow[b0 + bl], cp + (mi >> 1)), r[bl]);
#pragma unroll
                    for (int bl = 0; bl < 2; ++bl)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = r[bl][2 * h] ^ 0x80808080u, y = r[bl][2 * h + 1] ^ 0x80808080u;
                            const uint32_t af[4] = {codes_f16<0x4240>(x), codes_f16<0x4341>(x), codes_f16<0x4240>(y),
                                                    codes_f16<0x4341>(y)};
                            if (!kPacked) mma16816<false>(ot[h], af, pe[b0 + bl][0], pe[b0 + bl][1]);
                            mma16816<false>(ot[h], af, ph[b0 + bl][0], ph[b0 + bl][1]);
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    o[cp + h][0] = ffma2(make_float2(ot[h][0], ot[h][1]), f2, o[cp + h][0]);
                    o[cp + h][1] = ffma2(make_float2(ot[h][2], ot[h][3]), f2, o[cp + h][1]);
                }
            }
            // the slot's next tile
            __syncwarp();
            ++taken;
            send(slot);
            if (++slot == S) {
                slot = 0;
                phase ^= 1u;
            }
        }
        if (!ok) break;
        // ---- l summed over the lanes of each head slot; rows to the merge warp ----
#pragma unroll
        for (int ofs = 4; ofs < 32; ofs <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], ofs);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], ofs);
        }
        if (kPacked) {  // the remainders' sums (slots 4-7: lanes 2 further on) to the heads'
#pragma unroll
            for (int mt = 0; mt < kChunks; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    o[mt][k].x += __shfl_xor_sync(0xffffffffu, o[mt][k].x, 2);
                    o[mt][k].y += __shfl_xor_sync(0xffffffffu, o[mt][k].y, 2);
                }
        }
        const int splits = ONE ? 1 : (ut.lens[c.b] + chunk - 1) / chunk;
#pragma unroll
        for (int g0 = 0; g0 < G && ok; g0 += kMH) {  // the heads g0 .. g0 + kMH - 1
            if (!(ok = warp_wait(read, mphase ^ 1u, abort_flag, a.err))) break;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int g = 2 * tig + jj;
                if (g >= g0 && g < g0 + kMH && g < G) {
                    float *row = merge + ((size_t)warp * kMH + g - g0) * kMergeRow<D>;
#pragma unroll
                    for (int mt = 0; mt < kChunks; ++mt)  // M slot gid: dim 2gid of the chunk; gid + 8: dim 2gid + 1
                        *reinterpret_cast<float2 *>(row + mt * 16 + 2 * gid) =
                            jj ? make_float2(o[mt][0].y, o[mt][1].y) : make_float2(o[mt][0].x, o[mt][1].x);
                    // (every score NaN: the maximum passed over them; 0 lets the NaN sum through the merge)
                    if (gid == 0)
                        *reinterpret_cast<float2 *>(row + D) =
                            make_float2(m[jj] == -INFINITY && l[jj] != l[jj] ? 0.f : m[jj], l[jj]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(written);
            if (!(ok = warp_wait(written, mphase, abort_flag, a.err))) break;
            // ---- the merge of head g0 + warp: M = max m, weights 2^(m_w - M), out = sum w acc / sum w l ----
            const int g = g0 + warp;
            if (warp < kMH && g < G) {
                const float *row = merge + (size_t)warp * kMergeRow<D>;
                float2 ml[kWarps];
                float M = -INFINITY, sum = 0.f, acc[D / 32];
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    ml[i] = *reinterpret_cast<const float2 *>(row + (size_t)i * kMH * kMergeRow<D> + D);
                    M = fmaxf(M, ml[i].x);
                }
#pragma unroll
                for (int v = 0; v < D / 32; ++v) acc[v] = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float wt = ml[i].x == -INFINITY ? 0.f : ex2f(ml[i].x - M);
                    sum = fmaf(wt, ml[i].y, sum);
                    const float *r = row + (size_t)i * kMH * kMergeRow<D> + lane * (D / 32);
#pragma unroll
                    for (int v = 0; v < D / 32; ++v) acc[v] = fmaf(wt, r[v], acc[v]);
                }
                if constexpr (ONE) {  // the CTA's row, relative to M
                    float *mine = cta_rows + (size_t)g * kMergeRow<D>;
#pragma unroll
                    for (int v = 0; v < D / 32; ++v) mine[lane * (D / 32) + v] = acc[v];
                    if (lane == 0) *reinterpret_cast<float2 *>(mine + D) = make_float2(M, sum);
                } else {
                    const float inv = 1.f / sum;  // (a unit has a token, so the sum is above 0, or NaN)
#pragma unroll
                    for (int v = 0; v < D / 32; ++v) acc[v] *= inv;
                    const float lse = (M + __log2f(sum)) * kLn2;
                    const size_t head = (size_t)c.kvh * G + g;
                    if (splits == 1) {
                        const size_t row_o = (size_t)ut.qrow[c.b] * a.num_q_heads + head;
                        store_out_vec<D / 32>(a.out, row_o * D + lane * (D / 32), acc, a.out_dtype);
                        if (a.lse && lane == 0) a.lse[row_o] = lse;
                    } else {
                        const size_t row_p = ((size_t)c.b * a.num_q_heads + head) * a.s_max + c.split;
                        store_out_vec<D / 32>(a.part_o, row_p * D + lane * (D / 32), acc, 2);
                        if (lane == 0) a.part_lse[row_p] = lse;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(read);
            mphase ^= 1u;
        }
        if (!ok) break;
    }
    if (!ok) {
        // let copies in flight land before the CTA exits (bounded)
        volatile int no_abort = 0;
        for (; taken < issued; ++taken) mbar_wait(&full[taken % S], (taken / S) & 1u, &no_abort, nullptr);
    }
    if constexpr (ONE) {
        // ---- the cluster's rows: head g by warp g / n of CTA g % n; every CTA comes here, whatever its waits did ----
        cluster_barrier();
        const int n = cluster_size();
        for (int g = warp * n + cluster_rank(); g < G; g += n * kWarps) {
            const float *row = cta_rows + (size_t)g * kMergeRow<D>;
            const float2 ml = lane < n ? ld_cluster2(smem_of(row + D, lane)) : make_float2(-INFINITY, 0.f);
            float M = ml.x;
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
            const float wt = ml.x == -INFINITY ? 0.f : ex2f(ml.x - M);
            float sum = ml.x == -INFINITY ? 0.f : wt * ml.y;  // (a CTA without keys: 0; a NaN stays one at any weight)
            float2 acc[D / 64];
#pragma unroll
            for (int v = 0; v < D / 64; ++v) acc[v] = make_float2(0.f, 0.f);
            for (int i0 = 0; i0 < n; i0 += 4) {
                float2 x[4][D / 64];
#pragma unroll
                for (int i = 0; i < 4; ++i)  // (n is 1, 2 or a multiple of 4)
#pragma unroll
                    for (int v = 0; v < D / 64; ++v)
                        x[i][v] = ld_cluster2(smem_of(row + v * 64 + lane * 2, i0 + i < n ? i0 + i : i0));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = i0 + i < n ? __shfl_sync(0xffffffffu, wt, i0 + i) : 0.f;
#pragma unroll
                    for (int v = 0; v < D / 64; ++v) acc[v] = ffma2(make_float2(w, w), x[i][v], acc[v]);
                }
            }
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            const bool empty = M == -INFINITY;  // an empty context
            const float inv = empty ? 0.f : 1.f / sum;
            const size_t row_o = (size_t)one_row * a.num_q_heads + (size_t)one.kvh * G + g;
            if (ok && one_mine) {
#pragma unroll
                for (int v = 0; v < D / 64; ++v) {
                    const float o2[2] = {acc[v].x * inv, acc[v].y * inv};
                    store_out_vec<2>(a.out, row_o * D + v * 64 + lane * 2, o2, a.out_dtype);
                }
                if (a.lse && lane == 0) a.lse[row_o] = empty ? -INFINITY : (M + __log2f(sum)) * kLn2;
            }
        }
        cluster_barrier();  // (no CTA leaves before its rows have been read)
    }
    pdl_launch_dependents();  // (at the start instead: one request 9.7 -> 9.4 us, but the mixed batch 37 -> 40)
}

// (volatile: issued where they stand, ahead of the arithmetic)
__device__ __forceinline__ float ld_part(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void ld_part_vec(const float *p, float (&v)[4]) {
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
}
__device__ __forceinline__ void ld_part_vec(const float *p, float (&v)[2]) {
    asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
}

// Log-sum-exp merge of the splits' partials: one CTA a row (sequence, query head), its warps a share of the splits each,
// all of a warp's loads in flight at once (combine_kernel, a warp a row, takes 33 splits in five rounds of
// loads: 3 us of a single request's 12).
template <int D>
__global__ void __launch_bounds__(128) merge_splits_kernel(CombineArgs a) {
    constexpr int W = 4, V = D / 32, kBatch = 8;
    __shared__ float part[W][D + 2];
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = row / a.rows_per_seq;
    pdl_wait();  // lengths may come from the kernel before the split kernel, the partials come from it
    const int len = max(__ldg(a.context_lens + b), 0);
    const int S = min(len > 0 ? (len - 1) / a.chunk + 1 : 0, a.num_splits);
    size_t out_row = row;
    if (a.cu_q_lens) {  // mixed batch: rows of prefill chunks are not this kernel's
        const int q0 = __ldg(a.cu_q_lens + b);
        if (__ldg(a.cu_q_lens + b + 1) - q0 != 1) return;
        out_row = (size_t)q0 * a.rows_per_seq + (row - b * a.rows_per_seq);
    }
    if (S == 1) return;  // finished by the split kernel
    const float *pl = a.part_lse + (size_t)row * a.num_splits;
    const float *po = a.part_o + (size_t)row * a.num_splits * D + V * lane;
    float M = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int s0 = warp; s0 < S; s0 += W * kBatch) {
        float x[kBatch][V], ls[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int s = s0 + i * W;
            ls[i] = -INFINITY;
            if (s < S) {
                ls[i] = ld_part(pl + s);
                ld_part_vec(po + (size_t)s * D, x[i]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) x[i][v] = 0.f;
            }
        }
        float m = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m = fmaxf(m, ls[i]);
        // (every lse NaN so far: 0 lets them through)
        const float mm = m == -INFINITY ? 0.f : m, al = M == -INFINITY ? 0.f : ex2f((M - mm) * kLog2e);
        if (M != -INFINITY || sum != sum) {
            sum *= M == -INFINITY ? 1.f : al;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= M == -INFINITY ? 1.f : al;
        }
        M = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float w = ls[i] == -INFINITY ? 0.f : ex2f((ls[i] - mm) * kLog2e);
            sum += w;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[i][v], acc[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) part[warp][V * lane + v] = acc[v];
    if (lane == 0) {
        part[warp][D] = M;
        part[warp][D + 1] = sum;
    }
    __syncthreads();
    float top = -INFINITY, total = 0.f, wt[W];
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, part[i][D]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        // (a warp without a maximum has a sum of 0, or one of NaN relative to 0)
        wt[i] = part[i][D] == -INFINITY ? 1.f : ex2f((part[i][D] - ref) * kLog2e);
        total = fmaf(wt[i], part[i][D + 1], total);
    }
    const float inv = S > 0 ? 1.f / total : 0.f;
    if (threadIdx.x < D / 2) {
        float o[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int v = 0; v < 2; ++v) o[v] = fmaf(wt[i], part[i][2 * threadIdx.x + v], o[v]);
        o[0] *= inv;
        o[1] *= inv;
        store_out_vec<2>(a.out, out_row * D + 2 * threadIdx.x, o, a.out_dtype);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[out_row] = S > 0 ? ref + logf(total) : -INFINITY;
    pdl_launch_dependents();
}

template <int D, int G, bool ONE>
auto configured_kernel(cudaError_t &e) {
    auto kern = decode_int8_kernel<D, G, ONE>;
    static DeviceFlags configured;
    const int dev = device_info().device;
    e = cudaSuccess;
    if (!configured.test(dev)) {
        e = set_smem_attributes(kern, device_info().max_smem);
        if (ONE && e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) configured.set(dev);
    }
    return kern;
}

// Asked once a device: the cluster sizes that have a place on it (0 where the device does not say: then it is asked again).
template <int D, int G>
int cluster_sizes() {
    static std::atomic<int> known[64];  // the sizes, and 32 once they are
    const int dev = device_info().device;
    if (dev < 0 || dev >= 64) return 0;
    int sizes = known[dev].load(std::memory_order_relaxed);
    if (sizes) return sizes & 31;
    cudaError_t e;
    auto kern = configured_kernel<D, G, true>(e);
    for (int n = 1; n <= 16 && e == cudaSuccess; n *= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)n);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Int8Layout<D, G>::smem_bytes_one();
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)n;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
        // (a size that the device refuses outright is one without a place)
        if (e == cudaErrorInvalidClusterSize) {
            (void)cudaGetLastError();
            e = cudaSuccess;
            clusters = 0;
        }
        if (clusters > 0) sizes |= n;
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[dev].store(sizes | 32, std::memory_order_relaxed);
    return sizes;
}

template <int D, int G, bool ONE>
cudaError_t launch_t(const DecodeArgs &a, int grid, cudaStream_t s) {
    CUtensorMap tm;
    cudaError_t e = encode_int8_map(a.cache, a.cache.block_size < kTile<D> ? a.cache.block_size : kTile<D>, 2, &tm);
    if (e != cudaSuccess) return e;
    auto kern = configured_kernel<D, G, ONE>(e);
    if (e != cudaSuccess) return e;
    if (ONE) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(a.batch * a.cache.num_kv_heads * a.head_groups * a.cluster));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Int8Layout<D, G>::smem_bytes_one();
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)a.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kern, tm, a);
    }
    // as many CTAs an SM as fit in its shared memory (one CTA's maximum plus its 1 KB reserve, less a reserve each)
    const size_t smem = Int8Layout<D, G>::smem_bytes(a.batch, a.s_max);
    int ctas = (int)(((size_t)device_info().max_smem + 1024) / (smem + 1024));
    ctas = ctas > kCtasPerSm ? kCtasPerSm : ctas < 1 ? 1 : ctas;
    return launch_pdl(kern, dim3(grid * ctas), dim3(kThreads), smem, s, tm, a);
}

template <int D, int G>
cudaError_t launch_g(const DecodeArgs &a, int grid, cudaStream_t s) {
    return a.cluster > 0 ? launch_t<D, G, true>(a, grid, s) : launch_t<D, G, false>(a, grid, s);
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

template <int D>
int cluster_sizes_of(int heads) {
    switch (heads) {
        case 1: return cluster_sizes<D, 1>();
        case 2: return cluster_sizes<D, 2>();
        case 3: return cluster_sizes<D, 3>();
        case 4: return cluster_sizes<D, 4>();
        case 5: return cluster_sizes<D, 5>();
        case 6: return cluster_sizes<D, 6>();
        case 7: return cluster_sizes<D, 7>();
        case 8: return cluster_sizes<D, 8>();
        default: return 0;
    }
}

}  // namespace

int decode_int8_cluster_sizes(int head_dim, int heads) {
    return head_dim == 128 ? cluster_sizes_of<128>(heads) : head_dim == 64 ? cluster_sizes_of<64>(heads) : 0;
}

cudaError_t launch_merge_splits(const CombineArgs &a, cudaStream_t s) {
    if (a.n_rows == 0) return cudaSuccess;
    if (a.head_dim == 128) return launch_pdl(merge_splits_kernel<128>, dim3(a.n_rows), dim3(128), 0, s, a);
    return launch_pdl(merge_splits_kernel<64>, dim3(a.n_rows), dim3(128), 0, s, a);
}

cudaError_t launch_decode_int8(const DecodeArgs &a, int grid, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    return a.cache.head_dim == 128 ? launch_d<128>(a, grid, s) : launch_d<64>(a, grid, s);
}

}  // namespace pkv

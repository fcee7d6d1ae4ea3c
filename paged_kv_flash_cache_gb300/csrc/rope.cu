// rope.cu -- rope_append: what stands between a layer's projections and its attention over the paged
// cache, in one pass: the RMS norm of each query and key head (optional), the rotation of their leading
// rotary_dim elements by the token's position, the queries written out and the keys and values written
// into their pages ("企业官网建设流程全解析", section 2.1; layout of "Flash Attention与Paged Attention如何
// 共同优化大模型推理？", section 3).
//
// Mathematics, per head row x of D elements, in FP32:
//   norm     x <- x * rsqrt(mean(x^2) + eps) * w
//   rotation pair i of rotary_dim / 2 (elements i and i + rotary_dim / 2, or 2i and 2i + 1) turned by
//            the angle t = position * inv_freq[i], times mscale:
//            (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t)
// and one rounding to the 16-bit type (or, for the keys of an FP8 cache, straight to E4M3 codes and the
// row's scale, as the append quantises).
//
// The angle: position * inv_freq reaches 10^5 radians and more in a long context, where an FP32 product
// is off by hundredths. Only the angle's fraction of a turn matters, and integers wrap for free: with
// F = frac(inv_freq / 2 pi) as a 64-bit fraction (a few FP64 operations per frequency and warp, 1 / 2 pi in two FP64
// words), F * position modulo 2^64 is the fraction of a turn, to 2^-24 of a turn or better for every int32 position and
// |inv_freq| up to 2^40; its top 32 bits, as a signed number of half turns, go to sincospif.
//
// One warp per (token, share of its rows). A row is held by D / 16 lanes, each with two 16-byte vectors that hold whole
// pairs: vectors j and j + rotary_dim / 16 of the half layout, 2j and 2j + 1 of the interleaved one and of the elements
// behind rotary_dim. Either way lane j's pairs are those of frequencies 8j .. 8j + 7, so its cosines and sines,
// multiplied by the norm's weights, stay in registers over the token's query rows and over its key rows. The
// warp evaluates each frequency of its token once (a lane per frequency) and hands them out through shared memory, and
// looks up where its next 32 tokens go, a lane a token. A group of rows (kUnroll passes of 512 / D rows, 4 KB) is one
// run of memory and arrives by one bulk copy, kSlots groups ahead of the arithmetic: 192 KB an SM on their way, where
// registers held 64.
// Bound: HBM (a row is read once and written once), close behind it the instructions: two elements each where there is an
// instruction for it (fma.rn.f32x2), and rows of one kind in a straight line. 8192 tokens of 32 + 8 + 8 heads x 128, normed
// (201 MB): 37 us, 81% of the copy rate; 47 us with scalar arithmetic and the kind of row decided row by row, 66 us so with one
// vector a lane and the other element by shuffle (41 against 25 million warp instructions).
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kWarps = kRopeThreads / 32;
constexpr int kUnroll = 4;  // passes (of 512 / D rows) of a group
constexpr int kGroupBytes = kUnroll * 1024;
// CTAs an SM, and groups of a warp on their way or in work: with a norm the coefficients of two kinds of weights take
// registers for 4 CTAs (3 slots each: 37 us for the prompts above; 6 of 2 spill, 48 us). Without one 6 are better (4099 tokens
// into an FP8 cache: 33 us against 38), though their 80 registers make most of those kernels spill a little, 8 to 52 bytes
// (the prompts above without norms: 37.5 us; 5 CTAs have not been tried there).
template <bool NORM>
struct RopeShape {
    static constexpr int kCtas = NORM ? 4 : 6;
    static constexpr int kSlots = NORM ? 3 : 2;
    static constexpr int kSmem = kWarps * kSlots * kGroupBytes;
};

// 1 / 2 pi in two FP64 words
constexpr double kInvTwoPi = 0.15915494309189533577, kInvTwoPiLow = -9.839338337591243e-18;

template <bool BF16>
__device__ __forceinline__ void unpack_row(const uint4 &raw, float2 (&f)[4]) {
    if constexpr (BF16) unpack8x2(raw, f, BF16Tag());
    else unpack8x2(raw, f, F16Tag());
}

template <bool BF16>
__device__ __forceinline__ uint4 pack_row(const float2 (&f)[4]) {
    return make_uint4(pack_pair<BF16>(f[0].x, f[0].y), pack_pair<BF16>(f[1].x, f[1].y), pack_pair<BF16>(f[2].x, f[2].y),
                      pack_pair<BF16>(f[3].x, f[3].y));
}

// Eight E4M3 codes of f * inv.
__device__ __forceinline__ uint2 codes_of(const float2 (&f)[4], float inv) {
    float2 g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = fmul2(f[i], make_float2(inv, inv));
    return make_uint2(pack_e4m3x2(g[0].x, g[0].y) | (pack_e4m3x2(g[1].x, g[1].y) << 16),
                      pack_e4m3x2(g[2].x, g[2].y) | (pack_e4m3x2(g[3].x, g[3].y) << 16));
}

// Sequence of new token t: the last b with cu[b] <= t (t < cu[batch]).
__device__ __forceinline__ int sequence_of(const int *cu, int batch, int t) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Row of new token t's K in head 0 of its page (rows of the cache counted [page][K, V][head][offset]), or -1 (error
// word set) for a position outside the table or a page outside the pool.
__device__ __forceinline__ long long token_row(const RopeArgs &a, int t) {
    const int b = sequence_of(a.cu_new_lens, a.batch, t);
    const long long pos = (long long)a.ctx_before[b] + (t - a.cu_new_lens[b]);
    const long long logical = pos >> a.log2_block_size;
    int pb = -1;
    if (pos >= 0 && logical < a.max_blocks_per_seq) pb = __ldg(a.block_tables + (size_t)b * a.max_blocks_per_seq + logical);
    if (pb < 0 || pb >= a.num_blocks) {
        set_error(a.err, kErrDeviceRange);
        return -1;
    }
    return (long long)pb * 2 * a.num_kv_heads * a.block_size + (pos & (a.block_size - 1));
}

// What a lane multiplies its two vectors of a row by. Half layout: (a, b) -> (a c0 + b s1, b c1 + a s0) with c0, s0 =
// cos, sin times a's weight and c1, s1 = cos, -sin times b's. Interleaved: the pair (x0, x1) of one vector -> x c +
// (x1, x0) s with c = (w0 cos, w1 cos), s = (-w1 sin, w0 sin). Lanes behind rotary_dim: the weights (c) alone.
struct Coefficients {
    float2 c0[4], c1[4], s0[4], s1[4];
};

template <bool BF16, bool INTER, bool NORM>
__device__ __forceinline__ void fill(Coefficients &k, const void *w, const float *cosines, const float *sines, int va,
                                     int vb, bool rotates) {
    float2 wa[4], wb[4];
    if (NORM && w) {
        unpack_row<BF16>(__ldg(static_cast<const uint4 *>(w) + va), wa);
        unpack_row<BF16>(__ldg(static_cast<const uint4 *>(w) + vb), wb);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[i] = wb[i] = make_float2(1.f, 1.f);
    }
    if (!rotates) {
#pragma unroll
        for (int i = 0; i < 4; ++i) k.c0[i] = wa[i], k.c1[i] = wb[i], k.s0[i] = k.s1[i] = make_float2(0.f, 0.f);
        return;
    }
    float2 c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = reinterpret_cast<const float2 *>(cosines)[i];
        s[i] = reinterpret_cast<const float2 *>(sines)[i];
    }
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // pairs i of vector a, 4 + i of vector b
            const float ca = i & 1 ? c[i / 2].y : c[i / 2].x, sa = i & 1 ? s[i / 2].y : s[i / 2].x;
            const float cb = i & 1 ? c[2 + i / 2].y : c[2 + i / 2].x, sb = i & 1 ? s[2 + i / 2].y : s[2 + i / 2].x;
            k.c0[i] = make_float2(wa[i].x * ca, wa[i].y * ca);
            k.s0[i] = make_float2(-wa[i].y * sa, wa[i].x * sa);
            k.c1[i] = make_float2(wb[i].x * cb, wb[i].y * cb);
            k.s1[i] = make_float2(-wb[i].y * sb, wb[i].x * sb);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k.c0[i] = fmul2(c[i], wa[i]);
            k.s0[i] = fmul2(s[i], wa[i]);
            k.c1[i] = fmul2(c[i], wb[i]);
            k.s1[i] = fmul2(make_float2(-s[i].x, -s[i].y), wb[i]);
        }
    }
}

// Norm (if `normed`) and rotation of a lane's two vectors of a row.
template <int D, bool INTER, bool NORM>
__device__ __forceinline__ void turn_row(float2 (&fa)[4], float2 (&fb)[4], const Coefficients &k, bool normed, float eps,
                                         bool rotates) {
    float2 rs2 = make_float2(1.f, 1.f);
    if (NORM) {
        float2 q = fmul2(fa[0], fa[0]), r = fmul2(fb[0], fb[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) q = ffma2(fa[i], fa[i], q), r = ffma2(fb[i], fb[i], r);
        q = fadd2(q, r);
        float ss = q.x + q.y;
#pragma unroll
        for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = normed ? rsqrtf(ss * (1.f / D) + eps) : 1.f;
        rs2 = make_float2(rs, rs);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = fa[i], y = fb[i];
        fa[i] = fmul2(x, k.c0[i]);
        fb[i] = fmul2(y, k.c1[i]);
        if (rotates) {  // (an element behind rotary_dim meets no other one: not even as 0 * infinity)
            fa[i] = ffma2(INTER ? make_float2(x.y, x.x) : y, INTER ? k.s0[i] : k.s1[i], fa[i]);
            fb[i] = ffma2(INTER ? make_float2(y.y, y.x) : x, INTER ? k.s1[i] : k.s0[i], fb[i]);
        }
        if (NORM) fa[i] = fmul2(fa[i], rs2), fb[i] = fmul2(fb[i], rs2);
    }
}

// An FP8 row: the codes of a lane's two vectors and the row's scale. A row with a NaN gets the scale NaN (and codes of 0
// where its elements are finite), one with an infinity an infinite scale and NaN codes: none of its elements reads as a number.
// A row of magnitudes up to kZeroRow, whose 448 / amax may be beyond FP32, is stored as one of zeros.
constexpr float kZeroRow = 0x1p-119f;

template <int D>
__device__ __forceinline__ void store_codes(const RopeArgs &a, size_t row, const float2 (&fa)[4], const float2 (&fb)[4],
                                            int va, int vb, bool first, bool live) {
    float amax = kZeroRow;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        amax = fmax3_nan(fmax3_nan(amax, fabsf(fa[i].x), fabsf(fa[i].y)), fabsf(fb[i].x), fabsf(fb[i].y));
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // one division: the row's first lane makes the scale, the others 448 / amax, which the first takes from its neighbour
    const float quotient = (first ? amax : 448.0f) / (first ? 448.0f : amax);
    const float inv = __shfl_down_sync(0xffffffffu, quotient, first ? 1 : 0);
    if (!live) return;
    uint2 ca = make_uint2(0u, 0u), cb = ca;
    float scale = 0.f;
    if (amax != kZeroRow) {
        scale = quotient;
        const float times = amax > 0.f ? inv : 0.f;  // (not of a NaN)
        ca = codes_of(fa, times);
        cb = codes_of(fb, times);
    }
    uint2 *dst = static_cast<uint2 *>(a.cache) + row * (D / 8);
    dst[va] = ca;
    dst[vb] = cb;
    if (first) a.scales[row] = scale;
}

// NORM: a query or key weight is given (a missing one of the two: that side is not normed).
template <int D, bool BF16, bool FP8, bool INTER, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, RopeShape<NORM>::kCtas) rope_append_kernel(RopeArgs a) {
    constexpr int kSlots = RopeShape<NORM>::kSlots;
    constexpr int kLanes = D / 16;         // lanes a row
    constexpr int kRows = 32 / kLanes;     // rows a pass
    constexpr int kGroup = kUnroll * kRows;  // rows a group
    constexpr int kFreqs = D / 2;
    constexpr int kPer = (kFreqs + 31) / 32;  // frequencies a lane evaluates
    extern __shared__ __align__(128) uint8_t s_rows[];  // [kWarps][kSlots] groups
    __shared__ uint64_t s_full[kWarps][kSlots];
    __shared__ volatile int s_abort;
    __shared__ __align__(16) float s_cos[kWarps][kFreqs], s_sin[kWarps][kFreqs];
    __shared__ long long s_row[kWarps][32];  // token_row and position of the warp's next 32 tokens
    __shared__ int s_pos[kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = lane % kLanes, sub = lane / kLanes;
    const int rot_lanes = a.rotary_dim / 16;
    const bool rotates = j < rot_lanes;
    const int va = (!INTER && rotates) ? j : 2 * j, vb = (!INTER && rotates) ? j + rot_lanes : 2 * j + 1;
    const int hq = a.num_q_heads, hkv = a.num_kv_heads;
    // groups of rows: the query rows', the key rows', the value rows'; this warp's share of every token of its own
    const int gq = (hq + kGroup - 1) / kGroup, gk = (hkv + kGroup - 1) / kGroup;
    const int share = blockIdx.y, g_begin = share * a.share_groups, g_end = min(gq + 2 * gk, g_begin + a.share_groups);

    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < kSlots; ++i) mbar_init(&s_full[w][i], 1);
        s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();  // the projections come from the previous kernel, which may also still read the pages
    // F = frac(inv_freq / 2 pi) in 64 bits, signed: what the product is from the nearest whole turn, rounded once, and the
    // second word's part, which counts for frequencies above one radian a position
    unsigned long long turn[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int f = lane + 32 * i;
        turn[i] = 0;
        if (f < a.rotary_dim / 2) {
            const double w = (double)__ldg(a.inv_freq + f);
            const double x = __fma_rn(w, kInvTwoPi, -rint(__dmul_rn(w, kInvTwoPi)));
            turn[i] = (unsigned long long)(long long)(x * 0x1p64) +
                      (unsigned long long)(long long)(w * (kInvTwoPiLow * 0x1p64));
        }
    }
    const int total = min(a.num_new_tokens, __ldg(a.cu_new_lens + a.batch));  // tokens behind the last sequence: left alone
    const int stride = gridDim.x * kWarps;
    // the groups of this warp's tokens in order: the next one to fetch, and the fetched and used ones so far
    const uint64_t pol = l2_policy_evict_first();
    uint8_t *const my_rows = s_rows + warp * kSlots * kGroupBytes;
    int ft = blockIdx.x * kWarps + warp, fg = g_begin;
    uint32_t fetched = 0, used = 0;
    auto fetch = [&]() {
        if (ft >= total) return;
        const int kind = fg < gq ? 0 : fg < gq + gk ? 1 : 2;
        const int h0 = (fg - (kind == 0 ? 0 : kind == 1 ? gq : gq + gk)) * kGroup;
        if (tc::elect_one()) {
            const uint16_t *src = static_cast<const uint16_t *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                                  (size_t)ft * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (size_t)h0 * D;
            const uint32_t bytes = (uint32_t)min(kGroup, (kind == 0 ? hq : hkv) - h0) * D * 2u;
            uint64_t *bar = &s_full[warp][fetched % kSlots];
            mbar_arrive_expect_tx(bar, bytes);
            bulk_g2s(my_rows + (fetched % kSlots) * kGroupBytes, src, bytes, bar, pol);
        }
        ++fetched;
        if (++fg == g_end) {
            fg = g_begin;
            ft += stride;
        }
    };
    // this lane's vectors of row u * kRows + sub of the group in work
    const uint4 *group = nullptr;
    auto next_group = [&]() -> bool {
        group = reinterpret_cast<const uint4 *>(my_rows + (used % kSlots) * kGroupBytes) + sub * (D / 8);
        return mbar_wait(&s_full[warp][used % kSlots], (used / kSlots) & 1u, &s_abort, a.err);
    };
    auto done_group = [&]() {
        ++used;
        __syncwarp();  // every lane has read it
        fetch();
    };
#pragma unroll
    for (int i = 0; i < kSlots; ++i) fetch();
    bool ok = true;
    int n = 0;  // tokens of this warp so far
    for (int t = blockIdx.x * kWarps + warp; ok && t < total; t += stride, ++n) {
        const int at = n & 31;
        if (at == 0) {
            __syncwarp();
            const long long mine = t + (long long)lane * stride;
            if (mine < total) {
                s_pos[warp][lane] = __ldg(a.positions + mine);
                if (g_end > gq) s_row[warp][lane] = token_row(a, (int)mine);
            }
        }
        __syncwarp();  // (and the last token's cosines are read)
        const int pos = s_pos[warp][at];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int f = lane + 32 * i;
            if (f < a.rotary_dim / 2) {
                const int half_turns = (int)((turn[i] * (unsigned long long)(long long)pos) >> 32);  // of 2^-31
                float sn, cs;
                sincospif((float)half_turns * 4.656612873077393e-10f, &sn, &cs);
                s_cos[warp][f] = cs * a.mscale;
                s_sin[warp][f] = sn * a.mscale;
            }
        }
        __syncwarp();
        Coefficients k;
        if (g_begin < gq) {
            fill<BF16, INTER, NORM>(k, a.q_weight, &s_cos[warp][8 * j], &s_sin[warp][8 * j], va, vb, rotates);
            const int end = min(g_end, gq);
            for (int g = g_begin; ok && g < end; ++g) {
                const int h0 = g * kGroup;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.q_out) + (size_t)t * a.q_out_stride) +
                             (size_t)(h0 + sub) * (D / 8);
                if (!(ok = next_group())) break;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float2 fa[4], fb[4];
                    unpack_row<BF16>(group[64 * u + va], fa);
                    unpack_row<BF16>(group[64 * u + vb], fb);
                    turn_row<D, INTER, NORM>(fa, fb, k, a.q_weight != nullptr, a.eps, rotates);
                    if (h0 + u * kRows + sub < hq) {
                        dst[va + 64 * u] = pack_row<BF16>(fa);
                        dst[vb + 64 * u] = pack_row<BF16>(fb);
                    }
                }
                done_group();
            }
        }
        if (g_end <= gq) continue;
        const long long page_row = s_row[warp][at];  // K of head 0
        for (int g = max(g_begin, gq); ok && g < g_end; ++g) {
            const bool is_v = g >= gq + gk;
            const int h0 = (g - gq - (is_v ? gk : 0)) * kGroup;
            size_t row = (size_t)page_row + (size_t)((is_v ? hkv : 0) + h0 + sub) * a.block_size;
            if (!is_v && (g == gq || g == g_begin))
                fill<BF16, INTER, NORM>(k, a.k_weight, &s_cos[warp][8 * j], &s_sin[warp][8 * j], va, vb, rotates);
            if (!(ok = next_group())) break;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u, row += (size_t)kRows * a.block_size) {
                const bool live = h0 + u * kRows + sub < hkv && page_row >= 0;
                if (h0 + u * kRows >= hkv) break;  // uniform
                const uint4 xa = group[64 * u + va], xb = group[64 * u + vb];
                float2 fa[4], fb[4];
                if (FP8 || !is_v) {
                    unpack_row<BF16>(xa, fa);
                    unpack_row<BF16>(xb, fb);
                }
                if (!is_v) turn_row<D, INTER, NORM>(fa, fb, k, a.k_weight != nullptr, a.eps, rotates);
                if constexpr (FP8) {
                    store_codes<D>(a, row, fa, fb, va, vb, j == 0, live);
                } else if (live) {
                    uint4 *dst = static_cast<uint4 *>(a.cache) + row * (D / 8);
                    dst[va] = is_v ? xa : pack_row<BF16>(fa);  // values: the input's bits
                    dst[vb] = is_v ? xb : pack_row<BF16>(fb);
                }
            }
            done_group();
        }
    }
    if (!ok) {  // a copy did not land in time: let the others land before the CTA exits (bounded)
        volatile int no_abort = 0;
        for (; used != fetched; ++used) mbar_wait(&s_full[warp][used % kSlots], (used / kSlots) & 1u, &no_abort, nullptr);
    }
    pdl_launch_dependents();
}

template <int D, bool BF16, bool FP8, bool INTER, bool NORM>
cudaError_t launch_rope_n(const RopeArgs &a, dim3 grid, cudaStream_t s) {
    auto kern = rope_append_kernel<D, BF16, FP8, INTER, NORM>;
    static DeviceFlags configured;
    const int dev = device_info().device;
    if (!configured.test(dev)) {
        const cudaError_t e = set_smem_attributes(kern, RopeShape<NORM>::kSmem);
        if (e != cudaSuccess) return e;
        configured.set(dev);
    }
    return launch_pdl(kern, grid, dim3(kRopeThreads), RopeShape<NORM>::kSmem, s, a);
}

template <int D, bool BF16, bool FP8, bool INTER>
cudaError_t launch_rope_i(const RopeArgs &a, dim3 grid, cudaStream_t s) {
    return a.q_weight || a.k_weight ? launch_rope_n<D, BF16, FP8, INTER, true>(a, grid, s)
                                    : launch_rope_n<D, BF16, FP8, INTER, false>(a, grid, s);
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_rope_t(const RopeArgs &a, dim3 grid, cudaStream_t s) {
    return a.interleaved ? launch_rope_i<D, BF16, FP8, true>(a, grid, s) : launch_rope_i<D, BF16, FP8, false>(a, grid, s);
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs &a, dim3 grid, cudaStream_t s) {
    if constexpr (D <= 128) {
        if (a.fp8)
            return a.dtype == 1 ? launch_rope_t<D, true, true>(a, grid, s) : launch_rope_t<D, false, true>(a, grid, s);
    }
    return a.dtype == 1 ? launch_rope_t<D, true, false>(a, grid, s) : launch_rope_t<D, false, false>(a, grid, s);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t s) {
    const int rows = kUnroll * 512 / a.head_dim;  // of a group
    const int groups = (a.num_q_heads + rows - 1) / rows + 2 * ((a.num_kv_heads + rows - 1) / rows);
    // A token a warp over the CTAs that are resident together; a token's groups go to several warps while there are fewer
    // than eight tokens for each of those (a few tokens a warp would not divide evenly).
    const int cap = device_info().num_sms * (a.q_weight || a.k_weight ? RopeShape<true>::kCtas : RopeShape<false>::kCtas);
    const long long warps = (long long)cap * kWarps;
    long long shares = (8 * warps + a.num_new_tokens - 1) / a.num_new_tokens;
    if (shares > groups) shares = groups;
    RopeArgs r = a;
    r.share_groups = (int)((groups + shares - 1) / shares);
    const int y = (groups + r.share_groups - 1) / r.share_groups;
    const int ctas = (a.num_new_tokens + kWarps - 1) / kWarps, most = (cap + y - 1) / y;
    const dim3 grid(ctas < most ? ctas : most, y);
    if (a.head_dim == 256) return launch_rope_d<256>(r, grid, s);
    if (a.head_dim == 128) return launch_rope_d<128>(r, grid, s);
    return launch_rope_d<64>(r, grid, s);
}

}  // namespace pkv

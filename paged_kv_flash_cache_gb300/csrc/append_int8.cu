// append_int8.cu -- kv_cache_append into an INT8 cache: one scale per (page, K or V, KV head).
//
// element = code * scale, codes in [-127, 127]. For the rows that a call writes into one page of one head, of
// largest magnitude a, the page's scale becomes
//   the least power of two s >= 2^-126 with a <= 127 s (0 for a = 0) where the page has no older rows;
//   the old scale where it has some and a <= 127 s_old; else the power of two again, and the older codes c become
//   rne(c * s_old / s).
// New codes are rne(x / s). Powers of two make both scalings exact, so each code is one rounding away from what it
// stands for, and a row that was rounded again k times is off by at most 1/2 + 1/4 + ... < 1 step of the last
// scale, however often the scale grew. A row that holds a NaN or an infinity makes the scale NaN: the page reads
// as NaN until it starts again.
//
// The unit of work is a page of a head, so that the rows that share a scale meet in one group of warps: no atomics,
// no second launch. The pages that a call touches are not known on the host (lengths live on the device), but
// sequence b's are at most new_b / bs + 2, so slot numbers base_b = cu[b] / bs + 2 b leave room for all of them and
// a warp finds its sequence by a search over base_b; where that is more slots than tokens (decode steps), the slots
// are the tokens and the first one of each page does the page. Rows stay in registers between the maximum and the
// codes (16 rows of 128 a warp); a page of more rows than its warps hold reads the rest twice, the second time from L2.
//
// Measured, back to back: 4 x 2048 tokens of 8 heads x 128 in pages of 16 (50 MB) 10.5 us, 70% of the copy rate; 3 x 1367
// tokens of 32 heads in pages of 64 (101 MB) 18.0 us, 82%; a token each of 64 sequences 2.7 us. 72 registers a thread, so that
// seven CTAs fit; f16 with one warp a page spills 40 bytes for it (the prompts again and again into L2: 7.5 us, bf16 7.2). A warp's one chain (lengths,
// page id, scale; its rows; the maximum; the codes) and the launch's ramp bound it, not the arithmetic (a third of the issue
// slots): with 16 vectors a lane the prompts take 15.7 us, with 4 13.6; six CTAs an SM instead of seven 10.9, eight 11.9.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarpsCta = kThreads / 32;
constexpr int kVecs = 8;  // 16-byte vectors a lane holds: 4 KB of rows a warp

__device__ __forceinline__ uint4 ld_row(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Largest magnitudes of two 16-bit lanes, NaN if one is NaN.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x, F16Tag) {
    __half2 a, b;
    memcpy(&a, &m, 4);
    memcpy(&b, &x, 4);
    a = __hmax2_nan(a, __habs2(b));
    memcpy(&m, &a, 4);
    return m;
}
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x, BF16Tag) {
    __nv_bfloat162 a, b;
    memcpy(&a, &m, 4);
    memcpy(&b, &x, 4);
    a = __hmax2_nan(a, __habs2(b));
    memcpy(&m, &a, 4);
    return m;
}

// The least power of two s >= 2^-126 with a <= 127 s, for finite a > 0: 127 = 1.984375 * 2^6.
__device__ __forceinline__ float pow2_scale(float a) {
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// Eight 16-bit values to eight codes rne(x * inv): x * inv + 1.5 * 2^23 keeps the rounded integer in the low bits.
template <typename Tag>
__device__ __forceinline__ uint2 codes8(const uint4 &raw, float inv) {
    constexpr float kMagic = 12582912.0f;
    float2 f[4];
    unpack8x2(raw, f, Tag());
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = ffma2(f[i], make_float2(inv, inv), make_float2(kMagic, kMagic));
        w[i] = __byte_perm(__float_as_uint(f[i].x), __float_as_uint(f[i].y), 0x0040);
    }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// Four codes times ratio, rounded to nearest even (|ratio| <= 1 after a growth).
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
    constexpr float kMagic = 12582912.0f;
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = (float)(signed char)(c >> (8 * i));
        r |= (__float_as_uint(fmaf(x, ratio, kMagic)) & 0xffu) << (8 * i);
    }
    return r;
}

// The last b in [0, batch) with base(b) <= slot (base non-decreasing, base(0) <= slot): 32 probes a round.
template <typename Base>
__device__ __forceinline__ int last_at_most(int batch, int lane, long long slot, Base base) {
    int lo = 0, n = batch;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, i < n && (lane == 0 || base(lo + i) <= slot));
        const int k = (__popc(in) - 1) * step;
        lo += k;
        n = min(step, n - k);
    }
    return lo;
}

// W warps a page of a head.
template <int D, int W, typename Tag>
__global__ void __launch_bounds__(kThreads, 7) append_int8_kernel(AppendArgs a, long long tasks, int by_token) {
    constexpr int kLanes = D / 8;               // lanes a row (16 bytes each)
    constexpr int kRowsLoad = 32 / kLanes;      // rows a load of the warp
    constexpr int kRowsWarp = kVecs * kRowsLoad;
    constexpr int kGroups = kWarpsCta / W;
    __shared__ float smax[kWarpsCta];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp % W, group = warp / W;
    const int sub = lane / kLanes, chk = lane % kLanes;
    const int hkv = a.num_kv_heads, bs = a.block_size;
    const long long task = (long long)blockIdx.x * kGroups + group;
    pdl_wait();  // the previous kernel may still read the pages this call writes
    if (task >= tasks) return;  // (all warps of the group)
    const long long slot = task / (2 * hkv);
    const int kvh = (int)(task - slot * (2 * hkv));
    const int kv = kvh >= hkv ? 1 : 0, h = kvh - kv * hkv;

    // ---- the page's new rows: tokens t0 .. t0 + n - 1, page rows off .. off + n - 1 ----
    int b;
    long long pos0, end;  // positions of the page's first new row, and behind the sequence's last
    int t0;
    if (!a.cu_new_lens) {  // one token a sequence
        b = (int)slot;
        t0 = b;
        pos0 = __ldg(a.ctx_before + b);
        end = pos0 + 1;
    } else {
        const int *cu = a.cu_new_lens;
        const int lb = a.log2_block_size;
        int c0, c1, ctx0;
        if (a.batch <= 32) {  // everything in one round trip
            const bool in = lane < a.batch;
            c0 = in ? __ldg(cu + lane) : 0;
            c1 = in ? __ldg(cu + lane + 1) : 0;
            ctx0 = in ? __ldg(a.ctx_before + lane) : 0;
            const long long base = by_token ? (long long)c0 : (long long)(c0 >> lb) + 2ll * lane;
            b = __popc(__ballot_sync(0xffffffffu, in && (lane == 0 || base <= slot))) - 1;
            c0 = __shfl_sync(0xffffffffu, c0, b);
            c1 = __shfl_sync(0xffffffffu, c1, b);
            ctx0 = __shfl_sync(0xffffffffu, ctx0, b);
        } else {
            b = by_token ? last_at_most(a.batch, lane, slot, [cu](int i) { return (long long)__ldg(cu + i); })
                         : last_at_most(a.batch, lane, slot,
                                        [cu, lb](int i) { return (long long)(__ldg(cu + i) >> lb) + 2ll * i; });
            c0 = __ldg(cu + b);
            c1 = __ldg(cu + b + 1);
            ctx0 = __ldg(a.ctx_before + b);
        }
        c1 = min(c1, a.num_new_tokens);
        if (c0 < 0) {
            if (lane == 0) set_error(a.err, kErrDeviceRange);
            return;
        }
        const long long ctx = ctx0;
        end = ctx + (c1 - c0);
        if (by_token) {
            pos0 = ctx + (slot - c0);
            if (slot >= c1 || (slot > c0 && (pos0 & (bs - 1)) != 0)) return;
        } else {
            const long long page = (ctx >> lb) + (slot - ((long long)(c0 >> lb) + 2ll * b));
            pos0 = page << lb;
            if (pos0 < ctx) pos0 = ctx;
            if (pos0 >= end) return;
        }
        t0 = c0 + (int)(pos0 - ctx);
    }
    const int off = (int)(pos0 & (bs - 1));
    const int n = (int)min((long long)(bs - off), end - pos0);

    // ---- the rows, and while they come the page and its scale ----
    const uint4 *src = static_cast<const uint4 *>(kv ? a.v_new : a.k_new) + ((size_t)t0 * hkv + h) * kLanes + chk;
    const size_t stride = (size_t)hkv * kLanes;
    uint4 raw[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int r = w * kRowsWarp + i * kRowsLoad + sub;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < n) raw[i] = ld_row(src + r * stride);
    }
    const long long logical = pos0 >> a.log2_block_size;
    if (pos0 < 0 || logical >= a.max_blocks_per_seq) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return;
    }
    const int pb = __ldg(a.block_tables + (size_t)b * a.max_blocks_per_seq + logical);
    if (pb < 0 || pb >= a.num_blocks) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return;
    }
    const size_t page = ((size_t)pb * 2 + kv) * hkv + h;
    float s_old = off > 0 ? a.scales[page] : 0.f;
    if (s_old < 1.17549435e-38f) s_old = 0.f;  // (written elsewhere: below 2^-126, whose reciprocal can overflow)

    // ---- the largest magnitude ----
    uint32_t m2 = 0u;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        m2 = amax2(m2, raw[i].x, Tag());
        m2 = amax2(m2, raw[i].y, Tag());
        m2 = amax2(m2, raw[i].z, Tag());
        m2 = amax2(m2, raw[i].w, Tag());
    }
    for (int r0 = (W + w) * kRowsWarp; r0 < n; r0 += W * kRowsWarp) {  // rows beyond those in registers
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int r = r0 + i * kRowsLoad + sub;
            if (r < n) {
                const uint4 x = ld_row(src + r * stride);
                m2 = amax2(m2, x.x, Tag());
                m2 = amax2(m2, x.y, Tag());
                m2 = amax2(m2, x.z, Tag());
                m2 = amax2(m2, x.w, Tag());
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m2 = amax2(m2, __shfl_xor_sync(0xffffffffu, m2, o), Tag());
    float2 f[4];
    unpack8x2(make_uint4(m2, 0u, 0u, 0u), f, Tag());
    float amax = fmax_nan(f[0].x, f[0].y);
    if constexpr (W > 1) {
        if (lane == 0) smax[warp] = amax;
        named_barrier(1 + group, W * 32);  // (also: every warp has read the old scale)
        amax = smax[group * W];
#pragma unroll
        for (int i = 1; i < W; ++i) amax = fmax_nan(amax, smax[group * W + i]);
    }

    // ---- the scale ----
    float s = s_old;
    if (!(amax < INFINITY) || !(s_old < INFINITY)) s = __uint_as_float(0x7fc00000u);  // not finite, or already so
    else if (amax > 127.f * s_old) s = pow2_scale(amax);
    // 1 / s: exact for a power of two; a NaN or zero scale leaves codes of 0
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const bool bad = !(s < INFINITY);
    if (w == 0 && lane == 0) a.scales[page] = s;
    int8_t *codes = static_cast<int8_t *>(a.cache) + page * bs * D;

    // ---- older rows, rounded again where the scale grew ----
    if (off > 0 && s > s_old) {
        const float ratio = s_old * inv;
        constexpr int kVecRow = D / 16;
        uint4 *old = reinterpret_cast<uint4 *>(codes);
        for (int v = w * 32 + lane; v < off * kVecRow; v += W * 32) {
            uint4 x = old[v];
            x.x = rescale4(x.x, ratio);
            x.y = rescale4(x.y, ratio);
            x.z = rescale4(x.z, ratio);
            x.w = rescale4(x.w, ratio);
            old[v] = x;
        }
    }

    // ---- the codes ----
    uint2 *dst = reinterpret_cast<uint2 *>(codes + (size_t)off * D) + chk;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int r = w * kRowsWarp + i * kRowsLoad + sub;
        if (r < n) dst[r * kLanes] = bad ? make_uint2(0u, 0u) : codes8<Tag>(raw[i], inv);
    }
    for (int r0 = (W + w) * kRowsWarp; r0 < n; r0 += W * kRowsWarp) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int r = r0 + i * kRowsLoad + sub;
            if (r < n) dst[r * kLanes] = bad ? make_uint2(0u, 0u) : codes8<Tag>(ld_row(src + r * stride), inv);
        }
    }
    pdl_launch_dependents();
}

template <int D, int W, typename Tag>
cudaError_t launch_w(const AppendArgs &a, long long slots, int by_token, cudaStream_t s) {
    const long long tasks = slots * 2 * a.num_kv_heads;
    const long long ctas = (tasks + kWarpsCta / W - 1) / (kWarpsCta / W);
    if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
    return launch_pdl(append_int8_kernel<D, W, Tag>, dim3((unsigned)ctas), dim3(kThreads), 0, s, a, tasks, by_token);
}

template <int D, typename Tag>
cudaError_t launch_d(const AppendArgs &a, cudaStream_t s) {
    const long long by_page = (long long)a.num_new_tokens / a.block_size + 2ll * a.batch;
    const int by_token = a.num_new_tokens <= by_page ? 1 : 0;
    const long long slots = by_token ? a.num_new_tokens : by_page;
    // warps a page: enough to hold its rows in registers, where pages fill up in one call; one where a
    // page gets a row or two
    const int rows = by_token ? 1 : a.block_size, per_warp = kVecs * 256 / D;
    if (rows <= per_warp) return launch_w<D, 1, Tag>(a, slots, by_token, s);
    if (rows <= 2 * per_warp) return launch_w<D, 2, Tag>(a, slots, by_token, s);
    return launch_w<D, 4, Tag>(a, slots, by_token, s);
}

}  // namespace

cudaError_t launch_append_int8(const AppendArgs &a, cudaStream_t s) {
    if (a.num_new_tokens == 0 || a.batch == 0) return cudaSuccess;
    if (a.dtype == 1) return a.head_dim == 128 ? launch_d<128, BF16Tag>(a, s) : launch_d<64, BF16Tag>(a, s);
    return a.head_dim == 128 ? launch_d<128, F16Tag>(a, s) : launch_d<64, F16Tag>(a, s);
}

}  // namespace pkv

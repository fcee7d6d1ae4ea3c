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
// F = frac(inv_freq / 2 pi) as a 64-bit fraction (one FP64 product per frequency and warp), F * position
// modulo 2^64 is the fraction of a turn, to 2^-24 of a turn or better for every int32 position; its top 32 bits,
// as a signed number of half turns, go to sincospif.
//
// One warp per (token, chunk of its head rows). A row is held by D / 16 lanes, each with two 16-byte
// vectors that hold whole pairs: vectors j and j + rotary_dim / 16 of the half layout, 2j and 2j + 1 of
// the interleaved one and of the elements behind rotary_dim. Either way lane j's pairs are those of
// frequencies 8j .. 8j + 7, so its cosines and sines stay in registers over all rows of the token. The
// warp evaluates each frequency of its token once (a lane per frequency) and hands them out through
// shared memory. kUnroll passes of rows are loaded before any is used.
// Bound: HBM (a row is read once and written once).
#include <climits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kWarps = kRopeThreads / 32;
constexpr int kUnroll = 4;  // passes (of 512 / D rows) in flight

// plain loads, not the read-only path: q_out may be q itself
__device__ __forceinline__ uint4 ld_row(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <bool BF16>
__device__ __forceinline__ void unpack_row(const uint4 &raw, float (&f)[8]) {
    if constexpr (BF16) unpack8(raw, f, BF16Tag());
    else unpack8(raw, f, F16Tag());
}

template <bool BF16>
__device__ __forceinline__ uint4 pack_row(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &h, 4);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &h, 4);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sequence, page and in-page row of new token t (every lane the same t < cu_new_lens[batch]). False
// (error word set) for a position outside the table or a page outside the pool.
__device__ __forceinline__ bool rope_slot(const RopeArgs &a, int t, int lane, int &pb, int &off) {
    int b;
    if (a.batch <= 32) {
        // sequences 1 .. batch - 1 that start at or before t
        const int cu_j = (lane >= 1 && lane < a.batch) ? __ldg(a.cu_new_lens + lane) : INT_MAX;
        b = __popc(__ballot_sync(0xffffffffu, cu_j <= t));
    } else {
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.cu_new_lens + mid) <= t) lo = mid; else hi = mid;
        }
        b = lo;
    }
    const long long pos = (long long)__ldg(a.ctx_before + b) + (t - __ldg(a.cu_new_lens + b));
    const long long logical = pos >> a.log2_block_size;
    if (pos < 0 || logical >= a.max_blocks_per_seq) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return false;
    }
    pb = __ldg(a.block_tables + (size_t)b * a.max_blocks_per_seq + logical);
    if (pb < 0 || pb >= a.num_blocks) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return false;
    }
    off = (int)(pos & (a.block_size - 1));
    return true;
}

template <int D, bool BF16, bool FP8, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeArgs a) {
    constexpr int kLanes = D / 16;         // lanes a row
    constexpr int kRows = 32 / kLanes;     // rows a pass
    constexpr int kFreqs = D / 2;
    constexpr int kPer = (kFreqs + 31) / 32;  // frequencies a lane evaluates
    __shared__ __align__(16) float s_cos[kWarps][kFreqs], s_sin[kWarps][kFreqs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = lane % kLanes, sub = lane / kLanes;
    const int rot_lanes = a.rotary_dim / 16;
    const bool rotates = j < rot_lanes;
    const int va = (!INTER && rotates) ? j : 2 * j, vb = (!INTER && rotates) ? j + rot_lanes : 2 * j + 1;
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int kv_rows = a.num_q_heads + a.num_kv_heads;  // first V row

    pdl_wait();  // the projections come from the previous kernel, which may also still read the pages
    // F = frac(inv_freq / 2 pi) in 64 bits
    unsigned long long turn[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int f = lane + 32 * i;
        turn[i] = 0;
        if (f < a.rotary_dim / 2) {
            double x = (double)__ldg(a.inv_freq + f) * 0.15915494309189533577;
            x -= floor(x);
            turn[i] = (unsigned long long)(x * 18446744073709551616.0);
        }
    }
    const int total = min(a.num_new_tokens, __ldg(a.cu_new_lens + a.batch));  // tokens behind the last sequence: left alone
    const long long items = (long long)(total > 0 ? total : 0) * a.chunks;
    for (long long it = (long long)blockIdx.x * kWarps + warp; it < items; it += (long long)gridDim.x * kWarps) {
        const int t = (int)(it / a.chunks);
        const int c = (int)(it - (long long)t * a.chunks);
        const int r_begin = c * a.chunk_rows, r_end = min(rows, r_begin + a.chunk_rows);
        uint4 xa[kUnroll], xb[kUnroll];
        auto load = [&](int r0) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = r0 + u * kRows + sub;
                if (r >= r_end) continue;
                const uint16_t *p = r < a.num_q_heads ? static_cast<const uint16_t *>(a.q) + (size_t)t * a.q_stride + (size_t)r * D
                                    : r < kv_rows
                                        ? static_cast<const uint16_t *>(a.k) + (size_t)t * a.k_stride + (size_t)(r - a.num_q_heads) * D
                                        : static_cast<const uint16_t *>(a.v) + (size_t)t * a.v_stride + (size_t)(r - kv_rows) * D;
                xa[u] = ld_row(reinterpret_cast<const uint4 *>(p) + va);
                xb[u] = ld_row(reinterpret_cast<const uint4 *>(p) + vb);
            }
        };
        load(r_begin);
        // cosines and sines of the token, a frequency a lane
        const int pos = __ldg(a.positions + t);
        __syncwarp();  // the previous token's are read
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
        int pb = 0, off = 0;
        const bool slot_ok = r_end > a.num_q_heads && rope_slot(a, t, lane, pb, off);
        __syncwarp();
        float cs[8], sn[8];
        if (rotates) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 c4 = *reinterpret_cast<const float4 *>(&s_cos[warp][8 * j + i]);
                const float4 s4 = *reinterpret_cast<const float4 *>(&s_sin[warp][8 * j + i]);
                cs[i] = c4.x, cs[i + 1] = c4.y, cs[i + 2] = c4.z, cs[i + 3] = c4.w;
                sn[i] = s4.x, sn[i + 1] = s4.y, sn[i + 2] = s4.z, sn[i + 3] = s4.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
        }
        for (int r0 = r_begin; r0 < r_end; r0 += kUnroll * kRows) {
            if (r0 != r_begin) load(r0);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = r0 + u * kRows + sub;
                if (r0 + u * kRows >= r_end) break;  // uniform
                const bool live = r < r_end;
                const bool is_q = r < a.num_q_heads, is_v = r >= kv_rows;
                float fa[8], fb[8];
                if (live) {
                    unpack_row<BF16>(xa[u], fa);
                    unpack_row<BF16>(xb[u], fb);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) fa[i] = fb[i] = 0.f;
                }
                const void *w = is_q ? a.q_weight : a.k_weight;
                if (a.q_weight || a.k_weight) {  // uniform
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], ss));
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (w && live && !is_v) {
                        const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                        float wa[8], wb[8];
                        unpack_row<BF16>(__ldg(static_cast<const uint4 *>(w) + va), wa);
                        unpack_row<BF16>(__ldg(static_cast<const uint4 *>(w) + vb), wb);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            fa[i] = fa[i] * rs * wa[i];
                            fb[i] = fb[i] * rs * wb[i];
                        }
                    }
                }
                if (rotates && !is_v) {
                    if constexpr (INTER) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a0 = fa[2 * i], a1 = fa[2 * i + 1], b0 = fb[2 * i], b1 = fb[2 * i + 1];
                            fa[2 * i] = a0 * cs[i] - a1 * sn[i];
                            fa[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
                            fb[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
                            fb[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float a0 = fa[i], b0 = fb[i];
                            fa[i] = a0 * cs[i] - b0 * sn[i];
                            fb[i] = b0 * cs[i] + a0 * sn[i];
                        }
                    }
                }
                if constexpr (FP8) {
                    float amax = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(fa[i]), fabsf(fb[i])));
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (live && !is_q && slot_ok) {
                        const int h = is_v ? r - kv_rows : r - a.num_q_heads;
                        const size_t row = (((size_t)pb * 2 + (is_v ? 1 : 0)) * a.num_kv_heads + h) * a.block_size + off;
                        uint2 ca = make_uint2(0u, 0u), cb = ca;
                        float scale = 0.f;
                        if (amax > 0.f) {
                            scale = amax / 448.0f;
                            const float inv = 448.0f / amax;
                            ca.x = pack_e4m3x2(fa[0] * inv, fa[1] * inv) | (pack_e4m3x2(fa[2] * inv, fa[3] * inv) << 16);
                            ca.y = pack_e4m3x2(fa[4] * inv, fa[5] * inv) | (pack_e4m3x2(fa[6] * inv, fa[7] * inv) << 16);
                            cb.x = pack_e4m3x2(fb[0] * inv, fb[1] * inv) | (pack_e4m3x2(fb[2] * inv, fb[3] * inv) << 16);
                            cb.y = pack_e4m3x2(fb[4] * inv, fb[5] * inv) | (pack_e4m3x2(fb[6] * inv, fb[7] * inv) << 16);
                        }
                        uint8_t *dst = static_cast<uint8_t *>(a.cache) + row * D;
                        *reinterpret_cast<uint2 *>(dst + va * 8) = ca;
                        *reinterpret_cast<uint2 *>(dst + vb * 8) = cb;
                        if (j == 0) a.scales[row] = scale;
                    }
                }
                if (live && (is_q || (!FP8 && slot_ok))) {
                    uint16_t *dst;
                    if (is_q) {
                        dst = static_cast<uint16_t *>(a.q_out) + (size_t)t * a.q_out_stride + (size_t)r * D;
                    } else {
                        const int h = is_v ? r - kv_rows : r - a.num_q_heads;
                        dst = static_cast<uint16_t *>(a.cache) +
                              ((((size_t)pb * 2 + (is_v ? 1 : 0)) * a.num_kv_heads + h) * a.block_size + off) * D;
                    }
                    // V rows are the input's bits
                    reinterpret_cast<uint4 *>(dst)[va] = is_v ? xa[u] : pack_row<BF16>(fa);
                    reinterpret_cast<uint4 *>(dst)[vb] = is_v ? xb[u] : pack_row<BF16>(fb);
                }
            }
        }
    }
    pdl_launch_dependents();
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_rope_t(const RopeArgs &a, int grid, cudaStream_t s) {
    return a.interleaved ? launch_pdl(rope_append_kernel<D, BF16, FP8, true>, dim3(grid), dim3(kRopeThreads), 0, s, a)
                         : launch_pdl(rope_append_kernel<D, BF16, FP8, false>, dim3(grid), dim3(kRopeThreads), 0, s, a);
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs &a, int grid, cudaStream_t s) {
    if constexpr (D <= 128) {
        if (a.fp8) return a.dtype == 1 ? launch_rope_t<D, true, true>(a, grid, s) : launch_rope_t<D, false, true>(a, grid, s);
    }
    return a.dtype == 1 ? launch_rope_t<D, true, false>(a, grid, s) : launch_rope_t<D, false, false>(a, grid, s);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t s) {
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int group = kUnroll * (512 / a.head_dim);  // rows a warp has in flight
    const int sms = device_info().num_sms;
    // Rows of a token per warp: one group while the tokens leave warps to spare, whole tokens when they
    // fill the GPU by themselves (the token's cosines are then evaluated once, not once a group).
    RopeArgs r = a;
    const int most = (rows + group - 1) / group;
    const long long want = ((long long)sms * 16 + a.num_new_tokens - 1) / a.num_new_tokens;
    const int chunks = (int)(want < most ? want : most);
    r.chunk_rows = (most + chunks - 1) / chunks * group;
    r.chunks = (rows + r.chunk_rows - 1) / r.chunk_rows;
    const long long items = (long long)a.num_new_tokens * r.chunks;
    const long long ctas = (items + kWarps - 1) / kWarps, cap = (long long)sms * 16;
    const int grid = (int)(ctas < cap ? ctas : cap);
    if (a.head_dim == 256) return launch_rope_d<256>(r, grid, s);
    if (a.head_dim == 128) return launch_rope_d<128>(r, grid, s);
    return launch_rope_d<64>(r, grid, s);
}

}  // namespace pkv

// compact.cu -- kv_cache_compact: the cached rows of each sequence that are kept (the accepted path
// of a drafted tree, the tokens a window or an eviction rule leaves) move to consecutive positions,
// in place, every KV head's K and V.
//
// Row k of sequence b goes from position keep_pos[cu_keep[b] + k] to dst_start[b] + k, both read
// through the block table ("企业官网建设流程全解析", section 2.1: block i / block_size, offset
// i % block_size). Every source lies at or behind its destination (src >= dst, checked per row). That
// alone makes the move safe in ascending order: the destination of row k is the source of a row j only
// if src_j = dst_k >= dst_j, so j <= k -- a row written is never one that a later row still reads.
//
// Pure bandwidth: each moved row is read once and written once. A slice is one (sequence, K or V,
// head) and a column part of its rows; slices touch disjoint bytes, so they run as independent CTAs.
// Inside a slice the CTA moves chunks of kUnroll x (256 / VP) rows in order: the loads of chunk c + 1
// are issued before the stores of chunk c, with one barrier between a chunk's loads and its stores
// (a store of chunk c can only meet a source of chunk c or earlier, whose loads precede the barrier).
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kCompactThreads = 256;
constexpr int kUnroll = 4;

// The rows of one chunk held by a thread: a 16-byte vector and, from the first thread of a row's
// part 0 over an FP8 cache, the row's scale; dst < 0: nothing to store.
struct Chunk {
    uint4 v[kUnroll];
    float sc[kUnroll];
    long long dst[kUnroll];
};

__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// VP: 16-byte vectors of a row that the CTA moves (a power of two; the row's vectors / VP parts).
template <int VP>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(CompactArgs a) {
    constexpr int kRows = kCompactThreads / VP;
    const int e = threadIdx.x % VP, tr = threadIdx.x / VP;
    uint4 *cache = static_cast<uint4 *>(a.cache);
    const int row_vecs = VP * a.parts;
    const long long cap = (long long)a.max_blocks_per_seq << a.log2_block_size;

    pdl_wait();  // the previous kernel may still read or write the pages
    for (long long s = blockIdx.x; s < a.slices; s += gridDim.x) {
        const int part = (int)(s % a.parts);
        long long rest = s / a.parts;
        const int h = (int)(rest % a.num_kv_heads);
        rest /= a.num_kv_heads;
        const int kv = (int)(rest & 1);
        const int b = (int)(rest >> 1);
        const int r0 = __ldg(a.cu_keep + b), r1 = __ldg(a.cu_keep + b + 1);
        const int start = __ldg(a.dst_start + b);
        if (r0 < 0 || r1 < r0 || r1 > a.num_keep || start < 0) {
            if (threadIdx.x == 0) set_error(a.err, kErrDeviceRange);
            continue;
        }
        const int n = r1 - r0;
        const int *bt = a.block_tables + (size_t)b * a.max_blocks_per_seq;
        const bool first_lane = e == 0 && part == 0;  // carries the row's scale

        // row index of position pos in this slice's (K or V, head), or -1 (flagged)
        auto row_of = [&](long long pos) -> long long {
            const int pb = __ldg(bt + (pos >> a.log2_block_size));
            if (pb < 0 || pb >= a.num_blocks) {
                set_error(a.err, kErrDeviceRange);
                return -1;
            }
            return (((long long)pb * 2 + kv) * a.num_kv_heads + h) * a.block_size + (pos & (a.block_size - 1));
        };
        auto load = [&](int base, Chunk &c) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int k = base + u * kRows + tr;
                c.dst[u] = -1;
                if (k >= n) continue;
                const long long src = __ldg(a.keep_pos + r0 + k), dst = (long long)start + k;
                if (src == dst && src < cap) continue;
                if (src < dst || src >= cap) {
                    set_error(a.err, kErrDeviceRange);
                    continue;
                }
                const long long rs = row_of(src), rd = row_of(dst);
                if (rs < 0 || rd < 0) continue;
                c.dst[u] = rd;
                c.v[u] = ld_once(cache + rs * row_vecs + part * VP + e);
                if (a.scales && first_lane) c.sc[u] = __ldcg(a.scales + rs);
            }
        };
        auto store = [&](const Chunk &c) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (c.dst[u] < 0) continue;
                cache[c.dst[u] * row_vecs + part * VP + e] = c.v[u];
                if (a.scales && first_lane) a.scales[c.dst[u]] = c.sc[u];
            }
        };
        Chunk cur, nxt;
        load(0, cur);
        for (int base = 0; base < n; base += kUnroll * kRows) {
            load(base + kUnroll * kRows, nxt);
            __syncthreads();  // every load of this chunk (and of the next) precedes this chunk's stores
            store(cur);
            cur = nxt;
        }
        __syncthreads();  // slices of one CTA may share nothing, but its next loads follow these stores
    }
    pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t s) {
    const int row_vecs = a.head_dim * (a.scales ? 1 : 2) / 16;  // 4 .. 32
    // Column parts of 64 bytes or more until there are two CTAs an SM (a single sequence has only
    // 2 Hkv rows of slices); whole rows otherwise.
    CompactArgs c = a;
    const long long rows = (long long)a.batch * 2 * a.num_kv_heads;
    int vp = row_vecs;
    while (vp > 4 && rows * (row_vecs / vp) < 2ll * device_info().num_sms) vp /= 2;
    c.parts = row_vecs / vp;
    c.slices = rows * c.parts;
    const long long cap = 32ll * device_info().num_sms;
    const dim3 grid((unsigned)(c.slices < cap ? c.slices : cap)), block(kCompactThreads);
    switch (vp) {
        case 4: return launch_pdl(compact_kernel<4>, grid, block, 0, s, c);
        case 8: return launch_pdl(compact_kernel<8>, grid, block, 0, s, c);
        case 16: return launch_pdl(compact_kernel<16>, grid, block, 0, s, c);
        default: return launch_pdl(compact_kernel<32>, grid, block, 0, s, c);
    }
}

}  // namespace pkv

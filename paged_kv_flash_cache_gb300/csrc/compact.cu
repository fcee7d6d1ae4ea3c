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
// head); slices touch disjoint rows. A group of threads moves a slice's rows chunk by chunk, kUnroll 16-byte
// vectors a thread: the rows' places are looked up a chunk ahead, a thread a row, into shared memory, so that the
// moves themselves wait for one read only; a barrier stands between a chunk's loads and its stores (a
// store of chunk c can only meet a source of chunk c or earlier, whose loads precede the barrier).
// The batch's average number of rows chooses (counts on the device do not reach the launch), so a batch in which one list is much
// longer than the others takes as long as that list does with what the average gives it:
//   few rows   a warp a slice;
//   more       `shares` CTAs a slice, each moving an equal piece of its rows. Pieces are independent
//              when no row's source lies in a later piece's destinations (a window moved up behind a prompt);
//              every CTA of the slice looks the list over and finds the same answer. Otherwise the rows go in order
//              and the CTAs take a share of each row's columns instead, as far as 64 bytes a share.
// 8 x 8192 rows of 8 heads x 128 (537 MB read and written): 242 us with column shares only (64 bytes of a row at
// different times), 147 us with pieces and each vector's thread looking its row up, 97 us (82% of the copy rate) as it is.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kCompactThreads = 256;
constexpr int kUnroll = 8;
constexpr int kResident = 3;  // CTAs an SM (registers)
// Rows of the pool are counted in 32 bits (the entry point refuses a pool of more).
constexpr uint32_t kNoRow = 0xffffffffu;  // nothing to move

__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// kGroup threads (a warp, or the CTA) a slice.
template <int kGroup>
__global__ void __launch_bounds__(kCompactThreads, kResident) compact_kernel(CompactArgs a) {
    constexpr int kGroups = kCompactThreads / kGroup;
    // a chunk's source and destination rows, three chunks in turn: kUnroll * kGroup vectors are at most 2 * kGroup rows
    __shared__ uint32_t s_src[3][2 * kCompactThreads], s_dst[3][2 * kCompactThreads];
    const int tid = threadIdx.x % kGroup, s0 = threadIdx.x / kGroup * 2 * kGroup;
    uint4 *cache = static_cast<uint4 *>(a.cache);
    const long long cap = (long long)a.max_blocks_per_seq << a.log2_block_size;
    auto sync = [] {
        if constexpr (kGroup == 32) __syncwarp();
        else __syncthreads();
    };

    pdl_wait();  // the previous kernel may still read or write the pages
    const long long total = a.slices * a.shares;
    for (long long s = (long long)blockIdx.x * kGroups + threadIdx.x / kGroup; s < total; s += (long long)gridDim.x * kGroups) {
        // heads first: the CTAs that run together move the same tokens' rows, which are neighbours in their pages
        const int h = (int)(s % a.num_kv_heads);
        long long rest = s / a.num_kv_heads;
        const int kv = (int)(rest & 1);
        rest >>= 1;
        const int share = (int)(rest % a.shares), b = (int)(rest / a.shares);
        const int r0 = __ldg(a.cu_keep + b), r1 = __ldg(a.cu_keep + b + 1);
        const int start = __ldg(a.dst_start + b);
        if (r0 < 0 || r1 < r0 || r1 > a.num_keep || start < 0) {
            if (tid == 0) set_error(a.err, kErrDeviceRange);
            continue;
        }
        const int n = r1 - r0;
        const int *keep = a.keep_pos + r0;
        const int *bt = a.block_tables + (size_t)b * a.max_blocks_per_seq;

        // this group's rows [k0, k_end), 2^log2_v vectors of each from vector col on
        int k0 = 0, k_end = n, log2_v = a.log2_row_vecs, col = 0;
        if constexpr (kGroup > 32) {
            if (a.shares > 1) {
                const int piece = (n + a.shares - 1) / a.shares;
                // does a row read what a later piece writes?
                bool meets = false;
                int piece_end = piece;  // of k's piece
                for (int k8 = tid; k8 < n; k8 += 8 * kGroup) {
                    int src[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) src[u] = k8 + u * kGroup < n ? __ldg(keep + k8 + u * kGroup) : start;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const long long at = (long long)src[u] - start;  // the row that goes to the source of k
                        while (k8 + u * kGroup >= piece_end) piece_end += piece;
                        meets |= at >= piece_end && at < n;
                    }
                }
                if (!__syncthreads_or(meets)) {
                    k0 = share * piece;
                    k_end = min(n, k0 + piece);
                } else {
                    if (share >= 1 << a.log2_col_shares) continue;
                    log2_v -= a.log2_col_shares;
                    col = share << log2_v;
                }
            }
        }
        // rows of a chunk (with fewer columns: fewer vectors a thread)
        const int rows = (kUnroll * kGroup) >> a.log2_row_vecs;
        // row index of position pos in this slice's (K or V, head), or kNoRow (flagged)
        auto row_of = [&](long long pos) -> uint32_t {
            const int pb = __ldg(bt + (pos >> a.log2_block_size));
            if (pb < 0 || pb >= a.num_blocks) {
                set_error(a.err, kErrDeviceRange);
                return kNoRow;
            }
            return (((uint32_t)pb * 2 + kv) * a.num_kv_heads + h) * a.block_size + (uint32_t)(pos & (a.block_size - 1));
        };
        auto look_up = [&](int buf, int base) {
#pragma unroll
            for (int r = tid; r < rows; r += kGroup) {
                uint32_t rs = kNoRow, rd = kNoRow;
                const int k = base + r;
                if (k < k_end) {
                    const long long src = __ldg(keep + k), dst = (long long)start + k;
                    if (src < dst || src >= cap) {
                        set_error(a.err, kErrDeviceRange);
                    } else if (src != dst) {
                        rs = row_of(src);
                        rd = row_of(dst);
                        if (rs == kNoRow) rd = kNoRow;
                    }
                }
                s_src[buf][s0 + r] = rs;
                s_dst[buf][s0 + r] = rd;
            }
        };
        // vector u of this thread: row ra + u * rb of the chunk (the same vector of each)
        const int ra = tid >> log2_v, rb = kGroup >> log2_v;
        uint4 *const base_v = cache + col + (tid & ((1 << log2_v) - 1));
        const bool scales = a.scales && col == 0;
        int buf = 0;
        look_up(0, k0);
        sync();
        for (int base = k0; base < k_end; base += rows) {
            uint4 v[kUnroll];
            float sc[2];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = ra + u * rb;
                if (r < rows && s_dst[buf][s0 + r] != kNoRow)
                    v[u] = ld_once(base_v + ((size_t)s_src[buf][s0 + r] << a.log2_row_vecs));
            }
            if (scales)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = tid + u * kGroup;
                    if (r < rows && s_dst[buf][s0 + r] != kNoRow) sc[u] = __ldcg(a.scales + s_src[buf][s0 + r]);
                }
            const int next = buf == 2 ? 0 : buf + 1;
            if (base + rows < k_end) look_up(next, base + rows);
            sync();  // every load of this chunk precedes its stores
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = ra + u * rb;
                if (r < rows && s_dst[buf][s0 + r] != kNoRow) base_v[(size_t)s_dst[buf][s0 + r] << a.log2_row_vecs] = v[u];
            }
            if (scales)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = tid + u * kGroup;
                    if (r < rows && s_dst[buf][s0 + r] != kNoRow) a.scales[s_dst[buf][s0 + r]] = sc[u];
                }
            buf = next;
        }
        sync();  // the next slice's look-ups overwrite these
    }
    pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t s) {
    CompactArgs c = a;
    const int row_vecs = a.head_dim * (a.scales ? 1 : 2) / 16;  // 4, 8, 16 or 32
    c.log2_row_vecs = row_vecs == 4 ? 2 : row_vecs == 8 ? 3 : row_vecs == 16 ? 4 : 5;
    c.slices = (long long)a.batch * 2 * a.num_kv_heads;
    c.shares = 1;
    c.log2_col_shares = 0;
    const int sms = device_info().num_sms;
    // the rows of a sequence on average: what a warp moves in one chunk is a warp's (accepted paths)
    if ((long long)a.num_keep * row_vecs <= (long long)a.batch * 32 * kUnroll) {
        const long long ctas = (c.slices + kCompactThreads / 32 - 1) / (kCompactThreads / 32), cap = 32ll * sms;
        return launch_pdl(compact_kernel<32>, dim3((unsigned)(ctas < cap ? ctas : cap)), dim3(kCompactThreads), 0, s, c);
    }
    // CTAs a slice: four rounds of the SMs' (8 x 8192 rows of 8 heads: 97 us; two rounds 112, eight 105), and for each
    // two chunks of an average sequence's rows at least
    const long long round = (long long)kResident * sms, chunk = kUnroll * kCompactThreads / row_vecs;
    const long long avg = (a.num_keep + a.batch - 1) / a.batch;
    long long shares = 4 * round / c.slices;
    if (shares > avg / (2 * chunk)) shares = avg / (2 * chunk);
    c.shares = shares < 1 ? 1 : shares > 64 ? 64 : (int)shares;
    while ((2 << c.log2_col_shares) <= c.shares && c.log2_row_vecs - c.log2_col_shares > 2) ++c.log2_col_shares;
    const long long ctas = c.slices * c.shares, cap = 32ll * sms;
    return launch_pdl(compact_kernel<kCompactThreads>, dim3((unsigned)(ctas < cap ? ctas : cap)), dim3(kCompactThreads), 0, s, c);
}

}  // namespace pkv

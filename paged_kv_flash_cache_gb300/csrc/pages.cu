// pages.cu -- kv_cache_copy and kv_cache_fork: pages, or their first rows, moved bit for bit.
//
// A page that several block tables share can be written by none of them; a sequence that continues another one gets
// its own copy of the half-filled last page and shares the full ones. Pages of a pool [num_blocks, 2, Hkv, bs, D] are
// contiguous; the first rows of a page are 2 * Hkv runs. Pure bandwidth: a byte read and a byte written.
//
// A warp moves up to 4 KB of one run, all its loads in flight before the first store; whole pages are one run of all
// their bytes. Runs and their shares are numbered by the host's bounds alone (row counts live on the device); a
// warp whose share begins behind its run's end has nothing to do. 2048 pages of 64 KB (268 MB moved): 41.2 us, 96% of the copy
// rate; the first rows of 64 pages 2.2 us, forks of 1 to 4 and 64 to 64 sequences 2.0 and 3.3 us: a launch and two round trips.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;
constexpr int kShare = kVecs * 32;  // 16-byte vectors a warp moves
constexpr int kTableShare = 1024;   // entries of a block table a CTA of a fork writes

__device__ __forceinline__ void move_share(const uint4 *src, uint4 *dst, long long first, long long end, int lane) {
    uint4 x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const long long v = first + i * 32 + lane;
        if (v < end) x[i] = __ldg(src + v);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const long long v = first + i * 32 + lane;
        if (v < end) dst[v] = x[i];
    }
}

// The share `share` of run `run` of a page: rows < rows of it (whole: the page as one run, whatever rows is).
__device__ __forceinline__ void move_run(const PagesArgs &a, long long sp, long long dp, int rows, int run, int share,
                                         int lane) {
    const uint4 *src = static_cast<const uint4 *>(a.src) + sp * a.page_vecs;
    uint4 *dst = static_cast<uint4 *>(a.dst) + dp * a.page_vecs;
    const long long first = (long long)share * kShare;
    if (a.whole) {
        move_share(src, dst, first, a.page_vecs, lane);
    } else {
        const size_t at = (size_t)run * a.block_size * a.row_vecs;
        move_share(src + at, dst + at, first, (long long)rows * a.row_vecs, lane);
    }
    if (!a.scales_per_page) return;
    // scales: of the page (whole) or of the run's rows, shared out like the vectors
    const float *ss = a.src_scales + sp * a.scales_per_page;
    float *ds = a.dst_scales + dp * a.scales_per_page;
    const int per_run = a.scales_per_page / a.slices;  // 1 (a page of a head) or block_size (its rows)
    int lo, hi;
    if (a.whole) {
        const int part = (a.scales_per_page + a.shares - 1) / a.shares;
        lo = share * part;
        hi = min(lo + part, a.scales_per_page);
    } else {
        if (share != 0) return;
        lo = run * per_run;
        hi = lo + (per_run == 1 ? (rows > 0 ? 1 : 0) : rows);
    }
    for (int i = lo + lane; i < hi; i += 32) ds[i] = __ldg(ss + i);
}

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(PagesArgs a) {
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    const long long per_page = (long long)(a.whole ? 1 : a.slices) * a.shares;
    const long long i = u / per_page;
    if (i >= a.num_pages) return;
    const int j = (int)(u - i * per_page);
    const int run = j / a.shares, share = j - run * a.shares;
    const int sp = __ldg(a.src_pages + i), dp = __ldg(a.dst_pages + i);
    const int rows = a.num_rows ? __ldg(a.num_rows + i) : a.block_size;
    if (sp < 0 || sp >= a.src_blocks || dp < 0 || dp >= a.dst_blocks || rows < 0 || rows > a.block_size) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return;
    }
    move_run(a, sp, dp, rows, run, share, lane);
    pdl_launch_dependents();
}

// CTAs [0, table_ctas): block tables and lengths of the children; the others: the rows of their last pages.
__global__ void __launch_bounds__(kThreads) fork_kernel(PagesArgs a, ForkArgs f) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int mb = f.max_blocks_per_seq;
    const long long cap = (long long)mb * a.block_size;
    if ((long long)blockIdx.x < f.table_ctas) {
        const int c = blockIdx.x / f.table_parts, part = blockIdx.x - c * f.table_parts;
        const int p = __ldg(f.parents + c), fresh = __ldg(f.new_pages + c);
        int len = p >= 0 && p < f.num_parents ? __ldg(f.context_lens + p) : -1;
        const bool ok = len >= 0 && len <= cap;
        if (!ok) len = 0;
        const int full = len >> a.log2_block_size, rest = len & (a.block_size - 1);
        const bool fits = fresh < a.dst_blocks;
        if (part == 0 && threadIdx.x == 0) {
            f.out_lens[c] = len;
            if (!ok || !fits) set_error(a.err, kErrDeviceRange);
        }
        const int *row = f.block_tables + (size_t)(ok ? p : 0) * mb;
        for (int i = part * kTableShare + threadIdx.x; i < min(mb, (part + 1) * kTableShare); i += kThreads) {
            int page = -1;
            if (ok) {
                if (i < full || (i == full && rest > 0 && fresh < 0)) page = __ldg(row + i);
                else if (i == full && fresh >= 0 && fits) page = fresh;
            }
            f.out_tables[(size_t)c * mb + i] = page;
        }
        return;
    }
    const long long u = (long long)(blockIdx.x - f.table_ctas) * (kThreads / 32) + (threadIdx.x >> 5);
    const long long per_child = (long long)a.slices * a.shares;
    const long long c = u / per_child;
    if (c >= f.num_children) return;
    const int j = (int)(u - c * per_child);
    const int run = j / a.shares, share = j - run * a.shares;
    const int p = __ldg(f.parents + c), fresh = __ldg(f.new_pages + c);
    if (p < 0 || p >= f.num_parents || fresh < 0 || fresh >= a.dst_blocks) return;  // (flagged above, or no copy asked for)
    const int len = __ldg(f.context_lens + p);
    if (len <= 0 || len > cap) return;
    const int rest = len & (a.block_size - 1);
    if (rest == 0) return;
    const int last = __ldg(f.block_tables + (size_t)p * mb + (len >> a.log2_block_size));
    if (last < 0 || last >= a.dst_blocks) {
        if (lane == 0) set_error(a.err, kErrDeviceRange);
        return;
    }
    move_run(a, last, fresh, rest, run, share, lane);
    pdl_launch_dependents();
}

int shares_of(long long vecs) { return (int)((vecs + kShare - 1) / kShare); }

}  // namespace

cudaError_t launch_copy_pages(PagesArgs a, cudaStream_t s) {
    a.whole = a.num_rows ? 0 : 1;
    a.shares = shares_of(a.whole ? a.page_vecs : (long long)a.block_size * a.row_vecs);
    const long long warps = (long long)a.num_pages * (a.whole ? 1 : a.slices) * a.shares;
    const long long ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
    return launch_pdl(copy_pages_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, s, a);
}

cudaError_t launch_fork(PagesArgs a, ForkArgs f, cudaStream_t s) {
    a.whole = 0;
    a.shares = shares_of((long long)a.block_size * a.row_vecs);
    f.table_parts = (f.max_blocks_per_seq + kTableShare - 1) / kTableShare;
    const long long tables = (long long)f.num_children * f.table_parts;
    const long long warps = (long long)f.num_children * a.slices * a.shares;
    const long long ctas = tables + (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
    f.table_ctas = (int)tables;
    return launch_pdl(fork_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, s, a, f);
}

}  // namespace pkv

// decode_rules.h -- how a decode is cut: tokens per split for every cache format, and over an INT8 cache the query heads of
// a unit, clusters or splits. Functions of the sizes and of the device's SMs alone, so that calls, workspace sizes and tests
// without a GPU use the same ones.
#pragma once

namespace pkv {

constexpr int kSplitAlign = 128;         // decode splits start at multiples of this many tokens
constexpr int kDecodeMaxSplits = 2048;   // splits of one context (bounds the split size from below)
constexpr int kDecodeMaxBatch = 2048;    // sequences of one launch
constexpr int kInt8CtasPerSm = 3;        // decode_int8.cu: resident CTAs an SM
constexpr int kInt8ClusterCtasPerSm = 2; // and, in clusters, at most

// Tokens per decode split.  Automatic: enough (sequence, KV head, split) units for about
// eight per SM at full capacity, in [128, 768] tokens; explicit: capacity / num_splits
// rounded up to kSplitAlign (128, the tensor-core decode's key tile).  Either way at least
// capacity / kDecodeMaxSplits, rounded up, so that a full context has at most kDecodeMaxSplits
// splits.
inline int decode_split_tokens(int num_sms, int batch, int num_kv_heads, int block_size, int max_blocks_per_seq,
                               int num_splits) {
    const long long cap = (long long)max_blocks_per_seq * block_size;
    const long long tile = kSplitAlign;
    long long c;
    if (num_splits > 0) {
        c = (cap + num_splits - 1) / num_splits;
    } else {
        const long long want = (long long)batch * num_kv_heads * cap / (num_sms * 8ll);
        // the largest of these at or below want (at least 128): 768-token splits measured best on
        // the streaming paths (7B-like, FP8 and mixed batches against 512, 640 and 1024)
        constexpr int kSizes[] = {768, 512, 384, 256, 128};
        int i = 0;
        while (kSizes[i] > 128 && kSizes[i] > want) ++i;
        c = kSizes[i];
    }
    const long long floor_c = (cap + kDecodeMaxSplits - 1) / kDecodeMaxSplits;
    if (c < floor_c) c = floor_c;
    c = (c + tile - 1) / tile * tile;
    return (int)(c < tile ? tile : c);
}

// ---- an INT8 cache ----

// CTAs of the cluster that takes a unit's whole context, 0: the split kernel and its merge. A cluster saves the unit tables,
// the partials and the second launch, but has to leave SMs idle where the units times 16 are fewer. Measured against the
// splits, 8 KV heads of 4 query heads: one sequence of 4096 tokens 7.8 us for 9.6, of 8192 10.5 for 11.5, of 16384
// (not taken) 15.5 for 14.1; four of 4096 10.2 for 12.2, of 16384 26.1 for 29.2; 32 of 2048 25.5 for 28.4; 16 of 8192 47.6
// for 47.2 (not taken: more units than CTAs at two an SM in clusters of one). Clusters of 16 only where they are alone on
// their SMs: 16 units of 8192 tokens in 256 CTAs took 20.4 for 17.0. The lengths live on the device: capacity is the table's.
// sizes: the cluster sizes that the device can place, ored (a cluster lies in one GPC, and sizes above 8 are no device's duty).
inline int decode_int8_cluster(int num_sms, int sizes, int batch, int units_per_seq, long long capacity) {
    const long long units = (long long)batch * units_per_seq;
    for (int c = 16; c >= 1; c >>= 1)
        if ((sizes & c) && units * c <= (long long)(c == 16 ? 1 : kInt8ClusterCtasPerSm) * num_sms)
            return capacity <= (units * c <= num_sms ? 640ll : 4096ll) * c ? c : 0;
    return 0;
}

// Tokens per split (a multiple of 128, 256 to 1024, and at most kDecodeMaxSplits splits): units are dealt round-robin
// to the CTAs, so a launch takes about ceil(units / CTAs) times a unit's tokens and what a unit costs besides (150 tokens'
// time), for contexts that fill the table but its last page. (4 sequences of 8192 tokens, 8 KV heads: 26 us with splits of
// 128 tokens, 16 with 640.) With work for more rounds than four the contexts' own lengths matter more: 768 tokens, the best
// for ragged batches (mixed serving batch 37 us; 384 tokens 40, 1024 43).
inline int decode_int8_split(int num_sms, int batch, int units_per_seq, int block_size, long long capacity) {
    const long long ctas = (long long)kInt8CtasPerSm * num_sms;
    const long long tokens = capacity > block_size ? capacity - block_size : capacity;
    long long least = (capacity + kDecodeMaxSplits - 1) / kDecodeMaxSplits;
    least = (least + 127) / 128 * 128;
    if (least < 256) least = 256;
    if (least <= 768 && (long long)batch * units_per_seq * ((tokens + 767) / 768) >= 4 * ctas) return 768;
    long long best = least, best_cost = -1;
    for (long long c = least; c <= (least > 1024 ? least : 1024); c += 128) {
        const long long units = (long long)batch * units_per_seq * ((tokens + c - 1) / c);
        const long long cost = (units + ctas - 1) / ctas * (c + 150);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return (int)best;
}

// The same for tcgen05 units: a CTA an SM, so a launch takes about ceil(units / SMs) times a unit's tokens and what a CTA's
// start and end cost (600 tokens' time), for contexts that fill the table but its last page; 768 tokens at least.
inline int decode_int8_wide_split(int num_sms, int batch, int units_per_seq, int block_size, long long capacity) {
    const long long ctas = num_sms;
    const long long tokens = capacity > block_size ? capacity - block_size : capacity;
    long long least = (capacity + kDecodeMaxSplits - 1) / kDecodeMaxSplits;
    least = (least + 255) / 256 * 256;
    if (least < 768) least = 768;
    long long best = least, best_cost = -1;
    for (long long c = least; c <= (least > 8192 ? least : 8192); c += 256) {
        const long long units = (long long)batch * units_per_seq * ((tokens + c - 1) / c);
        const long long cost = (units + ctas - 1) / ctas * (c + 600);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return (int)best;
}

inline int largest_divisor(int group, int most) {
    int n = group;
    for (int d = most; n > most; --d)
        if (group % d == 0) n = d;
    return n;
}

// How a decode over an INT8 cache runs: query heads of a unit, the cluster's CTAs (0: splits and a merge), tokens per split,
// and whether the units are tcgen05's.
//   few units and short tables: clusters (decode_int8_cluster), units of the group or, above 8 heads, of its largest
//   divisor up to 8; more than 8 heads per KV head otherwise: tcgen05 units of the group or its largest divisor up to 128;
//   else splits of mma.sync units.
// Never more splits than decode_split_tokens makes: a workspace sized for the other formats serves this one too. (Their
// splits are the larger ones for about 1 in 200 sizes: 3 sequences of 9728 tokens, 32 heads, 768 tokens for 512.)
struct Int8Decode {
    int unit_heads, cluster, chunk;
    bool wide;
};

inline Int8Decode decode_int8_plan(int num_sms, int batch, int num_q_heads, int num_kv_heads, int block_size,
                                   int max_blocks_per_seq, int num_splits, int cluster_sizes = 31) {
    const long long cap = (long long)max_blocks_per_seq * block_size;
    const int group = num_q_heads / num_kv_heads;
    Int8Decode d;
    d.unit_heads = largest_divisor(group, 8);
    d.cluster = num_splits > 0 || batch > kDecodeMaxBatch
                    ? 0
                    : decode_int8_cluster(num_sms, cluster_sizes, batch, num_q_heads / d.unit_heads, cap);
    d.wide = d.cluster == 0 && group > 8;
    if (d.wide) d.unit_heads = largest_divisor(group, 128);
    const int units = num_q_heads / d.unit_heads;
    const int most = decode_split_tokens(num_sms, batch, num_kv_heads, block_size, max_blocks_per_seq, num_splits);
    d.chunk = num_splits > 0 ? most
              : d.wide       ? decode_int8_wide_split(num_sms, batch, units, block_size, cap)
                             : decode_int8_split(num_sms, batch, units, block_size, cap);
    if ((cap + d.chunk - 1) / d.chunk > (cap + most - 1) / most) d.chunk = most;
    return d;
}

}  // namespace pkv

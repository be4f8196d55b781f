// tri_chunk.cuh -- attention of a chunk of new tokens over the cache, for sm_100a.
//
// Sequence s brings n tokens (their rows already in the cache as its last n of len). For query head
// h of new token i, with the KV head g = h / G of its group,
//   out = sum_j softmax_j(scale q . k_j) v_j,  j < len - n + i + 1 (causal) or j < len,
//   lse = log sum_j exp(scale q . k_j),
// zeros and -inf where no key is left. The running maximum m and sum l of a row turn this into one
// pass over the keys: with p_j = 2^((x_j - m) c), c = scale log2(e), out = sum p_j v_j / sum p_j.
//
// Three launches. The plan kernel (one CTA, or one per sequence for many sequences or long block tables) checks
// the sequences (range of tokens, length, pages) and lists the work, so that nothing waits on the host. An
// item is a block of kChunkRows rows of a KV head's packed query matrix (row = token * G + head in group, so
// that all G query heads of a key share its one read), over a range of 128-key tiles. Where there are too few
// items to fill the SMs evenly, items are split over the keys, and the merge kernel joins their parts in the
// order of the keys, so that the result does not depend on which part finished first. Items are handed out
// longest first, in rounds that run forth and back over the CTAs.
//
// The attention kernel, one persistent CTA per SM: warp 0 loads (TMA, 128-byte swizzle: the item's
// query rows, then K and V tiles through a ring), and two warpgroups take one 128-row query tile each,
// a row per thread, with a warp each (1 and 2) that issues its tcgen05 MMAs:
//   S_q = Q_q K^T            128 x 128 x D into TMEM columns [128 q, 128 q + 128)
//   P_q = 2^((S_q - m) c)    read, masked, exponentiated, rounded to bf16 and written to TMEM
//   O_q += P_q V             A from TMEM, V as the N-major operand: the tile lies as it came
// An item of at most 128 rows (single and drafted tokens) gives its one query tile to both warpgroups, which take
// its key tiles in turn and join their (m, l, O) at the end: twice the keys in flight.
// Head 128: S_0, S_1, O_0 and O_1 fill the tensor memory, so P_q lies over S_q, and an MMA warp runs O_q += P_q V(i) and
// S_q = Q_q K(i+1)^T back to back; one warpgroup's exponentials overlap the other's MMAs. S_q(i+1) complete implies P_q
// V(i) complete, so O_q is the warpgroup's own until it hands over P_q(i+1): it rescales O_q itself, and only where
// the maximum has grown by more than 2^8 since the last rescale (p then stays below 2^8; the quotient is the same).
// Head 64: P has columns of its own, and S_q(i+1) is computed as soon as S_q(i) has been read.
//
// Precision: logits, m, l and O are fp32. P is rounded to bf16 (the MMA's A has V's type): each
// weight moves by at most 2^-8 relative, independent from key to key, which adds about as much to the
// result as its own final rounding to bf16: against 64 bits the error is 1.4 times that of the final rounding alone. l sums
// the unrounded weights. Weights in two bf16 parts would double the MMAs of P V.
//
// Bound, measured on a B200 with everything but one part of the kernel taken out (512 tokens of 64 heads over 32768
// rows of 128 dims: 128 items of 256 tiles on 148 SMs; 510 to 514 us): the loads alone 343 us, the MMAs with their barriers 426 us,
// the rest is the chain of a tile from S through the exponentials (1100 clocks) to P V and the next S, whose barriers cost
// about 300 clocks each way. 64-key steps with two S buffers take that chain apart, but an MMA of 64 keys takes
// as long as one of 128, and the MMAs alone then took 3100 of 3900 clocks a tile: the same time. Few rows: the HBM (16 single
// tokens over 2176 rows stream at 7 TB/s for 19 of 38 us; the rest is the plan, the first tiles' latency and the end).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tri_kernel.cuh"
#include "tri_maxdelta.cuh"
#include "tri_rope.cuh"

namespace tri {

constexpr int kChunkRows = 256;     // packed query rows of an item: two MMA tiles
constexpr int kChunkThreads = 384;  // a warpgroup with the load and the MMA warps, two for the softmax
// Registers a thread after the split: 128 * 72 + 256 * 216 = 64512, the 384 * 168 that the
// block is launched with. A softmax thread holds a row of 128 logits.
constexpr int kChunkRegsFew = 72, kChunkRegsMany = 216;
constexpr int kChunkPlanThreads = 256;
// Ring stages: as many as fit beside the query tiles, which also keeps it to one CTA per SM (each allocates
// the whole tensor memory).
__host__ __device__ constexpr int chunk_stages(int D) { return D == 128 ? 5 : 8; }

// One line of the plan: a block of rows of one sequence over the key tiles [kt0, kt1), for every
// layer and KV head.
struct __align__(16) ChunkEntry {
    int s, tok0, ntok, len;   // sequence, first token (global row), tokens of the block, cached rows
    int first, kt0, kt1;      // keys seen by the block's first row, key tiles
    int pair;                 // one row tile whose key tiles the two warpgroups take in turn
    int nsplit, split, slot;  // splits of the block; this one; its first partial
};

struct __align__(16) ChunkSeq {
    int q0, n, len, bad;
};

struct ChunkHead {
    int n_entries;            // lines of the plan
    int n_groups;             // blocks that are split
};

struct ChunkArgs {
    const int32_t *cu;        // [batch + 1]
    const int32_t *lens;
    const int32_t *block_table;
    int n_tokens, batch, n_kv, n_layers, group;
    int paged, page_size, max_pages, n_pages, cap_u;
    int causal;
    int piece_rows;           // rows of a key box
    int sm_count, max_slots, max_entries;
    float c;                  // scale * log2(e)
    // where the query rows and results are (strides in elements)
    const uint16_t *q;
    long long q_l, q_t, q_h;
    uint16_t *out;
    long long o_l, o_t, o_h;
    float *lse;               // [n_layers][n_tokens][Hq] or null
    const uint16_t *K, *V;
    // workspace
    ChunkHead *head;
    ChunkSeq *seqs;           // [batch]
    int *base;                // [batch + 1] blocks before each sequence
    int *tiles;               // [max blocks] key tiles of each block
    ChunkEntry *entries;
    float *part;              // [slot][tile][D / 4][128][4], then [slot][tile][128][2] (m, l)
    float *part_ml;
    ChunkEntry *merges;       // the blocks that are split
    // the context's status word, and behind it the count of the plan's CTAs that are done, back to 0 at the end. (A pointer of
    // its own, 8 bytes more of arguments, cost 1.3 us of host time in every call.)
    unsigned long long *status;
    int wait_tries;
    long long inject_unit;
};

__host__ __device__ inline int chunk_blocks(int n, int G) { return (n + kChunkRows / G - 1) / (kChunkRows / G); }

// ---------------------------------------------------------------------------------
// The plan.
// ---------------------------------------------------------------------------------
// Costs in units of one key tile of an item: what a further item costs its CTA (filling and draining
// the pipeline, the result), and what the merge of a split adds at the end.
constexpr int kChunkItemCost = 3;
constexpr int kChunkMergeCost = 3, kChunkMergeRows = 2;  // a merge: the first, and the second for a full block
constexpr int kChunkPlanSeqs = 512, kChunkPlanBlocks = 2048;  // what the plan keeps in shared memory, at most
constexpr int kChunkSortBins = 1024;
constexpr int kChunkCandidates = 16;
constexpr int kChunkPlanAlone = 8192;  // block table entries that one CTA checks by itself

__global__ void __launch_bounds__(kChunkPlanThreads) tri_chunk_plan_kernel(const ChunkArgs a) {
    constexpr unsigned FULL = 0xffffffffu;
    __shared__ int sh_bad, sh_last, sh_scan[kChunkPlanThreads / 32], sh_run;
    __shared__ int hist[kChunkSortBins];
    __shared__ ChunkSeq sh_seqs[kChunkPlanSeqs];
    __shared__ int sh_base[kChunkPlanSeqs + 1], sh_tiles[kChunkPlanBlocks];
    __shared__ float est[kChunkCandidates];
    __shared__ int est_chunk[kChunkCandidates];
    __shared__ long long sh_sum;
    __shared__ int sh_max, sh_entries, sh_slots, sh_groups, sh_chunk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool alone = gridDim.x == 1;  // one CTA checks every sequence (it needs no hand-over between CTAs)
    if (alone) {
        // (one CTA only where its shared memory holds the sequences)
        for (int s = tid; s < a.batch; s += kChunkPlanThreads) {
            const int lo = __ldg(a.cu + s), hi = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
            const int bad = lo < 0 || lo > hi || hi > a.n_tokens ? kDevBadRange : len < 0 || len > a.cap_u ? 1 : 0;
            sh_seqs[s] = ChunkSeq{lo, hi - lo, len, bad};
        }
        if (tid == 0) sh_bad = 0;
        __syncthreads();
        if (a.paged) {
            const int total = a.batch * a.max_pages;
            for (int x = tid; x < total; x += kChunkPlanThreads) {
                const int s = x / a.max_pages, p = x - s * a.max_pages;
                const int id = __ldg(a.block_table + x);
                if (p * a.page_size < sh_seqs[s].len && sh_seqs[s].n > 0 && sh_seqs[s].bad == 0 && (id < 0 || id >= a.n_pages))
                    sh_bad = 1;
            }
            __syncthreads();
            if (sh_bad) {  // some page is missing: which sequences lack one
                for (int s = warp; s < a.batch; s += kChunkPlanThreads / 32) {
                    bool ok = true;
                    if (sh_seqs[s].n > 0 && sh_seqs[s].bad == 0)
                        for (int p = lane; p * a.page_size < sh_seqs[s].len; p += 32) {
                            const int id = __ldg(a.block_table + (long long)s * a.max_pages + p);
                            ok = ok && id >= 0 && id < a.n_pages;
                        }
                    ok = __all_sync(FULL, ok);
                    if (!ok && lane == 0) sh_seqs[s].bad = 2;  // TRI_DEV_BAD_PAGE
                }
                __syncthreads();
            }
        }
        for (int s = tid; s < a.batch; s += kChunkPlanThreads)
            if (sh_seqs[s].bad) record_status(a.status, sh_seqs[s].bad, (long long)s * a.n_kv);
    } else {
        const int s0 = blockIdx.x;
        const int lo = __ldg(a.cu + s0), hi = __ldg(a.cu + s0 + 1), len = __ldg(a.lens + s0);
        const long long cap = a.cap_u;
        int bad = 0;
        if (lo < 0 || lo > hi || hi > a.n_tokens) bad = kDevBadRange;
        else if (len < 0 || len > cap) bad = 1;  // TRI_DEV_LEN_GT_CAP
        if (tid == 0) sh_bad = 0;
        __syncthreads();
        if (!bad && a.paged && hi > lo) {
            const int np = (len + a.page_size - 1) / a.page_size;
            bool ok = true;
            for (int p = tid; p < np; p += kChunkPlanThreads) {
                const int id = __ldg(a.block_table + (long long)s0 * a.max_pages + p);
                ok = ok && id >= 0 && id < a.n_pages;
            }
            if (!ok) sh_bad = 2;                 // TRI_DEV_BAD_PAGE
        }
        __syncthreads();
        if (!bad) bad = sh_bad;
        if (tid == 0) {
            a.seqs[s0] = ChunkSeq{lo, hi - lo, len, bad};
            if (bad) record_status(a.status, bad, (long long)s0 * a.n_kv);
            __threadfence();
            sh_last = atomicAdd(reinterpret_cast<unsigned *>(a.status + 1), 1u) == gridDim.x - 1;
        }
    }
    if (!alone) {
        __syncthreads();
        if (!sh_last) return;
        __threadfence();
    }

    // small plans are worked out in shared memory, larger ones in the workspace
    const ChunkSeq *seqs = a.batch <= kChunkPlanSeqs ? sh_seqs : a.seqs;
    int *base = a.batch <= kChunkPlanSeqs ? sh_base : a.base;
    // blocks before each sequence; a bad range refuses every sequence (the ranges may overlap)
    bool range_ok = true;
    for (int s = tid; s < a.batch; s += kChunkPlanThreads) {
        if (!alone) {
            const int4 v = __ldcg(reinterpret_cast<const int4 *>(a.seqs + s));
            if (a.batch <= kChunkPlanSeqs) sh_seqs[s] = ChunkSeq{v.x, v.y, v.z, v.w};
            range_ok = range_ok && v.w != kDevBadRange;
        } else {
            range_ok = range_ok && sh_seqs[s].bad != kDevBadRange;
        }
    }
    range_ok = __syncthreads_and(range_ok);
    if (tid == 0) {
        sh_run = 0;
        sh_sum = 0;
        sh_max = 0;
        if (!alone) *reinterpret_cast<unsigned *>(a.status + 1) = 0;
    }
    __syncthreads();
    const int G = a.group, tpb = kChunkRows / G;
    for (int c0 = 0; c0 < a.batch; c0 += kChunkPlanThreads) {
        const int s = c0 + tid;
        int nb = 0;
        if (range_ok && s < a.batch && seqs[s].bad == 0) nb = chunk_blocks(seqs[s].n, G);
        int inc = nb;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sh_scan[warp] = inc;
        __syncthreads();
        int before = sh_run;
        for (int w = 0; w < warp; ++w) before += sh_scan[w];
        if (s < a.batch) base[s] = before + inc - nb;
        __syncthreads();
        if (tid == kChunkPlanThreads - 1) sh_run = before + inc;
        __syncthreads();
    }
    const int n_blocks = sh_run;
    int *tiles = n_blocks <= kChunkPlanBlocks ? sh_tiles : a.tiles;
    __syncthreads();
    const int LH = a.n_layers * a.n_kv;
    // sequence of block e, and its line without splits
    auto block_of = [&](int e) {
        int lo = 0, hi = a.batch;  // the last s with base[s] <= e: empty sequences before it are skipped
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (base[mid] <= e) lo = mid; else hi = mid;
        }
        const int n = seqs[lo].n, len = seqs[lo].len;
        const int b = e - base[lo];
        ChunkEntry x;
        x.s = lo;
        x.tok0 = seqs[lo].q0 + b * tpb;
        x.ntok = min(tpb, n - b * tpb);
        x.len = len;
        x.first = a.causal ? len - n + b * tpb + 1 : len;
        const int end = a.causal ? min(len, max(0, x.first + x.ntok - 1)) : len;
        x.kt0 = 0;
        x.kt1 = (end + 127) / 128;
        x.nsplit = 1;
        x.split = 0;
        x.slot = 0;
        x.pair = 0;
        return x;
    };
    {
        long long sum = 0;
        int mx = 0;
        for (int e = tid; e < n_blocks; e += kChunkPlanThreads) {
            const ChunkEntry x = block_of(e);
            tiles[e] = x.kt1;
            sum += x.kt1;
            mx = max(mx, x.kt1);
        }
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(FULL, sum, o);
            mx = max(mx, __shfl_xor_sync(FULL, mx, o));
        }
        if (lane == 0) {
            atomicAdd(reinterpret_cast<unsigned long long *>(&sh_sum), (unsigned long long)sum);
            atomicMax(&sh_max, mx);
        }
    }
    __syncthreads();
    // the longest split: the warps weigh candidates, each a share of an SM's even part of the work. The
    // time of a candidate is at most rounds * longest and at most even part + longest (both bounds
    // of handing items out longest first); the smaller of them counts.
    {
        const float per_sm = 1.f / (float)a.sm_count, even = (float)sh_sum * (float)LH * per_sm;
        // the first candidate does not split
        __shared__ float share[kChunkCandidates];
        if (tid < kChunkCandidates)  // 1.6, 1.3, 1.15, 1.07, 1, and 1 / n of it down to 1/6
            share[tid] = tid < 5 ? 1.f + (tid == 1 ? .6f : tid == 2 ? .3f : tid == 3 ? .15f : .07f) : 2.f / (float)(tid - 3);
        __syncthreads();
#pragma unroll 1
        for (int cand = warp; cand < kChunkCandidates; cand += kChunkPlanThreads / 32) {
            const float want = ceilf(even * share[cand]);
            const int chunk = cand == 0 ? max(1, sh_max) : max(2, (int)fminf((float)max(1, sh_max), want));
            int items = 0, work = 0, longest = 0, slots = 0, merge_rows = 0;
#pragma unroll 1
            for (int e = lane; e < n_blocks; e += 32) {
                const int t = tiles[e];
                int ns = max(1, (t + chunk - 1) / chunk);
                const int per = (t + ns - 1) / ns;
                if (t > 0) ns = (t + per - 1) / per;
                items += ns;
                work += t + ns * kChunkItemCost;
                longest = max(longest, per);
                if (ns > 1) {
                    slots += ns;
                    merge_rows = max(merge_rows, min(tpb, a.n_tokens));
                }
            }
            items = __reduce_add_sync(FULL, items);
            work = __reduce_add_sync(FULL, work);
            longest = __reduce_max_sync(FULL, longest);
            slots = __reduce_add_sync(FULL, slots);
            merge_rows = __reduce_max_sync(FULL, merge_rows);
            if (lane == 0) {
                const float one = (float)(longest + kChunkItemCost);
                float cost = fminf(ceilf((float)items * (float)LH * per_sm) * one, (float)work * (float)LH * per_sm + one);
                if (slots > 0) cost += (float)(kChunkMergeCost + kChunkMergeRows * merge_rows / tpb);
                if ((long long)slots * LH > a.max_slots || items > a.max_entries) cost = 3e38f;
                est[cand] = cost;
                est_chunk[cand] = chunk;
            }
        }
    }
    // (only the bins of lengths up to the longest are used)
    const int bin0 = (kChunkSortBins - 1 - min(sh_max, kChunkSortBins - 1)) & ~31;
    for (int i = bin0 + tid; i < kChunkSortBins; i += kChunkPlanThreads) hist[i] = 0;
    __syncthreads();
    if (tid == 0) {
        int best = 0;
        for (int w = 1; w < kChunkCandidates; ++w)
            if (est[w] < est[best]) best = w;
        sh_chunk = est_chunk[best];
        sh_slots = 0;
        sh_groups = 0;
    }
    __syncthreads();
    // lines of each length, longest first
    const int chunk = sh_chunk;
    auto bin_of = [](int per) { return kChunkSortBins - 1 - min(per, kChunkSortBins - 1); };
    for (int e = tid; e < n_blocks; e += kChunkPlanThreads) {
        const int t = tiles[e];
        int ns = max(1, (t + chunk - 1) / chunk);
        const int per = (t + ns - 1) / ns;
        if (t > 0) ns = (t + per - 1) / per;
        atomicAdd(&hist[bin_of(per)], ns);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix sums of the bins
        int run = 0;
        for (int i0 = bin0; i0 < kChunkSortBins; i0 += 32) {
            const int x = hist[i0 + lane];
            int inc = x;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(FULL, inc, o);
                if (lane >= o) inc += y;
            }
            hist[i0 + lane] = run + inc - x;
            run += __shfl_sync(FULL, inc, 31);
        }
        if (lane == 0) sh_entries = run;
    }
    __syncthreads();
    for (int e = tid; e < n_blocks; e += kChunkPlanThreads) {
        ChunkEntry x = block_of(e);
        const int t = x.kt1;
        int ns = max(1, (t + chunk - 1) / chunk);
        const int per = (t + ns - 1) / ns;
        if (t > 0) ns = (t + per - 1) / per;
        const int at = atomicAdd(&hist[bin_of(per)], ns);
        x.nsplit = ns;
        if (ns > 1) {
            x.slot = atomicAdd(&sh_slots, ns);
            a.merges[atomicAdd(&sh_groups, 1)] = x;
        }
        for (int k = 0; k < ns; ++k) {
            x.split = k;
            x.kt0 = k * per;
            x.kt1 = min(t, (k + 1) * per);
            x.pair = x.ntok * G <= 128 && x.kt1 - x.kt0 >= 2;
            a.entries[at + k] = x;
        }
    }
    __syncthreads();
    if (tid == 0) {
        a.head->n_entries = sh_entries;
        a.head->n_groups = sh_groups;
    }
}

// ---------------------------------------------------------------------------------
// PTX of the attention kernel.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ void tma_tile_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// Shared-memory matrix descriptors in the 128-byte swizzle as (low, high) words: the start address and
// the leading offset, in units of 16 bytes, are the low word, to which a k-step adds a constant. The
// high word: 8-row groups 1024 bytes apart, descriptor version 1, swizzle mode.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr, unsigned lead_bytes) {
    return (smem_addr >> 4) | ((lead_bytes >> 4) << 16);
}
// In the roles below an instruction that one lane issues carries its predicate (`on`) with it instead of
// standing in a branch: a warp that diverges and joins again around each of them lost more time in a
// step than its MMAs take.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
__device__ __forceinline__ void chunk_mma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, int acc,
                                             uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(acc), "r"(kDescHigh), "r"(on)
        : "memory");
}
// A (bf16 pairs, one row per lane) in tensor memory.
__device__ __forceinline__ void chunk_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, int acc,
                                             uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(acc), "r"(kDescHigh), "r"(on)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint64_t *bar, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(on)
        : "memory");
}
__device__ __forceinline__ void arrive_if(uint64_t *bar, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(on)
        : "memory");
}
__device__ __forceinline__ void expect_tx_if(uint64_t *bar, unsigned bytes, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(on)
        : "memory");
}
__device__ __forceinline__ void tma_tile_2d_if(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "r"(on)
        : "memory");
}
// Three-input maximum that keeps a NaN.
__device__ __forceinline__ float max3nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// A position in the ring of tiles.
template <int NST>
struct ChunkRing {
    int stage = 0;
    unsigned phase = 0;
    __device__ __forceinline__ void step() {
        if (++stage == NST) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

#define TRI_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define TRI_U8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
#define TRI_W8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])

// 32 columns of this warp's 32 TMEM lanes; valid after tmem_wait32 on the same registers.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : TRI_R8(r, 0), TRI_R8(r, 8), TRI_R8(r, 16), TRI_R8(r, 24)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::TRI_U8(r, 0),
        TRI_U8(r, 8), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : TRI_W8(r, 0), TRI_W8(r, 8), TRI_W8(r, 16), TRI_W8(r, 24) : : "memory");
}
// Orders later uses of r after a tmem_wait32 issued just before (no instruction).
__device__ __forceinline__ void tmem_after32(uint32_t (&r)[32]) {
    asm volatile("" : TRI_W8(r, 0), TRI_W8(r, 8), TRI_W8(r, 16), TRI_W8(r, 24) : : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x of a pair on the FMA pipe: x = n + f with |f| <= 1/2 (round to nearest by adding 1.5 * 2^23, the
// reduction of Cody and Waite), 2^f by the degree-4 polynomial of least largest relative error on
// [-1/2, 1/2] (2.6e-6, found by Remez exchange), n added to the exponent. x <= 127. What x = -126 gives is taken off
// again, so that everything from there down to -infinity is exactly 0: a key that is not seen weighs nothing, however
// large its value (2^-126 times 3e38 would be 3.5). For a NaN: 0; such a row is told by its maximum.
__device__ __forceinline__ float2 exp2_pair(float2 x) {
    x.x = fmaxf(x.x, -126.f);
    x.y = fmaxf(x.y, -126.f);
    const float2 magic = make_float2(12582912.f, 12582912.f), unmagic = make_float2(-12582912.f, -12582912.f);
    const float2 t = __fadd2_rn(x, magic);
    const float2 n = __fadd2_rn(t, unmagic);
    const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
    float2 p = __ffma2_rn(f, make_float2(0.009570102207362652f, 0.009570102207362652f),
                          make_float2(0.05591785907745361f, 0.05591785907745361f));
    p = __ffma2_rn(p, f, make_float2(0.240247443318367f, 0.240247443318367f));
    p = __ffma2_rn(p, f, make_float2(0.6931217908859253f, 0.6931217908859253f));
    p = __ffma2_rn(p, f, make_float2(0.9999992847442627f, 0.9999992847442627f));
    p = make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                    __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
    // at x = -126 f is 0 and p the last coefficient, its exponent 126 lower (a subnormal, which the sum keeps)
    constexpr int kLowest = 0x3f7ffff4 - (126 << 23);  // 0x3f7ffff4: 0.9999992847442627f
    const float low = -__int_as_float(kLowest);
    return __fadd2_rn(p, make_float2(low, low));
}

// Heads of 64 leave 128 columns of tensor memory free: P has columns of its own there, so that the next S is
// computed while the warpgroup still exponentiates this one (at head 128 P lies over S).
__host__ __device__ constexpr bool chunk_apart(int D) { return D == 64; }

struct ChunkSmem {
    unsigned q, ring, ml, bars, total;
};
__host__ __device__ inline ChunkSmem chunk_smem(int D) {
    ChunkSmem L;
    const unsigned NST = (unsigned)chunk_stages(D);
    L.q = 0;
    L.ring = 2u * (unsigned)D * 256u;               // two query tiles of 128 rows
    L.ml = L.ring + NST * (unsigned)D * 256u;  // a paired item's second (m, l) of each row
    L.bars = L.ml + 128u * 8u;
    // full, empty [stages each], q full and empty, S, P, most of P and O full [2 each], done, S free and
    // P V done [2 each], exchange full and free,
    // turns [2], TMEM address, abort
    L.total = L.bars + (2u * NST + 19u) * 8u + 32u + 1024u;  // + alignment slack
    return L;
}

// E consecutive bf16 elements, a lane's share of a row.
template <int E>
struct ChunkLane {
    using Vec = unsigned;
    using Acc = float2;
};
template <>
struct ChunkLane<4> {
    using Vec = uint2;
    using Acc = float4;
};
template <int E>
__device__ __forceinline__ void chunk_lane(const typename ChunkLane<E>::Vec &w, float (&x)[E]) {
    const unsigned *u = reinterpret_cast<const unsigned *>(&w);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        x[e] = bf16lo(u[e / 2]);
        x[e + 1] = bf16hi(u[e / 2]);
    }
}
// An MMA multiplies what a row does not see by a zero weight, which leaves nothing of a finite value but makes a NaN of
// an infinity or a NaN among the values. So a dim of a row that came out not finite, where the item goes on past the
// keys that the row sees and one of those hidden values is not finite in that dim, is computed again over the seen
// keys of the item alone: by a warp, on the CUDA cores (weights in fp32, about 0.2 us a key), until every dim in question has
// met a NaN. What is not finite for a reason that the row does see stays as it is; telling so costs a look at the item's
// hidden values (at most 383 keys). `in_block`: the row among the block's, `slot` where the item's part lies.
// Its code is kept small, for calls that never run it pay for its size: 1 us here (of the 40 for 16 single tokens), 5 us
// when the merge kernel held it in a faster form.
template <int D>
__device__ __forceinline__ void chunk_row_again(const ChunkArgs &a, const ChunkEntry &en, int lr, int g, long long slot, int in_block) {
    constexpr int E = D / 32;  // lane's dims: [lane * E, + E)
    constexpr unsigned FULL = 0xffffffffu;
    const float NEG_INF = __int_as_float(0xff800000);
    using Vec = typename ChunkLane<E>::Vec;
    const int lane = threadIdx.x & 31, shift = __ffs(a.group) - 1;
    const int tok = en.tok0 + (in_block >> shift), head = g * a.group + (in_block & (a.group - 1));
    const int k0 = en.kt0 * 128, end = min(en.len, en.kt1 * 128);
    const int seen = max(k0, min(end, en.first + (in_block >> shift))), hide = end - seen;
    const bool part = en.nsplit > 1;
    if (hide <= 0) return;
    using Acc = typename ChunkLane<E>::Acc;
    Vec *out = reinterpret_cast<Vec *>(a.out + lr * a.o_l + tok * a.o_t + head * a.o_h + lane * E);
    Acc *acc_out = reinterpret_cast<Acc *>(a.part + ((slot * (D / 4) + lane * E / 4) * 128 + (in_block & 127)) * 4 + lane * E % 4);
    unsigned todo = 0, hidden = 0;  // this lane's dims that are not finite here, and in a hidden value
    alignas(16) float was[E];
    float qv[E], acc[E], m = NEG_INF, l = 0.f;
    if (part) *reinterpret_cast<Acc *>(was) = *acc_out; else chunk_lane<E>(*out, was);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (!(fabsf(was[e]) < __int_as_float(0x7f800000))) todo |= 1u << e;
        acc[e] = 0.f;
    }
    if (!__any_sync(FULL, todo != 0)) return;
    chunk_lane<E>(*reinterpret_cast<const Vec *>(a.q + lr * a.q_l + tok * a.q_t + head * a.q_h + lane * E), qv);
#pragma unroll 1
    for (int i = 0; i < end - k0; ++i) {
        const int j = i < hide ? seen + i : k0 + i - hide;  // the hidden keys, then those that it sees
        int unit = lr * a.batch + en.s, rows = a.cap_u, off = j;
        if (a.paged) {
            const int p = j / a.page_size;
            rows = a.page_size;
            off = j - p * rows;
            unit = lr * a.n_pages + __ldg(a.block_table + (long long)en.s * a.max_pages + p);
        }
        const long long at = (((long long)unit * a.n_kv + g) * rows + off) * D + lane * E;
        float v[E], k[E], x = 0.f;
        chunk_lane<E>(*reinterpret_cast<const Vec *>(a.V + at), v);
        chunk_lane<E>(*reinterpret_cast<const Vec *>(a.K + at), k);
        if (i < hide) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!(fabsf(v[e]) < __int_as_float(0x7f800000))) hidden |= 1u << e;
            if (i == hide - 1) {
                todo &= hidden;
                if (!__any_sync(FULL, todo != 0)) return;
            }
            continue;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x += qv[e] * k[e];
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
        x *= a.c;
        const float mn = fmaxf(m, x), z = mn == NEG_INF ? 0.f : mn;
        const float corr = ex2_approx(m - z), p = ex2_approx(x - z);
        m = mn;
        l = l * corr + p;
        bool open = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[e] = acc[e] * corr + p * v[e];
            open = open || ((todo >> e & 1u) && acc[e] == acc[e]);
        }
        if (!__any_sync(FULL, open)) break;
    }
    // a part goes by the maximum that it was written with; one that sees no key weighs nothing, whatever it holds
    const float scale = l == 0.f ? 0.f : part ? ex2_approx(m - a.part_ml[(slot * 128 + (in_block & 127)) * 2]) : 1.f / l;
    alignas(8) unsigned w[E / 2];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (todo >> e & 1u) was[e] = acc[e] * scale;
        if (e & 1) w[e / 2] = pack_bf16(was[e - 1], was[e]);
    }
    if (part) *acc_out = *reinterpret_cast<Acc *>(was); else *out = *reinterpret_cast<Vec *>(w);
}
// A CTA's item of round r: forth in even rounds, back in odd ones.
__device__ __forceinline__ unsigned chunk_item(int r) {
    const int pos = (r & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
    return (unsigned)r * gridDim.x + (unsigned)pos;
}

// (Not inline: inlined in the five places that call it, it cost every call 1 us by its size.)
__device__ __noinline__ void chunk_timed_out(unsigned long long *status, int n_kv, int batch, int s, int lh) {
    record_status(status, kDevTimeout, ((long long)(lh / n_kv) * batch + s) * n_kv + lh % n_kv);
}

// A 128-key tile of one row: S from tensor memory, masked, into the running (m, l); P over S. `left`: the
// tile's keys that the row sees (cut: some row of the tile sees fewer than 128). `fresh`: the first tile.
//
// The hardware exponential takes 8 clocks a warp, 1024 for the tile; `kEmu` of every 8 pairs are evaluated on the
// FMA pipe instead. Measured with 0, 1, 2 of 8: 844, 835, 854 us (two causal prompts of 8192 and 6145 tokens, head 128) and 522,
// 510, 507 us (512 tokens over 32768 rows); head 64 (two prompts of 4096 tokens): 244, 250, 247 us.
template <int D>
__device__ __forceinline__ bool chunk_softmax_tile(uint32_t ts, uint32_t tp, uint32_t to, float c, bool cut, int left,
                                                   bool fresh, float &m, float &l, int lane, uint64_t *most,
                                                   uint64_t *sfree, uint64_t *pv, unsigned pv_parity, int tries) {
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int kEmu = D == 128 ? 1 : 0;
    const float NEG_INF = __int_as_float(0xff800000);
    uint32_t s0[32], s1[32], s2[32], s3[32];
    float x0 = NEG_INF, x1 = NEG_INF, x2 = NEG_INF, x3 = NEG_INF;
    auto top = [&](uint32_t(&s)[32], int at) {
        if (cut) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (at + j >= left) s[j] = 0xff800000u;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            x0 = max3nan(x0, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            x1 = max3nan(x1, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
            x2 = max3nan(x2, __uint_as_float(s[j + 4]), __uint_as_float(s[j + 5]));
            x3 = max3nan(x3, __uint_as_float(s[j + 6]), __uint_as_float(s[j + 7]));
        }
    };
    tmem_ld32(ts, s0);
    tmem_wait32(s0);
    tmem_ld32(ts + 32u, s1);
    tmem_ld32(ts + 64u, s2);
    tmem_ld32(ts + 96u, s3);
    top(s0, 0);
    tmem_wait32(s1);
    tmem_after32(s2);
    tmem_after32(s3);
    if (chunk_apart(D)) {  // the next S may come
        tc_fence_before();
        __syncwarp();
        arrive_if(sfree, lane == 0);
    }
    top(s1, 32);
    top(s2, 64);
    top(s3, 96);
    const float mx = max3nan(max3nan(x0, x1, x2), x3, x3);
    if (fresh) {
        m = mx;
    } else if (__any_sync(FULL, mx != NEG_INF && !((mx - m) * c <= 8.f))) {
        // once P V of the tiles before is complete, O is this warpgroup's to rescale
        if (chunk_apart(D) && !__all_sync(FULL, mbar_wait_bounded(pv, pv_parity, tries))) return false;
        tc_fence_after();
        const float mn = max3nan(m, mx, mx);
        const float f = m == mn ? 1.f : ex2_approx((m - mn) * c);
        m = mn;
        l *= f;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t o[16];
            tmem_ld16_issue(to + c0, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(to + c0, o);
        }
    }
    // a NaN logit, or an infinite one (inf - inf), makes the row's maximum NaN and with it all its weights
    const float mc = m == NEG_INF ? 0.f : (m + (m - m)) * c;
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
    const float2 c2 = make_float2(c, c), m2 = make_float2(-mc, -mc);
    uint32_t p[16];
    auto weights = [&](const uint32_t(&s)[32], int from, int upto) {
#pragma unroll
        for (int j = from; j < upto; j += 2) {
            float2 y = __ffma2_rn(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), c2, m2);
            if (j / 2 * kEmu % 8 + kEmu > 7 && kEmu > 0)
                y = exp2_pair(y);
            else
                y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            if (j % 4 == 0) sum0 = __fadd2_rn(sum0, y); else sum1 = __fadd2_rn(sum1, y);
            p[j / 2] = pack_bf16(y.x, y.y);
        }
    };
    weights(s0, 0, 32);
    if (chunk_apart(D) && !fresh) {  // the P before has been read
        if (!__all_sync(FULL, mbar_wait_bounded(pv, pv_parity, tries))) return false;
        tc_fence_after();
    }
    tmem_st16(tp, p);
    weights(s1, 0, 32);
    tmem_st16(tp + 16u, p);
    weights(s2, 0, 32);
    tmem_st16(tp + 32u, p);
    // the first 96 keys' weights are handed over once their stores, by now under way for a while, are done,
    // so that most of P V runs during the rest
    weights(s3, 0, 16);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    arrive_if(most, lane == 0);
    weights(s3, 16, 32);
    tmem_st16(tp + 48u, p);
    l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
    tmem_wait_st();
    return true;
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    tri_chunk_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const ChunkArgs a) {
    constexpr int KCH = D / 64;                       // 64-dim (128-byte) chunks of a row
    constexpr unsigned kTileBytes = (unsigned)D * 256u;
    constexpr unsigned kChunkBytes = 128u * 128u;
    constexpr unsigned FULL = 0xffffffffu;
    const float NEG_INF = __int_as_float(0xff800000);
    extern __shared__ unsigned char chunk_smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(chunk_smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    constexpr int NST = chunk_stages(D);
    const ChunkSmem Ly = chunk_smem(D);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Ly.bars);
    uint64_t *empty = full + NST;
    uint64_t *qfull = empty + NST;
    uint64_t *qempty = qfull + 1;
    uint64_t *sfull = qempty + 1;   // [2]
    uint64_t *pfull = sfull + 2;    // [2]
    uint64_t *pmost = pfull + 2;    // [2]
    uint64_t *ofull = pmost + 2;    // [2]
    uint64_t *done = ofull + 2;
    uint64_t *sfree = done + 1;     // [2] (heads of 64)
    uint64_t *pv = sfree + 2;       // [2] (heads of 64)
    uint64_t *xfull = pv + 2;
    uint64_t *xfree = xfull + 1;
    uint64_t *turn = xfree + 1;     // [2]
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(turn + 2);
    float2 *ml_x = reinterpret_cast<float2 *>(smem + Ly.ml);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 2);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 2);        // an arrival of each MMA warp
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 4);  // the warpgroup's warps
            mbar_init(pmost + i, 4);
            mbar_init(ofull + i, 1);
            mbar_init(sfree + i, 4);
            mbar_init(pv + i, 1);
            mbar_init(turn + i, 1);
        }
        mbar_init(done, 2);
        mbar_init(xfull, 4);
        mbar_init(xfree, 4);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) {  // one CTA per SM: the whole tensor memory
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // a programmatic dependent of the plan kernel: the plan is read after this
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int G = a.group, LH = a.n_layers * a.n_kv;
    const unsigned n_items = (unsigned)a.head->n_entries * (unsigned)LH;  // below 2^31
    auto fail = [&](const ChunkEntry &e, int lh) {
        chunk_timed_out(a.status, a.n_kv, a.batch, e.s, lh);
        *abort_flag = 1;
    };

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChunkRegsFew));
    if (warp == 0) {
        // ---------------- loads ----------------
        ChunkRing<NST> fill;
        int k = 0, nq = 0;      // ring fills so far, query tiles loaded so far
        bool ok = true;
        for (int r = 0; ok && !*abort_flag; ++r) {
            const unsigned it = chunk_item(r);
            if (it >= n_items) break;
            const ChunkEntry e = a.entries[it / LH];
            const int lh = (int)(it % LH), lr = lh / a.n_kv, g = lh % a.n_kv;
            if (e.kt1 <= e.kt0) continue;
            const int ntile = e.ntok * G > 128 ? 2 : 1;
            if (nq > 0 && !__all_sync(FULL, mbar_wait_bounded(qempty, (unsigned)((nq - 1) & 1), a.wait_tries))) {
                if (lane == 0) fail(e, lh);
                break;
            }
            if (lane == 0) {
                mbar_expect_tx(qfull, (unsigned)ntile * kTileBytes);
                for (int q = 0; q < ntile; ++q)
                    for (int c = 0; c < KCH; ++c)
                        tma_tile_4d(smem + Ly.q + q * kTileBytes + c * kChunkBytes, &qmap, c * 64, g * G,
                                    e.tok0 + q * (128 / G), lr, qfull);
            }
            ++nq;
            const int pr = a.piece_rows, np = 128 / pr;
            const int p = lane / KCH, c = lane % KCH;  // this lane's box of a tile
            const bool withhold = e.kt0 == 0 && ((long long)lr * a.batch + e.s) * a.n_kv + g == a.inject_unit;
            auto page_of = [&](int kt) {
                const int r0 = kt * 128 + p * pr;
                return (a.paged && p < np && r0 < e.len && kt < e.kt1)
                           ? __ldg(a.block_table + (long long)e.s * a.max_pages + r0 / a.page_size) : 0;
            };
            // tiles in the order in which the MMA warp takes them: the first key tile (two of a paired
            // item), then each value tile followed by the key tile `lead` after it
            const int lead = e.pair ? 2 : 1, n = e.kt1 - e.kt0;
            int pages[3] = {page_of(e.kt0), page_of(e.kt0 + 1), page_of(e.kt0 + 2)};  // of the next value tile on
            auto tile = [&](int kt, int page, const CUtensorMap *map, bool skip) {
                const int r0 = kt * 128 + p * pr;
                long long row;
                if (a.paged)
                    row = (((long long)lr * a.n_pages + page) * a.n_kv + g) * (long long)a.page_size + r0 % a.page_size;
                else
                    row = (((long long)lr * a.batch + e.s) * a.n_kv + g) * (long long)a.cap_u + r0;
                const int pieces = min(np, (e.len - kt * 128 + pr - 1) / pr);
                const int st = fill.stage;
                if (k >= NST && !__all_sync(FULL, mbar_wait_bounded(empty + st, fill.phase ^ 1u, a.wait_tries))) {
                    if (lane == 0) fail(e, lh);
                    return false;
                }
                // (an MMA warp may have written zeros to this stage with the generic proxy)
                fence_proxy_async_smem();
                expect_tx_if(full + st, (unsigned)(pieces * pr) * 128u * KCH, lane == 0);
                __syncwarp();
                tma_tile_2d_if(smem + Ly.ring + (unsigned)st * kTileBytes + c * kChunkBytes + (unsigned)(p * pr) * 128u, map,
                                c * 64, (int)row, full + st, p < np && r0 < e.len && !skip);
                ++k;
                fill.step();
                return true;
            };
            // test hook: the unit's first key tile is armed but never loaded
            ok = tile(e.kt0, pages[0], &kmap, withhold);
            if (ok && e.pair) ok = tile(e.kt0 + 1, pages[1], &kmap, false);
            for (int i = 0; ok && i < n; ++i) {
                const int next = page_of(e.kt0 + i + 3);
                ok = tile(e.kt0 + i, pages[0], &vmap, false);
                if (ok && i + lead < n) ok = tile(e.kt0 + i + lead, pages[lead], &kmap, false);
                pages[0] = pages[1];
                pages[1] = pages[2];
                pages[2] = next;
            }
        }
        // copies still in flight must land before the CTA exits
        for (int j = k > NST ? k - NST : 0; j < k; ++j)
            (void)mbar_wait_bounded(full + j % NST, (unsigned)((j / NST) & 1), a.wait_tries);
        if (nq > 0) (void)mbar_wait_bounded(qfull, (unsigned)((nq - 1) & 1), a.wait_tries);
        __syncwarp();
    } else if (warp <= 2) {
        // ---------------- MMAs: one warp for each warpgroup's, so that one's bookkeeping and waits run beside
        // the other's MMAs (a single warp left the tensor core idle for about 900 of 4100 clocks a tile)
        const int q = warp - 1;
        const uint32_t id_s = mx_idesc(128), id_o = mx_idesc(D) | (1u << 16);  // V is N-major
        const uint32_t q_low = desc_low(smem_u32(smem + Ly.q), 16u), k_low = desc_low(smem_u32(smem + Ly.ring), 16u);
        const uint32_t v_low = desc_low(smem_u32(smem + Ly.ring), kChunkBytes);
        const uint32_t sd = tmem + 128u * q, od = tmem + 256u + (uint32_t)(D * q);
        const uint32_t pd = chunk_apart(D) ? tmem + 384u + 64u * q : sd;
        const uint32_t lead_lane = elect_one();
        ChunkRing<NST> at;            // the next tile
        unsigned nq = 0, np = 0;      // items, P tiles so far
        unsigned nt = 0;              // turns waited for
        bool owed = false;            // the other warp's turn comes before this one's next
        bool ok = true;
        auto wait = [&](uint64_t *bar, unsigned phase) {
            return __all_sync(FULL, mbar_wait_bounded(bar, phase & 1u, a.wait_tries));
        };
        // a tile that is the other warp's: its release takes an arrival of each
        auto skip = [&] {
            ok = ok && wait(full + at.stage, at.phase);
            arrive_if(empty + at.stage, ok && lane == 0);
            at.step();
        };
        for (int r = 0; ok && !*abort_flag; ++r) {
            const unsigned it = chunk_item(r);
            if (it >= n_items) break;
            const ChunkEntry e = a.entries[it / LH];
            // (values that the compiler shall know to be the same in every lane go through a shuffle)
            const int n = __shfl_sync(FULL, e.kt1 - e.kt0, 0);
            if (n <= 0) continue;
            const bool pair = __shfl_sync(FULL, e.pair, 0) != 0;
            const bool both = pair || __shfl_sync(FULL, e.ntok * G, 0) > 128, idle = q == 1 && !both;
            const int lead = pair ? 2 : 1, left = __shfl_sync(FULL, e.len - e.kt0 * 128, 0);
            const uint32_t ql = q_low + (pair ? 0u : (uint32_t)q * (kTileBytes >> 4));
            auto mma_s = [&](uint32_t bl, uint32_t on) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const unsigned off = ((unsigned)(ks >> 2) * kChunkBytes + (unsigned)(ks & 3) * 32u) >> 4;
                    chunk_mma_ss(sd, ql + off, bl + off, id_s, ks > 0, on);
                }
                commit_if(sfull + q, on);
            };
            ok = wait(qfull, nq);
            ++nq;
            if (!ok || idle) {
                for (int i = 0; ok && i < 2 * n; ++i) skip();
                arrive_if(qempty, ok && lane == 0);
            } else {
                // the last key tile of this warp: after it the query tile is free
                const int end = pair ? n - 1 - ((n - 1 - q) & 1) : n - 1;
                for (int t = 0; ok && t < lead; ++t) {
                    if (pair && t != q) {
                        skip();
                        continue;
                    }
                    ok = wait(full + at.stage, at.phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t bl = __shfl_sync(FULL, k_low + (unsigned)at.stage * (kTileBytes >> 4), 0);
                    mma_s(bl, lead_lane);
                    commit_if(empty + at.stage, lead_lane);
                    commit_if(qempty, lead_lane && t == end);
                    at.step();
                }
                for (int i = 0; ok && i < n; ++i) {
                    const bool more = i + lead < n;
                    if (pair && (i & 1) != q) {
                        skip();
                        if (more) skip();
                        continue;
                    }
                    const ChunkRing<NST> av = at;  // this tile's V; `at`: the K `lead` tiles on
                    at.step();
                    ok = wait(full + av.stage, av.phase);
                    if (!ok) break;
                    // value rows past the length hold whatever was there: zero them, for a zero weight does
                    // not clear a NaN (both warps of a tile that they share write the same zeros)
                    const int valid = left - i * 128;
                    if (valid < 128) {
                        unsigned char *Vs = smem + Ly.ring + (unsigned)av.stage * kTileBytes;
                        const int words = (128 - valid) * 8;  // 16-byte words of a chunk
                        for (int w = lane; w < words * KCH; w += 32) {
                            const int c = w / words, x = w % words;
                            *reinterpret_cast<uint4 *>(Vs + c * kChunkBytes + (unsigned)valid * 128u + (unsigned)x * 16u) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const uint32_t vl = __shfl_sync(FULL, v_low + (unsigned)av.stage * (kTileBytes >> 4), 0);
                    const uint32_t bl = __shfl_sync(FULL, k_low + (unsigned)at.stage * (kTileBytes >> 4), 0);
                    ok = !more || wait(full + at.stage, at.phase);
                    if (chunk_apart(D) && more && ok) {
                        ok = wait(sfree + q, np);
                        tc_fence_after();
                        mma_s(bl, lead_lane && ok);
                        commit_if(empty + at.stage, lead_lane && ok);
                        commit_if(qempty, lead_lane && ok && i + lead == end);
                    }
                    ok = ok && wait(pmost + q, np);
                    // the two warps take turns: MMAs of both at once would share the tensor core, end together
                    // and leave it idle while both warpgroups exponentiate
                    if (!chunk_apart(D) && ok && (q == 1 || owed)) ok = wait(turn + (q ^ 1), nt++);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 6; ++ks)  // 16 keys: 16 rows of 128 bytes of each chunk
                        chunk_mma_ts(od, pd + 8u * ks, vl + ks * 128u, id_o, (i >= lead || ks > 0), lead_lane);
                    ok = wait(pfull + q, np);
                    ++np;
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 6; ks < 8; ++ks) chunk_mma_ts(od, pd + 8u * ks, vl + ks * 128u, id_o, 1, lead_lane);
                    if (chunk_apart(D)) {
                        commit_if(pv + q, lead_lane);
                    } else if (more) {
                        mma_s(bl, lead_lane);
                        commit_if(empty + at.stage, lead_lane);
                        commit_if(qempty, lead_lane && i + lead == end);
                    }
                    commit_if(empty + av.stage, lead_lane);
                    commit_if(ofull + q, lead_lane && !more);
                    owed = !chunk_apart(D) && q == 0 && (pair ? i + 1 < n : both);
                    arrive_if(turn + q, lane == 0 && !chunk_apart(D) && (q == 1 || owed));
                    if (more) at.step();
                }
            }
            if (!ok) {
                if (lane == 0) fail(e, (int)(it % LH));
                break;
            }
        }
        // MMAs may still run (after a wait that ran out): they must end before the TMEM is released
        commit_if(done, lead_lane);
        __syncwarp();
        (void)mbar_wait_bounded(done, 0u, a.wait_tries);
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChunkRegsMany));
        // ---------------- softmax: warpgroup q, one row per thread ----------------
        const int q = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;          // TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128u * q, to = tmem + lanes + 256u + (uint32_t)(D * q);
        const uint32_t tp = chunk_apart(D) ? tmem + lanes + 384u + 64u * q : ts;
        unsigned ns = 0, no = 0, nx = 0;  // S tiles, items, paired items so far
        bool ok = true, again = false;    // again: a row of this thread may need chunk_row_again
        for (int r = 0; ok && !*abort_flag; ++r) {
            const unsigned it = chunk_item(r);
            if (it >= n_items) {
                // what hidden values spoilt is mended last, when no role waits for this warp any more: it may take far
                // longer than their bounded waits
                if (__any_sync(FULL, again)) {
                    __syncwarp();  // the rows that other lanes wrote
#pragma unroll 1
                    for (int x = 0; x < r; ++x) {
                        const unsigned xt = chunk_item(x);
                        const ChunkEntry &e = a.entries[xt / LH];
                        if (e.pair && q == 1) continue;
                        const int lh = (int)(xt % LH), lr = lh / a.n_kv, tile = e.pair ? 0 : q;
                        const long long slot = ((long long)e.slot * LH + (long long)lh * e.nsplit + e.split) * 2 + tile;
                        const int row0 = 128 * tile + (warp & 3) * 32;
#pragma unroll 1
                        for (int row = row0; row < min(e.ntok * G, row0 + 32); ++row)
                            chunk_row_again<D>(a, e, lr, lh - lr * a.n_kv, slot, row);
                    }
                }
                break;
            }
            const ChunkEntry *ep = a.entries + it / LH;
            const int lh = (int)(it % LH);
            float m = NEG_INF, l = 0.f;
            int n, rows, limit;
            bool pair;
            {
                const ChunkEntry e = *ep;
                pair = e.pair;
                n = e.kt1 - e.kt0;
                rows = e.ntok * G - (pair ? 0 : 128 * q);     // rows of this warpgroup's tile
                if (rows <= 0) continue;
                const int r0 = pair ? 0 : 128 * q;
                limit = min(e.len, a.causal ? e.first + (r0 + row) / G : e.len);
                const int sure = min(e.len, a.causal ? e.first + r0 / G : e.len);  // seen by every row
                const bool work = (warp & 3) * 32 < rows;     // a warp without rows only keeps the step
                const int step = pair ? 2 : 1;
                for (int i = pair ? q : 0; i < n; i += step) {
                    ok = __all_sync(FULL, mbar_wait_bounded(sfull + q, ns & 1u, a.wait_tries));
                    if (!ok) break;
                    ++ns;
                    if (work) {
                        tc_fence_after();
                        const int key0 = (e.kt0 + i) * 128;
                        ok = chunk_softmax_tile<D>(ts, tp, to, a.c, key0 + 128 > sure, limit - key0, i < step, m, l, lane,
                                                   pmost + q, sfree + q, pv + q, ns & 1u, a.wait_tries);
                        if (!ok) break;
                        tc_fence_before();
                    } else {
                        if (chunk_apart(D)) {
                            arrive_if(sfree + q, lane == 0);
                            // no earlier than a warp with rows could: this arrival belongs to this tile's phase
                            if (i >= step) ok = __all_sync(FULL, mbar_wait_bounded(pv + q, ns & 1u, a.wait_tries));
                            if (!ok) break;
                        }
                        arrive_if(pmost + q, lane == 0);
                    }
                    __syncwarp();
                    arrive_if(pfull + q, lane == 0);
                }
                if (ok && n > (pair ? q : 0)) {
                    ok = __all_sync(FULL, mbar_wait_bounded(ofull + q, no & 1u, a.wait_tries));
                    ++no;
                    tc_fence_after();
                }
                if (!ok) {
                    if (lane == 0) fail(e, lh);
                    break;
                }
            }
            // ---- the result of the item, or its part ----
            const int4 *e4 = reinterpret_cast<const int4 *>(ep);
            const int4 ea = __ldcg(e4), eb = __ldcg(e4 + 1), ec = __ldcg(e4 + 2);
            const int len = ea.w, kt1 = eb.z, nsplit = ec.x;
            float w0 = 1.f, w1 = 0.f;
            if (m == NEG_INF) l = 0.f;                        // no key: what is left of its zero weights goes
            m *= a.c;                                         // the log2 domain (-inf stays)
            if (pair) {
                // the second warpgroup hands its rows' (m, l) over and its O, in the tensor memory lanes of the
                // same rows, which the first joins to its own
                if (q == 1) {
                    ml_x[row] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(xfull);
                    ok = __all_sync(FULL, mbar_wait_bounded(xfree, nx & 1u, a.wait_tries));
                    ++nx;
                    if (ok) continue;
                } else {
                    ok = __all_sync(FULL, mbar_wait_bounded(xfull, nx & 1u, a.wait_tries));
                    ++nx;
                    tc_fence_after();
                    const float2 o = ml_x[row];
                    const float M = fmaxf(m, o.x);
                    w0 = l == 0.f ? 0.f : ex2_approx(m - M);
                    w1 = o.y == 0.f ? 0.f : ex2_approx(o.x - M);
                    l = (l == 0.f ? 0.f : l * w0) + (o.y == 0.f ? 0.f : o.y * w1);
                    m = M;
                }
                if (!ok) {
                    if (lane == 0) fail(*ep, lh);
                    break;
                }
            }
            const int r0 = pair ? 0 : 128 * q;
            const int lr = lh / a.n_kv, g = lh % a.n_kv;
            const int tok = (r0 + row) / G, hd = (r0 + row) % G;
            const bool mine = row < rows;
            const long long trow = ea.y + tok;
            const int head = g * G + hd;
            uint16_t *orow = a.out + lr * a.o_l + trow * a.o_t + head * a.o_h;
            const int tile = pair ? 0 : q;
            const long long slot = ((long long)ec.z * LH + (long long)lh * nsplit + ec.y) * 2 + tile;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            bool odd = false;
            if ((warp & 3) * 32 < rows) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(to + c0, o);
                        tmem_wait32(o);
                        if (pair) {
                            uint32_t o1[32];
                            tmem_ld32(to + D + c0, o1);
                            tmem_wait32(o1);
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float x = w0 == 0.f ? 0.f : __uint_as_float(o[j]) * w0;
                                o[j] = __float_as_uint(w1 == 0.f ? x : fmaf(__uint_as_float(o1[j]), w1, x));
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) odd |= (o[j] & 0x7f800000u) == 0x7f800000u;
                    if (nsplit == 1) {
                        if (mine) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                uint4 w;
                                w.x = pack_bf16(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv);
                                w.y = pack_bf16(__uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
                                w.z = pack_bf16(__uint_as_float(o[j + 4]) * inv, __uint_as_float(o[j + 5]) * inv);
                                w.w = pack_bf16(__uint_as_float(o[j + 6]) * inv, __uint_as_float(o[j + 7]) * inv);
                                *reinterpret_cast<uint4 *>(orow + c0 + j) = w;
                            }
                        }
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(a.part + ((slot * (D / 4) + (c0 + j) / 4) * 128 + row) * 4) =
                                make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), __uint_as_float(o[j + 2]),
                                            __uint_as_float(o[j + 3]));
                    }
                }
            }
            tc_fence_before();
            if (pair) {
                __syncwarp();
                if (lane == 0) mbar_arrive(xfree);
            }
            if (mine) {
                if (nsplit > 1)
                    *reinterpret_cast<float2 *>(a.part_ml + (slot * 128 + row) * 2) = make_float2(m, l);
                else if (a.lse)
                    a.lse[((long long)lr * a.n_tokens + trow) * (a.n_kv * G) + head] =
                        l == 0.f ? NEG_INF : (m + log2f(l)) * 0.6931471805599453f;
            }
            again |= mine && odd && limit < min(len, kt1 * 128);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// Joins the parts of every block that was split, in the order of the keys: out = sum_k 2^(m_k - M) acc_k / sum_k
// 2^(m_k - M) l_k. A programmatic dependent of the attention kernel. In a launch of its own because the last
// CTA of a block did it far slower: one CTA per block against all of them, and code that no CTA had fetched
// yet in the middle of the kernel (18 parts of 8 rows took 18 us).
constexpr int kChunkMergeThreads = 256;
constexpr int kChunkMergeShare = 8;  // CTAs that share the rows of a block's query tile
template <int D>
__global__ void __launch_bounds__(kChunkMergeThreads) tri_chunk_merge_kernel(const ChunkArgs a) {
    const float NEG_INF = __int_as_float(0xff800000);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int G = a.group, LH = a.n_layers * a.n_kv;
    const int units = a.head->n_groups * LH * 2 * kChunkMergeShare;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int share = u % kChunkMergeShare, tile = u / kChunkMergeShare % 2;
        const int lh = u / (2 * kChunkMergeShare) % LH, grp = u / (2 * kChunkMergeShare) / LH;
        const ChunkEntry e = a.merges[grp];
        const int nv = min(128, e.ntok * G - 128 * tile);
        if (nv <= 0) continue;
        const int lr = lh / a.n_kv, g = lh % a.n_kv;
        const long long first = ((long long)e.slot * LH + (long long)lh * e.nsplit) * 2 + tile;
        const float2 *ml0 = reinterpret_cast<const float2 *>(a.part_ml) + first * 128;
        const float4 *part0 = reinterpret_cast<const float4 *>(a.part) + first * (D / 4) * 128;
        const int shift = 32 - __clz(nv - 1);  // rows rounded up to a power of two, so that neighbours read neighbours
        for (int x = share * kChunkMergeThreads + threadIdx.x; x < (D / 4) << shift; x += kChunkMergeShare * kChunkMergeThreads) {
            const int rr = x & ((1 << shift) - 1), c = x >> shift;
            if (rr >= nv) continue;
            float M = NEG_INF, L = 0.f;
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
            for (int k = 0; k < e.nsplit; ++k) M = fmaxf(M, ml0[k * 256 + rr].x);
#pragma unroll 16
            for (int k = 0; k < e.nsplit; ++k) {
                const float2 ml = ml0[k * 256 + rr];
                const float4 v = part0[((long long)k * 2 * (D / 4) + c) * 128 + rr];
                if (ml.y != 0.f) {  // a part that sees no key of the row weighs nothing
                    const float w = ex2_approx(ml.x - M);
                    L = fmaf(ml.y, w, L);
                    A.x = fmaf(v.x, w, A.x);
                    A.y = fmaf(v.y, w, A.y);
                    A.z = fmaf(v.z, w, A.z);
                    A.w = fmaf(v.w, w, A.w);
                }
            }
            const float li = L == 0.f ? 0.f : 1.f / L;
            const int row = 128 * tile + rr, rh = g * G + row % G;
            const long long tok = e.tok0 + row / G;
            uint2 w;
            w.x = pack_bf16(A.x * li, A.y * li);
            w.y = pack_bf16(A.z * li, A.w * li);
            *reinterpret_cast<uint2 *>(a.out + lr * a.o_l + tok * a.o_t + rh * a.o_h + 4 * c) = w;
            if (c == 0 && a.lse)
                a.lse[((long long)lr * a.n_tokens + tok) * (a.n_kv * G) + rh] =
                    L == 0.f ? NEG_INF : (M + log2f(L)) * 0.6931471805599453f;
        }
    }
}

}  // namespace tri

// tri_rope.cuh -- rotary positions, and appending runs of new tokens to a cache, for sm_100a.
//
// The rotation. Band f < r/2 of a row x at position p is the complex number x_a + i x_b, with
// (a, b) = (f, f + r/2) in the half layout and (2f, 2f + 1) in the interleaved one, times
// M e^{i omega_f p}; dims at r and beyond are copied. The inverse divides by it. omega_f and the
// magnitude M are the caller's table (position scalings for long contexts are other tables).
//
// Angles. omega_f is held as turns per position, omega_f / 2 pi, in fp64: the constant, the quotient and pos * turns are
// off by at most 2^-53 each, relative, the fraction of a turn is exact, and only that fraction (at most half a turn)
// is rounded to fp32 for sincospi: at most 2^-23.3 radians plus 3 * 2^-53 omega_f pos. Found against 60 digits for frequencies
// up to 1: 2^-23.3 up to position 2^24, 2^-22.9 up to 2^28, 2^-21.3 at the ends of int32
// (a product in fp32 would lose the whole angle past 2^24 positions of the fastest band). The
// rotation is one fp32 product sum per component, rounded to bf16 once.
//
// Bound: HBM, 4 bytes an element (one read, one write); 3 flops an element. One CTA takes
// `tpc` consecutive tokens of one layer with all their rows (queries, keys and values), so the
// sines of a token are evaluated once per layer and shared through shared memory by all its heads.
// A thread's unit is 32 bytes of a row: the 8 + 8 dims of 8 bands, or 16 copied dims; a thread
// loads kRopeBatch units before the sines are ready, so that the loads, the sines and (for an
// append) the walk from the token to its slot overlap.
//
// Measured on a B200: 2 x 10240 tokens of 32 heads of 128 rotated back in 50 us (6.7 TB/s, the rate of a plain copy);
// 13758 prompt tokens of one layer appended (8 KV heads, their 32 query heads rotated) in 67 us (5.0 TB/s): there a CTA
// is one token and lives for the chain starts -> page -> store. 128 threads and 3 units in flight: 67 us; 256 threads
// with 2, 3, 4: 69 to 87, 74, 72; fewer registers for more CTAs an SM (10, 12, 14 instead of 9): 70, 83, 93. The smallest calls (16 tokens
// rotated, 8 tokens of 36 layers appended): 2 and 6 us on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tri_kernel.cuh"

namespace tri {

constexpr int kRopeThreads = 128;
constexpr int kRopeBatch = 3;      // units a thread has in flight
constexpr int kRopeMaxTokens = 32; // tokens of a CTA, at most
constexpr int kDevBadRange = 6;    // TRI_DEV_BAD_RANGE

struct RowSet {                   // rows [n_layers][n_tokens][heads] of D elements; strides in elements
    const uint16_t *src;
    uint16_t *dst;                // null: the row goes to the cache
    long long src_l, src_t, src_h;
    long long dst_l, dst_t, dst_h;
    int heads;
};

struct RopeArgs {
    RowSet q, k, v;               // heads 0: absent
    const int32_t *pos;           // [n_tokens]
    const double *turns;          // [rot / 2] turns per position
    float mag_c, mag_s;           // factors of the cosine and of the sine (inverse: 1/M and -1/M)
    int rot;                      // rotated dims, a multiple of 16 (0: rows are copied)
    int n_tokens, tpc;
    int units;                    // units of a token: (q + k + v heads) * D / 16
    unsigned units_magic;         // ceil(2^32 / units): idx / units by a high product (idx < 2^16)
    // append only
    uint16_t *K, *V;
    int32_t *P;
    const int32_t *cu;            // [batch + 1] first token of each sequence
    const int32_t *lens;
    int32_t *lens_out;
    const int32_t *block_table;
    int batch, n_kv, page_size, max_pages, n_pages, cap;  // page_size 0: dense
    int32_t *new_len;             // [batch] scratch: the lengths to publish
    unsigned *ticket;             // CTAs that have read the lengths (back to 0 at the end)
    unsigned long long *status;
};

__device__ __forceinline__ float2 rope_pair(float a, float b, float c, float s) {
    return make_float2(fmaf(-b, s, a * c), fmaf(b, c, a * s));
}
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
    unsigned r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where a new token goes, decided by one warp for one token (every lane returns the same):
// seq < 0: nowhere (behind the last sequence, or its sequence is refused).
struct TokenPlace {
    int seq, slot, page;
};

// The sequence of token t by counting the ends at or below it (32 at a time: one load for up to 32
// sequences, against log2(batch) dependent ones of a bisection), with the check that the starts
// ascend within [0, n_tokens]; if they do not, no token has a place. Then the sequence's verdict:
// all its new slots below the capacity and all their pages allocated, so that a refused sequence
// is refused by every CTA alike. Each token looks at all the pages of its run, 32 a load: nothing beside the rows for the
// prompts of the figures above, but it grows with the square of the run (131072 tokens in pages of 16: 1.74 ms, of 64: 0.88).
__device__ __forceinline__ TokenPlace token_place(const RopeArgs &a, int t, int lane, int *bad_code) {
    constexpr unsigned FULL = 0xffffffffu;
    int s = -1, t0 = 0, t1 = 0, len = 0;
    bool sane = true;
    for (int i0 = 0; i0 < a.batch; i0 += 32) {
        const int i = i0 + lane;
        int lo = 0, hi = 0, ln = 0;
        if (i < a.batch) {
            lo = __ldg(a.cu + i);
            hi = __ldg(a.cu + i + 1);
            ln = a.lens[i];  // a plain load: lens_out may be lens
        }
        sane = sane && lo >= 0 && lo <= hi && hi <= a.n_tokens;
        const unsigned past = __ballot_sync(FULL, i < a.batch && hi <= t), all = __ballot_sync(FULL, i < a.batch);
        if (s < 0 && past != all) {
            const int src = __popc(past);
            s = i0 + src;
            t0 = __shfl_sync(FULL, lo, src);
            t1 = __shfl_sync(FULL, hi, src);
            len = __shfl_sync(FULL, ln, src);
        }
    }
    *bad_code = 0;
    TokenPlace r{-1, 0, 0};
    // not ascending, or behind the last sequence, or before the first
    if (!__all_sync(FULL, sane) || s < 0 || t < t0) return r;
    const int n = t1 - t0;
    const long long cap = a.page_size ? (long long)a.page_size * a.max_pages : a.cap;
    if (len < 0 || (long long)len + n > cap) {
        *bad_code = 1;           // TRI_DEV_LEN_GT_CAP
        r.seq = s;
        return r;
    }
    if (a.page_size) {
        const int p0 = len / a.page_size, p1 = (len + n - 1) / a.page_size;
        const int32_t *row = a.block_table + (long long)s * a.max_pages;
        const int slot = len + (t - t0);
        r.page = __ldg(row + slot / a.page_size);
        int bad = 0;
#pragma unroll 4
        for (int p = p0 + lane; p <= p1; p += 32) bad |= (unsigned)__ldg(row + p) >= (unsigned)a.n_pages;
        if (__any_sync(FULL, bad)) {
            *bad_code = 2;       // TRI_DEV_BAD_PAGE
            r.seq = s;
            return r;
        }
        r.slot = slot % a.page_size;
    } else {
        r.page = s;
        r.slot = len + (t - t0);
    }
    r.seq = s;
    return r;
}

template <int D, int LAYOUT, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) tri_rope_kernel(const RopeArgs a) {
    constexpr int UPR = D / 16;  // units of a row
    constexpr int MAXU = D / 16; // rotated units of a row, at most
    __shared__ float4 trig[kRopeMaxTokens * MAXU * 4];  // [token][pair of bands e][unit]: c, s, c, s
    __shared__ TokenPlace place[kRopeMaxTokens];
    __shared__ int last_cta;
    // a programmatic dependent of the launch before it: nothing is read before that has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int layer = blockIdx.y;
    const int t0 = blockIdx.x * a.tpc;
    const int nt = min(a.tpc, a.n_tokens - t0);
    const int total = nt > 0 ? nt * a.units : 0;
    const int ru = a.rot >> 4;   // rotated units of a query or key row

    struct Unit {
        int tok, head, j, set;   // set 0: q, 1: k, 2: v
    };
    auto unit_of = [&](int idx) {
        Unit u;
        u.tok = a.tpc == 1 ? 0 : (int)__umulhi((unsigned)idx, a.units_magic);
        const int rem = idx - u.tok * a.units;
        const int row = rem / UPR;
        u.j = rem % UPR;
        u.set = row < a.q.heads ? 0 : row < a.q.heads + a.k.heads ? 1 : 2;
        u.head = u.set == 0 ? row : u.set == 1 ? row - a.q.heads : row - a.q.heads - a.k.heads;
        return u;
    };
    // element offsets of the unit's two 16-byte halves within its row
    auto halves = [&](const Unit &u, int &oa, int &ob) {
        const bool rotated = u.set < 2 && u.j < ru;
        oa = (LAYOUT == 0 && rotated) ? 8 * u.j : 16 * u.j;
        ob = (LAYOUT == 0 && rotated) ? (a.rot >> 1) + 8 * u.j : 16 * u.j + 8;
        return rotated;
    };
    uint4 xa[kRopeBatch], xb[kRopeBatch];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int idx = base + k * kRopeThreads;
            if (idx < total) {
                const Unit u = unit_of(idx);
                const RowSet &rs = u.set == 0 ? a.q : u.set == 1 ? a.k : a.v;
                const uint16_t *row = rs.src + layer * rs.src_l + (long long)(t0 + u.tok) * rs.src_t + u.head * rs.src_h;
                int oa, ob;
                halves(u, oa, ob);
                xa[k] = *reinterpret_cast<const uint4 *>(row + oa);
                xb[k] = *reinterpret_cast<const uint4 *>(row + ob);
            }
        }
    };
    load(tid);

    if (APPEND) {  // the last warps look the tokens up while the first ones evaluate the sines
        constexpr int NW = kRopeThreads / 32;
        for (int i = NW - 1 - warp; i < nt; i += NW) {
            int code;
            const int t = t0 + i;
            TokenPlace p = token_place(a, t, lane, &code);
            if (lane == 0) {
                if (layer == 0 && p.seq >= 0 && t == __ldg(a.cu + p.seq)) {
                    const int n = __ldg(a.cu + p.seq + 1) - t;
                    const int len = a.lens[p.seq];
                    a.new_len[p.seq] = code ? len : len + n;
                    if (code) record_status(a.status, code, (long long)p.seq * a.n_kv);
                }
                if (code) p.seq = -1;
                place[i] = p;
            }
        }
    }
    for (int i = tid; i < nt * (a.rot >> 1); i += kRopeThreads) {
        const int tok = i / (a.rot >> 1), f = i % (a.rot >> 1);
        const double turn = (double)__ldg(a.pos + t0 + tok) * __ldg(a.turns + f);
        const float part = (float)(2.0 * (turn - rint(turn)));
        float s, c;
        sincospif(part, &s, &c);
        float2 *dst = reinterpret_cast<float2 *>(trig + (tok * 4 + ((f & 7) >> 1)) * MAXU + (f >> 3)) + (f & 1);
        *dst = make_float2(c * a.mag_c, s * a.mag_s);
    }
    __syncthreads();

    for (int base = tid; base < total; base += kRopeBatch * kRopeThreads) {
        if (base != tid) load(base);
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int idx = base + k * kRopeThreads;
            if (idx >= total) continue;
            const Unit u = unit_of(idx);
            TokenPlace p{0, 0, 0};
            if (APPEND) {
                p = place[u.tok];
                if (p.seq < 0) continue;  // left as it was
            }
            int oa, ob;
            if (halves(u, oa, ob)) {
                unsigned wa[4] = {xa[k].x, xa[k].y, xa[k].z, xa[k].w}, wb[4] = {xb[k].x, xb[k].y, xb[k].z, xb[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 cs = trig[(u.tok * 4 + e) * MAXU + u.j];
                    if (LAYOUT == 0) {  // bands 2e, 2e + 1 of the unit: real parts in wa, imaginary in wb
                        const float2 y0 = rope_pair(bf16lo(wa[e]), bf16lo(wb[e]), cs.x, cs.y);
                        const float2 y1 = rope_pair(bf16hi(wa[e]), bf16hi(wb[e]), cs.z, cs.w);
                        wa[e] = pack_bf16(y0.x, y1.x);
                        wb[e] = pack_bf16(y0.y, y1.y);
                    } else {            // band 2e is one word, band 2e + 1 the next
                        unsigned &w0 = e < 2 ? wa[2 * e] : wb[2 * e - 4];
                        unsigned &w1 = e < 2 ? wa[2 * e + 1] : wb[2 * e - 3];
                        const float2 y0 = rope_pair(bf16lo(w0), bf16hi(w0), cs.x, cs.y);
                        const float2 y1 = rope_pair(bf16lo(w1), bf16hi(w1), cs.z, cs.w);
                        w0 = pack_bf16(y0.x, y0.y);
                        w1 = pack_bf16(y1.x, y1.y);
                    }
                }
                xa[k] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
                xb[k] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
            }
            uint16_t *row;
            if (!APPEND || u.set == 0) {
                row = a.q.dst + layer * a.q.dst_l + (long long)(t0 + u.tok) * a.q.dst_t + u.head * a.q.dst_h;
            } else {
                const long long units = a.page_size ? a.n_pages : a.batch;
                const long long rows = a.page_size ? a.page_size : a.cap;
                const long long r = ((layer * units + p.page) * a.n_kv + u.head) * rows + p.slot;
                row = (u.set == 1 ? a.K : a.V) + r * D;
                if (u.set == 1 && u.j == 0) a.P[r] = __ldg(a.pos + t0 + u.tok);
            }
            *reinterpret_cast<uint4 *>(row + oa) = xa[k];
            *reinterpret_cast<uint4 *>(row + ob) = xb[k];
        }
    }

    if (APPEND) {
        // the last CTA to have read the lengths publishes the new ones (lens_out may be lens): every
        // other CTA's reads and its new_len precede its ticket
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            last_cta = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
        }
        __syncthreads();
        if (last_cta) {
            __threadfence();
            if (tid == 0) *a.ticket = 0;
            bool sane = true;
            for (int s = tid; s < a.batch; s += kRopeThreads) {
                const int lo = __ldg(a.cu + s), hi = __ldg(a.cu + s + 1);
                if (lo < 0 || lo > hi || hi > a.n_tokens) {
                    sane = false;
                    record_status(a.status, kDevBadRange, (long long)s * a.n_kv);
                }
            }
            sane = __syncthreads_and(sane);
            for (int s = tid; s < a.batch; s += kRopeThreads) {
                const int n = __ldg(a.cu + s + 1) - __ldg(a.cu + s);
                const int len = a.lens[s];
                int out = len;
                if (sane && n > 0) out = __ldcg(a.new_len + s);
                // a sequence without new tokens was looked at by no CTA
                if (sane && n == 0 && (len < 0 || len > (a.page_size ? (long long)a.page_size * a.max_pages : a.cap)))
                    record_status(a.status, 1, (long long)s * a.n_kv);
                a.lens_out[s] = out;
            }
        }
    }
}

}  // namespace tri

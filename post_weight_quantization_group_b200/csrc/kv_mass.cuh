// kv_mass.cuh -- the attention weight that cached tokens received from chunks
// of new tokens, for head_dim above 128 (below: kv_mass_tc.cuh; decode steps:
// kv_attention.cuh),
//   mass[j, h] += sum over the new tokens' rows r of KV head h that see j
//                 of exp(scale (q_r . kq_j) sk_j - lse_r),
// lse_r being the log-sum-exp that the attention call returned for the row.
//
// The keys stay and the rows go by: a warp holds 16 tokens' K codes as the A
// fragments of S^T = K q^T (mma.sync m16n8k16) and walks over the rows that see
// any of its tokens, so a key's sum is a thread's own and needs no partial
// results.  Every warp reads the rows for itself, through L2 (256 new tokens over 8192,
// 16/8 heads of 256: 346 us).  The result is added
// with one atomic per token and head: a slot that one sequence names gets one
// addend (any order gives the same sum); a page that several sequences share
// gets all of theirs.
#pragma once

#include <stdint.h>

#include "kv_attention.cuh"
#include "kv_paged.cuh"

namespace q4dev {

struct KvMass {
    KvPool pool;
    KvBatch batch;
    KvGeom geom;  // R: tokens of a unit's tile, kKvTile; KT unused
    const uint16_t* q;
    const float* lse;  // [tokens, q_heads]
    float* mass;       // [pages, heads, page_size], pages mass_page apart
    int64_t q_stride, mass_page;
    int q_heads;
    float scale_log2;
    unsigned* status;
};

// Key tiles of a sequence: those that its new tokens may see.
__device__ __forceinline__ int kv_mass_tiles(const KvMass& a, const KvSeq& s, int* lo) {
    if (s.n == 0) {
        *lo = 0;
        return 0;
    }
    const int first = a.geom.window ? max(s.len - s.n + 1 - a.geom.window, 0) : 0;
    *lo = first / kKvTile;
    return max((s.len + kKvTile - 1) / kKvTile - *lo, 0);
}

template <bool BF16>
__global__ void __launch_bounds__(kKvWarps * 32, 1) kv_mass_kernel(const __grid_constant__ KvMass a) {
    constexpr int DP = 256;  // head_dim, padded
    constexpr int U = DP / 64;
    constexpr int NT = kKvWarps * 32;
    __shared__ int64_t s_sums[32];
    __shared__ int64_t s_at;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const KvPool& c = a.pool;
    const int d = c.d;
    grid_launch_dependents();
    grid_dependency_wait();

    // this CTA's range of (sequence, head, key tile)
    int64_t all = 0;
    for (int b0 = 0; b0 < a.batch.seqs; b0 += NT) {
        const int b = b0 + tid;
        int lo;
        int64_t sum;
        const int64_t mine =
            b < a.batch.seqs
                ? static_cast<int64_t>(kv_mass_tiles(a, kv_seq(a.batch, b, a.status), &lo)) * c.heads
                : 0;
        kv_block_scan<NT>(mine, s_sums, &sum);
        all += sum;
    }
    int64_t it = all * blockIdx.x / gridDim.x;
    const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
    if (it == end) return;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch.seqs; b0 += NT) {
        const int b = b0 + tid;
        int lo;
        int64_t sum;
        const int64_t mine =
            b < a.batch.seqs
                ? static_cast<int64_t>(kv_mass_tiles(a, kv_seq(a.batch, b, a.status), &lo)) * c.heads
                : 0;
        const int64_t incl = kv_block_scan<NT>(mine, s_sums, &sum);
        const int64_t x = it - (base + incl - mine);
        if (x >= 0 && x < mine) {
            s_b = b;
            s_at = x;
        }
        base += sum;
    }
    __syncthreads();
    int b = s_b;
    int64_t at = s_at;  // place inside the sequence's tiles: tile-major over heads
    KvSeq seq = kv_seq(a.batch, b, a.status);
    int lo;
    int tiles = kv_mass_tiles(a, seq, &lo);

    for (; it < end; ++it, ++at) {
        while (at >= static_cast<int64_t>(tiles) * c.heads) {
            at = 0;
            seq = kv_seq(a.batch, ++b, a.status);
            tiles = kv_mass_tiles(a, seq, &lo);
        }
        const int h = static_cast<int>(at / tiles);
        const int tile = static_cast<int>(at - static_cast<int64_t>(h) * tiles);
        const int j0 = (lo + tile) * kKvTile + warp * 16;
        if (j0 >= seq.len) continue;

        uint32_t kf[DP / 16][4];
        float sk[2];
        int64_t page[2], row[2];
        bool named[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = j0 + g + 8 * e;
            const bool in = j < seq.len;
            const int32_t entry = in ? kv_entry(a.batch, b, j / c.ps) : 0;
            page[e] = kv_page(c, entry, a.status);
            named[e] = in && entry >= 0 && entry < c.pages;
            row[e] = in ? kv_row(c, h, j % c.ps) : 0;
            const int8_t* p = c.kc + page[e] * c.kc_page + row[e] * d;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint4 x = in && u * 64 + t * 16 < d ? kv_ldg16(p + u * 64 + t * 16)
                                                          : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kf[u * 4 + i][e] = q8_pair<BF16>(xw[i], 0x4140u);
                    kf[u * 4 + i][e + 2] = q8_pair<BF16>(xw[i], 0x4342u);
                }
            }
            sk[e] = in ? cache_value<BF16>(kv_ld(c.ks + page[e] * c.ks_page + row[e])) * a.scale_log2 : 0.f;
        }
        // rows that see any of the 16 tokens: those of new tokens with at >= j0 and,
        // under a window, at - window < j0 + 15
        const int i_lo = max(j0 - (seq.len - seq.n), 0);
        const int i_hi = a.geom.window ? static_cast<int>(min(static_cast<int64_t>(seq.n),
                                             static_cast<int64_t>(j0) + 15 + a.geom.window - (seq.len - seq.n)))
                                       : seq.n;
        const int r_lo = i_lo * a.geom.group, r_hi = i_hi * a.geom.group;
        float sum[2] = {0.f, 0.f};
        for (int r0 = r_lo; r0 < r_hi; r0 += 8) {
            const int r = r0 + g;
            const int tok = r / a.geom.group;
            const uint16_t* qp = a.q + (seq.first + tok) * a.q_stride +
                                 static_cast<int64_t>(h * a.geom.group + r - tok * a.geom.group) * d;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const int e = (s >> 2) * 64 + t * 16 + (s & 3) * 4;
                const uint2 qf = r < r_hi && e < d ? kv_ld(reinterpret_cast<const uint2*>(qp + e))
                                                   : make_uint2(0u, 0u);
                mma_16816<BF16>(x, kf[s], qf.x, qf.y);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = r0 + 2 * t + e;
                if (rr < r_hi) {
                    const int tk = rr / a.geom.group;
                    const float ls = kv_ld(a.lse + (seq.first + tk) * a.q_heads + h * a.geom.group +
                                           rr - tk * a.geom.group) * 1.44269504f;
                    const int last = seq.len - seq.n + tk;
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int j = j0 + g + 8 * f;
                        if (j <= last && (!a.geom.window || j > last - a.geom.window))
                            sum[f] += kv_exp2(fmaf(x[2 * f + e], sk[f], -ls));
                    }
                }
            }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            sum[f] += __shfl_xor_sync(0xFFFFFFFFu, sum[f], 1);
            sum[f] += __shfl_xor_sync(0xFFFFFFFFu, sum[f], 2);
            if (t == 0 && named[f])
                atomicAdd(a.mass + page[f] * a.mass_page + row[f], sum[f]);
        }
    }
}

}  // namespace q4dev

// kv_evict.cuh -- eviction from the paged INT8 cache by accumulated attention
// weight: of each sequence and KV head, the first `sinks` tokens, the last
// `recent` tokens and, of the others, those of the largest mass (ties to the
// lower index) up to `budget` in all are kept, in their order, and moved to
// slots 0 .. of the destination pages.
#pragma once

#include <stdint.h>

#include "kv_paged.cuh"

namespace q4dev {

struct KvEvict {
    KvPool pool;
    KvBatch batch;             // table, lens, seqs; cu and tokens unused
    const int32_t* dst_table;  // [seqs, dst_width]
    int64_t dst_width;
    float* mass;  // [pages, heads, page_size], pages mass_page apart
    int64_t mass_page;
    int budget, recent, sinks;
    int32_t* new_lens;  // [seqs]
    int32_t* src;       // [seqs, heads, budget]: kept tokens in order
    int32_t* len;       // [seqs]: the lengths as the selection saw them
    unsigned* status;
};

__device__ __forceinline__ int kv_evict_len(const KvEvict& a, int b) {
    int len = __ldg(a.batch.lens + b);
    if (len < 0 || len > a.batch.cap) {
        atomicOr(a.status, kStatusBadIndex);
        len = min(max(len, 0), a.batch.cap);
    }
    return len;
}

// A mass as an unsigned number of the same order; NaN counts as the lowest.
__device__ __forceinline__ uint32_t kv_mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = __float_as_uint(m == 0.f ? 0.f : m);  // -0 and 0 are equal
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvThreads = 1024;
constexpr int kEvHeld = 32;  // keys a thread keeps in registers: 32,768 tokens need no second read

// The kept tokens of one (sequence, KV head): the mass of rank K = budget -
// sinks - recent among the others is found digit by digit from the top (four
// histograms of 8 bits), then one pass in order writes the tokens above it and
// the first of those equal to it.
__global__ void __launch_bounds__(kEvThreads) kv_evict_select_kernel(const __grid_constant__ KvEvict a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_digit, s_rank;
    __shared__ uint32_t s_warp[2][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const KvPool& c = a.pool;
    const int b = blockIdx.x / c.heads, h = blockIdx.x - b * c.heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = kv_evict_len(a, b);
    if (h == 0 && tid == 0) a.len[b] = len;
    if (len <= a.budget) return;  // all are kept: the move knows
    int32_t* src = a.src + (static_cast<int64_t>(b) * c.heads + h) * a.budget;

    // the tokens that compete: [lo, hi), K of them stay
    const int lo = a.sinks, hi = len - a.recent;
    const int K = a.budget - a.sinks - a.recent;
    const int n = hi - lo;
    auto key_at = [&](int j) -> uint32_t {
        const int64_t page = kv_page(c, kv_entry(a.batch, b, j / c.ps), a.status);
        return kv_mass_key(__ldg(a.mass + page * a.mass_page + kv_row(c, h, j % c.ps)));
    };
    uint32_t held[kEvHeld];
#pragma unroll
    for (int i = 0; i < kEvHeld; ++i) {
        const int x = i * kEvThreads + tid;
        held[i] = x < n ? key_at(lo + x) : 0u;
    }

    // the K-th largest key: `prefix`, and `rank` of the keys equal to it stay
    uint32_t prefix = 0, mask = 0, rank = static_cast<uint32_t>(K);
    if (K > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            auto add = [&](uint32_t k, bool in) {
                // neighbours often share a digit (tokens nobody looked at): one add for equal ones
                const bool use = in && (k & mask) == prefix;
                const uint32_t dg = use ? (k >> shift) & 255u : 256u;
                const uint32_t peers = __match_any_sync(0xFFFFFFFFu, dg);
                if (use && lane == __ffs(peers) - 1) atomicAdd(&hist[dg], __popc(peers));
            };
#pragma unroll
            for (int i = 0; i < kEvHeld; ++i)
                if (i * kEvThreads < n) add(held[i], i * kEvThreads + tid < n);
            for (int x0 = kEvHeld * kEvThreads; x0 < n; x0 += kEvThreads) {
                const bool in = x0 + tid < n;
                add(in ? key_at(lo + x0 + tid) : 0u, in);
            }
            __syncthreads();
            if (warp == 0) {
                // counts of the digits from the top: lane holds digits 255 - 8 lane - i
                uint32_t cnt[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += cnt[i] = hist[255 - 8 * lane - i];
                uint32_t incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += u;
                }
                uint32_t above = incl - sum;
                if (above < rank && rank <= incl) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < rank && rank <= above + cnt[i]) {
                            s_digit = 255 - 8 * lane - i;
                            s_rank = rank - above;
                        }
                        above += cnt[i];
                    }
                }
            }
            __syncthreads();
            prefix |= s_digit << shift;
            mask |= 255u << shift;
            rank = s_rank;
            __syncthreads();
        }
    }

    // in order: sinks, those above the border and the first `rank` at it, recent
    for (int j = tid; j < a.sinks; j += kEvThreads) src[j] = j;
    for (int j = tid; j < a.recent; j += kEvThreads) src[a.budget - a.recent + j] = hi + j;
    if (K == 0) return;
    uint32_t done = 0, ties = 0;  // written, and border keys seen, in earlier steps
    auto emit = [&](uint32_t k, int x, bool in) {
        const bool gt = in && k > prefix, eq = in && k == prefix;
        const uint32_t bg = __ballot_sync(0xFFFFFFFFu, gt), be = __ballot_sync(0xFFFFFFFFu, eq);
        if (lane == 0) {
            s_warp[0][warp] = __popc(bg);
            s_warp[1][warp] = __popc(be);
        }
        __syncthreads();
        uint32_t g0 = 0, e0 = 0, gall = 0, eall = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const uint32_t u = s_warp[0][w], v = s_warp[1][w];
            if (w < warp) {
                g0 += u;
                e0 += v;
            }
            gall += u;
            eall += v;
        }
        const uint32_t below = (1u << lane) - 1u;
        g0 += __popc(bg & below);
        const uint32_t er = ties + e0 + __popc(be & below);  // border keys before this one
        if (gt || (eq && er < rank))
            src[a.sinks + done + g0 + (min(er, rank) - min(ties, rank))] = lo + x;
        done += gall + min(ties + eall, rank) - min(ties, rank);
        ties += eall;
        __syncthreads();
    };
#pragma unroll
    for (int i = 0; i < kEvHeld; ++i)
        if (i * kEvThreads < n) emit(held[i], i * kEvThreads + tid, i * kEvThreads + tid < n);
    for (int x0 = kEvHeld * kEvThreads; x0 < n; x0 += kEvThreads) {
        const bool in = x0 + tid < n;
        emit(in ? key_at(lo + x0 + tid) : 0u, x0 + tid, in);
    }
}

// The moves read the lengths that the selection wrote down, not seq_lens: that
// may be the array new_lens is written to.
//
// Source token of the i-th kept one.
__device__ __forceinline__ int kv_evict_src(const KvEvict& a, int b, int h, int i, int len) {
    return len <= a.budget ? i
                           : __ldg(a.src + (static_cast<int64_t>(b) * a.pool.heads + h) * a.budget + i);
}
__device__ __forceinline__ int64_t kv_evict_dst_page(const KvEvict& a, int b, int i) {
    return kv_page(a.pool, __ldg(a.dst_table + static_cast<int64_t>(b) * a.dst_width + i / a.pool.ps),
                   a.status);
}

// Destination pages apart from the source pages: every kept row on its own.  A
// team of TS lanes moves a row of K and of V (16 bytes a lane), its scales and
// its mass.
template <int TS>
__global__ void __launch_bounds__(256) kv_evict_copy_kernel(const __grid_constant__ KvEvict a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const KvPool& c = a.pool;
    const int sub = threadIdx.x % TS;
    const int d = c.d;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < a.batch.seqs; b += 256) a.new_lens[b] = min(a.len[b], a.budget);
    for (int u = blockIdx.y; u < a.batch.seqs * c.heads; u += gridDim.y) {
        const int b = u / c.heads, h = u - b * c.heads;
        const int len = a.len[b], kept = min(len, a.budget);
        for (int i = blockIdx.x * (256 / TS) + threadIdx.x / TS; i < kept; i += gridDim.x * (256 / TS)) {
            const int j = kv_evict_src(a, b, h, i, len);
            const int64_t sp = kv_page(c, kv_entry(a.batch, b, j / c.ps), a.status);
            const int64_t dp = kv_evict_dst_page(a, b, i);
            const int64_t sr = kv_row(c, h, j % c.ps), dr = kv_row(c, h, i % c.ps);
            if (sub * 16 < d) {
                const uint4 k = *reinterpret_cast<const uint4*>(c.kc + sp * c.kc_page + sr * d + sub * 16);
                const uint4 v = *reinterpret_cast<const uint4*>(c.vc + sp * c.vc_page + sr * d + sub * 16);
                *reinterpret_cast<uint4*>(c.kc + dp * c.kc_page + dr * d + sub * 16) = k;
                *reinterpret_cast<uint4*>(c.vc + dp * c.vc_page + dr * d + sub * 16) = v;
            }
            if (sub == 0) {
                c.ks[dp * c.ks_page + dr] = c.ks[sp * c.ks_page + sr];
                c.vs[dp * c.vs_page + dr] = c.vs[sp * c.vs_page + sr];
                a.mass[dp * a.mass_page + dr] = a.mass[sp * a.mass_page + sr];
            }
        }
    }
}

// In place: a kept token never moves up (its new index is at most its old
// one), so rows moved in order, a block of 256 read before any of it is
// written, overwrite nothing that is still to be read.  The order binds only
// rows of the same bytes: a CTA takes one (sequence, head) and one 32-byte
// column of the K or the V codes, or the scales and mass (blockIdx.x).
__global__ void __launch_bounds__(256) kv_evict_inplace_kernel(const __grid_constant__ KvEvict a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const KvPool& c = a.pool;
    const int d = c.d, cols = (d + 31) / 32;
    const int piece = blockIdx.x;  // [0, cols): K, [cols, 2 cols): V, 2 cols: scales and mass
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < a.batch.seqs; b += 256) a.new_lens[b] = min(a.len[b], a.budget);
    for (int u = blockIdx.y; u < a.batch.seqs * c.heads; u += gridDim.y) {
        const int b = u / c.heads, h = u - b * c.heads;
        if (a.len[b] <= a.budget) continue;  // everything stays where it is
        const int kept = a.budget;
        for (int i0 = 0; i0 < kept; i0 += 256) {
            const int i = i0 + threadIdx.x;
            int j = i;
            if (i < kept) j = __ldg(a.src + static_cast<int64_t>(u) * a.budget + i);
            const bool move = i < kept && j > i;
            int64_t sp = 0, dp = 0, sr = 0, dr = 0;
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            const bool wide = piece < 2 * cols;
            const int col = (piece < cols ? piece : piece - cols) * 32;
            int8_t* base = piece < cols ? c.kc : c.vc;
            const int64_t stride = piece < cols ? c.kc_page : c.vc_page;
            if (move) {
                sp = kv_page(c, kv_entry(a.batch, b, j / c.ps), a.status);
                dp = kv_evict_dst_page(a, b, i);
                sr = kv_row(c, h, j % c.ps);
                dr = kv_row(c, h, i % c.ps);
                if (wide) {
                    const int8_t* p = base + sp * stride + sr * d + col;
                    x0 = *reinterpret_cast<const uint4*>(p);
                    if (col + 16 < d) x1 = *reinterpret_cast<const uint4*>(p + 16);
                } else {
                    x0.x = c.ks[sp * c.ks_page + sr];
                    x0.y = c.vs[sp * c.vs_page + sr];
                    x0.z = __float_as_uint(a.mass[sp * a.mass_page + sr]);
                }
            }
            __syncthreads();
            if (move) {
                if (wide) {
                    int8_t* p = base + dp * stride + dr * d + col;
                    *reinterpret_cast<uint4*>(p) = x0;
                    if (col + 16 < d) *reinterpret_cast<uint4*>(p + 16) = x1;
                } else {
                    c.ks[dp * c.ks_page + dr] = static_cast<uint16_t>(x0.x);
                    c.vs[dp * c.vs_page + dr] = static_cast<uint16_t>(x0.y);
                    a.mass[dp * a.mass_page + dr] = __uint_as_float(x0.z);
                }
            }
        }
    }
}

}  // namespace q4dev

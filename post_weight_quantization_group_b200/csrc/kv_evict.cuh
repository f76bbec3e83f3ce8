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
    int32_t* src;       // [seqs, heads, budget]: kept tokens in order (none if budget >= batch.cap)
    int32_t* len;       // [seqs]: the lengths as the selection saw them
    unsigned* status;
};

__device__ __forceinline__ int kv_evict_len(const KvEvict& a, int b) {
    int len = kv_ld(a.batch.lens + b);
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
constexpr int kEvHeld = 4;  // times four keys that a thread keeps in registers: 16,384 tokens of a CTA

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The kept tokens of one (sequence, KV head), by a cluster of C CTAs that take
// C consecutive parts of the sequence: the mass of rank K = budget - sinks -
// recent among the tokens that compete is found digit by digit from the top
// (four histograms of 8 bits, added up through distributed shared memory),
// then one pass in order writes the tokens above it and the first of those
// equal to it, each CTA behind what the ones before it wrote.  Bound by
// latency: 8 heads of 32,768 tokens took 100 us in 8 CTAs, and each digit
// 5.5 us when one warp read the 8 CTAs' counts one after another; now 12 us in
// 64 CTAs.  A thread takes four consecutive tokens at a time (one 16-byte load
// where vec allows).
__global__ void __launch_bounds__(kEvThreads) kv_evict_select_kernel(const __grid_constant__ KvEvict a, int C,
                                                                    int vec) {
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t s_total[256];
    __shared__ uint32_t s_digit, s_rank;
    __shared__ uint32_t s_warp[32];
    __shared__ uint32_t s_count[2];  // this CTA's tokens above the border, and at it
    grid_launch_dependents();
    grid_dependency_wait();
    const KvPool& c = a.pool;
    const int unit = blockIdx.x / C, part = blockIdx.x - unit * C;
    const int b = unit / c.heads, h = unit - b * c.heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = kv_evict_len(a, b);
    if (h == 0 && part == 0 && tid == 0) a.len[b] = len;
    if (len <= a.budget) return;  // all are kept: the move knows
    int32_t* src = a.src + static_cast<int64_t>(unit) * a.budget;
    reinterpret_cast<uint32_t*>(hist)[tid] = 0;

    // the tokens that compete: [lo, hi), K of them stay; this CTA's: [j_beg, j_end)
    const int lo = a.sinks, hi = len - a.recent;
    const int K = a.budget - a.sinks - a.recent;
    const int chunk = ((len + C - 1) / C + 3) & ~3;
    const int j_beg = part * chunk, j_end = min(j_beg + chunk, len);
    const int steps = j_end > j_beg ? (j_end - j_beg + 4 * kEvThreads - 1) / (4 * kEvThreads) : 0;
    const int shift = (c.ps & (c.ps - 1)) == 0 ? 31 - __clz(c.ps) : -1;
    const int32_t* trow = a.batch.table + static_cast<int64_t>(b) * a.batch.width;
    const float* mass = a.mass + static_cast<int64_t>(h) * c.ps;
    auto in = [&](int j) { return j >= lo && j < hi && j < j_end; };
    // keys of tokens j .. j + 3 (a multiple of four); 0 where there is none
    auto keys_at = [&](int j, uint32_t (&k)[4]) {
        k[0] = k[1] = k[2] = k[3] = 0u;
        if (j >= j_end) return;
        if (vec) {
            const int e = shift >= 0 ? j >> shift : j / c.ps;
            const int64_t page = kv_page(c, kv_ld(trow + e), a.status);
            const float4 m = kv_ld(reinterpret_cast<const float4*>(mass + page * a.mass_page + (j - e * c.ps)));
            k[0] = kv_mass_key(m.x);
            k[1] = kv_mass_key(m.y);
            k[2] = kv_mass_key(m.z);
            k[3] = kv_mass_key(m.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (j + i >= j_end) break;
                const int e = shift >= 0 ? (j + i) >> shift : (j + i) / c.ps;
                const int64_t page = kv_page(c, kv_ld(trow + e), a.status);
                k[i] = kv_mass_key(kv_ld(mass + page * a.mass_page + (j + i - e * c.ps)));
            }
        }
    };
    auto first_of = [&](int step) { return j_beg + (step * kEvThreads + tid) * 4; };
    uint32_t held[kEvHeld][4];
#pragma unroll
    for (int s = 0; s < kEvHeld; ++s) keys_at(first_of(s), held[s]);
    __syncthreads();  // the histograms are zero

    // the K-th largest key: `prefix`, and `rank` of the keys equal to it stay
    uint32_t prefix = 0, mask = 0, rank = static_cast<uint32_t>(K);
    for (int pass = 0; pass < 4; ++pass) {
        const int sh = 24 - 8 * pass;
        auto add = [&](const uint32_t (&k)[4], int j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool use = in(j + i) && (k[i] & mask) == prefix;
                // many tokens that nobody looked at share a key: one add for a warp of them
                const uint32_t dg = use ? (k[i] >> sh) & 255u : 256u;
                int same;
                __match_all_sync(0xFFFFFFFFu, dg, &same);
                if (same) {
                    if (use && lane == 0) atomicAdd(&hist[pass][dg], 32u);
                } else if (use) {
                    atomicAdd(&hist[pass][dg], 1u);
                }
            }
        };
#pragma unroll
        for (int s = 0; s < kEvHeld; ++s)
            if (s < steps) add(held[s], first_of(s));
        for (int s = kEvHeld; s < steps; ++s) {
            uint32_t k[4];
            keys_at(first_of(s), k);
            add(k, first_of(s));
        }
        if (C > 1) {
            cluster_sync_all();
        } else {
            __syncthreads();
        }
        if (tid < 256) {  // a thread per digit: its loads from the other CTAs are all in flight
            uint32_t v[8], n = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = q < C && q != part ? ld_shared_cluster_u32(mapa_shared(smem_u32(&hist[pass][tid]), q)) : 0u;
#pragma unroll
            for (int q = 0; q < 8; ++q) n += v[q];
            s_total[tid] = n + hist[pass][tid];
        }
        __syncthreads();
        if (warp == 0) {
            // counts of the digits from the top: lane holds digits 255 - 8 lane - i
            uint32_t cnt[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += cnt[i] = s_total[255 - 8 * lane - i];
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += u;
            }
            uint32_t above = incl - sum;
            if (K > 0 && above < rank && rank <= incl) {
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
        if (K > 0) {
            prefix |= s_digit << sh;
            mask |= 255u << sh;
            rank = s_rank;
        }
        __syncthreads();  // the next pass writes s_digit
    }

    // this CTA's tokens above the border and at it, and what stands before them
    auto counts_of = [&](const uint32_t (&k)[4], int j) {  // two counts of at most 4
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in(j + i)) n += k[i] > prefix ? 1u : k[i] == prefix ? 1u << 16 : 0u;
        return n;
    };
    uint32_t done = 0, ties = 0;  // tokens above the border, and at it, in earlier parts and steps
    if (C > 1) {
        uint32_t n = 0, gt = 0, eq = 0;
#pragma unroll
        for (int s = 0; s < kEvHeld; ++s)
            if (s < steps) n += counts_of(held[s], first_of(s));
        gt = n & 0xFFFFu;
        eq = n >> 16;
        for (int s = kEvHeld; s < steps; ++s) {
            uint32_t k[4];
            keys_at(first_of(s), k);
            n = counts_of(k, first_of(s));
            gt += n & 0xFFFFu;
            eq += n >> 16;
        }
        if (tid < 2) s_count[tid] = 0;
        __syncthreads();
        gt = __reduce_add_sync(0xFFFFFFFFu, gt);
        eq = __reduce_add_sync(0xFFFFFFFFu, eq);
        if (lane == 0) {
            atomicAdd(&s_count[0], gt);
            atomicAdd(&s_count[1], eq);
        }
        cluster_sync_all();
        {
            const bool before = lane < part;
            const uint32_t at = mapa_shared(smem_u32(s_count), before ? lane : part);
            const uint32_t x = ld_shared_cluster_u32(at), y = ld_shared_cluster_u32(at + 4);
            done = __reduce_add_sync(0xFFFFFFFFu, before ? x : 0u);
            ties = __reduce_add_sync(0xFFFFFFFFu, before ? y : 0u);
        }
        cluster_sync_all();  // no CTA leaves while another reads its shared memory
    }

    // in order: sinks, those above the border and the first `rank` at it, recent
    if (part == 0) {
        for (int j = tid; j < a.sinks; j += kEvThreads) src[j] = j;
        for (int j = tid; j < a.recent; j += kEvThreads) src[a.budget - a.recent + j] = hi + j;
    }
    if (K == 0) return;
    auto emit = [&](const uint32_t (&k)[4], int j) {
        const uint32_t n = counts_of(k, j);
        uint32_t incl = n;  // two 16-bit sums: a step has 4096 tokens
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        const uint32_t w = s_warp[lane];
        uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
        const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, w);
        before += incl - n;
        uint32_t g = done + (before & 0xFFFFu), e = ties + (before >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!in(j + i)) continue;
            if (k[i] > prefix) {
                src[a.sinks + g + min(e, rank)] = j + i;
                ++g;
            } else if (k[i] == prefix) {
                if (e < rank) src[a.sinks + g + e] = j + i;
                ++e;
            }
        }
        done += all & 0xFFFFu;
        ties += all >> 16;
        __syncthreads();
    };
#pragma unroll
    for (int s = 0; s < kEvHeld; ++s)
        if (s < steps) emit(held[s], first_of(s));
    for (int s = kEvHeld; s < steps; ++s) {
        uint32_t k[4];
        keys_at(first_of(s), k);
        emit(k, first_of(s));
    }
}

// The moves read the lengths that the selection wrote down, not seq_lens: that
// may be the array new_lens is written to.
//
// Source token of the i-th kept one.
__device__ __forceinline__ int kv_evict_src(const KvEvict& a, int b, int h, int i, int len) {
    return len <= a.budget ? i
                           : kv_ld(a.src + (static_cast<int64_t>(b) * a.pool.heads + h) * a.budget + i);
}
// Its page among the destination's, or -1: what has no page is not moved.
__device__ __forceinline__ int64_t kv_evict_dst_page(const KvEvict& a, int b, int i) {
    const int32_t e = kv_ld(a.dst_table + static_cast<int64_t>(b) * a.dst_width + i / a.pool.ps);
    return kv_valid_page(a.pool, e, a.status) ? e : -1;
}

// Destination pages apart from the source pages: every kept row on its own (16
// sequences of 1023 kept rows and 8 heads: 12 us).  A team of TS lanes moves a
// row of K and of V (16 bytes a lane), its scales and its mass.
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
            if (dp < 0) continue;
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
// column of the K or the V codes, or the scales and mass (blockIdx.x).  With the
// selection, 8 heads of 32,768 tokens to 4096: 40 us (into other pages 19).
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
            if (i < kept) j = kv_ld(a.src + static_cast<int64_t>(u) * a.budget + i);
            const int64_t dp = i < kept && j > i ? kv_evict_dst_page(a, b, i) : -1;
            const bool move = dp >= 0;
            int64_t sp = 0, sr = 0, dr = 0;
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            const bool wide = piece < 2 * cols;
            const int col = (piece < cols ? piece : piece - cols) * 32;
            int8_t* base = piece < cols ? c.kc : c.vc;
            const int64_t stride = piece < cols ? c.kc_page : c.vc_page;
            if (move) {
                sp = kv_page(c, kv_entry(a.batch, b, j / c.ps), a.status);
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

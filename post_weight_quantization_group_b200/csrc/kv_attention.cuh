// kv_attention.cuh -- attention of new tokens over the paged INT8 cache, the
// kernel of few rows (decode steps and short chunks).
//
//   S[r, j] = scale * (q_r . kq_j) * sk_j,   visible: at_r - window < j <= at_r,
//   out_r = sum_j 2^(S log2e - m) sv_j vq_j / sum_j 2^(S log2e - m).
//
// The V scale goes into the exponent: with x = S log2e + log2 sv and
// p' = 2^(x - m'), m' a little below the running maximum of x, the numerator is
// sum p' vq and the denominator sum p' / sv.  p' has its maximum at 2^7 to 2^15 whatever
// the V scales are, so it can be rounded to fp16 (2^-11, as fine as the
// codes' own exact fp16 form allows for the product) without leaving fp16's
// range above, and down to 2^-21 of the row's largest p' without leaving its normals;
// below that it is off by up to 2^-32 of the largest (with the maximum near 1 that would be
// 2^-25, and 10^5 tokens far below one other lost 1% of the output).  The
// denominator adds the unrounded fp32 p'.  V scales below 2^-80 are taken as 2^-80 (an
// absolute error below 2^-73): the denominator of 2^30 tokens, at most 2^(15 + 80 + 30),
// stays in fp32.
//
// Bound by the cache bytes read once from HBM.  A warp works alone on blocks
// of 16 tokens: cp.async brings a block's codes into its own ring of shared
// memory kKvStages ahead (128 KB in flight per SM), with no barrier but the
// warp's.  The products are transposed, S^T = K q^T and O^T = V^T P^T
// (mma.sync m16n8k16), so that a thread's fragment of K is 16-byte pieces of
// a row and of V 16-byte pieces of four rows, because the order of head_dim
// inside the dot product and of head_dim in the accumulator's rows is free;
// the ring's pieces are XOR-ed with their row so that both reads are free of
// bank conflicts.  The eight query rows of an MMA's N are one KV head's group
// at a decode step.  P^T comes out of S^T's accumulator by one movmatrix per
// 8 tokens.
//
// Codes become fp16 for both products (5 instructions for 4 codes; bf16 would
// take 8): the queries are scaled by a power of two per row into fp16's range
// first, which is exact for every element above 2^-31 of the row's largest,
// and below that within 2^-40 of it: finer than the fp32 sums.
//
// Measured (B200, 64 query heads over 8 of 128): one token over 131,071, 65 us
// = 4.2 TB/s, of which the loop takes 45 (6.0 TB/s); 32 ragged sequences of up
// to 8192, 66 us; one of 1001 (32 heads), 9.5 us.
//
// Work split: kv_paged.cuh (equal ranges of 128-token tiles over the CTAs; a
// warp takes 16 tokens of each tile).  The warps of a CTA keep their own
// maxima and sums and are joined at the end of a segment; a unit that
// several CTAs share goes through the workspace, and the CTA that arrives
// last on the unit's counter adds the parts in CTA order and re-zeroes the
// counter, so the result does not depend on timing.
#pragma once

#include <stdint.h>

#include "kv_paged.cuh"

namespace q4dev {

struct KvAttn {
    KvPool pool;
    KvBatch batch;
    KvGeom geom;
    const uint16_t* q;
    uint16_t* out;
    float* lse;  // [tokens, q_heads]: written (may be null) by attention, read by mass
    float* mass;  // [pages, heads, page_size], pages mass_page apart
    int64_t mass_page;
    int64_t q_stride, out_stride;
    int q_heads;
    float scale_log2;  // scale * log2(e)
    float* part;       // partial slots, two per CTA: m [R], l [R], O [R, DP]
    unsigned* count;   // one per CTA
    unsigned* status;
    int fill;  // of the rows that no sequence names: 1: zeros to out, 2: -inf to lse
};

constexpr int kKvWarps = 8;
constexpr int kKvTile = 16 * kKvWarps;  // tokens of a tile
constexpr float kKvNone = -1e30f;       // the maximum of nothing: finite, so that m - m' is not NaN
// A warp takes another m' only when an x passes it by more than kKvTop: p' stays
// below 2^15, inside fp16, and most blocks skip the rescale.  The new m' lies kKvBelow under
// that x, so a row's largest p' is 2^7 or more, and that of the token that set m',
// often by far the largest, is 2^7 itself and loses nothing to the rounding.  (A whole m',
// which makes rescales exact, rounds that one too: fp16 outputs of 1001 tokens were
// 3.0e-4 off fp64 instead of 2.1e-4.)
constexpr float kKvTop = 15.0f, kKvBelow = 7.0f;
__device__ __forceinline__ float kv_new_max(float m, float x) { return x > m + kKvTop ? x - kKvBelow : m; }

__device__ __forceinline__ uint4 kv_ldg16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ float kv_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t kv_pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// Two codes of a word whose bytes have had 0x80 added, bytes 0, 1 or 2, 3, as exact fp16:
// a byte under 0x64 is 1024 + (code + 128).
__device__ __forceinline__ uint32_t kv_codes01(uint32_t w) {
    return sub2<false>(prmt(w, 0x64u, 0x4140u), 0x64806480u);
}
__device__ __forceinline__ uint32_t kv_codes23(uint32_t w) {
    return sub2<false>(prmt(w, 0x64u, 0x4342u), 0x64806480u);
}
__device__ __forceinline__ uint32_t kv_transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// What a cached token's V scale contributes: log2 to the exponent, 1 / sv to the denominator.
struct KvVScale {
    float lg, inv;
};
__device__ __forceinline__ KvVScale kv_vscale(float sv) {
    KvVScale r;
    const float c = fmaxf(sv, 0x1p-80f);  // a NaN becomes 2^-80 here ...
    r.lg = sv == sv ? __log2f(c) : sv;         // ... and stays in the exponent, where masks drop it
    // within 1 ulp; c is normal and, as 1/127 of a finite value, below 2^121
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(c));
    return r;
}

// A warp's ring in shared memory: stages of a block's K and V codes, then of its
// tokens' scales (sk, log2 sv, 1 / sv).  For the mass: K alone, with sk and the
// tokens' places in the mass (64 bits each).
template <int DP, bool MASS>
struct KvRing {
    static constexpr int stages = DP == 64 ? (MASS ? 6 : 5) : (MASS ? 4 : 3);
    static constexpr uint32_t half = 16 * DP;  // bytes of a block's K, of its V
    static constexpr uint32_t stage = (MASS ? 1 : 2) * half;
    static constexpr uint32_t off_sc = stages * stage;
    static constexpr uint32_t total = off_sc + stages * 3 * 16 * 4;
    static constexpr int lanes = DP / 16;        // lanes of a row, 16 bytes each
    static constexpr int rows = 32 / lanes;      // rows of one cp.async of the warp
    static constexpr int copies = 16 / rows;
    // Byte offset of 16-byte piece p of token r.  K is read by lanes (two rows, four
    // pieces) at a time, V by (four even or odd rows, two pieces).
    static __device__ __forceinline__ uint32_t k_at(int r, int p) {
        return DP == 64 ? r * 64 + p * 16 : r * DP + ((p ^ ((r & 1) << 2)) << 4);
    }
    static __device__ __forceinline__ uint32_t v_at(int r, int p) {
        if constexpr (DP == 64)
            return ((r & ~3) | ((r & 1) << 1) | ((r >> 1) & 1)) * 64 + ((p ^ ((r >> 1) & 2)) << 4);
        else
            return r * DP + ((p ^ (r & 6)) << 4);
    }
};

__device__ __forceinline__ void kv_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void kv_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void kv_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The rows of q that no sequence names, after kv_locate: before the first one's and behind
// the last one's.
template <int NT>
__device__ __forceinline__ void kv_fill_unnamed(const KvAttn& a, const KvLocateShared& sh) {
    if (!a.fill) return;
    const int64_t chunks = static_cast<int64_t>(a.q_heads) * a.pool.d / 8;  // of 16 bytes
    const int64_t lo = sh.named[0], hi = max(sh.named[1], lo);
    for (int64_t u = blockIdx.x; u < a.batch.tokens - (hi - lo); u += gridDim.x) {
        const int64_t row = u < lo ? u : u + (hi - lo);
        if (a.fill & 1)
            for (int64_t i = threadIdx.x; i < chunks; i += NT)
                reinterpret_cast<uint4*>(a.out + row * a.out_stride)[i] = make_uint4(0u, 0u, 0u, 0u);
        if ((a.fill & 2) && a.lse)
            for (int i = threadIdx.x; i < a.q_heads; i += NT) a.lse[row * a.q_heads + i] = -INFINITY;
    }
}

// DP: head_dim padded to 64, 128 or 256.  NR: blocks of 8 rows (R = 8 NR).
// MASS: not attention but the weight that each token receives, given the rows'
// log-sum-exps: mass[j, h] += sum over the rows r that see j of exp(S[r, j] - lse_r).
// S^T has a token's rows in one quad, so its sum is a thread's and two
// shuffles; it is added with one atomic, the token's only one where the rows
// fit one unit and no other sequence shares the page (any order then gives the
// same sum).
// P16: the page size is a multiple of 16, so a block of 16 tokens is in one
// page and its rows follow one another; else every row looks up its own page.
template <bool BF16, int DP, int NR, bool P16, bool MASS>
__global__ void __launch_bounds__(kKvWarps * 32, DP * NR > 128 ? 1 : 2)
    kv_attention_kernel(const __grid_constant__ KvAttn a) {
    constexpr int R = 8 * NR;
    constexpr int U = DP / 64, MT = DP / 16;
    constexpr int ROW = DP + 8;  // padded row of the join buffer (floats): rows 2t apart by 16 banks
    using Ring = KvRing<DP, MASS>;
    extern __shared__ __align__(128) float smem[];
    // the warps' rings; at the end of a segment the same memory joins their parts
    float* s_o = smem;                                // [warps][R][ROW]
    float* s_m = smem + kKvWarps * R * ROW;           // [warps][R]
    float* s_l = s_m + kKvWarps * R;                  // [warps][R]
    __shared__ KvLocateShared s_loc;
    __shared__ unsigned s_last;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const KvPool& c = a.pool;
    const int d = c.d;
    grid_launch_dependents();
    grid_dependency_wait();

    int64_t T, P, beg, end;
    KvPlace w;
    kv_locate<kKvWarps * 32>(a.batch, a.geom, blockIdx.x, gridDim.x, 1, a.status, &s_loc, &T, &P,
                             &beg, &end, &w);
    if constexpr (!MASS) kv_fill_unnamed<kKvWarps * 32>(a, s_loc);
    if (beg == end) return;
    KvSeq seq = kv_seq(a.batch, w.b, a.status);
    const int shift = (c.ps & (c.ps - 1)) == 0 ? 31 - __clz(c.ps) : -1;
    auto page_index = [&](int j) { return shift >= 0 ? j >> shift : j / c.ps; };
    const uint32_t ring = smem_u32(smem) + warp * Ring::total;
    const bool same = c.kc_page == c.vc_page && c.ks_page == c.vs_page;
    // this lane's part of a copy: row crow (and every Ring::rows after it), piece cp; pieces
    // beyond head_dim repeat piece 0: their K meets zeros of q, their V is not stored
    const int crow = lane / Ring::lanes, cp = lane % Ring::lanes;
    const int ccol = cp * 16 < d ? cp * 16 : 0;

    int64_t it = beg;
    while (it < end) {
        int tile_lo;
        const int ntiles = kv_tiles(a.geom, seq, w.rt, &tile_lo);
        const int64_t unit_beg = it - w.tile, unit_end = unit_beg + ntiles;
        const int nseg = static_cast<int>(min(unit_end, end) - it);
        const int rows = seq.n * a.geom.group;
        const int row0 = w.rt * R;

        int at[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + n * 8 + 2 * t + e;
                at[n][e] = r < rows ? seq.len - seq.n + r / a.geom.group : -1;
            }
        const int at_min = seq.len - seq.n + row0 / a.geom.group;
        const int at_max = seq.len - seq.n + (min(row0 + R, rows) - 1) / a.geom.group;

        float o[MT][NR][4], m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n][0] = m[n][1] = kKvNone;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        }

        const int32_t* trow = a.batch.table + static_cast<int64_t>(w.b) * a.batch.width;
        auto entry_of = [&](int j0) -> int32_t {
            return P16 && j0 < seq.len ? kv_ld(trow + page_index(j0)) : 0;
        };
        // Element offsets of a token's row (of its scale; times d, of its codes) in the pools.
        struct Place {
            int64_t kc, vc, ks, vs;  // vs: of the mass, where that is asked for
        };
        const uint32_t hrow = static_cast<uint32_t>(w.h) * c.ps;
        auto place = [&](int j, int32_t entry) {
            const uint64_t page = static_cast<uint32_t>(kv_page(c, entry, a.status));
            const uint32_t row = hrow + static_cast<uint32_t>(j - page_index(j) * c.ps);
            Place p;
            p.kc = page * c.kc_page + static_cast<uint64_t>(row) * d;
            p.ks = page * c.ks_page + row;
            p.vc = p.kc;
            p.vs = p.ks;
            if constexpr (MASS) {
                // -1: not added
                p.vs = entry >= 0 && entry < c.pages ? static_cast<int64_t>(page * a.mass_page + row) : -1;
            } else if (!same) {
                p.vc = page * c.vc_page + static_cast<uint64_t>(row) * d;
                p.vs = page * c.vs_page + row;
            }
            return p;
        };

        const int jw = (tile_lo + w.tile) * kKvTile + warp * 16;  // block 0's first token
        uint32_t put = 0, put_sc = 0;  // stage of block i, of block i - 1
        uint16_t sc = 0;  // a scale of the block issued last: of K in lanes 0-15, of V in 16-31
        int64_t sc_mass = 0;  // or, in 16-31, a token's place in the mass
        int32_t entry_next = entry_of(jw);
        // starts the copy of block i of the segment into its stage and the load of its
        // scales, and stores those of block i - 1, which have had a step to arrive
        auto issue = [&](int i) {
            const int j0 = jw + i * kKvTile;
            const bool on = i < nseg && j0 < seq.len;  // else nothing of the block is visible
            const int last = min(15, seq.len - 1 - j0), rs = min(lane & 15, last);
            const uint32_t st = ring + put * Ring::stage;
            Place b{0, 0, 0, 0};
            if (on) {
                if constexpr (P16) {
                    b = place(j0, entry_next);
                    const int8_t* kp = c.kc + b.kc + ccol;
                    const int8_t* vp = c.vc + b.vc + ccol;
                    if (last == 15) {
                        kp += crow * d;
                        vp += crow * d;
#pragma unroll
                        for (int x = 0; x < Ring::copies; ++x) {
                            const int r = crow | (x * Ring::rows);
                            kv_cp16(st + Ring::k_at(r, cp), kp);
                            if constexpr (!MASS) kv_cp16(st + Ring::half + Ring::v_at(r, cp), vp);
                            kp += Ring::rows * d;
                            vp += Ring::rows * d;
                        }
                    } else {  // tokens behind the last one repeat it; the masks drop them
#pragma unroll 1
                        for (int x = 0; x < Ring::copies; ++x) {
                            const int r = crow | (x * Ring::rows), rd = min(r, last) * d;
                            kv_cp16(st + Ring::k_at(r, cp), kp + rd);
                            if constexpr (!MASS) kv_cp16(st + Ring::half + Ring::v_at(r, cp), vp + rd);
                        }
                    }
                    b.ks += rs;
                    if (!MASS || b.vs >= 0) b.vs += rs;
                } else {
#pragma unroll 1
                    for (int x = 0; x < Ring::copies; ++x) {
                        const int r = crow + x * Ring::rows, j = j0 + min(r, last);
                        b = place(j, kv_ld(trow + page_index(j)));
                        kv_cp16(st + Ring::k_at(r, cp), c.kc + b.kc + ccol);
                        if constexpr (!MASS) kv_cp16(st + Ring::half + Ring::v_at(r, cp), c.vc + b.vc + ccol);
                    }
                    b = place(j0 + rs, kv_ld(trow + page_index(j0 + rs)));
                }
            }
            kv_cp_commit();
            if (i >= 1 && i <= nseg) {
                const uint32_t at = ring + Ring::off_sc + put_sc * 192u + (lane & 15) * 4u;
                const float v = cache_value<BF16>(sc);
                if (lane < 16) {
                    sts32(at, __float_as_uint(v * a.scale_log2));
                } else if constexpr (MASS) {
                    sts64(at + (lane & 15) * 4u + 64u, static_cast<uint64_t>(sc_mass));
                } else {
                    const KvVScale x = kv_vscale(v);
                    sts32(at + 64u, __float_as_uint(x.lg));
                    sts32(at + 128u, __float_as_uint(x.inv));
                }
            }
            sc = 0;
            if constexpr (MASS) {
                sc_mass = b.vs;
                if (on && lane < 16) sc = kv_ld(c.ks + b.ks);
            } else {
                if (on) sc = kv_ld(lane < 16 ? c.ks + b.ks : c.vs + b.vs);
            }
            if (i + 1 < nseg) entry_next = entry_of(j0 + kKvTile);
            put_sc = put;
            put = put + 1 == Ring::stages ? 0 : put + 1;
        };
#pragma unroll 1
        for (int i = 0; i < Ring::stages - 1; ++i) issue(i);
        // query fragments in fp16, scaled by 2^-ex of their row, and the last visible token
        // of this thread's rows
        uint2 qf[NR][DP / 16];
        float undo[NR][2];  // 2^ex of rows 2 t, 2 t + 1
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int r = row0 + n * 8 + g;
            const int tok = r / a.geom.group;
            const int hd = r - tok * a.geom.group;
            const uint16_t* qp = a.q + (seq.first + tok) * a.q_stride +
                                 static_cast<int64_t>(w.h * a.geom.group + hd) * d;
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const int e = (s >> 2) * 64 + t * 16 + (s & 3) * 4;
                qf[n][s] = r < rows && e < d ? *reinterpret_cast<const uint2*>(qp + e)
                                             : make_uint2(0u, 0u);
            }
            float scale = 1.f;
            if constexpr (BF16) {
                // bits of a bf16 magnitude order like the magnitudes
                uint32_t mx = 0;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    mx = max(max(mx, max(qf[n][s].x & 0x7FFFu, (qf[n][s].x >> 16) & 0x7FFFu)),
                             max(qf[n][s].y & 0x7FFFu, (qf[n][s].y >> 16) & 0x7FFFu));
                mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                // the largest element to [2^14, 2^15); scales stay normal (an element of 2^127 or
                // of 2^-120 is still in range), and infinities and NaN stay themselves
                const int ex = min(max(static_cast<int>(mx >> 7) - 127 - 14, -120), 120);
                const float down = __int_as_float((127 - ex) << 23);
                scale = __int_as_float((127 + ex) << 23);
                auto to_half = [&](uint32_t v) {
                    return kv_pack_f16(cache_value<true>(static_cast<uint16_t>(v & 0xFFFFu)) * down,
                                       cache_value<true>(static_cast<uint16_t>(v >> 16)) * down);
                };
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    qf[n][s] = make_uint2(to_half(qf[n][s].x), to_half(qf[n][s].y));
            }
            undo[n][0] = __shfl_sync(0xFFFFFFFFu, scale, 8 * t);      // row 2 t's quad
            undo[n][1] = __shfl_sync(0xFFFFFFFFu, scale, 8 * t + 4);  // row 2 t + 1's
        }
        float ls[NR][2];  // the rows' log-sum-exps in log2
        if constexpr (MASS) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = row0 + n * 8 + 2 * t + e, tok = r / a.geom.group;
                    ls[n][e] = r < rows ? 1.44269504f * kv_ld(a.lse + (seq.first + tok) * a.q_heads +
                                                              w.h * a.geom.group + r - tok * a.geom.group)
                                        : 0.f;
                }
        }
        uint32_t take = 0;  // stage of block s
#pragma unroll 1
        for (int s = 0; s < nseg; ++s) {
            const int j0 = jw + s * kKvTile;
            kv_cp_wait<Ring::stages - 2>();
            __syncwarp();  // every lane's copies of block s are there, and block s - 1 is done with
            issue(s + Ring::stages - 1);
            const uint32_t st = ring + take * Ring::stage;
            const uint32_t scs = ring + Ring::off_sc + take * 192u + g * 4u;
            take = take + 1 == Ring::stages ? 0 : take + 1;
            // nothing of this block is visible to any row: at the ends of a unit's range
            if (j0 > at_max || (a.geom.window && j0 + 15 <= at_min - a.geom.window)) continue;

            // S^T = K q^T
            float x[NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint4 ka = lds128(st + Ring::k_at(g, u * 4 + t));
                const uint4 kb = lds128(st + Ring::k_at(g + 8, u * 4 + t));
                const uint32_t k0[4] = {ka.x ^ 0x80808080u, ka.y ^ 0x80808080u, ka.z ^ 0x80808080u,
                                        ka.w ^ 0x80808080u};
                const uint32_t k1[4] = {kb.x ^ 0x80808080u, kb.y ^ 0x80808080u, kb.z ^ 0x80808080u,
                                        kb.w ^ 0x80808080u};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t af[4] = {kv_codes01(k0[i]), kv_codes01(k1[i]), kv_codes23(k0[i]),
                                            kv_codes23(k1[i])};
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        mma_16816<false>(x[n], af, qf[n][u * 4 + i].x, qf[n][u * 4 + i].y);
                }
            }
            // scores in log2, with the V scale; masks
            const float sk0 = __uint_as_float(lds32(scs)), sk1 = __uint_as_float(lds32(scs + 32u));
            const bool open = j0 + 15 <= at_min && (!a.geom.window || j0 > at_max - a.geom.window);
            if constexpr (MASS) {
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + g + 8 * (e >> 1), top = at[n][e & 1];
                        const float y = fmaf(x[n][e], (e >> 1 ? sk1 : sk0) * undo[n][e & 1], -ls[n][e & 1]);
                        // a row of the tile that is none sees nothing (its top is -1)
                        const bool see = (open && top >= 0) ||
                                         (j <= top && (!a.geom.window || j > top - a.geom.window));
                        sum[e >> 1] += see ? kv_exp2(y) : 0.f;
                    }
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    sum[f] += __shfl_xor_sync(0xFFFFFFFFu, sum[f], 1);
                    sum[f] += __shfl_xor_sync(0xFFFFFFFFu, sum[f], 2);
                    if (t == 0 && j0 + g + 8 * f < seq.len) {
                        const uint2 o = lds64(scs + g * 4u + 64u + 64u * f);
                        const int64_t to = static_cast<int64_t>((static_cast<uint64_t>(o.y) << 32) | o.x);
                        if (to >= 0) atomicAdd(a.mass + to, sum[f]);
                    }
                }
                continue;
            }
            const KvVScale v0{__uint_as_float(lds32(scs + 64u)), __uint_as_float(lds32(scs + 128u))};
            const KvVScale v1{__uint_as_float(lds32(scs + 96u)), __uint_as_float(lds32(scs + 160u))};
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                x[n][0] = fmaf(x[n][0], sk0 * undo[n][0], v0.lg);
                x[n][1] = fmaf(x[n][1], sk0 * undo[n][1], v0.lg);
                x[n][2] = fmaf(x[n][2], sk1 * undo[n][0], v1.lg);
                x[n][3] = fmaf(x[n][3], sk1 * undo[n][1], v1.lg);
                if (!open) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + g + 8 * (e >> 1);
                        const bool see = j <= at[n][e & 1] &&
                                         (!a.geom.window || j > at[n][e & 1] - a.geom.window);
                        if (!see) x[n][e] = -INFINITY;
                    }
                }
                grow |= fmaxf(x[n][0], x[n][2]) > m[n][0] + kKvTop ||
                        fmaxf(x[n][1], x[n][3]) > m[n][1] + kKvTop;
            }
            if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[n][e], x[n][e + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                        // a row of its own: what other rows of the warp do leaves it alone
                        mx = kv_new_max(m[n][e], mx);
                        f[e] = kv_exp2(m[n][e] - mx);
                        m[n][e] = mx;
                        l[n][e] *= f[e];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[i][n][0] *= f[0];
                        o[i][n][1] *= f[1];
                        o[i][n][2] *= f[0];
                        o[i][n][3] *= f[1];
                    }
                }
            }
            uint32_t pb[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float p0 = kv_exp2(x[n][0] - m[n][0]), p1 = kv_exp2(x[n][1] - m[n][1]);
                const float p2 = kv_exp2(x[n][2] - m[n][0]), p3 = kv_exp2(x[n][3] - m[n][1]);
                l[n][0] = fmaf(p2, v1.inv, fmaf(p0, v0.inv, l[n][0]));
                l[n][1] = fmaf(p3, v1.inv, fmaf(p1, v0.inv, l[n][1]));
                pb[n][0] = kv_transpose8x8(kv_pack_f16(p0, p1));
                pb[n][1] = kv_transpose8x8(kv_pack_f16(p2, p3));
            }
            // O^T += V^T P^T
#pragma unroll
            for (int u = 0; u < (DP == 64 ? 1 : DP / 128); ++u) {
                uint32_t vw[4][4];  // this thread's pieces of rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 2 * t + (e & 1) + 8 * (e >> 1);
                    if constexpr (DP == 64) {
                        const uint2 y = lds64(st + Ring::half + Ring::v_at(r, g >> 1) + (g & 1) * 8);
                        vw[e][0] = y.x;
                        vw[e][1] = y.y;
                    } else {
                        const uint4 y = lds128(st + Ring::half + Ring::v_at(r, u * 8 + g));
                        vw[e][0] = y.x;
                        vw[e][1] = y.y;
                        vw[e][2] = y.z;
                        vw[e][3] = y.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < (DP == 64 ? 2 : 4); ++i) {
                    const uint32_t y0 = vw[0][i] ^ 0x80808080u, y1 = vw[1][i] ^ 0x80808080u;
                    const uint32_t y2 = vw[2][i] ^ 0x80808080u, y3 = vw[3][i] ^ 0x80808080u;
#pragma unroll
                    for (int hw = 0; hw < 2; ++hw) {
                        const uint32_t sel = hw ? 0x7362u : 0x5140u;  // bytes 2, 3 or 0, 1 of both rows
                        const uint32_t a01 = prmt(y0, y1, sel), a23 = prmt(y2, y3, sel);
                        const uint32_t af[4] = {kv_codes01(a01), kv_codes23(a01), kv_codes01(a23),
                                                kv_codes23(a23)};
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            mma_16816<false>(o[u * 8 + 2 * i + hw][n], af, pb[n][0], pb[n][1]);
                    }
                }
            }
        }

        if constexpr (MASS) {
            __syncwarp();  // the ring is done with
            it += nseg + a.geom.lead;
            if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
            continue;
        }
        // ------------------------------------------- join of the CTA's warps
        // Element (row, pos) of O: pos = 16 i + 2 g + e for the accumulator tile i, so
        // that a warp's stores and the join's loads are free of bank conflicts.
        __syncthreads();  // the rings are done with
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], off);
                const int r = n * 8 + 2 * t + e;
                if (g == 0) {
                    s_m[warp * R + r] = m[n][e];
                    s_l[warp * R + r] = l[n][e];
                }
                float* dst = s_o + (warp * R + r) * ROW + 2 * g;
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][n][e], o[i][n][e + 2]);
            }
        __syncthreads();
        const bool whole = it == unit_beg && it + nseg == unit_end;
        const int64_t first_cta = whole ? 0 : kv_owner(unit_beg, T, P);
        const int64_t last_cta = whole ? 0 : kv_owner(unit_end - 1, T, P);
        constexpr int64_t SLOT = static_cast<int64_t>(R) * (DP + 2);
        float* slot = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (it == beg ? 0 : 1)) * SLOT;

        // writes the row's pair of elements at pos (two head_dim values)
        auto finish = [&](int r, int pos, float mm, float ll, float2 v) {
            const int rr = row0 + r;
            if (rr >= rows) return;
            const int tok = rr / a.geom.group;
            const int head = w.h * a.geom.group + rr - tok * a.geom.group;
            const int i = pos >> 4, gg = (pos & 15) >> 1;
            const int dd = DP == 64 ? gg * 8 + 2 * i : (i >> 3) * 128 + gg * 16 + 2 * (i & 7);
            const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : ll == 0.f ? 0.f : ll;
            if (dd < d) {
                const uint32_t pair = static_cast<uint32_t>(cache_bits<BF16>(v.x * inv)) |
                                      (static_cast<uint32_t>(cache_bits<BF16>(v.y * inv)) << 16);
                *reinterpret_cast<uint32_t*>(a.out + (seq.first + tok) * a.out_stride +
                                             static_cast<int64_t>(head) * d + dd) = pair;
            }
            if (pos == 0 && a.lse)
                a.lse[(seq.first + tok) * a.q_heads + head] =
                    ll == 0.f ? -INFINITY : 0.69314718f * (mm + __log2f(ll));
        };

        for (int x = tid; x < R * DP / 2; x += kKvWarps * 32) {
            const int r = x / (DP / 2), pos = (x % (DP / 2)) * 2;
            float mm = s_m[r];
#pragma unroll
            for (int ww = 1; ww < kKvWarps; ++ww) mm = fmaxf(mm, s_m[ww * R + r]);
            float ll = 0.f;
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int ww = 0; ww < kKvWarps; ++ww) {
                const float f = kv_exp2(s_m[ww * R + r] - mm);
                const float2 u = *reinterpret_cast<const float2*>(s_o + (ww * R + r) * ROW + pos);
                ll = fmaf(f, s_l[ww * R + r], ll);
                v.x = fmaf(f, u.x, v.x);
                v.y = fmaf(f, u.y, v.y);
            }
            if (whole) {
                finish(r, pos, mm, ll, v);
            } else {
                if (pos == 0) {
                    __stcg(slot + r, mm);
                    __stcg(slot + R + r, ll);
                }
                __stcg(reinterpret_cast<float2*>(slot + 2 * R + r * DP + pos), v);
            }
        }
        __syncthreads();  // the join buffer is free again; the slot is written
        if (!whole) {
            if (tid == 0) {
                const unsigned prev = kv_arrive(a.count + first_cta);
                s_last = prev == static_cast<unsigned>(last_cta - first_cta);
                if (s_last) a.count[first_cta] = 0u;  // zero again for the next call
            }
            __syncthreads();
            if (s_last) {
                // The parts' weights 2^(m_p - m) first, a warp per row, then the sum: all its
                // loads are independent.  (One running rescale over the 37 parts of a 131K-token
                // unit took 28 us, a load's latency for each part; this takes 3.)
                __threadfence();
                const int n = static_cast<int>(last_cta - first_cta) + 1;
                // only the first of the unit's CTAs can have begun before it
                const int first_slot = T * first_cta / P >= unit_beg - a.geom.lead ? 0 : 1;
                auto slot_of = [&](int i) -> const float* {
                    return a.part + (2 * (first_cta + i) + (i == 0 ? first_slot : 0)) * SLOT;
                };
                float* s_f = smem;            // [n][R]: m, then weights; n <= CTAs of the device
                float* s_n = smem + n * R;    // [R] m, [R] l
                for (int r = warp; r < R; r += kKvWarps) {
                    float mm = kKvNone, ll = 0.f;
                    for (int i = lane; i < n; i += 32) {
                        const float x = __ldcg(slot_of(i) + r);
                        s_f[i * R + r] = x;
                        mm = fmaxf(mm, x);
                    }
#pragma unroll
                    for (int o2 = 16; o2 >= 1; o2 >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o2));
                    for (int i = lane; i < n; i += 32) {
                        const float f = kv_exp2(s_f[i * R + r] - mm);
                        s_f[i * R + r] = f;
                        ll = fmaf(f, __ldcg(slot_of(i) + R + r), ll);
                    }
#pragma unroll
                    for (int o2 = 16; o2 >= 1; o2 >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o2);
                    if (lane == 0) {
                        s_n[r] = mm;
                        s_n[R + r] = ll;
                    }
                }
                __syncthreads();
                for (int x = tid; x < R * DP / 4; x += kKvWarps * 32) {
                    const int r = x / (DP / 4), pos = (x % (DP / 4)) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int i = 0; i < n; ++i) {
                        const float f = s_f[i * R + r];
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(slot_of(i) + 2 * R + r * DP + pos));
                        v.x = fmaf(f, u.x, v.x);
                        v.y = fmaf(f, u.y, v.y);
                        v.z = fmaf(f, u.z, v.z);
                        v.w = fmaf(f, u.w, v.w);
                    }
                    finish(r, pos, s_n[r], s_n[R + r], make_float2(v.x, v.y));
                    finish(r, pos + 2, s_n[r], s_n[R + r], make_float2(v.z, v.w));
                }
                __syncthreads();  // the memory goes back to the rings
            }
        }
        it += nseg + a.geom.lead;
        if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
    }
}

template <int DP, int NR, bool MASS>
constexpr size_t kv_attention_smem() {
    constexpr size_t join = static_cast<size_t>(kKvWarps) * 8 * NR * (DP + 8 + 2) * 4;
    constexpr size_t rings = static_cast<size_t>(kKvWarps) * KvRing<DP, MASS>::total;
    return MASS || rings > join ? rings : join;
}

}  // namespace q4dev

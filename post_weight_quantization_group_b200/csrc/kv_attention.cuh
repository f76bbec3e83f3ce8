// kv_attention.cuh -- attention of new tokens over the paged INT8 cache, the
// kernel of few rows (decode steps and short chunks).
//
//   S[r, j] = scale * (q_r . kq_j) * sk_j,   visible: at_r - window < j <= at_r,
//   out_r = sum_j 2^(S log2e - m) sv_j vq_j / sum_j 2^(S log2e - m).
//
// The V scale goes into the exponent: with x = S log2e + log2 sv and
// p' = 2^(x - m'), m' the running maximum of x, the numerator is
// sum p' vq and the denominator sum p' / sv.  p' has its maximum near 1 whatever
// the V scales are, so it can be rounded to fp16 (2^-11, as fine as the
// codes' own exact fp16 form allows for the product) without leaving fp16's
// range; the denominator adds the unrounded fp32 p'.  V scales below 2^-100
// are taken as 2^-100 (an absolute error below 2^-93).
//
// Bound by the cache bytes read once from HBM.  Nothing of a cached row goes
// through shared memory: with the products transposed, S^T = K q^T and
// O^T = V^T P^T (mma.sync m16n8k16), a thread's fragment of K is 16-byte
// pieces of a row and of V 16-byte pieces of four rows, loaded straight to
// registers one block of 16 tokens ahead, because the order of head_dim
// inside the dot product and of head_dim in the accumulator's rows is free.
// The eight query rows of an MMA's N are one KV head's group at a decode step
// (the tensor pipe is far from a bound here: 8 warps issue 16 MMAs per 4 KB).
// P^T comes out of S^T's accumulator by one movmatrix per 8 tokens.
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
    float* lse;  // [tokens, q_heads] or null
    int64_t q_stride, out_stride;
    int q_heads;
    float scale_log2;  // scale * log2(e)
    float* part;       // partial slots, two per CTA: m [R], l [R], O [R, DP]
    unsigned* count;   // one per CTA
    unsigned* status;
};

constexpr int kKvWarps = 8;
constexpr int kKvTile = 16 * kKvWarps;  // tokens of a tile
constexpr float kKvNone = -1e30f;       // the maximum of nothing: finite, so that m - m' is not NaN
// A warp rescales only when a score passes its maximum by more than this
// (log2): p' stays below 2^8, inside fp16, and most blocks skip the rescale.
constexpr float kKvLazy = 8.0f;

__device__ __forceinline__ uint4 kv_ldg16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 kv_ldg8(const void* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
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
    const float c = fmaxf(sv, 7.888609e-31f);  // 2^-100; a NaN becomes 2^-100 here ...
    r.lg = sv == sv ? __log2f(c) : sv;         // ... and stays in the exponent, where masks drop it
    // within 1 ulp; c is normal and, as 1/127 of a finite value, below 2^121
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(c));
    return r;
}

// A block of 16 cached tokens as one thread holds it.
template <int DP>
struct KvBlock {
    static constexpr int U = DP / 64;                 // 64-byte pieces of a K row
    static constexpr int VW = DP / 32;                // words of a thread's piece of a V row
    uint4 k[2][U];                                    // rows g, g + 8
    uint32_t v[4][VW];                                // rows 2t, 2t + 1, 2t + 8, 2t + 9
    uint16_t ks[2], vs[2];                            // scales of tokens g, g + 8
};

// DP: head_dim padded to 64, 128 or 256.  NR: blocks of 8 rows (R = 8 NR).
// P16: the page size is a multiple of 16, so a block of 16 tokens is in one
// page and its rows follow one another; else every row looks up its own page.
template <bool BF16, int DP, int NR, bool P16>
__global__ void __launch_bounds__(kKvWarps * 32, DP * NR > 128 ? 1 : 2)
    kv_attention_kernel(const __grid_constant__ KvAttn a) {
    constexpr int R = 8 * NR;
    constexpr int U = DP / 64, VW = DP / 32, MT = DP / 16;
    constexpr int ROW = DP + 8;  // padded row of the join buffer (floats): rows 2t apart by 16 banks
    extern __shared__ float smem[];
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
    if (beg == end) return;
    KvSeq seq = kv_seq(a.batch, w.b, a.status);
    const int shift = (c.ps & (c.ps - 1)) == 0 ? 31 - __clz(c.ps) : -1;
    auto page_index = [&](int j) { return shift >= 0 ? j >> shift : j / c.ps; };
    // pieces beyond head_dim repeat piece 0: their K meets zeros of q, their V is not stored
    int kcol[U], vcol[DP == 64 ? 1 : DP / 128];
#pragma unroll
    for (int u = 0; u < U; ++u) kcol[u] = u * 64 + t * 16 < d ? u * 64 + t * 16 : 0;
#pragma unroll
    for (int u = 0; u < (DP == 64 ? 1 : DP / 128); ++u) {
        const int col = DP == 64 ? g * 8 : u * 128 + g * 16;
        vcol[u] = col < d ? col : 0;
    }

    int64_t it = beg;
    while (it < end) {
        int tile_lo;
        const int ntiles = kv_tiles(a.geom, seq, w.rt, &tile_lo);
        const int64_t unit_beg = it - w.tile, unit_end = unit_beg + ntiles;
        const int nseg = static_cast<int>(min(unit_end, end) - it);
        const int rows = seq.n * a.geom.group;
        const int row0 = w.rt * R;

        // query fragments and the last visible token of this thread's rows
        uint2 qf[NR][DP / 16];
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
        }
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

        auto entry_of = [&](int j0) -> int32_t {
            return P16 && j0 < seq.len ? kv_entry(a.batch, w.b, page_index(j0)) : 0;
        };
        // Where a block's rows are: offsets of token j0's row (P16), of a token's otherwise.
        // Tokens behind the last one repeat it; the masks drop them.
        struct Place {
            int64_t kc, vc, ks, vs;
        };
        auto place = [&](int j, int32_t entry) {
            const int64_t page = kv_page(c, entry, a.status);
            const int64_t row = kv_row(c, w.h, j - page_index(j) * c.ps);
            return Place{page * c.kc_page + row * d, page * c.vc_page + row * d, page * c.ks_page + row,
                         page * c.vs_page + row};
        };
        auto row_of = [&](const Place& base, int j0, int r) {  // of token j0 + r
            const int rr = min(r, seq.len - 1 - j0);
            if constexpr (P16)
                return Place{base.kc + rr * d, base.vc + rr * d, base.ks + rr, base.vs + rr};
            else
                return place(j0 + rr, kv_entry(a.batch, w.b, page_index(j0 + rr)));
        };
        KvBlock<DP> bk;
        auto fetch_k = [&](int j0, const Place& base) {
            if (j0 >= seq.len) return;  // nothing of the block is visible either
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int8_t* p = c.kc + row_of(base, j0, g + 8 * e).kc;
#pragma unroll
                for (int u = 0; u < U; ++u) bk.k[e][u] = kv_ldg16(p + kcol[u]);
            }
        };
        auto fetch_scales = [&](int j0, const Place& base) {
            if (j0 >= seq.len) return;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Place r = row_of(base, j0, g + 8 * e);
                bk.ks[e] = __ldg(c.ks + r.ks);
                bk.vs[e] = __ldg(c.vs + r.vs);
            }
        };
        auto fetch_v = [&](int j0, const Place& base) {
            if (j0 >= seq.len) return;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int8_t* p = c.vc + row_of(base, j0, 2 * t + (e & 1) + 8 * (e >> 1)).vc;
                if constexpr (DP == 64) {
                    const uint2 x = kv_ldg8(p + vcol[0]);
                    bk.v[e][0] = x.x;
                    bk.v[e][1] = x.y;
                } else {
#pragma unroll
                    for (int u = 0; u < DP / 128; ++u) {
                        const uint4 x = kv_ldg16(p + vcol[u]);
                        bk.v[e][4 * u] = x.x;
                        bk.v[e][4 * u + 1] = x.y;
                        bk.v[e][4 * u + 2] = x.z;
                        bk.v[e][4 * u + 3] = x.w;
                    }
                }
            }
        };

        // One block is held: its K registers take the next block's K as soon as S is
        // computed, its V registers as soon as P V is, so each load is in flight for the
        // other half of a step (and the 16 warps of an SM hold 64 KB between them)
        // without a second set of registers.
        int j0 = (tile_lo + w.tile) * kKvTile + warp * 16;
        auto base_of = [&](int j0, int32_t entry) {
            return P16 && j0 < seq.len ? place(j0, entry) : Place{0, 0, 0, 0};
        };
        Place nb = base_of(j0, entry_of(j0));
        int32_t entry_next = nseg > 1 ? entry_of(j0 + kKvTile) : 0;
        fetch_k(j0, nb);
        fetch_scales(j0, nb);
        fetch_v(j0, nb);
        for (int s = 0; s < nseg; ++s, j0 += kKvTile) {
            const bool more = s + 1 < nseg;
            if (more) nb = base_of(j0 + kKvTile, entry_next);
            if (s + 2 < nseg) entry_next = entry_of(j0 + 2 * kKvTile);
            // nothing of this block is visible to any row: at the ends of a unit's range
            if (j0 > at_max || (a.geom.window && j0 + 15 <= at_min - a.geom.window)) {
                if (more) {
                    fetch_k(j0 + kKvTile, nb);
                    fetch_scales(j0 + kKvTile, nb);
                    fetch_v(j0 + kKvTile, nb);
                }
                continue;
            }

            // S^T = K q^T
            float x[NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k0[4] = {bk.k[0][u].x, bk.k[0][u].y, bk.k[0][u].z, bk.k[0][u].w};
                const uint32_t k1[4] = {bk.k[1][u].x, bk.k[1][u].y, bk.k[1][u].z, bk.k[1][u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t af[4] = {q8_pair<BF16>(k0[i], 0x4140u), q8_pair<BF16>(k1[i], 0x4140u),
                                            q8_pair<BF16>(k0[i], 0x4342u), q8_pair<BF16>(k1[i], 0x4342u)};
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        mma_16816<BF16>(x[n], af, qf[n][u * 4 + i].x, qf[n][u * 4 + i].y);
                }
            }
            if (more) fetch_k(j0 + kKvTile, nb);
            // scores in log2, with the V scale; masks
            const float sk0 = cache_value<BF16>(bk.ks[0]) * a.scale_log2;
            const float sk1 = cache_value<BF16>(bk.ks[1]) * a.scale_log2;
            const KvVScale v0 = kv_vscale(cache_value<BF16>(bk.vs[0]));
            const KvVScale v1 = kv_vscale(cache_value<BF16>(bk.vs[1]));
            if (more) fetch_scales(j0 + kKvTile, nb);
            const bool open = j0 + 15 <= at_min && (!a.geom.window || j0 > at_max - a.geom.window);
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                x[n][0] = fmaf(x[n][0], sk0, v0.lg);
                x[n][1] = fmaf(x[n][1], sk0, v0.lg);
                x[n][2] = fmaf(x[n][2], sk1, v1.lg);
                x[n][3] = fmaf(x[n][3], sk1, v1.lg);
                if (!open) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + g + 8 * (e >> 1);
                        const bool see = j <= at[n][e & 1] &&
                                         (!a.geom.window || j > at[n][e & 1] - a.geom.window);
                        if (!see) x[n][e] = -INFINITY;
                    }
                }
                grow |= fmaxf(x[n][0], x[n][2]) > m[n][0] + kKvLazy ||
                        fmaxf(x[n][1], x[n][3]) > m[n][1] + kKvLazy;
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
                        mx = mx > m[n][e] + kKvLazy ? mx : m[n][e];
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
            for (int i = 0; i < VW; ++i) {
                const uint32_t y0 = bk.v[0][i] ^ 0x80808080u, y1 = bk.v[1][i] ^ 0x80808080u;
                const uint32_t y2 = bk.v[2][i] ^ 0x80808080u, y3 = bk.v[3][i] ^ 0x80808080u;
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {
                    const uint32_t sel = hw ? 0x7362u : 0x5140u;  // bytes 2, 3 or 0, 1 of both rows
                    const uint32_t a01 = prmt(y0, y1, sel), a23 = prmt(y2, y3, sel);
                    const uint32_t af[4] = {sub2<false>(prmt(a01, 0x64u, 0x4140u), 0x64806480u),
                                            sub2<false>(prmt(a01, 0x64u, 0x4342u), 0x64806480u),
                                            sub2<false>(prmt(a23, 0x64u, 0x4140u), 0x64806480u),
                                            sub2<false>(prmt(a23, 0x64u, 0x4342u), 0x64806480u)};
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        mma_16816<false>(o[2 * i + hw][n], af, pb[n][0], pb[n][1]);
                }
            }
            if (more) fetch_v(j0 + kKvTile, nb);
        }

        // ------------------------------------------- join of the CTA's warps
        // Element (row, pos) of O: pos = 16 i + 2 g + e for the accumulator tile i, so
        // that a warp's stores and the join's loads are free of bank conflicts.
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
                __threadfence();
                for (int x = tid; x < R * DP / 2; x += kKvWarps * 32) {
                    const int r = x / (DP / 2), pos = (x % (DP / 2)) * 2;
                    float mm = kKvNone, ll = 0.f;
                    float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
                    for (int64_t p = first_cta; p <= last_cta; ++p) {
                        const int64_t pb = T * p / P;
                        const float* src = a.part + (2 * p + (pb >= unit_beg ? 0 : 1)) * SLOT;
                        const float mp = __ldcg(src + r), lp = __ldcg(src + R + r);
                        const float2 u = __ldcg(reinterpret_cast<const float2*>(src + 2 * R + r * DP + pos));
                        const float mn = fmaxf(mm, mp);
                        const float f0 = kv_exp2(mm - mn), f1 = kv_exp2(mp - mn);
                        ll = fmaf(lp, f1, ll * f0);
                        v.x = fmaf(u.x, f1, v.x * f0);
                        v.y = fmaf(u.y, f1, v.y * f0);
                        mm = mn;
                    }
                    finish(r, pos, mm, ll, v);
                }
            }
        }
        it += nseg;
        if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
    }
}

template <int DP, int NR>
constexpr size_t kv_attention_smem() {
    return static_cast<size_t>(kKvWarps) * 8 * NR * (DP + 8 + 2) * 4;
}

}  // namespace q4dev

// kv_attention_tc.cuh -- attention of chunks of new tokens over the paged INT8
// cache on the tcgen05 tensor cores (head_dim up to 128).  The mathematics,
// the division of work and the join of a unit's parts are those of
// kv_attention.cuh; a unit has 256 rows, two M = 128 halves A and B that share
// every converted tile of the cache.
//
// Per 128-token tile and half, S = Q K^T goes to tensor memory, a softmax
// thread owns one row of it (no shuffles), writes p' as fp16 over the same
// columns, and O += P V reads it there as the A operand.  While one half is
// in its softmax the tensor pipe works on the other.  O stays in tensor
// memory; it is rescaled only when a row's maximum grows by more than kKvLazy.
//
//   warps 0-3 / 4-7   softmax of half A / B
//   warps 8-11        conversion: codes from the pages (16-byte loads, a tile
//                     ahead in registers) to 16-bit floats in shared memory,
//                     K in the cache type, V in fp16; the tile's scales; the
//                     unit's Q
//   warp 12           tcgen05.mma issue
//
// K [token, d] is a K-major operand of S and V [token, d] an N-major operand
// of P V: the same storage, [d / 64] blocks of 128-byte rows, one per token,
// 128-byte swizzle.
#pragma once

#include <stdint.h>

#include "kv_attention.cuh"
#include "q4_tcgen05.cuh"

namespace q4dev {

constexpr int kTcaThreads = 512;
constexpr int kTcaRows = 256;
constexpr int kTcaKT = 128;  // tokens of a tile

template <int DP>
struct TcaGeom {
    static constexpr uint32_t tile = DP * 256;  // bytes of 128 rows of DP 16-bit elements
    static constexpr uint32_t off_q = 0;        // two halves
    static constexpr uint32_t off_k = 2 * tile; // two stages
    static constexpr uint32_t off_v = 4 * tile;
    static constexpr uint32_t off_sc = 6 * tile;                 // two slots of sk, lg, inv
    static constexpr uint32_t off_bar = off_sc + 2 * 3 * 128 * 4;
    static constexpr uint32_t total = off_bar + 256 + 1024;
};

// Sixteen codes of token `row`, unit `u` of its DP / 16, as 16-bit floats into
// a tile.  The second half of a 128-element row stores its chunks in the other
// order, so that eight lanes of a row hit eight different 16-byte columns.
template <bool BF16>
__device__ __forceinline__ void tca_store16(uint32_t tile, int row, int u, const uint4& raw) {
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            o[2 * i] = q8_pair<true>(w[i], 0x4140u);
            o[2 * i + 1] = q8_pair<true>(w[i], 0x4342u);
        } else {
            const uint32_t y = w[i] ^ 0x80808080u;
            o[2 * i] = sub2<false>(prmt(y, 0x64u, 0x4140u), 0x64806480u);
            o[2 * i + 1] = sub2<false>(prmt(y, 0x64u, 0x4342u), 0x64806480u);
        }
    }
    const uint32_t base = tile + (u >> 2) * 16384u + static_cast<uint32_t>(row) * 128u;
    const uint32_t c = static_cast<uint32_t>(u & 3) * 2, x = static_cast<uint32_t>(row & 7);
    const bool odd = (u >> 2) & 1;
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    sts128(base + (((odd ? c + 1 : c) ^ x) << 4), odd ? hi : lo);
    sts128(base + (((odd ? c : c + 1) ^ x) << 4), odd ? lo : hi);
}

// A warp's bounded wait, with one outcome for all of its lanes: a wait that
// ran out must not part the lanes of a warp that goes on to collective steps.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity & 1u, status, kWaitLimitNs));
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kTcaThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ KvAttn a) {
    using G = TcaGeom<DP>;
    constexpr uint32_t kIdescS = umma_idesc_f16<BF16, 128, kTcaKT>();
    constexpr uint32_t kIdescO = umma_idesc_f16<false, 128, DP>() | kIdescNMajorB;
    constexpr uint32_t kColO = 256;  // tensor memory: S_A, S_B (128 columns each), O_A, O_B (DP each)
    constexpr int64_t SLOT = static_cast<int64_t>(kTcaRows) * (DP + 2);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::off_bar);
    uint64_t* k_full = bars;        // [2] conversion -> MMA, softmax (scales)
    uint64_t* k_empty = bars + 2;   // [2] S of both halves done
    uint64_t* v_full = bars + 4;    // [2]
    uint64_t* v_empty = bars + 6;   // [2] P V of both halves done
    uint64_t* sc_free = bars + 8;   // [2] softmax has read the slot's scales
    uint64_t* s_full = bars + 10;   // [half]
    uint64_t* p_ready = bars + 12;  // [half]
    uint64_t* pv_done = bars + 14;  // [half]
    uint64_t* q_full = bars + 16;
    uint64_t* q_free = bars + 17;
    uint64_t* drain = bars + 18;
    uint32_t* tbase_s = reinterpret_cast<uint32_t*>(bars + 19);
    __shared__ KvLocateShared s_loc;
    __shared__ unsigned s_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
            mbar_init(&sc_free[i], 8);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 4);
        mbar_init(q_free, 1);
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 12) tmem_alloc(tbase_s, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tbase_s;
    grid_launch_dependents();
    grid_dependency_wait();

    int64_t T, P, beg, end;
    KvPlace w;
    kv_locate<kTcaThreads>(a.batch, a.geom, blockIdx.x, gridDim.x, 1, a.status, &s_loc, &T, &P, &beg,
                           &end, &w);
    const int group = a.geom.group, window = a.geom.window;

    // Every role walks the same segments: (unit, tiles) of this CTA's range.
    struct Segment {
        KvSeq seq;
        int tile0, tiles, rows, row0;
        int64_t unit_beg, unit_end;
        bool both;  // half B has rows
    };
    auto segment = [&](int64_t it, const KvPlace& p, const KvSeq& s) {
        Segment g;
        int lo;
        const int n = kv_tiles(a.geom, s, p.rt, &lo);
        g.seq = s;
        g.tile0 = lo + p.tile;
        g.unit_beg = it - p.tile;
        g.unit_end = g.unit_beg + n;
        g.tiles = static_cast<int>(min(g.unit_end, end) - it);
        g.rows = s.n * group;
        g.row0 = p.rt * kTcaRows;
        g.both = g.rows - g.row0 > 128;
        return g;
    };

    if (beg < end) {
        KvSeq seq = kv_seq(a.batch, w.b, a.status);
        if (warp < 8) {
            // ------------------------------------------------------ softmax
            regs_inc<184>();
            const int half = warp >> 2;
            const uint32_t tl = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
            const uint32_t ts = tl + half * 128, to = tl + kColO + half * DP;
            const int r = half * 128 + (warp & 3) * 32 + lane;  // row of the unit
            int c = 0;        // tiles so far: the K stage and scale slot
            uint32_t n = 0;   // tiles of this half so far
            bool ok = true;
            for (int64_t it = beg; it < end;) {  // a failed wait still goes through the barriers
                const Segment g = segment(it, w, seq);
                const bool active = half == 0 || g.both;
                const bool live = g.row0 + r < g.rows;
                const bool warp_live = g.row0 + r - lane < g.rows;
                const int past = g.seq.len - g.seq.n;
                const int at = live ? past + (g.row0 + r) / group : -1;
                const int at_min = past + (g.row0 + half * 128) / group;
                const int at_max = past + (min(g.row0 + half * 128 + 128, g.rows) - 1) / group;
                float m = kKvNone, l = 0.f;
                for (int i = 0; i < g.tiles && ok; ++i, ++c) {
                    const int slot = c & 1;
                    if (active) ok = warp_wait(&s_full[half], n, a.status);
                    if (ok) ok = warp_wait(&k_full[slot], c >> 1, a.status);
                    if (!ok) break;
                    if (!active || !warp_live) {
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sc_free[slot]);
                            if (active) mbar_arrive(&p_ready[half]);
                        }
                        if (active) ++n;
                        continue;
                    }
                    tc_fence_after();
                    const float* sc = reinterpret_cast<const float*>(smem + G::off_sc) + slot * 384;
                    float x[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tmem_ld32(ts + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * q]));
                    tmem_wait_ld();
                    const int j0 = (g.tile0 + i) * kTcaKT;
                    float mx = kKvNone;
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const float4 sk = *reinterpret_cast<const float4*>(sc + 4 * q);
                        const float4 lg = *reinterpret_cast<const float4*>(sc + 128 + 4 * q);
                        x[4 * q] = fmaf(x[4 * q], sk.x, lg.x);
                        x[4 * q + 1] = fmaf(x[4 * q + 1], sk.y, lg.y);
                        x[4 * q + 2] = fmaf(x[4 * q + 2], sk.z, lg.z);
                        x[4 * q + 3] = fmaf(x[4 * q + 3], sk.w, lg.w);
                    }
                    // every row of the half sees the whole tile, or masks
                    if (!(j0 + kTcaKT - 1 <= at_min && (!window || j0 > at_max - window))) {
                        const int hi = at - j0;                       // columns <= hi
                        const int lo = window ? at - window - j0 : -1;  // and > lo
#pragma unroll
                        for (int q = 0; q < 128; ++q)
                            if (q > hi || q <= lo) x[q] = -INFINITY;
                    }
#pragma unroll
                    for (int q = 0; q < 128; ++q) mx = fmaxf(mx, x[q]);
                    if (__any_sync(0xFFFFFFFFu, mx > m + kKvLazy)) {
                        const float mn = fmaxf(m, mx), f = kv_exp2(m - mn);
                        m = mn;
                        l *= f;
                        if (i > 0) {
                            ok = warp_wait(&pv_done[half], n - 1, a.status);
                            tc_fence_after();
#pragma unroll
                            for (int q = 0; q < DP / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld16(to + 16 * q, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st8(to + 16 * q, *reinterpret_cast<uint32_t(*)[8]>(&o[0]));
                                tmem_st8(to + 16 * q + 8, *reinterpret_cast<uint32_t(*)[8]>(&o[8]));
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t p[32];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int y = 64 * q + 4 * e;
                            const float4 inv = *reinterpret_cast<const float4*>(sc + 256 + y);
                            const float p0 = kv_exp2(x[y] - m), p1 = kv_exp2(x[y + 1] - m);
                            const float p2 = kv_exp2(x[y + 2] - m), p3 = kv_exp2(x[y + 3] - m);
                            l = fmaf(p0, inv.x, l);
                            l = fmaf(p1, inv.y, l);
                            l = fmaf(p2, inv.z, l);
                            l = fmaf(p3, inv.w, l);
                            p[2 * e] = kv_pack_f16(p0, p1);
                            p[2 * e + 1] = kv_pack_f16(p2, p3);
                        }
                        tmem_st32(ts + 32 * q, p);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&p_ready[half]);
                        mbar_arrive(&sc_free[slot]);
                    }
                    ++n;
                }
                // ------------------------------------- end of the segment
                const bool whole = it == g.unit_beg && it + g.tiles == g.unit_end;
                const int row = g.row0 + r, tok = row / group;
                const int head = w.h * group + row - tok * group;
                uint16_t* out = a.out + (g.seq.first + tok) * a.out_stride + static_cast<int64_t>(head) * a.pool.d;
                auto store_lse = [&](float mm, float ll) {
                    if (a.lse)
                        a.lse[(g.seq.first + tok) * a.q_heads + head] =
                            ll == 0.f ? -INFINITY : 0.69314718f * (mm + __log2f(ll));
                };
                // eight elements of the row from column e0 on
                auto store8 = [&](int e0, float ll, const float (&v)[8]) {
                    const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : ll == 0.f ? 0.f : ll;
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = v[e] * inv;
                    if (e0 < a.pool.d) *reinterpret_cast<uint4*>(out + e0) = pack8<BF16>(y);
                };
                const int64_t first_cta = whole ? 0 : kv_owner(g.unit_beg, T, P);
                const int64_t last_cta = whole ? 0 : kv_owner(g.unit_end - 1, T, P);
                if (ok && active && warp_live) {
                    ok = warp_wait(&pv_done[half], n - 1, a.status);
                    tc_fence_after();
                    // a slot: m [256], l [256], O [DP][256] (a column of rows together)
                    float* part = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (it == beg ? 0 : 1)) * SLOT;
                    if (whole) {
                        if (live) store_lse(m, l);
                    } else {
                        __stcg(part + r, m);
                        __stcg(part + kTcaRows + r, l);
                    }
#pragma unroll
                    for (int q = 0; q < DP / 16; ++q) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * q, o);
                        tmem_wait_ld();
                        if (whole) {
                            if (live) {
                                store8(16 * q, l, *reinterpret_cast<float(*)[8]>(&o[0]));
                                store8(16 * q + 8, l, *reinterpret_cast<float(*)[8]>(&o[8]));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                __stcg(part + 2 * kTcaRows + (16 * q + e) * kTcaRows + r, __uint_as_float(o[e]));
                        }
                    }
                    tc_fence_before();
                }
                if (!whole) {
                    named_bar_sync(1, 256);
                    if (tid == 0) {
                        const unsigned prev = kv_arrive(a.count + first_cta);
                        s_last = prev == static_cast<unsigned>(last_cta - first_cta);
                        if (s_last) a.count[first_cta] = 0u;  // zero again for the next call
                    }
                    named_bar_sync(1, 256);
                    if (ok && s_last && active && live) {
                        __threadfence();
                        auto slot_of = [&](int64_t p) -> const float* {
                            return a.part + (2 * p + (T * p / P >= g.unit_beg ? 0 : 1)) * SLOT;
                        };
                        float mm = kKvNone;
                        for (int64_t p = first_cta; p <= last_cta; ++p) mm = fmaxf(mm, __ldcg(slot_of(p) + r));
                        float ll = 0.f;
                        for (int64_t p = first_cta; p <= last_cta; ++p) {
                            const float* s = slot_of(p);
                            ll = fmaf(__ldcg(s + kTcaRows + r), kv_exp2(__ldcg(s + r) - mm), ll);
                        }
                        store_lse(mm, ll);
                        for (int e0 = 0; e0 < DP; e0 += 8) {
                            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                            for (int64_t p = first_cta; p <= last_cta; ++p) {
                                const float* s = slot_of(p);
                                const float f = kv_exp2(__ldcg(s + r) - mm);
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    v[e] = fmaf(f, __ldcg(s + 2 * kTcaRows + (e0 + e) * kTcaRows + r), v[e]);
                            }
                            store8(e0, ll, v);
                        }
                    }
                }
                it += g.tiles;
                if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
            }
        } else if (warp < 12) {
            // --------------------------------------------------- conversion
            regs_dec<104>();
            constexpr int UPR = DP / 16;           // 16-code units of a row
            constexpr int NI = 128 * UPR / 128;    // units of a thread
            constexpr int RSTEP = 128 / UPR;       // rows between them
            const KvPool& pc = a.pool;
            const int ct = tid - 256, u = ct % UPR, rb = ct / UPR;
            const bool unit_on = u * 16 < pc.d;
            const int shift = (pc.ps & (pc.ps - 1)) == 0 ? 31 - __clz(pc.ps) : -1;
            auto entry_of = [&](int j, int* off) {  // table entry and place in the page of token j
                const int e = shift >= 0 ? j >> shift : j / pc.ps;
                *off = j - e * pc.ps;
                return e;
            };
            bool ok = true;
            int c = 0, segs = 0;
            for (int64_t it = beg; it < end && ok; ++segs) {
                const Segment g = segment(it, w, seq);
                uint4 kr[NI], vr[NI];
                int32_t ent[NI], ent_sc = 0;
                uint16_t ks = 0, vs = 0;
                auto entries = [&](int j0) {
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int j = j0 + rb + i * RSTEP;
                        int off;
                        ent[i] = j < g.seq.len ? kv_entry(a.batch, w.b, entry_of(j, &off)) : 0;
                    }
                    int off;
                    const int j = j0 + ct;
                    ent_sc = j < g.seq.len ? kv_entry(a.batch, w.b, entry_of(j, &off)) : 0;
                };
                auto load = [&](uint4 (&x)[NI], const int8_t* base, int64_t stride, int j0) {
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int j = j0 + rb + i * RSTEP;
                        x[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (j < g.seq.len && unit_on) {
                            int off;
                            entry_of(j, &off);
                            const int64_t page = kv_page(pc, ent[i], a.status);
                            x[i] = __ldg(reinterpret_cast<const uint4*>(
                                base + page * stride + kv_row(pc, w.h, off) * pc.d + u * 16));
                        }
                    }
                };
                auto load_scales = [&](int j0) {
                    const int j = j0 + ct;
                    ks = vs = 0;
                    if (j < g.seq.len) {
                        int off;
                        entry_of(j, &off);
                        const int64_t page = kv_page(pc, ent_sc, a.status), row = kv_row(pc, w.h, off);
                        ks = __ldg(pc.ks + page * pc.ks_page + row);
                        vs = __ldg(pc.vs + page * pc.vs_page + row);
                    }
                };
                int j0 = g.tile0 * kTcaKT;
                entries(j0);
                load(kr, pc.kc, pc.kc_page, j0);
                load_scales(j0);
                load(vr, pc.vc, pc.vc_page, j0);

                // the unit's queries, once the products of the last one have read theirs
                if (segs > 0) ok = warp_wait(q_free, segs - 1, a.status);
                if (!ok) break;
                {
                    constexpr int CPR = DP / 8;  // 16-byte chunks of a row
                    const int qrows = g.both ? 256 : 128;
                    const int ch = ct % CPR;
#pragma unroll 4
                    for (int rr = ct / CPR; rr < qrows; rr += 128 / CPR) {
                        const int row = g.row0 + rr;
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (row < g.rows && ch * 8 < pc.d) {
                            const int tok = row / group;
                            x = *reinterpret_cast<const uint4*>(
                                a.q + (g.seq.first + tok) * a.q_stride +
                                static_cast<int64_t>(w.h * group + row - tok * group) * pc.d + ch * 8);
                        }
                        const int rh = rr & 127;
                        sts128(sbase + G::off_q + (rr >> 7) * G::tile + (ch >> 3) * 16384u + rh * 128u +
                                   (static_cast<uint32_t>((ch & 7) ^ (rh & 7)) << 4), x);
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);

                for (int i = 0; i < g.tiles && ok; ++i, ++c, j0 += kTcaKT) {
                    const int st = c & 1;
                    const uint32_t use = static_cast<uint32_t>(c >> 1);  // earlier uses of the stage
                    const bool more = i + 1 < g.tiles;
                    if (more) entries(j0 + kTcaKT);
                    if (use > 0) {
                        ok = warp_wait(&k_empty[st], use - 1, a.status) &&
                             warp_wait(&sc_free[st], use - 1, a.status);
                        if (!ok) break;
                    }
                    {
                        const uint32_t tile = sbase + G::off_k + st * G::tile;
#pragma unroll
                        for (int q = 0; q < NI; ++q) tca_store16<BF16>(tile, rb + q * RSTEP, u, kr[q]);
                        float* sc = reinterpret_cast<float*>(smem + G::off_sc) + st * 384;
                        const KvVScale v = kv_vscale(cache_value<BF16>(vs));
                        const bool in = j0 + ct < g.seq.len;
                        sc[ct] = cache_value<BF16>(ks) * a.scale_log2;
                        sc[128 + ct] = in ? v.lg : 0.f;
                        sc[256 + ct] = in ? v.inv : 0.f;
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&k_full[st]);
                    if (more) {
                        load(kr, pc.kc, pc.kc_page, j0 + kTcaKT);
                        load_scales(j0 + kTcaKT);
                    }
                    if (use > 0) {
                        ok = warp_wait(&v_empty[st], use - 1, a.status);
                        if (!ok) break;
                    }
                    {
                        const uint32_t tile = sbase + G::off_v + st * G::tile;
#pragma unroll
                        for (int q = 0; q < NI; ++q) tca_store16<false>(tile, rb + q * RSTEP, u, vr[q]);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[st]);
                    if (more) load(vr, pc.vc, pc.vc_page, j0 + kTcaKT);
                }
                it += g.tiles;
                if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
            }
        } else {
            regs_dec<40>();
            if (warp == 12 && lane == 0) {
                // ---------------------------------------------- MMA issue
                bool ok = true;
                int c = 0, segs = 0;
                uint32_t n[2] = {0, 0};
                auto issue_s = [&](int half, int st) {
                    const uint32_t q = sbase + G::off_q + half * G::tile, k = sbase + G::off_k + st * G::tile;
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * 16384u + (kk & 3) * 32u;
                        umma_f16_ss(tbase + half * 128, umma_desc_sw128_kmajor(q + off),
                                    umma_desc_sw128_kmajor(k + off), kIdescS, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&s_full[half]);
                };
                auto issue_pv = [&](int half, int st, bool add) {
                    const uint32_t v = sbase + G::off_v + st * G::tile;
#pragma unroll
                    for (int kk = 0; kk < kTcaKT / 16; ++kk)
                        umma_f16_ts(tbase + kColO + half * DP, tbase + half * 128 + kk * 8,
                                    umma_desc_sw128_nmajor(v + kk * 2048u, 16384u), kIdescO,
                                    (add || kk > 0) ? 1u : 0u);
                    umma_commit(&pv_done[half]);
                };
                auto wait = [&](uint64_t* b, uint32_t ph) {
                    if (ok) ok = mbar_wait_bounded(b, ph & 1u, a.status, kWaitLimitNs);
                    tc_fence_after();
                    return ok;
                };
                for (int64_t it = beg; it < end && ok; ++segs) {
                    const Segment g = segment(it, w, seq);
                    if (!wait(q_full, segs)) break;
                    if (!wait(&k_full[c & 1], c >> 1)) break;
                    issue_s(0, c & 1);
                    if (g.both) issue_s(1, c & 1);
                    umma_commit(&k_empty[c & 1]);
                    if (g.tiles == 1) umma_commit(q_free);
                    for (int i = 0; i < g.tiles; ++i, ++c) {
                        const int st = c & 1, sn = (c + 1) & 1;
                        const bool more = i + 1 < g.tiles;
                        if (!wait(&v_full[st], c >> 1)) break;
                        if (!wait(&p_ready[0], n[0]++)) break;
                        issue_pv(0, st, i > 0);
                        if (more) {
                            if (!wait(&k_full[sn], (c + 1) >> 1)) break;
                            issue_s(0, sn);
                        }
                        if (g.both) {
                            if (!wait(&p_ready[1], n[1]++)) break;
                            issue_pv(1, st, i > 0);
                        }
                        umma_commit(&v_empty[st]);
                        if (more) {
                            if (g.both) issue_s(1, sn);
                            umma_commit(&k_empty[sn]);
                            if (i + 2 == g.tiles) umma_commit(q_free);
                        }
                    }
                    it += g.tiles;
                    if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
                }
                // every MMA has completed before tensor memory is released
                umma_commit(drain);
                mbar_wait_bounded(drain, 0, a.status, kWaitLimitNs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

}  // namespace q4dev

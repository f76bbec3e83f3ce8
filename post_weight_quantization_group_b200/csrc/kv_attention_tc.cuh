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
// memory; it is rescaled only when a row's x passes its m' by more than kKvTop.
//
// Measured (B200): 1024 new tokens over 32,768, 64 query heads over 8 of 128,
// 1.68 ms = 650 TFLOP/s.  A tile takes 6050 cycles, of which its products need 2050: a
// softmax warp works 3600 and waits 1800 to 2100 for its half's next scores, which
// wait for the P V before them (P lies over S).
//
//   warps 0-3 / 4-7   softmax of half A / B
//   warps 8-11        conversion: codes from the pages (16-byte loads, a tile
//                     ahead in registers) to 16-bit floats in shared memory,
//                     K in the cache type, V in fp16; the unit's Q
//   warp 12           tcgen05.mma issue
//   warp 13           walks the CTA's work and leaves for the others, ahead of
//                     them, its segments (TcaSeg) and the tiles' row addresses
//                     (block table) and scales
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

constexpr int kTcaRowSlots = 3;  // tiles of row addresses
constexpr int kTcaScSlots = 4;   // tiles of scales
constexpr int kTcaSegSlots = 4;  // segments

// Consecutive tiles of one unit, the work of a CTA one after another; tiles =
// 0 ends the list.
struct TcaSeg {
    int64_t first;             // the sequence's first row of q
    int past;                  // cached tokens before its new ones
    int rows, row0, h;         // rows of the sequence and head, the unit's first, the head
    int tile0, tiles;
    int first_cta, last_cta;   // the CTAs that share the unit
    int whole;                 // it is all this CTA's
    int slot, first_slot;      // partial slot (0 or 1) of this CTA and of first_cta
    int pad[3];
};
static_assert(sizeof(TcaSeg) == 64, "segment ring");

template <int DP>
struct TcaGeom {
    static constexpr uint32_t tile = DP * 256;  // bytes of 128 rows of DP 16-bit elements
    static constexpr uint32_t off_q = 0;        // two halves
    static constexpr uint32_t off_k = 2 * tile; // two stages
    static constexpr uint32_t off_v = 4 * tile;
    static constexpr uint32_t off_sc = 6 * tile;                          // sk, lg, inv [128]
    static constexpr uint32_t off_row = off_sc + kTcaScSlots * 3 * 128 * 4;  // K, V offsets [128]
    static constexpr uint32_t off_bar = off_row + kTcaRowSlots * 2 * 128 * 8;
    static constexpr uint32_t off_seg = off_bar + 512;
    static constexpr uint32_t off_at = off_seg + kTcaSegSlots * 64;  // last visible token, per row
    static constexpr uint32_t off_one = off_at + 1024;               // 128 ones, 128 zeros
    static constexpr uint32_t total = off_one + 1024 + 1024;
};

// Packed fp32 pairs: one instruction for both.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float f_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// An fp32 pair from shared memory.
__device__ __forceinline__ uint64_t lds_f2(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(addr));
    return v;
}

// Sixteen codes of token `row`, unit `u` of its DP / 16, as 16-bit floats into
// a tile.
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
    const uint32_t at = (static_cast<uint32_t>(u & 3) * 2u ^ static_cast<uint32_t>(row & 7)) << 4;
    sts128(base + at, make_uint4(o[0], o[1], o[2], o[3]));
    sts128(base + (at ^ 16u), make_uint4(o[4], o[5], o[6], o[7]));
}

// mbar_wait_bounded without a suspend time in its polls.
__device__ __forceinline__ bool mbar_wait_poll(uint64_t* bar, uint32_t parity, unsigned* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, kStatusTimeout);
            return false;
        }
    }
}

// A warp's bounded wait, with one outcome for all of its lanes: a wait that
// ran out must not part the lanes of a warp that goes on to collective steps.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_poll(bar, parity & 1u, status));
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
    uint64_t* k_full = bars;        // [2] conversion -> MMA
    uint64_t* k_empty = bars + 2;   // [2] S of both halves done
    uint64_t* v_full = bars + 4;    // [2]
    uint64_t* v_empty = bars + 6;   // [2] P V of both halves done
    uint64_t* s_full = bars + 8;    // [half]
    uint64_t* p_ready = bars + 10;  // [half]
    uint64_t* pv_done = bars + 12;  // [half]
    uint64_t* q_full = bars + 14;
    uint64_t* q_free = bars + 15;
    uint64_t* drain = bars + 16;
    uint64_t* sc_full = bars + 17;             // [kTcaScSlots]
    uint64_t* sc_free = sc_full + kTcaScSlots;
    uint64_t* row_full = sc_free + kTcaScSlots;  // [kTcaRowSlots]
    uint64_t* row_free = row_full + kTcaRowSlots;
    uint64_t* seg_full = row_free + kTcaRowSlots;  // [kTcaSegSlots]
    uint64_t* seg_free = seg_full + kTcaSegSlots;
    uint64_t* join = seg_free + kTcaSegSlots;  // [2] the halves' parts are stored; the count is known
    uint32_t* tbase_s = reinterpret_cast<uint32_t*>(join + 2);
    TcaSeg* segs = reinterpret_cast<TcaSeg*>(smem + G::off_seg);
    __shared__ KvLocateShared s_loc;
    __shared__ unsigned s_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < kTcaScSlots; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_free[i], 8);
        }
        for (int i = 0; i < kTcaRowSlots; ++i) {
            mbar_init(&row_full[i], 1);
            mbar_init(&row_free[i], 4);
        }
        for (int i = 0; i < kTcaSegSlots; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_free[i], 13);  // 8 softmax and 4 conversion warps, the MMA thread
        }
        mbar_init(&join[0], 8);
        mbar_init(&join[1], 1);
        mbar_init(q_full, 4);
        mbar_init(q_free, 1);
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (tid < 256) reinterpret_cast<float*>(smem + G::off_one)[tid] = tid < 128 ? 1.f : 0.f;
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
    kv_fill_unnamed<kTcaThreads>(a, s_loc);
    const int group = a.geom.group, window = a.geom.window;
    if (warp < 8) {
        // ------------------------------------------------------ softmax
        const int half = warp >> 2;
        const uint32_t tl = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + half * 128, to = tl + kColO + half * DP;
        const int r = half * 128 + (warp & 3) * 32 + lane;  // row of the unit
        int c = 0;        // tiles so far: the scale slot
        uint32_t n = 0;   // tiles of this half so far
        bool ok = true;
        uint32_t parts = 0;  // shared units so far
        const uint32_t s_at = sbase + G::off_at + warp * 128u;
        // the value of row `lane` of the warp, from the quad that holds it as its k-th
        auto by_lane = [&](const float (&v)[4]) {
            const int src = (lane & 7) * 4;
            float y = __shfl_sync(0xFFFFFFFFu, v[0], src);
#pragma unroll
            for (int k = 1; k < 4; ++k) {
                const float z = __shfl_sync(0xFFFFFFFFu, v[k], src);
                if ((lane >> 3) == k) y = z;
            }
            return y;
        };
        // no warp waits without a limit: one that gave up leaves the others to theirs
        for (int sg = 0;; ++sg) {
            if (!warp_wait(&seg_full[sg % kTcaSegSlots], sg / kTcaSegSlots, a.status)) break;
            const volatile TcaSeg& g = segs[sg % kTcaSegSlots];
            const int tiles = g.tiles, tile0 = g.tile0;
            if (tiles == 0) break;
            const bool active = half == 0 || g.rows - g.row0 > 128;
            const bool warp_live = g.row0 + r - lane < g.rows;
            // the rows' last visible tokens, read back where a tile needs masks
            __syncwarp();
            sts32(s_at + (lane << 2), g.row0 + r < g.rows ? g.past + (g.row0 + r) / group : -1);
            __syncwarp();
            // a tile at j0 is open to every row of the half if j0 <= open_hi, > open_lo
            const int open_hi = g.past + (g.row0 + half * 128) / group - (kTcaKT - 1);
            const int open_lo =
                window ? g.past + (min(g.row0 + half * 128 + 128, g.rows) - 1) / group - window : -1;
            float m[4] = {kKvNone, kKvNone, kKvNone, kKvNone};
            float l[4] = {0.f, 0.f, 0.f, 0.f};
            for (int i = 0; i < tiles && ok; ++i, ++c) {
                const int slot = c % kTcaScSlots;
                if (active) ok = warp_wait(&s_full[half], n, a.status);
                if (ok) ok = warp_wait(&sc_full[slot], c / kTcaScSlots, a.status);
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
                const uint32_t sc = sbase + G::off_sc + slot * 1536u + (lane & 3) * 8u;
                const int j0 = (tile0 + i) * kTcaKT;
                // S of columns 16 q .. 16 q + 15: the warp's lanes 0-15, then 16-31
                auto read_s = [&](int q, uint32_t (&v)[16]) {
                    tmem_ld_frag16(ts + 16 * q, v);
                    tmem_ld_frag16(ts + 16 * q + (16u << 16), v + 8);
                };
                // A tile that some row does not see whole: its scores are scaled and masked in
                // tensor memory first, and the pass below finds scales of one and zero.
                uint32_t scx = sc;
                if (!(j0 <= open_hi && j0 > open_lo)) {
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        uint32_t v[16];
                        read_s(q, v);
                        tmem_wait_ld_for(v);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint64_t sk = lds_f2(sc + 64 * q + 32 * y);
                            const uint64_t lg = lds_f2(sc + 512 + 64 * q + 32 * y);
                            const int col = j0 + 16 * q + 8 * y + 2 * (lane & 3);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t* w2 = v + 8 * (k >> 1) + 4 * y + 2 * (k & 1);
                                const int top = static_cast<int>(lds32(s_at + ((8 * k + (lane >> 2)) << 2)));
                                const int low = window ? top - window : INT32_MIN;
                                float u, t;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(w2[0]), __uint_as_float(w2[1])), sk, lg),
                                          u, t);
                                if (col > top || col <= low) u = -INFINITY;
                                if (col + 1 > top || col + 1 <= low) t = -INFINITY;
                                w2[0] = __float_as_uint(u);
                                w2[1] = __float_as_uint(t);
                            }
                        }
                        tmem_st_frag16w(ts + 16 * q, v);
                        tmem_st_frag16w(ts + 16 * q + (16u << 16), v + 8);
                    }
                    tmem_wait_st();
                    scx = sbase + G::off_one + (lane & 3) * 8u;
                }
                // One pass, 32 columns at a time, the next ones' S on its way: x = S sk + lg,
                // p' = 2^(x - m) with the m' known so far, their sum with 1 / sv into l. The
                // packed p' of columns 16 q .. go over columns 8 q .. of S, which have been read.
                // Columns whose maximum is more than kKvTop above m (rare after a segment's
                // first tile) raise m first and rescale what has been added with the old one:
                // l, O and this tile's earlier weights (a second rounding to fp16 for those).
                uint64_t lx[4], neg_m[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lx[k] = f2_pack(l[k], 0.f);
                    neg_m[k] = f2_pack(-m[k], -m[k]);
                }
                uint32_t sv[2][16];
                read_s(0, sv[0]);
                read_s(1, sv[1]);
#pragma unroll 1
                for (int q = 0; q < 8; q += 2) {  // two groups of 16 columns
                    uint64_t x[16];
                    tmem_wait_ld_for(sv[0]);
                    tmem_wait_ld_for(sv[1]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint64_t sk = lds_f2(scx + 64 * q + 32 * y);
                        const uint64_t lg = lds_f2(scx + 512 + 64 * q + 32 * y);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t* w2 = sv[y >> 1] + 8 * (k >> 1) + 4 * (y & 1) + 2 * (k & 1);
                            x[4 * y + k] = f2_fma(f2_pack(__uint_as_float(w2[0]), __uint_as_float(w2[1])), sk, lg);
                        }
                    }
                    if (q < 6) {
                        read_s(q + 2, sv[0]);
                        read_s(q + 3, sv[1]);
                    }
                    float mx[4];
                    bool grow = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float u[4], t[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) f2_unpack(x[4 * y + k], u[y], t[y]);
                        mx[k] = fmaxf(f_max3(f_max3(u[0], t[0], u[1]), t[1], u[2]), f_max3(t[2], u[3], t[3]));
                        grow |= mx[k] > m[k] + kKvTop;
                    }
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        float f[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 1));
                            mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 2));
                            // each row of its own: what the warp's other rows do leaves it alone
                            const float mn = kv_new_max(m[k], mx[k]);
                            f[k] = kv_exp2(m[k] - mn);
                            m[k] = mn;
                            lx[k] = f2_fma(lx[k], f2_pack(f[k], f[k]), 0ull);
                            neg_m[k] = f2_pack(-mn, -mn);
                        }
                        const float fr = by_lane(f);
                        if (i > 0) {
                            ok = warp_wait(&pv_done[half], n - 1, a.status) && ok;
                            tc_fence_after();
#pragma unroll 1
                            for (int o8 = 0; o8 < DP / 8; ++o8) {
                                uint32_t o[8];
                                tmem_ld8(to + 8 * o8, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fr);
                                tmem_st8(to + 8 * o8, o);
                            }
                        }
                        tmem_wait_st();  // the earlier groups' weights
#pragma unroll 1
                        for (int o8 = 0; o8 < q; ++o8) {
                            uint32_t o[8];
                            tmem_ld8(ts + 8 * o8, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __half2 h2 = *reinterpret_cast<__half2*>(&o[e]);
                                o[e] = kv_pack_f16(__low2float(h2) * fr, __high2float(h2) * fr);
                            }
                            tmem_st8(ts + 8 * o8, o);
                        }
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint64_t inv = lds_f2(sc + 1024 + 64 * q + 32 * y);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float u, t;
                            f2_unpack(f2_add(x[4 * y + k], neg_m[k]), u, t);
                            u = kv_exp2(u);
                            t = kv_exp2(t);
                            lx[k] = f2_fma(f2_pack(u, t), inv, lx[k]);
                            p[8 * (y >> 1) + 4 * (k >> 1) + 2 * (y & 1) + (k & 1)] = kv_pack_f16(u, t);
                        }
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        tmem_st_pairs8(ts + 8 * (q + z), p + 8 * z);
                        tmem_st_pairs8(ts + 8 * (q + z) + (16u << 16), p + 8 * z + 4);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float u, t;
                    f2_unpack(lx[k], u, t);
                    l[k] = u + t;
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
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 1);
                l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 2);
            }
            const float ls = by_lane(l), ms = by_lane(m);  // this lane's row's
            // ------------------------------------- end of the segment
            const bool whole = g.whole != 0;
            const int row = g.row0 + r, tok = row / group;
            const bool live = row < g.rows;
            const int head = g.h * group + row - tok * group;
            const int64_t qrow = g.first + tok;
            uint16_t* out = a.out + qrow * a.out_stride + static_cast<int64_t>(head) * a.pool.d;
            auto store_lse = [&](float mm, float ll) {
                if (a.lse)
                    a.lse[qrow * a.q_heads + head] =
                        ll == 0.f ? -INFINITY : 0.69314718f * (mm + __log2f(ll));
            };
            auto inverse = [](float ll) { return ll > 0.f ? __fdiv_rn(1.f, ll) : ll == 0.f ? 0.f : ll; };
            // eight elements of the row from column e0 on
            auto store8 = [&](int e0, float inv, const float (&v)[8]) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = v[e] * inv;
                if (e0 < a.pool.d) *reinterpret_cast<uint4*>(out + e0) = pack8<BF16>(y);
            };
            const int first_cta = g.first_cta, last_cta = g.last_cta;
            if (ok && active && warp_live) {
                ok = warp_wait(&pv_done[half], n - 1, a.status);
                tc_fence_after();
                // a slot: m [256], l [256], O [DP][256] (a column of rows together)
                float* part = a.part + (2 * static_cast<int64_t>(blockIdx.x) + g.slot) * SLOT;
                if (whole) {
                    if (live) store_lse(ms, ls);
                } else {
                    __stcg(part + r, ms);
                    __stcg(part + kTcaRows + r, ls);
                }
                const float inv = inverse(ls);
#pragma unroll 1
                for (int q = 0; q < DP / 16; ++q) {
                    uint32_t o[16];
                    tmem_ld16(to + 16 * q, o);
                    tmem_wait_ld();
                    if (whole) {
                        if (live) {
                            store8(16 * q, inv, *reinterpret_cast<float(*)[8]>(&o[0]));
                            store8(16 * q + 8, inv, *reinterpret_cast<float(*)[8]>(&o[8]));
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
                __syncwarp();
                if (lane == 0) mbar_arrive(&join[0]);
                if (warp == 0) {
                    ok = warp_wait(&join[0], parts, a.status) && ok;
                    if (lane == 0) {
                        const unsigned prev = kv_arrive(a.count + first_cta);
                        s_last = prev == static_cast<unsigned>(last_cta - first_cta);
                        if (s_last) a.count[first_cta] = 0u;  // zero again for the next call
                        mbar_arrive(&join[1]);
                    }
                }
                ok = warp_wait(&join[1], parts, a.status) && ok;
                ++parts;
                if (ok && s_last && active && live) {
                    __threadfence();
                    // only the first of the unit's CTAs can have begun before it
                    const int first_slot = g.first_slot;
                    auto slot_of = [&](int p) -> const float* {
                        return a.part + (2 * static_cast<int64_t>(p) + (p == first_cta ? first_slot : 0)) * SLOT;
                    };
                    float mm = kKvNone;
#pragma unroll 4
                    for (int p = first_cta; p <= last_cta; ++p) mm = fmaxf(mm, __ldcg(slot_of(p) + r));
                    float ll = 0.f;
#pragma unroll 4
                    for (int p = first_cta; p <= last_cta; ++p) {
                        const float* s = slot_of(p);
                        ll = fmaf(__ldcg(s + kTcaRows + r), kv_exp2(__ldcg(s + r) - mm), ll);
                    }
                    store_lse(mm, ll);
                    const float inv = inverse(ll);
#pragma unroll 1
                    for (int e0 = 0; e0 < DP; e0 += 32) {  // 32 loads of a part in flight
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0.f;
#pragma unroll 1
                        for (int p = first_cta; p <= last_cta; ++p) {
                            const float* s = slot_of(p);
                            const float f = kv_exp2(__ldcg(s + r) - mm);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = fmaf(f, __ldcg(s + 2 * kTcaRows + (e0 + e) * kTcaRows + r), v[e]);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            store8(e0 + e, inv, *reinterpret_cast<float(*)[8]>(&v[e]));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_free[sg % kTcaSegSlots]);
        }
    } else if (warp < 12) {
        // --------------------------------------------------- conversion
        constexpr int UPR = DP / 16;       // 16-code units of a row
        constexpr int NI = UPR;            // units of a thread: 128 rows of UPR over 128 threads
        constexpr int RSTEP = 128 / UPR;   // rows between them
        const int d = a.pool.d;
        // The eight lanes of a 128-element row take its first half from row rb and the
        // second from its neighbour, so that their stores hit eight different columns.
        const int ct = tid - 256, u = ct % UPR, rb = (ct / UPR) ^ (u >> 2);
        const bool unit_on = u * 16 < d;
        // units beyond head_dim repeat unit 0: their K meets zeros of Q, their V columns are not stored
        const int8_t* kbase = a.pool.kc + (unit_on ? u * 16 : 0);
        const int8_t* vbase = a.pool.vc + (unit_on ? u * 16 : 0);
        // this thread's units of a tile, by the row offsets that warp 13 left
        auto load = [&](uint4 (&x)[NI], const int8_t* base, uint32_t rows) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint2 o = lds64(rows + static_cast<uint32_t>(rb + i * RSTEP) * 8u);
                x[i] = kv_ldg16(base + ((static_cast<int64_t>(o.y) << 32) | o.x));
            }
        };
        auto rows_of = [&](int c) { return sbase + G::off_row + (c % kTcaRowSlots) * 2048u; };
        bool ok = true;
        int c = 0;
        for (int sg = 0; ok; ++sg) {
            ok = warp_wait(&seg_full[sg % kTcaSegSlots], sg / kTcaSegSlots, a.status);
            if (!ok) break;
            const volatile TcaSeg& g = segs[sg % kTcaSegSlots];
            const int tiles = g.tiles;
            if (tiles == 0) break;
            uint4 kr[NI], vr[NI];
            ok = warp_wait(&row_full[c % kTcaRowSlots], c / kTcaRowSlots, a.status);
            if (!ok) break;
            load(kr, kbase, rows_of(c));
            load(vr, vbase, rows_of(c) + 1024u);
            __syncwarp();
            if (lane == 0) mbar_arrive(&row_free[c % kTcaRowSlots]);

            // the unit's queries, once the products of the last one have read theirs
            if (sg > 0) ok = warp_wait(q_free, sg - 1, a.status);
            if (!ok) break;
            {
                constexpr int CPR = DP / 8;  // 16-byte chunks of a row
                const int rows = g.rows, row0 = g.row0, h = g.h;
                const int64_t first = g.first;
                const int qrows = rows - row0 > 128 ? 256 : 128;
                const int ch = ct % CPR;
#pragma unroll 4
                for (int rr = ct / CPR; rr < qrows; rr += 128 / CPR) {
                    const int row = row0 + rr;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (row < rows && ch * 8 < d) {
                        const int tok = row / group;
                        x = *reinterpret_cast<const uint4*>(
                            a.q + (first + tok) * a.q_stride +
                            static_cast<int64_t>(h * group + row - tok * group) * d + ch * 8);
                    }
                    const int rh = rr & 127;
                    sts128(sbase + G::off_q + (rr >> 7) * G::tile + (ch >> 3) * 16384u + rh * 128u +
                               (static_cast<uint32_t>((ch & 7) ^ (rh & 7)) << 4), x);
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(q_full);
                mbar_arrive(&seg_free[sg % kTcaSegSlots]);
            }

            for (int i = 0; i < tiles && ok; ++i, ++c) {
                const int st = c & 1;
                const uint32_t use = static_cast<uint32_t>(c >> 1);  // earlier uses of the stage
                const bool more = i + 1 < tiles;
                const int rs = (c + 1) % kTcaRowSlots;
                if (use > 0) ok = warp_wait(&k_empty[st], use - 1, a.status);
                if (!ok) break;
                {
                    const uint32_t tile = sbase + G::off_k + st * G::tile;
#pragma unroll
                    for (int q = 0; q < NI; ++q) tca_store16<BF16>(tile, rb + q * RSTEP, u, kr[q]);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[st]);
                if (more) {
                    ok = warp_wait(&row_full[rs], (c + 1) / kTcaRowSlots, a.status);
                    if (!ok) break;
                    load(kr, kbase, rows_of(c + 1));
                }
                if (use > 0) ok = warp_wait(&v_empty[st], use - 1, a.status);
                if (!ok) break;
                {
                    const uint32_t tile = sbase + G::off_v + st * G::tile;
#pragma unroll
                    for (int q = 0; q < NI; ++q) tca_store16<false>(tile, rb + q * RSTEP, u, vr[q]);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_full[st]);
                if (more) {
                    load(vr, vbase, rows_of(c + 1) + 1024u);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&row_free[rs]);
                }
            }
        }
    } else {
        if (warp == 12 && lane == 0) {
            // ---------------------------------------------- MMA issue
            bool ok = true;
            int c = 0;
            uint32_t n[2] = {0, 0};
            // A descriptor's low word is an address and grows by constants from step to
            // step.  (Where this thread had 40 registers the loop's descriptors were computed
            // ahead of it and spilled: with shared memory this full there is next to no L1, each
            // reload took 350 cycles, and a tile 17,000.)
            auto desc = [](uint32_t lo, uint32_t hi) {
                uint64_t v;
                asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
                return v;
            };
            const uint64_t kd = umma_desc_sw128_kmajor(sbase), nd = umma_desc_sw128_nmajor(sbase, 16384u);
            const uint32_t klo = static_cast<uint32_t>(kd), khi = static_cast<uint32_t>(kd >> 32);
            const uint32_t nlo = static_cast<uint32_t>(nd), nhi = static_cast<uint32_t>(nd >> 32);
            auto issue_s = [&](int half, int st) {
                const uint32_t q = klo + ((G::off_q + half * G::tile) >> 4);
                const uint32_t k = klo + ((G::off_k + st * G::tile) >> 4);
                const uint32_t ds = tbase + half * 128;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                    umma_f16_ss(ds, desc(q + off, khi), desc(k + off, khi), kIdescS, kk > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[half]);
            };
            auto issue_pv = [&](int half, int st, bool add) {
                const uint32_t v = nlo + ((G::off_v + st * G::tile) >> 4);
                const uint32_t ds = tbase + kColO + half * DP, pa = tbase + half * 128;
#pragma unroll
                for (int kk = 0; kk < kTcaKT / 16; ++kk)
                    umma_f16_ts(ds, pa + kk * 8, desc(v + kk * 128u, nhi), kIdescO,
                                (add || kk > 0) ? 1u : 0u);
                umma_commit(&pv_done[half]);
            };
            auto wait = [&](uint64_t* b, uint32_t ph) {
                if (ok) ok = mbar_wait_poll(b, ph & 1u, a.status);
                tc_fence_after();
                return ok;
            };
            for (int sg = 0; ok; ++sg) {
                if (!wait(&seg_full[sg % kTcaSegSlots], sg / kTcaSegSlots)) break;
                const volatile TcaSeg& g = segs[sg % kTcaSegSlots];
                const int tiles = g.tiles;
                if (tiles == 0) break;
                const bool both = g.rows - g.row0 > 128;
                mbar_arrive(&seg_free[sg % kTcaSegSlots]);
                if (!wait(q_full, sg)) break;
                if (!wait(&k_full[c & 1], c >> 1)) break;
                issue_s(0, c & 1);
                if (both) issue_s(1, c & 1);
                umma_commit(&k_empty[c & 1]);
                if (tiles == 1) umma_commit(q_free);
                for (int i = 0; i < tiles; ++i, ++c) {
                    const int st = c & 1, sn = (c + 1) & 1;
                    const bool more = i + 1 < tiles;
                    if (!wait(&v_full[st], c >> 1)) break;
                    if (!wait(&p_ready[0], n[0]++)) break;
                    issue_pv(0, st, i > 0);
                    if (more) {
                        if (!wait(&k_full[sn], (c + 1) >> 1)) break;
                        issue_s(0, sn);
                    }
                    if (both) {
                        if (!wait(&p_ready[1], n[1]++)) break;
                        issue_pv(1, st, i > 0);
                    }
                    umma_commit(&v_empty[st]);
                    if (more) {
                        if (both) issue_s(1, sn);
                        umma_commit(&k_empty[sn]);
                        if (i + 2 == tiles) umma_commit(q_free);
                    }
                }
            }
            // every MMA has completed before tensor memory is released
            umma_commit(drain);
            mbar_wait_bounded(drain, 0, a.status, kWaitLimitNs);
        } else if (warp == 13) {
            // ------------------------------- row addresses and scales
            const KvPool& pc = a.pool;
            const int shift = (pc.ps & (pc.ps - 1)) == 0 ? 31 - __clz(pc.ps) : -1;
            auto page_index = [&](int j) { return shift >= 0 ? j >> shift : j / pc.ps; };
            bool ok = true;
            int c = 0, sg = 0;
            KvSeq seq{};
            if (beg < end) seq = kv_seq(a.batch, w.b, a.status);
            for (int64_t it = beg; ok; ++sg) {
                // the next segment, or the end of the list
                TcaSeg g{};
                if (it < end) {
                    int lo;
                    const int n = kv_tiles(a.geom, seq, w.rt, &lo);
                    const int64_t unit_beg = it - w.tile, unit_end = unit_beg + n;
                    g.first = seq.first;
                    g.past = seq.len - seq.n;
                    g.rows = seq.n * group;
                    g.row0 = w.rt * kTcaRows;
                    g.h = w.h;
                    g.tile0 = lo + w.tile;
                    g.tiles = static_cast<int>(min(unit_end, end) - it);
                    g.whole = it == unit_beg && it + g.tiles == unit_end;
                    g.slot = it == beg ? 0 : 1;
                    const int64_t fc = kv_owner(unit_beg, T, P);
                    g.first_cta = static_cast<int>(fc);
                    g.last_cta = static_cast<int>(kv_owner(unit_end - 1, T, P));
                    g.first_slot = T * fc / P >= unit_beg - a.geom.lead ? 0 : 1;
                }
                const int gs = sg % kTcaSegSlots;
                if (sg >= kTcaSegSlots) ok = warp_wait(&seg_free[gs], sg / kTcaSegSlots - 1, a.status);
                if (!ok) break;
                if (lane == 0) {
                    segs[gs] = g;
                    mbar_arrive(&seg_full[gs]);
                }
                __syncwarp();
                if (g.tiles == 0) break;
                int j = g.tile0 * kTcaKT + lane;
                int32_t ent[4];
                auto entries = [&](int jj) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ent[e] = jj + 32 * e < seq.len
                                     ? kv_entry(a.batch, w.b, page_index(jj + 32 * e)) : 0;
                };
                entries(j);
                for (int i = 0; i < g.tiles; ++i, ++c, j += kTcaKT) {
                    const int rs = c % kTcaRowSlots, ss = c % kTcaScSlots;
                    if (c >= kTcaRowSlots) ok = warp_wait(&row_free[rs], c / kTcaRowSlots - 1, a.status);
                    if (!ok) break;
                    uint16_t ks[4], vs[4];
                    const uint32_t rows = sbase + G::off_row + rs * 2048u + lane * 8u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int64_t ko = 0, vo = 0;  // no token: any row, its scores are masked
                        ks[e] = vs[e] = 0;
                        if (j + 32 * e < seq.len) {
                            const int64_t page = kv_page(pc, ent[e], a.status);
                            const int64_t row =
                                kv_row(pc, w.h, j + 32 * e - page_index(j + 32 * e) * pc.ps);
                            ko = page * pc.kc_page + row * pc.d;
                            vo = page * pc.vc_page + row * pc.d;
                            ks[e] = kv_ld(pc.ks + page * pc.ks_page + row);
                            vs[e] = kv_ld(pc.vs + page * pc.vs_page + row);
                        }
                        sts64(rows + 256u * e, static_cast<uint64_t>(ko));
                        sts64(rows + 1024u + 256u * e, static_cast<uint64_t>(vo));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&row_full[rs]);
                    if (i + 1 < g.tiles) entries(j + kTcaKT);
                    if (c >= kTcaScSlots) ok = warp_wait(&sc_free[ss], c / kTcaScSlots - 1, a.status);
                    if (!ok) break;
                    float* sc = reinterpret_cast<float*>(smem + G::off_sc) + ss * 384 + lane;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const KvVScale v = kv_vscale(cache_value<BF16>(vs[e]));
                        const bool in = j + 32 * e < seq.len;
                        sc[32 * e] = cache_value<BF16>(ks[e]) * a.scale_log2;
                        sc[128 + 32 * e] = in ? v.lg : 0.f;
                        sc[256 + 32 * e] = in ? v.inv : 0.f;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[ss]);
                }
                it += g.tiles + a.geom.lead;
                if (it < end) kv_next_unit(a.batch, a.geom, &w, &seq, a.status);
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

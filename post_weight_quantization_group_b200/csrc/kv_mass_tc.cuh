// kv_mass_tc.cuh -- the attention weight that cached tokens received from
// chunks of new tokens, on the tcgen05 tensor cores (head_dim up to 128):
//   mass[j, h] += sum over the rows r that see j of exp(S[r, j] - lse_r).
//
// The keys stay and the rows go by: a unit is 128 tokens of a sequence and KV
// head, converted once to 16-bit floats as the A operand of S^T = K Q^T; the
// rows pass as tiles of 128 (B, copied by cp.async into the swizzled layout).
// A lane of tensor memory is a token, so its scale is a register, its sum a
// thread's own, and no row statistics are carried: per element one packed FMA
// (S sk - lse), one exponential, one packed add.  Bound by the exponentials
// (16 a clock and SM): 128 x 128 of them take 1024 cycles, the MMA 512.
//
// Measured (B200): 256 new tokens over 32,768, 64 query heads over 8 of 128,
// 256 us (the exponentials alone: 119).
//
//   warps 0-3, 4-7   exponentials and sums of the even / odd row tiles (one
//                    accumulator buffer each); their sums of a unit are joined
//                    in a fixed order and added to the mass once per token
//   warps 8-11       copies: the unit's K (converted), the row tiles and their
//                    log-sum-exps
//   warp 12          tcgen05.mma issue
//   warp 13          walks the CTA's units
#pragma once

#include <stdint.h>

#include "kv_attention_tc.cuh"

namespace q4dev {

struct KvMassTc {
    KvPool pool;
    KvBatch batch;
    int group, window, q_heads;
    const uint16_t* q;
    const float* lse;  // [tokens, q_heads]
    float* mass;       // [pages, heads, page_size], pages mass_page apart
    int64_t q_stride, mass_page;
    float scale_log2;
    unsigned* status;
};

constexpr int kTcmQStages = 3;
constexpr int kTcmLsSlots = 4;
constexpr int kTcmUnits = 4;  // units in flight between the roles

// A unit: tokens j0 .. of sequence b and head h, seen by rows [r_lo, r_hi);
// tiles = 0 ends the list.
struct TcmUnit {
    int64_t first;  // the sequence's first row of q
    int b, h, j0, len, past, r_lo, r_hi, tiles;
    int pad[6];
};
static_assert(sizeof(TcmUnit) == 64, "unit ring");

template <int DP>
struct TcmGeom {
    static constexpr uint32_t tile = DP * 256;
    static constexpr uint32_t off_k = 0;  // two units
    static constexpr uint32_t off_q = 2 * tile;
    static constexpr uint32_t off_ls = off_q + kTcmQStages * tile;    // -lse [128], last visible token [128]
    static constexpr uint32_t off_sum = off_ls + kTcmLsSlots * 1024;  // the odd tiles' sums
    static constexpr uint32_t off_unit = off_sum + 512;
    static constexpr uint32_t off_bar = off_unit + kTcmUnits * 64;
    static constexpr uint32_t total = off_bar + 512 + 1024;
};

// Row tiles of 128 that a sequence's keys cost each (the whole of its rows).
__device__ __forceinline__ int tcm_rows(const KvMassTc& a, const KvSeq& s) {
    return (s.n * a.group + 127) / 128;
}
// Key tiles of a sequence that its new tokens may see.
__device__ __forceinline__ int tcm_keys(const KvMassTc& a, const KvSeq& s, int* lo) {
    const int first = a.window ? max(s.len - s.n + 1 - a.window, 0) : 0;
    *lo = first / 128;
    return s.n > 0 ? max((s.len + 127) / 128 - *lo, 0) : 0;
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kTcaThreads, 1) kv_mass_tc_kernel(const __grid_constant__ KvMassTc a) {
    using G = TcmGeom<DP>;
    constexpr uint32_t kIdesc = umma_idesc_f16<BF16, 128, 128>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::off_bar);
    uint64_t* k_full = bars;       // [2]
    uint64_t* k_free = bars + 2;   // [2]
    uint64_t* d_full = bars + 4;   // [2] accumulators
    uint64_t* d_free = bars + 6;   // [2]
    uint64_t* q_full = bars + 8;   // [kTcmQStages]
    uint64_t* q_free = q_full + kTcmQStages;
    uint64_t* ls_full = q_free + kTcmQStages;  // [kTcmLsSlots]
    uint64_t* ls_free = ls_full + kTcmLsSlots;
    uint64_t* u_full = ls_free + kTcmLsSlots;  // [kTcmUnits]
    uint64_t* u_free = u_full + kTcmUnits;
    uint64_t* sum_full = u_free + kTcmUnits;
    uint64_t* sum_free = sum_full + 1;
    uint64_t* drain = sum_full + 2;
    uint32_t* tbase_s = reinterpret_cast<uint32_t*>(sum_full + 3);
    TcmUnit* units = reinterpret_cast<TcmUnit*>(smem + G::off_unit);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_free[i], 1);
            mbar_init(&d_full[i], 1);
            mbar_init(&d_free[i], 4);
        }
        for (int i = 0; i < kTcmQStages; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&q_free[i], 1);
        }
        for (int i = 0; i < kTcmLsSlots; ++i) {
            mbar_init(&ls_full[i], 4);
            mbar_init(&ls_free[i], 4);
        }
        for (int i = 0; i < kTcmUnits; ++i) {
            mbar_init(&u_full[i], 1);
            mbar_init(&u_free[i], 13);  // 8 summing and 4 copying warps, the MMA thread
        }
        mbar_init(sum_full, 4);
        mbar_init(sum_free, 4);
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 12) tmem_alloc(tbase_s, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tbase_s;
    grid_launch_dependents();
    grid_dependency_wait();

    if (warp < 8) {
        // ------------------------------------------ exponentials and sums
        const int wg = warp >> 2, key = (warp & 3) * 32 + lane;
        const uint32_t td = tbase + wg * 128 + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        float* s_sum = reinterpret_cast<float*>(smem + G::off_sum);
        int t = 0;         // row tiles so far: the log-sum-exps' slot
        uint32_t n = 0;    // this group's of them
        bool ok = true;
        for (int u = 0; ok; ++u) {
            ok = warp_wait(&u_full[u % kTcmUnits], u / kTcmUnits, a.status);
            if (!ok) break;
            const volatile TcmUnit& g = units[u % kTcmUnits];
            const int tiles = g.tiles, j = g.j0 + key;
            if (tiles == 0) break;
            bool live = j < g.len;
            float sk = 0.f;
            int64_t place = 0;
            if (live) {
                const int e = j / a.pool.ps;
                const int32_t entry = kv_entry(a.batch, g.b, e);
                live = kv_valid_page(a.pool, entry, a.status);  // else there is nothing to add to
                const int64_t page = live ? entry : 0;
                const int64_t row = kv_row(a.pool, g.h, j - e * a.pool.ps);
                sk = cache_value<BF16>(kv_ld(a.pool.ks + page * a.pool.ks_page + row)) * a.scale_log2;
                place = page * a.mass_page + row;
            }
            const uint64_t sk2 = f2_pack(sk, sk);
            // a row tile is open if its first row sees the unit's last token and, under a
            // window, its last row still the first
            const int j0 = g.j0, past = g.past, r_lo = g.r_lo, r_hi = g.r_hi;
            uint64_t sum2[2] = {0ull, 0ull};
            for (int i = 0; i < tiles && ok; ++i, ++t) {
                if ((t & 1) != wg) continue;
                const int slot = t % kTcmLsSlots;
                ok = warp_wait(&d_full[wg], n, a.status) &&
                     warp_wait(&ls_full[slot], t / kTcmLsSlots, a.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ls = sbase + G::off_ls + slot * 1024u;
                const int r0 = r_lo + i * 128, r1 = min(r0 + 128, r_hi) - 1;
                const bool open = past + r0 / a.group >= j0 + 127 &&
                                  (!a.window || past + r1 / a.group - a.window < j0);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[32];
                    tmem_ld16(td + 32 * q, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
                    tmem_ld16(td + 32 * q + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
                    uint4 l4[8];  // -lse of the chunk's rows
#pragma unroll
                    for (int e = 0; e < 8; ++e) l4[e] = lds128(ls + 128u * q + 16u * e);
                    tmem_wait_ld();
                    float x[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t lw[4] = {l4[e].x, l4[e].y, l4[e].z, l4[e].w};
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            float y0, y1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[4 * e + 2 * z]),
                                                     __uint_as_float(v[4 * e + 2 * z + 1])),
                                             sk2, f2_pack(__uint_as_float(lw[2 * z]), __uint_as_float(lw[2 * z + 1]))),
                                      y0, y1);
                            x[4 * e + 2 * z] = kv_exp2(y0);
                            x[4 * e + 2 * z + 1] = kv_exp2(y1);
                        }
                    }
                    if (!open) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int at = static_cast<int>(lds32(ls + 512u + 128u * q + 4u * e));
                            if (j > at || (a.window && j <= at - a.window)) x[e] = 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(x[2 * e], x[2 * e + 1]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&d_free[wg]);
                    mbar_arrive(&ls_free[slot]);
                }
                ++n;
            }
            if (!ok) break;
            float s0, s1, s2, s3;
            f2_unpack(sum2[0], s0, s1);
            f2_unpack(sum2[1], s2, s3);
            const float sum = (s0 + s1) + (s2 + s3);
            // the odd tiles' sums to the even ones', one unit after another
            if (wg == 1) {
                if (u > 0) ok = warp_wait(sum_free, u - 1, a.status);
                if (!ok) break;
                s_sum[key] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(sum_full);
            } else {
                ok = warp_wait(sum_full, u, a.status);
                if (!ok) break;
                const float total = sum + s_sum[key];
                __syncwarp();
                if (lane == 0) mbar_arrive(sum_free);
                if (live) atomicAdd(a.mass + place, total);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_free[u % kTcmUnits]);
        }
    } else if (warp < 12) {
        // ----------------------------------------------------------- copies
        constexpr int UPR = DP / 16, NI = UPR, RSTEP = 128 / UPR;
        constexpr int CPR = DP / 8, QSTEP = 128 / CPR;  // 16-byte chunks of a row of Q, rows a step
        const int d = a.pool.d;
        const int ct = tid - 256, un = ct % UPR, rb = (ct / UPR) ^ (un >> 2);
        const int ucol = un * 16 < d ? un * 16 : 0;  // columns beyond head_dim meet zeros of Q
        const int ch = ct % CPR;
        const int step_r = QSTEP % a.group;
        const int64_t step = QSTEP / a.group * a.q_stride + static_cast<int64_t>(step_r) * d;
        const int64_t wrap = a.q_stride - static_cast<int64_t>(a.group) * d;  // to the next token's head 0
        int t = 0;
        bool ok = true;
        // a row tile's copies arrive while the next one's are issued
        int pending = -1;
        auto arrived = [&]() {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&q_full[pending % kTcmQStages]);
                mbar_arrive(&ls_full[pending % kTcmLsSlots]);
            }
            pending = -1;
        };
        for (int u = 0; ok; ++u) {
            ok = warp_wait(&u_full[u % kTcmUnits], u / kTcmUnits, a.status);
            if (!ok) break;
            const volatile TcmUnit& g = units[u % kTcmUnits];
            const int tiles = g.tiles;
            if (tiles == 0) {
                if (pending >= 0) {
                    kv_cp_wait<0>();
                    arrived();
                }
                break;
            }
            const int b = g.b, h = g.h, j0 = g.j0, len = g.len, past = g.past, r_lo = g.r_lo, r_hi = g.r_hi;
            const int64_t first = g.first;
            // the unit's K
            {
                uint4 kr[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int j = min(j0 + rb + i * RSTEP, len - 1);  // tokens behind the last repeat it
                    const int e = j / a.pool.ps;
                    const int64_t page = kv_page(a.pool, kv_entry(a.batch, b, e), a.status);
                    kr[i] = kv_ldg16(a.pool.kc + page * a.pool.kc_page +
                                     kv_row(a.pool, h, j - e * a.pool.ps) * d + ucol);
                }
                if (pending >= 0) {
                    kv_cp_wait<0>();
                    arrived();
                }
                if (u >= 2) ok = warp_wait(&k_free[u & 1], u / 2 - 1, a.status);
                if (!ok) break;
                const uint32_t tile = sbase + G::off_k + (u & 1) * G::tile;
#pragma unroll
                for (int i = 0; i < NI; ++i) tca_store16<BF16>(tile, rb + i * RSTEP, un, kr[i]);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[u & 1]);
            }
            for (int i = 0; i < tiles && ok; ++i, ++t) {
                const int st = t % kTcmQStages, slot = t % kTcmLsSlots;
                if (t >= kTcmQStages) ok = warp_wait(&q_free[st], t / kTcmQStages - 1, a.status);
                if (ok && t >= kTcmLsSlots) ok = warp_wait(&ls_free[slot], t / kTcmLsSlots - 1, a.status);
                if (!ok) break;
                const int r0 = r_lo + i * 128;
                const uint32_t q0 = sbase + G::off_q + st * G::tile;
                // row by row of this thread's: QSTEP rows on are step_t tokens and step_r heads
                const int tok0 = (r0 + ct / CPR) / a.group;
                int rem = r0 + ct / CPR - tok0 * a.group;
                const uint16_t* src = a.q + (first + tok0) * a.q_stride +
                                      static_cast<int64_t>(h * a.group + rem) * d + ch * 8;
                const uint32_t dst0 = q0 + (ch >> 3) * 16384u + (ct / CPR) * 128u;
#pragma unroll
                for (int x = 0; x < 128 / QSTEP; ++x) {
                    const int rr = ct / CPR + x * QSTEP;
                    const uint32_t dst = dst0 + x * QSTEP * 128u +
                                         (static_cast<uint32_t>((ch & 7) ^ (rr & 7)) << 4);
                    if (r0 + rr < r_hi && ch * 8 < d)
                        kv_cp16(dst, src);
                    else
                        sts128(dst, make_uint4(0u, 0u, 0u, 0u));
                    src += step;
                    rem += step_r;
                    if (rem >= a.group) {
                        rem -= a.group;
                        src += wrap;
                    }
                }
                {
                    const int row = r0 + ct;
                    float nl = -INFINITY;  // a row that is none: its weights are 2^-inf
                    int at = -1;
                    if (row < r_hi) {
                        const int tok = row / a.group;
                        nl = -1.44269504f * kv_ld(a.lse + (first + tok) * a.q_heads + h * a.group + row -
                                                  tok * a.group);
                        at = past + tok;
                    }
                    float* ls = reinterpret_cast<float*>(smem + G::off_ls + slot * 1024u);
                    ls[ct] = nl;
                    reinterpret_cast<int*>(ls)[128 + ct] = at;
                }
                kv_cp_commit();
                if (pending >= 0) {
                    kv_cp_wait<1>();
                    arrived();
                }
                pending = t;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_free[u % kTcmUnits]);
        }
        kv_cp_wait<0>();  // none in flight at the exit, whatever ended the loop
    } else if (warp == 12 && lane == 0) {
        // -------------------------------------------------------- MMA issue
        auto opaque = [](uint32_t v) {
            asm volatile("" : "+r"(v));
            return v;
        };
        auto desc = [](uint32_t lo, uint32_t hi) {
            uint64_t v;
            asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
            return v;
        };
        const uint64_t kd = umma_desc_sw128_kmajor(sbase);
        const uint32_t klo = static_cast<uint32_t>(kd), khi = static_cast<uint32_t>(kd >> 32);
        bool ok = true;
        auto wait = [&](uint64_t* b, uint32_t ph) {
            if (ok) ok = mbar_wait_poll(b, ph & 1u, a.status);
            tc_fence_after();
            return ok;
        };
        int t = 0;
        for (int u = 0; ok; ++u) {
            if (!wait(&u_full[u % kTcmUnits], u / kTcmUnits)) break;
            const int tiles = static_cast<const volatile TcmUnit&>(units[u % kTcmUnits]).tiles;
            if (tiles == 0) break;
            mbar_arrive(&u_free[u % kTcmUnits]);
            if (!wait(&k_full[u & 1], u / 2)) break;
            for (int i = 0; i < tiles; ++i, ++t) {
                const int st = t % kTcmQStages, buf = t & 1;
                if (!wait(&q_full[st], t / kTcmQStages)) break;
                if (t >= 2 && !wait(&d_free[buf], t / 2 - 1)) break;
                const uint32_t k = opaque(klo + ((G::off_k + (u & 1) * G::tile) >> 4));
                const uint32_t q = opaque(klo + ((G::off_q + st * G::tile) >> 4));
                const uint32_t dd = opaque(tbase + buf * 128);
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                    umma_f16_ss(dd, desc(k + off, khi), desc(q + off, khi), kIdesc, kk > 0 ? 1u : 0u);
                }
                umma_commit(&d_full[buf]);
                umma_commit(&q_free[st]);
            }
            umma_commit(&k_free[u & 1]);
        }
        umma_commit(drain);
        mbar_wait_bounded(drain, 0, a.status, kWaitLimitNs);
    } else if (warp == 13) {
        // ------------------------------------------------------------ units
        // The sequences' units lie one after another, each as long as its row tiles; this
        // CTA takes those that begin in its share of the whole.
        auto work = [&](int b, int* keys, int* rt) -> int64_t {
            const KvSeq s = kv_seq(a.batch, b, a.status);
            int lo;
            *keys = tcm_keys(a, s, &lo);
            *rt = tcm_rows(a, s);
            return static_cast<int64_t>(*keys) * a.pool.heads * *rt;
        };
        int64_t all = 0;
        int keys, rt;
        for (int b = lane; b < a.batch.seqs; b += 32) all += work(b, &keys, &rt);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
        const int64_t beg = all * blockIdx.x / gridDim.x, end = all * (blockIdx.x + 1) / gridDim.x;
        // the sequence that holds place beg, and its own first place
        int b = 0;
        int64_t x0 = 0;
        for (int b0 = 0; b0 < a.batch.seqs; b0 += 32) {
            int64_t mine = b0 + lane < a.batch.seqs ? work(b0 + lane, &keys, &rt) : 0, incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned past_beg = __ballot_sync(0xFFFFFFFFu, x0 + incl > beg);
            if (past_beg) {
                const int f = __ffs(past_beg) - 1;
                b = b0 + f;
                x0 += __shfl_sync(0xFFFFFFFFu, incl - mine, f);
                break;
            }
            x0 += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        bool ok = true;
        int u = 0;
        if (beg < end) {
            int64_t size = work(b, &keys, &rt);
            int64_t at = (beg - x0 + rt - 1) / rt;  // unit of the sequence
            while (ok) {
                if (at * rt >= size) {  // on to the next sequence that has any
                    x0 += size;
                    if (++b >= a.batch.seqs || x0 >= end) break;
                    size = work(b, &keys, &rt);
                    at = 0;
                    continue;
                }
                if (x0 + at * rt >= end) break;
                const KvSeq s = kv_seq(a.batch, b, a.status);
                int lo;
                tcm_keys(a, s, &lo);
                TcmUnit g{};
                g.first = s.first;
                g.b = b;
                g.h = static_cast<int>(at / keys);
                g.j0 = (lo + static_cast<int>(at - static_cast<int64_t>(g.h) * keys)) * 128;
                g.len = s.len;
                g.past = s.len - s.n;
                // rows that see any of the unit's tokens
                g.r_lo = max(g.j0 - g.past, 0) * a.group;
                g.r_hi = static_cast<int>(a.window ? min(static_cast<int64_t>(s.n),
                                                         static_cast<int64_t>(g.j0) + 127 + a.window - g.past)
                                                   : static_cast<int64_t>(s.n)) * a.group;
                g.tiles = max((g.r_hi - g.r_lo + 127) / 128, 0);
                ++at;
                if (g.tiles == 0) continue;
                const int gs = u % kTcmUnits;
                if (u >= kTcmUnits) ok = warp_wait(&u_free[gs], u / kTcmUnits - 1, a.status);
                if (!ok) break;
                if (lane == 0) {
                    units[gs] = g;
                    mbar_arrive(&u_full[gs]);
                }
                __syncwarp();
                ++u;
            }
        }
        // the end of the list
        if (ok && u >= kTcmUnits) ok = warp_wait(&u_free[u % kTcmUnits], u / kTcmUnits - 1, a.status);
        if (ok && lane == 0) {
            units[u % kTcmUnits] = TcmUnit{};
            mbar_arrive(&u_full[u % kTcmUnits]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tbase, 256);
    }
}

}  // namespace q4dev

// kv_paged.cuh -- the paged INT8 KV cache: the device view of a layer's pool
// and of a batch of sequences, the write of new tokens (query / key norm,
// rotation, quantization, one pass) and the read-back of cached rows.
//
// A pool holds pages of [heads, page_size] rows of head_dim codes with one
// scale per row, quantized as kv_quantize_int8 does ("压缩算法"
// (cs-knowledge-wiki) section 7.4.1.1): s = cache_type(amax / 127),
// q = clamp(rne(x / s), -128, 127).
#pragma once

#include <stdint.h>

#include "q4_device.cuh"
#include "q8_codes.cuh"

namespace q4dev {

// A load of what another kernel of the stream may have written: a plain one.
// These kernels begin while the one ahead of them still runs (programmatic
// launch), so nothing they read is constant for as long as they run, which is
// what the read-only path asks for: a line of it that an earlier kernel left in
// the SM could be stale.
template <typename T>
__device__ __forceinline__ T kv_ld(const T* p) {
    return *p;
}

struct KvPool {
    int8_t *kc, *vc;
    uint16_t *ks, *vs;
    int64_t kc_page, vc_page, ks_page, vs_page;  // elements from a page to the next
    int64_t pages;
    int heads, ps, d;
};

// Element offset of a cached row's scale inside its page; times d, of its codes.
__device__ __forceinline__ int64_t kv_row(const KvPool& c, int head, int off) {
    return static_cast<int64_t>(head) * c.ps + off;
}

struct KvBatch {
    const int32_t* table;  // [seqs, width] page of every page_size cached tokens
    const int32_t* lens;   // [seqs] cached tokens, the new ones among them
    const int32_t* cu;     // [seqs + 1] first new token of each sequence; null: one each
    int64_t width;
    int64_t tokens;        // rows of q
    int seqs;
    int cap;               // tokens that a table row can name
};

struct KvSeq {
    int len, n;     // cached tokens, new tokens
    int64_t first;  // the first new token's row of q
};

// A sequence's extents, brought into range (and the caller told) where the
// device arrays say more than the buffers hold.
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int i, unsigned* status) {
    KvSeq s;
    int len = kv_ld(b.lens + i);
    int64_t lo, hi;
    if (b.cu) {
        lo = kv_ld(b.cu + i);
        hi = kv_ld(b.cu + i + 1);
    } else {
        lo = i;
        hi = i + 1;
    }
    if (len < 0 || len > b.cap || lo < 0 || hi < lo || hi > b.tokens) {
        atomicOr(status, kStatusBadIndex);
        len = min(max(len, 0), b.cap);
        lo = min(max(lo, int64_t(0)), b.tokens);
        hi = min(max(hi, lo), b.tokens);
    }
    s.len = len;
    s.first = lo;
    s.n = static_cast<int>(hi - lo);
    return s;
}

// Table entry e of sequence i, and the page it names, brought into [0, pages)
// likewise.  Two steps, so that a kernel can load an entry ahead of its use.
__device__ __forceinline__ int32_t kv_entry(const KvBatch& b, int i, int e) {
    return kv_ld(b.table + static_cast<int64_t>(i) * b.width + e);
}
__device__ __forceinline__ bool kv_valid_page(const KvPool& c, int32_t entry, unsigned* status) {
    if (entry >= 0 && entry < c.pages) return true;
    atomicOr(status, kStatusBadIndex);
    return false;
}
// For reads; nothing is written to a page that was not named.
__device__ __forceinline__ int64_t kv_page(const KvPool& c, int32_t entry, unsigned* status) {
    return kv_valid_page(c, entry, status) ? entry : entry < 0 ? 0 : c.pages - 1;
}

// ---------------------------------------------------------------- append

struct KvAppend {
    KvPool pool;
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, qo_stride;  // elements from a token to the next
    const uint16_t *q_norm, *k_norm;                  // [d] or null
    const int64_t* slots;
    const int32_t* positions;
    const float* inv_freq;  // [rot / 2]
    float* mass;            // [pages, heads, page_size], pages mass_page apart, or null
    int64_t mass_page;
    int64_t tokens;
    int q_heads, rot, heads_per_cta;
    float eps;
    unsigned* status;
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = cache_value<BF16>(static_cast<uint16_t>(w[i] & 0xFFFFu));
        v[2 * i + 1] = cache_value<BF16>(static_cast<uint16_t>(w[i] >> 16));
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        else
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA takes a token's heads (or heads_per_cta of them: blockIdx.y), a team
// of TS lanes one head, a lane eight consecutive elements (d <= 8 TS), so the
// norm and the row maximum are shuffles and nothing of a row is read twice.
// The heads run q, k, v.  The angles of a token are the same for all of its
// heads: they are computed once per CTA while the token before is worked on, and
// a lane keeps its eight of them in registers:
//   pos * inv_freq in turns, reduced in fp64 (53 bits keep a position of 2^31
//   within 2e-7 of a turn), then sine and cosine of the remainder in fp32.
// K is quantized from its fp32 rotated value: a rounding to the cache type in
// between would add an error of its own.  Every element is read and written
// once; the instruction rate is its nearest bound (0.71 of the issue slots, half of HBM's rate), so a warp
// whose heads are all queries has a path of its own, without the quantization
// and without branches (8191 tokens of 64/8 heads of 128: 98 us, 3.1 TB/s; with
// branches and one path 130; three heads under way instead of one 98; the
// weights multiplied into the angles and packed fp32 pairs 103, as they cost
// each token more than its five heads a warp save).  PAIRS: interleaved rotation.
template <bool BF16, int TS, bool PAIRS>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const __grid_constant__ KvAppend a) {
    constexpr int TEAMS = 256 / TS;
    __shared__ float2 cs[2][128];
    grid_launch_dependents();
    grid_dependency_wait();
    const KvPool& c = a.pool;
    const int d = c.d, sub = threadIdx.x % TS, team = threadIdx.x / TS;
    const int lane0 = (threadIdx.x & 31) - sub;  // first lane of the team
    const int half = a.rot >> 1, hl = half >> 3;
    const bool on = sub * 8 < d;
    const int h_beg = blockIdx.y * a.heads_per_cta;
    const int h_end = min(h_beg + a.heads_per_cta, a.q_heads + 2 * c.heads);
    const int shift = (c.ps & (c.ps - 1)) == 0 ? 31 - __clz(c.ps) : -1;
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if (on && a.q_norm) wq = kv_ld(reinterpret_cast<const uint4*>(a.q_norm) + sub);
    if (on && a.k_norm) wk = kv_ld(reinterpret_cast<const uint4*>(a.k_norm) + sub);
    const float inv_d = 1.f / static_cast<float>(d);

    auto load = [&](int64_t tok, int h) -> uint4 {
        if (!on || h >= h_end) return make_uint4(0, 0, 0, 0);
        const uint16_t* p;
        if (h < a.q_heads)
            p = a.q + tok * a.q_stride + h * d;
        else if (h < a.q_heads + c.heads)
            p = a.k + tok * a.k_stride + (h - a.q_heads) * d;
        else
            p = a.v + tok * a.v_stride + (h - a.q_heads - c.heads) * d;
        return *reinterpret_cast<const uint4*>(p + sub * 8);
    };
    auto angles = [&](int64_t tok, float2* to) {
        for (int i = threadIdx.x; i < half; i += 256) {
            double t = static_cast<double>(kv_ld(a.positions + tok)) *
                       static_cast<double>(kv_ld(a.inv_freq + i)) * 0.15915494309189533577;
            t -= rint(t);
            float s, co;
            sincospif(static_cast<float>(2.0 * t), &s, &co);
            to[i] = make_float2(co, s);
        }
    };

    int64_t tok = blockIdx.x;
    if (tok >= a.tokens) return;
    uint4 nxt = load(tok, h_beg + team);
    angles(tok, cs[0]);
    int64_t slot = kv_ld(a.slots + tok);
    __syncthreads();
    for (int buf = 0; tok < a.tokens; buf ^= 1) {
        const int64_t next = tok + gridDim.x;
        // where the token's key and value go
        const int64_t page = shift >= 0 ? slot >> shift : slot / c.ps;
        const int off = static_cast<int>(slot - page * c.ps);
        const bool write = slot >= 0 && page < c.pages;
        if (slot >= 0 && !write && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
        if (next < a.tokens) {
            slot = kv_ld(a.slots + next);
            angles(next, cs[buf ^ 1]);
        }
        // This lane's part of the rotation: v' = v f.x + partner f.y, element by element, or
        // pair by pair.  Elements behind rot_dim keep what they hold, an infinity too.
        float2 f[PAIRS ? 4 : 8];
        const bool lo = sub < hl;
        const int peer = PAIRS ? 0 : lane0 + (lo ? sub + hl : sub < 2 * hl ? sub - hl : sub);
#pragma unroll
        for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
            const int at = PAIRS ? sub * 4 + i : (lo ? sub : sub - hl) * 8 + i;
            const bool rot = PAIRS ? at < half : sub < 2 * hl;
            f[i] = rot ? cs[buf][at] : make_float2(1.f, 0.f);
            if (!PAIRS && lo) f[i].y = -f[i].y;
        }
        auto rotate = [&](float (&v)[8]) {
            if constexpr (PAIRS) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = v[2 * i], y = v[2 * i + 1];
                    if (sub * 4 + i >= half) continue;
                    v[2 * i] = x * f[i].x - y * f[i].y;
                    v[2 * i + 1] = y * f[i].x + x * f[i].y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = __shfl_sync(0xFFFFFFFFu, v[i], peer);
                    if (sub < 2 * hl) v[i] = fmaf(v[i], f[i].x, y * f[i].y);
                }
            }
        };
        auto normalize = [&](float (&v)[8], const uint4& weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
            for (int o = TS / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            const float r = rsqrtf(ss * inv_d + a.eps);
            float w[8];
            unpack8<BF16>(weight, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
        };
        // uniform over the warp's teams, so that all lanes take part in the shuffles
        const uint16_t* qp = a.q + tok * a.q_stride + sub * 8;
        uint16_t* qo = a.q_out + tok * a.qo_stride + sub * 8;
        for (int hb = h_beg; hb < h_end; hb += TEAMS) {
            const int h = hb + team;
            const uint4 raw = nxt;
            if (hb + 2 * TEAMS <= min(a.q_heads, h_end))
                nxt = on ? *reinterpret_cast<const uint4*>(qp + (h + TEAMS) * d) : make_uint4(0, 0, 0, 0);
            else if (hb + TEAMS < h_end)
                nxt = load(tok, h + TEAMS);
            else if (next < a.tokens)
                nxt = load(next, h_beg + team);
            float v[8];
            unpack8<BF16>(raw, v);
            if (hb + TEAMS <= min(a.q_heads, h_end)) {  // all queries
                if (a.q_norm) normalize(v, wq);
                if (half) rotate(v);
                if (on) *reinterpret_cast<uint4*>(qo + h * d) = pack8<BF16>(v);
                continue;
            }
            const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + c.heads;
            if (__any_sync(0xFFFFFFFFu, !is_v)) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = v[i];
                const uint4 weight = is_q ? wq : wk;
                if (a.q_norm || a.k_norm) {
                    normalize(u, weight);
                    if (is_q ? a.q_norm == nullptr : a.k_norm == nullptr) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = v[i];
                    }
                }
                if (half) rotate(u);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = is_v ? v[i] : u[i];
            }
            if (is_q && on && h < h_end) *reinterpret_cast<uint4*>(qo + h * d) = pack8<BF16>(v);
            if (!__any_sync(0xFFFFFFFFu, !is_q && h < h_end)) continue;
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
            for (int o = TS / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (is_q || !on || h >= h_end || !write) continue;
            const uint16_t sbits = cache_bits<BF16>(__fdiv_rn(m, 127.0f));
            const float s = cache_value<BF16>(sbits);
            const float rs = quot_recip(s);
            uint2 packed = make_uint2(0u, 0u);
            if (s != 0.f) {
                int qc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) qc[i] = int8_code(v[i], s, rs, -128);
                packed = pack8_bytes(qc);
            }
            const int64_t row = kv_row(c, h - a.q_heads - (is_v ? c.heads : 0), off);
            int8_t* codes = (is_v ? c.vc + page * c.vc_page : c.kc + page * c.kc_page) + row * d;
            *reinterpret_cast<uint2*>(codes + sub * 8) = packed;
            if (sub == 0) {
                (is_v ? c.vs + page * c.vs_page : c.ks + page * c.ks_page)[row] = sbits;
                // what the slot's last token received is not the new one's
                if (a.mass && !is_v) a.mass[page * a.mass_page + row] = 0.f;
            }
        }
        __syncthreads();  // the next token's angles are there, and this one's are done with
        tok = next;
    }
}

// Cached rows by slot, dequantized: out[t, h] = cache_type(q * s), one
// rounding of an exact product.  A team per (token, K or V, head).
template <bool BF16, int TS>
__global__ void __launch_bounds__(256)
    kv_gather_kernel(const __grid_constant__ KvPool c, const int64_t* slots, int64_t tokens,
                     uint16_t* k_out, uint16_t* v_out, unsigned* status) {
    constexpr int TEAMS = 256 / TS;
    grid_launch_dependents();
    grid_dependency_wait();
    const int sub = threadIdx.x % TS;
    const int64_t items = tokens * 2 * c.heads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TS; it < items;
         it += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t tok = it / (2 * c.heads);
        const int hh = static_cast<int>(it - tok * (2 * c.heads));
        const int64_t slot = kv_ld(slots + tok);
        const int64_t page = slot / c.ps;
        if (slot < 0 || sub * 8 >= c.d) continue;
        if (page >= c.pages) {
            atomicOr(status, kStatusBadIndex);
            continue;
        }
        const bool is_v = hh >= c.heads;
        const int h = is_v ? hh - c.heads : hh;
        const int64_t row = kv_row(c, h, static_cast<int>(slot - page * c.ps));
        const int8_t* codes = (is_v ? c.vc + page * c.vc_page : c.kc + page * c.kc_page) + row * c.d;
        const float s = cache_value<BF16>((is_v ? c.vs + page * c.vs_page : c.ks + page * c.ks_page)[row]);
        const uint2 raw = *reinterpret_cast<const uint2*>(codes + sub * 8);
        const uint32_t w[2] = {raw.x, raw.y};
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = static_cast<float>(static_cast<int8_t>((w[j >> 2] >> (8 * (j & 3))) & 0xFFu)) * s;
        *reinterpret_cast<uint4*>((is_v ? v_out : k_out) + (tok * c.heads + h) * c.d + sub * 8) =
            pack8<BF16>(o);
    }
}

// ------------------------------------------------------ division of work
//
// The attention kernels split their work by what the device arrays say, with
// no plan from the host: a unit is (sequence, row tile, KV head), rows being
// the new tokens times the query heads of a KV head (row = token * group +
// head, fewer
// than 2^31 - 2^16 of them), R to a tile; a unit's tiles are the KT-token tiles of the cache that
// any of its rows sees, one at least (a unit that sees nothing still writes
// its zeros).  The units lie one after another on a line, each as `lead` empty
// places (what beginning and ending a unit costs, in tiles) and then its
// tiles, and the line is cut into P equal ranges, one per CTA, whatever the
// sequences' lengths.

struct KvGeom {
    int R, KT, group, heads, window, lead;
    // sequences with more than rows_lo and at most rows_hi rows; the others are left alone
    int rows_lo, rows_hi;
};

// Row tiles of a sequence.
__device__ __forceinline__ int kv_row_tiles(const KvGeom& g, const KvSeq& s) {
    const int rows = s.n * g.group;
    return rows > g.rows_lo && rows <= g.rows_hi ? (rows + g.R - 1) / g.R : 0;
}

// Tiles [lo, lo + count) that the rows of tile rt see.
__device__ __forceinline__ int kv_tiles(const KvGeom& g, const KvSeq& s, int rt, int* lo) {
    const int r0 = rt * g.R, r1 = min(r0 + g.R, s.n * g.group) - 1;
    const int t0 = r0 / g.group, t1 = r1 / g.group;
    const int hi = max(s.len - s.n + t1 + 1, 0);
    const int first = g.window ? max(s.len - s.n + t0 + 1 - g.window, 0) : 0;
    *lo = first / g.KT;
    return max((hi + g.KT - 1) / g.KT - *lo, 1);
}

__device__ __forceinline__ int64_t kv_seq_work(const KvGeom& g, const KvSeq& s) {
    const int rts = kv_row_tiles(g, s);
    int64_t sum = 0;
    for (int rt = 0; rt < rts; ++rt) {
        int lo;
        sum += kv_tiles(g, s, rt, &lo) + g.lead;
    }
    return sum * g.heads;
}

// A place in the work: tile `tile` (counted from the unit's first) of unit
// (b, rt, h).
struct KvPlace {
    int b, rt, h, tile;
};

// Inclusive prefix sum over the block (NT threads, a multiple of 32; every
// thread calls); `sums` holds NT / 32 values.  Returns the block's total too.
template <int NT>
__device__ __forceinline__ int64_t kv_block_scan(int64_t v, int64_t* sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // sums may still be read from an earlier call
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const int64_t u = sums[w];
        if (w < warp) before += u;
        all += u;
    }
    *total = all;
    return v + before;
}

// The line's length T, the number of ranges P, this CTA's range (beginning at a
// tile: a range that holds none is empty) and the tile where it begins.  Every
// thread of the block calls it; `sh` is shared scratch.
struct KvLocateShared {
    int64_t sums[32];
    KvPlace place;
    int skip;          // empty places before the first tile
    int64_t named[2];  // rows of q [first, last) that the sequences name
};
template <int NT>
__device__ __forceinline__ void kv_locate(const KvBatch& bt, const KvGeom& g, int64_t p, int64_t P,
                                          int64_t min_tiles, unsigned* status, KvLocateShared* sh,
                                          int64_t* T, int64_t* Pused, int64_t* beg, int64_t* end,
                                          KvPlace* place) {
    int64_t all = 0, mine = 0, incl = 0;
    if (bt.seqs == 0) {
        if (threadIdx.x < 2) sh->named[threadIdx.x] = 0;
        __syncthreads();
    }
    // one pass when a block covers the sequences, else a pass for the total first
    const bool one = bt.seqs <= NT;
    for (int b0 = 0; b0 < bt.seqs; b0 += NT) {
        const int b = b0 + threadIdx.x;
        mine = 0;
        if (b < bt.seqs) {
            const KvSeq s = kv_seq(bt, b, status);
            mine = kv_seq_work(g, s);
            if (b == 0) sh->named[0] = s.first;
            if (b == bt.seqs - 1) sh->named[1] = s.first + s.n;
        }
        int64_t t;
        incl = kv_block_scan<NT>(mine, sh->sums, &t);
        all += t;
    }
    // no more CTAs than give each min_tiles tiles
    const int64_t Pu = max(min(P, all / min_tiles), int64_t(1));
    *T = all;
    *Pused = Pu;
    if (p >= Pu || all == 0) {
        *beg = *end = 0;
        return;
    }
    const int64_t lo = all * p / Pu;
    *beg = lo;
    *end = all * (p + 1) / Pu;
    int64_t base = 0;
    for (int b0 = 0; b0 < bt.seqs; b0 += NT) {
        const int b = b0 + threadIdx.x;
        int64_t t = all;
        if (!one) {
            mine = b < bt.seqs ? kv_seq_work(g, kv_seq(bt, b, status)) : 0;
            incl = kv_block_scan<NT>(mine, sh->sums, &t);
        }
        int64_t x = lo - (base + incl - mine);
        if (mine > 0 && x >= 0 && x < mine) {
            const KvSeq s = kv_seq(bt, b, status);
            KvPlace w{b, 0, 0, 0};
            for (;; ++w.rt) {
                int tl;
                const int64_t n = kv_tiles(g, s, w.rt, &tl) + g.lead;
                if (x < n * g.heads) {
                    w.h = static_cast<int>(x / n);
                    w.tile = static_cast<int>(x - w.h * n) - g.lead;
                    break;
                }
                x -= n * g.heads;
            }
            sh->skip = max(-w.tile, 0);
            w.tile = max(w.tile, 0);
            sh->place = w;
        }
        base += t;
    }
    __syncthreads();
    *place = sh->place;
    *beg += sh->skip;
    if (*beg >= *end) *beg = *end = 0;
}

// The next unit's tile 0, g.lead places behind the last one's end; the caller
// checks that its range goes so far.
__device__ __forceinline__ void kv_next_unit(const KvBatch& bt, const KvGeom& g, KvPlace* w,
                                             KvSeq* s, unsigned* status) {
    w->tile = 0;
    if (++w->h < g.heads) return;
    w->h = 0;
    if (++w->rt < kv_row_tiles(g, *s)) return;
    w->rt = 0;
    do {
        ++w->b;
        if (w->b >= bt.seqs) return;
        *s = kv_seq(bt, w->b, status);
    } while (kv_row_tiles(g, *s) == 0);
}

// CTA that owns place i when T places are cut into P ranges [T p / P, T (p + 1) / P).
__device__ __forceinline__ int64_t kv_owner(int64_t i, int64_t T, int64_t P) {
    return ((i + 1) * P - 1) / T;
}

__device__ __forceinline__ unsigned kv_arrive(unsigned* p) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(1u) : "memory");
    return old;
}

}  // namespace q4dev

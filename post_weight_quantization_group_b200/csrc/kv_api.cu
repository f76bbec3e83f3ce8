// kv_api.cu -- the paged INT8 KV cache's part of the C ABI of include/q4.h:
// argument validation, choice of kernel and launches (kv_paged.cuh,
// kv_attention.cuh, kv_mass.cuh, kv_evict.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "q4.h"
#include "q4_device.cuh"
#include "q4_host.cuh"
#include "kv_paged.cuh"
#include "kv_attention.cuh"
#include "kv_attention_tc.cuh"
#include "kv_mass.cuh"
#include "kv_mass_tc.cuh"
#include "kv_evict.cuh"

namespace {

using namespace q4dev;

constexpr int64_t kMaxRows = int64_t(1) << 30;  // 32-bit arithmetic on rows,
constexpr int64_t kMaxLen = int64_t(1) << 30;   // and on tokens less a window less new tokens

q4_status check_pool(const kv_paged_int8* c) {
    if (!c) return Q4_ERR_INVALID_ARG;
    if (!valid_dtype(c->dtype)) return Q4_ERR_INVALID_ARG;
    if (c->dtype == Q4_F32) return Q4_ERR_UNSUPPORTED;
    if (c->head_dim < 16 || c->head_dim > 256 || (c->head_dim % 16) != 0) return Q4_ERR_SHAPE;
    if (c->heads < 1 || c->heads > 4096 || c->page_size < 1 || c->page_size > (1 << 20) ||
        c->pages < 1 || c->pages > INT32_MAX)
        return Q4_ERR_SHAPE;
    const int64_t rows = static_cast<int64_t>(c->heads) * c->page_size;
    if (c->k_codes_stride < rows * c->head_dim || c->v_codes_stride < rows * c->head_dim ||
        c->k_scales_stride < rows || c->v_scales_stride < rows)
        return Q4_ERR_SHAPE;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return Q4_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 2) ||
        !aligned(c->v_scales, 2) || (c->k_codes_stride % 16) || (c->v_codes_stride % 16))
        return Q4_ERR_ALIGNMENT;
    return Q4_OK;
}

KvPool pool_of(const kv_paged_int8* c) {
    KvPool p{};
    p.kc = c->k_codes;
    p.vc = c->v_codes;
    p.ks = static_cast<uint16_t*>(c->k_scales);
    p.vs = static_cast<uint16_t*>(c->v_scales);
    p.kc_page = c->k_codes_stride;
    p.vc_page = c->v_codes_stride;
    p.ks_page = c->k_scales_stride;
    p.vs_page = c->v_scales_stride;
    p.pages = c->pages;
    p.heads = c->heads;
    p.ps = c->page_size;
    p.d = c->head_dim;
    return p;
}

// A matrix of `rows` rows of `cols` 16-bit elements, `stride` apart, read 16 bytes at a time.
q4_status check_rows(const void* p, int64_t stride, int64_t cols) {
    if (!p) return Q4_ERR_INVALID_ARG;
    if (stride < cols) return Q4_ERR_SHAPE;
    if (!aligned(p, 16) || (stride % 8)) return Q4_ERR_ALIGNMENT;
    return Q4_OK;
}

q4_status check_batch(const kv_batch* b, int page_size, bool queries) {
    if (!b) return Q4_ERR_INVALID_ARG;
    if (b->seqs < 0 || b->table_width < 0) return Q4_ERR_SHAPE;
    if (queries && (b->tokens < 0 || b->max_new < 1)) return Q4_ERR_SHAPE;
    if (b->table_width > kMaxLen / page_size) return Q4_ERR_SHAPE;
    if (b->seqs == 0) return Q4_OK;
    if (!b->seq_lens || (b->table_width > 0 && !b->block_table)) return Q4_ERR_INVALID_ARG;
    if (!aligned(b->seq_lens, 4) || !aligned(b->block_table, 4) || !aligned(b->cu_new, 4))
        return Q4_ERR_ALIGNMENT;
    return Q4_OK;
}

KvBatch batch_of(const kv_batch* b, int page_size) {
    KvBatch k{};
    k.table = b->block_table;
    k.lens = b->seq_lens;
    k.cu = b->cu_new;
    k.width = b->table_width;
    k.tokens = b->tokens;
    k.seqs = b->seqs;
    k.cap = static_cast<int>(b->table_width * page_size);
    return k;
}

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Team of 8-element lanes for a head of d elements.
int team_size(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

// ------------------------------------------------------------- attention

// Which kernel: the tensor-core one from more than kTcMinRows rows of a
// sequence and KV head on (head_dim up to 128), the other for decode steps.
constexpr int64_t kTcMinRows = 16;
// What a unit's beginning and end cost the decode kernel, in tiles (4.5 us against
// 1.6 us a tile): a ragged batch of 32 takes 66 us with it and 87 without.
constexpr int kKvLead = 3;

struct AttnPlan {
    bool tc;
    int nr;               // the other kernel's blocks of 8 rows of a unit
    int rows;             // rows of a unit
    int lead;             // what beginning and ending a unit costs, in tiles
    int64_t ctas;         // at most so many
    size_t bytes;         // of workspace
};

// CTAs of the few-rows kernel that the device holds at once.
int64_t rows_ctas(int dp, int nr, int sms) { return (dp * nr > 128 ? 1LL : 2LL) * sms; }

AttnPlan attn_plan(int d, int64_t group, int64_t max_new, int sms) {
    AttnPlan p{};
    const int dp = padded_dim(d);
    p.tc = dp <= 128 && max_new * group > kTcMinRows;
    p.nr = max_new * group <= 8 ? 1 : 2;
    p.rows = p.tc ? kTcaRows : 8 * p.nr;
    p.lead = p.tc ? 1 : kKvLead;
    // the other kernel's parts never need more than the tensor-core one's, which a mixed
    // batch takes after it
    p.ctas = p.tc ? sms : rows_ctas(dp, p.nr, sms);
    const size_t slot = static_cast<size_t>(p.rows) * (dp + 2);  // floats of a partial slot
    p.bytes = kWsCounterBytes + 2 * static_cast<size_t>(p.ctas) * slot * 4;
    return p;
}

// At most `ctas` CTAs, and no more than there can be places in the division of work.
int64_t attn_grid(const KvAttn& a, int64_t ctas) {
    const int64_t tiles = std::max<int64_t>((a.batch.cap + kKvTile - 1) / kKvTile, 1);
    const int64_t units = (a.batch.seqs + a.batch.tokens * a.geom.group / a.geom.R) * a.geom.heads;
    return units < ctas ? std::min(ctas, units * (tiles + a.geom.lead)) : ctas;
}

template <bool BF16, int DP, int NR, bool MASS>
q4_status run_attention(const KvAttn& a, int64_t grid, cudaStream_t st) {
    constexpr size_t smem = kv_attention_smem<DP, NR, MASS>();
    auto kernel = (a.pool.ps % 16) == 0 ? kv_attention_kernel<BF16, DP, NR, true, MASS>
                                        : kv_attention_kernel<BF16, DP, NR, false, MASS>;
    if (!set_kernel_attrs(kernel, static_cast<int>(smem), false)) return Q4_ERR_CUDA;
    return launch_ex(kernel, dim3(static_cast<unsigned>(grid)), dim3(kKvWarps * 32), smem, 1, true,
                     st, a);
}

template <bool BF16, int DP>
q4_status run_attention_tc(const KvAttn& a, int64_t grid, cudaStream_t st) {
    constexpr size_t smem = TcaGeom<DP>::total;
    auto kernel = kv_attention_tc_kernel<BF16, DP>;
    if (!set_kernel_attrs(kernel, static_cast<int>(smem), false)) return Q4_ERR_CUDA;
    return launch_ex(kernel, dim3(static_cast<unsigned>(grid)), dim3(kTcaThreads), smem, 1, true, st, a);
}

template <bool BF16, bool MASS>
q4_status dispatch_rows(const KvAttn& a, int nr, int64_t grid, cudaStream_t st) {
    switch (padded_dim(a.pool.d)) {
        case 64: return nr == 1 ? run_attention<BF16, 64, 1, MASS>(a, grid, st)
                                : run_attention<BF16, 64, 2, MASS>(a, grid, st);
        case 128: return nr == 1 ? run_attention<BF16, 128, 1, MASS>(a, grid, st)
                                 : run_attention<BF16, 128, 2, MASS>(a, grid, st);
        default: return nr == 1 ? run_attention<BF16, 256, 1, MASS>(a, grid, st)
                                : run_attention<BF16, 256, 2, MASS>(a, grid, st);
    }
}

template <bool BF16>
q4_status dispatch_attention(const KvAttn& a, const AttnPlan& p, int64_t grid, cudaStream_t st) {
    if (!p.tc) return dispatch_rows<BF16, false>(a, p.nr, grid, st);
    return padded_dim(a.pool.d) == 64 ? run_attention_tc<BF16, 64>(a, grid, st)
                                      : run_attention_tc<BF16, 128>(a, grid, st);
}

template <bool BF16, int DP>
q4_status run_mass_tc(const KvMassTc& a, int64_t grid, cudaStream_t st) {
    constexpr size_t smem = TcmGeom<DP>::total;
    auto kernel = kv_mass_tc_kernel<BF16, DP>;
    if (!set_kernel_attrs(kernel, static_cast<int>(smem), false)) return Q4_ERR_CUDA;
    return launch_ex(kernel, dim3(static_cast<unsigned>(grid)), dim3(kTcaThreads), smem, 1, true, st, a);
}

// Chunks with head_dim above 128.
template <bool BF16>
q4_status run_mass(const KvMass& a, int64_t grid, cudaStream_t st) {
    return launch_ex(kv_mass_kernel<BF16>, dim3(static_cast<unsigned>(grid)), dim3(kKvWarps * 32), 0,
                     1, true, st, a);
}

template <bool BF16, bool PAIRS>
q4_status run_append(const KvAppend& a, dim3 grid, cudaStream_t st) {
    switch (team_size(a.pool.d)) {
        case 8: return launch_ex(kv_append_kernel<BF16, 8, PAIRS>, grid, dim3(256), 0, 1, true, st, a);
        case 16: return launch_ex(kv_append_kernel<BF16, 16, PAIRS>, grid, dim3(256), 0, 1, true, st, a);
        default: return launch_ex(kv_append_kernel<BF16, 32, PAIRS>, grid, dim3(256), 0, 1, true, st, a);
    }
}

template <bool BF16>
q4_status run_gather(const KvPool& c, const int64_t* slots, int64_t tokens, uint16_t* k, uint16_t* v,
                     unsigned* status, dim3 grid, cudaStream_t st) {
    switch (team_size(c.d)) {
        case 8: return launch_ex(kv_gather_kernel<BF16, 8>, grid, dim3(256), 0, 1, true, st, c,
                                 slots, tokens, k, v, status);
        case 16: return launch_ex(kv_gather_kernel<BF16, 16>, grid, dim3(256), 0, 1, true, st, c,
                                  slots, tokens, k, v, status);
        default: return launch_ex(kv_gather_kernel<BF16, 32>, grid, dim3(256), 0, 1, true, st, c,
                                  slots, tokens, k, v, status);
    }
}

// What attention and mass check alike.
q4_status check_attention(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                          int32_t q_heads, const kv_batch* batch, float scale, int64_t window) {
    q4_status s = check_pool(cache);
    if (s != Q4_OK) return s;
    s = check_batch(batch, cache->page_size, true);
    if (s != Q4_OK) return s;
    if (q_heads < 1 || (q_heads % cache->heads) != 0) return Q4_ERR_SHAPE;
    if (!std::isfinite(scale) || window < 0) return Q4_ERR_INVALID_ARG;
    if (batch->tokens > kMaxRows / q_heads) return Q4_ERR_SHAPE;
    if (batch->tokens == 0 || batch->seqs == 0) return Q4_OK;
    return check_rows(q, q_stride, static_cast<int64_t>(q_heads) * cache->head_dim);
}

}  // namespace

extern "C" {

q4_status kv_append_int8_paged(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                               int32_t q_heads, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, int64_t tokens, const int64_t* slots,
                               const int32_t* positions, const float* inv_freq, int32_t rot_dim,
                               int32_t interleaved, const void* q_norm, const void* k_norm,
                               float eps, void* q_out, int64_t q_out_stride, q4_stream stream) {
    return kv_append_mass_int8_paged(cache, q, q_stride, q_heads, k, k_stride, v, v_stride, tokens, slots,
                                     positions, inv_freq, rot_dim, interleaved, q_norm, k_norm, eps, q_out,
                                     q_out_stride, nullptr, 0, stream);
}

q4_status kv_append_mass_int8_paged(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                                    int32_t q_heads, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, int64_t tokens, const int64_t* slots,
                                    const int32_t* positions, const float* inv_freq, int32_t rot_dim,
                                    int32_t interleaved, const void* q_norm, const void* k_norm,
                                    float eps, void* q_out, int64_t q_out_stride, float* mass,
                                    int64_t mass_stride, q4_stream stream) {
    q4_status s = check_pool(cache);
    if (s != Q4_OK) return s;
    if (tokens < 0 || q_heads < 0 || q_heads > (1 << 20)) return Q4_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > cache->head_dim || (rot_dim % (interleaved ? 2 : 16)) != 0)
        return Q4_ERR_SHAPE;
    if (interleaved != 0 && interleaved != 1) return Q4_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return Q4_ERR_INVALID_ARG;
    if (mass && mass_stride < static_cast<int64_t>(cache->heads) * cache->page_size) return Q4_ERR_SHAPE;
    if (tokens == 0) return Q4_OK;
    const int64_t d = cache->head_dim;
    if (!slots || (rot_dim > 0 && (!positions || !inv_freq))) return Q4_ERR_INVALID_ARG;
    if ((s = check_rows(k, k_stride, cache->heads * d)) != Q4_OK) return s;
    if ((s = check_rows(v, v_stride, cache->heads * d)) != Q4_OK) return s;
    if (q_heads > 0) {
        if ((s = check_rows(q, q_stride, q_heads * d)) != Q4_OK) return s;
        if ((s = check_rows(q_out, q_out_stride, q_heads * d)) != Q4_OK) return s;
    }
    if (!aligned(slots, 8) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(q_norm, 16) || !aligned(k_norm, 16) || !aligned(mass, 4))
        return Q4_ERR_ALIGNMENT;
    KvAppend a{};
    a.pool = pool_of(cache);
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.q_norm = static_cast<const uint16_t*>(q_norm);
    a.k_norm = static_cast<const uint16_t*>(k_norm);
    a.slots = slots;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.mass = mass;
    a.mass_page = mass_stride;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.rot = rot_dim;
    a.eps = eps;
    a.status = q4_status_word();
    if (!a.status) return Q4_ERR_CUDA;
    const int sms = sm_count(current_device());
    const int heads = q_heads + 2 * cache->heads;
    const int teams = 256 / team_size(cache->head_dim);
    // few tokens: one round of heads per CTA, so that a token's heads go side by side
    const bool few = tokens * heads <= 8LL * sms * teams;
    a.heads_per_cta = few ? teams : heads;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(tokens, 8LL * sms)),
                    static_cast<unsigned>((heads + a.heads_per_cta - 1) / a.heads_per_cta));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->dtype == Q4_BF16)
        return interleaved ? run_append<true, true>(a, grid, st) : run_append<true, false>(a, grid, st);
    return interleaved ? run_append<false, true>(a, grid, st) : run_append<false, false>(a, grid, st);
}

q4_status kv_gather_int8_paged(const kv_paged_int8* cache, const int64_t* slots, int64_t tokens,
                               void* k_out, void* v_out, q4_stream stream) {
    q4_status s = check_pool(cache);
    if (s != Q4_OK) return s;
    if (tokens < 0 || tokens > kMaxRows / (2 * cache->heads)) return Q4_ERR_SHAPE;
    if (tokens == 0) return Q4_OK;
    if (!slots || !k_out || !v_out) return Q4_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return Q4_ERR_ALIGNMENT;
    unsigned* status = q4_status_word();
    if (!status) return Q4_ERR_CUDA;
    const int sms = sm_count(current_device());
    const int teams = 256 / team_size(cache->head_dim);
    const int64_t want = (tokens * 2 * cache->heads + teams - 1) / teams;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(want, 16LL * sms)));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint16_t* ko = static_cast<uint16_t*>(k_out);
    uint16_t* vo = static_cast<uint16_t*>(v_out);
    return cache->dtype == Q4_BF16
               ? run_gather<true>(pool_of(cache), slots, tokens, ko, vo, status, grid, st)
               : run_gather<false>(pool_of(cache), slots, tokens, ko, vo, status, grid, st);
}

size_t kv_attention_workspace_bytes(int32_t head_dim, int32_t q_heads, int32_t kv_heads,
                                    int64_t max_new) {
    if (head_dim < 16 || head_dim > 256 || (head_dim % 16) != 0 || kv_heads < 1 || q_heads < 1 ||
        (q_heads % kv_heads) != 0 || max_new < 1 || max_new > kMaxRows / q_heads)
        return 0;
    return attn_plan(head_dim, q_heads / kv_heads, max_new, sm_count(current_device())).bytes;
}

q4_status kv_attention_int8_paged(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                                  int32_t q_heads, const kv_batch* batch, float scale,
                                  int64_t window, void* out, int64_t out_stride, float* lse,
                                  void* workspace, size_t workspace_bytes, q4_stream stream) {
    return kv_attention_fill_int8_paged(cache, q, q_stride, q_heads, batch, scale, window, out, out_stride, lse,
                                        workspace, workspace_bytes, 0, stream);
}

q4_status kv_attention_fill_int8_paged(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                                       int32_t q_heads, const kv_batch* batch, float scale,
                                       int64_t window, void* out, int64_t out_stride, float* lse,
                                       void* workspace, size_t workspace_bytes, int32_t fill,
                                       q4_stream stream) {
    q4_status s = check_attention(cache, q, q_stride, q_heads, batch, scale, window);
    if (s != Q4_OK) return s;
    if (fill < 0 || fill > 3) return Q4_ERR_INVALID_ARG;
    if (batch->tokens == 0 || (batch->seqs == 0 && !fill)) return Q4_OK;
    const int64_t d = cache->head_dim;
    if ((s = check_rows(out, out_stride, q_heads * d)) != Q4_OK) return s;
    if (!aligned(lse, 4)) return Q4_ERR_ALIGNMENT;
    const int group = q_heads / cache->heads;
    const int64_t max_new = std::min(batch->max_new, batch->tokens);
    const int sms = sm_count(current_device());
    const AttnPlan p = attn_plan(cache->head_dim, group, max_new, sms);
    if (!workspace || workspace_bytes < p.bytes) return Q4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return Q4_ERR_ALIGNMENT;
    KvAttn a{};
    a.pool = pool_of(cache);
    a.batch = batch_of(batch, cache->page_size);
    a.geom = {p.rows, kKvTile, group, cache->heads,
              static_cast<int>(std::min<int64_t>(window, kMaxLen)), p.lead, 0, INT32_MAX};
    if (window >= a.batch.cap) a.geom.window = 0;  // hides nothing
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.q_heads = q_heads;
    a.scale_log2 = scale * 1.44269504f;
    a.fill = fill;
    a.count = static_cast<unsigned*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsCounterBytes);
    a.status = q4_status_word();
    if (!a.status) return Q4_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = cache->dtype == Q4_BF16;
    if (batch->seqs == 0) {  // nothing but rows to fill
        const int64_t ctas = std::min<int64_t>(batch->tokens, sms);
        return bf ? dispatch_rows<true, false>(a, 1, ctas, st) : dispatch_rows<false, false>(a, 1, ctas, st);
    }
    if (p.tc && batch->tokens < max_new * batch->seqs) {
        // Chunks beside decode steps: those go to the other kernel, since a tile costs the
        // tensor-core kernel the same however few of its 256 rows are any (4 chunks of 257 and
        // 12 single tokens over up to 8100: 183 us in one kernel).
        AttnPlan few = p;
        few.tc = false;
        few.nr = group <= 8 ? 1 : 2;
        few.ctas = rows_ctas(padded_dim(cache->head_dim), few.nr, sms);
        KvAttn b = a;
        b.geom.R = 8 * few.nr;
        b.geom.lead = kKvLead;
        b.geom.rows_hi = 8 * few.nr;
        a.geom.rows_lo = 8 * few.nr;
        a.fill = 0;
        s = bf ? dispatch_attention<true>(b, few, attn_grid(b, few.ctas), st)
               : dispatch_attention<false>(b, few, attn_grid(b, few.ctas), st);
        if (s != Q4_OK) return s;
    }
    const int64_t grid = attn_grid(a, p.ctas);
    return bf ? dispatch_attention<true>(a, p, grid, st) : dispatch_attention<false>(a, p, grid, st);
}

q4_status kv_attention_mass_int8_paged(const kv_paged_int8* cache, const void* q, int64_t q_stride,
                                       int32_t q_heads, const float* lse, const kv_batch* batch,
                                       float scale, int64_t window, float* mass,
                                       int64_t mass_stride, q4_stream stream) {
    q4_status s = check_attention(cache, q, q_stride, q_heads, batch, scale, window);
    if (s != Q4_OK) return s;
    if (mass_stride < static_cast<int64_t>(cache->heads) * cache->page_size) return Q4_ERR_SHAPE;
    if (batch->tokens == 0 || batch->seqs == 0) return Q4_OK;
    if (!lse || !mass) return Q4_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(mass, 4)) return Q4_ERR_ALIGNMENT;
    const int group = q_heads / cache->heads;
    const int sms = sm_count(current_device());
    const int64_t max_new = std::min(batch->max_new, batch->tokens);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (max_new * group <= kTcMinRows) {  // decode steps: the rows stay and the keys go by
        KvAttn k{};
        k.pool = pool_of(cache);
        k.batch = batch_of(batch, cache->page_size);
        const int nr = max_new * group <= 8 ? 1 : 2;
        k.geom = {8 * nr, kKvTile, group, cache->heads,
                  static_cast<int>(std::min<int64_t>(window, kMaxLen)), kKvLead, 0, INT32_MAX};
        if (window >= k.batch.cap) k.geom.window = 0;  // hides nothing
        k.q = static_cast<const uint16_t*>(q);
        k.lse = const_cast<float*>(lse);  // read
        k.mass = mass;
        k.mass_page = mass_stride;
        k.q_stride = q_stride;
        k.q_heads = q_heads;
        k.scale_log2 = scale * 1.44269504f;
        k.status = q4_status_word();
        if (!k.status) return Q4_ERR_CUDA;
        const int64_t grid = attn_grid(k, 2LL * sms);
        return cache->dtype == Q4_BF16 ? dispatch_rows<true, true>(k, nr, grid, st)
                                       : dispatch_rows<false, true>(k, nr, grid, st);
    }
    if (cache->head_dim <= 128) {
        KvMassTc k{};
        k.pool = pool_of(cache);
        k.batch = batch_of(batch, cache->page_size);
        k.group = group;
        k.window = window >= k.batch.cap ? 0 : static_cast<int>(window);
        k.q_heads = q_heads;
        k.q = static_cast<const uint16_t*>(q);
        k.lse = lse;
        k.mass = mass;
        k.q_stride = q_stride;
        k.mass_page = mass_stride;
        k.scale_log2 = scale * 1.44269504f;
        k.status = q4_status_word();
        if (!k.status) return Q4_ERR_CUDA;
        const int64_t keys = std::max<int64_t>((k.batch.cap + 127) / 128, 1);
        const int64_t units = static_cast<int64_t>(batch->seqs) * cache->heads;
        const int64_t grid = units < sms ? std::min<int64_t>(sms, units * keys) : sms;
        if (cache->dtype == Q4_BF16)
            return cache->head_dim <= 64 ? run_mass_tc<true, 64>(k, grid, st) : run_mass_tc<true, 128>(k, grid, st);
        return cache->head_dim <= 64 ? run_mass_tc<false, 64>(k, grid, st) : run_mass_tc<false, 128>(k, grid, st);
    }
    KvMass a{};
    a.pool = pool_of(cache);
    a.batch = batch_of(batch, cache->page_size);
    a.geom = {kKvTile, kKvTile, q_heads / cache->heads, cache->heads,
              static_cast<int>(std::min<int64_t>(window, kMaxLen)), 0, 0, INT32_MAX};
    if (window >= a.batch.cap) a.geom.window = 0;  // hides nothing
    a.q = static_cast<const uint16_t*>(q);
    a.lse = lse;
    a.mass = mass;
    a.q_stride = q_stride;
    a.mass_page = mass_stride;
    a.q_heads = q_heads;
    a.scale_log2 = scale * 1.44269504f;
    a.status = q4_status_word();
    if (!a.status) return Q4_ERR_CUDA;
    const int64_t tiles = std::max<int64_t>((a.batch.cap + kKvTile - 1) / kKvTile, 1);
    int64_t grid = sms;
    if (static_cast<int64_t>(batch->seqs) * cache->heads < grid)
        grid = std::min(grid, batch->seqs * cache->heads * tiles);
    return cache->dtype == Q4_BF16 ? run_mass<true>(a, grid, st) : run_mass<false>(a, grid, st);
}

size_t kv_evict_workspace_bytes(int32_t seqs, int32_t heads, int64_t budget) {
    if (seqs < 1 || heads < 1 || heads > 4096 || budget < 1 || budget > kMaxLen) return 0;
    return (static_cast<size_t>(seqs) * heads * budget + seqs) * 4;
}

q4_status kv_evict_int8_paged(const kv_paged_int8* cache, float* mass, int64_t mass_stride,
                              const kv_batch* batch, int64_t budget, int64_t recent, int64_t sinks,
                              const int32_t* dst_table, int64_t dst_width, int32_t* new_lens,
                              void* workspace, size_t workspace_bytes, q4_stream stream) {
    q4_status s = check_pool(cache);
    if (s != Q4_OK) return s;
    if ((s = check_batch(batch, cache->page_size, false)) != Q4_OK) return s;
    if (mass_stride < static_cast<int64_t>(cache->heads) * cache->page_size) return Q4_ERR_SHAPE;
    if (budget < 1 || budget > kMaxLen || recent < 0 || sinks < 0 || recent > budget ||
        sinks > budget - recent)
        return Q4_ERR_INVALID_ARG;
    const bool in_place = !dst_table || dst_table == batch->block_table;
    const int64_t cap = batch->table_width * cache->page_size;
    if (!in_place && (dst_width < 0 || dst_width > kMaxLen / cache->page_size ||
                      dst_width * cache->page_size < std::min(budget, cap)))
        return Q4_ERR_SHAPE;
    if (static_cast<int64_t>(batch->seqs) * cache->heads > INT32_MAX) return Q4_ERR_SHAPE;
    if (batch->seqs == 0) return Q4_OK;
    if (!mass || !new_lens) return Q4_ERR_INVALID_ARG;
    if (!aligned(mass, 4) || !aligned(new_lens, 4) || !aligned(dst_table, 4)) return Q4_ERR_ALIGNMENT;
    // no sequence can be longer than cap: where that is within the budget nothing is selected
    const size_t need = budget >= cap ? static_cast<size_t>(batch->seqs) * 4
                                      : kv_evict_workspace_bytes(batch->seqs, cache->heads, budget);
    if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return Q4_ERR_ALIGNMENT;
    KvEvict a{};
    a.pool = pool_of(cache);
    a.batch = batch_of(batch, cache->page_size);
    a.dst_table = in_place ? batch->block_table : dst_table;
    a.dst_width = in_place ? batch->table_width : dst_width;
    a.mass = mass;
    a.mass_page = mass_stride;
    a.budget = static_cast<int>(budget);
    a.recent = static_cast<int>(recent);
    a.sinks = static_cast<int>(sinks);
    a.new_lens = new_lens;
    a.len = static_cast<int32_t*>(workspace);
    a.src = a.len + batch->seqs;
    a.status = q4_status_word();
    if (!a.status) return Q4_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int units = batch->seqs * cache->heads;
    const int sms = sm_count(current_device());
    // CTAs of a unit (each takes an SM): up to 8 that are all resident at once, with 2048
    // tokens or more each
    int parts = 1;
    while (parts < 8 && units * parts * 2 <= sms && cap / (2 * parts) >= 2048) parts *= 2;
    const int vec = (cache->page_size % 4) == 0 && aligned(mass, 16) && (mass_stride % 4) == 0;
    if (static_cast<int64_t>(units) * parts > INT32_MAX) return Q4_ERR_SHAPE;
    s = launch_ex(kv_evict_select_kernel, dim3(static_cast<unsigned>(units * parts)), dim3(kEvThreads), 0,
                  parts, true, st, a, parts, vec);
    if (s != Q4_OK) return s;
    const unsigned gy = static_cast<unsigned>(std::min(units, 65535));
    if (in_place) {
        const int cols = (cache->head_dim + 31) / 32;
        return launch_ex(kv_evict_inplace_kernel, dim3(2 * cols + 1, gy), dim3(256), 0, 1, true, st, a);
    }
    const int ts = cache->head_dim <= 64 ? 4 : cache->head_dim <= 128 ? 8 : 16;
    const int64_t rows = 256 / ts;
    const int64_t want = (std::min(budget, std::max<int64_t>(cap, 1)) + rows - 1) / rows;
    const int64_t room = std::max<int64_t>(1, 16LL * sms / gy);
    const dim3 grid(static_cast<unsigned>(std::min(want, room)), gy);
    switch (ts) {
        case 4: return launch_ex(kv_evict_copy_kernel<4>, grid, dim3(256), 0, 1, true, st, a);
        case 8: return launch_ex(kv_evict_copy_kernel<8>, grid, dim3(256), 0, 1, true, st, a);
        default: return launch_ex(kv_evict_copy_kernel<16>, grid, dim3(256), 0, 1, true, st, a);
    }
}

}  // extern "C"

// kpa_paged_api.cu -- the extern "C" entry points of the paged factor cache: argument
// checks, split planning, workspace layout and launches.
#include <math.h>

#include <algorithm>

#include "kpa_paged.cuh"

namespace kpa {
namespace {

kpa_status fail(cudaError_t e) {
    record_cuda_error(e);
    return KPA_ERR_CUDA;
}

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Config and pool description; *s gets everything but the device pointers.
kpa_status check_paged(const kpa_config *cfg, const kpa_pages *pg, PagedShape *s) {
    kpa_status st = config_check(cfg);
    if (st != KPA_OK) return st;
    if (!pg || pg->page_size <= 0 || pg->page_size % paged::kSlots16 != 0 || pg->page_size > 4096 || pg->n_pages <= 0 ||
        pg->table_stride <= 0 || (int64_t)pg->page_size * pg->table_stride > INT32_MAX)
        return KPA_ERR_INVALID_ARG;
    if (pg->format != KPA_PAGE_BF16 && pg->format != KPA_PAGE_E4M3) return KPA_ERR_INVALID_ARG;
    if (cfg->dtype != KPA_BF16 || cfg->order == 3 || cfg->shared_b) return KPA_ERR_UNSUPPORTED;
    const int64_t part = (int64_t)cfg->h1 * cfg->d1 + (int64_t)cfg->h2 * cfg->d2;
    if (part * std::max(cfg->r_k, cfg->r_v) > (1 << 24)) return KPA_ERR_UNSUPPORTED;
    s->d = config_dims(cfg);
    paged::Pool &p = s->pool;
    p.k = p.v = nullptr;
    p.table = nullptr;
    p.table_stride = pg->table_stride;
    p.n_pages = pg->n_pages;
    p.pg = pg->page_size / paged::kSlots16;
    p.magic = ((1ull << 36) + p.pg - 1) / p.pg;
    p.e4m3 = pg->format == KPA_PAGE_E4M3;
    p.kg = p.e4m3 ? (s->d.ek + 2) * 16 : s->d.ek * 32;
    p.vg = p.e4m3 ? (s->d.ev + 2) * 16 : s->d.ev * 32;
    return KPA_OK;
}

struct AttnPlan {
    int variant;                 // of the single-token kernel, or -1: a chunk kernel
    bool tcgen05;                // (chunk kernels) the tcgen05 one
    int groups_per_split;        // (single-token kernel)
    bool cluster;                // (single-token kernel) a sequence's splits merge in a cluster: no workspace
    int n_slots;                 // (single-token kernel) blocks that size the splits themselves, or 0
    int n_split;
    size_t ml_off, slots_off, bytes;
};

// How the rows' key range is split.
//  - The chunk kernels: with fewer CTAs than two per SM, into runs of at least four tiles
//    (shorter ones cost more in partials than they gain), as many as make the last wave of
//    CTAs end soonest when a CTA costs its tiles and three more.
//  - The single-token kernel: one CTA per slot of the SMs where that is one wave for the
//    longest sequences there may be.  Where a batch would take more than that, or where its
//    splits are long, the lengths decide, which the host does not see: the blocks of one wave
//    (of up to four, to keep three splits a sequence) find the split size themselves.
AttnPlan plan_attn(const PagedShape &ps, int batch, int n_rows, bool chunks, int max_len, int window, int sinks,
                   int sms) {
    const Dims &d = ps.d;
    const bool e4m3 = ps.pool.e4m3 != 0;
    AttnPlan p = {};
    p.variant = chunks ? -1 : paged_decode_variant(d);
    p.tcgen05 = chunks && paged_prefill_supported(ps);
    const int tr = p.tcgen05 ? paged_prefill_rows() : paged_mma_rows();
    auto visible = [&](int64_t T, int64_t rows) {          // units of T slots that a set of rows sees at most
        const int64_t all = ((int64_t)max_len + T - 1) / T;
        return window > 0 ? std::min(all, ((int64_t)sinks + T - 1) / T + ((int64_t)window + rows) / T + 2) : all;
    };
    if (p.variant >= 0) {
        int tg = 1, per_sm = 1;
        paged_decode_shape(p.variant, e4m3, &tg, &per_sm);
        const int64_t groups = std::max<int64_t>(1, visible(16, 1)), tiles = (groups + tg - 1) / tg;
        const int64_t per_seq = std::max<int64_t>(1, (int64_t)sms * per_sm / batch);
        int64_t per = (tiles + per_seq - 1) / per_seq;
        const int64_t wave = (int64_t)sms * per_sm;
        // Long batches: the lengths, which are not known here, may differ, so the blocks size the splits (32
        // sequences of 1024 .. 8192 tokens, R = 4: 82 us, splits sized from the longest 91).  Short ones do
        // not repay the search.  (It sums the sequences' tiles in 32 bits.)
        if (batch > 1 && batch <= kPagedMaxSlotSeqs && (per >= 16 || per_seq == 1) && tiles >= 8 &&
            batch * tiles <= INT32_MAX) {
            p.n_slots = (int)(wave * std::min<int64_t>(4, (3 * (int64_t)batch + wave - 1) / wave));
            p.n_slots = std::max(p.n_slots, batch);
            p.n_split = 2;                                 // (partials, in slots)
            const size_t rh = (size_t)p.n_slots * d.h;
            p.ml_off = (rh * d.dh * sizeof(float) + 255) & ~(size_t)255;
            p.slots_off = p.ml_off + ((rh * 2 * sizeof(float) + 255) & ~(size_t)255);
            p.bytes = p.slots_off + (((size_t)batch * sizeof(int2) + 255) & ~(size_t)255);
            return p;
        }
        // A sequence's splits merge in one cluster, without a second kernel, where every CTA is resident at
        // once (a cluster holds its SMs until its longest split ends) and the splits get no more than two
        // tiles or a quarter longer for it: the second kernel and its launch cost about as much (8 x 4096
        // tokens of 16 heads of 64, bf16: 10.7 us in a replayed graph and 6.2 of the host against 10.0 and 8.2;
        // 64 x 4096 of 32 heads of 64, e4m3: 25.1 and 6.0 against 26.7 and 8.0).
        const int64_t most = std::min<int64_t>(kPagedMaxCluster, (int64_t)sms * per_sm / batch);
        for (int64_t t = per; t <= std::max(per + 2, per + per / 4) && most > 1; ++t) {
            const int64_t n = (tiles + t - 1) / t;
            if (n > 1 && n <= most && paged_decode_max_clusters(p.variant, e4m3, (int)n) >= batch) {
                per = t;
                p.cluster = true;
                break;
            }
        }
        p.groups_per_split = (int)(per * tg);
        p.n_split = (int)((groups + p.groups_per_split - 1) / p.groups_per_split);
    } else {
        constexpr int kMinTiles = 4;
        const int kTile = p.tcgen05 ? 128 : 64;
        // (the rows of a sequence are not known here: half a tile of each is taken as empty)
        const int64_t row_tiles = chunks ? (n_rows + (int64_t)std::min(batch, n_rows) * (tr / 2) + tr - 1) / tr : batch;
        const int64_t ctas = std::max<int64_t>(1, row_tiles * d.h);
        const int64_t tiles = visible(kTile, chunks ? tr : 1);
        int64_t best = 0;
        p.n_split = 1;
        if (ctas < 2 * (int64_t)sms)
            for (int64_t k = 1; k <= std::min<int64_t>(4096, std::max<int64_t>(1, tiles / kMinTiles)) && ctas * k <= 4 * (int64_t)sms + ctas; ++k) {
                const int64_t cost = ((ctas * k + sms - 1) / sms) * ((tiles + k - 1) / k + 3);
                if (k == 1 || cost < best) {
                    best = cost;
                    p.n_split = (int)k;
                }
            }
    }
    const size_t rh = (size_t)n_rows * d.h * p.n_split;
    p.ml_off = (rh * d.dh * sizeof(float) + 255) & ~(size_t)255;
    p.bytes = p.n_split > 1 && !p.cluster ? p.ml_off + ((rh * 2 * sizeof(float) + 255) & ~(size_t)255) : 0;
    return p;
}

kpa_status check_attn(const kpa_config *cfg, const kpa_pages *pg, int32_t batch, int32_t n_rows, bool chunks,
                      int32_t max_len, int32_t window, int32_t sinks, PagedShape *s) {
    kpa_status st = check_paged(cfg, pg, s);
    if (st != KPA_OK && st != KPA_ERR_UNSUPPORTED) return st;
    if (batch < 0 || n_rows < 0 || max_len < 0 || window < 0 || sinks < 0) return KPA_ERR_INVALID_ARG;
    if ((int64_t)max_len > (int64_t)pg->page_size * pg->table_stride) return KPA_ERR_INVALID_ARG;
    if (st != KPA_OK) return st;
    if (!paged_mma_supported(s->d, s->pool.e4m3 != 0)) return KPA_ERR_UNSUPPORTED;
    // row tiles (of chunks) and sequences (single tokens) are blocks in y or z
    if (batch > 65535 || (chunks && n_rows / paged_mma_rows() + (int64_t)batch > 65535)) return KPA_ERR_UNSUPPORTED;
    return KPA_OK;
}

kpa_status workspace_size(const kpa_config *cfg, const kpa_pages *pg, int32_t batch, int32_t n_rows, bool chunks,
                          int32_t max_len, int32_t window, int32_t sinks, size_t *bytes) {
    PagedShape s;
    kpa_status st = check_attn(cfg, pg, batch, n_rows, chunks, max_len, window, sinks, &s);
    if (st != KPA_OK) return st;
    if (!bytes) return KPA_ERR_INVALID_ARG;
    *bytes = 0;
    if (batch == 0 || n_rows == 0) return KPA_OK;
    int sms = 0;
    st = device_info(nullptr, &sms);
    if (st != KPA_OK) return st;
    *bytes = plan_attn(s, batch, n_rows, chunks, max_len, window, sinks, sms).bytes;
    return KPA_OK;
}

// Both attentions: rows of chunks (cu, start) or one row per sequence (seq_len).
kpa_status attn(const kpa_config *cfg, const kpa_pages *pg, int32_t batch, int32_t n_rows, bool chunks, const void *q,
                const int32_t *cu, const int32_t *start, const int32_t *seq_len, const int32_t *table,
                const void *kpool, const void *vpool, int32_t max_len, int32_t window, int32_t sinks, float sm_scale,
                void *out, void *workspace, size_t ws_bytes, kpa_stream stream) {
    PagedShape s;
    kpa_status st = check_attn(cfg, pg, batch, n_rows, chunks, max_len, window, sinks, &s);
    if (st != KPA_OK && st != KPA_ERR_UNSUPPORTED) return st;
    if (!isfinite(sm_scale)) return KPA_ERR_INVALID_ARG;
    if (st != KPA_OK) return st;
    if (batch == 0 || n_rows == 0) return KPA_OK;
    if (!q || !table || !kpool || !vpool || !out || (chunks ? !cu || !start : !seq_len)) return KPA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kpool, 16) || !aligned(vpool, 16) || !aligned(out, 16) || !aligned(table, 4) ||
        !aligned(cu, 4) || !aligned(start, 4) || !aligned(seq_len, 4))
        return KPA_ERR_INVALID_ARG;
    int *err = nullptr, sms = 0;
    st = device_info(&err, &sms);
    if (st != KPA_OK) return st;
    const AttnPlan p = plan_attn(s, batch, n_rows, chunks, max_len, window, sinks, sms);
    if (p.bytes > 0) {
        if (!workspace || ws_bytes < p.bytes) return KPA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return KPA_ERR_INVALID_ARG;
    }
    s.pool.k = static_cast<const unsigned char *>(kpool);
    s.pool.v = static_cast<const unsigned char *>(vpool);
    s.pool.table = table;
    PagedAttnArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.cu = chunks ? cu : nullptr;
    a.start = start;
    a.seq_len = seq_len;
    a.batch = batch;
    a.n_rows = n_rows;
    a.max_len = max_len;
    a.mask.window = window;
    a.mask.sinks = sinks;
    a.qscale = (float)((double)sm_scale / (double)s.d.rk * 1.4426950408889634);
    a.out_scale = (float)(1.0 / (double)s.d.rv);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.n_split = p.n_split;
    if (p.bytes > 0) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.ml_off);
        if (p.n_slots > 0) a.slots = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + p.slots_off);
    }
    a.err = err;
    const cudaError_t e = p.variant >= 0 ? launch_paged_decode(p.variant, s, a, p.groups_per_split, p.n_slots, p.cluster,
                                                               device_wait_limit_ns(), (cudaStream_t)stream)
                          : p.tcgen05      ? launch_paged_prefill(s, a, device_wait_limit_ns(), (cudaStream_t)stream)
                                           : launch_paged_mma(s, a, (cudaStream_t)stream);
    return e == cudaSuccess ? KPA_OK : fail(e);
}

kpa_status records(const kpa_config *cfg, const kpa_pages *pg, int32_t batch, int32_t n_rows, const void *kf,
                   const void *vf, const int32_t *cu, const int32_t *start, const int32_t *table, const void *kpool,
                   const void *vpool, PagedShape *s, int **err, bool *empty) {
    kpa_status st = check_paged(cfg, pg, s);
    if (st != KPA_OK && st != KPA_ERR_UNSUPPORTED) return st;
    if (batch < 0 || n_rows < 0) return KPA_ERR_INVALID_ARG;
    if (st != KPA_OK) return st;
    *empty = batch == 0 || n_rows == 0;
    if (*empty) return KPA_OK;
    if (batch > INT32_MAX / 256 || n_rows > INT32_MAX / 2) return KPA_ERR_UNSUPPORTED;
    if (!kf || !vf || !cu || !start || !table || !kpool || !vpool) return KPA_ERR_INVALID_ARG;
    if (!aligned(kf, 16) || !aligned(vf, 16) || !aligned(kpool, 16) || !aligned(vpool, 16) || !aligned(cu, 4) ||
        !aligned(start, 4) || !aligned(table, 4))
        return KPA_ERR_INVALID_ARG;
    s->pool.k = static_cast<const unsigned char *>(kpool);
    s->pool.v = static_cast<const unsigned char *>(vpool);
    s->pool.table = table;
    return device_info(err, nullptr);
}

}  // namespace
}  // namespace kpa

using namespace kpa;

extern "C" {

kpa_status kpa_paged_page_bytes(const kpa_config *cfg, const kpa_pages *pages, size_t *k_bytes, size_t *v_bytes) {
    PagedShape s;
    const kpa_status st = check_paged(cfg, pages, &s);
    if (st != KPA_OK) return st;
    if (k_bytes) *k_bytes = (size_t)s.pool.pg * s.pool.kg;
    if (v_bytes) *v_bytes = (size_t)s.pool.pg * s.pool.vg;
    return KPA_OK;
}

kpa_status kpa_paged_append_factors(const kpa_config *cfg, const kpa_pages *pages, int32_t batch, int32_t n_rows,
                                    const void *k_factors, const void *v_factors, const int32_t *cu_rows,
                                    const int32_t *start_pos, const int32_t *page_table, void *kpool, void *vpool,
                                    kpa_stream stream) {
    PagedShape s;
    int *err = nullptr;
    bool empty = false;
    const kpa_status st = records(cfg, pages, batch, n_rows, k_factors, v_factors, cu_rows, start_pos, page_table,
                                  kpool, vpool, &s, &err, &empty);
    if (st != KPA_OK || empty) return st;
    const cudaError_t e = launch_paged_append(s, batch, n_rows, k_factors, v_factors, cu_rows, start_pos, kpool, vpool,
                                              config_rope(cfg), err, (cudaStream_t)stream);
    return e == cudaSuccess ? KPA_OK : fail(e);
}

kpa_status kpa_paged_read_factors(const kpa_config *cfg, const kpa_pages *pages, int32_t batch, int32_t n_rows,
                                  const int32_t *cu_rows, const int32_t *start_pos, const int32_t *page_table,
                                  const void *kpool, const void *vpool, void *k_factors, void *v_factors,
                                  kpa_stream stream) {
    PagedShape s;
    int *err = nullptr;
    bool empty = false;
    const kpa_status st = records(cfg, pages, batch, n_rows, k_factors, v_factors, cu_rows, start_pos, page_table,
                                  kpool, vpool, &s, &err, &empty);
    if (st != KPA_OK || empty) return st;
    const cudaError_t e = launch_paged_read(s, batch, n_rows, cu_rows, start_pos, k_factors, v_factors, err,
                                            (cudaStream_t)stream);
    return e == cudaSuccess ? KPA_OK : fail(e);
}

kpa_status kpa_paged_prefill_workspace_size(const kpa_config *cfg, const kpa_pages *pages, int32_t batch,
                                            int32_t n_rows, int32_t max_len, int32_t window, int32_t sinks,
                                            size_t *bytes) {
    return workspace_size(cfg, pages, batch, n_rows, true, max_len, window, sinks, bytes);
}

kpa_status kpa_paged_prefill(const kpa_config *cfg, const kpa_pages *pages, int32_t batch, int32_t n_rows,
                             const void *q, const int32_t *cu_rows, const int32_t *start_pos,
                             const int32_t *page_table, const void *kpool, const void *vpool, int32_t max_len,
                             int32_t window, int32_t sinks, float sm_scale, void *out, void *workspace,
                             size_t ws_bytes, kpa_stream stream) {
    return attn(cfg, pages, batch, n_rows, true, q, cu_rows, start_pos, nullptr, page_table, kpool, vpool, max_len,
                window, sinks, sm_scale, out, workspace, ws_bytes, stream);
}

static kpa_status kernel_kind(const kpa_config *cfg, const kpa_pages *pages, bool chunks, int32_t *kind) {
    PagedShape s;
    const kpa_status st = check_paged(cfg, pages, &s);
    if (st != KPA_OK) return st;
    if (!kind) return KPA_ERR_INVALID_ARG;
    if (!paged_mma_supported(s.d, s.pool.e4m3 != 0)) return KPA_ERR_UNSUPPORTED;
    *kind = KPA_PAGED_KERNEL_CHUNKS;
    if (!chunks && paged_decode_variant(s.d) >= 0) *kind = KPA_PAGED_KERNEL_FACTORS;
    if (chunks && paged_prefill_supported(s)) *kind = KPA_PAGED_KERNEL_TCGEN05;
    return KPA_OK;
}

kpa_status kpa_paged_decode_kernel_kind(const kpa_config *cfg, const kpa_pages *pages, int32_t *kind) {
    return kernel_kind(cfg, pages, false, kind);
}

kpa_status kpa_paged_prefill_kernel_kind(const kpa_config *cfg, const kpa_pages *pages, int32_t *kind) {
    return kernel_kind(cfg, pages, true, kind);
}

kpa_status kpa_paged_decode_workspace_size(const kpa_config *cfg, const kpa_pages *pages, int32_t batch,
                                           int32_t max_len, int32_t window, int32_t sinks, size_t *bytes) {
    return workspace_size(cfg, pages, batch, batch, false, max_len, window, sinks, bytes);
}

kpa_status kpa_paged_decode(const kpa_config *cfg, const kpa_pages *pages, int32_t batch, const void *q,
                            const int32_t *seq_len, const int32_t *page_table, const void *kpool, const void *vpool,
                            int32_t max_len, int32_t window, int32_t sinks, float sm_scale, void *out,
                            void *workspace, size_t ws_bytes, kpa_stream stream) {
    return attn(cfg, pages, batch, batch, false, q, nullptr, nullptr, seq_len, page_table, kpool, vpool, max_len,
                window, sinks, sm_scale, out, workspace, ws_bytes, stream);
}

}  // extern "C"

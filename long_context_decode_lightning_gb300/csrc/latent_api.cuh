// C-ABI entry points of the latent cache: host-side validation and launch
// shapes. Included by hsi.cu after paged_api.cuh.
#pragma once
#include <algorithm>
#include <cmath>

#include "latent.cuh"
#include "latent_attend.cuh"

namespace {

hsi_status latent_view(const hsi_latent_cache* c, LatentView* v) {
    if (!c || !c->data || !c->kv_len || c->B <= 0 || c->n_pages <= 0) return HSI_ERR_INVALID_ARG;
    if (c->format < HSI_LATENT_BF16 || c->format > HSI_LATENT_FP4) return HSI_ERR_INVALID_ARG;
    if (!(c->dim == 512 || (c->dim == 576 && c->format != HSI_LATENT_FP4)) || c->B > 65535) return HSI_ERR_UNSUPPORTED;
    const int64_t bytes = latent_entry_bytes(c->format, c->dim), far = int64_t(1) << 40;
    if (!aligned(c->data, 16) || c->token_stride < bytes || c->token_stride % 16 || c->token_stride >= far)
        return HSI_ERR_INVALID_ARG;
    v->data = static_cast<uint8_t*>(c->data);
    v->token_stride = c->token_stride;
    v->n_pages = c->n_pages;
    v->kv_len = c->kv_len;
    v->B = c->B;
    v->dim = c->dim;
    if (!c->table) {
        if (!c->offsets || !aligned(c->offsets, 8)) return HSI_ERR_INVALID_ARG;
        v->off = c->offsets;
        v->capacity = (int)(c->n_pages < INT32_MAX ? c->n_pages : INT32_MAX);
        return HSI_OK;
    }
    if (c->ld_table <= 0 || c->table_width < 0 || c->table_width > c->ld_table || c->page_size <= 0 ||
        c->n_pages >= INT32_MAX)
        return HSI_ERR_INVALID_ARG;
    if (c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return HSI_ERR_UNSUPPORTED;
    v->page_stride = c->n_pages == 1 ? c->token_stride : c->page_stride;  // never used where there is one page
    if (v->page_stride < bytes || v->page_stride % 16 || v->page_stride >= far) return HSI_ERR_INVALID_ARG;
    v->table = c->table;
    v->ld_table = c->ld_table;
    const int64_t width = c->table_width ? c->table_width : c->ld_table, most = INT32_MAX / c->page_size;
    v->capacity = width > most ? INT32_MAX : (int)(width * c->page_size);  // lengths are 32-bit
    while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
    return HSI_OK;
}

// The distance of n rows; of one row none, whatever the caller's.
int64_t row_stride(int64_t n, int64_t stride) { return n > 1 ? stride : 0; }

// (a k without lists is the list of a caller whose tensor holds nothing and so has no address)
bool lists_ok(const int32_t* idx, int64_t ld_idx, int32_t k) {
    return idx ? k > 0 && ld_idx >= k && aligned(idx, 4) : k == 0;
}

// How heads and tokens make units of at most 64 rows.
struct LatentTiles {
    int nht, hp, tpt;  // head tiles of a token, heads of one, tokens of a unit
    LatentTiles(int32_t H, bool lists) {
        nht = (H + LA_ROWS - 1) / LA_ROWS;
        hp = (H + nht - 1) / nht;
        tpt = lists || nht > 1 ? 1 : LA_ROWS / H;
    }
};

// Units of a head tile, at the host's bounds. Sequences without tokens have none, so there are no more than tokens.
int64_t latent_units(const LatentTiles& t, int32_t B, int64_t T, int64_t max_q, int32_t k) {
    return k > 0 ? T : std::min(T, B * ((max_q + t.tpt - 1) / t.tpt));
}

// Tiles of the line, at the host's bounds; more than 2^31 where they pass it.
int64_t latent_tiles(const LatentTiles& t, int32_t B, int64_t T, int64_t max_q, int64_t max_kv, int32_t k) {
    const int64_t keys = k > 0 ? k : max_kv, nt = (keys + LA_KEYS - 1) / LA_KEYS, units = latent_units(t, B, T, max_q, k);
    return units > INT32_MAX || nt > INT32_MAX ? int64_t(1) << 62 : units * nt;
}

// Runs: a CTA per SM and head tile, no more than there can be tiles; one at least.
int64_t latent_runs(const LatentTiles& t, int64_t tiles) {
    const int64_t sms = sm_count(), room = sms > t.nht ? sms / t.nht : 1;
    return tiles < room ? tiles : room;
}

size_t latent_desc_bytes(const LatentTiles& t, int64_t runs) { return align_up((size_t)runs * t.nht * sizeof(int4), 256); }

// Whether units go whole to blocks (no partial sums, no second kernel): where the most tiles that a block then has are
// no more than those of the line's runs and what the join costs, eight tiles' time where all SMs leave partial sums.
// Measured, 64 heads over bf16 entries of 576, us whole against line. Taken whole: 64 tokens of 512 listed entries 20.3
// and 26.6 (FP4 24.3 and 27.6, FP8 28.3 and 29.5), 150 tokens of 256 listed 15.5 and 22.2, and on the wrong side of the
// border 20 tokens of 512 listed 19.8 and 19.2 (FP4 22.8 and 20.4), 30 sequences of 600 entries 21.7 and 20.3. Taken
// along the line: eight tokens of 1024 listed 29.6 and 19.8, four sequences of 1000 entries 29.8 and 16.0, 12 of 400 17.2
// and 17.4, and on the wrong side 60 of 1000 30.7 and 35.4. (Clusters of 2, 4 or 8 blocks a unit, joined through
// distributed shared memory, were slower than the better of the two in at least fourteen of sixteen cases.)
bool latent_whole(const LatentAttendParams& p, int64_t tiles) {
    const int64_t keys = p.idx ? p.k : p.max_kv, nt = (keys + LA_KEYS - 1) / LA_KEYS, room = sm_count() / p.nht;
    const int64_t units = p.idx ? p.T : (int64_t)p.c.B * p.n_rt;
    if (room <= 0 || (!p.idx && units > room)) return false;
    return (units + room - 1) / room * nt <= (tiles + p.runs - 1) / p.runs + 1 + 7 * p.runs / room;
}

template <typename T, int DIM, int FMT>
hsi_status launch_latent_attend(const LatentAttendParams& p, int64_t units, cudaStream_t s) {
    using C = LatentCfg<DIM, FMT>;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (smem_attr_once(latent_attend_kernel<T, DIM, FMT>, C::SMEM_BYTES, attr_set) != HSI_OK) return HSI_ERR_CUDA;
    const unsigned grid = (unsigned)(p.runs * p.nht);
    const hsi_status st = launch(latent_attend_kernel<T, DIM, FMT>, dim3(grid), dim3(latent_threads(FMT)), C::SMEM_BYTES, s, p);
    if (st != HSI_OK || p.runs == 1 || p.whole) return st;
    const unsigned rows = (p.tpt * p.hp + 3) / 4;  // (the last four may pass the unit's rows, not the slot's)
    if (units >= p.runs / 8) return launch(latent_join_kernel<T, 1>, dim3(rows, grid), dim3(LJ_THREADS), 0, s, p);
    return launch(latent_join_kernel<T, 8>, dim3(rows * 8, (unsigned)units * p.nht), dim3(LJ_THREADS), 0, s, p);
}

}  // namespace

extern "C" {

size_t hsi_latent_entry_bytes(hsi_latent_format format, int32_t dim) {
    if (format < HSI_LATENT_BF16 || format > HSI_LATENT_FP4) return 0;
    if (!(dim == 512 || (dim == 576 && format != HSI_LATENT_FP4))) return 0;
    return (size_t)latent_entry_bytes(format, dim);
}

hsi_status hsi_latent_append(const hsi_latent_cache* cache, const void* x, int64_t x_token_stride,
                             const int32_t* q_start, int64_t T, const int32_t* positions, const uint64_t* steps,
                             int32_t rot, int32_t rot_offset, int32_t interleaved, float gain, cudaStream_t stream) {
    LatentAppendParams p{};
    const hsi_status st = latent_view(cache, &p.c);
    if (st != HSI_OK) return st;
    p.xt = row_stride(T, x_token_stride);
    if (!q_start || T <= 0 || T > INT32_MAX || !rows_ok(x, p.xt, 0)) return HSI_ERR_INVALID_ARG;
    if (steps) {
        if (!positions || !aligned(positions, 4) || !aligned(steps, 8) || !turn_ok(cache->dim, rot, rot_offset) ||
            !(gain == gain))
            return HSI_ERR_INVALID_ARG;
        if (rot % 16 || rot_offset % 8) return HSI_ERR_UNSUPPORTED;
        p.r = {reinterpret_cast<const unsigned long long*>(steps), positions, rot, rot_offset, interleaved != 0, gain, 1.f};
    }
    p.x = x;
    p.T = T;
    p.q_start = q_start;
    const dim3 grid((unsigned)((T + LT_WARPS - 1) / LT_WARPS)), block(32 * LT_WARPS);
    switch (cache->format) {
        case HSI_LATENT_BF16: return launch(latent_append_kernel<__nv_bfloat16, LF_BF16>, grid, block, 0, stream, p);
        case HSI_LATENT_FP16: return launch(latent_append_kernel<__half, LF_FP16>, grid, block, 0, stream, p);
        case HSI_LATENT_FP8: return launch(latent_append_kernel<__nv_bfloat16, LF_FP8>, grid, block, 0, stream, p);
        default: return launch(latent_append_kernel<__nv_bfloat16, LF_FP4>, grid, block, 0, stream, p);
    }
}

hsi_status hsi_latent_read(const hsi_latent_cache* cache, const int32_t* row_start, int64_t T, const int32_t* first,
                           const int32_t* idx, int64_t ld_idx, int32_t k, void* out, int64_t out_stride,
                           cudaStream_t stream) {
    LatentReadParams p{};
    const hsi_status st = latent_view(cache, &p.c);
    if (st != HSI_OK) return st;
    p.ot = row_stride(T, out_stride);
    if (!row_start || T <= 0 || T > INT32_MAX || !rows_ok(out, p.ot, 0)) return HSI_ERR_INVALID_ARG;
    if (!lists_ok(idx, ld_idx, k) || (idx && first)) return HSI_ERR_INVALID_ARG;
    if (T > 1 && p.ot < (int64_t)cache->dim * (idx ? k : 1)) return HSI_ERR_INVALID_ARG;  // two results in one place
    p.start = row_start;
    p.first = first;
    p.idx = idx;
    p.ld_idx = ld_idx;
    p.k = k;
    p.T = T;
    p.rows = idx ? T * k : T;
    p.out = static_cast<uint16_t*>(out);
    const int64_t blocks = (p.rows + LT_WARPS * LT_RPW - 1) / (LT_WARPS * LT_RPW);
    if (blocks > INT32_MAX) return HSI_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks), block(32 * LT_WARPS);
    switch (cache->format) {
        case HSI_LATENT_FP8: return launch(latent_read_kernel<LF_FP8>, grid, block, 0, stream, p);
        case HSI_LATENT_FP4: return launch(latent_read_kernel<LF_FP4>, grid, block, 0, stream, p);
        default: return launch(latent_read_kernel<LF_BF16>, grid, block, 0, stream, p);
    }
}

size_t hsi_latent_attention_ws(int32_t B, int32_t q_heads, int64_t T, int32_t max_q, int64_t max_kv, int32_t k) {
    if (B <= 0 || q_heads <= 0 || T <= 0 || max_q <= 0 || max_kv <= 0 || k < 0) return 0;
    const LatentTiles t(q_heads, k > 0);
    const int64_t runs = latent_runs(t, latent_tiles(t, B, T, max_q, max_kv, k));
    return latent_desc_bytes(t, runs) + align_up((size_t)runs * 2 * t.nht * LA_SLOT * 4, 256);
}

hsi_status hsi_latent_attention(const hsi_latent_cache* cache, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, int32_t q_heads, const int32_t* q_start, int64_t T,
                                int32_t max_q, int64_t max_kv, const int32_t* idx, int64_t ld_idx, int32_t k,
                                float scale, int32_t causal, void* out, int64_t o_token_stride, int64_t o_head_stride,
                                float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
    LatentAttendParams p{};
    const hsi_status st = latent_view(cache, &p.c);
    if (st != HSI_OK) return st;
    p.qt = row_stride(T, q_token_stride);
    p.qh = row_stride(q_heads, q_head_stride);
    p.ot = row_stride(T, o_token_stride);
    p.oh = row_stride(q_heads, o_head_stride);
    if (!q_start || T <= 0 || T > INT32_MAX || max_q <= 0 || max_kv <= 0 || max_kv > INT32_MAX || q_heads <= 0 ||
        !rows_ok(q, p.qt, p.qh) || !(scale == scale) || !lists_ok(idx, ld_idx, k))
        return HSI_ERR_INVALID_ARG;
    if (!rows_ok(out, p.ot, p.oh) || out == q || (T > 1 && p.ot < LT_VALUE) || (q_heads > 1 && p.oh < LT_VALUE))
        return HSI_ERR_INVALID_ARG;
    if (q_heads > 65535) return HSI_ERR_UNSUPPORTED;
    p.max_kv = (int)(max_kv < p.c.capacity ? max_kv : p.c.capacity);
    p.max_q = (int)(max_q < T ? max_q : T);
    if (p.max_kv > INT32_MAX - 4096 || k > INT32_MAX - 4096) return HSI_ERR_UNSUPPORTED;  // rounded up to tiles in 32 bits
    const LatentTiles tiles(q_heads, idx != nullptr);
    const int64_t most = latent_tiles(tiles, cache->B, T, p.max_q, p.max_kv, idx ? k : 0);
    if (most > INT32_MAX) return HSI_ERR_UNSUPPORTED;  // the kernels count them in 31 bits
    const size_t need = hsi_latent_attention_ws(cache->B, q_heads, T, p.max_q, p.max_kv, idx ? k : 0);
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return HSI_ERR_WORKSPACE;
    p.q = q;
    p.q_start = q_start;
    p.T = T;
    p.H = q_heads;
    p.nht = tiles.nht;
    p.hp = tiles.hp;
    p.tpt = tiles.tpt;
    p.idx = idx;
    p.ld_idx = ld_idx;
    p.k = idx ? k : 0;
    p.negate = scale < 0.f;
    p.sl2 = std::fmax(std::fabs(scale * LOG2E), 1e-30f);  // above 0, so that -inf stays -inf: at scale 0 every p is 1
    p.causal = causal != 0;
    p.out = out;
    p.lse = lse;
    if (sm_count() <= 0) return HSI_ERR_CUDA;
    p.runs = (int)latent_runs(tiles, most);
    p.desc = static_cast<int4*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + latent_desc_bytes(tiles, p.runs));
    p.inv_hp = 65536 / p.hp + 1;
    p.n_rt = (p.max_q + p.tpt - 1) / p.tpt;
    p.whole = latent_whole(p, most);
    // (a list's runs are of whole units then, a sequence's units are runs)
    if (p.whole) p.runs = (int)(idx ? std::min<int64_t>(T, sm_count() / p.nht) : (int64_t)cache->B * p.n_rt);
    const int64_t units = latent_units(tiles, cache->B, T, p.max_q, p.k);
    const bool wide = cache->dim > LT_VALUE;
    switch (cache->format) {
        case HSI_LATENT_BF16:
            return wide ? launch_latent_attend<__nv_bfloat16, 576, LF_BF16>(p, units, stream)
                        : launch_latent_attend<__nv_bfloat16, 512, LF_BF16>(p, units, stream);
        case HSI_LATENT_FP16:
            return wide ? launch_latent_attend<__half, 576, LF_FP16>(p, units, stream)
                        : launch_latent_attend<__half, 512, LF_FP16>(p, units, stream);
        case HSI_LATENT_FP8:
            return wide ? launch_latent_attend<__nv_bfloat16, 576, LF_FP8>(p, units, stream)
                        : launch_latent_attend<__nv_bfloat16, 512, LF_FP8>(p, units, stream);
        default: return launch_latent_attend<__nv_bfloat16, 512, LF_FP4>(p, units, stream);
    }
}

}  // extern "C"

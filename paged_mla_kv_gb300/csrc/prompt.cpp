// The C entries of the prompt path (include/tf_prompt.h): argument checks on the host, the rotary table,
// and the launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "tf_internal.h"

using namespace tf;

static constexpr uint32_t kRopeMade = 0x45504F52u;   // "ROPE"

extern "C" int tf_rope_make(const tf_rope_desc *d, tf_rope *out) {
    if (!d || !out) return TF_E_ARG;
    out->made = 0;
    if (d->dim < 16 || d->dim > TF_ROPE_MAX_DIM || d->dim % 16 != 0 || d->reserved != 0) return TF_E_ARG;
    if (d->layout != TF_ROPE_INTERLEAVED && d->layout != TF_ROPE_HALF) return TF_E_ARG;
    if (d->scaling != TF_ROPE_PLAIN && d->scaling != TF_ROPE_LINEAR && d->scaling != TF_ROPE_YARN) return TF_E_ARG;
    if (!(d->base > 1.0) || !std::isfinite(d->base) || !(d->amplitude >= 0.0) || !std::isfinite((float)d->amplitude)) return TF_E_ARG;
    const double pi = 3.14159265358979323846;
    double factor = 1.0, amplitude = 1.0, lo = 0.0, hi = 0.0;
    if (d->scaling != TF_ROPE_PLAIN) {
        if (!(d->factor >= 1.0) || !std::isfinite(d->factor)) return TF_E_ARG;
        factor = d->factor;
    }
    if (d->scaling == TF_ROPE_YARN) {
        if (!(d->original >= 1.0) || !std::isfinite(d->original) || !(d->beta_slow > 0.0) || !(d->beta_fast > d->beta_slow) ||
            !std::isfinite(d->beta_fast))
            return TF_E_ARG;
        auto pair_of = [&](double turns) { return d->dim * std::log(d->original / (2.0 * pi * turns)) / (2.0 * std::log(d->base)); };
        lo = std::fmax(0.0, std::floor(pair_of(d->beta_fast)));
        hi = std::fmin(d->dim - 1.0, std::ceil(pair_of(d->beta_slow)));
        amplitude = 0.1 * std::log(factor) + 1.0;
    }
    for (int i = 0; i < d->dim / 2; ++i) {
        double f = std::pow(d->base, -2.0 * i / d->dim);
        if (d->scaling == TF_ROPE_LINEAR) f /= factor;
        if (d->scaling == TF_ROPE_YARN) {
            const double r = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
            f = f * (1.0 - r) + f / factor * r;
        }
        // f <= 1 radian, a sixth of a turn: below 2^62
        out->turn[i] = (uint64_t)std::llround(std::ldexp(f / (2.0 * pi), 64));
    }
    for (int i = d->dim / 2; i < TF_ROPE_MAX_DIM / 2; ++i) out->turn[i] = 0;
    out->dim = d->dim;
    out->layout = d->layout;
    out->amplitude = (float)(d->amplitude > 0.0 ? d->amplitude : amplitude);
    out->made = kRopeMade;
    return TF_OK;
}

// Packed rows: the streams' counts and positions, below `limit` rows of a stream.  *rows: all of them.
static int packed_checks(const int64_t *h_pos, const int64_t *h_n, int32_t S, int64_t limit, int64_t *rows) {
    if (!h_pos || !h_n || S < 1 || S > TF_MAX_STREAMS) return TF_E_ARG;
    for (int s = 0; s < S; ++s)
        if (h_n[s] < 0) return TF_E_ARG;
    *rows = 0;
    for (int s = 0; s < S; ++s) {
        if (h_pos[s] < 0 || h_n[s] > limit || h_pos[s] > limit - h_n[s]) return TF_E_RANGE;
        *rows += h_n[s];   // at most TF_MAX_STREAMS times 2^31
    }
    return *rows > INT32_MAX ? TF_E_UNSUPPORTED : TF_OK;
}

static bool unaligned(const void *p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether two of rows x heads blocks of `width` values, at r * row + h * head, have a value in common.
static bool overlap(int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t width) {
    using wide = __int128;
    const wide a = row < 0 ? -(wide)row : row, b = head < 0 ? -(wide)head : head;
    if ((rows > 1 && a < width) || (heads > 1 && b < width)) return true;
    if (rows <= 1 || heads <= 1 || a >= b * (heads - 1) + width || b >= a * (rows - 1) + width) return false;
    // heads and rows that lie among one another: the rows nearest to each distance of two heads
    for (int64_t h = 1; h < heads; ++h)
        for (wide r = b * h / a, last = r + 1; r <= last; ++r)
            if (r < rows && r * a - b * h < width && b * h - r * a < width) return true;
    return false;
}

extern "C" int tf_rope_apply(const tf_rope *rope, const int64_t *h_pos, const int64_t *h_n, int32_t S, int32_t H,
                             const void *d_x, int64_t x_row, int64_t x_head, void *d_y, int64_t y_row, int64_t y_head,
                             void *stream) {
    if (!rope || rope->made != kRopeMade || H < 1 || H > TF_MAX_HEADS) return TF_E_ARG;
    if (x_row % 8 != 0 || x_head % 8 != 0 || y_row % 8 != 0 || y_head % 8 != 0) return TF_E_ARG;
    int64_t n = 0;
    const int rc = packed_checks(h_pos, h_n, S, (int64_t)INT32_MAX + 1, &n);
    if (rc != TF_OK) return rc;
    if (n == 0) return TF_OK;
    if (!d_x || !d_y || unaligned(d_x) || unaligned(d_y) || overlap(n, y_row, H, y_head, rope->dim)) return TF_E_ARG;
    return no_throw([&] { return launch_rope(rope, h_pos, h_n, S, H, d_x, x_row, x_head, d_y, y_row, y_head, (cudaStream_t)stream); });
}

// What the calls over pages refuse.
static int paged_checks(const tf_kvpool *p, int32_t cache, const int32_t *d_pt, int32_t max_pages, const int64_t *h_pos,
                        const int64_t *h_n, int32_t S, int64_t *rows) {
    if (!p || max_pages < 1 || unaligned(d_pt, 4)) return TF_E_ARG;
    const int64_t limit = std::min<int64_t>((int64_t)max_pages * kPageRows, (int64_t)INT32_MAX + 1);
    const int rc = packed_checks(h_pos, h_n, S, limit, rows);
    if (rc == TF_E_ARG) return rc;
    if (cache < 0 || cache >= p->desc.num_caches) return TF_E_RANGE;
    if (!d_pt && (int64_t)S * max_pages > p->desc.num_pages) return TF_E_RANGE;
    return rc;
}

extern "C" int tf_paged_append_rope(tf_kvpool *p, int32_t cache, const int32_t *d_pt, int32_t max_pages,
                                    const int64_t *h_pos, const int64_t *h_n, int32_t S, const void *d_rows,
                                    int64_t row_stride, const void *d_gain, float eps, const tf_rope *rope, void *stream) {
    if (rope && (rope->made != kRopeMade || rope->dim != kRope)) return TF_E_ARG;
    if (row_stride % 8 != 0 || row_stride < kDk || unaligned(d_gain) || (d_gain && (!(eps > 0.0f) || !std::isfinite(eps)))) return TF_E_ARG;
    int64_t n = 0;
    const int rc = paged_checks(p, cache, d_pt, max_pages, h_pos, h_n, S, &n);
    if (rc != TF_OK) return rc;
    if (n == 0) return TF_OK;
    if (!d_rows || unaligned(d_rows)) return TF_E_ARG;
    return no_throw([&] {
        return launch_append_rope(p, cache, d_pt, max_pages, h_pos, h_n, S, d_rows, row_stride, d_gain, eps, rope, (cudaStream_t)stream);
    });
}

extern "C" int tf_paged_read(tf_kvpool *p, int32_t cache, const int32_t *d_pt, int32_t max_pages, const int64_t *h_from,
                             const int64_t *h_n, int32_t S, void *d_latent, int64_t lat_stride, void *d_rope,
                             int64_t rope_stride, void *stream) {
    if (!d_latent && !d_rope) return TF_E_ARG;
    if (d_latent && (unaligned(d_latent) || lat_stride % 8 != 0 || lat_stride < kLat)) return TF_E_ARG;
    if (d_rope && (unaligned(d_rope) || rope_stride % 8 != 0 || rope_stride < kRope)) return TF_E_ARG;
    int64_t n = 0;
    const int rc = paged_checks(p, cache, d_pt, max_pages, h_from, h_n, S, &n);
    if (rc != TF_OK) return rc;
    if (n == 0) return TF_OK;
    return no_throw([&] {
        return launch_paged_read(p, cache, d_pt, max_pages, h_from, h_n, S, d_latent, lat_stride, d_rope, rope_stride, (cudaStream_t)stream);
    });
}

// ---- attention of prompts ----
static int prompt_checks(const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv, int32_t dqk, int32_t dv,
                         int32_t causal, int64_t *rows, int64_t *keys) {
    if (!h_nq || !h_nk || S < 1 || S > TF_MAX_STREAMS || H < 1 || H > TF_MAX_HEADS || Hkv < 1 || H % Hkv != 0 ||
        (causal != 0 && causal != 1))
        return TF_E_ARG;
    for (int s = 0; s < S; ++s)
        if (h_nq[s] < 0 || h_nk[s] < 0) return TF_E_ARG;
    if (!((dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 192 && dv == 128))) return TF_E_UNSUPPORTED;
    *rows = *keys = 0;
    for (int s = 0; s < S; ++s) {
        if (h_nq[s] > INT32_MAX - *rows || h_nk[s] > INT32_MAX - *keys) return TF_E_UNSUPPORTED;
        *rows += h_nq[s];
        *keys += h_nk[s];
    }
    return TF_OK;
}

extern "C" size_t tf_prompt_workspace_bytes(const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv,
                                            int32_t dqk, int32_t dv, int32_t causal) {
    int64_t rows, keys;
    if (prompt_checks(h_nq, h_nk, S, H, Hkv, dqk, dv, causal, &rows, &keys) != TF_OK) return 0;
    size_t n = 0;
    const int rc = no_throw([&] { return prompt_plan(h_nq, h_nk, S, H, Hkv, dqk, dv, causal, 0, nullptr, &n); });
    return rc == TF_OK ? n : 0;
}

extern "C" int tf_prompt_plan_info(const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv, int32_t dqk,
                                   int32_t dv, int32_t causal, int32_t sms, tf_prompt_plan *info) {
    if (!info) return TF_E_ARG;
    int64_t rows, keys;
    const int rc = prompt_checks(h_nq, h_nk, S, H, Hkv, dqk, dv, causal, &rows, &keys);
    if (rc != TF_OK) return rc;
    return no_throw([&] { return prompt_plan(h_nq, h_nk, S, H, Hkv, dqk, dv, causal, sms, info, nullptr); });
}

// A TMA view's pointer and strides: 16 bytes, strides up to 2^36 values.
static bool bad_view(const void *p, int64_t row, int64_t head, int32_t heads) {
    constexpr int64_t most = (int64_t)1 << 36;
    return !p || unaligned(p) || row % 8 != 0 || row < 1 || row > most ||
           (heads > 1 && (head % 8 != 0 || head < 1 || head > most));
}

extern "C" int tf_prompt_attend(tf_kvpool *p, const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv,
                                int32_t dqk, int32_t dv, const tf_heads *q, const tf_heads *k, const void *d_kr,
                                int64_t kr_row, const tf_heads *v, float scale, int32_t causal, const tf_heads *out,
                                float *d_lse, void *d_ws, size_t ws_bytes, void *stream) {
    if (!p || unaligned(d_lse, 4) || !(scale > 0.0f) || !std::isfinite(2.0f * scale)) return TF_E_ARG;
    int64_t rows = 0, keys = 0;
    const int rc = prompt_checks(h_nq, h_nk, S, H, Hkv, dqk, dv, causal, &rows, &keys);
    if (rc != TF_OK) return rc;
    if (d_kr && dqk == 64) return TF_E_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    if (!q || !out || bad_view(q->d_p, q->row, q->head, H)) return TF_E_ARG;
    if (keys > 0 && (!k || !v || bad_view(k->d_p, k->row, k->head, Hkv) || bad_view(v->d_p, v->row, v->head, Hkv) ||
                     (d_kr && bad_view(d_kr, kr_row, 8, 1))))
        return TF_E_ARG;
    if (!out->d_p || unaligned(out->d_p) || out->row % 8 != 0 || out->head % 8 != 0 || overlap(rows, out->row, H, out->head, dv)) return TF_E_ARG;
    return no_throw([&] {
        return launch_prompt_attend(p, h_nq, h_nk, S, H, Hkv, dqk, dv, q, k, keys > 0 ? d_kr : nullptr, kr_row, v, scale, causal, out,
                                    d_lse, d_ws, ws_bytes, (cudaStream_t)stream);
    });
}

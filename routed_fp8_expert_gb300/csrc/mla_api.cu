// C ABI of the latent attention (declared in include/moe_fp8.h): argument checks,
// tensor maps and workspace layout.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "mla.cuh"
#include "moe_fp8.h"

using namespace moe;

namespace {

int fail(int code, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return report_error(code, msg);
}

#define MLA_CUDA(call, what)                                                                             \
    do {                                                                                                 \
        cudaError_t e_ = (call);                                                                         \
        if (e_ != cudaSuccess)                                                                           \
            return fail(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e_), cudaGetErrorString(e_)); \
    } while (0)

#define MLA_CHECK(expr)              \
    do {                             \
        int s_ = (expr);             \
        if (s_ != MOE_OK) return s_; \
    } while (0)

int ptr(const void *p, const char *name, unsigned align = 16) {
    if (!p) return fail(MOE_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1)) return fail(MOE_ERR_ARG, "%s is not %u-byte aligned", name, align);
    return MOE_OK;
}

// A stride of 16-bit elements: at least `least` (0: rows may not overlap only in the
// caller's care), a multiple of 8, and below the tensor maps' 2^40-byte limit.
int stride(int64_t s, int64_t least, const char *name) {
    if (s < least || s <= 0 || s % 8 || s >= (int64_t{1} << 38))
        return fail(MOE_ERR_ARG, "%s=%lld must be a multiple of 8, at least %lld and below 2^38", name,
                    static_cast<long long>(s), static_cast<long long>(least));
    return MOE_OK;
}

int range(int64_t v, int64_t lo, int64_t hi, const char *name) {
    if (v < lo || v > hi)
        return fail(MOE_ERR_UNSUPPORTED, "%s=%lld must be in [%lld, %lld]", name, static_cast<long long>(v),
                    static_cast<long long>(lo), static_cast<long long>(hi));
    return MOE_OK;
}

int dtype_ok(int dtype) {
    if (dtype != MLA_BF16 && dtype != MLA_FP16) return fail(MOE_ERR_ARG, "dtype=%d must be MLA_BF16 or MLA_FP16", dtype);
    return MOE_OK;
}

int count(int64_t n, const char *name) {
    if (n < 0) return fail(MOE_ERR_ARG, "%s=%lld is negative", name, static_cast<long long>(n));
    return range(n, 0, (int64_t{1} << 31) - 1024, name);
}

// A tensor map of 16-bit elements with the 128-byte swizzle; dims and box innermost
// first, strides in elements from the second dimension on.
int tensor_map(CUtensorMap *m, const void *p, int dtype, int rank, const int64_t *dims, const int64_t *strides,
               const int *box, const char *name) {
    auto fn = encode_fn();
    if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], e[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        b[i] = static_cast<cuuint32_t>(box[i]);
        if (i + 1 < rank) s[i] = static_cast<cuuint64_t>(strides[i]) * 2;
    }
    const CUresult r = fn(m, dtype == MLA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          rank, const_cast<void *>(p), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (%s) failed (%d)", name, static_cast<int>(r));
    return MOE_OK;
}

// (the offsets on the device say which rows the sequences hold; without any, no row is)
int sequences(int B, int64_t Tq) {
    if (B == 0) return fail(MOE_ERR_ARG, "B=0 sequences for Tq=%lld rows", static_cast<long long>(Tq));
    return MOE_OK;
}

int proj_sizes(int T, int H, int K, int N) {
    MLA_CHECK(range(H, 1, 1024, "H"));
    if (K < 8 || K > 8192 || K % 8) return fail(MOE_ERR_UNSUPPORTED, "K=%d must be a multiple of 8 in [8, 8192]", K);
    if (N < 8 || N > 8192 || N % 8) return fail(MOE_ERR_UNSUPPORTED, "N=%d must be a multiple of 8 in [8, 8192]", N);
    MLA_CHECK(count(T, "T"));
    MLA_CHECK(range(T, 0, 1 << 20, "T"));
    return MOE_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

int scale_ok(float scale) {
    if (!std::isfinite(scale) || scale <= 0.f) return fail(MOE_ERR_ARG, "scale must be positive and finite");
    return MOE_OK;
}

// mla_attn_paged's workspace for a grid of n CTAs: two partial results of 64 rows per
// CTA (fp32 sums, then their reference maxima and exponential sums), one join entry each.
constexpr size_t kPartBytes = 64 * kMlaLatent * 4;
size_t paged_ws(int n) {
    return static_cast<size_t>(n) * 2 * (kPartBytes + 64 * sizeof(float2)) + static_cast<size_t>(n) * sizeof(int4);
}

}  // namespace

extern "C" {

int mla_rope_freqs(int dim, double base, double factor, int original_ctx, double beta_fast, double beta_slow,
                   uint64_t *freq) {
    report_launches(0);
    if (dim < 2 || dim > 256 || dim % 2) return fail(MOE_ERR_UNSUPPORTED, "dim=%d must be even and in [2, 256]", dim);
    if (!std::isfinite(base) || base <= 1.0) return fail(MOE_ERR_ARG, "base must be finite and above 1");
    if (!std::isfinite(factor) || factor < 1.0) return fail(MOE_ERR_ARG, "factor must be finite and at least 1");
    if (!freq) return fail(MOE_ERR_ARG, "freq is NULL");
    const double two_pi = 6.283185307179586476925;
    double low = 0.0, high = 0.0;
    if (factor > 1.0) {
        if (original_ctx < 1) return fail(MOE_ERR_ARG, "original_ctx=%d must be positive", original_ctx);
        if (!(beta_fast > 0.0) || !(beta_slow > 0.0) || !std::isfinite(beta_fast) || !std::isfinite(beta_slow))
            return fail(MOE_ERR_ARG, "beta_fast and beta_slow must be positive and finite");
        auto pair = [&](double turns) { return dim * std::log(original_ctx / (two_pi * turns)) / (2.0 * std::log(base)); };
        low = std::fmax(std::floor(pair(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair(beta_slow)), dim - 1.0);
    }
    for (int i = 0; i < dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / dim) / two_pi;
        if (factor > 1.0) {
            const double ramp = std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 0.001)));
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        freq[i] = static_cast<uint64_t>(std::ldexp(f, 64));   // f < 1 / (2 pi): below 2^62
    }
    return MOE_OK;
}

int mla_rope_append(const void *q, int64_t q_st, int64_t q_sh, void *q_out, int64_t qo_st, int64_t qo_sh,
                    const void *kv, int64_t kv_st, const void *gamma, float eps, void *kv_out, int64_t kvo_st,
                    void *cache, int64_t page_st, int64_t row_st, int64_t num_pages, int page_size,
                    const int32_t *slots, const int32_t *positions, const uint64_t *freq, float amplitude,
                    int layout, int T, int H, int dim, int latent, int dtype, void *stream) {
    report_launches(0);
    MLA_CHECK(dtype_ok(dtype));
    if (dim < 16 || dim > 256 || dim % 16)
        return fail(MOE_ERR_UNSUPPORTED, "dim=%d must be a multiple of 16 in [16, 256]", dim);
    if (layout != 0 && layout != 1) return fail(MOE_ERR_ARG, "layout=%d must be 0 or 1", layout);
    if (!std::isfinite(amplitude)) return fail(MOE_ERR_ARG, "amplitude is not finite");
    MLA_CHECK(count(T, "T"));
    if (T == 0) return MOE_OK;
    if (!q && !kv) return fail(MOE_ERR_ARG, "q and kv are both NULL");
    if (kv && (latent < 8 || latent % 8 || latent + dim > 2048))
        return fail(MOE_ERR_UNSUPPORTED, "latent=%d must be a positive multiple of 8, latent + dim at most 2048", latent);
    if (q) MLA_CHECK(range(H, 1, 1024, "H"));
    if (q) {
        MLA_CHECK(ptr(q, "q"));
        MLA_CHECK(ptr(q_out, "q_out"));
        MLA_CHECK(stride(q_st, 8, "q_st"));
        MLA_CHECK(stride(q_sh, 8, "q_sh"));
        MLA_CHECK(stride(qo_st, dim, "qo_st"));
        MLA_CHECK(stride(qo_sh, H > 1 ? dim : 8, "qo_sh"));
    }
    if (kv) {
        MLA_CHECK(ptr(kv, "kv"));
        MLA_CHECK(stride(kv_st, 8, "kv_st"));
        if (gamma) {
            MLA_CHECK(ptr(gamma, "gamma"));
            if (!std::isfinite(eps) || eps < 0.f) return fail(MOE_ERR_ARG, "eps must be finite and not negative");
        }
        if (!kv_out && !cache) return fail(MOE_ERR_ARG, "kv is given, but neither kv_out nor cache");
        if (kv_out) {
            MLA_CHECK(ptr(kv_out, "kv_out"));
            MLA_CHECK(stride(kvo_st, latent + dim, "kvo_st"));
        }
        if (cache) {
            MLA_CHECK(ptr(cache, "cache"));
            MLA_CHECK(ptr(slots, "slots", 4));
            MLA_CHECK(range(page_size, 1, 1 << 20, "page_size"));
            MLA_CHECK(range(num_pages, 0, (int64_t{1} << 31) - 1, "num_pages"));
            MLA_CHECK(stride(row_st, latent + dim, "row_st"));
            MLA_CHECK(stride(page_st, latent + dim, "page_st"));
        }
    }
    MLA_CHECK(ptr(positions, "positions", 4));
    MLA_CHECK(ptr(freq, "freq", 8));
    RopeArgs a{};
    a.q = q, a.q_st = q_st, a.q_sh = q_sh, a.q_out = q_out, a.qo_st = qo_st, a.qo_sh = qo_sh;
    a.kv = kv, a.kv_st = kv_st, a.gamma = gamma, a.kv_out = kv_out, a.kvo_st = kvo_st;
    a.cache = kv ? cache : nullptr;
    a.page_st = page_st, a.row_st = row_st, a.num_pages = num_pages, a.page_size = page_size;
    a.slots = slots, a.positions = positions, a.freq = freq;
    a.T = T, a.H = H, a.dim = dim, a.latent = latent, a.layout = layout;
    a.amplitude = amplitude, a.eps = eps;
    MLA_CUDA(device_error_word(&a.err), "error word address");
    MLA_CUDA(launch_rope(a, dtype == MLA_BF16, static_cast<cudaStream_t>(stream)), "rotary launch");
    report_launches(1);
    return MOE_OK;
}

size_t mla_paged_workspace_bytes(void) { return paged_ws(num_sms()); }

int mla_attn_paged(const void *q, int64_t q_st, int64_t q_sh, int64_t Tq, const void *cache, int64_t page_st,
                   int64_t row_st, int64_t num_pages, int page_size, const int32_t *table, int64_t table_st,
                   int max_pages, const int32_t *ctx, const int32_t *cu_q, int B, int H, float scale, int dtype,
                   void *out, int64_t o_st, int64_t o_sh, float *lse, void *workspace, size_t workspace_bytes,
                   void *stream) {
    report_launches(0);
    MLA_CHECK(dtype_ok(dtype));
    MLA_CHECK(scale_ok(scale));
    MLA_CHECK(range(H, 1, 128, "H"));
    if (B < 0) return fail(MOE_ERR_ARG, "B=%d is negative", B);
    MLA_CHECK(range(B, 0, 8192, "B"));
    MLA_CHECK(count(Tq, "Tq"));
    MLA_CHECK(range(Tq * H, 0, (int64_t{1} << 31) - 1024, "Tq * H"));
    if (!cu_q && Tq != B)
        return fail(MOE_ERR_ARG, "Tq=%lld must equal B=%d when cu_q is NULL", static_cast<long long>(Tq), B);
    if (page_size <= 0 || page_size % 8 || page_size > (1 << 20))
        return fail(MOE_ERR_UNSUPPORTED, "page_size=%d must be a multiple of 8 in [8, 2^20]", page_size);
    MLA_CHECK(range(num_pages, 1, (int64_t{1} << 31) - 2, "num_pages"));
    if (Tq == 0) return MOE_OK;
    MLA_CHECK(sequences(B, Tq));
    MLA_CHECK(range(max_pages, 0, (int64_t{1} << 31) - 1, "max_pages"));
    MLA_CHECK(ptr(q, "q"));
    MLA_CHECK(stride(q_st, 8, "q_st"));
    MLA_CHECK(stride(q_sh, 8, "q_sh"));
    MLA_CHECK(ptr(cache, "cache"));
    MLA_CHECK(stride(row_st, kMlaWidth, "row_st"));
    MLA_CHECK(stride(page_st, kMlaWidth, "page_st"));
    if (max_pages > 0) MLA_CHECK(ptr(table, "table", 4));   // (without pages no sequence has keys)
    if (table_st < max_pages && B > 1)
        return fail(MOE_ERR_ARG, "table_st=%lld is below max_pages=%d", static_cast<long long>(table_st), max_pages);
    MLA_CHECK(ptr(ctx, "ctx", 4));
    if (cu_q) MLA_CHECK(ptr(cu_q, "cu_q", 4));
    MLA_CHECK(ptr(out, "out"));
    MLA_CHECK(stride(o_st, kMlaLatent, "o_st"));
    MLA_CHECK(stride(o_sh, H > 1 ? kMlaLatent : 8, "o_sh"));
    if (lse) MLA_CHECK(ptr(lse, "lse", 4));
    const int grid = num_sms();
    if (workspace_bytes < paged_ws(grid))
        return fail(MOE_ERR_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, paged_ws(grid));
    MLA_CHECK(ptr(workspace, "workspace"));

    PagedArgs a{};
    a.Tq = Tq;
    a.table = table, a.table_st = table_st, a.ctx = ctx, a.cu_q = cu_q;
    a.out = out, a.o_st = o_st, a.o_sh = o_sh, a.lse = lse;
    a.num_pages = num_pages, a.max_pages = max_pages, a.page_size = page_size;
    // rows of one load: the largest of 64, 32, 16, 8 that divides the page, so that a
    // load never crosses a page
    a.box_rows = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : 8;
    a.B = B, a.H = H;
    a.scale_log2 = scale * kLog2e;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.part_o = reinterpret_cast<float *>(ws);
    ws += static_cast<size_t>(grid) * 2 * kPartBytes;
    a.part_ml = reinterpret_cast<float2 *>(ws);
    ws += static_cast<size_t>(grid) * 2 * 64 * sizeof(float2);
    a.joins = reinterpret_cast<int4 *>(ws);
    MLA_CUDA(device_error_word(&a.err), "error word address");

    // the queries as (column of a 64-column group, head, group, token): one load takes the
    // largest power-of-two share of the heads that also divides the 64 rows of a tile,
    // so that loads start on multiples of it and never cross a token
    a.q_box = std::min(64, H & -H);
    PagedMaps m;
    {
        const int64_t d[4] = {64, H, kMlaWidth / 64, Tq}, s[3] = {q_sh, 64, q_st};
        const int box[4] = {64, a.q_box, a.q_box == 64 ? kMlaWidth / 64 : 1, 1};
        MLA_CHECK(tensor_map(&m.q, q, dtype, 4, d, s, box, "q"));
    }
    // the cache as (column of a 64-column group, row of a page, group, page)
    const int64_t dims[4] = {64, page_size, kMlaWidth / 64, num_pages};
    const int64_t strides[3] = {row_st, 64, page_st};
    for (int groups : {1, 2}) {
        const int box[4] = {64, a.box_rows, groups, 1};
        MLA_CHECK(tensor_map(groups == 1 ? &m.group : &m.pair, cache, dtype, 4, dims, strides, box, "cache"));
    }
    MLA_CUDA(launch_paged(m, a, dtype == MLA_BF16, grid, static_cast<cudaStream_t>(stream)), "paged attention launch");
    report_launches(2);
    return MOE_OK;
}

int mla_attn_ragged(const void *q, int64_t q_st, int64_t q_sh, int64_t Tq, const void *k_nope, int64_t kn_st,
                    int64_t kn_sh, const void *k_pe, int64_t kp_st, const void *v, int64_t v_st, int64_t v_sh,
                    int64_t Tk, const int32_t *cu_q, const int32_t *cu_k, int B, int max_q, int H, float scale,
                    int causal, int dtype, void *out, int64_t o_st, int64_t o_sh, float *lse, void *stream) {
    report_launches(0);
    MLA_CHECK(dtype_ok(dtype));
    MLA_CHECK(scale_ok(scale));
    if (causal != 0 && causal != 1) return fail(MOE_ERR_ARG, "causal=%d must be 0 or 1", causal);
    MLA_CHECK(range(H, 1, 1024, "H"));
    if (B < 0) return fail(MOE_ERR_ARG, "B=%d is negative", B);
    MLA_CHECK(range(B, 0, 65535, "B"));
    MLA_CHECK(count(Tq, "Tq"));
    MLA_CHECK(count(Tk, "Tk"));
    MLA_CHECK(count(max_q, "max_q"));
    if (Tq == 0) return MOE_OK;
    MLA_CHECK(sequences(B, Tq));
    MLA_CHECK(ptr(q, "q"));
    MLA_CHECK(stride(q_st, 8, "q_st"));
    MLA_CHECK(stride(q_sh, 8, "q_sh"));
    if (Tk > 0) {
        MLA_CHECK(ptr(k_nope, "k_nope"));
        MLA_CHECK(stride(kn_st, 8, "kn_st"));
        MLA_CHECK(stride(kn_sh, 8, "kn_sh"));
        MLA_CHECK(ptr(k_pe, "k_pe"));
        MLA_CHECK(stride(kp_st, 8, "kp_st"));
        MLA_CHECK(ptr(v, "v"));
        MLA_CHECK(stride(v_st, 8, "v_st"));
        MLA_CHECK(stride(v_sh, 8, "v_sh"));
    }
    MLA_CHECK(ptr(cu_q, "cu_q", 4));
    MLA_CHECK(ptr(cu_k, "cu_k", 4));
    MLA_CHECK(ptr(out, "out"));
    MLA_CHECK(stride(o_st, kMlaV, "o_st"));
    MLA_CHECK(stride(o_sh, H > 1 ? kMlaV : 8, "o_sh"));
    if (lse) MLA_CHECK(ptr(lse, "lse", 4));

    RaggedArgs a{};
    a.cu_q = cu_q, a.cu_k = cu_k, a.Tq = Tq, a.Tk = Tk;
    a.out = out, a.o_st = o_st, a.o_sh = o_sh, a.lse = lse;
    a.B = B, a.H = H, a.max_q = max_q, a.causal = causal;
    a.scale_log2 = scale * kLog2e;
    MLA_CUDA(device_error_word(&a.err), "error word address");
    CUtensorMap mq, mkn, mkp, mv;
    const int box[3] = {64, 1, 128};
    {
        const int64_t d[3] = {kMlaNope + kMlaRope, H, Tq}, s[2] = {q_sh, q_st};
        MLA_CHECK(tensor_map(&mq, q, dtype, 3, d, s, box, "q"));
    }
    if (Tk > 0) {
        const int64_t d[3] = {kMlaNope, H, Tk}, s[2] = {kn_sh, kn_st};
        MLA_CHECK(tensor_map(&mkn, k_nope, dtype, 3, d, s, box, "k_nope"));
        const int64_t dp[2] = {kMlaRope, Tk}, sp[1] = {kp_st};
        const int boxp[2] = {64, 128};
        MLA_CHECK(tensor_map(&mkp, k_pe, dtype, 2, dp, sp, boxp, "k_pe"));
        const int64_t dv[3] = {kMlaV, H, Tk}, sv[2] = {v_sh, v_st};
        MLA_CHECK(tensor_map(&mv, v, dtype, 3, dv, sv, box, "v"));
    } else {
        mkn = mkp = mv = mq;   // no key exists: nothing is loaded through them
    }
    MLA_CUDA(launch_ragged(mq, mkn, mkp, mv, a, dtype == MLA_BF16, static_cast<cudaStream_t>(stream)),
             "ragged attention launch");
    report_launches(1);
    return MOE_OK;
}

int mla_head_proj(const void *x, int64_t x_st, int64_t x_sh, int x_shared, const void *w, int64_t w_sh,
                  int64_t w_sr, int w_kn, int T, int H, int K, int N, int dtype, void *out, int64_t o_st,
                  int64_t o_sh, void *stream) {
    report_launches(0);
    MLA_CHECK(dtype_ok(dtype));
    if (x_shared != 0 && x_shared != 1) return fail(MOE_ERR_ARG, "x_shared=%d must be 0 or 1", x_shared);
    if (w_kn != 0 && w_kn != 1) return fail(MOE_ERR_ARG, "w_kn=%d must be 0 or 1", w_kn);
    MLA_CHECK(proj_sizes(T, H, K, N));
    if (T == 0) return MOE_OK;
    MLA_CHECK(ptr(x, "x"));
    MLA_CHECK(stride(x_st, 8, "x_st"));
    if (!x_shared) MLA_CHECK(stride(x_sh, 8, "x_sh"));
    MLA_CHECK(ptr(w, "w"));
    MLA_CHECK(stride(w_sr, w_kn ? N : K, "w_sr"));
    MLA_CHECK(stride(w_sh, 8, "w_sh"));
    MLA_CHECK(ptr(out, "out"));
    MLA_CHECK(stride(o_st, N, "o_st"));
    MLA_CHECK(stride(o_sh, H > 1 ? N : 8, "o_sh"));
    ProjArgs a{};
    a.T = T, a.H = H, a.K = K, a.N = N, a.shared_x = x_shared;
    // no more rows than the call has, up to the next power of two: rows past T would cost a
    // request each, and all CTAs' at the same place when the heads share x (one token,
    // 512 -> 64 x 256, 20.7 us with 128-row loads)
    for (a.x_rows = 128; a.x_rows > 8 && a.x_rows / 2 >= T;) a.x_rows /= 2;
    MLA_CUDA(device_error_word(&a.err), "error word address");
    CUtensorMap mx, mw, mo;
    {
        const int64_t d[3] = {N, H, T}, s[2] = {o_sh, o_st};
        const int box[3] = {64, 1, 32};
        MLA_CHECK(tensor_map(&mo, out, dtype, 3, d, s, box, "out"));
    }
    {
        const int64_t d[3] = {K, x_shared ? 1 : H, T}, s[2] = {x_shared ? x_st : x_sh, x_st};
        const int box[3] = {64, 1, a.x_rows};
        MLA_CHECK(tensor_map(&mx, x, dtype, 3, d, s, box, "x"));
    }
    {
        const int64_t d[3] = {w_kn ? N : K, w_kn ? K : N, H}, s[2] = {w_sr, w_sh};
        const int box[3] = {64, w_kn ? 64 : 128, 1};
        MLA_CHECK(tensor_map(&mw, w, dtype, 3, d, s, box, "w"));
    }
    MLA_CUDA(launch_proj(mx, mw, mo, a, dtype == MLA_BF16, w_kn != 0, num_sms(), static_cast<cudaStream_t>(stream)),
             "head projection launch");
    report_launches(1);
    return MOE_OK;
}

int mla_head_proj_form(int T, int H, int K, int N, int x_shared) {
    report_launches(0);
    if (x_shared != 0 && x_shared != 1) return fail(MOE_ERR_ARG, "x_shared=%d must be 0 or 1", x_shared);
    MLA_CHECK(proj_sizes(T, H, K, N));
    return T > 0 && proj_uses_pairs(T, H, K, N, x_shared != 0) ? 1 : 0;
}

}  // extern "C"

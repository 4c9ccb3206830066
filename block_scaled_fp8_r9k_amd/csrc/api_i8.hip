// The C ABI of the 8-bit integer products and of the router's training operators: argument
// checks, plans and launches.  Declarations, argument meanings and error behaviour: r9k.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_checks.h"
#include "i8_internal.h"

using namespace r9k;

namespace r9k {
I8Tuning &i8_tuning() {
    static I8Tuning t{};
    return t;
}
}  // namespace r9k

static std::atomic<int> g_i8_setting{0};  // counts the changes of the plan control

// The plan of a shape under the present setting, kept for each thread's last shapes:
// planning takes longer than a launch.
static const I8Plan &i8_plan(int64_t M, int64_t K, int64_t N, int64_t E, bool silu, bool quant, bool wide = false) {
    struct Entry {
        int64_t M = -1, K, N, E;
        int setting, kind;
        I8Plan plan;
    };
    static thread_local Entry table[64];
    const int kind = silu + 2 * quant + 4 * wide, setting = g_i8_setting.load(std::memory_order_relaxed);
    const uint64_t h = ((uint64_t)M * 0x9E3779B97F4A7C15u) ^ ((uint64_t)K * 0xC2B2AE3D27D4EB4Fu) ^
                       ((uint64_t)N * 0x165667B19E3779F9u) ^ ((uint64_t)(8 * E + kind) * 0x27D4EB2F165667C5u);
    Entry &t = table[h >> 58];
    if (t.M != M || t.K != K || t.N != N || t.E != E || t.kind != kind || t.setting != setting) {
        t.plan = i8_plan_new(M, K, N, E, silu, quant, wide);
        t.M = M, t.K = K, t.N = N, t.E = E, t.kind = kind, t.setting = setting;
    }
    return t.plan;
}

extern "C" {

// ---- products -------------------------------------------------------------------

static bool i8_k(int64_t K) { return K > 0 && K % 128 == 0 && K < int64_t(1) << 17; }
static bool i8_shape(int64_t N, int64_t K, int64_t nmul) { return N > 0 && N % nmul == 0 && N <= MAX_DIM && i8_k(K); }

int r9k_quant_i8(const uint16_t *x, int64_t rows, int64_t K, int8_t *q, float *s, void *stream) {
    if (!x || !q || !s) return R9K_ERR_NULLPTR;
    if (rows < 0 || rows >= 128 * MAX_DIM || !i8_k(K)) return R9K_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return R9K_ERR_ALIGN;
    if (clash({{q, rows * K}, {s, 4 * rows}}, {{x, 2 * rows * K}})) return R9K_ERR_ARG;
    if (rows == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    return launch_result(launch_quant_i8(x, rows, K, q, s, (hipStream_t)stream));
}

int r9k_pack_weight_i8(const int8_t *wq, int64_t N, int64_t K, int8_t *wp, void *stream) {
    if (!wq || !wp) return R9K_ERR_NULLPTR;
    if (N <= 0 || N % 16 || !i8_k(K) || N >= (int64_t(1) << 36) / K) return R9K_ERR_SHAPE;
    if (!aligned16(wq) || !aligned16(wp)) return R9K_ERR_ALIGN;
    if (clash({{wp, N * K}}, {{wq, N * K}})) return R9K_ERR_ARG;
    if (int rc = check_device()) return rc;
    return launch_result(launch_pack_weight((const uint8_t *)wq, N, K, (uint8_t *)wp, (hipStream_t)stream));
}

// The workspace: the codes and scales of a call that quantises, then a split's sums
struct I8Layout {
    size_t scales, part, total;
};
static I8Layout i8_layout(int64_t M, int64_t K, int64_t N, const I8Plan &p, bool quant) {
    I8Layout l{};
    if (quant && !p.fused) {
        l.scales = align_up((size_t)(M * K), 256);
        l.part = l.scales + align_up((size_t)M * 4, 256);
    }
    l.total = l.part + (p.ksplit() > 1 ? align_up((size_t)p.ksplit() * (size_t)(M * N) * 4, 256) : 0);
    return l;
}
static hipError_t launch_i8(const I8Args &a, const I8Plan &p, hipStream_t s) {
    return p.tile ? launch_gemm_i8_tiled(a, p.tiled, s) : launch_gemm_i8(a, p.cfg, s);
}

static int i8_workspace(int64_t M, int64_t K, int64_t N, std::initializer_list<bool> forms, size_t *bytes) {
    if (!bytes) return R9K_ERR_NULLPTR;
    if (M < 0 || M > MAX_DIM || !i8_shape(N, K, 16)) return R9K_ERR_SHAPE;
    *bytes = 0;
    for (const bool quant : forms)
        if (M) *bytes = std::max(*bytes, i8_layout(M, K, N, i8_plan(M, K, N, 0, false, quant), quant).total);
    return R9K_OK;
}
int r9k_gemm_i8_workspace(int64_t M, int64_t K, int64_t N, size_t *bytes) {
    return i8_workspace(M, K, N, {false, true}, bytes);
}
int r9k_gemm_i8_codes_workspace(int64_t M, int64_t K, int64_t N, size_t *bytes) {
    return i8_workspace(M, K, N, {false}, bytes);
}

static int run_gemm_i8(const uint16_t *a, const int8_t *aq, const float *as, int64_t M, int64_t K, const int8_t *wp,
                       const float *ws, int64_t N, uint16_t *c, void *workspace, size_t ws_bytes, hipStream_t s) {
    if (!(a ? (const void *)a : (const void *)aq) || (!a && !as) || !wp || !ws || !c) return R9K_ERR_NULLPTR;
    if (M < 0 || M > MAX_DIM || !i8_shape(N, K, 16)) return R9K_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(aq) || !aligned16(as) || !aligned16(wp) || !aligned16(ws) || !aligned16(c) ||
        !aligned16(workspace))
        return R9K_ERR_ALIGN;
    if (M == 0) return R9K_OK;
    const I8Plan &plan = i8_plan(M, K, N, 0, false, a != nullptr);
    const I8Layout l = i8_layout(M, K, N, plan, a != nullptr);
    const bool quant = a && !plan.fused;
    if (l.total && !workspace) return R9K_ERR_NULLPTR;
    if (ws_bytes < l.total) return R9K_ERR_WORKSPACE;
    if (clash({{c, 2 * M * N}, {workspace, (int64_t)l.total}},
              {{a, 2 * M * K}, {aq, M * K}, {as, 4 * M}, {wp, N * K}, {ws, 4 * N}}))
        return R9K_ERR_ARG;
    if (int rc = check_device()) return rc;
    uint8_t *w = (uint8_t *)workspace;
    if (quant) {
        aq = (const int8_t *)w;
        as = (const float *)(w + l.scales);
        const hipError_t err = launch_quant_i8(a, M, K, (int8_t *)w, (float *)(w + l.scales), s);
        if (err != hipSuccess) return launch_result(err);
    }
    I8Args g{aq, as, wp, ws, c, M, K, N, nullptr, nullptr, 1, 1, M, 0, plan.ksplit() > 1 ? (int32_t *)(w + l.part) : nullptr,
             quant ? nullptr : a};
    return launch_result(launch_i8(g, plan, s));
}

int r9k_gemm_i8(const int8_t *aq, const float *as, int64_t M, int64_t K, const int8_t *wp, const float *ws, int64_t N,
                uint16_t *c, void *workspace, size_t ws_bytes, void *stream) {
    return run_gemm_i8(nullptr, aq, as, M, K, wp, ws, N, c, workspace, ws_bytes, (hipStream_t)stream);
}

int r9k_gemm_i8_qa(const uint16_t *a, int64_t M, int64_t K, const int8_t *wp, const float *ws, int64_t N, uint16_t *c,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (!a) return R9K_ERR_NULLPTR;
    return run_gemm_i8(a, nullptr, nullptr, M, K, wp, ws, N, c, workspace, ws_bytes, (hipStream_t)stream);
}

int r9k_moe_gemm_i8(const int8_t *aq, const float *as, int64_t arows, const int32_t *src, int64_t topk,
                    const int32_t *offsets, int64_t E, int64_t R, int64_t K, const int8_t *wp, const float *ws,
                    int64_t N, int act, uint16_t *c, void *stream) {
    if (!aq || !as || !offsets || !wp || !ws || !c) return R9K_ERR_NULLPTR;
    const bool silu = act == R9K_ACT_SILU_MUL;
    if (R < 0 || R >= 128 * MAX_DIM || E < 1 || E > MOE_MAX_E || arows < 0 || arows >= 128 * MAX_DIM ||
        !i8_shape(N, K, silu ? 32 : 16) || (R > 0 && arows < 1) || topk < 1 || topk > MAX_DIM ||
        R > arows * (src ? topk : 1))
        return R9K_ERR_SHAPE;
    if (act != R9K_ACT_NONE && !silu) return R9K_ERR_ARG;
    if (!aligned16(aq) || !aligned16(as) || !aligned16(src) || !aligned16(offsets) || !aligned16(wp) ||
        !aligned16(ws) || !aligned16(c))
        return R9K_ERR_ALIGN;
    if (clash({{c, (silu ? 1 : 2) * R * N}},
              {{aq, arows * K}, {as, 4 * arows}, {src, 4 * R}, {offsets, 4 * (E + 1)}, {wp, E * N * K}, {ws, 4 * E * N}}))
        return R9K_ERR_ARG;
    if (R == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    I8Args g{aq, as, wp, ws, c, R, K, N, offsets, src, E, topk, arows, silu ? 1 : 0, nullptr, nullptr};
    return launch_result(launch_i8(g, i8_plan(R, K, N, E, silu, false, src && arows * K >= int64_t(1) << 32), (hipStream_t)stream));
}

int r9k_i8_plan(int64_t M, int64_t K, int64_t N, int64_t E, int act, int quant, int *plan) {
    if (!plan) return R9K_ERR_NULLPTR;
    const bool silu = act == R9K_ACT_SILU_MUL;
    if (M < 0 || E < 0 || E > MOE_MAX_E || M > (E ? 128 * MAX_DIM - 1 : MAX_DIM) || !i8_shape(N, K, silu ? 32 : 16))
        return R9K_ERR_SHAPE;
    if ((act != R9K_ACT_NONE && !(silu && E)) || (quant != 0 && !(quant == 1 && E == 0))) return R9K_ERR_ARG;
    std::fill(plan, plan + R9K_I8_PLAN_INTS, 0);
    if (M == 0) return R9K_OK;
    const I8Plan &p = i8_plan(M, K, N, E, silu, quant != 0);
    const int *tile = I8_TILES[p.tiled.shape];
    const int tiled[] = {R9K_I8_TILED, tile[0], tile[1], 0, p.tiled.ksplit, 0, 0};
    const int stream[] = {R9K_I8_STREAM, p.cfg.nt, p.cfg.wn, p.cfg.wk, p.cfg.ksplit, p.cfg.mt, p.fused};
    std::copy_n(p.tile ? tiled : stream, R9K_I8_PLAN_INTS, plan);
    return R9K_OK;
}

int r9k_set_i8_plan(int kernel, int a, int b, int c, int ksplit, int rows) {
    if (ksplit < 0) return R9K_ERR_ARG;
    const bool shape = a || b || c || rows;
    if (kernel == R9K_I8_STREAM) {
        bool known = !shape && ksplit == 0;
        for (const auto &t : I8_STREAMS) known |= t[0] == rows && t[1] == a && t[2] == b && t[3] == c;
        if (!known) return R9K_ERR_ARG;
    } else if (kernel == R9K_I8_TILED) {
        bool known = !shape;
        for (const auto &t : I8_TILES) known |= t[0] == a && t[1] == b && !c && !rows;
        if (!known) return R9K_ERR_ARG;
    } else if (kernel != R9K_I8_AUTO || shape || ksplit) {
        return R9K_ERR_ARG;
    }
    i8_tuning() = I8Tuning{kernel, a, b, c, rows, ksplit};
    ++g_i8_setting;
    return R9K_OK;
}

// ---- the router ------------------------------------------------------------------

static int check_router_shape(int64_t T, int64_t E, int64_t topk, int64_t most) {
    return T < 0 || T >= MAX_BLOCKS || E < 1 || E > most || topk < 1 || topk > 64 ? R9K_ERR_SHAPE : R9K_OK;
}
int r9k_moe_balance_loss_workspace(int64_t T, int64_t E, int64_t topk, size_t *bytes) {
    if (!bytes) return R9K_ERR_NULLPTR;
    if (int rc = check_router_shape(T, E, topk, MOE_MAX_E)) return rc;
    *bytes = balance_workspace(T, E);
    return R9K_OK;
}

int r9k_moe_balance_loss(const void *logits, int dtype, int64_t T, int64_t E, const int32_t *topk_ids, int64_t topk,
                         const uint8_t *mask, float *loss, int32_t *counts, float *psum, void *workspace,
                         size_t ws_bytes, void *stream) {
    if (!logits || !topk_ids || !loss || !counts || !psum) return R9K_ERR_NULLPTR;
    if (int rc = check_router_shape(T, E, topk, MOE_MAX_E)) return rc;
    if (dtype != R9K_BF16 && dtype != R9K_F32) return R9K_ERR_ARG;
    if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(mask) || !aligned16(loss) || !aligned16(counts) ||
        !aligned16(psum) || !aligned16(workspace))
        return R9K_ERR_ALIGN;
    const size_t need = balance_workspace(T, E);
    if (need && !workspace) return R9K_ERR_NULLPTR;
    if (ws_bytes < need) return R9K_ERR_WORKSPACE;
    if (clash({{loss, 4}, {counts, 4 * (E + 1)}, {psum, 4 * E}, {workspace, (int64_t)need}},
              {{logits, T * E * (dtype == R9K_F32 ? 4 : 2)}, {topk_ids, 4 * T * topk}, {mask, T}}))
        return R9K_ERR_ARG;
    if (int rc = check_device()) return rc;
    const BalanceArgs a{logits, dtype == R9K_F32, T, E, topk, topk_ids, mask, loss, counts, psum};
    return launch_result(launch_balance_loss(a, workspace, (hipStream_t)stream));
}

int r9k_moe_balance_loss_backward(const float *gloss, const void *logits, int dtype, int64_t T, int64_t E, int64_t topk,
                                  const int32_t *counts, const uint8_t *mask, const float *gw, const int32_t *topk_ids,
                                  const float *topk_w, void *glogits, void *stream) {
    if (!gloss || !logits || !counts || !glogits || (gw == nullptr) != (topk_ids == nullptr) ||
        (gw == nullptr) != (topk_w == nullptr))
        return R9K_ERR_NULLPTR;
    if (int rc = check_router_shape(T, E, topk, MOE_MAX_E)) return rc;
    if (dtype != R9K_BF16 && dtype != R9K_F32) return R9K_ERR_ARG;
    if (!aligned16(gloss) || !aligned16(logits) || !aligned16(counts) || !aligned16(mask) || !aligned16(gw) ||
        !aligned16(topk_ids) || !aligned16(topk_w) || !aligned16(glogits))
        return R9K_ERR_ALIGN;
    const int64_t rows = T * E * (dtype == R9K_F32 ? 4 : 2), slots = 4 * T * topk;
    if (clash({{glogits, rows}}, {{gloss, 4}, {logits, rows}, {counts, 4 * (E + 1)}, {mask, T}, {gw, slots},
                                  {topk_ids, slots}, {topk_w, slots}}))
        return R9K_ERR_ARG;
    if (T == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    const RouterGradArgs a{gw, topk_ids, topk_w, T, E, topk, gloss, logits, dtype == R9K_F32, counts, mask, glogits};
    return launch_result(launch_router_backward(a, (hipStream_t)stream));
}

int r9k_moe_route_backward(const float *gw, const int32_t *topk_ids, const float *topk_w, int64_t T, int64_t E,
                           int64_t topk, float *glogits, void *stream) {
    if (!gw || !topk_ids || !topk_w || !glogits) return R9K_ERR_NULLPTR;
    if (int rc = check_router_shape(T, E, topk, 65536)) return rc;
    if (!aligned16(gw) || !aligned16(topk_ids) || !aligned16(topk_w) || !aligned16(glogits)) return R9K_ERR_ALIGN;
    const int64_t slots = 4 * T * topk;
    if (clash({{glogits, 4 * T * E}}, {{gw, slots}, {topk_ids, slots}, {topk_w, slots}})) return R9K_ERR_ARG;
    if (T == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    const RouterGradArgs a{gw, topk_ids, topk_w, T, E, topk, nullptr, nullptr, true, nullptr, nullptr, glogits};
    return launch_result(launch_router_backward(a, (hipStream_t)stream));
}

}  // extern "C"

// The C ABI of the 4-bit weights and of the rows sorted by expert: argument checks,
// plans and launches.  Declarations, argument meanings and error behaviour: r9k.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "r9k.h"
#include "w4_internal.h"

using namespace r9k;

namespace r9k {
W4Tuning &w4_tuning() {
    static W4Tuning t{{0, 0, 0, 0}, {-1, 0, 0}};
    static std::once_flag once;
    std::call_once(once, [] {
        if (const char *e = getenv("R9K_W4")) sscanf(e, "%d,%d,%d,%d", &t.stream[0], &t.stream[1], &t.stream[2], &t.stream[3]);
        if (const char *e = getenv("R9K_W4_TILED"))
            if (sscanf(e, "%d,%d,%d", &t.tiled[0], &t.tiled[1], &t.tiled[2]) < 1) t.tiled[0] = -1;
    });
    return t;
}
}  // namespace r9k

namespace {

// Device check, cached per device id: 1 = gfx950, 2 = not usable.
constexpr int MAX_DEV = 64;
std::atomic<int> g_dev_ok[MAX_DEV];

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return R9K_ERR_DEVICE;
    }
    const int st = dev < MAX_DEV ? g_dev_ok[dev].load() : 0;
    if (st) return st == 1 ? R9K_OK : R9K_ERR_DEVICE;
    hipDeviceProp_t prop;
    const bool ok = hipGetDeviceProperties(&prop, dev) == hipSuccess && strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    (void)hipGetLastError();
    if (dev < MAX_DEV) g_dev_ok[dev] = ok ? 1 : 2;
    return ok ? R9K_OK : R9K_ERR_DEVICE;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline int launch_result(hipError_t e) { return e == hipSuccess ? R9K_OK : R9K_ERR_LAUNCH; }

constexpr int64_t MAX_DIM = int64_t(1) << 24;

// Blocks of 256 threads in a launch: the runtime refuses 2^32 threads and more
constexpr int64_t MAX_BLOCKS = int64_t(1) << 24;

// Experts that the sort and the expert products take: the sort keeps four counters an
// expert in a CTA's LDS
constexpr int64_t MOE_MAX_E = 2048;

}  // namespace

extern "C" {

// ---- 4-bit weights ------------------------------------------------------------

static bool w4_known(int format, int group, bool zeros) {
    if (format == R9K_W4_INT) return group == 32 || group == 64 || group == 128;
    return format == R9K_W4_MXFP4 && group == 32 && !zeros;
}

static bool w4_shape(int64_t N, int64_t K, int64_t nmul) {
    return N > 0 && K > 0 && N % nmul == 0 && K % 128 == 0 && N <= 128 * MAX_DIM && K <= MAX_DIM &&
           N <= (int64_t(1) << 46) / K;
}

// Bytes that a call reads or writes.  Its CTAs read while others write, so an output
// (a workspace too) may lie on no input and on no other output.
struct Span {
    const void *p;
    int64_t n;
};
static bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.n > 0 && b.n > 0 && x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n;
}
static bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(*o, i)) return true;
        for (auto q = outs.begin(); q != o; ++q)
            if (overlap(*o, *q)) return true;
    }
    return false;
}
static int64_t w4_scale_bytes(int64_t N, int64_t K, int format, int group) {
    return N * (K / group) * (format == R9K_W4_INT ? 2 : 1);
}

int r9k_quant_weight_w4(const uint16_t *w, int64_t N, int64_t K, int format, int group, uint8_t *wq, void *s,
                        uint8_t *z, void *stream) {
    if (!w || !wq || !s) return R9K_ERR_NULLPTR;
    if (!w4_shape(N, K, 16) || N * K / 8 / 256 >= MAX_BLOCKS) return R9K_ERR_SHAPE;
    if (!w4_known(format, group, z != nullptr)) return R9K_ERR_ARG;
    if (!aligned16(w) || !aligned16(wq) || !aligned16(s) || !aligned16(z)) return R9K_ERR_ALIGN;
    if (clash({{wq, N * K / 2}, {s, w4_scale_bytes(N, K, format, group)}, {z, N * (K / group)}}, {{w, 2 * N * K}}))
        return R9K_ERR_ARG;
    if (int rc = check_device()) return rc;
    return launch_result(launch_quant_weight_w4(w, N, K, format, group, wq, s, z, (hipStream_t)stream));
}

int r9k_pack_weight_w4(const uint8_t *wq, const void *s, const uint8_t *z, int64_t N, int64_t K, int format,
                       int group, uint8_t *wp, void *sp, uint8_t *zp, void *stream) {
    if (!wq || !s || !wp || !sp) return R9K_ERR_NULLPTR;
    if (!w4_shape(N, K, 16) || N / 16 * (K / 128) / 4 >= MAX_BLOCKS) return R9K_ERR_SHAPE;
    if (!w4_known(format, group, z != nullptr) || (z == nullptr) != (zp == nullptr)) return R9K_ERR_ARG;
    if (!aligned16(wq) || !aligned16(s) || !aligned16(z) || !aligned16(wp) || !aligned16(sp) || !aligned16(zp))
        return R9K_ERR_ALIGN;
    const int64_t cb = N * K / 2, sb = w4_scale_bytes(N, K, format, group), zb = N * (K / group);
    if (clash({{wp, cb}, {sp, sb}, {zp, zb}}, {{wq, cb}, {s, sb}, {z, zb}})) return R9K_ERR_ARG;  // in place too
    if (int rc = check_device()) return rc;
    return launch_result(launch_pack_weight_w4(wq, s, z, N, K, format, group, wp, sp, zp, (hipStream_t)stream));
}

// A 4-bit product's kernel, and its workspace: the partial sums of a K split, which
// only dense products take.
struct W4Plan {
    W4TiledCfg tiled;
    W4Cfg cfg;
    bool tile[2];  // the tiled kernel takes it; [1]: int4 in groups of 32
    size_t bytes;  // of either choice, since the workspace query does not know the format
};
static W4Plan w4_plan_new(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    W4Plan w{w4_tiled_config(M, K, N, E, silu), w4_config(M, K, N, E, silu), {}, 0};
    for (int fine = 0; fine < 2; ++fine) {
        // The kernel of the least estimated time (measured around it: gemm_w4_tiled.hip).  A dense
        // product's row blocks share the weight in the caches, 8% less for the streaming kernel than
        // estimated; groups of 32 cost it 10% more than the tiled kernel (100 rows of 4096 x 4096:
        // 21.6 against 20.1 us, in groups of 128 16.9 against 18.3).  Its grid holds 65535 row
        // blocks; 2^19 rows of 2048 experts stay below.
        const double stream = w.cfg.us * (E ? 1.0 : 0.92) * (fine ? 1.1 : 1.0);
        bool &tile = w.tile[fine];
        tile = w.tiled.on;
        if (tile && w4_tuning().tiled[0] < 0) tile = w.tiled.us < stream || M >= 1 << 19;
        const int split = tile ? w.tiled.ksplit : w.cfg.ksplit;
        if (split > 1) w.bytes = std::max(w.bytes, align_up((size_t)split * (size_t)(M * N) * sizeof(float), 256));
    }
    return w;
}

static std::atomic<int> g_plan_setting{0};  // counts the changes of the plan control

// The plan of a shape under the present setting, kept for each thread's last shapes:
// planning takes about a microsecond, a third of a launch.
static const W4Plan &w4_plan(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    struct Entry {
        int64_t M = -1, K, N, E;
        int setting;
        bool silu;
        W4Plan plan;
    };
    static thread_local Entry table[64];
    const uint64_t h = ((uint64_t)M * 0x9E3779B97F4A7C15u) ^ ((uint64_t)K * 0xC2B2AE3D27D4EB4Fu) ^
                       ((uint64_t)N * 0x165667B19E3779F9u) ^ ((uint64_t)(2 * E + silu) * 0x27D4EB2F165667C5u);
    Entry &t = table[h >> 58];
    const int setting = g_plan_setting.load(std::memory_order_relaxed);
    if (t.M != M || t.K != K || t.N != N || t.E != E || t.silu != silu || t.setting != setting) {
        t.plan = w4_plan_new(M, K, N, E, silu);
        t.M = M, t.K = K, t.N = N, t.E = E, t.silu = silu, t.setting = setting;
    }
    return t.plan;
}

static bool w4_takes_tile(const W4Plan &w, int format, int group) {
    return w.tile[format == R9K_W4_INT && group == 32];
}

static int run_w4(W4Args &a, int format, int group, void *workspace, size_t ws_bytes, hipStream_t s) {
    const W4Plan &w = w4_plan(a.M, a.K, a.N, a.offsets ? a.E : 0, a.silu != 0);
    if (w.bytes && !workspace) return R9K_ERR_NULLPTR;
    if (ws_bytes < w.bytes) return R9K_ERR_WORKSPACE;
    // (what a dense product reads: a split, which alone takes a workspace, is none of the experts')
    if (w.bytes && clash({{workspace, (int64_t)w.bytes}},
                         {{a.a, 2 * a.M * a.K}, {a.wp, a.N * a.K / 2}, {a.sp, w4_scale_bytes(a.N, a.K, format, group)},
                          {a.zp, a.N * (a.K / group)}, {a.c, 2 * a.M * a.N}}))
        return R9K_ERR_ARG;
    if (int rc = check_device()) return rc;
    a.part = (float *)workspace;
    return launch_result(w4_takes_tile(w, format, group) ? launch_gemm_w4_tiled(a, format, group, w.tiled, s)
                                                         : launch_gemm_w4(a, format, group, w.cfg, s));
}

int r9k_gemm_w4_workspace(int64_t M, int64_t K, int64_t N, size_t *bytes) {
    if (!bytes) return R9K_ERR_NULLPTR;
    if (M < 0 || M > MAX_DIM || !w4_shape(N, K, 16) || N > MAX_DIM) return R9K_ERR_SHAPE;
    *bytes = M ? w4_plan(M, K, N, 0, false).bytes : 0;
    return R9K_OK;
}

int r9k_gemm_w4(const uint16_t *a, int64_t M, int64_t K, const uint8_t *wp, const void *sp, const uint8_t *zp,
                int format, int group, int64_t N, uint16_t *c, void *workspace, size_t ws_bytes, void *stream) {
    if (!a || !wp || !sp || !c) return R9K_ERR_NULLPTR;
    if (M < 0 || M > MAX_DIM || !w4_shape(N, K, 16) || N > MAX_DIM) return R9K_ERR_SHAPE;
    if (!w4_known(format, group, zp != nullptr)) return R9K_ERR_ARG;
    if (!aligned16(a) || !aligned16(wp) || !aligned16(sp) || !aligned16(zp) || !aligned16(c) || !aligned16(workspace))
        return R9K_ERR_ALIGN;
    if (clash({{c, 2 * M * N}}, {{a, 2 * M * K}, {wp, N * K / 2}, {sp, w4_scale_bytes(N, K, format, group)},
                                 {zp, N * (K / group)}}))
        return R9K_ERR_ARG;
    if (M == 0) return R9K_OK;
    W4Args w{a, wp, sp, zp, c, M, K, N, nullptr, nullptr, 1, 1, M, 0, nullptr};
    return run_w4(w, format, group, workspace, ws_bytes, (hipStream_t)stream);
}

static bool w4_moe_shape(int64_t arows, int64_t E, int64_t R, int64_t K, int64_t N, bool silu) {
    return R >= 0 && R < 128 * MAX_DIM && E >= 1 && E <= MOE_MAX_E && arows >= 0 && arows < 128 * MAX_DIM &&
           w4_shape(N, K, silu ? 32 : 16) && N <= MAX_DIM && (R == 0 || arows >= 1);
}

int r9k_moe_gemm_w4(const uint16_t *a, int64_t arows, const int32_t *src, int64_t topk, const int32_t *offsets,
                    int64_t E, int64_t R, int64_t K, const uint8_t *wp, const void *sp, const uint8_t *zp,
                    int format, int group, int64_t N, int act, uint16_t *c, void *stream) {
    if (!a || !offsets || !wp || !sp || !c) return R9K_ERR_NULLPTR;
    const bool silu = act == R9K_ACT_SILU_MUL;
    if (!w4_moe_shape(arows, E, R, K, N, silu) || topk < 1 || topk > MAX_DIM || R > arows * (src ? topk : 1))
        return R9K_ERR_SHAPE;  // more rows than there are slots (or, without an index, rows of a)
    if (!w4_known(format, group, zp != nullptr) || (act != R9K_ACT_NONE && !silu)) return R9K_ERR_ARG;
    if (!aligned16(a) || !aligned16(src) || !aligned16(offsets) || !aligned16(wp) || !aligned16(sp) ||
        !aligned16(zp) || !aligned16(c))
        return R9K_ERR_ALIGN;
    if (clash({{c, (silu ? 1 : 2) * R * N}},
              {{a, 2 * arows * K}, {src, 4 * R}, {offsets, 4 * (E + 1)}, {wp, E * N * K / 2},
               {sp, E * w4_scale_bytes(N, K, format, group)}, {zp, E * N * (K / group)}}))
        return R9K_ERR_ARG;
    if (R == 0) return R9K_OK;
    W4Args w{a, wp, sp, zp, c, R, K, N, offsets, src, E, topk, arows, silu ? 1 : 0, nullptr};
    return run_w4(w, format, group, nullptr, 0, (hipStream_t)stream);
}

int r9k_w4_plan(int64_t M, int64_t K, int64_t N, int64_t E, int act, int format, int group, int *plan) {
    if (!plan) return R9K_ERR_NULLPTR;
    const bool silu = act == R9K_ACT_SILU_MUL;
    if (E < 0 || (E ? !w4_moe_shape(M, E, M, K, N, silu) : M < 0 || M > MAX_DIM || !w4_shape(N, K, 16) || N > MAX_DIM))
        return R9K_ERR_SHAPE;
    if (!w4_known(format, group, false) || (act != R9K_ACT_NONE && !(silu && E))) return R9K_ERR_ARG;
    std::fill(plan, plan + R9K_W4_PLAN_INTS, 0);
    if (M == 0) return R9K_OK;
    const W4Plan &w = w4_plan(M, K, N, E, silu);
    const int tiled[] = {R9K_W4_TILED, w.tiled.tn, 4, 1, w.tiled.ksplit, 0};
    const int stream[] = {R9K_W4_STREAM, w.cfg.nt, w.cfg.wn, w.cfg.wk, w.cfg.ksplit, w4_segments(w.cfg, K, format, group)};
    std::copy_n(w4_takes_tile(w, format, group) ? tiled : stream, R9K_W4_PLAN_INTS, plan);
    return R9K_OK;
}

int r9k_set_w4_plan(int kernel, int tiles, int waves, int slices, int ksplit) {
    const bool shape = tiles || waves || slices;
    if (ksplit < 0) return R9K_ERR_ARG;
    W4Tuning t{{0, 0, 0, 0}, {-1, 0, 0}};
    if (kernel == R9K_W4_STREAM) {
        if (shape ? !w4_stream_shape(tiles, waves, slices) : ksplit != 0) return R9K_ERR_ARG;
        t = W4Tuning{{tiles, waves, slices, ksplit}, {0, 0, 0}};
    } else if (kernel == R9K_W4_TILED) {
        if (waves || slices || (tiles != 0 && tiles != 1 && tiles != 2 && tiles != 4)) return R9K_ERR_ARG;
        t = W4Tuning{{0, 0, 0, 0}, {1, tiles, ksplit}};
    } else if (kernel != R9K_W4_AUTO || shape || ksplit) {
        return R9K_ERR_ARG;
    }
    w4_tuning() = t;
    ++g_plan_setting;
    return R9K_OK;
}

// ---- rows sorted by expert -----------------------------------------------------

static int check_sort_shape(int64_t T, int64_t topk) {
    if (T < 0 || T >= MAX_BLOCKS || topk < 1 || topk > 64) return R9K_ERR_SHAPE;  // up to a block a token
    return R9K_OK;
}

// bytes of a row, or 0 if the rows' type or width is not one the library moves
static int64_t row_bytes(int dtype, int64_t H) {
    if (H <= 0 || H > MAX_DIM) return 0;
    const int64_t b = H * (dtype == R9K_F32 ? 4 : 2);
    return b % 16 ? 0 : b;
}

int r9k_moe_permute_workspace(int64_t T, int64_t E, int64_t topk, size_t *bytes) {
    if (!bytes) return R9K_ERR_NULLPTR;
    if (int rc = check_sort_shape(T, topk)) return rc;
    if (E < 1 || E > MOE_MAX_E) return R9K_ERR_SHAPE;
    *bytes = moe_sort_workspace(T * topk, E);
    return R9K_OK;
}

int r9k_moe_permute(const void *x, int dtype, int64_t T, int64_t H, const int32_t *topk_ids, int64_t topk, int64_t E,
                    void *xs, int32_t *src, int32_t *pos, int32_t *offsets, void *workspace, size_t ws_bytes,
                    void *stream) {
    if (!topk_ids || !src || !pos || !offsets || (x == nullptr) != (xs == nullptr)) return R9K_ERR_NULLPTR;
    if (int rc = check_sort_shape(T, topk)) return rc;
    if (E < 1 || E > MOE_MAX_E) return R9K_ERR_SHAPE;
    int64_t rb = 0;
    if (x) {
        if (dtype != R9K_BF16 && dtype != R9K_F32) return R9K_ERR_ARG;
        rb = row_bytes(dtype, H);
        if (!rb) return R9K_ERR_SHAPE;
    }
    if (!aligned16(x) || !aligned16(xs) || !aligned16(topk_ids) || !aligned16(src) || !aligned16(pos) ||
        !aligned16(offsets) || !aligned16(workspace))
        return R9K_ERR_ALIGN;
    const size_t need = moe_sort_workspace(T * topk, E);
    const int64_t slots = 4 * T * topk;  // bytes of an index
    if (clash({{xs, T * topk * rb}, {src, slots}, {pos, slots}, {offsets, 4 * (E + 1)}, {workspace, (int64_t)need}},
              {{x, T * rb}, {topk_ids, slots}}))
        return R9K_ERR_ARG;
    if (need && !workspace) return R9K_ERR_NULLPTR;
    if (ws_bytes < need) return R9K_ERR_WORKSPACE;
    if (int rc = check_device()) return rc;
    const SortArgs a{topk_ids, x, xs, src, pos, offsets, (int32_t *)workspace, T, topk, E, rb};
    return launch_result(launch_moe_permute(a, (hipStream_t)stream));
}

static int run_unpermute(const void *y, int dtype, int64_t T, int64_t H, const int32_t *pos, const float *w,
                         int64_t topk, void *out, void *stream) {
    if (!y || !pos || !out) return R9K_ERR_NULLPTR;
    if (int rc = check_sort_shape(T, topk)) return rc;
    if (dtype != R9K_BF16 && dtype != R9K_F32) return R9K_ERR_ARG;
    const int64_t rb = row_bytes(dtype, H);
    if (!rb) return R9K_ERR_SHAPE;
    if (!aligned16(y) || !aligned16(pos) || !aligned16(w) || !aligned16(out)) return R9K_ERR_ALIGN;
    if (clash({{out, T * rb}}, {{y, T * topk * rb}, {pos, 4 * T * topk}, {w, 4 * T * topk}})) return R9K_ERR_ARG;
    if (T == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    return launch_result(
        launch_moe_unpermute(y, dtype == R9K_F32, rb, T, topk, pos, w, out, (hipStream_t)stream));
}

int r9k_moe_unpermute(const void *y, int dtype, int64_t T, int64_t H, const int32_t *pos, const float *w,
                      int64_t topk, void *out, void *stream) {
    return run_unpermute(y, dtype, T, H, pos, w, topk, out, stream);
}

int r9k_moe_permute_backward(const void *gxs, int dtype, int64_t T, int64_t H, const int32_t *pos, int64_t topk,
                             void *gx, void *stream) {
    return run_unpermute(gxs, dtype, T, H, pos, nullptr, topk, gx, stream);
}

int r9k_moe_unpermute_backward(const void *gout, const void *y, int dtype, int64_t T, int64_t H, const int32_t *pos,
                               const float *w, int64_t topk, void *gy, float *gw, void *stream) {
    if (!gout || !y || !pos || !w || !gy || !gw) return R9K_ERR_NULLPTR;
    if (int rc = check_sort_shape(T, topk)) return rc;
    if (dtype != R9K_BF16 && dtype != R9K_F32) return R9K_ERR_ARG;
    const int64_t rb = row_bytes(dtype, H);
    if (!rb) return R9K_ERR_SHAPE;
    if (!aligned16(gout) || !aligned16(y) || !aligned16(pos) || !aligned16(w) || !aligned16(gy) || !aligned16(gw))
        return R9K_ERR_ALIGN;
    const int64_t slots = 4 * T * topk;  // bytes of pos, w and gw
    if (clash({{gy, T * topk * rb}, {gw, slots}}, {{gout, T * rb}, {y, T * topk * rb}, {pos, slots}, {w, slots}}))
        return R9K_ERR_ARG;
    if (T == 0) return R9K_OK;
    if (int rc = check_device()) return rc;
    return launch_result(launch_moe_unpermute_backward(gout, y, dtype == R9K_F32, rb, T, topk, pos, w, gy, gw,
                                                       (hipStream_t)stream));
}

}  // extern "C"

// C-ABI of the 8-bit matrices: argument checks, the workspaces' layouts and the
// order of the launches.  Nothing here allocates device memory or waits: the
// caller gives the workspace, so calls can be captured into a graph, and two
// graphs (or streams) with a workspace each never meet.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <string>

#include "../../include/mkp.h"
#include "internal.h"
#include "kernels.h"
#include "q8.h"

namespace mkp {

const char* q8_launch_name(int i) {
    static const char* const names[QL_COUNT] = {"q8_quantize", "q8_dequantize", "q8_pack",    "i8_product",
                                                "i8_finish",   "q8_slopes",     "q8_product", "q8_finish"};
    return i >= 0 && i < QL_COUNT ? names[i] : "q8";
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool real_type(int t) { return t == MKP_BF16 || t == MKP_F32; }
double size_of(int t) { return t == MKP_F32 ? 4.0 : t == MKP_I8 ? 1.0 : 2.0; }

constexpr int64_t kMaxRows = (int64_t(1) << 24) - 1;   // at least 256 threads a row, counted in 32 bits
constexpr int64_t kMaxCols = int64_t(1) << 22;         // and leading dimensions: a tile's rows stay within 32-bit offsets
constexpr int64_t kMaxDepth = 131071;                  // 128^2 times this is below 2^31

int check_extents(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return report(MKP_ERR_INVALID_ARG, "negative dimension");
    if (M > kMaxRows || N > kMaxCols || K > kMaxCols)
        return report(MKP_ERR_UNSUPPORTED, "more than 2^24 - 1 rows or 2^22 columns");
    return MKP_OK;
}
int check_ld(int64_t ld, int64_t cols, const char* name) {
    if (ld < cols) return report(MKP_ERR_INVALID_ARG, std::string(name) + " is less than a row");
    if (ld > 4 * kMaxCols) return report(MKP_ERR_UNSUPPORTED, std::string(name) + " exceeds 2^24");
    return MKP_OK;
}
int check_group(int64_t group) {
    if (group == 0 || group == 32 || group == 64 || group == 128 || group == kQ8MaxGroup) return MKP_OK;
    return report(MKP_ERR_INVALID_ARG, "group must be 0, 32, 64, 128 or 256");
}
int64_t groups_of(int64_t K, int64_t group) { return group == 0 ? 1 : ceil_div(K, group); }

#define MKP_TRY(call)               \
    do {                            \
        const int rc_ = (call);     \
        if (rc_ != MKP_OK) return rc_; \
    } while (0)

int go(hipStream_t st, int what, double flops, double bytes, const std::function<hipError_t()>& fn) {
    const hipError_t e = traced_launch(st, kTraceQ8 - what, flops, bytes, fn);
    if (e == hipSuccess) return MKP_OK;
    return report(MKP_ERR_HIP, std::string(q8_launch_name(what)) + " launch: " + hipGetErrorString(e));
}

int check_workspace(const void* ws, int64_t have, size_t need) {
    if (need == 0 || (ws && have >= 0 && (size_t)have >= need && aligned16(ws))) return MKP_OK;
    return report(MKP_ERR_INVALID_ARG, "workspace of " + std::to_string(need) + " bytes, 16-byte aligned, needed");
}

// ---- quantisation ----------------------------------------------------------

int convert(bool back, int64_t M, int64_t K, void* X, int64_t ldx, int type, int64_t group, int8_t* Q, int64_t ldq, float* S,
            int64_t lds, void* stream) {
    MKP_TRY(check_extents(M, 0, K));
    MKP_TRY(check_group(group));
    if (!real_type(type)) return report(MKP_ERR_INVALID_ARG, "type must be MKP_BF16 or MKP_F32");
    MKP_TRY(check_ld(ldx, K, "ldx"));
    MKP_TRY(check_ld(ldq, K, "ldq"));
    MKP_TRY(check_ld(lds, groups_of(K, group), "lds"));
    if (M == 0 || K == 0) return MKP_OK;
    if (!X || !Q || !S) return report(MKP_ERR_INVALID_ARG, "X, Q or S is NULL");
    begin_call();
    const QuantArgs a{M, (int)K, X, ldx, type == MKP_F32, (int)group, Q, ldq, S, lds, 0};
    const double m = (double)M, k = (double)K;
    const double bytes = (size_of(type) + 1.0) * m * k + 4.0 * m * (double)groups_of(K, group);
    const hipStream_t st = (hipStream_t)stream;
    return back ? go(st, QL_DEQUANTIZE, m * k, bytes, [&] { return launch_dequantize(a, st); })
                : go(st, QL_QUANTIZE, 3.0 * m * k, bytes, [&] { return launch_quantize(a, st); });
}

// ---- linear layer ------------------------------------------------------------

struct LinearLayout {
    int tile = 256, splits = 1;
    bool stream = false, quantise = false, pack_a = false, pack_b = false;
    int64_t Ka = 0, Kb = 0, ldp = 0;   // bytes of a packed row, a row of partial sums
    size_t a = 0, s = 0, b = 0, part = 0, bytes = 0;
};

// What a product takes, in us, on tiles of one size: a launch's start, a
// workgroup's ends, and one of its steps (128 bytes of an operand's row) where n
// workgroups share a CU: n `step`, at least `alone`; `fit` of them do.  The busiest
// CU counts.  (The constants are those whose choices lose least, not each one a time
// of its own.)
struct TileCost {
    int tile;
    double start, end, step, alone;
    int64_t fit;
};

// The tile, and the parts of the sum, that cost least; `joined` is what several
// parts cost on top.
template <size_t n, class F>
void choose_tile(const TileCost (&tiles)[n], int64_t rows, int64_t cols, int64_t depth, int& tile, int& splits, F&& joined) {
    const uint32_t steps = (uint32_t)std::max<int64_t>(depth, 1);
    double best = INFINITY;
    for (const TileCost& t : tiles) {
        const int64_t count = ceil_div(rows, t.tile) * ceil_div(cols, t.tile);
        if (t.tile < 256 && count > (int64_t(1) << 22)) break;   // (launch limits)
        for (const uint32_t want : {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16, 20, 24, 28, 32}) {
            if (want > steps || (want > 1 && count * want > 8 * 256)) break;
            const uint32_t per = (steps + want - 1) / want, s = (steps + per - 1) / per;
            const int64_t busiest = (count * s + 255) >> 8, full = busiest / t.fit, rest = busiest - full * t.fit;
            const double step = (double)full * std::max(t.alone, (double)t.fit * t.step) +
                                (rest > 0 ? std::max(t.alone, (double)rest * t.step) : 0.0);
            const double us = t.start + (double)per * step + t.end * (double)(full + (rest > 0)) + (s > 1 ? joined((double)s) : 0.0);
            if (us < best) {
                best = us;
                tile = t.tile;
                splits = (int)s;
            }
        }
    }
}

// linear_i8's.  Fitted to measurements of 200 extents (33 to 8192 x 128 to 12544 x 128
// to 12544): the choice is 0.6 % behind the fastest in the mean, 14 % at most (of 200
// others 1.2 % and 23 %).  One tile for all: 256 loses 7.5 us to 64's 4.1 at 109 x 887 x
// 144, 64 loses 563 to 256's 300 at 8192 x 11008 x 4096.  No splits: 105 x 1024 x 12544
// takes 36 us on the 64 tile, in eight parts 8.3 + 4.0.  (Parts are written and read, and
// joined by a launch that costs the caller 3 us.)
constexpr TileCost kI8Tiles[] = {
    {256, 0.1, 7.4, 1.2, 1.2, 1}, {128, 2.3, 4.0, 0.5, 0.5, 2}, {64, 1.9, 1.5, 0.28, 0.29, 4}};
double i8_joined(double mn, double splits) {
    return 0.8e-6 * mn * splits + 3.0 + std::max(4.0, 2.1 + 1e-6 * mn * (0.71 + 0.59 * splits));
}

// linear_q8_backward's dW.  Fitted to measurements of 100 extents (32 to 8192 x 128 to
// 12544 x 128 to 12544): 0.7 % behind the fastest in the mean, 15 % at most (of 100
// others 0 % and 12 %).  One tile for all: 256 loses 14.3 us to 128's 7.4 at 333 x 768 x
// 768, 128 loses 869 to 583 at 8192 x 11008 x 4096.  No splits: 8192 x 768 x 768 takes 71
// us on the 128 tile, in six parts 17.4 + 4.0.
constexpr TileCost kGradTiles[] = {{256, 0.9, 11.0, 0.65, 0.65, 1}, {128, 2.6, 4.9, 0.335, 0.43, 2}};
double grad_joined(double nk, double splits) {
    return 0.8e-6 * nk * splits + std::max(4.1, 1e-6 * nk * (0.28 + 0.67 * splits));
}

// choose() fills in tile and splits; a thread keeps its last choices by extents (the
// call and its workspace's size ask for the same one, a model's layers for a few).
template <int which, class F>
void remembered(int64_t M, int64_t N, int64_t K, int& tile, int& splits, F&& choose) {
    struct Entry {
        int64_t M, N, K;
        int tile, splits;
    };
    thread_local Entry table[64] = {};   // (tile 0: empty)
    Entry& e = table[((uint64_t)M * 0x9E3779B97F4A7C15u ^ (uint64_t)N * 0xC2B2AE3D27D4EB4Fu ^ (uint64_t)K * 0x165667B19E3779F9u) >> 58];
    if (e.tile == 0 || e.M != M || e.N != N || e.K != K) {
        choose();
        e = Entry{M, N, K, tile, splits};
        return;
    }
    tile = e.tile;
    splits = e.splits;
}

LinearLayout linear_layout(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, int x_type, const void* W,
                           int64_t ldw) {
    LinearLayout l;
    l.pack_b = !aligned16(W) || ldw % 16 != 0;
    // Every workgroup of the product for few tokens reads the whole of X, which takes
    // it 3 us per 100 KB: past 128 KB tiles, with parts of K, are faster (us a call, X in
    // 8 bits, few tokens / tiles: 32 x 1024 x 4096 7.2 / 7.9, x 12544 16.2 / 9.3; 8 x 1024 x
    // 12544 8.6 / 8.6, x 32768 17.8 / 12.3; of 880 extents to 32 x 8192 x 32768 the choice is
    // 1 % behind the faster in the mean) unless all of W were to be copied for them.
    l.stream = M <= kI8StreamRows && (M * K <= kI8StreamInput || l.pack_b);
    if (l.stream) {
        l.pack_b = false;   // (rows of any alignment; few enough features are quantised by the product)
        l.quantise = x_type != MKP_I8 && M * ceil_div(K, 512) > kI8StreamUnits;
        l.Ka = round_up(K, 16);
        if (l.quantise) {
            l.s = (size_t)round_up(M * l.Ka, 256);
            l.bytes = l.s + (size_t)(4 * M);
        }
        return l;
    }
    l.quantise = x_type != MKP_I8;
    l.pack_a = !l.quantise && (!aligned16(X) || ldx % 16 != 0 || K % 16 != 0);
    l.Ka = round_up(K, 16);
    l.Kb = round_up(K, 16);
    remembered<0>(M, N, K, l.tile, l.splits, [&] {
        choose_tile(kI8Tiles, M, N, ceil_div(K, 128), l.tile, l.splits, [&](double s) { return i8_joined((double)(M * N), s); });
    });
    l.ldp = round_up(N, 4);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (size_t)round_up(bytes, 256);
        return here;
    };
    if (l.quantise || l.pack_a) l.a = take(M * l.Ka);
    if (l.quantise) l.s = take(4 * M);
    if (l.pack_b) l.b = take(N * l.Kb);
    if (l.splits > 1) l.part = take(4 * M * l.ldp * l.splits);
    l.bytes = at;
    return l;
}

int check_linear(int64_t M, int64_t N, int64_t K, int64_t ldx, int x_type, int64_t ldw) {
    MKP_TRY(check_extents(M, N, K));
    if (K > kMaxDepth) return report(MKP_ERR_UNSUPPORTED, "K exceeds 131071: a sum need not fit 32 bits");
    if (x_type != MKP_I8 && !real_type(x_type)) return report(MKP_ERR_INVALID_ARG, "x_type must be MKP_BF16, MKP_F32 or MKP_I8");
    MKP_TRY(check_ld(ldx, K, "ldx"));
    MKP_TRY(check_ld(ldw, K, "ldw"));
    return MKP_OK;
}

int linear(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, int x_type, const float* x_scale, const int8_t* W,
           int64_t ldw, const float* w_scale, const float* bias, int act, void* Y, int64_t ldy, int y_type, void* workspace,
           int64_t workspace_bytes, void* stream) {
    MKP_TRY(check_linear(M, N, K, ldx, x_type, ldw));
    MKP_TRY(check_ld(ldy, N, "ldy"));
    if (!real_type(y_type)) return report(MKP_ERR_INVALID_ARG, "y_type must be MKP_BF16 or MKP_F32");
    if (act < 0 || act >= ACT_COUNT) return report(MKP_ERR_INVALID_ARG, "unknown activation");
    if (M == 0 || N == 0) return MKP_OK;
    if (!Y || !w_scale || (x_type == MKP_I8 && !x_scale)) return report(MKP_ERR_INVALID_ARG, "Y, w_scale or x_scale is NULL");
    if (K > 0 && (!X || !W)) return report(MKP_ERR_INVALID_ARG, "X or W is NULL");
    const LinearLayout l = linear_layout(M, N, K, X, ldx, x_type, W, ldw);
    MKP_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    const int64_t tiles = l.stream ? 0 : ceil_div(M, l.tile) * ceil_div(N, l.tile) * l.splits;
    if (tiles > UINT32_MAX / 512 || (l.splits > 1 && M * ceil_div(N, 4) > (int64_t)UINT32_MAX - 255))
        return report(MKP_ERR_UNSUPPORTED, "grid too large");
    begin_call();
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const double m = (double)M, n = (double)N, k = (double)K;
    I8Args a{};
    a.M = M;
    a.N = (int)N;
    a.K = (int)K;
    a.A = (const int8_t*)X;
    a.lda = ldx;
    a.sa = x_scale;
    a.B = W;
    a.ldb = ldw;
    a.sb = w_scale;
    a.bias = bias;
    a.act = act;
    a.C = Y;
    a.ldc = ldy;
    a.bf16 = y_type == MKP_BF16;
    a.tile = l.tile;
    a.splits = l.splits;
    a.part = (int*)(ws + l.part);
    a.ldp = l.ldp;
    if (l.quantise) {
        const QuantArgs q{M, (int)K, (void*)X, ldx, x_type == MKP_F32, 0, (int8_t*)(ws + l.a), l.Ka, (float*)(ws + l.s), 1,
                          (int)(l.Ka - K)};
        MKP_TRY(go(st, QL_QUANTIZE, 3.0 * m * k, (size_of(x_type) + 1.0) * m * k, [&] { return launch_quantize(q, st); }));
        a.sa = q.s;
    } else if (l.pack_a) {
        MKP_TRY(go(st, QL_PACK, 0.0, 2.0 * m * k,
                   [&] { return launch_q8_pack((const int8_t*)X, ldx, (int8_t*)(ws + l.a), l.Ka, M, (int)K, st); }));
    }
    if (l.quantise || l.pack_a) {
        a.A = (const int8_t*)(ws + l.a);
        a.lda = l.Ka;
    }
    if (l.pack_b) {
        MKP_TRY(go(st, QL_PACK, 0.0, 2.0 * n * k,
                   [&] { return launch_q8_pack(W, ldw, (int8_t*)(ws + l.b), l.Kb, N, (int)K, st); }));
        a.B = (const int8_t*)(ws + l.b);
        a.ldb = l.Kb;
    }
    if (l.stream && !l.quantise && x_type != MKP_I8) {
        a.quantise = true;
        a.x = X;
        a.x_f32 = x_type == MKP_F32;
    }
    const double out = size_of(y_type) * m * n, parts = 4.0 * m * n * (double)l.splits;
    MKP_TRY(go(st, QL_I8_PRODUCT, 2.0 * m * n * k, (m + n) * k + (l.splits > 1 ? parts : out),
               [&] { return l.stream ? launch_i8_stream(a, st) : launch_i8_product(a, st); }));
    if (l.splits == 1) return MKP_OK;
    return go(st, QL_I8_FINISH, 0.0, parts + out, [&] { return launch_i8_finish(a, st); });
}

// ---- backward ------------------------------------------------------------------

struct GradLayout {
    int tile = 256, splits = 1, sum_rows = 64;
    int64_t Mr = 0, Np = 0, Kp = 0;
    size_t a = 0, xb = 0, part = 0, dbp = 0, bytes = 0;
};

GradLayout grad_layout(int64_t M, int64_t N, int64_t K, bool dw, bool dbias) {
    GradLayout l;
    l.Mr = round_up(M, 64);
    l.Np = round_up(N, 8);
    l.Kp = round_up(K, 8);
    // (dW's bits are the same whatever else is asked for: the launch that joins its
    // parts, there for dbias anyway, counts as half of one)
    remembered<1>(M, N, K, l.tile, l.splits, [&] {
        choose_tile(kGradTiles, N, K, l.Mr / 64, l.tile, l.splits, [&](double s) { return grad_joined((double)(N * K), s); });
    });
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (size_t)round_up(bytes, 256);
        return here;
    };
    if (dw) {
        l.a = take(2 * l.Mr * l.Np);
        l.xb = take(2 * M * l.Kp);
        if (l.splits > 1) l.part = take(4 * N * l.Kp * l.splits);
    }
    // rows of a workgroup of the slopes: 64, fewer until there are two workgroups a CU
    while (l.sum_rows > 16 && ceil_div(l.Mr, l.sum_rows) * ceil_div(l.Np, 512) < 512) l.sum_rows /= 2;
    if (dbias) l.dbp = take(4 * ceil_div(l.Mr, l.sum_rows) * l.Np);
    l.bytes = at;
    return l;
}

int backward(int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy, int dy_type, const int8_t* X, int64_t ldx,
             const float* x_scale, const int8_t* Z, int64_t ldz, const float* z_scale, int64_t ldzs, int64_t z_group, int act,
             void* dZ, int64_t lddz, void* dW, int64_t lddw, int dw_type, float* dbias, void* workspace,
             int64_t workspace_bytes, void* stream) {
    MKP_TRY(check_extents(M, N, K));
    if (!real_type(dy_type)) return report(MKP_ERR_INVALID_ARG, "dy_type must be MKP_BF16 or MKP_F32");
    if (act < 0 || act >= ACT_COUNT) return report(MKP_ERR_INVALID_ARG, "unknown activation");
    MKP_TRY(check_ld(lddy, N, "lddy"));
    const bool sloped = act != ACT_NONE;
    if (sloped) {
        MKP_TRY(check_group(z_group));
        MKP_TRY(check_ld(ldz, N, "ldz"));
        MKP_TRY(check_ld(ldzs, groups_of(N, z_group), "ldzs"));
    }
    if (dZ) MKP_TRY(check_ld(lddz, N, "lddz"));
    if (dW) {
        if (!real_type(dw_type)) return report(MKP_ERR_INVALID_ARG, "dw_type must be MKP_BF16 or MKP_F32");
        MKP_TRY(check_ld(ldx, K, "ldx"));
        MKP_TRY(check_ld(lddw, K, "lddw"));
    }
    if (N == 0) return MKP_OK;
    if (K == 0) dW = nullptr;
    if (!dZ && !dW && !dbias) return MKP_OK;
    if (M > 0 && (!dY || (sloped && (!Z || !z_scale)))) return report(MKP_ERR_INVALID_ARG, "dY, Z or z_scale is NULL");
    if (M > 0 && dW && (!X || !x_scale)) return report(MKP_ERR_INVALID_ARG, "X or x_scale is NULL");
    const GradLayout l = grad_layout(M, N, K, dW != nullptr, dbias != nullptr);
    MKP_TRY(check_workspace(workspace, workspace_bytes, l.bytes));
    const int64_t slopes = ceil_div(l.Mr, l.sum_rows) * ceil_div(l.Np, 512) + ceil_div(M, 4);
    const int64_t tiles = dW ? ceil_div(N, l.tile) * ceil_div(K, l.tile) * l.splits : 0;
    const int64_t joined = dW && l.splits > 1 ? N * (l.Kp / 8) : 0;
    if (std::max(slopes * 256, std::max(tiles * 512 + 16 * N + 1024, joined + 8 * N + 1024)) > (int64_t)UINT32_MAX)
        return report(MKP_ERR_UNSUPPORTED, "grid too large");
    if (M == 0 && !dW && !dbias) return MKP_OK;
    begin_call();
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    Q8GradArgs a{};
    a.M = M;
    a.N = (int)N;
    a.K = (int)K;
    a.dy = dY;
    a.lddy = lddy;
    a.dy_f32 = dy_type == MKP_F32;
    a.act = act;
    a.z = Z;
    a.ldz = ldz;
    a.zs = z_scale;
    a.ldzs = ldzs;
    a.zgroup = sloped ? (int)z_group : 0;
    a.x = X;
    a.ldx = ldx;
    a.xs = dW ? x_scale : nullptr;
    a.dz = (uint16_t*)dZ;
    a.lddz = lddz;
    a.dw = dW;
    a.lddw = lddw;
    a.dw_f32 = dw_type == MKP_F32;
    a.dbias = dbias;
    a.a = dW ? (uint16_t*)(ws + l.a) : nullptr;
    a.xb = dW ? (uint16_t*)(ws + l.xb) : nullptr;
    a.part = (float*)(ws + l.part);
    a.dbp = (float*)(ws + l.dbp);
    a.Mr = (int)l.Mr;
    a.Np = (int)l.Np;
    a.Kp = (int)l.Kp;
    a.sum_rows = l.sum_rows;
    a.tile = l.tile;
    a.splits = l.splits;
    const double m = (double)M, n = (double)N, k = (double)K, wb = size_of(dw_type);
    auto pass = [&]() -> int {
        if (M > 0)
            MKP_TRY(go(st, QL_SLOPES, 4.0 * m * n,
                       (size_of(dy_type) + (sloped ? 1.0 : 0.0) + (a.dz ? 2.0 : 0.0) + (dW ? 2.0 : 0.0)) * m * n +
                           (dW && !a.low ? 3.0 * m * k : 0.0),
                       [&] { return launch_q8_slopes(a, st); }));
        const double parts = 4.0 * n * k * (double)l.splits, sums = a.dbias ? 4.0 * n * (double)ceil_div(M, l.sum_rows) : 0.0;
        const double grad = (a.low ? 2.0 : 1.0) * wb * n * k;
        if (dW)
            MKP_TRY(go(st, QL_Q8_PRODUCT, 2.0 * m * n * k, 2.0 * m * (n + k) + (l.splits > 1 ? parts : grad + sums),
                       [&] { return launch_q8_product(a, st); }));
        if (dW ? l.splits == 1 : a.dbias == nullptr) return MKP_OK;
        return go(st, QL_Q8_FINISH, 0.0, (dW ? parts + grad : 0.0) + sums, [&] { return launch_q8_finish(a, st); });
    };
    MKP_TRY(pass());
    if (!dW || !a.dw_f32 || M == 0) return MKP_OK;
    // A binary32 dW: what bf16 left of the operand, through the same workspace, added to it.
    a.low = true;
    a.dz = nullptr;
    a.dbias = nullptr;
    return pass();
}

}  // namespace
}  // namespace mkp

using namespace mkp;

extern "C" {

int mkp_quantize_rows(int64_t M, int64_t K, const void* X, int64_t ldx, int x_type, int64_t group, int8_t* Q, int64_t ldq,
                      float* S, int64_t lds, void* stream) {
    return guarded([&] { return convert(false, M, K, (void*)X, ldx, x_type, group, Q, ldq, S, lds, stream); });
}

int mkp_dequantize_rows(int64_t M, int64_t K, const int8_t* Q, int64_t ldq, const float* S, int64_t lds, int64_t group, void* Y,
                        int64_t ldy, int y_type, void* stream) {
    return guarded([&] { return convert(true, M, K, Y, ldy, y_type, group, (int8_t*)Q, ldq, (float*)S, lds, stream); });
}

int mkp_linear_i8_workspace(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, int x_type, const int8_t* W,
                            int64_t ldw, int64_t* bytes) {
    return guarded([&] {
        if (!bytes) return report(MKP_ERR_INVALID_ARG, "bytes is NULL");
        MKP_TRY(check_linear(M, N, K, ldx, x_type, ldw));
        *bytes = (int64_t)linear_layout(M, N, K, X, ldx, x_type, W, ldw).bytes;
        return (int)MKP_OK;
    });
}

int mkp_linear_i8(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, int x_type, const float* x_scale, const int8_t* W,
                  int64_t ldw, const float* w_scale, const float* bias, int act, void* Y, int64_t ldy, int y_type,
                  void* workspace, int64_t workspace_bytes, void* stream) {
    return guarded([&] {
        return linear(M, N, K, X, ldx, x_type, x_scale, W, ldw, w_scale, bias, act, Y, ldy, y_type, workspace, workspace_bytes,
                      stream);
    });
}

int mkp_linear_q8_backward_workspace(int64_t M, int64_t N, int64_t K, int need_dw, int need_dbias, int64_t* bytes) {
    return guarded([&] {
        if (!bytes) return report(MKP_ERR_INVALID_ARG, "bytes is NULL");
        MKP_TRY(check_extents(M, N, K));
        *bytes = (int64_t)grad_layout(M, N, K, need_dw != 0 && K > 0, need_dbias != 0).bytes;
        return (int)MKP_OK;
    });
}

int mkp_linear_q8_backward(int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy, int dy_type, const int8_t* X,
                           int64_t ldx, const float* x_scale, const int8_t* Z, int64_t ldz, const float* z_scale, int64_t ldzs,
                           int64_t z_group, int act, void* dZ, int64_t lddz, void* dW, int64_t lddw, int dw_type, float* dbias,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    return guarded([&] {
        return backward(M, N, K, dY, lddy, dy_type, X, ldx, x_scale, Z, ldz, z_scale, ldzs, z_group, act, dZ, lddz, dW, lddw,
                        dw_type, dbias, workspace, workspace_bytes, stream);
    });
}

}  // extern "C"

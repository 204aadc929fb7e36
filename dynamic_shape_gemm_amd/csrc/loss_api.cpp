// C-ABI of the vocabulary losses: argument checks, the workspace's layout and
// the order of the launches.  Nothing here allocates device memory or waits:
// the caller gives the workspace, so calls can be captured into a graph, and
// two graphs (or streams) with a workspace each never meet.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <exception>
#include <string>

#include "../../include/mkp.h"
#include "internal.h"
#include "kernels.h"
#include "loss.h"

namespace mkp {

const char* loss_launch_name(int i) {
    static const char* const names[LL_COUNT] = {"loss_flags",  "loss_scan", "loss_gather",   "loss_forward",
                                                "loss_finish", "loss_grad", "loss_products", "loss_outputs"};
    return i >= 0 && i < LL_COUNT ? names[i] : "loss";
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// columns of X and W: a tile's 256 rows stay within 32-bit byte offsets
constexpr int64_t kMaxK = int64_t(1) << 21;
// above this many rows one workgroup counts the live ones; below, every
// workgroup of the gather does so for itself
// (rows x features, scan and gather apart / in one: 4096 x 768 11.0 / 9.1 us,
// 8192 x 768 14.2 / 21.8)
constexpr int64_t kManyRows = 4096;
// up to here the forward pass takes rows as they come, which saves a launch or
// two.  As they come / gathered, us: 32000 x 4096 at 64 rows 63 / 68, at 256 89 /
// 95; 30522 x 768 at 64 21 / 23, at 256 21 / 25, whatever part of the rows is
// labelled.  It loses only where dropping rows spares a row of tiles of a
// product that is not bound by W: 256 x 32000 x 4096 with 50 % labelled 90 / 84,
// 15 % 90 / 76.
constexpr int64_t kDirectRows = 256;
// G of one piece: 8192 rows of which 15 % are live, 30522 x 768, took 372 us a
// step in pieces of 256 MB (two), 325 of 512 and 335 of 1024 (one); 8192 x
// 128256 x 4096 the same within 0.5 % in 2, 4 or 8 pieces
constexpr int64_t kPieceBytes = int64_t(512) << 20;

// A call's extents and where its workspace's parts lie.
struct Layout {
    int tile = 256;
    int64_t Mr = 0, Kp = 0, Vp = 0, kp = 1, ntiles = 0;
    int pieces = 1, slots = 256;
    bool pack_w = false, stream = false;
    size_t hdr = 0, map = 0, pos = 0, live = 0, xc = 0, ids = 0, targets = 0, rws = 0, part = 0, sumz = 0, zt = 0, g = 0,
           dxp = 0, dbp = 0, w = 0, bytes = 0;
};

// What a call costs on tiles of one size, in K steps of all CUs on 256 x 256
// tiles (1.37 us).  Of those one workgroup runs per CU, of 128 x 128 tiles two,
// which reuse half as much of what they load (a step of theirs, a quarter of
// the work in each, 0.7) but have smaller ends.  The logits take rounds of as
// many tiles as run at once, a last one that is at most half full little more
// than half the time (halved tiles, or one workgroup a CU); a tile's ends (its
// exponentials, the pipeline's filling) come on top of its steps.  Backward,
// dX's and dW's tiles share a launch without rounds; dW's have a step per 64
// rows, and ends again.
double tile_cost(int64_t M, int64_t V, int64_t K, bool backward, int tile) {
    const bool big = tile == 256;
    const double step = big ? 1.0 : 0.7, end = big ? 4.0 : 1.75;
    const int64_t slots = big ? 256 : 512, tiles = ceil_div(M, tile) * ceil_div(V, tile), last = tiles % slots;
    const double rounds = (double)(tiles / slots) + (last == 0 ? 0.0 : 2 * last <= slots ? 0.55 : 1.0);
    double cost = rounds * (step * (double)ceil_div(K, 64) + end);
    if (backward) {
        const double one = (double)ceil_div(M, 64) + (big ? 10.0 : 5.5), cols = (double)ceil_div(K, tile);
        const double all = cols * ((double)ceil_div(V, tile) * one + (double)ceil_div(M, tile) * (double)ceil_div(V, 64));
        cost += step * (all / (double)slots + 0.5 * one);
    }
    return cost;
}

// The tile that costs less.  Over 528 extents of 48 to 8000 rows x 1000 to
// 128256 x 64 to 5120 it is within 0.5 % in the mean of the faster of the two,
// forward and backward (always 256: 5 and 10 %; 128 up to 256 rows only: 4 and
// 8).  Forward, 128 / 256: 256 rows x 50257 x 4096 153 us / 108, 384 x 8000 x
// 4096 52 / 72, 320 x 50257 x 768 51 / 56; backward, 320 x 50257 x 768 131 /
// 149, 512 x 50257 x 4096 732 / 623, 8000 x 1000 x 640 104 / 187.
int tile_for(int64_t M, int64_t V, int64_t K, bool backward) {
    // (small tiles only where a launch can count them, with room to spare)
    const int64_t rows = ceil_div(M, 128), cols = ceil_div(V, 128), most = int64_t(1) << 22;
    if (rows > most || cols > most || rows * cols > most || (rows + cols) * ceil_div(K, 128) > most) return 256;
    return tile_cost(M, V, K, backward, 128) < tile_cost(M, V, K, backward, 256) ? 128 : 256;
}

Layout layout_of(int64_t M, int64_t V, int64_t K, int64_t k, const void* W, int64_t ldw, bool backward) {
    Layout l;
    l.tile = tile_for(M, V, K, backward);
    l.Mr = round_up(M, 256);
    l.Kp = round_up(K, 64);
    l.kp = k > 0 ? round_up(k, 4) : 1;
    l.ntiles = ceil_div(V, l.tile);
    l.pack_w = !aligned16(W) || ldw % 8 != 0 || K % 8 != 0;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (size_t)round_up(std::max<int64_t>(bytes, 1), 256);
        return here;
    };
    l.hdr = take(sizeof(LossHeader));
    l.map = take(4 * M);
    l.pos = take(M > kManyRows ? 4 * M : 0);
    l.live = take(k > 0 ? M : 0);
    l.xc = take(2 * l.Mr * l.Kp);
    l.ids = take(k > 0 && backward ? 0 : 4 * l.Mr * l.kp);
    if (l.pack_w) l.w = take(2 * V * l.Kp);
    if (!backward) {
        l.stream = M <= kStreamRows && !l.pack_w && K % 64 == 0;
        if (l.stream) l.ntiles = std::max<int64_t>(l.ntiles, kStreamGroups);
        l.part = take(8 * M * l.ntiles);
        l.sumz = take(4 * M * l.ntiles * loss_sumz_parts(l.tile));
        l.zt = take(4 * l.Mr * l.kp);
    } else {
        l.targets = take(k > 0 ? 8 * l.Mr * l.kp : 0);
        l.rws = take((int64_t)sizeof(LossRow) * l.Mr);
        // pieces of the vocabulary, about equal, whose G fits kPieceBytes
        const int64_t most = std::max<int64_t>(256, kPieceBytes / (2 * std::max<int64_t>(l.Mr, 1)) / 256 * 256);
        l.pieces = (int)ceil_div(V, most);
        l.Vp = round_up(ceil_div(V, l.pieces), 256);
        l.pieces = (int)ceil_div(V, l.Vp);
        l.g = take(2 * l.Mr * l.Vp);
        // dX: one partial, or splits of at most two rounds of tiles and at
        // least four vocabulary steps each
        l.slots = l.tile == 256 ? 256 : 512;
        const int64_t one = l.Mr * l.Kp, steps = l.Vp / 64;
        const int64_t split = std::min<int64_t>(2 * l.slots * l.tile * l.tile, std::max<int64_t>(1, steps / 4) * one);
        l.dxp = take(4 * std::max(one, split));
        l.dbp = take(4 * std::max<int64_t>(1, l.Mr / kDbiasRows) * l.Vp * l.pieces);
    }
    l.bytes = at;
    return l;
}

struct Call {
    int64_t M, V, K;
    const void* X;
    int64_t ldx;
    const void* W;
    int64_t ldw;
    const float* bias;
    bool distill;
    const int64_t* labels;
    float smoothing, z_loss;
    int64_t k;
    const int64_t* ids;
    int64_t ldids;
    const float* teacher;
    int64_t ldt;
    const float* teacher_lse;
    float T, scale, cap;
    bool backward;
    float* loss;
    float* lse;
    const float* dloss;
    void* dX;
    int64_t lddx;
    void* dW;
    int64_t lddw;
    float* dbias;
    int grad_type;
    void* ws;
    int64_t ws_bytes;
    void* stream;
};

int check_shape(int64_t M, int64_t V, int64_t K, int64_t k, int64_t ldw) {
    if (M < 0 || V < 0 || K < 0) return report(MKP_ERR_INVALID_ARG, "negative dimension");
    if (V == 0 || K == 0) return report(MKP_ERR_INVALID_ARG, "an empty vocabulary or no features");
    if (M > INT_MAX / 2 || V > INT_MAX / 2) return report(MKP_ERR_INVALID_ARG, "dimension exceeds 2^30");
    if (K > kMaxK || ldw > 2 * kMaxK) return report(MKP_ERR_INVALID_ARG, "K or ldw too large");
    if (ldw < K) return report(MKP_ERR_INVALID_ARG, "ldw < K");
    if (k < 0 || k > kMaxTargets)
        return report(MKP_ERR_INVALID_ARG, "targets per row must be 1.." + std::to_string(kMaxTargets));
    return MKP_OK;
}

int check(const Call& c) {
    int rc = check_shape(c.M, c.V, c.K, c.distill ? c.k : 0, c.ldw);
    if (rc != MKP_OK) return rc;
    if (c.ldx < c.K) return report(MKP_ERR_INVALID_ARG, "ldx < K");
    if (!c.W) return report(MKP_ERR_INVALID_ARG, "W is NULL");
    if (c.M > 0 && !c.X) return report(MKP_ERR_INVALID_ARG, "X is NULL");
    if (!std::isfinite(c.scale)) return report(MKP_ERR_INVALID_ARG, "scale is not finite");
    // (1 / softcap and log2(e) / T are factors in the kernels)
    if (!(c.cap >= 0.0f) || !std::isfinite(c.cap) || (c.cap > 0.0f && !std::isfinite(1.0f / c.cap)))
        return report(MKP_ERR_INVALID_ARG, "softcap must be 0 or more, its reciprocal finite");
    if (!c.distill) {
        if (c.M > 0 && !c.labels) return report(MKP_ERR_INVALID_ARG, "labels is NULL");
        if (!(c.smoothing >= 0.0f && c.smoothing <= 1.0f))
            return report(MKP_ERR_INVALID_ARG, "smoothing must lie in [0, 1]");
        if (!std::isfinite(c.z_loss)) return report(MKP_ERR_INVALID_ARG, "z_loss is not finite");
    } else {
        if (c.k < 1) return report(MKP_ERR_INVALID_ARG, "targets per row must be 1.." + std::to_string(kMaxTargets));
        if (c.M > 0 && (!c.ids || !c.teacher)) return report(MKP_ERR_INVALID_ARG, "ids or teacher is NULL");
        if (c.ldids < c.k || c.ldt < c.k) return report(MKP_ERR_INVALID_ARG, "ldids < k or ldt < k");
        // (T^2 is a factor of the loss: infinite, or 0 times an infinite divergence, it would be NaN)
        if (!(c.T > 0.0f) || !std::isfinite(c.T) || !std::isnormal(c.T * c.T))
            return report(MKP_ERR_INVALID_ARG, "temperature must be more than 0, its square finite and normal");
    }
    if (c.M > 0 && !c.lse) return report(MKP_ERR_INVALID_ARG, "lse is NULL");
    if (!c.backward) {
        if (c.M > 0 && !c.loss) return report(MKP_ERR_INVALID_ARG, "loss is NULL");
    } else {
        if (c.M > 0 && !c.dloss) return report(MKP_ERR_INVALID_ARG, "dloss is NULL");
        if (c.grad_type != MKP_BF16 && c.grad_type != MKP_F32) return report(MKP_ERR_INVALID_ARG, "unknown grad_type");
        if (c.dX && c.lddx < c.K) return report(MKP_ERR_INVALID_ARG, "lddx < K");
        if (c.dW && c.lddw < c.K) return report(MKP_ERR_INVALID_ARG, "lddw < K");
    }
    return MKP_OK;
}

int run(const Call& c) {
    int rc = check(c);
    if (rc != MKP_OK) return rc;
    if (c.M == 0 && (!c.backward || (!c.dW && !c.dbias))) return MKP_OK;
    if (c.backward && !c.dX && !c.dW && !c.dbias) return MKP_OK;
    const Layout l = layout_of(c.M, c.V, c.K, c.distill ? c.k : 0, c.W, c.ldw, c.backward);
    if (!c.ws || c.ws_bytes < 0 || (size_t)c.ws_bytes < l.bytes || !aligned16(c.ws))
        return report(MKP_ERR_INVALID_ARG,
                      "workspace of " + std::to_string(l.bytes) + " bytes, 16-byte aligned, needed");
    // a launch counts its threads in 32 bits: the tile kernels' (and the halves
    // and splits that they may add), a workgroup per row, a packed row's chunks
    const int64_t row_tiles = ceil_div(c.M, l.tile), col_tiles = ceil_div(c.K, l.tile);
    const int64_t logit_tiles = row_tiles * ceil_div(c.V, l.tile) + l.slots;
    const int64_t grad_tiles = c.backward ? (row_tiles + ceil_div(l.Vp, l.tile)) * col_tiles + 2 * l.slots : 0;
    const int64_t most = UINT32_MAX;
    if (std::max(logit_tiles, grad_tiles) > most / (l.tile == 256 ? 512 : 256) ||
        c.M + ceil_div(c.V, 256) > most / 256 || (l.pack_w && c.V * (l.Kp / 8) > most - 255))
        return report(MKP_ERR_UNSUPPORTED, "grid too large");
    begin_call();
    hipStream_t st = (hipStream_t)c.stream;
    char* ws = (char*)c.ws;
    LossArgs a{};
    a.M = c.M;
    a.V = (int)c.V;
    a.K = (int)c.K;
    a.X = (const uint16_t*)c.X;
    a.ldx = c.ldx;
    a.W = (const uint16_t*)c.W;
    a.ldw = c.ldw;
    a.Kw = (int)c.K;
    a.bias = c.bias;
    a.scale = c.scale;
    a.cap = c.cap;
    a.T = c.distill ? c.T : 1.0f;
    // (x.w times a factor that is 0, or more than there is, would lose what z has)
    a.plain = !c.bias && c.cap == 0.0f && c.scale > 0.0f && std::isnormal(1.4427f * c.scale / a.T);
    a.s2 = (float)(1.4426950408889634 * (a.plain ? (double)c.scale : 1.0) / (double)a.T);
    a.labels = c.distill ? nullptr : c.labels;
    a.smoothing = c.smoothing;
    a.z_loss = c.z_loss;
    a.k = c.distill ? (int)c.k : 1;
    a.ids = c.ids;
    a.ldids = c.ldids;
    a.teacher = c.teacher;
    a.ldt = c.ldt;
    a.teacher_lse = c.teacher_lse;
    a.loss = c.loss;
    a.lse = c.lse;
    a.dloss = c.backward ? c.dloss : nullptr;
    a.dX = c.dX;
    a.lddx = c.lddx;
    a.dW = c.dW;
    a.lddw = c.lddw;
    a.dbias = c.dbias;
    a.grad_f32 = c.grad_type == MKP_F32;
    a.hdr = (LossHeader*)(ws + l.hdr);
    a.map = (int*)(ws + l.map);
    a.pos = (int*)(ws + l.pos);
    a.live = (uint8_t*)(ws + l.live);
    a.Xc = (uint16_t*)(ws + l.xc);
    a.ids32 = (int*)(ws + l.ids);
    a.Mr = (int)l.Mr;
    a.Kp = (int)l.Kp;
    a.Vp = (int)l.Vp;
    a.kp = (int)l.kp;
    a.ntiles = (int)ceil_div(c.V, l.tile);
    a.tile = l.tile;
    a.slots = l.slots;
    const double elem = 2.0, m = (double)c.M, v = (double)c.V, k = (double)c.K;
    const double gb = a.grad_f32 ? 4.0 : 2.0;

    auto go = [&](int what, double flops, double bytes, const std::function<hipError_t()>& fn) -> int {
        hipError_t e = traced_launch(st, what < 0 ? what : kTraceLoss - what, flops, bytes, fn);
        if (e == hipSuccess) return MKP_OK;
        return report(MKP_ERR_HIP, std::string(what < 0 ? "pack" : loss_launch_name(what)) +
                                       " launch: " + hipGetErrorString(e));
    };

    if (l.pack_w) {
        uint16_t* dst = (uint16_t*)(ws + l.w);
        rc = go(-3, 0.0, v * (2.0 * k + 2.0 * (double)l.Kp), [&] {
            return launch_pack_rows((const uint16_t*)c.W, c.ldw, 0, dst, l.Kp, (int)c.V, (int)c.K, 1, st);
        });
        if (rc != MKP_OK) return rc;
        a.W = dst;
        a.ldw = l.Kp;
        a.Kw = (int)l.Kp;
    }
    const double target_bytes = c.distill ? 12.0 * m * (double)c.k : 8.0 * m;
    const bool scanned = c.M > kManyRows;
    auto compact = [&]() -> int {
        if (c.distill && c.M > 0)
            if ((rc = go(LL_FLAGS, 0.0, target_bytes, [&] { return launch_loss_flags(a, st); })) != MKP_OK) return rc;
        if (scanned)
            if ((rc = go(LL_SCAN, 0.0, 8.0 * m, [&] { return launch_loss_scan(a, st); })) != MKP_OK) return rc;
        return go(LL_GATHER, 0.0, 4.0 * m * k + target_bytes, [&] { return launch_loss_gather(a, scanned, st); });
    };

    if (!c.backward) {
        a.part = (float*)(ws + l.part);
        a.sumz = !c.distill && c.smoothing > 0.0f ? (float*)(ws + l.sumz) : nullptr;
        a.zt = (float*)(ws + l.zt);
        a.direct = c.M <= kDirectRows && !l.pack_w && aligned16(c.X) && c.ldx % 8 == 0 && c.ldx <= 2 * kMaxK &&
                   c.K % 64 == 0;
        a.stream = l.stream && a.direct;
        if (a.stream) a.ntiles = kStreamGroups;
        if (!a.direct && (rc = compact()) != MKP_OK) return rc;
        if ((rc = go(LL_FORWARD, 2.0 * m * v * k, elem * (m + v) * k, [&] {
                 return a.stream ? launch_loss_stream(a, st) : launch_loss_forward(a, st);
             })) != MKP_OK)
            return rc;
        return go(LL_FINISH, 0.0, 8.0 * m * (double)l.ntiles, [&] { return launch_loss_finish(a, st); });
    }

    a.targets = (int2*)(ws + l.targets);
    a.rows = (LossRow*)(ws + l.rws);
    a.G = (uint16_t*)(ws + l.g);
    a.dxp = (float*)(ws + l.dxp);
    a.dbp = c.dbias ? (float*)(ws + l.dbp) : nullptr;
    a.ldb = (int)(l.Vp * l.pieces);
    if ((rc = compact()) != MKP_OK) return rc;
    for (int p = 0; p < l.pieces; ++p) {
        a.v0 = (int)(p * l.Vp);
        a.vn = (int)std::min<int64_t>(l.Vp, c.V - a.v0);
        a.first = p == 0;
        const double pv = a.vn, both = (c.dX ? 1.0 : 0.0) + (c.dW ? 1.0 : 0.0);
        if (c.M > 0)
            if ((rc = go(LL_GRAD, 2.0 * m * pv * k, elem * ((m + pv) * k + m * pv),
                         [&] { return launch_loss_grad(a, st); })) != MKP_OK)
                return rc;
        if (c.dX || c.dW)
            if ((rc = go(LL_PRODUCTS, 2.0 * both * m * pv * k,
                         both * elem * m * pv + (c.dX ? elem * pv * k + (p ? 8.0 : 4.0) * m * k : 0.0) +
                             (c.dW ? elem * m * k + gb * pv * k : 0.0),
                         [&] { return launch_loss_products(a, st); })) != MKP_OK)
                return rc;
    }
    if (!(c.dX && c.M > 0) && !c.dbias) return MKP_OK;
    return go(LL_OUTPUTS, 0.0,
              (c.dX ? (4.0 + gb) * m * k : 0.0) + (c.dbias ? 4.0 * v * (double)ceil_div(c.M, kDbiasRows) : 0.0),
              [&] { return launch_loss_outputs(a, st); });
}

// No exception leaves the C entry points.
template <class F>
int guarded(F&& fn) {
    try {
        return fn();
    } catch (const std::exception& e) {
        try {
            return report(MKP_ERR_HIP, e.what());
        } catch (...) {
        }
    } catch (...) {
    }
    return MKP_ERR_HIP;
}

}  // namespace
}  // namespace mkp

using namespace mkp;

extern "C" {

int mkp_linear_loss_workspace(int64_t M, int64_t V, int64_t K, int64_t k, const void* W, int64_t ldw, int backward,
                              int64_t* bytes) {
    return guarded([&] {
        if (!bytes) return report(MKP_ERR_INVALID_ARG, "bytes is NULL");
        const int rc = check_shape(M, V, K, k, ldw);
        if (rc != MKP_OK) return rc;
        *bytes = (int64_t)layout_of(M, V, K, k, W, ldw, backward != 0).bytes;
        return (int)MKP_OK;
    });
}

int mkp_linear_xent(int64_t M, int64_t V, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                    const float* bias, const int64_t* labels, float scale, float softcap, float smoothing, float z_loss,
                    float* loss, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    Call c{};
    c.M = M, c.V = V, c.K = K, c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw, c.bias = bias, c.labels = labels;
    c.scale = scale, c.cap = softcap, c.smoothing = smoothing, c.z_loss = z_loss, c.loss = loss, c.lse = lse;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return guarded([&] { return run(c); });
}

int mkp_linear_xent_backward(int64_t M, int64_t V, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                             const float* bias, const int64_t* labels, float scale, float softcap, float smoothing,
                             float z_loss, const float* lse, const float* dloss, void* dX, int64_t lddx, void* dW,
                             int64_t lddw, float* dbias, int grad_type, void* workspace, int64_t workspace_bytes,
                             void* stream) {
    Call c{};
    c.M = M, c.V = V, c.K = K, c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw, c.bias = bias, c.labels = labels;
    c.scale = scale, c.cap = softcap, c.smoothing = smoothing, c.z_loss = z_loss, c.lse = (float*)lse, c.dloss = dloss;
    c.backward = true, c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw, c.dbias = dbias, c.grad_type = grad_type;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return guarded([&] { return run(c); });
}

int mkp_linear_distill(int64_t M, int64_t V, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                       const float* bias, int64_t k, const int64_t* ids, int64_t ldids, const float* teacher, int64_t ldt,
                       const float* teacher_lse, float temperature, float scale, float softcap, float* loss, float* lse,
                       void* workspace, int64_t workspace_bytes, void* stream) {
    Call c{};
    c.M = M, c.V = V, c.K = K, c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw, c.bias = bias;
    c.distill = true, c.k = k, c.ids = ids, c.ldids = ldids, c.teacher = teacher, c.ldt = ldt, c.teacher_lse = teacher_lse;
    c.T = temperature, c.scale = scale, c.cap = softcap, c.loss = loss, c.lse = lse;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return guarded([&] { return run(c); });
}

int mkp_linear_distill_backward(int64_t M, int64_t V, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                const float* bias, int64_t k, const int64_t* ids, int64_t ldids, const float* teacher,
                                int64_t ldt, const float* teacher_lse, float temperature, float scale, float softcap,
                                const float* lse, const float* dloss, void* dX, int64_t lddx, void* dW, int64_t lddw,
                                float* dbias, int grad_type, void* workspace, int64_t workspace_bytes, void* stream) {
    Call c{};
    c.M = M, c.V = V, c.K = K, c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw, c.bias = bias;
    c.distill = true, c.k = k, c.ids = ids, c.ldids = ldids, c.teacher = teacher, c.ldt = ldt, c.teacher_lse = teacher_lse;
    c.T = temperature, c.scale = scale, c.cap = softcap, c.lse = (float*)lse, c.dloss = dloss;
    c.backward = true, c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw, c.dbias = dbias, c.grad_type = grad_type;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return guarded([&] { return run(c); });
}

}  // extern "C"

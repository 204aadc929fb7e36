// Host-side view of the vocabulary-loss kernels: the losses behind a linear
// layer whose output columns are a vocabulary, computed from the layer's
// input X (M x K) and weight W (V x K) without storing the M x V logits.
//
//   s = scale x.w_v + b_v,  z = cap tanh(s / cap) (or s),  zh = z / T
//   lse = log sum_v e^{zh_v},  q_v = e^{zh_v - lse}
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace mkp {

constexpr int kMaxTargets = 1024;   // per row (distillation)
constexpr int kDbiasRows = 128;     // rows of one partial sum of dbias
constexpr int kStreamRows = 32;     // most rows of the kernel for few rows
constexpr int kStreamGroups = 256;   // workgroups of the kernel for few rows: one per CU

// What a call keeps in its workspace besides the large arrays; written by
// the row-scan kernel, read by every later one.
struct LossHeader {
    int n;          // rows that carry a target ("live"), compacted to the front
    float gref;     // backward: the largest |dloss| of a live row (1 if that is 0 or not finite)
    int splits;     // backward: partials of dX
};

// One live row's constants in the gradient (compact order):
//   dL/ds_v / (gref * unit) = (q_v rq - ru - [v a target] w) * slope
struct LossRow {
    float lse2;     // log2(e) * lse
    float rq, ru;
    float rp;       // weight of the one target (cross entropy)
};

struct LossArgs {
    int64_t M;              // rows of X
    int V, K;               // vocabulary, features
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* W;      // rows 16-byte aligned: the caller's, or a copy padded with zeros
    int64_t ldw;
    int Kw;                 // W's columns: K (a multiple of 8), or Kp for the padded copy
    const float* bias;      // V values or null
    float scale, cap, T;
    bool plain;             // z = scale x.w with scale > 0: the kernels keep x.w instead of z
    float s2;               // from what they keep to the base-2 logit, log2(e) z / T
    bool stream;            // forward: the kernel for few rows (then direct too)
    bool direct;            // forward on few aligned rows: X and targets as the caller has them
    // cross entropy
    const int64_t* labels;  // M, or null for distillation
    float smoothing, z_loss;
    // distillation
    int k;                  // targets per row (1 for cross entropy)
    const int64_t* ids;     // M x k
    int64_t ldids;
    const float* teacher;   // M x k
    int64_t ldt;
    const float* teacher_lse;   // M or null
    // forward results (backward: lse is an input)
    float* loss;
    float* lse;
    // backward
    const float* dloss;
    void* dX;
    int64_t lddx;
    void* dW;
    int64_t lddw;
    float* dbias;
    bool grad_f32;          // dX and dW hold binary32 instead of bf16
    // workspace
    LossHeader* hdr;
    int* map;               // compact row -> row
    int* pos;               // row -> compact row (calls of many rows)
    uint8_t* live;          // M (distillation)
    uint16_t* Xc;           // live rows of X, Mr x Kp, zero padded
    int* ids32;             // compact, n x kp: the targets (-1: none; distillation: forward)
    int2* targets;          // backward, distillation: compact, n x kp: the targets and the bits of their weights
    LossRow* rows;          // compact
    float* part;            // forward: per (row, vocabulary tile) maximum and sum of exponentials
    float* sumz;            // forward with smoothing: per (row, vocabulary tile, wave column) sum of kept values
    float* zt;              // forward: the targets' kept values, compact n x kp
    uint16_t* G;            // backward: one piece's gradient by s, Mr x Vp
    float* dxp;             // backward: dX partials, [splits][rows of live tiles][Kp]
    float* dbp;             // backward: sums of G's columns over kDbiasRows rows each, [Mr / kDbiasRows][ldb]
    int ldb;
    int Mr, Kp, Vp, kp;     // padded extents
    int tile;               // rows and columns of the tile kernels' tiles: 256 or 128
    int ntiles;             // vocabulary tiles of the forward pass
    // the piece of the vocabulary a backward launch works on
    int v0, vn;
    int slots;              // workgroups of a tile kernel that run at once
    bool first;             // dX partials are written, not added to
};

// Partial sums of z per row and tile (LossArgs::sumz).
int loss_sumz_parts(int tile);

// Launches; each returns the launch's status.
hipError_t launch_loss_flags(const LossArgs& a, hipStream_t st);       // distillation: live
hipError_t launch_loss_scan(const LossArgs& a, hipStream_t st);        // hdr, pos (calls of many rows)
hipError_t launch_loss_gather(const LossArgs& a, bool scanned, hipStream_t st);   // hdr, map, Xc, targets, rows
hipError_t launch_loss_forward(const LossArgs& a, hipStream_t st);     // part, sumz, zt
hipError_t launch_loss_stream(const LossArgs& a, hipStream_t st);      // the same for at most kStreamRows rows
hipError_t launch_loss_finish(const LossArgs& a, hipStream_t st);      // loss, lse
hipError_t launch_loss_grad(const LossArgs& a, hipStream_t st);        // G (and dbp) of a piece
hipError_t launch_loss_products(const LossArgs& a, hipStream_t st);    // dxp and dW of a piece
hipError_t launch_loss_outputs(const LossArgs& a, hipStream_t st);     // dX and dbias from their partials

}  // namespace mkp

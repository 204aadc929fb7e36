// Host-side view of the 8-bit kernels: matrices held row by row as integers of
// -127 .. 127 times binary32 scales, a linear layer on them, and the backward
// pass of a layer whose input and pre-activation are held so.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace mkp {

constexpr int kI8StreamRows = 32;   // most tokens of the product for few
constexpr int kI8StreamInput = 131072;   // and, where tiles take W as it is, most integers of X
constexpr int kI8StreamUnits = 64;  // runs of 512 features that it quantises by itself
constexpr int kQ8MaxGroup = 256;   // columns of one scale, if not the whole row

// A matrix <-> its 8-bit form.
struct QuantArgs {
    int64_t M;
    int K;
    void* x;               // M x K, bf16 or binary32: the source, or what is read back
    int64_t ldx;
    bool f32;
    int group;             // columns of a scale: 0 (the row), or a power of two
    int8_t* q;
    int64_t ldq;
    float* s;              // row m, group j: s[m * lds + j]
    int64_t lds;
    int pad;               // columns from K on that are set to 0 with a row (quantise)
};

// C = act(sa sb (A . B^T) + bias) of 8-bit A (M x K) and B (N x K).
struct I8Args {
    int64_t M;
    int N, K;
    const int8_t* A;       // rows 16-byte aligned on tiles, of any alignment in the stream
    int64_t lda;
    const float* sa;       // M
    const int8_t* B;       // as A's
    int64_t ldb;
    const float* sb;       // N
    const float* bias;     // N or null
    int act;
    void* C;
    int64_t ldc;
    bool bf16;             // C holds bf16 instead of binary32
    bool quantise;         // few tokens: x is X itself (lda its leading dimension), quantised by the product
    const void* x;
    bool x_f32;
    int tile;              // rows and columns of a tile: 256, 128 or 64
    int splits;            // of K; more than one: partial sums, joined by another launch
    int* part;             // [splits][M][ldp]
    int64_t ldp;
};

// Gradients of y = act(z), z = x w^T + bias from dy, with x and z in 8 bits.
struct Q8GradArgs {
    int64_t M;
    int N, K;
    const void* dy;        // M x N
    int64_t lddy;
    bool dy_f32;
    int act;
    const int8_t* z;       // M x N (unless act is ACT_NONE)
    int64_t ldz;
    const float* zs;
    int64_t ldzs;
    int zgroup;
    const int8_t* x;       // M x K
    int64_t ldx;
    const float* xs;       // M
    uint16_t* dz;          // M x N bf16, or null
    int64_t lddz;
    void* dw;              // N x K, or null
    int64_t lddw;
    bool dw_f32;
    float* dbias;          // N, or null
    // workspace
    uint16_t* a;           // dz times its row's scale in bf16, Mr x Np (rows past M zero)
    uint16_t* xb;          // x's integers in bf16, M x Kp
    float* part;           // dW's partials [splits][N][Kp] (several splits)
    float* dbp;            // column sums of dz over sum_rows rows each, [M / sum_rows][Np]
    int Mr, Np, Kp;
    int sum_rows;          // a multiple of 16
    bool low;              // a binary32 dW's second pass: a is what bf16 left of dz x_scale, dW is added to
    int tile, splits;
};

// Launches; each returns the launch's status.
hipError_t launch_quantize(const QuantArgs& a, hipStream_t st);
hipError_t launch_dequantize(const QuantArgs& a, hipStream_t st);
// Rows of 8-bit integers copied to rows of `ldd` bytes (a multiple of 16), the rest zero.
hipError_t launch_q8_pack(const int8_t* src, int64_t lds, int8_t* dst, int64_t ldd, int64_t rows, int cols,
                          hipStream_t st);
hipError_t launch_i8_product(const I8Args& a, hipStream_t st);
hipError_t launch_i8_stream(const I8Args& a, hipStream_t st);     // at most kI8StreamRows tokens, rows of any alignment
hipError_t launch_i8_finish(const I8Args& a, hipStream_t st);     // C from its partial sums
hipError_t launch_q8_slopes(const Q8GradArgs& a, hipStream_t st);  // dz, a, xb, dbp
hipError_t launch_q8_product(const Q8GradArgs& a, hipStream_t st); // dW and dbias (one split), or dW's partials
hipError_t launch_q8_finish(const Q8GradArgs& a, hipStream_t st);  // dW from its partials, and dbias

}  // namespace mkp

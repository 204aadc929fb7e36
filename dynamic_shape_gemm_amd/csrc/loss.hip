// Vocabulary losses on CDNA4 (gfx950): softmax cross entropy and top-logit
// distillation straight from a linear layer's input X (M x K) and weight W
// (V x K), forward and backward, the M x V logits never stored.
//
//   forward   each workgroup multiplies one tile of X . W^T on bf16 MFMA and
//             reduces it, still in registers, to every row's maximum and sum
//             of exponentials (base 2) over the tile's columns; a second
//             kernel joins a row's tiles into its log-partition and loss.
//   backward  a piece of the vocabulary at a time: the same product again
//             (that costs 2MVK operations and saves holding 4MV bytes), its
//             tile turned in registers into the gradient by the logits, G,
//             which goes to the workspace in bf16; then dX += G . W and
//             dW = G^T . X over the piece.
//
// Rows without a target are dropped first: the live rows of X are copied
// together (zero padded), so a batch of which 15 % carry a label costs 15 %,
// and whatever the dropped rows hold (NaN as well) reaches no output.  Their
// number stays on the device; the grids cover the most there can be and the
// surplus workgroups leave at once.
#include "loss.h"

#include "kernels.h"

#include <hip/hip_ext.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mkp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char lds_t;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

template <typename F, typename... Args>
hipError_t launch_kernel(F kernel, dim3 grid, dim3 block, hipStream_t st, Args... args) {
    LaunchEvents& ev = launch_events();
    if (ev.start != nullptr) {
        const LaunchEvents use = ev;
        ev = LaunchEvents{};
        hipExtLaunchKernelGGL(kernel, grid, block, 0, st, use.start, use.stop, 0, args...);
    } else {
        hipLaunchKernelGGL(kernel, grid, block, 0, st, args...);
    }
    return hipGetLastError();
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Round to nearest even, NaN kept a NaN: the conversion instruction.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// tanh: an odd polynomial (its Taylor series, next term below 1e-8 relative)
// where 1 - 2/(1 + e^2x) would cancel, that form elsewhere.
__device__ __forceinline__ float tanh_fast(float x) {
    const float x2 = x * x;
    const float p = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f),
                                      -1.0f / 3.0f), 1.0f);
    const float e = exp2_fast(2.0f * kLog2e * x);
    const float f = fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + e), 1.0f);
    return fabsf(x) < 0.25f ? p : f;
}

// ---- tiles -----------------------------------------------------------------
//
// One workgroup multiplies a BM x BN tile over K steps of 64 on 16x16x32
// MFMAs.  Each operand's tile is two halves of BM / 2 (BN / 2) rows, each in
// a block of its own in LDS, and a wave's part of the tile is one block of
// every half pair: the four quadrants are what a wave works through in turn.
//
// An operand is read either along its rows (the reduction is contiguous:
// X and W for the logits, G for dX) or across them (the reduction is the
// row: W for dX, G and X for dW); the second form goes through the LDS
// transpose read, which hands each lane four values of one column.
template <int WGM_, int WGN_, int FM_, int FN_, bool AT_, bool BT_>
struct LTile {
    static constexpr int WGM = WGM_, WGN = WGN_, FM = FM_, FN = FN_;   // FM, FN: 16-row fragments per wave and half
    static constexpr bool AT = AT_, BT = BT_;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int HA = WGM * FM * 16, HB = WGN * FN * 16;
    static constexpr int BM = 2 * HA, BN = 2 * HB, BK = 64;
    static constexpr int HA_BYTES = HA * 128, HB_BYTES = HB * 128;
    static constexpr int STAGE = 2 * (HA_BYTES + HB_BYTES);
    static constexpr int IA = HA_BYTES / 1024 / NW, IB = HB_BYTES / 1024 / NW;   // direct loads per wave and half
    static constexpr int LDS = 2 * STAGE;
    static_assert(HA_BYTES % (1024 * NW) == 0 && HB_BYTES % (1024 * NW) == 0, "halves are whole loads");
    static_assert(!AT || HA == 128 || HA == 64, "transposed rows of 256 or 128 bytes");
    static_assert(!BT || HB == 128 || HB == 64, "transposed rows of 256 or 128 bytes");
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

// Chunk swizzle of a 128-byte row (eight 16-byte chunks): the 16 rows of a
// fragment read meet 16 distinct bank windows.
__device__ __forceinline__ int swz_row(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Segment swizzle of a transposed row (32-byte segments): the eight rows a
// 32-lane pass of the transpose read touches (8g .. 8g+3 for two g) meet
// eight distinct bank windows.
template <int H>
__device__ __forceinline__ int swz_tr(int k) {
    if constexpr (H == 128) return (k & 3) | (((k >> 3) & 1) << 2);
    else return ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
}

// Where one lane's 16 bytes of a half's load `p` (load * 64 + lane) come
// from: row r and first element c of the half.
template <int H, bool TR>
__device__ __forceinline__ void half_slot(int p, int& r, int& c) {
    if constexpr (!TR) {
        r = p >> 3;
        c = ((p & 7) ^ swz_row(r)) * 8;
    } else {
        constexpr int CPR = H / 8;
        r = p / CPR;
        const int q = p % CPR;
        c = ((((q >> 1) ^ swz_tr<H>(r)) << 1) | (q & 1)) * 8;
    }
}

// One direct global->LDS load, 16 bytes a lane from base + off (bytes), the
// wave's 64 chunks in lane order at `lds` (wave-uniform).  In asm because the
// compiler cannot tell the stages apart and would wait for every load in
// flight before any fragment read; the main loop's own waits order them.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand of a tile: where its halves' loads come from.
//   rows (not TR): `lim` valid rows of the tile; a last step of fewer than 64
//     columns (`tail` > 0 of them) repeats the step's first chunk in the
//     missing ones, where the other operand holds zeros
//   columns (TR): `lim` valid columns of the tile; a last step of fewer than
//     64 rows repeats its last row likewise
// Both need `lim` and `tail` to be multiples of 8 columns.
template <int H, bool TR, int I, int NW>
struct Operand {
    const char* base;      // tile origin, step 0
    int64_t step_bytes;
    int64_t ld;
    uint32_t off[2][I];
    int lim, steps, tail;

    __device__ __forceinline__ uint32_t offset(int h, int i, int wave, int lane, int most) const {
        int r, c;
        half_slot<H, TR>((i * NW + wave) * 64 + lane, r, c);
        if constexpr (!TR) {
            if (c >= most) c = 0;
            r = min(h * H + r, lim - 1);
        } else {
            r = min(r, most - 1);
            c = min(h * H + c, lim - 8);
        }
        return (uint32_t)((r * ld + c) * 2);
    }
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int lim_, int steps_, int tail_, int wave,
                                         int lane) {
        base = (const char*)p;
        ld = ld_;
        lim = lim_;
        steps = steps_;
        tail = tail_;
        step_bytes = TR ? ld * 128 : 128;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < I; ++i) off[h][i] = offset(h, i, wave, lane, 64);
    }
    __device__ __forceinline__ void issue(int h, int step, uint32_t lds, int wave, int lane) const {
        const char* b = base + step * step_bytes;
        if (tail > 0 && step == steps - 1) {
#pragma unroll
            for (int i = 0; i < I; ++i) dma16(b, offset(h, i, wave, lane, tail), lds + (i * NW + wave) * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < I; ++i) dma16(b, off[h][i], lds + (i * NW + wave) * 1024);
        }
    }
};

// Fragments of one half from LDS: F 16-row fragments x 2 K halves of 32.
// Lane 16 g + s holds row s, K values 32 ks + 8 g + 0..7.
template <int H, bool TR, int F>
struct FragReader {
    uint32_t addr[TR ? F : 2];   // TR: per fragment; else: per K half
    __device__ __forceinline__ void init(int wpos, int lane) {
        const int g = lane >> 4, s = lane & 15;
        if constexpr (!TR) {
            const int row = wpos * F * 16 + s;
            addr[0] = row * 128 + ((g ^ swz_row(s)) << 4);
            addr[1] = addr[0] ^ 64;
        } else {
            const int k = 8 * g + (s >> 2);
#pragma unroll
            for (int i = 0; i < F; ++i)
                addr[i] = k * (H * 2) + (((wpos * F + i) ^ swz_tr<H>(k)) << 5) + (s & 3) * 8;
        }
    }
    __device__ __forceinline__ bf16x8 read(const lds_t* half, int i, int ks) const {
        if constexpr (!TR) {
            return __builtin_bit_cast(
                bf16x8, *(const u32x4 __attribute__((address_space(3)))*)(half + addr[ks] + i * 2048));
        } else {
            const lds_t* p = half + addr[i] + ks * 32 * H * 2;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 __attribute__((address_space(3)))*)p);
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 __attribute__((address_space(3)))*)(p + 4 * H * 2));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

template <class T>
using Acc = f32x4[2][2][T::FM][T::FN];

// Wait until at most N of this wave's direct loads are in flight and its LDS
// reads are done, then meet the other waves; nothing is scheduled across.
template <int N>
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void plain_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// acc := the tile's product over `steps` K steps, two LDS stages.
//
// A step is four phases, one quadrant of the wave's tile each:
//     phase   reads into registers      loads issued     multiplies
//       0     A0 of step s              B0 of step s+2   A0 x B0
//       1     B1 of step s              A0 of step s+2   A0 x B1
//       2     A1 of step s              B1 of step s+2   A1 x B0
//       3     B0 of step s+1            A1 of step s+2   A1 x B1
// Every half's LDS block is read in one phase only and refilled from the next
// phase on, so loads have six phases (one and a half steps) to arrive with two
// stages: at each phase's end six later halves may still be in flight.
// Within a phase: the reads and loads, a barrier, the multiplications.  With
// eight waves the second four run half a phase behind the first (one barrier
// more at the start, one less at the end), so on every SIMD one wave
// multiplies while the other reads.
template <class T>
__device__ __forceinline__ void main_loop(const Operand<T::HA, T::AT, T::IA, T::NW>& A,
                                          const Operand<T::HB, T::BT, T::IB, T::NW>& B, int steps, lds_t* smem,
                                          int wave, int lane, Acc<T>& acc) {
    constexpr bool PP = T::NW == 8;
    constexpr int I = T::IA;
    static_assert(T::IA == T::IB, "halves are counted in loads");
    const int wm = wave % T::WGM, wn = wave / T::WGM;
    FragReader<T::HA, T::AT, T::FM> ra;
    FragReader<T::HB, T::BT, T::FN> rb;
    ra.init(wm, lane);
    rb.init(wn, lane);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
    auto issue_a = [&](int h, int s) { A.issue(h, s, lds0 + (s & 1) * T::STAGE + h * T::HA_BYTES, wave, lane); };
    auto issue_b = [&](int h, int s) {
        B.issue(h, s, lds0 + (s & 1) * T::STAGE + 2 * T::HA_BYTES + h * T::HB_BYTES, wave, lane);
    };
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) acc[ha][hb][i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (steps <= 0) {
        __syncthreads();
        return;
    }
    bf16x8 ya[2][T::FM], xb[2][2][T::FN];
    auto read_a = [&](int h, int s) {
        const lds_t* p = smem + (s & 1) * T::STAGE + h * T::HA_BYTES;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) ya[ks][i] = ra.read(p, i, ks);
    };
    auto read_b = [&](int h, int s) {
        const lds_t* p = smem + (s & 1) * T::STAGE + 2 * T::HA_BYTES + h * T::HB_BYTES;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) xb[h][ks][j] = rb.read(p, j, ks);
    };
    auto multiply = [&](int ha, int hb) {
        if constexpr (PP) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
                    acc[ha][hb][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[hb][ks][j], ya[ks][i],
                                                                               acc[ha][hb][i][j], 0, 0, 0);
        if constexpr (PP) {
            __builtin_amdgcn_s_setprio(0);
            plain_barrier();
        } else {
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // LEFT: steps after this one (2: two or more)
    auto step = [&](auto left, int s) {
        constexpr int LEFT = decltype(left)::value;
        // loads that may still be in flight at each phase's end: six halves,
        // fewer where nothing more is issued
        constexpr int W0 = LEFT == 2 ? 6 : LEFT == 1 ? 5 : 1, W1 = LEFT == 2 ? 6 : LEFT == 1 ? 4 : 0;
        constexpr int W2 = LEFT == 2 ? 6 : LEFT == 1 ? 3 : 0, W3 = LEFT == 2 ? 6 : LEFT == 1 ? 2 : 0;
        read_a(0, s);
        if constexpr (LEFT == 2) issue_b(0, s + 2);
        phase_barrier<W0 * I>();
        multiply(0, 0);
        read_b(1, s);
        if constexpr (LEFT == 2) issue_a(0, s + 2);
        phase_barrier<W1 * I>();
        multiply(0, 1);
        read_a(1, s);
        if constexpr (LEFT == 2) issue_b(1, s + 2);
        phase_barrier<W2 * I>();
        multiply(1, 0);
        if constexpr (LEFT >= 1) read_b(0, s + 1);
        if constexpr (LEFT == 2) issue_a(1, s + 2);
        phase_barrier<W3 * I>();
        multiply(1, 1);
    };
    // the first two steps' loads, in the order of their use
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s < steps) {
            issue_b(0, s);
            issue_a(0, s);
            issue_b(1, s);
            issue_a(1, s);
        }
    }
    if (steps > 1) phase_barrier<6 * I>();
    else phase_barrier<2 * I>();
    read_b(0, 0);
    phase_barrier<6 * I>();
    if (PP && wave >= T::NW / 2) plain_barrier();
    int s = 0;
    for (; s + 2 < steps; ++s) step(std::integral_constant<int, 2>{}, s);
    if (steps > 1) step(std::integral_constant<int, 1>{}, s++);
    step(std::integral_constant<int, 0>{}, s);
    if (PP && wave < T::NW / 2) plain_barrier();
    __syncthreads();   // the stages are free for the epilogue
}

// A lane's places in the tile: the value acc[ha][hb][i][j][r] is row
// row(ha, i), column col(hb, j) + r.
template <class T>
struct Place {
    int wm, wn, g, s;
    __device__ __forceinline__ Place(int wave, int lane)
        : wm(wave % T::WGM), wn(wave / T::WGM), g(lane >> 4), s(lane & 15) {}
    __device__ __forceinline__ int row(int ha, int i) const { return ha * T::HA + (wm * T::FM + i) * 16 + s; }
    __device__ __forceinline__ int col(int hb, int j) const { return hb * T::HB + (wn * T::FN + j) * 16 + g * 4; }
};

// Workgroup -> tile.  Workgroups are dealt round-robin to the 8 XCDs; ids are
// regrouped so that each XCD gets a contiguous run of tiles, which walk eight
// tile rows per tile column (neighbours on one XCD share rows and columns in
// its L2).  The run is cut from the live tiles, so that a batch with few live
// rows still spreads over every XCD.
__device__ __forceinline__ bool map_tile(int bid, int tm_n, int tn_n, int& tm, int& tn, int& rest, int parts) {
    const int T = tm_n * tn_n, G = T * parts;
    if (bid >= G) return false;
    const int q = G >> 3, r = G & 7, x = bid & 7;
    const int L = x * q + min(x, r) + (bid >> 3);
    rest = L / T;
    const int tile = L - rest * T;
    constexpr int GROUP = 8;
    const int per = GROUP * tn_n, g = tile / per, first = g * GROUP;
    const int gsz = min(tm_n - first, GROUP), in = tile - g * per;
    tm = first + in % gsz;
    tn = in / gsz;
    return true;
}

// ---- the logits of a tile ---------------------------------------------------

// acc (x.w) -> z in place.
template <class T>
__device__ __forceinline__ void to_logits(Acc<T>& acc, const LossArgs& a, const Place<T>& at, int v_tile) {
    if (a.bias != nullptr) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                f32x4 b;
#pragma unroll
                for (int r = 0; r < 4; ++r) b[r] = a.bias[min(v_tile + at.col(hb, j) + r, a.V - 1)];
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int i = 0; i < T::FM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[ha][hb][i][j][r] = fmaf(a.scale, acc[ha][hb][i][j][r], b[r]);
            }
    } else if (a.scale != 1.0f) {
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int i = 0; i < T::FM; ++i)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) acc[ha][hb][i][j] *= a.scale;
    }
    if (a.cap > 0.0f) {
        const float inv = 1.0f / a.cap;
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[ha][hb][i][j][r] = a.cap * tanh_fast(acc[ha][hb][i][j][r] * inv);
                __builtin_amdgcn_sched_barrier(0);   // (a row of fragments at a time, or the registers spill)
            }
    }
}

// The tile's product X . W^T, as logits z.
template <class T>
__device__ __forceinline__ void logits_tile(const LossArgs& a, int m0, int v_tile, lds_t* smem, int wave, int lane,
                                            Acc<T>& acc) {
    const int steps = (a.Kw + 63) >> 6;
    Operand<T::HA, false, T::IA, T::NW> A;
    Operand<T::HB, false, T::IB, T::NW> B;
    A.init(a.Xc + (int64_t)m0 * a.Kp, a.Kp, T::BM, steps, 0, wave, lane);
    B.init(a.W + (int64_t)v_tile * a.ldw, a.ldw, a.V - v_tile, steps, a.Kw & 63, wave, lane);
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    to_logits<T>(acc, a, Place<T>(wave, lane), v_tile);
}

// ---- forward ----------------------------------------------------------------

// Statistics of one logit tile.  TG: the targets' z are picked from the tile
// staged in LDS, half its rows at a time (several targets a row); else each
// lane compares its columns with the row's one label.
template <class T, bool TG>
__global__ __launch_bounds__(T::NT) void loss_forward_kernel(LossArgs a) {
    constexpr int TAB = TG ? T::HA * (T::BN + 4) * 4 : 0;
    constexpr int RED = 3 * T::WGN * T::BM * 4;
    constexpr int NEED = TAB > RED ? TAB : RED;
    __shared__ __attribute__((aligned(1024))) unsigned char raw[T::LDS > NEED ? T::LDS : NEED];
    lds_t* smem = (lds_t*)raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.hdr->n;
    int tm, tn, rest;
    if (!map_tile(blockIdx.x, (n + T::BM - 1) / T::BM, a.ntiles, tm, tn, rest, 1)) return;
    const int m0 = tm * T::BM, v0 = tn * T::BN;
    Acc<T> acc;
    logits_tile<T>(a, m0, v0, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    const int vr = a.V - v0;   // valid columns
    if constexpr (TG) {
        float __attribute__((address_space(3)))* tab = (float __attribute__((address_space(3)))*)smem;
        constexpr int LD = T::BN + 4;
#pragma unroll
        for (int ha = 0; ha < 2; ++ha) {
            if (ha) __syncthreads();
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int i = 0; i < T::FM; ++i)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
                        *(f32x4 __attribute__((address_space(3)))*)(tab + (at.row(ha, i) - ha * T::HA) * LD +
                                                                    at.col(hb, j)) = acc[ha][hb][i][j];
            __syncthreads();
            constexpr int PER = T::NT / T::HA;   // threads per row
            const int r = tid / PER, m = m0 + ha * T::HA + r;
            if (m < n) {
                const int* ids = a.ids32 + (int64_t)m * a.kp;
                for (int q = (tid % PER) * 4; q < a.kp; q += PER * 4) {
                    const int4 id = *(const int4*)(ids + q);
                    const int c[4] = {id.x - v0, id.y - v0, id.z - v0, id.w - v0};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((unsigned)c[e] < (unsigned)T::BN)
                            a.zt[(int64_t)m * a.kp + q + e] = tab[r * LD + c[e]];
                }
            }
        }
        __syncthreads();
    }
    // per row: maximum, sum of 2^((z - maximum) c), and sum of z where asked for
    const float c2 = kLog2e / a.T;
    const bool smooth = a.sumz != nullptr;
    float __attribute__((address_space(3)))* red = (float __attribute__((address_space(3)))*)smem;
    if (smooth) {
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                float sz = 0.0f;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) sz += at.col(hb, j) + r < vr ? acc[ha][hb][i][j][r] : 0.0f;
                sz += __shfl_xor(sz, 16);
                sz += __shfl_xor(sz, 32);
                if (at.g == 0) red[(2 * T::WGN + at.wn) * T::BM + at.row(ha, i)] = sz;
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    if (vr < T::BN) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = at.col(hb, j) + r < vr;
#pragma unroll
                    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                        for (int i = 0; i < T::FM; ++i)
                            acc[ha][hb][i][j][r] = in ? acc[ha][hb][i][j][r] : -INFINITY;
                }
    }
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int row = at.row(ha, i);
            if constexpr (!TG) {
                const int m = m0 + row;
                const int lab = (m < n ? a.ids32[m] : -1) - v0;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) {
                        const int d = lab - at.col(hb, j);
                        if ((unsigned)d < 4u) {
                            const f32x4 v = acc[ha][hb][i][j];
                            a.zt[m] = d == 0 ? v[0] : d == 1 ? v[1] : d == 2 ? v[2] : v[3];
                        }
                    }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) mx = fmaxf(mx, acc[ha][hb][i][j][r]);
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float base = mx == -INFINITY ? 0.0f : mx;   // a row of -inf only: a sum of zeros
            float sm = 0.0f;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sm += exp2_fast((acc[ha][hb][i][j][r] - base) * c2);
            sm += __shfl_xor(sm, 16);
            sm += __shfl_xor(sm, 32);
            if (at.g == 0) {
                red[(0 * T::WGN + at.wn) * T::BM + row] = mx;
                red[(1 * T::WGN + at.wn) * T::BM + row] = sm;
            }
            __builtin_amdgcn_sched_barrier(0);   // one row of fragments at a time keeps the registers within bounds
        }
    __syncthreads();
    for (int row = tid; row < T::BM; row += T::NT) {
        const int m = m0 + row;
        if (m >= n) continue;
        float mx = -INFINITY, sm = 0.0f, sz = 0.0f;
#pragma unroll
        for (int w = 0; w < T::WGN; ++w) mx = fmaxf(mx, red[w * T::BM + row]);
        const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
        for (int w = 0; w < T::WGN; ++w) {
            const float mw = red[w * T::BM + row];
            sm += red[(T::WGN + w) * T::BM + row] * exp2_fast((mw - base) * c2);
            if (smooth) sz += red[(2 * T::WGN + w) * T::BM + row];
        }
        *(float2*)(a.part + ((int64_t)m * a.ntiles + tn) * 2) = make_float2(mx, sm);
        if (smooth) a.sumz[(int64_t)m * a.ntiles + tn] = sz;
    }
}

// Join a row's tiles: one wave per row.
//   lse = max / T + log sum; a row without any finite logit has lse -inf
//   cross entropy: lse - (1 - e) z_y - e / V sum z + c lse^2
//   distillation:  T^2 sum_j p_j (log p_j - (z_j / T - lse))
// The differences from z are taken to the maximum first and the logarithm
// added last: a label that is nearly certain has a small loss, and rounding
// lse before the difference would leave it few digits.
// Rows without a target get 0.  With COMPACT rows are looked up through the
// map (every row's results were cleared by the gather kernel).
template <bool COMPACT>
__global__ __launch_bounds__(256) void loss_finish_kernel(LossArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (c >= (COMPACT ? (int64_t)a.hdr->n : a.M)) return;
    const int64_t m = COMPACT ? (int64_t)a.map[c] : c;
    const float* part = a.part + c * a.ntiles * 2;
    float mx = -INFINITY;
    for (int t = lane; t < a.ntiles; t += 64) mx = fmaxf(mx, part[2 * t]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    const float base = mx == -INFINITY ? 0.0f : mx;
    const float c2 = kLog2e / a.T, it = 1.0f / a.T;
    float sm = 0.0f, sz = 0.0f;
    for (int t = lane; t < a.ntiles; t += 64) {
        sm += part[2 * t + 1] * exp2_fast((part[2 * t] - base) * c2);
        if (a.sumz) sz += a.sumz[c * a.ntiles + t];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        sm += __shfl_xor(sm, o);
        sz += __shfl_xor(sz, o);
    }
    const float ls = kLn2 * __builtin_amdgcn_logf(sm);
    const float lse = fmaf(base, it, ls);
    if (a.labels != nullptr) {
        const int64_t y = a.labels[m];
        const bool live = y >= 0 && y < a.V;
        if (lane == 0) {
            float v = (base - a.zt[c]) + ls + (a.smoothing > 0.0f ? a.smoothing * (a.zt[c] - sz / (float)a.V) : 0.0f) +
                      (a.z_loss != 0.0f ? a.z_loss * lse * lse : 0.0f);
            if (a.zt[c] == -INFINITY) v = INFINITY;   // the label is masked out, whatever else is
            a.loss[m] = live ? v : 0.0f;
            a.lse[m] = live ? lse : 0.0f;
        }
        return;
    }
    // distillation (always compact): the teacher's log-partition over the row
    const float* t = a.teacher + m * a.ldt;
    const int* ids = a.ids32 + c * a.kp;
    float tl;
    if (a.teacher_lse != nullptr) {
        tl = a.teacher_lse[m];
    } else {
        float tm = -INFINITY, ts = 0.0f;
        for (int j = lane; j < a.k; j += 64)
            if (ids[j] >= 0) tm = fmaxf(tm, t[j] * it);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) tm = fmaxf(tm, __shfl_xor(tm, o));
        for (int j = lane; j < a.k; j += 64)
            if (ids[j] >= 0) ts += exp2_fast(kLog2e * (t[j] * it - tm));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) ts += __shfl_xor(ts, o);
        tl = tm + kLn2 * __builtin_amdgcn_logf(ts);
    }
    float kl = 0.0f;
    for (int j = lane; j < a.k; j += 64) {
        if (ids[j] < 0) continue;
        const float lp = t[j] * it - tl;
        const float p = exp2_fast(kLog2e * lp);
        const float z = a.zt[c * a.kp + j];
        if (p != 0.0f) kl += z == -INFINITY ? INFINITY : p * (lp - ((z - base) * it - ls));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) kl += __shfl_xor(kl, o);
    if (lane == 0) {
        a.loss[m] = a.T * a.T * kl;
        a.lse[m] = lse;
    }
}

// ---- rows with a target -----------------------------------------------------

__device__ __forceinline__ bool target_ok(const LossArgs& a, int64_t m, int j) {
    const int64_t id = a.ids[m * a.ldids + j];
    return id >= 0 && id < a.V && a.teacher[m * a.ldt + j] != -INFINITY;
}

// Distillation: a row is live when it names a target of the vocabulary whose
// teacher logit is not -inf.  One wave per row.
__global__ __launch_bounds__(256) void loss_flags_kernel(LossArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= a.M) return;
    bool any = false;
    for (int j = lane; j < a.k; j += 64) any = any || target_ok(a, m, j);
    any = __ballot(any) != 0;
    if (lane == 0) a.live[m] = any ? 1 : 0;
}

// Compact the live rows in order (map), count them, and (backward) find the
// largest |dloss| among them.  One workgroup, so the order is the rows' own.
__global__ __launch_bounds__(1024) void loss_scan_kernel(LossArgs a) {
    __shared__ int wsum[16];
    __shared__ float wmax[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0;
    float g = 0.0f;
    for (int64_t m0 = 0; m0 < a.M; m0 += 1024) {
        const int64_t m = m0 + tid;
        bool on = false;
        if (m < a.M) {
            if (a.labels != nullptr) {
                const int64_t y = a.labels[m];
                on = y >= 0 && y < a.V;
            } else {
                on = a.live[m] != 0;
            }
        }
        const unsigned long long b = __ballot(on);
        if (lane == 0) wsum[wave] = __popcll(b);
        __syncthreads();
        int before = base, all = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            before += w < wave ? wsum[w] : 0;
            all += wsum[w];
        }
        if (on) {
            a.map[before + __popcll(b & ((1ull << lane) - 1ull))] = (int)m;
            if (a.dloss != nullptr) g = fmaxf(g, fabsf(a.dloss[m]));
        }
        base += all;
        __syncthreads();
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) g = fmaxf(g, __shfl_xor(g, o));
    if (lane == 0) wmax[wave] = g;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 0; w < 16; ++w) g = fmaxf(g, wmax[w]);
        a.hdr->n = base;
        a.hdr->gref = (g > 0.0f && g < INFINITY) ? g : 1.0f;
    }
}

// Workgroup b < M: if it is compact row c = b < n, copies X's row together
// with its targets; rows n .. the next multiple of 256 are zeroed.  Then, for
// row m = b of the call, clears what a row without a target gets.
template <bool BWD>
__global__ __launch_bounds__(256) void loss_gather_kernel(LossArgs a) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int c = blockIdx.x;
    const int n = a.hdr->n;
    const int nr = min((n + 255) & ~255, a.Mr);
    // clear the outputs of rows without a target
    if (c < a.M) {
        bool on;
        if (a.labels != nullptr) {
            const int64_t y = a.labels[c];
            on = y >= 0 && y < a.V;
        } else {
            on = a.live[c] != 0;
        }
        if (!on) {
            if constexpr (!BWD) {
                if (tid == 0) a.loss[c] = a.lse[c] = 0.0f;
            } else if (a.dX != nullptr) {
                for (int k = tid; k < a.K; k += 256) {
                    if (a.grad_f32) ((float*)a.dX)[(int64_t)c * a.lddx + k] = 0.0f;
                    else ((uint16_t*)a.dX)[(int64_t)c * a.lddx + k] = 0;
                }
            }
        }
    }
    if (c >= nr) return;
    const int64_t m = c < n ? (int64_t)a.map[c] : -1;
    // the row of X, zero padded to Kp columns
    const uint16_t* src = a.X + m * a.ldx;
    uint16_t* dst = a.Xc + (int64_t)c * a.Kp;
    const bool vec = ((uintptr_t)src & 15) == 0;
    for (int k = tid * 8; k < a.Kp; k += 2048) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (m >= 0) {
            if (vec && k + 8 <= a.K) {
                v = *(const u32x4*)(src + k);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < a.K) v[e >> 1] |= (uint32_t)src[k + e] << (16 * (e & 1));
            }
        }
        *(u32x4*)(dst + k) = v;
    }
    if (tid >= 64) return;
    if (m < 0) {
        if (BWD && lane == 0) a.rows[c] = LossRow{INFINITY, 0.0f, 0.0f, 0.0f};
        for (int j = lane; j < a.kp; j += 64) a.ids32[(int64_t)c * a.kp + j] = -1;
        return;
    }
    float rel = 1.0f, lse2 = 0.0f;
    if constexpr (BWD) {
        rel = a.dloss[m] / a.hdr->gref;
        const float l = a.lse[m];
        // a row without any finite logit: every probability 0
        lse2 = l == -INFINITY ? INFINITY : l * kLog2e;
    }
    if (a.labels != nullptr) {
        if (lane == 0) {
            a.ids32[(int64_t)c * a.kp] = (int)a.labels[m];
            if constexpr (BWD) {
                // everything over (1 - smoothing), so that a label's own
                // weight is exactly the row's share of gref
                const float unit = a.smoothing < 1.0f ? 1.0f - a.smoothing : 1.0f;
                const float cq = a.z_loss != 0.0f ? 1.0f + 2.0f * a.z_loss * a.lse[m] : 1.0f;
                a.rows[c] = LossRow{lse2, rel * cq / unit, rel * a.smoothing / ((float)a.V * unit),
                                    a.smoothing < 1.0f ? rel : 0.0f};
            }
        }
        return;
    }
    int* ids = a.ids32 + (int64_t)c * a.kp;
    const float* t = a.teacher + m * a.ldt;
    for (int j = lane; j < a.kp; j += 64) ids[j] = j < a.k && target_ok(a, m, j) ? (int)a.ids[m * a.ldids + j] : -1;
    if constexpr (BWD) {
        const float it = 1.0f / a.T;
        float tl;
        if (a.teacher_lse != nullptr) {
            tl = a.teacher_lse[m];
        } else {
            float tm = -INFINITY, ts = 0.0f;
            for (int j = lane; j < a.k; j += 64)
                if (target_ok(a, m, j)) tm = fmaxf(tm, t[j] * it);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) tm = fmaxf(tm, __shfl_xor(tm, o));
            for (int j = lane; j < a.k; j += 64)
                if (target_ok(a, m, j)) ts += exp2_fast(kLog2e * (t[j] * it - tm));
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) ts += __shfl_xor(ts, o);
            tl = tm + kLn2 * __builtin_amdgcn_logf(ts);
        }
        // weights; a target named twice keeps its weight at its first place
        float all = 0.0f;
        float* w = a.wts + (int64_t)c * a.kp;
        for (int j = lane; j < a.kp; j += 64) {
            float p = 0.0f;
            int keep = -1;
            if (j < a.k && target_ok(a, m, j)) {
                const int64_t id = a.ids[m * a.ldids + j];
                keep = (int)id;
                all += exp2_fast(kLog2e * (t[j] * it - tl));
                for (int u = 0; u < a.k; ++u) {
                    if (a.ids[m * a.ldids + u] != id || !target_ok(a, m, u)) continue;
                    if (u < j) {
                        keep = -1;
                        break;
                    }
                    p += exp2_fast(kLog2e * (t[u] * it - tl));
                }
            }
            ids[j] = keep;
            w[j] = keep >= 0 ? rel * p : 0.0f;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) all += __shfl_xor(all, o);
        if (lane == 0) a.rows[c] = LossRow{lse2, rel * all, 0.0f, 0.0f};
    }
}

// ---- backward ---------------------------------------------------------------

// One tile of G, the gradient by s over gref (and over the call's unit: the
// label's weight, or T): what multiplies it is put back, in 32 bits, where
// dX, dW and dbias are made.  So the entry of a label that is far from
// learnt is near -1 and survives bf16 nearly exactly, whatever the loss is
// divided by.  G is rounded to bf16 (relative 2^-9 of each entry, to
// nearest) because the products that follow run on bf16 MFMA.
template <class T, bool TG>
__global__ __launch_bounds__(T::NT) void loss_grad_kernel(LossArgs a) {
    constexpr int LDG = T::BN * 2 + 16;   // bytes of a staged row
    constexpr int TAB = TG ? T::HA * (T::BN + 4) * 4 : 0;
    constexpr int STG = T::BM * LDG;
    constexpr int NEED = TAB > STG ? TAB : STG;
    __shared__ __attribute__((aligned(1024))) unsigned char raw[T::LDS > NEED ? T::LDS : NEED];
    lds_t* smem = (lds_t*)raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.hdr->n;
    int tm, tn, rest;
    if (!map_tile(blockIdx.x, (n + T::BM - 1) / T::BM, (a.vn + T::BN - 1) / T::BN, tm, tn, rest, 1)) return;
    const int m0 = tm * T::BM, p0 = tn * T::BN, v0 = a.v0 + p0;
    Acc<T> acc;
    logits_tile<T>(a, m0, v0, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    const int vr = a.V - v0;
    const float c2 = kLog2e / a.T;
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
        if constexpr (TG) {
            // the weights of the targets in these rows, as a table
            float __attribute__((address_space(3)))* tab = (float __attribute__((address_space(3)))*)smem;
            constexpr int LD = T::BN + 4;
            if (ha) __syncthreads();
            for (int e = tid * 4; e < T::HA * LD; e += T::NT * 4)
                *(f32x4 __attribute__((address_space(3)))*)(tab + e) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            __syncthreads();
            constexpr int PER = T::NT / T::HA;
            const int r = tid / PER, m = m0 + ha * T::HA + r;
            if (m < n) {
                const int* ids = a.ids32 + (int64_t)m * a.kp;
                const float* w = a.wts + (int64_t)m * a.kp;
                for (int q = (tid % PER) * 4; q < a.kp; q += PER * 4) {
                    const int4 id = *(const int4*)(ids + q);
                    const int v[4] = {id.x, id.y, id.z, id.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (v[e] >= 0 && (unsigned)(v[e] - v0) < (unsigned)T::BN) tab[r * LD + v[e] - v0] = w[q + e];
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int row = at.row(ha, i);
            const LossRow c = a.rows[m0 + row];   // (rows past the live ones: all entries come out 0)
            int lab = 0;
            if constexpr (!TG) lab = a.ids32[m0 + row] - v0;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const int col = at.col(hb, j);
                    const f32x4 z = acc[ha][hb][i][j];
                    f32x4 v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = fmaf(exp2_fast(fmaf(z[r], c2, -c.lse2)), c.rq, -c.ru);
                    if constexpr (TG) {
                        v -= *(const f32x4 __attribute__((address_space(3)))*)(
                            (float __attribute__((address_space(3)))*)smem + (row - ha * T::HA) * (T::BN + 4) + col);
                    } else {
                        const int d = lab - col;
                        if ((unsigned)d < 4u) {   // (rarely taken by any lane)
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] -= d == r ? c.rp : 0.0f;
                        }
                    }
                    if (a.cap > 0.0f) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] *= fmaf(-z[r] * inv_cap, z[r] * inv_cap, 1.0f);
                    }
                    acc[ha][hb][i][j] = v;
                }
            __builtin_amdgcn_sched_barrier(0);   // one row of fragments at a time keeps the registers within bounds
        }
    }
    if (vr < T::BN) {   // columns past the vocabulary
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = at.col(hb, j) + r < vr;
#pragma unroll
                    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                        for (int i = 0; i < T::FM; ++i) acc[ha][hb][i][j][r] = in ? acc[ha][hb][i][j][r] : 0.0f;
                }
    }
    if constexpr (TG) __syncthreads();
    if (a.dbp != nullptr) {
        // column sums over the tile's rows: a lane's rows, the 16 lanes of a
        // group, then (through LDS) the waves that share the columns
        float __attribute__((address_space(3)))* red = (float __attribute__((address_space(3)))*)smem;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int i = 0; i < T::FM; ++i) t += acc[ha][hb][i][j];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) t[r] += __shfl_xor(t[r], o);
                    if (at.s == 0) red[at.wm * T::BN + at.col(hb, j) + r] = t[r];
                }
            }
        __syncthreads();
        for (int c = tid; c < T::BN; c += T::NT) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < T::WGM; ++w) t += red[w * T::BN + c];
            a.dbp[(int64_t)tm * a.Vp + p0 + c] = t;
        }
        __syncthreads();
    }
    // bf16, through LDS, so that the stores write whole row segments
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const f32x4 v = acc[ha][hb][i][j];
                    const u32x2 w = {(uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16),
                                     (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16)};
                    *(u32x2 __attribute__((address_space(3)))*)(smem + at.row(ha, i) * LDG + at.col(hb, j) * 2) = w;
                }
    __syncthreads();
    uint16_t* G = a.G + (int64_t)m0 * a.Vp + p0;
    constexpr int CPR = T::BN / 8;
    for (int p = tid; p < T::BM * CPR; p += T::NT) {
        const int r = p / CPR, c = p % CPR;
        *(u32x4*)(G + (int64_t)r * a.Vp + c * 8) =
            *(const u32x4 __attribute__((address_space(3)))*)(smem + r * LDG + c * 16);
    }
}

// How dX's product over a piece is cut: its tiles are few where the live rows
// or the features are, so the vocabulary steps are split over workgroups, each
// split with a partial dX of its own.  Counted in steps of a workgroup, with
// what a tile costs besides its steps (filling and draining the pipeline,
// writing and summing the partial) taken as 8 of them: the cheapest of the
// whole numbers of splits that give at most two rounds of workgroups.
struct DxCut {
    int tm, tk, splits;
};
__device__ __forceinline__ DxCut dx_cut(int n, int K, int Vp, int tile, int slots) {
    DxCut c;
    c.tm = (n + tile - 1) / tile;
    c.tk = (K + tile - 1) / tile;
    const int tiles = max(1, c.tm * c.tk), all = Vp >> 6;
    c.splits = 1;
    int best = ((tiles + slots - 1) / slots) * (all + 8);
    for (int s = 2; s * tiles <= 2 * slots && s * 4 <= all; ++s) {
        const int cost = ((tiles * s + slots - 1) / slots) * ((all + s - 1) / s + 8);
        if (cost < best) {
            best = cost;
            c.splits = s;
        }
    }
    return c;
}

// dX partials: [split] (+)= G(piece) . W(piece), a split's share of the
// vocabulary steps.
template <class T>
__global__ __launch_bounds__(T::NT) void loss_dx_kernel(LossArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[T::LDS];
    lds_t* smem = (lds_t*)raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.hdr->n;
    const DxCut cut = dx_cut(n, a.K, a.Vp, T::BM, a.slots);
    int tm, tn, split;
    if (!map_tile(blockIdx.x, cut.tm, cut.tk, tm, tn, split, cut.splits)) return;
    const int m0 = tm * T::BM, k0 = tn * T::BN;
    const int all = (a.vn + 63) >> 6;
    const int per = (all + cut.splits - 1) / cut.splits;
    const int s0 = min(split * per, all), steps = min(per, all - s0);
    Operand<T::HA, false, T::IA, T::NW> A;
    Operand<T::HB, true, T::IB, T::NW> B;
    A.init(a.G + (int64_t)m0 * a.Vp + s0 * 64, a.Vp, T::BM, steps, 0, wave, lane);
    B.init(a.W + (int64_t)(a.v0 + s0 * 64) * a.ldw + k0, a.ldw, a.Kw - k0, steps,
           s0 + steps == all ? a.vn & 63 : 0, wave, lane);
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    float* P = a.dxp + ((int64_t)split * cut.tm * T::BM + m0) * a.Kp + k0;
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const int col = at.col(hb, j);
                    if (k0 + col >= a.Kp) continue;
                    f32x4* p = (f32x4*)(P + (int64_t)at.row(ha, i) * a.Kp + col);
                    *p = a.first ? acc[ha][hb][i][j] : *p + acc[ha][hb][i][j];
                }
}

// dX = gref unit scale (sum of the partials), in the rows' own places.
__global__ __launch_bounds__(256) void loss_dx_finish_kernel(LossArgs a, float mul, int tile) {
    const int c = blockIdx.x, n = a.hdr->n;
    if (c >= n) return;
    const DxCut cut = dx_cut(n, a.K, a.Vp, tile, a.slots);
    const int64_t m = a.map[c];
    const float f = mul * a.hdr->gref;
    const int64_t sp = (int64_t)cut.tm * tile * a.Kp;
    for (int k = threadIdx.x * 4; k < a.K; k += 1024) {
        const float* p = a.dxp + (int64_t)c * a.Kp + k;
        f32x4 v = *(const f32x4*)p;
        for (int s = 1; s < cut.splits; ++s) v += *(const f32x4*)(p + s * sp);
        v *= f;
        if (a.grad_f32) {
            float* d = (float*)a.dX + m * a.lddx + k;
            if (k + 4 <= a.K && ((uintptr_t)d & 15) == 0) *(f32x4*)d = v;
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (k + r < a.K) d[r] = v[r];
        } else {
            uint16_t* d = (uint16_t*)a.dX + m * a.lddx + k;
            if (k + 4 <= a.K && ((uintptr_t)d & 7) == 0)
                *(u32x2*)d = u32x2{(uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16),
                                   (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16)};
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (k + r < a.K) d[r] = f32_to_bf16(v[r]);
        }
    }
}

// dW of a piece: gref unit scale G^T . X.
template <class T>
__global__ __launch_bounds__(T::NT) void loss_dw_kernel(LossArgs a, float mul) {
    constexpr int LDG = T::BN * 2 + 16;
    constexpr int NEED = T::BM * LDG;
    __shared__ __attribute__((aligned(1024))) unsigned char raw[T::LDS > NEED ? T::LDS : NEED];
    lds_t* smem = (lds_t*)raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.hdr->n;
    int tm, tn, rest;
    if (!map_tile(blockIdx.x, (a.vn + T::BM - 1) / T::BM, (a.K + T::BN - 1) / T::BN, tm, tn, rest, 1)) return;
    const int p0 = tm * T::BM, k0 = tn * T::BN;
    const int steps = (n + 63) >> 6;
    Operand<T::HA, true, T::IA, T::NW> A;
    Operand<T::HB, true, T::IB, T::NW> B;
    A.init(a.G + p0, a.Vp, T::BM, steps, 0, wave, lane);
    B.init(a.Xc + k0, a.Kp, a.Kp - k0, steps, 0, wave, lane);
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    const float f = mul * a.hdr->gref;
    const int vr = a.vn - p0, kr = a.K - k0;
    if (a.grad_f32) {
        float* D = (float*)a.dW + (int64_t)(a.v0 + p0) * a.lddw + k0;
        const bool vec = ((uintptr_t)D & 15) == 0 && a.lddw % 4 == 0;
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) {
                        const int row = at.row(ha, i), col = at.col(hb, j);
                        if (row >= vr) continue;
                        const f32x4 v = acc[ha][hb][i][j] * f;
                        float* p = D + (int64_t)row * a.lddw + col;
                        if (vec && col + 4 <= kr) *(f32x4*)p = v;
                        else
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (col + r < kr) p[r] = v[r];
                    }
        return;
    }
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const f32x4 v = acc[ha][hb][i][j] * f;
                    const u32x2 w = {(uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16),
                                     (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16)};
                    *(u32x2 __attribute__((address_space(3)))*)(smem + at.row(ha, i) * LDG + at.col(hb, j) * 2) = w;
                }
    __syncthreads();
    uint16_t* D = (uint16_t*)a.dW + (int64_t)(a.v0 + p0) * a.lddw + k0;
    const bool vec = ((uintptr_t)D & 15) == 0 && a.lddw % 8 == 0;
    constexpr int CPR = T::BN / 8;
    for (int p = tid; p < T::BM * CPR; p += T::NT) {
        const int r = p / CPR, c = (p % CPR) * 8;
        if (r >= vr || c >= kr) continue;
        const u32x4 w = *(const u32x4 __attribute__((address_space(3)))*)(smem + r * LDG + c * 2);
        uint16_t* d = D + (int64_t)r * a.lddw + c;
        if (vec && c + 8 <= kr) *(u32x4*)d = w;
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < kr) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// dbias of a piece: gref unit (sum over the row tiles, in order).
__global__ __launch_bounds__(256) void loss_dbias_kernel(LossArgs a, float mul, int row_tile) {
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= a.vn) return;
    const int tiles = (a.hdr->n + row_tile - 1) / row_tile;
    float t = 0.0f;
    for (int i = 0; i < tiles; ++i) t += a.dbp[(int64_t)i * a.Vp + p];
    a.dbias[a.v0 + p] = t * (mul * a.hdr->gref);
}

template <bool AT, bool BT>
using L256 = LTile<2, 4, 4, 2, AT, BT>;
template <bool AT, bool BT>
using L128 = LTile<2, 2, 2, 2, AT, BT>;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What G is over besides gref: T (whose square the loss carries, over one
// temperature from its derivative), or the label's own weight.
float unit_of(const LossArgs& a) {
    return a.labels == nullptr ? a.T : a.smoothing < 1.0f ? 1.0f - a.smoothing : 1.0f;
}

}  // namespace

int loss_tile_rows(int tile) { return tile == LT_256 ? 256 : 128; }

hipError_t launch_loss_flags(const LossArgs& a, hipStream_t st) {
    return launch_kernel(loss_flags_kernel, dim3((unsigned)up(a.M, 4)), dim3(256), st, a);
}

hipError_t launch_loss_scan(const LossArgs& a, hipStream_t st) {
    return launch_kernel(loss_scan_kernel, dim3(1), dim3(1024), st, a);
}

hipError_t launch_loss_gather(const LossArgs& a, bool backward, hipStream_t st) {
    const dim3 grid((unsigned)a.Mr);
    return backward ? launch_kernel(loss_gather_kernel<true>, grid, dim3(256), st, a)
                    : launch_kernel(loss_gather_kernel<false>, grid, dim3(256), st, a);
}

hipError_t launch_loss_forward(const LossArgs& a, int tile, hipStream_t st) {
    const bool tg = a.labels == nullptr;
    if (tile == LT_256) {
        using T = L256<false, false>;
        const dim3 grid((unsigned)(up(a.M, T::BM) * a.ntiles));
        return tg ? launch_kernel(loss_forward_kernel<T, true>, grid, dim3(T::NT), st, a)
                  : launch_kernel(loss_forward_kernel<T, false>, grid, dim3(T::NT), st, a);
    }
    using T = L128<false, false>;
    const dim3 grid((unsigned)(up(a.M, T::BM) * a.ntiles));
    return tg ? launch_kernel(loss_forward_kernel<T, true>, grid, dim3(T::NT), st, a)
              : launch_kernel(loss_forward_kernel<T, false>, grid, dim3(T::NT), st, a);
}

hipError_t launch_loss_finish(const LossArgs& a, bool compact, hipStream_t st) {
    const dim3 grid((unsigned)up(a.M, 4));
    return compact ? launch_kernel(loss_finish_kernel<true>, grid, dim3(256), st, a)
                   : launch_kernel(loss_finish_kernel<false>, grid, dim3(256), st, a);
}

hipError_t launch_loss_grad(const LossArgs& a, int tile, hipStream_t st) {
    const bool tg = a.labels == nullptr;
    if (tile == LT_256) {
        using T = L256<false, false>;
        const dim3 grid((unsigned)(up(a.M, T::BM) * up(a.vn, T::BN)));
        return tg ? launch_kernel(loss_grad_kernel<T, true>, grid, dim3(T::NT), st, a)
                  : launch_kernel(loss_grad_kernel<T, false>, grid, dim3(T::NT), st, a);
    }
    using T = L128<false, false>;
    const dim3 grid((unsigned)(up(a.M, T::BM) * up(a.vn, T::BN)));
    return tg ? launch_kernel(loss_grad_kernel<T, true>, grid, dim3(T::NT), st, a)
              : launch_kernel(loss_grad_kernel<T, false>, grid, dim3(T::NT), st, a);
}

hipError_t launch_loss_dx(const LossArgs& a, int tile, hipStream_t st) {
    const int b = loss_tile_rows(tile);
    // (at most two rounds, or one workgroup a tile)
    const dim3 grid((unsigned)std::max<int64_t>(up(a.M, b) * up(a.K, b), 2 * a.slots));
    if (tile == LT_256) {
        using T = L256<false, true>;
        return launch_kernel(loss_dx_kernel<T>, grid, dim3(T::NT), st, a);
    }
    using T = L128<false, true>;
    return launch_kernel(loss_dx_kernel<T>, grid, dim3(T::NT), st, a);
}

hipError_t launch_loss_dx_finish(const LossArgs& a, int tile, hipStream_t st) {
    return launch_kernel(loss_dx_finish_kernel, dim3((unsigned)a.M), dim3(256), st, a, unit_of(a) * a.scale,
                         loss_tile_rows(tile));
}

hipError_t launch_loss_dw(const LossArgs& a, int tile, hipStream_t st) {
    const int b = loss_tile_rows(tile);
    const dim3 grid((unsigned)(up(a.vn, b) * up(a.K, b)));
    const float mul = unit_of(a) * a.scale;
    if (tile == LT_256) {
        using T = L256<true, true>;
        return launch_kernel(loss_dw_kernel<T>, grid, dim3(T::NT), st, a, mul);
    }
    using T = L128<true, true>;
    return launch_kernel(loss_dw_kernel<T>, grid, dim3(T::NT), st, a, mul);
}

hipError_t launch_loss_dbias(const LossArgs& a, int row_tile, hipStream_t st) {
    return launch_kernel(loss_dbias_kernel, dim3((unsigned)up(a.vn, 256)), dim3(256), st, a, unit_of(a), row_tile);
}

}  // namespace mkp

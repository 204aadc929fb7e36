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
#include "load8.h"

#include <hip/hip_ext.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mkp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
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

// A product rounded by itself, never part of a fused multiply-add.
__device__ __forceinline__ float mul_rn(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

// The base-2 value that the row's (lane's, tile's) exponentials are taken
// relative to, from its largest u; 0 where even that is -inf in base 2, so
// that every exponential there is 0 and none is NaN.
__device__ __forceinline__ float stat_base(float umax, float s2) {
    const float b = mul_rn(umax, s2);
    return b == -INFINITY ? 0.0f : b;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Round to nearest even, NaN kept a NaN: the conversion instruction.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// tanh: x (1 + x^2 p(x^2)), p fitted to the least largest relative error (0.25 of
// U = 2^-24) below 1/2, where 1 - 2/(1 + e^2|x|) would cancel; that form elsewhere.
// Relative error at most 2.2 U below 1/2 and 6.5 U above (1.7 and 3.4 found over
// 400000 points); a longer p instead costs 7 % of 4096 x 30522 x 768 forward.
// slope: 1 - tanh^2 = 4 r (1 - r), r = 1/(1 + e^2|x|) <= 1/2, without a difference
// of nearly equal values however close to 1 the tanh is.
__device__ __forceinline__ float tanh_fast(float x, float& slope) {
    const float x2 = x * x;
    const float p = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 0.017241468653082848f, -0.05304548516869545f),
                                               0.13325878977775574f), -0.333331435918808f), 1.0f);
    const float e = exp2_fast(2.0f * kLog2e * fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float f = copysignf(fmaf(-2.0f, r, 1.0f), x);
    slope = 4.0f * fmaf(-r, r, r);
    return fabsf(x) < 0.5f ? p : f;
}
__device__ __forceinline__ float tanh_fast(float x) {
    float slope;
    return tanh_fast(x, slope);
}

// At the head of a branch that few calls or lanes take: keeps the compiler
// from computing the branch's work ahead of it, for everyone.
__device__ __forceinline__ void rarely() { asm volatile("; rarely taken"); }

// Sum over the 16 lanes of a row (lanes 16 r .. 16 r + 15), by rotations
// within it.
template <int N>
__device__ __forceinline__ float row_rotate(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float v) {
    v += row_rotate<8>(v);
    v += row_rotate<4>(v);
    v += row_rotate<2>(v);
    return v + row_rotate<1>(v);
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

// Chunk swizzle of a 128-byte row (eight 16-byte chunks).  A 128-bit read of
// 64 lanes goes in four passes of 16 lanes, lanes 0-3, 12-15 and 20-27 of each
// 32 in one and the others in the next; with lane 16 g + s on row s, chunk c +
// g, the rows' low three bits spread each pass over all 16 bank windows
// (measured: no conflict cycles; with the third bit folded in as well, half of
// all LDS cycles were).
__device__ __forceinline__ int swz_row(int row) { return row & 7; }

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
// The same from an address of each lane's own.
__device__ __forceinline__ void dma16_at(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand of a tile: where its halves' loads come from.
//   rows (not TR): `lim` valid rows of the tile; a last step of fewer than 64
//     columns (`tail` > 0 of them) takes the missing ones from `zeros`, 16 bytes
//     of them, as does the other operand: an infinity times 0 would be NaN
//   columns (TR): `lim` valid columns of the tile; a last step of fewer than
//     64 rows repeats its last row, where the other operand holds zeros (an
//     infinity in that row leaves no finite dX in any case)
// Both need `lim` and `tail` to be multiples of 8 columns.
template <int H, bool TR, int I, int NW>
struct Operand {
    const char* base;      // tile origin, step 0
    int64_t step_bytes;
    int64_t ld;
    uint32_t off[2][I];
    int lim, steps, tail;
    const uint16_t* zeros;

    // (most: TR, the rows there are)
    __device__ __forceinline__ uint32_t offset(int h, int i, int wave, int lane, int most) const {
        int r, c;
        half_slot<H, TR>((i * NW + wave) * 64 + lane, r, c);
        if constexpr (!TR) {
            r = min(h * H + r, lim - 1);
        } else {
            r = min(r, most - 1);
            c = min(h * H + c, lim - 8);
        }
        return (uint32_t)((r * ld + c) * 2);
    }
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int lim_, int steps_, int tail_, int wave,
                                         int lane, const uint16_t* zeros_ = nullptr) {
        base = (const char*)p;
        zeros = zeros_;
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
            for (int i = 0; i < I; ++i) {
                if constexpr (TR) {
                    dma16(b, offset(h, i, wave, lane, tail), lds + (i * NW + wave) * 1024);
                } else {
                    int r, c;
                    half_slot<H, TR>((i * NW + wave) * 64 + lane, r, c);
                    dma16_at(c < tail ? b + off[h][i] : (const char*)zeros, lds + (i * NW + wave) * 1024);
                }
            }
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
// Measured (256 x 256 tile, one per CU): 1.43 us a step, 1500 TFLOP/s over the
// device, whichever way the operands are read; the waves' MFMAs fill 76-78 %
// of the cycles at the 1.6-1.9 GHz that the card's power leaves.  Two phases
// of 32 MFMAs ran out of registers (5-25 % slower), one stage a step ahead
// with all waves in step took 1.7 us.
template <class T>
__device__ __forceinline__ void main_loop(const Operand<T::HA, T::AT, T::IA, T::NW>& A,
                                          const Operand<T::HB, T::BT, T::IB, T::NW>& B, int steps, lds_t* smem,
                                          int wave, int lane, Acc<T>& acc) {
    constexpr bool PP = T::NW == 8;
    constexpr int IA = T::IA, IB = T::IB;
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
        // loads that may still be in flight at each phase's end: six halves
        // (three of each operand), fewer where nothing more is issued
        constexpr int W0 = LEFT == 2 ? 3 * IA + 3 * IB : LEFT == 1 ? 3 * IA + 2 * IB : IA;
        constexpr int W1 = LEFT == 2 ? 3 * IA + 3 * IB : LEFT == 1 ? 2 * IA + 2 * IB : 0;
        constexpr int W2 = LEFT == 2 ? 3 * IA + 3 * IB : LEFT == 1 ? 2 * IA + IB : 0;
        constexpr int W3 = LEFT == 2 ? 3 * IA + 3 * IB : LEFT == 1 ? IA + IB : 0;
        read_a(0, s);
        if constexpr (LEFT == 2) issue_b(0, s + 2);
        phase_barrier<W0>();
        multiply(0, 0);
        read_b(1, s);
        if constexpr (LEFT == 2) issue_a(0, s + 2);
        phase_barrier<W1>();
        multiply(0, 1);
        read_a(1, s);
        if constexpr (LEFT == 2) issue_b(1, s + 2);
        phase_barrier<W2>();
        multiply(1, 0);
        if constexpr (LEFT >= 1) read_b(0, s + 1);
        if constexpr (LEFT == 2) issue_a(1, s + 2);
        phase_barrier<W3>();
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
    if (steps > 1) phase_barrier<3 * IA + 3 * IB>();
    else phase_barrier<IA + IB>();
    read_b(0, 0);
    phase_barrier<3 * IA + 3 * IB>();
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
__device__ __forceinline__ int xcd_run(int bid, int G) {
    const int q = G >> 3, r = G & 7, x = bid & 7;
    return x * q + min(x, r) + (bid >> 3);
}
__device__ __forceinline__ void tile_at(int tile, int tm_n, int tn_n, int& tm, int& tn) {
    constexpr int GROUP = 8;
    const int per = GROUP * tn_n, g = tile / per, first = g * GROUP;
    const int gsz = min(tm_n - first, GROUP), in = tile - g * per;
    tm = first + in % gsz;
    tn = in / gsz;
}
__device__ __forceinline__ bool map_tile(int bid, int tm_n, int tn_n, int& tm, int& tn, int& rest, int parts) {
    const int T = tm_n * tn_n, G = T * parts;
    if (bid >= G) return false;
    const int L = xcd_run(bid, G);
    rest = L / T;
    tile_at(L - rest * T, tm_n, tn_n, tm, tn);
    return true;
}

// The logit tiles of a launch.  Tiles of one size run in rounds of `slots`
// workgroups; when the last round would be at most half full, its tiles are
// halved (two workgroups of half the rows each), which takes about 0.6 of a
// whole tile's round instead of one (256 workgroups at 768 features: 19.8 us
// of halves, 33.6 of whole tiles).  half: -1 a whole tile, else which half.
__device__ __forceinline__ bool map_rounds(int bid, int tm_n, int tn_n, int slots, bool halves, int& tm, int& tn,
                                           int& half) {
    const int T = tm_n * tn_n, full = T / slots * slots, r = T - full;
    half = -1;
    if (!halves || 2 * r > slots) {
        if (bid >= T) return false;
        tile_at(xcd_run(bid, T), tm_n, tn_n, tm, tn);
        return true;
    }
    if (bid < full) {
        tile_at(xcd_run(bid, full), tm_n, tn_n, tm, tn);
        return true;
    }
    bid -= full;
    if (bid >= 2 * r) return false;
    half = bid >= r ? 1 : 0;
    tile_at(full + bid - half * r, tm_n, tn_n, tm, tn);
    return true;
}

// ---- the logits of a tile ---------------------------------------------------

// A lane's 16 bias values (0 without a bias).
template <class T>
struct BiasRegs {
    f32x4 b[2][T::FN];
    __device__ __forceinline__ void read(const LossArgs& a, const Place<T>& at, int v_tile) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    b[hb][j][r] = a.bias != nullptr ? a.bias[min(v_tile + at.col(hb, j) + r, a.V - 1)] : 0.0f;
    }
};

// One row of fragments: acc (x.w) -> s in place.
template <class T>
__device__ __forceinline__ void row_affine(const LossArgs& a, const BiasRegs<T>& bias, Acc<T>& acc, int ha, int i) {
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[ha][hb][i][j][r] = fmaf(a.scale, acc[ha][hb][i][j][r], bias.b[hb][j][r]);
}

// One row of fragments: acc (x.w) -> z in place.
template <class T>
__device__ __forceinline__ void row_logits(const LossArgs& a, const BiasRegs<T>& bias, float inv_cap, Acc<T>& acc, int ha,
                                           int i) {
    row_affine<T>(a, bias, acc, ha, i);
    if (a.cap > 0.0f) {
        rarely();
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[ha][hb][i][j][r] = a.cap * tanh_fast(acc[ha][hb][i][j][r] * inv_cap);
    }
}

// The tile's product X . W^T, from the compacted rows or (direct: few rows,
// nothing dropped) the caller's.
template <class T>
__device__ __forceinline__ void logits_tile(const LossArgs& a, int m0, int v_tile, int n, lds_t* smem, int wave, int lane,
                                            Acc<T>& acc) {
    const int steps = (a.Kw + 63) >> 6;
    const uint16_t* X = a.direct ? a.X : a.Xc;
    const int64_t ldx = a.direct ? a.ldx : a.Kp;
    Operand<T::HA, false, T::IA, T::NW> A;
    Operand<T::HB, false, T::IB, T::NW> B;
    A.init(X + (int64_t)m0 * ldx, ldx, n - m0, steps, 0, wave, lane);
    // (K not a multiple of 64: the compacted rows end in zeros, at least eight)
    B.init(a.W + (int64_t)v_tile * a.ldw, a.ldw, a.V - v_tile, steps, a.Kw & 63, wave, lane, a.Xc + a.Kp - 8);
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
}

// Compact row m's label (forward: the caller's where nothing is compacted).
__device__ __forceinline__ int row_label(const LossArgs& a, int m, int n) {
    if (m >= n) return -1;
    if (!a.direct) return a.ids32[m];
    const int64_t y = a.labels[m];
    return y >= 0 && y < a.V ? (int)y : -1;
}

// ---- forward ----------------------------------------------------------------

// Statistics of one logit tile.  TG: the targets' values are picked from the
// tile staged in LDS, half its rows at a time (several targets a row); else
// each lane compares its columns with the row's one label.
//
// Kept are u = x.w with y = u s2 the logit in base 2, or, where a bias, a cap
// or a scale below 0 asks for it, u = z (a.plain tells which): per row the
// largest u and the sum of 2^(y - fl(umax s2)).  The subtraction is part of
// the fused multiply, so an exponent keeps its digits, and what rounding umax
// s2 loses is put back where the tiles are joined.  A lane reduces its own 16
// values of a row; the 4 lanes and the waves that share the row meet in LDS.
// Bound by the product at many K steps (4096 x 32000 x 4096: 750 us, 1430
// TFLOP/s), at few by this epilogue too, about 6 us a tile, most of it the
// 65536 exponentials (1024 x 16384 x 768, one tile a CU: 29.6 us).
template <class T, bool TG>
constexpr int forward_lds() {
    const int tab = TG ? T::HA * (T::BN + 4) * 4 : 0, red = T::BM * (8 * T::WGN + 2) * 4;
    return std::max(T::LDS, std::max(tab, red));
}
template <class T, bool TG>
__device__ __forceinline__ void forward_tile(const LossArgs& a, int n, int m0, int tn, lds_t* smem, int wave, int lane) {
    constexpr int PARTS = 4 * T::WGN, LDP = 2 * PARTS + 2;   // floats per row
    const int tid = wave * 64 + lane, v0 = tn * T::BN;
    const Place<T> at(wave, lane);
    int labs[2][T::FM];
    if constexpr (!TG) {   // (read ahead of the product, whose loop hides it)
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) labs[ha][i] = row_label(a, m0 + at.row(ha, i), n) - v0 - at.wn * T::FN * 16;
    }
    Acc<T> acc;
    logits_tile<T>(a, m0, v0, n, smem, wave, lane, acc);
    const int vr = a.V - v0;   // valid columns
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
    BiasRegs<T> bias;
    if (!a.plain) bias.read(a, at, v0);
    if constexpr (TG) {
        float __attribute__((address_space(3)))* tab = (float __attribute__((address_space(3)))*)smem;
        constexpr int LD = T::BN + 4;
        // a row's first targets, AHEAD fours for each of its PER threads, are
        // read while the half is staged (-1 past the last)
        constexpr int PER = T::NT / T::HA, AHEAD = 16 / PER;
        int4 tg[AHEAD];
#pragma unroll
        for (int ha = 0; ha < 2; ++ha) {
            const int r = tid / PER, m = m0 + ha * T::HA + r;
            if (!a.direct) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int q = (tid % PER + PER * i) * 4;
                    tg[i] = m < n && q < a.kp ? *(const int4*)(a.ids32 + (int64_t)m * a.kp + q) : int4{-1, -1, -1, -1};
                }
            }
            if (ha) __syncthreads();
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                if (!a.plain) row_logits<T>(a, bias, inv_cap, acc, ha, i);
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
                        *(f32x4 __attribute__((address_space(3)))*)(tab + (at.row(ha, i) - ha * T::HA) * LD +
                                                                    at.col(hb, j)) = acc[ha][hb][i][j];
                __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
            auto pick = [&](int q, int id) {
                if ((unsigned)(id - v0) < (unsigned)T::BN) a.zt[(int64_t)m * a.kp + q] = tab[r * LD + id - v0];
            };
            if (m < n && a.direct) {
                const int64_t* ids = a.ids + (int64_t)m * a.ldids;
                for (int q = tid % PER; q < a.k; q += PER)
                    if (ids[q] >= 0 && ids[q] < a.V) pick(q, (int)ids[q]);
            } else if (m < n) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int q = (tid % PER + PER * i) * 4;
                    pick(q, tg[i].x);
                    pick(q + 1, tg[i].y);
                    pick(q + 2, tg[i].z);
                    pick(q + 3, tg[i].w);
                }
                for (int q = (tid % PER + PER * AHEAD) * 4; q < a.kp; q += PER * 4) {
                    const int4 id = *(const int4*)(a.ids32 + (int64_t)m * a.kp + q);
                    pick(q, id.x);
                    pick(q + 1, id.y);
                    pick(q + 2, id.z);
                    pick(q + 3, id.w);
                }
            }
        }
        __syncthreads();
    }
    const float s2 = a.s2;
    const bool smooth = a.sumz != nullptr;
    float __attribute__((address_space(3)))* red = (float __attribute__((address_space(3)))*)smem;
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int row = at.row(ha, i);
            if constexpr (!TG) {
                if (!a.plain) row_logits<T>(a, bias, inv_cap, acc, ha, i);
                // (the wave's columns are two runs of FN * 16)
                const unsigned lab = (unsigned)labs[ha][i];
                if (lab < (unsigned)T::BN && (lab & (T::HB - 1)) < (unsigned)(T::FN * 16)) {
                    rarely();
                    float u = 0.0f;
                    bool mine = false;
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int j = 0; j < T::FN; ++j)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const bool is = lab == (unsigned)(hb * T::HB + j * 16 + at.g * 4 + r);
                                u = is ? acc[ha][hb][i][j][r] : u;
                                mine |= is;
                            }
                    if (mine) a.zt[m0 + row] = u;
                }
            }
            if (smooth) {
                rarely();
                float sz = 0.0f;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) sz += at.col(hb, j) + r < vr ? acc[ha][hb][i][j][r] : 0.0f;
                sz += __shfl_xor(sz, 16);
                sz += __shfl_xor(sz, 32);
                // (one value a row and wave, kept apart from the partials below)
                if (at.g == 0 && m0 + row < n)
                    a.sumz[((int64_t)(m0 + row) * a.ntiles + tn) * T::WGN + at.wn] = sz;
            }
            if (vr < T::BN) {
                rarely();
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[ha][hb][i][j][r] = at.col(hb, j) + r < vr ? acc[ha][hb][i][j][r] : -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) mx = fmaxf(mx, acc[ha][hb][i][j][r]);
            const float base = stat_base(mx, s2);
            f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) part[r] += exp2_fast(fmaf(acc[ha][hb][i][j][r], s2, -base));
            const float sm = (part[0] + part[1]) + (part[2] + part[3]);
            *(f32x2 __attribute__((address_space(3)))*)(red + row * LDP + (at.wn * 4 + at.g) * 2) = f32x2{mx, sm};
            __builtin_amdgcn_sched_barrier(0);   // one row of fragments at a time keeps the registers within bounds
        }
    __syncthreads();
    for (int row = tid; row < T::BM; row += T::NT) {
        const int m = m0 + row;
        if (m >= n) continue;
        f32x2 p[PARTS];
        float mx = -INFINITY, sm = 0.0f;
#pragma unroll
        for (int w = 0; w < PARTS; ++w) {
            p[w] = *(const f32x2 __attribute__((address_space(3)))*)(red + row * LDP + w * 2);
            mx = fmaxf(mx, p[w].x);
        }
        const float base = stat_base(mx, s2);
#pragma unroll
        for (int w = 0; w < PARTS; ++w) sm += p[w].y * exp2_fast(mul_rn(p[w].x, s2) - base);
        *(float2*)(a.part + ((int64_t)m * a.ntiles + tn) * 2) = make_float2(mx, sm);
    }
}

// (At least two waves a SIMD: LossArgs::slots counts two workgroups of a 128 x
// 128 tile on a CU.  Without that bound the distillation gradient took 269
// registers and ran one: 99 us a step of 160 x 30522 x 768, 91 with it.)
template <class T, class H, bool TG>
__global__ __launch_bounds__(T::NT, 2) void loss_forward_kernel(LossArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[std::max(forward_lds<T, TG>(), forward_lds<H, TG>())];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = a.direct ? (int)a.M : a.hdr->n;
    int tm, tn, half;
    if (!map_rounds(blockIdx.x, (n + T::BM - 1) / T::BM, a.ntiles, a.slots, T::BM > H::BM, tm, tn, half)) return;
    if (half < 0) {
        forward_tile<T, TG>(a, n, tm * T::BM, tn, (lds_t*)raw, wave, lane);
    } else if (tm * T::BM + half * H::BM < n) {
        forward_tile<H, TG>(a, n, tm * T::BM + half * H::BM, tn, (lds_t*)raw, wave, lane);
    }
}

// Forward for few rows: the weight streams past them, so what counts is how
// many of its bytes are on their way.  One workgroup per CU takes a run of
// the vocabulary, in blocks of at most 64 rows of W, and walks (block, K step)
// as one sequence through a ring of S stages of BK columns, so the loads of a
// block's first steps are under way while the block before is finished.  Each
// wave multiplies 16 rows of W with the FM * 16 rows of X and keeps every
// row's running maximum and sum over the blocks; a workgroup leaves one
// partial per row.  Long K steps: 512 contiguous bytes of a row of W at a time.
// Measured, with cold weights (and on 128 x 128 tiles, a quarter of the bytes
// in flight): 8 x 32000 x 4096 in 49 us (60), 32 rows 50 (60), 8 x 30522 x 768
// 10.2 (12.6), 32 rows 11.6 (13.7); a form for 33 to 64 rows, its ring of 128
// columns, took 67 (61), 17 (14) at 33 rows and was dropped.  24 x 128256 x
// 4096: 175 us, 6.0 TB/s.
template <int FM_, int BK_, int S_>
struct Stream {
    static constexpr int FM = FM_, BK = BK_, S = S_;
    static constexpr int NW = 4, NT = 256, BN = 64;
    static constexpr int CPR = BK / 8;                       // chunks per LDS row
    static constexpr int W_BYTES = BN * BK * 2, X_BYTES = FM * 16 * BK * 2, STAGE = W_BYTES + X_BYTES;
    static constexpr int IW = W_BYTES / 1024 / NW, IX = X_BYTES / 1024 / NW;
    static constexpr int LD = BN + 4;                        // staged logits
    static constexpr int LDS = S * STAGE;
    static_assert(X_BYTES % (1024 * NW) == 0 && LDS <= 160 * 1024 && (S - 1) * (IW + IX) <= 63, "stages");
};

template <class T, bool TG>
__global__ __launch_bounds__(T::NT) void loss_stream_kernel(LossArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[T::LDS];
    __shared__ float tab[TG ? T::FM * 16 * T::LD : 1];
    __shared__ float red[T::NW][3][T::FM * 16];
    const lds_t* smem = (const lds_t*)raw;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, s16 = lane & 15, M = (int)a.M;
    // this workgroup's run of the vocabulary, in equal blocks
    const int vb = (int)((int64_t)a.V * blockIdx.x / gridDim.x), ve = (int)((int64_t)a.V * (blockIdx.x + 1) / gridDim.x);
    const int blocks = (ve - vb + T::BN - 1) / T::BN, rows = blocks > 0 ? (ve - vb + blocks - 1) / blocks : 0;
    const int ksteps = (a.K + T::BK - 1) / T::BK, steps = blocks * ksteps;

    int ib = 0, ik = 0, is = 0;   // the next loads' block, K step and stage
    auto issue = [&]() {
        const int v0 = vb + ib * rows, k0 = ik * T::BK;
        const int vl = min(rows, ve - v0) - 1, kl = min(T::BK, a.K - k0);
        const char* wb = (const char*)(a.W + (int64_t)v0 * a.ldw + k0);
        const char* xb = (const char*)(a.X + k0);
        const uint32_t st = lds0 + is * T::STAGE;
#pragma unroll
        for (int i = 0; i < T::IW + T::IX; ++i) {
            const bool w = i < T::IW;
            const int grp = (w ? i : i - T::IW) * T::NW + wave, p = grp * 64 + lane;
            const int r = p / T::CPR;
            int c = ((p % T::CPR) ^ (r & 15)) * 8;
            if (c >= kl) c = 0;   // past K: not multiplied
            if (w) dma16(wb, (uint32_t)((min(r, vl) * a.ldw + c) * 2), st + grp * 1024);
            else dma16(xb, (uint32_t)((min(r, M - 1) * a.ldx + c) * 2), st + T::W_BYTES + grp * 1024);
        }
        is = is + 1 == T::S ? 0 : is + 1;
        if (++ik == ksteps) {
            ik = 0;
            ++ib;
        }
    };
    // The targets, read before the ring starts: a load of the compiler's among
    // the ring's would be waited for together with all of them.  Several a
    // row: up to NID per thread, of all rows in a line; more are read again
    // for every block.
    constexpr int NID = TG ? 8 : 1;
    const bool few = TG && M * a.k <= NID * 256;
    int labs[T::FM], ids[NID];
    if constexpr (TG) {
        if (few) {
#pragma unroll
            for (int e = 0; e < NID; ++e) {
                const int at = tid + 256 * e;
                const int64_t id = at < M * a.k ? a.ids[(int64_t)(at / a.k) * a.ldids + at % a.k] : -1;
                ids[e] = id >= 0 && id < a.V ? (int)id : -1;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < T::FM; ++i) labs[i] = row_label(a, i * 16 + s16, M);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);   // (vmcnt 0)
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f, s2 = a.s2;
    const bool smooth = a.sumz != nullptr;
    float mx[T::FM], sm[T::FM], sz[T::FM];
    f32x4 acc[T::FM];
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
        mx[i] = -INFINITY;
        sm[i] = sz[i] = 0.0f;
        acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int s = 0; s < T::S - 1; ++s)
        if (s < steps) issue();
    int blk = 0, ks = 0, st = 0;
    for (int s = 0; s < steps; ++s) {
        // the step's loads have landed (S - 2 later steps may be in flight,
        // none counted on near the end), in every wave, and every wave is done
        // with the stage that is filled next
        if (s + T::S - 1 <= steps) phase_barrier<(T::S - 2) * (T::IW + T::IX)>();
        else phase_barrier<0>();
        if (s + T::S - 1 < steps) issue();
        const lds_t* ws = smem + st * T::STAGE;
        const int wrow = (wave * 16 + s16) * T::BK * 2, xrow = T::W_BYTES + s16 * T::BK * 2;
        const int kn = min(T::BK, a.K - ks * T::BK) / 32;
        auto part = [&](int q) {
            const int off = ((q * 4 + g) ^ s16) << 4;
            const bf16x8 wv = __builtin_bit_cast(bf16x8, *(const u32x4 __attribute__((address_space(3)))*)(ws + wrow + off));
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const bf16x8 xv = __builtin_bit_cast(
                    bf16x8, *(const u32x4 __attribute__((address_space(3)))*)(ws + xrow + i * 16 * T::BK * 2 + off));
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv, acc[i], 0, 0, 0);
            }
        };
        if (kn == T::BK / 32) {
#pragma unroll
            for (int q = 0; q < T::BK / 32; ++q) part(q);
        } else {
            for (int q = 0; q < kn; ++q) part(q);
        }
        st = st + 1 == T::S ? 0 : st + 1;
        if (++ks < ksteps) continue;
        // a block is done: lane 16 g + s holds X row 16 i + s, columns 4 g + 0..3 of the wave's 16
        const int v0 = vb + blk * rows, v = v0 + wave * 16 + g * 4, left = min(ve, v0 + rows) - v;   // valid from v on
        ks = 0;
        ++blk;
        if (!a.plain) {
            f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
            if (a.bias != nullptr) {
#pragma unroll
                for (int r = 0; r < 4; ++r) b[r] = a.bias[min(v + r, a.V - 1)];
            }
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float z = fmaf(a.scale, acc[i][r], b[r]);
                    acc[i][r] = a.cap > 0.0f ? a.cap * tanh_fast(z * inv_cap) : z;
                }
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            f32x4 u = acc[i];
            acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (TG) {
                *(f32x4*)(tab + (i * 16 + s16) * T::LD + wave * 16 + g * 4) = u;
            } else {
                const int d = labs[i] - v;
                if ((unsigned)d < 4u && d < left) a.zt[i * 16 + s16] = d == 0 ? u[0] : d == 1 ? u[1] : d == 2 ? u[2] : u[3];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (smooth) sz[i] += r < left ? u[r] : 0.0f;
                u[r] = r < left ? u[r] : -INFINITY;
            }
            const float top = fmaxf(fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])), mx[i]);
            const float base = stat_base(top, s2);
            float t = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) t += exp2_fast(fmaf(u[r], s2, -base));
            sm[i] = fmaf(sm[i], exp2_fast(mul_rn(mx[i], s2) - base), t);
            mx[i] = top;
        }
        if constexpr (TG) {
            // the targets among the block's columns: its logits are in LDS
            // (the direct loads in flight write elsewhere)
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            const int vn = min(ve, v0 + rows);
            if (few) {
#pragma unroll
                for (int e = 0; e < NID; ++e)
                    if (ids[e] >= v0 && ids[e] < vn)
                        a.zt[(tid + 256 * e) / a.k * a.kp + (tid + 256 * e) % a.k] =
                            tab[(tid + 256 * e) / a.k * T::LD + ids[e] - v0];
            } else {
                for (int m = tid >> 3; m < M; m += 32)
                    for (int q = tid & 7; q < a.k; q += 8) {
                        const int64_t id = a.ids[(int64_t)m * a.ldids + q];
                        if (id >= v0 && id < vn) a.zt[(int64_t)m * a.kp + q] = tab[m * T::LD + (int)(id - v0)];
                    }
            }
        }
    }
    // join the four lanes, then the waves, that share a row
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
        float top = fmaxf(mx[i], __shfl_xor(mx[i], 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float t = sm[i] * exp2_fast(mul_rn(mx[i], s2) - stat_base(top, s2));
        t += __shfl_xor(t, 16);
        t += __shfl_xor(t, 32);
        float z = sz[i];
        z += __shfl_xor(z, 16);
        z += __shfl_xor(z, 32);
        if (g == 0) {
            red[wave][0][i * 16 + s16] = top;
            red[wave][1][i * 16 + s16] = t;
            red[wave][2][i * 16 + s16] = z;
        }
    }
    __syncthreads();
    if (tid < M) {
        float top = -INFINITY, t = 0.0f, z = 0.0f;
#pragma unroll
        for (int w = 0; w < T::NW; ++w) top = fmaxf(top, red[w][0][tid]);
        const float base = stat_base(top, s2);
#pragma unroll
        for (int w = 0; w < T::NW; ++w) {
            t += red[w][1][tid] * exp2_fast(mul_rn(red[w][0][tid], s2) - base);
            z += red[w][2][tid];
        }
        *(float2*)(a.part + ((int64_t)tid * a.ntiles + blockIdx.x) * 2) = make_float2(top, t);
        if (smooth) a.sumz[(int64_t)tid * a.ntiles + blockIdx.x] = z;
    }
}

// Sum and maximum over the workgroup's 256 threads.
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}
__device__ __forceinline__ float block_max(float v, float* buf) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(buf[0], buf[1]), fmaxf(buf[2], buf[3]));
}

__device__ __forceinline__ bool target_ok(const LossArgs& a, int64_t m, int j) {
    const int64_t id = a.ids[m * a.ldids + j];
    const float t = a.teacher[m * a.ldt + j];   // (read with the id, not after it)
    return (id >= 0) & (id < a.V) & (t * (1.0f / a.T) != -INFINITY);
}

// Join a row's tiles, one workgroup per row.  With s2 the factor to base 2:
//   lse = ln2 (umax s2 + log2 sum); a row without any finite logit has -inf
//   cross entropy: lse - (1 - e) z_y - e / V sum z + c lse^2
//   distillation:  T^2 sum_j p_j (log p_j - (z_j / T - lse))
// The differences from the targets are taken to umax first and the logarithm
// added last, so a loss is good to some 40 x 2^-24 (17 found, of losses below 1)
// however large lse is; rounding lse before the difference would cost that of
// lse (1300 at 980).  Not less than that: a label that is the row's largest adds
// its own exponential, 1, to the others', so a loss of 1e-5 has one digit or two.
// Bound by latencies: what a thread needs first is read ahead of the
// reductions, all at once.
__global__ __launch_bounds__(256) void loss_finish_kernel(LossArgs a, int wgn) {
    __shared__ float buf[4];
    const int tid = threadIdx.x;
    const int64_t c = blockIdx.x;
    const int n = a.direct ? (int)a.M : a.hdr->n;
    if (c >= n) return;   // (rows without a target were cleared by the gather kernel)
    const int64_t m = a.direct ? c : (int64_t)a.map[c];
    const float* part = a.part + c * a.ntiles * 2;
    constexpr int U = 2;
    float2 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        p[u] = tid + 256 * u < a.ntiles ? *(const float2*)(part + 2 * (tid + 256 * u)) : make_float2(-INFINITY, 0.0f);
    const bool xent = a.labels != nullptr;
    const int64_t y = xent ? a.labels[m] : 0;
    // the label's kept value, or the thread's first target's, with that target
    const float* zt = a.zt + c * a.kp;
    const float* t = xent ? nullptr : a.teacher + m * a.ldt;
    const float it = 1.0f / a.T;
    bool ok = false;
    float u0 = 0.0f, t0 = 0.0f;
    if (xent) {
        u0 = zt[0];
    } else if (tid < a.k) {
        ok = target_ok(a, m, tid);
        t0 = t[tid] * it;
        u0 = zt[tid];
    }
    const float s2 = a.s2;
    float mx = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, p[u].x);
    for (int i = tid + 256 * U; i < a.ntiles; i += 256) mx = fmaxf(mx, part[2 * i]);
    mx = block_max(mx, buf);
    const float base = stat_base(mx, s2);
    float sm = 0.0f, sz = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) sm += p[u].y * exp2_fast(mul_rn(p[u].x, s2) - base);
    for (int i = tid + 256 * U; i < a.ntiles; i += 256) sm += part[2 * i + 1] * exp2_fast(mul_rn(part[2 * i], s2) - base);
    if (a.sumz != nullptr) {
        for (int i = tid; i < a.ntiles * wgn; i += 256) sz += a.sumz[c * a.ntiles * wgn + i];
        sz = block_sum(sz, buf);
    }
    sm = block_sum(sm, buf);
    // log2 of the sum over 2^(umax s2): what rounding base lost, put back
    const float top = mul_rn(mx, s2) == -INFINITY ? 0.0f : mx;
    const float l2 = __builtin_amdgcn_logf(sm) + fmaf(-top, s2, base);
    const float lse = kLn2 * fmaf(top, s2, l2);
    const float uz = a.plain ? a.scale : 1.0f;   // u to z
    if (xent) {
        const bool live = y >= 0 && y < a.V;
        if (tid == 0) {
            const float u = live ? u0 : 0.0f;
            float v = kLn2 * fmaf(top - u, s2, l2);
            if (a.smoothing > 0.0f) v += a.smoothing * uz * (u - sz / (float)a.V);
            if (a.z_loss != 0.0f) v += a.z_loss * lse * lse;
            if (u * s2 == -INFINITY) v = INFINITY;   // the label is masked out, whatever else is
            a.loss[m] = live ? v : 0.0f;
            a.lse[m] = live ? lse : 0.0f;
        }
        return;
    }
    // the teacher's log-partition over the row
    float any = ok ? 1.0f : 0.0f, tm = ok ? t0 : -INFINITY;
    for (int j = tid + 256; j < a.k; j += 256)
        if (target_ok(a, m, j)) {
            any = 1.0f;
            tm = fmaxf(tm, t[j] * it);
        }
    any = block_max(any, buf);
    float tl;
    if (a.teacher_lse != nullptr) {
        tl = a.teacher_lse[m];
    } else {
        tm = block_max(tm, buf);
        float ts = ok ? exp2_fast(kLog2e * (t0 - tm)) : 0.0f;
        for (int j = tid + 256; j < a.k; j += 256)
            if (target_ok(a, m, j)) ts += exp2_fast(kLog2e * (t[j] * it - tm));
        tl = tm + kLn2 * __builtin_amdgcn_logf(block_sum(ts, buf));
    }
    float kl = 0.0f;
    auto add = [&](float tj, float u) {
        const float lp = tj - tl;
        const float q = exp2_fast(kLog2e * lp);
        if (q != 0.0f) kl += u * s2 == -INFINITY ? INFINITY : q * (lp + kLn2 * fmaf(top - u, s2, l2));
    };
    if (ok) add(t0, u0);
    for (int j = tid + 256; j < a.k; j += 256)
        if (target_ok(a, m, j)) add(t[j] * it, zt[j]);
    kl = block_sum(kl, buf);
    if (tid == 0) {
        a.loss[m] = any != 0.0f ? a.T * a.T * kl : 0.0f;
        a.lse[m] = any != 0.0f ? lse : 0.0f;
    }
}

// ---- rows with a target -----------------------------------------------------

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

// Which of U rows from m on, `by` apart, are live (false past the last), their
// loads issued together.
template <int U>
__device__ __forceinline__ void rows_live(const LossArgs& a, int64_t m, int by, bool (&on)[U]) {
    if (a.labels != nullptr) {
        int64_t y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = a.labels[min(m + by * u, a.M - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) on[u] = y[u] >= 0 && y[u] < a.V && m + by * u < a.M;
    } else {
        uint8_t y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = a.live[min(m + by * u, a.M - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) on[u] = y[u] != 0 && m + by * u < a.M;
    }
}

__device__ __forceinline__ float usable_gref(float g) { return (g > 0.0f && g < INFINITY) ? g : 1.0f; }

// How dX's product over a piece is cut: its tiles are few where the live rows
// or the features are, so the vocabulary steps are split over workgroups, each
// split with a partial dX of its own.  In units of one K step of a workgroup,
// with what a tile costs besides (filling and draining the pipeline, writing
// and summing a partial) taken as 10: the whole number of splits, of at most
// two rounds of workgroups and at least four steps each, for which the work
// of dX's and dW's tiles (they run in one launch, dX's first) over the
// workgroups that run at once, and half a tile of what runs last, come out
// least.  One wave.
__device__ __forceinline__ int dx_splits(const LossArgs& a, int n, int lane) {
    const int tile = a.tile, tk = (a.K + tile - 1) / tile;
    const int tiles = max(1, (n + tile - 1) / tile * tk), all = a.Vp >> 6;
    const float rest = a.dW != nullptr ? (float)((a.Vp + tile - 1) / tile * tk) * ((n + 63) / 64 + 10.0f) : 0.0f;
    const float rest_one = a.dW != nullptr ? (n + 63) / 64 + 10.0f : 0.0f;
    float best = -INFINITY;   // minus the cost
    int mine = 1;
    for (int s = 1 + lane; s == 1 || (s * tiles <= 2 * a.slots && s * 4 <= all); s += 64) {
        const float one = (float)((all + s - 1) / s) + 10.0f;
        const float work = rest + (float)(tiles * s) * one;
        const float cost = fmaxf(work / (float)a.slots, one) + 0.5f * (rest > 0.0f ? rest_one : one);
        if (-cost > best) {
            best = -cost;
            mine = s;
        }
    }
    float top = best;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    int least = best == top ? mine : 1 << 30;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) least = min(least, __shfl_xor(least, o));
    return least;
}

// For more than a few thousand rows: each row's place among the live ones
// (pos, -1 without a target), their number, the largest |dloss| and dX's
// splits.  One workgroup, 8192 rows at a time: eight runs of 1024, a row of
// each per thread, whose live rows the waves count with a ballot per run
// (5.7 us for 8192 rows).
__global__ __launch_bounds__(1024) void loss_scan_kernel(LossArgs a) {
    constexpr int U = 8, NW = 16;
    __shared__ int cnt[U * NW];
    __shared__ float buf[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0;
    float g = 0.0f;
    for (int64_t m0 = 0; m0 < a.M; m0 += 1024 * U) {
        bool on[U];
        float d[U] = {};
        rows_live<U>(a, m0 + tid, 1024, on);
        if (a.dloss != nullptr) {
#pragma unroll
            for (int u = 0; u < U; ++u) d[u] = a.dloss[min(m0 + tid + 1024 * u, a.M - 1)];
        }
        unsigned long long bits[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bits[u] = __ballot(on[u]);
            if (lane == 0) cnt[u * NW + wave] = __popcll(bits[u]);
            if (on[u]) g = fmaxf(g, fabsf(d[u]));
        }
        __syncthreads();
        // live rows up to and with each (run, wave), over the 128 of them
        static_assert(U * NW == 128, "two counts a lane");
        int lo = cnt[lane], hi = cnt[64 + lane];
        const int lo1 = lo, hi1 = hi;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int p = __shfl_up(lo, o), q = __shfl_up(hi, o);
            if (lane >= o) {
                lo += p;
                hi += q;
            }
        }
        const int half = __shfl(lo, 63);
        hi += half;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u * NW + wave;
            const int before = at < 64 ? __shfl(lo - lo1, at) : __shfl(hi - hi1, at - 64);
            const int64_t m = m0 + tid + 1024 * u;
            if (m < a.M) a.pos[m] = on[u] ? base + before + __popcll(bits[u] & ((1ull << lane) - 1ull)) : -1;
        }
        base += __shfl(hi, 63);
        __syncthreads();
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) g = fmaxf(g, __shfl_xor(g, o));
    if (lane == 0) buf[wave] = g;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < NW; ++w) g = fmaxf(g, buf[w]);
    const int splits = a.dloss != nullptr ? dx_splits(a, base, lane) : 1;
    if (tid == 0) *a.hdr = LossHeader{base, usable_gref(g), splits};
}

// 8 values of row m of X from column k on, zeros past K (and for m < 0).
__device__ __forceinline__ u32x4 row_chunk(const LossArgs& a, int64_t m, int k) {
    if (m < 0 || k >= a.K) return u32x4{0u, 0u, 0u, 0u};
    const uint16_t* src = a.X + m * a.ldx + k;
    if (((uintptr_t)src & 15) == 0 && k + 8 <= a.K) return *(const u32x4*)src;
    return load8_any(src, a.K - k);
}

// What a wave reads of its row before it knows the row's place: the label, or
// lane j's first target, and the row's gradient.
struct RowInput {
    int64_t id = -1;
    float t = 0.0f, tl = 0.0f, dloss = 0.0f, lse = 0.0f;
};
template <bool BWD>
__device__ __forceinline__ RowInput row_input(const LossArgs& a, int64_t m, int lane) {
    RowInput in;
    if (a.labels != nullptr) {
        in.id = a.labels[m];
    } else if (lane < a.k) {
        in.id = a.ids[m * a.ldids + lane];
        in.t = a.teacher[m * a.ldt + lane];
    }
    if constexpr (BWD) {
        in.dloss = a.dloss[m];
        in.lse = a.lse[m];
        if (a.labels == nullptr && a.teacher_lse != nullptr) in.tl = a.teacher_lse[m];
    }
    return in;
}

// One wave: compact row c's targets and gradient constants, from row m.
template <bool BWD>
__device__ __forceinline__ void row_targets(const LossArgs& a, int64_t m, int c, const RowInput& in, float gref, int lane,
                                            int* sid, float* sp) {
    float rel = 1.0f, lse2 = 0.0f;
    if constexpr (BWD) {
        rel = in.dloss / gref;
        // a row without any finite logit: every probability 0
        lse2 = in.lse == -INFINITY ? INFINITY : in.lse * kLog2e;
    }
    if (a.labels != nullptr) {
        if (lane == 0) {
            a.ids32[(int64_t)c * a.kp] = (int)in.id;
            if constexpr (BWD) {
                // everything over (1 - smoothing), so that a label's own
                // weight is exactly the row's share of gref
                const float unit = a.smoothing < 1.0f ? 1.0f - a.smoothing : 1.0f;
                // (no probability: nothing for the penalty to weigh either)
                const float cq = a.z_loss != 0.0f && lse2 != INFINITY ? 1.0f + 2.0f * a.z_loss * in.lse : 1.0f;
                a.rows[c] = LossRow{lse2, rel * cq / unit, rel * a.smoothing / ((float)a.V * unit),
                                    a.smoothing < 1.0f ? rel : 0.0f};
            }
        }
        return;
    }
    const float it = 1.0f / a.T;
    // lane j's first target, then those 64 on: the id (-1: left out) and t / T
    auto target = [&](int j, float& t) {
        const int64_t id = j < 64 ? in.id : a.ids[m * a.ldids + j];
        t = (j < 64 ? in.t : a.teacher[m * a.ldt + j]) * it;
        return id >= 0 && id < a.V && t != -INFINITY ? (int)id : -1;
    };
    if constexpr (!BWD) {
        int* ids = a.ids32 + (int64_t)c * a.kp;
        float t;
        for (int j = lane; j < a.kp; j += 64) ids[j] = j < a.k ? target(j, t) : -1;
    } else {
        // the row's ids and t / T, then its probabilities, staged in LDS
        float tl = in.tl, tm = -INFINITY, ts = 0.0f, all = 0.0f;
        for (int j = lane; j < a.k; j += 64) {
            float t;
            sid[j] = target(j, t);
            sp[j] = t;
            if (sid[j] >= 0) tm = fmaxf(tm, t);
        }
        if (a.teacher_lse == nullptr) {
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) tm = fmaxf(tm, __shfl_xor(tm, o));
            for (int j = lane; j < a.k; j += 64)
                if (sid[j] >= 0) ts += exp2_fast(kLog2e * (sp[j] - tm));
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) ts += __shfl_xor(ts, o);
            tl = tm + kLn2 * __builtin_amdgcn_logf(ts);
        }
        for (int j = lane; j < a.k; j += 64) {
            sp[j] = sid[j] >= 0 ? exp2_fast(kLog2e * (sp[j] - tl)) : 0.0f;
            all += sp[j];
        }
        __builtin_amdgcn_wave_barrier();   // (one wave's own LDS: its operations stay in order)
        // weights; a target named twice keeps its weight at its first place
        int2* out = a.targets + (int64_t)c * a.kp;
        for (int j = lane; j < a.kp; j += 64) {
            const int id = j < a.k ? sid[j] : -1;
            bool first = id >= 0;
            float p = 0.0f;
            for (int u = 0; u < a.k; ++u) {
                const bool same = sid[u] == id;
                if (same && u < j) first = false;
                if (same) p += sp[u];
            }
            out[j] = make_int2(first ? id : -1, __builtin_bit_cast(int, first ? rel * p : 0.0f));
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) all += __shfl_xor(all, o);
        if (lane == 0) a.rows[c] = LossRow{lse2, rel * all, 0.0f, 0.0f};
    }
}

// Compacts the live rows of X with their targets, and clears what rows without
// a target get.  A workgroup takes four rows, a wave each; unless SCANNED (many
// rows: loss_scan_kernel has run) it counts the live rows before them and
// altogether by itself, which is cheaper than a launch that does.  The rows
// behind the last live one, up to a whole K step of dW's product, are zeroed.
// Bound by latencies: 333 x 768 in 5.7 us, 4096 x 4096 in 16 (67 MB).
constexpr int kGatherRows = 4;
template <bool BWD, bool SCANNED>
__global__ __launch_bounds__(256) void loss_gather_kernel(LossArgs a) {
    __shared__ float buf[4];
    __shared__ int cnt[2][4];
    __shared__ int places[kGatherRows];
    __shared__ int sid[BWD ? 4 : 1][BWD ? kMaxTargets : 1];
    __shared__ float sp[BWD ? 4 : 1][BWD ? kMaxTargets : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t r0 = (int64_t)blockIdx.x * kGatherRows;
    // the wave's row, its first loads (all of them up to 4096 features) and
    // what its place hangs on under way while the live rows are counted
    const int64_t m = r0 + wave;
    constexpr int U = 8;
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = row_chunk(a, m < a.M ? m : -1, lane * 8 + 512 * u);
    RowInput in;
    if (m < a.M) in = row_input<BWD>(a, m, lane);
    int64_t own = -1;
    if (!SCANNED && lane < kGatherRows && r0 + lane < a.M)
        own = a.labels != nullptr ? a.labels[r0 + lane] : a.live[r0 + lane] != 0 ? 0 : -1;
    int n, before = 0;
    float gref = 1.0f;
    if constexpr (SCANNED) {
        n = a.hdr->n;
        gref = a.hdr->gref;
        if (tid < kGatherRows) places[tid] = r0 + tid < a.M ? a.pos[r0 + tid] : -2;
    } else {
        int b = 0, all = 0;
        float g = 0.0f;
        // (eight rows a thread at a time, so that their loads overlap)
        for (int64_t m0 = tid; m0 < a.M; m0 += 256 * U) {
            bool on[U];
            float d[U] = {};
            rows_live<U>(a, m0, 256, on);
            if constexpr (BWD) {
#pragma unroll
                for (int u = 0; u < U; ++u) d[u] = a.dloss[min(m0 + 256 * u, a.M - 1)];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                b += on[u] && m0 + 256 * u < r0 ? 1 : 0;
                all += on[u] ? 1 : 0;
                if (on[u]) g = fmaxf(g, fabsf(d[u]));
            }
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            b += __shfl_xor(b, o);
            all += __shfl_xor(all, o);
        }
        if (lane == 0) {
            cnt[0][wave] = b;
            cnt[1][wave] = all;
        }
        __syncthreads();
        before = (cnt[0][0] + cnt[0][1]) + (cnt[0][2] + cnt[0][3]);
        n = (cnt[1][0] + cnt[1][1]) + (cnt[1][2] + cnt[1][3]);
        if constexpr (BWD) gref = usable_gref(block_max(g, buf));
        if (blockIdx.x == 0 && wave == 1) {
            const int splits = BWD ? dx_splits(a, n, lane) : 1;
            if (lane == 0) *a.hdr = LossHeader{n, gref, splits};
        }
        if (wave == 0) {
            const bool on = own >= 0 && own < a.V;
            const unsigned long long bits = __ballot(on);
            if (lane < kGatherRows)
                places[lane] = r0 + lane >= a.M ? -2 : on ? before + __popcll(bits & ((1ull << lane) - 1ull)) : -1;
        }
    }
    __syncthreads();
    const int c = places[wave];
    if (c != -2) {
        if (c < 0) {
            if constexpr (!BWD) {
                if (lane == 0) a.loss[m] = a.lse[m] = 0.0f;
            } else if (a.dX != nullptr) {
                // 16 bytes at a time from the row's first such boundary on
                const int es = a.grad_f32 ? 4 : 2;
                char* d = (char*)a.dX + m * a.lddx * es;
                const int64_t bytes = (int64_t)a.K * es;
                const int64_t head = min(bytes, (int64_t)((16 - ((uintptr_t)d & 15)) & 15));
                const int64_t body = head + ((bytes - head) & ~int64_t(15));
                for (int64_t b = head + lane * 16; b < body; b += 1024) *(u32x4*)(d + b) = u32x4{0u, 0u, 0u, 0u};
                for (int64_t b = lane * 2; b < head; b += 128) *(uint16_t*)(d + b) = 0;
                for (int64_t b = body + lane * 2; b < bytes; b += 128) *(uint16_t*)(d + b) = 0;
            }
        } else {
            if (lane == 0) a.map[c] = (int)m;
            // the row itself, then its targets
            for (int k0 = lane * 8; k0 < a.Kp; k0 += 512 * U) {
                if (k0 >= 512 * U) {
#pragma unroll
                    for (int u = 0; u < U; ++u) v[u] = row_chunk(a, m, k0 + 512 * u);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k0 + 512 * u < a.Kp) *(u32x4*)(a.Xc + (int64_t)c * a.Kp + k0 + 512 * u) = v[u];
            }
            row_targets<BWD>(a, m, c, in, gref, lane, sid[BWD ? wave : 0], sp[BWD ? wave : 0]);
        }
    }
    // (at most 63 rows, over the workgroups' waves)
    const int pad = ((n + 63) & ~63) - n;
    for (int p = blockIdx.x * 4 + wave; p < pad; p += gridDim.x * 4)
        for (int k = lane * 8; k < a.Kp; k += 512) *(u32x4*)(a.Xc + (int64_t)(n + p) * a.Kp + k) = row_chunk(a, -1, k);
}

// ---- backward ---------------------------------------------------------------

// One tile of G, the gradient by s over gref (and over the call's unit: the
// label's weight, or T): what multiplies it is put back, in 32 bits, where
// dX, dW and dbias are made.  So the entry of a label that is far from learnt
// is near -1 and survives bf16 nearly exactly, whatever the loss is divided
// by.  Bound as the forward tile is, with 128 KB of G a tile to write: 4096 x
// 32000 x 4096 in 780 us.  G is rounded to bf16 (at most 2^-8 of each entry, to
// nearest) because the products that follow run on bf16 MFMA.
template <class T, bool TG>
constexpr int grad_lds() {
    const int tab = TG ? T::HA * (T::BN + 4) * 4 : 0, stage = T::BM * (T::BN * 2 + 16);
    return std::max(T::LDS, std::max(tab, stage));
}
template <class T, bool TG>
__device__ __forceinline__ void grad_tile(const LossArgs& a, int n, int m0, int tn, lds_t* smem, int wave, int lane) {
    constexpr int LDG = T::BN * 2 + 16;   // bytes of a staged row
    const int tid = wave * 64 + lane;
    const int p0 = tn * T::BN, v0 = a.v0 + p0;
    Acc<T> acc;
    logits_tile<T>(a, m0, v0, n, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    const int vr = a.V - v0;
    const float s2 = a.s2;
    const float inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
    // several targets a row: the first AHEAD pairs of them per thread of a
    // row's PER, read a half of the rows ahead (-1 past the last)
    constexpr int PER = T::NT / T::HA, AHEAD = TG ? 32 / PER : 1;
    int4 tg[AHEAD];
    [[maybe_unused]] auto targets_ahead = [&](int ha) {
        const int m = m0 + ha * T::HA + tid / PER;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int q = (tid % PER + PER * i) * 2;
            tg[i] = m < n && q < a.kp ? *(const int4*)(a.targets + (int64_t)m * a.kp + q) : int4{-1, 0, -1, 0};
        }
    };
    if constexpr (TG) targets_ahead(0);
    BiasRegs<T> bias;
    if (!a.plain) bias.read(a, at, v0);
    LossRow rows[2][T::FM];
    int labs[2][T::FM];
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int m = m0 + at.row(ha, i);
            rows[ha][i] = a.rows[min(m, n - 1)];
            if constexpr (!TG) labs[ha][i] = row_label(a, m, n) - v0 - at.wn * T::FN * 16;
        }
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
        if constexpr (TG) {
            // the weights of the targets in these rows, as a table; the
            // targets themselves were read a half ahead
            float __attribute__((address_space(3)))* tab = (float __attribute__((address_space(3)))*)smem;
            constexpr int LD = T::BN + 4;
            if (ha) __syncthreads();
            for (int e = tid * 4; e < T::HA * LD; e += T::NT * 4)
                *(f32x4 __attribute__((address_space(3)))*)(tab + e) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            __syncthreads();
            const int r = tid / PER, m = m0 + ha * T::HA + r;
            auto put = [&](int id, int w) {
                if ((unsigned)(id - v0) < (unsigned)T::BN) tab[r * LD + id - v0] = __builtin_bit_cast(float, w);
            };
            if (m < n) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    put(tg[i].x, tg[i].y);
                    put(tg[i].z, tg[i].w);
                }
                for (int q = (tid % PER + PER * AHEAD) * 2; q < a.kp; q += PER * 2) {
                    const int4 p = *(const int4*)(a.targets + (int64_t)m * a.kp + q);
                    put(p.x, p.y);
                    put(p.z, p.w);
                }
            }
            __syncthreads();
            if (ha == 0) targets_ahead(1);
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int row = at.row(ha, i);
            const LossRow c = rows[ha][i];
            if (!a.plain) row_affine<T>(a, bias, acc, ha, i);
            f32x4 v[2][T::FN];
            if (a.cap > 0.0f) {   // acc becomes dz/ds
                rarely();
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            float slope;
                            const float z = a.cap * tanh_fast(acc[ha][hb][i][j][r] * inv_cap, slope);
                            v[hb][j][r] = fmaf(exp2_fast(fmaf(z, s2, -c.lse2)), c.rq, -c.ru);
                            acc[ha][hb][i][j][r] = slope;
                        }
            } else {
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[hb][j][r] = fmaf(exp2_fast(fmaf(acc[ha][hb][i][j][r], s2, -c.lse2)), c.rq, -c.ru);
            }
            if constexpr (TG) {
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
                        v[hb][j] -= *(const f32x4 __attribute__((address_space(3)))*)(
                            (float __attribute__((address_space(3)))*)smem + (row - ha * T::HA) * (T::BN + 4) +
                            at.col(hb, j));
            }
            if constexpr (!TG) {
                // (the wave's columns are two runs of FN * 16)
                const unsigned lab = (unsigned)labs[ha][i];
                if (lab < (unsigned)T::BN && (lab & (T::HB - 1)) < (unsigned)(T::FN * 16)) {
                    rarely();
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int j = 0; j < T::FN; ++j)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                v[hb][j][r] -= lab == (unsigned)(hb * T::HB + j * 16 + at.g * 4 + r) ? c.rp : 0.0f;
                }
            }
            if (a.cap > 0.0f) {
                rarely();
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) v[hb][j] *= acc[ha][hb][i][j];
            }
            if (m0 + T::BM > n) {   // rows past the live ones
                rarely();
                const bool on = m0 + row < n;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[hb][j][r] = on ? v[hb][j][r] : 0.0f;
            }
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) acc[ha][hb][i][j] = v[hb][j];
            __builtin_amdgcn_sched_barrier(0);   // one row of fragments at a time keeps the registers within bounds
        }
    }
    if (vr < T::BN) {   // columns past the vocabulary
        rarely();
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
        // column sums over 128 rows each (all of the tile's, or each half's):
        // a lane's rows, the 16 lanes of a group, then (through LDS) the waves
        // that share the columns
        constexpr int PARTS = T::BM / kDbiasRows, PER = 2 / PARTS;
        static_assert(T::BM == 128 || T::BM == 256, "column sums of 128 rows");
        float __attribute__((address_space(3)))* red = (float __attribute__((address_space(3)))*)smem;
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < PER; ++h)
#pragma unroll
                        for (int i = 0; i < T::FM; ++i) t += acc[part * PER + h][hb][i][j];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        t[r] = row_sum(t[r]);
                        if (at.s == 0) red[(part * T::WGM + at.wm) * T::BN + at.col(hb, j) + r] = t[r];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        __syncthreads();
        for (int e = tid; e < PARTS * T::BN; e += T::NT) {
            const int part = e / T::BN, c = e % T::BN;
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < T::WGM; ++w) t += red[(part * T::WGM + w) * T::BN + c];
            a.dbp[(int64_t)(m0 / kDbiasRows + part) * a.ldb + v0 + c] = t;
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

template <class T, class H, bool TG>
__global__ __launch_bounds__(T::NT, 2) void loss_grad_kernel(LossArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[std::max(grad_lds<T, TG>(), grad_lds<H, TG>())];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = a.hdr->n;
    int tm, tn, half;
    if (!map_rounds(blockIdx.x, (n + T::BM - 1) / T::BM, (a.vn + T::BN - 1) / T::BN, a.slots, T::BM > H::BM, tm, tn, half))
        return;
    // (a half without a live row is not multiplied: an operand's rows are
    // clamped to the live ones, of which it has none)
    if (half < 0) {
        grad_tile<T, TG>(a, n, tm * T::BM, tn, (lds_t*)raw, wave, lane);
    } else if (tm * T::BM + half * H::BM < n) {
        grad_tile<H, TG>(a, n, tm * T::BM + half * H::BM, tn, (lds_t*)raw, wave, lane);
    }
}

// A finished tile times f as rows of a gradient matrix D (bf16 or binary32),
// columns k0 on: row r of the tile is row where(r) of D; rows of them and cols
// columns exist.  bf16 goes through LDS, so that the stores write whole row
// segments.
template <class T, class Where>
__device__ __forceinline__ void store_tile(const Acc<T>& acc, float f, void* Dv, bool f32, int64_t ld, int k0, int rows,
                                           int cols, lds_t* smem, int wave, int lane, Where where) {
    constexpr int LDG = T::BN * 2 + 16;
    const Place<T> at(wave, lane);
    if (f32) {
        float* D = (float*)Dv + k0;
        const bool vec = ((uintptr_t)D & 15) == 0 && ld % 4 == 0;
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const int row = at.row(ha, i);
                if (row >= rows) continue;
                float* d = D + where(row) * ld;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) {
                        const int col = at.col(hb, j);
                        const f32x4 v = acc[ha][hb][i][j] * f;
                        if (vec && col + 4 <= cols) *(f32x4*)(d + col) = v;
                        else
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (col + r < cols) d[col + r] = v[r];
                    }
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
    uint16_t* D = (uint16_t*)Dv + k0;
    const bool vec = ((uintptr_t)D & 15) == 0 && ld % 8 == 0;
    constexpr int CPR = T::BN / 8;
    for (int p = wave * 64 + lane; p < T::BM * CPR; p += T::NT) {
        const int r = p / CPR, c = (p % CPR) * 8;
        if (r >= rows || c >= cols) continue;
        const u32x4 w = *(const u32x4 __attribute__((address_space(3)))*)(smem + r * LDG + c * 2);
        uint16_t* d = D + where(r) * ld + c;
        if (vec && c + 8 <= cols) *(u32x4*)d = w;
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// Whether dX's tiles are its final values: one split of one piece.
__device__ __forceinline__ bool dx_at_once(const LossArgs& a, int splits) { return splits == 1 && a.vn == a.V; }

// A workgroup's share of dX: G(piece) . W(piece) over the split's vocabulary
// steps, as the result's own rows where that is all of it, else as a partial
// ([split] (+)=, live rows only).
template <class T>
__device__ __forceinline__ void dx_tile(const LossArgs& a, int n, int tm, int tn, int split, int splits, float f,
                                        lds_t* smem, int wave, int lane) {
    const int m0 = tm * T::BM, k0 = tn * T::BN;
    const int all = (a.vn + 63) >> 6;
    const int per = (all + splits - 1) / splits;
    const int s0 = min(split * per, all), steps = min(per, all - s0);
    Operand<T::HA, false, T::IA, T::NW> A;
    Operand<T::HB, true, T::IB, T::NW> B;
    A.init(a.G + (int64_t)m0 * a.Vp + s0 * 64, a.Vp, T::BM, steps, 0, wave, lane);
    B.init(a.W + (int64_t)(a.v0 + s0 * 64) * a.ldw + k0, a.ldw, a.Kw - k0, steps,
           s0 + steps == all ? a.vn & 63 : 0, wave, lane);
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    if (dx_at_once(a, splits)) {
        store_tile<T>(acc, f, a.dX, a.grad_f32, a.lddx, k0, n - m0, a.K - k0, smem, wave, lane,
                      [&](int r) { return (int64_t)a.map[m0 + r]; });
        return;
    }
    float* P = a.dxp + ((int64_t)split * ((n + T::BM - 1) / T::BM) * T::BM + m0) * a.Kp + k0;
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j) {
                    const int col = at.col(hb, j);
                    if (k0 + col >= a.Kp || m0 + at.row(ha, i) >= n) continue;
                    f32x4* p = (f32x4*)(P + (int64_t)at.row(ha, i) * a.Kp + col);
                    *p = a.first ? acc[ha][hb][i][j] : *p + acc[ha][hb][i][j];
                }
}

// The results that are made from partials (bound by their bytes: 7373 x 4096
// from one partial in 33 us, 5.5 TB/s).  Workgroups from `dx_groups` on:
// dbias = gref unit (the sum over the row blocks, in order).  Before them, one
// per row, unless the products wrote dX themselves: dX = gref unit scale (the
// sum of its partials), in the row's own place; where a row has fewer than 128
// runs of four features, several threads share each run's splits and join
// through LDS, in order.
__global__ __launch_bounds__(256) void loss_outputs_kernel(LossArgs a, float unit, int dx_groups) {
    __shared__ f32x4 buf[256];
    const int c = blockIdx.x, n = a.hdr->n, splits = a.hdr->splits, tile = a.tile;
    if (c >= dx_groups) {
        const int v = (c - dx_groups) * 256 + threadIdx.x;
        if (v >= a.V) return;
        const int parts = (n + kDbiasRows - 1) / kDbiasRows;
        constexpr int U = 8;
        float t = 0.0f;
        for (int i0 = 0; i0 < parts; i0 += U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = i0 + u < parts ? a.dbp[(int64_t)(i0 + u) * a.ldb + v] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) t += x[u];
        }
        a.dbias[v] = t * (unit * a.hdr->gref);
        return;
    }
    if (c >= n || dx_at_once(a, splits)) return;
    const float mul = unit * a.scale;
    const int64_t m = a.map[c];
    const float f = mul * a.hdr->gref;
    const int64_t sp = (int64_t)((n + tile - 1) / tile) * tile * a.Kp;
    const int runs = (a.K + 3) >> 2;
    int width = 256;   // threads along the row
    while (width > runs && width > 16) width >>= 1;
    const int groups = 256 / width, grp = threadIdx.x / width;
    for (int k0 = 0; k0 < a.K; k0 += width * 4) {
        const int k = k0 + (threadIdx.x % width) * 4;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (k < a.K) {
            const float* p = a.dxp + (int64_t)c * a.Kp + k;
            constexpr int U = 8;
            for (int s0 = grp; s0 < splits; s0 += groups * U) {
                f32x4 t[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int s = s0 + u * groups;
                    t[u] = s < splits ? *(const f32x4*)(p + s * sp) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
#pragma unroll
                for (int u = 0; u < U; ++u) v += t[u];
            }
        }
        if (groups > 1) {
            __syncthreads();
            buf[threadIdx.x] = v;
            __syncthreads();
            if (grp > 0) continue;
            for (int g = 1; g < groups; ++g) v += buf[g * width + threadIdx.x];
        }
        if (k >= a.K) continue;
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

// One tile of a piece's dW: gref unit scale G^T . X.
template <class T>
__device__ __forceinline__ void dw_tile(const LossArgs& a, int n, int tm, int tn, float f, lds_t* smem, int wave, int lane) {
    const int p0 = tm * T::BM, k0 = tn * T::BN;
    const int steps = (n + 63) >> 6;
    Operand<T::HA, true, T::IA, T::NW> A;
    Operand<T::HB, true, T::IB, T::NW> B;
    A.init(a.G + p0, a.Vp, T::BM, steps, 0, wave, lane);
    B.init(a.Xc + k0, a.Kp, a.Kp - k0, steps, 0, wave, lane);
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    store_tile<T>(acc, f, a.dW, a.grad_f32, a.lddw, k0, a.vn - p0, a.K - k0, smem, wave, lane,
                  [&](int r) { return (int64_t)(a.v0 + p0 + r); });
}

// Both products of a piece in one launch, dX's workgroups first: they need
// the same G, and together they fill the device better than one after the
// other (950 x 50257 x 768: 140 us against 80 and 82; 4096 x 32000 x 4096:
// 1440 us, 1490 TFLOP/s, bound by the matrix pipe; 333 x 30522 x 768: 47 us, of
// which the bytes of dX's partials (9 MB) and of dW (47 MB) are a quarter, the
// ends of dW's tiles of six K steps most of the rest).
template <class TX, class TW>
__global__ __launch_bounds__(TX::NT, 2) void loss_products_kernel(LossArgs a, float mul) {
    constexpr int NEED = TW::BM * (TW::BN * 2 + 16);
    __shared__ __attribute__((aligned(1024))) unsigned char raw[TX::LDS > NEED ? TX::LDS : NEED];
    lds_t* smem = (lds_t*)raw;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.hdr->n, splits = a.hdr->splits;
    const int tk = (a.K + TX::BN - 1) / TX::BN, tr = (n + TX::BM - 1) / TX::BM;
    const int ndx = a.dX != nullptr ? tr * tk * splits : 0;
    int tm, tn, split;
    if ((int)blockIdx.x < ndx) {
        map_tile(blockIdx.x, tr, tk, tm, tn, split, splits);
        dx_tile<TX>(a, n, tm, tn, split, splits, mul * a.hdr->gref, smem, wave, lane);
    } else if (a.dW != nullptr) {
        if (!map_tile(blockIdx.x - ndx, (a.vn + TW::BM - 1) / TW::BM, tk, tm, tn, split, 1)) return;
        dw_tile<TW>(a, n, tm, tn, mul * a.hdr->gref, smem, wave, lane);
    }
}

template <bool AT, bool BT>
using L256 = LTile<2, 4, 4, 2, AT, BT>;
template <bool AT, bool BT>
using L256Half = LTile<2, 4, 2, 2, AT, BT>;   // half the rows of L256
template <bool AT, bool BT>
using L128 = LTile<2, 2, 2, 2, AT, BT>;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What G is over besides gref: T (whose square the loss carries, over one
// temperature from its derivative), or the label's own weight.
float unit_of(const LossArgs& a) {
    return a.labels == nullptr ? a.T : a.smoothing < 1.0f ? 1.0f - a.smoothing : 1.0f;
}

}  // namespace

int loss_sumz_parts(int tile) { return tile == 256 ? L256<false, false>::WGN : L128<false, false>::WGN; }

hipError_t launch_loss_flags(const LossArgs& a, hipStream_t st) {
    return launch_kernel(loss_flags_kernel, dim3((unsigned)up(a.M, 4)), dim3(256), st, a);
}

hipError_t launch_loss_scan(const LossArgs& a, hipStream_t st) {
    return launch_kernel(loss_scan_kernel, dim3(1), dim3(1024), st, a);
}

hipError_t launch_loss_gather(const LossArgs& a, bool scanned, hipStream_t st) {
    const dim3 grid((unsigned)std::max<int64_t>(1, up(a.M, kGatherRows)));
    if (a.dloss != nullptr)
        return scanned ? launch_kernel(loss_gather_kernel<true, true>, grid, dim3(256), st, a)
                       : launch_kernel(loss_gather_kernel<true, false>, grid, dim3(256), st, a);
    return scanned ? launch_kernel(loss_gather_kernel<false, true>, grid, dim3(256), st, a)
                   : launch_kernel(loss_gather_kernel<false, false>, grid, dim3(256), st, a);
}

hipError_t launch_loss_forward(const LossArgs& a, hipStream_t st) {
    const bool tg = a.labels == nullptr;
    // (halved tiles of a last round: at most slots / 2 workgroups more)
    const dim3 grid((unsigned)(up(a.M, a.tile) * a.ntiles + (a.tile == 256 ? a.slots / 2 : 0)));
    if (a.tile == 256) {
        using T = L256<false, false>;
        using H = L256Half<false, false>;
        return tg ? launch_kernel(loss_forward_kernel<T, H, true>, grid, dim3(T::NT), st, a)
                  : launch_kernel(loss_forward_kernel<T, H, false>, grid, dim3(T::NT), st, a);
    }
    using T = L128<false, false>;
    return tg ? launch_kernel(loss_forward_kernel<T, T, true>, grid, dim3(T::NT), st, a)
              : launch_kernel(loss_forward_kernel<T, T, false>, grid, dim3(T::NT), st, a);
}

hipError_t launch_loss_stream(const LossArgs& a, hipStream_t st) {
    const bool tg = a.labels == nullptr;
    const dim3 grid((unsigned)a.ntiles);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return tg ? launch_kernel(loss_stream_kernel<T, true>, grid, dim3(T::NT), st, a)
                  : launch_kernel(loss_stream_kernel<T, false>, grid, dim3(T::NT), st, a);
    };
    static_assert(kStreamRows == 32, "rows of the larger form");
    return a.M <= 16 ? go(Stream<1, 256, 3>{}) : go(Stream<2, 256, 3>{});
}

hipError_t launch_loss_finish(const LossArgs& a, hipStream_t st) {
    return launch_kernel(loss_finish_kernel, dim3((unsigned)a.M), dim3(256), st, a,
                         a.stream ? 1 : loss_sumz_parts(a.tile));
}

hipError_t launch_loss_grad(const LossArgs& a, hipStream_t st) {
    const bool tg = a.labels == nullptr;
    // (halved tiles of a last round: at most slots / 2 workgroups more)
    const dim3 grid((unsigned)(up(a.M, a.tile) * up(a.vn, a.tile) + (a.tile == 256 ? a.slots / 2 : 0)));
    if (a.tile == 256) {
        using T = L256<false, false>;
        using H = L256Half<false, false>;
        return tg ? launch_kernel(loss_grad_kernel<T, H, true>, grid, dim3(T::NT), st, a)
                  : launch_kernel(loss_grad_kernel<T, H, false>, grid, dim3(T::NT), st, a);
    }
    using T = L128<false, false>;
    return tg ? launch_kernel(loss_grad_kernel<T, T, true>, grid, dim3(T::NT), st, a)
              : launch_kernel(loss_grad_kernel<T, T, false>, grid, dim3(T::NT), st, a);
}

hipError_t launch_loss_products(const LossArgs& a, hipStream_t st) {
    const int b = a.tile;
    // (dX: at most two rounds of workgroups, or one a tile)
    const int64_t dx = a.dX != nullptr ? std::max<int64_t>(up(a.M, b) * up(a.K, b), 2 * a.slots) : 0;
    const int64_t dw = a.dW != nullptr ? up(a.vn, b) * up(a.K, b) : 0;
    const dim3 grid((unsigned)(dx + dw));
    const float mul = unit_of(a) * a.scale;
    if (b == 256)
        return launch_kernel(loss_products_kernel<L256<false, true>, L256<true, true>>, grid, dim3(512), st, a, mul);
    return launch_kernel(loss_products_kernel<L128<false, true>, L128<true, true>>, grid, dim3(256), st, a, mul);
}

hipError_t launch_loss_outputs(const LossArgs& a, hipStream_t st) {
    const int64_t dx = a.dX != nullptr ? a.M : 0, db = a.dbias != nullptr ? up(a.V, 256) : 0;
    return launch_kernel(loss_outputs_kernel, dim3((unsigned)(dx + db)), dim3(256), st, a, unit_of(a), (int)dx);
}

}  // namespace mkp

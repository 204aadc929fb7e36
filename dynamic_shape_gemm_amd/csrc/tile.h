// The tile multiplier of this library's fused products (device code): a
// workgroup's BM x BN tile over direct global->LDS loads in two stages, the
// accumulators left in registers for the kernel around it.  Operands are read
// along their rows or across them; elements are bf16, or 8-bit integers taken in
// pairs (an 8-bit matrix is one of half as many 16-bit columns).
#pragma once

#include "kernels.h"
#include "load8.h"

#include <hip/hip_ext.h>

#include <type_traits>

namespace mkp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char lds_t;

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

// Round to nearest even, NaN kept a NaN: the conversion instruction.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// What the 16 bytes a lane that make a fragment are multiplied as: eight bf16
// values (16x16x32) or sixteen 8-bit integers (16x16x64), at the same cycles.
struct MulBf16 {
    typedef f32x4 acc;
    static __device__ __forceinline__ acc mul(bf16x8 b, bf16x8 a, acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    }
};
struct MulI8 {
    typedef i32x4 acc;
    static __device__ __forceinline__ acc mul(bf16x8 b, bf16x8 a, acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
    }
};

// ---- tiles -----------------------------------------------------------------
//
// One workgroup multiplies a BM x BN tile over K steps of 64 (16-bit columns).  Each operand's tile is two halves of BM / 2 (BN / 2) rows, each in
// a block of its own in LDS, and a wave's part of the tile is one block of
// every half pair: the four quadrants are what a wave works through in turn.
//
// An operand is read either along its rows (the reduction is contiguous:
// X and W for the logits, G for dX) or across them (the reduction is the
// row: W for dX, G and X for dW); the second form goes through the LDS
// transpose read, which hands each lane four values of one column.
template <int WGM_, int WGN_, int FM_, int FN_, bool AT_, bool BT_, class MUL_ = MulBf16>
struct LTile {
    using MUL = MUL_;
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
using Acc = typename T::MUL::acc[2][2][T::FM][T::FN];

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
// Measured (256 x 256 tile of bf16, one per CU): 1.43 us a step, 1500 TFLOP/s over the
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
                for (int j = 0; j < T::FN; ++j) acc[ha][hb][i][j] = typename T::MUL::acc{0, 0, 0, 0};
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
                    acc[ha][hb][i][j] = T::MUL::mul(xb[hb][ks][j], ya[ks][i], acc[ha][hb][i][j]);
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

// A tile's bf16 values, staged in LDS in rows of staged_ld<T> bytes, as rows of D:
// the stores write whole row segments.
template <class T>
constexpr int staged_ld = T::BN * 2 + 16;
template <class T, class Where>
__device__ __forceinline__ void store_staged(uint16_t* D, int64_t ld, int rows, int cols, const lds_t* smem, int wave, int lane,
                                             Where where) {
    constexpr int LDG = staged_ld<T>;
    __syncthreads();
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

// A finished tile times f as rows of a gradient matrix D (bf16 or binary32),
// columns k0 on: row r of the tile is row where(r) of D; rows of them and cols
// columns exist.  bf16 goes through LDS, so that the stores write whole row
// segments.
template <class T, class Where>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[2][2][T::FM][T::FN], float f, void* Dv, bool f32, int64_t ld, int k0, int rows,
                                           int cols, lds_t* smem, int wave, int lane, Where where) {
    constexpr int LDG = staged_ld<T>;
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
    store_staged<T>((uint16_t*)Dv + k0, ld, rows, cols, smem, wave, lane, where);
}

}  // namespace
}  // namespace mkp

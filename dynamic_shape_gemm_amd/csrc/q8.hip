// 8-bit matrices on CDNA4 (gfx950): quantisation by rows and back, a linear
// layer in 8-bit integers, and the backward pass of a layer whose input and
// pre-activation were kept in 8 bits.
//
// Row m (or a group of columns of it) is held as integers q = rne(x / s) of
// -127 .. 127 and one binary32 scale s = max(max |x| / 127, 2^-126); where the
// row holds an infinity or NaN, s is NaN and q is 0, so that every product with
// it is NaN.
#include "q8.h"

#include "act.h"
#include "tile.h"

#include <algorithm>
#include <cmath>

namespace mkp {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2a1 __attribute__((ext_vector_type(2), aligned(1)));
// (memory of any alignment of its elements is read and written by whole vectors:
// the same instructions as for aligned ones)
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __attribute__((aligned(16))) const uint32_t kZeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};

// Device memory's own address space: what is chosen between two pointers is
// otherwise read by instructions that wait for LDS too.  ALIGN: p's alignment.
template <class V, int ALIGN>
__device__ __forceinline__ V load_global(const void* p) {
    typedef V U __attribute__((aligned(ALIGN)));
    return *(const U __attribute__((address_space(1)))*)p;
}

template <class V, int ALIGN>
__device__ __forceinline__ V load_once(const void* p) {
    typedef V U __attribute__((aligned(ALIGN)));
    return __builtin_nontemporal_load((const U __attribute__((address_space(1)))*)p);
}

constexpr float kTiny = 1.17549435e-38f;   // 2^-126

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
// (a vector's element by value: __builtin_bit_cast of one in place reads element 0)
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// Eight consecutive values of a row as read: bf16 or binary32, zeros past `nvalid`.
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    u32x4 w;
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void read(const void* p) { w = load_global<u32x4, 2>(p); }
    __device__ __forceinline__ void load(const void* row, int64_t c, int nvalid) {
        const uint16_t* p = (const uint16_t*)row + c;
        if (nvalid >= 8) read(p);
        else w = load8_elems(p, nvalid);
    }
    // The largest |x|, as the bits of a value of X's type: all infinities and
    // NaN are above every finite one.
    __device__ __forceinline__ uint32_t top() const {
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
        return std::max((uint32_t)m[0], (uint32_t)m[1]);
    }
    static __device__ __forceinline__ float top_value(uint32_t t) { return __builtin_bit_cast(float, t << 16); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};
template <>
struct Raw8<true> {
    f32x4 a, b;
    __device__ __forceinline__ void zero() { a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ void read(const void* p) {
        a = load_global<f32x4, 4>(p);
        b = load_global<f32x4, 4>((const float*)p + 4);
    }
    __device__ __forceinline__ void load(const void* row, int64_t c, int nvalid) {
        const float* p = (const float*)row + c;
        if (nvalid >= 8) {
            read(p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = i < nvalid ? p[i] : 0.0f;
                b[i] = i + 4 < nvalid ? p[i + 4] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = std::max(m, abs_bits(a[i]));
            m = std::max(m, abs_bits(b[i]));
        }
        return m;
    }
    static __device__ __forceinline__ float top_value(uint32_t t) { return __builtin_bit_cast(float, t); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[i + 4] = b[i];
        }
    }
};

// A row's (group's) scale, and what its values are multiplied by.
struct Scale8 {
    float s, inv;
    bool ok;
    __device__ __forceinline__ explicit Scale8(float top) {
        // top / 127 rounded to nearest, from the rounded reciprocal of 127 and the exact
        // rest (Markstein; right for every mantissa); below 2^-126 it does not count
        ok = top < INFINITY;
        constexpr float r = 1.0f / 127.0f;
        const float q = top * r;
        s = fmaxf(fmaf(fmaf(-127.0f, q, top), r, q), kTiny);
        inv = __builtin_amdgcn_rcpf(s);
        if (!ok) {
            s = __builtin_nanf("");
            inv = 0.0f;
        }
    }
};

// Eight values to integers, a byte each.  x * inv + 1.5 * 2^23 rounds to the
// nearest integer n, whose low byte is the sum's; inv is 1 / s to a unit, so n can
// be the neighbour of the nearest when x / s is next to a half.  The rest r = x -
// n s is exact (a multiple of half a unit of s below 2^24 of them), so where 2 |r|
// reaches s -- rarely, and a branch for the whole wave -- n is put right: away
// from r beyond s, and to the even neighbour at s.
__device__ __forceinline__ u32x2 to_i8(const float (&v)[8], const Scale8& sc) {
    constexpr float kMagic = 12582912.0f;
    float t[8], most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = fmaf(v[i], sc.inv, kMagic);
        most = fmaxf(most, fabsf(fmaf(kMagic - t[i], sc.s, v[i])));
    }
    if (2.0f * most >= sc.s) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = t[i] - kMagic, r = fmaf(-n, sc.s, v[i]), r2 = 2.0f * fabsf(r);
            const bool odd = (__builtin_bit_cast(uint32_t, t[i]) & 1) != 0;
            if (r2 > sc.s || (r2 == sc.s && odd)) t[i] += copysignf(1.0f, r);
        }
    }
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __builtin_bit_cast(uint32_t, t[4 * h + i]);
        out[h] = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
        out[h] = sc.ok ? out[h] : 0u;
    }
    return out;
}

// What rounding v to bf16 leaves of it, exactly (of an infinity or NaN: nothing).
__device__ __forceinline__ float bf16_rest(float v) {
    const float hi = bf16_lo(f32_to_bf16(v));
    return fabsf(hi) < INFINITY ? v - hi : 0.0f;
}

// Up to eight bytes to a row (any alignment).
__device__ __forceinline__ void store_i8(int8_t* p, u32x2 w, int n) {
    if (n >= 8) {
        *(u32x2a1*)p = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return std::max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true));
}
// The largest of the 4, 8, 16 or 32 lanes around this one, or of the wave.
__device__ __forceinline__ uint32_t max4(uint32_t v) { return dpp_max<0x4E>(dpp_max<0xB1>(v)); }
__device__ __forceinline__ uint32_t max16(uint32_t v) { return dpp_max<0x140>(dpp_max<0x141>(max4(v))); }
__device__ __forceinline__ uint32_t max_wave(uint32_t v) {
    v = max16(v);
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return std::max(std::max(a, b), std::max(c, d));
}

// ---- a scale for each row ----------------------------------------------------

// TPR threads hold a row, C chunks of eight values each, between its maximum and
// its integers, so X is read once; a row of more than 65536 (LOOP) is read twice.  A
// wave a row up to 1024 columns (no barrier), a workgroup above, of 1024 threads from
// 8192 columns on (bf16, 256 threads of eight or, LOOP, four chunks / 1024: 105 x 12544
// 6.0 / 4.1 us, 4096 x 12544 27.5 / 28.8, 32 x 30000 11.5 / 5.1, 2048 x 30000 50.8 /
// 32.2; below, 4096 x 8192, 16.9 / 19.0).  Bound by the bytes (8192 x 4096 bf16: 16 us in
// a row of calls, 6.2 TB/s), one row by latencies (1 x 4096: 4.0 us, a launch's 2.5 in it).
template <bool F32, int TPR, int C, bool LOOP>
__global__ __launch_bounds__(std::max(TPR, 256)) void quantize_row_kernel(QuantArgs a) {
    constexpr int NT = std::max(TPR, 256), NW = TPR / 64;
    __shared__ uint32_t buf[16];
    const int tid = threadIdx.x, at = tid % TPR;
    const int64_t m = (int64_t)blockIdx.x * (NT / TPR) + tid / TPR;
    if (TPR < 256 && m >= a.M) return;   // (whole waves)
    const char* row = (const char*)a.x + m * a.ldx * (F32 ? 4 : 2);
    Raw8<F32> raw[C];
    auto load = [&](int c0) {   // (without branches: a load behind one is waited for before the next)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + (i * TPR + at) * 8;
            raw[i].read(c + 8 <= a.K ? row + (int64_t)c * (F32 ? 4 : 2) : (const char*)kZeros);
        }
        if ((a.K & 7) != 0)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int c = c0 + (i * TPR + at) * 8;
                if (c < a.K && c + 8 > a.K) raw[i].load(row, c, a.K - c);
            }
    };
    uint32_t top = 0;
    for (int c0 = 0; c0 < a.K; c0 += TPR * 8 * C) {
        load(c0);
#pragma unroll
        for (int i = 0; i < C; ++i) top = std::max(top, raw[i].top());
        if constexpr (!LOOP) break;
    }
    top = max_wave(top);
    if constexpr (NW > 1) {
        if ((tid & 63) == 0) buf[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) top = std::max(top, buf[w]);
    }
    const Scale8 sc(Raw8<F32>::top_value(top));
    if (at == 0) a.s[m * a.lds] = sc.s;
    int8_t* q = a.q + m * a.ldq;
    for (int c0 = 0; c0 < a.K + a.pad; c0 += TPR * 8 * C) {
        if constexpr (LOOP) load(c0);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + (i * TPR + at) * 8;
            float v[8];
            raw[i].values(v);
            store_i8(q + c, to_i8(v, sc), a.K + a.pad - c);
        }
        if constexpr (!LOOP) break;
    }
}

// ---- a scale for each group of columns ----------------------------------------

// A workgroup's chunks of eight columns: `rows` rows of `cpr` chunks, row after
// row; a thread takes every 256th of them.
struct Walk {
    int r, c, dr, dc, cpr;
    __device__ __forceinline__ Walk(int cpr_) : cpr(cpr_) {
        r = threadIdx.x / cpr;
        c = threadIdx.x - r * cpr;
        dr = 256 / cpr;
        dc = 256 - dr * cpr;
    }
    __device__ __forceinline__ void next() {
        r += dr;
        c += dc;
        if (c >= cpr) {
            c -= cpr;
            ++r;
        }
    }
};

// G lanes (2 .. 16) hold a group, sixteen columns each; a row's chunks are padded to
// whole groups.  Bound by the bytes and, half as much, by some 10 instructions an
// element (8192 x 11008 bf16 in groups of 128: 47 us, 5.7 TB/s; eight columns a lane,
// with a scale's two divisions for each eight, took 70).
template <bool F32, int G>
__global__ __launch_bounds__(256) void quantize_group_kernel(QuantArgs a, int rows, int cpr) {
    constexpr int U = 2;
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int rn = (int)std::min<int64_t>(rows, a.M - m0);
    Walk w(cpr);
    while (true) {
        Raw8<F32> raw[U][2];
        int r[U], c[U];
        // (a thread that is past the end stays with its wave: the lanes of a group meet below)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u] = w.r;
            c[u] = w.c * 16;
            w.next();
            const char* row = (const char*)a.x + (m0 + r[u]) * a.ldx * (F32 ? 4 : 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = c[u] + 8 * h;
                if (r[u] < rn && k < a.K) raw[u][h].load(row, k, a.K - k);
                else raw[u][h].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t top = dpp_max<0xB1>(std::max(raw[u][0].top(), raw[u][1].top()));
            if constexpr (G >= 4) top = dpp_max<0x4E>(top);
            if constexpr (G >= 8) top = dpp_max<0x141>(top);
            if constexpr (G >= 16) top = dpp_max<0x140>(top);
            const Scale8 sc(Raw8<F32>::top_value(top));
            u32x2 q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
                raw[u][h].values(v);
                q[h] = to_i8(v, sc);
            }
            const int n = a.K + a.pad - c[u];
            if (r[u] >= rn || n <= 0) continue;
            if (c[u] % (G * 16) == 0 && c[u] < a.K) a.s[(m0 + r[u]) * a.lds + c[u] / (G * 16)] = sc.s;
            int8_t* d = a.q + (m0 + r[u]) * a.ldq + c[u];
            if (n >= 16) {
                *(u32x4a1*)d = u32x4{q[0][0], q[0][1], q[1][0], q[1][1]};
            } else {
                store_i8(d, q[0], n);
                store_i8(d + 8, q[1], n - 8);
            }
        }
        if (__ballot(w.r < rn) == 0) break;
    }
}

// ---- and back ------------------------------------------------------------------

__device__ __forceinline__ u32x2 load_i8(const int8_t* p, int n) {
    u32x2 w = {0, 0};
    if (n >= 8) {
        w = *(const u32x2a1*)p;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    }
    return w;
}
__device__ __forceinline__ float i8_at(u32x2 w, int i) { return (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))); }

// ONCE: past the caches (streaming stores).
template <class V, int ALIGN, bool ONCE>
__device__ __forceinline__ void store_vec(void* p, V v) {
    typedef V U __attribute__((aligned(ALIGN)));
    typedef U __attribute__((address_space(1))) * at;
    if constexpr (ONCE) __builtin_nontemporal_store(v, (at)p);
    else *(at)p = v;
}

// Up to eight values to a row of bf16 or binary32 (any alignment of its elements).
template <bool F32, bool ONCE = false>
__device__ __forceinline__ void store_values(void* row, int64_t c, const float (&v)[8], int n) {
    if constexpr (F32) {
        float* p = (float*)row + c;
        if (n >= 8) {
            store_vec<f32x4, 4, ONCE>(p, f32x4{v[0], v[1], v[2], v[3]});
            store_vec<f32x4, 4, ONCE>(p + 4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        }
    } else {
        uint16_t* p = (uint16_t*)row + c;
        if (n >= 8) {
            store_vec<u32x4, 2, ONCE>(
                p, u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = f32_to_bf16(v[i]);
        }
    }
}

// y = q s, eight columns a thread, four chunks read before the first is used.  Bound
// by the bytes (8192 x 11008 to bf16: 41.5 us, 6.5 TB/s).  ONCE: an output that would
// take much of the last-level cache is written past it (quantised, read back and
// added to, us, into the cache / past it: 90 MB of bf16 82 / 81, 135 MB 129 / 120, 180
// MB 180 / 159; 67 MB 57 / 58).
template <bool F32, bool ONCE>
__global__ __launch_bounds__(256) void dequantize_kernel(QuantArgs a, int rows, int cpr, int shift) {
    constexpr int U = 4;
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int rn = (int)std::min<int64_t>(rows, a.M - m0);
    Walk w(cpr);
    while (w.r < rn) {
        u32x2 q[U];
        float s[U];
        int r[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u] = w.r;
            c[u] = w.c * 8;
            w.next();
            if (r[u] >= rn) continue;
            q[u] = load_i8(a.q + (m0 + r[u]) * a.ldq + c[u], a.K - c[u]);
            s[u] = a.s[(m0 + r[u]) * a.lds + (c[u] >> shift)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r[u] >= rn) continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i8_at(q[u], i) * s[u];
            store_values<F32, ONCE>((char*)a.x + (m0 + r[u]) * a.ldx * (F32 ? 4 : 2), c[u], v, a.K - c[u]);
        }
    }
}

// ---- rows of any alignment into aligned ones -------------------------------------

// A wave a row.
__global__ __launch_bounds__(256) void q8_pack_kernel(const int8_t* src, int64_t lds, int8_t* dst, int64_t ldd, int64_t rows,
                                                      int cols) {
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= rows) return;
    const int8_t* s = src + m * lds;
    int8_t* d = dst + m * ldd;
    for (int c = (threadIdx.x & 63) * 8; c < ldd; c += 512) *(u32x2*)(d + c) = c < cols ? load_i8(s + c, cols - c) : u32x2{0, 0};
}

// ---- the product in 8-bit integers -------------------------------------------------

// (a row or channel of scale NaN stays NaN; the GEMM's rectifier makes it 0)
template <int ACT>
__device__ __forceinline__ float act_keep(float v) {
    if constexpr (ACT == ACT_RELU) return v <= 0.0f ? 0.0f : v;
    return act_t<ACT>(v);
}
template <int ACT, int N>
__device__ __forceinline__ void act_run(f32x4* v) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[i][r] = act_keep<ACT>(v[i][r]);
}
// act of 4 N values.
template <int N>
__device__ __forceinline__ void act_run(int act, f32x4* v) {
    switch (act) {
        case ACT_RELU: return act_run<ACT_RELU, N>(v);
        case ACT_GELU: return act_run<ACT_GELU, N>(v);
        case ACT_GELU_TANH: return act_run<ACT_GELU_TANH, N>(v);
        case ACT_SILU: return act_run<ACT_SILU, N>(v);
    }
}

// A tile's bf16 values, staged in LDS, to rows of any alignment.
template <class T>
__device__ __forceinline__ void store_rows16(uint16_t* D, int64_t ld, int rows, int cols, const lds_t* smem, int tid) {
    __syncthreads();
    constexpr int CPR = T::BN / 8;
    for (int q = tid; q < T::BM * CPR; q += T::NT) {
        const int r = q / CPR, c = (q % CPR) * 8;
        if (r >= rows || c >= cols) continue;
        const u32x4 w = *(const u32x4 __attribute__((address_space(3)))*)(smem + r * staged_ld<T> + c * 2);
        uint16_t* d = D + r * ld + c;
        if (c + 8 <= cols) *(u32x4a2*)d = w;
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

template <class T>
constexpr int staged_ld32 = T::BN * 4 + 16;
// One tile over one split's K steps (of 128 integers).  256 x 256 tiles, one a CU: 1.4
// us a step, as long as of bf16 for twice the work.  MFMAs take 64-68 % of that time
// (48-60 % of the launch's, whose ends are not hidden with one tile a CU), LDS 21-25 %,
// the rest are the waves' waits for each other and for a step's loads; 4096 x 4096 x
// 4096 57 us, 2420 TOPS.  64 x 64 tiles, four a CU, for latency: 509 x 2304 x
// 768 6.2 us, where 128 x 128 take 8.1 and 256 x 256 10.2.  The sums are exact in 32
// bits (K at most 131071); what is past K reads as zeros in both operands, or, in
// the last 16 bytes, as zeros in A.
template <class T, int ACT>
__device__ __forceinline__ void i8_tile(const I8Args& a, int m0, int n0, int split, lds_t* smem, float* edge, int wave,
                                        int lane) {
    const int kp = (a.K + 15) >> 4 << 3;   // 16-bit columns
    const int all = (kp + 63) >> 6, per = (all + a.splits - 1) / a.splits;
    const int s0 = std::min(split * per, all), steps = std::min(per, all - s0);
    const int tail = s0 + steps == all ? kp & 63 : 0;
    const int rows = (int)std::min<int64_t>(a.M - m0, T::BM), cols = a.N - n0;
    Operand<T::HA, false, T::IA, T::NW> A;
    Operand<T::HB, false, T::IB, T::NW> B;
    A.init((const uint16_t*)(a.A + (int64_t)m0 * a.lda) + s0 * 64, a.lda >> 1, rows, steps, tail, wave, lane,
           (const uint16_t*)kZeros);
    B.init((const uint16_t*)(a.B + (int64_t)n0 * a.ldb) + s0 * 64, a.ldb >> 1, cols, steps, tail, wave, lane,
           (const uint16_t*)kZeros);
    // The epilogue's operands are read ahead of the product, into LDS: read after
    // it, row by row, they cost a 128 x 128 tile 4 us of 8.5 (109 x 887 x 144).
    const int tid = wave * 64 + lane;
    if (a.splits == 1) {
        for (int i = tid; i < T::BN; i += T::NT) {
            const int n = n0 + std::min(i, cols - 1);
            edge[i] = a.sb[n];
            edge[T::BN + i] = a.bias != nullptr ? a.bias[n] : 0.0f;
        }
        for (int i = tid; i < T::BM; i += T::NT) edge[2 * T::BN + i] = a.sa[m0 + std::min(i, rows - 1)];
    }
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    if (a.splits > 1) {
        int* P = a.part + ((int64_t)split * a.M + m0) * a.ldp + n0;
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const int row = at.row(ha, i);
                if (row >= rows) continue;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j)
                        if (n0 + at.col(hb, j) < a.ldp) *(i32x4*)(P + row * a.ldp + at.col(hb, j)) = acc[ha][hb][i][j];
            }
        return;
    }
    // One row of fragments (registers: a row at a time), to LDS.  Both types go
    // through it, binary32 half the tile's rows at a time, and leave by one loop in
    // whole row segments: stores beside each fragment's arithmetic are code that is
    // jumped over, and fetched, for every fragment (bf16, 109 x 887 x 144 on 128 x
    // 128 tiles: 8.0 us so, 6.6 now).
    f32x4 sb[2][T::FN], bias[2][T::FN];
    auto columns = [&] {
        asm volatile("" ::: "memory");   // (by each type's branch for itself: nothing of a row is worked out ahead of both)
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) {
                sb[hb][j] = *(const f32x4*)(edge + at.col(hb, j));
                bias[hb][j] = *(const f32x4*)(edge + T::BN + at.col(hb, j));
            }
    };
    auto row_to = [&](int ha, int i, auto&& put) {
        const float sa = edge[2 * T::BN + at.row(ha, i)];
        f32x4 v[2][T::FN];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[hb][j][r] = fmaf((float)acc[ha][hb][i][j][r] * sb[hb][j][r], sa, bias[hb][j][r]);
        act_run<ACT, 2 * T::FN>(&v[0][0]);
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) put(at.row(ha, i), at.col(hb, j), v[hb][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (a.bf16) {
        columns();
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
                row_to(ha, i, [&](int row, int col, f32x4 y) {
                    *(u32x2 __attribute__((address_space(3)))*)(smem + row * staged_ld<T> + col * 2) =
                        u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
                });
        store_rows16<T>((uint16_t*)a.C + (int64_t)m0 * a.ldc + n0, a.ldc, rows, cols, smem, tid);
        return;
    }
    columns();
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
        if (ha) __syncthreads();
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
            row_to(ha, i, [&](int row, int col, f32x4 y) {
                *(f32x4 __attribute__((address_space(3)))*)(smem + (row - ha * T::HA) * staged_ld32<T> + col * 4) = y;
            });
        __syncthreads();
        float* D = (float*)a.C + (int64_t)(m0 + ha * T::HA) * a.ldc + n0;
        constexpr int CPR = T::BN / 4;
        for (int q = tid; q < T::HA * CPR; q += T::NT) {
            const int r = q / CPR, c = (q % CPR) * 4;
            if (r >= rows - ha * T::HA || c >= cols) continue;
            const f32x4 y = *(const f32x4 __attribute__((address_space(3)))*)(smem + r * staged_ld32<T> + c * 4);
            float* d = D + r * a.ldc + c;
            if (c + 4 <= cols) *(f32x4a4*)d = y;
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) d[e] = y[e];
        }
    }
}

template <class T>
constexpr int tile_lds() {
    return std::max(T::LDS, T::BM * staged_ld<T>);
}
template <class T>
constexpr int i8_lds() {
    return std::max(tile_lds<T>(), T::HA * staged_ld32<T>);
}

// H: T, or the tile of half its rows that a last round of unsplit tiles is cut
// into.  An instance for each activation: a switch between them inside an epilogue
// costs its jumps' instruction fetches, 4 us of 9 for the smallest products on
// 128 x 128 tiles.
template <class T, class H, int ACT>
__global__ __launch_bounds__(T::NT, 2) void i8_tile_kernel(I8Args a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[std::max(i8_lds<T>(), i8_lds<H>())];
    __shared__ __attribute__((aligned(16))) float edge[T::BM + 2 * T::BN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)((a.M + T::BM - 1) / T::BM), cols = (a.N + T::BN - 1) / T::BN;
    int tm, tn, split;
    if constexpr (T::BM > H::BM) {
        if (a.splits == 1) {
            int half;
            if (!map_rounds(blockIdx.x, rows, cols, 256, true, tm, tn, half)) return;
            if (half < 0) i8_tile<T, ACT>(a, tm * T::BM, tn * T::BN, 0, (lds_t*)raw, edge, wave, lane);
            else if (tm * T::BM + half * H::BM < a.M)
                i8_tile<H, ACT>(a, tm * T::BM + half * H::BM, tn * T::BN, 0, (lds_t*)raw, edge, wave, lane);
            return;
        }
    }
    if (!map_tile(blockIdx.x, rows, cols, tm, tn, split, a.splits)) return;
    i8_tile<T, ACT>(a, tm * T::BM, tn * T::BN, split, (lds_t*)raw, edge, wave, lane);
}

// Up to four consecutive values of C.
__device__ __forceinline__ void store4(const I8Args& a, int64_t at, f32x4 v, int n) {
    if (n >= 4) {
        if (a.bf16) *(u32x2a1*)((uint16_t*)a.C + at) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        else *(f32x4a4*)((float*)a.C + at) = v;
        return;
    }
#pragma unroll
    for (int r = 0; r < 3; ++r) {
        if (r >= n) break;
        if (a.bf16) ((uint16_t*)a.C)[at + r] = f32_to_bf16(v[r]);
        else ((float*)a.C)[at + r] = v[r];
    }
}

// Four columns a thread: the partial sums, joined exactly, and the epilogue.  Bound by
// latency where it is used most (105 x 1024 in eight parts: 3.9 us), by the parts'
// bytes else (2048 x 4096 in two: 17 us, 4.9 TB/s).
__global__ __launch_bounds__(256) void i8_finish_kernel(I8Args a) {
    const int quads = (a.N + 3) >> 2;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    if (m >= a.M) return;
    const int* p = a.part + m * a.ldp + n;
    const float sa = a.sa[m];
    f32x4 sb, bias;   // (read with the sums, not after them)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = std::min(n + r, a.N - 1);
        sb[r] = a.sb[c];
        bias[r] = a.bias != nullptr ? a.bias[c] : 0.0f;
    }
    i32x4 t = {0, 0, 0, 0};
    constexpr int U = 8;
    for (int s0 = 0; s0 < a.splits; s0 += U) {
        i32x4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = s0 + u < a.splits ? *(const i32x4*)(p + (s0 + u) * a.M * a.ldp) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < U; ++u) t += x[u];
    }
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = fmaf((float)t[r] * sb[r], sa, bias[r]);
    act_run<1>(a.act, &v);
    store4(a, m * a.ldc + n, v, a.N - n);
}

// ---- few tokens ------------------------------------------------------------------------

// Up to sixteen bytes of a row (any alignment), zeros from `n` on.
__device__ __forceinline__ u32x4 load16(const int8_t* p, int n) {
    if (n >= 16) return *(const u32x4a1*)p;
    const u32x2 lo = load_i8(p, n), hi = load_i8(p + 8, n - 8);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// a (rows 0-7 in lanes of low s, and their second 64 bytes in those of high s) and b
// (rows 8-15 likewise) into rows 0-15 of the first and of the second 64 bytes.
__device__ __forceinline__ void exchange(u32x4 a, u32x4 b, u32x4 (&out)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = (int)a[i], y = (int)b[i];
        out[0][i] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xf, 0xc, false);   // (lanes rotated by 8 of 16)
        out[1][i] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false);
    }
}

// At most 16 FM tokens: the weight streams past them, through registers.  A
// workgroup takes a run of output channels, in NF fragments of 16, and its eight
// waves a part of the features each (128 at a step), so every byte of W is read
// once, by one lane, D steps ahead of its use; the waves' sums meet in LDS.
//
// A load takes whole lines, 128 bytes of each of eight rows: lane 16 g + s row s % 8,
// bytes 16 (g + 4 (s / 8)).  Two of them, of a fragment's first and last eight rows,
// make the two multiplications' operands (row s, bytes 16 g and 64 + 16 g) by
// exchanging halves of every 16 lanes.  (As the multiplication wants them, 64 bytes of
// each of 16 rows a load: 32 x 4096 x 11008 21.8 us, 17.0 so; 24 x 11008 x 4096 14.7,
// 12.9.)  W's loads are marked as read once: nothing of it stays in the caches for
// the next layers' (cold, 1 x 32000 x 4096 29.6 us without, 25.9 so, 5.1 TB/s; 1 x 11008
// x 4096 11.8, 10.5, 4.3 TB/s of a launch that takes 2.5 by itself; a weight that the
// last-level cache still holds: 9.7, 9.5).  Two steps ahead: four took 31.6 and 12.3,
// the requests in the other's way; one 9.2 us against 7.1 at 1 x 1024 x 12544.
//
// UNITS > 0: X is bf16 or binary32 and quantised here, by every workgroup for
// itself, into LDS, while the weight's first loads are on their way.  A wave
// holds up to UNITS runs of 512 features in registers between their row's
// maximum and their integers.
template <int FM, int NF, int UNITS, bool F32>
__global__ __launch_bounds__(512) void i8_stream_kernel(I8Args a, int cols) {
    constexpr int NW = 8, D = 2;
    // [M][K to 128, and 16]: at most 8 UNITS runs of 512
    __shared__ __attribute__((aligned(16))) unsigned char xq[UNITS > 0 ? 4096 * UNITS + 256 * FM : 16];
    __shared__ i32x4 red[NW][NF * FM][64];
    __shared__ uint32_t tops[16 * FM];
    __shared__ float sx[16 * FM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, s16 = lane & 15, M = (int)a.M;
    const int n0 = blockIdx.x * cols, left = std::min(cols, a.N - n0);
    const int steps = a.K >> 7, tail = a.K & 127;   // (a last step that is not full is one wave's, at the end)
    const int s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
    const int xld = (a.K + 127) / 128 * 128 + 16;
    const int r8 = s16 & 7, chunk = (g + 4 * (s16 >> 3)) * 16;

    // X's own loads come first: they are waited for first
    const int parts = std::max((a.K + 511) >> 9, 1), units = M * parts;
    Raw8<F32> raw[UNITS > 0 ? UNITS : 1];
    if constexpr (UNITS > 0) {
        if (tid < 16 * FM) tops[tid] = 0;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            // (without branches: a load behind one is waited for with all that follow it)
            const int unit = wave + u * NW, m = unit / parts, c = (unit - m * parts) * 512 + lane * 8;
            const char* p = (const char*)a.x + (m * a.lda + c) * (F32 ? 4 : 2);
            raw[u].read(unit < units && c + 8 <= a.K ? p : (const char*)kZeros);
            if ((a.K & 7) != 0 && unit < units && c < a.K && c + 8 > a.K) raw[u].load(p, 0, a.K - c);
        }
    }
    const int8_t *wp[2 * NF], *xp[2 * FM];
#pragma unroll
    for (int f = 0; f < 2 * NF; ++f) wp[f] = a.B + (int64_t)(n0 + std::min(f * 8 + r8, left - 1)) * a.ldb + chunk;
#pragma unroll
    for (int m = 0; m < 2 * FM; ++m) xp[m] = UNITS > 0 ? nullptr : a.A + std::min(m * 8 + r8, M - 1) * a.lda + chunk;
    u32x4 wb[D][2 * NF], xb[UNITS > 0 ? 1 : D][2 * FM];
    auto load = [&](int i, int s) {
#pragma unroll
        for (int f = 0; f < 2 * NF; ++f) wb[i][f] = load_once<u32x4, 1>(steps > 0 ? wp[f] + s * 128 : (const int8_t*)kZeros);
        if constexpr (UNITS == 0) {
#pragma unroll
            for (int m = 0; m < 2 * FM; ++m) xb[i][m] = load_global<u32x4, 1>(steps > 0 ? xp[m] + s * 128 : (const int8_t*)kZeros);
        }
    };
    // (and the epilogue's operands: a fragment a wave, NF FM of them)
    static_assert(NF * FM <= NW, "a fragment a wave");
    const int ef = wave / FM, em = (wave - ef * FM) * 16 + s16, ec = ef * 16 + g * 4;
    f32x4 sb, bias = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = n0 + std::min(ec + r, left - 1);
        sb[r] = a.sb[n];
        if (a.bias != nullptr) bias[r] = a.bias[n];
    }
    float sa = 0.0f;
    if constexpr (UNITS == 0) sa = a.sa[std::min(em, M - 1)];
    const int last = std::max(s1 - 1, 0);   // (a wave without a step reads one of another's, unused)
#pragma unroll
    for (int i = 0; i < D; ++i) load(i, std::min(s0 + i, last));
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (UNITS > 0) {
        uint32_t top[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) top[u] = max_wave(raw[u].top());
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
            if (lane == 0 && wave + u * NW < units) atomicMax(&tops[(wave + u * NW) / parts], top[u]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int unit = wave + u * NW, m = unit / parts, part = unit - m * parts, c = part * 512 + lane * 8;
            if (unit >= units) break;
            const Scale8 sc(Raw8<F32>::top_value(tops[m]));
            if (part == 0 && lane == 0) sx[m] = sc.s;
            float v[8];
            raw[u].values(v);
            if (c < xld - 16) *(u32x2*)(xq + m * xld + c) = to_i8(v, sc);
        }
        __syncthreads();
    }
    i32x4 acc[NF][FM];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) acc[f][m] = i32x4{0, 0, 0, 0};
    auto multiply = [&](int i, int s) {
        u32x4 w[NF][2];
#pragma unroll
        for (int f = 0; f < NF; ++f) exchange(wb[i][2 * f], wb[i][2 * f + 1], w[f]);
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            u32x4 x[2];
            if constexpr (UNITS > 0) {
                const unsigned char* p = xq + std::min(m * 16 + s16, M - 1) * xld + s * 128 + g * 16;
                x[0] = *(const u32x4*)p;
                x[1] = *(const u32x4*)(p + 64);
            } else {
                exchange(xb[i][2 * m], xb[i][2 * m + 1], x);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[f][m] = MulI8::mul(__builtin_bit_cast(bf16x8, w[f][h]), __builtin_bit_cast(bf16x8, x[h]), acc[f][m]);
        }
    };
    int s = s0;
    for (; s + D < s1; s += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            multiply(i, s + i);
            load(i, std::min(s + D + i, last));
            __builtin_amdgcn_sched_barrier(0);   // (kept in this order: the compiler puts the loads last)
        }
    }
#pragma unroll
    for (int i = 0; i < D; ++i)
        if (s + i < s1) multiply(i, s + i);
    if (tail > 0 && wave == NW - 1) {
        const int n = tail - chunk;
#pragma unroll
        for (int f = 0; f < 2 * NF; ++f) wb[0][f] = load16(wp[f] + steps * 128, n);
        if constexpr (UNITS == 0) {
#pragma unroll
            for (int m = 0; m < 2 * FM; ++m) xb[0][m] = load16(xp[m] + steps * 128, n);
        }
        multiply(0, steps);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m) red[wave][f * FM + m][lane] = acc[f][m];
    __syncthreads();
    if (wave >= NF * FM || em >= M || ec >= left) return;
    i32x4 t = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) t += red[w][wave][lane];
    if constexpr (UNITS > 0) sa = sx[em];
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = fmaf((float)t[r] * sb[r], sa, bias[r]);
    act_run<1>(a.act, &v);
    store4(a, (int64_t)em * a.ldc + n0 + ec, v, left - ec);
}

// ---- backward -----------------------------------------------------------------------

// dz = dy act'(z), what is made of it, and the input's integers in bf16.
// Workgroups of the first kind take sum_rows rows of 512 columns, a wave every
// fourth row; of the second 4 rows of the input.  The product's operand dz x_scale is
// rounded here, once, from binary32 (made from the bf16 dz in the product it would be
// rounded twice), and x's integers become bf16 here, exactly, so that the product's
// loop does nothing but multiply.  For a binary32 dW another pass makes that operand
// of what the rounding left: dz x_scale in two bf16 parts, relative 2^-16 (8192 x 2304 x
// 768, against 64 bits: 2.5e-6 of dW's norm in 138 us a call; one part 1.7e-3, 71 us).
// Bound by the bytes: 8192 x 11008 with 8192 x 4096 of x, 730 MB, 118 us, 6.2 TB/s.
// (Loads behind branches: 120; 8192 x 2304 with 8192 x 768, binary32 dy, 33.4 us against
// 29.8; 333 x 768 with 333 x 12544 14.5, one load of x ahead, against 10.4.)
template <bool F32, int ACT>
__global__ __launch_bounds__(256) void q8_slopes_kernel(Q8GradArgs a, int first, int cols, int zshift) {
    __shared__ float red[4][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const char* const zeros = (const char*)kZeros;
    if ((int)blockIdx.x >= first) {
        const int64_t m = (int64_t)(blockIdx.x - first) * 4 + wave;
        if (m >= a.M) return;
        const int8_t* x = a.x + m * a.ldx;
        uint16_t* d = a.xb + m * a.Kp;
        constexpr int U = 4;
        for (int k0 = lane * 8; k0 < a.Kp; k0 += 512 * U) {
            u32x2 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + 512 * u;
                w[u] = load_global<u32x2, 1>(k + 8 <= a.K ? (const char*)x + k : zeros);
            }
            if ((a.K & 7) != 0)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = k0 + 512 * u;
                    if (k < a.K && k + 8 > a.K) w[u] = load_i8(x + k, a.K - k);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + 512 * u;
                if (k >= a.Kp) break;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = i8_at(w[u], i);
                store_values<false>(d, k, v, 8);
            }
        }
        return;
    }
    const int rb = blockIdx.x / cols, n = (blockIdx.x - rb * cols) * 512 + lane * 8;
    const int left = a.N - n;
    const int64_t m0 = (int64_t)rb * a.sum_rows;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr int U = 4;
    if (n < a.Np) {
        for (int r0 = wave; r0 < a.sum_rows; r0 += 4 * U) {
            Raw8<F32> dy[U];
            u32x2 z[U];
            float zs[U], xs[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {   // (without branches: see quantize_row_kernel)
                const int64_t m = m0 + r0 + 4 * u;
                const bool on = m < a.M, whole = on && left >= 8;
                dy[u].read(whole ? (const char*)a.dy + (m * a.lddy + n) * (F32 ? 4 : 2) : zeros);
                if constexpr (ACT != ACT_NONE) {
                    z[u] = load_global<u32x2, 1>(whole ? (const char*)a.z + m * a.ldz + n : zeros);
                    zs[u] = load_global<float, 4>(on ? (const char*)(a.zs + m * a.ldzs + (n >> zshift)) : zeros);
                }
                xs[u] = load_global<float, 4>(on && a.xs != nullptr ? (const char*)(a.xs + m) : zeros);
            }
            if ((a.N & 7) != 0 && left < 8)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t m = m0 + r0 + 4 * u;
                    if (m >= a.M) continue;
                    dy[u].load((const char*)a.dy + m * a.lddy * (F32 ? 4 : 2), n, left);
                    if constexpr (ACT != ACT_NONE) z[u] = load_i8(a.z + m * a.ldz + n, left);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t m = m0 + r0 + 4 * u;
                float g[8];
                dy[u].values(g);
                if constexpr (ACT != ACT_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] *= act_slope<ACT>(i8_at(z[u], i) * zs[u]);
                }
                if (m < a.M) {
                    if (a.dz != nullptr) store_values<false>(a.dz + m * a.lddz, n, g, left);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += g[i];
                }
                if (a.a != nullptr && m < a.Mr) {   // (rows from M on: zeros)
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = m < a.M ? g[i] * xs[u] : 0.0f;
                    if (a.low)
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] = bf16_rest(g[i]);
                    store_values<false>(a.a + m * a.Np, n, g, 8);
                }
            }
        }
    }
    if (a.dbias == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave][lane * 8 + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 512; i += 256) {
        const int c = (blockIdx.x - rb * cols) * 512 + i;
        if (c < a.Np) a.dbp[(int64_t)rb * a.Np + c] = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
    }
}

// dbias of 32 columns from its column sums, every NT / 32-th sum a thread, in a fixed
// order whatever NT is: eight interleaved series of sums, then those.
template <int NT>
__device__ __forceinline__ void q8_dbias(const Q8GradArgs& a, int n0, float* red) {
    const int c = threadIdx.x & 31, grp = threadIdx.x >> 5, n = n0 + c;
    const int parts = (int)((a.M + a.sum_rows - 1) / a.sum_rows);
    if (grp < 8) {
        constexpr int U = 8;
        float t = 0.0f;
        for (int i0 = grp; i0 < parts; i0 += 8 * U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u] = i0 + 8 * u < parts && n < a.N ? a.dbp[(int64_t)(i0 + 8 * u) * a.Np + n] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) t += x[u];
        }
        red[grp * 32 + c] = t;
    }
    __syncthreads();
    if (grp == 0 && n < a.N)
        a.dbias[n] = ((red[c] + red[32 + c]) + (red[64 + c] + red[96 + c])) +
                     ((red[128 + c] + red[160 + c]) + (red[192 + c] + red[224 + c]));
}

// Four values of a row of K, zeros past it.
__device__ __forceinline__ f32x4 load4_f32(const float* row, int k, int K) {
    if (k + 4 <= K) return *(const f32x4a4*)(row + k);
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 3; ++r)
        if (k + r < K) v[r] = row[k + r];
    return v;
}

// A tile of dW = a^T . xb over one split of the rows (64 a step), both operands read
// across their rows.  256 x 256 tiles, one a CU, come at 1.43 us a step, 1500 TFLOP/s in
// full rounds (8192 x 11008 x 4096, two rounds and 0.69: 570 us, 1300); 128 x 128 tiles,
// two a CU, where the result is small (8192 x 2304 x 768 in four parts: 33 us).  The
// workgroups past the tiles make dbias, which spares small calls a launch (unsplit
// ones: else the launch that joins the partials does).
template <class T>
__global__ __launch_bounds__(T::NT, 2) void q8_product_kernel(Q8GradArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char raw[tile_lds<T>()];
    lds_t* smem = (lds_t*)raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tm, tn, split;
    const int rows = (a.N + T::BM - 1) / T::BM, cols = (a.K + T::BN - 1) / T::BN;
    if ((int)blockIdx.x >= rows * cols * a.splits) {
        q8_dbias<T::NT>(a, (blockIdx.x - rows * cols * a.splits) * 32, (float*)raw);
        return;
    }
    if (!map_tile(blockIdx.x, rows, cols, tm, tn, split, a.splits)) return;
    const int n0 = tm * T::BM, k0 = tn * T::BN;
    const int all = a.Mr >> 6, per = (all + a.splits - 1) / a.splits;
    const int s0 = std::min(split * per, all), steps = std::min(per, all - s0);
    Operand<T::HA, true, T::IA, T::NW> A;
    Operand<T::HB, true, T::IB, T::NW> B;
    A.init(a.a + (int64_t)s0 * 64 * a.Np + n0, a.Np, a.Np - n0, steps, 0, wave, lane);
    B.init(a.xb + (int64_t)s0 * 64 * a.Kp + k0, a.Kp, a.Kp - k0, steps, s0 + steps == all ? (int)(a.M & 63) : 0, wave, lane);
    Acc<T> acc;
    main_loop<T>(A, B, steps, smem, wave, lane, acc);
    const Place<T> at(wave, lane);
    if (a.splits == 1 && !a.dw_f32) {
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                    for (int j = 0; j < T::FN; ++j) {
                        const f32x4 v = acc[ha][hb][i][j];
                        *(u32x2 __attribute__((address_space(3)))*)(smem + at.row(ha, i) * staged_ld<T> + at.col(hb, j) * 2) =
                            u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                    }
        store_rows16<T>((uint16_t*)a.dw + (int64_t)n0 * a.lddw + k0, a.lddw, a.N - n0, a.K - k0, smem, wave * 64 + lane);
        return;
    }
    if (a.splits == 1) {
        if (a.low)
#pragma unroll
            for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                for (int i = 0; i < T::FM; ++i) {
                    const int row = n0 + at.row(ha, i);
                    if (row >= a.N) continue;
                    const float* d = (const float*)a.dw + row * a.lddw;
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int j = 0; j < T::FN; ++j) acc[ha][hb][i][j] += load4_f32(d, k0 + at.col(hb, j), a.K);
                }
        store_tile<T>(acc, 1.0f, a.dw, true, a.lddw, k0, a.N - n0, a.K - k0, smem, wave, lane,
                      [&](int r) { return (int64_t)n0 + r; });
        return;
    }
    float* P = a.part + ((int64_t)split * a.N + n0) * a.Kp + k0;
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            if (n0 + at.row(ha, i) >= a.N) continue;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
                    if (k0 + at.col(hb, j) < a.Kp)
                        *(f32x4*)(P + (int64_t)at.row(ha, i) * a.Kp + at.col(hb, j)) = acc[ha][hb][i][j];
        }
}

// dW from its partials (and, in a second pass, from itself), eight columns a thread; then dbias.
__global__ __launch_bounds__(256) void q8_finish_kernel(Q8GradArgs a, int first) {
    __shared__ float red[256];
    if ((int)blockIdx.x >= first) {
        q8_dbias<256>(a, (blockIdx.x - first) * 32, red);
        return;
    }
    const int cpr = a.Kp >> 3;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = i / cpr;
    const int k = (int)(i - n * cpr) * 8;
    if (n >= a.N) return;
    const float* p = a.part + n * a.Kp + k;
    const int64_t sp = (int64_t)a.N * a.Kp;
    f32x4 lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
    constexpr int U = 4;
    for (int s0 = 0; s0 < a.splits; s0 += U) {
        f32x4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = s0 + u < a.splits;
            x[u] = on ? *(const f32x4*)(p + (s0 + u) * sp) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            y[u] = on ? *(const f32x4*)(p + (s0 + u) * sp + 4) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo += x[u];
            hi += y[u];
        }
    }
    if (a.low) {
        const float* d = (const float*)a.dw + n * a.lddw;
        lo += load4_f32(d, k, a.K);
        hi += load4_f32(d, k + 4, a.K);
    }
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    if (a.dw_f32) store_values<true>((float*)a.dw + n * a.lddw, k, v, a.K - k);
    else store_values<false>((uint16_t*)a.dw + n * a.lddw, k, v, a.K - k);
}

using I256 = LTile<2, 4, 4, 2, false, false, MulI8>;
using I256Half = LTile<2, 4, 2, 2, false, false, MulI8>;
using I64 = LTile<2, 2, 1, 1, false, false, MulI8>;
using I128 = LTile<2, 2, 2, 2, false, false, MulI8>;
using G256 = LTile<2, 4, 4, 2, true, true>;
using G128 = LTile<2, 2, 2, 2, true, true>;

template <int N>
using Int = std::integral_constant<int, N>;

constexpr int64_t kOnceBytes = int64_t(100) << 20;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
template <class F>
hipError_t by_act(int act, F&& f) {
    switch (act) {
        case ACT_RELU: return f(Int<ACT_RELU>{});
        case ACT_GELU: return f(Int<ACT_GELU>{});
        case ACT_GELU_TANH: return f(Int<ACT_GELU_TANH>{});
        case ACT_SILU: return f(Int<ACT_SILU>{});
        default: return f(Int<ACT_NONE>{});
    }
}
int log2i(int v) { return 31 - __builtin_clz((unsigned)v); }

// Rows of a workgroup that walks chunks: about 1024 of them, fewer (to 256) until
// there are two workgroups a CU (509 x 770 binary32 in groups of 64: 6.1 us with
// 1024, 4.1 so).
int walk_rows(int64_t M, int cpr) {
    const int64_t chunks = std::min<int64_t>(1024, std::max<int64_t>(256, M * cpr / 512));
    return (int)std::max<int64_t>(1, std::min<int64_t>(M, chunks / cpr));
}

template <bool F32>
hipError_t quantize(const QuantArgs& a, hipStream_t st) {
    if (a.group == 0) {
        const int K = a.K + a.pad;
        const dim3 waves((unsigned)up(a.M, 4)), wgs((unsigned)a.M), b(256), wide(1024);
        if (K <= 512) return launch_kernel(quantize_row_kernel<F32, 64, 1, false>, waves, b, st, a);
        if (K <= 1024) return launch_kernel(quantize_row_kernel<F32, 64, 2, false>, waves, b, st, a);
        if (K <= 2048) return launch_kernel(quantize_row_kernel<F32, 256, 1, false>, wgs, b, st, a);
        if (K <= 4096) return launch_kernel(quantize_row_kernel<F32, 256, 2, false>, wgs, b, st, a);
        if (K <= 8192) return launch_kernel(quantize_row_kernel<F32, 256, 4, false>, wgs, b, st, a);
        // (a launch counts its threads in 32 bits, so 2^22 rows and more take 256 each: bf16, one
        // row less / these, 8200 columns 20.3 / 20.0 ms, 12544 27.6 / 27.8, 16400 36.9 / 43.7)
        if (a.M * 1024 > (int64_t)UINT32_MAX)
            return K <= 16384 ? launch_kernel(quantize_row_kernel<F32, 256, 8, false>, wgs, b, st, a)
                              : launch_kernel(quantize_row_kernel<F32, 256, 4, true>, wgs, b, st, a);
        if (K <= 16384) return launch_kernel(quantize_row_kernel<F32, 1024, 2, false>, wgs, wide, st, a);
        if (K <= 32768) return launch_kernel(quantize_row_kernel<F32, 1024, 4, false>, wgs, wide, st, a);
        if (K <= 65536) return launch_kernel(quantize_row_kernel<F32, 1024, 8, false>, wgs, wide, st, a);
        return launch_kernel(quantize_row_kernel<F32, 1024, 4, true>, wgs, wide, st, a);
    }
    const int cpr = (int)up(a.K, a.group) * (a.group / 16), rows = walk_rows(a.M, cpr);
    const dim3 grid((unsigned)up(a.M, rows)), b(256);
    switch (a.group) {
        case 32: return launch_kernel(quantize_group_kernel<F32, 2>, grid, b, st, a, rows, cpr);
        case 64: return launch_kernel(quantize_group_kernel<F32, 4>, grid, b, st, a, rows, cpr);
        case 128: return launch_kernel(quantize_group_kernel<F32, 8>, grid, b, st, a, rows, cpr);
        default: return launch_kernel(quantize_group_kernel<F32, 16>, grid, b, st, a, rows, cpr);
    }
}

}  // namespace

hipError_t launch_quantize(const QuantArgs& a, hipStream_t st) { return a.f32 ? quantize<true>(a, st) : quantize<false>(a, st); }

hipError_t launch_dequantize(const QuantArgs& a, hipStream_t st) {
    const int cpr = (int)up(a.K, 8), rows = walk_rows(a.M, cpr), shift = a.group == 0 ? 31 : log2i(a.group);
    const dim3 grid((unsigned)up(a.M, rows));
    const bool once = a.M * a.K * (a.f32 ? 4 : 2) >= kOnceBytes;
    auto go = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value != 0;
        return once ? launch_kernel(dequantize_kernel<F32, true>, grid, dim3(256), st, a, rows, cpr, shift)
                    : launch_kernel(dequantize_kernel<F32, false>, grid, dim3(256), st, a, rows, cpr, shift);
    };
    return a.f32 ? go(Int<1>{}) : go(Int<0>{});
}

hipError_t launch_q8_pack(const int8_t* src, int64_t lds, int8_t* dst, int64_t ldd, int64_t rows, int cols, hipStream_t st) {
    return launch_kernel(q8_pack_kernel, dim3((unsigned)up(rows, 4)), dim3(256), st, src, lds, dst, ldd, rows, cols);
}

hipError_t launch_i8_product(const I8Args& a, hipStream_t st) {
    // (halved tiles of a last round: at most 128 workgroups more)
    const dim3 grid((unsigned)(up(a.M, a.tile) * up(a.N, a.tile) * a.splits + (a.tile == 256 && a.splits == 1 ? 128 : 0)));
    return by_act(a.splits > 1 ? ACT_NONE : a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        switch (a.tile) {
            case 256: return launch_kernel(i8_tile_kernel<I256, I256Half, ACT>, grid, dim3(I256::NT), st, a);
            case 128: return launch_kernel(i8_tile_kernel<I128, I128, ACT>, grid, dim3(I128::NT), st, a);
            default: return launch_kernel(i8_tile_kernel<I64, I64, ACT>, grid, dim3(I64::NT), st, a);
        }
    });
}

hipError_t launch_i8_stream(const I8Args& a, hipStream_t st) {
    // every CU a run of channels, at most 64 of them at a time
    const int passes = (int)up(a.N, 256 * 64), cols = (int)up(a.N, 256 * passes);
    const dim3 grid((unsigned)up(a.N, cols)), b(512);
    // (a row without features takes a run too: its scale is made there)
    const int units = a.quantise ? (int)up(a.M * std::max<int64_t>(up(a.K, 512), 1), 8) : 0;
    auto go = [&](auto fm, auto nf, auto un, auto f32) {
        return launch_kernel(i8_stream_kernel<decltype(fm)::value, decltype(nf)::value, decltype(un)::value,
                                                  decltype(f32)::value>, grid, b, st, a, cols);
    };
    auto by_units = [&](auto fm, auto nf) {
        if (units == 0) return go(fm, nf, Int<0>{}, Int<0>{});
        if constexpr (decltype(fm)::value == 1) {
            if (a.x_f32) return units <= 1 ? go(fm, nf, Int<1>{}, Int<1>{}) : units <= 4 ? go(fm, nf, Int<4>{}, Int<1>{})
                                                                                        : go(fm, nf, Int<8>{}, Int<1>{});
            return units <= 1 ? go(fm, nf, Int<1>{}, Int<0>{}) : units <= 4 ? go(fm, nf, Int<4>{}, Int<0>{})
                                                                            : go(fm, nf, Int<8>{}, Int<0>{});
        } else {
            return a.x_f32 ? go(fm, nf, Int<8>{}, Int<1>{}) : go(fm, nf, Int<8>{}, Int<0>{});
        }
    };
    auto by_cols = [&](auto fm) {
        return cols <= 16 ? by_units(fm, Int<1>{}) : cols <= 32 ? by_units(fm, Int<2>{})
               : cols <= 48 ? by_units(fm, Int<3>{}) : by_units(fm, Int<4>{});
    };
    return a.M <= 16 ? by_cols(Int<1>{}) : by_cols(Int<2>{});
}

hipError_t launch_i8_finish(const I8Args& a, hipStream_t st) {
    return launch_kernel(i8_finish_kernel, dim3((unsigned)up(a.M * up(a.N, 4), 256)), dim3(256), st, a);
}

hipError_t launch_q8_slopes(const Q8GradArgs& a, hipStream_t st) {
    const int cols = (int)up(a.Np, 512), shift = a.zgroup == 0 ? 31 : log2i(a.zgroup);
    const int64_t rows = a.a != nullptr ? a.Mr : a.M;
    const int64_t first = up(rows, a.sum_rows) * cols, second = a.xb != nullptr && !a.low ? up(a.M, 4) : 0;
    const dim3 grid((unsigned)(first + second));
    return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return a.dy_f32 ? launch_kernel(q8_slopes_kernel<true, ACT>, grid, dim3(256), st, a, (int)first, cols, shift)
                        : launch_kernel(q8_slopes_kernel<false, ACT>, grid, dim3(256), st, a, (int)first, cols, shift);
    });
}

hipError_t launch_q8_product(const Q8GradArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)(up(a.N, a.tile) * up(a.K, a.tile) * a.splits + (a.dbias != nullptr && a.splits == 1 ? up(a.N, 32) : 0)));
    return a.tile == 256 ? launch_kernel(q8_product_kernel<G256>, grid, dim3(G256::NT), st, a)
                         : launch_kernel(q8_product_kernel<G128>, grid, dim3(G128::NT), st, a);
}

hipError_t launch_q8_finish(const Q8GradArgs& a, hipStream_t st) {
    const int64_t first = a.dw != nullptr && a.splits > 1 ? up((int64_t)a.N * (a.Kp >> 3), 256) : 0;
    const int64_t second = a.dbias != nullptr ? up(a.N, 32) : 0;
    return launch_kernel(q8_finish_kernel, dim3((unsigned)(first + second)), dim3(256), st, a, (int)first);
}

}  // namespace mkp

// ns_f8.hip -- gfx950 kernels of the layers in 8-bit floating point with a scale for
// each block of 128 (include/ns.h, ns_f8_*): matrices to 8-bit floats and back, and
// the product C = beta C + A B^T.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "ns.h"
#include "ns_device.h"
#include "ns_f8.h"

namespace ns {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// f(0), f(1), .. f(N - 1) with the numbers as constants (immediates of builtins).
template <typename F, int... I>
__device__ __forceinline__ void unroll_of(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unroll(F&& f)
{
    unroll_of(f, std::make_integer_sequence<int, N>{});
}

// ---------------------------------------------------------------------------
// Values to 8-bit floats and back.

template <int FMT> constexpr float kTop = FMT == NS_F8_E4M3 ? 448.f : 57344.f;

// The scale of a block from the largest magnitude's bits: NaN for Inf or NaN.
template <int FMT, bool POW2>
__device__ __forceinline__ float f8_scale(uint32_t m)
{
    if (m >= 0x7F800000u)
        return __uint_as_float(0x7FC00000u);
    if constexpr (POW2) {
        // m = f 2^x with f in [1, 2), top = 1.75 2^h: top 2^e >= m first holds at
        // e = x - h when f <= 1.75, else at x - h + 1 (subnormals: 2^-126)
        constexpr int h = FMT == NS_F8_E4M3 ? 8 : 15;
        const int e = (int)(m >> 23) - 127 - h + ((m & 0x7FFFFFu) > 0x600000u);
        return m < 0x00800000u || e < -126 ? 0x1p-126f : __uint_as_float((uint32_t)(e + 127) << 23);
    }
    return fmaxf(__uint_as_float(m) / kTop<FMT>, 0x1p-126f);
}

// What a block's values are divided by: its scale and the scale's reciprocal, exact for
// powers of two, else within 2 units of its last place.
struct Divisor { float s, inv; };
template <bool POW2>
__device__ __forceinline__ Divisor divisor(float s)
{
    if constexpr (POW2)
        return {s, __uint_as_float(0x7F000000u - __float_as_uint(s))};   // (NaN: not used)
    return {s, __builtin_amdgcn_rcpf(s)};
}

// x / s of eight values such that rounding them to 8-bit floats is rounding the quotients
// themselves. Power-of-two scales: the quotients, exactly. Otherwise x (1 / s), off by a
// few units of its last place, is good enough unless it lies that near to a border between
// 8-bit floats, which all have 19 zeros at the end: then the nearest fp32 to the quotient,
// whose last bit is set where the remainder says that the quotient lies beside it, and on
// which side. A fused multiply-add gives the remainder exactly (for tiny scales from 2^60
// times the values, so that it is not subnormal). Zeros go the same way, though no border is
// near: 8192 x 6144 values half of which are 0 take 41 us instead of 38 (bf16, rows), and
// the same as others in the other forms and in fp32.
template <bool POW2>
__device__ __forceinline__ void quotients(const float (&x)[8], const Divisor& d, float (&r)[8])
{
    uint32_t near = ~0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r[e] = x[e] * d.inv;
        if constexpr (!POW2)
            near = min(near, (__float_as_uint(r[e]) + 8) & 0x7FFFFu);
    }
    if constexpr (!POW2)
        if (near <= 16) {
            const float mul = d.s < 0x1p-60f ? 0x1p60f : 1.f, s = d.s * mul;
            const float inv = 1.f / s;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = x[e] * mul;
                float q = v * inv;
                q = fmaf(fmaf(-q, s, v), inv, q);
                const float left = fmaf(-q, s, v);
                const uint32_t bits = __float_as_uint(q);
                const bool beyond = (left > 0.f) == (v > 0.f);
                if (left != 0.f && q != 0.f)
                    q = __uint_as_float((beyond ? bits : bits - 1) | 1u);
                r[e] = q;
            }
        }
}

// Four floats as four 8-bit ones.
template <int FMT>
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d)
{
    int w = 0;
    if constexpr (FMT == NS_F8_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return (uint32_t)w;
}

// The largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
}

template <bool POW2>
__device__ __forceinline__ void put_scale(char* base, int64_t at, float s)
{
    if constexpr (POW2)
        gbl(base)[at] = (char)(s == s ? __float_as_uint(s) >> 23 : 255u);
    else
        *(NS_GLOBAL float*)gbl(base + 4 * at) = s;
}

// Bytes i of four words as one word each (a 4 x 4 transpose).
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4])
{
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u), cd = __builtin_amdgcn_perm(d, c, 0x05010400u);
    const uint32_t AB = __builtin_amdgcn_perm(b, a, 0x07030602u), CD = __builtin_amdgcn_perm(d, c, 0x07030602u);
    o[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
    o[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
    o[2] = __builtin_amdgcn_perm(CD, AB, 0x05040100u);
    o[3] = __builtin_amdgcn_perm(CD, AB, 0x07060302u);
}

// Eight values of each of a thread's eight rows, 0 past the end, as fp32 on request: bf16
// ones stay packed (half the registers, and their magnitudes compare in pairs), columns
// 8 cg .. + 7; fp32 ones are columns 4 cg .. + 3 and 64 + 4 cg .. + 3, so that 16 lanes
// read and write whole lines.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <int DT> struct Patch;
template <> struct Patch<0> {
    u32x4 w[8];
    static __device__ __forceinline__ int column(int cg, int e) { return 8 * cg + e; }
    static __device__ __forceinline__ int lanes_of(int column) { return column >> 3; }
    __device__ __forceinline__ void clear(int p) { w[p] = u32x4{0u, 0u, 0u, 0u}; }
    // Lanes at a row's end read its last 16 bytes, with the others and without a branch;
    // `settle`, after all loads, moves these values to their places. (Value by value
    // they wait for memory once a row: 8 of 2043 x 6101 took 85 us instead of 71.) Rows of fewer
    // values go one by one.
    __device__ __forceinline__ void load(int p, const bf16* row, int cg, int cols, bool whole)
    {
        const int c = 8 * cg;
        if (whole) {
            w[p] = load16_any(row + min(c, cols - 8));
        } else {
            clear(p);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols)
                    w[p][e >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, gbl(row)[c + e]) << (16 * (e & 1));
        }
    }
    __device__ __forceinline__ void settle(int cg, int cols)
    {
        const int over = 8 * cg - (cols - 8);
        if (over <= 0)
            return;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            u32x4 v = w[p];
            if (over & 4)
                v = u32x4{v[2], v[3], 0u, 0u};
            if (over & 2)
                v = u32x4{v[1], v[2], v[3], 0u};
            if (over & 1)
                v = u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], 2), __builtin_amdgcn_alignbyte(v[2], v[1], 2),
                          __builtin_amdgcn_alignbyte(v[3], v[2], 2), v[3] >> 16};
            w[p] = over < 8 ? v : u32x4{0u, 0u, 0u, 0u};
        }
    }
    __device__ __forceinline__ float at(int p, int e) const
    {
        return __uint_as_float(e & 1 ? w[p][e >> 1] & 0xFFFF0000u : w[p][e >> 1] << 16);
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                      __builtin_bit_cast(u16x2, b)));
    }
    __device__ __forceinline__ uint32_t row_max(int p) const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = larger(m, w[p][i] & 0x7FFF7FFFu);
        return max(m << 16, m & 0xFFFF0000u);
    }
    // of all rows that 4 lanes of a wavefront hold, by column
    __device__ __forceinline__ void column_max(uint32_t (&m)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                v = larger(v, w[p][i] & 0x7FFF7FFFu);
            v = larger(v, (uint32_t)__shfl_xor((int)v, 16, 64));
            v = larger(v, (uint32_t)__shfl_xor((int)v, 32, 64));
            m[2 * i] = v << 16;
            m[2 * i + 1] = v & 0xFFFF0000u;
        }
    }
};
template <> struct Patch<1> {
    float x[8][8];
    static __device__ __forceinline__ int column(int cg, int e) { return (e < 4 ? 0 : 60) + 4 * cg + e; }
    static __device__ __forceinline__ int lanes_of(int column) { return (column & 63) >> 2; }
    __device__ __forceinline__ void clear(int p)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[p][e] = 0.f;
    }
    // (fp32 rows gain nothing by loads of their last 16 bytes: 4 of 2043 x 6144 in 58 us
    // instead of 46)
    __device__ __forceinline__ void load(int p, const float* row, int cg, int cols, bool)
    {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            const int c = column(cg, h);
            if (c + 4 <= cols) {
                const f32x4 v = __builtin_bit_cast(f32x4, load16_any(row + c));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[p][h + e] = v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[p][h + e] = c + e < cols ? gbl(row)[c + e] : 0.f;
            }
        }
    }
    __device__ __forceinline__ void settle(int, int) {}
    __device__ __forceinline__ float at(int p, int e) const { return x[p][e]; }
    __device__ __forceinline__ uint32_t row_max(int p) const
    {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max(m, mag(x[p][e]));
        return m;
    }
    __device__ __forceinline__ void column_max(uint32_t (&m)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t v = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                v = max(v, mag(x[p][e]));
            v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
            m[e] = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
        }
    }
};

// A workgroup takes a tile of 128 x 128 values, which holds whole blocks of either
// form: thread t the rows 8 (t / 16) .. + 7 and the columns of lane t % 16 (Patch), so that
// values are read once for both forms. Row blocks lie in 16 lanes, column
// blocks in a thread's 8 rows, 4 of a wavefront's lanes and 4 wavefronts; one lane for
// each block divides, the others take what it finds from LDS. The transposed bytes cross
// through LDS: a thread has 8 bytes in a row of each of 8 columns, stored at 8-byte place
// (t / 16) ^ (t % 16) of the column, which keeps the lanes of a store apart. Squares
// give the same bytes both ways, which are turned instead. Memory bounds it: 8192 x 6144
// bf16 values to both forms in 38 us, 5.2 TB/s (46 between calls that leave 200 MB of
// written lines behind), to one in 27; 8172 x 6144 fp32 ones, squares, to one in 46, 5.4 TB/s.
template <int DT, int FMT, bool POW2, int N>
__global__ __launch_bounds__(kThreads) void k_f8_quantize(const F8RowsBatchOf<N> batch)
{
    using T = typename Elt<DT>::type;
    __shared__ __attribute__((aligned(16))) char bytes[16384];
    __shared__ uint32_t colmax[4][128];
    __shared__ __attribute__((aligned(16))) float row_s[128], row_inv[128], col_s[128], col_inv[128];
    const F8RowsItem it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin;
    const int tr = b / it.ntn, tc = b - tr * it.ntn;
    const int r0 = tr * 128, c0 = tc * 128;
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
    const bool square = batch.square != 0;
    const int rows = min(128, it.rows - r0), cols = min(128, it.cols - c0);

    const bool whole = it.cols >= 16 / (int)sizeof(T);
    Patch<DT> x;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = 8 * rg + p;
        if (r < rows)
            x.load(p, reinterpret_cast<const T*>(it.values) + (r0 + r) * it.ldv + c0, cg, cols, whole);
        else
            x.clear(p);
    }
    if (whole)
        x.settle(cg, cols);

    // The largest magnitude of a row block for lane p of its 16 (p < 8), or of the square.
    uint32_t mine = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        uint32_t m = x.row_max(p);
        if (!square)
            m = max16(m);
        mine = square ? max(mine, m) : cg == p ? m : mine;
    }
    if (square) {
        mine = max16(mine);
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 16, 64));
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 32, 64));
        if ((t & 63) == 0)
            colmax[wave][0] = mine;
        __syncthreads();
        mine = max(max(colmax[0][0], colmax[1][0]), max(colmax[2][0], colmax[3][0]));
    } else if (it.qt) {
        uint32_t m[8];
        x.column_max(m);
        if ((t & 48) == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                colmax[wave][x.column(cg, e)] = m[e];
    }
    Divisor all{};   // of a square
    if (square) {
        all = divisor<POW2>(f8_scale<FMT, POW2>(mine));
        if (t == 0) {
            if (it.q)
                put_scale<POW2>(it.scale, (int64_t)tc * it.lds + tr, all.s);
            if (it.qt)
                put_scale<POW2>(it.scale_t, (int64_t)tr * it.ldst + tc, all.s);
        }
    } else if (it.q && cg < 8) {
        const int r = 8 * rg + cg;
        const Divisor d = divisor<POW2>(f8_scale<FMT, POW2>(mine));
        row_s[r] = d.s;
        row_inv[r] = d.inv;
        if (r < rows)
            put_scale<POW2>(it.scale, (int64_t)tc * it.lds + r0 + r, d.s);
    }
    // (a row's lanes are of one wavefront)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    auto eight = [&](const float (&v)[8], const Divisor& d) __attribute__((always_inline)) {
        float r[8];
        quotients<POW2>(v, d, r);
        const u32x2 w = {pack_f8<FMT>(r[0], r[1], r[2], r[3]), pack_f8<FMT>(r[4], r[5], r[6], r[7])};
        return d.s == d.s ? w : u32x2{0u, 0u};
    };
    u32x2 w[8];
    if (it.q || square) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int r = 8 * rg + p;
            w[p] = eight({x.at(p, 0), x.at(p, 1), x.at(p, 2), x.at(p, 3), x.at(p, 4), x.at(p, 5), x.at(p, 6), x.at(p, 7)},
                         square ? all : Divisor{row_s[r], row_inv[r]});
            if (!it.q || r >= rows)
                continue;
            char* q = it.q + (int64_t)(r0 + r) * it.ldq + c0;
            if (DT == 0 && x.column(cg, 7) < cols) {
                *(NS_GLOBAL u32x2*)gbl(q + x.column(cg, 0)) = w[p];
            } else if (DT == 1 && x.column(cg, 7) < cols) {
                *(NS_GLOBAL uint32_t*)gbl(q + x.column(cg, 0)) = w[p].x;
                *(NS_GLOBAL uint32_t*)gbl(q + x.column(cg, 4)) = w[p].y;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (x.column(cg, e) < cols)
                        gbl(q)[x.column(cg, e)] = (char)((e < 4 ? w[p].x : w[p].y) >> (8 * (e & 3)));
            }
        }
    }
    if (!it.qt)
        return;
    auto turned = [&](int e, u32x2 v) __attribute__((always_inline)) {
        *reinterpret_cast<u32x2*>(bytes + x.column(cg, e) * 128 + ((rg ^ cg) << 3)) = v;
    };
    if (square) {
        uint32_t lo[4], hi[4];
        turn4(w[0].x, w[1].x, w[2].x, w[3].x, lo);
        turn4(w[4].x, w[5].x, w[6].x, w[7].x, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            turned(e, u32x2{lo[e], hi[e]});
        turn4(w[0].y, w[1].y, w[2].y, w[3].y, lo);
        turn4(w[4].y, w[5].y, w[6].y, w[7].y, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            turned(4 + e, u32x2{lo[e], hi[e]});
    } else {
        __syncthreads();
        if (t < 128) {
            const Divisor d = divisor<POW2>(
                f8_scale<FMT, POW2>(max(max(colmax[0][t], colmax[1][t]), max(colmax[2][t], colmax[3][t]))));
            col_s[t] = d.s;
            col_inv[t] = d.inv;
            if (t < cols)
                put_scale<POW2>(it.scale_t, (int64_t)tr * it.ldst + c0 + t, d.s);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = x.column(cg, e);
            turned(e, eight({x.at(0, e), x.at(1, e), x.at(2, e), x.at(3, e), x.at(4, e), x.at(5, e), x.at(6, e), x.at(7, e)},
                            Divisor{col_s[c], col_inv[c]}));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = t + kThreads * i, c = u >> 3, g = (u & 7) * 2;
        const int turn = x.lanes_of(c);
        const u32x2 lo = *reinterpret_cast<const u32x2*>(bytes + c * 128 + ((g ^ turn) << 3));
        const u32x2 hi = *reinterpret_cast<const u32x2*>(bytes + c * 128 + (((g + 1) ^ turn) << 3));
        const u32x4 v = {lo.x, lo.y, hi.x, hi.y};
        if (c >= cols)
            continue;
        char* q = it.qt + (int64_t)(c0 + c) * it.ldqt + r0 + 8 * g;
        if (8 * g + 16 <= rows) {
            *(NS_GLOBAL u32x4*)gbl(q) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * g + e < rows)
                    gbl(q)[e] = (char)(v[e >> 2] >> (8 * (e & 3)));
        }
    }
}

// Pieces of 16 bytes of values a thread, so that a wavefront writes whole lines, a few of
// them one after the other, their loads in flight together. Memory bounds it: two forms of
// 8192 x 6144 to bf16 in 49 us, 6.2 TB/s (8-bit values from the last-level cache).
template <int DT, int N>
__global__ __launch_bounds__(kThreads) void k_f8_dequantize(const F8ValuesBatchOf<N> batch)
{
    using T = typename Elt<DT>::type;
    constexpr int V = 16 / (int)sizeof(T), kEach = kF8ValuesPieces / kThreads;
    const F8ValuesItem it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin;
    const int g = (it.cols + V - 1) / V;   // pieces a row
    const bool many = g <= kF8ValuesPieces;
    const int per = many ? kF8ValuesPieces / g : 1, seg = many ? 1 : (g + kF8ValuesPieces - 1) / kF8ValuesPieces;
    const int row0 = many ? b * per : b / seg, piece0 = many ? 0 : (b - row0 * seg) * kF8ValuesPieces;
    int row[kEach], c[kEach];
    uint32_t w[kEach][V / 4] = {};
    float s[kEach];
    bool in[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int k = threadIdx.x + kThreads * i, r = many ? k / g : 0;
        row[i] = row0 + r;
        c[i] = (piece0 + k - r * g) * V;
        in[i] = r < per && row[i] < it.rows && c[i] < it.cols;
        if (!in[i])
            continue;
        const int64_t at = (int64_t)(c[i] >> 7) * it.lds + (it.kind & 4 ? row[i] >> 7 : row[i]);
        const char* q = it.q + row[i] * it.ldq + c[i];
        // (q is aligned to 16 bytes, as are its rows: past a row's end, what fills its last 16
        // bytes is read and not used)
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[i][j] = ((const NS_GLOBAL uint32_t*)gbl(q))[j];
        if (it.kind & 2) {
            const uint32_t e = (uint8_t)gbl(it.scale)[at];
            s[i] = e == 255 ? __uint_as_float(0x7FC00000u) : e == 0 ? 0x1p-127f : __uint_as_float(e << 23);
        } else {
            s[i] = *(const NS_GLOBAL float*)gbl(it.scale + 4 * at);
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (!in[i])
            continue;
        float v[V];
        unroll<V>([&](auto e) __attribute__((always_inline)) {
            constexpr int E = decltype(e)::value;
            v[E] = s[i] * (it.kind & 1 ? __builtin_amdgcn_cvt_f32_bf8((int)w[i][E / 4], E % 4)
                                       : __builtin_amdgcn_cvt_f32_fp8((int)w[i][E / 4], E % 4));
        });
        T* x = reinterpret_cast<T*>(it.values) + row[i] * it.ldv + c[i];
        if (c[i] + V > it.cols) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c[i] + e < it.cols)
                    gbl(x)[e] = from_f32<T>(v[e]);
        } else if constexpr (DT == 0) {
            bf16x8 h;
#pragma unroll
            for (int e = 0; e < V; ++e)
                h[e] = (bf16)v[e];
            store16_any(x, __builtin_bit_cast(u32x4, h));
        } else {
            store16_any(x, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
        }
    }
}

// ---------------------------------------------------------------------------
// The product C = beta C + A B^T, in tiles of C.

// The shape of a tile kernel: WM x WN wavefronts of MI x NJ blocks of 32 x 32 each,
// RING slots of SLOT bytes of k a row in LDS.
template <int WM_, int WN_, int MI_, int NJ_, int SLOT_, int RING_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, MI = MI_, NJ = NJ_, SLOT = SLOT_, RING = RING_;
    static constexpr int kWaves = WM * WN, kLanes = 64 * kWaves;
    static constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN;
    static constexpr int kBytes = (BM + BN) * SLOT;      // LDS of a slot: A's rows, then B's
    static constexpr int kChunks = SLOT / 16;            // 16-byte pieces of a row
    static constexpr int kRows = 64 / kChunks;           // rows a load instruction covers
    static constexpr int LA = BM / (kRows * kWaves), LB = BN / (kRows * kWaves);   // a wavefront's loads a slot
    static constexpr int kUnits = SLOT / 64;             // MFMA steps a slot
};

#ifdef __HIP_DEVICE_COMPILE__
__device__ __forceinline__ int up16(int v) { return (v + 15) & ~15; }

// D = A B + C on blocks of 32 x 32 outputs and 64 k, operands times the powers of two
// in byte I and J of the lanes' scale words. A in format FA, B in e4m3. The unit adds the
// products of eight neighbouring k first, cut at 2^-13 of the largest one's power of two,
// toward 0; these sums and C add up in fp32. That is 1.5e-5 of the result's norm for normal
// values, and what twice the bf16 unit's rate costs: bf16 outputs round by 1.7e-3. fp32
// outputs take the bf16 unit, which cuts nothing.
template <int FA, int I, int J>
__device__ __forceinline__ f32x16 mfma_f8(i32x8 a, i32x8 b, f32x16 c, int sa, int sb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, FA, NS_F8_E4M3, I, sa, J, sb);
}
// The same on 16 x 16 outputs and 128 k.
template <int FA>
__device__ __forceinline__ f32x4 mfma_f8_16(i32x8 a, i32x8 b, f32x4 c, int sa, int sb)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, FA, NS_F8_E4M3, 0, sa, 0, sb);
}

// Eight 8-bit floats times the power of two of s's exponent, as bf16.
template <int FMT>
__device__ __forceinline__ bf16x8 widen(int lo, int hi, float s)
{
    bf16x2 v[4];
    if constexpr (FMT == NS_F8_E4M3) {
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
    } else {
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, s, false);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, s, true);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, s, false);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, s, true);
    }
    return bf16x8{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
}

// An fp32 scale as 2^(e - 127) m: e goes to the matrix units or into the widening, m
// in [1, 2) multiplies the block's sum. (0 and subnormals: e = 0, m < 1.)
struct Split { uint32_t e; float m; };
__device__ __forceinline__ Split split(uint32_t bits, bool pow2)
{
    const uint32_t e = (bits >> 23) & 255u;
    const float normal = __uint_as_float((bits & 0x807FFFFFu) | 0x3F800000u);
    const float m = e == 0 ? __uint_as_float(bits) * 0x1p127f : normal;
    return {e, pow2 ? 1.f : m};
}

// Scales of an operand's rows, block by block. at: a row's index among a block's
// scales (the row, or its square's).
struct Scales {
    const char* base;
    int64_t pitch;   // bytes
    int bytes;       // of a block's scales, those of one byte rounded up to 4
    int blocks;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t at(int b) const
    {
        return buffer(base + b * pitch, b < blocks ? bytes : 0);
    }
};
__device__ __forceinline__ Scales scales(const char* base, int ld, int rows, int blocks, bool pow2, bool square)
{
    const int count = square ? (rows + 127) >> 7 : rows;
    return {base, (int64_t)ld * (pow2 ? 1 : 4), pow2 ? (count + 3) & ~3 : count * 4, blocks};
}
// One scale's bits in fp32 (a byte of 0 stays 0).
__device__ __forceinline__ uint32_t scale_bits(__amdgpu_buffer_rsrc_t r, int at, bool pow2)
{
    const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(r, pow2 ? at & ~3 : at * 4, 0, 0);
    return pow2 ? ((w >> (8 * (at & 3))) & 255u) << 23 : w;
}

// The tile at (m0, n0) over slots [s0, s1) of k; piece: which of it.nsplit.
// ANY: fp32 scales, 1 with a scale for each row of B, 2 with squares of B.
//
// Both operands arrive by buffer_load ... lds, 16 bytes a lane and whole cache lines a
// row: rows of 128 bytes load at 7 to 10 ns an instruction and compute unit, rows of 64 at
// 16 to 17. Row r of a slot takes 128 bytes, its chunk c at chunk c ^ (r / 2 & 7): the 64
// banks hold two rows, so that 16 lanes of a fragment's read fall on different ones
// whether they are neighbours or not (by r & 7 half of the LDS cycles were conflicts). While a slot is multiplied, those after it stream in; the
// fragments of the next 64 k are read while the matrix units work on these.
//
// Rows of C: block i of a wavefront takes every MI-th of its rows from i on, columns
// likewise: a lane's rows lie side by side in the scales, so that one word holds all
// that it needs of them, and its NJ columns side by side in C. A and B lie in LDS in
// that order.
//
// Buffer resources end with the operand, so rows past the end read as 0. Along a row,
// what lies past the end in memory may be anything (a NaN): lanes whose 16 bytes of k are
// not whole get an offset behind the resource, and the last k that do not fill 16 bytes
// are multiplied by themselves, before the loop, from registers. So the loop has no
// branches, across which the compiler would move the products.
template <bool WIDE, int FA, int ANY, typename S>
__device__ __forceinline__ void f8_tile(const F8Item& it, int m0, int n0, int s0, int s1, int piece, float beta,
                                        char* (&sl)[S::RING], float* lman)
{
    static_assert(S::SLOT == kF8Block && (S::RING == 3 || S::RING == 2), "see step");
    constexpr int MI = S::MI, NJ = S::NJ, SLOT = S::SLOT, RING = S::RING;
    const int K = it.k, ns = (K + SLOT - 1) / SLOT;
    const int rows = min(S::BM, it.m - m0), cols = min(S::BN, it.n - n0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave / S::WN, wc = wave % S::WN;
    const int fr = lane & 31, fg = lane >> 5;
    const bool powa = !ANY || (it.flags & kF8PowA), powb = !ANY || (it.flags & kF8PowB);
    const bool sqa = it.flags & kF8SquareA, sqb = it.flags & kF8SquareB;

    const char* A = it.a + (int64_t)m0 * it.lda;
    const char* B = it.b + (int64_t)n0 * it.ldb;
    constexpr int kBehind = (int)0x80000000;
    const int whole = K & ~15;   // k in whole pieces of 16
    const int size_a = (rows - 1) * it.lda + up16(K), size_b = (cols - 1) * it.ldb + up16(K);
    const __amdgpu_buffer_rsrc_t ra = buffer(A, size_a), rb = buffer(B, size_b);
    const int blocks = (K + kF8Block - 1) / kF8Block;
    const Scales ca = scales(it.sa, it.ldsa, it.m, blocks, powa, sqa);
    const Scales cb = scales(it.sb, it.ldsb, it.n, blocks, powb, sqb);

    auto swz = [](int r) { return (r >> 1) & 7; };
    // Load q of a wavefront: LDS rows kRows (wave + kWaves q) .. + kRows - 1.
    const int lrow = lane / S::kChunks, lchunk = lane % S::kChunks;
    int voff_a[S::LA], voff_b[S::LB];
#pragma unroll
    for (int q = 0; q < S::LA; ++q) {
        const int r = S::kRows * (wave + S::kWaves * q) + lrow, rem = r % (32 * MI);
        voff_a[q] = (r - rem + MI * (rem % 32) + rem / 32) * it.lda + ((lchunk ^ swz(r)) << 4);
    }
#pragma unroll
    for (int q = 0; q < S::LB; ++q) {
        const int r = S::kRows * (wave + S::kWaves * q) + lrow, rem = r % (32 * NJ);
        voff_b[q] = (r - rem + NJ * (rem % 32) + rem / 32) * it.ldb + ((lchunk ^ swz(r)) << 4);
    }
    // A lane's first byte of a slot, the same in all of its loads: kWaves is even.
    const int first = (lchunk ^ swz(S::kRows * wave + lrow)) << 4;
    auto issue = [&](char* sp, int s) __attribute__((always_inline)) {
        // slots past the end read as 0 and keep the count of loads uniform
        const bool in = first < (s < s1 ? whole - s * SLOT : 0);
#pragma unroll
        for (int q = 0; q < S::LA; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(sp + (wave + S::kWaves * q) * 1024), 16,
                                                     in ? voff_a[q] : kBehind, s * SLOT, 0, 0);
#pragma unroll
        for (int q = 0; q < S::LB; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb, (lds_ptr)(sp + S::BM * SLOT + (wave + S::kWaves * q) * 1024), 16, in ? voff_b[q] : kBehind,
                s * SLOT, 0, 0);
    };

    // The scales of a lane's rows of A and of B: one byte each in a word, exponents; and
    // where some are fp32, the factors m that they leave.
    const int row_a = m0 + wr * 32 * MI + MI * fr, row_b = n0 + wc * 32 * NJ + NJ * fr;
    auto pick = [](int at, int n, bool square) {
        uint32_t sel = 0;
        for (int i = 0; i < n; ++i)
            sel |= (uint32_t)((at & 3) + (square ? 0 : i)) << (8 * i);
        return sel;
    };
    const int at_a = sqa ? row_a >> 7 : row_a, at_b = sqb ? row_b >> 7 : row_b;
    const uint32_t sel_a = pick(at_a, MI, sqa), sel_b = pick(at_b, NJ, sqb);
    struct Scale {
        int a, b;
        uint32_t ra[ANY ? MI : 1], rb[ANY ? NJ : 1];   // ANY: as loaded
    };
    auto load_scale = [&](Scale& c, int block) __attribute__((always_inline)) {
        // (past the end: 0)
        const __amdgpu_buffer_rsrc_t qa = ca.at(block), qb = cb.at(block);
        if constexpr (ANY) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
                c.ra[i] = scale_bits(qa, sqa ? at_a : at_a + i, powa);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                c.rb[j] = scale_bits(qb, sqb ? at_b : at_b + j, powb);
        } else {
            c.ra[0] = __builtin_amdgcn_raw_buffer_load_b32(qa, at_a & ~3, 0, 0);
            c.rb[0] = __builtin_amdgcn_raw_buffer_load_b32(qb, at_b & ~3, 0, 0);
        }
    };
    // The words from what was loaded; A's factors go to LDS, from where every lane
    // takes those of its rows of C.
    float mb[NJ];
    float* const man = lman + wave * 32 * MI;
    auto ready = [&](Scale& c) __attribute__((always_inline)) {
        if constexpr (ANY) {
            c.a = c.b = 0;
            float m[MI];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const Split p = split(c.ra[i], powa);
                c.a |= (int)(p.e << (8 * i));
                m[i] = p.m;
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const Split p = split(c.rb[j], powb);
                c.b |= (int)(p.e << (8 * j));
                mb[j] = p.m;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < MI; ++i)
                man[MI * fr + i] = ANY == 2 ? m[i] * mb[0] : m[i];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        } else {
            c.a = (int)__builtin_amdgcn_perm(c.ra[0], c.ra[0], sel_a);
            c.b = (int)__builtin_amdgcn_perm(c.rb[0], c.rb[0], sel_b);
        }
    };

    // Fragments: lane l takes row l & 31 of its block and of unit u the 16-byte chunks
    // 4 u + (l >> 5) and 4 u + 2 + (l >> 5); which k that is does not matter, as long
    // as A and B agree.
    const int frag = fr * SLOT + ((fg ^ swz(fr)) << 4);
    const int base_a = wr * 32 * MI * SLOT, base_b = S::BM * SLOT + wc * 32 * NJ * SLOT;
    auto read_frags = [&](const char* sp, int u, i32x8 (&af)[MI], i32x8 (&bf)[NJ]) __attribute__((always_inline)) {
        auto one = [&](int base) __attribute__((always_inline)) {
            const u32x4 lo = *reinterpret_cast<const u32x4*>(sp + base + (frag ^ (u << 6)));
            const u32x4 hi = *reinterpret_cast<const u32x4*>(sp + base + (frag ^ (u << 6) ^ 32));
            return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        };
#pragma unroll
        for (int i = 0; i < MI; ++i)
            af[i] = one(base_a + i * 32 * SLOT);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            bf[j] = one(base_b + j * 32 * SLOT);
    };

    f32x16 acc[MI][NJ], tmp[ANY ? MI : 1][ANY ? NJ : 1];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            acc[i][j] = f32x16{};
    // 64 k of a block, `first` or more; in halves of the work, part 0 and 1 (2: all).
    auto multiply = [&](auto first, auto part, const i32x8 (&af)[MI], const i32x8 (&bf)[NJ], const Scale& c)
        __attribute__((always_inline)) {
        constexpr int P = decltype(part)::value;
        auto mine = [](int i, int n) constexpr { return P == 2 || i * 2 / n == P; };
        if constexpr (ANY && decltype(first)::value && !(WIDE && P == 1))
            unroll<MI>([&](auto i) __attribute__((always_inline)) {
                if constexpr (WIDE || mine(decltype(i)::value, MI))
                    unroll<NJ>([&](auto j) __attribute__((always_inline)) { tmp[i][j] = f32x16{}; });
            });
        auto& sum = [&]() -> auto& {
            if constexpr (ANY)
                return tmp;
            else
                return acc;
        }();
        if constexpr (WIDE) {
            float fa[MI], fb[NJ];
            unroll<MI>([&](auto i) __attribute__((always_inline)) {
                fa[i] = __uint_as_float((((uint32_t)c.a >> (8 * i)) & 255u) << 23);
            });
            unroll<NJ>([&](auto j) __attribute__((always_inline)) {
                fb[j] = __uint_as_float((((uint32_t)c.b >> (8 * j)) & 255u) << 23);
            });
            unroll<4>([&](auto q) __attribute__((always_inline)) {
                if constexpr (mine(decltype(q)::value, 4)) {
                    bf16x8 wa[MI], wb[NJ];
                    unroll<MI>([&](auto i) __attribute__((always_inline)) {
                        wa[i] = widen<FA>(af[i][2 * q], af[i][2 * q + 1], fa[i]);
                    });
                    unroll<NJ>([&](auto j) __attribute__((always_inline)) {
                        wb[j] = widen<NS_F8_E4M3>(bf[j][2 * q], bf[j][2 * q + 1], fb[j]);
                    });
                    unroll<MI>([&](auto i) __attribute__((always_inline)) {
                        unroll<NJ>([&](auto j) __attribute__((always_inline)) {
                            sum[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa[i], wb[j], sum[i][j], 0, 0, 0);
                        });
                    });
                }
            });
        } else {
            unroll<MI>([&](auto i) __attribute__((always_inline)) {
                if constexpr (mine(decltype(i)::value, MI))
                    unroll<NJ>([&](auto j) __attribute__((always_inline)) {
                        sum[i][j] =
                            mfma_f8<FA, decltype(i)::value, decltype(j)::value>(af[i], bf[j], sum[i][j], c.a, c.b);
                    });
            });
        }
    };
    // ANY: a block's sums, times the factors of their row and column.
    auto fold = [&]() __attribute__((always_inline)) {
        if constexpr (ANY) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float m[4 * MI];
#pragma unroll
                for (int e = 0; e < MI; ++e)
                    *reinterpret_cast<f32x4*>(m + 4 * e) =
                        *reinterpret_cast<const f32x4*>(man + MI * (8 * g + 4 * fg) + 4 * e);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            acc[i][j][4 * g + e] =
                                fmaf(tmp[i][j][4 * g + e], ANY == 2 ? m[MI * e + i] : m[MI * e + i] * mb[j],
                                     acc[i][j][4 * g + e]);
            }
        }
    };

    Scale c[3];
    const std::true_type begin{};
    const std::false_type more{};
    const std::integral_constant<int, 0> half0{};
    const std::integral_constant<int, 1> half1{};
    const std::integral_constant<int, 2> all{};
    if (whole < K && s1 == ns) {
        // the last k: chunk 0 of a unit whose others are 0
        auto load = [&](__amdgpu_buffer_rsrc_t r, int off) __attribute__((always_inline)) {
            const u32x4 v = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, fg == 0 ? off + whole : kBehind, 0, 0));
            i32x8 f = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int over = K - whole - 4 * e;   // bytes of this word to keep
                f[e] = over >= 4 ? (int)v[e] : over <= 0 ? 0 : (int)(v[e] & (0xFFFFFFFFu >> (32 - 8 * over)));
            }
            return f;
        };
        i32x8 af[MI], bf[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i)
            af[i] = load(ra, (wr * 32 * MI + MI * fr + i) * it.lda);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            bf[j] = load(rb, (wc * 32 * NJ + NJ * fr + j) * it.ldb);
        load_scale(c[0], blocks - 1);
        ready(c[0]);
        multiply(begin, all, af, bf, c[0]);
        fold();
    }

    // Step s multiplies slot s, the one at place I of the ring, in two units of 64 k; the
    // second unit's fragments are read while the first one's are multiplied, the next
    // slot's first while the second one's are.
    //
    // A ring of three: behind the barrier in the middle slot s + 1 is whole for everyone,
    // and slot s, which all have read, is refilled. Its wait leaves in flight what was
    // issued after slot s + 1 (loads of scales not counted, so that it can only wait for
    // more).
    //
    // A ring of two, the large tiles': slot s is refilled as soon as all have read it,
    // behind a barrier after half of the first unit; slot s + 1 is waited for half a step
    // before its end, behind another, so that its loads have a step and a half to arrive.
    constexpr int kLoads = S::LA + S::LB;
    constexpr bool kTwo = RING == 2;
    i32x8 fa[2][MI], fb[2][NJ];
    // The order within a part of a step: products with the reads and loads between them.
    // (All reads at once would fill the LDS queue and keep the first product waiting.)
    auto interleave = [&](auto products, auto reads, auto loads) __attribute__((always_inline)) {
        constexpr int F = decltype(products)::value, R = decltype(reads)::value, M = decltype(loads)::value;
        if constexpr (!ANY || WIDE)
            unroll<F>([&](auto f) __attribute__((always_inline)) {
                constexpr int q = decltype(f)::value;
                constexpr int r = R * (q + 1) / F - R * q / F, m = M * (q + 1) / F - M * q / F;
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if constexpr (m > 0)
                    __builtin_amdgcn_sched_group_barrier(0x010, m, 0);
                if constexpr (r > 0)
                    __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
            });
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kProducts = MI * NJ * (WIDE ? 4 : 1), kReads = 2 * (MI + NJ);
    const std::integral_constant<int, 0> none{};
    const std::integral_constant<int, kLoads> loads{};
    const std::integral_constant<int, kReads> reads{};
    const std::integral_constant<int, kProducts> products{};
    const std::integral_constant<int, kProducts / 2> some{};
    auto step = [&](auto place, int s) __attribute__((always_inline)) {
        constexpr int I = decltype(place)::value, N = (I + 1) % RING;
        if constexpr (kTwo) {
            ready(c[I]);
            read_frags(sl[I], 1, fa[1], fb[1]);
            multiply(begin, half0, fa[0], fb[0], c[I]);
            interleave(some, reads, none);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            load_scale(c[I], s + 2);
            asm volatile("" ::: "memory");
            issue(sl[I], s + 2);
            multiply(begin, half1, fa[0], fb[0], c[I]);
            multiply(more, half0, fa[1], fb[1], c[I]);
            interleave(products, none, loads);
            asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
            read_frags(sl[N], 0, fa[0], fb[0]);
            multiply(more, half1, fa[1], fb[1], c[I]);
            interleave(some, reads, none);
            fold();
            __builtin_amdgcn_sched_barrier(0);
        } else {
            ready(c[I]);
            read_frags(sl[I], 1, fa[1], fb[1]);
            multiply(begin, all, fa[0], fb[0], c[I]);
            interleave(products, reads, none);
            asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
            load_scale(c[(I + 2) % 3], s + 2);
            asm volatile("" ::: "memory");
            issue(sl[I], s + RING);
            read_frags(sl[N], 0, fa[0], fb[0]);
            multiply(more, all, fa[1], fb[1], c[I]);
            interleave(products, reads, loads);
            fold();
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    load_scale(c[0], s0);
    load_scale(c[1], s0 + 1);
    asm volatile("" ::: "memory");
    unroll<RING>([&](auto i) __attribute__((always_inline)) { issue(sl[i], s0 + i); });
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"((RING - 1) * kLoads) : "memory");
    read_frags(sl[0], 0, fa[0], fb[0]);
    int s = s0;
    for (; s + RING <= s1; s += RING)
        unroll<RING>([&](auto i) __attribute__((always_inline)) { step(i, s + i); });
    unroll<RING - 1>([&](auto i) __attribute__((always_inline)) {
        if (s + i < s1)
            step(i, s + i);
    });
    // (loads of slots past the end are still to land in LDS: they are not to outlive
    // the workgroup)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // The output. Register r of lane l, block (i, j): row MI (8 (r >> 2) + 4 (l >> 5) +
    // (r & 3)) + i, column NJ (l & 31) + j of the wavefront's part. Rows past the end
    // fall behind the buffer resource, and lanes with columns past the end get an
    // offset behind it.
    const bool split = it.nsplit > 1;   // a piece of the sums goes as it is, in fp32
    const int row0 = wr * 32 * MI + MI * 4 * fg, col0 = wc * 32 * NJ + NJ * fr;
    // Row g, e, i of a lane's: its NJ sums, plus beta times what is there; as one piece
    // where the alignment and n allow.
    auto store = [&](auto out, __amdgpu_buffer_rsrc_t ro, int ldo, auto fits, auto adds) __attribute__((always_inline)) {
        using T = decltype(out);
        constexpr int kElt = sizeof(T), kWords = NJ * kElt / 4;
        constexpr bool kFits = decltype(fits)::value, kAdds = decltype(adds)::value;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const int at = (row0 + MI * (8 * g + e) + i) * ldo + col0 * kElt;
                    float v[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        v[j] = acc[i][j][4 * g + e];
                    if constexpr (kFits) {
                        const int place = col0 < cols ? at : kBehind;
                        uint32_t w[kWords];
                        if constexpr (kAdds) {
                            load_words(w, ro, place);
#pragma unroll
                            for (int j = 0; j < NJ; ++j) {
                                const uint32_t o = w[kElt == 2 ? j >> 1 : j];
                                v[j] = fmaf(beta, __uint_as_float(kElt == 4 ? o : j & 1 ? o & 0xFFFF0000u : o << 16),
                                            v[j]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < kWords; ++j)
                            w[j] = kElt == 4 ? __float_as_uint(v[j])
                                             : __builtin_bit_cast(uint32_t, bf16x2{(bf16)v[(2 * j) % NJ],
                                                                                   (bf16)v[(2 * j + 1) % NJ]});
                        store_words(w, ro, place);
                    } else {
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const int place = col0 + j < cols ? at + kElt * j : kBehind;
                            if constexpr (kElt == 2) {
                                if constexpr (kAdds) {
                                    const uint32_t o = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ro, place, 0, 0);
                                    v[j] = fmaf(beta, __uint_as_float(o << 16), v[j]);
                                }
                                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)v[j]), ro, place,
                                                                      0, 0);
                            } else {
                                if constexpr (kAdds)
                                    v[j] = fmaf(beta,
                                                __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ro, place, 0, 0)),
                                                v[j]);
                                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), ro, place, 0, 0);
                            }
                        }
                    }
                }
            __builtin_amdgcn_sched_barrier(0);   // (a group's registers at a time)
        }
    };
    const std::true_type yes{};
    const std::false_type no{};
    using T = typename std::conditional<WIDE, float, bf16>::type;
    const int ldo = it.ldo * (int)sizeof(T);
    const __amdgpu_buffer_rsrc_t ro = buffer(static_cast<const T*>(it.out) + (int64_t)m0 * it.ldo + n0,
                                             (rows - 1) * ldo + cols * (int)sizeof(T));
    if constexpr (MI * NJ > 4) {
        // Large tiles, whose sums fill half of the registers: one way to store them, whole
        // pieces, in which only the loads of what is there are left out where nothing is to
        // be added. (Ways of their own would copy all sums at once where they part.)
        constexpr int kElt = sizeof(T), kWords = NJ * kElt / 4;
        const int place = col0 < cols ? row0 * ldo + col0 * kElt : kBehind;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t w[4][MI][kWords] = {};
            if (beta != 0.f)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < MI; ++i)
                        load_words(w[e][i], ro, place + (MI * (8 * g + e) + i) * ldo);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float v[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const uint32_t o = w[e][i][kElt == 2 ? j >> 1 : j];
                        v[j] = fmaf(beta, __uint_as_float(kElt == 4 ? o : j & 1 ? o & 0xFFFF0000u : o << 16),
                                    acc[i][j][4 * g + e]);
                    }
                    uint32_t y[kWords];
#pragma unroll
                    for (int j = 0; j < kWords; ++j)
                        y[j] = kElt == 4 ? __float_as_uint(v[j])
                                         : __builtin_bit_cast(uint32_t, bf16x2{(bf16)v[(2 * j) % NJ],
                                                                               (bf16)v[(2 * j + 1) % NJ]});
                    store_words(y, ro, place + (MI * (8 * g + e) + i) * ldo);
                }
            __builtin_amdgcn_sched_barrier(0);   // (a group's registers at a time)
        }
        return;
    }
    if (split) {
        const __amdgpu_buffer_rsrc_t rp =
            buffer(it.part + ((int64_t)piece * it.m + m0) * it.n + n0, ((rows - 1) * it.n + cols) * 4);
        if (it.n % NJ == 0)
            store(0.f, rp, it.n * 4, yes, no);
        else
            store(0.f, rp, it.n * 4, no, no);
        return;
    }
    const bool fits = it.n % NJ == 0 && it.ldo % NJ == 0 && reinterpret_cast<uintptr_t>(it.out) % (NJ * sizeof(T)) == 0;
    if (fits && beta == 0.f)
        store(T(0.f), ro, ldo, yes, no);
    else if (fits)
        store(T(0.f), ro, ldo, yes, yes);
    else if (beta == 0.f)
        store(T(0.f), ro, ldo, no, no);
    else
        store(T(0.f), ro, ldo, no, yes);
}
#endif

using Small = Shape<2, 2, 2, 2, 128, 2>;
using Mid = Shape<2, 4, 2, 2, 128, 3>;
using Big = Shape<2, 2, 4, 4, 128, 2>;
static_assert(Small::BM == kF8SmallM && Small::BN == kF8SmallN && Mid::BM == kF8MidM && Mid::BN == kF8MidN &&
                  Big::BM == kF8Big && Big::BN == kF8Big,
              "the planner's tiles");

// Mid, 16 experts of 2048 x 6144, 3001 tokens: 60 us, matrix units 38% busy, 247 MB a call
// from memory at 4.1 TB/s. What holds memory there is not known: operands at pitches of 6144
// + 128 to 1024 bytes take 62 to 64. Small with fp32 scales, 4 experts of 2048 x 6144, 1999
// tokens: 53 us, matrix units 21% busy, vector ones 22%: there is one wavefront a SIMD, so
// that nothing is multiplied beside its fold, and 272 tiles give 16 of 256 compute units two
// (256 tiles: 46 us).
//
// Small: tiles of 128 x 128, two workgroups of four wavefronts a compute unit, a ring of
// two slots each. Mid: tiles of 128 x 256, one workgroup of eight wavefronts a compute
// unit, a ring of three slots, two of them (96 KB) in flight.
template <bool WIDE, int FA, int ANY, typename S, int N>
__global__ __launch_bounds__(S::kLanes, 2) void k_f8_tiles(const F8BatchOf<N> batch, int nwg)
{
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __attribute__((aligned(1024))) char sl0[S::kBytes];
    __shared__ __attribute__((aligned(1024))) char sl1[S::kBytes];
    __shared__ __attribute__((aligned(1024))) char sl2[S::RING == 3 ? S::kBytes : 16];
    __shared__ __attribute__((aligned(16))) float lman[ANY ? S::kWaves * 32 * S::MI : 4];
    char* sl[S::RING];
    sl[0] = sl0;
    sl[1] = sl1;
    if constexpr (S::RING == 3)
        sl[2] = sl2;
    const int t = by_xcd(blockIdx.x, nwg);
    const F8Item it = batch.it[find_item(batch, t)];
    const int ntm = (it.m + S::BM - 1) / S::BM, tiles = ntm * it.ntn, own = t - it.begin;
    const int piece = own / tiles, blocks = (it.k + kF8Block - 1) / kF8Block;
    int bm, bn;
    tile_at(own - piece * tiles, ntm, it.ntn, &bm, &bn);
    const int s0 = piece * it.per, s1 = min(blocks, s0 + it.per);
    f8_tile<WIDE, FA, ANY, S>(it, bm * S::BM, bn * S::BN, s0, s1, piece, batch.beta, sl, lman);
#endif
}

// Tiles of 256 x 256, one workgroup of four wavefronts a compute unit, 128 x 128 outputs
// a wavefront in 256 registers of each lane, a ring of two slots of 128 bytes a row. Matrix
// units bound it: 4096 x 8192 by k = 6144 in 156 to 169 us (bf16, 71% busy, 2.4 to 2.6
// PFLOP/s), 8192 x 6144 by 4001 into fp32 in 355 to 373 (60%, 1.1).
template <bool WIDE, int FA>
__global__ __launch_bounds__(Big::kLanes, 1) void k_f8_big(const F8Batch batch, int nwg)
{
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __attribute__((aligned(1024))) char sl0[Big::kBytes];
    __shared__ __attribute__((aligned(1024))) char sl1[Big::kBytes];
    char* sl[2] = {sl0, sl1};
    const int t = by_xcd(blockIdx.x, nwg);
    const F8Item it = batch.it[find_item(batch, t)];
    int bm, bn;
    tile_at(t - it.begin, (it.m + Big::BM - 1) / Big::BM, it.ntn, &bm, &bn);
    f8_tile<WIDE, FA, 0, Big>(it, bm * Big::BM, bn * Big::BN, 0, (it.k + kF8Block - 1) / kF8Block, 0,
                                  batch.beta, sl, nullptr);
#endif
}

// Products of at most 32 rows of A (few tokens): B, the weights, streams from memory
// straight into the MFMAs. A workgroup of eight wavefronts takes 16 NB rows of B, a
// wavefront every eighth block of them, all loads of several blocks in flight at once: lane
// l the 32 bytes from 32 (l / 16) on of the block of row l % 16. The wavefronts' sums meet
// in LDS. Memory bounds it: one token through 8192 x 6144 in 9.9 us, 5.1 TB/s.
constexpr int kFewLanes = 512;
template <bool WIDE, int FA, bool ANY, int NB, int N>
__global__ __launch_bounds__(kFewLanes, 2) void k_f8_few(const F8BatchOf<N> batch)
{
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __attribute__((aligned(16))) f32x4 red[2][NB][8][64];
    const F8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int n0 = (blockIdx.x - it.begin) * 16 * NB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const int K = it.k, blocks = (K + kF8Block - 1) / kF8Block;
    const int cols = min(16 * NB, it.n - n0);
    const bool two = it.m > 16;
    const bool powa = !ANY || (it.flags & kF8PowA), powb = !ANY || (it.flags & kF8PowB);
    const bool sqa = it.flags & kF8SquareA, sqb = it.flags & kF8SquareB;
    const __amdgpu_buffer_rsrc_t ra = buffer(it.a, (it.m - 1) * it.lda + up16(K));
    const __amdgpu_buffer_rsrc_t rb = buffer(it.b + (int64_t)n0 * it.ldb, (cols - 1) * it.ldb + up16(K));
    const Scales ca = scales(it.sa, it.ldsa, it.m, blocks, powa, sqa);
    const Scales cb = scales(it.sb, it.ldsb, it.n, blocks, powb, sqb);
    // 32 bytes of k from `at` of a row at `off`, 0 past the row's end (whole chunks of 16
    // by an offset behind the resource, the rest byte by byte)
    constexpr int kBehind = (int)0x80000000;
    auto fetch = [&](__amdgpu_buffer_rsrc_t r, int off, int at) __attribute__((always_inline)) {
        const u32x4 lo = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at < K ? off + at : kBehind, 0, 0));
        const u32x4 hi = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 < K ? off + at + 16 : kBehind, 0, 0));
        return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto clear = [&](i32x8& v, int at) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int over = K - (at + 4 * e);   // bytes of this word to keep
            v[e] = over >= 4 ? v[e] : over <= 0 ? 0 : (int)((uint32_t)v[e] & (0xFFFFFFFFu >> (32 - 8 * over)));
        }
    };
    f32x4 acc[2][NB] = {};
    auto tiles = [&](auto second) __attribute__((always_inline)) {
        constexpr int MT = decltype(second)::value ? 2 : 1;
        // blocks in flight: what the registers hold (6 of a wavefront are all of k = 6144)
        constexpr int D = MT == 2 && NB == 2 ? 3 : 6;
        for (int b0 = wave; b0 < blocks; b0 += 8 * D) {
            i32x8 va[D][MT], vb[D][NB];
            uint32_t xa[D][MT], xb[D][NB];
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int b = b0 + 8 * d, at = b * kF8Block + 32 * fg;
                const __amdgpu_buffer_rsrc_t qa = ca.at(b), qb = cb.at(b);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int row = 16 * j + fr;
                    vb[d][j] = fetch(rb, row * it.ldb, at);
                    xb[d][j] = scale_bits(qb, sqb ? (n0 + row) >> 7 : n0 + row, powb);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int row = 16 * i + fr;
                    va[d][i] = fetch(ra, row * it.lda, at);
                    xa[d][i] = scale_bits(qa, sqa ? row >> 7 : row, powa);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int b = b0 + 8 * d, at = b * kF8Block + 32 * fg;
                if (b == blocks - 1 && (K & 127)) {
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        clear(vb[d][j], at);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        clear(va[d][i], at);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const Split pa = split(xa[d][i], powa);
                    float ma[ANY ? 4 : 1];
                    if constexpr (ANY)   // (rows of C: 4 (l / 16) + r, whose factors lanes of those numbers hold)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            ma[r] = __shfl(pa.m, 4 * fg + r, 64);
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const Split pb = split(xb[d][j], powb);
                        f32x4 sum = ANY ? f32x4{} : acc[i][j];
                        if constexpr (WIDE) {
                            const float fa = __uint_as_float(pa.e << 23), fb = __uint_as_float(pb.e << 23);
                            unroll<4>([&](auto q) __attribute__((always_inline)) {
                                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    widen<FA>(va[d][i][2 * q], va[d][i][2 * q + 1], fa),
                                    widen<NS_F8_E4M3>(vb[d][j][2 * q], vb[d][j][2 * q + 1], fb), sum, 0, 0, 0);
                            });
                        } else {
                            sum = mfma_f8_16<FA>(va[d][i], vb[d][j], sum, (int)pa.e, (int)pb.e);
                        }
                        if constexpr (ANY) {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                acc[i][j][r] = fmaf(sum[r], ma[r] * pb.m, acc[i][j][r]);
                        } else {
                            acc[i][j] = sum;
                        }
                    }
                }
            }
        }
    };
    if (two)
        tiles(std::true_type{});
    else
        tiles(std::false_type{});
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        red[0][j][wave][lane] = acc[0][j];
        red[1][j][wave][lane] = acc[1][j];
    }
    __syncthreads();
    // one wavefront adds up each block of 16 x 16
    const int half = wave / NB, j = wave % NB;
    if (half > (two ? 1 : 0))
        return;
    f32x4 sum = red[half][j][0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w)
        sum += red[half][j][w][lane];
    if (16 * j + fr >= cols)
        return;
    using T = typename std::conditional<WIDE, float, bf16>::type;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 16 * half + 4 * fg + r;
        if (row < it.m) {
            NS_GLOBAL T* o = gbl(static_cast<T*>(it.out)) + (int64_t)row * it.ldo + n0 + 16 * j + fr;
            const float v = batch.beta != 0.f ? fmaf(batch.beta, to_f32(*o), sum[r]) : sum[r];
            *o = from_f32<T>(v);
        }
    }
#endif
}

// The pieces of split sums, added in order; sums over nothing. Four outputs a thread where
// n and the alignment allow, eight pieces in flight. About 5 us beside its bytes.
template <int DT, int N>
__global__ __launch_bounds__(kThreads) void k_f8_join(const F8BatchOf<N> batch)
{
    using T = typename Elt<DT>::type;
    typedef T T4 __attribute__((ext_vector_type(4)));
    const F8Item it = batch.it[find_item(batch, blockIdx.x)];
    const float beta = batch.beta;
    const int64_t total = (int64_t)it.m * it.n, e0 = (int64_t)(blockIdx.x - it.begin) * kF8JoinElems;
    const NS_GLOBAL float* part = gbl(static_cast<const float*>(it.part));
    if (((it.n | it.ldo) & 3) == 0 && reinterpret_cast<uintptr_t>(it.out) % sizeof(T4) == 0) {
        const int64_t e = e0 + 4 * threadIdx.x;
        if (e >= total)
            return;
        const int r = (int)(e / it.n), c = (int)(e - (int64_t)r * it.n);
        NS_GLOBAL T4* p = (NS_GLOBAL T4*)(gbl(static_cast<T*>(it.out)) + (int64_t)r * it.ldo + c);
        const T4 old = beta != 0.f ? *p : T4{};
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int q0 = 0; q0 < it.nsplit; q0 += 8) {
            f32x4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = q0 + q < it.nsplit ? *(const NS_GLOBAL f32x4*)(part + (q0 + q) * total + e) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                sum += v[q];
        }
        T4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = from_f32<T>(beta != 0.f ? fmaf(beta, to_f32(old[i]), sum[i]) : sum[i]);
        *p = y;
        return;
    }
    for (int i = 0; i < kF8JoinElems / kThreads; ++i) {
        const int64_t e = e0 + threadIdx.x + i * kThreads;
        if (e >= total)
            return;
        float sum = 0.f;
        for (int q = 0; q < it.nsplit; ++q)
            sum += part[q * total + e];
        const int r = (int)(e / it.n), c = (int)(e - (int64_t)r * it.n);
        NS_GLOBAL T* p = gbl(static_cast<T*>(it.out)) + (int64_t)r * it.ldo + c;
        *p = from_f32<T>(beta != 0.f ? fmaf(beta, to_f32(*p), sum) : sum);
    }
}

// The first items of a batch, for a launch with fewer argument bytes.
template <int M, typename B>
B first_of(const F8BatchOf<M>& b)
{
    B h;
    for (int i = 0; i < kF8FewItems; ++i)
        h.it[i] = b.it[i];
    h.count = b.count;
    h.beta = b.beta;
    return h;
}
F8BatchOf<kF8FewItems> head(const F8Batch& b) { return first_of<kF8Items, F8BatchOf<kF8FewItems>>(b); }

}  // namespace

hipError_t launch_f8_quantize(const F8RowsBatch& b, int nwg, int format, int pow2, int dtype, hipStream_t stream)
{
    auto go = [&](auto dt, auto fmt, auto p) {
        if (b.count <= kF8FewItems) {
            F8RowsBatchOf<kF8FewItems> h;
            for (int i = 0; i < kF8FewItems; ++i)
                h.it[i] = b.it[i];
            h.count = b.count;
            h.square = b.square;
            hipLaunchKernelGGL((k_f8_quantize<decltype(dt)::value, decltype(fmt)::value, decltype(p)::value, kF8FewItems>),
                               dim3(nwg), dim3(kThreads), 0, stream, h);
        } else {
            hipLaunchKernelGGL((k_f8_quantize<decltype(dt)::value, decltype(fmt)::value, decltype(p)::value, kF8RowsItems>),
                               dim3(nwg), dim3(kThreads), 0, stream, b);
        }
    };
    auto by_type = [&](auto fmt, auto p) {
        if (dtype == 0)
            go(std::integral_constant<int, 0>{}, fmt, p);
        else
            go(std::integral_constant<int, 1>{}, fmt, p);
    };
    auto by_format = [&](auto p) {
        if (format == NS_F8_E4M3)
            by_type(std::integral_constant<int, 0>{}, p);
        else
            by_type(std::integral_constant<int, 1>{}, p);
    };
    if (pow2)
        by_format(std::true_type{});
    else
        by_format(std::false_type{});
    return hipGetLastError();
}

hipError_t launch_f8_dequantize(const F8ValuesBatch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kThreads);
    if (b.count <= kF8FewItems) {
        F8ValuesBatchOf<kF8FewItems> h;
        for (int i = 0; i < kF8FewItems; ++i)
            h.it[i] = b.it[i];
        h.count = b.count;
        if (dtype == 0)
            hipLaunchKernelGGL((k_f8_dequantize<0, kF8FewItems>), grid, block, 0, stream, h);
        else
            hipLaunchKernelGGL((k_f8_dequantize<1, kF8FewItems>), grid, block, 0, stream, h);
    } else if (dtype == 0) {
        hipLaunchKernelGGL((k_f8_dequantize<0, kF8ValuesItems>), grid, block, 0, stream, b);
    } else {
        hipLaunchKernelGGL((k_f8_dequantize<1, kF8ValuesItems>), grid, block, 0, stream, b);
    }
    return hipGetLastError();
}

namespace {
// go(output is fp32, A's format, any) with the values as constants
template <typename F>
void by_kind(int format, int any, int dtype, F&& go)
{
    auto two = [&](auto wide, auto fmt) {
        if (any == 0)
            go(wide, fmt, std::integral_constant<int, 0>{});
        else if (any == 1)
            go(wide, fmt, std::integral_constant<int, 1>{});
        else
            go(wide, fmt, std::integral_constant<int, 2>{});
    };
    auto one = [&](auto wide) {
        if (format == NS_F8_E4M3)
            two(wide, std::integral_constant<int, 0>{});
        else
            two(wide, std::integral_constant<int, 1>{});
    };
    if (dtype == NS_FP32)
        one(std::true_type{});
    else
        one(std::false_type{});
}

template <typename S>
hipError_t launch_tiles(const F8Batch& b, int nwg, int format, int any, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(S::kLanes);
    bool done = false;
    by_kind(format, any, dtype, [&](auto wide, auto fmt, auto a) {
        constexpr bool W = decltype(wide)::value;
        constexpr int F = decltype(fmt)::value, Y = decltype(a)::value;
        if constexpr (!std::is_same_v<S, Mid> || has_mid(Y, W ? NS_FP32 : NS_BF16)) {
            if (b.count <= kF8FewItems)
                hipLaunchKernelGGL((k_f8_tiles<W, F, Y, S, kF8FewItems>), grid, block, 0, stream, head(b), nwg);
            else
                hipLaunchKernelGGL((k_f8_tiles<W, F, Y, S, kF8Items>), grid, block, 0, stream, b, nwg);
            done = true;
        }
    });
    return done ? hipGetLastError() : hipErrorInvalidValue;
}
}  // namespace

hipError_t launch_f8_small(const F8Batch& b, int nwg, int format, int any, int dtype, hipStream_t stream)
{
    return launch_tiles<Small>(b, nwg, format, any, dtype, stream);
}

hipError_t launch_f8_mid(const F8Batch& b, int nwg, int format, int any, int dtype, hipStream_t stream)
{
    return launch_tiles<Mid>(b, nwg, format, any, dtype, stream);
}

hipError_t launch_f8_big(const F8Batch& b, int nwg, int format, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(Big::kLanes);
    by_kind(format, 0, dtype, [&](auto wide, auto fmt, auto) {
        hipLaunchKernelGGL((k_f8_big<decltype(wide)::value, decltype(fmt)::value>), grid, block, 0, stream, b, nwg);
    });
    return hipGetLastError();
}

hipError_t launch_f8_few(const F8Batch& b, int nwg, int rows, int format, int any, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kFewLanes);
    by_kind(format, any ? 1 : 0, dtype, [&](auto wide, auto fmt, auto a) {
        constexpr bool W = decltype(wide)::value, Y = decltype(a)::value != 0;
        constexpr int F = decltype(fmt)::value;
        auto go = [&](auto nb) {
            constexpr int NB = decltype(nb)::value;
            if (b.count <= kF8FewItems)
                hipLaunchKernelGGL((k_f8_few<W, F, Y, NB, kF8FewItems>), grid, block, 0, stream, head(b));
            else
                hipLaunchKernelGGL((k_f8_few<W, F, Y, NB, kF8Items>), grid, block, 0, stream, b);
        };
        if (rows == 16)
            go(std::integral_constant<int, 1>{});
        else
            go(std::integral_constant<int, 2>{});
    });
    return hipGetLastError();
}

hipError_t launch_f8_join(const F8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kThreads);
    if (dtype == 0)
        hipLaunchKernelGGL((k_f8_join<0, kF8Items>), grid, block, 0, stream, b);
    else
        hipLaunchKernelGGL((k_f8_join<1, kF8Items>), grid, block, 0, stream, b);
    return hipGetLastError();
}

}  // namespace ns

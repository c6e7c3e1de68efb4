// ns_q8.hip -- gfx950 kernels of the 8-bit linear layers (include/ns.h,
// ns_q8_*): rows to int8 with a scale each and back, and the three products of
// a layer, Y = Xq Wq^T, dX = dY Wq and G = beta G + dY^T Xq.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ns.h"
#include "ns_q8.h"

namespace ns {
namespace {

typedef __bf16 bf16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define NS_GLOBAL __attribute__((address_space(1)))
// Global-memory view of a pointer (generic accesses would count on the LDS
// counter as well).
template <typename T>
__device__ __forceinline__ NS_GLOBAL T* gbl(T* p)
{
    return (NS_GLOBAL T*)p;
}

// 16- and 8-byte accesses at any byte address: the target's unaligned access
// mode makes them one instruction whatever the alignment.
struct __attribute__((packed, aligned(1))) Any16 { u32x4 v; };
struct __attribute__((packed, aligned(1))) Any8 { u32x2 v; };
__device__ __forceinline__ u32x4 load16_any(const void* p)
{
    return ((NS_GLOBAL const Any16*)gbl(static_cast<const char*>(p)))->v;
}
__device__ __forceinline__ u32x2 load8_any(const void* p)
{
    return ((NS_GLOBAL const Any8*)gbl(static_cast<const char*>(p)))->v;
}
__device__ __forceinline__ void store8_any(void* p, u32x2 v)
{
    ((NS_GLOBAL Any8*)gbl(static_cast<char*>(p)))->v = v;
}
__device__ __forceinline__ void store16_any(void* p, u32x4 v)
{
    ((NS_GLOBAL Any16*)gbl(static_cast<char*>(p)))->v = v;
}

template <int DT> struct Elt;
template <> struct Elt<0> { using type = bf16; };
template <> struct Elt<1> { using type = float; };
__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return (bf16)v; }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

constexpr int kThreads = 256;

// Item that owns workgroup b: the largest i with begin <= b.
template <typename B>
__device__ __forceinline__ int find_item(const B& batch, int b)
{
    int lo = 0, hi = batch.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (batch.it[mid].begin <= b)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------------------
// Rows to int8 and back.
//
// s from m = max |x| of the row, q = rne(x / s). Both kernels move every byte
// once (a row longer than its workgroup's registers is read twice), so memory
// bandwidth bounds them.

// Eight values of a row from column c on (0 past the end), as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, float (&v)[8])
{
    if (c + 8 <= cols) {
        if constexpr (sizeof(T) == 2) {
            const bf16x8 h = __builtin_bit_cast(bf16x8, load16_any(row + c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (float)h[e];
        } else {
            const f32x4 a = __builtin_bit_cast(f32x4, load16_any(row + c));
            const f32x4 b = __builtin_bit_cast(f32x4, load16_any(row + c + 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = c + e < cols ? to_f32(gbl(row)[c + e]) : 0.f;
    }
}

// Magnitude as an integer: orders like |x|, with Inf and NaN on top.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a row from the largest magnitude's bits: NaN for Inf or NaN.
__device__ __forceinline__ float q8_scale(uint32_t m, int mode)
{
    if (m >= 0x7F800000u)
        return __uint_as_float(0x7FC00000u);
    const float amax = __uint_as_float(m);
    if (mode == NS_Q8_POW2) {
        // amax = f 2^x with f in [1, 2): 127 2^e >= amax first holds at
        // e = x - 6 when f <= 127 / 64, else at x - 5 (subnormals: 2^-126)
        const int x = (int)(m >> 23) - 127;
        const int e = x - 6 + ((m & 0x7FFFFFu) > 0x7E0000u);
        return m < 0x00800000u || e < -126 ? 0x1p-126f : __uint_as_float((uint32_t)(e + 127) << 23);
    }
    return fmaxf(amax / 127.f, 0x1p-126f);
}

// Four integers of magnitude at most 127, held as floats, as the bytes of a
// word. Adding 1.5 2^23 leaves the integer in the float's low bits.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    const float big = 12582912.f;
    const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(b + big), __float_as_uint(a + big), 0x0C0C0400u);
    const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(d + big), __float_as_uint(c + big), 0x04000C0Cu);
    return ab | cd;
}

// q of eight values. `mul` is 1, or 2^60 for rows whose scale is so small that
// the tie test below would meet subnormals; s and inv = 1 / s come multiplied.
// x inv is off by at most 127 2^-23 from the quotient, so its rounding is the
// quotient's unless it lies that near a half: there the side of the tie is
// the sign of x - (q +- 1/2) s, which one fma gives exactly (q +- 1/2 has 8
// bits, s 24).
__device__ __forceinline__ u32x2 quant8(const float (&x)[8], float s, float inv, float mul)
{
    float q[8], v[8];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = x[e] * mul;
        const float r = v[e] * inv;
        q[e] = rintf(r);
        far = fmaxf(far, fabsf(r - q[e]));
    }
    if (far > 0.4999f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool odd = ((int)q[e]) & 1;
            const float up = fmaf(-(q[e] + 0.5f), s, v[e]);
            const float dn = fmaf(-(q[e] - 0.5f), s, v[e]);
            if (up > 0.f || (up == 0.f && odd))
                q[e] += 1.f;
            else if (dn < 0.f || (dn == 0.f && odd))
                q[e] -= 1.f;
        }
    }
    return u32x2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
}

// W wavefronts per row (1 or 4), NV groups of 8 values per lane in registers.
template <int DT, int W>
__device__ __forceinline__ void quantize_row(const Q8RowsItem& it, int row, int mode, uint32_t* red)
{
    using T = typename Elt<DT>::type;
    constexpr int NV = 4;
    constexpr int L = W * 64, kSpan = L * 8;   // lanes, values per group
    const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    const T* x = static_cast<const T*>(it.values) + row * it.ldv;
    int8_t* q = it.q + row * it.ldq;
    const int cols = it.cols;
    float v[NV][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kSpan + t * 8;
        if (c < cols)
            load8<T>(x, c, cols, v[i]);
        else
            for (int e = 0; e < 8; ++e)
                v[i][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max(m, mag(v[i][e]));
    for (int c = NV * kSpan + t * 8; c < cols; c += kSpan) {
        float w[8];
        load8<T>(x, c, cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max(m, mag(w[e]));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    const float s = q8_scale(m, mode);
    if (t == 0)
        gbl(it.scale)[row] = s;
    const bool bad = !(s == s);
    const float mul = s < 0x1p-90f ? 0x1p60f : 1.f;
    const float sm = s * mul, inv = 1.f / sm;
    auto put = [&](int c, const float (&w)[8]) __attribute__((always_inline)) {
        const u32x2 p = bad ? u32x2{0u, 0u} : quant8(w, sm, inv, mul);
        if (c + 8 <= cols) {
            store8_any(q + c, p);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < cols)
                    gbl(q)[c + e] = (int8_t)((e < 4 ? p.x : p.y) >> (8 * (e & 3)));
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * kSpan + t * 8;
        if (c < cols)
            put(c, v[i]);
    }
    for (int c = NV * kSpan + t * 8; c < cols; c += kSpan) {
        float w[8];
        load8<T>(x, c, cols, w);
        put(c, w);
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_q8_quantize(const Q8RowsBatch batch)
{
    __shared__ uint32_t red[4];
    const Q8RowsItem it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin;
    if (it.cols <= kQ8WaveCols) {
        const int row = 4 * b + (threadIdx.x >> 6);
        if (row < it.rows)
            quantize_row<DT, 1>(it, row, batch.mode, red);
    } else {
        quantize_row<DT, 4>(it, b, batch.mode, red);
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_q8_dequantize(const Q8RowsBatch batch)
{
    using T = typename Elt<DT>::type;
    const Q8RowsItem it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin;
    const bool wave = it.cols <= kQ8WaveCols;
    const int row = wave ? 4 * b + (int)(threadIdx.x >> 6) : b;
    if (row >= it.rows)
        return;
    const int t = wave ? threadIdx.x & 63 : threadIdx.x, step = wave ? 512 : 2048;
    T* x = static_cast<T*>(it.values) + row * it.ldv;
    const int8_t* q = it.q + row * it.ldq;
    const float s = gbl(it.scale)[row];
    for (int c = t * 8; c < it.cols; c += step) {
        if (c + 8 <= it.cols) {
            const u32x2 p = load8_any(q + c);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (float)(int8_t)((e < 4 ? p.x : p.y) >> (8 * (e & 3))) * s;
            if constexpr (DT == 0) {
                bf16x8 h;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[e] = (bf16)v[e];
                store16_any(x + c, __builtin_bit_cast(u32x4, h));
            } else {
                store16_any(x + c, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
                store16_any(x + c + 4, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
            }
        } else {
            for (int e = 0; c + e < it.cols; ++e)
                gbl(x)[c + e] = from_f32<T>((float)gbl(q)[c + e] * s);
        }
    }
}

// ---------------------------------------------------------------------------
// The plain tile kernel: any sizes, pitches and alignments. One workgroup
// computes a 64 x 64 tile of C = A B over one piece of the k axis, a 32 x 32
// MFMA block per wavefront, in slots of 64 bytes of k (64 int8 or 32 bf16)
// that pass through registers into LDS.
//
// Operands with k along their rows (A of matmul and grad_input, B of matmul)
// lie in LDS as 64 rows of 64 bytes at a pitch of 80: the 16-byte reads of
// eight lanes then meet 32 different banks. Those with k down their rows (dY
// of grad_weight, the 8-bit operand of both gradients) lie as 32 k-rows of 64
// bf16 at a pitch of 160 bytes and are read with ds_read_b64_tr_b16, which
// hands lane x of a 16-lane group the four k values of column x. The 8-bit
// operand of the gradients becomes q s, rounded to bf16, on its way into LDS.
constexpr int kPitchRow = 80, kPitchTr = 160;

typedef short v4i16 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 ds_read_tr(const char* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16*)(p)));
}

// 16 bytes of row r from element c on; elements past `cols` and rows past
// `rows` are 0.
template <typename T>
__device__ __forceinline__ u32x4 chunk16(const T* base, int64_t ld, int r, int rows, int c, int cols)
{
    constexpr int N = 16 / sizeof(T);
    if (r >= rows || c >= cols)
        return u32x4{0u, 0u, 0u, 0u};
    const T* p = base + r * ld + c;
    if (c + N <= cols)
        return load16_any(p);
    union { T t[N]; u32x4 v; } u;
    u.v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (c + e < cols)
            u.t[e] = gbl(p)[e];
    return u.v;
}

__device__ __forceinline__ u32x2 chunk8(const int8_t* base, int64_t ld, int r, int rows, int c, int cols)
{
    if (r >= rows || c >= cols)
        return u32x2{0u, 0u};
    const int8_t* p = base + r * ld + c;
    if (c + 8 <= cols)
        return load8_any(p);
    u32x2 v = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < cols)
            v[e >> 2] |= (uint32_t)(uint8_t)gbl(p)[e] << (8 * (e & 3));
    return v;
}

// Byte b of a word, as a signed integer in fp32.
__device__ __forceinline__ float byte_f32(uint32_t p, int b)
{
    return (float)(int)__builtin_amdgcn_sbfe((int)p, 8 * b, 8);
}

// Eight int8 as bf16(q s).
__device__ __forceinline__ u32x4 widen8(u32x2 p, float s)
{
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = (bf16)(byte_f32(p[e >> 2], e & 3) * s);
    return __builtin_bit_cast(u32x4, h);
}

// C element (r, c) from its sum.
template <int OP, int DT, typename AccT>
__device__ __forceinline__ void finish(const Q8Item& it, int r, int c, AccT sum, float beta)
{
    using T = typename Elt<DT>::type;
    NS_GLOBAL T* p = gbl(static_cast<T*>(it.out)) + (int64_t)r * it.ldo + c;
    float v = (float)sum;
    if (OP == kQ8Matmul)
        v = v * gbl(it.sa)[r] * gbl(it.sb)[c];
    if (OP == kQ8GradWeight && beta != 0.f)
        v = fmaf(beta, to_f32(*p), v);
    *p = from_f32<T>(v);
}

template <int OP, int DT>
__global__ __launch_bounds__(kThreads) void k_q8_tile(const Q8Batch batch)
{
    constexpr bool kInt = OP == kQ8Matmul;
    constexpr int kSlot = kInt ? 64 : 32;   // k values per slot
    using AccT = typename std::conditional<kInt, int, float>::type;
    using Acc = typename std::conditional<kInt, i32x16, f32x16>::type;
    __shared__ __attribute__((aligned(16))) char la[64 * kPitchRow];
    __shared__ __attribute__((aligned(16))) char lb[64 * kPitchRow];
    static_assert(32 * kPitchTr <= 64 * kPitchRow, "a k-row operand fits the same LDS");

    const Q8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin;
    const int tile = b / it.nsplit, piece = b - tile * it.nsplit;
    const int m0 = tile / it.ntn * kQ8Tile, n0 = tile % it.ntn * kQ8Tile;
    const int nslots = (it.k + kSlot - 1) / kSlot;
    const int s0 = piece * it.per, s1 = min(nslots, s0 + it.per);

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wr = wave >> 1, wc = wave & 1;
    const int row = tid >> 2, ch = tid & 3;      // of an operand with k along its rows
    const int kr = tid >> 3, c8 = (tid & 7) * 8; // of one with k down its rows

    u32x4 ra{}, rb{};
    u32x2 rq{};
    float rs = 0.f;
    auto fetch = [&](int s) __attribute__((always_inline)) {
        const int k0 = s * kSlot;
        if constexpr (OP == kQ8Matmul) {
            ra = chunk16(static_cast<const int8_t*>(it.a), it.lda, m0 + row, it.m, k0 + ch * 16, it.k);
            rb = chunk16(it.b, it.ldb, n0 + row, it.n, k0 + ch * 16, it.k);
        } else {
            if constexpr (OP == kQ8GradInput)
                ra = chunk16(static_cast<const bf16*>(it.a), it.lda, m0 + row, it.m, k0 + ch * 8, it.k);
            else
                ra = chunk16(static_cast<const bf16*>(it.a), it.lda, k0 + kr, it.k, m0 + c8, it.m);
            rq = chunk8(it.b, it.ldb, k0 + kr, it.k, n0 + c8, it.n);
            rs = k0 + kr < it.k ? gbl(it.sb)[k0 + kr] : 0.f;
        }
    };
    auto stash = [&]() __attribute__((always_inline)) {
        if constexpr (OP == kQ8GradWeight)
            *reinterpret_cast<u32x4*>(la + kr * kPitchTr + c8 * 2) = ra;
        else
            *reinterpret_cast<u32x4*>(la + row * kPitchRow + ch * 16) = ra;
        if constexpr (OP == kQ8Matmul)
            *reinterpret_cast<u32x4*>(lb + row * kPitchRow + ch * 16) = rb;
        else
            *reinterpret_cast<u32x4*>(lb + kr * kPitchTr + c8 * 2) = widen8(rq, rs);
    };
    // MFMA operand of k-step ks (32 int8 or 16 bf16): lane l takes row or
    // column l & 31 of its block, 16 bytes of k from (l >> 5) on
    const int fr = lane & 31, fg = lane >> 5;
    auto along = [&](const char* base, int blk, int ks) {
        return *reinterpret_cast<const u32x4*>(base + (blk * 32 + fr) * kPitchRow + (2 * ks + fg) * 16);
    };
    auto down = [&](const char* base, int blk, int ks) {
        const int g = lane >> 4, x = lane & 15;
        const char* p = base + (16 * ks + 8 * (g >> 1) + (x >> 2)) * kPitchTr +
                        (blk * 32 + 16 * (g & 1) + 4 * (x & 3)) * 2;
        const u32x2 v0 = ds_read_tr(p), v1 = ds_read_tr(p + 4 * kPitchTr);
        return u32x4{v0.x, v0.y, v1.x, v1.y};
    };

    Acc acc{};
    if (s0 < s1)
        fetch(s0);
    for (int s = s0; s < s1; ++s) {
        __syncthreads();
        stash();
        __syncthreads();
        if (s + 1 < s1)
            fetch(s + 1);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const u32x4 av = OP == kQ8GradWeight ? down(la, wr, ks) : along(la, wr, ks);
            const u32x4 bv = OP == kQ8Matmul ? along(lb, wc, ks) : down(lb, wc, ks);
            if constexpr (kInt)
                acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, av),
                                                            __builtin_bit_cast(i32x4, bv), acc, 0, 0, 0);
            else
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, av),
                                                              __builtin_bit_cast(bf16x8, bv), acc, 0, 0, 0);
        }
    }
    // register r of lane l: row 8 (r >> 2) + 4 (l >> 5) + (r & 3), column l & 31
    const int c = n0 + wc * 32 + fr;
    if (c < it.n) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int rr = m0 + wr * 32 + 8 * (r >> 2) + 4 * fg + (r & 3);
            if (rr < it.m) {
                if (it.nsplit == 1)
                    finish<OP, DT>(it, rr, c, (AccT)acc[r], batch.beta);
                else
                    gbl(reinterpret_cast<AccT*>(it.part))[((int64_t)piece * it.m + rr) * it.n + c] = acc[r];
            }
        }
    }
}

// C from the pieces of split sums, added in piece order. A thread takes
// elements 256 apart, so every piece is read in whole lines.
template <int OP, int DT>
__global__ __launch_bounds__(kThreads) void k_q8_join(const Q8Batch batch)
{
    using AccT = typename std::conditional<OP == kQ8Matmul, int, float>::type;
    const Q8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int64_t total = (int64_t)it.m * it.n;
    const int64_t e0 = (int64_t)(blockIdx.x - it.begin) * kQ8JoinElems;
    const NS_GLOBAL AccT* part = gbl(reinterpret_cast<const AccT*>(it.part));
#pragma unroll 4
    for (int64_t e = e0 + threadIdx.x; e < min(total, e0 + kQ8JoinElems); e += kThreads) {
        AccT sum = part[e];
        for (int p = 1; p < it.nsplit; ++p)
            sum += part[p * total + e];
        const int r = (int)(e / it.n);
        finish<OP, DT>(it, r, (int)(e - (int64_t)r * it.n), sum, batch.beta);
    }
}

// ---------------------------------------------------------------------------
// The large tile kernel: 256 x 256 outputs per workgroup of four wavefronts
// (2 x 2), 128 x 128 = 4 x 4 MFMA blocks of 32 x 32 each, the accumulators in
// the 256 AGPRs of each lane. k advances in slots of 64 bytes (64 int8 or 32
// bf16) through a ring of four LDS slots of 32 KB: while slot s is multiplied,
// slots s + 1 .. s + 3 stream in.
//
// Per slot a wavefront issues 32 MFMAs (about 1024 cycles) and reads 16 KB of
// fragments; the compute unit's LDS moves 64 KB of reads and 32 KB of writes in
// that time, three quarters of what it can, so the tile cannot be smaller and
// the matrix units still be fed.
//
// Operands with k along their rows (both of matmul, dY of grad_input) arrive
// by buffer_load ... lds, 16 bytes a lane: row r takes the 64 bytes at 64 r,
// its chunk c stored at chunk c ^ ((r >> 2) & 3). dY of grad_weight (k down its
// rows) arrives the same way as 32 k-rows of 512 bytes, chunk c of row k
// at c ^ ((k & 3) << 2), and is read transposing. The 8-bit operand of the
// gradients passes through registers: 32 bytes a lane, loaded five slots
// ahead, widened to bf16(q s) and written three slots ahead in the same k-row
// layout. Widening costs 2.5 vector operations a value, 32 values a lane and
// slot, which issue between the MFMAs.
//
// Buffer resources end with the operand (rounded up to the 16 bytes that its
// alignment allows), so rows past the end and k-rows past the end read as 0.
// Along a row, k past the end is not zero in memory: the one slot that holds
// it is cleared in LDS before it is read.
constexpr int kOpBytes = kQ8Big * 64;   // one operand of a slot
typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ int up16(int v) { return (v + 15) & ~15; }
__device__ __forceinline__ int swz_row(int r) { return (r >> 2) & 3; }
__device__ __forceinline__ int swz_tr(int k) { return (k & 3) << 2; }

// Workgroup b of n, with neighbours in the list on the same XCD (workgroups go
// round the eight XCDs), so that tiles which share operands share an L2.
__device__ __forceinline__ int by_xcd(int b, int n)
{
    const int x = b & 7, per = n >> 3, rem = n & 7;
    return x * per + min(x, rem) + (b >> 3);
}

template <int OP, int DT>
__global__ __launch_bounds__(kThreads, 1) void k_q8_big(const Q8Batch batch, int nwg)
{
    constexpr bool kInt = OP == kQ8Matmul;
    constexpr bool kWiden = !kInt;              // B passes through registers
    constexpr bool kTA = OP == kQ8GradWeight;   // A with k down its rows
    constexpr int kSlot = kInt ? 64 : 32;
    constexpr int kEltA = kInt ? 1 : 2;
    using AccT = typename std::conditional<kInt, int, float>::type;
    using Acc = typename std::conditional<kInt, i32x16, f32x16>::type;
    // One object per slot, so that every access names its slot statically, and
    // one more for an operand that is written from registers: the compiler
    // lets such a write wait for every DMA into the same object.
    constexpr int kObjA = kInt ? 2 * kOpBytes : kOpBytes, kObjB = kInt ? 16 : kOpBytes;
    __shared__ __attribute__((aligned(1024))) char sa0[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa1[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa2[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa3[kObjA];
    __shared__ __attribute__((aligned(1024))) char sb0[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb1[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb2[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb3[kObjB];
    __shared__ __attribute__((aligned(16))) float lscale[kInt ? 512 : 4];   // of the tile's rows, of its columns
    struct Slot { char *a, *b; };
    const Slot sl0 = {sa0, kInt ? sa0 + kOpBytes : sb0}, sl1 = {sa1, kInt ? sa1 + kOpBytes : sb1};
    const Slot sl2 = {sa2, kInt ? sa2 + kOpBytes : sb2}, sl3 = {sa3, kInt ? sa3 + kOpBytes : sb3};

    const int wg = by_xcd(blockIdx.x, nwg);
    const Q8Item it = batch.it[find_item(batch, wg)];
    const int t = wg - it.begin;
    // four tile rows at a time, down each column of them: the 32 workgroups
    // of an XCD then share 4 blocks of A and 8 of B
    const int ntm = (it.m + kQ8Big - 1) / kQ8Big;
    const int grp = t / (4 * it.ntn), left = t - grp * 4 * it.ntn;
    const int gh = min(4, ntm - 4 * grp);
    const int m0 = (4 * grp + left % gh) * kQ8Big, n0 = left / gh * kQ8Big;
    const int K = it.k, ns = (K + kSlot - 1) / kSlot;
    const int rows = min(kQ8Big, it.m - m0), cols = min(kQ8Big, it.n - n0);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave >> 1, wc = wave & 1;
    const int fr = lane & 31, fg = lane >> 5;

    const char* A = static_cast<const char*>(it.a) + (kTA ? (int64_t)m0 * 2 : (int64_t)m0 * it.lda * kEltA);
    const char* B = reinterpret_cast<const char*>(it.b) + (kInt ? (int64_t)n0 * it.ldb : (int64_t)n0);
    const int lda = it.lda * kEltA, ldb = it.ldb;   // bytes
    const __amdgpu_buffer_rsrc_t ra = buffer(A, kTA ? 0 : up16((rows - 1) * lda + K * kEltA));
    const __amdgpu_buffer_rsrc_t rb = buffer(B, kInt ? up16((cols - 1) * ldb + K) : 0);
    const __amdgpu_buffer_rsrc_t rs = buffer(it.sb, kWiden ? K * 4 : 0);

    // DMA: wavefront w fills instructions w + 4 q of a slot operand, 1 KB each:
    // rows 16 I .. + 15 (lane l the stored chunk l & 3 of row l >> 2), or k-rows
    // 2 I, 2 I + 1 (lane l the stored chunk l & 31 of row l >> 5).
    const int row_n = 16 * wave + (lane >> 2), row_t = 2 * wave + (lane >> 5);
    const int chunk_n = ((lane & 3) ^ swz_row(row_n)) << 4;
    const int voff_a = kTA ? row_t * lda + (((lane & 31) ^ swz_tr(row_t)) << 4) : row_n * lda + chunk_n;
    const int voff_b = row_n * ldb + chunk_n;
    auto issue = [&](const Slot& sp, int s, int q0, int q1) __attribute__((always_inline)) {
        // slots past the end read as 0 and keep the count of loads uniform
        if constexpr (kTA) {
            // (a pitch is at least a row: no k-rows left give 0 bytes)
            const int k0 = s * kSlot;
            const __amdgpu_buffer_rsrc_t r =
                buffer(A + (int64_t)k0 * lda, max(0, (min(kSlot, K - k0) - 1) * lda + up16(rows * 2)));
#pragma unroll
            for (int q = q0; q < q1; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(sp.a + (wave + 4 * q) * 1024), 16, voff_a,
                                                         8 * q * lda, 0, 0);
        } else {
#pragma unroll
            for (int q = q0; q < q1; ++q) {
                const int so = s < ns ? s * 64 : 0x40000000;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(sp.a + (wave + 4 * q) * 1024), 16, voff_a,
                                                         so + (s < ns ? 64 * q * lda : 0), 0, 0);
                if constexpr (kInt)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(sp.b + (wave + 4 * q) * 1024),
                                                             16, voff_b, so + (s < ns ? 64 * q * ldb : 0), 0, 0);
            }
        }
    };

    // The 8-bit operand of the gradients: thread t holds k-row t >> 3, columns
    // 16 (t & 7) + 0 .. 15 and the same 128 further, of the slot.
    struct Raw { u32x4 lo, hi; float s; };
    const int krow = tid >> 3, kcol = (tid & 7) * 16;
    auto fetch = [&](int s) __attribute__((always_inline)) {
        const int k0 = s * kSlot;
        const __amdgpu_buffer_rsrc_t r =
            buffer(B + (int64_t)k0 * ldb, max(0, (min(kSlot, K - k0) - 1) * ldb + up16(cols)));
        Raw w;
        w.lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, krow * ldb + kcol, 0, 0));
        w.hi = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, krow * ldb + kcol + 128, 0, 0));
        w.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (k0 + krow) * 4, 0, 0));
        return w;
    };
    // columns kcol + 128 h + 0 .. 15: chunks 2 (t & 7) + 16 h and the next
    const int wide_at = krow * 512, wide_c = 2 * (tid & 7);
    auto widen = [&](const Slot& sp, const Raw& w, int h) __attribute__((always_inline)) {
        const u32x4 v = h ? w.hi : w.lo;
        *reinterpret_cast<u32x4*>(sp.b + wide_at + (((wide_c + 16 * h) ^ swz_tr(krow)) << 4)) =
            widen8(u32x2{v.x, v.y}, w.s);
        *reinterpret_cast<u32x4*>(sp.b + wide_at + (((wide_c + 16 * h + 1) ^ swz_tr(krow)) << 4)) =
            widen8(u32x2{v.z, v.w}, w.s);
    };

    // Fragments: lane l of k-step ks takes row l & 31 of its block and 16 bytes
    // of k from 2 ks + (l >> 5) on; a transposing read covers k-rows
    // 16 ks + 8 (g >> 1) + (x >> 2) (+ 4) and columns 16 (g & 1) + 4 (x & 3).
    auto off_n = [&](int base) {
        const int r = base + fr;
        return r * 64 + ((fg ^ swz_row(r)) << 4);
    };
    auto off_t = [&](int base) {
        const int g = lane >> 4, x = lane & 15;
        const int kr = 8 * (g >> 1) + (x >> 2), cl = base + 16 * (g & 1) + 4 * (x & 3);
        return kr * 512 + (((cl >> 3) ^ swz_tr(kr)) << 4) + (cl & 7) * 2;
    };
    int aoff[4], boff[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        aoff[i] = kTA ? off_t(wr * 128 + i * 32) : off_n(wr * 128 + i * 32);
        boff[i] = kInt ? off_n(wc * 128 + i * 32) : off_t(wc * 128 + i * 32);
    }
    auto read_frag = [&](const char* sp, int off, int ks, bool tr) __attribute__((always_inline)) {
        if (tr) {
            const u32x2 v0 = ds_read_tr(sp + off + ks * 8192), v1 = ds_read_tr(sp + off + ks * 8192 + 2048);
            return u32x4{v0.x, v0.y, v1.x, v1.y};
        }
        return *reinterpret_cast<const u32x4*>(sp + (off ^ (ks << 5)));
    };
    auto read_frags = [&](const Slot& sp, int ks, u32x4 (&af)[4], u32x4 (&bf)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            af[i] = read_frag(sp.a, aoff[i], ks, kTA);
            bf[i] = read_frag(sp.b, boff[i], ks, kWiden);
        }
    };
    Acc acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = Acc{};
    auto multiply = [&](const u32x4 (&af)[4], const u32x4 (&bf)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (kInt)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                        __builtin_bit_cast(i32x4, af[i]), __builtin_bit_cast(i32x4, bf[j]), acc[i][j], 0, 0, 0);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, af[i]), __builtin_bit_cast(bf16x8, bf[j]), acc[i][j], 0, 0, 0);
            }
    };
    // The order within half a step: the reads of the next k-step, the loads
    // and the widening spread between the 16 MFMAs.
    auto interleave = []() __attribute__((always_inline)) {
        constexpr int reads = (kTA ? 8 : 4) + (kWiden ? 8 : 4);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            if (q % 4 == 0)
                __builtin_amdgcn_sched_group_barrier(0x010, kWiden ? 2 : 1, 0);
            if (q < reads)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (kWiden)
                __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
            if (kWiden && (q == 8 || q == 15))
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
    };
    // k past the end in the slot that holds it: 0 in A (its B is 0 or finite)
    const int tail = K % kSlot;   // k values in it, when not whole
    const int tail_slot = !kTA && tail ? ns - 1 : -1;
    auto clear_tail = [&](const Slot& sp) __attribute__((always_inline)) {
        // thread t clears row t
        const int r = tid, b0 = tail * kEltA;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (16 * c + 16 <= b0)
                continue;
            u32x4* p = reinterpret_cast<u32x4*>(sp.a + r * 64 + ((c ^ swz_row(r)) << 4));
            u32x4 v = *p;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int over = b0 - (16 * c + 4 * e);   // bytes of this word to keep
                v[e] = over >= 4 ? v[e] : over <= 0 ? 0u : v[e] & (0xFFFFFFFFu >> (32 - 8 * over));
            }
            *p = v;
        }
        __syncthreads();
    };

    // The pipeline. Step s multiplies slot s; it refills the ring position of
    // slot s - 1 (free since the barrier in step s - 1) with slot s + 3. Its
    // wait leaves the loads younger than slot s + 1 in flight (matmul: the 8 of
    // slot s + 2 and 4 of slot s + 3; gradients: 7 and 5 with the widened
    // operand's), the barrier then makes slot s + 1 whole for everyone.
    u32x4 fa[4], fb[4], ga[4], gb[4];
    Raw w0{}, w1{};
    auto step = [&](const Slot& cur, const Slot& refill, const Slot& next, int s, Raw& w) __attribute__((always_inline)) {
        Raw fresh{};
        issue(refill, s + 3, 0, 2);
        if constexpr (kWiden)
            fresh = fetch(s + 5);
        read_frags(cur, 1, ga, gb);
        if constexpr (kWiden)
            widen(refill, w, 0);
        multiply(fa, fb);
        interleave();
        asm volatile("s_waitcnt vmcnt(12)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if constexpr (!kTA)
            if (s + 1 == tail_slot)
                clear_tail(next);
        issue(refill, s + 3, 2, 4);
        read_frags(next, 0, fa, fb);
        if constexpr (kWiden)
            widen(refill, w, 1);
        multiply(ga, gb);
        interleave();
        w = fresh;
    };
    if constexpr (kInt) {
        lscale[tid] = tid < rows ? gbl(it.sa)[m0 + tid] : 0.f;
        lscale[256 + tid] = tid < cols ? gbl(it.sb)[n0 + tid] : 0.f;
    }
    // (slot 2's loads go last: the first wait leaves them alone in flight)
    if constexpr (kWiden) {
        // slots 0 .. 2 whole, 3 and 4 in registers
        const Raw p0 = fetch(0), p1 = fetch(1), p2 = fetch(2);
        w0 = fetch(3);
        w1 = fetch(4);
        widen(sl0, p0, 0);
        widen(sl0, p0, 1);
        widen(sl1, p1, 0);
        widen(sl1, p1, 1);
        widen(sl2, p2, 0);
        widen(sl2, p2, 1);
    }
    issue(sl0, 0, 0, 4);
    issue(sl1, 1, 0, 4);
    asm volatile("" ::: "memory");
    issue(sl2, 2, 0, 4);
    if constexpr (kInt)
        asm volatile("s_waitcnt vmcnt(8)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
        asm volatile("s_waitcnt vmcnt(4)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (tail_slot == 0)
        clear_tail(sl0);
    read_frags(sl0, 0, fa, fb);
    for (int s = 0; s < ns; s += 4) {
        step(sl0, sl3, sl1, s, w0);
        step(sl1, sl0, sl2, s + 1, w1);
        step(sl2, sl1, sl3, s + 2, w0);
        step(sl3, sl2, sl0, s + 3, w1);
    }
    // (loads of slots past the end are still to land in LDS, which outlives them)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // Register r of lane l, block (i, j): row 32 i + 8 (r >> 2) + 4 (l >> 5) +
    // (r & 3), column 32 j + (l & 31) of the wavefront's 128 x 128. The tile is
    // written through a buffer resource: rows past the end fall behind it,
    // and lanes with columns past the end get an offset behind it.
    using T = typename Elt<DT>::type;
    constexpr int kElt = sizeof(T);
    const int ldo = it.ldo * kElt;
    const __amdgpu_buffer_rsrc_t ro =
        buffer(static_cast<const T*>(it.out) + (int64_t)m0 * it.ldo + n0, (rows - 1) * ldo + cols * kElt);
    const float beta = batch.beta;
    const int row0 = wr * 128, col0 = wc * 128 + fr;
    // row scales of the four rows of a register group, and the column scale
    auto value = [&](int i, int j, int r, const f32x4& sa, float sb) __attribute__((always_inline)) {
        const float v = (float)(AccT)acc[i][j][r];
        return kInt ? v * sa[r & 3] * sb : v;
    };
    float colscale[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (kInt) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            colscale[j] = lscale[256 + col0 + 32 * j];
    }
    if (DT == 0 && ((it.n | it.ldo) & 1) == 0 && (reinterpret_cast<uintptr_t>(it.out) & 3) == 0) {
        // bf16 in pairs of columns: of two rows, an even lane takes the first
        // and its neighbour's value of it, an odd lane the second
        const bool odd = fr & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = col0 + 32 * j - odd;
            const int vo = c < cols ? (4 * fg + odd) * ldo + c * kElt : (int)0x80000000;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t g[8];
                if (OP == kQ8GradWeight && beta != 0.f) {
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        g[p] = __builtin_amdgcn_raw_buffer_load_b32(
                            ro, vo, (row0 + 32 * i + 8 * (p >> 1) + 2 * (p & 1)) * ldo, 0);
                }
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const int r = 2 * p, lr = row0 + 32 * i + 8 * (r >> 2);
                    f32x4 sa{};
                    if constexpr (kInt)
                        sa = *reinterpret_cast<const f32x4*>(&lscale[lr + 4 * fg]);
                    const float v0 = value(i, j, r, sa, colscale[j]), v1 = value(i, j, r + 1, sa, colscale[j]);
                    const float other = __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(
                        __builtin_bit_cast(int, odd ? v0 : v1), 0xB1, 0xF, 0xF, true));
                    float lo = odd ? other : v0, hi = odd ? v1 : other;
                    if (OP == kQ8GradWeight && beta != 0.f) {
                        lo = fmaf(beta, __uint_as_float(g[p] << 16), lo);
                        hi = fmaf(beta, __uint_as_float(g[p] & 0xFFFF0000u), hi);
                    }
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    const bf16x2 h = {(bf16)lo, (bf16)hi};
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, h), ro, vo,
                                                          (lr + (r & 3)) * ldo, 0);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = col0 + 32 * j;
        const int vo = c < cols ? 4 * fg * ldo + c * kElt : (int)0x80000000;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float g[16];
            if (OP == kQ8GradWeight && beta != 0.f) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int so = (row0 + 32 * i + 8 * (r >> 2) + (r & 3)) * ldo;
                    if constexpr (DT == 0)
                        g[r] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ro, vo, so, 0) << 16);
                    else
                        g[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ro, vo, so, 0));
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int lr = row0 + 32 * i + 8 * (r >> 2), so = (lr + (r & 3)) * ldo;
                f32x4 sa{};
                if constexpr (kInt)
                    sa = *reinterpret_cast<const f32x4*>(&lscale[lr + 4 * fg]);
                float v = value(i, j, r, sa, colscale[j]);
                if (OP == kQ8GradWeight && beta != 0.f)
                    v = fmaf(beta, g[r], v);
                if constexpr (DT == 0)
                    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)v), ro, vo, so, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ro, vo, so, 0);
            }
        }
    }
}

}  // namespace

hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream)
{
    if (dtype == 0)
        hipLaunchKernelGGL(k_q8_quantize<0>, dim3(nwg), dim3(kThreads), 0, stream, b);
    else
        hipLaunchKernelGGL(k_q8_quantize<1>, dim3(nwg), dim3(kThreads), 0, stream, b);
    return hipGetLastError();
}

hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream)
{
    if (dtype == 0)
        hipLaunchKernelGGL(k_q8_dequantize<0>, dim3(nwg), dim3(kThreads), 0, stream, b);
    else
        hipLaunchKernelGGL(k_q8_dequantize<1>, dim3(nwg), dim3(kThreads), 0, stream, b);
    return hipGetLastError();
}

// The instantiation of kernel template K<op, dtype> for run-time op and dtype
// (grad_input's output is always bf16).
#define NS_Q8_LAUNCH(K, threads)                                                                    \
    do {                                                                                            \
        if (op == kQ8Matmul && dtype == 0)                                                          \
            hipLaunchKernelGGL((K<kQ8Matmul, 0>), dim3(nwg), dim3(threads), 0, stream, b);          \
        else if (op == kQ8Matmul)                                                                   \
            hipLaunchKernelGGL((K<kQ8Matmul, 1>), dim3(nwg), dim3(threads), 0, stream, b);          \
        else if (op == kQ8GradInput)                                                                \
            hipLaunchKernelGGL((K<kQ8GradInput, 0>), dim3(nwg), dim3(threads), 0, stream, b);       \
        else if (dtype == 0)                                                                        \
            hipLaunchKernelGGL((K<kQ8GradWeight, 0>), dim3(nwg), dim3(threads), 0, stream, b);      \
        else                                                                                        \
            hipLaunchKernelGGL((K<kQ8GradWeight, 1>), dim3(nwg), dim3(threads), 0, stream, b);      \
    } while (0)

hipError_t launch_q8_tile(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    NS_Q8_LAUNCH(k_q8_tile, kThreads);
    return hipGetLastError();
}

hipError_t launch_q8_big(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    if (op == kQ8Matmul && dtype == 0)
        hipLaunchKernelGGL((k_q8_big<kQ8Matmul, 0>), dim3(nwg), dim3(kThreads), 0, stream, b, nwg);
    else if (op == kQ8Matmul)
        hipLaunchKernelGGL((k_q8_big<kQ8Matmul, 1>), dim3(nwg), dim3(kThreads), 0, stream, b, nwg);
    else if (op == kQ8GradInput)
        hipLaunchKernelGGL((k_q8_big<kQ8GradInput, 0>), dim3(nwg), dim3(kThreads), 0, stream, b, nwg);
    else if (dtype == 0)
        hipLaunchKernelGGL((k_q8_big<kQ8GradWeight, 0>), dim3(nwg), dim3(kThreads), 0, stream, b, nwg);
    else
        hipLaunchKernelGGL((k_q8_big<kQ8GradWeight, 1>), dim3(nwg), dim3(kThreads), 0, stream, b, nwg);
    return hipGetLastError();
}

hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    NS_Q8_LAUNCH(k_q8_join, kThreads);
    return hipGetLastError();
}

}  // namespace ns

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

// Eight int8 as bf16(q s).
__device__ __forceinline__ u32x4 widen8(u32x2 p, float s)
{
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = (bf16)((float)(int8_t)(p[e >> 2] >> (8 * (e & 3))) * s);
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

hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    NS_Q8_LAUNCH(k_q8_join, kThreads);
    return hipGetLastError();
}

}  // namespace ns

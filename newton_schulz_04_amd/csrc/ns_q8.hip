// ns_q8.hip -- gfx950 kernels of the 8-bit linear layers (include/ns.h,
// ns_q8_*): rows to int8 with a scale each and back, and the three products of
// a layer, Y = Xq Wq^T, dX = dY Wq and G = beta G + dY^T Xq.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ns.h"
#include "ns_device.h"
#include "ns_q8.h"

namespace ns {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Rows to int8 and back.
//
// s from m = max |x| of the row, q = rne(x / s). Both kernels move every byte
// once (a row longer than its workgroup's registers is read twice), so memory
// bandwidth bounds them: 8192 x 6144 bf16 36 us to int8 (4.2 TB/s) and 23 us back
// (6.6 TB/s: what was just written partly comes from the last-level cache), 59
// us together at 5.1 TB/s, the rate of a large copy; 24 fp32 matrices of 1531 x
// 1027 45 and 31 us.

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

template <int DT, int N>
__global__ __launch_bounds__(kThreads) void k_q8_quantize(const Q8RowsBatchOf<N> batch)
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

template <int DT, int N>
__global__ __launch_bounds__(kThreads) void k_q8_dequantize(const Q8RowsBatchOf<N> batch)
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
// The products C = A B, in tiles of C.
//
// A workgroup of four wavefronts (2 x 2) computes a tile of 64 MI x 64 NJ
// outputs, MI x NJ MFMA blocks of 32 x 32 a wavefront. k advances in slots of
// 64 bytes (64 int8 or 32 bf16) through a ring of RING = 3 or 4 LDS slots:
// while slot s is multiplied, the RING - 1 after it stream in.
//
// Operands with k along their rows (both of matmul, dY of grad_input) arrive
// by buffer_load ... lds, 16 bytes a lane: row r takes the 64 bytes at 64 r,
// its chunk c stored at chunk c ^ ((r >> 2) & 3). dY of grad_weight (k down its
// rows) arrives the same way as 32 k-rows, chunk c of row k at
// c ^ ((k & 3) << 2), and is read with ds_read_b64_tr_b16, which hands lane x of
// a 16-lane group four k values of column x. The 8-bit operand of the
// gradients passes through registers: loaded five slots ahead, widened to bf16
// and written RING - 1 slots ahead in the same k-row layout. Widening costs 2.5
// vector operations a value, which issue between the MFMAs.
//
// q s has 8 + 24 bits, bf16 8. Its leading 8 bits alone are all of it when s is
// a power of two. Otherwise their cut would be off by up to 2^-7 of every term,
// more than the output's own rounding, so the sum runs over k again with what
// they left out (see `widen8_rest`): once more for bf16 outputs, twice more for
// fp32 ones, into the same sums. A workgroup looks at the scales of its part of
// k first, and takes the one pass where all are powers of two: 4096 tokens,
// 8192 x 6144, dX 747 us in two parts and 361 in one. (A second operand beside
// the first in each slot would not fit the LDS of the large tiles, whose time the
// matrix units bound either way.)
//
// Buffer resources end with the operand (rounded up to the 16 bytes that its
// alignment allows), so rows past the end and k-rows past the end read as 0.
// Along a row, k past the end is not zero in memory: the one slot that holds
// it is cleared in LDS before it is read.
//
// Every tile size and both ways of cutting the output run a sum's terms in the
// same order, so which one a call takes does not show in the bits.
#ifdef __HIP_DEVICE_COMPILE__   // (the tiles' builtins and resources do not exist on the host)
typedef short v4i16 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 ds_read_tr(const char* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16*)(p)));
}

// Byte b of a word, as a signed integer in fp32.
__device__ __forceinline__ float byte_f32(uint32_t p, int b)
{
    return (float)(int)__builtin_amdgcn_sbfe((int)p, 8 * b, 8);
}

// The leading 8 bits of a float, as a float, and those of eight as bf16.
__device__ __forceinline__ float lead(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
__device__ __forceinline__ u32x4 leads8(const float (&v)[8])
{
    u32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = __builtin_amdgcn_perm(__float_as_uint(v[2 * e + 1]), __float_as_uint(v[2 * e]), 0x07060302u);
    return h;
}

// Eight int8 times s, rounded to fp32, to their leading bits: value e is byte
// b[e] of word w[e].
template <typename W, typename B>
__device__ __forceinline__ u32x4 widen8(W&& w, B&& b, float s)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = byte_f32(w(e), b(e)) * s;
    return leads8(v);
}

// What widen8 leaves of v = q s. In two parts (P == 2) the rest of it, rounded
// to bf16: off by at most 2^-7 2^-8 v. In three, the rest's leading 8 bits
// (part 1) or what they leave in turn (part 2): all 24 bits of v. 2^-48 v is
// added to each, which no sum of a 2^-24 v shows, so that a part beside a v that
// is not zero is not zero either, and has v's sign: an Inf of dY times the parts
// then adds up to the Inf that it is times v, and never to a NaN.
template <int P, typename W, typename B>
__device__ __forceinline__ u32x4 widen8_rest(W&& w, B&& b, float s, int part)
{
#pragma clang fp contract(off)   // (v is the rounded product that widen8 cuts)
    const uint32_t cut = P == 3 && part == 2 ? 0xFFFF0000u : 0u;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = byte_f32(w(e), b(e)) * s;
        r[e] = fmaf(v, 0x1p-48f, v - lead(v));
        if constexpr (P == 3)
            r[e] = fmaf(v, 0x1p-48f, r[e] - __uint_as_float(__float_as_uint(r[e]) & cut));
    }
    if constexpr (P == 3)
        return leads8(r);
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = (bf16)r[e];
    return __builtin_bit_cast(u32x4, h);
}

__device__ __forceinline__ int up16(int v) { return (v + 15) & ~15; }
__device__ __forceinline__ int swz_row(int r) { return (r >> 2) & 3; }
__device__ __forceinline__ int swz_tr(int k) { return (k & 3) << 2; }

#endif

// A token's scale for matmul's outputs, sum s_t s_o: sum s_t alone would pass
// fp32's range from s_t = 2^97 on, so large scales enter 2^-64 times themselves,
// which `back` undoes at the end (one multiplication an output, by 1 for all
// other tokens; neither factor rounds).
struct TokenScale { float s, back; };
__device__ __forceinline__ TokenScale token_scale(float s)
{
    const bool large = s > 0x1p90f;
    return {large ? s * 0x1p-64f : s, large ? 0x1p64f : 1.f};
}
__device__ __forceinline__ float scaled(int sum, TokenScale t, float channel)
{
    return (float)sum * t.s * channel * t.back;
}

// LDS of one slot: its operands (one object each where the second is written
// from registers, as the compiler lets such a write wait for every DMA into
// the same object).
struct Slot { char *a, *b; };

// k values a slot holds.
template <int OP> constexpr int slot_k() { return OP == kQ8Matmul ? 64 : 32; }
// Parts that the 8-bit operand enters in, by the output's type.
template <int OP, int DT> constexpr int parts() { return OP == kQ8Matmul ? 1 : DT == 0 ? 2 : 3; }

// The tile at (m0, n0) over slots [s0, s1) of k; piece: which of it.nsplit.
// P: parts that the 8-bit operand enters in. lscale: LDS for the scales of
// matmul, 64 (MI + NJ) floats.
template <int OP, int DT, int MI, int NJ, int RING, int P>
__device__ __forceinline__ void q8_tile(const Q8Item& it, int m0, int n0, int s0, int s1, int piece, float beta,
                                        const Slot sl0, const Slot sl1, const Slot sl2, const Slot sl3,
                                        float* lscale)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr bool kInt = OP == kQ8Matmul;
    constexpr bool kWiden = !kInt;              // B passes through registers
    constexpr bool kTA = OP == kQ8GradWeight;   // A with k down its rows
    constexpr int kSlot = slot_k<OP>();
    constexpr int kEltA = kInt ? 1 : 2;
    constexpr int BM = 64 * MI, BN = 64 * NJ;
    using AccT = typename std::conditional<kInt, int, float>::type;
    using Acc = typename std::conditional<kInt, i32x16, f32x16>::type;

    const int K = it.k, ns = (K + kSlot - 1) / kSlot;
    const int rows = min(BM, it.m - m0), cols = min(BN, it.n - n0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave >> 1, wc = wave & 1;
    const int fr = lane & 31, fg = lane >> 5;

    const char* A = static_cast<const char*>(it.a) + (kTA ? (int64_t)m0 * 2 : (int64_t)m0 * it.lda * kEltA);
    const char* B = reinterpret_cast<const char*>(it.b) + (kInt ? (int64_t)n0 * it.ldb : (int64_t)n0);
    const int lda = it.lda * kEltA, ldb = it.ldb;   // bytes
    const int size_a = kTA ? 0 : up16((rows - 1) * lda + K * kEltA), size_b = kInt ? up16((cols - 1) * ldb + K) : 0;
    const __amdgpu_buffer_rsrc_t ra = buffer(A, size_a), rb = buffer(B, size_b);
    const __amdgpu_buffer_rsrc_t rs = buffer(it.sb, kWiden ? K * 4 : 0);

    // Columns of C: block j of a wavefront's kCols takes every NJ-th of them
    // from j on, so that lane l holds columns NJ (l & 31) + 0 .. NJ - 1 of each of
    // its rows, and a row's part leaves as one piece of 32 lanes. B lies in LDS
    // in that order.
    constexpr int kCols = 32 * NJ;

    // DMA: wavefront w fills instructions w + 4 q of a slot operand, 1 KB each:
    // rows 16 I .. + 15 (lane l the stored chunk l & 3 of row l >> 2), or k-rows
    // of BM / 8 chunks, kRows of them.
    constexpr int kChunks = BM / 8, kRows = 64 / kChunks;
    const int row_n = 16 * wave + (lane >> 2), row_t = kRows * wave + lane / kChunks;
    const int chunk_n = ((lane & 3) ^ swz_row(row_n)) << 4;
    // Whatever may lie past an operand's end (rows of A and B, k-rows) is in
    // the lanes' offsets, which the resource checks; the scalar offset is the
    // position along the rows, or the operand's size for slots past the end.
    int voff_a[MI], voff_b[NJ];
#pragma unroll
    for (int q = 0; q < MI; ++q)
        voff_a[q] = kTA ? (row_t + 4 * kRows * q) * lda + (((lane % kChunks) ^ swz_tr(row_t)) << 4)
                        : (row_n + 64 * q) * lda + chunk_n;
#pragma unroll
    for (int q = 0; q < NJ; ++q) {
        // LDS row 32 NJ part + 32 j + p holds row 32 NJ part + NJ p + j (see kCols)
        const int r = row_n + 64 * q, rem = r % kCols;
        voff_b[q] = (r - rem + NJ * (rem % 32) + rem / 32) * ldb + chunk_n;
    }
    // Bytes of 32 k-rows at a pitch of which `left` exist, `width` bytes used
    // of each.
    auto krows = [&](int left, int pitch, int width) __attribute__((always_inline)) {
        const int live = left > 0 ? -1 : 0;
        return ((min(kSlot, left) - 1) * pitch + up16(width)) & live;
    };
    auto issue = [&](const Slot& sp, int s, bool second) __attribute__((always_inline)) {
        // slots past the end read as 0 and keep the count of loads uniform
        const bool in = s < s1;
        if constexpr (kTA) {
            const int k0 = s * kSlot;
            const __amdgpu_buffer_rsrc_t r =
                buffer(A + (int64_t)k0 * lda, krows(in ? K - k0 : 0, lda, rows * 2));
#pragma unroll
            for (int q = second ? (MI + 1) / 2 : 0; q < (second ? MI : (MI + 1) / 2); ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(sp.a + (wave + 4 * q) * 1024), 16, voff_a[q],
                                                         0, 0, 0);
        } else {
            const int so_a = in ? s * 64 : size_a, so_b = in ? s * 64 : size_b;
#pragma unroll
            for (int q = second ? (MI + 1) / 2 : 0; q < (second ? MI : (MI + 1) / 2); ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(sp.a + (wave + 4 * q) * 1024), 16, voff_a[q],
                                                         so_a, 0, 0);
            if constexpr (kInt) {
#pragma unroll
                for (int q = second ? (NJ + 1) / 2 : 0; q < (second ? NJ : (NJ + 1) / 2); ++q)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(sp.b + (wave + 4 * q) * 1024), 16,
                                                             voff_b[q], so_b, 0, 0);
            }
        }
    };

    // The 8-bit operand of the gradients: thread t holds k-row t >> 3 of the
    // slot, columns 8 NJ (t & 7) + 0 .. 8 NJ - 1, and writes eight of them to
    // each of NJ blocks.
    constexpr int kLoads = NJ / 2;   // of 16 bytes
    static_assert(!kWiden || NJ == 2 || NJ == 4, "tiles of 128 or 256 columns");
    struct Raw { u32x4 v[kWiden ? kLoads : 1]; float s; };
    const int krow = tid >> 3;
    auto fetch = [&](int s) __attribute__((always_inline)) {
        const int k0 = s * kSlot;
        const __amdgpu_buffer_rsrc_t r = buffer(B + (int64_t)k0 * ldb, krows(s < s1 ? K - k0 : 0, ldb, cols));
        Raw w;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            w.v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   r, krow * ldb + 8 * NJ * (tid & 7) + 16 * i, 0, 0));
        w.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (k0 + krow) * 4, 0, 0));
        return w;
    };
    // 16-byte chunk c of k-row k in LDS, c < 8 NJ: the rows' swizzle, and (512
    // byte rows) one that keeps the two wavefront columns' writes apart
    auto chunk_b = [&](int k, int c) { return (c ^ swz_tr(k) ^ (NJ == 4 ? (c >> 4) << 2 : 0)) << 4; };
    // Half of the blocks, h = 0 or 1, of what a thread holds, in the part that
    // the pass over k adds.
    int part = 0;
    auto widen = [&](auto rest, const Slot& sp, const Raw& w, int h) __attribute__((always_inline)) {
        char* row = sp.b + krow * (2 * BN);
#pragma unroll
        for (int j = h * kLoads; j < (h + 1) * kLoads; ++j) {
            auto word = [&](int e) { return NJ == 4 ? w.v[e >> 2][e & 3] : w.v[0][e >> 1]; };
            auto byte = [&](int e) { return NJ == 4 ? j : j + 2 * (e & 1); };
            const int c = (tid >> 2 & 1) * 4 * NJ + 4 * j + (tid & 3);
            u32x4* p = reinterpret_cast<u32x4*>(row + chunk_b(krow, c));
            if constexpr (decltype(rest)::value)
                *p = widen8_rest<P>(word, byte, w.s, part);
            else
                *p = widen8(word, byte, w.s);
        }
    };

    // Fragments: lane l of k-step ks takes row l & 31 of its block and 16 bytes
    // of k from 2 ks + (l >> 5) on; a transposing read covers k-rows
    // 16 ks + 8 (g >> 1) + (x >> 2) (+ 4) and columns 16 (g & 1) + 4 (x & 3).
    auto off_n = [&](int base) {
        const int r = base + fr;
        return r * 64 + ((fg ^ swz_row(r)) << 4);
    };
    auto off_t = [&](int base, int pitch, auto chunk) {
        const int g = lane >> 4, x = lane & 15;
        const int kr = 8 * (g >> 1) + (x >> 2), cl = base + 16 * (g & 1) + 4 * (x & 3);
        return kr * pitch + chunk(kr, cl >> 3) + (cl & 7) * 2;
    };
    auto chunk_a = [&](int k, int c) { return (c ^ swz_tr(k)) << 4; };
    int aoff[MI], boff[NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
        aoff[i] = kTA ? off_t(wr * 32 * MI + i * 32, 2 * BM, chunk_a) : off_n(wr * 32 * MI + i * 32);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        boff[j] = kInt ? off_n(wc * 32 * NJ + j * 32) : off_t(wc * 32 * NJ + j * 32, 2 * BN, chunk_b);
    auto read_frag = [&](const char* sp, int off, int ks, int tr_pitch) __attribute__((always_inline)) {
        if (tr_pitch) {
            const u32x2 v0 = ds_read_tr(sp + off + ks * 16 * tr_pitch);
            const u32x2 v1 = ds_read_tr(sp + off + ks * 16 * tr_pitch + 4 * tr_pitch);
            return u32x4{v0.x, v0.y, v1.x, v1.y};
        }
        return *reinterpret_cast<const u32x4*>(sp + (off ^ (ks << 5)));
    };
    auto read_frags = [&](const Slot& sp, int ks, u32x4 (&af)[MI], u32x4 (&bf)[NJ]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (MI > NJ ? MI : NJ); ++i) {
            if (i < MI)
                af[i] = read_frag(sp.a, aoff[i], ks, kTA ? 2 * BM : 0);
            if (i < NJ)
                bf[i] = read_frag(sp.b, boff[i], ks, kWiden ? 2 * BN : 0);
        }
    };
    Acc acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            acc[i][j] = Acc{};
    auto multiply = [&](const u32x4 (&af)[MI], const u32x4 (&bf)[NJ]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if constexpr (kInt)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                        __builtin_bit_cast(i32x4, af[i]), __builtin_bit_cast(i32x4, bf[j]), acc[i][j], 0, 0, 0);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, af[i]), __builtin_bit_cast(bf16x8, bf[j]), acc[i][j], 0, 0, 0);
            }
    };
    // The order within half a step: the reads of the next k-step, the loads
    // and the widening spread between the MFMAs. (Smaller tiles run two or
    // three workgroups a compute unit, which fill each other's gaps.)
    auto interleave = []() __attribute__((always_inline)) {
        if constexpr (MI * NJ >= 8) {
            constexpr int reads = (kTA ? 2 : 1) * MI + (kWiden ? 2 : 1) * NJ;
            constexpr int nmf = MI * NJ, per = (reads + nmf - 1) / nmf;
#pragma unroll
            for (int q = 0; q < nmf; ++q) {
                if (q % (nmf / 4) == 0)
                    __builtin_amdgcn_sched_group_barrier(0x010, kWiden ? 2 : 1, 0);
                if (q < reads)
                    __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
                if (kWiden)
                    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                if (kWiden && (q == nmf / 2 || q == nmf - 1))
                    __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
        }
    };
    // k past the end in the slot that holds it: 0 in A (its B is 0 or finite)
    const int tail = K % kSlot;   // k values in it, when not whole
    const int tail_slot = !kTA && tail ? ns - 1 : -1;
    auto clear_tail = [&](const Slot& sp) __attribute__((always_inline)) {
        // thread t clears row t
        const int r = tid, b0 = tail * kEltA;
        if (r < BM) {
#pragma unroll 1
            for (int c = b0 >> 4; c < 4; ++c) {
                u32x4* p = reinterpret_cast<u32x4*>(sp.a + r * 64 + ((c ^ swz_row(r)) << 4));
                u32x4 v = *p;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int over = b0 - (16 * c + 4 * e);   // bytes of this word to keep
                    v[e] = over >= 4 ? v[e] : over <= 0 ? 0u : v[e] & (0xFFFFFFFFu >> (32 - 8 * over));
                }
                *p = v;
            }
        }
        __syncthreads();
    };

    if constexpr (kInt) {
        for (int e = tid; e < BM + BN; e += kThreads)
            lscale[e] = e < BM ? (e < rows ? gbl(it.sa)[m0 + e] : 0.f)
                               : (e - BM < cols ? gbl(it.sb)[n0 + e - BM] : 0.f);
    }

    // The output. Register r of lane l, block (i, j): row 32 i + 8 (r >> 2) +
    // 4 (l >> 5) + (r & 3), column NJ (l & 31) + j of the wavefront's part. It is
    // addressed through a buffer resource: rows past the end fall behind it,
    // and lanes with columns past the end get an offset behind it. Where the
    // alignment and n allow (`fits`), a lane's NJ columns go as one.
    using T = typename Elt<DT>::type;
    constexpr int kElt = sizeof(T);
    constexpr int kBehind = (int)0x80000000;
    constexpr bool kBeta = OP == kQ8GradWeight;
    constexpr bool kSplit = MI * NJ < 8;   // (large tiles are not split)
    const int row0 = wr * 32 * MI + 4 * fg, col0 = wc * kCols + NJ * fr;
    const bool fits = it.n % NJ == 0 && it.ldo % NJ == 0 &&
                      reinterpret_cast<uintptr_t>(it.out) % (NJ * kElt) == 0;
    const int ldo = it.ldo * kElt;
    const __amdgpu_buffer_rsrc_t ro =
        buffer(static_cast<const T*>(it.out) + (int64_t)m0 * it.ldo + n0, (rows - 1) * ldo + cols * kElt);
    const int place = col0 < cols ? row0 * ldo + col0 * kElt : kBehind;
    // beta G: groups of four rows (r >> 2), the first from before the products
    // on, so that reading G is not waited for group by group. As many of them
    // as 16 registers hold (24 in small bf16 tiles): in the small tiles a value
    // too many is spilled, and the spill waits for it before the first product (16
    // experts of 2048 x 6144: 398 us with 32 registers, 309 with 24 in the same
    // code). The large bf16 tiles spill some of their 16 all the same; with 8
    // they take as long (8192 x 6144, 4096 tokens: 362 and 369 us).
    constexpr int kWords = NJ * kElt / 4;   // of a lane's columns
    constexpr int kGroups = 4 * MI, kAhead = MI * NJ >= 8 ? 4 / kWords : kWords == 1 ? 6 : 2;
    uint32_t g[kBeta ? kAhead : 1][4][kWords];
    auto ahead = [&](int b) __attribute__((always_inline)) {
        if constexpr (kBeta) {
            if (beta != 0.f && fits) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    load_words(g[b % kAhead][e], ro, place + (8 * b + e) * ldo);
            }
        }
    };
    auto first_ahead = [&]() __attribute__((always_inline)) {
        if (!kSplit || it.nsplit == 1)
#pragma unroll
            for (int b = 0; b < kAhead; ++b)
                ahead(b);
    };
    // (the further passes take registers of their own: behind them then)
    if constexpr (P == 1)
        first_ahead();

    // The pipeline. Step s multiplies slot s; it refills the ring position of
    // slot s - 1 (free since the barrier in step s - 1) with slot s + kDeep. Its
    // wait leaves in flight what was issued after slot s + 1 (with a ring of
    // four the loads of step s - 1 and of this step's first half, with one of
    // three the latter); the barrier then makes slot s + 1 whole for everyone.
    // The widened operand is written kDeep slots ahead, from registers loaded
    // kRaw steps before that.
    constexpr int kDeep = RING - 1, kRaw = RING == 4 ? 2 : 3;
    constexpr int kStepLoads = MI + (kInt ? NJ : kLoads + 1);
    constexpr int kHalfLoads = (MI + 1) / 2 + (kInt ? (NJ + 1) / 2 : kLoads + 1);
    // In small tiles of matmul, whose operands all arrive by DMA, the first half
    // of a slot's loads goes half a step earlier, behind the barrier of step s
    // into slot s itself, which everyone has read by then, and the second half
    // at the start of the next step: cold operands, 2048 x 2048 of k = 6144, 43 to
    // 41 us, the 16 experts below 87 to 85 us. (All of the slot that early: 44 and
    // 80 us, but 5 to 11% slower than this for short sums.)
    constexpr bool kEarly = kInt && MI * NJ < 8;
    constexpr int kInFlight = kEarly        ? (kDeep - 1) * kStepLoads
                              : RING == 4 ? kStepLoads + kHalfLoads
                                          : kHalfLoads;
    constexpr int kFirst = kEarly ? (kDeep - 1) * kStepLoads + kHalfLoads : kInt ? MI + NJ : MI;
    u32x4 fa[MI], fb[NJ], ga[MI], gb[NJ];
    Raw w0{}, w1{}, w2{};
    // A step after the loop, whose loads to registers nobody uses, makes none:
    // the compiler would drop them, and a wait that counts them would leave as
    // many older loads in flight.
    auto step = [&](auto rest, auto after, const Slot& cur, const Slot& refill, const Slot& next, int s, Raw& w)
        __attribute__((always_inline)) {
        constexpr bool kAfter = decltype(after)::value;
        constexpr int kLeft = kAfter ? kInFlight - (kWiden ? kLoads + 1 : 0) : kInFlight;
        Raw fresh{};
        // (loads in this order, which the wait below counts: the previous
        // step's second half, this step's first, those to registers)
        asm volatile("" ::: "memory");
        issue(refill, s + kDeep, kEarly);
        if constexpr (kWiden && !kAfter)
            fresh = fetch(s + kDeep + kRaw);
        read_frags(cur, 1, ga, gb);
        if constexpr (kWiden)
            widen(rest, refill, w, 0);
        multiply(fa, fb);
        interleave();
        // (small tiles: keeps the widening of the next slot's values, and the
        // wait for them, behind this one's)
        if constexpr (MI * NJ < 8)
            __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
        if constexpr (!kTA)
            if (s + 1 == tail_slot)
                clear_tail(next);
        if constexpr (kEarly)
            issue(cur, s + RING, false);
        else
            issue(refill, s + kDeep, true);
        read_frags(next, 0, fa, fb);
        if constexpr (kWiden)
            widen(rest, refill, w, 1);
        multiply(ga, gb);
        interleave();
        if constexpr (MI * NJ < 8)
            __builtin_amdgcn_sched_barrier(0);
        w = fresh;
    };
    // slots s0 .. s0 + kDeep - 1 whole, the next kRaw of the widened operand in
    // registers; the last slot's loads go last, so that the first wait leaves
    // them alone in flight
    auto whole = [&](const Slot& sp, int s) __attribute__((always_inline)) {
        issue(sp, s, false);
        issue(sp, s, true);
    };
    // One pass over this workgroup's slots, `rest` with the 8-bit operand's
    // further parts.
    auto pass = [&](auto rest) __attribute__((always_inline)) {
        if constexpr (kWiden) {
            const Raw p0 = fetch(s0), p1 = fetch(s0 + 1), p2 = kDeep == 3 ? fetch(s0 + 2) : Raw{};
            w0 = fetch(s0 + kDeep);
            w1 = fetch(s0 + kDeep + 1);
            if constexpr (kRaw == 3)
                w2 = fetch(s0 + kDeep + 2);
            whole(sl0, s0);
            if constexpr (kDeep == 3)
                whole(sl1, s0 + 1);
            widen(rest, sl0, p0, 0);
            widen(rest, sl0, p0, 1);
            widen(rest, sl1, p1, 0);
            widen(rest, sl1, p1, 1);
            if constexpr (kDeep == 3) {
                widen(rest, sl2, p2, 0);
                widen(rest, sl2, p2, 1);
            }
        } else {
            whole(sl0, s0);
            if constexpr (kDeep == 3)
                whole(sl1, s0 + 1);
        }
        asm volatile("" ::: "memory");
        whole(kDeep == 3 ? sl2 : sl1, s0 + kDeep - 1);
        if constexpr (kEarly)
            issue(kDeep == 3 ? sl3 : sl2, s0 + kDeep, false);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(kFirst) : "memory");
        if (s0 == tail_slot)
            clear_tail(sl0);
        read_frags(sl0, 0, fa, fb);
        const std::false_type in{};
        if constexpr (RING == 4) {
            for (int s = s0; s < s1; s += 4) {
                step(rest, in, sl0, sl3, sl1, s, w0);
                step(rest, in, sl1, sl0, sl2, s + 1, w1);
                step(rest, in, sl2, sl1, sl3, s + 2, w0);
                step(rest, in, sl3, sl2, sl0, s + 3, w1);
            }
        } else {
            const std::true_type after{};
            int s = s0;
            for (; s + 3 <= s1; s += 3) {
                step(rest, in, sl0, sl2, sl1, s, w0);
                step(rest, in, sl1, sl0, sl2, s + 1, w1);
                step(rest, in, sl2, sl1, sl0, s + 2, w2);
            }
            if (s < s1)
                step(rest, after, sl0, sl2, sl1, s, w0);
            if (s + 1 < s1)
                step(rest, after, sl1, sl0, sl2, s + 1, w1);
        }
        // (loads of slots past the end are still to land in LDS: they are not to
        // meet the next pass, or outlive the workgroup)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    };
    pass(std::false_type{});
    if constexpr (P > 1) {
#pragma unroll 1
        for (part = 1; part < P; ++part) {
            __syncthreads();   // everyone is done with the slots
            pass(std::true_type{});
        }
        first_ahead();
    }

    if constexpr (kSplit) {
        if (it.nsplit > 1) {
            // a piece of the sums, as it is
            const int ldp = it.n * 4;
            const __amdgpu_buffer_rsrc_t rp =
                buffer(it.part + ((int64_t)piece * it.m + m0) * it.n + n0, (rows - 1) * ldp + cols * 4);
#pragma unroll
            for (int b = 0; b < kGroups; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t v[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const AccT a = acc[b >> 2][j][4 * (b & 3) + e];
                        v[j] = __builtin_bit_cast(uint32_t, a);
                    }
                    const int at = (row0 + 8 * b + e) * ldp + col0 * 4;
                    if (it.n % NJ == 0) {
                        store_words(v, rp, col0 < cols ? at : kBehind);
                    } else {
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            __builtin_amdgcn_raw_buffer_store_b32(v[j], rp, col0 + j < cols ? at + 4 * j : kBehind,
                                                                  0, 0);
                    }
                }
            return;
        }
    }
    float colscale[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        colscale[j] = kInt ? lscale[BM + col0 + j] : 1.f;
    // row b, e of the lane's: its NJ sums, scaled
    auto values = [&](int b, int e, const f32x4& rowscale, float (&v)[NJ]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const AccT a = acc[b >> 2][j][4 * (b & 3) + e];
            if constexpr (kInt)
                v[j] = scaled(a, token_scale(rowscale[e]), colscale[j]);
            else
                v[j] = a;
        }
    };
    if (fits) {
#pragma unroll
        for (int b = 0; b < kGroups; ++b) {
            f32x4 rowscale{};
            if constexpr (kInt)
                rowscale = *reinterpret_cast<const f32x4*>(&lscale[row0 + 8 * b]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[NJ];
                values(b, e, rowscale, v);
                if (kBeta && beta != 0.f) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const uint32_t w = g[b % kAhead][e][DT == 0 ? j >> 1 : j];
                        const uint32_t f = DT == 1 ? w : j & 1 ? w & 0xFFFF0000u : w << 16;
                        v[j] = fmaf(beta, __uint_as_float(f), v[j]);
                    }
                }
                uint32_t w[kWords];
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    w[j] = DT == 1 ? __float_as_uint(v[j])
                                   : __builtin_bit_cast(uint32_t, bf16x2{(bf16)v[(2 * j) % NJ],
                                                                         (bf16)v[(2 * j + 1) % NJ]});
                }
                store_words(w, ro, place + (8 * b + e) * ldo);
            }
            if (b + kAhead < kGroups)
                ahead(b + kAhead);
            __builtin_amdgcn_sched_barrier(0);   // (a group's registers at a time)
        }
        return;
    }
#pragma unroll
    for (int b = 0; b < kGroups; ++b) {
        f32x4 rowscale{};
        if constexpr (kInt)
            rowscale = *reinterpret_cast<const f32x4*>(&lscale[row0 + 8 * b]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v[NJ];
            values(b, e, rowscale, v);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int at = col0 + j < cols ? place + (8 * b + e) * ldo + kElt * j : kBehind;
                if constexpr (DT == 0) {
                    if (kBeta && beta != 0.f)
                        v[j] = fmaf(
                            beta,
                            __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ro, at, 0, 0) << 16), v[j]);
                    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)v[j]), ro, at, 0, 0);
                } else {
                    if (kBeta && beta != 0.f)
                        v[j] = fmaf(beta, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ro, at, 0, 0)), v[j]);
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), ro, at, 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#endif
}

// A tile in one part where the scales of its part of k, slots [s0, s1), are all
// powers of two, else in as many as its output's type asks for.
template <int OP, int DT, int MI, int NJ, int RING>
__device__ __forceinline__ void q8_tile_in_parts(const Q8Item& it, int m0, int n0, int s0, int s1, int piece,
                                                 float beta, const Slot sl0, const Slot sl1, const Slot sl2,
                                                 const Slot sl3, float* lscale)
{
    constexpr int kParts = parts<OP, DT>();
    if constexpr (kParts > 1) {
        const int first = s0 * slot_k<OP>(), n = min(it.k, s1 * slot_k<OP>()) - first, wave = threadIdx.x >> 6;
        const float* sb = it.sb + first;
        u32x4 bits = {0u, 0u, 0u, 0u};
        if (n >= 4) {   // four a load, the last of them perhaps again
#pragma unroll 4
            for (int k = 4 * threadIdx.x; k < n; k += 4 * kThreads)
                bits |= load16_any(sb + min(k, n - 4));
        } else if ((int)threadIdx.x < n) {
            bits.x = __float_as_uint(gbl(sb)[threadIdx.x]);
        }
        const bool any = __ballot(((bits.x | bits.y | bits.z | bits.w) & 0x007FFFFFu) != 0) != 0;
        if ((threadIdx.x & 63) == 0)
            lscale[wave] = any ? 1.f : 0.f;
        __syncthreads();
        if (lscale[0] + lscale[1] + lscale[2] + lscale[3] > 0.f) {
            q8_tile<OP, DT, MI, NJ, RING, kParts>(it, m0, n0, s0, s1, piece, beta, sl0, sl1, sl2, sl3, lscale);
            return;
        }
    }
    q8_tile<OP, DT, MI, NJ, RING, 1>(it, m0, n0, s0, s1, piece, beta, sl0, sl1, sl2, sl3, lscale);
}

// Tiles of 256 x 256, one workgroup a compute unit: 128 x 128 outputs a
// wavefront, in the 256 AGPRs of each lane. Per slot a wavefront issues 32
// MFMAs (about 1024 cycles) and reads 16 KB of fragments; the compute unit's
// LDS moves 64 KB of reads and 32 KB of writes in that time, three quarters of
// what it can, so the tile cannot be smaller and the matrix units still be fed.
// 4096 tokens, 8192 x 6144, scales of dX and dW powers of two: Y 181 to 191 us
// (2.2 to 2.3 POP/s; 63% of the matrix units' cycles), dX 361 to 375 us (1.10 to
// 1.14 PFLOP/s), fp32 G + dW 366 to 375 us (1.10 to 1.13 PFLOP/s; 56%). Other
// scales: dX 747 to 773 us. The chip's clock under this load bounds them:
// a library's product of 8192 x 8192 x 8192 reaches 2.08 POP/s and 1.22 PFLOP/s.
//
// When the last round of tiles would keep at most half of the compute units
// busy, its tiles run as two halves of 256 x 128 each (workgroups from nwhole
// on, two for each tile from there).
template <int OP, int DT>
__global__ __launch_bounds__(kThreads, 1) void k_q8_big(const Q8Batch batch, int nwg, int nwhole)
{
    constexpr bool kInt = OP == kQ8Matmul;
    constexpr int kOp = 16384;   // one operand of a slot: 256 rows of 64 bytes
    constexpr int kObjA = kInt ? 2 * kOp : kOp, kObjB = kInt ? 16 : kOp;
    __shared__ __attribute__((aligned(1024))) char sa0[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa1[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa2[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa3[kObjA];
    __shared__ __attribute__((aligned(1024))) char sb0[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb1[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb2[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb3[kObjB];
    __shared__ __attribute__((aligned(16))) float lscale[kInt ? 512 : 4];
    const Slot sl0 = {sa0, kInt ? sa0 + kOp : sb0}, sl1 = {sa1, kInt ? sa1 + kOp : sb1};
    const Slot sl2 = {sa2, kInt ? sa2 + kOp : sb2}, sl3 = {sa3, kInt ? sa3 + kOp : sb3};

    const bool half = (int)blockIdx.x >= nwhole;
    // whole tiles first, over the XCDs; then the halves, likewise
    const int h = half ? by_xcd(blockIdx.x - nwhole, nwg - nwhole) : 0;
    // (each item's over the XCDs where their sums differ in length, as below)
    constexpr bool kEach = OP == kQ8GradWeight;
    const int t = half ? nwhole + (h >> 1) : kEach ? (int)blockIdx.x : by_xcd(blockIdx.x, nwhole);
    const Q8Item it = batch.it[find_item(batch, t)];
    const int ntm = (it.m + kQ8Big - 1) / kQ8Big, ns = (it.k + slot_k<OP>() - 1) / slot_k<OP>();
    const int own = t - it.begin;
    int bm, bn;
    tile_at(kEach && !half ? by_xcd(own, min(ntm * it.ntn, nwhole - it.begin)) : own, ntm, it.ntn, &bm, &bn);
    const int m0 = bm * kQ8Big, n0 = bn * kQ8Big + (half ? 128 * (h & 1) : 0);
    if (!half)
        q8_tile_in_parts<OP, DT, 4, 4, 4>(it, m0, n0, 0, ns, 0, batch.beta, sl0, sl1, sl2, sl3, lscale);
    else if (n0 < it.n)
        q8_tile_in_parts<OP, DT, 4, 2, 4>(it, m0, n0, 0, ns, 0, batch.beta, sl0, sl1, sl2, sl3, lscale);
}

// Tiles of 128 x 128 over a ring of three slots, three workgroups a compute
// unit: for outputs too small for the large tiles, and sums so short that a
// tile's loads and stores have to overlap another's products. What bounds them is
// the latency of the slots' loads, which two slots ahead of three workgroups do
// not quite hide. matmul with no more than two tiles a compute unit has a ring of
// four instead (gradients gain nothing from it, their matrix instructions taking
// twice the time a slot): 2048 x 2048 of k = 6144 from 37 to 33 us, 16 experts of
// 2048 x 6144, 3001 tokens and cold weights, from 94 to 87 us (now 85, 2.6 TB/s).
// Gradients, 8 experts of 512 x 10240, 1999 tokens: dX 35 us, 66 in two parts; 16
// of 2048 x 6144, 3001 tokens, beta G + dW in bf16: 207 us, 4.0 TB/s, of which
// reading and writing G without products takes 150, and 304 us in two parts.
template <int OP, int DT, int N, int RING>
__global__ __launch_bounds__(kThreads, RING == 3 ? 3 : 2) void k_q8_mid(const Q8BatchOf<N> batch, int nwg)
{
    constexpr bool kInt = OP == kQ8Matmul;
    constexpr int kOp = 8192;
    constexpr int kObjA = kInt ? 2 * kOp : kOp, kObjB = kInt ? 16 : kOp;
    __shared__ __attribute__((aligned(1024))) char sa0[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa1[kObjA];
    __shared__ __attribute__((aligned(1024))) char sa2[kObjA];
    __shared__ __attribute__((aligned(1024))) char sb0[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb1[kObjB];
    __shared__ __attribute__((aligned(1024))) char sb2[kObjB];
    __shared__ __attribute__((aligned(1024))) char sa3[RING == 3 ? 16 : kObjA];
    __shared__ __attribute__((aligned(1024))) char sb3[RING == 3 ? 16 : kObjB];
    __shared__ __attribute__((aligned(16))) float lscale[kInt ? 256 : 4];
    const Slot sl0 = {sa0, kInt ? sa0 + kOp : sb0}, sl1 = {sa1, kInt ? sa1 + kOp : sb1};
    const Slot sl2 = {sa2, kInt ? sa2 + kOp : sb2}, sl3 = {sa3, kInt ? sa3 + kOp : sb3};

    // Sums over tokens differ in length from item to item, so each item's tiles
    // are spread over the XCDs; else the launch's are.
    const int wg = OP == kQ8GradWeight ? (int)blockIdx.x : by_xcd(blockIdx.x, nwg);
    const Q8Item it = batch.it[find_item(batch, wg)];
    const int ntm = (it.m + kQ8Mid - 1) / kQ8Mid, ns = (it.k + slot_k<OP>() - 1) / slot_k<OP>();
    // the tiles of one piece of k, then those of the next
    const int tiles = ntm * it.ntn;
    const int b = OP == kQ8GradWeight ? by_xcd(wg - it.begin, tiles * it.nsplit) : wg - it.begin;
    const int piece = b / tiles;
    int bm, bn;
    tile_at(b - piece * tiles, ntm, it.ntn, &bm, &bn);
    const int s0 = piece * it.per;
    q8_tile_in_parts<OP, DT, 2, 2, RING>(it, bm * kQ8Mid, bn * kQ8Mid, s0, min(ns, s0 + it.per), piece, batch.beta,
                                         sl0, sl1, sl2, RING == 3 ? sl2 : sl3, lscale);
}

// grad_weight of few rows (m <= 64, an attention gate's): a stream over the
// tokens, which memory latency bounds. Tiles of 64 x 128, a 32 x 64 part a
// wavefront; both operands pass through registers, kDeep slots of 32 tokens
// ahead, 36 bytes a thread and slot, into two LDS slots in turn. dY at any
// alignment: at pitches of 16 bytes and more, 16 bytes that start in a row of any
// slot but the last end within the operand's next row, and what they hold past
// their row only reaches outputs that are not written; the last slot is loaded
// value by value. All parts of the 8-bit operand lie side by side in LDS; the
// further ones are made and multiplied in slots with a scale that is no power of
// two. Three 18 x 2304 outputs over 16384 tokens: 29 us a call, 1.3 TB/s, 4 us of
// it for their sums; where all scales are powers of two, 2.5 vector operations a
// value instead of 8, 24.
template <int DT, int N>
__global__ __launch_bounds__(kThreads, DT == 0 ? 3 : 2) void k_q8_thin(const Q8BatchOf<N> batch)
{
#ifdef __HIP_DEVICE_COMPILE__
    using T = typename Elt<DT>::type;
    constexpr int kDeep = 6, kSlot = 32, kPitchA = 128, kPitchB = 256;
    constexpr int kParts = parts<kQ8GradWeight, DT>();
    __shared__ __attribute__((aligned(1024))) char la[2][kSlot * kPitchA];
    __shared__ __attribute__((aligned(1024))) char lb[2][kParts][kSlot * kPitchB];
    const Q8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int b = blockIdx.x - it.begin, piece = b / it.ntn;
    const int n0 = (b - piece * it.ntn) * 128;
    const int last = (it.k + kSlot - 1) / kSlot - 1;   // the last slot
    const int s0 = piece * it.per, s1 = min(last, s0 + it.per);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wr = wave >> 1, wc = wave & 1, fr = lane & 31, fg = lane >> 5;
    const int krow = tid >> 3, t8 = tid & 7;

    const char* A = static_cast<const char*>(it.a);
    const char* B = reinterpret_cast<const char*>(it.b) + n0;
    const int lda = 2 * it.lda, ldb = it.ldb, cols = min(128, it.n - n0);
    // columns past the end: the first ones again
    const int va = krow * lda + (8 * t8 < it.m ? 16 * t8 : 0), vb = krow * ldb + (16 * t8 < cols ? 16 * t8 : 0);
    struct Raw { u32x4 a, b; float s; uint32_t all; };   // all: the slot's scales, one a lane
    auto fetch = [&](int s) __attribute__((always_inline)) {
        // (a slot that is not this piece's loads nothing: its resources are empty)
        const bool in = s < s1;
        const __amdgpu_buffer_rsrc_t ra = buffer(A + (int64_t)s * kSlot * lda, in ? kSlot * lda + 16 : 0);
        const __amdgpu_buffer_rsrc_t rb = buffer(B + (int64_t)s * kSlot * ldb, in ? kSlot * ldb + 16 : 0);
        const __amdgpu_buffer_rsrc_t rs = buffer(it.sb + (int64_t)s * kSlot, in ? kSlot * 4 : 0);
        Raw w;
        w.a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, va, 0, 0));
        w.b = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, vb, 0, 0));
        w.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * krow, 0, 0));
        w.all = __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * (lane & 31), 0, 0);
        return w;
    };
    // Whether a slot's further parts are multiplied (the same in every wavefront).
    auto more = [](const Raw& w) __attribute__((always_inline)) {
        return __ballot((w.all & 0x007FFFFFu) != 0) != 0;
    };
    // B's columns lie as in the tiles above: block j of a wavefront's 64 takes
    // every other one from j on. A's rows of 128 bytes alternate between the
    // halves of the banks; the swizzle does the rest.
    auto swz_a = [](int k) { return (k & 2) << 1; };
    auto stash = [&](int buf, const Raw& w) __attribute__((always_inline)) {
        const bool rest = more(w);
        *reinterpret_cast<u32x4*>(la[buf] + krow * kPitchA + ((t8 ^ swz_a(krow)) << 4)) = w.a;
        auto word = [&](int e) { return w.b[e >> 1]; };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            auto byte = [&](int e) { return j + 2 * (e & 1); };
            const int at = krow * kPitchB + ((((t8 >> 2) * 8 + 4 * j + (t8 & 3)) ^ swz_tr(krow)) << 4);
            *reinterpret_cast<u32x4*>(lb[buf][0] + at) = widen8(word, byte, w.s);
            if (rest) {
#pragma unroll
                for (int p = 1; p < kParts; ++p)
                    *reinterpret_cast<u32x4*>(lb[buf][p] + at) = widen8_rest<kParts>(word, byte, w.s, p);
            }
        }
        return rest;
    };
    auto frag = [&](const char* base, int pitch, int col, bool narrow, int ks) __attribute__((always_inline)) {
        const int g = lane >> 4, x = lane & 15;
        const int kr = 16 * ks + 8 * (g >> 1) + (x >> 2), cl = col + 16 * (g & 1) + 4 * (x & 3);
        const char* p = base + kr * pitch + (((cl >> 3) ^ (narrow ? swz_a(kr) : swz_tr(kr))) << 4) + (cl & 7) * 2;
        const u32x2 v0 = ds_read_tr(p), v1 = ds_read_tr(p + 4 * pitch);
        return __builtin_bit_cast(bf16x8, u32x4{v0.x, v0.y, v1.x, v1.y});
    };
    f32x16 acc[2] = {};
    auto multiply = [&](int buf, bool rest) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        auto add = [&](int part) __attribute__((always_inline)) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 a = frag(la[buf], kPitchA, 32 * wr, true, ks);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        a, frag(lb[buf][part], kPitchB, 64 * wc + 32 * j, false, ks), acc[j], 0, 0, 0);
            }
        };
        add(0);
        if (rest) {
#pragma unroll
            for (int p = 1; p < kParts; ++p)
                add(p);
        }
    };
    Raw w[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
        w[d] = fetch(s0 + d);
        asm volatile("" ::: "memory");   // (in this order, as they are waited for)
    }
    // (a slot past the end is all zeros, in both operands)
    for (int s = s0; s < s1; s += kDeep)
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const bool rest = stash(d & 1, w[d]);
            w[d] = fetch(s + d + kDeep);
            multiply(d & 1, rest);
        }
    if (s0 <= last && last < s0 + it.per) {
        const int k = last * kSlot + krow;
        union { bf16 t[8]; u32x4 v; } a;
        union { int8_t t[16]; u32x4 v; } q;
        a.v = q.v = u32x4{0u, 0u, 0u, 0u};
        float scale = 0.f;
        uint32_t all = 0;
        if (last * kSlot + (lane & 31) < it.k)
            all = __float_as_uint(gbl(it.sb)[last * kSlot + (lane & 31)]);
        if (k < it.k) {
            const NS_GLOBAL bf16* pa = gbl(static_cast<const bf16*>(it.a)) + (int64_t)k * it.lda;
            const NS_GLOBAL int8_t* pb = gbl(it.b) + (int64_t)k * it.ldb + n0;
            for (int e = 0; e < 8; ++e)
                if (8 * t8 + e < it.m)
                    a.t[e] = pa[8 * t8 + e];
            for (int e = 0; e < 16; ++e)
                if (16 * t8 + e < cols)
                    q.t[e] = pb[16 * t8 + e];
            scale = gbl(it.sb)[k];
        }
        const bool rest = stash(0, Raw{a.v, q.v, scale, all});
        multiply(0, rest);
    }

    // register r of lane l, block j: row 8 (r >> 2) + 4 (l >> 5) + (r & 3),
    // column 2 (l & 31) + j
    const int c0 = n0 + 64 * wc + 2 * fr;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = 32 * wr + 8 * (r >> 2) + 4 * fg + (r & 3);
        if (row >= it.m)
            continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (c0 + j >= it.n)
                continue;
            if (it.nsplit > 1) {
                gbl(it.part)[((int64_t)piece * it.m + row) * it.n + c0 + j] = acc[j][r];
            } else {
                NS_GLOBAL T* p = gbl(static_cast<T*>(it.out)) + (int64_t)row * it.ldo + c0 + j;
                *p = from_f32<T>(batch.beta != 0.f ? fmaf(batch.beta, to_f32(*p), acc[j][r]) : acc[j][r]);
            }
        }
    }
#endif
}

// Few tokens (T <= 32): Y = Xq Wq^T as a stream over the weights, which memory
// bounds. A workgroup of eight wavefronts takes 16 R channels of Wq and all T
// tokens; its wavefronts take k in turns of 64 bytes a row, each with its
// weights straight from memory into the MFMAs (16 x 16 x 64: lane l holds
// channel or token l & 15, bytes 16 (l >> 4) + 0 .. 15 of the step), eight
// steps in flight, and their integer sums meet in LDS. Channels and tokens past
// the end repeat the last one and are not written. Any pitch and alignment.
// 8192 x 6144: 10 us with one token (5.0 TB/s, the rate of a large copy), 14 with
// 32, where the tiles take 16 with 33.
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;

// 16 bytes of a row from byte c on, 0 past `len`.
__device__ __forceinline__ u32x4 tail16(const int8_t* row, int c, int len)
{
    if (c + 16 <= len)
        return load16_any(row + c);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (c + e < len)
            v[e >> 2] |= (uint32_t)(uint8_t)gbl(row)[c + e] << (8 * (e & 3));
    return v;
}

template <int DT, int R, int NT>
__device__ __forceinline__ void few_tokens(const Q8Item& it, int o0, int* red)
{
    using T = typename Elt<DT>::type;
    constexpr int O = 16 * R, N = 16 * NT;   // channels, tokens of the workgroup
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int fr = lane & 15, fg = lane >> 4;
    const int8_t* x[NT];
    const int8_t* w[R];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        x[j] = static_cast<const int8_t*>(it.a) + (int64_t)min(16 * j + fr, it.m - 1) * it.lda;
#pragma unroll
    for (int i = 0; i < R; ++i)
        w[i] = it.b + (int64_t)min(o0 + 16 * i + fr, it.n - 1) * it.ldb;
    i32x4 acc[R][NT];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    auto mac = [&](const u32x4 (&wv)[R], const u32x4 (&xv)[NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[i]),
                                                                  __builtin_bit_cast(i32x4, xv[j]), acc[i][j], 0, 0, 0);
    };
    constexpr int kDeep = 8 / R;   // steps in flight
    const int full = it.k >> 6;    // whole steps of 64
    int s = wave;
    for (; s + (kDeep - 1) * kFewWaves < full; s += kDeep * kFewWaves) {
        u32x4 wv[kDeep][R], xv[kDeep][NT];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int c = 64 * (s + d * kFewWaves) + 16 * fg;
#pragma unroll
            for (int i = 0; i < R; ++i)
                wv[d][i] = load16_any(w[i] + c);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                xv[d][j] = load16_any(x[j] + c);
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
            mac(wv[d], xv[d]);
    }
    for (; 64 * s < it.k; s += kFewWaves) {
        const int c = 64 * s + 16 * fg;
        u32x4 wv[R], xv[NT];
#pragma unroll
        for (int i = 0; i < R; ++i)
            wv[i] = tail16(w[i], c, it.k);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            xv[j] = tail16(x[j], c, it.k);
        mac(wv, xv);
    }
    // register r of lane l: channel 4 (l >> 4) + r, token l & 15
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<i32x4*>(red + (wave * N + 16 * j + fr) * O + 16 * i + 4 * fg) = acc[i][j];
    __syncthreads();
    for (int e = tid; e < N * O; e += kFewThreads) {
        const int t = e / O, o = o0 + e % O;
        if (t < it.m && o < it.n) {
            int sum = red[e];
#pragma unroll
            for (int v = 1; v < kFewWaves; ++v)
                sum += red[v * N * O + e];
            const float y = scaled(sum, token_scale(gbl(it.sa)[t]), gbl(it.sb)[o]);
            gbl(static_cast<T*>(it.out))[(int64_t)t * it.ldo + o] = from_f32<T>(y);
        }
    }
}

// Channels a workgroup takes: more with more tokens, so that Xq is read less.
template <int DT, int N>
__global__ __launch_bounds__(kFewThreads) void k_q8_few(const Q8BatchOf<N> batch)
{
    __shared__ __attribute__((aligned(16))) int red[kFewWaves * 2 * 16 * 32];
    const Q8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int o0 = (blockIdx.x - it.begin) * q8_few_channels(it.m);
    if (it.m <= 16)
        few_tokens<DT, 1, 1>(it, o0, red);
    else
        few_tokens<DT, 2, 2>(it, o0, red);
}

// C from the pieces of split sums, added in piece order: four elements of a row
// a thread (where n and the alignment allow; else four elements 256 apart),
// eight pieces' loads in flight at once. Latency bounds it: 4 us for 9 pieces of
// three 18 x 2304 sums. Also the sum over nothing (no pieces).
template <int OP, int DT, int N>
__global__ __launch_bounds__(kThreads) void k_q8_join(const Q8BatchOf<N> batch)
{
    using T = typename Elt<DT>::type;
    using AccT = typename std::conditional<OP == kQ8Matmul, int, float>::type;
    typedef AccT Acc4 __attribute__((ext_vector_type(4)));
    typedef T T4 __attribute__((ext_vector_type(4)));
    const Q8Item it = batch.it[find_item(batch, blockIdx.x)];
    const int64_t total = (int64_t)it.m * it.n;
    const int64_t e0 = (int64_t)(blockIdx.x - it.begin) * kQ8JoinElems;
    const NS_GLOBAL AccT* part = gbl(reinterpret_cast<const AccT*>(it.part));
    const float beta = batch.beta;
    auto value = [&](AccT sum, int r, int c, float old) {
        if constexpr (OP == kQ8Matmul)
            return scaled(sum, token_scale(gbl(it.sa)[r]), gbl(it.sb)[c]);
        const float v = sum;
        return OP == kQ8GradWeight && beta != 0.f ? fmaf(beta, old, v) : v;
    };
    if (((it.n | it.ldo) & 3) == 0 && reinterpret_cast<uintptr_t>(it.out) % sizeof(T4) == 0) {
        const int64_t e = e0 + 4 * threadIdx.x;
        if (e >= total)
            return;
        Acc4 sum = {0, 0, 0, 0};
        for (int q0 = 0; q0 < it.nsplit; q0 += 8) {
            Acc4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = q0 + q < it.nsplit ? *(const NS_GLOBAL Acc4*)(part + (q0 + q) * total + e) : Acc4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q0 + q < it.nsplit)
                    sum += v[q];
        }
        const int r = (int)(e / it.n), c = (int)(e - (int64_t)r * it.n);
        NS_GLOBAL T4* p = (NS_GLOBAL T4*)(gbl(static_cast<T*>(it.out)) + (int64_t)r * it.ldo + c);
        const bool read = OP == kQ8GradWeight && beta != 0.f;
        const T4 old = read ? *p : T4{};
        T4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = from_f32<T>(value(sum[i], r, c + i, to_f32(old[i])));
        *p = y;
        return;
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t e = e0 + threadIdx.x + i * kThreads;
        if (e >= total)
            return;
        AccT sum = 0;
        for (int q = 0; q < it.nsplit; ++q)
            sum += part[q * total + e];
        const int r = (int)(e / it.n), c = (int)(e - (int64_t)r * it.n);
        NS_GLOBAL T* p = gbl(static_cast<T*>(it.out)) + (int64_t)r * it.ldo + c;
        const bool read = OP == kQ8GradWeight && beta != 0.f;
        *p = from_f32<T>(value(sum, r, c, read ? to_f32(*p) : 0.f));
    }
}

// Operands at other alignments or pitches, copied once to rows of a multiple
// of 16 bytes for the tiles' loads: 16 bytes a thread. What follows a row's
// last value in its last 16 bytes is not used by anyone. Memory bounds it (3.6 us
// for 16384 x 18 bf16); loading 4 or 8 bytes at a time in the tiles instead
// would cost every slot two to four times the load instructions.
__global__ __launch_bounds__(kThreads) void k_q8_align(const Q8AlignBatch batch)
{
    const Q8AlignItem it = batch.it[find_item(batch, blockIdx.x)];
    const int64_t chunk = (int64_t)(blockIdx.x - it.begin) * kThreads + threadIdx.x;
    const int per = (it.len + 15) >> 4;
    const int64_t row = chunk / per;
    if (row >= it.rows)
        return;
    const int c = (int)(chunk - row * per) * 16;
    const char* src = static_cast<const char*>(it.src) + row * it.pitch + c;
    u32x4 v;
    if (c + 16 <= it.len) {
        v = load16_any(src);
    } else {
        v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (c + e < it.len)
                v[e >> 2] |= (uint32_t)(uint8_t)gbl(src)[e] << (8 * (e & 3));
    }
    *(NS_GLOBAL u32x4*)gbl(static_cast<char*>(it.dst) + row * (16 * (int64_t)per) + c) = v;
}

}  // namespace

namespace {

// The first kQ8FewItems of a batch, for a launch with fewer argument bytes.
Q8BatchOf<kQ8FewItems> head(const Q8Batch& b)
{
    Q8BatchOf<kQ8FewItems> h;
    for (int i = 0; i < kQ8FewItems; ++i)
        h.it[i] = b.it[i];
    h.count = b.count;
    h.beta = b.beta;
    return h;
}

Q8RowsBatchOf<kQ8FewItems> head(const Q8RowsBatch& b)
{
    Q8RowsBatchOf<kQ8FewItems> h;
    for (int i = 0; i < kQ8FewItems; ++i)
        h.it[i] = b.it[i];
    h.count = b.count;
    h.mode = b.mode;
    return h;
}

}  // namespace

// Kernel template K<op, dtype, ...> for run-time op and dtype (grad_input's
// output is always bf16).
#define NS_Q8_LAUNCH(K, ...)                                                                              \
    do {                                                                                                  \
        if (op == kQ8Matmul && dtype == 0)                                                                \
            hipLaunchKernelGGL((K(kQ8Matmul, 0)), dim3(nwg), dim3(kThreads), 0, stream, __VA_ARGS__);     \
        else if (op == kQ8Matmul)                                                                         \
            hipLaunchKernelGGL((K(kQ8Matmul, 1)), dim3(nwg), dim3(kThreads), 0, stream, __VA_ARGS__);     \
        else if (op == kQ8GradInput)                                                                      \
            hipLaunchKernelGGL((K(kQ8GradInput, 0)), dim3(nwg), dim3(kThreads), 0, stream, __VA_ARGS__);  \
        else if (dtype == 0)                                                                              \
            hipLaunchKernelGGL((K(kQ8GradWeight, 0)), dim3(nwg), dim3(kThreads), 0, stream, __VA_ARGS__); \
        else                                                                                              \
            hipLaunchKernelGGL((K(kQ8GradWeight, 1)), dim3(nwg), dim3(kThreads), 0, stream, __VA_ARGS__); \
    } while (0)
#define NS_Q8_BIG(op, dt) k_q8_big<op, dt>
#define NS_Q8_MID(op, dt) k_q8_mid<op, dt, kQ8Items, 3>
#define NS_Q8_MID_FEW(op, dt) k_q8_mid<op, dt, kQ8FewItems, 3>
#define NS_Q8_JOIN(op, dt) k_q8_join<op, dt, kQ8Items>
#define NS_Q8_JOIN_FEW(op, dt) k_q8_join<op, dt, kQ8FewItems>

hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kThreads);
    if (b.count <= kQ8FewItems) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_q8_quantize<0, kQ8FewItems>), grid, block, 0, stream, head(b));
        else
            hipLaunchKernelGGL((k_q8_quantize<1, kQ8FewItems>), grid, block, 0, stream, head(b));
    } else if (dtype == 0) {
        hipLaunchKernelGGL((k_q8_quantize<0, kQ8RowsItems>), grid, block, 0, stream, b);
    } else {
        hipLaunchKernelGGL((k_q8_quantize<1, kQ8RowsItems>), grid, block, 0, stream, b);
    }
    return hipGetLastError();
}

hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kThreads);
    if (b.count <= kQ8FewItems) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_q8_dequantize<0, kQ8FewItems>), grid, block, 0, stream, head(b));
        else
            hipLaunchKernelGGL((k_q8_dequantize<1, kQ8FewItems>), grid, block, 0, stream, head(b));
    } else if (dtype == 0) {
        hipLaunchKernelGGL((k_q8_dequantize<0, kQ8RowsItems>), grid, block, 0, stream, b);
    } else {
        hipLaunchKernelGGL((k_q8_dequantize<1, kQ8RowsItems>), grid, block, 0, stream, b);
    }
    return hipGetLastError();
}

hipError_t launch_q8_big(int op, const Q8Batch& b, int nwg, int nwhole, int dtype, hipStream_t stream)
{
    NS_Q8_LAUNCH(NS_Q8_BIG, b, nwg, nwhole);
    return hipGetLastError();
}

hipError_t launch_q8_mid(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    // Up to two tiles a compute unit, matmul: deeper rings (see the kernel).
    if (op == kQ8Matmul && nwg <= 512) {
        const dim3 grid(nwg), block(kThreads);
        if (b.count <= kQ8FewItems) {
            if (dtype == 0)
                hipLaunchKernelGGL((k_q8_mid<kQ8Matmul, 0, kQ8FewItems, 4>), grid, block, 0, stream, head(b), nwg);
            else
                hipLaunchKernelGGL((k_q8_mid<kQ8Matmul, 1, kQ8FewItems, 4>), grid, block, 0, stream, head(b), nwg);
        } else if (dtype == 0) {
            hipLaunchKernelGGL((k_q8_mid<kQ8Matmul, 0, kQ8Items, 4>), grid, block, 0, stream, b, nwg);
        } else {
            hipLaunchKernelGGL((k_q8_mid<kQ8Matmul, 1, kQ8Items, 4>), grid, block, 0, stream, b, nwg);
        }
    } else if (b.count <= kQ8FewItems) {
        NS_Q8_LAUNCH(NS_Q8_MID_FEW, head(b), nwg);
    } else {
        NS_Q8_LAUNCH(NS_Q8_MID, b, nwg);
    }
    return hipGetLastError();
}

hipError_t launch_q8_thin(const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kThreads);
    if (b.count <= kQ8FewItems) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_q8_thin<0, kQ8FewItems>), grid, block, 0, stream, head(b));
        else
            hipLaunchKernelGGL((k_q8_thin<1, kQ8FewItems>), grid, block, 0, stream, head(b));
    } else if (dtype == 0) {
        hipLaunchKernelGGL((k_q8_thin<0, kQ8Items>), grid, block, 0, stream, b);
    } else {
        hipLaunchKernelGGL((k_q8_thin<1, kQ8Items>), grid, block, 0, stream, b);
    }
    return hipGetLastError();
}

hipError_t launch_q8_few(const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    const dim3 grid(nwg), block(kFewThreads);
    if (b.count <= kQ8FewItems) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_q8_few<0, kQ8FewItems>), grid, block, 0, stream, head(b));
        else
            hipLaunchKernelGGL((k_q8_few<1, kQ8FewItems>), grid, block, 0, stream, head(b));
    } else if (dtype == 0) {
        hipLaunchKernelGGL((k_q8_few<0, kQ8Items>), grid, block, 0, stream, b);
    } else {
        hipLaunchKernelGGL((k_q8_few<1, kQ8Items>), grid, block, 0, stream, b);
    }
    return hipGetLastError();
}

hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream)
{
    if (b.count <= kQ8FewItems)
        NS_Q8_LAUNCH(NS_Q8_JOIN_FEW, head(b));
    else
        NS_Q8_LAUNCH(NS_Q8_JOIN, b);
    return hipGetLastError();
}

hipError_t launch_q8_align(const Q8AlignBatch& b, int nwg, hipStream_t stream)
{
    hipLaunchKernelGGL(k_q8_align, dim3(nwg), dim3(kThreads), 0, stream, b);
    return hipGetLastError();
}

}  // namespace ns

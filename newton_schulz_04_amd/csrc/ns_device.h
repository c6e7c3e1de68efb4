// ns_device.h -- device helpers shared by the kernels of the layers in 8 bits
// (ns_q8.hip, ns_f8.hip) and of the experts' router (ns_route.hip). Everything is
// local to the file that includes it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

#ifdef __HIP_DEVICE_COMPILE__   // (builtins and resources that do not exist on the host)
typedef __attribute__((address_space(3))) void* lds_ptr;
// A buffer resource over bytes [0, bytes) from p, the same for all lanes:
// saying so keeps it in scalar registers wherever its parts were computed.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)a);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(hi << 32 | lo), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
// One, two or four words at byte `at` of a resource.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], __amdgpu_buffer_rsrc_t r, int at)
{
    if constexpr (N == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
    } else if constexpr (N == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
        w[0] = v.x, w[1] = v.y;
    } else {
        static_assert(N == 4, "1, 2 or 4 words");
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}
template <int N>
__device__ __forceinline__ void store_words(const uint32_t (&w)[N], __amdgpu_buffer_rsrc_t r, int at)
{
    if constexpr (N == 1)
        __builtin_amdgcn_raw_buffer_store_b32(w[0], r, at, 0, 0);
    else if constexpr (N == 2)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, r, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, r, at, 0, 0);
}
#endif

// Workgroup b of n, with neighbours in the list on the same XCD (workgroups go
// round the eight XCDs), so that tiles which share operands share an L2.
__device__ __forceinline__ int by_xcd(int b, int n)
{
    const int x = b & 7, per = n >> 3, rem = n & 7;
    return x * per + min(x, rem) + (b >> 3);
}

// Tile t of ntm x ntn, four tile rows at a time, down each column of them:
// consecutive tiles share few blocks of A and of B.
__device__ __forceinline__ void tile_at(int t, int ntm, int ntn, int* bm, int* bn)
{
    const int grp = t / (4 * ntn), left = t - grp * 4 * ntn;
    const int h = min(4, ntm - 4 * grp);
    *bm = 4 * grp + left % h;
    *bn = left / h;
}

}  // namespace
}  // namespace ns

// ns_check.h -- argument checks shared by the entry points of the layers in 8 bits
// and of the experts' router (ns_q8_api.cpp, ns_f8_api.cpp, ns_route_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <new>
#include <string>
#include <vector>

#include "ns.h"
#include "ns_enqueue.h"

namespace ns {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxPitch = int64_t(1) << 21;    // of the products' operands

std::string nth(int32_t i, const char* what) { return "matrix " + std::to_string(i) + ": " + what; }

// NS_CHECK=1: wait for the stream after every launch (see ns.h).
[[maybe_unused]] ns_status launched(hipError_t e, const char* what, hipStream_t stream)
{
    if (e != hipSuccess)
        return hip_fail(e, what);
    const char* v = std::getenv("NS_CHECK");
    if (v && v[0] == '1' && v[1] == 0) {
        e = hipStreamSynchronize(stream);
        if (e == hipSuccess)
            e = hipGetLastError();
        if (e != hipSuccess)
            return fail(NS_EHIP, std::string("NS_CHECK: the ") + what + " kernel failed (" + hipGetErrorString(e) + ")");
    }
    return NS_OK;
}

// --- outputs -----------------------------------------------------------------
// An output: rows of `len` bytes at a pitch of `pitch` bytes.
struct Span {
    uintptr_t at;
    int64_t rows, len, pitch;
    int32_t index;
    uintptr_t end() const { return at + (uintptr_t)((rows - 1) * pitch + len); }
};

// Two outputs whose byte ranges meet may still be column slices of one wide
// matrix: the same pitch, and columns that do not meet.
bool meet(const Span& a, const Span& b)
{
    if (a.at >= b.end() || b.at >= a.end())
        return false;
    if (a.rows == 1 && b.rows == 1)
        return true;
    const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
    if ((a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) || a.len > pitch || b.len > pitch)
        return true;
    const Span& lo = a.at <= b.at ? a : b;
    const Span& hi = a.at <= b.at ? b : a;
    const int64_t d = (int64_t)((hi.at - lo.at) % (uintptr_t)pitch);   // hi's column in lo's rows
    return !(d >= lo.len && d + hi.len <= pitch);
}

[[maybe_unused]] ns_status check_spans(std::vector<Span>& s)
{
    std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
    for (size_t i = 0; i < s.size(); ++i)
        for (size_t j = i + 1; j < s.size() && s[j].at < s[i].end(); ++j)
            if (meet(s[i], s[j]))
                return fail(NS_EINVAL, "the outputs of matrices " + std::to_string(std::min(s[i].index, s[j].index)) +
                                           " and " + std::to_string(std::max(s[i].index, s[j].index)) + " overlap");
    return NS_OK;
}

// A rows x cols operand that the call reads or writes.
[[maybe_unused]] ns_status check_operand(int32_t i, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld,
                        int64_t max_ld, size_t elt)
{
    if (rows == 0 || cols == 0)
        return NS_OK;
    if (!p)
        return fail(NS_EINVAL, nth(i, name) + " is non-empty but its pointer is NULL");
    if (reinterpret_cast<uintptr_t>(p) % elt)
        return fail(NS_EINVAL, nth(i, name) + " is not aligned to its element size");
    if (ld < cols)
        return fail(NS_EINVAL, nth(i, name) + " has a pitch below its row length");
    if (ld > max_ld)
        return fail(NS_EINVAL, nth(i, name) + " has a pitch above " + std::to_string(max_ld));
    return NS_OK;
}

[[maybe_unused]] ns_status check_dim(int32_t i, int64_t v)
{
    if (v < 0)
        return fail(NS_EINVAL, nth(i, "a dimension is negative"));
    if (v > kMaxDim)
        return fail(NS_EINVAL, nth(i, "a dimension is above 2^24"));
    return NS_OK;
}

// Runs an entry point's body: host allocations that fail are NS_ENOMEM.
template <typename F>
ns_status guarded(F&& f)
{
    clear_error();
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return fail(NS_ENOMEM, "host allocation failed");
    }
}

}  // namespace
}  // namespace ns

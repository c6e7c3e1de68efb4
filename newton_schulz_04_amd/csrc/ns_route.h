// ns_route.h -- descriptors and launch wrappers of the router's kernels (ns_route.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ns {

struct RouteArgs {
    const char* logits;
    int64_t ld;
    const uint8_t* mask;
    int32_t* chosen;
    float* weights;
    int32_t* counts;
    float* probs;
    int32_t* routed;
    float* loss;
    float* part_probs;      // the workgroups' sums of p, kRouteJoin experts at a time
    int32_t* part_counts;   // the same of counts
    int32_t* part_routed;   // workgroups
    uint32_t* arrived;      // workgroups of the join that are done
    int32_t tokens, experts, top_k, normalize;
};

struct RouteGradArgs {
    const char* logits;
    int64_t ld;
    const int32_t* chosen;
    const int32_t* counts;
    const int32_t* routed;
    const float* dweights;
    const float* dloss;
    char* out;
    int64_t ldo;
    int32_t tokens, experts, top_k, normalize;
};

// Lanes that share a token: 16 where 16 values each hold its logits, else 64.
constexpr int kRouteThreads = 512;
inline int route_lanes(int64_t experts) { return experts <= 256 ? 16 : 64; }
// Tokens a workgroup takes at a time.
inline int route_tokens(int64_t experts) { return kRouteThreads / route_lanes(experts); }
// Workgroups: one token a group of lanes until the chip is full, then several.
constexpr int64_t kRouteGroups = 512;
inline int64_t route_groups(int64_t tokens, int64_t experts)
{
    const int64_t per = route_tokens(experts), n = (tokens + per - 1) / per;
    // (a workgroup alone, which needs no join, as long as its tokens are few)
    return n <= 4 ? 1 : n < kRouteGroups ? n : kRouteGroups;
}
// Experts that a workgroup of the join adds up.
constexpr int kRouteJoin = 16;

hipError_t launch_route(const RouteArgs& a, int nwg, int dtype, hipStream_t stream);
hipError_t launch_route_join(const RouteArgs& a, int nwg, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradArgs& a, int nwg, int dtype, hipStream_t stream);

}  // namespace ns

// route.hip - experts and weights of given router logits (select.hpp).
//
// The same selection as a layer with a rule makes, for logits that come from
// elsewhere, or ahead of the layer: a host that fetches experts has to know
// them before («Colibri 是什么» (xxqk.cn) §3.3, expert prefetch).
#include "select.hpp"

namespace cmoe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float logit_of(const float* p) { return *p; }
__device__ __forceinline__ float logit_of(const uint16_t* p) { return bf16_to_f32(*p); }

// One wave per token.
template <typename T, int NQ>
__global__ __launch_bounds__(kThreads) void route_kernel(const T* logits, int64_t ld, int tokens, int E, int k,
                                                         SelectRule rule, int32_t* ids, float* w)
{
    const int waves = (int)gridDim.x * (kThreads / kWave);
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; t < tokens; t += waves) {
        const T* row = logits + t * ld;
        select_token<NQ>([&](int e) { return logit_of(row + e); }, E, k, rule, ids + t * k, w + t * k);
    }
}

template <typename T>
hipError_t launch(const RouteArgs& a, hipStream_t s)
{
    const unsigned blocks = (unsigned)std::min<int64_t>(((int64_t)a.T + 3) / 4, 8192);
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3(blocks), dim3(kThreads), 0, s, (const T*)a.logits, a.ld, a.T, a.E, a.k, a.rule,
                           a.ids, a.w);
    };
    if (a.E <= 64)
        go(route_kernel<T, 1>);
    else if (a.E <= 128)
        go(route_kernel<T, 2>);
    else
        go(route_kernel<T, 4>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    return a.bf16 ? launch<uint16_t>(a, s) : launch<float>(a, s);
}

}  // namespace cmoe

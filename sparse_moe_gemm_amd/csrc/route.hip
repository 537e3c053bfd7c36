// route.hip - experts and weights of given router logits (select.hpp).
//
// The same selection as a layer with a rule makes, for logits that come from
// elsewhere, or ahead of the layer: a host that fetches experts has to know
// them before («Colibri 是什么» (xxqk.cn) §3.3, expert prefetch).
#include "select.hpp"

namespace cmoe {

namespace {

constexpr int kThreads = 256;

// A token's logits in memory.
template <typename T, bool VEC>
struct RowLogits {
    const T* row;
    int E;
    __device__ __forceinline__ float one(int e) const { return element(row, e); }
    template <int NQ>
    __device__ __forceinline__ void all(int e0, float (&l)[NQ]) const
    {
        load_row<VEC>(row, e0, E, -INFINITY, l);
    }
};

template <typename T, bool VEC, int NQ>
__global__ __launch_bounds__(kThreads) void route_kernel(const T* logits, int64_t ld, int tokens, int E, int k,
                                                         SelectRule rule, int32_t* ids, float* w)
{
    const int64_t t = (int64_t)blockIdx.x * (kThreads / kRow) + threadIdx.x / kRow;
    select_token<NQ>(RowLogits<T, VEC>{logits + min(t, (int64_t)tokens - 1) * ld, E}, E, k, rule, t < tokens, ids + t * k,
                     w + t * k);
}

template <typename T>
hipError_t launch(const RouteArgs& a, hipStream_t s)
{
    constexpr int kRows = kThreads / kRow;
    constexpr int64_t kMost = 1 << 27;  // tokens of a launch, which has fewer than 2^32 threads
    auto go = [&](auto kern) {
        for (int64_t t = 0; t < a.T; t += kMost) {
            const int n = (int)std::min<int64_t>(a.T - t, kMost);
            hipLaunchKernelGGL(kern, dim3((unsigned)((n + kRows - 1) / kRows)), dim3(kThreads), 0, s,
                               (const T*)a.logits + t * a.ld, a.ld, n, a.E, a.k, a.rule, a.ids + t * a.k, a.w + t * a.k);
        }
    };
    auto width = [&](auto nq) {
        if (((uintptr_t)a.logits & 15u) == 0 && a.ld * sizeof(T) % 16 == 0)  // every row
            go(route_kernel<T, true, nq()>);
        else
            go(route_kernel<T, false, nq()>);
    };
    switch (select_width(a.E)) {
    case 4: width(std::integral_constant<int, 4>{}); break;
    case 8: width(std::integral_constant<int, 8>{}); break;
    default: width(std::integral_constant<int, 16>{}); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    return a.bf16 ? launch<uint16_t>(a, s) : launch<float>(a, s);
}

}  // namespace cmoe

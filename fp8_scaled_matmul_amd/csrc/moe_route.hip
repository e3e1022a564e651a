// A mixture of experts' router in training, for gfx950: of each token's logits
// the top_k experts and their weights; of the batch the tokens of each expert
// and the balance loss
//   E sum_e f_e P_e,  f_e = counts_e / (N top_k),  P_e = mean softmax(l)_e,
// N the tokens that count; and the logits' gradient.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"

namespace fp8mi {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = 4, kParts = 256;     // waves of a workgroup, workgroups at most

struct RouteKArgs {
    const void* logits;
    int tokens, experts, top_k;
    int64_t ld;
    int renormalize;
    const uint8_t* mask;
    int32_t* ids;
    float* weights;
    float* part_p;          // [workgroups, experts]
    int32_t* part_c;        // [workgroups, experts]
    int32_t* part_n;        // [workgroups]
    const int32_t* counts;  // backward
    const float* grad_weights;
    const float* grad_balance;
    void* dlogits;
    int64_t ldd;
};

__device__ inline float get(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
__device__ inline float get(const float* p) { return *p; }
__device__ inline void put(uint16_t* p, float v) { *p = gemm::to_bf16(v); }
__device__ inline void put(float* p, float v) { *p = v; }

__device__ inline float wave_fmax(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ inline float wave_fsum(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// A token's logits, V to a lane (expert lane + 64 i), -Inf past the last;
// returns false where all are -Inf.
template <typename T, int V>
__device__ inline bool load_row(const RouteKArgs& a, int64_t t, float (&l)[V], float& mx)
{
    const int lane = threadIdx.x & 63;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    mx = -__builtin_inff();
    bool some = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < a.experts ? get(row + e) : -__builtin_inff();
        mx = fmaxf(mx, l[i]);
        some |= !(l[i] == -__builtin_inff());
    }
    mx = wave_fmax(mx);
    return __any(some);
}

// exp(l - max) in place of l, and their sum.
template <int V>
__device__ inline float exponentials(float (&l)[V], float mx)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        l[i] = __builtin_amdgcn_exp2f((l[i] - mx) * kLog2e);
        s += l[i];
    }
    return wave_fsum(s);
}

template <typename T, int V>
__global__ void __launch_bounds__(64 * kWaves) k_route(RouteKArgs a)
{
    __shared__ int32_t count[512];
    __shared__ float prob[kWaves][512];
    __shared__ int32_t number[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int e = threadIdx.x; e < 512; e += 64 * kWaves) count[e] = 0;
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    int n = 0;
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
        float l[V], mx;
        bool on = !a.mask || a.mask[t] != 0;
        if (on) on = load_row<T, V>(a, t, l, mx);
        if (!on) {
            if (lane < a.top_k) {
                a.ids[t * a.top_k + lane] = -1;
                a.weights[t * a.top_k + lane] = 0.0f;
            }
            continue;
        }
        ++n;
        // order: larger logits, then lower experts, NaN last; 0: not there
        uint64_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            const uint32_t u = __builtin_bit_cast(uint32_t, l[i] + 0.0f);
            const uint32_t k = l[i] != l[i] ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
            key[i] = e < a.experts ? (uint64_t)k << 32 | (uint32_t)~e : 0;
        }
        const float total = exponentials<V>(l, mx);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += l[i] / total;
        int mine = 0;
        float w = 0.0f, chosen = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            uint64_t best = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) {
                const uint64_t other = __shfl_xor((unsigned long long)best, off, 64);
                best = other > best ? other : best;
            }
            const int e = (int)~(uint32_t)best;
            float p = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (e == lane + 64 * i) {
                    key[i] = 0;
                    p = l[i];
                }
            }
            p = __shfl(p, e & 63, 64);
            chosen += p;
            if (lane == j) {
                mine = e;
                w = p;
            }
        }
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = mine;
            a.weights[t * a.top_k + lane] = w / (a.renormalize ? chosen : total);
            atomicAdd(&count[mine], 1);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) prob[wave][lane + 64 * i] = sum[i];
    if (lane == 0) number[wave] = n;
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += 64 * kWaves) {
        float s = 0.0f;
        for (int w = 0; w < kWaves; ++w) s += prob[w][e];
        a.part_p[(int64_t)blockIdx.x * a.experts + e] = s;
        a.part_c[(int64_t)blockIdx.x * a.experts + e] = count[e];
    }
    if (threadIdx.x == 0) {
        int s = 0;
        for (int w = 0; w < kWaves; ++w) s += number[w];
        a.part_n[blockIdx.x] = s;
    }
}

// The parts' sums, the balance loss.
__global__ void __launch_bounds__(1024) k_route_finish(const float* part_p, const int32_t* part_c, const int32_t* part_n,
                                                       int parts, int experts, int top_k, int32_t* counts, float* balance)
{
    __shared__ double sh[1024];
    __shared__ int32_t shc[1024];
    __shared__ double loss;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    if (threadIdx.x == 0) loss = 0.0;
    int64_t n = 0;
    for (int i = 0; i < parts; ++i) n += part_n[i];
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + x;
        double s = 0.0;
        int32_t c = 0;
        if (e < experts)
            for (int i = y; i < parts; i += 32) {
                s += part_p[(int64_t)i * experts + e];
                c += part_c[(int64_t)i * experts + e];
            }
        sh[threadIdx.x] = s;
        shc[threadIdx.x] = c;
        __syncthreads();
        for (int h = 16; h >= 1; h >>= 1) {
            if (y < h) {
                sh[threadIdx.x] += sh[threadIdx.x + 32 * h];
                shc[threadIdx.x] += shc[threadIdx.x + 32 * h];
            }
            __syncthreads();
        }
        if (threadIdx.x == 0)
            for (int i = 0; i < 32 && e0 + i < experts; ++i) loss += sh[i] * shc[i];
        if (y == 0 && e < experts) counts[e] = shc[x];
        __syncthreads();
    }
    if (threadIdx.x == 0) *balance = n ? (float)(loss * experts / ((double)n * n * top_k)) : 0.0f;
}

template <typename T, int V>
__global__ void __launch_bounds__(64 * kWaves) k_route_backward(RouteKArgs a)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float gb = a.grad_balance ? *a.grad_balance : 0.0f;
    // the balance loss' gradient for each probability, times the tokens' 1 / N
    float share[V];
    int64_t pairs = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        const int32_t c = e < a.experts ? a.counts[e] : 0;
        share[i] = (float)c;
        pairs += c;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) pairs += __shfl_xor((long long)pairs, off, 64);
    const double n = (double)pairs / a.top_k;
    const float to_share = n > 0.0 ? (float)(gb * (double)a.experts / (n * n * a.top_k)) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) share[i] *= to_share;
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
        T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
        const int32_t* ids = a.ids + t * a.top_k;
        if (ids[0] < 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 64 * i < a.experts) put(out + lane + 64 * i, 0.0f);
            continue;
        }
        float p[V], mx;
        load_row<T, V>(a, t, p, mx);
        const float total = exponentials<V>(p, mx);
        float down = 0.0f;      // sum of p times its gradient
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] /= total;
            down = __builtin_fmaf(p[i], share[i], down);
        }
        down = wave_fsum(down);
        float inner = 0.0f, extra[V];
#pragma unroll
        for (int i = 0; i < V; ++i) extra[i] = 0.0f;
        if (a.grad_weights) {
            for (int j = 0; j < a.top_k; ++j) {
                const float w = a.weights[t * a.top_k + j], g = a.grad_weights[t * a.top_k + j];
                inner = __builtin_fmaf(w, g, inner);
            }
            for (int j = 0; j < a.top_k; ++j) {
                const float w = a.weights[t * a.top_k + j], g = a.grad_weights[t * a.top_k + j];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (ids[j] == lane + 64 * i) extra[i] = a.renormalize ? w * (g - inner) : w * g;
            }
            if (!a.renormalize) down += inner;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 64 * i < a.experts) put(out + lane + 64 * i, __builtin_fmaf(p[i], share[i] - down, extra[i]));
    }
}

int parts_of(int64_t tokens) { return (int)std::min<int64_t>((tokens + kWaves - 1) / kWaves, kParts); }

template <typename F>
void by_experts(int experts, int dtype, F f)
{
    const auto with = [&](auto t) {
        if (experts <= 64) f(t, std::integral_constant<int, 1>{});
        else if (experts <= 128) f(t, std::integral_constant<int, 2>{});
        else if (experts <= 256) f(t, std::integral_constant<int, 4>{});
        else f(t, std::integral_constant<int, 8>{});
    };
    dtype == FP8_IN_BF16 ? with(uint16_t{}) : with(float{});
}

RouteKArgs kernel_args(const RouteArgs& g)
{
    RouteKArgs a = {};
    a.logits = g.logits;
    a.tokens = (int)g.tokens;
    a.experts = (int)g.experts;
    a.top_k = (int)g.top_k;
    a.ld = g.ld;
    a.renormalize = g.renormalize;
    a.mask = g.mask;
    a.ids = g.ids;
    a.weights = g.weights;
    return a;
}

}  // namespace

size_t route_workspace(int64_t tokens, int64_t experts)
{
    return (size_t)parts_of(tokens) * (size_t)(2 * experts + 1) * 4;
}

hipError_t launch_route(const RouteArgs& g, hipStream_t stream)
{
    RouteKArgs a = kernel_args(g);
    const int parts = parts_of(g.tokens);
    a.part_p = static_cast<float*>(g.ws);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + (int64_t)parts * g.experts);
    a.part_n = a.part_c + (int64_t)parts * g.experts;
    if (parts)
        by_experts(a.experts, g.dtype, [&](auto t, auto v) {
            hipLaunchKernelGGL((k_route<decltype(t), decltype(v)::value>), dim3(parts), dim3(64 * kWaves), 0, stream, a);
        });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_finish, dim3(1), dim3(1024), 0, stream, a.part_p, a.part_c, a.part_n, parts, a.experts, a.top_k,
                       g.counts, g.balance);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& g, hipStream_t stream)
{
    if (g.tokens == 0) return hipSuccess;
    RouteKArgs a = kernel_args(g);
    a.counts = g.counts;
    a.grad_weights = g.grad_weights;
    a.grad_balance = g.grad_balance;
    a.dlogits = g.dlogits;
    a.ldd = g.ldd;
    const int grid = (int)std::min<int64_t>((g.tokens + kWaves - 1) / kWaves, 8 * gemm_num_cus());
    by_experts(a.experts, g.dtype, [&](auto t, auto v) {
        hipLaunchKernelGGL((k_route_backward<decltype(t), decltype(v)::value>), dim3(grid), dim3(64 * kWaves), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace fp8mi

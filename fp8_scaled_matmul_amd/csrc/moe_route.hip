// A mixture of experts' router in training, for gfx950: of each token's logits
// the top_k experts and their weights; of the batch the tokens of each expert
// and the balance loss
//   E sum_e f_e P_e,  f_e = counts_e / (N top_k),  P_e = mean softmax(l)_e,
// N the tokens that count; and the logits' gradient.
//
// 65536 x 128, top 8: bf16 forward 16 us and 5 for the sums (4.0 us of traffic),
// backward 14.5 to 15 (7.7); fp32 25 and 5.7 (7.3), backward 15.6 (14).  The forward is
// bound by arithmetic: it sorts each lane's keys and takes top_k times the largest
// of the lanes' first ones; VALU instructions take 84 % (fp32: 89 %) of the cycles in
// which the shader engines are busy.  In the backward they take 54 % (49 %): the rest is
// the latency of a token's chain (loads, reductions, LDS) with four waves a SIMD.
// One token: 3.4, 4.6 and 3.6 us, launches and a trip or two to memory.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"

namespace fp8mi {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
// Waves of a workgroup, and workgroups at most: each brings a part of the sums
// (512 parts: 24.1 us against 20.9 for 65536 x 128).
constexpr int kWaves = 16, kParts = 256;
constexpr int kBackwardBlocks = 1;          // the backward's workgroups a CU at most (2: 16.3 us against 14.5)

struct RouteKArgs {
    const void* logits;
    int tokens, experts, top_k;
    int64_t ld;
    int renormalize;
    const uint8_t* mask;
    int32_t* ids;
    float* weights;
    int32_t* counts;
    float* balance;
    float* part_p;          // [parts, experts]
    int32_t* part_c;        // [parts, experts]
    int32_t* part_n;        // [parts]
    int parts;
    double* part_loss;      // [blocks of 32 experts]
    int32_t* ticket;
    const float* grad_weights;
    const float* grad_balance;
    void* dlogits;
    int64_t ldd;
};

// A token is handled by L = 16, 32 or 64 lanes with V experts each, V sub .. V
// sub + V - 1: up to 128 experts by 16 lanes, so that a wave has 4 tokens at
// work (65536 x 128 bf16, forward and backward: 20.9 and 14.5 us; 32 lanes of 4
// experts 28.8 and 19.1, 64 lanes of 2 41.3 and 23.9).  Reductions over a token's lanes
// are rotations inside 16 (DPP) and, for more, exchanges of groups.
template <int N>
__device__ inline uint32_t rotated(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
__device__ inline float rotated(float v) { return __builtin_bit_cast(float, rotated<N>(__builtin_bit_cast(uint32_t, v))); }
template <int N>
__device__ inline double rotated(double v)
{
    const uint2 b = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, uint2{rotated<N>(b.x), rotated<N>(b.y)});
}
// v of the lane's own and of the other group of 16 (32)
__device__ inline uint2 both16(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return uint2{r[0], r[1]};
}
__device__ inline uint2 both32(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return uint2{r[0], r[1]};
}
template <int L, typename T, typename F>
__device__ inline T reduce(T v, F f)
{
    v = f(v, rotated<8>(v));
    v = f(v, rotated<4>(v));
    v = f(v, rotated<2>(v));
    v = f(v, rotated<1>(v));
    const auto across = [&](auto both) {
        if constexpr (sizeof(T) == 4) {
            const uint2 r = both(__builtin_bit_cast(uint32_t, v));
            v = f(__builtin_bit_cast(T, r.x), __builtin_bit_cast(T, r.y));
        } else {
            const uint2 b = __builtin_bit_cast(uint2, v);
            const uint2 x = both(b.x), y = both(b.y);
            v = f(__builtin_bit_cast(T, uint2{x.x, y.x}), __builtin_bit_cast(T, uint2{x.y, y.y}));
        }
    };
    if constexpr (L >= 32) across(both16);
    if constexpr (L >= 64) across(both32);
    return v;
}

// Keys that order as the selection does: larger logits first, then lower
// experts, NaN last; distinct, and what no expert has is below them all.
//   bf16: the ordered bits above the expert's complement, one 32-bit word
//   fp32: the value as a double, whose 29 free bits hold the expert so that a
//         lower one is larger (infinities and NaN beyond the type's range)
struct Key16 {
    typedef uint32_t T;
    static __device__ T none() { return 0; }
    static __device__ T make(float l, int e)
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);     // -0 as 0
        const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
        return l != l ? (uint32_t)(0xFFFF - e) : (k & 0xFFFF0000u) | (uint32_t)(0xFFFF - e);
    }
    static __device__ int expert(T k) { return 0xFFFF - (int)(k & 0xFFFFu); }
    static __device__ float value(T k)
    {
        const uint32_t o = k & 0xFFFF0000u, b = o & 0x80000000u ? o ^ 0x80000000u : ~o & 0xFFFF0000u;
        return __builtin_bit_cast(float, o == 0 ? 0x7FC00000u : b);
    }
    static __device__ T largest(T a, T b) { return max(a, b); }
    static __device__ T smallest(T a, T b) { return min(a, b); }
};
struct Key32 {
    typedef double T;
    static constexpr double kFar = 0x1p200;
    static __device__ T none() { return -4 * kFar; }
    static __device__ T make(float l, int e)
    {
        // (beyond fp32's range by far; NaN below -Inf)
        const double v = l != l ? -2 * kFar : __builtin_fabsf(l) == __builtin_inff() ? (double)__builtin_copysignf(1.0f, l) * kFar : (double)(l + 0.0f);
        uint64_t b = __builtin_bit_cast(uint64_t, v);
        b |= (b >> 63) ? (uint32_t)e : (uint32_t)(511 - e);
        return __builtin_bit_cast(double, b);
    }
    static __device__ int expert(T k)
    {
        const uint64_t b = __builtin_bit_cast(uint64_t, k);
        const int low = (int)(b & 511u);
        return (b >> 63) ? low : 511 - low;
    }
    static __device__ float value(T k)
    {
        const double v = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~511ull);
        return v <= -2 * kFar ? __builtin_nanf("") : __builtin_fabs(v) >= kFar ? __builtin_copysignf(__builtin_inff(), (float)v) : (float)v;
    }
    static __device__ T largest(T a, T b) { return __builtin_fmax(a, b); }
    static __device__ T smallest(T a, T b) { return __builtin_fmin(a, b); }
};

// a where the mask's bits are set, b elsewhere.
__device__ inline uint32_t choose(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }
__device__ inline double choose(uint32_t mask, double a, double b)
{
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    return __builtin_bit_cast(double, uint2{choose(mask, x.x, y.x), choose(mask, x.y, y.y)});
}

// A lane's V keys in falling order.
template <typename K, int V>
__device__ inline void sort_keys(typename K::T (&k)[V])
{
    const auto order = [&](int i, int j) {
        const auto a = k[i], b = k[j];
        k[i] = K::largest(a, b);
        k[j] = K::smallest(a, b);
    };
    // merge sort of pairs, fours, eights (odd-even merges)
#pragma unroll
    for (int i = 0; i + 1 < V; i += 2) order(i, i + 1);
#pragma unroll
    for (int i = 0; i + 3 < V; i += 4) {
        order(i, i + 2);
        order(i + 1, i + 3);
        order(i + 1, i + 2);
    }
    if constexpr (V == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) order(i, i + 4);
        order(2, 4);
        order(3, 5);
#pragma unroll
        for (int i = 1; i < 7; i += 2) order(i, i + 1);
    }
}

struct __attribute__((packed, aligned(2))) Bf16s {
    uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) Floats {
    float v[8];
};
template <int V>
__device__ inline void load_row(const uint16_t* row, int e0, int experts, float (&l)[V])
{
    if (V == 8 && e0 + V <= experts) {
        const Bf16s b = *reinterpret_cast<const Bf16s*>(row + e0);
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = __builtin_bit_cast(float, i & 1 ? b.w[i / 2] & 0xFFFF0000u : b.w[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            l[i] = e0 + i < experts ? __builtin_bit_cast(float, (uint32_t)row[e0 + i] << 16) : -__builtin_inff();
    }
}
template <int V>
__device__ inline void load_row(const float* row, int e0, int experts, float (&l)[V])
{
    if (V == 8 && e0 + V <= experts) {
        const Floats b = *reinterpret_cast<const Floats*>(row + e0);
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = b.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? row[e0 + i] : -__builtin_inff();
    }
}
template <int V>
__device__ inline void store_row(uint16_t* row, int e0, int experts, const float (&v)[V])
{
    if (V == 8 && e0 + V <= experts) {
        Bf16s b;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) b.w[i] = gemm::pack_bf16(v[2 * i], v[(2 * i + 1) % V]);
        *reinterpret_cast<Bf16s*>(row + e0) = b;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < experts) row[e0 + i] = gemm::to_bf16(v[i]);
    }
}
template <int V>
__device__ inline void store_row(float* row, int e0, int experts, const float (&v)[V])
{
    if (V == 8 && e0 + V <= experts) {
        Floats b;
#pragma unroll
        for (int i = 0; i < V; ++i) b.v[i] = v[i];
        *reinterpret_cast<Floats*>(row + e0) = b;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < experts) row[e0 + i] = v[i];
    }
}

__device__ inline float add(float a, float b) { return a + b; }

// Each lane sorts its keys; then top_k times the largest of the lanes' first
// ones is taken out.  Lane j of a token keeps the j-th.
template <typename T, int L, int V>
__global__ void __launch_bounds__(64 * kWaves) k_route(RouteKArgs a)
{
    using K = std::conditional_t<sizeof(T) == 2, Key16, Key32>;
    constexpr int G = 64 / L;       // tokens of a wave
    __shared__ int32_t count[512];
    __shared__ float prob[kWaves][L * V];
    __shared__ int32_t number[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane % L, e0 = V * sub;
    if (threadIdx.x < 512) count[threadIdx.x] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    int n = 0;
    const int64_t step = (int64_t)gridDim.x * kWaves * G;
    // a token's row, read while the one before is worked on
    float l[V], next[V];
    bool on, next_on;
    const auto fetch = [&](int64_t t0, float (&row)[V], bool& live) {
        const int64_t t = t0 + lane / L;
        live = t < a.tokens && (!a.mask || a.mask[t] != 0);
#pragma unroll
        for (int i = 0; i < V; ++i) row[i] = -__builtin_inff();
        if (live) load_row<V>(static_cast<const T*>(a.logits) + t * a.ld, e0, a.experts, row);
    };
    const int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * G;
    fetch(first, next, next_on);
    for (int64_t t0 = first; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool there = t < a.tokens;
        on = next_on;
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = next[i];
        fetch(t0 + step, next, next_on);
        typename K::T key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = e0 + i < a.experts ? K::make(l[i], e0 + i) : K::none();
        sort_keys<K, V>(key);
        typename K::T mine = K::none();
        float mx = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const typename K::T best = reduce<L>(key[0], K::largest);
            if (j == 0) mx = K::value(best);
            if (sub == j) mine = best;
            // the winner's list moves up; by a mask that the compiler does not see
            // through, else it makes the moves an indexed access
            uint32_t won = key[0] == best ? ~0u : 0u;
            asm("" : "+v"(won));
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = choose(won, i + 1 < V ? key[(i + 1) % V] : K::none(), key[i]);
        }
        // exp(l - max): of all for the sum, of the chosen for the weights.  Over 0
        // where the first choice is -Inf: 0 then says that the row has nothing else,
        // NaN that it has NaN.
        const bool low = mx == -__builtin_inff();
        mx = low ? 0.0f : mx;
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = __builtin_amdgcn_exp2f((l[i] - mx) * kLog2e);
            total += l[i];
        }
        total = reduce<L>(total, add);
        on = on && !(low && total == 0.0f);
        const float chosen = sub < a.top_k ? __builtin_amdgcn_exp2f((K::value(mine) - mx) * kLog2e) : 0.0f;
        const float below = a.renormalize ? reduce<L>(chosen, add) : total;
        if (on) {
            n += sub == 0;
            const float inv = __builtin_amdgcn_rcpf(total);     // off by one step at most
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = __builtin_fmaf(l[i], inv, sum[i]);
        }
        if (there && sub < a.top_k) {
            const int e = on ? K::expert(mine) : -1;
            a.ids[t * a.top_k + sub] = e;
            a.weights[t * a.top_k + sub] = on ? chosen * __builtin_amdgcn_rcpf(below) : 0.0f;
            if (on) atomicAdd(&count[e], 1);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // the wave's tokens together, in a fixed order
        if constexpr (L <= 16) {
            const uint2 r = both16(__builtin_bit_cast(uint32_t, sum[i]));
            sum[i] = __builtin_bit_cast(float, r.x) + __builtin_bit_cast(float, r.y);
        }
        if constexpr (L <= 32) {
            const uint2 r = both32(__builtin_bit_cast(uint32_t, sum[i]));
            sum[i] = __builtin_bit_cast(float, r.x) + __builtin_bit_cast(float, r.y);
        }
        if (lane < L) prob[wave][e0 + i] = sum[i];
    }
    n = (int)wave_sum((uint32_t)n);
    if (lane == 0) number[wave] = n;
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += 64 * kWaves) {
        float s = 0.0f;
#pragma unroll
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

// The parts' sums; the last of the workgroups (32 experts each) adds up the
// balance loss, in their order.
__global__ void __launch_bounds__(1024) k_route_finish(RouteKArgs a)
{
    __shared__ double sh[1024];
    __shared__ int32_t shc[1024], shn[1024];
    __shared__ int last;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + x;
    double s = 0.0;
    int32_t c = 0;
    if (e < a.experts) {
#pragma unroll 4
        for (int i = y; i < a.parts; i += 32) {
            s += a.part_p[(int64_t)i * a.experts + e];
            c += a.part_c[(int64_t)i * a.experts + e];
        }
    }
    sh[threadIdx.x] = s;
    shc[threadIdx.x] = c;
    shn[threadIdx.x] = (int)threadIdx.x < a.parts ? a.part_n[threadIdx.x] : 0;
    static_assert(kParts <= 1024, "a part a thread");
    __syncthreads();
    for (int h = 512; h >= 32; h >>= 1) {
        if ((int)threadIdx.x < h) {
            sh[threadIdx.x] += sh[threadIdx.x + h];
            shc[threadIdx.x] += shc[threadIdx.x + h];
            shn[threadIdx.x] += shn[threadIdx.x + h];
        }
        __syncthreads();
    }
    // the first wave's lower half: in the order of the exchanges
    double loss = threadIdx.x < 32 ? sh[threadIdx.x] * shc[threadIdx.x] : 0.0;
    int n = threadIdx.x < 32 ? shn[threadIdx.x] : 0;
    if (threadIdx.x < 64) {
        for (int off = 16; off >= 1; off >>= 1) {
            loss += __shfl_xor(loss, off, 64);
            n += __shfl_xor(n, off, 64);
        }
    }
    if (threadIdx.x == 0) {
        const double nn = (double)n;
        loss = n ? loss * a.experts / (nn * nn * a.top_k) : 0.0;
        a.part_loss[blockIdx.x] = loss;
        __threadfence();
        last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    }
    if (y == 0 && e < a.experts) a.counts[e] = shc[x];
    __syncthreads();
    if (last && threadIdx.x == 0) {
        __threadfence();
        double loss = 0.0;
        for (int i = 0; i < (int)gridDim.x; ++i) loss += __hip_atomic_load(a.part_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *a.balance = (float)loss;
    }
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(64 * kWaves) k_route_backward(RouteKArgs a)
{
    constexpr int G = 64 / L;
    // what the chosen experts get beside the rest; a lane's V floats in runs of 4,
    // so that its 16 bytes lie beside its neighbours'
    constexpr int R = V < 4 ? V : 4;
    const auto place = [](int e) { return (e % V) / R * (L * R) + e / V * R + e % R; };
    __shared__ __attribute__((aligned(16))) float extra[kWaves][G][L * V];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane % L, e0 = V * sub;
    float* own = extra[wave][lane / L];
    const int64_t step = (int64_t)gridDim.x * kWaves * G, first = ((int64_t)blockIdx.x * kWaves + wave) * G;
    // what belongs to a token, read while the one before is worked on
    struct Row {
        float p[V];
        int id;
        float w, g;
    } next;
    const auto fetch = [&](int64_t t0, Row& r) {
        const int64_t t = t0 + lane / L;
        const bool there = t < a.tokens;
#pragma unroll
        for (int i = 0; i < V; ++i) r.p[i] = -__builtin_inff();
        if (there) load_row<V>(static_cast<const T*>(a.logits) + t * a.ld, e0, a.experts, r.p);
        r.id = -1;
        r.w = r.g = 0.0f;
        if (there && sub < a.top_k) {
            r.id = a.ids[t * a.top_k + sub];
            if (a.grad_weights) {
                r.w = a.weights[t * a.top_k + sub];
                r.g = a.grad_weights[t * a.top_k + sub];
            }
        }
    };
    fetch(first, next);
    // the balance loss' gradient for each probability
    float share[V];
    int c = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t k = e0 + i < a.experts ? a.counts[e0 + i] : 0;
        share[i] = (float)k;
        c += k;
    }
    c = (int)wave_sum(lane < L ? (uint32_t)c : 0u);
    const double n = (double)c / a.top_k;
    const float gb = a.grad_balance ? *a.grad_balance : 0.0f;
    const float to_share = n > 0.0 ? (float)(gb * (double)a.experts / (n * n * a.top_k)) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) share[i] *= to_share;
    for (int64_t t0 = first; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool there = t < a.tokens;
        Row now = next;
        fetch(t0 + step, next);
        float (&p)[V] = now.p;
        const int id = now.id;
        float w = now.w, g = now.g;
        // of a token that is left out the gradient may hold anything
        w = id >= 0 ? w : 0.0f;
        g = id >= 0 ? g : 0.0f;
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            own[place(e0 + i)] = 0.0f;
            mx = fmaxf(mx, p[i]);
        }
        mx = reduce<L>(mx, [](float x, float y) { return fmaxf(x, y); });
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = __builtin_amdgcn_exp2f((p[i] - mx) * kLog2e);
            total += p[i];
        }
        total = reduce<L>(total, add);
        const float inv = __builtin_amdgcn_rcpf(total);
        float down = 0.0f;      // sum of p times its gradient
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] *= inv;
            down = __builtin_fmaf(p[i], share[i], down);
        }
        down = reduce<L>(down, add);
        const float inner = reduce<L>(w * g, add);
        if (!a.renormalize) down += inner;
        // a wave's LDS operations are done in their order, if the compiler keeps it
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (id >= 0 && id < L * V) own[place(id)] = a.renormalize ? w * (g - inner) : w * g;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const bool on = __shfl(id, lane / L * L, 64) >= 0;
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = on ? __builtin_fmaf(p[i], share[i] - down, own[place(e0 + i)]) : 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (there) store_row<V>(static_cast<T*>(a.dlogits) + t * a.ldd, e0, a.experts, d);
    }
}

// Lanes of a token and experts of a lane.
template <typename F>
void by_experts(int experts, int dtype, F f)
{
    const auto with = [&](auto t) {
        const auto go = [&](auto l, auto v) { f(t, l, v); };
        using std::integral_constant;
        if (experts <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
        else if (experts <= 32) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
        else if (experts <= 64) go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
        else if (experts <= 128) go(integral_constant<int, 16>{}, integral_constant<int, 8>{});
        else if (experts <= 256) go(integral_constant<int, 32>{}, integral_constant<int, 8>{});
        else go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    };
    dtype == FP8_IN_BF16 ? with(uint16_t{}) : with(float{});
}
int tokens_of_wave(int64_t experts) { return experts <= 128 ? 4 : experts <= 256 ? 2 : 1; }

// Workgroups of the forward, whose sums the second kernel adds up.
int parts_of(int64_t tokens, int64_t experts)
{
    const int64_t per = kWaves * tokens_of_wave(experts);
    return (int)std::min<int64_t>((tokens + per - 1) / per, kParts);
}
int blocks_of(int64_t experts) { return (int)((experts + 31) / 32); }

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
    a.counts = g.counts;
    return a;
}

__global__ void __launch_bounds__(512) k_route_nothing(int32_t* counts, int experts, float* balance)
{
    if ((int)threadIdx.x < experts) counts[threadIdx.x] = 0;
    if (threadIdx.x == 0) *balance = 0.0f;
}

}  // namespace

size_t route_workspace(int64_t tokens, int64_t experts)
{
    return (size_t)blocks_of(experts) * 8 + 16 + (size_t)parts_of(tokens, experts) * (size_t)(2 * experts + 1) * 4;
}

hipError_t launch_route(const RouteArgs& g, hipStream_t stream)
{
    RouteKArgs a = kernel_args(g);
    a.balance = g.balance;
    if (g.tokens == 0) {
        hipLaunchKernelGGL(k_route_nothing, dim3(1), dim3(512), 0, stream, g.counts, a.experts, g.balance);
        return hipGetLastError();
    }
    a.parts = parts_of(g.tokens, g.experts);
    a.part_loss = static_cast<double*>(g.ws);
    a.ticket = reinterpret_cast<int32_t*>(a.part_loss + blocks_of(g.experts));
    a.part_p = reinterpret_cast<float*>(a.ticket + 4);
    a.part_c = reinterpret_cast<int32_t*>(a.part_p + (int64_t)a.parts * g.experts);
    a.part_n = a.part_c + (int64_t)a.parts * g.experts;
    by_experts(a.experts, g.dtype, [&](auto t, auto l, auto v) {
        hipLaunchKernelGGL((k_route<decltype(t), decltype(l)::value, decltype(v)::value>), dim3(a.parts), dim3(64 * kWaves), 0,
                           stream, a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_finish, dim3(blocks_of(g.experts)), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& g, hipStream_t stream)
{
    if (g.tokens == 0) return hipSuccess;
    RouteKArgs a = kernel_args(g);
    a.grad_weights = g.grad_weights;
    a.grad_balance = g.grad_balance;
    a.dlogits = g.dlogits;
    a.ldd = g.ldd;
    const int64_t per = kWaves * tokens_of_wave(g.experts);
    const int grid = (int)std::min<int64_t>((g.tokens + per - 1) / per, kBackwardBlocks * gemm_num_cus());
    by_experts(a.experts, g.dtype, [&](auto t, auto l, auto v) {
        hipLaunchKernelGGL((k_route_backward<decltype(t), decltype(l)::value, decltype(v)::value>), dim3(grid),
                           dim3(64 * kWaves), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace fp8mi

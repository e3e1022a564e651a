// A mixture-of-experts layer with 4-bit (OCP MXFP4) weights for at most 64
// tokens, gfx950.
//
//   l[t, e]  = sum_c x[t, c] R[e, c]                          (router, float64 sums)
//   E(t)     = the top_k experts by l, equal logits to the lower expert
//   p[t, e]  = exp(l - max) / sum exp(l - max), over E(t) or over all experts
//   g, u     = W1[e] x[t]  (gate rows, then up rows)
//   a[t, e]  = p g / (1 + exp(-g)) u
//   y[t]     = sum over e in E(t) of W2[e] a[t, e]
//
// What bounds it is the read of the chosen experts' codes, half a byte a
// weight, each read once; so the weights go from memory to registers as they
// lie and are decoded there, two to an instruction, to bf16, which holds code
// times scale exactly.  The products are v_mfma_f32_16x16x32_bf16's: 16 rows
// of weights by 16 columns of activations, exact products, fp32 sums.  A
// column of the first layer is a token's x as it is.  The second layer's
// activations are fp32 numbers, each the exact sum of three bf16 pieces of 8
// bits; a column there is one piece of one token, and the columns of a token
// are added at the end.  (E4M3 pieces and undecoded weights through
// v_mfma_scale_f32_16x16x128_f8f6f4 take no decoding, but that instruction adds
// the products of neighbouring elements aligned to the largest of them
// and drops what lies 2^-13 below it: measured, errors of 2^-18 of the summed
// sizes for normal data and 2^-13 at worst, against 2^-22 with bf16 operands.)
// Sums are in an order that only the sizes and the chosen experts set: no
// atomics on values.
//
// Three launches: the router, which also lists the reached experts and their
// tokens; up; down.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

using gemm::v4f;
typedef double v4d __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kUnit = 256;          // K elements of a row of codes: rows are padded to whole units
constexpr int kPieces = 3;          // bf16 numbers that add up to an fp32 one

// Some tokens of an expert: the first ones of the mask, which lie among all
// chosen (token, expert) pairs, in order of the experts, then of the tokens,
// at places off, off + 1, ..  The first layer takes an expert's tokens 16 at a
// time, the second 5 (a column each piece).
struct MoeGroup {
    int32_t expert, off;
    uint64_t mask;
};
constexpr int kUpTokens = 16;
constexpr int kDownTokens = 16 / kPieces;

// Workspace.  What workgroups of one launch hand to each other goes through
// agent-scope atomics.
struct MoeArgs {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* router;
    int64_t ldr;
    int tokens, experts, top_k, hidden, inner, renormalize;
    int hp, ip;                     // hidden, inner in whole panels of 512
    const uint8_t* q1;
    const uint8_t* s1;
    int64_t ldq1, eq1, ps1, es1;    // bytes between rows, experts, scale panels, experts' scales
    const uint8_t* q2;
    const uint8_t* s2;
    int64_t ldq2, eq2, ps2, es2;
    uint16_t* y;
    int64_t ldy;
    int32_t* ids;
    float* weights;
    uint32_t* arrived;              // [5] router workgroups done: of each 16 tokens, and token tiles; zero between calls
    double* logits;                 // [splits, tokens, experts] partial sums
    uint16_t* xq;                   // [tokens, hp] x in the order of place_of, zeros past hidden
    int32_t* count;                 // [2] groups of the first layer, of the second
    MoeGroup* up_groups;            // [max_groups(kUpTokens)], by expert
    MoeGroup* groups;               // [max_groups(kDownTokens)], by expert
    float* prob;                    // [tokens top_k] the weight at each place
    uint16_t* aq;                   // [tokens top_k, 3, ip] pieces at each place, in the order of place_of
    fp8_counters* ctr;
    float* part;                    // [shares, tokens, hidden] partial sums of y
    uint32_t* arrived_rows;         // [row blocks of y] workgroups done; zero between calls
    int tiles_e, tiles_t, splits;   // router tiles of 16 x 16, K splits
    int shares;                     // workgroups that share a row block of y
    int max_up_groups, max_groups;  // most groups there can be
};

template <typename T>
__device__ inline void agent_store(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ inline T agent_load(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// ------------------------------------------------------------------ matrix instruction
// One unit (256 K) of a lane's row of weights, and of its column.  16 rows x
// 16 columns x 128 K in four instructions: lane l holds 32 weights of row
// l % 16, K 32 (l / 16) on, one scale block, 8 of them an instruction, and the
// same K of column l % 16.  The columns' memory has each 128 elements in the
// order in which the instructions take them.
struct UnitW {
    uint4 q[2];
};
struct UnitX {
    uint4 q[2][4];
};
// Where element k of a column lies; eight from a multiple of eight on stay together.
__device__ inline int place_of(int k) { return (k & ~127) | (k & 24) << 2 | (k & 96) >> 2 | (k & 7); }

template <typename T>
__device__ inline T load_at(const uint8_t* base, uint32_t off)
{
    return *reinterpret_cast<const T*>(base + off);
}
// base uniform; off: the lane's row (column), 16 (l / 16) bytes in.
__device__ inline void load_w(UnitW& o, const uint8_t* base, uint32_t off)
{
    o.q[0] = load_at<uint4>(base, off);
    o.q[1] = load_at<uint4>(base + 64, off);
}
__device__ inline void load_x(UnitX& o, const uint16_t* base, uint32_t off)
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o.q[k][j] = load_at<uint4>(reinterpret_cast<const uint8_t*>(base) + 256 * k + 64 * j, off);
}
// Eight weights, times their scale.
__device__ inline v8bf decode8(uint32_t w, float s)
{
    const uint4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
    return __builtin_bit_cast(v8bf, v);
}
// sw: the unit's 8 scale bytes.
__device__ inline void unit_mma(v4f& acc, const UnitW& w, const UnitX& x, const uint2& sw)
{
    const int sh = 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float s = mx4::scale_float(((k ? sw.y : sw.x) >> sh) & 255u);
        const uint32_t q[4] = {w.q[k].x, w.q[k].y, w.q[k].z, w.q[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(q[j], s), __builtin_bit_cast(v8bf, x.q[k][j]), acc, 0, 0,
                                                          0);
    }
}

// A neighbour's value within 16 lanes.
template <int CTRL>
__device__ inline float dpp_f(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
constexpr int kDppNext1 = 0x101, kDppNext2 = 0x102;     // lanes l + 1, l + 2

// ------------------------------------------------------------------ router
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxSplits = 8;
constexpr int kChunk = 32;          // K of 8 fp64 matrix instructions
constexpr int kRouteDepth = 2;      // chunks read at a time

// Eight elements of a row from column c on (a multiple of 8), in two steps, so
// that several reads are on their way at once: read8 takes 16 bytes, wherever
// an element may lie, and where the row ends before c + 8 its last eight;
// trim8 moves those to their places, zeros past the end.
typedef uint32_t u4x2 __attribute__((ext_vector_type(4), aligned(2)));
__device__ inline uint4 read8(const uint16_t* row, int c, int cols)
{
    if (cols >= 8) {
        const u4x2 v = *reinterpret_cast<const u4x2*>(row + min(c, cols - 8));
        return uint4{v.x, v.y, v.z, v.w};
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < cols) w[j >> 1] |= (uint32_t)row[j] << (16 * (j & 1));
    return uint4{w[0], w[1], w[2], w[3]};
}
__device__ inline uint4 trim8(uint4 v, int c, int cols)
{
    const int past = c - min(c, max(cols - 8, 0));
    if (past & 1)
        v = uint4{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
    if (past & 2) v = uint4{v.y, v.z, v.w, 0};
    if (past & 4) v = uint4{v.z, v.w, 0, 0};
    return past >= 8 ? uint4{0, 0, 0, 0} : v;
}

// One wave: 512 columns of a token to their places.  A block of 32 that holds
// an Inf or NaN becomes NaN.
__device__ inline void place_x(const MoeArgs& p, int item)
{
    const int lane = threadIdx.x & 63;
    const int panels = (p.hp + mx4::kPanel - 1) / mx4::kPanel;
    const int t = item / panels, c = (item - t * panels) * mx4::kPanel + 8 * lane;
    if (t >= p.tokens || c >= p.hp) return;
    uint4 v = trim8(read8(p.x + t * p.ldx, c, p.hidden), c, p.hidden);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFF0000u, (w[j] << 16) & 0x7FFF0000u));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
    if (amax >= 0x7F800000u) v = uint4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    *reinterpret_cast<uint4*>(p.xq + (int64_t)t * p.hp + place_of(c)) = v;
}

// fp64 as an unsigned key over 1 of the same order; NaN lowest, +0 and -0
// alike
__device__ inline uint64_t key_of(double v)
{
    if (v != v) return 1;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// The largest value of the wave's lanes, in every lane.
__device__ inline uint32_t max_of_wave(uint32_t v)
{
    const auto step = [](uint32_t a, int moved) { return max(a, (uint32_t)moved); };
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));      // l ^ 1
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));      // l ^ 2
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));     // 4, then 8 across of 16
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}

// One wave: the top_k experts of token t and their weights, to `ids` and
// `weights` too.  Lane l holds experts l, l + 64, .. up to 64 N.
template <int N>
__device__ inline void select(const MoeArgs& p, int t, int* ids, float* weights)
{
    const int lane = threadIdx.x & 63;
    const int64_t split = (int64_t)p.tokens * p.experts;
    const uint64_t* at = reinterpret_cast<const uint64_t*>(p.logits) + (int64_t)t * p.experts;
    double l[N];
#pragma unroll
    for (int j = 0; j < N; ++j) l[j] = 0;
    constexpr int kAtOnce = kMaxSplits / N;
    for (int s0 = 0; s0 < p.splits; s0 += kAtOnce) {
        uint64_t part[N][kAtOnce];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int s = 0; s < kAtOnce; ++s)
                part[j][s] =
                    s0 + s < p.splits ? agent_load(at + (s0 + s) * split + min(64 * j + lane, p.experts - 1)) : 0;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int s = 0; s < kAtOnce; ++s) l[j] += __builtin_bit_cast(double, part[j][s]);
    }
    // a lane's own in falling order (equal ones as they come); key 0: none, or taken
    uint32_t hi[N], lo[N], slot[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint64_t key = 64 * j + lane < p.experts ? key_of(l[j]) : 0;
        hi[j] = (uint32_t)(key >> 32);
        lo[j] = (uint32_t)key;
        slot[j] = j;
    }
#pragma unroll
    for (int i = N - 1; i > 0; --i)
#pragma unroll
        for (int j = 0; j < i; ++j) {
            const uint64_t x = (uint64_t)hi[j] << 32 | lo[j], y = (uint64_t)hi[j + 1] << 32 | lo[j + 1];
            const bool swap = y > x;
            const uint32_t h = hi[j], w = lo[j], k = slot[j];
            hi[j] = swap ? hi[j + 1] : h;
            lo[j] = swap ? lo[j + 1] : w;
            slot[j] = swap ? slot[j + 1] : k;
            hi[j + 1] = swap ? h : hi[j + 1];
            lo[j + 1] = swap ? w : lo[j + 1];
            slot[j + 1] = swap ? k : slot[j + 1];
        }
    int id = 0;                         // lane r: rank r's
    for (int r = 0; r < p.top_k; ++r) {
        // the lanes that hold the largest: by the high words; where those are
        // alike by the low words, then the expert
        const uint32_t top_hi = max_of_wave(hi[0]);
        uint64_t who = __ballot(hi[0] == top_hi);
        const uint32_t e = 64 * slot[0] + lane;
        if (who & (who - 1)) {
            const bool in = who >> lane & 1;
            const uint32_t top_lo = max_of_wave(in ? lo[0] : 0u);
            const bool still = in && lo[0] == top_lo;
            const uint32_t first = ~max_of_wave(still ? ~e : 0u);
            who = __ballot(still && e == first);
        }
        const int owner = __builtin_ctzll(who);
        const int chosen = __builtin_amdgcn_readlane((int)e, owner);
        id = lane == r ? chosen : id;
        const bool took = lane == owner;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            hi[j] = took ? (j + 1 < N ? hi[j + 1] : 0u) : hi[j];
            lo[j] = took ? (j + 1 < N ? lo[j + 1] : 0u) : lo[j];
            slot[j] = took ? (j + 1 < N ? slot[j + 1] : 0u) : slot[j];
        }
    }
    double mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const double v = __shfl(l[j], id & 63, 64);
        mine = id >> 6 == j ? v : mine;
    }
    const double top = __shfl(mine, 0, 64);
    const float z = lane < p.top_k ? expf((float)(mine - top)) : 0.0f;
    float sum = z;
    if (!p.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) sum += 64 * j + lane < p.experts ? expf((float)(l[j] - top)) : 0.0f;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane < p.top_k) {
        const int i = t * p.top_k + lane;
        agent_store(p.ids + i, id);
        agent_store(p.weights + i, z / sum);
        ids[i] = id;
        weights[i] = z / sum;
    }
}

// Adds this workgroup to a count of `all`, after its stores have completed.
// True in the last of them, which leaves the count zero.
__device__ inline bool last_of(uint32_t* count, uint32_t all)
{
    __shared__ int s_last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        s_last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == all;
        if (s_last) agent_store(count, 0u);
    }
    __syncthreads();
    return s_last;
}

// The groups of the reached experts in order.  ids and
// weights: of every pair.
__device__ inline void list_reached(const MoeArgs& p, unsigned long long* mask, uint32_t* off, const int* ids,
                                    const float* weights)
{
    __shared__ uint32_t s_sum[kRouteWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    static_assert(kRouteThreads >= kMoeMaxExperts && kRouteThreads >= kMoeMaxTokens * kMoeMaxTopK, "a thread each");
    mask[threadIdx.x] = 0;
    __syncthreads();
    const int t = threadIdx.x / p.top_k;
    const int e = t < p.tokens ? min(max(ids[threadIdx.x], 0), p.experts - 1) : -1;
    if (e >= 0) atomicOr(&mask[e], 1ull << t);
    __syncthreads();
    const int n = __builtin_popcountll(mask[threadIdx.x]);
    const int groups = (n + kDownTokens - 1) / kDownTokens, up_groups = (n + kUpTokens - 1) / kUpTokens;
    // inclusive sums over the wave, of all three at once: at most 1024 pairs,
    // which makes at most 717 and 576 groups
    const uint32_t all = (uint32_t)(n | groups << 11 | up_groups << 21);
    uint32_t sum = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)sum, d, 64);
        sum += lane >= d ? o : 0;
    }
    if (lane == 63) s_sum[wave] = sum;
    __syncthreads();
    sum -= all;
    uint32_t total = 0;
    const int waves = (p.experts + 63) / 64;
    for (int i = 0; i < waves; ++i) {
        sum += i < wave ? s_sum[i] : 0u;
        total += s_sum[i];
    }
    off[threadIdx.x] = sum;
    // sums: of expert e; left: its tokens from the nth on
    const auto list = [&](uint32_t sums, int e, int nth, uint64_t left) {
        const MoeGroup group{e, (int)(sums & 0x7FF) + nth, left};
        if (nth % kDownTokens == 0) p.groups[((sums >> 11) & 0x3FF) + nth / kDownTokens] = group;
        if (nth % kUpTokens == 0) p.up_groups[(sums >> 21) + nth / kUpTokens] = group;
    };
    if (n) list(sum, threadIdx.x, 0, mask[threadIdx.x]);
    if (threadIdx.x == 0) {
        p.count[0] = total >> 21;
        p.count[1] = (total >> 11) & 0x3FF;
    }
    __syncthreads();
    if (e < 0) return;
    // each pair to its place; those that begin a further group write it (the
    // first ones are on their way before the wait: 0.5 us of one token's 26)
    const uint64_t before = mask[e] & ((1ull << t) - 1);
    const int nth = __builtin_popcountll(before);
    const uint32_t sums = off[e];
    p.prob[(sums & 0x7FF) + nth] = weights[threadIdx.x];
    if (nth) list(sums, e, nth, mask[e] ^ before);
}

// Workgroups below tiles_e tiles_t splits take 16 tokens x 16 experts of the
// logits and a share of K, which their waves split.  The last of 16 tokens to
// arrive selects, the last of those lists the reached experts.  The others
// bring x to its places.  fp64 sums: products of bf16 are exact in fp64, so that
// another order of a sum could choose other experts only between logits equal
// to about 2^-50.  One token, 64 experts of 2048: 7.6 us (9.5 under a profiler),
// of which the logits 3.7, their way to one workgroup 0.6, the selection 2.0 and
// the lists 1.3; 64 tokens, 128 experts of 4096: 14 us.
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(MoeArgs p)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nroute = p.tiles_e * p.tiles_t * p.splits;
    if ((int)blockIdx.x >= nroute) {
        place_x(p, ((int)blockIdx.x - nroute) * kRouteWaves + wave);
        return;
    }
    __shared__ __attribute__((aligned(16))) double red[kRouteWaves][256];
    __shared__ int s_ids[kMoeMaxTokens * kMoeMaxTopK];
    __shared__ float s_weights[kMoeMaxTokens * kMoeMaxTopK];
    static_assert(sizeof(red) >= kRouteThreads * (sizeof(uint64_t) + sizeof(uint32_t)), "the lists' masks and places");
    const int tt = blockIdx.x / (p.tiles_e * p.splits), rest = blockIdx.x - tt * p.tiles_e * p.splits;
    const int split = rest / p.tiles_e, te = rest - split * p.tiles_e;
    const int t = min(16 * tt + (lane & 15), p.tokens - 1), e = min(16 * te + (lane & 15), p.experts - 1);
    const uint16_t* xr = p.x + t * p.ldx;
    const uint16_t* rr = p.router + e * p.ldr;
    v4d acc = {0, 0, 0, 0};
    const int chunks = (p.hidden + kChunk - 1) / kChunk;
    const int stride = kRouteWaves * p.splits;
    for (int c0 = split * kRouteWaves + wave; c0 < chunks; c0 += kRouteDepth * stride) {
        uint4 a[kRouteDepth], b[kRouteDepth];
#pragma unroll
        for (int d = 0; d < kRouteDepth; ++d) {
            const int from = kChunk * (c0 + d * stride), c = from + 8 * (lane >> 4);
            if (from >= p.hidden) break;
            a[d] = read8(rr, c, p.hidden);
            b[d] = read8(xr, c, p.hidden);
        }
#pragma unroll
        for (int d = 0; d < kRouteDepth; ++d) {
            const int from = kChunk * (c0 + d * stride);
            if (from >= p.hidden) break;
            if (from + kChunk > p.hidden) {
                a[d] = trim8(a[d], from + 8 * (lane >> 4), p.hidden);
                b[d] = trim8(b[d], from + 8 * (lane >> 4), p.hidden);
            }
            const uint32_t aw[4] = {a[d].x, a[d].y, a[d].z, a[d].w}, bw[4] = {b[d].x, b[d].y, b[d].z, b[d].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_lo(aw[j]), (double)bf16_lo(bw[j]), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_hi(aw[j]), (double)bf16_hi(bw[j]), acc, 0, 0, 0);
            }
        }
    }
    // register i of lane l: expert 4 i + l / 16, token l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(4 * i + (lane >> 4)) * 16 + (lane & 15)] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        double s = red[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kRouteWaves; ++w) s += red[w][threadIdx.x];
        const int oe = 16 * te + (threadIdx.x >> 4), ot = 16 * tt + (threadIdx.x & 15);
        if (oe < p.experts && ot < p.tokens)
            agent_store(reinterpret_cast<uint64_t*>(p.logits) + ((int64_t)split * p.tokens + ot) * p.experts + oe,
                        __builtin_bit_cast(uint64_t, s));
    }
    if (!last_of(p.arrived + tt, (uint32_t)(p.tiles_e * p.splits))) return;
    static_assert(kRouteWaves == 16, "a wave each token");
    if (16 * tt + wave < p.tokens) {
        const int at = 16 * tt + wave;
        if (p.experts <= 64)
            select<1>(p, at, s_ids, s_weights);
        else if (p.experts <= 128)
            select<2>(p, at, s_ids, s_weights);
        else if (p.experts <= 256)
            select<4>(p, at, s_ids, s_weights);
        else
            select<8>(p, at, s_ids, s_weights);
    }
    if (p.tiles_t > 1) {
        if (!last_of(p.arrived + kMoeMaxTokens / 16, (uint32_t)p.tiles_t)) return;
        if ((int)threadIdx.x < p.tokens * p.top_k) {
            s_ids[threadIdx.x] = agent_load(p.ids + threadIdx.x);
            s_weights[threadIdx.x] = agent_load(p.weights + threadIdx.x);
        }
    }
    __syncthreads();
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(&red[0][0]);
    list_reached(p, mask, reinterpret_cast<uint32_t*>(mask + kRouteThreads), s_ids, s_weights);
}

// Lists that an earlier launch wrote, at uniform places: read through the
// scalar cache, beside the vector reads and not in their order.
template <typename T>
__device__ inline T listed(const T* list, int i)
{
    return ((const __attribute__((address_space(4))) T*)list)[i];
}
// What the lists hold, within their bounds whatever is there: a workspace
// that was not zeroed makes wrong results, not wild reads.
__device__ inline int up_group_count(const MoeArgs& p) { return min(max(listed(p.count, 0), 0), p.max_up_groups); }
__device__ inline int group_count(const MoeArgs& p) { return min(max(listed(p.count, 1), 0), p.max_groups); }
__device__ inline MoeGroup group_at(const MoeArgs& p, const MoeGroup* list, int i)
{
    const uint32_t* words = reinterpret_cast<const uint32_t*>(list + i);
    MoeGroup r;
    r.expert = min(max((int)listed(words, 0), 0), p.experts - 1);
    r.mask = ((uint64_t)listed(words, 2) | (uint64_t)listed(words, 3) << 32) & (~0ull >> (64 - p.tokens));
    r.mask = r.mask ? r.mask : 1ull;
    r.off = min(max((int)listed(words, 1), 0), p.tokens * p.top_k - __builtin_popcountll(r.mask));
    return r;
}
// The c-th token of a mask.
__device__ inline int token_of(uint64_t mask, int c)
{
    for (int j = 0; j < c; ++j) mask &= mask - 1;
    return __builtin_ctzll(mask);
}

// ------------------------------------------------------------------ up
constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / 64;

// v as three bf16 numbers, in the high halves of words: 8 bits of it each, so
// that they add up to v (an fp32 number has 24; bits under 2^-133 are lost).
// Inf and NaN stand in the first alone.
__device__ inline void split(float v, uint32_t& a, uint32_t& b, uint32_t& c)
{
    const auto top = [](float f) { return __builtin_bit_cast(uint32_t, f) & 0xFFFF0000u; };
    const auto val = [](uint32_t w) { return __builtin_bit_cast(float, w); };
    const bool finite = (__builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu) < 0x7F800000u;
    a = finite ? top(v) : v != v ? 0x7FC00000u : __builtin_bit_cast(uint32_t, v);
    const float r = finite ? v - val(a) : 0.0f;
    b = top(r);
    c = top(r - val(b));
}

// A workgroup takes an expert's 32 gate rows and the 32 up rows of the same
// outputs, K over its waves, for a group of up to 16 tokens, a column each.
// 64 tokens, 128 experts of 4096 x 1024: 105 us, 5.3 TB/s; one token, 8 experts
// of 2048 x 1408: 9.5 us for 24.5 MB.  (64 tokens, the whole layer, 203 us: 201
// with 8 waves a workgroup, 205 with 2, 214 with the next unit's weights read
// ahead; without the barrier below the compiler puts half of the reads off
// until others have arrived: 212.)
__global__ void __launch_bounds__(kUpThreads, 3) k_moe_up(MoeArgs p)
{
    __shared__ v4f red[kUpWaves][4][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (p.inner + 31) / 32;
    const int group = blockIdx.x / tiles, tile = blockIdx.x - group * tiles;
    const MoeGroup at = group_at(p, p.up_groups, group);
    if (group >= up_group_count(p)) return;
    const int e = at.expert, off = at.off;
    const int n = min(__builtin_popcountll(at.mask), kUpTokens);
    const int c16 = lane & 15, q = lane >> 4;

    // gate rows; up rows lie `inner` rows on
    const uint8_t* wq = p.q1 + e * p.eq1 + 32 * tile * p.ldq1;
    const uint8_t* ws = p.s1 + e * p.es1 + 32 * tile * 16;
    uint32_t woff[2], soff[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = min(16 * h + c16, p.inner - 1 - 32 * tile);
        woff[h] = (uint32_t)(row * p.ldq1 + 16 * q);
        soff[h] = (uint32_t)(row * 16);
    }
    const int units = (p.hidden + kUnit - 1) / kUnit;
    const int c = min(c16, n - 1);
    const uint32_t xoff = (uint32_t)(token_of(at.mask, c) * p.hp) * 2 + 16 * q;
    const float prob = p.prob[off + c];
    v4f acc[4] = {};
    for (int u = wave; u < units; u += kUpWaves) {
        UnitW w[4];
        uint2 sw[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t far = (r >> 1) * (int64_t)p.inner;
            sw[r] = load_at<uint2>(ws + far * 16 + (u >> 1) * p.ps1 + 8 * (u & 1), soff[r & 1]);
            load_w(w[r], wq + far * p.ldq1 + u * 128, woff[r & 1]);
        }
        UnitX x;
        load_x(x, p.xq + u * kUnit, xoff);
        __builtin_amdgcn_sched_barrier(0);      // every read of the unit on its way first
#pragma unroll
        for (int r = 0; r < 4; ++r) unit_mma(acc[r], w[r], x, sw[r]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
    // wave r: 16 r + 4 q + i of the 32 outputs, token c16
    if (wave > 1 || c16 >= n) return;
    v4f g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kUpWaves; ++w) {
        g += red[w][wave][lane];
        u += red[w][wave + 2][lane];
    }
    uint32_t o[kPieces][4];
    const int k = 16 * wave + 4 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = prob * (g[i] / (1.0f + expf(-g[i])) * u[i]);
        split(32 * tile + k + i < p.inner ? v : 0.0f, o[0][i], o[1][i], o[2][i]);
    }
    uint16_t* aq = p.aq + (int64_t)(off + c) * kPieces * p.ip;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        *reinterpret_cast<uint2*>(aq + (int64_t)i * p.ip + place_of(32 * tile + k)) =
            uint2{o[i][0] >> 16 | o[i][1], o[i][2] >> 16 | o[i][3]};
    // zeros to the end of the last panel
    if (tile == tiles - 1)
        for (int z = 32 * tiles; z < p.ip; z += 32)
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                *reinterpret_cast<uint2*>(aq + (int64_t)i * p.ip + place_of(z + k)) = uint2{0, 0};
}

// ------------------------------------------------------------------ down
constexpr int kDownThreads = 256;
constexpr int kDownWaves = kDownThreads / 64;
constexpr int kMaxShares = 8;

// `shares` workgroups take the same 16 R rows of y for every token.  Their waves
// share the steps (up to five tokens of an expert, a unit of K) in a fixed
// order, each with sums of its own in LDS, which are added in wave order at the
// end, and over the workgroups by the last of them to arrive.  A step's weights
// are read two steps ahead and its columns one: reads come back in order, so
// the columns of the next step are asked for before the weights of the one
// after it, and no read in the loop hangs on a branch.
// 64 tokens, 128 experts of 4096 x 1024: 80 us, 3.5 TB/s, of which 19 us are the
// columns (from L2); one token, 8 experts of 2048 x 1408: 9 us for 12.2 MB.
template <int R>
__global__ void __launch_bounds__(kDownThreads, 2) k_moe_down(MoeArgs p)
{
    constexpr int kDownRows = 16 * R;
    extern __shared__ __attribute__((aligned(16))) float ysum[];     // [waves, tokens, 16 R]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int block = blockIdx.x / p.shares, share = blockIdx.x - block * p.shares;
    const int row0 = kDownRows * block;
    const int groups = group_count(p);

    const int c16 = lane & 15, q = lane >> 4;
    uint32_t woff[R], soff[R];
#pragma unroll
    for (int h = 0; h < R; ++h) {
        const int row = min(16 * h + c16, p.hidden - 1 - row0);
        woff[h] = (uint32_t)(row * p.ldq2 + 16 * q);
        soff[h] = (uint32_t)(row * 16);
    }
    const int units = (p.inner + kUnit - 1) / kUnit;
    const int steps = groups * units;
    float* mine = ysum + wave * p.tokens * kDownRows;

    struct At {
        int e, row, n, unit;        // row: of the first token's first piece; n tokens
        uint64_t mask;
    };
    struct Entry {
        MoeGroup r;
        int unit;
    };
    // what the list holds for step i, then what it means
    const auto entry = [&](int i) {
        i = min(i, steps - 1);
        const int g = i / units;
        return Entry{group_at(p, p.groups, g), i - g * units};
    };
    const auto at_step = [&](const Entry& x) {
        At a;
        a.unit = x.unit;
        a.mask = x.r.mask;
        a.e = x.r.expert;
        a.row = kPieces * x.r.off;
        a.n = min(__builtin_popcountll(x.r.mask), kDownTokens);
        return a;
    };
    struct W {
        UnitW u[R];
        uint2 s[R];
    };
    const auto get_w = [&](W& w, const At& a) {
        const uint8_t* base = p.q2 + a.e * p.eq2 + row0 * p.ldq2 + 128 * a.unit;
        const uint8_t* sbase = p.s2 + a.e * p.es2 + (a.unit >> 1) * p.ps2 + row0 * 16 + 8 * (a.unit & 1);
#pragma unroll
        for (int h = 0; h < R; ++h) {
            w.s[h] = load_at<uint2>(sbase, soff[h]);
            load_w(w.u[h], base, woff[h]);
        }
    };
    const auto get_x = [&](UnitX& x, const At& a) {
        const uint32_t col = (uint32_t)min(c16, kPieces * a.n - 1);
        load_x(x, p.aq + (int64_t)a.row * p.ip + kUnit * a.unit, col * (uint32_t)p.ip * 2 + 16 * q);
    };
    // 16 R rows x the tokens of 15 columns, added to this wave's sums
    const auto compute = [&](const W& w, const UnitX& x, const At& a) {
        static_assert(kPieces == 3, "two neighbours");
        const int c = c16 / kPieces;
        const bool mine_to_add = c16 % kPieces == 0 && c < a.n;
        v4f* to = reinterpret_cast<v4f*>(mine + token_of(a.mask, min(c, a.n - 1)) * kDownRows + 4 * q);
#pragma unroll
        for (int h = 0; h < R; ++h) {
            v4f acc = {0, 0, 0, 0};
            unit_mma(acc, w.u[h], x, w.s[h]);
            v4f sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = acc[i] + (dpp_f<kDppNext1>(acc[i]) + dpp_f<kDppNext2>(acc[i]));
            if (mine_to_add) to[4 * h] += sum;
        }
    };

    // this wave's steps, neighbours in memory
    const int who = share * kDownWaves + wave, all = p.shares * kDownWaves;
    const int first = (int)((int64_t)steps * who / all), end = (int)((int64_t)steps * (who + 1) / all);
    W w0, w1;
    UnitX x0, x1;
    At a0, a1;
    if (first < end) {
        const Entry e0 = entry(first), e1 = entry(first + 1);
        a0 = at_step(e0);
        a1 = at_step(e1);
        get_w(w0, a0);
        get_x(x0, a0);
        get_w(w1, a1);
    }
    for (int i = lane; i < p.tokens * kDownRows; i += 64) mine[i] = 0.0f;
    if (first < end) {
        int i = first;
        for (; i + 2 < end; i += 2) {
            get_x(x1, a1);
            const Entry e0 = entry(i + 2);
            compute(w0, x0, a0);
            a0 = at_step(e0);
            get_w(w0, a0);
            get_x(x0, a0);
            const Entry e1 = entry(i + 3);
            compute(w1, x1, a1);
            a1 = at_step(e1);
            get_w(w1, a1);
        }
        const bool two = i + 1 < end;
        if (two) get_x(x1, a1);
        compute(w0, x0, a0);
        if (two) compute(w1, x1, a1);
    }
    __syncthreads();
    uint32_t nonfinite = 0;
    const int rows = min(p.hidden - row0, kDownRows);
    const auto put = [&](int t, int r, float v) {
        const uint16_t h = gemm::to_bf16(v);
        nonfinite += (h & 0x7F80u) == 0x7F80u;
        p.y[t * p.ldy + row0 + r] = h;
    };
    for (int i = threadIdx.x; i < p.tokens * kDownRows; i += kDownThreads) {
        const int t = i / kDownRows, r = i % kDownRows;
        float s = ysum[i];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) s += ysum[w * p.tokens * kDownRows + i];
        if (r >= rows) continue;
        if (p.shares == 1)
            put(t, r, s);
        else
            agent_store(p.part + ((int64_t)share * p.tokens + t) * p.hidden + row0 + r, s);
    }
    if (p.shares > 1) {
        if (!last_of(p.arrived_rows + block, (uint32_t)p.shares)) return;
        // all reads of 8 outputs a thread (of 64 tokens) in flight at once
        constexpr int kAt = kMoeMaxTokens * kDownRows / kDownThreads;
        const int r = threadIdx.x % kDownRows, t0 = threadIdx.x / kDownRows;
        constexpr int kApart = kDownThreads / kDownRows;
        const float* from = p.part + row0 + min(r, rows - 1);
        float v[kAt];
#pragma unroll
        for (int i = 0; i < kAt; ++i) v[i] = 0.0f;
        for (int j0 = 0; j0 < p.shares; j0 += 4) {
            float w[kAt][4];
#pragma unroll
            for (int i = 0; i < kAt; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + kApart * i < p.tokens && j0 + j < p.shares)
                        w[i][j] = agent_load(from + ((int64_t)(j0 + j) * p.tokens + t0 + kApart * i) * p.hidden);
                    else
                        w[i][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kAt; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i] += w[i][j];
        }
#pragma unroll
        for (int i = 0; i < kAt; ++i)
            if (t0 + kApart * i < p.tokens && r < rows) put(t0 + kApart * i, r, v[i]);
    }
    flush_counters(p.ctr, 0, 0, 0, nonfinite);
}

// Rows of y a workgroup takes: 64, which halves the reads of the columns, from 64
// wave steps of such a workgroup a CU on.  The layer, us, the chosen one first:
//   1 token, 8 of 64 experts of 2048 x 1408      32: 26.4    64: 29.5
//   64 tokens, 4 of 64 of 1024 x 700             32: 41.5    64: 49.1
//   8 tokens, 8 of 128 of 4096 x 1024            64: 83.5    32: 86.7
//   64 tokens, 8 of 128 of 4096 x 1024           64: 203     32: 217
constexpr int kDownRowsFew = 32, kDownRowsMany = 64;
int down_rows(int64_t tokens, int64_t top_k, int64_t hidden, int64_t inner)
{
    const int64_t steps = tokens * top_k * ((inner + kUnit - 1) / kUnit) * ((hidden + 63) / 64);
    return steps < 64 * (int64_t)gemm_num_cus() ? kDownRowsFew : kDownRowsMany;
}

// Workgroups that share a row block of y: enough for one on each CU,
// of two steps a wave at least.  (64 tokens, 128 experts of 4096 x 1024: 213
// us with 3, 197 with 4, 203 with 8; one token of 2048 x 1408: 26.6 with 4, 28.2
// with 8.)
int down_shares(int64_t tokens, int64_t top_k, int64_t hidden, int64_t inner, int64_t rows)
{
    const int64_t blocks = (hidden + rows - 1) / rows;
    const int64_t steps = tokens * top_k * ((inner + kUnit - 1) / kUnit);
    return (int)std::clamp<int64_t>(std::min((gemm_num_cus() + blocks - 1) / blocks, steps / (2 * kDownWaves)), 1, kMaxShares);
}

// K splits of the router: one round of reads a wave, as far as the partial sums
// of 16 tokens, which one workgroup reads, stay under 64 KB (64 tokens, 128
// experts of 4096: 4 splits, the launch 2 us shorter than with 8).
constexpr int64_t kSplitBytes = 65536;
int route_splits(int64_t tokens, int64_t experts, int64_t hidden)
{
    const int64_t chunks = (hidden + kChunk - 1) / kChunk, bytes = std::min<int64_t>(tokens, 16) * experts * 8;
    return (int)std::clamp<int64_t>(std::min((chunks + kRouteWaves - 1) / kRouteWaves, kSplitBytes / bytes), 1, kMaxSplits);
}

struct MoeLayout {
    size_t arrived_rows, logits, xq, count, up_groups, groups, prob, aq, part, total;
    int64_t max_up_groups, max_groups;
};
// Most groups of `size` tokens: an expert's last may be short.
int64_t most_groups(int64_t pairs, int64_t experts, int64_t size)
{
    return std::min(pairs, std::min(pairs, experts) + pairs / size);
}
MoeLayout moe_layout(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inner)
{
    const auto up = [](int64_t v, int64_t a) { return (v + a - 1) / a * a; };
    const int64_t hp = up(hidden, mx4::kPanel), ip = up(inner, mx4::kPanel), pairs = tokens * top_k;
    MoeLayout m;
    int64_t at = 256;                                       // arrival counts
    const auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at = up(at + bytes, 256);
        return (size_t)o;
    };
    m.arrived_rows = take((hidden + kDownRowsFew - 1) / kDownRowsFew * 4);
    // fewer tokens may take more splits, in as many bytes
    m.logits = take(std::max<int64_t>(kSplitBytes, route_splits(tokens, experts, hidden) * tokens * experts * 8));
    m.xq = take(tokens * hp * 2);
    m.count = take(8);
    m.max_up_groups = most_groups(pairs, experts, kUpTokens);
    m.max_groups = most_groups(pairs, experts, kDownTokens);
    m.up_groups = take(m.max_up_groups * (int64_t)sizeof(MoeGroup));
    m.groups = take(m.max_groups * (int64_t)sizeof(MoeGroup));
    m.prob = take(pairs * 4);
    m.aq = take(pairs * kPieces * ip * 2);
    m.part = take(kMaxShares * tokens * hidden * 4);
    m.total = (size_t)at;
    return m;
}

}  // namespace

size_t mx4_moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inner)
{
    return moe_layout(tokens, experts, top_k, hidden, inner).total;
}

int64_t mx4_moe_items(int64_t tokens, int64_t experts, int64_t top_k, int64_t inner)
{
    return most_groups(tokens * top_k, experts, kUpTokens) * ((inner + 31) / 32) * kUpThreads;
}

hipError_t launch_mx4_moe(const Mx4MoeArgs& g, hipStream_t stream)
{
    if (g.tokens == 0) return hipSuccess;
    const MoeLayout m = moe_layout(g.tokens, g.experts, g.top_k, g.hidden, g.inner);
    uint8_t* ws = static_cast<uint8_t*>(g.ws);
    MoeArgs p;
    p.x = static_cast<const uint16_t*>(g.x);
    p.ldx = g.ldx;
    p.router = static_cast<const uint16_t*>(g.router);
    p.ldr = g.ldr;
    p.tokens = (int)g.tokens;
    p.experts = (int)g.experts;
    p.top_k = (int)g.top_k;
    p.hidden = (int)g.hidden;
    p.inner = (int)g.inner;
    p.renormalize = g.renormalize;
    p.hp = (int)((g.hidden + mx4::kPanel - 1) / mx4::kPanel * mx4::kPanel);
    p.ip = (int)((g.inner + mx4::kPanel - 1) / mx4::kPanel * mx4::kPanel);
    p.q1 = g.w1.q;
    p.s1 = g.w1.s;
    p.ldq1 = g.w1.ldq;
    p.eq1 = g.w1.eq;
    p.ps1 = g.w1.ps;
    p.es1 = g.w1.es;
    p.q2 = g.w2.q;
    p.s2 = g.w2.s;
    p.ldq2 = g.w2.ldq;
    p.eq2 = g.w2.eq;
    p.ps2 = g.w2.ps;
    p.es2 = g.w2.es;
    p.y = static_cast<uint16_t*>(g.y);
    p.ldy = g.ldy;
    p.ids = g.ids;
    p.weights = g.weights;
    p.arrived = reinterpret_cast<uint32_t*>(ws);
    p.logits = reinterpret_cast<double*>(ws + m.logits);
    p.xq = reinterpret_cast<uint16_t*>(ws + m.xq);
    p.count = reinterpret_cast<int32_t*>(ws + m.count);
    p.up_groups = reinterpret_cast<MoeGroup*>(ws + m.up_groups);
    p.max_up_groups = (int)m.max_up_groups;
    p.groups = reinterpret_cast<MoeGroup*>(ws + m.groups);
    p.max_groups = (int)m.max_groups;
    p.prob = reinterpret_cast<float*>(ws + m.prob);
    p.part = reinterpret_cast<float*>(ws + m.part);
    p.arrived_rows = reinterpret_cast<uint32_t*>(ws + m.arrived_rows);
    const int rows = down_rows(g.tokens, g.top_k, g.hidden, g.inner);
    p.shares = down_shares(g.tokens, g.top_k, g.hidden, g.inner, rows);
    p.aq = reinterpret_cast<uint16_t*>(ws + m.aq);
    p.ctr = g.ctr;
    p.tiles_e = (p.experts + 15) / 16;
    p.tiles_t = (p.tokens + 15) / 16;
    p.splits = route_splits(g.tokens, g.experts, g.hidden);

    const int items = p.tokens * ((p.hp + mx4::kPanel - 1) / mx4::kPanel);
    const int route = p.tiles_e * p.tiles_t * p.splits + (items + kRouteWaves - 1) / kRouteWaves;
    hipLaunchKernelGGL(k_moe_route, dim3(route), dim3(kRouteThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_moe_up, dim3(p.max_up_groups * ((p.inner + 31) / 32)), dim3(kUpThreads), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int lds = kDownWaves * p.tokens * rows * 4;
    const int blocks = (p.hidden + rows - 1) / rows;
    const auto kernel = rows == kDownRowsFew ? k_moe_down<kDownRowsFew / 16> : k_moe_down<kDownRowsMany / 16>;
    if (rows == kDownRowsMany) {
        static mx4::LdsLimit limit;
        e = limit.raise(reinterpret_cast<const void*>(kernel), kDownWaves * kMoeMaxTokens * kDownRowsMany * 4);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(blocks * p.shares), dim3(kDownThreads), lds, stream, p);
    return hipGetLastError();
}

}  // namespace fp8mi

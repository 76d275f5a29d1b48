// The router of a mixture-of-experts layer: logits l = x R^T, scores, and the k best experts of every token.
//
// Which expert a token goes to is a whole number, so the logits are summed in 64 bits: products of fp16 numbers are exact
// there and the sum's rounding (2^-53 of its terms) stays below any gap between two different logits that matters; the choice
// then depends neither on the batch nor on how the sum is split.  Equal logits (equal rows of R) tie, and the
// lower index wins.
//
// route_logits_kernel: tiles of 16 experts x 16 tokens on the 64-bit matrix instruction; a wave takes every fourth step of
// 32 inputs of its workgroup's share of them, and the shares' sums go to the workspace.
// route_pick_kernel: a wave a token adds the shares in order, scores them, and takes the largest score k times.
#include <algorithm>

#include "aqlm_device.h"
#include "moe_launch.h"

namespace aqlm {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16, kWaves = 4, kStep = 32, kAhead = 4;

__global__ __launch_bounds__(kWaves* kWave) void route_logits_kernel(const f16* __restrict__ x, const f16* __restrict__ r,
                                                                     double* __restrict__ part, int in, int T, int E,
                                                                     int tiles_e, int tiles_t, int splits) {
    __shared__ double red[kWaves][kTile * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int e0 = ((int)blockIdx.x % tiles_e) * kTile;
    const int t0 = ((int)blockIdx.x / tiles_e % tiles_t) * kTile;
    const int split = (int)blockIdx.x / tiles_e / tiles_t;
    const int steps = (in + kStep - 1) / kStep;
    const f16* rr = r + (size_t)min(e0 + (lane & 15), E - 1) * in;
    const f16* xr = x + (size_t)min(t0 + (lane & 15), T - 1) * in;
    f64x4 acc = {0., 0., 0., 0.};
    const int stride = splits * kWaves;
    for (int s0 = split * kWaves + wave; s0 < steps; s0 += kAhead * stride) {   // kAhead steps' loads in flight
        f16x8 a[kAhead], b[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int at = min((s0 + q * stride) * kStep + 8 * (lane >> 4), in - 8);
            a[q] = as_f16x8(load16(rr + at));
            b[q] = as_f16x8(load16(xr + at));
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            // in % 8 == 0: a lane's 8 inputs are inside or outside together
            const bool in_row = (s0 + q * stride) * kStep + 8 * (lane >> 4) < in;
            a[q] = in_row ? a[q] : f16x8{};
            b[q] = in_row ? b[q] : f16x8{};
            if (s0 + q * stride >= steps) break;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)a[q][i], (double)b[q][i], acc, 0, 0, 0);
        }
    }
    // lane l holds rows l / 16 + 4 i of column l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(lane & 15) * kTile + (lane >> 4) + 4 * i] = acc[i];
    __syncthreads();
    const int t = threadIdx.x / kTile, e = threadIdx.x % kTile;
    if (t0 + t < T && e0 + e < E) {
        double v = 0.;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += red[w][t * kTile + e];
        part[((size_t)split * T + t0 + t) * E + e0 + e] = v;
    }
}

// Scores as whole numbers in the same order; NaN below everything, 0 for experts already taken.
__device__ __forceinline__ uint64_t rank_key(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v);
    return v != v ? 1ull : b < 0 ? ~(uint64_t)b : (uint64_t)b | (1ull << 63);
}

template <int CTRL>
__device__ __forceinline__ uint64_t max_dpp(uint64_t v) {   // lanes without a source keep their own value
    const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
    const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp((int)lo, (int)lo, CTRL, 0xf, 0xf, false);
    const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp((int)hi, (int)hi, CTRL, 0xf, 0xf, false);
    return max(v, (uint64_t)h << 32 | l);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    v = max_dpp<0x111>(v);   // from 1, 2, 4, 8 lanes below in a row of 16
    v = max_dpp<0x112>(v);
    v = max_dpp<0x114>(v);
    v = max_dpp<0x118>(v);
    v = max_dpp<0x142>(v);   // the last lane of a row to the next row
    v = max_dpp<0x143>(v);   // lane 31 to the upper half
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// N: experts a lane holds (expert lane + 64 j).
template <int N>
__global__ __launch_bounds__(kWaves* kWave) void route_pick_kernel(const double* __restrict__ part,
                                                                   const float* __restrict__ bias,
                                                                   int32_t* __restrict__ ids, float* __restrict__ weights,
                                                                   int T, int E, int splits, int k, int score, int renorm,
                                                                   float scale) {
    const int lane = threadIdx.x & 63;
    const int t = (int)blockIdx.x * kWaves + (int)threadIdx.x / 64;
    if (t >= T) return;   // whole waves
    double v[N];
    uint64_t key[N];
    const double kInf = __builtin_inf();
    constexpr int kParts = N == 1 ? 8 : 4;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 64 * j;
        v[j] = e < E ? 0. : -kInf;
        if (e < E) {
            for (int s0 = 0; s0 < splits; s0 += kParts) {   // kParts loads in flight
                double d[kParts];
#pragma unroll
                for (int s = 0; s < kParts; ++s) d[s] = part[((size_t)min(s0 + s, splits - 1) * T + t) * E + e];
#pragma unroll
                for (int s = 0; s < kParts; ++s)
                    if (s0 + s < splits) v[j] += d[s];
            }
        }
        key[j] = e < E ? rank_key(v[j]) : 0ull;
    }
    if (score == kScoreSoftmax) {
        uint64_t m = key[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = max(m, key[j]);
        m = wave_max(m);
        // the largest logit back from its key (NaN where there is none)
        const double top = m <= 1 ? __builtin_nan("") : __builtin_bit_cast(double, m >> 63 ? m & ~(1ull << 63) : ~m);
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            v[j] = lane + 64 * j < E ? exp(v[j] - top) : 0.;
            sum += v[j];
        }
        const double total = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] /= total;
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 1. / (1. + exp(-v[j]));
    }
    if (score == kScoreSigmoid || bias != nullptr) {   // softmax keeps the order of the logits
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 64 * j;
            if (e < E) key[j] = rank_key(bias != nullptr ? v[j] + (double)bias[e] : v[j]);
        }
    }
    double mine = 0.;   // lane i keeps the i-th choice
    int id = 0;
    for (int i = 0; i < k; ++i) {
        uint64_t m = key[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = max(m, key[j]);
        m = wave_max(m);
        bool done = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t who = done ? 0ull : __ballot(key[j] == m);
            if (who != 0) {
                const int l = __builtin_ctzll(who);
                const double s = __shfl(v[j], l, 64);
                if (lane == i) {
                    mine = s;
                    id = l + 64 * j;
                }
                if (lane == l) key[j] = 0;
                done = true;
            }
        }
    }
    if (renorm) {
        const double total = wave_sum(lane < k ? mine : 0.);
        mine /= total;
    }
    if (lane < k) {
        ids[(size_t)t * k + lane] = id;
        weights[(size_t)t * k + lane] = (float)(mine * (double)scale);
    }
}

// Workgroups that fill the chip, by splitting the sums of small batches.
constexpr int kWantTiles = 128;
struct RoutePlan {
    int tiles_e, tiles_t, splits;
};
constexpr int kMaxSplits = 8;   // each a load more for the pick
int max_splits(int64_t in) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, in / (kStep * kWaves))); }
RoutePlan route_plan(int64_t experts, int64_t in, int64_t tokens) {
    RoutePlan p;
    p.tiles_e = (int)((experts + kTile - 1) / kTile);
    p.tiles_t = (int)((tokens + kTile - 1) / kTile);
    p.splits = std::max(1, std::min(max_splits(in), kWantTiles / p.tiles_e / p.tiles_t));
    return p;
}

}  // namespace

int64_t route_workspace(int64_t experts, int64_t in, int64_t tokens) {
    if (tokens == 0) return 0;
    const RoutePlan p = route_plan(experts, in, tokens);
    // splits * tiles_t grows with the batch up to its cap, so a larger batch never needs less
    const int64_t tiles = std::max<int64_t>(p.tiles_t, std::min<int64_t>((int64_t)max_splits(in) * p.tiles_t, kWantTiles / p.tiles_e));
    return tiles * kTile * experts * (int64_t)sizeof(double);
}

hipError_t launch_route(const RouteCall& c, void* workspace, hipStream_t stream) {
    const RoutePlan p = route_plan(c.experts, c.in, c.tokens);
    double* part = static_cast<double*>(workspace);
    hipLaunchKernelGGL(route_logits_kernel, dim3((unsigned)((int64_t)p.tiles_e * p.tiles_t * p.splits)), dim3(kWaves * kWave),
                       0, stream, static_cast<const f16*>(c.x), static_cast<const f16*>(c.router), part, (int)c.in,
                       (int)c.tokens, c.experts, p.tiles_e, p.tiles_t, p.splits);
    hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    const dim3 grid((unsigned)((c.tokens + kWaves - 1) / kWaves));
#define AQLM_PICK(N)                                                                                                   \
    hipLaunchKernelGGL(route_pick_kernel<N>, grid, dim3(kWaves * kWave), 0, stream, part, c.bias, c.ids, c.weights,       \
                       (int)c.tokens, c.experts, p.splits, c.k, c.score, c.renorm, c.scale)
    if (c.experts <= 64) AQLM_PICK(1);
    else if (c.experts <= 128) AQLM_PICK(2);
    else if (c.experts <= 256) AQLM_PICK(4);
    else AQLM_PICK(8);
#undef AQLM_PICK
    return hipGetLastError();
}

}  // namespace aqlm

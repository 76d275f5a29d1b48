// The router of a mixture-of-experts layer: logits l = x R^T, scores, and the k best experts of every token.
//
// Which expert a token goes to is a whole number, so the logits are summed in 64 bits: products of fp16 numbers are exact
// there and the sum's rounding (2^-53 of its terms) stays below any gap between two different logits that matters; the choice
// then depends neither on the batch nor on how the sum is split.  Equal logits (equal rows of R) tie, and the
// lower index wins.
//
// Few tokens, route_logits_kernel: tiles of 16 experts x 16 tokens on the 64-bit matrix instruction; a wave takes every
// fourth step of 32 inputs of its workgroup's share of them, and the shares' sums go to the workspace.
// route_pick_kernel: a wave a token adds the shares in order, scores them, and takes the largest score k times.
//
// Many tokens: the 64-bit instruction would bound the time (256 experts, 4096 inputs, 2048 tokens: 55 us of 102 at its peak).
// route_fast_kernel multiplies on the fp16 instruction and adds its fp32 sums in 64 bits every 64 inputs.  A sum of 64 products
// p in fp32 is off by at most 64 2^-23 sum |p|, so a logit by at most eb = 2^-17 |x| |r|.  The pick then knows which of its
// comparisons eb could turn, and computes those logits again in 64 bits (one token in ten, two or three logits): the choice is
// the same.  Weights come from the faster sums: their error against 64 bits is within 4 % of that of an fp32 number's rounding
// (2.9e-8 against 2.8e-8, relative, 2048 tokens), at most 2^-22.  All chosen logits in 64 bits too took 62 us instead of 47
// (2048 tokens, k 8), 132 instead of 72 (3000, 512 experts of 2048 inputs, k 16), 148 instead of 111 (8192).  Not for softmax scores with a bias, whose
// comparisons need every logit of a token.  Together 48 us: the product 20 (134 MB through LDS), the pick 26, of which the
// last token's exact logits are 10.
#include <algorithm>

#include "act_launch.h"
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

// 64 experts x 64 tokens a workgroup, 32 x 32 a wave.  Blocks of 64 inputs go through a ring of kStages in LDS, loaded
// there directly; the 16-byte chunk c of a row lies at c ^ (row & 7), so that 16 rows are read without conflicts.
constexpr int kFastTile = 64, kFastSteps = 2;   // steps of 32 inputs that fp32 adds
constexpr int kStages = 5, kStageBytes = 2 * kFastTile * 128, kFastLoads = kStageBytes / 1024 / kWaves;

__global__ __launch_bounds__(kWaves* kWave) void route_fast_kernel(const f16* __restrict__ x, const f16* __restrict__ r,
                                                                   double* __restrict__ part, float* __restrict__ xn,
                                                                   float* __restrict__ rn, int in, int T, int E, int tiles_e,
                                                                   int tiles_t, int splits) {
    __shared__ __attribute__((aligned(16))) uint8_t ring[kStages * kStageBytes];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int id = xcd_run((int)blockIdx.x, (int)gridDim.x);   // tiles of the same tokens on one XCD
    const int te = id % tiles_e, split = id / tiles_e % splits, tt = id / tiles_e / splits;
    const int blocks = (in + 63) / 64, per = (blocks + splits - 1) / splits;
    const int b0 = split * per, b1 = min(b0 + per, blocks);
    // Waves 0 and 1 load experts, 2 and 3 tokens: 8 rows of 128 bytes at a time.
    const bool of_x = wave >= 2;
    const int first = of_x ? tt * kFastTile : te * kFastTile, rows = of_x ? T : E;
    const f16* base = (of_x ? x : r) + (size_t)first * in;
    uint32_t row_at[kFastLoads];
#pragma unroll
    for (int i = 0; i < kFastLoads; ++i)
        row_at[i] = (uint32_t)min((wave & 1) * 32 + i * 8 + (lane >> 3), rows - 1 - first) * (uint32_t)in * 2u;
    const int chunk = (lane & 7) ^ (lane >> 3);
    const uint32_t lds0 = lds_address(ring);
    auto load = [&](int blk) {
        const uint32_t at = (uint32_t)min(blk * 64 + 8 * chunk, in - 8) * 2u;
        const uint32_t to = lds0 + (uint32_t)((blk - b0) % kStages * kStageBytes + wave * kFastLoads * 1024);
#pragma unroll
        for (int i = 0; i < kFastLoads; ++i) load_to_lds(to + i * 1024, base, row_at[i] + at);
    };
    f64x4 acc[2][2];
    float n2[2][2] = {{0.f, 0.f}, {0.f, 0.f}};   // sums of squares of the lane's inputs: of experts, of tokens
    const bool norm_r = tt == 0 && wave < 2, norm_x = te == 0 && (wave & 1) == 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f64x4{0., 0., 0., 0.};
    auto squares = [](const f16x8 v) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += (float)v[q] * (float)v[q];
        return s;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(b0 + s);
    for (int blk = b0; blk < b1; ++blk) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kFastLoads * (kStages - 2)) : "memory");
        load(blk + kStages - 1);   // over the block that every wave has read; behind the last block nothing uses it
        const uint8_t* at = ring + (blk - b0) % kStages * kStageBytes;
        f32x4 c[2][2] = {};
#pragma unroll
        for (int s = 0; s < kFastSteps; ++s) {
            const bool in_row = blk * 64 + s * 32 + 8 * (lane >> 4) < in;   // in % 8 == 0
            f16x8 a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ra = (wave & 1) * 32 + 16 * i + (lane & 15), rb = kFastTile + (wave >> 1) * 32 + 16 * i + (lane & 15);
                const int to = ((s * 4 + (lane >> 4)) ^ (lane & 7)) * 16;
                a[i] = *reinterpret_cast<const f16x8*>(at + ra * 128 + to);
                b[i] = *reinterpret_cast<const f16x8*>(at + rb * 128 + to);
                a[i] = in_row ? a[i] : f16x8{};
                b[i] = in_row ? b[i] : f16x8{};
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) c[i][j] = mfma16x16x32(a[i], b[j], c[i][j]);
            if (norm_r)
#pragma unroll
                for (int i = 0; i < 2; ++i) n2[0][i] += squares(a[i]);
            if (norm_x)
#pragma unroll
                for (int i = 0; i < 2; ++i) n2[1][i] += squares(b[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] += (double)c[i][j][q];
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the workgroup's LDS is given up with no load on its way
    const int e0 = te * kFastTile + (wave & 1) * 32, t0 = tt * kFastTile + (wave >> 1) * 32;
    // lane l holds experts 4 (l / 16) + q of token l % 16
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = t0 + 16 * j + (lane & 15), e = e0 + 16 * i + 4 * (lane >> 4);
            double* to = part + ((size_t)split * T + t) * E + e;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t < T && e + q < E) to[q] = acc[i][j][q];
        }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float s = n2[w][i];
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            const int at = (w ? t0 : e0) + 16 * i + (lane & 15);
            if (lane < 16 && w == 0 && norm_r && at < E) rn[(size_t)split * E + at] = s;
            if (lane < 16 && w == 1 && norm_x && at < T) xn[(size_t)split * T + at] = s;
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

// x . r[e_i] in 64 bits by a wave; every lane gets them.
// Rows at once, steps with their loads in flight: mostly two are wanted, and a token that wants more waits for memory again
// (2048 tokens of 256 experts: the pick 26 us, with 4 rows 28, with 3 rows of 2 steps 30).
constexpr int kExact = 2, kExactSteps = 4;
__device__ __forceinline__ void exact_logits(const f16* __restrict__ x, const f16* __restrict__ r, const int (&e)[kExact], int in,
                                             int lane, double (&s)[kExact]) {
#pragma unroll
    for (int i = 0; i < kExact; ++i) s[i] = 0.;
    for (int k0 = 8 * lane; k0 < in; k0 += kExactSteps * 512) {
        f16x8 a[kExactSteps], b[kExactSteps][kExact];
#pragma unroll
        for (int u = 0; u < kExactSteps; ++u) {
            const int k = min(k0 + 512 * u, in - 8);
            a[u] = as_f16x8(load16(x + k));
#pragma unroll
            for (int i = 0; i < kExact; ++i) b[u][i] = as_f16x8(load16(r + (size_t)e[i] * in + k));
        }
        __builtin_amdgcn_sched_barrier(0);   // the loads stay in front
#pragma unroll
        for (int u = 0; u < kExactSteps; ++u) {
            const bool in_row = k0 + 512 * u < in;
            a[u] = in_row ? a[u] : f16x8{};
#pragma unroll
            for (int i = 0; i < kExact; ++i) {
                b[u][i] = in_row ? b[u][i] : f16x8{};
#pragma unroll
                for (int q = 0; q < 8; ++q) s[i] += (double)((float)a[u][q] * (float)b[u][i][q]);   // the product is exact in fp32
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kExact; ++i) s[i] = wave_sum(s[i]);
}

__device__ __forceinline__ double lane_value(double v, int l) {   // l uniform
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// What the pick needs to make sure of sums that may be off.
struct RouteCheck {
    const f16 *x, *r;
    const float *xn, *rn;   // [splits][tokens], [splits][experts]: sums of squares
    int in;
};

// N: experts a lane holds (expert lane + 64 j).  CHECK: the logits are route_fast_kernel's.
template <int N, bool CHECK>
__global__ __launch_bounds__(kWaves* kWave) void route_pick_kernel(const double* __restrict__ part,
                                                                   const float* __restrict__ bias,
                                                                   int32_t* __restrict__ ids, float* __restrict__ weights,
                                                                   int T, int E, int splits, int k, int score, int renorm,
                                                                   float scale, RouteCheck c) {
    const int lane = threadIdx.x & 63;
    const int t = (int)blockIdx.x * kWaves + (int)threadIdx.x / 64;
    if (t >= T) return;   // whole waves
    const double kInf = __builtin_inf();
    double v[N];   // logits
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
    }
    double eb = 0.;   // how far a logit may be off
    if (CHECK) {
        float r2 = 0.f, x2 = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float s = 0.f;
            if (lane + 64 * j < E)
                for (int q = 0; q < splits; ++q) s += c.rn[(size_t)q * E + lane + 64 * j];
            r2 = s > r2 || s != s ? s : r2;
        }
        for (int q = 0; q < splits; ++q) x2 += c.xn[(size_t)q * T + t];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const float s = __shfl_xor(r2, o, 64);
            r2 = s > r2 || s != s ? s : r2;
        }
        eb = 0x1.02p-17 * sqrt((double)x2) * sqrt((double)r2);   // the norms' own rounding included
        if (!(eb < kInf)) eb = kInf;   // a NaN or an infinity in the token or in any expert
    }
    double top = 0., total = 1.;   // softmax: the largest logit and the sum of exp(l - top)
    if (score == kScoreSoftmax) {
        uint64_t m = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) m = max(m, lane + 64 * j < E ? rank_key(v[j]) : 0ull);
        m = wave_max(m);
        // the largest logit back from its key (NaN where there is none)
        top = m <= 1 ? __builtin_nan("") : __builtin_bit_cast(double, m >> 63 ? m & ~(1ull << 63) : ~m);
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < N; ++j) sum += lane + 64 * j < E ? exp(v[j] - top) : 0.;
        total = wave_sum(sum);
    }
    auto score_of = [&](double l) { return score == kScoreSoftmax ? exp(l - top) / total : 1. / (1. + exp(-l)); };
    const bool by_logit = score == kScoreSoftmax && bias == nullptr;   // softmax keeps the order of the logits
    double rank[N], off[N];   // what is compared, and how far it may be off
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const double s = by_logit ? 0. : score_of(v[j]);
        rank[j] = by_logit ? v[j] : bias != nullptr && lane + 64 * j < E ? s + (double)bias[lane + 64 * j] : s;
        // The logistic function's slope is s (1 - s), and changes by less than a factor e^eb over eb; then the sum's rounding.
        // An infinite bias decides alone.
        off[j] = !CHECK || eb == 0. ? 0.
                 : by_logit         ? eb
                 : fabs(rank[j]) == kInf
                     ? 0.
                     : (eb < 1. ? 3. * eb * s * (1. - s) : 1.) + 0x1p-50 * (1. + (rank[j] == rank[j] ? fabs(rank[j]) : 0.));
    }
    double mine = 0.;   // lane i keeps the i-th choice's logit
    int id = 0;
    for (int round = 0;; ++round) {
        uint64_t key[N];
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = lane + 64 * j < E ? rank_key(rank[j]) : 0ull;
        double my_rank = 0., my_off = 0.;
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
                    const double lv = lane_value(v[j], l);
                    if (lane == i) {
                        mine = lv;
                        id = l + 64 * j;
                    }
                    if (CHECK) {
                        const double lr = lane_value(rank[j], l), lo = lane_value(off[j], l);
                        if (lane == i) {
                            my_rank = lr;
                            my_off = lo;
                        }
                    }
                    if (lane == l) key[j] = 0;
                    done = true;
                }
            }
        }
        if (!CHECK) break;
        // Comparisons that the errors could turn: neighbours among the chosen, and the last of them against all others.
        const double next_rank = __shfl_down(my_rank, 1, 64), next_off = __shfl_down(my_off, 1, 64);
        const bool close = lane + 1 < k && my_off + next_off > 0. && !(my_rank - next_rank > my_off + next_off);
        const uint64_t pairs = __ballot(close);
        const double last = lane_value(my_rank, k - 1), last_off = lane_value(my_off, k - 1);
        uint64_t again[N];   // a bit a lane: logits to be computed again
        uint64_t others = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            // key 0: among the chosen, or no expert
            again[j] = __ballot(key[j] != 0 && off[j] + last_off > 0. && !(last - rank[j] > off[j] + last_off));
            others |= again[j];
        }
        if ((pairs | others) == 0) break;
        const uint64_t chosen = pairs | pairs << 1 | (others != 0 ? 1ull << (k - 1) : 0ull);
        for (uint64_t w = chosen; w != 0; w &= w - 1) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(w));
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (e >> 6 == j) again[j] |= 1ull << (e & 63);
        }
        // After a few rounds (logits that are all alike) everything.  Exact ones are left; as one of every pair is not, the
        // rounds end.
#pragma unroll
        for (int j = 0; j < N; ++j) again[j] = (round >= 3 ? __ballot(lane + 64 * j < E) : again[j]) & __ballot(off[j] > 0.);
        for (;;) {
            int e[kExact], n = 0;
#pragma unroll
            for (int i = 0; i < kExact; ++i) {
                e[i] = i == 0 ? -1 : e[0];
                bool found = false;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (!found && again[j] != 0) {
                        e[i] = __builtin_ctzll(again[j]) + 64 * j;
                        again[j] &= again[j] - 1;
                        found = true;
                    }
                n += found;
            }
            if (n == 0) break;
            double s[kExact];
            exact_logits(c.x + (size_t)t * c.in, c.r, e, c.in, lane, s);
#pragma unroll
            for (int i = 0; i < kExact; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (e[i] == lane + 64 * j) {
                        v[j] = s[i];
                        off[j] = 0.;
                    }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const double s = by_logit ? v[j] : 1. / (1. + exp(-v[j]));
            if (off[j] == 0.) rank[j] = bias != nullptr && lane + 64 * j < E ? s + (double)bias[lane + 64 * j] : s;
        }
    }
    mine = score_of(mine);
    if (renorm) mine /= wave_sum(lane < k ? mine : 0.);
    if (lane < k) {
        ids[(size_t)t * k + lane] = id;
        weights[(size_t)t * k + lane] = (float)(mine * (double)scale);
    }
}

// Workgroups that fill the chip, by splitting the sums of small batches.
constexpr int kWantTiles = 128;
struct RoutePlan {
    bool fast;
    int tiles_e, tiles_t, splits;
};
constexpr int kMaxSplits = 8;   // each a load more for the pick
int max_splits(int64_t in) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, in / (kStep * kWaves))); }
// From here on route_fast_kernel: products of tokens, experts and inputs.  4096 inputs, 64 experts: 1024 tokens 28 us against
// 24 in 64 bits, 2048 tokens 30 against 36; 256 experts: 512 tokens 38 against 40, 1024 tokens 43 against 61.
constexpr int64_t kFastFrom = (int64_t)1 << 29;
constexpr int kFastMaxSplits = 4;
// Tokens of a launch: a grid has fewer than 2^32 threads, and 512 experts take 512 threads a token in 64 bits.
constexpr int64_t kLaunchTokens = (int64_t)1 << 22;
RoutePlan route_plan(int64_t experts, int64_t in, int64_t tokens, bool fast) {
    RoutePlan p;
    p.fast = fast;
    const int tile = p.fast ? kFastTile : kTile;
    p.tiles_e = (int)((experts + tile - 1) / tile);
    p.tiles_t = (int)((tokens + tile - 1) / tile);
    const int64_t tiles = (int64_t)p.tiles_e * p.tiles_t;
    if (p.fast) {
        const int64_t blocks = (in + 32 * kFastSteps - 1) / (32 * kFastSteps);
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({kFastMaxSplits, 512 / tiles, blocks / 8}));
        while (p.splits > 1 && (blocks + p.splits - 1) / p.splits * (p.splits - 1) >= blocks) --p.splits;   // no empty part
    } else {
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(max_splits(in), kWantTiles / tiles));
    }
    return p;
}

}  // namespace

int64_t route_workspace(int64_t experts, int64_t in, int64_t tokens) {
    if (tokens == 0) return 0;
    tokens = std::min(tokens, kLaunchTokens);   // parts of a larger batch take turns
    // Sums: splits * tokens * experts.  splits * tiles grows with the batch up to its cap and then with the batch alone, so
    // the larger of both bounds covers this batch and every smaller one.  Norms behind them.
    const int64_t te = (experts + kTile - 1) / kTile, tt = (tokens + kTile - 1) / kTile;
    const int64_t rows = kTile * std::max<int64_t>(tt, std::min<int64_t>(max_splits(in) * tt, kWantTiles / te));
    const int64_t fe = (experts + kFastTile - 1) / kFastTile, ft = (tokens + kFastTile - 1) / kFastTile;
    const int64_t fast_rows = kFastTile * std::max<int64_t>(ft, std::min<int64_t>(kFastMaxSplits * ft, 512 / fe));
    return std::max(rows, fast_rows) * experts * (int64_t)sizeof(double) + kFastMaxSplits * (tokens + experts) * (int64_t)sizeof(float);
}

namespace {

// The tokens of c, at most kLaunchTokens, by plan p.
hipError_t launch_part(const RouteCall& c, const RoutePlan& p, void* workspace, hipStream_t stream) {
    double* part = static_cast<double*>(workspace);
    const f16 *x = static_cast<const f16*>(c.x), *r = static_cast<const f16*>(c.router);
    const dim3 tiles((unsigned)((int64_t)p.tiles_e * p.tiles_t * p.splits));
    RouteCheck check = {};
    if (p.fast) {
        float* xn = reinterpret_cast<float*>(part + (int64_t)p.splits * c.tokens * c.experts);
        float* rn = xn + (int64_t)p.splits * c.tokens;
        check = RouteCheck{x, r, xn, rn, (int)c.in};
        hipLaunchKernelGGL(route_fast_kernel, tiles, dim3(kWaves * kWave), 0, stream, x, r, part, xn, rn, (int)c.in, (int)c.tokens,
                           c.experts, p.tiles_e, p.tiles_t, p.splits);
    } else {
        hipLaunchKernelGGL(route_logits_kernel, tiles, dim3(kWaves * kWave), 0, stream, x, r, part, (int)c.in, (int)c.tokens, c.experts,
                           p.tiles_e, p.tiles_t, p.splits);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid((unsigned)((c.tokens + kWaves - 1) / kWaves));
#define AQLM_PICK(N)                                                                                                   \
    hipLaunchKernelGGL((p.fast ? route_pick_kernel<N, true> : route_pick_kernel<N, false>), grid, dim3(kWaves * kWave), 0,  \
                       stream, part, c.bias, c.ids, c.weights, (int)c.tokens, c.experts, p.splits, c.k, c.score, c.renorm,  \
                       c.scale, check)
    if (c.experts <= 64) AQLM_PICK(1);
    else if (c.experts <= 128) AQLM_PICK(2);
    else if (c.experts <= 256) AQLM_PICK(4);
    else AQLM_PICK(8);
#undef AQLM_PICK
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteCall& c, void* workspace, hipStream_t stream) {
    // for all parts of the batch alike; softmax scores with a bias compare sums over all logits
    const bool fast = (c.score == kScoreSigmoid || c.bias == nullptr) && c.tokens * c.experts * c.in >= kFastFrom;
    for (int64_t t = 0; t < c.tokens; t += kLaunchTokens) {
        RouteCall part = c;
        part.tokens = std::min(kLaunchTokens, c.tokens - t);
        part.x = static_cast<const f16*>(c.x) + t * c.in;
        part.ids = c.ids + t * c.k;
        part.weights = c.weights + t * c.k;
        const hipError_t e = launch_part(part, route_plan(c.experts, c.in, part.tokens, fast), workspace, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace aqlm

// How a mixture-of-experts launch finds its work (device helpers).
//
// Which experts are asked for, and by whom, is known on the device only.  Every workgroup sorts the layer's pairs (token,
// choice) by expert in its LDS, at most 1024 of them: it counts each expert's, and finds the pairs of the items that it takes by a
// vote of 64 lanes at a time.  A launch of its own would take two microseconds.  Up to `chunk` pairs of one expert are an item: its
// weights are read once for them.  chunk is what the kernel has columns for, whatever tokens they belong to: a token may name an
// expert more than once, so an expert can have more pairs than there are tokens.  Items are cut into `parts` so that parts x items
// fill the launch's workgroups evenly.
#pragma once
#include "aqlm_device.h"
#include "moe_launch.h"

namespace aqlm {

constexpr uint32_t kMoeNone = 0xffff;   // an id that is no expert
constexpr int kMoeIdBits = 9;
static_assert(kMoeMaxExperts <= 1 << kMoeIdBits, "bits of an id");

struct MoeLds {
    int count[kMoeMaxExperts];
    int item0[kMoeMaxExperts + 1];   // first item of an expert
    uint16_t id[kMoeMaxPairs];       // the expert of a pair, or kMoeNone
    int expert;                      // of the item at hand
    uint16_t x[16], y[16];           // its columns: rows of the input, pairs
};

// What a workgroup knows about the items.  few: at most FEW pairs, and no expert has more than an item takes, so every expert that is
// asked for is one item; lane p of each wave then holds pair p: its expert, the pairs of the same expert, and (all lanes) the first pair of each expert.
struct MoeItems {
    int n;
    bool few;
    uint32_t expert;
    uint64_t same, firsts;
};

// The lanes whose e equals this lane's, by a vote on each of its bits, among those with an expert.
__device__ __forceinline__ uint64_t same_expert(uint32_t e) {
    uint64_t same = __ballot(e != kMoeNone);
#pragma unroll
    for (int b = 0; b < kMoeIdBits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1u);
        same &= (e >> b) & 1u ? set : ~set;
    }
    return same;
}

// Counts the pairs.  All threads of the workgroup (at least 512) call it.  A pair whose id is no expert is left out.
template <int FEW>
__device__ __forceinline__ MoeItems moe_items(const int32_t* __restrict__ ids, int pairs, int experts, int chunk, MoeLds& m) {
    static_assert(FEW <= kWave, "a lane a pair");
    if (pairs <= FEW) {
        const int lane = threadIdx.x & (kWave - 1);
        const int id = ids[min(lane, pairs - 1)];
        const uint32_t e = lane < pairs && id >= 0 && id < experts ? (uint32_t)id : kMoeNone;
        const uint64_t same = same_expert(e);
        const uint64_t firsts = __ballot(e != kMoeNone && __builtin_ctzll(same | 1ull << 63) == lane);
        // all waves read the same ids: the workgroup goes one way
        if (pairs <= chunk || __ballot(e != kMoeNone && __popcll(same) > chunk) == 0)
            return MoeItems{(int)__popcll(firsts), true, e, same, firsts};
    }
    const int tid = threadIdx.x, n = blockDim.x;
    if (tid < kMoeMaxExperts) m.count[tid] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += n) {
        const int e = ids[p];
        const bool some = e >= 0 && e < experts;
        m.id[p] = (uint16_t)(some ? e : kMoeNone);
        if (some) atomicAdd(&m.count[e], 1);   // whole numbers: in any order the same
    }
    __syncthreads();
    if (tid < kWave) {
        constexpr int kPer = kMoeMaxExperts / kWave;
        const uint32_t inverse = 65536u / (uint32_t)chunk + 1u;   // n inverse >> 16 is n / chunk for n < 1040, chunk <= 16
        int c[kPer], items = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            c[i] = (int)((uint32_t)(m.count[tid * kPer + i] + chunk - 1) * inverse >> 16);
            items += c[i];
        }
        int t = items;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int to = __shfl_up(t, o, kWave);
            t += tid >= o ? to : 0;
        }
        if (tid == kWave - 1) m.item0[kMoeMaxExperts] = t;
        t -= items;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            m.item0[tid * kPer + i] = t;
            t += c[i];
        }
    }
    __syncthreads();
    return MoeItems{__builtin_amdgcn_readfirstlane(m.item0[kMoeMaxExperts]), false, 0u, 0ull, 0ull};
}

// Parts an item is cut into: `rounds` rounds of `wgs` workgroups take n * parts <= rounds * wgs units, each 1 / parts of an
// item and the fixed cost `fixed` (in items) of starting on one.
__device__ __forceinline__ int moe_parts(int n, int wgs, int most, float fixed) {
    int best = 1;
    float cost = (float)((n + wgs - 1) / wgs) * (1.f + fixed);
    for (int r = 1; r <= 4; ++r) {
        const int p = min(r * wgs / max(n, 1), most);
        if (p < 1) continue;
        const float c = (float)((n * p + wgs - 1) / wgs) * (1.f / (float)p + fixed);
        if (c < cost) {
            cost = c;
            best = p;
        }
    }
    return best;
}

// Makes item v the one at hand: its expert e, and m.x (rows of the input) and m.y (pairs) for its pairs; returns how
// many there are.  An expert's pairs keep their order: workgroups that take parts of one item must agree on its pairs.  PAIRED: the
// input has two rows for a pair (2 pair, 2 pair + 1), else one for its token.  chunk: as for moe_items.  Ends with a barrier.
template <bool PAIRED>
__device__ __forceinline__ int moe_item(const MoeItems& items, int v, int pairs, int k, int chunk, MoeLds& m, int& e) {
    const int tid = threadIdx.x;
    int n;
    auto keep = [&](int place, int p) {
        m.y[place] = (uint16_t)p;
        if constexpr (PAIRED) {
            m.x[2 * place] = (uint16_t)(2 * p);
            m.x[2 * place + 1] = (uint16_t)(2 * p + 1);
        } else {
            m.x[place] = (uint16_t)(p / k);
        }
    };
    const int lane = tid & (kWave - 1);
    const uint64_t below = (1ull << lane) - 1ull;
    __syncthreads();
    if (items.few) {
        const uint64_t first = __ballot((items.firsts >> lane & 1ull) && __popcll(items.firsts & below) == v);
        const int l = __builtin_ctzll(first);
        e = __builtin_amdgcn_readlane((int)items.expert, l);
        const uint64_t same = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(items.same >> 32), l) << 32 |
                              (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)items.same, l);
        n = __popcll(same);
        if (tid < kWave && (same >> lane & 1ull)) keep(__popcll(same & below), lane);
    } else {
        if (tid < kMoeMaxExperts && m.item0[tid] <= v && v < m.item0[tid + 1]) m.expert = tid;
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(m.expert);
        const int from = __builtin_amdgcn_readfirstlane((v - m.item0[e]) * chunk);   // the item's first pair among the expert's
        n = min(chunk, m.count[e] - from);
        if (tid < kWave) {
            int before = 0;   // of the expert's pairs
            for (int p0 = 0; p0 < pairs && before < from + n; p0 += kWave) {
                const bool mine = p0 + lane < pairs && m.id[p0 + lane] == e;
                const uint64_t same = __ballot(mine);
                const int place = before + __popcll(same & below) - from;
                if (mine && place >= 0 && place < n) keep(place, p0 + lane);
                before += __popcll(same);
            }
        }
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(n);
}

}  // namespace aqlm

// A workgroup's part of a product of MX4 rows with up to 64 columns of activations: mx4_linear.hip describes the kernel
// that it carries; the mixture-of-experts layer (moe_mx4.hip) runs it on experts.
//
// The workgroup walks tiles of 16 matrix-core rows in groups of TILES: tiles bid + i nwg.  Its 8 waves share the
// inputs: wave w takes NK steps of 128 inputs (a block for each quarter of a wave) out of every chunk of 8 NK, with their activations in registers for all tiles
// of the group.  What a step has used is loaded again at once for the next chunk or group, so that loads are a whole round
// ahead.  The waves' partial tiles are added in LDS in the order of the waves.
//
// Past a workgroup's last tile nothing is loaded: loads that repeat a tile cost what others do (8192 -> 28672, 7 tiles a workgroup in
// groups of 4, 1 token: 27.6 us, with an eighth load repeated 29.9; in groups of 6, with 12 instead of 7, 41).
#pragma once
#include <type_traits>

#include "hidden_pair.h"
#include "mx4.h"

namespace aqlm {

constexpr int kMxWaves = 8;
constexpr int kMxThreads = kMxWaves * kWave;
// Tiles of a group: the codes of this many are in flight.  Four column tiles leave registers for two.
constexpr int mx4_tiles(int ct) { return ct == 4 ? 2 : 4; }
constexpr int kMxRows = 16;       // matrix-core rows of a tile

// WIDE (rows of at least kMxWideBlocks blocks; else NK = 1): a wave loads the 16 scale bytes of its steps' blocks at once, the same
// for the lanes of a row, and each lane takes its byte out where it is used; in front of a row's end 16 bytes earlier, moved back
// then.  A byte a lane and step takes as many cache lines as the codes do.  Bytes | wide: 28672x8192 at 1 token 34 | 29 us,
// 32 experts 2048x1056 at 40 tokens 51 | 49.
constexpr int kMxWideBlocks = 16;

// How the inputs are dealt to the waves: `chunks` of kMxWaves nk steps, nk <= nk_max (the kernel's NK).
struct MxSteps {
    int nb;        // blocks of a row
    int chunks;
};
inline MxSteps mx4_steps(int64_t in, int nk_max, int* nk) {
    MxSteps s;
    s.nb = (int)(in / kMxBlock);
    const int steps = (s.nb + 3) / 4;
    s.chunks = (steps + kMxWaves * nk_max - 1) / (kMxWaves * nk_max);
    *nk = (steps + kMxWaves * s.chunks - 1) / (kMxWaves * s.chunks);
    return s;
}

// Rows of activations.
//   FMT kFmt16: fp16, piece e of 8 values of block b of row r at x + r rs + b bs + e es (mx4_rows16: plain rows)
//   FMT kFmt4: MX4, codes [..][nb][16 bytes] and scale bytes [..][nb]
template <int FMT>
struct MxInputRows;
template <>
struct MxInputRows<kFmt16> {
    const f16* x;
    int rs, bs, es;
};
inline __host__ __device__ MxInputRows<kFmt16> mx4_rows16(const f16* x, int nb) { return {x, nb * kMxBlock, kMxBlock, 8}; }
template <>
struct MxInputRows<kFmt4> {
    const uint8_t* codes;
    const uint8_t* scales;
    int nb;
};

// What a lane holds of a step: the block `block` of row `row`.
template <int FMT>
struct MxOperand;
template <>
struct MxOperand<kFmt16> {
    f16x8 v[4];
    __device__ __forceinline__ void load(const MxInputRows<kFmt16>& x, int row, int block) {
        const f16* at = x.x + (size_t)row * x.rs + (size_t)block * x.bs;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = as_f16x8(load16(at + i * x.es));
    }
};
template <>
struct MxOperand<kFmt4> {
    u32x4 q;
    uint32_t s;
    __device__ __forceinline__ void load(const MxInputRows<kFmt4>& x, int row, int block) {
        const size_t at = (size_t)row * x.nb + block;
        q = load16(x.codes + at * kMxBlockBytes);
        s = x.scales[at];
    }
};

// Up to 16 rows of fp16 activations in LDS: a row takes 256 bytes a step, its 16-byte piece p of a step lies in slot p ^ fold(row).  The
// 16 lanes that one clock of a 16-byte read serves (0-3, 12-15, 20-27; 4-11, 16-19, 28-31; likewise above 32) then find 16 slots.
struct MxStaged {
    static constexpr int kSteps = 512;   // steps of all rows that fit: 128 KB
    const u32x4* lds;
    uint32_t at;   // their address
    int steps;     // of a row, at least 4
    __host__ __device__ static int row_steps(int nb) { return (nb + 3) / 4; }
    __device__ static __forceinline__ int fold(int r) { return (r & 3) | (r >> 1 & 4) | ((r >> 3 ^ r >> 2) & 1) << 3; }
    // Sends the rows there, straight from memory.  Past a row comes its last piece, which meets weights of 0.
    __device__ __forceinline__ void send(const f16* __restrict__ x, int rows, int nb) const {
        const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
        const int per = (steps + 3) / 4;   // loads of a row: 64 pieces, the last may begin earlier
        for (int n = wave; n < rows * per; n += kMxWaves) {
            const int r = n / per, s0 = min((n - r * per) * 4, steps - 4);
            const int piece = min((s0 * 16 + lane) ^ fold(r), nb * 4 - 1);
            load_to_lds(at + (uint32_t)(r * steps + s0) * 256u, x + (size_t)r * nb * kMxBlock, (uint32_t)piece * 16u);
        }
    }
    // Until this wave's have arrived, where at least LATER of its loads came after; a barrier says so for all.
    template <int LATER>
    __device__ static __forceinline__ void wait() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
};

// A lane's row of a tile: tile TR + lane_row, at most the last of `rows`.
struct MxTileRows {
    int lane_row, rows;
};

// wq, ws: the lane's own layer (gate or up, where a tile has rows of both).
// PAIR: column tiles 0 and 1 are the two numbers of the same columns (hidden_pair.h), added here: fin sees one.
// fin(t0, n, sum): called by all threads of the workgroup once per group, after a barrier: tiles t0 + i nwg for i < n;
// sum(i, col, r) adds the waves' partial products of matrix-core row r and column col of the i-th.
// STAGED: the activations go to LDS, and a step's are read when its turn comes; else they are in registers, from xin.
template <int CT, int NK, int FMT, int TILES, bool WIDE, int TR = kMxRows, bool PAIR = false, bool STAGED = false, class Fin>
__device__ __forceinline__ void mx4_body(const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws,
                                         const MxInputRows<FMT>& xin, const int (&xrow)[CT], const MxSteps st,
                                         const int bid, const int nwg, const int n_tiles, float* red, const MxTileRows of, Fin fin,
                                         const MxStaged staged = {}) {
    static_assert(!STAGED || (CT == 1 && FMT == kFmt16), "one column tile in LDS");
    static_assert(!PAIR || (CT == 2 && FMT == kFmt16), "two numbers a column");
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int q = lane >> 4;
    const int nb = st.nb;
    constexpr int RT = PAIR ? 1 : CT;   // column tiles that fin sees

    if (bid >= n_tiles) return;   // uniform
    const int last = bid + (n_tiles - 1 - bid) / nwg * nwg;
    auto first = [&](int c) { return (c * kMxWaves + wave) * NK; };   // this wave's first step of chunk c
    // First block of a tile (uniform), and the lane's row from there, in blocks.
    auto tile_block = [&](int tile) { return (size_t)tile * TR * nb; };
    const uint32_t lane_whole = (uint32_t)(of.lane_row * nb);
    const uint32_t lane_last = (uint32_t)(min(of.lane_row, of.rows - 1 - (n_tiles - 1) * TR) * nb);
    auto lane_block = [&](int tile) { return tile == n_tiles - 1 ? lane_last : lane_whole; };

    constexpr int kScales = WIDE ? 4 : NK;
    u32x4 cw[TILES][NK];
    uint32_t cs[TILES][kScales];
    auto load_codes = [&](int i, int j, int tile, int c) {
        // not with the streaming hint: a step reads half of a line, the wave's next step the other (36 us with it, 34 without)
        cw[i][j] = load16(wq + tile_block(tile) * kMxBlockBytes +
                          (lane_block(tile) + (uint32_t)min(4 * (first(c) + j) + q, nb - 1)) * (uint32_t)kMxBlockBytes);
    };
    auto load_scales = [&](uint32_t (&to)[kScales], int tile, int c) {
        const uint8_t* at = ws + tile_block(tile) + lane_block(tile);
        if constexpr (WIDE) {
            typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
            const u32x4_any v = *reinterpret_cast<const u32x4_any*>(at + min(4 * first(c), nb - kMxWideBlocks));
#pragma unroll
            for (int d = 0; d < 4; ++d) to[d] = v[d];
        } else {
#pragma unroll
            for (int j = 0; j < NK; ++j) to[j] = at[min(4 * (first(c) + j) + q, nb - 1)];
        }
    };
    constexpr int kHeld = !STAGED ? NK : TILES > 2 ? 1 : 2;   // steps in registers: one ahead where registers allow
    MxOperand<FMT> x[CT][kHeld];
    int piece[4];   // STAGED: the lane's of step 0
    if constexpr (STAGED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) piece[e] = xrow[0] * staged.steps * 16 + ((4 * q + e) ^ MxStaged::fold(xrow[0]));
    }
    auto read_x = [&](int j, int c) {
        if constexpr (STAGED) {
            const int s = min(first(c) + j, staged.steps - 1);   // past the row: weights of 0
#pragma unroll
            for (int e = 0; e < 4; ++e) x[0][j % kHeld].v[e] = as_f16x8(staged.lds[piece[e] + 16 * s]);
        }
    };
    auto load_x = [&](int j, int c) {   // past the row: its last block, which meets weights of 0
        const int b = min(4 * (first(c) + j) + q, nb - 1);
#pragma unroll
        for (int t = 0; t < CT; ++t) x[t][j].load(xin, xrow[t], b);
    };
    // A tile with odd blocks (mx4.h) from its beginning: steps without them, and those blocks one at a time.  In no hurry.
    auto again = [&](int tile, f32x4 (&acc)[CT]) {
        if constexpr (FMT == kFmt16) {
            f32x4 odd[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[t] = odd[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            const size_t row = tile_block(tile) + lane_block(tile);
#pragma unroll 1
            for (int n = 0; n < st.chunks * NK; ++n) {
                const int b = 4 * (first(n / NK) + n % NK) + q;
                const size_t at = row + min(b, nb - 1);
                const uint32_t s = b < nb ? ws[at] : 0u;
                const bool mine = odd_scale(s);
                const u32x4 a = load16(wq + at * kMxBlockBytes);
                MxOperand<kFmt16> v[CT];
#pragma unroll
                for (int t = 0; t < CT; ++t) v[t].load(xin, xrow[t], min(b, nb - 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f16x8 w = decode8(a[e], plain_scale(s) ? scale_value(s) : 0.f);
#pragma unroll
                    for (int t = 0; t < CT; ++t) acc[t] = mfma16x16x32(w, v[t].v[e], acc[t]);
                }
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    if (__ballot(mine && q == g) == 0) continue;
                    f32x4 d[CT] = {};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f16x8 w = decode8(mine && q == g ? a[e] : 0u, 1.f);
#pragma unroll
                        for (int t = 0; t < CT; ++t) d[t] = mfma16x16x32(w, v[t].v[e], d[t]);
                    }
#pragma unroll
                    for (int t = 0; t < CT; ++t) pin(d[t]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {   // rows 4 q + r of the result; those without the block have sums of 0
                        const uint32_t sr = (uint32_t)__shfl(mine ? (int)s : 127, g * 16 + 4 * q + r, kWave);
#pragma unroll
                        for (int t = 0; t < CT; ++t) odd[t][r] += odd_sum(d[t][r], sr);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                pin(acc[t]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][r] = no_infinity(acc[t][r]) + odd[t][r];
            }
        }
    };

    const bool idle = st.chunks == 1 && 4 * first(0) >= nb;   // a wave without a step of its own (uniform)
    const bool whole = bid + (TILES - 1) * nwg < n_tiles;     // the first group
    if (idle) {
        if constexpr (STAGED) MxStaged::wait<0>();
    } else if constexpr (FMT == kFmt4) {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
            if (bid + i * nwg < n_tiles) {
                load_scales(cs[i], bid + i * nwg, 0);
#pragma unroll
                for (int j = 0; j < NK; ++j) load_codes(i, j, bid + i * nwg, 0);
            }
#pragma unroll
        for (int j = 0; j < NK; ++j) load_x(j, 0);
    } else {
#pragma unroll
        for (int i = 0; i < TILES; ++i) load_scales(cs[i], min(bid + i * nwg, last), 0);
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            if constexpr (!STAGED) load_x(j, 0);
#pragma unroll
            for (int i = 0; i < TILES; ++i)
                if (bid + i * nwg < n_tiles) load_codes(i, j, bid + i * nwg, 0);
        }
        if constexpr (STAGED) {
            if (whole) MxStaged::wait<TILES + TILES * NK>();
            else MxStaged::wait<TILES + NK>();
        }
    }
    if constexpr (STAGED) asm volatile("s_barrier" ::: "memory");

    f32x4 acc[TILES][CT];
    uint32_t least, most;   // scales met in a group, 0 apart: least is one less than their least
    // The products of chunk c, `left` tiles.  LOAD: what comes next, chunk cn of the tiles from tn on, XLOAD: and its activations.
    auto run = [&](auto load, auto xload, int left, int c, int tn, int cn) {
        constexpr bool LOAD = decltype(load)::value, XLOAD = decltype(xload)::value;
        const int coming = (n_tiles - tn + nwg - 1) / nwg;   // tiles from tn on
        // The lane's scale bytes of the round, one word a tile; zeros past the row.
        uint32_t sc[TILES][WIDE ? 1 : NK];
        if constexpr (WIDE) {
            const int d = min(max(4 * first(c) - (nb - kMxWideBlocks), 0), kMxWideBlocks);   // uniform
            if (d != 0) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    const u32x4 v = move_bytes(u32x4{cs[i][0], cs[i][1], cs[i][2], cs[i][3]}, d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) cs[i][j] = v[j];
                }
            }
            const uint32_t low = 0x0c0c0400u + 0x0101u * (uint32_t)q, high = 0x04000c0cu + 0x01010000u * (uint32_t)q;   // 0x0c: zero
#pragma unroll
            for (int i = 0; i < TILES; ++i)
                sc[i][0] = __builtin_amdgcn_perm(cs[i][1], cs[i][0], low) | __builtin_amdgcn_perm(cs[i][3], cs[i][2], high);
        } else {
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int j = 0; j < NK; ++j) sc[i][j] = 4 * (first(c) + j) + q < nb ? cs[i][j] : 0u;
        }
        if constexpr (LOAD) {
#pragma unroll
            for (int i = 0; i < TILES; ++i) load_scales(cs[i], min(tn + i * nwg, last), cn);
        }
        if constexpr (kHeld == 2) read_x(0, c);
        __builtin_amdgcn_sched_barrier(0);
        // Step j of tile i, and the load of what takes the place of its codes.
        auto step = [&](int j, int i) {
            if (i < left && 4 * (first(c) + j) < nb) {   // uniform
                if constexpr (FMT == kFmt4) {
                    // past the row: codes 0 on both sides with scales of 1, whatever was loaded
                    const bool in_row = 4 * (first(c) + j) + q < nb;
                    i32x8 a = operand4(cw[i][j]);
#pragma unroll
                    for (int d = 0; d < 4; ++d) a[d] = in_row ? a[d] : 0;
                    const uint32_t sa = in_row ? WIDE ? sc[i][0] >> 8 * j : sc[i][j] : 127u;   // its low byte counts
#pragma unroll
                    for (int t = 0; t < CT; ++t) {
                        i32x8 v = operand4(x[t][j].q);
#pragma unroll
                        for (int d = 0; d < 4; ++d) v[d] = in_row ? v[d] : 0;
                        acc[i][t] = mfma_mx(a, v, acc[i][t], sa, in_row ? x[t][j].s : 127u);
                    }
                } else {
                    const uint32_t s = WIDE ? sc[i][0] >> 8 * j & 255u : sc[i][j];
                    least = min(least, s - 1u);
                    most = max(most, s);
                    const float f = scale_value(s);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f16x8 w = decode8(cw[i][j][e], f);
#pragma unroll
                        for (int t = 0; t < CT; ++t) acc[i][t] = mfma16x16x32(w, x[t][j % kHeld].v[e], acc[i][t]);
                    }
                }
            }
        };
        if constexpr (FMT == kFmt4) {   // little work a step: a branch a tile
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
#pragma unroll
                for (int j = 0; j < NK; ++j) step(j, i);
                if constexpr (LOAD) {
                    if (i < coming && (!XLOAD || 4 * first(cn) < nb)) {
#pragma unroll
                        for (int j = 0; j < NK; ++j) load_codes(i, j, tn + i * nwg, cn);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (LOAD && XLOAD) {
                if (4 * first(cn) < nb) {
#pragma unroll
                    for (int j = 0; j < NK; ++j) load_x(j, cn);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                if (kHeld == 1) read_x(j, c);
                else if (j + 1 < NK) read_x(j + 1, c);
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    step(j, i);
                    if constexpr (LOAD) {
                        if (i < coming && (!XLOAD || 4 * (first(cn) + j) < nb)) load_codes(i, j, tn + i * nwg, cn);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (LOAD && XLOAD && !STAGED) {
                    if (4 * (first(cn) + j) < nb) load_x(j, cn);
                }
            }
        }
    };
    for (int t0 = bid; t0 < n_tiles; t0 += nwg * TILES) {
        const int after = t0 + nwg * TILES;
        const int left = (n_tiles - t0 + nwg - 1) / nwg;   // tiles of this group
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        least = ~0u;
        most = 0u;
        const bool end = after >= n_tiles;
        if (idle) {
        } else if (st.chunks > 1) {
            for (int c = 0; c < st.chunks - (int)end; ++c) {
                const bool same = c + 1 < st.chunks;
                run(std::true_type{}, std::true_type{}, left, c, same ? t0 : after, same ? c + 1 : 0);
            }
        } else if (!end) {
            run(std::true_type{}, std::false_type{}, left, 0, after, 0);
        }
        if (end && !idle) run(std::false_type{}, std::false_type{}, left, st.chunks - 1, 0, 0);
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t) pin(acc[i][t]);
        if constexpr (FMT == kFmt16) {
            const bool odd = __ballot(odd_scale(least + 1u) || odd_scale(most)) != 0;
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
#pragma unroll
                for (int t = 0; t < CT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][t][r] = no_infinity(acc[i][t][r]);
                if (odd && i < left) again(t0 + i * nwg, acc[i]);
                if constexpr (PAIR) acc[i][0] += acc[i][1] * (1.f / kPairFine);
            }
        }
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if (i >= left) continue;
                *reinterpret_cast<f32x4*>(red + ((i * kMxWaves + wave) * RT + t) * 256 + (lane & 15) * kMxRows + 4 * q) = acc[i][t];
            }
        __syncthreads();
        fin(t0, min(left, TILES), [&](int i, int col, int r) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kMxWaves; ++w) s += red[(i * kMxWaves + w) * RT * 256 + col * kMxRows + r];
            return s;
        });
        __syncthreads();
    }
}

}  // namespace aqlm

// A workgroup's part of a product of MX4 rows with up to 64 columns of activations: mx4_linear.hip describes the kernel
// that it carries; the mixture-of-experts layer (moe_mx4.hip) runs it on experts.
//
// The workgroup walks tiles of 16 matrix-core rows in groups of mx4_tiles: tiles bid + i nwg, or, RUN, 4 neighbours
// each (4 (bid + i nwg) + 0 .. 3).  Its 8 waves share the
// inputs: wave w takes `nk` <= NK steps of 128 inputs out of every chunk of 8 nk, keeps their activations in registers
// for all tiles of the group, and streams the codes of its steps, a group ahead.  The waves' partial tiles are
// added in LDS in the order of the waves.
#pragma once
#include <type_traits>

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

// LDS floats of the partial tiles of a group, CT column tiles.
constexpr int mx4_red_floats(int ct) { return mx4_tiles(ct) * kMxWaves * ct * 256; }

// How the inputs are dealt to the waves.
struct MxSteps {
    int nb;        // blocks of a row
    int nk;        // steps a wave takes of a chunk
    int chunks;
};
inline MxSteps mx4_steps(int64_t in, int nk_max) {
    MxSteps s;
    s.nb = (int)(in / kMxBlock);
    const int steps = (s.nb + 3) / 4;
    s.chunks = (steps + kMxWaves * nk_max - 1) / (kMxWaves * nk_max);
    s.nk = (steps + kMxWaves * s.chunks - 1) / (kMxWaves * s.chunks);
    return s;
}

// Activations of one lane, the block `block` of token `row`.
//   FMT kFmt6: split records (mx4.h)
//   FMT kFmt4: MX4 rows, codes [..][nb][16 bytes] and scale bytes [..][nb]
template <int FMT>
struct MxInputRows;
template <>
struct MxInputRows<kFmt6> {
    SplitRows rows;
};
template <>
struct MxInputRows<kFmt4> {
    const uint8_t* codes;
    const uint8_t* scales;
    int nb;
};

template <int FMT>
struct MxOperand {
    static constexpr int kParts = FMT == kFmt6 ? kPieces : 1;
    using Part = std::conditional_t<FMT == kFmt6, u32x6, u32x4>;
    Part q[kParts];
    uint32_t s;
    __device__ __forceinline__ void load(const MxInputRows<FMT>& x, int row, int block, bool in_row) {
        if constexpr (FMT == kFmt6) {
            char* rec = x.rows.record(row, block);
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const u32x4 a = *x.rows.first(rec, row, p);
                const u32x2 b = *x.rows.rest(rec, row, p);
                q[p] = u32x6{a[0], a[1], a[2], a[3], b[0], b[1]};
            }
            s = *x.rows.scales(rec, row);
        } else {
            const size_t at = (size_t)row * x.nb + block;
            q[0] = load16(x.codes + at * kMxBlockBytes);
            s = x.scales[at];
        }
        if (!in_row) {
#pragma unroll
            for (int p = 0; p < kParts; ++p) q[p] = Part{};
            s = 0x7f7f7f7fu;
        }
    }
    __device__ __forceinline__ f32x4 product(u32x4 a, uint32_t sa, f32x4 acc) const {
        const i32x8 av = operand4(a);
        if constexpr (FMT == kFmt4) {
            return mfma_mx<kFmt4, 0>(av, operand4(q[0]), acc, sa, s);
        } else {
            acc = mfma_mx<kFmt6, 3>(av, operand6(q[3]), acc, sa, s);   // small terms first
            acc = mfma_mx<kFmt6, 2>(av, operand6(q[2]), acc, sa, s);
            acc = mfma_mx<kFmt6, 1>(av, operand6(q[1]), acc, sa, s);
            return mfma_mx<kFmt6, 0>(av, operand6(q[0]), acc, sa, s);
        }
    }
};

// row_of(tile): this lane's row of the tile inside wq / ws, which are the lane's own layer (clamped into it).
// prepare(): called once the first codes are on their way; what the activations wait for.
// fin(t0, n, sum): called by all threads of the workgroup once per group, after a barrier: tiles t0 + i step for i < n, step 1
// with RUN, else nwg; sum(i, col, r) adds the waves' partial products of matrix-core row r and column col of the i-th.
template <int CT, int NK, int FMT, bool RUN, int TILES, bool WIDE, class RowOf, class Prepare, class Fin>
__device__ __forceinline__ void mx4_body(const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws,
                                         const MxInputRows<FMT>& xin, const int (&xrow)[CT], const MxSteps st,
                                         const int bid, const int nwg, const int n_tiles, float* red, RowOf row_of,
                                         Prepare prepare, Fin fin) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int q = lane >> 4;
    const int nb = st.nb;
    constexpr int kMxTiles = TILES;

    const int scale_bit = WIDE ? 8 * q : 0;
    u32x4 cw[kMxTiles][NK];
    uint32_t cs[kMxTiles][WIDE ? 4 : NK];
    auto first = [&](int c) { return (c * kMxWaves + wave) * st.nk; };   // this wave's first step of chunk c
    auto load_tile = [&](int i, int tile, int c) {
        const size_t row = (size_t)row_of(min(tile, n_tiles - 1));
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            if (j < st.nk) {
                const size_t at = row * nb + min(4 * (first(c) + j) + q, nb - 1);
                // not with the streaming hint: a step reads half of a line, the wave's next step the other (36 us with it, 34 without)
                cw[i][j] = load16(wq + at * kMxBlockBytes);
                if constexpr (!WIDE) cs[i][j] = ws[at];
            }
        }
        if constexpr (WIDE) {
            typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
            const u32x4_any v = *reinterpret_cast<const u32x4_any*>(ws + row * nb + min(4 * first(c), nb - kMxWideBlocks));
#pragma unroll
            for (int d = 0; d < 4; ++d) cs[i][d] = v[d];
        }
    };
    auto settle_scales = [&](int i, int c) {
        if constexpr (WIDE) {
            const int d = min(max(4 * first(c) - (nb - kMxWideBlocks), 0), kMxWideBlocks);   // uniform
            if (d == 0) return;
            u32x4 v = {cs[i][0], cs[i][1], cs[i][2], cs[i][3]};
            v = move_bytes(v, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[i][j] = v[j];
        }
    };
    MxOperand<FMT> x[CT][NK];
    auto load_x = [&](int c) {
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            if (j < st.nk) {
                const int b = 4 * (first(c) + j) + q;
#pragma unroll
                for (int t = 0; t < CT; ++t) x[t][j].load(xin, xrow[t], min(b, nb - 1), b < nb);
            }
        }
    };

    const int step = RUN ? 1 : nwg, begin = RUN ? bid * kMxTiles : bid;
#pragma unroll
    for (int i = 0; i < kMxTiles; ++i)
        if (begin + i * step < n_tiles) load_tile(i, begin + i * step, 0);
    prepare();
    load_x(0);

    for (int t0 = begin; t0 < n_tiles; t0 += nwg * kMxTiles) {
        f32x4 acc[kMxTiles][CT];
#pragma unroll
        for (int i = 0; i < kMxTiles; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < st.chunks; ++c) {
            const int cn = c + 1 < st.chunks ? c + 1 : 0;                      // what comes next
            const int tn = cn != 0 ? t0 : t0 + nwg * kMxTiles;
#pragma unroll
            for (int i = 0; i < kMxTiles; ++i) {
                if (t0 + i * step < n_tiles) {
                    settle_scales(i, c);
#pragma unroll
                    for (int j = 0; j < NK; ++j) {
                        if (j < st.nk) {
                            // past the row: codes 0 with a scale of 1, whatever was loaded
                            const bool in_row = 4 * (first(c) + j) + q < nb;
                            u32x4 a = cw[i][j];
#pragma unroll
                            for (int d = 0; d < 4; ++d) a[d] = in_row ? a[d] : 0u;
                            const uint32_t sa = in_row ? cs[i][j] >> scale_bit : 127u;   // its low byte counts
#pragma unroll
                            for (int t = 0; t < CT; ++t) acc[i][t] = x[t][j].product(a, sa, acc[i][t]);
                        }
                    }
                    if (tn + i * step < n_tiles) load_tile(i, tn + i * step, cn);
                }
            }
            if (st.chunks > 1 && tn < n_tiles) load_x(cn);
        }
#pragma unroll
        for (int i = 0; i < kMxTiles; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t) pin(acc[i][t]);
        const int left = (n_tiles - t0 + step - 1) / step;   // tiles of this group
#pragma unroll
        for (int i = 0; i < kMxTiles; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                if (i >= left) continue;
                *reinterpret_cast<f32x4*>(red + ((i * kMxWaves + wave) * CT + t) * 256 + (lane & 15) * kMxRows + 4 * q) = acc[i][t];
            }
        __syncthreads();
        fin(t0, min(left, kMxTiles), [&](int i, int col, int r) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kMxWaves; ++w) s += red[(i * kMxWaves + w) * CT * 256 + col * kMxRows + r];
            return s;
        });
        __syncthreads();
    }
}

// The same for up to 16 columns of split activations in LDS, rows of at least kMxWideBlocks blocks, and workgroups of few tiles.  A
// step's activations are read when its turn comes, for all tiles of the group; that leaves registers to write the loads without
// branches.  The compiler counts the loads in flight and waits for the oldest; where paths with and without a load meet it waits for all
// of them, so the last round, which loads nothing, is code of its own.  Past a workgroup's last tile its loads repeat that tile.
template <int NK, int TILES, class RowOf, class Prepare, class Fin>
__device__ __forceinline__ void mx4_body_lds(const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws, const SplitRows xs,
                                             const int xrow, const MxSteps st, const int bid, const int nwg, const int n_tiles,
                                             float* red, RowOf row_of, Prepare prepare, Fin fin) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int q = lane >> 4;
    const int nb = st.nb;
    if (bid >= n_tiles) return;   // uniform
    const int last = bid + (n_tiles - 1 - bid) / nwg * nwg;
    auto first = [&](int c) { return (c * kMxWaves + wave) * NK; };   // this wave's first step of chunk c
    auto base = [&](int tile) { return (size_t)row_of(min(tile, last)) * nb; };

    u32x4 cw[TILES][NK];
    uint32_t cs[TILES][4], next[TILES][4];
    auto load_codes = [&](int i, int j, size_t row, int c) {
        cw[i][j] = load16(wq + (row + min(4 * (first(c) + j) + q, nb - 1)) * kMxBlockBytes);
    };
    auto load_scales = [&](uint32_t (&to)[4], size_t row, int c) {
        typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(ws + row + min(4 * first(c), nb - kMxWideBlocks));
#pragma unroll
        for (int d = 0; d < 4; ++d) to[d] = v[d];
    };
#pragma unroll
    for (int i = 0; i < TILES; ++i) load_scales(cs[i], base(bid + i * nwg), 0);
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int i = 0; i < TILES; ++i) load_codes(i, j, base(bid + i * nwg), 0);
    prepare();

    f32x4 acc[TILES];
    auto run = [&](auto more, int c, int tn, int cn) {
        const int d = min(max(4 * first(c) - (nb - kMxWideBlocks), 0), kMxWideBlocks);   // uniform
        if (d != 0) {
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const u32x4 v = move_bytes(u32x4{cs[i][0], cs[i][1], cs[i][2], cs[i][3]}, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) cs[i][j] = v[j];
            }
        }
        size_t row[TILES];
        if constexpr (decltype(more)::value) {
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                row[i] = base(tn + i * nwg);
                load_scales(next[i], row[i], cn);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int b = 4 * (first(c) + j) + q;
            const bool in_row = b < nb;
            MxOperand<kFmt6> x;
            x.load(MxInputRows<kFmt6>{xs}, xrow, min(b, nb - 1), in_row);
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                // past the row: codes 0 with a scale of 1, whatever was loaded
                u32x4 a = cw[i][j];
#pragma unroll
                for (int w = 0; w < 4; ++w) a[w] = in_row ? a[w] : 0u;
                acc[i] = x.product(a, in_row ? cs[i][j] >> 8 * q : 127u, acc[i]);
                if constexpr (decltype(more)::value) load_codes(i, j, row[i], cn);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (decltype(more)::value) {
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) cs[i][w] = next[i][w];
        }
    };
    for (int t0 = bid; t0 < n_tiles; t0 += nwg * TILES) {
        const int after = t0 + nwg * TILES;
#pragma unroll
        for (int i = 0; i < TILES; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool end = after >= n_tiles;
        for (int c = 0; c < st.chunks - (int)end; ++c) {
            const bool same = c + 1 < st.chunks;
            run(std::true_type{}, c, same ? t0 : after, same ? c + 1 : 0);
        }
        if (end) run(std::false_type{}, st.chunks - 1, 0, 0);
#pragma unroll
        for (int i = 0; i < TILES; ++i) pin(acc[i]);
        const int left = (n_tiles - t0 + nwg - 1) / nwg;   // tiles of this group
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            if (i >= left) continue;
            *reinterpret_cast<f32x4*>(red + (i * kMxWaves + wave) * 256 + (lane & 15) * kMxRows + 4 * q) = acc[i];
        }
        __syncthreads();
        fin(t0, min(left, TILES), [&](int i, int col, int r) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kMxWaves; ++w) s += red[(i * kMxWaves + w) * 256 + col * kMxRows + r];
            return s;
        });
        __syncthreads();
    }
}

}  // namespace aqlm

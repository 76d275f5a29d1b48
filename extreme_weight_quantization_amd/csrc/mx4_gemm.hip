// Products of MX4 weights with many tokens: z[t][i] = sum_k W[i][k] x[t][k], then mx4_linear.hip's epilogue.
//
// With x in MX4 the scaled matrix instructions take codes and scales as they are; with x in fp16 a wave converts its codes to fp16
// in its registers, which is exact (mx4.h).  The work is to bring the operands on time.  A workgroup of
// WM x WN waves owns a tile of rows of W x tokens; a wave a part of MT x NT squares of 32 x 32, which each take one
// instruction a step of 64 inputs (four with x in fp16).  Inputs pass through LDS in stages of KB blocks of 32, loaded
// straight from memory, with one barrier a stage.  Between two matrix instructions of a step a wave reads a piece of the
// next step's operands, or issues a load of a later stage.
//
// LDS of a stage:
//   rows of MX4 (W, and x where it is MX4): KB blocks of 16 bytes a row; block b of row r lies in slot b ^ fold(r), so that the
//     16 lanes that one clock of a 16-byte read serves (0-3, 12-15, 20-27; 4-11, 16-19, 28-31; likewise above 32) find 16
//     distinct banks, and KB neighbouring lanes of a load still read 16 * KB contiguous bytes;
//   rows of fp16 x: 4 KB chunks of 8 values; chunk c of row r lies in slot c ^ (r & 15), for the same reason.
// Scale bytes of MX4 rows: 16 bytes a row at a time, 16 blocks' worth, into LDS of their own (two buffers): straight where
// rows and array are 16-byte aligned (in % 512 == 0), else through registers from any address.  A lane reads the bytes of
// its row and stage and moves its half of the wave's to where the instruction's byte selection finds it.
// Odd blocks (mx4.h) are zero in all this; a wave that has met one goes over its scales again and adds them one by one.
//
// At the end a wave turns its squares in LDS, so that a lane has 8 neighbouring outputs of a token, and finishes them in a
// loop that is not unrolled: with a copy of the activations' code for every square the epilogue took 70 us of 360.
//
// Bound by the matrix cores where tiles fill the chip: x in MX4, 8192 -> 28672, 2048 tokens 290 us (3.3 PF/s; 59 % busy, the rest waits
// at a stage's barrier and half a round of tiles), x fp16, 4096 -> 11008 184 us (1.0 PF/s); else by the codes: 8192 -> 28672, 64 tokens, 25
// and 42 us.
#include <algorithm>
#include <type_traits>

#include "act_bias.h"
#include "act_math.h"
#include "mx4_gemm.h"

namespace aqlm {

namespace {

constexpr int kChunkBlocks = 16;       // blocks that a load of scales serves

struct GemmArgs {
    const uint8_t* w;        // codes, scales of W
    const uint8_t* ws;
    const uint8_t* x;        // codes, scales of x; or its fp16 rows (xs NULL)
    const uint8_t* xs;
    const f16* bias;
    const f16* residual;     // may be y
    f16* y;
    float* part;             // [split][token][op], for splits > 1
    int act, out, T, nb, op;
    int tiles_m, tiles_n, splits, chunks;   // chunks of kChunkBlocks of the whole row
};

template <int FMT, int WM, int WN, int MT, int NT, int KB, int STAGES>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int kM = WM * MT * 32, kN = WN * NT * 32;
    static constexpr int kABytes = kM * KB * 16;
    static constexpr int kXBlock = FMT == kFmt4 ? kMxBlockBytes : 2 * kMxBlock;   // bytes of a block of x
    static constexpr int kBBytes = kN * KB * kXBlock;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kScaleLoads = (kM + (FMT == kFmt4 ? kN : 0) + kThreads - 1) / kThreads;   // rows a thread
    static constexpr int kScaleRows = kScaleLoads * kThreads;              // the last may repeat
    static constexpr int kScales = STAGES * kStage;                        // their place in LDS
    static constexpr int kPipe = kScales + 2 * kScaleRows * 16;
    static constexpr int kEpiRow = MT * 32 * 4 + 16;                       // bytes of a token in a wave's LDS of the epilogue
    static constexpr int kLds = kPipe > kWaves * 32 * kEpiRow ? kPipe : kWaves * 32 * kEpiRow;
    static constexpr int kLoads = (kStage / 1024 + kWaves - 1) / kWaves;   // a wave, a stage
    static constexpr int kSteps = KB / 2;
    static constexpr int kChunkStages = kChunkBlocks / KB;
    static_assert(kLds <= 163840 && kStage % 1024 == 0 && kM % 64 == 0 && kN % 64 == 0);
};

// 16 bytes of an array of `total` >= 16 from any offset; bytes past its end are zero.
__device__ __forceinline__ u32x4 load_bytes16(const uint8_t* __restrict__ p, int64_t at, int64_t total) {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
    const int64_t from = at < total - 16 ? at : total - 16;
    const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p + from);
    return move_bytes(u32x4{v[0], v[1], v[2], v[3]}, (int)(at - from < 16 ? at - from : 16));
}

template <int KB>
__device__ __forceinline__ int fold(int r) { return KB == 8 ? r & 7 : (r >> 2) & 3; }

// The operands of a step of 64 inputs.
template <int FMT, int MT, int NT>
struct StepOperands {
    u32x4 a[MT];
    u32x4 b[NT][FMT == kFmt4 ? 1 : 4];
};

// The scales of MX4 rows of a stage: KB / 4 words a square.
template <int FMT, int MT, int NT, int KB>
struct StageScales {
    uint32_t a[MT][KB / 4], b[FMT == kFmt4 ? NT : 1][KB / 4];
};

template <int FMT, int WM, int WN, int MT, int NT, int KB, int STAGES, bool PART, bool STRAIGHT>
__global__ __launch_bounds__(WM* WN * 64) void mx4_gemm_kernel(GemmArgs g) {
    using L = Tile<FMT, WM, WN, MT, NT, KB, STAGES>;
    extern __shared__ u32x4 smem[];
    char* lds = reinterpret_cast<char*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int l32 = lane & 31, half = lane >> 5;
    // An XCD's workgroups are neighbours in an order of kBand token tiles next to each other, row tile after row tile: what
    // 32 of them read in a stage is then about as little as it can be (x in fp16: 4 x 32 KB and 8 x 16 KB, where all
    // 16 token tiles of 2048 tokens would make 540 KB), and comes out of the XCD's L2 when it is shared.
    constexpr int kBand = FMT == kFmt4 ? 8 : 4;
    const int tiles = g.tiles_m * g.tiles_n, u = xcd_run((int)blockIdx.x, (int)gridDim.x), split = u / tiles;
    const int band = u % tiles / (kBand * g.tiles_m), in_band = u % tiles - band * kBand * g.tiles_m;
    const int width = min(kBand, g.tiles_n - band * kBand);
    const int n0 = (band * kBand + in_band % width) * L::kN, m0 = in_band / width * L::kM;
    const int nb = g.nb;
    const int per = (g.chunks + g.splits - 1) / g.splits;               // chunks of a part
    const int block0 = split * per * kChunkBlocks, blocks = min(per * kChunkBlocks, nb - block0);
    const int n_stage = (blocks + KB - 1) / KB;
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t lds0 = lds_address(lds);

    // Load j of this wave in a stage: 64 chunks of 16 bytes, from chunk 64 (wave + kWaves j) on (past the stage: the last 64
    // again).  The lane's chunk of stage 0 lies row_off from the operand's base.  Blocks past a row of MX4 are whatever follows it, and
    // the array's last 16 bytes where nothing does: the products leave them out.  Past a row of fp16 x comes its own last chunk: it meets
    // weights of 0, and what it may hold of infinities and NaN the row's outputs are NaN of anyway.
    const uint8_t* const wbase = g.w + (size_t)m0 * nb * kMxBlockBytes;
    const uint8_t* const xbase = g.x + (size_t)n0 * nb * L::kXBlock;
    auto last16 = [](int64_t bytes) { return (uint32_t)(bytes - 16 < (int64_t)0xfffffff0 ? bytes - 16 : (int64_t)0xfffffff0); };
    const uint32_t wlast = last16((int64_t)(g.out - m0) * nb * kMxBlockBytes);
    const uint32_t xlast = last16((int64_t)(g.T - n0) * nb * kMxBlockBytes);   // MX4
    uint32_t row_off[L::kLoads], row_last[L::kLoads];   // row_last: of fp16 x
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        const int i = min(wave + j * L::kWaves, L::kStage / 1024 - 1), c = i * 64 + lane;
        if (i < L::kABytes / 1024) {
            const int r = c / KB;
            row_off[j] = (uint32_t)((min(r, g.out - 1 - m0) * nb + block0 + ((c & (KB - 1)) ^ fold<KB>(r))) * kMxBlockBytes);
        } else if constexpr (FMT == kFmt4) {
            const int cb = c - L::kABytes / 16, r = cb / KB;
            row_off[j] = (uint32_t)((min(r, g.T - 1 - n0) * nb + block0 + ((cb & (KB - 1)) ^ fold<KB>(r))) * kMxBlockBytes);
        } else {
            const int cb = c - L::kABytes / 16, r = cb / (4 * KB);
            const uint32_t row = (uint32_t)(min(r, g.T - 1 - n0) * nb) * L::kXBlock;
            row_off[j] = row + (uint32_t)block0 * L::kXBlock + (uint32_t)((cb & (4 * KB - 1)) ^ (r & 15)) * 16;
            row_last[j] = row + (uint32_t)nb * L::kXBlock - 16;
        }
    }
    static_assert(L::kABytes / 1024 % L::kWaves == 0, "a load is of W or x for all waves");
    auto load = [&](int s, int j) {
        const int i = min(wave + j * L::kWaves, L::kStage / 1024 - 1);   // uniform
        const bool of_w = j * L::kWaves < L::kABytes / 1024;
        const uint32_t off = row_off[j] + (uint32_t)(s * KB * (of_w ? kMxBlockBytes : L::kXBlock));
        load_to_lds(lds0 + s % STAGES * L::kStage + i * 1024, of_w ? wbase : xbase,
                    min(off, of_w ? wlast : FMT == kFmt4 ? xlast : row_last[j]));
    };

    // Scales of a chunk: a thread has rows tid, tid + kThreads, ... of W, then, where x is MX4, of x (then the last again).
    auto scales_of_w = [&](int q) { return FMT != kFmt4 || wave * 64 + q * L::kThreads < L::kM; };   // all of a wave's 64
    const uint8_t* sbase[L::kScaleLoads];
    int64_t srow[L::kScaleLoads], sbytes[L::kScaleLoads];
#pragma unroll
    for (int q = 0; q < L::kScaleLoads; ++q) {
        const bool of_w = scales_of_w(q);
        const int r = tid + q * L::kThreads, rows = of_w ? g.out : g.T;
        sbase[q] = of_w ? g.ws : g.xs;
        srow[q] = (int64_t)min(of_w ? m0 + r : n0 + r - L::kM, rows - 1) * nb;
        sbytes[q] = (int64_t)rows * nb;
    }
    auto load_scales = [&](int c, u32x4 (&v)[L::kScaleLoads]) {   // into registers
#pragma unroll
        for (int q = 0; q < L::kScaleLoads; ++q) v[q] = load_bytes16(sbase[q], srow[q] + block0 + c * kChunkBlocks, sbytes[q]);
    };
    auto keep_scales = [&](const u32x4 (&v)[L::kScaleLoads], int c) {
#pragma unroll
        for (int q = 0; q < L::kScaleLoads; ++q)
            *reinterpret_cast<u32x4*>(lds + L::kScales + ((c & 1) * L::kScaleRows + tid + q * L::kThreads) * 16) = v[q];
    };
    auto send_scales = [&](int c) {   // straight into LDS
        const int b = min(block0 + c * kChunkBlocks, nb - kChunkBlocks);
#pragma unroll
        for (int q = 0; q < L::kScaleLoads; ++q) {
            const int64_t row0 = (int64_t)(scales_of_w(q) ? m0 : n0) * nb;
            load_to_lds(lds0 + L::kScales + ((c & 1) * L::kScaleRows + wave * 64 + q * L::kThreads) * 16, sbase[q] + row0,
                        (uint32_t)(srow[q] - row0) + b);
        }
    };

    f32x16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x16{};

    u32x4 sc[L::kScaleLoads] = {};
    if constexpr (STRAIGHT) {
        send_scales(0);
    } else {
        load_scales(0, sc);
        keep_scales(sc, 0);
        load_scales(1, sc);
    }
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) load(s, j);

    // Places of the lane's operands in a stage, at block b ^ its row's fold.
    const int fd = fold<KB>(l32);
    const uint32_t pa = (uint32_t)(wm * MT * 32 + l32) * (KB * 16);
    const uint32_t pb4 = L::kABytes + (uint32_t)(wn * NT * 32 + l32) * (KB * 16);
    const uint32_t pb16 = L::kABytes + (uint32_t)(wn * NT * 32 + l32) * (KB * 64);
    const uint32_t psa = L::kScales + (uint32_t)(wm * MT * 32 + l32) * 16;
    const uint32_t psb = L::kScales + (uint32_t)(L::kM + wn * NT * 32 + l32) * 16;

    using Operands = StepOperands<FMT, MT, NT>;
    using Scales = StageScales<FMT, MT, NT, KB>;
    // Reads of step k of the stage at `st`, one of kReads.
    constexpr int kReads = MT + NT * (FMT == kFmt4 ? 1 : 4);
    auto read = [&](Operands& o, const char* st, int k, int q) {
        const int slot = ((2 * k + half) ^ fd) * 16;
        if (q < MT) {
            o.a[q] = *reinterpret_cast<const u32x4*>(st + pa + slot + q * 32 * KB * 16);
        } else if constexpr (FMT == kFmt4) {
            o.b[q - MT][0] = *reinterpret_cast<const u32x4*>(st + pb4 + slot + (q - MT) * 32 * KB * 16);
        } else {
            const int j = (q - MT) / 4, e = (q - MT) % 4;
            o.b[j][e] = *reinterpret_cast<const u32x4*>(st + pb16 + j * 32 * KB * 64 + (((2 * k + half) * 4 + e) ^ (l32 & 15)) * 16);
        }
    };
    auto read_scales = [&](Scales& sc, int s) {
        const char* at = lds + (s / L::kChunkStages & 1) * L::kScaleRows * 16 + s % L::kChunkStages * KB;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int d = 0; d < KB / 4; ++d) sc.a[i][d] = *reinterpret_cast<const uint32_t*>(at + psa + i * 512 + d * 4);
        if constexpr (FMT == kFmt4) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int d = 0; d < KB / 4; ++d) sc.b[j][d] = *reinterpret_cast<const uint32_t*>(at + psb + j * 512 + d * 4);
        }
    };
    auto half_scales = [&](Scales& sc) {   // byte 2 k + half to byte 2 k of word k / 2
#pragma unroll
        for (int d = 0; d < KB / 4; ++d) {
#pragma unroll
            for (int i = 0; i < MT; ++i) sc.a[i][d] >>= 8 * half;
            if constexpr (FMT == kFmt4) {
#pragma unroll
                for (int j = 0; j < NT; ++j) sc.b[j][d] >>= 8 * half;
            }
        }
    };

    // acc += the products of step K, and between them what between(n) does.  Next to MX4 activations, blocks past the row, whatever was
    // loaded for them, count with scales of 2^-127 and 1: below 2^-118, which no fp16 result feels.
    constexpr int kProducts = MT * NT * (FMT == kFmt4 ? 1 : 4);
    uint32_t odd = 0u;   // whether this lane has met an odd block
    auto multiply = [&](const Operands& o, const Scales& sc, int s, auto k_const, auto between) {
        constexpr int K = decltype(k_const)::value;
        const bool in_row = block0 + s * KB + half + 2 * K < nb;
        constexpr int SA = 2 * (K % 2);
        if constexpr (FMT == kFmt4) {
            uint32_t sa[MT], sb[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) sa[i] = in_row ? sc.a[i][K / 2] : 0u;
#pragma unroll
            for (int j = 0; j < NT; ++j) sb[j] = in_row ? sc.b[j][K / 2] : 0x7f7f7f7fu;
#pragma unroll
            for (int n = 0; n < kProducts; ++n) {
                const int i = n % MT, j = n / MT;
                acc[i][j] = mfma_mx32<SA>(operand4(o.a[i]), operand4(o.b[j][0]), acc[i][j], sa[i], sb[j]);
                between(n);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            float f[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t b = in_row ? sc.a[i][K / 2] >> (8 * SA) & 255u : 0u;
                odd |= odd_scale(b) ? 1u : 0u;
                f[i] = plain_scale(b) ? scale_value(b) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const f16x8 w = decode8(o.a[i][e], f[i]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        acc[i][j] = mfma32x32x16(w, as_f16x8(o.b[j][e]), acc[i][j]);
                        between((e * MT + i) * NT + j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
        }
    };
    // The odd blocks of this wave's rows and part, found 16 blocks of all rows at a time and taken one at a time: both halves of the
    // wave take one block, in two instructions.
    auto add_odd = [&]() {
        if constexpr (FMT != kFmt4) {
            size_t row[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) row[i] = (size_t)min(m0 + (wm * MT + i) * 32 + l32, g.out - 1) * nb;
            for (int c = 0; c < blocks; c += 16) {
                uint32_t here = 0u;   // a bit a block
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const u32x4 v = load_bytes16(g.ws, row[i] + block0 + c, (int64_t)g.out * nb);
#pragma unroll
                    for (int k = 0; k < 16; ++k) here |= c + k < blocks && odd_scale(v[k / 4] >> 8 * (k % 4) & 255u) ? 1u << k : 0u;
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) here |= (uint32_t)__shfl_xor((int)here, o, kWave);
                for (uint32_t left = (uint32_t)__builtin_amdgcn_readfirstlane((int)here); left != 0; left &= left - 1) {
                    const int b = block0 + c + __builtin_ctz(left);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const size_t at = row[i] + b;
                        const uint32_t s = g.ws[at];
                        const bool mine = odd_scale(s);
                        if (__ballot(mine) == 0) continue;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const f16* xr = reinterpret_cast<const f16*>(g.x) +
                                            ((size_t)min(n0 + (wn * NT + j) * 32 + l32, g.T - 1) * nb + b) * kMxBlock + 8 * half;
                            f32x16 d = {};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t w = *reinterpret_cast<const uint32_t*>(g.w + at * kMxBlockBytes + 4 * (2 * e + half));
                                d = mfma32x32x16(decode8(mine ? w : 0u, 1.f), as_f16x8(load16(xr + 16 * e)), d);
                            }
                            pin(d);
#pragma unroll
                            for (int r = 0; r < 16; ++r)   // rows without the block have sums of 0
                                acc[i][j][r] += odd_sum(d[r], (uint32_t)__shfl(mine ? (int)s : 127, 8 * (r / 4) + 4 * half + r % 4, kWave));
                        }
                    }
                }
            }
        }
    };

    // This wave's loads of a stage have landed (those of the STAGES - 2 behind it may be in flight), and the barrier says so for
    // all; every wave has read the stage before it, whose place is loaded next.  Loads go on past the last stage, unused.
    auto arrive = [&]() { asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(L::kLoads * (STAGES - 2)) : "memory"); };
    auto place = [&](int s) { return lds + s % STAGES * L::kStage; };

    Operands o[2];
    Scales cur, nxt;
    arrive();
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(o[0], place(0), 0, q);
    read_scales(cur, 0);
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) load(STAGES - 1, j);
    half_scales(cur);
    static_assert(L::kSteps == 2 || L::kSteps == 4);
    auto read_next = [&](Operands& to, const char* from, int k, int n) {
#pragma unroll
        for (int q = n * kReads / kProducts; q < (n + 1) * kReads / kProducts; ++q) read(to, from, k, q);
    };
    auto stage = [&](int s) {
        using std::integral_constant;
        multiply(o[0], cur, s, integral_constant<int, 0>{}, [&](int n) { read_next(o[1], place(s), 1, n); });
        if constexpr (L::kSteps == 4) {
            multiply(o[1], cur, s, integral_constant<int, 1>{}, [&](int n) { read_next(o[0], place(s), 2, n); });
            multiply(o[0], cur, s, integral_constant<int, 2>{}, [&](int n) { read_next(o[1], place(s), 3, n); });
        }
        arrive();   // stage s + 1
        read_scales(nxt, s + 1);
        multiply(o[1], cur, s, integral_constant<int, L::kSteps - 1>{}, [&](int n) {
            read_next(o[0], place(s + 1), 0, n);
#pragma unroll
            for (int j = n * L::kLoads / kProducts; j < (n + 1) * L::kLoads / kProducts; ++j) load(s + STAGES, j);
        });
        cur = nxt;
        half_scales(cur);
    };
    for (int c = 0; c * L::kChunkStages < n_stage; ++c) {
        // the scales of the chunk after this one: their place was last read in the chunk before it
        if constexpr (STRAIGHT) {
            send_scales(c + 1);
        } else {
            keep_scales(sc, c + 1);
            load_scales(c + 2, sc);
        }
#pragma unroll
        for (int t = 0; t < L::kChunkStages; ++t) {
            if (t > 0 && c * L::kChunkStages + t >= n_stage) break;
            stage(c * L::kChunkStages + t);
        }
    }
    // nothing is on its way into LDS, and nobody reads the stages
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if constexpr (FMT != kFmt4) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = no_infinity(acc[i][j][r]);
        if (__ballot(odd != 0u) != 0) add_odd();
    }
    char* const turn = lds + wave * 32 * L::kEpiRow;
    constexpr int kLanes = MT * 4;   // a token
    const int row = m0 + wm * MT * 32 + 8 * (lane % kLanes), left = g.out - row;
    const bool vec = g.out % 8 == 0;
    float bias[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) bias[q] = !PART && g.bias != nullptr && q < left ? (float)g.bias[row + q] : 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(turn + l32 * L::kEpiRow + (i * 32 + 8 * q + 4 * half) * 4) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        __builtin_amdgcn_wave_barrier();
        const char* from = turn + lane / kLanes * L::kEpiRow + (lane % kLanes) * 32;
        int token = n0 + (wn * NT + j) * 32 + lane / kLanes;
#pragma unroll 1
        for (int t = 0; t < 32; t += 64 / kLanes, token += 64 / kLanes, from += 64 / kLanes * L::kEpiRow) {
            const f32x4 z0 = *reinterpret_cast<const f32x4*>(from), z1 = *reinterpret_cast<const f32x4*>(from + 16);
            if (token >= g.T || left <= 0) continue;
            if constexpr (PART) {
                float* to = g.part + ((size_t)split * g.T + token) * g.op + row;
                *reinterpret_cast<f32x4*>(to) = z0;
                if (left > 4) *reinterpret_cast<f32x4*>(to + 4) = z1;
            } else {
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = (q < 4 ? z0[q & 3] : z1[q & 3]) + bias[q];
                act_values(g.act, v);
                const size_t at = (size_t)token * g.out + row;
                if (vec) {
                    if (g.residual != nullptr) {
                        const f16x8 res = as_f16x8(load16(g.residual + at));
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] += (float)res[q];
                    }
                    f16x8 y;
#pragma unroll
                    for (int q = 0; q < 8; ++q) y[q] = (f16)v[q];
                    *reinterpret_cast<u32x4*>(g.y + at) = as_u32x4(y);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if (q < left) {
                            if (g.residual != nullptr) v[q] += (float)g.residual[at + q];
                            g.y[at + q] = (f16)v[q];
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Tiles of W's rows x tokens: 256 x 256 (x fp16: 256 x 128), 128 x 128, 128 x 64.
enum TileKind { kBig, kSmall, kNarrowTile };
constexpr int64_t kNarrow = 64;
struct GemmPlan {
    TileKind kind;
    int splits;
};

template <int FMT, int WM, int WN, int MT, int NT, int KB, int STAGES, bool PART>
hipError_t launch_tile(GemmArgs& g, bool straight, hipStream_t stream) {
    using L = Tile<FMT, WM, WN, MT, NT, KB, STAGES>;
    g.tiles_m = (g.out + L::kM - 1) / L::kM;
    g.tiles_n = (g.T + L::kN - 1) / L::kN;
    auto kern = straight ? mx4_gemm_kernel<FMT, WM, WN, MT, NT, KB, STAGES, PART, true>
                         : mx4_gemm_kernel<FMT, WM, WN, MT, NT, KB, STAGES, PART, false>;
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, L::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits)), dim3(L::kThreads), L::kLds, stream, g);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_plan(const GemmPlan& p, GemmArgs& g, hipStream_t stream) {
    // scales in 16-byte pieces that start on 16 bytes
    const bool straight = g.nb % kChunkBlocks == 0 && (uintptr_t)g.ws % 16 == 0 && (uintptr_t)g.xs % 16 == 0;
    constexpr bool kX4 = FMT == kFmt4;
    if (p.kind == kBig) {   // 8 waves of 128 x 64, stages of 256 inputs; x fp16: 4 waves of 128 x 64, stages of 128
        if constexpr (kX4) return launch_tile<FMT, 2, 4, 4, 2, 8, 2, false>(g, straight, stream);
        else return launch_tile<FMT, 2, 2, 4, 2, 4, 3, false>(g, straight, stream);
    }
    if (p.kind == kSmall) {   // 8 waves of 64 x 32
        constexpr int kStages = kX4 ? 4 : 3;
        return p.splits > 1 ? launch_tile<FMT, 2, 4, 2, 1, 4, kStages, true>(g, straight, stream)
                            : launch_tile<FMT, 2, 4, 2, 1, 4, kStages, false>(g, straight, stream);
    }
    constexpr int kStages = kX4 ? 5 : 4;   // 8 waves of 32 x 32
    return p.splits > 1 ? launch_tile<FMT, 4, 2, 1, 1, 4, kStages, true>(g, straight, stream)
                        : launch_tile<FMT, 4, 2, 1, 1, 4, kStages, false>(g, straight, stream);
}

int64_t round4(int64_t v) { return (v + 3) / 4 * 4; }

constexpr int kSmallRows = 128;   // of W, in both small tiles
constexpr int kFill = 256;        // workgroups that fill the chip: a tile's sum is split as long as there are no more
int max_splits(int64_t in) { return (int)std::max<int64_t>(1, in / (2 * kChunkBlocks * kMxBlock)); }

// Up to 64 tokens the narrow tile (128 x 128 at 64 tokens, 8192 -> 28672: 71 us against 43, x in MX4 28 against 26); also where
// narrow tiles of whole, short rows fit the chip at once, which then needs fewer parts.  Narrow | 128 x 128, us, x fp16, x in MX4:
//   4096 -> 4096: 128 tokens 18 | 21, 15 | 15, 400 tokens 24 | 32, 13 | 18    4096 -> 11008: 128 tokens 22 | 28, 13 | 17
//   past the chip, 130 tokens: 39 | 33, 17 | 13    long rows, 11008 -> 4096, 300 tokens: 54.5 | 53.6, 37 | 27
// The big tile from three quarters of the chip on: fewer leave CUs without work for a whole tile's time.
GemmPlan gemm_plan(bool x_mx4, int64_t out, int64_t in, int64_t batch) {
    const int64_t rows = (out + kSmallRows - 1) / kSmallRows, narrow = rows * ((batch + kNarrow - 1) / kNarrow);
    const int64_t big = (out + 255) / 256 * (x_mx4 ? (batch + 255) / 256 : (batch + 127) / 128);
    GemmPlan p;
    p.kind = batch <= kNarrow || (in <= 4096 && narrow <= kFill) ? kNarrowTile : big >= kFill * 3 / 4 ? kBig : kSmall;
    const int64_t tiles = p.kind == kNarrowTile ? narrow : rows * ((batch + 127) / 128);
    p.splits = p.kind == kBig ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(max_splits(in), kFill / tiles));
    // no empty part
    const int64_t chunks = (in / kMxBlock + kChunkBlocks - 1) / kChunkBlocks;
    while (p.splits > 1 && (chunks + p.splits - 1) / p.splits * (p.splits - 1) >= chunks) --p.splits;
    return p;
}

}  // namespace

// Against mx4_linear.hip's kernel, which walks a row from end to end in one workgroup (x fp16 | x MX4, us, its time first):
//   33 tokens   8192 -> 1024: 25 11 | 15 9    4096 -> 2048: 14 11 | 9 9    2048 -> 4096: 9 11 | 6 8
//   17 tokens   8192 -> 28672: 51 41 | 39 24    4096 -> 16384: 16.9 17.1 (x fp16)    8192 -> 11008, 32 tokens, x in MX4: 22 17
//   x in MX4, 1 token   8192 -> 28672: 28 22    8192 -> 16384: 17 18    4096 -> 28672: 15 14
bool mx4_gemm_serves(bool x_mx4, int64_t out, int64_t in, int64_t batch) {
    // load_bytes16's least array: the scales of W, and of x where they are read
    if ((x_mx4 ? std::min(out, batch) : out) * (in / kMxBlock) < 16) return false;
    return batch > kNarrow || (batch > 32 && (in >= 4096 || out * in >= (int64_t)1 << 25)) ||
           (batch > 16 && out * in > (int64_t)1 << 26) || (x_mx4 && out * in > (int64_t)1 << 27);
}

int64_t mx4_gemm_part_bytes(int64_t out, int64_t in, int64_t batch) {
    // splits <= max_splits and splits * token tiles <= kFill / tiles_m: the most of any batch up to this one
    const int64_t tiles_m = (out + kSmallRows - 1) / kSmallRows, cap = std::max<int64_t>(1, kFill / tiles_m) * 128;
    return std::min(max_splits(in) * batch, cap) * round4(out) * (int64_t)sizeof(float);
}

hipError_t launch_mx4_gemm(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* part, int64_t out, int64_t in,
                           int64_t batch, hipStream_t stream) {
    const GemmPlan p = gemm_plan(x.scales != nullptr, out, in, batch);
    GemmArgs g = {};
    g.w = static_cast<const uint8_t*>(codes);
    g.ws = static_cast<const uint8_t*>(scales);
    g.x = static_cast<const uint8_t*>(x.x);
    g.xs = static_cast<const uint8_t*>(x.scales);
    g.bias = static_cast<const f16*>(e.bias[0]);
    g.residual = static_cast<const f16*>(e.residual);
    g.y = static_cast<f16*>(e.y);
    g.part = static_cast<float*>(part);
    g.act = e.act;
    g.out = (int)out;
    g.T = (int)batch;
    g.nb = (int)(in / kMxBlock);
    g.op = (int)round4(out);
    g.splits = p.splits;
    g.chunks = (g.nb + kChunkBlocks - 1) / kChunkBlocks;
    const hipError_t r = x.scales != nullptr ? launch_plan<kFmt4>(p, g, stream) : launch_plan<kFmt16>(p, g, stream);
    if (r != hipSuccess || p.splits == 1) return r;
    return launch_finish(1, g.part, nullptr, e, out, g.op, batch, p.splits, BiasSum{}, stream);
}

}  // namespace aqlm

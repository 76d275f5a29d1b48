// C ABI of the fused products and their backward passes (declared in include/aqlm.h):
// argument checks on the host, then the launches on the caller's stream.
//
// Forward at batch 1..16 the codes are multiplied as they are decoded, in one launch; 2x8, 1x16
// and 4x8 g16 at up to some hundreds of tokens likewise, with partial sums in the workspace
// (skinny.hip), and so are their gradients (skinny_back.hip).  Otherwise the products run in passes:
// the weights decoded once into the workspace as fp16, then a dense matrix-core product over them.  Forward, the decoded rows are padded to whole
// steps of 64 inputs; backward, they are written transposed (dx = dz W sums over the rows
// of W).  With one codebook (M = 1) a codeword is exactly an fp16 weight: forward, the row
// scale then goes into the fp32 epilogue and the weights are not rounded at all; backward,
// it goes into dz, which is rounded to fp16 anyway (where dz is dy as it is, it stays with the
// weights).  With several codebooks a weight is the fp32 sum times the scale, rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/aqlm.h"
#include "act_bias.h"
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_validate.h"

namespace aqlm {

static_assert((int)kActNone == AQLM_ACT_NONE && (int)kActRelu == AQLM_ACT_RELU && (int)kActSilu == AQLM_ACT_SILU &&
                  (int)kActGelu == AQLM_ACT_GELU && (int)kActGeluTanh == AQLM_ACT_GELU_TANH,
              "activation codes");

namespace {

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Parts of a workspace, each 256-byte aligned.  Sizes are added in 128 bits: `total` is -1
// once they leave int64.
struct Parts {
    int64_t total = 0;
    int64_t add(int64_t a, int64_t b, int64_t c) {   // a * b * c bytes; its offset
        const int64_t at = total;
        if (total < 0) return 0;
        const __int128 end = (__int128)total + ((__int128)a * b * c + 255) / 256 * 256;
        total = end > (__int128)INT64_MAX / 2 ? -1 : (int64_t)end;
        return at;
    }
};

struct ForwardPlan {
    int64_t kp = 0, w[2] = {0, 0}, xp = 0, partial = 0, bytes = 0;
    bool pad = false, skinny = false;
};

// n layers: their weights as rows of kp inputs, then x padded to them.
ForwardPlan forward_plan(int n, const GenericScheme& sc, int64_t out, int64_t in, int64_t batch) {
    ForwardPlan p;
    Parts parts;
    p.kp = round_up(in, 64);
    p.pad = p.kp != in;
    if (out == 0 || batch <= AQLM_GEMV_MAX_BATCH) return p;   // one launch straight from the codes
    if (skinny_serves(sc, n, out, in, batch)) {
        p.skinny = true;
        p.bytes = skinny_partial_bytes(sc, n, out, in, batch);
        return p;
    }
    for (int l = 0; l < n; ++l) p.w[l] = parts.add(out, p.kp, 2);
    if (p.pad) p.xp = parts.add(batch, p.kp, 2);
    p.partial = parts.add(dense_partial_bytes(n, out, p.kp, batch), 1, 1);
    p.bytes = parts.total;
    // not less than the batches below need that are served straight from the codes
    for (int64_t t : {kSkinnyMaxBatch1x16Few, skinny_max_batch(sc, n)})
        if (p.bytes >= 0 && t < batch && skinny_serves(sc, n, out, in, t))
            p.bytes = std::max(p.bytes, skinny_partial_bytes(sc, n, out, in, t));
    return p;
}

struct BackwardPlan {
    int64_t op = 0, wt = 0, dz = 0, partial = 0, parts = 0, bytes = 0;
    bool grad = false;   // a pass over dy writes dz (else the product takes dy itself)
    bool skinny = false;
};

BackwardPlan backward_plan(int n, int act, const GenericScheme& sc, int64_t out, int64_t in, int64_t batch) {
    BackwardPlan p;
    Parts parts;
    p.op = round_up(out, 64);
    auto add_dz = [&]() {   // with its levels and units behind it (act_launch.h)
        p.dz = parts.add(batch, n * p.op, 2);
        parts.add(batch, n * grad_level_cols(p.op), 1);
        parts.add(batch, 4, 1);
    };
    p.skinny = skinny_back_serves(sc, out, in, batch);
    if (p.skinny) {
        p.grad = !skinny_back_grads(sc, n, out, in, batch);
        if (p.grad) {
            add_dz();
            p.partial = parts.add(grad_chunks_room(out, batch), n * out, 4);
        }
        p.parts = out == 0 || batch == 0 ? 0 : parts.add(skinny_back_partial_bytes(sc, n, out, in, batch), 1, 1);
        p.bytes = (out == 0 || batch == 0) ? 0 : parts.total;
        return p;
    }
    p.grad = n > 1 || act != kActNone || p.op != out;
    p.wt = parts.add(in, n * p.op, 2);
    add_dz();
    p.partial = parts.add(grad_chunks_room(out, batch), n * out, 4);
    p.parts = parts.add(dense_partial_bytes(1, in, n * p.op, batch), 1, 1);
    p.bytes = (out == 0 || batch == 0) ? 0 : parts.total;
    const int64_t direct = sc.M == 1 ? kSkinnyBackMaxBatch1x16 : sc.M == 2 ? kSkinnyBackMaxBatch2x8 : kSkinnyBackMaxBatch4x8;
    if (p.bytes > 0 && direct < batch && skinny_back_serves(sc, out, in, direct))
        p.bytes = std::max(p.bytes, backward_plan(n, act, sc, out, in, direct).bytes);
    return p;
}

bool act_ok(int act) { return act >= AQLM_ACT_NONE && act <= AQLM_ACT_GELU_TANH; }

// Scheme and sizes of the calls of this file, apart from any pointer.
int check_sizes(int act, int M, int B, int g, int64_t out, int64_t in, int64_t batch) {
    if (!generic_scheme_ok(M, B, g)) return AQLM_ERR_SCHEME;
    if (!act_ok(act)) return AQLM_ERR_ACT;
    if (in < 1 || in > AQLM_MAX_IN || in % g != 0) return AQLM_ERR_SHAPE;
    if (out < 0 || out > AQLM_ACT_MAX_OUT || batch < 0 || batch > (int64_t)INT32_MAX - 256) return AQLM_ERR_SHAPE;
    const int64_t kp = round_up(in, 64), op = round_up(out, 64);
    // decoded pieces, code groups, output tiles and gradient workgroups are counted in 32 bits
    if ((uint64_t)op * (uint64_t)(kp / 8) > UINT32_MAX || (uint64_t)out * (uint64_t)(in / g) > UINT32_MAX)
        return AQLM_ERR_SHAPE;
    const int64_t bt = (batch + 255) / 256, wide = op > kp ? op : kp;
    if ((wide / 64 + 8) * bt > INT32_MAX / 2 || grad_chunks(out, batch) * (op / 512 + 1) > INT32_MAX) return AQLM_ERR_SHAPE;
    return AQLM_OK;
}

int check_layers(const ActLayers& L) {
    for (int l = 0; l < L.n; ++l) {
        if (!L.codes[l] || !L.codebooks[l] || !L.scales[l]) return AQLM_ERR_NULL;
        if (!aligned(L.codes[l], 16) || !aligned(L.codebooks[l], 16) || !aligned(L.scales[l], 2)) return AQLM_ERR_ALIGN;
    }
    return AQLM_OK;
}

int check_workspace(const void* workspace, int64_t have, int64_t need) {
    if (need < 0) return AQLM_ERR_SHAPE;   // more than int64 counts
    if (need == 0) return AQLM_OK;
    if (!workspace) return AQLM_ERR_NULL;
    if (!aligned(workspace, 16)) return AQLM_ERR_ALIGN;
    return have < need ? AQLM_ERR_SHAPE : AQLM_OK;
}

// Two host arrays' entries, or NULL for an absent array.
template <class T>
T entry(T const* a, int l) { return a ? a[l] : nullptr; }

int forward(const ActLayers& L, const void* x, const Epilogue& epi, void* workspace, int64_t workspace_bytes, int M,
            int B, int g, int64_t out, int64_t in, int64_t batch, void* stream) {
    const int st = check_sizes(epi.act, M, B, g, out, in, batch);
    if (st != AQLM_OK) return st;
    if (out == 0 || batch == 0) return AQLM_OK;
    const int lt = check_layers(L);
    if (lt != AQLM_OK) return lt;
    if (!x || !epi.y) return AQLM_ERR_NULL;
    if (!aligned(x, 16) || !aligned(epi.y, 16) || !aligned(epi.residual, 16)) return AQLM_ERR_ALIGN;
    for (int l = 0; l < L.n; ++l)
        if (!aligned(epi.z[l], 16) || !aligned(epi.bias[l], 2)) return AQLM_ERR_ALIGN;
    const ForwardPlan p = forward_plan(L.n, GenericScheme{M, B, g}, out, in, batch);
    const int wt = check_workspace(workspace, workspace_bytes, p.bytes);
    if (wt != AQLM_OK) return wt;
    const hipStream_t s = (hipStream_t)stream;
    if (batch <= AQLM_GEMV_MAX_BATCH)
        return finish(launch_gemv_act(GenericScheme{M, B, g}, L, x, epi, out, in, batch, s));
    if (p.skinny)
        return finish(launch_skinny(GenericScheme{M, B, g}, L, x, workspace, epi, out, in, batch, s));
    char* base = static_cast<char*>(workspace);
    void* w[2] = {base + p.w[0], base + p.w[1]};
    const WeightScale ws = M == 1 ? WeightScale::kNone : WeightScale::kFull;
    int r = finish(launch_decode_rows(GenericScheme{M, B, g}, L, ws, w, out, in, p.kp, s));
    if (r != AQLM_OK) return r;
    if (p.pad) {
        r = finish(launch_pad_rows(x, base + p.xp, batch, in, p.kp, s));
        if (r != AQLM_OK) return r;
        x = base + p.xp;
    }
    return finish(launch_gemm_dense_act(x, w, ws == WeightScale::kNone ? L.scales : nullptr, L.n, epi, base + p.partial, out,
                                        p.kp, batch, BiasSum{}, s));
}

int backward(const ActLayers& L, const void* dy, const void* const* z, void* dx, void* const* dbias, int act,
             void* workspace, int64_t workspace_bytes, int M, int B, int g, int64_t out, int64_t in, int64_t batch,
             void* stream) {
    const int st = check_sizes(act, M, B, g, out, in, batch);
    if (st != AQLM_OK) return st;
    const bool want_bias = dbias[0] != nullptr;
    if (L.n > 1 && (dbias[1] != nullptr) != want_bias) return AQLM_ERR_NULL;   // both sums or none
    for (int l = 0; l < L.n; ++l)
        if (!aligned(dbias[l], 2)) return AQLM_ERR_ALIGN;
    const hipStream_t s = (hipStream_t)stream;
    if (batch == 0) {   // sums over no tokens
        for (int l = 0; l < L.n && want_bias && out > 0; ++l) {
            const int r = finish(launch_zero16(dbias[l], out, s));
            if (r != AQLM_OK) return r;
        }
        return AQLM_OK;
    }
    if (!dx) return AQLM_ERR_NULL;
    if (!aligned(dx, 16)) return AQLM_ERR_ALIGN;
    if (out == 0) return finish(launch_zero16(dx, batch * in, s));   // a sum over no rows
    const int lt = check_layers(L);
    if (lt != AQLM_OK) return lt;
    if (!dy) return AQLM_ERR_NULL;
    if (!aligned(dy, 16)) return AQLM_ERR_ALIGN;
    for (int l = 0; l < L.n; ++l) {
        if ((L.n > 1 || act != kActNone) && !z[l]) return AQLM_ERR_NULL;
        if (!aligned(z[l], 16)) return AQLM_ERR_ALIGN;
    }
    const BackwardPlan p = backward_plan(L.n, act, GenericScheme{M, B, g}, out, in, batch);
    const int wt = check_workspace(workspace, workspace_bytes, p.bytes);
    if (wt != AQLM_OK) return wt;
    char* base = static_cast<char*>(workspace);
    if (p.skinny && !p.grad) {   // two launches
        const BackGrads grads = {dy, {z[0], z[1]}, {dbias[0], dbias[1]}, act};
        return finish(launch_skinny_back(GenericScheme{M, B, g}, L, nullptr, &grads, base + p.parts, dx, out, in, p.op,
                                         batch, BiasSum{}, s));
    }
    // the scale goes into dz where the codewords are multiplied as they are
    const WeightScale ws = (p.skinny || (M == 1 && p.grad)) ? WeightScale::kNone : WeightScale::kFull;
    if (p.grad || want_bias) {
        const int r = finish(launch_act_grad(dy, z, ws == WeightScale::kNone ? L.scales : nullptr, L.n, act,
                                             p.grad ? base + p.dz : nullptr,
                                             want_bias ? reinterpret_cast<float*>(base + p.partial) : nullptr, out, p.op,
                                             batch, s));
        if (r != AQLM_OK) return r;
    }
    BiasSum bias = {};   // added by the launch that finishes dx, or by one of its own
    if (want_bias)
        bias = BiasSum{reinterpret_cast<const float*>(base + p.partial),
                       {static_cast<f16*>(dbias[0]), static_cast<f16*>(dbias[1])}, L.n, (int)out, (int)grad_chunks(out, batch)};
    if (p.skinny)
        return finish(launch_skinny_back(GenericScheme{M, B, g}, L, base + p.dz, nullptr, base + p.parts, dx, out, in, p.op, batch,
                                         bias, s));
    ActLayers decoded = L;
    if (p.grad) decoded.grads = {base + p.dz, batch};
    const int r = finish(launch_decode_transposed(GenericScheme{M, B, g}, decoded, ws, base + p.wt, out, in, p.op, s));
    if (r != AQLM_OK) return r;
    const void* wt16 = base + p.wt;
    Epilogue plain = {{nullptr, nullptr}, nullptr, {nullptr, nullptr}, dx, kActNone};
    if (p.grad) plain.units = grad_units(base + p.dz, L.n, p.op, batch);
    return finish(launch_gemm_dense_act(p.grad ? base + p.dz : dy, &wt16, nullptr, 1, plain, base + p.parts, in,
                                        L.n * p.op, batch, bias, s));
}

// The slice-list product of n layers at batch 1.
int lists_forward(int n, const void* const* tables, const void* const* entries, const int64_t* entries_bytes,
                  const void* const* codebooks, const void* const* scales, const void* x, const Epilogue& epi,
                  void* workspace, int64_t workspace_bytes, int M, int B, int g, int64_t out, int64_t in, int64_t batch,
                  void* stream) {
    const int st = validate_lists(M, B, g, out, in);
    if (st != AQLM_OK) return st;
    if (!act_ok(epi.act)) return AQLM_ERR_ACT;
    if (batch < 0 || batch > 1 || workspace_bytes < 0) return AQLM_ERR_SHAPE;
    if (out == 0 || batch == 0) return AQLM_OK;
    if (!x || !epi.y || !workspace) return AQLM_ERR_NULL;
    ListsLayers L{};
    L.n = n;
    const int64_t part = lists_workspace_bytes_aligned(out, in);
    for (int l = 0; l < n; ++l) {
        if (entries_bytes[l] < 0) return AQLM_ERR_SHAPE;
        if (!tables[l] || !entries[l] || !codebooks[l] || !scales[l]) return AQLM_ERR_NULL;
        if (!aligned(tables[l], 16) || !aligned(entries[l], 16) || !aligned(codebooks[l], 16) || !aligned(scales[l], 2) ||
            !aligned(epi.z[l], 16) || !aligned(epi.bias[l], 2))
            return AQLM_ERR_ALIGN;
        L.table[l] = static_cast<const uint32_t*>(tables[l]);
        L.entries[l] = static_cast<const uint32_t*>(entries[l]);
        L.cap[l] = (uint64_t)(entries_bytes[l] / 256);
        L.codebook[l] = codebooks[l];
        L.scales[l] = scales[l];
        L.out[l] = (int)out;
        L.partial[l] = reinterpret_cast<float*>(static_cast<char*>(workspace) + l * part);
    }
    if (!aligned(x, 16) || !aligned(epi.y, 16) || !aligned(epi.residual, 16) || !aligned(workspace, 16))
        return AQLM_ERR_ALIGN;
    if (workspace_bytes < (n - 1) * part + lists_workspace_bytes(out, in)) return AQLM_ERR_SHAPE;
    return finish(launch_lists_act(L, x, epi, in, (hipStream_t)stream));
}

int workspace_bytes_of(int n, bool back, int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes) {
    if (!bytes) return AQLM_ERR_NULL;
    const int st = check_sizes(AQLM_ACT_RELU, M, B, g, out, in, batch);
    if (st != AQLM_OK) return st;
    const int64_t need = back ? backward_plan(n, AQLM_ACT_RELU, GenericScheme{M, B, g}, out, in, batch).bytes
                              : forward_plan(n, GenericScheme{M, B, g}, out, in, batch).bytes;
    if (need < 0) return AQLM_ERR_SHAPE;
    *bytes = need;
    return AQLM_OK;
}

}  // namespace
}  // namespace aqlm

using namespace aqlm;

extern "C" {

int aqlm_linear_act_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes) {
    return workspace_bytes_of(1, false, M, B, g, out, in, batch, bytes);
}

int aqlm_gated_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes) {
    return workspace_bytes_of(2, false, M, B, g, out, in, batch, bytes);
}

int aqlm_linear_act_backward_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch,
                                             int64_t* bytes) {
    return workspace_bytes_of(1, true, M, B, g, out, in, batch, bytes);
}

int aqlm_gated_backward_workspace_bytes(int M, int B, int g, int64_t out, int64_t in, int64_t batch, int64_t* bytes) {
    return workspace_bytes_of(2, true, M, B, g, out, in, batch, bytes);
}

int aqlm_linear_act(const void* codes, const void* codebooks, const void* scales, const void* x, const void* bias,
                    const void* residual, void* z, void* y, void* workspace, int64_t workspace_bytes, int act, int M,
                    int B, int g, int64_t out, int64_t in, int64_t batch, void* stream) {
    const ActLayers L = {{codes, nullptr}, {codebooks, nullptr}, {scales, nullptr}, 1};
    const Epilogue epi = {{bias, nullptr}, residual, {z, nullptr}, y, act};
    return forward(L, x, epi, workspace, workspace_bytes, M, B, g, out, in, batch, stream);
}

int aqlm_gated(const void* const* codes, const void* const* codebooks, const void* const* scales, const void* x,
               const void* const* bias, void* const* z, void* y, void* workspace, int64_t workspace_bytes, int act,
               int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream) {
    if (!codes || !codebooks || !scales) return AQLM_ERR_NULL;
    const ActLayers L = {{codes[0], codes[1]}, {codebooks[0], codebooks[1]}, {scales[0], scales[1]}, 2};
    const Epilogue epi = {{entry(bias, 0), entry(bias, 1)}, nullptr, {entry(z, 0), entry(z, 1)}, y, act};
    return forward(L, x, epi, workspace, workspace_bytes, M, B, g, out, in, batch, stream);
}

int aqlm_linear_act_lists(const void* table, const void* entries, int64_t entries_bytes, const void* codebooks,
                          const void* scales, const void* x, const void* bias, const void* residual, void* z, void* y,
                          void* workspace, int64_t workspace_bytes, int act, int M, int B, int g, int64_t out,
                          int64_t in, int64_t batch, void* stream) {
    const Epilogue epi = {{bias, nullptr}, residual, {z, nullptr}, y, act};
    return lists_forward(1, &table, &entries, &entries_bytes, &codebooks, &scales, x, epi, workspace, workspace_bytes, M,
                         B, g, out, in, batch, stream);
}

int aqlm_gated_lists(const void* const* tables, const void* const* entries, const int64_t* entries_bytes,
                     const void* const* codebooks, const void* const* scales, const void* x, const void* const* bias,
                     void* const* z, void* y, void* workspace, int64_t workspace_bytes, int act, int M, int B, int g,
                     int64_t out, int64_t in, int64_t batch, void* stream) {
    if (!tables || !entries || !entries_bytes || !codebooks || !scales) return AQLM_ERR_NULL;
    const Epilogue epi = {{entry(bias, 0), entry(bias, 1)}, nullptr, {entry(z, 0), entry(z, 1)}, y, act};
    return lists_forward(2, tables, entries, entries_bytes, codebooks, scales, x, epi, workspace, workspace_bytes, M, B,
                         g, out, in, batch, stream);
}

int aqlm_linear_act_backward(const void* codes, const void* codebooks, const void* scales, const void* dy,
                             const void* z, void* dx, void* dbias, void* workspace, int64_t workspace_bytes, int act,
                             int M, int B, int g, int64_t out, int64_t in, int64_t batch, void* stream) {
    const ActLayers L = {{codes, nullptr}, {codebooks, nullptr}, {scales, nullptr}, 1};
    const void* zs[2] = {z, nullptr};
    void* db[2] = {dbias, nullptr};
    return backward(L, dy, zs, dx, db, act, workspace, workspace_bytes, M, B, g, out, in, batch, stream);
}

int aqlm_gated_backward(const void* const* codes, const void* const* codebooks, const void* const* scales,
                        const void* dy, const void* const* z, void* dx, void* const* dbias, void* workspace,
                        int64_t workspace_bytes, int act, int M, int B, int g, int64_t out, int64_t in, int64_t batch,
                        void* stream) {
    if (!codes || !codebooks || !scales || !z) return AQLM_ERR_NULL;
    const ActLayers L = {{codes[0], codes[1]}, {codebooks[0], codebooks[1]}, {scales[0], scales[1]}, 2};
    const void* zs[2] = {z[0], z[1]};
    void* db[2] = {entry(dbias, 0), entry(dbias, 1)};
    return backward(L, dy, zs, dx, db, act, workspace, workspace_bytes, M, B, g, out, in, batch, stream);
}

}  // extern "C"

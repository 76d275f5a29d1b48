// Host-only driver of the argument checks and workspace plans of the fused products
// (act_api.hip), built as api_validation_driver.hip is and on top of its stubs
// (tests/test_fused_host_sanitizers.py).  Host arrays have exactly two entries, sizes
// reach INT64_MIN/MAX, and no stub dereferences a "device" pointer.
#define main api_validation_main
#include "api_validation_driver.hip"
#undef main

#include "../../extreme_weight_quantization_amd/csrc/act_bias.h"
#include "../../extreme_weight_quantization_amd/csrc/act_launch.h"

namespace {
bool g_skinny = false, g_grads = false;
}

namespace aqlm {
hipError_t launch_decode_rows(const GenericScheme&, const ActLayers&, WeightScale, void* const*, int64_t, int64_t,
                              int64_t, hipStream_t) { return stub(); }
hipError_t launch_decode_transposed(const GenericScheme&, const ActLayers&, WeightScale, void*, int64_t, int64_t,
                                    int64_t, hipStream_t) { return stub(); }
hipError_t launch_pad_rows(const void*, void*, int64_t, int64_t, int64_t, hipStream_t) { return stub(); }
hipError_t launch_zero16(void*, int64_t, hipStream_t) { return stub(); }
int64_t dense_partial_bytes(int n, int64_t out, int64_t, int64_t batch) { return 4 * n * out * batch; }
hipError_t launch_gemm_dense_act(const void*, const void* const*, const void* const*, int, const Epilogue&, void*,
                                 int64_t, int64_t, int64_t, const BiasSum&, hipStream_t) { return stub(); }
int64_t grad_chunks(int64_t, int64_t batch) { return (batch + 3) / 4; }
hipError_t launch_act_grad(const void*, const void* const*, const void* const*, int, int, void*, float*, int64_t,
                           int64_t, int64_t, hipStream_t) { return stub(); }
hipError_t launch_gemv_act(const GenericScheme&, const ActLayers&, const void*, const Epilogue&, int64_t, int64_t,
                           int64_t, hipStream_t) { return stub(); }
bool skinny_serves(const GenericScheme&, int, int64_t, int64_t, int64_t) { return g_skinny; }
int64_t skinny_partial_bytes(const GenericScheme&, int n, int64_t out, int64_t, int64_t batch) { return 4 * n * out * batch; }
hipError_t launch_skinny(const GenericScheme&, const ActLayers&, const void*, void*, const Epilogue&, int64_t, int64_t,
                         int64_t, hipStream_t) { return stub(); }
bool skinny_back_serves(const GenericScheme&, int64_t, int64_t, int64_t) { return g_skinny; }
int64_t skinny_back_partial_bytes(const GenericScheme&, int n, int64_t, int64_t in, int64_t batch) { return 4 * n * in * batch; }
bool skinny_back_grads(const GenericScheme&, int, int64_t, int64_t, int64_t) { return g_grads; }
hipError_t launch_skinny_back(const GenericScheme&, const ActLayers&, const void*, const BackGrads*, void*, void*,
                              int64_t, int64_t, int64_t, int64_t, const BiasSum&, hipStream_t) { return stub(); }
hipError_t launch_lists_act(ListsLayers, const void*, const Epilogue&, int64_t, hipStream_t) { return stub(); }
}  // namespace aqlm

namespace {

// A host array of exactly two pointers (one where a read past its end is planted).
void** two(void* a, void* b) {
#ifdef AQLM_PLANT_OVERREAD
    void** p = static_cast<void**>(malloc(sizeof(void*)));
    p[0] = a;
    (void)b;
#else
    void** p = static_cast<void**>(malloc(2 * sizeof(void*)));
    p[0] = a;
    p[1] = b;
#endif
    return p;
}

}  // namespace

int main() {
    char* buf = static_cast<char*>(aligned_alloc(256, 1 << 16));
    void *p = buf, *odd = buf + 8, *st = nullptr;
    const int64_t ws = INT64_MAX;
    void** a = two(p, p);
    void** half = two(p, nullptr);
    const int64_t ext[] = {INT64_MIN, -1, 0, 1, 8, 64, 72, 4096, 1 << 20, (1 << 20) + 8, 1 << 24, (1 << 24) + 1,
                           (int64_t)INT32_MAX - 256, INT32_MAX, (int64_t)1 << 32, INT64_MAX / 2, INT64_MAX};

    for (int v = 0; v < 4; ++v) {
        g_skinny = v & 1;
        g_grads = (v & 2) != 0;
        // launches: one straight from the codes (up to 16 tokens, or skinny), else decode (, pad) and product
        const int fwd = g_skinny ? 1 : 2, pad = g_skinny ? 0 : 1;
        CHECK(aqlm_linear_act(p, p, p, p, p, p, p, p, p, ws, 2, 2, 8, 8, 64, 256, 40, st), AQLM_OK, fwd);
        CHECK(aqlm_linear_act(p, p, p, p, p, p, p, p, p, ws, 2, 2, 8, 8, 64, 248, 40, st), AQLM_OK, fwd + pad);
        CHECK(aqlm_linear_act(p, p, p, p, nullptr, nullptr, nullptr, p, nullptr, 0, 0, 2, 8, 8, 64, 256, 16, st), AQLM_OK, 1);
        CHECK(aqlm_gated(a, a, a, p, a, a, p, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_OK, fwd);
        CHECK(aqlm_gated(a, a, a, p, half, half, p, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_OK, fwd);
        CHECK(aqlm_gated(a, a, a, p, nullptr, nullptr, p, nullptr, 0, 2, 1, 16, 8, 64, 256, 3, st), AQLM_OK, 1);
        CHECK(aqlm_gated(a, half, a, p, a, a, p, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_ERR_NULL, 0);
        // backward: gradients (, in the product), transposed weights, product
        const int back = g_skinny ? (g_grads ? 1 : 2) : 3;
        CHECK(aqlm_linear_act_backward(p, p, p, p, p, p, p, p, ws, 2, 2, 8, 8, 64, 256, 40, st), AQLM_OK, back);
        CHECK(aqlm_linear_act_backward(p, p, p, p, nullptr, p, nullptr, p, ws, 0, 2, 8, 8, 64, 256, 40, st), AQLM_OK,
              g_skinny ? back : 2);
        CHECK(aqlm_linear_act_backward(p, p, p, p, nullptr, p, p, p, ws, 0, 2, 8, 8, 72, 256, 40, st), AQLM_OK, back);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_OK, back);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, nullptr, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_OK, back);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, half, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_ERR_NULL, 0);
        CHECK(aqlm_gated_backward(a, a, a, p, half, p, a, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_ERR_NULL, 0);
        CHECK(aqlm_gated_backward(a, a, a, p, nullptr, p, a, p, ws, 2, 1, 16, 8, 64, 256, 40, st), AQLM_ERR_NULL, 0);
        // nothing to compute, or only zeros to write
        CHECK(aqlm_gated_backward(nullptr, a, a, p, a, p, a, p, ws, 2, 1, 16, 8, 64, 256, 0, st), AQLM_ERR_NULL, 0);
        CHECK(aqlm_gated_backward(a, a, a, nullptr, a, nullptr, a, nullptr, 0, 2, 1, 16, 8, 64, 256, 0, st), AQLM_OK, 2);
        CHECK(aqlm_linear_act_backward(p, p, p, p, p, p, p, nullptr, 0, 2, 2, 8, 8, 0, 256, 40, st), AQLM_OK, 1);
        // exactly the workspace of the query, one byte less, misaligned, absent
        int64_t n = 0;
        CHECK(aqlm_gated_backward_workspace_bytes(2, 8, 8, 1000, 1000, 100, &n), AQLM_OK, 0);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, p, n, 2, 2, 8, 8, 1000, 1000, 100, st), AQLM_OK, back);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, p, n - 1, 2, 2, 8, 8, 1000, 1000, 100, st), AQLM_ERR_SHAPE, 0);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, odd, n, 2, 2, 8, 8, 1000, 1000, 100, st), AQLM_ERR_ALIGN, 0);
        CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, nullptr, n, 2, 2, 8, 8, 1000, 1000, 100, st), AQLM_ERR_NULL, 0);
        CHECK(aqlm_linear_act_workspace_bytes(2, 8, 8, 64, 64, 64, nullptr), AQLM_ERR_NULL, 0);
        // every combination of extreme sizes is refused or served without overflow
        for (int64_t out : ext)
            for (int64_t in : ext)
                for (int64_t batch : ext) {
                    for (int M = 1; M <= 2; ++M) {
                        const int B = M == 1 ? 16 : 8;
                        const int r[] = {aqlm_linear_act_workspace_bytes(M, B, 8, out, in, batch, &n),
                                         aqlm_gated_workspace_bytes(M, B, 8, out, in, batch, &n),
                                         aqlm_linear_act_backward_workspace_bytes(M, B, 8, out, in, batch, &n),
                                         aqlm_gated_backward_workspace_bytes(M, B, 8, out, in, batch, &n)};
                        for (int q : r)
                            if (q != AQLM_OK && q != AQLM_ERR_SHAPE) ++g_failures;
                        const int s[] = {aqlm_linear_act(p, p, p, p, p, p, p, p, p, ws, 1, M, B, 8, out, in, batch, st),
                                         aqlm_gated(a, a, a, p, a, a, p, p, ws, 1, M, B, 8, out, in, batch, st),
                                         aqlm_linear_act_backward(p, p, p, p, p, p, p, p, ws, 1, M, B, 8, out, in, batch, st),
                                         aqlm_gated_backward(a, a, a, p, a, p, a, p, ws, 1, M, B, 8, out, in, batch, st)};
                        for (int i = 0; i < 4; ++i)
                            if ((s[i] == AQLM_OK) != (r[i] == AQLM_OK)) {
                                fprintf(stderr, "out %lld in %lld batch %lld: call %d gives %d, its workspace %d\n",
                                        (long long)out, (long long)in, (long long)batch, i, s[i], r[i]);
                                ++g_failures;
                            }
                    }
                }
    }
    int64_t* eb = static_cast<int64_t*>(malloc(2 * sizeof(int64_t)));
    eb[0] = eb[1] = 4096;
    CHECK(aqlm_gated_lists(a, a, eb, a, a, p, a, a, p, p, ws, 2, 1, 16, 8, 64, 256, 1, st), AQLM_OK, 1);
    CHECK(aqlm_gated_lists(a, a, eb, a, half, p, a, a, p, p, ws, 2, 1, 16, 8, 64, 256, 1, st), AQLM_ERR_NULL, 0);
    CHECK(aqlm_gated_lists(a, a, eb, a, a, p, nullptr, nullptr, p, nullptr, ws, 2, 1, 16, 8, 64, 256, 1, st), AQLM_ERR_NULL, 0);
    for (int64_t v : ext) {
        eb[1] = v;
        CHECK(aqlm_gated_lists(a, a, eb, a, a, p, half, half, p, p, ws, 2, 1, 16, 8, 64, 256, 1, st),
              v < 0 ? AQLM_ERR_SHAPE : AQLM_OK, v < 0 ? 0 : 1);
        CHECK(aqlm_linear_act_lists(p, p, 4096, p, p, p, p, p, p, p, p, v, 2, 1, 16, 8, 64, 256, 1, st),
              v >= 2048 ? AQLM_OK : AQLM_ERR_SHAPE, v >= 2048 ? 1 : 0);
    }
    // an error of a launch stops the call there
    g_skinny = g_grads = false;
    g_result = hipErrorInvalidValue;
    CHECK(aqlm_gated(a, a, a, p, a, a, p, p, ws, 2, 2, 8, 8, 64, 256, 40, st), AQLM_ERR_HIP, 1);
    CHECK(aqlm_gated_backward(a, a, a, p, a, p, a, p, ws, 2, 2, 8, 8, 64, 256, 40, st), AQLM_ERR_HIP, 1);
    g_result = hipSuccess;
    free(eb);
    free(half);
    free(a);
    free(buf);
    if (g_failures) return 1;
    printf("act validation ok\n");
    return 0;
}

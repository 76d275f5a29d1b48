// Host-side argument checks shared by the C ABI's sources (defined in aqlm_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace aqlm {

enum class Op { kGemv, kGemm, kDecode };

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 1 <= M <= 8, 1 <= B <= 16, g in {1, 2, 4, 8, 16, 32}
bool generic_scheme_ok(int M, int B, int g);

// Scheme, shape, pointers and alignment of one layer's call: AQLM_OK and the scheme
// id, or an error status; *empty: the call has nothing to compute.
int validate(Op op, const void* codes, const void* codebooks, const void* scales, const void* x, const void* y,
             int M, int B, int g, int64_t out, int64_t in, int64_t batch, int* scheme, bool* empty,
             uintptr_t codes_align = 16);
// The same for the slice-list layout (scheme and shape only).
int validate_lists(int M, int B, int g, int64_t out, int64_t in);

// The 2x8 GEMV kernel's scheme id for another 2-bit scheme with B = 8, or -1.
int gemv_b8_scheme(int M, int B, int g, int64_t in, int64_t batch);

// AQLM_OK, or AQLM_ERR_HIP with the error kept for aqlm_last_hip_error.
int finish(hipError_t e);

}  // namespace aqlm

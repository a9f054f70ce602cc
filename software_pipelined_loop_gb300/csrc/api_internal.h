// api_internal.h -- what the entry points of gemmpipe_api.cpp share with the
// other host translation units: device lookup, pointer checks, the stream
// workspace, tensor maps and launch accounting.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemmpipe.h"

namespace gp {

struct ApiDevice {
    int dev = 0;
    int sms = 0;
    int smem_optin = 0;
};

// The current device, or GEMMPIPE_ERR_UNSUPPORTED_DEVICE.
gemmpipe_status_t api_device(ApiDevice *out);

// A non-null device or managed pointer aligned to `align` bytes.
gemmpipe_status_t api_check_pointer(const void *p, int align);

// The operand workspace of (device, stream), at least `bytes` long.
gemmpipe_status_t api_workspace(int dev, cudaStream_t s, int64_t bytes, void **out);

// The workspace of (device, stream) for sums in parts: `counts` bytes that
// start as zeros and stay what the kernels make them, then `bytes` of parts.
gemmpipe_status_t api_parts_workspace(int dev, cudaStream_t s, int64_t counts, int64_t bytes, void **out);

// Runs fn(ctx), which launches `kernels` kernels on `s`, inside the timing
// region of the main (gemm) or auxiliary kernels, and counts the launches.
gemmpipe_status_t api_timed_launch(bool gemm, cudaStream_t s, int kernels, cudaError_t (*fn)(void *), void *ctx);

template <class F>
gemmpipe_status_t api_launch(bool gemm, cudaStream_t s, int kernels, F f)
{
    return api_timed_launch(
        gemm, s, kernels, [](void *c) { return (*static_cast<F *>(c))(); }, &f);
}

// The k-block of the armed test stall (-1: none), whose time limit replaces
// *timeout_ns; consumes the hook.
int64_t api_take_stall(uint64_t *timeout_ns);

// Tiled tensor map of 16-bit elements in the 128-byte swizzle: dims and box
// from the innermost, strides (bytes) of dims 1 .. rank - 1, zero fill
// outside.
bool api_encode_16bit(CUtensorMap *m, bool bf16, int rank, const void *base, const uint64_t *dims,
                      const uint64_t *strides, const uint32_t *box);

}  // namespace gp

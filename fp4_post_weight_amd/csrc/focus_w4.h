// focus_w4.h -- arguments and launchers of the linear layers with 4-bit
// weights and 8- or 16-bit activations, shared by focus_w4.hip and the C
// ABI.  Arguments reaching the launchers have been validated on the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace focus {

enum W4Kind {
    kW4Mx = 0,         // MXFP8 activations, MXFP4 weights
    kW4Bf16Nvfp4 = 1,  // BF16 activations, NVFP4 weights
    kW4Bf16Mxfp4 = 2,  // BF16 activations, MXFP4 weights
};

struct W4Args {
    const uint8_t* x;    // MXFP8 codes [M, K], or BF16 [M, K]
    const uint8_t* xs;   // MXFP8 scale bytes [M, K/32]
    int64_t M;
    const uint8_t* wc;   // weight codes [N, K/2]
    const uint8_t* ws;   // E8M0 [N, K/32] or E4M3 [N, K/16] scale bytes
    const float* ws2;    // NVFP4: one value
    int64_t N, K;
    void* y;             // [M, N] FP32 or BF16
};

// Largest K: a workgroup's rows (at most 256) are addressed by 32-bit offsets.
constexpr int64_t kMaxW4K = (int64_t)1 << 22;

hipError_t launch_w4_linear(const W4Args& a, W4Kind kind, bool bf16_out, hipStream_t stream);

}  // namespace focus

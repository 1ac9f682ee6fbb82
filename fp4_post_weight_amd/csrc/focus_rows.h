// focus_rows.h -- arguments and launchers of the row operators (root-mean-
// square norm with the residual's addition, gated activation, MXFP8
// quantizer), shared by focus_rows.hip and the C ABI.  Arguments reaching the
// launchers have been validated on the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace focus {

enum RowSource { kRowPlain = 0, kRowNorm = 1, kRowSilu = 2 };
enum RowOutput { kRowBf16 = 0, kRowNvfp4 = 1, kRowMxfp8 = 2 };

struct RowArgs {
    const uint16_t* x;   // input rows; the gate of the gated activation
    const uint16_t* r;   // norm: residual rows or NULL; gated activation: up
    const uint16_t* w;   // norm: weight [hidden]
    int64_t x_stride;    // elements from row to row of x (gated activation;
    int64_t r_stride;    // dense otherwise) and of r
    uint16_t* res_out;   // norm: BF16(x + r) or NULL
    float eps;           // norm
    int64_t tokens, hidden;
    uint8_t* codes;      // NVFP4 or MXFP8 codes
    uint8_t* scales;     // their block scale bytes
    float* s2;           // NVFP4: one per row
    uint16_t* y;         // BF16 result, or the dequantized values or NULL
};

// Rows whose result needs a whole-row reduction (the norm; NVFP4's token
// scale): one row per wavefront or workgroup.
hipError_t launch_rows(const RowArgs& a, RowSource src, RowOutput out, hipStream_t stream);

// No reduction (gated activation or plain input, BF16 or MXFP8 out).
hipError_t launch_flat(const RowArgs& a, RowSource src, RowOutput out, hipStream_t stream);

}  // namespace focus

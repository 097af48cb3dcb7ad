// Launch parameters of the norms around a block.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

struct NormVec {            // a [D] (or [group]) vector: weight or channel gate
    const void* p;
    int32_t bf16;
};

struct NormParams {
    int64_t T;
    int32_t D, group, w1_len;   // w1_len: D, or group when all groups share the weight
    int32_t act;                // 0 none, 1 sigmoid, 2 silu
    int32_t gate_mode;          // 0 none, 1 per token [T, D], 2 per channel [D]
    float c, eps;
    const void* y; int64_t y_row;
    const void* x; int64_t x_row;       // residual or nullptr
    const void* gate; int64_t gate_row;
    NormVec gate_c, w1, w2;
    void* h; int64_t h_row;
    void* n; int64_t n_row;             // nullptr unless w2
    // backward
    const void* dh; int64_t dh_row;
    const void* dn; int64_t dn_row;
    void* dx; int64_t dx_row;
    void* dy; int64_t dy_row;
    void* dgate; int64_t dgate_row;     // per token
    int32_t parts;                      // workgroups of the backward
    float *pw1, *pw2, *pgate;           // [parts, w1_len], [parts, D], [parts, D] or nullptr
};

struct NormReduce {
    const float* part;
    int32_t parts, n, out_bf16;
    void* out;
};

constexpr int kNormMaxDim = 16384;

// Workgroups that share the backward's rows.
int norm_parts(int64_t T, int D);

// Threads of a forward's workgroup; one workgroup a row.
int norm_threads(const NormParams& p);

hipError_t launch_norm(const NormParams& p, bool work_bf16, hipStream_t s);
hipError_t launch_norm_bwd(const NormParams& p, bool work_bf16, hipStream_t s);
hipError_t launch_norm_reduce(const NormReduce* r, int count, hipStream_t s);

}  // namespace gdr

// Launch parameters of the selective state space scan, the convolution's
// gradient and history fold, and the verification of drafted tokens.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// States [slots or rows, D, N] with a dense D x N block each.
struct ScanState {
    const void* p;          // nullptr: zeros (read), nothing (written)
    int64_t outer;          // elements from one slot (or row) to the next
    int32_t bf16;
};

struct ScanRows {           // a [T, D] operand
    const void* p;
    int64_t tok;
};

struct ScanHeads {          // B or C: [T, G, N]
    const void* p;
    int64_t tok, grp;
};

struct ScanParams {
    int32_t B, T, D, N, G, gd;      // gd: channels a group
    int32_t softplus, keep;         // keep: states are read and not written
    const uint32_t* offsets;        // [B+1], or nullptr: token t is row t
    const uint32_t* slot_idx;       // [B] or nullptr (slot = row)
    const uint32_t* accepted;       // [B] or nullptr (the whole row)
    ScanRows x, dt, z;
    void* out; int64_t o_tok;       // nullptr: states only
    const float *A, *skip, *bias;   // [D, N]; [D] or nullptr
    ScanHeads b, c;
    ScanState in;
    void* last; int64_t last_outer; // written states (in's type), or nullptr
    int32_t narrow_most;            // rows up to this many tokens are taken by the narrow walk
    int32_t hand_on;                // the narrow walk writes the states of empty rows too
    int32_t lane_most;              // longer rows up to this many are taken by the lane walk
    // long rows, cut into segments of seg_len tokens (0: none is cut)
    int32_t seg_skip;               // rows up to this many tokens have no segment
    int32_t seg_len, segs, tiles;   // tiles: waves over one group's channels
    float* seg_state;               // [segs, D, N]
    float* seg_delta;               // [segs, D]
};

// The gradient's operands beside the forward's.
struct ScanGrad {
    ScanRows d_o, dx, ddt, dz;
    ScanHeads db, dc;               // outputs
    float *dA, *dskip, *dbias;      // [D, N], [D], [D]; dskip and dbias may be nullptr
    ScanState dfinal;               // nullptr: zeros
    void* dinit; int64_t dinit_outer; int32_t dinit_bf16;
    int32_t tiles;                  // workgroups over one group's channels
    float* check;                   // [parts, N + 1, D] local states before each part, and the
                                    // step sizes from the segment's start (parts: T/kScanPart + B)
    float* seg_rev;                 // [segs, N, D] what a segment hands to its past; the
                                    // gradient keeps seg_state in that order too
    float* turned;                  // [parts, G, 2, N, kScanPart] B and C
    float* part_bc;                 // [tiles of a group, T, G, 2, N]
    float* part_a;                  // [segs, N, D]
    float* part_d;                  // [segs, 2, D]
};

struct ConvFold {
    int32_t B, C, H;                // H: entries of history
    const uint32_t *offsets, *slot_idx, *accepted;
    ScanRows x;
    void* state; int64_t st_slot, st_tok;
};

struct ConvGrad {
    int32_t B, T, C, W, silu;
    const uint32_t* offsets;
    ScanRows d_o, x, dx;
    const float* weight; int64_t w_chan;
    const float* bias;
    float* dweight; int64_t dw_chan;
    float* dbias;
    int32_t run, runs;              // tokens a thread walks, and how many such runs
    float* part;                    // [runs, W + 1, C]
};

struct DraftParams {
    int32_t B, T, V, splits, span;  // span: values a split covers
    const uint32_t* offsets;
    const int32_t* tokens; int64_t tok_stride;
    const void *p, *q; int64_t p_tok, q_tok; int32_t bf16;
    const float* u; int64_t u_stride;
    int32_t *accepted, *next;
    double* part;                   // sampled: [B, 2, splits]; greedy: [T, splits] pairs
};

// Workgroups of four waves that need nothing of one another: one for each SIMD.
constexpr int kScanThreads = 256;
inline unsigned scan_blocks(int64_t waves) { return static_cast<unsigned>((waves + 3) / 4); }
constexpr int kScanNarrowThreads = 256;
constexpr int kScanLaneChannels = 16;  // channels of a lane walk's workgroup
constexpr int kScanPart = 16;       // tokens that a gradient holds in registers
int scan_grad_channels(int N);      // channels of a gradient's workgroup

hipError_t launch_scan_narrow(const ScanParams& p, bool work_bf16, hipStream_t s);
hipError_t launch_scan_wide(const ScanParams& p, bool work_bf16, bool sums, hipStream_t s);
hipError_t launch_scan_lanes(const ScanParams& p, bool work_bf16, hipStream_t s);
hipError_t launch_scan_chain(const ScanParams& p, hipStream_t s);

hipError_t launch_scan_bwd(const ScanParams& p, const ScanGrad& g, bool work_bf16, hipStream_t s);

hipError_t launch_conv_fold(const ConvFold& p, bool work_bf16, hipStream_t s);
hipError_t launch_conv_bwd(const ConvGrad& p, bool work_bf16, hipStream_t s);

hipError_t launch_drafts(const DraftParams& p, hipStream_t s);

}  // namespace gdr

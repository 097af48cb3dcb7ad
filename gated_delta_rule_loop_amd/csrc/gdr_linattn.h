// Launch parameters shared by the host entry points and the gfx950 kernels of
// linear attention with a decay for each head.  Not part of the public ABI.
//
// Per (row, value head) a K x V state S is carried token by token,
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,     o_t = scale S_t^T q_t.
// Everything the library computes for more than a few tokens - the forward
// and the gradients of q, k and v - is one kind of walk over a row:
//     out_i = scale (sum_{j <= i} exp(G_i - G_j) (x_i . y_j) z_j + exp(G_i) S^T x_i)
// in walk order, with G the running sum of g and S the state [Kd, Vd] that the
// walk starts from:
//     forward  x, y, z = q, k, v    (from the first token; the state is S)
//     dq       x, y, z = do, v, k   (from the first token; S transposed)
//     dv       x, y, z = k, q, do   (from the last token; dL/dS over scale)
//     dk       x, y, z = v, do, q   (from the last token; that transposed)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// A per-token operand; value head hv reads head hv / div.  Strides in elements.
struct LaTensor {
    const void* p;
    int64_t tok, head;
    int32_t div;
};

// Where a walk's state comes from or goes to; element (kd, z) of a head lies
// at kd * sk + z * sz.
struct LaState {
    void* p;                // nullptr: zeros (source), no store (destination)
    int64_t outer, head;    // per slot, row or segment; per value head
    int32_t sk, sz;
    int32_t bf16;
    int32_t by_segment;     // indexed by segment instead of by slot or row
    float mult;             // value = mult * stored (source), stored = mult * value
};

struct LaWalk {
    LaTensor x, y, z;
    int32_t Kd, Vd, tiles;  // tiles: workgroups over Vd
    int32_t reverse;        // walk from the row's last token
    void* out;
    int64_t out_tok, out_head;
    int32_t out_f32;        // float32 output whatever the work type
    int32_t third;          // a third bf16 term in the state's sums (float32 states)
    LaState in, last;
    // by_cut: a row of one segment starts from in_row; `in` holds states by the
    // number of a segment among those of rows that have several.
    LaState in_row;
    int32_t by_cut;
    // Sums for the decays' gradient (row_sum != nullptr): row_sum[part, head,
    // token] += partner . out without the token's own pair, and phi[segment,
    // head, part] = scale <state at the walk's end, phi_in>.
    LaTensor partner;
    float* row_sum;
    float* phi;
    LaState phi_in;
    int32_t phi_rows;       // phi only where the walk leaves its row
};

constexpr int kLaMaxWalks = 3;
// Where a call has many rows, those of a few tokens go token by token and only the
// others are walked, each row by its own length (a batch of single tokens and a
// prompt is common).  A short row is mostly its state, which the token-by-token
// form streams in whole lines; the walk's layout reads it in pieces.  Measured at
// 32 value heads, K = V = 128, us token by token and walked: 64 rows of 1, 8 and 16
// tokens bf16 29 and 57, 57 and 60, 89 and 55, float32 54 and 89, 91 and 91, 117 and
// 95; 256 rows of 8 bf16 196 and 268; 4 rows of 1 token 14.4 and 15.7.  A prompt of
// 190 tokens beside 63 single ones: 57 us, 332 where the call went token by token,
// 59 where it was walked; one of 512 beside 255: 158, 968 and 272.
constexpr int kLaStepTokens = 8, kLaStepRows = 16;

struct LaParams {
    int32_t B, nv, T;
    int32_t seg_len;        // tokens per segment; 0: one segment per row
    int32_t walk_from;      // rows of fewer tokens are not walked (then seg_len > 0)
    int32_t segs;           // segments launched (rows, or their upper bound)
    int32_t nwalks, max_tiles;
    const uint32_t* offsets;
    const uint32_t* slot_idx;  // states by slot; nullptr: by row
    const void* g;          // log decays [T, nv]; nullptr: none (a = 1)
    int64_t g_tok, g_head;
    int32_t g_bf16;
    float scale;
    LaWalk w[kLaMaxWalks];
};

// Segment sums -> the state that each segment's walk starts from, in place.
struct LaScan {
    int32_t B, nv, T, seg_len, walk_from, segs;
    int32_t rows;           // rows of walk_from tokens and more, or their upper bound
    const uint32_t* offsets;
    const uint32_t* slot_idx;
    int32_t n;              // elements per state
    int32_t V;              // columns of a state row (for dense sources)
    int32_t reverse;
    float* state;           // [segs, nv, n]
    const float* tot;       // [segs, nv] log2 decay of a segment
    LaState in;             // the row's first state ([K, V] dense) or absent
};

struct LaDecayGrad {
    int32_t B, nv, T, seg_len, segs;
    const uint32_t* offsets;
    const float *rq, *rk;   // [parts, nv, T]
    const float* phi;       // [segs, nv, parts] at the segments' ends, or nullptr (zeros)
    const float* phi0;      // [segs, nv, parts0] where rows start, or nullptr (zeros)
    int32_t parts, parts0;  // multiples of 4
    void* dg; int64_t dg_tok, dg_head; int32_t dg_bf16;
};

struct LaHeadSum {          // out[t, hk, :] = sum over the group of part[t, hv, :]
    int32_t T, nk, G, K, B;
    const uint32_t* offsets;   // tokens outside [offsets[0], offsets[B]) have no parts
    const float* part;      // [T, nk * G, K]
    void* out; int64_t out_tok, out_head;
};

// Token-by-token form for rows of one or a few tokens.
struct LaStep {
    int32_t B, nv, G, K, V;
    const uint32_t* offsets;   // nullptr: row b is token b
    const uint32_t* slot_idx;
    const void* q; int64_t q_tok, q_head;
    const void* k; int64_t k_tok, k_head;
    const void* v; int64_t v_tok, v_head;
    const void* g; int64_t g_tok, g_head; int32_t g_bf16;
    void* out; int64_t o_tok, o_head;
    LaState in, last;
    float scale;
    int32_t most;              // with offsets: rows of more tokens are left out
};

// Waves of a walk's workgroup, of 16 columns of the state each.
inline int la_waves(int Vd) { return Vd <= 64 ? 4 : 8; }

// Threads of a step's workgroup: 8 x 8 elements of the state each.
inline int64_t la_step_threads(int64_t K, int64_t V) { return ((K / 8) * (V / 8) + 63) / 64 * 64; }

// Workgroups of a scan over one state of n elements, 4 a thread.
constexpr int kLaScanThreads = 256;
__host__ __device__ inline int la_scan_blocks(int n) {
    return (n / 4 + kLaScanThreads - 1) / kLaScanThreads;
}

hipError_t launch_la_walks(const LaParams& p, bool work_bf16, hipStream_t s);
hipError_t launch_la_segments(const LaParams& p, bool work_bf16, float* tot, hipStream_t s);
hipError_t launch_la_scans(const LaScan* c, int count, hipStream_t s);
hipError_t launch_la_decay_grad(const LaDecayGrad& p, hipStream_t s);
hipError_t launch_la_head_sum(const LaHeadSum& p, bool work_bf16, hipStream_t s);
hipError_t launch_la_step(const LaStep& p, bool work_bf16, hipStream_t s);

}  // namespace gdr

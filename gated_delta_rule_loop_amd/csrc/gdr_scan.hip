// gfx950 kernels of the selective state space scan:
//     delta = softplus(dt + dt_bias)     a = exp(delta A[d, n])
//     h_t = a h_{t-1} + delta x B_t[n]   out = (sum_n C_t[n] h_t + skip x) silu(z)
// for every channel d and its N states n, in float32.  The decay is a number of
// its own for every token, channel and state, so there is no form as matrix
// products: the work is 6 vector-unit slots a token, channel and state (product,
// exponential, which takes two, product, two multiply-adds).
//
// Wide walk (prompts): a lane owns a channel and all its states, in registers;
// B and C of a token are the same for the whole wave and come through scalar
// loads.  Long rows are cut into segments so that few channels still fill the
// chip: one launch takes each segment's own end state from zero and the sum of
// its step sizes (a segment's decay is exp(A sum delta)), one chains them to the
// states the segments start from, and the walk follows.
//
// Narrow walk (single tokens, drafted windows, folds): a lane owns 16 bytes of a
// channel's state, so that states are read and written in whole lines; the
// output is summed over a channel's 1 to 16 lanes by lane permutations.
#include "gdr_scan_dev.h"

namespace gdr {
namespace {

// ------------------------------------------------------------- narrow walk ---

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)),
                                                       CTRL, 0xf, 0xf, false));
}
// Sum over n neighbouring lanes (a power of two up to 16, aligned), in each.
template <int n> __device__ __forceinline__ float lane_sum(float v) {
    if constexpr (n >= 2) v += dpp<0xB1>(v);   // quad lanes 1 0 3 2
    if constexpr (n >= 4) v += dpp<0x4E>(v);   // quad lanes 2 3 0 1
    if constexpr (n >= 8) v += dpp<0x141>(v);  // mirrored within 8
    if constexpr (n >= 16) v += dpp<0x140>(v); // mirrored within 16
    return v;
}

template <typename WT, int S> struct Token {  // one token's operands of a lane
    float x, dt, z, b[S], c[S];
};

template <typename WT, typename ST, int N, bool OUT>
__global__ void __launch_bounds__(kScanNarrowThreads) scan_narrow(const ScanParams p) {
    constexpr int S = N < static_cast<int>(16 / sizeof(ST)) ? N : 16 / sizeof(ST);
    constexpr int L = N / S;                       // lanes a channel
    const int per = kScanNarrowThreads / L;        // channels a workgroup
    const int tiles = (p.D + per - 1) / per;
    const int row = blockIdx.x / tiles, tile = blockIdx.x - row * tiles;
    int t0 = row, n = 1;
    if (p.offsets) {
        t0 = static_cast<int>(p.offsets[row]);
        n = static_cast<int>(p.offsets[row + 1]) - t0;
        if (n > p.narrow_most || (n <= 0 && !p.hand_on)) return;
    }
    const uint32_t slot = p.slot_idx ? p.slot_idx[row] : static_cast<uint32_t>(row);
    const bool pad = p.slot_idx != nullptr && slot == kPadSlot;
    if (p.accepted) {  // a fold takes the row's accepted prefix, and none beyond the row
        const uint32_t a = p.accepted[row];
        if (a == 0 || a > static_cast<uint32_t>(n) || pad) return;
        n = static_cast<int>(a);
    }
    const int d = tile * per + threadIdx.x / L, sub = threadIdx.x % L;
    if (d >= p.D) return;  // whole groups of L lanes
    if (pad) {
        if (OUT && sub == 0)
            for (int t = 0; t < n; ++t)
                scan_put(static_cast<WT*>(p.out) + static_cast<int64_t>(t0 + t) * p.o_tok + d, 0.0f);
        return;
    }
    const int n0 = sub * S;
    const int64_t at = static_cast<int64_t>(d) * N + n0;
    float h[S], a2[S];
#pragma unroll
    for (int i = 0; i < S; ++i) h[i] = 0.0f;
    if (p.in.p)
        scan_load<S>(static_cast<const ST*>(p.in.p) + static_cast<int64_t>(slot) * p.in.outer + at, h);
    scan_load<S>(p.A + at, a2);
    const float bias = p.bias ? p.bias[d] : 0.0f;
    const float skip = OUT && p.skip ? p.skip[d] : 0.0f;
    const int g = d / p.gd;
    const WT* x = static_cast<const WT*>(p.x.p) + d;
    const WT* dt = static_cast<const WT*>(p.dt.p) + d;
    const WT* z = OUT && p.z.p ? static_cast<const WT*>(p.z.p) + d : nullptr;
    const WT* b = static_cast<const WT*>(p.b.p) + static_cast<int64_t>(g) * p.b.grp + n0;
    const WT* c = OUT ? static_cast<const WT*>(p.c.p) + static_cast<int64_t>(g) * p.c.grp + n0
                      : nullptr;
    auto fetch = [&](int t, Token<WT, S>& k) {
        const int64_t i = t0 + t;
        k.x = scan_value(x[i * p.x.tok]);
        k.dt = scan_value(dt[i * p.dt.tok]);
        if (OUT && z) k.z = scan_value(z[i * p.z.tok]);
        scan_load<S>(b + i * p.b.tok, k.b);
        if constexpr (OUT) scan_load<S>(c + i * p.c.tok, k.c);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) a2[i] *= kScanLog2e;
    Token<WT, S> next;
    if (n > 0) fetch(0, next);
    for (int t = 0; t < n; ++t) {
        const Token<WT, S> k = next;
        if (t + 1 < n) fetch(t + 1, next);
        float delta = k.dt + bias;
        if (p.softplus) delta = scan_softplus(delta);
        const float u = delta * k.x;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[i]), h[i], u * k.b[i]);
            if constexpr (OUT) y = __builtin_fmaf(h[i], k.c[i], y);
        }
        if constexpr (OUT) {
            y = __builtin_fmaf(skip, k.x, lane_sum<L>(y));
            if (z) y *= k.z * scan_sigmoid(k.z);
            if (sub == 0)
                scan_put(static_cast<WT*>(p.out) + static_cast<int64_t>(t0 + t) * p.o_tok + d, y);
        }
    }
    if (p.last && !p.keep)
        scan_store<S>(static_cast<ST*>(p.last) + static_cast<int64_t>(slot) * p.last_outer + at, h);
}

template <typename WT, typename ST, int N>
hipError_t narrow_out(const ScanParams& p, hipStream_t s) {
    constexpr int S = N < static_cast<int>(16 / sizeof(ST)) ? N : 16 / sizeof(ST);
    const int per = kScanNarrowThreads / (N / S);
    const dim3 grid(static_cast<unsigned>(p.B) * ((p.D + per - 1) / per));
    if (p.out)
        hipLaunchKernelGGL((scan_narrow<WT, ST, N, true>), grid, dim3(kScanNarrowThreads), 0, s, p);
    else
        hipLaunchKernelGGL((scan_narrow<WT, ST, N, false>), grid, dim3(kScanNarrowThreads), 0, s, p);
    return hipGetLastError();
}

template <typename WT, typename ST> hipError_t narrow_n(const ScanParams& p, hipStream_t s) {
    switch (p.N) {
        case 8: return narrow_out<WT, ST, 8>(p, s);
        case 16: return narrow_out<WT, ST, 16>(p, s);
        case 32: return narrow_out<WT, ST, 32>(p, s);
        case 64: return narrow_out<WT, ST, 64>(p, s);
        default: return hipErrorInvalidValue;
    }
}

// --------------------------------------------------------------- wide walk ---

constexpr int kAhead = 4;  // tokens whose x, dt and z are loaded before those in work

template <typename WT, int N, bool SUMS>
__global__ void __launch_bounds__(kScanThreads) scan_wide(const ScanParams p) {
    const int ctiles = p.G * p.tiles;
    const int seg = blockIdx.x / ctiles, tile = blockIdx.x - seg * ctiles;
    ScanSpan o;
    if (!scan_locate(p, seg, o)) return;
    if (o.n <= 0 || (o.count == 1 && o.n <= p.narrow_most)) return;
    if (SUMS && o.s == o.count - 1) return;
    const int g = tile / p.tiles;
    const int cg = (tile - g * p.tiles) * kScanThreads + static_cast<int>(threadIdx.x);
    const bool live = cg < p.gd;
    const int d = g * p.gd + min(cg, p.gd - 1);
    const uint32_t slot = p.slot_idx ? scan_index(p.slot_idx, o.row) : static_cast<uint32_t>(o.row);
    const bool pad = p.slot_idx != nullptr && slot == kPadSlot;
    if (pad) {
        if (!SUMS && live && p.out)
            for (int t = 0; t < o.n; ++t)
                scan_put(static_cast<WT*>(p.out) + static_cast<int64_t>(o.t0 + t) * p.o_tok + d, 0.0f);
        return;
    }
    const int64_t at = static_cast<int64_t>(d) * N;
    float h[N], a2[N];
    scan_load<N>(p.A + at, a2);
#pragma unroll
    for (int i = 0; i < N; ++i) a2[i] *= kScanLog2e;
    const int64_t mine = static_cast<int64_t>(seg) * p.D * N + at;
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = 0.0f;
    if constexpr (!SUMS) {
        if (o.count > 1) {
            scan_load<N>(p.seg_state + mine, h);
        } else if (p.in.p) {
            const int64_t i = static_cast<int64_t>(slot) * p.in.outer + at;
            if (p.in.bf16) scan_load<N>(static_cast<const uint16_t*>(p.in.p) + i, h);
            else scan_load<N>(static_cast<const float*>(p.in.p) + i, h);
        }
    }
    const float bias = p.bias ? p.bias[d] : 0.0f;
    const float skip = !SUMS && p.skip ? p.skip[d] : 0.0f;
    const WT* x = static_cast<const WT*>(p.x.p) + static_cast<int64_t>(o.t0) * p.x.tok;
    const WT* dt = static_cast<const WT*>(p.dt.p) + static_cast<int64_t>(o.t0) * p.dt.tok;
    const bool gated = !SUMS && p.z.p != nullptr;
    const WT* z = gated ? static_cast<const WT*>(p.z.p) + static_cast<int64_t>(o.t0) * p.z.tok : x;
    const int64_t z_tok = gated ? p.z.tok : p.x.tok;
    WT* out = static_cast<WT*>(p.out) + (SUMS ? 0 : static_cast<int64_t>(o.t0) * p.o_tok);
    const int64_t b0 = static_cast<int64_t>(o.t0) * p.b.tok + static_cast<int64_t>(g) * p.b.grp;
    const int64_t c0 = SUMS ? 0 : static_cast<int64_t>(o.t0) * p.c.tok + static_cast<int64_t>(g) * p.c.grp;
    WT xs[kAhead], ds[kAhead], zs[kAhead];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t u = min(t + i, o.n - 1);
            xs[i] = (x + u * p.x.tok)[d];
            ds[i] = (dt + u * p.dt.tok)[d];
            if constexpr (!SUMS) zs[i] = (z + u * z_tok)[d];
        }
    };
    float total = 0.0f;
    auto token = [&](int t, WT xr, WT dr, WT zr) {
        const float xv = scan_value(xr);
        float delta = scan_value(dr) + bias;
        if (p.softplus) delta = scan_softplus(delta);
        const float u = delta * xv;
        float b[N];
        uniform_row<WT, N>(p.b.p, b0 + t * p.b.tok, b);
        if constexpr (SUMS) {
            total += delta;
#pragma unroll
            for (int i = 0; i < N; ++i)
                h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[i]), h[i], u * b[i]);
        } else {
            float c[N], y0 = 0.0f, y1 = 0.0f;
            uniform_row<WT, N>(p.c.p, c0 + t * p.c.tok, c);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[i]), h[i], u * b[i]);
                if (i & 1) y1 = __builtin_fmaf(h[i], c[i], y1);
                else y0 = __builtin_fmaf(h[i], c[i], y0);
            }
            float y = __builtin_fmaf(skip, xv, y0 + y1);
            if (gated) {
                const float zv = scan_value(zr);
                y *= zv * scan_sigmoid(zv);
            }
            if (live) scan_put(out + t * p.o_tok + d, y);
        }
    };
    fetch(0);
    for (int t = 0; t < o.n; t += kAhead) {
        WT xc[kAhead], dc[kAhead], zc[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            xc[i] = xs[i];
            dc[i] = ds[i];
            if constexpr (!SUMS) zc[i] = zs[i];
        }
        if (t + kAhead < o.n) fetch(t + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t + i < o.n) token(t + i, xc[i], dc[i], SUMS ? xc[i] : zc[i]);
    }
    if (!live) return;
    if constexpr (SUMS) {
        scan_store<N>(p.seg_state + mine, h);
        p.seg_delta[static_cast<int64_t>(seg) * p.D + d] = total;
    } else if (o.s == o.count - 1 && p.last && !p.keep) {
        const int64_t i = static_cast<int64_t>(slot) * p.last_outer + at;
        if (p.in.bf16) scan_store<N>(static_cast<uint16_t*>(p.last) + i, h);
        else scan_store<N>(static_cast<float*>(p.last) + i, h);
    }
}

// seg_state of a cut row: from the segments' own end states to the states that
// they start from.
__global__ void __launch_bounds__(256) scan_chain(const ScanParams p) {
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const int blocks = static_cast<int>((DN + 255) / 256);
    const int row = blockIdx.x / blocks;
    const int64_t i = static_cast<int64_t>(blockIdx.x - row * blocks) * 256 + threadIdx.x;
    const uint32_t a = p.offsets[row];
    const int n = static_cast<int>(p.offsets[row + 1] - a);
    if (i >= DN || n <= p.seg_len) return;
    const uint32_t slot = p.slot_idx ? p.slot_idx[row] : static_cast<uint32_t>(row);
    if (p.slot_idx != nullptr && slot == kPadSlot) return;
    const int count = (n + p.seg_len - 1) / p.seg_len;
    const int64_t first = scan_first_seg(a, row, p.seg_len);
    const float a2 = p.A[i] * kScanLog2e;
    float h = 0.0f;
    if (p.in.p) {
        const int64_t j = static_cast<int64_t>(slot) * p.in.outer + i;
        h = p.in.bf16 ? scan_widen(static_cast<const uint16_t*>(p.in.p)[j])
                      : static_cast<const float*>(p.in.p)[j];
    }
    float* st = p.seg_state + first * DN + i;
    const float* dl = p.seg_delta + first * p.D + i / p.N;
    constexpr int U = 8;  // segments whose sums are in flight together
    for (int s = 0; s < count; s += U) {
        float e[U], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (s + j < count - 1) {
                e[j] = st[(s + j) * DN];
                d[j] = dl[static_cast<int64_t>(s + j) * p.D];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (s + j < count) {
                st[(s + j) * DN] = h;
                if (s + j < count - 1)
                    h = __builtin_fmaf(__builtin_amdgcn_exp2f(a2 * d[j]), h, e[j]);
            }
    }
}

template <typename WT, int N> hipError_t wide_sums(const ScanParams& p, bool sums, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.segs) * p.G * p.tiles);
    if (sums)
        hipLaunchKernelGGL((scan_wide<WT, N, true>), grid, dim3(kScanThreads), 0, s, p);
    else
        hipLaunchKernelGGL((scan_wide<WT, N, false>), grid, dim3(kScanThreads), 0, s, p);
    return hipGetLastError();
}

template <typename WT> hipError_t wide_n(const ScanParams& p, bool sums, hipStream_t s) {
    switch (p.N) {
        case 8: return wide_sums<WT, 8>(p, sums, s);
        case 16: return wide_sums<WT, 16>(p, sums, s);
        case 32: return wide_sums<WT, 32>(p, sums, s);
        case 64: return wide_sums<WT, 64>(p, sums, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_scan_narrow(const ScanParams& p, bool work_bf16, hipStream_t s) {
    if (work_bf16)
        return p.in.bf16 ? narrow_n<uint16_t, uint16_t>(p, s) : narrow_n<uint16_t, float>(p, s);
    return p.in.bf16 ? narrow_n<float, uint16_t>(p, s) : narrow_n<float, float>(p, s);
}

hipError_t launch_scan_wide(const ScanParams& p, bool work_bf16, bool sums, hipStream_t s) {
    return work_bf16 ? wide_n<uint16_t>(p, sums, s) : wide_n<float>(p, sums, s);
}

hipError_t launch_scan_chain(const ScanParams& p, hipStream_t s) {
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const dim3 grid(static_cast<unsigned>(p.B) * static_cast<unsigned>((DN + 255) / 256));
    hipLaunchKernelGGL(scan_chain, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gdr

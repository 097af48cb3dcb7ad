// gfx950 kernels around the causal Conv1d: its gradient, and the fold of its
// history over an accepted prefix.
//
// Gradient of out_t = act(pre_t), pre_t = bias + sum_j w[j] x[t - (W-1-j)] within
// a row (inputs before the row are zeros):
//     g_t = dout_t act'(pre_t)              dx_s = sum_k w[W-1-k] g[s+k]  (s + k in the row)
//     dw[j] = sum_t g_t x[t - (W-1-j)]      dbias = sum_t g_t
// A thread owns 4 neighbouring channels and walks a run of tokens, and W - 1 tokens
// past it for the inputs' gradients: it recomputes pre from a window of inputs,
// so that x and dout are read once and nothing else is, and keeps the run's part
// of the weights' gradient in registers.  A second launch adds the runs' parts
// in float64 in a fixed order.  A stream over x, dout and dx: bound by HBM.  4096 bf16
// tokens of 8192 channels 52 us (201 MB, 3.9 TB/s; a copy 5.1) and 5 for the runs' parts.
#include <type_traits>

#include "gdr_scan_dev.h"

namespace gdr {
namespace {

constexpr int kConvBwdAhead = 4;

__device__ __forceinline__ void put4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put4(uint16_t* p, const float (&v)[4]) {
    const uint32_t a = scan_round(v[0]) | (static_cast<uint32_t>(scan_round(v[1])) << 16);
    const uint32_t b = scan_round(v[2]) | (static_cast<uint32_t>(scan_round(v[3])) << 16);
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
}

// 4 values as they stand in memory.
__device__ __forceinline__ float4 raw4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint2 raw4(const uint16_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void wide4(const float4& w, float (&v)[4]) {
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}
__device__ __forceinline__ void wide4(const uint2& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

template <int W, typename WT, bool SILU>
__global__ void __launch_bounds__(kScanThreads) conv_bwd_kernel(const ConvGrad p) {
    constexpr int H = W - 1;
    const int ctiles = (p.C / 4 + 63) / 64, wave = scan_wave();
    const int run = wave / ctiles;
    const int c0 = ((wave - run * ctiles) * 64 + static_cast<int>(threadIdx.x & 63)) * 4;
    if (run >= p.runs || c0 >= p.C) return;
    const int first = static_cast<int>(scan_index(p.offsets, 0));
    const int end = static_cast<int>(scan_index(p.offsets, p.B));  // rows hold tokens [first, end)
    const int a = run * p.run, b = a + min(p.run, p.T - a);  // this run's tokens
    const WT* x = static_cast<const WT*>(p.x.p) + c0;
    const WT* d_o = static_cast<const WT*>(p.d_o.p) + c0;
    WT* dx = static_cast<WT*>(const_cast<void*>(p.dx.p)) + c0;
    float w[W][4], bias[4], dw[W][4], db[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j][v] = p.weight[static_cast<int64_t>(c0 + v) * p.w_chan + j];
            dw[j][v] = 0.0f;
        }
        bias[v] = p.bias ? p.bias[c0 + v] : 0.0f;
        db[v] = 0.0f;
    }
    const int from = max(a, first), upto = min(b, end);
    if (from < upto) {
        int row = 0, hi = p.B - 1;
        while (row < hi) {
            const int mid = (row + hi + 1) >> 1;
            if (static_cast<int>(scan_index(p.offsets, mid)) <= from) row = mid; else hi = mid - 1;
        }
        int t0 = static_cast<int>(scan_index(p.offsets, row)), t1 = static_cast<int>(scan_index(p.offsets, row + 1));
        float xw[H][4], acc[W][4];  // acc[k]: gradient of the input of token t - k so far
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const int s = from - H + k;
#pragma unroll
            for (int v = 0; v < 4; ++v) xw[k][v] = 0.0f;
            if (s >= t0) scan_load<4>(x + static_cast<int64_t>(s) * p.x.tok, xw[k]);
        }
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[k][v] = 0.0f;
        const int last = min(upto + H, end);   // tokens read
        typedef decltype(raw4(x)) Raw;
        Raw xn[kConvBwdAhead], gn[kConvBwdAhead];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < kConvBwdAhead; ++i) {
                const int64_t u = min(t + i, last - 1);
                xn[i] = raw4(x + u * p.x.tok);
                gn[i] = raw4(d_o + u * p.d_o.tok);
            }
        };
        fetch(from);
        // FULL: every token and those that it is summed into are in one row and in the run.
        auto block = [&](int tb, auto full) __attribute__((always_inline)) {
            constexpr bool FULL = decltype(full)::value;
            Raw xr[kConvBwdAhead], gr[kConvBwdAhead];
#pragma unroll
            for (int i = 0; i < kConvBwdAhead; ++i) {
                xr[i] = xn[i];
                gr[i] = gn[i];
            }
            if (tb + kConvBwdAhead < last) fetch(tb + kConvBwdAhead);
#pragma unroll
            for (int i = 0; i < kConvBwdAhead; ++i) {
                const int t = tb + i;
                float xc[4], gc[4];
                wide4(xr[i], xc);
                wide4(gr[i], gc);
                if (FULL || t < last) {
                    if (!FULL && t >= t1) {  // the next row that has tokens; nothing passes between rows
                        do {
                            ++row;
                            t0 = t1;
                            t1 = static_cast<int>(scan_index(p.offsets, row + 1));
                        } while (t >= t1);
#pragma unroll
                        for (int k = 0; k < H; ++k)
#pragma unroll
                            for (int v = 0; v < 4; ++v) xw[k][v] = 0.0f;
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float g = gc[v];
                        if constexpr (SILU) {
                            float pre = bias[v];
#pragma unroll
                            for (int j = 0; j < H; ++j) pre = __builtin_fmaf(w[j][v], xw[j][v], pre);
                            pre = __builtin_fmaf(w[H][v], xc[v], pre);
                            const float sig = scan_sigmoid(pre);
                            g *= sig * __builtin_fmaf(pre, 1.0f - sig, 1.0f);
                        }
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            if (FULL || t - k >= t0) acc[k][v] = __builtin_fmaf(g, w[H - k][v], acc[k][v]);
                        if (FULL || t < upto) {
#pragma unroll
                            for (int j = 0; j < H; ++j)
                                dw[j][v] = __builtin_fmaf(g, xw[j][v], dw[j][v]);
                            dw[H][v] = __builtin_fmaf(g, xc[v], dw[H][v]);
                            db[v] += g;
                        }
#pragma unroll
                        for (int k = 0; k + 1 < H; ++k) xw[k][v] = xw[k + 1][v];
                        xw[H - 1][v] = xc[v];
                    }
                }
                const int s = t - H;  // complete now
                if (FULL || (s >= from && s < upto)) put4(dx + static_cast<int64_t>(s) * p.dx.tok, acc[H]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
#pragma unroll
                    for (int k = H; k > 0; --k) acc[k][v] = acc[k - 1][v];
                    acc[0][v] = 0.0f;
                }
            }
        };
        for (int tb = from; tb < upto + H; tb += kConvBwdAhead) {
            if (tb - H >= max(t0, from) && tb + kConvBwdAhead <= min(t1, upto))
                block(tb, std::true_type());
            else
                block(tb, std::false_type());
        }
    }
    float* part = p.part + static_cast<int64_t>(run) * (W + 1) * p.C + c0;
#pragma unroll
    for (int j = 0; j < W; ++j) put4(part + static_cast<int64_t>(j) * p.C, dw[j]);
    put4(part + static_cast<int64_t>(W) * p.C, db);
}

__global__ void __launch_bounds__(256) conv_bwd_reduce(const ConvGrad p) {
    const int64_t n = static_cast<int64_t>(p.W + 1) * p.C;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    double s0 = 0.0, s1 = 0.0;
    int r = 0;
    for (; r + 8 <= p.runs; r += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p.part[(r + k) * n + i];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            s0 += static_cast<double>(v[k]);
            s1 += static_cast<double>(v[k + 1]);
        }
    }
    for (; r < p.runs; ++r) s0 += static_cast<double>(p.part[r * n + i]);
    const int j = static_cast<int>(i / p.C), c = static_cast<int>(i - static_cast<int64_t>(j) * p.C);
    const float v = static_cast<float>(s0 + s1);
    if (j < p.W) p.dweight[c * p.dw_chan + j] = v;
    else if (p.dbias) p.dbias[c] = v;
}

template <int W, typename WT> hipError_t conv_bwd_w(const ConvGrad& p, hipStream_t s) {
    const dim3 grid(scan_blocks(static_cast<int64_t>(p.runs) * ((p.C / 4 + 63) / 64)));
    if (p.runs) {
        if (p.silu)
            hipLaunchKernelGGL((conv_bwd_kernel<W, WT, true>), grid, dim3(kScanThreads), 0, s, p);
        else
            hipLaunchKernelGGL((conv_bwd_kernel<W, WT, false>), grid, dim3(kScanThreads), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t n = static_cast<int64_t>(W + 1) * p.C;
    hipLaunchKernelGGL(conv_bwd_reduce, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0,
                       s, p);
    return hipGetLastError();
}

template <typename WT> hipError_t conv_bwd_wt(const ConvGrad& p, hipStream_t s) {
    switch (p.W) {
        case 2: return conv_bwd_w<2, WT>(p, s);
        case 3: return conv_bwd_w<3, WT>(p, s);
        case 4: return conv_bwd_w<4, WT>(p, s);
        default: return hipErrorInvalidValue;
    }
}

// ------------------------------------------------------------------- fold ---

// History behind the first n tokens of a row: entry i is the input H - i tokens
// back, from the row or, where the row has none, from the history before it.
// A thread reads all that it replaces before it writes.
template <typename WT> __global__ void __launch_bounds__(256) conv_fold_kernel(const ConvFold p) {
    const int ctiles = (p.C / 4 + 255) / 256;
    const int b = blockIdx.x / ctiles;
    const int c0 = ((blockIdx.x - b * ctiles) * 256 + threadIdx.x) * 4;
    const uint32_t t0 = p.offsets[b], len = p.offsets[b + 1] - t0, n = p.accepted[b];
    const uint32_t slot = p.slot_idx ? p.slot_idx[b] : static_cast<uint32_t>(b);
    if (c0 >= p.C || n == 0 || n > len || (p.slot_idx != nullptr && slot == kPadSlot)) return;
    WT* st = static_cast<WT*>(p.state) + static_cast<int64_t>(slot) * p.st_slot + c0;
    const WT* x = static_cast<const WT*>(p.x.p) + c0;
    float v[3][4];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i >= p.H) break;
        const int64_t at = static_cast<int64_t>(n) - p.H + i;  // in the row
        if (at >= 0) scan_load<4>(x + (static_cast<int64_t>(t0) + at) * p.x.tok, v[i]);
        else scan_load<4>(st + (at + p.H) * p.st_tok, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i >= p.H) break;
        put4(st + i * p.st_tok, v[i]);
    }
}

}  // namespace

hipError_t launch_conv_bwd(const ConvGrad& p, bool work_bf16, hipStream_t s) {
    return work_bf16 ? conv_bwd_wt<uint16_t>(p, s) : conv_bwd_wt<float>(p, s);
}

hipError_t launch_conv_fold(const ConvFold& p, bool work_bf16, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.B) * ((p.C / 4 + 255) / 256));
    if (work_bf16) hipLaunchKernelGGL(conv_fold_kernel<uint16_t>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(conv_fold_kernel<float>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gdr

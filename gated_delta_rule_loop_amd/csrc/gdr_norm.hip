// gfx950 kernels of the norms before and after a block, fused with the
// block's gate and residual scale:
//     p = y / rms_group(y) * w1,   h = x + c act(gate) p,   n = h / rms(h) * w2
// and their gradients.  One workgroup holds a whole row of D values in
// registers (8 neighbouring values a thread and step), so every input is read
// once and every output written once; the arithmetic and the sums of squares
// are float32.  Bound by HBM: 16384 rows of 4096 bf16 with a gate and a norm per
// head (403 MB) take 86 us, 4.7 TB/s of the 5.2 that a large copy reaches.
#include "gdr_norm.h"

#include <algorithm>

#include "gdr_linattn_dev.h"

namespace gdr {
namespace {

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = la_round(v[2 * i]) | (static_cast<uint32_t>(la_round(v[2 * i + 1])) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8(const NormVec& w, int i, float (&v)[8]) {
    if (w.bf16) load8(static_cast<const uint16_t*>(w.p) + i, v);
    else load8(static_cast<const float*>(w.p) + i, v);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Sums over the workgroup, the same bits in every thread, with one barrier
// each: `red` holds a float per wave in each of kSlots slots used in turn, so
// that a slot's last readers are barriers away from its next writers.
constexpr int kSlots = 4;
struct BlockSums {
    float* red;
    int slot = 0;
    __device__ explicit BlockSums(float* r) : red(r) {}
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
        const int waves = blockDim.x >> 6;
        if (waves == 1) return;
        float* const r = red + slot * 16 * 2;
        slot = (slot + 1) % kSlots;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) r[i * 16 + (threadIdx.x >> 6)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float sum = 0.0f;
            for (int k = 0; k < waves; ++k) sum += r[i * 16 + k];
            v[i] = sum;
        }
    }
};
constexpr int kRedFloats = kSlots * 2 * 16;

// How the values of a group share a sum (group / 8 units of 8 values each).
enum GroupMode { kNoNorm, kWholeRow, kLanes, kAny };

// Sums of v[i] (one value per unit tid + i * threads) over each unit's group.
template <int NV, int GM>
__device__ __forceinline__ void group_sum(float (&v)[NV], int gu, int units, BlockSums& block,
                                          float* per_unit) {
    if constexpr (GM == kWholeRow) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) s[0] += v[i];
        block(s);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = s[0];
    } else if constexpr (GM == kLanes) {  // gu is a power of two up to 64
        for (int d = 1; d < gu; d <<= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], d);
    } else if constexpr (GM == kAny) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) per_unit[u] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            float s = 0.0f;
            if (u < units)
                for (int k = u / gu * gu, e = k + gu; k < e; ++k) s += per_unit[k];
            v[i] = s;
        }
        __syncthreads();
    }
}

template <typename T, int NV, int GM, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormParams p) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    BlockSums block(lds);
    float* per_unit = lds + kRedFloats;   // [units], kAny only
    const int64_t t = blockIdx.x;
    const int units = p.D >> 3, gu = p.group >> 3;
    const T* y = static_cast<const T*>(p.y) + t * p.y_row;
    const T* x = static_cast<const T*>(p.x) + t * p.x_row;
    const T* gt = static_cast<const T*>(p.gate) + t * p.gate_row;
    float yv[NV][8], xv[NV][8], gv[NV][8], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < p.D) {
            load8(y + c, yv[i]);
            if (p.x) load8(x + c, xv[i]);
            if (p.gate_mode == 1) load8(gt + c, gv[i]);
            else if (p.gate_mode == 2) load8(p.gate_c, c, gv[i]);
        }
        r[i] = 0.0f;
        if (GM != kNoNorm && c < p.D)
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i] = fmaf(yv[i][e], yv[i][e], r[i]);
    }
    if constexpr (GM != kNoNorm) {
        group_sum<NV, GM>(r, gu, units, block, per_unit);
#pragma unroll
        for (int i = 0; i < NV; ++i) r[i] = 1.0f / sqrtf(r[i] / static_cast<float>(p.group) + p.eps);
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < p.D) {
            if constexpr (GM != kNoNorm) {
                float w[8];
                load8(p.w1, p.w1_len == p.D ? c : c % p.w1_len, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) yv[i][e] *= r[i] * w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = p.c * yv[i][e];
                if (p.gate_mode) {
                    const float z = gv[i][e];
                    u *= p.act == 0 ? z : p.act == 1 ? sigmoid(z) : z * sigmoid(z);
                }
                if (p.x) u += xv[i][e];
                yv[i][e] = u;
                sq[0] = fmaf(u, u, sq[0]);
            }
            store8(static_cast<T*>(p.h) + t * p.h_row + c, yv[i]);
        }
    }
    if (!p.w2.p) return;
    // n is the norm of h before h's rounding
    block(sq);
    const float rh = 1.0f / sqrtf(sq[0] / static_cast<float>(p.D) + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < p.D) {
            float w[8];
            load8(p.w2, c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) yv[i][e] *= rh * w[e];
            store8(static_cast<T*>(p.n) + t * p.n_row + c, yv[i]);
        }
    }
}

// The gradients.  With H = dh + (the pre-norm's gradient by h) the total
// gradient of h: dx = H; dgate = c H p act'; dp = c H act;
// dy = r (dp w1 - y^ mean_group(dp w1 y^)), y^ = y r.  Workgroup b takes rows
// b, b + parts, ...; it sums its rows' weight gradients in registers and writes
// them once, and norm_reduce_kernel adds the parts in order.  8192 rows of 4096 bf16,
// gated per head (336 MB): 80 us with the reduction, 4.2 TB/s.
template <typename T, int NV, int GM, int THREADS>
__global__ void __launch_bounds__(THREADS, 4) norm_bwd_kernel(const NormParams p) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    BlockSums block(lds);
    float* per_unit = lds + kRedFloats;   // [units] kAny, [D] to fold a shared weight
    const int units = p.D >> 3, gu = p.group >> 3;
    float a1[NV][8], a2[NV][8], ag[NV][8], w1[NV][8], w2[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) a1[i][e] = a2[i][e] = ag[i][e] = 0.0f;
        if (c < p.D) {
            if (GM != kNoNorm) load8(p.w1, p.w1_len == p.D ? c : c % p.w1_len, w1[i]);
            if (p.w2.p) load8(p.w2, c, w2[i]);
        }
    }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float H[NV][8], yv[NV][8], gv[NV][8], r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            r[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) H[i][e] = yv[i][e] = gv[i][e] = 0.0f;
            if (c < p.D) {
                load8(static_cast<const T*>(p.dh) + t * p.dh_row + c, H[i]);
                load8(static_cast<const T*>(p.y) + t * p.y_row + c, yv[i]);
                if (p.gate_mode == 1)
                    load8(static_cast<const T*>(p.gate) + t * p.gate_row + c, gv[i]);
                else if (p.gate_mode == 2)
                    load8(p.gate_c, c, gv[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[i] = fmaf(yv[i][e], yv[i][e], r[i]);
            }
        }
        if (p.w2.p) {
            // with a norm over whole rows its squares are summed along
            float hv[NV][8], tv[NV][8], sq[2] = {0.0f, 0.0f}, dot[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) hv[i][e] = tv[i][e] = 0.0f;
                if (c < p.D) {
                    load8(static_cast<const T*>(p.h) + t * p.h_row + c, hv[i]);
                    load8(static_cast<const T*>(p.dn) + t * p.dn_row + c, tv[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq[0] = fmaf(hv[i][e], hv[i][e], sq[0]);
                }
                sq[1] += r[i];
            }
            block(sq);
            if constexpr (GM == kWholeRow)
#pragma unroll
                for (int i = 0; i < NV; ++i) r[i] = sq[1];
            const float rh = 1.0f / sqrtf(sq[0] / static_cast<float>(p.D) + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
                if (c < p.D) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        hv[i][e] *= rh;
                        a2[i][e] = fmaf(tv[i][e], hv[i][e], a2[i][e]);
                        tv[i][e] *= w2[i][e];
                        dot[0] = fmaf(tv[i][e], hv[i][e], dot[0]);
                    }
                }
            }
            block(dot);
            const float mean = dot[0] / static_cast<float>(p.D);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
                if (c < p.D) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        H[i][e] = fmaf(rh, fmaf(-hv[i][e], mean, tv[i][e]), H[i][e]);
                    if (p.dx) store8(static_cast<T*>(p.dx) + t * p.dx_row + c, H[i]);
                }
            }
        } else if (p.dx) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
                if (c < p.D) store8(static_cast<T*>(p.dx) + t * p.dx_row + c, H[i]);
            }
        }
        if constexpr (GM != kNoNorm) {
            if (GM != kWholeRow || !p.w2.p) group_sum<NV, GM>(r, gu, units, block, per_unit);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                r[i] = 1.0f / sqrtf(r[i] / static_cast<float>(p.group) + p.eps);
        }
        float dot[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            dot[i] = 0.0f;
            if (c < p.D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float hat = GM == kNoNorm ? yv[i][e] : yv[i][e] * r[i];
                    const float wt = GM == kNoNorm ? 1.0f : w1[i][e];
                    float dp = p.c * H[i][e];
                    if (p.gate_mode) {
                        const float z = gv[i][e];
                        float a = z, d = 1.0f;
                        if (p.act) {
                            const float s = sigmoid(z);
                            a = p.act == 1 ? s : z * s;
                            d = p.act == 1 ? s * (1.0f - s) : s * fmaf(z, 1.0f - s, 1.0f);
                        }
                        const float dg = dp * hat * wt * d;
                        gv[i][e] = dg;
                        ag[i][e] += dg;
                        dp *= a;
                    }
                    if constexpr (GM != kNoNorm) {
                        a1[i][e] = fmaf(dp, hat, a1[i][e]);
                        dp *= wt;
                        dot[i] = fmaf(dp, hat, dot[i]);
                    }
                    yv[i][e] = hat;
                    H[i][e] = dp;
                }
                if (p.dgate) store8(static_cast<T*>(p.dgate) + t * p.dgate_row + c, gv[i]);
            }
        }
        if constexpr (GM != kNoNorm) group_sum<NV, GM>(dot, gu, units, block, per_unit);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            if (c < p.D) {
                if constexpr (GM != kNoNorm) {
                    const float mean = dot[i] / static_cast<float>(p.group);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        H[i][e] = r[i] * fmaf(-yv[i][e], mean, H[i][e]);
                }
                store8(static_cast<T*>(p.dy) + t * p.dy_row + c, H[i]);
            }
        }
    }
    const int64_t b = blockIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < p.D) {
            if (p.pw2) store8(p.pw2 + b * p.D + c, a2[i]);
            if (p.pgate) store8(p.pgate + b * p.D + c, ag[i]);
            if (p.pw1 && p.w1_len == p.D) store8(p.pw1 + b * p.D + c, a1[i]);
        }
    }
    if (p.pw1 && p.w1_len != p.D) {       // the groups share the weight: add them up
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            if (c < p.D) store8(per_unit + c, a1[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.w1_len; c += blockDim.x) {
            float s = 0.0f;
            for (int k = c; k < p.D; k += p.w1_len) s += per_unit[k];
            p.pw1[b * p.w1_len + c] = s;
        }
    }
}

// Sums of up to three arrays of parts over the parts: 16 columns a workgroup,
// 64 threads down the parts of each column, whose sums are added in order.  Bound
// by its launch and two trips to memory: 512 parts of 128, 5 us.
struct NormReduces { NormReduce r[3]; };
constexpr int kReduceCols = 16, kReduceWalk = 64;
__global__ void __launch_bounds__(kReduceCols * kReduceWalk)
    norm_reduce_kernel(const NormReduces a) {
    __shared__ float lds[kReduceWalk][kReduceCols];
    const NormReduce& r = a.r[blockIdx.y];
    const int col = threadIdx.x % kReduceCols, walk = threadIdx.x / kReduceCols;
    const int c = blockIdx.x * kReduceCols + col;
    if (static_cast<int>(blockIdx.x) * kReduceCols >= r.n) return;
    float s = 0.0f;
    if (c < r.n) {
        const float* q = r.part + c;
        int k = walk;
        for (; k + 3 * kReduceWalk < r.parts; k += 4 * kReduceWalk) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = q[int64_t{k + i * kReduceWalk} * r.n];
#pragma unroll
            for (int i = 0; i < 4; ++i) s += v[i];
        }
        for (; k < r.parts; k += kReduceWalk) s += q[int64_t{k} * r.n];
    }
    lds[walk][col] = s;
    __syncthreads();
    if (walk < 4) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kReduceWalk / 4; ++k) sum += lds[walk * (kReduceWalk / 4) + k][col];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (walk == 0 && c < r.n) la_store(r.out, c, r.out_bf16, sum);
    }
}

// Threads of a workgroup that holds a row at NV units of 8 values a thread.
int row_threads(int D, int nv) {
    const int units = D / 8;
    int t = 64;
    while (t * nv < units && t < 1024) t *= 2;
    return t;
}

// Units of 8 values a thread, where a row fits 1024 threads that way.  bf16, us with
// one and two: residual and both norms 8192 x 8192 147 and 150, 4096 x 4096 34.6 and
// 36.2, 4096 x 2048 21.2 and 23.0; a gate alone (fewer loads in flight a thread)
// 16384 x 4096 103 and 101.  Gradients hold three times the values: one.
constexpr int kBwdUnits = 1;
int fwd_units(const NormParams& p) { return p.x ? 1 : 2; }

int group_mode(const NormParams& p) {
    if (!p.w1.p) return kNoNorm;
    if (p.group == p.D) return kWholeRow;
    const int gu = p.group / 8;
    return gu <= 64 && (gu & (gu - 1)) == 0 ? kLanes : kAny;
}

template <typename T, int NV, int THREADS, bool BWD>
hipError_t run_mode(const NormParams& p, int threads, hipStream_t s) {
    const int gm = group_mode(p);
    uint32_t lds = kRedFloats * sizeof(float);
    if (gm == kAny) lds += p.D / 8 * sizeof(float);
    if (BWD && p.pw1 && p.w1_len != p.D) lds = static_cast<uint32_t>((kRedFloats + p.D) * sizeof(float));
    const dim3 grid(static_cast<uint32_t>(BWD ? p.parts : p.T));
#define GDR_NORM_RUN(GM)                                                        \
    do {                                                                        \
        if constexpr (BWD) norm_bwd_kernel<T, NV, GM, THREADS><<<grid, threads, lds, s>>>(p); \
        else norm_kernel<T, NV, GM, THREADS><<<grid, threads, lds, s>>>(p);     \
    } while (0)
    if (gm == kNoNorm) GDR_NORM_RUN(kNoNorm);
    else if (gm == kWholeRow) GDR_NORM_RUN(kWholeRow);
    else if (gm == kLanes) GDR_NORM_RUN(kLanes);
    else GDR_NORM_RUN(kAny);
#undef GDR_NORM_RUN
    return hipGetLastError();
}

template <typename T, bool BWD, int units>
hipError_t run(const NormParams& p, hipStream_t s) {
    const int threads = row_threads(p.D, units);
    if (threads * units * 8 < p.D) return run_mode<T, 2, 1024, BWD>(p, 1024, s);
    if (threads <= 256) return run_mode<T, units, 256, BWD>(p, threads, s);
    if (threads <= 512) return run_mode<T, units, 512, BWD>(p, threads, s);
    return run_mode<T, units, 1024, BWD>(p, threads, s);
}

}  // namespace

int norm_parts(int64_t T, int D) {
    // as many workgroups as the chip holds at 16 waves a compute unit, with rows
    // shared evenly
    const int64_t most = std::min<int64_t>(1024, 256 * 16 * 64 / row_threads(D, kBwdUnits));
    const int64_t rows = (T + most - 1) / most;  // of the fullest workgroup
    return static_cast<int>((T + rows - 1) / rows);
}

int norm_threads(const NormParams& p) { return row_threads(p.D, fwd_units(p)); }

hipError_t launch_norm(const NormParams& p, bool work_bf16, hipStream_t s) {
    if (fwd_units(p) == 1)
        return work_bf16 ? run<uint16_t, false, 1>(p, s) : run<float, false, 1>(p, s);
    return work_bf16 ? run<uint16_t, false, 2>(p, s) : run<float, false, 2>(p, s);
}
hipError_t launch_norm_bwd(const NormParams& p, bool work_bf16, hipStream_t s) {
    return work_bf16 ? run<uint16_t, true, kBwdUnits>(p, s) : run<float, true, kBwdUnits>(p, s);
}
hipError_t launch_norm_reduce(const NormReduce* r, int count, hipStream_t s) {
    NormReduces a{};
    int n = 0;
    for (int i = 0; i < count; ++i) {
        a.r[i] = r[i];
        n = r[i].n > n ? r[i].n : n;
    }
    norm_reduce_kernel<<<dim3((n + kReduceCols - 1) / kReduceCols, count),
                         kReduceCols * kReduceWalk, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdr

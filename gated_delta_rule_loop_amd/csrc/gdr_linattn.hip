// gfx950 kernels around the walks of linear attention with a decay for each
// head: the token-by-token form, the scan that turns the segments' sums into
// the states they start from, the decays' gradient, and the sum over a group's
// heads.
#include "gdr_linattn_dev.h"

namespace gdr {
namespace {

// ------------------------------------------------------------------- step ---

// Rows of one or a few tokens.  A workgroup holds one (row, value head) state:
// thread (rg, cg) of K/8 x V/8 threads holds rows rg + i * K/8, i < 8, of 8
// neighbouring columns, so a wave's accesses cover whole rows.  Per token
// every thread updates its block and sums its rows' share of the read-out;
// the shares of a column's K/8 threads meet in LDS and are added in order.
// Bound by HBM: the state is read and written once (bytes = 2 K V per head).
// 256 rows, 32 heads, K = V = 128, bf16 states: 107 us, 5.1 TB/s (a large copy
// reaches 5.2; through the caches 114 us).  One row: 5.8 us, three dependent
// trips to memory and the launch.
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

// A state is read and written once a call: its lines are streamed past the
// caches (16 bytes a lane, whole lines a wave).
template <typename E> __device__ __forceinline__ void stream_in(const E* p, float (&v)[8]) {
    constexpr int N = sizeof(E) / 2;
    __attribute__((aligned(16))) E raw[8];
#pragma unroll
    for (int i = 0; i < N; ++i)
        reinterpret_cast<la_u4*>(raw)[i] =
            __builtin_nontemporal_load(reinterpret_cast<const la_u4*>(p) + i);
    load8(raw, v);
}
template <typename E> __device__ __forceinline__ void stream_out(E* p, const float (&v)[8]) {
    constexpr int N = sizeof(E) / 2;
    __attribute__((aligned(16))) E raw[8];
    store8(raw, v);
#pragma unroll
    for (int i = 0; i < N; ++i)
        __builtin_nontemporal_store(reinterpret_cast<const la_u4*>(raw)[i],
                                    reinterpret_cast<la_u4*>(p) + i);
}

template <typename T, typename ST, int THREADS>
__global__ void __launch_bounds__(THREADS) step_kernel(const LaStep p) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int K8 = p.K >> 3, V8 = p.V >> 3;
    float* qs = lds;                      // [K]
    float* ks = lds + p.K;                // [K]
    float* part = lds + 2 * p.K;          // [K8][V]
    const int head = blockIdx.x % p.nv, row = blockIdx.x / p.nv;
    const int tid = threadIdx.x;
    const int rg = tid / V8, cg = tid % V8;
    const bool on = rg < K8;
    int t0 = row, n = 1;
    if (p.offsets) {
        t0 = static_cast<int>(p.offsets[row]);
        n = static_cast<int>(p.offsets[row + 1]) - t0;
        if (n > p.most) return;           // walked in chunks
    }
    T* out = static_cast<T*>(p.out) + head * p.o_head;
    const uint32_t slot = p.slot_idx ? p.slot_idx[row] : static_cast<uint32_t>(row);
    if (slot == kPadSlot) {
        for (int t = 0; t < n; ++t)
            for (int c = tid; c < p.V; c += blockDim.x) out[(int64_t{t0} + t) * p.o_tok + c] = T(0);
        return;
    }
    if (n <= 0 && p.in.p == p.last.p) return;
    float S[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) S[i][c] = 0.0f;
    if (on && p.in.p) {
        const ST* s = static_cast<const ST*>(p.in.p) + int64_t{slot} * p.in.outer +
                      head * p.in.head + rg * p.V + cg * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) stream_in(s + i * K8 * p.V, S[i]);
    }
    const T* q = static_cast<const T*>(p.q) + (head / p.G) * p.q_head;
    const T* k = static_cast<const T*>(p.k) + (head / p.G) * p.k_head;
    const T* v = static_cast<const T*>(p.v) + head * p.v_head + cg * 8;
    for (int t = 0; t < n; ++t) {
        const int64_t at = int64_t{t0} + t;
        float vv[8];
        if (on) load8(v + at * p.v_tok, vv);
        for (int i = tid; i < p.K; i += blockDim.x) {
            qs[i] = la_load(q, at * p.q_tok + i, sizeof(T) == 2);
            ks[i] = la_load(k, at * p.k_tok + i, sizeof(T) == 2);
        }
        const float a = p.g ? expf(la_clamp_g(la_load(p.g, at * p.g_tok + head * p.g_head,
                                                      p.g_bf16)))
                            : 1.0f;
        __syncthreads();
        if (on) {
            float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float kk = ks[rg + i * K8], qq = qs[rg + i * K8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    S[i][c] = fmaf(kk, vv[c], a * S[i][c]);
                    o[c] = fmaf(qq, S[i][c], o[c]);
                }
            }
            store8(part + rg * p.V + cg * 8, o);
        }
        __syncthreads();
        for (int c = tid; c < p.V; c += blockDim.x) {
            float o = 0.0f;
            for (int r = 0; r < K8; ++r) o += part[r * p.V + c];
            o *= p.scale;
            la_store(out, at * p.o_tok + c, sizeof(T) == 2, o);
        }
    }
    if (on && p.last.p) {
        ST* s = static_cast<ST*>(p.last.p) + int64_t{slot} * p.last.outer + head * p.last.head +
                rg * p.V + cg * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) stream_out(s + i * K8 * p.V, S[i]);
    }
}

template <typename T, typename ST>
hipError_t run_step(const LaStep& p, hipStream_t s) {
    const int threads = static_cast<int>(la_step_threads(p.K, p.V));
    const uint32_t lds = static_cast<uint32_t>((2 * p.K + (p.K / 8) * p.V) * sizeof(float));
    const dim3 grid(static_cast<uint32_t>(p.B) * p.nv);
    if (threads <= 256)
        step_kernel<T, ST, 256><<<grid, threads, lds, s>>>(p);
    else
        step_kernel<T, ST, 1024><<<grid, threads, lds, s>>>(p);
    return hipGetLastError();
}

// ------------------------------------------------------------------- scan ---

// A thread carries 4 elements of a (row, head) state over the row's segments:
// each segment's sum is replaced by the state that its walk starts from.  The
// sums are loaded four steps ahead.  blockIdx.y: the scans of one launch.
// Bound by the latency of a row's segments in turn: the 16 of 32768 tokens at 32
// heads, K = V = 128: 14 us for 67 MB.
struct LaScans { LaScan c[2]; };
__global__ void __launch_bounds__(kLaScanThreads) scan_kernel(const LaScans both) {
    const LaScan& p = both.c[blockIdx.y];
    const int blocks = la_scan_blocks(p.n);      // of a state
    const int which = blockIdx.x / blocks;
    const int head = which % p.nv;
    LaSpan sp;                            // of the rows that are walked, as one segment each
    if (!la_locate(p.offsets, p.B, p.walk_from ? 0x7FFFFFFF : 0, p.walk_from, which / p.nv, sp))
        return;
    const int row = __builtin_amdgcn_readfirstlane(sp.row);
    const int i = ((blockIdx.x % blocks) * kLaScanThreads + threadIdx.x) * 4;
    // the row's first segment
    int first = 0;
    for (int b = threadIdx.x & 63; b < row; b += 64)
        first += la_row_segs(static_cast<int>(p.offsets[b + 1] - p.offsets[b]), p.seg_len,
                             p.walk_from);
    for (int d = 1; d < 64; d <<= 1) first += __shfl_xor(first, d);
    first = __builtin_amdgcn_readfirstlane(first);
    const int count = la_row_segs(static_cast<int>(p.offsets[row + 1] - p.offsets[row]),
                                  p.seg_len, p.walk_from);
    if (i >= p.n) return;
    const uint32_t slot = p.slot_idx ? p.slot_idx[row] : static_cast<uint32_t>(row);
    if (slot == kPadSlot) return;
    la_f4 run = {0, 0, 0, 0};
    if (p.in.p) {
        const int64_t base = int64_t{slot} * p.in.outer + head * p.in.head + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) run[e] = p.in.mult * la_load(p.in.p, base + e, p.in.bf16);
    }
    const int64_t step = (p.reverse ? -1 : 1) * int64_t{p.nv} * p.n;
    const int from = first + (p.reverse ? count - 1 : 0);
    float* q = p.state + (int64_t{from} * p.nv + head) * p.n + i;
    const float* tot = p.tot + (int64_t{p.reverse} * p.segs + from) * p.nv + head;
    const int tot_step = p.reverse ? -p.nv : p.nv;
    constexpr int AHEAD = 4;
    la_f4 own[AHEAD];
    float a[AHEAD];
    auto fetch = [&](int j, int e) {      // of the last segment nothing is needed
        const int c = min(j, count - 2);
        own[e] = *reinterpret_cast<const la_f4*>(q + c * step);
        a[e] = tot[c * tot_step];
    };
    if (count > 1)
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) fetch(e, e);
    for (int j = 0; j < count; j += AHEAD) {
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            if (j + e >= count) break;
            *reinterpret_cast<la_f4*>(q + (j + e) * step) = run;
            if (j + e + 1 < count) {
                run = run * exp2f(a[e]) + own[e];
                if (j + e + AHEAD < count - 1) fetch(j + e + AHEAD, e);
            }
        }
    }
}

// ---------------------------------------------------------- decay gradient ---

// dg_j = sum_{i >= j} (q_i . dq_i - k_i . dk_i) + phi(end), the tokens' own pairs
// left out of both products, phi = <S, dL/dS> at a segment's end.  One workgroup
// per (segment, head) sums from the segment's end, 256 tokens at a time, in
// float64: the terms telescope, so what is left is a small difference of sums
// whose rounding errors add up like a random walk.  The sum over the whole
// segment has to be phi(start) - phi(end), both known; what it misses is the sum
// of the terms' errors.  A term's error is a few roundings of its parts, so each
// term takes back its share by the square of the parts' absolute sum: the likeliest
// split of a sum of independent errors of those sizes.  A few large tokens thus
// keep their own error (by equal shares they would put it on the small terms of
// others).  float32, 512 tokens of unit size: 0.5 to 0.95 of the error without;
// with the first 4 of 180 a hundred times the others' size, the later half's
// error is 5.1e-7 of its values, as with all alike (by equal shares 7.7e-3).
// Bound by the launch and a few dependent loads: 2 x 2048 tokens, 16 heads, 7 us.
__device__ __forceinline__ double phi_at(const float* phi, int64_t i, int parts) {
    const float* f = phi + i * parts;
    double sum = 0.0;
    for (int k = 0; k < parts; k += 4)
        sum += (static_cast<double>(f[k]) + f[k + 1]) + (static_cast<double>(f[k + 2]) + f[k + 3]);
    return sum;
}

__global__ void __launch_bounds__(256) decay_grad_kernel(const LaDecayGrad p) {
    __shared__ double wsum[8];
    const int head = blockIdx.x % p.nv, seg = blockIdx.x / p.nv;
    LaSpan sp;
    if (!la_locate(p.offsets, p.B, p.seg_len, 0, seg, sp)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t at = int64_t{seg} * p.nv + head, part = int64_t{p.nv} * p.T;
    const double end = p.phi ? phi_at(p.phi, at, p.parts) : 0.0;
    double begin = 0.0;
    if (sp.s > 0) begin = phi_at(p.phi, at - p.nv, p.parts);
    else if (p.phi0) begin = phi_at(p.phi0, at, p.parts0);
    // the term of the r-th token from the segment's end, and the square of its size
    auto term = [&](int r, double& square) {
        double v = 0.0, size = 0.0;
        if (r < sp.n) {
            const int64_t i = int64_t{head} * p.T + sp.t0 + sp.n - 1 - r;
            for (int k = 0; k < p.parts; k += 4) {  // in flight together
                float a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = p.rq[(k + e) * part + i];
                    b[e] = p.rk[(k + e) * part + i];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v += static_cast<double>(a[e]) - b[e];
                    size += static_cast<double>(fabsf(a[e])) + fabsf(b[e]);
                }
            }
        }
        square = size * size;
        return v;
    };
    double first_square, squares;
    const double first = term(tid, first_square);
    double all = first;
    squares = first_square;
    for (int r = 256 + tid; r < sp.n; r += 256) {
        double square;
        all += term(r, square);
        squares += square;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        all += __shfl_xor(all, d);
        squares += __shfl_xor(squares, d);
    }
    if (lane == 0) {
        wsum[wave] = all;
        wsum[4 + wave] = squares;
    }
    __syncthreads();
    all = (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
    squares = (wsum[4] + wsum[5]) + (wsum[6] + wsum[7]);
    __syncthreads();
    // by each square; nothing where the terms are zeros or not finite
    double missed = (begin - end - all) / squares;
    if (!isfinite(missed)) missed = 0.0;
    double carry = end;
    for (int r0 = 0; r0 < sp.n; r0 += 256) {  // r counts from the segment's end
        const int r = r0 + tid;
        double square = first_square;
        double v = r0 ? term(r, square) : first;
        if (missed != 0.0) v += missed * square;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(v, d);
            if (lane >= d) v += up;
        }
        if (lane == 63) wsum[wave] = v;
        __syncthreads();
        double before = carry;
        for (int i = 0; i < 4; ++i) {
            if (i < wave) before += wsum[i];
            carry += wsum[i];
        }
        if (r < sp.n)
            la_store(p.dg, (int64_t{sp.t0} + sp.n - 1 - r) * p.dg_tok + head * p.dg_head, p.dg_bf16,
                     static_cast<float>(before + v));
        __syncthreads();
    }
}

// --------------------------------------------------------------- head sums ---

// Gradients of key heads that G value heads share: the heads' float32 parts
// added in order and rounded once.  Tokens of no row are left alone: the walks
// wrote no parts for them.  1507 tokens, 4 key heads of 64: 4.3 us, the launch's
// own time.
template <typename T>
__global__ void __launch_bounds__(256) head_sum_kernel(const LaHeadSum p) {
    const int K4 = p.K >> 2;
    const int64_t i = int64_t{blockIdx.x} * 256 + threadIdx.x;
    if (i >= int64_t{p.T} * p.nk * K4) return;
    const int c = static_cast<int>(i % K4) * 4;
    const int64_t th = i / K4, t = th / p.nk;
    if (t < int64_t{p.offsets[0]} || t >= int64_t{p.offsets[p.B]}) return;
    const float* s = p.part + th * p.G * p.K + c;
    la_f4 sum = {0, 0, 0, 0};
    for (int m = 0; m < p.G; ++m) sum += *reinterpret_cast<const la_f4*>(s + int64_t{m} * p.K);
    T* o = static_cast<T*>(p.out) + t * p.out_tok + th % p.nk * p.out_head + c;
    if constexpr (sizeof(T) == 2) {
        la_b4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = static_cast<__bf16>(sum[e]);
        *reinterpret_cast<la_b4*>(o) = b;
    } else {
        *reinterpret_cast<la_f4*>(o) = sum;
    }
}

}  // namespace

hipError_t launch_la_step(const LaStep& p, bool work_bf16, hipStream_t s) {
    const bool st16 = (p.in.p ? p.in.bf16 : p.last.bf16) != 0;
    if (work_bf16)
        return st16 ? run_step<uint16_t, uint16_t>(p, s) : run_step<uint16_t, float>(p, s);
    return st16 ? run_step<float, uint16_t>(p, s) : run_step<float, float>(p, s);
}

hipError_t launch_la_scans(const LaScan* c, int count, hipStream_t s) {
    LaScans both{};
    for (int i = 0; i < count; ++i) both.c[i] = c[i];
    const dim3 grid(static_cast<uint32_t>(la_scan_blocks(c->n)) * c->rows * c->nv,
                    static_cast<uint32_t>(count));
    scan_kernel<<<grid, kLaScanThreads, 0, s>>>(both);
    return hipGetLastError();
}

hipError_t launch_la_decay_grad(const LaDecayGrad& p, hipStream_t s) {
    decay_grad_kernel<<<dim3(static_cast<uint32_t>(p.segs) * p.nv), 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_la_head_sum(const LaHeadSum& p, bool work_bf16, hipStream_t s) {
    const int64_t n = int64_t{p.T} * p.nk * (p.K / 4);
    const dim3 grid(static_cast<uint32_t>((n + 255) / 256));
    if (work_bf16) head_sum_kernel<uint16_t><<<grid, 256, 0, s>>>(p);
    else head_sum_kernel<float><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t la_walks_f32(const LaParams& p, hipStream_t s);
hipError_t la_walks_bf16(const LaParams& p, hipStream_t s);
hipError_t la_segments_f32(const LaParams& p, float* tot, hipStream_t s);
hipError_t la_segments_bf16(const LaParams& p, float* tot, hipStream_t s);

hipError_t launch_la_walks(const LaParams& p, bool work_bf16, hipStream_t s) {
    return work_bf16 ? la_walks_bf16(p, s) : la_walks_f32(p, s);
}
hipError_t launch_la_segments(const LaParams& p, bool work_bf16, float* tot, hipStream_t s) {
    return work_bf16 ? la_segments_bf16(p, tot, s) : la_segments_f32(p, tot, s);
}

}  // namespace gdr

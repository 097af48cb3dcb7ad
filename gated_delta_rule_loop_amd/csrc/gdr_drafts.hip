// gfx950 kernels that verify drafted tokens against the target's probabilities.
//
// Token i >= 1 of a row's window is a draft; the target's row i - 1 says how
// likely it is.  Sampled: it stands while u_i q_i(x_i) < p_{i-1}(x_i), and the row
// goes on with a token drawn by u_0 from max(p - q, 0) at the first draft that
// falls, from p behind the last one otherwise.  The test compares exact products
// (24-bit factors in float64); the draw is the first index whose running sum of
// weights, in float64, exceeds u_0 times their whole sum.  One launch finds what
// stands (every workgroup for itself: two dependent loads) and sums the weights of a
// slice of the vocabulary, one picks the slice, then the index.  Greedy: one
// launch takes every target row's largest value and its lowest index by slices,
// one compares.  Bound by HBM (one vocabulary row of p and q a sequence, all of the
// target's rows greedily) and, for few rows, by the launches.  64 rows of 412 tokens together,
// 131072 bf16 scores each: 19 us and 4 (108 MB, 5.7 TB/s; a copy 5.1); 256
// rows of 50021 float32 probabilities 13 and 11 us; one row of 32000 4 and 7.
#include "gdr_scan_dev.h"

namespace gdr {
namespace {

constexpr int kDraftThreads = 256;

typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 neighbouring values from any address of their type.
__device__ __forceinline__ void any8(const float* p, float (&v)[8]) {
    const f4_any a = *reinterpret_cast<const f4_any*>(p);
    const f4_any b = *reinterpret_cast<const f4_any*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}
__device__ __forceinline__ void any8(const uint16_t* p, float (&v)[8]) {
    const u4_any a = *reinterpret_cast<const u4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}
template <typename PT> __device__ __forceinline__ void load8(const PT* p, int64_t n, float (&v)[8]) {
    if (n >= 8) {
        any8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? scan_value(p[i]) : 0.0f;
    }
}

__device__ __forceinline__ double weight(double w) {  // NaN, infinities and what is not positive: 0
    return w > 0.0 && w < __builtin_inf() ? w : 0.0;
}

// The row of the target that a sequence goes on from, and what is taken off it.
template <typename PT> struct Rest {
    const PT *p, *q;  // q: nullptr where nothing, or one token, is taken off
    int one;          // that token, -1: none
    __device__ __forceinline__ double at(int64_t j, float pv, float qv) const {
        double w = static_cast<double>(pv);
        if (q) w -= static_cast<double>(qv);
        if (j == one) w -= 1.0;
        return weight(w);
    }
};

template <typename PT>
__device__ __forceinline__ Rest<PT> rest_of(const DraftParams& p, int64_t a, int n, int len) {
    Rest<PT> r;
    r.p = static_cast<const PT*>(p.p) + (a + n - 1) * p.p_tok;
    r.q = n < len && p.q ? static_cast<const PT*>(p.q) + (a + n) * p.q_tok : nullptr;
    r.one = n < len && !p.q ? p.tokens[(a + n) * p.tok_stride] : -1;
    return r;
}

// Tokens of the window that stand (the first always does); the same in every lane.
template <typename PT>
__device__ __forceinline__ int standing(const DraftParams& p, int64_t a, int len) {
    const int lane = threadIdx.x & 63;
    for (int i0 = 1; i0 < len; i0 += 64) {
        const int i = i0 + lane;
        bool falls = false;
        if (i < len) {
            const int64_t x = p.tokens[(a + i) * p.tok_stride];
            falls = true;
            if (x >= 0 && x < p.V) {
                const double pv = scan_value((static_cast<const PT*>(p.p) + (a + i - 1) * p.p_tok)[x]);
                const double qv =
                    p.q ? static_cast<double>(scan_value((static_cast<const PT*>(p.q) + (a + i) * p.q_tok)[x]))
                        : 1.0;
                falls = !(static_cast<double>(p.u[(a + i) * p.u_stride]) * qv < pv);
            }
        }
        const uint64_t any = __ballot(falls);
        if (any) return i0 + __ffsll(static_cast<unsigned long long>(any)) - 1;
    }
    return len;
}

__device__ __forceinline__ double wave_sum(double v) {
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

template <typename PT>
__global__ void __launch_bounds__(kDraftThreads) drafts_sums(const DraftParams p) {
    __shared__ double red[2][kDraftThreads / 64];
    const int b = blockIdx.x / p.splits, s = blockIdx.x - b * p.splits;
    const int64_t a = p.offsets[b];
    const int len = static_cast<int>(p.offsets[b + 1] - p.offsets[b]);
    if (len <= 0) {
        if (s == 0 && threadIdx.x == 0) {
            p.accepted[b] = 0;
            p.next[b] = -1;
        }
        return;
    }
    const int n = standing<PT>(p, a, len);
    if (s == 0 && threadIdx.x == 0) p.accepted[b] = n;
    const Rest<PT> r = rest_of<PT>(p, a, n, len);
    const int64_t from = static_cast<int64_t>(s) * p.span;
    const int64_t upto = min(from + p.span, static_cast<int64_t>(p.V));
    double sum = 0.0, whole = 0.0;
    constexpr int kStep = kDraftThreads * 8;
    auto add = [&](int64_t j, const float (&pv)[8], const float (&qv)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum += r.at(j + i, pv[i], qv[i]);
            whole += weight(static_cast<double>(pv[i]));
        }
    };
    int64_t j = from + threadIdx.x * 8;
    for (; j + kStep + 8 <= upto; j += 2 * kStep) {  // two loads of each in flight
        float p0[8], p1[8], q0[8] = {}, q1[8] = {};
        any8(r.p + j, p0);
        any8(r.p + j + kStep, p1);
        if (r.q) {
            any8(r.q + j, q0);
            any8(r.q + j + kStep, q1);
        }
        add(j, p0, q0);
        add(j + kStep, p1, q1);
    }
    for (; j < upto; j += kStep) {
        float pv[8], qv[8] = {};
        load8(r.p + j, upto - j, pv);
        if (r.q) load8(r.q + j, upto - j, qv);
        add(j, pv, qv);
    }
    sum = wave_sum(sum);
    whole = wave_sum(whole);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        red[0][wave] = sum;
        red[1][wave] = whole;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double t = 0.0;
        for (int w = 0; w < kDraftThreads / 64; ++w) t += red[threadIdx.x][w];
        p.part[(static_cast<int64_t>(b) * 2 + threadIdx.x) * p.splits + s] = t;
    }
}

// Running sums over the workgroup's threads; `before`: of the threads before
// this one.  Returns the whole sum.
__device__ __forceinline__ double block_scan(double v, double* red, double& before) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double inc = v;
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    __syncthreads();  // red may still be read from an earlier scan
    if (lane == 63) red[wave] = inc;
    __syncthreads();
    double base = 0.0, all = 0.0;
    for (int w = 0; w < kDraftThreads / 64; ++w) {
        if (w == wave) base = all;
        all += red[w];
    }
    before = base + inc - v;
    return all;
}

// The first thread whose `yes` holds, else the last whose `some` does, else -1.
__device__ __forceinline__ int block_pick(bool yes, bool some, int* box) {
    __syncthreads();
    if (threadIdx.x == 0) {
        box[0] = kDraftThreads;
        box[1] = -1;
    }
    __syncthreads();
    if (yes) atomicMin(&box[0], static_cast<int>(threadIdx.x));
    if (some) atomicMax(&box[1], static_cast<int>(threadIdx.x));
    __syncthreads();
    return box[0] < kDraftThreads ? box[0] : box[1];
}

template <typename PT>
__global__ void __launch_bounds__(kDraftThreads) drafts_draw(const DraftParams p) {
    __shared__ double red[kDraftThreads / 64];
    __shared__ double carried, run_before;
    __shared__ int box[2], offset;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int64_t a = p.offsets[b];
    const int len = static_cast<int>(p.offsets[b + 1] - p.offsets[b]);
    if (len <= 0) return;
    const int n = p.accepted[b];
    Rest<PT> r = rest_of<PT>(p, a, n, len);
    const double* part = p.part + static_cast<int64_t>(b) * 2 * p.splits;
    double v = tid < p.splits ? part[tid] : 0.0, before;
    double all = block_scan(v, red, before);
    if (!(all > 0.0)) {  // nothing is left of it: draw from p itself
        r.q = nullptr;
        r.one = -1;
        v = tid < p.splits ? part[p.splits + tid] : 0.0;
        all = block_scan(v, red, before);
    }
    const double goal = static_cast<double>(p.u[a * p.u_stride]) * all;
    const int s = block_pick(v > 0.0 && before + v > goal, v > 0.0, box);
    if (s < 0) {  // no weight anywhere
        if (tid == 0) p.next[b] = -1;
        return;
    }
    if (tid == s) carried = before;
    __syncthreads();
    const double base = carried;
    // the slice's values, neighbouring ones to each thread
    const int each = p.span / kDraftThreads;
    const int64_t from = static_cast<int64_t>(s) * p.span + static_cast<int64_t>(tid) * each;
    const int64_t upto = min(from + each, static_cast<int64_t>(p.V));
    double sum = 0.0;
    for (int64_t j = from; j < upto; j += 8) {
        float pv[8], qv[8];
        load8(r.p + j, upto - j, pv);
        if (r.q) load8(r.q + j, upto - j, qv);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += r.at(j + i, pv[i], r.q ? qv[i] : 0.0f);
    }
    block_scan(sum, red, before);
    const int t = block_pick(sum > 0.0 && base + (before + sum) > goal, sum > 0.0, box);
    if (tid == t) {
        run_before = base + before;
        offset = static_cast<int>(from - static_cast<int64_t>(s) * p.span);
    }
    __syncthreads();
    // that thread's values, 64 at a time, one a lane of the first wave
    if (tid >= 64) return;
    const int64_t first = static_cast<int64_t>(s) * p.span + offset;
    const int64_t last = min(first + each, static_cast<int64_t>(p.V));
    double run = run_before;
    int64_t found = -1;  // the first that passes, else the last that has a weight
    for (int64_t j0 = first; j0 < last; j0 += 64) {
        const int64_t j = j0 + tid;
        double w = 0.0;
        if (j < last) w = r.at(j, scan_value(r.p[j]), r.q ? scan_value(r.q[j]) : 0.0f);
        double inc = w;
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(inc, d);
            if (tid >= d) inc += up;
        }
        const uint64_t some = __ballot(w > 0.0), yes = __ballot(w > 0.0 && run + inc > goal);
        if (yes) {
            found = j0 + __ffsll(static_cast<unsigned long long>(yes)) - 1;
            break;
        }
        if (some) found = j0 + 63 - __clzll(static_cast<long long>(some));
        run += __shfl(inc, 63);
    }
    if (tid == 0) p.next[b] = static_cast<int32_t>(found);
}

// ----------------------------------------------------------------- greedy ---

// Larger values first, then lower indices; 0: none (NaN is no value).
__device__ __forceinline__ uint64_t key_of(float v, uint32_t j) {
    if (v != v) return 0;
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 is 0
    const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<uint64_t>(o) << 32 | (0xFFFFFFFFu - j);
}
__device__ __forceinline__ uint64_t later(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <typename PT>
__global__ void __launch_bounds__(kDraftThreads) drafts_best(const DraftParams p) {
    __shared__ uint64_t red[kDraftThreads / 64];
    const int64_t t = blockIdx.x / p.splits;
    const int s = blockIdx.x - static_cast<int>(t) * p.splits;
    if (t < p.offsets[0] || t >= p.offsets[p.B]) return;
    const PT* row = static_cast<const PT*>(p.p) + t * p.p_tok;
    const int64_t from = static_cast<int64_t>(s) * p.span;
    const int64_t upto = min(from + p.span, static_cast<int64_t>(p.V));
    // A thread meets its values in rising order: the first of the largest stays.
    constexpr int kStep = kDraftThreads * 8, kAhead = 4;
    float top = -__builtin_inff();
    int at = -1;
    auto look = [&](int64_t j, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v[i] > top) {
                top = v[i];
                at = static_cast<int>(j) + i;
            }
    };
    const int64_t mine = from + threadIdx.x * 8;
    int64_t j = mine;
    for (; j + (kAhead - 1) * kStep + 8 <= upto; j += kAhead * kStep) {
        float v[kAhead][8];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) any8(row + j + k * kStep, v[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) look(j + k * kStep, v[k]);
    }
    for (; j < upto; j += kStep) {
        if (j + 8 <= upto) {
            float v[8];
            any8(row + j, v);
            look(j, v);
        } else {
            for (int64_t i = j; i < upto; ++i) {
                const float v = scan_value(row[i]);
                if (v > top) {
                    top = v;
                    at = static_cast<int>(i);
                }
            }
        }
    }
    if (at < 0)  // nothing above -inf: the first -inf itself, if there is one
        for (int64_t k = mine; k < upto && at < 0; k += kStep)
            for (int64_t i = k; i < min(k + 8, upto); ++i)
                if (at < 0 && scan_value(row[i]) == top) at = static_cast<int>(i);
    uint64_t best = at < 0 ? 0 : key_of(top, static_cast<uint32_t>(at));
    for (int d = 32; d; d >>= 1) best = later(best, __shfl_xor(best, d));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kDraftThreads / 64; ++w) best = later(best, red[w]);
        reinterpret_cast<uint64_t*>(p.part)[t * p.splits + s] = best;
    }
}

// 16 lanes a target row, 16 rows at a time.
__global__ void __launch_bounds__(kDraftThreads) drafts_compare(const DraftParams p) {
    __shared__ int best[kDraftThreads / 16];
    const int b = blockIdx.x;
    const int64_t a = p.offsets[b];
    const int len = static_cast<int>(p.offsets[b + 1] - p.offsets[b]);
    const uint64_t* part = reinterpret_cast<const uint64_t*>(p.part);
    const int lane = threadIdx.x & 15, mine = threadIdx.x >> 4;
    int n = 0, go = -1;
    bool done = len <= 0;
    for (int i0 = 0; i0 < len && !done; i0 += kDraftThreads / 16) {
        uint64_t k = 0;
        if (i0 + mine < len)
            for (int s = lane; s < p.splits; s += 16)
                k = later(k, part[(a + i0 + mine) * p.splits + s]);
        for (int d = 8; d; d >>= 1) k = later(k, __shfl_xor(k, d));
        __syncthreads();
        if (lane == 0)
            best[mine] = k ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)) : -1;
        __syncthreads();
        for (int i = 0; i < kDraftThreads / 16 && i0 + i < len; ++i) {
            n = i0 + i + 1;  // token i0 + i stands; the row goes on with its best
            go = best[i];
            if (n == len || go < 0 || p.tokens[(a + n) * p.tok_stride] != go) {
                done = true;
                break;
            }
        }
    }
    if (threadIdx.x == 0) {
        p.accepted[b] = n;
        p.next[b] = go;
    }
}

template <typename PT> hipError_t launch_pt(const DraftParams& p, hipStream_t s) {
    if (p.u) {
        hipLaunchKernelGGL(drafts_sums<PT>, dim3(static_cast<unsigned>(p.B) * p.splits),
                           dim3(kDraftThreads), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(drafts_draw<PT>, dim3(p.B), dim3(kDraftThreads), 0, s, p);
        return hipGetLastError();
    }
    if (p.T > 0) {
        hipLaunchKernelGGL(drafts_best<PT>, dim3(static_cast<unsigned>(p.T) * p.splits),
                           dim3(kDraftThreads), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(drafts_compare, dim3(p.B), dim3(kDraftThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_drafts(const DraftParams& p, hipStream_t s) {
    return p.bf16 ? launch_pt<uint16_t>(p, s) : launch_pt<float>(p, s);
}

}  // namespace gdr

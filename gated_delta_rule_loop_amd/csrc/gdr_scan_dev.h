// Device helpers of the selective scan (gfx950).
#pragma once

#include "gdr_internal.h"
#include "gdr_scan.h"

namespace gdr {

constexpr float kScanLog2e = 1.44269504088896341f;

__device__ __forceinline__ float scan_widen(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ uint16_t scan_round(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));  // to nearest even
}
__device__ __forceinline__ float scan_value(float v) { return v; }
__device__ __forceinline__ float scan_value(uint16_t v) { return scan_widen(v); }
__device__ __forceinline__ void scan_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void scan_put(uint16_t* p, float v) { *p = scan_round(v); }

// n values from p, as float32; p aligned to all of them (16 bytes at most).
template <int n> __device__ __forceinline__ void scan_load(const float* p, float (&v)[n]) {
    if constexpr (n % 4 == 0) {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(p + i);
            v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = p[i];
    }
}
template <int n> __device__ __forceinline__ void scan_load(const uint16_t* p, float (&v)[n]) {
    if constexpr (n % 8 == 0) {
#pragma unroll
        for (int i = 0; i < n; i += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i + 2 * j] = __uint_as_float(u[j] << 16);
                v[i + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
            }
        }
    } else if constexpr (n % 4 == 0) {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + i);
            v[i] = __uint_as_float(w.x << 16); v[i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
            v[i + 2] = __uint_as_float(w.y << 16); v[i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = scan_widen(p[i]);
    }
}
template <int n> __device__ __forceinline__ void scan_store(float* p, const float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int n> __device__ __forceinline__ void scan_store(uint16_t* p, const float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; i += 8) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = scan_round(v[i + 2 * j]) |
                   (static_cast<uint32_t>(scan_round(v[i + 2 * j + 1])) << 16);
        *reinterpret_cast<uint4*>(p + i) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)),
                                                       CTRL, 0xf, 0xf, false));
}
// What a lane and its partner (named by CTRL) hold of x and y, added: x's in the
// lanes where `up` is false, y's in their partners.
template <int CTRL> __device__ __forceinline__ float halve(bool up, float x, float y) {
    return (up ? y : x) + dpp<CTRL>(up ? x : y);
}

// halve() of four pairs at a distance whose lanes are whole banks of four: two additions a
// pair, the second into the banks MASK alone, where halve() takes two selects and one.
// The waits are those between a write of a register and its use by another lane, which
// the compiler does not see to here.  Gradients of 2 x 2048 tokens 355 us, 366 with
// selects; the lane walk 1 to 2 % less.
#define GDR_SCAN_HALVE4(NAME, CTRL, MASK)                                                      \
    __device__ __forceinline__ void NAME(float* x, const float* y) {                           \
        asm("s_nop 1\n\t"                                                                      \
            "v_add_f32_dpp %0, %0, %0 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                 \
            "v_add_f32_dpp %1, %1, %1 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                 \
            "v_add_f32_dpp %2, %2, %2 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                 \
            "v_add_f32_dpp %3, %3, %3 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                 \
            "v_add_f32_dpp %0, %4, %4 " CTRL " row_mask:0xf bank_mask:" MASK "\n\t"            \
            "v_add_f32_dpp %1, %5, %5 " CTRL " row_mask:0xf bank_mask:" MASK "\n\t"            \
            "v_add_f32_dpp %2, %6, %6 " CTRL " row_mask:0xf bank_mask:" MASK "\n\t"            \
            "v_add_f32_dpp %3, %7, %7 " CTRL " row_mask:0xf bank_mask:" MASK "\n\t"            \
            "s_nop 1"                                                                          \
            : "+&v"(x[0]), "+&v"(x[1]), "+&v"(x[2]), "+&v"(x[3])                               \
            : "v"(y[0]), "v"(y[1]), "v"(y[2]), "v"(y[3]));                                     \
    }
GDR_SCAN_HALVE4(halve_by_8, "row_ror:8", "0xc")           // lanes with bit 3 take y's sums
GDR_SCAN_HALVE4(halve_by_4, "row_half_mirror", "0xa")     // bit 2
#undef GDR_SCAN_HALVE4

// Lane l: the sum over its 16 lanes (an aligned row) of x[l % 16].
__device__ __forceinline__ float row_sums16(float (&x)[16]) {
    const int lane = threadIdx.x;
    halve_by_8(x, x + 8);
    halve_by_8(x + 4, x + 12);
    halve_by_4(x, x + 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = halve<0x4E>(lane & 2, x[i], x[i + 2]);
    return halve<0xB1>(lane & 1, x[0], x[1]);
}

// The value `off` bytes behind a wave-uniform base: one 32-bit register a lane.
template <typename WT> __device__ __forceinline__ WT scan_at(const char* base, uint32_t off) {
    return *reinterpret_cast<const WT*>(base + off);
}
template <typename WT>
__device__ __forceinline__ const char* scan_base(const ScanRows& r, int64_t tok) {
    return static_cast<const char*>(r.p) + tok * r.tok * static_cast<int64_t>(sizeof(WT));
}
template <typename WT> __device__ __forceinline__ uint32_t scan_step(const ScanRows& r) {
    return static_cast<uint32_t>(r.tok) * static_cast<uint32_t>(sizeof(WT));
}

// e^x = 2^hi 2^lo: hi, and in lo what x log2(e) loses when it is rounded to hi.
__device__ __forceinline__ float scan_exponent(float x, float& lo) {
    const float hi = x * kScanLog2e;
    lo = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, kScanLog2e, -hi));
    return hi;
}
// e^x to about one float32 rounding (the compensated product: 2^hi (1 + lo ln 2)) for
// finite x up to 88; where 2^hi is infinite the sum would be no number.  Results
// below 2^-126 are 0.
__device__ __forceinline__ float scan_exp(float x) {
    float lo;
    const float e = __builtin_amdgcn_exp2f(scan_exponent(x, lo));
    return __builtin_fmaf(e, lo * 0.693147181f, e);
}
// 1 / (1 + e^-x); of NaN it is a number (callers multiply by x, which is none).  e^-x
// passes float32's largest value from -x = 88.8 on: as a product with a factor near 1,
// which costs a rounding more than the sum, it is infinite there and the sigmoid 0.
__device__ __forceinline__ float scan_sigmoid(float x) {
    float lo;
    const float e = __builtin_amdgcn_exp2f(scan_exponent(__builtin_amdgcn_fmed3f(-x, -150.0f, 128.0f), lo));
    return __builtin_amdgcn_rcpf(1.0f + e * __builtin_fmaf(lo, 0.693147181f, 1.0f));
}
// log(1 + e^x) = max(x, 0) + log(1 + t), t = e^-|x|.  log(1 + t) = 2 atanh(s) with
// s = t / (2 + t) <= 1/3: an odd series in s, its tail after s fitted by a cubic
// in s^2 (off by 1.6e-8 of the result at most), so that small t keep all their bits.
// `slope`: its derivative, the sigmoid.
__device__ __forceinline__ float scan_softplus(float x, float& slope) {
    const float t = scan_exp(__builtin_fmaxf(-__builtin_fabsf(x), -150.0f));
    const float s = t * __builtin_amdgcn_rcpf(2.0f + t), v = s * s;
    float q = __builtin_fmaf(0.134337738f, v, 0.141169786f);
    q = __builtin_fmaf(q, v, 0.200038359f);
    q = __builtin_fmaf(q, v, 0.333333194f);
    const float l = __builtin_fmaf(2.0f * s, v * q, 2.0f * s);
    slope = (x > 0.0f ? 1.0f : t) * __builtin_amdgcn_rcpf(1.0f + t);
    return (x <= 0.0f ? 0.0f : x) + l;  // NaN stays NaN
}
__device__ __forceinline__ float scan_softplus(float x) {
    float slope;
    return scan_softplus(x, slope);
}

// A pointer whose loads at wave-uniform addresses are scalar loads.
#define GDR_UNIFORM __attribute__((address_space(4)))

// An index vector's element at a wave-uniform place.
__device__ __forceinline__ uint32_t scan_index(const uint32_t* v, int64_t i) {
    return *reinterpret_cast<const GDR_UNIFORM uint32_t*>(reinterpret_cast<uint64_t>(v + i));
}

// N values of a [.., N] operand at a wave-uniform place.
template <typename WT, int N>
__device__ __forceinline__ void uniform_row(const void* base, int64_t elem, float (&v)[N]) {
    const uint64_t at = reinterpret_cast<uint64_t>(base) + static_cast<uint64_t>(elem) * sizeof(WT);
    const GDR_UNIFORM uint32_t* q = reinterpret_cast<const GDR_UNIFORM uint32_t*>(at);
    if constexpr (sizeof(WT) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint32_t w = q[i];
            v[2 * i] = __uint_as_float(w << 16);
            v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
}

// B and C of some tokens as they stand in memory, in scalar registers.
template <typename WT, int N, int S, bool TWO> struct ScalarRows {
    static constexpr int R = N * static_cast<int>(sizeof(WT)) / 4;
    uint32_t b[S][R], c[S][TWO ? R : 1];
    __device__ __forceinline__ void load(const char* pb, const char* pc, uint32_t sb, uint32_t sc,
                                         int t, int n) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const uint64_t u = static_cast<uint64_t>(min(t + i, n - 1));
            const GDR_UNIFORM uint32_t* q =
                reinterpret_cast<const GDR_UNIFORM uint32_t*>(reinterpret_cast<uint64_t>(pb) + u * sb);
#pragma unroll
            for (int k = 0; k < R; ++k) b[i][k] = q[k];
            if constexpr (TWO) {
                q = reinterpret_cast<const GDR_UNIFORM uint32_t*>(reinterpret_cast<uint64_t>(pc) + u * sc);
#pragma unroll
                for (int k = 0; k < R; ++k) c[i][k] = q[k];
            }
        }
    }
    // Scalar loads return in any order, so that a wait for one is a wait for all: these
    // have to be there before the next are asked for.
    __device__ __forceinline__ void arrive() {
        asm volatile("" : "+s"(b[S - 1][R - 1]));
        if constexpr (TWO) asm volatile("" : "+s"(c[S - 1][R - 1]));
        __builtin_amdgcn_sched_barrier(0);
    }
    static __device__ __forceinline__ float value(const uint32_t (&r)[R], int i) {
        if constexpr (sizeof(WT) == 4) return __uint_as_float(r[i]);
        return __uint_as_float(i & 1 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
    }
};

// Tokens that B and C are loaded ahead: as many as leave scalar registers beside two
// sets of them.
template <typename WT> constexpr int scan_ahead(int N) {
    return N * static_cast<int>(sizeof(WT)) <= 32 ? 2 : 1;
}

// The number of row b's first part, when rows are cut into parts of `len` tokens:
// rows own disjoint ranges of numbers, with at most one unused at the end of each.
__device__ __forceinline__ int64_t scan_first_part(uint32_t off, int b, int len) {
    return static_cast<int64_t>(off / static_cast<uint32_t>(len)) + b;
}

// The wave's number in a launch of kScanThreads.
__device__ __forceinline__ int scan_wave() {
    return static_cast<int>(blockIdx.x) * (kScanThreads / 64) +
           __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
}

// Segments of a row of n tokens: none up to `skip` tokens, one at least above.  They are
// numbered without gaps: waves that find nothing to do would leave the others
// unevenly spread (32 rows of 512 tokens 353 us, 588 with every second segment
// empty).
__device__ __forceinline__ int scan_segs(int n, int len, int skip) {
    return n <= skip ? 0 : len == 0 || n <= len ? 1 : (n + len - 1) / len;
}

struct ScanSpan {
    int row, s, count;  // the segment's row, its number there, the row's segments
    int t0, n;          // its tokens
};

// Which tokens segment `seg` spans; false past the last one.  The whole wave calls
// it with one `seg`: rows are counted 64 at a time, so that every wave's time grows with
// the number of rows before its own (4096 channels, rows of 4 tokens: 1024 rows 282 us, 4096
// 2.5 ms, 16384 31 ms).
__device__ __forceinline__ bool scan_locate(const ScanParams& p, int seg, ScanSpan& o) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 64) {
        const int b = b0 + lane;
        int a = 0, n = 0, c = 0;
        if (b < p.B) {
            a = static_cast<int>(p.offsets[b]);
            n = static_cast<int>(p.offsets[b + 1]) - a;
            c = scan_segs(n, p.seg_len, p.seg_skip);
        }
        int sum = c;
        for (int d = 1; d < min(64, p.B); d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const uint64_t past = __ballot(before + sum > seg);
        if (past) {
            const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
            auto of = [at](int v) { return __builtin_amdgcn_readlane(v, at); };
            o.row = b0 + at;
            o.count = of(c);
            o.s = seg - (before + of(sum) - o.count);
            const int len = p.seg_len ? p.seg_len : of(n);
            o.t0 = of(a) + o.s * len;
            o.n = o.count > 1 ? min(len, of(n) - o.s * len) : of(n);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, min(64, p.B) - 1);
    }
    return false;
}

// The number of a row's first segment; the whole wave calls it with one row.
__device__ __forceinline__ int scan_first_seg(const ScanParams& p, int row) {
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int b = lane; b < row; b += 64)
        sum += scan_segs(static_cast<int>(p.offsets[b + 1] - p.offsets[b]), p.seg_len, p.seg_skip);
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    return __builtin_amdgcn_readfirstlane(sum);
}

}  // namespace gdr

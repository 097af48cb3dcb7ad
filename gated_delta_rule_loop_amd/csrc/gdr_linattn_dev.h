// Device helpers of the linear-attention kernels (gfx950).
#pragma once

#include "gdr_linattn.h"
#include "gdr_internal.h"

namespace gdr {

typedef float la_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t la_u4 __attribute__((ext_vector_type(4)));
typedef short la_s4 __attribute__((ext_vector_type(4)));
typedef short la_s8 __attribute__((ext_vector_type(8)));
typedef __bf16 la_b4 __attribute__((ext_vector_type(4)));
typedef __bf16 la_b8 __attribute__((ext_vector_type(8)));

constexpr double kLog2e = 1.4426950408889634;
// exp(-700) is zero in float32; the clamp keeps sums of exponents finite, so
// that a decay of exactly zero (g = -inf) never makes inf - inf.
constexpr float kLogDecayMin = -700.0f;

__device__ __forceinline__ float la_widen(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ uint16_t la_round(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ float la_load(const void* p, int64_t i, int bf16) {
    return bf16 ? la_widen(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void la_store(void* p, int64_t i, int bf16, float x) {
    if (bf16) static_cast<uint16_t*>(p)[i] = la_round(x);
    else static_cast<float*>(p)[i] = x;
}
__device__ __forceinline__ float la_clamp_g(float g) { return g < kLogDecayMin ? kLogDecayMin : g; }

// A double from the lane that the DPP control names, 0 where there is none or
// the lane's row is not in ROWS.
template <int CTRL, int ROWS> __device__ __forceinline__ double la_lanes(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(u), CTRL, ROWS, 0xf, false));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double la_lane(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), lane));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32),
                                                                        lane));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Sum over the four lanes that share lane % 16.
__device__ __forceinline__ float la_sum_rows(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t s = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(s, s, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Segments of a row of n tokens (one at least: it carries the row's state); none
// of a row below `from` tokens, which is not walked.
__device__ __forceinline__ int la_row_segs(int n, int seg_len, int from) {
    return n < from ? 0 : n <= seg_len ? 1 : (n + seg_len - 1) / seg_len;
}

struct LaSpan {
    int row, s, count;   // the segment's row, its number there, the row's segments
    int t0, n;           // its tokens
    int first;           // the row's first segment
    int cut;             // ... and among the segments of rows that have several
};

// Which tokens segment `seg` spans; false past the last one.  Each wave scans
// the rows' segment counts, 64 rows at a time.
__device__ __forceinline__ bool la_locate(const uint32_t* off, int B, int seg_len, int from,
                                          int seg, LaSpan& o) {
    if (seg_len == 0) {
        if (seg >= B) return false;
        o.row = seg;
        o.s = 0;
        o.count = 1;
        o.t0 = static_cast<int>(off[seg]);
        o.n = static_cast<int>(off[seg + 1]) - o.t0;
        o.first = seg;
        o.cut = 0;
        return true;
    }
    const int lane = threadIdx.x & 63;
    int base = 0, cut_base = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int b = b0 + lane;
        int a = 0, n = 0, c = 0;
        if (b < B) {
            a = static_cast<int>(off[b]);
            n = static_cast<int>(off[b + 1]) - a;
            c = la_row_segs(n, seg_len, from);
        }
        const int cuts = c > 1 ? c : 0;
        int sum = c, cut_sum = cuts;
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d), cut_up = __shfl_up(cut_sum, d);
            if (lane >= d) {
                sum += up;
                cut_sum += cut_up;
            }
        }
        const uint64_t past = __ballot(base + sum > seg);
        if (past) {
            const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
            auto of = [at](int v) { return __builtin_amdgcn_readlane(v, at); };
            o.row = b0 + at;
            o.count = of(c);
            o.first = base + of(sum) - o.count;
            o.cut = cut_base + of(cut_sum) - of(cuts);
            o.s = seg - o.first;
            const int ra = of(a), rn = of(n);
            o.t0 = ra + o.s * seg_len;
            o.n = min(seg_len, rn - o.s * seg_len);
            if (o.n < 0) o.n = 0;
            return true;
        }
        base += __builtin_amdgcn_readlane(sum, 63);
        cut_base += __builtin_amdgcn_readlane(cut_sum, 63);
    }
    return false;
}

// blockIdx -> logical index such that consecutive logical indices run on one
// of the 8 dies (workgroups are dealt to them in turn) and share its L2.
__device__ __forceinline__ int la_logical(int bid, int total) {
    const int q = total >> 3, r = total & 7, die = bid & 7;
    return die * q + min(die, r) + (bid >> 3);
}

}  // namespace gdr

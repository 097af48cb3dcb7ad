// gfx950 walk kernels of linear attention with a decay for each head, in the
// chunked matrix form.  Compiled once per work type (GDR_WT: float, or
// uint16_t for bf16 bits).
//
// A workgroup of four or eight waves walks one segment of a row for one value
// head and 64 or 128 columns of the state, C tokens (a chunk) at a time:
//     P_ij = exp(G_i - G_j) (x_i . y_j), j <= i         (C x C, per chunk)
//     out  = scale (P Z + diag(exp(G)) X S)
//     S   <- exp(G_C) S + Y^T diag(exp(G_C - G)) Z
// The state stays in registers for the whole segment: each wave owns all Kd
// rows of 16 columns, in the accumulator layout of the matrix
// instructions, which is at once the operand layout of the product X S (the
// order of a contraction is free as long as both operands agree on it), so
// the state is never moved.  X, Y and Z are staged row by row in LDS; the
// operands that run along tokens (Y^T, Z) come from there through the
// transposing LDS read.  The outputs are computed transposed (columns in the
// registers of a lane), so a lane stores four neighbouring columns at once.
// A walk from the last token is the same with the tokens taken in reverse and
// the decays summed exclusively instead of inclusively.
//
// Precision.  Products of bf16 operands are exact in the float32 accumulators.
// What is computed and then multiplied again - P, S, and Z times its decay -
// is split into two bf16 terms (the value's rounding and the rounding of the
// rest, within 2^-16 of the value; three terms, 2^-24, for what goes into a
// float32 state), so outputs carry little more than their own rounding, and the
// sums that the decays' gradient takes over a segment stay small differences of
// accurate terms.  One term would leave 2^-8 there, as much as the rounding of
// the bf16 output itself, and useless decay gradients.  float32 work uses the float32 matrix
// instructions throughout.  Decay exponents are summed in float64 and kept as
// a pair of float32.
//
// Measured, 32 value heads, K = V = 128.  bf16, 32768 tokens in 16 segments: 367 us a
// call (with one term everywhere 317, of 378 then).  By the kernel trace, which slows
// the calls down, the walk takes 304 us on average and 255 at best (544 MB: q, k, v
// once a value head's share through the caches, the outputs), the segments' sums 122
// and 108, the scan 15.  Of the walk's cycles the VALU issues in 53%, the LDS is busy
// in 49%, a third of that in bank conflicts, and the matrix instructions in 30%, at 16
// waves a compute unit.  float32, 8336 tokens: 276 us, the matrix instructions at half
// their rate.  Eight waves of 16 columns instead of four of 32: 408 against 424 us, for
// twice the waves a SIMD.
#include <type_traits>

#include "gdr_linattn_dev.h"

#ifndef GDR_WT
#error "compile with -DGDR_WT=float or -DGDR_WT=uint16_t"
#endif

namespace gdr {
namespace {

// The matrix instructions of a work type.  An operand fragment (Fr) holds 4
// values a lane: index lane % 16, contraction 4 * (lane / 16) + e.
template <typename T> struct Mat;

template <> struct Mat<uint16_t> {
    typedef la_s4 Fr;
    enum { kTerms = 2, kVec = 8, kPad = 0 };  // kVec: elements per 16 bytes
    // Place of (row r0 + r, column c), r0 a multiple of 16, in a tile of rows
    // of S elements (64 at least).  The 16-byte slots of a row are permuted by
    // the row's number, to spread the lanes of a transposing read (16 at a time:
    // 4 rows, 32 bytes each) over the banks.
    static __device__ __forceinline__ int at(int r0, int r, int c, int S) {
        // rows of 64 lie two to a round of the banks: the row's parity tells them apart
        const int h = S == 64 ? ((r >> 1 & 3) << 1 | r >> 3) : ((r & 7) << 1 | (r >> 3 & 1));
        return (r0 + r) * S + (((c >> 3) ^ h) << 3) + (c & 7);
    }
    // D[a][b] += sum over 32: two fragments of 16 on each side
    static __device__ __forceinline__ la_f4 mma(Fr a0, Fr a1, Fr b0, Fr b1, la_f4 c) {
        const la_s8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
        const la_s8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(la_b8, a),
                                                       __builtin_bit_cast(la_b8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ Fr row(const uint16_t* p) {
        return *reinterpret_cast<const la_s4*>(p);
    }
    // v as a sum of terms, largest first.  What a pair's rounding leaves comes
    // from one dot product a value: v - 1 * (its own half) - 0 * (the other).
    template <int N> static __device__ __forceinline__ void split(la_f4 v, Fr (&out)[N]) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        // (-1, 0) and (0, -1), from registers: as an inline constant of this
        // instruction -1.0 stands for the float32 pattern, which is (0, -1)
        uint32_t low = 0x0000BF80u, high = 0xBF800000u;
        asm("" : "+s"(low), "+s"(high));
        const b2 first = __builtin_bit_cast(b2, low), second = __builtin_bit_cast(b2, high);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u2 packed;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const b2 b = {static_cast<__bf16>(v[2 * h]), static_cast<__bf16>(v[2 * h + 1])};
                packed[h] = __builtin_bit_cast(uint32_t, b);
                if (i + 1 < N) {
                    v[2 * h] = __builtin_amdgcn_fdot2_f32_bf16(b, first, v[2 * h], false);
                    v[2 * h + 1] = __builtin_amdgcn_fdot2_f32_bf16(b, second, v[2 * h + 1], false);
                }
            }
            out[i] = __builtin_bit_cast(la_s4, packed);
        }
    }
    // X is only read along its rows, 32 values a time: their order in LDS is that
    // of the state's registers (4 g + e, then 16 + 4 g + e), so that a lane reads
    // them as 16 bytes.  Its slots are permuted to spread 8 lanes of such a read
    // over the banks.
    static __device__ __forceinline__ void put_x(uint16_t* p, int r, int c, int S, la_u4 v) {
        const int q = c >> 3 & 3;
        const int a = r * S + ((((c >> 5) * 4 + (q & 1) * 2) ^ (r & 7)) << 3) + (q >> 1) * 4;
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        *reinterpret_cast<u2*>(p + a) = u2{v[0], v[1]};
        *reinterpret_cast<u2*>(p + (a ^ 8)) = u2{v[2], v[3]};
    }
    static __device__ __forceinline__ int x_place(int lane, int S) {
        const int r = lane & 15;
        return r * S + (((lane >> 4) ^ (r & 7)) << 3);
    }
    static __device__ __forceinline__ void x_pair(const uint16_t* p, int a, int kt, Fr& f0, Fr& f1) {
        const la_s8 v = *reinterpret_cast<const la_s8*>(p + (a ^ (kt * 16)));
        f0 = __builtin_shufflevector(v, v, 0, 1, 2, 3);
        f1 = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    }
    // The same for column c + 16 ct from the place `a` of column c (below 16):
    // only the slot's number changes, by bits that are zero in it.
    static __device__ __forceinline__ int step(int a, int ct) { return a ^ (ct * 16); }
    // A fragment with rows r0 + 4 * (lane / 16) + e, column lane % 16 of a 16 x 16
    // block is read from `a`, the place of its own lane
    static __device__ __forceinline__ int col_place(int lane, int S) {
        return at(0, 4 * (lane >> 4) + ((lane & 15) >> 2), (lane & 3) * 4, S);
    }
    static __device__ __forceinline__ Fr col(const uint16_t* p, int) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) la_s4*)p);
    }
    static __device__ __forceinline__ la_f4 widen(Fr f) {
        la_f4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = la_widen(static_cast<uint16_t>(f[e]));
        return r;
    }
    static __device__ __forceinline__ Fr narrow(la_f4 v) {
        la_b4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = static_cast<__bf16>(v[e]);
        return __builtin_bit_cast(la_s4, b);
    }
};

template <> struct Mat<float> {
    typedef la_f4 Fr;
    enum { kTerms = 1, kVec = 4, kPad = 4 };
    static __device__ __forceinline__ int at(int r0, int r, int c, int S) {
        return (r0 + r) * S + c;
    }
    template <int N> static __device__ __forceinline__ void split(la_f4 v, Fr (&out)[N]) {
        static_assert(N == 1, "float32 operands are exact");
        out[0] = v;
    }
    static __device__ __forceinline__ void put_x(float* p, int r, int c, int S, la_u4 v) {
        *reinterpret_cast<la_u4*>(p + r * S + c) = v;
    }
    static __device__ __forceinline__ int x_place(int lane, int S) {
        return (lane & 15) * S + (lane >> 4) * 4;
    }
    static __device__ __forceinline__ void x_pair(const float* p, int a, int kt, Fr& f0, Fr& f1) {
        f0 = row(p + a + kt * 16);
        f1 = row(p + a + kt * 16 + 16);
    }
    static __device__ __forceinline__ la_f4 mma(Fr a0, Fr a1, Fr b0, Fr b1, la_f4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[e], b0[e], c, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[e], b1[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Fr row(const float* p) {
        return *reinterpret_cast<const la_f4*>(p);
    }
    static __device__ __forceinline__ int step(int a, int ct) { return a + ct * 16; }
    static __device__ __forceinline__ int col_place(int lane, int S) {
        return at(0, 4 * (lane >> 4), lane & 15, S);
    }
    static __device__ __forceinline__ Fr col(const float* p, int S) {
        Fr r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = p[e * S];
        return r;
    }
    static __device__ __forceinline__ la_f4 widen(Fr f) { return f; }
    static __device__ __forceinline__ Fr narrow(la_f4 v) { return v; }
};

// KP: Kd rounded up to the built size (the rest is zeros); W waves of 16
// columns per workgroup; C tokens per chunk.  Modes: the walk; the walk with the sums for the
// decays' gradient; only the segment's own sum of the state.
enum { kWalk = 0, kWalkSums = 1, kSegment = 2 };
template <typename T, int KP, int W, int C, int MODE>
__global__ void __launch_bounds__(64 * W, KP > 128 || W == 4 ? 2 : 4) walk_kernel(const LaParams p, float* __restrict__ tot) {
    typedef Mat<T> M;
    typedef typename M::Fr Fr;
    constexpr bool SEG = MODE == kSegment, SUMS = MODE == kWalkSums;
    constexpr int N = M::kTerms;
    constexpr int VEC = M::kVec, ES = sizeof(T);
    constexpr int XS = KP + M::kPad;      // LDS rows
    constexpr int TH = 64 * W, ZC = 16 * W;
    constexpr int ZS = ZC + M::kPad;
    constexpr int PS = C + VEC;           // one 16-byte slot of padding
    constexpr int IT = C / 16;            // token tiles
    constexpr int KT = KP / 16;           // state row tiles
    constexpr int XV = C * KP / VEC / TH;
    constexpr int ZV = C * ZC / VEC / TH;
    static_assert(XV >= 1 && ZV >= 1, "a chunk fills the workgroup's loads");

    __shared__ __attribute__((aligned(16))) T Xs[SEG ? 8 : C * XS];
    __shared__ __attribute__((aligned(16))) T Ys[C * XS];
    __shared__ __attribute__((aligned(16))) T Zs[C * ZS];
    __shared__ __attribute__((aligned(16))) T Ps[SEG ? 8 : N * C * PS];
    // decay exponents and factors of two chunks: the one at work and the next
    __shared__ __attribute__((aligned(16))) float g_hi[2][C], g_lo[2][C], g_in[2][C], g_out[2][C];
    __shared__ float g_all[2], own[SUMS ? C : 1];

    const int id = la_logical(blockIdx.x, gridDim.x);
    const int tile = id % p.max_tiles;
    const int wi = (id / p.max_tiles) % p.nwalks;
    // segments before heads: those past the last one are spread over the dies
    const int seg = (id / (p.max_tiles * p.nwalks)) % p.segs;
    const int head = id / (p.max_tiles * p.nwalks * p.segs);
    const LaWalk& w = p.w[wi];
    if (tile >= w.tiles) return;
    LaSpan sp;
    if (!la_locate(p.offsets, p.B, p.seg_len, p.walk_from, seg, sp)) return;
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    sp = LaSpan{uniform(sp.row), uniform(sp.s), uniform(sp.count), uniform(sp.t0), uniform(sp.n),
                uniform(sp.first), uniform(sp.cut)};
    const int Kd = w.Kd, Vd = w.Vd, n = sp.n;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = (lane >> 4) * 4, i16 = lane & 15;
    const int zbase = tile * ZC + wave * 16;        // this wave's columns
    const uint32_t slot = p.slot_idx ? p.slot_idx[sp.row] : static_cast<uint32_t>(sp.row);
    const bool third = w.third != 0, out_f32 = w.out_f32 != 0;
    const LaState& in = w.by_cut && sp.count == 1 ? w.in_row : w.in;
    const int state_seg = w.by_cut ? sp.cut + sp.s : seg;
    const bool at_last = w.reverse ? sp.s == 0 : sp.s == sp.count - 1;
    // A segment's sum is taken from its far end: the state needs no decay on the
    // way (the factor of a chunk's tokens takes what was walked), and the walk
    // that follows starts with what was read last.
    const bool reverse = SEG ? !w.reverse : w.reverse != 0;
    if (SEG && at_last) return;           // no segment after it in the walk needs its sum
    const bool sums = SUMS && w.row_sum != nullptr;

    // Walk position r is token start + dir * r.
    const int64_t start = reverse ? int64_t{sp.t0} + n - 1 : sp.t0;
    const int dir = reverse ? -1 : 1;
    if (!SEG && slot == kPadSlot) {       // a padding row: zeros out, no state
        for (int64_t i = tid; i < int64_t{n} * ZC; i += TH) {
            const int z = tile * ZC + static_cast<int>(i % ZC);
            const int64_t at = (sp.t0 + i / ZC) * w.out_tok + head * w.out_head + z;
            if (z < Vd) {
                if (out_f32) static_cast<float*>(w.out)[at] = 0.0f;
                else static_cast<T*>(w.out)[at] = T(0);
            }
        }
        return;
    }

    // ---- a chunk's loads, held in registers until its LDS is free.  A load
    // takes XR (ZR) rows: its first token in memory is a uniform address that
    // moves on by `inc`, a thread's own row and column a 32-bit offset from it.
    // In the last chunk, rows past the end are clamped instead; they, and
    // columns past the head dim, are written to LDS as zeros.
    constexpr int XR = TH / (KP / VEC), ZR = TH / (ZC / VEC);
    // What is derived from the thread's number is computed anew for each chunk
    // (`fresh`): kept over the chunks it takes registers that others would have
    // to be spilled from.
    auto fresh = [](int v) {
        asm volatile("" : "+v"(v));
        return v;
    };
    struct Mine { int xr, xc, zr, zc; };
    auto mine = [](int t) {
        return Mine{t / (KP / VEC), t % (KP / VEC) * VEC, t / (ZC / VEC), t % (ZC / VEC) * VEC};
    };
    struct Stream {
        const char* q;                    // the next load's first token in memory
        int32_t tok;                      // bytes from token to token, below 2^26
    };
    auto stream = [&](const LaTensor& t, int R) {
        return Stream{static_cast<const char*>(t.p) +
                          (head / t.div * t.head + (reverse ? start - (R - 1) : start) * t.tok) * ES,
                      static_cast<int32_t>(t.tok * ES)};
    };
    Stream xs = stream(w.x, XR), ys = stream(w.y, XR), zs = stream(w.z, ZR);
    la_u4 px[SEG ? 1 : XV], py[XV], pz[ZV];
    uint32_t pg = 0;                      // g as it is stored
    // The first token in memory of the R at walk positions r, r + 1, ...
    auto lead = [&](int r, int R) { return reverse ? start - r - (R - 1) : start + r; };
    auto fetch = [&](int c0) {
        const int t = fresh(tid);
        const Mine at = mine(t);
        const int m = n - 1 - c0;         // the last token's place in the chunk
        if (p.g && wave == W - 1) {
            const int64_t i = (start + dir * (c0 + min(t & 63, m))) * p.g_tok + head * p.g_head;
            if (p.g_bf16) pg = static_cast<const uint16_t*>(p.g)[i];
            else pg = static_cast<const uint32_t*>(p.g)[i];
        }
        const uint32_t xcol = at.xc < Kd ? at.xc * ES : 0;
        const uint32_t zcol = tile * ZC + at.zc < Vd ? (tile * ZC + at.zc) * ES : 0;
        if (m >= C - 1) {
            auto load = [&](Stream& s, int R, int r, uint32_t col) {
                const uint32_t row = __umul24(static_cast<uint32_t>(reverse ? R - 1 - r : r),
                                              static_cast<uint32_t>(s.tok >> 4)) << 4;
                const la_u4 v = *reinterpret_cast<const la_u4*>(s.q + (row + col));
                s.q += int64_t{dir * R} * s.tok;
                return v;
            };
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                if constexpr (!SEG) px[i] = load(xs, XR, at.xr, xcol);
                py[i] = load(ys, XR, at.xr, xcol);
            }
#pragma unroll
            for (int i = 0; i < ZV; ++i) pz[i] = load(zs, ZR, at.zr, zcol);
        } else {
            auto load = [&](const Stream& s, int R, int r, uint32_t col) {
                // from the chunk's first load, rows in walk order
                const int64_t row = dir * min(r, m) + (reverse ? R - 1 : 0);
                return *reinterpret_cast<const la_u4*>(s.q + row * s.tok + col);
            };
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                if constexpr (!SEG) px[i] = load(xs, XR, at.xr + i * XR, xcol);
                py[i] = load(ys, XR, at.xr + i * XR, xcol);
            }
#pragma unroll
            for (int i = 0; i < ZV; ++i) pz[i] = load(zs, ZR, at.zr + i * ZR, zcol);
        }
    };
    auto place = [](int r, int c, int stride) { return M::at(r & ~15, r & 15, c, stride); };
    auto stage = [&](int c0) {
        const Mine at_ = mine(fresh(tid));
        const int xr0 = at_.xr, xc = at_.xc, zr0 = at_.zr, zc = at_.zc;
        const bool xok = xc < Kd, zok = tile * ZC + zc < Vd;
        const int m = n - c0;
        if (m >= C && Kd == KP && (tile + 1) * ZC <= Vd) {
#pragma unroll
            for (int i = 0; i < XV; ++i) {
                if constexpr (!SEG) M::put_x(Xs, xr0 + i * XR, xc, XS, px[i]);
                *reinterpret_cast<la_u4*>(&Ys[place(xr0 + i * XR, xc, XS)]) = py[i];
            }
#pragma unroll
            for (int i = 0; i < ZV; ++i)
                *reinterpret_cast<la_u4*>(&Zs[place(zr0 + i * ZR, zc, ZS)]) = pz[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            const int r = xr0 + i * XR;
            const uint32_t keep = xok && r < m ? ~0u : 0u;
            if constexpr (!SEG) M::put_x(Xs, r, xc, XS, px[i] & keep);
            *reinterpret_cast<la_u4*>(&Ys[place(r, xc, XS)]) = py[i] & keep;
        }
#pragma unroll
        for (int i = 0; i < ZV; ++i) {
            const int r = zr0 + i * ZR;
            const uint32_t keep = zok && r < m ? ~0u : 0u;
            *reinterpret_cast<la_u4*>(&Zs[place(r, zc, ZS)]) = pz[i] & keep;
        }
    };
    // The next 16 outputs' first token in memory, at this wave's columns
    const int oes = out_f32 ? 4 : ES;
    const int32_t out_tok = static_cast<int32_t>(w.out_tok);
    char* out = static_cast<char*>(w.out) +
                ((reverse ? start - 15 : start) * w.out_tok + head * w.out_head + zbase) * oes;
    const float scale = p.scale;
    double walked = 0.0;                  // log2 decay of the chunks so far (SEG)
    // A chunk's decay exponents (base 2), by the last wave: a lane per token,
    // summed over rows of 16 lanes and then across them without leaving the
    // registers.
    auto decays = [&](int c0, int b) {
        const int ln = fresh(lane);
        const float g = __uint_as_float(p.g_bf16 ? pg << 16 : pg);
        const double own_g = p.g && ln < C && ln < n - c0
                                 ? static_cast<double>(la_clamp_g(g)) * kLog2e : 0.0;
        double sum = own_g;
        sum += la_lanes<0x111, 0xf>(sum);             // lane - 1 of the row of 16
        sum += la_lanes<0x112, 0xf>(sum);             // lane - 2
        sum += la_lanes<0x114, 0xf>(sum);
        sum += la_lanes<0x118, 0xf>(sum);
        sum += la_lanes<0x142, 0xa>(sum);             // row 0's last to row 1, 2's to 3
        if constexpr (C > 32) sum += la_lanes<0x143, 0xc>(sum);  // row 1's last to rows 2, 3
        const double all = la_lane(sum, C - 1);
        if (reverse) sum -= own_g;
        if (ln < C) {
            const float hi = static_cast<float>(sum);
            g_hi[b][ln] = hi;
            g_lo[b][ln] = static_cast<float>(sum - static_cast<double>(hi));
            g_in[b][ln] = scale * __builtin_amdgcn_exp2f(static_cast<float>(sum));
            g_out[b][ln] =
                __builtin_amdgcn_exp2f(static_cast<float>(SEG ? walked + sum : all - sum));
        }
        if (ln == 0) g_all[b] = __builtin_amdgcn_exp2f(static_cast<float>(all));
        if (SEG) walked += all;
    };

    if (n > 0) fetch(0);

    // ---- the state.  A lane's 4 rows of a tile are neighbours: one vector where
    // the walk's state is stored transposed.  Places are 32-bit offsets from a
    // uniform base; all loads are in flight before the first value is used.
    la_f4 S[KT];
    const bool has_z = zbase + i16 < Vd;
    auto load_as = [&](const LaState& s, auto* p0, la_f4 (&v)[KT]) {
        typedef typename std::remove_const<typename std::remove_pointer<decltype(p0)>::type>::type E;
        const char* base = reinterpret_cast<const char*>(
            p0 + int64_t{s.by_segment ? static_cast<uint32_t>(state_seg) : slot} * s.outer +
            head * s.head);
        const uint32_t off = static_cast<uint32_t>((g4 * s.sk + (zbase + i16) * s.sz) *
                                                   static_cast<int>(sizeof(E)));
        const uint32_t row = static_cast<uint32_t>(s.sk * static_cast<int>(sizeof(E)));
        typedef E E4 __attribute__((ext_vector_type(4)));
        E4 raw[KT];
        if (s.sk == 1) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                raw[kt] = E4{0, 0, 0, 0};
                if (has_z && kt * 16 + g4 < Kd)
                    raw[kt] = *reinterpret_cast<const E4*>(base + kt * 16 * row + off);
            }
        } else {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                raw[kt] = E4{0, 0, 0, 0};
                if (has_z && kt * 16 + g4 < Kd)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        raw[kt][r] = *reinterpret_cast<const E*>(base + (kt * 16 + r) * row + off);
            }
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (sizeof(E) == 2) v[kt][r] = s.mult * la_widen(raw[kt][r]);
                else v[kt][r] = s.mult * raw[kt][r];
            }
    };
    auto load_state = [&](const LaState& s, la_f4 (&v)[KT]) {
        if (s.bf16) load_as(s, static_cast<const uint16_t*>(s.p), v);
        else load_as(s, static_cast<const float*>(s.p), v);
    };
    if (!SEG && in.p) {
        load_state(in, S);
    } else {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = la_f4{0, 0, 0, 0};
    }
    if (n > 0 && wave == W - 1) decays(0, 0);
    for (int c0 = 0, b = 0; c0 < n; c0 += C, b ^= 1) {
        stage(c0);
        __syncthreads();
        const bool more = c0 + C < n;
        const int ln = fresh(lane);
        const int g4 = (ln >> 4) * 4, i16 = ln & 15;
        const int row_x = M::x_place(ln, XS), col_y = M::col_place(ln, XS);
        // a wave's own columns start at a multiple of 16 within a tile's rows
        const int col_z = M::step(M::col_place(ln, ZS), wave);
        // the partner's values at this wave's outputs, before the next chunk's
        // loads: what is loaded in order is waited for in order
        Fr partner[SUMS ? IT : 1];
        if (sums) {
            const int64_t from = lead(c0, C);
            const char* const qp = static_cast<const char*>(w.partner.p) +
                                   (head / w.partner.div * w.partner.head +
                                    from * w.partner.tok) * ES;
            const uint32_t q_tok = static_cast<uint32_t>(w.partner.tok / 4);
            const uint32_t z = static_cast<uint32_t>(min(zbase + g4, Vd - 4)) / 4;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int r = min(it * 16 + i16, n - 1 - c0);
                const uint32_t at = __umul24(reverse ? C - 1 - r : r, q_tok) + z;
                partner[it] = *reinterpret_cast<const Fr*>(qp + at * static_cast<uint32_t>(4 * ES));
            }
        }
        if (more) fetch(c0 + C);
        la_f4 O[SEG ? 1 : IT];
        if constexpr (!SEG) {
            // scale exp(G_i) (S^T X^T): rows are columns of the state, columns tokens
#pragma unroll
            for (int it = 0; it < IT; ++it) O[it] = la_f4{0, 0, 0, 0};
            // Two token tiles at a time, the next two's operands on their way: a
            // wave that waits for each read before its products takes 2 to 3 times
            // as long.
            Fr x[2][2][2];                // [of two steps][tile][half]
            auto read_x = [&](int step) {
                const int kt = step / (IT / 2) * 2, it = step % (IT / 2) * 2;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    M::x_pair(&Xs[(it + j) * 16 * XS], row_x, kt, x[step & 1][j][0],
                              x[step & 1][j][1]);
            };
            constexpr int STEPS = KT / 2 * (IT / 2);
            Fr s0[N], s1[N];
            read_x(0);
#pragma unroll
            for (int step = 0; step < STEPS; ++step) {
                const int kt = step / (IT / 2) * 2, it = step % (IT / 2) * 2;
                if (it == 0) {
                    M::template split<N>(S[kt], s0);
                    M::template split<N>(S[kt + 1], s1);
                }
                if (step + 1 < STEPS) read_x(step + 1);
#pragma unroll
                for (int t = 0; t < N; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        O[it + j] = M::mma(s0[t], s1[t], x[step & 1][j][0], x[step & 1][j][1],
                                           O[it + j]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) O[it] *= g_in[b][it * 16 + i16];
            // scale P by tiles of 16 x 16 on and below the diagonal, dealt to the waves
            for (int t = wave; t < IT * (IT + 1) / 2; t += W) {
                const int it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
                const int jt = t - it * (it + 1) / 2;
                la_f4 acc = {0, 0, 0, 0};
                const int ry = M::at(0, i16, g4, XS) + jt * 16 * XS;
#pragma unroll
                for (int kt = 0; kt < KT; kt += 2) {
                    Fr x0, x1;
                    M::x_pair(&Xs[it * 16 * XS], row_x, kt, x0, x1);
                    acc = M::mma(M::row(&Ys[M::step(ry, kt)]), M::row(&Ys[M::step(ry, kt + 1)]),
                                 x0, x1, acc);
                }
                acc *= scale;
                const int i = it * 16 + i16;
                const float hi = g_hi[b][i], lo = g_lo[b][i];
                const la_f4 hj = *reinterpret_cast<const la_f4*>(&g_hi[b][jt * 16 + g4]);
                const la_f4 lj = *reinterpret_cast<const la_f4*>(&g_lo[b][jt * 16 + g4]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = jt * 16 + g4 + r;
                    const float e = __builtin_amdgcn_exp2f((hi - hj[r]) + (lo - lj[r]));
                    if (SUMS && i == j) own[i] = acc[r];
                    const bool keep = sums ? j < i : j <= i;
                    acc[r] = keep ? acc[r] * e : 0.0f;
                }
                Fr pf[N];
                M::template split<N>(acc, pf);
#pragma unroll
                for (int u = 0; u < N; ++u)
                    *reinterpret_cast<Fr*>(&Ps[(u * C + i) * PS + jt * 16 + g4]) = pf[u];
            }
            if (more && wave == W - 1) decays(c0 + C, b ^ 1);
            __syncthreads();
            if (SUMS) __builtin_amdgcn_sched_barrier(0);
        }
        // Z by columns: operand of P Z as it is, of the state's sum with its decay
        Fr zf[IT];
#pragma unroll
        for (int jt = 0; jt < IT; ++jt) zf[jt] = M::col(&Zs[jt * 16 * ZS + col_z], ZS);
        if constexpr (!SEG) {
            const Fr none = M::narrow(la_f4{0, 0, 0, 0});
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int jt = 0; jt <= it; jt += 2)
#pragma unroll
                    for (int u = 0; u < N; ++u) {
                        const T* pr = &Ps[(u * C + it * 16 + i16) * PS + jt * 16 + g4];
                        const Fr p0 = M::row(pr), p1 = jt + 1 <= it ? M::row(pr + 16) : none;
                        O[it] = M::mma(zf[jt], zf[jt + 1], p0, p1, O[it]);
                    }
            if (sums) {
                // partner . out without the token's own pair, then that pair
                const int row_z = M::step(M::at(0, i16, g4, ZS), wave);
                float* const rs = w.row_sum + (int64_t{tile} * W + wave) * p.nv * p.T +
                                  int64_t{head} * p.T + lead(c0, C);
                const bool has = zbase + g4 < Vd;
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int i = it * 16 + i16;
                    const la_f4 a = M::widen(partner[it]);
                    float sum = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum = fmaf(a[r], O[it][r], sum);
                    sum = la_sum_rows(has ? sum : 0.0f);
                    if (ln < 16 && c0 + i < n) rs[reverse ? C - 1 - i : i] = sum;
                    const float d = own[i];
                    const la_f4 zz = M::widen(M::row(&Zs[it * 16 * ZS + row_z]));
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[it][r] = fmaf(d, zz[r], O[it][r]);
                }
            }
            auto put = [&](auto narrow) {
                typedef decltype(narrow(O[0])) Vec;
                constexpr int OES = sizeof(Vec) / 4;
                const uint32_t at = __umul24(static_cast<uint32_t>(reverse ? 15 - i16 : i16),
                                             static_cast<uint32_t>(out_tok / 4)) * sizeof(Vec) +
                                    g4 * OES;
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    if (c0 + it * 16 + i16 < n && zbase + g4 < Vd)
                        *reinterpret_cast<Vec*>(out + at) = narrow(O[it]);
                    out += int64_t{dir * 16} * (out_tok * OES);
                }
            };
            if (out_f32) put([](la_f4 v) { return v; });
            else put([](la_f4 v) { return M::narrow(v); });
        }
        if (SEG && more && wave == W - 1) decays(c0 + C, b ^ 1);
        // ---- S <- exp(G_C) S + Y^T (decayed Z)
        if constexpr (!SEG) {
            const float all = g_all[b];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) S[kt] *= all;
        }
#pragma unroll
        for (int jt = 0; jt < IT; jt += 2) {
            const la_f4 w0 = *reinterpret_cast<const la_f4*>(&g_out[b][jt * 16 + g4]);
            const la_f4 w1 = *reinterpret_cast<const la_f4*>(&g_out[b][jt * 16 + 16 + g4]);
            Fr z0[N], z1[N];
            M::template split<N>(M::widen(zf[jt]) * w0, z0);
            M::template split<N>(M::widen(zf[jt + 1]) * w1, z1);
            Fr y[2][2][2];                // [of two steps][row tile][half]
            auto read_y = [&](int kt) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        y[kt >> 1 & 1][j][h] = M::col(
                            &Ys[(jt + h) * 16 * XS + M::step(col_y, kt + j)], XS);
            };
            read_y(0);
#pragma unroll
            for (int kt = 0; kt < KT; kt += 2) {
                if (kt + 2 < KT) read_y(kt + 2);
#pragma unroll
                for (int u = 0; u < N; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        S[kt + j] = M::mma(y[kt >> 1 & 1][j][0], y[kt >> 1 & 1][j][1], z0[u],
                                           z1[u], S[kt + j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (N > 1) {
            if (third) {                  // what two terms leave, for a float32 state
#pragma unroll 1
                for (int jt = 0; jt < IT; jt += 2) {
                    const la_f4 w0 = *reinterpret_cast<const la_f4*>(&g_out[b][jt * 16 + g4]);
                    const la_f4 w1 = *reinterpret_cast<const la_f4*>(&g_out[b][jt * 16 + 16 + g4]);
                    Fr z0[3], z1[3];
                    const T* z = &Zs[jt * 16 * ZS + col_z];
                    M::template split<3>(M::widen(M::col(z, ZS)) * w0, z0);
                    M::template split<3>(M::widen(M::col(z + 16 * ZS, ZS)) * w1, z1);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const Fr y0 = M::col(&Ys[jt * 16 * XS + M::step(col_y, kt)], XS);
                        const Fr y1 = M::col(&Ys[(jt + 1) * 16 * XS + M::step(col_y, kt)], XS);
                        S[kt] = M::mma(y0, y1, z0[2], z1[2], S[kt]);
                    }
                }
            }
        }
        __syncthreads();
    }

    // ---- what is left
    auto store_as = [&](const LaState& s, auto* p0) {
        typedef typename std::remove_pointer<decltype(p0)>::type E;
        typedef E E4 __attribute__((ext_vector_type(4)));
        char* base = reinterpret_cast<char*>(p0);
        const uint32_t off = static_cast<uint32_t>((g4 * s.sk + (zbase + i16) * s.sz) *
                                                   static_cast<int>(sizeof(E)));
        const uint32_t row = static_cast<uint32_t>(s.sk * static_cast<int>(sizeof(E)));
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if (!has_z || kt * 16 + g4 >= Kd) continue;
            E4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (sizeof(E) == 2) v[r] = la_round(s.mult * S[kt][r]);
                else v[r] = s.mult * S[kt][r];
            }
            if (s.sk == 1) {
                *reinterpret_cast<E4*>(base + kt * 16 * row + off) = v;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<E*>(base + (kt * 16 + r) * row + off) = v[r];
            }
        }
    };
    auto store_state = [&](const LaState& s, int64_t at) {
        if (s.bf16) store_as(s, static_cast<uint16_t*>(s.p) + at);
        else store_as(s, static_cast<float*>(s.p) + at);
    };
    if (SEG) {
        store_state(w.last, int64_t{seg} * w.last.outer + head * w.last.head);
        if (tid == TH - 1 && tile == 0 && tot)
            tot[(int64_t{w.reverse} * p.segs + seg) * p.nv + head] = static_cast<float>(walked);
        return;
    }
    if (SUMS && w.phi && (!w.phi_rows || at_last)) {
        float sum = 0.0f;
        if (w.phi_in.p) {
            la_f4 back[KT];
            load_state(w.phi_in, back);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = fmaf(S[kt][r], back[kt][r], sum);
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane == 0)
            w.phi[((int64_t{seg} * p.nv + head) * w.tiles + tile) * W + wave] =
                scale * sum;
    }
    // a row without tokens leaves its pool slot alone
    if (w.last.p && at_last && (n > 0 || w.last.p != in.p))
        store_state(w.last, int64_t{slot} * w.last.outer + head * w.last.head);
}

template <int KP, int W, int C, int MODE>
hipError_t run(const LaParams& p, float* tot, hipStream_t s) {
    const int64_t blocks = int64_t{p.segs} * p.nv * p.nwalks * p.max_tiles;
    walk_kernel<GDR_WT, KP, W, C, MODE>
        <<<dim3(static_cast<uint32_t>(blocks)), 64 * W, 0, s>>>(p, tot);
    return hipGetLastError();
}

// The walks of one call that share a built shape, in one launch.
template <int MODE>
hipError_t dispatch(const LaParams& p, float* tot, hipStream_t s) {
    constexpr int C = sizeof(GDR_WT) == 2 ? 64 : 32;
    const int Kd = p.w[0].Kd;
    if (la_waves(p.w[0].Vd) == 4) {
        if (Kd <= 64) return run<64, 4, C, MODE>(p, tot, s);
        if (Kd <= 128) return run<128, 4, C, MODE>(p, tot, s);
        return run<256, 4, 32, MODE>(p, tot, s);
    }
    if (Kd <= 64) return run<64, 8, C, MODE>(p, tot, s);
    // with the decays' sums a chunk of 64 does not fit the registers of four waves
    // a SIMD (gradient of 8192 tokens, 32 heads, K = V = 128: 502 us, 484 by 32)
    if (Kd <= 128) return run<128, 8, MODE == kWalkSums ? 32 : C, MODE>(p, tot, s);
    return run<256, 8, 32, MODE>(p, tot, s);
}

}  // namespace

hipError_t GDR_LA_WALK(const LaParams& p, hipStream_t s) {
    bool sums = false;
    for (int i = 0; i < p.nwalks; ++i) sums = sums || p.w[i].row_sum || p.w[i].phi;
    return sums ? dispatch<kWalkSums>(p, nullptr, s) : dispatch<kWalk>(p, nullptr, s);
}
hipError_t GDR_LA_SEG(const LaParams& p, float* tot, hipStream_t s) {
    return dispatch<kSegment>(p, tot, s);
}

}  // namespace gdr

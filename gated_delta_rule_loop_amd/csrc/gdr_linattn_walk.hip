// gfx950 walk kernels of linear attention with a decay for each head, in the
// chunked matrix form.  Compiled once per work type (GDR_WT: float, or
// uint16_t for bf16 bits).
//
// A workgroup of four waves walks one segment of a row for one value head and
// up to 128 columns of the state, C tokens (a chunk) at a time:
//     P_ij = exp(G_i - G_j) (x_i . y_j), j <= i         (C x C, per chunk)
//     out  = scale (P Z + diag(exp(G)) X S)
//     S   <- exp(G_C) S + Y^T diag(exp(G_C - G)) Z
// The state stays in registers for the whole segment: each wave owns all Kd
// rows of 16 NT columns, in the accumulator layout of the matrix
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
    enum { kTerms = 2, kVec = 8 };    // kVec: elements per 16 bytes
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
    // rows 4 * (lane / 16) + e, column lane % 16 of the 16 x 16 block at p
    static __device__ __forceinline__ Fr col(const uint16_t* p, int stride, int lane) {
        const int g = lane >> 4, i = lane & 15;
        auto* q = (__attribute__((address_space(3))) la_s4*)(p + (4 * g + (i >> 2)) * stride +
                                                             (i & 3) * 4);
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(q);
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
    enum { kTerms = 1, kVec = 4 };
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
    static __device__ __forceinline__ Fr col(const float* p, int stride, int lane) {
        const int g = lane >> 4, i = lane & 15;
        Fr r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = p[(4 * g + e) * stride + i];
        return r;
    }
    static __device__ __forceinline__ la_f4 widen(Fr f) { return f; }
    static __device__ __forceinline__ Fr narrow(la_f4 v) { return v; }
};

// v as a sum of N work-type terms, largest first.
template <typename T, int N>
__device__ __forceinline__ void split(la_f4 v, typename Mat<T>::Fr (&out)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        out[i] = Mat<T>::narrow(v);
        if (i + 1 < N) v = v - Mat<T>::widen(out[i]);
    }
}

// KP: Kd rounded up to the built size (the rest is zeros); 64 * NT columns per
// workgroup; C tokens per chunk.  Modes: the walk; the walk with the sums for the
// decays' gradient; only the segment's own sum of the state.
enum { kWalk = 0, kWalkSums = 1, kSegment = 2 };
template <typename T, int KP, int NT, int C, int MODE>
__global__ void __launch_bounds__(256, 2) walk_kernel(const LaParams p, float* __restrict__ tot) {
    typedef Mat<T> M;
    typedef typename M::Fr Fr;
    constexpr bool SEG = MODE == kSegment, SUMS = MODE == kWalkSums;
    constexpr int N = M::kTerms;
    constexpr int VEC = M::kVec;
    constexpr int XS = KP + VEC;          // LDS row strides: one 16-byte slot of padding
    constexpr int ZC = 64 * NT;
    constexpr int ZS = ZC + VEC;
    constexpr int PS = C + VEC;
    constexpr int IT = C / 16;            // token tiles
    constexpr int KT = KP / 16;           // state row tiles
    constexpr int XV = C * KP / VEC / 256;
    constexpr int ZV = C * ZC / VEC / 256;
    static_assert(XV >= 1 && ZV >= 1, "a chunk fills the workgroup's loads");

    __shared__ __attribute__((aligned(16))) T Xs[SEG ? 8 : C * XS];
    __shared__ __attribute__((aligned(16))) T Ys[C * XS];
    __shared__ __attribute__((aligned(16))) T Zs[C * ZS];
    __shared__ __attribute__((aligned(16))) T Ps[SEG ? 8 : N * C * PS];
    __shared__ __attribute__((aligned(16))) float g_hi[C], g_lo[C], g_in[C], g_out[C], own[C];
    __shared__ float g_all;

    const int id = la_logical(blockIdx.x, gridDim.x);
    const int tile = id % p.max_tiles;
    const int wi = (id / p.max_tiles) % p.nwalks;
    // segments before heads: those past the last one are spread over the dies
    const int seg = (id / (p.max_tiles * p.nwalks)) % p.segs;
    const int head = id / (p.max_tiles * p.nwalks * p.segs);
    const LaWalk& w = p.w[wi];
    if (tile >= w.tiles) return;
    LaSpan sp;
    if (!la_locate(p.offsets, p.B, p.seg_len, seg, sp)) return;
    const int Kd = w.Kd, Vd = w.Vd, n = sp.n;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g4 = (lane >> 4) * 4, i16 = lane & 15;
    const int zbase = tile * ZC + wave * 16 * NT;   // this wave's columns
    const int lz = wave * 16 * NT;                  // the same within the workgroup's
    const uint32_t slot = p.slot_idx ? p.slot_idx[sp.row] : static_cast<uint32_t>(sp.row);
    const bool at_last = w.reverse != 0 ? sp.s == 0 : sp.s == sp.count - 1;
    if (SEG && at_last) return;           // no later segment needs its sum

    const bool third = w.third != 0, reverse = w.reverse != 0, out_f32 = w.out_f32 != 0;
    const bool sums = SUMS && w.row_sum != nullptr;
    char* const out = static_cast<char*>(w.out);
    const int64_t out_tok = w.out_tok, out_head = w.out_head;

    // Walk position r is token start + dir * r.
    const int64_t start = reverse ? int64_t{sp.t0} + n - 1 : sp.t0;
    const int64_t dir = reverse ? -1 : 1;
    if (!SEG && slot == kPadSlot) {       // a padding row: zeros out, no state
        for (int64_t i = tid; i < int64_t{n} * ZC; i += 256) {
            const int z = tile * ZC + static_cast<int>(i % ZC);
            const int64_t at = (sp.t0 + i / ZC) * out_tok + head * out_head + z;
            if (z < Vd) {
                if (out_f32) reinterpret_cast<float*>(out)[at] = 0.0f;
                else reinterpret_cast<T*>(out)[at] = T(0);
            }
        }
        return;
    }

    // ---- the state.  All loads are issued together: indices past the state
    // are clamped into it and their values replaced.
    la_f4 S[KT][NT];
    auto load_as = [&](const LaState& s, auto* base, auto&& use) {
        base += (s.by_segment ? int64_t{seg} : int64_t{slot}) * s.outer + head * s.head;
        int zo[NT];
#pragma unroll
        for (int zt = 0; zt < NT; ++zt) zo[zt] = min(zbase + zt * 16 + i16, Vd - 1) * s.sz;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int zt = 0; zt < NT; ++zt) {
                la_f4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kd = kt * 16 + g4 + r;
                    const auto raw = base[min(kd, Kd - 1) * s.sk + zo[zt]];
                    float f;
                    if constexpr (sizeof(raw) == 2) f = la_widen(raw);
                    else f = raw;
                    v[r] = kd < Kd && zbase + zt * 16 + i16 < Vd ? s.mult * f : 0.0f;
                }
                use(kt, zt, v);
            }
    };
    auto load_state = [&](const LaState& s, auto&& use) {
        if (s.bf16) load_as(s, static_cast<const uint16_t*>(s.p), use);
        else load_as(s, static_cast<const float*>(s.p), use);
    };
    if (!SEG && w.in.p) {
        load_state(w.in, [&](int kt, int zt, la_f4 v) { S[kt][zt] = v; });
    } else {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int zt = 0; zt < NT; ++zt) S[kt][zt] = la_f4{0, 0, 0, 0};
    }

    // ---- a chunk's loads, held in registers until its LDS is free.  They are
    // unconditional too: rows past the end and columns past the head dim are
    // clamped, and written to LDS as zeros.
    constexpr int XR = 256 / (KP / VEC), ZR = 256 / (ZC / VEC);  // rows per load
    const int xr0 = tid / (KP / VEC), xc = tid % (KP / VEC) * VEC;
    const int zr0 = tid / (ZC / VEC), zc = tid % (ZC / VEC) * VEC;
    const bool xok = xc < Kd, zok = tile * ZC + zc < Vd;
    const int64_t xt = dir * w.x.tok, yt = dir * w.y.tok, zt_ = dir * w.z.tok;
    const T* xp = static_cast<const T*>(w.x.p) + (head / w.x.div) * w.x.head + start * w.x.tok +
                  (xok ? xc : 0);
    const T* yp = static_cast<const T*>(w.y.p) + (head / w.y.div) * w.y.head + start * w.y.tok +
                  (xok ? xc : 0);
    const T* zp = static_cast<const T*>(w.z.p) + (head / w.z.div) * w.z.head + start * w.z.tok +
                  (zok ? tile * ZC + zc : 0);
    la_u4 px[SEG ? 1 : XV], py[XV], pz[ZV];
    float pg = 0.0f;
    const int64_t gdir = dir * p.g_tok;
    const char* gp = static_cast<const char*>(p.g) +
                     (start * p.g_tok + head * p.g_head) * (p.g_bf16 ? 2 : 4);
    auto fetch = [&](int c0) {
        const int m = n - 1 - c0;         // the last token's place in the chunk
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            const int r = c0 + min(xr0 + i * XR, m);
            if constexpr (!SEG) px[i] = *reinterpret_cast<const la_u4*>(xp + r * xt);
            py[i] = *reinterpret_cast<const la_u4*>(yp + r * yt);
        }
#pragma unroll
        for (int i = 0; i < ZV; ++i)
            pz[i] = *reinterpret_cast<const la_u4*>(zp + (c0 + min(zr0 + i * ZR, m)) * zt_);
        if (p.g && wave == 0) {
            const int64_t at = (c0 + min(lane, m)) * gdir;
            pg = p.g_bf16 ? la_widen(reinterpret_cast<const uint16_t*>(gp)[at])
                          : reinterpret_cast<const float*>(gp)[at];
        }
    };
    double walked = 0.0;                  // log2 decay of the chunks before (SEG)
    auto stage = [&](int c0) {
        const int m = n - c0;
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            const int r = xr0 + i * XR;
            const uint32_t keep = xok && r < m ? ~0u : 0u;
            if constexpr (!SEG) *reinterpret_cast<la_u4*>(&Xs[r * XS + xc]) = px[i] & keep;
            *reinterpret_cast<la_u4*>(&Ys[r * XS + xc]) = py[i] & keep;
        }
#pragma unroll
        for (int i = 0; i < ZV; ++i) {
            const int r = zr0 + i * ZR;
            const uint32_t keep = zok && r < m ? ~0u : 0u;
            *reinterpret_cast<la_u4*>(&Zs[r * ZS + zc]) = pz[i] & keep;
        }
        if (wave == 0) {                  // the chunk's decay exponents, base 2
            const double own_g = lane < C && lane < m ? static_cast<double>(la_clamp_g(pg)) * kLog2e
                                                      : 0.0;
            double sum = own_g;
#pragma unroll
            for (int d = 1; d < C; d <<= 1) {
                const double up = __shfl_up(sum, d);
                if (lane >= d) sum += up;
            }
            const double all = __shfl(sum, C - 1);
            if (reverse) sum -= own_g;
            if (lane < C) {
                const float hi = static_cast<float>(sum);
                g_hi[lane] = hi;
                g_lo[lane] = static_cast<float>(sum - static_cast<double>(hi));
                g_in[lane] = exp2f(static_cast<float>(sum));
                g_out[lane] = exp2f(static_cast<float>(all - sum));
            }
            if (lane == 0) g_all = exp2f(static_cast<float>(all));
            if (SEG) walked += all;
        }
    };

    const float scale = p.scale;
    if (n > 0) fetch(0);
    for (int c0 = 0; c0 < n; c0 += C) {
        stage(c0);
        __syncthreads();
        if (c0 + C < n) fetch(c0 + C);
        la_f4 O[SEG ? 1 : IT][NT];
        if constexpr (!SEG) {
            // exp(G_i) (S^T X^T): rows are columns of the state, columns tokens
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int zt = 0; zt < NT; ++zt) O[it][zt] = la_f4{0, 0, 0, 0};
#pragma unroll
            for (int kt = 0; kt < KT; kt += 2) {
                Fr s0[NT][N], s1[NT][N];
#pragma unroll
                for (int zt = 0; zt < NT; ++zt) {
                    split<T, N>(S[kt][zt], s0[zt]);
                    split<T, N>(S[kt + 1][zt], s1[zt]);
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const T* xr = &Xs[(it * 16 + i16) * XS + kt * 16 + g4];
                    const Fr x0 = M::row(xr), x1 = M::row(xr + 16);
#pragma unroll
                    for (int zt = 0; zt < NT; ++zt)
#pragma unroll
                        for (int t = 0; t < N; ++t)
                            O[it][zt] = M::mma(s0[zt][t], s1[zt][t], x0, x1, O[it][zt]);
                }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const float wgt = g_in[it * 16 + i16];
#pragma unroll
                for (int zt = 0; zt < NT; ++zt) O[it][zt] *= wgt;
            }
            // P by tiles of 16 x 16 on and below the diagonal, dealt to the waves
            for (int t = wave; t < IT * (IT + 1) / 2; t += kLaWaves) {
                const int it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
                const int jt = t - it * (it + 1) / 2;
                la_f4 acc = {0, 0, 0, 0};
                const T* xr = &Xs[(it * 16 + i16) * XS + g4];
                const T* yr = &Ys[(jt * 16 + i16) * XS + g4];
#pragma unroll
                for (int kt = 0; kt < KT; kt += 2)
                    acc = M::mma(M::row(yr + kt * 16), M::row(yr + kt * 16 + 16),
                                 M::row(xr + kt * 16), M::row(xr + kt * 16 + 16), acc);
                const int i = it * 16 + i16;
                const float hi = g_hi[i], lo = g_lo[i];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = jt * 16 + g4 + r;
                    const float e = exp2f((hi - g_hi[j]) + (lo - g_lo[j]));
                    if (SUMS && i == j) own[i] = acc[r];
                    const bool keep = sums ? j < i : j <= i;
                    acc[r] = keep ? acc[r] * e : 0.0f;
                }
                Fr pf[N];
                split<T, N>(acc, pf);
#pragma unroll
                for (int u = 0; u < N; ++u)
                    *reinterpret_cast<Fr*>(&Ps[(u * C + i) * PS + jt * 16 + g4]) = pf[u];
            }
            __syncthreads();
        }
        // Z by columns: operand of P Z as it is, of the state's sum with its decay
        Fr zf[IT][NT];
#pragma unroll
        for (int jt = 0; jt < IT; ++jt)
#pragma unroll
            for (int zt = 0; zt < NT; ++zt)
                zf[jt][zt] = M::col(&Zs[jt * 16 * ZS + lz + zt * 16], ZS, lane);
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
#pragma unroll
                        for (int zt = 0; zt < NT; ++zt)
                            O[it][zt] = M::mma(zf[jt][zt], zf[jt + 1][zt], p0, p1, O[it][zt]);
                    }
            if (sums) {
                // partner . out without the token's own pair, then that pair
                const int64_t qt = dir * w.partner.tok;
                const T* qp = static_cast<const T*>(w.partner.p) +
                              (head / w.partner.div) * w.partner.head + start * w.partner.tok;
                float* rs = w.row_sum + (int64_t{tile} * kLaWaves + wave) * p.nv * p.T +
                            int64_t{head} * p.T;
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int i = it * 16 + i16;
                    float sum = 0.0f;
#pragma unroll
                    for (int zt = 0; zt < NT; ++zt) {
                        const int z = zbase + zt * 16 + g4;
                        const T* q = qp + min(c0 + i, n - 1) * qt + min(z, Vd - 4);
                        const la_f4 a = M::widen(*reinterpret_cast<const Fr*>(q));
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            sum = z < Vd ? fmaf(a[r], O[it][zt][r], sum) : sum;
                    }
                    sum += __shfl_xor(sum, 16);
                    sum += __shfl_xor(sum, 32);
                    if (lane < 16 && c0 + i < n) rs[start + dir * (c0 + i)] = sum;
                    const float d = own[i];
#pragma unroll
                    for (int zt = 0; zt < NT; ++zt) {
                        const la_f4 z = M::widen(M::row(&Zs[i * ZS + lz + zt * 16 + g4]));
#pragma unroll
                        for (int r = 0; r < 4; ++r) O[it][zt][r] = fmaf(d, z[r], O[it][zt][r]);
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = it * 16 + i16;
                if (c0 + i < n) {
                    const int64_t at = (start + dir * (c0 + i)) * out_tok + head * out_head;
#pragma unroll
                    for (int zt = 0; zt < NT; ++zt) {
                        const int z = zbase + zt * 16 + g4;
                        if (z < Vd) {
                            const la_f4 o = O[it][zt] * scale;
                            if (out_f32)
                                *reinterpret_cast<la_f4*>(reinterpret_cast<float*>(out) + at + z) = o;
                            else
                                *reinterpret_cast<Fr*>(reinterpret_cast<T*>(out) + at + z) =
                                    M::narrow(o);
                        }
                    }
                }
            }
        }
        // ---- S <- exp(G_C) S + Y^T (decayed Z)
        const float all = g_all;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int zt = 0; zt < NT; ++zt) S[kt][zt] *= all;
#pragma unroll
        for (int jt = 0; jt < IT; jt += 2) {
            const la_f4 w0 = *reinterpret_cast<const la_f4*>(&g_out[jt * 16 + g4]);
            const la_f4 w1 = *reinterpret_cast<const la_f4*>(&g_out[jt * 16 + 16 + g4]);
            constexpr int NW = N == 1 ? 1 : 3;
            Fr z0[NT][NW], z1[NT][NW];
#pragma unroll
            for (int zt = 0; zt < NT; ++zt) {
                split<T, NW>(M::widen(zf[jt][zt]) * w0, z0[zt]);
                split<T, NW>(M::widen(zf[jt + 1][zt]) * w1, z1[zt]);
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Fr y0 = M::col(&Ys[jt * 16 * XS + kt * 16], XS, lane);
                const Fr y1 = M::col(&Ys[(jt + 1) * 16 * XS + kt * 16], XS, lane);
#pragma unroll
                for (int zt = 0; zt < NT; ++zt) {
#pragma unroll
                    for (int u = 0; u < N; ++u)
                        S[kt][zt] = M::mma(y0, y1, z0[zt][u], z1[zt][u], S[kt][zt]);
                    if constexpr (NW == 3)
                        if (third)
                            S[kt][zt] = M::mma(y0, y1, z0[zt][2], z1[zt][2], S[kt][zt]);
                }
            }
        }
        __syncthreads();
    }

    // ---- what is left
    auto store_as = [&](const LaState& s, auto* base) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int zt = 0; zt < NT; ++zt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kd = kt * 16 + g4 + r, z = zbase + zt * 16 + i16;
                    if (kd < Kd && z < Vd) {
                        const float v = s.mult * S[kt][zt][r];
                        if constexpr (sizeof(*base) == 2) base[kd * s.sk + z * s.sz] = la_round(v);
                        else base[kd * s.sk + z * s.sz] = v;
                    }
                }
    };
    auto store_state = [&](const LaState& s, int64_t at) {
        if (s.bf16) store_as(s, static_cast<uint16_t*>(s.p) + at);
        else store_as(s, static_cast<float*>(s.p) + at);
    };
    if (SEG) {
        store_state(w.last, int64_t{seg} * w.last.outer + head * w.last.head);
        if (tid == 0 && tile == 0 && tot)
            tot[(int64_t{reverse} * p.segs + seg) * p.nv + head] = static_cast<float>(walked);
        return;
    }
    if (SUMS && w.phi) {
        float sum = 0.0f;
        if (w.phi_in.p)
            load_state(w.phi_in, [&](int kt, int zt, la_f4 v) {
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = fmaf(S[kt][zt][r], v[r], sum);
            });
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane == 0)
            w.phi[(int64_t{seg} * p.nv + head) * w.tiles * kLaWaves + tile * kLaWaves + wave] = sum;
    }
    // a row without tokens leaves its pool slot alone
    if (w.last.p && at_last && (n > 0 || w.last.p != w.in.p))
        store_state(w.last, int64_t{slot} * w.last.outer + head * w.last.head);
}

template <int KP, int NT, int C, int MODE>
hipError_t run(const LaParams& p, float* tot, hipStream_t s) {
    const int64_t blocks = int64_t{p.segs} * p.nv * p.nwalks * p.max_tiles;
    walk_kernel<GDR_WT, KP, NT, C, MODE><<<dim3(static_cast<uint32_t>(blocks)), 256, 0, s>>>(p, tot);
    return hipGetLastError();
}

// The walks of one call that share a built shape, in one launch.
template <int MODE>
hipError_t dispatch(const LaParams& p, float* tot, hipStream_t s) {
    const int Kd = p.w[0].Kd, cols = la_columns(Kd, p.w[0].Vd);
    constexpr bool b16 = sizeof(GDR_WT) == 2;
    constexpr int C = b16 ? 64 : 32;
    if (Kd <= 64)
        return cols == 64 ? run<64, 1, C, MODE>(p, tot, s) : run<64, 2, C, MODE>(p, tot, s);
    if (Kd <= 128)
        return cols == 64 ? run<128, 1, C, MODE>(p, tot, s) : run<128, 2, C, MODE>(p, tot, s);
    return run<256, 1, 32, MODE>(p, tot, s);
}

}  // namespace

hipError_t GDR_LA_WALK(const LaParams& p, hipStream_t s) {
    bool sums = false;
    for (int i = 0; i < p.nwalks; ++i) sums = sums || p.w[i].row_sum != nullptr;
    return sums ? dispatch<kWalkSums>(p, nullptr, s) : dispatch<kWalk>(p, nullptr, s);
}
hipError_t GDR_LA_SEG(const LaParams& p, float* tot, hipStream_t s) {
    return dispatch<kSegment>(p, tot, s);
}

}  // namespace gdr

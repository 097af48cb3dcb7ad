// gfx950 kernels of the selective scan's gradient.  With dy = dout silu(z):
//     lam_t = dy_t C_t + a_{t+1} lam_{t+1}      w_t = lam_t a_t h_{t-1}
//     dx = skip dy + delta sum_n lam B          ddelta = x sum_n lam B + sum_n A w
//     dA = sum_t delta w     dB = sum_d lam delta x     dC = sum_d dy h
//     dz = dout y silu'(z)   ddt = ddelta softplus'     dskip = sum dy x
// The states h run forward and lam backward, and neither is kept by the forward.
// Rows are cut into segments and segments into parts of kPart tokens:
//   1. every segment walks forward from a zero state and leaves its state before
//      each part, its end state, the sums of its step sizes, and what its tokens'
//      dy C hand to its past (decayed from where each stands: a running product);
//   2. both chains over a row's segments give the state that each starts from and
//      the gradient that reaches its end;
//   3. every segment goes through its parts from the last, one state n at a time:
//      16 tokens' decays and states forward into registers (the part's local
//      state plus what is left of the segment's start), then backward.  A lane
//      owns a channel; dB and dC, sums over channels, are reduced over the wave by
//      halving: 32 values in 64 lanes take about 75 slots, not 6 each;
//   4. the parts of dB, dC (over channels), dA, dskip and dt_bias's gradient (over
//      segments) are added in a fixed order.
// Everything is float32; sums over segments are float64.  Bound by the vector
// units: a part takes about 310 slots a channel and state and 1900 a channel, the
// first launch about 150 a token and channel of 16 states.  2 x 2048 bf16 tokens of
// 4096 gated channels of 16 states: 355 us, of which the slots take 250.
#include <type_traits>

#include "gdr_scan_dev.h"

namespace gdr {
namespace {

constexpr int kPart = kScanPart;
// Waves of a gradient's workgroup: what it holds of every state takes 1156 bytes of LDS a
// wave and state (four floats a lane and 33 sums), 73984 a workgroup of 16 states or more, so
// that two workgroups fit a compute unit.
constexpr int grad_waves(int N) { return N > 32 ? 1 : N > 16 ? 2 : 4; }
// States that one wave of the first launch carries.
constexpr int sum_states(int N) { return N < 16 ? N : 16; }

// The number of a segment's first part (segments are whole parts but for a row's last).
__device__ __forceinline__ int64_t first_part(const ScanParams& p, const ScanSpan& o) {
    return scan_first_part(scan_index(p.offsets, o.row), o.row, kPart) + static_cast<int64_t>(o.s) * (p.seg_len / kPart);
}

// ------------------------------------------------------------ 1: own sums ---

// B and C of a segment's parts as float32 [n][token], so that the walk reads a state's
// tokens with scalar loads; zeros past the row's end.
template <typename WT>
__device__ __forceinline__ void turn_parts(const ScanParams& p, const ScanGrad& q,
                                           const ScanSpan& o, int g) {
    const int64_t first = first_part(p, o);
    for (int part = 0; part * kPart < o.n; ++part) {
        const int m = o.n - part * kPart;
        float* to = q.turned + ((first + part) * p.G + g) * 2 * p.N * kPart;
        for (int i = threadIdx.x & 63; i < 2 * p.N * kPart; i += 64) {
            const int n = i % p.N, v = i / p.N, t = v % kPart;  // v: B's tokens, then C's
            const ScanHeads& from = v < kPart ? p.b : p.c;
            float x = 0.0f;
            if (t < m)
                x = scan_value(static_cast<const WT*>(
                    from.p)[(static_cast<int64_t>(o.t0) + part * kPart + t) * from.tok +
                            g * from.grp + n]);
            to[(v / kPart * p.N + n) * kPart + t] = x;
        }
    }
}

// N: the states of this wave, of the channels' p.N.
template <typename WT, int N>
__global__ void __launch_bounds__(kScanThreads, 3) grad_sums(const ScanParams p, const ScanGrad q) {
    const int ctiles = p.G * p.tiles, nblocks = p.N / N, wave = scan_wave();
    const int block = wave / ctiles, tile = wave - block * ctiles;
    const int seg = block / nblocks, n0 = (block - seg * nblocks) * N;
    ScanSpan o;
    if (seg >= p.segs) {  // the last waves turn B and C
        const int job = wave - p.segs * nblocks * ctiles;
        if (job < p.segs * p.G && scan_locate(p, job / p.G, o))
            turn_parts<WT>(p, q, o, job % p.G);
        return;
    }
    if (!scan_locate(p, seg, o)) return;
    const bool ends = o.s < o.count - 1, rev = o.s > 0;
    if (o.n <= kPart && !ends && !rev) return;
    const int g = tile / p.tiles;
    const int cg = (tile - g * p.tiles) * 64 + static_cast<int>(threadIdx.x & 63);
    const bool live = cg < p.gd;
    const int d = g * p.gd + min(cg, p.gd - 1);
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    float h[N], a2[N], P[N], R[N];
    scan_load<N>(p.A + static_cast<int64_t>(d) * p.N + n0, a2);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a2[i] *= kScanLog2e;
        h[i] = 0.0f;
        P[i] = 1.0f;
        R[i] = 0.0f;
    }
    const float bias = p.bias ? p.bias[d] : 0.0f;
    const bool gated = p.z.p != nullptr;
    const ScanRows zrow = gated ? p.z : q.d_o;
    const uint32_t at = static_cast<uint32_t>(d) * sizeof(WT);
    const uint32_t sx = scan_step<WT>(p.x), sd = scan_step<WT>(p.dt), so = scan_step<WT>(q.d_o),
                   sz = scan_step<WT>(zrow);
    const char* pb = static_cast<const char*>(p.b.p) +
                     (o.t0 * p.b.tok + g * p.b.grp + n0) * static_cast<int64_t>(sizeof(WT));
    const char* pc = static_cast<const char*>(p.c.p) +
                     (o.t0 * p.c.tok + g * p.c.grp + n0) * static_cast<int64_t>(sizeof(WT));
    const uint32_t sb = static_cast<uint32_t>(p.b.tok) * sizeof(WT);
    const uint32_t sc = static_cast<uint32_t>(p.c.tok) * sizeof(WT);
    float* check = q.check + first_part(p, o) * (DN + p.D) + d;
    float total = 0.0f;
    constexpr int U = 4;
    WT xs[U], ds[U], os[U], zs[U];
    auto fetch = [&](int t) {
        const char *bx = scan_base<WT>(p.x, o.t0 + t), *bd = scan_base<WT>(p.dt, o.t0 + t);
        const char *bo = scan_base<WT>(q.d_o, o.t0 + t), *bz = scan_base<WT>(zrow, o.t0 + t);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t k = min(i, o.n - 1 - t);
            xs[i] = scan_at<WT>(bx, at + k * sx);
            ds[i] = scan_at<WT>(bd, at + k * sd);
            if (rev) {
                os[i] = scan_at<WT>(bo, at + k * so);
                zs[i] = scan_at<WT>(bz, at + k * sz);
            }
        }
    };
    constexpr int S = scan_ahead<WT>(N);
    typedef ScalarRows<WT, N, S, true> Rows;
    auto token = [&](const Rows& r, int i, WT xr, WT dr, WT gr, WT zr, auto back) {
        float delta = scan_value(dr) + bias;
        if (p.softplus) delta = scan_softplus(delta);
        const float u = delta * scan_value(xr);
        total += delta;
        if constexpr (decltype(back)::value) {
            float dy = scan_value(gr);
            if (gated) {
                const float zv = scan_value(zr);
                dy *= zv * scan_sigmoid(zv);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float a = __builtin_amdgcn_exp2f(delta * a2[k]);
                h[k] = __builtin_fmaf(a, h[k], u * Rows::value(r.b[i], k));
                P[k] *= a;
                R[k] = __builtin_fmaf(P[k], dy * Rows::value(r.c[i], k), R[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[k]), h[k],
                                      u * Rows::value(r.b[i], k));
        }
    };
    Rows rows[2];
    auto step = [&](int t, auto full, auto back) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        WT xc[U], dc[U], oc[U], zc[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            xc[i] = xs[i];
            dc[i] = ds[i];
            oc[i] = os[i];
            zc[i] = zs[i];
        }
        if (t + U < o.n) fetch(t + U);
        if (t % kPart == 0 && t && live) {  // the state before part t / kPart
            float* to = check + (t / kPart) * (DN + p.D);
#pragma unroll
            for (int i = 0; i < N; ++i) to[static_cast<int64_t>(n0 + i) * p.D] = h[i];
            if (n0 == 0) to[DN] = total;
        }
#pragma unroll
        for (int i = 0; i < U; i += S) {
            Rows &now = rows[(i / S) & 1], &next = rows[(i / S + 1) & 1];
            now.arrive();
            next.load(pb, pc, sb, sc, t + i + S, o.n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (FULL || t + i + j < o.n)
                    token(now, j, xc[i + j], dc[i + j], oc[i + j], zc[i + j], back);
        }
    };
    auto walk = [&](auto back) __attribute__((always_inline)) {
        fetch(0);
        rows[0].load(pb, pc, sb, sc, 0, o.n);
        int t = 0;
        for (; t + U <= o.n; t += U) step(t, std::true_type(), back);
        if (t < o.n) step(t, std::false_type(), back);
    };
    if (rev) walk(std::true_type());
    else walk(std::false_type());
    if (!live) return;
    const int64_t mine = static_cast<int64_t>(seg) * DN + static_cast<int64_t>(n0) * p.D + d;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (ends) p.seg_state[mine + static_cast<int64_t>(k) * p.D] = h[k];
        if (rev) q.seg_rev[mine + static_cast<int64_t>(k) * p.D] = R[k];
    }
    // Without cut rows the workspace has no place for it.
    if (n0 == 0 && (ends || rev)) p.seg_delta[static_cast<int64_t>(seg) * p.D + d] = total;
}

// --------------------------------------------------------------- 2: chains ---

__device__ __forceinline__ float state_at(const ScanState& s, int64_t outer, int64_t i) {
    if (!s.p) return 0.0f;
    const int64_t j = outer * s.outer + i;
    return s.bf16 ? scan_widen(static_cast<const uint16_t*>(s.p)[j])
                  : static_cast<const float*>(s.p)[j];
}

template <int N>
__device__ __forceinline__ void state_row(const ScanState& s, int64_t outer, int64_t i,
                                          float (&v)[N]) {
    const int64_t j = outer * s.outer + i;
    if (!s.p) {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = 0.0f;
    } else if (s.bf16) {
        scan_load<N>(static_cast<const uint16_t*>(s.p) + j, v);
    } else {
        scan_load<N>(static_cast<const float*>(s.p) + j, v);
    }
}

__global__ void __launch_bounds__(256) grad_chains(const ScanParams p, const ScanGrad q) {
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const int blocks = static_cast<int>((DN + 255) / 256);
    const int job = blockIdx.x / blocks, row = job >> 1;
    const bool back = job & 1;
    const int64_t i = static_cast<int64_t>(blockIdx.x - job * blocks) * 256 + threadIdx.x;
    const int n = static_cast<int>(p.offsets[row + 1] - p.offsets[row]);
    if (n <= p.seg_len) return;
    const int64_t first = scan_first_seg(p, row);
    if (i >= DN) return;
    const int count = (n + p.seg_len - 1) / p.seg_len;
    const int k = static_cast<int>(i / p.D), d = static_cast<int>(i - static_cast<int64_t>(k) * p.D);
    const int64_t in_slot = static_cast<int64_t>(d) * p.N + k;
    const float a2 = p.A[in_slot] * kScanLog2e;
    float v = state_at(back ? q.dfinal : p.in, row, in_slot);
    float* st = (back ? q.seg_rev : p.seg_state) + first * DN + i;
    const float* dl = p.seg_delta + first * p.D + d;
    constexpr int U = 8;
    for (int j0 = 0; j0 < count; j0 += U) {
        float e[U], s[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j0 + j < count - 1) {
                const int64_t at = back ? count - 1 - (j0 + j) : j0 + j;
                e[j] = st[at * DN];
                s[j] = dl[at * p.D];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j0 + j < count) {
                const int64_t at = back ? count - 1 - (j0 + j) : j0 + j;
                st[at * DN] = v;
                if (j0 + j < count - 1)
                    v = __builtin_fmaf(__builtin_amdgcn_exp2f(a2 * s[j]), v, e[j]);
            }
    }
}

// ------------------------------------------------------------- 3: gradients ---

// Sums over the wave of x[0..15] and y[0..15]: lane l gets that of x[l % 16] below 32
// and of y[l % 16] from there on.
__device__ __forceinline__ float sums32(float (&x)[16], float (&y)[16]) {
    const uint32_t rx = __float_as_uint(row_sums16(x)), ry = __float_as_uint(row_sums16(y));
    const auto s = __builtin_amdgcn_permlane32_swap(rx, ry, false, false);
    const float r = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(r), __float_as_uint(r), false,
                                                    false);
    return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

// A part's raw operands, all loaded before the first is used; past the row's end
// its last token again.
template <typename WT, bool FULL> struct PartRows {
    WT v[kPart];
    __device__ __forceinline__ void load(const ScanRows& r, int64_t t0, int m, uint32_t off) {
        const char* base = scan_base<WT>(r, t0);
        const uint32_t step = scan_step<WT>(r);
        asm volatile("" : "+v"(off));  // the same for every part: not kept in registers
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            v[i] = scan_at<WT>(base, off);
            off += FULL || i + 1 < m ? step : 0;
        }
    }
};
template <typename WT, bool FULL>
__device__ __forceinline__ void part_store(const ScanRows& r, int64_t t0, int m, uint32_t off,
                                           const float (&v)[kPart]) {
    char* base = const_cast<char*>(scan_base<WT>(r, t0));
    const uint32_t step = scan_step<WT>(r);
    asm volatile("" : "+v"(off));
#pragma unroll
    for (int i = 0; i < kPart; ++i) {
        if (FULL || i < m) scan_put(reinterpret_cast<WT*>(base + off), v[i]);
        off += step;
    }
}

template <typename WT, int N, bool GATED>
__global__ void __launch_bounds__(64 * grad_waves(N), N > 16 ? 1 : 2)
grad_walk(const ScanParams p, const ScanGrad q) {
    constexpr int kGradWaves = grad_waves(N), kGradThreads = 64 * kGradWaves;
    // a lane's own: what comes from behind, A, dA so far, the state before the part
    __shared__ float carry[kGradWaves][N][64], as[kGradWaves][N][64], da[kGradWaves][N][64];
    __shared__ float hs[kGradWaves][N][64];
    __shared__ float red[kGradWaves][N][2 * kPart + 1];
    const int gtiles = q.tiles, ctiles = p.G * gtiles;
    const int seg = blockIdx.x / ctiles, tile = blockIdx.x - seg * ctiles;
    const int g = tile / gtiles, gt = tile - g * gtiles;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int cg = gt * kGradThreads + tid;
    const bool live = cg < p.gd;
    const int d = g * p.gd + min(cg, p.gd - 1);
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const int64_t mine = static_cast<int64_t>(seg) * DN + d;
    float* part_a = q.part_a + mine;
    float* part_d = q.part_d + static_cast<int64_t>(seg) * 2 * p.D + d;
    ScanSpan o;
    if (!scan_locate(p, seg, o)) {
        if (live) {
            for (int n = 0; n < N; ++n) part_a[static_cast<int64_t>(n) * p.D] = 0.0f;
            part_d[0] = 0.0f;
            part_d[p.D] = 0.0f;
        }
        return;
    }
    const bool cut = o.count > 1;
    {
        float v[N], a[N];
        scan_load<N>(p.A + static_cast<int64_t>(d) * N, a);
        if (cut) {
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = q.seg_rev[mine + static_cast<int64_t>(n) * p.D];
        } else {
            state_row<N>(q.dfinal, o.row, static_cast<int64_t>(d) * N, v);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            carry[wave][n][lane] = v[n];
            as[wave][n][lane] = a[n];
            da[wave][n][lane] = 0.0f;
        }
    }
    const float bias = p.bias ? p.bias[d] : 0.0f;
    const float skip = p.skip ? p.skip[d] : 0.0f;
    float dskip = 0.0f, dbias = 0.0f;
    const uint32_t at = static_cast<uint32_t>(d) * sizeof(WT);  // within a token
    const int64_t first = first_part(p, o);
    const float* check = q.check + first * (DN + p.D) + d;
    // One part; FULL: of kPart tokens.
    auto walk = [&](int part, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t t0 = o.t0 + part * kPart;
        const int m = min(kPart, o.n - part * kPart);
        PartRows<WT, FULL> xr, dr, gr, zr;
        dr.load(p.dt, t0, m, at);
        xr.load(p.x, t0, m, at);
        gr.load(q.d_o, t0, m, at);
        if constexpr (GATED) zr.load(p.z, t0, m, at);
        const float* ck = check + part * (DN + p.D);
        {   // all of the states' loads at once
            float st[N], at_part[N];
            if (cut) {
#pragma unroll
                for (int n = 0; n < N; ++n) st[n] = p.seg_state[mine + static_cast<int64_t>(n) * p.D];
            } else {
                state_row<N>(p.in, o.row, static_cast<int64_t>(d) * N, st);
            }
            if (part) {
                const float since = ck[DN] * kScanLog2e;  // step sizes from the segment's start
#pragma unroll
                for (int n = 0; n < N; ++n) at_part[n] = ck[static_cast<int64_t>(n) * p.D];
#pragma unroll
                for (int n = 0; n < N; ++n)
                    st[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(as[wave][n][lane] * since), st[n],
                                           at_part[n]);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) hs[wave][n][lane] = st[n];
        }
        const float* bc = q.turned + ((first + part) * p.G + g) * 2 * N * kPart;
        // delta, delta x, dy, and the sums over n.
        // Tokens past the row's end have no step and no gradient.
        float delta[kPart], u[kPart], dy[kPart], s1[kPart], s2[kPart], y[kPart];
#pragma unroll
        for (int i = 0; i < kPart; ++i) delta[i] = scan_value(dr.v[i]) + bias;
        if (p.softplus) {
#pragma unroll
            for (int i = 0; i < kPart; ++i) delta[i] = scan_softplus(delta[i]);
        }
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const bool in = (FULL || i < m) && live;
            float gy = scan_value(gr.v[i]);
            if constexpr (GATED) {
                const float zv = scan_value(zr.v[i]);
                gy *= zv * scan_sigmoid(zv);
            }
            delta[i] = FULL || i < m ? delta[i] : 0.0f;
            dy[i] = in ? gy : 0.0f;
            u[i] = in ? delta[i] * scan_value(xr.v[i]) : 0.0f;
            s1[i] = s2[i] = y[i] = 0.0f;
        }
        __syncthreads();  // the sums of the part before have been read
        // The next state's operands are fetched a state ahead (gradients of 2 x 2048 tokens
        // without a gate 315 us, 338 without; 1024 channels of 64 states 295 and 334), but not
        // with a gate and few states, where registers run out (402 us, 384 without).
        constexpr bool AHEAD = !GATED || N > 16;
        float b1[kPart], c1[kPart], an1, st1, mu1;
        if constexpr (AHEAD) {
            uniform_row<float, kPart>(bc, 0, b1);
            uniform_row<float, kPart>(bc, N * kPart, c1);
            an1 = as[wave][0][lane];
            st1 = hs[wave][0][lane];
            mu1 = carry[wave][0][lane];
        }
        for (int n = 0; n < N; ++n) {
            if constexpr (!AHEAD) {
                an1 = as[wave][n][lane];
                st1 = hs[wave][n][lane];
                mu1 = carry[wave][n][lane];
            }
            const float an = an1, a2 = an * kScanLog2e, start = st1;
            float mu = mu1;
            if (AHEAD && n + 1 < N) {
                an1 = as[wave][n + 1][lane];
                st1 = hs[wave][n + 1][lane];
                mu1 = carry[wave][n + 1][lane];
            }
            float b[kPart], c[kPart];
            if constexpr (AHEAD) {
#pragma unroll
                for (int i = 0; i < kPart; ++i) {
                    b[i] = b1[i];
                    c[i] = c1[i];
                }
                if (n + 1 < N) {
                    uniform_row<float, kPart>(bc, (n + 1) * kPart, b1);
                    uniform_row<float, kPart>(bc, (N + n + 1) * kPart, c1);
                }
            } else {
                uniform_row<float, kPart>(bc, n * kPart, b);
                uniform_row<float, kPart>(bc, (N + n) * kPart, c);
            }
            float a[kPart], h[kPart], hp = start;
#pragma unroll
            for (int i = 0; i < kPart; ++i) {
                a[i] = __builtin_amdgcn_exp2f(delta[i] * a2);
                h[i] = __builtin_fmaf(a[i], hp, u[i] * b[i]);
                hp = h[i];
                if constexpr (GATED) y[i] = __builtin_fmaf(c[i], h[i], y[i]);
            }
            float ga = 0.0f;
#pragma unroll
            for (int i = kPart - 1; i >= 0; --i) {
                const float lam = __builtin_fmaf(dy[i], c[i], mu);
                s1[i] = __builtin_fmaf(lam, b[i], s1[i]);
                mu = a[i] * lam;
                const float w = mu * (i ? h[i - 1] : start);
                s2[i] = __builtin_fmaf(an, w, s2[i]);
                ga = __builtin_fmaf(delta[i], w, ga);
                a[i] = lam * u[i];
                h[i] = dy[i] * h[i];
            }
            carry[wave][n][lane] = mu;
            da[wave][n][lane] += ga;
            const float sum = sums32(a, h);
            if (!(lane & 16)) red[wave][n][(lane >> 5) * kPart + (lane & 15)] = sum;
        }
        // The raw operands once more (from the caches): kept through the loop above they
        // would take 48 registers that it does not have.
        xr.load(p.x, t0, m, at);
        if (p.softplus) {
            dr.load(p.dt, t0, m, at);
#pragma unroll
            for (int i = 0; i < kPart; ++i) {
                float slope;
                scan_softplus(scan_value(dr.v[i]) + bias, slope);
                s2[i] = __builtin_fmaf(scan_value(xr.v[i]), s1[i], s2[i]) * slope;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPart; ++i) s2[i] = __builtin_fmaf(scan_value(xr.v[i]), s1[i], s2[i]);
        }
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const float xv = scan_value(xr.v[i]);
            dbias += FULL || i < m ? s2[i] : 0.0f;
            dskip = __builtin_fmaf(dy[i], xv, dskip);
            s1[i] = __builtin_fmaf(skip, dy[i], delta[i] * s1[i]);
            if constexpr (GATED) y[i] = __builtin_fmaf(skip, xv, y[i]);
        }
        if constexpr (GATED) {
            gr.load(q.d_o, t0, m, at);
            zr.load(p.z, t0, m, at);
#pragma unroll
            for (int i = 0; i < kPart; ++i) {
                const float zv = scan_value(zr.v[i]), sig = scan_sigmoid(zv);
                y[i] *= scan_value(gr.v[i]) * (sig * __builtin_fmaf(zv, 1.0f - sig, 1.0f));
            }
        }
        if (live) {
            part_store<WT, FULL>(q.dx, t0, m, at, s1);
            part_store<WT, FULL>(q.ddt, t0, m, at, s2);
            if constexpr (GATED) part_store<WT, FULL>(q.dz, t0, m, at, y);
        }
        __syncthreads();
        for (int i = tid; i < 2 * kPart * N; i += kGradThreads) {
            const int n = i % N, v = i / N;  // v: dB's tokens, then dC's
            const int t = v % kPart;
            if (!FULL && t >= m) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kGradWaves; ++w) s += red[w][n][v];
            q.part_bc[((static_cast<int64_t>(gt) * p.T + t0 + t) * p.G + g) * 2 * N +
                      (v / kPart) * N + n] = s;
        }
    };
    const int parts = (o.n + kPart - 1) / kPart;
    for (int part = parts - 1; part >= 0; --part) {
        if ((part + 1) * kPart <= o.n) walk(part, std::true_type());
        else walk(part, std::false_type());
    }
    if (!live) return;
    for (int n = 0; n < N; ++n) {
        part_a[static_cast<int64_t>(n) * p.D] = da[wave][n][lane];
        if (q.dinit && o.s == 0) {
            const int64_t at = o.row * q.dinit_outer + static_cast<int64_t>(d) * N + n;
            if (q.dinit_bf16) static_cast<uint16_t*>(q.dinit)[at] = scan_round(carry[wave][n][lane]);
            else static_cast<float*>(q.dinit)[at] = carry[wave][n][lane];
        }
    }
    part_d[0] = dskip;
    part_d[p.D] = dbias;
}

// ---------------------------------------------------------- 4: sums of parts ---

// Workgroups [0, n_bc): dB and dC; [n_bc, n_bc + n_a): dA; then dskip and dt_bias's.
template <typename WT>
__global__ void __launch_bounds__(256) grad_reduce(const ScanParams p, const ScanGrad q, int n_bc,
                                                   int n_a) {
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const int gtiles = q.tiles;
    const int block = blockIdx.x;
    if (block < n_bc) {
        const int64_t per = static_cast<int64_t>(p.G) * 2 * p.N, n = p.T * per;
        const int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x;
        if (i >= n) return;
        const int64_t t = i / per;
        if (t < p.offsets[0] || t >= p.offsets[p.B]) return;
        float s = 0.0f;
        for (int k = 0; k < gtiles; ++k) s += q.part_bc[k * n + i];
        const int r = static_cast<int>(i - t * per), g = r / (2 * p.N), v = r - g * 2 * p.N;
        const ScanHeads& out = v < p.N ? q.db : q.dc;
        scan_put(static_cast<WT*>(const_cast<void*>(out.p)) + t * out.tok + g * out.grp +
                     (v < p.N ? v : v - p.N), s);
        return;
    }
    const bool isa = block < n_bc + n_a;
    const int64_t n = isa ? DN : 2 * static_cast<int64_t>(p.D);
    const int64_t i = static_cast<int64_t>(block - n_bc - (isa ? 0 : n_a)) * 256 + threadIdx.x;
    if (i >= n) return;
    const float* part = (isa ? q.part_a : q.part_d) + i;
    double s0 = 0.0, s1 = 0.0;
    int r = 0;
    for (; r + 8 <= p.segs; r += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = part[(r + k) * n];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            s0 += static_cast<double>(v[k]);
            s1 += static_cast<double>(v[k + 1]);
        }
    }
    for (; r < p.segs; ++r) s0 += static_cast<double>(part[r * n]);
    const float s = static_cast<float>(s0 + s1);
    if (isa) {
        const int64_t k = i / p.D, d = i - k * p.D;
        q.dA[d * p.N + k] = s;
    } else if (i < p.D) {
        if (q.dskip) q.dskip[i] = s;
    } else if (q.dbias) {
        q.dbias[i - p.D] = s;
    }
}

template <typename WT, int N>
hipError_t bwd_n(const ScanParams& p, const ScanGrad& q, hipStream_t s) {
    const int64_t DN = static_cast<int64_t>(p.D) * N;
    hipError_t e;
    if (p.segs) {
        constexpr int S = sum_states(N);
        hipLaunchKernelGGL((grad_sums<WT, S>),
                           dim3(scan_blocks(static_cast<int64_t>(p.segs) * p.G * (N / S * p.tiles + 1))),
                           dim3(kScanThreads), 0, s, p, q);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.seg_len) {
        const unsigned blocks = static_cast<unsigned>((DN + 255) / 256);
        hipLaunchKernelGGL(grad_chains, dim3(2u * p.B * blocks), dim3(256), 0, s, p, q);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.segs) {
        const dim3 grid(static_cast<unsigned>(p.segs) * p.G * q.tiles), block(64 * grad_waves(N));
        if (p.z.p) hipLaunchKernelGGL((grad_walk<WT, N, true>), grid, block, 0, s, p, q);
        else hipLaunchKernelGGL((grad_walk<WT, N, false>), grid, block, 0, s, p, q);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t bc = p.B > 0 ? static_cast<int64_t>(p.T) * p.G * 2 * N : 0;
    const int n_bc = static_cast<int>((bc + 255) / 256), n_a = static_cast<int>((DN + 255) / 256);
    const int n_d = (2 * p.D + 255) / 256;
    hipLaunchKernelGGL(grad_reduce<WT>, dim3(n_bc + n_a + n_d), dim3(256), 0, s, p, q, n_bc, n_a);
    return hipGetLastError();
}

template <typename WT> hipError_t bwd_wt(const ScanParams& p, const ScanGrad& q, hipStream_t s) {
    switch (p.N) {
        case 8: return bwd_n<WT, 8>(p, q, s);
        case 16: return bwd_n<WT, 16>(p, q, s);
        case 32: return bwd_n<WT, 32>(p, q, s);
        case 64: return bwd_n<WT, 64>(p, q, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

int scan_grad_channels(int N) { return 64 * grad_waves(N); }

hipError_t launch_scan_bwd(const ScanParams& p, const ScanGrad& q, bool work_bf16, hipStream_t s) {
    return work_bf16 ? bwd_wt<uint16_t>(p, q, s) : bwd_wt<float>(p, q, s);
}

}  // namespace gdr

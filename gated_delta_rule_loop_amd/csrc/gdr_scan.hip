// gfx950 kernels of the selective state space scan:
//     delta = softplus(dt + dt_bias)     a = exp(delta A[d, n])
//     h_t = a h_{t-1} + delta x B_t[n]   out = (sum_n C_t[n] h_t + skip x) silu(z)
// for every channel d and its N states n, in float32.  The decay is a number of
// its own for every token, channel and state, so there is no form as matrix
// products: the work is 6 vector-unit slots a token, channel and state (product,
// exponential, which takes two, product, two multiply-adds).  At 39e12 slots a second,
// what the unit issues, they bound every walk over long rows.
//
// Wide walk (prompts): a lane owns a channel and all its states, in registers;
// B and C of a token are the same for the whole wave and come through scalar
// loads.  Long rows are cut into segments so that few channels still fill the
// chip: one launch takes each segment's own end state from zero and the sum of
// its step sizes (a segment's decay is exp(A sum delta)), one chains them to the
// states the segments start from, and the walk follows.  16384 bf16 tokens of 4096
// channels of 16 states 471 us (183, 18 and 268), where the 275 slots a token and channel of
// both passes take 469; 32 rows of 512, enough for one piece a row, 348 (150 slots, 256 us).
//
// Lane walk (prompts of few tokens or many states): 16 lanes own a channel, so that
// one launch has 16 times the waves and nothing is walked twice.  97 tokens of 4096
// channels of 16 states 17 us (segments 25), 1500 of 2048 channels of 64 122 (168).
//
// Narrow walk (single tokens, folds): a lane owns 16 bytes of a
// channel's state, so that states are read and written in whole lines; the
// output is summed over a channel's 1 to 16 lanes by lane permutations.  256 single
// tokens of 4096 channels of 16 bf16 states: 19 us for 74 MB.
#include <type_traits>

#include "gdr_scan_dev.h"

namespace gdr {
namespace {

// ------------------------------------------------------------- narrow walk ---

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

// U: tokens whose operands are loaded ahead of those in work.
template <typename WT, typename ST, int N, bool OUT, int U>
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
    Token<WT, S> next[U];
    auto fetch_all = [&](int t) {
#pragma unroll
        for (int j = 0; j < U; ++j) fetch(min(t + j, n - 1), next[j]);
    };
    // U tokens: what does not depend on the state for all of them first, so that their
    // long chains (softplus, sigmoid) run beside one another.  FULL: none is past the row.
    auto block = [&](int t, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        Token<WT, S> now[U];
        float delta[U], gate[U], y[U];
#pragma unroll
        for (int j = 0; j < U; ++j) now[j] = next[j];
        if (t + U < n) fetch_all(t + U);
#pragma unroll
        for (int j = 0; j < U; ++j) delta[j] = now[j].dt + bias;
        if (p.softplus) {
#pragma unroll
            for (int j = 0; j < U; ++j) delta[j] = scan_softplus(delta[j]);
        }
        if constexpr (OUT) {
#pragma unroll
            for (int j = 0; j < U; ++j) gate[j] = 1.0f;
            if (z) {
#pragma unroll
                for (int j = 0; j < U; ++j) gate[j] = now[j].z * scan_sigmoid(now[j].z);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!FULL && t + j >= n) continue;
            const float u = delta[j] * now[j].x;
            y[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta[j] * a2[i]), h[i], u * now[j].b[i]);
                if constexpr (OUT) y[j] = __builtin_fmaf(h[i], now[j].c[i], y[j]);
            }
        }
        if constexpr (OUT) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                y[j] = __builtin_fmaf(skip, now[j].x, lane_sum<L>(y[j])) * gate[j];
            if (sub == 0) {
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (FULL || t + j < n)
                        scan_put(static_cast<WT*>(p.out) + static_cast<int64_t>(t0 + t + j) * p.o_tok + d,
                                 y[j]);
            }
        }
    };
    if (n > 0) fetch_all(0);
    int t = 0;
    for (; t + U <= n; t += U) block(t, std::true_type());
    if (t < n) block(t, std::false_type());
    if (p.last && !p.keep)
        scan_store<S>(static_cast<ST*>(p.last) + static_cast<int64_t>(slot) * p.last_outer + at, h);
}

template <typename WT, typename ST, int N>
hipError_t narrow_out(const ScanParams& p, hipStream_t s) {
    constexpr int S = N < static_cast<int>(16 / sizeof(ST)) ? N : 16 / sizeof(ST);
    const int per = kScanNarrowThreads / (N / S);
    const dim3 grid(static_cast<unsigned>(p.B) * ((p.D + per - 1) / per));
    // Rows of about one token have nothing to load ahead for; longer ones come here in
    // folds and, without a lane walk, in calls of few tokens (64 tokens of 8 states 32 us, one
    // token ahead 38; the fold of 64 windows of 1 to 12 tokens 14 us with either).
    const bool one = p.T <= p.B + p.B / 2;
    if constexpr (N < 16) {
        if (p.out && !one) {
            hipLaunchKernelGGL((scan_narrow<WT, ST, N, true, 4>), grid, dim3(kScanNarrowThreads), 0, s, p);
            return hipGetLastError();
        }
    }
    if (p.out)
        hipLaunchKernelGGL((scan_narrow<WT, ST, N, true, 1>), grid, dim3(kScanNarrowThreads), 0, s, p);
    else if (one)
        hipLaunchKernelGGL((scan_narrow<WT, ST, N, false, 1>), grid, dim3(kScanNarrowThreads), 0, s, p);
    else
        hipLaunchKernelGGL((scan_narrow<WT, ST, N, false, 4>), grid, dim3(kScanNarrowThreads), 0, s, p);
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
    const int ctiles = p.G * p.tiles, wave = scan_wave();
    const int seg = wave / ctiles, tile = wave - seg * ctiles;
    ScanSpan o;
    if (seg >= p.segs || !scan_locate(p, seg, o)) return;
    if (SUMS && o.s == o.count - 1) return;
    const int g = tile / p.tiles;
    const int cg = (tile - g * p.tiles) * 64 + static_cast<int>(threadIdx.x & 63);
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
    const bool gated = !SUMS && p.z.p != nullptr;
    const ScanRows zrow = gated ? p.z : p.x;
    const uint32_t off = static_cast<uint32_t>(d) * sizeof(WT);
    const uint32_t sx = scan_step<WT>(p.x), sd = scan_step<WT>(p.dt), sz = scan_step<WT>(zrow);
    const ScanRows orow = {p.out, p.o_tok};
    char* out = const_cast<char*>(scan_base<WT>(orow, o.t0));
    const uint32_t so = scan_step<WT>(orow);
    const char* pb = static_cast<const char*>(p.b.p) +
                     (static_cast<int64_t>(o.t0) * p.b.tok + static_cast<int64_t>(g) * p.b.grp) * static_cast<int64_t>(sizeof(WT));
    const char* pc = SUMS ? pb : static_cast<const char*>(p.c.p) +
                     (static_cast<int64_t>(o.t0) * p.c.tok + static_cast<int64_t>(g) * p.c.grp) * static_cast<int64_t>(sizeof(WT));
    const uint32_t sb = static_cast<uint32_t>(p.b.tok) * sizeof(WT);
    const uint32_t sc = static_cast<uint32_t>(p.c.tok) * sizeof(WT);
    WT xs[kAhead], ds[kAhead], zs[kAhead];
    auto fetch = [&](int t) {
        const char *bx = scan_base<WT>(p.x, o.t0 + t), *bd = scan_base<WT>(p.dt, o.t0 + t);
        const char* bz = scan_base<WT>(zrow, o.t0 + t);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t k = min(i, o.n - 1 - t);
            xs[i] = scan_at<WT>(bx, off + k * sx);
            ds[i] = scan_at<WT>(bd, off + k * sd);
            if constexpr (!SUMS) zs[i] = scan_at<WT>(bz, off + k * sz);
        }
    };
    float total = 0.0f;
    constexpr int S = scan_ahead<WT>(N);
    typedef ScalarRows<WT, N, S, !SUMS> Rows;
    auto token = [&](const Rows& r, int i, WT xr, WT dr, WT zr, char* to) {
        const float xv = scan_value(xr);
        float delta = scan_value(dr) + bias;
        if (p.softplus) delta = scan_softplus(delta);
        const float u = delta * xv;
        if constexpr (SUMS) {
            total += delta;
#pragma unroll
            for (int k = 0; k < N; ++k)
                h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[k]), h[k],
                                      u * Rows::value(r.b[i], k));
        } else {
            float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * a2[k]), h[k],
                                      u * Rows::value(r.b[i], k));
                if (k & 1) y1 = __builtin_fmaf(h[k], Rows::value(r.c[i], k), y1);
                else y0 = __builtin_fmaf(h[k], Rows::value(r.c[i], k), y0);
            }
            float y = __builtin_fmaf(skip, xv, y0 + y1);
            if (gated) {
                const float zv = scan_value(zr);
                y *= zv * scan_sigmoid(zv);
            }
            if (live) scan_put(reinterpret_cast<WT*>(to + off), y);
        }
    };
    fetch(0);
    Rows rows[2];
    rows[0].load(pb, pc, sb, sc, 0, o.n);
    auto block = [&](int t, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        WT xc[kAhead], dc[kAhead], zc[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            xc[i] = xs[i];
            dc[i] = ds[i];
            if constexpr (!SUMS) zc[i] = zs[i];
        }
        if (t + kAhead < o.n) fetch(t + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; i += S) {
            Rows &now = rows[(i / S) & 1], &next = rows[(i / S + 1) & 1];
            now.arrive();
            next.load(pb, pc, sb, sc, t + i + S, o.n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (FULL || t + i + j < o.n)
                    token(now, j, xc[i + j], dc[i + j], SUMS ? xc[i + j] : zc[i + j],
                          out + static_cast<uint64_t>(t + i + j) * so);
        }
    };
    int t = 0;
    for (; t + kAhead <= o.n; t += kAhead) block(t, std::true_type());
    if (t < o.n) block(t, std::false_type());
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

// --------------------------------------------------------------- lane walk ---

// A wave takes four channels, 16 lanes each, and 16 tokens at a time.  Lane j of a
// channel holds N / 16 of its states and is also the one that reads token j's x, dt and z
// and takes their softplus and gate, once for all states; step sizes go to the
// channel's lanes as broadcast operands.  The 16 tokens' outputs, sums over the
// lanes, are added by halving (15 exchanges instead of 64), which leaves token j's in
// lane j.  B and C come 16 tokens at a time through LDS, turned to a state's tokens.
// No wave needs another's work.
constexpr int kLanes = 16;
constexpr int kLanePad = 20;  // floats from one state's tokens to the next's in LDS

template <int K> __device__ __forceinline__ float from_lane(float v) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)),
                                                    0x150 + K, 0xf, 0xf, true));
}

template <typename WT, int N> struct LaneWalk {
    static constexpr int S = N / kLanes;   // states a lane
    static constexpr int V = N / 2;        // values of B or C that a lane brings
    float h[S], a2[S];
    float y[kLanes];

    template <int K, bool FULL>
    __device__ __forceinline__ void token(float delta, float u, const float (&b)[S], const float (&c)[S],
                                          int left) {
        y[K] = 0.0f;
        if (!FULL && K >= left) return;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const float e = __builtin_amdgcn_exp2f(from_lane<K>(delta) * a2[i]);
            h[i] = __builtin_fmaf(e, h[i], from_lane<K>(u) * b[i]);
            y[K] = i ? __builtin_fmaf(h[i], c[i], y[K]) : h[i] * c[i];
        }
    }
    // Tokens 4 Q to 4 Q + 3 of the block in work, of which the first `left` are the row's;
    // lds: B's states, then C's.
    template <int Q, bool FULL>
    __device__ __forceinline__ void four(float delta, float u, const float* lds, int j, int left) {
        float b[4][S], c[4][S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const float* at = lds + (j * S + i) * kLanePad + 4 * Q;
            const float4 p = *reinterpret_cast<const float4*>(at);
            const float4 q = *reinterpret_cast<const float4*>(at + N * kLanePad);
            b[0][i] = p.x; b[1][i] = p.y; b[2][i] = p.z; b[3][i] = p.w;
            c[0][i] = q.x; c[1][i] = q.y; c[2][i] = q.z; c[3][i] = q.w;
        }
        token<4 * Q, FULL>(delta, u, b[0], c[0], left);
        token<4 * Q + 1, FULL>(delta, u, b[1], c[1], left);
        token<4 * Q + 2, FULL>(delta, u, b[2], c[2], left);
        token<4 * Q + 3, FULL>(delta, u, b[3], c[3], left);
    }
};

template <typename WT, typename ST, int N>
__global__ void __launch_bounds__(kScanThreads) scan_lanes(const ScanParams p) {
    typedef LaneWalk<WT, N> Walk;
    constexpr int S = Walk::S, V = Walk::V;
    __shared__ __attribute__((aligned(16))) float staged[kScanThreads / 64][2][2 * N * kLanePad];
    const int tiles = (p.D + kScanLaneChannels - 1) / kScanLaneChannels;
    const int row = blockIdx.x / tiles;
    int tile = blockIdx.x - row * tiles;
    // Four neighbouring tiles of bf16 share the lines of a token: the dies take workgroups
    // in turn, so that every eighth gets the next of four.
    if (tile < (tiles & ~31)) tile = (tile & ~31) | ((tile & 7) << 2) | ((tile >> 3) & 3);
    const int t0 = static_cast<int>(scan_index(p.offsets, row));
    const int n = static_cast<int>(scan_index(p.offsets, row + 1)) - t0;
    if (n <= p.narrow_most || n > p.lane_most) return;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int first = tile * kScanLaneChannels + wave * 4;  // of the wave's channels
    if (first >= p.D) return;
    const int lane = threadIdx.x & 63, j = lane & (kLanes - 1);
    const int d = first + (lane >> 4), g = first / p.gd;    // groups are whole fours
    const uint32_t slot = p.slot_idx ? scan_index(p.slot_idx, row) : static_cast<uint32_t>(row);
    const ScanRows orow = {p.out, p.o_tok};
    if (p.slot_idx != nullptr && slot == kPadSlot) {
        for (int t = j; t < n; t += kLanes)
            scan_put(static_cast<WT*>(p.out) + static_cast<int64_t>(t0 + t) * p.o_tok + d, 0.0f);
        return;
    }
    const int64_t at = static_cast<int64_t>(d) * N + j * S;
    Walk w;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        w.a2[i] = p.A[at + i] * kScanLog2e;
        w.h[i] = p.in.p ? scan_value(static_cast<const ST*>(p.in.p)[static_cast<int64_t>(slot) * p.in.outer + at + i])
                        : 0.0f;
    }
    const float bias = p.bias ? p.bias[d] : 0.0f, skip = p.skip ? p.skip[d] : 0.0f;
    const bool gated = p.z.p != nullptr;
    const ScanRows zrow = gated ? p.z : p.x;
    // token j's operands, and a quarter of token lane / 4's B or C
    const uint32_t off = static_cast<uint32_t>(d) * sizeof(WT);
    const uint32_t sx = scan_step<WT>(p.x), sd = scan_step<WT>(p.dt), sz = scan_step<WT>(zrow),
                   so = scan_step<WT>(orow);
    const int mine = lane >> 2, part = lane & 3;
    const ScanHeads bc = part < 2 ? p.b : p.c;
    const WT* bcp = static_cast<const WT*>(bc.p) + static_cast<int64_t>(t0) * bc.tok +
                    static_cast<int64_t>(g) * bc.grp + (part & 1) * V;
    const int to = ((part >> 1) * N + (part & 1) * V) * kLanePad + mine;
    // Three blocks are in work at once: the operands of the one after the next are being
    // loaded, the next one's go to LDS and through softplus and gate, and this one's
    // states are stepped.
    const int final = (n - 1) / kLanes * kLanes;  // the last block's first token
    struct Raw {
        WT x, dt, z;
        float bc[V];
    };
    struct Ready {
        float x, delta, u, gate;
    };
    Raw raw;
    Ready next;
    auto fetch = [&](int t) {
        t = min(t, final);
        const uint32_t k = min(j, n - 1 - t);
        raw.x = scan_at<WT>(scan_base<WT>(p.x, t0 + t), off + k * sx);
        raw.dt = scan_at<WT>(scan_base<WT>(p.dt, t0 + t), off + k * sd);
        raw.z = scan_at<WT>(scan_base<WT>(zrow, t0 + t), off + k * sz);
        scan_load<V>(bcp + static_cast<int64_t>(min(t + mine, n - 1)) * bc.tok, raw.bc);
    };
    auto ready = [&](int t) {  // of block t, which was loaded last
        float* lds = staged[wave][(t / kLanes) & 1] + to;
#pragma unroll
        for (int i = 0; i < V; ++i) lds[i * kLanePad] = raw.bc[i];
        const float dt = scan_value(raw.dt) + bias, z = scan_value(raw.z);
        const float delta = p.softplus ? scan_softplus(dt) : dt;
        next.x = scan_value(raw.x);
        next.delta = delta;
        next.u = delta * next.x;
        next.gate = gated ? z * scan_sigmoid(z) : 1.0f;
    };
    fetch(0);
    ready(0);
    fetch(kLanes);
    auto block = [&](int t, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const Ready now = next;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // LDS serves a wave in order
        ready(t + kLanes);
        fetch(t + 2 * kLanes);
        const float* lds = staged[wave][(t / kLanes) & 1];
        w.template four<0, FULL>(now.delta, now.u, lds, j, n - t);
        w.template four<1, FULL>(now.delta, now.u, lds, j, n - t);
        w.template four<2, FULL>(now.delta, now.u, lds, j, n - t);
        w.template four<3, FULL>(now.delta, now.u, lds, j, n - t);
        const float y = __builtin_fmaf(skip, now.x, row_sums16(w.y)) * now.gate;
        if (FULL || t + j < n)
            scan_put(reinterpret_cast<WT*>(const_cast<char*>(scan_base<WT>(orow, t0 + t)) + off + j * so), y);
    };
    int t = 0;
    for (; t + kLanes <= n; t += kLanes) block(t, std::true_type());
    if (t < n) block(t, std::false_type());
    if (p.last && !p.keep) {
        ST* last = static_cast<ST*>(p.last) + static_cast<int64_t>(slot) * p.last_outer + at;
#pragma unroll
        for (int i = 0; i < S; ++i) scan_put(last + i, w.h[i]);
    }
}

template <typename WT, typename ST> hipError_t lanes_n(const ScanParams& p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.B) * ((p.D + kScanLaneChannels - 1) / kScanLaneChannels));
    switch (p.N) {
        case 16: hipLaunchKernelGGL((scan_lanes<WT, ST, 16>), grid, dim3(kScanThreads), 0, s, p); break;
        case 32: hipLaunchKernelGGL((scan_lanes<WT, ST, 32>), grid, dim3(kScanThreads), 0, s, p); break;
        case 64: hipLaunchKernelGGL((scan_lanes<WT, ST, 64>), grid, dim3(kScanThreads), 0, s, p); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// seg_state of a cut row: from the segments' own end states to the states that
// they start from.
__global__ void __launch_bounds__(256) scan_chain(const ScanParams p) {
    const int64_t DN = static_cast<int64_t>(p.D) * p.N;
    const int blocks = static_cast<int>((DN + 255) / 256);
    const int row = blockIdx.x / blocks;
    const int64_t i = static_cast<int64_t>(blockIdx.x - row * blocks) * 256 + threadIdx.x;
    const int n = static_cast<int>(p.offsets[row + 1] - p.offsets[row]);
    // Uncut rows have nothing to chain, and rows that another walk takes no segment at all:
    // the places from scan_first_seg on would be the next cut row's.
    if (n <= max(p.seg_len, p.seg_skip)) return;
    const int64_t first = scan_first_seg(p, row);
    if (i >= DN) return;
    const uint32_t slot = p.slot_idx ? p.slot_idx[row] : static_cast<uint32_t>(row);
    if (p.slot_idx != nullptr && slot == kPadSlot) return;
    const int count = (n + p.seg_len - 1) / p.seg_len;
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
    const dim3 grid(scan_blocks(static_cast<int64_t>(p.segs) * p.G * p.tiles));
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

hipError_t launch_scan_lanes(const ScanParams& p, bool work_bf16, hipStream_t s) {
    if (work_bf16)
        return p.in.bf16 ? lanes_n<uint16_t, uint16_t>(p, s) : lanes_n<uint16_t, float>(p, s);
    return p.in.bf16 ? lanes_n<float, uint16_t>(p, s) : lanes_n<float, float>(p, s);
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

// Host side of the selective scan, of the Conv1d's gradient and history fold and
// of the verification of drafted tokens (include/gdr.h): argument validation,
// workspace layout, launch choice.
#include <algorithm>
#include <climits>
#include <initializer_list>

#include "gdr_host.h"
#include "gdr_scan.h"

using namespace gdr;

namespace {

typedef long long ll;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

constexpr int64_t kMaxTokens = INT32_MAX - 65536;
constexpr int64_t kMaxChannels = int64_t{1} << 24;

struct ScanDims {
    int64_t T, D, N, G, B;
    int32_t work;
    int64_t tiles() const { return ceil_div(D / G, 64); }
};

// Tokens are addressed by unsigned 32-bit offsets from a part's first.
constexpr int64_t kMaxTokenStride = (int64_t{1} << 24) - 1;

int check_token_stride(const char* fn, const char* name, const gdr_tensor* t) {
    if (t->shape[0] > 1 && !empty(t) && (t->stride[0] < 0 || t->stride[0] > kMaxTokenStride))
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s has a token stride outside 0..%lld elements", fn,
                    name, static_cast<ll>(kMaxTokenStride));
    return GDR_OK;
}

// [T, D] operand: unit innermost stride, 16-byte rows.
int check_rows(const char* fn, const char* name, const gdr_tensor* t, const ScanDims& d, bool out) {
    const int64_t shape[2] = {d.T, d.D};
    int rc = check_tensor(fn, name, t, 2, shape, true, true, false);
    if (rc || (rc = check_work_dtype(fn, name, t, d.work)) ||
        (rc = check_layout(fn, name, t, vec_mult(d.work))) ||
        (rc = check_token_stride(fn, name, t)))
        return rc;
    return out ? check_distinct(fn, name, t) : GDR_OK;
}

int check_groups(const char* fn, const char* name, const gdr_tensor* t, const ScanDims& d,
                 bool out) {
    const int64_t shape[3] = {d.T, d.G, d.N};
    int rc = check_tensor(fn, name, t, 3, shape, true, true, false);
    if (rc || (rc = check_work_dtype(fn, name, t, d.work)) ||
        (rc = check_layout(fn, name, t, vec_mult(d.work))) ||
        (rc = check_token_stride(fn, name, t)))
        return rc;
    return out ? check_distinct(fn, name, t) : GDR_OK;
}

// float32 [D], contiguous.
int check_channels(const char* fn, const char* name, const gdr_tensor* t, int64_t D) {
    const int64_t shape[1] = {D};
    const int rc = check_tensor(fn, name, t, 1, shape, true, false, false);
    if (rc) return rc;
    if (D > 1 && t->stride[0] != 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s must be contiguous", fn, name);
    return GDR_OK;
}

// States [slots or rows, D, N], each D x N block dense.
int check_scan_state(const char* fn, const char* name, const gdr_tensor* t, int64_t rows,
                     const ScanDims& d, bool out) {
    const int64_t shape[3] = {rows, d.D, d.N};
    int rc = check_tensor(fn, name, t, 3, shape, true, true, false);
    if (rc) return rc;
    if (!empty(t) && (t->stride[2] != 1 || t->stride[1] != d.N))
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s needs a dense D x N block per slot", fn, name);
    if ((rc = check_layout(fn, name, t, vec_mult(t->dtype)))) return rc;
    return out ? check_distinct(fn, name, t) : GDR_OK;
}

int check_decay(const char* fn, const char* name, const gdr_tensor* t, const ScanDims& d) {
    const int64_t shape[2] = {d.D, d.N};
    const int rc = check_tensor(fn, name, t, 2, shape, true, false, false);
    if (rc) return rc;
    if (!empty(t) && (t->stride[1] != 1 || (d.D > 1 && t->stride[0] != d.N)))
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s must be contiguous", fn, name);
    if (!empty(t) && !aligned16(t->data))
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s base must be 16-byte aligned", fn, name);
    return GDR_OK;
}

// What every entry of the scan has: x, dt, A, B and dt_bias.
int check_scan(const char* fn, const gdr_tensor* x, const gdr_tensor* dt, const gdr_tensor* A,
               const gdr_tensor* Bm, const gdr_tensor* dt_bias, uint32_t flags, uint32_t known,
               ScanDims& d) {
    int rc;
    if (flags & ~known) return fail(GDR_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if ((rc = check_tensor(fn, "x", x, 2, nullptr, true, true, false)) ||
        (rc = check_tensor(fn, "B", Bm, 3, nullptr, true, true, false)))
        return rc;
    d.T = x->shape[0];
    d.D = x->shape[1];
    d.G = Bm->shape[1];
    d.N = Bm->shape[2];
    d.work = x->dtype;
    if (d.N != 8 && d.N != 16 && d.N != 32 && d.N != 64)
        return fail(GDR_ERR_UNSUPPORTED, "%s: state size %lld not built (8, 16, 32, 64)", fn,
                    static_cast<ll>(d.N));
    if (d.G < 1 || d.D < 1 || d.D % d.G != 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: channels (%lld) must be a positive multiple of B's "
                    "groups (%lld)", fn, static_cast<ll>(d.D), static_cast<ll>(d.G));
    if (d.D / d.G % 4 != 0)
        return fail(GDR_ERR_UNSUPPORTED, "%s: channels of a group must be a multiple of 4", fn);
    if (d.T > kMaxTokens || d.D > kMaxChannels)
        return fail(GDR_ERR_INVALID_ARG, "%s: too many tokens or channels", fn);
    if ((rc = check_rows(fn, "x", x, d, false)) || (rc = check_rows(fn, "dt", dt, d, false)) ||
        (rc = check_decay(fn, "A", A, d)) || (rc = check_groups(fn, "B", Bm, d, false)))
        return rc;
    if (present(dt_bias) && (rc = check_channels(fn, "dt_bias", dt_bias, d.D))) return rc;
    return GDR_OK;
}

int check_offsets(const char* fn, const gdr_tensor* off, int64_t& B) {
    const int rc = check_tensor(fn, "input_row_offsets", off, 1, nullptr, false, false, true);
    if (rc) return rc;
    B = off->shape[0] - 1;
    if (B < 0) return fail(GDR_ERR_INVALID_ARG, "%s: input_row_offsets is empty", fn);
    if (B > kMaxTokens) return fail(GDR_ERR_INVALID_ARG, "%s: too many rows", fn);
    return check_index_vec(fn, "input_row_offsets", off, B + 1);
}

ScanRows rows_of(const gdr_tensor* t) {
    ScanRows r{};
    if (!present(t)) return r;
    r.p = t->data;
    r.tok = t->shape[0] > 1 ? t->stride[0] : 0;  // a single token's stride can be anything
    return r;
}

ScanHeads heads_of(const gdr_tensor* t) {
    ScanHeads h{};
    if (!present(t)) return h;
    h.p = t->data;
    h.tok = t->shape[0] > 1 ? t->stride[0] : 0;
    h.grp = t->shape[1] > 1 ? t->stride[1] : 0;
    return h;
}

ScanState state_of(const gdr_tensor* t) {
    ScanState s{};
    if (!present(t)) return s;
    s.p = t->data;
    s.outer = t->stride[0];
    s.bf16 = t->dtype == GDR_DTYPE_BF16;
    return s;
}

const float* floats(const gdr_tensor* t) {
    return present(t) ? static_cast<const float*>(t->data) : nullptr;
}

ScanParams scan_params(const ScanDims& d, const gdr_tensor* x, const gdr_tensor* dt,
                       const gdr_tensor* A, const gdr_tensor* Bm, const gdr_tensor* dt_bias,
                       const gdr_tensor* off, const gdr_tensor* slots, uint32_t flags) {
    ScanParams p{};
    p.B = static_cast<int32_t>(d.B);
    p.T = static_cast<int32_t>(d.T);
    p.D = static_cast<int32_t>(d.D);
    p.N = static_cast<int32_t>(d.N);
    p.G = static_cast<int32_t>(d.G);
    p.gd = static_cast<int32_t>(d.D / d.G);
    p.tiles = static_cast<int32_t>(d.tiles());
    p.softplus = (flags & GDR_FLAG_DT_SOFTPLUS) != 0;
    p.keep = (flags & GDR_FLAG_KEEP_STATE) != 0;
    p.offsets = as_u32(off);
    p.slot_idx = as_u32(slots);
    p.x = rows_of(x);
    p.dt = rows_of(dt);
    p.A = static_cast<const float*>(A->data);
    p.bias = floats(dt_bias);
    p.b = heads_of(Bm);
    return p;
}

int64_t narrow_blocks(const ScanDims& d, bool state_bf16) {
    const int64_t states = std::min<int64_t>(d.N, state_bf16 ? 8 : 4);
    return d.B * ceil_div(d.D, kScanNarrowThreads / (d.N / states));
}

// How a forward is cut: rows up to `narrow` tokens take the narrow walk, longer ones up to
// `lane` the lane walk, and longer ones still the wide walk in segments of seg_len tokens
// (0: uncut).  All walks leave the same bits in the states of rows that are not cut.
//   - Calls of about a token a row go narrowly, those of few tokens too where there is no
//     lane walk: 64 rows of 1 token of 4096 channels of 16 states 13 us (widely 30). Above
//     64 tokens the launches for longer rows, which may be among them, come behind it and
//     both ways take about as long: 256 rows of 1 token 59 us (widely 53), of 64 states 172
//     (208), 250 rows of 1 beside 40 and 80 tokens 95 (73), 511 beside 200 141 (145). A call
//     of single tokens alone is gdr_selective_scan_step's (256 rows 19 us).
//   - Calls whose rows fill the chip walk widely, rows cut only where they are longer than
//     all tokens' share of 2048 waves: 64 windows of 1 to 12 tokens of 4096 channels of 16
//     states 27 us (lane walk 32, narrow 37), 256 rows of 3 53 (113, 104), 32 rows of 512 348
//     (cut 480).  32 rows of 12 to 1023 tokens 648, cut at twice the share 958.
//   - Other calls take the lane walk or segments, as lanes_first says: 63 single tokens
//     beside a row of 190 35 us, the single ones narrowly 45; 16 rows of 16 beside one of 200
//     35 and 30.
// The wide walk's waves find their rows in time that grows with the number of rows (see
// scan_locate).
// Segments number as many as 8192 waves hold where the chip is not full: 16384 tokens of
// 4096 channels 470 us (4096 waves 508, 16384 469), 8 ragged rows in float32 165 (184, 169).
struct FwdPlan {
    int64_t narrow, lane, seg_len, segs, state, delta, end;
    bool wide;
};

constexpr int64_t kUncut = 64;  // tokens of a call up to which no row is cut

// Whether the lane walk takes a call whose rows do not fill the chip.  It goes along a row at about
// 6 + 1.5 N ns a token after 10 us, whatever the width (too few waves to hide what a token
// waits for); segments, their chain and the walk take 12 + 0.85 N us and D N / 2000 ns a
// token.  Measured, lane walk and segments, us: 97 tokens of 4096 channels x 16 states 17
// and 25, 800 of them 35 and 53, 1200 52 and 63, 2048 108 and 88; of 512 channels 350
// tokens 18 and 26; of 8192 channels 2048 tokens 130 and 138, 12000 904 and 698.  32
// states: 300 of 2048 channels 25 and 39, 1500 of 4096 104 and 116.  64 states: 300 of
// 1024 channels 41 and 67, 700 87 and 82, 3000 of 4096 352 and 489.  The longest row is
// not known here: all tokens may be one row's.
bool lanes_first(int64_t T, int64_t D, int64_t N) {
    return N >= 16 && T <= 96 * N && T * (12000 + 3000 * N - D * N) < 2000 * (2000 + 850 * N);
}

FwdPlan fwd_plan(int64_t T, int64_t B, int64_t D, int64_t N, int64_t G) {
    FwdPlan p{};
    const int64_t ctiles = G * ceil_div(D / G, 64);
    p.segs = B;
    const bool few = T <= kUncut;
    p.narrow = T <= B + B / 2 || (few && N < 16) ? kUncut : 0;
    p.lane = p.narrow;
    if (T <= p.narrow) return p;
    const bool full = !few && B * ctiles >= 2048;
    if (!full && lanes_first(T, D, N)) p.lane = T;
    p.wide = T > p.lane;
    if (p.wide) {
        const int64_t want = std::max<int64_t>(1, (full ? 2048 : 8192) / ctiles);
        const int64_t len = std::max<int64_t>(16, round_up(ceil_div(T, want), 16));
        if (len < T) {
            p.seg_len = len;
            p.segs = T / len + B;
            p.delta = round_up(p.segs * D * N, 64);
            p.end = p.delta + round_up(p.segs * D, 64);
        }
    }
    return p;
}

// How a gradient is cut, and where its workspace holds what.  Segments for 1024 workgroups
// (2 x 2048 tokens of 4096 channels 358 us, for 512 364, for 2048 367) of 16 tokens at least
// (511 tokens of 512 channels 57 us, of 64 at least 134) and 512 at most (8 x 2048 tokens of
// 16384 channels 4.80 ms, uncut 4.96).
struct BwdPlan {
    int64_t gtiles, seg_len, segs, parts;
    int64_t state, rev, delta, check, turned, bc, a, dd, end;
};

BwdPlan bwd_plan(int64_t T, int64_t B, int64_t D, int64_t N, int64_t G) {
    BwdPlan p{};
    p.gtiles = ceil_div(D / G, scan_grad_channels(static_cast<int>(N)));
    if (B == 0) return p;  // no row: the weights' gradients are zeros
    const int64_t want = std::max<int64_t>(1, 1024 / (G * p.gtiles));
    const int64_t len = std::min<int64_t>(512, std::max<int64_t>(16, round_up(ceil_div(T, want), 16)));
    p.seg_len = len < T ? len : 0;
    p.segs = p.seg_len ? T / len + B : B;
    p.parts = T / kScanPart + B;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t here = at;
        at += round_up(n, 64);
        return here;
    };
    if (p.seg_len) {
        p.state = take(p.segs * D * N);
        p.rev = take(p.segs * D * N);
        p.delta = take(p.segs * D);
    }
    p.check = take(p.parts * (D * N + D));
    p.turned = take(p.parts * G * 2 * N * kScanPart);
    p.bc = take(p.gtiles * T * G * 2 * N);
    p.a = take(p.segs * D * N);
    p.dd = take(p.segs * 2 * D);
    p.end = at;
    return p;
}

// A pool and the rows' slots in it.
int check_pool(const char* fn, const ScanDims& d, const gdr_tensor* state,
               const gdr_tensor* slots) {
    const int rc = check_scan_state(fn, "state", state, -1, d, true);
    if (rc) return rc;
    if (present(slots)) return check_index_vec(fn, "slot_idx", slots, d.B);
    if (state->shape[0] < d.B)
        return fail(GDR_ERR_INVALID_ARG, "%s: state has fewer slots than rows", fn);
    return GDR_OK;
}

int check_states(const char* fn, const ScanDims& d, const gdr_tensor* initial,
                 const gdr_tensor* final_, const gdr_tensor* state, const gdr_tensor* slots) {
    int rc;
    if (present(state)) {
        if (present(initial) || present(final_))
            return fail(GDR_ERR_INVALID_ARG, "%s: give state, or initial_state and final_state", fn);
        return check_pool(fn, d, state, slots);
    }
    if (present(slots)) return fail(GDR_ERR_INVALID_ARG, "%s: slot_idx needs state", fn);
    if (present(initial) && (rc = check_scan_state(fn, "initial_state", initial, d.B, d, false)))
        return rc;
    if (present(final_) && (rc = check_scan_state(fn, "final_state", final_, d.B, d, true)))
        return rc;
    if (present(initial) && present(final_) && initial->dtype != final_->dtype)
        return fail(GDR_ERR_UNSUPPORTED, "%s: final_state must have initial_state's dtype", fn);
    if (present(initial) && present(final_) && !empty(final_) && initial->data == final_->data)
        return fail(GDR_ERR_INVALID_ARG, "%s: final_state must not alias initial_state", fn);
    return GDR_OK;
}

void set_states(ScanParams& p, const gdr_tensor* initial, const gdr_tensor* final_,
                const gdr_tensor* state) {
    const gdr_tensor* in = present(state) ? state : initial;
    const gdr_tensor* last = present(state) ? state : final_;
    p.in = state_of(in);
    if (present(last)) {
        p.last = last->data;
        p.last_outer = last->stride[0];
        p.in.bf16 = last->dtype == GDR_DTYPE_BF16;
    }
}

IndexCheck index_check(const ScanDims& d, const gdr_tensor* off, const gdr_tensor* state,
                       const gdr_tensor* slots) {
    IndexCheck ic;
    ic.offsets = off;
    ic.total_tokens = d.T;
    if (present(state) && present(slots)) {
        ic.slots = slots;
        ic.num_slots = state->shape[0];
    }
    return ic;
}

// Tokens of a run of the Conv1d's gradient: enough runs to fill the chip, few
// enough that their parts of the weights' gradient stay small beside the inputs.  For 2048
// runs of 256 channels (4096 tokens of 8192 channels 51 us, for 1024 or 4096 56), of 16 tokens
// at least (700 of 4096 channels 20.6 us, of 32 22.9) and 128 at most (32768 of 8192 channels
// 346 us, of 512 381).
int64_t conv_run(int64_t T, int64_t C) {
    const int64_t run = ceil_div(T * ceil_div(C, 256), 2048);
    return std::min<int64_t>(128, std::max<int64_t>(16, round_up(run, 4)));
}

struct DraftPlan {
    int64_t span, splits;
};

// Slices of a vocabulary row: a multiple of 2048 values each, 256 of them at most (the
// threads that go through them), enough of them to fill the chip: 2048 in all (256 rows of
// 50021 values 23.8 us, 1024 26.5, 4096 23.3; 64 rows greedily 38.4, 39.3 and 38.2).
DraftPlan draft_plan(int64_t jobs, int64_t V) {
    const int64_t want = std::min<int64_t>(256, std::max<int64_t>(1, 2048 / std::max<int64_t>(1, jobs)));
    DraftPlan p{};
    p.span = std::max<int64_t>(2048, round_up(ceil_div(V, want), 2048));
    p.splits = std::max<int64_t>(1, ceil_div(V, p.span));
    return p;
}

}  // namespace

extern "C" {

int64_t gdr_selective_scan_workspace(int64_t tokens, int64_t rows, int64_t channels,
                                     int32_t state_size, int32_t groups, int backward) {
    if (tokens < 0 || rows < 0 || channels < 1 || state_size < 1 || groups < 1 ||
        channels % groups != 0)
        return -1;
    if (backward) return bwd_plan(tokens, rows, channels, state_size, groups).end;
    return rows ? fwd_plan(tokens, rows, channels, state_size, groups).end : 0;
}

int gdr_selective_scan_fwd(const gdr_tensor* out, const gdr_tensor* x, const gdr_tensor* dt,
                           const gdr_tensor* A, const gdr_tensor* Bm, const gdr_tensor* Cm,
                           const gdr_tensor* D, const gdr_tensor* z, const gdr_tensor* dt_bias,
                           const gdr_tensor* input_row_offsets, const gdr_tensor* initial_state,
                           const gdr_tensor* final_state, const gdr_tensor* state,
                           const gdr_tensor* slot_idx, uint32_t flags,
                           const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_selective_scan_fwd";
    ScanDims d{};
    int rc;
    if ((rc = check_scan(fn, x, dt, A, Bm, dt_bias, flags,
                         GDR_FLAG_DT_SOFTPLUS | GDR_FLAG_KEEP_STATE, d)) ||
        (rc = check_groups(fn, "C", Cm, d, false)) || (rc = check_rows(fn, "out", out, d, true)) ||
        (present(D) && (rc = check_channels(fn, "D", D, d.D))) ||
        (present(z) && (rc = check_rows(fn, "z", z, d, false))) ||
        (rc = check_offsets(fn, input_row_offsets, d.B)) ||
        (rc = no_alias(fn, out, "out", {x, dt, Bm, Cm, z})) ||
        (rc = check_states(fn, d, initial_state, final_state, state, slot_idx)))
        return rc;
    if ((flags & GDR_FLAG_KEEP_STATE) && !present(state))
        return fail(GDR_ERR_INVALID_ARG, "%s: GDR_FLAG_KEEP_STATE needs state", fn);
    if (d.B == 0) return done();
    const FwdPlan pl = fwd_plan(d.T, d.B, d.D, d.N, d.G);
    if ((rc = check_workspace(fn, workspace, pl.end))) return rc;
    ScanParams p = scan_params(d, x, dt, A, Bm, dt_bias, input_row_offsets, slot_idx, flags);
    p.z = rows_of(z);
    p.c = heads_of(Cm);
    p.skip = floats(D);
    p.out = out->data;
    p.o_tok = rows_of(out).tok;
    set_states(p, initial_state, final_state, state);
    p.narrow_most = static_cast<int32_t>(pl.narrow);
    p.hand_on = present(final_state);  // also of rows without tokens
    p.lane_most = static_cast<int32_t>(pl.lane);
    p.seg_skip = p.lane_most;
    p.seg_len = static_cast<int32_t>(pl.seg_len);
    p.segs = static_cast<int32_t>(pl.segs);
    if (pl.seg_len) {
        p.seg_state = static_cast<float*>(workspace->data);
        p.seg_delta = p.seg_state + pl.delta;
    }
    if ((rc = check_grid(fn, narrow_blocks(d, p.in.bf16), kScanNarrowThreads)) ||
        (pl.lane > pl.narrow &&
         (rc = check_grid(fn, d.B * ceil_div(d.D, kScanLaneChannels), kScanThreads))) ||
        (pl.wide && (rc = check_grid(fn, ceil_div(pl.segs * d.G * d.tiles(), 4), kScanThreads))) ||
        (pl.seg_len && (rc = check_grid(fn, d.B * ceil_div(d.D * d.N, 256), 256))) ||
        (rc = run_debug_check(fn, d.B, index_check(d, input_row_offsets, state, slot_idx), stream)))
        return rc;
    if (d.T == 0 && (present(state) || !present(final_state))) return done();
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool b16 = d.work == GDR_DTYPE_BF16;
    hipError_t e = hipSuccess;
    if (pl.narrow || p.hand_on) e = launch_scan_narrow(p, b16, s);
    if (e == hipSuccess && pl.lane > pl.narrow) e = launch_scan_lanes(p, b16, s);
    if (e == hipSuccess && pl.seg_len) {
        e = launch_scan_wide(p, b16, true, s);
        if (e == hipSuccess) e = launch_scan_chain(p, s);
    }
    if (e == hipSuccess && pl.wide) e = launch_scan_wide(p, b16, false, s);
    return hip_status(fn, e);
}

int gdr_selective_scan_step(const gdr_tensor* out, const gdr_tensor* x, const gdr_tensor* dt,
                            const gdr_tensor* A, const gdr_tensor* Bm, const gdr_tensor* Cm,
                            const gdr_tensor* D, const gdr_tensor* z, const gdr_tensor* dt_bias,
                            const gdr_tensor* state, const gdr_tensor* slot_idx, uint32_t flags,
                            void* stream) {
    const char* fn = "gdr_selective_scan_step";
    ScanDims d{};
    int rc;
    if ((rc = check_scan(fn, x, dt, A, Bm, dt_bias, flags, GDR_FLAG_DT_SOFTPLUS, d)) ||
        (rc = check_groups(fn, "C", Cm, d, false)) || (rc = check_rows(fn, "out", out, d, true)) ||
        (present(D) && (rc = check_channels(fn, "D", D, d.D))) ||
        (present(z) && (rc = check_rows(fn, "z", z, d, false))) ||
        (rc = no_alias(fn, out, "out", {x, dt, Bm, Cm, z})))
        return rc;
    d.B = d.T;
    if ((rc = check_pool(fn, d, state, slot_idx))) return rc;
    if (d.B == 0) return done();
    ScanParams p = scan_params(d, x, dt, A, Bm, dt_bias, nullptr, slot_idx, flags);
    p.z = rows_of(z);
    p.c = heads_of(Cm);
    p.skip = floats(D);
    p.out = out->data;
    p.o_tok = rows_of(out).tok;
    set_states(p, nullptr, nullptr, state);
    if ((rc = check_grid(fn, narrow_blocks(d, p.in.bf16), kScanNarrowThreads)) ||
        (rc = run_debug_check(fn, d.B, index_check(d, nullptr, state, slot_idx), stream)))
        return rc;
    return hip_status(fn, launch_scan_narrow(p, d.work == GDR_DTYPE_BF16,
                                             static_cast<hipStream_t>(stream)));
}

int gdr_selective_scan_fold(const gdr_tensor* state, const gdr_tensor* x, const gdr_tensor* dt,
                            const gdr_tensor* A, const gdr_tensor* Bm, const gdr_tensor* dt_bias,
                            const gdr_tensor* input_row_offsets, const gdr_tensor* accepted,
                            const gdr_tensor* slot_idx, uint32_t flags, void* stream) {
    const char* fn = "gdr_selective_scan_fold";
    ScanDims d{};
    int rc;
    if ((rc = check_scan(fn, x, dt, A, Bm, dt_bias, flags, GDR_FLAG_DT_SOFTPLUS, d)) ||
        (rc = check_offsets(fn, input_row_offsets, d.B)) ||
        (rc = check_index_vec(fn, "accepted", accepted, d.B)))
        return rc;
    if ((rc = check_pool(fn, d, state, slot_idx))) return rc;
    if (d.B == 0 || d.T == 0) return done();
    ScanParams p = scan_params(d, x, dt, A, Bm, dt_bias, input_row_offsets, slot_idx, flags);
    p.accepted = as_u32(accepted);
    p.narrow_most = INT32_MAX;
    set_states(p, nullptr, nullptr, state);
    if ((rc = check_grid(fn, narrow_blocks(d, p.in.bf16), kScanNarrowThreads)) ||
        (rc = run_debug_check(fn, d.B, index_check(d, input_row_offsets, state, slot_idx), stream)))
        return rc;
    return hip_status(fn, launch_scan_narrow(p, d.work == GDR_DTYPE_BF16,
                                             static_cast<hipStream_t>(stream)));
}

int gdr_selective_scan_bwd(const gdr_tensor* dout, const gdr_tensor* x, const gdr_tensor* dt,
                           const gdr_tensor* A, const gdr_tensor* Bm, const gdr_tensor* Cm,
                           const gdr_tensor* D, const gdr_tensor* z, const gdr_tensor* dt_bias,
                           const gdr_tensor* input_row_offsets, const gdr_tensor* initial_state,
                           const gdr_tensor* dfinal_state, const gdr_tensor* dx,
                           const gdr_tensor* ddt, const gdr_tensor* dA, const gdr_tensor* dB,
                           const gdr_tensor* dC, const gdr_tensor* dD, const gdr_tensor* dz,
                           const gdr_tensor* ddt_bias, const gdr_tensor* dinitial_state,
                           uint32_t flags, const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_selective_scan_bwd";
    ScanDims d{};
    int rc;
    if ((rc = check_scan(fn, x, dt, A, Bm, dt_bias, flags, GDR_FLAG_DT_SOFTPLUS, d)) ||
        (rc = check_groups(fn, "C", Cm, d, false)) || (rc = check_rows(fn, "dout", dout, d, false)) ||
        (present(D) && (rc = check_channels(fn, "D", D, d.D))) ||
        (present(z) && (rc = check_rows(fn, "z", z, d, false))) ||
        (rc = check_offsets(fn, input_row_offsets, d.B)) ||
        (present(initial_state) &&
         (rc = check_scan_state(fn, "initial_state", initial_state, d.B, d, false))) ||
        (present(dfinal_state) &&
         (rc = check_scan_state(fn, "dfinal_state", dfinal_state, d.B, d, false))) ||
        (rc = check_rows(fn, "dx", dx, d, true)) || (rc = check_rows(fn, "ddt", ddt, d, true)) ||
        (rc = check_decay(fn, "dA", dA, d)) || (rc = check_groups(fn, "dB", dB, d, true)) ||
        (rc = check_groups(fn, "dC", dC, d, true)) ||
        (present(dinitial_state) &&
         (rc = check_scan_state(fn, "dinitial_state", dinitial_state, d.B, d, true))))
        return rc;
    const struct { const gdr_tensor *in, *grad; const char* name; } pairs[] = {
        {D, dD, "dD"}, {z, dz, "dz"}, {dt_bias, ddt_bias, "ddt_bias"}};
    for (const auto& q : pairs)
        if (present(q.in) != present(q.grad) && !(q.in && empty(q.in)))
            return fail(GDR_ERR_INVALID_ARG, "%s: %s is given exactly when its input is", fn, q.name);
    if ((present(dz) && (rc = check_rows(fn, "dz", dz, d, true))) ||
        (present(dD) && (rc = check_channels(fn, "dD", dD, d.D))) ||
        (present(ddt_bias) && (rc = check_channels(fn, "ddt_bias", ddt_bias, d.D))))
        return rc;
    const gdr_tensor* outs[] = {dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state};
    const char* names[] = {"dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial_state"};
    for (int i = 0; i < 9; ++i) {
        if (!present(outs[i])) continue;
        if ((rc = no_alias(fn, outs[i], names[i], {dout, x, dt, A, Bm, Cm, D, z, dt_bias,
                                                   initial_state, dfinal_state})))
            return rc;
        for (int j = 0; j < i; ++j)
            if (present(outs[j]) && !empty(outs[j]) && outs[j]->data == outs[i]->data)
                return fail(GDR_ERR_INVALID_ARG, "%s: %s and %s share memory", fn, names[j], names[i]);
    }
    const BwdPlan pl = bwd_plan(d.T, d.B, d.D, d.N, d.G);
    if ((rc = check_workspace(fn, workspace, pl.end))) return rc;
    ScanParams p = scan_params(d, x, dt, A, Bm, dt_bias, input_row_offsets, nullptr, flags);
    p.z = rows_of(z);
    p.c = heads_of(Cm);
    p.skip = floats(D);
    p.in = state_of(initial_state);
    p.seg_skip = -1;  // rows without tokens too: they hand on the state's gradient
    p.seg_len = static_cast<int32_t>(pl.seg_len);
    p.segs = static_cast<int32_t>(pl.segs);
    float* ws = present(workspace) ? static_cast<float*>(workspace->data) : nullptr;
    ScanGrad g{};
    if (pl.seg_len) {
        p.seg_state = ws + pl.state;
        p.seg_delta = ws + pl.delta;
        g.seg_rev = ws + pl.rev;
    }
    g.d_o = rows_of(dout);
    g.dx = rows_of(dx);
    g.ddt = rows_of(ddt);
    g.dz = rows_of(dz);
    g.db = heads_of(dB);
    g.dc = heads_of(dC);
    g.dA = static_cast<float*>(dA->data);
    g.dskip = present(dD) ? static_cast<float*>(dD->data) : nullptr;
    g.dbias = present(ddt_bias) ? static_cast<float*>(ddt_bias->data) : nullptr;
    g.dfinal = state_of(dfinal_state);
    if (present(dinitial_state)) {
        g.dinit = dinitial_state->data;
        g.dinit_outer = dinitial_state->stride[0];
        g.dinit_bf16 = dinitial_state->dtype == GDR_DTYPE_BF16;
    }
    g.tiles = static_cast<int32_t>(pl.gtiles);
    g.check = ws + pl.check;
    g.turned = ws + pl.turned;
    g.part_bc = ws + pl.bc;
    g.part_a = ws + pl.a;
    g.part_d = ws + pl.dd;
    const int64_t threads = scan_grad_channels(static_cast<int>(d.N));
    const int64_t DN = d.D * d.N;
    if ((rc = check_grid(fn, ceil_div(pl.segs * d.G * ((d.N > 16 ? d.N / 16 : 1) * d.tiles() + 1), 4),
                         kScanThreads)) ||
        (rc = check_grid(fn, 2 * d.B * ceil_div(DN, 256), 256)) ||
        (rc = check_grid(fn, pl.segs * d.G * pl.gtiles, threads)) ||
        (rc = check_grid(fn, ceil_div(d.T * d.G * 2 * d.N, 256) + ceil_div(DN, 256) +
                                 ceil_div(2 * d.D, 256), 256)) ||
        (rc = run_debug_check(fn, d.B, index_check(d, input_row_offsets, nullptr, nullptr), stream)))
        return rc;
    return hip_status(fn, launch_scan_bwd(p, g, d.work == GDR_DTYPE_BF16,
                                          static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ Conv1d ---

int gdr_causal_conv1d_fold(const gdr_tensor* conv_state, const gdr_tensor* x,
                           const gdr_tensor* input_row_offsets, const gdr_tensor* accepted,
                           const gdr_tensor* slot_idx, void* stream) {
    const char* fn = "gdr_causal_conv1d_fold";
    int rc;
    int64_t B = 0;
    if ((rc = check_tensor(fn, "x", x, 2, nullptr, true, true, false))) return rc;
    const int64_t T = x->shape[0], C = x->shape[1];
    if (C % 4 != 0) return fail(GDR_ERR_UNSUPPORTED, "%s: channels must be a multiple of 4", fn);
    const int64_t shape[3] = {-1, -1, C};
    if ((rc = check_layout(fn, "x", x, 4)) ||
        (rc = check_tensor(fn, "conv_state", conv_state, 3, shape, true, true, false)) ||
        (rc = check_work_dtype(fn, "conv_state", conv_state, x->dtype)) ||
        (rc = check_layout(fn, "conv_state", conv_state, 4)) ||
        (rc = check_distinct(fn, "conv_state", conv_state)) ||
        (rc = check_offsets(fn, input_row_offsets, B)) ||
        (rc = check_index_vec(fn, "accepted", accepted, B)))
        return rc;
    const int64_t H = conv_state->shape[1];
    if (H < 1 || H > 3)
        return fail(GDR_ERR_UNSUPPORTED, "%s: a history of %lld inputs is not built (1, 2, 3)", fn,
                    static_cast<ll>(H));
    if (present(slot_idx)) {
        if ((rc = check_index_vec(fn, "slot_idx", slot_idx, B))) return rc;
    } else if (conv_state->shape[0] < B) {
        return fail(GDR_ERR_INVALID_ARG, "%s: conv_state has fewer slots than rows", fn);
    }
    if (T > kMaxTokens || C > kMaxChannels)
        return fail(GDR_ERR_INVALID_ARG, "%s: too many tokens or channels", fn);
    if (B == 0 || T == 0 || C == 0) return done();
    if ((rc = check_grid(fn, B * ceil_div(C / 4, 256), 256))) return rc;
    ConvFold p{};
    p.B = static_cast<int32_t>(B);
    p.C = static_cast<int32_t>(C);
    p.H = static_cast<int32_t>(H);
    p.offsets = as_u32(input_row_offsets);
    p.slot_idx = as_u32(slot_idx);
    p.accepted = as_u32(accepted);
    p.x = rows_of(x);
    p.state = conv_state->data;
    p.st_slot = conv_state->stride[0];
    p.st_tok = conv_state->stride[1];
    IndexCheck ic;
    ic.offsets = input_row_offsets;
    ic.total_tokens = T;
    if (present(slot_idx)) {
        ic.slots = slot_idx;
        ic.num_slots = conv_state->shape[0];
    }
    if ((rc = run_debug_check(fn, B, ic, stream))) return rc;
    return hip_status(fn, launch_conv_fold(p, x->dtype == GDR_DTYPE_BF16,
                                           static_cast<hipStream_t>(stream)));
}

int64_t gdr_causal_conv1d_workspace(int64_t tokens, int64_t channels, int32_t width) {
    if (tokens < 0 || channels < 0 || width < 1) return -1;
    return ceil_div(tokens, conv_run(tokens, channels)) * (width + 1) * channels;
}

int gdr_causal_conv1d_bwd(const gdr_tensor* dout, const gdr_tensor* x, const gdr_tensor* weight,
                          const gdr_tensor* bias, const gdr_tensor* input_row_offsets,
                          const gdr_tensor* dx, const gdr_tensor* dweight, const gdr_tensor* dbias,
                          uint32_t flags, const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_causal_conv1d_bwd";
    int rc;
    int64_t B = 0;
    if (flags & ~GDR_FLAG_CONV_SILU)
        return fail(GDR_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if ((rc = check_tensor(fn, "x", x, 2, nullptr, true, true, false))) return rc;
    const int64_t T = x->shape[0], C = x->shape[1];
    if (C % 4 != 0) return fail(GDR_ERR_UNSUPPORTED, "%s: channels must be a multiple of 4", fn);
    const struct { const gdr_tensor* t; const char* name; bool out; } rows[] = {
        {x, "x", false}, {dout, "dout", false}, {dx, "dx", true}};
    for (const auto& r : rows)
        if ((rc = check_tensor(fn, r.name, r.t, 2, x->shape, true, true, false)) ||
            (rc = check_work_dtype(fn, r.name, r.t, x->dtype)) ||
            (rc = check_layout(fn, r.name, r.t, 4)) ||
            (r.out && (rc = check_distinct(fn, r.name, r.t))))
            return rc;
    const int64_t wshape[2] = {C, -1};
    if ((rc = check_tensor(fn, "weight", weight, 2, wshape, true, false, false))) return rc;
    const int64_t W = weight->shape[1], dwshape[2] = {C, W};
    if (W < 2 || W > 4)
        return fail(GDR_ERR_UNSUPPORTED, "%s: kernel width %lld not built (2, 3, 4)", fn,
                    static_cast<ll>(W));
    if ((rc = check_tensor(fn, "dweight", dweight, 2, dwshape, true, false, false)) ||
        (rc = check_distinct(fn, "dweight", dweight)))
        return rc;
    if ((weight->stride[1] != 1 && !empty(weight)) || (dweight->stride[1] != 1 && !empty(dweight)))
        return fail(GDR_ERR_UNSUPPORTED, "%s: weight and dweight need unit stride over the taps", fn);
    if ((present(bias) && (rc = check_channels(fn, "bias", bias, C))) ||
        (present(dbias) && (rc = check_channels(fn, "dbias", dbias, C))))
        return rc;
    if (present(dbias) && !present(bias))
        return fail(GDR_ERR_INVALID_ARG, "%s: dbias needs bias", fn);
    if ((rc = check_offsets(fn, input_row_offsets, B)) ||
        (rc = no_alias(fn, dx, "dx", {x, dout})) ||
        (rc = no_alias(fn, dweight, "dweight", {weight, dx})) ||
        (present(dbias) && (rc = no_alias(fn, dbias, "dbias", {bias, dx, dweight}))))
        return rc;
    if (T > kMaxTokens || C > kMaxChannels)
        return fail(GDR_ERR_INVALID_ARG, "%s: too many tokens or channels", fn);
    const int64_t need = gdr_causal_conv1d_workspace(T, C, static_cast<int32_t>(W));
    if ((rc = check_workspace(fn, workspace, need))) return rc;
    if (C == 0) return done();
    ConvGrad p{};
    p.B = static_cast<int32_t>(B);
    p.T = static_cast<int32_t>(T);
    p.C = static_cast<int32_t>(C);
    p.W = static_cast<int32_t>(W);
    p.silu = (flags & GDR_FLAG_CONV_SILU) != 0;
    p.offsets = as_u32(input_row_offsets);
    p.d_o = rows_of(dout);
    p.x = rows_of(x);
    p.dx = rows_of(dx);
    p.weight = static_cast<const float*>(weight->data);
    p.w_chan = weight->stride[0];
    p.bias = floats(bias);
    p.dweight = static_cast<float*>(dweight->data);
    p.dw_chan = dweight->stride[0];
    p.dbias = present(dbias) ? static_cast<float*>(dbias->data) : nullptr;
    p.run = static_cast<int32_t>(conv_run(T, C));
    p.runs = static_cast<int32_t>(ceil_div(T, p.run));
    p.part = present(workspace) ? static_cast<float*>(workspace->data) : nullptr;
    IndexCheck ic;
    ic.offsets = input_row_offsets;
    ic.total_tokens = T;
    if ((rc = check_grid(fn, ceil_div(p.runs * ceil_div(C / 4, 64), 4), kScanThreads)) ||
        (rc = check_grid(fn, ceil_div((W + 1) * C, 256), 256)) ||
        (rc = run_debug_check(fn, B, ic, stream)))
        return rc;
    return hip_status(fn, launch_conv_bwd(p, x->dtype == GDR_DTYPE_BF16,
                                          static_cast<hipStream_t>(stream)));
}

// ----------------------------------------------------------- drafted tokens ---

int64_t gdr_verify_drafts_workspace(int64_t tokens, int64_t rows, int64_t vocab) {
    if (tokens < 0 || rows < 0 || vocab < 1) return -1;
    return std::max(4 * rows * draft_plan(rows, vocab).splits,
                    2 * tokens * draft_plan(tokens, vocab).splits);
}

int gdr_verify_drafts(const gdr_tensor* accepted, const gdr_tensor* next_token,
                      const gdr_tensor* tokens, const gdr_tensor* target, const gdr_tensor* draft,
                      const gdr_tensor* uniform, const gdr_tensor* input_row_offsets,
                      const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_verify_drafts";
    int rc;
    int64_t B = 0;
    if ((rc = check_tensor(fn, "target", target, 2, nullptr, true, true, false))) return rc;
    const int64_t T = target->shape[0], V = target->shape[1];
    if (V < 1 || V > kMaxTokens)
        return fail(GDR_ERR_INVALID_ARG, "%s: a vocabulary of %lld", fn, static_cast<ll>(V));
    if (T > kMaxTokens) return fail(GDR_ERR_INVALID_ARG, "%s: too many tokens", fn);
    if (!empty(target) && V > 1 && target->stride[1] != 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: target must have unit innermost stride", fn);
    if (present(draft)) {
        if ((rc = check_tensor(fn, "draft", draft, 2, target->shape, true, true, false)) ||
            (rc = check_work_dtype(fn, "draft", draft, target->dtype)))
            return rc;
        if (!empty(draft) && V > 1 && draft->stride[1] != 1)
            return fail(GDR_ERR_UNSUPPORTED, "%s: draft must have unit innermost stride", fn);
        if (!present(uniform) && T > 0)
            return fail(GDR_ERR_INVALID_ARG, "%s: draft needs uniform", fn);
    }
    const int64_t tshape[1] = {T};
    if ((rc = check_index_vec(fn, "tokens", tokens, T)) ||
        (present(uniform) && (rc = check_tensor(fn, "uniform", uniform, 1, tshape, true, false, false))) ||
        (rc = check_offsets(fn, input_row_offsets, B)) ||
        (rc = check_index_vec(fn, "accepted", accepted, B)) ||
        (rc = check_index_vec(fn, "next_token", next_token, B)) ||
        (rc = no_alias(fn, accepted, "accepted", {tokens, input_row_offsets, next_token})) ||
        (rc = no_alias(fn, next_token, "next_token", {tokens, input_row_offsets})) ||
        (rc = check_workspace(fn, workspace, gdr_verify_drafts_workspace(T, B, V))))
        return rc;
    if (B == 0) return done();
    DraftParams p{};
    p.B = static_cast<int32_t>(B);
    p.T = static_cast<int32_t>(T);
    p.V = static_cast<int32_t>(V);
    const bool sampled = present(uniform);
    const DraftPlan pl = draft_plan(sampled ? B : T, V);
    p.span = static_cast<int32_t>(pl.span);
    p.splits = static_cast<int32_t>(pl.splits);
    p.offsets = as_u32(input_row_offsets);
    p.tokens = static_cast<const int32_t*>(tokens->data);
    p.tok_stride = 1;
    p.p = target->data;
    p.p_tok = T > 1 ? target->stride[0] : 0;
    p.q = present(draft) ? draft->data : nullptr;
    p.q_tok = present(draft) && T > 1 ? draft->stride[0] : 0;
    p.bf16 = target->dtype == GDR_DTYPE_BF16;
    p.u = floats(uniform);
    p.u_stride = sampled && T > 1 ? uniform->stride[0] : 0;
    p.accepted = static_cast<int32_t*>(accepted->data);
    p.next = static_cast<int32_t*>(next_token->data);
    p.part = present(workspace) ? static_cast<double*>(workspace->data) : nullptr;
    IndexCheck ic;
    ic.offsets = input_row_offsets;
    ic.total_tokens = T;
    if ((rc = check_grid(fn, std::max(B, T) * pl.splits, 256)) ||
        (rc = run_debug_check(fn, B, ic, stream)))
        return rc;
    return hip_status(fn, launch_drafts(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// Host side of the linear-attention and block-norm entry points declared in
// include/gdr.h: argument validation, workspace layout, launch choice.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <initializer_list>

#include "gdr_host.h"
#include "gdr_linattn.h"
#include "gdr_norm.h"

using namespace gdr;

namespace {

typedef long long ll;

constexpr int64_t kLaMaxTokenStride = (int64_t{1} << 24) - 1;

// [tokens, heads, dim] operand: unit innermost stride, 16-byte rows.  `walked`:
// the walks read it, which address a chunk's tokens from one 64-bit base by
// unsigned 32-bit offsets.
int check_heads(const char* fn, const char* name, const gdr_tensor* t, int64_t T, int64_t heads,
                int64_t dim, int32_t work, bool walked) {
    const int64_t shape[3] = {T, heads, dim};
    int rc = check_tensor(fn, name, t, 3, shape, true, true, false);
    if (rc || (rc = check_work_dtype(fn, name, t, work))) return rc;
    if ((rc = check_layout(fn, name, t, vec_mult(work)))) return rc;
    if (T > 1 && heads > 0 && walked && t->stride[0] < 0)
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s has a negative token stride", fn, name);
    if (T > 1 && heads > 0 && std::llabs(t->stride[0]) > kLaMaxTokenStride)
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s has a token stride above %lld elements", fn, name,
                    static_cast<ll>(kLaMaxTokenStride));
    return GDR_OK;
}

// Outputs are written by many workgroups: no two elements may share memory.
int check_distinct(const char* fn, const char* name, const gdr_tensor* t) {
    if (empty(t)) return GDR_OK;
    int64_t need = 1;                     // sorted by stride, each covers the ones before
    bool used[GDR_MAX_DIMS] = {};
    for (int k = 0; k < t->ndim; ++k) {
        int at = -1;
        for (int i = 0; i < t->ndim; ++i)
            if (!used[i] && (at < 0 || t->stride[i] < t->stride[at] ||
                             (t->stride[i] == t->stride[at] && t->shape[i] < t->shape[at])))
                at = i;
        used[at] = true;
        if (t->shape[at] == 1) continue;
        if (t->stride[at] < need)
            return fail(GDR_ERR_INVALID_ARG, "%s: %s is an output whose elements overlap", fn,
                        name);
        need = t->stride[at] * (t->shape[at] - 1) + need;
    }
    return GDR_OK;
}

int check_out_heads(const char* fn, const char* name, const gdr_tensor* t, int64_t T,
                    int64_t heads, int64_t dim, int32_t work) {
    int rc = check_heads(fn, name, t, T, heads, dim, work, false);
    return rc ? rc : check_distinct(fn, name, t);
}

// States [N, heads, K, V] with a dense K x V block per head.
int check_la_state(const char* fn, const char* name, const gdr_tensor* t, int64_t N, int64_t nv,
                   int64_t K, int64_t V, bool out) {
    const int64_t shape[4] = {N, nv, K, V};
    int rc = check_tensor(fn, name, t, 4, shape, true, true, false);
    if (rc) return rc;
    if (!empty(t) && (t->stride[3] != 1 || t->stride[2] != V))
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s needs a dense K x V block per head", fn, name);
    if ((rc = check_layout(fn, name, t, vec_mult(t->dtype)))) return rc;
    return out ? check_distinct(fn, name, t) : GDR_OK;
}

LaTensor la_tensor(const gdr_tensor* t, int64_t div) {
    LaTensor r{};
    r.p = t->data;
    r.tok = t->shape[0] > 1 ? t->stride[0] : 0;  // a single token's stride can be anything
    r.head = t->stride[1];
    r.div = static_cast<int32_t>(div);
    return r;
}

// Dense states by slot or row; `flip`: the walk's state is the transpose.
LaState la_state(const gdr_tensor* t, int64_t V, bool flip, float mult) {
    LaState s{};
    if (!present(t)) return s;
    s.p = t->data;
    s.outer = t->stride[0];
    s.head = t->stride[1];
    s.sk = flip ? 1 : static_cast<int32_t>(V);
    s.sz = flip ? static_cast<int32_t>(V) : 1;
    s.bf16 = t->dtype == GDR_DTYPE_BF16;
    s.mult = mult;
    return s;
}

LaState la_segment_state(float* p, int64_t nv, int64_t K, int64_t V, bool flip) {
    LaState s{};
    s.p = p;
    s.outer = nv * K * V;
    s.head = K * V;
    s.sk = flip ? 1 : static_cast<int32_t>(V);
    s.sz = flip ? static_cast<int32_t>(V) : 1;
    s.by_segment = 1;
    s.mult = 1.0f;
    return s;
}

constexpr int64_t kLaUncut = 192;         // tokens of a call up to which no row is cut,
constexpr int64_t kLaUncutMany = 1024;    // and of a forward with rows enough to fill the chip
constexpr int64_t kLaSumTokens = 512;     // longest segment of a gradient

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a call is cut into segments and what its workspace holds (float32
// elements; every part starts at a multiple of 64).
struct LaPlan {
    int64_t seg_len, segs;
    int64_t cuts, cut_rows;               // segments that have states of their own; their rows
    int64_t q_tiles, v_tiles;             // workgroups over K (dq, dk) and over V (fwd, dv)
    int64_t s_fwd, s_rev, tot, rq, rk, phi, phi0, pq, pk, end;
};

LaPlan la_plan(int64_t T, int64_t B, int64_t nk, int64_t nv, int64_t K, int64_t V, bool backward) {
    LaPlan p{};
    const int64_t q_waves = la_waves(static_cast<int>(K));
    p.v_tiles = ceil_div(V, 16 * la_waves(static_cast<int>(V)));
    p.q_tiles = ceil_div(K, 16 * q_waves);
    // Rows are walked chunk by chunk, so few (row, head) pairs leave most of the
    // 256 compute units idle: rows are cut into segments, whose own sums a first
    // pass takes and a scan turns into states, until about two workgroups a unit
    // are walking (64 segments at most, as the scan goes through a row's in turn; a
    // gradient's are 512 tokens long at most, however many that makes).
    // Measured at 16 value heads, K = V = 128, us uncut and in segments of 64
    // tokens: bf16 forward of 200 tokens 24 and 26, of 300 (by 256) 38 and 27,
    // float32 46 and 35, 82 and 37; the two more launches cost up to 5 us where
    // they gain nothing.
    const int64_t per_seg = nv * (backward ? p.v_tiles + 2 * p.q_tiles : p.v_tiles);
    const int64_t want = std::min<int64_t>(64, ceil_div(512, per_seg));
    p.segs = B;
    int64_t len = T;
    // With rows enough only those are cut that are longer than their share, so that
    // none walks on alone.  32 heads, K = V = 128, us uncut and cut: 32768 tokens beside
    // 255 single ones bf16 2612 and 623, 16 rows of 64 to 2048 tokens 195 and 204, in
    // float32 571 and 523, 64 rows of 16 to 1024 271 and 261, 766 and 639; 16 equal
    // rows of 512, none of them cut, 80 and 90.
    if (B < want ? T > kLaUncut : !backward && T > kLaUncutMany) {
        const int64_t full = B < want ? want - B / 2 : want;  // rows end in part segments
        len = std::max<int64_t>(64, ceil_div(ceil_div(T, full), 64) * 64);
    }
    // the decays' gradient is summed over a segment, with errors as its root
    if (backward) len = std::min(len, kLaSumTokens);
    if (len < T) {
        p.seg_len = len;
        p.segs = T / len + B;
        p.cut_rows = backward ? B : std::min(B, T / (len + 1));
        p.cuts = backward ? p.segs : T / len + p.cut_rows;
    }
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t here = at;
        at += ceil_div(n, 64) * 64;
        return here;
    };
    if (p.seg_len) {
        p.s_fwd = take(p.cuts * nv * K * V);
        if (backward) p.s_rev = take(p.cuts * nv * K * V);
        p.tot = take(2 * p.cuts * nv);
    }
    if (backward) {
        p.rq = take(p.q_tiles * q_waves * nv * T);
        p.rk = take(p.q_tiles * q_waves * nv * T);
        p.phi = take(p.segs * nv * p.q_tiles * q_waves);
        p.phi0 = take(p.segs * nv * p.v_tiles * la_waves(static_cast<int>(V)));
        if (nv != nk) {
            p.pq = take(T * nv * K);
            p.pk = take(T * nv * K);
        }
    }
    p.end = at;
    return p;
}

int check_workspace(const char* fn, const gdr_tensor* ws, int64_t need) {
    if (need == 0) return GDR_OK;
    if (!present(ws))
        return fail(GDR_ERR_INVALID_ARG, "%s: workspace is null (%lld floats needed, see "
                    "gdr_linear_attention_workspace and gdr_block_norm_workspace)", fn,
                    static_cast<ll>(need));
    if (ws->ndim != 1 || ws->dtype != GDR_DTYPE_F32)
        return fail(GDR_ERR_INVALID_ARG, "%s: workspace must be a float32 vector", fn);
    if (ws->shape[0] < need)
        return fail(GDR_ERR_INVALID_ARG, "%s: workspace has %lld floats, %lld needed", fn,
                    static_cast<ll>(ws->shape[0]), static_cast<ll>(need));
    if (ws->shape[0] > 1 && ws->stride[0] != 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: workspace must be contiguous", fn);
    if (!aligned16(ws->data))
        return fail(GDR_ERR_UNSUPPORTED, "%s: workspace base must be 16-byte aligned", fn);
    return GDR_OK;
}

// The sizes that the linear-attention entries share, from q, k, v, g.
struct LaDims {
    int64_t T, nk, nv, K, V, B;
    int32_t work;
};

int check_la(const char* fn, const gdr_tensor* q, const gdr_tensor* k, const gdr_tensor* v,
             const gdr_tensor* g, bool walked, LaDims& d) {
    int rc = check_tensor(fn, "q", q, 3, nullptr, true, true, false);
    if (rc || (rc = check_tensor(fn, "v", v, 3, nullptr, true, true, false))) return rc;
    d.T = q->shape[0];
    d.nk = q->shape[1];
    d.K = q->shape[2];
    d.nv = v->shape[1];
    d.V = v->shape[2];
    d.work = q->dtype;
    if (d.nk < 1 || d.nv < d.nk || d.nv % d.nk != 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: v's heads (%lld) must be a positive multiple of q's "
                    "(%lld)", fn, static_cast<ll>(d.nv), static_cast<ll>(d.nk));
    if (d.K < 8 || d.V < 8 || d.K % 8 || d.V % 8 || d.K > GDR_MAX_HEAD_DIM ||
        d.V > GDR_MAX_HEAD_DIM)
        return fail(GDR_ERR_UNSUPPORTED, "%s: head dims K=%lld V=%lld (multiples of 8 up to %d)",
                    fn, static_cast<ll>(d.K), static_cast<ll>(d.V), GDR_MAX_HEAD_DIM);
    if ((rc = check_heads(fn, "q", q, d.T, d.nk, d.K, d.work, walked)) ||
        (rc = check_heads(fn, "k", k, d.T, d.nk, d.K, d.work, walked)) ||
        (rc = check_heads(fn, "v", v, d.T, d.nv, d.V, d.work, walked)))
        return rc;
    const int64_t gs[2] = {d.T, d.nv};
    if (present(g) && (rc = check_tensor(fn, "g", g, 2, gs, true, true, false))) return rc;
    if (d.T > INT32_MAX - 65536 || d.nv > 65535)
        return fail(GDR_ERR_INVALID_ARG, "%s: too many tokens or heads", fn);
    return GDR_OK;
}

int check_offsets(const char* fn, const gdr_tensor* off, LaDims& d) {
    int rc = check_tensor(fn, "input_row_offsets", off, 1, nullptr, false, false, true);
    if (rc) return rc;
    d.B = off->shape[0] - 1;
    if (d.B < 0) return fail(GDR_ERR_INVALID_ARG, "%s: input_row_offsets is empty", fn);
    return check_index_vec(fn, "input_row_offsets", off, d.B + 1);
}

// A launch holds fewer than 2^32 threads in a dimension.  Every launch of a call is
// checked before the first, which may already change states.
int check_grid(const char* fn, int64_t blocks, int64_t threads) {
    if (blocks > UINT32_MAX / threads)
        return fail(GDR_ERR_INVALID_ARG, "%s: batch too large for one launch", fn);
    return GDR_OK;
}

int check_scan(const char* fn, const LaDims& d, int64_t rows) {
    return check_grid(fn, la_scan_blocks(static_cast<int>(d.K * d.V)) * rows * d.nv,
                      kLaScanThreads);
}

void set_decay(const gdr_tensor* g, const void*& p, int64_t& tok, int64_t& head, int32_t& bf16) {
    p = present(g) ? g->data : nullptr;
    tok = p ? g->stride[0] : 0;
    head = p ? g->stride[1] : 0;
    bf16 = p && g->dtype == GDR_DTYPE_BF16;
}

LaParams la_params(const LaDims& d, const LaPlan& pl, const gdr_tensor* off,
                   const gdr_tensor* slots, const gdr_tensor* g, float scale) {
    LaParams p{};
    p.B = static_cast<int32_t>(d.B);
    p.nv = static_cast<int32_t>(d.nv);
    p.T = static_cast<int32_t>(d.T);
    p.seg_len = static_cast<int32_t>(pl.seg_len);
    p.segs = static_cast<int32_t>(pl.segs);
    p.offsets = as_u32(off);
    p.slot_idx = as_u32(slots);
    set_decay(g, p.g, p.g_tok, p.g_head, p.g_bf16);
    p.scale = scale;
    return p;
}

LaWalk la_walk(const LaTensor& x, const LaTensor& y, const LaTensor& z, int64_t Kd, int64_t Vd,
               bool reverse) {
    LaWalk w{};
    w.x = x;
    w.y = y;
    w.z = z;
    w.Kd = static_cast<int32_t>(Kd);
    w.Vd = static_cast<int32_t>(Vd);
    w.tiles = static_cast<int32_t>(ceil_div(Vd, 16 * la_waves(w.Vd)));
    w.reverse = reverse;
    return w;
}

// Walks of one built shape in one launch.
hipError_t run_walks(LaParams p, const LaWalk* w, int n, bool b16, hipStream_t s) {
    p.nwalks = n;
    p.max_tiles = 1;
    for (int i = 0; i < n; ++i) {
        p.w[i] = w[i];
        p.max_tiles = std::max(p.max_tiles, w[i].tiles);
    }
    return launch_la_walks(p, b16, s);
}

// Walks of one class run the same kernel.
int size_class(int Kd, int Vd) { return (Kd <= 64 ? 0 : Kd <= 128 ? 1 : 2) * 16 + la_waves(Vd); }

LaScan la_scan(const LaParams& p, const LaDims& d, int64_t rows, float* state, const float* tot,
               bool reverse, const LaState& in) {
    LaScan c{};
    c.B = p.B;
    c.rows = static_cast<int32_t>(rows);
    c.nv = p.nv;
    c.T = p.T;
    c.seg_len = p.seg_len;
    c.walk_from = p.walk_from;
    c.segs = p.segs;
    c.offsets = p.offsets;
    c.slot_idx = p.slot_idx;
    c.n = static_cast<int32_t>(d.K * d.V);
    c.V = static_cast<int32_t>(d.V);
    c.reverse = reverse;
    c.state = state;
    c.tot = tot;
    c.in = in;
    return c;
}

hipError_t run_step(const LaDims& d, const gdr_tensor* o, const gdr_tensor* q, const gdr_tensor* k,
                    const gdr_tensor* v, const gdr_tensor* g, const gdr_tensor* off,
                    const gdr_tensor* slots, const LaState& in, const LaState& last, float scale,
                    hipStream_t s) {
    LaStep p{};
    p.B = static_cast<int32_t>(d.B);
    p.nv = static_cast<int32_t>(d.nv);
    p.G = static_cast<int32_t>(d.nv / d.nk);
    p.K = static_cast<int32_t>(d.K);
    p.V = static_cast<int32_t>(d.V);
    p.offsets = as_u32(off);
    p.slot_idx = as_u32(slots);
    p.q = q->data; p.q_tok = q->stride[0]; p.q_head = q->stride[1];
    p.k = k->data; p.k_tok = k->stride[0]; p.k_head = k->stride[1];
    p.v = v->data; p.v_tok = v->stride[0]; p.v_head = v->stride[1];
    set_decay(g, p.g, p.g_tok, p.g_head, p.g_bf16);
    p.out = o->data; p.o_tok = o->stride[0]; p.o_head = o->stride[1];
    p.in = in;
    p.last = last;
    p.most = kLaStepTokens;
    p.scale = scale;
    return launch_la_step(p, d.work == GDR_DTYPE_BF16, s);
}

int no_alias(const char* fn, const gdr_tensor* out, const char* name,
             std::initializer_list<const gdr_tensor*> ins) {
    if (empty(out)) return GDR_OK;
    for (const gdr_tensor* t : ins)
        if (present(t) && t->data == out->data)
            return fail(GDR_ERR_INVALID_ARG, "%s: %s must not alias an input", fn, name);
    return GDR_OK;
}

int done() {
    clear_error();
    return GDR_OK;
}

}  // namespace

extern "C" {

int64_t gdr_linear_attention_workspace(int64_t tokens, int64_t rows, int32_t num_key_heads,
                                       int32_t num_value_heads, int32_t key_head_dim,
                                       int32_t value_head_dim, int backward) {
    if (tokens < 0 || rows < 0 || num_key_heads < 1 || num_value_heads < 1 || key_head_dim < 1 ||
        value_head_dim < 1)
        return -1;
    if (rows == 0) return 0;
    return la_plan(tokens, rows, num_key_heads, num_value_heads, key_head_dim, value_head_dim,
                   backward != 0)
        .end;
}

int gdr_linear_attention_fwd(const gdr_tensor* o, const gdr_tensor* q, const gdr_tensor* k,
                             const gdr_tensor* v, const gdr_tensor* g,
                             const gdr_tensor* input_row_offsets, float scale,
                             const gdr_tensor* initial_state, const gdr_tensor* final_state,
                             const gdr_tensor* state, const gdr_tensor* slot_idx,
                             const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_linear_attention_fwd";
    LaDims d{};
    int rc;
    if ((rc = check_la(fn, q, k, v, g, true, d)) || (rc = check_offsets(fn, input_row_offsets, d)) ||
        (rc = check_out_heads(fn, "o", o, d.T, d.nv, d.V, d.work)) ||
        (rc = no_alias(fn, o, "o", {q, k, v, g})))
        return rc;
    const bool pool = present(state);
    if (pool) {
        if (present(initial_state) || present(final_state))
            return fail(GDR_ERR_INVALID_ARG, "%s: give state, or initial_state and final_state", fn);
        if ((rc = check_la_state(fn, "state", state, -1, d.nv, d.K, d.V, true))) return rc;
        if (present(slot_idx)) {
            if ((rc = check_index_vec(fn, "slot_idx", slot_idx, d.B))) return rc;
        } else if (state->shape[0] < d.B) {
            return fail(GDR_ERR_INVALID_ARG, "%s: state has fewer slots than rows", fn);
        }
    } else {
        if (present(slot_idx))
            return fail(GDR_ERR_INVALID_ARG, "%s: slot_idx needs state", fn);
        if (present(initial_state) &&
            (rc = check_la_state(fn, "initial_state", initial_state, d.B, d.nv, d.K, d.V, false)))
            return rc;
        if (present(final_state) &&
            (rc = check_la_state(fn, "final_state", final_state, d.B, d.nv, d.K, d.V, true)))
            return rc;
        if (present(initial_state) && present(final_state) &&
            initial_state->dtype != final_state->dtype)
            return fail(GDR_ERR_UNSUPPORTED, "%s: final_state must have initial_state's dtype", fn);
    }
    if (d.B == 0) return done();
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool b16 = d.work == GDR_DTYPE_BF16;
    const float sc = resolve_scale(scale, d.K);
    const LaState in = la_state(pool ? state : initial_state, d.V, false, 1.0f);
    const LaState last = la_state(pool ? state : final_state, d.V, false, 1.0f);
    const LaPlan pl = la_plan(d.T, d.B, d.nk, d.nv, d.K, d.V, false);
    // with rows enough those of few tokens go token by token, and these are walked
    const bool split = d.B >= kLaStepRows;
    const int64_t rows = split ? std::min(d.B, d.T / (kLaStepTokens + 1)) : d.B;
    const int64_t segs = !split ? pl.segs : rows + (pl.seg_len ? d.T / pl.seg_len : 0);
    const int64_t wide = 64 * la_waves(static_cast<int>(d.V));
    if ((rc = check_workspace(fn, workspace, pl.end)) ||
        (split && (rc = check_grid(fn, d.B * d.nv, la_step_threads(d.K, d.V)))) ||
        (rows && (rc = check_grid(fn, segs * d.nv * pl.v_tiles, wide))) ||
        (pl.seg_len && ((rc = check_grid(fn, pl.cuts * d.nv * pl.v_tiles, wide)) ||
                        (rc = check_scan(fn, d, pl.cut_rows)))))
        return rc;
    IndexCheck ic;
    ic.offsets = input_row_offsets;
    ic.total_tokens = d.T;
    if (pool && present(slot_idx)) {
        ic.slots = slot_idx;
        ic.num_slots = state->shape[0];
    }
    if ((rc = run_debug_check(fn, d.B, ic, stream))) return rc;
    const int64_t G = d.nv / d.nk;
    LaParams p = la_params(d, pl, input_row_offsets, slot_idx, g, sc);
    hipError_t e = hipSuccess;
    if (split) {
        e = run_step(d, o, q, k, v, g, input_row_offsets, slot_idx, in, last, sc, s);
        if (e != hipSuccess || rows == 0) return hip_status(fn, e);
        p.walk_from = kLaStepTokens + 1;
        p.segs = static_cast<int32_t>(segs);
        if (!pl.seg_len) p.seg_len = p.T;
    }
    LaWalk w = la_walk(la_tensor(q, G), la_tensor(k, G), la_tensor(v, 1), d.K, d.V, false);
    w.out = o->data;
    w.out_tok = d.T > 1 ? o->stride[0] : 0;
    w.out_head = o->stride[1];
    w.in = in;
    w.last = last;
    w.third = last.p && !last.bf16;
    if (pl.seg_len && e == hipSuccess) {
        float* ws = static_cast<float*>(workspace->data);
        LaWalk sum = w;
        sum.last = la_segment_state(ws + pl.s_fwd, d.nv, d.K, d.V, false);
        LaParams ps = p;                  // of the rows that are cut
        ps.walk_from = static_cast<int32_t>(pl.seg_len) + 1;
        ps.segs = static_cast<int32_t>(pl.cuts);
        ps.nwalks = 1;
        ps.max_tiles = w.tiles;
        ps.w[0] = sum;
        e = launch_la_segments(ps, b16, ws + pl.tot, s);
        const LaScan scan = la_scan(ps, d, pl.cut_rows, ws + pl.s_fwd, ws + pl.tot, false, in);
        if (e == hipSuccess) e = launch_la_scans(&scan, 1, s);
        w.in_row = in;
        w.in = sum.last;
        w.by_cut = 1;
    }
    if (e == hipSuccess) e = run_walks(p, &w, 1, b16, s);
    return hip_status(fn, e);
}

int gdr_linear_attention_step(const gdr_tensor* o, const gdr_tensor* q, const gdr_tensor* k,
                              const gdr_tensor* v, const gdr_tensor* g, const gdr_tensor* state,
                              const gdr_tensor* slot_idx, float scale, void* stream) {
    const char* fn = "gdr_linear_attention_step";
    LaDims d{};
    int rc;
    if ((rc = check_la(fn, q, k, v, g, false, d)) ||
        (rc = check_out_heads(fn, "o", o, d.T, d.nv, d.V, d.work)) ||
        (rc = no_alias(fn, o, "o", {q, k, v, g})) ||
        (rc = check_la_state(fn, "state", state, -1, d.nv, d.K, d.V, true)))
        return rc;
    d.B = d.T;
    if (present(slot_idx)) {
        if ((rc = check_index_vec(fn, "slot_idx", slot_idx, d.B))) return rc;
    } else if (state->shape[0] < d.B) {
        return fail(GDR_ERR_INVALID_ARG, "%s: state has fewer slots than rows", fn);
    }
    if (d.B == 0) return done();
    if ((rc = check_grid(fn, d.B * d.nv, la_step_threads(d.K, d.V)))) return rc;
    IndexCheck ic;
    if (present(slot_idx)) {
        ic.slots = slot_idx;
        ic.num_slots = state->shape[0];
    }
    if ((rc = run_debug_check(fn, d.B, ic, stream))) return rc;
    const LaState st = la_state(state, d.V, false, 1.0f);
    return hip_status(fn, run_step(d, o, q, k, v, g, nullptr, slot_idx, st, st,
                                   resolve_scale(scale, d.K), static_cast<hipStream_t>(stream)));
}

int gdr_linear_attention_bwd(const gdr_tensor* d_o, const gdr_tensor* q, const gdr_tensor* k,
                             const gdr_tensor* v, const gdr_tensor* g,
                             const gdr_tensor* input_row_offsets, float scale,
                             const gdr_tensor* initial_state, const gdr_tensor* dfinal_state,
                             const gdr_tensor* dq, const gdr_tensor* dk, const gdr_tensor* dv,
                             const gdr_tensor* dg, const gdr_tensor* dinitial_state,
                             const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_linear_attention_bwd";
    LaDims d{};
    int rc;
    if ((rc = check_la(fn, q, k, v, g, true, d)) || (rc = check_offsets(fn, input_row_offsets, d)) ||
        (rc = check_heads(fn, "do", d_o, d.T, d.nv, d.V, d.work, true)) ||
        (rc = check_out_heads(fn, "dq", dq, d.T, d.nk, d.K, d.work)) ||
        (rc = check_out_heads(fn, "dk", dk, d.T, d.nk, d.K, d.work)) ||
        (rc = check_out_heads(fn, "dv", dv, d.T, d.nv, d.V, d.work)) ||
        (rc = no_alias(fn, dq, "dq", {d_o, q, k, v, g, dk, dv})) ||
        (rc = no_alias(fn, dk, "dk", {d_o, q, k, v, g, dv})) ||
        (rc = no_alias(fn, dv, "dv", {d_o, q, k, v, g})))
        return rc;
    if (present(initial_state) &&
        (rc = check_la_state(fn, "initial_state", initial_state, d.B, d.nv, d.K, d.V, false)))
        return rc;
    if (present(dfinal_state) &&
        (rc = check_la_state(fn, "dfinal_state", dfinal_state, d.B, d.nv, d.K, d.V, false)))
        return rc;
    if (present(dinitial_state) &&
        ((rc = check_la_state(fn, "dinitial_state", dinitial_state, d.B, d.nv, d.K, d.V, true)) ||
         (rc = no_alias(fn, dinitial_state, "dinitial_state", {initial_state, dfinal_state}))))
        return rc;
    if (present(dg)) {
        const int64_t gs[2] = {d.T, d.nv};
        if (!present(g) && d.T) return fail(GDR_ERR_INVALID_ARG, "%s: dg needs g", fn);
        if ((rc = check_tensor(fn, "dg", dg, 2, gs, true, true, false)) ||
            (rc = check_distinct(fn, "dg", dg)) ||
            (rc = no_alias(fn, dg, "dg", {d_o, q, k, v, g})))
            return rc;
    }
    if (d.nv * d.K > kLaMaxTokenStride)
        return fail(GDR_ERR_UNSUPPORTED, "%s: v's heads times K above %lld", fn,
                    static_cast<ll>(kLaMaxTokenStride));
    if (d.B == 0) return done();
    const LaPlan pl = la_plan(d.T, d.B, d.nk, d.nv, d.K, d.V, true);
    const int K = static_cast<int>(d.K), V = static_cast<int>(d.V);
    const bool one = size_class(V, K) == size_class(K, V);  // launch of the three walks
    const int64_t rows = pl.segs * d.nv, wide_k = 64 * la_waves(K), wide_v = 64 * la_waves(V);
    if ((rc = check_workspace(fn, workspace, pl.end)) ||
        (one ? (rc = check_grid(fn, rows * 3 * std::max(pl.q_tiles, pl.v_tiles), wide_v))
             : (rc = check_grid(fn, rows * 2 * pl.q_tiles, wide_k)) ||
                   (rc = check_grid(fn, rows * pl.v_tiles, wide_v))) ||
        (pl.seg_len && ((rc = check_grid(fn, pl.cuts * d.nv * 2 * pl.v_tiles, wide_v)) ||
                        (rc = check_scan(fn, d, pl.cut_rows)))) ||
        (present(dg) && (rc = check_grid(fn, rows, 256))) ||
        (d.nv != d.nk && (rc = check_grid(fn, ceil_div(d.T * d.nk * (d.K / 4), 256), 256))))
        return rc;
    IndexCheck ic;
    ic.offsets = input_row_offsets;
    ic.total_tokens = d.T;
    if ((rc = run_debug_check(fn, d.B, ic, stream))) return rc;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool b16 = d.work == GDR_DTYPE_BF16, sums = present(dg), parts = d.nv != d.nk;
    const float sc = resolve_scale(scale, d.K);
    const int64_t G = d.nv / d.nk;
    float* ws = static_cast<float*>(workspace->data);
    const LaTensor tq = la_tensor(q, G), tk = la_tensor(k, G), tv = la_tensor(v, 1),
                   to = la_tensor(d_o, 1);
    LaParams p = la_params(d, pl, input_row_offsets, nullptr, g, sc);

    LaWalk wq = la_walk(to, tv, tk, d.V, d.K, false);
    LaWalk wv = la_walk(tk, tq, to, d.K, d.V, true);
    LaWalk wk = la_walk(tv, to, tq, d.V, d.K, true);
    wq.in = la_state(initial_state, d.V, true, 1.0f);
    wv.in = la_state(dfinal_state, d.V, false, 1.0f / sc);
    wk.in = la_state(dfinal_state, d.V, true, 1.0f / sc);
    wv.last = la_state(dinitial_state, d.V, false, sc);
    wv.third = wv.last.p && !wv.last.bf16;
    hipError_t e = hipSuccess;
    if (pl.seg_len) {
        float *sf = ws + pl.s_fwd, *sr = ws + pl.s_rev, *tot = ws + pl.tot;
        LaParams ps = p;
        ps.nwalks = 2;
        ps.w[0] = la_walk(tq, tk, tv, d.K, d.V, false);
        ps.w[0].last = la_segment_state(sf, d.nv, d.K, d.V, false);
        ps.w[1] = la_walk(tk, tq, to, d.K, d.V, true);
        ps.w[1].last = la_segment_state(sr, d.nv, d.K, d.V, false);
        ps.w[1].third = wv.third;
        ps.max_tiles = ps.w[0].tiles;
        e = launch_la_segments(ps, b16, tot, s);
        const LaScan scans[2] = {
            la_scan(p, d, pl.cut_rows, sf, tot, false, la_state(initial_state, d.V, false, 1.0f)),
            la_scan(p, d, pl.cut_rows, sr, tot, true, la_state(dfinal_state, d.V, false, 1.0f / sc))};
        if (e == hipSuccess) e = launch_la_scans(scans, 2, s);
        wq.in = la_segment_state(sf, d.nv, d.K, d.V, true);
        wv.in = la_segment_state(sr, d.nv, d.K, d.V, false);
        wk.in = la_segment_state(sr, d.nv, d.K, d.V, true);
    }
    wv.out = dv->data;
    wv.out_tok = d.T > 1 ? dv->stride[0] : 0;
    wv.out_head = dv->stride[1];
    if (parts) {
        wq.out = ws + pl.pq;
        wk.out = ws + pl.pk;
        wq.out_tok = wk.out_tok = d.nv * d.K;
        wq.out_head = wk.out_head = d.K;
        wq.out_f32 = wk.out_f32 = 1;
    } else {
        wq.out = dq->data;
        wq.out_tok = d.T > 1 ? dq->stride[0] : 0;
        wq.out_head = dq->stride[1];
        wk.out = dk->data;
        wk.out_tok = d.T > 1 ? dk->stride[0] : 0;
        wk.out_head = dk->stride[1];
    }
    if (sums) {
        wq.row_sum = ws + pl.rq;
        wq.partner = tq;
        wk.row_sum = ws + pl.rk;
        wk.partner = tk;
        if (wk.in.p) {                    // nothing comes back into the rows' ends otherwise
            wq.phi = ws + pl.phi;
            wq.phi_in = wk.in;
        }
        if (present(initial_state)) {     // and into their starts
            wv.phi = ws + pl.phi0;
            wv.phi_in = la_state(initial_state, d.V, false, 1.0f);
            wv.phi_rows = 1;
        }
    }
    const LaWalk all[3] = {wq, wv, wk};
    if (e == hipSuccess) {
        if (one) {
            e = run_walks(p, all, 3, b16, s);
        } else {
            const LaWalk two[2] = {wq, wk};
            e = run_walks(p, two, 2, b16, s);
            if (e == hipSuccess) e = run_walks(p, &wv, 1, b16, s);
        }
    }
    if (e == hipSuccess && sums) {
        LaDecayGrad c{};
        c.B = p.B;
        c.nv = p.nv;
        c.T = p.T;
        c.seg_len = p.seg_len;
        c.segs = p.segs;
        c.offsets = p.offsets;
        c.rq = ws + pl.rq;
        c.rk = ws + pl.rk;
        c.phi = wq.phi;
        c.parts = wq.tiles * la_waves(wq.Vd);
        c.phi0 = wv.phi;
        c.parts0 = wv.tiles * la_waves(wv.Vd);
        c.dg = dg->data;
        c.dg_tok = dg->stride[0];
        c.dg_head = dg->stride[1];
        c.dg_bf16 = dg->dtype == GDR_DTYPE_BF16;
        e = launch_la_decay_grad(c, s);
    }
    if (parts && d.T > 0) {
        LaHeadSum h{};
        h.T = p.T;
        h.nk = static_cast<int32_t>(d.nk);
        h.G = static_cast<int32_t>(G);
        h.K = static_cast<int32_t>(d.K);
        h.B = p.B;
        h.offsets = p.offsets;
        const gdr_tensor* outs[2] = {dq, dk};
        const int64_t from[2] = {pl.pq, pl.pk};
        for (int i = 0; i < 2 && e == hipSuccess; ++i) {
            h.part = ws + from[i];
            h.out = outs[i]->data;
            h.out_tok = outs[i]->stride[0];
            h.out_head = outs[i]->stride[1];
            e = launch_la_head_sum(h, b16, s);
        }
    }
    return hip_status(fn, e);
}

}  // extern "C"

// ------------------------------------------------------------------ norms ---

namespace {

int check_rows(const char* fn, const char* name, const gdr_tensor* t, int64_t T, int64_t D,
               int32_t work, bool out) {
    const int64_t shape[2] = {T, D};
    int rc = check_tensor(fn, name, t, 2, shape, true, true, false);
    if (rc || (rc = check_work_dtype(fn, name, t, work)) ||
        (rc = check_layout(fn, name, t, vec_mult(work))))
        return rc;
    return out ? check_distinct(fn, name, t) : GDR_OK;
}

// A [n] vector in float32 or the work dtype.
int check_vec(const char* fn, const char* name, const gdr_tensor* t, int64_t n, int32_t work) {
    const int64_t shape[1] = {n};
    int rc = check_tensor(fn, name, t, 1, shape, true, true, false);
    if (rc) return rc;
    if (t->dtype != GDR_DTYPE_F32 && t->dtype != work)
        return fail(GDR_ERR_UNSUPPORTED, "%s: %s must be f32 or the work dtype", fn, name);
    return check_layout(fn, name, t, 1);
}

NormVec norm_vec(const gdr_tensor* t) {
    NormVec v{};
    if (present(t)) {
        v.p = t->data;
        v.bf16 = t->dtype == GDR_DTYPE_BF16;
    }
    return v;
}

// The arguments that the norm and its gradient share.
int check_norm(const char* fn, const gdr_tensor* y, const gdr_tensor* gate,
               const gdr_tensor* post_weight, const gdr_tensor* pre_weight, int64_t group,
               float residual_scale, float eps, uint32_t flags, NormParams& p, int32_t& work) {
    int rc = check_tensor(fn, "y", y, 2, nullptr, true, true, false);
    if (rc) return rc;
    if (flags & ~(GDR_FLAG_GATE_SIGMOID | GDR_FLAG_GATE_SILU))
        return fail(GDR_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (flags == (GDR_FLAG_GATE_SIGMOID | GDR_FLAG_GATE_SILU))
        return fail(GDR_ERR_INVALID_ARG, "%s: one activation at most", fn);
    const int64_t T = y->shape[0], D = y->shape[1];
    work = y->dtype;
    if (D % 8 || D > kNormMaxDim)
        return fail(GDR_ERR_UNSUPPORTED, "%s: rows of %lld values (multiples of 8 up to %d)", fn,
                    static_cast<ll>(D), kNormMaxDim);
    if (T > INT32_MAX) return fail(GDR_ERR_INVALID_ARG, "%s: too many rows", fn);
    if ((rc = check_rows(fn, "y", y, T, D, work, false))) return rc;
    if (group <= 0) group = D;
    if (D && (group % 8 || D % group))
        return fail(GDR_ERR_INVALID_ARG, "%s: groups of %lld values (a multiple of 8 that divides "
                    "%lld)", fn, static_cast<ll>(group), static_cast<ll>(D));
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(GDR_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    p.T = T;
    p.D = static_cast<int32_t>(D);
    p.group = static_cast<int32_t>(group);
    p.act = flags & GDR_FLAG_GATE_SIGMOID ? 1 : flags & GDR_FLAG_GATE_SILU ? 2 : 0;
    p.c = residual_scale;
    p.eps = eps;
    p.y = y->data;
    p.y_row = y->stride[0];
    if (present(post_weight)) {
        const int64_t n = post_weight->ndim == 1 && post_weight->shape[0] == group ? group : D;
        if ((rc = check_vec(fn, "post_weight", post_weight, n, work))) return rc;
        p.w1 = norm_vec(post_weight);
        p.w1_len = static_cast<int32_t>(n);
    } else if (group != D) {
        return fail(GDR_ERR_INVALID_ARG, "%s: groups need post_weight", fn);
    }
    if (present(gate)) {
        if (gate->ndim == 1) {
            if ((rc = check_vec(fn, "gate", gate, D, work))) return rc;
            p.gate_mode = 2;
            p.gate_c = norm_vec(gate);
        } else {
            if ((rc = check_rows(fn, "gate", gate, T, D, work, false))) return rc;
            p.gate_mode = 1;
            p.gate = gate->data;
            p.gate_row = gate->stride[0];
        }
    } else {
        p.act = 0;  // an activation of nothing
    }
    if (present(pre_weight)) {
        if ((rc = check_vec(fn, "pre_weight", pre_weight, D, work))) return rc;
        p.w2 = norm_vec(pre_weight);
    }
    return GDR_OK;
}

// Floats of the backward's workspace: parts of each weight's gradient.
int64_t norm_workspace(int64_t T, int64_t D, int64_t w1_len, bool pre, bool channel_gate,
                       int64_t* parts, int64_t* w2_at, int64_t* gate_at, int64_t* end) {
    *parts = norm_parts(T, static_cast<int>(D));
    int64_t at = ceil_div(*parts * w1_len, 64) * 64;
    *w2_at = at;
    at += pre ? *parts * D : 0;
    *gate_at = at = ceil_div(at, 64) * 64;
    at += channel_gate ? *parts * D : 0;
    *end = at;
    return at;
}

}  // namespace

extern "C" {

int64_t gdr_block_norm_workspace(int64_t tokens, int64_t dim) {
    if (tokens < 0 || dim < 0 || dim > kNormMaxDim) return -1;
    if (tokens == 0 || dim == 0) return 0;
    int64_t parts, a, b, end;
    return norm_workspace(tokens, dim, dim, true, true, &parts, &a, &b, &end);
}

int gdr_block_norm(const gdr_tensor* h, const gdr_tensor* n, const gdr_tensor* y,
                   const gdr_tensor* residual, const gdr_tensor* gate,
                   const gdr_tensor* post_weight, const gdr_tensor* pre_weight, int64_t group,
                   float residual_scale, float eps, uint32_t flags, void* stream) {
    const char* fn = "gdr_block_norm";
    NormParams p{};
    int32_t work;
    int rc = check_norm(fn, y, gate, post_weight, pre_weight, group, residual_scale, eps, flags, p,
                        work);
    if (rc || (rc = check_rows(fn, "h", h, p.T, p.D, work, true))) return rc;
    if (present(residual)) {
        if ((rc = check_rows(fn, "residual", residual, p.T, p.D, work, false))) return rc;
        p.x = residual->data;
        p.x_row = residual->stride[0];
    }
    const bool none = p.T == 0 || p.D == 0;
    if (!none && present(n) != present(pre_weight))
        return fail(GDR_ERR_INVALID_ARG, "%s: n and pre_weight go together", fn);
    if (present(n)) {
        if ((rc = check_rows(fn, "n", n, p.T, p.D, work, true))) return rc;
        if (n->data == h->data) return fail(GDR_ERR_INVALID_ARG, "%s: n must not alias h", fn);
        p.n = n->data;
        p.n_row = n->stride[0];
    }
    p.h = h->data;
    p.h_row = h->stride[0];
    if (none) return done();
    if ((rc = check_grid(fn, p.T, norm_threads(p)))) return rc;
    return hip_status(fn, launch_norm(p, work == GDR_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

int gdr_block_norm_bwd(const gdr_tensor* dresidual, const gdr_tensor* dy, const gdr_tensor* dgate,
                       const gdr_tensor* dpost_weight, const gdr_tensor* dpre_weight,
                       const gdr_tensor* dh, const gdr_tensor* dn, const gdr_tensor* y,
                       const gdr_tensor* h, const gdr_tensor* gate, const gdr_tensor* post_weight,
                       const gdr_tensor* pre_weight, int64_t group, float residual_scale,
                       float eps, uint32_t flags, const gdr_tensor* workspace, void* stream) {
    const char* fn = "gdr_block_norm_bwd";
    NormParams p{};
    int32_t work;
    int rc = check_norm(fn, y, gate, post_weight, pre_weight, group, residual_scale, eps, flags, p,
                        work);
    if (rc || (rc = check_rows(fn, "dh", dh, p.T, p.D, work, false)) ||
        (rc = check_rows(fn, "dy", dy, p.T, p.D, work, true)))
        return rc;
    const bool pre = present(pre_weight), none = p.T == 0 || p.D == 0;
    if (pre) {
        if ((rc = check_rows(fn, "dn", dn, p.T, p.D, work, false)) ||
            (rc = check_rows(fn, "h", h, p.T, p.D, work, false)))
            return rc;
        p.dn = dn->data;
        p.dn_row = dn->stride[0];
        p.h = h->data;
        p.h_row = h->stride[0];
    } else if (present(dn)) {
        return fail(GDR_ERR_INVALID_ARG, "%s: dn needs pre_weight", fn);
    }
    if (present(dresidual)) {
        if ((rc = check_rows(fn, "dresidual", dresidual, p.T, p.D, work, true))) return rc;
        p.dx = dresidual->data;
        p.dx_row = dresidual->stride[0];
    }
    const bool row_gate = p.gate_mode == 1, channel_gate = p.gate_mode == 2;
    if (row_gate) {
        if ((rc = check_rows(fn, "dgate", dgate, p.T, p.D, work, true))) return rc;
        p.dgate = dgate->data;
        p.dgate_row = dgate->stride[0];
    } else if (channel_gate) {
        if ((rc = check_vec(fn, "dgate", dgate, p.D, work))) return rc;
    } else if (present(dgate)) {
        return fail(GDR_ERR_INVALID_ARG, "%s: dgate needs gate", fn);
    }
    if (p.w1.p) {
        if ((rc = check_vec(fn, "dpost_weight", dpost_weight, p.w1_len, work))) return rc;
    } else if (present(dpost_weight)) {
        return fail(GDR_ERR_INVALID_ARG, "%s: dpost_weight needs post_weight", fn);
    }
    if (pre) {
        if ((rc = check_vec(fn, "dpre_weight", dpre_weight, p.D, work))) return rc;
    } else if (present(dpre_weight)) {
        return fail(GDR_ERR_INVALID_ARG, "%s: dpre_weight needs pre_weight", fn);
    }
    const gdr_tensor* outs[5] = {dresidual, dy, row_gate ? dgate : nullptr, nullptr, nullptr};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (present(outs[i]) && present(outs[j]) && outs[i]->data == outs[j]->data)
                return fail(GDR_ERR_INVALID_ARG, "%s: two outputs share memory", fn);
    if (p.D == 0) return done();
    int64_t parts, w2_at, gate_at, end;
    norm_workspace(std::max<int64_t>(p.T, 1), p.D, p.w1.p ? p.w1_len : 0, pre, channel_gate,
                   &parts, &w2_at, &gate_at, &end);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!none && (rc = check_workspace(fn, workspace, end))) return rc;
    NormReduce r[3] = {};
    int count = 0;
    float* ws = none || end == 0 ? nullptr : static_cast<float*>(workspace->data);
    p.parts = static_cast<int32_t>(parts);
    p.y = y->data;
    p.dh = dh->data;
    p.dh_row = dh->stride[0];
    p.dy = dy->data;
    p.dy_row = dy->stride[0];
    auto reduce = [&](const gdr_tensor* out, float* part, int64_t n) {
        r[count].part = part;
        r[count].parts = none ? 0 : p.parts;
        r[count].n = static_cast<int32_t>(n);
        r[count].out = out->data;
        r[count].out_bf16 = out->dtype == GDR_DTYPE_BF16;
        ++count;
    };
    if (p.w1.p) reduce(dpost_weight, p.pw1 = ws, p.w1_len);
    if (pre) reduce(dpre_weight, p.pw2 = ws ? ws + w2_at : nullptr, p.D);
    if (channel_gate) reduce(dgate, p.pgate = ws ? ws + gate_at : nullptr, p.D);
    hipError_t e = none ? hipSuccess : launch_norm_bwd(p, work == GDR_DTYPE_BF16, s);
    if (e == hipSuccess && count) e = launch_norm_reduce(r, count, s);
    return hip_status(fn, e);
}

}  // extern "C"

// Entry points of the attention calls: host checks, the cut of a call into
// workgroups, workspaces.  The kernels are in attention.h.
#include "attention.h"

namespace spc {
namespace attn {
namespace {

constexpr int D_MAX = 128;

// Rows of one side that work is cut over (positions times the heads that share
// them), and the other side's.
Cut cut_of(int64_t rows, int64_t other, int64_t n_seg, int heads, int D) {
    Cut c;
    // Four waves share the staged tiles where samples have rows for them and
    // the call fills the chip; else as few as there can be, which leave fewer lanes idle.
    c.nw = rows >= 64 * n_seg && slots_of(rows, n_seg, 128) * heads >= 512 ? 4 : few_waves(D);
    c.slots = slots_of(rows, n_seg, 32 * c.nw);
    // Few workgroups: the other side is split too, and the parts are joined by
    // a second launch, to 4 waves a SIMD.  A split is worth at least 128 rows of the
    // longest sample, which may be several times the mean (only the device knows):
    // taken as 8 times.  Forward + backward in us where it is taken as the mean, 3, 8
    // and 32 times that, ragged causal samples: 5,003 x 6 over 2 x 48 fp32 in 23 of
    // them 163 + 392, 91 + 275, 91 + 274, 91 + 275; 8,000 x 2 x 32 bf16 in 50 40 +
    // 123, 24 + 67, 23 + 60, 23 + 60; even ones pay a little for parts that are
    // empty: 2,000 x 4 x 32 fp32 in 4 36 + 98, 38 + 104, 36 + 104, 36 + 104.  Samples
    // of fewer than 128 rows in the mean are not split.
    const int64_t want = 4096 / c.nw, have = (rows / (32 * c.nw) + n_seg) * heads;
    const int64_t mean = other / n_seg, longest = mean < 128 ? 0 : 8 * mean < other ? 8 * mean : other, most = longest / 128;
    c.splits = int32_t(have * 2 > want || most < 2 ? 1 : (want / have < most ? want / have : most));
    c.blocks = (c.slots * c.splits + 8 * (32 / c.nw)) * heads;   // with what rounding up to groups of an XCD adds
    return c;
}

struct Plan {
    Cut q, k;
    size_t fwd, bwd;    // workspace bytes
};

spc_status check_sizes(spc_dtype dtype, const spc_attention* a, Plan& w) {
    if (dtype != SPC_F32 && dtype != SPC_F16 && dtype != SPC_BF16) return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
    if (!a) return fail(SPC_ERR_ARG, "the attention descriptor is NULL");
    if (a->n_q < 0 || a->n_q >= ROWS_END) return fail(SPC_ERR_ARG, "n_q=%lld is out of range", (long long)a->n_q);
    if (a->n_kv < 0 || a->n_kv >= ROWS_END) return fail(SPC_ERR_ARG, "n_kv=%lld is out of range", (long long)a->n_kv);
    if (a->n_seg < 1 || a->n_seg >= ROWS_END) return fail(SPC_ERR_ARG, "n_seg=%lld is out of range", (long long)a->n_seg);
    if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads)
        return fail(SPC_ERR_ARG, "heads=%d is not a positive multiple of kv_heads=%d", a->heads, a->kv_heads);
    if (a->head_dim < 1 || a->head_dim % 16 || a->head_dim > D_MAX)
        return fail(SPC_ERR_UNSUPPORTED, "head_dim=%d: a multiple of 16 up to %d", a->head_dim, D_MAX);
    if (int64_t(a->heads) * a->head_dim > C_MAX) return fail(SPC_ERR_UNSUPPORTED, "%d heads of %d are too many", a->heads, a->head_dim);
    if (a->n_q * a->heads >= ROWS_END || a->n_kv * a->kv_heads >= ROWS_END)
        return fail(SPC_ERR_UNSUPPORTED, "rows x heads exceed 31 bits");
    if (!(a->scale > 0.f && a->scale <= 1e38f)) return fail(SPC_ERR_ARG, "scale=%g must be positive and at most 1e38", double(a->scale));
    const int64_t rows = a->n_q * (a->heads / a->kv_heads);
    w.q = cut_of(rows, a->n_kv, a->n_seg, a->kv_heads, a->head_dim);
    w.k = cut_of(a->n_kv, rows, a->n_seg, a->kv_heads, a->head_dim);
    // (a call that is split has few workgroups, so its join has too)
    if (!launchable(w.q.blocks, 64 * w.q.nw) || !launchable(w.k.blocks, 64 * w.k.nw))
        return fail(SPC_ERR_UNSUPPORTED, "%lld samples of %lld and %lld rows exceed one launch", (long long)a->n_seg, (long long)a->n_q,
                    (long long)a->n_kv);
    const size_t hq = size_t(a->n_q) * size_t(a->heads), hk = size_t(a->n_kv) * size_t(a->kv_heads), D = size_t(a->head_dim);
    w.fwd = w.q.splits > 1 ? size_t(w.q.splits) * hq * (D + 4) * 4 : 0;
    const size_t pq = w.q.splits > 1 ? size_t(w.q.splits) * hq * D * 4 : 0, pk = w.k.splits > 1 ? size_t(w.k.splits) * hk * 2 * D * 4 : 0;
    w.bwd = align_up(hq * 4, 256) + (pq > pk ? pq : pk);
    return SPC_OK;
}

struct Side {
    const void* p;
    int64_t ld;
    int32_t heads;
    const char* name;
};

spc_status check_call(spc_dtype dtype, const spc_attention* a, const void* ws, size_t need, size_t ws_bytes, Args& p) {
    if ((!a->q_ptr || !a->kv_ptr) && a->n_seg != 1) return fail(SPC_ERR_ARG, "q_ptr or kv_ptr is NULL with n_seg=%lld", (long long)a->n_seg);
    for (const void* q : {(const void*)a->q_ptr, (const void*)a->kv_ptr, (const void*)a->q_order, (const void*)a->kv_order, ws})
        if (q && !aligned16(q)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (!ws && need) return fail(SPC_ERR_ARG, "ws is NULL");
    if (ws_bytes < need) return fail(SPC_ERR_WORKSPACE, "ws_bytes=%zu, need %zu", ws_bytes, need);
    p = Args{};
    p.qs = Segs{a->q_ptr, int32_t(a->n_seg), int32_t(a->n_q)};
    p.ks = Segs{a->kv_ptr, int32_t(a->n_seg), int32_t(a->n_kv)};
    p.q_order = a->q_order, p.kv_order = a->kv_order;
    p.hk = a->kv_heads, p.g = a->heads / a->kv_heads, p.D = a->head_dim, p.causal = a->causal != 0;
    p.inv_g = p.g > 1 ? uint32_t(((uint64_t(1) << 32) + uint64_t(p.g) - 1) / uint64_t(p.g)) : 0u;
    p.scale = a->scale, p.c = float(double(a->scale) * 1.4426950408889634);
    return SPC_OK;
}

spc_status check_rows(spc_dtype dtype, const spc_attention* a, const Side& s, int64_t n) {
    if (s.ld < int64_t(s.heads) * a->head_dim || s.ld * dtype_size(dtype) % 16 || s.ld >= (int64_t(1) << 31))
        return fail(SPC_ERR_ARG, "row stride %lld of %s: at least heads x head_dim, a multiple of 16 bytes, below 2^31", (long long)s.ld, s.name);
    if (n > 0 && !s.p) return fail(SPC_ERR_ARG, "%s is NULL", s.name);
    if (s.p && !aligned16(s.p)) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    return SPC_OK;
}

Rows rows_of(spc_dtype dtype, const spc_attention* a, const Side& s, int64_t n) {
    const int64_t e = dtype_size(dtype);
    return Rows{s.p, n, int64_t(s.heads) * a->head_dim * e, s.ld * e, s.name};
}

}  // namespace
}  // namespace attn
}  // namespace spc

using namespace spc;
using namespace spc::attn;

extern "C" spc_status spc_attention_workspace(spc_dtype dtype, const spc_attention* a, size_t* fwd, size_t* bwd) {
    clear_error();
    if (!fwd || !bwd) return fail(SPC_ERR_ARG, "fwd or bwd is NULL");
    Plan w;
    const spc_status st = check_sizes(dtype, a, w);
    if (st == SPC_OK) *fwd = w.fwd, *bwd = w.bwd;
    return st;
}

extern "C" spc_status spc_attention_fwd(spc_dtype dtype, const spc_attention* a, const void* q, int64_t ldq, const void* k,
                                        int64_t ldk, const void* v, int64_t ldv, void* out, int64_t ldo, float* stats, void* rest,
                                        void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    Plan w;
    Args p;
    spc_status st = check_sizes(dtype, a, w);
    if (st == SPC_OK) st = check_call(dtype, a, ws, w.fwd, ws_bytes, p);
    if (st != SPC_OK) return st;
    const Side sq{q, ldq, a->heads, "q"}, sk{k, ldk, a->kv_heads, "k"}, sv{v, ldv, a->kv_heads, "v"}, so{out, ldo, a->heads, "out"},
        sr{dtype == SPC_F32 ? nullptr : rest, int64_t(a->heads) * a->head_dim, a->heads, "rest"};
    for (const Side* s : {&sq, &so})
        if ((st = check_rows(dtype, a, *s, a->n_q)) != SPC_OK) return st;
    for (const Side* s : {&sk, &sv})
        if ((st = check_rows(dtype, a, *s, a->n_kv)) != SPC_OK) return st;
    if ((stats && !aligned16(stats)) || (rest && !aligned16(rest))) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    if (a->n_q == 0) return SPC_OK;
    const Rows ro = rows_of(dtype, a, so, a->n_q), rr = rows_of(dtype, a, sr, a->n_q);
    for (const Rows* o : {&ro, &rr})
        for (const Rows& in : {rows_of(dtype, a, sq, a->n_q), rows_of(dtype, a, sk, a->n_kv), rows_of(dtype, a, sv, a->n_kv)})
            if ((st = check_overlap(*o, in)) != SPC_OK) return st;
    if ((st = check_overlap(ro, rr)) != SPC_OK) return st;
    const int64_t e = dtype_size(dtype);
    p.q = static_cast<const char*>(q), p.k = static_cast<const char*>(k), p.v = static_cast<const char*>(v), p.out = static_cast<char*>(out);
    p.ldq = ldq * e, p.ldk = ldk * e, p.ldv = ldv * e, p.ldo = ldo * e;
    p.stats = reinterpret_cast<float2*>(stats), p.rest = static_cast<char*>(rest);
    p.part = static_cast<float*>(ws);
    switch (dtype) {
        case SPC_F32: return launch_fwd_f32(p, w.q, stream);
        case SPC_F16: return launch_fwd_f16(p, w.q, stream);
        case SPC_BF16: return launch_fwd_bf16(p, w.q, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}

extern "C" spc_status spc_attention_bwd(spc_dtype dtype, const spc_attention* a, const void* dout, int64_t lddo, const void* q,
                                        int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, const void* out,
                                        int64_t ldo, const float* stats, const void* rest, void* dq, int64_t lddq, void* dk, int64_t lddk,
                                        void* dv, int64_t lddv, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    Plan w;
    Args p;
    spc_status st = check_sizes(dtype, a, w);
    if (st == SPC_OK) st = check_call(dtype, a, ws, w.bwd, ws_bytes, p);
    if (st != SPC_OK) return st;
    const Side queries[] = {{dout, lddo, a->heads, "dout"}, {q, ldq, a->heads, "q"}, {out, ldo, a->heads, "out"}, {dq, lddq, a->heads, "dq"}};
    const Side keys[] = {{k, ldk, a->kv_heads, "k"}, {v, ldv, a->kv_heads, "v"}, {dk, lddk, a->kv_heads, "dk"}, {dv, lddv, a->kv_heads, "dv"}};
    for (const Side& s : queries)
        if ((st = check_rows(dtype, a, s, a->n_q)) != SPC_OK) return st;
    for (const Side& s : keys)
        if ((st = check_rows(dtype, a, s, a->n_kv)) != SPC_OK) return st;
    if (a->n_q > 0 && !stats) return fail(SPC_ERR_ARG, "stats is NULL");
    if ((stats && !aligned16(stats)) || (rest && !aligned16(rest))) return fail(SPC_ERR_ARG, "device pointers must be 16-byte aligned");
    // the inputs, and the gradients behind them
    const Side sr{dtype == SPC_F32 ? nullptr : rest, int64_t(a->heads) * a->head_dim, a->heads, "rest"};
    const Rows all[] = {rows_of(dtype, a, queries[0], a->n_q), rows_of(dtype, a, queries[1], a->n_q), rows_of(dtype, a, queries[2], a->n_q),
                        rows_of(dtype, a, keys[0], a->n_kv),   rows_of(dtype, a, keys[1], a->n_kv),   rows_of(dtype, a, sr, a->n_q),
                        rows_of(dtype, a, queries[3], a->n_q), rows_of(dtype, a, keys[2], a->n_kv),   rows_of(dtype, a, keys[3], a->n_kv)};
    for (int o = 6; o < 9; ++o)
        for (int i = 0; i < o; ++i)
            if ((st = check_overlap(all[o], all[i])) != SPC_OK) return st;
    const int64_t e = dtype_size(dtype);
    p.q = static_cast<const char*>(q), p.k = static_cast<const char*>(k), p.v = static_cast<const char*>(v);
    p.o = static_cast<const char*>(out), p.dout = static_cast<const char*>(dout);
    p.dq = static_cast<char*>(dq), p.dk = static_cast<char*>(dk), p.dv = static_cast<char*>(dv);
    p.ldq = ldq * e, p.ldk = ldk * e, p.ldv = ldv * e, p.ldo = ldo * e, p.lddo = lddo * e;
    p.lddq = lddq * e, p.lddk = lddk * e, p.lddv = lddv * e;
    p.stats = reinterpret_cast<float2*>(const_cast<float*>(stats)), p.rest = static_cast<char*>(const_cast<void*>(rest));
    p.delta = static_cast<float*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(size_t(a->n_q) * size_t(a->heads) * 4, 256));
    switch (dtype) {
        case SPC_F32: return launch_bwd_f32(p, w.q, w.k, stream);
        case SPC_F16: return launch_bwd_f16(p, w.q, w.k, stream);
        case SPC_BF16: return launch_bwd_bf16(p, w.q, w.k, stream);
    }
    return fail(SPC_ERR_ARG, "unknown dtype %d", int(dtype));
}

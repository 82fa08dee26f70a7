// C ABI of the building-block operators: argument validation, workspace
// layout and the launch sequence of permute / unpermute and linear.  Host
// code only.
#include <initializer_list>

#include "../../include/moe.h"
#include "common.h"
#include "launch.h"

using namespace moe;

namespace {

bool at(const void* p, size_t a) { return p && ((uintptr_t)p % a) == 0; }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// ---------------------------------------------------------------- permute / unpermute
moe_status rows_args(const moe_config* cfg, const moe_sched* sched, int dtype, void* ws, size_t ws_bytes,
                     RowsArgs& a) {
    const moe_status s = moe_validate_config(cfg);
    if (s != MOE_OK) return s;
    if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16 && dtype != MOE_DT_FP32) return MOE_ERR_INVALID_ARG;
    if (!sched || !at(sched->row_of_slot, 4)) return MOE_ERR_INVALID_ARG;
    if (!at(ws, 256) || ws_bytes < 256) return MOE_ERR_WORKSPACE;
    a = {cfg->T, cfg->H, cfg->k, cfg->T * cfg->k, dtype, sched->row_of_slot, (int32_t*)ws};
    return MOE_OK;
}

// ---------------------------------------------------------------- linear
struct LinLayout {
    size_t lists[3], dz, part, sums, total;
};

moe_status lin_check(const moe_linear_config* c) {
    if (!c || c->M < 1 || c->M > (1 << 24) || c->N < 8 || c->N > (1 << 16) || c->N % 8 || c->K < 8 ||
        c->K > (1 << 16) || c->K % 8 || c->E < 0 || c->E > kMaxExperts || c->flags != 0)
        return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_FP16) return MOE_ERR_INVALID_ARG;
    if (c->act < 0 || c->act >= LIN_ACTS) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

LinLayout lin_layout(const moe_linear_config& c) {
    LinLayout L{};
    size_t n = 256;                                   // the device error word
    auto take = [&](size_t bytes) {
        const size_t here = n;
        n += up256(bytes);
        return here;
    };
    for (size_t& l : L.lists) l = take((size_t)(c.E + 1) * 4);
    L.dz = take(c.act == MOE_ACT_NONE ? 0 : (size_t)c.M * c.N * 2);
    const int rows = linear_dz_rows(c.M, c.E, c.N);
    L.part = take((((size_t)c.M + rows - 1) / rows + c.E) * c.N * 4);
    const size_t f = linear_part_floats(linear_plan(c.M, c.E, c.K, c.N, false), c.M, c.N);
    const size_t b = linear_part_floats(linear_plan(c.M, c.E, c.N, c.K, true), c.M, c.K);
    L.sums = take((f > b ? f : b) * 4);
    L.total = n;
    return L;
}

// Fills in the tiles of a call: the offsets, and a list for each set whose
// blocks do not find their tiles themselves, all lists in one launch.  C: the
// columns of its product's output.
struct Tiles {
    LinTiles* t;
    int C, tn;
};
int lin_tiles(const moe_linear_config& c, const int32_t* offsets, char* ws, const LinLayout& L,
              std::initializer_list<Tiles> sets, hipStream_t st) {
    LinPrefix p{};
    for (const Tiles& s : sets) {
        s.t->err = (int32_t*)ws;
        if (c.E == 0) continue;
        s.t->offsets = offsets;
        if (s.t->tm == 0 || linear_inline_tiles(*s.t, s.C, s.tn)) continue;
        s.t->list = (const int32_t*)(ws + L.lists[p.n]);
        p.t[p.n++] = *s.t;
    }
    return p.n ? launch_linear_prefix(p, st) : 0;
}

moe_status lin_common(const moe_linear_config* c, const int32_t* offsets, void* ws, size_t ws_bytes, LinLayout& L) {
    const moe_status s = lin_check(c);
    if (s != MOE_OK) return s;
    L = lin_layout(*c);
    if (!at(ws, 256) || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if (c->E > 0 ? !at(offsets, 4) : offsets != nullptr) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

bool at_or_null(const void* p) { return !p || at(p, 16); }

// whether an output is one of these (other) buffers
bool among(const void* out, std::initializer_list<const void*> others) {
    for (const void* p : others)
        if (out && p == out) return true;
    return false;
}

}  // namespace

extern "C" {

moe_status moe_permute_forward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* x,
                               void* xs, void* workspace, size_t workspace_bytes, void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(x, 16) || !at(xs, 16) || among(xs, {x, sched->row_of_slot})) return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_permute(a, x, xs, (hipStream_t)stream) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_permute_backward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* dxs,
                                void* dx, void* workspace, size_t workspace_bytes, void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(dxs, 16) || !at(dx, 16) || among(dx, {dxs, sched->row_of_slot})) return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_permute_bwd(a, dxs, dx, (hipStream_t)stream) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_unpermute_forward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* o,
                                 const void* residual, void* y, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(o, 16) || !at_or_null(residual) || !at(y, 16) || !at(sched->topk_w, 4) ||
        among(y, {o, sched->row_of_slot, sched->topk_w}))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_unpermute(a, o, sched->topk_w, residual, y, (hipStream_t)stream) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_unpermute_backward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* o,
                                  const void* dy, void* d_o, float* dw, float* d_logits, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(o, 16) || !at(dy, 16) || !at(d_o, 16) || !at(dw, 4) || !at(sched->topk_w, 4) ||
        (d_logits && (!at(d_logits, 4) || !at(sched->topk_idx, 4))))
        return MOE_ERR_INVALID_ARG;
    const void *row = sched->row_of_slot, *w = sched->topk_w, *idx = d_logits ? sched->topk_idx : nullptr;
    if (among(d_o, {o, dy, row, w, idx, dw, d_logits}) || among(dw, {o, dy, row, w, idx, d_logits}) ||
        among(d_logits, {o, dy, row, w, idx}))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_unpermute_bwd(a, o, dy, sched->topk_idx, sched->topk_w, cfg->E, d_o, dw, d_logits,
                                (hipStream_t)stream)
               ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_linear_workspace_size(const moe_linear_config* cfg, size_t* bytes) {
    const moe_status s = lin_check(cfg);
    if (s != MOE_OK) return s;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = lin_layout(*cfg).total;
    return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_config* c, const int32_t* offsets, const void* x, const void* w,
                              const void* bias, const void* residual, void* y, void* z, void* workspace,
                              size_t workspace_bytes, void* stream) {
    LinLayout L;
    const moe_status s = lin_common(c, offsets, workspace, workspace_bytes, L);
    if (s != MOE_OK) return s;
    if (!at(x, 16) || !at(w, 16) || !at(y, 16) || !at_or_null(bias) || !at_or_null(residual) || !at_or_null(z) ||
        among(y, {offsets, x, w, bias, z}) || among(z, {offsets, x, w, bias, residual}))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    LinPlan p = linear_plan(c->M, c->E, c->K, c->N, false);
    if (lin_tiles(*c, offsets, ws, L, {{&p.small, c->N, p.stream ? 32 : 128}, {&p.big, c->N, 256}}, st))
        return MOE_ERR_HIP;
    const LinFwdArgs a{{}, c->dtype, c->act, c->N, c->K, (const uint16_t*)x, (const uint16_t*)w,
                       (const uint16_t*)bias, (const uint16_t*)residual, (uint16_t*)y, (uint16_t*)z, 1,
                       (float*)(ws + L.sums)};
    return launch_linear_fwd(p, a, st) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_linear_backward(const moe_linear_config* c, const int32_t* offsets, const void* x, const void* w,
                               const void* z, const void* dy, void* dx, void* dw, void* db, void* workspace,
                               size_t workspace_bytes, void* stream) {
    LinLayout L;
    const moe_status s = lin_common(c, offsets, workspace, workspace_bytes, L);
    if (s != MOE_OK) return s;
    const bool none = c->act == MOE_ACT_NONE;
    if (!at(dy, 16) || (none ? !at_or_null(z) : !at(z, 16)) || (!dx && !dw && !db) || !at_or_null(dx) ||
        !at_or_null(dw) || !at_or_null(db) || (dx ? !at(w, 16) : !at_or_null(w)) || (dw ? !at(x, 16) : !at_or_null(x)) ||
        among(dx, {offsets, x, w, z, dy, dw, db}) || among(dw, {offsets, x, w, z, dy, db}) ||
        among(db, {offsets, x, w, z, dy}))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    LinPlan p = linear_plan(c->M, c->E, c->N, c->K, true);
    LinTiles strips{nullptr, nullptr, c->E, c->M, linear_dz_rows(c->M, c->E, c->N), nullptr};
    if (lin_tiles(*c, offsets, ws, L, {{&p.small, c->K, 128}, {&p.big, c->K, 256}, {&strips, c->N, 512}}, st))
        return MOE_ERR_HIP;
    uint16_t* dz = (uint16_t*)(ws + L.dz);
    float* part = db ? (float*)(ws + L.part) : nullptr;
    const LinDzArgs d{strips, c->dtype, c->act, c->N, (const uint16_t*)dy, (const uint16_t*)z, dz, part};
    if ((db || !none) && launch_linear_dz(d, st)) return MOE_ERR_HIP;
    const LinBwdArgs b{p.small, strips, c->dtype, c->N, c->K, none ? (const uint16_t*)dy : dz, (const uint16_t*)x,
                       (const uint16_t*)w, (uint16_t*)dx, (uint16_t*)dw, (uint16_t*)db, part,
                       (float*)(ws + L.sums), 0, 0, 0};
    if (launch_linear_bwd(p, b, st)) return MOE_ERR_HIP;
    return MOE_OK;
}

}  // extern "C"

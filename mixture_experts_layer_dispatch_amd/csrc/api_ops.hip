// C ABI of the building-block operators: argument validation, workspace
// layout and the launch sequence of permute / unpermute and linear.  Host
// code only.
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
    size_t tiles, big, rows32, dz, part, total;
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
    const size_t pre = (size_t)(c.E + 1) * 4;
    L.tiles = take(pre);
    L.big = take(pre);
    L.rows32 = take(pre);
    L.dz = take(c.act == MOE_ACT_NONE ? 0 : (size_t)c.M * c.N * 2);
    L.part = take(((size_t)(c.M + kLinDzRows - 1) / kLinDzRows + c.E) * c.N * 4);
    L.total = n;
    return L;
}

GroupRows lin_group(const moe_linear_config& c, const int32_t* offsets, char* ws) {
    GroupRows g{};
    g.E = c.E > 0 ? c.E : 1;
    g.rows = c.M;
    g.err = (int32_t*)ws;
    if (c.E > 0) g.offsets = offsets;
    else g.dense_rows = c.M;
    return g;
}

// The tile forms of one product and, for groups, the prefixes of its tiles
// (and of the kLinDzRows-row tiles, if wanted) in one launch.
int lin_tiles(const moe_linear_config& c, const int32_t* offsets, const LinForm& f, int32_t* tiles, int32_t* big,
              int32_t* rows32, GroupRows& g, hipStream_t st) {
    if (c.E == 0) {
        g.tm = f.dense_big ? 256 : f.small;
        return 0;
    }
    g.tm = f.small;
    g.tile_off = tiles;
    LinPrefix p{1, {f.small}, {0}, {f.split ? 256 : INT32_MAX}, {tiles}};
    auto add = [&](int tm, int lo, int32_t* out) {
        p.tm[p.n] = tm;
        p.lo[p.n] = lo;
        p.hi[p.n] = INT32_MAX;
        p.out[p.n++] = out;
    };
    if (f.split) {
        add(256, 256, big);
        g.tile_big = big;
    }
    if (rows32) add(kLinDzRows, 0, rows32);
    return launch_linear_prefix(offsets, c.E, c.M, p, g.err, st);
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

}  // namespace

extern "C" {

moe_status moe_permute_forward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* x,
                               void* xs, void* workspace, size_t workspace_bytes, void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(x, 16) || !at(xs, 16)) return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_permute(a, x, xs, (hipStream_t)stream) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_permute_backward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* dxs,
                                void* dx, void* workspace, size_t workspace_bytes, void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(dxs, 16) || !at(dx, 16)) return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    return launch_permute_bwd(a, dxs, dx, (hipStream_t)stream) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_unpermute_forward(const moe_config* cfg, const moe_sched* sched, moe_dtype dtype, const void* o,
                                 const void* residual, void* y, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    RowsArgs a;
    const moe_status s = rows_args(cfg, sched, dtype, workspace, workspace_bytes, a);
    if (s != MOE_OK) return s;
    if (!at(o, 16) || !at_or_null(residual) || !at(y, 16) || !at(sched->topk_w, 4)) return MOE_ERR_INVALID_ARG;
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
    if (!at(x, 16) || !at(w, 16) || !at(y, 16) || !at_or_null(bias) || !at_or_null(residual) || !at_or_null(z))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    LinFwdArgs a{lin_group(*c, offsets, ws), c->dtype, c->act, c->N, c->K, (const uint16_t*)x, (const uint16_t*)w,
                 (const uint16_t*)bias, (const uint16_t*)residual, (uint16_t*)y, (uint16_t*)z};
    int32_t *tiles = (int32_t*)(ws + L.tiles), *big = (int32_t*)(ws + L.big);
    const LinForm f = linear_form(c->M, c->E, c->N, false);
    a.stream = f.stream;
    if (lin_tiles(*c, offsets, f, tiles, big, nullptr, a.g, st)) return MOE_ERR_HIP;
    return launch_linear_fwd(a, st) ? MOE_ERR_HIP : MOE_OK;
}

moe_status moe_linear_backward(const moe_linear_config* c, const int32_t* offsets, const void* x, const void* w,
                               const void* z, const void* dy, void* dx, void* dw, void* db, void* workspace,
                               size_t workspace_bytes, void* stream) {
    LinLayout L;
    const moe_status s = lin_common(c, offsets, workspace, workspace_bytes, L);
    if (s != MOE_OK) return s;
    const bool none = c->act == MOE_ACT_NONE;
    if (!at(dy, 16) || (none ? !at_or_null(z) : !at(z, 16)) || (!dx && !dw && !db) || !at_or_null(dx) ||
        !at_or_null(dw) || !at_or_null(db) || (dx ? !at(w, 16) : !at_or_null(w)) || (dw ? !at(x, 16) : !at_or_null(x)))
        return MOE_ERR_INVALID_ARG;
    if (!device_ok()) return MOE_ERR_UNSUPPORTED_DEVICE;
    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const GroupRows g = lin_group(*c, offsets, ws);
    int32_t *tiles = (int32_t*)(ws + L.tiles), *big = (int32_t*)(ws + L.big), *rows32 = (int32_t*)(ws + L.rows32);
    GroupRows gx = g;                                 // dx's tiles
    if (lin_tiles(*c, offsets, linear_form(c->M, c->E, c->K, true), tiles, big, rows32, gx, st)) return MOE_ERR_HIP;
    uint16_t* dz = (uint16_t*)(ws + L.dz);
    LinDzArgs d{g, c->dtype, c->act, c->N, (const uint16_t*)dy, (const uint16_t*)z, dz,
                db ? (float*)(ws + L.part) : nullptr};
    if (c->E > 0) d.g.tile_off = rows32;
    if ((db || !none) && launch_linear_dz(d, st)) return MOE_ERR_HIP;
    const LinBwdArgs b{gx, d.g, c->dtype, c->N, c->K, none ? (const uint16_t*)dy : dz, (const uint16_t*)x,
                       (const uint16_t*)w, (uint16_t*)dx, (uint16_t*)dw, (uint16_t*)db, d.part,
                       linear_dw_form(c->M, c->E, c->N, c->K), 0, 0};
    if (launch_linear_bwd(b, st)) return MOE_ERR_HIP;
    return MOE_OK;
}

}  // extern "C"

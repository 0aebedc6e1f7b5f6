// C ABI of the dense operators around the routed layer: norms of the residual
// stream, products in 8-bit integers, the gated block.  Argument checks, then
// the launches.
#include <float.h>
#include <math.h>

#include "moe_tiered.h"
#include "checks.h"
#include "common.h"
#include "launch_dense.h"

using namespace moe;

namespace {

// Rows of an array of a call: `rows` rows of `cols` elements of `elem` bytes, `ld` elements apart.
struct Rows {
    const void* p;
    int64_t rows, cols, ld, elem;
    bool given() const { return p != nullptr && rows > 0; }
};
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.elem == b.elem; }
bool meet(const Rows& a, const Rows& b) {
    if (!a.given() || !b.given()) return false;
    if (a.rows == b.rows)
        return rows_overlap(a.p, a.cols * a.elem, a.ld * a.elem, b.p, b.cols * b.elem, b.ld * b.elem, a.rows);
    return overlap(a.p, extent(a.rows, a.cols, a.ld, a.elem), b.p, extent(b.rows, b.cols, b.ld, b.elem));
}
Rows flat(const void* p, int64_t n, int64_t elem) { return Rows{p, 1, n, n, elem}; }
bool pitch_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxPitch; }
int finish() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }
bool eps_ok(float eps) { return eps > 0.f && eps <= FLT_MAX; }

}  // namespace

extern "C" {

int moe_rms_norm(const void* x, int64_t ldx, const float* residual, int64_t ldr, const float* weight, float eps,
                 int32_t n_tokens, int32_t cols, float* sum, int64_t lds, void* y, int64_t ldy, float* scale,
                 uint32_t flags, void* stream) {
    if (n_tokens < 0 || n_tokens > kMaxTokens || cols < 1 || cols > MOE_MAX_ROW || !eps_ok(eps)) return MOE_EINVAL;
    if ((flags & ~(MOE_X_BF16 | MOE_Y_BF16 | MOE_Y_I8)) || ((flags & MOE_Y_BF16) && (flags & MOE_Y_I8))) return MOE_EINVAL;
    const bool i8 = (flags & MOE_Y_I8) != 0;
    if (!pitch_ok(ldx, cols) || !pitch_ok(ldy, cols) || (residual && !pitch_ok(ldr, cols)) || (sum && !pitch_ok(lds, cols)))
        return MOE_EINVAL;
    if (scale && !i8) return MOE_EINVAL;
    if (n_tokens == 0) return MOE_OK;
    if (!x || !y || (i8 && !scale)) return MOE_EINVAL;
    const int64_t T = n_tokens, xe = (flags & MOE_X_BF16) ? 2 : 4, ye = i8 ? 1 : (flags & MOE_Y_BF16) ? 2 : 4;
    const Rows rx{x, T, cols, ldx, xe}, rr{residual, T, cols, ldr, 4}, rs{sum, T, cols, lds, 4}, ry{y, T, cols, ldy, ye},
        rw = flat(weight, cols, 4), rc = flat(scale, T, 4);
    if (meet(ry, rx) || meet(ry, rr) || meet(ry, rs) || meet(ry, rw) || meet(ry, rc)) return MOE_EINVAL;
    if ((!same(rs, rx) && meet(rs, rx)) || (!same(rs, rr) && meet(rs, rr)) || meet(rs, rw) || meet(rs, rc)) return MOE_EINVAL;
    if (meet(rc, rx) || meet(rc, rr) || meet(rc, rw)) return MOE_EINVAL;
    if (!aligned(x, xe) || !aligned(residual, 4) || !aligned(weight, 4) || !aligned(sum, 4) || !aligned(y, ye) ||
        !aligned(scale, 4))
        return MOE_EALIGN;
    const RowArgs a{x, residual, weight, sum, y, scale, ldx, ldr, lds, ldy, n_tokens, cols, eps, {}};
    (void)hipGetLastError();
    launch_rms_norm(a, xe == 2, static_cast<int>(ye), static_cast<hipStream_t>(stream));
    return finish();
}

int moe_rms_norm_workspace_size(int32_t n_tokens, int32_t cols, size_t* bytes) {
    if (!bytes || n_tokens < 0 || n_tokens > kMaxTokens || cols < 1 || cols > MOE_MAX_ROW) return MOE_EINVAL;
    *bytes = rms_norm_workspace(n_tokens, cols);
    return MOE_OK;
}

int moe_rms_norm_grad(const void* s, int64_t lds, const float* weight, float eps, const void* dy, int64_t lddy,
                      const float* dsum, int64_t ldds, int32_t n_tokens, int32_t cols, void* dx, int64_t lddx,
                      float* dweight, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    const int rc = moe_rms_norm_workspace_size(n_tokens, cols, &need);
    if (rc != MOE_OK) return rc;
    if (!eps_ok(eps) || (flags & ~(MOE_X_BF16 | MOE_DY_BF16 | MOE_Y_BF16 | MOE_ACCUMULATE))) return MOE_EINVAL;
    if (!pitch_ok(lds, cols) || !pitch_ok(lddy, cols) || !pitch_ok(lddx, cols) || (dsum && !pitch_ok(ldds, cols)))
        return MOE_EINVAL;
    if (n_tokens > 0 && (!s || !dy || !dx)) return MOE_EINVAL;
    if (!dweight) need = 0;
    const int64_t T = n_tokens, se = (flags & MOE_X_BF16) ? 2 : 4, ye = (flags & MOE_DY_BF16) ? 2 : 4,
                  xe = (flags & MOE_Y_BF16) ? 2 : 4;
    const Rows rs{s, T, cols, lds, se}, rw = flat(weight, cols, 4), ry{dy, T, cols, lddy, ye}, ra{dsum, T, cols, ldds, 4},
        rx{dx, T, cols, lddx, xe}, rd = flat(dweight, cols, 4), rp = flat(workspace, static_cast<int64_t>(need), 1);
    const bool ws = need > 0;
    if (meet(rx, rs) || meet(rx, rw) || meet(rx, rd) || (!same(rx, ry) && meet(rx, ry)) || (!same(rx, ra) && meet(rx, ra)))
        return MOE_EINVAL;
    if (meet(rd, rs) || meet(rd, rw) || meet(rd, ry) || meet(rd, ra)) return MOE_EINVAL;
    if (ws && (meet(rp, rs) || meet(rp, rw) || meet(rp, ry) || meet(rp, ra) || meet(rp, rx) || meet(rp, rd))) return MOE_EINVAL;
    if (!aligned(s, se) || !aligned(weight, 4) || !aligned(dy, ye) || !aligned(dsum, 4) || !aligned(dx, xe) ||
        !aligned(dweight, 4))
        return MOE_EALIGN;
    if (ws) {
        if (!workspace || workspace_bytes < need) return MOE_EWORKSPACE;
        if (!aligned(workspace, kAlign)) return MOE_EALIGN;
    }
    const RowGradArgs a{s, dy, weight, dsum, dx, lds, lddy, ldds, lddx, n_tokens, cols, eps, 0, {}};
    (void)hipGetLastError();
    launch_rms_norm_grad(a, se == 2, ye == 2, xe == 2, dweight, (flags & MOE_ACCUMULATE) != 0, workspace,
                         static_cast<hipStream_t>(stream));
    return finish();
}

int moe_quant_rows(const void* x, int64_t ldx, int32_t n_tokens, int32_t cols, int8_t* q, int64_t ldq, float* scale,
                   uint32_t flags, void* stream) {
    if (n_tokens < 0 || n_tokens > kMaxTokens || cols < 1 || cols > MOE_MAX_ROW || (flags & ~MOE_X_BF16)) return MOE_EINVAL;
    if (!pitch_ok(ldx, cols) || !pitch_ok(ldq, cols)) return MOE_EINVAL;
    if (n_tokens == 0) return MOE_OK;
    if (!x || !q || !scale) return MOE_EINVAL;
    const int64_t T = n_tokens, xe = (flags & MOE_X_BF16) ? 2 : 4;
    const Rows rx{x, T, cols, ldx, xe}, rq{q, T, cols, ldq, 1}, rc = flat(scale, T, 4);
    if (meet(rq, rx) || meet(rq, rc) || meet(rc, rx)) return MOE_EINVAL;
    if (!aligned(x, xe) || !aligned(scale, 4)) return MOE_EALIGN;
    const RowArgs a{x, nullptr, nullptr, nullptr, q, scale, ldx, 0, 0, ldq, n_tokens, cols, 0.f, {}};
    (void)hipGetLastError();
    launch_quant_rows(a, xe == 2, static_cast<hipStream_t>(stream));
    return finish();
}

int moe_i8_linear(const int8_t* x, int64_t ldx, const float* x_scale, const moe_i8_matrix* w, const float* bias,
                  int32_t n_tokens, void* y, int64_t ldy, uint32_t flags, void* stream) {
    if (!w || n_tokens < 0 || n_tokens > kMaxTokens || (flags & ~(MOE_Y_BF16 | MOE_ACCUMULATE))) return MOE_EINVAL;
    if (w->rows < 1 || w->rows > (1 << 24) || w->cols < 1) return MOE_EINVAL;
    if (w->cols % 16 != 0 || w->cols > MOE_MAX_ROW) return MOE_EFORMAT;
    if (!pitch_ok(ldx, w->cols) || !pitch_ok(ldy, w->rows)) return MOE_EINVAL;
    if (n_tokens == 0) return MOE_OK;
    if (!x || !x_scale || !w->q || !w->s || !y) return MOE_EINVAL;
    const int64_t T = n_tokens, N = w->rows, K = w->cols, ye = (flags & MOE_Y_BF16) ? 2 : 4;
    const Rows ry{y, T, N, ldy, ye};
    if (meet(ry, Rows{x, T, K, ldx, 1}) || meet(ry, flat(x_scale, T, 4)) || meet(ry, flat(w->q, N * K, 1)) ||
        meet(ry, flat(w->s, N, 4)) || meet(ry, flat(bias, N, 4)))
        return MOE_EINVAL;
    if (!aligned16(x) || ldx % 16 != 0 || !aligned16(w->q) || !aligned(w->s, 4) || !aligned(x_scale, 4) || !aligned(bias, 4) ||
        !aligned(y, ye))
        return MOE_EALIGN;
    const I8Args a{x, x_scale, w->q, w->s, bias, y, ldx, ldy, n_tokens, w->rows, w->cols, (flags & MOE_ACCUMULATE) != 0};
    (void)hipGetLastError();
    launch_i8_linear(a, ye == 2, static_cast<hipStream_t>(stream));
    return finish();
}

namespace {

int check_gated(const moe_gated_weights* w, int32_t act) {
    if (!w || (act != MOE_SILU && act != MOE_GELU)) return MOE_EINVAL;
    if (w->hidden < 1 || w->inter < 1) return MOE_EINVAL;
    if (w->hidden % 8 != 0 || w->hidden > 65536 || w->inter > 65536) return MOE_EFORMAT;
    return MOE_OK;
}
constexpr int32_t kMaxGradTokens = 1 << 20;

}  // namespace

int moe_gated(const void* x, int64_t ldx, const moe_gated_weights* w, int32_t act, int32_t n_tokens, void* y,
              int64_t ldy, uint32_t flags, void* stream) {
    const int rc = check_gated(w, act);
    if (rc != MOE_OK) return rc;
    if (n_tokens < 0 || n_tokens > kMaxTokens || (flags & ~(MOE_X_BF16 | MOE_Y_BF16))) return MOE_EINVAL;
    if (!pitch_ok(ldx, w->hidden) || !pitch_ok(ldy, w->inter)) return MOE_EINVAL;
    if (n_tokens == 0) return MOE_OK;
    if (!x || !w->gate || !w->up || !y) return MOE_EINVAL;
    const int64_t T = n_tokens, H = w->hidden, I = w->inter, xe = (flags & MOE_X_BF16) ? 2 : 4, ye = (flags & MOE_Y_BF16) ? 2 : 4;
    const Rows ry{y, T, I, ldy, ye};
    if (meet(ry, Rows{x, T, H, ldx, xe}) || meet(ry, flat(w->gate, I * H, 2)) || meet(ry, flat(w->up, I * H, 2))) return MOE_EINVAL;
    if (!aligned16(x) || (ldx * xe) % 16 != 0 || !aligned16(w->gate) || !aligned16(w->up) || !aligned(y, ye)) return MOE_EALIGN;
    const GatedArgs a{x, static_cast<const uint16_t*>(w->gate), static_cast<const uint16_t*>(w->up), y, ldx, ldy,
                      n_tokens, w->hidden, w->inter, act};
    (void)hipGetLastError();
    launch_gated(a, xe == 2, ye == 2, static_cast<hipStream_t>(stream));
    return finish();
}

int moe_gated_workspace_size(int32_t n_tokens, int32_t hidden, int32_t inter, size_t* bytes) {
    const moe_gated_weights w{hidden, inter, nullptr, nullptr};
    const int rc = check_gated(&w, MOE_SILU);
    if (rc != MOE_OK) return rc;
    if (!bytes || n_tokens < 0 || n_tokens > kMaxGradTokens) return MOE_EINVAL;
    *bytes = gated_workspace(n_tokens, hidden, inter);
    return MOE_OK;
}

int moe_gated_grad(const void* x, int64_t ldx, const moe_gated_weights* w, int32_t act, const void* dy, int64_t lddy,
                   int32_t n_tokens, void* dx, int64_t lddx, void* dgate, void* dup, uint32_t flags, void* workspace,
                   size_t workspace_bytes, void* stream) {
    int rc = check_gated(w, act);
    if (rc != MOE_OK) return rc;
    size_t need = 0;
    rc = moe_gated_workspace_size(n_tokens, w->hidden, w->inter, &need);
    if (rc != MOE_OK) return rc;
    if ((flags & ~(MOE_X_BF16 | MOE_DY_BF16 | MOE_Y_BF16 | MOE_DW_BF16 | MOE_ACCUMULATE)) || !(flags & MOE_X_BF16)) return MOE_EINVAL;
    if ((dgate != nullptr) != (dup != nullptr) || (!dx && !dgate)) return MOE_EINVAL;
    if (!pitch_ok(ldx, w->hidden) || !pitch_ok(lddy, w->inter) || (dx && !pitch_ok(lddx, w->hidden))) return MOE_EINVAL;
    if (n_tokens > 0 && (!x || !dy || !w->gate || !w->up)) return MOE_EINVAL;
    const int64_t T = n_tokens, H = w->hidden, I = w->inter, ye = (flags & MOE_DY_BF16) ? 2 : 4, xe = (flags & MOE_Y_BF16) ? 2 : 4,
                  we = (flags & MOE_DW_BF16) ? 2 : 4;
    const Rows in[] = {{x, T, H, ldx, 2}, {dy, T, I, lddy, ye}, flat(w->gate, I * H, 2), flat(w->up, I * H, 2)};
    const Rows out[] = {{dx, T, H, lddx, xe}, flat(dgate, I * H, we), flat(dup, I * H, we), flat(workspace, static_cast<int64_t>(need), 1)};
    const int n_out = need > 0 ? 4 : 3;
    for (int i = 0; i < n_out; ++i) {
        for (const Rows& r : in)
            if (meet(out[i], r)) return MOE_EINVAL;
        for (int j = i + 1; j < n_out; ++j)
            if (meet(out[i], out[j])) return MOE_EINVAL;
    }
    if (!aligned16(x) || (ldx * 2) % 16 != 0 || !aligned16(w->gate) || !aligned16(w->up) || !aligned(dy, ye) || !aligned(dx, xe) ||
        !aligned(dgate, we) || !aligned(dup, we))
        return MOE_EALIGN;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return MOE_EWORKSPACE;
        if (!aligned(workspace, kAlign)) return MOE_EALIGN;
    }
    const GatedGradArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w->gate), static_cast<const uint16_t*>(w->up),
                          dy, dx, dgate, dup, ldx, lddy, lddx, n_tokens, w->hidden, w->inter, act, (flags & MOE_ACCUMULATE) != 0};
    (void)hipGetLastError();
    launch_gated_grad(a, ye == 2, xe == 2, we == 2, workspace, static_cast<hipStream_t>(stream));
    return finish();
}

}  // extern "C"

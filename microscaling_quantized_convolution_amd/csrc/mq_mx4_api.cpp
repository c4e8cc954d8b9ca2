// mq_mx4_api.cpp -- C ABI of the microscaled 4-bit linear layers: host-side validation, and the
// launches that make up a call.
//
// As in mq_api.cpp, every call validates its arguments on the host, then enqueues kernels on the
// caller's stream; nothing here allocates, synchronizes or reads device memory.
#include "mq_mx4.hpp"

namespace {

constexpr int32_t kMaxDim = 1 << 30;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

size_t pieces(int32_t cols) { return ((size_t)cols + mq::kMxPiece - 1) / mq::kMxPiece; }

// Codes and scales of a quantized matrix in a workspace, each from a multiple of 256 bytes.
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t held_bytes(int32_t rows, int32_t cols)
{
    return round256(pieces(cols) * rows * 128) + round256(pieces(cols) * rows * 8);
}

bool matrix_ok(const mq_matrix *m)
{
    if (!m || m->rows < 0 || m->cols < 0 || m->stride < m->cols) return false;
    if (m->dtype != MQ_F16 && m->dtype != MQ_BF16 && m->dtype != MQ_F32) return false;
    return (m->data || m->rows == 0 || m->cols == 0) && aligned(m->data, m->dtype == MQ_F32 ? 4 : 2);
}

bool held_ok(const mq_mx4 *q)
{
    return q && q->rows >= 0 && q->cols >= 0 && aligned(q->codes, 16) && aligned(q->scales, 8) &&
           ((q->codes && q->scales) || q->rows == 0 || q->cols == 0);
}

bool round_ok(int32_t rnd) { return rnd == MQ_RNE || rnd == MQ_SR; }

bool fits(int32_t a, int32_t b = 0, int32_t c = 0) { return a < kMaxDim && b < kMaxDim && c < kMaxDim; }

bool is(const mq_matrix *m, int32_t rows, int32_t cols) { return m->rows == rows && m->cols == cols; }
bool is(const mq_mx4 *q, int32_t rows, int32_t cols) { return q->rows == rows && q->cols == cols; }

mq::MatView view(const mq_matrix *m)
{
    return m ? mq::MatView{m->data, m->stride, m->dtype} : mq::MatView{nullptr, 0, 0};
}
mq::Mx4View view(const mq_mx4 *q)
{
    return q ? mq::Mx4View{q->codes, q->scales, q->rows, q->cols} : mq::Mx4View{nullptr, nullptr, 0, 0};
}

mq_status launched(hipError_t e)
{
    return e == hipSuccess ? MQ_OK : (e == hipErrorInvalidValue ? MQ_ERR_UNSUPPORTED : MQ_ERR_LAUNCH);
}

// The next quantized matrix of a workspace.
mq::Mx4View take(uint8_t *&at, int32_t rows, int32_t cols)
{
    const size_t codes = round256(pieces(cols) * rows * 128);
    const mq::Mx4View q = {at, at + codes, rows, cols};
    at += held_bytes(rows, cols);
    return q;
}

mq::Mx4QuantArgs quantize_args(const mq_matrix *x, int32_t rnd, uint64_t seed)
{
    mq::Mx4QuantArgs a = {};
    a.x = view(x);
    a.rows = x->rows;
    a.cols = x->cols;
    a.sr = rnd == MQ_SR;
    a.seed_lo = (uint32_t)seed;
    a.seed_hi = (uint32_t)(seed >> 32);
    return a;
}

mq::Mx4MatmulArgs matmul_args(const mq::Mx4View &a, const mq::Mx4View &b, const mq_matrix *y)
{
    mq::Mx4MatmulArgs m = {};
    m.a[0][0] = a;
    m.b[0][0] = b;
    m.y[0] = view(y);
    m.jobs = 1;
    m.m = y->rows;
    m.n = y->cols;
    m.pieces[0] = a.pieces();
    return m;
}

// A layer's input: quantized along its rows into the workspace (unless the product does that) and
// along its columns into x_col, if given.
mq_status quantize_input(const mq_matrix *x, const mq_mx4 *x_col, bool inside, uint8_t *&at, mq::Mx4View &row, hipStream_t stream)
{
    mq::Mx4QuantArgs q = quantize_args(x, MQ_RNE, 0);
    row = take(at, x->rows, x->cols);
    if (!inside) q.row = row;
    q.col = view(x_col);
    return inside || x->rows == 0 || x->cols == 0 ? MQ_OK : launched(mq::launch_mx4_quantize(q, stream));
}

bool sizes_ok(int32_t a, int32_t b, int32_t c) { return a >= 0 && b >= 0 && c >= 0 && fits(a, b, c); }

} // namespace

extern "C" {

size_t mq_mx4_codes_bytes(int32_t rows, int32_t cols)
{
    return rows < 0 || cols < 0 ? 0 : pieces(cols) * rows * 128;
}

size_t mq_mx4_scales_bytes(int32_t rows, int32_t cols)
{
    return rows < 0 || cols < 0 ? 0 : pieces(cols) * rows * 8;
}

mq_status mq_mx4_quantize(const mq_matrix *x, const mq_mx4 *row, const mq_mx4 *col, int32_t rnd,
                          uint64_t seed, hipStream_t stream)
{
    if (!matrix_ok(x) || (!row && !col) || (row && !held_ok(row)) || (col && !held_ok(col)) || !round_ok(rnd))
        return MQ_ERR_ARG;
    if ((row && !is(row, x->rows, x->cols)) || (col && !is(col, x->cols, x->rows))) return MQ_ERR_SHAPE;
    if (!fits(x->rows, x->cols)) return MQ_ERR_UNSUPPORTED;
    if (x->rows == 0 || x->cols == 0) return MQ_OK;
    mq::Mx4QuantArgs a = quantize_args(x, rnd, seed);
    a.row = view(row);
    a.col = view(col);
    return launched(mq::launch_mx4_quantize(a, stream));
}

mq_status mq_mx4_dequantize(const mq_mx4 *q, const mq_matrix *out, hipStream_t stream)
{
    if (!held_ok(q) || !matrix_ok(out)) return MQ_ERR_ARG;
    if (!is(q, out->rows, out->cols)) return MQ_ERR_SHAPE;
    if (!fits(q->rows, q->cols)) return MQ_ERR_UNSUPPORTED;
    return launched(mq::launch_mx4_dequantize(view(q), view(out), stream));
}

size_t mq_mx4_matmul_workspace_bytes(int32_t, int32_t, int32_t) { return 0; }

mq_status mq_mx4_matmul(const mq_mx4 *a, const mq_mx4 *b, const mq_matrix *y, void *ws,
                        size_t, hipStream_t stream)
{
    if (!held_ok(a) || !held_ok(b) || !matrix_ok(y) || !aligned(ws, 16)) return MQ_ERR_ARG;
    if (a->cols != b->cols || !is(y, a->rows, b->rows)) return MQ_ERR_SHAPE;
    if (!fits(a->rows, b->rows, a->cols)) return MQ_ERR_UNSUPPORTED;
    return launched(mq::launch_mx4_matmul(matmul_args(view(a), view(b), y), stream));
}

size_t mq_mx4_linear_workspace_bytes(int32_t m, int32_t n, int32_t k)
{
    return sizes_ok(m, n, k) ? held_bytes(m, k) : 0;
}

mq_status mq_mx4_linear(const mq_matrix *x, const mq_mx4 *w, const mq_matrix *y,
                        const mq_mx4 *x_col, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!matrix_ok(x) || !held_ok(w) || !matrix_ok(y) || (x_col && !held_ok(x_col)) || !aligned(ws, 16))
        return MQ_ERR_ARG;
    if (x->cols != w->cols || !is(y, x->rows, w->rows) || (x_col && !is(x_col, x->cols, x->rows)))
        return MQ_ERR_SHAPE;
    if (!fits(x->rows, x->cols, w->rows)) return MQ_ERR_UNSUPPORTED;
    const size_t need = mq_mx4_linear_workspace_bytes(x->rows, w->rows, x->cols);
    if (need && (!ws || ws_bytes < need)) return MQ_ERR_WORKSPACE;
    mq::Mx4View row;
    uint8_t *at = static_cast<uint8_t *>(ws);
    const bool inside = !x_col && mq::mx4_quantizes_rows(x->rows, w->rows, x->cols);
    const mq_status st = quantize_input(x, x_col, inside, at, row, stream);
    if (st != MQ_OK) return st;
    mq::Mx4MatmulArgs a = matmul_args(row, view(w), y);
    if (inside) a.x = view(x), a.cols = x->cols;
    return launched(mq::launch_mx4_matmul(a, stream));
}

size_t mq_mx4_linear_backward_workspace_bytes(int32_t m, int32_t n, int32_t k)
{
    return sizes_ok(m, n, k) ? held_bytes(m, n) + held_bytes(n, m) : 0;
}

mq_status mq_mx4_linear_backward(const mq_matrix *dy, const mq_mx4 *x_col, const mq_mx4 *w_col,
                                 const mq_matrix *dx, const mq_matrix *dw, int32_t rnd,
                                 uint64_t seed, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!matrix_ok(dy) || (!dx && !dw) || !round_ok(rnd) || !aligned(ws, 16)) return MQ_ERR_ARG;
    if ((dx && (!matrix_ok(dx) || !held_ok(w_col))) || (dw && (!matrix_ok(dw) || !held_ok(x_col)))) return MQ_ERR_ARG;
    const int32_t m = dy->rows, n = dy->cols, k = dx ? dx->cols : dw->cols;
    if (dx && (!is(dx, m, k) || !is(w_col, k, n))) return MQ_ERR_SHAPE;
    if (dw && (!is(dw, n, k) || !is(x_col, k, m))) return MQ_ERR_SHAPE;
    if (!fits(m, n, k)) return MQ_ERR_UNSUPPORTED;
    const size_t need = mq_mx4_linear_backward_workspace_bytes(m, n, k);
    if (need && (!ws || ws_bytes < need)) return MQ_ERR_WORKSPACE;
    uint8_t *at = static_cast<uint8_t *>(ws);
    mq::Mx4QuantArgs q = quantize_args(dy, rnd, seed);
    const mq::Mx4View row = take(at, m, n), col = take(at, n, m);
    if (dx) q.row = row;
    if (dw) q.col = col;
    mq_status st = MQ_OK;
    if (m && n) st = launched(mq::launch_mx4_quantize(q, stream));
    if (st == MQ_OK && dx) st = launched(mq::launch_mx4_matmul(matmul_args(row, view(w_col), dx), stream));
    if (st == MQ_OK && dw) st = launched(mq::launch_mx4_matmul(matmul_args(col, view(x_col), dw), stream));
    return st;
}

size_t mq_mx4_gated_workspace_bytes(int32_t m, int32_t f, int32_t k)
{
    return sizes_ok(m, f, k) ? held_bytes(m, k) : 0;
}

mq_status mq_mx4_gated(const mq_matrix *x, const mq_mx4 *wg, const mq_mx4 *wu, const mq_matrix *h,
                       const mq_matrix *g, const mq_matrix *u, const mq_mx4 *x_col, void *ws,
                       size_t ws_bytes, hipStream_t stream)
{
    if (!matrix_ok(x) || !held_ok(wg) || !held_ok(wu) || !matrix_ok(h) || (x_col && !held_ok(x_col)) ||
        !g != !u || (g && (!matrix_ok(g) || !matrix_ok(u))) || !aligned(ws, 16))
        return MQ_ERR_ARG;
    const int32_t m = x->rows, k = x->cols, f = h->cols;
    if (!is(wg, f, k) || !is(wu, f, k) || h->rows != m || (x_col && !is(x_col, k, m))) return MQ_ERR_SHAPE;
    if (g && (!is(g, m, f) || !is(u, m, f) || g->dtype != h->dtype || u->dtype != h->dtype)) return MQ_ERR_SHAPE;
    if (!fits(m, f, k)) return MQ_ERR_UNSUPPORTED;
    const size_t need = mq_mx4_gated_workspace_bytes(m, f, k);
    if (need && (!ws || ws_bytes < need)) return MQ_ERR_WORKSPACE;
    mq::Mx4View row;
    uint8_t *at = static_cast<uint8_t *>(ws);
    const bool inside = !x_col && mq::mx4_takes_rows(m, f, true) && mq::mx4_quantizes_rows(m, f, k);
    const mq_status st = quantize_input(x, x_col, inside, at, row, stream);
    if (st != MQ_OK) return st;
    mq::Mx4MatmulArgs a = matmul_args(row, view(wg), h);
    if (inside) a.x = view(x), a.cols = k;
    a.b[0][1] = view(wu);
    a.g = view(g);
    a.u = view(u);
    a.gated = true;
    return launched(mq::launch_mx4_matmul(a, stream));
}

size_t mq_mx4_gated_backward_workspace_bytes(int32_t m, int32_t f, int32_t k)
{
    return sizes_ok(m, f, k) ? 2 * (held_bytes(m, f) + held_bytes(f, m)) : 0;
}

mq_status mq_mx4_gated_backward(const mq_matrix *dh, const mq_matrix *g, const mq_matrix *u,
                                const mq_mx4 *x_col, const mq_mx4 *wg_col, const mq_mx4 *wu_col,
                                const mq_matrix *dx, const mq_matrix *dwg, const mq_matrix *dwu,
                                int32_t rnd, uint64_t seed, void *ws, size_t ws_bytes,
                                hipStream_t stream)
{
    if (!matrix_ok(dh) || !matrix_ok(g) || !matrix_ok(u) || !dwg != !dwu || (!dx && !dwg) || !round_ok(rnd) ||
        !aligned(ws, 16))
        return MQ_ERR_ARG;
    if (dx && (!matrix_ok(dx) || !held_ok(wg_col) || !held_ok(wu_col))) return MQ_ERR_ARG;
    if (dwg && (!matrix_ok(dwg) || !matrix_ok(dwu) || !held_ok(x_col))) return MQ_ERR_ARG;
    const int32_t m = dh->rows, f = dh->cols, k = dx ? dx->cols : dwg->cols;
    if (!is(g, m, f) || !is(u, m, f) || g->dtype != dh->dtype || u->dtype != dh->dtype) return MQ_ERR_SHAPE;
    if (dx && (!is(dx, m, k) || !is(wg_col, k, f) || !is(wu_col, k, f))) return MQ_ERR_SHAPE;
    if (dwg && (!is(dwg, f, k) || !is(dwu, f, k) || !is(x_col, k, m) || dwg->dtype != dwu->dtype)) return MQ_ERR_SHAPE;
    if (!fits(m, f, k)) return MQ_ERR_UNSUPPORTED;
    const size_t need = mq_mx4_gated_backward_workspace_bytes(m, f, k);
    if (need && (!ws || ws_bytes < need)) return MQ_ERR_WORKSPACE;
    uint8_t *at = static_cast<uint8_t *>(ws);
    mq::Mx4QuantArgs q = quantize_args(dh, rnd, seed);
    q.g = view(g);
    q.u = view(u);
    const mq::Mx4View row = take(at, m, f), row2 = take(at, m, f), col = take(at, f, m), col2 = take(at, f, m);
    if (dx) q.row = row, q.row2 = row2;
    if (dwg) q.col = col, q.col2 = col2;
    mq_status st = MQ_OK;
    if (m && f) st = launched(mq::launch_mx4_gradients(q, stream));
    if (st == MQ_OK && dx) {
        mq::Mx4MatmulArgs a = matmul_args(row, view(wg_col), dx);
        a.a[0][1] = row2;
        a.b[0][1] = view(wu_col);
        a.pieces[1] = a.pieces[0];
        st = launched(mq::launch_mx4_matmul(a, stream));
    }
    if (st == MQ_OK && dwg) {
        mq::Mx4MatmulArgs a = matmul_args(col, view(x_col), dwg);
        a.a[1][0] = col2;
        a.b[1][0] = a.b[0][0];
        a.y[1] = view(dwu);
        a.jobs = 2;
        st = launched(mq::launch_mx4_matmul(a, stream));
    }
    return st;
}

} // extern "C"

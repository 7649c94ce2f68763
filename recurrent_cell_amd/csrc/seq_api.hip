// C ABI of the sequence-block operators (declared in include/seq.h): argument
// checks, workspace layout and the launch sequences.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/seq.h"
#include "api_common.h"
#include "seq_kernels.h"

namespace {

using cfc_host::fail;

int64_t elem(int dtype) { return dtype == SEQ_F32 ? 4 : 2; }
int64_t round64(int64_t floats) { return (floats + 63) / 64 * 64; }

// A row-strided operand, in bytes.
struct Mat {
    const void* p;
    int64_t rows, width, ld;
};

Mat mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) { return {p, rows, cols * size, ld * size}; }
Mat flat(const void* p, int64_t n, int64_t size) { return {p, 1, n * size, n * size}; }

// Whether two operands share a byte.  Columns of one buffer (equal strides)
// may interleave without doing so; other strides are taken by their spans.
bool share(const Mat& a, const Mat& b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + (uintptr_t)((a.rows - 1) * a.ld + a.width), b1 = b0 + (uintptr_t)((b.rows - 1) * b.ld + b.width);
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.ld != b.ld || a.ld <= 0) return true;
    const int64_t ld = a.ld;
    const int64_t off = (int64_t)(b0 >= a0 ? (b0 - a0) % (uintptr_t)ld : ((uintptr_t)ld - (a0 - b0) % (uintptr_t)ld) % (uintptr_t)ld);
    return off < a.width || ld - off < b.width;
}

int check_overlap(const char* fn, std::initializer_list<Mat> outs, std::initializer_list<Mat> ins)
{
    for (const Mat* o = outs.begin(); o != outs.end(); ++o) {
        for (const Mat& i : ins)
            if (share(*o, i)) return fail(CFC_EINVAL, "%s: an output overlaps an input", fn);
        for (const Mat* q = o + 1; q != outs.end(); ++q)
            if (share(*o, *q)) return fail(CFC_EINVAL, "%s: two outputs overlap", fn);
    }
    return CFC_OK;
}

int check_type(const char* fn, int dtype)
{
    if (dtype != SEQ_F32 && dtype != SEQ_BF16 && dtype != SEQ_F16) return fail(CFC_EINVAL, "%s: dtype=%d is none of seq_dtype", fn, dtype);
    return CFC_OK;
}

int check_rows(const char* fn, int64_t rows, int64_t cols, int64_t max_cols)
{
    if (rows < 0 || rows > SEQ_MAX_ROWS) return fail(CFC_EINVAL, "%s: rows=%lld out of range [0, %d]", fn, (long long)rows, SEQ_MAX_ROWS);
    if (cols < 1 || cols > max_cols) return fail(CFC_EINVAL, "%s: columns=%lld out of range [1, %lld]", fn, (long long)cols, (long long)max_cols);
    return CFC_OK;
}

// A required operand with rows, its stride and the element's alignment.
int check_mat(const char* fn, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype)
{
    if (rows <= 0) return CFC_OK;
    if (!p) return fail(CFC_EINVAL, "%s: %s is NULL", fn, name);
    if (ld < cols || ld > (int64_t)1 << 31) return fail(CFC_EINVAL, "%s: the row stride of %s, %lld, is out of range [%lld, 2^31]", fn, name, (long long)ld, (long long)cols);
    if ((uintptr_t)p % (uintptr_t)elem(dtype)) return fail(CFC_EINVAL, "%s: %s is not aligned to its elements", fn, name);
    return CFC_OK;
}

int check_f32(const char* fn, const char* name, const void* p, bool needed)
{
    if (!p) return needed ? fail(CFC_EINVAL, "%s: %s is NULL", fn, name) : CFC_OK;
    if ((uintptr_t)p % 4) return fail(CFC_EINVAL, "%s: %s is not aligned to its elements", fn, name);
    return CFC_OK;
}

int check_ws(const char* fn, const void* ws, size_t have, size_t need)
{
    if (need == 0) return CFC_OK;
    if (!ws || have < need) return fail(CFC_EINVAL, "%s: the workspace has %zu bytes, %zu are needed", fn, ws ? have : (size_t)0, need);
    if ((uintptr_t)ws % 4) return fail(CFC_EINVAL, "%s: the workspace is not aligned to 4 bytes", fn);
    return CFC_OK;
}

int check_seqs(const char* fn, const int* cu, int n_seq, int64_t total, int64_t len)
{
    if (n_seq < 0 || n_seq > SEQ_MAX_SEQS) return fail(CFC_EINVAL, "%s: n_seq=%d out of range [0, %d]", fn, n_seq, SEQ_MAX_SEQS);
    if (total < 0 || total > SEQ_MAX_ROWS) return fail(CFC_EINVAL, "%s: total=%lld out of range [0, %d]", fn, (long long)total, SEQ_MAX_ROWS);
    if (n_seq == 0 && total > 0) return fail(CFC_EINVAL, "%s: %lld rows but no sequence", fn, (long long)total);
    if ((uintptr_t)cu % 4) return fail(CFC_EINVAL, "%s: cu_seqlens is not aligned to its elements", fn);
    if (!cu && (len < 0 || len > SEQ_MAX_ROWS || len * n_seq != total))
        return fail(CFC_EINVAL, "%s: total=%lld is not n_seq * len = %d * %lld", fn, (long long)total, n_seq, (long long)len);
    return CFC_OK;
}

#define SEQ_TRY(call)                 \
    do {                              \
        if (int rc_ = (call)) return rc_; \
    } while (0)

// ---------------------------------------------------------------- convolution

int check_conv(const char* fn, const int* cu, int n_seq, int64_t total, int64_t len, int D, int K, int dtype)
{
    SEQ_TRY(check_type(fn, dtype));
    SEQ_TRY(check_rows(fn, total, D, SEQ_MAX_D));
    if (K < 2 || K > 4) return fail(CFC_EINVAL, "%s: K=%d out of range [2, 4]", fn, K);
    return check_seqs(fn, cu, n_seq, total, len);
}

int check_conv_seqs(const char* fn, const int* cu, int n_seq, int64_t total, int64_t len, int D, int K, int dtype)
{
    SEQ_TRY(check_conv(fn, cu, n_seq, total, len, D, K, dtype));
    if (!seq::conv_fits(seq::Rows{cu, total, len, n_seq}, D))
        return fail(CFC_EINVAL, "%s: %d sequences of %lld rows and %d channels need more workgroups than a launch has", fn, n_seq, (long long)total, D);
    return CFC_OK;
}

// ---------------------------------------------------------------- scan

seq::Rows rows_of(const seq_scan& a) { return seq::Rows{a.cu_seqlens, a.total, a.len, a.n_seq}; }

int check_scan_sizes(const char* fn, int64_t total, int D, int N, int G, int dtype)
{
    SEQ_TRY(check_type(fn, dtype));
    SEQ_TRY(check_rows(fn, total, D, SEQ_MAX_D));
    if (N < 1 || N > SEQ_MAX_N) return fail(CFC_EINVAL, "%s: N=%d out of range [1, %d]", fn, N, SEQ_MAX_N);
    if (G < 1 || D % G) return fail(CFC_EINVAL, "%s: G=%d does not divide D=%d", fn, G, D);
    return CFC_OK;
}

int check_scan(const char* fn, const seq_scan* a)
{
    if (!a) return fail(CFC_EINVAL, "%s: the arguments are NULL", fn);
    SEQ_TRY(check_scan_sizes(fn, a->total, a->D, a->N, a->G, a->dtype));
    SEQ_TRY(check_seqs(fn, a->cu_seqlens, a->n_seq, a->total, a->len));
    if (!seq::scan_fits(rows_of(*a), a->D, a->G))
        return fail(CFC_EINVAL, "%s: %d sequences of %lld rows and %d channels need more workgroups than a launch has", fn, a->n_seq, (long long)a->total, a->D);
    return CFC_OK;
}

int check_scan_inputs(const char* fn, const seq_scan& a)
{
    const int64_t R = a.total, GN = (int64_t)a.G * a.N;
    SEQ_TRY(check_mat(fn, "u", a.u, R, a.D, a.ldu, a.dtype));
    SEQ_TRY(check_mat(fn, "dt", a.dt, R, a.D, a.lddt, a.dtype));
    if (a.z) SEQ_TRY(check_mat(fn, "z", a.z, R, a.D, a.ldz, a.dtype));
    SEQ_TRY(check_mat(fn, "B", a.B, R, GN, a.ldb, a.dtype));
    SEQ_TRY(check_mat(fn, "C", a.C, R, GN, a.ldc, a.dtype));
    SEQ_TRY(check_f32(fn, "A", a.A, true));
    SEQ_TRY(check_f32(fn, "skip", a.skip, false));
    SEQ_TRY(check_f32(fn, "dt_bias", a.dt_bias, false));
    return check_f32(fn, "h0", a.h0, false);
}

struct ScanWs {
    int piece = 0, chans = 0;
    int64_t slots = 0, st = -1, sd = -1, bc = -1, pp = -1, total = 0;   // offsets in floats, -1: not used
};

ScanWs scan_fwd_ws(const seq_scan& a)
{
    ScanWs w;
    const seq::Rows r = rows_of(a);
    w.piece = seq::scan_piece(r, a.D, a.G);
    w.slots = seq::scan_slots(r, w.piece);
    if (!seq::scan_one_piece(r, w.piece)) {
        w.st = 0;
        w.sd = round64(w.slots * a.N * a.D);
        w.total = w.sd + round64(w.slots * a.D);
    }
    return w;
}

ScanWs scan_bwd_ws(const seq_scan& a)
{
    ScanWs w;
    const seq::Rows r = rows_of(a);
    w.piece = seq::kScanKeep;
    w.slots = seq::scan_slots(r, w.piece);
    w.chans = seq::scan_bwd_chans(r, a.D, a.G);
    const int64_t blocks = seq::scan_bwd_blocks(a.D, a.G, w.chans);
    // the joined gradients, also where every sequence is one piece: whether
    // dh0 is wanted is not known yet
    w.st = 0;
    w.sd = round64(w.slots * a.N * a.D);
    w.bc = w.sd + round64(w.slots * a.D);
    w.pp = w.bc + round64(blocks * 2 * a.total * a.G * a.N);
    w.total = w.pp + round64(w.slots * (a.N + 2) * a.D);
    return w;
}

// The backward pass's last launch, the sums of the partial gradients, has lanes
// by the values of dB and dC as well.
int check_scan_bwd(const char* fn, const seq_scan* a)
{
    SEQ_TRY(check_scan(fn, a));
    const ScanWs w = scan_bwd_ws(*a);
    const int64_t bc = a->total * a->G * a->N, blocks = seq::scan_bwd_blocks(a->D, a->G, w.chans);
    const int64_t need = 2 * seq::sum_rows_blocks(blocks, bc) + seq::sum_rows_blocks(w.slots, (int64_t)a->N * a->D) +
                         2 * seq::sum_rows_blocks(w.slots, a->D);
    if (need >= (int64_t)1 << 24)
        return fail(CFC_EINVAL, "%s: the gradients of %lld rows, %d groups and %d states need more workgroups than a launch has", fn, (long long)a->total, a->G, a->N);
    return CFC_OK;
}

seq::ScanArgs scan_args(const seq_scan& a)
{
    seq::ScanArgs k{};
    k.u = a.u;
    k.dt = a.dt;
    k.z = a.z;
    k.B = a.B;
    k.C = a.C;
    k.ldu = a.ldu;
    k.lddt = a.lddt;
    k.ldz = a.ldz;
    k.ldb = a.ldb;
    k.ldc = a.ldc;
    k.A = a.A;
    k.skip = a.skip;
    k.dt_bias = a.dt_bias;
    k.h0 = a.h0;
    k.rows = rows_of(a);
    k.D = a.D;
    k.N = a.N;
    k.G = a.G;
    k.type = a.dtype;
    k.softplus = a.softplus ? 1 : 0;
    return k;
}

int dropout(const char* fn, const char* in, const char* out, const void* x, int64_t ldx, const void* r, int64_t ldr, void* y,
            int64_t ldy, int64_t rows, int64_t C, double p, uint64_t seed, uint64_t offset, int dtype, void* stream)
{
    SEQ_TRY(check_type(fn, dtype));
    SEQ_TRY(check_rows(fn, rows, C, (int64_t)1 << 31));
    if (rows > 0 && C > ((int64_t)1 << 33) / rows) return fail(CFC_EINVAL, "%s: more than 2^33 elements", fn);
    if (!(p >= 0.0 && p < 1.0)) return fail(CFC_EINVAL, "%s: p=%g out of range [0, 1)", fn, p);
    SEQ_TRY(check_mat(fn, in, x, rows, C, ldx, dtype));
    if (r) SEQ_TRY(check_mat(fn, "residual", r, rows, C, ldr, dtype));
    SEQ_TRY(check_mat(fn, out, y, rows, C, ldy, dtype));
    const int64_t e = elem(dtype);
    SEQ_TRY(check_overlap(fn, {mat(y, rows, C, ldy, e)}, {mat(x, rows, C, ldx, e), mat(r, rows, C, ldr, e)}));
    if (rows == 0) return CFC_OK;
    const double t = std::nearbyint(p * 4294967296.0);
    seq::DropArgs a{x, r, y, ldx, ldr, ldy, rows, C, seed, offset, (uint32_t)(t < 4294967295.0 ? t : 4294967295.0),
                    (float)(1.0 / (1.0 - p)), dtype};
    CFC_HIP(seq::launch_dropout(a, (hipStream_t)stream), "dropout launch");
    return CFC_OK;
}

}  // namespace

extern "C" {

int seq_layer_norm_fwd(const void* x, int64_t ldx, const float* w, const float* b, void* y, int64_t ldy, float* mean,
                       float* rstd, int64_t rows, int C, float eps, int dtype, void* stream)
{
    const char* fn = "seq_layer_norm_fwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_type(fn, dtype));
    SEQ_TRY(check_rows(fn, rows, C, SEQ_MAX_C));
    if (!(eps >= 0.0f)) return fail(CFC_EINVAL, "%s: eps=%g is negative", fn, (double)eps);
    SEQ_TRY(check_mat(fn, "x", x, rows, C, ldx, dtype));
    SEQ_TRY(check_mat(fn, "y", y, rows, C, ldy, dtype));
    SEQ_TRY(check_f32(fn, "w", w, false));
    SEQ_TRY(check_f32(fn, "b", b, false));
    SEQ_TRY(check_f32(fn, "mean", mean, false));
    SEQ_TRY(check_f32(fn, "rstd", rstd, false));
    const int64_t e = elem(dtype);
    SEQ_TRY(check_overlap(fn, {mat(y, rows, C, ldy, e), flat(mean, rows, 4), flat(rstd, rows, 4)},
                          {mat(x, rows, C, ldx, e), flat(w, C, 4), flat(b, C, 4)}));
    if (rows == 0) return CFC_OK;
    seq::LnArgs a{};
    a.x = x;
    a.out = y;
    a.ldx = ldx;
    a.ldo = ldy;
    a.w = w;
    a.b = b;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.C = C;
    a.type = dtype;
    a.eps = eps;
    CFC_HIP(seq::launch_ln_fwd(a, (hipStream_t)stream), "layer norm launch");
    return CFC_OK;
}

size_t seq_layer_norm_bwd_workspace_bytes(int64_t rows, int C, int dtype)
{
    const char* fn = "seq_layer_norm_bwd_workspace_bytes";
    if (check_type(fn, dtype) || check_rows(fn, rows, C, SEQ_MAX_C)) return 0;
    return sizeof(float) * (size_t)seq::ln_bwd_parts(rows, C, dtype) * 2 * (size_t)C;
}

int seq_layer_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* w, const float* mean,
                       const float* rstd, void* dx, int64_t lddx, float* dw, float* db, int64_t rows, int C, int dtype,
                       void* ws, size_t ws_bytes, void* stream)
{
    const char* fn = "seq_layer_norm_bwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_type(fn, dtype));
    SEQ_TRY(check_rows(fn, rows, C, SEQ_MAX_C));
    SEQ_TRY(check_mat(fn, "dy", dy, rows, C, lddy, dtype));
    SEQ_TRY(check_mat(fn, "x", x, rows, C, ldx, dtype));
    SEQ_TRY(check_mat(fn, "dx", dx, rows, C, lddx, dtype));
    SEQ_TRY(check_f32(fn, "w", w, false));
    SEQ_TRY(check_f32(fn, "mean", mean, rows > 0));
    SEQ_TRY(check_f32(fn, "rstd", rstd, rows > 0));
    SEQ_TRY(check_f32(fn, "dw", dw, false));
    SEQ_TRY(check_f32(fn, "db", db, false));
    const bool params = dw || db;
    const size_t need = params && rows > 0 ? seq_layer_norm_bwd_workspace_bytes(rows, C, dtype) : 0;
    SEQ_TRY(check_ws(fn, ws, ws_bytes, need));
    const int64_t e = elem(dtype);
    SEQ_TRY(check_overlap(fn, {mat(dx, rows, C, lddx, e), flat(dw, C, 4), flat(db, C, 4), flat(need ? ws : nullptr, (int64_t)need, 1)},
                          {mat(dy, rows, C, lddy, e), mat(x, rows, C, ldx, e), flat(w, C, 4), flat(mean, rows, 4), flat(rstd, rows, 4)}));
    hipStream_t s = (hipStream_t)stream;
    const int parts = rows > 0 ? seq::ln_bwd_parts(rows, C, dtype) : 0;
    if (rows > 0) {
        seq::LnArgs a{};
        a.x = x;
        a.dy = dy;
        a.out = dx;
        a.ldx = ldx;
        a.lddy = lddy;
        a.ldo = lddx;
        a.w = w;
        a.mean = const_cast<float*>(mean);
        a.rstd = const_cast<float*>(rstd);
        a.part = params ? (float*)ws : nullptr;
        a.rows = rows;
        a.C = C;
        a.type = dtype;
        a.parts = parts;
        CFC_HIP(seq::launch_ln_bwd(a, s), "layer norm backward launch");
    }
    if (params) {
        const float* p = (const float*)ws;
        seq::SumArgs q{};
        q.nseg = 2;
        q.seg[0] = seq::SumSeg{p, dw, parts, C, 2 * (int64_t)C, SEQ_F32, 0};
        q.seg[1] = seq::SumSeg{p + C, db, parts, C, 2 * (int64_t)C, SEQ_F32, 0};
        CFC_HIP(seq::launch_sum_rows(q, s), "layer norm weight-gradient launch");
    }
    return CFC_OK;
}

int seq_dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t rows,
                    int64_t C, double p, uint64_t seed, uint64_t offset, int dtype, void* stream)
{
    cfc_host::last_error().clear();
    return dropout("seq_dropout_fwd", "x", "y", x, ldx, residual, ldr, y, ldy, rows, C, p, seed, offset, dtype, stream);
}

int seq_dropout_bwd(const void* dy, int64_t lddy, void* dx, int64_t lddx, int64_t rows, int64_t C, double p,
                    uint64_t seed, uint64_t offset, int dtype, void* stream)
{
    cfc_host::last_error().clear();
    return dropout("seq_dropout_bwd", "dy", "dx", dy, lddy, nullptr, 0, dx, lddx, rows, C, p, seed, offset, dtype, stream);
}

int seq_causal_conv_fwd(const void* x, int64_t ldx, const float* w, const float* b, const void* state_in, void* y,
                        int64_t ldy, void* state_out, const int* cu_seqlens, int n_seq, int64_t total, int64_t len,
                        int D, int K, int silu, int dtype, void* stream)
{
    const char* fn = "seq_causal_conv_fwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_conv_seqs(fn, cu_seqlens, n_seq, total, len, D, K, dtype));
    SEQ_TRY(check_mat(fn, "x", x, total, D, ldx, dtype));
    SEQ_TRY(check_mat(fn, "y", y, total, D, ldy, dtype));
    SEQ_TRY(check_f32(fn, "w", w, true));
    SEQ_TRY(check_f32(fn, "b", b, false));
    const int64_t e = elem(dtype), st = (int64_t)n_seq * (K - 1);
    if (state_in) SEQ_TRY(check_mat(fn, "state_in", state_in, st, D, D, dtype));
    if (state_out) SEQ_TRY(check_mat(fn, "state_out", state_out, st, D, D, dtype));
    SEQ_TRY(check_overlap(fn, {mat(y, total, D, ldy, e), flat(state_out, st * D, e)},
                          {mat(x, total, D, ldx, e), flat(w, (int64_t)D * K, 4), flat(b, D, 4), flat(state_in, st * D, e),
                           flat(cu_seqlens, n_seq + 1, 4)}));
    if (n_seq == 0) return CFC_OK;
    seq::ConvArgs a{};
    a.x = x;
    a.out = y;
    a.ldx = ldx;
    a.ldo = ldy;
    a.w = w;
    a.b = b;
    a.state_in = state_in;
    a.state_out = state_out;
    a.rows = seq::Rows{cu_seqlens, total, len, n_seq};
    a.D = D;
    a.K = K;
    a.type = dtype;
    a.silu = silu ? 1 : 0;
    CFC_HIP(seq::launch_conv_fwd(a, (hipStream_t)stream), "convolution launch");
    return CFC_OK;
}

size_t seq_causal_conv_bwd_workspace_bytes(int n_seq, int64_t total, int64_t len, int packed, int D, int K)
{
    const int any = 0;   // stands for a device address: only whether there is one matters here
    const int* cu = packed ? &any : nullptr;
    if (check_conv_seqs("seq_causal_conv_bwd_workspace_bytes", cu, n_seq, total, len, D, K, SEQ_F32)) return 0;
    return sizeof(float) * (size_t)seq::conv_bwd_parts(seq::Rows{cu, total, len, n_seq}, D) * (size_t)D * (size_t)(K + 1);
}

int seq_causal_conv_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* w, const float* b,
                        const void* state_in, void* dx, int64_t lddx, float* dw, float* db, const int* cu_seqlens,
                        int n_seq, int64_t total, int64_t len, int D, int K, int silu, int dtype, void* ws,
                        size_t ws_bytes, void* stream)
{
    const char* fn = "seq_causal_conv_bwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_conv_seqs(fn, cu_seqlens, n_seq, total, len, D, K, dtype));
    SEQ_TRY(check_mat(fn, "dy", dy, total, D, lddy, dtype));
    SEQ_TRY(check_mat(fn, "x", x, total, D, ldx, dtype));
    SEQ_TRY(check_mat(fn, "dx", dx, total, D, lddx, dtype));
    SEQ_TRY(check_f32(fn, "w", w, true));
    SEQ_TRY(check_f32(fn, "b", b, false));
    SEQ_TRY(check_f32(fn, "dw", dw, true));
    SEQ_TRY(check_f32(fn, "db", db, false));
    const int64_t e = elem(dtype), st = (int64_t)n_seq * (K - 1);
    if (state_in) SEQ_TRY(check_mat(fn, "state_in", state_in, st, D, D, dtype));
    const size_t need = seq_causal_conv_bwd_workspace_bytes(n_seq, total, len, cu_seqlens != nullptr, D, K);
    SEQ_TRY(check_ws(fn, ws, ws_bytes, need));
    SEQ_TRY(check_overlap(fn, {mat(dx, total, D, lddx, e), flat(dw, (int64_t)D * K, 4), flat(db, D, 4), flat(need ? ws : nullptr, (int64_t)need, 1)},
                          {mat(dy, total, D, lddy, e), mat(x, total, D, ldx, e), flat(w, (int64_t)D * K, 4), flat(b, D, 4),
                           flat(state_in, st * D, e), flat(cu_seqlens, n_seq + 1, 4)}));
    hipStream_t s = (hipStream_t)stream;
    seq::ConvArgs a{};
    a.x = x;
    a.dy = dy;
    a.out = dx;
    a.ldx = ldx;
    a.lddy = lddy;
    a.ldo = lddx;
    a.w = w;
    a.b = b;
    a.state_in = state_in;
    a.part = (float*)ws;
    a.rows = seq::Rows{cu_seqlens, total, len, n_seq};
    a.D = D;
    a.K = K;
    a.type = dtype;
    a.silu = silu ? 1 : 0;
    if (n_seq > 0) CFC_HIP(seq::launch_conv_bwd(a, s), "convolution backward launch");
    const int64_t parts = seq::conv_bwd_parts(a.rows, D), DK = (int64_t)D * K;
    seq::SumArgs q{};
    q.nseg = 2;
    q.seg[0] = seq::SumSeg{a.part, dw, parts, DK, DK + D, SEQ_F32, 0};
    q.seg[1] = seq::SumSeg{a.part + DK, db, parts, D, DK + D, SEQ_F32, 0};
    CFC_HIP(seq::launch_sum_rows(q, s), "convolution weight-gradient launch");
    return CFC_OK;
}

int seq_causal_conv_step(const void* x, int64_t ldx, void* state, const float* w, const float* b, void* y, int64_t ldy,
                         int64_t S, int D, int K, int silu, int dtype, void* stream)
{
    const char* fn = "seq_causal_conv_step";
    cfc_host::last_error().clear();
    SEQ_TRY(check_conv(fn, nullptr, S >= 0 && S <= SEQ_MAX_SEQS ? (int)S : -1, S, 1, D, K, dtype));
    SEQ_TRY(check_mat(fn, "x", x, S, D, ldx, dtype));
    SEQ_TRY(check_mat(fn, "y", y, S, D, ldy, dtype));
    SEQ_TRY(check_mat(fn, "state", state, S * (K - 1), D, D, dtype));
    SEQ_TRY(check_f32(fn, "w", w, true));
    SEQ_TRY(check_f32(fn, "b", b, false));
    const int64_t e = elem(dtype);
    SEQ_TRY(check_overlap(fn, {mat(y, S, D, ldy, e), flat(state, S * (K - 1) * D, e)},
                          {mat(x, S, D, ldx, e), flat(w, (int64_t)D * K, 4), flat(b, D, 4)}));
    if (S == 0) return CFC_OK;
    seq::ConvStepArgs a{x, state, y, ldx, ldy, w, b, S, D, K, dtype, silu ? 1 : 0};
    CFC_HIP(seq::launch_conv_step(a, (hipStream_t)stream), "convolution step launch");
    return CFC_OK;
}

size_t seq_selective_scan_hist_floats(const seq_scan* a)
{
    if (check_scan("seq_selective_scan_hist_floats", a)) return 0;
    return (size_t)seq::scan_slots(rows_of(*a), seq::kScanKeep) * (size_t)a->N * (size_t)a->D;
}

size_t seq_selective_scan_fwd_workspace_bytes(const seq_scan* a)
{
    if (check_scan("seq_selective_scan_fwd_workspace_bytes", a)) return 0;
    return sizeof(float) * (size_t)scan_fwd_ws(*a).total;
}

size_t seq_selective_scan_bwd_workspace_bytes(const seq_scan* a)
{
    if (check_scan_bwd("seq_selective_scan_bwd_workspace_bytes", a)) return 0;
    return sizeof(float) * (size_t)scan_bwd_ws(*a).total;
}

int seq_selective_scan_fwd(const seq_scan* a, void* y, int64_t ldy, float* h_last, float* hist, void* ws,
                           size_t ws_bytes, void* stream)
{
    const char* fn = "seq_selective_scan_fwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_scan(fn, a));
    SEQ_TRY(check_scan_inputs(fn, *a));
    SEQ_TRY(check_mat(fn, "y", y, a->total, a->D, ldy, a->dtype));
    SEQ_TRY(check_f32(fn, "h_last", h_last, false));
    SEQ_TRY(check_f32(fn, "hist", hist, false));
    const ScanWs w = scan_fwd_ws(*a);
    SEQ_TRY(check_ws(fn, ws, ws_bytes, sizeof(float) * (size_t)w.total));
    const int64_t e = elem(a->dtype), R = a->total, D = a->D, ND = (int64_t)a->N * D, GN = (int64_t)a->G * a->N;
    SEQ_TRY(check_overlap(fn, {mat(y, R, D, ldy, e), flat(h_last, a->n_seq * ND, 4), flat(hist, (int64_t)(hist ? seq_selective_scan_hist_floats(a) : 0), 4),
                               flat(w.total ? ws : nullptr, w.total, 4)},
                          {mat(a->u, R, D, a->ldu, e), mat(a->dt, R, D, a->lddt, e), mat(a->z, R, D, a->ldz, e),
                           mat(a->B, R, GN, a->ldb, e), mat(a->C, R, GN, a->ldc, e), flat(a->A, ND, 4), flat(a->skip, D, 4),
                           flat(a->dt_bias, D, 4), flat(a->h0, a->n_seq * ND, 4), flat(a->cu_seqlens, a->n_seq + 1, 4)}));
    if (a->n_seq == 0) return CFC_OK;
    hipStream_t s = (hipStream_t)stream;
    seq::ScanArgs k = scan_args(*a);
    k.y = y;
    k.ldy = ldy;
    k.h_last = h_last;
    k.hist = hist;
    k.piece = w.piece;
    if (w.total) {
        k.st = (float*)ws + w.st;
        k.sd = (float*)ws + w.sd;
        CFC_HIP(seq::launch_scan_state(k, false, s), "scan piece-state launch");
        k.join = seq::scan_joins(k.rows, a->D, a->G);
        if (!k.join) CFC_HIP(seq::launch_scan_join(k, false, s), "scan join launch");
    }
    CFC_HIP(seq::launch_scan_fwd(k, s), "scan launch");
    return CFC_OK;
}

int seq_selective_scan_bwd(const seq_scan* a, const void* dy, int64_t lddy, const float* hist, const float* dh_last,
                           const seq_scan_grads* g, void* ws, size_t ws_bytes, void* stream)
{
    const char* fn = "seq_selective_scan_bwd";
    cfc_host::last_error().clear();
    SEQ_TRY(check_scan_bwd(fn, a));
    SEQ_TRY(check_scan_inputs(fn, *a));
    if (!g) return fail(CFC_EINVAL, "%s: the gradients are NULL", fn);
    const int dtype = a->dtype;
    const int64_t e = elem(dtype), R = a->total, D = a->D, ND = (int64_t)a->N * D, GN = (int64_t)a->G * a->N;
    SEQ_TRY(check_mat(fn, "dy", dy, R, D, lddy, dtype));
    SEQ_TRY(check_mat(fn, "du", g->du, R, D, g->lddu, dtype));
    SEQ_TRY(check_mat(fn, "ddt", g->ddt, R, D, g->ldddt, dtype));
    if (a->z) SEQ_TRY(check_mat(fn, "dz", g->dz, R, D, g->lddz, dtype));
    else if (g->dz) return fail(CFC_EINVAL, "%s: dz without z", fn);
    SEQ_TRY(check_mat(fn, "dB", g->dB, R, GN, GN, dtype));
    SEQ_TRY(check_mat(fn, "dC", g->dC, R, GN, GN, dtype));
    SEQ_TRY(check_f32(fn, "dA", g->dA, true));
    SEQ_TRY(check_f32(fn, "dskip", g->dskip, false));
    SEQ_TRY(check_f32(fn, "ddt_bias", g->ddt_bias, false));
    SEQ_TRY(check_f32(fn, "dh0", g->dh0, false));
    SEQ_TRY(check_f32(fn, "hist", hist, R > 0));
    SEQ_TRY(check_f32(fn, "dh_last", dh_last, false));
    const ScanWs w = scan_bwd_ws(*a);
    SEQ_TRY(check_ws(fn, ws, ws_bytes, sizeof(float) * (size_t)w.total));
    const Mat outs_w = flat(w.total ? ws : nullptr, w.total, 4);
    SEQ_TRY(check_overlap(fn,
                          {mat(g->du, R, D, g->lddu, e), mat(g->ddt, R, D, g->ldddt, e), mat(g->dz, R, D, g->lddz, e), flat(g->dB, R * GN, e),
                           flat(g->dC, R * GN, e), flat(g->dA, ND, 4), flat(g->dskip, D, 4), flat(g->ddt_bias, D, 4),
                           flat(g->dh0, a->n_seq * ND, 4), outs_w},
                          {mat(a->u, R, D, a->ldu, e), mat(a->dt, R, D, a->lddt, e), mat(a->z, R, D, a->ldz, e),
                           mat(a->B, R, GN, a->ldb, e), mat(a->C, R, GN, a->ldc, e), flat(a->A, ND, 4), flat(a->skip, D, 4),
                           flat(a->dt_bias, D, 4), flat(a->cu_seqlens, a->n_seq + 1, 4), mat(dy, R, D, lddy, e),
                           flat(hist, (int64_t)seq_selective_scan_hist_floats(a), 4), flat(dh_last, a->n_seq * ND, 4)}));
    hipStream_t s = (hipStream_t)stream;
    seq::ScanArgs k = scan_args(*a);
    float* f = (float*)ws;
    if (a->n_seq > 0) {
        k.dy = dy;
        k.lddy = lddy;
        k.du = g->du;
        k.ddt = g->ddt;
        k.dz = g->dz;
        k.lddu = g->lddu;
        k.ldddt = g->ldddt;
        k.lddz = g->lddz;
        k.dh_last = dh_last;
        k.dh0 = g->dh0;
        k.hist = const_cast<float*>(hist);
        k.piece = w.piece;
        k.chans = w.chans;
        k.part_bc = f + w.bc;
        k.part_p = f + w.pp;
        // one piece per sequence and no dh0: what enters from the right is dh_last itself
        if (g->dh0 || !seq::scan_one_piece(k.rows, w.piece)) {
            k.st = f + w.st;
            k.sd = f + w.sd;
            CFC_HIP(seq::launch_scan_state(k, true, s), "scan backward piece-state launch");
            k.join = seq::scan_joins(k.rows, a->D, a->G);
            if (!k.join) CFC_HIP(seq::launch_scan_join(k, true, s), "scan backward join launch");
        }
        CFC_HIP(seq::launch_scan_bwd(k, s), "scan backward launch");
    }
    const int64_t blocks = seq::scan_bwd_blocks(a->D, a->G, w.chans), stride = ND + 2 * D;
    seq::SumArgs q{};
    q.nseg = 5;
    q.seg[0] = seq::SumSeg{f + w.bc, g->dB, blocks, R * GN, 2 * R * GN, dtype, 0};
    q.seg[1] = seq::SumSeg{f + w.bc + R * GN, g->dC, blocks, R * GN, 2 * R * GN, dtype, 0};
    q.seg[2] = seq::SumSeg{f + w.pp, g->dA, w.slots, ND, stride, SEQ_F32, 0};
    q.seg[3] = seq::SumSeg{f + w.pp + ND, g->dskip, w.slots, D, stride, SEQ_F32, 0};
    q.seg[4] = seq::SumSeg{f + w.pp + ND + D, g->ddt_bias, w.slots, D, stride, SEQ_F32, 0};
    CFC_HIP(seq::launch_sum_rows(q, s), "scan gradient-sum launch");
    return CFC_OK;
}

int seq_selective_scan_step(float* h, const void* u, int64_t ldu, const void* dt, int64_t lddt, const float* A,
                            const void* B, int64_t ldb, const void* C, int64_t ldc, const float* skip, const void* z,
                            int64_t ldz, const float* dt_bias, void* y, int64_t ldy, int64_t S, int D, int N, int G,
                            int softplus, int dtype, void* stream)
{
    const char* fn = "seq_selective_scan_step";
    cfc_host::last_error().clear();
    SEQ_TRY(check_scan_sizes(fn, S, D, N, G, dtype));
    if (S > SEQ_MAX_SEQS) return fail(CFC_EINVAL, "%s: S=%lld out of range [0, %d]", fn, (long long)S, SEQ_MAX_SEQS);
    const int64_t e = elem(dtype), ND = (int64_t)N * D, GN = (int64_t)G * N;
    SEQ_TRY(check_mat(fn, "u", u, S, D, ldu, dtype));
    SEQ_TRY(check_mat(fn, "dt", dt, S, D, lddt, dtype));
    if (z) SEQ_TRY(check_mat(fn, "z", z, S, D, ldz, dtype));
    SEQ_TRY(check_mat(fn, "B", B, S, GN, ldb, dtype));
    SEQ_TRY(check_mat(fn, "C", C, S, GN, ldc, dtype));
    SEQ_TRY(check_mat(fn, "y", y, S, D, ldy, dtype));
    SEQ_TRY(check_f32(fn, "h", h, S > 0));
    SEQ_TRY(check_f32(fn, "A", A, true));
    SEQ_TRY(check_f32(fn, "skip", skip, false));
    SEQ_TRY(check_f32(fn, "dt_bias", dt_bias, false));
    SEQ_TRY(check_overlap(fn, {mat(y, S, D, ldy, e), flat(h, S * ND, 4)},
                          {mat(u, S, D, ldu, e), mat(dt, S, D, lddt, e), mat(z, S, D, ldz, e), mat(B, S, GN, ldb, e),
                           mat(C, S, GN, ldc, e), flat(A, ND, 4), flat(skip, D, 4), flat(dt_bias, D, 4)}));
    if (S == 0) return CFC_OK;
    seq::ScanStepArgs a{u, dt, z, B, C, ldu, lddt, ldz, ldb, ldc, ldy, y, A, skip, dt_bias, h, S, D, N, G, dtype, softplus ? 1 : 0};
    CFC_HIP(seq::launch_scan_step(a, (hipStream_t)stream), "scan step launch");
    return CFC_OK;
}

}  // extern "C"

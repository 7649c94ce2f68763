"""Sequence-block operators on the GPU at the sizes where a launch takes another
shape: more rows than workers, longer pieces.  Against the fp64 oracle; tolerances:
tests/tolerances.py."""
import numpy as np
import pytest
import torch

from oracle import seq_oracle as so
from tests.test_gpu_seq import S, dev, f64, ok, rng, say, scan_inputs, split, strided  # noqa: F401
from tests.tolerances import check_seq, scan_k, seq_ln_bounds

pytestmark = pytest.mark.gpu

# Backward passes whose workers (16, 32 or 64 lanes, 4 or 8 wavefronts, by C and
# type) take two rows or more each: more than 8,192, 4,096, 2,048, 512 and 256 rows.
LN_ROWS = [(9000, 3, "f32", 0), (9000, 33, "f32", 2), (8300, 100, "bf16", 0), (5000, 100, "f32", 0), (4500, 200, "bf16", 3),
           (2200, 300, "f32", 0), (2200, 1000, "f16", 0), (4200, 1025, "bf16", 0), (600, 1025, "f32", 1), (600, 3001, "f32", 0),
           (600, 3000, "bf16", 0), (300, 5000, "f32", 0), (300, 8193, "f32", 0), (300, 9001, "f16", 0)]


@pytest.mark.parametrize("M,C,dtype,pad", LN_ROWS)
def test_layer_norm_many_rows(S, M, C, dtype, pad):  # noqa: F811
    say("layer_norm", M, C, dtype, pad)
    r = rng(30, M, C)
    x, dy = dev(r.normal(size=(M, C)) + 0.7, dtype), dev(r.normal(size=(M, C)), dtype)
    w, b = dev(1 + 0.3 * r.normal(size=C)), dev(r.normal(size=C))
    X, DY, W, Bv = f64(x), f64(dy), f64(w), f64(b)
    x, dy = strided(x, pad), strided(dy, pad)
    y, mean, rstd = S.layer_norm_fwd(x, w, b)
    my, mdx, mdw, mdb = seq_ln_bounds(X, W, Bv, 1e-5, DY)
    ok(check_seq("y", f64(y), so.layer_norm(X, W, Bv, 1e-5)[0], my, dtype, 1))
    dx, dw, db = S.layer_norm_bwd(dy, x, w, mean, rstd)
    rdx, rdw, rdb = so.layer_norm_bwd(DY, X, W, 1e-5)
    ok(check_seq("dx", f64(dx), rdx, mdx, dtype, 1))
    # dw and db are fp32 sums over a worker's rows (at most 3 here) and over 32
    # workers, then fp64: 44 roundings instead of the bounds' M + 8, so that a row
    # left out or counted twice fails
    xh = (X - X.mean(1, keepdims=True)) / np.sqrt(X.var(1, keepdims=True) + 1e-5)
    fewer = M + 8 - 44
    ok(check_seq("dw", f64(dw), rdw, mdw - fewer * np.abs(DY * xh).sum(0), "f32", 1))
    ok(check_seq("db", f64(db), rdb, mdb - fewer * np.abs(DY).sum(0), "f32", 1))


# Forward passes whose workgroups (4,096 at most, of 16, 8, 4 or one row) go round again.
LN_ROUNDS = [(66000, 5, "f16", 0), (66000, 40, "f32", 0), (33000, 130, "bf16", 1), (17000, 260, "f32", 0), (4200, 1025, "f32", 0),
             (4200, 2050, "f16", 0), (4200, 4200, "f32", 0), (4200, 8200, "bf16", 0)]


@pytest.mark.parametrize("M,C,dtype,pad", LN_ROUNDS)
def test_layer_norm_more_rows_than_workers(S, M, C, dtype, pad):  # noqa: F811
    say("layer_norm", M, C, dtype, pad)
    r = rng(31, M, C)
    x = dev(r.standard_normal((M, C), np.float32) + np.float32(0.7), dtype)
    w, b = dev(1 + 0.3 * r.normal(size=C)), dev(r.normal(size=C))
    X, W, Bv = f64(x), f64(w), f64(b)
    y, mean, rstd = S.layer_norm_fwd(strided(x, pad), w, b)
    ref, rm, rr = so.layer_norm(X, W, Bv, 1e-5)
    ok(check_seq("y", f64(y), ref, seq_ln_bounds(X, W, Bv, 1e-5), dtype, 1))
    ok(check_seq("mean", f64(mean), rm, np.abs(X).mean(1), "f32", 56))
    ok(check_seq("rstd", f64(rstd), rr, rr * (1 + np.abs(X).mean(1) * rr), "f32", 100))


# The backward pass takes pieces of 32 rows from 384 units of 64 rows x 128
# channels on and of 64 rows from 2,048 on (units: 8 x 50 and 8 x 257 here).
@pytest.mark.parametrize("n,dtype,K,silu", [([1700, 0, 1, 31, 33, 65, 1400], "f32", 4, True), ([3231], "bf16", 3, True),
                                            ([9001, 0, 63, 64, 1, 65, 7300], "bf16", 4, True), ([16500], "f16", 2, False)])
def test_conv_long_pieces(S, n, dtype, K, silu):  # noqa: F811
    say("conv", n, dtype, K, silu)
    rows, D, cu = sum(n), 999, np.concatenate([[0], np.cumsum(n)])
    r = rng(32, rows, K)
    x, dy = dev(r.standard_normal((rows, D), np.float32), dtype), dev(r.standard_normal((rows, D), np.float32), dtype)
    w, b, st = dev(r.normal(size=(D, K))), dev(r.normal(size=D)), dev(r.normal(size=(len(n), K - 1, D)), dtype)
    cud = torch.from_numpy(cu.astype(np.int32)).cuda() if len(n) > 1 else None
    d = S.causal_conv_bwd(dy, x, w, b, silu=silu, state=st, cu_seqlens=cud)
    refs, masses = so.causal_conv_bwd(f64(dy), f64(x), f64(w), f64(b), silu, f64(st), so.spans(rows, cu))
    for name, t, ref, m, k in zip(("dx", "dw", "db"), d, refs, masses, (24 + K, 24 + 64, 24 + 64)):
        ok(check_seq(name, f64(t), ref, m, dtype if name == "dx" else "f32", k))


# With a channel per lane the forward pieces grow with the rows (to 128 and 192
# here), while the states kept and the backward pieces stay 64 rows apart.
@pytest.mark.parametrize("n,N,dtype", [([700, 0, 130, 270], 4, "f32"), ([700, 0, 130, 270], 3, "bf16"), ([1500, 3, 600], 4, "f32"), ([1100], 2, "f16")])
def test_scan_long_pieces(S, n, N, dtype):  # noqa: F811
    say("scan", n, N, dtype)
    D = G = 256
    a, ref, where = scan_inputs(n, D, N, G, dtype)
    args, kw = split(a)
    r = rng(33, N, sum(n))
    f = S.selective_scan_fwd(*args, save=True, **kw)
    (y, h), (my, mh) = so.selective_scan(*ref, where)
    k = scan_k(ref[1], ref[7], ref[2], ref[8], N)
    ok(check_seq("y", f64(f.y), y, my, dtype, k))
    ok(check_seq("h_last", f64(f.h_last), h, mh, "f32", k))
    dy, dh = dev(r.normal(size=y.shape), dtype), dev(r.normal(size=h.shape))
    d = S.selective_scan_bwd(dy, *args, f.hist, dh_last=dh, **kw)
    g, m = so.selective_scan_bwd(f64(dy), *ref, f64(dh), where)
    chain = {"dB": 1, "dC": 1, "du": N, "ddt": N, "dz": N}   # a group is one channel
    for key in g:
        ok(check_seq(key, f64(getattr(d, key)), g[key], m[key], dtype if key in ("du", "ddt", "dz", "dB", "dC") else "f32",
                     scan_k(ref[1], ref[7], ref[2], ref[8], chain.get(key, 16))))

"""Sequence-block operators on the GPU where single values are not finite,
against the fp64 oracle.  Tolerances: tests/tolerances.py."""
import numpy as np
import pytest
import torch

from oracle import seq_oracle as so
from tests.test_gpu_seq import MANY, S, dev, f64, ok, rng, say, scan_inputs, split  # noqa: F401
from tests.tolerances import check_seq, scan_k

pytestmark = pytest.mark.gpu

# in rows and, with many sequences, with a channel per lane
LAYOUTS = [([1], 1, "f32"), ([40], 1, "f16"), ([70, 9, 0, 130], 2, "bf16"), ([300], 1, "f32"), (MANY, 1, "f32"), (MANY, 2, "bf16")]


@pytest.mark.parametrize("n,G,dtype", LAYOUTS)
def test_scan_steps_of_minus_infinity(S, n, G, dtype):  # noqa: F811
    """dt = -inf (a masked row) and dt_bias = -inf (a channel switched off):
    delta = softplus(-inf) = 0, so the state is kept, and no gradient reaches
    dt.  The oracle's values are those of -1e4, where softplus and its slope are
    0 in fp64 too but the masses stay finite."""
    say("scan -inf", len(n), G, dtype)
    D, N = 6, 5
    a, ref, where = scan_inputs(n, D, N, G, dtype)
    r = rng(20, len(n), G)
    rows = r.random(sum(n)) < 0.3
    rows[-1] = True
    off = np.arange(D) == 2
    low, high = a["dt"].clone(), a["dt_bias"].clone()
    a["dt"][torch.from_numpy(rows).cuda()] = -float("inf")
    a["dt_bias"][2] = -float("inf")
    low[torch.from_numpy(rows).cuda()] = -1e4
    high[2] = -1e4
    ref = ref[:1] + (f64(low),) + ref[2:7] + (f64(high),) + ref[8:]
    with np.errstate(invalid="ignore"):
        inf = so.selective_scan(*(ref[:1] + (f64(a["dt"]),) + ref[2:7] + (f64(a["dt_bias"]),) + ref[8:]), where)[0]
    (y, h), (my, mh) = so.selective_scan(*ref, where)
    assert np.array_equal(inf[0], y) and np.array_equal(inf[1], h)

    args, kw = split(a)
    x = np.where(rows[:, None] | off[None], -1e4, ref[1] + ref[7])
    k = scan_k(x, 0.0, ref[2], True, N)
    f = S.selective_scan_fwd(*args, save=True, **kw)
    ok(check_seq("y", f64(f.y), y, my, dtype, k))
    ok(check_seq("h_last", f64(f.h_last), h, mh, "f32", k))
    dy, dh = dev(r.normal(size=y.shape), dtype), dev(r.normal(size=h.shape))
    d = S.selective_scan_bwd(dy, *args, f.hist, dh_last=dh, **kw)
    g, m = so.selective_scan_bwd(f64(dy), *ref, f64(dh), where)
    for key in g:
        ok(check_seq(key, f64(getattr(d, key)), g[key], m[key], dtype if key in ("du", "ddt", "dz", "dB", "dC") else "f32",
                     scan_k(x, 0.0, ref[2], True, {"dB": D, "dC": D}.get(key, 16))))
    assert not f64(d.ddt)[rows].any() and not f64(d.ddt)[:, off].any() and f64(d.ddt_bias)[2] == 0

    # the same rows as single tokens: a sequence each
    T = min(sum(n), 200)
    one = [v if i == 2 else v[:T].contiguous() for i, v in enumerate(args)]
    h0 = dev(r.normal(size=(T, N, D)))
    state = h0.clone()
    ys = S.selective_scan_step(state, *one, skip=kw["skip"], z=kw["z"][:T].contiguous(), dt_bias=kw["dt_bias"])
    cut = [ref[0][:T], ref[1][:T], ref[2], ref[3][:T], ref[4][:T], ref[5], ref[6][:T], ref[7], ref[8], f64(h0)]
    (y, h), (my, mh) = so.selective_scan(*cut, so.spans(T, np.arange(T + 1)))
    ok(check_seq("y", f64(ys), y, my, dtype, k))
    ok(check_seq("h", f64(state), h, mh, "f32", k))
    kept = np.zeros((T, 1, D), bool) | rows[:T, None, None] | off
    assert np.array_equal(f64(state)[np.broadcast_to(kept, state.shape)], f64(h0)[np.broadcast_to(kept, state.shape)])


def finite_or_equal(name, x, ref, mass, dtype, k):
    """Where the definition is finite, its bound; where it is infinite, the same
    infinity; where it is NaN (infinities of both signs), anything."""
    fin, inf = np.isfinite(ref), np.isinf(ref)
    assert np.array_equal(x[inf], ref[inf]), (name, int((x[inf] != ref[inf]).sum()), "of", int(inf.sum()))
    ok(check_seq(name, x[fin], ref[fin], mass[fin], dtype, k))


@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("N", [1, 3, 5, 6, 11, 12, 16, 17, 20, 33, 48])
def test_scan_infinite_inputs(S, N, layout):  # noqa: F811
    """An infinite u leaves what the definition makes of it: infinities, not NaN,
    in its channel from its row on, also where N states do not fill their tile;
    and nothing in the gradients that do not meet it."""
    say("scan inf", N, layout)
    n, dtype = [([40], "f32"), ([130, 7, 70], "bf16"), (MANY, "f32")][layout]
    D, rows = 3, sum(n)
    a, ref, where = scan_inputs(n, D, N, 1, dtype)
    r = rng(21, N, layout)
    # all positive, decays that stay above 0: every infinity has one sign
    for key in ("B", "C", "z", "u"):
        a[key] = a[key].abs() + 0.125
    a["dt_bias"] = dev(r.uniform(-6, -5, size=D))
    a["h0"], a["skip"] = a["h0"].abs(), a["skip"].abs()
    dy, dh = dev(r.uniform(0.1, 1, size=(rows, D)), dtype), dev(r.uniform(0.1, 1, size=(len(n), N, D)))
    a["u"][n[0] // 2, 0] = float("inf")
    ref = (f64(a["u"]), ref[1], ref[2], f64(a["B"]), f64(a["C"]), f64(a["skip"]), f64(a["z"]), f64(a["dt_bias"]), True, f64(a["h0"]))
    args, kw = split(a)
    with np.errstate(invalid="ignore"):
        (y, h), (my, mh) = so.selective_scan(*ref, where)
        g, m = so.selective_scan_bwd(f64(dy), *ref, f64(dh), where)
    assert np.isinf(y[n[0] // 2:n[0], 0]).all() and np.isfinite(y[:, 1:]).all() and np.isinf(g["dA"][:, 0]).all()
    k = scan_k(ref[1], ref[7], ref[2], True, N)
    f = S.selective_scan_fwd(*args, save=True, **kw)
    finite_or_equal("y", f64(f.y), y, my, dtype, k)
    finite_or_equal("h_last", f64(f.h_last), h, mh, "f32", k)
    d = S.selective_scan_bwd(dy, *args, f.hist, dh_last=dh, **kw)
    for key in g:
        finite_or_equal(key, f64(getattr(d, key)), g[key], m[key], dtype if key in ("du", "ddt", "dz", "dB", "dC") else "f32",
                        scan_k(ref[1], ref[7], ref[2], True, {"dB": D, "dC": D}.get(key, N)))


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("n", [[3], [40], [16, 5, 33]])
def test_conv_infinite_inputs(S, K, n):  # noqa: F811
    """An infinite x without an activation: infinities in the dw of the taps that
    meet it and in y, nothing elsewhere.  In one channel it is a sequence's last
    row, in one the first after 16 rows (a piece), in one the first of all."""
    say("conv inf", K, n)
    rows, D, cu = sum(n), 5, np.concatenate([[0], np.cumsum(n)])
    r = rng(22, K, rows)
    x, dy, w, b = r.normal(size=(rows, D)), r.normal(size=(rows, D)), r.normal(size=(D, K)), r.normal(size=D)
    x, dy, w, b = dev(x), dev(dy), dev(w), dev(b)
    x[n[0] - 1, 0] = x[min(16, rows - 1), 1] = float("inf")
    x[0, 3] = -float("inf")
    where, st = so.spans(rows, cu), np.zeros((len(n), K - 1, D))
    cud = torch.from_numpy(cu.astype(np.int32)).cuda()
    with np.errstate(invalid="ignore"):
        y, _ = so.causal_conv(f64(x), f64(w), f64(b), False, st, where)
        mass, _ = so.causal_conv(np.abs(f64(x)), np.abs(f64(w)), np.abs(f64(b)), False, st, where)
        g, m = so.causal_conv_bwd(f64(dy), f64(x), f64(w), f64(b), False, st, where)
    assert np.isinf(g[1]).any() and not np.isnan(g[1]).any() and np.isfinite(g[1][[2, 4]]).all()
    finite_or_equal("y", f64(S.causal_conv_fwd(x, w, b, silu=False, cu_seqlens=cud)), y, mass, "f32", 12)
    d = S.causal_conv_bwd(dy, x, w, b, silu=False, cu_seqlens=cud)
    for name, t, ref, ma, k in zip(("dx", "dw", "db"), d, g, m, (24 + K, 24 + 64, 24 + 64)):
        finite_or_equal(name, f64(t), ref, ma, "f32", k)

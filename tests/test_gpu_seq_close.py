"""The selective scan on the GPU held to what fp32 can do: its outputs and
gradients against the definition differentiated in fp64, off by at most four
times what the same definition loses in fp32 (or 16 half steps of the output's
own size), in norm and, with twice that, in the worst element.  First-order bounds grow with
the steps a term goes through; these do not, so a row left out of a sum fails."""
import numpy as np
import pytest
import torch

from tests.test_gpu_seq import MANY, S, dev, rng, say, scan_inputs, split  # noqa: F401
from tests.tolerances import U32

pytestmark = pytest.mark.gpu


def plain_scan(v, ends, G):
    """(y, h_last) in the type of v's values, one row at a time."""
    D = v["u"].shape[1]
    per = lambda m: m.repeat_interleave(D // G, 0).t()  # noqa: E731  [G, N] -> [N, D]
    delta = torch.nn.functional.softplus(v["dt"] + v["dt_bias"])
    ys, hs = [], []
    for s, (p, e) in enumerate(zip(ends, ends[1:])):
        h = v["h0"][s]
        for t in range(p, e):
            h = torch.exp(delta[t] * v["A"]) * h + (delta[t] * v["u"][t]) * per(v["B"][t])
            ys.append((per(v["C"][t]) * h).sum(0) + v["skip"] * v["u"][t])
        hs.append(h)
    return torch.stack(ys) * (v["z"] * torch.sigmoid(v["z"])), torch.stack(hs)


def plain_all(v, dy, dh, dtype, ends, G):
    v = {k: t.detach().cpu().to(dtype).requires_grad_() for k, t in v.items()}
    y, h = plain_scan(v, ends, G)
    g = torch.autograd.grad((y * dy.cpu().to(dtype)).sum() + (h * dh.cpu().to(dtype)).sum(), list(v.values()))
    return {k: t.detach().double() for k, t in zip(["y", "h_last"] + ["d" + k for k in v], (y, h) + g)}


@pytest.mark.parametrize("n,D,N,G", [([300], 40, 16, 2), ([5, 0, 1, 130, 64, 0, 257], 36, 11, 1), ([100], 130, 64, 1), ([70, 200], 48, 32, 3),
                                     ([250], 20, 6, 1), (MANY, 6, 16, 1), (MANY, 5, 11, 1), ([700, 0, 130, 270], 256, 4, 256)])
def test_scan_close(S, n, D, N, G):  # noqa: F811
    say("scan close", len(n), D, N, G)
    a, _, _ = scan_inputs(n, D, N, G, "f32", seed=40)
    r = rng(41, D, N, sum(n))
    a["dt_bias"] = dev(r.uniform(-3, -1, size=D))
    ends = [0] + np.cumsum(n).tolist()
    dy, dh = dev(r.normal(size=(sum(n), D))), dev(r.normal(size=(len(n), N, D)))
    v = {k: a[k] for k in ("u", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")}
    ref, low = (plain_all(v, dy, dh, t, ends, G) for t in (torch.float64, torch.float32))
    args, kw = split(a)
    f = S.selective_scan_fwd(*args, save=True, **kw)
    d = S.selective_scan_bwd(dy, *args, f.hist, dh_last=dh, **kw)
    got = dict({"d" + k: getattr(d, "d" + k) for k in v}, y=f.y, h_last=f.h_last)
    assert set(got) == set(ref)
    for name, want in ref.items():
        e, e32 = got[name].double().cpu() - want, low[name] - want
        norm = 4 * max(float(e32.norm()), 16 * U32 * float(want.norm()))
        worst = 8 * max(float(e32.abs().max()), 16 * U32 * float(want.abs().max()))
        say("   ", name, "norm %.3f worst %.3f of the allowed" % (float(e.norm()) / norm, float(e.abs().max()) / worst))
        assert float(e.norm()) <= norm and float(e.abs().max()) <= worst, name

"""Host-side checks of the sequence operators' C ABI and binding (CPU only:
no call here reaches a kernel; every refused call is refused by the checks that
run before anything is enqueued, so fake addresses are safe)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from recurrent_cell_amd import build as hbuild
    hbuild.build(force=False)
    from recurrent_cell_amd import seq
    return seq.lib()


def at(i):
    return FAKE + i * (1 << 34)


def err(L):
    return L.cfc_last_error().decode()


def test_header_matches_the_library_and_the_binding(L):
    from recurrent_cell_amd import seq
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "seq.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|size_t)\s+(seq_\w+)\s*\(([^)]*)\)", text, flags=re.M)
    assert len(names) == 15
    for name, args in names:
        f = getattr(L, name)
        assert len(f.argtypes) == len(args.split(",")), name
    for struct, cls in (("seq_scan", seq._Scan), ("seq_scan_grads", seq._ScanGrads)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, flags=re.S).group(1)
        fields = re.findall(r"\*?(\w+)\s*[;,]", body)
        assert fields == [n for n, _ in cls._fields_]


def test_kernel_sources_have_no_atomics():
    csrc = os.path.join(ROOT, "recurrent_cell_amd", "csrc")
    for fn in ("seq_norm.hip", "seq_conv.hip", "seq_scan.hip", "seq_device.h", "seq_kernels.h"):
        assert not re.search(r"\batomic\w*\s*\(|_atomic_|std::atomic", open(os.path.join(csrc, fn)).read()), fn


def test_layer_norm_refusals(L):
    def fwd(x=at(0), ldx=64, w=at(1), b=at(2), y=at(3), ldy=64, mean=at(4), rstd=at(5), rows=8, C=64, eps=1e-5, dtype=F32):
        return L.seq_layer_norm_fwd(x, ldx, w, b, y, ldy, mean, rstd, rows, C, eps, dtype, None)

    for bad in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(C=0), dict(C=16385, ldx=20000, ldy=20000),
                dict(x=None), dict(y=None), dict(ldx=63), dict(ldy=63), dict(ldx=(1 << 31) + 1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=at(0) + 2), dict(w=at(1) + 2), dict(mean=at(4) + 1),
                dict(y=at(0) + 64), dict(mean=at(0) + 16), dict(w=at(3)), dict(mean=at(5))):
        assert fwd(**bad) == -1, bad
        assert err(L).startswith("seq_layer_norm_fwd"), bad
    assert fwd(x=None, y=None, rows=0) == 0
    need = L.seq_layer_norm_bwd_workspace_bytes(1000, 64, F32)
    assert need == 4 * 32 * 2 * 64   # 1000 rows, 32 to a workgroup
    assert L.seq_layer_norm_bwd_workspace_bytes(-1, 64, F32) == 0
    assert L.seq_layer_norm_bwd_workspace_bytes(1000, 64, 7) == 0

    def bwd(dy=at(0), x=at(1), w=at(2), mean=at(3), rstd=at(4), dx=at(5), dw=at(6), db=at(7), ws=at(8), nws=need, ld=64, rows=1000):
        return L.seq_layer_norm_bwd(dy, ld, x, 64, w, mean, rstd, dx, 64, dw, db, rows, 64, F32, ws, nws, None)

    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None), dict(nws=need - 4),
                dict(ld=3), dict(dx=at(0)), dict(dw=at(7)), dict(ws=at(1)), dict(rows=-5)):
        assert bwd(**bad) == -1, bad


def test_dropout_refusals(L):
    def fwd(x=at(0), ldx=64, r=at(1), ldr=64, y=at(2), ldy=64, rows=8, C=64, p=0.5, dtype=F16):
        return L.seq_dropout_fwd(x, ldx, r, ldr, y, ldy, rows, C, p, 1, 2, dtype, None)

    for bad in (dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(rows=-1), dict(C=0), dict(x=None), dict(y=None), dict(ldr=10),
                dict(y=at(0)), dict(y=at(1)), dict(dtype=5), dict(rows=1 << 20, C=1 << 20, ldx=1 << 20, ldr=1 << 20, ldy=1 << 20)):
        assert fwd(**bad) == -1, bad
        assert err(L).startswith("seq_dropout_fwd"), bad
    assert L.seq_dropout_bwd(at(0), 64, at(0), 64, 8, 64, 0.5, 1, 2, F32, None) == -1
    assert fwd(rows=0, x=None, r=None, y=None) == 0


def test_interleaved_columns_do_not_overlap(L):
    """An output that is another half of the input's buffer is not refused for
    its span; one that shares a column is."""
    e = 4
    # x is columns [0, 64), y columns [64, 128) of [8, 128]: no shared byte, so the refusal is p's
    assert L.seq_dropout_fwd(at(0), 128, None, 0, at(0) + 64 * e, 128, 8, 64, 2.0, 1, 2, F32, None) == -1
    assert "p=2" in err(L)
    assert L.seq_dropout_fwd(at(0), 128, None, 0, at(0) + 63 * e, 128, 8, 64, 0.5, 1, 2, F32, None) == -1
    assert "overlap" in err(L)
    assert L.seq_dropout_fwd(at(0) + 63 * e, 128, None, 0, at(0), 128, 8, 64, 0.5, 1, 2, F32, None) == -1
    assert "overlap" in err(L)


def test_conv_refusals(L):
    def fwd(x=at(0), ldx=64, w=at(1), b=at(2), si=at(3), y=at(4), ldy=64, so=at(5), cu=None, S=2, total=16, ln=8, D=64, K=4, dtype=BF16):
        return L.seq_causal_conv_fwd(x, ldx, w, b, si, y, ldy, so, cu, S, total, ln, D, K, 1, dtype, None)

    for bad in (dict(K=1), dict(K=5), dict(D=0), dict(D=16385, ldx=20000, ldy=20000), dict(S=-1), dict(S=0), dict(total=15), dict(ln=7),
                dict(total=-16), dict(x=None), dict(w=None), dict(y=None), dict(y=at(0)), dict(so=at(3)), dict(cu=at(6) + 2),
                dict(ldx=60), dict(dtype=9), dict(x=at(0) + 1), dict(S=(1 << 20) + 1, cu=at(6))):
        assert fwd(**bad) == -1, bad
        assert err(L).startswith("seq_causal_conv_fwd"), bad
    assert fwd(S=0, total=0, ln=0, x=None, y=None, si=None, so=None) == 0
    need = L.seq_causal_conv_bwd_workspace_bytes(2, 16, 8, 0, 64, 4)
    assert need == 4 * 1 * 64 * 5
    assert L.seq_causal_conv_bwd_workspace_bytes(2, 16, 8, 0, 64, 7) == 0

    def bwd(dy=at(0), x=at(1), dx=at(2), dw=at(3), db=at(4), ws=at(5), nws=need):
        return L.seq_causal_conv_bwd(dy, 64, x, 64, at(6), at(7), None, dx, 64, dw, db, None, 2, 16, 8, 64, 4, 1, F32, ws, nws, None)

    for bad in (dict(dy=None), dict(x=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(nws=need - 1), dict(dx=at(0)),
                dict(db=at(3)), dict(ws=at(2))):
        assert bwd(**bad) == -1, bad

    def step(x=at(0), st=at(1), y=at(2), S=3, K=4):
        return L.seq_causal_conv_step(x, 64, st, at(3), None, y, 64, S, 64, K, 1, F32, None)

    for bad in (dict(x=None), dict(st=None), dict(y=None), dict(S=-1), dict(K=0), dict(y=at(1)), dict(st=at(0)), dict(S=1 << 21)):
        assert step(**bad) == -1, bad
    assert step(S=0, x=None, st=None, y=None) == 0


def test_launches_beyond_a_grid_are_refused(L):
    """2^20 sequences of one row: 2^18 workgroups of four times 128 blocks of 128
    channels are 2^25, of 2^24 that 2^32 lanes make; half the channels, less one
    sequence, pass this check and fail at the next (a NULL operand)."""
    n = 1 << 20

    def conv(S, D):
        return L.seq_causal_conv_fwd(None, D, at(1), None, None, at(2), D, None, None, S, S, 1, D, 4, 1, BF16, None)

    assert conv(n, 16384) == -1 and "workgroups" in err(L)
    assert conv(n, 8192) == -1 and "workgroups" in err(L)
    assert conv(n - 4, 8192) == -1 and "x is NULL" in err(L)
    assert L.seq_causal_conv_bwd_workspace_bytes(n, n, 1, 0, 16384, 4) == 0
    big = dict(total=n, n_seq=n, len=1, ldu=16384, lddt=16384, ldz=16384, D=16384)
    # a wavefront per group of one channel, and per 64 channels of one group
    for more in (dict(G=16384, N=1, ldb=16384, ldc=16384), dict(G=1, N=1)):
        a = scan(**dict(big, **more))
        assert L.seq_selective_scan_fwd_workspace_bytes(a) == 0 and "workgroups" in err(L)
        assert L.seq_selective_scan_hist_floats(a) == 0
        assert L.seq_selective_scan_fwd(a, at(10), 16384, None, None, None, 0, None) == -1 and "workgroups" in err(L)
    a = scan(**dict(big, G=1, N=1, D=4096))
    assert L.seq_selective_scan_hist_floats(a) == 0
    a = scan(**dict(big, G=1, N=1, D=4032))
    assert L.seq_selective_scan_hist_floats(a) == n * 4032


def scan(**more):
    from recurrent_cell_amd import seq
    a = dict(u=at(0), ldu=64, dt=at(1), lddt=64, z=at(2), ldz=64, B=at(3), ldb=32, C=at(4), ldc=32, A=at(5), skip=at(6), dt_bias=at(7),
             h0=at(8), cu_seqlens=None, total=600, len=300, n_seq=2, D=64, N=16, G=2, softplus=1, dtype=F32)
    a.update(more)
    return seq._Scan(*[a[n] for n, _ in seq._Scan._fields_])


def test_scan_refusals(L):
    from recurrent_cell_amd import seq

    def fwd(a, y=at(10), ldy=64, hl=at(11), hist=at(12), ws=at(13), nws=None):
        n = L.seq_selective_scan_fwd_workspace_bytes(a) if nws is None else nws
        return L.seq_selective_scan_fwd(a, y, ldy, hl, hist, ws, n, None)

    assert L.seq_selective_scan_fwd(None, at(10), 64, None, None, None, 0, None) == -1
    for bad in (dict(D=0), dict(N=0), dict(N=65), dict(G=3), dict(G=0), dict(dtype=3), dict(total=601), dict(n_seq=0), dict(n_seq=-1),
                dict(u=None), dict(dt=None), dict(B=None), dict(C=None), dict(A=None), dict(ldu=63), dict(ldb=31), dict(A=at(5) + 2),
                dict(h0=at(8) + 1)):
        assert fwd(scan(**bad)) == -1, bad
        assert err(L).startswith("seq_selective_scan_fwd"), bad
    ok = scan()
    need = L.seq_selective_scan_fwd_workspace_bytes(ok)
    assert need > 0
    for bad in (dict(y=None), dict(ldy=63), dict(ws=None), dict(nws=need - 4), dict(y=at(0)), dict(hl=at(8)), dict(hist=at(11)), dict(ws=at(3))):
        assert fwd(ok, **bad) == -1, bad
    assert L.seq_selective_scan_hist_floats(ok) == 2 * 5 * 16 * 64
    assert L.seq_selective_scan_hist_floats(scan(cu_seqlens=at(9))) == (600 // 64 + 2) * 16 * 64
    assert L.seq_selective_scan_hist_floats(scan(N=99)) == 0
    assert L.seq_selective_scan_fwd_workspace_bytes(scan(total=128, len=64)) == 0   # one piece per sequence
    assert fwd(scan(n_seq=0, total=0, len=0, u=None, dt=None, z=None, B=None, C=None), y=None) == 0

    def bwd(a=ok, dy=at(10), hist=at(11), dh=at(12), ws=at(13), nws=None, **more):
        g = dict(du=at(14), lddu=64, ddt=at(15), ldddt=64, dz=at(16), lddz=64, dB=at(17), dC=at(18), dA=at(19), dskip=at(20),
                 ddt_bias=at(21), dh0=at(22))
        g.update(more)
        n = L.seq_selective_scan_bwd_workspace_bytes(a) if nws is None else nws
        return L.seq_selective_scan_bwd(a, dy, 64, hist, dh, seq._ScanGrads(*[g[n] for n, _ in seq._ScanGrads._fields_]), ws, n, None)

    for bad in (dict(dy=None), dict(hist=None), dict(ws=None), dict(nws=64), dict(du=None), dict(ddt=None), dict(dz=None), dict(dB=None),
                dict(dC=None), dict(dA=None), dict(lddu=60), dict(du=at(0)), dict(dB=at(18)), dict(dh0=at(12)), dict(ws=at(11)),
                dict(a=scan(z=None))):
        assert bwd(**bad) == -1, bad
        assert err(L).startswith("seq_selective_scan_bwd"), bad
    assert L.seq_selective_scan_bwd(ok, at(10), 64, at(11), None, None, at(13), 1 << 30, None) == -1


def test_scan_step_refusals(L):
    def step(h=at(0), u=at(1), dt=at(2), A=at(3), B=at(4), C=at(5), z=at(6), y=at(7), S=4, D=64, N=16, G=1, ldb=16, dtype=F32):
        return L.seq_selective_scan_step(h, u, 64, dt, 64, A, B, ldb, C, 16, None, z, 64, None, y, 64, S, D, N, G, 1, dtype, None)

    for bad in (dict(h=None), dict(u=None), dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(y=None), dict(S=-1), dict(D=65),
                dict(N=0), dict(N=65), dict(G=5), dict(ldb=15), dict(y=at(0)), dict(h=at(1)), dict(dtype=4), dict(S=1 << 21)):
        assert step(**bad) == -1, bad
        assert err(L).startswith("seq_selective_scan_step"), bad
    assert step(S=0, h=None, u=None, dt=None, B=None, C=None, z=None, y=None) == 0


def test_binding_refuses_cpu_tensors(L):
    from recurrent_cell_amd import seq
    x = torch.zeros(4, 8)
    for call in (lambda: seq.layer_norm_fwd(x), lambda: seq.dropout_fwd(x, 0.5, 1), lambda: seq.causal_conv_fwd(x, torch.zeros(8, 4)),
                 lambda: seq.causal_conv_step(x, torch.zeros(4, 3, 8), torch.zeros(8, 4)),
                 lambda: seq.selective_scan_fwd(x, x, torch.zeros(2, 8), torch.zeros(4, 2), torch.zeros(4, 2))):
        with pytest.raises(TypeError, match="GPU tensor"):
            call()


def test_row_strides():
    """Row strides that the binding finds or refuses (host logic alone)."""
    from recurrent_cell_amd.seq import _row_stride
    x = torch.zeros(3, 5, 16)
    assert _row_stride(x, "x", 2) == 16
    assert _row_stride(x[..., :7], "x", 2) == 16
    assert _row_stride(x[:1, :, :7], "x", 2) == 16
    assert _row_stride(x[:, :1, :7], "x", 2) == 80
    assert _row_stride(x[:1, :1, :7], "x", 2) == 7
    assert _row_stride(x.view(3, 5, 2, 8)[..., :8], "x", 2) == 16
    assert _row_stride(torch.zeros(0, 4), "x", 1) == 4
    for bad, lead in ((x[:, :4], 2), (x.transpose(0, 1), 2), (x[..., ::2], 2), (x.view(3, 5, 2, 8)[..., :7], 2),
                      (torch.zeros(1, 8).expand(4, 8), 1)):
        with pytest.raises(TypeError):
            _row_stride(bad, "x", lead)


def test_gradient_sums_beyond_a_grid_are_refused(L):
    """dB and dC of 8,192 rows x 16,384 groups x 64 states are 2^34 values, four
    to a lane of the launch that sums them: 2^32 lanes.  The forward pass has no
    such launch; 64 rows fewer pass this check and fail at the next."""
    from recurrent_cell_amd import seq

    def bwd(a):
        return L.seq_selective_scan_bwd(a, at(10), 16384, at(11), None, seq._ScanGrads(
            at(14), 16384, at(15), 16384, at(16), 16384, at(17), at(19), at(21), at(22), at(23), at(24)), at(40), 1 << 40, None)

    def args(rows):
        return scan(total=rows, len=rows, n_seq=1, D=16384, G=16384, N=64, ldu=16384, lddt=16384, ldz=16384, ldb=1 << 20, ldc=1 << 20,
                    dtype=BF16, u=None, C=at(60))

    a = args(8192)
    assert L.seq_selective_scan_bwd_workspace_bytes(a) == 0 and "workgroups" in err(L)
    assert bwd(a) == -1 and "workgroups" in err(L)
    assert L.seq_selective_scan_hist_floats(a) == 8192 // 64 * 64 * 16384
    assert L.seq_selective_scan_fwd(a, at(10), 16384, None, at(11), at(40), 1 << 40, None) == -1 and "u is NULL" in err(L)
    a = args(8192 - 64)
    assert L.seq_selective_scan_bwd_workspace_bytes(a) > 1 << 36
    assert bwd(a) == -1 and "u is NULL" in err(L)

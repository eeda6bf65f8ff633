"""The parts of a layer (conv, scan, gated norm, dense projection): refusals of bad
arguments before anything is enqueued, and pins of their fp64 forms against the layer
oracle."""
import ctypes as C

import numpy as np
import pytest

from bit_scaffold_quantized_b200 import dfssm as F
from bit_scaffold_quantized_b200 import synth as S
from oracle import dfssm_oracle as O
from oracle import parts_oracle as PO

FAKE = 1 << 20     # aligned, never dereferenced: the checks fail first
NULL = None


def rows(ptr=FAKE, stride=1 << 20, dtype=F.DTYPE_F32):
    return C.byref(F.CRows(ptr, stride, dtype))


def seqs(n=2, r=8, slots=4, start=FAKE, slot=FAKE, fresh=0, status=0):
    return C.byref(F.CSeqs(n, r, slots, start, slot, fresh, status))


def scan(h=8, p=64, n=16, g=1, st=F.DTYPE_F32, bias=FAKE, a=FAKE, d=FAKE):
    return C.byref(F.CScan(h, p, n, g, st, bias, a, d))


def expect(code, rc, text):
    assert rc == code, (rc, F.last_error())
    assert text in F.last_error(), F.last_error()


INV, SHAPE, MIS, SMALL = F.ERR_INVALID_ARG, F.ERR_UNSUPPORTED_SHAPE, F.ERR_MISALIGNED, F.ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("token", [False, True])
def test_conv_refusals(token):
    L = F.lib()
    fn = L.dfssm_conv_token if token else L.dfssm_conv_prompt
    good = seqs(n=8, start=0) if token else seqs()

    def call(c=64, w=4, x=rows(), wt=FAKE, b=FAKE, q=good, st=FAKE, y=rows(ptr=2 * FAKE)):
        return fn(c, w, 1, x, wt, b, q, st, y, None)
    expect(INV, call(c=0), "channels")
    expect(SHAPE, call(c=(1 << 28) + 4, x=rows(stride=1 << 30)), "channels")
    expect(SHAPE, call(w=1), "d_conv")
    expect(SHAPE, call(w=5), "d_conv")
    expect(INV, call(x=NULL), "x is NULL")
    expect(INV, call(x=rows(ptr=0)), "x is NULL")
    expect(INV, call(y=rows(dtype=2)), "dtype")
    expect(INV, call(x=rows(stride=63)), "stride")
    expect(INV, call(x=rows(stride=-64)), "stride")
    expect(MIS, call(x=rows(ptr=FAKE + 2)), "aligned")
    expect(INV, call(y=rows(ptr=FAKE)), "y may not")
    expect(INV, call(wt=0), "w is NULL")
    expect(MIS, call(wt=FAKE + 2), "w is not")
    expect(MIS, call(b=FAKE + 8), "b is not")
    expect(MIS, call(st=FAKE + 4), "conv_state")
    expect(INV, call(q=NULL), "seqs")
    expect(INV, call(q=seqs(n=-1, start=0 if token else FAKE)), "n_seqs")
    expect(MIS, call(q=seqs(n=8, slot=FAKE + 2, start=0 if token else FAKE)), "slot")
    expect(INV, call(q=seqs(n=8, slot=0, slots=4, start=0 if token else FAKE)), "slot numbers")
    if token:
        expect(INV, call(q=seqs(n=8)), "start must be NULL")
        expect(INV, call(q=seqs(n=7, start=0)), "n_rows")
        expect(INV, call(st=0), "conv_state is NULL")
    else:
        expect(INV, call(q=seqs(start=0)), "start is NULL")
    # nothing to do
    assert call(q=seqs(n=0, r=0, start=0 if token else FAKE)) == 0


@pytest.mark.parametrize("token", [False, True])
def test_scan_refusals(token):
    L = F.lib()
    good = seqs(n=8, start=0) if token else seqs()

    def call(s=scan(), x=rows(), dt=rows(), B=rows(), Cm=rows(), q=good, st=FAKE, y=rows(ptr=2 * FAKE), ws=FAKE, n=1 << 30):
        if token:
            return L.dfssm_scan_token(s, x, dt, B, Cm, q, st, y, None)
        return L.dfssm_scan_prompt(s, x, dt, B, Cm, q, st, y, ws, n, None)
    expect(INV, call(s=NULL), "scan is NULL")
    expect(INV, call(s=scan(h=0)), "positive")
    expect(SHAPE, call(s=scan(h=8, g=3)), "ngroups")
    expect(SHAPE, call(s=scan(p=60)), "headdim")
    expect(SHAPE, call(s=scan(p=144)), "headdim")
    expect(SHAPE, call(s=scan(n=18)), "d_state")
    expect(SHAPE, call(s=scan(n=260)), "d_state")
    expect(SHAPE, call(s=scan(h=65536)), "nheads")
    expect(INV, call(s=scan(st=2)), "state_dtype")
    expect(INV, call(s=scan(bias=0)), "dt_bias")
    expect(MIS, call(s=scan(d=FAKE + 4)), "D is not")
    expect(INV, call(x=rows(stride=511)), "stride")
    expect(INV, call(dt=rows(stride=7)), "stride")
    expect(INV, call(B=rows(dtype=F.DTYPE_F16)), "one dtype")
    expect(MIS, call(Cm=rows(ptr=FAKE + 2)), "aligned")
    for k in ("x", "dt", "B", "Cm"):
        expect(INV, call(**{k: rows(ptr=2 * FAKE)}), "y may not")
    expect(MIS, call(st=FAKE + 8), "state")
    if token:
        expect(INV, call(st=0), "state is NULL")
        expect(INV, call(q=seqs(n=8)), "start must be NULL")
    else:
        expect(INV, call(q=seqs(start=0)), "start is NULL")
        expect(INV, call(ws=0), "ws is NULL")
        expect(MIS, call(ws=FAKE + 8), "ws is not")
        expect(SMALL, call(n=8), "workspace")
    assert call(q=seqs(n=0, r=0, start=0 if token else FAKE)) == 0


def test_scan_workspace_query():
    L = F.lib()
    assert L.dfssm_scan_workspace_bytes(scan(p=60), F.DTYPE_F32, 1, 1) == 0
    assert L.dfssm_scan_workspace_bytes(scan(), 5, 1, 1) == 0
    assert L.dfssm_scan_workspace_bytes(scan(), F.DTYPE_F32, -1, 1) == 0
    one = F.scan_workspace_bytes(64, 64, 128, 1, 1, 1)
    long = F.scan_workspace_bytes(64, 64, 128, 1, 1, 8192)
    assert 0 < one <= long
    # offsets past 32 bits: a long prompt's states between segments
    assert F.scan_workspace_bytes(80, 128, 256, 1, 65536, 1 << 20, half=True) > 0


def test_norm_and_dense_refusals():
    L = F.lib()

    def norm(r=4, c=512, g=1, y=rows(), z=rows(), w=FAKE, out=rows(ptr=2 * FAKE)):
        return L.dfssm_gated_norm(r, c, g, y, z, w, out, None)
    expect(INV, norm(r=-1), "rows")
    expect(INV, norm(g=0), "ngroups")
    expect(SHAPE, norm(g=3), "ngroups")
    expect(SHAPE, norm(c=(1 << 30) + 8), "cols")
    expect(INV, norm(y=NULL), "y is NULL")
    expect(INV, norm(w=0), "w is NULL")
    expect(INV, norm(z=rows(stride=511)), "z: stride")
    expect(INV, norm(out=rows(dtype=F.DTYPE_F16)), "shares")
    expect(INV, norm(out=rows(stride=1 << 19)), "shares")
    expect(SHAPE, norm(r=1 << 30, c=512, g=8), "out of range")
    assert norm(r=0) == 0

    def dense(o=64, k=64, n=4, w=FAKE, b=FAKE, x=rows(dtype=F.DTYPE_F16), r=NULL, y=rows(ptr=2 * FAKE), st=NULL):
        return L.dfssm_dense_forward(o, k, n, w, b, 0, x, r, y, st, None)
    expect(INV, dense(o=0), "rows")
    expect(INV, dense(n=-1), "batch")
    for k in "okn":
        expect(SHAPE, dense(**{k: (1 << 30) + 8}), "2^30")
    expect(INV, dense(w=0), "w is NULL")
    expect(MIS, dense(w=FAKE + 2), "w is not")
    expect(MIS, dense(b=FAKE + 2), "b is not")
    expect(INV, dense(x=rows()), "x must be fp16")
    expect(INV, dense(x=rows(dtype=F.DTYPE_F16, stride=63)), "x: stride")
    expect(INV, dense(r=rows(ptr=2 * FAKE, dtype=F.DTYPE_F16)), "shares")
    expect(INV, dense(r=rows(ptr=0)), "residual is NULL")
    expect(INV, dense(y=rows()), "y may not")
    expect(MIS, dense(st=FAKE + 2), "status")
    assert dense(n=0) == 0


def test_binding_refuses_before_the_library_is_called():
    """Shapes, types and devices, checked before any pointer is taken (host tensors here: the
    device is looked at last)."""
    import torch
    x, w = torch.zeros(4, 8), torch.zeros(8, dtype=torch.float16)

    def no(text, fn, *args, **kw):
        with pytest.raises(ValueError, match=text):
            fn(*args, **kw)
    for other in (torch.zeros(4, 9), torch.zeros(3, 8), torch.zeros(8, 4).t(), torch.zeros(4, 8, dtype=torch.float64)):
        no("CUDA|out must", F.gated_norm, x, x, w, other)
    no("CUDA device", F.gated_norm, x, x, w, x)
    no("matri", F.gated_norm, x[0], x, w, x)
    no("CUDA", F.conv_token, x, torch.zeros(8, 4).half(), None, torch.zeros(4, 3, 8), x)
    no("start", F.conv_prompt, x, torch.zeros(8, 4).half(), None, torch.zeros(4, 3, 8), x, None)
    no("headdim", F.scan_prompt, x, x, x, x, torch.zeros(1), torch.zeros(1), None, None, x, torch.zeros(2).int(), x)
    no("state", F.scan_token, x, x, x, x, torch.zeros(1), torch.zeros(1), None, torch.zeros(2, 2, 8, 8), x)
    no("CUDA", F.dense_forward, torch.zeros(8, 8).half(), x, x)


def test_live_sequences():
    f = PO.live_sequences
    assert f(3, 10, [0, 4, 4, 10], None, 3) == [(0, 0, 4, 0), (2, 4, 10, 2)]
    assert f(3, 10, [2, 4, 9, 10], [5, -1, 5], 6) == [(0, 2, 4, 5)]
    assert f(2, 10, [0, 11, 12], None, 2) == []
    assert f(2, 2, None, [3, 1], 3) == [(1, 1, 2, 1)]


@pytest.mark.parametrize("cuts", [[0, 1, 4, 70], [0, 3, 3, 5]])
def test_fp64_forms_equal_the_layer_oracle(cuts):
    """Each packed prompt through the plain forms equals the layer oracle's own prompt pass."""
    d = S.LAYER_SMALL
    rng = np.random.default_rng(5)
    lw = S.gen_layer(rng, d)
    n = len(cuts) - 1
    E, Cd, N = d.d_inner, d.conv_dim, d.d_state
    conv0 = rng.normal(size=(n, d.d_conv - 1, Cd)).astype(np.float32)
    ssm0 = rng.normal(size=(n, d.nheads, d.headdim, N)).astype(np.float32)
    res = [S.gen_layer_inputs(rng, d, max(b - a, 1)).transpose(1, 0, 2)[:, :b - a].copy()
           for a, b in zip(cuts, cuts[1:])]
    traces = {i: O.layer_prefill(r, lw, O.State(conv0[i:i + 1], ssm0[i:i + 1]), d)
              for i, r in enumerate(res) if r.shape[1]}
    z = np.concatenate([t.zxbcdt.reshape(-1, d.in_rows) for t in traces.values()])
    xc, _, cs = PO.conv(z[:, E:E + Cd], lw.conv_w, lw.conv_b, cuts, None, None, conv0)
    y, _, hs, _ = PO.scan(xc[:, :E], z[:, E + Cd:], xc[:, E:E + N], xc[:, E + N:], lw.dt_bias, lw.A_log, lw.D, cuts, None,
                          None, ssm0)
    xo = PO.gated_norm(y, z[:, :E], lw.gnorm_w)
    for i, t in traces.items():
        a, b = cuts[i], cuts[i + 1]
        np.testing.assert_allclose(xc[a:b], t.xc.reshape(-1, Cd), rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(y[a:b] * PO.silu(z[a:b, :E]), t.g.reshape(-1, E), rtol=1e-6, atol=1e-9)
        np.testing.assert_allclose(hs[i], t.ssm[0], rtol=1e-6, atol=1e-6)
        np.testing.assert_allclose(cs[i], t.conv[0], rtol=1e-6, atol=1e-7)
        np.testing.assert_allclose(xo[a:b], np.float64(t.x_out.reshape(-1, E)), rtol=2e-3, atol=1e-6)
    for i in set(range(n)) - set(traces):
        assert np.array_equal(hs[i], np.float64(ssm0[i])) and np.array_equal(cs[i], np.float64(conv0[i]))

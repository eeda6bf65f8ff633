"""GPU tests of the parts of a layer (conv, scan, gated norm, dense projection) against
their plain fp64 forms.

Tolerances.  A sum of terms of total magnitude A that is evaluated in fp32 through k
roundings is off by at most k 2^-24 A; the result is rounded once more to its row's type
(half a step: eps / 2 of the value, plus half the smallest subnormal).  k counts:
conv: the taps and the bias.  Scan: the d_state products of a row, the rows of a chunk
(at most 128), two roundings per chunk of the carried state and per join of segments, and
the decays: exp of an fp32 exponent v is off by |v| 2^-24 of itself, |v| exp(-|v|) <= 0.37,
so a few roundings.  Dense: the products; adds on the tensor cores do not round to
nearest and count twice.  SiLU: slope at most 1.1, its own error within 8 2^-24."""
import numpy as np
import pytest
import torch

from bit_scaffold_quantized_b200 import dfssm as F
from bit_scaffold_quantized_b200 import synth as S
from oracle import dfssm_oracle as O
from oracle import parts_oracle as PO

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
MARK = 7.5          # fills outputs beforehand: rows that are not to be written keep it
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    F.lib()


def half_step(t, v):
    tiny = 2.0 ** -25 if t == F16 else 2.0 ** -150
    return torch.finfo(t).eps / 2 * np.abs(v) + tiny


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def wide(a, dtype, pad):
    """a as a view of wider rows, `pad` values to the left, on the device."""
    t = torch.full((a.shape[0], a.shape[1] + pad), 3.25, dtype=dtype, device=DEV)
    t[:, pad:] = dev(a).to(dtype)
    return t[:, pad:]


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)


def check(name, got, want, tol):
    """Rows with NaN in `want` were not to be written; elsewhere |got - want| <= tol."""
    keep = np.isnan(want)
    assert np.all(got[keep] == MARK), f"{name}: rows of no sequence were written"
    bad = np.abs(got - want)[~keep] > tol[~keep]
    assert np.all(np.isfinite(got[~keep])) and not bad.any(), (
        f"{name}: {bad.sum()} of {bad.size} off, worst {np.max((np.abs(got - want) / tol)[~keep])} times the bound")


# lengths, first row, rows behind the last sequence, slots (None: own), pool size, fresh
PACKS = {
    "one row": ([1], 0, 0, None, 1, None),
    "two rows": ([2], 0, 0, [2], 3, None),
    "three rows": ([3], 1, 2, None, 1, None),
    "empty ones": ([0, 5, 0, 0, 2, 0], 0, 1, [4, 0, 1, 5, 3, 2], 6, [1, 0, 1, 0, 1, 1]),
    "tile edges": ([31, 33, 64, 1, 65, 127], 0, 0, [6, 2, 0, 1, 5, 3], 7, [0, 1, 0, 1, 0, 0]),
    "many short": ([1, 2, 3, 1, 1, 4] * 9, 2, 3, None, 54, None),
    "chunk edges": ([128, 129, 256, 255], 3, 5, [3, 1, 0, 2], 4, [0, 0, 1, 0]),
    "left out": ([5, 40, 7, 3, 9], 0, 0, [1, -1, 1, 9, 2], 4, None),
    "all left out": ([5, 6], 0, 0, [-1, -1], 2, None),
}


def pack(key):
    lens, first, behind, slot, slots, fresh = PACKS[key]
    cuts = list(first + np.concatenate([[0], np.cumsum(lens)]))
    return [int(c) for c in cuts], int(cuts[-1]) + behind, slot, slots, fresh


# ------------------------------------------------------------------ conv

def conv_case(rows, C, W, xt, seed, slots, bias=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, C)).astype(np.float16 if xt == F16 else np.float32)
    w = rng.uniform(-0.5, 0.5, size=(C, W)).astype(np.float16)
    b = rng.uniform(-0.5, 0.5, size=C).astype(np.float16) if bias else None
    return x, w, b, rng.normal(size=(slots, W - 1, C)).astype(np.float32)


def conv_tol(yt, y, A, W, act):
    err = (W + 2) * U * A
    if act:
        err = 1.1 * err + 8 * U * np.abs(y)
    return err + half_step(yt, y)


@pytest.mark.parametrize("key", list(PACKS))
@pytest.mark.parametrize("xt,yt,C,W,pad,act,bias", [
    (F32, F16, 544, 4, 516, True, True), (F16, F16, 544, 4, 0, True, True), (F16, F32, 33, 3, 0, True, False),
    (F32, F32, 7, 2, 5, False, True), (F32, F32, 516, 4, 3, True, True)])
def test_conv_prompt(key, xt, yt, C, W, pad, act, bias):
    cuts, rows, slot, slots, fresh = pack(key)
    x, w, b, st = conv_case(rows, C, W, xt, 11, slots, bias)
    y, A, new = PO.conv(x, w, b, cuts, slot, fresh, st, act)
    yd, sd = torch.full((rows, C), MARK, dtype=yt, device=DEV), dev(st)
    F.conv_prompt(wide(x, xt, pad), dev(w), None if b is None else dev(b), sd, yd, ints(cuts), ints(slot), ints(fresh),
                  silu=act)
    check("y", host(yd), y, conv_tol(yt, y, A, W, act))
    assert np.array_equal(host(sd), new)             # the state holds inputs, unrounded


def test_conv_prompt_without_state():
    cuts, rows, _, _, _ = pack("tile edges")
    x, w, b, _ = conv_case(rows, 544, 4, F16, 12, 1)
    y, A, _ = PO.conv(x, w, b, cuts, None, None, None)
    yd = torch.full((rows, 544), MARK, dtype=F32, device=DEV)
    F.conv_prompt(dev(x), dev(w), dev(b), None, yd, ints(cuts), slot=ints([-1] * 6))
    check("y", host(yd), y, conv_tol(F32, y, A, 4, True))


@pytest.mark.parametrize("xt,yt,C,W,pad", [(F32, F16, 544, 4, 516), (F16, F32, 33, 3, 1), (F16, F16, 7, 2, 0)])
@pytest.mark.parametrize("slot,slots,fresh", [
    (None, 5, None), ([3, -1, 0, 3, 5], 5, [0, 0, 1, 0, 0]), ([4, 3, 2, 1, 0], 6, [1, 1, 1, 1, 1])])
def test_conv_token(xt, yt, C, W, pad, slot, slots, fresh):
    x, w, b, st = conv_case(5, C, W, xt, 13, slots)
    y, A, new = PO.conv(x, w, b, None, slot, fresh, st)
    yd, sd = torch.full((5, C), MARK, dtype=yt, device=DEV), dev(st)
    F.conv_token(wide(x, xt, pad), dev(w), dev(b), sd, yd, ints(slot), ints(fresh))
    check("y", host(yd), y, conv_tol(yt, y, A, W, True))
    assert np.array_equal(host(sd), new)


def test_conv_pieces_equal_the_whole():
    """A prompt in pieces, then token by token, gives the bits of the prompt in one call."""
    C, T = 544, 90
    x, w, b, st = conv_case(T, C, 4, F32, 14, 2)
    xd, wd, bd = dev(x), dev(w), dev(b)
    whole, s1 = torch.empty(T, C, dtype=F32, device=DEV), dev(st)
    F.conv_prompt(xd, wd, bd, s1, whole, ints([0, T]), ints([1]))
    parts, s2 = torch.empty_like(whole), dev(st)
    cuts = [0, 1, 3, 40, 41, 86]
    for a, e in zip(cuts, cuts[1:]):
        F.conv_prompt(xd[a:e], wd, bd, s2, parts[a:e], ints([0, e - a]), ints([1]))
    for t in range(86, T):
        F.conv_token(xd[t:t + 1], wd, bd, s2, parts[t:t + 1], ints([1]))
    assert torch.equal(whole, parts) and torch.equal(s1, s2)


# ------------------------------------------------------------------ scan

SHAPES = [(8, 64, 16, 1), (4, 64, 128, 1), (3, 16, 4, 3), (6, 32, 20, 2), (2, 128, 256, 1), (5, 48, 200, 5),
          (2, 96, 64, 1), (1, 64, 128, 1), (6, 64, 64, 2),
          (8, 64, 64, 2), (4, 64, 128, 2)]


def scan_case(rows, shape, xt, dtt, st, slots, seed, decay=16.0):
    H, P, N, G = shape
    rng = np.random.default_rng(seed)
    cast = lambda v, t: v.astype(np.float16 if t == F16 else np.float32)  # noqa: E731
    return dict(x=cast(rng.normal(size=(rows, H * P)), xt), dt=cast(rng.normal(size=(rows, H)), dtt),
                B=cast(rng.normal(size=(rows, G * N)), xt), C=cast(rng.normal(size=(rows, G * N)), xt),
                dt_bias=rng.uniform(-5, 1, size=H).astype(np.float32),
                A_log=np.log(rng.uniform(0.02, decay, size=H)).astype(np.float32),
                D=rng.normal(size=H).astype(np.float32),
                state=cast(rng.normal(size=(slots, H, P, N)), st))


def scan_oracle(c, cuts, slot, fresh, D=True):
    return PO.scan(c["x"], c["dt"], c["B"], c["C"], c["dt_bias"], c["A_log"], c["D"] if D else None, cuts, slot, fresh,
                   c["state"])


def scan_k(shape, rows):
    return shape[2] + 160 + rows // 4


def run_scan(c, cuts, slot, fresh, yt, xt, D=True, pads=(0, 0, 0, 0), status=None, stream=None, ws=None):
    rows = c["x"].shape[0]
    H, P, N = c["state"].shape[1:]
    yd, sd = torch.full((rows, H * P), MARK, dtype=yt, device=DEV), dev(c["state"])
    a = [wide(c[k], xt if k != "dt" else (F16 if c["dt"].dtype == np.float16 else F32), p)
         for k, p in zip(("x", "dt", "B", "C"), pads)]
    par = [dev(c["dt_bias"]), dev(c["A_log"]), dev(c["D"]) if D else None]
    if cuts is None:
        F.scan_token(*a, *par, sd, yd, slot=ints(slot), fresh=ints(fresh), status=status, stream=stream)
    else:
        ws = F.scan_workspace(a[0], sd, len(cuts) - 1, a[2].shape[1] // N) if ws is None else ws
        ws.fill_(255)           # NaNs, should anything be read before it is written
        F.scan_prompt(*a, *par, sd, yd, ints(cuts), ws, slot=ints(slot), fresh=ints(fresh), status=status, stream=stream)
    return yd, sd


def check_scan(c, got, want, shape, yt, rows):
    (yd, sd), (y, A, new, newA) = got, want
    k = scan_k(shape, rows)
    check("y", host(yd), y, k * U * A + half_step(yt, y))
    tol = k * U * newA + half_step(sd.dtype, new)
    same = newA == np.abs(np.float64(c["state"]))        # untouched slots (or unchanged values)
    assert np.array_equal(host(sd)[same], new[same])
    bad = np.abs(host(sd) - new) > tol
    assert not bad.any(), f"state: {bad.sum()} off, worst {np.max(np.abs(host(sd) - new) / tol)} times the bound"


@pytest.mark.parametrize("key", list(PACKS))
@pytest.mark.parametrize("shape", SHAPES[:2] + SHAPES[3:4])
@pytest.mark.parametrize("xt,yt,st", [(F16, F16, F32), (F32, F32, F32), (F16, F32, F16)])
def test_scan_prompt_packs(key, shape, xt, yt, st):
    cuts, rows, slot, slots, fresh = pack(key)
    c = scan_case(rows, shape, xt, F32, st, slots, 21)
    got = run_scan(c, cuts, slot, fresh, yt, xt)
    check_scan(c, got, scan_oracle(c, cuts, slot, fresh), shape, yt, rows)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("xt,yt,st,dtt,D,pads", [
    (F16, F16, F32, F16, True, (8, 0, 8, 16)), (F32, F32, F16, F16, False, (4, 1, 4, 8)),
    (F16, F16, F32, F32, False, (1, 3, 3, 5)), (F32, F16, F32, F32, True, (0, 0, 1, 2))])
def test_scan_prompt_shapes(shape, xt, yt, st, dtt, D, pads):
    cuts, rows, slot, fresh = [0, 70, 70, 231], 233, [2, 0, 1], [0, 0, 1]
    c = scan_case(rows, shape, xt, dtt, st, 3, 22)
    got = run_scan(c, cuts, slot, fresh, yt, xt, D, pads)
    check_scan(c, got, scan_oracle(c, cuts, slot, fresh, D), shape, yt, rows)


@pytest.mark.parametrize("xt,yt", [(F16, F16), (F32, F32), (F16, F32)])
@pytest.mark.parametrize("rows,cuts", [(2000, [0, 2000]), (1500, [0, 3, 1100, 1497]), (1024, [0, 512, 1024])])
def test_scan_prompt_in_segments(xt, yt, rows, cuts):
    """Long prompts of few heads, whose rows are divided among blocks, little decay: what
    the segments hand on matters to the end."""
    shape = (2, 64, 128, 1)
    c = scan_case(rows, shape, xt, F32, F32, 4, 23, decay=0.5)
    c["dt_bias"] -= 3
    got = run_scan(c, cuts, [3, 0, 1][:len(cuts) - 1], None, yt, xt, D=False)
    check_scan(c, got, scan_oracle(c, cuts, [3, 0, 1][:len(cuts) - 1], None, False), shape, yt, rows)


@pytest.mark.parametrize("xt", [F16, F32])
def test_scan_prompt_strong_and_no_decay(xt):
    """Steps from 0 (the state stands still) to huge (the state is forgotten at once)."""
    shape, rows, cuts = (4, 64, 128, 1), 200, [0, 130, 200]
    c = scan_case(rows, shape, xt, F32, F32, 2, 24)
    c["dt"][::3] = -200.0        # dt = 0
    c["dt"][1::7] = 60.0         # dt = 60: decay exp(-960)
    got = run_scan(c, cuts, None, None, F32, xt)
    check_scan(c, got, scan_oracle(c, cuts, None, None), shape, F32, rows)


@pytest.mark.parametrize("xt", [F16, F32])
@pytest.mark.parametrize("scale", [2.0 ** -14, 1.0, 2.0 ** 12])
def test_scan_prompt_scales(xt, scale):
    """Tiny and large activations: nothing under- or overflows on the way."""
    shape, rows, cuts = (4, 64, 128, 1), 300, [0, 300]
    c = scan_case(rows, shape, xt, F32, F32, 1, 25)
    c["x"] = (np.float64(c["x"]) * scale).astype(c["x"].dtype)
    c["state"] = (c["state"] * scale).astype(np.float32)
    got = run_scan(c, cuts, None, None, F32, xt, D=False)
    check_scan(c, got, scan_oracle(c, cuts, None, None, False), shape, F32, rows)


def test_scan_prompt_large_b_and_c():
    shape, rows, cuts = (4, 64, 128, 1), 140, [0, 140]
    c = scan_case(rows, shape, F16, F32, F32, 1, 26)
    c["B"], c["C"] = c["B"] * np.float16(300), c["C"] * np.float16(300)      # sums of products beyond fp16
    got = run_scan(c, cuts, None, None, F32, F16)
    check_scan(c, got, scan_oracle(c, cuts, None, None), shape, F32, rows)


@pytest.mark.parametrize("xt", [F16, F32])
@pytest.mark.parametrize("poison", [np.nan, np.inf])
def test_scan_and_conv_keep_neighbours_clean(xt, poison):
    """NaN or infinity in one prompt, behind the last one and in a slot that is begun anew
    reach no other prompt."""
    shape, cuts, rows = (4, 64, 128, 1), [2, 90, 100, 233], 240
    c = scan_case(rows, shape, xt, F32, F32, 3, 27)
    want = scan_oracle(c, [2, 90, 90, 90], [0, 1, 2], [1, 0, 0])
    last = scan_oracle(c, [100, 100, 100, 233], [0, 1, 2], [1, 0, 0])
    for k in ("x", "dt", "B", "C"):
        c[k][90:100] = poison
        c[k][:2] = poison
        c[k][233:] = poison
    c["state"][0] = poison
    yd, sd = run_scan(c, cuts, [0, 1, 2], [1, 0, 0], F32, xt)
    k = scan_k(shape, rows)
    for (y, A, new, newA), (a, e), s in ((want, (2, 90), 0), (last, (100, 233), 2)):
        assert np.all(np.abs(host(yd)[a:e] - y[a:e]) <= k * U * A[a:e] + half_step(F32, y[a:e]))
        assert np.all(np.abs(host(sd)[s] - new[s]) <= k * U * newA[s] + half_step(F32, new[s]))
    x, w, b, st = conv_case(rows, 64, 4, xt, 28, 3)
    y, A, new = PO.conv(x, w, b, cuts, None, [1, 0, 0], st)
    x[90:100] = poison
    x[:2] = poison
    x[233:] = poison
    st[0] = poison
    yd, sd = torch.full((rows, 64), MARK, dtype=F32, device=DEV), dev(st)
    F.conv_prompt(dev(x), dev(w), dev(b), sd, yd, ints(cuts), None, ints([1, 0, 0]))
    for a, e, s in ((2, 90, 0), (100, 233, 2)):
        assert np.all(np.abs(host(yd)[a:e] - y[a:e]) <= conv_tol(F32, y, A, 4, True)[a:e])
        assert np.array_equal(host(sd)[s], new[s])


@pytest.mark.parametrize("shape,xt,pads", [((4, 64, 128, 1), F16, (0, 0, 0, 0)), ((4, 64, 128, 1), F16, (1, 0, 1, 1)),
                                           ((4, 64, 128, 1), F32, (0, 0, 0, 0)), ((2, 128, 160, 1), F32, (0, 0, 0, 0)),
                                           ((2, 48, 20, 2), F16, (0, 0, 0, 0))])
@pytest.mark.parametrize("name", ["x", "dt", "B", "C"])
@pytest.mark.parametrize("poison", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("at,rows", [(0, 140), (77, 140), (139, 140), (700, 1500)])
def test_scan_prompt_no_number_reaches_earlier_rows(shape, xt, pads, name, poison, at, rows):
    """NaN or infinity at one place of a prompt: the rows before it and the heads, channels and
    states that do not depend on it are as the recurrence has them, the others no numbers
    (dt of -inf is a step of 0: all are)."""
    c = scan_case(rows, shape, xt, F32, F32, 1, 61, decay=0.5)
    c[name][at, 1] = poison
    with np.errstate(all="ignore"):
        y, A, new, newA = scan_oracle(c, [0, rows], None, None)
    yd, sd = run_scan(c, [0, rows], None, None, F32, xt, True, pads)
    k = scan_k(shape, rows)
    assert np.all(np.isfinite(y[:at])) and (name == "dt" and poison < 0) == (np.isfinite(y).all() and np.isfinite(new).all())
    for got, want, size in ((host(yd), y, A), (host(sd), new, newA)):
        fine = np.isfinite(want)
        assert not np.isfinite(got[~fine]).any()
        size = np.where(fine, size, 0)
        assert np.all(np.abs(got[fine] - want[fine]) <= (k * U * size + half_step(F32, np.where(fine, want, 0)))[fine])


def test_scan_prompt_without_state():
    shape, cuts, rows = (4, 64, 128, 1), [0, 70, 200], 200
    for xt in (F16, F32):
        c = scan_case(rows, shape, xt, F32, F32, 2, 29)
        c["state"][:] = 0
        y, A, _, _ = scan_oracle(c, cuts, None, None)
        yd = torch.full((rows, 256), MARK, dtype=F32, device=DEV)
        x = dev(c["x"])
        n = F.scan_workspace_bytes(4, 64, 128, 1, 2, rows, xt == F16)
        F.scan_prompt(x, dev(c["dt"]), dev(c["B"]), dev(c["C"]), dev(c["dt_bias"]), dev(c["A_log"]), dev(c["D"]), None, yd,
                      ints(cuts), torch.empty(n, dtype=torch.uint8, device=DEV), headdim=64, groups=1)
        check("y", host(yd), y, scan_k(shape, rows) * U * A + half_step(F32, y))


@pytest.mark.parametrize("shape", SHAPES + [(64, 64, 128, 1)])
@pytest.mark.parametrize("xt,yt,st,dtt,D,pads", [
    (F16, F16, F32, F16, True, (8, 0, 8, 16)), (F32, F32, F16, F32, False, (1, 3, 1, 2)),
    (F16, F32, F32, F32, True, (1, 0, 3, 5))])
@pytest.mark.parametrize("slot,slots,fresh", [(None, 7, None), ([3, -1, 0, 3, 5, 9, 8], 9, [0, 0, 1, 0, 0, 0, 1])])
def test_scan_token(shape, xt, yt, st, dtt, D, pads, slot, slots, fresh):
    c = scan_case(7, shape, xt, dtt, st, slots, 31)
    got = run_scan(c, None, slot, fresh, yt, xt, D, pads)
    check_scan(c, got, scan_oracle(c, None, slot, fresh, D), shape, yt, 0)


def test_scan_token_many_sequences():
    """Enough sequences for the blocks that take several passes."""
    shape = (8, 64, 128, 1)
    for n in (64, 400):
        c = scan_case(n, shape, F16, F32, F32, n, 32)
        got = run_scan(c, None, None, None, F16, F16)
        check_scan(c, got, scan_oracle(c, None, None, None), shape, F16, 0)


def test_status_bits():
    shape = (2, 64, 16, 1)
    c = scan_case(20, shape, F32, F32, F32, 3, 33)
    w = np.zeros((6, 4), np.float16)

    def bits(cuts, slot):
        out = []
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        run_scan(c, cuts, slot, None, F32, F32, status=status)
        out.append(int(status))
        status.zero_()
        x = torch.zeros(20, 6, device=DEV)
        y = torch.zeros_like(x)
        if cuts is None:
            F.conv_token(x, dev(w), None, torch.zeros(3, 3, 6, device=DEV), y, ints(slot), status=status)
        else:
            F.conv_prompt(x, dev(w), None, torch.zeros(3, 3, 6, device=DEV), y, ints(cuts), ints(slot), status=status)
        out.append(int(status))
        return out
    assert bits([0, 5, 10, 20], [0, 1, 2]) == [0, 0]
    assert bits([0, 5, 10, 20], [0, -1, 2]) == [0, 0]        # -1 is a padded batch's own
    assert bits([0, 5, 10, 20], [0, 3, 2]) == [1, 1]
    assert bits([0, 5, 10, 20], [0, -2, 2]) == [1, 1]
    assert bits([0, 5, 10, 20], [2, 1, 2]) == [2, 2]
    assert bits([0, 5, 21, 21], [0, 1, 2]) == [4, 4]
    assert bits(None, list(range(3)) + [-1] * 16 + [1]) == [2, 2]


def test_broken_starts_stay_in_bounds():
    """Starts that fall, or lie outside the rows: the call ends, says so, and touches
    nothing outside its buffers (guard rows and slots keep their bits)."""
    shape = (2, 64, 128, 1)
    for xt in (F16, F32):
        for cuts in ([0, 50, 20, 70], [-5, 10, 70, 90], [90, 95, 99, 200], [60, 40, 20, 0], [2 ** 31 - 1, -2 ** 31, 0, 5]):
            c = scan_case(70, shape, xt, F32, F32, 5, 34)
            pool = torch.full((7,) + c["state"].shape[1:], MARK, device=DEV)
            out = torch.full((74, 128), MARK, device=DEV)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            x, ws = dev(c["x"]), F.scan_workspace(dev(c["x"]), pool, 3)
            F.scan_prompt(x, dev(c["dt"]), dev(c["B"]), dev(c["C"]), dev(c["dt_bias"]), dev(c["A_log"]), None, pool[1:6],
                          out[2:72], ints(cuts), ws, status=status)
            assert int(status) == 4
            assert bool((out[:2] == MARK).all()) and bool((out[72:] == MARK).all())
            assert bool((pool[0] == MARK).all()) and bool((pool[4:] == MARK).all())
            status.zero_()
            cst = torch.full((7, 3, 128), MARK, device=DEV)
            out.fill_(MARK)
            F.conv_prompt(x, torch.ones(128, 4, dtype=F16, device=DEV), None, cst[1:6], out[2:72], ints(cuts), status=status)
            assert bool((out[:2] == MARK).all()) and bool((out[72:] == MARK).all())
            assert bool((cst[0] == MARK).all()) and bool((cst[4:] == MARK).all())


# ------------------------------------------------------------------ norm

def norm_tol(y, cols, ot):
    # the mean square is a sum of cols / groups positive terms (each rounded, summed as a
    # tree of at most 64 adds per thread and 8 levels), its root and the three products
    return (8 + 72 / 2 + 16) * U * np.abs(y) + half_step(ot, y)


@pytest.mark.parametrize("rows,cols,groups", [
    (1, 1, 1), (3, 7, 1), (5, 256, 1), (2, 512, 4), (4, 1000, 1), (3, 1024, 1), (2, 1032, 1), (2, 2048, 1), (3, 4096, 1),
    (2, 4096, 8), (2, 8192, 1), (1, 9000, 1), (1, 16384, 1), (2, 999, 3), (300, 520, 1)])
@pytest.mark.parametrize("yt,zt,ot,pads", [(F32, F32, F16, (0, 0)), (F16, F16, F16, (8, 16)), (F16, F32, F32, (1, 3)),
                                           (F32, None, F16, (4, 0))])
def test_gated_norm(rows, cols, groups, yt, zt, ot, pads):
    rng = np.random.default_rng(41)
    y = rng.normal(size=(rows, cols)).astype(np.float16 if yt == F16 else np.float32)
    z = None if zt is None else rng.normal(size=(rows, cols), scale=3).astype(np.float16 if zt == F16 else np.float32)
    w = rng.normal(size=cols, loc=1.0, scale=0.1).astype(np.float16)
    want = PO.gated_norm(y, z, w, groups)
    out = torch.full((rows, cols), MARK, dtype=ot, device=DEV)
    F.gated_norm(wide(y, yt, pads[0]), None if z is None else wide(z, zt, pads[1]), dev(w), out, groups)
    check("out", host(out), want, norm_tol(want, cols // groups, ot))


@pytest.mark.parametrize("rows,cols,groups", [(1500, 520, 1), (700, 2048, 2), (1300, 1024, 1)])
def test_gated_norm_many_rows(rows, cols, groups):
    """Enough parts for a warp each."""
    rng = np.random.default_rng(43)
    y, z = rng.normal(size=(rows, cols)).astype(np.float32), rng.normal(size=(rows, cols)).astype(np.float16)
    w = rng.normal(size=cols, loc=1.0, scale=0.1).astype(np.float16)
    want = PO.gated_norm(y, z, w, groups)
    out = torch.full((rows, cols), MARK, dtype=F16, device=DEV)
    F.gated_norm(dev(y), dev(z), dev(w), out, groups)
    check("out", host(out), want, norm_tol(want, cols // groups, F16))


def test_gated_norm_in_place_and_extremes():
    rng = np.random.default_rng(42)
    for cols in (512, 4096, 9000):
        y, z = rng.normal(size=(4, cols)).astype(np.float32), rng.normal(size=(4, cols)).astype(np.float32)
        y[1] = 0.0                                  # rsqrt(eps), no division by zero
        y[2] *= 1e15                                # squares near the top of fp32
        z[3] = -100.0                               # gates that are 0 in fp32
        w = np.ones(cols, np.float16)
        want = PO.gated_norm(y, z, w)
        yd = dev(y)
        F.gated_norm(yd, dev(z), dev(w), yd)
        tol = norm_tol(want, cols, F32) + 1e-30
        assert np.all(np.abs(host(yd) - want) <= tol)


# ------------------------------------------------------------------ dense

def dense_case(n, rows, cols, seed, bias, rt):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n, cols)).astype(np.float16)
    w = (rng.normal(size=(rows, cols)) / np.sqrt(cols)).astype(np.float16)
    b = rng.normal(size=rows).astype(np.float16) if bias else None
    r = None if rt is None else rng.normal(size=(n, rows)).astype(np.float16 if rt == F16 else np.float32)
    return x, w, b, r


def dense_tol(yt, y, A, cols, act):
    err = (2 * (cols // 16 + 16) + 4) * U * A
    return (1.1 * err + 8 * U * np.abs(y) if act else err + 2 * U * np.abs(y)) + half_step(yt, y)


@pytest.mark.parametrize("n", [1, 2, 7, 16, 17, 33, 64, 100, 200, 257, 520])
@pytest.mark.parametrize("rows,cols,pad", [(1064, 256, 0), (256, 512, 8), (130, 72, 0), (17, 8, 0), (65, 129, 3), (256, 264, 1)])
@pytest.mark.parametrize("yt,rt,bias,act", [(F32, None, False, False), (F16, F32, True, True), (F32, F16, True, False)])
def test_dense_forward(n, rows, cols, pad, yt, rt, bias, act):
    x, w, b, r = dense_case(n, rows, cols, 51, bias, rt)
    want, A = PO.dense(x, w, b, r, act)
    y = torch.full((n, rows), MARK, dtype=yt, device=DEV)
    F.dense_forward(dev(w), wide(x, F16, pad), y, None if b is None else dev(b), None if r is None else wide(r, rt, 5), act)
    check("y", host(y), want, dense_tol(yt, want, A, cols, act))


@pytest.mark.parametrize("n,rows,cols", [(1, 8512, 2048), (16, 8512, 2048), (3, 2048, 4096), (300, 2048, 4096), (64, 8512, 2048)])
def test_dense_forward_layer_shapes(n, rows, cols):
    x, w, _, r = dense_case(n, rows, cols, 52, False, F32)
    want, A = PO.dense(x, w, None, r, False)
    y = dev(r)
    F.dense_forward(dev(w), dev(x), y, residual=y)                  # onto the residual itself
    check("y", host(y), want, dense_tol(F32, want, A, cols, False))
    # no bias either: of K terms of spread s added one by one, the partial sums are of size
    # sqrt(j) s, each rounded by U / sqrt(3) of that, in all sqrt(K / 6) U of the sum's own
    # size; sums that lean to one side (256 chained adds that round towards zero come to
    # 170 U) break sqrt(K) U = 64 U
    plain = x.astype(np.float64) @ w.astype(np.float64).T
    assert np.linalg.norm(host(y) - want) <= cols ** 0.5 * U * np.linalg.norm(plain) + U * np.linalg.norm(want)


def test_dense_forward_leaves_the_rest_alone():
    x, w, _, _ = dense_case(37, 200, 64, 53, False, None)
    out = torch.full((40, 210), MARK, device=DEV)
    F.dense_forward(dev(w), dev(x), out[1:38, 4:204])
    want, A = PO.dense(x, w, None, None, False)
    check("y", host(out[1:38, 4:204]), want, dense_tol(F32, want, A, 64, False))
    out[1:38, 4:204] = MARK
    assert bool((out == MARK).all())


# ------------------------------------------------------------------ together

def layer_parts(d, lw, z, cuts, slot, conv, ssm, act=F32):
    """conv, scan and gated norm on in_proj's fp32 rows z, as a layer runs them."""
    n, E, Cd, N, H = z.shape[0], d.d_inner, d.conv_dim, d.d_state, d.nheads
    xc = torch.empty(n, Cd, dtype=act, device=DEV)
    y = torch.empty(n, E, dtype=act, device=DEV)
    xo = torch.empty(n, E, dtype=F16, device=DEV)
    par = (dev(lw.dt_bias), dev(lw.A_log), dev(lw.D))
    xbc, dt = z[:, E:E + Cd], z[:, E + Cd:]
    parts = (xc[:, :E], dt, xc[:, E:E + N], xc[:, E + N:]) + par + (ssm, y)
    if cuts is None:
        F.conv_token(xbc, dev(lw.conv_w), dev(lw.conv_b), conv, xc, slot)
        F.scan_token(*parts, slot=slot)
    else:
        F.conv_prompt(xbc, dev(lw.conv_w), dev(lw.conv_b), conv, xc, cuts, slot)
        F.scan_prompt(*parts, cuts, F.scan_workspace(xc, ssm, len(cuts) - 1), slot=slot)
    F.gated_norm(y, z[:, :E], dev(lw.gnorm_w), xo)
    return xc, y, xo


def test_a_layer_from_its_parts():
    """The 1.3B layer: pre-norm and scaffold projection of packed prompts, conv, scan, gated
    norm, out_proj, then two token steps from the states left, against the layer oracle
    run on each prompt alone."""
    d = S.LAYER_1P3B
    rng = np.random.default_rng(61)
    lw = S.gen_layer(rng, d)
    lens, slots = [70, 5, 129], [2, 0, 3]
    cuts = [0, 70, 75, 204]
    res = [S.gen_layer_inputs(rng, d, n + 2).transpose(1, 0, 2).copy() for n in lens]
    pin, pout = F.DeviceProj.from_host(lw.inp), F.DeviceProj.from_host(lw.out)
    conv = torch.zeros(4, d.d_conv - 1, d.conv_dim, device=DEV)
    ssm = torch.zeros(4, d.nheads, d.headdim, d.d_state, device=DEV)

    def step(rows, cuts_, res_rows, oracle):
        x = torch.empty(rows, d.d_model, dtype=F16, device=DEV)
        F.gated_norm(dev(res_rows), None, dev(lw.prenorm_w), x)
        x_in = np.concatenate([t.x_in.reshape(-1, d.d_model) for t in oracle])
        np.testing.assert_allclose(host(x), np.float64(x_in), rtol=2.0 ** -10, atol=2.0 ** -24)     # one fp16 step
        x = dev(x_in)             # the projection's own codes depend on the last bit of x
        z = torch.empty(rows, d.in_rows, dtype=F32, device=DEV)
        F.proj_forward(pin, d.rank, x, z, F.proj_workspace(d.in_rows, d.d_model, d.rank, rows))
        xc, y, xo = layer_parts(d, lw, z, cuts_, ints(slots), conv, ssm)
        ref = lambda k, n: np.concatenate([np.float64(getattr(t, k)).reshape(-1, n) for t in oracle])  # noqa: E731
        near = lambda g, w: np.linalg.norm(host(g) - w) <= 2e-6 * np.linalg.norm(w)  # noqa: E731
        assert near(z, ref("zxbcdt", d.in_rows)) and near(xc, ref("xc", d.conv_dim))
        zr = ref("zxbcdt", d.in_rows)[:, :d.d_inner]
        assert near(y * torch.nn.functional.silu(z[:, :d.d_inner]), ref("g", d.d_inner)) and np.isfinite(zr).all()
        np.testing.assert_allclose(host(xo), ref("x_out", d.d_inner), rtol=2.0 ** -10, atol=2.0 ** -18)
        out = torch.empty(rows, d.d_model, dtype=F32, device=DEV)
        F.proj_forward(pout, d.rank, xo, out, F.proj_workspace(d.d_model, d.d_inner, d.rank, rows))
        assert near(out, np.float64(O.project(xo.cpu().numpy(), lw.out).y))

    st = [O.State(np.zeros((1, 3, d.conv_dim), np.float32), np.zeros((1, d.nheads, d.headdim, d.d_state), np.float32))
          for _ in lens]
    traces = [O.layer_prefill(r[:, :n], lw, s, d) for r, n, s in zip(res, lens, st)]
    step(204, ints(cuts), np.concatenate([r[0, :n] for r, n in zip(res, lens)]), traces)
    for k in range(2):
        st = [O.State(t.conv, t.ssm) for t in traces]
        traces = [O.layer_step(r[:, n + k], lw, s, d) for r, n, s in zip(res, lens, st)]
        step(3, None, np.concatenate([r[:, n + k] for r, n in zip(res, lens)]), traces)
    for i, t in zip(slots, traces):
        assert np.linalg.norm(host(ssm[i]) - t.ssm[0]) <= 2e-6 * np.linalg.norm(t.ssm)
        assert np.linalg.norm(host(conv[i]) - t.conv[0]) <= 2e-6 * np.linalg.norm(t.conv)
    assert not bool(ssm[1].any()) and not bool(conv[1].any())


def dense_layer(d, w_in, w_out, lw, res, cuts, slot, conv, ssm, bufs):
    """A layer with dense projections, fp16 between its parts; everything preallocated."""
    x, z, xc, y, xo, ws = bufs
    E, Cd, N = d.d_inner, d.conv_dim, d.d_state
    F.gated_norm(res, None, lw["prenorm_w"], x)
    F.dense_forward(w_in, x, z)
    xbc, dt = z[:, E:E + Cd], z[:, E + Cd:]
    args = (xc[:, :E], dt, xc[:, E:E + N], xc[:, E + N:], lw["dt_bias"], lw["A_log"], lw["D"], ssm, y)
    if cuts is None:
        F.conv_token(xbc, lw["conv_w"], lw["conv_b"], conv, xc, slot)
        F.scan_token(*args, slot=slot)
    else:
        F.conv_prompt(xbc, lw["conv_w"], lw["conv_b"], conv, xc, cuts, slot)
        F.scan_prompt(*args, cuts, ws, slot=slot)
    F.gated_norm(y, z[:, :E], lw["gnorm_w"], xo)
    F.dense_forward(w_out, xo, res, residual=res)


def dense_setup(rows, n_slots, seed=71):
    d = S.LAYER_SMALL
    rng = np.random.default_rng(seed)
    lw = S.gen_layer(rng, d)
    par = {k: dev(getattr(lw, k)) for k in ("prenorm_w", "conv_w", "conv_b", "dt_bias", "A_log", "D", "gnorm_w")}
    w_in = dev((rng.normal(size=(d.in_rows, d.d_model)) / 16).astype(np.float16))
    w_out = dev((rng.normal(size=(d.d_model, d.d_inner)) / 22).astype(np.float16))
    conv = torch.zeros(n_slots, 3, d.conv_dim, device=DEV)
    ssm = torch.zeros(n_slots, d.nheads, d.headdim, d.d_state, device=DEV)
    bufs = [torch.empty(rows, n, dtype=t, device=DEV) for n, t in
            ((d.d_model, F16), (d.in_rows, F32), (d.conv_dim, F16), (d.d_inner, F16), (d.d_inner, F16))]
    bufs.append(torch.empty(F.scan_workspace_bytes(d.nheads, d.headdim, d.d_state, 1, rows, rows, True), dtype=torch.uint8,
                            device=DEV))
    return d, par, w_in, w_out, conv, ssm, bufs


def test_prompts_in_one_pack_equal_prompts_alone():
    """Prompts packed together leave the bits that each leaves alone: nothing of a prompt
    depends on its neighbours or on where it lies."""
    lens = [1, 64, 130, 3, 33]
    cuts = [0] + list(np.cumsum(lens))
    d, par, w_in, w_out, conv, ssm, bufs = dense_setup(cuts[-1], 5)
    res = torch.randn(cuts[-1], d.d_model, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    packed = res.clone()
    dense_layer(d, w_in, w_out, par, packed, ints(cuts), None, conv, ssm, bufs)
    for i, n in enumerate(lens):
        _, _, _, _, c1, s1, b1 = dense_setup(n, 1)
        alone = res[cuts[i]:cuts[i + 1]].clone()
        dense_layer(d, w_in, w_out, par, alone, ints([0, n]), None, c1, s1, b1)
        # the dense tile and the chunk a row falls into may differ: fp32 sums in another order
        assert torch.allclose(alone, packed[cuts[i]:cuts[i + 1]], rtol=0, atol=2e-3 * float(alone.abs().max()))
        assert torch.allclose(s1[0], ssm[i], rtol=0, atol=2e-3 * float(s1.abs().max()))


def test_captured_and_replayed_on_another_stream():
    """A prompt call and a token call in one captured graph, on a side stream, replayed with
    new inputs, give the bits of the eager calls; two graphs with workspaces of their own
    replay side by side."""
    cuts, n = [0, 40, 41, 200], 200

    def capture(seed):
        d, par, w_in, w_out, conv, ssm, bufs = dense_setup(n, 3, seed)
        tb = dense_setup(3, 3, seed)[6]
        res = torch.zeros(n, d.d_model, device=DEV)
        tok = torch.zeros(3, d.d_model, device=DEV)
        start, slot = ints(cuts), ints([2, 0, 1])

        def both():
            dense_layer(d, w_in, w_out, par, res, start, slot, conv, ssm, bufs)
            dense_layer(d, w_in, w_out, par, tok, None, slot, conv, ssm, tb)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both()
        return g, res, tok, conv, ssm, both, side
    graphs = [capture(81), capture(82)]
    gen = torch.Generator(DEV).manual_seed(2)
    wanted = []
    for g, res, tok, conv, ssm, both, side in graphs:
        r0, t0 = (torch.randn(v.shape, device=DEV, generator=gen) for v in (res, tok))
        out = []
        for run in (both, None):
            res.copy_(r0)
            tok.copy_(t0)
            conv.zero_()
            ssm.zero_()
            if run:
                run()
                out = [v.clone() for v in (res, tok, conv, ssm)]
        wanted.append(out)
    torch.cuda.synchronize()
    for g, *_, side in graphs:
        with torch.cuda.stream(side):
            g.replay()
    torch.cuda.synchronize()
    for (g, res, tok, conv, ssm, both, side), out in zip(graphs, wanted):
        assert all(torch.equal(a, b) for a, b in zip((res, tok, conv, ssm), out))


def test_results_do_not_change_between_calls():
    shape, rows, cuts = (4, 64, 128, 1), 900, [0, 500, 900]
    for xt in (F16, F32):
        c = scan_case(rows, shape, xt, F32, F32, 2, 91)
        first = run_scan(c, cuts, None, None, F32, xt)
        for _ in range(5):
            again = run_scan(c, cuts, None, None, F32, xt)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_tensors_of_two_devices_are_refused():
    if torch.cuda.device_count() < 2:
        y = torch.zeros(1, 8, device=DEV)
        with pytest.raises(ValueError):
            F.gated_norm(y, None, torch.zeros(8, dtype=F16), y)
        return
    y = torch.randn(2, 64, device="cuda:1")
    w = torch.ones(64, dtype=F16, device="cuda:1")
    out = torch.empty_like(y)
    F.gated_norm(y, None, w, out)            # not the current device
    assert torch.allclose(out, y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-5), atol=1e-5)
    with pytest.raises(ValueError):
        F.gated_norm(y, None, w.to("cuda:0"), out)


def test_rows_and_slots_beyond_32_bits():
    """Rows 16 MiB apart and slots far into their pool give the bits of compact ones."""
    n, S, slots = 300, 2 ** 23 + 8, 65700
    big = torch.empty(n * S, dtype=F16, device=DEV)              # 2.5e9 values
    far = lambda at, width: big.as_strided((n, width), (S, 1), at)  # noqa: E731
    rng = np.random.default_rng(95)
    c = scan_case(n, (4, 64, 128, 1), F16, F16, F32, 1, 95)
    near = {k: dev(c[k]) for k in ("x", "dt", "B", "C")}
    wide_ = {}
    for i, (k, v) in enumerate(near.items()):
        wide_[k] = far(512 * i, v.shape[1])
        wide_[k].copy_(v)
    pool = torch.empty(slots, 4, 64, 128, device=DEV)            # 2.15e9 values
    par = [dev(c[k]) for k in ("dt_bias", "A_log", "D")]
    start = ints([0, n])

    def run(rows, y, state, slot):
        state[slot].copy_(dev(c["state"])[0])
        ws = F.scan_workspace(rows["x"], state, 1)
        F.scan_prompt(*[rows[k] for k in ("x", "dt", "B", "C")], *par, state, y, start, ws, ints([slot]))
        one = [rows[k][-1:] for k in ("x", "dt", "B", "C")]
        F.scan_token(*one, *par, state, y[:1], ints([slot]))
        return y.clone(), state[slot].clone()
    small = run(near, torch.zeros(n, 256, dtype=F16, device=DEV), torch.zeros(1, 4, 64, 128, device=DEV), 0)
    y = far(2048, 256)
    large = run(wide_, y, pool, slots - 50)
    assert torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    # fp32 rows take another kernel
    f = {k: v.float() for k, v in near.items()}
    small = run(f, torch.zeros(n, 256, device=DEV), torch.zeros(1, 4, 64, 128, device=DEV), 0)
    large = run(f, torch.zeros(n, 256, device=DEV), pool, slots - 50)
    assert torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    # conv
    m = 2 ** 31 // 768 + 100
    cpool = pool.view(-1)[:m * 768].view(m, 3, 256)
    w, st = dev(rng.normal(size=(256, 4)).astype(np.float16)), dev(rng.normal(size=(1, 3, 256)).astype(np.float32))
    got = []
    for x, yy, state, slot in ((near["x"], torch.zeros(n, 256, dtype=F16, device=DEV), st.clone(), 0), (wide_["x"], y, cpool, m - 1)):
        state[slot].copy_(st[0])
        F.conv_prompt(x, w, None, state, yy, start, ints([slot]))
        F.conv_token(x[-1:], w, None, state, yy[:1], ints([slot]))
        got.append((yy.clone(), state[slot].clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    # norm, dense (few rows and many)
    wn, wd = dev(np.ones(256, np.float16)), dev(rng.normal(size=(256, 256)).astype(np.float16))
    out = torch.zeros(n, 256, dtype=F16, device=DEV)
    F.gated_norm(near["x"], None, wn, out)
    F.gated_norm(wide_["x"], None, wn, y)
    assert torch.equal(out, y)
    for k in (n, 20):
        F.dense_forward(wd, near["x"][-k:], out[-k:])
        F.dense_forward(wd, wide_["x"][-k:], y[-k:])
        assert torch.equal(out, y)


def test_no_number_stays_in_its_row():
    """Projections and norms of a batch: rows do not reach each other."""
    for n in (5, 70):
        x, w, _, _ = dense_case(n, 200, 512, 96, False, None)
        x[3, 7] = np.nan
        y, out = torch.zeros(n, 200, device=DEV), torch.zeros(n, 512, device=DEV)
        F.dense_forward(dev(w), dev(x), y)
        F.gated_norm(dev(x), None, dev(np.ones(512, np.float16)), out)
        for v in (y, out):
            assert torch.isnan(v[3]).all() and torch.isfinite(v[:3]).all() and torch.isfinite(v[4:]).all()


def test_calls_of_two_host_threads():
    """Calls of different sizes at once, from two threads on streams of their own."""
    import ctypes as C
    import threading
    L = F.lib()
    jobs, errors = [], []
    for i, (n, rows, cols) in enumerate([(70, 512, 256), (300, 2048, 1024), (20, 512, 4096), (20, 8512, 256)]):
        x, w, _, _ = dense_case(n, rows, cols, 97 + i, False, None)
        jobs.append((dev(w), dev(x), torch.zeros(n, rows, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(mine):
        for _ in range(50):
            for w, x, y, s in mine:      # the C call itself: it runs without the interpreter's lock
                rc = L.dfssm_dense_forward(w.shape[0], w.shape[1], x.shape[0], w.data_ptr(), None, 0,
                                           C.byref(F.CRows(x.data_ptr(), x.shape[1], F.DTYPE_F16)), None,
                                           C.byref(F.CRows(y.data_ptr(), y.shape[1], F.DTYPE_F32)), None, s.cuda_stream)
                if rc != F.OK:
                    errors.append((rc, F.last_error()))
    threads = [threading.Thread(target=work, args=(jobs[i::2],)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for w, x, y, _ in jobs:
        alone = torch.zeros_like(y)
        F.dense_forward(w, x, alone)
        assert torch.equal(alone, y)


FIRST_IN_A_CAPTURE = """
import torch
from bit_scaffold_quantized_b200 import dfssm as F
d = dict(device="cuda", dtype=torch.float16)
x, B, C, dt = torch.randn(300, 128, **d), torch.randn(300, 64, **d), torch.randn(300, 64, **d), torch.randn(300, 2, **d)
w, wn, wd = torch.randn(128, 4, **d), torch.ones(128, **d), torch.randn(128, 128, **d)
par = [torch.zeros(2, device="cuda") for _ in range(3)]
start = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
conv, ssm = torch.zeros(2, 3, 128, device="cuda"), torch.zeros(2, 2, 64, 64, device="cuda")
y = [torch.zeros(300, 128, **d) for _ in range(6)]
ws = F.scan_workspace(x, ssm, 2)

def run():
    F.conv_prompt(x, w, None, conv, y[0], start)
    F.scan_prompt(y[0], dt, B, C, *par, ssm, y[1], start, ws)
    F.gated_norm(y[1], x, wn, y[2])
    F.dense_forward(wd, y[2], y[3])
    F.conv_token(y[3][:2], w, None, conv, y[4][:2])
    F.scan_token(y[4][:2], dt[:2], B[:2], C[:2], *par, ssm, y[5][:2])
    F.dense_forward(wd, y[5][:2], y[4][2:4])

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (*y, conv, ssm)]
for v in (*y, conv, ssm):
    v.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (*y, conv, ssm)))
print("the same bits")
"""


def test_first_calls_of_a_process_in_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the same bits" in r.stdout, r.stdout + r.stderr

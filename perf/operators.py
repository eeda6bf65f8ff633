"""What is measured of the operators that a Mamba-2 layer is put together from when its
prompts are packed one behind the other and its projections may be dense: the causal
conv and the selective scan (for packed prompts and for single tokens), the gated
RMSNorm and the dense projection with its epilogue.

With `own` false, `run` computes them from elementary torch operations in 32 bits (the
running sums of the decay exponents, whose differences matter, in 64); with `own` true it
calls the library's entry points through bit_scaffold_quantized_b200.dfssm.

Sizes are those of this repository's layers (d_model 256: 8 heads of 64, d_state 16;
d_model 2048: 64 heads of 64, d_state 128, in_proj 8512 rows) and general ones."""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
CHUNK = 64
TYPES = {"f16": torch.float16, "f32": torch.float32}
SIZE = {"f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _conv(form, tokens, seqs, channels, x, y, pad=0, fresh=0.5, skip=False, width=4, silu=True, bias=True):
    return dict(op="conv", form=form, tokens=tokens, seqs=seqs, channels=channels, x=x, y=y, pad=pad, fresh=fresh,
                skip=skip, width=width, silu=silu, bias=bias)


def _scan(form, tokens, seqs, heads, headdim, d_state, groups, x, y, dt="f32", state="f32", fresh=0.5, skip=False,
          D=True):
    return dict(op="scan", form=form, tokens=tokens, seqs=seqs, heads=heads, headdim=headdim, d_state=d_state,
                groups=groups, x=x, y=y, dt=dt, state=state, fresh=fresh, skip=skip, D=D)


def _norm(rows, cols, groups, y, z, out, gate=True):
    return dict(op="norm", rows=rows, cols=cols, groups=groups, y=y, z=z, out=out, gate=gate)


def _dense(batch, rows, cols, y, bias=False, silu=False, residual="none"):
    return dict(op="dense", batch=batch, rows=rows, cols=cols, y=y, bias=bias, silu=silu, residual=residual)


def listed():
    return [
        # a server admits 24 prompts together, a part of them further pieces of prompts begun before: the
        # conv reads the fp32 in_proj rows in place and leaves 16-bit rows for the scan
        dict(_conv("prompt", 6007, 24, 4352, "f32", "f16", pad=4160), name="conv_prompts_packed"),
        # one decode step of 64 users
        dict(_conv("token", 64, 64, 4352, "f32", "f16", pad=4160, fresh=0.0), name="conv_token_b64"),
        # one long document through one layer
        dict(_scan("prompt", 8192, 1, 64, 64, 128, 1, "f16", "f16", fresh=1.0), name="scan_prompt_long"),
        # the 24 packed prompts
        dict(_scan("prompt", 6007, 24, 64, 64, 128, 1, "f16", "f16"), name="scan_prompts_packed"),
        # 32 bits throughout, for callers that hold the layer to the prompt pass of the library
        dict(_scan("prompt", 1000, 3, 64, 64, 128, 1, "f32", "f32"), name="scan_prompts_f32"),
        # the small layer over two short prompts: latency
        dict(_scan("prompt", 77, 2, 8, 64, 16, 1, "f32", "f32"), name="scan_prompt_small_f32"),
        # one user's next token: latency
        dict(_scan("token", 1, 1, 64, 64, 128, 1, "f16", "f16", fresh=0.0), name="scan_token_b1"),
        # one decode step of up to 128 users in a graph that is padded with empty rows, half-size states
        dict(_scan("token", 128, 128, 64, 64, 128, 1, "f16", "f32", state="f16", fresh=0.0, skip=True),
             name="scan_token_b128_state16"),
        # the gate and the norm before out_proj: one decode step of 64 users, and a long prompt
        dict(_norm(64, 4096, 1, "f32", "f32", "f16"), name="norm_b64"),
        dict(_norm(8192, 4096, 1, "f16", "f16", "f16"), name="norm_prompt_8192"),
        # a dense in_proj for one user's next token: reading the weights is all of the work
        dict(_dense(1, 8512, 2048, "f32"), name="dense_in_b1"),
        # a dense out_proj of a 4096-token prompt, added to the fp32 residual stream
        dict(_dense(4096, 2048, 4096, "f32", residual="f32"), name="dense_out_prompt_4096"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "norm", "dense", "dense"])
    typ = lambda: rng.choice(["f16", "f32"])  # noqa: E731
    form = rng.choice(["prompt", "prompt", "token"])
    if op == "conv":
        channels = _log(rng, 32, 5000)
        most = 16384 if form == "prompt" else 512
        tokens = _log(rng, 1, most)
        seqs = min(tokens, _log(rng, 1, 64)) if form == "prompt" else tokens
        return _conv(form, tokens, seqs, channels, typ(), typ(), pad=rng.choice([0, 0, 8, 33, 4160]),
                     fresh=rng.choice([0.0, 0.5, 1.0]), skip=rng.random() < 0.3, width=rng.choice([2, 3, 4, 4, 4]),
                     silu=rng.random() < 0.8, bias=rng.random() < 0.8)
    if op == "scan":
        heads, groups = rng.choice([(8, 1), (64, 1), (16, 2), (24, 8), (5, 1), (1, 1), (80, 1), (32, 4)])
        headdim = rng.choice([16, 32, 64, 64, 64, 96, 128])
        d_state = rng.choice([4, 16, 20, 64, 64, 128, 128, 128, 200, 256])
        if form == "prompt":
            tokens = _log(rng, 1, min(8192, 8192 * 64 * 64 * 128 // (heads * headdim * d_state)))
            seqs = min(tokens, _log(rng, 1, 48))
        else:
            tokens = seqs = _log(rng, 1, min(256, 256 * 64 * 64 * 64 // (heads * headdim * d_state)))
        x = rng.choice(["f16", "f16", "f32"])
        return _scan(form, tokens, seqs, heads, headdim, d_state, groups, x, rng.choice([x, x, "f32"]), dt=typ(),
                     state=rng.choice(["f32", "f32", "f16"]), fresh=rng.choice([0.0, 0.5, 1.0]),
                     skip=rng.random() < 0.3, D=rng.random() < 0.8)
    if op == "norm":
        groups = rng.choice([1, 1, 1, 2, 8])
        return _norm(_log(rng, 1, 8192), groups * _log(rng, 16, 4096 // groups), groups, typ(), typ(), typ(),
                     gate=rng.random() < 0.8)
    rows, cols = rng.choice([(8512, 2048), (2048, 4096), (1064, 256), (256, 512), (None, None)])
    if rows is None:
        rows, cols = _log(rng, 16, 8192), 8 * _log(rng, 4, 512)
    return _dense(_log(rng, 1, min(4096, 4096 * 4096 * 2048 // (rows * cols))), rows, cols, typ(),
                  bias=rng.random() < 0.5, silu=rng.random() < 0.3, residual=rng.choice(["none", "f16", "f32"]))


# ------------------------------------------------------------------ inputs

def _lengths(tokens, seqs, seed):
    """`seqs` lengths of uneven size that add up to `tokens`; now and then one is empty."""
    r = random.Random(seed)
    w = [0.0 if seqs > 2 and r.random() < 0.05 else r.lognormvariate(0.0, 1.0) for _ in range(seqs)]
    total = sum(w) or 1.0
    cuts, run = [0], 0.0
    for v in w[:-1]:
        run += v
        cuts.append(min(tokens, int(round(tokens * run / total))))
    cuts.append(tokens)
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _sequences(case, seed, g, st):
    """Where the sequences lie in the packed rows, which state slot each has, which of them begin anew."""
    n = case["seqs"]
    if case["form"] == "prompt":
        cuts = [0]
        for v in _lengths(case["tokens"], n, seed):
            cuts.append(cuts[-1] + v)
        st["start"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    else:
        st["start"] = None
    slots = n + 3
    slot = torch.randperm(slots, generator=g, device=DEV)[:n].to(torch.int32)
    if case["skip"] and n > 1:      # the last rows of a padded batch hold no sequence
        slot[n - max(1, n // 8):] = -1
    st["slot"], st["slots"] = slot, slots
    st["fresh"] = (torch.rand(n, generator=g, device=DEV) < case["fresh"]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    f32 = torch.float32

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=f32) * std + mean

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=DEV, dtype=f32) * (hi - lo) + lo

    st = {"case": case}
    op = case["op"]
    if op == "conv":
        _sequences(case, seed, g, st)
        C, W = case["channels"], case["width"]
        wide = normal(case["tokens"], C + case["pad"]).to(TYPES[case["x"]])
        st["x"] = wide[:, case["pad"]:] if case["pad"] else wide     # a view of the projection's wider rows
        st["w"] = uniform(-0.5, 0.5, C, W).half()
        st["b"] = uniform(-0.5, 0.5, C).half() if case["bias"] else None
        st["state"] = normal(st["slots"], W - 1, C)
        st["y"] = torch.zeros(case["tokens"], C, dtype=TYPES[case["y"]], device=DEV)
    elif op == "scan":
        _sequences(case, seed, g, st)
        H, P, N, G, T = case["heads"], case["headdim"], case["d_state"], case["groups"], case["tokens"]
        E, GN = H * P, case["groups"] * N
        xbc = normal(T, E + 2 * GN)
        xbc = (xbc * torch.sigmoid(xbc)).to(TYPES[case["x"]])          # what the conv leaves
        st["x"], st["B"], st["C"] = xbc[:, :E], xbc[:, E:E + GN], xbc[:, E + GN:]
        st["dt"] = normal(T, H, std=0.5).to(TYPES[case["dt"]])
        # step sizes around exp(U(ln 1e-3, ln 1e-1)) and decay rates in [1, 16], as such layers are initialised
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["A_log"] = torch.log(uniform(1.0, 16.0, H))
        st["D"] = normal(H, std=0.1, mean=1.0) if case["D"] else None
        st["state"] = normal(st["slots"], H, P, N, std=0.02).to(TYPES[case["state"]])
        st["y"] = torch.zeros(T, E, dtype=TYPES[case["y"]], device=DEV)
    elif op == "norm":
        R, C = case["rows"], case["cols"]
        st["in"] = normal(R, C).to(TYPES[case["y"]])
        st["z"] = normal(R, C).to(TYPES[case["z"]]) if case["gate"] else None
        st["w"] = normal(C, std=0.1, mean=1.0).half()
        st["y"] = torch.empty(R, C, dtype=TYPES[case["out"]], device=DEV)
    else:
        M, R, K = case["batch"], case["rows"], case["cols"]
        st["x"] = normal(M, K).half()
        st["w"] = normal(R, K, std=1.0 / math.sqrt(K)).half()
        st["b"] = normal(R, std=0.1).half() if case["bias"] else None
        st["r"] = normal(M, R).to(TYPES[case["residual"]]) if case["residual"] != "none" else None
        st["y"] = torch.empty(M, R, dtype=TYPES[case["y"]], device=DEV)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st, st["case"])
    return _PLAIN[op](st, st["case"])


def _own_conv(st, case):
    from bit_scaffold_quantized_b200 import dfssm
    call = dfssm.conv_prompt if case["form"] == "prompt" else dfssm.conv_token
    where = {"start": st["start"]} if case["form"] == "prompt" else {}
    call(st["x"], st["w"], st["b"], st["state"], st["y"], slot=st["slot"], fresh=st["fresh"], silu=case["silu"], **where)
    return st["y"], st["state"]


def _own_scan(st, case):
    from bit_scaffold_quantized_b200 import dfssm
    args = (st["x"], st["dt"], st["B"], st["C"], st["dt_bias"], st["A_log"], st["D"], st["state"], st["y"])
    if case["form"] == "token":
        dfssm.scan_token(*args, slot=st["slot"], fresh=st["fresh"])
        return st["y"], st["state"]
    if "ws" not in st:
        st["ws"] = dfssm.scan_workspace(st["x"], st["state"], case["seqs"], case["groups"])
    dfssm.scan_prompt(*args, st["start"], st["ws"], slot=st["slot"], fresh=st["fresh"])
    return st["y"], st["state"]


def _own_norm(st, case):
    from bit_scaffold_quantized_b200 import dfssm
    dfssm.gated_norm(st["in"], st["z"], st["w"], st["y"], groups=case["groups"])
    return st["y"]


def _own_dense(st, case):
    from bit_scaffold_quantized_b200 import dfssm
    dfssm.dense_forward(st["w"], st["x"], st["y"], bias=st["b"], residual=st["r"], silu=case["silu"])
    return st["y"]


_OWN = {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm, "dense": _own_dense}


# ------------------------------------------------------------------ plain forms

def _places(st):
    """For every packed row: its sequence, its place in it and whether it belongs to one that has a slot."""
    T = st["x"].shape[0]
    row = torch.arange(T, device=DEV)
    if st["start"] is None:
        seq, pos = row, torch.zeros_like(row)
    else:
        start = st["start"].long()
        seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
        pos = row - start[seq]
    return row, seq, pos, st["slot"][seq] >= 0


def _lens(st):
    return torch.ones_like(st["slot"]).long() if st["start"] is None else (st["start"][1:] - st["start"][:-1]).long()


def _plain_conv(st, case):
    C, W = case["channels"], case["width"]
    x, state = st["x"].float(), st["state"]
    row, seq, pos, live = _places(st)
    slot, begins = st["slot"].long(), st["fresh"].bool()
    old = torch.where(begins[:, None, None], 0.0, state[slot.clamp(min=0)])         # [seqs, W-1, C]
    ext = torch.cat([old.reshape(-1, C), x])
    first = old.shape[0] * (W - 1)
    back = torch.arange(W - 1, -1, -1, device=DEV)                                  # tap j looks back W-1-j rows
    at = torch.where(pos[:, None] >= back, first + row[:, None] - back,
                     seq[:, None] * (W - 1) + (W - 1) + pos[:, None] - back)
    v = (ext[at] * st["w"].float().t()).sum(1)
    if case["bias"]:
        v = v + st["b"].float()
    if case["silu"]:
        v = v * torch.sigmoid(v)
    st["y"].copy_(torch.where(live[:, None], v, st["y"].float()))
    n = _lens(st)
    begin = torch.arange(len(n), device=DEV) if st["start"] is None else st["start"][:-1].long()
    k = torch.arange(W - 1, device=DEV) + n[:, None] - (W - 1)                      # place in the sequence, < 0: old rows
    at = torch.where(k >= 0, first + begin[:, None] + k,
                     torch.arange(len(n), device=DEV)[:, None] * (W - 1) + (W - 1) + k)
    keep = (slot >= 0) & (n > 0)
    state[slot[keep]] = ext[at[keep]]
    return st["y"], state


def _steps(st):
    """Step sizes, and the exponents of the decay per step in 64 bits."""
    v = st["dt"].float() + st["dt_bias"]
    step = torch.where(v > 20.0, v, torch.log1p(torch.exp(v)))
    return step, step.double() * -torch.exp(st["A_log"].double())


def _plain_scan(st, case):
    H, P, N, G = case["heads"], case["headdim"], case["d_state"], case["groups"]
    T, R = case["tokens"], case["heads"] // case["groups"]
    x, Bm, Cm = st["x"].float().view(T, H, P), st["B"].float().view(T, G, N), st["C"].float().view(T, G, N)
    step, expo = _steps(st)
    state, slot = st["state"], st["slot"].long()
    row, seq, pos, live = _places(st)
    h0 = torch.where(st["fresh"].bool()[:, None, None, None], 0.0, state[slot.clamp(min=0)].float())
    if st["start"] is None:
        Bh, Ch = Bm.repeat_interleave(R, 1), Cm.repeat_interleave(R, 1)
        h = h0 * torch.exp(expo).float()[:, :, None, None] + (step[:, :, None] * x)[..., None] * Bh[:, :, None, :]
        y = (h * Ch[:, :, None, :]).sum(-1)
        keep = slot >= 0
        state[slot[keep]] = h[keep].to(state.dtype)
    else:
        # every sequence in chunks of its own; what the chunks hand on is summed over the chunks before them
        n = _lens(st)
        count = (n + CHUNK - 1) // CHUNK
        upto = torch.cumsum(count, 0)
        i = torch.arange(T // CHUNK + len(n), device=DEV)
        cseq = torch.searchsorted(upto, i, right=True).clamp(max=len(n) - 1)
        k = i - (upto - count)[cseq]
        tok = st["start"].long()[cseq][:, None] + k[:, None] * CHUNK + torch.arange(CHUNK, device=DEV)
        has = (tok < st["start"].long()[cseq + 1][:, None]) & (i < upto[-1])[:, None]
        tok = tok.clamp(max=T - 1)
        w = torch.where(has[..., None], step[tok], 0.0)                                     # [c, Q, H]
        cs = torch.cumsum(torch.where(has[..., None], expo[tok], 0.0), 1)                   # [c, Q, H], 64 bits
        xs, bs, ct = x[tok], Bm[tok], Cm[tok]
        csh = cs.transpose(1, 2)                                                             # [c, H, Q]
        ahead = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).triu(1)
        L = torch.exp((csh[..., :, None] - csh[..., None, :]).float().masked_fill(ahead, -math.inf))
        cb = torch.matmul(ct.permute(0, 2, 1, 3), bs.permute(0, 2, 3, 1))                    # [c, G, Q, Q]
        M = cb.repeat_interleave(R, 1) * L * w.transpose(1, 2)[:, :, None, :]
        yc = torch.matmul(M, xs.transpose(1, 2))                                             # [c, H, Q, P]
        total = cs[:, -1]                                                                    # [c, H]
        u = xs * (torch.exp(total[:, None] - cs).float() * w)[..., None]                     # [c, Q, H, P]
        S = torch.matmul(u.permute(0, 2, 3, 1), bs.repeat_interleave(R, 2).permute(0, 2, 1, 3))   # [c, H, P, N]
        run_ = torch.cumsum(total, 0)
        before = (run_ - total).t()                                                          # [H, c]
        part = (before[:, :, None] - run_.t()[:, None, :]).masked_fill(
            (cseq[:, None] != cseq[None, :]) | (i[:, None] <= i[None, :]), -math.inf)
        hin = torch.matmul(torch.exp(part).float(), S.transpose(0, 1).reshape(H, len(i), P * N)).view(H, len(i), P, N)
        begins = (upto - count).clamp(max=len(i) - 1)
        hin = hin.transpose(0, 1) + torch.exp(before.t() - before.t()[begins][cseq]).float()[..., None, None] * h0[cseq]
        inter = torch.matmul(ct.repeat_interleave(R, 2).permute(0, 2, 1, 3), hin.transpose(2, 3))
        yc = yc + inter * torch.exp(csh).float()[..., None]
        y = torch.zeros(T, H, P, device=DEV)
        y[tok[has]] = yc.transpose(1, 2)[has]
        keep = (slot >= 0) & (n > 0)
        last = (upto - 1).clamp(min=0)[keep]
        state[slot[keep]] = (torch.exp(total[last]).float()[..., None, None] * hin[last] + S[last]).to(state.dtype)
    if case["D"]:
        y = y + st["D"][:, None] * x
    st["y"].copy_(torch.where(live[:, None], y.reshape(T, H * P), st["y"].float()))
    return st["y"], state


def _plain_norm(st, case):
    v = st["in"].float()
    if case["gate"]:
        z = st["z"].float()
        v = v * (z * torch.sigmoid(z))
    v = v.view(case["rows"], case["groups"], -1)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return (v.view(case["rows"], case["cols"]) * st["w"].float()).to(st["y"].dtype)


def _plain_dense(st, case):
    v = torch.matmul(st["x"].float(), st["w"].float().t())
    if case["bias"]:
        v = v + st["b"].float()
    if case["silu"]:
        v = v * torch.sigmoid(v)
    if st["r"] is not None:
        v = v + st["r"].float()
    return v.to(st["y"].dtype)


_PLAIN = {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm, "dense": _plain_dense}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "conv":
        T, C, W = case["tokens"], case["channels"], case["width"]
        return {"bytes": T * C * (SIZE[case["x"]] + SIZE[case["y"]]) + 2 * C * (W + 1) + 8 * case["seqs"] * (W - 1) * C,
                "flops": 2 * T * C * W}
    if op == "scan":
        H, P, N, T = case["heads"], case["headdim"], case["d_state"], case["tokens"]
        rows = H * P * (SIZE[case["x"]] + SIZE[case["y"]]) + 2 * case["groups"] * N * SIZE[case["x"]] + H * SIZE[case["dt"]]
        return {"bytes": T * rows + 2 * case["seqs"] * H * P * N * SIZE[case["state"]], "flops": 4 * T * H * P * N}
    if op == "norm":
        z = SIZE[case["z"]] if case["gate"] else 0
        return {"bytes": case["rows"] * case["cols"] * (SIZE[case["y"]] + z + SIZE[case["out"]]) + 2 * case["cols"],
                "flops": 8 * case["rows"] * case["cols"]}
    M, R, K = case["batch"], case["rows"], case["cols"]
    return {"bytes": 2 * R * K + 2 * M * K + M * R * (SIZE[case["y"]] + SIZE.get(case["residual"], 0)),
            "flops": 2 * M * R * K}


# ------------------------------------------------------------------ the definitions, in 64 bits

def _exact_tokens(st, case):
    """For each place in a sequence: which sequences reach it, and their packed rows there."""
    if st["start"] is None:
        yield torch.arange(case["tokens"], device=DEV), torch.arange(case["tokens"], device=DEV)
        return
    cuts = st["start"].tolist()
    lens = [b - a for a, b in zip(cuts, cuts[1:])]
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    seqs, starts = torch.tensor(order, device=DEV), torch.tensor([cuts[s] for s in order], device=DEV)
    for t in range(max(lens)):
        m = sum(v > t for v in lens)
        yield seqs[:m], starts[:m] + t


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "dense":
        v = st["x"].to(f64) @ st["w"].to(f64).t()
        v = v + st["b"].to(f64) if case["bias"] else v
        v = v / (1 + torch.exp(-v)) if case["silu"] else v
        return v + st["r"].to(f64) if st["r"] is not None else v
    if op == "norm":
        g = st["in"].to(f64)
        if case["gate"]:
            z = st["z"].to(f64)
            g = g * z / (1 + torch.exp(-z))
        g = g.reshape(case["rows"], case["groups"], -1)
        g = g / torch.sqrt(g.pow(2).sum(-1, keepdim=True) / g.shape[-1] + EPS)
        return g.reshape(case["rows"], -1) * st["w"].to(f64)
    pool, y = st["state"].to(f64), st["y"].to(f64)
    live, fresh = (st["slot"] >= 0), st["fresh"].bool()
    cur = pool[st["slot"].long().clamp(min=0)].clone()
    cur[fresh] = 0
    if op == "conv":
        x, w, W = st["x"].to(f64), st["w"].to(f64), case["width"]
        # y_t = sum_j w_j x_{t - (W-1) + j}: each sequence behind its own old rows
        cuts = list(range(case["tokens"] + 1)) if st["start"] is None else st["start"].tolist()
        for s, (a, b) in enumerate(zip(cuts, cuts[1:])):
            if b > a and bool(live[s]):
                line = torch.cat([cur[s], x[a:b]])
                v = sum(line[j:j + b - a] * w[:, j] for j in range(W))
                v = v + st["b"].to(f64) if case["bias"] else v
                y[a:b] = v / (1 + torch.exp(-v)) if case["silu"] else v
                pool[int(st["slot"][s])] = line[b - a:]
        return y, pool
    if case["tokens"] * case["seqs"] * case["heads"] * case["headdim"] * case["d_state"] > 3e11:
        return None
    H, P, N, G = case["heads"], case["headdim"], case["d_state"], case["groups"]
    raw = st["dt"].to(f64) + st["dt_bias"].to(f64)
    step = torch.nn.functional.softplus(raw, threshold=20.0)
    keepf = torch.exp(step * -torch.exp(st["A_log"].to(f64)))
    out = torch.zeros(case["tokens"], H, P, dtype=f64, device=DEV)
    for seqs, rows in _exact_tokens(st, case):
        m = len(rows)
        xt = st["x"][rows].to(f64).view(m, H, P)
        Bt = st["B"][rows].to(f64).view(m, G, 1, N).expand(m, G, H // G, N).reshape(m, H, 1, N)
        Ct = st["C"][rows].to(f64).view(m, G, 1, N).expand(m, G, H // G, N).reshape(m, H, N, 1)
        h = cur[seqs] * keepf[rows][..., None, None] + (xt * step[rows][..., None])[..., None] * Bt
        cur[seqs] = h
        out[rows] = torch.matmul(h, Ct)[..., 0]
        if case["D"]:
            out[rows] += st["D"].to(f64)[:, None] * xt
    rows = torch.arange(case["tokens"], device=DEV)
    seq = rows if st["start"] is None else torch.searchsorted(st["start"][1:].long(), rows, right=True)
    ok = live[seq]
    y[ok] = out.reshape(case["tokens"], H * P)[ok]
    n = _lens(st)
    done = live & (n > 0)
    pool[st["slot"].long()[done]] = cur[done]
    return y, pool

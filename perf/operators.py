"""The training-side operators around the expert products, as cases that can be timed and compared.

Four operators of one mixture-of-experts block, each in two forms: a plain one (elementary torch operations in
32 bits, one rounding at the end) and the library's own call.

  norm     layer norm over the hidden width, and its backward pass with the gradients of weight and bias
  ckpt     an activation kept in 8 bits between forward and backward pass, and read back
  swiglu   the experts' gated activation, kept in 8 bits, and its backward pass from what was kept
  wgrad    the experts' weight gradients over the static buffer, [E, H, H'] and the slots' [R, B, H, H']

The 8-bit form, called a checkpoint row below: C signed bytes q, from byte align16(C) on one scale byte s for each
block of 128 columns, and padding to a multiple of 32 bytes. A value is q * 2^(s - 127). The step is
2^max(floor(log2(largest magnitude of the block)) - 6, -126), q is rounded to the nearest even and kept within
+-127. A scale byte of 255 says that the block held an infinity or a NaN; its values come back as NaN.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
BLOCK = 128


# ---------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # The framework's smallest workload (R2 S64 H128): one launch's latency.
        dict(name="norm-tiny-fwd", op="norm_fwd", N=128, H=128, dtype="bf16", saved=False),
        # The medium workload's tokens (R8 S4096 H2048): the norm in front of the router, its output also kept in 8 bits.
        dict(name="norm-medium-fwd-saved", op="norm_fwd", N=32768, H=2048, dtype="bf16", saved=True),
        # Its backward pass, the norm's input kept in 8 bits.
        dict(name="norm-medium-bwd-saved", op="norm_bwd", N=32768, H=2048, dtype="bf16", saved=True),
        # The large workload's tokens (R8 S8192 H7168), input kept as it was.
        dict(name="norm-large-bwd", op="norm_bwd", N=65536, H=7168, dtype="bf16", saved=False),
        # A ragged batch in 32 bits whose rows start at odd addresses: no wide access fits.
        dict(name="norm-odd-bwd-f32", op="norm_bwd", N=777, H=1001, dtype="f32", saved=False),
        # The medium tokens to 8 bits and back.
        dict(name="ckpt-medium", op="ckpt", N=32768, H=2048, dtype="bf16"),
        # A ragged one in 32 bits: the last block is cut, rows at odd addresses.
        dict(name="ckpt-odd-f32", op="ckpt", N=1501, H=1407, dtype="f32"),
        # The medium workload's buffer (R8 S4096 K6) between its two projections (H' 1408): forward, then backward.
        dict(name="swiglu-medium-step", op="swiglu", rows=196608, F=1408),
        # A short buffer with an odd width.
        dict(name="swiglu-odd-step", op="swiglu", rows=1501, F=333),
        # The framework's smallest workload: every group is less than a tile.
        dict(name="wgrad-tiny", op="wgrad", R=2, S=64, K=2, E=8, B=4, H=128, Hp=64, skew=1.0, saved=False),
        # The medium workload's first projection, the dispatched rows kept in 8 bits.
        dict(name="wgrad-medium-saved", op="wgrad", R=8, S=4096, K=6, E=64, B=8, H=2048, Hp=1408, skew=0.3, saved=True),
        # Few, uneven groups, sizes that end inside a tile, the rows as they were.
        dict(name="wgrad-ragged", op="wgrad", R=4, S=1111, K=5, E=12, B=6, H=1160, Hp=520, skew=1.0, saved=False),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ckpt", "swiglu", "wgrad"])
    if op in ("norm_fwd", "norm_bwd", "ckpt"):
        H = _spread(rng, 64, 7168)
        if rng.random() < 0.7:  # a model's width is a multiple of 8 more often than not
            H = H // 8 * 8
        c = dict(op=op, N=_spread(rng, 16, 65536), H=H, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op != "ckpt":
            c["saved"] = rng.random() < 0.5
        return c
    if op == "swiglu":
        F = _spread(rng, 32, 1408)
        if rng.random() < 0.7:
            F = F // 8 * 8
        return dict(op=op, rows=_spread(rng, 64, 196608), F=F)
    while True:
        R = rng.choice([1, 2, 4, 8])
        E = R * rng.randint(1, 8)
        K = rng.randint(1, min(8, E))
        c = dict(op="wgrad", R=R, S=_spread(rng, 16, 4096), K=K, E=E, B=rng.randint(0, 8), H=_spread(rng, 64, 2048) // 8 * 8,
                 Hp=_spread(rng, 64, 1408) // 8 * 8, skew=round(rng.uniform(0.0, 1.5), 2), saved=rng.random() < 0.5)
        rows = R * c["S"] * K
        if rows <= 65536 and rows * c["H"] * c["Hp"] <= 65536 * 2048 * 1408 // 4:
            return c


# ---------------------------------------------------------------------------------------------------- inputs


def _row_bytes(C):
    return -(-(-(-C // 16) * 16 + -(-C // BLOCK)) // 32) * 32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _stream(g, N, H, dtype):
    """A residual stream: channels of different spread and offset, a few of them far out, rows of different size."""
    spread = torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))
    spread[torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] *= 12.0
    offset = 0.3 * torch.randn(H, generator=g, device="cuda")
    size = torch.exp(0.4 * torch.randn(N, 1, generator=g, device="cuda"))
    x = torch.randn(N, H, generator=g, device="cuda")
    return x.mul_(spread).add_(offset).mul_(size).to(dtype)


def _groups(case, seed):
    """Group sizes [R, E+B] as a plan gives them: every rank has S*K rows, its own experts' first, then its used slots'."""
    R, E, B, SK = case["R"], case["E"], case["B"], case["S"] * case["K"]
    rng = np.random.default_rng([seed, 17])
    per, n = E // R, np.zeros((R, E + B), np.int64)
    for r in range(R):
        used = int(rng.integers(0, min(B, 2) + 1))
        share = (np.arange(per + used) + 1.0) ** -case["skew"]
        share = rng.permutation(share) * rng.uniform(0.7, 1.3, per + used)
        got = rng.multinomial(SK, share / share.sum())
        n[r, r * per:(r + 1) * per] = got[:per]
        n[r, E:E + used] = got[per:]
    return n


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        N, H, dt = case["N"], case["H"], _dtype(case)
        st["x"] = _stream(g, N, H, dt)
        st["w"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        st["b"] = 0.1 * torch.randn(H, generator=g, device="cuda")
        if op == "norm_bwd":
            x = st["x"].float()
            st["mean"] = x.mean(1)
            st["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt()
            del x
            st["dy"] = (1e-3 * torch.randn(N, H, generator=g, device="cuda")).to(dt)
            if case["saved"]:
                st["x"] = _save(st["x"])
    elif op == "ckpt":
        st["x"] = _stream(g, case["N"], case["H"], _dtype(case))
    elif op == "swiglu":
        rows, F = case["rows"], case["F"]
        st["gu"] = torch.randn(rows, 2 * F, generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
        st["da"] = (1e-3 * torch.randn(rows, F, generator=g, device="cuda")).to(torch.bfloat16)
    else:
        R, E, B, H, Hp = (case[k] for k in ("R", "E", "B", "H", "Hp"))
        n = _groups(case, seed)
        rows = R * case["S"] * case["K"]
        st["cu"] = torch.from_numpy(np.cumsum(n, 1).astype(np.int32)).cuda()
        # what the plain form goes by instead of ragged groups: the weight rows that have to be written, the longest group
        st["slots"] = torch.from_numpy(np.flatnonzero(n[:, E:].reshape(-1))).cuda()
        st["longest"] = int(n.max())
        x = torch.randn(rows, H, generator=g, device="cuda").to(torch.bfloat16)
        st["x"] = _save(x) if case["saved"] else x
        st["dy"] = (1e-3 * torch.randn(rows, Hp, generator=g, device="cuda")).to(torch.bfloat16)
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["home"] = torch.zeros(E, H, Hp, device="cuda")
        st["slot"] = torch.zeros(R, B, H, Hp, device="cuda")
    return st


# ------------------------------------------------------------------------------------------ the plain forms


def _blocks(x):
    """x [N, C] in 32 bits as [N, blocks, 128], filled up with zeros."""
    N, C = x.shape
    n = -(-C // BLOCK)
    return torch.nn.functional.pad(x.float(), (0, n * BLOCK - C)).view(N, n, BLOCK)


def _quantise(x):
    """The bytes q [N, C] and scale bytes s [N, blocks] of x [N, C]."""
    b = _blocks(x)
    top = b.abs().amax(2, keepdim=True)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine, top, torch.ones_like(top)))[1] - 7
    k = torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    up = ((127 - k) << 23).view(torch.float32)
    q = torch.where(fine, b * up, torch.zeros_like(b)).round().clamp(-127, 127)
    s = torch.where(fine, k + 127, torch.full_like(k, 255))
    return q.to(torch.int8).flatten(1)[:, : x.shape[1]], s.squeeze(2).to(torch.uint8)


def _values(q, s):
    """The values in 32 bits of bytes q [N, C] and scale bytes s [N, blocks]."""
    s = s.int()
    step = torch.where(s == 255, torch.full_like(s, 0x7FC00000), s << 23).view(torch.float32)
    return (_blocks(q) * step.unsqueeze(2)).flatten(1)[:, : q.shape[1]]


def _save(x):
    """Checkpoint rows, uint8 [N, row bytes], of x [N, C]."""
    N, C = x.shape
    q, s = _quantise(x)
    rows = torch.zeros(N, _row_bytes(C), dtype=torch.uint8, device=x.device)
    rows[:, :C] = q.view(torch.uint8)
    at = -(-C // 16) * 16
    rows[:, at:at + s.shape[1]] = s
    return rows


def _load(rows, C):
    """The values in 32 bits, [N, C], of checkpoint rows."""
    at = -(-C // 16) * 16
    return _values(rows[:, :C].contiguous().view(torch.int8), rows[:, at:at + -(-C // BLOCK)])


def _norm_fwd(st):
    x = st["x"].float()
    mean = x.mean(1)
    c = x - mean.unsqueeze(1)
    rstd = (c.square().mean(1) + EPS).rsqrt()
    y = (c * rstd.unsqueeze(1) * st["w"] + st["b"]).to(st["x"].dtype)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if st["case"]["saved"]:
        out["kept"] = _load(_save(y), y.shape[1]).to(y.dtype)
    return out


def _norm_bwd(st):
    H = st["case"]["H"]
    x = _load(st["x"], H) if st["case"]["saved"] else st["x"].float()
    dy, mean, rstd = st["dy"].float(), st["mean"].unsqueeze(1), st["rstd"].unsqueeze(1)
    xhat = (x - mean) * rstd
    t = dy * st["w"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(st["dy"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _swiglu(st):
    rows, F = st["case"]["rows"], st["case"]["F"]
    gu = st["gu"].float()
    a = (gu[:, :F] * (1 / (1 + torch.exp(-gu[:, :F]))) * gu[:, F:]).to(torch.bfloat16)
    kept = _save(st["gu"].view(2 * rows, F))
    g, u = _load(kept, F).view(rows, 2, F).unbind(1)
    da, sig = st["da"].float(), 1 / (1 + torch.exp(-g))
    dg = da * u * sig * (1 + g * (1 - sig))
    du = da * g * sig
    return {"a": a, "dgu": torch.cat([dg, du], 1).to(torch.bfloat16), "a_again": (g * sig * u).to(torch.bfloat16)}


def _wgrad(st):
    c = st["case"]
    R, E, B, H = c["R"], c["E"], c["B"], c["H"]
    dev, cu, SK = st["dy"].device, st["cu"].long(), c["S"] * c["K"]
    x = _load(st["x"], H) if c["saved"] else st["x"].float()
    dy = st["dy"].float()
    # one group for each weight row: expert e's on its own rank, slot b's on the slot's
    begin = torch.nn.functional.pad(cu, (1, 0))[:, :-1]
    e = torch.arange(E, device=dev)
    rank = torch.cat([e // (E // R), st["slots"] // max(1, B)])
    group = torch.cat([e, E + st["slots"] % max(1, B)])
    first, length = rank * SK + begin[rank, group], (cu - begin)[rank, group]
    step = torch.arange(st["longest"], device=dev)
    row = (first.unsqueeze(1) + step).clamp(max=x.shape[0] - 1)
    there = (step < length.unsqueeze(1)).unsqueeze(2)
    grads = torch.bmm((x[row] * there).transpose(1, 2), dy[row] * there)
    st["home"].copy_(grads[:E])
    st["slot"].view(R * B, H, -1)[st["slots"]] = grads[E:]
    return {"home": st["home"], "slot": st["slot"]}


def _plain(st):
    op = st["case"]["op"]
    if op == "norm_fwd":
        return _norm_fwd(st)
    if op == "norm_bwd":
        return _norm_bwd(st)
    if op == "ckpt":
        return {"kept": _load(_save(st["x"]), st["case"]["H"]).to(st["x"].dtype)}
    return _swiglu(st) if op == "swiglu" else _wgrad(st)


# --------------------------------------------------------------------------------------- the library's calls


def _own(st):
    import load_balancing_topk_gb300 as mep

    c, op = st["case"], st["case"]["op"]
    if op == "norm_fwd":
        x = st["x"]
        kept = torch.empty(c["N"], mep.ckpt_row_bytes(c["H"]), dtype=torch.uint8, device=x.device) if c["saved"] else None
        y, mean, rstd = mep.mep_layer_norm(x, st["w"], st["b"], EPS, y_ckpt=kept)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if c["saved"]:
            out["kept"] = mep.mep_ckpt_load(kept, c["H"], dtype=x.dtype)
        return out
    if op == "norm_bwd":
        dx, dw, db = mep.mep_layer_norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "ckpt":
        return {"kept": mep.mep_ckpt_load(mep.mep_ckpt_save(st["x"]), c["H"], dtype=st["x"].dtype)}
    if op == "swiglu":
        kept = torch.empty(c["rows"], 2, mep.ckpt_row_bytes(c["F"]), dtype=torch.uint8, device=st["gu"].device)
        a = mep.mep_swiglu(st["gu"], ckpt=kept)
        dgu, again = mep.mep_swiglu_backward(st["da"], kept)
        return {"a": a, "dgu": dgu, "a_again": again}
    mep.mep_grouped_wgrad(st["x"], st["dy"], st["cu"], st["home"], st["slot"], st["status"], c["R"], c["S"], c["K"])
    return {"home": st["home"], "slot": st["slot"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------- work and values


def work(case):
    op = case["op"]
    if op == "wgrad":
        rows = case["R"] * case["S"] * case["K"]
        x = case["H"] + -(-case["H"] // BLOCK) if case["saved"] else 2 * case["H"]
        return {"bytes": rows * (x + 2 * case["Hp"]) + 4 * case["E"] * case["H"] * case["Hp"], "flops": 2 * rows * case["H"] * case["Hp"]}
    if op == "swiglu":
        rows, F = case["rows"], case["F"]
        kept = 2 * (F + -(-F // BLOCK))
        return {"bytes": rows * (4 * F + 2 * F + kept + kept + 2 * F + 4 * F + 2 * F), "flops": 40 * rows * F}
    N, H, size = case["N"], case["H"], 2 if case["dtype"] == "bf16" else 4
    kept = H + -(-H // BLOCK)
    if op == "norm_fwd":
        row = 2 * size * H + 8 + ((2 * kept + size * H) if case["saved"] else 0)
        return {"bytes": N * row + 8 * H, "flops": 8 * N * H}
    if op == "norm_bwd":
        row = (kept if case["saved"] else size * H) + 2 * size * H + 8
        return {"bytes": N * row + 12 * H, "flops": 14 * N * H}
    return {"bytes": N * (2 * size * H + 2 * kept), "flops": 4 * N * H}


def _exact_kept(v, dt):
    """In 64 bits, what v (already in the kept type) stands for after 8 bits; its blocks by reshaping and log2."""
    N, C = v.shape
    out = torch.zeros(N, -(-C // BLOCK) * BLOCK, dtype=torch.float64, device=v.device)
    out[:, :C] = v.to(dt).double()
    out = out.view(N, -1, BLOCK)
    top = out.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, torch.where(torch.exp2(e) > top, e - 1, e))
    step = torch.exp2((e - 6).clamp(min=-126))
    return (torch.round(out / step).clamp(-127, 127) * step).view(N, -1)[:, :C]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    dt = _dtype(case)
    if op == "ckpt":
        return {"kept": _exact_kept(st["x"], dt)}
    if op == "norm_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = 1 / torch.sqrt(var + EPS)
        y = x.sub_(mean[:, None]).mul_(rstd[:, None]).mul_(st["w"].double()).add_(st["b"].double())
        out = {"y": y, "mean": mean, "rstd": rstd}
        if case["saved"]:
            out["kept"] = _exact_kept(y, dt)
        return out
    if op == "norm_bwd":
        H = case["H"]
        if case["saved"]:
            at = -(-H // 16) * 16
            s = st["x"][:, at:at + -(-H // BLOCK)].double()
            x = st["x"][:, :H].contiguous().view(torch.int8).double() * torch.exp2(s - 127).repeat_interleave(BLOCK, 1)[:, :H]
        else:
            x = st["x"].double()
        r = st["rstd"].double()[:, None]
        xhat = x.sub_(st["mean"].double()[:, None]).mul_(r)
        dy = st["dy"].double()
        dweight, dbias = torch.einsum("nh,nh->h", dy, xhat), dy.sum(0)
        t = dy.mul_(st["w"].double())
        c1, c2 = t.sum(1, keepdim=True) / H, torch.einsum("nh,nh->n", t, xhat)[:, None] / H
        return {"dx": t.sub_(c1).sub_(xhat.mul_(c2)).mul_(r), "dweight": dweight, "dbias": dbias}
    if op == "swiglu":
        rows, F = case["rows"], case["F"]
        g, u = st["gu"][:, :F].double(), st["gu"][:, F:].double()
        a = g * torch.sigmoid(g) * u
        g, u, da = _exact_kept(st["gu"][:, :F], dt), _exact_kept(st["gu"][:, F:], dt), st["da"].double()
        s = torch.sigmoid(g)
        dgu = torch.empty(rows, 2 * F, dtype=torch.float64, device=g.device)
        dgu[:, :F] = da * u * (s + g * s * (1 - s))
        dgu[:, F:] = da * g * s
        return {"a": a, "dgu": dgu, "a_again": g.mul_(s).mul_(u)}
    R, E, B, H, Hp = (case[k] for k in ("R", "E", "B", "H", "Hp"))
    n, SK = _groups(case, seed), case["S"] * case["K"]
    if case["saved"]:
        at = -(-H // 16) * 16
        s = st["x"][:, at:at + -(-H // BLOCK)].double()
        x = st["x"][:, :H].contiguous().view(torch.int8).double() * torch.exp2(s - 127).repeat_interleave(BLOCK, 1)[:, :H]
    else:
        x = st["x"].double()
    home = torch.zeros(E, H, Hp, dtype=torch.float64, device=x.device)
    slot = torch.zeros(R, B, H, Hp, dtype=torch.float64, device=x.device)
    for r in range(R):
        at = r * SK
        for j in range(E + B):
            if n[r, j]:
                part = x[at:at + n[r, j]].t() @ st["dy"][at:at + n[r, j]].double()
                if j < E:
                    home[j] += part
                else:
                    slot[r, j - E] += part
            at += int(n[r, j])
    return {"home": home, "slot": slot}

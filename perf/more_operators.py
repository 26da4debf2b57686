"""The serving-side operators around the experts, and the router, as cases that can be timed and compared.

Each operator in two forms: a plain one (elementary torch operations in 32 bits, one rounding at the end) and the
library's own call.

  layer    the whole mixture-of-experts layer for a few tokens, experts in bf16 or in 4 bits
  product  a few rows times a matrix held in 4 bits
  save     a matrix to 4 bits with one scale for each group of rows of a column, and its values back
  route    from logits to each token's experts and weights, and the logits' gradient

The 4-bit form of a matrix [K, N], in groups of G rows (32, 64 or 128). A group's scale is the bf16 nearest to (its
largest magnitude) / 7, and q = w / scale to the nearest whole number, ties to even, within -7 .. 7; a value is
q * scale. A group of scale 0 stands for zeros, one that holds an infinity or a NaN has a NaN for a scale. Columns lie
in panels of 64, rows in blocks of 128 (the last ones filled up with zeros); a panel's blocks follow one another, and
the panels. A block is 4096 bytes of pairs and then its scales. With k = 64 h + 16 j + 8 i + 2 t + e a row of the block
and n = 16 c + 8 l + g a column of the panel, (q + 8) is the low (l = 0) or high half of the byte
((((4 h + c) * 8 + g) * 4 + t) * 4 + j) * 4 + 2 e + i, and a column's scale is the bf16 number 16 c + 2 g + l of its
group's 64.
"""

import math

import numpy as np
import torch

own = False

ROWS, COLS = 128, 64  # of a block


# ---------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # The framework's smallest workload (H128, E8, K2) with four tokens: a launch's latency.
        dict(name="layer-tiny", op="layer", T=4, K=2, E=8, H=128, F=64, bits=16, group=128, skew=1.0, pad=0),
        # One token of the medium workload (E64 K6 H2048 H'1408): the next token of a single sequence.
        dict(name="layer-medium-one", op="layer", T=1, K=6, E=64, H=2048, F=1408, bits=16, group=128, skew=0.3, pad=0),
        # The large workload (E256 K8 H7168) with the most tokens that the layer takes, nearly every expert in use.
        dict(name="layer-large-64", op="layer", T=64, K=8, E=256, H=7168, F=1408, bits=16, group=128, skew=0.3, pad=0),
        # The large workload's next token, experts in 4 bits.
        dict(name="layer-large-4bit-one", op="layer", T=1, K=8, E=256, H=7168, F=1408, bits=4, group=128, skew=0.3, pad=0),
        # The same for a captured batch of 16 places, three of them empty.
        dict(name="layer-large-4bit-16", op="layer", T=16, K=8, E=256, H=7168, F=1408, bits=4, group=64, skew=0.3, pad=3),
        # A projection of the large workload's width for one token.
        dict(name="product-large-one", op="product", T=1, K=7168, N=7168, group=128, dtype="bf16"),
        # The most rows, to a vocabulary's logits in 32 bits.
        dict(name="product-wide-64", op="product", T=64, K=2048, N=65536, group=128, dtype="f32"),
        # Sizes that end inside a panel, a block and a group, rows at odd addresses.
        dict(name="product-odd", op="product", T=5, K=1001, N=1407, group=32, dtype="bf16"),
        # The medium workload's first projections of all experts, gate and up as parts of their own.
        dict(name="save-medium", op="save", M=64, K=2048, N=2816, parts=2, group=128, dtype="bf16"),
        # A ragged matrix in 32 bits.
        dict(name="save-odd-f32", op="save", M=3, K=777, N=1001, parts=1, group=64, dtype="f32"),
        # The large workload's tokens (R8 S8192 E256 K8) through the router, forward and backward, with a selection bias.
        dict(name="route-large-step", op="route", N=65536, E=256, K=8, skew=0.5, bias=True, masked=False, dtype="f32"),
        # A ragged batch of bf16 logits, which tie often, some experts masked out, some rows without any.
        dict(name="route-odd-step", op="route", N=777, E=43, K=5, skew=0.5, bias=False, masked=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over the logarithm of its range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "layer", "layer", "product", "save", "route"])
    if op == "layer":
        while True:
            E = _spread(rng, 2, 256)
            T = _spread(rng, 1, 64)
            c = dict(op=op, T=T, K=rng.randint(1, min(8, E)), E=E, H=_spread(rng, 64, 7168) // 8 * 8,
                     F=_spread(rng, 32, 1408) // 8 * 8, bits=rng.choice([16, 4]), group=rng.choice([32, 64, 128]),
                     skew=round(rng.uniform(0.0, 1.5), 2), pad=rng.choice([0, 0, rng.randint(0, T - 1)]))
            if E * c["H"] * c["F"] <= 64 * 2048 * 1408:
                return c
    if op == "product":
        while True:
            K, N = _spread(rng, 32, 7168), _spread(rng, 32, 65536)
            if rng.random() < 0.7:  # a model's widths are multiples of 8 more often than not
                K, N = K // 8 * 8, N // 8 * 8
            if K * N <= 2048 * 65536:
                return dict(op=op, T=_spread(rng, 1, 64), K=K, N=N, group=rng.choice([32, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
    if op == "save":
        while True:
            parts = rng.choice([1, 2])
            c = dict(op=op, M=_spread(rng, 1, 64), K=_spread(rng, 32, 7168), N=_spread(rng, 32, 2816) * parts, parts=parts,
                     group=rng.choice([32, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
            if c["M"] * c["K"] * c["N"] <= 64 * 2048 * 1408:
                return c
    E = _spread(rng, 4, 384)
    return dict(op=op, N=_spread(rng, 16, 65536), E=E, K=rng.randint(1, min(8, E)), skew=round(rng.uniform(0.0, 1.5), 2),
                bias=rng.random() < 0.5, masked=rng.random() < 0.3, dtype=rng.choice(["f32", "f32", "bf16"]))


# ---------------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _choice(case, seed):
    """Experts [T, K] of a layer's tokens, -1 for the empty places, and their weights."""
    T, K, E = case["T"], case["K"], case["E"]
    rng = np.random.default_rng([seed, 23])
    logits = rng.normal(size=(T, E)) - case["skew"] * np.log(rng.permutation(E) + 1.0)
    idx = np.argsort(-logits, 1)[:, :K]
    top = np.exp(np.take_along_axis(logits, idx, 1))
    idx[T - case["pad"]:] = -1
    return idx, (top / top.sum(1, keepdims=True)).astype(np.float32)


def _weights(g, M, K, N, parts, group):
    """4-bit matrices [M, parts, bytes] of normal weights [M, K, N]; a few at a time, so that they fit."""
    out, most = [], max(1, (1 << 28) // (K * N))
    for m in range(0, M, most):
        w = torch.randn(min(most, M - m), K, N, generator=g, device="cuda").mul_(K ** -0.5).to(torch.bfloat16)
        out.append(_w4_save(w, parts, group))
    return torch.cat(out)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "layer":
        T, K, E, H, F = (case[k] for k in ("T", "K", "E", "H", "F"))
        idx, top = _choice(case, seed)
        st["x"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        st["idx"] = torch.from_numpy(idx.astype(np.int32)).cuda()
        st["w"] = torch.from_numpy(top).cuda()
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["bits"] == 4:
            st["w1"] = _weights(g, E, H, 2 * F, 2, case["group"])
            st["w2"] = _weights(g, E, F, H, 1, case["group"])
        else:
            st["w1"] = torch.empty(E, H, 2 * F, dtype=torch.bfloat16, device="cuda").normal_(0, H ** -0.5, generator=g)
            st["w2"] = torch.empty(E, F, H, dtype=torch.bfloat16, device="cuda").normal_(0, F ** -0.5, generator=g)
        # what the plain form goes by instead of ragged groups: the experts in use, each one's tokens, each assignment's place
        used, most = np.unique(idx[idx >= 0]), 1
        token, place = np.zeros((len(used), T), np.int64), np.zeros((T, K), np.int64)
        for i, e in enumerate(used):
            t, k = np.nonzero(idx == e)
            token[i, :len(t)], most = t, max(most, len(t))
            place[t, k] = i * T + np.arange(len(t))
        st["used"] = torch.from_numpy(used).cuda()
        st["token"] = torch.from_numpy(token[:, :most]).cuda()
        st["place"] = torch.from_numpy(place // T * most + place % T).cuda()
    elif op == "product":
        st["x"] = torch.randn(case["T"], case["K"], generator=g, device="cuda").to(torch.bfloat16)
        st["w4"] = _weights(g, 1, case["K"], case["N"], 1, case["group"])[0]
    elif op == "save":
        w = torch.randn(case["M"], case["K"], case["N"], generator=g, device="cuda")
        st["w"] = w.mul_(case["K"] ** -0.5).to(_dtype(case))
    else:
        N, E, K = case["N"], case["E"], case["K"]
        popular = torch.randperm(E, generator=g, device="cuda").float()
        logits = torch.randn(N, E, generator=g, device="cuda") - case["skew"] * torch.log(popular + 1)
        if case["masked"]:
            logits[torch.rand(N, E, generator=g, device="cuda") < 0.3] = -math.inf
            logits[torch.randint(0, N, (1 + N // 16,), generator=g, device="cuda")] = -math.inf
        st["logits"] = logits.to(_dtype(case))
        st["bias"] = 0.3 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        st["dw"] = 1e-3 * torch.randn(N, K, generator=g, device="cuda")
    return st


# ------------------------------------------------------------------------------------------ the plain forms


def _w4_save(w, parts, group):
    """w [M, K, N] in 4 bits, uint8 [M, parts, bytes]."""
    M, K, N = w.shape
    n = N // parts
    kb, p = -(-K // ROWS), -(-n // COLS)
    w = torch.nn.functional.pad(w.view(M, K, parts, n).transpose(1, 2).float(), (0, p * COLS - n, 0, kb * ROWS - K))
    w = w.reshape(M * parts, kb * ROWS // group, group, p * COLS)
    top = w.abs().amax(2, keepdim=True)
    scale = torch.where(torch.isfinite(top), top / 7, torch.full_like(top, math.nan)).to(torch.bfloat16)
    s = scale.float()
    q = torch.where(s > 0, w / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(w)).round().clamp(-7, 7) + 8
    # rows (block, h, j, i, t, e), columns (panel, c, l, g)
    q = q.to(torch.uint8).view(-1, kb, 2, 4, 2, 4, 2, p, 4, 2, 8).permute(0, 7, 1, 2, 8, 10, 5, 3, 6, 4, 9)
    pairs = (q[..., 0] | (q[..., 1] << 4)).reshape(M * parts, p, kb, -1)
    scale = scale.view(-1, kb, ROWS // group, p, 4, 2, 8).permute(0, 3, 1, 2, 4, 6, 5).contiguous()
    return torch.cat([pairs, scale.view(torch.uint8).reshape(M * parts, p, kb, -1)], 3).view(M, parts, -1)


def _w4_load(w4, K, N, group):
    """The values in 32 bits, [M, K, N], of matrices in 4 bits, uint8 [M, bytes]."""
    kb, p = -(-K // ROWS), -(-N // COLS)
    w4 = w4.view(-1, p, kb, ROWS * COLS // 2 + ROWS // group * COLS * 2)
    pairs, scale = w4[..., :ROWS * COLS // 2], w4[..., ROWS * COLS // 2:].contiguous().view(torch.bfloat16)
    q = torch.stack([pairs & 15, pairs >> 4], -1).view(-1, p, kb, 2, 4, 8, 4, 4, 2, 2, 2).float() - 8
    q = q.permute(0, 2, 3, 7, 9, 6, 8, 1, 4, 10, 5).reshape(-1, kb * ROWS // group, group, p * COLS)
    scale = scale.view(-1, p, kb, ROWS // group, 4, 8, 2).permute(0, 2, 3, 1, 4, 6, 5).reshape(-1, kb * ROWS // group, 1, p * COLS)
    return (q * scale.float()).view(-1, kb * ROWS, p * COLS)[:, :K, :N]


def _layer(st):
    c = st["case"]
    H, F = c["H"], c["F"]
    used, x, here = st["used"], st["x"].float(), st["idx"] >= 0
    if c["bits"] == 4:
        w = _w4_load(st["w1"][used].flatten(0, 1), H, F, c["group"])
        g, u = torch.bmm(x[st["token"]], w[0::2]), torch.bmm(x[st["token"]], w[1::2])
        w2 = _w4_load(st["w2"][used].flatten(0, 1), F, H, c["group"])
    else:
        g, u = torch.bmm(x[st["token"]], st["w1"][used].float()).split(F, 2)
        w2 = st["w2"][used].float()
    y = torch.bmm(g * (1 / (1 + torch.exp(-g))) * u, w2).flatten(0, 1)
    weight = torch.where(here, st["w"], torch.zeros_like(st["w"]))
    return {"out": (weight.unsqueeze(2) * y[st["place"]]).sum(1).to(torch.bfloat16), "status": st["status"]}


def _route(st):
    c = st["case"]
    logits = st["logits"].float()
    key = logits if st["bias"] is None else logits + st["bias"]
    idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : c["K"]]
    top = torch.gather(logits, 1, idx)
    there = top > -math.inf
    most = top.amax(1, keepdim=True)
    e = torch.where(there, torch.exp(top - torch.where(most > -math.inf, most, torch.zeros_like(most))), torch.zeros_like(top))
    w = e / torch.where(there.any(1, keepdim=True), e.sum(1, keepdim=True), torch.ones_like(most))
    d = w * (st["dw"] - (w * st["dw"]).sum(1, keepdim=True))
    dlogits = torch.zeros_like(logits).scatter_(1, idx, d).to(st["logits"].dtype)
    return {"idx": torch.where(there, idx, torch.full_like(idx, -1)).to(torch.int32), "w": w, "dlogits": dlogits}


def _plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "layer":
        return _layer(st)
    if op == "product":
        return {"y": (st["x"].float() @ _w4_load(st["w4"], c["K"], c["N"], c["group"])[0]).to(_dtype(c))}
    if op == "save":
        M, K, N, n = c["M"], c["K"], c["N"], c["N"] // c["parts"]
        w = _w4_load(_w4_save(st["w"], c["parts"], c["group"]).flatten(0, 1), K, n, c["group"])
        return {"kept": w.view(M, -1, K, n).transpose(1, 2).reshape(M, K, N).to(_dtype(c))}
    return _route(st)


# --------------------------------------------------------------------------------------- the library's calls


def _own(st):
    import load_balancing_topk_gb300 as mep

    c, op = st["case"], st["case"]["op"]
    if op == "layer":
        kind = dict(F=c["F"], group=c["group"]) if c["bits"] == 4 else {}
        return {"out": mep.mep_expert_layer(st["x"], st["idx"], st["w"], st["w1"], st["w2"], st["status"], **kind), "status": st["status"]}
    if op == "product":
        return {"y": mep.mep_w4_product(st["x"], st["w4"], c["N"], group=c["group"], dtype=_dtype(c))}
    if op == "save":
        w4 = mep.mep_w4_save(st["w"], group=c["group"], parts=c["parts"])
        return {"kept": mep.mep_w4_load(w4, c["K"], c["N"], group=c["group"], dtype=_dtype(c))}
    idx, w = mep.mep_route(st["logits"], c["K"], st["bias"], skip_masked=True)
    return {"idx": idx, "w": w, "dlogits": mep.mep_route_backward(st["dw"], w, idx, c["E"], dtype=st["logits"].dtype)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------- work and values


def _w4_bytes(K, N, group):
    return K * N / 2 + 2 * -(-K // group) * N


def work(case):
    op = case["op"]
    if op == "layer":
        T, K, H, F = (case[k] for k in ("T", "K", "H", "F"))
        idx, _ = _choice(case, 0)
        used, rows = len(np.unique(idx[idx >= 0])), int((idx >= 0).sum())
        expert = 6 * H * F if case["bits"] == 16 else _w4_bytes(H, 2 * F, case["group"]) + _w4_bytes(F, H, case["group"])
        return {"bytes": used * expert + 4 * T * H + 8 * T * K, "flops": 6 * rows * H * F}
    if op == "product":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": _w4_bytes(K, N, case["group"]) + 2 * T * K + (2 if case["dtype"] == "bf16" else 4) * T * N, "flops": 2 * T * K * N}
    if op == "save":
        M, K, N, size = case["M"], case["K"], case["N"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * (2 * size * K * N + 2 * _w4_bytes(K, N, case["group"])), "flops": 5 * M * K * N}
    N, E, K, size = case["N"], case["E"], case["K"], 2 if case["dtype"] == "bf16" else 4
    return {"bytes": N * (2 * size * E + 20 * K), "flops": 4 * N * E}


def _exact_w4(w4, K, N, group):
    """In 64 bits, the values [K, N] of one matrix in 4 bits, each fetched from where it lies."""
    k = torch.arange(K, device=w4.device)[:, None]
    n = torch.arange(N, device=w4.device)[None, :]
    size = 4096 + 128 * (128 // group)
    block = (n // 64 * -(-K // 128) + k // 128) * size
    b, m = k % 128, n % 64
    h, j, i, t, e = b // 64, b // 16 % 4, b // 8 % 2, b // 2 % 4, b % 2
    c, l, g = m // 16, m // 8 % 2, m % 8
    pair = w4[block + ((((4 * h + c) * 8 + g) * 4 + t) * 4 + j) * 4 + 2 * e + i].long()
    q = (pair // 16 ** l) % 16 - 8
    at = block + 4096 + 2 * (b // group * 64 + 16 * c + 2 * g + l)
    bits = w4[at].int() + 256 * w4[at + 1].int()
    return q.double() * (bits << 16).view(torch.float32).double()


def _exact_kept(w, group):
    """In 64 bits, what one matrix [K, N] stands for after 4 bits."""
    out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    for k in range(0, w.shape[0], group):
        v = w[k:k + group].double()
        s = (v.abs().amax(0) / 7).to(torch.bfloat16).double()
        out[k:k + group] = torch.where(s > 0, torch.round(v / s.clamp(min=1e-300)), 0.0) * s
    return out


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "layer":
        H, F, group = case["H"], case["F"], case["group"]
        idx, _ = _choice(case, seed)
        out = torch.zeros(case["T"], H, dtype=torch.float64, device="cuda")
        for e in np.unique(idx[idx >= 0]):
            t, k = (torch.from_numpy(v).cuda() for v in np.nonzero(idx == e))
            if case["bits"] == 4:
                g, u = (st["x"][t].double() @ _exact_w4(st["w1"][e, part], H, F, group) for part in (0, 1))
                w2 = _exact_w4(st["w2"][e, 0], F, H, group)
            else:
                gu = st["x"][t].double() @ st["w1"][e].double()
                g, u, w2 = gu[:, :F], gu[:, F:], st["w2"][e].double()
            out.index_add_(0, t, st["w"][t, k].double()[:, None] * ((torch.sigmoid(g) * g * u) @ w2))
        return {"out": out, "status": None}
    if op == "product":
        K, N = case["K"], case["N"]
        return {"y": st["x"].double() @ _exact_w4(st["w4"][0], K, N, case["group"])}
    if op == "save":
        M, K, N, n = case["M"], case["K"], case["N"], case["N"] // case["parts"]
        kept = torch.empty(M, K, N, dtype=torch.float64, device="cuda")
        for m in range(M):
            kept[m] = _exact_kept(st["w"][m], case["group"])
        return {"kept": kept}
    logits, K = st["logits"].cpu().float().numpy(), case["K"]
    key = logits if st["bias"] is None else logits + st["bias"].cpu().numpy()
    N, E = key.shape
    idx = np.lexsort((np.broadcast_to(np.arange(E), key.shape), -key.astype(np.float64)), axis=1)[:, :K]
    top = np.take_along_axis(logits, idx, 1).astype(np.float64)
    most = np.maximum(top.max(1, keepdims=True), -1e300)
    w = np.exp(top - most) * (top > -np.inf)
    w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
    dw = st["dw"].cpu().numpy().astype(np.float64)
    d = np.zeros((N, E))
    np.put_along_axis(d, idx, w * (dw - (w * dw).sum(1, keepdims=True)), 1)
    return {"idx": torch.from_numpy(np.where(top > -np.inf, idx, -1)), "w": torch.from_numpy(w), "dlogits": torch.from_numpy(d)}

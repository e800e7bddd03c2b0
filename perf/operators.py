"""The products of wide experts and of 8-bit integers: what they are, their plain form, their
definition in 64 bits, and the sizes at which they are measured.

Three operators, as a program uses them beside the routed layer:

- "product": y[r] = (SiLU of) x[token of r] . W[e]^T for the rows r of each expert's group, the
  groups of ragged sizes and one after another in the row order (what routing, then scheduling
  with one expert per group, leaves behind);
- "gradient": its backward, dx[r] = dy[r] . W[e] and dW[e] = sum over the group's rows of
  dy[r]^T x[token of r];
- "int8": y = (SiLU of) x . W^T with W in 8-bit integers and one scale per output channel, the
  tokens' rows quantised in the call with one scale each; for one matrix, or by expert.

A case's sizes: tokens; topk experts of E per token (rows = tokens * topk); n_in and n_out, the
widths of a weight matrix [n_out, n_in].  skew: how unevenly the tokens choose (0: alike)."""
import numpy as np
import torch

own = False


def listed():
    return [
        # one token being decoded: latency and the bytes of its eight experts
        dict(name="product-one-token", op="product", tokens=1, topk=8, E=64, n_in=2048,
             n_out=1024, skew=0.0, gather=True, silu=False, f32=False),
        # a decode batch: most experts have a few rows, and every weight is read once
        dict(name="product-decode", op="product", tokens=64, topk=8, E=64, n_in=2048, n_out=1024,
             skew=0.5, gather=True, silu=True, f32=False),
        # a short ragged batch, odd widths, experts without rows, fp32 output
        dict(name="product-ragged", op="product", tokens=1201, topk=3, E=24, n_in=1000, n_out=712,
             skew=1.1, gather=False, silu=False, f32=True),
        # prefill of 8 sequences of 2048 tokens
        dict(name="product-prefill", op="product", tokens=16384, topk=8, E=64, n_in=2048,
             n_out=1024, skew=0.3, gather=True, silu=True, f32=False),
        # the gradients of a small odd batch
        dict(name="gradient-ragged", op="gradient", tokens=130, topk=2, E=16, n_in=200, n_out=328,
             skew=0.8, gather=False, silu=False, f32=True),
        # a training step's first product: tokens gathered by expert
        dict(name="gradient-step", op="gradient", tokens=4096, topk=8, E=32, n_in=1024,
             n_out=2048, skew=0.3, gather=True, silu=False, f32=False),
        # its second product, many experts: the weights' gradients are most of the bytes
        dict(name="gradient-many-experts", op="gradient", tokens=2048, topk=8, E=128, n_in=512,
             n_out=2048, skew=0.3, gather=False, silu=False, f32=False),
        # few experts, long groups
        dict(name="gradient-long-groups", op="gradient", tokens=16384, topk=2, E=8, n_in=2048,
             n_out=2048, skew=0.2, gather=False, silu=False, f32=False),
        # the shared MLP's first product in 8 bits: one token, a decode batch, a prefill
        dict(name="int8-one-token", op="int8", tokens=1, topk=0, E=1, n_in=2048, n_out=8192,
             skew=0.0, gather=False, silu=False, f32=False),
        dict(name="int8-decode", op="int8", tokens=64, topk=0, E=1, n_in=2048, n_out=8192,
             skew=0.0, gather=False, silu=True, f32=False),
        dict(name="int8-prefill", op="int8", tokens=16384, topk=0, E=1, n_in=2048, n_out=8192,
             skew=0.0, gather=False, silu=True, f32=False),
        # a decode batch's experts in 8 bits
        dict(name="int8-experts", op="int8", tokens=64, topk=8, E=64, n_in=2048, n_out=1024,
             skew=0.5, gather=True, silu=False, f32=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["product", "gradient", "int8"])
    one = op == "int8" and rng.random() < 0.6
    E = 1 if one else _log(rng, 4, 128)
    topk = 0 if one else rng.randint(1, min(8, E))
    step = 16 if op == "int8" else 8
    while True:
        tokens = _log(rng, 1, 16384)
        n_in = step * _log(rng, 64 // step, 4096 // step)
        n_out = 8 * _log(rng, 8, 1024)
        rows = tokens * max(topk, 1)
        if rows * n_in * n_out <= (1 << 36 if op == "gradient" else 1 << 38) \
                and E * n_in * n_out <= 1 << 28:
            break
    return dict(op=op, tokens=tokens, topk=topk, E=E, n_in=n_in, n_out=n_out,
                skew=round(rng.uniform(0.0, 1.2), 2) if E > 1 else 0.0,
                gather=topk > 0 and (op == "int8" or rng.random() < 0.5),
                silu=op != "gradient" and rng.random() < 0.5, f32=rng.random() < 0.25)


def _groups(case, seed):
    """Which experts the tokens choose, and the rows in expert order: offsets of the experts that
    have rows, those experts' ids, and each row's token (numpy)."""
    T, K, E = case["tokens"], case["topk"], case["E"]
    rng = np.random.default_rng(seed)
    taste = -case["skew"] * np.log(np.arange(1, E + 1))
    score = taste[rng.permutation(E)] + rng.gumbel(size=(T, E))  # the K largest: K distinct draws
    ids = np.argpartition(-score, K - 1, axis=1)[:, :K].reshape(-1)
    token = np.repeat(np.arange(T), K)
    order = np.lexsort((token, ids))
    count = np.bincount(ids, minlength=E)
    return count, token[order]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, K, E, n_in, n_out = (case[k] for k in ("tokens", "topk", "E", "n_in", "n_out"))

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)

    s = {"case": case}
    rows = T * K if K else T
    if K:
        count, token = _groups(case, seed)
        # decode lists the experts that have rows (as a schedule does, its count on the device);
        # the other batches list every expert
        ids = np.nonzero(count)[0] if case["gather"] else np.arange(E)
        off = np.concatenate(([0], np.cumsum(count[ids])))
        s["longest"] = int(count.max())
        s["off"] = torch.from_numpy(off.astype(np.int32)).to(dev)
        if case["gather"]:
            room = min(E, rows) - len(ids)
            s["off"] = torch.cat([s["off"], torch.full((room,), rows, dtype=torch.int32, device=dev)])
            s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(dev)
            s["ids"] = torch.cat([s["ids"], torch.zeros(room, dtype=torch.int32, device=dev)])
            s["n"] = torch.tensor([len(ids)], dtype=torch.int32, device=dev)
            s["rows"] = torch.from_numpy(token.astype(np.int32)).to(dev)
    W = normal(E, n_out, n_in, std=n_in ** -0.5)
    if case["op"] == "int8":
        # outlier channels, as activations have them
        loud = 1.0 + 20.0 * (torch.rand(n_in, generator=g, device=dev) < 0.01)
        s["x"] = (torch.randn((T, n_in), generator=g, device=dev) * loud).to(torch.bfloat16)
        # the weights are quantised once, when they are loaded
        w = W.float()
        scale = w.abs().amax(-1) / torch.full((), 127.0, device=dev)
        s["Wq"] = torch.round(w / scale[..., None]).clamp(-127, 127).to(torch.int8)
        s["Ws"] = scale
        if not K:
            s["Wq"], s["Ws"] = s["Wq"][0], s["Ws"][0]
    else:
        s["W"] = W
        s["x"] = normal(T if case["gather"] else rows, n_in)
        if case["op"] == "gradient":
            s["dy"] = normal(rows, n_out)
    return s


def _kind(case):
    return torch.float32 if case["f32"] else torch.bfloat16


def _spread(off, n, longest):
    """Row numbers of each group [n, longest], and which of them exist."""
    at = off[:n, None].long() + torch.arange(longest, device=off.device)
    return at, at < off[1:n + 1, None]


def _padded(v, at, real):
    """v's rows by group, in 32 bits: [groups, longest, width], zeros behind a group's end."""
    return v.float()[at.clamp(max=v.shape[0] - 1)] * real[..., None]


def _place(off, n, rows):
    """Each row's group, and its place there."""
    r = torch.arange(rows, device=off.device)
    grp = torch.searchsorted(off[1:n + 1].contiguous(), r.int(), right=True)
    return grp, r - off[grp].long()


def _plain_product(s):
    case = s["case"]
    x = s["x"][s["rows"].long()] if case["gather"] else s["x"]
    off = s["off"]
    n = off.numel() - 1
    at, real = _spread(off, n, s["longest"])
    W = s["W"][s["ids"].long()] if case["gather"] else s["W"]
    y = _padded(x, at, real) @ W.float().transpose(1, 2)
    grp, place = _place(off, n, x.shape[0])
    y = y[grp, place]
    if case["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return y.to(_kind(case))


def _plain_gradient(s):
    case = s["case"]
    x = s["x"][s["rows"].long()] if case["gather"] else s["x"]
    off = s["off"]
    n = off.numel() - 1
    at, real = _spread(off, n, s["longest"])
    W = s["W"][s["ids"].long()] if case["gather"] else s["W"]
    dy = _padded(s["dy"], at, real)
    dx = dy @ W.float()
    dW = dy.transpose(1, 2) @ _padded(x, at, real)
    if case["gather"]:
        # unused places hold id 0 and no rows: adding them changes nothing
        dW = torch.zeros_like(s["W"], dtype=torch.float32).index_add_(0, s["ids"].long(), dW)
    grp, place = _place(off, n, x.shape[0])
    return {"dx": dx[grp, place].to(_kind(case)), "dW": dW}


def _plain_int8(s):
    case = s["case"]
    x = s["x"].double()
    # the scale is held in 32 bits; a row's values go to the nearest step, ties to even: in 64
    # bits, so that a value next to a border falls on its side
    scale = (x.abs().amax(-1, keepdim=True) / 127.0).float()
    q = torch.round(x / scale.double()).clamp(-127, 127).float()
    if case["topk"]:
        q, scale = q[s["rows"].long()], scale[s["rows"].long()]
        off = s["off"]
        n = off.numel() - 1
        at, real = _spread(off, n, s["longest"])
        ids = s["ids"].long()
        y = _padded(q, at, real) @ s["Wq"][ids].float().transpose(1, 2)
        grp, place = _place(off, n, q.shape[0])
        y = y[grp, place] * scale * s["Ws"][ids][grp]
    else:
        y = (q @ s["Wq"].float().T) * scale * s["Ws"]
    if case["silu"]:
        y = y / (1.0 + torch.exp(-y))
    return y.to(_kind(case))


def run(s):
    case = s["case"]
    if not own:
        return {"product": _plain_product, "gradient": _plain_gradient,
                "int8": _plain_int8}[case["op"]](s)
    import atomic_expert_routing_b200 as omni

    where = {"ids": s["ids"], "n_groups": s["n"], "rows": s["rows"]} if case["gather"] else {}
    if case["op"] == "product":
        return omni.grouped_linear(s["x"], s["W"], s["off"], silu=case["silu"],
                                   out_dtype=_kind(case), **where)
    if case["op"] == "gradient":
        g = omni.grouped_linear_backward(s["x"], s["W"], s["dy"], s["off"],
                                         out_dtype=_kind(case), **where)
        return {"dx": g["dx"], "dW": g["dW"]}
    q, scale = omni.quantize_rows(s["x"])
    return omni.quantized_linear(q, scale, s["Wq"], s["Ws"], s.get("off"), silu=case["silu"],
                                 out_dtype=_kind(case), **where)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    T, K, E, n_in, n_out = (case[k] for k in ("tokens", "topk", "E", "n_in", "n_out"))
    rows = T * K if K else T
    if rows * n_in * n_out > 1 << 39:
        return None
    act = (lambda v: v * torch.sigmoid(v)) if case["silu"] else (lambda v: v)
    if K:
        count, token = _groups(case, seed)
        ends = np.cumsum(count)
        if case["gather"]:
            x = x[torch.from_numpy(token).to(x.device)]
    else:
        count, ends = np.array([rows]), np.array([rows])
    if case["op"] == "int8":
        step = (x.abs().max(dim=1).values / 127).to(torch.float32).double()
        code = torch.round(x / step[:, None])  # |x| / step <= 127.00001: never past 127
        Wq, Ws = s["Wq"].reshape(-1, n_out, n_in), s["Ws"].reshape(-1, n_out).double()
    y = torch.empty((rows, n_out), dtype=torch.float64, device=x.device)
    dx = torch.empty((rows, n_in), dtype=torch.float64, device=x.device)
    dW = torch.zeros((E, n_out, n_in), dtype=torch.float64, device=x.device) \
        if case["op"] == "gradient" else None
    for e in range(len(count)):
        a, b = int(ends[e] - count[e]), int(ends[e])
        if a == b:
            continue
        if case["op"] == "product":
            y[a:b] = act(torch.einsum("rc,oc->ro", x[a:b], s["W"][e].double()))
        elif case["op"] == "gradient":
            up = s["dy"][a:b].double()
            dx[a:b] = torch.einsum("ro,oc->rc", up, s["W"][e].double())
            dW[e] = torch.einsum("ro,rc->oc", up, x[a:b])
        else:
            total = torch.einsum("rc,oc->ro", code[a:b], Wq[e].double())
            y[a:b] = act(torch.einsum("ro,r,o->ro", total, step[a:b], Ws[e]))
    return {"dx": dx, "dW": dW} if case["op"] == "gradient" else y


def work(case):
    T, K, E, n_in, n_out = (case[k] for k in ("tokens", "topk", "E", "n_in", "n_out"))
    rows = T * K if K else T
    # the experts that can have rows: all of them, or as many as there are rows
    live = min(E, rows)
    y = rows * n_out * (4 if case["f32"] else 2)
    x = (T if case["gather"] or not K else rows) * n_in * 2
    flops = 2.0 * rows * n_in * n_out
    if case["op"] == "product":
        return {"bytes": x + live * n_in * n_out * 2 + y, "flops": flops}
    if case["op"] == "gradient":
        dx = rows * n_in * (4 if case["f32"] else 2)
        return {"bytes": x + rows * n_out * 2 + live * n_in * n_out * 2 + dx
                + E * n_in * n_out * 4, "flops": 2 * flops}
    return {"bytes": x + live * n_in * n_out + live * n_out * 4 + y, "flops": flops}

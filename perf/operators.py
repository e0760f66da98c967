"""The operators of a text-conditioned diffusion-transformer block around the
ternary linear layer, as cases to be timed and checked:

* ``attention``: attention of image (or decoder) tokens to an encoder's states
  of another length, with a key mask and shared key-value heads, forward and
  backward;
* ``norm``: the norms before and after a block fused with its gate, its residual
  scale and the modulation of the next block, forward and backward;
* ``rope``: rotary positions with several axes (time, height, width), forward
  and its transpose.

``run`` computes a case in elementary torch operations in fp32 (``own`` false)
or by the package's entry points (``own`` true); ``exact`` computes the same in
64 bits from the definitions.  Sizes are those of the layers this repository
names: hidden 1152 with 16 heads of 72 at 256 tokens times batch 8, and hidden
3072 with 24 heads of 128 at 4096 image and 512 text tokens.
"""
import math

import torch

own = False

DEV = "cuda"
_package = None


def _tern():
    global _package
    if _package is None:
        import ternary_weight_quantized_tern_amd as package
        _package = package
    return _package


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _attention(name, direction, b, sq, sk, hq, hkv, d, mask, fused):
    return {"name": name, "op": "attention", "direction": direction, "b": b, "sq": sq, "sk": sk,
            "hq": hq, "hkv": hkv, "d": d, "mask": mask, "fused": fused}


def _norm(name, direction, b, t, c, dtype, pre, post, weights):
    return {"name": name, "op": "norm", "direction": direction, "b": b, "t": t, "c": c,
            "dtype": dtype, "pre": pre, "post": post, "weights": weights}


def _rope(name, direction, b, t, h, d, axes, layout, dtype, fused):
    return {"name": name, "op": "rope", "direction": direction, "b": b, "t": t, "h": h, "d": d,
            "axis0": axes[0], "axis1": axes[1], "axis2": axes[2], "layout": layout, "dtype": dtype,
            "fused": fused}


def listed():
    return [
        # One new token of each of four sequences over an encoder's states,
        # four query heads on each key-value head: a stream of keys and values.
        _attention("attention_one_token", "forward", 4, 1, 4608, 24, 6, 128, "none", False),
        # The small transformer's cross attention to padded captions, head width 72.
        _attention("attention_caption", "forward", 8, 256, 120, 16, 16, 72, "prefix", True),
        # Image tokens of a guidance pair to 512 padded text states.
        _attention("attention_text", "forward", 2, 4096, 512, 24, 24, 128, "prefix", True),
        # Image and text tokens together, the longest ordinary call.
        _attention("attention_joint", "forward", 1, 4608, 4608, 24, 24, 128, "none", True),
        # Training: ragged lengths, shared heads, a mask with holes and one
        # sample whose caption was dropped (nothing to attend to).
        _attention("attention_backward_ragged", "backward", 3, 1021, 333, 16, 4, 72, "holes", False),
        # Training: image tokens to padded text states.
        _attention("attention_backward_text", "backward", 2, 4096, 512, 24, 24, 128, "prefix", True),
        # A block boundary at one token of each of 8 samples: the smallest call.
        _norm("norm_eight_rows", "forward", 8, 1, 1152, "bf16", "layer", "none", False),
        # A block boundary of the large transformer, one image.
        _norm("norm_large", "forward", 1, 4608, 3072, "bf16", "layer", "none", False),
        # Training the small transformer: fp32 residual stream, RMS norms with
        # weights before and after the block.
        _norm("norm_backward_small", "backward", 8, 256, 1152, "f32", "rms", "rms", True),
        # Training the large transformer.
        _norm("norm_backward_large", "backward", 2, 2304, 3072, "bf16", "layer", "none", False),
        # The query and key heads of one image inside a fused projection.
        _rope("rope_image", "forward", 1, 4608, 48, 128, (16, 56, 56), "interleaved", "bf16", True),
        # Training on short clips: time, height and width, fp32 gradients.
        _rope("rope_video_backward", "backward", 3, 1001, 16, 72, (24, 24, 24), "halves", "f32",
              False),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], evenly over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    largest = {op: _cost([c for c in listed() if c["op"] == op])
               for op in ("attention", "norm", "rope")}
    while True:
        case = _draw(rng)
        if _cost([case]) <= largest[case["op"]]:
            return case


def _cost(cases):
    """The larger of the case's work in bytes and, at 100 operations a byte, in operations."""
    return max(max(work(c)["bytes"], work(c)["flops"] / 100.0) for c in cases)


def _draw(rng):
    op = rng.choice(["attention", "attention", "norm", "rope"])
    direction = rng.choice(["forward", "backward"])
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 6, 8, 16, 24])
        hq = hkv * rng.choice([1, 1, 1, 2, 4])
        sq = 1 if rng.random() < 0.2 else _spread(rng, 2, 4608)
        return _attention("", direction, rng.choice([1, 2, 3, 4, 8]), sq, _spread(rng, 1, 4608), hq,
                          hkv, rng.choice([40, 64, 72, 80, 96, 128]),
                          rng.choice(["none", "prefix", "holes"]), rng.random() < 0.5)
    if op == "norm":
        c = rng.choice([1152, 3072, 8 * _spread(rng, 8, 640), _spread(rng, 63, 5001)])
        return _norm("", direction, rng.choice([1, 2, 3, 8]), _spread(rng, 1, 4608), c,
                     rng.choice(["bf16", "f32"]), rng.choice(["layer", "rms"]),
                     rng.choice(["none", "layer", "rms"]), rng.random() < 0.5)
    d = rng.choice([64, 72, 96, 128])
    axes = {64: (16, 24, 24), 72: (24, 24, 24), 96: (32, 32, 32), 128: (16, 56, 56)}[d]
    if rng.random() < 0.3:
        axes = (axes[0], axes[1], axes[2] - 8)  # the last channels pass unturned
    return _rope("", direction, rng.choice([1, 2, 3, 8]), _spread(rng, 1, 4608),
                 rng.choice([1, 4, 12, 16, 24, 48]), d, axes, rng.choice(["interleaved", "halves"]),
                 rng.choice(["bf16", "f32"]), rng.random() < 0.5)


def _kept(case):
    """The keys that the mask leaves of each sample."""
    b, sk = case["b"], case["sk"]
    if case["mask"] == "none":
        return [sk] * b
    if case["mask"] == "prefix":  # from a quarter of the longest caption to all of it
        return [max(1, sk - (3 * sk * i) // (4 * b)) for i in range(b)]
    # every fourth key or so is missing, and the last sample of several keeps none
    return [0 if b > 1 and i == b - 1 else sk - sk // 4 for i in range(b)]


def work(case):
    if case["op"] == "attention":
        rows = case["b"] * case["sq"] * case["hq"]
        kept, d = sum(_kept(case)), case["d"]
        q, kv = 2 * rows * d, 2 * kept * case["hkv"] * d
        pairs = kept * case["sq"] * case["hq"]
        mask = case["b"] * case["sk"] if case["mask"] != "none" else 0
        if case["direction"] == "forward":  # q, k, v; o and its log-sum-exp
            return {"bytes": 2 * q + 2 * kv + 4 * rows + mask, "flops": 4 * pairs * d}
        # do, q, k, v, o, lse; dq and all of dk, dv
        dkv = 2 * case["b"] * case["sk"] * case["hkv"] * d
        return {"bytes": 4 * q + 2 * kv + 2 * dkv + 4 * rows + mask, "flops": 10 * pairs * d}
    if case["op"] == "norm":
        n, c = case["b"] * case["t"] * case["c"], case["b"] * case["c"]
        e = 2 if case["dtype"] == "bf16" else 4
        if case["direction"] == "forward":  # r, y; r', h; gate, scale, shift
            return {"bytes": n * (2 * e + 4) + 12 * c, "flops": 16 * n}
        # dr', dh, r', y, statistics; dr, dy; gate, scale; their gradients
        return {"bytes": n * (3 * e + 6) + 16 * case["b"] * case["t"] + 20 * c, "flops": 32 * n}
    n = case["b"] * case["t"] * case["h"] * case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 2 * n * e + 12 * case["b"] * case["t"], "flops": 3 * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _heads(g, b, s, heads, d, spread, fused):
    """One [b, s, heads[i], d] bf16 tensor for each i: views of one fused
    projection's output, or tensors of their own."""
    if not fused:
        return [(_normal(g, b, s, h, d) * spread).to(torch.bfloat16) for h in heads]
    whole = (_normal(g, b, s, sum(heads), d) * spread).to(torch.bfloat16)
    return list(whole.split(heads, dim=2))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"attention": _prepare_attention, "norm": _prepare_norm, "rope": _prepare_rope}[
        case["op"]](case, g)


def _prepare_attention(case, g):
    b, sq, sk, hq, hkv, d = (case[n] for n in ("b", "sq", "sk", "hq", "hkv", "d"))
    # Logits of standard deviation 2: attention that prefers some keys.
    spread = math.sqrt(2.0)
    if case["fused"] and sq == sk and case["mask"] == "none":
        q, k, v = _heads(g, b, sq, [hq, hkv, hkv], d, spread, True)
    else:
        (q,) = _heads(g, b, sq, [hq], d, spread, False)
        k, v = _heads(g, b, sk, [hkv, hkv], d, spread, case["fused"])
    mask = None
    if case["mask"] != "none":
        if case["mask"] == "prefix":
            order = torch.arange(sk, device=DEV).expand(b, sk)
        else:
            order = torch.rand(b, sk, generator=g, device=DEV).argsort(dim=1)
        mask = order < torch.tensor(_kept(case), device=DEV)[:, None]
    st = {"case": case, "q": q, "k": k, "v": v, "mask": mask, "scale": 1.0 / math.sqrt(d)}
    if case["direction"] == "backward":
        st["o"], st["lse"] = _attention_forward(st)
        st["do"] = _normal(g, b, sq, hq, d).to(torch.bfloat16)
    return st


def _prepare_norm(case, g):
    b, t, c = case["b"], case["t"], case["c"]
    m = b * t
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # A residual stream with some channels much larger than the others.
    large = 1.0 + 9.0 * (torch.rand(c, generator=g, device=DEV) < 0.01)
    r = (_normal(g, m, c) * large + 0.1).to(dtype)
    y = _normal(g, m, c).to(torch.bfloat16)
    modulation = _normal(g, b, 3 * c) * 0.3  # one projection of the conditioning
    shift, scale, gate = modulation.split(c, dim=1)
    weight = [1.0 + 0.1 * _normal(g, c) if case["weights"] else None for _ in range(2)]
    post = None if case["post"] == "none" else case["post"]
    st = {"case": case, "r": r, "y": y, "gate": gate, "scale": scale, "shift": shift,
          "options": {"tokens": t, "pre": case["pre"], "post": post, "pre_weight": weight[0],
                      "post_weight": weight[1] if post else None, "residual_scale": 0.75,
                      "eps": 1e-6}}
    if case["direction"] == "backward":
        st["r_out"], _, st["stats"] = _norm_forward(st)
        st["dr_out"] = _normal(g, m, c).to(dtype)
        st["dh"] = _normal(g, m, c).to(torch.bfloat16)
    return st


def _axes(case):
    return (case["axis0"], case["axis1"], case["axis2"])


def _prepare_rope(case, g):
    b, t, h, d = case["b"], case["t"], case["h"], case["d"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = _normal(g, b, t, 2 * h if case["fused"] else h, d).to(dtype)[:, :, :h]
    # Frames of a grid as near to square as its tokens fill, eight frames to a clip.
    frames = 1 if case["b"] == 1 else min(8, t)
    width = max(1, math.isqrt(-(-t // frames)))
    token = torch.arange(t, device=DEV)
    height = -(-t // (frames * width))
    grid = torch.stack([token // (width * height), token // width % height, token % width], dim=1)
    start = torch.randint(0, 32, (b, 1, 3), generator=g, device=DEV)
    return {"case": case, "x": x, "pos": (grid + start).float(), "theta": 10000.0}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    case = state["case"]
    forward = case["direction"] == "forward"
    if case["op"] == "attention":
        if not own:
            return _attention_forward(state) if forward else _attention_backward(state)
        if forward:
            return _tern().attention(state["q"], state["k"], state["v"], mask=state["mask"],
                                     scale=state["scale"])
        return _tern().attention_backward(state["do"], state["q"], state["k"], state["v"],
                                          state["o"], state["lse"], mask=state["mask"],
                                          scale=state["scale"])
    if case["op"] == "norm":
        if not own:
            return _norm_forward(state)[:2] if forward else _norm_backward(state)
        if forward:
            return _tern().residual_norm(state["r"], state["y"], gate=state["gate"],
                                         scale=state["scale"], shift=state["shift"],
                                         **state["options"])
        return _tern().residual_norm_backward(state["dr_out"], state["dh"], state["r_out"],
                                              state["y"], state["stats"], gate=state["gate"],
                                              scale=state["scale"], **state["options"])
    if not own:
        return _rope_plain(state, inverse=not forward)
    return _tern().rope(state["x"], state["pos"], _axes(case), theta=state["theta"],
                        layout=case["layout"], inverse=not forward)


def _by_group(x, hkv):
    """[b, s, h, d] -> fp32 [b, hkv, h / hkv * s, d]: the rows that share a key-value head."""
    b, s, h, d = x.shape
    return x.float().reshape(b, s, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(
        b, hkv, h // hkv * s, d)


def _by_token(x, h):
    """The inverse of _by_group."""
    b, hkv, rows, d = x.shape
    g = h // hkv
    return x.reshape(b, hkv, g, rows // g, d).permute(0, 3, 1, 2, 4).reshape(b, rows // g, h, d)


def _transposed(x):
    return x.transpose(-1, -2).contiguous()


def _attention_operands(st):
    hkv = st["k"].shape[2]
    q, k, v = (_by_group(st[n], hkv) for n in ("q", "k", "v"))
    off = None if st["mask"] is None else ~st["mask"][:, None, None, :]
    return q, k, v, off


def _attention_forward(st):
    q, k, v, off = _attention_operands(st)
    hq = st["q"].shape[2]
    s = q @ _transposed(k) * st["scale"]
    if off is not None:
        s = s.masked_fill(off, -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (s - top).exp()
    total = p.sum(dim=-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = _by_token(top + total.log(), hq)[..., 0].transpose(1, 2)
    return _by_token(o, hq).to(torch.bfloat16), lse.contiguous()


def _attention_backward(st):
    q, k, v, off = _attention_operands(st)
    hq, hkv = st["q"].shape[2], st["k"].shape[2]
    do, o = _by_group(st["do"], hkv), _by_group(st["o"], hkv)
    lse = _by_group(st["lse"].transpose(1, 2)[..., None], hkv)
    p = (q @ _transposed(k) * st["scale"] - torch.where(lse == -math.inf, 0.0, lse)).exp()
    if off is not None:
        p = p.masked_fill(off, 0.0)
    dv = _transposed(p) @ do
    ds = p * (do @ _transposed(v) - (do * o).sum(dim=-1, keepdim=True)) * st["scale"]
    dq, dk = ds @ k, _transposed(ds) @ q
    return tuple(_by_token(x, h).to(torch.bfloat16) for x, h in ((dq, hq), (dk, hkv), (dv, hkv)))


def _statistics(x, kind, eps):
    mean = x.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, ((x - mean).square().mean(dim=1, keepdim=True) + eps).rsqrt()


def _times(x, w):
    return x if w is None else x * w


def _each(x, t):
    """[b, c] -> [b * t, c]: a sample's vector for each of its tokens."""
    return x[:, None, :].expand(x.shape[0], t, x.shape[1]).reshape(-1, x.shape[1])


def _norm_forward(st):
    a = st["options"]
    z, t = st["y"].float(), a["tokens"]
    mean2 = rstd2 = torch.zeros_like(z[:, :1])
    if a["post"]:
        mean2, rstd2 = _statistics(z, a["post"], a["eps"])
        z = _times((z - mean2) * rstd2, a["post_weight"])
    r_out = (st["r"].float() + a["residual_scale"] * _each(st["gate"], t) * z).to(st["r"].dtype)
    x = r_out.float()
    mean, rstd = _statistics(x, a["pre"], a["eps"])
    n = _times((x - mean) * rstd, a["pre_weight"])
    h = n * (1.0 + _each(st["scale"], t)) + _each(st["shift"], t)
    return r_out, h.to(torch.bfloat16), torch.cat([mean, rstd, mean2, rstd2], dim=1)


def _through_norm(dn, n, rstd, kind):
    """The gradient of a norm's input from that of its normalised rows n."""
    dx = dn - n * (dn * n).mean(dim=1, keepdim=True)
    if kind == "layer":
        dx = dx - dn.mean(dim=1, keepdim=True)
    return dx * rstd


def _norm_backward(st):
    a = st["options"]
    t, c = a["tokens"], st["r_out"].shape[1]
    mean, rstd, mean2, rstd2 = st["stats"].split(1, dim=1)
    gate = a["residual_scale"] * _each(st["gate"], t)
    dh = st["dh"].float()
    n = (st["r_out"].float() - mean) * rstd
    dn = dh * (1.0 + _each(st["scale"], t))
    dr = st["dr_out"].float() + _through_norm(_times(dn, a["pre_weight"]), n, rstd, a["pre"])
    y = z = st["y"].float()
    dz = gate * dr
    dy = dz
    if a["post"]:
        y = (y - mean2) * rstd2
        z = _times(y, a["post_weight"])
        dy = _through_norm(_times(dz, a["post_weight"]), y, rstd2, a["post"])
    by_sample = lambda v: v.view(-1, t, c).sum(dim=1)  # noqa: E731
    return (dr.to(st["r_out"].dtype), dy.to(torch.bfloat16),
            by_sample(dr * z) * a["residual_scale"],
            by_sample(dh * _times(n, a["pre_weight"])), by_sample(dh),
            (dn * n).sum(dim=0) if a["pre_weight"] is not None else None,
            (dz * y).sum(dim=0) if a["post_weight"] is not None else None)


def _rope_plain(st, inverse):
    case, x = st["case"], st["x"].float()
    axes = _axes(case)
    turn = torch.cat([torch.arange(0, n, 2, device=DEV, dtype=torch.float32) / n for n in axes])
    axis = torch.repeat_interleave(torch.arange(3, device=DEV),
                                   torch.tensor(axes, device=DEV) // 2)
    angle = (st["pos"][..., axis] * torch.pow(st["theta"], -turn))[:, :, None, :]
    cos, sin = angle.cos(), (-angle if inverse else angle).sin()
    p = sum(axes) // 2
    rest = x[..., 2 * p:]
    if case["layout"] == "interleaved":
        u, v = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(-2)
    else:
        u, v = x[..., :p], x[..., p:2 * p]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    return torch.cat([turned, rest], dim=-1).to(st["x"].dtype)


# --------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# --------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    forward = case["direction"] == "forward"
    if case["op"] == "attention":
        return _exact_attention(st) if forward else _exact_attention_backward(st)
    if case["op"] == "norm":
        return _exact_norm(st) if forward else _exact_norm_backward(st)
    return _exact_rope(st, 1.0 if forward else -1.0)


def _exact_attention(st):
    q, k, v = st["q"], st["k"], st["v"]
    b, sq, hq, d = q.shape
    share = hq // k.shape[2]
    o = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, sq), -math.inf, dtype=torch.float64, device=DEV)
    for i in range(b):
        keep = slice(None) if st["mask"] is None else st["mask"][i].nonzero()[:, 0]
        for h in range(hq):
            ki, vi = k[i, keep, h // share].double(), v[i, keep, h // share].double()
            if ki.shape[0] == 0:
                continue
            logits = st["scale"] * torch.mm(q[i, :, h].double(), ki.T.contiguous())
            lse[i, h] = torch.logsumexp(logits, dim=1)
            o[i, :, h] = torch.mm(torch.softmax(logits, dim=1), vi)
    return o, lse


def _exact_attention_backward(st):
    q, k, v, do, o = (st[n].double() for n in ("q", "k", "v", "do", "o"))
    b, sq, hq, d = q.shape
    share = hq // k.shape[2]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(b):
        keep = (torch.arange(k.shape[1], device=DEV) if st["mask"] is None
                else st["mask"][i].nonzero()[:, 0])
        if keep.numel() == 0:
            continue
        for h in range(hq):
            j = h // share
            qi, ki, vi, doi = q[i, :, h], k[i, keep, j], v[i, keep, j], do[i, :, h]
            logits = st["scale"] * torch.mm(qi, ki.T.contiguous())
            p = torch.exp(logits - st["lse"][i, h].double()[:, None])
            delta = torch.einsum("sd,sd->s", doi, o[i, :, h])
            dlogits = p * (torch.mm(doi, vi.T.contiguous()) - delta[:, None])
            dq[i, :, h] = st["scale"] * torch.mm(dlogits, ki)
            dk[i, keep, j] += st["scale"] * torch.mm(dlogits.T.contiguous(), qi)
            dv[i, keep, j] += torch.mm(p.T.contiguous(), doi)
    return dq, dk, dv


def _exact_normalised(x, kind, eps):
    if kind == "layer":
        return (x - x.mean(1, True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + eps)
    return x / torch.sqrt((x * x).mean(1, True) + eps)


def _exact_norm(st):
    a, case = st["options"], st["case"]
    b, t, c = case["b"], case["t"], case["c"]
    z = st["y"].double()
    if a["post"]:
        z = _exact_normalised(z, a["post"], a["eps"])
        z = z if a["post_weight"] is None else z * a["post_weight"].double()
    gate, scale, shift = (st[n].double()[:, None] for n in ("gate", "scale", "shift"))
    r_out = st["r"].double().view(b, t, c) + a["residual_scale"] * gate * z.view(b, t, c)
    # The norm is taken of the residual stream as it is stored.
    n = _exact_normalised(r_out.to(st["r"].dtype).double().view(-1, c), a["pre"], a["eps"])
    n = n if a["pre_weight"] is None else n * a["pre_weight"].double()
    return r_out.view(-1, c), (n.view(b, t, c) * (1 + scale) + shift).view(-1, c)


def _exact_norm_backward(st):
    a, case = st["options"], st["case"]
    b, t, c = case["b"], case["t"], case["c"]
    mean, rstd, mean2, rstd2 = (st["stats"][:, i].double()[:, None] for i in range(4))
    n = (st["r_out"].double() - mean) * rstd
    wpre = 1.0 if a["pre_weight"] is None else a["pre_weight"].double()
    wpost = 1.0 if a["post_weight"] is None else a["post_weight"].double()
    dh = st["dh"].double()
    one = (1.0 + st["scale"].double()).repeat_interleave(t, dim=0)
    gate = a["residual_scale"] * st["gate"].double().repeat_interleave(t, dim=0)
    grad = dh * one * wpre
    inner = grad - n * torch.sum(grad * n, 1, True) / c
    if a["pre"] == "layer":
        inner = inner - torch.sum(grad, 1, True) / c
    dr = st["dr_out"].double() + rstd * inner
    y = st["y"].double()
    if a["post"]:
        yn = (y - mean2) * rstd2
        z, grad = yn * wpost, gate * dr * wpost
        dy = grad - yn * torch.sum(grad * yn, 1, True) / c
        if a["post"] == "layer":
            dy = dy - torch.sum(grad, 1, True) / c
        dy = dy * rstd2
    else:
        yn, z, dy = y, y, gate * dr
    total = lambda v: torch.stack([part.sum(0) for part in v.split(t)])  # noqa: E731
    return (dr, dy, a["residual_scale"] * total(dr * z), total(dh * n * wpre), total(dh),
            None if a["pre_weight"] is None else (dh * one * n).sum(0),
            None if a["post_weight"] is None else (gate * dr * yn).sum(0))


def _exact_rope(st, sign):
    x, case = st["x"].double(), st["case"]
    y = x.clone()
    half = sum(_axes(case)) // 2
    pair = 0
    for axis, n in enumerate(_axes(case)):
        for i in range(n // 2):
            angle = sign * st["pos"][:, :, axis].double() * st["theta"] ** (-2.0 * i / n)
            lo, hi = ((2 * pair, 2 * pair + 1) if case["layout"] == "interleaved"
                      else (pair, pair + half))
            c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
            y[..., lo] = c * x[..., lo] - s * x[..., hi]
            y[..., hi] = s * x[..., lo] + c * x[..., hi]
            pair += 1
    return y

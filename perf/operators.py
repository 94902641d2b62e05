"""Cases and plain forms of the operators around pair-biased attention: the
learned relative position bias by buckets with its gradient, the norms before
and after a block fused with its gate and residual scale with their gradients,
and cross attention to an encoder's states of another length with its
gradients.

``own`` selects what ``run`` does: the plain form (elementary torch operations
in 32 bits, in 64 for bucket borders and for the long sums of the table's
gradient, rounded once at the end) or the package's public calls.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token's bias row against a causal cache: latency
        dict(name="relpos_token", op="relpos", dtype="bf16", B=1, H=16, Nq=1, Nk=2047, rule="log_causal", buckets=32,
             distance=128, groups=False, base=False),
        # the bias of a 4096-token complex of several chains, added to a projected pair bias
        dict(name="relpos_pair4k", op="relpos", dtype="bf16", B=1, H=16, Nq=4096, Nk=4096, rule="clip", buckets=65,
             distance=0, groups=True, base=True),
        # a padded batch in fp32 with its own positions per sequence, queries and keys of different ragged lengths
        dict(name="relpos_ragged_f32", op="relpos", dtype="f32", B=3, H=8, Nq=777, Nk=1301, rule="log", buckets=32,
             distance=128, groups=False, base=False),
        # the table's gradient from the attention backward's dbias at the 4096-token complex
        dict(name="relpos_grad_pair4k", op="relpos_grad", dtype="bf16", B=1, H=16, Nq=4096, Nk=4096, rule="clip",
             buckets=65, distance=0, groups=True, base=False),
        # the same gradient for a padded fp32 batch
        dict(name="relpos_grad_ragged_f32", op="relpos_grad", dtype="f32", B=2, H=5, Nq=1000, Nk=651, rule="log",
             buckets=32, distance=128, groups=False, base=False),
        # a decoder step of four sequences: residual add and the next block's norm, latency
        dict(name="norm_token", op="norm", dtype="bf16", rows=4, C=768, kind="rms", post=False, gate=False,
             scale=False, pre=True),
        # the pair representation of 1024 tokens between two triangle blocks
        dict(name="norm_pair1024", op="norm", dtype="bf16", rows=1024 * 1024, C=128, kind="layer", post=True, gate=True,
             scale=True, pre=True),
        # its gradients at 512 tokens
        dict(name="norm_grad_pair512", op="norm_grad", dtype="bf16", rows=512 * 512, C=128, kind="layer", post=True,
             gate=True, scale=True, pre=True),
        # gradients of the token representation's residual scale and norm in fp32, an odd row count
        dict(name="norm_grad_single_f32", op="norm_grad", dtype="f32", rows=4099, C=384, kind="rms", post=False,
             gate=False, scale=True, pre=True),
        # one new token per sequence against the encoder states of a padded batch, grouped heads
        dict(name="cross_token", op="cross", B=16, H=16, Hkv=4, Nq=1, Nk=8192, D=64, pad=0.5, mask=False),
        # a long encoder read by 2048 decoder tokens
        dict(name="cross_long", op="cross", B=2, H=16, Hkv=16, Nq=2048, Nk=8192, D=64, pad=0.25, mask=False),
        # one training pass of a decoder layer's cross attention, masked encoder states, grouped heads
        dict(name="cross_train2k", op="cross_train", B=2, H=16, Hkv=8, Nq=2048, Nk=2048, D=64, pad=0.1, mask=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["relpos", "relpos_grad", "norm", "norm_grad", "cross", "cross_train"])
    if op in ("relpos", "relpos_grad"):
        rule = rng.choice(["clip", "log", "log_causal"])
        case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=rng.randint(1, 4), H=rng.randint(1, 16),
                    Nq=_log_int(rng, 1, 2048), Nk=_log_int(rng, 1, 2048), rule=rule,
                    buckets=2 * rng.randint(4, 64) + 1 if rule == "clip" else 2 * rng.randint(4, 32),
                    distance=0 if rule == "clip" else rng.choice([128, 300, 1024]), groups=rng.random() < 0.5,
                    base=op == "relpos" and rng.random() < 0.5)
    elif op in ("norm", "norm_grad"):
        C = rng.choice([64, 100, 128, 256, 384, 768, 1021, 2048])
        case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_log_int(rng, 1, 33554432 // C), C=C,
                    kind=rng.choice(["layer", "rms"]), post=rng.random() < 0.5, gate=rng.random() < 0.5,
                    scale=rng.random() < 0.5, pre=rng.random() < 0.8)
    else:
        Hkv = rng.choice([1, 2, 4, 8])
        case = dict(op=op, B=rng.randint(1, 4), H=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv,
                    Nq=_log_int(rng, 1, 2048) if op == "cross" else _log_int(rng, 16, 1024),
                    Nk=_log_int(rng, 1, 8192) if op == "cross" else _log_int(rng, 16, 2048), D=rng.choice([32, 64]),
                    pad=rng.choice([0.0, 0.3, 0.9]), mask=rng.random() < 0.5)
        while case["B"] * case["H"] * case["Nq"] * case["Nk"] > 2 * 16 * 2048 * 4096:
            case["Nq"] = (case["Nq"] + 1) // 2
    return case


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _key_lengths(case):
    """Valid keys of each sequence: from Nk down to (1 - pad) Nk."""
    B, Nk = case["B"], case["Nk"]
    return [Nk - int(case["pad"] * Nk * (b + 1) / B) for b in range(B)]


def _normal(g, shape, dtype, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda")
    return t.normal_(mean, std, generator=g).to(dtype)


def _positions(g, B, n):
    """Positions and chain numbers of B sequences: rising numbers with gaps,
    starting over at each chain."""
    chain = torch.randint(0, 1000, (B, n), generator=g, device="cuda").lt(4).cumsum(1)
    step = 1 + torch.randint(0, 50, (B, n), generator=g, device="cuda").eq(0).long() * 7
    pos = step.cumsum(1)
    first = torch.zeros((B, n + 1), dtype=torch.long, device="cuda")
    first.scatter_reduce_(1, chain, pos, "amin", include_self=False)
    return (pos - first.gather(1, chain)).int(), chain.int()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    op, dt = case["op"], _dtype(case)
    if op in ("relpos", "relpos_grad"):
        B, H, Nq, Nk = (case[n] for n in ("B", "H", "Nq", "Nk"))
        rows = case["buckets"] + int(case["groups"])
        k_pos, k_group = _positions(g, B, max(Nk, Nq))
        # the queries are the last of the keys' positions (a decoder's newest tokens), or all of them
        q_pos, q_group = k_pos[:, -Nq:].contiguous(), k_group[:, -Nq:].contiguous()
        k_pos, k_group = k_pos[:, :Nk].contiguous(), k_group[:, :Nk].contiguous()
        s = dict(case=case, q_pos=q_pos, k_pos=k_pos, q_group=q_group if case["groups"] else None,
                 k_group=k_group if case["groups"] else None)
        if op == "relpos":
            s["table"] = _normal(g, (rows, H), dt, 0.7)
            s["base"] = _normal(g, (B, H, Nq, Nk), dt) if case["base"] else None
        else:
            s["dbias"] = _normal(g, (B, H, Nq, Nk), dt, 0.01)
        return s
    if op in ("norm", "norm_grad"):
        rows, C = case["rows"], case["C"]
        layer = case["kind"] == "layer"

        def params(want):
            return (_normal(g, (C,), dt, 0.2, 1.0), _normal(g, (C,), dt, 0.1) if layer else None) if want else None

        s = dict(case=case, f=_normal(g, (rows, C), dt), gate=_normal(g, (rows, C), dt, 1.5) if case["gate"] else None,
                 scale=_normal(g, (C,), dt, 0.3, 0.5) if case["scale"] else None, post=params(case["post"]),
                 pre=params(case["pre"]))
        s["x" if op == "norm" else "h"] = _normal(g, (rows, C), dt, 2.0, 0.3)
        if op == "norm_grad":
            s["dh"] = _normal(g, (rows, C), dt)
            s["dy"] = _normal(g, (rows, C), dt) if case["pre"] else None
        return s
    B, H, Hkv, Nq, Nk, D = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "D"))
    order = torch.randperm(B, generator=torch.Generator().manual_seed(int(seed)))
    s = dict(case=case, q=_normal(g, (B, H, Nq, D), dt), k=_normal(g, (B, Hkv, Nk, D), dt),
             v=_normal(g, (B, Hkv, Nk, D), dt),
             k_len=torch.tensor(_key_lengths(case), dtype=torch.int32)[order].cuda(), key_mask=None)
    if case["mask"]:
        s["key_mask"] = torch.rand((B, Nk), generator=g, device="cuda").ge(0.1).to(torch.uint8)
    if op == "cross_train":
        s["dout"] = _normal(g, (B, H, Nq, D), dt)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_rows(s):
    """Table row of every (batch, query, key)."""
    case = s["case"]
    rel = s["k_pos"].long()[:, None, :] - s["q_pos"].long()[:, :, None]
    n = case["buckets"]
    if case["rule"] == "clip":
        row = rel.clamp(-(n // 2), n // 2) + n // 2
    else:
        both = case["rule"] == "log"
        n = n // 2 if both else n
        d = rel.abs() if both else (-rel).clamp(min=0)
        e = n // 2
        # floor(e + ln(d / e) / ln(distance / e) (n - e)); a quotient that is whole up to the logarithm's rounding counts as whole
        far = (d.clamp(min=1).double() / e).log() / math.log(case["distance"] / e) * (n - e)
        row = torch.where(d < e, d, (e + (far + 1e-9).floor().long()).clamp(max=n - 1))
        if both:
            row = row + (rel > 0).long() * n
    if s["q_group"] is not None:
        same = s["q_group"][:, :, None] == s["k_group"][:, None, :]
        row = torch.where(same, row, case["buckets"])
    return row


def _plain_relpos(s):
    out = s["table"].float().t()[:, _plain_rows(s)].transpose(0, 1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(s["table"].dtype).contiguous()


def _plain_relpos_grad(s):
    case = s["case"]
    rows, order = _plain_rows(s).reshape(-1).sort()
    H = case["H"]
    d = s["dbias"].transpose(0, 1).reshape(H, -1)[:, order].double()
    sums = torch.cat([d.new_zeros(H, 1), d.cumsum(1)], 1)
    n = case["buckets"] + int(case["groups"])
    ends = torch.searchsorted(rows, torch.arange(n + 1, device=rows.device))
    return (sums[:, ends[1:]] - sums[:, ends[:-1]]).t().float().contiguous()


def _unit(x, kind):
    """x brought to mean 0 (layer) and mean square 1, and what it was divided by."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r


def _affine(u, params):
    u = u * params[0].float()
    return u if params[1] is None else u + params[1].float()


def _plain_norm(s):
    kind, dt = s["case"]["kind"], s["x"].dtype
    u = s["f"].float()
    if s["post"] is not None:
        u = _affine(_unit(u, kind)[0], s["post"])
    if s["gate"] is not None:
        u = u * torch.sigmoid(s["gate"].float())
    if s["scale"] is not None:
        u = u * s["scale"].float()
    h = s["x"].float() + u
    y = _affine(_unit(h, kind)[0], s["pre"]).to(dt) if s["pre"] is not None else None
    return h.to(dt), y


def _unit_grad(du, u, r, kind):
    g = du - u * (du * u).mean(-1, keepdim=True)
    if kind == "layer":
        g = g - du.mean(-1, keepdim=True)
    return g * r


def _column_sums(x):
    return x.sum(0, dtype=torch.float64).float()


def _plain_norm_grad(s):
    kind, dt = s["case"]["kind"], s["h"].dtype
    post, pre, scale, gate = s["post"], s["pre"], s["scale"], s["gate"]
    t = s["dh"].float()
    dscale = dpost = dpost_b = dpre = dpre_b = dgate = None
    if pre is not None:
        u, r = _unit(s["h"].float(), kind)
        dy = s["dy"].float()
        dpre = _column_sums(dy * u)
        dpre_b = _column_sums(dy) if pre[1] is not None else None
        t = t + _unit_grad(dy * pre[0].float(), u, r, kind)
    f = s["f"].float()
    if post is not None:
        fu, fr = _unit(f, kind)
        a = _affine(fu, post)
    else:
        a = f
    sig = torch.sigmoid(gate.float()) if gate is not None else 1.0
    if scale is not None:
        dscale = _column_sums(t * a * sig)
    da = t if scale is None else t * scale.float()
    if gate is not None:
        dgate = (da * a * sig * (1 - sig)).to(dt)
    da = da * sig
    if post is not None:
        dpost = _column_sums(da * fu)
        dpost_b = _column_sums(da) if post[1] is not None else None
        da = _unit_grad(da * post[0].float(), fu, fr, kind)
    return t.to(dt), da.to(dt), dgate, dscale, dpost, dpost_b, dpre, dpre_b


def _plain_cross(s):
    """out, lse and what the gradients need: the probabilities [B,Hkv,G,Nq,Nk] and the fp32 inputs."""
    case = s["case"]
    B, H, Hkv, Nq, Nk, D = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "D"))
    q = s["q"].float().reshape(B, Hkv, (H // Hkv) * Nq, D)
    k, v = s["k"].float(), s["v"].float()
    keep = torch.arange(Nk, device="cuda")[None, :] < s["k_len"][:, None]
    if s["key_mask"] is not None:
        keep = keep & (s["key_mask"] != 0)
    x = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    x = x.masked_fill(~keep[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m.masked_fill(m == -math.inf, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).reshape(B, H, Nq)
    p = p / total.masked_fill(total == 0, 1.0)
    return p @ v, lse, p, q, k, v


def _plain_cross_train(s):
    case = s["case"]
    out, lse, p, q, k, v = _plain_cross(s)
    do = s["dout"].float().reshape(q.shape)
    dv = p.transpose(-1, -2) @ do
    ds = p * (do @ v.transpose(-1, -2) - (do * out).sum(-1, keepdim=True)) / math.sqrt(case["D"])
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    dt = s["q"].dtype
    return out.reshape(s["q"].shape).to(dt), lse, dq.reshape(s["q"].shape).to(dt), dk.to(dt), dv.to(dt)


def run(s):
    op = s["case"]["op"]
    if own:
        import pair_biased_attention_b200 as pba

        case = s["case"]
        if op == "relpos":
            return pba.pba_relpos_bias_forward(s["table"], s["q_pos"], s["k_pos"], case["rule"], case["distance"],
                                               q_group=s["q_group"], k_group=s["k_group"], base=s["base"])
        if op == "relpos_grad":
            return pba.pba_relpos_bias_backward(s["dbias"], s["q_pos"], s["k_pos"],
                                                case["buckets"] + int(case["groups"]), case["rule"],
                                                case["distance"], q_group=s["q_group"], k_group=s["k_group"])
        if op == "norm":
            return pba.pba_block_norm_forward(s["x"], s["f"], s["gate"], s["scale"], s["post"], s["pre"],
                                              case["kind"], EPS)
        if op == "norm_grad":
            return pba.pba_block_norm_backward(s["h"], s["dh"], s["dy"], s["f"], s["gate"], s["scale"], s["post"],
                                               s["pre"], case["kind"], EPS)
        out, lse = pba.pba_cross_attn_forward(s["q"], s["k"], s["v"], s["k_len"], s["key_mask"])
        if op == "cross":
            return out, lse
        return out, lse, *pba.pba_cross_attn_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["k_len"],
                                                      s["key_mask"])
    if op == "relpos":
        return _plain_relpos(s)
    if op == "relpos_grad":
        return _plain_relpos_grad(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "cross":
        out, lse = _plain_cross(s)[:2]
        return out.reshape(s["q"].shape).to(s["q"].dtype), lse
    return _plain_cross_train(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, size = case["op"], 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op in ("relpos", "relpos_grad"):
        n = case["B"] * case["H"] * case["Nq"] * case["Nk"]
        small = case["B"] * (case["Nq"] + case["Nk"]) * (8 if case["groups"] else 4)
        small += (case["buckets"] + int(case["groups"])) * case["H"] * 4
        return dict(bytes=n * size * (2 if case["base"] else 1) + small, flops=n)
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["C"]
        if op == "norm":  # x, f, gate read; h, y written
            return dict(bytes=n * size * (3 + case["gate"] + case["pre"]), flops=n * 12)
        # f, dh, gate, h and dy read (h only for the norm after it); dx, df, dgate written
        return dict(bytes=n * size * (4 + 2 * case["gate"] + 2 * case["pre"]), flops=n * 30)
    keys = sum(_key_lengths(case)) * (0.9 if case["mask"] else 1.0)
    B, H, Hkv, Nq, Nk, D = (case[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "D"))
    qbytes, kbytes, pairs = B * H * Nq * D * 2, 2 * Hkv * keys * D * 2, H * Nq * keys
    lse = B * H * Nq * 4
    if op == "cross":
        return dict(bytes=2 * qbytes + kbytes + lse, flops=4 * D * pairs)
    return dict(bytes=4 * qbytes + 2 * kbytes + lse, flops=14 * D * pairs)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_borders(n, distance):
    """Smallest distance of each row e+1 .. n-1 of the logarithmic rule, by whole numbers: d is at or past the border of
    row e + t where d^(n-e) >= e^(n-e-t) distance^t."""
    e = n // 2
    borders = []
    for t in range(1, n - e):
        need = e ** (n - e - t) * distance ** t
        lo, hi = e, max(distance, e + 1)
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if mid ** (n - e) >= need else (mid + 1, hi)
        borders.append(lo)
    return borders


def _exact_rows(s):
    case = s["case"]
    q, k = s["q_pos"].long().unsqueeze(2), s["k_pos"].long().unsqueeze(1)
    n = case["buckets"]
    if case["rule"] == "clip":
        r = n // 2
        row = (k - q + r).clamp(0, 2 * r)
    else:
        half = n // 2 if case["rule"] == "log" else n
        e = half // 2
        edges = torch.tensor(list(range(1, e + 1)) + _exact_borders(half, case["distance"]), device="cuda")
        back = torch.bucketize((q - k).clamp(min=0), edges, right=True)
        row = back
        if case["rule"] == "log":
            row = torch.where(k > q, half + torch.bucketize((k - q).clamp(min=0), edges, right=True), back)
    if s["q_group"] is not None:
        row = row.masked_fill(s["q_group"].unsqueeze(2) != s["k_group"].unsqueeze(1), n)
    return row


def _exact_norm(x, params, kind):
    x = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return x * params[0] + (params[1] if params[1] is not None else 0.0)


def _exact_block(x, f, gate, scale, post, pre, kind):
    u = f if post is None else _exact_norm(f, post, kind)
    u = u if gate is None else u / (1.0 + torch.exp(-gate))
    h = x + (u if scale is None else scale * u)
    return h, None if pre is None else _exact_norm(h, pre, kind)


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _grad(t):
    return None if t is None else t.grad


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "relpos":
        table, rows = s["table"].double(), _exact_rows(s)
        out = torch.stack([table[:, h][rows] for h in range(case["H"])], 1)
        return out if s["base"] is None else out + s["base"].double()
    if op == "relpos_grad":
        rows, n = _exact_rows(s), case["buckets"] + int(case["groups"])
        out = torch.zeros((n, case["H"]), dtype=torch.float64, device="cuda")
        for r in range(n):
            at = (rows == r).double()
            for h in range(case["H"]):
                out[r, h] = (s["dbias"][:, h].double() * at).sum()
        return out
    if op == "norm":
        as64 = [None if t is None else t.double() for t in (s["x"], s["f"], s["gate"], s["scale"])]
        wide = [None if p is None else tuple(None if t is None else t.double() for t in p) for p in (s["post"], s["pre"])]
        return _exact_block(*as64, *wide, case["kind"])
    if op == "norm_grad":
        f, gate, scale, h = _leaf(s["f"]), _leaf(s["gate"]), _leaf(s["scale"]), _leaf(s["h"])
        post = None if s["post"] is None else tuple(_leaf(t) for t in s["post"])
        pre = None if s["pre"] is None else tuple(_leaf(t) for t in s["pre"])
        through = s["dh"].double()
        if pre is not None:
            _exact_norm(h, pre, case["kind"]).backward(s["dy"].double())
            through = through + h.grad
        branch = _exact_block(torch.zeros_like(through), f, gate, scale, post, None, case["kind"])[0]
        branch.backward(through)
        pw, pb = post or (None, None)
        nw, nb = pre or (None, None)
        return through, f.grad, _grad(gate), _grad(scale), _grad(pw), _grad(pb), _grad(nw), _grad(nb)
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    train = op == "cross_train"
    outs, lses = [], []
    grads = [torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")] if train else []
    for b in range(B):
        keep = torch.arange(case["Nk"], device="cuda") < s["k_len"][b]
        if s["key_mask"] is not None:
            keep = keep & (s["key_mask"][b] != 0)
        at = keep.nonzero()[:, 0]
        for h in range(H):
            j = h * Hkv // H
            q, k, v = (t.double().requires_grad_(train) for t in (s["q"][b, h], s["k"][b, j, at], s["v"][b, j, at]))
            x = q @ k.t() * D ** -0.5
            if at.numel():
                lse = torch.logsumexp(x, 1)
                out = torch.exp(x - lse[:, None]) @ v
            else:
                lse, out = x.new_full((case["Nq"],), -math.inf), torch.zeros_like(q)
            if train and at.numel():
                out.backward(s["dout"][b, h].double())
                grads[0][b, h] = q.grad
                grads[1][b, j, at] += k.grad
                grads[2][b, j, at] += v.grad
            outs.append(out.detach())
            lses.append(lse.detach())
    out = torch.stack(outs).reshape(s["q"].shape)
    return (out, torch.stack(lses).reshape(B, H, case["Nq"]), *grads)

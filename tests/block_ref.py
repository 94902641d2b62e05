"""fp64 references of the operators around the attention block, from their
definitions, on the CPU: the relative position bias, the block norms and
cross attention.  Gradients come from autograd over these definitions, which
tests/test_block_ref.py compares with differences."""
from __future__ import annotations

import math

import torch


def d64(t):
    return None if t is None else t.detach().double().cpu()


# ------------------------------------------------------------------ relative position bias
def log_row(d: int, side: int, far: int) -> int:
    """Row of distance d >= 0 among the `side` rows of a logarithmic side: the
    largest e + t with d^m >= e^(m-t) far^t, in whole numbers."""
    e = side // 2
    if d < e:
        return d
    m, t = side - e, 0
    while t + 1 < m and d ** m >= e ** (m - t - 1) * far ** (t + 1):
        t += 1
    return e + t


def relpos_rows(q_pos, k_pos, rows, rule, max_distance, q_group=None, k_group=None):
    """[B, Nq, Nk] table rows; position arrays [n] or [B, n]."""
    q, k = (t.cpu().long().reshape(-1, t.shape[-1]) for t in (q_pos, k_pos))
    n = rows - (q_group is not None)
    rel = k[:, None, :] - q[:, :, None]
    if rule == "clip":
        out = rel.clamp(-(n // 2), n // 2) + n // 2
    else:
        side = n // 2 if rule == "log" else n
        known = {}

        def row(x):
            if x not in known:
                d = abs(x) if rule == "log" else max(-x, 0)
                known[x] = log_row(min(d, max_distance), side, max_distance) + (side if rule == "log" and x > 0 else 0)
            return known[x]

        out = torch.tensor([row(x) for x in rel.reshape(-1).tolist()], dtype=torch.long).reshape(rel.shape)
    if q_group is not None:
        qg, kg = (t.cpu().long().reshape(-1, t.shape[-1]) for t in (q_group, k_group))
        out = torch.where(qg[:, :, None] == kg[:, None, :], out, torch.full_like(out, n))
    return out


def relpos_bias(table, rows_index, base=None):
    out = d64(table)[rows_index].permute(0, 3, 1, 2)
    return out if base is None else out + d64(base)


def relpos_table_grad(dbias, rows_index, rows):
    """Sums of dbias per row and head, and of its magnitudes (for bounds)."""
    d = d64(dbias)
    H = d.shape[1]
    idx = rows_index.expand(d.shape[0], -1, -1).reshape(-1)
    flat = d.permute(0, 2, 3, 1).reshape(-1, H)
    out = torch.zeros(rows, H, dtype=torch.float64).index_add_(0, idx, flat)
    mag = torch.zeros(rows, H, dtype=torch.float64).index_add_(0, idx, flat.abs())
    return out, mag


# ------------------------------------------------------------------ block norms
def norm(v, params, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    v = v * params[0]
    return v if params[1] is None else v + params[1]


def block(x, f, gate, scale, post, pre, kind, eps):
    h = x
    if f is not None:
        u = f if post is None else norm(f, post, kind, eps)
        if gate is not None:
            u = u * torch.sigmoid(gate)
        if scale is not None:
            u = u * scale
        h = x + u
    return h, None if pre is None else norm(h, pre, kind, eps)


# ------------------------------------------------------------------ cross attention
def cross(q, k, v, keep, scale=None):
    """q [B,H,Nq,D], k, v [B,Hkv,Nk,D] in fp64, keep [B,Nk] bool -> out, lse.
    Rows without a key give 0 and -inf."""
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    # what a masked key holds does not matter: it is taken out before any product
    k = torch.where(keep[:, None, :, None], k, torch.zeros_like(k))
    v = torch.where(keep[:, None, :, None], v, torch.zeros_like(v))
    x = (q @ k.transpose(-1, -2)) * scale
    x = x.masked_fill(~keep[:, None, None, :], -math.inf)
    some = keep.any(-1)[:, None, None]
    lse = torch.where(some, torch.logsumexp(torch.where(some[..., None], x, torch.zeros_like(x)), -1),
                      torch.full(x.shape[:-1], -math.inf, dtype=x.dtype))
    p = torch.exp(x - torch.where(some, lse, torch.zeros_like(lse))[..., None])
    return p @ v, lse

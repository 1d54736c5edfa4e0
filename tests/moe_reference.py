"""Plain 64-bit definitions of the router's choice, the experts' FP8 products
and the few-token layer, with the error bounds that the tests hold the
kernels to.  Nothing here uses the package.

Bounds, with u = 2^-24 (half an ulp of fp32) and 2^-8 the half ulp of bf16
relative to its value:
  * A sum of n fp32 products in any order, each step rounded or truncated, is
    off by at most 2 (n + 8) u S, S the sum of the products' magnitudes
    (`gamma(n) * S`).
  * e4m3 rounding of v in units of the block scale s: at most 2^-4 |v| or
    2^-10 s, the subnormal half step.
"""
import torch

U = 2.0 ** -24


def gamma(n):
    return 2.0 * (n + 8) * U


def decode(q):
    """Values of e4m3 codes, from the format."""
    b = torch.arange(256, dtype=torch.float64)
    e, m = torch.div(b % 128, 8, rounding_mode="floor"), b % 8
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10))
    v[127] = float("nan")
    v[255] = float("nan")
    v = torch.where(b >= 128, -v, v)
    return v.to(q.device)[q.long()]


def rows64(q, scale):
    return decode(q) * scale.double().repeat_interleave(128, dim=-1)


def weights64(q, scale):
    """Codes [..., N, K] with a scale per 128 x 128 block."""
    s = scale.double().repeat_interleave(128, dim=-1).repeat_interleave(128, dim=-2)
    return decode(q) * s[..., : q.shape[-2], :]


def quantise_f32(x, reciprocal=False):
    """The FP8 cast of bf16 or float32 rows by its fp32 definition: (the codes'
    values as float64; scales float32).  448 / amax is the IEEE quotient of
    two tensors, or with `reciprocal` 1 / amax times 448, each rounded."""
    f = x.float()
    b = f.view(*f.shape[:-1], -1, 128)
    a = b.abs().amax(-1).clamp_min(1e-4)
    c = torch.full_like(a, 448.0)
    inv = (torch.ones_like(a) / a) * 448.0 if reciprocal else c / a
    v = (b * inv.unsqueeze(-1)).clamp(-448.0, 448.0)
    return v.to(torch.float8_e4m3fn).double().view(f.shape), a / c


def segments(counts, offsets, kind, capacity, rows):
    """[(expert, first, last)] of the rows that belong to an expert."""
    out = []
    for e, n in enumerate(counts.tolist()):
        a = e * capacity if kind == "masked" else int(offsets[e])
        n = min(n, capacity) if kind == "masked" else min(n, rows - a)
        if n > 0:
            out.append((e, a, a + n))
    return out


def product(a_q, a_scale, w_q, w_scale, first, last, e):
    """(y, bound of the fp32 error) of one expert's rows, in 64 bits."""
    a = rows64(a_q[first:last], a_scale[first:last])
    w = weights64(w_q[e], w_scale[e])
    y = a @ w.T
    return y, gamma(w.shape[1]) * (a.abs() @ w.abs().T)


def silu_mul(g, u, dg, du):
    """(h, bound of its fp32 error) of h = g / (1 + exp(-g)) * u for errors dg,
    du of its arguments.  |silu'| <= 1.1; expf, the add, the quotient and the
    product are off by a few ulp, the argument of exp being exact."""
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * U * (s * u).abs() + 1e-37


def flip_slack(h, dh):
    """Where an error of dh can move a value of h [m, n] across a midpoint of
    its e4m3 grid: (codes' values times the scale, bound of what the cast can
    be off).  The scale itself moves by max(dh) over the block."""
    b = h.view(*h.shape[:-1], -1, 128)
    db = dh.view(b.shape)
    a = b.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    da = db.amax(-1, keepdim=True) + 4 * U * a
    v = b * 448.0 / a
    dv = (db * 448.0 / a) + v.abs() * da / a + 4 * U * v.abs()
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 4).int())
    q = (torch.round(v / step) * step).clamp(-448.0, 448.0)
    near = (0.5 - (v / step - q / step).abs()) * step <= dv  # within dv of a midpoint
    slack = torch.where(near, step, torch.zeros_like(step)) * a / 448.0 + q.abs() * da / 448.0
    return (q * a / 448.0).view(h.shape), slack.view(h.shape), (a / 448.0).squeeze(-1), (da / 448.0).squeeze(-1)


def route(logits, k, bias=None, groups=1, groups_per_token=None, scoring="softmax", renormalize=True, scale=1.0):
    """The router's choice, one token at a time: (ids, weights in 64 bits)."""
    T, E = logits.shape
    lg = logits.float().cpu()
    key = lg if bias is None else lg + bias.float().cpu()
    ids = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=torch.float64)
    ninf = float("-inf")
    per = E // groups
    for t in range(T):
        kt = [x if x == x else ninf for x in key[t].tolist()]
        if groups_per_token is not None and groups_per_token < groups:
            best = [max(kt[g * per:(g + 1) * per]) for g in range(groups)]
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:groups_per_token]
            kt = [x if e // per in keep else ninf for e, x in enumerate(kt)]
        order = [e for e in sorted(range(E), key=lambda e: (-kt[e], e)) if kt[e] > ninf][:k]
        if not order:
            continue
        l = lg[t].double()
        chosen = l[order]
        if scoring == "softmax":
            over = chosen if renormalize else l[l == l]
            m = chosen.max() if renormalize else over.max()
            d = lambda v: torch.where(v == m, torch.zeros_like(v), v - m)  # noqa: E731
            p = torch.exp(d(chosen)) / torch.exp(d(over)).sum()
        else:
            p = 1.0 / (1.0 + torch.exp(-chosen))
            if renormalize:
                s = p.sum()
                p = p / s if s > 0 else torch.zeros_like(p)
        ids[t, :len(order)] = torch.tensor(order)
        w[t, :len(order)] = p * scale
    return ids, w

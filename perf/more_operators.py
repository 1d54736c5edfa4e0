"""Cases for measuring the BF16 products of an expert layer and their
gradients: the experts' products over a dispatched buffer (plain and gated,
with the gradients of their inputs and weights), the dense product beside them
(router logits, shared experts: bias, activation and residual in its epilogue)
with its gradients, and the gradient of the weighted combine.

`run` computes a case either in plain float32 torch operations (`own` false)
or through the package's calls (`own` true).
"""
import math

import torch

own = False


def listed():
    return [
        # second expert product of a decode batch of the small configuration:
        # 4 rows per expert, all weights read
        dict(name="product_decode", op="product", T=64, E=128, k=8, N=2048, K=1024, kind="contiguous", zipf=0.0),
        # first product of gated experts in training, pre-activations kept for
        # the backward pass; experts unevenly loaded
        dict(name="swiglu_train", op="swiglu", T=8192, E=64, k=8, N=2048, K=7168, kind="contiguous", zipf=0.25,
             keep=True),
        # gradient of the second product's input in masked buffers of 2,048
        # rows of the small configuration, odd widths
        dict(name="dgrad_masked", op="dgrad", T=2048, E=128, k=8, N=2056, K=1000, kind="masked", zipf=0.0),
        # the same through SwiGLU to the pre-activations, at the training size
        dict(name="swiglu_dgrad_train", op="swiglu_dgrad", T=8192, E=64, k=8, N=2048, K=7168, kind="contiguous",
             zipf=0.25),
        # gradient of the weights of a small batch, kept in bf16: about 19
        # ragged rows per expert
        dict(name="wgrad_small", op="wgrad", T=300, E=128, k=8, N=2048, K=1024, kind="contiguous", zipf=0.0,
             out="bfloat16"),
        # gradient of the second product's weights in training, kept in float32
        dict(name="wgrad_train", op="wgrad", T=8192, E=64, k=8, N=7168, K=2048, kind="contiguous", zipf=0.25,
             out="float32"),
        # router logits of one token: nothing but latency
        dict(name="linear_one", op="linear", M=1, N=256, K=7168, activation="none", bias="none", residual=False,
             out="float32", keep=False),
        # gate and up projection of a shared expert, eight requests decoding
        dict(name="linear_few", op="linear", M=8, N=2048, K=7168, activation="swiglu", bias="none", residual=False,
             out="bfloat16", keep=False),
        # down projection of a shared expert in prefill, added to the layer's
        # residual; a ragged batch
        dict(name="linear_shared", op="linear", M=4091, N=7168, K=2048, activation="none", bias="bfloat16",
             residual=True, out="bfloat16", keep=False),
        # backward pass of a dense layer with bias and GELU, float32 gradients
        # of the weights
        dict(name="linear_back", op="linear_back", M=4096, N=2048, K=7168, activation="gelu", bias="float32",
             out="float32"),
        # gradient of the combine for a batch of the small configuration, some
        # pairs dropped by a capacity limit
        dict(name="combine_back_small", op="combine_back", T=128, H=2048, E=128, k=8, dropped=0.05),
        # and for a training batch
        dict(name="combine_back_train", op="combine_back", T=16384, H=7168, E=256, k=8, dropped=0.0),
    ]


_WIDTHS = [8, 24, 64, 128, 136, 256, 520, 768, 1000, 1024, 1536, 2048, 2056, 4096, 5000, 7168]
_INNER = [16, 48, 128, 256, 400, 768, 1024, 1408, 2048]
_LARGEST = 2.0 * 8192 * 8 * 4096 * 7168  # products of the largest listed case, in operations


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _rows(rng, hi):
    """1 to hi, odd above 64."""
    t = _log(rng, 1, max(1, hi))
    return t if t <= 64 else (t - 1) | 1


def draw(rng):
    op = rng.choice(["product", "swiglu", "dgrad", "swiglu_dgrad", "wgrad", "linear", "linear", "linear_back",
                     "combine_back"])
    if op == "combine_back":
        H, k = rng.choice(_WIDTHS), rng.choice([1, 2, 4, 6, 8, 8])
        return dict(op=op, T=_rows(rng, min(65535, 16384 * 7168 * 8 // (H * k))), H=H, E=rng.choice([8, 60, 128, 256]), k=k,
                    dropped=rng.choice([0.0, 0.0, 0.1]))
    if op in ("linear", "linear_back"):
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
        N = rng.choice(_INNER) if act == "swiglu" else rng.choice(_WIDTHS)
        K = rng.choice(_WIDTHS)
        c = dict(op=op, M=_rows(rng, min(32767, int(_LARGEST / (8.0 * N * K)))), N=N, K=K, activation=act,
                 bias=rng.choice(["none", "float32", "bfloat16"]))
        if op == "linear_back":
            return dict(c, out=rng.choice(["float32", "bfloat16"]))
        return dict(c, residual=rng.random() < 0.4, out="bfloat16" if act == "swiglu" else rng.choice(["float32", "bfloat16"]),
                    keep=act != "none" and rng.random() < 0.4)
    E = rng.choice([1, 8, 16, 60, 64, 128])
    k = min(E, rng.choice([1, 2, 4, 6, 8, 8]))
    K = rng.choice(_WIDTHS)
    N = rng.choice(_INNER) if "swiglu" in op else rng.choice(_WIDTHS)
    T = _rows(rng, min(8191, int(_LARGEST / (4.0 * k * N * K))))
    c = dict(op=op, T=T, E=E, k=k, N=N, K=K, kind=rng.choice(["contiguous", "masked"]), zipf=rng.choice([0.0, 0.25, 0.5]))
    if op == "swiglu":
        c["keep"] = rng.random() < 0.6
    if op == "wgrad":
        c["out"] = rng.choice(["float32", "bfloat16"])
    return c


# ---- inputs -----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, amp=1.0, dtype=torch.bfloat16):
    n = math.prod(shape)
    out = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, 1 << 28):
        b = min(n, a + (1 << 28))
        out[a:b] = torch.randn(b - a, generator=g, device="cuda").mul_(amp)
    return out.view(shape)


def _zeros(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _route(T, E, k, zipf, g):
    """k distinct experts per token, popularity (e+1)^-zipf."""
    u = torch.rand(T, E, generator=g, device="cuda").clamp_min(1e-30)
    keys = -torch.log(-torch.log(u)) - zipf * torch.log(torch.arange(1, E + 1, device="cuda").float())
    return torch.topk(keys, k, dim=1).indices.to(torch.int32)


def _prepare_group(c, g):
    T, E, k, N, K, op = c["T"], c["E"], c["k"], c["N"], c["K"], c["op"]
    idx = _route(T, E, k, c["zipf"], g).view(-1)
    counts = torch.bincount(idx.long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    capacity = T if c["kind"] == "masked" else 0
    rows = E * capacity if capacity else T * k
    first = torch.arange(E, device="cuda") * capacity if capacity else offsets[:-1]
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    used = first[expert] + torch.arange(T * k, device="cuda") - offsets[:-1][expert]

    def buffer(width):
        # padding rows of a masked buffer hold whatever was there before: NaN here
        b = torch.full((rows, width), float("nan"), dtype=torch.bfloat16, device="cuda")
        b[used] = _normal((T * k, width), g)
        return b

    s = dict(counts=counts.to(torch.int32), offsets=offsets.to(torch.int32), kind=c["kind"], capacity=capacity,
             most=int(counts.max()))
    # the buffers that a training or serving loop keeps; rows that hold no pair stay as they are
    if op == "product":
        s.update(x=buffer(K), w=_normal((E, N, K), g, K ** -0.5), out=_zeros((rows, N)))
    elif op == "swiglu":
        s.update(x=buffer(K), w=_normal((E, 2 * N, K), g, K ** -0.5), out=_zeros((rows, N)),
                 z=_zeros((rows, 2 * N)) if c["keep"] else None)
    elif op == "dgrad":
        s.update(dy=buffer(N), w=_normal((E, N, K), g, K ** -0.5), out=_zeros((rows, K)))
    elif op == "swiglu_dgrad":  # the second product's weights are [E, K, N]: N inner channels
        s.update(dy=buffer(K), w=_normal((E, K, N), g, N ** -0.5), z=buffer(2 * N), out=_zeros((rows, 2 * N)))
    else:
        s.update(dy=buffer(N), x=buffer(K), out=_zeros((E, N, K), getattr(torch, c["out"])))
    return s


def _prepare_linear(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    wide = 2 * N if c["activation"] == "swiglu" else N
    s = dict(x=_normal((M, K), g), w=_normal((wide, K), g, K ** -0.5), bias=None)
    if c["bias"] != "none":
        s["bias"] = _normal((wide,), g, 0.5, getattr(torch, c["bias"]))
    if c["op"] == "linear":
        dt = getattr(torch, c["out"])
        s.update(out=_zeros((M, N), dt), z=_zeros((M, wide)) if c["keep"] else None,
                 residual=_normal((M, N), g, 1.0, dt) if c["residual"] else None)
    else:
        s.update(dy=_normal((M, N), g), z=_normal((M, wide), g) if c["activation"] != "none" else None,
                 dz=_zeros((M, wide)) if c["activation"] != "none" else None, dx=_zeros((M, K)),
                 dw=_zeros((wide, K), getattr(torch, c["out"])), dbias=_zeros((wide,), torch.float32))
    return s


def _prepare_combine(c, g):
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    idx = _route(T, E, k, 0.0, g)
    if c["dropped"] > 0:
        idx.masked_fill_(torch.rand(T, k, generator=g, device="cuda") < c["dropped"], -1)
    live = idx.view(-1) >= 0
    order = torch.sort(idx.view(-1), stable=True).indices
    order = order[live[order]]
    dst = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    dst[order] = torch.arange(order.numel(), dtype=torch.int32, device="cuda")
    return dict(dout=_normal((T, H), g), y=_normal((T * k, H), g), dst_row=dst.view(T, k),
                topk_w=torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1),
                dy=_zeros((T * k, H)), dw=_zeros((T, k), torch.float32))


def prepare(case, seed):
    g = _gen(seed)
    make = dict(linear=_prepare_linear, linear_back=_prepare_linear, combine_back=_prepare_combine)
    s = make.get(case["op"], _prepare_group)(case, g)
    s["case"] = dict(case)
    return s


# ---- the plain form ---------------------------------------------------------


def _padded(s):
    """[E, longest] rows of every expert, and which of them it has."""
    E = s["counts"].numel()
    first = torch.arange(E, device="cuda") * s["capacity"] if s["capacity"] else s["offsets"][:-1].long()
    slot = torch.arange(s["most"], device="cuda")
    return first[:, None] + slot, slot < s["counts"][:, None]


def _take(buf, row, valid):
    """Rows as float32, zero where the expert has none."""
    v = buf[row.clamp_max(buf.shape[0] - 1)].float()
    return v.masked_fill_(~valid.unsqueeze(2), 0.0)


def _place(v, row, valid, rows):
    """Back into a buffer; rows without a pair land in one past the end, which is cut off."""
    out = torch.zeros(rows + 1, v.shape[2], dtype=torch.bfloat16, device="cuda")
    out[torch.where(valid, row, rows).view(-1)] = v.to(torch.bfloat16).view(-1, v.shape[2])
    return out[:rows]


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _plain_group(s):
    op = s["case"]["op"]
    row, valid = _padded(s)
    if op == "wgrad":
        return dict(dw=torch.bmm(_take(s["dy"], row, valid).transpose(1, 2), _take(s["x"], row, valid)).to(s["out"].dtype))
    if op in ("product", "swiglu"):
        rows = s["x"].shape[0]
        y = torch.bmm(_take(s["x"], row, valid), s["w"].float().transpose(1, 2))
        if op == "product":
            return dict(out=_place(y, row, valid, rows))
        gate, up = y.chunk(2, dim=2)
        out = dict(out=_place(gate * _sigmoid(gate) * up, row, valid, rows))
        if s["z"] is not None:
            out["z"] = _place(y, row, valid, rows)
        return out
    rows = s["dy"].shape[0]
    dx = torch.bmm(_take(s["dy"], row, valid), s["w"].float())
    if op == "dgrad":
        return dict(dx=_place(dx, row, valid, rows))
    gate, up = _take(s["z"], row, valid).chunk(2, dim=2)
    p = _sigmoid(gate)
    dz = torch.cat([dx * up * p * (1.0 + gate * (1.0 - p)), dx * gate * p], dim=2)
    return dict(dz=_place(dz, row, valid, rows))


def _activate(v, kind):
    if kind == "relu":
        return v.clamp_min(0.0)
    if kind == "silu":
        return v * _sigmoid(v)
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if kind == "swiglu":
        gate, up = v.chunk(2, dim=1)
        return gate * _sigmoid(gate) * up
    return v


def _gradient(z, dy, kind):
    """Gradient of the pre-activations."""
    if kind == "relu":
        return dy * (z > 0)
    if kind == "silu":
        p = _sigmoid(z)
        return dy * p * (1.0 + z * (1.0 - p))
    if kind == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    gate, up = z.chunk(2, dim=1)
    p = _sigmoid(gate)
    return torch.cat([dy * up * p * (1.0 + gate * (1.0 - p)), dy * gate * p], dim=1)


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    v = _activate(y, c["activation"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    out = dict(out=v.to(s["out"].dtype))
    if s["z"] is not None:
        out["z"] = y.to(torch.bfloat16)
    return out


def _plain_linear_back(s):
    # the gradient of the pre-activations is an output in bf16; the products take it as it is
    c = s["case"]
    dz = s["dy"].float() if s["z"] is None else _gradient(s["z"].float(), s["dy"].float(), c["activation"])
    out = {} if s["bias"] is None else dict(dbias=dz.sum(0))
    if s["z"] is not None:
        dz = dz.to(torch.bfloat16)
        out["dz"] = dz
        dz = dz.float()
    return dict(out, dx=(dz @ s["w"].float()).to(torch.bfloat16), dw=(dz.T @ s["x"].float()).to(s["dw"].dtype))


def _plain_combine(s):
    live = s["dst_row"] >= 0
    at = s["dst_row"].long().clamp_min(0)
    dout = s["dout"].float()
    T, H = dout.shape
    k = at.shape[1]
    rows = s["y"].shape[0]
    dw = (s["y"][at.view(-1)].float().view(T, k, H) * dout[:, None, :]).sum(2)
    dy = torch.zeros(rows + 1, H, dtype=torch.bfloat16, device="cuda")
    dy[torch.where(live, at, rows).view(-1)] = (s["topk_w"].unsqueeze(2) * dout[:, None, :]).to(torch.bfloat16).view(T * k, H)
    return dict(dy=dy[:rows], dw=dw.masked_fill(~live, 0.0))


# ---- the package's calls ----------------------------------------------------


def _own(s):
    import combine_ep_layout_02_gb300 as ep
    c = s["case"]
    op = c["op"]
    if op == "linear":
        out = dict(out=ep.linear(s["x"], s["w"], s["bias"], activation=c["activation"], residual=s["residual"],
                                 out=s["out"], z=s["z"]))
        return out if s["z"] is None else dict(out, z=s["z"])
    if op == "linear_back":
        grads = ep.linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=c["activation"], dz=s["dz"], dx=s["dx"],
                                   dw=s["dw"], dbias=s["dbias"] if s["bias"] is not None else None,
                                   with_dbias=s["bias"] is not None)
        out = dict(dx=grads.dx, dw=grads.dw)
        if s["bias"] is not None:
            out["dbias"] = grads.dbias
        return out if s["z"] is None else dict(out, dz=grads.dz)
    if op == "combine_back":
        dy, dw = ep.combine_backward(s["dout"], s["y"], s["topk_w"], s["dst_row"], dy=s["dy"], dw=s["dw"])
        return dict(dy=dy, dw=dw)
    at = (s["counts"], s["offsets"], s["kind"], s["capacity"])
    if op == "product":
        return dict(out=ep.group_gemm(s["x"], s["w"], *at, out=s["out"]))
    if op == "swiglu":
        out = dict(out=ep.group_gemm_swiglu(s["x"], s["w"], *at, out=s["out"], z=s["z"]))
        return out if s["z"] is None else dict(out, z=s["z"])
    if op == "dgrad":
        return dict(dx=ep.group_gemm_dgrad(s["dy"], s["w"], *at, dx=s["out"]))
    if op == "swiglu_dgrad":
        return dict(dz=ep.group_gemm_swiglu_dgrad(s["dy"], s["w"], s["z"], *at, dz=s["out"]))
    return dict(dw=ep.group_gemm_wgrad(s["dy"], s["x"], *at, dw=s["out"]))


def run(state):
    if own:
        return _own(state)
    plain = dict(linear=_plain_linear, linear_back=_plain_linear_back, combine_back=_plain_combine)
    return plain.get(state["case"]["op"], _plain_group)(state)


# ---- what a pass cannot do without ------------------------------------------


def _active(c):
    """Experts that a uniform route reaches, on average."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = case
    op = c["op"]
    if op == "combine_back":
        pairs = c["T"] * c["k"] * (1.0 - c["dropped"])
        return dict(bytes=2.0 * c["T"] * c["H"] + 4.0 * pairs * c["H"] + 12.0 * c["T"] * c["k"], flops=3.0 * pairs * c["H"])
    N, K = c["N"], c["K"]
    size = 4.0 if c.get("out") == "float32" else 2.0
    if op in ("linear", "linear_back"):
        M, wide = c["M"], N * (2 if c["activation"] == "swiglu" else 1)
        if op == "linear":
            return dict(bytes=2.0 * M * K + 2.0 * wide * K + size * M * N * (2 if c["residual"] else 1)
                        + (2.0 * M * wide if c["keep"] else 0.0), flops=2.0 * M * wide * K)
        kept = 2.0 * 2.0 * M * wide if c["activation"] != "none" else 0.0  # z read, dz written
        return dict(bytes=2.0 * M * N + kept + 4.0 * M * K + (2.0 + size) * wide * K, flops=4.0 * M * wide * K)
    rows = c["T"] * c["k"]
    wide = N * (2 if op == "swiglu" else 1)
    if op == "wgrad":
        return dict(bytes=2.0 * rows * (N + K) + size * c["E"] * N * K, flops=2.0 * rows * N * K)
    moved = 2.0 * rows * (N + K) + 2.0 * _active(c) * wide * K
    if op == "swiglu" and c["keep"]:
        moved += 2.0 * rows * 2 * N
    if op == "swiglu_dgrad":
        moved += 2.0 * rows * 3 * N  # z read, one half of dz beside what the product itself would write
    return dict(bytes=moved, flops=2.0 * rows * wide * K)


# ---- the definition in 64 bits ----------------------------------------------


def _silu64(v):
    return v * torch.special.expit(v)


def _dsilu64(v):
    p = torch.special.expit(v)
    return p + v * p * (1.0 - p)


def _exact_group(s, c):
    E, op = c["E"], c["op"]
    N, K = c["N"], c["K"]
    counts, offsets = s["counts"].tolist(), s["offsets"].tolist()
    rows = (s["x"] if "x" in s else s["dy"]).shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "wgrad":
        out = dict(dw=torch.zeros(E, N, K, **f64))
    elif op == "dgrad":
        out = dict(dx=torch.zeros(rows, K, **f64))
    elif op == "swiglu_dgrad":
        out = dict(dz=torch.zeros(rows, 2 * N, **f64))
    else:
        out = dict(out=torch.zeros(rows, N, **f64))
        if op == "swiglu" and c["keep"]:
            out["z"] = torch.zeros(rows, 2 * N, **f64)
    for e in range(E):
        if counts[e] == 0:
            continue
        a = e * s["capacity"] if s["capacity"] else offsets[e]
        b = a + counts[e]
        if op == "wgrad":
            out["dw"][e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
            continue
        w = s["w"][e].double()
        if op == "dgrad":
            out["dx"][a:b] = s["dy"][a:b].double() @ w
        elif op == "swiglu_dgrad":
            dh = s["dy"][a:b].double() @ w
            gate, up = s["z"][a:b, :N].double(), s["z"][a:b, N:].double()
            out["dz"][a:b, :N] = dh * up * _dsilu64(gate)
            out["dz"][a:b, N:] = dh * _silu64(gate)
        else:
            y = s["x"][a:b].double() @ w.T
            out["out"][a:b] = _silu64(y[:, :N]) * y[:, N:] if op == "swiglu" else y
            if "z" in out:
                out["z"][a:b] = y
    return out


def _exact_linear(s, c):
    N = c["N"]
    z = s["x"].double() @ s["w"].double().T
    if s["bias"] is not None:
        z += s["bias"].double()
    act = c["activation"]
    if act == "relu":
        v = torch.where(z > 0, z, 0.0)
    elif act == "silu":
        v = _silu64(z)
    elif act == "gelu":
        v = z * torch.special.ndtr(z)
    elif act == "swiglu":
        v = _silu64(z[:, :N]) * z[:, N:]
    else:
        v = z
    out = dict(out=v if s["residual"] is None else v + s["residual"].double())
    return out if s["z"] is None else dict(out, z=z)


def _exact_linear_back(s, c):
    N, act = c["N"], c["activation"]
    dz = s["dy"].double()
    if act != "none":
        z = s["z"].double()
        if act == "relu":
            dz = torch.where(z > 0, dz, 0.0)
        elif act == "silu":
            dz = dz * _dsilu64(z)
        elif act == "gelu":
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        else:
            dz = torch.cat([dz * z[:, N:] * _dsilu64(z[:, :N]), dz * _silu64(z[:, :N])], dim=1)
    out = {} if s["bias"] is None else dict(dbias=dz.sum(0))
    if act != "none":
        out["dz"] = dz
        dz = dz.float().to(torch.bfloat16).double()  # the products are those of the gradient as it is kept
    return dict(out, dx=dz @ s["w"].double(), dw=dz.T @ s["x"].double())


def _exact_combine(s, c):
    T, k = c["T"], c["k"]
    dout = s["dout"].double()
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["dst_row"][:, j] >= 0).view(-1)
        r = s["dst_row"][t, j].long()
        dw[t, j] = torch.einsum("th,th->t", dout[t], s["y"][r].double())
        dy[r] = s["topk_w"][t, j].double()[:, None] * dout[t]
    return dict(dy=dy, dw=dw)


def exact(case, seed):
    # about 1 TFLOP/s in 64 bits
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    make = dict(linear=_exact_linear, linear_back=_exact_linear_back, combine_back=_exact_combine)
    return make.get(case["op"], _exact_group)(s, case)

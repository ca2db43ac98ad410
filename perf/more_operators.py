"""What is measured of the root-mean-square norm in front of the MoE layer, with its backward pass, and of the grouped
products in 8-bit floating point: one projection, and the experts' feed-forward network.

``run`` computes them either in their plain form (elementary torch operations) or, where ``own`` is
true, with the calls of ``sparse_mixture_experts_level_amd.ops``.

Formulas (T tokens of d values, w the norm's weight; rows r of group g, W_g the group's weights):

    h = x + residual, rounded to the type of x;  rstd = 1 / sqrt(mean h^2 + eps);  y = (h rstd) w
    dx = dh + rstd (dy w) - h rstd^3 / d sum(dy w h);  dw = sum_t dy h rstd
    linear: y_r = W_g x_r
    experts: y_r = D_g q(silu(G_g x_r) * (U_g x_r)),  silu(z) = z / (1 + exp(-z))

8-bit values: e4m3 codes with a scale 2^e for each block of 128 values along the contraction of a row, of 128 x 128
values of a weight matrix (gate and up rows apart); e is the least with (largest magnitude) <= 448 2^e, and the code of v
the nearest to v 2^-e (ties to the even one). q is this rounding of a row. Blocks at an end hold fewer values.
The mean of h^2 is formed in 64 bits and h rstd and its product with w are each rounded to 32, so that the codes, which
jump next to a border, are the same for everybody.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0
EPS = 1e-6


def listed():
    return [
        # the norm in front of a gpt-oss-shaped decode step of one token: one call's latency
        dict(name="norm, 1 x 2880", kind="norm", T=1, d=2880, bf16=True, residual=True),
        # a float layer of odd width, first block of a network (nothing to add)
        dict(name="norm, 5003 x 1091 float", kind="norm", T=5003, d=1091, bf16=False, residual=False),
        # a DeepSeek-V3-shaped layer's batch
        dict(name="norm, 16384 x 7168", kind="norm", T=16384, d=7168, bf16=True, residual=True),
        # training a Mixtral-shaped layer
        dict(name="norm grad, 4096 x 4096", kind="norm_backward", T=4096, d=4096, bf16=True, residual=True),
        # training a float layer of odd width
        dict(name="norm grad, 5003 x 1091 float", kind="norm_backward", T=5003, d=1091, bf16=False, residual=False),
        # a shared expert's down projection, one token
        dict(name="linear, 1 x 7168 x 2048", kind="linear", T=1, E=1, k=1, N=7168, K=2048, skew=False, tail=0),
        # 64 ragged groups, some of them empty, odd widths, rows behind the last group
        dict(name="linear, 64 ragged odd", kind="linear", T=1500, E=64, k=1, N=1000, K=1091, skew=True, tail=9),
        # a dense product of a Mixtral-shaped down projection
        dict(name="linear, 4096 x 4096 x 14336", kind="linear", T=4096, E=1, k=1, N=4096, K=14336, skew=False, tail=0),
        # a gpt-oss-shaped decode step: one token
        dict(name="experts, decode 1 token", kind="experts", T=1, E=32, k=4, d=2880, f=2880, skew=False, tail=0),
        # the same, 16 tokens
        dict(name="experts, decode 16 tokens", kind="experts", T=16, E=32, k=4, d=2880, f=2880, skew=False, tail=0),
        # one rank of eight of a DeepSeek-V3-shaped layer: 80 rows an expert
        dict(name="experts, 32 x 80 rows", kind="experts", T=320, E=32, k=8, d=7168, f=2048, skew=False, tail=0),
        # a Mixtral-shaped layer: a thousand rows an expert
        dict(name="experts, 8 x 1024 rows", kind="experts", T=4096, E=8, k=2, d=4096, f=14336, skew=False, tail=0),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(max(a, b))))))  # noqa: E731
    kind = rng.choice(["norm", "norm_backward", "linear", "linear", "experts", "experts", "experts"])
    if kind.startswith("norm"):
        d = log(16, 16384) if rng.random() < 0.5 else 64 * log(1, 256)
        return dict(kind=kind, T=log(1, 117_000_000 // d), d=d, bf16=rng.random() < 0.7, residual=rng.random() < 0.6)
    E = log(1, 64)
    k = rng.randint(1, min(E, 8))
    odd = rng.random() < 0.4
    size = lambda a, b: log(a, b) if odd else 64 * log(max(1, a // 64), b // 64)  # noqa: E731
    wide = 1_400_000_000 // E  # weights of a group at most
    if kind == "linear":
        K = size(64, min(14336, wide // 64))
        shape = dict(N=size(16 if odd else 64, min(28672, wide // K)), K=K)
        values = shape["N"] * K
    else:
        d = size(64, min(7168, wide // 192))
        shape = dict(d=d, f=size(64, min(14336, wide // (3 * d))))
        values = 3 * d * shape["f"]
    # no more work than the largest listed case, nor in the plain form, whose groups are all as long as the longest
    skew = rng.random() < 0.5
    longest = 1.0 if skew else min(1.0, 1.3 * k / E)  # share of the tokens
    T = log(1, min(8192, int(1.5e12 / (max(E * longest, k) * values))))
    return dict(kind=kind, T=T, E=E, k=k, skew=skew, tail=rng.choice([0, rng.randint(1, 40)]), **shape)


# ---------------------------------------------------------------------------------------------- inputs


def _rand(seed, tag, shape, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + tag)
    return (torch.randn(shape, generator=g, device=DEV, dtype=dtype) * scale).to(dtype)


def prepare(case, seed):
    return _prepare_norm(case, seed) if case["kind"].startswith("norm") else _prepare_grouped(case, seed)


def _prepare_norm(case, seed):
    T, d = case["T"], case["d"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    spread = torch.exp(_rand(seed, 1, (T, 1)))  # tokens' magnitudes differ
    s = dict(case=case, weight=(1 + _rand(seed, 2, (d,), 0.2)).to(dt))
    blank = lambda dtype, *shape: torch.zeros(shape, dtype=dtype, device=DEV)  # noqa: E731
    if case["kind"] == "norm":
        s["x"] = (_rand(seed, 3, (T, d)) * spread).to(dt)
        s["residual"] = (_rand(seed, 4, (T, d)) * spread).to(dt) if case["residual"] else None
        s["y"] = blank(dt, T, d)
        s["h"] = blank(dt, T, d) if case["residual"] else None
        s["rstd"] = blank(torch.float32, T)
        if own:
            from sparse_mixture_experts_level_amd import ops
            s["y8"] = blank(torch.uint8, T, ops.moe_fp8_row_bytes(d))
            s["y_scale"] = blank(torch.uint8, T, ops.moe_fp8_scale_bytes(d))
            s["values"] = blank(torch.bfloat16, T, d)
        return s
    s["h"] = (_rand(seed, 3, (T, d)) * spread).to(dt)
    s["rstd"] = _rstd(s["h"])[:, 0]
    s["dy"] = _rand(seed, 5, (T, d), 1e-2).to(dt)
    s["dh"] = _rand(seed, 6, (T, d), 1e-2).to(dt) if case["residual"] else None
    s["dx"], s["dweight"] = blank(dt, T, d), blank(torch.float32, d)
    if own:
        from sparse_mixture_experts_level_amd import ops
        s["ws"] = ops.workspace(ops.moe_rms_norm_backward_workspace_size(T, d), DEV)
    return s


def _matrices(case):
    """Name, tag, rows and columns of each weight matrix of a group."""
    if case["kind"] == "linear":
        return [("w", 1, case["N"], case["K"])]
    return [("gate_up", 1, 2 * case["f"], case["d"]), ("down", 2, case["d"], case["f"])]


def _prepare_grouped(case, seed):
    T, E, k = case["T"], case["E"], case["k"]
    K = case["K"] if case["kind"] == "linear" else case["d"]
    N = case["N"] if case["kind"] == "linear" else case["d"]
    s = dict(case=case)
    # a router's choices, sorted by group
    logits = _rand(seed, 3, (T, E))
    if case["skew"]:
        logits -= 1.1 * torch.log(torch.arange(E, device=DEV) + 1.0)
    ids = torch.topk(logits, k, dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    order = torch.argsort(ids, stable=True)
    s["group"] = ids[order]
    s["place"] = torch.arange(T * k, device=DEV) - s["offsets"].long()[s["group"]]  # of a row in its group
    s["longest"] = int(counts.max())
    # tokens that the experts' rows are gathered from; a projection's rows stand in order
    s["index"] = (order // k).to(torch.int32) if case["kind"] == "experts" else None
    rows = T * k + case["tail"]
    if s["index"] is not None:  # what stands behind the last group is no token
        s["index"] = torch.cat([s["index"], s["index"].new_full((case["tail"],), -1)])
    x = _rand(seed, 4, (T if s["index"] is not None else rows, K))
    s["x8"], s["x_scale"] = _quantize(x)
    s["y"] = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    if own:
        from sparse_mixture_experts_level_amd import ops
    for name, tag, n, kk in _matrices(case):
        w = _rand(seed, 4 + tag, (E, n, kk), kk ** -0.5, torch.bfloat16)
        if own:  # the library's own form, written once
            s[name] = ops.fp8_weights(w, swiglu=name == "gate_up")
        else:
            parts = [w[:, :n // 2], w[:, n // 2:]] if name == "gate_up" else [w]
            s[name] = [_quantize_weights(p) for p in parts]
        del w
    if own:
        s["x8"] = s["x8"].view(torch.uint8)
        exponents = s["x_scale"]  # bytes, each row's padded to what the library reads
        s["x_scale"] = torch.zeros((len(x), ops.moe_fp8_scale_bytes(K)), dtype=torch.uint8, device=DEV)
        s["x_scale"][:, :exponents.shape[1]] = (exponents + 127).to(torch.uint8)
        if case["kind"] == "linear":
            s["ws"] = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(E, rows, T, N, K), DEV)
        else:
            s["ws"] = ops.workspace(ops.moe_grouped_swiglu_gemm_fp8_workspace_size(E, rows, T, K, case["f"]), DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _exponent(largest):
    """The least e with largest <= 448 2^e (448 = 0.875 * 2^9); 0 where all is zero."""
    m, e = torch.frexp(largest)
    return torch.where(largest > 0, e - 9 + (m > 0.875), torch.zeros_like(e))


def _quantize(x):
    """Codes [rows, K up to a whole block] with zeros behind K, exponents [rows, blocks] of float rows."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x, (0, _padded(K) - K)).view(rows, -1, BLOCK)
    e = _exponent(x.abs().amax(dim=2))
    return torch.ldexp(x, -e[:, :, None]).to(torch.float8_e4m3fn).view(rows, -1), e


def _values(codes, e):
    return torch.ldexp(codes.float().view(*e.shape, BLOCK), e[..., None]).view(codes.shape)


def _quantize_weights(w):
    """Codes [G, K, N] (both up to whole blocks), exponents [G, K / 128, N / 128] of [G, N, K]."""
    G, N, K = w.shape
    w = torch.nn.functional.pad(w.float(), (0, _padded(K) - K, 0, _padded(N) - N))
    w = w.transpose(1, 2).contiguous().view(G, -1, BLOCK, _padded(N) // BLOCK, BLOCK)
    e = _exponent(w.abs().amax(dim=(2, 4)))
    return torch.ldexp(w, -e[:, :, None, :, None]).to(torch.float8_e4m3fn).view(G, _padded(K), _padded(N)), e


def _weight_values(codes, e):
    G, K, N = codes.shape
    v = codes.float().view(G, e.shape[1], BLOCK, e.shape[2], BLOCK)
    return torch.ldexp(v, e[:, :, None, :, None]).view(G, K, N)


def _rstd(h):
    mean = h.double().square().mean(dim=1, keepdim=True)
    return (1.0 / torch.sqrt(mean + EPS)).float()


def _plain_norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    rstd = _rstd(h)
    y = (h.float() * rstd) * s["weight"].float()
    values = _values(*_quantize(y))[:, :h.shape[1]].to(torch.bfloat16)
    return dict(h=h if s["residual"] is not None else None, y=y.to(h.dtype), values=values, rstd=rstd[:, 0])


def _plain_norm_backward(s):
    h, rstd = s["h"].float(), s["rstd"][:, None]
    g = s["dy"].float() * s["weight"].float()
    xhat = h * rstd
    dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dweight = (s["dy"].float() * xhat).double().sum(dim=0).float()
    return dict(dx=dx.to(s["h"].dtype), dweight=dweight)


def _plain_grouped(s):
    """Groups side by side, each as long as the longest, so that one batched product does for all."""
    case = s["case"]
    x = _values(s["x8"], s["x_scale"])
    n = s["group"].numel()
    x = x[:n] if s["index"] is None else x[s["index"][:n].long()]
    side = torch.zeros((case["E"], s["longest"], x.shape[1]), device=DEV)
    side[s["group"], s["place"]] = x
    if case["kind"] == "experts":
        gate, up = (torch.bmm(side, _weight_values(*w)) for w in s["gate_up"])
        h = gate / (1 + torch.exp(-gate)) * up
        codes, e = _quantize(h.view(-1, h.shape[2]))
        side = _values(codes, e).view(case["E"], s["longest"], -1)
    w, = s["w"] if case["kind"] == "linear" else s["down"]
    out = torch.bmm(side, _weight_values(*w))
    y = torch.zeros_like(s["y"])
    y[:n] = out[s["group"], s["place"]][:, :y.shape[1]].to(torch.bfloat16)
    return y


# ---------------------------------------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return _plain_norm(s) if kind == "norm" else _plain_norm_backward(s) if kind == "norm_backward" else _plain_grouped(s)
    from sparse_mixture_experts_level_amd import ops
    if kind == "norm":
        ops.moe_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], y=s["y"], y8=s["y8"],
                         y_scale=s["y_scale"], rstd=s["rstd"])
        ops.moe_dequantize_rows_fp8(s["y8"], s["y_scale"], s["values"])  # codes as the values they stand for
        return dict(h=s["h"], y=s["y"], values=s["values"], rstd=s["rstd"])
    if kind == "norm_backward":
        ops.moe_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], s["ws"], dh=s["dh"])
        return dict(dx=s["dx"], dweight=s["dweight"])
    rows = len(s["y"])
    if kind == "linear":
        ops.moe_grouped_linear_fp8(case["E"], rows, case["T"], case["N"], case["K"], s["x8"], s["x_scale"], s["offsets"],
                                   *s["w"], s["y"], s["ws"])
    else:
        ops.moe_grouped_swiglu_gemm_fp8(case["E"], rows, case["T"], case["d"], case["f"], s["x8"], s["x_scale"],
                                        s["offsets"], *s["gate_up"], *s["down"], s["y"], s["ws"], row_index=s["index"])
    return s["y"]


def work(case):
    kind = case["kind"]
    if kind.startswith("norm"):
        T, d, size = case["T"], case["d"], 2 if case["bf16"] else 4
        moved = (4 if case["residual"] else 2) if kind == "norm" else (4 if case["residual"] else 3)
        codes = T * d + T * (-(-d // BLOCK)) + 2 * T * d if kind == "norm" else 0  # and the values they stand for
        return dict(bytes=T * d * size * moved + codes + d * size + 4 * T, flops=12 * T * d)
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * k
    touched = E * (1 - (1 - k / E) ** T)  # of equal load
    K, N = (case["K"], case["N"]) if kind == "linear" else (case["d"], case["d"])
    values = sum(n * kk for _, _, n, kk in _matrices(case))
    read = (rows if kind == "linear" else T) * K * (1 + 1 / BLOCK)
    return dict(bytes=read + touched * values + 2 * rows * N, flops=2 * rows * values)


# ---------------------------------------------------------------------------------------------- in 64 bits


def _levels():
    """The 127 magnitudes of e4m3, and the borders between neighbours."""
    code = torch.arange(127, dtype=torch.float64, device=DEV)
    e, m = torch.floor(code / 8), code % 8
    level = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    return level, (level[1:] + level[:-1]) / 2


def _exact_held(v):
    """What the nearest codes of rows v [rows, K] stand for, block by block."""
    level, border = _levels()
    out = []
    for a in v.split(BLOCK, dim=1):
        largest = a.abs().amax(dim=1, keepdim=True)
        scale = 2.0 ** torch.ceil(torch.log2(largest.clamp(min=1e-300) / TOP))
        scale = torch.where(largest > TOP * scale, 2 * scale, torch.where(largest <= TOP / 2 * scale, scale / 2, scale))
        share = a.abs() / scale
        code = torch.searchsorted(border, share)
        on = border[code.clamp(max=125)] == share
        code = code + (on & (code % 2 == 1))
        out.append(level[code.clamp(max=126)] * torch.sign(a) * scale)
    return torch.cat(out, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h = s["x"].to(torch.float64)
        if s["residual"] is not None:  # held in the type of x
            h = (h + s["residual"].to(torch.float64)).to(s["x"].dtype).to(torch.float64)
        norm = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["d"] + EPS)
        y = h / norm * s["weight"].to(torch.float64)
        return dict(h=h if s["residual"] is not None else None, y=y, values=_exact_held(y), rstd=1 / norm[:, 0])
    if kind == "norm_backward":  # by automatic differentiation
        h = s["h"].to(torch.float64).requires_grad_()
        w = s["weight"].to(torch.float64).requires_grad_()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * w
        loss = (y * s["dy"].to(torch.float64)).sum()
        if s["dh"] is not None:
            loss = loss + (h * s["dh"].to(torch.float64)).sum()
        dx, dw = torch.autograd.grad(loss, (h, w))
        return dict(dx=dx, dweight=dw)
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    x = s["x8"].to(torch.float64) * (2.0 ** s["x_scale"].double()).repeat_interleave(BLOCK, dim=1)

    def matrix(name, g):
        def one(codes, e):
            scale = (2.0 ** e[g].double()).repeat_interleave(BLOCK, dim=0).repeat_interleave(BLOCK, dim=1)
            return codes[g].to(torch.float64) * scale
        return [one(*part) for part in s[name]]

    ends = s["offsets"].tolist()
    for g, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            continue
        rows = x[a:b] if s["index"] is None else x[s["index"][a:b].long()]
        if kind == "experts":
            gate, up = (rows @ w for w in matrix("gate_up", g))
            rows = _exact_held(torch.sigmoid(gate) * gate * up)
        w, = matrix("w" if kind == "linear" else "down", g)
        y[a:b] = (rows @ w)[:, :y.shape[1]]
    return y

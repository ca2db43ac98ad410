"""What is measured of the training operators beside the MoE layer: the balance and z losses of the
router with their gradient, the gradient norm over many tensors, and the AdamW step over many tensors
with its states in 32 or in 8 bits.

``run`` computes them either in their plain form (elementary torch operations) or, where ``own`` is
true, with the calls of ``sparse_mixture_experts_level_amd.ops``.

Formulas (T tokens, E experts, k choices a token; sequences s of the batch, each the tokens
seq_offsets[s] .. seq_offsets[s + 1] - 1 less the masked ones, N_s tokens counted, N in all, S' sequences
that count any):

    p_t = softmax(l_t), z_t = log sum exp l_t
    c_si = the counted tokens' choices of expert i, f_si = c_si / (k N_s), P_si = mean of p_ti over s
    balance = alpha E / S' sum_s sum_i f_si P_si,  z = beta / N sum_t z_t^2
    d/dl_ti = p_ti (alpha E / (S' N_s) (f_si - sum_j f_sj p_tj) + 2 beta / N z_t), f held fixed

    norm = sqrt(sum of g^2 over every tensor), scale = min(1, max_norm / (norm + 1e-6))

    g' = scale g;  m' = b1 m + (1 - b1) g';  v' = b2 v + (1 - b2) g'^2
    w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)

States in 8 bits: blocks of 256 values with one float scale, the largest magnitude of the block. m is held
as a signed code c that stands for scale c |c| / 127^2, v as a code c that stands for scale (c / 255)^4;
each takes the code whose value, for v whose value's root, is nearest, and a v above zero takes one at least.
m' and v' that are to be held so are formed and compared in 64 bits, each operation rounded by itself, so that
the choice next to a border is the same for everybody (with b1 = 0.9 a block's largest often lies halfway
between two floats).
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 256   # values that share a scale
ALIGN = 1024  # every tensor of an arena starts at a multiple of this many values
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1


def listed():
    return [
        # a training step on a few tokens: one call's latency
        dict(name="balance, 16 tokens", kind="balance", T=16, E=32, k=4, seqs=1, masked=False, tail=0),
        # a Switch-style layer, one sequence
        dict(name="balance, 8192 x 64", kind="balance", T=8192, E=64, k=1, seqs=1, masked=False, tail=0),
        # a DeepSeek-V3-shaped layer, ragged sequences with padding tokens
        dict(name="balance, 16384 x 256 ragged", kind="balance", T=16384, E=256, k=8, seqs=9, masked=True, tail=0),
        # gradient alone, as a program does whose loss is scaled after its forward pass: few experts
        dict(name="balance grad, 4096 x 8", kind="balance_backward", T=4096, E=8, k=2, seqs=1, masked=False, tail=0),
        # gradient alone: a large batch, an odd number of experts, rows behind the last sequence
        dict(name="balance grad, 60001 x 161 odd", kind="balance_backward", T=60001, E=161, k=6, seqs=33, masked=True,
             tail=77),
        # clipping over many small and odd tensors (forty layers)
        dict(name="grad norm, 120 tensors", kind="norm", layers=40, E=4, d=192, f=128, odd=True, bf16=True),
        # clipping over the gradients of one Mixtral-shaped expert
        dict(name="grad norm, 176 M", kind="norm", layers=1, E=1, d=4096, f=14336, odd=False, bf16=True),
        # the tiny float layer: latency
        dict(name="adamw, tiny float", kind="adamw", bits=32, layers=1, E=8, d=128, f=256, odd=False, bf16=False,
             master=False, clip=False),
        # many small tensors of odd sizes (forty layers), clipped
        dict(name="adamw, 120 tensors", kind="adamw", bits=32, layers=40, E=4, d=192, f=128, odd=True, bf16=True,
             master=True, clip=True),
        # one Mixtral-shaped expert
        dict(name="adamw, 176 M", kind="adamw", bits=32, layers=1, E=1, d=4096, f=14336, odd=False, bf16=True,
             master=True, clip=False),
        # small layers with states in 8 bits and no float copy of the weights
        dict(name="adamw 8 bit, 18 tensors odd", kind="adamw", bits=8, layers=6, E=5, d=320, f=448, odd=True, bf16=True,
             master=False, clip=False),
        # 16 experts of a Switch-style layer with states in 8 bits, clipped
        dict(name="adamw 8 bit, 201 M", kind="adamw", bits=8, layers=1, E=16, d=1024, f=4096, odd=False, bf16=True,
             master=True, clip=True),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    kind = rng.choice(["balance", "balance", "balance_backward", "norm", "adamw", "adamw", "adamw"])
    if kind.startswith("balance"):
        E = log(2, 512)
        T = log(1, min(65536, (1 << 23) // E))
        seqs = rng.choice([1, 1, log(1, 48)])
        return dict(kind=kind, T=T, E=E, k=rng.randint(1, min(E, 8)), seqs=seqs, masked=rng.random() < 0.5,
                    tail=rng.choice([0, 0, rng.randint(0, T // 2)]))
    layers, E = log(1, 40), log(1, 32)
    d = 8 * log(4, 512)
    f = max(1, log(1 << 16, 150_000_000) // (layers * E * 3 * d))
    shape = dict(kind=kind, layers=layers, E=E, d=d, f=f, odd=rng.random() < 0.5, bf16=rng.random() < 0.75)
    if kind == "norm":
        return shape
    return dict(shape, bits=rng.choice([32, 8]), master=shape["bf16"] and rng.random() < 0.5, clip=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------- inputs


def _sizes(case):
    """Values of each tensor: a layer's router, gate_up and down weights."""
    E, d, f = case["E"], case["d"], case["f"]
    sizes = [E * d, E * 2 * f * d, E * d * f] * case["layers"]
    return [max(1, n - 1 - i % 7) for i, n in enumerate(sizes)] if case["odd"] else sizes


def _starts(sizes):
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // ALIGN) * ALIGN
    return starts, at


def _rand(seed, n, scale, tag):
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + tag)
    return torch.randn(n, generator=g, device=DEV, dtype=torch.float32) * scale


def prepare(case, seed):
    if case["kind"].startswith("balance"):
        return _prepare_balance(case, seed)
    sizes = _sizes(case)
    starts, total = _starts(sizes)
    # which places of the arena hold a value of a tensor
    place = torch.arange(ALIGN, device=DEV)
    used = torch.cat([torch.full((-(-n // ALIGN),), ALIGN, device=DEV) for n in sizes])
    last = torch.tensor([-(-(a + n) // ALIGN) - 1 for a, n in zip(starts, sizes)], device=DEV)
    used[last] = torch.tensor([(n - 1) % ALIGN + 1 for n in sizes], device=DEV)
    live = (place < used[:, None]).reshape(-1)
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    # gradients of a wide spread from block to block, as the experts' are
    spread = torch.exp(_rand(seed, total // ALIGN, 1.5, 1)).repeat_interleave(ALIGN)
    grad = (_rand(seed, total, 1e-3, 2) * spread * live).to(dt)
    s = dict(case=case, sizes=sizes, starts=starts, grad=grad, out=torch.zeros(2, device=DEV))
    views = lambda t, per=1: [t[a // per: a // per + -(-n // per)] for a, n in zip(starts, sizes)]  # noqa: E731
    if case["kind"] == "norm":
        s["grads"] = views(grad)
        if own:
            from sparse_mixture_experts_level_amd import ops
            s["tensors"] = ops.grad_list(s["grads"])
            s["ws"] = ops.workspace(ops.moe_grad_norm_workspace_size(s["tensors"]), DEV)
        return s
    s["step"] = 500
    w = _rand(seed, total, 0.02, 3) * live
    s["param"] = w.to(dt)
    s["master"] = w if case["master"] else None
    m = _rand(seed, total, 3e-4, 4) * spread * live
    v = (_rand(seed, total, 1e-3, 5) * spread * live) ** 2
    if case["bits"] == 32:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    else:
        s["m"], s["m_scale"] = _encode_m(m.double())
        s["v"], s["v_scale"] = _encode_v(v.double())
        s["m_value"], s["v_value"] = torch.zeros(total, device=DEV), torch.zeros(total, device=DEV)
    # the routers are not decayed
    decay = [0.0 if i % 3 == 0 else DECAY for i in range(len(sizes))]
    s["decay"] = torch.cat([torch.full((-(-n // ALIGN),), 1.0 - LR * x, dtype=torch.float64, device=DEV)
                            for n, x in zip(sizes, decay)]).float()
    if own:
        from sparse_mixture_experts_level_amd import ops
        part = lambda name, per=1: views(s[name], per) if s[name] is not None else [None] * len(sizes)  # noqa: E731
        states = [dict(m=a, v=b, m_scale=c, v_scale=d, master=e) for a, b, c, d, e in zip(
            part("m"), part("v"), part("m_scale", BLOCK), part("v_scale", BLOCK), part("master"))]
        s["opt"] = ops.MoEAdamW(views(s["param"]), views(grad), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=decay,
                                max_grad_norm=1.0 if case["clip"] else None, state_bits=case["bits"], states=states,
                                step=s["step"])
        if case["bits"] == 8:
            s["values"] = views(s["m_value"]), views(s["v_value"])
    return s


def _prepare_balance(case, seed):
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + 11)
    logits = torch.randn((T, E), generator=g, device=DEV)
    logits -= 1.1 * torch.log(torch.arange(E, device=DEV) + 1.0)  # unequal load
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    s = dict(case=case, logits=logits, ids=ids, alpha=0.01, beta=0.001, offsets=None, mask=None)
    if S > 1 or case["tail"]:
        ends = T - case["tail"]
        cuts = torch.randint(0, ends + 1, (S - 1,), generator=g, device=DEV).sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), ends)]).to(torch.int32)
    if case["masked"]:
        s["mask"] = (torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8)
    s["dloss"] = torch.rand(2, generator=g, device=DEV) + 0.5
    s["counts"] = torch.zeros((S, E), dtype=torch.int32, device=DEV)
    s["seq_tokens"] = torch.zeros(S, dtype=torch.int32, device=DEV)
    s["probs"] = torch.zeros((S, E), device=DEV)
    s["losses"] = torch.zeros(2, device=DEV)
    s["dlogits"] = torch.zeros((T, E), device=DEV)
    if case["kind"] == "balance_backward":  # the forward pass's tables
        s["counts"], s["seq_tokens"] = _count(s, _members(s, *_sequences(s)))
    if own:
        from sparse_mixture_experts_level_amd import ops
        s["desc"] = ops.make_desc(T, 64, 64, E, k, None)
        s["ws"] = ops.workspace(ops.moe_balance_workspace_size(s["desc"], S), DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _sequences(s):
    """The sequence of each token, and whether the token is counted."""
    T = s["case"]["T"]
    counted = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0
    at = torch.arange(T, device=DEV)
    if s["offsets"] is None:
        return torch.zeros_like(at), counted
    seq = torch.bucketize(at, s["offsets"][1:].long(), right=True)
    counted = counted & (at >= s["offsets"][0]) & (seq < s["case"]["seqs"])
    return seq.clamp(max=s["case"]["seqs"] - 1), counted


def _members(s, seq, counted):
    """[seqs, T]: one where the token is counted in the sequence."""
    return ((seq == torch.arange(s["case"]["seqs"], device=DEV)[:, None]) & counted).double()


def _count(s, members):
    """Counts of choices [seqs, E] and of tokens [seqs] (whole numbers, exact in 64 bits)."""
    chosen = torch.zeros((s["case"]["T"], s["case"]["E"]), dtype=torch.float64, device=DEV)
    chosen.scatter_(1, s["ids"].long(), 1.0)  # a token's choices differ
    return (members @ chosen).to(torch.int32), members.sum(dim=1).to(torch.int32)


def _plain_balance(s, backward_alone):
    E, k = s["case"]["E"], s["case"]["k"]
    seq, counted = _sequences(s)
    members = None if backward_alone else _members(s, seq, counted)
    counts, tokens = (s["counts"], s["seq_tokens"]) if backward_alone else _count(s, members)
    n = tokens.clamp(min=1).float()
    live, total = (tokens > 0).sum().clamp(min=1).float(), tokens.sum().clamp(min=1).float()
    logits = torch.where(counted[:, None], s["logits"], torch.zeros_like(s["logits"]))
    top = logits.amax(dim=1, keepdim=True)
    e = torch.exp(logits - top)
    total_e = e.sum(dim=1, keepdim=True)
    p = e / total_e * counted[:, None]
    z = (top + torch.log(total_e)) * counted[:, None]
    f = counts.float() / (n * k)[:, None]
    ft = f[seq]
    scale = s["alpha"] * E / (live * n)
    up = s["dloss"] if backward_alone else torch.ones_like(s["dloss"])
    dlogits = p * (up[0] * scale[seq][:, None] * (ft - (ft * p).sum(dim=1, keepdim=True))
                   + up[1] * (2 * s["beta"]) / total * z)
    if backward_alone:
        return dlogits
    probs = members @ p.double() / n.double()[:, None]
    balance = s["alpha"] * E * (f.double() * probs).sum() / live
    zloss = s["beta"] * z.double().square().sum() / total
    return dict(counts=counts, seq_tokens=tokens, probs=probs.float(), losses=torch.stack([balance, zloss]).float(),
                dlogits=dlogits)


def _plain_norm(grad, max_norm):
    norm = grad.double().square().sum().sqrt()
    return torch.stack([norm, (max_norm / (norm + 1e-6)).clamp(max=1.0)]).float()


def _scale(a):
    """Block scales of magnitudes [blocks, BLOCK], and what a block's values are multiplied by for shares of one."""
    scale = a.amax(dim=1).float()
    scale = torch.where(scale < torch.finfo(torch.float32).tiny, torch.zeros_like(scale), scale)
    inverse = torch.where(scale > 0, 1.0 / scale.double(), torch.zeros_like(scale, dtype=torch.float64))
    return scale, inverse[:, None]


def _nearest(u):
    """The c whose square is nearest to u: c (c - 1) + 1/2 <= u < c (c + 1) + 1/2."""
    return torch.floor(torch.sqrt((u - 0.25).clamp(min=0)) + 0.5)


def _encode_m(m):
    a = m.abs().view(-1, BLOCK)
    scale, inverse = _scale(a)
    c = _nearest(a * inverse * 127.0 ** 2).view(-1)
    return torch.where(m < 0, -c, c).to(torch.int8), scale


def _encode_v(v):
    a = v.view(-1, BLOCK)
    scale, inverse = _scale(a)
    share = a * inverse
    c = torch.maximum(_nearest(share.sqrt() * 255.0 ** 2), (share > 0).double())
    return c.view(-1).to(torch.uint8), scale


def _decode_m(c, scale):
    c = c.double().view(-1, BLOCK)
    return (c * c.abs() * (scale.double() * (1.0 / 127.0 ** 2))[:, None]).view(-1)


def _decode_v(c, scale):
    square = c.double().view(-1, BLOCK).square()
    return (square * square * (scale.double() * (1.0 / 255.0 ** 4))[:, None]).view(-1)


def _plain_adamw(s):
    case, t = s["case"], s["step"] + 1
    s["step"] = t
    eight = case["bits"] == 8
    g = s["grad"].float()
    if case["clip"]:
        s["out"] = _plain_norm(s["grad"], 1.0)
        g = g.double() * s["out"][1] if eight else g * s["out"][1]
    w = s["master"] if case["master"] else s["param"].float()
    if eight:
        g = g.double()
        m = _decode_m(s["m"], s["m_scale"]) * BETA1 + g * (1.0 - BETA1)
        v = _decode_v(s["v"], s["v_scale"]) * BETA2 + (g * g) * (1.0 - BETA2)
        s["m"], s["m_scale"] = _encode_m(m)
        s["v"], s["v_scale"] = _encode_v(v)
        m, v = m.float(), v.float()
    else:
        m = s["m"] * BETA1 + g * (1.0 - BETA1)
        v = s["v"] * BETA2 + (g * g) * (1.0 - BETA2)
        s["m"], s["v"] = m, v
    u = m / (torch.sqrt(v) * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + EPS)
    w = (w.view(-1, ALIGN) * s["decay"][:, None]).view(-1) - u * (LR / (1.0 - BETA1 ** t))
    s["param"] = w.to(s["param"].dtype)
    if case["master"]:
        s["master"] = w
    if eight:
        m, v = _decode_m(s["m"], s["m_scale"]).float(), _decode_v(s["v"], s["v_scale"]).float()
    return dict(param=s["param"], master=s["master"], m=m, v=v, clip=s["out"] if case["clip"] else None)


# ---------------------------------------------------------------------------------------------- one pass


def run(s):
    kind = s["case"]["kind"]
    if not own:
        if kind.startswith("balance"):
            return _plain_balance(s, kind == "balance_backward")
        return _plain_norm(s["grad"], 1.0) if kind == "norm" else _plain_adamw(s)
    from sparse_mixture_experts_level_amd import ops
    if kind == "balance":
        ops.moe_balance_loss(s["desc"], s["logits"], s["ids"], s["alpha"], s["beta"], s["counts"], s["seq_tokens"],
                             s["probs"], s["losses"], s["ws"], token_mask=s["mask"], seq_offsets=s["offsets"],
                             dlogits=s["dlogits"])
        return dict(counts=s["counts"], seq_tokens=s["seq_tokens"], probs=s["probs"], losses=s["losses"],
                    dlogits=s["dlogits"])
    if kind == "balance_backward":
        ops.moe_balance_loss_backward(s["desc"], s["logits"], s["counts"], s["seq_tokens"], s["alpha"], s["beta"],
                                      s["dlogits"], token_mask=s["mask"], seq_offsets=s["offsets"], dloss=s["dloss"])
        return s["dlogits"]
    if kind == "norm":
        ops.moe_grad_norm(s["tensors"], 1.0, s["out"], s["ws"])
        return s["out"]
    opt = s["opt"]
    opt.step()
    clip = opt.grad_norm if s["case"]["clip"] else None
    if s["case"]["bits"] == 32:
        return dict(param=s["param"], master=s["master"], m=s["m"], v=s["v"], clip=clip)
    opt.read_states(*s["values"])  # states in 8 bits as the values they stand for
    return dict(param=s["param"], master=s["master"], m=s["m_value"], v=s["v_value"], clip=clip)


def work(case):
    if case["kind"].startswith("balance"):
        T, E, S = case["T"], case["E"], case["seqs"]
        more = T * case["k"] * 4 if case["kind"] == "balance" else 0
        tables = S * E * (8 if case["kind"] == "balance" else 4) + S * 8
        return dict(bytes=8 * T * E + more + tables + (T if case["masked"] else 0), flops=20 * T * E)
    n = sum(_sizes(case))
    value = 2 if case["bf16"] else 4
    if case["kind"] == "norm":
        return dict(bytes=n * value + 8, flops=2 * n)
    weights = value + 8 if case["master"] else 2 * value  # a float copy is read in the weights' place
    # states in 8 bits: codes and scales read and written, and the values they stand for
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
    return dict(bytes=n * (value + weights + states), flops=n * (20 if case["bits"] == 32 else 60))


# ---------------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("balance"):
        return _exact_balance(s, case["kind"] == "balance_backward")
    g = s["grad"].to(torch.float64)
    norm = torch.linalg.vector_norm(g)
    clip = torch.stack([norm, torch.minimum(torch.ones_like(norm), 1.0 / (norm + 1e-6))])
    if case["kind"] == "norm":
        return clip
    if case["clip"]:
        g = g * clip[1].float()  # held as a float
    t = s["step"] + 1
    old = s["master"] if case["master"] else s["param"]
    if case["bits"] == 8:  # whole numbers times the share of the scale that one of them stands for
        one = (s["m_scale"].to(torch.float64) * (1 / 127 ** 2)).repeat_interleave(BLOCK)
        m = one * (s["m"].long() * s["m"].long().abs()).to(torch.float64)
        one = (s["v_scale"].to(torch.float64) * (1 / 255 ** 4)).repeat_interleave(BLOCK)
        v = one * (s["v"].long() ** 4).to(torch.float64)
    else:
        m, v = s["m"].to(torch.float64), s["v"].to(torch.float64)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    step = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    decay = [0.0 if i % 3 == 0 else DECAY for i in range(len(s["sizes"]))]
    lengths = torch.tensor([-(-n // ALIGN) * ALIGN for n in s["sizes"]], device=DEV)
    rate = torch.repeat_interleave(torch.tensor(decay, dtype=torch.float64, device=DEV), lengths)
    w = old.to(torch.float64) - LR * (step + rate * old.to(torch.float64))
    if case["bits"] == 8:
        m, v = _exact_held(m, 127, 1), _exact_held(v, 255, 2)
    return dict(param=w, master=w if case["master"] else None, m=m, v=v, clip=clip if case["clip"] else None)


def _exact_held(x, top, root):
    """The values that stand for x in 8 bits: the block's level whose `root`-th root is nearest to x's."""
    level = (torch.arange(top + 1, dtype=torch.float64, device=DEV) / top) ** 2
    border = ((level[1:] + level[:-1]) / 2) ** root
    a = x.abs().view(-1, BLOCK)
    largest = a.amax(dim=1, keepdim=True).float().double()  # held as a float
    share = a / torch.where(largest > 0, largest, torch.ones_like(largest))
    code = torch.searchsorted(border, share, right=True)
    if root == 2:
        code = torch.where(share > 0, code.clamp(min=1), code)
    return (level[code] ** root * largest).view(-1) * torch.sign(x)


def _exact_balance(s, backward_alone):
    """Sequence by sequence in 64 bits, the gradient by automatic differentiation."""
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    ends = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    logits = s["logits"].to(torch.float64).requires_grad_()
    balance, z, counts, tokens, probs = [], [], [], [], []
    for a, b in zip(ends, ends[1:]):
        keep = torch.arange(a, b, device=DEV)
        keep = keep if s["mask"] is None else keep[s["mask"][a:b] != 0]
        chosen = torch.bincount(s["ids"][keep].reshape(-1).long(), minlength=E)
        counts.append(chosen)
        tokens.append(len(keep))
        if not len(keep):
            probs.append(torch.zeros(E, dtype=torch.float64, device=DEV))
            continue
        mean = torch.softmax(logits[keep], dim=1).mean(dim=0)
        probs.append(mean)
        balance.append(E * (mean * chosen / (len(keep) * k)).sum())
        z.append(torch.logsumexp(logits[keep], dim=1).square().sum())
    if not z:
        losses = torch.zeros(2, dtype=torch.float64, device=DEV)
        grad = torch.zeros_like(logits)
    else:
        losses = torch.stack([s["alpha"] * sum(balance) / len(balance), s["beta"] * sum(z) / sum(tokens)])
        up = s["dloss"].to(torch.float64) if backward_alone else torch.ones_like(losses)
        grad, = torch.autograd.grad((losses * up).sum(), logits)
    if backward_alone:
        return grad
    return dict(counts=torch.stack(counts).to(torch.int32), seq_tokens=torch.tensor(tokens, dtype=torch.int32),
                probs=torch.stack(probs).detach(), losses=losses.detach(), dlogits=grad)

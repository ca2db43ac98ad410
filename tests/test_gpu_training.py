"""GPU parity of the training operators (balance loss with its gradient, gradient norm, AdamW with
states in 32 or 8 bits) against the 64-bit oracle, and of the whole training step.

Tolerances, u = 2^-24 (half a step of a float) and B = 2^-8 (of bf16), derived as the errors of the
float operations on the way:
  * balance: exp(l - m) of a float argument is off by (R + 4) 2u relative, R the largest |l - m| of
    the case's finite logits (the argument's rounding, times log2 e, and the exponential's own last place);
    the sum over E adds at most 11 roundings and the division 2: p is off by K u with K = 2 R + 24.  Means over
    tokens add the roundings of a lane's and a block's sums, at most 32.  A gradient p (a (f - d) + b z) is
    off by (K + 16) u of p (a (f + d) + b (|z| + 1)) (z is off by that share of |z| + 1: the logarithm of a sum
    next to one is off absolutely).
  * AdamW: m' and v' are sums of two products of which each factor and product is rounded: 4 u of
    |b1 m| + |(1 - b1) g|, 6 u of v'.  The step u = m' / (sqrt(v') c + eps) adds v's half, the root, c,
    the sum and the division: 16 u of (|b1 m| + |(1 - b1) g|) / denominator; w' two roundings of w more.
    A bf16 parameter without a float copy adds B of |w'|; with one it is the copy's rounding, exactly.
  * 8-bit states: codes and scales equal the oracle's, which tries every level in 64 bits.
  * the norm: 64-bit sums, rounded once: 2 u.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_mixture_experts_level_amd import workloads as wl
from tests.moe_testlib import BF16_TOL, HostExperts, row_rel_err, say, to_np

pytestmark = pytest.mark.gpu
ops = pytest.importorskip("sparse_mixture_experts_level_amd.ops")
DEV = "cuda"
U, B = 2.0 ** -24, 2.0 ** -8


# ------------------------------------------------------------------------------ balance loss

GUARD = 64  # values behind every output that have to stay as they were


class Outputs:
    """The balance loss's output tensors, each at the front of a buffer with a guard behind it."""

    def __init__(self, T, E, S):
        self.whole = {}
        for name, shape, dt in [("counts", (S, E), torch.int32), ("seq_tokens", (S,), torch.int32),
                                ("mean_probs", (S, E), torch.float32), ("losses", (2,), torch.float32),
                                ("dlogits", (T, E), torch.float32)]:
            n = math.prod(shape)
            self.whole[name] = torch.full((n + GUARD,), 7, dtype=dt, device=DEV)
            setattr(self, name, self.whole[name][:n].view(shape))

    def check_guards(self):
        for name, t in self.whole.items():
            assert torch.all(t[-GUARD:] == 7), name


def _balance(logits, ids, alpha=0.3, z=0.05, mask=None, off=None, ws_fill=255):
    T, E = logits.shape
    S = 1 if off is None else len(off) - 1
    dev = lambda a, dt: None if a is None else torch.as_tensor(np.ascontiguousarray(a)).to(dt).to(DEV)  # noqa: E731
    lg, ig = dev(logits, torch.float32), dev(ids, torch.int32)
    mg, og = dev(mask, torch.uint8), dev(off, torch.int32)
    desc = ops.make_desc(T, 64, 64, E, ids.shape[1], None)
    out = Outputs(T, E, S)
    need = ops.moe_balance_workspace_size(desc, S)
    ws = torch.full((need + GUARD,), ws_fill, dtype=torch.uint8, device=DEV)
    ops.moe_balance_loss(desc, lg, ig, alpha, z, out.counts, out.seq_tokens, out.mean_probs, out.losses, ws[:need],
                         token_mask=mg, seq_offsets=og, dlogits=out.dlogits)
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == ws_fill)
    out.check_guards()
    return desc, lg, ig, mg, og, out


def _gradient_bound(ref, logits, alpha, z, mask, off, dloss=(1.0, 1.0)):
    """(K + 16) u of p (a (f + d) + b (|z| + 1)), from the oracle's gradients of the positive parts."""
    T, E = logits.shape
    fin = np.where(np.isfinite(logits), logits, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            R = np.nan_to_num(np.nanmax(np.nanmax(fin, 1) - np.nanmin(fin, 1))) if np.isfinite(fin).any() else 0.0
    K = 2 * min(R, 104.0) + 24  # below exp(-104) a float is zero
    bound = np.zeros((T, E))
    tokens = ref["seq_tokens"]
    live, total = max(int((tokens > 0).sum()), 1), max(int(tokens.sum()), 1)
    offs = [0, T] if off is None else off
    for s in range(len(offs) - 1):
        n = max(int(tokens[s]), 1)
        k = ref["k"]
        f = ref["counts"][s] / (k * n)
        for t in range(offs[s], offs[s + 1]):
            if mask is not None and not mask[t]:
                continue
            top = logits[t].max()
            if not np.isfinite(top):
                continue
            e = np.exp(logits[t] - top)
            p, lse = e / e.sum(), top + np.log(e.sum())
            bound[t] = p * (abs(dloss[0]) * alpha * E / (live * n) * (f + (f * p).sum())
                            + abs(dloss[1]) * 2 * z / total * (abs(lse) + 1))
    return (K + 16) * U * bound + 1e-37, K


def _check_balance(logits, ids, alpha=0.3, z=0.05, mask=None, off=None):
    logits = np.asarray(logits, dtype=np.float32).astype(np.float64)
    desc, lg, ig, mg, og, out = _balance(logits, ids, alpha, z, mask, off)
    E = logits.shape[1]
    with np.errstate(all="ignore"):
        ref = oracle.balance_loss(logits, ids, E, alpha, z, mask, off)
    ref["k"] = ids.shape[1]
    assert np.array_equal(to_np(out.counts), ref["counts"])
    assert np.array_equal(to_np(out.seq_tokens), ref["seq_tokens"])
    with np.errstate(all="ignore"):
        bound, K = _gradient_bound(ref, logits, alpha, z, mask, off)
    err = np.abs(to_np(out.dlogits) - ref["dlogits"])
    assert np.all(err <= bound), (err.max(), (err / bound).max())
    assert np.all(np.abs(to_np(out.mean_probs) - ref["mean_probs"]) <= (K + 32) * U * ref["mean_probs"] + 1e-37)
    losses = to_np(out.losses)
    assert abs(losses[0] - ref["losses"][0]) <= (K + 34) * U * abs(ref["losses"][0])
    # z^2 is off by 2 |z| K u (|z| + 1); sum over tokens of |z| (|z| + 1) from the loss: at most 2 z^2 + 1
    assert abs(losses[1] - ref["losses"][1]) <= 2 * (K + 34) * U * (2 * abs(ref["losses"][1]) + z)
    # the gradient alone, bit for bit the same; and weighted by upstream gradients
    alone = torch.full((logits.shape[0] * E + GUARD,), 7.0, device=DEV)
    d2 = alone[:logits.shape[0] * E].view(logits.shape)
    args = dict(token_mask=mg, seq_offsets=og)
    ops.moe_balance_loss_backward(desc, lg, out.counts, out.seq_tokens, alpha, z, d2, **args)
    assert torch.equal(d2, out.dlogits) and torch.all(alone[-GUARD:] == 7)
    up = (-1.5, 0.25)
    ops.moe_balance_loss_backward(desc, lg, out.counts, out.seq_tokens, alpha, z, d2,
                                  dloss=torch.tensor(up, device=DEV), **args)
    with np.errstate(all="ignore"):
        ref2 = oracle.balance_loss(logits, ids, E, alpha, z, mask, off, up)
        bound, _ = _gradient_bound(ref, logits, alpha, z, mask, off, up)
    assert np.all(np.abs(to_np(d2) - ref2["dlogits"]) <= bound)
    return out


def _draw(seed, T, E, k, spread=2.0):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * spread).astype(np.float32)
    return rng, l, np.argsort(-l, axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (2, 2, 2), (3, 3, 1), (16, 32, 4), (63, 5, 5), (64, 64, 1), (65, 7, 3), (257, 8, 2),
    (100, 33, 6), (130, 65, 2), (129, 128, 8), (200, 130, 4), (300, 256, 8), (77, 257, 3), (40, 512, 8),
    (33, 513, 2), (20, 1000, 8), (10, 1024, 16), (5000, 16, 2), (4097, 12, 3),
])
def test_balance_loss_one_sequence(T, E, k):
    say(f"balance T={T} E={E} k={k}")
    _, l, ids = _draw(T + E, T, E, k)
    _check_balance(l, ids)


@pytest.mark.parametrize("T,E,k,off,masked", [
    (10, 4, 2, [0, 10], False),
    (100, 8, 2, [0, 1, 2, 40, 100], False),
    (300, 33, 4, [0, 0, 100, 100, 299, 300, 300], True),   # empty sequences
    (500, 64, 2, [17, 50, 320, 450], True),                # rows before the first and behind the last
    (90, 256, 8, [5, 5, 5], True),                         # no rows at all
    (1500, 24, 3, list(range(0, 1501, 10)), True),         # 150 sequences: more than a wavefront
    (700, 6, 2, [0, 699], False),                          # one sequence and one row behind it
    (2600, 40, 2, [1, 1200, 2500], True),                  # chunks end inside sequences
    (9000, 8, 4, [0, 4000, 9000], True),                   # counted apart, few experts
    (12000, 160, 8, list(range(0, 12001, 200)), False),    # 60 sequences, counts added up by each block
    (7000, 700, 6, [0, 10, 6990], True),                   # ... and through the tables
    (4200, 4, 1, list(range(0, 4201, 2)), True),           # 2100 sequences of two tokens
])
def test_balance_loss_sequences(T, E, k, off, masked):
    say(f"balance sequences T={T} E={E} k={k} S={len(off) - 1}")
    rng, l, ids = _draw(T * 3 + E, T, E, k)
    mask = (rng.random(T) < 0.6).astype(np.uint8) if masked else None
    out = _check_balance(l, ids, mask=mask, off=off)
    if off[-1] == off[0]:
        assert not to_np(out.losses).any() and not to_np(out.dlogits).any()


@pytest.mark.parametrize("E", [6, 7, 9, 11, 12, 13, 15, 17, 20, 23, 25, 31, 36, 47, 49, 63, 68, 95, 97, 127, 132, 191, 193,
                               255, 260, 383, 385, 511, 516, 639, 641, 767, 768, 769, 772, 1023])
def test_balance_loss_at_the_ends_of_each_way_to_hold_a_row(E):
    """Fewest and most experts of each number of lanes and values a row is held in."""
    say(f"balance E={E}")
    rng, l, ids = _draw(72 + E, 70, E, min(E, 5))
    _check_balance(l, ids, mask=rng.random(70) < 0.8, off=[3, 40, 66])


def test_balance_debug_library_rejects_offsets_that_are_none():
    """libmoe_debug.so checks the offsets on the host before any launch, in both directions."""
    say("balance offsets refused by the debug library")
    T, E, k, S = 50, 8, 2, 3
    _, l, ids = _draw(73, T, E, k)
    desc, lg, ig, _, _, out = _balance(l, ids, off=[0, 20, 20, 50])
    D = ops.debug_lib()
    ws = ops.workspace(ops.moe_balance_workspace_size(desc, S))
    kept = {n: w.clone() for n, w in out.whole.items()}
    for off, ok in [([0, 20, 20, 50], True), ([4, 20, 21, 47], True), ([0, 21, 20, 50], False), ([-1, 20, 20, 50], False),
                    ([0, 20, 20, 51], False)]:
        og = torch.tensor(off, dtype=torch.int32, device=DEV)
        fwd = D.moe_balance_loss(ops.ctypes.byref(desc), lg.data_ptr(), ig.data_ptr(), None, og.data_ptr(), S, 0.3, 0.05,
                                 out.counts.data_ptr(), out.seq_tokens.data_ptr(), out.mean_probs.data_ptr(),
                                 out.losses.data_ptr(), out.dlogits.data_ptr(), ws.data_ptr(), ws.numel(), None)
        torch.cuda.synchronize()
        bwd = D.moe_balance_loss_backward(ops.ctypes.byref(desc), lg.data_ptr(), None, og.data_ptr(), S,
                                          out.counts.data_ptr(), out.seq_tokens.data_ptr(), 0.3, 0.05, None,
                                          out.dlogits.data_ptr(), None)
        torch.cuda.synchronize()
        if ok:
            assert fwd == bwd == ops.MOE_OK
            kept = {n: w.clone() for n, w in out.whole.items()}
        else:
            assert fwd == bwd == ops.MOE_ERR_INVALID and b"seq_offsets" in D.moe_last_error()
            assert all(torch.equal(w, kept[n]) for n, w in out.whole.items())


def test_balance_loss_masked_rows_may_hold_anything():
    say("balance masked rows with NaN and infinities")
    rng, l, ids = _draw(5, 200, 20, 3)
    mask = (rng.random(200) < 0.5).astype(np.uint8)
    l[mask == 0] = rng.choice(np.array([np.nan, np.inf, -np.inf, np.finfo(np.float32).min], dtype=np.float32),
                              size=((mask == 0).sum(), 20))
    ids = np.where(mask[:, None] == 0, 10 ** 6, ids)
    clean = np.where(mask[:, None] == 0, 0, l)
    out = _check_balance(np.where(mask[:, None] == 0, 0.0, l), ids, mask=mask)
    _, _, _, _, _, dirty = _balance(l, ids, mask=mask)
    for name in out.whole:
        assert torch.equal(out.whole[name], dirty.whole[name]), name
    assert np.isfinite(clean).all()
    # every token masked: nothing is counted
    _, _, _, _, _, none = _balance(l, ids, mask=np.zeros(200, dtype=np.uint8))
    assert not none.losses.any() and not none.dlogits.any() and not none.mean_probs.any() and not none.counts.any()


def test_balance_loss_infinite_logits():
    """-inf is an expert with probability 0, a row of them has no probabilities; the type's lowest value is
    finite; NaN and +inf of a counted token show up."""
    say("balance with -inf logits")
    rng, l, ids = _draw(6, 70, 12, 2)
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[3] = -np.inf
    l[10] = np.finfo(np.float32).min
    l[11, 1:] = np.finfo(np.float32).min
    # row 10's z is 3.4e38, whose square no float holds: checked without the z loss
    _check_balance(l, ids, z=0.0)
    l[10], l[11] = 0.0, 1.0
    _check_balance(l, ids)
    for bad in (np.nan, np.inf):
        q = np.where(np.isfinite(l), l, 0.0)
        q[20, 4] = bad
        _, _, _, _, _, out = _balance(q, ids)
        assert torch.isnan(out.losses).all() and torch.isnan(out.dlogits[20]).all()
        assert torch.isfinite(out.dlogits[19]).all() and torch.isfinite(out.dlogits[21]).all()


def test_balance_loss_ids_outside_are_not_counted():
    say("balance with ids outside the experts")
    rng, l, ids = _draw(7, 300, 10, 4)
    ids = ids.copy()
    ids[rng.random(ids.shape) < 0.2] = -1
    ids[rng.random(ids.shape) < 0.1] = 10
    ids[5] = [2 ** 31 - 1, -2 ** 31, 10, -1]
    out = _check_balance(l, ids)
    assert int(out.counts.sum()) == int(((ids >= 0) & (ids < 10)).sum())


def test_balance_loss_collapsed_router():
    """Every token on one expert: the counts' atomics all meet."""
    say("balance collapsed")
    l = np.zeros((3000, 16), dtype=np.float32)
    l[:, 5] = 9.0
    out = _check_balance(l, np.full((3000, 1), 5))
    assert int(out.counts[0, 5]) == 3000


def test_balance_loss_far_logits_and_large_batch():
    say("balance T=40000 E=24, logits in the hundreds")
    _, l, ids = _draw(8, 3000, 24, 2, spread=60.0)
    _check_balance(l, ids)
    rng, l, ids = _draw(9, 40000, 24, 2)
    _check_balance(l, ids, mask=(rng.random(40000) < 0.9).astype(np.uint8), off=[0, 11, 20000, 39990])


@pytest.mark.parametrize("off", [None, [5, 2 ** 20, 2 ** 21 + 70]])
def test_balance_loss_past_32_bits(off):
    """More than 2^31 logits: sums against 64 bits, gradients against the same rows alone."""
    say(f"balance T=2^21+77 E=1024 off={off}")
    T, E, alpha, z = 2 ** 21 + 77, 1024, 0.3, 0.05
    gen = torch.Generator(device=DEV).manual_seed(3)
    lg = torch.randn((T, E), generator=gen, device=DEV)
    ids = torch.randint(0, E, (T, 1), generator=gen, device=DEV, dtype=torch.int32)
    S = 1 if off is None else len(off) - 1
    offs = [0, T] if off is None else off
    og = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    desc, out = ops.make_desc(T, 64, 64, E, 1, None), Outputs(T, E, S)
    ops.moe_balance_loss(desc, lg, ids, alpha, z, out.counts, out.seq_tokens, out.mean_probs, out.losses,
                         ops.workspace(ops.moe_balance_workspace_size(desc, S)), seq_offsets=og, dlogits=out.dlogits)
    torch.cuda.synchronize()
    out.check_guards()
    # K = 2 range + 24 as above; a lane adds up at most 4096 rows one after another, each of relative error u
    K = 2 * float(lg.max() - lg.min()) + 24 + 4096
    balance, squares, n = 0.0, 0.0, 0
    for s in range(S):
        b, e = offs[s], offs[s + 1]
        assert torch.equal(out.counts[s].long(), torch.bincount(ids[b:e, 0].long(), minlength=E))
        assert int(out.seq_tokens[s]) == e - b
        probs = torch.zeros(E, dtype=torch.float64, device=DEV)
        for i in range(b, e, 1 << 16):
            l = lg[i:min(i + (1 << 16), e)].double()
            lse = torch.logsumexp(l, 1)
            probs += (l - lse[:, None]).exp().sum(0)
            squares += float((lse * lse).sum())
        probs /= e - b
        assert torch.all((out.mean_probs[s] - probs).abs() <= (K + 32) * U * probs)
        balance += float((out.counts[s].double() / (e - b) * probs).sum())
        n += e - b
    losses = to_np(out.losses)
    want = (alpha * E * balance / S, z * squares / n)
    assert abs(losses[0] - want[0]) <= (K + 34) * U * want[0]
    assert abs(losses[1] - want[1]) <= 2 * (K + 34) * U * (2 * want[1] + z)
    # rows at the start, on both sides of 2^31 values (row 2^21), at a sequence's end and at the batch's
    for i in (0, 2 ** 20 - 8, 2 ** 21 - 8, T - 16):
        rows = slice(i, i + 16)
        seq = None
        if off is not None:
            seq = torch.tensor([min(max(o - i, 0), 16) for o in off], dtype=torch.int32, device=DEV)
        part = torch.full((16, E), 7.0, device=DEV)
        ops.moe_balance_loss_backward(ops.make_desc(16, 64, 64, E, 1, None), lg[rows], out.counts, out.seq_tokens,
                                      alpha, z, part, seq_offsets=seq)
        assert torch.equal(part, out.dlogits[rows]) and bool(part.any())


def test_balance_sums_past_32_bits():
    """More than 2^31 logits, R their largest range within a row.  A probability is off by 4 R + 41 u (twice the
    exponential's 2 R + 8, 22 roundings of the row's sum, reciprocal and product); a mean adds what one lane adds up in
    floats (a quarter of a 512th of the rows) and 8 u.  The losses are sums in 64 bits: 25 u for the row's dot product,
    and z off by (2 R + 33) u (|z| + 1)."""
    say("balance sums T=2^21+77 E=1024")
    T, E, alpha, z = 2 ** 21 + 77, 1024, 0.3, 0.05
    gen = torch.Generator(device=DEV).manual_seed(75)
    lg = torch.randn((T, E), generator=gen, device=DEV)
    ids = torch.randint(0, E, (T, 1), generator=gen, device=DEV, dtype=torch.int32)
    desc, out = ops.make_desc(T, 64, 64, E, 1, None), Outputs(1, E, 1)
    ops.moe_balance_loss(desc, lg, ids, alpha, z, out.counts, out.seq_tokens, out.mean_probs, out.losses,
                         ops.workspace(ops.moe_balance_workspace_size(desc)))
    torch.cuda.synchronize()
    out.check_guards()
    probs, squares, R = torch.zeros(E, dtype=torch.float64, device=DEV), 0.0, 0.0
    for i in range(0, T, 1 << 16):
        l = lg[i:min(i + (1 << 16), T)].double()
        lse = torch.logsumexp(l, 1)
        probs += (l - lse[:, None]).exp().sum(0)
        squares += float((lse * lse).sum())
        R = max(R, float((l.amax(1) - l.amin(1)).max()))
    probs /= T
    rows = -(--(-T // 512) // 4)
    assert torch.all((out.mean_probs[0] - probs).abs() <= (4 * R + 41 + rows + 8) * U * probs)
    losses = to_np(out.losses)
    want = alpha * E * float((out.counts[0].double() / T * probs).sum()), z * squares / T
    assert abs(losses[0] - want[0]) <= (4 * R + 41 + 25) * U * want[0]
    assert abs(losses[1] - want[1]) <= 2 * (2 * R + 34) * U * (2 * want[1] + z)


@pytest.mark.parametrize("T,E,k,off", [(200, 32, 4, None), (300, 33, 3, [4, 100, 100, 290]), (70, 64, 2, [0, 70]),
                                       (40, 1, 1, None), (40, 700, 8, None), (40, 1023, 8, None)])
def test_balance_gradient_of_uncounted_tokens_is_zero_whatever_comes_from_above(T, E, k, off):
    """An upstream gradient that is not finite (an overflowed loss scale) or a product of coefficients past the floats:
    zero for masked tokens, for tokens of no sequence and for those without a finite logit, all the same."""
    say(f"balance gradient under infinite factors T={T} E={E}")
    rng, l, ids = _draw(70, T, E, k)
    mask = rng.random(T) < 0.6
    l[10:13] = -np.inf
    mask[10:13] = [True, False, True]
    none = ~mask
    none[10:13] = True
    if off is not None:
        none[:off[0]] = none[off[-1]:] = True
    desc, lg, ig, mg, og, out = _balance(l, ids, 0.3, 0.05, mask, off)
    dl = torch.full_like(out.dlogits, 7.0)
    for up in ((float("inf"), 1.0), (1.0, -float("inf")), (float("nan"), float("nan"))):
        ops.moe_balance_loss_backward(desc, lg, out.counts, out.seq_tokens, 0.3, 0.05, dl, token_mask=mg, seq_offsets=og,
                                      dloss=torch.tensor(up, device=DEV))
        got = to_np(dl)
        assert np.all(got[none] == 0.0)
        assert not np.isfinite(got[~none]).all()
    _, _, _, _, _, out = _balance(l, ids, 3e38, 3e38, mask, off)
    assert np.all(to_np(out.dlogits)[none] == 0.0)


def test_balance_loss_equals_the_aux_loss_and_needs_no_gradient():
    say("balance against moe_router_aux_loss; without dlogits")
    for T, E, k in [(64, 8, 2), (1000, 64, 1)]:
        _, l, ids = _draw(T, T, E, k)
        desc, lg, ig, _, _, out = _balance(l, ids, alpha=0.02)
        loss = torch.empty(4, device=DEV)
        ws = ops.workspace(ops.moe_workspace_size(desc))
        ops.moe_router_aux_loss(desc, lg, out.counts[0], 0.02, loss, ws)
        assert abs(float(loss[0]) - float(out.losses[0])) <= 1e-5 * float(loss[0])
        bare = Outputs(T, E, 1)
        ops.moe_balance_loss(desc, lg, ig, 0.02, 0.05, bare.counts, bare.seq_tokens, bare.mean_probs, bare.losses,
                             ops.workspace(ops.moe_balance_workspace_size(desc)))
        assert torch.equal(bare.losses, out.losses) and torch.equal(bare.mean_probs, out.mean_probs)
        assert torch.all(bare.dlogits == 7)


@pytest.mark.parametrize("T,E,k,S", [(16, 32, 4, 1), (3000, 64, 2, 1), (2000, 33, 3, 5)])
def test_balance_loss_is_deterministic_and_replays_from_a_graph(T, E, k, S):
    say(f"balance graph T={T} E={E} S={S}")
    _, l, ids = _draw(T + 1, T, E, k)
    off = None if S == 1 else [0] + [T * (i + 1) // S - 3 for i in range(S)]
    desc, lg, ig, mg, og, want = _balance(l, ids, off=off)
    out = Outputs(T, E, S)
    ws = ops.workspace(ops.moe_balance_workspace_size(desc, S))

    def call():
        ops.moe_balance_loss(desc, lg, ig, 0.3, 0.05, out.counts, out.seq_tokens, out.mean_probs, out.losses, ws,
                             seq_offsets=og, dlogits=out.dlogits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for n in want.whole:
        assert torch.equal(want.whole[n], out.whole[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        for t in out.whole.values():
            t[:-GUARD].fill_(3)
        ws.fill_(17 * i)
        g.replay()
        torch.cuda.synchronize()
        for n in want.whole:
            assert torch.equal(want.whole[n], out.whole[n]), (i, n)


def test_balance_loss_on_two_streams_and_its_gradient_from_a_graph():
    """Two batches at once, each with its own buffers; the gradient alone captured and replayed."""
    say("balance on two streams")
    runs = []
    for i, (T, E, k, S) in enumerate([(3000, 48, 2, 3), (5000, 33, 4, 1)]):
        _, l, ids = _draw(50 + i, T, E, k)
        off = None if S == 1 else [3, 900, 950, T - 10]
        runs.append((k, S) + _balance(l, ids, off=off)[:5] + (_balance(l, ids, off=off)[5],))
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (k, S, desc, lg, ig, mg, og, want), st in zip(runs, streams):
            out = Outputs(lg.shape[0], lg.shape[1], S)
            ws = ops.workspace(ops.moe_balance_workspace_size(desc, S))
            st.wait_stream(torch.cuda.current_stream())
            ops.moe_balance_loss(desc, lg, ig, 0.3, 0.05, out.counts, out.seq_tokens, out.mean_probs, out.losses, ws,
                                 seq_offsets=og, dlogits=out.dlogits, stream=st)
            outs.append((want, out, ws))
    torch.cuda.synchronize()
    for want, out, _ in outs:
        assert all(torch.equal(want.whole[n], out.whole[n]) for n in want.whole)
    k, S, desc, lg, ig, mg, og, want = runs[0]
    d, up = torch.empty_like(lg), torch.ones(2, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.moe_balance_loss_backward(desc, lg, want.counts, want.seq_tokens, 0.3, 0.05, d, seq_offsets=og, dloss=up)
    for factor in (1.0, 2.0, -0.5):
        up.fill_(factor)
        d.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want.dlogits * factor)  # powers of two: exact


# ----------------------------------------------------------------------------- gradient norm

def _norm(grads, max_norm):
    lst = ops.grad_list(grads)
    need = ops.moe_grad_norm_workspace_size(lst)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((2 + GUARD,), 7.0, device=DEV)
    ops.moe_grad_norm(lst, max_norm, out[:2], ws[:need])
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == 255) and torch.all(out[2:] == 7)
    return out[:2].cpu().double().numpy()


@pytest.mark.parametrize("sizes,dts", [
    ([1], "f"), ([1], "b"), ([7, 8, 9], "fb"), ([2047, 2048, 2049, 0, 1], "b"), ([100003, 5], "fb"),
    ([4096 * 3 + 1] * 3, "f"), (list(range(1, 150)), "fb"), ([1 << 20, 3, (1 << 22) + 5], "b"), ([], "f"), ([0, 0], "b"),
])
def test_grad_norm(sizes, dts):
    say(f"grad norm {len(sizes)} tensors {dts}")
    gen = torch.Generator(device=DEV).manual_seed(len(sizes))
    grads = [torch.randn(n, generator=gen, device=DEV).to(torch.float32 if dts[i % len(dts)] == "f" else torch.bfloat16)
             for i, n in enumerate(sizes)]
    for max_norm in (0.5, 1e9, float("inf")):
        got = _norm(grads, max_norm)
        norm, scale = oracle.grad_norm([to_np(g) for g in grads], max_norm)
        assert abs(got[0] - norm) <= 2 * U * norm
        assert abs(got[1] - scale) <= 2 * U * scale


def test_grad_norm_extremes():
    say("grad norm extremes")
    big = torch.full((3000,), 1e38, device=DEV)  # squares that no float holds
    got = _norm([big], 1.0)
    norm, scale = oracle.grad_norm([to_np(big)], 1.0)  # 5.5e39: past the largest float
    assert np.isinf(got[0]) and abs(got[1] - scale) <= 1.5e-45
    mid = torch.full((3000,), 1e30, device=DEV)
    assert abs(_norm([mid], 1.0)[0] - oracle.grad_norm([to_np(mid)], 1.0)[0]) <= 2 * U * 6e31
    small = torch.full((3000,), 1e-30, device=DEV)
    assert abs(_norm([small], 1.0)[0] - oracle.grad_norm([to_np(small)], 1.0)[0]) <= 2 * U * 6e-29
    for bad in (float("inf"), float("nan"), -float("inf")):
        g = torch.ones(70000, device=DEV, dtype=torch.bfloat16)
        g[-1] = bad
        got = _norm([torch.ones(3, device=DEV), g], 1.0)
        assert not np.isfinite(got[0]) and np.isnan(got[1])


# --------------------------------------------------------------------------------- AdamW step

H = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8)


def _make(sizes, bits, pf, gf, master, seed, zero_state=False):
    """Parameters, gradients and states at the front of buffers with guards behind them."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda n, s: torch.randn(n, generator=gen, device=DEV) * s  # noqa: E731
    whole, params, grads, states = [], [], [], []

    def guarded(t):
        w = torch.full((t.numel() + GUARD,), 7, dtype=t.dtype, device=DEV)
        w[:t.numel()] = t
        whole.append(w)
        return w[:t.numel()]
    for i, n in enumerate(sizes):
        w = rnd(n, 0.1)
        p32 = pf[i % len(pf)] == "f"
        params.append(guarded(w if p32 else w.bfloat16()))
        spread = torch.exp(rnd(n, 1.0))
        grads.append(guarded((rnd(n, 1e-3) * spread).to(torch.float32 if gf[i % len(gf)] == "f" else torch.bfloat16)))
        m, v = rnd(n, 5e-4) * spread, (rnd(n, 1e-3) * spread) ** 2
        if zero_state:
            m, v = m * 0, v * 0
        if bits == 32:
            s = dict(m=guarded(m), v=guarded(v))
        else:
            cm, sm = oracle.held_m(to_np(m))
            cv, sv = oracle.held_v(to_np(v))
            s = dict(m=guarded(torch.tensor(cm, dtype=torch.int8, device=DEV)),
                     v=guarded(torch.tensor(cv, dtype=torch.uint8, device=DEV)),
                     m_scale=guarded(torch.tensor(sm, device=DEV)), v_scale=guarded(torch.tensor(sv, device=DEV)))
        if master and not p32:
            s["master"] = guarded(w)
        states.append(s)
    return whole, params, grads, states


def _snapshot(params, grads, states):
    get = lambda t: None if t is None else to_np(t).copy()  # noqa: E731
    return [(get(p), get(g), {k: get(t) for k, t in s.items()}) for p, g, s in zip(params, grads, states)]


def _check_step(before, params, states, bits, decay, t, scale=1.0, lr=1e-2):
    """Every tensor after a step against the oracle's step from the tensors before it."""
    b1, b2 = H["betas"]
    for i, ((p0, g0, s0), p, s) in enumerate(zip(before, params, states)):
        if p0.size == 0:
            continue
        w0 = (s0["master"] if "master" in s0 else p0).astype(np.float64)
        if bits == 32:
            m0, v0 = s0["m"].astype(np.float64), s0["v"].astype(np.float64)
        else:
            m0, v0 = oracle.read_m(s0["m"], s0["m_scale"]), oracle.read_v(s0["v"], s0["v_scale"])
        g0 = g0.astype(np.float64)
        w, m, v = oracle.adamw_step(w0, g0, m0, v0, t, lr, b1, b2, H["eps"], decay[i], scale)
        parts = np.abs(b1 * m0) + np.abs((1 - b1) * g0 * scale)
        if bits == 32:
            assert np.all(np.abs(to_np(s["m"]) - m) <= 4 * U * parts + 1e-44), i
            assert np.all(np.abs(to_np(s["v"]) - v) <= 6 * U * v + 1e-44), i
        else:
            cm, sm = oracle.held_m(m)
            cv, sv = oracle.held_v(v)
            assert np.array_equal(to_np(s["m_scale"]), sm) and np.array_equal(to_np(s["v_scale"]), sv), i
            assert np.array_equal(to_np(s["m"]), cm), (i, np.nonzero(to_np(s["m"]) != cm)[0][:5])
            assert np.array_equal(to_np(s["v"]), cv), (i, np.nonzero(to_np(s["v"]) != cv)[0][:5])
        den = np.sqrt(v) / np.sqrt(1 - b2 ** t) + H["eps"]
        bound = 3 * U * np.abs(w0) + 16 * U * lr / (1 - b1 ** t) * parts / den + 1e-44
        got = to_np(p).astype(np.float64)
        if "master" in s0:
            assert np.all(np.abs(to_np(s["master"]) - w) <= bound), i
            assert torch.equal(s["master"].to(torch.bfloat16), p), i
        elif p.dtype == torch.float32:
            assert np.all(np.abs(got - w) <= bound), (i, (np.abs(got - w) / bound).max())
        else:
            assert np.all(np.abs(got - w) <= bound * (1 + B) + B * np.abs(w)), i


def _guards(whole):
    for w in whole:
        assert torch.all(w[-GUARD:] == 7)


ODD = [1, 2, 7, 8, 9, 255, 256, 257, 511, 2047, 2048, 2049, 4100, 0, 10007]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pf,gf,master", [("f", "f", False), ("b", "b", False), ("b", "b", True), ("b", "f", True),
                                          ("fb", "fbb", True), ("f", "b", False)])
def test_adamw_sizes_and_types(bits, pf, gf, master):
    say(f"adamw bits={bits} params={pf} grads={gf} master={master}")
    whole, params, grads, states = _make(ODD, bits, pf, gf, master, seed=bits + len(pf))
    decay = [0.0 if i % 2 else 0.1 for i in range(len(ODD))]
    opt = ops.MoEAdamW(params, grads, weight_decay=decay, state_bits=bits, states=states, step=10, **H)
    for t in (11, 12):
        before = _snapshot(params, grads, states)
        opt.step()
        torch.cuda.synchronize()
        _guards(whole)
        _check_step(before, params, states, bits, decay, t)
        assert all(np.array_equal(to_np(g), b[1]) for g, b in zip(grads, before))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors_clipped(bits):
    say(f"adamw 137 tensors clipped bits={bits}")
    sizes = [1 + (i * 37) % 700 for i in range(137)]
    whole, params, grads, states = _make(sizes, bits, "bf", "b", True, seed=3)
    opt = ops.MoEAdamW(params, grads, weight_decay=0.05, state_bits=bits, states=states, max_grad_norm=0.01, **H)
    before = _snapshot(params, grads, states)
    opt.step()
    torch.cuda.synchronize()
    _guards(whole)
    norm, scale = oracle.grad_norm([b[1] for b in before], 0.01)
    assert scale < 1 and abs(float(opt.grad_norm[0]) - norm) <= 2 * U * norm
    # the factor is held as a float: the step is checked from the float the device holds
    assert abs(float(opt.grad_norm[1]) - scale) <= 2 * U
    _check_step(before, params, states, bits, [0.05] * 137, 1, scale=float(opt.grad_norm[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_first_steps_from_zero_states(bits):
    say(f"adamw from zeros bits={bits}")
    g = torch.Generator(device=DEV).manual_seed(1)
    params = [torch.randn((33, 40), generator=g, device=DEV).bfloat16(), torch.randn(1000, generator=g, device=DEV)]
    grads = [torch.randn(p.shape, generator=g, device=DEV).to(p.dtype) * 1e-2 for p in params]
    grads[0][3] = 0  # an expert without tokens: no gradient at all
    opt = ops.MoEAdamW(params, grads, weight_decay=0.1, state_bits=bits, master_weights=True, **H)
    for t in range(1, 5):
        before = _snapshot([p.view(-1) for p in params], [q.view(-1) for q in grads],
                           [{k: x.view(-1) for k, x in s.items()} for s in opt.states])
        opt.step()
        torch.cuda.synchronize()
        _check_step(before, [p.view(-1) for p in params], [{k: x.view(-1) for k, x in s.items()} for s in opt.states],
                    bits, [0.1, 0.1], t)
        for q in grads:
            q.mul_(-0.7)
    assert torch.isfinite(params[0]).all()


def test_adamw_8bit_blocks_of_extremes():
    """Blocks of zeros, of values below the smallest normal float, of one large value among small ones, and of
    values that are not finite."""
    say("adamw 8-bit extremes")
    n = 256 * 6 + 40
    p = torch.ones(n, device=DEV)
    g = torch.zeros(n, device=DEV)
    g[256:512] = 1e-38
    g[512:768] = 1e-6
    g[600] = 1e3
    g[768 + 5] = float("nan")
    g[1024 + 9] = float("inf")
    g[1536:] = -2.0
    opt = ops.MoEAdamW([p], [g], weight_decay=0.0, state_bits=8, **H)
    before = _snapshot([p], [g], opt.states)
    opt.step()
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        w, m, v = oracle.adamw_step(before[0][0], before[0][1], np.zeros(n), np.zeros(n), 1, 1e-2, 0.9, 0.99, 1e-8, 0)
    s = opt.states[0]
    (cm, sm), (cv, sv) = oracle.held_m(m), oracle.held_v(v)
    assert np.array_equal(to_np(s["m_scale"]), sm, equal_nan=True)
    assert np.array_equal(to_np(s["v_scale"]), sv, equal_nan=True)
    assert np.isnan(sm[3]) and np.isnan(sm[4]) and sm[0] == 0 and sv[1] == 0
    assert np.array_equal(to_np(s["m"]), cm) and np.array_equal(to_np(s["v"]), cv)
    assert int(s["v"][512:600].min()) == 1  # above zero: never held as zero
    got = to_np(p)
    fine = np.isfinite(w)
    assert np.array_equal(np.isfinite(got), fine) and fine.sum() == n - 2
    m_out, v_out = opt.read_states()
    want = oracle.read_m(cm, sm)
    assert np.allclose(to_np(m_out[0]), want, rtol=4 * U, atol=0, equal_nan=True)
    assert np.allclose(to_np(v_out[0]), oracle.read_v(cv, sv), rtol=4 * U, atol=0, equal_nan=True)


def test_adamw_read_states_of_some():
    say("adamw read states of some tensors")
    _, params, grads, states = _make([5, 3000, 700], 8, "b", "b", False, seed=60)
    opt = ops.MoEAdamW(params, grads, state_bits=8, states=states, **H)
    whole = torch.full((3000 + GUARD,), 7.0, device=DEV)
    m = [None, whole[:3000], None]
    assert opt.read_states(m, None)[1] is None
    torch.cuda.synchronize()
    want = oracle.read_m(to_np(states[1]["m"]), to_np(states[1]["m_scale"]))
    assert np.array_equal(to_np(m[1]), want.astype(np.float32)) and torch.all(whole[3000:] == 7)
    v = [None, None, torch.empty(700, device=DEV)]
    opt.read_states(None, v)
    want = oracle.read_v(to_np(states[2]["v"]), to_np(states[2]["v_scale"]))
    assert np.array_equal(to_np(v[2]), want.astype(np.float32))
    with pytest.raises(ValueError, match="holds"):
        opt.read_states([None, whole[:2999], None], None)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_states_may_name_what_they_lack(bits):
    say(f"adamw states with None bits={bits}")
    got = []
    for none in (False, True):
        whole, params, grads, states = _make([300, 9], bits, "b", "b", False, seed=61)
        if none:
            states = [dict(s, master=None, **({} if bits == 8 else dict(m_scale=None, v_scale=None))) for s in states]
        ops.MoEAdamW(params, grads, state_bits=bits, states=states, **H).step()
        torch.cuda.synchronize()
        got.append(whole)
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_balance_of_an_empty_batch_is_zero():
    say("balance of no tokens")
    E, S = 33, 3
    desc = ops.MoeDesc(num_tokens=0, d_model=64, d_ff=64, num_experts=E, top_k=2, capacity=ops.MOE_NO_CAPACITY)
    counts = torch.full((S, E), 7, dtype=torch.int32, device=DEV)
    tokens = torch.full((S,), 7, dtype=torch.int32, device=DEV)
    probs, losses = torch.full((S, E), 7.0, device=DEV), torch.full((2,), 7.0, device=DEV)
    none = torch.empty((0, E), device=DEV)
    ops.moe_balance_loss(desc, none, torch.empty((0, 2), dtype=torch.int32, device=DEV), 0.1, 0.1, counts, tokens, probs,
                         losses, None, seq_offsets=torch.zeros(S + 1, dtype=torch.int32, device=DEV), dlogits=none)
    assert not counts.any() and not tokens.any() and not probs.any() and not losses.any()


def test_adamw_states_read_on_another_stream():
    say("adamw read_states on another stream")
    _, params, grads, states = _make([5000], 8, "b", "b", False, seed=62)
    opt = ops.MoEAdamW(params, grads, state_bits=8, states=states, **H)
    opt.step()
    want = opt.read_states()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = opt.read_states(stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))


def test_adamw_refuses_wrong_options_when_built():
    p, g = torch.ones(8, device=DEV), torch.ones(8, device=DEV)
    for kw, error in [(dict(lr=-1.0), ValueError), (dict(lr=float("nan")), ValueError),
                      (dict(max_grad_norm=0.0), ValueError), (dict(betas=(1.0, 0.9)), ops.MoEError),
                      (dict(eps=0.0), ops.MoEError), (dict(step=-1), ops.MoEError)]:
        for capturable in (False, True):
            if capturable and "step" in kw:
                continue
            with pytest.raises(error):
                ops.MoEAdamW([p], [g], capturable=capturable, **{**H, **kw})
    opt = ops.MoEAdamW([p], [g], capturable=True, **H)
    with pytest.raises(ValueError):
        opt.set_lr(float("inf"))


def test_adamw_nan_gradient_stays_where_it_is():
    say("adamw NaN gradient, 32 bits")
    p, g = torch.ones(1000, device=DEV), torch.full((1000,), 0.1, device=DEV)
    g[17] = float("nan")
    opt = ops.MoEAdamW([p], [g], state_bits=32, **H)
    opt.step()
    bad = torch.isnan(p).nonzero().flatten().tolist()
    assert bad == [17] and torch.isnan(opt.states[0]["m"]).sum() == 1 and torch.isnan(opt.states[0]["v"]).sum() == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_leaves_everything_when_the_norm_is_not_finite(bits):
    say(f"adamw skipped step bits={bits}")
    whole, params, grads, states = _make([300, 5, 4000], bits, "b", "b", True, seed=9)
    grads[1][2] = float("inf")
    before = [w.clone() for w in whole]
    opt = ops.MoEAdamW(params, grads, state_bits=bits, states=states, max_grad_norm=1.0, **H)
    opt.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, whole))
    assert not torch.isfinite(opt.grad_norm[0]) and torch.isnan(opt.grad_norm[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_captured_steps_count_on(bits):
    """A capturable step replayed from a graph, with eager work between, equals eager steps bit for bit; the rate
    changes between replays."""
    say(f"adamw graph bits={bits}")
    sizes = [700, 3, 5000]

    def build(capturable):
        whole, params, grads, states = _make(sizes, bits, "b", "b", True, seed=21)
        return whole, grads, ops.MoEAdamW(params, grads, weight_decay=0.1, state_bits=bits, states=states,
                                          max_grad_norm=0.05, capturable=capturable, **H)
    w1, g1, eager = build(True)
    w2, g2, captured = build(True)
    captured.step()  # warm up, then back to the start
    torch.cuda.synchronize()
    w0, _, plain = build(False)
    for a, b in zip(w2, w0):
        a.copy_(b)
    captured.step_dev.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    captured.step_dev.zero_()
    for i in range(4):
        for a, b in zip(g1, g2):
            a.mul_(-0.8)
            b.mul_(-0.8)
        eager.set_lr(1e-2 / (i + 1))
        captured.set_lr(1e-2 / (i + 1))
        eager.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w1, w2)), i
        assert torch.equal(eager.grad_norm, captured.grad_norm)
    assert int(captured.step_dev) == 4 == int(eager.step_dev)
    # host scalars give the device scalars' step (the rate is a float there)
    w3, g3, other = build(True)
    plain.set_lr(float(np.float32(1e-2)))
    plain.step()
    other.step()
    torch.cuda.synchronize()
    for a, b in zip(w0, w3):
        assert torch.allclose(a.float(), b.float(), rtol=1e-6, atol=0)


def test_adamw_refuses_a_capture_that_would_repeat_its_step():
    say("adamw capture refused")
    p, g = torch.ones(100, device=DEV), torch.ones(100, device=DEV)
    opt = ops.MoEAdamW([p], [g], **H)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="capturable"):
            opt.step()
    torch.cuda.synchronize()
    opt.step()
    assert opt.step_count == 1


def test_adamw_refuses_moved_tensors_and_another_device():
    say("adamw refusals of moved tensors")
    p, g = torch.ones(100, device=DEV), torch.ones(100, device=DEV)
    opt = ops.MoEAdamW([p], [g], max_grad_norm=1.0, **H)
    opt.step()
    kept, old = p.clone(), p.data
    p.data = torch.ones(100, device=DEV)
    with pytest.raises(RuntimeError, match="replaced"):
        opt.step()
    p.data = old
    # gradients: the memory that the list was built with stays alive and is what is read
    lst, out = ops.grad_list([g]), torch.zeros(2, device=DEV)
    g.data = torch.full((100,), 7.0, device=DEV)
    ops.moe_grad_norm(lst, 1.0, out, ops.workspace(ops.moe_grad_norm_workspace_size(lst)))
    assert float(out[0]) == 10.0
    opt._device += 1
    lst.device += 1
    for call in (opt.step, opt.read_states, lambda: ops.moe_grad_norm(lst, 1.0, out, opt._ws)):
        with pytest.raises(RuntimeError, match="current"):
            call()
    assert torch.equal(p, kept) and opt.step_count == 1


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.0, 0.99), (0.9, 0.0)])
def test_adamw_without_memory(bits, betas):
    """beta1 or beta2 of zero, with the step's number on the host and on the device."""
    say(f"adamw betas={betas} bits={bits}")
    got = []
    for capturable in (False, True):
        whole, params, grads, states = _make([777], bits, "f", "f", False, seed=40)
        before = _snapshot(params, grads, states)
        ops.MoEAdamW(params, grads, lr=2.0 ** -7, betas=betas, eps=1e-8, weight_decay=0.5, state_bits=bits,
                     states=states, step=2, capturable=capturable).step()
        torch.cuda.synchronize()
        got.append([w.clone() for w in whole])
    s0 = before[0][2]
    m0 = s0["m"].astype(np.float64) if bits == 32 else oracle.read_m(s0["m"], s0["m_scale"])
    v0 = s0["v"].astype(np.float64) if bits == 32 else oracle.read_v(s0["v"], s0["v_scale"])
    g0 = before[0][1].astype(np.float64)
    w, m, v = oracle.adamw_step(before[0][0], g0, m0, v0, 3, 2.0 ** -7, betas[0], betas[1], 1e-8, 0.5)
    parts = np.abs(betas[0] * m0) + np.abs((1 - betas[0]) * g0)
    den = np.sqrt(v) / np.sqrt(1 - betas[1] ** 3) + 1e-8
    bound = 3 * U * np.abs(before[0][0]) + 16 * U * 2.0 ** -7 / (1 - betas[0] ** 3) * parts / den + 1e-44
    assert np.all(np.abs(to_np(params[0]) - w) <= bound)
    if bits == 8:
        assert np.array_equal(to_np(states[0]["m"]), oracle.held_m(m)[0])
        assert np.array_equal(to_np(states[0]["v"]), oracle.held_v(v)[0])
    assert all(torch.equal(a, b) for a, b in zip(*got))  # the same scalars: a rate that is a float


def test_adamw_8bit_blocks_of_the_smallest_floats():
    """Scales from the smallest normal float up to where the float path takes over, and values far below them."""
    say("adamw 8-bit blocks of tiny values")
    rng = np.random.default_rng(41)
    scales = 10.0 ** np.arange(-19, -9, 0.25)  # gradients; their squares reach 1e-38
    g = np.concatenate([s * rng.standard_normal(256) * np.exp(-rng.random(256) * 9) for s in scales])
    p, gd = torch.ones(g.size, device=DEV), torch.tensor(g, dtype=torch.float32, device=DEV)
    opt = ops.MoEAdamW([p], [gd], lr=1e-2, betas=(0.5, 0.5), eps=1e-18, weight_decay=0.0, state_bits=8)
    for t in (1, 2, 3):
        before = _snapshot([p], [gd], opt.states)
        opt.step()
        torch.cuda.synchronize()
        s0, s = before[0][2], opt.states[0]
        m0, v0 = oracle.read_m(s0["m"], s0["m_scale"]), oracle.read_v(s0["v"], s0["v_scale"])
        g0 = before[0][1].astype(np.float64)
        w, m, v = oracle.adamw_step(before[0][0], g0, m0, v0, t, 1e-2, 0.5, 0.5, 1e-18, 0.0)
        (cm, sm), (cv, sv) = oracle.held_m(m), oracle.held_v(v)
        assert np.array_equal(to_np(s["m_scale"]), sm) and np.array_equal(to_np(s["v_scale"]), sv)
        assert np.array_equal(to_np(s["m"]), cm) and np.array_equal(to_np(s["v"]), cv)
        parts = np.abs(0.5 * m0) + np.abs(0.5 * g0)
        den = np.sqrt(v) / np.sqrt(1 - 0.5 ** t) + 1e-18
        assert np.all(np.abs(to_np(p) - w) <= 3 * U * np.abs(w) + 16 * U * 1e-2 / (1 - 0.5 ** t) * parts / den)
        gd.mul_(-0.6)


def test_adamw_on_another_stream_and_two_lists_at_once():
    say("adamw on two streams")
    runs = []
    for streams in (None, [torch.cuda.Stream(), torch.cuda.Stream()]):
        sets = [_make([20000, 77], bits, "b", "b", True, seed=31 + bits) for bits in (32, 8)]
        opts = [ops.MoEAdamW(p, g, state_bits=bits, states=s, max_grad_norm=0.1, **H)
                for bits, (_, p, g, s) in zip((32, 8), sets)]
        torch.cuda.synchronize()
        for _ in range(3):
            for i, o in enumerate(opts):
                o.step(stream=streams[i] if streams else None)
        torch.cuda.synchronize()
        runs.append([w for s in sets for w in s[0]])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_adamw_and_norm_past_32_bits():
    """A tensor of more than 2^31 values: the last values against the oracle, one in the middle too."""
    say("adamw 8 bits, 2^31 + 777 values")
    n = 2 ** 31 + 777
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = 1200
    gen = torch.Generator(device=DEV).manual_seed(2)
    p[-tail:] = torch.randn(tail, generator=gen, device=DEV).bfloat16()
    g[-tail:] = torch.randn(tail, generator=gen, device=DEV).bfloat16()
    p[2 ** 31 - 5], g[2 ** 31 - 5] = 1.0, 2.0
    opt = ops.MoEAdamW([p], [g], weight_decay=0.1, state_bits=8, max_grad_norm=1.0, **H)
    w0, g0 = to_np(p[-tail:]).astype(np.float64), to_np(g[-tail:]).astype(np.float64)
    opt.step()
    torch.cuda.synchronize()
    norm, _ = oracle.grad_norm([g0, np.array([0.0])], 1.0)
    inside = 2 ** 31 - 5 >= n - tail
    if not inside:
        norm = math.hypot(norm, 2.0)
    assert abs(float(opt.grad_norm[0]) - norm) <= 2 * U * norm
    scale = float(opt.grad_norm[1])
    w, m, v = oracle.adamw_step(w0, g0, 0 * g0, 0 * g0, 1, 1e-2, 0.9, 0.99, 1e-8, 0.1, scale)
    # whole blocks from the tail's first block on
    first = (n - tail + 255) // 256 * 256
    skip = first - (n - tail)
    cm, sm = oracle.held_m(m[skip:])
    s = opt.states[0]
    assert np.array_equal(to_np(s["m"][first:]), cm) and np.array_equal(to_np(s["m_scale"][first // 256:]), sm)
    # |u| <= sqrt(10) (m' against the root of v' after one step): 16 u lr of that, and the bf16 rounding
    assert np.all(np.abs(to_np(p[-tail:]) - w) <= B * np.abs(w) + 1e-7)
    assert int(torch.count_nonzero(p)) <= tail + 1


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_given_states_with_master_weights(bits):
    """States without a float copy of the weights, as a checkpoint of bf16 weights leaves them: master_weights makes
    it, and steps far below a weight's last place add up.  A copy that the states hold is taken as it is."""
    say(f"adamw given states and master_weights bits={bits}")
    for lacking in ({}, dict(master=None)):
        _, params, grads, states = _make([300, 40], bits, "bf", "b", False, seed=63, zero_state=True)
        given = [dict(s, **lacking) for s in states]
        start = [p.clone() for p in params]
        opt = ops.MoEAdamW(params, grads, weight_decay=0.0, state_bits=bits, states=given, master_weights=True,
                           lr=2.0 ** -20, betas=(0.0, 0.0), eps=1e-30)
        assert opt.states[1].get("master") is None and given[0].get("master") is None
        assert torch.equal(opt.states[0]["master"], start[0].float())
        opt.step()
        torch.cuda.synchronize()
        # betas of zero: the step is lr times the gradient's sign, off by 16 u of it; the copy rounds itself
        moved = to_np(opt.states[0]["master"]).astype(np.float64) - to_np(start[0]).astype(np.float64)
        want = -2.0 ** -20 * np.sign(to_np(grads[0]).astype(np.float64))
        assert np.all(np.abs(moved - want) <= 2.0 ** -20 * 16 * U + 2 * U * np.abs(to_np(start[0])))
    _, params, grads, states = _make([300], bits, "b", "b", True, seed=64)
    for asked in (False, True):
        opt = ops.MoEAdamW(params, grads, state_bits=bits, states=states, master_weights=asked, **H)
        assert opt.states[0]["master"] is states[0]["master"]


def _norm_of(grads, to):
    """Writes value `to` over the first of the gradients: a norm that is not finite, or the way back."""
    grads[0].view(-1)[0] = to


@pytest.mark.parametrize("bits,n", [(32, 3), (8, 3), (32, 137), (8, 137)])
@pytest.mark.parametrize("capturable", [False, True])
def test_adamw_bias_corrections_count_the_updates_made(bits, n, capturable):
    """A step that the norm's infinity or NaN leaves undone does not count in t (one launch, and several)."""
    say(f"adamw t after skipped steps bits={bits} tensors={n} capturable={capturable}")
    sizes = [300, 5, 4000] + [1 + (i * 37) % 700 for i in range(n - 3)]
    whole, params, grads, states = _make(sizes, bits, "b", "b", True, seed=65, zero_state=True)
    opt = ops.MoEAdamW(params, grads, weight_decay=0.0, state_bits=bits, states=states, max_grad_norm=1.0,
                       capturable=capturable, **{**H, "lr": 2.0 ** -7})
    kept = float(grads[0][0])
    done = 0
    for bad in (float("inf"), None, float("nan"), -float("inf"), None, None):
        _norm_of(grads, kept if bad is None else bad)
        start = [w.clone() for w in whole]
        before = _snapshot(params, grads, states)
        opt.step()
        torch.cuda.synchronize()
        if bad is not None:
            assert all(torch.equal(a, b) for a, b, g in zip(start, whole, whole) if not torch.isnan(g.float()).any())
            assert all(np.array_equal(to_np(p), b[0]) for p, b in zip(params, before))
            continue
        done += 1
        _check_step(before, params, states, bits, [0.0] * n, done, scale=float(opt.grad_norm[1]), lr=2.0 ** -7)
        assert opt.updates_done() == done
    assert opt.step_count == 6 and int(opt.skipped) == 3


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_captured_steps_that_are_skipped(bits):
    say(f"adamw graph with skipped steps bits={bits}")
    whole, params, grads, states = _make([700, 3, 5000], bits, "b", "b", True, seed=66, zero_state=True)
    opt = ops.MoEAdamW(params, grads, weight_decay=0.1, state_bits=bits, states=states, max_grad_norm=0.05,
                       capturable=True, **H)
    kept = float(grads[0][0])
    _norm_of(grads, float("inf"))
    opt.step()  # warms up, and leaves everything as it is
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    opt.step_dev.zero_()
    opt.skipped.zero_()
    for i, bad in enumerate((float("inf"), float("nan"), None, float("inf"), None)):
        _norm_of(grads, kept if bad is None else bad)
        before = _snapshot(params, grads, states)
        graph.replay()
        torch.cuda.synchronize()
        if bad is None:
            _check_step(before, params, states, bits, [0.1] * 3, {2: 1, 4: 2}[i], scale=float(opt.grad_norm[1]))
    assert int(opt.step_dev) == 5 and int(opt.skipped) == 3 and opt.updates_done() == 2


def test_adamw_skipped_counts_once_a_step_of_both_kinds():
    """Tensors with 32-bit and with 8-bit states in one call: two launches, one step."""
    say("adamw skipped steps of both kinds")
    made = [_make([3000, 40], bits, "b", "b", True, seed=67 + bits) for bits in (32, 8)]
    opts = [ops.MoEAdamW(p, g, state_bits=bits, states=s, **H) for bits, (_, p, g, s) in zip((32, 8), made)]
    norm = torch.tensor([float("inf"), float("nan")], device=DEV)
    skipped = torch.full((1,), 4, dtype=torch.int64, device=DEV)
    start = [w.clone() for m in made for w in m[0]]
    for order in ((0, 1), (1, 0), (0,), (1,)):
        tensors = [opts[o].tensors[i] for o in order for i in range(2)]
        arr = (ops.MoeAdamwTensor * len(tensors))(*tensors)
        skipped.fill_(4)
        h = ops.MoeAdamwHparams(1e-2, 0.9, 0.99, 1e-8, 7, None, None, norm.data_ptr(), skipped.data_ptr())
        ops.moe_adamw_step(arr, len(tensors), h)
        assert int(skipped) == 5, order
    assert all(torch.equal(a, b) for a, b in zip(start, (w for m in made for w in m[0])))
    # a norm to go by again: t is 7 - 5 for both kinds
    norm.copy_(torch.tensor([1.0, 0.5]))
    before = [_snapshot(p, g, s) for _, p, g, s in made]
    tensors = [o.tensors[i] for o in opts for i in range(2)]
    ops.moe_adamw_step((ops.MoeAdamwTensor * 4)(*tensors), 4, h)
    torch.cuda.synchronize()
    assert int(skipped) == 5
    for bits, b, (_, p, _, s) in zip((32, 8), before, made):
        _check_step(b, p, s, bits, [0.01, 0.01], 2, scale=0.5)


def test_adamw_refuses_gradients_whose_memory_was_replaced():
    """As for parameters: the memory that the optimizer was built with would be read, an old gradient."""
    say("adamw refuses replaced gradients")
    for kw in (dict(), dict(max_grad_norm=1.0), dict(capturable=True)):
        p, g = torch.ones(100, device=DEV), torch.ones(100, device=DEV)
        opt = ops.MoEAdamW([p], [g], **{**H, **kw})
        opt.step()
        kept, old = p.clone(), g.data
        g.data = torch.full((100,), 7.0, device=DEV)
        with pytest.raises(RuntimeError, match="gradient's memory has been replaced"):
            opt.step()
        assert torch.equal(p, kept) and opt.step_count == 1
        assert not opt.capturable or int(opt.step_dev) == 1
        g.data = old
        opt.step()
        assert opt.step_count == 2


def test_adamw_refuses_a_norm_that_is_no_float_and_counts_no_refused_step():
    say("adamw max_grad_norm below the floats")
    p, g = torch.ones(100, device=DEV), torch.ones(100, device=DEV)
    for capturable in (False, True):
        with pytest.raises(ValueError, match="max_grad_norm"):
            ops.MoEAdamW([p], [g], max_grad_norm=1e-60, capturable=capturable, **H)
        ops.MoEAdamW([p], [g], max_grad_norm=1e60, capturable=capturable, **H).step()  # infinity: no clipping
    opt = ops.MoEAdamW([p], [g], max_grad_norm=1.0, capturable=True, **H)
    opt.max_grad_norm = -1.0
    with pytest.raises(ops.MoEError, match="max_norm"):
        opt.step()
    assert int(opt.step_dev) == 0 and opt.step_count == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_steps_under_a_norm_past_the_floats(bits):
    """Finite gradients whose norm no float holds: grad_norm[0] is infinite, the factor and the step are not."""
    say(f"adamw norm past the floats bits={bits}")
    n = 3000
    gen = torch.Generator(device=DEV).manual_seed(71)
    p = torch.randn(n, generator=gen, device=DEV)
    g = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.5, -1e38, 1e38)
    opt = ops.MoEAdamW([p], [g], weight_decay=0.1, state_bits=bits, max_grad_norm=1.0, **H)
    before = _snapshot([p], [g], opt.states)
    opt.step()
    torch.cuda.synchronize()
    norm, scale = oracle.grad_norm([before[0][1]], 1.0)
    got = to_np(opt.grad_norm)
    assert np.isinf(got[0]) and abs(got[1] - scale) <= 1.5e-45  # one step among the smallest floats
    assert int(opt.skipped) == 0
    _check_step(before, [p], opt.states, bits, [0.1], 1, scale=float(got[1]))


@pytest.mark.parametrize("bits,gdt", [(32, torch.float32), (32, torch.bfloat16), (8, torch.float32)])
def test_adamw_steps_and_states_past_32_bits(bits, gdt):
    """More than 2^31 values, zero but for four places: the start, one far before 2^31, the values around it, the end.
    Two steps of weights, copies, both states and their scales against the oracle's, and the states read back."""
    n = 2 ** 31 + 777
    say(f"adamw bits={bits} gradients {gdt}, 2^31 + 777 values")
    places = [(0, 512), (2 ** 30 + 256, 2 ** 30 + 1024), (2 ** 31 - 512, 2 ** 31 + 256), (2 ** 31 + 512, n)]
    gen = torch.Generator(device=DEV).manual_seed(74)
    p, g = torch.zeros(n, dtype=torch.bfloat16, device=DEV), torch.zeros(n, dtype=gdt, device=DEV)
    for a, b in places:
        p[a:b] = torch.randn(b - a, generator=gen, device=DEV).bfloat16()
        g[a:b] = torch.randn(b - a, generator=gen, device=DEV).to(gdt)
    opt = ops.MoEAdamW([p], [g], weight_decay=0.1, state_bits=bits, master_weights=True, max_grad_norm=1.0, **H)
    s = opt.states[0]
    parts = [(p[a:b], g[a:b], {k: t[a // 256:-(-b // 256)] if k.endswith("scale") else t[a:b] for k, t in s.items()})
             for a, b in places]
    cut = [list(x) for x in zip(*parts)]
    for t in (1, 2):
        before = _snapshot(*cut)
        opt.step()
        torch.cuda.synchronize()
        norm, _ = oracle.grad_norm([b[1] for b in before], 1.0)
        assert abs(float(opt.grad_norm[0]) - norm) <= 2 * U * norm
        _check_step(before, cut[0], cut[2], bits, [0.1] * len(places), t, scale=float(opt.grad_norm[1]))
        g.mul_(-0.75)
    live = sum(b - a for a, b in places)
    for name, x in [("param", p)] + list(s.items()):
        assert int(torch.count_nonzero(x)) <= (live + 255 if name.endswith("scale") else live), name
    if bits == 8:
        m, v = opt.read_states()
        for (a, b), st in zip(places, cut[2]):
            assert np.array_equal(to_np(m[0][a:b]), oracle.read_m(to_np(st["m"]), to_np(st["m_scale"])).astype(np.float32))
            assert np.array_equal(to_np(v[0][a:b]), oracle.read_v(to_np(st["v"]), to_np(st["v_scale"])).astype(np.float32))
        assert int(torch.count_nonzero(m[0])) <= live and int(torch.count_nonzero(v[0])) <= live


@pytest.mark.parametrize("beta2", [0.9, 0.95, 0.98, 0.99, 0.992, 0.993, 0.999])
def test_adamw_8bit_v_falls_where_the_formula_says(beta2):
    """Codes 1 .. 255 of v without gradients, beside a largest that stays: a step lowers a code where its v' = beta2 v
    is past the border (c (c - 1) + 1/2)^2 below it, and nowhere else; after many steps the codes above are gone."""
    say(f"adamw 8-bit v falling, beta2={beta2}")
    codes = np.arange(256)
    codes[0] = 255  # the block's largest, under a gradient that keeps it
    p, g = torch.ones(256, device=DEV), torch.zeros(256, device=DEV)
    g[0] = 1.0
    s = dict(m=torch.zeros(256, dtype=torch.int8, device=DEV), m_scale=torch.zeros(1, device=DEV),
             v=torch.tensor(codes, dtype=torch.uint8, device=DEV), v_scale=torch.ones(1, device=DEV))
    opt = ops.MoEAdamW([p], [g], lr=0.0, betas=(0.9, beta2), state_bits=8, states=[s])
    opt.step()
    c = np.arange(1, 256).astype(np.float64)
    falls = beta2 * c ** 4 < (c * (c - 1) + 0.5) ** 2  # no code is within 1e-8 of it
    falls[0] = False                                   # above zero: one at least
    assert np.array_equal(to_np(s["v"])[1:] < codes[1:], falls)
    assert falls.any() == (beta2 < 0.9922) and (beta2 != 0.95 or falls.nonzero()[0][0] + 1 == 39)
    for _ in range(260):
        opt.step()
    left = to_np(s["v"])[1:]
    if falls.any():
        assert np.array_equal(left, np.minimum(codes[1:], falls.nonzero()[0][0]))  # codes below the lowest that falls
    else:
        assert np.array_equal(left, codes[1:])


@pytest.mark.parametrize("beta2", [0.95, 0.98])
def test_adamw_8bit_v_follows_32_bits_over_many_steps(beta2):
    """300 steps of the same gradients, half of which shrink tenfold: v in 8 bits is off from v in 32 by no more than
    each step's half cell (c^2 + c + 1/2)^2 - c^4 of scale / 255^4, carried on by beta2 (and 6 u of v a step)."""
    n, steps = 256 * 40, 300
    gen = torch.Generator(device=DEV).manual_seed(76)
    p = torch.zeros(n, device=DEV)
    grad = torch.zeros(n, device=DEV)
    opts = [ops.MoEAdamW([p.clone()], [grad], lr=0.0, betas=(0.9, beta2), state_bits=bits) for bits in (8, 32)]
    size = torch.exp(torch.randn(n, generator=gen, device=DEV))
    bound = torch.zeros(n, dtype=torch.float64, device=DEV)
    s8, s32 = opts[0].states[0], opts[1].states[0]
    for t in range(steps):
        if t == 100:
            size[::2] *= 0.1
        grad.copy_(torch.randn(n, generator=gen, device=DEV) * size)
        for o in opts:
            o.step()
        c = s8["v"].double()
        cell = ((c * c + c + 0.5) ** 2 - c ** 4) * (s8["v_scale"].double() / 255.0 ** 4).repeat_interleave(256)
        bound = beta2 * bound + cell * (1 + 4 * U)  # (the scale is the largest rounded to a float)
    v8 = opts[0].read_states()[1][0].double()
    v32 = s32["v"].double()
    assert torch.all((v8 - v32).abs() <= bound + 2 * U * v8 + 6 * U * steps * v32)
    off = (v8.sqrt() / v32.sqrt() - 1).abs()
    print(f"root of v off: median {float(off.median()):.4f}")


@pytest.mark.parametrize("largest", [1e-3, 0.5, 100.0, 3e4, 1e9])
def test_adamw_8bit_tiny_values_beside_large_ones(largest):
    """A block's smallest v' may be below the smallest normal float while its largest is above one: roots of 1e-20 and
    up weigh against an eps of 1e-16 all the same."""
    say(f"adamw 8-bit tiny values beside {largest}")
    rng = np.random.default_rng(77)
    n, lr, b1, b2, eps = 512, 1.0, 0.9, 0.99, 1e-16
    g = rng.standard_normal(n) * 10.0 ** -rng.uniform(15, 20, n)
    g[[5, 300]] = largest
    p, gd = torch.zeros(n, device=DEV), torch.tensor(g, dtype=torch.float32, device=DEV)
    opt = ops.MoEAdamW([p], [gd], lr=lr, betas=(b1, b2), eps=eps, weight_decay=0.0, state_bits=8)
    opt.step()
    torch.cuda.synchronize()
    z = np.zeros(n)
    w, m, v = oracle.adamw_step(z, to_np(gd).astype(np.float64), z, z, 1, lr, b1, b2, eps, 0.0)
    assert v.min() < 1e-38
    bound = 16 * U * lr / (1 - b1) * np.abs(m) / (np.sqrt(v) / np.sqrt(1 - b2) + eps) + 1e-44
    assert np.all(np.abs(to_np(p) - w) <= bound), (np.abs(to_np(p) - w) / bound).max()
    (cm, sm), (cv, sv), s = oracle.held_m(m), oracle.held_v(v), opt.states[0]
    assert np.array_equal(to_np(s["m_scale"]), sm) and np.array_equal(to_np(s["v_scale"]), sv)
    assert np.array_equal(to_np(s["m"]), cm) and np.array_equal(to_np(s["v"]), cv)


def test_adamw_8bit_scales_next_to_the_largest_float():
    """A block of m whose scale's reciprocal is below the smallest normal float (states that were given so)."""
    say("adamw 8-bit m_scale 3e38")
    n = 512
    c = (np.arange(n) % 255 - 127).astype(np.int8)
    c[[0, 256]] = 127
    s = dict(m=torch.tensor(c, device=DEV), m_scale=torch.tensor([3e38, 9e37], device=DEV),
             v=torch.full((n,), 255, dtype=torch.uint8, device=DEV), v_scale=torch.full((2,), 1e38, device=DEV))
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    before = _snapshot([p], [g], [s])
    opt = ops.MoEAdamW([p], [g], lr=1e-2, betas=(0.99, 0.99), eps=1e-8, weight_decay=0.0, state_bits=8, states=[s])
    opt.step()
    torch.cuda.synchronize()
    m = 0.99 * oracle.read_m(before[0][2]["m"], before[0][2]["m_scale"])
    cm, sm = oracle.held_m(m)
    assert np.array_equal(to_np(s["m_scale"]), sm) and np.array_equal(to_np(s["m"]), cm) and np.abs(cm).max() == 127


# ------------------------------------------------------------------------------ the run together

def _layer(T=300, d=128, E=8, k=2, f=192, cf=1.25, fs=64, seed=4, **kw):
    w = wl.Workload("train", T, d, E, k, f, cf, "bf16", d_ff_shared=fs, offset="boost4", **kw)
    inp = wl.make_inputs(w, seed=seed, device=DEV)
    return w, inp, ops.moe_capacity(T, E, cf)


def test_backward_with_dlogits_of_zeros_is_the_backward():
    say("backward with a zero gradient on the logits")
    w, inp, cap = _layer()
    tr = ops.MoETrainer(inp, cap)
    dy = torch.randn((300, 128), device=DEV).bfloat16()
    tr.forward()
    args = (tr.layer.desc, inp.w_router, inp.w_gate_up, inp.w_down, inp.x, tr.layer.routing, dy)
    got = []
    for dl in (None, torch.zeros_like(tr.dlogits)):
        dx = torch.empty_like(inp.x)
        grads = {n: torch.empty_like(t) for n, t in tr.grads.items()}
        ops.moe_backward(*args, dx, grads, tr.backward_ws, w_shared_gate_up=inp.w_shared_gate_up,
                         w_shared_down=inp.w_shared_down, dlogits=dl)
        got.append([dx] + list(grads.values()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("T,k,off,overflow", [(300, 2, None, "drop"), (257, 1, [0, 100, 250], "drop"),
                                              (300, 2, [0, 140, 300], "reroute")])
def test_layer_gradients_with_the_balance_loss(T, k, off, overflow):
    """dx, dW_router and the experts' gradients of sum(dy out) + balance + z against the oracle's."""
    say(f"training gradients T={T} k={k} S={1 if off is None else len(off) - 1} {overflow}")
    w, inp, cap = _layer(T=T, k=k)
    mask = np.random.default_rng(5).random(T) < 0.8
    alpha, z = 30.0, 2.0  # large, so that the losses' gradients weigh as much as the layer's
    tr = ops.MoETrainer(inp, cap, alpha=alpha, z_coeff=z, overflow=overflow,
                        seq_offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV),
                        token_mask=torch.as_tensor(mask).to(DEV))
    dy = torch.randn((T, 128), generator=torch.Generator(device=DEV).manual_seed(6), device=DEV).bfloat16()
    tr.forward()
    dx = tr.backward(dy)
    torch.cuda.synchronize()
    h = lambda t: to_np(t).astype(np.float64)  # noqa: E731
    ids = to_np(tr.layer.routing["topk_ids"])
    ref = oracle.moe_backward(h(inp.x), h(inp.w_router), HostExperts(inp.w_gate_up), HostExperts(inp.w_down), k, cap,
                              h(dy), h(inp.logit_offset), w_shared_gate_up=h(inp.w_shared_gate_up),
                              w_shared_down=h(inp.w_shared_down), ids=ids, overflow=overflow)
    logits = oracle.router_logits(h(inp.x), h(inp.w_router), h(inp.logit_offset))
    bal = oracle.balance_loss(logits, ids, 8, alpha, z, mask, off)
    assert np.array_equal(to_np(tr.counts), bal["counts"])
    # logits are float sums of bf16 products here: off by some 1e-6
    assert np.allclose(to_np(tr.losses), bal["losses"], rtol=1e-4)
    assert row_rel_err(to_np(dx), ref["dx"] + bal["dlogits"] @ h(inp.w_router)) <= BF16_TOL
    assert row_rel_err(to_np(tr.grads["dw_router"]), ref["dw_router"] + bal["dlogits"].T @ h(inp.x)) <= BF16_TOL
    gu = to_np(tr.grads["dw_gate_up"])
    assert max(row_rel_err(gu[e], ref["dw_gate_up"][e]) for e in range(8)) <= BF16_TOL


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_run(bits):
    """Three steps with tile-major copies: the weights follow AdamW from the gradients on the device, the next
    forward reads the new weights, and a fresh layer with them gives its outputs bit for bit."""
    say(f"training steps bits={bits}")
    w, inp, cap = _layer(T=700, d=256, E=2, f=256, cf=None, fs=256)  # large-tile kernels
    tr = ops.MoETrainer(inp, cap, tiled=True, shared_tiled=True, state_bits=bits, master_weights=True, lr=1e-2,
                        betas=H["betas"], eps=H["eps"], weight_decay=0.1, max_grad_norm=1.0)
    dy = torch.randn((700, 256), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV).bfloat16()
    flat = lambda: ([p.view(-1) for p in tr.optimizer.params], [g.view(-1) for g in tr.optimizer.grads],  # noqa: E731
                    [{k: x.view(-1) for k, x in s.items()} for s in tr.optimizer.states])
    for t in range(1, 4):
        tr.forward()
        tr.backward(dy)
        before = _snapshot(*flat())
        tr.step()
        torch.cuda.synchronize()
        p, _, s = flat()
        _check_step(before, p, s, bits, [0.0] + [0.1] * 4, t, scale=float(tr.optimizer.grad_norm[1]))
        after = tr.forward().clone()
        fresh = ops.MoELayer(inp, cap, tiled=True, shared_tiled=True)
        assert torch.equal(fresh.forward(), after)
        untiled = ops.MoELayer(inp, cap)
        assert row_rel_err(to_np(untiled.forward()), to_np(after).astype(np.float64)) <= BF16_TOL
    assert torch.isfinite(tr.losses).all()


def test_training_step_replays_from_a_graph():
    """The whole step captured: replays, with eager work between, follow the eager trainer bit for bit."""
    say("training step graph")
    made = []
    for _ in range(2):
        w, inp, cap = _layer(T=200, d=128, E=4, f=128, cf=1.25, fs=64)
        made.append(ops.MoETrainer(inp, cap, state_bits=8, master_weights=True, lr=1e-2, max_grad_norm=1.0,
                                   capturable=True))
    eager, other = made
    dy = torch.randn((200, 128), generator=torch.Generator(device=DEV).manual_seed(8), device=DEV).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other.train_step(dy)
    torch.cuda.current_stream().wait_stream(side)
    eager.train_step(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.train_step(dy)
    for i in range(3):
        eager.train_step(dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.optimizer.params, other.optimizer.params):
            assert torch.equal(a, b), i
        assert torch.equal(eager.losses, other.losses) and torch.equal(eager.dx, other.dx)


def test_training_step_refuses_weights_and_gradients_that_were_replaced():
    """The optimizer holds the tensors that the trainer was built with: the layer would run on others."""
    say("trainer refuses replaced weights and gradients")
    w, inp, cap = _layer(T=40, d=128, E=4, f=128)
    tr = ops.MoETrainer(inp, cap)
    dy = torch.randn((40, 128), device=DEV).bfloat16()
    tr.train_step(dy)
    for name in ("w_router", "w_gate_up", "w_down", "w_shared_gate_up", "w_shared_down"):
        old = getattr(inp, name)
        setattr(inp, name, old.clone())
        with pytest.raises(RuntimeError, match=name):
            tr.step()
        setattr(inp, name, old)
    old = tr.grads["dw_down"]
    tr.grads["dw_down"] = old.clone()
    with pytest.raises(RuntimeError, match="dw_down"):
        tr.step()
    tr.grads["dw_down"] = old
    tr.train_step(dy)
    assert tr.optimizer.step_count == 2


def test_binding_refuses_wrong_tensors():
    say("binding refusals on the device")
    desc = ops.make_desc(10, 64, 64, 4, 2, None)
    out = Outputs(10, 4, 1)
    l, i = torch.zeros((10, 4), device=DEV), torch.zeros((10, 2), dtype=torch.int32, device=DEV)
    ws = ops.workspace(ops.moe_balance_workspace_size(desc))
    with pytest.raises(ValueError, match="shape"):
        ops.moe_balance_loss(desc, l, i[:, :1].contiguous(), 1.0, 0.0, out.counts, out.seq_tokens, out.mean_probs,
                             out.losses, ws)
    with pytest.raises(ValueError, match="dtype"):
        ops.moe_balance_loss(desc, l.double(), i, 1.0, 0.0, out.counts, out.seq_tokens, out.mean_probs, out.losses, ws)
    w = wl.Workload("f32", 8, 16, 2, 1, 16, None, "f32")
    with pytest.raises(ValueError, match="bf16"):
        ops.MoETrainer(wl.make_inputs(w, device=DEV), None)
    p = torch.zeros(8, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        ops.MoEAdamW([torch.zeros((4, 4), device=DEV).t()], [torch.zeros((4, 4), device=DEV)])
    with pytest.raises(ValueError, match="dtype"):
        ops.MoEAdamW([p.half()], [p])
    with pytest.raises(ValueError, match="values"):
        ops.MoEAdamW([p], [torch.zeros(9, device=DEV)])
    with pytest.raises(ops.MoEError, match="aligned"):
        ops.MoEAdamW([torch.zeros(9, device=DEV)[1:]], [p])
    with pytest.raises(ops.MoEError, match="overlaps"):
        ops.MoEAdamW([p, p], [torch.zeros(8, device=DEV)] * 2)
    with pytest.raises(ops.MoEError, match="overlaps"):
        ops.MoEAdamW([p], [p])

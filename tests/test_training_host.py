"""CPU tests of the training operators: pins of their oracle (automatic differentiation, central
differences, an independent optimizer, brute force over the 8-bit levels), and the argument
checks of their C entry points, which return before any device work."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle

ops = pytest.importorskip("sparse_mixture_experts_level_amd.ops")
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
needs_lib = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="libmoe.so not built")


# ------------------------------------------------------------------------------ oracle pins

def _batch(rng, T, E, k, masked=False):
    l = rng.standard_normal((T, E)) * 2
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    return l, ids, (rng.random(T) < 0.7 if masked else None)


def test_balance_of_one_sequence_is_the_aux_loss():
    rng = np.random.default_rng(0)
    l, ids, _ = _batch(rng, 57, 9, 3)
    r = oracle.balance_loss(l, ids, 9, 0.02, 0.0)
    assert r["losses"][0] == pytest.approx(oracle.aux_load_balancing_loss(ids, oracle.softmax(l), 9, 0.02), rel=1e-12)
    assert r["counts"].sum() == 57 * 3 and r["seq_tokens"].tolist() == [57]


@pytest.mark.parametrize("masked,off", [(False, None), (True, None), (True, [0, 5, 5, 17, 29]), (False, [3, 10, 26])])
def test_balance_gradient_against_autograd_and_differences(masked, off):
    rng = np.random.default_rng(1)
    T, E, k = 29, 6, 2
    l, ids, mask = _batch(rng, T, E, k, masked)
    up = (0.7, 1.3)
    r = oracle.balance_loss(l, ids, E, 0.05, 0.01, mask, off, up)

    # written apart, differentiated by torch (f held fixed: counts carry no gradient)
    x = torch.tensor(l, requires_grad=True)
    bounds = [0, T] if off is None else off
    terms, z, n_all = [], [], 0
    for a, b in zip(bounds, bounds[1:]):
        keep = torch.tensor([t for t in range(a, b) if mask is None or mask[t]], dtype=torch.long)
        if keep.numel() == 0:
            continue
        n_all += keep.numel()
        f = torch.bincount(torch.tensor(ids)[keep].reshape(-1), minlength=E).double() / (keep.numel() * k)
        terms.append((f * torch.softmax(x[keep], 1).mean(0)).sum())
        z.append(torch.logsumexp(x[keep], 1).square().sum())
    losses = torch.stack([0.05 * E * torch.stack(terms).mean(), 0.01 * torch.stack(z).sum() / n_all])
    assert np.allclose(losses.detach().numpy(), r["losses"], rtol=1e-12)
    grad, = torch.autograd.grad((losses * torch.tensor(up, dtype=torch.float64)).sum(), x)
    assert np.allclose(grad.numpy(), r["dlogits"], rtol=1e-10, atol=1e-15)

    # central differences (ids fixed): error h^2 / 6 times the third derivative, some 1e-9 here
    h = 1e-4
    for t, e in [(0, 0), (4, 3), (12, 5), (28, 1)]:
        up_l, dn_l = l.copy(), l.copy()
        up_l[t, e] += h
        dn_l[t, e] -= h
        d = [oracle.balance_loss(q, ids, E, 0.05, 0.01, mask, off)["losses"] @ np.array(up) for q in (up_l, dn_l)]
        assert (d[0] - d[1]) / (2 * h) == pytest.approx(r["dlogits"][t, e], abs=1e-8)


def test_balance_of_nothing_is_zero():
    l, ids, _ = _batch(np.random.default_rng(2), 7, 4, 2)
    r = oracle.balance_loss(l, ids, 4, 0.1, 0.1, np.zeros(7, dtype=bool))
    assert not r["losses"].any() and not r["dlogits"].any() and not r["counts"].any()


def test_adamw_against_torch():
    rng = np.random.default_rng(3)
    w = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.tensor(w))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1, foreach=False)
    m = v = np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        w, m, v = oracle.adamw_step(w, g, m, v, t, 3e-3, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p.detach().numpy(), w, rtol=1e-12, atol=1e-14)


def test_grad_norm_and_clipping():
    n, c = oracle.grad_norm([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert n == 5.0 and c == pytest.approx(1 / 5.000001, rel=1e-12)
    assert oracle.grad_norm([np.array([0.1])], 1.0)[1] == 1.0
    assert np.isnan(oracle.grad_norm([np.array([np.inf])], 1.0)[1])


def test_held_states():
    rng = np.random.default_rng(4)
    m = rng.standard_normal(700) * np.exp(rng.standard_normal(700) * 3)
    c, s = oracle.held_m(m)
    assert len(s) == 3 and np.abs(c).max() == 127
    back = oracle.read_m(c, s)
    # neighbours are (2 c + 1) / 127^2 of the scale apart: off by half of that at most, and by the scale's rounding
    step = (2 * np.abs(c) + 1) / 127.0 ** 2 * np.repeat(s.astype(np.float64), 256)[:700]
    assert np.all(np.abs(back - m) <= step / 2 * (1 + 1e-5) + np.abs(m) * 2.0 ** -23)
    v = m * m
    c, s = oracle.held_v(v)
    root, held = np.sqrt(v), np.sqrt(oracle.read_v(c, s))
    step = (2 * c + 1) / 255.0 ** 2 * np.sqrt(np.repeat(s.astype(np.float64), 256)[:700])
    assert np.all(np.abs(held - root)[c > 1] <= (step / 2 * (1 + 1e-5) + root * 2.0 ** -23)[c > 1])
    assert c.min() >= 1  # above zero: never held as zero
    assert oracle.held_v(np.zeros(5))[0].tolist() == [0] * 5 and oracle.held_m(np.full(3, 1e-39))[1].tolist() == [0.0]
    assert np.isnan(oracle.held_m(np.array([1.0, np.nan]))[1][0])


# ----------------------------------------------------------------------------------- refusals

def _desc(**kw):
    base = dict(num_tokens=64, d_model=128, d_ff=256, num_experts=8, top_k=2, capacity=-1, d_ff_shared=0,
                dtype=ops.MOE_DTYPE_BF16)
    base.update(kw)
    return ops.MoeDesc(**base)


def _last():
    return ops.lib().moe_last_error().decode()


def _loss(desc=None, logits=FAKE, ids=FAKE, mask=None, off=None, S=1, alpha=0.1, z=0.1, counts=FAKE, tokens=FAKE,
          probs=FAKE, losses=FAKE, dlogits=None, ws=FAKE, nbytes=1 << 30):
    return ops.lib().moe_balance_loss(ctypes.byref(desc or _desc()), logits, ids, mask, off, S, alpha, z, counts,
                                      tokens, probs, losses, dlogits, ws, nbytes, None)


@needs_lib
@pytest.mark.parametrize("kw,status,word", [
    (dict(logits=None), ops.MOE_ERR_INVALID, "logits"),
    (dict(logits=FAKE + 4), ops.MOE_ERR_INVALID, "aligned"),
    (dict(ids=None), ops.MOE_ERR_INVALID, "topk_ids"),
    (dict(mask=FAKE + 1), ops.MOE_ERR_INVALID, "token_mask"),
    (dict(off=FAKE + 4), ops.MOE_ERR_INVALID, "seq_offsets"),
    (dict(S=0), ops.MOE_ERR_INVALID, "num_seqs"),
    (dict(S=2), ops.MOE_ERR_INVALID, "without seq_offsets"),
    (dict(off=FAKE, S=ops.MOE_MAX_SEQS + 1), ops.MOE_ERR_INVALID, "num_seqs"),
    (dict(alpha=float("nan")), ops.MOE_ERR_INVALID, "alpha"),
    (dict(z=float("inf")), ops.MOE_ERR_INVALID, "z_coeff"),
    (dict(counts=None), ops.MOE_ERR_INVALID, "counts"),
    (dict(tokens=None), ops.MOE_ERR_INVALID, "seq_tokens"),
    (dict(probs=None), ops.MOE_ERR_INVALID, "mean_probs"),
    (dict(losses=None), ops.MOE_ERR_INVALID, "losses"),
    (dict(dlogits=FAKE + 8), ops.MOE_ERR_INVALID, "dlogits"),
    (dict(dlogits=FAKE), ops.MOE_ERR_INVALID, "overlaps"),
    (dict(ws=None), ops.MOE_ERR_WORKSPACE, "workspace"),
    (dict(nbytes=8), ops.MOE_ERR_WORKSPACE, "workspace"),
    (dict(desc=_desc(top_k=9)), ops.MOE_ERR_INVALID, "top_k"),
])
def test_balance_loss_refusals(kw, status, word):
    assert _loss(**kw) == status
    assert word in _last()


@needs_lib
def test_balance_of_an_empty_batch_needs_its_outputs_only():
    d = _desc(num_tokens=0)
    for name in ("counts", "tokens", "probs", "losses"):
        assert _loss(d, None, None, ws=None, nbytes=0, **{name: None}) == ops.MOE_ERR_INVALID
    L = ops.lib()
    assert L.moe_balance_loss_backward(ctypes.byref(d), None, None, None, 1, None, None, 0.1, 0.1, None, None,
                                       None) == ops.MOE_OK


@needs_lib
def test_balance_backward_refusals():
    L, d = ops.lib(), _desc()

    def call(logits=FAKE, mask=None, off=None, S=1, counts=FAKE, tokens=FAKE, alpha=0.1, z=0.1, dloss=None, dl=FAKE):
        return L.moe_balance_loss_backward(ctypes.byref(d), logits, mask, off, S, counts, tokens, alpha, z, dloss, dl,
                                           None)
    for kw, word in [(dict(logits=None), "logits"), (dict(counts=None), "counts"), (dict(tokens=None), "seq_tokens"),
                     (dict(dl=None), "dlogits"), (dict(dl=FAKE), "overlaps"), (dict(dl=FAKE + 16), "overlaps"),
                     (dict(dl=FAKE - 16), "overlaps"), (dict(dloss=FAKE + 4), "dloss"), (dict(S=3), "seq_offsets"),
                     (dict(alpha=float("inf")), "alpha")]:
        assert call(**kw) == ops.MOE_ERR_INVALID
        assert word in _last()


@needs_lib
def test_balance_workspace_size():
    assert ops.moe_balance_workspace_size(_desc(), 1) > 0
    assert ops.moe_balance_workspace_size(_desc(), 0) == 0
    assert ops.moe_balance_workspace_size(_desc(), ops.MOE_MAX_SEQS + 1) == 0
    assert ops.moe_balance_workspace_size(_desc(num_experts=0), 1) == 0
    assert ops.moe_balance_workspace_size(_desc(), 64) > ops.moe_balance_workspace_size(_desc(), 1)


@needs_lib
def test_backward_with_dlogits_refuses_what_the_backward_refuses():
    L, d = ops.lib(), _desc()
    W, R, G = ops.MoeWeights(), ops.MoeRouting(), ops.MoeGrads()
    call = lambda desc, dl: L.moe_backward_with_dlogits(  # noqa: E731
        ctypes.byref(desc), ctypes.byref(W), FAKE, ctypes.byref(R), FAKE, dl, FAKE, ctypes.byref(G), FAKE, 1 << 40, None)
    assert call(d, None) == ops.MOE_ERR_INVALID and "dlogits" in _last()
    assert call(d, FAKE) == ops.MOE_ERR_INVALID and "w_router" in _last()
    assert call(_desc(dtype=ops.MOE_DTYPE_F32), FAKE) == ops.MOE_ERR_UNSUPPORTED


def _views(*entries):
    return (ops.MoeGradView * len(entries))(*[ops.MoeGradView(*e) for e in entries])


@needs_lib
def test_grad_norm_refusals():
    L = ops.lib()
    good = (FAKE, 100, ops.MOE_DTYPE_BF16, 0)
    assert L.moe_grad_norm_workspace_size(_views(good), 1) > 0
    for entry, status, word in [((None, 5, 0, 0), ops.MOE_ERR_INVALID, "NULL"),
                                ((FAKE + 2, 5, 1, 0), ops.MOE_ERR_INVALID, "aligned"),
                                ((FAKE, -1, 1, 0), ops.MOE_ERR_INVALID, "< 0"),
                                ((FAKE, (1 << 33) + 1, 1, 0), ops.MOE_ERR_UNSUPPORTED, "2^33"),
                                ((FAKE, 5, 7, 0), ops.MOE_ERR_UNSUPPORTED, "dtype")]:
        v = _views(good, entry)
        assert L.moe_grad_norm_workspace_size(v, 2) == 0
        assert L.moe_grad_norm(v, 2, 1.0, FAKE, FAKE, 1 << 20, None) == status
        assert word in _last() and "grads[1]" in _last()
    v = _views(good)
    for bad in (0.0, -1.0, float("nan")):
        assert L.moe_grad_norm(v, 1, bad, FAKE, FAKE, 1 << 20, None) == ops.MOE_ERR_INVALID
    assert L.moe_grad_norm(v, 1, 1.0, None, FAKE, 1 << 20, None) == ops.MOE_ERR_INVALID
    assert L.moe_grad_norm(v, 1, 1.0, FAKE, None, 0, None) == ops.MOE_ERR_WORKSPACE
    assert L.moe_grad_norm(v, 1, 1.0, FAKE, FAKE, 8, None) == ops.MOE_ERR_WORKSPACE
    assert L.moe_grad_norm(v, -1, 1.0, FAKE, FAKE, 1 << 20, None) == ops.MOE_ERR_INVALID
    assert L.moe_grad_norm(None, 1, 1.0, FAKE, FAKE, 1 << 20, None) == ops.MOE_ERR_INVALID


def _tensor(**kw):
    n = kw.pop("n", 1000)
    base = dict(param=0x100000, grad=0x200000, master=None, m=0x300000, v=0x400000, m_scale=0x500000, v_scale=0x600000,
                n=n, param_dtype=ops.MOE_DTYPE_BF16, grad_dtype=ops.MOE_DTYPE_BF16, state_bits=8, weight_decay=0.1)
    base.update(kw)
    return ops.MoeAdamwTensor(**base)


def _tensors(*t):
    return (ops.MoeAdamwTensor * len(t))(*t)


@needs_lib
@pytest.mark.parametrize("kw,status,word", [
    (dict(param=None), ops.MOE_ERR_INVALID, "param is NULL"),
    (dict(grad=0x200004), ops.MOE_ERR_INVALID, "grad is not 16-byte aligned"),
    (dict(m=None), ops.MOE_ERR_INVALID, "m is NULL"),
    (dict(v=None), ops.MOE_ERR_INVALID, "v is NULL"),
    (dict(m_scale=None), ops.MOE_ERR_INVALID, "m_scale is NULL"),
    (dict(v_scale=None), ops.MOE_ERR_INVALID, "v_scale is NULL"),
    (dict(master=0x700004), ops.MOE_ERR_INVALID, "master is not"),
    (dict(n=-1), ops.MOE_ERR_INVALID, "< 0"),
    (dict(n=(1 << 33) + 1), ops.MOE_ERR_UNSUPPORTED, "2^33"),
    (dict(param_dtype=5), ops.MOE_ERR_UNSUPPORTED, "dtype"),
    (dict(grad_dtype=-1), ops.MOE_ERR_UNSUPPORTED, "dtype"),
    (dict(state_bits=16), ops.MOE_ERR_UNSUPPORTED, "state_bits"),
    (dict(weight_decay=-0.1), ops.MOE_ERR_INVALID, "weight_decay"),
    (dict(weight_decay=float("nan")), ops.MOE_ERR_INVALID, "weight_decay"),
    (dict(master=0x700000, param_dtype=ops.MOE_DTYPE_F32), ops.MOE_ERR_INVALID, "master"),
    # overlaps: within one tensor, a gradient with a state, the end of a range
    (dict(m=0x100000), ops.MOE_ERR_INVALID, "overlaps"),
    (dict(grad=0x100010), ops.MOE_ERR_INVALID, "overlaps"),
    (dict(v=0x300000 + 992), ops.MOE_ERR_INVALID, "overlaps"),
    (dict(v_scale=0x500000), ops.MOE_ERR_INVALID, "overlaps"),
])
def test_adamw_tensor_refusals(kw, status, word):
    L = ops.lib()
    first = _tensor(**{f: getattr(_tensor(), f) + 0x1000000 for f in ("param", "grad", "m", "v", "m_scale", "v_scale")})
    t = _tensors(first, _tensor(**kw))
    assert L.moe_adamw_check_tensors(t, 2) == status
    assert word in _last() and "tensors[1]" in _last()
    if word != "overlaps":
        h = ops.MoeAdamwHparams(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None)
        assert L.moe_adamw_step(t, 2, ctypes.byref(h), None) == status


@needs_lib
def test_adamw_tensors_that_touch_or_share_a_gradient_are_fine():
    a = _tensor()
    b = _tensor(param=0x100000 + 2000, m=0x300000 + 1008, v=0x400000 + 1008, m_scale=0x500010, v_scale=0x600010)
    ops.moe_adamw_check_tensors(_tensors(a, b), 2)  # the same gradient for both
    ops.moe_adamw_check_tensors(_tensors(_tensor(n=0, param=None, m=None)), 1)
    ops.moe_adamw_check_tensors((ops.MoeAdamwTensor * 1)(), 0)


@needs_lib
def test_adamw_refuses_the_same_tensor_twice():
    L = ops.lib()
    h = ops.MoeAdamwHparams(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None)
    t = _tensors(_tensor(), _tensor(m=0x800000, v=0x900000, m_scale=0xa00000, v_scale=0xb00000))
    assert L.moe_adamw_step(t, 2, ctypes.byref(h), None) == ops.MOE_ERR_INVALID
    assert "tensors[1].param overlaps" in _last() or "tensors[0].param overlaps" in _last()


@needs_lib
@pytest.mark.parametrize("kw,word", [
    (dict(lr=-1.0), "lr"), (dict(lr=float("nan")), "lr"), (dict(beta1=1.0), "beta"), (dict(beta2=-0.1), "beta"),
    (dict(eps=0.0), "eps"), (dict(step=0), "step"), (dict(lr_dev=FAKE + 4), "lr_dev"),
    (dict(step_dev=FAKE + 8), "step_dev"), (dict(norm=FAKE + 4), "norm"),
])
def test_adamw_hparam_refusals(kw, word):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, lr_dev=None, step_dev=None, norm=None)
    base.update(kw)
    h = ops.MoeAdamwHparams(**base)
    assert ops.lib().moe_adamw_step(_tensors(_tensor()), 1, ctypes.byref(h), None) == ops.MOE_ERR_INVALID
    assert word in _last()
    assert ops.lib().moe_adamw_step(_tensors(_tensor()), 1, None, None) == ops.MOE_ERR_INVALID


@needs_lib
def test_adamw_refuses_a_count_of_skipped_steps_that_is_not_aligned():
    h = ops.MoeAdamwHparams(1e-3, 0.9, 0.999, 1e-8, 1, None, None, FAKE, FAKE + 8)
    assert ops.lib().moe_adamw_step(_tensors(_tensor()), 1, ctypes.byref(h), None) == ops.MOE_ERR_INVALID
    assert "skipped" in _last()


@needs_lib
def test_adamw_read_refusals():
    L = ops.lib()
    out = (ctypes.c_void_p * 1)(FAKE)
    t32 = _tensor(state_bits=32)
    assert L.moe_adamw_read_states(_tensors(t32), 1, out, out, None) == ops.MOE_ERR_INVALID
    assert L.moe_adamw_read_states(_tensors(_tensor(m=None)), 1, out, None, None) == ops.MOE_ERR_INVALID
    assert L.moe_adamw_read_states(_tensors(_tensor(m_scale=None)), 1, out, None, None) == ops.MOE_ERR_INVALID
    bad = (ctypes.c_void_p * 1)(FAKE + 4)
    assert L.moe_adamw_read_states(_tensors(_tensor()), 1, bad, None, None) == ops.MOE_ERR_INVALID
    assert L.moe_adamw_read_states(_tensors(_tensor(param=None, grad=None)), 1, None, None, None) == ops.MOE_OK


@needs_lib
def test_debug_library_checks_the_whole_list():
    D = ops.debug_lib()
    h = ops.MoeAdamwHparams(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None)
    assert D.moe_adamw_step(_tensors(_tensor(m=0x400000)), 1, ctypes.byref(h), None) == ops.MOE_ERR_INVALID
    assert b"overlaps" in D.moe_last_error()


def test_binding_checks_types_shapes_and_device():
    x = torch.zeros((4, 8))
    for t, kinds, shape, word in [(x, torch.int32, None, "dtype"), (x, torch.float32, (4, 9), "shape"),
                                  (x.t(), torch.float32, None, "contiguous"), (x, torch.float32, (4, 8), "GPU")]:
        with pytest.raises(ValueError, match=word):
            ops._tensor(t, "x", kinds, shape)
    assert ops._tensor(None, "x", torch.float32) is None
    with pytest.raises(ValueError, match="state_bits"):
        ops.MoEAdamW([], [], state_bits=16)
    with pytest.raises(ValueError, match="one entry per tensor"):
        ops.MoEAdamW([x], [])
    with pytest.raises(ValueError, match="one value or one per tensor"):
        ops.MoEAdamW([x], [x], weight_decay=[0.1, 0.2])

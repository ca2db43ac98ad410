"""GPU parity of the norm with its backward and of the products in 8 bits against the 64-bit oracle, and of a layer
that runs them together.

Tolerances, u = 2^-24 (half a step of a float), B = 2^-8 (of bf16):
  * conversions: codes, scales and layouts equal the oracle's, which tries every level.
  * norm: h is one sum, rounded once: equal.  rstd is formed in 64 bits and rounded once: 2 u.  y adds two float roundings
    (and the output's): 4 u, or B + 4 u.  Codes are those of y formed from the call's own rstd with these two
    roundings: equal to the oracle's of that y.
  * norm backward: g, xhat and their products each rounded (8 u of the magnitudes with the rstd's), a sum over d
    by at most NV * 8 + 16 additions a thread and between threads, of magnitudes: 100 u covers it; dx within 100 u of
    |dh| + rstd (|g| + |xhat| mean |g xhat|) plus its own rounding.  dweight: at most ceil(T / 512) additions in a
    workgroup and 512 / 4 + 2 between: (T / 512 + 140) u of sum |dy xhat|.
  * products of small whole numbers (|x|, |w| <= 4, scales powers of two close together): every product and sum is exact
    in the instruction and in a float below 2^24 steps, so the bf16 outputs EQUAL the rounded oracle's.
  * products of normal rows: within a lane's 16 products what lies below 2^-13 of the largest may be lost, 15 * 2^-13 <
    2^-9 of the largest: |err| <= B |y| + 2^-9 sum |x w|, and over all values, where losses average out (1.5e-5) and
    roundings are spread evenly over half a step, at most B / sqrt(3): 2.3e-3; 2.5e-3 is asked.
  * FFN: H's float errors (1.5e-5 of its size, see above) move a code over a border with probability 2 * 1.5e-5 /
    2^-4 or so, by 2^-3 of the value at most: 2^-3 sqrt(5e-4) = 2.8e-3 of H's norm; with the output's rounding
    sqrt(2.3^2 + 2.8^2) = 3.6e-3: 4e-3 is asked of the norm.  Of each row 2e-2 of its largest (the layers'
    tolerance) and, since one moved code is a step of up to 2^-3 |h_j| |w_ij| whatever the row's sum (f = 256: one h of
    four times the others' size, 2^-3 * 4 * 2.5 / (16 * 3) = 2.6e-2 of a row's largest), three such steps of the largest h and
    w: codes move with probability 5e-4 and less, so that more than three of a row's f <= 1091 do with 1.8e-3 and less,
    and then not all of the largest.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_mixture_experts_level_amd import workloads as wl
from tests.moe_testlib import BF16_TOL, row_rel_err, say, to_np

pytestmark = pytest.mark.gpu
ops = pytest.importorskip("sparse_mixture_experts_level_amd.ops")
DEV = "cuda"
U, B = 2.0 ** -24, 2.0 ** -8
GUARD = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dt=torch.float32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dt).to(DEV)


def f64(t):
    return to_np(t).astype(np.float64)


def guarded(shape, dt, fill=7):
    """A tensor at the front of a buffer, and a check that nothing behind it was written."""
    n = math.prod(shape)
    whole = torch.full((n + GUARD,), fill, dtype=dt, device=DEV)

    def check():
        assert torch.all(whole[n:] == fill), "written past the end"
    return whole[:n].view(shape), check


# ------------------------------------------------------------------------------ conversions

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 128), (5, 127), (2, 129), (7, 300), (33, 640), (4, 1091), (2, 2880)])
def test_rows_to_8_bits(dt, rows, K):
    say(f"rows {rows} x {K} {dt}")
    rng = np.random.default_rng(rows * 10000 + K)
    x = rng.standard_normal((rows, K)) * np.exp(3 * rng.standard_normal((rows, 1)))
    x[0, :min(K, 128)] = 0
    xg = dev(x, TYPES[dt])
    x = f64(xg)
    (codes, c1), (scale, c2) = guarded((rows, ops.moe_fp8_row_bytes(K)), torch.uint8), guarded((rows, ops.moe_fp8_scale_bytes(K)),
                                                                                             torch.uint8)
    ops.moe_quantize_rows_fp8(xg, codes, scale)
    want, e = oracle.fp8_quantize_rows(x)
    nb = e.shape[1]
    assert np.array_equal(to_np(codes)[:, :K], want[:, :K]) and not to_np(codes)[:, K:].any()
    assert np.array_equal(to_np(scale)[:, :nb].astype(int) - 127, e) and np.all(to_np(scale)[:, nb:] == 127)
    for back in TYPES.values():
        out, c3 = guarded((rows, K), back)
        ops.moe_dequantize_rows_fp8(codes, scale, out)
        assert np.array_equal(f64(out), oracle.fp8_row_values(want, e, K))
        c3()
    c1(), c2()


def test_rows_to_8_bits_at_the_ends_of_the_range():
    lv = oracle.e4m3_levels()
    mid = (lv[1:] + lv[:-1]) / 2
    v = np.concatenate([[448.0], lv, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))])
    rows = []
    for s in (1.0, 2.0 ** -130, 2.0 ** 118, 2.0 ** -60, 1.001):  # ties, subnormal floats, the largest
        row = np.zeros(512)
        row[:len(v)] = v * s
        row[128::128] = 448 * s
        rows.append(row)
    rows.append(np.full(512, 1e-45))
    rows.append(np.where(np.arange(512) % 5 == 0, np.inf, -3.0))
    rows.append(np.where(np.arange(512) < 128, np.nan, np.where(np.arange(512) % 3 == 0, -np.inf, 2.5)))
    x = np.array(rows, dtype=np.float32)
    codes, scale = ops.fp8_rows(len(x), 512)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    want, e = oracle.fp8_quantize_rows(x)
    got = to_np(codes)
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(to_np(scale).astype(int) - 127, e)
    out = torch.empty((len(x), 512), device=DEV)
    ops.moe_dequantize_rows_fp8(codes, scale, out)
    assert np.array_equal(f64(out), oracle.fp8_row_values(want, e, 512), equal_nan=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("G,n,K,swiglu", [(1, 1, 1, False), (2, 17, 130, False), (3, 128, 128, True), (2, 129, 64, True),
                                          (1, 200, 520, True), (2, 257, 300, False)])
def test_weights_to_8_bits(dt, G, n, K, swiglu):
    say(f"weights {G} x {n} x {K} swiglu {swiglu} {dt}")
    rng = np.random.default_rng(n * 1000 + K)
    w = dev(rng.standard_normal((G, n * (2 if swiglu else 1), K)) * np.exp(rng.standard_normal((G, 1, K))), TYPES[dt])
    sizes = ops.moe_fp8_weights_bytes(G, n, K, swiglu), ops.moe_fp8_weight_scales_bytes(G, n, K, swiglu)
    (codes, c1), (scale, c2) = guarded(sizes[:1], torch.uint8, 99), guarded(sizes[1:], torch.uint8, 99)
    ops.moe_quantize_weights_fp8(G, n, K, swiglu, w, codes, scale)
    codes, scale, wh = to_np(codes).reshape(G, -1), to_np(scale).reshape(G, -1), f64(w)
    for g in range(G):
        parts = [wh[g, :n], wh[g, n:]] if swiglu else [wh[g]]
        want, ws = oracle.fp8_pack_weights([oracle.fp8_quantize_weights(p) for p in parts])
        assert np.array_equal(codes[g], want) and np.array_equal(scale[g], ws)
    c1(), c2()


def test_rows_past_2_to_31_values():
    x = dev(np.random.default_rng(6).standard_normal((1000, 512)), torch.bfloat16)
    codes, scale = ops.fp8_rows(1000, 512)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    X = x.repeat(4300, 1)
    C, S = ops.fp8_rows(len(X), 512)
    ops.moe_quantize_rows_fp8(X, C, S)
    assert torch.all(C.view(4300, 1000, 512) == codes) and torch.all(S.view(4300, 1000, 4) == scale)
    back = torch.empty_like(x)
    ops.moe_dequantize_rows_fp8(codes, scale, back)
    ops.moe_dequantize_rows_fp8(C, S, X)
    assert torch.all(X.view(4300, 1000, 512) == back)


def test_calls_without_rows():
    """Nothing is written but the gradient of the weight, which is zeros."""
    none, w = torch.empty((0, 200), dtype=torch.bfloat16, device=DEV), torch.ones(200, dtype=torch.bfloat16, device=DEV)
    codes, scale = ops.fp8_rows(0, 200)
    ops.moe_quantize_rows_fp8(none, codes, scale)
    ops.moe_dequantize_rows_fp8(codes, scale, none)
    ops.moe_rms_norm(none, w, 1e-6, y=torch.empty_like(none))
    dw = torch.full((200,), 7.0, device=DEV)
    ops.moe_rms_norm_backward(none, none, w, torch.empty(0, device=DEV), torch.empty_like(none), dw,
                              ops.workspace(ops.moe_rms_norm_backward_workspace_size(0, 200)))
    assert torch.all(dw == 0)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    w8 = ops.fp8_weights(torch.ones((2, 30, 200), dtype=torch.bfloat16, device=DEV))
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(2, 0, 1, 30, 200))
    ops.moe_grouped_linear_fp8(2, 0, 1, 30, 200, codes, scale, off, *w8, none[:, :30].contiguous(), ws)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------ norm

def _held(dt):
    return lambda a: torch.tensor(a).to(TYPES[dt]).double().numpy()


def _check_norm(dt, T, d, residual, eps=1e-6, x=None, r=None, eight=True):
    rng = np.random.default_rng(T * 100000 + d)
    spread = np.exp(2 * rng.standard_normal((T, 1)))
    xg = dev(rng.standard_normal((T, d)) * spread if x is None else x, TYPES[dt])
    rg = dev(rng.standard_normal((T, d)) * spread if r is None else r, TYPES[dt]) if residual else None
    wg = dev(1 + 0.3 * rng.standard_normal(d), TYPES[dt])
    (h, c1), (y, c2), (rstd, c3) = guarded((T, d), TYPES[dt]), guarded((T, d), TYPES[dt]), guarded((T,), torch.float32)
    (y8, c4), (ys, c5) = (guarded((T, ops.moe_fp8_row_bytes(d)), torch.uint8), guarded((T, ops.moe_fp8_scale_bytes(d)),
                                                                                     torch.uint8))
    ops.moe_rms_norm(xg, wg, eps, residual=rg, h=h, y=y, rstd=rstd, **(dict(y8=y8, y_scale=ys) if eight else {}))
    with np.errstate(all="ignore"):
        hw, rw, yw = oracle.rms_norm(f64(xg), None if rg is None else f64(rg), f64(wg), float(np.float32(eps)), _held(dt))
    assert np.array_equal(f64(h), hw, equal_nan=True)
    got_r = f64(rstd)
    fine = np.isfinite(rw) & (rw < 3e38) & (rw > 1e-37)
    assert np.all(np.abs(got_r - rw)[fine] <= 2 * U * rw[fine])
    tol = (4 * U + (B if dt == "bf16" else 0)) * np.abs(yw) + 1e-37
    assert np.all(np.abs(f64(y) - yw)[fine] <= tol[fine])
    if eight:
        w32, r32, h32 = f64(wg).astype(np.float32), to_np(rstd), f64(h).astype(np.float32)
        with np.errstate(all="ignore"):
            y32 = (h32 * r32[:, None]) * w32
        want, e = oracle.fp8_quantize_rows(y32)
        got, nan = to_np(y8), (want & 127) == 127
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])
        assert np.array_equal(to_np(ys)[:, :e.shape[1]].astype(int) - 127, e) and np.all(to_np(ys)[:, e.shape[1]:] == 127)
    for c in (c1, c2, c3, c4, c5):
        c()
    return y, rstd


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,residual", [
    (1, 1, False), (3, 7, True), (5, 64, True), (4, 127, False), (9, 128, True), (6, 512, True), (5, 513, False),
    (2, 1024, True), (3, 1091, True), (7, 2048, False), (5, 2055, True), (1, 2880, True), (2, 4096, True), (3, 7168, True),
    (2, 8200, False), (2, 16384, True), (1, 16391, True), (2, 32768, False)])
def test_norm(dt, T, d, residual):
    say(f"norm {T} x {d} {dt} residual {residual}")
    _check_norm(dt, T, d, residual)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_of_rows_of_zeros_large_and_tiny_values(dt):
    d = 300
    x = np.random.default_rng(3).standard_normal((6, d))
    x[0] = 0
    x[1] *= 1e18   # squares past the floats' range
    x[2] *= 1e-25  # and below it: eps decides
    x[3] = 0
    x[3, 299] = 5
    _check_norm(dt, 6, d, False, x=x)
    _check_norm(dt, 3, d, False, eps=0.0, x=x[1:4] * np.array([[1], [1e8], [1]]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_keeps_a_row_that_is_not_finite_to_itself(dt):
    x = np.random.default_rng(4).standard_normal((5, 256))
    x[1, 3], x[3, 200] = np.nan, np.inf
    clean = x.copy()
    clean[[1, 3]] = 1
    w = dev(np.ones(256), TYPES[dt])
    outs = []
    for a in (x, clean):
        y, y8 = torch.zeros((5, 256), dtype=TYPES[dt], device=DEV), torch.zeros((5, 256), dtype=torch.uint8, device=DEV)
        ys = torch.zeros((5, 4), dtype=torch.uint8, device=DEV)
        ops.moe_rms_norm(dev(a, TYPES[dt]), w, 1e-6, y=y, y8=y8, y_scale=ys)
        outs.append((f64(y), to_np(y8)))
    keep = [0, 2, 4]
    assert np.array_equal(outs[0][0][keep], outs[1][0][keep]) and np.array_equal(outs[0][1][keep], outs[1][1][keep])
    assert np.isnan(outs[0][0][1]).all() and np.isnan(outs[0][0][3, 200])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_in_place_and_outputs_left_out(dt):
    T, d = 6, 1091
    rng = np.random.default_rng(5)
    x, r, w = (dev(rng.standard_normal(s), TYPES[dt]) for s in ((T, d), (T, d), (d,)))
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    ops.moe_rms_norm(x, w, 1e-5, residual=r, h=h, y=y, rstd=rstd)
    for inplace in ("h is x", "h is residual", "y is x, no h"):
        a, b = x.clone(), r.clone()
        y2 = torch.empty_like(x)
        if inplace == "h is x":
            ops.moe_rms_norm(a, w, 1e-5, residual=b, h=a, y=y2)
            assert torch.equal(a, h) and torch.equal(y2, y)
        elif inplace == "h is residual":
            ops.moe_rms_norm(a, w, 1e-5, residual=b, h=b, y=y2)
            assert torch.equal(b, h) and torch.equal(y2, y) and torch.equal(a, x)
        else:
            ops.moe_rms_norm(a, w, 1e-5, residual=b, y=a)
            assert torch.equal(a, y)
    only = torch.empty(T, device=DEV)
    ops.moe_rms_norm(x, w, 1e-5, residual=r, rstd=only)
    assert torch.equal(only, rstd)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,with_dh", [(1, 1, False), (2, 65, True), (7, 128, False), (600, 65, True), (2100, 40, True),
                                         (5, 1024, True), (513, 1091, False), (3, 2055, True), (4, 4096, True),
                                         (2, 8200, False), (3, 16384, True), (2, 16391, True)])
def test_norm_backward(dt, T, d, with_dh):
    say(f"norm backward {T} x {d} {dt} dh {with_dh}")
    rng = np.random.default_rng(T * 1000 + d)
    hg, dyg = (dev(rng.standard_normal((T, d)) * np.exp(rng.standard_normal((T, 1))), TYPES[dt]) for _ in range(2))
    dhg = dev(rng.standard_normal((T, d)), TYPES[dt]) if with_dh else None
    wg = dev(1 + 0.3 * rng.standard_normal(d), TYPES[dt])
    rstd = torch.empty(T, device=DEV)
    ops.moe_rms_norm(hg, wg, 1e-6, rstd=rstd)
    (dx, c1), (dw, c2) = guarded((T, d), TYPES[dt]), guarded((d,), torch.float32)
    need = ops.moe_rms_norm_backward_workspace_size(T, d)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    ops.moe_rms_norm_backward(dyg, hg, wg, rstd, dx, dw, ws[:need], dh=dhg)
    h, dy, w, r = f64(hg), f64(dyg), f64(wg), f64(rstd)
    wantx, wantw = oracle.rms_norm_backward(dy, h, w, r, None if dhg is None else f64(dhg))
    g, xh = np.abs(dy * w), np.abs(h * r[:, None])
    size = r[:, None] * (g + xh * (g * xh).mean(axis=1, keepdims=True)) + (0 if dhg is None else np.abs(f64(dhg)))
    assert np.all(np.abs(f64(dx) - wantx) <= 100 * U * size + (B if dt == "bf16" else U) * np.abs(wantx) + 1e-37)
    assert np.all(np.abs(f64(dw) - wantw) <= (T / 512 + 140) * U * (np.abs(dy) * xh).sum(axis=0) + 1e-37)
    assert torch.all(ws[need:] == 255)
    c1(), c2()
    for inplace in (dyg, hg) + ((dhg,) if with_dh else ()):  # and again: equal bit for bit
        a = {id(t): t.clone() for t in (dyg, hg) + ((dhg,) if with_dh else ())}
        out, dw2 = a[id(inplace)], torch.empty_like(dw)
        ops.moe_rms_norm_backward(a[id(dyg)], a[id(hg)], wg, rstd, out, dw2, ws[:need], dh=a[id(dhg)] if with_dh else None)
        assert torch.equal(out, dx) and torch.equal(dw2, dw)


def test_norm_backward_against_differences_of_the_kernel():
    """Float rows: the kernel's own forward, stepped by s, is off by some 2 u |y| / s of each difference."""
    T, d, s = 3, 96, 2.0 ** -6
    rng = np.random.default_rng(11)
    h, dy, w = rng.standard_normal((T, d)), rng.standard_normal((T, d)), 1 + 0.2 * rng.standard_normal(d)
    wg, rstd = dev(w), torch.empty(T, device=DEV)

    def value(a, ww):
        y = torch.empty((T, d), device=DEV)
        ops.moe_rms_norm(dev(a), dev(ww), 1e-6, y=y, rstd=rstd)
        return (f64(y) * dy).sum()
    value(h, w)
    base = rstd.clone()
    dx, dw = torch.empty((T, d), device=DEV), torch.empty(d, device=DEV)
    ops.moe_rms_norm_backward(dev(dy), dev(h), wg, base, dx, dw, ops.workspace(ops.moe_rms_norm_backward_workspace_size(T, d)))
    for t, c in [(0, 0), (1, 50), (2, 95)]:
        up, dn = h.copy(), h.copy()
        up[t, c] += s
        dn[t, c] -= s
        # third derivative: some |dy| (1 / d + ...) below one; s^2 / 6 = 4e-5, and float noise 4 u sqrt(T d) / s = 3e-4
        assert (value(up, w) - value(dn, w)) / (2 * s) == pytest.approx(f64(dx)[t, c], abs=5e-4)
    for c in (0, 95):
        up, dn = w.copy(), w.copy()
        up[c] += s
        dn[c] -= s
        assert (value(h, up) - value(h, dn)) / (2 * s) == pytest.approx(f64(dw)[c], abs=5e-4)


def test_norm_and_gradients_past_2_to_31_values():
    """Rows that repeat have outputs that repeat; dweight within its bound of the sum over all."""
    n, d, times = 1000, 512, 4300
    T = n * times
    rng = np.random.default_rng(12)
    w = dev(1 + 0.3 * rng.standard_normal(d), torch.bfloat16)
    x, r, dy = (dev(rng.standard_normal((n, d)), torch.bfloat16) for _ in range(3))
    h, y, rstd, dx, dw = (torch.empty_like(x), torch.empty_like(x), torch.empty(n, device=DEV), torch.empty_like(x),
                          torch.empty(d, device=DEV))
    y8, ys = ops.fp8_rows(n, d)
    ops.moe_rms_norm(x, w, 1e-6, residual=r, h=h, y=y, rstd=rstd, y8=y8, y_scale=ys)
    ops.moe_rms_norm_backward(dy, h, w, rstd, dx, dw, ops.workspace(ops.moe_rms_norm_backward_workspace_size(n, d)))
    X, R, DY = (t.repeat(times, 1) for t in (x, r, dy))
    RSTD, DW, (Y8, YS) = torch.empty(T, device=DEV), torch.empty(d, device=DEV), ops.fp8_rows(T, d)
    Y = torch.empty_like(X)
    ops.moe_rms_norm(X, w, 1e-6, residual=R, h=R, y=Y, rstd=RSTD, y8=Y8, y_scale=YS)
    for big, small in ((R, h), (Y, y), (RSTD, rstd), (Y8, y8), (YS, ys)):
        assert torch.all(big.view(times, *small.shape) == small)
    ops.moe_rms_norm_backward(DY, R, w, RSTD, Y, DW, ops.workspace(ops.moe_rms_norm_backward_workspace_size(T, d)))
    assert torch.all(Y.view(times, n, d) == dx)
    size = times * (np.abs(f64(dy)) * np.abs(f64(h)) * f64(rstd)[:, None]).sum(axis=0)
    want = times * (f64(dy) * f64(h) * f64(rstd)[:, None]).sum(axis=0)
    assert np.all(np.abs(f64(DW) - want) <= (T / 512 + 140) * U * size)


def test_norm_of_more_rows_than_a_launch_takes():
    n, d, times = 1000, 9, 9001  # 2^22 rows a launch
    rng = np.random.default_rng(13)
    x, r = (dev(rng.standard_normal((n, d)), torch.bfloat16).repeat(times, 1) for _ in range(2))
    w = dev(1 + 0.3 * rng.standard_normal(d), torch.bfloat16)
    T = n * times
    h, y, rstd, (y8, ys) = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV), ops.fp8_rows(T, d)
    ops.moe_rms_norm(x, w, 1e-6, residual=r, h=h, y=y, rstd=rstd, y8=y8, y_scale=ys)
    want = [torch.empty_like(t[:n]) for t in (h, y, rstd, y8, ys)]
    ops.moe_rms_norm(x[:n], w, 1e-6, residual=r[:n], h=want[0], y=want[1], rstd=want[2], y8=want[3], y_scale=want[4])
    for big, small in zip((h, y, rstd, y8, ys), want):
        assert torch.all(big.view(times, *small.shape) == small)


def test_codes_as_torch_holds_them():
    """float8_e4m3fn tensors are taken for codes."""
    x = dev(np.random.default_rng(14).standard_normal((5, 256)), torch.bfloat16)
    codes, scale = ops.fp8_rows(5, 256)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    own, scale2 = torch.empty((5, 256), dtype=torch.float8_e4m3fn, device=DEV), torch.empty_like(scale)
    ops.moe_quantize_rows_fp8(x, own, scale2)
    assert torch.equal(own.view(torch.uint8), codes) and torch.equal(scale, scale2)
    values = torch.empty((5, 256), device=DEV)
    ops.moe_dequantize_rows_fp8(own, scale, values)
    want = own.float().view(5, 2, 128) * torch.exp2(scale[:, :2].float() - 127)[:, :, None]
    assert torch.equal(values, want.view(5, 256))


# ------------------------------------------------------------------------------ products

def _offsets(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def _whole(rng, shape, block_axis_exponents):
    """Whole numbers up to 4 by powers of two a block, which 8 bits hold exactly."""
    v = rng.integers(-4, 5, shape).astype(np.float64)
    v[v == 3] = 4
    return v * block_axis_exponents


def _linear(counts, n, K, whole, gather, seed, tail=0, hint=None, first=0):
    rng = np.random.default_rng(seed)
    G, off = len(counts), _offsets(counts, first)
    rows = int(off[-1]) + tail
    kb = -(-K // 128)
    n_x = max(1, rows // 2) if gather else rows
    if whole:
        x = _whole(rng, (n_x, K), np.repeat(2.0 ** rng.integers(-2, 3, (n_x, kb)), 128, axis=1)[:, :K])
        w = _whole(rng, (G, n, K), np.repeat(2.0 ** rng.integers(-2, 3, (G, 1, kb)), 128, axis=2)[:, :, :K])
    else:
        x = rng.standard_normal((n_x, K)) * np.exp(rng.standard_normal((n_x, 1)))
        w = rng.standard_normal((G, n, K)) / np.sqrt(K)
    xg, wg = dev(x), dev(w)
    codes, scale = ops.fp8_rows(n_x, K)
    ops.moe_quantize_rows_fp8(xg, codes, scale)
    x8, xs = oracle.fp8_quantize_rows(f64(xg))
    xv = oracle.fp8_row_values(x8, xs, K)
    index = rng.integers(0, n_x, rows).astype(np.int32) if gather else None
    w8 = ops.fp8_weights(wg)
    y, guard = guarded((rows, n), torch.bfloat16, 3)
    need = ops.moe_grouped_linear_fp8_workspace_size(G, rows, hint or max(max(counts), 1), n, K)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    ops.moe_grouped_linear_fp8(G, rows, hint or max(max(counts), 1), n, K, codes, scale, dev(off, torch.int32), *w8, y,
                               ws[:need], row_index=None if index is None else dev(index, torch.int32))
    got = f64(y)
    guard()
    assert torch.all(ws[need:] == 255)
    assert np.all(got[:first] == 3) and np.all(got[off[-1]:] == 3)  # rows of no group stay as they were
    num = den = 0.0
    for g in range(G):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        src = xv[a:b] if index is None else xv[index[a:b]]
        m = oracle.fp8_quantize_weights(f64(wg)[g])
        want = oracle.fp8_linear(src, m)
        if whole:
            held = torch.tensor(want).float().to(torch.bfloat16).double().numpy()
            assert np.array_equal(got[a:b], held), (g, np.abs(got[a:b] - held).max())
        else:
            bound = B * np.abs(want) + 2.0 ** -9 * (np.abs(src) @ np.abs(oracle.fp8_weight_values(*m)).T) + 1e-37
            assert np.all(np.abs(got[a:b] - want) <= bound), g
            num, den = num + ((got[a:b] - want) ** 2).sum(), den + (want ** 2).sum()
    if not whole and sum(counts) * n > 2000:
        assert math.sqrt(num / den) <= 2.5e-3, math.sqrt(num / den)


SHAPES = [  # rows of each group, n_out, K
    ([1], 1, 1), ([1], 16, 128), ([0, 3, 0, 1], 17, 130), ([16, 2, 31], 64, 256), ([33], 130, 640), ([5, 0, 0], 300, 1091),
    ([40, 7, 64, 1], 128, 384), ([130], 96, 512), ([200, 17], 257, 300), ([300, 0, 256, 70], 272, 520), ([257], 520, 1152),
    ([0, 0], 64, 64), ([600], 256, 1024), ([129, 128, 127], 144, 129)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_linear_of_whole_numbers_is_exact(i, gather):
    counts, n, K = SHAPES[i]
    say(f"linear {counts} {n} x {K} gather {gather}")
    _linear(counts, n, K, True, gather, i)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_linear_of_normal_rows(i, gather):
    counts, n, K = SHAPES[i]
    say(f"linear, normal {counts} {n} x {K} gather {gather}")
    _linear(counts, n, K, False, gather, 100 + i, tail=5, first=0 if gather else 3)


@pytest.mark.parametrize("hint", [1, 5, 64, 300, 100000])
def test_linear_with_any_hint(hint):
    say(f"linear, hint {hint}")
    _linear([70, 0, 300, 5], 144, 384, True, True, 7, hint=hint)


LONG = [  # few tiles and a long K, cut along K: rows of each group, n_out, K
    ([100], 300, 2700), ([300], 257, 2700), ([20, 0, 150, 3], 130, 4100), ([17], 1, 5200), ([129, 64], 40, 2600), ([1, 40], 64, 9000)]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_linear_in_parts_of_k(i, whole):
    """Sums of whole numbers as above: 16 * 16 * 9000 / 2^-4 = 2^25 steps at most, 2^21 or so at 5 sigma."""
    counts, n, K = LONG[i]
    say(f"linear, parts {counts} {n} x {K} whole {whole}")
    _linear(counts, n, K, whole, bool(i % 2), 200 + i, tail=2, first=i % 3)
    _linear(counts, n, K, whole, not i % 2, 300 + i, hint=700)


def _whole_on_device(gen, *shape):
    return torch.randint(-4, 5, shape, generator=gen, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("counts,n", [([5000], 3300), ([2000, 1500, 0, 1500], 3300), ([4900, 100], 3300), ([700, 260], 28000)])
def test_linear_whose_last_round_is_cut(counts, n):
    """A few tiles more than whole rounds of 256; sums of whole numbers are the same in any order, so that the call equals
    calls of 600 rows, whose tiles are not that many.  With a group of few rows nothing is cut."""
    say(f"linear, last round {counts} x {n}")
    K, rows, G = 7300, sum(counts), len(counts)
    gen = torch.Generator(device=DEV).manual_seed(rows)
    x, w = _whole_on_device(gen, rows, K), _whole_on_device(gen, G, n, K)
    codes, scale = ops.fp8_rows(rows, K)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    c8, s8 = ops.fp8_weights(w)
    off = _offsets(counts)
    y, guard = guarded((rows, n), torch.bfloat16, 3)
    need = ops.moe_grouped_linear_fp8_workspace_size(G, rows, max(counts), n, K)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        ops.moe_grouped_linear_fp8(G, rows, max(counts), n, K, codes, scale, dev(off, torch.int32), c8, s8, y, ws[:need])
    guard()
    assert torch.all(ws[need:] == 255)
    c8, s8 = c8.view(G, -1), s8.view(G, -1)
    for g in range(G):
        for a in range(off[g], off[g + 1], 600):
            b = min(a + 600, off[g + 1])
            want = torch.empty((b - a, n), dtype=torch.bfloat16, device=DEV)
            own = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(1, b - a, b - a, n, K))
            ops.moe_grouped_linear_fp8(1, b - a, b - a, n, K, codes[a:b].clone(), scale[a:b].clone(), dev([0, b - a], torch.int32),
                                       c8[g].clone(), s8[g].clone(), want, own)
            assert torch.equal(y[a:b], want), (g, a)
    few = torch.arange(0, rows, rows // 40, device=DEV)
    for g in range(G):
        r = few[(few >= int(off[g])) & (few < int(off[g + 1]))]
        assert torch.equal(y[r], (x[r].double() @ w[g].double().T).float().to(torch.bfloat16)), g


def test_ffn_whose_last_round_is_cut():
    """Gate and up sums of whole numbers, so that H, and what it gives, is the same as that of 250 rows at a time."""
    rows, d, f = 2100, 7300, 3700
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, gu = _whole_on_device(gen, rows, d), _whole_on_device(gen, 1, 2 * f, d)
    dn = torch.randn((1, 300, f), generator=gen, device=DEV).to(torch.bfloat16)
    gu[:, :, 300:] *= (torch.rand((1, 2 * f, 1), generator=gen, device=DEV) < 0.02)  # sums of a size for silu
    gu = gu * 2.0 ** -7
    dn = torch.cat([dn, torch.zeros((1, d - 300, f), dtype=dn.dtype, device=DEV)], dim=1)
    codes, scale = ops.fp8_rows(rows, d)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    gu8, dn8 = ops.fp8_weights(gu, swiglu=True), ops.fp8_weights(dn)

    def run(a, b):
        y = torch.empty((b - a, d), dtype=torch.bfloat16, device=DEV)
        ws = ops.workspace(ops.moe_grouped_swiglu_gemm_fp8_workspace_size(1, b - a, b - a, d, f))
        ops.moe_grouped_swiglu_gemm_fp8(1, b - a, b - a, d, f, codes[a:b].clone(), scale[a:b].clone(), dev([0, b - a], torch.int32),
                                        *gu8, *dn8, y, ws)
        return y
    y = run(0, rows)
    assert y.isfinite().all() and y[:, :300].abs().mean() > 0
    for a in range(0, rows, 250):
        part = run(a, min(a + 250, rows))
        err = (y[a:a + 250].double() - part.double()).abs()
        assert torch.all(err <= 2 * B * part.double().abs() + 1e-5 * part.double().abs().max()), a


@pytest.mark.parametrize("counts", [[1, 0, 2] * 50, [40, 0, 1, 17] * 35, [0, 140, 3] * 30 + [300] * 12 + [0] * 64 + [5, 129]])
def test_linear_of_many_groups(counts):
    say(f"linear, {len(counts)} groups, up to {max(counts)} rows")
    _linear(counts, 40, 130, True, True, len(counts))


@pytest.mark.parametrize("counts,n,K", [([20, 0, 3] * 30, 1100, 130), ([17, 128] * 60 + [129, 300], 900, 130),
                                        ([1, 40] * 130, 300, 260)])
def test_linear_of_several_column_tiles_a_workgroup(counts, n, K):
    say(f"linear, {len(counts)} groups, {n} x {K}")
    _linear(counts, n, K, True, True, len(counts), hint=max(counts))
    _linear(counts, n, K, False, False, len(counts) + 1, hint=128)


@pytest.mark.parametrize("scale_rows,k", [(1, 200), (5, 200), (30, 200), (30, 2700)])
def test_offsets_that_decrease(scale_rows, k):
    """Not allowed, and harmless: rows are left out or one of their groups', and nothing else is written."""
    rng = np.random.default_rng(8)
    n, m = 12 * scale_rows, 40
    off = np.array([0, 10, 4, 12], dtype=np.int32) * scale_rows
    x, w = _whole(rng, (n, k), 1.0), _whole(rng, (3, m, k), 1.0)
    codes, scale = ops.fp8_rows(n, k)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    y, guard = guarded((n, m), torch.bfloat16, 3)
    need = ops.moe_grouped_linear_fp8_workspace_size(3, n, n, m, k)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    ops.moe_grouped_linear_fp8(3, n, n, m, k, codes, scale, dev(off, torch.int32), *ops.fp8_weights(dev(w)), y, ws[:need])
    got = f64(y)
    guard()
    assert torch.all(ws[need:] == 255)
    held = [torch.tensor(x @ w[g].T).float().to(torch.bfloat16).double().numpy() for g in range(3)]
    r = np.arange(n)[:, None]
    fine = (got == 3) | ((r < off[1]) & (got == held[0])) | ((r >= off[2]) & (got == held[2]))
    assert fine.all(), np.argwhere(~fine)[:5]


@pytest.mark.parametrize("hint", [16, 128, 1000])
def test_more_than_4_gib_of_rows(hint):
    """Codes, packed copies and outputs past 2^32 bytes and values: rows that repeat have outputs that repeat."""
    rng = np.random.default_rng(9)
    n, k, m, times = 1000, 128, 64, 34000
    x, w = _whole(rng, (n, k), 1.0), _whole(rng, (2, m, k), 1.0)
    codes, scale = ops.fp8_rows(n, k)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    codes, scale = codes.repeat(times, 1), scale.repeat(times, 1)
    rows = n * times
    # nearly all rows in few groups where those of many rows are split over tiles, else in as many as the hint asks for
    G, off = 2, [0, rows - 1500, rows]
    if hint <= 128:
        G, off = 3, [rows - 2 * hint - 5, rows - 2 * hint - 5, rows - hint - 5, rows - 5]
        w = np.concatenate([w[:1], w])
    y = torch.full((rows, m), 3.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(G, rows, hint, m, k))
    ops.moe_grouped_linear_fp8(G, rows, hint, m, k, codes, scale, dev(off, torch.int32), *ops.fp8_weights(dev(w)), y, ws)
    want = [torch.tensor(x @ w[g].T).float().to(torch.bfloat16).to(DEV) for g in range(G)]
    if hint > 128:
        assert torch.equal(y[:rows - 2000].view(-1, n, m), want[0].expand(times - 2, n, m))
    for g in range(G):
        a, b = max(off[g], rows - 2000), off[g + 1]
        assert torch.equal(y[a:b], want[g].repeat(2, 1)[a - (rows - 2000):b - (rows - 2000)]), g
    assert torch.all(y[off[-1]:] == 3)


def test_products_on_two_streams_at_once():
    """Each with its own workspace; with parts of K, packed rows and few rows between them."""
    rng = np.random.default_rng(11)
    k, m = 2700, 300
    w8 = ops.fp8_weights(dev(rng.standard_normal((2, m, k))))
    calls = []
    for rows, hint in ((400, 400), (90, 90), (20, 10), (300, 300)):
        codes, scale = ops.fp8_rows(rows, k)
        ops.moe_quantize_rows_fp8(dev(rng.standard_normal((rows, k))), codes, scale)
        y = torch.empty((rows, m), dtype=torch.bfloat16, device=DEV)
        ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(2, rows, hint, m, k))
        calls.append((rows, hint, codes, scale, dev([0, rows // 2, rows], torch.int32), y, ws, torch.cuda.Stream()))

    def run(c, stream):
        rows, hint, codes, scale, off, y, ws, _ = c
        ops.moe_grouped_linear_fp8(2, rows, hint, m, k, codes, scale, off, *w8, y, ws, stream=stream)
    want = []
    for c in calls:
        run(c, None)
        torch.cuda.synchronize()
        want.append(c[5].clone())
        c[5].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for c in calls:
            run(c, c[7])
    torch.cuda.synchronize()
    for c, y in zip(calls, want):
        assert torch.equal(c[5], y), c[0]


def test_offsets_and_indexes_out_of_range():
    """Offsets count as the ends of [0, rows_max], indexes outside as rows of zeros."""
    rng = np.random.default_rng(0)
    x, w = _whole(rng, (6, 64), 1.0), _whole(rng, (3, 32, 64), 1.0)
    codes, scale = ops.fp8_rows(6, 64)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    y = torch.full((8, 32), 3.0, dtype=torch.bfloat16, device=DEV)
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(3, 8, 8, 32, 64))
    index = np.array([0, -1, 5, 6, 2 ** 31 - 1, 1, -2 ** 31, 3], dtype=np.int32)
    off = np.array([-5, 4, 6, 900], dtype=np.int32)
    ops.moe_grouped_linear_fp8(3, 8, 8, 32, 64, codes, scale, dev(off, torch.int32), *ops.fp8_weights(dev(w)), y, ws,
                               row_index=dev(index, torch.int32))
    ends, got = [0, 4, 6, 8], f64(y)
    for g in range(3):
        for r in range(ends[g], ends[g + 1]):
            want = x[index[r]] @ w[g].T if 0 <= index[r] < 6 else np.zeros(32)
            assert np.array_equal(got[r], want), r


def test_nan_stays_in_its_row_and_column():
    rng = np.random.default_rng(1)
    x, w = _whole(rng, (20, 300), 1.0), _whole(rng, (1, 150, 300), 1.0)
    x[3, 299], x[17, 0], w[0, 40, 129], w[0, 149, 5] = np.nan, np.inf, np.nan, -np.inf
    codes, scale = ops.fp8_rows(20, 300)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    y = torch.empty((20, 150), dtype=torch.bfloat16, device=DEV)
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(1, 20, 20, 150, 300))
    ops.moe_grouped_linear_fp8(1, 20, 20, 150, 300, codes, scale, dev([0, 20], torch.int32), *ops.fp8_weights(dev(w)), y, ws)
    bad = np.zeros((20, 150), dtype=bool)
    bad[[3, 17]] = True
    bad[:, [40, 149]] = True
    got = f64(y)
    assert np.array_equal(np.isnan(got), bad)
    x[[3, 17]], w[0, [40, 149]] = 0, 0
    want = torch.tensor(x @ w[0].T).float().to(torch.bfloat16).double().numpy()
    assert np.array_equal(got[~bad], want[~bad])


def test_padding_scales_are_not_looked_at():
    rng = np.random.default_rng(2)
    x, w = _whole(rng, (5, 200), 1.0), _whole(rng, (1, 40, 200), 1.0)
    codes, scale = ops.fp8_rows(5, 200)
    ops.moe_quantize_rows_fp8(dev(x), codes, scale)
    c8, s8 = ops.fp8_weights(dev(w))
    scale[:, 2:] = 255
    s8.view(-1, 4)[:, 2:] = 255
    y = torch.empty((5, 40), dtype=torch.bfloat16, device=DEV)
    ws = ops.workspace(ops.moe_grouped_linear_fp8_workspace_size(1, 5, 5, 40, 200))
    ops.moe_grouped_linear_fp8(1, 5, 5, 40, 200, codes, scale, dev([0, 5], torch.int32), c8, s8, y, ws)
    assert np.array_equal(f64(y), torch.tensor(x @ w[0].T).float().to(torch.bfloat16).double().numpy())


# ------------------------------------------------------------------------------ the experts' FFN

def _ffn_case(counts, d, f, seed, tail=0):
    rng = np.random.default_rng(seed)
    G, off = len(counts), _offsets(counts)
    rows = int(off[-1]) + tail
    T = max(1, rows // 2)
    x = dev(rng.standard_normal((T, d)))
    gu, dn = dev(rng.standard_normal((G, 2 * f, d)) / np.sqrt(d)), dev(rng.standard_normal((G, d, f)) / np.sqrt(f))
    codes, scale = ops.fp8_rows(T, d)
    ops.moe_quantize_rows_fp8(x, codes, scale)
    index = rng.integers(0, T, rows).astype(np.int32)
    return dict(G=G, off=off, rows=rows, x=x, gu=gu, dn=dn, codes=codes, scale=scale, index=index, d=d, f=f,
                gu8=ops.fp8_weights(gu, swiglu=True), dn8=ops.fp8_weights(dn), top=max(max(counts), 1))


def _run_ffn(c, y, ws, stream=None):
    ops.moe_grouped_swiglu_gemm_fp8(c["G"], c["rows"], c["top"], c["d"], c["f"], c["codes"], c["scale"], c["goff"], *c["gu8"],
                                    *c["dn8"], y, ws, row_index=c["gindex"], stream=stream)


FFNS = [([1], 1, 1), ([2, 0, 1], 64, 64), ([16, 5], 130, 200), ([33, 0, 1], 256, 384), ([70], 520, 130), ([140, 128], 384, 256),
        ([300, 20, 0, 257], 256, 320), ([520], 300, 1091)]


LONG_FFNS = [([100], 2700, 130), ([300, 0, 20], 2700, 257), ([90, 30], 140, 2700), ([300, 129], 130, 2700),
             ([1, 0, 2] * 50, 130, 200), ([20, 0, 3] * 30, 130, 200), ([140, 3] * 40, 130, 200), ([20, 0, 3] * 30, 530, 300)]


@pytest.mark.parametrize("i", range(len(FFNS) + len(LONG_FFNS)))
def test_ffn(i):
    """Of the longer ones some are cut along K, some have more than 64 groups.  f of 2700: 1.4 codes of a row move on
    average, more than ten in 1e-7 of the rows."""
    counts, d, f = (FFNS + LONG_FFNS)[i]
    say(f"ffn {counts} d {d} f {f}")
    c = _ffn_case(counts, d, f, i, tail=3)
    c["goff"], c["gindex"] = dev(c["off"], torch.int32), dev(c["index"], torch.int32)
    y, guard = guarded((c["rows"], d), torch.bfloat16, 3)
    need = ops.moe_grouped_swiglu_gemm_fp8_workspace_size(c["G"], c["rows"], c["top"], d, f)
    ws = torch.full((need + GUARD,), 255, dtype=torch.uint8, device=DEV)
    _run_ffn(c, y, ws[:need])
    got = f64(y)
    guard()
    assert torch.all(ws[need:] == 255) and np.all(got[c["off"][-1]:] == 3)
    xv = oracle.fp8_row_values(*oracle.fp8_quantize_rows(f64(c["x"])), d)
    num = den = 0.0
    for g in range(c["G"]):
        a, b = c["off"][g], c["off"][g + 1]
        if a == b:
            continue
        q = oracle.fp8_quantize_weights
        gu = f64(c["gu"])[g]
        down = q(f64(c["dn"])[g])
        want, h, _ = oracle.fp8_ffn(xv[c["index"][a:b]], q(gu[:f]), q(gu[f:]), down)
        steps = (3 if f < 2000 else 10) * 2.0 ** -3 * np.abs(h).max(axis=1) * np.abs(oracle.fp8_weight_values(*down)).max()
        err = np.abs(got[a:b] - want).max(axis=1)
        assert np.all(err <= BF16_TOL * np.abs(want).max(axis=1) + steps), (g, err.max())
        num, den = num + ((got[a:b] - want) ** 2).sum(), den + (want ** 2).sum()
    if sum(counts) * d > 2000:
        assert math.sqrt(num / den) <= 4e-3, math.sqrt(num / den)
    y2 = torch.full_like(y, 3)
    _run_ffn(c, y2, ws[:need])
    assert torch.equal(y, y2)  # bit for bit


@pytest.mark.parametrize("counts,d,f", [([40, 0, 200, 3], 256, 384), ([40, 0, 200, 3], 2700, 2600), ([9, 2], 256, 384),
                                        ([60, 90], 2600, 256)])
def test_ffn_on_another_stream_and_captured(counts, d, f):
    c = _ffn_case(counts, d, f, 9)
    c["goff"], c["gindex"] = dev(c["off"], torch.int32), dev(c["index"], torch.int32)
    ws = ops.workspace(ops.moe_grouped_swiglu_gemm_fp8_workspace_size(c["G"], c["rows"], c["top"], d, f))
    want = torch.empty((c["rows"], d), dtype=torch.bfloat16, device=DEV)
    _run_ffn(c, want, ws)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    y = torch.zeros_like(want)
    other.wait_stream(torch.cuda.current_stream())
    _run_ffn(c, y, ws, stream=other)
    other.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_quantize_rows_fp8(c["x"], c["codes"], c["scale"])
        _run_ffn(c, y, ws)
    x0 = c["x"].clone()
    for k in range(3):  # replays follow the inputs, with eager work between
        c["x"].copy_(x0 if k != 1 else x0.flip(0))
        y.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        eager = torch.empty_like(y)
        ops.moe_quantize_rows_fp8(c["x"], c["codes"], c["scale"])
        _run_ffn(c, eager, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, eager), k
        assert k == 1 or torch.equal(got, want)


# ------------------------------------------------------------------------------ together: norm, layer in 8 bits

LAYERS = {
    "few tokens": wl.Workload("few", 5, 256, 8, 2, 128, None, "bf16"),
    "capacity, shared, skewed": wl.Workload("cap", 200, 320, 8, 2, 192, 1.25, "bf16", d_ff_shared=64, offset="boost4"),
    "many rows an expert": wl.Workload("many", 900, 256, 3, 2, 384, None, "bf16", d_ff_shared=128),
}


def _layer(w, **kw):
    inputs = wl.make_inputs(w, seed=0, device=DEV)
    return inputs, ops.MoELayer(inputs, ops.moe_capacity(w.num_tokens, w.num_experts, w.capacity_factor), device=DEV, **kw)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("name", LAYERS)
def test_layer_in_8_bits(name, norm):
    """Routing and combine as the bf16 layer's (bit for bit on the same input); each kept row's FFN as the oracle's in 8 bits."""
    w = LAYERS[name]
    say(f"layer in 8 bits: {name}, norm {norm}")
    weight = (1 + 0.1 * torch.randn(w.d_model, device=DEV, generator=torch.Generator(DEV).manual_seed(5))).bfloat16()
    inputs, layer = _layer(w, fp8=True, norm_weight=weight if norm else None)
    res = torch.randn(inputs.x.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(6)).bfloat16() if norm else None
    out = f64(layer.forward(residual=res))
    x = inputs.x
    if norm:
        h = (inputs.x.float() + res.float()).bfloat16()
        assert torch.equal(layer.h, h)
        x = layer.normed
        yw = oracle.rms_norm(f64(h), None, f64(weight), 1e-6)[2]
        assert np.all(np.abs(f64(x) - yw) <= (B + 4 * U) * np.abs(yw))
    plain, bf16 = _layer(w)
    plain.x.copy_(x)
    bf16.forward()
    for n in ("topk_ids", "slot", "expert_offsets", "topk_gates"):
        assert torch.equal(layer.routing[n], bf16.routing[n]), n
    # the norm quantises from its float y, the layer alone from the bf16 x
    codes, scale = (layer.x8, layer.x_scale) if norm else ops.fp8_rows(*x.shape)
    if not norm:
        ops.moe_quantize_rows_fp8(x, codes, scale)
    xv = torch.empty(x.shape, device=DEV)
    ops.moe_dequantize_rows_fp8(codes, scale, xv)
    xv, q = f64(xv), oracle.fp8_quantize_weights
    f, fs = w.d_ff, w.d_ff_shared
    off, rows = to_np(layer.routing["expert_offsets"]), to_np(layer.routing["row_token"])
    y = np.zeros((off[-1], w.d_model))
    for e in range(w.num_experts):
        a, b = off[e], off[e + 1]
        if a < b:
            gu = f64(inputs.w_gate_up[e])
            y[a:b] = oracle.fp8_ffn(xv[rows[a:b]], q(gu[:f]), q(gu[f:]), q(f64(inputs.w_down[e])))[0]
    want = np.zeros(out.shape)
    if fs:
        gu = f64(inputs.w_shared_gate_up)
        want += oracle.fp8_ffn(xv, q(gu[:fs]), q(gu[fs:]), q(f64(inputs.w_shared_down)))[0]
    ids, slot, gates = (to_np(layer.routing[n]) for n in ("topk_ids", "slot", "topk_gates"))
    for t in range(w.num_tokens):
        for j in range(w.top_k):
            if slot[t, j] >= 0:
                want[t] += gates[t, j] * y[off[ids[t, j]] + slot[t, j]]
    assert row_rel_err(out, want) <= BF16_TOL
    again = f64(layer.forward(residual=res))
    assert np.array_equal(again, out)
    # near the bf16 layer's: two roundings of 2^-4 / sqrt(3) a product, averaging out over sums: some 5% of the norm
    ref = f64(bf16.out)
    assert np.linalg.norm(out - ref) < 0.12 * np.linalg.norm(ref)


def test_layer_in_8_bits_redirects_overflow_as_the_bf16_layer():
    w = LAYERS["capacity, shared, skewed"]
    _, layer = _layer(w, fp8=True, overflow="reroute")
    _, bf16 = _layer(w, overflow="reroute")
    a, b = f64(layer.forward()), f64(bf16.forward())
    assert torch.equal(layer.routing["assigned_ids"], bf16.routing["assigned_ids"])
    assert torch.equal(layer.routing["slot"], bf16.routing["slot"])
    assert np.linalg.norm(a - b) < 0.12 * np.linalg.norm(b)


def test_blocks_of_norm_and_layer_captured():
    """Two blocks as a model runs them, h of the one the residual of the next, captured into a graph and replayed."""
    w = LAYERS["few tokens"]
    weight = torch.ones(w.d_model, dtype=torch.bfloat16, device=DEV)
    (i1, l1), (i2, l2) = (_layer(w, fp8=True, norm_weight=weight) for _ in range(2))
    i2.x = l1.out
    res = torch.zeros_like(i1.x)

    def both():
        l1.forward(residual=res)
        return l2.forward(residual=l1.h)
    want = both().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        l1.ws.fill_(255), l2.ws.fill_(255), l2.out.zero_()
        if k == 1:
            res.fill_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = l2.out.clone()
        assert torch.equal(got, both()), k
        assert torch.equal(got, want) == (k == 0), k


def test_layer_options_refused():
    w = LAYERS["few tokens"]
    with pytest.raises(ValueError, match="tile-major"):
        _layer(w, fp8=True, tiled=True)
    with pytest.raises(ValueError, match="bf16 layers"):
        _layer(wl.get_workload("tiny_f32"), fp8=True)
    inputs, layer = _layer(w, fp8=True)
    with pytest.raises(ValueError, match="norm_weight"):
        layer.forward(residual=inputs.x)
    with pytest.raises(ValueError, match="forward_staged"):
        layer.forward_staged(ops.stage_events())


def test_trainer_with_a_norm():
    """The step's gradients with a norm in front, against the composed oracle's, and the weight's update."""
    w = wl.Workload("train", 96, 256, 4, 2, 128, None, "bf16", d_ff_shared=64)
    inputs = wl.make_inputs(w, seed=0, device=DEV)
    gen = torch.Generator(DEV).manual_seed(9)
    rand = lambda s: torch.randn((w.num_tokens, w.d_model), generator=gen, device=DEV).mul_(s).bfloat16()  # noqa: E731
    weight = torch.ones(w.d_model, dtype=torch.bfloat16, device=DEV)
    res, dy, dh = rand(1.0), rand(1e-2), rand(1e-2)
    tr = ops.MoETrainer(inputs, None, device=DEV, norm_weight=weight, alpha=0.0, z_coeff=0.0, lr=1e-3, max_grad_norm=1.0,
                        master_weights=True)
    tr.forward(residual=res)
    dx = f64(tr.backward(dy, dh=dh))
    # the same layer without the norm, run on the norm's output, gives the gradient that reaches it
    plain = wl.make_inputs(w, seed=0, device=DEV)
    plain.x.copy_(tr.layer.normed)
    p = ops.MoETrainer(plain, None, device=DEV, alpha=0.0, z_coeff=0.0)
    p.forward()
    dn = f64(p.backward(dy))
    for n in p.grads:
        assert torch.equal(tr.grads[n], p.grads[n]), n
    h, wt = f64(tr.layer.h), f64(weight)
    wantx, wantw = oracle.rms_norm_backward(dn, h, wt, f64(tr.layer.rstd), f64(dh))
    size = np.abs(wantx) + np.abs(f64(dh)) + f64(tr.layer.rstd)[:, None] * (np.abs(dn) + np.abs(dn).mean())
    assert np.all(np.abs(dx - wantx) <= B * np.abs(wantx) + 400 * U * size)
    assert np.allclose(f64(tr.grads["dw_norm"]), wantw, rtol=0, atol=200 * U * np.abs(dn * h).sum(axis=0).max() + 1e-12)
    tr.step()
    torch.cuda.synchronize()
    # the first step moves a value by lr = 1e-3: less than half of bf16's step below one, 2^-9, so the weight itself stays and
    # its float copy moves, against the gradient
    master = tr.optimizer.states[-1]["master"]
    moved = f64(master) - 1
    assert np.all(np.abs(np.abs(moved) - 1e-3)[np.abs(wantw) > 1e-4] < 1e-5)
    assert np.array_equal(np.sign(moved)[np.abs(wantw) > 1e-4], -np.sign(wantw)[np.abs(wantw) > 1e-4])
    assert torch.equal(weight, master.bfloat16()) and torch.isfinite(tr.optimizer.grad_norm).all()
    with pytest.raises(ValueError, match="norm_weight"):
        p.backward(dy, dh=dh)
    tr.layer.norm_weight = weight.clone()
    with pytest.raises(RuntimeError, match="norm_weight"):
        tr.step()

"""CPU tests of the norm and of the products in 8 bits: pins of their oracle (torch's own 8-bit type, automatic
differentiation, differences, hand-worked layouts), and the argument checks of their C entry points and of the binding,
which return before any device work."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle

ops = pytest.importorskip("sparse_mixture_experts_level_amd.ops")
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
needs_lib = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="libmoe.so not built")
F32, BF16 = ops.MOE_DTYPE_F32, ops.MOE_DTYPE_BF16
INVALID, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


# ------------------------------------------------------------------------------ oracle pins

def test_levels_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_decode(codes.numpy()), want, equal_nan=True)


def test_codes_are_torchs():
    rng = np.random.default_rng(0)
    lv = oracle.e4m3_levels()
    # values, levels, the borders between them (ties) and their neighbours
    mid = (lv[1:] + lv[:-1]) / 2
    v = np.concatenate([rng.standard_normal(2000) * 100, lv, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    v = np.concatenate([v, -v]).astype(np.float32)
    v = v[np.abs(v) <= 448]
    assert len(v) > 4000
    for c in np.array_split(v, -(-len(v) // 120)):
        row = np.concatenate([c, [448.0]])[None]  # which keeps the scale at one
        codes, e = oracle.fp8_quantize_rows(row)
        assert e.tolist() == [[0]]
        want = torch.tensor(row).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes[0, :row.shape[1]], want[0])


def test_scales():
    for top, e in [(448.0, 0), (448.1, 1), (224.0, -1), (224.01, 0), (1.75, -8), (1.0, -8), (1.76, -7), (0.0, 0),
                   (2.0 ** -140, -126), (3e38, 120)]:
        assert oracle.fp8_scale_exponent(top) == e
    # a value that is not finite has no part in the scale, and the NaN code
    codes, e = oracle.fp8_quantize_rows(np.array([[np.inf, 3.0, -np.inf, np.nan, -448.0]]))
    assert e.tolist() == [[0]] and (codes[0, [0, 2, 3]] & 127).tolist() == [127] * 3 and codes[0, 4] == 0xfe
    codes, e = oracle.fp8_quantize_rows(np.array([[np.nan, np.inf]]))
    assert e.tolist() == [[0]] and (codes[0, :2] & 127).tolist() == [127] * 2


def test_packed_layout_by_hand():
    w = np.arange(17 * 130).reshape(17, 130) % 7 - 3.0
    codes, e = oracle.fp8_quantize_weights(w)
    out, scale = oracle.fp8_pack_weights([(codes, e)])
    assert out.shape == (2 * 2 * 2048,) and scale.shape == (4,)
    # two blocks, one tile: pieces [2 steps][2 halves][2 blocks] of 1 KB
    assert out[(2 * 2 + 0) * 1024 + 1 * 1024 + 1] == codes[16, 129]     # row 16: block 1; k 129: step 1, half 0, byte 1
    assert out[(1 * 2 + 0) * 1024 + 256 * 2 + 16 * 5 + 3] == codes[5, 99]  # row 5, k 99: half 1, c 2, i 3
    assert scale[:2].tolist() == (e[0] + 127).tolist()
    both, s2 = oracle.fp8_pack_weights([(codes, e), (codes, e)])
    both = both.reshape(2, 2, 2, 2, 1024)  # [step][half][block of rows][gate, up]
    assert np.array_equal(both[:, :, :, 0].reshape(-1), out) and np.array_equal(both[:, :, :, 1].reshape(-1), out) and len(s2) == 8
    tall = oracle.fp8_quantize_weights(np.arange(290 * 64).reshape(290, 64) % 9 - 4.0)
    out, _ = oracle.fp8_pack_weights([tall])  # 19 blocks: a tile of 16 and one of 3
    assert out[16 * 2048 + 1024 * 2 + 16 * 1 + 7] == tall[0][16 * 18 + 1, 7]


@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_gradient_against_autograd_and_differences(with_dh):
    rng = np.random.default_rng(1)
    T, d, eps = 5, 7, 1e-3
    h, w, dy = rng.standard_normal((T, d)) * 3, rng.standard_normal(d), rng.standard_normal((T, d))
    dh = rng.standard_normal((T, d)) if with_dh else None
    _, rstd, y = oracle.rms_norm(h, None, w, eps)
    dx, dw = oracle.rms_norm_backward(dy, h, w, rstd, dh)
    ht, wt = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    yt = torch.nn.functional.rms_norm(ht, (d,), wt, eps)
    assert np.allclose(yt.detach().numpy(), y, rtol=1e-12)
    loss = (yt * torch.tensor(dy)).sum() + (0 if dh is None else (ht * torch.tensor(dh)).sum())
    a, b = torch.autograd.grad(loss, (ht, wt))
    assert np.allclose(a.numpy(), dx, rtol=1e-10, atol=1e-13) and np.allclose(b.numpy(), dw, rtol=1e-10)
    step = 1e-5  # central differences: off by step^2 times the third derivative, some 1e-9 here

    def value(h):
        return (oracle.rms_norm(h, None, w, eps)[2] * dy).sum() + (0 if dh is None else (h * dh).sum())
    for t, c in [(0, 0), (2, 5), (4, 6)]:
        up, dn = h.copy(), h.copy()
        up[t, c] += step
        dn[t, c] -= step
        assert (value(up) - value(dn)) / (2 * step) == pytest.approx(dx[t, c], abs=1e-7)


def test_norm_of_a_sum():
    rng = np.random.default_rng(2)
    x, r, w = rng.standard_normal((3, 9)), rng.standard_normal((3, 9)), np.ones(9)
    h, rstd, y = oracle.rms_norm(x, r, w, 0.0)
    assert np.array_equal(h, x + r) and np.allclose((y * y).mean(axis=1), 1.0)


def test_ffn_is_the_layers_of_the_held_values():
    rng = np.random.default_rng(3)
    d, f = 40, 150
    gate, up, down = (oracle.fp8_quantize_weights(rng.standard_normal(s) * 0.2) for s in ((f, d), (f, d), (d, f)))
    rows = oracle.fp8_row_values(*oracle.fp8_quantize_rows(rng.standard_normal((6, d))), d)
    y, h, held = oracle.fp8_ffn(rows, gate, up, down)
    gu = np.concatenate([oracle.fp8_weight_values(*gate), oracle.fp8_weight_values(*up)])
    ref = oracle.swiglu_ffn(rows, gu, oracle.fp8_weight_values(*down))
    # a code is off by at most 2^-4 of its value, or half a subnormal step, 2^-10 of the scale
    assert np.all(np.abs(held - h) <= np.abs(h) * 2.0 ** -4 + np.abs(h).max(axis=1, keepdims=True) * 2.0 ** -17)
    assert np.abs(y - ref).max() < 0.1 * np.abs(ref).max() and not np.array_equal(y, ref)


# ------------------------------------------------------------------------------ refusals of the C entry points

def _norm(L, T=4, d=64, dt=BF16, x=FAKE, res=None, w=FAKE, eps=1e-6, h=None, y=None, y8=None, ys=None, rstd=None):
    return L.moe_rms_norm(T, d, dt, x, res, w, eps, h, y, y8, ys, rstd, None)


@needs_lib
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769), UNSUPPORTED), (dict(dt=5), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=FAKE + 2), INVALID), (dict(w=None), INVALID), (dict(res=FAKE + 8), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y8=FAKE), INVALID), (dict(ys=FAKE), INVALID), (dict(rstd=FAKE + 4), INVALID),
    (dict(h=FAKE + 16), INVALID), (dict(y=FAKE + 64), INVALID), (dict(res=0x90000, y=0x90010), INVALID),
    (dict(h=0x90000, y=0x90000), INVALID), (dict(h=0x90000, y=0x90010), INVALID)])
def test_norm_refusals(kw, status):
    L = ops.lib()
    assert _norm(L, **kw) == status and L.moe_last_error()


@needs_lib
def test_empty_calls_look_at_nothing():
    L = ops.lib()
    assert _norm(L, T=0, x=None, w=None) == ops.MOE_OK
    assert L.moe_quantize_rows_fp8(0, 64, BF16, None, None, None, None) == ops.MOE_OK
    assert L.moe_dequantize_rows_fp8(0, 64, F32, None, None, None, None) == ops.MOE_OK
    assert L.moe_grouped_linear_fp8(2, 0, 1, 64, 64, None, None, None, 0, None, None, None, None, None, 0, None) == ops.MOE_OK
    assert L.moe_grouped_swiglu_gemm_fp8(2, 0, 1, 64, 64, None, None, None, 0, None, None, None, None, None, None, None, 0,
                                         None) == ops.MOE_OK


@needs_lib
@pytest.mark.parametrize("kw,status", [
    (dict(d=0), INVALID), (dict(d=40000), UNSUPPORTED), (dict(dy=None), INVALID), (dict(h=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dw=FAKE + 4), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE), (dict(dx=FAKE + 16), INVALID),
    (dict(ws=FAKE + 8), INVALID), (dict(T=0, dw=None), INVALID)])
def test_norm_backward_refusals(kw, status):
    L = ops.lib()
    a = dict(T=4, d=64, dt=BF16, dy=FAKE, h=FAKE + 0x10000, w=FAKE + 0x20000, rstd=FAKE + 0x30000, dh=None,
             dx=FAKE + 0x40000, dw=FAKE + 0x50000, ws=FAKE + 0x60000, ws_bytes=1 << 20)
    a.update(kw)
    assert L.moe_rms_norm_backward(a["T"], a["d"], a["dt"], a["dy"], a["h"], a["w"], a["rstd"], a["dh"], a["dx"], a["dw"],
                                   a["ws"], a["ws_bytes"], None) == status
    assert L.moe_last_error()


@needs_lib
def test_sizes():
    assert [ops.moe_fp8_row_bytes(k) for k in (0, 1, 128, 129, 2880)] == [0, 128, 128, 256, 2944]
    assert [ops.moe_fp8_scale_bytes(k) for k in (-1, 1, 512, 513, 2880)] == [0, 4, 4, 8, 24]
    assert ops.moe_fp8_weights_bytes(3, 17, 130, False) == 3 * 2 * 2 * 2048
    assert ops.moe_fp8_weights_bytes(3, 17, 130, True) == 3 * 2 * 2 * 2 * 2048
    assert ops.moe_fp8_weight_scales_bytes(3, 129, 600, True) == 3 * 2 * 2 * 8
    assert ops.moe_fp8_weights_bytes(0, 17, 130, False) == 0 and ops.moe_fp8_weights_bytes(1025, 17, 130, False) == 0
    assert ops.moe_fp8_weights_bytes(1, 1 << 16, 1 << 15, False) == 0  # 2 GiB
    assert ops.moe_rms_norm_backward_workspace_size(5, 0) == 0 and ops.moe_rms_norm_backward_workspace_size(0, 8) > 0
    assert ops.moe_grouped_linear_fp8_workspace_size(4, -1, 1, 64, 64) == 0
    assert ops.moe_grouped_linear_fp8_workspace_size(4, 10, 0, 64, 64) == 0
    assert ops.moe_grouped_swiglu_gemm_fp8_workspace_size(4, 10, 10, 64, 200) >= 10 * 256 + 10 * 4
    assert ops.moe_forward_fp8_workspace_size(ops.make_desc(8, 64, 64, 4, 2, None, dtype=torch.float32)) == 0
    assert ops.moe_forward_fp8_workspace_size(ops.make_desc(8, 64, 64, 4, 2, None)) > 0


def _linear(L, **kw):
    a = dict(G=4, rows=32, top=32, n=64, k=64, x8=FAKE, xs=FAKE, idx=None, xr=32, off=FAKE, w8=FAKE, ws8=FAKE, y=FAKE,
             ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return L.moe_grouped_linear_fp8(a["G"], a["rows"], a["top"], a["n"], a["k"], a["x8"], a["xs"], a["idx"], a["xr"], a["off"],
                                    a["w8"], a["ws8"], a["y"], a["ws"], a["ws_bytes"], None)


def _ffn(L, **kw):
    a = dict(G=4, rows=32, top=32, d=64, f=64, x8=FAKE, xs=FAKE, idx=None, xr=32, off=FAKE, gu=FAKE, gus=FAKE, dn=FAKE,
             dns=FAKE, y=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return L.moe_grouped_swiglu_gemm_fp8(a["G"], a["rows"], a["top"], a["d"], a["f"], a["x8"], a["xs"], a["idx"], a["xr"],
                                         a["off"], a["gu"], a["gus"], a["dn"], a["dns"], a["y"], a["ws"], a["ws_bytes"],
                                         None)


COMMON = [(dict(G=0), INVALID), (dict(G=1025), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID),
          (dict(top=0), INVALID), (dict(x8=None), INVALID), (dict(x8=FAKE + 1), INVALID), (dict(xs=None), INVALID),
          (dict(off=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
          (dict(idx=FAKE, xr=-1), INVALID), (dict(idx=FAKE, xr=1 << 25), UNSUPPORTED), (dict(idx=FAKE + 4), INVALID)]


@needs_lib
def test_workspaces_of_the_most_rows():
    top = 2 ** 31 - 1
    assert 512 * 4 <= ops.moe_rms_norm_backward_workspace_size(top, 1) <= 1024 * 4
    assert ops.moe_rms_norm_backward_workspace_size(top, 32768) <= 1024 * 32768 * 4
    # codes packed for every tile that there can be, no more than a tile a group above the rows' own
    need = ops.moe_grouped_linear_fp8_workspace_size(1024, top, top, 4096, 128)
    assert top * 132 <= need <= (2 * top + 1025 * 256) * 132
    assert ops.moe_grouped_linear_fp8_workspace_size(1024, top, 16, 4096, 128) <= 256


@needs_lib
@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(n=1 << 16, k=1 << 15), UNSUPPORTED), (dict(w8=None), INVALID),
    (dict(ws8=None), INVALID), (dict(ws8=FAKE + 4), INVALID), (dict(k=1 << 24), UNSUPPORTED),
    (dict(k=1 << 23, n=1), UNSUPPORTED), (dict(k=1, n=1 << 23), UNSUPPORTED)])
def test_linear_refusals(kw, status):
    L = ops.lib()
    assert _linear(L, **kw) == status and L.moe_last_error()


@needs_lib
@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(d=0), INVALID), (dict(f=-3), INVALID), (dict(d=1 << 15, f=1 << 15), UNSUPPORTED), (dict(gu=None), INVALID),
    (dict(gus=None), INVALID), (dict(dn=None), INVALID), (dict(dns=FAKE + 2), INVALID)])
def test_ffn_refusals(kw, status):
    L = ops.lib()
    assert _ffn(L, **kw) == status and L.moe_last_error()


@needs_lib
@pytest.mark.parametrize("kw,status", [(dict(dt=9), UNSUPPORTED), (dict(k=0), INVALID), (dict(rows=-1), INVALID),
                                       (dict(rows=1 << 31), INVALID), (dict(a=None), INVALID), (dict(b=FAKE + 8), INVALID),
                                       (dict(c=None), INVALID)])
def test_conversion_refusals(kw, status):
    L = ops.lib()
    a = dict(rows=3, k=64, dt=BF16, a=FAKE, b=FAKE, c=FAKE)
    a.update(kw)
    assert L.moe_quantize_rows_fp8(a["rows"], a["k"], a["dt"], a["a"], a["b"], a["c"], None) == status
    assert L.moe_dequantize_rows_fp8(a["rows"], a["k"], a["dt"], a["a"], a["b"], a["c"], None) == status


@needs_lib
def test_weight_conversion_refusals():
    L = ops.lib()
    call = lambda g, n, k, dt=BF16, w=FAKE, c=FAKE, s=FAKE: L.moe_quantize_weights_fp8(g, n, k, 0, dt, w, c, s, None)  # noqa: E731
    assert call(0, 64, 64) == INVALID and call(1, 0, 64) == INVALID and call(1, 64, 64, dt=3) == UNSUPPORTED
    assert call(1, 64, 64, w=None) == INVALID and call(1, 64, 64, c=FAKE + 8) == INVALID
    assert call(1, 9_000_000, 128) == UNSUPPORTED


@needs_lib
def test_forward_fp8_refusals():
    L = ops.lib()
    m = ops.MoeFp8Matrix(FAKE, FAKE)
    none = ops.MoeFp8Matrix(None, None)

    def call(desc, w, x=FAKE, x8=None, xs=None, ws=FAKE, n=1 << 40):
        return L.moe_forward_fp8(ctypes.byref(desc), ctypes.byref(w) if w is not None else None, x, x8, xs, None, FAKE, None,
                                 ws, n, None)
    d = ops.make_desc(8, 64, 64, 4, 2, None)
    good = ops.MoeWeightsFp8(FAKE, m, m, none, none)
    assert call(ops.make_desc(8, 64, 64, 4, 2, None, dtype=torch.float32), good) == UNSUPPORTED
    assert call(ops.make_desc(8, 64, 64, 4, 5, None), good) == INVALID
    assert call(d, None) == INVALID
    assert call(d, ops.MoeWeightsFp8(None, m, m, none, none)) == INVALID
    assert call(d, ops.MoeWeightsFp8(FAKE, none, m, none, none)) == INVALID
    assert call(d, ops.MoeWeightsFp8(FAKE, m, ops.MoeFp8Matrix(FAKE, None), none, none)) == INVALID
    assert call(ops.make_desc(8, 64, 64, 4, 2, None, d_ff_shared=64), good) == INVALID
    assert call(d, good, x8=FAKE) == INVALID and call(d, good, x=None) == INVALID
    assert call(d, good, n=100) == WORKSPACE and call(d, good, ws=None) == WORKSPACE
    assert call(ops.make_desc(0, 64, 64, 4, 2, None), good) == ops.MOE_OK


# ------------------------------------------------------------------------------ refusals of the binding

@needs_lib
def test_binding_refuses_other_shapes_types_and_devices():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current GPU"):
        ops.moe_rms_norm(x, w, 1e-6)
    with pytest.raises(ValueError, match="unsupported dtype"):
        ops.moe_rms_norm(x.half(), w, 1e-6)
    codes, scale = ops.fp8_rows(4, 64, "cpu")
    assert codes.shape == (4, 128) and scale.shape == (4, 4)
    with pytest.raises(ValueError, match="shape"):
        ops._rows8(codes[:3], scale, ("c", "s"), 4, 64, -1)
    with pytest.raises(ValueError, match="shape"):
        ops._rows8(codes, scale[:, :2], ("c", "s"), 4, 64, -1)
    with pytest.raises(ValueError, match="as many gate as up rows"):
        ops.fp8_weights(torch.zeros((1, 3, 64), dtype=torch.bfloat16), swiglu=True)
    with pytest.raises(ValueError, match="contiguous"):
        ops.moe_rms_norm(torch.zeros((64, 4), dtype=torch.bfloat16).t(), w, 1e-6)


# ------------------------------------------------------------------------------ tiles of rows, compiled for the host

def _host_program(tmp_path, body):
    """What a program prints that includes the launchers' header, compiled by the host's compiler (signed sums wrap)."""
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("needs g++ and HIP's headers")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include "kernels.hpp"\n#include <cstdio>\nusing namespace moe;\nint main() {\n' + body + "\n}\n")
    csrc = os.path.join(os.path.dirname(ops.__file__), "csrc")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + csrc, str(src),
                    "-o", str(exe)], check=True)
    return [[int(v) for v in line.split()] for line in
            subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.splitlines()]


def test_tiles_of_groups_up_to_the_most_rows(tmp_path):
    """Of a group past 128 rows: the least number of tiles of 256, equal but for whole 32s, none of them empty."""
    rows = [0, 1, 128, 129, 256, 257, 300, 1040, 1537, 2 ** 20 + 1, 2 ** 30 - 1, 2 ** 30, 1_900_000_001, 1_950_000_000,
            2 ** 31 - 257, 2 ** 31 - 256, 2 ** 31 - 255, 2 ** 31 - 1]
    body = "".join(f"{{ int t = fp8_large_tiles({r}); std::printf(\"%d %d %d\\n\", {r}, t, t > 0 ? fp8_tile_rows({r}, t) : 0); }}\n"
                   for r in rows)
    got = _host_program(tmp_path, body)
    assert [g[0] for g in got] == rows
    for r, tiles, per in got:
        assert tiles == (0 if r <= 128 else -(-r // 256)), r
        if tiles:
            assert per % 32 == 0 and 0 < per <= 256 and (tiles - 1) * per < r <= tiles * per, (r, tiles, per)

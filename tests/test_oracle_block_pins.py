"""Pins of the block operators' oracle (oracle/block.py): closed forms, brute force, differences, torch."""
import numpy as np
import pytest
import torch

from oracle import block as o


def test_norm_against_torch():
    rng = np.random.default_rng(0)
    x, w, b = rng.normal(2, 3, (5, 33)), rng.normal(1, 0.2, 33), rng.normal(0, 1, 33)
    t = [torch.from_numpy(v) for v in (x, w, b)]
    ref = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], 1e-5).numpy()
    assert np.allclose(o.norm(x, "layer", 1e-5, w, b), ref, rtol=1e-12, atol=1e-12)
    ref = torch.nn.functional.rms_norm(t[0], (33,), t[1] + 1.0, 1e-5).numpy()
    assert np.allclose(o.norm(x, "rms", 1e-5, w, None, 1.0), ref, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
def test_gradients_against_autograd(kind):
    rng = np.random.default_rng(1)
    T, d = 4, 17
    v = {n: torch.from_numpy(rng.normal(m, 1, s)).requires_grad_() for n, s, m in
         (("r", (T, d), 0), ("y", (T, d), 1), ("w", (d,), 1), ("b", (d,), 0), ("g", (T, 1), 1))}
    dout = rng.normal(0, 1, (T, d))
    y = v["y"]
    c = y - y.mean(1, keepdim=True) if kind == "layer" else y
    n = y if kind == "none" else c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-3) * (v["w"] + 1.0) + v["b"]
    out = 0.5 * v["r"] + 2.0 * v["g"] * n
    out.backward(torch.from_numpy(dout))
    num = {k: t.detach().numpy() for k, t in v.items()}
    w, b = (num["w"], num["b"]) if kind != "none" else (None, None)
    assert np.allclose(o.norm_residual(num["r"], num["y"], kind, 1e-3, w, b, 1.0, num["g"], 0.5, 2.0), out.detach().numpy())
    dr, dy, dw, db, dg = o.norm_residual_backward(num["y"], dout, kind, 1e-3, w, b, 1.0, num["g"], 0.5, 2.0)
    assert np.allclose(dr, v["r"].grad) and np.allclose(dy, v["y"].grad)
    assert np.allclose(dg.sum(1, keepdims=True), v["g"].grad)
    if kind != "none":
        assert np.allclose(dw, v["w"].grad) and np.allclose(db, v["b"].grad)


def test_e4m3_values_are_torch_s():
    u = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(u.copy()).view(torch.float8_e4m3fn).double().numpy()
    got = o.e4m3_values(u)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])


def test_rounding_takes_the_nearest_and_ties_to_even():
    grid = np.unique(o.e4m3_values(np.arange(0x7F)))  # the finite non-negative values
    rng = np.random.default_rng(2)
    v = np.concatenate([rng.uniform(0, 460, 3000), 2.0 ** rng.uniform(-12, 9, 3000), (grid[1:] + grid[:-1]) / 2])
    got = o.round_e4m3(v)
    best = np.abs(np.minimum(v, 448.0)[:, None] - grid).min(1)
    assert np.array_equal(np.abs(np.minimum(v, 448.0) - got), best)
    mid = o.round_e4m3((grid[1:] + grid[:-1]) / 2)
    assert np.array_equal(np.searchsorted(grid, mid) % 2, np.zeros(mid.size, int))  # even fraction
    assert np.array_equal(o.round_e4m3(-v), -got) and np.isnan(o.round_e4m3(np.nan))


def test_scales_and_blocks():
    assert o.block_scale(448.0) == 1 and o.block_scale(0.0) == np.float32(2.0 ** -126)
    x = np.zeros((2, 144), np.float32)
    x[0, 0], x[0, 143], x[1, 130] = 448, -7, 1
    q, s = o.quantize_rows(x)
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[1, 0] == np.float32(7) / np.float32(448)
    assert q[0, 0] == 448 and q[0, 143] == -448 and q[1, 130] == 448
    assert np.allclose(o.dequantize_rows(q, s), x, rtol=1e-6)
    w = np.random.default_rng(3).normal(0, 1, (200, 272)).astype(np.float32)
    q, s = o.quantize_weights(w)
    assert s.shape == (2, 3) and np.abs(q).max() == 448
    back = o.dequantize_weights(q, s)
    assert (np.abs(back - w) <= 2.0 ** -4 * np.abs(w) * 1.001 + np.repeat(np.repeat(s, 128, 0)[:200], 128, 1)[:, :272] * 2.0 ** -10).all()


def test_matmul_and_gated_by_loops():
    rng = np.random.default_rng(4)
    a, W = rng.normal(0, 1, (5, 6)), rng.normal(0, 1, (3, 4, 6))
    got = o.matmul(a, [0, 2, 2, 4], lambda e: W[e])
    for r, e in ((0, 0), (1, 0), (2, 2), (3, 2)):
        assert np.allclose(got[r], [sum(a[r, k] * W[e, n, k] for k in range(6)) for n in range(4)])
    assert np.isnan(got[4]).all()
    assert np.isclose(o.gated(1.0, 3.0, 0.0), 3 / (1 + np.exp(-1))) and np.isclose(o.gated(9.0, -9.0, 2.0), -4 / (1 + np.exp(-2)))
    assert o.gated(np.array(-1e4), 1.0, 0.0) == 0

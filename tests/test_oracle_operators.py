"""Pins of ``oracle/operators.py``: nearest-value brute force, the workload encoders (torch, written
apart), torch's own functions, and differences for the gradients."""

import numpy as np
import pytest
import torch

from oracle import formats, operators as oo
from workloads import generate as wg


def test_encode_e2m1_is_the_nearest_value_with_ties_to_even():
    grid = formats.decode_e2m1(np.arange(8))
    mids = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mids, np.nextafter(mids, 0), np.nextafter(mids, 9), np.linspace(0, 6, 1201)])
    for s in (1.0, -1.0):
        codes = oo.encode_e2m1(s * v)
        for x, c in zip(s * v, codes):
            far = np.abs(grid - abs(x))
            best = np.flatnonzero(far == far.min())
            want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
            assert c & 7 == want and bool(c >> 3) == bool(np.signbit(x))


@pytest.mark.parametrize("elem,kind", oo.FORMS)
def test_quantize_agrees_with_the_workload_encoders(elem, kind):
    rng = np.random.default_rng(5)
    y = (rng.standard_normal((9, 512)) * np.exp2(rng.integers(-12, 12, (9, 1)))).astype(np.float32)
    y[2, :128] = 0
    y[3] *= 1e-30
    q, s = oo.quantize(y, elem, kind)
    t = torch.from_numpy(y)
    tq, ts = (wg.quantize_e4m3_rowblocks(t) if kind == "blockwise" else wg.quantize_nvfp4(t) if kind == "nv"
              else wg.quantize_mx(t, elem))
    assert np.array_equal(s, ts.numpy())
    assert np.array_equal(formats.decode_elements(q, elem), formats.decode_elements(tq.numpy(), elem))


def test_silu_mul_against_torch():
    x = torch.randn(7, 256, dtype=torch.float64) * 30
    want = torch.nn.functional.silu(x[:, :128]) * x[:, 128:]
    assert np.allclose(oo.silu_mul(x.numpy()), want.numpy(), rtol=1e-12, atol=1e-300)


def test_silu_mul_backward_against_torch():
    x = (torch.randn(7, 256, dtype=torch.float64, generator=torch.Generator().manual_seed(6)) * 8).requires_grad_()
    dy = torch.randn(7, 128, dtype=torch.float64, generator=torch.Generator().manual_seed(7))
    (torch.nn.functional.silu(x[:, :128]) * x[:, 128:]).backward(dy)
    assert np.allclose(oo.silu_mul_backward(dy.numpy(), x.detach().numpy()), x.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_rms_norm_gradient_against_autograd_and_differences():
    g = torch.Generator().manual_seed(1)
    h, dy, dres = (torch.randn(5, 128, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(128, generator=g, dtype=torch.float64)
    y, rstd = oo.rms_norm(h.numpy(), w.numpy(), 1e-3)
    hg, wgd = h.clone().requires_grad_(), w.clone().requires_grad_()
    (torch.nn.functional.rms_norm(hg, (128,), wgd, 1e-3) * dy + hg * dres).sum().backward()
    dx, dw = oo.rms_norm_backward(dy.numpy(), h.numpy(), w.numpy(), rstd, dres.numpy())
    assert np.allclose(dx, hg.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(dw, wgd.grad.numpy(), rtol=1e-10, atol=1e-12)
    # differences along one direction: error of order step^2
    v, step = torch.randn(5, 128, generator=g, dtype=torch.float64).numpy(), 1e-5
    loss = lambda a: (oo.rms_norm(a, w.numpy(), 1e-3)[0] * dy.numpy() + a * dres.numpy()).sum()  # noqa: E731
    slope = (loss(h.numpy() + step * v) - loss(h.numpy() - step * v)) / (2 * step)
    assert abs(slope - (dx * v).sum()) <= 1e-7 * np.abs(dx * v).sum()


def test_rows_there_and_back_are_adjoint_and_the_weighted_sum_has_its_gradient():
    rng = np.random.default_rng(2)
    dest = np.array([[0, 4], [1, -1], [-1, -1], [5, 2]], np.int32)
    counts, offsets = [3, 2], [0, 4, 8]                     # rows 3, 6 and 7 are padding
    x, r = rng.standard_normal((4, 8)), rng.standard_normal((9, 8))
    out = oo.permute_rows(x, dest, counts, offsets, np.full((9, 8), 7.0))
    assert np.all(out[[3, 6, 7]] == 0) and np.all(out[8] == 7)
    out[8] = 0
    assert np.isclose((out * r).sum(), (x * oo.combine(r, dest)).sum())
    w, dout = rng.random((4, 2)), rng.standard_normal((4, 8))
    y = rng.standard_normal((9, 8))
    dy, dw = oo.combine_backward(dout, y, dest, w, counts, offsets, np.full((9, 8), 7.0))
    assert np.all(dy[[3, 6, 7]] == 0) and np.all(dy[8] == 7) and np.all(dw[dest < 0] == 0)
    step, va, vb = 1e-6, rng.standard_normal(y.shape), rng.standard_normal(w.shape)
    f = lambda s: (oo.combine(y + s * va, dest, w + s * vb) * dout).sum()  # noqa: E731
    dy[8] = 0
    assert np.isclose((f(step) - f(-step)) / (2 * step), (dy * va).sum() + (dw * vb).sum(), rtol=1e-7)


def test_planted_mistakes_are_seen():
    """A scale of the wrong block, a tie rounded away from even and a lost padding row each differ."""
    y = np.random.default_rng(3).standard_normal((2, 256)).astype(np.float32)
    y[:, 128:] *= 4
    q, s = oo.quantize(y, "e4m3", "blockwise")
    assert not np.array_equal(s[:, 0], s[:, 1])
    assert oo.encode_e2m1([2.5])[0] == 4 and oo.encode_e2m1([5.0])[0] == 6 and oo.encode_e2m1([0.25])[0] == 0


def test_e4m3_blocks_of_the_smallest_values_have_finite_codes_and_scales():
    """amax from 2^-149 on, where amax / 448 has few bits or rounds to 0: clamped codes, the scale never 0."""
    n = np.arange(1, 9000, dtype=np.uint32)
    y = np.zeros((n.size, 128), np.float32)
    y[:, 0], y[:, 1] = n.view(np.float32), -n.view(np.float32)
    q, s = oo.quantize(y, "e4m3", "blockwise")
    v = formats.decode_e4m3fn(q)
    assert np.all(np.isfinite(v)) and np.all(s > 0) and np.all(v[:, 2:] == 0) and np.array_equal(v[:, 0], -v[:, 1])
    # the scale is amax / 448 to half of 2^-149, the code 448 of it or, cut, at most 224 steps of 2^-149 less
    err = np.abs(v[:, 0] * s[:, 0].astype(np.float64) - y[:, 0])
    assert np.all(err <= np.maximum(y[:, 0] * 2.0 ** -4, s[:, 0] * 2.0 ** -10) + 224 * 2.0 ** -149)

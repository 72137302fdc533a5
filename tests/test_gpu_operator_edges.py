"""The operators around the grouped GEMM where their values or sizes leave the ordinary range. Tolerances are
derived where they are used; U, the fp32 rounding, is 2^-24.
"""

import numpy as np
import pytest
import torch

import mx_grouped_gemm_amd as bsg
from examples import moe_block
from oracle import formats, operators as oo
from tests.parity import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LEAST = 2.0 ** -149
E4M3_BLOCK = bsg.make_quant("e4m3", "blockwise")


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say(f"\n[gpu-test] {request.node.name}")


# --------------------------------------------------------------------------------------
# blocks of the smallest fp32 values
# --------------------------------------------------------------------------------------
def tiny_blocks():
    """A row of one block for each amax: every one to 2^-136, 4096 more to 2^-126. The other elements are 0, -0, the
    amax with its sign changed, and multiples of 2^-149 in between."""
    rng = np.random.default_rng(1)
    n = np.unique(np.concatenate([np.arange(1, 8193), rng.integers(8193, 1 << 23, 4096), 2 ** np.arange(24)]))
    bits = rng.integers(0, n[:, None] + 1, (n.size, 128)).astype(np.uint32) | (rng.integers(0, 2, (n.size, 128)).astype(np.uint32) << 31)
    bits[:, 5], bits[:, 77] = n, n | (1 << 31)
    bits[:, 9], bits[:, 10] = 0, 1 << 31
    return bits.view(np.float32)


def test_blocks_of_the_smallest_values_to_e4m3():
    """Scales that are subnormal, or would round to 0: the codes are the clamped ones, none is NaN."""
    x = tiny_blocks()
    q, s = bsg.bsgemm_quantize(torch.from_numpy(x).cuda(), E4M3_BLOCK)
    qr, sr = oo.quantize(x, "e4m3", "blockwise")
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    assert not np.any((qr & 0x7F) == 0x7F) and np.all(sr > 0)


def near(q, s, y):
    """Codes and scales stand for y within half a step of e4m3 (2^-4 of y, or 2^-10 of the scale), 448 times the
    rounding of a subnormal scale, and y's own fp32 roundings."""
    v = formats.decode_elements(q.cpu().numpy(), "e4m3")
    scale = np.repeat(s.cpu().double().numpy(), 128, 1)
    assert not np.any(np.isnan(v))
    return np.all(np.abs(v * scale - y) <= np.abs(y) * (2.0 ** -4 + 32 * U) + scale * 2.0 ** -10 + 226 * LEAST)


def test_smallest_products_of_swiglu_and_the_norm_to_e4m3():
    """SwiGLU and norm outputs down to 2^-149 of ordinary inputs in fp32, and products of their rows."""
    g = torch.Generator().manual_seed(3)
    rows, K = 600, 256
    scale = torch.exp2(-torch.linspace(124, 149, rows, dtype=torch.float64))[:, None]
    gate = torch.randn(rows, K, generator=g) + 4
    up = (torch.randn(rows, K, generator=g).double() * scale).float()
    x = torch.cat([gate, up], 1)
    q, s = bsg.bsgemm_quantize(x.cuda(), E4M3_BLOCK, act="swiglu")
    assert near(q, s, oo.silu_mul(x.numpy()))
    B, bs = torch.full((256, K), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, device="cuda")
    C = torch.full((rows, 256), float("nan"), device="cuda")
    bsg.bsgemm_grouped(q, s, B, bs, None, None, C, rows, 256, K, bsg.make_fmt("e4m3", "e4m3", "blockwise", "f32"))
    assert torch.isfinite(C).all()
    h = torch.randn(40, K, generator=g)
    for power in (126, 138, 141, 143, 146, 149):
        w = (torch.randn(K, generator=g).double() * 2.0 ** -power).float()
        q, s, _, _ = bsg.bsgemm_rms_norm_quantize(h.cuda(), w.cuda(), E4M3_BLOCK, 1e-5)
        # (h rstd) w with rstd to (K / 64 + 20) U
        assert near(q, s, oo.rms_norm(h.numpy(), w.numpy(), 1e-5)[0])


# --------------------------------------------------------------------------------------
# gates that are not finite
# --------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("elem,kind", oo.FORMS)
def test_swiglu_shows_infinite_gates(elem, kind, dtype):
    """A gate of -inf, +inf or NaN, with an ordinary other factor, gives its block a scale that is not finite: g / (1 +
    exp(-g)) is NaN at -inf. Every other block is what it is without, gates far below 0 (0 there) among them."""
    K, B = 384, oo.BLOCK[kind]
    x = torch.randn(40, 2 * K, generator=torch.Generator().manual_seed(6)).to(dtype)
    x[:, 5:K:97] = torch.finfo(dtype).min
    x[:, 6:K:89] = -88.0
    fmt = bsg.make_quant(elem, kind)
    q0, s0 = (t.cpu().numpy() for t in bsg.bsgemm_quantize(x.cuda(), fmt, act="swiglu"))
    bad = np.zeros((40, K // B), bool)
    for r in range(1, 40):
        at = (r * 61) % K
        x[r, at] = (-float("inf"), float("inf"), float("nan"))[r % 3]
        bad[r, at // B] = True
    q, s = (t.cpu().numpy() for t in bsg.bsgemm_quantize(x.cuda(), fmt, act="swiglu"))
    lost = {"blockwise": lambda v: ~np.isfinite(v), "mx": lambda v: v == 255, "nv": lambda v: v == 0x7F}[kind]
    assert not lost(s0).any() and np.array_equal(lost(s), bad)
    assert np.array_equal(s[~bad], s0[~bad])
    q, q0 = (t.reshape(40, K // B, -1) for t in (q, q0))
    assert np.array_equal(q[~bad], q0[~bad])


# --------------------------------------------------------------------------------------
# no rows
# --------------------------------------------------------------------------------------
def test_a_block_without_tokens():
    """Every operator with empty tensors, forward and gradient: a rank that got no tokens."""
    block = moe_block.random_block(4, 256, 128, 2)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    out, saved = moe_block.forward(block, x, x)
    assert out.shape == (0, 256) and not saved["counts"].any() and not saved["offsets"].any()
    dx, dnorm, drouter = moe_block.backward(block, saved, out, x)
    assert dx.shape == (0, 256) and not dnorm.any() and not drouter.any()

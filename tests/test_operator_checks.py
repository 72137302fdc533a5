"""Refusals of the operators around the grouped GEMM (no GPU needed): status codes of the C ABI on
fake addresses, before any device is touched, and the binding's checks of tensors."""

import ctypes
import os

import pytest
import torch

import mx_grouped_gemm_amd as bsg

pytestmark = pytest.mark.skipif(not os.path.exists(bsg.library_path()), reason="libbsgemm.so not built")

P, ODD, P4 = 0x10000, 0x10001, 0x10004
BF16 = 2
OK, NULL, SHAPE, ALIGN, FMT, DEVICE = 0, -1, -2, -3, -4, -5
E4M3_BLOCK, E4M3_MX, E2M1_MX, E2M1_NV = (bsg.make_quant(*f) for f in
                                         (("e4m3", "blockwise"), ("e4m3", "mx"), ("e2m1", "mx"), ("e2m1", "nv")))


def call(name, base, **over):
    args = dict(base)
    assert set(over) <= set(args), over
    args.update(over)
    return getattr(bsg.load_library(), name)(*args.values())


def check(name, base, cases):
    # without a device the well-formed call gets as far as the device check (with one it would launch)
    if not torch.cuda.is_available():
        assert call(name, base) == DEVICE
    for want, over in cases:
        assert call(name, base, **over) == want, (over, want)


def test_quantize():
    base = dict(x=P, x_dtype=BF16, act=0, rows=4, K=256, q_fmt=E2M1_MX, q=P, scales=P, stream=None)
    check("bsgemm_quantize", base, [
        (FMT, dict(x_dtype=0)), (FMT, dict(x_dtype=4)), (FMT, dict(act=2)), (FMT, dict(q_fmt=0)),
        (FMT, dict(q_fmt=2 | (1 << 8))), (FMT, dict(q_fmt=1 | (3 << 8))), (FMT, dict(q_fmt=E4M3_MX | (1 << 12))),
        (SHAPE, dict(rows=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(K=96)), (SHAPE, dict(K=-128)),
        (SHAPE, dict(rows=(1 << 31) - 1, K=1 << 20)),
        (NULL, dict(x=None)), (NULL, dict(q=None)), (NULL, dict(scales=None)),
        (ALIGN, dict(x=P4)), (ALIGN, dict(q=P4)), (ALIGN, dict(scales=ODD, q_fmt=E4M3_BLOCK)),
        (OK, dict(rows=0, x=None, q=None, scales=None))])


def test_swiglu_backward():
    base = dict(dy=P, x=P, dtype=BF16, rows=4, K=24, dx=P, stream=None)
    check("bsgemm_swiglu_backward", base, [
        (FMT, dict(dtype=0)), (FMT, dict(dtype=4)), (SHAPE, dict(rows=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(K=12)),
        (SHAPE, dict(rows=(1 << 14) + 1, K=1 << 20)), (NULL, dict(dy=None)), (NULL, dict(x=None)), (NULL, dict(dx=None)),
        (ALIGN, dict(dy=P4)), (ALIGN, dict(x=P4)), (ALIGN, dict(dx=P4)), (OK, dict(rows=0, dy=None, x=None, dx=None))])


def test_rms_norm_quantize():
    base = dict(x=P, residual=P, weight=P, dtype=BF16, rows=4, K=256, eps=1e-6, q_fmt=E4M3_BLOCK, residual_out=P, rstd=P,
                q=P, scales=P, stream=None)
    check("bsgemm_rms_norm_quantize", base, [
        (FMT, dict(dtype=7)), (FMT, dict(q_fmt=5)), (SHAPE, dict(rows=-1)), (SHAPE, dict(K=130)), (SHAPE, dict(K=32896)),
        (SHAPE, dict(rows=1 << 22)), (SHAPE, dict(eps=-1.0)), (SHAPE, dict(eps=float("nan"))),
        (NULL, dict(x=None)), (NULL, dict(weight=None)), (NULL, dict(q=None)), (NULL, dict(scales=None)),
        (NULL, dict(residual=None)), (NULL, dict(residual_out=None)),
        (ALIGN, dict(x=P4)), (ALIGN, dict(residual=P4)), (ALIGN, dict(weight=P4)), (ALIGN, dict(residual_out=P4)),
        (ALIGN, dict(rstd=ODD)), (ALIGN, dict(q=P4)), (ALIGN, dict(scales=ODD)), (OK, dict(rows=0))])


def test_rms_norm_backward():
    base = dict(dy=P, h=P, weight=P, rstd=P, dresidual=P, dtype=BF16, rows=4, K=256, dx=P, dweight=P, workspace=P, nbytes=1 << 30,
                stream=None)
    check("bsgemm_rms_norm_backward", base, [
        (FMT, dict(dtype=0)), (SHAPE, dict(rows=-2)), (SHAPE, dict(K=100)), (SHAPE, dict(K=1 << 20)),
        (NULL, dict(dy=None)), (NULL, dict(h=None)), (NULL, dict(weight=None)), (NULL, dict(rstd=None)), (NULL, dict(dx=None)),
        (NULL, dict(dweight=None)), (NULL, dict(workspace=None)), (NULL, dict(rows=0, dweight=None)),
        (ALIGN, dict(dy=P4)), (ALIGN, dict(h=P4)), (ALIGN, dict(rstd=ODD)), (ALIGN, dict(dresidual=P4)), (ALIGN, dict(dx=P4)),
        (ALIGN, dict(dweight=ODD)), (ALIGN, dict(workspace=P4))])
    n = ctypes.c_size_t(0)
    size = bsg.load_library().bsgemm_rms_norm_backward_workspace_size
    assert size(-1, 256, ctypes.byref(n)) == SHAPE and size(4, 100, ctypes.byref(n)) == SHAPE and size(4, 256, None) == NULL


def test_route_sort():
    base = dict(ids=P, n=64, E=8, T=4, padded=1, M=512, counts=P, offsets=P, tile_offsets=P, expert_ids=P, dest=P, workspace=None,
                nbytes=0, stream=None)
    check("bsgemm_route_sort", base, [
        (SHAPE, dict(n=-1)), (SHAPE, dict(n=(1 << 24) + 1)), (SHAPE, dict(E=0)), (SHAPE, dict(E=4097)), (SHAPE, dict(T=-1)),
        (SHAPE, dict(T=(1 << 31) - 1)), (SHAPE, dict(M=-1)),
        (NULL, dict(ids=None)), (NULL, dict(counts=None)), (NULL, dict(offsets=None)), (NULL, dict(tile_offsets=None)),
        (NULL, dict(expert_ids=None)), (NULL, dict(dest=None)), (NULL, dict(n=1 << 20)),
        (SHAPE, dict(n=1 << 20, workspace=P, nbytes=64)),
        (ALIGN, dict(ids=ODD)), (ALIGN, dict(dest=ODD)), (ALIGN, dict(counts=ODD)), (ALIGN, dict(offsets=ODD)),
        (ALIGN, dict(tile_offsets=ODD)), (ALIGN, dict(expert_ids=ODD))])
    assert bsg.bsgemm_route_sort_workspace_size(1024, 32) == 0          # a decode batch needs none
    assert bsg.bsgemm_route_sort_workspace_size(1 << 20, 32) > 0
    with pytest.raises(bsg.BsgemmError):
        bsg.bsgemm_route_sort_workspace_size(-1, 32)


def test_permute_rows():
    base = dict(x=P, row_bytes=64, dest=P, tokens=4, top_k=2, counts=P, offsets=P, E=2, M=256, out=P, stream=None)
    check("bsgemm_permute_rows", base, [
        (SHAPE, dict(row_bytes=0)), (SHAPE, dict(row_bytes=6)), (SHAPE, dict(tokens=-1)), (SHAPE, dict(top_k=0)), (SHAPE, dict(E=0)),
        (SHAPE, dict(M=-1)), (SHAPE, dict(tokens=1 << 30, top_k=4)), (SHAPE, dict(tokens=1 << 30)),
        (NULL, dict(x=None)), (NULL, dict(dest=None)), (NULL, dict(counts=None)), (NULL, dict(offsets=None)), (NULL, dict(out=None)),
        (ALIGN, dict(x=ODD)), (ALIGN, dict(out=ODD)), (ALIGN, dict(dest=ODD)), (OK, dict(M=0, out=None))])


def test_combine():
    base = dict(y=P, dtype=BF16, dest=P, weights=P, tokens=4, top_k=2, K=64, M=256, out=P, stream=None)
    check("bsgemm_combine_rows", base, [
        (FMT, dict(dtype=9)), (SHAPE, dict(K=60)), (SHAPE, dict(K=0)), (SHAPE, dict(tokens=-1)), (SHAPE, dict(top_k=0)),
        (SHAPE, dict(M=-1)), (SHAPE, dict(tokens=1 << 30, K=1024)), (NULL, dict(y=None)), (NULL, dict(dest=None)),
        (NULL, dict(out=None)), (ALIGN, dict(y=P4)), (ALIGN, dict(out=P4)), (ALIGN, dict(weights=ODD)), (OK, dict(tokens=0))])
    base = dict(dout=P, y=P, dtype=BF16, dest=P, weights=P, tokens=4, top_k=2, K=64, counts=P, offsets=P, E=2, M=256, dy=P,
                dweights=P, stream=None)
    check("bsgemm_combine_backward", base, [
        (FMT, dict(dtype=0)), (SHAPE, dict(K=4)), (SHAPE, dict(E=0)), (SHAPE, dict(top_k=0)), (SHAPE, dict(tokens=(1 << 23) + 1)),
        (NULL, dict(dout=None)), (NULL, dict(y=None)), (NULL, dict(dest=None)), (NULL, dict(weights=None)), (NULL, dict(counts=None)),
        (NULL, dict(offsets=None)), (NULL, dict(dy=None)), (NULL, dict(dweights=None)),
        (ALIGN, dict(dout=P4)), (ALIGN, dict(y=P4)), (ALIGN, dict(dy=P4)), (ALIGN, dict(dweights=ODD))])


def test_grouped_few_rows():
    mx = bsg.make_fmt("e2m1", "e2m1", "mx", "bf16")
    base = dict(A=P, sa=P, B=P, sb=P, ei=P, to=P, T=2, C=P, M=64, N=256, K=640, E=2, fmt=mx, stream=None)
    check("bsgemm_grouped_few_rows", base, [
        (FMT, dict(fmt=bsg.make_fmt("e4m3", "e4m3", "blockwise", "bf16"))), (FMT, dict(fmt=bsg.make_fmt("e2m1", "e2m1", "nv", "bf16"))),
        (FMT, dict(fmt=bsg.make_fmt("e4m3", "e4m3", "mx", "bf16"))), (FMT, dict(fmt=mx | bsg.SCHED_SMALL_M)), (FMT, dict(fmt=(mx & ~0xF) | 3)), (FMT, dict(fmt=mx & ~0xF000)),
        (SHAPE, dict(N=192)), (SHAPE, dict(K=96)), (SHAPE, dict(K=1 << 25)), (SHAPE, dict(M=-1)), (SHAPE, dict(E=0)), (SHAPE, dict(T=-1)),
        (SHAPE, dict(T=1 << 22)),
        (NULL, dict(A=None)), (NULL, dict(C=None)), (NULL, dict(sb=None)), (NULL, dict(ei=None)), (NULL, dict(to=None)),
        (ALIGN, dict(A=P4)), (ALIGN, dict(B=P4)), (ALIGN, dict(C=P4)), (ALIGN, dict(sa=ODD)), (ALIGN, dict(ei=ODD)),
        (OK, dict(M=0)), (OK, dict(T=0))])


def test_make_quant():
    assert bsg.quant_shapes(E2M1_NV, 3, 256) == ((3, 128), (3, 16), torch.uint8)
    assert bsg.quant_shapes(E4M3_BLOCK, 3, 256) == ((3, 256), (3, 2), torch.float32)
    with pytest.raises(ValueError, match="unsupported"):
        bsg.make_quant("e2m1", "blockwise")
    with pytest.raises(ValueError, match="unknown"):
        bsg.quant_shapes(0, 1, 128)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


U8, I32, F32 = torch.uint8, torch.int32, torch.float32


@pytest.mark.parametrize("fn,good,bad", [
    (bsg.check_quantize_args, dict(x=z(4, 256), q_fmt=E2M1_MX, act="none", q=z(4, 128, dtype=U8), scales=z(4, 8, dtype=U8)),
     [dict(x=z(4, 256, dtype=torch.float64)), dict(x=z(256)), dict(act="gelu"), dict(q=z(4, 256, dtype=U8)),
      dict(scales=z(4, 8)), dict(act="swiglu")]),
    (bsg.check_swiglu_backward_args, dict(dy=z(4, 24), x=z(4, 48), dx=z(4, 48)),
     [dict(x=z(4, 24)), dict(x=z(4, 48, dtype=F32)), dict(dx=z(4, 24)), dict(dx=z(5, 48)), dict(dy=z(24)), dict(dy=z(4, 24, dtype=U8))]),
    (bsg.check_norm_args, dict(x=z(4, 256), weight=z(256), q_fmt=E4M3_BLOCK, residual=z(4, 256), residual_out=z(4, 256),
                               rstd=z(4, dtype=F32), q=z(4, 256, dtype=U8), scales=z(4, 2, dtype=F32)),
     [dict(weight=z(256, dtype=F32)), dict(weight=z(128)), dict(residual=None), dict(residual=z(5, 256)), dict(rstd=z(4)),
      dict(scales=z(4, 8, dtype=U8)), dict(q=z(4, 128, dtype=U8))]),
    (bsg.check_norm_backward_args, dict(dy=z(4, 256), h=z(4, 256), weight=z(256), rstd=z(4, dtype=F32), dresidual=z(4, 256),
                                        dx=z(4, 256), dweight=z(256, dtype=F32)),
     [dict(h=z(4, 128)), dict(h=z(4, 256, dtype=F32)), dict(rstd=z(5, dtype=F32)), dict(dweight=z(256)), dict(dresidual=z(3, 256)),
      dict(dx=z(4, 256, dtype=F32))]),
    (bsg.check_route_sort_args, dict(topk_ids=z(4, 2, dtype=I32), num_experts=3, num_tiles=5, dest=z(4, 2, dtype=I32),
                                     counts=z(3, dtype=I32), expert_offsets=z(4, dtype=I32), tile_offsets=z(6, dtype=I32),
                                     expert_ids=z(5, dtype=I32)),
     [dict(topk_ids=z(4, 2, dtype=torch.int64)), dict(dest=z(8, dtype=I32)), dict(counts=z(4, dtype=I32)),
      dict(expert_offsets=z(3, dtype=I32)), dict(tile_offsets=z(5, dtype=I32)), dict(expert_ids=z(5))]),
    (bsg.check_permute_rows_args, dict(x=z(4, 64), dest=z(4, 2, dtype=I32), counts=z(3, dtype=I32), expert_offsets=z(4, dtype=I32),
                                       M=128, out=z(128, 64)),
     [dict(x=z(5, 64)), dict(dest=z(4, dtype=I32)), dict(dest=z(4, 2, dtype=torch.int64)), dict(expert_offsets=z(3, dtype=I32)),
      dict(out=z(127, 64)), dict(out=z(128, 64, dtype=U8))]),
    (bsg.check_combine_args, dict(y=z(128, 64), dest=z(4, 2, dtype=I32), weights=z(4, 2, dtype=F32), out=z(4, 64)),
     [dict(y=z(128, 64, dtype=U8)), dict(weights=z(4, 2)), dict(weights=z(2, 4, dtype=F32)), dict(out=z(5, 64)),
      dict(dest=z(4, dtype=I32))]),
    (bsg.check_combine_backward_args, dict(dout=z(4, 64), y=z(128, 64), dest=z(4, 2, dtype=I32), weights=z(4, 2, dtype=F32),
                                           counts=z(3, dtype=I32), expert_offsets=z(4, dtype=I32), dy=z(128, 64),
                                           dweights=z(4, 2, dtype=F32)),
     [dict(dout=z(4, 32)), dict(dout=z(5, 64)), dict(weights=z(4, 3, dtype=F32)), dict(dy=z(127, 64)), dict(dweights=z(4, 2)),
      dict(counts=z(4, dtype=I32))]),
])
def test_binding_checks(fn, good, bad):
    fn(**good)
    for over in bad:
        with pytest.raises(ValueError):
            fn(**{**good, **over})


def test_grouped_few_rows_without_rows_takes_the_null_pointers_of_empty_tensors():
    assert torch.empty(0, 128).data_ptr() == 0
    base = dict(A=None, sa=None, B=P, sb=P, ei=P, to=P, T=2, C=None, M=0, N=256, K=640, E=2,
                fmt=bsg.make_fmt("e2m1", "e2m1", "mx", "bf16"), stream=None)
    for want, over in [(OK, {}), (OK, dict(ei=None, to=None)), (OK, dict(T=0, ei=None)), (OK, dict(T=0, ei=None, M=4)),
                       (OK, dict(B=None, sb=None)), (NULL, dict(ei=None)), (NULL, dict(to=None)), (NULL, dict(M=4)),
                       (NULL, dict(T=0, to=None)), (SHAPE, dict(N=100)), (ALIGN, dict(B=P4))]:
        assert call("bsgemm_grouped_few_rows", base, **over) == want, (over, want)

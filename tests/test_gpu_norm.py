"""dit_rms_norm against the fp64 definition: odd widths, every type, strided and in-place rows."""

import numpy as np
import pytest

from oracle import block, fp8

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24                                  # half a step of fp32


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _make(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * 1.7).to(dtype)


def _tol(C):
    """Relative error of y in fp32 before its last rounding: the sum of C squares (at most C / 32
    terms one after another in a lane, then 5 + 5 steps across lanes and warps, halved by the root),
    the mean, rsqrt (2 ulps of 2 * U32) and the two products."""
    return (C / 64 + 5 + 1 + 4 + 2 + 2) * U32


def _check(y, ds, ref, C, group):
    import torch
    if ds is None:
        half = torch.finfo(y.dtype).eps / 2 if y.dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(_np(y) - ref) <= np.abs(ref) * (half + _tol(C)) * (1 + half) + 1e-37)
        return
    codes, d = fp8.e4m3_decode(y.cpu().numpy()).astype(np.float64), _np(ds)
    g = group or C
    for i in range(d.shape[-1]):
        r, c, di = ref[:, i * g:(i + 1) * g], codes[:, i * g:(i + 1) * g], d[:, i:i + 1]
        amax = np.abs(r).max(1, keepdims=True)
        want = np.where(amax > 0, amax / 448.0, 1.0)
        assert np.all(np.abs(di - want) <= want * (_tol(C) + 2 * U32))
        # half a step of E4M3: 2^-4 of a normal value, 2^-10 scales below that
        assert np.all(np.abs(c * di - r) <= np.maximum(np.abs(r) * 2.0 ** -4, di * 2.0 ** -10) * 1.001 + 2 * _tol(C) * amax)


CASES = [(1, 1), (3, 7), (5, 64), (2, 127), (4, 129), (333, 1001), (7, 1536), (130, 2304), (3, 5120), (2, 8192),
         (2, 20001), (1, 70000), (3, 40960)]


@pytest.mark.parametrize("rows,C", CASES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("out,group", [("bfloat16", 0), ("float32", 0), ("uint8", 0), ("uint8", 128)])
def test_types_and_widths(cuda_lib, rows, C, dtype, out, group):
    import torch
    t = getattr(torch, dtype)
    x, r, w = _make((rows, C), t, 1), _make((rows, C), t, 2), _make((C,), t, 3)
    for res, wt in ((r, w), (None, w), (r, None)):
        y, h, ds = cuda_lib.rms_norm(x, wt, residual=res, eps=1e-5, out_dtype=getattr(torch, out), group=group)
        ref, rh = block.rms_norm(_np(x), None if wt is None else _np(wt), None if res is None else _np(res), 1e-5)
        _check(y, ds, ref, C, group)
        if res is None:
            assert h is None
        else:
            half = torch.finfo(t).eps / 2
            assert h.dtype == t and np.all(np.abs(_np(h) - rh) <= np.abs(rh) * half + 1e-37)


def test_rows_out_of_a_wider_matrix_and_in_place(cuda_lib):
    import torch
    for C, ld, off in ((256, 640, 128), (256, 643, 3), (99, 128, 1)):
        wide = _make((37, ld), torch.bfloat16, 4)
        x, w, r = wide[:, off:off + C], _make((C,), torch.bfloat16, 5), _make((37, C), torch.bfloat16, 6)
        keep, r0 = wide.clone(), r.clone()
        y, h, _ = cuda_lib.rms_norm(x, w, residual=r, inplace=True)
        ref, rh = block.rms_norm(_np(x), _np(w), _np(r0))
        _check(y, None, ref, C, 0)
        assert h is r and torch.equal(wide, keep)
        assert torch.equal(r, (x.float() + r0.float()).to(torch.bfloat16))
        # the stream over x itself (dense rows), through the C entry
        xd = x.contiguous()
        y2 = torch.empty_like(xd)
        cuda_lib.dit_rms_norm(xd, C, r0, w, y2, xd, None, 37, C, 1e-6)
        assert torch.equal(y2, y) and torch.equal(xd, r)


def test_leading_dimensions_and_empty(cuda_lib):
    import torch
    x = _make((2, 3, 5, 128), torch.float32, 7)
    y, h, ds = cuda_lib.rms_norm(x, out_dtype=torch.uint8, group=128)
    assert y.shape == x.shape and ds.shape == (2, 3, 5, 1) and h is None
    y, _, _ = cuda_lib.rms_norm(x[:0])
    assert y.shape == (0, 3, 5, 128)
    z, _, ds = cuda_lib.rms_norm(torch.zeros(2, 256, device="cuda"), out_dtype=torch.uint8, group=128)
    assert torch.all(z == 0) and torch.all(ds == 1.0)


def test_a_bad_row_stays_in_its_row(cuda_lib):
    import torch
    x = _make((9, 1536), torch.bfloat16, 8)
    good = cuda_lib.rms_norm(x)[0]
    x[4, 17] = float("nan")
    x[7, 3] = float("inf")
    y = cuda_lib.rms_norm(x)[0]
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(y[keep], good[keep]) and torch.all(torch.isnan(y[4].float()))
    y = y[7].float()
    assert torch.isnan(y[3]) and torch.all(y[:3] == 0) and torch.all(y[4:] == 0)


def test_large_and_small_magnitudes(cuda_lib):
    import torch
    for s in (1e-15, 1e15):
        x = _make((5, 640), torch.float32, 9) * s
        y = cuda_lib.rms_norm(x, eps=0.0)[0]
        _check(y, None, block.rms_norm(_np(x), eps=0.0)[0], 640, 0)


def test_e4m3_of_tiny_rows(cuda_lib):
    """Down to 2^-119 the scale holds; below, a group counts as zeros (never NaN)."""
    import torch
    x = torch.zeros(4, 256, device="cuda")
    x[0, 5], x[1, 200], x[2, 7], x[3] = 1e-30, -2e-36, 1e-37, 1e-44
    for group in (0, 128):
        c, _, d = cuda_lib.rms_norm(x, eps=1.0, out_dtype=torch.uint8, group=group)
        back = c.view(torch.float8_e4m3fn).float().view(4, -1, 128) * d.view(4, -1, 1)
        assert not torch.any(torch.isnan(back)) and torch.all(back[2:] == 0)
        assert abs(back[0].max() / 1e-30 - 1) < 2.0 ** -4 and abs(back[1].min() / -2e-36 - 1) < 2.0 ** -4


def test_streams_and_graph(cuda_lib):
    import torch
    x, r = _make((64, 5120), torch.bfloat16, 10), _make((64, 5120), torch.bfloat16, 11)
    want = cuda_lib.rms_norm(x, residual=r, out_dtype=torch.uint8, group=128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = cuda_lib.rms_norm(x, residual=r, out_dtype=torch.uint8, group=128, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = cuda_lib.rms_norm(x, residual=r, out_dtype=torch.uint8, group=128)
    x.mul_(2.0)
    g.replay()
    want = cuda_lib.rms_norm(x, residual=r, out_dtype=torch.uint8, group=128)
    assert all(torch.equal(a, b) for a, b in zip(want, cap))

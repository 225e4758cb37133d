"""What must stay apart where rows of several adapters share a matrix-core block: above 512
rows, and above 64 rows where rows times rank passes 16384.  Adapters, unused rank slots and
rows that are not finite reach the rows they belong to and no others."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import x_values
from lora_bounds import (adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern, mlp_lora_bound)
from test_gpu_lora import _check, _gemm, _mlp, _x

pytestmark = pytest.mark.gpu

BLOCKS = [(600, 16), (130, 128), (513, 8), (90, 256), (1100, 72)]


def _ids(M, n):
    """Adapters that alternate row by row, and rows without one among them."""
    ids = (np.arange(M) % n).astype(np.int32)
    ids[7::29] = -1
    ids[-1] = -1
    return ids


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,R", BLOCKS)
def test_a_bad_adapter_or_row_stays_its_own(M, R, dtype):
    K, N, n = 256, 128, 5
    w, lo = device_weight(codes(K, N, 80)), adapters(n, R, K, N, 81)
    ids = _ids(M, n)
    dev_ids = torch.from_numpy(ids).cuda()
    x = _x(M, K, dtype, 82)
    want = _gemm(x, w, device_lora(lo), dev_ids, torch.float32)
    assert bool(torch.isfinite(want).all())
    others = torch.from_numpy(ids != 2).cuda()
    for which in (0, 1, 2):  # A, B and the scale
        bad = [lo[0].copy(), lo[1].copy(), lo[2].copy(), None]
        if which == 2:
            bad[2][2] = np.nan
        else:
            bad[which][2, ::2], bad[which][2, 1::2] = np.inf, np.nan
        got = _gemm(x, w, device_lora(tuple(bad)), dev_ids, torch.float32)
        assert torch.equal(got[others], want[others])
        if which == 1:  # every other column of B
            assert not bool(torch.isfinite(got[~others]).any())
        else:
            assert bool(torch.isnan(got[~others]).all())
    for value in (float("nan"), float("inf")):
        rows = torch.tensor([0, 1, 7, 70, M - 1], device="cuda")  # (7 and the last have no adapter)
        x2 = x.clone()
        x2[rows] = value
        got = _gemm(x2, w, device_lora(lo), dev_ids, torch.float32)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert torch.equal(got[keep], want[keep])
        assert not bool(torch.isfinite(got[rows]).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fill", [np.nan, np.inf])
@pytest.mark.parametrize("M,R", BLOCKS)
def test_unused_slots(M, R, fill, dtype):
    """Ranks past ranks[id] hold NaN or infinities; ranks beyond [0, R] are clamped."""
    K, N, n = 256, 128, 6
    w = codes(K, N, 83)
    lo = adapters(n, R, K, N, 84, ranks=[R, 0, 1, R // 2 + 3, R + 9, -3])
    A, B = lo[0].copy(), lo[1].copy()
    for a in range(n):
        r = O.lora_rank(lo[3], a, R)
        A[a, r:] = fill
        B[a, :, r:] = fill
    ids = _ids(M, n)
    x = _x(M, K, dtype, 85)
    y = _gemm(x, device_weight(w), device_lora((A, B, lo[2], lo[3])), torch.from_numpy(ids).cuda(), torch.float32)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32),
           f"gemm_lora unused slots M={M} R={R} {dtype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("have", [7, 3, 5, 2])
@pytest.mark.parametrize("M,R", [(600, 16), (130, 128)])
def test_mlp(M, R, have, dtype):
    """Unused slots of NaN in every adapter, a bad adapter on one projection, a row with one NaN."""
    H, I, n = 128, 320, 5
    shapes = ((H, I), (H, I), (I, H))
    ws3 = [codes(K, N, 86 + i) for i, (K, N) in enumerate(shapes)]
    dw = [device_weight(w) for w in ws3]
    ids = _ids(M, n)
    dev_ids = torch.from_numpy(ids).cuda()
    los, holed = [], []
    for i, (K, N) in enumerate(shapes):
        lo = adapters(n, R, K, N, 89 + i, ranks=[R, 3, R // 2, 0, R]) if have >> i & 1 else None
        los.append(lo)
        if lo is not None:
            A, B = lo[0].copy(), lo[1].copy()
            for a in range(n):
                r = O.lora_rank(lo[3], a, R)
                A[a, r:] = np.nan
                B[a, :, r:] = np.nan
            lo = (A, B, lo[2], lo[3])
        holed.append(lo)
    x = _x(M, H, dtype, 92)
    y = _mlp(x, dw, [device_lora(l) for l in holed], dev_ids, torch.float32)
    xv = x_values(x)
    _check(y, O.swiglu_mlp_lora64(xv, *ws3, *los, ids), mlp_lora_bound(xv, *ws3, *los, ids, dtype, torch.float32),
           f"mlp_lora unused slots M={M} R={R} have={have} {dtype}", dtype)
    for i in range(3):
        if los[i] is None:
            continue
        A = holed[i][0].copy()
        A[4] = np.nan
        bad = [device_lora((A,) + holed[i][1:] if j == i else l) for j, l in enumerate(holed)]
        got = _mlp(x, dw, bad, dev_ids, torch.float32)
        others = torch.from_numpy(ids != 4).cuda()
        assert torch.equal(got[others], y[others])
        assert bool(torch.isnan(got[~others]).all())
    rows = torch.tensor([0, 1, 7, 70, M - 1], device="cuda")
    x2 = x.clone()
    x2[rows, 3] = float("nan")
    got = _mlp(x2, dw, [device_lora(l) for l in holed], dev_ids, torch.float32)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], y[keep])
    assert bool(torch.isnan(got[rows]).all())

"""MXFP4 calls and block_norm on matrices of more than 2^32 values: the last rows and columns, whose
offsets pass 32 bits, are those of the same call on them alone, or within the products' bounds."""
import pytest
import torch

import int4_w4a16_group_g32_amd as L
from mx_bounds import check, gemm_bound, out_bound

pytestmark = pytest.mark.gpu

ROWS, K, LAST = (1 << 17) + 16, 1 << 15, 16


@pytest.fixture(scope="module")
def long():
    """(x bf16 [ROWS][K], its MXFP4 rows)."""
    torch.manual_seed(3)
    x = torch.empty((ROWS, K), dtype=torch.bfloat16, device="cuda").normal_()
    m = L.mx_empty(ROWS, K)
    L.mx_quantize(x, m)
    yield x, m
    del x, m
    torch.cuda.empty_cache()


def _tail(x):
    """MXFP4 of the last rows alone, and its values in float64 (bf16 holds them exactly)."""
    t = L.mx_empty(LAST, K)
    L.mx_quantize(x[-LAST:].clone(), t)
    v = torch.empty((LAST, K), dtype=torch.bfloat16, device="cuda")
    L.mx_dequantize(t, v)
    return t, v


def test_formats(long):
    x, m = long
    t, v = _tail(x)
    assert torch.equal(m.codes[-LAST:], t.codes) and torch.equal(m.scales[-LAST:], t.scales)
    out = torch.empty_like(x)
    L.mx_dequantize(m, out)
    assert torch.equal(out[-LAST:], v)
    w = L.mx_prepack(m, L.mx_empty(ROWS, K, L.MX_TILED))
    out.zero_()
    L.mx_dequantize(w, out)
    assert torch.equal(out[-LAST:], v)
    back = L.mx_empty(ROWS, K)
    L.mx_quantize_weight(out.t().contiguous(), back)
    assert torch.equal(back.codes[-LAST:], t.codes) and torch.equal(back.scales[-LAST:], t.scales)


@pytest.mark.parametrize("M", [2, 40, 130])
@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_columns_of_a_long_weight(long, M, kind):
    x, m = long
    w = L.mx_prepack(m, L.mx_empty(ROWS, K, L.MX_TILED))
    wv = _tail(x)[1].double().cpu().numpy()
    a = x[7:7 + M].clone()
    if kind == "mx":
        q = L.mx_empty(M, K)
        L.mx_quantize(a, q)
        L.mx_dequantize(q, a)
    av = a.double().cpu().numpy()
    y = torch.empty((M, ROWS), device="cuda")
    code = L.MXFP4 if kind == "mx" else L.BF16
    L.mx_gemm(q if kind == "mx" else a, w, y, L.new_workspace(L.mx_gemm_workspace_bytes(M, code, w)))
    ref = av @ wv.T
    check(y[:, -LAST:], ref, out_bound(ref, gemm_bound(av, wv, kind), torch.float32), kind)


@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_rows_of_a_long_batch(long, kind):
    x, m = long
    t, v = _tail(x)
    n = L.mx_empty(48, K)
    L.mx_quantize(x[100:148].clone(), n)
    w = L.mx_prepack(n, L.mx_empty(48, K, L.MX_TILED))
    wv = torch.empty((48, K), device="cuda")
    L.mx_dequantize(n, wv)
    wv = wv.double().cpu().numpy()
    av = (v if kind == "mx" else x[-LAST:]).double().cpu().numpy()
    y = torch.empty((ROWS, 48), device="cuda")
    code = L.MXFP4 if kind == "mx" else L.BF16
    L.mx_gemm(m if kind == "mx" else x, w, y, L.new_workspace(L.mx_gemm_workspace_bytes(ROWS, code, w)))
    ref = av @ wv.T
    check(y[-LAST:], ref, out_bound(ref, gemm_bound(av, wv, kind), torch.float32), kind)


def test_norm_to_mxfp4_rows(long):
    x, m = long
    pre = torch.rand(K, device="cuda").bfloat16() + 0.5
    s, n = torch.empty_like(x), L.mx_empty(ROWS, K)
    L.block_norm(x, x, s, n, pre_w=pre, post_w=pre, gate=x)
    s1, n1, tail = torch.empty((LAST, K), dtype=torch.bfloat16, device="cuda"), L.mx_empty(LAST, K), x[-LAST:].clone()
    L.block_norm(tail, tail, s1, n1, pre_w=pre, post_w=pre, gate=tail)
    assert torch.equal(s[-LAST:], s1)
    assert torch.equal(n.codes[-LAST:], n1.codes) and torch.equal(n.scales[-LAST:], n1.scales)

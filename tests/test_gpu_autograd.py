"""The calls beside autograd: they record nothing, and what they write into a
caller's tensor counts as a write."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16 = torch.float16


def _operands():
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(F16)
    return rand(6, 32), rand(2, 16, 32), torch.tensor([0, 2, 6], dtype=torch.int32).cuda(), rand


def test_results_require_no_grad():
    from bit_quantized_moe_token_amd import moeq
    x, w, off, rand = _operands()
    wq, sw = moeq.quantize_i8(w)
    x.requires_grad_()
    w.requires_grad_()
    y = moeq.grouped_gemm(x, w, off)
    outs = [y, moeq.grouped_wgrad(y, x, off), moeq.linear_i8(x, wq, sw, offsets=off), *moeq.block_norm(x, x)]
    assert not any(t.requires_grad for t in outs)


def test_writes_are_counted():
    from bit_quantized_moe_token_amd import moeq
    x, w, off, rand = _operands()
    wq, sw = moeq.quantize_i8(w)
    xq, sx = moeq.quantize_i8(x)
    y, dw, r, n = rand(6, 16), torch.zeros(2, 16, 32, device="cuda"), rand(6, 32), rand(6, 32)
    for out, call in ((y, lambda: moeq.grouped_gemm(x, w, off, out=y)), (dw, lambda: moeq.grouped_wgrad(y, x, off, out=dw)),
                      (y, lambda: moeq.linear_i8(x, wq, sw, offsets=off, out=y)),
                      (y, lambda: moeq.gemm_i8(xq, sx, wq, sw, offsets=off, out=y)),
                      (r, lambda: moeq.block_norm(r, n, res_out=r, n_out=n)),
                      (n, lambda: moeq.block_norm(r, n, res_out=r, n_out=n))):
        before = out._version
        call()
        assert out._version > before
    # a pass that saved the residual reports that it was overwritten
    leaf = torch.ones(6, 32, device="cuda", requires_grad=True)
    res = rand(6, 32).float()
    loss = (leaf * res).sum()
    moeq.block_norm(res, n.float(), res_out=res)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                       # (such tensors count no writes)
        moeq.grouped_gemm(x, w, off, out=torch.empty(6, 16, dtype=F16, device="cuda"))

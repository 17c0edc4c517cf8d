"""Limits of the gated activation that its documentation states."""
import ctypes

import pytest
import torch

import expert_ref as X

pytestmark = pytest.mark.gpu


def test_most_features_of_the_activation(gpu):
    m, most = gpu, gpu.MOE_MAX_FEATURES // 2
    c = X.Case(m, T=3, k=1, E=2)
    gu, d = c.randn(3, 2 * most), c.randn(3, most)
    gud, dd = gu.cuda(), d.cuda()
    out, codes, scales = torch.empty_like(dd), torch.empty(3, most, dtype=torch.uint8, device="cuda"), torch.empty(3, most // 128, device="cuda")
    lib, h = m.load_library(), ctypes.byref(c.handle.c)

    def calls(features):
        return (lib.moe_swiglu(c.ctx.handle, gud.data_ptr(), features, 0, h, out.data_ptr(), None),
                lib.moe_swiglu_fp8(c.ctx.handle, gud.data_ptr(), features, 0, h, codes.data_ptr(), scales.data_ptr(), None),
                lib.moe_swiglu_backward(c.ctx.handle, dd.data_ptr(), gud.data_ptr(), features, 0, h, gud.data_ptr(), None))
    for features in (most + 8, most + 128, 2 * most):
        assert set(calls(features)) == {m.MOE_ERR_UNSUPPORTED}
    assert set(calls(0)) == set(calls(-8)) == {m.MOE_ERR_INVALID_ARG}
    assert torch.equal(gud.cpu(), gu)
    assert set(calls(most)) == {m.MOE_OK}
    ref = X.swiglu64(gu)
    X.check(out.cpu(), ref, (X.BF16_HALF + 128 * X.F32_STEP) * ref.abs() + 2.0 ** -120, "act")
    c.close()


def test_gates_past_the_range_of_the_exponential(gpu):
    """exp(-g) is infinite in binary32 below -88.73: the sigmoid is 0 there, and so are the product and its gradient."""
    c = X.Case(gpu, T=1, k=1, E=1)
    g = torch.tensor([-86.0, -87.0, -88.5, -89.0, -90.0, -100.0, -1000.0, -3e38])
    gu = torch.cat((g, torch.full((8,), 1e30))).bfloat16().reshape(1, 16)
    out = gpu.moe_swiglu(c.ctx, gu.cuda(), c.handle)[0].double().cpu()
    ref = X.swiglu64(gu)[0]
    # e^-g is off by at most |g| + 4 half steps of binary32, the rest by a few more
    assert ((out[:3] - ref[:3]).abs() <= (X.BF16_HALF + 128 * X.F32_STEP) * ref[:3].abs()).all()
    assert (out[3:] == 0).all()
    grad = gpu.moe_swiglu_backward(c.ctx, torch.ones(1, 8, dtype=torch.bfloat16, device="cuda"), gu.cuda(), c.handle)[0].double().cpu()
    assert (grad[3:8] == 0).all() and (grad[11:] == 0).all() and torch.isfinite(grad).all()
    c.close()

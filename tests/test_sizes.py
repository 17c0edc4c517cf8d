"""Sizes and settings of more than 32 bits, of which ctypes would pass the lower half, are refused."""
import pytest
import torch

import combine_moe_dispatch_layout_amd as moe

gpu_only = pytest.mark.gpu
B = moe._binding
LONG = 2 ** 32


def refused(status, f, *args, **kwargs):
    with pytest.raises(moe.MoeError) as e:
        f(*args, **kwargs)
    assert e.value.status == status


def meta(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device="meta")


@pytest.mark.parametrize("args", [(LONG + 24, 7168, 256), (24, LONG + 7168, 256), (24, 7168, LONG + 256), (24, 7168, 256, LONG)])
def test_workspace_queries(args):
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_linear_workspace, *args)
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_linear_backward_workspace, *args)


@pytest.mark.parametrize("place", range(4))
def test_router_settings(place):
    settings = [0, 1, 1, 1]
    settings[place] += LONG
    refused(moe.MOE_ERR_UNSUPPORTED, B._router, *settings, True, 1.0)


def test_shapes():
    class Ctx:
        cfg, device, handle = moe.make_config(4, 8, 1, 1, 1), 0, None
    refused(moe.MOE_ERR_CAPACITY, moe.moe_layer, Ctx(), meta(LONG + 1, 8), None, None, None, meta(1, 8, 16))
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_layer, Ctx(), meta(1, 8), None, None, None, meta(1, 8, LONG + 16))
    for shape in ((1, LONG + 8, 8), (1, 8, LONG + 8)):
        refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_expert_gemm, Ctx(), meta(1, 8), meta(*shape), None)
        refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_expert_gemm_fp8, Ctx(), meta(1, 8), None, meta(*shape), None, None)
        refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_expert_gemm_backward_rows, Ctx(), meta(1, 8), meta(*shape), None)
        refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_expert_gemm_backward_weights, Ctx(), meta(1, shape[1]), meta(1, shape[2]), None)
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_swiglu, Ctx(), meta(1, 2 * LONG + 16), None)
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_swiglu_fp8, Ctx(), meta(1, 2 * LONG + 256), None)
    refused(moe.MOE_ERR_UNSUPPORTED, moe.moe_swiglu_backward, Ctx(), meta(1, LONG + 8), meta(1, 2 * LONG + 16), None)


@gpu_only
def test_batches_of_more_than_32_bits(gpu):
    """2^32 and a few rows: not taken for a few."""
    T = LONG + 3
    if torch.cuda.mem_get_info()[0] < 120 * 2 ** 30:
        pytest.skip("needs 110 GB")
    ctx = gpu.Context(gpu.make_config(8, 8, 1, 1, 1))
    idx = torch.empty(T, 1, dtype=torch.int64, device="cuda")
    refused(gpu.MOE_ERR_CAPACITY, gpu.moe_dispatch_layout, ctx, idx)
    x = torch.empty(T, 8, dtype=torch.bfloat16, device="cuda")
    bufs, handle = gpu.DispatchBuffers(ctx), gpu.Handle(ctx)
    refused(gpu.MOE_ERR_CAPACITY, gpu.moe_dispatch, ctx, x, idx)
    refused(gpu.MOE_ERR_CAPACITY, gpu.prepare_dispatch, ctx, x, idx, False, bufs, handle)
    refused(gpu.MOE_ERR_CAPACITY, gpu.moe_dispatch_noalloc, ctx, x, idx, bufs, handle)
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    del idx
    refused(gpu.MOE_ERR_UNSUPPORTED, gpu.moe_linear, ctx, x, w)
    refused(gpu.MOE_ERR_UNSUPPORTED, gpu.moe_linear_backward, ctx, x, x, w, need_x=False)
    del x
    logits, d = (torch.empty(T, 1, device="cuda") for _ in range(2))
    idx = torch.empty(T, 1, dtype=torch.int64, device="cuda")
    refused(gpu.MOE_ERR_CAPACITY, gpu.moe_route, ctx, logits)
    refused(gpu.MOE_ERR_CAPACITY, gpu.moe_route_backward, ctx, d, logits, idx)
    ctx.close()
    del logits, d, idx
    torch.cuda.empty_cache()

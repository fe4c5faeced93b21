"""Host-side checks of the 4-bit weight entry points (no GPU): sizes, refusals in the
order and with the codes that the header states, and nothing enqueued for zero tokens."""
import ctypes

import pytest

import mixture_experts_layer_align_gb300 as moe

FP8, BF16, FP32 = moe.MOE_DT_FP8_E4M3, moe.MOE_DT_BF16, moe.MOE_DT_FP32


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_align_gb300 import build
    build.build()
    return moe.load()


def weight(**kw):
    base = dict(codes=16, scales=16, zeros=None, scale_dtype=FP32, group=64)
    base.update(kw)
    return moe.MoeW4Tensor(**base)


def test_workspace_size(lib):
    small = moe.moe_w4_workspace_size(1, 2048, 768, 128, 8)
    assert 0 < small < moe.moe_w4_workspace_size(64, 2048, 768, 128, 8)
    assert small % 256 == 0
    assert moe.moe_w4_workspace_size(1, 128, 128, 4, 5) == 0
    assert moe.moe_w4_workspace_size(1, 128, 128, 1025, 1) == 0
    assert moe.moe_w4_workspace_size(-1, 128, 128, 4, 1) == 0


def test_launch_count(lib):
    assert moe.moe_w4_launch_count(0, 2048, 768, 128, 8) == 0
    assert 1 <= moe.moe_w4_launch_count(1, 2048, 768, 128, 8) <= 7
    assert moe.moe_w4_launch_count(1, 2040, 768, 128, 8) == -1
    assert moe.moe_w4_launch_count(1, 2048, 700, 128, 8) == -1
    assert moe.moe_w4_launch_count(1, 2048, 768, 128, 129) == -1


@pytest.mark.parametrize("kw,w,code", [
    (dict(T=-1), {}, 1), (dict(N=0), {}, 1), (dict(K=0), {}, 1), (dict(K=48), {}, 2),
    (dict(dtype=FP8), {}, 1), (dict(dtype=9), {}, 1), (dict(x=None), {}, 1),
    (dict(x=24), {}, 1), (dict(out=None), {}, 1), (dict(out=18), {}, 1),
    (dict(out=17, dtype=BF16), {}, 1), ({}, dict(codes=None), 1), ({}, dict(codes=8), 1),
    ({}, dict(scales=None), 1), ({}, dict(scales=18), 1), ({}, dict(group=0), 1),
    ({}, dict(group=48), 1), ({}, dict(scale_dtype=FP8), 1), (dict(T=1 << 20), {}, 2),
    (dict(T=1 << 19, N=1 << 12), {}, 2), (dict(K=1 << 21), {}, 2),
    (dict(T=1 << 13, K=1 << 18), {}, 2), (dict(T=0), {}, 0), (dict(T=0, x=None, out=None), {}, 0),
])
def test_matvec_refusals(lib, kw, w, code):
    a = dict(x=16, T=2, K=64, N=8, out=16, dtype=FP32)
    a.update(kw)
    st = lib.moe_w4_matvec(ctypes.c_void_p(a["x"]), a["T"], a["K"], a["N"],
                           ctypes.byref(weight(**w)), ctypes.c_void_p(a["out"]), a["dtype"],
                           ctypes.c_void_p(16), 1 << 40, None)
    assert st == code


def test_matvec_null_weight(lib):
    assert lib.moe_w4_matvec(ctypes.c_void_p(16), 1, 32, 1, None, ctypes.c_void_p(16), FP32,
                             ctypes.c_void_p(16), 1 << 40, None) == 1


def test_matvec_scratch(lib):
    need = moe.moe_w4_matvec_scratch_size(5, 96)
    assert 0 < need < moe.moe_w4_matvec_scratch_size(9, 96)
    assert moe.moe_w4_matvec_scratch_size(0, 96) == 0
    for ptr, size in ((None, need), (8, need), (16, need - 1)):
        assert lib.moe_w4_matvec(ctypes.c_void_p(16), 5, 96, 3, ctypes.byref(weight()),
                                 ctypes.c_void_p(16), FP32, ctypes.c_void_p(ptr), size, None) == 3


def layer_args(**kw):
    base = dict(x=16, router_logits=16, w13=weight(), w2=weight(), T=4, H=128, I=64, E=8, top_k=2,
                renormalize=1, out=16, topk_ids_out=None, topk_w_out=None, counts_out=None)
    base.update(kw)
    return moe.MoeW4Args(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(top_k=0), 1), (dict(top_k=9), 1), (dict(E=1025), 1), (dict(T=-1), 1), (dict(H=0), 1),
    (dict(H=100), 2), (dict(I=72), 2), (dict(x=None), 1), (dict(x=20), 1), (dict(out=8), 1),
    (dict(router_logits=None), 1), (dict(topk_ids_out=2), 1), (dict(topk_w_out=2), 1),
    (dict(counts_out=2), 1), (dict(w13=weight(codes=None)), 1), (dict(w2=weight(scales=None)), 1),
    (dict(w2=weight(group=100)), 1), (dict(w13=weight(scale_dtype=FP8)), 1), (dict(T=0), 0),
    (dict(T=0, x=None, out=None, w13=weight(codes=None)), 0),
])
def test_layer_refusals(lib, kw, code):
    a = layer_args(**kw)
    assert lib.moe_w4_forward(ctypes.byref(a), ctypes.c_void_p(256), 1 << 40, None) == code


def test_layer_workspace_refusals(lib):
    a = layer_args()
    need = moe.moe_w4_workspace_size(4, 128, 64, 8, 2)
    assert lib.moe_w4_forward(ctypes.byref(a), ctypes.c_void_p(256), need - 1, None) == 3
    assert lib.moe_w4_forward(ctypes.byref(a), None, need, None) == 3
    assert lib.moe_w4_forward(ctypes.byref(a), ctypes.c_void_p(272), need, None) == 3
    assert lib.moe_w4_forward(None, ctypes.c_void_p(256), need, None) == 1

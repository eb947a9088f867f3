"""CPU checks of the MXFP4 calls: every refusal happens on the host before any HIP call."""
import ctypes

import pytest
import torch

from expert_routed_grouped_amd import moe

P = ctypes.c_void_p
A, B, C, D = P(0x10000000), P(0x20000000), P(0x30000000), P(0x40000000)  # never dereferenced


def off(p, n):
    return P(p.value + n)


def quantize(**kw):
    a = dict(x=A, xd=1, rows=4, K=64, c=B, s=C)
    a.update(kw)
    return moe.lib().moe_quantize_mx4(a["x"], a["xd"], a["rows"], a["K"], a["c"], a["s"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), -2), (dict(K=48), -2), (dict(rows=-1), -2), (dict(rows=1 << 40), -2), (dict(xd=2), -3), (dict(xd=5), -3),
    (dict(x=None), -1), (dict(c=None), -1), (dict(s=None), -1), (dict(x=off(A, 8)), -6), (dict(c=off(B, 2)), -6),
    (dict(rows=0, x=None), 0),
])
def test_quantize_validation(kw, code):
    assert quantize(**kw) == code


def dequantize(**kw):
    a = dict(c=A, s=B, md=5, rows=4, K=64, o=C, od=0)
    a.update(kw)
    return moe.lib().moe_dequantize_mx(a["c"], a["s"], a["md"], a["rows"], a["K"], a["o"], a["od"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=33), -2), (dict(rows=-1), -2), (dict(md=2), -3), (dict(md=4), -3), (dict(od=2), -3), (dict(od=3), -3),
    (dict(c=None), -1), (dict(s=None), -1), (dict(o=None), -1), (dict(o=off(C, 4)), -6), (dict(md=3, c=off(A, 4)), -6),
    (dict(c=off(A, 2)), -6), (dict(rows=0), 0),
])
def test_dequantize_validation(kw, code):
    assert dequantize(**kw) == code


def pack(**kw):
    a = dict(c=A, s=B, rows=32, K=256, pc=C, ps=D)
    a.update(kw)
    return moe.lib().moe_pack_mx4(a["c"], a["s"], a["rows"], a["K"], a["pc"], a["ps"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -2), (dict(rows=24), -2), (dict(K=64), -2), (dict(K=192), -2), (dict(rows=1 << 40), -2),
    (dict(c=None), -1), (dict(s=None), -1), (dict(pc=None), -1), (dict(ps=None), -1), (dict(c=off(A, 8)), -6),
    (dict(pc=off(C, 4)), -6), (dict(ps=off(D, 4)), -6),
    (dict(pc=A), -2), (dict(pc=off(A, 16)), -2), (dict(ps=B), -2), (dict(ps=off(C, 4080)), -2), (dict(pc=off(B, 16)), -2),
])
def test_pack_validation(kw, code):
    assert pack(**kw) == code


def test_packed_scale_bytes():
    f = moe.lib().moe_mx4_packed_scale_bytes
    assert f(32, 256) == 2 * 256 and f(16, 512) == 256 and f(48, 640) == 3 * 2 * 256
    assert f(8, 256) == 0 and f(16, 64) == 0 and f(-16, 128) == 0 and f(0, 128) == 0


def ffn(**kw):
    a = dict(a=A, s=A, ad=3, off=A, rt=A, rw=A, tr=A, El=8, T=16, k=2, H=256, I=128, gc=A, gs=A, dc=A, ds=A, y=A, yd=1,
             ws=A, wsb=1 << 30)
    a.update(kw)
    return moe.lib().moe_grouped_ffn_mx4(a["a"], a["s"], a["ad"], a["off"], a["rt"], a["rw"], a["tr"], a["El"], a["T"],
                                         a["k"], a["H"], a["I"], a["gc"], a["gs"], a["dc"], a["ds"], a["y"], a["yd"],
                                         a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(El=0), -2), (dict(El=1025), -2), (dict(k=0), -2), (dict(k=33), -2), (dict(H=192), -2),
    (dict(I=64), -2), (dict(I=192), -2), (dict(T=1 << 24), -2), (dict(T=1 << 23, I=1536), -2),
    (dict(H=1 << 16, I=1 << 15), -2), (dict(ad=1), -3), (dict(ad=2), -3), (dict(yd=3), -3),
    (dict(a=None), -1), (dict(s=None), -1), (dict(off=None), -1), (dict(rt=None), -1), (dict(rw=None), -1),
    (dict(tr=None), -1), (dict(gc=None), -1), (dict(gs=None), -1), (dict(dc=None), -1), (dict(ds=None), -1),
    (dict(y=None), -1), (dict(ws=None), -4), (dict(wsb=1000), -4), (dict(a=off(A, 8)), -6), (dict(s=off(A, 2)), -6),
    (dict(gs=off(A, 4)), -6), (dict(y=off(A, 8)), -6), (dict(ws=off(A, 128)), -6), (dict(T=0, a=None, y=None), 0),
])
def test_ffn_validation(kw, code):
    assert ffn(**kw) == code


def test_ffn_workspace_size():
    f = moe.moe_ffn_mx4_workspace_size
    assert f(100, 8, 128, 4096, 1536, moe.MOE_F32) >= 800 * (1536 + 48 + 4 * 4096)
    assert f(100, 8, 128, 4096, 1536, moe.MOE_BF16) >= 800 * (1536 + 48 + 2 * 4096)
    assert f(100, 8, 4, 4096, 1536, moe.MOE_F32) >= 400 * (1536 + 48 + 4 * 4096)
    assert f(100, 8, 128, 4096, 1500, moe.MOE_F32) == 0 and f(100, 8, 128, 4096, 1536, 3) == 0
    assert moe.moe_workspace_size(moe.MOE_OP_GROUPED_FFN_MX4, 100, 8, 128, 4096, 1536) == f(100, 8, 128, 4096, 1536)


def layer(**kw):
    a = dict(x=A, wr=A, b=None, T=4, H=256, E=16, k=2, lo=0, hi=16, I=128, gc=A, gs=A, dc=A, ds=A, ids=A, w=A, y=A, yd=1,
             ws=A, wsb=1 << 30)
    a.update(kw)
    return moe.lib().moe_decode_layer_mx4(a["x"], a["wr"], a["b"], a["T"], a["H"], a["E"], a["k"], a["lo"], a["hi"], a["I"],
                                          a["gc"], a["gs"], a["dc"], a["ds"], a["ids"], a["w"], a["y"], a["yd"], a["ws"],
                                          a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(T=65), -2), (dict(E=257, hi=257), -2), (dict(k=0), -2), (dict(k=17), -2),
    (dict(E=64, k=33, hi=64), -2), (dict(lo=-1), -2), (dict(lo=3, hi=3), -2), (dict(hi=17), -2), (dict(H=200), -2),
    (dict(H=8320), -2), (dict(I=96), -2), (dict(yd=2), -3), (dict(x=None), -1), (dict(wr=None), -1), (dict(gc=None), -1),
    (dict(gs=None), -1), (dict(dc=None), -1), (dict(ds=None), -1), (dict(ids=None), -1), (dict(w=None), -1),
    (dict(y=None), -1), (dict(ws=None), -4), (dict(wsb=5000), -4), (dict(x=off(A, 8)), -6), (dict(wr=off(A, 8)), -6),
    (dict(ds=off(A, 8)), -6), (dict(y=off(A, 4)), -6), (dict(ws=off(A, 64)), -6), (dict(T=0, x=None, ws=None), 0),
])
def test_layer_validation(kw, code):
    assert layer(**kw) == code


def test_layer_workspace_size():
    f = moe.lib().moe_decode_layer_mx4_workspace_size
    assert f(8, 8, 128, 4096, 1536) >= 256 + 8 * 4096 + 64 * (1536 + 48)
    assert f(65, 8, 128, 4096, 1536) == 0 and f(8, 8, 257, 4096, 1536) == 0 and f(8, 8, 128, 8320, 1536) == 0
    assert f(8, 8, 128, 4100, 1536) == 0
    assert all(f(t, 8, 128, 4096, 1536) <= f(t + 1, 8, 128, 4096, 1536) for t in range(64 - 1))
    assert moe.moe_workspace_size(moe.MOE_OP_DECODE_LAYER_MX4, 8, 8, 128, 4096, 1536) == f(8, 8, 128, 4096, 1536)


def test_binding_refuses_host_and_misshapen_tensors():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):
        moe.moe_quantize_mx4(torch.zeros(4, 64))  # host memory
    with pytest.raises(TypeError):
        moe.moe_quantize_mx4(torch.zeros((4, 64), dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.moe_quantize_mx4(torch.zeros(4, 64), codes=u8(4, 64))
    with pytest.raises(ValueError):
        moe.moe_dequantize_mx(u8(4, 48), u8(4, 2))
    with pytest.raises(TypeError):
        moe.moe_dequantize_mx(u8(4, 32), u8(4, 2), dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_pack_mx4(u8(2, 32, 64), u8(2, 32, 5))
    with pytest.raises(moe.MoEError):
        moe.moe_pack_mx4(u8(24, 64), u8(24, 4))
    wgu, wd = (u8(2, 16, 2, 1024), u8(2, 16, 1, 256)), (u8(2, 16, 1, 1024), u8(2, 16, 1, 256))  # H = 256, I = 128
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(a_codes=u8(3, 256), a_scales=u8(3, 8), offsets=i32(3), row_token=i32(6), row_w=torch.zeros(6),
              token_row=i32(3, 2), wgu=wgu, wd=wd)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_grouped_ffn_mx4(**ok)
    for bad in (dict(a_codes=u8(3, 200)), dict(a_scales=u8(3, 16)), dict(offsets=i32(2)), dict(row_token=i32(5)),
                dict(token_row=torch.zeros((3, 2))), dict(wd=(u8(2, 16, 2, 1024), u8(2, 16, 1, 256))),
                dict(wgu=(u8(2, 15, 2, 1024), u8(2, 15, 1, 256))), dict(y=torch.zeros((3, 128)))):
        with pytest.raises(ValueError) as err:
            moe.moe_grouped_ffn_mx4(**{**ok, **bad})
        assert "on the GPU" not in str(err.value)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    ok = dict(x=bf(3, 256), w_router_packed=torch.zeros(64, 8, 4), bias=None, k=2, e_begin=0, e_end=2, wgu=wgu, wd=wd,
              workspace=u8(100000))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_decode_layer_mx4(**ok)
    for bad in (dict(x=bf(3, 128)), dict(x=torch.zeros(3, 256)), dict(w_router_packed=torch.zeros(8, 256)),
                dict(w_router_packed=torch.zeros(32, 8, 4)), dict(e_end=3), dict(bias=torch.zeros(7)),
                dict(topk_ids=i32(3, 3)), dict(y=bf(2, 256)), dict(workspace=torch.zeros(1000))):
        with pytest.raises(ValueError) as err:
            moe.moe_decode_layer_mx4(**{**ok, **bad})
        assert "on the GPU" not in str(err.value)

"""CPU checks of the calls that train a MoE block: every refusal happens on the host before any HIP call, and what a call
on a given stream allocates by itself belongs to that stream."""
import ctypes

import pytest
import torch

from expert_routed_grouped_amd import moe

P = ctypes.c_void_p
BUF = [P(0x100000000 * (i + 1)) for i in range(24)]  # far apart, never dereferenced
A, B, C, D, E_, F, G, H_, I_, J, K_, L_, M_, N_, O_, Q, R, S = BUF[:18]
ODD = P(A.value + 4)


def off(p, n):
    return P(p.value + n)


def call(fn, order, defaults):
    def f(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a)
        a.update(kw)
        return getattr(moe.lib(), fn)(*[a[n] for n in order], None)
    return f


mm = call("moe_grouped_mm", "a idx ar w dt off El R N K out ot fl".split(),
          dict(a=A, idx=B, ar=10, w=C, dt=1, off=D, El=4, R=8, N=64, K=32, out=E_, ot=1, fl=0))


@pytest.mark.parametrize("kw,code", [
    (dict(El=0), -2), (dict(El=1025), -2), (dict(R=-1), -2), (dict(R=1 << 28), -2), (dict(N=0), -2), (dict(K=0), -2),
    (dict(N=1 << 15, K=1 << 14), -2), (dict(N=1 << 24), -2), (dict(ar=-1), -2), (dict(ar=0), -2), (dict(fl=2), -2), (dict(fl=3), -2),
    (dict(idx=None, ar=7), -2), (dict(R=(1 << 28) - 1, N=1 << 19, K=8), -2),
    (dict(dt=2), -3), (dict(dt=5), -3), (dict(ot=2), -3), (dict(dt=0, ot=1), -3),
    (dict(a=None), -1), (dict(w=None), -1), (dict(off=None), -1), (dict(out=None), -1),
    (dict(a=off(A, 8)), -6), (dict(w=off(C, 2)), -6), (dict(out=off(E_, 8)), -6), (dict(idx=off(B, 2)), -6), (dict(off=off(D, 1)), -6),
    (dict(out=A), -2), (dict(out=off(A, 10 * 64 - 16)), -2), (dict(out=off(A, -8 * 128 + 16)), -2), (dict(out=C), -2), (dict(out=B), -2),
    (dict(out=D), -2), (dict(R=0, a=None, out=None), 0),
])
def test_grouped_mm(kw, code):
    assert mm(**kw) == code


wgrad = call("moe_grouped_wgrad", "a ai ar b bi br dt off El R M N dw ot ws nws fl".split(),
             dict(a=A, ai=None, ar=8, b=B, bi=C, br=3, dt=1, off=D, El=4, R=8, M=64, N=32, dw=E_, ot=0, ws=F, nws=1 << 30, fl=0))


@pytest.mark.parametrize("kw,code", [
    (dict(El=0), -2), (dict(El=1025), -2), (dict(R=-1), -2), (dict(R=1 << 28), -2), (dict(M=0), -2), (dict(N=0), -2),
    (dict(M=1 << 15, N=1 << 14), -2), (dict(ar=7), -2), (dict(bi=None, br=7), -2), (dict(br=0), -2), (dict(ar=-1), -2), (dict(fl=2), -2),
    (dict(dt=2), -3), (dict(ot=2), -3), (dict(dt=0, ot=1), -3),
    (dict(a=None), -1), (dict(b=None), -1), (dict(off=None), -1), (dict(dw=None), -1),
    (dict(a=off(A, 8)), -6), (dict(b=off(B, 8)), -6), (dict(dw=off(E_, 4)), -6), (dict(bi=off(C, 2)), -6), (dict(off=off(D, 2)), -6),
    (dict(dw=A), -2), (dict(dw=B), -2), (dict(dw=C), -2), (dict(dw=D), -2), (dict(dw=off(A, -4 * 64 * 32 * 4 + 16)), -2),
])
def test_grouped_wgrad(kw, code):
    assert wgrad(**kw) == code


def test_grouped_wgrad_workspace():
    size = moe.moe_grouped_wgrad_workspace_size
    assert size(0, 8, 8, 8) == 0 and size(2, -1, 8, 8) == 0 and size(2, 8, 0, 8) == 0
    need = size(1, 100000, 32, 32)
    if need:
        kw = dict(El=1, R=100000, ar=100000, M=32, N=32, nws=need)
        assert wgrad(**kw, ws=None) == -4 and wgrad(**{**kw, "nws": need - 1}) == -4
        assert wgrad(**kw, ws=off(F, 16)) == -6
        assert wgrad(**kw, ws=A) == -2 and wgrad(**kw, ws=off(E_, 256)) == -2


swiglu = call("moe_swiglu", "gu dt off w El R I h".split(), dict(gu=A, dt=1, off=B, w=C, El=4, R=8, I=64, h=D))


@pytest.mark.parametrize("kw,code", [
    (dict(El=0), -2), (dict(El=1025), -2), (dict(R=-1), -2), (dict(R=1 << 28), -2), (dict(I=0), -2), (dict(I=1 << 24), -2),
    (dict(dt=2), -3), (dict(dt=5), -3), (dict(gu=None), -1), (dict(h=None), -1), (dict(gu=off(A, 8)), -6), (dict(h=off(D, 8)), -6),
    (dict(w=off(C, 2)), -6), (dict(h=A), -2), (dict(h=off(A, 8 * 256 - 16)), -2), (dict(h=C), -2), (dict(h=B), -2), (dict(R=0, gu=None), 0),
])
def test_swiglu(kw, code):
    assert swiglu(**kw) == code


backward = call("moe_swiglu_backward", "gu dh dt off w El R I dgu h dw".split(),
                dict(gu=A, dh=B, dt=0, off=C, w=D, El=4, R=8, I=64, dgu=E_, h=F, dw=G))


@pytest.mark.parametrize("kw,code", [
    (dict(El=0), -2), (dict(R=-1), -2), (dict(I=0), -2), (dict(dt=3), -3), (dict(gu=None), -1), (dict(dh=None), -1), (dict(dgu=None), -1),
    (dict(gu=off(A, 4)), -6), (dict(dh=off(B, 4)), -6), (dict(dgu=off(E_, 4)), -6), (dict(h=off(F, 4)), -6), (dict(dw=off(G, 2)), -6),
    (dict(dgu=off(A, 16)), -2), (dict(dgu=B), -2), (dict(h=A), -2), (dict(h=off(B, 16)), -2), (dict(dw=D), -2), (dict(dw=A), -2),
    (dict(h=E_), -2), (dict(dw=F), -2), (dict(dgu=D), -2), (dict(h=C), -2), (dict(R=0, gu=None, dgu=None), 0),
])
def test_swiglu_backward(kw, code):
    assert backward(**kw) == code


route = call("moe_route_backward", "ids g d T k E H x wr dt off rt rows rd at R dx xd dw db".split(),
             dict(ids=A, g=B, d=C, T=8, k=2, E=4, H=64, x=D, wr=E_, dt=1, off=F, rt=G, rows=I_, rd=1, at=J, R=16, dx=K_, xd=0,
                  dw=L_, db=M_))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(k=0), -2), (dict(k=5), -2), (dict(k=33, E=64), -2), (dict(E=1025), -2), (dict(H=0), -2), (dict(H=(1 << 20) + 1), -2),
    (dict(T=1 << 27), -2), (dict(R=-1), -2), (dict(dt=2), -3), (dict(xd=2), -3), (dict(rd=2), -3),
    (dict(ids=None), -1), (dict(g=None), -1), (dict(d=None), -1), (dict(x=None), -1), (dict(wr=None), -1), (dict(off=None), -1),
    (dict(rt=None), -1), (dict(at=None), -1), (dict(dx=None, dw=None, db=None), -1),
    (dict(x=off(D, 8)), -6), (dict(wr=off(E_, 8)), -6), (dict(rows=off(I_, 8)), -6),
    (dict(dx=off(K_, 8)), -6), (dict(dw=off(L_, 4)), -6), (dict(ids=ODD.value and off(A, 2)), -6),
    (dict(dx=D), -2), (dict(dx=I_), -2), (dict(dw=E_), -2), (dict(db=L_), -2), (dict(db=B), -2),
    (dict(T=0, dw=None, db=None), 0),
])
def test_route_backward(kw, code):
    assert route(**kw) == code


norm = call("moe_block_norm", "x xd y yd wn wp g wd gk sc eps T H xo n rn rp".split(),
            dict(x=A, xd=1, y=B, yd=0, wn=C, wp=D, g=E_, wd=0, gk=1, sc=1.0, eps=1e-6, T=8, H=64, xo=F, n=G, rn=H_, rp=I_))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(T=1 << 30), -2), (dict(H=0), -2), (dict(H=16385), -2), (dict(eps=0.0), -2), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2), (dict(gk=3), -2), (dict(gk=-1), -2), (dict(gk=0), -2), (dict(g=None), -2), (dict(y=None), -2),
    (dict(y=None, xo=None, wp=None, g=None, gk=0, rp=None, sc=0.5), -2), (dict(wp=None), -2),
    (dict(xd=2), -3), (dict(yd=2), -3), (dict(wd=2), -3), (dict(x=None), -1), (dict(n=None), -1), (dict(wn=None), -1),
    (dict(wn=None, n=None, xo=None), -1), (dict(x=off(A, 8)), -6), (dict(y=off(B, 8)), -6), (dict(wn=off(C, 8)), -6), (dict(n=off(G, 8)), -6),
    (dict(g=off(E_, 4)), -6), (dict(rn=off(H_, 2)), -6),
    (dict(xo=off(A, 16)), -2), (dict(n=A), -2), (dict(n=B), -2), (dict(n=F), -2), (dict(rn=G), -2), (dict(rp=H_), -2), (dict(xo=B), -2),
    (dict(T=0, x=None), 0),
])
def test_block_norm(kw, code):
    assert norm(**kw) == code


norm_back = call("moe_block_norm_backward", "xo xd y yd wn wp g wd gk sc rn rp dxo dn T H dx dy dyd dwn dwp dg ws nws".split(),
                 dict(xo=A, xd=1, y=B, yd=0, wn=C, wp=D, g=E_, wd=0, gk=1, sc=1.0, rn=F, rp=G, dxo=H_, dn=I_, T=8, H=64, dx=J, dy=K_, dyd=0,
                      dwn=L_, dwp=M_, dg=N_, ws=O_, nws=1 << 20))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(H=0), -2), (dict(H=16385), -2), (dict(gk=3), -2), (dict(gk=0), -2), (dict(g=None, dg=None), -2), (dict(y=None), -2),
    (dict(wn=None), -2), (dict(wp=None), -2), (dict(xd=2), -3), (dict(yd=5), -3), (dict(dyd=2), -3), (dict(wd=2), -3), (dict(dn=None, dxo=None), -1),
    (dict(xo=None), -1), (dict(rn=None), -1), (dict(rp=None), -1), (dict(wn=None, dwn=None), -1), (dict(dx=None, dy=None, dwn=None, dwp=None, dg=None), -1),
    (dict(ws=None), -4), (dict(nws=16), -4), (dict(xo=off(A, 8)), -6), (dict(dx=off(J, 8)), -6), (dict(dwn=off(L_, 4)), -6), (dict(ws=off(O_, 16)), -6),
    (dict(dx=A), -2), (dict(dx=off(H_, 16)), -2), (dict(dy=B), -2), (dict(dy=J), -2), (dict(dwn=C), -2), (dict(dwp=L_), -2), (dict(ws=J), -2),
    (dict(dg=E_), -2), (dict(T=0, dwn=None, dwp=None, dg=None), 0),
])
def test_block_norm_backward(kw, code):
    assert norm_back(**kw) == code


# ------------------------------------------------------------------ the binding
T, E, K, H, I = 4, 4, 2, 64, 32
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
f32 = lambda *s: torch.zeros(s)  # noqa: E731
PERM = dict(offsets=i32(E + 1), row_token=i32(T * K))
CALLS = {  # name: (tensors it allocates, the call)
    "moe_grouped_mm": (1, lambda s: moe.moe_grouped_mm(bf(T, H), bf(E, I, H), i32(E + 1), row_index=i32(T * K), stream=s)),
    "moe_swiglu": (1, lambda s: moe.moe_swiglu(bf(T, 2 * I), stream=s)),
    "moe_swiglu_backward": (3, lambda s: moe.moe_swiglu_backward(bf(T, 2 * I), bf(T, I), row_w=f32(T), stream=s)),
    "moe_route_backward": (3, lambda s: moe.moe_route_backward(i32(T, K), f32(T, K), f32(T, K), bf(T, H), bf(E, H), PERM, stream=s)),
    "moe_block_norm": (4, lambda s: moe.moe_block_norm(bf(T, H), f32(H), y=f32(T, H), w_post=f32(H), stats=True, stream=s)),
    "moe_block_norm_backward": (5, lambda s: moe.moe_block_norm_backward(
        bf(T, H), f32(H), f32(T), bf(T, H), y=f32(T, H), w_post=f32(H), rstd_post=f32(T), gate=f32(H), stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_own_buffers_belong_to_the_stream(name, monkeypatch):
    """Every buffer goes through ``_new`` with the stream of the call.  (Host tensors: the call ends before the library.)"""
    n, run = CALLS[name]
    made, empty, stream = [], torch.empty, object()
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream: made.append(stream) or empty(shape, dtype=dtype))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, lambda *a, **k: pytest.fail("allocated on the current stream"))
    with pytest.raises(ValueError, match="on the GPU"):
        run(stream)
    assert made == [stream] * n


def test_wgrad_buffers_belong_to_the_stream(monkeypatch):
    made, empty, stream = [], torch.empty, object()
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream: made.append(stream) or empty(shape, dtype=dtype))
    R = 100000
    with pytest.raises(ValueError, match="on the GPU"):
        moe.moe_grouped_wgrad(bf(R, 8), bf(R, 8), i32(2), stream=stream)
    assert made == [stream] * (1 + (moe.moe_grouped_wgrad_workspace_size(1, R, 8, 8) > 0))


@pytest.mark.parametrize("run", [
    lambda: moe.moe_grouped_mm(bf(T, H), bf(E, I, H + 8), i32(E + 1)),
    lambda: moe.moe_grouped_mm(bf(T, H), f32(E, I, H), i32(E + 1)),
    lambda: moe.moe_grouped_mm(bf(T, H), bf(I, H), i32(2)),
    lambda: moe.moe_grouped_mm(bf(T, H), bf(E, I, H), i32(E)),
    lambda: moe.moe_grouped_mm(bf(T, 2 * H)[:, ::2], bf(E, I, H), i32(E + 1)),
    lambda: moe.moe_grouped_mm(bf(T, H), bf(E, I, H), i32(E + 1), row_index=i32(2), out=bf(4, I)),
    lambda: moe.moe_grouped_mm(bf(T, H), bf(E, I, H), torch.zeros(E + 1, dtype=torch.int64)),
    lambda: moe.moe_grouped_wgrad(bf(T, H), f32(T, I), i32(E + 1)),
    lambda: moe.moe_grouped_wgrad(bf(T, H), bf(T, I), i32(E + 1), add=True),
    lambda: moe.moe_grouped_wgrad(bf(T, H), bf(T, I), i32(E + 1), out=bf(E, I, H)),
    lambda: moe.moe_swiglu(bf(T, 33)),
    lambda: moe.moe_swiglu(bf(T, 2 * I), row_w=bf(T)),
    lambda: moe.moe_swiglu_backward(bf(T, 2 * I), bf(T, I + 1)),
    lambda: moe.moe_route_backward(i32(T, K), f32(T, K), f32(T, K), bf(T, H), f32(E, H), PERM),
    lambda: moe.moe_route_backward(i32(T, K), f32(T, K), f32(T, K), bf(T, H), bf(E, H), dict(PERM, row_token=i32(3))),
    lambda: moe.moe_block_norm(bf(T, H), f32(H + 1)),
    lambda: moe.moe_block_norm(bf(T, H), f32(H), y=f32(T, H), w_post=bf(H)),
    lambda: moe.moe_block_norm(bf(T, H), f32(H), y=f32(T, H), gate=f32(T)),
    lambda: moe.moe_block_norm(bf(T, H), f32(H), y=f32(T, H), gate=f32(H, 1)),
    lambda: moe.moe_block_norm_backward(bf(T, H), f32(H), f32(T), f32(T, H)),
])
def test_binding_refuses(run):
    with pytest.raises((ValueError, TypeError)):
        run()

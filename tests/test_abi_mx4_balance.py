"""The entry points of the 4-bit experts and of the balance loss refuse bad arguments
on the host (CPU only: no call here reaches a kernel)."""
import ctypes
import os

import pytest
import torch

from mixture_experts_layer_sort_amd import _lib as L

FAKE = 0x10000  # never dereferenced
BAD = 2 ** 64 - 1
W, R = L.MOE_MX4_WEIGHTS, L.MOE_MX4_ROWS


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from mixture_experts_layer_sort_amd.build import build
        build()
    return L.lib()


def at(i):
    """Distinct, well separated addresses."""
    return FAKE + i * (1 << 32)


def q(i, scales=None):
    return L.moe_mx4(at(i), at(i + 1) if scales is None else scales)


def D(N=8, H=128, F=256, E=4, K=2, dtype=L.MOE_BF16):
    return L.dims(N, H, F, E, K, dtype)


def test_mx4_bytes(lib):
    assert L.moe_mx4_code_bytes(W, 3, 256, 384) == 3 * 256 * 384 // 2
    assert L.moe_mx4_scale_bytes(W, 3, 256, 384) == 3 * 384 * 16
    assert L.moe_mx4_scale_bytes(W, 3, 640, 128) == 3 * 128 * 32
    assert L.moe_mx4_code_bytes(R, 5, 1024, 1) == 5 * 512
    assert L.moe_mx4_scale_bytes(R, 5, 1024, 1) == 5 * 32
    assert L.moe_mx4_code_bytes(R, 0, 128, 1) == 0


SIZES = [((2, 1, 128, 128), L.MOE_EINVAL), ((W, -1, 128, 128), L.MOE_EINVAL), ((W, 1, 0, 128), L.MOE_EINVAL),
         ((W, 1, 128, 0), L.MOE_EINVAL), ((W, 1, 96, 128), L.MOE_EINVAL), ((W, 1, 128, 64), L.MOE_EINVAL),
         ((R, 1, 128, 128), L.MOE_EINVAL), ((R, 1, 64, 1), L.MOE_EINVAL),
         ((W, 1, (1 << 20) + 128, 128), L.MOE_EUNSUPPORTED), ((W, 1, 128, (1 << 20) + 128), L.MOE_EUNSUPPORTED),
         ((R, 1 << 31, 128, 1), L.MOE_EUNSUPPORTED), ((R, 1 << 27, 128, 1), L.MOE_EUNSUPPORTED),
         ((R, (1 << 16) + 1, 1 << 20, 1), L.MOE_EUNSUPPORTED), ((W, 2, 1 << 20, 1 << 20), L.MOE_EUNSUPPORTED)]


@pytest.mark.parametrize("sizes,status", SIZES)
def test_mx4_sizes_refused(lib, sizes, status):
    assert L.moe_mx4_code_bytes(*sizes) == BAD and L.moe_mx4_scale_bytes(*sizes) == BAD
    p = ctypes.byref(q(2))
    assert lib.moe_mx4_quantize(*sizes, L.MOE_BF16, at(1), p, None) == status
    assert lib.moe_mx4_dequantize(*sizes, L.MOE_BF16, p, at(1), None) == status


def test_mx4_quantize_pointers(lib):
    def both(v=at(1), t=q(2), dtype=L.MOE_BF16, count=4):
        p = None if t is None else ctypes.byref(t)
        got = {lib.moe_mx4_quantize(W, count, 128, 128, dtype, v, p, None),
               lib.moe_mx4_dequantize(W, count, 128, 128, dtype, p, v, None)}
        assert len(got) == 1
        return got.pop()

    assert both(dtype=2) == L.MOE_EUNSUPPORTED
    for kw in (dict(v=None), dict(v=at(1) + 8), dict(t=None), dict(t=L.moe_mx4(None, at(3))),
               dict(t=L.moe_mx4(at(2), None)), dict(t=L.moe_mx4(at(2) + 4, at(3))), dict(t=L.moe_mx4(at(2), at(3) + 8))):
        assert both(**kw) == L.MOE_EINVAL, kw
    n = 4 * 128 * 128
    for t in (L.moe_mx4(at(1), at(3)), L.moe_mx4(at(1) + 2 * n - 16, at(3)), L.moe_mx4(at(2), at(1) + 16),
              L.moe_mx4(at(2), at(2)), L.moe_mx4(at(2), at(2) + n // 2 - 16)):
        assert both(t=t) == L.MOE_EINVAL
    assert both(count=0) == L.MOE_OK


def gate_up(d, x=q(1), flat=at(3), wg=q(4), wu=q(6), tiles=at(8), nt=at(9), act=at(10)):
    r = lambda t: None if t is None else ctypes.byref(t)
    return L.lib().moe_mx4_gate_up(ctypes.byref(d), r(x), flat, r(wg), r(wu), tiles, nt, act, None)


def down(d, a=q(1), w=q(4), tiles=at(8), nt=at(9), ys=at(10)):
    r = lambda t: None if t is None else ctypes.byref(t)
    return L.lib().moe_mx4_down(ctypes.byref(d), r(a), r(w), tiles, nt, ys, None)


def test_mx4_products_refuse(lib):
    for kw in (dict(x=None), dict(x=L.moe_mx4(None, at(2))), dict(wg=L.moe_mx4(at(4), at(5) + 4)), dict(wu=None),
               dict(flat=None), dict(tiles=None), dict(nt=at(9) + 2), dict(act=None), dict(act=at(10) + 8),
               dict(act=at(1)), dict(act=at(2)), dict(act=at(3)), dict(act=at(4)), dict(act=at(7)), dict(act=at(8)),
               dict(act=at(9))):
        assert gate_up(D(), **kw) == L.MOE_EINVAL, kw
    for kw in (dict(a=None), dict(w=None), dict(w=L.moe_mx4(at(4) + 8, at(5))), dict(tiles=None), dict(nt=None),
               dict(ys=None), dict(ys=at(10) + 4), dict(ys=at(1)), dict(ys=at(2)), dict(ys=at(4)), dict(ys=at(5)),
               dict(ys=at(8)), dict(ys=at(9))):
        assert down(D(), **kw) == L.MOE_EINVAL, kw
    for d, st in ((D(H=100), L.MOE_EINVAL), (D(E=300), L.MOE_EUNSUPPORTED), (D(dtype=5), L.MOE_EUNSUPPORTED)):
        assert gate_up(d) == st and down(d) == st
    assert gate_up(D(N=0)) == L.MOE_OK and down(D(N=0)) == L.MOE_OK
    for d in (D(H=(1 << 20) + 128), D(F=(1 << 20) + 128)):  # no 4-bit tensor has such a side
        assert gate_up(d) == down(d) == L.MOE_EUNSUPPORTED
        assert L.moe_mx4_decode_workspace_bytes(d) == 2 ** 64 - 1 and decode(d, nb=1 << 40) == L.MOE_EUNSUPPORTED
    # the rows' codes have 32-bit offsets
    assert gate_up(D(N=1 << 20, H=1 << 13), act=at(1)) == L.MOE_EUNSUPPORTED
    assert gate_up(D(N=(1 << 20) - 1, H=1 << 13), act=at(1)) == L.MOE_EINVAL  # the next check's


def decode(d, ds=None, shared=(None, None, None), nb=None, ws=at(30), **kw):
    a = dict(x=at(1), w_r=at(2), bias=None, wg=q(3), wu=q(5), wd=q(7), topk=at(9), gates=at(10), y=at(11))
    a.update(kw)
    r = lambda t: None if t is None else ctypes.byref(t)
    nb = L.moe_mx4_decode_workspace_bytes(d, ds) if nb is None else nb
    return L.lib().moe_mx4_decode(ctypes.byref(d), a["x"], a["w_r"], a["bias"], r(a["wg"]), r(a["wu"]), r(a["wd"]),
                                  r(ds), *(r(s) for s in shared), a["topk"], a["gates"], a["y"], ws, nb, None)


def test_mx4_decode_refuses(lib):
    assert 0 < L.moe_mx4_decode_workspace_bytes(D()) < BAD
    assert L.moe_mx4_decode_workspace_bytes(D(N=0)) == 0
    for d, st in ((D(N=L.MOE_DECODE_MAX_TOKENS + 1), L.MOE_EUNSUPPORTED), (D(H=100), L.MOE_EINVAL),
                  (D(K=5), L.MOE_EUNSUPPORTED), (D(N=-1), L.MOE_EINVAL), (D(dtype=5), L.MOE_EUNSUPPORTED)):
        assert L.moe_mx4_decode_workspace_bytes(d) == BAD
        assert decode(d, nb=1 << 30) == st
    need = L.moe_mx4_decode_workspace_bytes(D())
    assert decode(D(), nb=need - 1) == L.MOE_EWORKSPACE
    assert decode(D(), ws=None) == L.MOE_EWORKSPACE
    assert decode(D(), ws=at(30) + 8) == L.MOE_EWORKSPACE
    for name in ("x", "w_r", "topk", "gates", "y"):
        assert decode(D(), **{name: None}) == L.MOE_EINVAL, name
        assert decode(D(), **{name: at(20) + 2}) == L.MOE_EINVAL, name
    for name in ("wg", "wu", "wd"):
        assert decode(D(), **{name: None}) == L.MOE_EINVAL, name
        assert decode(D(), **{name: L.moe_mx4(at(20), None)}) == L.MOE_EINVAL, name
    assert decode(D(), bias=at(21) + 4) == L.MOE_EINVAL
    inputs = dict(x=at(1), w_r=at(2), bias=at(20), wg=at(3), wgs=at(4), wu=at(5), wus=at(6), wd=at(7), wds=at(8))
    for name, a in inputs.items():
        for out in ("topk", "gates", "y"):
            assert decode(D(), bias=at(20), **{out: a}) == L.MOE_EINVAL, (out, name)
        assert decode(D(), bias=at(20), ws=a) == L.MOE_EINVAL, name
    for i, j in (("topk", "gates"), ("topk", "y"), ("gates", "y")):
        assert decode(D(), **{i: at(25), j: at(25)}) == L.MOE_EINVAL
    assert decode(D(), y=at(30) + need - 16) == L.MOE_EINVAL
    assert decode(D(N=0), nb=0, ws=None) == L.MOE_OK


def test_mx4_decode_shared_expert_dims(lib):
    s = (q(12), q(14), q(16))
    good = D(F=384, E=1, K=1)
    need = L.moe_mx4_decode_workspace_bytes(D(), good)
    assert L.moe_mx4_decode_workspace_bytes(D()) < need < BAD
    assert decode(D(), good, s, nb=need - 1) == L.MOE_EWORKSPACE
    assert decode(D(), good, (q(12), None, q(16))) == L.MOE_EINVAL
    assert decode(D(), good, (q(12), L.moe_mx4(at(14), None), q(16))) == L.MOE_EINVAL
    assert decode(D(), None, s) == L.MOE_EINVAL
    assert decode(D(), good, s, y=at(17)) == L.MOE_EINVAL
    for ds in (D(E=2, K=1), D(E=1, K=1, H=256), D(E=1, K=1, N=7), D(E=1, K=1, dtype=L.MOE_F32)):
        assert L.moe_mx4_decode_workspace_bytes(D(), ds) == BAD
        assert decode(D(), ds, s, nb=1 << 30) == L.MOE_EINVAL


def B(N=64, E=8, K=2, seq_len=16, dtype=L.MOE_F32, score=L.MOE_SCORE_SOFTMAX, alpha=0.01, z_coef=0.0):
    return L.moe_balance(N, E, K, seq_len, dtype, score, alpha, z_coef)


def loss(b, sb=None, wb=None, **kw):
    a = dict(logits=at(1), topk=at(2), bias=None, mask=at(3), loss=at(4), counts=at(5), state=at(6), ws=at(7))
    a.update(kw)
    sb = L.moe_balance_state_bytes(b) if sb is None else sb
    wb = L.moe_balance_workspace_bytes(b) if wb is None else wb
    return L.lib().moe_balance_loss(ctypes.byref(b), a["logits"], a["topk"], a["bias"], a["mask"], a["loss"],
                                    a["counts"], a["state"], sb, a["ws"], wb, None)


def bwd(b, **kw):
    a = dict(logits=at(1), mask=at(3), state=at(6), dloss=at(8), d=at(9))
    a.update(kw)
    return L.lib().moe_balance_loss_bwd(ctypes.byref(b), a["logits"], a["mask"], a["state"], a["dloss"], a["d"], None)


@pytest.mark.parametrize("b,status", [
    (B(N=-1), L.MOE_EINVAL), (B(N=65), L.MOE_EINVAL), (B(seq_len=0), L.MOE_EINVAL), (B(E=0), L.MOE_EINVAL),
    (B(K=0), L.MOE_EINVAL), (B(K=9, E=16), L.MOE_EUNSUPPORTED), (B(K=5, E=4), L.MOE_EUNSUPPORTED),
    (B(E=257), L.MOE_EUNSUPPORTED), (B(dtype=3), L.MOE_EUNSUPPORTED), (B(score=2), L.MOE_EINVAL),
    (B(alpha=float("nan")), L.MOE_EINVAL), (B(z_coef=float("inf")), L.MOE_EINVAL),
    (B(N=1 << 30, seq_len=1, E=8), L.MOE_EUNSUPPORTED), (B(N=1 << 28, seq_len=1 << 20, E=2, K=1), L.MOE_EUNSUPPORTED),
    (B(N=(1 << 23) + 1, seq_len=1, E=2, K=1), L.MOE_EUNSUPPORTED)])
def test_balance_options_refused(lib, b, status):
    assert L.moe_balance_state_bytes(b) == BAD and L.moe_balance_workspace_bytes(b) == BAD
    assert loss(b, 1 << 40, 1 << 40) == status
    assert bwd(b) == status


def test_balance_pointers(lib):
    b = B()
    sb, wb = L.moe_balance_state_bytes(b), L.moe_balance_workspace_bytes(b)
    for kw in (dict(sb=sb - 1), dict(wb=wb - 1), dict(state=None), dict(ws=None), dict(ws=at(7) + 8)):
        assert loss(b, **kw) == L.MOE_EWORKSPACE, kw
    for name in ("logits", "loss", "counts"):
        assert loss(b, **{name: None}) == L.MOE_EINVAL, name
        assert loss(b, **{name: at(20) + 8}) == L.MOE_EINVAL, name
    for kw in (dict(topk=at(2) + 4), dict(mask=at(3) + 1), dict(bias=at(20)), dict(topk=None, bias=at(20) + 4)):
        assert loss(b, **kw) == L.MOE_EINVAL, kw
    for out in ("loss", "counts", "state", "ws"):
        for i in (1, 2, 3):
            assert loss(b, **{out: at(i)}) == L.MOE_EINVAL, (out, i)
        for other in ("loss", "counts", "state", "ws"):
            if other != out:
                assert loss(b, **{out: at(30), other: at(30)}) == L.MOE_EINVAL
    for kw in (dict(logits=None), dict(state=None), dict(d=None), dict(d=at(9) + 4), dict(dloss=at(8) + 2),
               dict(mask=at(3) + 1), dict(d=at(1) + 16), dict(d=at(3)), dict(d=at(6)), dict(d=at(8) - 16)):
        assert bwd(b, **kw) == L.MOE_EINVAL, kw
    assert loss(B(N=0), sb=0, wb=0, state=None, ws=None) == L.MOE_OK and bwd(B(N=0)) == L.MOE_OK


@pytest.mark.parametrize("B_,T,E", [(1, 1, 1), (1, 203, 8), (7, 1, 256), (64, 1024, 64), (1, 1 << 22, 256), (3, 77, 12)])
def test_balance_scratch_grows_with_sequences(lib, B_, T, E):
    b = B(N=B_ * T, E=E, K=1, seq_len=T)
    assert L.moe_balance_state_bytes(b) >= 4 * B_ * (E + 1)
    assert 4 * B_ * (2 * E + 2) <= L.moe_balance_workspace_bytes(b) < BAD
    assert L.moe_balance_workspace_bytes(b) <= 4 * (B_ + 1024) * (2 * E + 2) + B_ * (E * 4 + 24) + 1024


def test_products_before_any_grouping_are_refused(monkeypatch):
    """gate_up() and down() of a runner that has no tile list yet (CPU tensors, the 4-bit ones without addresses)."""
    from mixture_experts_layer_sort_amd import mx4
    monkeypatch.setattr(L, "mx4", lambda codes, scales: None)
    r = mx4.MoEMx4Runner(5, 128, 256, 2, 2, torch.float32, "cpu")
    x, a = mx4.MoEMx4Tensor(R, (5, 128), "cpu"), mx4.MoEMx4Tensor(R, (10, 256), "cpu")
    up, down = mx4.MoEMx4Tensor(W, (2, 128, 256), "cpu"), mx4.MoEMx4Tensor(W, (2, 256, 128), "cpu")
    with pytest.raises(RuntimeError, match="before meta"):
        r.gate_up(x, up, up)
    with pytest.raises(RuntimeError, match="before meta"):
        r.down(a, down)
    assert int(r.num_tiles) == 0
    with pytest.raises(ValueError):  # a refused grouping is none
        r.meta(torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(RuntimeError):
        r.down(a, down)
    none = mx4.MoEMx4Runner(0, 128, 256, 2, 2, torch.float32, "cpu")
    assert none.gate_up(mx4.MoEMx4Tensor(R, (0, 128), "cpu"), up, up).shape == (0, 256)

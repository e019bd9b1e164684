"""The entry points for few tokens, the residual RMS norm and gradient clipping
refuse bad arguments on the host (CPU only: no call here reaches a kernel)."""
import ctypes
import os

import pytest
import torch

from mixture_experts_layer_sort_amd import _lib as L

FAKE = 0x10000  # never dereferenced
BAD = 2 ** 64 - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from mixture_experts_layer_sort_amd.build import build
        build()
    return L.lib()


def D(N=8, H=128, F=256, E=4, K=2, dtype=L.MOE_BF16):
    return L.dims(N, H, F, E, K, dtype)


def at(i):
    """Distinct, well separated addresses."""
    return FAKE + i * (1 << 32)


def decode(d, ds=None, shared=(None, None, None), y=at(7), ws=at(8), nb=None, **kw):
    a = dict(x=at(1), w_r=at(2), bias=None, wg=at(3), wu=at(4), wd=at(5), topk=at(6), gates=at(9))
    a.update(kw)
    nb = L.moe_decode_workspace_bytes(d, ds) if nb is None else nb
    return L.lib().moe_decode(ctypes.byref(d), a["x"], a["w_r"], a["bias"], a["wg"], a["wu"], a["wd"],
                              None if ds is None else ctypes.byref(ds), *shared, a["topk"], a["gates"], y, ws, nb, None)


def test_decode_limits_and_workspace(lib):
    assert 0 < L.moe_decode_workspace_bytes(D()) < BAD
    assert L.moe_decode_workspace_bytes(D(N=0)) == 0
    assert L.moe_decode_workspace_bytes(D(N=L.MOE_DECODE_MAX_TOKENS)) < BAD
    for d, st in ((D(N=L.MOE_DECODE_MAX_TOKENS + 1), L.MOE_EUNSUPPORTED), (D(H=100), L.MOE_EINVAL),
                  (D(E=300), L.MOE_EUNSUPPORTED), (D(K=5), L.MOE_EUNSUPPORTED), (D(N=-1), L.MOE_EINVAL),
                  (D(dtype=5), L.MOE_EUNSUPPORTED)):
        assert L.moe_decode_workspace_bytes(d) == BAD
        assert decode(d, nb=1 << 30) == st
    need = L.moe_decode_workspace_bytes(D())
    assert decode(D(), nb=need - 1) == L.MOE_EWORKSPACE
    assert decode(D(), ws=None) == L.MOE_EWORKSPACE
    assert decode(D(), ws=at(8) + 8) == L.MOE_EWORKSPACE


def test_decode_pointers(lib):
    for name in ("x", "w_r", "wg", "wu", "wd", "topk", "gates"):
        assert decode(D(), **{name: None}) == L.MOE_EINVAL, name
        assert decode(D(), **{name: at(20) + 2}) == L.MOE_EINVAL, name
    assert decode(D(), y=None) == L.MOE_EINVAL
    assert decode(D(), bias=at(21) + 4) == L.MOE_EINVAL
    assert decode(D(), y=at(1)) == L.MOE_EINVAL                 # y on x
    assert decode(D(), y=at(1) + 8 * 128 * 2 - 16) == L.MOE_EINVAL
    assert decode(D(N=0), nb=0, ws=None) == L.MOE_OK            # nothing to do


def test_decode_outputs_and_workspace_overlap_nothing(lib):
    need = L.moe_decode_workspace_bytes(D())
    a = dict(topk=at(30), gates=at(31), y=at(32), x=at(33))
    for name in a:
        for other in a:
            if name < other:
                assert decode(D(), ws=at(40), **{**a, name: a[other]}) == L.MOE_EINVAL, (name, other)
    assert decode(D(), ws=at(40), **{**a, "topk": at(40)}) == L.MOE_EINVAL
    assert decode(D(), ws=at(40), **{**a, "gates": at(40) + need - 16}) == L.MOE_EINVAL
    assert decode(D(), ws=at(40), **{**a, "y": at(40) - 256}) == L.MOE_EINVAL


def test_decode_shared_expert_dims(lib):
    s = (at(10), at(11), at(12))
    good = D(F=384, E=1, K=1)
    need = L.moe_decode_workspace_bytes(D(), good)
    assert L.moe_decode_workspace_bytes(D()) < need < BAD
    assert decode(D(), good, s, nb=need - 1) == L.MOE_EWORKSPACE
    assert decode(D(), good, (at(10), None, at(12))) == L.MOE_EINVAL
    assert decode(D(), None, s) == L.MOE_EINVAL                 # weights without dims
    for ds in (D(E=2, K=1), D(E=1, K=1, H=256), D(E=1, K=1, N=7), D(E=1, K=1, dtype=L.MOE_F32)):
        assert L.moe_decode_workspace_bytes(D(), ds) == BAD
        assert decode(D(), ds, s, nb=1 << 30) == L.MOE_EINVAL


def norm(d, eps=1e-6, **kw):
    a = dict(x=at(1), residual=at(2), weight=at(3), h=at(4), y=at(5), rstd=at(6))
    a.update(kw)
    return L.lib().moe_rms_norm(ctypes.byref(d), a["x"], a["residual"], a["weight"], eps, a["h"], a["y"], a["rstd"], None)


def test_norm_refusals(lib):
    d = D()
    for name in ("x", "weight", "y"):
        assert norm(d, **{name: None}) == L.MOE_EINVAL, name
    for name in ("x", "weight", "y", "residual", "h", "rstd"):
        assert norm(d, **{name: at(20) + 8}) == L.MOE_EINVAL, name
    assert norm(d, residual=None) == L.MOE_EINVAL and norm(d, h=None) == L.MOE_EINVAL
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(d, eps=eps) == L.MOE_EINVAL, eps
    assert norm(D(H=L.MOE_NORM_MAX_H + 128)) == L.MOE_EUNSUPPORTED
    row = 128 * 2
    for kw in (dict(y=at(1)), dict(y=at(2)), dict(y=at(4)), dict(y=at(3)), dict(h=at(1) + row), dict(h=at(2) + row),
               dict(y=at(1) + 7 * row), dict(rstd=at(5)), dict(rstd=at(1)), dict(h=at(3))):
        assert norm(d, **kw) == L.MOE_EINVAL, kw
    assert norm(D(N=0), residual=None, h=None, rstd=None) == L.MOE_OK


def norm_bwd(d, ws=at(8), nb=None, **kw):
    a = dict(dy=at(1), h=at(2), weight=at(3), rstd=at(4), dh=at(5), dx=at(6), dw=at(7))
    a.update(kw)
    nb = L.moe_workspace_bytes(d, L.MOE_ENTRY_RMS_NORM_BWD) if nb is None else nb
    return L.lib().moe_rms_norm_bwd(ctypes.byref(d), a["dy"], a["h"], a["weight"], a["rstd"], a["dh"], a["dx"], a["dw"],
                                    ws, nb, None)


def test_norm_backward_refusals(lib):
    d = D()
    need = L.moe_workspace_bytes(d, L.MOE_ENTRY_RMS_NORM_BWD)
    assert 0 < need < BAD
    assert L.moe_workspace_bytes(D(H=L.MOE_NORM_MAX_H + 128), L.MOE_ENTRY_RMS_NORM_BWD) == BAD
    for name in ("dy", "h", "weight", "rstd", "dx", "dw"):
        assert norm_bwd(d, **{name: None}) == L.MOE_EINVAL, name
        assert norm_bwd(d, **{name: at(20) + 4}) == L.MOE_EINVAL, name
    assert norm_bwd(d, dh=at(20) + 4) == L.MOE_EINVAL
    for kw in (dict(dx=at(2)), dict(dx=at(1) + 256), dict(dx=at(5) + 256), dict(dx=at(3)), dict(dx=at(4))):
        assert norm_bwd(d, **kw) == L.MOE_EINVAL, kw
    assert norm_bwd(d, nb=need - 4) == L.MOE_EWORKSPACE
    assert norm_bwd(d, ws=None) == L.MOE_EWORKSPACE
    assert norm_bwd(D(H=L.MOE_NORM_MAX_H + 128), nb=1 << 40) == L.MOE_EUNSUPPORTED
    assert norm_bwd(D(N=0), ws=None, nb=0, dh=None) == L.MOE_OK


def test_norm_backward_refuses_a_dweight_on_other_arguments(lib):
    for other in (1, 2, 3, 4, 5, 6):
        assert norm_bwd(D(), dw=at(other)) == L.MOE_EINVAL, other
    assert norm_bwd(D(), dw=at(1) - 128 * 4 + 16) == L.MOE_EINVAL      # its end on dy


def test_decode_workspace_of_a_wide_shared_expert(lib):
    """Partial sums of the shared expert's down product: at most a piece per CU (256) over the
    strips of 256 columns, whatever the ratio of the experts' lengths."""
    N, H, F, Fs = 64, 8192, 128, 65536
    d, ds = D(N=N, H=H, F=F, E=8, K=2), D(N=N, H=H, F=Fs, E=1, K=1)
    acts = 2 * 4 * N * Fs * 4 + N * Fs * 4          # sums of gate and up in four pieces at most, activations
    parts = 256 // (H // 256) * N * H * 4
    assert L.moe_decode_workspace_bytes(d, ds) <= L.moe_decode_workspace_bytes(d) + acts + parts + 4096


def clip(rows, max_norm=1.0, norm=at(100), ws=at(101), nb=L.MOE_GRAD_WS_BYTES, count=None, entry="moe_grad_clip"):
    arr = (L.moe_grad * max(1, len(rows)))(*rows)
    count = len(rows) if count is None else count
    if entry == "moe_grad_norm":
        return L.lib().moe_grad_norm(arr, count, norm, ws, nb, None)
    return L.lib().moe_grad_clip(arr, count, max_norm, norm, ws, nb, None)


F32, BF16 = L.MOE_F32, L.MOE_BF16


@pytest.mark.parametrize("entry", ["moe_grad_norm", "moe_grad_clip"])
def test_grad_list_refusals(lib, entry):
    ok = (at(1), at(2), 100, F32, F32)
    assert clip([ok], entry=entry, count=-1) == L.MOE_EINVAL
    assert clip([ok], entry=entry, count=L.MOE_GRAD_MAX_TENSORS + 1) == L.MOE_EUNSUPPORTED
    assert clip([(None, at(2), 100, F32, F32)], entry=entry) == L.MOE_EINVAL
    assert clip([(at(1) + 2, at(2), 100, F32, F32)], entry=entry) == L.MOE_EINVAL
    assert clip([(at(1) + 1, at(2), 100, BF16, F32)], entry=entry) == L.MOE_EINVAL
    assert clip([(at(1), at(2), -1, F32, F32)], entry=entry) == L.MOE_EINVAL
    assert clip([(at(1), at(2), 100, 2, F32)], entry=entry) == L.MOE_EINVAL
    assert clip([(at(1), at(2), 1 << 45, F32, F32)], entry=entry) == L.MOE_EUNSUPPORTED
    assert clip([(FAKE, at(2), 1 << 43, F32, F32)] * 3, entry=entry) == L.MOE_EUNSUPPORTED
    assert clip([ok], entry=entry, norm=None) == L.MOE_EINVAL
    assert clip([ok], entry=entry, norm=at(100) + 2) == L.MOE_EINVAL
    assert clip([ok], entry=entry, ws=None) == L.MOE_EWORKSPACE
    assert clip([ok], entry=entry, ws=at(101) + 8) == L.MOE_EWORKSPACE
    assert clip([ok], entry=entry, nb=L.MOE_GRAD_WS_BYTES - 1) == L.MOE_EWORKSPACE
    fn = getattr(L.lib(), entry)
    args = (None, 1, at(100), at(101), 8192, None) if entry == "moe_grad_norm" else (None, 1, 1.0, at(100), at(101), 8192, None)
    assert fn(*args) == L.MOE_EINVAL                            # no list


def test_clip_refuses_overlapping_outputs(lib):
    for mn in (float("nan"), float("inf"), -1.0):
        assert clip([(at(1), at(2), 100, F32, F32)], max_norm=mn) == L.MOE_EINVAL
    for rows in (
        [(at(1), at(2), 100, F32, 3)],                                       # unknown output type
        [(at(1), None, 100, F32, F32)],
        [(at(1), at(2) + 2, 100, F32, F32)],
        [(at(1), at(1), 100, F32, F32)] * 2,                                 # the same tensor twice, in place
        [(at(1), at(2), 100, F32, F32), (at(3), at(2), 100, F32, F32)],      # the same output twice
        [(at(1), at(1), 100, F32, BF16)],                                    # in place, another type
        [(at(1), at(1) + 16, 100, F32, F32)],                                # output shifted into its input
        [(at(1), at(2), 100, F32, F32), (at(2) + 396, at(4), 10, F32, F32)],  # one output on another's input
        [(at(1), at(1), 100, F32, F32), (at(1) + 200, at(5), 4, F32, F32)],  # an input inside one in place
        [(at(1), at(100), 100, F32, F32)],                                   # output on norm
        [(at(101), at(2), 100, F32, F32)],                                   # input on the workspace
    ):
        assert clip(rows) == L.MOE_EINVAL, rows


def test_python_entries_check_their_arguments(lib):
    """Checks that run before any device is touched."""
    import mixture_experts_layer_sort_amd as M
    with pytest.raises(L.MoEError):
        M.MoEDecodeRunner(65, 128, 128, 4, 2, torch.bfloat16, "cpu")
    with pytest.raises(L.MoEError):
        M.MoEDecodeRunner(4, 100, 128, 4, 2, torch.bfloat16, "cpu")
    with pytest.raises(ValueError):
        M.MoEDecodeRunner(4, 128, 128, 4, 2, torch.float16, "cpu")
    with pytest.raises(L.MoEError):
        M.MoENormRunner(4, L.MOE_NORM_MAX_H + 128, torch.float32, "cpu")
    r = M.MoEDecodeRunner(4, 128, 256, 4, 2, torch.float32, "cpu")
    x, w_r = torch.zeros(3, 128), torch.zeros(128, 4)
    wg, wd = torch.zeros(4, 128, 256), torch.zeros(4, 256, 128)
    for bad in ((torch.zeros(5, 128), w_r, wg, wg, wd), (x.bfloat16(), w_r, wg, wg, wd), (x, w_r.t(), wg, wg, wd),
                (x, w_r, wg[:3], wg, wd), (x, w_r, wg, wg, wg), (x, w_r, wg, wg, wd, torch.zeros(3))):
        with pytest.raises(ValueError):
            r.forward(*bad)
    with pytest.raises(ValueError):
        r.forward(x, w_r, wg, wg, wd, shared=(wg[0], wg[0], wd[0]))
    with pytest.raises(ValueError):
        r.forward(x, w_r, wg, wg, wd)                          # host tensors
    n = M.MoENormRunner(4, 128, torch.float32, "cpu")
    with pytest.raises(RuntimeError):
        n.backward(x)
    with pytest.raises(ValueError):
        n.forward(torch.zeros(5, 128), torch.zeros(128))
    with pytest.raises(ValueError):
        n.forward(x, torch.zeros(128), residual=torch.zeros(2, 128))
    with pytest.raises(RuntimeError):
        M.MoENormRunner(4, 128, torch.float32, "cpu", backward=False).backward(x)
    for bad in (dict(grads=[x], max_norm=1.0, out=[x, x]), dict(grads=[x], max_norm=1.0),
                dict(grads=[x], max_norm=1.0, out=[torch.zeros(2)]), dict(grads=[x.double()], max_norm=1.0)):
        with pytest.raises(ValueError):
            M.moe_clip_grads(**bad)


def test_refused_calls_leave_the_runners_as_they_were(lib):
    """The host tensors are refused where their addresses are taken, behind the checks of shapes."""
    import mixture_experts_layer_sort_amd as M
    n = M.MoENormRunner(4, 128, torch.float32, "cpu")
    before = n.d, n.h, n.y, n.rstd, n.inputs
    for residual in (None, torch.zeros(3, 128)):
        with pytest.raises(ValueError):
            n.forward(torch.zeros(3, 128), torch.zeros(128), residual=residual)
        assert all(a is b for a, b in zip(before, (n.d, n.h, n.y, n.rstd, n.inputs)))
    r = M.MoEDecodeRunner(4, 128, 256, 4, 2, torch.float32, "cpu")
    before = r.topk, r.gates, r.y
    wg, wd = torch.zeros(4, 128, 256), torch.zeros(4, 256, 128)
    with pytest.raises(ValueError):
        r.forward(torch.zeros(3, 128), torch.zeros(128, 4), wg, wg, wd)
    assert all(a is b for a, b in zip(before, (r.topk, r.gates, r.y)))


def test_norm_backward_refuses_a_workspace_on_other_arguments(lib):
    d = D(N=40)                                                  # ten workgroups' partial sums
    need = L.moe_workspace_bytes(d, L.MOE_ENTRY_RMS_NORM_BWD)
    for other in (1, 2, 3, 4, 5, 6, 7):
        assert norm_bwd(d, ws=at(other)) == L.MOE_EINVAL, other
        assert norm_bwd(d, ws=at(other) - need + 16) == L.MOE_EINVAL, other      # its end on the argument
    assert norm_bwd(D(N=0), ws=at(7), nb=0) == L.MOE_OK          # no byte of it is used


def test_grad_norm_refuses_a_norm_or_workspace_on_its_tensors(lib):
    ok = (at(1), at(2), 100, F32, F32)
    for rows, kw in (
        ([ok, (at(101), None, 100, F32, F32)], {}),                      # a tensor inside the workspace
        ([(at(101) - 400 + 4, None, 100, F32, F32)], {}),                # its end
        ([(at(101) + L.MOE_GRAD_WS_BYTES - 2, None, 9, BF16, F32)], {}),  # its start
        ([ok, (at(100), None, 1, F32, F32)], {}),                        # a tensor on norm
        ([(at(100) - 8, None, 5, BF16, F32)], {}),
        ([ok], dict(norm=at(101) + 64)),                                 # norm inside the workspace
        ([], dict(norm=at(101))),
    ):
        assert clip(rows, entry="moe_grad_norm", **kw) == L.MOE_EINVAL, rows
    # an empty tensor may point anywhere
    assert clip([(at(101), None, 0, F32, F32)], entry="moe_grad_norm", nb=0) == L.MOE_EWORKSPACE


@pytest.mark.parametrize("entry", ["moe_grad_norm", "moe_grad_clip"])
def test_grad_lists_have_at_most_two_to_the_31_chunks(lib, entry):
    """Chunks of 4096 elements; the refusal of a missing norm comes behind the list's own."""
    one = 1 << 43
    for sizes, st in (([one], L.MOE_EINVAL), ([one + 1], L.MOE_EUNSUPPORTED), ([one // 2] * 2, L.MOE_EINVAL),
                      ([one // 2, one // 2 + 1], L.MOE_EUNSUPPORTED), ([one, 1], L.MOE_EUNSUPPORTED),
                      ([one - 4096, 0, 1], L.MOE_EINVAL), ([one - 4096, 1, 1], L.MOE_EUNSUPPORTED),
                      ([(1 << 63) - 1], L.MOE_EUNSUPPORTED)):
        assert clip([(at(1), at(2), n, BF16, BF16) for n in sizes], entry=entry, norm=None) == st, sizes


def test_decode_outputs_and_workspace_overlap_no_weights(lib):
    d, ds, s = D(), D(F=384, E=1, K=1), (at(10), at(11), at(12))
    need = L.moe_decode_workspace_bytes(d, ds)
    full, shared = 4 * 128 * 256 * 2, 128 * 384 * 2              # bytes of a weight tensor
    ends = {2: 128 * 4 * 2, 3: full, 4: full, 5: full, 10: shared, 11: shared, 12: shared, 13: 16}
    for i, n in ends.items():
        for where in (at(i), at(i) + n - 16):                    # its start, its last bytes
            for out in ("y", "topk", "gates", "ws"):
                assert decode(d, ds, s, bias=at(13), nb=need, **{out: where}) == L.MOE_EINVAL, (i, out)
        assert decode(d, ds, s, bias=at(13), ws=at(i) - need + 16) == L.MOE_EINVAL, i
    assert decode(D(N=0), D(N=0, F=384, E=1, K=1), s, y=at(3), bias=at(13), ws=at(4), nb=0) == L.MOE_OK


def test_clip_grads_needs_a_backward(lib):
    """The runner's gradient buffers hold nothing before."""
    import mixture_experts_layer_sort_amd as M
    with pytest.raises(RuntimeError, match="before backward"):
        M.MoELayerRunner(8, 128, 128, 4, 2, torch.float32, "cpu").clip_grads(1.0)
    with pytest.raises(RuntimeError, match="without backward buffers"):
        M.MoELayerRunner(8, 128, 128, 4, 2, torch.float32, "cpu", backward=False).clip_grads(1.0)

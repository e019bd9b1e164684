"""Global gradient norm and clipping against a plain float64 evaluation.

Tolerances, u = 2^-24: squares and their sums are float64, so norm is off by
its rounding to float32, u (1 + 2^-20).  The factor is rounded to float32 once
(u), the product to the output's type once (s = 2^-8 or 2^-24): an output is off
by at most (s + u) (1 + 2^-7) relative to the exact one, where that is a normal
number."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _grads(sizes, dtypes, scale=1e-3, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def _norm64(grads):
    return math.sqrt(math.fsum(g.double().square().sum().item() for g in grads))


def check(grads, outs, norm, max_norm):
    ref = _norm64(grads)
    assert abs(norm.item() - ref) <= U * (1 + 2.0 ** -20) * ref
    coef = min(1.0, max_norm / (ref + 1e-6))
    for g, o in zip(grads, outs):
        want = g.double() * coef
        s = 2.0 ** -8 if o.dtype == BF16 else U
        assert ((o.double() - want).abs() <= (s + U) * (1 + 2.0 ** -7) * want.abs()).all()


LISTS = {
    "one": [1],
    "tiny": [1, 2, 3, 5, 7, 8, 9, 0, 15, 16, 17],
    "chunk_edges": [8191, 8192, 8193, 2047, 2048, 2049, 16384],
    "layer": [128, 128 * 8, 8 * 128 * 256, 8 * 128 * 256, 8 * 256 * 128],
    "empty_ends": [0, 0, 100, 0],
    "many": [(i * 37) % 301 for i in range(200)],
    "table_edge": [50] * 64,
    "large": [30_000_001, 77],
}


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)],
                         ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("name", LISTS)
def test_clip_matches_float64(name, types):
    from mixture_experts_layer_sort_amd import moe_clip_grads, moe_grad_norm
    grads = _grads(LISTS[name], [types[0]], scale=1.0, seed=1)
    outs = [torch.full_like(g, 9.0, dtype=types[1]) for g in grads]
    keep = [g.clone() for g in grads]
    for max_norm in (0.25, 1e9):
        got, norm = moe_clip_grads(grads, max_norm, out=outs)
        check(grads, got, norm, max_norm)
        assert norm.item() == moe_grad_norm(grads).item()
    for g, k in zip(grads, keep):
        assert torch.equal(g, k)
    if types[0] == types[1]:
        want = [o.clone() for o in moe_clip_grads(grads, 0.25, out=outs)[0]]
        moe_clip_grads(grads, 0.25)                 # in place
        for g, o in zip(grads, want):
            assert torch.equal(g, o)


def test_mixed_types_and_alignments():
    """Views at odd elements, both types in one list; neighbours keep their values."""
    from mixture_experts_layer_sort_amd import moe_clip_grads
    flat, fb = _grads([100_000, 100_000], [F32, BF16], scale=1.0, seed=2)
    of, ob = torch.full((100_000,), 3.0, device="cuda"), torch.full((100_000,), 3.0, device="cuda", dtype=BF16)
    cuts = [(1, 5000), (5001, 5002), (5003, 30_011), (40_004, 99_999)]
    grads = [flat[a:b] for a, b in cuts] + [fb[a:b] for a, b in cuts]
    outs = [ob[a:b] for a, b in cuts] + [of[a + 1:b + 1] for a, b in cuts]
    got, norm = moe_clip_grads(grads, 0.1, out=outs)
    check(grads, got, norm, 0.1)
    for o, shift in ((ob, 0), (of, 1)):
        hit = torch.zeros(100_000, dtype=torch.bool, device="cuda")
        for a, b in cuts:
            hit[a + shift:b + shift] = True
        assert (o[~hit] == 3).all()


def test_range_of_values():
    """Squares that overflow or vanish in float32 count; zeros, one huge value."""
    from mixture_experts_layer_sort_amd import moe_clip_grads, moe_grad_norm
    for scale in (1e-30, 1e30, 3e38):
        grads = [torch.full((1000,), scale, device="cuda"), torch.zeros(77, device="cuda")]
        ref = _norm64(grads)
        got = moe_grad_norm(grads).item()
        assert got == math.inf if ref > 3.4028235677973366e38 else abs(got - ref) <= U * 1.001 * ref
    grads = [torch.full((1000,), 1e30, device="cuda")]
    outs, _ = moe_clip_grads(grads, 1.0)
    assert (outs[0].double() - 1000 ** -0.5).abs().max() <= 3 * U * 1000 ** -0.5
    z = [torch.zeros(100, device="cuda")]
    outs, norm = moe_clip_grads(z, 1.0)
    assert norm.item() == 0 and (outs[0] == 0).all()
    outs, norm = moe_clip_grads([torch.ones(100, device="cuda")], 0.0)
    assert norm.item() == 10 and (outs[0] == 0).all()
    assert moe_clip_grads([], 1.0)[1].item() == 0 and moe_grad_norm([]).item() == 0


def test_non_finite_gradients():
    from mixture_experts_layer_sort_amd import moe_clip_grads
    a, b = torch.ones(5000, device="cuda"), torch.ones(300, device="cuda", dtype=BF16)
    a[4999] = float("inf")
    (oa, ob), norm = moe_clip_grads([a, b], 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
    assert norm.item() == math.inf and (oa[:4999] == 0).all() and torch.isnan(oa[4999]) and (ob == 0).all()
    a[4999] = float("nan")
    (oa, ob), norm = moe_clip_grads([a, b], 1.0, out=[oa, ob])
    assert math.isnan(norm.item()) and torch.isnan(oa).all() and torch.isnan(ob).all()


def test_repeated_and_overlapping_tensors():
    from mixture_experts_layer_sort_amd import MoEError, moe_clip_grads, moe_grad_norm
    g = _grads([4000], [F32])[0]
    assert abs(moe_grad_norm([g, g]).item() - _norm64([g, g])) <= U * 1.001 * _norm64([g, g])
    keep = g.clone()
    for bad in (dict(grads=[g, g]), dict(grads=[g, g[10:20]]), dict(grads=[g[:100]], out=[g[4:104]]),
                dict(grads=[g[:10], g[10:20]], out=[g[20:30], g[25:35]])):
        with pytest.raises(MoEError):
            moe_clip_grads(max_norm=1.0, **bad)
    with pytest.raises(ValueError):
        moe_clip_grads([g.view(40, 100).t()], 1.0)
    assert torch.equal(g, keep)
    # both inputs the same, outputs apart: allowed
    outs, norm = moe_clip_grads([g, g], 0.01, out=[torch.empty_like(g), torch.empty_like(g)])
    check([g, g], outs, norm, 0.01)


def test_same_bits_again_in_a_graph_and_on_another_stream():
    from mixture_experts_layer_sort_amd import _lib as L, moe_clip_grads
    grads = _grads([1_000_003, 5, 70_000, 0, 1] + [333] * 90, [F32, BF16], scale=1.0, seed=4)
    outs = [torch.empty(g.shape, dtype=BF16, device="cuda") for g in grads]
    want = [o.clone() for o in moe_clip_grads(grads, 2.0, out=outs)[0]]
    norm0 = moe_clip_grads(grads, 2.0, out=outs)[1].clone()
    check(grads, want, norm0, 2.0)
    ws, norm = torch.empty(L.MOE_GRAD_WS_BYTES, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.moe_grad_clip(grads, outs, 2.0, norm, ws, side)
    side.synchronize()
    assert torch.equal(norm, norm0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.moe_grad_clip(grads, outs, 2.0, norm, ws)     # the list is gone after the call: the graph holds its own
    for i in range(4):
        for o in outs:
            o.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, norm0)
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
        torch.randn(1000, device="cuda").sum().item()
    grads[0].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    check(grads, outs, norm, 2.0)


def test_runner_clips_its_own_gradients():
    from mixture_experts_layer_sort_amd import MoELayerRunner
    from moe_workloads import TEST_CONFIGS, make_inputs, make_shared_weights
    c = TEST_CONFIGS["t_ragged"]
    t = make_inputs(c, 0, device="cuda")
    r = MoELayerRunner(c.N, c.H, c.F, c.E, c.K, c.torch_dtype, shared_ffn=256)
    r.forward(t["x"], t["w_r"], t["w_gate"], t["w_up"], t["w_down"],
              shared=make_shared_weights(c, 0, 256, "cuda"))
    g = r.backward(t["dy"])
    names = [k for k in g if k.startswith("dw")]
    assert len(names) == 7
    before = [g[k].clone() for k in names]
    extra = torch.randn(256, device="cuda")
    e0 = extra.clone()
    norm = r.clip_grads(1.0, extra=[extra])
    check(before + [e0], [g[k] for k in names] + [extra], norm, 1.0)

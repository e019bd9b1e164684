"""Residual addition and RMS norm, forward and backward, against a plain
float64 evaluation, and the step norm -> layer -> backward -> clipping.

Tolerances.  u = 2^-24, s = 2^-8 (bf16) or 2^-24 (float32).  h is one float32
addition and one rounding of it: equal bits.  A row's sum of squares has at most
32 terms a thread, 6 steps in a wave and 16 waves, each off by u of a positive
sum; the mean, the root and the quotient add 4 u: rstd is good to (54 / 2 + 5) u
= 32 u, y to 35 u before its rounding (two products).  The backward's row sum is
off by (54 + 6) u mean|t xhat|, so, with B = rstd (|t| + |xhat| mean|t xhat|) +
|dh|, dx is good to s |dx| + 80 u B.  dweight adds ceil(N / 512) rows in float32
(4 at once in a workgroup of 4 waves, and 4 sums), the rest in float64: good to
(ceil(N / 512) + 12) u sum|dy xhat|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _make(N, H, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return r(N, H), (2 * r(N, H)).to(dtype), (1 + 0.1 * r(H)).to(dtype), r(N, H), r(N, H)


def _s(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def check_forward(h, w, y, rstd, eps=EPS):
    hd, wd = h.double(), w.double()
    ref_r = (hd.square().mean(1) + eps).rsqrt()
    ref = hd * ref_r[:, None] * wd
    assert ((rstd.double() - ref_r).abs() <= 32 * U * ref_r).all()
    assert ((y.double() - ref).abs() <= (_s(h.dtype) + 36 * U) * ref.abs()).all()


def check_backward(h, w, dy, dh, dx, dw, eps=EPS):
    N, H = h.shape
    hd, wd, g = h.double(), w.double(), dy.double()
    r = (hd.square().mean(1, keepdim=True) + eps).rsqrt()
    xh, t = hd * r, g * wd
    ref = r * (t - xh * (t * xh).mean(1, keepdim=True))
    B = r * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        ref, B = ref + dh.double(), B + dh.double().abs()
    assert ((dx.double() - ref).abs() <= _s(h.dtype) * ref.abs() + 80 * U * B).all()
    tol = (-(-N // 512) + 12) * U * (g * xh).abs().sum(0)
    # rstd itself is off by up to 32 u, alike in all of a row's terms
    assert ((dw.double() - (g * xh).sum(0)).abs() <= tol + 34 * U * (g * xh).abs().sum(0)).all()


SHAPES = [(1, 128), (1, 7168), (2, 512), (3, 640), (5, 1024), (4, 1152), (7, 2048), (9, 2176), (513, 256), (1030, 2048), (8200, 2048),
          (600, 4096), (5, 8192), (3, 12288), (2, 16384), (2, 16512), (3, 32768)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES)
def test_norm_matches_float64(N, H, dtype):
    from mixture_experts_layer_sort_amd import MoENormRunner
    x, res, w, dy, dh = _make(N, H, dtype, seed=N + H)
    r = MoENormRunner(N, H, dtype, "cuda", eps=EPS)
    y = r.forward(x, w, residual=res)
    assert torch.equal(r.h, (x.float() + res.float()).to(dtype))
    check_forward(r.h, w, y, r.rstd)
    dx, dw = r.backward(dy, dh=dh)
    check_backward(r.h, w, dy, dh, dx, dw)
    first = [t.clone() for t in (y, r.h, r.rstd, dx, dw)]
    r.ws.fill_(255)
    r.forward(x, w, residual=res)
    dx, dw = r.backward(dy, dh=dh)
    for a, b in zip(first, (r.y, r.h, r.rstd, dx, dw)):
        assert torch.equal(a, b)
    # without a residual, and without a gradient of the residual stream
    y = r.forward(x, w)
    assert r.h is x
    check_forward(x, w, y, r.rstd)
    dx, dw = r.backward(dy)
    check_backward(x, w, dy, None, dx, dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 15, 16, 17, 1003, 20011])
@pytest.mark.parametrize("H", [128, 256, 384])
def test_short_rows_share_a_wave(N, H, dtype):
    """dweight joins up to 16 rows' sums in a workgroup here instead of 4, but a row's sum of
    squares has at most 8 terms a thread and 5 steps, so rstd is good to (13 / 2 + 5) u: 15 joins
    and 12 u stay within the 12 + 34 u that the check allows besides ceil(N / 512)."""
    test_norm_matches_float64(N, H, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_in_place_and_partial_rows(dtype):
    from mixture_experts_layer_sort_amd import MoENormRunner, _lib as L
    x, res, w, dy, dh = _make(11, 4096, dtype, seed=1)
    r = MoENormRunner(16, 4096, dtype, "cuda", eps=EPS)
    r._y.fill_(5)
    r._h.fill_(5)
    y = r.forward(x, w, residual=res)
    assert y.shape == x.shape and (r._y[11:] == 5).all() and (r._h[11:] == 5).all()
    want = [t.clone() for t in (r.h, y, r.rstd)]
    dx, dw = (t.clone() for t in r.backward(dy, dh=dh))
    for where in ("x", "residual"):
        a, b = x.clone(), res.clone()
        h = a if where == "x" else b
        L.moe_rms_norm(r.d, a, b, w, EPS, h, y, r.rstd)
        for p, q in zip(want, (h, y, r.rstd)):
            assert torch.equal(p, q)
    for where in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        o = a if where == "dy" else b
        L.moe_rms_norm_bwd(r.d, a, want[0], w, r.rstd, b, o, r.dweight, r.ws)
        assert torch.equal(o, dx) and torch.equal(r.dweight, dw)
    assert r.forward(x[:0], w).shape == (0, 4096)
    dx, dw = r.backward(dy[:0])
    assert dx.shape == (0, 4096) and (dw == 0).all()


def test_special_values():
    """Zero rows give zeros, a NaN or an infinity stays in its row."""
    from mixture_experts_layer_sort_amd import MoENormRunner
    x, _, w, dy, _ = _make(6, 1024, torch.bfloat16, seed=2)
    r = MoENormRunner(6, 1024, torch.bfloat16, "cuda", eps=EPS)
    x[1] = 0
    good = r.forward(x, w).clone()
    assert (good[1] == 0).all() and r.rstd[1].item() == pytest.approx(1e3, rel=1e-6)
    gdx, _ = r.backward(dy)
    gdx = gdx.clone()
    x[3, 7], x[4, 9] = float("nan"), float("inf")
    y = r.forward(x, w)
    dx, _ = r.backward(dy)
    assert torch.isnan(y[3]).all() and r.rstd[4] == 0 and torch.isnan(y[4, 9]) and (y[4, :9] == 0).all()
    for n in (0, 1, 2, 5):
        assert torch.equal(y[n], good[n]) and torch.equal(dx[n], gdx[n])


def test_more_rows_than_one_launch_has_workgroups():
    """Rows behind 2^20 workgroups of 4 rows, element offsets behind 2^31 bytes."""
    from mixture_experts_layer_sort_amd import MoENormRunner
    N, H = (1 << 22) + 3 * 4 + 1, 512
    r = MoENormRunner(N, H, torch.bfloat16, "cuda", eps=EPS, backward=False)
    x = torch.zeros((N, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, N - 1], device="cuda")
    part = torch.randn((5, H), device="cuda").bfloat16()
    x[rows] = part
    y = r.forward(x, w)
    check_forward(part, w, y[rows], r.rstd[rows])
    assert (y[2:(1 << 22) - 1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_autograd_function(dtype):
    from mixture_experts_layer_sort_amd import moe_rms_norm
    x, res, w, dy, dh = (t.detach() for t in _make(12, 640, dtype, seed=3))
    leaves = [t.clone().view(3, 4, 640).requires_grad_() for t in (x, res)] + [w.clone().requires_grad_()]
    y, h = moe_rms_norm(leaves[0], leaves[2], residual=leaves[1], eps=EPS)
    assert y.shape == (3, 4, 640) == h.shape
    torch.autograd.backward([y, h], [dy.view(3, 4, 640), dh.view(3, 4, 640)])
    assert leaves[0].grad.dtype == dtype and torch.equal(leaves[0].grad, leaves[1].grad)
    check_backward(h.detach().view(12, 640), w, dy, dh, leaves[0].grad.view(12, 640),
                   torch.autograd.grad(moe_rms_norm(x, wd := w.clone().requires_grad_(), res)[0], wd, dy)[0]
                   if dtype == torch.float32 else _dw(h.detach().view(12, 640), dy))
    # only h used: its gradient passes through; only y used; no residual; a strided input
    a, b = x.clone().requires_grad_(), res.clone().requires_grad_()
    moe_rms_norm(a, w, residual=b)[1].backward(dh)
    assert torch.equal(a.grad, dh) and torch.equal(b.grad, dh)
    a = x.clone().requires_grad_()
    moe_rms_norm(a, w).backward(dy)
    ref = a.grad.clone()
    wide = torch.zeros((12, 1280), dtype=dtype, device="cuda")
    wide[:, :640] = x
    a = wide[:, :640].detach().requires_grad_()
    assert not a.is_contiguous()
    moe_rms_norm(a, w).backward(dy)
    assert torch.equal(a.grad, ref)
    # a broadcast upstream gradient (stride 0)
    a = x.clone().requires_grad_()
    moe_rms_norm(a, w).sum().backward()
    assert torch.isfinite(a.grad).all()
    # no rows
    a, ww = x[:0].clone().requires_grad_(), w.clone().requires_grad_()
    moe_rms_norm(a, ww).sum().backward()
    assert (ww.grad == 0).all() and a.grad.shape == (0, 640)


def _dw(h, dy):
    hd = h.double()
    return (dy.double() * hd * (hd.square().mean(1, keepdim=True) + EPS).rsqrt()).sum(0)


def test_autograd_function_captured_with_its_backward():
    from mixture_experts_layer_sort_amd import moe_rms_norm
    x, res, w, dy, dh = _make(40, 512, torch.bfloat16, seed=11)
    leaves = [t.clone().requires_grad_() for t in (x, res, w)]

    def step():
        y, h = moe_rms_norm(leaves[0], leaves[2], residual=leaves[1], eps=EPS)
        return (y.detach(), *torch.autograd.grad([y, h], leaves, [dy, dh]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(4):
        with torch.no_grad():
            leaves[0].copy_(x * (i + 1))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """Central differences in float64 of the plain formula at the kernel's own h,
    along random directions: f(h + d) - f(h - d) over 2 d, truncation of order d^2."""
    from mixture_experts_layer_sort_amd import moe_rms_norm
    x, _, w, dy, _ = _make(4, 256, torch.float32, seed=4)
    a, ww = x.clone().requires_grad_(), w.clone().requires_grad_()
    moe_rms_norm(a, ww, eps=EPS).backward(dy)

    def f(xd, wd):
        return ((xd * (xd.square().mean(1, keepdim=True) + EPS).rsqrt() * wd) * dy.double()).sum()

    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-4
        num = (f(x.double() + eps * vx, w.double() + eps * vw) - f(x.double() - eps * vx, w.double() - eps * vw)) / (2 * eps)
        ana = (a.grad.double() * vx).sum() + (ww.grad.double() * vw).sum()
        # truncation: eps^2 times third derivatives of order |dy||w||v|^3/|h|^2 ~ 1e3; float32 gradients: 80 u each
        scale = (a.grad.double() * vx).abs().sum() + (ww.grad.double() * vw).abs().sum()
        assert abs(num - ana) <= 100 * U * scale + 1e-8 * 1e3


def test_norm_in_a_graph_and_on_another_stream():
    from mixture_experts_layer_sort_amd import MoENormRunner
    x, res, w, dy, dh = _make(300, 1024, torch.bfloat16, seed=5)
    r = MoENormRunner(300, 1024, torch.bfloat16, "cuda", eps=EPS)
    want = [t.clone() for t in (r.forward(x, w, residual=res), r.h, *r.backward(dy, dh=dh))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.forward(x, w, residual=res, stream=side)
    got = r.backward(dy, dh=dh, stream=side)
    side.synchronize()
    for a, b in zip(want, (r.y, r.h, *got)):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.forward(x, w, residual=res)
        r.backward(dy, dh=dh)
    for i in range(4):
        for t in (r._y, r._h, r._dx, r.dweight):
            t.zero_()
        r.ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (r.y, r.h, *got)):
            assert torch.equal(a, b)
        torch.randn(1000, device="cuda").sum().item()


def test_training_step_norm_layer_backward_clip():
    """norm -> layer -> backward -> norm's backward -> clipping in float32, against
    the same step in float64.  Every sum here has at most 256 terms of order one and
    there are fewer than 20 steps: 20 * 256 u < 4e-4 relative to each tensor's
    largest value is the worst case that sums in any order allow."""
    from mixture_experts_layer_sort_amd import MoELayerRunner, MoENormRunner
    N, H, F, E, K = 96, 256, 256, 6, 2
    x, res, w, dy, _ = _make(N, H, torch.float32, seed=6)
    g = torch.Generator(device="cuda")
    g.manual_seed(60)
    ws = [torch.randn(s, generator=g, device="cuda") * c for s, c in
          (((H, E), 0.02), ((E, H, F), H ** -0.5), ((E, H, F), H ** -0.5), ((E, F, H), F ** -0.5))]
    norm, layer = MoENormRunner(N, H, torch.float32, "cuda", eps=EPS), MoELayerRunner(N, H, F, E, K, torch.float32)
    xn = norm.forward(x, w, residual=res)
    y = layer.forward(xn, *ws)
    out = norm.h + y                                          # the block's output
    grads = layer.backward(dy)
    dx, dw = norm.backward(grads["dx"], dh=dy)                # dy also flows along the residual stream
    raw = [t.clone() for t in (layer.dw_r, layer.dw_gate, layer.dw_up, layer.dw_down, dw)]
    total = layer.clip_grads(0.5, extra=[dw])
    torch.cuda.synchronize()

    leaves = [t.double().requires_grad_() for t in (x, res, w, *ws)]
    xd, rd, wd, wr, wg, wu, wdn = leaves
    h = xd + rd
    n = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * wd
    ids = layer.topk.long()
    gates = torch.softmax(torch.gather(n @ wr, 1, ids), 1)
    yd = torch.zeros_like(h)
    for e in range(E):
        tok, k = torch.nonzero(ids == e, as_tuple=True)
        a = n[tok]
        o = (torch.nn.functional.silu(a @ wg[e]) * (a @ wu[e])) @ wdn[e]
        yd = yd.index_add(0, tok, gates[tok, k][:, None] * o)
    ref_out = h + yd
    ref_out.backward(dy.double())
    close = lambda a, b: (a.double() - b).abs().max() <= 4e-4 * b.abs().max()  # noqa: E731
    assert close(out, ref_out.detach()) and close(dx, xd.grad) and torch.equal(xd.grad, rd.grad)
    refs = [wr.grad, wg.grad, wu.grad, wdn.grad, wd.grad]
    ref_total = torch.stack([t.square().sum() for t in refs]).sum().sqrt()
    assert abs(total.double() - ref_total) <= 4e-4 * ref_total and ref_total > 0.5
    for got, before, ref in zip((layer.dw_r, layer.dw_gate, layer.dw_up, layer.dw_down, dw), raw, refs):
        assert close(before, ref)
        assert close(got, ref * (0.5 / (ref_total + 1e-6)))


def test_serving_step_norm_decode():
    """norm -> layer for few tokens -> the next block's norm, captured once and replayed on new tokens."""
    from mixture_experts_layer_sort_amd import MoEDecodeRunner, MoENormRunner
    N, H, F, E, K = 5, 512, 256, 16, 4
    x, res, w, _, _ = _make(N, H, torch.bfloat16, seed=7)
    g = torch.Generator(device="cuda")
    g.manual_seed(70)
    ws = [(torch.randn(s, generator=g, device="cuda") * c).bfloat16() for s, c in
          (((H, E), 0.02), ((E, H, F), H ** -0.5), ((E, H, F), H ** -0.5), ((E, F, H), F ** -0.5))]
    n1, n2 = (MoENormRunner(N, H, torch.bfloat16, "cuda", eps=EPS, backward=False) for _ in range(2))
    dec = MoEDecodeRunner(N, H, F, E, K, torch.bfloat16)

    def step():
        y = dec.forward(n1.forward(x, w, residual=res), *ws)
        return n2.forward(y, w, residual=n1.h)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(_make(N, H, torch.bfloat16, seed=80 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (n1.y, dec.y, n2.h, n2.y)]
        step()
        for a, b in zip(got, (n1.y, dec.y, n2.h, n2.y)):
            assert torch.equal(a, b)
        check_forward(n2.h, w, n2.y, n2.rstd)
        assert torch.equal(n2.h, (dec.y.float() + n1.h.float()).bfloat16())


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_no_rows_clear_dweight_on_the_given_stream(raw):
    """A step without rows behind a step with rows, both on a stream that is still busy: its
    gradient is zero there, also when the handle is passed."""
    from mixture_experts_layer_sort_amd import MoENormRunner
    x, _, w, dy, _ = _make(64, 512, torch.float32, seed=12)
    r = MoENormRunner(64, 512, torch.float32, "cuda", eps=EPS)
    r.forward(x, w)
    want = r.backward(dy)[1].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = side.cuda_stream if raw else side
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)               # some milliseconds of a waiting kernel
    r.forward(x, w, stream=s)
    r.backward(dy, stream=s)
    with torch.cuda.stream(side):
        first = r.dweight.clone()
    r.forward(x[:0], w, stream=s)
    dx, dw = r.backward(dy[:0], stream=s)
    side.synchronize()
    assert dx.shape == (0, 512) and torch.equal(first, want) and (dw == 0).all()
    if not raw:
        return
    r.backward(dy[:0], stream=0)                    # the null stream's handle
    torch.cuda.synchronize()
    assert (r.dweight == 0).all()


def test_backward_behind_a_refused_forward_is_the_last_ones():
    from mixture_experts_layer_sort_amd import MoEError, MoENormRunner
    x, res, w, dy, dh = _make(8, 256, torch.bfloat16, seed=13)
    r = MoENormRunner(8, 256, torch.bfloat16, "cuda", eps=EPS)
    r.forward(x, w, residual=res)
    want = [t.clone() for t in r.backward(dy, dh=dh)]
    odd = torch.zeros(8 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 256)
    for bad in (odd, odd[:5], r.y):                 # misaligned; on the output
        with pytest.raises(MoEError):
            r.forward(bad, w)
    assert r.y.shape == (8, 256)
    for a, b in zip(want, r.backward(dy, dh=dh)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_autograd_function_takes_views_at_any_element(dtype):
    """Inputs and gradients that start at odd elements give the same bits as aligned ones."""
    from mixture_experts_layer_sort_amd import moe_rms_norm
    x, res, w, dy, dh = _make(6, 256, dtype, seed=14)

    def run(move, through):
        leaves = [t.clone().requires_grad_() for t in (x, res, w)]
        y, h = moe_rms_norm(*(move(t) for t in (leaves[0], leaves[2], leaves[1])), eps=EPS)
        return (y.detach(), h.detach(), *torch.autograd.grad([through(y), through(h)], leaves, [move(dy), move(dh)]))

    def odd(t):                                     # the same values, one element behind the start
        return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)

    want = run(lambda t: t, lambda t: t)
    assert odd(x).is_contiguous() and odd(x).data_ptr() % 16
    for a, b in zip(want, run(odd, lambda t: t)):
        assert torch.equal(a, b)
    # the gradient of the cat's second part starts behind its first
    for a, b in zip(want, run(lambda t: t, lambda t: torch.cat([t.new_zeros(3), t.flatten()])[3:].view(t.shape))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 12, 1600])
@pytest.mark.parametrize("used", ["y", "y and h"])
def test_autograd_function_weight_gradient(dtype, N, used):
    """The weight's gradient in the weight's type against float64: dweight's own bound, as
    check_backward has it, and one rounding to the type."""
    from mixture_experts_layer_sort_amd import moe_rms_norm
    x, res, w, dy, dh = _make(N, 640, dtype, seed=15 + N)
    leaves = [t.clone().requires_grad_() for t in (x, res, w)]
    y, h = moe_rms_norm(leaves[0], leaves[2], residual=leaves[1], eps=EPS)
    torch.autograd.backward([y] if used == "y" else [y, h], [dy] if used == "y" else [dy, dh])
    hd, g = h.detach().double(), dy.double()
    terms = g * hd * (hd.square().mean(1, keepdim=True) + EPS).rsqrt()
    ref, own = terms.sum(0), (-(-N // 512) + 12 + 34) * U * terms.abs().sum(0)
    got = leaves[2].grad
    assert got.dtype == dtype and got.shape == (640,)
    assert ((got.double() - ref).abs() <= own + _s(dtype) * (ref.abs() + own)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [128, 7168, 32768])
def test_rows_around_the_largest_sum_of_squares(H, dtype):
    """Up to a 2-norm of 2^64 (1.84e19) rows are as good as any; behind it rstd and y are 0."""
    from mixture_experts_layer_sort_amd import MoENormRunner
    w = (1 + 0.1 * torch.randn(H, device="cuda")).to(dtype)
    sign = 1 - 2 * (torch.arange(H, device="cuda") % 2)
    x = torch.stack([(2.0 ** 64 * c / H ** 0.5 * sign).to(dtype) for c in (0.98, 1.02, 1e-9)])
    x = torch.cat([x, torch.zeros((1, H), dtype=dtype, device="cuda")])
    x[3, H - 3] = 0.98 * 2.0 ** 64                  # all of it in one value
    r = MoENormRunner(4, H, dtype, "cuda", eps=EPS, backward=False)
    y = r.forward(x, w)
    keep = [0, 2, 3]
    check_forward(x[keep], w, y[keep], r.rstd[keep])
    assert r.rstd[1] == 0 and (y[1] == 0).all()

"""Balance and z loss of router logits (moe_balance_loss) against plain float64.

Tolerances.  u = 2^-24.  expf, logf and the quotients are good to a few u; a float32 sum of m
positive terms is off by at most m u of it.  With R = max|l| + 10 over finite l:
  a softmax probability is exp(l - max) / sum: the difference rounded once (R u), so (R + E + 16) u
  of it; a normalised sigmoid alike;
  P_s,e adds up a chunk's tokens in float32, sixteen sums of chunk / 16 of them, then these: with
  chunk <= max(64, N / 768 + 16) at most (N / 512 + 64) u more;
  lse: R u + (E + 8) u absolutely, at most (R + E + 8) u, and its square 2 |lse| times that.
The loss adds alpha times the first and z times the second, and is rounded once.  A gradient
    c p_e (f_e - f.p) [1 - sigmoid] + zc lse softmax_e
is off by c p_e (max f (E + 4) u + (|f_e| + |f.p|) (R + E + 24) u) + zc softmax_e (|lse| + 1) (R + E + 24) u, then
rounded to its type.  Counts are whole numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def logits_of(N, E, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    l = torch.randn((N, E), generator=g, device="cuda") * scale + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    return l.to(dtype)


def order(l, bias, K):
    """K experts by (value desc, id asc), NaN last, float32 values."""
    v = l.float() if bias is None else l.float() + bias
    key = torch.where(torch.isnan(v), torch.full_like(v, -float("inf")), v)
    rank = torch.sort(torch.isnan(v).int() * 2, dim=1, stable=True)  # NaN behind -inf
    ids = rank[1]
    key = torch.gather(key, 1, ids)
    i = torch.sort(key, dim=1, descending=True, stable=True)[1]
    return torch.gather(ids, 1, i)[:, :K]


def reference(l, topk, mask, T, alpha, z, score):
    """loss, its bound, counts, gradient and its bound before the rounding, float64."""
    N, E = l.shape
    K = topk.shape[1]
    keep = torch.ones(N, dtype=torch.bool, device=l.device) if mask is None else mask.reshape(N).bool()
    x = torch.where(keep[:, None], l.double(), torch.zeros_like(l, dtype=torch.float64))
    ok = (topk >= 0) & (topk < E) & keep[:, None]
    hits = torch.zeros((N, E), dtype=torch.float64, device=l.device)
    hits.scatter_add_(1, torch.where(ok, topk, torch.zeros_like(topk)).long(), ok.double())
    soft, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    sig = torch.sigmoid(x)
    if score == "softmax":
        p, rest = soft, torch.ones_like(soft)
    else:
        p, rest = torch.exp(torch.nn.functional.logsigmoid(x)), 1 - sig
        p = p / p.sum(1, keepdim=True)
    kd = keep.double()[:, None]
    n = kd.reshape(-1, T).sum(1)
    seqs, total = int((n > 0).sum()), float(n.sum())
    nz = n.clamp(min=1)[:, None]
    f = (hits.reshape(-1, T, E).sum(1)) * E / (K * nz)
    P = (p * kd).reshape(-1, T, E).sum(1) / nz
    R = float(x[torch.isfinite(x)].abs().max()) + 10 if x.numel() else 10.0  # exp(-inf) is exactly 0
    rel = (R + E + 24) * U
    balance = float((f * P).sum()) * alpha / max(1, seqs)
    zed = float((lse ** 2 * kd[:, 0]).sum()) * z / max(1.0, total)
    bound = abs(balance) * (rel + (N / 512 + 64) * U) + abs(z) / max(1.0, total) * float(
        (2 * lse.abs() * rel * (1 + lse.abs()) + lse ** 2 * (N / 512 + 64) * U).sum())
    fr = f.repeat_interleave(T, 0)
    c = (alpha / max(1, seqs) / nz[:, 0]).repeat_interleave(T)[:, None]
    fp = (fr * p).sum(1, keepdim=True)
    zc = 2 * z / max(1.0, total)
    d = (c * p * (fr - fp) * rest + zc * lse[:, None] * soft) * kd
    ed = abs(c) * p * rest * (fr.amax(1, keepdim=True) * (E + 4) * U + (fr + fp) * rel) + abs(zc) * soft * (
        lse.abs()[:, None] + 1) * rel
    return balance + zed, bound + U * abs(balance + zed), hits.sum(0).long(), d, ed * kd


def check(l, K, T, alpha, z, score, topk=None, mask=None, bias=None, loss=None, counts=None, d=None):
    ids = topk if topk is not None else order(l, bias, K)
    want, tol, hits, dw, ed = reference(l, ids, mask, T, alpha, z, score)
    assert torch.equal(counts.long(), hits)
    assert abs(float(loss) - want) <= 1.01 * tol, (float(loss), want, tol)
    s = 2.0 ** -8 if l.dtype == torch.bfloat16 else U
    err, lim = (d.double() - dw).abs(), s * dw.abs() + 1.01 * ed + 1e-40
    assert bool((err <= lim).all()), float((err / lim).max())


CASES = [(1, 1, 1, 1), (1, 203, 8, 2), (3, 67, 12, 3), (1, 1, 256, 8), (5, 64, 7, 7), (1, 5000, 64, 6), (4, 513, 60, 4),
         (2, 300, 33, 5), (8, 16, 128, 8), (3, 130, 100, 2), (1, 700, 255, 8), (2, 1025, 256, 8), (300, 1, 16, 2),
         (77, 3, 250, 1), (1, 40000, 4, 2), (1, 100, 33, 4), (1, 128, 64, 6), (1, 129, 64, 6), (1, 256, 16, 2),
         (1, 257, 16, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,E,K", CASES)
def test_runner(B, T, E, K, dtype, score):
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    N = B * T
    l = logits_of(N, E, dtype, seed=N + E)
    r = MoEBalanceRunner(N, E, K, dtype, seq_len=T, alpha=0.02, z_coef=0.005, score=score)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    mask = torch.rand(N, generator=g, device="cuda") < 0.7
    given = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(min(N, 50))])
    given = given.repeat((N + len(given) - 1) // len(given), 1)[:N].to(torch.int32).contiguous()
    bias = torch.randn(E, generator=g, device="cuda")
    for kw in (dict(), dict(mask=mask), dict(topk=given), dict(topk=given, mask=mask), dict(bias=bias, mask=mask)):
        loss = r.forward(l, **kw).clone()
        d = r.backward().clone()
        check(l, K, T, 0.02, 0.005, score, loss=loss, counts=r.counts, d=d, **kw)
        again = r.forward(l, **kw)
        assert torch.equal(again, loss) and torch.equal(r.backward(), d)  # bit for bit


def test_ties_infinities_and_nan():
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    N, E, K = 64, 40, 5
    l = torch.round(logits_of(N, E, torch.float32, seed=2))     # many equal logits, 0 and -0 among them
    l[0] = 0.0
    l[1] = -0.0
    l[2, ::2] = -float("inf")
    r = MoEBalanceRunner(N, E, K, torch.float32, alpha=0.1, z_coef=0.01)
    loss = r.forward(l)
    check(l, K, N, 0.1, 0.01, "softmax", loss=loss, counts=r.counts, d=r.backward())
    assert float(r.dlogits[2, ::2].abs().max()) == 0.0
    # NaN in a token that counts: its gradients and the loss; the others' gradients stay
    clean = r.dlogits.clone()
    ids = order(l, None, K).to(torch.int32).contiguous()
    l[7, 3] = float("nan")
    loss = r.forward(l, topk=ids)
    d = r.backward()
    others = torch.arange(N, device="cuda") != 7
    assert bool(torch.isnan(loss).all()) and bool(torch.isnan(d[7]).all()) and torch.equal(d[others], clean[others])
    # in padding it is not looked at
    mask = others
    loss = r.forward(l, topk=ids, mask=mask)
    check(torch.where(mask[:, None], l, torch.zeros_like(l)), K, N, 0.1, 0.01, "softmax", topk=ids, mask=mask, loss=loss,
          counts=r.counts, d=r.backward())
    # NaN logits are chosen last
    l = logits_of(N, E, torch.float32, seed=3)
    l[:, :E - K] = float("nan")
    r.forward(l)
    assert r.counts.tolist() == [0] * (E - K) + [N] * K
    l[:] = float("nan")
    r.forward(l)
    assert r.counts.tolist() == [N] * K + [0] * (E - K)


@pytest.mark.parametrize("E", [12, 20, 60, 100])
def test_choice_among_few_numbers(E):
    """Tokens of 0 to 12 logits that are numbers, 0 to 10 of these -inf, the others NaN: -inf in front of
    NaN, NaN by its expert, and K chosen experts for every token, also where the numbers and the places
    behind the last expert are K together."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    N, K = 13 * 11, 8
    l = logits_of(N, E, torch.float32, seed=E)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    place = torch.argsort(torch.rand((N, E), generator=g, device="cuda"), dim=1)
    i = torch.arange(N, device="cuda")[:, None]
    l = torch.where(place < i % 13, l, torch.full_like(l, float("nan")))
    l = torch.where(place < torch.minimum(i % 13, i // 13), torch.full_like(l, -float("inf")), l)
    r = MoEBalanceRunner(N, E, K, torch.float32)
    r.forward(l)
    want = torch.bincount(order(l, None, K).reshape(-1), minlength=E)
    assert int(want.sum()) == N * K and torch.equal(r.counts.long(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-300.0, -80.0, 60.0, 300.0])
def test_large_logits(score, shift):
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    N, E, K = 200, 24, 2
    l = logits_of(N, E, torch.float32, seed=5, scale=3.0) + shift
    r = MoEBalanceRunner(N, E, K, torch.float32, alpha=0.1, z_coef=1e-4, score=score)
    loss = r.forward(l)
    check(l, K, N, 0.1, 1e-4, score, loss=loss, counts=r.counts, d=r.backward())


def test_sequences_without_tokens_and_ids_outside():
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    B, T, E, K = 6, 50, 16, 4
    l = logits_of(B * T, E, torch.bfloat16)
    r = MoEBalanceRunner(B * T, E, K, torch.bfloat16, seq_len=T, alpha=0.3, z_coef=0.01)
    mask = torch.ones((B, T), dtype=torch.uint8, device="cuda")
    mask[1] = 0
    mask[4] = 0
    mask[2, 1:] = 0
    ids = order(l, None, K).to(torch.int32)
    ids[::3, 2] = -1
    ids[::5, 0] = E
    ids[::7, 1] = 2 ** 31 - 1
    ids = ids.contiguous()
    loss = r.forward(l, topk=ids, mask=mask)
    check(l, K, T, 0.3, 0.01, "softmax", topk=ids, mask=mask, loss=loss, counts=r.counts, d=r.backward())
    mask.zero_()
    loss = r.forward(l, topk=ids, mask=mask)
    assert float(loss) == 0.0 and int(r.counts.abs().max()) == 0 and float(r.backward().abs().max()) == 0.0
    one = MoEBalanceRunner(T, E, K, torch.bfloat16, alpha=0.3, z_coef=0.01)
    loss = one.forward(l[:T].contiguous(), mask=mask[0].contiguous())
    assert float(loss) == 0.0 and float(one.backward().abs().max()) == 0.0


def test_agrees_with_the_layers_own_loss():
    """One sequence, softmax scores, no padding: moe_aux_loss on the same logits."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner, MoELayerRunner
    N, H, F, E, K = 500, 128, 128, 8, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn((N, H), generator=g, device="cuda")
    w = [torch.randn(s, generator=g, device="cuda") * 0.1 for s in ((H, E), (E, H, F), (E, H, F), (E, F, H))]
    layer = MoELayerRunner(N, H, F, E, K, torch.float32, aux_alpha=0.05)
    layer.forward(x, *w)
    r = MoEBalanceRunner(N, E, K, torch.float32, alpha=0.05)
    loss = r.forward((x.double() @ w[0].double()).float(), topk=layer.topk)
    assert torch.equal(r.counts, layer.counts)
    assert abs(float(loss) - float(layer.aux_loss)) <= 1e-6 * float(loss)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_autograd(score):
    from mixture_experts_layer_sort_amd import moe_balance_loss
    B, T, E, K = 4, 30, 10, 3
    l = logits_of(B * T, E, torch.float32, seed=9).reshape(B, T, E)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    mask = torch.rand((B, T), generator=g, device="cuda") < 0.8
    leaf = l.clone().requires_grad_()
    loss, counts = moe_balance_loss(leaf, K, mask=mask, seq_len=T, alpha=0.2, z_coef=0.03, score=score)
    assert loss.requires_grad and not counts.requires_grad and counts.dtype == torch.int32
    (3.0 * loss).sum().backward()
    flat = l.reshape(B * T, E)
    check(flat, K, T, 0.2, 0.03, score, mask=mask, loss=loss.detach(), counts=counts, d=leaf.grad.reshape(B * T, E) / 3.0)
    # against differences of the float64 loss, the choice of experts held
    ids = order(flat, None, K)
    h = 1e-6
    for n, e in ((0, 0), (17, 4), (B * T - 1, 9), (50, 7)):
        up, dn = flat.double().clone(), flat.double().clone()
        up[n, e] += h
        dn[n, e] -= h
        diff = (reference(up, ids, mask, T, 0.2, 0.03, score)[0] - reference(dn, ids, mask, T, 0.2, 0.03, score)[0]) / (2 * h)
        # the third derivative's h^2 and the loss's rounding over h, both below 1e-9; the gradient's own 1e-6 of its size
        assert abs(float(leaf.grad.reshape(-1, E)[n, e]) / 3.0 - diff) <= 1e-8 + 1e-5 * abs(diff)
    # views at any element, a double use, and a loss that nothing depends on
    wide = torch.randn((B * T, E + 1), device="cuda", requires_grad=True)
    a, _ = moe_balance_loss(wide[:, 1:], K, alpha=0.1)
    b, _ = moe_balance_loss(wide[:, 1:], K, alpha=0.1, z_coef=0.1)
    (a + b).backward()
    assert wide.grad.shape == wide.shape and float(wide.grad[:, 0].abs().max()) == 0.0
    assert bool(torch.isfinite(wide.grad).all()) and float(wide.grad.abs().max()) > 0.0
    empty = torch.zeros((0, E), device="cuda", requires_grad=True)
    loss, counts = moe_balance_loss(empty, K)
    loss.backward()
    assert float(loss) == 0.0 and int(counts.sum()) == 0 and empty.grad.shape == (0, E)


def test_training_step_with_the_layer():
    """The loss next to the layer in one training step, as a user writes it: gradients reach x and W_r along
    both paths, the sum of the two taken apart."""
    from mixture_experts_layer_sort_amd import moe_balance_loss, moe_layer
    N, H, F, E, K = 96, 128, 128, 8, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((N, H), generator=g, device="cuda")
    w = [torch.randn(s, generator=g, device="cuda") * 0.1 for s in ((H, E), (E, H, F), (E, H, F), (E, F, H))]

    def grads(task, balance):
        leaves = [t.clone().requires_grad_() for t in (x, *w)]
        total = 0.0
        if task:
            total = total + moe_layer(*leaves, K).square().mean()
        if balance:
            total = total + moe_balance_loss(leaves[0] @ leaves[1], K, seq_len=N // 2, alpha=0.5, z_coef=0.1)[0].sum()
        return torch.autograd.grad(total, leaves, allow_unused=True)

    whole, one, two = grads(True, True), grads(True, False), grads(False, True)
    for i in range(5):
        want = one[i] if two[i] is None else one[i] + two[i]
        assert torch.allclose(whole[i], want, rtol=1e-6, atol=1e-9)
    assert float(two[0].abs().max()) > 0 and float(two[1].abs().max()) > 0 and two[2] is None


def test_refusals_change_nothing():
    from mixture_experts_layer_sort_amd import MoEBalanceRunner, MoEError, moe_balance_loss
    N, E, K = 32, 8, 2
    l = logits_of(N, E, torch.float32)
    r = MoEBalanceRunner(N, E, K, torch.float32)
    with pytest.raises(RuntimeError):
        r.backward()
    loss = float(r.forward(l))
    ids = torch.zeros((N, K), dtype=torch.int32, device="cuda")
    bias = torch.zeros(E, device="cuda")
    for args in (dict(logits=l[:16]), dict(logits=l.bfloat16()), dict(logits=l, topk=ids.long()),
                 dict(logits=l, topk=ids[:, :1]), dict(logits=l, topk=ids, bias=bias), dict(logits=l, bias=bias[:4]),
                 dict(logits=l, mask=torch.ones(N, device="cuda")), dict(logits=l, mask=ids[:16, 0] > 0)):
        with pytest.raises(ValueError):
            r.forward(**args)
    with pytest.raises(ValueError):
        r.backward(torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        MoEBalanceRunner(N, E, K, torch.float32, score="relu")
    for kw in (dict(seq_len=5), dict(alpha=float("nan"))):
        with pytest.raises(MoEError):
            MoEBalanceRunner(N, E, K, torch.float32, **kw)
        with pytest.raises(MoEError):
            moe_balance_loss(l, K, **kw)
    with pytest.raises(ValueError):
        moe_balance_loss(l, K, topk=ids, bias=bias)
    assert float(r.loss) == loss
    none = MoEBalanceRunner(0, E, K, torch.float32)
    assert float(none.forward(l[:0])) == 0.0 and none.backward().shape == (0, E)
    up = torch.full((1,), -2.5, device="cuda")
    d = r.backward().clone()
    assert torch.allclose(r.backward(up), -2.5 * d, rtol=1e-6, atol=0)


def test_on_another_stream_and_captured():
    from mixture_experts_layer_sort_amd import MoEBalanceRunner, moe_balance_loss
    B, T, E, K = 4, 300, 64, 6
    l = logits_of(B * T, E, torch.bfloat16)
    r = MoEBalanceRunner(B * T, E, K, torch.bfloat16, seq_len=T, z_coef=0.01)
    want = r.forward(l).clone(), r.counts.clone(), r.backward().clone()
    side = torch.cuda.Stream()
    for t in (r.loss, r.counts, r.dlogits):
        t.zero_()
    torch.cuda.synchronize()
    r.forward(l, stream=side)
    r.backward(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((r.loss, r.counts, r.dlogits), want))
    graph, leaf = torch.cuda.CUDAGraph(), l.clone().requires_grad_()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        torch.autograd.grad(moe_balance_loss(leaf, K, seq_len=T, z_coef=0.01)[0], leaf)
    torch.cuda.current_stream().wait_stream(warm)
    with torch.cuda.graph(graph):
        r.forward(l)
        r.backward()
        out = moe_balance_loss(leaf, K, seq_len=T, z_coef=0.01)
        grad, = torch.autograd.grad(out[0], leaf)
    for i in range(4):
        new = logits_of(B * T, E, torch.bfloat16, seed=20 + i)
        l.copy_(new)
        leaf.data.copy_(new)
        fresh = MoEBalanceRunner(B * T, E, K, torch.bfloat16, seq_len=T, z_coef=0.01)
        want = fresh.forward(new).clone(), fresh.counts.clone(), fresh.backward().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((r.loss, r.counts, r.dlogits), want))
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(grad, want[2])


def test_two_streams_at_once():
    """Runners of their own on two streams, one with its sums in one workgroup: the results of one after the other."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    l = [logits_of(203, 8, torch.float32, seed=1), logits_of(4096, 64, torch.float32, seed=2)]
    r = [MoEBalanceRunner(203, 8, 2, torch.float32, z_coef=0.01), MoEBalanceRunner(4096, 64, 6, torch.float32, seq_len=512)]
    want = []
    for run, v in zip(r, l):
        loss = run.forward(v).clone()
        want.append((loss, run.counts.clone(), run.backward().clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for run, v, s in zip(r, l, streams):
            run.forward(v, stream=s)
            run.backward(stream=s)
    torch.cuda.synchronize()
    for run, (loss, counts, d) in zip(r, want):
        assert torch.equal(run.loss, loss) and torch.equal(run.counts, counts) and torch.equal(run.dlogits, d)


def test_runner_of_another_stream():
    """A runner made behind work of the current stream and called on another one: its first values (zeros) come
    before the call's, not after them."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    l = logits_of(203, 8, torch.float32)
    r = MoEBalanceRunner(203, 8, 2, torch.float32, z_coef=0.01)
    want = r.forward(l).clone(), r.counts.clone(), r.backward().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    v = torch.zeros(1 << 28, device="cuda")
    for _ in range(40):
        v.add_(1.0)
    r = MoEBalanceRunner(203, 8, 2, torch.float32, z_coef=0.01)
    r.forward(l, stream=side)
    r.backward(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((r.loss, r.counts, r.dlogits), want))


@pytest.mark.parametrize("top", [0.0, 1.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [4, 40, 256])
def test_small_probabilities(E, score, top):
    """Tokens whose first logit is 0 or 1 and whose others go down to -85 in steps of 2^-10, so that differences are
    exact.  A gradient is c p_e (f_e - f.p) [1 - sigmoid].  A sum over the experts, of one sign, adds up E / 16 values in
    a lane and sixteen lanes pairwise: E / 16 + 5 u of itself.  p_e: 3 u of an exponential, 3 u of a sigmoid, the sum, 2 u
    of the quotient; f.p: the same and a product, and the sum; f_e 1 u; 10 u of the products.  So its error is at most
    (E / 8 + 39) u c p_e (f_e + f.p) [1 - sigmoid].  An exponential that is off by |x| u alone is past that at 4 and
    40 experts (61 to 65 u)."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    N = 512
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    l = -torch.randint(1024, 85 * 1024, (N, E), generator=g, device="cuda").float() / 1024
    l[:, 0] = top
    ids = torch.randint(1, E, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    ids[:E - 1, 0] = torch.arange(1, E, device="cuda")
    r = MoEBalanceRunner(N, E, 1, torch.float32, alpha=float(N), score=score)
    r.forward(l, topk=ids)
    d = r.backward().double()
    x = l.double()
    f = torch.bincount(ids[:, 0].long(), minlength=E).double() * E / N
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x) / torch.sigmoid(x).sum(1, keepdim=True)
    rest = torch.ones_like(x) if score == "softmax" else torch.sigmoid(-x)
    fp = (p * f).sum(1, keepdim=True)
    worst = float(((d - p * (f - fp) * rest).abs() / (p * (f + fp) * rest)).max() / U)
    print(f"[balance] worst {worst:.1f} u", flush=True)
    assert worst <= E / 8 + 39


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [1, 16, 33, 60, 128, 250, 256])
def test_gradient_in_place_of_the_logits(E, dtype):
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    from mixture_experts_layer_sort_amd import _lib as L
    N = 700
    l = logits_of(N, E, dtype, seed=E)
    mask = torch.arange(N, device="cuda") % 5 != 0
    for score in ("softmax", "sigmoid"):
        r = MoEBalanceRunner(N, E, 1, dtype, seq_len=100, alpha=0.3, z_coef=0.01, score=score)
        r.forward(l, mask=mask)
        want, d = r.backward().clone(), l.clone()
        L.moe_balance_loss_bwd(r.b, d, mask, r.state, None, d)
        assert torch.equal(d, want)


def test_the_layers_own_choice_in_bf16():
    """A bf16 training step as a user writes it: the loss counts the experts that the layer chose, which a choice made
    again on bf16 logits does not; gradients are those of the loss and of the layer taken apart."""
    from mixture_experts_layer_sort_amd import MoELayerRunner, moe_balance_loss, moe_layer
    N, H, F, E, K = 4000, 128, 128, 64, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x = torch.randn((N, H), generator=g, device="cuda").bfloat16()
    w = [(torch.randn(s, generator=g, device="cuda") * 0.1).bfloat16() for s in ((H, E), (E, H, F), (E, H, F), (E, F, H))]
    leaves = [t.clone().requires_grad_() for t in (x, *w)]
    y, topk = moe_layer(*leaves, K, return_topk=True)
    assert topk.dtype == torch.int32 and topk.shape == (N, K) and not topk.requires_grad
    loss, counts = moe_balance_loss(leaves[0].float() @ leaves[1].float(), K, topk=topk, alpha=0.1)
    kept = topk.clone()
    r = MoELayerRunner(N, H, F, E, K, torch.bfloat16)
    r.forward(x, *w)
    assert torch.equal(topk, r.topk) and torch.equal(counts, r.counts)
    again = moe_balance_loss(x @ w[0], K)[1]
    assert not torch.equal(again, counts)
    # float32 logits are off by (H + 1) u |x|.|W_r|, probabilities by twice that of themselves
    want, tol = reference((x.double() @ w[0].double()).float(), topk, None, N, 0.1, 0.0, "softmax")[:2]
    off = (H + 1) * U * float((x.double().abs() @ w[0].double().abs()).max())
    assert abs(float(loss.detach()) - want) <= 1.01 * (tol + 2 * off * want)
    both = torch.autograd.grad(y.float().square().mean() + loss.sum(), leaves, retain_graph=True)
    topk.zero_()  # the caller's own
    again = torch.autograd.grad(y.float().square().mean(), leaves)
    ref = r.backward((2 * y.detach().float() / y.numel()).bfloat16())
    assert torch.equal(again[0], ref["dx"]) and torch.equal(again[1], ref["dw_r"].bfloat16())
    assert not torch.equal(both[1], again[1])
    # in the order y, aux loss, choice; and y alone as before
    out = moe_layer(x, *w, K, aux_alpha=0.01, return_topk=True)
    assert len(out) == 3 and torch.equal(out[0], y.detach()) and torch.equal(out[2], kept)
    assert torch.equal(moe_layer(x, *w, K), y.detach())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,T", [(2, 1), (64, 1), (40, 2), (900, 1), (7, 17)])
def test_short_sequences_of_padding(B, T, score):
    """Sequences that are nothing but padding, one token long too, among others: they count neither as sequences nor
    as tokens."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    E, K = 24, 3
    l = logits_of(B * T, E, torch.float32, seed=B)
    ends = torch.arange(B, device="cuda") * 5 % (T + 1)
    ends[0] = T
    mask = (torch.arange(T, device="cuda") < ends[:, None])
    assert B < 3 or bool((ends < T).any())
    l[~mask.reshape(-1)] = float("nan")
    r = MoEBalanceRunner(B * T, E, K, torch.float32, seq_len=T, alpha=0.3, z_coef=0.01, score=score)
    loss = r.forward(l, mask=mask)
    check(torch.where(mask.reshape(-1, 1), l, torch.zeros_like(l)), K, T, 0.3, 0.01, score, mask=mask, loss=loss,
          counts=r.counts, d=r.backward())


def test_runner_made_on_a_side_stream():
    """Made on a side stream, called on the default one, by its raw handle too; first called in a capture."""
    from mixture_experts_layer_sort_amd import MoEBalanceRunner
    l = logits_of(500, 40, torch.float32)
    want = MoEBalanceRunner(500, 40, 2, torch.float32).forward(l).clone()
    side = torch.cuda.Stream()
    for stream in (None, torch.cuda.current_stream().cuda_stream, torch.cuda.current_stream()):
        with torch.cuda.stream(side):
            r = MoEBalanceRunner(500, 40, 2, torch.float32)
        assert torch.equal(r.forward(l, stream=stream), want)
    r, g = MoEBalanceRunner(500, 40, 2, torch.float32), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.forward(l)
    for _ in range(3):
        r.loss.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.loss, want)
    r.loss.zero_()
    assert torch.equal(r.forward(l), want)

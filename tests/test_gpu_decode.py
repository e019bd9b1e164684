"""The layer for a few tokens (moe_decode) against a plain float64 evaluation.

Tolerances.  u = 2^-24, s = 2^-8 (bf16) or 2^-24 (float32), the largest
relative error of one rounding.  A float32 sum of n products, in any order, is
off by at most (n + 1) u sum|products| (to first order).  So, element by
element, with eG = (H + 8) u (|x|.|W_gate|) and eU alike, and |silu'| <= 1.1:
  eA = 1.1 |U| eG + |silu(G)| eU + (8 u + s^2) |A|      (bf16: A = hi + lo)
  e  = sum_k g_k (eA.|W_down| + (F + 16) u |A|.|W_down|)   (+ the shared expert's)
  |y - ref| <= s |ref| + 1.01 (e + gate error).
Gates: expf and the softmax's sum and quotient are good to a few u; the
difference of two logits is rounded to float32 once, so the relative error is at
most (16 + max|difference|) u.  Beside the worst case, a bf16 y that is rounded
once has a root-mean-square error of 2^-8 / sqrt(3) * sqrt(0.75 / (2 ln 2)) =
1.66e-3 of its own (mantissas spread evenly over a logarithm); with an
activation rounded to bf16 it would be about 2.3e-3.  2e-3 separates the two."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(N, H, F, E, K, dtype, Fs=0, bias=False, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(shape, s):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(dtype)

    sh = (r((H, Fs), H ** -0.5), r((H, Fs), H ** -0.5), r((Fs, H), Fs ** -0.5)) if Fs else None
    b = torch.randn((E,), generator=g, device="cuda") * 0.3 if bias else None
    return dict(x=r((N, H), 1.0), w_r=r((H, E), 0.02), w_gate=r((E, H, F), H ** -0.5), w_up=r((E, H, F), H ** -0.5),
                w_down=r((E, F, H), F ** -0.5), bias=b, shared=sh)


def _runner(N, t, K, Fs=0):
    from mixture_experts_layer_sort_amd import MoEDecodeRunner
    E, H, F = t["w_gate"].shape
    return MoEDecodeRunner(N, H, F, E, K, t["x"].dtype, "cuda", shared_ffn=Fs or None)


def _forward(r, t, **kw):
    return r.forward(t["x"], t["w_r"], t["w_gate"], t["w_up"], t["w_down"], bias=t["bias"], shared=t["shared"], **kw)


def _ffn(x, wg, wu, wd, s):
    """Output and error bound of one expert for the rows x (float64)."""
    x, wg, wu, wd = x.double(), wg.double(), wu.double(), wd.double()
    H, F = wg.shape
    G, Uu = x @ wg, x @ wu
    eG, eU = (H + 8) * U * (x.abs() @ wg.abs()), (H + 8) * U * (x.abs() @ wu.abs())
    silu = G * torch.sigmoid(G)
    A = silu * Uu
    eA = 1.1 * Uu.abs() * eG + silu.abs() * eU + (8 * U + (s * s if s > U else 0.0)) * A.abs()
    return A @ wd, (eA + (F + 16) * U * A.abs()) @ wd.abs()


def reference(t, K):
    """topk, gates, y and y's error bound before the last rounding."""
    x = t["x"]
    s = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    l = x.double() @ t["w_r"].double()
    if t["bias"] is not None:
        l = l + t["bias"].double()
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    gates = torch.softmax(top, 1)
    ge = (16 + (top[:, :1] - top).max().item()) * U
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    e = torch.zeros_like(y)
    for ex in range(t["w_r"].shape[1]):
        n, k = torch.nonzero(ids == ex, as_tuple=True)
        if n.numel():
            o, eo = _ffn(x[n], t["w_gate"][ex], t["w_up"][ex], t["w_down"][ex], s)
            y[n] += gates[n, k, None] * o
            e[n] += gates[n, k, None] * (eo + (ge + 8 * U) * o.abs())
    if t["shared"] is not None:
        o, eo = _ffn(x, *t["shared"], s)
        y += o
        e += eo + 4 * U * o.abs()
    return ids, gates, ge, y, e, s


def check(t, K, r, y, rows=None):
    ids, gates, ge, ry, e, s = reference(t, K)
    keep = slice(None) if rows is None else rows
    assert torch.equal(r.topk[keep].long(), ids[keep])
    assert ((r.gates[keep].double() - gates[keep]).abs() <= ge * gates[keep]).all()
    err = (y.double() - ry).abs()[keep]
    tol = (s * ry.abs() + 1.01 * e)[keep]
    worst = (err / tol.clamp_min(1e-300)).max().item()
    rms = (err.square().mean().sqrt() / ry[keep].square().mean().sqrt()).item()
    print(f"[decode] worst err/tol {worst:.3f} rel-RMS {rms:.2e}", flush=True)
    assert (err <= tol).all(), worst
    if s > U and err.numel() >= 8192:
        assert rms <= 2e-3, rms


# (N, H, F, E, K, Fs, bias)
SHAPES = [
    (1, 128, 128, 1, 1, 0, False),        # one expert, one token, one panel of F per wave
    (1, 512, 1024, 8, 2, 0, False),
    (2, 128, 256, 5, 5, 128, True),       # every expert chosen
    (3, 256, 384, 256, 8, 0, True),       # far more experts than slots
    (7, 384, 128, 13, 3, 0, False),       # odd expert count: rows of W_r unaligned
    (15, 256, 256, 3, 2, 384, False),
    (16, 128, 640, 4, 1, 0, True),
    (17, 256, 256, 4, 2, 0, False),       # a second row tile
    (32, 640, 128, 64, 6, 256, True),
    (33, 128, 384, 1, 1, 0, False),       # one expert has all 33 rows
    (47, 256, 128, 100, 7, 0, False),
    (64, 512, 256, 8, 8, 128, True),      # the most tokens, every expert has all of them
    (64, 128, 128, 256, 8, 0, False),
    (5, 2048, 128, 6, 2, 0, False),
    (4, 128, 2048, 6, 2, 0, False),
    # many strips of columns and many rows each: gate and up in one workgroup
    (16, 128, 6528, 8, 8, 128, False),
    (40, 256, 6528, 8, 4, 384, True),     # a last single segment, two row tiles
    (64, 128, 6656, 8, 8, 0, False),      # more rows than two row tiles
    (64, 128, 6528, 8, 8, 128, False),
    (24, 1152, 256, 4, 3, 1408, False),   # a shared expert much longer than the routed ones
    (2, 640, 384, 64, 8, 256, True),      # the workgroups route by themselves, logits from the first kernel
    (2, 256, 128, 16, 4, 0, True),        # ... and the logits too
    (1, 128, 384, 200, 7, 0, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "n{}_h{}_f{}_e{}_k{}_s{}_b{}".format(*map(int, s)))
def test_decode_matches_float64(shape, dtype):
    N, H, F, E, K, Fs, bias = shape
    t = _inputs(N, H, F, E, K, dtype, Fs, bias, seed=N + E)
    r = _runner(N, t, K, Fs)
    y = _forward(r, t)
    torch.cuda.synchronize()
    check(t, K, r, y)


@pytest.mark.parametrize("seed", range(24))
def test_random_sizes(seed):
    """Sizes spread over the whole range of tokens, experts and types."""
    import random
    rng = random.Random(1000 + seed)
    N = rng.choice([1, 2, 3, rng.randint(4, 16), rng.randint(17, 32), rng.randint(33, 64)])
    E = rng.choice([1, 2, rng.randint(3, 16), rng.randint(17, 64), rng.randint(65, 256)])
    K, dtype = rng.randint(1, min(8, E)), rng.choice([torch.bfloat16, torch.float32])
    H = 128 * rng.randint(1, 12)
    F = 128 * rng.randint(1, max(1, min(24, (1 << 26) // (E * H * 128))))
    Fs, bias = rng.choice([0, 128 * rng.randint(1, 12)]), rng.random() < 0.5
    print("[decode]", N, H, F, E, K, Fs, bias, dtype, flush=True)
    t = _inputs(N, H, F, E, K, dtype, Fs, bias, seed=seed)
    r = _runner(N, t, K, Fs)
    r.ws.fill_(255)
    y = _forward(r, t)
    torch.cuda.synchronize()
    check(t, K, r, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,H,Fs", [(17, 8192, 8320), (64, 256, 16384), (40, 4224, 2176), (12, 512, 8192)])
def test_shared_expert_much_longer_than_the_routed_ones(N, H, Fs, dtype):
    t = _inputs(N, H, 128, 3, 2, dtype, Fs, seed=N)
    r = _runner(N, t, 2, Fs)
    check(t, 2, r, _forward(r, t))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("F", [256, 6528])               # gate and up apart, and in one workgroup
@pytest.mark.parametrize("N", [16, 17, 32, 33, 48, 49, 64])
def test_every_number_of_row_tiles(N, F, dtype):
    """Every expert has all N rows."""
    t = _inputs(N, 128, F, 8, 8, dtype, 384, True, seed=N)
    r = _runner(N, t, 8, 384)
    check(t, 8, r, _forward(r, t))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,E", [(8, 8), (13, 8), (16, 4)])
def test_few_tokens_of_wide_experts(N, E, dtype):
    """About as many strips as CUs, all rows in one tile: gate and up in one workgroup."""
    t = _inputs(N, 512, 4480, E, E, dtype, 384, True, seed=N)
    r = _runner(N, t, E, 384)
    check(t, E, r, _forward(r, t))


@pytest.mark.parametrize("H", [128, 640, 1152])
@pytest.mark.parametrize("N,E,K", [(16, 16, 8), (8, 32, 5), (15, 17, 3), (3, 85, 8), (1, 256, 8), (9, 29, 4), (2, 129, 8)])
def test_routing_around_one_pair_a_thread(N, E, K, H):
    t = _inputs(N, H, 128, E, K, torch.bfloat16, 0, True, seed=E)
    r = _runner(N, t, K)
    check(t, K, r, _forward(r, t))


@pytest.mark.parametrize("N,E,K", [(64, 8, 2), (40, 64, 6), (64, 256, 1)])
def test_skewed_routing(N, E, K):
    """A bias that sends every token to the same experts (rows of all others empty)."""
    t = _inputs(N, 256, 256, E, K, torch.bfloat16, seed=3)
    t["bias"] = torch.zeros(E, device="cuda")
    t["bias"][E - K:] = 50.0
    r = _runner(N, t, K)
    y = _forward(r, t)
    assert (r.topk >= E - K).all()
    check(t, K, r, y)


def test_fewer_tokens_than_the_runner_holds():
    """Rows behind the last token keep what they held; no tokens at all is fine."""
    t = _inputs(9, 256, 256, 16, 4, torch.bfloat16, Fs=128, seed=5)
    r = _runner(24, t, 4, 128)
    r._y.fill_(7.0)
    r._gates.fill_(7.0)
    r._topk.fill_(7)
    y = _forward(r, t)
    assert y.shape == (9, 256) and r.topk.shape == (9, 4)
    check(t, 4, r, y)
    assert (r._y[9:] == 7).all() and (r._gates[9:] == 7).all() and (r._topk[9:] == 7).all()
    t["x"] = t["x"][:0]
    assert _forward(r, t).shape == (0, 256)
    assert (r._y[9:] == 7).all()


def test_equal_logits_go_to_the_lowest_experts():
    t = _inputs(6, 128, 128, 40, 5, torch.bfloat16, seed=6)
    t["x"][2] = 0                                   # all logits equal
    t["w_r"][:, 20:] = t["w_r"][:, :20]             # pairs of equal logits
    r = _runner(6, t, 5)
    y = _forward(r, t)
    check(t, 5, r, y)
    assert r.topk[2].tolist() == [0, 1, 2, 3, 4] and (y[2] == 0).all()


def test_nan_and_infinite_tokens_stay_in_their_rows():
    """A NaN token ranks experts by id; the other rows are the same bits as without it."""
    t = _inputs(5, 256, 128, 8, 2, torch.bfloat16, seed=7)
    r = _runner(5, t, 2)
    t["x"][1], t["x"][3] = 0, 0
    before = _forward(r, t).clone()
    t["x"][1, 5] = float("nan")
    t["x"][3] = 3e38
    y = _forward(r, t)
    assert r.topk[1].tolist() == [0, 1]
    assert torch.isnan(y[1]).all()
    for n in (0, 2, 4):
        assert torch.equal(y[n], before[n])


def test_nan_logits_rank_last():
    t = _inputs(3, 128, 128, 6, 3, torch.float32, seed=8)
    t["bias"] = torch.zeros(6, device="cuda")
    t["bias"][[0, 2]] = float("nan")
    r = _runner(3, t, 3)
    _forward(r, t)
    assert not torch.isin(r.topk, torch.tensor([0, 2], device="cuda", dtype=torch.int32)).any()
    assert torch.isfinite(r.gates).all()
    t["bias"][:] = float("-inf")
    t["bias"][4] = 0.0
    _forward(r, t)
    assert r.topk.tolist() == [[4, 0, 1]] * 3
    assert r.gates.tolist() == [[1.0, 0.0, 0.0]] * 3


def test_gates_of_zero_add_nothing_and_weights_stay_unread_elsewhere():
    """Experts that no token chose may hold anything."""
    t = _inputs(4, 256, 256, 12, 2, torch.bfloat16, seed=9)
    t["bias"] = torch.zeros(12, device="cuda")
    t["bias"][4:] = -100.0
    r = _runner(4, t, 2)
    good = _forward(r, t).clone()
    for w in ("w_gate", "w_up", "w_down"):
        t[w][4:] = float("nan")
    assert torch.equal(_forward(r, t), good)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_every_number_of_tokens_on_one_runner(dtype):
    t = _inputs(64, 256, 384, 12, 3, dtype, Fs=128, bias=True, seed=14)
    r = _runner(64, t, 3, 128)
    x = t["x"]
    for n in list(range(1, 65)) + [1, 40, 2]:
        t["x"] = x[:n].contiguous()
        check(t, 3, r, _forward(r, t))


def test_two_runners_on_two_streams_at_once():
    jobs = []
    for i, (N, E) in enumerate(((1, 16), (12, 16), (50, 8))):
        t = _inputs(N, 512, 1024, E, 2, torch.bfloat16, seed=20 + i)
        r = _runner(N, t, 2)
        jobs.append((t, r, _forward(r, t).clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for t, r, _, s in jobs:
            r._y.fill_(float("nan"))
        torch.cuda.synchronize()
        for t, r, _, s in jobs:
            _forward(r, t, stream=s)
        torch.cuda.synchronize()
        for _, r, want, _ in jobs:
            assert torch.equal(r.y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 12, 24])
def test_non_finite_weights_reach_only_the_tokens_that_chose_them(N, dtype):
    """An expert with infinite and NaN weights: tokens routed elsewhere are as without it."""
    t = _inputs(N, 256, 256, 8, 2, dtype, Fs=128, seed=13)
    t["bias"] = torch.zeros(8, device="cuda")
    t["x"][:] *= 0.5
    r = _runner(N, t, 2, 128)
    good = _forward(r, t).clone()
    bad = int(r.topk[0, 0])
    hit = (r.topk == bad).any(1)
    assert hit.any() and not hit.all()
    for w, v in (("w_gate", float("nan")), ("w_up", float("inf")), ("w_down", float("inf"))):
        for value in (v, float("nan")):
            keep = t[w][bad].clone()
            t[w][bad, 3, 7] = value
            y = _forward(r, t)
            assert torch.equal(y[~hit], good[~hit]), w
            assert not torch.isfinite(y[hit]).all(), w
            t[w][bad] = keep


def test_same_bits_with_a_dirty_workspace_another_stream_and_a_graph():
    t = _inputs(19, 384, 512, 32, 4, torch.bfloat16, Fs=256, bias=True, seed=10)
    r = _runner(32, t, 4, 256)
    y = _forward(r, t).clone()
    topk, gates = r.topk.clone(), r.gates.clone()
    check(t, 4, r, y)
    for fill in (0, 255, 127):
        r.ws.fill_(fill)
        assert torch.equal(_forward(r, t), y) and torch.equal(r.topk, topk) and torch.equal(r.gates, gates)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.ws.fill_(255)
    side.wait_stream(torch.cuda.current_stream())
    out = _forward(r, t, stream=side)
    side.synchronize()
    assert torch.equal(out, y)
    # two graphs on one runner (one workspace), replayed in turn with eager work between
    t2 = dict(t, x=t["x"][:3].contiguous())
    y2 = _forward(r, t2).clone()
    graphs = []
    for ti in (t, t2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _forward(r, ti)
        graphs.append((g, r.y))
    x0 = t["x"].clone()
    for i in range(4):
        for (g, out), want in zip(graphs, (y, y2)):
            r.ws.fill_(i * 85)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            torch.randn(1000, device="cuda").sum().item()
    t["x"].copy_(x0.flip(0))                        # a replay reads the tokens that are there then
    graphs[0][0].replay()
    torch.cuda.synchronize()
    got = graphs[0][1].clone()
    assert torch.equal(got, _forward(r, t)) and not torch.equal(got, y)


def test_agrees_with_the_layer():
    """The same layer as MoELayerRunner: equal choices; y within the roundings of both
    (the layer stores G, U, A and the expert rows in bf16)."""
    from mixture_experts_layer_sort_amd import MoELayerRunner
    t = _inputs(48, 512, 768, 16, 4, torch.bfloat16, Fs=256, bias=True, seed=11)
    r = _runner(48, t, 4, 256)
    y = _forward(r, t)
    lr = MoELayerRunner(48, 512, 768, 16, 4, torch.bfloat16, "cuda", backward=False, shared_ffn=256)
    ly = lr.forward(t["x"], t["w_r"], t["w_gate"], t["w_up"], t["w_down"], bias=t["bias"], shared=t["shared"])
    torch.cuda.synchronize()
    assert torch.equal(lr.topk, r.topk)
    d = (ly.double() - y.double())
    # five roundings of 1.66e-3 rms at most on either path's way
    assert (d.square().mean().sqrt() / y.double().square().mean().sqrt()).item() <= 5 * 1.66e-3


def test_decode_reads_offsets_beyond_32_bits():
    """Expert matrices that start behind 2^32 bytes of the weight tensor."""
    E, H, F = 72, 2048, 8192                        # 32 MiB each in bf16: 2.25 GiB a tensor of E
    t = _inputs(2, H, F, 1, 1, torch.bfloat16, seed=12)
    big = {}
    for w in ("w_gate", "w_up", "w_down"):
        src = t[w][0]
        big[w] = torch.zeros((E * 2, *src.shape), dtype=src.dtype, device="cuda")
        big[w][-1] = src
    t.update(big)
    t["w_r"] = torch.zeros((H, 2 * E), dtype=torch.bfloat16, device="cuda")
    t["bias"] = torch.zeros(2 * E, device="cuda")
    t["bias"][-1] = 1.0
    r = _runner(2, t, 1)
    y = _forward(r, t)
    assert (r.topk == 2 * E - 1).all()
    o, e = _ffn(t["x"], t["w_gate"][-1], t["w_up"][-1], t["w_down"][-1], 2.0 ** -8)
    assert ((y.double() - o).abs() <= 2.0 ** -8 * o.abs() + 1.01 * e).all()


def _cancelling_down(A, g):
    """W_down [F, H] with three weights a column, chosen so that the sum over the activations A
    (float64) nearly cancels: about 2^-18 of its terms is left."""
    F = A.numel()
    wd = torch.zeros((F, 128), dtype=torch.float64)
    r = lambda v: v.to(torch.bfloat16).double()  # noqa: E731
    for h in range(128):
        f = torch.randperm(F, generator=g)[:3]
        f = f[torch.argsort(A[f].abs(), descending=True)]
        a = A[f]
        w1 = r(-a[0] / a[1])
        wd[f, h] = torch.stack([torch.ones((), dtype=torch.float64), w1, r(-(a[0] + a[1] * w1) / a[2])])
    return wd


@pytest.mark.parametrize("N,F,E", [(1, 128, 1), (3, 256, 2), (16, 128, 1), (24, 256, 2), (40, 384, 1), (64, 128, 2),
                                   (16, 6528, 8), (24, 6528, 8), (64, 6656, 8)])
def test_activations_keep_float32_accuracy_in_bf16(N, F, E):
    """Tokens with one nonzero value: G and U are single exact products.  All E experts are chosen
    with gates of 1/E (exact), all but one have a W_down of zero, and that one's columns cancel.
    So the sum has three terms: with 8 u of an activation's own, 4 u of the sum's, y is good to
    s |ref| + 12 u |A|.|W_down|.  An activation of two bf16 values (16 bits) misses that for two
    columns of three, by up to a factor of seven."""
    g = torch.Generator()
    g.manual_seed(N + F)
    t = {k: torch.zeros(s, dtype=torch.bfloat16) for k, s in
         dict(x=(N, 128), w_r=(128, E), w_gate=(E, 128, F), w_up=(E, 128, F), w_down=(E, F, 128)).items()}
    t["x"][:, 77] = 1.0
    e = E // 2
    t["w_gate"][:, 77], t["w_up"][:, 77] = torch.randn(E, F, generator=g), torch.randn(E, F, generator=g)
    G, Uu = t["w_gate"][e, 77].double(), t["w_up"][e, 77].double()
    A = G * torch.sigmoid(G) * Uu / E
    wd = _cancelling_down(A, g)
    t["w_down"][e] = wd
    t = {k: v.cuda() for k, v in t.items()}
    t.update(bias=None, shared=None)
    y = _forward(_runner(N, t, E), t).cpu().double()
    ref, tol = A @ wd, 2.0 ** -8 * (A @ wd).abs() + 1.01 * 12 * U * (A.abs() @ wd.abs())
    worst = ((y - ref).abs() / tol).max().item()
    print(f"[decode] worst err/tol {worst:.3f}", flush=True)
    assert worst <= 1.0

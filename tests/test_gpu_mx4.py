"""Microscaled 4-bit tensors and the layer with 4-bit experts against plain float64.

Quantisation is held to equality: scales are powers of two and codes are rounded once
from exact quotients, so there is one right value.

Tolerances of the products.  u = 2^-24, s = 2^-8 (bf16) or 2^-24 (float32), the largest
relative error of one rounding.  Products of two codes, and of a code and a bf16 operand,
are exact in float32; a float32 sum of n of them, in any order, is off by at most
(n + 1) u sum|products| (to first order).  So for the 4-bit products, element by element,
with eG = (H + 8) u (|x|.|W_gate|), eU alike, and |silu'| <= 1.1:
  act: eA = 1.1 |U| eG + |silu(G)| eU + 8 u |A|, then one rounding s |A|;
  ys:  (F + 8) u (|a|.|W_down|), then one rounding.
For the layer over few tokens (weights alone in 4 bits) the activation is split into bf16
operands whose sum is off by at most 2^-16 of it (bf16 layers) or exact, so
  eA = 1.1 |U| eG + |silu(G)| eU + (8 u + split) |A|
  e  = sum_k g_k (eA.|W_down| + (F + 16) u |A|.|W_down|)   (+ the shared expert's)
  |y - ref| <= s |ref| + 1.01 (e + gate error),
gates to (16 + max|logit difference|) u as softmax of float64 logits in float32."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def quantised(v):
    """Values and scale exponents of v [count, K, cols] or [N, K] in 4 bits, float64: the nearest
    magnitude, ties to the even code."""
    v = v.double()
    rows = v.dim() == 2
    b = (v[:, :, None] if rows else v).reshape(v.shape[0], -1, 32, 1 if rows else v.shape[2])
    top = b.abs().amax(2, keepdim=True)
    bad = ~torch.isfinite(top)
    e = torch.floor(torch.log2(torch.where((top > 0) & ~bad, top, torch.ones_like(top)))) - 2
    e = torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(min=-127)
    a = (b / torch.exp2(e)).abs()
    grid = GRID.to(v.device)
    d = (a[..., None] - grid).abs()
    d = d + 1e-9 * (torch.arange(8, device=v.device) % 2) * (d == d.amin(-1, keepdim=True))  # odd codes lose ties
    out = torch.copysign(grid[d.argmin(-1)], b) * torch.exp2(e)
    out = torch.where(bad, torch.full_like(out, float("nan")), out)
    return out.reshape(v.shape), torch.where(bad, torch.full_like(e, 128.0), e)


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128, 128), (3, 128, 256), (2, 640, 384), (1, 1408, 128), (5, 512, 128),
                                   (1, 128), (7, 256), (33, 512), (3, 640), (129, 1408), (2, 4096)])
def test_quantise(dtype, shape):
    from mixture_experts_layer_sort_amd import MoEMx4Tensor as Q
    v = randn(1, *shape)
    v *= torch.exp2(torch.randint(-20, 21, shape, device="cuda", dtype=torch.float32))
    v.view(-1)[::97] = 0
    v = v.to(dtype)
    make = Q.rows if len(shape) == 2 else Q.weights
    q = make(v)
    want, _ = quantised(v)
    for out in (torch.float32, torch.bfloat16):
        got = q.dequantize(out)
        assert got.dtype == out and torch.equal(got.double(), want)
    again = make(q.dequantize(dtype))  # the values are their own 4-bit form
    assert torch.equal(again.dequantize(torch.float32).double(), want)


def borders():
    """Blocks whose values lie on, below and above every border between two magnitudes."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    block = [6.0] + [m * f for m in mids for f in (1.0, 1.0 - 2 ** -7, 1.0 + 2 ** -7)] + [0.0, -0.0, 7.9, -6.0, 4.0, -4.99,
                                                                                        5.01, 0.5, 1.0, -3.0]
    return torch.tensor(block[:32], dtype=torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [True, False])
def test_quantise_borders_and_extremes(dtype, rows):
    from mixture_experts_layer_sort_amd import MoEMx4Tensor as Q
    one = borders()
    tiny, huge = 2.0 ** -126, 2.0 ** 120
    blocks = [one, -one, one * 2.0 ** 100, one * 2.0 ** -100, one * huge, torch.zeros(32), one * tiny, one * tiny / 4,
              one * tiny / 64, torch.full((32,), torch.finfo(dtype).max), torch.full((32,), -torch.finfo(dtype).max),
              torch.full((32,), tiny), torch.full((32,), tiny / 128)]
    for bad in (float("nan"), float("inf"), -float("inf")):
        b = one.clone()
        b[17] = bad
        blocks.append(b)
    lonely = torch.zeros(32)
    lonely[31] = -1e-30
    blocks += [lonely, one * 3.0, one / 3.0, one]
    flat = torch.cat(blocks).to(dtype)          # 20 blocks = 640 values
    assert flat.numel() == 640
    if rows:
        v = torch.stack([flat, flat.flip(0), -flat]).cuda().contiguous()
    else:
        v = torch.stack([flat.roll(32 * i) for i in range(128)], 1)[None].cuda().contiguous()
    q = Q.rows(v) if rows else Q.weights(v)
    want, e = quantised(v)
    got = q.dequantize(torch.float32).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    # the values below 2^-126 may have become 0
    ok = torch.isnan(want) | (got == want) | ((want.abs() < 2.0 ** -126) & (got == 0))
    assert bool(ok.all())
    # scale bytes, where the documentation puts them
    if rows:
        s = q.scales.reshape(3, 2, 4, 4)        # [row][group][g][kt]
        byte = s.permute(0, 1, 3, 2).reshape(3, 32)
        assert torch.equal(byte[:, :20].double(), e[:, :, 0, 0] + 127) and int(byte[:, 20:].max()) == 0
    else:
        s = q.scales.reshape(8, 2, 4, 16, 4)    # [strip][group][g][column][kt]
        byte = s.permute(0, 3, 1, 4, 2).reshape(128, 32)
        assert torch.equal(byte[:, :20].double(), (e[0, :, 0, :] + 127).t()) and int(byte[:, 20:].max()) == 0


def test_codes_lie_where_the_documentation_says():
    from mixture_experts_layer_sort_amd import MoEMx4Tensor as Q
    # value (code) number (k + 3 * column) % 8, the largest in each block 6
    k, c = torch.arange(256), torch.arange(128)
    code = (k[:, None] + 3 * c[None]) % 8
    v = GRID[code].float()[None].cuda()
    q = Q.weights(v)
    byte = q.codes.reshape(8, 2, 4, 16, 16).cpu()   # [strip][tile][g][column][byte]
    for kk, cc in ((0, 0), (1, 0), (31, 5), (32, 17), (127, 127), (128, 64), (255, 126), (200, 33)):
        b = int(byte[cc // 16, kk // 128, kk % 128 // 32, cc % 16, kk % 32 // 2])
        assert (b >> 4 * (kk % 2)) & 15 == int(code[kk, cc]), (kk, cc)
    r = Q.rows(v[0].t().contiguous())
    byte = r.codes.reshape(128, 128).cpu()
    for kk, cc in ((0, 0), (1, 9), (130, 77), (255, 127)):
        assert (int(byte[cc, kk // 2]) >> 4 * (kk % 2)) & 15 == int(code[kk, cc])


def test_quantise_refusals_and_empty():
    from mixture_experts_layer_sort_amd import MoEError, MoEMx4Tensor as Q
    from mixture_experts_layer_sort_amd import _lib as L
    for shape in ((1, 100, 128), (1, 128, 100), (2, 96)):
        with pytest.raises(ValueError):
            (Q.rows if len(shape) == 2 else Q.weights)(randn(0, *shape))
    with pytest.raises(ValueError):
        Q.rows(randn(0, 2, 128).half())
    with pytest.raises(ValueError):
        Q.rows(randn(0, 128, 4).t())
    q = Q.rows(randn(0, 4, 128))
    for bad in (randn(0, 5, 128), randn(0, 4, 256)):
        with pytest.raises(ValueError):
            q.quantize(bad)
        with pytest.raises(ValueError):
            q.dequantize(out=bad)
    with pytest.raises(MoEError):
        q.quantize(randn(0, 4 * 128 + 1)[1:].view(4, 128))  # not aligned to 16 bytes
    assert Q.rows(randn(0, 0, 128)).dequantize().shape == (0, 128)
    assert Q.weights(randn(0, 0, 128, 128)).dequantize().shape == (0, 128, 128)
    assert Q.weights(randn(0, 128, 256)).shape == (1, 128, 256) and q.order == L.MOE_MX4_ROWS


def test_quantise_past_4_gib():
    """Offsets of a tensor longer than 32 bits: the last rows of 4.5 GiB of bf16 weights."""
    from mixture_experts_layer_sort_amd import MoEMx4Tensor as Q
    w = torch.zeros((9, 16384, 16384), dtype=torch.bfloat16, device="cuda")
    w[8] = randn(3, 16384, 16384, dtype=torch.bfloat16)
    q = Q.weights(w)
    del w
    got = q.dequantize(torch.bfloat16)
    assert int(torch.count_nonzero(got[:8])) == 0
    v = randn(3, 16384, 16384, dtype=torch.bfloat16)
    for part in (slice(0, 128), slice(16256, 16384)):
        want, _ = quantised(v[None, part, :512])
        assert torch.equal(got[8, part, :512].double(), want[0])
        want, _ = quantised(v[None, part, -256:])
        assert torch.equal(got[8, part, -256:].double(), want[0])


# ------------------------------------------------------------ the products


def ffn_parts(x, wg, wu):
    """silu(G) * U of float64 rows and weights, and the error bound of its float32 evaluation."""
    H = x.shape[1]
    G, Uu = x @ wg, x @ wu
    eG, eU = (H + 8) * U * (x.abs() @ wg.abs()), (H + 8) * U * (x.abs() @ wu.abs())
    silu = G * torch.sigmoid(G)
    A = silu * Uu
    return A, 1.1 * Uu.abs() * eG + silu.abs() * eU + 8 * U * A.abs()


def choice(seed, N, E, K, counts=None):
    """topk [N, K]: random, or (K = 1) the given rows per expert."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if counts is not None:
        flat = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
        return flat[torch.randperm(N, generator=g, device="cuda")].to(torch.int32)[:, None].contiguous()
    pull = torch.randn((N, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    return torch.topk(pull, K, dim=1)[1].to(torch.int32).contiguous()


# N, H, F, E, K, rows per expert
PRODUCTS = [(1, 128, 128, 1, 1, None), (3, 128, 256, 2, 2, None), (65, 256, 128, 5, 3, None),
            (70, 640, 384, 64, 8, None), (257, 512, 640, 1, 1, None), (300, 1408, 256, 3, 2, None),
            (513, 384, 512, 4, 1, [0, 256, 1, 256]), (400, 128, 1408, 4, 1, [17, 0, 383, 0]),
            (1000, 256, 256, 256, 8, None), (2100, 896, 384, 6, 4, None), (700, 2048, 256, 2, 1, [699, 1]),
            (500, 256, 384, 8, 1, [300, 1, 128, 71, 0, 0, 0, 0])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,F,E,K,counts", PRODUCTS)
def test_products(dtype, N, H, F, E, K, counts):
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    s = 2.0 ** -8 if dtype == torch.bfloat16 else U
    topk = choice(N, N, E, K, counts)
    r = MoEMx4Runner(N, H, F, E, K, dtype)
    r.meta(topk)
    x, a = randn(1, N, H, dtype=dtype), randn(2, N * K, F, dtype=dtype)
    wg, wu = (randn(i, E, H, F, dtype=dtype, scale=H ** -0.5) for i in (3, 4))
    wd = randn(5, E, F, H, dtype=dtype, scale=F ** -0.5)
    xq, aq = Q.rows(x), Q.rows(a)
    qg, qu, qd = Q.weights(wg), Q.weights(wu), Q.weights(wd)
    act = r.gate_up(xq, qg, qu).clone()
    ys = r.down(aq, qd).clone()
    xv, av, gv, uv, dv = (quantised(t)[0] for t in (x, a, wg, wu, wd))
    flat = topk.reshape(-1)
    at = 0
    for e in range(E):
        rows = torch.nonzero(flat == e)[:, 0]
        n = rows.numel()
        if n == 0:
            continue
        A, eA = ffn_parts(xv[rows // K], gv[e], uv[e])
        got = act[at:at + n].double()
        assert bool(((got - A).abs() <= s * A.abs() + 1.01 * eA).all()), f"act of expert {e}"
        y = av[at:at + n] @ dv[e]
        ey = (F + 8) * U * (av[at:at + n].abs() @ dv[e].abs())
        got = ys[at:at + n].double()
        assert bool(((got - y).abs() <= s * y.abs() + 1.01 * ey).all()), f"ys of expert {e}"
        at += n
    assert at == N * K
    assert torch.equal(r.gate_up(xq, qg, qu), act) and torch.equal(r.down(aq, qd), ys)  # bit for bit


def test_gathered_rows_past_2_gib():
    """The last of 400000 tokens of 16384 values, their codes 3 GiB from the first, as in a tensor of their own."""
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, last = 400000, 16384, 128, 333
    w = Q.weights(randn(1, 1, H, F, scale=H ** -0.5)), Q.weights(randn(2, 1, H, F, scale=H ** -0.5))
    some = Q.rows(randn(3, last, H))
    many = Q(some.order, (N, H), "cuda")
    many.codes.zero_()
    many.scales.fill_(127)
    many.codes.view(N, -1)[-last:] = some.codes.view(last, -1)
    many.scales.view(N, -1)[-last:] = some.scales.view(last, -1)
    out = []
    for q, n in ((many, N), (some, last)):
        r = MoEMx4Runner(n, H, F, 1, 1, torch.bfloat16)
        r.meta(torch.zeros((n, 1), dtype=torch.int32, device="cuda"))
        out.append(r.gate_up(q, *w)[-last:])
    assert bool(out[1].any()) and torch.equal(*out)


def test_products_leave_dropped_rows():
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 200, 256, 256, 3, 2
    r = MoEMx4Runner(N, H, F, E, K, torch.bfloat16, capacity=50)
    r.meta(choice(1, N, E, K))
    kept = int(r.offsets[-1])
    assert kept <= 150
    xq = Q.rows(randn(1, N, H, dtype=torch.bfloat16))
    w = [Q.weights(randn(i, E, H, F, dtype=torch.bfloat16)) for i in (2, 3, 4)]
    r.act.fill_(7.0)
    r.ys.fill_(9.0)
    r.gate_up(xq, w[0], w[1])
    assert bool((r.act[kept:] == 7.0).all()) and not bool((r.act[:kept] == 7.0).all())
    r.down(Q.rows(r.act), w[2])
    assert bool((r.ys[kept:] == 9.0).all())


def test_nan_rows_and_experts_stay_where_they_are():
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 90, 256, 256, 4, 1
    topk = choice(2, N, E, K)
    r = MoEMx4Runner(N, H, F, E, K, torch.float32)
    r.meta(topk)
    x = randn(1, N, H)
    wg, wu = randn(2, E, H, F), randn(3, E, H, F)
    clean = r.gate_up(Q.rows(x), Q.weights(wg), Q.weights(wu)).clone()
    x[5, 100] = float("nan")
    wg[2, 40, 30] = float("inf")
    got = r.gate_up(Q.rows(x), Q.weights(wg), Q.weights(wu))
    hurt = torch.zeros((N, F), dtype=torch.bool, device="cuda")
    hurt[r.inv[5].long()] = True
    mine = r.sorted_flat.long()
    hurt[topk.reshape(-1)[mine] == 2, 30] = True
    assert bool(torch.isnan(got[hurt]).all()) and torch.equal(got[~hurt], clean[~hurt])


def layer_reference(t, wv, K, split, s, shared=None):
    """topk, gates, y and y's error bound of the layer, from float64 weights."""
    x = t["x"].double()
    l = x @ t["w_r"].double()
    if t["bias"] is not None:
        l = l + t["bias"].double()
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    gates = torch.softmax(top, 1)
    ge = (16 + (top[:, :1] - top).max().item()) * U
    y = torch.zeros_like(x)
    e = torch.zeros_like(x)

    def one(rows, wg, wu, wd):
        A, eA = ffn_parts(rows, wg, wu)
        eA = eA + split * A.abs()
        return A @ wd, (eA + (wd.shape[0] + 16) * U * A.abs()) @ wd.abs()

    for ex in range(t["w_r"].shape[1]):
        n, k = torch.nonzero(ids == ex, as_tuple=True)
        if n.numel():
            o, eo = one(x[n], wv[0][ex], wv[1][ex], wv[2][ex])
            y[n] += gates[n, k, None] * o
            e[n] += gates[n, k, None] * (eo + (ge + 8 * U) * o.abs())
    if shared is not None:
        o, eo = one(x, shared[0][0], shared[1][0], shared[2][0])
        y += o
        e += eo + 4 * U * o.abs()
    return ids, gates, ge, y, e


def layer_inputs(N, H, F, E, dtype, Fs=0, bias=False, seed=0):
    t = dict(x=randn(seed + 1, N, H, dtype=dtype), w_r=randn(seed + 2, H, E, dtype=dtype, scale=0.05),
             bias=randn(seed + 3, E, scale=0.3) if bias else None)
    w = [randn(seed + 4, E, H, F, dtype=dtype, scale=H ** -0.5), randn(seed + 5, E, H, F, dtype=dtype, scale=H ** -0.5),
         randn(seed + 6, E, F, H, dtype=dtype, scale=F ** -0.5)]
    sh = [randn(seed + 7, 1, H, Fs, dtype=dtype, scale=H ** -0.5), randn(seed + 8, 1, H, Fs, dtype=dtype, scale=H ** -0.5),
          randn(seed + 9, 1, Fs, H, dtype=dtype, scale=Fs ** -0.5)] if Fs else None
    return t, w, sh


# N, H, F, E, K, Fs, bias
DECODE = [(1, 128, 128, 1, 1, 0, False), (1, 512, 1024, 8, 2, 0, False), (1, 640, 384, 6, 3, 256, True),
          (1, 1408, 256, 256, 8, 128, False), (2, 128, 256, 3, 3, 0, False), (5, 256, 128, 256, 8, 0, True),
          (13, 512, 640, 64, 6, 896, True), (16, 384, 512, 4, 1, 0, False), (17, 256, 384, 2, 2, 128, False),
          (24, 640, 256, 1, 1, 0, False), (33, 256, 256, 3, 2, 0, True), (48, 128, 640, 8, 2, 256, False),
          (64, 512, 384, 8, 2, 0, False), (64, 384, 256, 1, 1, 512, False), (64, 256, 256, 200, 8, 0, False),
          (40, 128, 2176, 2, 1, 0, False), (20, 128, 4096, 4, 2, 1152, False), (9, 128, 4352, 2, 1, 128, True),
          (2, 256, 6144, 3, 2, 0, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,F,E,K,Fs,bias", DECODE)
def test_decode(dtype, N, H, F, E, K, Fs, bias):
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    s, split = (2.0 ** -8, 2.0 ** -16) if dtype == torch.bfloat16 else (U, 0.0)
    t, w, sh = layer_inputs(N, H, F, E, dtype, Fs, bias)
    r = MoEMx4DecodeRunner(N, H, F, E, K, dtype, shared_ffn=Fs or None)
    q = [Q.weights(v) for v in w]
    qs = tuple(Q.weights(v) for v in sh) if sh else None
    y = r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs).clone()
    ids, gates, ge, ref, e = layer_reference(t, [quantised(v)[0] for v in w], K, split, s,
                                             [quantised(v)[0] for v in sh] if sh else None)
    assert torch.equal(r.topk.long(), ids)
    assert bool(((r.gates.double() - gates).abs() <= ge * gates).all())
    err, tol = (y.double() - ref).abs(), s * ref.abs() + 1.01 * e
    assert bool((err <= tol).all()), float((err / tol).max())
    if dtype == torch.bfloat16:
        # a y rounded once: 1.66e-3 of its own root mean square; 2.3e-3 with activations in bf16
        rms = float(((y.double() - ref) ** 2).mean().sqrt() / (ref ** 2).mean().sqrt())
        assert rms < 2e-3 + (0.0 if y.numel() >= 4096 else 1e-3)
    r.y.zero_()
    assert torch.equal(r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs), y)  # bit for bit


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_any_number_of_tokens(dtype):
    """One runner, every number of tokens from 0 to 64, rows behind the last one left alone."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    H, F, E, K = 256, 384, 5, 2
    s, split = (2.0 ** -8, 2.0 ** -16) if dtype == torch.bfloat16 else (U, 0.0)
    t, w, _ = layer_inputs(64, H, F, E, dtype)
    r = MoEMx4DecodeRunner(64, H, F, E, K, dtype)
    q = [Q.weights(v) for v in w]
    ids, gates, ge, ref, e = layer_reference(t, [quantised(v)[0] for v in w], K, split, s)
    for n in range(65):
        r._y.fill_(5.0)
        y = r.forward(t["x"][:n].contiguous(), t["w_r"], *q)
        assert y.shape == (n, H) and bool((r._y[n:] == 5.0).all())
        assert torch.equal(r.topk.long(), ids[:n])
        assert bool(((y.double() - ref[:n]).abs() <= s * ref[:n].abs() + 1.01 * e[:n]).all()), n


def test_decode_nan_and_infinite_values():
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    N, H, F, E, K = 12, 256, 256, 6, 2
    t, w, _ = layer_inputs(N, H, F, E, torch.bfloat16)
    r = MoEMx4DecodeRunner(N, H, F, E, K, torch.bfloat16)
    clean = r.forward(t["x"], t["w_r"], *(Q.weights(v) for v in w)).clone()
    topk = r.topk.clone()
    w[0][2, 17, 3] = float("nan")
    w[2][4, 200, 9] = float("inf")
    got = r.forward(t["x"], t["w_r"], *(Q.weights(v) for v in w))
    two, four = (topk == 2).any(1), (topk == 4).any(1)
    assert 0 < int(two.sum()) < N and 0 < int(four.sum()) < N
    assert bool(torch.isnan(got[two]).all())
    assert bool(torch.isnan(got[four, 9]).all())
    spared = ~two
    rest = torch.ones(H, dtype=torch.bool, device="cuda")
    rest[9] = False
    assert torch.equal(got[spared][:, rest], clean[spared][:, rest])
    assert torch.equal(got[~two & ~four], clean[~two & ~four])
    # a token's own NaN
    t, w, _ = layer_inputs(N, H, F, E, torch.bfloat16)
    q = [Q.weights(v) for v in w]
    t["x"][3, 7] = float("nan")
    got = r.forward(t["x"], t["w_r"], *q)
    others = torch.arange(N, device="cuda") != 3
    assert bool(torch.isnan(got[3]).all()) and torch.equal(got[others], clean[others])


def test_decode_refusals_change_nothing():
    from mixture_experts_layer_sort_amd import MoEError, MoEMx4DecodeRunner, MoEMx4Tensor as Q
    H, F, E, K = 128, 256, 4, 2
    t, w, sh = layer_inputs(8, H, F, E, torch.bfloat16, 128)
    q = [Q.weights(v) for v in w]
    r = MoEMx4DecodeRunner(8, H, F, E, K, torch.bfloat16)
    y = r.forward(t["x"], t["w_r"], *q).clone()
    qs = tuple(Q.weights(v) for v in sh)
    for args, kw in (((t["x"], t["w_r"], q[0], q[1], q[0]), {}), ((t["x"], t["w_r"], w[0], q[1], q[2]), {}),
                     ((t["x"].float(), t["w_r"], *q), {}), ((t["x"], t["w_r"], *q), dict(shared=qs)),
                     ((t["x"], t["w_r"], *q), dict(bias=t["x"][0, :4])),
                     ((torch.cat([t["x"], t["x"]]), t["w_r"], *q), {})):
        with pytest.raises(ValueError):
            r.forward(*args, **kw)
    with pytest.raises(MoEError):
        r.forward(r.y, t["w_r"], *q)            # x on y
    assert torch.equal(r.y, y)
    with pytest.raises(MoEError):
        MoEMx4DecodeRunner(65, H, F, E, K, torch.bfloat16)


def test_layer_over_many_and_few_tokens():
    """One set of quantised weights through both runners, as a server uses them: a prompt, then its
    next tokens.  The prompt's path quantises rows as well: against float64 on the values that it had."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 333, 256, 512, 6, 2
    t, w, _ = layer_inputs(N, H, F, E, torch.bfloat16, bias=True)
    q = [Q.weights(v) for v in w]
    r = MoEMx4Runner(N, H, F, E, K, torch.bfloat16)
    y = r.forward(t["x"], t["w_r"], *q, bias=t["bias"])
    wv = [quantised(v)[0] for v in w]
    xv, av = quantised(t["x"])[0], quantised(r.act)[0]
    s = 2.0 ** -8
    ref, tol = torch.zeros((N, H), dtype=torch.float64, device="cuda"), torch.zeros((N, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = int(r.offsets[e]), int(r.offsets[e + 1])
        f = r.sorted_flat[lo:hi].long()
        A, eA = ffn_parts(xv[f // K], wv[0][e], wv[1][e])
        assert bool(((r.act[lo:hi].double() - A).abs() <= s * A.abs() + 1.01 * eA).all())
        o = av[lo:hi] @ wv[2][e]
        eo = (F + 8) * U * (av[lo:hi].abs() @ wv[2][e].abs()) + s * o.abs()
        g = r.gates.reshape(-1)[f].double()[:, None]
        ref.index_add_(0, f // K, g * o)
        tol.index_add_(0, f // K, g * (eo + 8 * U * o.abs()))
    assert bool(((y.double() - ref).abs() <= s * ref.abs() + 1.01 * tol).all())
    few = MoEMx4DecodeRunner(16, H, F, E, K, torch.bfloat16)
    z = few.forward(t["x"][:16].contiguous(), t["w_r"], *q, bias=t["bias"])
    assert torch.equal(few.topk, r.topk[:16])
    # rows in 4 bits as well: each block's values are off by an eighth of its largest at most, a quarter where
    # that is cut off at 6; the two agree to what that leaves of independent errors
    cos = torch.nn.functional.cosine_similarity(z.float(), y[:16].float(), dim=1)
    assert float(cos.min()) > 0.9


def test_no_tokens():
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    t, w, _ = layer_inputs(1, 128, 128, 4, torch.bfloat16)
    r = MoEMx4Runner(0, 128, 128, 4, 2, torch.bfloat16)
    q = [Q.weights(v) for v in w]
    assert r.forward(t["x"][:0], t["w_r"], *q).shape == (0, 128)
    r.meta(torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert r.gate_up(Q.rows(t["x"][:0]), q[0], q[1]).shape == (0, 128)
    assert r.down(Q.rows(t["x"][:0]), q[2]).shape == (0, 128)


def test_on_another_stream_and_captured():
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor as Q
    H, F, E, K = 256, 384, 6, 2
    t, w, _ = layer_inputs(100, H, F, E, torch.bfloat16)
    q = [Q.weights(v) for v in w]
    many, few = MoEMx4Runner(100, H, F, E, K, torch.bfloat16), MoEMx4DecodeRunner(16, H, F, E, K, torch.bfloat16)
    x16 = t["x"][:16].contiguous()

    def both():
        return many.forward(t["x"], t["w_r"], *q), few.forward(x16, t["w_r"], *q)

    want = [v.clone() for v in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    many.y.zero_()
    few.y.zero_()
    torch.cuda.synchronize()
    y = many.forward(t["x"], t["w_r"], *q, stream=side)
    z = few.forward(x16, t["w_r"], *q, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    keep = t["x"].clone(), x16.clone()
    for i in range(4):
        scale = 1.0 if i % 2 == 0 else 0.5
        t["x"].copy_(keep[0] * scale)
        x16.copy_(keep[1] * scale)
        eager = [v.clone() for v in both()]
        many.y.zero_()
        few.y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(many.y, eager[0]) and torch.equal(few.y, eager[1])
        if scale == 1.0:
            assert torch.equal(many.y, want[0]) and torch.equal(few.y, want[1])


def test_two_streams_at_once():
    """Runners of their own on two streams, sharing the weights: the results of one after the other."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor as Q
    H, F, E, K = 512, 4096, 4, 2
    t, w, _ = layer_inputs(700, H, F, E, torch.bfloat16)
    q = [Q.weights(v) for v in w]
    x = [t["x"][:20].contiguous(), t["x"][20:40].contiguous()]
    few = [MoEMx4DecodeRunner(20, H, F, E, K, torch.bfloat16) for _ in x]
    many = MoEMx4Runner(700, H, F, E, K, torch.bfloat16)
    want = [r.forward(v, t["w_r"], *q).clone() for r, v in zip(few, x)] + [many.forward(t["x"], t["w_r"], *q).clone()]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, v, s in zip(few, x, streams):
            r.forward(v, t["w_r"], *q, stream=s)
        many.forward(t["x"], t["w_r"], *q, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(r.y, y) for r, y in zip(few + [many], want))


def test_the_same_expert_twice():
    """A given choice that names an expert twice for a token: two rows of it."""
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F = 37, 256, 128
    x = randn(1, N, H, dtype=torch.bfloat16)
    q = Q.weights(randn(2, 3, H, F, scale=H ** -0.5)), Q.weights(randn(3, 3, H, F, scale=H ** -0.5))
    r = MoEMx4Runner(N, H, F, 3, 2, torch.bfloat16)
    one = torch.arange(N, dtype=torch.int32, device="cuda")[:, None] % 3
    r.meta(one.expand(N, 2).contiguous())
    act = r.gate_up(Q.rows(x), *q)
    assert torch.equal(r.counts.cpu(), 2 * torch.bincount(one.cpu()[:, 0], minlength=3).int())
    i = r.inv.view(N, 2).long()
    assert torch.equal(act[i[:, 0]], act[i[:, 1]])
    s = MoEMx4Runner(N, H, F, 3, 1, torch.bfloat16)
    s.meta(one.contiguous())
    assert torch.equal(act[i[:, 0]], s.gate_up(Q.rows(x), *q)[s.inv.long()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,F,E", [(1, 128, 1), (3, 256, 2), (16, 128, 1), (24, 256, 2), (40, 384, 1), (64, 128, 2),
                                   (16, 6528, 8), (24, 6528, 8), (64, 6656, 8)])
def test_decode_activations_keep_24_bits(dtype, N, F, E):
    """Tokens with one nonzero value, so that G and U are single exact products.  Neighbouring hidden columns have
    the same G, and U of 3 : 1 (times powers of two), so their activations are as 3 : 1 too; each column of W_down
    weighs one such pair with 1 : -3, so that the sum is 0 but for the activations' own errors: 8 u of each, and
    4 u of the sum's.  |y| <= 12 u |A|.|W_down|.  All E experts are chosen with gates of 1/E (exact); all but one
    have a W_down of 0.  Activations of 16 bits are off by up to 2^-18 of themselves: five times that bound."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    g = torch.Generator()
    g.manual_seed(N + F)
    H, e, P = 128, E // 2, F // 2
    pick = lambda n, *shape: torch.randint(n, shape, generator=g)  # noqa: E731
    x, wr = torch.zeros(N, H), torch.zeros(H, E)
    x[:, 77] = (0.5 + 1.5 * torch.rand(N, generator=g)).bfloat16().float()
    wg, wu, wd = torch.zeros(E, H, F), torch.zeros(E, H, F), torch.zeros(E, F, H)
    same = GRID.float()[1 + pick(7, E, P)] * torch.exp2(-pick(4, E, P).float())
    wg[:, 77] = same.repeat_interleave(2, 1)
    i, j = pick(2, E, P).float(), pick(2, E, P).float()
    wu[:, 77, 0::2], wu[:, 77, 1::2] = 3 * torch.exp2(i), torch.exp2(j)
    pair, h = pick(P, H), torch.arange(H)
    wd[e, 2 * pair, h], wd[e, 2 * pair + 1, h] = torch.exp2(j - i)[e, pair], -3.0
    for w in (wg, wu, wd):
        assert torch.equal(quantised(w)[0], w.double())  # exact in 4 bits
    G, Uu = x.double()[:, 77:78] * wg[e, 77].double(), x.double()[:, 77:78] * wu[e, 77].double()
    A = G * torch.sigmoid(G) * Uu / E
    ref, bound = A @ wd[e].double(), 12 * U * (A.abs() @ wd[e].double().abs())
    assert bool((ref.abs() <= 2.0 ** -48 * bound / U).all())
    r = MoEMx4DecodeRunner(N, H, F, E, E, dtype)
    y = r.forward(x.cuda().to(dtype), wr.cuda().to(dtype), *(Q.weights(w.cuda()) for w in (wg, wu, wd)))
    s = 2.0 ** -8 if dtype == torch.bfloat16 else U
    worst = float(((y.cpu().double() - ref).abs() / ((1 + s) * 1.01 * bound)).max())
    print(f"[mx4 decode] worst err/tol {worst:.3f}", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 5, 24])
def test_decode_silu_far_below_zero(dtype, N):
    """G around -88, where 1 + exp(-G) is past 2^126 and silu(G) a normal 1e-36.  exp(G) below 2^-126 comes in steps
    of 2^-149, at -88.2 half of one is 2^-22 of it; 16 u of an activation and its gate, F + 16 of the sum, all of whose
    terms are equal: |y - ref| <= (s + 2^-21 + (F + 32) u) |ref|."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    H = F = 128
    x, wr = torch.zeros(N, H), torch.zeros(H, 1)
    x[:, 3] = torch.tensor([14.5625, 14.625, 14.6875])[torch.arange(N) % 3]
    wg, wu, wd = torch.zeros(1, H, F), torch.zeros(1, H, F), torch.zeros(1, F, H)
    wg[:, 3], wu[:, 3] = -6.0, 2.0 ** 20
    wd[:] = 2.0 ** 60
    G, Uu = x.double()[:, 3:4] * -6.0, x.double()[:, 3:4] * 2.0 ** 20
    assert bool((G < -87.35).all()) and bool((G > -88.2).all())
    ref = (G * torch.sigmoid(G) * Uu * F * 2.0 ** 60).expand(N, H)
    r = MoEMx4DecodeRunner(N, H, F, 1, 1, dtype)
    y = r.forward(x.cuda().to(dtype), wr.cuda().to(dtype), *(Q.weights(w.cuda()) for w in (wg, wu, wd))).cpu().double()
    s = 2.0 ** -8 if dtype == torch.bfloat16 else U
    worst = float(((y - ref).abs() / ((s + 2.0 ** -21 + (F + 32) * U) * ref.abs())).max())
    print(f"[mx4 decode] worst err/tol {worst:.3f}", flush=True)
    assert worst <= 1.0


def _busy():
    """Work of some ten milliseconds on the current stream."""
    v = torch.zeros(1 << 28, device="cuda")
    for _ in range(40):
        v.add_(1.0)


@pytest.mark.parametrize("rows", [True, False])
def test_tensors_of_another_stream(rows):
    """4-bit tensors and their values, made on a side stream while the current one still works on memory that it has
    given back: the values of a call on one stream."""
    from mixture_experts_layer_sort_amd import MoEMx4Tensor as Q
    v = randn(1, 2048, 2048)
    make = Q.rows if rows else Q.weights
    plain = make(v)
    want = plain.dequantize()
    sizes = [plain.codes.numel(), plain.scales.numel(), 2 * want.numel()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55)
    q = make(v, stream=side)
    got = q.dequantize(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(q.codes, plain.codes) and torch.equal(q.scales, plain.scales) and torch.equal(got, want)
    q.record_stream(torch.cuda.current_stream())


def test_runners_of_another_stream():
    """Runners made behind work of the current stream and called on another one: what they hold of their making
    (zeros of rows that a capacity drops) comes before the call, not after it."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 600, 512, 512, 4, 2
    t, w, _ = layer_inputs(N, H, F, E, torch.bfloat16)
    q = [Q.weights(v) for v in w]
    x16 = t["x"][:16].contiguous()
    make = lambda: (MoEMx4Runner(N, H, F, E, K, torch.bfloat16, capacity=200),  # noqa: E731
                    MoEMx4DecodeRunner(16, H, F, E, K, torch.bfloat16))
    many, few = make()
    want = many.forward(t["x"], t["w_r"], *q).clone(), few.forward(x16, t["w_r"], *q).clone(), many.act.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    many, few = make()
    many.forward(t["x"], t["w_r"], *q, stream=side)
    few.forward(x16, t["w_r"], *q, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(many.y, want[0]) and torch.equal(few.y, want[1]) and torch.equal(many.act, want[2])


def prompt_check(r, y, t, wv, N, K, s, shared=None):
    """y of MoEMx4Runner.forward against float64, step by step on the values that each product had (its quantised
    activations, as the runner holds them); rows that a capacity dropped count nothing."""
    F, H = wv[2].shape[1:]
    xv, av = quantised(t["x"])[0], quantised(r.act)[0]
    ref, tol = torch.zeros((N, H), dtype=torch.float64, device="cuda"), torch.zeros((N, H), dtype=torch.float64, device="cuda")
    for e in range(wv[0].shape[0]):
        lo, hi = int(r.offsets[e]), int(r.offsets[e + 1])
        f = r.sorted_flat[lo:hi].long()
        A, eA = ffn_parts(xv[f // K], wv[0][e], wv[1][e])
        assert bool(((r.act[lo:hi].double() - A).abs() <= s * A.abs() + 1.01 * eA).all()), e
        o = av[lo:hi] @ wv[2][e]
        eo = (F + 8) * U * (av[lo:hi].abs() @ wv[2][e].abs()) + s * o.abs()
        g = r.gates.reshape(-1)[f].double()[:, None]
        ref.index_add_(0, f // K, g * o)
        tol.index_add_(0, f // K, g * (eo + 8 * U * o.abs()))
    if shared is not None:
        A, eA = ffn_parts(xv, shared[0][0], shared[1][0])
        assert bool(((r.act_s.double() - A).abs() <= s * A.abs() + 1.01 * eA).all())
        a, Fs = quantised(r.act_s)[0], shared[2].shape[1]
        o = a @ shared[2][0]
        ref += o
        tol += (Fs + 8) * U * (a.abs() @ shared[2][0].abs()) + s * o.abs() + 8 * U * o.abs()
    err, lim = (y.double() - ref).abs(), s * ref.abs() + 1.01 * tol
    assert bool((err <= lim).all()), float((err / lim).max())


# N, H, F, E, K, Fs, capacity, bias
PROMPTS = [(1, 128, 128, 1, 1, 0, None, False), (333, 256, 512, 6, 2, 0, None, True), (333, 256, 512, 6, 2, 384, None, True),
           (256, 128, 256, 3, 1, 128, None, False), (257, 384, 640, 5, 3, 1408, None, False),
           (700, 640, 384, 4, 2, 0, 100, False), (700, 256, 1408, 8, 2, 640, 60, True), (90, 128, 128, 4, 2, 0, 0, False),
           (90, 128, 128, 4, 2, 256, 0, False), (1500, 512, 256, 64, 8, 256, None, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,F,E,K,Fs,capacity,bias", PROMPTS)
def test_prompt(dtype, N, H, F, E, K, Fs, capacity, bias):
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor as Q
    s = 2.0 ** -8 if dtype == torch.bfloat16 else U
    t, w, sh = layer_inputs(N, H, F, E, dtype, Fs, bias)
    r = MoEMx4Runner(N, H, F, E, K, dtype, capacity=capacity, shared_ffn=Fs or None)
    q = [Q.weights(v) for v in w]
    qs = tuple(Q.weights(v) for v in sh) if sh else None
    y = r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs).clone()
    kept = int(r.offsets[-1])
    assert kept == N * K if capacity is None else kept <= min(N * K, E * capacity)
    prompt_check(r, y, t, [quantised(v)[0] for v in w], N, K, s, [quantised(v)[0] for v in sh] if sh else None)
    # the same bits again, with NaN in the rows that were dropped
    r.act[kept:] = float("nan")
    r.ys[kept:] = float("nan")
    r.y.zero_()
    assert torch.equal(r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs), y)
    few = MoEMx4DecodeRunner(1, H, F, E, K, dtype, shared_ffn=Fs or None)
    few.forward(t["x"][:1].contiguous(), t["w_r"], *q, bias=t["bias"], shared=qs)
    assert torch.equal(few.topk, r.topk[:1])


def test_prompt_refuses_shared_weights_that_do_not_fit():
    from mixture_experts_layer_sort_amd import MoEError, MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 20, 128, 256, 4, 2
    t, w, sh = layer_inputs(N, H, F, E, torch.bfloat16, 384)
    q, qs = [Q.weights(v) for v in w], tuple(Q.weights(v) for v in sh)
    r, plain = (MoEMx4Runner(N, H, F, E, K, torch.bfloat16, shared_ffn=Fs) for Fs in (384, None))
    y = r.forward(t["x"], t["w_r"], *q, shared=qs).clone()
    for run, bad in ((r, None), (plain, qs), (r, (qs[0], qs[1], qs[0])), (r, (q[0], q[1], q[2])), (r, sh)):
        with pytest.raises(ValueError):
            run.forward(t["x"], t["w_r"], *q, shared=bad)
    assert torch.equal(r.y, y)
    with pytest.raises(MoEError):
        MoEMx4Runner(N, H, F, E, K, torch.bfloat16, shared_ffn=100)
    none = MoEMx4Runner(0, H, F, E, K, torch.bfloat16, shared_ffn=384)
    assert none.forward(t["x"][:0], t["w_r"], *q, shared=qs).shape == (0, H)


# N, H, F, E, K, Fs, the expert that all tokens choose: strips of a piece 1, 2, 4 of gate/up and 1, 2, 4, 8 of down,
# for kernels of one, two and four row tiles (N up to 16; experts of up to 24 rows on average; more, or a shared expert)
PIECES = [(9, 1024, 128, 64, 8, 0, None), (16, 1024, 512, 16, 4, 256, None), (16, 1024, 1024, 24, 4, 0, None),
          (20, 1024, 640, 16, 2, 0, None), (30, 1024, 1152, 20, 2, 0, None), (48, 2048, 256, 24, 2, 0, None),
          (41, 512, 384, 16, 2, 0, 3), (64, 512, 384, 16, 2, 0, 15), (64, 1024, 1152, 20, 2, 0, 0),
          (33, 512, 384, 32, 2, 256, None), (64, 1024, 1024, 20, 3, 128, 7), (64, 2048, 128, 24, 2, 128, None),
          (40, 2048, 768, 24, 4, 256, None), (64, 1024, 2304, 8, 4, 0, None), (17, 256, 1152, 16, 8, 1152, 2),
          (10, 512, 1152, 24, 4, 0, None), (16, 512, 640, 20, 4, 0, None)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,F,E,K,Fs,all_to", PIECES)
def test_decode_pieces(dtype, N, H, F, E, K, Fs, all_to):
    """As test_decode, over the ways in which the work is cut; rows of an expert in two turns of 32 too."""
    from mixture_experts_layer_sort_amd import MoEMx4DecodeRunner, MoEMx4Tensor as Q
    s = 2.0 ** -8 if dtype == torch.bfloat16 else U
    t, w, sh = layer_inputs(N, H, F, E, dtype, Fs, all_to is not None, seed=N + E)
    if all_to is not None:
        t["bias"][all_to] += 3.0
    r = MoEMx4DecodeRunner(N, H, F, E, K, dtype, shared_ffn=Fs or None)
    q = [Q.weights(v) for v in w]
    qs = tuple(Q.weights(v) for v in sh) if sh else None
    y = r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs).clone()
    ids, gates, ge, ref, e = layer_reference(t, [quantised(v)[0] for v in w], K, 0.0, s,
                                             [quantised(v)[0] for v in sh] if sh else None)
    assert torch.equal(r.topk.long(), ids)
    if all_to is not None:
        assert int((ids == all_to).sum()) > (32 if N > 32 else 16)
    assert bool(((r.gates.double() - gates).abs() <= ge * gates).all())
    err, tol = (y.double() - ref).abs(), s * ref.abs() + 1.01 * e
    assert bool((err <= tol).all()), float((err / tol).max())
    r.y.zero_()
    assert torch.equal(r.forward(t["x"], t["w_r"], *q, bias=t["bias"], shared=qs), y)  # bit for bit


def test_prompt_with_a_shared_expert_on_another_stream_and_captured():
    """A runner whose first call is on a side stream, and one whose first call is captured: the same bits; products
    behind the capture alone, before any replay, have no tiles and write nothing."""
    from mixture_experts_layer_sort_amd import MoEMx4Runner, MoEMx4Tensor as Q
    N, H, F, E, K = 300, 256, 384, 6, 2
    t, w, sh = layer_inputs(N, H, F, E, torch.bfloat16, 256)
    q, qs = [Q.weights(v) for v in w], tuple(Q.weights(v) for v in sh)
    make = lambda: MoEMx4Runner(N, H, F, E, K, torch.bfloat16, shared_ffn=256)  # noqa: E731
    r = make()
    want, xq = r.forward(t["x"], t["w_r"], *q, shared=qs).clone(), Q.rows(t["x"])
    side, r = torch.cuda.Stream(), make()
    side.wait_stream(torch.cuda.current_stream())
    r.forward(t["x"], t["w_r"], *q, shared=qs, stream=side)
    side.synchronize()
    assert torch.equal(r.y, want)
    r, g = make(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.forward(t["x"], t["w_r"], *q, shared=qs)
    r.act.fill_(7.0)
    assert bool((r.gate_up(xq, q[0], q[1]) == 7.0).all())
    for _ in range(3):
        r.y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.y, want)
    r.y.zero_()
    assert torch.equal(r.forward(t["x"], t["w_r"], *q, shared=qs), want)

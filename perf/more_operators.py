"""Cases of the router's balance loss and of the layer's experts in microscaled 4-bit floating point, and their plain
forms.

Four operators are measured:
  quantize  a tensor in blocks of 32 values along its contraction axis, each value one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with
            a sign, each block with a power of two of its own: to codes and scales and back (MoEMx4Tensor); weights
            [E, K, C] along K, or token rows [N, K] along K;
  decode    the whole layer for the few tokens of a decoding step with 4-bit experts (MoEMx4DecodeRunner);
  product   one of the experts' grouped products over many tokens, both operands in 4 bits: gate/up with its
            SwiGLU, or down (MoEMx4Runner);
  balance   the load-balancing and z loss of the router's logits, per sequence, padding left out, with the counts of
            every expert and the gradient of the logits (MoEBalanceRunner).

With ``own`` false, run() evaluates them in elementary torch operations; with ``own`` true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32
ALPHA, ZETA = 0.01, 0.001


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one weight matrix of the benchmark's default layer
        dict(name="quantize_w_bf16_e8", op="quantize", rows=False, dtype="bf16", E=8, K=512, C=1024),
        # one weight matrix of the 64-expert layer, from the float32 copy that its optimiser keeps
        dict(name="quantize_w_f32_e64", op="quantize", rows=False, dtype="f32", E=64, K=2048, C=1408),
        # the token rows of a long prompt in front of the large-FFN layer
        dict(name="quantize_rows_bf16_n16384", op="quantize", rows=True, dtype="bf16", E=16384, K=4096, C=1),
        # one user's next token on the default layer: launches and latency are all there is
        dict(name="decode_bf16_n1_e8", op="decode", dtype="bf16", N=1, H=512, F=1024, E=8, K=2, Fs=0, bias=False),
        # a small ragged batch on the 64-expert layer, with a balancing bias and a shared expert of two experts' size
        dict(name="decode_bf16_n13_e64_shared", op="decode", dtype="bf16", N=13, H=2048, F=1408, E=64, K=6, Fs=2816,
             bias=True),
        # 32 users' next tokens on the wide-expert layer: most of 6 GB of 4-bit weights is touched
        dict(name="decode_bf16_n32_wide", op="decode", dtype="bf16", N=32, H=7168, F=2048, E=256, K=8, Fs=0,
             bias=False),
        # the fullest batch: every expert of the large-FFN layer has about 16 of the 64 tokens
        dict(name="decode_bf16_n64_large_ffn", op="decode", dtype="bf16", N=64, H=4096, F=14336, E=8, K=2, Fs=0,
             bias=False),
        # a long prompt through the large-FFN layer: its gate and up products
        dict(name="product_gate_up_bf16_n16384_large_ffn", op="product", part="gate_up", dtype="bf16", N=16384, H=4096,
             F=14336, E=8, K=2),
        # a short prompt on the 64-expert layer: about 95 rows an expert, every one another number
        dict(name="product_down_bf16_n1013_e64", op="product", part="down", dtype="bf16", N=1013, H=2048, F=1408, E=64,
             K=6),
        # a short float32 batch of the default layer
        dict(name="balance_f32_n203_e8", op="balance", dtype="f32", score="softmax", B=1, T=203, E=8, K=2, pad=False,
             choose=True),
        # a training step's tokens on the 64-expert layer, four padded sequences
        dict(name="balance_bf16_n16384_e64_sequences", op="balance", dtype="bf16", score="softmax", B=4, T=4096, E=64,
             K=6, pad=True, choose=False),
        # a large batch on the wide-expert layer, sigmoid scores
        dict(name="balance_f32_n131072_e256_sigmoid", op="balance", dtype="f32", score="sigmoid", B=32, T=4096, E=256,
             K=8, pad=False, choose=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any of the operators, sizes spread over the logarithm of their ranges."""
    op = rng.choice(["quantize", "decode", "product", "balance"])
    if op == "quantize":
        # contraction axes and columns are multiples of 128, as the layer has them; any number of rows
        K, rows = 128 * _log(rng, 1, 112), rng.random() < 0.5
        C = 1 if rows else 128 * _log(rng, 1, 112)
        return dict(op=op, rows=rows, dtype=rng.choice(["bf16", "f32"]), E=_log(rng, 1, max(1, min(20000, (1 << 27) // (K * C)))),
                    K=K, C=C)
    if op == "decode":
        # 1 to 64 tokens, 1 to 256 experts
        N, E = _log(rng, 1, 64), _log(rng, 1, 256)
        H = 128 * _log(rng, 1, 56)
        F = 128 * _log(rng, 1, max(1, min(112, (1 << 30) // (E * H * 128))))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), N=N, H=H, F=F, E=E, K=rng.randint(1, min(8, E)),
                    Fs=rng.choice([0, 0, 128 * _log(rng, 1, 32)]), bias=rng.random() < 0.5)
    if op == "product":
        # some tokens more than a decoding step has, to a long prompt
        E = _log(rng, 1, 256)
        K = rng.randint(1, min(8, E))
        H, N = 128 * _log(rng, 1, 32), _log(rng, 65, 16384 // K)
        F = 128 * _log(rng, 1, max(1, min(112, (1 << 28) // (E * H * 128))))
        return dict(op=op, part=rng.choice(["gate_up", "down"]), dtype=rng.choice(["bf16", "bf16", "f32"]), N=N, H=H,
                    F=F, E=E, K=K)
    E, B = _log(rng, 1, 256), _log(rng, 1, 64)
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), score=rng.choice(["softmax", "sigmoid"]), B=B,
                T=_log(rng, 1, 65536 // B), E=E, K=rng.randint(1, min(8, E)), pad=rng.random() < 0.5,
                choose=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _randn(gen, shape, scale=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return t if scale == 1.0 else t.mul_(scale)


def _weights(case):
    """Shapes of the quantised weights, and the scale of their values."""
    H, F, E = case["H"], case["F"], case["E"]
    if case["op"] == "product":
        return [("w_gate", (E, H, F)), ("w_up", (E, H, F))] if case["part"] == "gate_up" else [("w_down", (E, F, H))]
    shapes = [("w_gate", (E, H, F)), ("w_up", (E, H, F)), ("w_down", (E, F, H))]
    if case["Fs"]:
        shapes += [("s_gate", (1, H, case["Fs"])), ("s_up", (1, H, case["Fs"])), ("s_down", (1, case["Fs"], H))]
    return shapes


def _inputs(case, seed, keep):
    """The case's inputs; keep(w) makes of a weight tensor (or of token rows) what the caller keeps of it."""
    gen, op, dt = _generator(seed), case["op"], TYPES[case["dtype"]]
    if op == "quantize":
        shape = (case["E"], case["K"]) if case["rows"] else (case["E"], case["K"], case["C"])
        w = _randn(gen, shape, 1.0 if case["rows"] else case["K"] ** -0.5, dt)
        if case["rows"]:  # token rows: some tokens much larger than others, some channels too
            w.mul_(torch.exp(_randn(gen, (shape[0], 1))).to(dt)).mul_(torch.exp(_randn(gen, (1, shape[1]))).to(dt))
        return dict(w=w)
    if op == "balance":
        N, E, K = case["B"] * case["T"], case["E"], case["K"]
        logits = (_randn(gen, (N, E)) + _randn(gen, (1, E), 0.5)).to(dt)
        mask = None
        if case["pad"]:  # each sequence ends in padding; a sequence may be all padding but for one of them
            ends = torch.randint(case["T"] // 2, case["T"] + 1, (case["B"], 1), generator=gen, device="cuda")
            ends[0] = case["T"]
            mask = (torch.arange(case["T"], device="cuda") < ends).reshape(N)
        topk = None
        if not case["choose"]:  # the choice of a router with a balancing bias of its own
            moved = logits.double() + _randn(gen, (1, E), 0.3).double()
            topk = torch.sort(moved, dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
        return dict(logits=logits, mask=mask, topk=topk)
    N, H, F, E, K = (case[k] for k in ("N", "H", "F", "E", "K"))
    s = dict(bias=None)
    if op == "decode":
        s.update(x=_randn(gen, (N, H), 1.0, dt), w_r=_randn(gen, (H, E), 0.02, dt))
        if case["bias"]:
            s["bias"] = _randn(gen, (E,), 0.1)
    else:
        # a router's choice, some experts more popular than others
        pull = _randn(gen, (N, E)) + _randn(gen, (1, E), 0.3)
        s["topk"] = torch.sort(pull, dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
        width = H if case["part"] == "gate_up" else F
        s["x"] = keep(_randn(gen, (N if case["part"] == "gate_up" else N * K, width), 1.0, dt))
    for name, shape in _weights(case):
        s[name] = keep(_randn(gen, shape, shape[1] ** -0.5, torch.bfloat16 if dt == torch.bfloat16 else dt))
    return s


# ------------------------------------------------- the 4-bit form, plainly

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(v):
    """Codes (0 to 15, a byte each) and scale exponents + 127 (bytes) of v [..., blocks, 32, C], along the 32."""
    v = v.float()
    amax = v.abs().amax(-2, keepdim=True)
    e = torch.frexp(amax)[1] - 3                             # floor(log2 amax) - 2
    e = torch.where(amax == 0, -127, e).clamp(-127, 127)
    a = torch.ldexp(v, -e).abs()
    step = torch.ldexp(torch.full_like(a, 0.5), (torch.frexp(a)[1] - 1).clamp(0, 2))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)  # ties to even
    code = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, a + 2.0, 0.5 * a + 4.0))
    return (code + 8.0 * torch.signbit(v)).to(torch.uint8), (e + 127).to(torch.uint8)


def _dequantize(code, scale):
    code = code.int()
    sign = 1.0 - 2.0 * (code >> 3)
    code = (code & 7).float()
    a = torch.where(code < 4.0, 0.5 * code, torch.where(code < 6.0, code - 2.0, 2.0 * code - 8.0))
    return torch.ldexp(sign * a, scale.int() - 127)


def _blocks(v):
    """v [..., K] or [E, K, C] as [..., K/32, 32, C]."""
    return v.reshape(v.shape[0], -1, BLOCK, 1 if v.dim() == 2 else v.shape[2])


def _keep_plain(v):
    """Two codes a byte, as a checkpoint holds them, and the scales; a part of the tensor at a time."""
    parts = []
    for part in v.split(max(1, (1 << 26) // max(1, v[0].numel()))):
        code, scale = _quantize(_blocks(part))
        parts.append((code[:, :, 0::2] | code[:, :, 1::2] << 4, scale))
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _values(packed, scale, at=None):
    """float32 values [E, K, C] of kept weights (of the experts `at` alone) or [N, K] of kept rows."""
    if at is not None:
        packed, scale = packed[at], scale[at]
    code = torch.stack((packed & 15, packed >> 4), 3).reshape(*packed.shape[:2], BLOCK, packed.shape[3])
    v = _dequantize(code, scale).reshape(packed.shape[0], -1, packed.shape[3])
    return v[:, :, 0] if v.shape[2] == 1 else v


def prepare(case, seed):
    op = case["op"]
    if not own:
        s = _inputs(case, seed, _keep_plain)
        if op == "product":
            # how the rows lie, grouped by expert in the order of their tokens
            flat = s["topk"].reshape(-1).long()
            s["order"] = torch.sort(flat, stable=True)[1]
            s["counts"] = torch.bincount(flat, minlength=case["E"])
            s["most"] = int(s["counts"].max())
        return dict(s, case=case)
    from mixture_experts_layer_sort_amd import (MoEBalanceRunner, MoEMx4DecodeRunner, MoEMx4Runner, MoEMx4Tensor)
    s = _inputs(case, seed, lambda v: MoEMx4Tensor.rows(v) if v.dim() == 2 else MoEMx4Tensor.weights(v))
    dev, dt = torch.device("cuda"), TYPES[case["dtype"]]
    if op == "quantize":
        # the buffers of the quantised tensor and of its values
        s["q"] = (MoEMx4Tensor.rows if case["rows"] else MoEMx4Tensor.weights)(s["w"])
        s["out"] = torch.empty_like(s["w"])
    elif op == "decode":
        s["runner"] = MoEMx4DecodeRunner(case["N"], case["H"], case["F"], case["E"], case["K"], dt, dev,
                                         shared_ffn=case["Fs"] or None)
    elif op == "product":
        s["runner"] = MoEMx4Runner(case["N"], case["H"], case["F"], case["E"], case["K"], dt, dev)
        s["runner"].meta(s["topk"])
    else:
        s["runner"] = MoEBalanceRunner(case["B"] * case["T"], case["E"], case["K"], dt, dev, seq_len=case["T"],
                                       alpha=ALPHA, z_coef=ZETA, score=case["score"])
    return dict(s, case=case)


# -------------------------------------------------------------------- run


def _swiglu(g, u):
    return g * u / (1.0 + torch.exp(-g))


def _plain_quantize(s):
    w = s["w"]
    return _dequantize(*_quantize(_blocks(w))).reshape(w.shape).to(w.dtype)


def _plain_decode(s):
    x, K = s["x"], s["case"]["K"]
    logits = x.double() @ s["w_r"].double()          # 64 bits: the choice next to a border
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    z = torch.exp(top - top[:, :1])
    gates = (z / z.sum(1, keepdim=True)).float()
    used = torch.unique(ids)                         # only the experts that some token chose
    share = ((ids[:, :, None] == used) * gates[:, :, None]).sum(1)          # [N, used]
    xf = x.float()
    xe = xf.expand(used.numel(), *xf.shape)
    a = _swiglu(torch.bmm(xe, _values(*s["w_gate"], used)), torch.bmm(xe, _values(*s["w_up"], used)))
    y = (share.t()[:, :, None] * torch.bmm(a, _values(*s["w_down"], used))).sum(0)
    if s["case"]["Fs"]:
        y = y + _swiglu(xf @ _values(*s["s_gate"])[0], xf @ _values(*s["s_up"])[0]) @ _values(*s["s_down"])[0]
    return y.to(x.dtype), ids.to(torch.int32), gates


def _plain_product(s):
    case, counts, order = s["case"], s["counts"], s["order"]
    E, dt = case["E"], TYPES[case["dtype"]]
    x = _values(*s["x"])
    if case["part"] == "gate_up":
        x = x[order // case["K"]]
    # each expert's rows padded to the largest count, one batched product
    expert = torch.repeat_interleave(torch.arange(E, device=x.device), counts, output_size=x.shape[0])
    at = expert * s["most"] + torch.arange(x.shape[0], device=x.device) - (torch.cumsum(counts, 0) - counts)[expert]
    padded = torch.zeros((E * s["most"], x.shape[1]), device=x.device).index_copy_(0, at, x).reshape(E, s["most"], -1)
    if case["part"] == "gate_up":
        out = _swiglu(torch.bmm(padded, _values(*s["w_gate"])), torch.bmm(padded, _values(*s["w_up"])))
    else:
        out = torch.bmm(padded, _values(*s["w_down"]))
    return out.reshape(E * s["most"], -1)[at].to(dt)


def _plain_balance(s):
    case, l = s["case"], s["logits"].float()
    B, T, E, K = (case[k] for k in ("B", "T", "E", "K"))
    valid = torch.ones(B * T, device=l.device) if s["mask"] is None else s["mask"].float()
    topk = s["topk"]
    if topk is None:
        topk = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :K]
    hits = torch.zeros_like(l).scatter_(1, topk.long(), 1.0) * valid[:, None]
    top = l.amax(1, keepdim=True)
    z = torch.exp(l - top)
    total = z.sum(1, keepdim=True)
    soft, lse = z / total, (top + torch.log(total))[:, 0]
    if case["score"] == "softmax":
        p = soft
    else:
        sig = 1.0 / (1.0 + torch.exp(-l))
        p = sig / sig.sum(1, keepdim=True)
    n = valid.reshape(B, T).sum(1, keepdim=True)             # [B, 1]
    n_all = n.sum()
    hits = hits.reshape(B, T, E).sum(1)
    f = hits * (E / (K * n))
    P = (p * valid[:, None]).reshape(B, T, E).sum(1) / n
    loss = ALPHA / B * (f * P).sum() + ZETA / n_all * (lse * lse * valid).sum()
    fr = f.repeat_interleave(T, 0)
    c = (ALPHA / B / n).repeat_interleave(T, 0)
    d = c * p * (fr - (fr * p).sum(1, keepdim=True))
    if case["score"] == "sigmoid":
        d = d * (1.0 - sig)
    d = (d + 2.0 * ZETA / n_all * lse[:, None] * soft) * valid[:, None]
    return loss.reshape(1), hits.sum(0).to(torch.int32), d.to(s["logits"].dtype)


def _own_quantize(s):
    s["q"].quantize(s["w"])
    return s["q"].dequantize(out=s["out"])


def _own_decode(s):
    r = s["runner"]
    shared = (s["s_gate"], s["s_up"], s["s_down"]) if s["case"]["Fs"] else None
    y = r.forward(s["x"], s["w_r"], s["w_gate"], s["w_up"], s["w_down"], bias=s["bias"], shared=shared)
    return y, r.topk, r.gates


def _own_product(s):
    r = s["runner"]
    return r.gate_up(s["x"], s["w_gate"], s["w_up"]) if s["case"]["part"] == "gate_up" else r.down(s["x"], s["w_down"])


def _own_balance(s):
    r = s["runner"]
    loss = r.forward(s["logits"], topk=s["topk"], mask=s["mask"])
    return loss, r.counts, r.backward()


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quantize": _own_quantize, "decode": _own_decode, "product": _own_product,
                "balance": _own_balance}[op](state)
    return {"quantize": _plain_quantize, "decode": _plain_decode, "product": _plain_product,
            "balance": _plain_balance}[op](state)


# ------------------------------------------------------------------- work


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    q = 17.0 / 32.0                                  # bytes of a value in 4 bits with its part of a scale
    if case["op"] == "quantize":
        # the values read, the codes and scales written and read again, the values written
        n = case["E"] * case["K"] * case["C"]
        return {"bytes": n * (2.0 * es + 2.0 * q), "flops": 4.0 * n}
    if case["op"] == "balance":
        N, E, K = case["B"] * case["T"], case["E"], case["K"]
        ids = 0.0 if case["choose"] else 4.0 * N * K
        return {"bytes": 2.0 * N * E * es + ids + (N if case["pad"] else 0.0) + 4.0 * E + 4.0, "flops": 20.0 * N * E}
    N, H, F, E, K = (case[k] for k in ("N", "H", "F", "E", "K"))
    used = E * (1.0 - (1.0 - K / E) ** N)            # experts that N tokens choose, on average
    if case["op"] == "decode":
        Fs = case["Fs"]
        rows = used * 3 * H * F * q + 3 * H * Fs * q + H * E * es + 2 * N * H * es + 8 * N * K
        return {"bytes": rows, "flops": 6.0 * H * (N * K * F + N * Fs) + 2.0 * N * H * E}
    if case["part"] == "gate_up":
        return {"bytes": used * 2 * H * F * q + N * H * q + N * K * (F * es + 4.0), "flops": 4.0 * N * K * H * F}
    return {"bytes": used * H * F * q + N * K * (F * q + H * es), "flops": 2.0 * N * K * H * F}


# ------------------------------------------------------------------ exact


def _nearest(v):
    """v [E, K, C] or [N, K] as its 4-bit values, in 64 bits: the nearest magnitude by its borders, ties to the even code."""
    shape = v.shape
    v = _blocks(v).double()
    a = v.abs()
    top = a.amax(2, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2.0)
    a = a / unit
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=v.device)
    lower = torch.bucketize(a, grid, right=True).sub_(1).clamp_(0, 7)
    upper = (lower + 1).clamp_(max=7)
    below, above = a - grid[lower], grid[upper] - a
    pick = torch.where((above < below) | ((above == below) & (lower % 2 == 1)), upper, lower)
    return (torch.sign(v) * grid[pick] * unit).reshape(shape)


def _keep_exact(v):
    """The values, which bfloat16 holds exactly."""
    return torch.cat([_nearest(part).to(torch.bfloat16) for part in v.split(max(1, (1 << 25) // max(1, v[0].numel())))])


def _exact_ffn(rows, wg, wu, wd):
    rows = rows.double()
    g, u = rows @ wg.double(), rows @ wu.double()
    return (g * torch.sigmoid(g) * u) @ wd.double()


def exact(case, seed):
    s = _inputs(case, seed, _keep_exact)
    if case["op"] == "quantize":
        return _keep_exact(s["w"]).double()
    if case["op"] == "balance":
        B, T, E, K = (case[k] for k in ("B", "T", "E", "K"))
        l = s["logits"].double().requires_grad_()
        ids = s["topk"]
        if ids is None:
            ids = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)[1][:, :K]
        hits = torch.nn.functional.one_hot(ids.long(), E).sum(1)
        score = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        score = score / score.sum(1, keepdim=True)
        keep = torch.ones(B * T, dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"]
        loss = ZETA * torch.logsumexp(l[keep], 1).square().mean()
        for b in range(B):
            mine = keep[b * T:(b + 1) * T]
            share = hits[b * T:(b + 1) * T][mine].double().mean(0) * E / K
            loss = loss + ALPHA / B * (share * score[b * T:(b + 1) * T][mine].mean(0)).sum()
        grad, = torch.autograd.grad(loss, l)
        return loss.detach().reshape(1), hits[keep].sum(0).to(torch.int32), grad
    x, E, K = s["x"], case["E"], case["K"]
    if case["op"] == "product":
        flat = s["topk"].reshape(-1)
        rows = []
        for e in range(E):
            at = torch.nonzero(flat == e)[:, 0]
            if at.numel() == 0:
                continue
            if case["part"] == "gate_up":
                v = x[at // K].double()
                g = v @ s["w_gate"][e].double()
                rows.append(g * torch.sigmoid(g) * (v @ s["w_up"][e].double()))
            else:
                done = sum(r.shape[0] for r in rows)
                rows.append(x[done:done + at.numel()].double() @ s["w_down"][e].double())
        return torch.cat(rows)
    N = case["N"]
    l = x.double() @ s["w_r"].double()
    if s["bias"] is not None:
        l = l + s["bias"].double()
    # rank of expert e for a token: how many come before it (larger logit, or the same and a lower id)
    i = torch.arange(E, device=x.device)
    before = (l[:, None, :] > l[:, :, None]) | ((l[:, None, :] == l[:, :, None]) & (i[None, :] < i[:, None]))
    ids = torch.argsort(before.sum(2), dim=1)[:, :K]
    gates = torch.softmax(torch.gather(l, 1, ids), 1)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(E):
        n, k = torch.nonzero(ids == e, as_tuple=True)
        if n.numel():
            y[n] += gates[n, k, None] * _exact_ffn(x[n], s["w_gate"][e], s["w_up"][e], s["w_down"][e])
    if case["Fs"]:
        y += _exact_ffn(x, s["s_gate"][0], s["s_up"][0], s["s_down"][0])
    return y, ids.to(torch.int32), gates

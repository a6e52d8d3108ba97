"""Cases of the training operators around the NVFP4 linear layer: the gated feed-forward block
(forward, the gradient of its two projections, the whole backward pass), the distillation loss
against a teacher's top logits, and the embedding lookup with its gradient.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true,
through the package's calls; ``exact`` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

SILU, GELU = "silu", "gelu"


# ---- the cases ---------------------------------------------------------------
def listed():
    return [
        # one token of a served model: the weights are read once, latency counts
        dict(name="ffn one token", op="ffn", m=1, f=10240, k=5120, act=SILU, dtype="bf16"),
        # a decode batch of odd size
        dict(name="ffn batch of 45", op="ffn", m=45, f=10240, k=5120, act=GELU, dtype="bf16"),
        # a short ragged prompt through a smaller layer, kept in float32
        dict(name="ffn ragged f32", op="ffn", m=1003, f=2736, k=2112, act=GELU, dtype="f32"),
        # the 12B layer's tokens and weight tensor, the weight's rows shared by gate and up
        dict(name="ffn training", op="ffn", m=8192, f=10240, k=5120, act=SILU, dtype="bf16"),
        # its gradient: both pre-activation gradients, recomputed from the quantized operands
        dict(name="ffn_grad training", op="ffn_grad", m=8192, f=10240, k=5120, act=SILU, dtype="bf16"),
        # a ragged micro-batch
        dict(name="ffn_grad ragged f32", op="ffn_grad", m=515, f=2736, k=2048, act=GELU, dtype="f32"),
        # the block's whole backward pass, down to the gradients of its input and weights
        dict(name="ffn_backward", op="ffn_backward", m=4096, f=5120, k=2560, act=SILU, dtype="bf16"),
        # a few rows of a small vocabulary: latency
        dict(name="distill few rows", op="distill", t=8, v=32000, k=20, dtype="f32", mode="both", tau=1.0),
        # a ragged batch over an odd vocabulary, a tail of which is masked; loss alone (evaluation)
        dict(name="distill odd loss", op="distill", t=1000, v=50021, k=100, dtype="bf16", mode="loss", tau=2.0),
        # a training batch: loss and gradient of every row
        dict(name="distill training", op="distill", t=4096, v=131072, k=64, dtype="bf16", mode="both", tau=1.0),
        # the lookup of a training batch
        dict(name="embed training", op="embed", t=8192, v=131072, d=5120, dtype="bf16"),
        # and the gradient of its table, held in float32
        dict(name="embed_grad training", op="embed_grad", t=8192, v=131072, d=5120, dtype="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(step, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_backward", "distill", "distill", "embed", "embed_grad"])
    act, dtype = rng.choice([SILU, GELU]), rng.choice(["bf16", "bf16", "f32"])
    if op in ("ffn", "ffn_grad"):
        return dict(op=op, m=_log(rng, 1, 8192), f=_log(rng, 256, 10240, 16), k=_log(rng, 256, 5120, 64), act=act,
                    dtype=dtype)
    if op == "ffn_backward":  # its gradients come as the next layer's quantizer takes them
        return dict(op=op, m=_log(rng, 64, 4096, 16), f=_log(rng, 256, 5120, 16), k=_log(rng, 256, 2560, 64), act=act,
                    dtype="bf16")
    if op == "distill":
        return dict(op=op, t=_log(rng, 1, 4096), v=_log(rng, 1000, 131072), k=rng.randint(1, 128),
                    dtype=rng.choice(["bf16", "f32"]) if rng.random() < 0.5 else "bf16",
                    mode=rng.choice(["both", "both", "loss", "grad"]), tau=rng.choice([1.0, 2.0, 0.7]))
    return dict(op=op, t=_log(rng, 1, 8192), v=_log(rng, 1000, 131072), d=_log(rng, 64, 5120), dtype=dtype)


# ---- inputs --------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x, square=False):
    """NVFP4 of x [rows][cols] along cols, nearest-even: codes [rows][cols/2], E4M3 bytes
    [rows][cols/16] and (S, amax); `square` gives each 16 x 16 block one scale."""
    x = x.float()
    rows, cols = x.shape
    amax = x.abs().max()
    # torch turns a division by (or of) a Python number into a product with a rounded reciprocal;
    # between tensors it is the correctly rounded quotient that the format's definition names
    full, six = torch.full_like(amax, 2688.0), torch.full_like(amax, 6.0)
    s_enc = torch.where(amax > 0, full / amax, torch.ones_like(amax)).clamp(max=torch.finfo(torch.float32).max)
    top = x.view(rows, cols // 16, 16).abs().amax(2)
    if square:
        top = top.view(rows // 16, 16, cols // 16).amax(1).repeat_interleave(16, 0)
    scale = ((top * s_enc) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    inv = torch.where(scale.float() > 0, s_enc / scale.float(), torch.zeros_like(top))
    y = x * inv.repeat_interleave(16, 1)
    a = y.abs()
    # nearest value of the grid, ties to the even code: below 2 in halves, below 4 in ones, then in twos
    code = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    code = (code.clamp(max=7) + 8.0 * torch.signbit(y)).to(torch.uint8)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return packed.contiguous(), scale.view(torch.uint8), torch.stack([s_enc, amax])


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + sum(ord(c) for c in case["op"]))
    return g


def prepare(case, seed):
    g, op = _gen(case, seed), case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if op.startswith("ffn"):
        m, f, k = case["m"], case["f"], case["k"]
        x = randn(m, k)
        x[:, (rand(max(1, k // 1000)) * k).long()] *= 30.0  # a few outlier channels
        x = x.bfloat16()
        w = (0.02 * randn(2 * f, k)).bfloat16()
        st = dict(case=case, x=_quantize(x), w=_quantize(w, square=True))
        st["lut"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        if op != "ffn":
            # gradients with heavier tails than a normal's
            st["dh"] = (1e-3 * randn(m, f) / (0.2 + rand(m, f))).to(_type(case))
        if op == "ffn_backward":
            st["x_t"] = _quantize(x.t().contiguous())
            st["w_t"] = _quantize(w.t().contiguous(), square=True)
        return st
    if op == "distill":
        t, v, k = case["t"], case["v"], case["k"]
        logits = torch.empty(t, v, device="cuda", dtype=_type(case))
        for r in range(0, t, 512):
            logits[r:r + 512] = 2.5 * randn(min(512, t - r), v)
        if v % 2:  # an odd vocabulary comes padded: its last entries are masked
            logits[:, v - v // 100:] = -math.inf
        live = v - v // 100
        # the teacher agrees in part: its top entries lie at random places, none twice
        idx = torch.stack([torch.randperm(live, generator=g, device="cuda")[:k] for _ in range(min(t, 64))])
        idx = (idx[torch.arange(t, device="cuda") % idx.shape[0]] + (rand(t, 1) * live).long()) % live
        top = (2.0 * randn(t, k) + 6.0).sort(1, descending=True)[0]
        idx = torch.where(rand(t, k) < 0.02, torch.full_like(idx, -1), idx)  # entries that the teacher left out
        weight = (rand(t) > 0.1).float() / t  # a tenth of the tokens are padding
        st = dict(case=case, logits=logits, idx=idx.int(), top=top, weight=weight)
        if case["mode"] == "grad":
            lse = [torch.logsumexp(logits[r:r + 512].float() / case["tau"], 1) for r in range(0, t, 512)]
            st["lse"] = torch.cat(lse)
        return st
    t, v, d = case["t"], case["v"], case["d"]
    tok = torch.pow(float(v), rand(t)).long().clamp(max=v) - 1  # frequencies as one over the rank
    tok = torch.where(rand(t) < 0.01, torch.full_like(tok, -1), tok).int()  # padding
    st = dict(case=case, tok=tok, scale=math.sqrt(d))
    if op == "embed":
        st["table"] = torch.empty(v, d, device="cuda", dtype=_type(case))
        for r in range(0, v, 16384):
            st["table"][r:r + 16384] = 0.02 * randn(min(16384, v - r), d)
    else:
        st["dout"] = (1e-3 * randn(t, d)).to(_type(case))
    return st


# ---- one pass --------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case["op"], case, state)


def _run_own(op, case, s):
    import bit_block_scaled_quant_amd as nv
    if op.startswith("ffn"):
        act = nv.SILU if case["act"] == SILU else nv.GELU
        x, w = nv.Quantized(*s["x"]), nv.Quantized(*s["w"])
        if op == "ffn":
            return nv.gated_ffn(x, w, act, dtype=_type(case))
        if op == "ffn_grad":
            return nv.gated_ffn_grad(s["dh"], x, w, act)
        w.codes_t, w.scales_t = s["w_t"][:2]
        return nv.gated_ffn_backward(s["dh"], x, nv.Quantized(*s["x_t"]), w, act, rounding=nv.RNE, rht_t=False,
                                     dtype=torch.bfloat16)
    if op == "distill":
        args = (s["logits"], s["idx"], s["top"])
        if case["mode"] == "loss":
            return nv.distill_topk(*args, weight=s["weight"], temperature=case["tau"])
        if case["mode"] == "grad":
            return nv.distill_topk_grad(*args, s["lse"], weight=s["weight"], temperature=case["tau"])
        return nv.distill_topk_loss_and_grad(*args, weight=s["weight"], temperature=case["tau"])
    if op == "embed":
        return nv.embed(s["tok"], s["table"], scale=s["scale"])
    return nv.embed_grad(s["tok"], s["dout"], case["v"], scale=s["scale"])


def _dequantize(q, lut):
    codes, scales, ts = q
    both = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    value = lut[both.int()].view(codes.shape[0], -1, 16) * scales.view(torch.float8_e4m3fn).float()[:, :, None]
    return value.view(codes.shape[0], -1) / ts[0]


def _gate(a, act):
    """The activation of a and its derivative."""
    if act == SILU:
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * c * (1.0 + 0.134145 * a * a)


def _run_plain(op, case, s):
    if op.startswith("ffn"):
        lut = s["lut"]
        x, w = _dequantize(s["x"], lut), _dequantize(s["w"], lut)
        f = case["f"]
        a, u = x @ w[:f].t(), x @ w[f:].t()
        h, dh_da = _gate(a, case["act"])
        if op == "ffn":
            return (h * u).to(_type(case))
        dh = s["dh"].float()
        dgu = torch.cat([dh * u * dh_da, dh * h], 1).to(_type(case))
        if op == "ffn_grad":
            return dgu
        dx = _dequantize(_quantize(dgu), lut) @ w
        dw = _dequantize(_quantize(dgu.t().contiguous()), lut) @ _dequantize(s["x_t"], lut).t()
        return dx.bfloat16(), dw.bfloat16()
    if op == "distill":
        z = s["logits"].float() / case["tau"]
        idx, k = s["idx"].long(), case["k"]
        ok = (idx >= 0) & (idx < case["v"])
        at = idx.clamp(0, case["v"] - 1)
        top = torch.where(ok, s["top"] / case["tau"], torch.full_like(s["top"], -math.inf))
        high = top.amax(1, keepdim=True)
        any_ = high > -math.inf
        shifted = top - torch.where(any_, high, torch.zeros_like(high))
        total = torch.exp(shifted).sum(1, keepdim=True)
        p = torch.exp(shifted) / torch.where(any_, total, torch.ones_like(total))
        if case["mode"] == "grad":
            lse = s["lse"][:, None]
        else:
            zmax = z.amax(1, keepdim=True)
            lse = zmax + torch.log(torch.exp(z - zmax).sum(1, keepdim=True))
        weight = (s["weight"] * any_[:, 0]).unsqueeze(1)
        terms = torch.where(p > 0, p * (shifted - torch.log(total) - (z.gather(1, at) - lse)), torch.zeros_like(p))
        loss = torch.where(weight[:, 0] != 0, terms.sum(1) * weight[:, 0], torch.zeros_like(weight[:, 0]))
        if case["mode"] == "loss":
            return loss, lse[:, 0]
        grad = torch.exp(z - lse).scatter_add_(1, at, -p)
        grad = (grad * (weight / case["tau"])).to(_type(case))
        return grad if case["mode"] == "grad" else (loss, lse[:, 0], grad)
    tok = s["tok"].long()
    ok = tok >= 0
    if op == "embed":
        return (s["table"][tok.clamp(min=0)].float() * (s["scale"] * ok[:, None])).to(_type(case))
    grad = torch.zeros(case["v"], case["d"], device="cuda")
    return grad.index_add_(0, tok.clamp(min=0), s["dout"].float() * (s["scale"] * ok[:, None]))


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("ffn"):
        m, f, k = case["m"], case["f"], case["k"]
        q = 0.5625
        read = q * (m * k + 2 * f * k)
        if case["op"] == "ffn":
            return dict(bytes=read + b * m * f, flops=4 * m * f * k)
        if case["op"] == "ffn_grad":
            return dict(bytes=read + 3 * b * m * f, flops=4 * m * f * k)
        return dict(bytes=2 * read + b * m * f + 2 * (m * k + 2 * f * k), flops=12 * m * f * k)
    if case["op"] == "distill":
        t, v, k = case["t"], case["v"], case["k"]
        return dict(bytes=t * (v * b * (1 if case["mode"] == "loss" else 2) + 8 * k + 12), flops=4 * t * v)
    t, v, d = case["t"], case["v"], case["d"]
    if case["op"] == "embed":
        return dict(bytes=t * (2 * d * b + 4), flops=t * d)
    return dict(bytes=t * (d * b + 4) + 4 * v * d, flops=t * d)


# ---- the definitions in 64 bits ---------------------------------------------------------
def _values(q):
    """The float64 values that NVFP4 codes stand for."""
    codes, scales, ts = q
    n, half = codes.shape
    out = torch.empty(n, half, 2, dtype=torch.float64, device=codes.device)
    for part, nib in enumerate((codes % 16, codes // 16)):
        e, man = (nib % 8) // 2, (nib % 2).double()
        mag = torch.where(e == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(e.double() - 1.0))
        out[:, :, part] = torch.where(nib >= 8, -mag, mag)
    byte = scales.long()
    e, man = byte // 8, (byte % 8).double()
    sc = torch.where(e == 0, man / 512.0, (1.0 + man / 8.0) * torch.exp2(e.double() - 7.0))
    return (out.view(n, 2 * half // 16, 16) * sc.unsqueeze(2) / ts[0].double()).view(n, 2 * half)


def _f32(v):
    """v rounded to binary32: a step that the format's definition rounds, where values next to a
    border, and the exact ties that 16-bit inputs bring, are decided by that rounding."""
    return v.float().double()


def _nvfp4(x):
    """The float64 values of the nearest-even NVFP4 quantization of x along its rows."""
    amax = x.abs().max()
    s = _f32(torch.full_like(amax, 2688.0) / amax) if amax else torch.ones_like(amax)
    b = x.view(x.shape[0], -1, 16)
    t = _f32(_f32(b.abs().amax(2, keepdim=True) * s) / 6.0).clamp(max=448.0)
    # E4M3: three bits after the leading one, the smallest step 2^-9
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3.0)
    sc = torch.round(t / step) * step
    y = torch.where(sc > 0, _f32(b * _f32(s / sc.clamp(min=2.0 ** -9))), torch.zeros_like(b))
    a = y.abs().clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0))) - 1.0)
    return (torch.copysign(torch.round(a / step) * step, y) * sc / s).view_as(x)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("ffn"):
        x, w = _values(s["x"]), _values(s["w"])
        gate, up = (x @ part.t() for part in w.chunk(2))
        if case["act"] == SILU:
            sig = torch.sigmoid(gate)
            act, slope = gate * sig, sig + gate * sig * (1 - sig)
        else:
            inner = math.sqrt(2 / math.pi) * (gate + 0.044715 * gate.pow(3))
            act = gate * torch.sigmoid(2 * inner)  # (1 + tanh(z)) / 2 is the sigmoid of 2 z
            slope = torch.sigmoid(2 * inner) + gate * torch.sigmoid(2 * inner) * torch.sigmoid(-2 * inner) * (
                2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * gate.pow(2)))
        if op == "ffn":
            return act * up
        dgu = torch.cat([s["dh"].double() * up * slope, s["dh"].double() * act], 1)
        if op == "ffn_grad":
            return dgu
        dgu = dgu.bfloat16().double()  # the gradients are handed to the quantizer in 16 bits
        return _nvfp4(dgu) @ w, _nvfp4(dgu.t().contiguous()) @ _values(s["x_t"]).t()
    if op == "distill":
        tau, losses, lses, grads = case["tau"], [], [], []
        for r in range(0, case["t"], 256):
            z = s["logits"][r:r + 256].double() / tau
            logq = torch.log_softmax(z, 1)
            lse = s["lse"][r:r + 256].double() if case["mode"] == "grad" else torch.logsumexp(z, 1)
            idx, w = s["idx"][r:r + 256].long(), s["weight"][r:r + 256].double()
            there = idx >= 0
            logp = torch.log_softmax((s["top"][r:r + 256].double() / tau).masked_fill(~there, -math.inf), 1)
            p = torch.exp(logp).nan_to_num(0.0)  # a row without entries
            w = torch.where(there.any(1), w, torch.zeros_like(w))
            term = p * (logp.masked_fill(~there, 0.0).nan_to_num(0.0) - logq.gather(1, idx.clamp(min=0)))
            losses.append(torch.where(there, term, torch.zeros_like(term)).sum(1) * w)
            lses.append(lse)
            if case["mode"] != "loss":
                target = torch.zeros_like(z).scatter_add_(1, idx.clamp(min=0), p)
                grads.append(((torch.exp(z - lse[:, None]) - target) * (w / tau)[:, None]).float()
                             if case["dtype"] == "bf16" else (torch.exp(z - lse[:, None]) - target) * (w / tau)[:, None])
        loss, lse = torch.cat(losses), torch.cat(lses)
        if case["mode"] == "loss":
            return loss, lse
        grad = torch.cat(grads)
        return grad if case["mode"] == "grad" else (loss, lse, grad)
    tok = s["tok"].long()
    if op == "embed":
        rows = s["table"][tok.clamp(min=0)].double() * s["scale"]
        return rows.masked_fill((tok < 0)[:, None], 0.0)
    grad = torch.zeros(case["v"], case["d"], dtype=torch.float64, device="cuda")
    keep = tok >= 0
    return grad.index_put_((tok[keep],), s["dout"].double()[keep] * s["scale"], accumulate=True)

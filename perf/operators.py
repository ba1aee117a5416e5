"""The operators around the compressed tensor-parallel sum, as measured cases.

A row-parallel layer of P tensor-parallel ranks in 8-bit integers, and what follows its sum:

  matmul   bf16 activations to int8 with one scale a token, times int8 weights with one scale a
           channel: every rank's partial sum [P, T, H] (``hq_quantize_tokens``, ``hq_int8_matmul``)
  wire     the same product leaving as the hybrid 4-bit/bf16 wire with no partial sum in memory,
           then the wire's rank-ordered sum [T, H] (``hq_int8_matmul_pack``, ``hq_dequant_reduce``)
  norm     the block's end: its output normalised, gated and added to the scaled residual, and the
           next block's norm of the new residual (``hq_residual_norm``)
  layer    all of it in a row: activations, wire, sum, residual and norm to int8, next projection
"""
import math

import torch

own = False

# Numbers of the partial sums' workloads: ranks, rows and widths are the repository's decode and
# prefill workloads; K is a rank's share of an attention output (H / P) or of a 4 H wide layer.
CASES = [
    # one token on one real rank: an attention output's share, where only latency counts
    dict(name="matmul-token", op="matmul", P=1, T=1, H=4096, K=512, quantize=True, bias=False, f32=False),
    # a decode batch over all ranks: bound by reading the weights
    dict(name="matmul-decode", op="matmul", P=8, T=32, H=8192, K=1024, quantize=True, bias=False, f32=False),
    # a prompt through a 4 H wide layer's down projection, its activations in int8 already
    dict(name="matmul-prefill-7b", op="matmul", P=8, T=4096, H=4096, K=2048, quantize=False, bias=False, f32=False),
    # the largest prompt, activations quantized in the pass
    dict(name="matmul-prefill-70b", op="matmul", P=8, T=8192, H=8192, K=1024, quantize=True, bias=False, f32=False),
    # nothing a multiple of anything: a ragged prompt, an odd K, bias and fp32 output
    dict(name="matmul-ragged", op="matmul", P=3, T=333, H=2056, K=1001, quantize=False, bias=True, f32=True),
    # the wire of a decode batch
    dict(name="wire-decode", op="wire", P=4, T=32, H=4096, K=1024, k=64),
    # the wire of a prompt: an attention output's share
    dict(name="wire-prefill-7b", op="wire", P=8, T=4096, H=4096, K=512, k=128),
    # the largest wire
    dict(name="wire-prefill-70b", op="wire", P=8, T=8192, H=8192, K=1024, k=256),
    # the end of a block for a decode batch
    dict(name="norm-decode", op="norm", T=32, H=8192, post="rms", pre="rms", gate=0, res_f32=False, y_f32=False),
    # the same for the largest prompt, with a learned gate on every feature
    dict(name="norm-prefill", op="norm", T=8192, H=8192, post="rms", pre="rms", gate=1, res_f32=False, y_f32=False),
    # layer norms, an fp32 residual, an fp32 sum and one gate row for each of three sequences
    dict(name="norm-ragged", op="norm", T=777, H=5000, post="none", pre="layer", gate=3, res_f32=True, y_f32=True),
    # a whole decode layer's path from activations to the next projection
    dict(name="layer-decode", op="layer", P=4, T=32, H=4096, K=1024, k=64, F=2048),
]
EPS = 1e-6
MOST_OPS, MOST_SUMS = 2.0 * 8 * 8192 * 8192 * 1024, 8 * 8192 * 8192


def listed():
    return [dict(c) for c in CASES]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "wire", "wire", "norm", "layer"])
    T, H = _log(rng, 1, 8192), 8 * _log(rng, 32, 1024)
    if op == "norm":
        gate = rng.choice([0, 1, T])
        return dict(op=op, T=T, H=H, post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                    gate=gate, res_f32=rng.random() < 0.5, y_f32=rng.random() < 0.5)
    P, K = rng.randint(1, 8), _log(rng, 64, 4096)
    T = max(1, min(T, int(MOST_SUMS / (P * H)), int(MOST_OPS / (2.0 * P * H * K))))
    if op == "matmul":
        return dict(op=op, P=P, T=T, H=H, K=K, quantize=rng.random() < 0.5, bias=rng.random() < 0.5, f32=rng.random() < 0.3)
    k = 8 * rng.randint(0, H // 128)
    if op == "wire":
        return dict(op=op, P=P, T=T, H=H, K=K, k=k)
    return dict(op=op, P=P, T=min(T, 512), H=H, K=K, k=k, F=8 * _log(rng, 32, 512))


# ---------------------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _pitched(t, multiple):
    """`t` with rows a multiple of `multiple` elements apart, as the tensors of a padded buffer are."""
    n = t.shape[-1]
    wide = torch.zeros(*t.shape[:-1], -(-n // multiple) * multiple, dtype=t.dtype, device=t.device)
    wide[..., :n] = t
    return wide[..., :n]


def _activations(g, P, T, K):
    """Tokens of different magnitude, a few channels far larger than the rest."""
    channel = torch.exp(0.5 * _randn(g, P, 1, K))
    channel = torch.where(torch.rand(P, 1, K, generator=g, device="cuda") < 0.004, 20 * channel, channel)
    token = torch.exp(0.5 * _randn(g, P, T, 1))
    x = _randn(g, P, T, K, dtype=torch.bfloat16)
    return _pitched((x * (channel * token)).to(torch.bfloat16), 8)


def _weights(g, P, N, K, outliers):
    """int8 weights of normal columns with a scale a channel; `outliers` channels are larger in every rank."""
    row = torch.exp(0.5 * _randn(g, N))
    big = torch.randperm(N, generator=g, device="cuda")[:outliers]
    row[big] *= 50
    q = torch.clamp(torch.round(32 * _randn(g, P, N, K, dtype=torch.bfloat16)), -127, 127).to(torch.int8)
    return _pitched(q, 16), (row * torch.exp(0.1 * _randn(g, P, N)) / (32 * math.sqrt(K))).contiguous()


def _int8_rows(x):
    """int8 activations with a scale a token, as they come out of an earlier layer."""
    x = x.float()
    s = (x.abs().amax(-1) / 127).clamp_min(1e-30)
    return _pitched(torch.round(x / s[..., None]).to(torch.int8), 16), s.contiguous()


def _selection(lo, hi, k):
    """The kept features and the 4-bit grids of the others, from every rank's ranges [P, H]."""
    lo, hi = lo.clamp_max(0), hi.clamp_min(0)
    order = torch.sort((hi - lo).sum(0), descending=True, stable=True).indices
    keep, rest = torch.sort(order[:k]).values.int(), torch.sort(order[k:]).values.int()
    scale = (hi - lo) / 15
    inv = 1 / scale
    zero = torch.clamp(torch.round(-lo * inv), 0, 15).to(torch.uint8)
    return dict(keep=keep, rest=rest, scale=scale.contiguous(), inv=inv.contiguous(), zero=zero.contiguous())


def _buffers(c):
    """What a program holds for its results."""
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    b = {}
    if c["op"] != "norm":
        P, T, H, K = c["P"], c["T"], c["H"], c["K"]
        b["q"] = new(P, T, -(-K // 16) * 16, dtype=torch.int8)[..., :K]
        b["qs"] = new(P, T, dtype=torch.float32)
    if c["op"] == "matmul":
        b["out"] = new(P, T, H, dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if c["op"] in ("wire", "layer"):
        b["codes"] = new(P, T, (H - c["k"]) // 8, dtype=torch.int32)
        b["side"] = new(P, c["k"], T)
        b["sum"] = new(T, H)
    if c["op"] in ("norm", "layer"):
        T, H = c["T"], c["H"]
        b["res"] = new(T, H, dtype=torch.float32 if c.get("res_f32") else torch.bfloat16)
    if c["op"] == "norm":
        b["h"] = new(T, H)
    if c["op"] == "layer":
        b["hq"], b["hs"] = new(1, T, -(-H // 16) * 16, dtype=torch.int8)[..., :H], new(1, T, dtype=torch.float32)
        b["up"] = new(1, T, c["F"])
    return b


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 17)
    s = {"c": c, "b": _buffers(c)}
    if c["op"] in ("norm", "layer"):
        T, H = c["T"], c["H"]
        s["post_w"], s["pre_w"] = 1 + 0.2 * _randn(g, H), 1 + 0.2 * _randn(g, H)
        s["post_b"], s["pre_b"] = 0.1 * _randn(g, H), 0.1 * _randn(g, H)
        res = _randn(g, T, H) * torch.exp(0.5 * _randn(g, H))
        s["res"] = res if c.get("res_f32") else res.bfloat16()
        s["alpha"], s["beta"] = 1.0, 0.75
        if c.get("gate"):
            s["gate"] = torch.tanh(_randn(g, c["gate"], H)).bfloat16()
        if c["op"] == "norm":
            y = 3 * _randn(g, T, H) + 0.3
            s["y"] = y if c["y_f32"] else y.bfloat16()
            return s
    P, T, H, K = c["P"], c["T"], c["H"], c["K"]
    x = _activations(g, P, T, K)
    w, ws = _weights(g, P, H, K, c.get("k", H // 64) // 2)
    if c["op"] == "matmul":
        s["w"], s["ws"] = w, ws
        if c["bias"]:
            s["bias"] = _randn(g, P, H).bfloat16()
        if c["quantize"]:
            s["x"] = x
        else:
            s["a"], s["as"] = _int8_rows(x)
        return s
    s["x"] = x
    # ranges of a calibration batch's partial sums, then the weights' rows in the wire's order
    cal, cal_s = _int8_rows(_activations(g, P, 64, K))
    y = torch.bmm(cal.float(), w.float().transpose(1, 2)) * cal_s[..., None] * ws[:, None]
    s.update(_selection(y.amin(1), y.amax(1), c["k"]))
    order = torch.cat([s["rest"], s["keep"]]).long()
    s["order"] = order
    s["w"], s["ws"] = _pitched(w[:, order], 16), ws[:, order].contiguous()
    if c["op"] == "layer":
        s["up_w"], s["up_s"] = _weights(g, 1, c["F"], H, 0)
    return s


# ---------------------------------------------------------------------------------- plain form
def _tokens_to_int8(x, t=torch.float32):
    """Whole numbers -127..127 and the scale of every row."""
    x = x.to(t)
    amax = x.abs().amax(-1, keepdim=True)
    some = amax > 0
    q = torch.where(some, torch.round(x * 127 / torch.where(some, amax, 1)), 0)
    return q, torch.where(some, amax / 127, 1)


def _product(a, a_s, w, w_s, t=torch.float32):
    return torch.bmm(a.to(t), w.to(t).transpose(1, 2)) * a_s.to(t)[..., None] * w_s.to(t)[:, None]


def _sum_of_wires(x, s, t=torch.float32):
    """The ranks' sum after the wire; x [P, T, H] holds the partial sums in the wire's order."""
    k, P = s["c"]["k"], s["c"]["P"]
    H = x.shape[-1]
    x = x.bfloat16()  # a partial sum is a bf16 number
    rest = s["rest"].long()
    inv, zero, scale = s["inv"][:, None, rest], s["zero"][:, None, rest].to(t), s["scale"][:, None, rest].to(t)
    code = torch.clamp(torch.round((x[..., :H - k].float() * inv)).to(t) + zero, 0, 15)
    out = torch.empty(x.shape[1], H, dtype=t, device=x.device)
    out[:, rest] = ((code - zero) * scale).sum(0)
    out[:, s["keep"].long()] = x[..., H - k:].to(t).sum(0)
    return out


def _normed(x, kind, w, b):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    return n + b.to(x.dtype) if kind == "layer" else n


def _residual(y, s, post, t=torch.float32):
    u = _normed(y.to(t), post, s["post_w"], s["post_b"])
    if "gate" in s:
        u = u * s["gate"].to(t).repeat_interleave(y.shape[0] // s["gate"].shape[0], 0)
    return (s["alpha"] * s["res"].to(t) + s["beta"] * u).to(s["res"].dtype)


def _plain(s, t=torch.float32):
    c = s["c"]
    narrow = (lambda v: v) if t == torch.float64 else (lambda v: v.bfloat16())
    if c["op"] == "norm":
        r = _residual(s["y"], s, c["post"], t)
        return {"res": r, "h": narrow(_normed(r.to(t), c["pre"], s["pre_w"], s["pre_b"]))}
    a, a_s = (s["a"], s["as"]) if "a" in s else _tokens_to_int8(s["x"], t)
    a_s = a_s.reshape(c["P"], c["T"])
    x = _product(a, a_s, s["w"], s["ws"], t)
    if c["op"] == "matmul":
        x = x + s["bias"].to(t)[:, None] if "bias" in s else x
        return x if c["f32"] else narrow(x)
    y = _sum_of_wires(x, s, t).bfloat16()
    if c["op"] == "wire":
        return y
    r = _residual(y, s, "rms", t)
    h, h_s = _tokens_to_int8(_normed(r.to(t), "rms", s["pre_w"], None).bfloat16(), t)
    return {"res": r, "up": narrow(_product(h[None], h_s.reshape(1, -1), s["up_w"], s["up_s"], t))}


# ---------------------------------------------------------------------------------- the framework's calls
def _calls(s):
    import bit_tensor_activation_b200 as hq

    c, b = s["c"], s["b"]
    norms = {"none": hq.HQ_NORM_NONE, "rms": hq.HQ_NORM_RMS, "layer": hq.HQ_NORM_LAYER}
    if c["op"] == "norm":
        hq.hq_residual_norm(s["y"], s["res"], b["res"], h=b["h"], post=norms[c["post"]], post_w=s["post_w"],
                            post_b=s["post_b"] if c["post"] == "layer" else None, gate=s.get("gate"),
                            alpha=s["alpha"], beta=s["beta"], pre=norms[c["pre"]], pre_w=s["pre_w"],
                            pre_b=s["pre_b"] if c["pre"] == "layer" else None, eps=EPS)
        return {"res": b["res"], "h": b["h"]}
    if "a" in s:
        a, a_s = s["a"], s["as"]
    else:
        a, a_s = b["q"], b["qs"]
        hq.hq_quantize_tokens(s["x"], a, a_s)
    if c["op"] == "matmul":
        hq.hq_int8_matmul(a, a_s, s["w"], s["ws"], b["out"], bias=s.get("bias"))
        return b["out"]
    hq.hq_int8_matmul_pack(a, a_s, s["w"], s["ws"], s["keep"], s["rest"], s["inv"], s["zero"], b["codes"], b["side"])
    hq.hq_dequant_reduce(b["codes"], b["side"], s["keep"], s["rest"], s["scale"], s["zero"], b["sum"])
    if c["op"] == "wire":
        return b["sum"]
    hq.hq_residual_norm(b["sum"], s["res"], b["res"], q=b["hq"][0], q_scale=b["hs"][0], post=hq.HQ_NORM_RMS,
                        post_w=s["post_w"], alpha=s["alpha"], beta=s["beta"], gate=s.get("gate"),
                        pre=hq.HQ_NORM_RMS, pre_w=s["pre_w"], eps=EPS)
    hq.hq_int8_matmul(b["hq"], b["hs"], s["up_w"], s["up_s"], b["up"])
    return {"res": b["res"], "up": b["up"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- work and definition
def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] == "norm":
        res, y = (4 if c["res_f32"] else 2), (4 if c["y_f32"] else 2)
        return {"bytes": T * H * (2 * res + y + 2) + 2 * c["gate"] * H + 8 * H, "flops": 16 * T * H}
    P, K = c["P"], c["K"]
    read = P * T * K * (2 if c.get("quantize", True) else 1) + P * H * K + 4 * P * H
    flops = 2 * P * T * H * K
    if c["op"] == "matmul":
        return {"bytes": read + P * T * H * (4 if c["f32"] else 2), "flops": flops}
    read += 9 * P * H  # the grids; the wire itself need not leave the chip on one GPU
    if c["op"] == "wire":
        return {"bytes": read + 2 * T * H, "flops": flops}
    F = c["F"]
    return {"bytes": read + 4 * T * H + H * F + 2 * T * F + 4 * (2 * H + F), "flops": flops + 2 * T * H * F}


def exact(case, seed):
    """The definitions in 64 bits, from the inputs alone: every product's sum, scale and norm in
    double; the roundings that are part of a definition (codes, a bf16 partial sum or norm that is
    quantized again, a stored residual) where they stand in it."""
    s = prepare(case, seed)
    c, D = s["c"], torch.float64

    def quantized(v):
        v = v.to(D)
        top = v.abs().max(dim=-1, keepdim=True).values
        step = torch.where(top == 0, torch.ones_like(top), top / 127)
        return torch.where(top == 0, torch.zeros_like(v), torch.round(v * 127 / torch.where(top == 0, 1.0, top))), step

    def norm(v, kind, w, b):
        v = v.to(D)
        if kind == "none":
            return v
        centre = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
        n = (v - centre) / torch.sqrt(((v - centre) ** 2).mean(-1, keepdim=True) + EPS)
        return n * w.to(D) + (b.to(D) if kind == "layer" else 0.0)

    def new_residual(y, kind):
        u = norm(y, kind, s["post_w"], s["post_b"])
        if "gate" in s:
            n = u.shape[0] // s["gate"].shape[0]
            u = u * s["gate"].to(D)[torch.arange(u.shape[0], device=u.device) // n]
        return s["alpha"] * s["res"].to(D) + s["beta"] * u

    if c["op"] == "norm":
        r = new_residual(s["y"], c["post"])
        return {"res": r, "h": norm(r.to(s["res"].dtype), c["pre"], s["pre_w"], s["pre_b"])}
    a, step = (s["a"].to(D), s["as"].to(D)[..., None]) if "a" in s else quantized(s["x"])
    x = torch.matmul(a, s["w"].to(D).mT) * step * s["ws"].to(D)[:, None, :]
    if c["op"] == "matmul":
        return x + s["bias"].to(D)[:, None, :] if "bias" in s else x
    # the wire's features in their own order, then the code of every feature that is not kept
    natural = torch.empty_like(x)
    natural[..., s["order"]] = x
    natural = natural.bfloat16().to(D)
    zero = s["zero"].to(D)[:, None, :]
    code = torch.round(natural * s["inv"].to(D)[:, None, :]) + zero
    value = (code.clamp(0, 15) - zero) * s["scale"].to(D)[:, None, :]
    kept = torch.zeros(c["H"], dtype=torch.bool, device=x.device)
    kept[s["keep"].long()] = True
    y = torch.where(kept, natural, value).sum(0)
    if c["op"] == "wire":
        return y
    r = new_residual(y.bfloat16(), "rms")
    h, h_step = quantized(norm(r.to(s["res"].dtype), "rms", s["pre_w"], None).bfloat16())
    return {"res": r, "up": (torch.matmul(h, s["up_w"][0].to(D).mT) * h_step * s["up_s"].to(D))[None]}

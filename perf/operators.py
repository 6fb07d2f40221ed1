"""Cases of the 8-bit linear path and of the query/key norm with rotation, for measurement.

The operators, each in a plain form of elementary torch operations and as the library's call:

  quantize  rows of a matrix to 8-bit integers, one scale a row:
            amax = max_j |x_j|,  scale = amax / 127,  q_j = round_half_even(127 x_j / amax)
            (a row of zeros: scale 0, q 0)
  ln        the same of h = LN(x) (1 + scale) + shift, the modulated LayerNorm before a block's projections
  swiglu    the same of h = SiLU(g) * u, with g | u the two halves of a row (the input of the down projection)
  gemm      C[m, n] = (sum_k A[m, k] B[n, k]) a_scale[m] b_scale[n] + bias[n], A and B 8-bit integers; with a
            gate and a residual: C = residual + gate[n] * that
  qk        per head of the queries and keys: RMSNorm with a gain, then the rotation of its pairs by the
            token's angles

An operand in 8 bits is returned as the values it stands for, q * scale.  Where the rows are computed before
they are rounded (ln, swiglu), an FP32 difference in the last place moves a value that lies on a border
between two integers by a whole step, so there the values come in BF16; quantize's own result is exact and
comes in FP32.
"""
import math

import torch

own = False

LN_EPS = 1e-6
QK_EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # A single token through the fused q|k|v projection: latency, the weights read once.
        dict(name="gemm one token", op="gemm", m=1, n=9216, k=3072, out="bf16", bias=False, resid=False),
        # A short prompt (77 tokens) through the text projection, encoder width 4096, with its bias.
        dict(name="gemm prompt projection", op="gemm", m=77, n=3072, k=4096, out="f32", bias=True, resid=False),
        # The q|k|v projection of both guidance branches of a 1024 x 1024 image with 512 prompt tokens.
        dict(name="gemm qkv both branches", op="gemm", m=9216, n=9216, k=3072, out="bf16", bias=False, resid=False),
        # The down projection of one branch into the FP32 residual stream, gated, a ragged prompt of 333 tokens.
        dict(name="gemm down gated residual", op="gemm", m=4429, n=3072, k=8192, out="f32", bias=False, resid=True),
        # The encoder states of a 512-token prompt before the text projection.
        dict(name="quantize encoder states", op="quantize", rows=512, dim=4096, x="bf16"),
        # The attention output of both branches before the output projection.
        dict(name="quantize attention out", op="quantize", rows=9216, dim=3072, x="bf16"),
        # A 256 x 256 image with 77 prompt tokens before its projections.
        dict(name="ln small image", op="ln", rows=333, dim=3072),
        # The residual stream of both branches at 1024 x 1024.
        dict(name="ln both branches", op="ln", rows=9216, dim=3072),
        # The feed-forward activation of a few tokens at the small width.
        dict(name="swiglu few tokens", op="swiglu", rows=37, dim=704),
        # The feed-forward activation of both branches.
        dict(name="swiglu both branches", op="swiglu", rows=9216, dim=8192),
        # One new token for each of 8 sequences, shared key heads, halves rotated, far positions.
        dict(name="qk one token each", op="qk", rows=8, hq=32, hk=8, dim=128, rot=128, pairing="halves", x="bf16",
             npos=32768, positions=True),
        # The queries and keys of both branches inside the fused projection's output.
        dict(name="qk both branches", op="qk", rows=9216, hq=24, hk=24, dim=128, rot=128, pairing="adjacent", x="bf16",
             npos=4608, positions=False),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over the logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quantize", "ln", "swiglu", "qk", "qk"])
    if op == "gemm":
        resid = rng.random() < 0.3
        out = "f32" if resid or rng.random() < 0.3 else "bf16"
        return dict(op=op, m=_log(rng, 1, 9216), n=_log(rng, 96, 9216, rng.choice([1, 8, 32])), k=_log(rng, 64, 8192, 16)
                    if rng.random() < 0.7 else _log(rng, 256, 3072, 256), out=out, bias=rng.random() < 0.4, resid=resid)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 9216), dim=_log(rng, 64, 4096, 16), x=rng.choice(["bf16", "f32"]))
    if op == "ln":
        return dict(op=op, rows=_log(rng, 1, 9216), dim=_log(rng, 256, 4096, 128))
    if op == "swiglu":
        return dict(op=op, rows=_log(rng, 1, 9216), dim=_log(rng, 64, 8192, 16))
    dim = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 8, 24])
    hq = hk * rng.choice([1, 1, 3, 4]) if hk < 24 else 24
    npos = _log(rng, 16, 65536)
    return dict(op=op, rows=_log(rng, 1, 9216), hq=hq, hk=hk, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                pairing=rng.choice(["adjacent", "halves"]), x=rng.choice(["bf16", "f32"]), npos=npos,
                positions=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        ob = 2 if case["out"] == "bf16" else 4
        b = m * k + n * k + 4 * (m + n) + m * n * ob
        b += 2 * n if case["bias"] else 0
        b += 4 * m * n + 4 * n if case["resid"] else 0
        return dict(bytes=b, flops=2 * m * n * k)
    if op == "qk":
        per = case["rows"] * (case["hq"] + case["hk"]) * case["dim"]
        xb = 2 if case["x"] == "bf16" else 4
        table = min(case["rows"], case["npos"]) * (case["rot"] // 2) * 8
        return dict(bytes=per * (xb + 2) + table + 8 * case["dim"], flops=8 * per)
    r, d = case["rows"], case["dim"]
    if op == "quantize":
        return dict(bytes=r * d * ((2 if case["x"] == "bf16" else 4) + 1) + 4 * r, flops=3 * r * d)
    if op == "ln":
        return dict(bytes=r * d * (4 + 1) + 8 * d + 4 * r, flops=10 * r * d)
    return dict(bytes=r * d * (2 * 2 + 1) + 4 * r, flops=8 * r * d)


# ------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, dim, dtype):
    """Normal values whose rows differ in size, with a few channels far larger than the others (what the streams
    of transformers look like) and, from 8 rows on, one row in 8 of zeros (a padded token)."""
    x = torch.randn(rows, dim, generator=g, device="cuda")
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)
    x *= 1.0 + 15.0 * (torch.rand(dim, generator=g, device="cuda") < 0.01)
    if rows >= 8:
        x[5::8] = 0.0
    return x.to(dtype)


_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s = dict(case=case)
        s["a"] = (torch.randn(m, k, generator=g, device="cuda") * 30).round().clamp(-127, 127).to(torch.int8)
        s["b"] = (torch.randn(n, k, generator=g, device="cuda") * 30).round().clamp(-127, 127).to(torch.int8)
        s["a_scale"] = torch.exp(torch.randn(m, generator=g, device="cuda") * 0.5) * (4.0 / 127)
        s["b_scale"] = torch.exp(torch.randn(n, generator=g, device="cuda") * 0.2) * (0.08 / 127)
        s["bias"] = (torch.randn(n, generator=g, device="cuda") * 0.02).bfloat16() if case["bias"] else None
        s["gate"] = torch.randn(n, generator=g, device="cuda") * 0.5 if case["resid"] else None
        s["residual"] = torch.randn(m, n, generator=g, device="cuda") if case["resid"] else None
        return s
    if op == "quantize":
        return dict(case=case, x=_activations(g, case["rows"], case["dim"], _DTYPE[case["x"]]))
    if op == "ln":
        d = case["dim"]
        return dict(case=case, x=_activations(g, case["rows"], d, torch.float32),
                    shift=torch.randn(d, generator=g, device="cuda") * 0.1,
                    scale=torch.randn(d, generator=g, device="cuda") * 0.1)
    if op == "swiglu":
        return dict(case=case, gu=_activations(g, case["rows"], 2 * case["dim"], torch.bfloat16))
    rows, hq, hk, d, rot, npos = (case[f] for f in ("rows", "hq", "hk", "dim", "rot", "npos"))
    qkv = torch.randn(rows, (hq + 2 * hk) * d, generator=g, device="cuda")  # the fused projection's output
    qkv = (qkv * torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)).to(_DTYPE[case["x"]])
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                    -torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
    ang = torch.arange(npos, dtype=torch.float64, device="cuda")[:, None] * inv
    s = dict(case=case, q=qkv[:, :hq * d].view(rows, hq, d), k=qkv[:, hq * d:(hq + hk) * d].view(rows, hk, d))
    s["rope"] = torch.stack([torch.cos(ang), torch.sin(ang)], dim=-1).float().contiguous()  # [npos, rot/2, 2]
    s["q_gain"] = 1 + torch.randn(d, generator=g, device="cuda") * 0.02
    s["k_gain"] = 1 + torch.randn(d, generator=g, device="cuda") * 0.02
    s["positions"] = (torch.randint(0, npos, (rows,), generator=g, device="cuda", dtype=torch.int32)
                      if case["positions"] else None)
    return s


# ------------------------------------------------------------------------------------------ one pass
def _plain_quantize(h):
    """(q * scale, scale) of FP32 rows; the quotient in 64 bits, since values lie on the borders."""
    amax = h.abs().amax(dim=1, keepdim=True)
    q = torch.round(h.double() * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)).double()).float()
    scale = amax / 127.0
    return q * scale, scale[:, 0]


def _plain_qk_one(x, gain, cos, sin, case):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + QK_EPS) * gain
    r = case["rot"]
    y = x.clone()
    if case["pairing"] == "adjacent":
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = a * cos - b * sin
        y[..., 1:r:2] = a * sin + b * cos
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = a * cos - b * sin
        y[..., r // 2:r] = a * sin + b * cos
    return y.bfloat16()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import diffusion_transformer_text_block_b200 as moss
        if op == "gemm":
            return moss.op_gemm_i8(state["a"], state["a_scale"], state["b"], state["b_scale"], bias=state["bias"],
                                   gate=state["gate"], residual=state["residual"], out_dtype=_DTYPE[case["out"]])
        if op == "qk":
            return moss.op_qk_norm_rope(state["q"], state["k"], state["q_gain"], state["k_gain"], state["rope"],
                                        positions=state["positions"], pairing=case["pairing"], eps=QK_EPS)
        if op == "quantize":
            q, scale = moss.op_quantize_i8(state["x"])
            return torch.mul(q, scale[:, None]), scale
        if op == "ln":
            q, scale = moss.op_ln_modulate_i8(state["x"], state["shift"], state["scale"])
        else:
            q, scale = moss.op_swiglu_i8(state["gu"])
        return torch.mul(q, scale[:, None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)), scale
    if op == "gemm":
        c = (state["a"].float() @ state["b"].float().T) * state["a_scale"][:, None] * state["b_scale"]
        if state["bias"] is not None:
            c = c + state["bias"].float()
        if state["residual"] is not None:
            c = state["residual"] + state["gate"] * c
        return c.to(_DTYPE[case["out"]])
    if op == "qk":
        rows, npos = case["rows"], case["npos"]
        at = state["positions"].long() if state["positions"] is not None else torch.arange(rows, device="cuda") % npos
        cos, sin = state["rope"][at][:, None, :, 0], state["rope"][at][:, None, :, 1]
        return (_plain_qk_one(state["q"], state["q_gain"], cos, sin, case),
                _plain_qk_one(state["k"], state["k_gain"], cos, sin, case))
    if op == "quantize":
        return _plain_quantize(state["x"].float())
    if op == "ln":
        x = state["x"]
        xc = x - x.mean(dim=1, keepdim=True)
        h = xc * torch.rsqrt((xc * xc).mean(dim=1, keepdim=True) + LN_EPS) * (1 + state["scale"]) + state["shift"]
    else:
        g, u = state["gu"].float().chunk(2, dim=1)
        h = g / (1 + torch.exp(-g)) * u
    v, scale = _plain_quantize(h)
    return v.bfloat16(), scale


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        c = torch.mm(s["a"].double(), s["b"].double().t())
        c.mul_(s["a_scale"].double().unsqueeze(1)).mul_(s["b_scale"].double().unsqueeze(0))
        if case["bias"]:
            c.add_(s["bias"].double())
        if case["resid"]:
            c.mul_(s["gate"].double()).add_(s["residual"].double())
        return c
    if op == "qk":
        d, rot = case["dim"], case["rot"]
        pos = s["positions"] if case["positions"] else torch.remainder(torch.arange(case["rows"], device="cuda"),
                                                                      case["npos"])
        turn = torch.view_as_complex(s["rope"].double().contiguous())[pos.long()].unsqueeze(1)
        outs = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            x = x.double()
            x = gain.double() * x / torch.sqrt(torch.sum(x ** 2, dim=-1, keepdim=True) / d + QK_EPS)
            head, tail = x[..., :rot], x[..., rot:]
            if case["pairing"] == "adjacent":
                z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
                head = torch.cat([z.real, z.imag], dim=-1)
            outs.append(torch.cat([head, tail], dim=-1))
        return tuple(outs)
    if op == "quantize":
        h = s["x"].double()
    elif op == "ln":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        h = (x - mean) / torch.sqrt(var + LN_EPS) * (s["scale"].double() + 1.0) + s["shift"].double()
    else:
        f = case["dim"]
        h = s["gu"][:, :f].double() * torch.sigmoid(s["gu"][:, :f].double()) * s["gu"][:, f:].double()
    scale = torch.amax(torch.abs(h), dim=1) / 127.0
    steps = torch.where(scale[:, None] > 0, h * 127.0 / (127.0 * scale[:, None]), torch.zeros_like(h))
    if op == "quantize":  # the largest value itself, so that ties stay ties
        top = torch.amax(torch.abs(h), dim=1, keepdim=True)
        steps = torch.where(top > 0, h * 127.0 / top, torch.zeros_like(h))
    return torch.round(steps) * scale[:, None], scale

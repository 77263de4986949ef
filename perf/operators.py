"""The feed-forward operators' workloads: their inputs, one pass through each operator, the
bytes and operations a pass cannot do without, and the 64-bit values it should give.

Four kinds of pass:

``gated``     H = act(X Wg) * (X Wu), the gated projection of a feed-forward block (serving:
              single tokens and prompts).
``train``     the same with its pre-activations kept, then its backward pass: H, dX, dWg, dWu.
``int8``      C = (Aq Bq^T) scaled by row and by column, or the gated projection from two such
              products.
``linear8``   the rows of a 16-bit or fp32 X brought to int8 with one scale each, then that
              product with int8 weights: a whole layer as a served model runs it.

``run`` computes the plain form (elementary torch operations, 32 bits or more, rounded once
at the end) unless ``own`` is true, when it calls this package's kernels.  Weights are stored
[K,N] ("kn") or [N,K] ("nk").
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_GELU_C, _GELU_A = 0.7978845608, 0.044715


def listed():
    return [
        # one token of a decoding step through a block's two projections: all of it is the
        # reading of the weights
        dict(name="gated_token", op="gated", M=1, N=12288, K=4096, dtype="bf16", layout="nk", act="silu"),
        # a small odd-sized block, rows that start at any 2-byte address
        dict(name="gated_ragged", op="gated", M=300, N=2731, K=1001, dtype="bf16", layout="nk", act="relu"),
        # a long prompt, or many short ones together
        dict(name="gated_prompt", op="gated", M=8192, N=12288, K=4096, dtype="bf16", layout="nk", act="silu"),
        # a small model's training step, weights stored [K,N]
        dict(name="train_small", op="train", M=2048, N=4096, K=1024, dtype="bf16", layout="kn", act="gelu_tanh"),
        # ... with odd sizes throughout, in fp16
        dict(name="train_ragged", op="train", M=511, N=1365, K=500, dtype="f16", layout="kn", act="gelu_tanh"),
        # a large model's training step: 4096 tokens on one GPU
        dict(name="train_large", op="train", M=4096, N=12288, K=4096, dtype="bf16", layout="nk", act="silu"),
        # the down projection of a few sequences' next tokens, their activations in int8 already
        dict(name="int8_tokens", op="int8", M=4, N=4096, K=12288, dtype="bf16", act="none"),
        # the gated projection in int8 for a batch of sequences' next tokens
        dict(name="int8_gated_batch", op="int8", M=64, N=8192, K=4096, dtype="bf16", act="silu"),
        # odd sizes: neither rows nor the reduction fill a tile
        dict(name="int8_ragged", op="int8", M=333, N=2050, K=1531, dtype="f32", act="none"),
        # one token through a square layer: two launches' latency
        dict(name="linear8_token", op="linear8", M=1, N=4096, K=4096, x="bf16", dtype="bf16", act="none"),
        # a gated projection of a short prompt, from fp16
        dict(name="linear8_gated", op="linear8", M=512, N=8192, K=2048, x="f16", dtype="f16", act="gelu_tanh"),
        # the down projection of a long prompt
        dict(name="linear8_prompt", op="linear8", M=8192, N=4096, K=12288, x="bf16", dtype="bf16", act="none"),
    ]


def draw(rng):
    def size(lo, hi):
        # log-uniform; half of the sizes whole multiples of 64, a quarter multiples of 8,
        # the rest whatever comes
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        g = rng.choice((64, 64, 8, 1))
        return min(hi, max(lo, int(v) if v < 2 * g else int(round(v / g)) * g))

    def rows(hi):
        # a third single tokens and small batches of them, the rest anything up to `hi`
        return rng.randint(1, 16) if rng.random() < 0.34 else int(math.exp(rng.uniform(math.log(17), math.log(hi + 1))))

    op = rng.choice(("gated", "train", "int8", "linear8"))
    half = rng.choice(("bf16", "bf16", "f16"))
    act = rng.choice(("silu", "silu", "gelu_tanh", "relu"))
    layout = rng.choice(("nk", "kn"))
    if op == "gated":
        return dict(op=op, M=rows(8192), N=size(48, 12288), K=size(40, 4096), dtype=half, layout=layout, act=act)
    if op == "train":
        return dict(op=op, M=rows(4096), N=size(48, 12288), K=size(40, 4096), dtype=half, layout=layout, act=act)
    n, k = size(48, 12288), size(40, 12288)
    m = rows(min(8192, 8192 * 4096 * 12288 // (n * k)))
    case = dict(op=op, M=m, N=n, K=k, dtype=rng.choice(("bf16", "f16", "f32")), act=rng.choice(("none", "none", act)))
    if op == "linear8":
        case["x"] = rng.choice(("bf16", "f16", "f32"))
    if case["act"] != "none":
        case["N"] = max(24, n // 2)   # two products: no dearer than one of the whole width
    return case


def _normal(gen, shape, std, dtype):
    t = torch.empty(shape, dtype=torch.float32, device=gen.device)
    t.normal_(0.0, std, generator=gen)
    return t.to(dtype)


def _weight(gen, layout, n, k, dtype):
    return _normal(gen, (n, k) if layout == "nk" else (k, n), 1.0 / math.sqrt(k), dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, k = case["op"], case["M"], case["K"]
    dt = _DTYPES[case["dtype"]]
    s = dict(case=case)
    n = case["N"]
    if op in ("int8", "linear8"):
        gated = case["act"] != "none"

        def ints(r):
            t = torch.empty(r, k, dtype=torch.float32, device="cuda").normal_(0.0, 32.0, generator=gen)
            return t.round_().clamp_(-127, 127).to(torch.int8)

        def scales(r, std):
            t = torch.empty(r, dtype=torch.float32, device="cuda").uniform_(0.5, 1.5, generator=gen)
            return t * (std / 32.0)

        if op == "int8":
            s["a"], s["sa"] = ints(m), scales(m, 1.0)
        else:
            # normalised activations with a few channels ten times as large, as they come
            # out of a transformer's blocks
            x = _normal(gen, (m, k), 1.0, torch.float32)
            x[:, torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 256)]] *= 10.0
            s["x"] = x.to(_DTYPES[case["x"]])
        s["b"], s["sb"] = ints(n), scales(n, 1.0 / math.sqrt(k))
        s["b2"], s["sb2"] = (ints(n), scales(n, 1.0 / math.sqrt(k))) if gated else (None, None)
        if own:
            import software_pipelined_tiled_gemm_amd as spg
            s["plan"] = spg.QuantizedGemm(m, n, k, case["dtype"], case["act"])
            s["c"] = torch.empty(m, n, dtype=dt, device="cuda")
            if op == "linear8":
                s["a"] = torch.empty(m, k, dtype=torch.int8, device="cuda")
                s["sa"] = torch.empty(m, dtype=torch.float32, device="cuda")
            s["ws"] = torch.empty(s["plan"].workspace_bytes(), dtype=torch.uint8, device="cuda")
        return s
    s["x"] = _normal(gen, (m, k), 1.0, dt)
    s["wg"] = _weight(gen, case["layout"], n, k, dt)
    s["wu"] = _weight(gen, case["layout"], n, k, dt)
    if op == "train":
        s["dh"] = _normal(gen, (m, n), 0.1, dt)
    if own:
        import software_pipelined_tiled_gemm_amd as spg
        s["plan"] = spg.Gated(m, n, k, case["dtype"], case["layout"], case["act"])
        s["h"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["ws"] = torch.empty(s["plan"].workspace_bytes(), dtype=torch.uint8, device="cuda")
        if op == "train":
            s["g"], s["u"] = torch.empty_like(s["h"]), torch.empty_like(s["h"])
            s["dx"] = torch.empty_like(s["x"])
            s["dwg"], s["dwu"] = torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import software_pipelined_tiled_gemm_amd as spg
    op = s["case"]["op"]
    if op == "linear8":
        spg.gemm_quantize_rows(s["x"], s["a"], s["sa"])
    if op in ("int8", "linear8"):
        return s["plan"](s["a"], s["sa"], s["b"], s["sb"], s["c"], B2=s["b2"], scale_b2=s["sb2"], workspace=s["ws"])
    if op == "gated":
        return s["plan"](s["x"], s["wg"], s["wu"], s["h"], workspace=s["ws"])
    s["plan"](s["x"], s["wg"], s["wu"], s["h"], G=s["g"], U=s["u"], workspace=s["ws"])
    s["plan"].backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], s["dx"], s["dwg"], s["dwu"], workspace=s["ws"])
    return s["h"], s["dx"], s["dwg"], s["dwu"]


def _act(g, act):
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g))
    z = g if act == "silu" else 2.0 * _GELU_C * (g + _GELU_A * g * g * g)
    return g / (1.0 + torch.exp(-z))


def _act_and_slope(g, act):
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "silu":
        z, dz = g, 1.0
    else:
        z = 2.0 * _GELU_C * (g + _GELU_A * g * g * g)
        dz = 2.0 * _GELU_C * (1.0 + 3.0 * _GELU_A * g * g)
    sig = 1.0 / (1.0 + torch.exp(-z))
    return g * sig, sig + g * sig * (1.0 - sig) * dz


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    dt = _DTYPES[case["dtype"]]
    if op in ("int8", "linear8"):
        # 64 bits: the sums pass 2^24, and a quotient next to a half must fall on its side of it
        if op == "int8":
            a, sa = s["a"].double(), s["sa"].double()[:, None]
        else:
            x = s["x"].double()
            amax = x.abs().amax(dim=1, keepdim=True)
            a = torch.round(x * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
            sa = (amax / 127.0).float().double()
        c = (a @ s["b"].double().t()) * sa * s["sb"].double()
        if s["b2"] is not None:
            up = (a @ s["b2"].double().t()) * sa * s["sb2"].double()
            c = _act(c, case["act"]) * up
        return c.to(dt)
    nk = case["layout"] == "nk"
    x = s["x"].float()
    wg, wu = s["wg"].float(), s["wu"].float()
    if nk:
        wg, wu = wg.t(), wu.t()
    g, u = x @ wg, x @ wu
    if op == "gated":
        return (_act(g, case["act"]) * u).to(dt)
    a, slope = _act_and_slope(g, case["act"])
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * a
    dx = dg @ wg.t() + du @ wu.t()
    if nk:
        dwg, dwu = dg.t() @ x, du.t() @ x
    else:
        dwg, dwu = x.t() @ dg, x.t() @ du
    return (a * u).to(dt), dx.to(dt), dwg.to(dt), dwu.to(dt)


def work(case):
    op, m, k = case["op"], case["M"], case["K"]
    e, n = _SIZE[case["dtype"]], case["N"]
    if op in ("int8", "linear8"):
        w = 1 if case["act"] == "none" else 2
        a = m * (k + 4) if op == "int8" else m * k * _SIZE[case["x"]]
        return {"bytes": a + w * n * (k + 4) + m * n * e, "flops": 2 * w * m * n * k}
    x, w, h = m * k, 2 * n * k, m * n
    if op == "gated":
        return {"bytes": (x + w + h) * e, "flops": 4 * m * n * k}
    # X, Wg, Wu and dH read; H, dX, dWg and dWu written; two products forward, four backward
    return {"bytes": (2 * x + 2 * w + 2 * h) * e, "flops": 12 * m * n * k}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    f64 = torch.float64
    def gate(g, act):
        if act == "silu":
            return g * torch.sigmoid(g)
        if act == "relu":
            return g.clamp(min=0)
        return 0.5 * g * (1 + torch.tanh(_GELU_C * (g + _GELU_A * g.pow(3))))

    if op in ("int8", "linear8"):
        if op == "int8":
            rows = s["a"].to(f64) * s["sa"].to(f64).unsqueeze(1)
        else:
            x = s["x"].to(f64)
            top = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
            step = torch.where(top > 0, top, torch.ones_like(top)).unsqueeze(1)
            rows = (x.mul(127).div(step)).round() * (step / 127)

        def scaled(b, sb):
            return torch.matmul(rows, (b.to(f64) * sb.to(f64).unsqueeze(1)).transpose(0, 1))

        first = scaled(s["b"], s["sb"])
        return first if case["act"] == "none" else gate(first, case["act"]) * scaled(s["b2"], s["sb2"])
    x = s["x"].to(f64)
    as_nk = (lambda w: w.to(f64)) if case["layout"] == "nk" else (lambda w: w.to(f64).transpose(0, 1).contiguous())
    wg, wu = as_nk(s["wg"]), as_nk(s["wu"])                     # [N,K]
    g, u = torch.matmul(x, wg.transpose(0, 1)), torch.matmul(x, wu.transpose(0, 1))
    a = gate(g, case["act"])
    h = a * u
    if op == "gated":
        return h
    if case["act"] == "silu":
        t = torch.sigmoid(g)
        da = t * (1 + g * (1 - t))
    elif case["act"] == "relu":
        da = (g > 0).to(f64)
    else:
        t = torch.tanh(_GELU_C * (g + _GELU_A * g.pow(3)))
        da = 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _GELU_C * (1 + 3 * _GELU_A * g * g)
    dh = s["dh"].to(f64)
    du, dg = dh * a, dh * u * da
    dx = torch.matmul(torch.cat((dg, du), 1), torch.cat((wg, wu), 0))
    dwg, dwu = torch.matmul(dg.transpose(0, 1), x), torch.matmul(du.transpose(0, 1), x)
    if case["layout"] == "kn":
        dwg, dwu = dwg.transpose(0, 1).contiguous(), dwu.transpose(0, 1).contiguous()
    return h, dx, dwg, dwu

"""Workloads of the operators that make a feed-forward block a mixture of experts: their
inputs, one pass through each, the bytes and operations a pass cannot do without, and the
64-bit values it should give.

``norm``      Y = (X - mean) / sqrt(var + eps) * weight + bias, row by row.
``route``     every token's k experts out of E from its logits, their gates, and the rows
              (token, choice) grouped by expert: a slot per row, a source per slot, the
              groups' offsets.
``gated``     H = act(X Wg[e]) * (X Wu[e]) for the rows of every expert e, read from the
              tokens by their source.
``grouped``   Y = X W[e] for the rows of every expert e.
``combine``   out[t] = sum over j of gate[t,j] Y[slot[t,j]]: the experts' rows back to tokens.

With ``train`` a pass is the forward and the backward pass.  Tokens behind the last ``used``
one are padding: their logits are -inf, they have no rows, and the rows behind the last group
stay as they are.  ``run`` computes the plain form (elementary torch operations, 32 bits or
more, rounded once at the end) unless ``own`` is true, when it calls this package's kernels.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_GELU_C, _GELU_A = 0.7978845608, 0.044715
_EPS = 1e-5


def listed():
    return [
        # one token of a decoding step: a single row, all of it latency
        dict(name="norm_token", op="norm", train=False, M=1, K=4096, dtype="bf16", params="bf16"),
        # the norm before a block in training, its weights kept in fp32
        dict(name="norm_train", op="norm", train=True, M=8192, K=4096, dtype="bf16", params="f32"),
        # rows that start at any 2-byte address
        dict(name="norm_ragged", op="norm", train=True, M=511, K=1001, dtype="f16", params="f16"),
        # the next tokens of a few sequences, in 16 bits, where equal logits are common
        dict(name="route_tokens", op="route", train=False, T=4, used=4, E=64, k=8, dtype="bf16", renormalise=True),
        # a padded training batch
        dict(name="route_train", op="route", train=True, T=16384, used=16000, E=64, k=8, dtype="f32", renormalise=True),
        # the experts' rows of a few next tokens
        dict(name="combine_tokens", op="combine", train=False, T=4, used=4, E=64, k=8, N=2048, dtype="bf16"),
        # a training batch, with the gates' gradients
        dict(name="combine_train", op="combine", train=True, T=8192, used=8192, E=8, k=2, N=4096, dtype="bf16"),
        # one token through two of eight wide experts: the reading of their weights
        dict(name="gated_token", op="gated", train=False, T=1, used=1, E=8, k=2, N=12288, K=4096, dtype="bf16",
             layout="nk", act="silu"),
        # a prompt through many narrow experts
        dict(name="gated_prompt", op="gated", train=False, T=4096, used=4096, E=64, k=6, N=1408, K=2048, dtype="bf16",
             layout="nk", act="silu"),
        # a training step on one GPU: eight wide experts, two a token
        dict(name="gated_train", op="gated", train=True, T=4096, used=4096, E=8, k=2, N=8192, K=4096, dtype="bf16",
             layout="nk", act="silu"),
        # the down projection of a decoding batch: a few rows an expert, all of the experts
        dict(name="grouped_batch", op="grouped", train=False, T=64, used=64, E=64, k=8, N=2048, K=1408, dtype="bf16",
             layout="nk"),
        # odd sizes throughout, padded, weights stored [K,N]
        dict(name="grouped_ragged", op="grouped", train=True, T=700, used=651, E=5, k=2, N=500, K=1365, dtype="f16",
             layout="kn"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    def size(lo, hi):
        # log-uniform; half of the sizes whole multiples of 64, a quarter multiples of 8,
        # the rest whatever comes
        v, g = log(lo, hi), rng.choice((64, 64, 8, 1))
        return min(hi, max(lo, v if v < 2 * g else int(round(v / g)) * g))

    def tokens(hi):
        # a third single tokens and small batches of them, the rest anything up to `hi`
        t = rng.randint(1, 16) if rng.random() < 0.34 else log(17, hi)
        return t, (t if rng.random() < 0.6 else rng.randint(max(1, t // 2), t))

    op = rng.choice(("norm", "route", "combine", "gated", "gated", "grouped", "grouped"))
    train = rng.random() < 0.5
    half = rng.choice(("bf16", "bf16", "f16"))
    if op == "norm":
        k = size(24, 16384)
        dtype = rng.choice((half, half, "f32"))
        return dict(op=op, train=train, M=tokens(min(32768, 8192 * 4096 // k))[0], K=k, dtype=dtype,
                    params=rng.choice((dtype, "f32")))
    e = rng.choice((log(2, 256), 8, 64, 128))
    k = rng.randint(1, min(8, e))
    if op == "route":
        t, used = tokens(16384)
        return dict(op=op, train=train, T=t, used=used, E=e, k=k, dtype=rng.choice(("f32", half)),
                    renormalise=rng.random() < 0.5)
    if op == "combine":
        n = size(24, 8192)
        t, used = tokens(max(17, 8192 * 2 * 4096 // (k * n)))
        return dict(op=op, train=train, T=t, used=used, E=e, k=k, N=n, dtype=rng.choice((half, half, "f32")))
    n, d = size(48, 12288), size(40, 4096)
    while e * n * d > 8 * 8192 * 4096:      # no more weights than the largest listed case
        n, d = max(48, n // 2), max(40, d // 2)
    t, used = tokens(max(17, 8192 // k))
    case = dict(op=op, train=train, T=t, used=used, E=e, k=k, N=n, K=d, dtype=half, layout=rng.choice(("nk", "kn")))
    if op == "gated":
        case["act"] = rng.choice(("silu", "silu", "gelu_tanh", "relu"))
    return case


def _normal(gen, shape, std, dtype):
    t = torch.empty(shape, dtype=torch.float32, device=gen.device)
    return t.normal_(0.0, std, generator=gen).to(dtype)


def _group(gen, case):
    """k different experts for every used token, some experts liked better than others:
    source of every row, rows' slots [T,k] (-1: padding), offsets on the GPU and here."""
    t, e, k, used = case["T"], case["E"], case["k"], case["used"]
    score = torch.empty(used, e, device="cuda").uniform_(0.0, 1.0, generator=gen)
    score += torch.empty(e, device="cuda").uniform_(0.0, 0.25, generator=gen)
    chosen = score.argsort(dim=1, descending=True, stable=True)[:, :k].reshape(-1)
    order = chosen.argsort(stable=True)
    slot = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
    slot[order] = torch.arange(used * k, dtype=torch.int32, device="cuda")
    source = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
    source[: used * k] = (order // k).int()
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(chosen, minlength=e).cumsum(0).int()
    return source, slot.view(t, k), offsets, offsets.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, train, dt = case["op"], case["train"], _DTYPES[case["dtype"]]
    s = dict(case=case)
    if own:
        import software_pipelined_tiled_gemm_amd as spg

    def new(*shape, dtype=dt, fill=0):
        return torch.full(shape, fill, dtype=dtype, device="cuda")

    def scratch(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    if op == "norm":
        m, k, pt = case["M"], case["K"], _DTYPES[case["params"]]
        # a residual stream: rows of their own mean and size
        x = _normal(gen, (m, k), 1.0, torch.float32)
        s["x"] = (x * _normal(gen, (m, 1), 1.0, torch.float32).exp_() + _normal(gen, (m, 1), 0.5, torch.float32)).to(dt)
        s["w"] = (1.0 + _normal(gen, (k,), 0.2, torch.float32)).to(pt)
        s["b"] = _normal(gen, (k,), 0.2, pt)
        if train:
            s["dy"] = _normal(gen, (m, k), 0.1, dt)
        if own:
            s["plan"] = spg.LayerNorm(m, k, case["dtype"], case["params"], eps=_EPS)
            s["y"] = new(m, k)
            if train:
                s["mean"], s["rstd"] = new(m, dtype=torch.float32), new(m, dtype=torch.float32)
                s["dx"], s["dw"], s["db"] = new(m, k), new(k, dtype=pt), new(k, dtype=pt)
                s["ws"] = scratch(s["plan"].workspace_bytes())
        return s
    t, e, k = case["T"], case["E"], case["k"]
    if op == "route":
        s["logits"] = _normal(gen, (t, e), 1.5, dt)
        s["logits"][case["used"]:] = float("-inf")
        if train:
            s["dgate"] = _normal(gen, (t, k), 0.1, torch.float32)
        if own:
            s["plan"] = spg.Router(t, e, k, case["dtype"], renormalise=case["renormalise"])
            s["gate"] = new(t, k, dtype=torch.float32)
            s["expert"], s["slot"] = new(t, k, dtype=torch.int32), new(t, k, dtype=torch.int32)
            s["source"] = new(t * k, dtype=torch.int32, fill=-1)
            s["offsets"] = new(e + 1, dtype=torch.int32)
            s["ws"] = scratch(s["plan"].workspace_bytes())
            if train:
                s["dlogits"] = new(t, e)
        return s
    s["source"], s["slot"], s["offsets"], s["host"] = _group(gen, case)
    rows, n = t * k, case["N"]
    if op == "combine":
        s["y"] = _normal(gen, (rows, n), 1.0, dt)
        s["gate"] = torch.empty(t, k, device="cuda").uniform_(0.05, 0.6, generator=gen)
        if train:
            s["dout"] = _normal(gen, (t, n), 0.1, dt)
        if own:
            s["plan"] = spg.Combine(t, k, rows, n, case["dtype"])
            s["out"] = new(t, n)
            if train:
                s["dy"], s["dgate"] = new(rows, n), new(t, k, dtype=torch.float32)
        return s
    d = case["K"]
    shape = (e, n, d) if case["layout"] == "nk" else (e, d, n)
    std = 1.0 / math.sqrt(d)
    if op == "grouped":
        s["x"], s["w"] = _normal(gen, (rows, d), 1.0, dt), _normal(gen, shape, std, dt)
        if train:
            s["dy"] = _normal(gen, (rows, n), 0.1, dt)
        if own:
            s["plan"] = spg.GroupedGemm(rows, n, d, e, case["dtype"], case["layout"])
            s["y"] = new(rows, n)
            s["ws"] = scratch(s["plan"].workspace_bytes(backward=train))
            if train:
                s["dx"], s["dw"] = new(rows, d), torch.empty_like(s["w"])
        return s
    s["x"] = _normal(gen, (t, d), 1.0, dt)
    s["wg"], s["wu"] = _normal(gen, shape, std, dt), _normal(gen, shape, std, dt)
    if train:
        s["dh"] = _normal(gen, (rows, n), 0.1, dt)
    if own:
        s["plan"] = spg.GroupedGated(rows, n, d, e, case["dtype"], case["layout"], case["act"], tokens=t)
        s["h"] = new(rows, n)
        s["ws"] = scratch(s["plan"].workspace_bytes(backward=train))
        if train:
            s["g"], s["u"], s["dx"] = new(rows, n), new(rows, n), new(rows, d)
            s["dwg"], s["dwu"] = torch.empty_like(s["wg"]), torch.empty_like(s["wu"])
    return s


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state, state["case"])


def _run_own(s):
    op, train, plan = s["case"]["op"], s["case"]["train"], s["plan"]
    if op == "norm":
        if not train:
            return plan(s["x"], s["w"], s["b"], s["y"])
        plan(s["x"], s["w"], s["b"], s["y"], mean=s["mean"], rstd=s["rstd"])
        plan.backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"], workspace=s["ws"])
        return s["y"], s["dx"], s["dw"], s["db"]
    if op == "route":
        plan(s["logits"], s["gate"], s["expert"], s["slot"], s["source"], s["offsets"], workspace=s["ws"])
        out = s["gate"], s["expert"], s["slot"], s["source"], s["offsets"]
        if not train:
            return out
        plan.backward(s["logits"], s["expert"], s["dgate"], s["dlogits"])
        return out + (s["dlogits"],)
    if op == "combine":
        plan(s["y"], s["slot"], s["gate"], s["out"])
        if not train:
            return s["out"]
        plan.backward(s["dout"], s["y"], s["slot"], s["gate"], s["dy"], s["dgate"])
        return s["out"], s["dy"], s["dgate"]
    if op == "grouped":
        plan(s["x"], s["w"], s["offsets"], s["y"], workspace=s["ws"])
        if not train:
            return s["y"]
        plan.backward(s["dy"], s["x"], s["w"], s["offsets"], s["dx"], s["dw"], workspace=s["ws"])
        return s["y"], s["dx"], s["dw"]
    if not train:
        return plan(s["x"], s["wg"], s["wu"], s["offsets"], s["h"], source=s["source"], workspace=s["ws"])
    plan(s["x"], s["wg"], s["wu"], s["offsets"], s["h"], source=s["source"], G=s["g"], U=s["u"], workspace=s["ws"])
    plan.backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], s["offsets"], s["dx"], s["dwg"], s["dwu"],
                  source=s["source"], workspace=s["ws"])
    return s["h"], s["dx"], s["dwg"], s["dwu"]


def _plain_norm(s, case):
    x = s["x"].float()
    k = case["K"]
    w, b = s["w"].float(), s["b"].float()
    c = x - x.sum(1, keepdim=True) / k
    r = 1.0 / torch.sqrt((c * c).sum(1, keepdim=True) / k + _EPS)
    n = c * r
    y = (n * w + b).to(s["x"].dtype)
    if not case["train"]:
        return y
    dy = s["dy"].float()
    g = dy * w
    dx = r * (g - g.sum(1, keepdim=True) / k - n * ((g * n).sum(1, keepdim=True) / k))
    return y, dx.to(y.dtype), (dy * n).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype)


def _plain_route(s, case):
    t, e, k = case["T"], case["E"], case["k"]
    dev = s["logits"].device
    x = s["logits"].float()
    # the k largest, the lowest index first among equals
    expert = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    value = x.gather(1, expert)
    live = value > float("-inf")
    top = x.amax(1, keepdim=True)
    top = torch.where(top > float("-inf"), top, torch.zeros_like(top))
    p = torch.exp(x - top)
    total = (torch.exp(value - top) if case["renormalise"] else p).sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    gate = torch.exp(value - top) / total
    group = torch.where(live, expert, torch.full_like(expert, e)).reshape(-1)
    order = group.sort(stable=True).indices
    slot = torch.empty(t * k, dtype=torch.int32, device=dev)
    slot[order] = torch.arange(t * k, dtype=torch.int32, device=dev)
    slot = torch.where(live, slot.view(t, k), -1)
    count = (group[:, None] == torch.arange(e, device=dev)).sum(0)
    offsets = torch.cat((torch.zeros_like(count[:1]), count.cumsum(0))).int()
    source = torch.where(group[order] < e, order // k, -1).int()
    out = gate, torch.where(live, expert, -1).int(), slot, source, offsets
    if not case["train"]:
        return out
    dg = torch.where(live, s["dgate"], torch.zeros_like(gate))
    inner = (gate * dg).sum(1, keepdim=True)
    if case["renormalise"]:
        d = torch.zeros_like(x).scatter_(1, expert, gate * (dg - inner))
    else:
        d = (p / total) * (torch.zeros_like(x).scatter_(1, expert, dg) - inner)
    return out + (d.to(s["logits"].dtype),)


def _plain_combine(s, case):
    t, n, slot = case["T"], case["N"], s["slot"]
    dt = s["y"].dtype
    live = (slot >= 0).unsqueeze(2)
    rows = torch.where(live, s["y"].float()[slot.clamp(min=0).long()], 0.0)           # [T,k,N]
    gate = torch.where(slot >= 0, s["gate"], 0.0)
    out = (gate.unsqueeze(2) * rows).sum(1).to(dt)
    if not case["train"]:
        return out
    do = s["dout"].float()
    dgate = (rows * do.unsqueeze(1)).sum(2)
    dy = torch.zeros(t * case["k"], n, dtype=dt, device=do.device)
    used = case["used"]
    dy[slot[:used].reshape(-1).long()] = (gate.unsqueeze(2) * do.unsqueeze(1))[:used].reshape(-1, n).to(dt)
    return out, dy, dgate


def _kn(w, layout):
    return w.float().t() if layout == "nk" else w.float()


def _plain_grouped(s, case):
    rows, host, lay = case["T"] * case["k"], s["host"], case["layout"]
    dt, dev = s["x"].dtype, s["x"].device
    y = torch.zeros(rows, case["N"], dtype=dt, device=dev)
    if case["train"]:
        dx, dw = torch.zeros(rows, case["K"], dtype=dt, device=dev), torch.zeros_like(s["w"])
    for e in range(case["E"]):
        a, b = host[e], host[e + 1]
        if a == b:
            continue
        x, w = s["x"][a:b].float(), _kn(s["w"][e], lay)
        y[a:b] = (x @ w).to(dt)
        if case["train"]:
            dy = s["dy"][a:b].float()
            dx[a:b] = (dy @ w.t()).to(dt)
            dw[e] = (dy.t() @ x if lay == "nk" else x.t() @ dy).to(dt)
    return (y, dx, dw) if case["train"] else y


def _act(g, act):
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


def _plain_gated(s, case):
    rows, host, lay = case["T"] * case["k"], s["host"], case["layout"]
    dt, dev = s["x"].dtype, s["x"].device
    h = torch.zeros(rows, case["N"], dtype=dt, device=dev)
    if case["train"]:
        dx = torch.zeros(rows, case["K"], dtype=dt, device=dev)
        dwg, dwu = torch.zeros_like(s["wg"]), torch.zeros_like(s["wu"])
    for e in range(case["E"]):
        a, b = host[e], host[e + 1]
        if a == b:
            continue
        x = s["x"][s["source"][a:b]].float()
        wg, wu = _kn(s["wg"][e], lay), _kn(s["wu"][e], lay)
        g, u = x @ wg, x @ wu
        act, slope = _act(g, case["act"])
        h[a:b] = (act * u).to(dt)
        if case["train"]:
            dh = s["dh"][a:b].float()
            dg, du = dh * u * slope, dh * act
            dx[a:b] = (dg @ wg.t() + du @ wu.t()).to(dt)
            dwg[e] = (dg.t() @ x if lay == "nk" else x.t() @ dg).to(dt)
            dwu[e] = (du.t() @ x if lay == "nk" else x.t() @ du).to(dt)
    return (h, dx, dwg, dwu) if case["train"] else h


_PLAIN = {"norm": _plain_norm, "route": _plain_route, "combine": _plain_combine, "grouped": _plain_grouped,
          "gated": _plain_gated}


def work(case):
    op, train, z = case["op"], case["train"], _SIZE[case["dtype"]]
    if op == "norm":
        m, k, p = case["M"], case["K"], _SIZE[case["params"]]
        # x, weight and bias read, y written; training: x and dy again, dx and the parameters' gradients
        return {"bytes": (4 if train else 2) * m * k * z + (4 if train else 2) * k * p, "flops": (20 if train else 8) * m * k}
    t, e, k, used = case["T"], case["E"], case["k"], case["used"]
    rows = used * k
    if op == "route":
        fwd = t * e * z + t * k * 12 + rows * 4 + (e + 1) * 4
        return {"bytes": fwd + (t * k * 4 + t * e * z if train else 0), "flops": (8 if train else 4) * t * e}
    n = case["N"]
    if op == "combine":
        fwd = rows * n * z + t * k * 8 + t * n * z
        return {"bytes": fwd + (t * n * z + rows * n * z + t * k * 4 if train else 0), "flops": (5 if train else 2) * rows * n}
    d = case["K"]
    # experts that have a row, on average: their weights are read (all gradients are written)
    live = e * (1.0 - (1.0 - k / e) ** used)
    w = (2 if op == "gated" else 1) * n * d * z
    x = used if op == "gated" else rows
    fwd = int(live * w) + x * d * z + rows * n * z + (e + 1) * 4 + (rows * 4 if op == "gated" else 0)
    one = 2 * rows * n * d * (2 if op == "gated" else 1)
    if not train:
        return {"bytes": fwd, "flops": one}
    return {"bytes": fwd + rows * n * z + rows * d * z + e * w, "flops": 3 * one}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op, train, f64 = case["op"], case["train"], torch.float64
    if op == "norm":
        x, w = s["x"].to(f64), s["w"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        std = torch.sqrt(var + _EPS)
        n = (x - mean) / std
        y = torch.addcmul(s["b"].to(f64), n, w)
        if not train:
            return y
        dy = s["dy"].to(f64)
        g = dy * w
        dx = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) / std
        return y, dx, torch.sum(n * dy, 0), torch.sum(dy, 0)
    t, e, k, used = case["T"], case["E"], case["k"], case["used"]
    if op == "route":
        return _exact_route(s, case)
    rows, n = t * k, case["N"]
    if op == "combine":
        # the padding's slots point at a row of zeros
        y = torch.cat((s["y"].to(f64), torch.zeros(1, n, dtype=f64, device="cuda")))
        slot = torch.where(s["slot"] < 0, rows, s["slot"]).long()
        gate = s["gate"].to(f64)
        out = torch.zeros(t, n, dtype=f64, device="cuda")
        for j in range(k):
            out += gate[:, j:j + 1] * y[slot[:, j]]
        if not train:
            return out
        do = s["dout"].to(f64)
        dy = torch.zeros(rows + 1, n, dtype=f64, device="cuda")
        dgate = torch.empty(t, k, dtype=f64, device="cuda")
        for j in range(k):
            dgate[:, j] = torch.sum(do * y[slot[:, j]], 1)
            dy[slot[:, j]] = gate[:, j:j + 1] * do
        return out, dy[:rows], dgate
    d, host, nk = case["K"], s["host"], case["layout"] == "nk"

    def put(grad, e_, m):      # m is [N,K]
        grad[e_] = m if nk else m.transpose(0, 1)

    def zeros(*shape):
        return torch.zeros(shape, dtype=f64, device="cuda")

    def weight(w):             # as [N,K]
        return w.to(f64) if nk else w.to(f64).transpose(0, 1).contiguous()

    first = zeros(rows, n)
    names = ("w",) if op == "grouped" else ("wg", "wu")
    dx = zeros(rows, d) if train else None
    dw = [zeros(*s[w].shape) for w in names] if train else []
    for i in range(e):
        r = slice(host[i], host[i + 1])
        if host[i] == host[i + 1]:
            continue
        if op == "grouped":
            x, w = s["x"][r].to(f64), weight(s["w"][i])
            first[r] = torch.matmul(x, w.transpose(0, 1))
            if train:
                dy = s["dy"][r].to(f64)
                dx[r] = torch.matmul(dy, w)
                put(dw[0], i, torch.matmul(dy.transpose(0, 1), x))
            continue
        x = s["x"].to(f64)[s["source"][r].long()]
        wg, wu = weight(s["wg"][i]), weight(s["wu"][i])
        g, u = torch.matmul(x, wg.transpose(0, 1)), torch.matmul(x, wu.transpose(0, 1))
        if case["act"] == "relu":
            a, da = g.clamp(min=0), (g > 0).to(f64)
        elif case["act"] == "silu":
            q = torch.sigmoid(g)
            a, da = g * q, q * (1 + g * (1 - q))
        else:
            q = torch.tanh(_GELU_C * (g + _GELU_A * g.pow(3)))
            a = 0.5 * g * (1 + q)
            da = 0.5 * (1 + q) + 0.5 * g * (1 - q * q) * _GELU_C * (1 + 3 * _GELU_A * g * g)
        first[r] = a * u
        if train:
            dh = s["dh"][r].to(f64)
            dg, du = dh * u * da, dh * a
            dx[r] = torch.matmul(torch.cat((dg, du), 1), torch.cat((wg, wu), 0))
            put(dw[0], i, torch.matmul(dg.transpose(0, 1), x))
            put(dw[1], i, torch.matmul(du.transpose(0, 1), x))
    return (first, dx, *dw) if train else first


def _exact_route(s, case):
    t, e, k, used = case["T"], case["E"], case["k"], case["used"]
    x = s["logits"].to(torch.float64)
    left = x.clone()
    row = torch.arange(t, device="cuda")
    expert = torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    picked = torch.zeros(t, e, dtype=torch.bool, device="cuda")
    column = torch.arange(e, device="cuda").expand(t, e)
    for j in range(k):
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, column, e).amin(1)           # the lowest index among equals
        expert[:used, j] = at[:used].int()
        picked[row[:used], at[:used]] = True
        left[row, at] = float("-inf")
    share = torch.where(picked, x, float("-inf")) if case["renormalise"] else x
    p = torch.zeros_like(x)
    p[:used] = torch.softmax(share[:used], dim=1)
    index = expert.clamp(min=0).long()
    gate = p.gather(1, index)
    gate[used:] = 0
    count = picked.sum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(count, 0).int()
    # a row's place: its group's start and the earlier tokens of that group
    before = torch.cumsum(picked.int(), 0) - picked.int()
    slot = (offsets[:-1] + before).gather(1, index).int()
    slot[used:] = -1
    source = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
    source[slot[:used].reshape(-1).long()] = row[:used].repeat_interleave(k).int()
    out = gate, expert, slot, source, offsets
    if not case["train"]:
        return out
    dp = torch.zeros_like(x).scatter_add_(1, index, s["dgate"].to(torch.float64))
    dp[used:] = 0
    return out + (p * (dp - torch.sum(p * dp, 1, keepdim=True)),)

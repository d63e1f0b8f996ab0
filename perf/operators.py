"""Cases of the routing and 4-bit operators: their inputs, plain forms and exact results.

Four operators of a served mixture-of-experts layer, each with its plain form in elementary torch
operations and, where `own` is true, the framework's call:

  route    scores, groups, top-K and weights from router logits
  quant    weights into 4-bit codes with group scales, and back
  linear   y = x W^T with 4-bit weights (one matrix)
  experts  the grouped SwiGLU FFN of routed and shared experts with 4-bit weights

The 4-bit format: W[r][c] = (q[r][c] - z[r][c // g]) * s[r][c // g], q and z in 0..15 (z = 8 where no
zero points are held), s in BF16, g = 32, 64 or 128. Codes are stored in 64 bytes for each row and
128 columns: sixteen 32-bit words of eight columns, word v at place 4 * (v % 4) + v // 4; inside a word
column 2i is at bits 4i and column 2i + 1 at bits 16 + 4i.
"""
import torch

own = False

E, K, D, I = 384, 6, 2560, 512      # the layer's experts, choices, width and expert width


def listed():
    return [
        # one token of one sequence: the call's latency
        dict(name="route-one-token", op="route", n=1, e=E, k=K, score="sigmoid", groups=1, keep=1, by="max", renorm=True,
             scale=1.0, bias=True, masked=0, dtype="f32"),
        # a decode batch with groups, as models that limit a token to some groups of experts route
        dict(name="route-decode", op="route", n=32, e=E, k=K, score="sigmoid", groups=8, keep=4, by="top2", renorm=True,
             scale=2.5, bias=True, masked=0, dtype="f32"),
        # a prefill chunk, softmax scores without a bias, logits in BF16, a few experts switched off
        dict(name="route-prefill", op="route", n=8192, e=E, k=K, score="softmax", groups=8, keep=3, by="max", renorm=False,
             scale=1.0, bias=False, masked=5, dtype="bf16"),
        # the longest batch of the layer's workloads
        dict(name="route-long", op="route", n=65536, e=E, k=K, score="sigmoid", groups=8, keep=4, by="top2", renorm=True,
             scale=2.5, bias=True, masked=0, dtype="f32"),
        # one expert's projection, symmetric codes
        dict(name="quant-matrix", op="quant", rows=I, cols=D, g=128, zeros=False, dtype="bf16"),
        # the projections of 64 experts held in FP32, with zero points
        dict(name="quant-experts", op="quant", rows=64 * I, cols=D, g=32, zeros=True, dtype="f32"),
        # a matrix-vector product of one token
        dict(name="linear-one-token", op="linear", n=1, rows=I, cols=D, g=128, zeros=False, out="f32"),
        # a ragged output width, a few tokens, small groups with zero points
        dict(name="linear-ragged", op="linear", n=13, rows=6001, cols=D, g=32, zeros=True, out="bf16"),
        # one token through its experts: latency of the whole FFN
        dict(name="experts-one-token", op="experts", n=1, d=D, i=I, e=E, k=K, g=128, zeros=False, skew=0.0, shared=True),
        # a decode batch
        dict(name="experts-decode", op="experts", n=32, d=D, i=I, e=E, k=K, g=128, zeros=False, skew=0.0, shared=True),
        # a large decode batch whose experts are unevenly popular, with zero points
        dict(name="experts-batch", op="experts", n=250, d=D, i=I, e=E, k=K, g=64, zeros=True, skew=0.5, shared=True),
        # a prefill chunk
        dict(name="experts-prefill", op="experts", n=4096, d=D, i=I, e=E, k=K, g=128, zeros=False, skew=0.0, shared=True),
    ]


def _between(rng, lo, hi):
    """A whole number, spread evenly over the logarithm of lo..hi."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("route", "quant", "linear", "experts"))
    g, zeros = rng.choice((32, 64, 128)), rng.random() < 0.5
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8, 6, 16))
        size = max(8, _between(rng, 16, 512) // groups)
        keep = rng.randint(1, groups)
        return dict(op=op, n=_between(rng, 1, 50000), e=groups * size, k=rng.randint(1, min(8, size)),
                    score=rng.choice(("sigmoid", "softmax")), groups=groups, keep=keep, by=rng.choice(("max", "top2")),
                    renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)), bias=rng.random() < 0.7,
                    masked=rng.choice((0, 0, 3)), dtype=rng.choice(("f32", "bf16")))
    if op == "quant":
        return dict(op=op, rows=_between(rng, 1, 30000), cols=128 * _between(rng, 1, 20), g=g, zeros=zeros,
                    dtype=rng.choice(("f32", "bf16")))
    if op == "linear":
        return dict(op=op, n=_between(rng, 1, 300), rows=_between(rng, 16, 6000), cols=128 * _between(rng, 1, 40), g=g,
                    zeros=zeros, out=rng.choice(("f32", "bf16")))
    return dict(op=op, n=_between(rng, 1, 3000), d=256 * rng.randint(2, 10), i=128 * rng.randint(1, 4),
                e=rng.choice((16, 61, 128, 256, 384)), k=rng.randint(1, 8), g=g, zeros=zeros,
                skew=rng.choice((0.0, 0.5)), shared=rng.random() < 0.8)


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]        # columns of a word in the order of its nibbles


def _pack(q):
    """Codes 0..15 [..., cols] (uint8) -> bytes [..., cols / 2] in the stored order."""
    w = q.unflatten(-1, (-1, 4, 4, 8)).transpose(-2, -3)[..., ORDER]
    return (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-4).contiguous()


def _unpack(codes):
    """The reverse of _pack."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    w = torch.empty_like(n).unflatten(-1, (-1, 4, 4, 8))
    w[..., ORDER] = n.unflatten(-1, (-1, 4, 4, 8))
    return w.transpose(-2, -3).flatten(-4)


def _quant(w, g, zeros):
    """The format of FP32 or BF16 w [..., cols]: codes 0..15, scales, zero points or None."""
    b = w.float().unflatten(-1, (-1, g))
    hi, lo = b.amax(-1).clamp(min=0), b.amin(-1).clamp(max=0)
    span = hi - lo if zeros else torch.maximum(hi, -lo)
    s = (span / torch.full_like(span, 15.0 if zeros else 7.0)).bfloat16()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = torch.round(-lo / s.float()).clamp(0, 15) if zeros else torch.full_like(lo, 8.0)
    q = (torch.round(b / s.float().unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
    return q.to(torch.uint8).flatten(-2), s, z.to(torch.uint8) if zeros else None


def _values(codes, s, z):
    """FP32 values of stored codes [..., cols / 2] with scales and zero points [..., cols / g]."""
    q = _unpack(codes).unflatten(-1, (s.shape[-1], -1)).float()
    q = q - (8.0 if z is None else z.unsqueeze(-1).float())
    return (q * s.unsqueeze(-1).float()).flatten(-2)


def _matrix(gen, lead, rows, cols, c):
    """Quantised weights of a trained layer's spread: N(0, 0.02)."""
    codes = torch.empty((lead, rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((lead, rows, cols // c["g"]), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((lead, rows, cols // c["g"]), dtype=torch.uint8, device="cuda") if c["zeros"] else None
    step = max(1, (1 << 26) // (rows * cols))
    for a in range(0, lead, step):
        n = min(step, lead - a)
        w = torch.randn((n, rows, cols), device="cuda", generator=gen) * 0.02
        if c["zeros"]:
            w += 0.01               # weights that are not centred, which zero points are for
        q, s[a:a + n], zz = _quant(w, c["g"], c["zeros"])
        codes[a:a + n] = _pack(q)
        if c["zeros"]:
            z[a:a + n] = zz
    return codes, s, z


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    if c["op"] == "route":
        c["logits"] = normal(c["n"], c["e"]).to(DTYPES[c["dtype"]])
        c["b"] = torch.rand(c["e"], device="cuda", generator=gen) * 0.2 - 0.1 if c["bias"] else None
        off = torch.randperm(c["e"], device="cuda", generator=gen)[:c["masked"]]
        if c["bias"]:
            c["b"][off] = float("-inf")             # switched off for every token
        else:
            c["logits"][:, off] = float("-inf")
    elif c["op"] == "quant":
        c["w"] = (normal(c["rows"], c["cols"]) * 0.02 + (0.01 if c["zeros"] else 0.0)).to(DTYPES[c["dtype"]])
    elif c["op"] == "linear":
        c["x"] = normal(c["n"], c["cols"]).bfloat16()
        codes, s, z = _matrix(gen, 1, c["rows"], c["cols"], c)
        c["codes"], c["s"], c["z"] = codes[0], s[0], None if z is None else z[0]
    else:
        n, d, i, e, k = c["n"], c["d"], c["i"], c["e"], c["k"]
        c["x"] = normal(n, d).bfloat16()
        popular = torch.log(torch.randperm(e, device="cuda", generator=gen).float() + 1.0) * -c["skew"]
        idx = torch.topk(normal(n, e) + popular, k, dim=1).indices
        flat = idx.flatten()
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=e)
        ends = counts.cumsum(0)
        c["offsets"] = torch.cat((ends.new_zeros(1), ends)).int()
        c["perm"] = (order // k).int()
        # the plain form's plan: experts that have rows, and their rows padded to the longest
        c["active"] = counts.nonzero().flatten()
        longest = int(counts.max())
        first = (ends - counts)[c["active"]]
        c["rows"] = (first[:, None] + torch.arange(longest, device="cuda")).clamp(max=n * k - 1)
        where = torch.empty(e, dtype=torch.long, device="cuda")
        where[c["active"]] = torch.arange(len(c["active"]), device="cuda")
        c["place"] = where[flat[order]] * longest + torch.arange(n * k, device="cuda") - (ends - counts)[flat[order]]
        g_, u_, d_ = (_matrix(gen, e + 1, r, cc, c) for r, cc in ((i, d), (i, d), (d, i)))
        c["layer"] = dict(w_gate=g_[0], s_gate=g_[1], z_gate=g_[2], w_up=u_[0], s_up=u_[1], z_up=u_[2],
                          w_down=d_[0], s_down=d_[1], z_down=d_[2])
    return c


def run(state):
    c = state
    if own:
        return _own(c)
    if c["op"] == "route":
        return _plain_route(c)
    if c["op"] == "quant":
        q, s, z = _quant(c["w"], c["g"], c["zeros"])
        out = dict(values=_values(_pack(q), s, z).to(c["w"].dtype), scales=s)
        return dict(out, zeros=z) if c["zeros"] else out
    if c["op"] == "linear":
        return (c["x"].float() @ _values(c["codes"], c["s"], c["z"]).t()).to(DTYPES[c["out"]])
    return _plain_experts(c)


def _plain_route(c):
    l = c["logits"].double()            # scores decide between neighbours
    b = torch.zeros(c["e"], device=l.device) if c["b"] is None else c["b"]
    l = torch.where(torch.isnan(l), float("-inf"), l)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(-1, keepdim=True)
        p = torch.exp(l - torch.where(torch.isinf(top), 0.0, top))
        total = p.sum(-1, keepdim=True)
        s = p / torch.where(total > 0, total, 1.0)
    masked = torch.isinf(l) & (l < 0) | torch.isnan(b) | (torch.isinf(b) & (b < 0))
    choice = torch.where(masked, float("-inf"), s + b.double())
    in_groups = choice.unflatten(-1, (c["groups"], -1))
    best = in_groups.sort(-1, descending=True).values
    score = best[..., 0]
    if c["by"] == "top2" and best.shape[-1] > 1:
        score = score + torch.where(torch.isinf(best[..., 1]), 0.0, best[..., 1])
    kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
    stays = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
    # an expert outside the kept groups comes behind the masked ones inside them
    rank = torch.where(stays.unsqueeze(-1).expand_as(in_groups).flatten(-2), choice.clamp(min=-1e300), float("-inf"))
    idx = rank.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.where(masked, 0.0, s).gather(1, idx)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return dict(idx=idx.int(), w=(w * c["scale"]).float())


def _plain_experts(c):
    L, a = c["layer"], c["active"]

    def ffn(x, which):          # x [experts, tokens, d]
        def w(m):
            z = L["z_" + m]
            return _values(L["w_" + m][which], L["s_" + m][which], None if z is None else z[which])
        gate, up = torch.bmm(x, w("gate").mT), torch.bmm(x, w("up").mT)
        return torch.bmm(gate / (1.0 + torch.exp(-gate)) * up, w("down").mT)

    x = c["x"].float()
    y = ffn(x[c["perm"].long()[c["rows"]]], a).flatten(0, 1)[c["place"]]
    out = dict(routed=y.bfloat16())
    if c["shared"]:
        out["shared"] = ffn(x[None], slice(c["e"], c["e"] + 1))[0].bfloat16()
    return out


def _own(c):
    from fine_grained_sparse_fp32_b200 import kmoe
    if c["op"] == "route":
        if "plan" not in c:
            c["plan"] = kmoe.Routing(score=c["score"], n_groups=c["groups"], topk_groups=c["keep"], group_score=c["by"],
                                     renormalise=c["renorm"], scale=c["scale"])
        idx, w = kmoe.moe_route(c["logits"], c["k"], bias=c["b"], routing=c["plan"])
        return dict(idx=idx, w=w)
    if c["op"] == "quant":
        w4 = kmoe.moe_quant_w4(c["w"], group=c["g"], zeros=c["zeros"])
        out = dict(values=kmoe.moe_dequant_w4(w4, dtype=c["w"].dtype), scales=w4.scales)
        return dict(out, zeros=w4.zeros) if c["zeros"] else out
    if c["op"] == "linear":
        if "plan" not in c:
            c["plan"] = kmoe.W4(c["codes"], c["s"], c["z"])
        return kmoe.moe_linear_w4(c["x"], c["plan"], y_dtype=DTYPES[c["out"]])
    if "plan" not in c:
        from fine_grained_sparse_fp32_b200.inputs import LayerConfig
        cfg = LayerConfig("w4", c["n"], c["d"], c["e"], c["k"], c["i"], "bf16", "w4")
        c["plan"] = kmoe.Layer(dict(c["layer"], cfg=cfg), max_tokens=c["n"])
    y, ys = c["plan"].grouped_ffn(c["x"], c["perm"], c["offsets"], with_shared=c["shared"])
    return dict(routed=y, shared=ys) if c["shared"] else dict(routed=y)


def work(case):
    c = case
    if c["op"] == "route":
        return dict(bytes=c["n"] * c["e"] * (4 if c["dtype"] == "f32" else 2) + c["n"] * c["k"] * 8, flops=8 * c["n"] * c["e"])
    if c["op"] == "quant":
        n = c["rows"] * c["cols"]
        # read w, write and read the format, write the values
        return dict(bytes=n * (4 if c["dtype"] == "f32" else 2) * 2 + 2 * _stored(n, c), flops=6 * n)
    if c["op"] == "linear":
        n = c["rows"] * c["cols"]
        return dict(bytes=_stored(n, c) + c["n"] * (c["cols"] * 2 + c["rows"] * (4 if c["out"] == "f32" else 2)),
                    flops=2 * n * c["n"])
    one = 3 * c["d"] * c["i"]
    touched = c["e"] * (1 - (1 - c["k"] / c["e"]) ** c["n"]) + c["shared"]
    rows = c["n"] * (c["k"] + c["shared"])
    return dict(bytes=touched * _stored(one, c) + c["n"] * c["d"] * 2 + rows * c["d"] * 2, flops=2 * one * rows)


def _stored(n, c):
    return n / 2 + n / c["g"] * (3 if c["zeros"] else 2)


def exact(case, seed):
    """From the definitions, in 64 bits, one row of scores, one matrix or one expert at a time."""
    c = prepare(case, seed)

    def decode(codes, s, z):
        """Codes [rows, cols / 2] by arithmetic on the words."""
        word = codes.view(torch.int32).long() & 0xffffffff
        n = word.shape[1] * 8
        col = torch.arange(n, device="cuda")
        v = col % 128 // 8
        q = (word[:, col // 128 * 16 + 4 * (v % 4) + v // 4] >> (col % 8 // 2 * 4 + col % 2 * 16)) & 15
        at = col // c["g"]
        return (q.double() - (z[:, at].double() if z is not None else 8.0)) * s[:, at].double()

    if c["op"] == "quant":
        w = c["w"].double()
        parts = w.reshape(w.shape[0], -1, c["g"])
        lo, hi = parts.amin(2).clamp(max=0), parts.amax(2).clamp(min=0)
        # the definition rounds in FP32: the span, its quotient, each weight's quotient
        span = (hi.float() - lo.float()) if c["zeros"] else torch.maximum(hi, -lo).float()
        s = (span.double() / (15 if c["zeros"] else 7)).float().bfloat16().double()
        s[s == 0] = 1.0
        z = torch.round((-lo / s).float()).clamp(0, 15) if c["zeros"] else torch.full_like(s, 8.0)
        q = (torch.round((parts / s[:, :, None]).float()) + z[:, :, None]).clamp(0, 15)
        out = dict(values=((q.double() - z[:, :, None].double()) * s[:, :, None]).reshape(w.shape), scales=s)
        return dict(out, zeros=None) if c["zeros"] else out
    if c["op"] == "linear":
        return c["x"].double() @ decode(c["codes"], c["s"], c["z"]).t()
    if c["op"] == "route":
        l = c["logits"].double()
        b = c["b"].double() if c["b"] is not None else torch.zeros(c["e"], dtype=torch.float64, device="cuda")
        off = l.isneginf() | b.isneginf()
        s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        s = s.masked_fill(off, 0.0)
        choice = (s + b).masked_fill(off, -1e300)
        size = c["e"] // c["groups"]
        group = torch.stack([choice[:, g * size:(g + 1) * size].amax(1) for g in range(c["groups"])], 1)
        if c["by"] == "top2" and size > 1:
            second = torch.stack([choice[:, g * size:(g + 1) * size].kthvalue(size - 1, 1).values for g in range(c["groups"])], 1)
            group = group + second.masked_fill(second == -1e300, 0.0)
        for _ in range(c["groups"] - c["keep"]):        # drop the worst group, the last of equals
            worst = group.amin(1, keepdim=True)
            last = c["groups"] - 1 - (group == worst).flip(1).int().argmax(1)
            group = group.scatter(1, last[:, None], float("inf"))
            choice = choice.masked_fill((torch.arange(c["e"], device="cuda") // size)[None] == last[:, None], -float("inf"))
        w = []
        for _ in range(c["k"]):
            best = (choice == choice.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
            w.append(s.gather(1, best))
            choice = choice.scatter(1, best, -float("inf"))
        w = torch.cat(w, 1)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = w / total.masked_fill(total == 0, 1.0)
        return dict(idx=None, w=w * c["scale"])
    L, x, offsets, perm = c["layer"], c["x"].double(), c["offsets"].tolist(), c["perm"].long()

    def ffn(e, x):
        g, u, d = (decode(L["w_" + m][e], L["s_" + m][e], L["z_" + m][e] if c["zeros"] else None) for m in ("gate", "up", "down"))
        a = x @ g.t()
        return (a * torch.sigmoid(a) * (x @ u.t())) @ d.t()

    y = torch.cat([ffn(e, x[perm[offsets[e]:offsets[e + 1]]]) for e in range(c["e"]) if offsets[e] < offsets[e + 1]])
    return dict(routed=y, shared=ffn(c["e"], x)) if c["shared"] else dict(routed=y)

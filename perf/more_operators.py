"""Cases of the operators of a decoder layer around tree attention and the
quantized products: the 8-bit product with a scale per token and per channel,
the gated feed-forward product, the residual update with the norms around it,
row quantization, and the position rotation of drafted queries and keys.

`run` computes a case in plain torch operations (own = False) or with the
library's entry points (own = True) on the state that `prepare` makes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    """5120, 8192 and 17408 are the widths of the weight stream; 64 and 8 heads
    of 128 make its 8192-wide projections; 16 rows are a full draft block."""
    return [
        # plain decoding of one user: a single token through one projection, latency counts
        dict(name="product 1 8192 to 5120", op="product", n=1, m=5120, k=8192, dtype="bf16", bias=False),
        # a full draft block through the widest projection
        dict(name="product 16 5120 to 17408", op="product", n=16, m=17408, k=5120, dtype="f16", bias=True),
        # prompts packed without padding: an odd number of rows
        dict(name="product 4093 17408 to 5120", op="product", n=4093, m=5120, k=17408, dtype="bf16", bias=False),
        # a few users' drafted trees of 61 nodes through the gated projections
        dict(name="gated 61 5120 to 17408", op="gated", n=61, f=17408, k=5120, dtype="bf16", act="silu"),
        # a prompt through the gated projections
        dict(name="gated 2048 5120 to 17408", op="gated", n=2048, f=17408, k=5120, dtype="f16", act="gelu_tanh"),
        # the whole feed-forward block of a draft block: norm to 8 bits, gated product, quantization, product back
        dict(name="block 16 5120 17408", op="block", n=16, c=5120, f=17408, dtype="bf16", act="silu"),
        # a draft block's residual update and the norm of the next block
        dict(name="norm 16 5120", op="norm", n=16, c=5120, dtype="bf16", res="bf16", post=False, gate="none", alpha=1.0),
        # a prompt's, with a norm and a gate for each channel behind the block, the residual kept in 32 bits
        dict(name="norm 8190 5120 sandwich", op="norm", n=8190, c=5120, dtype="bf16", res="f32", post=True,
             gate="channel", alpha=0.35),
        # a draft block's rows to 8 bits before the product back
        dict(name="quant 16 17408", op="quant", n=16, c=17408, dtype="bf16"),
        # a prompt's rows
        dict(name="quant 4093 17408", op="quant", n=4093, c=17408, dtype="f16"),
        # drafted trees of a served batch at ragged positions, straight from the fused projection
        dict(name="rotate tree 8x16 ctx 16k", op="rotate", batch=8, n=16, heads=64, kv_heads=8, dim=128, rot=128,
             pairs="half", dtype="bf16", ctx_lo=1024, ctx=16384, tree="tree", scaling=1.0, amp=1.0),
        # two prompts far into a long context, part of each head, neighbouring pairs, scaled frequencies
        dict(name="rotate prompt 2x8190 ctx 1M", op="rotate", batch=2, n=8190, heads=64, kv_heads=8, dim=128, rot=64,
             pairs="neighbours", dtype="f16", ctx_lo=500000, ctx=1000000, tree="chain", scaling=8.0, amp=1.2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["product", "product", "gated", "gated", "block", "norm", "quant", "rotate"])
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    half = rng.choice(["bf16", "f16"])
    if op == "product":
        c = dict(op=op, n=_log_int(rng, 1, 4093), m=_log_int(rng, 64, 17408), k=16 * _log_int(rng, 4, 1088),
                 dtype=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.3)
        return c
    if op == "gated":
        c = dict(op=op, n=_log_int(rng, 1, 4093), f=_log_int(rng, 64, 17408), k=16 * _log_int(rng, 4, 1088),
                 dtype=rng.choice(["bf16", "f16", "f32"]), act=act)
        c["n"] = max(1, min(c["n"], 2048 * 17408 * 5120 // (c["f"] * c["k"])))
        return c
    if op == "block":
        c = dict(op=op, n=_log_int(rng, 1, 512), c=16 * _log_int(rng, 16, 512), f=16 * _log_int(rng, 16, 1088),
                 dtype=half, act=act)
        return c
    if op == "norm":
        c = dict(op=op, n=_log_int(rng, 1, 8190), c=16 * _log_int(rng, 4, 1088), dtype=half,
                 res=rng.choice(["f32", half]), post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "row"]),
                 alpha=rng.choice([1.0, 0.35]))
        c["n"] = max(1, min(c["n"], 8190 * 5120 // c["c"]))
        return c
    if op == "quant":
        return dict(op=op, n=_log_int(rng, 1, 4093), c=16 * _log_int(rng, 4, 1088), dtype=rng.choice(["bf16", "f16"]))
    chain = rng.random() < 0.5
    c = dict(op=op, batch=_log_int(rng, 1, 32), n=_log_int(rng, 1, 8190) if chain else _log_int(rng, 1, 64),
             kv_heads=rng.choice([1, 2, 4, 8]), heads=0, dim=rng.choice([64, 128, 256]), rot=0,
             pairs=rng.choice(["half", "neighbours"]), dtype=half, ctx_lo=0, ctx=_log_int(rng, 1, 1000000),
             tree="chain" if chain else "tree", scaling=rng.choice([1.0, 4.0, 8.0]), amp=rng.choice([1.0, 1.2]))
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8])
    c["rot"] = rng.choice([c["dim"], c["dim"] // 2, c["dim"] // 4])
    c["n"] = max(1, min(c["n"], 2 * 8190 * 72 * 128 // (c["batch"] * (c["heads"] + c["kv_heads"]) * c["dim"])))
    c["ctx_lo"] = rng.randint(0, c["ctx"])
    return c


# ------------------------------------------------------------------ inputs

def _weights(m, k, gen, dev):
    """8-bit weights with a scale for each output channel: normal values, the
    largest of a channel at 127."""
    w = torch.randn(m, k, generator=gen, device=dev)
    top = w.abs().amax(-1, keepdim=True)
    codes = torch.round(w * (127.0 / top)).to(torch.int8)
    return codes, (top[:, 0] / 127.0 / math.sqrt(k)).contiguous()


def _activations(n, k, gen, dev):
    """Rows with heavy tails and a few channels far above the others, as the
    inputs of projections are."""
    x = torch.randn(n, k, generator=gen, device=dev)
    x = x / torch.sqrt(torch.rand(n, k, generator=gen, device=dev).clamp(min=0.02))
    loud = torch.randint(0, k, (max(1, k // 1000),), generator=gen, device=dev)
    x[:, loud] *= 8.0
    return x


def _codes(x):
    top = x.abs().amax(-1, keepdim=True)
    return torch.round(x * (127.0 / top)).to(torch.int8), (top[:, 0] / 127.0).contiguous()


def _spread(lo, hi, count):
    """`count` whole numbers spread over lo .. hi, the first of them hi."""
    return [hi - int((hi - lo) * ((0.6180339887 * b) % 1.0)) for b in range(count)]


def _tree_masks(batch, n, g):
    """int64 [B][n]: bit j of entry i where node j is i or one of its
    ancestors, in random trees."""
    masks = np.zeros((batch, n), dtype=np.uint64)
    for b in range(batch):
        for i in range(n):
            up = np.uint64(0) if i == 0 else masks[b, g.randint(max(0, i - 6), i)]
            masks[b, i] = up | (np.uint64(1) << np.uint64(i))
    return masks.view(np.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    st = dict(op=case["op"], case=case)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "product":
        n, m, k = case["n"], case["m"], case["k"]
        st["w"], st["ws"] = _weights(m, k, gen, dev)
        st["x"], st["xs"] = _codes(_activations(n, k, gen, dev))
        st["bias"] = 0.1 * torch.randn(m, generator=gen, device=dev) if case["bias"] else None
        st["out"] = torch.zeros(n, m, dtype=dt, device=dev)
    elif case["op"] == "gated":
        n, f, k = case["n"], case["f"], case["k"]
        # one matrix, the gate's rows first, as the weights of such blocks are kept
        st["w"], st["ws"] = _weights(2 * f, k, gen, dev)
        st["x"], st["xs"] = _codes(_activations(n, k, gen, dev))
        st["out"] = torch.zeros(n, f, dtype=dt, device=dev)
    elif case["op"] == "block":
        n, c, f = case["n"], case["c"], case["f"]
        st["y"], st["residual"] = (_activations(n, c, gen, dev).to(dt) for _ in range(2))
        st["weight"] = 1.0 + 0.2 * torch.randn(c, generator=gen, device=dev)
        st["w"], st["ws"] = _weights(2 * f, c, gen, dev)
        st["wd"], st["wds"] = _weights(c, f, gen, dev)
        st["residual_out"], st["h"], st["out"] = (torch.zeros(n, x, dtype=dt, device=dev) for x in (c, f, c))
        st["x"], st["hq"] = (torch.zeros(n, x, dtype=torch.int8, device=dev) for x in (c, f))
        st["xs"], st["hs"] = (torch.zeros(n, device=dev) for _ in range(2))
    elif case["op"] == "norm":
        n, c = case["n"], case["c"]
        st["y"] = _activations(n, c, gen, dev).to(dt)
        st["residual"] = (3.0 * _activations(n, c, gen, dev)).to(DTYPES[case["res"]])
        st["weight"] = 1.0 + 0.2 * torch.randn(c, generator=gen, device=dev)
        st["post"] = 1.0 + 0.2 * torch.randn(c, generator=gen, device=dev) if case["post"] else None
        st["gate"] = None
        if case["gate"] == "channel":
            st["gate"] = 0.5 * torch.randn(c, generator=gen, device=dev)
        elif case["gate"] == "row":
            st["gate"] = torch.sigmoid(torch.randn(n, c, generator=gen, device=dev)).to(dt)
        st["residual_out"] = torch.zeros_like(st["residual"])
        st["out"] = torch.zeros(n, c, dtype=dt, device=dev)
    elif case["op"] == "quant":
        n, c = case["n"], case["c"]
        st["x"] = _activations(n, c, gen, dev).to(dt)
        st["q_out"] = torch.zeros(n, c, dtype=torch.int8, device=dev)
        st["scales_out"] = torch.zeros(n, device=dev)
    else:
        B, n, D = case["batch"], case["n"], case["dim"]
        widths = [case["heads"] * D, case["kv_heads"] * D, case["kv_heads"] * D]
        fused = torch.randn(B, n, sum(widths), generator=gen, device=dev).to(dt)
        q, k, _ = torch.split(fused, widths, dim=-1)
        st["q"], st["k"] = q.unflatten(-1, (-1, D)), k.unflatten(-1, (-1, D))
        g = np.random.RandomState(int(seed) % (1 << 31))
        lens = np.array(_spread(case["ctx_lo"], case["ctx"], B), dtype=np.int32)
        st["ctx_len"] = torch.from_numpy(lens[g.permutation(B)]).to(dev)
        st["tree_mask"] = torch.from_numpy(_tree_masks(B, n, g)).to(dev) if case["tree"] == "tree" else None
        half = torch.arange(case["rot"] // 2, dtype=torch.float64)
        freq = 1e6 ** (-2.0 * half / case["rot"])
        # the slow half of the pairs is stretched for the longer context
        freq = torch.where(half >= case["rot"] // 4, freq / case["scaling"], freq)
        st["inv_freq"] = freq.to(torch.float32).to(dev)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"product": _plain_product, "gated": _plain_gated, "block": _plain_block, "norm": _plain_norm,
            "quant": _plain_quant, "rotate": _plain_rotate}[st["op"]](st)


def _run_own(st):
    import block_quantized_gemm_amd as vq
    case = st["case"]
    if st["op"] == "product":
        return vq.gemm_w8a8(st["w"], st["ws"], st["x"], st["xs"], st["out"], bias=st["bias"])
    if st["op"] == "gated":
        f = case["f"]
        return vq.gated_w8a8(st["w"][:f], st["ws"][:f], st["w"][f:], st["ws"][f:], st["x"], st["xs"], st["out"],
                             activation=case["act"])
    if st["op"] == "block":
        f = case["f"]
        vq.residual_norm(st["residual"], st["y"], st["weight"], out=st["x"], scales_out=st["xs"],
                         residual_out=st["residual_out"], eps=EPS)
        vq.gated_w8a8(st["w"][:f], st["ws"][:f], st["w"][f:], st["ws"][f:], st["x"], st["xs"], st["h"],
                      activation=case["act"])
        vq.quant_rows_int8(st["h"], st["hq"], st["hs"])
        return st["residual_out"], vq.gemm_w8a8(st["wd"], st["wds"], st["hq"], st["hs"], st["out"])
    if st["op"] == "norm":
        vq.residual_norm(st["residual"], st["y"], st["weight"], post_weight=st["post"], gate=st["gate"],
                         alpha=case["alpha"], eps=EPS, out=st["out"], residual_out=st["residual_out"])
        return st["residual_out"], st["out"]
    if st["op"] == "quant":
        return vq.quant_rows_int8(st["x"], st["q_out"], st["scales_out"])
    return vq.rotate(st["q"], st["k"], st["inv_freq"], st["ctx_len"], tree_mask=st["tree_mask"],
                     interleaved=case["pairs"] == "neighbours", scale=case["amp"])


def _dots(x, xs, w, ws):
    return torch.matmul(x.float(), w.float().t()) * xs[:, None] * ws


def _plain_product(st):
    y = _dots(st["x"], st["xs"], st["w"], st["ws"])
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(st["out"].dtype)


def _act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    if kind == "gelu_tanh":  # 0.5 g (1 + tanh z) = g / (1 + exp(-2 z))
        z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
        return g / (1.0 + torch.exp(-2.0 * z))
    return 0.5 * g * torch.special.erfc(g * -math.sqrt(0.5))


def _gated(x, xs, w, ws, kind):
    f = w.shape[0] // 2
    both = _dots(x, xs, w, ws)
    return _act(both[:, :f], kind) * both[:, f:]


def _plain_gated(st):
    return _gated(st["x"], st["xs"], st["w"], st["ws"], st["case"]["act"]).to(st["out"].dtype)


def _rms(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _quantize(x):
    top = x.abs().amax(-1, keepdim=True)
    s = top / torch.full_like(top, 127.0)
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))).clamp(-127, 127)
    return q.to(torch.int8), s[:, 0]


def _plain_block(st):
    r = st["residual"].float() + st["y"].float()
    x, xs = _quantize(_rms(r) * st["weight"])
    h = _gated(x, xs, st["w"], st["ws"], st["case"]["act"]).to(st["h"].dtype)
    hq, hs = _quantize(h.float())
    return r.to(st["residual"].dtype), _dots(hq, hs, st["wd"], st["wds"]).to(st["out"].dtype)


def _plain_norm(st):
    u = st["y"].float()
    if st["post"] is not None:
        u = _rms(u) * st["post"]
    if st["gate"] is not None:
        u = u * st["gate"].float()
    r = st["residual"].float() + st["case"]["alpha"] * u
    return r.to(st["residual"].dtype), (_rms(r) * st["weight"]).to(st["out"].dtype)


def _plain_quant(st):
    return _quantize(st["x"].float())


def _positions(st):
    """int64 [B][n]: the context's length and how many ancestors a node has."""
    n = st["q"].shape[1]
    node = torch.arange(n, device=st["q"].device)
    if st["tree_mask"] is None:
        depth = node[None, :]
    else:
        depth = (((st["tree_mask"][:, :, None] >> node) & 1) * (node < node[:, None])).sum(-1)
    return st["ctx_len"].long()[:, None] + depth


def _plain_rotate(st):
    case = st["case"]
    angle = _positions(st).double()[:, :, None, None] * st["inv_freq"].double()
    c, s = (case["amp"] * f(angle).float() for f in (torch.cos, torch.sin))
    rot = case["rot"]

    def turn(t):
        x = t.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["pairs"] == "neighbours" else \
            (x[..., :rot // 2], x[..., rot // 2:rot])
        y = [a * c - b * s, b * c + a * s]
        y = torch.stack(y, -1).flatten(-2) if case["pairs"] == "neighbours" else torch.cat(y, -1)
        return torch.cat([y, x[..., rot:]], -1).to(t.dtype)
    return turn(st["q"]), turn(st["k"])


# ------------------------------------------------------------------ what a pass cannot do without

def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op == "product":
        n, m, k = case["n"], case["m"], case["k"]
        return {"bytes": (m + n) * (k + 4) + n * m * e + (4 * m if case["bias"] else 0), "flops": 2 * n * m * k}
    if op == "gated":
        n, f, k = case["n"], case["f"], case["k"]
        return {"bytes": (2 * f + n) * (k + 4) + n * f * e, "flops": 4 * n * f * k}
    if op == "block":  # what lies between the four calls is not counted
        n, c, f = case["n"], case["c"], case["f"]
        return {"bytes": 3 * f * c + 4 * (2 * f + 2 * c) + 4 * n * c * e, "flops": 6 * n * f * c}
    if op == "norm":
        n, c, r = case["n"], case["c"], _size(case["res"])
        gate = {"none": 0, "channel": 4 * c, "row": n * c * e}[case["gate"]]
        return {"bytes": n * c * (2 * r + 2 * e) + 4 * c * (2 if case["post"] else 1) + gate, "flops": 8 * n * c}
    if op == "quant":
        return {"bytes": case["n"] * (case["c"] * (e + 1) + 4), "flops": 3 * case["n"] * case["c"]}
    rows = case["batch"] * case["n"]
    heads = case["heads"] + case["kv_heads"]
    return {"bytes": 2 * e * rows * heads * case["dim"] + (8 * rows if case["tree"] == "tree" else 0),
            "flops": 3 * rows * heads * case["rot"]}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"product": _exact_product, "gated": _exact_gated, "block": _exact_block, "norm": _exact_norm,
            "quant": _exact_quant, "rotate": _exact_rotate}[case["op"]](case, st)


def _product64(x, xs, w, ws):
    """sum_k of the dequantized values, some channels at a time."""
    out = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    a = x.double() * xs.double()[:, None]
    for at in range(0, w.shape[0], 2048):
        part = w[at:at + 2048].double() * ws[at:at + 2048].double()[:, None]
        out[:, at:at + 2048] = a @ part.t().contiguous()
    return out


def _exact_product(case, st):
    y = _product64(st["x"], st["xs"], st["w"], st["ws"])
    return y if st["bias"] is None else y + st["bias"].double()


def _gated64(x, xs, w, ws, kind):
    f = w.shape[0] // 2
    g, u = (_product64(x, xs, w[at:at + f], ws[at:at + f]) for at in (0, f))
    if kind == "silu":
        a = g * torch.sigmoid(g)
    elif kind == "gelu_tanh":
        a = 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    else:
        a = 0.5 * g * (1.0 + torch.erf(g / 2.0 ** 0.5))
    return a * u


def _exact_gated(case, st):
    return _gated64(st["x"], st["xs"], st["w"], st["ws"], case["act"])


def _norm64(x, weight):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * weight.double()


def _quantize64(x):
    s = (x.abs().max(dim=1).values / 127.0).float()  # the scale is kept in 32 bits
    q = torch.round(x / s.double()[:, None])
    return torch.clamp(torch.nan_to_num(q), -127, 127).to(torch.int8), s


def _exact_block(case, st):
    r = st["residual"].double() + st["y"].double()
    x, xs = _quantize64(_norm64(r, st["weight"]))
    h = _gated64(x, xs, st["w"], st["ws"], case["act"])
    h = h.to(DTYPES[case["dtype"]])  # what the gated product hands on is of this type
    hq, hs = _quantize64(h.double())
    return r, _product64(hq, hs, st["wd"], st["wds"])


def _exact_norm(case, st):
    u = st["y"].double()
    if case["post"]:
        u = _norm64(u, st["post"])
    if case["gate"] != "none":
        u = u * st["gate"].double()
    r = st["residual"].double() + case["alpha"] * u
    return r, _norm64(r, st["weight"])


def _exact_quant(case, st):
    return None, st["x"].double().abs().max(dim=1).values / 127.0


def _exact_rotate(case, st):
    rot, n = case["rot"], case["n"]
    freq = st["inv_freq"].double().cpu().numpy()
    masks = st["tree_mask"].cpu().numpy().view(np.uint64) if st["tree_mask"] is not None else None
    pos = np.zeros((case["batch"], n))
    for b, ctx in enumerate(st["ctx_len"].tolist()):
        for i in range(n):
            pos[b, i] = ctx + (i if masks is None else bin(int(masks[b, i]) & ((1 << i) - 1)).count("1"))
    turn = torch.polar(torch.full((1,), case["amp"], dtype=torch.float64),
                       torch.from_numpy(pos[:, :, None, None] * freq)).to(st["q"].device)

    def rotated(t):
        y = t.double()
        if case["pairs"] == "neighbours":
            z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot] = torch.cat([z.real, z.imag], -1)
        return y
    return rotated(st["q"]), rotated(st["k"])

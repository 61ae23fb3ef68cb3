"""Cases that measure the microscaled 4-bit operators: the layer's, the cache's and its attention.

Codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), 32 consecutive ones along the
contraction sharing a scale, which is a power of two kept as its exponent byte. With rotation k the
values are first multiplied by the Walsh-Hadamard matrix H_k along that axis, unnormalised, in fp32
butterflies of strides 1, 2, .. k / 2. s = the smallest power of two with absmax <= 6 s, at least
2^-126; a code is the value nearest to v / s (ties to even), or is rounded at random without bias.

Four operators, each in a plain form (elementary torch operations in 32 bits) and through the
framework's entry points:

  quant   a matrix to codes (and those of its transpose), and back to values
  linear  serve: Y = X W^T for given codes of W; train: the three products of a layer's step
  cache   keys and values of new tokens written to their slots in 4 bits, and read back
  attn    attention of a batch's queries over the paged cache, with the logarithms of the sums
"""
import math
import random

import torch

own = False

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
INF = float("inf")


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch's activations before a projection: latency
        dict(name="quant_decode", op="quant", rows=16, cols=4096, dtype="bf16", rot=32, t=False,
             random=False),
        # a training batch's output gradients, both layouts, rounded at random
        dict(name="quant_gradient", op="quant", rows=8192, cols=13824, dtype="bf16", rot=32, t=True,
             random=True),
        # one token through an MLP projection: the weights' bytes
        dict(name="serve_1", op="linear", train=False, N=1, C=4096, D=11008, dtype="bf16", rot=32),
        # a short prompt of an odd length
        dict(name="serve_1000", op="linear", train=False, N=1000, C=5120, D=13824, dtype="fp16",
             rot=32),
        # a small layer with ragged sizes on every axis, in fp32, not rotated
        dict(name="train_ragged", op="linear", train=True, N=1000, C=1030, D=778, dtype="fp32",
             rot=1, random=False),
        # the largest layer, gradients rounded at random
        dict(name="train_8192", op="linear", train=True, N=8192, C=13824, D=5120, dtype="bf16",
             rot=32, random=True),
        # a decode batch's new keys and values
        dict(name="cache_decode", op="cache", T=48, H=8, D=128, page=64, dtype="bf16", rot=True),
        # a prompt's keys and values
        dict(name="cache_prompt", op="cache", T=16384, H=8, D=128, page=64, dtype="bf16", rot=True),
        # one short conversation: latency
        dict(name="attn_one", op="attn", S=1, Q=1, L=777, Hq=32, Hkv=8, D=128, page=16, window=0,
             dtype="bf16", out="bf16", rot=True),
        # a decode batch of unlike lengths: the cache's bytes
        dict(name="attn_decode", op="attn", S=32, Q=1, L=16384, Hq=32, Hkv=8, D=128, page=64,
             window=0, dtype="bf16", out="bf16", rot=True),
        # a few drafted tokens for each of some sequences, a head each, in a window, not rotated
        dict(name="attn_draft", op="attn", S=5, Q=7, L=9001, Hq=16, Hkv=16, D=64, page=32,
             window=2500, dtype="fp16", out="fp32", rot=False),
        # pieces of two prompts behind what the cache holds of them
        dict(name="attn_prompt", op="attn", S=2, Q=1500, L=9000, Hq=40, Hkv=8, D=128, page=256,
             window=0, dtype="bf16", out="bf16", rot=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm, odd ones among them."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "cache", "attn", "attn"])
    if op == "quant":
        rows = _spread(rng, 1, 8192)
        cols = _spread(rng, 16, min(16384, max(16, (8192 * 13824) // rows)))
        if rng.random() < 0.5:   # feature counts are usually whole blocks
            cols = (cols + 31) // 32 * 32
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["fp32", "fp16", "bf16"]),
                    rot=rng.choice([1, 32]), t=rng.random() < 0.5, random=rng.random() < 0.5)
    if op == "linear":
        train = rng.random() < 0.5
        C, D = (_spread(rng, 128, 8192 if train else 13824) for _ in range(2))
        if rng.random() < 0.7:
            C, D = (C + 31) // 32 * 32, (D + 31) // 32 * 32
        c = dict(op=op, train=train, N=_spread(rng, 64, 8192) if train else _spread(rng, 1, 2048),
                 C=C, D=D, dtype=rng.choice(["fp32", "fp16", "bf16", "bf16"]),
                 rot=rng.choice([1, 32]))
        return dict(c, random=rng.random() < 0.5) if train else c
    head = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    rot, dtype = rng.random() < 0.7, rng.choice(["fp32", "fp16", "bf16", "bf16"])
    if op == "cache":
        H = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, T=_spread(rng, 1, 16384 * 8 * 128 // (H * head)), H=H, D=head, page=page,
                    dtype=dtype, rot=rot)
    Hkv, group = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 4, 5, 8, 16])
    if rng.random() < 0.65:   # decoding, with a few drafted tokens at most
        Q, S = rng.choice([1, 1, 1, 2, 5, 8]), _spread(rng, 1, 64)
        L = _spread(rng, Q + 10, min(32768, 32 * 16384 * 8 * 128 // (S * Hkv * head)))
    else:                     # pieces of prompts
        Q, S = _spread(rng, 9, 1500), rng.randint(1, 3)
        L = Q + _spread(rng, 1, 8000)
        while S * Q * L * Hkv * group * head > 2 * 1500 * 9000 * 40 * 128:
            group, S = max(1, group // 2), max(1, S - 1)
            Q, L = max(9, Q // 2), max(20, L // 2)
    return dict(op=op, S=S, Q=Q, L=L, Hq=Hkv * group, Hkv=Hkv, D=head, page=page,
                window=rng.choice([0, 0, 0, _spread(rng, 16, 4096)]), dtype=dtype, out=dtype, rot=rot)


# ------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _normal(g, rows, cols, dtype, scale=1.0, outliers=0):
    """Normal values, a few columns of which are 30 times larger (the outlier channels of
    activations)."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    if outliers:
        x[:, torch.randint(0, cols, (outliers,), generator=g, device="cuda")] *= 30.0
    return x.to(DT[dtype])


def _gradients(g, rows, cols, dtype):
    """Mostly small, with heavy tails."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (1e-3 * x * x.square()).to(DT[dtype])


def _kept(x, rot):
    """Codes (packed in pairs, rows padded to 16 bytes) and scale bytes (rows padded likewise) of a
    matrix, as a checkpoint holds them."""
    v, s = _quantized(_rotated(x.float(), rot))
    return _padded(_packed(v), 16), _padded(_bytes(s), 16)


def _padded(x, to):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % to)).contiguous()


def _packed(v):
    """Two code nibbles a byte, the even element in the low one."""
    m = v.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = _padded(code + 8 * torch.signbit(v).to(torch.uint8), 32)
    return code[..., ::2] + 16 * code[..., 1::2]


def _bytes(s):
    return (s.view(torch.int32) >> 23).to(torch.uint8)


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": dict(case)}
    op = case["op"]
    # of the random rounding
    st["seed"] = torch.tensor([int(seed) * 2654435761 & 0x7FFFFFFF], dtype=torch.int32, device="cuda")
    if op == "quant":
        make = _gradients if case["random"] else _normal
        st["x"] = make(g, case["rows"], case["cols"], case["dtype"])
        st["values"] = torch.empty_like(st["x"])
        st["values_t"] = st["x"].new_empty(case["cols"], case["rows"])
    elif op == "linear":
        N, C, D, dtype = case["N"], case["C"], case["D"], case["dtype"]
        st["x"] = _normal(g, N, C, dtype, 1.0, 4)
        st["y"] = torch.empty(N, D, dtype=DT[dtype], device="cuda")
        if case["train"]:
            st["w"] = _normal(g, D, C, dtype, 0.02)
            st["dy"] = _gradients(g, N, D, dtype)
            st["dx"], st["dw"] = torch.empty_like(st["x"]), torch.empty_like(st["w"])
        else:
            st["w_codes"], st["w_scales"] = _kept(_normal(g, D, C, "fp32", 0.02), case["rot"])
    elif op == "cache":
        T, H, D = case["T"], case["H"], case["D"]
        # keys and values lie in the projection's output, behind 4 H heads of queries
        qkv = torch.randn(T, 6 * H, D, generator=g, device="cuda")
        qkv[:, 4 * H:5 * H, 3:5] *= 10.0      # keys have outlier channels
        st["qkv"] = qkv.to(DT[case["dtype"]])
        pages = -(-T // case["page"]) + 3
        st["slots"] = torch.randperm(pages * case["page"], generator=g, device="cuda")[:T].contiguous()
        st["k"], st["v"] = (st["qkv"].new_empty(T, H, D) for _ in range(2))
    else:
        _prepare_attn(st, case, g)
    return st


def _prepare_attn(st, c, g):
    S, page, Hkv, D = c["S"], c["page"], c["Hkv"], c["D"]
    rng = random.Random(c["L"] * 4096 + c["Q"])    # the batch's lengths are the case's own
    news = [c["Q"] if i == 0 or c["Q"] < 9 else rng.randint(1, c["Q"]) for i in range(S)]
    lens = [c["L"] if i == 0 else rng.randint(max(news[i], c["L"] // 4), c["L"]) for i in range(S)]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table, at = torch.zeros(S, max(need), dtype=torch.int32, device="cuda"), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [sum(news[:i]) for i in range(S + 1)]
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for name in ("k", "v"):
        st[name + "_codes"] = torch.empty(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
        st[name + "_scales"] = torch.empty(pages, Hkv, page, D // 32, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 25) // (Hkv * page * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = torch.randn(n, Hkv, page, D, generator=g, device="cuda")
            if name == "k":
                x[..., 3:5] *= 6.0
            v, s = _quantized(_rotated(x, D if c["rot"] else 1))
            st[name + "_codes"][p:p + n], st[name + "_scales"][p:p + n] = _packed(v), _bytes(s)
    st["q"] = torch.randn(starts[-1], c["Hq"], D, generator=g, device="cuda").to(DT[c["dtype"]])
    st["out"] = torch.empty(starts[-1], c["Hq"], D, dtype=DT[c["out"]], device="cuda")
    st["lse"] = torch.empty(starts[-1], c["Hq"], dtype=torch.float32, device="cuda")
    st["scale"] = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------------------------- plain forms
def _rotated(x, k):
    """H_k on every k consecutive elements of the last axis (padded with zeros to whole ones)."""
    x = _padded(x, k)
    shape, h = x.shape, 1
    while h < k:
        x = x.reshape(*shape[:-1], -1, 2, h)
        a, b = x[..., 0, :], x[..., 1, :]
        x = torch.stack([a + b, a - b], -2)
        h *= 2
    return x.reshape(shape)


def _mix(h):
    """The 32-bit mixing steps of the random rounding (h: int64 holding 32 bits)."""
    h = h ^ (h >> 16)
    h = (h * 2654435761) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 2891336453) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _numbers(seed, shape):
    """16 random bits for each element: one hash of (seed, row, column / 2) for two columns."""
    dev = seed.device
    r, j = torch.arange(shape[0], device=dev), torch.arange(shape[1] // 2, device=dev)
    key = _mix((seed.long() + 2654435761 * r) & 0xFFFFFFFF)
    h = _mix(key[:, None] ^ j)
    return torch.stack([h & 0xFFFF, h >> 16], -1).view(shape)


def _quantized(x, seed=None):
    """The codes' values (the last axis padded to whole blocks) and the scales by block."""
    x = _padded(x, 32)
    b = x.view(*x.shape[:-1], -1, 32)
    exponent = ((b.abs().amax(-1).view(torch.int32) + 0x3FFFFF) >> 23) - 2
    s = (exponent.clamp_min(1) << 23).view(torch.float32)
    y = (b / s[..., None]).view(x.shape)
    m = y.abs()
    if seed is None:
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        m = torch.round(m / step) * step
    else:
        u = _numbers(seed, x.shape).int()
        high = ((m.view(torch.int32) + (u << 6)) & ~0x3FFFFF).view(torch.float32)
        m = torch.where(m >= 1, high, torch.floor(2 * m + u.float() / 65536) * 0.5)
    return torch.copysign(m, y), s


def _scaled(v, s):
    """What codes and scales stand for (in the rotated space)."""
    return (v.view(*s.shape, 32) * s[..., None]).view(v.shape)


def _values(x, rot, seed=None):
    return _scaled(*_quantized(_rotated(x.float(), rot), seed))


def _plain_quant(st):
    c = st["case"]
    seeds = [None, None] if not c["random"] else [st["seed"], st["seed"].long() + 0x9E3779B9]
    out = {}
    for name, x, seed in [("values", st["x"], seeds[0]), ("values_t", st["x"].t(), seeds[1])][:1 + c["t"]]:
        v = _rotated(_values(x, c["rot"], seed), c["rot"]) / c["rot"]
        st[name].copy_(v[:, :x.shape[1]])
        out[name] = st[name]
    return out


def _unpacked(codes):
    """The values of packed codes."""
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = codes & 7
    e = (m >> 1).float()
    v = torch.where(m < 2, m.float() * 0.5, (1 + (m & 1).float() * 0.5) * torch.exp2(e - 1))
    return torch.where(codes > 7, -v, v)


def _from_bytes(b):
    return (b.int() << 23).view(torch.float32)


def _plain_linear(st):
    c = st["case"]
    rot = c["rot"]
    if not c["train"]:
        x = _values(st["x"], rot)
        blocks = x.shape[1] // 32
        w = _scaled(_unpacked(st["w_codes"][:, :16 * blocks]), _from_bytes(st["w_scales"][:, :blocks]))
        st["y"].copy_(x @ w.t() / rot)
        return {"y": st["y"]}
    seed = seed_t = None
    if c["random"]:
        seed, seed_t = st["seed"], st["seed"].long() + 0x9E3779B9
    st["y"].copy_(_values(st["x"], rot) @ _values(st["w"], rot).t() / rot)
    st["dx"].copy_(_values(st["dy"], rot, seed) @ _values(st["w"].t(), rot).t() / rot)
    st["dw"].copy_(_values(st["dy"].t(), rot, seed_t) @ _values(st["x"].t(), rot).t() / rot)
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _plain_cache(st):
    c = st["case"]
    H, rot = c["H"], c["D"] if c["rot"] else 1
    pages = -(-c["T"] // c["page"]) + 3
    for name, at in (("k", 4 * H), ("v", 5 * H)):
        pool = torch.zeros(pages, c["page"], H, c["D"], device="cuda")
        page, row = st["slots"] // c["page"], st["slots"] % c["page"]
        pool[page, row] = _values(st["qkv"][:, at:at + H], rot)
        st[name].copy_(_rotated(pool[page, row], rot) / rot)
    return {"k": st["k"], "v": st["v"]}


def _cached(st, name):
    """The cache's values (in the rotated space) for each sequence's positions: S x Hkv x L x D."""
    table = st["table"].long()
    v = _scaled(_unpacked(st[name + "_codes"][table]), _from_bytes(st[name + "_scales"][table]))
    return v.transpose(1, 2).flatten(2, 3)    # S x pages x Hkv x page x D


def _plain_attn(st):
    c = st["case"]
    rot = c["D"] if c["rot"] else 1
    k = _cached(st, "k")
    S, Hkv, L, D = k.shape
    first, news = st["starts"][:-1].long(), st["starts"].long().diff()
    at = torch.arange(c["Q"], device="cuda")
    real = at < news[:, None]
    rows = (first[:, None] + at).clamp_max(st["q"].shape[0] - 1)
    q = _rotated(st["q"][rows].float(), rot).view(S, c["Q"], Hkv, -1, D)
    group = q.shape[3]
    s = q.permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D) @ k.transpose(2, 3) * (st["scale"] / rot)
    del k
    pos = ((st["lens"].long() - news)[:, None] + at).repeat_interleave(group, 1)[:, None, :, None]
    j = torch.arange(L, device="cuda")
    seen = j <= pos
    if c["window"]:
        seen &= j > pos - c["window"]
    s.masked_fill_(~seen, -INF)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = _rotated((p @ _cached(st, "v")) / total, rot) / rot
    lse = (m + total.log())[..., 0]

    def by_token(x):
        return x.view(S, Hkv, c["Q"], group, -1).permute(0, 2, 1, 3, 4).reshape(S, c["Q"], c["Hq"], -1)[real]

    st["out"].copy_(by_token(o))
    st["lse"].copy_(by_token(lse)[..., 0])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------------------------- own calls
def _own(st):
    from hadamard_rotated_precision_amd import binding as B
    from hadamard_rotated_precision_amd import tensors as T

    c, kept = st["case"], st.get("kept")
    seed = st["seed"] if c.get("random") else None
    if c["op"] == "quant":
        if kept is None:
            kept = st["kept"] = T.MxTensor(c["rows"], c["cols"], rot=c["rot"], codes_t=c["t"])
        kept.quantize(st["x"], seed=seed)
        kept.dequantize(st["values"])
        if not c["t"]:
            return {"values": st["values"]}
        kept.dequantize(st["values_t"], side=B.HQ_SIDE_COLS)
        return {"values": st["values"], "values_t": st["values_t"]}
    if c["op"] == "linear" and not c["train"]:
        if kept is None:   # the layer around the weights that a server keeps
            w = T.MxTensor.wrap(st["w_codes"], st["w_scales"], c["D"], c["C"], rot=c["rot"])
            kept = st["kept"] = T.MxLayer(c["N"], c["C"], c["D"], rot=c["rot"], weight=w, train=False)
        kept.fwd(st["x"], st["y"])
        return {"y": st["y"]}
    if c["op"] == "linear":
        if kept is None:
            kept = st["kept"] = T.MxLayer(c["N"], c["C"], c["D"], rot=c["rot"])
        kept.set_weight(st["w"])
        kept.fwd(st["x"], st["y"])
        kept.bwd_input(st["dy"], st["dx"], seed=seed)
        kept.bwd_weight(st["dw"])
        return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}
    if c["op"] == "cache":
        H = c["H"]
        if kept is None:
            kept = st["kept"] = T.KVCache(-(-c["T"] // c["page"]) + 3, c["page"], H, c["D"], rotate=c["rot"])
        kept.append(st["qkv"][:, 4 * H:5 * H], st["qkv"][:, 5 * H:], st["slots"])
        kept.read(st["slots"], st["k"], st["v"])
        return {"k": st["k"], "v": st["v"]}
    if kept is None:   # the cache and the workspace that a server keeps
        kept = st["kept"] = T.KVCache.wrap(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"],
                                           rotate=c["rot"])
        st["ws"] = kept.attention_workspace(c["S"], c["Hq"], max_q=c["Q"], max_len=c["L"])
    kept.attend(st["q"], st["out"], st["starts"], st["lens"], st["table"], max_q=c["Q"], max_len=c["L"],
                scale=st["scale"], window=c["window"], lse=st["lse"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "linear": _plain_linear, "cache": _plain_cache,
            "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- work
def _code_bytes(n, k):
    """Bytes of n rows of k codes with their scales."""
    return n * (-(-k // 2) + -(-k // 32))


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "quant":
        r, c = case["rows"], case["cols"]
        codes = _code_bytes(r, c) + (_code_bytes(c, r) if case["t"] else 0)
        return {"bytes": r * c * e * (2 + case["t"]) + codes, "flops": 0}
    if op == "linear":
        N, C, D = case["N"], case["C"], case["D"]
        if not case["train"]:
            return {"bytes": _code_bytes(D, C) + e * (N * C + N * D), "flops": 2 * N * C * D}
        return {"bytes": e * 2 * (N * C + D * C + N * D), "flops": 6 * N * C * D}
    if op == "cache":
        rows = 2 * case["T"] * case["H"]
        return {"bytes": rows * 2 * case["D"] * e + _code_bytes(rows, case["D"]) + 8 * case["T"],
                "flops": 0}
    # sequences after the first have half of its new tokens and 5/8 of its length on average
    S, Q, L, w = case["S"], case["Q"], case["L"], case["window"]
    others = max(0, S - 1)
    tokens = Q + others * (Q if Q < 9 else (1 + Q) / 2)
    lengths = [L] + [L * 5 / 8] * others
    news = [Q] + [tokens / S if Q < 9 else (1 + Q) / 2] * others
    read = sum(min(n, w + q) if w else n for n, q in zip(lengths, news))
    pairs = sum(q * (min(n - q / 2, w) if w else n - q / 2) for n, q in zip(lengths, news))
    io = tokens * case["Hq"] * case["D"] * (e + SIZE[case["out"]]) + 4 * tokens * case["Hq"]
    return {"bytes": int(_code_bytes(2 * read * case["Hkv"], case["D"]) + io),
            "flops": int(4 * case["D"] * case["Hq"] * pairs)}


# ------------------------------------------------------------------------------------- in 64 bits
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _turned64(x, k, cut=False):
    """H_k along the last axis, k = 1 or a power of two that divides it; cut: every stage's sums are
    fp32 numbers, as the quantizer's definition has them."""
    at = torch.arange(x.shape[-1], device=x.device)
    for bit in range(k.bit_length() - 1):
        upper = (at >> bit) & 1
        x = x[..., at ^ (1 << bit)] + x * (1 - 2 * upper)
        x = x.float().double() if cut else x
    return x


def _exact_values(x, rot, seed=None):
    """What the codes of a matrix stand for, in the rotated space (columns padded to blocks)."""
    n = -(-x.shape[-1] // 32) * 32
    v = torch.zeros(*x.shape[:-1], n, dtype=torch.float64, device=x.device)
    v[..., :x.shape[-1]] = x
    v = _turned64(v, rot, cut=True)
    a = v.unflatten(-1, (-1, 32)).abs().amax(-1)
    f, e = torch.frexp(a / 6.0)          # a / 6 = f 2^e, f in [0.5, 1)
    e = torch.where(f == 0.5, e - 1, e)
    # 6 has two significant bits, so the quotient's rounding cannot hide a <= 6 2^e
    e = torch.where(torch.ldexp(torch.full_like(a, 6.0), e - 1) >= a, e - 1, e)
    s = torch.exp2(torch.where(a > 0, e, -126).clamp_min(-126).double()).repeat_interleave(32, -1)
    y = v.abs() / s
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    low = (torch.searchsorted(grid, y, right=True) - 1).clamp_max(6)
    share = (y - grid[low]) / (grid[low + 1] - grid[low])
    if seed is None:
        up = torch.where(share == 0.5, low % 2 == 1, share > 0.5)
    else:
        at = torch.arange(n, device=x.device)
        row = torch.arange(x.shape[0], device=x.device)
        h = _hashed64(torch.bitwise_xor(_hashed64((seed.long() + row * 2654435761) % 2 ** 32)[:, None],
                                        at // 2))
        u = torch.where(at % 2 == 0, h % 65536, h // 65536).double() / 65536
        up = share + u >= 1
    return torch.copysign(grid[low + up.long()], v) * s


def _hashed64(h):
    for shift, factor in ((16, 2654435761), (15, 2891336453), (16, 1)):
        h = torch.bitwise_xor(h, torch.div(h, 2 ** shift, rounding_mode="floor"))
        # in two halves: the product of two 32-bit numbers need not fit 63 bits
        h = (h % 65536 * factor + (h // 65536 * factor % 65536) * 65536) % 2 ** 32
    return h


def _exact_codes(codes, scales):
    """Values of packed codes and scale bytes."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device=codes.device)
    v = torch.stack([grid[(codes % 16).long()], grid[(codes // 16).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_attn(st):
    c = st["case"]
    D, page, group = c["D"], c["page"], c["Hq"] // c["Hkv"]
    rot = D if c["rot"] else 1
    starts, lens = st["starts"].tolist(), st["lens"].tolist()
    out, lse = st["out"].double(), st["lse"].double()
    for i, n in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        pos = torch.arange(n - (b - a), n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        hidden = (j > pos) | ((j <= pos - c["window"]) if c["window"] else (j < 0))
        pages = st["table"][i, :-(-n // page)].long()
        for h in range(c["Hkv"]):
            k, v = (_turned64(_exact_codes(st[x + "_codes"][pages, h].flatten(0, 1)[:n],
                                           st[x + "_scales"][pages, h].flatten(0, 1)[:n]), rot) / rot
                    for x in ("k", "v"))
            heads = slice(h * group, (h + 1) * group)
            q = st["q"][a:b, heads].double().transpose(0, 1)
            s = torch.matmul(q, k.t().contiguous()) * st["scale"]
            s = s.masked_fill(hidden, -INF)
            lse[a:b, heads] = torch.logsumexp(s, -1).t()
            out[a:b, heads] = torch.matmul(torch.softmax(s, -1), v).transpose(0, 1)
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    rot = case.get("rot")
    seeds = [st["seed"].long(), st["seed"].long() + 0x9E3779B9] if case.get("random") else [None, None]
    if case["op"] == "quant":
        out = {}
        for name, x, s in (("values", st["x"], seeds[0]), ("values_t", st["x"].t(), seeds[1])):
            if name == "values" or case["t"]:
                out[name] = (_turned64(_exact_values(x, rot, s), rot) / rot)[:, :x.shape[1]]
        return out
    if case["op"] == "linear" and not case["train"]:
        x = _exact_values(st["x"], rot)
        n = x.shape[1]
        w = _exact_codes(st["w_codes"][:, :n // 2], st["w_scales"][:, :n // 32])
        return {"y": torch.mm(x, w.t().contiguous()) / rot}
    if case["op"] == "linear":
        def product(a, b, s=None):
            return torch.mm(_exact_values(a, rot, s), _exact_values(b, rot).t().contiguous()) / rot

        return {"y": product(st["x"], st["w"]), "dx": product(st["dy"], st["w"].t(), seeds[0]),
                "dw": product(st["dy"].t(), st["x"].t(), seeds[1])}
    if case["op"] == "cache":
        H, rot = case["H"], case["D"] if rot else 1
        return {name: _turned64(_exact_values(st["qkv"][:, at:at + H], rot), rot) / rot
                for name, at in (("k", 4 * H), ("v", 5 * H))}
    return _exact_attn(st)

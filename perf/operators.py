"""Cases that measure the block-scaled FP8 operators and the AdamW step.

Three operators, each in a plain form (elementary torch operations in 32 bits) and through the
framework's entry points:

  quant   a matrix to FP8 E4M3 codes with one scale for each block of 128: ROWS blocks are 1 x 128
          along the row (and, for the transposed codes, 128 x 1 along the column), TILES blocks are
          128 x 128. s = absmax / 448 in fp32 (POW2: the smallest power of two not below it),
          code = the E4M3 value nearest to fp32(v * fp32(1/s)).
  serve   Y = X W^T for a few tokens: X is quantized in ROWS blocks within the call, W is kept as
          TILES codes.
  train   one step of a linear layer: W quantized in TILES blocks, X and dY in ROWS blocks, then
          Y = X W^T, dX = dY W and dW = dY^T X, the last over blocks of 128 tokens.
  adamw   one AdamW step over many tensors, states in 32 bits, or in 8 bits (E4M3 codes of m and of
          sqrt(v), one scale for each 128 elements, rounded at random without bias).
"""
import math

import torch

own = False

F32, POW2 = "f32", "pow2"
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch's activations before a projection: latency
        dict(name="quant_decode_rows", op="quant", rows=16, cols=4096, dtype="bf16", shape="rows",
             scale=F32, t=False),
        # a training batch's activations, both layouts in one pass
        dict(name="quant_train_both", op="quant", rows=8192, cols=13824, dtype="bf16",
             shape="rows", scale=F32, t=True),
        # a layer's fp32 master weights into tiles with power-of-two scales, both layouts
        dict(name="quant_weight_tiles", op="quant", rows=11008, cols=4096, dtype="fp32",
             shape="tiles", scale=POW2, t=True),
        # one token through an MLP projection: the weights' bytes
        dict(name="serve_1", op="serve", N=1, C=4096, D=11008, dtype="bf16", scale=F32),
        # a few sequences decoded together, power-of-two scales, fp16
        dict(name="serve_13_pow2", op="serve", N=13, C=11008, D=4096, dtype="fp16", scale=POW2),
        # a short prompt of an odd length
        dict(name="serve_1000", op="serve", N=1000, C=5120, D=13824, dtype="bf16", scale=F32),
        # a small layer with ragged sizes on every axis, fp32 outputs
        dict(name="train_ragged_fp32", op="train", N=1000, C=1030, D=778, dtype="fp32", scale=F32),
        # the MLP layer shape at full size, power-of-two scales
        dict(name="train_4096_pow2", op="train", N=4096, C=4096, D=11008, dtype="bf16",
             scale=POW2),
        # the largest layer
        dict(name="train_8192", op="train", N=8192, C=13824, D=5120, dtype="bf16", scale=F32),
        # norm gains, biases and learned steps: many short tensors
        dict(name="adamw_short_32", op="adamw", n=20000, tensors=12, bits=32, param="fp32",
             grad="fp32", copy=False),
        # a layer's weights in 32 bits with a bf16 copy for the next forward
        dict(name="adamw_layer_32", op="adamw", n=70778880, tensors=3, bits=32, param="fp32",
             grad="bf16", copy=True),
        # the same with 8-bit states
        dict(name="adamw_layer_8", op="adamw", n=70778880, tensors=5, bits=8, param="fp32",
             grad="bf16", copy=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm, odd ones among them."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "serve", "train", "adamw"])
    scale = rng.choice([F32, POW2])
    if op == "quant":
        rows = _spread(rng, 1, 8192)
        cols = _spread(rng, 16, min(16384, max(16, (8192 * 13824) // rows)))
        if rng.random() < 0.5:   # feature counts are usually whole 16-byte rows
            cols = (cols + 15) // 16 * 16
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["fp32", "fp16", "bf16"]),
                    shape=rng.choice(["rows", "tiles"]), scale=scale, t=rng.random() < 0.5)
    if op == "serve":
        C, D = _spread(rng, 256, 13824), _spread(rng, 256, 13824)
        if rng.random() < 0.7:
            C, D = (C + 15) // 16 * 16, (D + 15) // 16 * 16
        return dict(op=op, N=_spread(rng, 1, 2048), C=C, D=D, dtype=rng.choice(["fp16", "bf16"]),
                    scale=scale)
    if op == "train":
        C, D = _spread(rng, 128, 8192), _spread(rng, 128, 8192)
        if rng.random() < 0.7:
            C, D = (C + 15) // 16 * 16, (D + 15) // 16 * 16
        return dict(op=op, N=_spread(rng, 64, 8192), C=C, D=D,
                    dtype=rng.choice(["fp32", "fp16", "bf16", "bf16"]), scale=scale)
    return dict(op=op, n=_spread(rng, 1000, 40000000), tensors=rng.randint(1, 24),
                bits=rng.choice([8, 32]), param=rng.choice(["fp32", "fp32", "bf16"]),
                grad=rng.choice(["fp32", "bf16", "fp16"]), copy=rng.random() < 0.5)


def _lengths(case):
    """Lengths of the case's tensors: a geometric spread down to one element, odd ones among them."""
    n, k = case["n"], case["tensors"]
    return [max(1, n // 5 ** i - (i % 2)) for i in range(k)]


# ------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _normal(g, rows, cols, dtype, scale=1.0, outliers=0):
    """Normal values, a few columns of which are 50 times larger (the outlier channels of
    activations)."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    if outliers:
        at = torch.randint(0, cols, (outliers,), generator=g, device="cuda")
        x[:, at] *= 50.0
    return x.to(DT[dtype])


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": dict(case)}
    if case["op"] == "quant":
        st["x"] = _normal(g, case["rows"], case["cols"], case["dtype"], 1.0, 4)
    elif case["op"] == "serve":
        N, C, D = case["N"], case["C"], case["D"]
        st["x"] = _normal(g, N, C, case["dtype"], 1.0, 4)
        w = torch.randn(D, C, generator=g, device="cuda") * 0.02
        q, s = _quant_tiles(w, case["scale"])
        st["w_codes"] = torch.zeros(D, (C + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
        st["w_codes"][:, :C] = q.view(torch.uint8)
        st["w_scales"] = s
        st["y"] = torch.empty(N, D, dtype=DT[case["dtype"]], device="cuda")
    elif case["op"] == "train":
        N, C, D = case["N"], case["C"], case["D"]
        st["x"] = _normal(g, N, C, case["dtype"], 1.0, 4)
        st["w"] = _normal(g, D, C, case["dtype"], 0.02)
        # gradients: mostly small, with heavy tails
        dy = torch.randn(N, D, generator=g, device="cuda")
        st["dy"] = (1e-3 * dy * dy.square()).to(DT[case["dtype"]])
        for name, shape in (("y", (N, D)), ("dx", (N, C)), ("dw", (D, C))):
            st[name] = torch.empty(shape, dtype=DT[case["dtype"]], device="cuda")
    else:
        st.update(t=100, seed=int(seed) & 0xFFFF, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)
        st["tensors"] = [_adamw_inputs(g, n, case) for n in _lengths(case)]
    return st


def _adamw_inputs(g, n, case):
    def normal(scale):
        return torch.randn(n, generator=g, device="cuda") * scale

    size = torch.exp(normal(1.0))   # gradients whose size differs from element to element
    t = {"p": normal(0.02).to(DT[case["param"]]), "g": (normal(1e-3) * size).to(DT[case["grad"]])}
    if case["copy"]:
        t["copy"] = t["p"].to(torch.bfloat16)
    m, v = normal(3e-4) * size, (normal(1.0).square() + 0.1) * (1e-3 * size).square()
    if case["bits"] == 32:
        t["m"], t["v"] = m, v
    else:   # the codes of an earlier step
        for name, x in (("m", m), ("v", v.sqrt())):
            q, s = _quant_rows(x.view(1, -1), F32)
            t[name], t[name + "_s"] = q.view(torch.uint8).view(-1).contiguous(), s.view(-1).contiguous()
    return t


# ------------------------------------------------------------------------------------- plain forms
def _padded(x, br, bc):
    rows, cols = x.shape
    p = x.new_zeros((rows + br - 1) // br * br, (cols + bc - 1) // bc * bc)
    p[:rows, :cols] = x
    return p


def _scale_of(a, kind):
    """The scale of blocks with the largest magnitudes a, and its reciprocal."""
    # correctly rounded quotients, through 64 bits: the codes next to a border hang on them
    s = (a.double() / a.new_full((), 448.0).double()).float()
    if kind == POW2:
        bits = s.view(torch.int32)
        s = ((bits + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    s = torch.where(a > 0, s.clamp_min(2.0 ** -126), torch.zeros_like(s))
    return s, torch.where(s > 0, s.double().reciprocal().float(), torch.zeros_like(s))


def _quant_rows(x, kind):
    """E4M3 codes (rows x cols) and scales (column blocks x rows) in blocks of 1 x 128."""
    rows, cols = x.shape
    v = _padded(x.float(), 1, 128).view(rows, -1, 128)
    s, r = _scale_of(v.abs().amax(2), kind)
    q = (v * r[:, :, None]).clamp(-448.0, 448.0).to(E4M3)
    return q.view(rows, -1)[:, :cols], s.t().contiguous()


def _quant_tiles(x, kind):
    """E4M3 codes (rows x cols) and scales (row blocks x column blocks) in blocks of 128 x 128."""
    rows, cols = x.shape
    p = _padded(x.float(), 128, 128)
    v = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    s, r = _scale_of(v.abs().amax(dim=(1, 3)), kind)
    q = (v * r[:, None, :, None]).clamp(-448.0, 448.0).to(E4M3)
    return q.view(p.shape)[:rows, :cols], s


def _values_rows(q, s):
    """What ROWS codes and scales stand for, in fp32."""
    return q.float() * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _values_tiles(q, s):
    every = s.repeat_interleave(128, 0).repeat_interleave(128, 1)
    return q.float() * every[:q.shape[0], :q.shape[1]]


def _plain_quant(st):
    c, x = st["case"], st["x"]
    one = _quant_rows if c["shape"] == "rows" else _quant_tiles
    q, s = one(x, c["scale"])
    out = {"codes": q.contiguous(), "scales": s}
    if c["t"] and c["shape"] == "rows":
        q, s = _quant_rows(x.t(), c["scale"])
        out.update(codes_t=q.contiguous(), scales_t=s)
    elif c["t"]:
        out["codes_t"] = q.view(torch.uint8).t().contiguous().view(E4M3)
    return out


def _plain_serve(st):
    c = st["case"]
    x = _values_rows(*_quant_rows(st["x"], c["scale"]))
    w = _values_tiles(st["w_codes"][:, :c["C"]].view(E4M3), st["w_scales"])
    st["y"].copy_(x @ w.t())
    return {"y": st["y"]}


def _plain_train(st):
    kind = st["case"]["scale"]
    w = _values_tiles(*_quant_tiles(st["w"], kind))
    st["y"].copy_(_values_rows(*_quant_rows(st["x"], kind)) @ w.t())
    st["dx"].copy_(_values_rows(*_quant_rows(st["dy"], kind)) @ w)
    gt = _values_rows(*_quant_rows(st["dy"].t(), kind))
    xt = _values_rows(*_quant_rows(st["x"].t(), kind))
    st["dw"].copy_(gt @ xt.t())
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _mix(h):
    """The 32-bit mixing steps of the rounding's random numbers (h: int64 holding 32 bits)."""
    h = h ^ (h >> 16)
    h = (h * 2654435761) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 2891336453) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _key(seed, step, ordinal):
    k = int(_mix(torch.tensor((seed + 2654435761 * step) & 0xFFFFFFFF)))
    return (k + 0x9E3779B9 * (ordinal + 1)) & 0xFFFFFFFF


def _blocks(x):
    return _padded(x.view(1, -1), 1, 128).view(-1, 128)


def _round_m(m, random):
    """8-bit codes and scales of m: the two neighbours on the E4M3 grid, the upper one with the
    probability that makes the mean m (random: 16 bits for each element)."""
    b = _blocks(m)
    s, r = _scale_of(b.abs().amax(1), F32)
    x = (b.abs() * r[:, None]).clamp(max=448.0).view(-1)[:m.numel()]
    normal = ((x.view(torch.int32) + (random << 4).to(torch.int32)) >> 20) - 960
    small = (x * 512.0 + random.float() / 65536.0).to(torch.int32)
    code = torch.where(x >= 2.0 ** -6, normal, small)
    return torch.where(m < 0, code + 128, code).to(torch.uint8), s


def _round_v(v, random):
    """8-bit codes and scales of sqrt(v), rounded so that the mean of the square is v; a value
    above zero keeps a code above zero."""
    y = v.sqrt()
    b = _blocks(y)
    s, r = _scale_of(b.amax(1), F32)
    x = (b * r[:, None]).clamp(max=448.0).view(-1)[:v.numel()]
    normal = x >= 2.0 ** -6
    bits = x.view(torch.int32)
    code = torch.where(normal, (bits >> 20) - 960, (x * 512.0).to(torch.int32))
    low = torch.where(normal, (bits & -0x100000).view(torch.float32), code.float() / 512.0)
    step = torch.where(normal, (((bits >> 23) - 3) << 23).view(torch.float32),
                       torch.full_like(x, 1.0 / 512.0))
    up = (random.float() / 65536.0) * (step * (2.0 * low + step)) < (x - low) * (x + low)
    code = code + up.to(torch.int32)
    return torch.where(v > 0, code.clamp_min(1), code).to(torch.uint8), s


def _from_codes(q, s):
    return q.view(E4M3).float() * s.repeat_interleave(128)[:q.numel()]


def _plain_adamw_one(st, t, ordinal):
    b1, b2 = st["beta1"], st["beta2"]
    eight = st["case"]["bits"] == 8
    m, v = t["m"], t["v"]
    if eight:
        m, v = _from_codes(m, t["m_s"]), _from_codes(v, t["v_s"]).square()
    g = t["g"].float()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    den = v.sqrt() * (1.0 / math.sqrt(1.0 - b2 ** st["t"])) + st["eps"]
    p = t["p"].float() * (1.0 - st["lr"] * st["wd"]) - (st["lr"] / (1.0 - b1 ** st["t"])) * m / den
    t["p"].copy_(p)
    if "copy" in t:
        t["copy"].copy_(p)
    if eight:
        i = torch.arange(m.numel(), device=m.device)
        h = _mix(i ^ _key(st["seed"], st["t"], ordinal))
        for name, (q, s) in (("m", _round_m(m, h & 0xFFFF)), ("v", _round_v(v, h >> 16))):
            t[name].copy_(q)
            t[name + "_s"].copy_(s)
    else:
        t["m"].copy_(m)
        t["v"].copy_(v)


def _adamw_out(st):
    """Parameters, copies and states; 8-bit codes as the values they hold."""
    def shown(x):
        return x.view(E4M3) if x.dtype == torch.uint8 else x

    return [{k: shown(x) for k, x in t.items() if k != "g"} for t in st["tensors"][:8]]


def _plain_adamw(st):
    st["t"] += 1
    for k, t in enumerate(st["tensors"]):
        _plain_adamw_one(st, t, k)
    return _adamw_out(st)


# ------------------------------------------------------------------------------------- own calls
def _own(st):
    from hadamard_rotated_precision_amd import binding as B
    from hadamard_rotated_precision_amd import tensors as T

    c = st["case"]
    if c["op"] == "adamw":
        opt = st.get("kept")
        if opt is None:   # the optimizer that a program keeps, over its parameters and states
            ts = st["tensors"]
            opt = st["kept"] = T.AdamW(
                [t["p"] for t in ts], lr=st["lr"], betas=(st["beta1"], st["beta2"]), eps=st["eps"],
                weight_decay=st["wd"], state_bits=c["bits"], seed=st["seed"], steps_done=st["t"],
                copies=[t["copy"] for t in ts] if c["copy"] else None,
                states=[{"m": t["m"], "v": t["v"], "m_scales": t.get("m_s"),
                         "v_scales": t.get("v_s")} for t in ts])
            st["grads"] = [t["g"] for t in ts]
        opt.step(st["grads"])
        return _adamw_out(st)
    scale = B.HQ_BSCALE_POW2 if c["scale"] == POW2 else B.HQ_BSCALE_F32
    if c["op"] == "quant":
        q = st.get("kept")
        if q is None:
            q = st["kept"] = T.BlockTensor(
                c["rows"], c["cols"],
                shape=B.HQ_BLOCK_ROWS if c["shape"] == "rows" else B.HQ_BLOCK_TILES,
                scale=scale, codes_t=c["t"])
        q.quantize(st["x"])
        out = {"codes": q.codes_view().view(E4M3), "scales": q.scales}
        if c["t"]:
            out["codes_t"] = q.codes_t_view().view(E4M3)
            if c["shape"] == "rows":
                out["scales_t"] = q.scales_t
        return out
    layer = st.get("kept")
    if c["op"] == "serve":
        if layer is None:   # the layer around the weights that a server keeps
            w = T.BlockTensor.wrap(st["w_codes"], st["w_scales"], c["D"], c["C"],
                                   shape=B.HQ_BLOCK_TILES, scale=scale)
            layer = st["kept"] = T.BlockLayer(c["N"], c["C"], c["D"], scale=scale, weight=w,
                                              train=False)
        layer.fwd(st["x"], st["y"])
        return {"y": st["y"]}
    if layer is None:
        layer = st["kept"] = T.BlockLayer(c["N"], c["C"], c["D"], scale=scale)
    layer.set_weight(st["w"])
    layer.fwd(st["x"], st["y"])
    layer.bwd_input(st["dy"], st["dx"])
    layer.bwd_weight(st["dw"])
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "serve": _plain_serve, "train": _plain_train,
            "adamw": _plain_adamw}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- work
def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if case["op"] == "quant":
        r, c = case["rows"], case["cols"]
        rb, cb = -(-r // 128), -(-c // 128)
        scales = 4 * (r * cb + (c * rb if case["t"] else 0)) if case["shape"] == "rows" else 4 * rb * cb
        return {"bytes": r * c * (size[case["dtype"]] + 1 + case["t"]) + scales, "flops": 0}
    if case["op"] in ("serve", "train"):
        N, C, D, e = case["N"], case["C"], case["D"], size[case["dtype"]]
        if case["op"] == "serve":
            return {"bytes": D * C + 4 * -(-D // 128) * -(-C // 128) + e * (N * C + N * D),
                    "flops": 2 * N * C * D}
        return {"bytes": e * 2 * (N * C + D * C + N * D), "flops": 6 * N * C * D}
    n = sum(_lengths(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / 128
    return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + 2 * case["copy"] + state),
            "flops": 12 * n}


# ------------------------------------------------------------------------------------- in 64 bits
def _grid64(x):
    """The E4M3 value nearest to x (64 bits), ties to the even one; |x| <= 448."""
    _, e = torch.frexp(x)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return torch.round(x / ulp) * ulp


def _largest64(x, br, bc):
    """The largest magnitude of each br x bc block, at every element of x."""
    rows, cols = x.shape
    rb, cb = -(-rows // br), -(-cols // bc)
    a = torch.zeros(rb * br, cb * bc, dtype=torch.float64, device=x.device)
    a[:rows, :cols] = x.abs()
    a = a.reshape(rb, br, cb, bc).amax(3).amax(1)
    return a


def _exact_quant(x, br, bc, kind):
    """(codes' values, scales of the blocks) by the definition: s and 1/s are fp32 numbers, the
    product v * (1/s) is rounded to fp32, the code is its nearest E4M3 value."""
    x = x.double()
    a = _largest64(x, br, bc)
    s = (a / 448.0).float().double()
    if kind == POW2:
        f, e = torch.frexp(s)
        s = torch.where(a > 0, torch.exp2((e - (f == 0.5).int()).double()), s)
    s = torch.where(a > 0, s.clamp_min(2.0 ** -126), torch.zeros_like(s))
    r = torch.where(s > 0, (1.0 / s).float().double(), torch.zeros_like(s))
    at_r = torch.arange(x.shape[0], device=x.device) // br
    at_c = torch.arange(x.shape[1], device=x.device) // bc
    y = (x * r[at_r][:, at_c]).float().double().clamp(-448.0, 448.0)
    return _grid64(y), s


def _exact_values(x, br, bc, kind):
    q, s = _exact_quant(x, br, bc, kind)
    at_r = torch.arange(x.shape[0], device=x.device) // br
    at_c = torch.arange(x.shape[1], device=x.device) // bc
    return q * s[at_r][:, at_c]


def _exact_hash(h):
    for shift, factor in ((16, 2654435761), (15, 2891336453), (16, 1)):
        h = torch.remainder(torch.bitwise_xor(h, torch.div(h, 2 ** shift, rounding_mode="floor"))
                            * factor, 2 ** 32)
    return h


def _exact_adamw(st):
    out = []
    step = st["t"] + 1
    key = int(_exact_hash(torch.tensor((st["seed"] + 2654435761 * step) % 2 ** 32)))
    for k, t in enumerate(st["tensors"][:8]):
        n = t["p"].numel()
        eight = st["case"]["bits"] == 8
        at = torch.arange(n, device=t["p"].device)
        m, v = t["m"], t["v"]
        if eight:
            m = m.view(E4M3).double() * t["m_s"].double()[at // 128]
            v = (v.view(E4M3).double() * t["v_s"].double()[at // 128]) ** 2
        g = t["g"].double()
        m = st["beta1"] * m.double() + (1 - st["beta1"]) * g
        v = st["beta2"] * v.double() + (1 - st["beta2"]) * g ** 2
        mhat, vhat = m / (1 - st["beta1"] ** step), v / (1 - st["beta2"] ** step)
        p = t["p"].double()
        p = p - st["lr"] * (st["wd"] * p + mhat / (vhat.sqrt() + st["eps"]))
        one = {"p": p}
        if "copy" in t:
            one["copy"] = p
        if eight:
            h = _exact_hash(torch.bitwise_xor(at, torch.tensor((key + 0x9E3779B9 * (k + 1)) % 2 ** 32)))
            for name, value, u in (("m", m, h % 65536), ("v", v.sqrt(), h // 65536)):
                a = _largest64(value.view(1, -1), 1, 128).view(-1)
                s = torch.where(a > 0, (a / 448.0).clamp_min(2.0 ** -126), a)
                x = torch.where(s[at // 128] > 0, value.abs() / s[at // 128], value.abs())
                _, e = torch.frexp(x)
                ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
                low = torch.floor(x / ulp) * ulp
                if name == "m":
                    share = (x - low) / ulp
                else:
                    share = (x ** 2 - low ** 2) / ((low + ulp) ** 2 - low ** 2)
                u = u.double() / 65536
                q = low + ulp * ((u >= 1 - share) if name == "m" else (u < share)).double()
                if name == "v":
                    q = torch.where(value > 0, q.clamp_min(2.0 ** -9), q)
                one[name], one[name + "_s"] = torch.copysign(q, value), s
        else:
            one["m"], one["v"] = m, v
        out.append(one)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case.get("scale")
    if case["op"] == "quant":
        x = st["x"]
        if case["shape"] == "tiles":
            q, s = _exact_quant(x, 128, 128, kind)
            return {"codes": q, "scales": s, **({"codes_t": q.t().contiguous()} if case["t"] else {})}
        q, s = _exact_quant(x, 1, 128, kind)
        out = {"codes": q, "scales": s.t().contiguous()}
        if case["t"]:
            q, s = _exact_quant(x, 128, 1, kind)
            out.update(codes_t=q.t().contiguous(), scales_t=s)
        return out
    if case["op"] == "serve":
        s = st["w_scales"].double()
        at_r = torch.arange(case["D"], device="cuda") // 128
        at_c = torch.arange(case["C"], device="cuda") // 128
        w = st["w_codes"][:, :case["C"]].view(E4M3).double() * s[at_r][:, at_c]
        return {"y": torch.mm(_exact_values(st["x"], 1, 128, kind), w.t().contiguous())}
    if case["op"] == "train":
        w = _exact_values(st["w"], 128, 128, kind)
        y = torch.mm(_exact_values(st["x"], 1, 128, kind), w.t().contiguous())
        dx = torch.mm(_exact_values(st["dy"], 1, 128, kind), w)
        del w
        g = _exact_values(st["dy"], 128, 1, kind)
        return {"y": y, "dx": dx,
                "dw": torch.mm(g.t().contiguous(), _exact_values(st["x"], 128, 1, kind))}
    return _exact_adamw(st)

"""Plain references of the microscaled 4-bit operators, in 64 bits.

The quantizer's definition names its fp32 roundings: the sums of the rotation's butterflies (each is
taken here by rounding the exact 64-bit sum once) and, below 1, the sum of the random rounding. The
division by a power of two is exact. So codes and scale bytes are compared for equality.
"""
import math

import torch

from hadamard_rotated_precision_amd import binding as B
from hadamard_rotated_precision_amd import tensors as T

DEV = "cuda"
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def draw(g, rows, cols, dtype=torch.float32, scale=1.0):
    x = torch.randn(rows, cols, generator=g, device=DEV) * scale
    if cols > 4:
        x[:, 3] *= 30
    return x.to(dtype)


def blocks(n):
    return -(-n // 32)


def hadamard(x, k, cut=False):
    """H_k on every k elements of the last axis; cut: each butterfly's sum is an fp32 number."""
    h = 1
    while h < k:
        y = x.unflatten(-1, (-1, 2, h))
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).flatten(-3)
        x = y.float().double() if cut else y
        h *= 2
    return x


def mix(h):
    h = h ^ (h >> 16)
    h = (h * 2654435761) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 2891336453) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(seed, rows, cols):
    r = torch.arange(rows, device=DEV)[:, None]
    c = torch.arange(cols, device=DEV)
    h = mix(mix((seed + 2654435761 * r) & 0xFFFFFFFF) ^ (c // 2))
    return torch.where(c % 2 == 0, h & 0xFFFF, h >> 16)


def quantize(x, rot=1, seed=None):
    """(codes 0 .. 15, scale bytes) of the rows of x (any leading axes; with a seed: two axes)."""
    n = 32 * blocks(x.shape[-1])
    v = torch.zeros(*x.shape[:-1], n, dtype=torch.float64, device=x.device)
    v[..., :x.shape[-1]] = x.double()
    v = hadamard(v, rot, cut=True)
    a = v.unflatten(-1, (-1, 32)).abs().amax(-1)     # a NaN stays one
    bad = ~(a < math.inf)
    a = torch.where(bad, torch.ones_like(a), a)
    _, e = torch.frexp(a)
    e = torch.where(a > 0, e - 4, -126)              # 6 * 2^e < a for certain, or a tiny
    for _ in range(3):
        e = torch.where(6.0 * torch.exp2(e.double()) < a, e + 1, e)
    e = e.clamp_min(-126)
    y = v / torch.exp2(e.double()).repeat_interleave(32, -1)
    m = torch.where(bad.repeat_interleave(32, -1), torch.zeros_like(y), y).abs()
    grid = GRID.to(x.device)
    low = (torch.searchsorted(grid, m, right=True) - 1).clamp_max(6)
    share = (m - grid[low]) / (grid[low + 1] - grid[low])
    if seed is None:
        up = torch.where(share == 0.5, low % 2 == 1, share > 0.5)
    else:
        u = random_bits(seed, *v.shape).double() / 65536
        # below 1 the sum is an fp32 number; above, 16 of the dropped bits take part exactly
        whole = torch.where(low < 2, (2 * m + u).float().double() >= low + 1, share + u >= 1)
        up = whole
    code = low + up.long() + 8 * torch.signbit(v)
    code = torch.where(bad.repeat_interleave(32, -1), torch.zeros_like(code), code)
    return code.to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def pack(code):
    return code[..., ::2] + 16 * code[..., 1::2]


def values(code, scale):
    """What codes and scale bytes stand for (in the rotated space); byte 255: NaN."""
    v = GRID.to(code.device)[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
    s = torch.where(scale == 255, math.nan, torch.exp2(scale.double() - 127))
    return v * s.repeat_interleave(32, -1)


def held(q, side=0):
    """What a layout of an MxTensor holds, read from its buffers, in the rotated space."""
    codes, scales, n = (q.codes, q.scales, q.cols) if side == 0 else (q.codes_t, q.scales_t, q.rows)
    nb = blocks(n)
    return values(unpack(codes[:, :16 * nb]), scales[:, :nb])


def product_bound(a, b, c, rot, dtype):
    """Largest error of c = a b^T / rot for values a (M x K) and b (N x K) of codes in 64 bits. S =
    sum |a b| / rot bounds every partial sum. Products of codes and sums of a block are multiples of
    a quarter below 32 * 36, so exact; the blocks are added in fp32, at most 4 in an instruction and one for
    each instruction, split sum or group: fewer than K / 32 + 32 additions of 2^-23 S each (an
    instruction may cut instead of rounding). Then the output's own rounding (half a step of its type;
    steps of 2^-24 below 2^-14 for fp16, sums below 2^-126 may be lost)."""
    S = torch.mm(a.abs(), b.abs().t().contiguous()) / rot
    err = (blocks(a.shape[1]) + 32) * 2.0 ** -23 * S
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    return err + HALF_STEP[dtype] * (c.abs() + err) + tiny


def assert_within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    n = int(bad.sum())
    worst = float((off / bound).max()) if off.numel() else 0.0
    print("[bound] %s: worst error / bound %.3g of %d values" % (what, worst, off.numel()), flush=True)
    assert n == 0, "%s: %d values outside the bound, worst error / bound %.3g" % (what, n, worst)


# ------------------------------------------------------------------ the cache and its attention
def rows_of(cache, slots):
    return slots // cache.page, slots % cache.page


def cached(cache, name, pages, rows):
    """Rotated-space values (n x heads x D) at page indexes and rows."""
    codes, scales = ((cache.k_codes, cache.k_scales) if name == "k" else (cache.v_codes, cache.v_scales))
    return values(unpack(codes[pages, :, rows]), scales[pages, :, rows])


def fill(cache, g, spread=4.0):
    """Random codes and scales (of 2^-spread .. 2^spread) in the whole cache."""
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        codes.random_(0, 256, generator=g)
        e = torch.rand(scales.shape, generator=g, device=DEV) * 2 * spread - spread
        scales.copy_((e + 127).round().to(torch.uint8))


def attention(cache, q, starts, lens, table, scale, window, dtype):
    """(out, lse, bound of out, bound of lse) in 64 bits, rows of no sequence as NaN.

    The bounds count, for parts = bf16 numbers that a probability is split into (3 with fp32 in or out:
    2^-25, else 2^-17) and a row that sees n tokens:
      scores    q: its rotation (log2 D stages and the scaling, each half a step of sums below sum |q|
                in magnitude), its split; the products' sum: parts D additions. d_j below.
                The split into 6-bit numbers (E2M3: steps of 1/8 below 2, 1/4 below 4, 1/2 up to 7.5),
                each with a scale s of the block of 32, the smallest power of two with max |q| <= 7.5 s,
                so s < max |q| / 3.75. The first leaves at most s / 4, which is 4 of the second's
                s / 16; that leaves 1/8 of its scale, 4 of the third's at 2^-5 of it, and so on. After
                four: s 2^(-3 - 4 - 5 - 5) = s 2^-17, below 2^-18 max |q|; after six (fp32): s 2^-27,
                below 2^-28 max |q|. It is relative to the block's largest, so an element's error is
                multiplied with |k| by itself.
      p_j       the score's error d_j, the rounding of s_j - m (in powers of two, twice half a step of
                |s_j| + |m|), the exponential's two steps, its split: e_j.
      sums      n + 64 additions in fp32 for each part, of sums below sum p |v|, and the same for l.
      output    two steps of the division, its rotation back (log2 D + 1), its own rounding."""
    heads, D = cache.heads, cache.head_dim
    rot = D if cache.st.rot > 1 else 1
    tokens, Hq = q.shape[:2]
    group = Hq // heads
    parts = 3 if torch.float32 in (q.dtype, dtype) else 2
    cut, u, stages = 2.0 ** (-25 if parts == 3 else -17), 2.0 ** -24, math.log2(D) + 1
    out = torch.full((tokens, Hq, D), math.nan, dtype=torch.float64, device=DEV)
    lse, out_err, lse_err = out[..., 0].clone(), out.clone(), out[..., 0].clone()
    qr = hadamard(q.double(), rot) if rot > 1 else q.double()
    for s in range(len(lens)):
        a, b, n = starts[s], starts[s + 1], lens[s]
        if b <= a:
            continue
        if n == 0:
            out[a:b], lse[a:b], out_err[a:b], lse_err[a:b] = 0.0, -math.inf, 0.0, 0.0
            continue
        at = torch.arange(n, device=DEV)
        entry = at // cache.page
        named = torch.full((n,), -1, dtype=torch.long, device=DEV)
        inside = entry < table.shape[1]
        named[inside] = table[s].long()[entry[inside]]
        ok = (named >= 0) & (named < cache.pages)
        named = torch.where(ok, named, 0)
        k, v = (cached(cache, x, named, at % cache.page) for x in ("k", "v"))
        pos = n - (b - a) + torch.arange(b - a, device=DEV)[:, None]
        seen = (at <= pos) & ok
        if window:
            seen &= at > pos - window
        for h in range(Hq):
            kh, vh, x = k[:, h // group], v[:, h // group], qr[a:b, h]
            kz = torch.where(seen.any(0)[:, None], kh, 0.0)
            sc = abs(scale) / rot
            sj = torch.mm(x, kz.t().contiguous()) * (scale / rot)
            big = torch.mm(x.abs(), kz.abs().t().contiguous()) * sc
            total = q[a:b, h].double().abs().sum(-1, keepdim=True) if rot > 1 else x.abs().amax(-1, keepdim=True)
            largest = x.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
            split = torch.mm(largest, kz.abs().t().contiguous()) * sc * 2.0 ** (-28 if parts == 3 else -18)
            d = split + big * parts * D * u + total * kz.abs().sum(-1) * sc * stages * u
            sj = sj.masked_fill(~seen, -math.inf)
            m = sj.amax(-1, keepdim=True)
            some = seen.any(-1)
            w = torch.softmax(torch.where(some[:, None], sj, 0.0), -1) * seen
            zero = torch.where(seen, sj, 0.0).abs() + torch.where(some[:, None], m, 0.0).abs()
            e = torch.expm1(d + 2 * u * zero + 4 * u) + cut + (n + 64) * parts * u
            # a weight of 0 hides whatever its value is
            def weighed(y):
                return torch.mm(w, torch.where(seen.any(0)[:, None], y, 0.0))

            o = weighed(vh)
            err = torch.mm(w * e, torch.where(seen.any(0)[:, None], vh.abs(), 0.0))
            off_l = (w * e).sum(-1, keepdim=True)
            err = err + off_l * o.abs() + 4 * u * o.abs()
            if rot > 1:
                err = err.sum(-1, keepdim=True) / D + stages * u * o.abs().sum(-1, keepdim=True) / D
                o = hadamard(o, D) / D
            tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
            out[a:b, h] = o
            out_err[a:b, h] = err * 1.01 + HALF_STEP[dtype] * (o.abs() + err) + tiny
            lse[a:b, h] = torch.where(some, torch.logsumexp(torch.where(some[:, None], sj, 0.0), -1), -math.inf)
            lse_err[a:b, h] = (off_l[:, 0] * 1.01 + torch.where(some, lse[a:b, h].abs() + m[:, 0].abs(), 0.0) * 4 * u
                               + 4 * u)
    return out, lse, out_err, lse_err


def batch(g, cache, news, lens, extra_pages=0):
    """(starts, lens, table) on the device, with pages of the cache in random order, each its own."""
    need = [-(-n // cache.page) for n in lens]
    order = torch.randperm(cache.pages, generator=g, device=DEV).int()
    assert sum(need) <= cache.pages
    table = torch.full((len(lens), max([1, *need]) + extra_pages), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = [sum(news[:i]) for i in range(len(news) + 1)]
    return starts, table


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def new_cache(pages, page, heads, D, rotate=True):
    return T.KVCache(pages, page, heads, D, rotate=rotate)


assert B.HQ_MX_BLOCK == 32

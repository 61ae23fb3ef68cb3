"""Plain references of the block-scaled FP8 operators and of AdamW, in 64 bits.

The quantizer's definition names its fp32 roundings (s = fp32(a / 448), r = fp32(1 / s), the
product fp32(v r)); each is taken here by rounding the exact 64-bit result once, so codes and
scales are compared for equality. (fp64 holds a product of two fp32 numbers exactly, and rounding
an fp64 quotient of fp32 numbers to fp32 is the correctly rounded quotient: 53 >= 2 * 24 + 2.)
"""
import torch

from hadamard_rotated_precision_amd import binding as B

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def grid(x):
    """The E4M3 value nearest to x (fp64, |x| <= 448), ties to the even one."""
    _, e = torch.frexp(x)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return torch.round(x / ulp) * ulp


def block_max(x, br, bc):
    rows, cols = x.shape
    rb, cb = -(-rows // br), -(-cols // bc)
    p = torch.zeros(rb * br, cb * bc, dtype=torch.float64, device=x.device)
    p[:rows, :cols] = x.abs()
    return p.reshape(rb, br, cb, bc).amax(3).amax(1)


def scales_of(a, kind):
    s = (a / 448.0).float().double()
    if kind == B.HQ_BSCALE_POW2:
        f, e = torch.frexp(s)
        s = torch.where(a > 0, torch.exp2((e - (f == 0.5).int()).double()), s)
    s = torch.where(a > 0, s.clamp_min(2.0 ** -126), torch.zeros_like(s))
    r = torch.where(s > 0, (1.0 / s).float().double(), torch.zeros_like(s))
    return s, r


def spread(s, br, bc, shape):
    at_r = torch.arange(shape[0], device=s.device) // br
    at_c = torch.arange(shape[1], device=s.device) // bc
    return s[at_r][:, at_c]


def quantize(x, br, bc, kind=B.HQ_BSCALE_F32):
    """(code values, scales by block) of x in br x bc blocks."""
    x = x.double()
    s, r = scales_of(block_max(x, br, bc), kind)
    y = (x * spread(r, br, bc, x.shape)).float().double().clamp(-448.0, 448.0)
    return grid(y), s


def values(x, br, bc, kind=B.HQ_BSCALE_F32):
    q, s = quantize(x, br, bc, kind)
    return q * spread(s, br, bc, x.shape)


def largest_of_groups(a, b):
    """Sum over the groups of eight consecutive k of the largest |a[m][k] b[n][k]|."""
    a, b = a.abs(), b.abs()
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 8):
        big = torch.zeros_like(out)
        for i in range(k, min(k + 8, a.shape[1])):
            torch.maximum(big, torch.outer(a[:, i], b[:, i]), out=big)
        out += big
    return out


def product_bound(a, b, c, dtype):
    """Largest error of a product of the values a (M x K) and b (N x K) of codes, both 64-bit,
    whose exact result is c. S = sum |a b| bounds every partial sum.
    fp32 outputs: sums of exact products in fp32, at most 128 additions inside a block, one per
    block, two roundings of the scales' product and its application: (128 + blocks + 3) 2^-24 S.
    16-bit outputs: the FP8 instruction aligns each group of eight consecutive products to the
    exponent of the largest (which is at most that product's magnitude P) and cuts the other seven
    13 bits below: a measured 2^16 + 2^3 is exact and 2^16 + x is 2^16 for every x < 2^3. So a group
    is off by less than 7 * 2^-13 P; the groups' sums are added in fp32, cut rather than rounded:
    2^-23 S for each of the K / 8.
    Then the output's own rounding (half a step of its type; fp16 has steps of 2^-24 below 2^-14,
    fp32 and bf16 sums below 2^-126 may be lost)."""
    S = torch.mm(a.abs(), b.abs().t().contiguous())
    nb = -(-a.shape[1] // 128)
    err = (128 + nb + 3) * 2.0 ** -24 * S
    if dtype != torch.float32:
        err = err + 7 * 2.0 ** -13 * largest_of_groups(a, b) + (a.shape[1] // 8 + 1) * 2.0 ** -23 * S
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    return err + HALF_STEP[dtype] * (c.abs() + err) + tiny


def assert_within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    n = int(bad.sum())
    worst = float((off / bound).max()) if off.numel() else 0.0
    print("[bound] %s: worst error / bound %.3g of %d values" % (what, worst, off.numel()), flush=True)
    assert n == 0, "%s: %d values outside the bound, worst error / bound %.3g" % (what, n, worst)

"""Microscaled 4-bit operators against 64-bit references: the quantizer (codes and scale bytes equal),
the products in every form, the layer calls, graphs, streams and refusals."""
import math

import pytest
import torch

import mx_testlib as R
from hadamard_rotated_precision_amd import binding as B
from hadamard_rotated_precision_amd import tensors as T
from mx_testlib import draw, gen

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
COLS = B.HQ_SIDE_COLS


def seed_of(n):
    return torch.tensor([n], dtype=torch.int32, device=DEV)


def check_quantized(q, x, seed=None):
    """Codes and scale bytes of an MxTensor equal the definition's, and what lies past them is zero."""
    for side, codes, scales, y in ((0, q.codes, q.scales, x), (1, q.codes_t, q.scales_t, x.t())):
        if codes is None:
            continue
        n = R.blocks(y.shape[1])
        key = None if seed is None else (seed + side * 0x9E3779B9) & 0xFFFFFFFF
        want, s = R.quantize(y, q.rot, key)
        assert torch.equal(scales[:, :n], s), "scales of side %d" % side
        assert torch.equal(R.unpack(codes[:, :16 * n]), want), "codes of side %d" % side
        assert not scales[:, n:T.pitch16(n)].any()
        if q.rot == 1:
            assert not (R.unpack(codes[:, :16 * n])[:, y.shape[1]:]).any()


def fresh(rows, cols, **kw):
    """An MxTensor whose buffers hold other bytes than it will."""
    q = T.MxTensor(rows, cols, **kw)
    for t in (q.codes, q.codes_t, q.scales, q.scales_t):
        if t is not None:
            t.fill_(0xA7)
    return q


SIZES = [(1, 1), (1, 32), (1, 4096), (3, 17), (16, 33), (31, 31), (32, 32), (33, 130), (127, 129),
         (128, 128), (257, 1000), (640, 384), (1000, 1030), (2, 20000), (20000, 3), (4100, 2050)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("rot", [1, 32])
@pytest.mark.parametrize("random", [False, True])
def test_quantize_sizes(rows, cols, rot, random):
    for k, dtype in enumerate(DTYPES):
        x = draw(gen(rows + cols + k), rows, cols, dtype)
        seed = 12345 + k if random else None
        for kw in (dict(), dict(codes=False), dict(codes_t=False)):
            q = fresh(rows, cols, rot=rot, **kw).quantize(x, seed=None if seed is None else seed_of(seed))
            check_quantized(q, x, seed)


@pytest.mark.parametrize("rot", [1, 32])
def test_quantize_many_scales(rot):
    x = draw(gen(3), 4096, 8192)
    x *= torch.exp2(torch.rand(4096, 1, generator=gen(4), device=DEV) * 60 - 30)
    q = T.MxTensor(4096, 8192, rot=rot).quantize(x)
    for r in range(0, 4096, 1024):
        want, s = R.quantize(x[r:r + 1024], rot)
        assert torch.equal(q.scales[r:r + 1024], s)
        assert torch.equal(R.unpack(q.codes[r:r + 1024]), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("random", [False, True])
def test_quantize_extreme_magnitudes(dtype, random):
    """Blocks of zeros (of either sign), of one value, of subnormals, near the largest number, and
    spread over the whole exponent range; values on grid points and on midpoints between them."""
    top = torch.finfo(dtype).max
    g = gen(9)
    x = torch.zeros(200, 512, dtype=torch.float64, device=DEV)
    x[0] = 1.0
    x[1] = 1e-40
    x[2] = top * torch.rand(512, generator=g, device=DEV).double()
    x[3] = torch.exp2(torch.rand(512, generator=g, device=DEV).double() * 250 - 126).clamp_max(top)
    x[4, ::2] = 6.0
    x[5] = 2.0 ** -126
    x[6] = 2.0 ** -126 * torch.rand(512, generator=g, device=DEV).double()
    x[7] = -0.0
    grid = R.GRID.to(DEV)
    x[8, :8], x[8, 8] = grid, -6.0
    x[9, :7], x[9, 7] = (grid[1:] + grid[:-1]) / 2, 6.0
    x[9, 32:39], x[9, 39] = -(grid[1:] + grid[:-1]) / 2, 6.0
    x[10, ::32] = 3.0 + 2.0 ** -7     # just above and at 6 s and 3 s
    x[11, ::32] = 1.5
    x[12, ::32], x[12, 1::32] = 1.5 * 2.0 ** -24, 2.0 ** -24
    x[13, 5] = -7.0
    x[20:] = draw(g, 180, 512)
    x = x.to(dtype)
    check_quantized(fresh(200, 512, rot=1).quantize(x, seed=seed_of(7) if random else None), x, 7 if random else None)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rot", [1, 32])
@pytest.mark.parametrize("random", [False, True])
def test_not_finite_blocks_are_nan_and_others_are_not(bad, rot, random):
    x = draw(gen(2), 200, 300, torch.bfloat16)
    x[130, 200] = bad
    seed = seed_of(3) if random else None
    q = fresh(200, 300, rot=rot).quantize(x, seed=seed)
    check_quantized(q, x, 3 if random else None)
    assert (q.scales[:, :10] == 255).sum() == 1 and q.scales[130, 6] == 255
    assert (q.scales_t[:, :7] == 255).sum() == 1 and q.scales_t[200, 4] == 255
    w = T.MxTensor(96, 300, rot=rot).quantize(draw(gen(3), 96, 300))
    for dtype in DTYPES:
        c = torch.zeros(200, 96, dtype=dtype, device=DEV)
        T.mx_gemm(q, w, c)
        assert c[130].isnan().all() and c.isnan().sum() == 96
        y = q.dequantize(torch.zeros(200, 300, dtype=dtype, device=DEV))
        assert y[130, 192:224].isnan().all() and y.isnan().sum() == 32


def test_a_rotated_sum_past_fp32_is_nan():
    x = torch.full((1, 64), 3e38, device=DEV)
    x[0, 32:] = 1.0
    q = T.MxTensor(1, 64, codes_t=False).quantize(x)
    check_quantized(q, x)
    assert q.scales[0, 0] == 255 and q.scales[0, 1] != 255


def test_random_rounding_is_unbiased_and_follows_its_seed():
    """The mean over seeds of a code is its value: 4000 roundings of 2048 values, whose mean has a
    standard deviation of at most half a step / sqrt(4000) (a rounding to either side at worst); six of
    them hold for 2048 values and more (a share of 2e-9 each lies outside)."""
    x = torch.empty(1, 2048, device=DEV).uniform_(-6.0, 6.0, generator=gen(5))
    x[0, ::32] = 6.0            # the scale is 1
    total = torch.zeros(1, 2048, dtype=torch.float64, device=DEV)
    q, seed, n = T.MxTensor(1, 2048, rot=1, codes_t=False), seed_of(0), 4000
    for i in range(n):
        seed.fill_(1000003 * i % 2 ** 31)
        total += R.held(q.quantize(x, seed=seed))
    m = x.abs().double()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    # 16 random bits: the mean may lie 2^-16 steps from the value
    assert ((total / n - x.double()).abs() <= 6 * 0.5 * step / math.sqrt(n) + step * 2.0 ** -16).all()
    a, b = T.MxTensor(64, 512), T.MxTensor(64, 512)
    y = draw(gen(6), 64, 512, torch.bfloat16)
    a.quantize(y, seed=seed_of(1))
    b.quantize(y, seed=seed_of(1))
    assert torch.equal(a.codes, b.codes) and torch.equal(a.codes_t, b.codes_t)
    b.quantize(y, seed=seed_of(2))
    assert not torch.equal(a.codes, b.codes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", [1, 3])
def test_any_element_may_be_the_first(dtype, off):
    rows, cols = 70, 133
    flat = draw(gen(8), 1, rows * cols + off, dtype).view(-1)
    x = flat[off:].view(rows, cols)
    q = fresh(rows, cols).quantize(x)
    check_quantized(q, x)
    buf = torch.zeros(rows * cols + off + 8, dtype=dtype, device=DEV)
    q.dequantize(buf[off:off + rows * cols].view(rows, cols))
    want = torch.empty(rows, cols, dtype=dtype, device=DEV)
    q.dequantize(want)
    assert torch.equal(buf[off:off + rows * cols].view(rows, cols), want)
    assert not buf[:off].any() and not buf[off + rows * cols:].any()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 17), (33, 130), (128, 4096), (300, 2081)])
@pytest.mark.parametrize("rot", [1, 32])
def test_dequantize(rows, cols, rot):
    """A value is rounded once: sums of 32 codes are exact. (fp32 values below 2^-126 have a coarser
    step, 2^-149, as fp16's below 2^-14 have.)"""
    x = draw(gen(rows + cols), rows, cols)
    x[0] *= 2.0 ** -120
    q = T.MxTensor(rows, cols, rot=rot).quantize(x)
    for side, shape in ((0, (rows, cols)), (COLS, (cols, rows))):
        want = R.hadamard(R.held(q, side), rot)[:, :shape[1]] / rot
        for dtype in DTYPES:
            got = q.dequantize(torch.full(shape, 7.0, dtype=dtype, device=DEV), side=side)
            assert torch.equal(got, want.to(dtype))


def test_dequantize_reads_every_scale_byte():
    """Bytes 0 (2^-127) to 254, and 255 as NaN."""
    codes = torch.full((256, 16), 0x21, dtype=torch.uint8, device=DEV)    # 0.5, 1.0, ...
    scales = torch.zeros(256, 16, dtype=torch.uint8, device=DEV)
    scales[:, 0] = torch.arange(256, device=DEV)
    q = T.MxTensor.wrap(codes, scales, 256, 32, rot=1)
    got = q.dequantize(torch.empty(256, 32, device=DEV)).double()
    want = torch.exp2(torch.arange(255, device=DEV).double() - 127)[:, None] * torch.tensor([0.5, 1.0], device=DEV).repeat(16)
    assert torch.equal(got[:255], want) and got[255].isnan().all()


# M, N, K: one row, tails on every axis, K below, at and above a block and a step; every tile size,
# split sums, more large tiles than compute units
PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 777, 1000), (2, 300, 4096), (13, 64, 255), (16, 513, 640),
            (16, 40, 11008), (17, 64, 31), (32, 100, 5000), (33, 129, 33), (33, 129, 9000), (64, 64, 256),
            (100, 1000, 272), (256, 256, 512), (300, 260, 1030), (513, 700, 384), (1, 4096, 16),
            (1000, 3, 200), (2000, 1500, 544), (4096, 2048, 320), (5000, 4100, 257), (1, 13000, 300)]


def operands(M, N, K, rot, seed=0, codes_t=False):
    g = gen(M + 3 * N + 7 * K + seed)
    a, b = draw(g, M, K, torch.bfloat16), draw(g, N, K, torch.bfloat16, 0.02)
    return [T.MxTensor(*x.shape, rot=rot, codes_t=codes_t).quantize(x) for x in (a, b)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("rot", [1, 32])
def test_products(M, N, K, rot):
    a, b = operands(M, N, K, rot)
    va, vb = R.held(a), R.held(b)
    want = torch.mm(va, vb.t().contiguous()) / rot
    for dtype in DTYPES:
        c = torch.full((M, N), math.nan, dtype=dtype, device=DEV)
        T.mx_gemm(a, b, c)
        R.assert_within(c, want, R.product_bound(va, vb, want, rot, dtype), "product %s" % dtype)
        again = torch.empty_like(c)
        T.mx_gemm(a, b, again)
        assert torch.equal(c, again)


@pytest.mark.parametrize("M,N,K", [(3, 50, 96), (70, 130, 333), (300, 520, 1000)])
def test_products_of_either_side_and_accumulation(M, N, K):
    g = gen(M)
    a = T.MxTensor(K, M).quantize(draw(g, K, M))          # its transpose is the operand
    b = T.MxTensor(K, N).quantize(draw(g, K, N))
    va, vb = R.held(a, 1), R.held(b, 1)
    product = torch.mm(va, vb.t().contiguous()) / 32
    for dtype in DTYPES:
        c0 = draw(g, M, N, dtype)
        c = c0.clone()
        T.mx_gemm(a, b, c, a_side=COLS, b_side=COLS, accumulate=True)
        want = product + c0.double()
        # one more addition in fp32
        more = 2.0 ** -23 * (c0.double().abs() + product.abs())
        R.assert_within(c, want, R.product_bound(va, vb, want, 32, dtype) + more, "accumulated %s" % dtype)
    mixed = T.MxTensor(N, K).quantize(draw(g, N, K))
    c = torch.empty(M, N, device=DEV)
    T.mx_gemm(a, mixed, c, a_side=COLS)
    vm = R.held(mixed)
    want = torch.mm(va, vm.t().contiguous()) / 32
    R.assert_within(c, want, R.product_bound(va, vm, want, 32, torch.float32), "mixed sides")


def test_products_over_the_whole_range_of_scales():
    """Scales from 2^-126 to 2^126 on one side against their inverses on the other, and scales whose
    product leaves fp32: infinite above, zero below."""
    g = gen(12)
    a, b = draw(g, 40, 256), draw(g, 50, 256)
    e = torch.arange(40, device=DEV) * 6 - 118
    a *= torch.exp2(e.float())[:, None]
    qa, qb = T.MxTensor(40, 256).quantize(a), T.MxTensor(50, 256).quantize(b)
    va, vb = R.held(qa), R.held(qb)
    want = torch.mm(va, vb.t().contiguous()) / 32
    c = torch.empty(40, 50, device=DEV)
    T.mx_gemm(qa, qb, c)
    bound = R.product_bound(va, vb, want, 32, torch.float32)
    # partial sums are below 32 sum |a b| / 32: where that passes fp32 they may be infinite
    fits = torch.mm(va.abs(), vb.abs().t().contiguous()) < 2.0 ** 128
    assert fits.float().mean() > 0.95
    R.assert_within(c[fits], want[fits], bound[fits], "wide scales")
    tiny = T.MxTensor(50, 256).quantize(b * 2.0 ** -100)
    T.mx_gemm(qa, tiny, c)
    low = torch.mm(va, R.held(tiny).t().contiguous()) / 32
    R.assert_within(c, low, R.product_bound(va, R.held(tiny), low, 32, torch.float32) + 2.0 ** -126, "small scales")
    huge = T.MxTensor(50, 256).quantize(b * 2.0 ** 100)
    T.mx_gemm(qa, huge, c)
    assert not c[-1].isfinite().any() and c[0].isfinite().all()


def test_few_tokens_take_the_same_values_as_their_codes():
    """The fused form quantizes as hq_mx_quantize does."""
    for N, C, D, rot in ((1, 4096, 1000, 32), (5, 333, 70, 32), (16, 1000, 130, 1), (8, 2048, 64, 32), (3, 50, 5, 1)):
        for dtype in DTYPES:
            x = draw(gen(N), N, C, dtype)
            w = T.MxTensor(D, C, rot=rot).quantize(draw(gen(C), D, C, torch.float32, 0.02))
            y = torch.empty(N, D, device=DEV)
            T.MxLayer(N, C, D, weight=w, train=False).fwd(x, y)
            q = T.MxTensor(N, C, rot=rot, codes_t=False).quantize(x)
            c = torch.empty_like(y)
            T.mx_gemm(q, w, c)
            assert torch.equal(y, c)


@pytest.mark.parametrize("N,C,D", [(1, 64, 40), (40, 100, 70), (130, 333, 260), (600, 512, 1000)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rot,random", [(32, False), (32, True), (1, True)])
def test_layer_step(N, C, D, dtype, rot, random):
    g = gen(N + C)
    x, w, dy = draw(g, N, C, dtype), draw(g, D, C, dtype, 0.05), draw(g, N, D, dtype, 1e-2)
    layer = T.MxLayer(N, C, D, rot=rot)
    seed = seed_of(77) if random else None
    y, dx, dw = (torch.empty(s, dtype=dtype, device=DEV) for s in ((N, D), (N, C), (D, C)))
    layer.set_weight(w)
    layer.fwd(x, y)
    layer.bwd_input(dy, dx, seed=seed)
    layer.bwd_weight(dw)
    check_quantized(layer.qw, w)
    check_quantized(layer.qx, x)
    check_quantized(layer.qg, dy, 77 if random else None)
    for name, got, a, b in (("y", y, R.held(layer.qx), R.held(layer.qw)),
                            ("dx", dx, R.held(layer.qg), R.held(layer.qw, 1)),
                            ("dw", dw, R.held(layer.qg, 1), R.held(layer.qx, 1))):
        want = torch.mm(a, b.t().contiguous()) / rot
        R.assert_within(got, want, R.product_bound(a, b, want, rot, dtype), name)
    before = dw.clone()
    layer.bwd_weight(dw, accumulate=True)
    a, b = R.held(layer.qg, 1), R.held(layer.qx, 1)
    want = torch.mm(a, b.t().contiguous()) / rot + before.double()
    R.assert_within(dw, want, R.product_bound(a, b, want, rot, dtype) + 2.0 ** -23 * (want.abs() + before.double().abs()),
                    "accumulated dw")


def test_gradients_against_differences():
    """On values that the codes hold exactly the layer is bilinear, so differences of sum(dy * y) are
    its gradients, without a remainder: whole numbers and halves whose sums stay exact in fp32."""
    N, C, D = 64, 96, 64
    g = gen(21)

    def on_grid(rows, cols):
        x = R.GRID.to(DEV)[torch.randint(0, 8, (rows, cols), generator=g, device=DEV)].float()
        x *= torch.randint(0, 2, (rows, cols), generator=g, device=DEV) * 2 - 1
        x[::32] = 6.0        # every block, of either layout, has the scale 1
        x[:, ::32] = 6.0
        return x

    x, w, dy = on_grid(N, C), on_grid(D, C), on_grid(N, D)
    layer = T.MxLayer(N, C, D, rot=1)

    def loss():
        y = torch.empty(N, D, device=DEV)
        layer.set_weight(w)
        layer.fwd(x, y)
        return float((y.double() * dy.double()).sum())

    at = loss()
    dx, dw = torch.empty(N, C, device=DEV), torch.empty(D, C, device=DEV)
    layer.bwd_input(dy, dx)
    layer.bwd_weight(dw)
    for t, grad in ((x, dx), (w, dw)):
        for i, j in ((1, 1), (5, 40), (33, 95), (63, 2)):
            old = float(t[i, j])
            step = -2.0 * old if old else 2.0      # to another value of the grid
            t[i, j] = old + step
            assert loss() - at == step * float(grad[i, j])
            t[i, j] = old


def test_a_captured_step_follows_its_inputs_and_seed():
    N, C, D = 64, 256, 96
    g = gen(31)
    x, w, dy = draw(g, N, C, torch.bfloat16), draw(g, D, C, torch.bfloat16), draw(g, N, D, torch.bfloat16)
    layer, seed = T.MxLayer(N, C, D), seed_of(1)
    y, dx, dw = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((N, D), (N, C), (D, C)))

    def step():
        layer.set_weight(w)
        layer.fwd(x, y)
        layer.bwd_input(dy, dx, seed=seed)
        layer.bwd_weight(dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(draw(g, N, C, torch.bfloat16))
        dy.copy_(draw(g, N, D, torch.bfloat16))
        seed.fill_(100 + i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.zero_()
        step()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    g = gen(41)
    jobs = []
    for k in range(2):
        N, C, D = 300 + k, 512, 700
        x = draw(g, N, C, torch.bfloat16)
        layer = T.MxLayer(N, C, D, train=False)
        layer.set_weight(draw(g, D, C, torch.bfloat16))
        want, got = (torch.zeros(N, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        layer.fwd(x, want)
        jobs.append((layer, x, want, got, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, x, want, got, stream in jobs:
            layer.fwd(x, got, stream=stream)
    torch.cuda.synchronize()
    for _, _, want, got, _ in jobs:
        assert torch.equal(want, got)


def test_wrapped_weights_of_a_wider_buffer():
    """Pitches beyond the codes' own, and neighbours that are not zero."""
    D, C, N = 70, 100, 5
    q = T.MxTensor(D, C, codes_t=False).quantize(draw(gen(51), D, C))
    codes = torch.full((D, 160), 0xFF, dtype=torch.uint8, device=DEV)
    scales = torch.full((D, 64), 0xFF, dtype=torch.uint8, device=DEV)
    codes[:, :64], scales[:, :16] = q.codes, q.scales
    w = T.MxTensor.wrap(codes, scales, D, C)
    x, y, z = draw(gen(52), N, C), torch.empty(N, D, device=DEV), torch.empty(N, D, device=DEV)
    T.MxLayer(N, C, D, weight=w, train=False).fwd(x, y)
    T.MxLayer(N, C, D, weight=q, train=False).fwd(x, z)
    assert torch.equal(y, z)
    big = draw(gen(53), 200, C)
    y, z = torch.empty(200, D, device=DEV), torch.empty(200, D, device=DEV)
    T.MxLayer(200, C, D, weight=w, train=False).fwd(big, y)
    T.MxLayer(200, C, D, weight=q, train=False).fwd(big, z)
    assert torch.equal(y, z)


def test_wrap_refuses_what_would_be_read_as_numbers():
    def fresh_pair():
        q = T.MxTensor(8, 40, rot=1, codes_t=False).quantize(draw(gen(5), 8, 40))
        return q.codes.clone(), q.scales.clone()

    T.MxTensor.wrap(*fresh_pair(), 8, 40, rot=1)
    codes, scales = fresh_pair()
    scales[3, 2] = 1
    with pytest.raises(ValueError, match="zero past"):
        T.MxTensor.wrap(codes, scales, 8, 40, rot=1)
    codes, scales = fresh_pair()
    codes[3, 20] = 1
    with pytest.raises(ValueError, match="zero past"):
        T.MxTensor.wrap(codes, scales, 8, 40, rot=1)
    with pytest.raises(ValueError, match="zero past"):
        T.MxTensor.wrap(codes, scales, 8, 39, rot=1)
    T.MxTensor.wrap(codes, scales, 8, 40, rot=32)       # a rotated block's codes all count
    with pytest.raises(ValueError, match="at least"):
        T.MxTensor.wrap(codes[:, :16], scales, 8, 40, rot=1)
    with pytest.raises(ValueError, match="at least"):
        T.MxTensor.wrap(codes, scales[:, :8], 8, 40, rot=1)


def test_refusals_of_the_helpers():
    x = draw(gen(1), 8, 64)
    q = T.MxTensor(8, 64)
    with pytest.raises(ValueError, match="shape"):
        q.quantize(x.t().contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        q.quantize(draw(gen(1), 64, 8).t())
    with pytest.raises(ValueError, match="dtype"):
        q.quantize(x.double())
    for seed in (torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV),
                 torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="seed"):
            q.quantize(x, seed=seed)
    with pytest.raises(ValueError, match="rot"):
        T.MxTensor(8, 64, rot=16)
    with pytest.raises(ValueError, match="weight is"):
        T.MxLayer(4, 64, 9, weight=q)
    q.quantize(x)
    other = T.MxTensor(16, 64, rot=1).quantize(draw(gen(2), 16, 64))
    with pytest.raises(B.HQError, match="MISMATCH"):
        T.mx_gemm(q, other, torch.empty(8, 16, device=DEV))
    with pytest.raises(ValueError, match="train=False"):
        T.MxLayer(4, 64, 8, weight=q, train=False).bwd_weight(torch.empty(8, 64, device=DEV))
    with pytest.raises(ValueError, match="ws"):
        T.mx_gemm(q, q, torch.empty(8, 8, device=DEV), ws=torch.empty(16, device=DEV))


def test_empty_matrices():
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        q = T.MxTensor(rows, cols).quantize(torch.empty(rows, cols, device=DEV))
        assert q.dequantize(torch.empty(rows, cols, device=DEV)).numel() == 0
    a, b = T.MxTensor(5, 0), T.MxTensor(7, 0)
    a.quantize(torch.empty(5, 0, device=DEV))
    b.quantize(torch.empty(7, 0, device=DEV))
    c = torch.ones(5, 7, device=DEV)
    T.mx_gemm(a, b, c, accumulate=True)
    assert (c == 1).all()
    T.mx_gemm(a, b, c)
    assert not c.any()
    layer = T.MxLayer(0, 64, 32)
    layer.set_weight(draw(gen(1), 32, 64))
    layer.fwd(torch.empty(0, 64, device=DEV), torch.empty(0, 32, device=DEV))
    layer.bwd_input(torch.empty(0, 32, device=DEV), torch.empty(0, 64, device=DEV))
    dw = torch.ones(32, 64, device=DEV)
    layer.bwd_weight(dw)
    assert not dw.any()

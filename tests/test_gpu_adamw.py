"""The AdamW step against the formula in 64 bits: 32-bit states, 8-bit states and their rounding,
many tensors, captured steps, refusals, and a whole training step of a block-scaled layer."""
import math

import pytest
import torch

import train_testlib as R
from hadamard_rotated_precision_amd import binding as B
from hadamard_rotated_precision_amd import tensors as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, n, scale=1.0):
    return torch.randn(n, generator=g, device=DEV) * scale


def formula(p, g, m, v, step, grad_scale=1.0, lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1):
    """(p, m, v, and bounds of fp32 errors) from 64-bit inputs. fp32: each constant and operation
    is off by at most U of its result. m: two products of rounded constants and a sum, under 5 U of
    the terms' magnitudes; v: under 7 U; den: sqrt halves v's, three more roundings, 8 U; the update
    adds a quotient, a product and the constant, p its own product, constant and difference."""
    b1, b2 = betas
    g = g * grad_scale
    size = (b1 * m).abs() + ((1 - b1) * g).abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = v.sqrt() / math.sqrt(1 - b2 ** step) + eps
    rate = lr / (1 - b1 ** step)
    new = p * (1 - lr * weight_decay) - rate * m / den
    bound = 4 * U * p.abs() + U * new.abs() + rate / den * (6 * U * size + 13 * U * m.abs())
    return new, m, v, (bound, 6 * U * size, 8 * U * v)


def stored(x64, bound, dtype):
    """Bound of x rounded to dtype."""
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    return bound + R.HALF_STEP[dtype] * (x64.abs() + bound) + tiny


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 127, 128, 129, 2047, 2048, 2049, 100003])
@pytest.mark.parametrize("pdt,gdt,cdt", [
    (torch.float32, torch.float32, None), (torch.float32, torch.bfloat16, torch.bfloat16),
    (torch.bfloat16, torch.bfloat16, None), (torch.float16, torch.float32, torch.float16),
    (torch.float32, torch.float16, torch.float32)])
def test_step_in_32_bits(n, pdt, gdt, cdt):
    g = gen(n)
    p, grad = randn(g, n, 0.02).to(pdt), randn(g, n, 1e-3).to(gdt)
    st = {"m": randn(g, n, 1e-3), "v": randn(g, n, 1e-3).square()}
    copy = None if cdt is None else torch.zeros(n, dtype=cdt, device=DEV)
    want, m, v, (bp, bm, bv) = formula(p.double(), grad.double(), st["m"].double(),
                                       st["v"].double(), 6, 0.5)
    opt = T.AdamW([p], states=[st], steps_done=5, copies=None if copy is None else [copy], **HYPER)
    opt.step([grad], grad_scale=0.5)
    R.assert_within(p, want, stored(want, bp, pdt), "p")
    if copy is not None:
        R.assert_within(copy, want, stored(want, bp, cdt), "copy")
    R.assert_within(st["m"], m, bm + 2.0 ** -149, "m")
    R.assert_within(st["v"], v, bv + 2.0 ** -149, "v")


def neighbours(x):
    """The grid values around x >= 0 (fp64): low <= x <= high."""
    _, e = torch.frexp(x)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    low = torch.floor(x / ulp) * ulp
    return low, low + ulp


def eight_bit_values(st, n):
    at = torch.arange(n, device=DEV) // 128
    m = st["m"].view(R.E4M3).double() * st["m_scales"].double()[at]
    return m, (st["v"].view(R.E4M3).double() * st["v_scales"].double()[at]).square()


@pytest.mark.parametrize("n", [1, 5, 8, 127, 128, 130, 2048, 2050, 70001])
def test_step_in_8_bits(n):
    """p as with 32-bit states of the same values; new states on a neighbour of the exact value."""
    g = gen(n)
    p, grad = randn(g, n, 0.02), (randn(g, n, 1e-3) * torch.exp(randn(g, n, 2.0)))
    opt = T.AdamW([p], state_bits=8, seed=5, **HYPER)
    st = opt.states[0]
    for step in range(1, 4):
        m0, v0 = eight_bit_values(st, n)
        want, m, v, (bp, bm, bv) = formula(p.double(), grad.double(), m0, v0, step)
        opt.step([grad])
        R.assert_within(p, want, stored(want, bp, torch.float32), "p")
        for name, exact, bound in (("m", m, bm), ("v", v.sqrt(), bv / v.sqrt().clamp_min(1e-30))):
            at = torch.arange(n, device=DEV) // 128
            s = st[name + "_scales"].double()
            a = R.block_max(exact.view(1, -1), 1, 128).view(-1)
            assert ((s - a / 448).abs() <= 16 * U * a / 448 + 2.0 ** -126).all()
            q = st[name].view(R.E4M3).double()
            assert (q * exact >= 0).all()
            x, q = exact.abs() / s[at].clamp_min(1e-300), q.abs()
            off = bound / s[at].clamp_min(1e-300) + 16 * U * x   # fp32 errors of x
            low, high = neighbours((x - off).clamp_min(0))[0], neighbours((x + off).clamp(max=448))[1]
            ok = (q >= low) & (q <= high)
            if name == "v":
                ok |= (q == 2.0 ** -9) & (v > 0) & (x < 2.0 ** -9)
                assert (q[v > 0] > 0).all()
            assert ok.all(), (name, int((~ok).sum()))
        grad = randn(g, n, 1e-3)


def test_8_bit_rounding_is_unbiased():
    """Many elements of one value: the mean of m, and of v, over the elements is the value itself,
    within five standard deviations (a rounded value differs by at most one step)."""
    n = 128 * 2000
    for value in (0.3, 0.011, 3.1e-4):   # steps of normal codes, and of the subnormal ones
        grad = torch.full((n,), value, device=DEV)
        grad[::128] = 1.0      # the block's largest
        p = torch.zeros(n, device=DEV)
        opt = T.AdamW([p], lr=1e-3, betas=(0.0, 0.0), state_bits=8, seed=1)   # m = g, v = g^2
        opt.step([grad])
        m, v = eight_bit_values(opt.states[0], n)
        keep = torch.ones(n, dtype=torch.bool, device=DEV)
        keep[::128] = False
        for got, want in ((m[keep], float(grad[1])), (v[keep], float(grad[1]) ** 2)):
            spread = float(got.std())
            assert spread > 0
            assert abs(float(got.mean()) - want) <= 5 * spread / math.sqrt(got.numel()) + 2.0 ** -16 * want


def test_8_bit_second_moment_decays():
    """Without gradients v falls by beta2 each step on average; nearest rounding would keep it."""
    n = 128 * 64
    p, g = torch.zeros(n, device=DEV), randn(gen(1), n, 1e-3)
    opt = T.AdamW([p], lr=0.0, betas=(0.9, 0.999), state_bits=8, weight_decay=0.0)
    opt.step([g])
    v0 = eight_bit_values(opt.states[0], n)[1].sum()
    zero = torch.zeros_like(g)
    for _ in range(300):
        opt.step([zero])
    ratio = float(eight_bit_values(opt.states[0], n)[1].sum() / v0)
    # the sum of 8192 unbiased terms: a few percent of spread around 0.999^300 = 0.741
    assert abs(ratio - 0.999 ** 300) < 0.05


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_are_each_alone(bits):
    """More tensors than one launch's table, lengths from zero to many workgroups: each tensor gets
    what a call with the others emptied gives it (its place in the list sets the random numbers)."""
    lengths = [0, 1, 5, 128, 129, 5000, 3, 0, 2048] * 11 + [100000]
    g = gen(3)
    params = [randn(g, n, 0.02) for n in lengths]
    grads = [randn(g, n, 1e-3) for n in lengths]
    decay = [0.1 * (i % 3) for i in range(len(lengths))]
    start = [p.clone() for p in params]
    kw = dict(HYPER, weight_decay=decay, state_bits=bits, seed=9)
    opt = T.AdamW(params, **kw)
    opt.step(grads)
    opt.step(grads)
    for i in (1, 5, 39, 40, 41, 80, 98, 99):
        n = lengths[i]
        alone = [start[j].clone() if j == i else start[j].new_zeros(0) for j in range(len(lengths))]
        one = T.AdamW(alone, **kw)
        for _ in range(2):
            one.step([grads[j] if j == i else grads[j].new_zeros(0) for j in range(len(lengths))])
        assert torch.equal(alone[i], params[i])
        for k in one.states[i]:
            assert torch.equal(one.states[i][k], opt.states[i][k]), (i, k)


def test_memory_around_a_tensor_is_left():
    for bits in (32, 8):
        n = 1003
        buf = torch.full((n + 64,), 3.0, device=DEV)
        st_buf = torch.full((n + 64,), 7, dtype=torch.uint8, device=DEV)
        p = buf[32:32 + n]
        opt = T.AdamW([p], state_bits=bits, **HYPER)
        if bits == 8:
            st = {"m": st_buf[32:32 + n].zero_(), "v": torch.zeros(n, dtype=torch.uint8, device=DEV),
                  "m_scales": torch.zeros(8, device=DEV), "v_scales": torch.zeros(8, device=DEV)}
            opt = T.AdamW([p], state_bits=8, states=[st], **HYPER)
        opt.step([randn(gen(1), n)])
        assert (buf[:32] == 3).all() and (buf[32 + n:] == 3).all()
        assert (st_buf[:32] == 7).all() and (st_buf[32 + n:] == 7).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_its_device_scalars(bits):
    """A captured step replayed with advance() between gives the eager steps' bits."""
    n = 5000
    g = gen(7)
    p, grad = randn(g, n, 0.02), randn(g, n, 1e-3)
    q = p.clone()
    eager = T.AdamW([p], state_bits=bits, seed=4, **HYPER)
    taken = T.AdamW([q], state_bits=bits, seed=4, **HYPER)
    taken.device_scalars
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken.step([grad], captured=True)
    for k in range(4):
        if k == 2:
            eager.set_lr(1e-2)
            taken.set_lr(1e-2)
        eager.step([grad], grad_scale=0.25 * (k + 1))
        taken.advance(grad_scale=0.25 * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, q)
        for name in eager.states[0]:
            assert torch.equal(eager.states[0][name], taken.states[0][name])
    assert taken.step_count == eager.step_count == 4


def test_not_finite_gradients_show():
    n = 1000
    for bits in (32, 8):
        p, g = torch.zeros(n, device=DEV), randn(gen(1), n)
        g[300] = float("nan")
        opt = T.AdamW([p], state_bits=bits, **HYPER)
        opt.step([g])
        assert p[300].isnan() and int(p.isnan().sum()) == 1
        if bits == 8:
            assert opt.states[0]["m_scales"][2].isnan() and opt.states[0]["v_scales"][2].isnan()
            assert int(opt.states[0]["m_scales"].isnan().sum()) == 1


def test_python_refusals():
    p = torch.zeros(10, device=DEV)
    for kw in (dict(state_bits=16), dict(copies=[]), dict(copies=[torch.zeros(9, device=DEV)]),
               dict(states=[{"m": p, "v": torch.zeros(9, device=DEV)}]), dict(weight_decay=[0.1, 0.2]),
               dict(states=[])):
        with pytest.raises(ValueError):
            T.AdamW([p], **kw)
    with pytest.raises(ValueError):
        T.AdamW([])
    with pytest.raises(ValueError):
        T.AdamW([p, p.half()])
    opt = T.AdamW([p])
    for bad in ([], [torch.zeros(9, device=DEV)], [torch.zeros(10)], [torch.zeros(10, device=DEV).double()],
                [torch.zeros(20, device=DEV)[::2]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(B.HQError):
        T.AdamW([p], betas=(1.0, 0.9)).step([p])


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_of_a_block_scaled_layer(bits):
    """The operators as they are used together: quantize W, forward, both gradients, update, and
    again from the updated bf16 weights; every stage against the 64-bit one on its own inputs."""
    N, C, D = 200, 384, 300
    g = gen(11)
    master = randn(g, D * C, 0.02)
    bias = randn(g, D, 0.1)
    w = master.to(torch.bfloat16).view(D, C)
    x, dy = randn(g, N * C).view(N, C).bfloat16(), randn(g, N * D, 1e-3).view(N, D).bfloat16()
    layer = T.BlockLayer(N, C, D)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    dw = torch.zeros(D, C, device=DEV)
    opt = T.AdamW([master, bias], state_bits=bits, copies=[w.view(-1), torch.zeros(D, dtype=torch.bfloat16, device=DEV)],
                  **HYPER)
    for step in range(1, 4):
        layer.set_weight(w)
        layer.fwd(x, y)
        layer.bwd_input(dy, dx)
        layer.bwd_weight(dw)
        vw = R.values(w, 128, 128)
        for got, a, b in ((y, R.values(x, 1, 128), vw), (dx, R.values(dy, 1, 128), vw.t().contiguous()),
                          (dw, R.values(dy, 128, 1).t().contiguous(), R.values(x, 128, 1).t().contiguous())):
            want = torch.mm(a, b.t().contiguous())
            R.assert_within(got, want, R.product_bound(a, b, want, got.dtype), "step %d" % step)
        grads = [dw.view(-1), dy.float().sum(0)]
        before = [p.double() for p in (master, bias)]
        states = [eight_bit_values(s, p.numel()) if bits == 8 else (s["m"].double(), s["v"].double())
                  for s, p in zip(opt.states, (master, bias))]
        opt.step(grads)
        for p, p0, gr, (m, v) in zip((master, bias), before, grads, states):
            want, _, _, (bp, _, _) = formula(p0, gr.double(), m, v, step)
            R.assert_within(p, want, stored(want, bp, torch.float32), "p at step %d" % step)
        assert torch.equal(w.view(-1), master.bfloat16())


def random_of(seed, step, tensor, element):
    """The documented random numbers of an element: (for m, for v), each 16 bits."""
    def mix(h):
        h ^= h >> 16
        h = h * 2654435761 & 0xFFFFFFFF
        h ^= h >> 15
        h = h * 2891336453 & 0xFFFFFFFF
        return h ^ h >> 16

    k = mix((seed + 2654435761 * step) & 0xFFFFFFFF) + 0x9E3779B9 * (tensor + 1)
    u = mix((element & 0xFFFFFFFF) ^ (k + 0x632BE5AB * (element >> 32) & 0xFFFFFFFF))
    return u & 0xFFFF, u >> 16


def check_rounding(st, lo, m, v, seed, step, tensor):
    """States of elements lo, lo + 1, ... (64-bit m, v) are rounded as the random numbers say, where
    they are not next to the border."""
    at = torch.arange(lo, lo + m.numel(), device=DEV) // 128
    tested = 0
    for name, exact, which in (("m", m.abs(), 0), ("v", v.sqrt(), 1)):
        x = (exact / st[name + "_scales"].double()[at]).clamp(max=448)
        low, high = neighbours(x)
        share = ((x - low) / (high - low) if name == "m"
                 else (x * x - low * low) / (high * high - low * low))
        got = st[name][lo:lo + m.numel()].view(R.E4M3).double().abs()
        for i in range(m.numel()):
            u = random_of(seed, step, tensor, lo + i)[which] / 65536
            edge = 1 - float(share[i])
            up = u >= edge if name == "m" else u < float(share[i])
            if min(abs(u - edge), abs(u - float(share[i])), float(share[i]), edge) < 1e-3 or float(x[i]) < 2.0 ** -6:
                continue
            assert float(got[i]) == float(high[i] if up else low[i]), (name, lo + i)
            tested += 1
    assert tested > m.numel()


def test_rounding_follows_the_documented_random_numbers():
    g = gen(5)
    params = [randn(g, n, 0.02) for n in (50, 400)]
    grads = [randn(g, n, 1e-3) for n in (50, 400)]
    opt = T.AdamW(params, state_bits=8, seed=77, steps_done=8, **HYPER)
    opt.step(grads)
    for k in (0, 1):
        gr = grads[k].double()
        check_rounding(opt.states[k], 0, 0.1 * gr, 0.05 * gr * gr, 77, 9, k)


def test_more_elements_than_32_bits():
    """2^32 + 1500 elements: the parameters and the states past every 32-bit border."""
    n = 2 ** 32 + 1500
    p = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    grad = torch.empty(n, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(1))
    opt = T.AdamW([p], state_bits=8, seed=3, lr=1e-1, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    opt.step([grad])
    st = opt.states[0]
    for lo in (2 ** 31 - 512, 2 ** 32 - 512, n - 1024):
        hi = min(lo + 1024, n)
        gr = grad[lo:hi].double()
        want, m, v, (bp, _, _) = formula(torch.full_like(gr, 0.5), gr, torch.zeros_like(gr),
                                         torch.zeros_like(gr), 1, lr=1e-1)
        R.assert_within(p[lo:hi], want, stored(want, bp, torch.bfloat16), "p")
        check_rounding(st, lo, m, v, 3, 1, 0)


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_at_any_element(bits):
    """Parameters, gradients, copies and states that are pieces of flat buffers, at odd places."""
    n, sizes = 5000, [1, 130, 2049, 77, 2743]
    g = gen(2)
    p, grad = randn(g, n, 0.02), randn(g, n, 1e-3).bfloat16()
    flat = {k: (torch.zeros(n, device=DEV) if bits == 32 else torch.zeros(n, dtype=torch.uint8, device=DEV)) for k in "mv"}
    flat["p"], flat["copy"], flat["g"] = p.clone(), torch.zeros(n, dtype=torch.float16, device=DEV), grad
    cut = lambda t: list(t.split(sizes))  # noqa: E731
    scales = {k: [torch.zeros(-(-s // 128), device=DEV) for s in sizes] for k in ("m_scales", "v_scales")}
    states = [dict(m=m, v=v, m_scales=a, v_scales=b) for m, v, a, b in
              zip(cut(flat["m"]), cut(flat["v"]), scales["m_scales"], scales["v_scales"])]
    one = T.AdamW(cut(flat["p"]), state_bits=bits, copies=cut(flat["copy"]), states=states, seed=1, **HYPER)
    other_p = [t.clone() for t in cut(p)]
    other = T.AdamW(other_p, state_bits=bits, copies=[torch.zeros_like(t, dtype=torch.float16) for t in other_p],
                    seed=1, **HYPER)
    for _ in range(2):
        one.step(cut(flat["g"]))
        other.step([t.clone() for t in cut(grad)])
    assert torch.equal(flat["p"], torch.cat(other_p))
    assert torch.equal(flat["copy"], torch.cat(other.copies))
    for k in "mv":
        assert torch.equal(flat[k], torch.cat([s[k] for s in other.states]))


@pytest.mark.parametrize("bits", [32, 8])
def test_capture_before_anything_else(bits):
    """The first call of an optimizer may be the captured one: replays keep its scalars."""
    p, grad = randn(gen(7), 700, 0.02), randn(gen(8), 700, 1e-3)
    q = p.clone()
    eager, taken = T.AdamW([p], state_bits=bits, **HYPER), T.AdamW([q], state_bits=bits, **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken.step([grad], captured=True)
    for _ in range(3):
        eager.step([grad])
        taken.advance()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, q)


def test_overlapping_tensors_are_refused():
    a, b, c = torch.zeros(100, device=DEV), torch.zeros(40, device=DEV), torch.zeros(100, device=DEV)
    whole = {"m": torch.zeros(140, device=DEV), "v": torch.zeros(100, device=DEV)}
    for params, kw in (([a, b, a], {}), ([a, a[90:]], {}), ([a, c], dict(copies=[c, a])),
                       ([a, b], dict(states=[{"m": whole["m"][:100], "v": whole["v"]},
                                             {"m": whole["m"][99:139], "v": torch.zeros(40, device=DEV)}]))):
        with pytest.raises(ValueError, match="overlap"):
            T.AdamW(params, **kw)
    T.AdamW([a[:50], a[50:], a[:0]])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_copy_may_be_its_own_parameter(bits):
    """bf16 parameters whose bf16 copies are themselves: the bits of a step without copies."""
    start = [randn(gen(k), n, 0.02).bfloat16() for k, n in enumerate((1, 300, 4097))]
    grads = [randn(gen(9), p.numel(), 1e-3) for p in start]
    alone, same = [p.clone() for p in start], [p.clone() for p in start]
    a = T.AdamW(alone, state_bits=bits, **HYPER)
    b = T.AdamW(same, state_bits=bits, copies=[p.to(torch.bfloat16) for p in same], **HYPER)
    for _ in range(3):
        a.step(grads)
        b.step(grads)
    for x, y, z in zip(alone, same, start):
        assert torch.equal(x, y) and not torch.equal(x, z)


@pytest.mark.parametrize("bits", [32, 8])
def test_rebound_tensors_give_the_bits_of_an_optimizer_made_anew(bits):
    """After p.data = ..., a state loaded by assignment and a new copy, steps go on from there and
    leave the old memory as it was."""
    n = 1003
    g = gen(21)
    p, grads = randn(g, n, 0.02), [randn(g, n, 1e-3) for _ in range(3)]
    copy = p.bfloat16()
    opt = T.AdamW([p], state_bits=bits, copies=[copy], seed=2, **HYPER)
    opt.step([grads[0]])
    q = T.AdamW([p.clone()], state_bits=bits, copies=[copy.clone()], seed=2, steps_done=1,
                states=[{k: t.clone() for k, t in opt.states[0].items()}], **HYPER)
    old = [p.data, copy.data] + list(opt.states[0].values())
    kept = [t.clone() for t in old]
    p.data, copy.data = p.data.clone(), copy.data.clone()
    for k in list(opt.states[0]):
        opt.states[0][k] = opt.states[0][k].clone()
    for grad in grads[1:]:
        opt.step([grad])
        q.step([grad])
    assert torch.equal(p, q.params[0]) and torch.equal(copy, q.copies[0])
    for k in opt.states[0]:
        assert torch.equal(opt.states[0][k], q.states[0][k]), k
    for was, now in zip(kept, old):
        assert torch.equal(was, now)


def busy(stream=None):
    """Tens of milliseconds of work on a stream, and the event behind it."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(stream):
        for _ in range(60):
            torch.mm(a, a)
        done.record()
    return done


def test_advance_does_not_wait_for_the_stream():
    opt = T.AdamW([torch.zeros(100, device=DEV)], **HYPER)
    opt.advance()       # the first call allocates
    done = busy()
    opt.advance()
    assert not done.query(), "the host waited for the work before it"
    torch.cuda.synchronize()
    assert done.query()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_run_ahead_on_a_stream_of_their_own(bits):
    """Many steps handed over at once, with the scalars of each in the order of the stream."""
    p, grad = randn(gen(7), 3000, 0.02), randn(gen(8), 3000, 1e-3)
    q = p.clone()
    eager, taken = T.AdamW([p], state_bits=bits, **HYPER), T.AdamW([q], state_bits=bits, **HYPER)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken.step([grad], captured=True)
    torch.cuda.synchronize()
    for k in range(50):
        eager.step([grad], grad_scale=1.0 + k)
    torch.cuda.synchronize()
    done = busy(s)
    for k in range(50):
        taken.advance(grad_scale=1.0 + k, stream=s)
        with torch.cuda.stream(s):
            graph.replay()
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(p, q)
    for name in eager.states[0]:
        assert torch.equal(eager.states[0][name], taken.states[0][name])


@pytest.mark.parametrize("value", [2e-5, 6e-6])
def test_8_bit_rounding_is_unbiased_among_subnormal_codes(value):
    """Beside a block's largest of 1 these are 4.6 and 1.4 steps of the subnormal codes (2^-9), so
    the codes 4 and 5, or 1 and 2: each appears, and the means of m and of v are the values, within
    five standard deviations, the 2^-16 grain of the probabilities and the fp32 errors of x (2^-20)."""
    n = 128 * 2000
    grad = torch.full((n,), value, device=DEV)
    grad[::128] = 1.0
    opt = T.AdamW([torch.zeros(n, device=DEV)], lr=1e-3, betas=(0.0, 0.0), state_bits=8, seed=1)
    opt.step([grad])
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[::128] = False
    x = value * 448
    low = math.floor(x * 512)
    assert x < 2.0 ** -6
    for name, got, power in zip("mv", eight_bit_values(opt.states[0], n), (1, 2)):
        assert sorted(opt.states[0][name][keep].unique().tolist()) == [low, low + 1]
        got, want = got[keep], float(grad[1]) ** power
        gap = (((low + 1) ** power - low ** power) / 512.0 ** power) / 448.0 ** power
        spread = float(got.std())
        off = abs(float(got.mean()) - want)
        print("[mean] %s %g: off by %.3g, five deviations %.3g" % (name, value, off, 5 * spread / math.sqrt(got.numel())), flush=True)
        assert off <= 5 * spread / math.sqrt(got.numel()) + 2.0 ** -16 * gap + 2.0 ** -20 * want


def test_subnormal_codes_follow_the_documented_random_numbers():
    """Every element whose fraction is away from the border (2^-10: the grain of 2^-16 and the fp32
    errors of x are below it) rounds as its random number says, v from the first code up."""
    n, seed, step = 128 * 300, 77, 9
    g = gen(31)
    grad = randn(g, n) * torch.exp2(-6 - 10 * torch.rand(n, generator=g, device=DEV)) / 448
    grad[::128] = 1.0
    opt = T.AdamW([torch.zeros(1, device=DEV), torch.zeros(n, device=DEV)], lr=1e-3, betas=(0.0, 0.0),
                  state_bits=8, seed=seed, steps_done=step - 1)
    opt.step([torch.zeros(1, device=DEV), grad])
    st, tensor = opt.states[1], 1

    def mix(h):
        for shift, factor in ((16, 2654435761), (15, 2891336453), (16, 1)):
            h = ((h ^ (h >> shift)) * factor) & 0xFFFFFFFF
        return h

    key = int(mix(torch.tensor((seed + 2654435761 * step) & 0xFFFFFFFF))) + 0x9E3779B9 * (tensor + 1)
    i = torch.arange(n, device=DEV)
    u = mix(i ^ (key & 0xFFFFFFFF))
    assert (int(u[5]) & 0xFFFF, int(u[5]) >> 16) == random_of(seed, step, tensor, 5)
    for name, r in (("m", u & 0xFFFF), ("v", u >> 16)):
        r = r.double() / 65536
        x = grad.double().abs() / st[name + "_scales"].double()[i // 128]
        low, high = neighbours(x)
        if name == "m":
            border = 1 - (x - low) / (high - low)
            up = r >= border
        else:
            border = (x * x - low * low) / (high * high - low * low)
            up = r < border
        tested = (x < 2.0 ** -6) & ((r - border).abs() > 2.0 ** -10)
        if name == "v":
            tested &= x >= 2.0 ** -9
        got = st[name].view(R.E4M3).double().abs()
        assert torch.equal(got[tested], torch.where(up, high, low)[tested]), name
        codes = st[name][tested] & 0x7F
        # of ten octaves of x the three from the first code up to 2^-6 count for v
        assert int(tested.sum()) > n // 8 and set(range(1, 8)) <= set(codes.unique().tolist())


def test_every_significand_of_the_denominator():
    """The update's 1 / den is the correctly rounded one for each of the 2^23 significands. With
    beta1 = 1/2, beta2 = 1/4, no gradient and states m = 2, v = 4 y^2: m becomes 1 and v y^2, whose
    rounded root is y again; far on, both bias corrections are 1, eps is lost beside y, and p = 0
    becomes -1 / y (lr 1, no decay)."""
    y = torch.arange(0x3F800000, 0x40000000, dtype=torch.int32, device=DEV).view(torch.float32)
    n = y.numel()
    root = (y * y).double().sqrt().float()
    assert torch.equal(root, y)
    p = torch.zeros(n, device=DEV)
    st = {"m": torch.full((n,), 2.0, device=DEV), "v": 4.0 * (y * y)}
    opt = T.AdamW([p], lr=1.0, betas=(0.5, 0.25), eps=1.2e-38, weight_decay=0.0, states=[st], steps_done=999)
    opt.step([torch.zeros(n, device=DEV)])
    assert (st["m"] == 1).all() and torch.equal(st["v"], y * y)
    assert torch.equal(p, -y.double().reciprocal().float())

"""The torch helpers of include/hq_train.h on the CPU: what they hand to the library (the launch is
replaced by a stand-in that looks at the arguments), and what they refuse before it."""
import pytest
import torch

from hadamard_rotated_precision_amd import binding as B
from hadamard_rotated_precision_amd import tensors as T


@pytest.fixture
def launches(monkeypatch):
    """Argument lists of the calls that would have reached the library."""
    calls = []
    monkeypatch.setattr(T, "_launch", lambda fn, t, stream, *args: calls.append(args) or B.HQ_OK)
    return calls


FIELDS = {32: ("m", "v"), 8: ("m", "v", "m_scales", "v_scales")}


def adamw(bits, copies=False):
    params = [torch.zeros(n) for n in (300, 7)]
    kw = dict(copies=[p.bfloat16() for p in params]) if copies else {}
    return T.AdamW(params, state_bits=bits, **kw), [torch.zeros(n) for n in (300, 7)]


def table_is_current(call, opt):
    table = call[0]
    for i, (p, s) in enumerate(zip(opt.params, opt.states)):
        assert table[i].p == p.data_ptr()
        for k in FIELDS[opt.state_bits]:
            assert getattr(table[i], k) == s[k].data_ptr(), k
        assert table[i].copy == (opt.copies[i].data_ptr() if opt.copies else None)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_follows_tensors_that_are_rebound(bits, launches):
    """p.data = ..., a state's entry, an entry of the lists: the step works on the new memory."""
    opt, grads = adamw(bits, copies=True)
    opt.step(grads)
    opt.params[0].data = torch.ones(300)
    opt.step(grads)
    for k in FIELDS[bits]:
        opt.states[1][k] = opt.states[1][k].clone()
    opt.step(grads)
    opt.copies[1].data = opt.copies[1].data.clone()
    opt.step(grads)
    opt.params[1] = torch.ones(7)
    opt.step(grads)
    opt.copies[1] = torch.ones(7, dtype=torch.bfloat16)
    opt.step(grads)
    assert len(launches) == 6 and opt.step_count == 6
    for call in launches[-1:]:
        table_is_current(call, opt)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("what", range(5))
def test_adamw_follows_each_rebinding_at_once(bits, what, launches):
    opt, grads = adamw(bits, copies=True)
    opt.step(grads)
    if what == 0:
        opt.params[0].data = torch.ones(300)
    elif what == 1:
        opt.states[0]["m"] = opt.states[0]["m"].clone()
    elif what == 2:
        opt.states[1]["v"].data = opt.states[1]["v"].clone()
    elif what == 3:
        opt.copies[0].data = opt.copies[0].clone()
    else:
        opt.states[0] = {k: t.clone() for k, t in opt.states[0].items()}
    opt.step(grads)
    table_is_current(launches[-1], opt)


def test_adamw_checks_what_is_rebound(launches):
    """The checks of the constructor hold for a tensor that takes another's place."""
    def broken(change, match):
        opt, grads = adamw(8, copies=True)
        change(opt)
        with pytest.raises(ValueError, match=match):
            opt.step(grads)
        with pytest.raises(ValueError, match=match):    # and again: it stays refused
            opt.step(grads)
        assert not launches and opt.step_count == 0

    def set_data(t, new):
        t.data = new

    broken(lambda o: set_data(o.params[0], torch.zeros(300).half()), "dtype")
    broken(lambda o: set_data(o.params[0], torch.zeros(299)), "300|299")
    broken(lambda o: set_data(o.params[0], torch.zeros(300, 2)[:, 0]), "contiguous")
    broken(lambda o: set_data(o.copies[1], torch.zeros(7)), "dtype")
    broken(lambda o: set_data(o.params[1], o.params[0].data[10:17]), "overlap")
    broken(lambda o: o.states[0].update(m=o.states[0]["v"]), "overlap")
    broken(lambda o: o.states[0].update(m=torch.zeros(300)), "state m")
    broken(lambda o: o.states[1].update(v_scales=torch.zeros(2)), "state v_scales")
    broken(lambda o: o.states[1].pop("m_scales"), "m_scales")
    broken(lambda o: o.params.append(torch.zeros(3)), "param")


@pytest.mark.parametrize("copy", [False, True])
def test_adamw_refuses_a_transposed_tensor_at_the_same_address(copy, launches):
    """p.data = p.data.t() keeps the address and changes the order of the elements."""
    p, c = torch.zeros(6, 5), torch.zeros(6, 5).half()
    opt = T.AdamW([p], copies=[c])
    opt.step([torch.zeros(6, 5)])
    if copy:
        c.data = c.data.t()
    else:
        p.data = p.data.t()
    with pytest.raises(ValueError, match="contiguous"):
        opt.step([torch.zeros(5, 6)])
    assert len(launches) == 1


class AnyStream:
    cuda_stream = 0


def test_host_memory_never_reaches_a_call(monkeypatch):
    """Tensors in host memory agree with one another about their device; the library would launch
    on their addresses all the same."""
    reached = []
    for name in ("hq_block_quantize", "hq_block_gemm", "hq_block_linear_fwd",
                 "hq_block_linear_bwd_input", "hq_block_linear_bwd_weight", "hq_adamw_step"):
        monkeypatch.setattr(B, name, lambda *a: reached.append(a) or B.HQ_OK)
    x, y, w = torch.zeros(4, 64), torch.zeros(4, 32), torch.zeros(32, 64)
    a, b = T.BlockTensor(4, 64, device="cpu"), T.BlockTensor(32, 64, shape=B.HQ_BLOCK_TILES, device="cpu")
    layer = T.BlockLayer(4, 64, 32, weight=b)
    opt = T.AdamW([torch.zeros(5)])
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda s: a.quantize(x, stream=s), lambda s: layer.set_weight(w, s),
                 lambda s: layer.fwd(x, y, s), lambda s: layer.bwd_input(y, x, s),
                 lambda s: layer.bwd_weight(w, stream=s),
                 lambda s: T.block_gemm(a, b, y, ws=ws, stream=s),
                 lambda s: opt.step([torch.zeros(5)], stream=s)):
        for stream in (AnyStream(), None):
            with pytest.raises(ValueError, match="GPU"):
                call(stream)
    assert not reached and opt.step_count == 0


def test_captured_step_takes_no_gradient_scale(launches):
    """A captured step reads its scale from device_scalars: one given to it would be lost."""
    opt, grads = adamw(32)
    with pytest.raises(ValueError, match="advance"):
        opt.step(grads, grad_scale=0.5, captured=True)
    assert not launches
    opt.step(grads, captured=True)
    assert len(launches) == 1 and opt.step_count == 0


@pytest.mark.parametrize("name", ["codes", "codes_t", "scales", "scales_t"])
def test_block_tensor_keeps_its_buffers(name):
    """The library's struct holds the buffers' addresses: another tensor in their place would leave
    it with those of freed memory."""
    for q in (T.BlockTensor(40, 300, device="cpu"),
              T.BlockTensor.wrap(torch.zeros(40, 304, dtype=torch.uint8), torch.zeros(1, 3), 40, 300)):
        old = getattr(q, name)
        with pytest.raises(AttributeError):
            setattr(q, name, torch.zeros(3))
        assert getattr(q, name) is old


def wrapped(shape, codes, codes_t, scales, scales_t, rows=200, cols=300):
    return T.BlockTensor.wrap(codes, scales, rows, cols, shape=shape, scale=B.HQ_BSCALE_POW2,
                              codes_t=codes_t, scales_t=scales_t)


def pow2_parts(shape):
    """Codes in both layouts and scales of 200 x 300 elements, with room behind what is read."""
    codes = torch.full((200, 320), 0x38, dtype=torch.uint8)
    codes_t = torch.full((300, 224), 0x38, dtype=torch.uint8)
    if shape == B.HQ_BLOCK_TILES:
        return codes, codes_t, torch.full((2, 5), 0.25), None
    return codes, codes_t, torch.full((3, 210), 0.25), torch.full((2, 310), 0.25)


@pytest.mark.parametrize("shape", [B.HQ_BLOCK_ROWS, B.HQ_BLOCK_TILES])
@pytest.mark.parametrize("bad", [3.0, -0.5, float("inf"), 2.0 ** -127, 2.0 ** -130, 2.0 ** -149, 0.0])
def test_wrap_refuses_scales_that_the_exponent_does_not_tell(shape, bad):
    """A power-of-two product reads a scale's exponent alone: a subnormal scale, or zero over codes
    that are not zero, would count as 2^-127."""
    for which in (2, 3) if shape == B.HQ_BLOCK_ROWS else (2,):
        parts = pow2_parts(shape)
        wrapped(shape, *parts)
        parts[which][1, 2] = bad
        with pytest.raises(ValueError, match="POW2"):
            wrapped(shape, *parts)


@pytest.mark.parametrize("shape", [B.HQ_BLOCK_ROWS, B.HQ_BLOCK_TILES])
def test_wrap_takes_every_scale_that_it_promises(shape):
    """From 2^-126 up, NaN, and zero over zero codes of either sign; what is behind is not read."""
    codes, codes_t, scales, scales_t = pow2_parts(shape)
    scales[0, 0], scales[0, 1], scales[1, 1] = 2.0 ** -126, 2.0 ** 127, float("nan")
    if shape == B.HQ_BLOCK_TILES:
        scales[1, 2] = 0.0
        codes[128:, 256:300], codes_t[256:, 128:200] = 0x80, 0
        scales[:, 3:] = 3.0
    else:
        scales[2, 7] = scales_t[1, 9] = 0.0
        codes[7, 256:300], codes_t[9, 128:200] = 0x80, 0
        scales[:, 200:] = scales_t[:, 300:] = 3.0
    wrapped(shape, codes, codes_t, scales, scales_t)
    codes_t[-1 if shape == B.HQ_BLOCK_TILES else 9, 199] = 1    # one code under a zero scale
    with pytest.raises(ValueError, match="POW2"):
        wrapped(shape, codes, codes_t, scales, scales_t)


@pytest.mark.parametrize("M,N,K,split", [(32, 1024, 16384, True), (17, 1024, 16384, True), (24, 4112, 4096, True),
                                         (17, 4096, 8192, False), (32, 4096, 6144, False), (32, 1024, 4096, False),
                                         (16, 1024, 16384, False)])
def test_few_tokens_split_a_long_contraction(M, N, K, split):
    """17 to 32 tokens against long or wide weights run on tiles with K split, whose sums need a
    workspace; the few-token form, which needs none, reads every token in every workgroup."""
    assert (B.hq_block_gemm_workspace_bytes(M, N, K) > 0) == split


def test_adamw_takes_its_lists_as_tuples(launches):
    opt, grads = adamw(8, copies=True)
    opt.params, opt.copies, opt.states = (tuple(t.clone() for t in opt.params), tuple(t.clone() for t in opt.copies),
                                          tuple({k: t.clone() for k, t in s.items()} for s in opt.states))
    opt.step(grads)
    table_is_current(launches[-1], opt)

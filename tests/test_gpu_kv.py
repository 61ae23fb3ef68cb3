"""The 4-bit cache and its attention against 64-bit references: written codes, values read back,
attention over every head size, length, window and page size, graphs, streams and wrong arguments."""
import math

import pytest
import torch

import mx_testlib as R
from hadamard_rotated_precision_amd import binding as B
from hadamard_rotated_precision_amd import tensors as T
from mx_testlib import gen, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def heads_of(g, n, heads, D, dtype, outlier=True):
    x = torch.randn(n, heads, D, generator=g, device=DEV)
    if outlier:
        x[..., 5] *= 20
    return x.to(dtype)


# ------------------------------------------------------------------------------ append and read
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (3, 2, 16), (77, 5, 64), (1000, 8, 256)])
def test_append_and_read(D, rotate, tokens, heads, page):
    for i, dtype in enumerate(DTYPES):
        g = gen(tokens + D + i)
        cache = R.new_cache(-(-tokens // page) + 2, page, heads, D, rotate)
        k, v = heads_of(g, tokens, heads, D, dtype), heads_of(g, tokens, heads, D, dtype)
        slots = torch.randperm(cache.pages * page, generator=g, device=DEV)[:tokens].contiguous()
        for codes in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
            codes.fill_(0xC3)
        cache.append(k, v, slots)
        rot, (at, row) = D if rotate else 1, R.rows_of(cache, slots)
        for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
            want, s = R.quantize(x, rot)
            assert torch.equal(R.unpack(codes[at, :, row]), want)
            assert torch.equal(scales[at, :, row], s)
            other = torch.ones(cache.pages, page, dtype=torch.bool, device=DEV)
            other[at, row] = False
            assert (codes.transpose(1, 2)[other] == 0xC3).all() and (scales.transpose(1, 2)[other] == 0xC3).all()
        outs = [torch.full((tokens, heads, D), 9.0, dtype=dtype, device=DEV) for _ in range(2)]
        cache.read(slots, *outs)
        for x, out in zip((k, v), outs):
            # sums of D codes times their scales in fp32: log2 D roundings of sums below sum |v|
            held = R.values(*R.quantize(x, rot))
            want = R.hadamard(held, rot) / rot
            total = held.abs().sum(-1, keepdim=True) / rot
            slack = (math.log2(D) + 1) * 2.0 ** -24 * total if rotate else 0.0
            tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
            R.assert_within(out, want, slack + R.HALF_STEP[dtype] * (want.abs() + slack) + tiny, "read back")
        one = torch.empty_like(outs[0])
        cache.read(slots, v=one)
        assert torch.equal(one, outs[1])
        cache.read(slots, k=one)
        assert torch.equal(one, outs[0])


def test_heads_of_a_projection_and_slots_outside():
    """Strided keys and values; tokens of slots outside the cache are left out, and read as zeros."""
    g = gen(3)
    heads, D, n = 4, 128, 37
    qkv = heads_of(g, n, 3 * heads, D, torch.bfloat16)
    cache = R.new_cache(4, 16, heads, D)
    slots = torch.randperm(64, generator=g, device=DEV)[:n]
    slots[::5] = torch.tensor([-1, 64, -2 ** 62, 2 ** 62, 1000, -7, 2 ** 31, 65], device=DEV)
    cache.append(qkv[:, heads:2 * heads], qkv[:, 2 * heads:], slots)
    whole = R.new_cache(4, 16, heads, D)
    inside = (slots >= 0) & (slots < 64)
    kept = slots[inside].contiguous()
    whole.append(qkv[inside][:, heads:2 * heads].contiguous(), qkv[inside][:, 2 * heads:].contiguous(), kept)
    for a, b in ((cache.k_codes, whole.k_codes), (cache.v_codes, whole.v_codes),
                 (cache.k_scales, whole.k_scales), (cache.v_scales, whole.v_scales)):
        assert torch.equal(a, b)
    k = torch.full((n, heads, D), 9.0, device=DEV)
    cache.read(slots, k=k)
    assert not k[~inside].any() and k[inside].abs().amax((1, 2)).min() > 0
    # heads of a head-major tensor, and one head for all
    heads_first = heads_of(g, n, heads, D, torch.float32).transpose(0, 1).contiguous().transpose(0, 1)
    shared = heads_of(g, n, 1, D, torch.float32).expand(n, heads, D)
    slots = torch.arange(n, device=DEV)
    cache.append(heads_first, shared, slots)
    whole.append(heads_first.contiguous(), shared.contiguous(), slots)
    assert torch.equal(cache.k_codes, whole.k_codes) and torch.equal(cache.v_codes, whole.v_codes)


def test_not_finite_blocks_of_the_cache():
    g = gen(4)
    k = heads_of(g, 6, 2, 128, torch.float32)
    k[2, 1, 70] = math.nan
    k[4, 0, 0] = math.inf
    for rotate in (True, False):
        cache = R.new_cache(1, 16, 2, 128, rotate)
        slots = torch.arange(6, device=DEV)
        cache.append(k, k, slots)
        out = torch.empty_like(k)
        cache.read(slots, k=out)
        bad = out.isnan()
        assert bad.any(-1).sum() == 2
        assert bad[2, 1, 64:96].all() and bad[4, 0, :32].all()
        assert bad.sum() == (2 * 128 if rotate else 2 * 32)


def test_a_cache_past_32_bit_offsets():
    """Pages whose codes lie beyond 2^32 bytes, written, read and attended."""
    heads, D, page = 16, 128, 256
    pages = (1 << 32) // (heads * page * D // 2) + 40
    cache = R.new_cache(pages, page, heads, D)
    g, n = gen(5), 300
    k, v = heads_of(g, n, heads, D, torch.bfloat16), heads_of(g, n, heads, D, torch.bfloat16)
    table = ints([[pages - 3, pages - 1]])
    at = torch.arange(n, device=DEV)
    cache.append(k, v, table[0].long()[at // page] * page + at % page)
    small = R.new_cache(2, page, heads, D)
    small.append(k, v, at)
    q = heads_of(g, 2, heads, D, torch.bfloat16, False)
    outs = []
    for c, t in ((cache, table), (small, ints([[0, 1]]))):
        out = torch.empty_like(q)
        c.attend(q, out, ints([0, 2]), ints([n]), t, max_q=2, max_len=n)
        back = torch.empty(n, heads, D, device=DEV)
        c.read(t[0].long()[at // page] * page + at % page, k=back)
        outs.append((out, back))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and a.abs().max() > 0


# ------------------------------------------------------------------------------------ attention
def run(cache, q, starts, lens, table, max_q=None, max_len=None, scale=None, window=0, dtype=None, **kw):
    out = torch.full(q.shape, 7.0, dtype=dtype or q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    news = [b - a for a, b in zip(starts, starts[1:])]
    cache.attend(q, out, ints(starts), ints(lens), table, max_q=max(news) if max_q is None else max_q,
                 max_len=max(lens) if max_len is None else max_len, scale=scale, window=window, lse=lse, **kw)
    return out, lse


def check(cache, q, starts, lens, table, scale=None, window=0, dtype=None, **kw):
    out, lse = run(cache, q, starts, lens, table, scale=scale, window=window, dtype=dtype, **kw)
    want, want_l, err, err_l = R.attention(cache, q, starts, lens, table,
                                           cache.head_dim ** -0.5 if scale is None else scale, window, out.dtype)
    mine = ~want_l.isnan()
    R.assert_within(out[mine], want[mine], err[mine], "attention")
    empty = mine & (want_l == -math.inf)
    assert (lse[empty] == -math.inf).all() and not out[empty].any()
    mine &= ~empty
    R.assert_within(lse[mine], want_l[mine], err_l[mine], "lse")
    assert (out[want_l.isnan()] == 7.0).all() and (lse[want_l.isnan()] == 7.0).all()
    return out, lse


# new tokens and lengths of a batch: single tokens, drafts, pieces of prompts, whole prompts, sequences
# without new tokens, of length 0 and 1, pages and chunks that end anywhere
BATCHES = [([1], [1]), ([1], [777]), ([1, 1, 1], [16, 17, 64]), ([1, 3, 0, 2], [65, 200, 50, 2]),
           ([5, 1, 7], [5, 300, 129]), ([40], [100]), ([33, 20, 1], [33, 500, 1024]), ([1, 1], [1500, 63])]


@pytest.mark.parametrize("news,lens", BATCHES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group,page,dtype,rotate",
                         [(2, 4, 16, torch.bfloat16, True), (3, 1, 64, torch.float16, False),
                          (1, 5, 32, torch.float32, True), (2, 16, 128, torch.bfloat16, False),
                          (1, 24, 256, torch.float16, True)])
def test_attention(news, lens, D, heads, group, page, dtype, rotate):
    g = gen(sum(lens) + D + group)
    cache = R.new_cache(sum(-(-n // page) for n in lens) + 3, page, heads, D, rotate)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, news, lens, extra_pages=2)
    q = heads_of(g, starts[-1], heads * group, D, dtype, False) * 0.3
    check(cache, q, starts, lens, table)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs,heads,group,new,longest",
                         [(3, 2, 4, 1, 9000), (300, 1, 3, 1, 13000), (40, 2, 4, 5, 6200), (40, 2, 12, 5, 13000),
                          (2, 2, 8, 5, 2500), (70, 4, 4, 1, 1500)])
def test_long_lengths_among_short_ones(seqs, heads, group, new, longest, D, dtype):
    """One long sequence, the others short, of length 0 or without new tokens: the pieces of the waves
    begin and end anywhere, and hold many sequences or a part of one."""
    g = gen(seqs + D)
    lens = [(37 * s) % 150 for s in range(seqs)]
    lens[seqs // 2], lens[-1] = longest, 0
    news = [min(new, n) if s % 7 else 0 for s, n in enumerate(lens)]
    news[seqs // 2] = new
    page = 64
    cache = R.new_cache(sum(-(-n // page) for n in lens) + 3, page, heads, D)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, news, lens)
    q = heads_of(g, starts[-1], heads * group, D, dtype, False)
    check(cache, q, starts, lens, table)
    check(cache, q, starts, lens, table, window=longest - 1000)
    if seqs < 100:      # two long ones, and every bound at once
        lens[0], news[0] = longest - 77, 0
        lens[1] = longest // 2
        cache = R.new_cache(sum(-(-n // page) for n in lens) + 3, page, heads, D, False)
        R.fill(cache, g, 2.0)
        starts, table = R.batch(g, cache, news, lens)
        q = heads_of(g, starts[-1], heads * group, D, dtype, False)
        out, _ = check(cache, q, starts, lens, table)
        for wrong in ([5] + starts[1:], [-4] + starts[1:], starts[:-1] + [2 ** 31 - 1], starts[::-1]):
            run(cache, q, wrong, [n * 3 - 70 for n in lens], table, max_q=new, max_len=longest)
        torch.cuda.synchronize()


@pytest.mark.parametrize("window", [1, 2, 33, 64, 200, 5000])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(window, D):
    g = gen(window)
    news, lens = [1, 9, 30], [700, 300, 30]
    cache = R.new_cache(40, 32, 2, D)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, news, lens)
    check(cache, heads_of(g, 40, 6, D, torch.bfloat16, False), starts, lens, table, window=window)


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_types_of_queries_and_outputs(dtype, out):
    g = gen(8)
    cache = R.new_cache(20, 16, 2, 128)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [2, 1], [90, 200])
    check(cache, heads_of(g, 3, 4, 128, dtype, False), starts, [90, 200], table, dtype=out)


def test_written_tokens_are_attended():
    """Real keys and values, a sharp softmax, and one that sees a single token."""
    g = gen(9)
    for rotate in (True, False):
        cache = R.new_cache(12, 64, 2, 128, rotate)
        n = 600
        starts, table = R.batch(g, cache, [3], [n])
        at = torch.arange(n, device=DEV)
        slots = table[0].long()[at // 64] * 64 + at % 64
        cache.append(heads_of(g, n, 2, 128, torch.bfloat16), heads_of(g, n, 2, 128, torch.bfloat16), slots)
        q = heads_of(g, 3, 8, 128, torch.bfloat16, False)
        for scale in (None, 3.0, -0.5, 0.0):
            check(cache, q, starts, [n], table, scale=scale)
        check(cache, q, starts, [n], table, window=1)


def test_rows_that_see_nothing_and_rows_of_no_sequence():
    """More new tokens than the sequence is long: the first rows stand before it. Length 0. Rows
    before, between (none) and behind the sequences stay as they were."""
    g = gen(10)
    cache = R.new_cache(10, 16, 2, 64)
    R.fill(cache, g)
    q = heads_of(g, 20, 4, 64, torch.bfloat16, False)
    starts, table = [2, 8, 11, 12], ints([[3], [5], [0]])
    out, lse = check(cache, q, starts, [2, 0, 7], table, max_len=64)
    assert (out[:2] == 7).all() and (out[12:] == 7).all()
    assert not out[2:6].any() and not out[8:11].any()
    check(cache, q, starts, [2, 0, 7], table, max_len=5000)     # most parts of the split are empty


def test_pages_that_do_not_exist_are_not_seen():
    g = gen(11)
    cache = R.new_cache(6, 32, 2, 128)
    R.fill(cache, g, 2.0)
    q = heads_of(g, 4, 4, 128, torch.float16, False)
    table = ints([[0, -1, 2, 6, 2 ** 31 - 1, -2 ** 31, 1], [-1, 99, -5, -1, -1, 7, 6]])
    starts = [0, 2, 4]
    check(cache, q, starts, [200, 100], table)
    # the table ends before the sequence does
    check(cache, q, starts, [200, 100], table[:, :3].contiguous())
    wide = table.new_full((2, 9), -1)
    out, lse = run(cache, q, starts, [200, 100], wide)
    assert not out.any() and (lse == -math.inf).all()


def test_bounds_cut_rows_and_tokens():
    """Rows past max_q are left, tokens past max_len are not seen; rows keep their positions. Query
    rows past the tensor's end are not touched."""
    g = gen(12)
    cache = R.new_cache(20, 16, 1, 64)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [6, 5], [90, 200])
    q = heads_of(g, 11, 2, 64, torch.float32, False)
    out, lse = run(cache, q, starts, [90, 200], table)
    cut, cut_l = run(cache, q, starts, [90, 200], table, max_q=2)
    left = torch.ones(11, dtype=torch.bool, device=DEV)
    left[[0, 1, 6, 7]] = False
    assert (cut[left] == 7).all() and torch.allclose(cut[~left], out[~left], rtol=1e-4, atol=1e-4)
    short, _ = run(cache, q, starts, [90, 200], table, max_len=100)
    assert torch.allclose(short[:6], out[:6], rtol=1e-4, atol=1e-4)
    masked = table.clone()
    masked[1, 7:] = -1          # sees the first 112 of 200 tokens
    a, _ = run(cache, q, starts, [90, 200], masked)
    b, _ = run(cache, q, starts, [90, 200], table, max_len=112)
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-4)
    few, _ = run(cache, q[:8], starts, [90, 200], table)
    assert torch.equal(few, out[:8])
    for wrong in ([0, 6, 3], [-4, 6, 11], [5, 5, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 11]):
        run(cache, q, wrong, [90, 200], table, max_q=6)
    run(cache, q, starts, [-5, 2 ** 31 - 1], table, max_len=200)
    torch.cuda.synchronize()


def test_values_that_are_not_numbers():
    """A token with a NaN block makes the rows that see it NaN and no others; what lies behind the
    lengths, in slots that nothing was written to, does not matter."""
    g = gen(13)
    for rotate in (True, False):
        cache = R.new_cache(8, 16, 1, 128, rotate)
        R.fill(cache, g, 2.0)
        starts, table = R.batch(g, cache, [30], [50])
        q = heads_of(g, 30, 2, 128, torch.bfloat16, False)
        clean, _ = run(cache, q, starts, [50], table)
        for scales in (cache.k_scales, cache.v_scales):
            for s in (50, 63):      # behind the length
                scales[table[0, s // 16], 0, s % 16] = 255
        cache.k_codes[table[0, 3], 0, 2:] = cache.v_codes[table[0, 3], 0, 2:] = 0x77
        again, _ = run(cache, q, starts, [50], table)
        assert torch.equal(clean, again)
        cache.k_scales[table[0, 3], 0, 2:] = cache.v_scales[table[0, 3], 0, 2:] = 254     # times 6: past fp32
        again, _ = run(cache, q, starts, [50], table)
        assert torch.equal(clean, again)
        for scales, blocks in ((cache.k_scales, None), (cache.v_scales, slice(32, 64))):
            kept = scales.clone()
            scales[table[0, 40 // 16], 0, 40 % 16, 1] = 255      # token 40: seen from row 20 on
            out, lse = run(cache, q, starts, [50], table)
            assert torch.equal(out[:20], clean[:20])
            bad = out[20:].isnan()
            assert bad.all() if blocks is None or rotate else bad[..., blocks].all() and bad.float().mean() == 0.25
            assert lse[20:].isnan().all() == (blocks is None)
            scales.copy_(kept)
        q[4, 1, 3] = math.nan
        out, _ = run(cache, q, starts, [50], table)
        assert out[4, 1].isnan().all() and out.isnan().sum() == 128


@pytest.mark.parametrize("n,L", [(30, 50), (1, 200), (1, 6000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_that_are_not_finite(D, n, L):
    """An infinity times codes of either sign has no softmax: its row is NaN, the others are as before."""
    g = gen(15)
    for rotate in (True, False):
        cache = R.new_cache(-(-L // 64) + 1, 64, 2, D, rotate)
        R.fill(cache, g, 2.0)
        starts, table = R.batch(g, cache, [n], [L])
        q = heads_of(g, n, 4, D, torch.float32, False)
        clean, _ = run(cache, q, starts, [L], table)
        for bad in (math.inf, -math.inf, math.nan):
            x = q.clone()
            x[n - 1, 2, 7] = bad
            out, lse = run(cache, x, starts, [L], table)
            assert out[n - 1, 2].isnan().all() and lse[n - 1, 2].isnan()
            out[n - 1, 2] = clean[n - 1, 2]
            assert torch.equal(out, clean)


def test_what_a_compute_unit_held_before_does_not_matter():
    """Parts of a chunk whose page does not exist are not loaded: after a call over codes and scales of
    all ones (NaN) and of the largest numbers, the next one's results are its own."""
    for D in (64, 128, 256):
        for byte in (254, 255):
            dirty = R.new_cache(64, 16, 2, D)
            for t in (dirty.k_scales, dirty.v_scales):
                t.fill_(byte)
            for t in (dirty.k_codes, dirty.v_codes):
                t.fill_(0x77)
            every = torch.arange(64, dtype=torch.int32, device=DEV).repeat(40, 1)
            for n in (1, 3, 20):
                q = heads_of(gen(n), 40 * n, 8, D, torch.bfloat16, False)
                run(dirty, q, [n * i for i in range(41)], [1000] * 40, every)
                cache = R.new_cache(20, 16, 2, D)
                R.fill(cache, gen(n), 2.0)
                starts, table = R.batch(gen(n + 1), cache, [n, n, 1], [20, 37, 5])
                table[1, 1] = -1
                check(cache, heads_of(gen(n + 2), starts[-1], 8, D, torch.bfloat16, False), starts, [20, 37, 5], table)


def test_strided_queries():
    g = gen(14)
    cache = R.new_cache(10, 16, 2, 128)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [4], [77])
    wide = heads_of(g, 4, 14, 128, torch.bfloat16, False)
    a, _ = run(cache, wide[:, 3:9], starts, [77], table)
    b, _ = run(cache, wide[:, 3:9].contiguous(), starts, [77], table)
    assert torch.equal(a, b)
    turned = wide[:, 3:9].transpose(0, 1).contiguous().transpose(0, 1)
    c, _ = run(cache, turned, starts, [77], table)
    assert torch.equal(b, c)


def test_the_same_bits_each_time_and_from_a_given_workspace():
    g = gen(15)
    cache = R.new_cache(200, 64, 2, 128)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [1, 2], [6000, 3000])
    q = heads_of(g, 3, 8, 128, torch.bfloat16, False)
    ws = cache.attention_workspace(2, 8, max_q=2, max_len=6000)
    ws.fill_(0xFF)
    first = run(cache, q, starts, [6000, 3000], table)
    for kw in ({}, dict(ws=ws), dict(ws=ws)):
        assert all(torch.equal(a, b) for a, b in zip(first, run(cache, q, starts, [6000, 3000], table, **kw)))
    with pytest.raises(B.HQError, match="WORKSPACE"):
        run(cache, q, starts, [6000, 3000], table, ws=ws[:-1])


def test_a_captured_decode_step_follows_lengths_and_pages():
    """Append and attend in a graph: the arrays on the device say where, at each replay."""
    g = gen(16)
    heads, D, page, seqs, most = 2, 128, 16, 3, 400
    cache, plain = R.new_cache(100, page, heads, D), R.new_cache(100, page, heads, D)
    for c in (cache, plain):
        R.fill(c, gen(17), 2.0)
    order = torch.randperm(100, generator=g, device=DEV).int()[:75].view(3, 25).contiguous()
    q, k, v = (heads_of(g, seqs, h, D, torch.bfloat16, False) for h in (8, heads, heads))
    lens, slots, starts = ints([100, 17, 385]), torch.zeros(seqs, dtype=torch.int64, device=DEV), ints([0, 1, 2, 3])
    out, lse = torch.empty_like(q), torch.empty(seqs, 8, device=DEV)
    ws = cache.attention_workspace(seqs, 8, max_q=1, max_len=most)

    def step(c, o, e, w):
        c.append(k, v, slots)
        c.attend(q, o, starts, lens, order, max_q=1, max_len=most, lse=e, ws=w)

    def place():
        at = lens.long() - 1
        slots.copy_(order.long().gather(1, (at // page)[:, None])[:, 0] * page + at % page)

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, out, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, lse, ws)
    step(plain, torch.empty_like(out), torch.empty_like(lse), None)
    for i in range(6):
        for t in (q, k, v):
            t.copy_(heads_of(g, *t.shape, torch.bfloat16, False))
        lens += 1 + i % 2
        place()
        graph.replay()
        torch.cuda.synchronize()
        o, e = torch.empty_like(out), torch.empty_like(lse)
        step(plain, o, e, None)
        assert torch.equal(out, o) and torch.equal(lse, e)
        assert torch.equal(cache.k_codes, plain.k_codes) and torch.equal(cache.v_scales, plain.v_scales)


def test_two_streams():
    g = gen(18)
    cache = R.new_cache(300, 32, 2, 64)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [1, 1], [5000, 2000])
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [heads_of(g, 2, 8, 64, torch.bfloat16, False) for _ in range(2)]
    want = [run(cache, q, starts, [5000, 2000], table)[0] for q in qs]
    dev = [ints(starts), ints([5000, 2000])]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, o, s in zip(qs, outs, streams):
            cache.attend(q, o, *dev, table, max_q=1, max_len=5000, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_the_whole_step_of_a_layer():
    """As a server runs it: projections of a token in 4 bits, its keys and values appended, attention,
    the output projection; each against the 64-bit reference on what the step before gave."""
    g = gen(19)
    width, heads, group, D, page = 512, 2, 2, 128, 16
    Hq = heads * group
    cache = R.new_cache(30, page, heads, D)
    lens, news = [70, 5, 130], [1, 1, 1]
    starts, table = R.batch(g, cache, news, [n + 1 for n in lens])
    for s, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        cache.append(heads_of(g, n, heads, D, torch.bfloat16), heads_of(g, n, heads, D, torch.bfloat16),
                     table[s].long()[at // page] * page + at % page)
    w_qkv, w_out = (R.draw(g, a, b, torch.bfloat16, 0.05) for a, b in (((Hq + 2 * heads) * D, width), (width, Hq * D)))
    proj, back = T.MxLayer(3, width, (Hq + 2 * heads) * D, train=False), T.MxLayer(3, Hq * D, width, train=False)
    proj.set_weight(w_qkv)
    back.set_weight(w_out)
    x = R.draw(g, 3, width, torch.bfloat16)
    qkv = torch.empty(3, (Hq + 2 * heads) * D, dtype=torch.bfloat16, device=DEV)
    proj.fwd(x, qkv)
    q, k, v = qkv.view(3, -1, D).split([Hq, heads, heads], 1)
    slots = torch.stack([table[s].long()[n // page] * page + n % page for s, n in enumerate(lens)])
    cache.append(k, v, slots)
    out, _ = check(cache, q, starts, [n + 1 for n in lens], table)
    y = torch.empty(3, width, dtype=torch.bfloat16, device=DEV)
    back.fwd(out.view(3, -1), y)
    for got, a, w in ((qkv, x, proj.qw), (y, out.view(3, -1), back.qw)):
        va, vb = R.values(*R.quantize(a, 32)), R.held(w)
        want = torch.mm(va, vb.t().contiguous()) / 32
        R.assert_within(got, want, R.product_bound(va, vb, want, 32, torch.bfloat16), "projection")
    # the layer in 4 bits stays near the one in 64: codes are off by a sixth of their value at most, errors
    # of many of them add like random ones; here only that nothing is scaled or mixed up
    dense = x.double() @ w_qkv.double().t()
    assert float((qkv.double() - dense).norm() / dense.norm()) < 0.25


def test_refusals_of_the_helpers():
    cache = R.new_cache(4, 16, 2, 64)
    k = torch.zeros(3, 2, 64, device=DEV)
    slots = torch.arange(3, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        cache.append(k[:2], k, slots)
    with pytest.raises(ValueError, match="dtypes"):
        cache.append(k, k.half(), slots)
    with pytest.raises(ValueError, match="slots"):
        cache.append(k, k, slots.int())
    with pytest.raises(ValueError, match="contiguous"):
        cache.append(torch.zeros(3, 2, 128, device=DEV)[..., ::2], k, slots)
    with pytest.raises(ValueError, match="needed"):
        cache.read(slots)
    with pytest.raises(ValueError, match="contiguous"):
        cache.read(slots, k=torch.zeros(3, 4, 64, device=DEV)[:, :2])
    q, out = torch.zeros(3, 4, 64, device=DEV), torch.zeros(3, 4, 64, device=DEV)
    args = (ints([0, 3]), ints([10]), ints([[0]]))
    with pytest.raises(ValueError, match="lens"):
        cache.attend(q, out, args[0], args[1].long(), args[2], max_q=3, max_len=10)
    with pytest.raises(ValueError, match="q_starts"):
        cache.attend(q, out, ints([0, 1, 3]), args[1], args[2], max_q=3, max_len=10)
    with pytest.raises(ValueError, match="lse"):
        cache.attend(q, out, *args, max_q=3, max_len=10, lse=torch.zeros(3, 4, dtype=torch.half, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        cache.attend(q, torch.zeros(3, 8, 64, device=DEV)[:, :4], *args, max_q=3, max_len=10)
    with pytest.raises(B.HQError, match="MISMATCH"):
        cache.attend(q[:, :3], out[:, :3].contiguous(), *args, max_q=3, max_len=10)
    with pytest.raises(ValueError, match="head_dim"):
        T.KVCache(4, 16, 2, 96)
    with pytest.raises(ValueError, match="power of two"):
        T.KVCache(4, 24, 2, 64)
    with pytest.raises(ValueError, match="k_scales"):
        T.KVCache.wrap(cache.k_codes, cache.k_scales[..., :1], cache.v_codes, cache.v_scales)


def test_empty_batches():
    cache = R.new_cache(4, 16, 2, 64)
    none = torch.empty(0, 2, 64, device=DEV)
    cache.append(none, none, torch.empty(0, dtype=torch.int64, device=DEV))
    cache.read(torch.empty(0, dtype=torch.int64, device=DEV), k=none)
    q = torch.empty(0, 2, 64, device=DEV)
    cache.attend(q, torch.empty_like(q), ints([0]), ints([]), torch.empty(0, 1, dtype=torch.int32, device=DEV),
                 max_q=0, max_len=0)
    q = torch.ones(2, 2, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    cache.attend(q, out, ints([0, 2]), ints([0]), torch.empty(1, 0, dtype=torch.int32, device=DEV), max_q=2, max_len=0)
    assert not out.any()


@pytest.mark.parametrize("rows,longest", [(1, 200), (7, 200), (1, 9000), (40, 200), (40, 9000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_far_past_the_bound_with_windows(D, rows, longest):
    """Positions near 2^31 see nothing of the tokens that the bound leaves, through a window that ends
    behind them; a window that reaches back to them changes nothing."""
    g = gen(20)
    cache = R.new_cache(-(-longest // 64), 64, 2, D)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [rows], [longest])
    table = table.repeat(3, 1)
    starts = [rows * s for s in range(4)]
    q = heads_of(g, starts[-1], 4, D, torch.bfloat16, False)
    far = [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30]
    for window in (1, 16, 64, 1000):
        out, lse = run(cache, q, starts, far, table, max_len=longest, window=window)
        assert not out.any() and (lse == -math.inf).all()
    whole = run(cache, q, starts, far, table, max_len=longest)
    assert all(torch.equal(a, b) for a, b in zip(whole, run(cache, q, starts, far, table, max_len=longest, window=2 ** 31 - 1)))


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_table_where_nothing_may_be_seen(D, rows):
    """With a bound of 0 on the lengths the table may be missing, whatever its pitch."""
    cache = R.new_cache(4, 16, 2, D)
    q = heads_of(gen(21), rows, 4, D, torch.bfloat16, False)
    out, lse = torch.full_like(q, 7.0), torch.full((rows, 4), 7.0, device=DEV)
    starts, lens = ints([0, rows]), ints([100])
    b = cache._batch(1, 4, rows, 0)
    b.q_starts, b.lens, b.table, b.table_ld = starts.data_ptr(), lens.data_ptr(), None, 100
    B.check(T._launch(B.hq_kv_attention, q, None, q.data_ptr(), T.HQ_DT[q.dtype], rows, *q.stride()[:2], cache.st, b,
                      out.data_ptr(), T.HQ_DT[out.dtype], lse.data_ptr(), None, 0), "hq_kv_attention")
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("byte,codes", [(253, 0x76), (254, 0x76), (253, 0x55)])
@pytest.mark.parametrize("n,before", [(12, 0), (80, 0), (12, 9000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_near_and_past_2_to_the_128(D, n, before, byte, codes):
    """A token whose values lie past fp32 (4 and 6 times its scale) leaves the rows that do not see it as
    they are, and for those that do may make the elements with such values infinite or NaN, but no others.
    Below (3 times 2^126) everything counts in full."""
    g = gen(22)
    first = before + 20
    L, at = first + n, first + 5
    cache = R.new_cache(-(-L // 16), 16, 2, D, False)
    R.fill(cache, g, 2.0)
    starts, table = R.batch(g, cache, [n], [L])
    q = heads_of(g, n, 4, D, torch.float32, False) * 0.3
    clean, _ = run(cache, q, starts, [L], table)
    page, row = table[0, at // 16], at % 16
    cache.v_scales[page, :, row, 1] = byte
    cache.v_codes[page, :, row, 16:32] = codes
    out, lse = run(cache, q, starts, [L], table)
    assert torch.equal(out[:at - first], clean[:at - first])
    want, want_l, err, err_l = R.attention(cache, q, starts, [L], table, D ** -0.5, 0, out.dtype)
    free = torch.zeros_like(out, dtype=torch.bool)
    if codes == 0x76:
        free[at - first:, :, 32:64] = ~out[at - first:, :, 32:64].isfinite()
    R.assert_within(out[~free], want[~free], err[~free], "attention")
    R.assert_within(lse, want_l, err_l, "lse")
    assert (out[at - first:, :, 32:64] != clean[at - first:, :, 32:64]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_come_back_from_the_rotation(D):
    """One element of 1e38 in a vector: its rotated codes stay below 2^128, and so do the sums that rotate them
    back, reading or behind the attention."""
    g = gen(23)
    cache, n = R.new_cache(2, 16, 1, D), 20
    x = heads_of(g, n, 1, D, torch.float32)
    x[3, 0, 7], x[11, 0, D - 1] = 1e38, -1e38
    slots = torch.randperm(32, generator=g, device=DEV)[:n].contiguous()
    cache.append(x, x, slots)
    k, v = torch.empty_like(x), torch.empty_like(x)
    cache.read(slots, k, v)
    held = R.values(*R.quantize(x, D))
    want = R.hadamard(held, D) / D
    slack = (math.log2(D) + 1) * 2.0 ** -24 * held.abs().sum(-1, keepdim=True) / D
    for got in (k, v):
        R.assert_within(got, want, slack + 2.0 ** -24 * (want.abs() + slack) + 2.0 ** -126, "read back")
    # rows that see one token each, in the form where waves share the rows and in the one where each has its own
    for rows in (1, 70):
        at = torch.tensor([3, 11], device=DEV)
        one = R.new_cache(2, 16, 1, D)
        one.append(heads_of(g, 2, 1, D, torch.float32, False), x[at].contiguous(), torch.tensor([0, 16], device=DEV))
        lens, starts = [rows, rows], [0, rows, 2 * rows]
        table = ints([[0] * 5, [1] * 5])
        q = heads_of(g, 2 * rows, 4, D, torch.bfloat16, False)
        out, _ = run(one, q, starts, lens, table, max_len=1, window=rows, dtype=torch.float32)
        # beside the rotation's steps: a weight split into three parts (2^-25), their products added (three steps that
        # may cut: 2^-23 each), two steps of the division: below 2^-20 of every element before the rotation
        for s in (0, 1):
            err = slack[at[s], 0] + 2.0 ** -20 * (want[at[s], 0].abs() + held[at[s], 0].abs().sum() / D)
            R.assert_within(out[s * rows:(s + 1) * rows], want[at[s], 0].expand(rows, 4, D), err.expand(rows, 4, D), "attention")


@pytest.mark.parametrize("scale", [-0.5, 0.0, 2.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_either_sign_where_waves_have_rows_of_their_own(D, dtype, scale):
    g = gen(24)
    for rotate in (True, False):
        cache = R.new_cache(30, 16, 2, D, rotate)
        R.fill(cache, g, 2.0)
        starts, table = R.batch(g, cache, [90, 3], [150, 200])
        check(cache, heads_of(g, 93, 4, D, dtype, False) * 0.2, starts, [150, 200], table, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("news,lens", [([1, 3], [300, 77]), ([1], [6000]), ([90], [200])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_with_outlier_channels(D, news, lens, dtype):
    """Channels of the queries 20 and 1000 times the others, where the cache holds outlier channels too and
    where it holds none: what a query's part of 6 bits leaves is counted by its block's largest element."""
    g = gen(25)
    for rotate in (True, False):
        page = 64
        cache = R.new_cache(sum(-(-n // page) for n in lens) + 1, page, 2, D, rotate)
        starts, table = R.batch(g, cache, news, lens)
        for s, n in enumerate(lens):
            at = torch.arange(n, device=DEV)
            k = heads_of(g, n, 2, D, torch.bfloat16, rotate)
            cache.append(k, heads_of(g, n, 2, D, torch.bfloat16), table[s].long()[at // page] * page + at % page)
        q = heads_of(g, starts[-1], 8, D, torch.float32) * 0.02
        q[..., 40] *= 1000
        check(cache, q.to(dtype), starts, lens, table)

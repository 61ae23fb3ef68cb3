"""C-ABI checks of include/hq_mx.h that need no GPU: exports and every refusal. The pointers are fake
addresses; every call below fails its argument checks, or stops at the device check, before any
launch."""
import ctypes
import os
import random
import re
import subprocess
import sys

import pytest

from hadamard_rotated_precision_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, OFF4, OFF2, ODD = 0x10000, 0x10004, 0x10002, 0x10001


def test_every_declared_symbol_is_exported():
    with open(os.path.join(ROOT, "include", "hq_mx.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(hq_[a-z0-9_]+)\s*\(", text))
    assert declared == set(B.MX_EXPORTS)
    lib = B.load_mx()
    for name in declared:
        assert hasattr(lib, name), name
    assert B.hq_mx_abi_version() == 1


def test_no_symbol_outside_the_header():
    out = subprocess.run(["nm", "-D", "--defined-only", B.MX_LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\bT (hq_[a-z0-9_]+)\b", out))
    assert set(B.MX_EXPORTS) <= exported
    if "HQ_MX_LIB_PATH" not in os.environ:   # the sanitizer build holds both C ABIs
        assert exported == set(B.MX_EXPORTS)


def test_the_header_stands_alone_in_c(tmp_path):
    src = tmp_path / "a.c"
    src.write_text('#include "hq_mx.h"\n'
                   "int main(void) { return sizeof(hq_mx_tensor) == %d && sizeof(hq_kv_cache) == %d && "
                   "sizeof(hq_kv_batch) == %d ? 0 : 1; }\n"
                   % (ctypes.sizeof(B.hq_mx_tensor), ctypes.sizeof(B.hq_kv_cache), ctypes.sizeof(B.hq_kv_batch)))
    exe = str(tmp_path / "a")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    subprocess.run([exe], check=True)


def mt(m, n, rot=32, **kw):
    q = B.hq_mx_tensor()
    nb = lambda x: -(-x // 32)  # noqa: E731
    vals = dict(codes=FAKE, codes_t=FAKE, scales=FAKE, scales_t=FAKE, rows=m, cols=n, ld=16 * nb(n),
                ld_t=16 * nb(m), lds=(nb(n) + 15) // 16 * 16, lds_t=(nb(m) + 15) // 16 * 16, rot=rot)
    vals.update(kw)
    for k, v in vals.items():
        setattr(q, k, v)
    return q


def name(status):
    return B.STATUS_NAMES[status]


LAYOUT = [(dict(codes=OFF4), "HQ_ERR_ALIGN"), (dict(scales=OFF4), "HQ_ERR_ALIGN"),
          (dict(ld=120), "HQ_ERR_ALIGN"), (dict(ld=96), "HQ_ERR_SHAPE"), (dict(lds=8), "HQ_ERR_ALIGN"),
          (dict(lds=0), "HQ_ERR_SHAPE"), (dict(scales=None), "HQ_ERR_NULL"),
          (dict(ld=1 << 23), "HQ_ERR_SHAPE"), (dict(lds=1 << 23), "HQ_ERR_SHAPE")]


@pytest.mark.parametrize("kw,want", [
    (dict(), "HQ_ERR_DEVICE"),     # every check passes; there is no device
    (dict(dt=7), "HQ_ERR_DTYPE"),
    (dict(rot=16), "HQ_ERR_K"),
    (dict(rot=0), "HQ_ERR_K"),
    (dict(rot=1), "HQ_ERR_DEVICE"),
    (dict(rows=-1), "HQ_ERR_SHAPE"),
    (dict(cols=1 << 23), "HQ_ERR_SHAPE"),
    (dict(rows=1 << 20, cols=1 << 20), "HQ_ERR_SHAPE"),
    (dict(src=None), "HQ_ERR_NULL"),
    (dict(src=ODD), "HQ_ERR_ALIGN"),
    (dict(src=OFF2), "HQ_ERR_DEVICE"),       # elements may start anywhere
    (dict(seed=OFF2), "HQ_ERR_ALIGN"),
    (dict(seed=OFF4), "HQ_ERR_DEVICE"),
    (dict(out=None), "HQ_ERR_NULL"),
    (dict(out=dict(codes=None, codes_t=None)), "HQ_ERR_NULL"),
    (dict(out=dict(codes=None, scales=None)), "HQ_ERR_DEVICE"),   # transposed codes alone
    (dict(out=dict(codes_t=OFF4)), "HQ_ERR_ALIGN"),
    (dict(out=dict(ld_t=48)), "HQ_ERR_SHAPE"),
    (dict(out=dict(scales_t=None)), "HQ_ERR_NULL"),
] + [(dict(out=kw), want) for kw, want in LAYOUT])
def test_quantize_refusals(kw, want):
    kw = dict(kw)
    out = kw.pop("out", {})
    q = None if out is None else mt(100, 200, **out)
    r = B.hq_mx_quantize(kw.get("src", FAKE), kw.get("dt", B.HQ_BF16), kw.get("rows", 100), kw.get("cols", 200),
                         kw.get("rot", 32), kw.get("seed"), q, None)
    assert name(r) == want


@pytest.mark.parametrize("q,kw,want", [
    ({}, {}, "HQ_ERR_DEVICE"),
    ({}, dict(side=2), "HQ_ERR_MODE"),
    ({}, dict(dt=3), "HQ_ERR_DTYPE"),
    ({}, dict(dst=None), "HQ_ERR_NULL"),
    ({}, dict(dst=OFF2), "HQ_ERR_ALIGN"),
    (dict(rot=2), {}, "HQ_ERR_K"),
    (dict(rows=-1), {}, "HQ_ERR_SHAPE"),
    (dict(codes=None), {}, "HQ_ERR_NULL"),
    (dict(codes=None), dict(side=1), "HQ_ERR_DEVICE"),
    (dict(codes_t=None), dict(side=1), "HQ_ERR_NULL"),
] + [(kw, {}, want) for kw, want in LAYOUT])
def test_dequantize_refusals(q, kw, want):
    r = B.hq_mx_dequantize(mt(100, 200, **q), kw.get("side", 0), kw.get("dst", FAKE), kw.get("dt", B.HQ_F32), None)
    assert name(r) == want


@pytest.mark.parametrize("a,b,kw,want", [
    ({}, {}, {}, "HQ_ERR_DEVICE"),
    ({}, {}, dict(c=None), "HQ_ERR_NULL"),
    ({}, {}, dict(c=OFF2), "HQ_ERR_ALIGN"),
    ({}, {}, dict(dt=5), "HQ_ERR_DTYPE"),
    ({}, {}, dict(a_side=2), "HQ_ERR_MODE"),
    ({}, {}, dict(b_side=-1), "HQ_ERR_MODE"),
    ({}, dict(rot=1), {}, "HQ_ERR_MISMATCH"),
    ({}, dict(cols=192), {}, "HQ_ERR_MISMATCH"),
    ({}, {}, dict(a_side=B.HQ_SIDE_COLS), "HQ_ERR_MISMATCH"),
    (dict(codes=None), {}, {}, "HQ_ERR_NULL"),
    ({}, dict(lds=0), {}, "HQ_ERR_SHAPE"),
])
def test_gemm_refusals(a, b, kw, want):
    r = B.hq_mx_gemm(mt(64, 256, **a), kw.get("a_side", 0), mt(96, 256, **b), kw.get("b_side", 0), kw.get("c", FAKE),
                     kw.get("dt", B.HQ_F32), 0, FAKE, 1 << 30, None)
    assert name(r) == want


def test_workspaces_are_asked_for():
    N, C, D = 64, 8192, 64
    need = B.hq_mx_workspace_bytes(N, C, D)
    assert need >= N * C // 2 + N * C // 32
    w = mt(D, C)
    for ws, size, want in ((None, need, "HQ_ERR_WORKSPACE"), (FAKE, 100, "HQ_ERR_WORKSPACE"), (OFF4, need, "HQ_ERR_ALIGN"),
                           (FAKE, need, "HQ_ERR_DEVICE")):
        assert name(B.hq_mx_linear_fwd(FAKE, 2, N, C, D, w, None, FAKE, 2, None, ws, size, None)) == want
    assert B.hq_mx_workspace_bytes(-1, 2, 3) == 0 and B.hq_mx_gemm_workspace_bytes(1 << 23, 1, 1) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(), "HQ_ERR_DEVICE"),
    (dict(x=None), "HQ_ERR_NULL"),
    (dict(y=None), "HQ_ERR_NULL"),
    (dict(w=None), "HQ_ERR_NULL"),
    (dict(w=mt(96, 100)), "HQ_ERR_MISMATCH"),
    (dict(w=mt(96, 128, rot=64)), "HQ_ERR_K"),
    (dict(dt=9), "HQ_ERR_DTYPE"),
    (dict(N=-1), "HQ_ERR_SHAPE"),
    (dict(seed=ODD), "HQ_ERR_ALIGN"),
    (dict(save=mt(40, 128, codes=None)), "HQ_ERR_NULL"),
    (dict(save=mt(40, 128, codes_t=None, scales_t=None)), "HQ_ERR_DEVICE"),
    (dict(save=mt(40, 128, lds_t=8)), "HQ_ERR_ALIGN"),
])
def test_layer_refusals(kw, want):
    for fn, w in ((B.hq_mx_linear_fwd, mt(96, 128)), (B.hq_mx_linear_bwd_input, mt(128, 96))):
        C, D = (128, 96) if fn is B.hq_mx_linear_fwd else (96, 128)
        w = kw.get("w", w)
        if w is not None and fn is B.hq_mx_linear_bwd_input and "w" in kw:
            w = mt(w.cols, w.rows, rot=w.rot)
        r = fn(kw.get("x", FAKE), kw.get("dt", 2), kw.get("N", 40), C, D, w, kw.get("seed"), kw.get("y", FAKE), 2,
               kw.get("save"), FAKE, 1 << 30, None)
        assert name(r) == want


@pytest.mark.parametrize("g,x,kw,want", [
    ({}, {}, {}, "HQ_ERR_DEVICE"),
    (dict(rot=1), {}, {}, "HQ_ERR_MISMATCH"),
    (dict(rows=41), {}, {}, "HQ_ERR_MISMATCH"),
    ({}, dict(codes_t=None), {}, "HQ_ERR_NULL"),
    ({}, {}, dict(dw=None), "HQ_ERR_NULL"),
    ({}, {}, dict(dw=OFF2), "HQ_ERR_ALIGN"),
    ({}, {}, dict(dt=-1), "HQ_ERR_DTYPE"),
])
def test_weight_gradient_refusals(g, x, kw, want):
    r = B.hq_mx_linear_bwd_weight(mt(40, 96, **g), mt(40, 128, **x), 40, 128, 96, kw.get("dw", FAKE), kw.get("dt", 0), 0,
                                  FAKE, 1 << 30, None)
    assert name(r) == want


def cache(**kw):
    c = B.hq_kv_cache()
    vals = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, pages=10, page=64, heads=8, head_dim=128, rot=128)
    vals.update(kw)
    for k, v in vals.items():
        setattr(c, k, v)
    return c


CACHES = [(dict(head_dim=96), "HQ_ERR_SHAPE"), (dict(page=24), "HQ_ERR_SHAPE"), (dict(page=8), "HQ_ERR_SHAPE"),
          (dict(page=0), "HQ_ERR_SHAPE"), (dict(page=1 << 21), "HQ_ERR_SHAPE"), (dict(heads=0), "HQ_ERR_SHAPE"),
          (dict(heads=1025), "HQ_ERR_SHAPE"), (dict(pages=-1), "HQ_ERR_SHAPE"), (dict(pages=1 << 30), "HQ_ERR_SHAPE"),
          (dict(rot=32), "HQ_ERR_K"), (dict(rot=1), "HQ_ERR_DEVICE"), (dict(k_codes=None), "HQ_ERR_NULL"),
          (dict(v_scales=None), "HQ_ERR_NULL"), (dict(v_codes=OFF4), "HQ_ERR_ALIGN"), (dict(k_scales=ODD), "HQ_ERR_ALIGN")]


@pytest.mark.parametrize("c,kw,want", [
    ({}, {}, "HQ_ERR_DEVICE"),
    ({}, dict(k=None), "HQ_ERR_NULL"),
    ({}, dict(slots=None), "HQ_ERR_NULL"),
    ({}, dict(slots=OFF4), "HQ_ERR_ALIGN"),
    ({}, dict(k=ODD), "HQ_ERR_ALIGN"),
    ({}, dict(k=OFF2), "HQ_ERR_DEVICE"),
    ({}, dict(dt=3), "HQ_ERR_DTYPE"),
    ({}, dict(n=-1), "HQ_ERR_SHAPE"),
    ({}, dict(n=1 << 28), "HQ_ERR_SHAPE"),
    ({}, dict(stride=-1), "HQ_ERR_SHAPE"),
] + [(kw, {}, want) for kw, want in CACHES])
def test_cache_refusals(c, kw, want):
    n, stride, dt, slots = kw.get("n", 7), kw.get("stride", 128), kw.get("dt", 2), kw.get("slots", FAKE)
    assert name(B.hq_kv_append(kw.get("k", FAKE), FAKE, dt, n, 1024, stride, 1024, 128, slots, cache(**c), None)) == want
    if "stride" not in kw:
        assert name(B.hq_kv_read(cache(**c), slots, n, kw.get("k", FAKE), None, dt, None)) == want


def batch(**kw):
    b = B.hq_kv_batch()
    vals = dict(q_starts=FAKE, lens=FAKE, table=FAKE, table_ld=100, seqs=3, max_q=4, max_len=5000, q_heads=32, window=0,
                scale=0.1)
    vals.update(kw)
    for k, v in vals.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("c,b,kw,want", [
    ({}, {}, {}, "HQ_ERR_DEVICE"),
    ({}, {}, dict(q=None), "HQ_ERR_NULL"),
    ({}, {}, dict(out=None), "HQ_ERR_NULL"),
    ({}, {}, dict(q=ODD), "HQ_ERR_ALIGN"),
    ({}, {}, dict(lse=OFF2), "HQ_ERR_ALIGN"),
    ({}, {}, dict(dt=4), "HQ_ERR_DTYPE"),
    ({}, {}, dict(n=-1), "HQ_ERR_SHAPE"),
    ({}, {}, dict(ws=None), "HQ_ERR_WORKSPACE"),
    ({}, {}, dict(ws=OFF4), "HQ_ERR_ALIGN"),
    ({}, dict(q_starts=None), {}, "HQ_ERR_NULL"),
    ({}, dict(lens=None), {}, "HQ_ERR_NULL"),
    ({}, dict(table=None), {}, "HQ_ERR_NULL"),
    ({}, dict(table=OFF2), {}, "HQ_ERR_ALIGN"),
    ({}, dict(seqs=-1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(max_q=-1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(max_len=-1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(max_len=(1 << 30) + 1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(table_ld=-1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(window=-1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(q_heads=12), {}, "HQ_ERR_MISMATCH"),
    ({}, dict(q_heads=0), {}, "HQ_ERR_MISMATCH"),
    ({}, dict(scale=float("nan")), {}, "HQ_ERR_MODE"),
    ({}, dict(scale=float("inf")), {}, "HQ_ERR_MODE"),
    ({}, dict(seqs=1 << 22), {}, "HQ_ERR_SHAPE"),
    ({}, dict(max_q=2 ** 31 - 1), {}, "HQ_ERR_SHAPE"),
    ({}, dict(seqs=0, q_starts=None, lens=None, table=None), {}, "HQ_ERR_DEVICE"),
    ({}, dict(max_len=0, table=None), {}, "HQ_ERR_DEVICE"),
] + [(kw, {}, {}, want) for kw, want in CACHES])
def test_attention_refusals(c, b, kw, want):
    r = B.hq_kv_attention(kw.get("q", FAKE), kw.get("dt", 2), kw.get("n", 9), 4096, 128, cache(**c), batch(**b),
                          kw.get("out", FAKE), 2, kw.get("lse"), kw.get("ws", FAKE), 1 << 40, None)
    assert name(r) == want


def test_attention_workspace():
    assert B.hq_kv_attention_workspace_bytes(cache(), batch()) > 0
    assert B.hq_kv_attention_workspace_bytes(cache(), batch(max_len=64)) == 0
    assert B.hq_kv_attention_workspace_bytes(cache(page=3), batch()) == 0
    assert B.hq_kv_attention_workspace_bytes(cache(), batch(seqs=0)) == 0
    assert B.hq_kv_attention_workspace_bytes(cache(), None) == 0


def test_no_call_reaches_the_device_where_there_is_one(tmp_path):
    """This file on the CPU as if there were a GPU: those of its tests that only the device check would
    stop are skipped."""
    from test_no_fake_pointers_on_a_gpu import PLUGIN
    (tmp_path / "as_if_there_were_a_gpu.py").write_text(PLUGIN)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), os.environ.get("PYTHONPATH", "")]),
               HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        "-p", "as_if_there_were_a_gpu", "-m", "not gpu", "-k", "not as_if and not where_there_is_one",
                        os.path.join("tests", "test_mx_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    print(r.stdout[-3000:] + r.stderr[-2000:])
    assert r.returncode == 0
    tail = r.stdout.strip().splitlines()[-1]
    assert "passed" in tail and "skipped" in tail


@pytest.mark.skipif("HQ_MX_LIB_PATH" in os.environ, reason="the sanitizer build has no launchers of its own")
def test_a_window_needs_no_more_workspace_than_none():
    rng = random.Random(1)
    for _ in range(3000):
        c = cache(head_dim=rng.choice([64, 128, 256]), heads=rng.choice([1, 2, 8, 16]), rot=1)
        b = dict(seqs=rng.choice([1, 2, 5, 33, 300]), q_heads=c.heads * rng.choice([1, 4, 12]),
                 max_q=rng.choice([1, 3, 9, 70, 1000]), max_len=int(2 ** rng.uniform(0, 18)))
        without = B.hq_kv_attention_workspace_bytes(c, batch(**b))
        window = int(2 ** rng.uniform(0, 18))
        assert B.hq_kv_attention_workspace_bytes(c, batch(window=window, **b)) <= without, (b, window)


@pytest.mark.skipif("HQ_MX_LIB_PATH" in os.environ, reason="the sanitizer build has no launchers of its own")
def test_a_window_needs_no_more_workspace_than_none_up_to_every_limit():
    """The same over all that the checks admit: lengths up to 2^30 and thousands of sequences of many heads."""
    c = cache(head_dim=64, heads=256, rot=1)
    far = dict(seqs=1645, q_heads=256, max_q=2, max_len=219732955)
    assert B.hq_kv_attention_workspace_bytes(c, batch(**far)) == B.hq_kv_attention_workspace_bytes(c, batch(window=10938102, **far))
    rng = random.Random(2)
    for _ in range(6000):
        c = cache(head_dim=rng.choice([64, 128, 256]), heads=int(2 ** rng.uniform(0, 10)), rot=1)
        b = dict(seqs=int(2 ** rng.uniform(0, 14)), q_heads=c.heads * rng.choice([1, 2, 8]), max_q=int(2 ** rng.uniform(0, 7)),
                 max_len=int(2 ** rng.uniform(0, 30)))
        without = B.hq_kv_attention_workspace_bytes(c, batch(**b))
        for window in (1, int(2 ** rng.uniform(0, 30)), b["max_len"], 2 ** 31 - 1):
            assert B.hq_kv_attention_workspace_bytes(c, batch(window=window, **b)) <= without, (b, window)


@pytest.mark.parametrize("heads,D", [(1, 64), (3, 128), (1024, 256)])
def test_a_call_of_the_cache_fits_one_launch(heads, D):
    """A thread takes eight elements of a key or value, 256 of them a workgroup, and a launch has fewer
    than 2^32 threads: the largest number of tokens that fits passes the checks, the next does not."""
    most = 0
    for bit in range(31, -1, -1):
        n = most + (1 << bit)
        if -(-2 * n * heads * (D // 8) // 256) * 256 < 1 << 32:
            most = n
    c = cache(heads=heads, head_dim=D, rot=1)
    for n, want in ((most, "HQ_ERR_DEVICE"), (most + 1, "HQ_ERR_SHAPE")):
        assert name(B.hq_kv_append(FAKE, FAKE, 2, n, 0, 0, 0, 0, FAKE, c, None)) == want
        assert name(B.hq_kv_read(c, FAKE, n, FAKE, None, 2, None)) == want

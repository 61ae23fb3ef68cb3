"""C-ABI checks of include/hq_train.h that need no GPU: exports, every refusal, the host-side
scalars, and the rounding's random numbers. The pointers are fake addresses; every call below
fails its argument checks, or stops at the device check, before any launch."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

from hadamard_rotated_precision_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MIS, ODD = 0x10000, 0x10004, 0x10001


def test_every_declared_symbol_is_exported():
    with open(os.path.join(ROOT, "include", "hq_train.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(hq_[a-z0-9_]+)\s*\(", text))
    assert declared == set(B.TRAIN_EXPORTS)
    lib = B.load_train()
    for name in declared:
        assert hasattr(lib, name), name
    assert B.hq_train_abi_version() == 1


def test_no_symbol_outside_the_header():
    out = subprocess.run(["nm", "-D", "--defined-only", B.TRAIN_LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\bT (hq_[a-z0-9_]+)\b", out))
    assert set(B.TRAIN_EXPORTS) <= exported
    if "HQ_TRAIN_LIB_PATH" not in os.environ:   # the sanitizer build holds both C ABIs
        assert exported == set(B.TRAIN_EXPORTS)


def bt(rows, cols, shape=B.HQ_BLOCK_ROWS, scale=B.HQ_BSCALE_F32, **kw):
    q = B.hq_block_tensor()
    nb = lambda n: -(-n // 128)  # noqa: E731
    rows_kind = shape == B.HQ_BLOCK_ROWS
    vals = dict(codes=FAKE, codes_t=FAKE, scales=FAKE, scales_t=FAKE if rows_kind else None,
                rows=rows, cols=cols, ld=(cols + 15) // 16 * 16, ld_t=(rows + 15) // 16 * 16,
                lds=rows if rows_kind else nb(cols), lds_t=cols, shape=shape, scale=scale)
    vals.update(kw)
    for k, v in vals.items():
        setattr(q, k, v)
    return q


def bt_of(kw, *default):
    """bt(*default) with fields replaced."""
    q = bt(*default)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


TILES = B.HQ_BLOCK_TILES


@pytest.mark.parametrize("kw,want", [
    (dict(), "HQ_ERR_DEVICE"),     # every check passes; there is no device
    (dict(dt=7), "HQ_ERR_DTYPE"),
    (dict(shape=2), "HQ_ERR_MODE"),
    (dict(scale=2), "HQ_ERR_MODE"),
    (dict(rows=-1), "HQ_ERR_SHAPE"),
    (dict(cols=1 << 23), "HQ_ERR_SHAPE"),
    (dict(src=None), "HQ_ERR_NULL"),
    (dict(src=ODD), "HQ_ERR_ALIGN"),
    (dict(src=MIS), "HQ_ERR_DEVICE"),       # elements may start anywhere
    (dict(out=None), "HQ_ERR_NULL"),
    (dict(out=dict(codes=None, codes_t=None)), "HQ_ERR_NULL"),
    (dict(out=dict(scales=None)), "HQ_ERR_NULL"),
    (dict(out=dict(scales_t=None)), "HQ_ERR_NULL"),
    (dict(out=dict(codes=MIS)), "HQ_ERR_ALIGN"),
    (dict(out=dict(codes_t=MIS)), "HQ_ERR_ALIGN"),
    (dict(out=dict(ld=210)), "HQ_ERR_ALIGN"),
    (dict(out=dict(ld=192)), "HQ_ERR_SHAPE"),
    (dict(out=dict(ld_t=96)), "HQ_ERR_SHAPE"),
    (dict(out=dict(lds=99)), "HQ_ERR_SHAPE"),
    (dict(out=dict(lds_t=199)), "HQ_ERR_SHAPE"),
    (dict(out=dict(scales=FAKE + 2)), "HQ_ERR_ALIGN"),
    (dict(out=dict(codes=None, lds=0, scales=None)), "HQ_ERR_DEVICE"),   # transposed codes alone
    (dict(shape=TILES, out=dict(lds=1)), "HQ_ERR_SHAPE"),
    (dict(shape=TILES, out=dict(scales=None)), "HQ_ERR_NULL"),
    (dict(shape=TILES), "HQ_ERR_DEVICE"),
])
def test_quantize_refusals(kw, want):
    kw = dict(kw)
    shape = kw.get("shape", B.HQ_BLOCK_ROWS)
    out = kw.pop("out", {})
    q = None if out is None else bt(100, 200, shape if shape < 2 else 0, **out)
    r = B.hq_block_quantize(kw.get("src", FAKE), kw.get("dt", B.HQ_BF16), kw.get("rows", 100),
                            kw.get("cols", 200), shape, kw.get("scale", 0), q, None)
    assert B.STATUS_NAMES[r] == want


@pytest.mark.parametrize("a,b,kw,want", [
    ({}, {}, {}, "HQ_ERR_DEVICE"),
    ({}, {}, dict(c=None), "HQ_ERR_NULL"),
    ({}, {}, dict(c=FAKE + 2), "HQ_ERR_ALIGN"),
    ({}, {}, dict(dt=5), "HQ_ERR_DTYPE"),
    ({}, {}, dict(a_side=2), "HQ_ERR_MODE"),
    (dict(shape=3), {}, {}, "HQ_ERR_MODE"),
    (dict(scale=-1), {}, {}, "HQ_ERR_MODE"),
    (dict(codes=None), {}, {}, "HQ_ERR_NULL"),
    (dict(scales=None), {}, {}, "HQ_ERR_NULL"),
    (dict(ld=250), {}, {}, "HQ_ERR_ALIGN"),
    (dict(ld=240), {}, {}, "HQ_ERR_SHAPE"),
    (dict(lds=63), {}, {}, "HQ_ERR_SHAPE"),
    (dict(rows=-1), {}, {}, "HQ_ERR_SHAPE"),
    ({}, dict(cols=240), {}, "HQ_ERR_MISMATCH"),
    ({}, {}, dict(a_side=B.HQ_SIDE_COLS), "HQ_ERR_MISMATCH"),   # 64 against 256
    ({}, dict(lds=1), {}, "HQ_ERR_SHAPE"),
])
def test_gemm_refusals(a, b, kw, want):
    r = B.hq_block_gemm(bt_of(a, 64, 256), kw.get("a_side", 0), bt_of(b, 96, 256, TILES), 0,
                        kw.get("c", FAKE), kw.get("dt", B.HQ_F32), 0, FAKE, 1 << 30, None)
    assert B.STATUS_NAMES[r] == want


def fwd(**kw):
    a = dict(x=FAKE, xdt=B.HQ_BF16, N=64, C=256, D=96, w=bt(96, 256, TILES), scale=0, y=FAKE,
             ydt=B.HQ_BF16, save=bt(64, 256), ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return B.STATUS_NAMES[B.hq_block_linear_fwd(a["x"], a["xdt"], a["N"], a["C"], a["D"], a["w"],
                                                a["scale"], a["y"], a["ydt"], a["save"], a["ws"],
                                                a["ws_bytes"], None)]


@pytest.mark.parametrize("kw,want", [
    (dict(), "HQ_ERR_DEVICE"),
    (dict(xdt=3), "HQ_ERR_DTYPE"), (dict(ydt=-1), "HQ_ERR_DTYPE"),
    (dict(N=-1), "HQ_ERR_SHAPE"),
    (dict(w=None), "HQ_ERR_NULL"), (dict(x=None), "HQ_ERR_NULL"), (dict(y=None), "HQ_ERR_NULL"),
    (dict(w=bt(96, 240, TILES)), "HQ_ERR_MISMATCH"),
    (dict(w=bt(96, 256, TILES, codes=None)), "HQ_ERR_NULL"),
    (dict(scale=2), "HQ_ERR_MODE"),
    (dict(x=ODD), "HQ_ERR_ALIGN"), (dict(y=ODD), "HQ_ERR_ALIGN"),
    (dict(save=bt(64, 256, codes=None)), "HQ_ERR_NULL"),
    (dict(save=bt(64, 256, ld=128)), "HQ_ERR_SHAPE"),
    (dict(save=None, ws=None), "HQ_ERR_WORKSPACE"),
    (dict(save=None, ws_bytes=100), "HQ_ERR_WORKSPACE"),
    (dict(save=None, ws=MIS), "HQ_ERR_ALIGN"),
    (dict(save=None), "HQ_ERR_DEVICE"),
])
def test_forward_refusals(kw, want):
    assert fwd(**kw) == want


def test_backward_refusals():
    w = bt(96, 256, TILES)

    def dx(w=w, save=None, **kw):
        return B.STATUS_NAMES[B.hq_block_linear_bwd_input(
            kw.get("dy", FAKE), B.HQ_BF16, 64, 256, 96, w, 0, FAKE, B.HQ_BF16, save, FAKE, 1 << 30,
            None)]

    assert dx() == "HQ_ERR_DEVICE"
    assert dx(w=bt(96, 256, TILES, codes_t=None)) == "HQ_ERR_NULL"
    assert dx(w=bt(96, 256, TILES, ld_t=80)) == "HQ_ERR_SHAPE"
    assert dx(dy=None) == "HQ_ERR_NULL"
    assert dx(save=bt(64, 96, lds=3)) == "HQ_ERR_SHAPE"

    def dw(g=None, x=None, **kw):
        return B.STATUS_NAMES[B.hq_block_linear_bwd_weight(
            g or bt(64, 96), x or bt(64, 256), 64, 256, 96, kw.get("dw", FAKE),
            kw.get("dt", B.HQ_F32), 1, FAKE, 1 << 30, None)]

    assert dw() == "HQ_ERR_DEVICE"
    assert dw(dt=4) == "HQ_ERR_DTYPE"
    assert dw(dw=None) == "HQ_ERR_NULL" and dw(dw=FAKE + 2) == "HQ_ERR_ALIGN"
    assert dw(g=bt(32, 96)) == "HQ_ERR_MISMATCH" and dw(x=bt(64, 240)) == "HQ_ERR_MISMATCH"
    assert dw(g=bt(64, 96, codes_t=None)) == "HQ_ERR_NULL"
    assert dw(x=bt(64, 256, scales_t=None)) == "HQ_ERR_NULL"


def test_workspace_sizes():
    assert B.hq_block_workspace_bytes(-1, 4, 4) == 0
    assert B.hq_block_workspace_bytes(1 << 23, 4, 4) == 0
    # the forward's codes and scales of X fit
    assert B.hq_block_workspace_bytes(100, 200, 16) >= 100 * 208 + 2 * 100 * 4
    assert B.hq_block_gemm_workspace_bytes(-1, 4, 4) == 0


def adamw_cfg(**kw):
    c = B.hq_adamw_config()
    vals = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, param_dtype=B.HQ_F32,
                grad_dtype=B.HQ_BF16, copy_dtype=B.HQ_BF16, state_bits=8, seed=3)
    vals.update(kw)
    for k, v in vals.items():
        setattr(c, k, v)
    return c


def adamw_step(cfg=None, scalars=True, count=1, device=None, **kw):
    t = (B.hq_adamw_tensor * 1)()
    vals = dict(p=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scales=FAKE, v_scales=FAKE, copy=None, n=1000,
                weight_decay=0.1)
    vals.update(kw)
    for k, v in vals.items():
        setattr(t[0], k, v)
    s = B.hq_adamw_scalars() if scalars else None
    return B.STATUS_NAMES[B.hq_adamw_step(t if count else None, count, cfg or adamw_cfg(), s,
                                          device, None)]


@pytest.mark.parametrize("kw,want", [
    (dict(), "HQ_ERR_DEVICE"),
    (dict(scalars=False), "HQ_ERR_NULL"),
    (dict(scalars=False, device=FAKE), "HQ_ERR_DEVICE"),
    (dict(device=FAKE + 1), "HQ_ERR_ALIGN"),
    (dict(count=-1), "HQ_ERR_SHAPE"),
    (dict(p=None), "HQ_ERR_NULL"), (dict(grad=None), "HQ_ERR_NULL"),
    (dict(m=None), "HQ_ERR_NULL"), (dict(v_scales=None), "HQ_ERR_NULL"),
    (dict(p=FAKE + 2), "HQ_ERR_ALIGN"), (dict(copy=ODD), "HQ_ERR_ALIGN"),
    (dict(m=ODD, v=ODD), "HQ_ERR_DEVICE"),      # 8-bit codes
    (dict(cfg=adamw_cfg(state_bits=32), m=FAKE + 2), "HQ_ERR_ALIGN"),
    (dict(m_scales=FAKE + 2), "HQ_ERR_ALIGN"),
    (dict(n=-1), "HQ_ERR_SHAPE"), (dict(n=2 ** 34 + 1), "HQ_ERR_SHAPE"), (dict(n=2 ** 34), "HQ_ERR_DEVICE"),
    (dict(weight_decay=-0.1), "HQ_ERR_MODE"), (dict(weight_decay=float("nan")), "HQ_ERR_MODE"),
    (dict(n=0, p=None, grad=None), "HQ_ERR_DEVICE"),    # an empty tensor needs no buffers
    (dict(cfg=adamw_cfg(state_bits=4)), "HQ_ERR_BITS"),
    (dict(cfg=adamw_cfg(beta1=1.0)), "HQ_ERR_MODE"),
    (dict(cfg=adamw_cfg(beta2=float("nan"))), "HQ_ERR_MODE"),
    (dict(cfg=adamw_cfg(eps=0.0)), "HQ_ERR_MODE"), (dict(cfg=adamw_cfg(lr=-1.0)), "HQ_ERR_MODE"),
    (dict(cfg=adamw_cfg(grad_dtype=8)), "HQ_ERR_DTYPE"),
])
def test_adamw_refusals(kw, want):
    assert adamw_step(**kw) == want


def test_adamw_scalars():
    s = B.hq_adamw_scalars()
    assert B.STATUS_NAMES[B.hq_adamw_scalars_at(adamw_cfg(), 0, 1.0, s)] == "HQ_ERR_SHAPE"
    assert B.STATUS_NAMES[B.hq_adamw_scalars_at(adamw_cfg(), 1, 1.0, None)] == "HQ_ERR_NULL"
    for t in (1, 2, 100, 10 ** 6):
        assert B.hq_adamw_scalars_at(adamw_cfg(), t, 0.5, s) == B.HQ_OK
        assert s.step_size == pytest.approx(1e-3 / (1 - 0.9 ** t), rel=2.0 ** -23)
        assert s.inv_sqrt_bias2 == pytest.approx(1 / math.sqrt(1 - 0.95 ** t), rel=2.0 ** -23)
        assert s.grad_scale == 0.5 and s.lr == np.float32(1e-3)


def mix(h):
    h = h ^ (h >> np.uint64(16))
    h = (h * np.uint64(2654435761)) & np.uint64(0xFFFFFFFF)
    h = h ^ (h >> np.uint64(15))
    h = (h * np.uint64(2891336453)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def test_rounding_random_numbers_are_uniform_and_unrelated():
    """The documented hash: each half of u is uniform, the halves, neighbouring elements and
    consecutive steps are uncorrelated (five standard deviations of n independent draws)."""
    s = B.hq_adamw_scalars()
    B.hq_adamw_scalars_at(adamw_cfg(seed=11), 7, 1.0, s)
    assert s.key == int(mix(np.uint64((11 + 2654435761 * 7) & 0xFFFFFFFF)))
    n = 1 << 20
    i = np.arange(n, dtype=np.uint64)
    draws = []
    for step in (7, 8):
        B.hq_adamw_scalars_at(adamw_cfg(seed=11), step, 1.0, s)
        u = mix(i ^ np.uint64((s.key + 0x9E3779B9) & 0xFFFFFFFF))
        draws += [(u & np.uint64(0xFFFF)).astype(float) / 65536, (u >> np.uint64(16)).astype(float) / 65536]
    for d in draws:
        counts = np.bincount((d * 256).astype(int), minlength=256)
        chi2 = float(((counts - n / 256) ** 2 / (n / 256)).sum())
        assert abs(chi2 - 255) < 5 * math.sqrt(2 * 255), chi2
        c = d - d.mean()
        for lag in (1, 2, 8, 128):
            assert abs((c[lag:] * c[:-lag]).mean() / c.var()) < 5 / math.sqrt(n)
    for a in range(4):
        for b in range(a):
            assert abs(np.corrcoef(draws[a], draws[b])[0, 1]) < 5 / math.sqrt(n)


def test_struct_sizes_match_the_header():
    """The ctypes mirrors are laid out as C lays the structs out (natural alignment)."""
    assert ctypes.sizeof(B.hq_block_tensor) == 4 * 8 + 6 * 8 + 2 * 4
    assert ctypes.sizeof(B.hq_adamw_tensor) == 7 * 8 + 8 + 4 + 4
    assert ctypes.sizeof(B.hq_adamw_config) == 4 * 8 + 6 * 4
    assert ctypes.sizeof(B.hq_adamw_scalars) == 20

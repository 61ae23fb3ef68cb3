"""Device-memory plumbing around the C ABI: torch allocates the buffers (codes, scales,
outputs, workspace) and names the stream; the binding passes raw pointers to libhq.
No arithmetic of the method happens here."""
import itertools
import operator

import numpy as np
import torch

from . import binding as B

TORCH_DT = {B.HQ_F32: torch.float32, B.HQ_F16: torch.float16, B.HQ_BF16: torch.bfloat16}
HQ_DT = {torch.float32: B.HQ_F32, torch.float16: B.HQ_F16, torch.bfloat16: B.HQ_BF16}


def pitch16(n):
    return (n + 15) // 16 * 16


def ptr(t):
    return None if t is None else t.data_ptr()


def stream_ptr(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def device_tensor_from_bits(bits, dtype, device="cuda"):
    """Upload a host array of raw bits (uint16 for fp16/bf16, float32 for fp32)."""
    if dtype == B.HQ_F32:
        return torch.from_numpy(np.ascontiguousarray(bits, dtype=np.float32)).to(device)
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.view(TORCH_DT[dtype]).to(device)


def bits_of(t):
    """Raw host bits of a device tensor (uint16 for 16-bit dtypes, float32 for fp32)."""
    h = t.detach().cpu()
    if h.dtype == torch.float32:
        return h.numpy()
    return h.view(torch.int16).numpy().view(np.uint16)


class QTensor:
    """Caller-owned storage of one quantized tensor: codes (rows x pitch), codes_t
    (cols x pitch), one device float scale, and the hq_qtensor struct pointing at them."""

    def __init__(self, rows, cols, codes=True, codes_t=True, device="cuda"):
        self.rows, self.cols = rows, cols
        self.codes = (torch.empty((rows, pitch16(cols)), dtype=torch.int8, device=device)
                      if codes else None)
        self.codes_t = (torch.empty((cols, pitch16(rows)), dtype=torch.int8, device=device)
                        if codes_t else None)
        self.scale = torch.zeros(1, dtype=torch.float32, device=device)
        self.st = B.hq_qtensor()
        self.st.codes = ptr(self.codes)
        self.st.codes_t = ptr(self.codes_t)
        self.st.scale = ptr(self.scale)
        self.st.ld = pitch16(cols)
        self.st.ld_t = pitch16(rows)

    def codes_view(self):
        return None if self.codes is None else self.codes[:, :self.cols]

    def codes_t_view(self):
        return None if self.codes_t is None else self.codes_t[:, :self.rows]


def config(k, bits, scale_mode, variant, fmt=B.HQ_FMT_INT):
    c = B.hq_config()
    c.k, c.bits, c.scale_mode, c.variant, c.format = k, bits, scale_mode, variant, fmt
    return c


class Layer:
    """Buffers for one linear layer (N tokens, C in, D out) and the three HQ-MM calls."""

    def __init__(self, N, C, D, k, bits, scale_mode, variant, device="cuda", fmt=B.HQ_FMT_INT):
        self.N, self.C, self.D = N, C, D
        self.cfg = config(k, bits, scale_mode, variant, fmt)
        self.variant = variant
        self.ws_bytes = B.hq_workspace_bytes(self.cfg, N, C, D)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)
        halo2 = variant == B.HQ_VARIANT_HALO2
        self.qx = QTensor(N, C, codes=True, codes_t=not halo2, device=device)
        self.qxt = QTensor(N, C, codes=False, codes_t=True, device=device) if halo2 else None
        self.qw = QTensor(D, C, codes=True, codes_t=True, device=device)
        self.qg = QTensor(N, D, codes=True, codes_t=True, device=device)

    def fwd(self, x, w, y, steps=None, stream=None):
        steps = steps or {}
        B.check(B.hq_linear_fwd(
            ptr(x), ptr(w), HQ_DT[x.dtype], self.N, self.C, self.D, self.cfg,
            ptr(steps.get("x")), ptr(steps.get("w")), ptr(steps.get("xt", steps.get("x"))),
            ptr(y), HQ_DT[y.dtype], self.qx.st, None if self.qxt is None else self.qxt.st,
            self.qw.st, ptr(self.ws), self.ws_bytes, stream_ptr(stream)), "hq_linear_fwd")

    def bwd_input(self, dy, dx, steps=None, stream=None):
        steps = steps or {}
        B.check(B.hq_linear_bwd_input(
            ptr(dy), HQ_DT[dy.dtype], self.N, self.C, self.D, self.cfg, ptr(steps.get("g")),
            self.qw.st, ptr(dx), HQ_DT[dx.dtype], self.qg.st, ptr(self.ws), self.ws_bytes,
            stream_ptr(stream)), "hq_linear_bwd_input")

    def bwd_weight(self, dw, stream=None):
        qx = self.qxt if self.qxt is not None else self.qx
        B.check(B.hq_linear_bwd_weight(
            self.qg.st, qx.st, self.N, self.C, self.D, self.cfg, ptr(dw), HQ_DT[dw.dtype],
            ptr(self.ws), self.ws_bytes, stream_ptr(stream)), "hq_linear_bwd_weight")


class BatchedLayer:
    """Buffers for a batched product (batch x (N x C) by batch x (D x C), e.g. attention
    heads) and the three batched calls; codes describe the stacked matrices."""

    def __init__(self, batch, N, C, D, k, bits, scale_mode, variant, device="cuda",
                 fmt=B.HQ_FMT_INT):
        self.batch, self.N, self.C, self.D = batch, N, C, D
        self.cfg = config(k, bits, scale_mode, variant, fmt)
        self.variant = variant
        self.ws_bytes = B.hq_bmm_workspace_bytes(self.cfg)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)
        halo2 = variant == B.HQ_VARIANT_HALO2
        NB, DB = batch * N, batch * D
        self.qx = QTensor(NB, C, codes=True, codes_t=not halo2, device=device)
        self.qxt = QTensor(NB, C, codes=False, codes_t=True, device=device) if halo2 else None
        self.qw = QTensor(DB, C, codes=True, codes_t=True, device=device)
        self.qg = QTensor(NB, D, codes=True, codes_t=True, device=device)

    def fwd(self, x, w, y, steps=None, stream=None):
        steps = steps or {}
        B.check(B.hq_bmm_fwd(
            ptr(x), ptr(w), HQ_DT[x.dtype], self.batch, self.N, self.C, self.D, self.cfg,
            ptr(steps.get("x")), ptr(steps.get("w")), ptr(steps.get("xt", steps.get("x"))),
            ptr(y), HQ_DT[y.dtype], self.qx.st, None if self.qxt is None else self.qxt.st,
            self.qw.st, ptr(self.ws), self.ws_bytes, stream_ptr(stream)), "hq_bmm_fwd")

    def bwd_input(self, dy, dx, steps=None, stream=None):
        steps = steps or {}
        B.check(B.hq_bmm_bwd_input(
            ptr(dy), HQ_DT[dy.dtype], self.batch, self.N, self.C, self.D, self.cfg,
            ptr(steps.get("g")), self.qw.st, ptr(dx), HQ_DT[dx.dtype], self.qg.st, ptr(self.ws),
            self.ws_bytes, stream_ptr(stream)), "hq_bmm_bwd_input")

    def bwd_weight(self, dw, stream=None):
        qx = self.qxt if self.qxt is not None else self.qx
        B.check(B.hq_bmm_bwd_weight(
            self.qg.st, qx.st, self.batch, self.N, self.C, self.D, self.cfg, ptr(dw),
            HQ_DT[dw.dtype], ptr(self.ws), self.ws_bytes, stream_ptr(stream)), "hq_bmm_bwd_weight")


class LssGrad:
    """Buffers for the sampled weight gradient (hq_lss_bwd_weight) of an N x C -> D layer:
    workspace, probabilities, kept-token list and the stats record (kept, s8, s_hi, s_lo)."""

    def __init__(self, N, C, D, k, variant=B.HQ_VARIANT_HQ, device="cuda"):
        self.N, self.C, self.D = N, C, D
        self.cfg = config(k, 4, B.HQ_SCALE_ABSMAX, variant)
        self.ws_bytes = B.hq_lss_workspace_bytes(N, C, D)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)
        self.probs = torch.empty(max(N, 1), dtype=torch.float64, device=device)
        self.kept_idx = torch.empty(max(N, 1), dtype=torch.int32, device=device)
        self.stats = torch.zeros(4, dtype=torch.int32, device=device)   # one hq_lss_stats

    def __call__(self, dy, saved_x, uniforms, dw, budget, stream=None):
        B.check(B.hq_lss_bwd_weight(
            ptr(dy), HQ_DT[dy.dtype], saved_x.st, self.N, self.C, self.D, self.cfg, float(budget),
            ptr(uniforms), ptr(dw), HQ_DT[dw.dtype], ptr(self.probs), ptr(self.kept_idx),
            ptr(self.stats), ptr(self.ws), self.ws_bytes, stream_ptr(stream)),
            "hq_lss_bwd_weight")

    def read_stats(self):
        """(kept, s8, s_hi, s_lo) on the host."""
        h = self.stats.cpu().numpy()
        f = h.view(np.float32)
        return int(h[0]), np.float32(f[1]), np.float32(f[2]), np.float32(f[3])


# ------------------------------------------------------------------ block-scaled FP8, AdamW
def _blocks(n):
    return (n + B.HQ_BLOCK - 1) // B.HQ_BLOCK


def _launch(fn, t, stream, *args):
    """fn(*args, stream) with t's device current (a call launches on the current device), on the
    given stream or the device's current one. The callers check that their other tensors are where
    t is; host memory is refused here, for a kernel would fault on it."""
    if not t.is_cuda:
        raise ValueError("tensors on a GPU are needed, not on %s" % t.device)
    dev = t.device.index
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def _check_matrix(t, rows, cols, name, device=None):
    """A call reads rows x cols contiguous elements at the tensor's address."""
    if tuple(t.shape) != (rows, cols):
        raise ValueError("%s has shape %s, not %s" % (name, tuple(t.shape), (rows, cols)))
    if t.dtype not in HQ_DT:
        raise ValueError("%s has dtype %s: fp32, fp16 or bf16 is needed" % (name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))


class BlockTensor:
    """Caller-owned storage of a block-scaled FP8 matrix (hq_block_tensor): E4M3 codes
    (rows x pitch), transposed codes (cols x pitch) and their scales. ROWS blocks (1 x 128) have
    scales (column blocks x rows) and scales_t (row blocks x cols); TILES (128 x 128) have one
    scales (row blocks x column blocks) for both layouts. New values go into the buffers; the
    buffers themselves stay, for the library's struct holds their addresses."""

    codes = property(operator.attrgetter("_codes"))
    codes_t = property(operator.attrgetter("_codes_t"))
    scales = property(operator.attrgetter("_scales"))
    scales_t = property(operator.attrgetter("_scales_t"))

    def __init__(self, rows, cols, shape=B.HQ_BLOCK_ROWS, scale=B.HQ_BSCALE_F32, codes=True,
                 codes_t=True, device="cuda"):
        if not (codes or codes_t):
            raise ValueError("a BlockTensor holds codes, codes_t or both")

        def new(wanted, *size, dtype=torch.float32):
            return torch.empty(size, dtype=dtype, device=device) if wanted else None

        rows_kind = shape == B.HQ_BLOCK_ROWS
        self._set(rows, cols, shape, scale,
                  new(codes, rows, pitch16(cols), dtype=torch.uint8),
                  new(codes_t, cols, pitch16(rows), dtype=torch.uint8),
                  new(codes, _blocks(cols), rows) if rows_kind
                  else new(True, _blocks(rows), _blocks(cols)),
                  new(codes_t, _blocks(rows), cols) if rows_kind else None)

    def _set(self, rows, cols, shape, scale, codes, codes_t, scales, scales_t):
        self.rows, self.cols, self.shape, self.scale = rows, cols, shape, scale
        self._codes, self._codes_t, self._scales, self._scales_t = codes, codes_t, scales, scales_t
        self.device = next(t for t in (codes, codes_t, scales) if t is not None).device
        st = self.st = B.hq_block_tensor()
        st.codes, st.codes_t = ptr(codes), ptr(codes_t)
        st.scales, st.scales_t = ptr(scales), ptr(scales_t)
        st.rows, st.cols, st.shape, st.scale = rows, cols, shape, scale
        st.ld, st.ld_t, st.lds, st.lds_t = (self._pitch(t) for t in (codes, codes_t, scales, scales_t))

    @staticmethod
    def _pitch(t):
        """Elements between rows (a single row's stride means nothing)."""
        return 0 if t is None else t.stride(0) if t.shape[0] > 1 else t.shape[1]

    @classmethod
    def wrap(cls, codes, scales, rows, cols, shape=B.HQ_BLOCK_TILES, scale=B.HQ_BSCALE_F32,
             codes_t=None, scales_t=None):
        """A matrix whose codes exist already (weights of a checkpoint): codes (rows x pitch, the
        bytes from cols to the next multiple of 16 zero), scales as above. The buffers are used
        as they are. Checks their shapes and, once, on the host, that scales of kind POW2 are
        powers of two from 2^-126 up, NaN, or 0 over codes that are zero."""
        self = cls.__new__(cls)
        parts = [("codes", codes, rows, cols, torch.uint8),
                 ("codes_t", codes_t, cols, rows, torch.uint8)]
        if shape == B.HQ_BLOCK_TILES:
            parts += [("scales", scales, _blocks(rows), _blocks(cols), torch.float32)]
        else:
            parts += [("scales", scales, _blocks(cols), rows, torch.float32),
                      ("scales_t", scales_t, _blocks(rows), cols, torch.float32)]
        for name, t, r, c, dtype in parts:
            if t is None:
                if name in ("codes", "scales"):
                    raise ValueError("%s is needed" % name)
                continue
            if t.dtype != dtype or t.dim() != 2 or t.shape[0] != r or t.shape[1] < c:
                raise ValueError("%s must be a %s tensor of at least %d x %d" % (name, dtype, r, c))
            if t.stride(1) != 1 and t.shape[1] > 1:
                raise ValueError("%s must have contiguous rows" % name)
            if t.device != scales.device:
                raise ValueError("%s is on %s, not on %s" % (name, t.device, scales.device))
            if dtype == torch.uint8 and r and c:   # whole 16-byte pieces of the last row are read
                end = t.storage_offset() + (r - 1) * cls._pitch(t) + pitch16(c)
                if end > t.untyped_storage().nbytes():
                    raise ValueError("%s: the last row must reach to the next multiple of 16 bytes" % name)
        if scale == B.HQ_BSCALE_POW2:
            # by row of codes and block of columns, for each layout
            if shape == B.HQ_BLOCK_TILES:
                every = scales[:, :_blocks(cols)]
                cls._check_pow2(every, codes, 128, cols)
                if codes_t is not None:
                    cls._check_pow2(every.t(), codes_t, 128, rows)
            else:
                cls._check_pow2(scales[:, :rows].t(), codes, 1, cols)
                if codes_t is not None and scales_t is not None:
                    cls._check_pow2(scales_t[:, :cols].t(), codes_t, 1, rows)
        self._set(rows, cols, shape, scale, codes, codes_t, scales, scales_t)
        return self

    @staticmethod
    def _check_pow2(scales, codes, height, cols):
        """Scales of blocks of height x 128 codes whose exponents alone tell them."""
        zero = scales == 0
        power = (scales.view(torch.int32) & 0x7FFFFF == 0) & (scales >= 2.0 ** -126) & scales.isfinite()
        if not bool((power | zero | scales.isnan()).all()):
            raise ValueError("scales of kind POW2 must be powers of two, at least 2^-126")
        if bool(zero.any()):
            under = zero.repeat_interleave(height, 0)[:codes.shape[0]].repeat_interleave(128, 1)
            if bool((codes[:, :cols] & 0x7F)[under[:, :cols]].any()):
                raise ValueError("codes under a scale of 0 (kind POW2) must be zero")

    def quantize(self, src, stream=None):
        """hq_block_quantize of src (rows x cols, contiguous) into these buffers."""
        _check_matrix(src, self.rows, self.cols, "src", self.device)
        B.check(_launch(B.hq_block_quantize, src, stream, src.data_ptr(), HQ_DT[src.dtype],
                        self.rows, self.cols, self.shape, self.scale, self.st),
                "hq_block_quantize")
        return self

    def codes_view(self):
        return None if self.codes is None else self.codes[:, :self.cols]

    def codes_t_view(self):
        return None if self.codes_t is None else self.codes_t[:, :self.rows]


def block_gemm(a, b, c, a_side=B.HQ_SIDE_ROWS, b_side=B.HQ_SIDE_ROWS, accumulate=False, ws=None,
               stream=None):
    """hq_block_gemm: c (+)= a b^T over BlockTensors (HQ_SIDE_COLS reads the transposed codes).
    ws: a uint8 tensor of hq_block_gemm_workspace_bytes, allocated here when missing, from the
    memory of the stream that uses it."""
    M, K = (a.rows, a.cols) if a_side == B.HQ_SIDE_ROWS else (a.cols, a.rows)
    N = b.rows if b_side == B.HQ_SIDE_ROWS else b.cols
    _check_matrix(c, M, N, "c", a.device)
    if b.device != a.device:
        raise ValueError("b is on %s, not on %s" % (b.device, a.device))
    if ws is None:
        with torch.cuda.stream(stream):
            ws = torch.empty(max(B.hq_block_gemm_workspace_bytes(M, N, K), 16), dtype=torch.uint8,
                             device=c.device)
    elif ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != a.device:
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % a.device)
    B.check(_launch(B.hq_block_gemm, c, stream, a.st, a_side, b.st, b_side, c.data_ptr(),
                    HQ_DT[c.dtype], int(accumulate), ws.data_ptr(), ws.numel()), "hq_block_gemm")


class BlockLayer:
    """Buffers for one linear layer (N tokens, C in, D out) in block-scaled FP8 and its calls.

    train=True keeps Q(X) and Q(dY) in both layouts for the weight gradient; train=False is the
    serving form (forward alone, nothing saved). weight: a BlockTensor that the layer reads (D x C,
    for instance BlockTensor.wrap of a checkpoint's codes); without it set_weight quantizes W into
    TILES of the layer's own."""

    def __init__(self, N, C, D, scale=B.HQ_BSCALE_F32, weight=None, train=True, device="cuda"):
        self.N, self.C, self.D, self.scale, self.train = N, C, D, scale, train
        if weight is not None:
            if (weight.rows, weight.cols) != (D, C):
                raise ValueError("weight is %d x %d, not %d x %d" % (weight.rows, weight.cols, D, C))
            device = weight.device
        self.qw = weight or BlockTensor(D, C, shape=B.HQ_BLOCK_TILES, scale=scale, codes_t=train,
                                        device=device)
        self.device = self.qw.device
        self.qx = BlockTensor(N, C, scale=scale, device=device) if train else None
        self.qg = BlockTensor(N, D, scale=scale, device=device) if train else None
        self.ws_bytes = B.hq_block_workspace_bytes(N, C, D)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)

    def set_weight(self, w, stream=None):
        self.qw.quantize(w, stream)

    def fwd(self, x, y, stream=None):
        _check_matrix(x, self.N, self.C, "x", self.device)
        _check_matrix(y, self.N, self.D, "y", self.device)
        B.check(_launch(B.hq_block_linear_fwd, x, stream, x.data_ptr(), HQ_DT[x.dtype], self.N,
                        self.C, self.D, self.qw.st, self.scale, y.data_ptr(), HQ_DT[y.dtype],
                        None if self.qx is None else self.qx.st, self.ws.data_ptr(),
                        self.ws_bytes), "hq_block_linear_fwd")

    def bwd_input(self, dy, dx, stream=None):
        _check_matrix(dy, self.N, self.D, "dy", self.device)
        _check_matrix(dx, self.N, self.C, "dx", self.device)
        B.check(_launch(B.hq_block_linear_bwd_input, dy, stream, dy.data_ptr(), HQ_DT[dy.dtype],
                        self.N, self.C, self.D, self.qw.st, self.scale, dx.data_ptr(),
                        HQ_DT[dx.dtype], None if self.qg is None else self.qg.st,
                        self.ws.data_ptr(), self.ws_bytes), "hq_block_linear_bwd_input")

    def bwd_weight(self, dw, accumulate=False, stream=None):
        """From the codes that fwd and bwd_input saved."""
        if not self.train:
            raise ValueError("a layer made with train=False saves nothing for the weight gradient")
        _check_matrix(dw, self.D, self.C, "dw", self.device)
        B.check(_launch(B.hq_block_linear_bwd_weight, dw, stream, self.qg.st, self.qx.st, self.N,
                        self.C, self.D, dw.data_ptr(), HQ_DT[dw.dtype], int(accumulate),
                        self.ws.data_ptr(), self.ws_bytes), "hq_block_linear_bwd_weight")


class AdamW:
    """AdamW over a list of parameter tensors of one dtype and device (hq_adamw_step).

    state_bits: 32 (fp32 states) or 8 (E4M3 codes with a scale for each 128 elements).
    weight_decay: one number, or one for each tensor. copies: tensors of one dtype that receive
    the updated parameters (the low-precision weights of the next forward); a copy may be its own
    parameter, which then is written once. states: dicts of m, v
    (and m_scales, v_scales for 8 bits) to go on from, used in place; zeros without it.
    steps_done: steps taken before.

    Parameters, copies and states may be bound anew (p.data = ..., opt.states[i]["m"] = ...): the
    next step checks them again and works on the new memory. A captured step keeps the addresses of
    its capture. Gradients share no memory with what a step writes.

    step(grads) takes the next step. Under HIP graph capture a step has to read its scalars from
    device memory: step(grads, captured=True) launches with `device_scalars` (a device tensor of
    five 32-bit words: lr, step_size, inv_sqrt_bias2, grad_scale as floats, then the key), and
    advance(grad_scale, stream) writes the next step's there before each replay, on the stream of
    the replay."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, copies=None, states=None, seed=0, steps_done=0):
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        decay = ([float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float))
                 else [float(w) for w in weight_decay])
        if len(decay) != len(params):
            raise ValueError("weight_decay needs one number for each tensor")
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        self.params, self.device, self.step_count = params, params[0].device, int(steps_done)
        self.state_bits, self._dtype = state_bits, params[0].dtype
        self._check("parameter", params, self._dtype)
        self.copies = None if copies is None else list(copies)
        self._copy_dtype = self.copies[0].dtype if self.copies else self._dtype
        self.states = [self._zeros(p) for p in params] if states is None else list(states)
        if len(self.states) != len(params):
            raise ValueError("one state for each parameter is needed")
        c = self.cfg = B.hq_adamw_config()
        c.lr, (c.beta1, c.beta2), c.eps = lr, betas, eps
        self._state_keys = ("m", "v") + (("m_scales", "v_scales") if state_bits == 8 else ())
        self._state_of = operator.itemgetter(*self._state_keys)
        self._table, self._decay = (B.hq_adamw_tensor * len(params))(), decay
        self._bind()
        c.param_dtype, c.copy_dtype = HQ_DT[self._dtype], HQ_DT[self._copy_dtype]
        c.grad_dtype, c.state_bits, c.seed = c.param_dtype, state_bits, seed & 0xFFFFFFFF
        self._scalars = B.hq_adamw_scalars()
        # made here: made under capture, it would be cleared again by each replay
        self.device_scalars = torch.zeros(5, dtype=torch.float32, device=self.device)

    def _addresses(self):
        """Those of every tensor that a step writes."""
        states = itertools.chain.from_iterable(map(self._state_of, self.states))
        return list(map(torch.Tensor.data_ptr,
                        itertools.chain(self.params, self.copies or (), states)))

    def _bind(self):
        """Check the tensors that a step works on and note their addresses."""
        if len(self.params) != len(self._table) or len(self.states) != len(self._table):
            raise ValueError("%d parameters and %d states for an optimizer of %d"
                             % (len(self.params), len(self.states), len(self._table)))
        self._check("parameter", self.params, self._dtype)
        if self.copies is not None:
            self._check("copy", self.copies, self._copy_dtype)
        for p, s in zip(self.params, self.states):
            self._check_state(s, p.numel())
        self._check_overlap()
        rows = []
        for i, (t, p, s) in enumerate(zip(self._table, self.params, self.states)):
            t.p, t.n, t.weight_decay = ptr(p), p.numel(), self._decay[i]
            t.m, t.v = ptr(s["m"]), ptr(s["v"])
            t.m_scales, t.v_scales = (ptr(s[k]) if self.state_bits == 8 else None
                                      for k in ("m_scales", "v_scales"))
            copy = self.copies[i] if self.copies else None
            t.copy = None if copy is None or self._is_same(copy, p) else ptr(copy)
            rows.append((t, p.numel()))
        self._rows = rows
        self._bound = self._addresses()

    def _is_bound(self):
        """The table's addresses are the tensors', whose elements are still in order. (A call for
        each tensor: 2 us on the host for 12 parameters with 32-bit states.)"""
        try:
            return (self._addresses() == self._bound
                    and all(map(torch.Tensor.is_contiguous,
                                itertools.chain(self.params, self.copies or ()))))
        except KeyError:    # a state's entry is gone
            return False

    @staticmethod
    def _is_same(copy, p):
        return copy.dtype == p.dtype and copy.data_ptr() == p.data_ptr()

    def _check_overlap(self):
        """All that a step writes has to be disjoint (a copy that is its own parameter aside): a
        parameter listed twice would be updated by two workgroups at once."""
        written = [*self.params] + [s[k] for s in self.states for k in self._state_keys]
        written += [c for c, p in zip(self.copies or [], self.params) if not self._is_same(c, p)]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                       for t in written if t.numel())
        for (_, end), (start, _) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("parameters, copies and states must not overlap")

    def _zeros(self, p):
        n, dev = p.numel(), p.device
        if self.state_bits == 32:
            return {k: torch.zeros(n, dtype=torch.float32, device=dev) for k in ("m", "v")}
        s = {k: torch.zeros(n, dtype=torch.uint8, device=dev) for k in ("m", "v")}
        s.update({k + "_scales": torch.zeros(_blocks(n), dtype=torch.float32, device=dev)
                  for k in ("m", "v")})
        return s

    def _check(self, what, tensors, dtype):
        if len(tensors) != len(self.params):
            raise ValueError("%d tensors of kind %s for %d parameters"
                             % (len(tensors), what, len(self.params)))
        for i, (t, p) in enumerate(zip(tensors, self.params)):
            if t.numel() != p.numel() or not t.is_contiguous() or t.device != self.device:
                raise ValueError("%s %d must be contiguous, on %s, with %d elements"
                                 % (what, i, self.device, p.numel()))
            if t.dtype != dtype or t.dtype not in HQ_DT:
                raise ValueError("%s %d has dtype %s: one of fp32, fp16, bf16 for all is needed"
                                 % (what, i, t.dtype))

    def _check_state(self, s, n):
        eight = self.state_bits == 8
        parts = [(k, n, torch.uint8 if eight else torch.float32) for k in ("m", "v")]
        if eight:
            parts += [(k, _blocks(n), torch.float32) for k in ("m_scales", "v_scales")]
        for k, size, dtype in parts:
            t = s.get(k)
            if (t is None or t.numel() != size or t.dtype != dtype or not t.is_contiguous()
                    or t.device != self.device):
                raise ValueError("state %s must be a contiguous %s tensor of %d elements on %s"
                                 % (k, dtype, size, self.device))

    def set_lr(self, lr):
        self.cfg.lr = lr

    def advance(self, grad_scale=1.0, stream=None):
        """Count one step and write its scalars to device_scalars, in the order of the given stream
        (or the current one), without waiting for it. Each call's words go through pinned memory of
        their own, which torch hands out again once their copy is done."""
        if stream is not None and stream.device != self.device:
            raise ValueError("the stream is of %s, not of %s" % (stream.device, self.device))
        s = self._scalars
        B.check(B.hq_adamw_scalars_at(self.cfg, self.step_count + 1, grad_scale, s),
                "hq_adamw_scalars_at")
        self.step_count += 1
        host = torch.frombuffer(bytearray(bytes(s)), dtype=torch.float32).pin_memory()
        with torch.cuda.stream(stream):
            self.device_scalars.copy_(host, non_blocking=True)

    def step(self, grads, grad_scale=1.0, captured=False, stream=None):
        """One step with one gradient for each parameter (one dtype for all). A captured one takes
        its gradient scale from advance()."""
        if captured and grad_scale != 1.0:
            raise ValueError("a captured step reads its gradient scale from what advance() wrote")
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(self.params)))
        dtype, index = grads[0].dtype, self.params[0].get_device()
        if dtype not in HQ_DT:
            raise ValueError("gradients have dtype %s: fp32, fp16 or bf16 is needed" % dtype)
        if not self._is_bound():
            self._bind()
        for g, (row, n) in zip(grads, self._rows):
            if g.dtype != dtype or g.numel() != n or g.get_device() != index or not g.is_contiguous():
                raise ValueError("gradients must be contiguous %s tensors on %s with their "
                                 "parameters' numbers of elements" % (dtype, self.device))
            row.grad = g.data_ptr()
        self.cfg.grad_dtype = HQ_DT[dtype]
        if captured:
            scalars = None
        else:
            scalars = self._scalars
            B.check(B.hq_adamw_scalars_at(self.cfg, self.step_count + 1, grad_scale, scalars),
                    "hq_adamw_scalars_at")
        B.check(_launch(B.hq_adamw_step, self.params[0], stream, self._table, len(self.params),
                        self.cfg, scalars, ptr(self.device_scalars) if captured else None),
                "hq_adamw_step")
        if not captured:
            self.step_count += 1

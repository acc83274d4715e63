"""8-bit projections on torch tensors over the C ABI: RMSNorm with E4M3 output, weights
quantised in 128 x 128 blocks, and the product of the two.  Marshalling only.

A quantised matrix of n rows of k values is a pair (q, scale): q [n, k] float8_e4m3fn (or uint8)
with a row pitch of k rounded up to 16 bytes, scale uint8 with one E8M0 byte (2^(byte - 127))
per 128 values at a pitch of ceil(k / 128) rounded up to 4: [n, pitch] for rows, [ceil(n / 128),
pitch] for weights.  ``empty`` allocates such a pair.

Calls run on the current stream of the tensors' device."""

from __future__ import annotations

import torch

from . import abi

_DTYPES = {torch.float32: abi.DS4C_F32, torch.bfloat16: abi.DS4C_BF16}
_BYTES = (torch.float8_e4m3fn, torch.uint8)


def row_bytes(k: int) -> int:
    """Pitch of a quantised row of k values."""
    return (k + 15) // 16 * 16


def scale_bytes(k: int) -> int:
    """Pitch of the scales of a row of k values."""
    return ((k + 127) // 128 + 3) // 4 * 4


def empty(n: int, k: int, device="cuda", rows_per_scale: int = 1):
    """Uninitialised (q, scale) for n rows of k values, one scale row per rows_per_scale rows."""
    q = torch.empty(n, row_bytes(k), dtype=torch.float8_e4m3fn, device=device)[:, :k]
    return q, torch.empty((n + rows_per_scale - 1) // rows_per_scale, scale_bytes(k), dtype=torch.uint8, device=device)


def _dtype(t, what):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{what}: {t.dtype} (float32 or bfloat16)")
    return d


def _pitch(t, n, k, what, device):
    """Row pitch of a [n, k] tensor with unit column stride."""
    if t.dim() != 2 or t.shape[0] != n or t.shape[1] != k:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {(n, k)}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if k > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the rows' elements must be contiguous")
    return t.stride(0) if n > 1 else max(k, t.stride(0))


def check_rows(q, scale, k: int, rows_per_scale: int = 1):
    """Raise unless (q, scale) is a quantised matrix of rows of k values on one CUDA device."""
    n = q.shape[0] if q.dim() == 2 else -1
    if q.dtype not in _BYTES or scale.dtype != torch.uint8 or q.device.type != "cuda":
        raise ValueError(f"quantised rows: {q.dtype} on {q.device} with {scale.dtype} scales")
    if n < 0 or q.shape[1] != k or (k > 1 and q.stride(1) != 1) or (n > 1 and q.stride(0) != row_bytes(k)):
        raise ValueError(f"quantised rows: shape {tuple(q.shape)} stride {q.stride()}, expected (*, {k}) at a pitch of "
                         f"{row_bytes(k)}")
    if scale.device != q.device or tuple(scale.shape) != ((n + rows_per_scale - 1) // rows_per_scale, scale_bytes(k)) \
            or not scale.is_contiguous():
        raise ValueError(f"scales: shape {tuple(scale.shape)} on {scale.device}, expected "
                         f"{((n + rows_per_scale - 1) // rows_per_scale, scale_bytes(k))}, contiguous, on {q.device}")


def _run(device, call):
    """call(stream) with `device` current, on its current stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}: a CUDA device is needed")
    if device.index == torch.cuda.current_device():
        return call(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        return call(torch.cuda.current_stream().cuda_stream)


def rmsnorm(x, gain=None, *, residual=None, residual_out=None, eps: float = 1e-6, q=None, scale=None, y=None):
    """RMSNorm of x [n, d] (float32 or bfloat16; rows may be strided), quantised: returns (q, scale).

    With a residual the norm is of h = x + residual rounded to x's type; h goes to residual_out, which
    may be x or residual itself.  gain: [d] float32 or None (ones).  q, scale: outputs as ``empty``
    gives them, allocated if None.  y: optional output of x's type, the norm before its quantisation."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected two dimensions")
    n, d = x.shape
    dev = x.device
    dt = _dtype(x, "x")
    a = abi.RmsnormArgs(n, d, dt, eps, x.data_ptr())
    a.x_ld = _pitch(x, n, d, "x", dev)
    for name, t in (("residual", residual), ("residual_out", residual_out), ("y", y)):
        if t is not None:
            if t.dtype != x.dtype:
                raise ValueError(f"{name}: {t.dtype}, expected x's {x.dtype}")
            setattr(a, "y_out" if name == "y" else name, t.data_ptr())
            setattr(a, name + "_ld", _pitch(t, n, d, name, dev))
    if gain is not None:
        if gain.dtype != torch.float32 or tuple(gain.shape) != (d,) or gain.device != dev or not gain.is_contiguous():
            raise ValueError(f"gain: {gain.dtype} {tuple(gain.shape)} on {gain.device}, expected contiguous float32 {(d,)}")
        a.gain = gain.data_ptr()
    if q is None and scale is None:
        q, scale = empty(n, d, dev)
    if q is None or scale is None:
        raise ValueError("q and scale: both or neither")
    check_rows(q, scale, d)
    if q.shape[0] != n or q.device != dev:
        raise ValueError(f"q: {q.shape[0]} rows on {q.device}, expected {n} on {dev}")
    a.q, a.scale = q.data_ptr(), scale.data_ptr()
    abi.check(_run(dev, lambda s: abi.ds4c_rmsnorm_quant(a, s)), "ds4c_rmsnorm_quant")
    return q, scale


class Fp8Weight:
    """A weight matrix [n, k] in E4M3 with one scale per 128 x 128 block."""

    def __init__(self, q, scale):
        check_rows(q, scale, q.shape[1], 128)
        self.q, self.scale = q, scale

    @property
    def shape(self):
        return self.q.shape


def quantize_weight(w, q=None, scale=None) -> Fp8Weight:
    """w [n, k] (float32 or bfloat16; rows may be strided) quantised in blocks of 128 x 128."""
    if w.dim() != 2:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected two dimensions")
    n, k = w.shape
    dt = _dtype(w, "w")
    ld = _pitch(w, n, k, "w", w.device)
    if q is None and scale is None:
        q, scale = empty(n, k, w.device, 128)
    if q is None or scale is None:
        raise ValueError("q and scale: both or neither")
    out = Fp8Weight(q, scale)
    if tuple(q.shape) != (n, k) or q.device != w.device:
        raise ValueError(f"q: shape {tuple(q.shape)} on {q.device}, expected {(n, k)} on {w.device}")
    abi.check(_run(w.device, lambda s: abi.ds4c_quant_weight(n, k, dt, w.data_ptr(), ld, q.data_ptr(), scale.data_ptr(), s)),
              "ds4c_quant_weight")
    return out


class Linear:
    """1 to 4 weight matrices of one width over the same rows: out_g = rows @ w_g.T in one launch."""

    def __init__(self, weights):
        self.weights = list(weights)
        if not 1 <= len(self.weights) <= 4:
            raise ValueError(f"{len(self.weights)} weight matrices: 1 to 4")
        self.k = self.weights[0].shape[1]
        self.device = self.weights[0].q.device
        for w in self.weights:
            if w.shape[1] != self.k or w.q.device != self.device:
                raise ValueError(f"weights of {w.shape[1]} columns on {w.q.device}, expected {self.k} on {self.device}")

    def __call__(self, q, scale, out=None, dtype=torch.float32):
        """q, scale: quantised rows [m, k].  out: list of [m, n_g] tensors of one type (float32 or bfloat16;
        rows may be strided), allocated in `dtype` if None.  Returns them."""
        check_rows(q, scale, self.k)
        m = q.shape[0]
        if q.device != self.device:
            raise ValueError(f"rows on {q.device}, weights on {self.device}")
        if out is None:
            out = [torch.empty(m, w.shape[0], dtype=dtype, device=self.device) for w in self.weights]
        if len(out) != len(self.weights) or any(o.dtype != out[0].dtype for o in out):
            raise ValueError(f"{len(out)} outputs for {len(self.weights)} weight matrices, of one type")
        dt = _dtype(out[0], "out")
        mats = (abi.QuantMatrix * len(out))()
        for g, (w, o) in enumerate(zip(self.weights, out)):
            n = w.shape[0]
            mats[g] = abi.QuantMatrix(w.q.data_ptr(), w.scale.data_ptr(), o.data_ptr(), _pitch(o, m, n, "out", self.device), n)
        abi.check(_run(self.device, lambda s: abi.ds4c_quant_matmul(m, self.k, q.data_ptr(), scale.data_ptr(), mats,
                                                                    len(out), dt, s)), "ds4c_quant_matmul")
        return out

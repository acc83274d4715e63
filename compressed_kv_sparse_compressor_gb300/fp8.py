"""8-bit projections on torch tensors over the C ABI: RMSNorm with E4M3 output, weights
quantised in 128 x 128 blocks, and the product of the two.  Marshalling only.

A quantised matrix of n rows of k values is a pair (q, scale): q [n, k] float8_e4m3fn (or uint8)
with a row pitch of k rounded up to 16 bytes, scale uint8 with one E8M0 byte (2^(byte - 127))
per 128 values at a pitch of ceil(k / 128) rounded up to 4: [n, pitch] for rows, [ceil(n / 128),
pitch] for weights.  ``empty`` allocates such a pair.

Calls run on the current stream of the tensors' device and report what the host can see.  A product
whose kernel gives up waiting (its waits are bounded) leaves outputs unwritten: ``sync`` waits for the
stream and raises in that case.

A decode step's kernels take a few microseconds, so the checks read each tensor's attributes once and
go to the stream's and the device's raw handles (``rmsnorm`` took 14.9 us of host time on torch's
stream objects)."""

from __future__ import annotations

import torch

from . import abi

_DTYPES = {torch.float32: abi.DS4C_F32, torch.bfloat16: abi.DS4C_BF16}
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_E8M0 = torch.uint8
_device, _stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


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


def _matrix(t, what):
    """(n, k, ABI dtype, device index, row pitch) of a float matrix with contiguous rows on a GPU."""
    shape = t.shape
    dt = _DTYPES.get(t.dtype)
    dev = t.get_device()
    if len(shape) != 2 or dt is None or dev < 0:
        raise ValueError(f"{what}: {t.dtype} {tuple(shape)} on {t.device}, expected a float32 or bfloat16 matrix on a "
                         "CUDA device")
    n, k = shape
    row, col = t.stride()
    if col != 1 and k > 1:
        raise ValueError(f"{what}: the rows' elements must be contiguous")
    return n, k, dt, dev, row if n > 1 else max(k, row)


def _pitch(t, n, k, dtype, dev, what):
    """Row pitch of a [n, k] tensor of `dtype` with unit column stride on device `dev`."""
    if t.shape != (n, k) or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} {(n, k)} on cuda:{dev}")
    row, col = t.stride()
    if col != 1 and k > 1:
        raise ValueError(f"{what}: the rows' elements must be contiguous")
    return row if n > 1 else max(k, row)


def check_rows(q, scale, k: int, rows_per_scale: int = 1):
    """Number of rows and device index of a quantised matrix (q, scale) of rows of k values on one CUDA
    device; raises if it is none."""
    shape, dev = q.shape, q.get_device()
    if len(shape) != 2 or shape[1] != k or dev < 0 or q.dtype not in _BYTES:
        raise ValueError(f"quantised rows: {q.dtype} {tuple(shape)} on {q.device}, expected E4M3 (*, {k}) on a CUDA device")
    n = shape[0]
    row, col = q.stride()
    if (row != (k + 15) // 16 * 16 and n > 1) or (col != 1 and k > 1):
        raise ValueError(f"quantised rows: stride {(row, col)}, expected {(row_bytes(k), 1)}")
    want = (n if rows_per_scale == 1 else (n + rows_per_scale - 1) // rows_per_scale, ((k + 127) // 128 + 3) // 4 * 4)
    if scale.shape != want or scale.dtype != _E8M0 or scale.get_device() != dev or not scale.is_contiguous():
        raise ValueError(f"scales: {scale.dtype} {tuple(scale.shape)} on {scale.device}, expected contiguous uint8 {want} on "
                         f"cuda:{dev}")
    return n, dev


def run(dev, fn, *args):
    """fn(*args, stream) with device `dev` current, on its current stream; raises the ABI's errors."""
    if dev == _device():
        status = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(dev))
    if status:
        raise abi.Ds4cError(status, fn.__name__)


def sync(device=None):
    """Waits for the current stream of `device` (the current device if None); raises Ds4cError if a kernel launched on
    the device since the last such check gave up, or if the stream failed."""
    dev = _device() if device is None else torch.device(device).index
    run(_device() if dev is None else dev, abi.ds4c_sync_status)


def rmsnorm(x, gain=None, *, residual=None, residual_out=None, eps: float = 1e-6, q=None, scale=None, y=None):
    """RMSNorm of x [n, d] (float32 or bfloat16; rows may be strided), quantised: returns (q, scale).

    With a residual the norm is of h = x + residual rounded to x's type; h goes to residual_out, which
    may be x or residual itself.  gain: [d] float32 or None (ones).  q, scale: outputs as ``empty``
    gives them, allocated if None.  y: optional output of x's type, the norm before its quantisation."""
    n, d, dt, dev, x_ld = _matrix(x, "x")
    if q is None or scale is None:
        if q is not scale:
            raise ValueError("q and scale: both or neither")
        q, scale = empty(n, d, x.device)
    if check_rows(q, scale, d) != (n, dev):
        raise ValueError(f"q: {q.shape[0]} rows on {q.device}, expected {n} on cuda:{dev}")
    xt = x.dtype
    r = h = yp = g = None
    r_ld = h_ld = y_ld = 0
    if residual is not None:
        r, r_ld = residual.data_ptr(), _pitch(residual, n, d, xt, dev, "residual")
    if residual_out is not None:
        h, h_ld = residual_out.data_ptr(), _pitch(residual_out, n, d, xt, dev, "residual_out")
    if y is not None:
        yp, y_ld = y.data_ptr(), _pitch(y, n, d, xt, dev, "y")
    if gain is not None:
        if gain.shape != (d,) or gain.dtype != torch.float32 or gain.get_device() != dev or not gain.is_contiguous():
            raise ValueError(f"gain: {gain.dtype} {tuple(gain.shape)} on {gain.device}, expected contiguous float32 {(d,)} on "
                             f"cuda:{dev}")
        g = gain.data_ptr()
    run(dev, abi.ds4c_rmsnorm_quant, abi.RmsnormArgs(n, d, dt, eps, x.data_ptr(), r, h, yp, x_ld, r_ld, h_ld, y_ld, g,
                                                      q.data_ptr(), scale.data_ptr()))
    return q, scale


class Fp8Weight:
    """A weight matrix [n, k] in E4M3 with one scale per 128 x 128 block."""

    def __init__(self, q, scale):
        self.device_index = check_rows(q, scale, q.shape[-1], 128)[1]
        self.q, self.scale = q, scale

    @property
    def shape(self):
        return self.q.shape


def quantize_weight(w, q=None, scale=None) -> Fp8Weight:
    """w [n, k] (float32 or bfloat16; rows may be strided) quantised in blocks of 128 x 128."""
    n, k, dt, dev, ld = _matrix(w, "w")
    if q is None or scale is None:
        if q is not scale:
            raise ValueError("q and scale: both or neither")
        q, scale = empty(n, k, w.device, 128)
    out = Fp8Weight(q, scale)
    if q.shape != (n, k) or out.device_index != dev:
        raise ValueError(f"q: {tuple(q.shape)} on {q.device}, expected {(n, k)} on cuda:{dev}")
    run(dev, abi.ds4c_quant_weight, n, k, dt, w.data_ptr(), ld, q.data_ptr(), scale.data_ptr())
    return out


class Linear:
    """1 to 4 weight matrices of one width over the same rows: out_g = rows @ w_g.T in one launch.

    Holds the weights; their addresses are read once, here.  ``sync`` says whether a launch gave up."""

    def __init__(self, weights):
        self.weights = list(weights)
        if not 1 <= len(self.weights) <= 4:
            raise ValueError(f"{len(self.weights)} weight matrices: 1 to 4")
        self.k = self.weights[0].shape[1]
        self.device_index = self.weights[0].device_index
        for w in self.weights:
            if w.shape[1] != self.k or w.device_index != self.device_index:
                raise ValueError(f"weights of {w.shape[1]} columns on {w.q.device}, expected {self.k} on "
                                 f"cuda:{self.device_index}")
        self._n = [w.shape[0] for w in self.weights]
        self._mats_t = abi.QuantMatrix * len(self.weights)
        self._mats = bytes(self._mats_t(*[abi.QuantMatrix(w.q.data_ptr(), w.scale.data_ptr(), None, 0, w.shape[0])
                                          for w in self.weights]))

    def __call__(self, q, scale, out=None, dtype=torch.float32):
        """q, scale: quantised rows [m, k].  out: list of [m, n_g] tensors of one type (float32 or bfloat16;
        rows may be strided), allocated in `dtype` if None.  Returns them."""
        m, dev = check_rows(q, scale, self.k)
        if dev != self.device_index:
            raise ValueError(f"rows on {q.device}, weights on cuda:{self.device_index}")
        if out is None:
            out = [torch.empty(m, n, dtype=dtype, device=q.device) for n in self._n]
        if len(out) != len(self._n):
            raise ValueError(f"{len(out)} outputs for {len(self._n)} weight matrices")
        odt = out[0].dtype
        dt = _DTYPES.get(odt)
        if dt is None:
            raise ValueError(f"out: {odt} (float32 or bfloat16)")
        mats = self._mats_t.from_buffer_copy(self._mats)        # of this call: another thread may be in its own
        for mat, o, n in zip(mats, out, self._n):
            if o.shape != (m, n) or o.dtype != odt or o.get_device() != dev:
                raise ValueError(f"out: {o.dtype} {tuple(o.shape)} on {o.device}, expected {odt} {(m, n)} on cuda:{dev}")
            row, col = o.stride()
            if col != 1 and n > 1:
                raise ValueError("out: the rows' elements must be contiguous")
            mat.out_ld = row if m > 1 else max(n, row)
            mat.out = o.data_ptr()
        run(dev, abi.ds4c_quant_matmul, m, self.k, q.data_ptr(), scale.data_ptr(), mats, len(out), dt)
        return out

"""Torch-facing helpers over the C ABI: allocate device buffers with torch, pass their
addresses and the current stream to libtcq.  No arithmetic happens here."""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import _lib


def nwords(k: int, T: int) -> int:
    return (k * T + 31) // 32


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


@dataclass
class Encoded:
    bitstream: torch.Tensor    # uint32 [blocks, nwords] (stored as int32)
    start_state: torch.Tensor  # uint32 [blocks] (stored as int32)
    cost: torch.Tensor         # float32 [blocks]
    recon: torch.Tensor | None  # float32 [M, N]


class Workspace:
    """Device workspace owned by torch's allocator."""

    def __init__(self, nbytes: int, device="cuda"):
        self.nbytes = int(nbytes)
        self.buf = torch.empty(max(self.nbytes, 1), dtype=torch.uint8, device=device)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def make_codebook(L: int, V: int, seed: int, device="cuda") -> torch.Tensor:
    host = _lib.tcq_make_codebook(L, V, seed)
    return torch.from_numpy(host).to(device)


def encode(W: torch.Tensor, d: torch.Tensor | None, codebook: torch.Tensor, L: int, k: int,
           V: int, T: int, recon: bool = False, workspace: Workspace | None = None,
           out: Encoded | None = None) -> Encoded:
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    M, N = W.shape
    assert codebook.is_cuda and codebook.dtype == torch.float32 and codebook.is_contiguous()
    if d is not None:
        assert d.is_cuda and d.dtype == torch.float32 and d.is_contiguous() and d.numel() == N
    nb = M * (N // T) if T > 0 else 0
    if out is None:
        dev = W.device
        out = Encoded(
            bitstream=torch.empty((nb, nwords(k, T)), dtype=torch.int32, device=dev),
            start_state=torch.empty(nb, dtype=torch.int32, device=dev),
            cost=torch.empty(nb, dtype=torch.float32, device=dev),
            recon=torch.empty((M, N), dtype=torch.float32, device=dev) if recon else None)
    if workspace is None:
        workspace = Workspace(_lib.tcq_encode_workspace_bytes(M, N, L, k, V, T), W.device)
    _lib.tcq_encode(W.data_ptr(), M, N, W.stride(0), None if d is None else d.data_ptr(),
                    codebook.data_ptr(), L, k, V, T, out.bitstream.data_ptr(),
                    out.start_state.data_ptr(), out.cost.data_ptr(),
                    None if out.recon is None else out.recon.data_ptr(),
                    N if out.recon is None else out.recon.stride(0), workspace.ptr,
                    workspace.nbytes, _stream())
    return out


def decode(bitstream: torch.Tensor, start_state: torch.Tensor, codebook: torch.Tensor, M: int,
           N: int, L: int, k: int, V: int, T: int) -> torch.Tensor:
    out = torch.empty((M, N), dtype=torch.float32, device=bitstream.device)
    _lib.tcq_decode(bitstream.data_ptr(), start_state.data_ptr(), codebook.data_ptr(), M, N,
                    L, k, V, T, out.data_ptr(), N, _stream())
    return out


def decode_gemv(bitstream: torch.Tensor, start_state: torch.Tensor, codebook: torch.Tensor,
                x: torch.Tensor, M: int, N: int, L: int, k: int, V: int, T: int) -> torch.Tensor:
    assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous() and x.numel() == N
    y = torch.empty(M, dtype=torch.float32, device=x.device)
    _lib.tcq_decode_gemv(bitstream.data_ptr(), start_state.data_ptr(), codebook.data_ptr(), M,
                         N, L, k, V, T, x.data_ptr(), y.data_ptr(), _stream())
    return y


@dataclass
class EncodedLdlq(Encoded):
    target: torch.Tensor | None = None  # float32 [M, N]


def encode_ldlq(W: torch.Tensor, U: torch.Tensor | None, d: torch.Tensor | None,
                codebook: torch.Tensor, L: int, k: int, V: int, T: int, recon: bool = True,
                target: bool = False, workspace: Workspace | None = None) -> EncodedLdlq:
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    M, N = W.shape
    if U is not None:
        assert U.is_cuda and U.dtype == torch.float32 and U.dim() == 2 and U.stride(1) == 1
    if d is not None:
        assert d.is_cuda and d.dtype == torch.float32 and d.is_contiguous() and d.numel() == N
    nb = M * (N // T)
    dev = W.device
    out = EncodedLdlq(
        bitstream=torch.empty((nb, nwords(k, T)), dtype=torch.int32, device=dev),
        start_state=torch.empty(nb, dtype=torch.int32, device=dev),
        cost=torch.empty(nb, dtype=torch.float32, device=dev),
        recon=torch.empty((M, N), dtype=torch.float32, device=dev) if recon else None,
        target=torch.empty((M, N), dtype=torch.float32, device=dev) if target else None)
    if workspace is None:
        workspace = Workspace(_lib.tcq_ldlq_workspace_bytes(M, N, L, k, V, T), dev)
    _lib.tcq_encode_ldlq(W.data_ptr(), M, N, W.stride(0),
                         None if U is None else U.data_ptr(), N if U is None else U.stride(0),
                         None if d is None else d.data_ptr(), codebook.data_ptr(), L, k, V, T,
                         out.bitstream.data_ptr(), out.start_state.data_ptr(),
                         out.cost.data_ptr(), None if out.recon is None else out.recon.data_ptr(),
                         N, None if out.target is None else out.target.data_ptr(), N,
                         workspace.ptr, workspace.nbytes, _stream())
    return out


def bcjr(W: torch.Tensor, d: torch.Tensor | None, codebook: torch.Tensor, L: int, k: int,
         V: int, T: int, tau: float, workspace: Workspace | None = None
         ) -> tuple[torch.Tensor, torch.Tensor]:
    """Soft codewords (float32 [M, N]) and log Z per block (float32 [M*N/T])."""
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    M, N = W.shape
    if d is not None:
        assert d.is_cuda and d.dtype == torch.float32 and d.is_contiguous() and d.numel() == N
    soft = torch.empty((M, N), dtype=torch.float32, device=W.device)
    logz = torch.empty(M * (N // T), dtype=torch.float32, device=W.device)
    if workspace is None:
        workspace = Workspace(_lib.tcq_bcjr_workspace_bytes(M, N, L, k, V, T), W.device)
    _lib.tcq_bcjr(W.data_ptr(), M, N, W.stride(0), None if d is None else d.data_ptr(),
                  codebook.data_ptr(), L, k, V, T, float(tau), soft.data_ptr(), N,
                  logz.data_ptr(), workspace.ptr, workspace.nbytes, _stream())
    return soft, logz


def hadamard(X: torch.Tensor, n: int, sigma: torch.Tensor | None = None, inverse: bool = False,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """Rows of X rotated by R = H_n diag(sigma)/sqrt(n) in chunks of n (inverse: R^T)."""
    assert X.is_cuda and X.dtype == torch.float32 and X.dim() == 2 and X.stride(1) == 1
    rows, length = X.shape
    if sigma is not None:
        assert sigma.is_cuda and sigma.dtype == torch.float32 and sigma.is_contiguous()
    if out is None:
        out = torch.empty_like(X)
    _lib.tcq_hadamard(X.data_ptr(), rows, length, X.stride(0), n,
                      None if sigma is None else sigma.data_ptr(), inverse, out.data_ptr(),
                      out.stride(0), _stream())
    return out


def scale_field(W: torch.Tensor, normalized: bool = True
                ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """(row_scale [M], col_scale [N], Wn [M, N] or None) with W = a_r b_c Wn_rc."""
    assert W.is_cuda and W.dtype == torch.float32 and W.dim() == 2 and W.stride(1) == 1
    M, N = W.shape
    a = torch.empty(M, dtype=torch.float32, device=W.device)
    b = torch.empty(N, dtype=torch.float32, device=W.device)
    Wn = torch.empty_like(W) if normalized else None
    ws = Workspace(_lib.tcq_scale_field_workspace_bytes(M, N), W.device)
    _lib.tcq_scale_field(W.data_ptr(), M, N, W.stride(0), a.data_ptr(), b.data_ptr(),
                         None if Wn is None else Wn.data_ptr(), N, ws.ptr, ws.nbytes, _stream())
    return a, b, Wn


_DTYPES = {torch.float32: _lib.TCQ_F32, torch.float16: _lib.TCQ_F16,
           torch.bfloat16: _lib.TCQ_BF16}
_ACTS = {"none": _lib.TCQ_ACT_NONE, "relu": _lib.TCQ_ACT_RELU, "silu": _lib.TCQ_ACT_SILU,
         "gelu": _lib.TCQ_ACT_GELU}
CHECKPOINT_GROUP = 32  # consecutive values of a row that share a scale byte


def _on(device: torch.device):
    """The tensors' device made current, where it is not: the launch and the stream are
    its own."""
    if device.index is None or device.index == torch.cuda.current_device():
        return nullcontext()
    return torch.cuda.device(device)


def _stream_of(device: torch.device) -> int:
    """The device's current stream, without the Stream object that the public query builds
    (2.7 us of a 12 us call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _rows(t: torch.Tensor, name: str, rows: int, cols: int, dtype: torch.dtype,
          device: torch.device) -> int:
    """Checks a rows x cols matrix whose rows are contiguous; its leading dimension."""
    assert t.device == device and t.dtype == dtype, f"{name}: {dtype} on {device}"
    assert t.shape == (rows, cols), f"{name}: shape {tuple(t.shape)}, not {(rows, cols)}"
    # a dimension of at most one element may carry any stride
    assert cols <= 1 or t.stride(1) == 1, f"{name}: rows must be contiguous"
    ld = t.stride(0) if rows > 1 else cols
    assert ld >= cols, f"{name}: rows overlap"
    return max(ld, 1)


def _workspace(workspace: Workspace | None, device: torch.device) -> tuple[int | None, int]:
    """Address and size of a call's workspace, which the tensors' device must hold."""
    if workspace is None:
        return None, 0
    assert workspace.buf.device == device, f"workspace: on {device}"
    return workspace.ptr, workspace.nbytes


def _vector(t: torch.Tensor | None, name: str, n: int, device: torch.device) -> int | None:
    if t is None:
        return None
    assert t.device == device and t.dtype == torch.float32 and t.is_contiguous() and \
        t.numel() == n, f"{name}: {n} contiguous float32 values on {device}"
    return t.data_ptr()


def _coded(bitstream: torch.Tensor, start_state: torch.Tensor, codebook: torch.Tensor, M: int,
           N: int, L: int, k: int, V: int, T: int, dtype: torch.dtype,
           device: torch.device) -> None:
    blocks = M * (N // T)
    assert bitstream.device == device and bitstream.is_contiguous() and \
        bitstream.element_size() == 4 and bitstream.numel() == blocks * nwords(k, T)
    assert start_state.device == device and start_state.is_contiguous() and \
        start_state.element_size() == 4 and start_state.numel() == blocks
    assert codebook.device == device and codebook.dtype == dtype and \
        codebook.is_contiguous() and codebook.numel() == V << L, \
        f"codebook: {V << L} contiguous values of the layer's type {dtype}"


def decode_linear(bitstream: torch.Tensor, start_state: torch.Tensor, codebook: torch.Tensor,
                  x: torch.Tensor, M: int, N: int, L: int, k: int, V: int, T: int,
                  row_scale: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                  act: str = "none", residual: torch.Tensor | None = None, pre: bool = False,
                  out: torch.Tensor | None = None, workspace: Workspace | None = None
                  ) -> torch.Tensor | tuple[torch.Tensor, torch.Tensor]:
    """act(row_scale (x W_hat^T) + bias) + residual for x [B, N] in float32, float16 or
    bfloat16 and the coded matrix W_hat [M, N] (codebook in x's type); [B, M], or with
    ``pre`` the pair of it and the pre-activation.  act: none, relu, silu or gelu.  ``out``
    may be ``residual``, but not overlap x.  The outputs carry no autograd graph, whatever x
    requires: the gradients are decode_linear_backward's."""
    dev, dt = x.device, x.dtype
    assert x.is_cuda and x.dim() == 2 and dt in _DTYPES
    B = x.shape[0]
    ldx = _rows(x, "x", B, N, dt, dev)
    _coded(bitstream, start_state, codebook, M, N, L, k, V, T, dt, dev)
    a, b = _vector(row_scale, "row_scale", M, dev), _vector(bias, "bias", M, dev)
    with _on(dev):
        y = torch.empty((B, M), dtype=dt, device=dev) if out is None else out
        ldy = M if out is None else _rows(out, "out", B, M, dt, dev)
        z = torch.empty((B, M), dtype=dt, device=dev) if pre else None
        if workspace is None:
            n = _lib.tcq_decode_linear_workspace_bytes(_DTYPES[dt], B, M, N, L, k, V, T)
            workspace = Workspace(n, dev) if n else None
        _lib.tcq_decode_linear(
            bitstream.data_ptr(), start_state.data_ptr(), codebook.data_ptr(), M, N, L, k, V, T,
            _DTYPES[dt], x.data_ptr(), B, ldx, a, b, _ACTS[act],
            None if residual is None else residual.data_ptr(),
            M if residual is None else _rows(residual, "residual", B, M, dt, dev),
            y.data_ptr(), ldy, None if z is None else z.data_ptr(), M,
            *_workspace(workspace, dev), _stream_of(dev))
    return y if z is None else (y, z)


@dataclass
class Packed:
    """An 8-bit checkpoint of a matrix [rows, cols] (see tcq_act_pack)."""
    codes: torch.Tensor  # int8 [rows, cols], rows contiguous
    scale: torch.Tensor  # uint8 [rows, ceil(cols / 32)]

    def check(self, name: str, rows: int, cols: int, device: torch.device) -> int:
        groups = -(-cols // CHECKPOINT_GROUP)
        assert self.scale.device == device and self.scale.dtype == torch.uint8 and \
            self.scale.shape == (rows, groups) and self.scale.is_contiguous(), \
            f"{name}: scale bytes [{rows}, {groups}]"
        return _rows(self.codes, name, rows, cols, torch.int8, device)


def act_pack(x: torch.Tensor) -> Packed:
    """8-bit checkpoint of x [rows, cols] (float32, float16 or bfloat16)."""
    assert x.is_cuda and x.dim() == 2 and x.dtype in _DTYPES
    rows, cols = x.shape
    ldx = _rows(x, "x", rows, cols, x.dtype, x.device)
    groups = -(-cols // CHECKPOINT_GROUP)
    with _on(x.device):
        # rows start on whole groups
        ldq = groups * CHECKPOINT_GROUP
        codes = torch.empty((rows, ldq), dtype=torch.int8, device=x.device)
        if ldq != cols:
            codes = codes[:, :cols]
        scale = torch.empty((rows, groups), dtype=torch.uint8, device=x.device)
        _lib.tcq_act_pack(x.data_ptr(), _DTYPES[x.dtype], rows, cols, ldx, codes.data_ptr(),
                          max(ldq, 1), scale.data_ptr(), _stream_of(x.device))
    return Packed(codes, scale)


def act_unpack(packed: Packed, dtype: torch.dtype) -> torch.Tensor:
    """The values a checkpoint stands for, [rows, cols] in float32, float16 or bfloat16."""
    assert packed.codes.is_cuda and packed.codes.dim() == 2 and dtype in _DTYPES
    rows, cols = packed.codes.shape
    dev = packed.codes.device
    ldq = packed.check("codes", rows, cols, dev)
    with _on(dev):
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
        _lib.tcq_act_unpack(packed.codes.data_ptr(), ldq, packed.scale.data_ptr(), rows, cols,
                            _DTYPES[dtype], out.data_ptr(), max(cols, 1), _stream_of(dev))
    return out


def decode_linear_backward(bitstream: torch.Tensor, start_state: torch.Tensor,
                           codebook: torch.Tensor, dy: torch.Tensor, M: int, N: int, L: int,
                           k: int, V: int, T: int, row_scale: torch.Tensor | None = None,
                           act: str = "none", z: Packed | None = None, x: Packed | None = None,
                           dx: bool = True, dbias: bool = True,
                           workspace: Workspace | None = None
                           ) -> tuple[torch.Tensor | None, torch.Tensor | None,
                                      torch.Tensor | None]:
    """Gradients (dx [B, N], dw [M, N], dbias [M]) of decode_linear from dy [B, M] and the
    checkpoints z of the pre-activation (needed unless act is "none") and x of the input
    (dw is computed where it is given).  dw is the gradient of W_hat; the residual's
    gradient is dy."""
    dev, dt = dy.device, dy.dtype
    assert dy.is_cuda and dy.dim() == 2 and dt in _DTYPES
    assert dx or dbias or x is not None, "no gradient is wanted"
    B = dy.shape[0]
    lddy = _rows(dy, "dy", B, M, dt, dev)
    if dx:
        _coded(bitstream, start_state, codebook, M, N, L, k, V, T, dt, dev)
    a = _vector(row_scale, "row_scale", M, dev)
    assert act == "none" or z is not None, "the slope of act needs the checkpoint of z"
    ldz = z.check("z", B, M, dev) if act != "none" else M
    ldx = x.check("x", B, N, dev) if x is not None else N
    with _on(dev):
        gx = torch.empty((B, N), dtype=dt, device=dev) if dx else None
        gw = torch.empty((M, N), dtype=dt, device=dev) if x is not None else None
        gb = torch.empty(M, dtype=torch.float32, device=dev) if dbias else None
        if workspace is None:
            n = _lib.tcq_decode_linear_backward_workspace_bytes(
                _DTYPES[dt], B, M, N, L, k, V, T, dx, x is not None, dbias)
            workspace = Workspace(n, dev) if n else None
        # an output of no elements has no address and nothing to be written
        empty = (gx is None or gx.numel() == 0) and (gw is None or gw.numel() == 0) and \
            (gb is None or gb.numel() == 0)
        if not empty:
            _lib.tcq_decode_linear_backward(
                bitstream.data_ptr() if dx else None, start_state.data_ptr() if dx else None,
                codebook.data_ptr() if dx else None, M, N, L, k, V, T, _DTYPES[dt],
                dy.data_ptr(), B, lddy, a, _ACTS[act],
                z.codes.data_ptr() if act != "none" else None, ldz,
                z.scale.data_ptr() if act != "none" else None,
                x.codes.data_ptr() if x is not None else None, ldx,
                x.scale.data_ptr() if x is not None else None,
                None if gx is None else gx.data_ptr(), N, None if gw is None else gw.data_ptr(),
                N, None if gb is None else gb.data_ptr(), *_workspace(workspace, dev),
                _stream_of(dev))
    return gx, gw, gb

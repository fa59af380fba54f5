"""Torch-facing convenience layer over the C ABI: allocates outputs and workspaces as
CUDA (HIP) tensors and calls the entry points on the current stream.  Only argument
marshalling happens here; every step of the path runs in the HIP kernels.  Autograd
records none of these calls: gradients come from the calls that compute them (bcjr_vjp,
gated_vjp, layer_norm_vjp, distill_topk, distill_topk_vjp).
"""
from __future__ import annotations

import torch

from . import _native as nat

CODES = {"1mad": nat.QTCQ_CODE_1MAD, "3inst": nat.QTCQ_CODE_3INST}


def xor_code(masks) -> int:
    """The XOR-Trellis palette code with parity masks (m0, m1, m2, m3): m0 and m1 pick the
    palette, m2 and m3 the branch shuffle; each an (L - 2)-bit history mask."""
    code = nat.qtcq_xor_code(*masks)
    if code == nat.QTCQ_CODE_INVALID:
        raise ValueError("XOR parity masks must fit in 14 bits")
    return code


def _code(code) -> int:
    """A code name ("1mad", "3inst"), ("xor", masks), or a qtcq_code descriptor."""
    if isinstance(code, str):
        return CODES[code]
    if isinstance(code, tuple) and len(code) == 2 and code[0] == "xor":
        return xor_code(code[1])
    return int(code)


def _stream(device: int | None = None) -> int:
    # the handle alone: building a torch Stream around it takes longer than the rest of a
    # small call's checks together
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None
                                              else device)


def _on_current_device(x: torch.Tensor, name: str) -> None:
    # the kernels run on the current device's current stream, and workspaces and outputs
    # are allocated there
    if x.device.index is not None and x.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, not on the current device cuda:%d"
                         % (name, x.device, torch.cuda.current_device()))


def _dev_f32(x: torch.Tensor, name: str) -> torch.Tensor:
    if not (x.is_cuda and x.dtype == torch.float32 and x.is_contiguous() and x.dim() == 2):
        raise ValueError("%s must be a contiguous 2-D float32 device tensor" % name)
    _on_current_device(x, name)
    return x


def _dev_workspace(ws, name: str = "workspace") -> int:
    """A caller-supplied device scratch tensor: contiguous and on the current device (the
    kernels write through its pointer).  Returns its size in bytes, whatever its dtype."""
    if not (isinstance(ws, torch.Tensor) and ws.is_cuda and ws.is_contiguous()):
        raise ValueError("%s must be a contiguous device tensor" % name)
    _on_current_device(ws, name)
    return ws.numel() * ws.element_size()


def _like_seq(x: torch.Tensor | None, seq: torch.Tensor, name: str) -> None:
    """An optional per-weight tensor (error weights, upstream gradient) shaped as seq."""
    if x is not None:
        _dev_f32(x, name)
        if x.shape != seq.shape:
            raise ValueError("%s must have the shape of seq" % name)


def _dev_words(bits: torch.Tensor, B: int, W: int) -> None:
    """Streams as the kernels read them: B rows of W contiguous 32-bit words."""
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.dtype in (torch.int32, torch.uint32) and tuple(bits.shape) == (B, W)):
        raise ValueError("bits must be a contiguous [%d][%d] 32-bit device tensor" % (B, W))
    _on_current_device(bits, "bits")


def _decode_inputs(bits, T, W, seq, weights, want_mse):
    B = bits.shape[0]
    if W < 0:
        raise ValueError("unsupported (L, k, T)")
    _dev_words(bits, B, W)
    if seq is not None:
        _dev_f32(seq, "seq")
        if tuple(seq.shape) != (B, T):
            raise ValueError("seq must be [B][T]")
        _like_seq(weights, seq, "weights")
    elif want_mse or weights is not None:
        raise ValueError("the MSE needs seq (and weights only come with seq)")
    return B


def bitstream_words(L: int = 16, k: int = 2, T: int = 256) -> int:
    return nat.qtcq_bitstream_words(L, k, T)


def code_table(code="1mad", L: int = 16) -> torch.Tensor:
    out = torch.empty(1 << L, dtype=torch.float32, device="cuda")
    nat.qtcq_code_table(_code(code), L, out.data_ptr(), _stream())
    return out


# Default workspace caps: a chunk of sequences is one launch, so the cap bounds HBM use
# while keeping each launch many workgroups deep (the 4096x4096 encode fits one chunk).
ENCODE_WS_CAP = 64 << 30
BCJR_WS_CAP = 16 << 30
VJP_WS_CAP = 32 << 30


def _chunk_bytes(B: int, per: int, max_bytes: int | None, seqs_per_wg: int = 1) -> int:
    """Workspace bytes for min(B, what max_bytes holds) sequences of `per` bytes.  A
    partial batch is rounded down to whole multiples of the device's CU count times the
    sequences one workgroup takes (two in the search once a chunk exceeds the CU count),
    so that no launch ends with a partly empty round of workgroups."""
    if max_bytes is None or B * per <= max_bytes:
        return max(1, B) * per
    n = max(1, max_bytes // per)
    cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    if n > cus * seqs_per_wg:
        n = n // (cus * seqs_per_wg) * (cus * seqs_per_wg)
    elif n > cus:
        n = n // cus * cus
    return n * per


def encode_workspace(B: int, T: int = 256, L: int = 16, k: int = 2,
                     max_bytes: int | None = ENCODE_WS_CAP) -> torch.Tensor:
    per = nat.qtcq_encode_workspace_bytes(1, T, L, k)
    return torch.empty(_chunk_bytes(B, per, max_bytes, 2), dtype=torch.uint8, device="cuda")


def bcjr_workspace(B: int, T: int = 256, L: int = 16, k: int = 2,
                   max_bytes: int | None = BCJR_WS_CAP) -> torch.Tensor:
    per = nat.qtcq_bcjr_workspace_bytes(1, T, L, k)
    return torch.empty(_chunk_bytes(B, per, max_bytes), dtype=torch.uint8, device="cuda")


def encode(seq: torch.Tensor, weights: torch.Tensor | None = None, L: int = 16, k: int = 2,
           code="1mad", want_states: bool = False, workspace: torch.Tensor | None = None):
    """Viterbi-encode [B][T] targets.  Returns (bits [B][W] int32 view of uint32 words,
    mse [B] float32, states [B][T] int32 view of uint32 or None)."""
    _dev_f32(seq, "seq")
    B, T = seq.shape
    _like_seq(weights, seq, "weights")
    W = nat.qtcq_bitstream_words(L, k, T)
    bits = torch.empty((B, W), dtype=torch.int32, device=seq.device)
    mse = torch.empty(B, dtype=torch.float32, device=seq.device)
    states = torch.empty((B, T), dtype=torch.int32, device=seq.device) if want_states else None
    if workspace is None:
        workspace = encode_workspace(B, T, L, k)
    ws_bytes = _dev_workspace(workspace)
    nat.qtcq_viterbi_encode(seq.data_ptr(), None if weights is None else weights.data_ptr(), B, T,
                            L, k, _code(code), bits.data_ptr(), mse.data_ptr(),
                            None if states is None else states.data_ptr(), workspace.data_ptr(),
                            ws_bytes, _stream())
    return bits, mse, states


def decode(bits: torch.Tensor, T: int, L: int = 16, k: int = 2, code="1mad",
           seq: torch.Tensor | None = None, weights: torch.Tensor | None = None,
           want_recon: bool = True, want_mse: bool = False):
    """Window-decode [B][W] streams.  Returns (recon [B][T] or None, mse [B] or None)."""
    B = _decode_inputs(bits, T, nat.qtcq_bitstream_words(L, k, T), seq, weights, want_mse)
    recon = torch.empty((B, T), dtype=torch.float32, device=bits.device) if want_recon else None
    mse = torch.empty(B, dtype=torch.float32, device=bits.device) if want_mse else None
    nat.qtcq_decode(bits.data_ptr(), B, T, L, k, _code(code),
                    None if recon is None else recon.data_ptr(),
                    None if seq is None else seq.data_ptr(),
                    None if weights is None else weights.data_ptr(),
                    None if mse is None else mse.data_ptr(), _stream())
    return recon, mse


def bcjr_soft(seq: torch.Tensor, temperature: float, weights: torch.Tensor | None = None,
              L: int = 16, k: int = 2, code="1mad", workspace: torch.Tensor | None = None):
    """BCJR soft codewords.  Returns (soft [B][T] float32, log_z [B] float32)."""
    _dev_f32(seq, "seq")
    _like_seq(weights, seq, "weights")
    B, T = seq.shape
    soft = torch.empty((B, T), dtype=torch.float32, device=seq.device)
    logz = torch.empty(B, dtype=torch.float32, device=seq.device)
    if workspace is None:
        workspace = bcjr_workspace(B, T, L, k)
    ws_bytes = _dev_workspace(workspace)
    nat.qtcq_bcjr_soft(seq.data_ptr(), None if weights is None else weights.data_ptr(), B, T, L, k,
                       _code(code), temperature, soft.data_ptr(), logz.data_ptr(),
                       workspace.data_ptr(), ws_bytes, _stream())
    return soft, logz


def bcjr_vjp_workspace(B: int, T: int = 256, L: int = 16, k: int = 2,
                       max_bytes: int | None = VJP_WS_CAP) -> torch.Tensor:
    per = nat.qtcq_bcjr_vjp_workspace_bytes(1, T, L, k)
    return torch.empty(_chunk_bytes(B, per, max_bytes), dtype=torch.uint8, device="cuda")


def bcjr_vjp(seq: torch.Tensor, temperature: float, grad_soft: torch.Tensor,
             weights: torch.Tensor | None = None, L: int = 16, k: int = 2, code="1mad",
             want_soft: bool = False, workspace: torch.Tensor | None = None):
    """Gradient of sum_t grad_soft[b][t] * soft[b][t] with respect to seq.  Returns
    (grad_seq [B][T] float32, soft [B][T] or None, log_z [B] or None)."""
    _dev_f32(seq, "seq")
    _like_seq(grad_soft, seq, "grad_soft")
    _like_seq(weights, seq, "weights")
    B, T = seq.shape
    grad = torch.empty((B, T), dtype=torch.float32, device=seq.device)
    soft = torch.empty((B, T), dtype=torch.float32, device=seq.device) if want_soft else None
    logz = torch.empty(B, dtype=torch.float32, device=seq.device) if want_soft else None
    if workspace is None:
        workspace = bcjr_vjp_workspace(B, T, L, k)
    ws_bytes = _dev_workspace(workspace)
    nat.qtcq_bcjr_vjp(seq.data_ptr(), None if weights is None else weights.data_ptr(), B, T, L, k,
                      _code(code), temperature, grad_soft.data_ptr(), grad.data_ptr(),
                      None if soft is None else soft.data_ptr(),
                      None if logz is None else logz.data_ptr(), workspace.data_ptr(),
                      ws_bytes, _stream())
    return grad, soft, logz


def tailbiting_words(L: int = 16, k: int = 2, T: int = 256) -> int:
    return nat.qtcq_tailbiting_words(L, k, T)


def tailbiting_workspace(B: int, T: int = 256, L: int = 16, k: int = 2,
                         max_bytes: int | None = ENCODE_WS_CAP) -> torch.Tensor:
    per = nat.qtcq_tailbiting_workspace_bytes(1, T, L, k)
    return torch.empty(_chunk_bytes(B, per, max_bytes, 2), dtype=torch.uint8, device="cuda")


def tailbiting_encode(seq: torch.Tensor, weights: torch.Tensor | None = None, L: int = 16,
                      k: int = 2, code="1mad", want_states: bool = False,
                      workspace: torch.Tensor | None = None):
    """Tail-biting encode (two searches per sequence) of [B][T] targets.  Returns
    (bits [B][ceil(kT/32)] int32 view of uint32 words, mse [B], states [B][T] or None)."""
    _dev_f32(seq, "seq")
    B, T = seq.shape
    _like_seq(weights, seq, "weights")
    W = nat.qtcq_tailbiting_words(L, k, T)
    if W < 0:
        raise ValueError("tail-biting needs k*T >= L")
    bits = torch.empty((B, W), dtype=torch.int32, device=seq.device)
    mse = torch.empty(B, dtype=torch.float32, device=seq.device)
    states = torch.empty((B, T), dtype=torch.int32, device=seq.device) if want_states else None
    if workspace is None:
        workspace = tailbiting_workspace(B, T, L, k)
    ws_bytes = _dev_workspace(workspace)
    nat.qtcq_tailbiting_encode(seq.data_ptr(), None if weights is None else weights.data_ptr(), B,
                               T, L, k, _code(code), bits.data_ptr(), mse.data_ptr(),
                               None if states is None else states.data_ptr(),
                               workspace.data_ptr(), ws_bytes, _stream())
    return bits, mse, states


def tailbiting_decode(bits: torch.Tensor, T: int, L: int = 16, k: int = 2, code="1mad",
                      seq: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                      want_recon: bool = True, want_mse: bool = False):
    """Cyclic window decode of [B][W] tail-biting streams.  Returns (recon or None,
    mse or None)."""
    B = _decode_inputs(bits, T, nat.qtcq_tailbiting_words(L, k, T), seq, weights, want_mse)
    recon = torch.empty((B, T), dtype=torch.float32, device=bits.device) if want_recon else None
    mse = torch.empty(B, dtype=torch.float32, device=bits.device) if want_mse else None
    nat.qtcq_tailbiting_decode(bits.data_ptr(), B, T, L, k, _code(code),
                               None if recon is None else recon.data_ptr(),
                               None if seq is None else seq.data_ptr(),
                               None if weights is None else weights.data_ptr(),
                               None if mse is None else mse.data_ptr(), _stream())
    return recon, mse


def decode_matvec(bits: torch.Tensor, M: int, N: int, x: torch.Tensor, L: int = 16, k: int = 2,
                  code="1mad", tailbiting: bool = False) -> torch.Tensor:
    """y [batch][M] = W x for the M x N matrix whose row-major 16x16 tiles are the
    T = 256 streams `bits` ([(M/16)(N/16)][W]); x [batch][N] (or [N]) float32 on device."""
    one = x.dim() == 1
    x2 = x.reshape(1, -1) if one else x
    _dev_f32(x2, "x")
    if x2.shape[1] != N:
        raise ValueError("x must have N columns")
    W = tailbiting_words(L, k, 256) if tailbiting else bitstream_words(L, k, 256)
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.numel() == (M // 16) * (N // 16) * W):
        raise ValueError("bits must hold (M/16)*(N/16) contiguous streams of %d words" % W)
    _on_current_device(bits, "bits")
    y = torch.empty((x2.shape[0], M), dtype=torch.float32, device=x.device)
    nat.qtcq_decode_matvec(bits.data_ptr(), M, N, L, k, _code(code), tailbiting, x2.data_ptr(),
                           x2.shape[0], y.data_ptr(), _stream())
    return y[0] if one else y


def matvec_mfma_workspace(N: int) -> torch.Tensor:
    """Device scratch for decode_matvec_mfma over N columns (reusable across calls on one
    stream)."""
    n = nat.qtcq_decode_matvec_mfma_workspace_bytes(N)
    if n == 0:
        raise ValueError("N must be a multiple of 16 in [0, 2^22]")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def decode_matvec_mfma(bits: torch.Tensor, M: int, N: int, x: torch.Tensor, L: int = 16,
                       k: int = 2, code="1mad", tailbiting: bool = False,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """decode_matvec with the products on the matrix cores: the code values (exact in fp16)
    times x split per 32-column block into two scaled fp16 parts.  Same arguments and
    result layout, with up to 32 rows of x; `workspace` (matvec_mfma_workspace(N)) is
    allocated when not given."""
    one = x.dim() == 1
    x2 = x.reshape(1, -1) if one else x
    _dev_f32(x2, "x")
    if x2.shape[1] != N:
        raise ValueError("x must have N columns")
    W = tailbiting_words(L, k, 256) if tailbiting else bitstream_words(L, k, 256)
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.numel() == (M // 16) * (N // 16) * W):
        raise ValueError("bits must hold (M/16)*(N/16) contiguous streams of %d words" % W)
    _on_current_device(bits, "bits")
    if workspace is None:
        workspace = matvec_mfma_workspace(N)
    ws_bytes = _dev_workspace(workspace)
    y = torch.empty((x2.shape[0], M), dtype=torch.float32, device=x.device)
    nat.qtcq_decode_matvec_mfma(bits.data_ptr(), M, N, L, k, _code(code), tailbiting,
                                x2.data_ptr(), x2.shape[0], y.data_ptr(), workspace.data_ptr(),
                                ws_bytes, _stream())
    return y[0] if one else y


class SplitX:
    """The split of x made by matvec_mfma_split_x: the device workspace holding it and the
    (N, batch) it was made for.  The product reads the fragments and block scales at
    offsets that depend on both, so decode_matvec_mfma_presplit checks them."""
    __slots__ = ("workspace", "N", "batch")

    def __init__(self, workspace: torch.Tensor, N: int, batch: int):
        self.workspace, self.N, self.batch = workspace, N, batch


def matvec_mfma_split_x(x: torch.Tensor, workspace: torch.Tensor | None = None) -> SplitX:
    """The split of x [batch][N] (or [N]) for decode_matvec_mfma_presplit, written into
    `workspace` (matvec_mfma_workspace(N), allocated when not given)."""
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    _dev_f32(x2, "x")
    N = x2.shape[1]
    if workspace is None:
        workspace = matvec_mfma_workspace(N)
    ws_bytes = _dev_workspace(workspace)
    nat.qtcq_matvec_mfma_split_x(x2.data_ptr(), N, x2.shape[0], workspace.data_ptr(), ws_bytes,
                                 _stream())
    return SplitX(workspace, N, x2.shape[0])


def decode_matvec_mfma_presplit(bits: torch.Tensor, M: int, N: int, split: SplitX,
                                L: int = 16, k: int = 2, code="1mad",
                                tailbiting: bool = False) -> torch.Tensor:
    """y [split.batch][M] = W x from a split made by matvec_mfma_split_x for this N (equal to
    decode_matvec_mfma bit for bit)."""
    if not isinstance(split, SplitX):
        raise ValueError("split must be the SplitX that matvec_mfma_split_x returned")
    if split.N != N:
        raise ValueError("split was made for N = %d, not %d" % (split.N, N))
    W = tailbiting_words(L, k, 256) if tailbiting else bitstream_words(L, k, 256)
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.numel() == (M // 16) * (N // 16) * W):
        raise ValueError("bits must hold (M/16)*(N/16) contiguous streams of %d words" % W)
    _on_current_device(bits, "bits")
    sp_bytes = _dev_workspace(split.workspace, "split")
    y = torch.empty((split.batch, M), dtype=torch.float32, device=bits.device)
    nat.qtcq_decode_matvec_mfma_presplit(bits.data_ptr(), M, N, L, k, _code(code), tailbiting,
                                         split.workspace.data_ptr(), sp_bytes, split.batch,
                                         y.data_ptr(), _stream())
    return y


def decode_matvec_mfma_noalloc(bits: torch.Tensor, M: int, N: int, x: torch.Tensor,
                               out: torch.Tensor, L: int = 16, k: int = 2, code="1mad",
                               tailbiting: bool = False) -> torch.Tensor:
    """decode_matvec_mfma with the split x in the library's per-device scratch array: no
    workspace, and nothing allocated here either -- the caller passes the output `out`
    ([batch][M] float32, or [M] for a 1-D x).  Calls that overlap on one GPU race."""
    one = x.dim() == 1
    x2 = x.reshape(1, -1) if one else x
    _dev_f32(x2, "x")
    if x2.shape[1] != N:
        raise ValueError("x must have N columns")
    W = tailbiting_words(L, k, 256) if tailbiting else bitstream_words(L, k, 256)
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.numel() == (M // 16) * (N // 16) * W):
        raise ValueError("bits must hold (M/16)*(N/16) contiguous streams of %d words" % W)
    _on_current_device(bits, "bits")
    o2 = out.reshape(1, -1) if one else out
    _dev_f32(o2, "out")
    if tuple(o2.shape) != (x2.shape[0], M):
        raise ValueError("out must be [batch][M]")
    nat.qtcq_decode_matvec_mfma_noalloc(bits.data_ptr(), M, N, L, k, _code(code), tailbiting,
                                        x2.data_ptr(), x2.shape[0], o2.data_ptr(), _stream())
    return out


# ---- dense operators around the codec --------------------------------------------------

DTYPES = {torch.float32: nat.QTCQ_F32, torch.bfloat16: nat.QTCQ_BF16, torch.float16: nat.QTCQ_F16,
          torch.int8: nat.QTCQ_I8}
ACTIVATIONS = {"silu": nat.QTCQ_ACT_SILU, "gelu": nat.QTCQ_ACT_GELU,
               "gelu_tanh": nat.QTCQ_ACT_GELU_TANH, "relu": nat.QTCQ_ACT_RELU,
               "sigmoid": nat.QTCQ_ACT_SIGMOID}


def _rows(x: torch.Tensor, name: str, dtypes, device: int, shape=None) -> int:
    """A 2-D tensor on the current device (its index: device) of rows that do not overlap,
    each contiguous (a slice of columns of a wider matrix too).  Returns its row stride."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2 and x.dtype in dtypes):
        raise ValueError("%s must be a 2-D device tensor of %s"
                         % (name, " or ".join(str(d) for d in dtypes)))
    if x.get_device() != device:
        _on_current_device(x, name)
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError("%s must be %s" % (name, list(shape)))
    cols = x.shape[1]
    if x.is_contiguous():
        return cols
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if x.shape[0] == 1:
        return cols
    if x.stride(0) < cols:
        raise ValueError("the rows of %s overlap" % name)
    return x.stride(0)


def _scales(s: torch.Tensor, name: str, n: int, device: int) -> None:
    if not (isinstance(s, torch.Tensor) and s.is_cuda and s.dtype == torch.float32
            and s.dim() == 1 and s.shape[0] == n and s.is_contiguous()):
        raise ValueError("%s must be a contiguous float32 device tensor of %d values" % (name, n))
    if s.get_device() != device:
        _on_current_device(s, name)


def _whole_rows(pointers: int, cols: int, size: int, *strides: int) -> bool:
    """Whether the kernels can read operands of `cols` columns in 16-byte chunks where they
    are (otherwise the workspace holds padded copies): their pointers ORed together, the
    bytes of an element, their row strides."""
    for ld in strides:
        cols |= ld
        if ld * size > 1 << 22:
            return False
    return (pointers | cols * size) & 15 == 0


def _workspace(workspace, nbytes: int, like: torch.Tensor):
    """(pointer or None, bytes) of a workspace, allocated when not given and needed; the
    tensor comes along so that it lives until the call."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = like.new_empty(nbytes, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), nbytes
    return workspace, workspace.data_ptr(), _dev_workspace(workspace)


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(ACTIVATIONS))
    return ACTIVATIONS[name]


def quantize_rows(x: torch.Tensor):
    """Rows of x ([R][C] float32, bfloat16 or float16) to 8-bit integers with one scale a
    row.  Returns (q [R][C] int8, scale [R] float32); x is about q * scale[:, None]."""
    dev = torch.cuda.current_device()
    ldx = _rows(x, "x", (torch.float32, torch.bfloat16, torch.float16), dev)
    R, C = x.shape
    q = torch.empty_like(x, dtype=torch.int8, memory_format=torch.contiguous_format)
    scale = x.new_empty(R, dtype=torch.float32)
    nat.qtcq_quantize_rows(x.data_ptr(), DTYPES[x.dtype], R, C, ldx, q.data_ptr(), C,
                           scale.data_ptr(), _stream(dev))
    return q, scale


def decode_matrix(bits: torch.Tensor, M: int, N: int, L: int = 16, k: int = 2, code="1mad",
                  tailbiting: bool = False, dtype: torch.dtype = torch.int8):
    """The M x N matrix whose row-major 16x16 tiles are the T = 256 streams `bits`
    ([(M/16)(N/16)][W]) as rows.  Returns (w [M][N] int8, scale [M] float32) for
    torch.int8, or w [M][N] in float32, bfloat16 or float16."""
    if dtype not in DTYPES:
        raise ValueError("dtype must be int8, float32, bfloat16 or float16")
    if M < 0 or N < 0 or M % 16 or N % 16:
        raise ValueError("M and N must be multiples of 16")
    W = tailbiting_words(L, k, 256) if tailbiting else bitstream_words(L, k, 256)
    if not (bits.is_cuda and bits.is_contiguous() and bits.element_size() == 4
            and bits.numel() == (M // 16) * (N // 16) * W):
        raise ValueError("bits must hold (M/16)*(N/16) contiguous streams of %d words" % W)
    _on_current_device(bits, "bits")
    w = bits.new_empty((M, N), dtype=dtype)
    scale = bits.new_empty(M, dtype=torch.float32) if dtype == torch.int8 else None
    nat.qtcq_decode_matrix(bits.data_ptr(), M, N, L, k, _code(code), tailbiting, DTYPES[dtype],
                           w.data_ptr(), N, None if scale is None else scale.data_ptr(), _stream())
    return w if scale is None else (w, scale)


def matmul_int8_workspace(M: int, N: int, K: int, whole_rows: bool = False) -> torch.Tensor:
    """Device scratch for matmul_int8 (reusable across calls on one stream).  whole_rows:
    the rows of a and w start on 16 bytes and are a multiple of 16 bytes long."""
    return torch.empty(nat.qtcq_matmul_int8_workspace_bytes(M, N, K, whole_rows),
                       dtype=torch.uint8, device="cuda")


def matmul_int8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                dtype: torch.dtype = torch.float32,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y [M][N] = (a w^T) a_scale[:, None] w_scale for a [M][K] and w [N][K] int8: exact
    integer sums, then a scale for each token and each channel.  dtype float32, bfloat16
    or float16; `workspace` (matmul_int8_workspace(M, N, K)) is allocated when not given
    and needed."""
    if dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError("dtype must be float32, bfloat16 or float16")
    dev = torch.cuda.current_device()
    lda = _rows(a, "a", (torch.int8,), dev)
    ldw = _rows(w, "w", (torch.int8,), dev)
    (M, K), N = a.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w must have the columns of a")
    _scales(a_scale, "a_scale", M, dev)
    _scales(w_scale, "w_scale", N, dev)
    ap, wp = a.data_ptr(), w.data_ptr()
    need = nat.qtcq_matmul_int8_workspace_bytes(M, N, K, _whole_rows(ap | wp, K, 1, lda, ldw))
    _keep, ws, ws_bytes = _workspace(workspace, need, a)
    y = a.new_empty((M, N), dtype=dtype)
    nat.qtcq_matmul_int8(ap, lda, a_scale.data_ptr(), wp, ldw, w_scale.data_ptr(), M, N, K,
                         DTYPES[dtype], y.data_ptr(), N, ws, ws_bytes, _stream(dev))
    return y


def _gated_inputs(x, w_gate, w_up, dev):
    """(ldx, ldw, whether x, w_gate and w_up are whole 16-byte chunks)"""
    ldx = _rows(x, "x", (torch.bfloat16, torch.float16), dev)
    ldw = _rows(w_gate, "w_gate", (x.dtype,), dev)
    if w_gate.shape[1] != x.shape[1]:
        raise ValueError("w_gate must have the columns of x")
    if _rows(w_up, "w_up", (x.dtype,), dev, w_gate.shape) != ldw:
        raise ValueError("w_up must have the row stride of w_gate")
    return ldx, ldw, _whole_rows(x.data_ptr() | w_gate.data_ptr() | w_up.data_ptr(), x.shape[1], 2,
                                 ldx, ldw)


def gated_workspace(M: int, F: int, K: int, whole_rows: bool = False) -> torch.Tensor:
    """Device scratch for gated (reusable across calls on one stream).  whole_rows: the rows
    of x, w_gate and w_up start on 16 bytes and are a multiple of 16 bytes long."""
    return torch.empty(nat.qtcq_gated_workspace_bytes(M, F, K, whole_rows), dtype=torch.uint8,
                       device="cuda")


def gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
          save: bool = False, workspace: torch.Tensor | None = None):
    """h [M][F] = act(x w_gate^T) * (x w_up^T) for x [M][K] and w_gate, w_up [F][K], all
    bfloat16 or all float16.  With save, returns (h, gate, up): the two projections too,
    for gated_vjp.  `workspace` (gated_workspace(M, F, K)) is allocated when not given and
    needed.  Autograd does not see the call, so inputs that require gradients are refused
    while it records (torch.no_grad() or detached inputs, and gated_vjp for the gradients)."""
    act = _activation(activation)
    dev = torch.cuda.current_device()
    ldx, ldw, whole = _gated_inputs(x, w_gate, w_up, dev)
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        raise ValueError("gated does not record gradients: call it under torch.no_grad() or with "
                         "detached inputs, and gated_vjp for the gradients")
    (M, K), F = x.shape, w_gate.shape[0]
    need = nat.qtcq_gated_workspace_bytes(M, F, K, whole)
    _keep, ws, ws_bytes = _workspace(workspace, need, x)
    h = x.new_empty((M, F))
    gate, up = (torch.empty_like(h), torch.empty_like(h)) if save else (None, None)
    nat.qtcq_gated_forward(x.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), ldw,
                           DTYPES[x.dtype], M, F, K, act, h.data_ptr(), F,
                           gate.data_ptr() if save else None, up.data_ptr() if save else None, F,
                           ws, ws_bytes, _stream(dev))
    return (h, gate, up) if save else h


def gated_vjp_workspace(M: int, F: int, K: int, whole_rows: bool = False) -> torch.Tensor:
    """Device scratch for gated_vjp (reusable across calls on one stream); whole_rows as
    gated_workspace."""
    return torch.empty(nat.qtcq_gated_vjp_workspace_bytes(M, F, K, whole_rows),
                       dtype=torch.uint8, device="cuda")


def gated_vjp(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, gate: torch.Tensor,
              up: torch.Tensor, grad_h: torch.Tensor, activation: str = "silu",
              want_x: bool = True, want_w: bool = True, workspace: torch.Tensor | None = None,
              round_slopes: bool = False):
    """Gradients of sum(grad_h * h) for h of gated(x, w_gate, w_up), with the gate and up
    that it saved.  Returns (grad_x [M][K], grad_w_gate [F][K], grad_w_up [F][K]), None
    where not wanted; `workspace` (gated_vjp_workspace(M, F, K)) is allocated when not
    given.  round_slopes: the gradients of the two projections are rounded to the type of x
    ahead of the products, which halves their work and adds about as much error as the
    rounding of the results."""
    act = _activation(activation) | (nat.QTCQ_ACT_ROUND_SLOPES if round_slopes else 0)
    dev = torch.cuda.current_device()
    ldx, ldw, whole = _gated_inputs(x, w_gate, w_up, dev)
    (M, K), F = x.shape, w_gate.shape[0]
    ldg = _rows(gate, "gate", (x.dtype,), dev, (M, F))
    if _rows(up, "up", (x.dtype,), dev, (M, F)) != ldg:
        raise ValueError("up must have the row stride of gate")
    ldgh = _rows(grad_h, "grad_h", (x.dtype,), dev, (M, F))
    need = nat.qtcq_gated_vjp_workspace_bytes(M, F, K, whole)
    _keep, ws, ws_bytes = _workspace(workspace, need, x)
    grad_x = x.new_empty((M, K)) if want_x else None
    grad_wg, grad_wu = (x.new_empty((F, K)), x.new_empty((F, K))) if want_w else (None, None)
    nat.qtcq_gated_vjp(x.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), ldw, gate.data_ptr(),
                       up.data_ptr(), ldg, grad_h.data_ptr(), ldgh, DTYPES[x.dtype], M, F, K, act,
                       None if grad_x is None else grad_x.data_ptr(), K,
                       None if grad_wg is None else grad_wg.data_ptr(),
                       None if grad_wu is None else grad_wu.data_ptr(), K, ws, ws_bytes,
                       _stream(dev))
    return grad_x, grad_wg, grad_wu


# ---- model operators on coded weights ---------------------------------------------------

FLOATS = (torch.float32, torch.bfloat16, torch.float16)


def _not_recorded(name: str) -> None:
    """For a call with inputs that require gradients: autograd does not see it, so it is refused
    while autograd records (in a backward pass too, if that is to be differentiated again)."""
    if torch.is_grad_enabled():
        raise ValueError("%s does not record gradients: call it under torch.no_grad() or with detached "
                         "inputs (gradients come from the calls that compute them)" % name)


def _grad(x) -> bool:
    return x is not None and x.requires_grad


def _vector(x, name: str, dtypes, n: int, device: int):
    """An optional contiguous device vector of n values: its pointer, or None."""
    if x is None:
        return None
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in dtypes
            and x.shape == (n,) and x.is_contiguous()):
        raise ValueError("%s must be a contiguous device tensor of %d values in %s"
                         % (name, n, " or ".join(str(d) for d in dtypes)))
    if x.get_device() != device:
        _on_current_device(x, name)
    return x.data_ptr()


def _result_rows(x: torch.Tensor) -> torch.Tensor:
    """Contiguous rows for a result of the shape and dtype of x."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _block_scales(s: torch.Tensor, name: str, shape, device: int):
    """A matrix of block scales with any strides, broadcast ones too.  Returns both strides."""
    if not (isinstance(s, torch.Tensor) and s.is_cuda and s.dtype == torch.float32
            and s.shape == shape):
        raise ValueError("%s must be a float32 device tensor of %s" % (name, list(shape)))
    if s.get_device() != device:
        _on_current_device(s, name)
    row, col = s.stride()
    return row if shape[0] > 1 else 0, col if shape[1] > 1 else 0


def quantize_blocks(x: torch.Tensor, block_rows: int = 1):
    """Rows of x ([R][C] float32, bfloat16 or float16) to 8-bit floating point with a float32
    scale for each block: block_rows = 1, of 128 columns of a row (activations), block_rows =
    128, of 128 x 128 elements (weights).  Returns (q [R][C] float8_e4m3fn, scale
    [R or ceil(R / 128)][ceil(C / 128)]); x is about q times its block's scale.  The scales
    of rows lie together (scale.t() is contiguous), as matmul_fp8 reads them fastest."""
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    dev = torch.cuda.current_device()
    ldx = _rows(x, "x", FLOATS, dev)
    if x.requires_grad:
        _not_recorded("quantize_blocks")
    R, C = x.shape
    q = x.new_empty((R, C), dtype=torch.float8_e4m3fn)
    down = R if block_rows == 1 else (R + 127) // 128
    scale = x.new_empty_strided((down, (C + 127) // 128), (1, down), dtype=torch.float32)
    nat.qtcq_quantize_blocks(x.data_ptr(), DTYPES[x.dtype], R, C, ldx, block_rows, q.data_ptr(), C,
                             scale.data_ptr(), 1, down, _stream(dev))
    return q, scale


def matmul_fp8_workspace(M: int, N: int, K: int, whole_rows: bool = False) -> torch.Tensor:
    """Device scratch for matmul_fp8 (reusable across calls on one stream).  whole_rows:
    the rows of a and w start on 16 bytes and are a multiple of 16 bytes long."""
    return torch.empty(nat.qtcq_matmul_fp8_workspace_bytes(M, N, K, whole_rows),
                       dtype=torch.uint8, device="cuda")


def matmul_fp8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
               dtype: torch.dtype = torch.float32,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y [M][N] = a w^T for a [M][K] and w [N][K] float8_e4m3fn with the scales of
    quantize_blocks: a_scale [M][ceil(K / 128)] (block_rows = 1) and w_scale [ceil(N / 128)]
    [ceil(K / 128)] (block_rows = 128), with any strides (of rows up to 2^20).  Sums in
    float32; dtype float32, bfloat16 or float16.  16-bit results of more than a few rows come
    from the 8-bit matrix instruction, which cuts each product off at 2^-13 of the largest power
    of two among its 8 neighbours of k (1.4e-5 of the results' norm on values of a Gaussian);
    float32 results, which may be rounded afterwards, have exact products.  `workspace`
    (matmul_fp8_workspace(M, N, K)) is allocated when not given and needed."""
    if dtype not in FLOATS:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    dev = torch.cuda.current_device()
    lda = _rows(a, "a", (torch.float8_e4m3fn,), dev)
    ldw = _rows(w, "w", (torch.float8_e4m3fn,), dev)
    (M, K), N = a.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError("w must have the columns of a")
    kb = (K + 127) // 128
    as_row, as_col = _block_scales(a_scale, "a_scale", (M, kb), dev)
    ws_row, ws_col = _block_scales(w_scale, "w_scale", ((N + 127) // 128, kb), dev)
    if a.requires_grad or a_scale.requires_grad or w.requires_grad or w_scale.requires_grad:
        _not_recorded("matmul_fp8")
    ap, wp = a.data_ptr(), w.data_ptr()
    need = nat.qtcq_matmul_fp8_workspace_bytes(M, N, K, _whole_rows(ap | wp, K, 1, lda, ldw))
    _keep, ws, ws_bytes = _workspace(workspace, need, a)
    y = a.new_empty((M, N), dtype=dtype)
    nat.qtcq_matmul_fp8(ap, lda, a_scale.data_ptr(), as_row, as_col, wp, ldw, w_scale.data_ptr(),
                        ws_row, ws_col, M, N, K, DTYPES[dtype], y.data_ptr(), N, ws, ws_bytes,
                        _stream(dev))
    return y


def _norm_weights(x, weight, bias, dev):
    """(pointers of weight and bias, their dtype): float32 or the dtype of x, both the same."""
    given = bias if weight is None else weight
    dtype = given.dtype if isinstance(given, torch.Tensor) else x.dtype
    kinds = (dtype,) if dtype in (torch.float32, x.dtype) else (torch.float32, x.dtype)
    return (_vector(weight, "weight", kinds, x.shape[1], dev),
            _vector(bias, "bias", kinds, x.shape[1], dev), dtype)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5, save: bool = False):
    """y = (x - mean) rstd weight + bias over the columns of x ([R][C] float32, bfloat16 or
    float16), with the mean of each row and rstd = 1 / sqrt(its variance + eps), in float32.
    weight and bias [C] are float32 or of the dtype of x (None: ones, zeros).  With save,
    returns (y, mean [R], rstd [R]) for layer_norm_vjp."""
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    dev = torch.cuda.current_device()
    ldx = _rows(x, "x", FLOATS, dev)
    wp, bp, wt = _norm_weights(x, weight, bias, dev)
    if x.requires_grad or _grad(weight) or _grad(bias):
        _not_recorded("layer_norm")
    R, C = x.shape
    y = _result_rows(x)
    mean = x.new_empty(R, dtype=torch.float32) if save else None
    rstd = torch.empty_like(mean) if save else None
    nat.qtcq_layer_norm(x.data_ptr(), DTYPES[x.dtype], R, C, ldx, wp, bp, DTYPES[wt], eps,
                        y.data_ptr(), C, mean.data_ptr() if save else None,
                        rstd.data_ptr() if save else None, _stream(dev))
    return (y, mean, rstd) if save else y


def layer_norm_vjp_workspace(R: int, C: int) -> torch.Tensor:
    """Device scratch for layer_norm_vjp (reusable across calls on one stream)."""
    return torch.empty(nat.qtcq_layer_norm_vjp_workspace_bytes(R, C), dtype=torch.uint8,
                       device="cuda")


def layer_norm_vjp(x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                   rstd: torch.Tensor, grad_y: torch.Tensor, want_x: bool = True,
                   want_w: bool = True, workspace: torch.Tensor | None = None,
                   weight_dtype: torch.dtype | None = None):
    """Gradients of sum(grad_y * y) for y of layer_norm(x, weight, bias), with the mean and
    rstd that it saved.  Returns (grad_x [R][C], grad_weight [C], grad_bias [C]), None where
    not wanted; the last two in the dtype of weight.  Where weight is None, in weight_dtype:
    float32 or the dtype of x, which it is when not given (a bias alone may be either).
    `workspace` (layer_norm_vjp_workspace(R, C)) is allocated when not given and needed."""
    dev = torch.cuda.current_device()
    ldx = _rows(x, "x", FLOATS, dev)
    ldgy = _rows(grad_y, "grad_y", (x.dtype,), dev, x.shape)
    wp, _, wt = _norm_weights(x, weight, None, dev)
    if weight_dtype is not None:
        if weight_dtype not in ((torch.float32, x.dtype) if weight is None else (wt,)):
            raise ValueError("weight_dtype must be the dtype of weight, or without one float32 or "
                             "the dtype of x")
        wt = weight_dtype
    R, C = x.shape
    mp = _vector(mean, "mean", (torch.float32,), R, dev)
    rp = _vector(rstd, "rstd", (torch.float32,), R, dev)
    if mp is None or rp is None:
        raise ValueError("mean and rstd are those that layer_norm saved")
    if x.requires_grad or grad_y.requires_grad or mean.requires_grad or rstd.requires_grad or _grad(weight):
        _not_recorded("layer_norm_vjp")
    need = nat.qtcq_layer_norm_vjp_workspace_bytes(R, C) if want_w else 0
    _keep, ws, ws_bytes = _workspace(workspace, need, x)
    grad_x = _result_rows(x) if want_x else None
    grad_w = grad_b = None
    if want_w:
        grad_w = x.new_empty(C, dtype=wt) if weight is None else torch.empty_like(weight)
        grad_b = torch.empty_like(grad_w)
    nat.qtcq_layer_norm_vjp(x.data_ptr(), DTYPES[x.dtype], R, C, ldx, wp, DTYPES[wt], mp, rp,
                            grad_y.data_ptr(), ldgy, grad_x.data_ptr() if want_x else None, C,
                            grad_w.data_ptr() if want_w else None,
                            grad_b.data_ptr() if want_w else None, ws, ws_bytes, _stream(dev))
    return grad_x, grad_w, grad_b


def _distill_inputs(logits, index, teacher, temperature, dev):
    """(row strides of logits, index and teacher)"""
    if not 2.0 ** -100 <= temperature <= 2.0 ** 100:
        raise ValueError("temperature must be positive, from 2^-100 to 2^100")
    ldl = _rows(logits, "logits", FLOATS, dev)
    ldi = _rows(index, "index", (torch.int64, torch.int32), dev)
    if index.shape[0] != logits.shape[0]:
        raise ValueError("index must have the rows of logits")
    return ldl, ldi, _rows(teacher, "teacher", FLOATS, dev, index.shape)


def distill_topk_workspace(R: int, V: int) -> torch.Tensor:
    """Device scratch for distill_topk (reusable across calls on one stream)."""
    return torch.empty(nat.qtcq_distill_topk_workspace_bytes(R, V), dtype=torch.uint8, device="cuda")


def distill_topk(logits: torch.Tensor, index: torch.Tensor, teacher: torch.Tensor,
                 temperature: float = 1.0, teacher_log_z: torch.Tensor | None = None,
                 grad_loss: torch.Tensor | None = None, save: bool = False,
                 workspace: torch.Tensor | None = None):
    """loss [R] = sum_j p_j (log p_j - log q[index_j]) of each row of logits ([R][V] float32,
    bfloat16 or float16), q = softmax(logits / temperature) and p = softmax(teacher /
    temperature) over the teacher's top logits [R][k] at the vocabulary entries index [R][k]
    (int64 or int32; one outside 0 .. V - 1 is padding; k at most 1024).  With teacher_log_z
    [R] (float32), p = exp(teacher / temperature - teacher_log_z): the teacher's probabilities
    over its whole vocabulary.

    With grad_loss [R] (float32: what each loss weighs in the total, 0 for tokens without
    one), returns (loss, grad_logits): the gradient of sum(grad_loss * loss) in the same pass.
    Otherwise, with save, returns (loss, stats) for distill_topk_vjp.  `workspace`
    (distill_topk_workspace(R, V)) is allocated when not given and needed."""
    if grad_loss is not None and save:
        raise ValueError("save is for distill_topk_vjp: not with grad_loss")
    dev = torch.cuda.current_device()
    ldl, ldi, ldt = _distill_inputs(logits, index, teacher, temperature, dev)
    (R, V), k = logits.shape, index.shape[1]
    zp = _vector(teacher_log_z, "teacher_log_z", (torch.float32,), R, dev)
    gp = _vector(grad_loss, "grad_loss", (torch.float32,), R, dev)
    if logits.requires_grad or teacher.requires_grad or _grad(teacher_log_z) or _grad(grad_loss):
        _not_recorded("distill_topk")
    _keep, ws, ws_bytes = _workspace(workspace, nat.qtcq_distill_topk_workspace_bytes(R, V), logits)
    loss = logits.new_empty(R, dtype=torch.float32)
    stats = logits.new_empty((R, 5), dtype=torch.float32) if save else None
    grad = _result_rows(logits) if grad_loss is not None else None
    nat.qtcq_distill_topk(logits.data_ptr(), DTYPES[logits.dtype], R, V, ldl, index.data_ptr(),
                          index.element_size(), ldi, teacher.data_ptr(), DTYPES[teacher.dtype], ldt,
                          k, temperature, zp, loss.data_ptr(), stats.data_ptr() if save else None,
                          gp, grad.data_ptr() if grad is not None else None, V, ws, ws_bytes,
                          _stream(dev))
    return (loss, stats) if save else loss if grad is None else (loss, grad)


def distill_topk_vjp(logits: torch.Tensor, index: torch.Tensor, teacher: torch.Tensor,
                     stats: torch.Tensor, grad_loss: torch.Tensor,
                     temperature: float = 1.0) -> torch.Tensor:
    """The gradient of sum(grad_loss * loss) with respect to the logits, for the loss of
    distill_topk and the stats that it saved for the same inputs: for a grad_loss [R]
    (float32) that is known only after the losses."""
    dev = torch.cuda.current_device()
    ldl, ldi, ldt = _distill_inputs(logits, index, teacher, temperature, dev)
    (R, V), k = logits.shape, index.shape[1]
    gp = _vector(grad_loss, "grad_loss", (torch.float32,), R, dev)
    if gp is None or not (isinstance(stats, torch.Tensor) and stats.shape == (R, 5)
                          and stats.is_contiguous()):
        raise ValueError("stats are those that distill_topk saved, grad_loss a value a row")
    sp = _vector(stats.view(-1), "stats", (torch.float32,), R * 5, dev)
    if logits.requires_grad or teacher.requires_grad or stats.requires_grad or grad_loss.requires_grad:
        _not_recorded("distill_topk_vjp")
    grad = _result_rows(logits)
    nat.qtcq_distill_topk_vjp(logits.data_ptr(), DTYPES[logits.dtype], R, V, ldl, index.data_ptr(),
                              index.element_size(), ldi, teacher.data_ptr(), DTYPES[teacher.dtype],
                              ldt, k, temperature, sp, gp, grad.data_ptr(), V, _stream(dev))
    return grad

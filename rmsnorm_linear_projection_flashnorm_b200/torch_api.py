"""torch-facing conveniences over the C ABI: allocate outputs and workspaces
with torch (device memory is torch's job here) and call the library.  No
arithmetic of the method happens in Python."""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import (FN_T_BF16, FN_T_FP16, FN_T_FP32, FN_W_BF16, FN_W_FP8_E4M3_B128, FN_W_MXFP8_E4M3, check, fn_adaln_shift_bias, fn_norm_proj_adaln,
               fn_norm_proj_swiglu_nvfp4_swizzled, fn_workspace_size_adaln, fn_fold_weights, fn_norm_proj, fn_norm_proj_swiglu,
               fn_norm_proj_partial, fn_norm_proj_swiglu_nvfp4, fn_post_scale, fn_query_device_status,
               fn_workspace_size, fn_workspace_size_moe, fn_workspace_size_proj, lib)


def weight_type(Wp: torch.Tensor, scales: Optional[torch.Tensor]) -> int:
    """The fn_wtype of a folded weight: bf16, e4m3 with fp32 block scales, or
    MXFP8 (e4m3 with ue8m0 scale bytes)."""
    if Wp.dtype == torch.bfloat16:
        return FN_W_BF16
    return FN_W_MXFP8_E4M3 if scales is not None and scales.dtype == torch.uint8 else FN_W_FP8_E4M3_B128


def fold(W0: torch.Tensor, g: torch.Tensor, W1: Optional[torch.Tensor] = None, wtype: int = FN_W_BF16,
         stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Fold g into W0 (and W1 for SwiGLU); returns (W', scales or None)."""
    d, N = W0.shape
    ncols = 2 * N if W1 is not None else N
    dev = W0.device
    if wtype == FN_W_BF16:
        Wp = torch.empty((d, ncols), dtype=torch.bfloat16, device=dev)
        scales = None
    elif wtype == FN_W_MXFP8_E4M3:
        Wp = torch.empty((d, ncols), dtype=torch.uint8, device=dev)
        scales = torch.empty(d * ncols // 32, dtype=torch.uint8, device=dev)   # chunked ue8m0 bytes
    else:
        Wp = torch.empty((d, ncols), dtype=torch.uint8, device=dev)
        scales = torch.empty((d // 128, ncols // 128), dtype=torch.float32, device=dev)
    check(fn_fold_weights(W0, W1, g, d, N, wtype, Wp, scales, stream), "fn_fold_weights")
    return Wp, scales


def _capturing(device) -> bool:
    return torch.device(device).type == "cuda" and torch.cuda.is_current_stream_capturing()


class Workspace:
    """A zero-initialised device workspace that grows on demand.

    A captured graph keeps the address it was captured with, so buffers that a
    larger one has replaced live as long as the workspace (each is at least
    twice the one before, so all of them together are less than twice the last).
    While the current stream is being captured the workspace does not grow: a
    call that needs more gets a zeroed buffer of its own, which belongs to the
    graph and is zeroed at every replay.  One call of the largest size before
    the capture saves that, and puts its status word where `status` reads it."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = torch.zeros(256, dtype=torch.uint8, device=device)
        self._replaced = []

    def get(self, M: int, d: int, N: int, wt: int, swiglu: bool) -> torch.Tensor:
        return self.reserve(fn_workspace_size(M, d, N, wt, int(swiglu)))

    def reserve(self, need: int) -> torch.Tensor:
        have = self.buf.numel()
        if have < need:
            if _capturing(self.device):
                return torch.zeros(need, dtype=torch.uint8, device=self.device)
            self._replaced.append(self.buf)
            self.buf = torch.zeros(max(need, 2 * have), dtype=torch.uint8, device=self.device)
        return self.buf

    def status(self, stream=None):
        return fn_query_device_status(self.buf, stream)


def norm_proj(x: torch.Tensor, Wp: torch.Tensor, N: int, eps: float, swiglu: bool = False,
              scales: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = RMSNorm(x) @ W through the fused kernels (W' already folded)."""
    M, d = x.shape
    wt = weight_type(Wp, scales)
    if ws is None:
        ws = Workspace(x.device)
    buf = ws.get(M, d, N, wt, swiglu)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    fn = fn_norm_proj_swiglu if swiglu else fn_norm_proj
    check(fn(x, M, d, Wp, scales, wt, N, eps, out, buf, buf.numel(), stream), fn.__name__)
    return out


def norm_proj_swiglu_nvfp4(x: torch.Tensor, Wp: torch.Tensor, N: int, eps: float, global_scale: torch.Tensor,
                           scales: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
                           out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """SwiGLU output in NVFP4: (codes uint8 [M, N/2], e4m3 scale bytes uint8
    [M, N/16]); global_scale is a one-element fp32 device tensor."""
    M, d = x.shape
    wt = weight_type(Wp, scales)
    if ws is None:
        ws = Workspace(x.device)
    buf = ws.get(M, d, N, wt, True)
    if out is None:
        out = (torch.empty((M, N // 2), dtype=torch.uint8, device=x.device),
               torch.empty((M, N // 16), dtype=torch.uint8, device=x.device))
    q, sf = out
    check(fn_norm_proj_swiglu_nvfp4(x, M, d, Wp, scales, wt, N, eps, global_scale, q, sf, buf, buf.numel(), stream),
          "fn_norm_proj_swiglu_nvfp4")
    return q, sf


def norm_proj_swiglu_nvfp4_swizzled(x: torch.Tensor, Wp: torch.Tensor, N: int, eps: float,
                                    global_scale: torch.Tensor, scales: Optional[torch.Tensor] = None,
                                    ws: Optional[Workspace] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """SwiGLU output in NVFP4 with the scale bytes in the chunked (swizzled)
    layout: (codes uint8 [M, N/2], scale bytes uint8 [ceil(M/128)*128 * N/16],
    zero-initialised so the padding rows read as 0)."""
    M, d = x.shape
    wt = weight_type(Wp, scales)
    if ws is None:
        ws = Workspace(x.device)
    buf = ws.get(M, d, N, wt, True)
    q = torch.empty((M, N // 2), dtype=torch.uint8, device=x.device)
    sf = torch.zeros(((M + 127) // 128) * 128 * (N // 16), dtype=torch.uint8, device=x.device)
    check(fn_norm_proj_swiglu_nvfp4_swizzled(x, M, d, Wp, scales, wt, N, eps, global_scale, q, sf, buf, buf.numel(),
                                             stream), "fn_norm_proj_swiglu_nvfp4_swizzled")
    return q, sf


def norm_proj_partial(x: torch.Tensor, Wp: torch.Tensor, ncols: int, scales: Optional[torch.Tensor] = None,
                      ws: Optional[Workspace] = None, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """One rank's share of a row-parallel projection: fp32 [M * ncols + M]
    (unscaled x @ Wp in stored column order, then the rows' sums of squares)."""
    M, d = x.shape
    wt = weight_type(Wp, scales)
    if ws is None:
        ws = Workspace(x.device)
    buf = ws.get(M, d, ncols, wt, False)
    if out is None:
        out = torch.empty(M * ncols + M, dtype=torch.float32, device=x.device)
    check(fn_norm_proj_partial(x, M, d, Wp, scales, wt, ncols, out, buf, buf.numel(), stream), "fn_norm_proj_partial")
    return out


def post_scale(partial: torch.Tensor, M: int, N: int, d_total: int, eps: float, swiglu: bool = False,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 [M, N] from a summed partial buffer (see fn_post_scale)."""
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=partial.device)
    check(fn_post_scale(partial, M, N, int(swiglu), d_total, eps, out, stream), "fn_post_scale")
    return out


def adaln_shift_bias(shift: torch.Tensor, W0: torch.Tensor, W1: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """fp32 [n_cond, ncols]: the AdaLN shift rows through the unfolded weight."""
    n_cond, d = shift.shape
    N = W0.shape[1]
    ncols = 2 * N if W1 is not None else N
    B = torch.empty((n_cond, ncols), dtype=torch.float32, device=shift.device)
    check(fn_adaln_shift_bias(shift, n_cond, W0, W1, d, N, B, stream), "fn_adaln_shift_bias")
    return B


def norm_proj_adaln(x: torch.Tensor, Wp: torch.Tensor, N: int, eps: float, adaln_scale: torch.Tensor,
                    shift_bias: torch.Tensor, adaln_index: torch.Tensor, swiglu: bool = False,
                    scales: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The AdaLN-modulated fused call (see fn_norm_proj_adaln)."""
    M, d = x.shape
    wt = weight_type(Wp, scales)
    if ws is None:
        ws = Workspace(x.device)
    buf = ws.reserve(fn_workspace_size_adaln(d, N, wt, int(swiglu)))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    check(fn_norm_proj_adaln(x, M, d, Wp, scales, wt, N, int(swiglu), eps, adaln_scale, shift_bias, adaln_index,
                             adaln_scale.shape[0], out, buf, buf.numel(), stream), "fn_norm_proj_adaln")
    return out


# --------------------------------------------------------------------------
# operators next to the fused projections
# --------------------------------------------------------------------------
_DTYPE = {torch.bfloat16: FN_T_BF16, torch.float16: FN_T_FP16, torch.float32: FN_T_FP32}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# The checks below run on every call of a decode step: each is one condition,
# and the message is put together only when it fails.
def _rows(t: torch.Tensor, name: str, dtypes, shape=None) -> int:
    """Check a matrix with contiguous rows; returns its row stride."""
    if t.dim() != 2 or t.dtype not in dtypes:
        raise ValueError(f"{name}: a matrix of {[str(d) for d in dtypes]} is needed")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name}: shape {(rows, cols)}, expected {shape}")
    ld, inner = t.stride()
    if inner != 1 and cols != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # a single row has no stride of its own; overlapping rows are refused by the library
    return ld if rows > 1 else max(ld, cols)


def _vec(t: Optional[torch.Tensor], name: str, dtype, n: int, dev) -> None:
    if t is not None and (t.dtype != dtype or t.shape != (n,) or not t.is_contiguous() or t.device != dev):
        raise ValueError(f"{name}: a contiguous {dtype} vector of {n} on {dev} is needed")


def _dense(t: Optional[torch.Tensor], name: str, dtype, shape, dev) -> None:
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != dev):
        raise ValueError(f"{name}: contiguous {dtype} {shape} on {dev} is needed")


class _Elsewhere:
    """Another device than the current one, or a stream of the caller's
    (torch.cuda.Stream or a raw handle): what is allocated or zeroed inside
    belongs to that stream, as under torch.cuda.stream."""

    def __init__(self, dev: torch.device, stream):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        self.parts = [torch.cuda.device(dev)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for part in self.parts:
            part.__enter__()

    def __exit__(self, *exc):
        for part in reversed(self.parts):
            part.__exit__(*exc)


def _elsewhere(dev: torch.device, stream) -> Optional[_Elsewhere]:
    """None where the tensors' device is the current one and its current stream
    is meant; else what to switch to (the callers then call themselves inside)."""
    if dev.type != "cuda":
        raise ValueError(f"tensors on {dev}: a CUDA device is needed")
    if stream is None and dev.index == torch.cuda.current_device():
        return None
    return _Elsewhere(dev, stream)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _handle(dev: torch.device) -> int:
    """The device's current stream, without the Stream object around it."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _workspace(ws: Optional[Workspace], dev: torch.device, need: int) -> torch.Tensor:
    """The caller's workspace, grown to `need` bytes, or one for this call."""
    if ws is None:
        return torch.zeros(need, dtype=torch.uint8, device=dev)
    buf = ws.reserve(need)
    if buf.device != dev:
        raise ValueError(f"workspace on {buf.device}, tensors on {dev}")
    return buf


_ACT = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_BF16 = (torch.bfloat16,)
_BF16_FP32 = (torch.bfloat16, torch.float32)


def proj(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
         residual: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None, out: Optional[torch.Tensor] = None,
         out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """act(x @ W + bias) + residual (see fn_proj): x bf16 [M, K], W bf16 [K, N],
    bias fp32 [N]; the output is bf16 or fp32, the type of `out`, else
    `out_dtype`, else the residual's, else bf16.  `out` may be the residual."""
    ldx = _rows(x, "x", _BF16)
    ldw = _rows(W, "W", _BF16)
    M, K = x.shape
    KW, N = W.shape
    dev = x.device
    if KW != K:
        raise ValueError(f"W: {K} rows are needed")
    if act not in _ACT:
        raise ValueError(f"act: one of {list(_ACT)}")
    _vec(bias, "bias", torch.float32, N, dev)
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return proj(x, W, bias, act, residual, ws, out, out_dtype)
    if out is None:
        dt = out_dtype or (residual.dtype if residual is not None else torch.bfloat16)
        out = torch.empty(M, N, dtype=dt, device=dev)
    ldy = _rows(out, "out", _BF16_FP32, (M, N))
    if residual is None:
        ldr = 0
    elif residual is out:
        ldr = ldy
    else:
        ldr = _rows(residual, "residual", (out.dtype,), (M, N))
    if W.device != dev or out.device != dev or (residual is not None and residual.device != dev):
        raise ValueError(f"every tensor must be on {dev}")
    # a single row's stride is free: the library wants multiples of 8
    if M <= 1:
        ldx = (ldx + 7) // 8 * 8
    if K == 1:
        ldw = (ldw + 7) // 8 * 8
    buf = _workspace(ws, dev, fn_workspace_size_proj(M, K, N))
    check(lib().fn_proj(x.data_ptr(), ldx, M, K, W.data_ptr(), ldw, N, _at(bias), _ACT[act], _at(residual), ldr,
                        _DTYPE[out.dtype], out.data_ptr(), ldy, buf.data_ptr(), buf.numel(), _handle(dev)), "fn_proj")
    return out


_SCORE = {"softmax": 0, "sigmoid": 1}


def fold_experts(W_gate: torch.Tensor, g: torch.Tensor, W_up: torch.Tensor, stream=None) -> torch.Tensor:
    """Fold the norm gain into every expert's gate and up weights [E, d, I]:
    bf16 [E, d, 2I], per expert the interleaved layout of `fold`."""
    _need(W_gate.dim() == 3, "W_gate [E, d, I] is needed")
    E, d, N = W_gate.shape
    dev = W_gate.device
    _dense(W_gate, "W_gate", torch.bfloat16, (E, d, N), dev)
    _dense(W_up, "W_up", torch.bfloat16, (E, d, N), dev)
    _vec(g, "g", torch.float32, d, dev)
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return fold_experts(W_gate, g, W_up)
    out = torch.empty((E, d, 2 * N), dtype=torch.bfloat16, device=dev)
    for e in range(E):
        check(fn_fold_weights(W_gate[e], W_up[e], g, d, N, FN_W_BF16, out[e], None, _handle(dev)), "fn_fold_weights")
    return out


def moe_swiglu(x: torch.Tensor, g: Optional[torch.Tensor], router: torch.Tensor, Wgu: torch.Tensor, Wd: torch.Tensor,
               top_k: int, eps: float, score: str = "softmax", select_bias: Optional[torch.Tensor] = None,
               renorm: bool = True, route_scale: float = 1.0, residual: Optional[torch.Tensor] = None,
               ws: Optional[Workspace] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A mixture-of-experts layer for at most 64 tokens (see fn_moe_swiglu):
    (y bf16 [M, d], expert ids int32 [M, top_k], routing weights fp32 [M, top_k]).
    Wgu [E, d, 2I] from `fold_experts`; `out` may be x or the residual."""
    dev = x.device
    if x.dim() != 2 or Wd.dim() != 3:
        raise ValueError("x [M, d], Wgu [E, d, 2I], Wd [E, I, d] are needed")
    M, d = x.shape
    E, I, _ = Wd.shape
    if score not in _SCORE:
        raise ValueError(f"score: one of {list(_SCORE)}")
    if not 0 < top_k <= E:
        raise ValueError(f"top_k: 1..{E}")
    bf = torch.bfloat16
    _dense(x, "x", bf, (M, d), dev)
    _dense(router, "router", bf, (E, d), dev)
    _dense(Wgu, "Wgu", bf, (E, d, 2 * I), dev)
    _dense(Wd, "Wd", bf, (E, I, d), dev)
    _dense(residual, "residual", bf, (M, d), dev)
    _dense(out, "out", bf, (M, d), dev)
    _vec(g, "g", torch.float32, d, dev)
    _vec(select_bias, "select_bias", torch.float32, E, dev)
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return moe_swiglu(x, g, router, Wgu, Wd, top_k, eps, score, select_bias, renorm, route_scale, residual, ws,
                              out)
    if out is None:
        out = torch.empty(M, d, dtype=bf, device=dev)
    ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
    w = torch.empty(M, top_k, dtype=torch.float32, device=dev)
    buf = _workspace(ws, dev, fn_workspace_size_moe(M, d, I, E, top_k))
    check(lib().fn_moe_swiglu(x.data_ptr(), M, d, _at(g), router.data_ptr(), E, Wgu.data_ptr(), Wd.data_ptr(), I, top_k,
                              _SCORE[score], _at(select_bias), 1 if renorm else 0, route_scale, eps, _at(residual),
                              out.data_ptr(), ids.data_ptr(), w.data_ptr(), buf.data_ptr(), buf.numel(), _handle(dev)),
          "fn_moe_swiglu")
    return out, ids, w


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]      # fp32 [M] (None without targets)
    entropy: torch.Tensor                # fp32 [M]
    lse: torch.Tensor                    # fp32 [M]
    top_ids: torch.Tensor                # int32 [M, top_k]
    top_logprobs: torch.Tensor           # fp32 [M, top_k]


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top_k: int = 0, scale: float = 1.0,
                   out: Optional[TokenLogprobs] = None, stream=None) -> TokenLogprobs:
    """Log probabilities of the int32 `targets` [M] under softmax(scale * logits),
    the rows' entropies and log sums, and the top_k alternatives (see
    fn_token_logprobs).  logits: bf16, fp16 or fp32 [M, V], rows contiguous.
    Not recorded by autograd: token_logprobs_backward gives the gradient."""
    ld = _rows(logits, "logits", _DTYPE)
    M, V = logits.shape
    dev = logits.device
    _vec(targets, "targets", torch.int32, M, dev)
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return token_logprobs(logits, targets, top_k, scale, out)
    if out is None:
        lp, ent, lse = torch.empty(3, M, dtype=torch.float32, device=dev).unbind()
        ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
        top = torch.empty(M, top_k, dtype=torch.float32, device=dev)
        if targets is None:
            lp = None
        out = TokenLogprobs(lp, ent, lse, ids, top)
    else:
        lp, ent, lse, ids, top = out
        _vec(lp, "logprob", torch.float32, M, dev)
        _vec(ent, "entropy", torch.float32, M, dev)
        _vec(lse, "lse", torch.float32, M, dev)
        _dense(ids, "top_ids", torch.int32, (M, top_k), dev)
        _dense(top, "top_logprobs", torch.float32, (M, top_k), dev)
    check(lib().fn_token_logprobs(logits.data_ptr(), _DTYPE[logits.dtype], M, V, ld, _at(targets), scale, top_k,
                                  _at(lp), _at(ent), _at(lse), _at(ids) if top_k else None,
                                  _at(top) if top_k else None, _handle(dev)), "fn_token_logprobs")
    return out


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor], lse: torch.Tensor,
                            entropy: Optional[torch.Tensor], grad_logprob: Optional[torch.Tensor],
                            grad_entropy: Optional[torch.Tensor] = None, scale: float = 1.0,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of token_logprobs' logprob and entropy with respect to the
    logits (see fn_token_logprobs_backward); `out` may be the logits."""
    ld = _rows(logits, "logits", _DTYPE)
    M, V = logits.shape
    dev = logits.device
    _vec(targets, "targets", torch.int32, M, dev)
    _vec(lse, "lse", torch.float32, M, dev)
    _vec(entropy, "entropy", torch.float32, M, dev)
    _vec(grad_logprob, "grad_logprob", torch.float32, M, dev)
    _vec(grad_entropy, "grad_entropy", torch.float32, M, dev)
    other = _elsewhere(dev, stream)
    if other is not None:
        with other:
            return token_logprobs_backward(logits, targets, lse, entropy, grad_logprob, grad_entropy, scale, out)
    if out is None:
        out = torch.empty(M, V, dtype=logits.dtype, device=dev)
    ldd = _rows(out, "out", (logits.dtype,), (M, V))
    if out.device != dev:
        raise ValueError(f"out on {out.device}, logits on {dev}")
    check(lib().fn_token_logprobs_backward(logits.data_ptr(), _DTYPE[logits.dtype], M, V, ld, _at(targets),
                                           lse.data_ptr(), _at(entropy), _at(grad_logprob), _at(grad_entropy), scale,
                                           out.data_ptr(), ldd, _handle(dev)), "fn_token_logprobs_backward")
    return out

"""MI355X (gfx950) sigmoid top-K routed MoE layer with Exact Quantile Balancing.

Thin binding over the C ABI of libmoe_mi355x.so (include/moe_mi355x.h):
``route``, ``eqb_bias`` and ``forward`` marshal torch tensors (device memory
and the current stream) into the library calls; every step of the layer runs
in the library's HIP kernels.  There is no CPU fallback: a missing library or
a non-GPU tensor raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
from dataclasses import dataclass, replace
from typing import Optional

from . import _lib
from ._lib import (MOE_KEY32, MOE_PACKED_GATEUP, MOE_RECOMPUTE_BIAS, MOE_ROUTE_FUSED, MoeAux,
                   MoeError,
                   MoeFp8Weights, MoeGrads, MoeProblem, MoeWeights)

__all__ = ["route", "eqb_bias", "eqb_workspace_bytes", "EqbState", "eqb_bias_parts",
           "route_stats", "read_route_stats", "lei_backward", "forward",
           "forward_workspace_bytes", "fp8_quantize_blocks", "fp8_quantize_rows",
           "Fp8ExpertWeights", "quantize_experts", "forward_fp8", "forward_fp8_workspace_bytes",
           "ExpertWeights", "MoeError", "load_library", "stage_timing", "stage_times",
           "forward_noalloc", "pack_gateup", "pack_gateup_weights", "rms_norm",
           "rms_norm_backward", "balance_loss", "balance_loss_backward", "backward",
           "backward_workspace_bytes"]

AUX_FIELDS = [f for f, _ in MoeAux._fields_]


def load_library():
    return _lib.load()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(t, name, dtype=None, shape=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU torch tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _stream(stream):
    torch = _torch()
    if stream is None:
        # the handle of torch.cuda.current_stream() without its object (0.5 us a
        # call instead of 2.9, of the 13 that a small call takes on the host);
        # not a public name of torch's, so it may be missing
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return C.c_void_p(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _on(stream):
    """Allocation context of a call: with an explicit stream, the outputs and
    temporaries of the call are allocated on that stream, so torch's caching
    allocator does not hand their memory to other work before the call's
    kernels on that stream are done."""
    torch = _torch()
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _on_device(t, stream):
    """_on(stream) with the device of t as the current one, for the calls that
    take tensors of another device than the current."""
    torch = _torch()
    if t.device.index == torch.cuda.current_device():
        return _on(stream)
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(t.device))
    ctx.enter_context(_on(stream))
    return ctx


def _one_device(first, **others):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


@functools.lru_cache(maxsize=None)
def _bf16():
    torch = _torch()
    return (torch.bfloat16, torch.uint16, torch.int16)


def route(logits, K: int, beta=None, stream=None):
    """Top-K selection on logits + beta, sigmoid weights of the unbiased
    logits.  Returns (ids int32 [N,K], weights fp32 [N,K], alpha fp32 [N],
    margin fp32 [N])."""
    torch = _torch()
    lib = _lib.load()
    logits = _dev(logits, "logits", torch.float32)
    N, E = logits.shape
    beta = _dev(beta, "beta", torch.float32, (E,))
    with _on(stream):
        dev = logits.device
        ids = torch.empty((N, K), dtype=torch.int32, device=dev)
        w = torch.empty((N, K), dtype=torch.float32, device=dev)
        alpha = torch.empty((N,), dtype=torch.float32, device=dev)
        margin = torch.empty((N,), dtype=torch.float32, device=dev)
        _lib.check(lib.moe_route(_ptr(logits), _ptr(beta), N, E, K, _ptr(ids), _ptr(w),
                                 _ptr(alpha), _ptr(margin), _stream(stream)))
    return ids, w, alpha, margin


def route_stats(topk_ids, E: int, topk_ids_unbiased=None, margin=None, tau: float = 1e-3,
                stream=None):
    """Routing diagnostics on the device (moe_route_stats): returns
    (counts [E] int32, stats) where stats is a 40-byte device tensor holding a
    moe_route_stats_t; read_route_stats(stats) copies it to a dict."""
    torch = _torch()
    lib = _lib.load()
    topk_ids = _dev(topk_ids, "topk_ids", torch.int32)
    N, K = topk_ids.shape
    topk_ids_unbiased = _dev(topk_ids_unbiased, "topk_ids_unbiased", torch.int32, (N, K))
    margin = _dev(margin, "margin", torch.float32, (N,))
    with _on(stream):
        counts = torch.empty((E,), dtype=torch.int32, device=topk_ids.device)
        stats = torch.empty((C.sizeof(_lib.MoeRouteStats) // 8,), dtype=torch.float64,
                            device=topk_ids.device)
        _lib.check(lib.moe_route_stats(_ptr(topk_ids), _ptr(topk_ids_unbiased), _ptr(margin), N, E,
                                       K, float(tau), _ptr(counts), _ptr(stats), _stream(stream)))
    return counts, stats


def read_route_stats(stats) -> dict:
    """Copy a moe_route_stats_t from the device (synchronises) into a dict."""
    raw = stats.cpu().numpy().tobytes()
    st = _lib.MoeRouteStats.from_buffer_copy(raw)
    return {f: getattr(st, f) for f, _ in _lib.MoeRouteStats._fields_}


def lei_backward(topk_ids, E: int, logits=None, grad_scores=None, lam: float = 1e-5,
                 tau: float = 1.0, scores_out: bool = True, logits_out: bool = True,
                 inplace: bool = False, stream=None):
    """Load-Error Injection on the score gradient of one microbatch
    (moe_lei_backward).  Returns (grad_scores' [N,E] or None,
    grad_logits [N,E] or None, injection [E]).  With inplace=True the
    injection is added into grad_scores itself."""
    torch = _torch()
    lib = _lib.load()
    topk_ids = _dev(topk_ids, "topk_ids", torch.int32)
    N, K = topk_ids.shape
    logits = _dev(logits, "logits", torch.float32, (N, E))
    grad_scores = _dev(grad_scores, "grad_scores", torch.float32, (N, E))
    with _on(stream):
        dev_ = topk_ids.device
        if inplace:
            if grad_scores is None:
                raise ValueError("inplace needs grad_scores")
            gout = grad_scores
        else:
            gout = torch.empty((N, E), dtype=torch.float32, device=dev_) if scores_out else None
        dz = torch.empty((N, E), dtype=torch.float32, device=dev_) if logits_out else None
        inj = torch.empty((E,), dtype=torch.float32, device=dev_)
        need = int(lib.moe_lei_workspace_bytes(E))
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev_)
        _lib.check(lib.moe_lei_backward(_ptr(logits), _ptr(topk_ids), _ptr(grad_scores), N, E, K,
                                        float(lam), float(tau), _ptr(gout), _ptr(dz), _ptr(inj),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    return gout, dz, inj


def eqb_workspace_bytes(N: int, E: int, key_bits: int = 16) -> int:
    return int(_lib.load().moe_eqb_workspace_bytes(N, E, key_bits))


def eqb_bias(logits, K: int, beta_in=None, alpha=None, key_bits: int = 16,
             workspace=None, stream=None):
    """One exact Quantile Balancing update.  Returns (beta_out [E],
    quantile [E]) in fp32."""
    torch = _torch()
    lib = _lib.load()
    logits = _dev(logits, "logits", torch.float32)
    N, E = logits.shape
    beta_in = _dev(beta_in, "beta_in", torch.float32, (E,))
    alpha = _dev(alpha, "alpha", torch.float32, (N,))
    with _on(stream):
        need = int(lib.moe_eqb_workspace_bytes(N, E, key_bits))
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=logits.device)
        beta_out = torch.empty((E,), dtype=torch.float32, device=logits.device)
        q = torch.empty((E,), dtype=torch.float32, device=logits.device)
        _lib.check(lib.moe_eqb_bias(_ptr(logits), _ptr(beta_in), _ptr(alpha), N, E, K, key_bits,
                                    _ptr(beta_out), _ptr(q), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))
    return beta_out, q


class EqbState:
    """Exact quantile update over a batch that arrives in parts
    (moe_eqb_begin / moe_eqb_accumulate / moe_eqb_select).  Owns the device
    state buffer; use: ``st = EqbState(E, K, n_total)``, then for every pass
    ``st.accumulate(pass_, Z_part, alpha_part)`` over all parts and
    ``st.select(pass_)``; the last select returns (beta_out, quantile)."""

    def __init__(self, E: int, K: int, n_total: int, key_bits: int = 16, device=None,
                 stream=None):
        torch = _torch()
        self.lib = _lib.load()
        self.E, self.K, self.n_total, self.key_bits = E, K, n_total, key_bits
        self.passes = key_bits // 8
        self.stream = stream
        nbytes = int(self.lib.moe_eqb_state_bytes(E, key_bits))
        if nbytes == 0:
            raise ValueError(f"unsupported E={E} / key_bits={key_bits}")
        self.state = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
        _lib.check(self.lib.moe_eqb_begin(E, key_bits, _ptr(self.state), nbytes,
                                          _stream(stream)))

    def accumulate(self, pass_: int, logits, alpha):
        torch = _torch()
        logits = _dev(logits, "logits", torch.float32)
        N, E = logits.shape
        if E != self.E:
            raise ValueError(f"logits have E={E}, state has E={self.E}")
        alpha = _dev(alpha, "alpha", torch.float32, (N,))
        _lib.check(self.lib.moe_eqb_accumulate(pass_, _ptr(logits), _ptr(alpha), N, E,
                                               self.key_bits, _ptr(self.state),
                                               self.state.numel(), _stream(self.stream)))

    def select(self, pass_: int):
        torch = _torch()
        last = pass_ == self.passes - 1
        beta = torch.empty((self.E,), dtype=torch.float32, device=self.state.device) if last else None
        q = torch.empty((self.E,), dtype=torch.float32, device=self.state.device) if last else None
        _lib.check(self.lib.moe_eqb_select(pass_, self.n_total, self.E, self.K, self.key_bits,
                                           _ptr(beta), _ptr(q), _ptr(self.state),
                                           self.state.numel(), _stream(self.stream)))
        return (beta, q) if last else None


def eqb_bias_parts(logits_parts, alpha_parts, K: int, key_bits: int = 16, stream=None):
    """moe_eqb_bias over the concatenation of the parts, computed part by part
    (histograms summed over the parts for every radix pass).  Returns
    (beta_out [E], quantile [E])."""
    n_total = sum(int(z.shape[0]) for z in logits_parts)
    E = int(logits_parts[0].shape[1])
    st = EqbState(E, K, n_total, key_bits, device=logits_parts[0].device, stream=stream)
    out = None
    for p in range(st.passes):
        for z, a in zip(logits_parts, alpha_parts):
            st.accumulate(p, z, a)
        out = st.select(p)
    return out


@dataclass
class ExpertWeights:
    """bf16 weights of one MoE layer (torch tensors on the GPU)."""
    w_router: object        # [E, d]
    w_gate: object          # [E, h, d]
    w_up: object            # [E, h, d]
    w_down: object          # [E, d, h]
    ws_gate: object = None  # [S, hs, d]
    ws_up: object = None    # [S, hs, d]
    ws_down: object = None  # [S, d, hs]
    packed: bool = False    # w_gate, w_up as [E, d/64, h, 64] (pack_gateup)


def _problem(N, d, E, K, h, n_shared, h_shared, flags, logit_offset, logits_in):
    return MoeProblem(N, d, E, K, h, n_shared, h_shared, flags,
                      _ptr(logit_offset), _ptr(logits_in))


def forward_workspace_bytes(N, d, E, K, h, n_shared=1, h_shared=None,
                            recompute_bias=False, key_bits=16) -> int:
    flags = (MOE_RECOMPUTE_BIAS if recompute_bias else 0) | (MOE_KEY32 if key_bits == 32 else 0)
    p = _problem(N, d, E, K, h, n_shared, h_shared or h, flags, None, None)
    return int(_lib.load().moe_forward_workspace_bytes(C.byref(p)))


def forward_fp8_workspace_bytes(N, d, E, K, h, n_shared=1, h_shared=None,
                                recompute_bias=False, key_bits=16) -> int:
    flags = (MOE_RECOMPUTE_BIAS if recompute_bias else 0) | (MOE_KEY32 if key_bits == 32 else 0)
    p = _problem(N, d, E, K, h, n_shared, h_shared or h, flags, None, None)
    return int(_lib.load().moe_forward_fp8_workspace_bytes(C.byref(p)))


def pack_gateup_weights(w, stream=None):
    """moe_pack_gateup_weights: bf16 [count, rows, cols] (cols % 64 == 0) ->
    [count, cols/64, rows, 64], out[c, k, r, j] = w[c, r, 64k + j]."""
    torch = _torch()
    w = _dev(w, "w", _bf16())
    if w.dim() != 3:
        raise ValueError("w must be [count, rows, cols]")
    cnt, R, Cc = w.shape
    with _on(stream):
        out = torch.empty((cnt, Cc // 64, R, 64), dtype=torch.bfloat16, device=w.device)
        _lib.check(_lib.load().moe_pack_gateup_weights(_ptr(w), cnt, R, Cc, _ptr(out),
                                                       _stream(stream)))
    return out


def pack_gateup(weights, stream=None):
    """The same layer (ExpertWeights or Fp8ExpertWeights) with its routed
    gate and up weights packed k-block-major (MOE_PACKED_GATEUP); forward()
    and forward_fp8() give bit-identical results with either form.  E4M3
    codes are packed as 16-bit words, so each row's 128-code k-blocks stay
    whole: [E, h, d] -> [E, d/128, h, 128]."""
    if weights.packed:
        return weights
    if isinstance(weights, Fp8ExpertWeights):
        torch = _torch()

        def pack_codes(c):
            c = _dev(c, "codes", torch.uint8)
            return pack_gateup_weights(c.view(torch.bfloat16), stream).view(torch.uint8)
        return replace(weights, w_gate=pack_codes(weights.w_gate),
                       w_up=pack_codes(weights.w_up), packed=True)
    return replace(weights, w_gate=pack_gateup_weights(weights.w_gate, stream),
                   w_up=pack_gateup_weights(weights.w_up, stream), packed=True)


def fp8_quantize_blocks(w, stream=None):
    """bf16 [count, R, C] (or [R, C]) -> (E4M3 codes uint8 of the same shape,
    fp32 scales [count, ceil(R/128), ceil(C/128)] (or without count)), one
    scale per 128 x 128 block."""
    torch = _torch()
    w = _dev(w, "w", _bf16())
    squeeze = w.dim() == 2
    w3 = w.unsqueeze(0) if squeeze else w
    if w3.dim() != 3:
        raise ValueError("w must be [R, C] or [count, R, C]")
    cnt, R, Cc = w3.shape
    with _on(stream):
        codes = torch.empty((cnt, R, Cc), dtype=torch.uint8, device=w.device)
        scales = torch.empty((cnt, (R + 127) // 128, (Cc + 127) // 128), dtype=torch.float32,
                             device=w.device)
        _lib.check(_lib.load().moe_fp8_quantize_blocks(_ptr(w3), cnt, R, Cc, _ptr(codes),
                                                       _ptr(scales), _stream(stream)))
    return (codes[0], scales[0]) if squeeze else (codes, scales)


def fp8_quantize_rows(x, stream=None):
    """bf16 rows [n, C] (C % 128 == 0) -> (codes uint8 [n, C], fp32 scales
    [n, C/128]), one scale per 1 x 128 group."""
    torch = _torch()
    x = _dev(x, "x", _bf16())
    n, Cc = x.shape
    with _on(stream):
        codes = torch.empty((n, Cc), dtype=torch.uint8, device=x.device)
        scales = torch.empty((n, Cc // 128), dtype=torch.float32, device=x.device)
        _lib.check(_lib.load().moe_fp8_quantize_rows(_ptr(x), n, Cc, _ptr(codes), _ptr(scales),
                                                     _stream(stream)))
    return codes, scales


@dataclass
class Fp8ExpertWeights:
    """E4M3 expert weights with 128 x 128 block scales (torch tensors on the
    GPU); the router stays bf16."""
    w_router: object                   # [E, d] bf16
    w_gate: object                     # [E, h, d] uint8 codes
    s_gate: object                     # [E, h/128, d/128] fp32
    w_up: object
    s_up: object
    w_down: object                     # [E, d, h]
    s_down: object                     # [E, d/128, h/128]
    ws_gate: object = None             # [S, hs, d]
    ss_gate: object = None
    ws_up: object = None
    ss_up: object = None
    ws_down: object = None             # [S, d, hs]
    ss_down: object = None
    packed: bool = False               # w_gate, w_up as [E, d/128, h, 128] (pack_gateup)


def quantize_experts(weights: ExpertWeights, stream=None) -> Fp8ExpertWeights:
    """Quantise the expert weights of a bf16 layer with the library's block
    quantiser; the router is kept as it is."""
    if weights.packed:
        raise ValueError("quantize_experts takes row-major weights, not packed ones")
    q = {}
    for name in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"):
        t = getattr(weights, name)
        codes, scales = (None, None) if t is None else fp8_quantize_blocks(t, stream)
        q[name] = codes
        q["s" + name[1:] if name.startswith("w_") else "ss" + name[2:]] = scales
    return Fp8ExpertWeights(w_router=weights.w_router, **q)


def _aux_tensors(aux, N, E, K, device):
    torch = _torch()
    shapes = {"logits": ((N, E), torch.float32), "topk_ids": ((N, K), torch.int32),
              "topk_weights": ((N, K), torch.float32), "alpha": ((N,), torch.float32),
              "margin": ((N,), torch.float32), "beta_out": ((E,), torch.float32),
              "quantile_out": ((E,), torch.float32), "counts_before": ((E,), torch.int32),
              "counts": ((E,), torch.int32), "offsets": ((E + 1,), torch.int32),
              "sorted_src": ((N * K,), torch.int32), "src_pos": ((N, K), torch.int32)}
    aux_t = {}
    for name in aux:
        if name not in shapes:
            raise ValueError(f"unknown aux output {name!r}")
        shp, dt = shapes[name]
        aux_t[name] = torch.empty(shp, dtype=dt, device=device)
    return aux_t


def _run_forward(fp8, x, wstruct, N, d, E, K, h, n_shared, h_shared, beta_in, recompute_bias,
                 key_bits, logit_offset, logits_in, aux, workspace, out, stream, extra_flags=0,
                 x_quant=None):
    torch = _torch()
    lib = _lib.load()
    beta_in = _dev(beta_in, "beta_in", torch.float32, (E,))
    logit_offset = _dev(logit_offset, "logit_offset", torch.float32, (E,))
    logits_in = _dev(logits_in, "logits_in", torch.float32, (N, E))
    flags = (MOE_RECOMPUTE_BIAS if recompute_bias else 0) | (MOE_KEY32 if key_bits == 32 else 0)
    p = _problem(N, d, E, K, h, n_shared, h_shared, flags | extra_flags, logit_offset, logits_in)
    ws_fn = lib.moe_forward_fp8_workspace_bytes if fp8 else lib.moe_forward_workspace_bytes
    fwd = lib.moe_forward_fp8 if fp8 else lib.moe_forward
    need = int(ws_fn(C.byref(p)))
    if need == 0:  # rejected shape: the call reports why
        _lib.check(fwd(C.byref(p), None, None, None, None, None, None, 0, None))
    with _on(stream):
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        y = out if out is not None else torch.empty((N, d), dtype=torch.bfloat16, device=x.device)
        _dev(y, "out", _bf16(), (N, d))
        aux_t = _aux_tensors(aux, N, E, K, x.device)
        a = MoeAux(*[_ptr(aux_t.get(f)) for f in AUX_FIELDS]) if aux_t else None
        given = () if x_quant is None else (_ptr(x_quant[0]), _ptr(x_quant[1]))
        if given:
            fwd = lib.moe_forward_fp8_quantized
        _lib.check(fwd(C.byref(p), C.byref(wstruct), _ptr(x), *given, _ptr(beta_in), _ptr(y),
                       C.byref(a) if a is not None else None, _ptr(workspace),
                       workspace.numel() * workspace.element_size(), _stream(stream)))
    return (y, aux_t) if aux else y


def _bf16_weights(x, weights: ExpertWeights):
    x = _dev(x, "x", _bf16())
    N, d = x.shape
    wg = _dev(weights.w_gate, "w_gate", _bf16())
    if weights.packed:
        if wg.dim() != 4 or wg.shape[1] * 64 != d or wg.shape[3] != 64:
            raise ValueError("packed w_gate must be [E, d/64, h, 64]")
        E, _, h, _ = wg.shape
        _dev(weights.w_up, "w_up", _bf16(), (E, d // 64, h, 64))
    else:
        E, h, _ = wg.shape
        _dev(weights.w_up, "w_up", _bf16(), (E, h, d))
    _dev(weights.w_down, "w_down", _bf16(), (E, d, h))
    if weights.w_router is not None:
        _dev(weights.w_router, "w_router", _bf16(), (E, d))
    n_shared = 0 if weights.ws_gate is None else int(weights.ws_gate.shape[0])
    h_shared = h if n_shared == 0 else int(weights.ws_gate.shape[1])
    if n_shared:
        _dev(weights.ws_gate, "ws_gate", _bf16(), (n_shared, h_shared, d))
        _dev(weights.ws_up, "ws_up", _bf16(), (n_shared, h_shared, d))
        _dev(weights.ws_down, "ws_down", _bf16(), (n_shared, d, h_shared))
    w = MoeWeights(_ptr(weights.w_router), _ptr(wg), _ptr(weights.w_up),
                   _ptr(weights.w_down), _ptr(weights.ws_gate), _ptr(weights.ws_up),
                   _ptr(weights.ws_down))
    return x, w, N, d, E, h, n_shared, h_shared


def forward(x, weights: ExpertWeights, K: int, beta_in=None, recompute_bias: bool = False,
            key_bits: int = 16, logit_offset=None, logits_in=None, aux=(),
            workspace=None, out=None, stream=None, route_fused: bool = False):
    """MoE layer forward.  x: [N, d] bf16.  Returns y [N, d] bf16, or
    (y, dict) when ``aux`` names optional outputs (see moe_aux_t).
    ``route_fused`` selects the experts inside the router GEMM's epilogue
    (MOE_ROUTE_FUSED; same outputs as the default separate pass)."""
    x, w, N, d, E, h, n_shared, h_shared = _bf16_weights(x, weights)
    flags = (MOE_PACKED_GATEUP if weights.packed else 0) | \
        (MOE_ROUTE_FUSED if route_fused else 0)
    return _run_forward(False, x, w, N, d, E, K, h, n_shared, h_shared, beta_in, recompute_bias,
                        key_bits, logit_offset, logits_in, aux, workspace, out, stream, flags)


def forward_noalloc(x, weights: ExpertWeights, K: int, beta_in=None,
                    recompute_bias: bool = False, key_bits: int = 16, logit_offset=None,
                    logits_in=None, aux=(), out=None, stream=None,
                    route_fused: bool = False):
    """moe_forward_noalloc: the layer forward with the library's fixed
    per-GPU scratch array as its workspace (for callers that cannot allocate
    device memory; problems needing more than 64 MiB of workspace are
    rejected).  Arguments and results as forward(); pass ``out`` and aux
    tensors from the caller to keep the call itself free of allocations."""
    torch = _torch()
    lib = _lib.load()
    x, w, N, d, E, h, n_shared, h_shared = _bf16_weights(x, weights)
    beta_in = _dev(beta_in, "beta_in", torch.float32, (E,))
    logit_offset = _dev(logit_offset, "logit_offset", torch.float32, (E,))
    logits_in = _dev(logits_in, "logits_in", torch.float32, (N, E))
    flags = (MOE_RECOMPUTE_BIAS if recompute_bias else 0) | (MOE_KEY32 if key_bits == 32 else 0)
    flags |= MOE_PACKED_GATEUP if weights.packed else 0
    flags |= MOE_ROUTE_FUSED if route_fused else 0
    p = _problem(N, d, E, K, h, n_shared, h_shared, flags, logit_offset, logits_in)
    with _on(stream):
        y = out if out is not None else torch.empty((N, d), dtype=torch.bfloat16, device=x.device)
        _dev(y, "out", _bf16(), (N, d))
        aux_t = aux if isinstance(aux, dict) else _aux_tensors(aux, N, E, K, x.device)
        a = MoeAux(*[_ptr(aux_t.get(f)) for f in AUX_FIELDS]) if aux_t else None
        _lib.check(lib.moe_forward_noalloc(C.byref(p), C.byref(w), _ptr(x), _ptr(beta_in),
                                           _ptr(y), C.byref(a) if a is not None else None,
                                           _stream(stream)))
    return (y, aux_t) if aux else y


def forward_fp8(x, weights: Fp8ExpertWeights, K: int, beta_in=None,
                recompute_bias: bool = False, key_bits: int = 16, logit_offset=None,
                logits_in=None, aux=(), workspace=None, out=None, stream=None,
                route_fused: bool = False, x_quant=None):
    """MoE layer forward with E4M3 experts (moe_forward_fp8).  x: [N, d] bf16;
    weights from ``quantize_experts`` or given codes and scales.  ``x_quant``:
    the (codes, scales) of x from ``rms_norm(..., quantize=True)`` or
    ``fp8_quantize_rows``; the call then quantises nothing
    (moe_forward_fp8_quantized)."""
    torch = _torch()
    x = _dev(x, "x", _bf16())
    N, d = x.shape
    u8, f32 = torch.uint8, torch.float32
    if x_quant is not None:
        _dev(x_quant[0], "x_quant codes", u8, (N, d))
        _dev(x_quant[1], "x_quant scales", f32, (N, d // 128))
        _one_device(x, codes=x_quant[0], scales=x_quant[1])
    wg = _dev(weights.w_gate, "w_gate", u8)
    if weights.packed:
        if wg.dim() != 4 or wg.shape[1] * 128 != d or wg.shape[3] != 128:
            raise ValueError("packed w_gate codes must be [E, d/128, h, 128]")
        E, _, h, _ = wg.shape
        _dev(weights.w_up, "w_up", u8, (E, d // 128, h, 128))
    else:
        E, h, _ = wg.shape
        _dev(weights.w_up, "w_up", u8, (E, h, d))
    _dev(weights.w_down, "w_down", u8, (E, d, h))
    for name, shp in (("s_gate", (E, h // 128, d // 128)), ("s_up", (E, h // 128, d // 128)),
                      ("s_down", (E, d // 128, h // 128))):
        _dev(getattr(weights, name), name, f32, shp)
    if weights.w_router is not None:
        _dev(weights.w_router, "w_router", _bf16(), (E, d))
    n_shared = 0 if weights.ws_gate is None else int(weights.ws_gate.shape[0])
    hs = h if n_shared == 0 else int(weights.ws_gate.shape[1])
    if n_shared:
        _dev(weights.ws_gate, "ws_gate", u8, (n_shared, hs, d))
        _dev(weights.ws_up, "ws_up", u8, (n_shared, hs, d))
        _dev(weights.ws_down, "ws_down", u8, (n_shared, d, hs))
        for name, shp in (("ss_gate", (n_shared, hs // 128, d // 128)),
                          ("ss_up", (n_shared, hs // 128, d // 128)),
                          ("ss_down", (n_shared, d // 128, hs // 128))):
            _dev(getattr(weights, name), name, f32, shp)
    w = MoeFp8Weights(*[_ptr(getattr(weights, f)) for f, _ in MoeFp8Weights._fields_])
    flags = (MOE_PACKED_GATEUP if weights.packed else 0) | \
        (MOE_ROUTE_FUSED if route_fused else 0)
    return _run_forward(True, x, w, N, d, E, K, h, n_shared, hs, beta_in, recompute_bias,
                        key_bits, logit_offset, logits_in, aux, workspace, out, stream, flags,
                        x_quant)


def backward_workspace_bytes(N, d, E, K, h, n_shared=1, h_shared=None) -> int:
    p = _problem(N, d, E, K, h, n_shared, h_shared or h, 0, None, None)
    return int(_lib.load().moe_backward_workspace_bytes(C.byref(p)))


def backward(grad_y, x, weights: ExpertWeights, logits, topk_ids, grad_logits=None,
             inplace: bool = False, workspace=None, stream=None):
    """Gradients of the layer (moe_backward): grad_y, x: [N, d] bf16; logits
    fp32 [N, E] and topk_ids int32 [N, K] of the forward call (aux outputs
    "logits" and "topk_ids"); grad_logits: fp32 [N, E], the logits' gradient
    from elsewhere (balance_loss_backward, lei_backward).  Row-major weights
    only; without w_router grad_x has no router term.

    Returns (grad_x [N, d] bf16, grad_logits [N, E] fp32, ExpertWeights holding
    the weights' gradients in bf16).  With ``inplace`` the logits' gradient is
    added into grad_logits itself."""
    torch = _torch()
    lib = _lib.load()
    if weights.packed:
        raise ValueError("backward takes row-major weights, not packed ones")
    x, w, N, d, E, h, n_shared, h_shared = _bf16_weights(x, weights)
    grad_y = _dev(grad_y, "grad_y", _bf16(), (N, d))
    logits = _dev(logits, "logits", torch.float32, (N, E))
    topk_ids = _dev(topk_ids, "topk_ids", torch.int32)
    if topk_ids is None or topk_ids.dim() != 2 or topk_ids.shape[0] != N:
        raise ValueError(f"topk_ids must be [{N}, K]")
    K = topk_ids.shape[1]
    grad_logits = _dev(grad_logits, "grad_logits", torch.float32, (N, E))
    if inplace and grad_logits is None:
        raise ValueError("inplace needs grad_logits")
    names = [f for f, _ in MoeWeights._fields_ if getattr(weights, f) is not None]
    _one_device(x, grad_y=grad_y, logits=logits, topk_ids=topk_ids, grad_logits=grad_logits,
                workspace=workspace, **{f: getattr(weights, f) for f in names})
    p = _problem(N, d, E, K, h, n_shared, h_shared, 0, None, None)
    with _on_device(x, stream):
        dev = x.device
        if workspace is None:
            need = int(lib.moe_backward_workspace_bytes(C.byref(p)))
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        dx = torch.empty((N, d), dtype=torch.bfloat16, device=dev)
        dz = grad_logits if inplace else torch.empty_like(logits)
        grads = {f: torch.empty(getattr(weights, f).shape, dtype=torch.bfloat16, device=dev)
                 for f in names}
        g = MoeGrads(_ptr(dx), _ptr(dz), *[_ptr(grads.get(f)) for f, _ in MoeWeights._fields_])
        _lib.check(lib.moe_backward(
            C.byref(p), C.byref(w), _ptr(x), _ptr(grad_y), _ptr(logits), _ptr(topk_ids),
            _ptr(grad_logits), C.byref(g), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
    return dx, dz, ExpertWeights(**{"w_router": None, **grads})


def _norm_weights(weight, post_weight, d):
    torch = _torch()
    weight = _dev(weight, "weight", (*_bf16(), torch.float32), (d,))
    post_weight = _dev(post_weight, "post_weight", weight.dtype, (d,))
    return weight, post_weight, _lib.MOE_NORM_WEIGHT_F32 if weight.dtype == torch.float32 else 0


def rms_norm(x, weight, eps: float = 1e-6, residual=None, post_weight=None,
             quantize: bool = False, norm_out: bool = True, inplace: bool = False, stream=None):
    """Root-mean-square norm of the residual stream (moe_rms_norm):
    r = residual + x (``post_weight``: the normed x times it is added instead,
    the sandwich form), y = r / rms(r) * weight.  x: [n, d] bf16; residual bf16
    or fp32; weights bf16 or fp32, both of one type.

    Returns (y, residual_out, quant): y [n, d] bf16 (None without
    ``norm_out``); residual_out = r in the type of residual (bf16 without one),
    or None where r is x itself; quant = (codes uint8 [n, d], fp32 scales
    [n, d/128]) with ``quantize``, else None.  With ``inplace`` r overwrites
    residual."""
    torch = _torch()
    lib = _lib.load()
    x = _dev(x, "x", _bf16())
    if x.dim() != 2:
        raise ValueError("x must be [n, d]")
    n, d = x.shape
    weight, post_weight, flags = _norm_weights(weight, post_weight, d)
    residual = _dev(residual, "residual", (*_bf16(), torch.float32), (n, d))
    _one_device(x, weight=weight, post_weight=post_weight, residual=residual)
    if inplace and residual is None:
        raise ValueError("inplace needs residual")
    if residual is not None and residual.dtype == torch.float32:
        flags |= _lib.MOE_NORM_STREAM_F32
    with _on_device(x, stream):
        dev = x.device
        y = torch.empty((n, d), dtype=torch.bfloat16, device=dev) if norm_out else None
        r = None
        if inplace:
            r = residual
        elif residual is not None:
            r = torch.empty_like(residual)
        elif post_weight is not None:
            r = torch.empty((n, d), dtype=torch.bfloat16, device=dev)
        codes = scales = None
        if quantize:
            codes = torch.empty((n, d), dtype=torch.uint8, device=dev)
            scales = torch.empty((n, d // 128), dtype=torch.float32, device=dev)
        _lib.check(lib.moe_rms_norm(_ptr(x), _ptr(residual), _ptr(post_weight), _ptr(weight), n,
                                    d, eps, flags, _ptr(y), _ptr(r), _ptr(codes), _ptr(scales),
                                    _stream(stream)))
    return y, r, (codes, scales) if quantize else None


def rms_norm_backward(grad_y, r, weight, eps: float = 1e-6, grad_residual=None, x=None,
                      post_weight=None, weight_grads: bool = True, workspace=None, stream=None):
    """Gradients of rms_norm (moe_rms_norm_backward).  grad_y: [n, d] bf16; r:
    the residual_out of the forward call, or its x where that was None;
    grad_residual: gradient that reaches r from elsewhere, in r's type; x and
    post_weight: both, for the sandwich form.

    Returns (grad_x bf16, grad_residual in r's type, grad_weight fp32 [d],
    grad_post_weight fp32 [d] or None); without post_weight and with a bf16 r
    the first two are one tensor.  Without ``weight_grads`` the last two are
    None."""
    torch = _torch()
    lib = _lib.load()
    grad_y = _dev(grad_y, "grad_y", _bf16())
    if grad_y.dim() != 2:
        raise ValueError("grad_y must be [n, d]")
    n, d = grad_y.shape
    weight, post_weight, flags = _norm_weights(weight, post_weight, d)
    r = _dev(r, "r", (*_bf16(), torch.float32), (n, d))
    grad_residual = _dev(grad_residual, "grad_residual", r.dtype, (n, d))
    x = _dev(x, "x", _bf16(), (n, d))
    if (x is None) != (post_weight is None):
        raise ValueError("x belongs to post_weight: both or neither")
    _one_device(grad_y, weight=weight, post_weight=post_weight, r=r, grad_residual=grad_residual,
                x=x, workspace=workspace)
    f32 = r.dtype == torch.float32
    if f32:
        flags |= _lib.MOE_NORM_STREAM_F32
    with _on_device(grad_y, stream):
        dev = grad_y.device
        dres = torch.empty((n, d), dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
        shared = post_weight is None and not f32
        dx = None if shared else torch.empty((n, d), dtype=torch.bfloat16, device=dev)
        dw = torch.empty((d,), dtype=torch.float32, device=dev) if weight_grads else None
        dp = torch.empty((d,), dtype=torch.float32, device=dev) \
            if weight_grads and post_weight is not None else None
        if workspace is None:
            need = int(lib.moe_rms_norm_backward_workspace_bytes(n, d))
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _lib.check(lib.moe_rms_norm_backward(
            _ptr(grad_y), _ptr(r), _ptr(x), _ptr(grad_residual), _ptr(weight), _ptr(post_weight),
            n, d, eps, flags, _ptr(dx), _ptr(dres), _ptr(dw), _ptr(dp), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
    return dres if shared else dx, dres, dw, dp


def _segments(segments, first):
    """(begin, end, n_seg) of the segments argument of the balance loss."""
    torch = _torch()
    if segments is None:
        return None, None, 1
    if isinstance(segments, torch.Tensor):
        cu = _dev(segments, "segments", torch.int32)
        if cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("segments must be [n_seg + 1] offsets or (begin, end)")
        begin, end = cu[:-1], cu[1:]
    else:
        begin, end = segments
        begin = _dev(begin, "segments begin", torch.int32)
        end = _dev(end, "segments end", torch.int32, (begin.numel(),))
    _one_device(first, segments=begin, segments_end=end)
    return begin, end, begin.numel()


def _score(score):
    if score not in _lib.SCORES:
        raise ValueError(f"score must be one of {sorted(_lib.SCORES)}, got {score!r}")
    return _lib.SCORES[score]


def balance_loss(logits, topk_ids=None, coef: float = 1e-2, score: str = "sigmoid_norm",
                 segments=None, counts=None, workspace=None, stream=None):
    """Balance loss of the router (moe_balance_loss): coef times the mean over
    the segments of sum_e f_e P_e, with f_e = E c_e / sum c over the segment's
    loads and P_e the mean score of its rows (``score``: "sigmoid",
    "sigmoid_norm" or "softmax" of the logits).  ``segments``: int32 offsets
    [n_seg + 1] of packed sequences, or (begin, end) int32 [n_seg] each, for
    padded ones; None: the batch is one segment.  ``counts``: int32 [n_seg, E]
    loads to use in place of the batch's own.

    Returns (loss fp32 [1], counts int32 [n_seg, E] of the batch's own
    topk_ids (the given ones without topk_ids), mean scores fp32
    [n_seg, E])."""
    torch = _torch()
    lib = _lib.load()
    logits = _dev(logits, "logits", torch.float32)
    N, E = logits.shape
    topk_ids = _dev(topk_ids, "topk_ids", torch.int32)
    K = 1
    if topk_ids is not None:
        if topk_ids.dim() != 2 or topk_ids.shape[0] != N:
            raise ValueError(f"topk_ids has shape {tuple(topk_ids.shape)}, expected ({N}, K)")
        K = topk_ids.shape[1]
    begin, end, n_seg = _segments(segments, logits)
    counts = _dev(counts, "counts", torch.int32, (n_seg, E))
    if topk_ids is None and counts is None:
        raise ValueError("topk_ids or counts is required")
    _one_device(logits, topk_ids=topk_ids, counts=counts, workspace=workspace)
    which = _score(score)
    with _on_device(logits, stream):
        dev = logits.device
        loss = torch.empty((1,), dtype=torch.float32, device=dev)
        mean = torch.empty((n_seg, E), dtype=torch.float32, device=dev)
        own = None
        if topk_ids is not None:
            own = torch.empty((n_seg, E), dtype=torch.int32, device=dev)
        if workspace is None:
            need = int(lib.moe_balance_workspace_bytes(N, E, n_seg))
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _lib.check(lib.moe_balance_loss(
            _ptr(logits), _ptr(topk_ids), _ptr(counts), _ptr(begin), _ptr(end), N, E, K, n_seg,
            which, coef, _ptr(loss), _ptr(own), _ptr(mean), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
    return loss, counts if own is None else own, mean


def balance_loss_backward(logits, counts, coef: float = 1e-2, score: str = "sigmoid_norm",
                          segments=None, grad_loss=None, grad_logits=None, inplace: bool = False,
                          stream=None):
    """Gradient of balance_loss with respect to the logits
    (moe_balance_loss_backward), the loads held constant: grad_logits (None:
    zero) + grad_loss (fp32 [1] on the device, None: 1) * d loss / d logits,
    fp32 [N, E].  ``counts``: the loads that the loss was formed with.  With
    ``inplace`` the gradient is added into grad_logits itself."""
    torch = _torch()
    lib = _lib.load()
    logits = _dev(logits, "logits", torch.float32)
    N, E = logits.shape
    begin, end, n_seg = _segments(segments, logits)
    counts = _dev(counts, "counts", torch.int32, (n_seg, E))
    if counts is None:
        raise ValueError("counts is required")
    grad_loss = _dev(grad_loss, "grad_loss", torch.float32)
    if grad_loss is not None and grad_loss.numel() != 1:
        raise ValueError("grad_loss must hold one value")
    grad_logits = _dev(grad_logits, "grad_logits", torch.float32, (N, E))
    if inplace and grad_logits is None:
        raise ValueError("inplace needs grad_logits")
    _one_device(logits, counts=counts, grad_loss=grad_loss, grad_logits=grad_logits)
    which = _score(score)
    with _on_device(logits, stream):
        out = grad_logits if inplace else torch.empty_like(logits)
        _lib.check(lib.moe_balance_loss_backward(
            _ptr(logits), _ptr(counts), _ptr(begin), _ptr(end), N, E, n_seg, which, coef,
            _ptr(grad_loss), _ptr(grad_logits), _ptr(out), _stream(stream)))
    return out


def stage_timing(enable=True):
    """Per-stage HIP-event timing of forward(): True or 1 = every stage,
    2 = only the routed gate/up GEMM (two events per call), False or 0 = off.
    Clears what was recorded."""
    mode = int(enable) if not isinstance(enable, bool) else (1 if enable else 0)
    _lib.check(_lib.load().moe_stage_timing(mode))


def stage_times():
    """(dict stage -> summed ms since the last read, number of calls)."""
    lib = _lib.load()
    ms = (C.c_double * _lib.NUM_STAGES)()
    calls = C.c_int64(0)
    _lib.check(lib.moe_stage_times(ms, C.byref(calls)))
    return {lib.moe_stage_name(i).decode(): ms[i] for i in range(_lib.NUM_STAGES)}, calls.value

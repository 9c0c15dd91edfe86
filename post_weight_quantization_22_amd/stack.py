"""Layer-sequential GPTQ over a stack of MLP blocks, as a sequence of C-ABI calls.

"GPTQ deep dive" (hncyxsy.com news 243429) §3.1 step 4 and "AWQ, MinMax, GPTQ
calibration in Model Optimizer" (gtnt.cn news 115337) §4: layers are quantized
in order, each on the calibration activations produced by the network whose
earlier layers are already quantized; layers that read the same input share its
Hessian.  The block is a Llama-style MLP with a residual:

    g = x Wg_q^T, u = x Wu_q^T       gate, up: one Hessian of x, one prepare
    h = bf16(silu(g) * u)            gptq_swiglu
    y = h Wd_q^T                     down: Hessian of h
    x' = bf16(x + y)                 gptq_residual_add

Every step runs in libgptq_mi355x.so (Hessian, prepare, quantize, processing-
order packing, the products, the elementwise steps); this module allocates the
caller-owned buffers and issues the calls on one stream.  Activations stay
resident in HBM (x and h of the current block); the products run over token
chunks so their fp32 outputs stay small.  The products multiply by the
quantized weights either as a dense bf16 matrix dequantized once per layer
(gptq_dequantize + gptq_gemm_bf16, the default: the calibration set is large,
so no tile should dequantize again) or straight from the packed codes
(gptq_dequant_gemm); both form the same weights, bf16(fma(q, s, -(z s))).
"""
from __future__ import annotations

import dataclasses
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib, pipeline


@dataclasses.dataclass
class QuantizedLayer:
    buf: pipeline.LayerBuffers  # codes, scales, zeros, g_idx (original order), U, perm
    packed: torch.Tensor        # processing-order packing, the product's input
    perm: Optional[torch.Tensor]  # None when the processing order is the identity
    wq: Optional[torch.Tensor] = None  # dense bf16 weights, processing order (dense products)


@dataclasses.dataclass
class QuantizedBlock:
    gate: QuantizedLayer
    up: QuantizedLayer
    down: QuantizedLayer
    x_in: Optional[torch.Tensor] = None  # kept on request (tests)
    h: Optional[torch.Tensor] = None


class _Products:
    """Preallocated outputs and workspaces of the chunked products."""

    def __init__(self, device):
        self.device = device
        self.ws = {}
        self.out = {}
        self.xp = {}

    def get(self, tokens: int, m: int, n: int, has_perm: bool, slot: str, need_ws: bool = True):
        key = (tokens, m, n, has_perm)
        if need_ws and key not in self.ws:
            nb = _lib.gptq_dequant_gemm_workspace_size(tokens, m, n, has_perm)
            self.ws[key] = torch.empty(max(nb, 1), dtype=torch.uint8, device=self.device)
        okey = (tokens, m, slot)
        if okey not in self.out:
            self.out[okey] = torch.empty((tokens, m), dtype=torch.float32, device=self.device)
        return self.ws.get(key), self.out[okey]


def _packed(buf: pipeline.LayerBuffers, desc_act: bool, dense: bool, stream) -> QuantizedLayer:
    nw = -(-(buf.n * buf.cfg.bits) // 32)
    packed = torch.empty((buf.m, nw), dtype=torch.int32, device=buf.codes.device)
    perm = buf.perm if desc_act else None
    _lib.gptq_pack_ordered(buf.codes, buf.cfg.bits, perm, packed, stream=stream)
    wq = None
    if dense:
        ldw = -(-buf.n // 8) * 8
        wq = torch.empty((buf.m, ldw), dtype=torch.bfloat16, device=packed.device)[:, :buf.n]
        _lib.gptq_dequantize(packed, buf.cfg.bits, buf.cfg.group_size, buf.scales, buf.zeros,
                             buf.n, wq, stream=stream)
    return QuantizedLayer(buf, packed, perm, wq)


def _gathered(prod: _Products, X: torch.Tensor, perm: Optional[torch.Tensor], slot: str,
              stream) -> torch.Tensor:
    """X in the layers' processing order (X itself without desc_act), formed
    once for every layer that reads it."""
    if perm is None:
        return X
    key = (X.shape[0], X.shape[1], slot)
    if key not in prod.xp:
        ldxp = -(-X.shape[1] // 8) * 8
        prod.xp[key] = torch.empty((X.shape[0], ldxp), dtype=torch.bfloat16,
                                   device=prod.device)[:, :X.shape[1]]
    Xp = prod.xp[key]
    _lib.gptq_gather_columns(X, perm, Xp, stream=stream)
    return Xp


def _product(prod: _Products, Xp: torch.Tensor, L: QuantizedLayer, slot: str,
             stream) -> torch.Tensor:
    """Y = X W_q^T from the activations already in L's processing order."""
    ws, Y = prod.get(Xp.shape[0], L.buf.m, L.buf.n, False, slot, need_ws=L.wq is None)
    if L.wq is not None:
        _lib.gptq_gemm_bf16(Xp, L.wq, Y, stream=stream)
    else:
        _lib.gptq_dequant_gemm(Xp, L.packed, L.buf.cfg.bits, L.buf.cfg.group_size, L.buf.scales,
                               L.buf.zeros, Y, perm=None, ws=ws, stream=stream)
    return Y


def quantize_stack(x0: torch.Tensor, weights: Sequence[Tuple[torch.Tensor, torch.Tensor,
                                                             torch.Tensor]],
                   cfg: _lib.GPTQConfig, chunk_tokens: int = 16384, keep: bool = False,
                   stream=None, marks: Optional[list] = None, dense: bool = True
                   ) -> Tuple[List[QuantizedBlock], torch.Tensor]:
    """Quantize every block of the stack in order; returns the blocks and the
    quantized network's output activations (bf16 [tokens, d]).

    x0: bf16 [tokens, d] calibration activations (device).  weights: per block
    (Wg [f, d], Wu [f, d], Wd [d, f]) bf16 or fp32 device tensors.  Enqueued on
    ``stream`` (default: the current stream); the data-error words of a block's
    three layers are checked (a synchronization) at the end of the block.  ``marks``: if a list,
    (phase, event) pairs are appended, each event recorded on ``stream`` at the
    end of the phase (timing only).  ``dense``: multiply by the dequantized bf16
    weights (gptq_gemm_bf16) instead of the packed codes (gptq_dequant_gemm)."""
    if stream is None:
        stream = torch.cuda.current_stream()
    dev = x0.device
    T, d = x0.shape
    desc = bool(cfg.desc_act)
    prod = _Products(dev)
    def mark(name):
        if marks is not None:
            ev = torch.cuda.Event(enable_timing=True)
            ev.record(stream)
            marks.append((name, ev))

    mark("start")
    x = x0
    blocks = []
    for Wg, Wu, Wd in weights:
        f = Wg.shape[0]
        # gate and up: one Hessian of x, one prepare, two quantizations
        bg = pipeline.allocate(f, d, cfg, T, device=dev)
        bu = pipeline.allocate(f, d, cfg, 0, device=dev)
        bg.S.zero_()
        pipeline.accumulate(bg, [x], stream)
        mark("hessian")
        pipeline.prepare(bg, T, stream)
        mark("prepare")
        bu.S, bu.U, bu.perm, bu.dead = bg.S, bg.U, bg.perm, bg.dead  # shared Hessian
        pipeline.quantize(bg, Wg, stream)
        pipeline.quantize(bu, Wu, stream)
        gate, up = _packed(bg, desc, dense, stream), _packed(bu, desc, dense, stream)
        mark("quantize")
        # h = silu(x Wg_q^T) * (x Wu_q^T), chunk by chunk
        h = torch.empty((T, f), dtype=torch.bfloat16, device=dev)
        for t0 in range(0, T, chunk_tokens):
            t1 = min(T, t0 + chunk_tokens)
            xp = _gathered(prod, x[t0:t1], gate.perm, "x", stream)  # gate and up: one order
            g = _product(prod, xp, gate, "g", stream)
            u = _product(prod, xp, up, "u", stream)
            _lib.gptq_swiglu(g, u, h[t0:t1], stream=stream)
        mark("forward")
        # down: Hessian of h
        bd = pipeline.allocate(d, f, cfg, T, device=dev)
        bd.S.zero_()
        pipeline.accumulate(bd, [h], stream)
        mark("hessian")
        pipeline.prepare(bd, T, stream)
        mark("prepare")
        pipeline.quantize(bd, Wd, stream)
        down = _packed(bd, desc, dense, stream)
        mark("quantize")
        # x' = x + h Wd_q^T
        x_next = torch.empty_like(x)
        for t0 in range(0, T, chunk_tokens):
            t1 = min(T, t0 + chunk_tokens)
            y = _product(prod, _gathered(prod, h[t0:t1], down.perm, "h", stream), down, "y",
                         stream)
            _lib.gptq_residual_add(x[t0:t1], y, x_next[t0:t1], stream=stream)
        mark("forward")
        for b in (bg, bu, bd):
            pipeline.check_info(b)
        blocks.append(QuantizedBlock(gate, up, down, x if keep else None, h if keep else None))
        x = x_next
    return blocks, x


# ---------------------------------------------------------------------------
# The same stack in 8-bit floating point: weights and activations in e4m3 with
# a scale per 128 x 128 block and per token and 128 columns ("AWQ, MinMax, GPTQ
# calibration in Model Optimizer", section 2: the max calibrator needs no
# calibration data, so a layer's weights are quantized on their own).
#
#     x8 = e4m3(x)                     fp8_quantize_rows
#     g = x8 Wg8^T, u = x8 Wu8^T       fp8_gated_gemm, g and u bf16
#     h8 = e4m3(silu(g) * u)
#     x' = bf16(x + h8 Wd8^T)          fp8_gemm with x as its residual
#
# g and u are rounded to bf16, half a step of 2^-8 relative, before h is rounded to
# e4m3's 2^-4: where they pass through memory they then take half the bytes.
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Fp8Layer:
    codes: torch.Tensor   # e4m3 [m, n], row stride a multiple of 16
    scales: torch.Tensor  # fp32 [ceil(m / 128), ceil(n / 128)]


@dataclasses.dataclass
class Fp8Block:
    gate: Fp8Layer
    up: Fp8Layer
    down: Fp8Layer


def quantize_layer_fp8(W: torch.Tensor, stream=None) -> Fp8Layer:
    """W[m, n] (bf16 or fp32) as e4m3 codes and block scales, enqueued on ``stream`` (default:
    the current stream of W's device), which their memory belongs to."""
    if stream is None:
        stream = torch.cuda.current_stream(W.device)
    if stream.device != W.device:
        raise ValueError(f"the stream is on {stream.device}, W on {W.device}")
    m, n = W.shape
    ld = -(-n // 16) * 16
    with torch.cuda.stream(stream):  # (memory of another stream may still be in use there)
        codes = torch.empty((m, ld), dtype=torch.float8_e4m3fn, device=W.device)[:, :n]
        scales = torch.empty((-(-m // _lib.FP8_BLOCK), -(-n // _lib.FP8_BLOCK)),
                             dtype=torch.float32, device=W.device)
        _lib.fp8_quantize_blocks(W, codes, scales)
    return Fp8Layer(codes, scales)


def forward_block_fp8(x: torch.Tensor, block: Fp8Block, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """x' [tokens, d] (bf16) of one block for x [tokens, d] (bf16); gate and up [f, d], down
    [d, f], d and f multiples of 16; out: bf16, at least [tokens, d],
    may be x.
    Enqueued on ``stream`` (default: the current stream of x's device)."""
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x: dtype {x.dtype}, expected bfloat16")
    T, d = x.shape
    f = block.gate.codes.shape[0]
    for name, shape in (("gate", (f, d)), ("up", (f, d)), ("down", (d, f))):
        got = tuple(getattr(block, name).codes.shape)
        if got != shape:
            raise ValueError(f"{name}: codes of shape {got}, expected {shape}")
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, x on {x.device}")
    with torch.cuda.stream(stream):  # the buffers between the steps belong to the stream
        def buf(rows, cols, dtype):
            return torch.empty((rows, cols), dtype=dtype, device=x.device)

        if out is None:
            out = buf(T, d, torch.bfloat16)
        x8, xs = buf(T, d, torch.float8_e4m3fn), buf(-(-d // _lib.FP8_BLOCK), T, torch.float32)
        _lib.fp8_quantize_rows(x, x8, xs)
        h8, hs = buf(T, f, torch.float8_e4m3fn), buf(-(-f // _lib.FP8_BLOCK), T, torch.float32)
        _lib.fp8_gated_gemm(x8, xs, block.gate.codes, block.gate.scales, block.up.codes,
                            block.up.scales, h8, hs)
        _lib.fp8_gemm(h8, hs, block.down.codes, block.down.scales, out, residual=x)
    return out


def quantize_stack_fp8(x0: torch.Tensor, weights: Sequence[Tuple[torch.Tensor, torch.Tensor,
                                                                 torch.Tensor]],
                       chunk_tokens: int = 16384, stream=None
                       ) -> Tuple[List[Fp8Block], torch.Tensor]:
    """Quantize every block of the stack to e4m3 and carry x0 (bf16 [tokens, d]) through it,
    ``chunk_tokens`` at a time (a token does not depend on the others, but the order of
    its fp32 sums does on a call's size, and a code where a sum lies on a border of it);
    returns the blocks and the quantized network's output activations."""
    if stream is None:
        stream = torch.cuda.current_stream(x0.device)
    blocks = []
    x = x0
    for ws in weights:
        with torch.cuda.stream(stream):
            block = Fp8Block(*(quantize_layer_fp8(W, stream) for W in ws))
            x_next = torch.empty_like(x)
            for t0 in range(0, x.shape[0], chunk_tokens):
                t1 = min(x.shape[0], t0 + chunk_tokens)
                forward_block_fp8(x[t0:t1], block, x_next[t0:t1], stream)
        blocks.append(block)
        x = x_next
    return blocks, x

"""torch-facing layer on top of the C ABI: custom ops and a drop-in linear module.

The issue "Revamp int4 MPS support in torchao" (issue text) asks for a
module built directly on the weight-only quantized linear that quantizes on
the fly and accepts a bias, and its thread shows a user broken by one missing
bit width: here an ``nn.Linear`` is replaced by a module that quantizes its
weight once, keeps the packed codes and the per-group scales and zeros, and
runs the low-bit kernel in ``forward``, for every bit width 1..7.  "Add
support for fbgemm int4 mm kernel" notes that an op without a shape (meta)
function cannot be traced by ``torch.compile``; the ops registered here carry
one.

Ops (namespace ``lowbit``):

* ``lowbit::quantize_pack(Tensor w, int bits, int group, ScalarType sz_dtype)
  -> (Tensor packed, Tensor scales, Tensor zeros)`` -- fp32 ``w[N, K]`` on the
  GPU to codes packed LSB-first, ``N x (K*bits/8)`` bytes, and scales / zeros
  ``N x (K/group)`` in ``sz_dtype``;
* ``lowbit::linear(Tensor x, Tensor packed, Tensor scales, Tensor zeros,
  Tensor? bias, int bits, int group) -> Tensor`` -- ``x[..., K]`` to
  ``y[..., N]`` in x's dtype, ``y = x . dequant(W)^T (+ bias)``;
* ``lowbit::linear_a8(...)`` -- the same signature with 8-bit dynamic
  activations: each row of x is quantized on the fly to int8 codes with one
  fp32 scale (symmetric, max |x| / 127), and the linear runs over the codes
  on the int8 matrix cores (the export mode with 8-bit dynamic activations
  and 4-bit weights in groups of 32 of "[MPS] Add support for Int4 groupwise
  quantization");
* ``lowbit::rmsnorm_q8(Tensor x, Tensor? weight, float eps, int fmt) ->
  (Tensor q, Tensor qscale)`` and ``lowbit::add_rmsnorm_q8(Tensor x, Tensor
  residual, Tensor? weight, float eps, int fmt) -> (Tensor q, Tensor qscale,
  Tensor h)`` -- RMS norm of ``x`` (of ``h = x + residual``) straight to 8-bit
  codes and scales: ``lowbit.Q8_I8`` (the input of ``lowbit_linear_a8``) or
  ``lowbit.Q8_F8`` (the input of the ops below);
* ``lowbit::quantize_act_f8``, ``lowbit::quantize_weight_f8`` -- e4m3 codes
  with an fp32 scale for each block of 128 (128 x 128);
* ``lowbit::linear_f8(Tensor xq, Tensor xscale, Tensor wq, Tensor wscale,
  Tensor? bias, ScalarType dtype) -> Tensor`` -- the linear over such codes on
  the fp8 matrix cores;
* ``lowbit::linear_f8_grouped(Tensor xq, Tensor xscale, Tensor? rows, Tensor
  offsets, Tensor wq, Tensor wscale, Tensor? bias, ScalarType dtype) ->
  Tensor`` -- the same for rows grouped by expert;
* ``lowbit::moe_route(Tensor logits, Tensor? bias, int topk, int score, int
  groups, int topk_groups, int group_best, bool renormalize, float scale) ->
  (Tensor experts, Tensor weights)`` -- each token's experts and their weights;
* ``lowbit::group_rows(Tensor ids, int num_experts) -> (Tensor rows, Tensor
  offsets, Tensor position)`` -- the slots of ``ids[T, k]`` in the order of their
  expert (or adapter);
* ``lowbit::moe_combine(Tensor y, Tensor position, Tensor weights, Tensor?
  residual) -> Tensor`` -- each token's weighted sum of its experts' rows;
* ``lowbit::lora(Tensor x, Tensor a, Tensor b, Tensor? scales, Tensor? rows,
  Tensor offsets, Tensor? base, bool all_rows=False) -> Tensor`` -- ``base`` plus
  the low-rank adapter of each row.  Rows that ``rows`` does not name keep
  ``base``, of which a copy is made first; ``all_rows`` says that it names every
  row, as group_rows makes it, so that none is needed (rows left out all the same
  are undefined then).

All run in liblowbit.so through :mod:`bit_groupwise_weight_amd.lowbit`;
nothing here computes on the CPU.
"""
from __future__ import annotations

from typing import Callable, NamedTuple, Optional, Tuple

import torch

from . import lowbit as _lb

_SZ_DTYPES = (torch.float16, torch.bfloat16, torch.float32)


def _check_bits_group(bits: int, group: int) -> None:
    if bits not in range(1, 8):
        raise ValueError(f"bits must be in 1..7, got {bits}")
    if group not in (32, 64, 128, 256):
        raise ValueError(f"group must be 32, 64, 128 or 256, got {group}")


def _check_linear_shapes(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                         zeros: torch.Tensor, bias: Optional[torch.Tensor], bits: int,
                         group: int) -> Tuple[int, int]:
    _check_bits_group(bits, group)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension (..., K)")
    K = x.shape[-1]
    if scales.dim() != 2 or zeros.shape != scales.shape:
        raise ValueError("scales and zeros must both be [N, K/group]")
    N = scales.shape[0]
    if K % group != 0 or scales.shape[1] != K // group:
        raise ValueError(f"x has K={K}, scales imply K={scales.shape[1] * group}")
    if packed.numel() != N * K * bits // 8:
        raise ValueError(f"packed holds {packed.numel()} bytes, expected N*K*bits/8 = {N * K * bits // 8}")
    if packed.dtype != torch.uint8:
        raise ValueError("packed must be uint8")
    if scales.dtype != x.dtype or zeros.dtype != x.dtype:
        raise ValueError("scales and zeros must have the activation dtype")
    if bias is not None and (bias.shape != (N,) or bias.dtype != x.dtype):
        raise ValueError("bias must be [N] in the activation dtype")
    return N, K


# ------------------------------------------------------------------ ops --

@torch.library.custom_op("lowbit::quantize_pack", mutates_args=())
def quantize_pack(w: torch.Tensor, bits: int, group: int,
                  sz_dtype: torch.dtype) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    _check_bits_group(bits, group)
    if sz_dtype not in _SZ_DTYPES:
        raise ValueError(f"sz_dtype must be one of {_SZ_DTYPES}")
    # fp32, fp16 and bf16 weights go in as they are (the kernel takes fp16 and
    # bf16 values exactly as fp32); other dtypes are converted to fp32 first
    if w.dtype not in (torch.float32, torch.float16, torch.bfloat16):
        w = w.float()
    packed, scales, zeros, _ = _lb.lowbit_quantize_pack(w.contiguous(), bits, group, sz_dtype)
    return packed, scales, zeros


@quantize_pack.register_fake
def _quantize_pack_fake(w, bits, group, sz_dtype):
    _check_bits_group(bits, group)
    N, K = w.shape
    if K % group != 0:
        raise ValueError(f"K={K} is not a multiple of group={group}")
    packed = w.new_empty((N, K * bits // 8), dtype=torch.uint8)
    scales = w.new_empty((N, K // group), dtype=sz_dtype)
    return packed, scales, torch.empty_like(scales)


@torch.library.custom_op("lowbit::linear", mutates_args=())
def linear(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
           bias: Optional[torch.Tensor], bits: int, group: int) -> torch.Tensor:
    N, K = _check_linear_shapes(x, packed, scales, zeros, bias, bits, group)
    lead = x.shape[:-1]
    x2 = x.reshape(-1, K).contiguous()
    y = _lb.lowbit_linear(x2, packed.contiguous(), scales.contiguous(), zeros.contiguous(),
                          None if bias is None else bias.contiguous(), bits, group)
    return y.reshape(*lead, N)


@linear.register_fake
def _linear_fake(x, packed, scales, zeros, bias, bits, group):
    N, _ = _check_linear_shapes(x, packed, scales, zeros, bias, bits, group)
    return x.new_empty((*x.shape[:-1], N))


@torch.library.custom_op("lowbit::linear_a8", mutates_args=())
def linear_a8(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
              bias: Optional[torch.Tensor], bits: int, group: int) -> torch.Tensor:
    N, K = _check_linear_shapes(x, packed, scales, zeros, bias, bits, group)
    lead = x.shape[:-1]
    x2 = x.reshape(-1, K).contiguous()
    xq, ascale = _lb.lowbit_quantize_act_i8(x2)
    y = _lb.lowbit_linear_a8(xq, ascale, packed.contiguous(), scales.contiguous(),
                             zeros.contiguous(), None if bias is None else bias.contiguous(),
                             bits, group)
    return y.reshape(*lead, N)


@linear_a8.register_fake
def _linear_a8_fake(x, packed, scales, zeros, bias, bits, group):
    N, _ = _check_linear_shapes(x, packed, scales, zeros, bias, bits, group)
    return x.new_empty((*x.shape[:-1], N))


# ------------------------------------------------------ ops, 8-bit path --

def _check_norm(x: torch.Tensor, weight: Optional[torch.Tensor], fmt: int) -> None:
    if x.dim() < 1 or x.dtype not in _SZ_DTYPES:
        raise ValueError(f"x must be [..., K] in one of {_SZ_DTYPES}")
    if fmt not in (_lb.Q8_I8, _lb.Q8_F8):
        raise ValueError(f"fmt must be Q8_I8 or Q8_F8, got {fmt}")
    unit = 32 if fmt == _lb.Q8_I8 else 16
    if x.shape[-1] == 0 or x.shape[-1] % unit:
        raise ValueError(f"K={x.shape[-1]} must be a positive multiple of {unit}")
    if weight is not None and (weight.shape != x.shape[-1:] or weight.dtype != x.dtype):
        raise ValueError("weight must be [K] in x's dtype")


def _norm_out(x: torch.Tensor, fmt: int) -> Tuple[torch.Tensor, torch.Tensor]:
    lead, K = x.shape[:-1], x.shape[-1]
    if fmt == _lb.Q8_I8:
        return x.new_empty(x.shape, dtype=torch.int8), x.new_empty(lead, dtype=torch.float32)
    return (x.new_empty(x.shape, dtype=torch.float8_e4m3fn),
            x.new_empty((*lead, _lb._f8_blocks(K)), dtype=torch.float32))


@torch.library.custom_op("lowbit::rmsnorm_q8", mutates_args=())
def rmsnorm_q8(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float,
               fmt: int) -> Tuple[torch.Tensor, torch.Tensor]:
    _check_norm(x, weight, fmt)
    q, s = _norm_out(x, fmt)
    K = x.shape[-1]
    _lb.lowbit_add_rmsnorm_q8(x.reshape(-1, K).contiguous(), None if weight is None else weight.contiguous(),
                              eps, fmt, q=q.view(-1, K),
                              qscale=s.view(-1) if fmt == _lb.Q8_I8 else s.view(-1, s.shape[-1]))
    return q, s


@rmsnorm_q8.register_fake
def _rmsnorm_q8_fake(x, weight, eps, fmt):
    _check_norm(x, weight, fmt)
    return _norm_out(x, fmt)


@torch.library.custom_op("lowbit::add_rmsnorm_q8", mutates_args=())
def add_rmsnorm_q8(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor], eps: float,
                   fmt: int) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    _check_norm(x, weight, fmt)
    if residual.shape != x.shape or residual.dtype != x.dtype:
        raise ValueError("residual must have x's shape and dtype")
    q, s = _norm_out(x, fmt)
    K = x.shape[-1]
    h = x.new_empty(x.shape)
    _lb.lowbit_add_rmsnorm_q8(x.reshape(-1, K).contiguous(), None if weight is None else weight.contiguous(),
                              eps, fmt, residual=residual.reshape(-1, K).contiguous(), q=q.view(-1, K),
                              qscale=s.view(-1) if fmt == _lb.Q8_I8 else s.view(-1, s.shape[-1]),
                              h=h.view(-1, K))
    return q, s, h


@add_rmsnorm_q8.register_fake
def _add_rmsnorm_q8_fake(x, residual, weight, eps, fmt):
    _check_norm(x, weight, fmt)
    if residual.shape != x.shape or residual.dtype != x.dtype:
        raise ValueError("residual must have x's shape and dtype")
    return (*_norm_out(x, fmt), x.new_empty(x.shape))


@torch.library.custom_op("lowbit::quantize_act_f8", mutates_args=())
def quantize_act_f8(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    _check_norm(x, None, _lb.Q8_F8)
    q, s = _norm_out(x, _lb.Q8_F8)
    K = x.shape[-1]
    _lb.lowbit_quantize_act_f8(x.reshape(-1, K).contiguous(), q.view(-1, K), s.view(-1, s.shape[-1]))
    return q, s


@quantize_act_f8.register_fake
def _quantize_act_f8_fake(x):
    _check_norm(x, None, _lb.Q8_F8)
    return _norm_out(x, _lb.Q8_F8)


def _check_weight(w: torch.Tensor) -> None:
    if w.dim() not in (2, 3) or w.numel() == 0:
        raise ValueError("w must be [N, K] or [E, N, K], not empty")
    if w.shape[-1] % 16:
        raise ValueError(f"K={w.shape[-1]} must be a multiple of 16")


@torch.library.custom_op("lowbit::quantize_weight_f8", mutates_args=())
def quantize_weight_f8(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    _check_weight(w)
    if w.dtype not in _SZ_DTYPES:
        w = w.float()
    return _lb.lowbit_quantize_weight_f8(w.contiguous())


@quantize_weight_f8.register_fake
def _quantize_weight_f8_fake(w):
    _check_weight(w)
    N, K = w.shape[-2:]
    spans = (*w.shape[:-2], _lb._f8_blocks(N), _lb._f8_blocks(K))
    return w.new_empty(w.shape, dtype=torch.float8_e4m3fn), w.new_empty(spans, dtype=torch.float32)


def _check_f8(xq, xscale, wq, wscale, bias, dtype, wdims=2) -> None:
    if xq.dim() < 1 or wq.dim() != wdims:
        raise ValueError(f"xq must be [..., K] and wq {'[N, K]' if wdims == 2 else '[E, N, K]'}")
    K = xq.shape[-1]
    if K == 0 or K % 16:
        raise ValueError(f"K={K} must be a positive multiple of 16")
    if wq.shape[-1] != K:
        raise ValueError(f"xq has K={K}, wq has K={wq.shape[-1]}")
    if xq.dtype != torch.float8_e4m3fn or wq.dtype != torch.float8_e4m3fn:
        raise ValueError("xq and wq must be float8_e4m3fn")
    if xscale.shape != (*xq.shape[:-1], _lb._f8_blocks(K)) or xscale.dtype != torch.float32:
        raise ValueError("xscale must be float32 [..., ceil(K/128)]")
    if (wscale.shape != (*wq.shape[:-2], _lb._f8_blocks(wq.shape[-2]), _lb._f8_blocks(K))
            or wscale.dtype != torch.float32):
        raise ValueError("wscale must be float32 [(E,) ceil(N/128), ceil(K/128)]")
    if dtype not in _SZ_DTYPES:
        raise ValueError(f"dtype must be one of {_SZ_DTYPES}")
    if bias is not None and (bias.shape != wq.shape[:-1] or bias.dtype != dtype):
        raise ValueError("bias must be [(E,) N] in the output dtype")


@torch.library.custom_op("lowbit::linear_f8", mutates_args=())
def linear_f8(xq: torch.Tensor, xscale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
              bias: Optional[torch.Tensor], dtype: torch.dtype) -> torch.Tensor:
    _check_f8(xq, xscale, wq, wscale, bias, dtype)
    K, N = xq.shape[-1], wq.shape[0]
    y = _lb.lowbit_linear_f8(xq.reshape(-1, K).contiguous(), xscale.reshape(-1, xscale.shape[-1]).contiguous(),
                             wq.contiguous(), wscale.contiguous(),
                             None if bias is None else bias.contiguous(), dtype)
    return y.reshape(*xq.shape[:-1], N)


@linear_f8.register_fake
def _linear_f8_fake(xq, xscale, wq, wscale, bias, dtype):
    _check_f8(xq, xscale, wq, wscale, bias, dtype)
    return xq.new_empty((*xq.shape[:-1], wq.shape[0]), dtype=dtype)


def _check_grouped(xq, xscale, rows, offsets, wq, wscale, bias, dtype) -> None:
    _check_f8(xq, xscale, wq, wscale, bias, dtype, wdims=3)
    if xq.dim() != 2:
        raise ValueError("xq must be [M, K]")
    if offsets.shape != (wq.shape[0] + 1,) or offsets.dtype != torch.int32:
        raise ValueError("offsets must be int32 [E + 1]")
    if rows is not None and (rows.dim() != 1 or rows.dtype != torch.int32):
        raise ValueError("rows must be int32 [T]")


@torch.library.custom_op("lowbit::linear_f8_grouped", mutates_args=())
def linear_f8_grouped(xq: torch.Tensor, xscale: torch.Tensor, rows: Optional[torch.Tensor],
                      offsets: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                      bias: Optional[torch.Tensor], dtype: torch.dtype) -> torch.Tensor:
    _check_grouped(xq, xscale, rows, offsets, wq, wscale, bias, dtype)
    return _lb.lowbit_linear_f8_grouped(xq.contiguous(), xscale.contiguous(), offsets, wq.contiguous(),
                                        wscale.contiguous(), None if bias is None else bias.contiguous(),
                                        dtype, rows=rows)


@linear_f8_grouped.register_fake
def _linear_f8_grouped_fake(xq, xscale, rows, offsets, wq, wscale, bias, dtype):
    _check_grouped(xq, xscale, rows, offsets, wq, wscale, bias, dtype)
    T = xq.shape[0] if rows is None else rows.shape[0]
    return xq.new_empty((T, wq.shape[1]), dtype=dtype)


# ------------------------------------------ ops, around the experts, adapters --

def _check_route(logits, bias, topk, score, groups, topk_groups, group_best, scale) -> int:
    if logits.dim() < 1 or logits.dtype not in _SZ_DTYPES:
        raise ValueError(f"logits must be [..., E] in one of {_SZ_DTYPES}")
    E = logits.shape[-1]
    if not 1 <= E <= _lb.ROUTE_MAX_EXPERTS:
        raise ValueError(f"E={E} not in 1..{_lb.ROUTE_MAX_EXPERTS}")
    if not 1 <= topk <= min(E, _lb.ROUTE_MAX_TOPK):
        raise ValueError(f"topk={topk} not in 1..min(E, {_lb.ROUTE_MAX_TOPK})")
    if score not in (_lb.ROUTE_SOFTMAX, _lb.ROUTE_SIGMOID):
        raise ValueError(f"score must be ROUTE_SOFTMAX or ROUTE_SIGMOID, got {score}")
    if not 1 <= groups <= _lb.ROUTE_MAX_GROUPS or E % groups:
        raise ValueError(f"groups={groups} must be a divisor of E={E}, at most {_lb.ROUTE_MAX_GROUPS}")
    if not 1 <= topk_groups <= groups or group_best not in (1, 2):
        raise ValueError("topk_groups must be in 1..groups, group_best 1 or 2")
    if bias is not None and (bias.shape != (E,) or bias.dtype != torch.float32):
        raise ValueError("bias must be float32 [E]")
    if not abs(scale) < float("inf"):
        raise ValueError(f"scale={scale} is not finite")
    return E


@torch.library.custom_op("lowbit::moe_route", mutates_args=())
def moe_route(logits: torch.Tensor, bias: Optional[torch.Tensor], topk: int, score: int, groups: int,
              topk_groups: int, group_best: int, renormalize: bool,
              scale: float) -> Tuple[torch.Tensor, torch.Tensor]:
    E = _check_route(logits, bias, topk, score, groups, topk_groups, group_best, scale)
    experts, weights = _lb.lowbit_moe_route(logits.reshape(-1, E).contiguous(), topk,
                                            None if bias is None else bias.contiguous(), score, groups,
                                            topk_groups, group_best, renormalize, scale)
    shape = (*logits.shape[:-1], topk)
    return experts.view(shape), weights.view(shape)


@moe_route.register_fake
def _moe_route_fake(logits, bias, topk, score, groups, topk_groups, group_best, renormalize, scale):
    _check_route(logits, bias, topk, score, groups, topk_groups, group_best, scale)
    shape = (*logits.shape[:-1], topk)
    return logits.new_empty(shape, dtype=torch.int32), logits.new_empty(shape, dtype=torch.float32)


def _check_group_rows(ids: torch.Tensor, num_experts: int) -> None:
    if ids.dim() != 2 or ids.shape[1] < 1 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be [T, k], int32 or int64")
    if not 1 <= num_experts <= 1 << 16:
        raise ValueError(f"num_experts={num_experts} not in 1..2^16")


@torch.library.custom_op("lowbit::group_rows", mutates_args=())
def group_rows(ids: torch.Tensor, num_experts: int) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    _check_group_rows(ids, num_experts)
    return _lb.lowbit_group_rows(ids.contiguous(), num_experts)


@group_rows.register_fake
def _group_rows_fake(ids, num_experts):
    _check_group_rows(ids, num_experts)
    T, k = ids.shape
    return (ids.new_empty((T * k,), dtype=torch.int32), ids.new_empty((num_experts + 1,), dtype=torch.int32),
            ids.new_empty((T, k), dtype=torch.int32))


def _check_combine(y, position, weights, residual) -> None:
    if y.dim() != 2 or y.shape[1] < 1 or y.dtype not in _SZ_DTYPES:
        raise ValueError(f"y must be [R, N] in one of {_SZ_DTYPES}")
    if position.dim() != 2 or position.shape[1] < 1 or position.dtype != torch.int32:
        raise ValueError("position must be int32 [T, k]")
    if position.shape[1] > _lb.COMBINE_MAX_TOPK:
        raise ValueError(f"k={position.shape[1]} is more than {_lb.COMBINE_MAX_TOPK}")
    if weights.shape != position.shape or weights.dtype != torch.float32:
        raise ValueError("weights must be float32 [T, k]")
    if residual is not None and (residual.shape != (position.shape[0], y.shape[1]) or residual.dtype != y.dtype):
        raise ValueError("residual must be [T, N] in y's dtype")


@torch.library.custom_op("lowbit::moe_combine", mutates_args=())
def moe_combine(y: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
                residual: Optional[torch.Tensor]) -> torch.Tensor:
    _check_combine(y, position, weights, residual)
    return _lb.lowbit_moe_combine(y.contiguous(), position.contiguous(), weights.contiguous(),
                                  None if residual is None else residual.contiguous())


@moe_combine.register_fake
def _moe_combine_fake(y, position, weights, residual):
    _check_combine(y, position, weights, residual)
    return y.new_empty((position.shape[0], y.shape[1]))


def _check_lora(x, a, b, scales, rows, offsets, base) -> Tuple[int, int]:
    if x.dim() < 1 or x.dtype not in _SZ_DTYPES:
        raise ValueError(f"x must be [..., K] in one of {_SZ_DTYPES}")
    if a.dim() != 3 or b.dim() != 3 or a.dtype != x.dtype or b.dtype != x.dtype:
        raise ValueError("a must be [L, rank, K] and b [L, N, rank] in x's dtype")
    L, rank, K = a.shape
    N = b.shape[1]
    if x.shape[-1] != K or b.shape[0] != L or b.shape[2] != rank:
        raise ValueError(f"x has K={x.shape[-1]}; a {list(a.shape)} and b {list(b.shape)} do not fit it and each other")
    if L < 1 or N < 1 or K == 0 or K % 16 or rank == 0 or rank % 8 or rank > _lb.LORA_MAX_RANK:
        raise ValueError(f"L and N must be positive, K a positive multiple of 16, rank one of 8 up to {_lb.LORA_MAX_RANK}")
    if L > _lb.LORA_MAX_ADAPTERS or max(N, K) > _lb.LORA_MAX_SIZE:
        raise ValueError(f"L={L}, N={N} and K={K} must be at most {_lb.LORA_MAX_ADAPTERS}, {_lb.LORA_MAX_SIZE} and "
                         f"{_lb.LORA_MAX_SIZE}")
    if offsets.shape != (L + 1,) or offsets.dtype != torch.int32:
        raise ValueError("offsets must be int32 [L + 1]")
    if scales is not None and (scales.shape != (L,) or scales.dtype != torch.float32):
        raise ValueError("scales must be float32 [L]")
    if rows is not None and (rows.dim() != 1 or rows.dtype != torch.int32):
        raise ValueError("rows must be int32 [T]")
    if base is not None and (base.shape != (*x.shape[:-1], N) or base.dtype != x.dtype):
        raise ValueError("base must be [..., N] in x's dtype")
    return N, K


@torch.library.custom_op("lowbit::lora", mutates_args=())
def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scales: Optional[torch.Tensor],
         rows: Optional[torch.Tensor], offsets: torch.Tensor, base: Optional[torch.Tensor],
         all_rows: bool = False) -> torch.Tensor:
    N, K = _check_lora(x, a, b, scales, rows, offsets, base)
    x2 = x.reshape(-1, K).contiguous()
    base2 = None if base is None else base.reshape(-1, N).contiguous()
    a, b, offsets, y = a.contiguous(), b.contiguous(), offsets.contiguous(), None
    rows, scales = (None if t is None else t.contiguous() for t in (rows, scales))
    if rows is not None and (not all_rows or rows.shape[0] < x2.shape[0]):
        y = x2.new_zeros((x2.shape[0], N)) if base2 is None else base2.clone()
        base2 = None if base2 is None else y                  # (in place)
    y = _lb.lowbit_lora(x2, a, b, scales, rows, offsets, base2, y=y)
    return y.reshape(*x.shape[:-1], N)


@lora.register_fake
def _lora_fake(x, a, b, scales, rows, offsets, base, all_rows=False):
    N, _ = _check_lora(x, a, b, scales, rows, offsets, base)
    return x.new_empty((*x.shape[:-1], N))


# --------------------------------------------------------------- module --

def _derived(t: torch.Tensor) -> bool:
    """Whether a derivative of t may be asked for: it requires one, carries a forward-mode tangent, or
    a transform of torch.func (a derivative of either mode, vmap) is at work, under which only torch's
    operations are differentiated and batched.  (torch has no public query for the last.)"""
    if torch._C._are_functorch_transforms_active():
        return True
    if torch.is_grad_enabled() and t.requires_grad:
        return True
    return torch.autograd.forward_ad.unpack_dual(t).tangent is not None


def _no_tangent(what: str, *tensors: Optional[torch.Tensor]) -> None:
    """Refuse tensors that carry a forward-mode tangent: the library's calls have no derivative, and
    torch would drop the tangent without a word.  (Of nested derivatives the innermost one's is seen;
    in a compiled program batched tensors are refused while forward mode is at work.)"""
    if torch.autograd.forward_ad._current_level < 0:
        return
    functorch = torch._C._functorch
    for t in tensors:
        if t is None:
            continue
        compiling = torch.compiler.is_compiling()
        while not compiling and functorch.is_batchedtensor(t):
            t = functorch.get_unwrapped(t)
        if functorch.is_batchedtensor(t) or torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{what} has no forward-mode derivative")


class LowbitLinear(torch.nn.Module):
    """``nn.Linear`` with a groupwise b-bit weight: w = s * q + z per group.

    Buffers: ``packed`` (uint8, ``[N, K*bits/8]``), ``scales`` and ``zeros``
    (``[N, K/group]``, activation dtype) and optional ``bias`` (``[N]``).
    Inputs must be on the GPU, in the activation dtype, with last dim K.
    ``act_bits=8`` quantizes the activations too, per row to int8 on every
    call (``lowbit::linear_a8``); ``None`` keeps them floating point.
    """

    def __init__(self, in_features: int, out_features: int, bits: int, group_size: int,
                 bias: bool = True, dtype: torch.dtype = torch.float16,
                 device: Optional[torch.device] = None, act_bits: Optional[int] = None):
        super().__init__()
        _check_bits_group(bits, group_size)
        if act_bits not in (None, 8):
            raise ValueError(f"act_bits must be None or 8, got {act_bits}")
        self.act_bits = act_bits
        if dtype not in _SZ_DTYPES:
            raise ValueError(f"dtype must be one of {_SZ_DTYPES}")
        if in_features % group_size != 0:
            raise ValueError(f"in_features={in_features} is not a multiple of group_size={group_size}")
        self.in_features, self.out_features = in_features, out_features
        self.bits, self.group_size, self.dtype = bits, group_size, dtype
        self._call = None            # prepared eager call (made on first use)
        G = in_features // group_size
        self.register_buffer("packed", torch.zeros((out_features, in_features * bits // 8),
                                                   dtype=torch.uint8, device=device))
        self.register_buffer("scales", torch.zeros((out_features, G), dtype=dtype, device=device))
        self.register_buffer("zeros", torch.zeros((out_features, G), dtype=dtype, device=device))
        if bias:
            self.register_buffer("bias", torch.zeros((out_features,), dtype=dtype, device=device))
        else:
            self.bias = None

    @torch.no_grad()
    def set_weight(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> "LowbitLinear":
        """Quantize a float ``weight[N, K]`` (on the GPU) into this module."""
        if tuple(weight.shape) != (self.out_features, self.in_features):
            raise ValueError(f"weight must be [{self.out_features}, {self.in_features}]")
        packed, scales, zeros = torch.ops.lowbit.quantize_pack(weight.detach(), self.bits,
                                                               self.group_size, self.dtype)
        self.packed.copy_(packed)
        self.scales.copy_(scales)
        self.zeros.copy_(zeros)
        if self.bias is not None:
            if bias is None:
                self.bias.zero_()
            else:
                self.bias.copy_(bias.detach().to(self.dtype))
        return self

    @classmethod
    def from_linear(cls, lin: torch.nn.Linear, bits: int, group_size: int,
                    dtype: Optional[torch.dtype] = None,
                    act_bits: Optional[int] = None) -> "LowbitLinear":
        """Quantize ``lin`` on the fly (its weight must live on the GPU)."""
        dt = dtype or (lin.weight.dtype if lin.weight.dtype in _SZ_DTYPES else torch.float16)
        m = cls(lin.in_features, lin.out_features, bits, group_size, bias=lin.bias is not None,
                dtype=dt, device=lin.weight.device, act_bits=act_bits)
        return m.set_weight(lin.weight, lin.bias)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.act_bits == 8:
            return torch.ops.lowbit.linear_a8(x, self.packed, self.scales, self.zeros, self.bias,
                                              self.bits, self.group_size)
        # Traced (torch.compile), autograd and non-GPU (e.g. meta) calls go
        # through the registered op; plain eager GPU calls take the prepared
        # call, which validated the weights once (buffers replaced by .to()
        # and the like make a new one).
        if (not x.is_cuda or torch.compiler.is_compiling()
                or (x.requires_grad and torch.is_grad_enabled())):
            return torch.ops.lowbit.linear(x, self.packed, self.scales, self.zeros, self.bias,
                                           self.bits, self.group_size)
        b = self._buffers
        call = self._call
        if (call is None or call._keep[0] is not b["packed"] or call._keep[1] is not b["scales"]
                or call._keep[2] is not b["zeros"] or call._keep[3] is not b.get("bias")):
            call = _lb.PreparedLinear(b["packed"], b["scales"], b["zeros"], b.get("bias"),
                                      self.bits, self.group_size)
            self._call = call
        if x.dim() == 2:
            return call(x.contiguous())
        y = call(x.reshape(-1, self.in_features).contiguous())
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, bits={self.bits}, "
                f"group_size={self.group_size}, dtype={self.dtype}, bias={self.bias is not None}"
                + ("" if self.act_bits is None else f", act_bits={self.act_bits}"))


def quantize_linears(model: torch.nn.Module, bits: int, group_size: int,
                     dtype: Optional[torch.dtype] = None,
                     filter_fn: Optional[Callable[[torch.nn.Module, str], bool]] = None,
                     act_bits: Optional[int] = None) -> torch.nn.Module:
    """Replace every ``nn.Linear`` of ``model`` (in place) by a LowbitLinear.

    ``filter_fn(module, qualified_name)`` may exclude layers; layers whose
    in_features is not a multiple of ``group_size`` are left as they are.
    ``act_bits=8`` makes every swapped layer quantize its activations too.
    """
    for name, child in list(model.named_children()):
        _swap(model, name, child, name, bits, group_size, dtype, filter_fn, act_bits)
    return model


def _swap(parent, name, child, qual, bits, group_size, dtype, filter_fn, act_bits):
    if isinstance(child, torch.nn.Linear):
        if child.in_features % group_size == 0 and (filter_fn is None or filter_fn(child, qual)):
            setattr(parent, name, LowbitLinear.from_linear(child, bits, group_size, dtype, act_bits))
        return
    for n, c in list(child.named_children()):
        _swap(child, n, c, f"{qual}.{n}", bits, group_size, dtype, filter_fn, act_bits)


class _F8Module(torch.nn.Module):
    """Base of the e4m3 modules.  Their codes and scales (every buffer but ``bias``) are a format, not
    numbers to be cast: ``.half()``, ``.to(dtype)`` and the like leave their types alone and set the
    type of the outputs and the bias."""

    def _apply(self, fn, recurse=True):
        def example(t, dtype):
            return fn(torch.empty(1, dtype=dtype, device=t.device))

        held = {id(b) for name, b in self._buffers.items() if name != "bias"}
        dtype = example(next(b for b in self._buffers.values() if b is not None), self.dtype).dtype
        if dtype not in _SZ_DTYPES:
            raise ValueError(f"{type(self).__name__} computes in one of {_SZ_DTYPES}, not {dtype}")

        def keep(t):
            if id(t) not in held:
                return fn(t)
            like = example(t, t.dtype)
            return fn(t) if like.dtype == t.dtype else t.to(like.device)

        super()._apply(keep, recurse)
        self.dtype = dtype
        return self


class F8Linear(_F8Module):
    """``nn.Linear`` with e4m3 weights and activations, an fp32 scale for each block of 128 x 128
    weights and of 128 activations of a row.

    Buffers: ``wq`` (float8_e4m3fn, ``[N, K]``), ``wscale`` (fp32, ``[ceil(N/128), ceil(K/128)]``)
    and optional ``bias`` (``[N]``).  ``forward(x)`` quantizes x's rows on the fly; where a norm
    made the codes already (``lowbit::add_rmsnorm_q8``), ``forward_codes(xq, xscale)`` takes them.
    """

    def __init__(self, in_features: int, out_features: int, bias: bool = True,
                 dtype: torch.dtype = torch.bfloat16, device: Optional[torch.device] = None):
        super().__init__()
        if dtype not in _SZ_DTYPES:
            raise ValueError(f"dtype must be one of {_SZ_DTYPES}")
        if in_features <= 0 or in_features % 16 != 0:
            raise ValueError(f"in_features={in_features} is not a positive multiple of 16")
        self.in_features, self.out_features, self.dtype = in_features, out_features, dtype
        self.register_buffer("wq", torch.zeros((out_features, in_features), dtype=torch.float8_e4m3fn,
                                               device=device))
        self.register_buffer("wscale", torch.zeros((_lb._f8_blocks(out_features), _lb._f8_blocks(in_features)),
                                                   dtype=torch.float32, device=device))
        if bias:
            self.register_buffer("bias", torch.zeros((out_features,), dtype=dtype, device=device))
        else:
            self.bias = None

    @torch.no_grad()
    def set_weight(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> "F8Linear":
        """Quantize a float ``weight[N, K]`` (on the GPU) into this module."""
        if tuple(weight.shape) != (self.out_features, self.in_features):
            raise ValueError(f"weight must be [{self.out_features}, {self.in_features}]")
        wq, wscale = torch.ops.lowbit.quantize_weight_f8(weight.detach())
        self.wq.copy_(wq)
        self.wscale.copy_(wscale)
        if self.bias is not None:
            if bias is None:
                self.bias.zero_()
            else:
                self.bias.copy_(bias.detach().to(self.dtype))
        return self

    @classmethod
    def from_linear(cls, lin: torch.nn.Linear, dtype: Optional[torch.dtype] = None) -> "F8Linear":
        """Quantize ``lin`` on the fly (its weight must live on the GPU)."""
        dt = dtype or (lin.weight.dtype if lin.weight.dtype in _SZ_DTYPES else torch.bfloat16)
        m = cls(lin.in_features, lin.out_features, bias=lin.bias is not None, dtype=dt,
                device=lin.weight.device)
        return m.set_weight(lin.weight, lin.bias)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        xq, xscale = torch.ops.lowbit.quantize_act_f8(x)
        return self.forward_codes(xq, xscale)

    def forward_codes(self, xq: torch.Tensor, xscale: torch.Tensor) -> torch.Tensor:
        return torch.ops.lowbit.linear_f8(xq, xscale, self.wq, self.wscale, self.bias, self.dtype)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, dtype={self.dtype}, "
                f"bias={self.bias is not None}")


def quantize_linears_f8(model: torch.nn.Module, dtype: Optional[torch.dtype] = None,
                        filter_fn: Optional[Callable[[torch.nn.Module, str], bool]] = None
                        ) -> torch.nn.Module:
    """Replace every ``nn.Linear`` of ``model`` (in place) by an F8Linear; layers whose in_features
    is not a multiple of 16, and those that ``filter_fn(module, qualified_name)`` excludes, are left
    as they are.  A layer that stands at several places is quantized once and shared by those that
    the filter admits."""
    made = {}
    linears = [(n, c) for n, c in model.named_modules(remove_duplicate=False)
               if isinstance(c, torch.nn.Linear) and n]
    for qual, child in linears:
        if child.in_features % 16 == 0 and (filter_fn is None or filter_fn(child, qual)):
            if id(child) not in made:
                made[id(child)] = F8Linear.from_linear(child, dtype)
            parent, _, name = qual.rpartition(".")
            setattr(model.get_submodule(parent), name, made[id(child)])
    return model


class F8Experts(_F8Module):
    """The experts of a mixture-of-experts block in the e4m3 format: for a token x and each of its
    experts e with routing weight r,

        out += r * down[e] (silu(gate[e] x) * (up[e] x))

    Buffers: ``gate_up`` (``[E, 2 I, H]``, gate rows first) and ``down`` (``[E, H, I]``) as e4m3
    codes with their block scales.  The tokens' codes are made once whatever number of experts a
    token goes to, and nothing waits for the routing on the host.
    """

    def __init__(self, num_experts: int, hidden: int, intermediate: int,
                 dtype: torch.dtype = torch.bfloat16, device: Optional[torch.device] = None):
        super().__init__()
        if dtype not in _SZ_DTYPES:
            raise ValueError(f"dtype must be one of {_SZ_DTYPES}")
        if num_experts < 1 or hidden <= 0 or intermediate <= 0 or hidden % 16 or intermediate % 16:
            raise ValueError("hidden and intermediate must be positive multiples of 16, num_experts >= 1")
        self.num_experts, self.hidden, self.intermediate, self.dtype = num_experts, hidden, intermediate, dtype
        b = _lb._f8_blocks
        for name, n, k in (("gate_up", 2 * intermediate, hidden), ("down", hidden, intermediate)):
            self.register_buffer(name, torch.zeros((num_experts, n, k), dtype=torch.float8_e4m3fn,
                                                   device=device))
            self.register_buffer(name + "_scale", torch.zeros((num_experts, b(n), b(k)),
                                                              dtype=torch.float32, device=device))

    @torch.no_grad()
    def set_weight(self, gate_up: torch.Tensor, down: torch.Tensor) -> "F8Experts":
        """Quantize float ``gate_up[E, 2 I, H]`` and ``down[E, H, I]`` (on the GPU) into this module."""
        for name, w in (("gate_up", gate_up), ("down", down)):
            if w.shape != getattr(self, name).shape:
                raise ValueError(f"{name} must be {list(getattr(self, name).shape)}, got {list(w.shape)}")
            q, s = torch.ops.lowbit.quantize_weight_f8(w.detach())
            getattr(self, name).copy_(q)
            getattr(self, name + "_scale").copy_(s)
        return self

    def forward(self, x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """x[..., H] (the module's dtype); experts (integer) and weights, both [..., k]: each
        token's experts and their routing weights.  An expert outside 0..E-1 (a padded slot)
        adds nothing."""
        xq, xscale = torch.ops.lowbit.quantize_act_f8(x.reshape(-1, self.hidden))
        return self.forward_codes(xq, xscale, experts, weights).reshape(x.shape)

    def forward_codes(self, xq: torch.Tensor, xscale: torch.Tensor, experts: torch.Tensor,
                      weights: torch.Tensor) -> torch.Tensor:
        """The same for tokens' codes and scales as ``lowbit::add_rmsnorm_q8`` makes them: [T, H]."""
        T, k = xq.shape[0], experts.shape[-1]
        if experts.shape != weights.shape or experts.numel() != T * k:
            raise ValueError("experts and weights must both be [T, k]")
        if k == 0:
            return weights.reshape(T, 0, 1).float().expand(T, 0, self.hidden).sum(1).to(self.dtype)
        ids = experts.reshape(T, k)
        if ids.dtype not in (torch.int32, torch.int64):
            ids = ids.long()
        rows, offsets, position = torch.ops.lowbit.group_rows(ids, self.num_experts)
        gu = torch.ops.lowbit.linear_f8_grouped(xq, xscale, rows, offsets, self.gate_up, self.gate_up_scale,
                                                None, self.dtype)
        gate, up = gu.split(self.intermediate, dim=-1)
        aq, ascale = torch.ops.lowbit.quantize_act_f8(torch.nn.functional.silu(gate) * up)
        slots = torch.ops.lowbit.linear_f8_grouped(aq, ascale, None, offsets, self.down, self.down_scale,
                                                   None, self.dtype)
        # (rows of no expert are undefined; their slots have position -1 and add nothing)
        weights = weights.reshape(T, k).float()
        if k > 31 or _derived(weights):
            # the same sum from torch's operations, which know the derivatives of the routing weights
            # (bit for bit up to 31 slots; from 32 on torch's sum adds in another order, and is kept)
            # (both factors of a slot without an expert are 0 before they meet, for the derivatives' sake)
            used = position >= 0
            out = torch.where(used.unsqueeze(-1), slots[position.clamp(min=0).long()].float(), 0.0)
            return (out * torch.where(used, weights, 0.0).unsqueeze(-1)).sum(1).to(self.dtype)
        return torch.ops.lowbit.moe_combine(slots, position, weights, None)

    def extra_repr(self) -> str:
        return (f"num_experts={self.num_experts}, hidden={self.hidden}, intermediate={self.intermediate}, "
                f"dtype={self.dtype}")


class MoeRouter(torch.nn.Module):
    """Chooses each token's experts for F8Experts from the router's logits.

    ``score`` "softmax" or "sigmoid"; the experts of largest score (plus ``bias`` where the router
    has one for balance, which the weights leave out) among the ``topk_groups`` best of ``groups``
    groups, a group's value being its largest choice (``group_best`` 1) or the sum of its two
    largest (2); weights renormalized over the chosen, times ``scale``.  The bias is a float32 buffer
    and stays one when the module is cast.
    """

    def __init__(self, num_experts: int, topk: int, score: str = "softmax", bias: bool = False, groups: int = 1,
                 topk_groups: int = 1, group_best: int = 1, renormalize: bool = True, scale: float = 1.0,
                 device: Optional[torch.device] = None):
        super().__init__()
        if score not in ("softmax", "sigmoid"):
            raise ValueError(f'score must be "softmax" or "sigmoid", got {score!r}')
        self.num_experts, self.topk, self.score, self.scale = num_experts, topk, score, float(scale)
        self.groups, self.topk_groups, self.group_best = groups, topk_groups, group_best
        self.renormalize = bool(renormalize)
        _check_route(torch.empty((1, num_experts), device="meta"), None, topk, self._score(), groups, topk_groups,
                     group_best, self.scale)
        if bias:
            self.register_buffer("bias", torch.zeros((num_experts,), dtype=torch.float32, device=device))
        else:
            self.bias = None

    def _score(self) -> int:
        return _lb.ROUTE_SOFTMAX if self.score == "softmax" else _lb.ROUTE_SIGMOID

    def _apply(self, fn, recurse=True):
        def keep(t):
            moved = fn(t)
            return moved if moved.dtype == t.dtype else t.to(moved.device)

        return super()._apply(keep, recurse)

    def forward(self, logits: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """logits[..., E] -> (experts int32, weights float32), both [..., topk]."""
        if logits.shape[-1:] != (self.num_experts,):
            raise ValueError(f"logits must be [..., {self.num_experts}], got {list(logits.shape)}")
        _no_tangent("MoeRouter", logits, self.bias)
        return torch.ops.lowbit.moe_route(logits, self.bias, self.topk, self._score(), self.groups,
                                          self.topk_groups, self.group_best, self.renormalize, self.scale)

    def extra_repr(self) -> str:
        return (f"num_experts={self.num_experts}, topk={self.topk}, score={self.score}, groups={self.groups}, "
                f"topk_groups={self.topk_groups}, group_best={self.group_best}, renormalize={self.renormalize}, "
                f"scale={self.scale}, bias={self.bias is not None}")


class AdapterPlan(NamedTuple):
    """A batch's rows in the order of their adapter, every row named once, and where each adapter's
    begin: ``rows`` and ``offsets`` of ``lowbit::group_rows``."""
    rows: torch.Tensor
    offsets: torch.Tensor


def adapter_plan(ids: torch.Tensor, num_adapters: int) -> AdapterPlan:
    """The plan of a batch for its LoraLinear layers, from each row's adapter (any integer type;
    outside 0..num_adapters-1: none): (rows, offsets), made on the GPU, good for every layer."""
    ids = ids.reshape(-1, 1)
    if ids.dtype not in (torch.int32, torch.int64):
        ids = ids.long()
    rows, offsets, _ = torch.ops.lowbit.group_rows(ids, num_adapters)
    return AdapterPlan(rows, offsets)


class LoraLinear(torch.nn.Module):
    """A linear (LowbitLinear, F8Linear, nn.Linear) shared by all rows with low-rank adapters of
    many requests beside it:

        y = linear(x) + scales[l] * b[l] (a[l] x),  l each row's adapter

    Buffers: ``a`` (``[num_adapters, rank, K]``), ``b`` (``[num_adapters, N, rank]``, both in
    ``dtype``, that of x and y) and ``scales`` (float32).  ``set_adapter`` puts an adapter of that
    rank or less into its place while others are in use.
    """

    def __init__(self, linear: torch.nn.Module, num_adapters: int, rank: int,
                 dtype: Optional[torch.dtype] = None, device: Optional[torch.device] = None):
        super().__init__()
        K, N = linear.in_features, linear.out_features
        held = next((t for t in (*linear.buffers(), *linear.parameters())), None)
        if device is None and held is not None:
            device = held.device
        if dtype is None:
            dtype = getattr(linear, "dtype", None) or linear.weight.dtype
        if dtype not in _SZ_DTYPES:
            raise ValueError(f"dtype must be one of {_SZ_DTYPES}")
        if num_adapters < 1 or K % 16 or rank <= 0 or rank % 8 or rank > _lb.LORA_MAX_RANK:
            raise ValueError(f"num_adapters must be positive, in_features a multiple of 16 and rank one of 8 up to "
                             f"{_lb.LORA_MAX_RANK}")
        self.linear, self.num_adapters, self.rank = linear, num_adapters, rank
        self.in_features, self.out_features = K, N
        self.register_buffer("a", torch.zeros((num_adapters, rank, K), dtype=dtype, device=device))
        self.register_buffer("b", torch.zeros((num_adapters, N, rank), dtype=dtype, device=device))
        self.register_buffer("scales", torch.ones((num_adapters,), dtype=torch.float32, device=device))

    def _apply(self, fn, recurse=True):
        scales = self.scales

        def keep(t):
            moved = fn(t)
            return t.to(moved.device) if t is scales and moved.dtype != t.dtype else moved

        return super()._apply(keep, recurse)

    @torch.no_grad()
    def set_adapter(self, index: int, a: torch.Tensor, b: torch.Tensor, scale: float = 1.0) -> "LoraLinear":
        """Adapter ``index``: ``a[r, K]``, ``b[N, r]`` (r up to ``rank``) and its factor."""
        r = a.shape[0]
        if not 0 <= index < self.num_adapters:
            raise ValueError(f"index={index} not in 0..{self.num_adapters - 1}")
        if a.shape != (r, self.in_features) or b.shape != (self.out_features, r) or r > self.rank:
            raise ValueError(f"a must be [r, {self.in_features}] and b [{self.out_features}, r], r at most {self.rank}")
        self.a[index].zero_()
        self.b[index].zero_()
        self.a[index, :r].copy_(a)
        self.b[index, :, :r].copy_(b)
        self.scales[index] = scale
        return self

    def forward(self, x: torch.Tensor, plan: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> torch.Tensor:
        """x[..., K] -> [..., N]; ``plan`` = adapter_plan(ids, num_adapters) for x's rows, None for
        no adapters.  Rows that a (rows, offsets) of another make does not name keep the linear's
        output; an AdapterPlan names all of them, which saves the copy that keeping it takes."""
        y = self.linear(x)
        if plan is None:
            return y
        _no_tangent("LoraLinear", x, y, self.a, self.b, self.scales)
        return torch.ops.lowbit.lora(x, self.a, self.b, self.scales, plan[0], plan[1], y,
                                     isinstance(plan, AdapterPlan))

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"num_adapters={self.num_adapters}, rank={self.rank}, dtype={self.a.dtype}")

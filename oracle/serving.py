"""The calls around a block, restated in fp64: the norms before and after it, the whole layer
for a few tokens and low-rank adapters beside a projection.  Test infrastructure like
``reference.py``, whose functions it builds on."""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np

from . import reference as ref

__all__ = ["round_f64_via_f32_to_bf16_bits", "bf16_candidates", "rms_norm", "combine_norm_residual", "moe_layer_few",
           "adapter_gemm"]


def round_f64_via_f32_to_bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp64 rounded to fp32, then to bf16 (both to nearest, ties to even)."""
    return ref.round_f64_to_bf16_bits(np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64))


def bf16_candidates(x: np.ndarray, rel: float) -> np.ndarray:
    """The bf16 patterns that a value within `rel` of x (relative) can round to: [2][...]."""
    x = np.asarray(x, dtype=np.float64)
    return np.stack([round_f64_via_f32_to_bf16_bits(x * (1 - rel)), round_f64_via_f32_to_bf16_bits(x * (1 + rel))])


def rms_norm(v: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """v / sqrt(mean(v^2) + eps) * weight per row, in fp64."""
    v = np.asarray(v, dtype=np.float64)
    ms = np.mean(v * v, axis=1, keepdims=True)
    return v / np.sqrt(ms + float(np.float32(eps))) * np.asarray(weight, dtype=np.float64)


def combine_norm_residual(rows: np.ndarray, residual: np.ndarray, slot_of: Optional[np.ndarray],
                          topk_w: Optional[np.ndarray], n_shared: int, post_weight: Optional[np.ndarray], eps: float,
                          gate: Optional[np.ndarray], scale: float) -> np.ndarray:
    """residual + scale * gate * norm(combined rows), in fp64 before its rounding."""
    T = residual.shape[0]
    topk = 0 if slot_of is None else slot_of.shape[1]
    y = np.zeros(residual.shape)
    for j in range(topk):
        y += np.asarray(topk_w[:, j:j + 1], dtype=np.float64) * np.asarray(rows, dtype=np.float64)[slot_of[:, j]]
    for s in range(n_shared):
        y += np.asarray(rows[T * topk + s * T:T * topk + (s + 1) * T], dtype=np.float64)
    if post_weight is not None:
        y = rms_norm(y, post_weight, eps)
    if gate is not None:
        y = y * np.asarray(gate, dtype=np.float64)
    return np.asarray(residual, dtype=np.float64) + float(np.float32(scale)) * y


def moe_layer_few(q: np.ndarray, scales: np.ndarray, logits: np.ndarray, gate, up, down, topk: int, n_shared: int,
                  act_bits: int, renormalize: bool = True, codes_h: Optional[tuple] = None) -> Dict:
    """The MoE layer on quantised tokens with h kept unrounded.  Rows are per choice: row
    t*topk + j is token t's j-th choice, row T*topk + s*T + t shared expert s.  codes_h
    (q [R][F], scales [R]) replaces the oracle's own codes of h (teacher forcing)."""
    T = q.shape[0]
    rt = ref.route(logits, topk, renormalize, n_shared)
    E = logits.shape[1]
    expert = np.concatenate([rt["ids"].ravel(), np.repeat(np.arange(E, E + n_shared), T)])
    token = np.concatenate([np.repeat(np.arange(T), topk), np.tile(np.arange(T), n_shared)])
    order = np.argsort(expert, kind="stable")
    offs = np.searchsorted(expert[order], np.arange(E + n_shared + 1))

    def grouped(qq, sc, tok, w):
        out = ref.expert_gemm(qq, sc, tok[order], offs, w.idx, w.codebook, w.K, w.bits)
        back = np.empty_like(out)
        back[order] = out
        return back

    g, u = grouped(q, scales, token, gate), grouped(q, scales, token, up)
    with np.errstate(over="ignore"):
        h = g * u / (1.0 + np.exp(-g))
    if codes_h is None:
        b = ref.block_size(h.shape[1])
        qh, sh = ref.quantize(ref.rotate_fp64(h, b).astype(np.float32), b, act_bits)
        qh = qh.astype(np.int64)
    else:
        qh, sh = codes_h
    out = grouped(qh, sh, np.arange(len(expert)), down)
    y = np.zeros((T, out.shape[1]))
    for j in range(topk):
        y += rt["weights64"][:, j:j + 1] * out[np.arange(T) * topk + j]
    for s in range(n_shared):
        y += out[T * topk + s * T:T * topk + (s + 1) * T]
    return dict(route=rt, h=h, qh=qh, sh=sh, out=out, y=y, expert=expert, token=token)


def adapter_gemm(q: np.ndarray, scales: np.ndarray, W: np.ndarray, x: np.ndarray, lora_a: np.ndarray,
                 lora_b: np.ndarray, adapter_of: np.ndarray, adapter_scale: Optional[np.ndarray]) -> np.ndarray:
    """scale_t * q W^T + s_a * B_a (A_a x) with a = adapter_of[t]; ids outside the set add nothing."""
    y = ref.dense_gemm(q, scales, W)
    for t in range(q.shape[0]):
        a = int(adapter_of[t])
        if 0 <= a < lora_a.shape[0]:
            s = 1.0 if adapter_scale is None else float(adapter_scale[a])
            y[t] += s * (np.asarray(lora_b[a], dtype=np.float64) @ (np.asarray(lora_a[a], dtype=np.float64) @ x[t]))
    return y

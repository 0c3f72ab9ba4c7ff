"""Shared helpers for the tests of the few-row operators: packed weights, quantised rows, and the
operators' definitions in 64 bits with the error bounds the kernels are held to.

Bounds (derived from the formulas; u = 2^-24, the fp32 rounding unit):
  product  fp32 sums of n terms in blocks of 16, each step off by at most 2 u of the partial sum of
           absolute values A, the low-rank factor's intermediate kept as BF16 hi + lo (2^-16 of its
           terms B), then one rounding to BF16 (half a step, 2^-8 of the value).  GELU has a slope
           below 1.13 and an evaluation error of 3e-7 max(1, |y|).
           The rows themselves enter as eight FP4 digits to the base 8: with the row's largest magnitude M
           in [2^e, 2^(e+1)) a value has digits of 2^(e-1) 8^-p, p = 0..7, each rounded to nearest, so what
           is left is at most 2^(e-1) 8^-7 / 2 = 2^(e-23) <= 2^-23 M.  Times the weights' magnitudes, summed.
  norm     a relative error of (C / 256 + 48) u: the sum of C squares in strides of at least 256
           threads and a tree, a division, a square root, a reciprocal and two products; then half a
           step of the format (BF16 2^-8, E4M3 2^-4 of the value, 2^-10 scales below its normal range).
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def bf16(t: torch.Tensor) -> torch.Tensor:
    return t.to(torch.bfloat16)


def e2m1_values(codes: np.ndarray) -> np.ndarray:
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
    return mag[codes & 7] * np.where(codes & 8, -1.0, 1.0)


class Weight:
    """A packed layer of random weights: the blob and factors for the device, and its values in 64 bits."""

    def __init__(self, dq, Ci, Co, rank, seed=0, bias=False, c2=False, scale=1.0):
        from dq_case import packed_weight_parts
        rng = np.random.default_rng(seed)
        W = rng.standard_normal((Co, Ci)) * scale / np.sqrt(Ci)
        W[:, rng.integers(0, Ci, max(1, Ci // 100))] *= 20
        self.l1 = bf16(torch.from_numpy(rng.standard_normal((Ci, rank)) / np.sqrt(Ci)))
        self.l2 = bf16(torch.from_numpy(rng.standard_normal((rank, Co)) * scale / np.sqrt(rank)))
        bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
        packed, l1m, l2s, _ = dq.dq_pack_weight_factors(bits(bf16(torch.from_numpy(W))), bits(self.l1), bits(self.l2),
                                                        pack_flags=dq.DQ_PACK_C2 if c2 else 0)
        self.bias = None
        if bias:
            self.bias = bf16(torch.from_numpy(rng.standard_normal(Co)))
            dq.dq_pack_bias(packed, bits(self.bias))
        self.Ci, self.Co, self.rank, self.packed = Ci, Co, rank, packed
        parts = packed_weight_parts(packed)
        codes = np.stack([parts["wcodes"] & 15, parts["wcodes"] >> 4], 2).reshape(Co, Ci)
        s = torch.from_numpy(parts["wscales"].copy()).view(torch.float8_e4m3fn).double().numpy()
        self.values = e2m1_values(codes) * np.repeat(s, 16, axis=1) * float(parts["S_w"])   # Co x Ci
        self._host = (packed, l1m.view(np.int16), l2s.view(np.int16))

    def device(self, dev="cuda"):
        return tuple(torch.from_numpy(a).to(dev) for a in self._host)


def rows_input(rows, Ci, fmt, seed=0, outliers=True):
    """(values in 64 bits, tensor for the device, scales or None); fmt 0, 1, 2 as DQ_ROWS_*."""
    rng = np.random.default_rng(seed + 17)
    x = rng.standard_normal((rows, Ci)) * np.exp(0.5 * rng.standard_normal(Ci))
    if outliers:
        x[:, rng.integers(0, Ci, max(1, Ci // 100))] *= 50
    x = torch.from_numpy(x)
    if fmt == 0:
        xb = bf16(x)
        return xb.double(), xb, None
    return quantise_rows(x, fmt)


def quantise_rows(x: torch.Tensor, fmt: int):
    rows, C = x.shape
    n = C if fmt == 1 else 64
    g = x.float().reshape(rows, C // n, n)
    s = g.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, g / s[:, :, None], torch.zeros(())).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = (q.double() * s.double()[:, :, None]).reshape(rows, C)
    return v, q.reshape(rows, C), s.contiguous()


def rows_reference(w: Weight, v: torch.Tensor, gelu: bool):
    """(Y in 64 bits, tolerance) of the product of the rows with values v."""
    wv, l1, l2 = torch.from_numpy(w.values), w.l1.double(), w.l2.double()
    y = v @ w_t(wv)
    A = v.abs() @ w_t(wv.abs())
    low = (v @ l1) @ l2
    B = (v.abs() @ l1.abs()) @ l2.abs()
    y = y + low
    if w.bias is not None:
        y = y + w.bias.double()
        A = A + w.bias.double().abs()
    digits = 2.0 ** -23 * v.abs().amax(1, keepdim=True).expand_as(v)
    tol = digits @ w_t(wv.abs()) + 2 * U * (w.Ci / 16 + 32) * A + (2 * U * (w.Ci / 16 + 2 * w.rank + 32) + 2.0 ** -16) * B
    if gelu:
        tol = 1.13 * tol + 3e-7 * y.abs().clamp(min=1.0)
        y = y * 0.5 * torch.special.erfc(-y / np.sqrt(2.0))
    return y, tol + 2.0 ** -8 * y.abs() + 2.0 ** -133


def w_t(t):
    return t.t().contiguous()


def assert_within(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what: str):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got.cpu()[tuple(i)])}, "
                             f"reference {float(ref[tuple(i)])}, bound {float(tol[tuple(i)])}")


def norm_reference(x, residual, gamma, eps):
    h = x.double() + (0 if residual is None else residual.double())
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    return h, y


def norm_rel(C):
    return (C / 256 + 48) * U


def check_norm(dq, h, y, C, fmt, got_sum, got_y, got_scales, what=""):
    """Outputs of dq_rmsnorm_forward (on the CPU) against h and y in 64 bits."""
    rel = norm_rel(C)
    if got_sum is not None:
        assert_within(got_sum, h, 2.0 ** -8 * (1 + 2.0 ** -12) * h.abs() + 2.0 ** -134, what + " sum")
    if fmt == 0:
        assert_within(got_y, y, (2.0 ** -8 + 2 * rel) * y.abs() + 2.0 ** -134, what + " Y")
        return
    n = C if fmt == 1 else 64
    groups = -(-C // n)
    pad = torch.nn.functional.pad(y, (0, groups * n - C)).reshape(y.shape[0], groups, n)
    s = pad.abs().amax(2) / 448.0
    assert_within(got_scales.reshape(s.shape), s, 2 * rel * s + 2.0 ** -149, what + " scales")
    sx = s.repeat_interleave(n, 1)[:, :C]
    v = got_y.double() * got_scales.double().reshape(s.shape).repeat_interleave(n, 1)[:, :C]
    assert_within(v, y, (2.0 ** -4 + 4 * rel) * y.abs() + 2.0 ** -10 * (1 + 4 * rel) * sx + 2.0 ** -148, what + " codes")

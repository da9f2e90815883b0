"""Attention over a shared prefix and own caches by its definition in fp64, and how far a
kernel that rounds queries, rows and weights to fp16 may be from it.

Tolerance of one output element d of a query row, in the rotated domain (q~ = H q scale,
y = H k_hat, softmax weights p_t, output o), with rho = 2^-11 / sqrt(3), the root mean square
of a rounding to fp16 whose half step is 2^-11 relative:
  - the score of token t is off by rho sqrt(1 + 3) |q~ * y_t| (elementwise product's norm: one
    rounding of q~, three of y - its scale, its mean's product, its sum) and by rho |s_t| from the
    scale that all dims of a token share; with the weight's own rounding (rho) this moves the
    output by at most that times the spread sqrt(sum p (v_d - o_d)^2) (Cauchy-Schwarz, so errors
    that the tokens share through q~ are covered);
  - the rows of V add sqrt(3) rho sqrt(sum p^2 |v_t|^2 / 128) from independent roundings that H
    spreads over the dims, and rho sqrt(sum p^2 v_td^2) from the shared scale.
Six of these root mean squares, the half step of the output type, and one row in 2^22 for the
fp32 sums and the approximate exponential."""
from __future__ import annotations

import numpy as np
import torch

import cache_testlib as ct

RHO = 2.0 ** -11 / np.sqrt(3.0)


def hadamard():
    h = np.ones((1, 1))
    while h.shape[0] < 128:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(128.0)


def reference(q, k, v, scale):
    """q [g, 128], k / v [n, 128] (fp64 numpy) -> (out, root-mean-square terms without the output's rounding)."""
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = q @ k.T * scale
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = p @ v
    h = hadamard()
    qr, kr = (q @ h) * scale, k @ h
    ds = 2 * RHO * np.sqrt((qr ** 2) @ (kr ** 2).T) + RHO * np.abs(s)
    spread = np.sqrt(np.maximum(p @ v ** 2 - out ** 2, 0.0))
    dw = np.sqrt((p * (ds + RHO) ** 2).sum(1, keepdims=True))
    dv = np.sqrt(3.0) * RHO * np.sqrt((p ** 2) @ (v ** 2).sum(1, keepdims=True) / 128) + RHO * np.sqrt((p ** 2) @ v ** 2)
    return out, dw * spread + dv


def tolerance(out, rms, dtype):
    return 6 * rms + np.abs(out) * torch.finfo(dtype).eps / 2 + np.abs(out).max(-1, keepdims=True) * 2.0 ** -22 + 2.0 ** -25


def check(pk, pv, kc, vc, q, out, cbk, cbv, mk, mv, scale, chunk=0, pick=None, skip_nan=False):
    """Every output row (of the (b, h) in `pick`) against the definition.  chunk 0: decode."""
    B, H = kc.batch, kc.n_kv_heads
    qf = q.double().cpu().numpy()
    got = out.double().cpu().numpy()
    if not chunk:
        qf, got = qf[:, None], got[:, None]
    g = qf.shape[2] // H
    prefix = {h: (ct.rows(pk, 0, h, cbk, mk), ct.rows(pv, 0, h, cbv, mv)) for h in range(H)}
    worst = 0.0
    for b in range(B):
        for h in range(H):
            if pick is not None and (b, h) not in pick:
                continue
            ok, ov = ct.rows(kc, b, h, cbk, mk), ct.rows(vc, b, h, cbv, mv)
            nw = int(kc.n_window[b, h])
            for c in range(qf.shape[1]):
                hide = min(nw, max(0, qf.shape[1] - 1 - c))
                k = np.concatenate([prefix[h][0], ok[:len(ok) - hide]])
                v = np.concatenate([prefix[h][1], ov[:len(ov) - hide]])
                want, rms = reference(qf[b, c, h * g:(h + 1) * g], k, v, scale)
                tol = tolerance(want, rms, out.dtype)
                diff = np.abs(got[b, c, h * g:(h + 1) * g] - want)
                assert np.isfinite(got[b, c, h * g:(h + 1) * g]).all(), f"(b={b}, c={c}, h={h}): not finite"
                worst = max(worst, float((diff / tol).max()))
                assert (diff <= tol).all(), f"(b={b}, c={c}, h={h}): {float((diff / tol).max()):.3g} tolerances off"
    return worst

"""Random compressed caches for the tests of the operators that read them: any mode,
with or without double quantization, ragged counts per (b, h), and stored bytes past the
counts that no result may depend on (NaN norms, means and window rows)."""
from __future__ import annotations

import numpy as np

import nsn_testlib as tl
from oracle import nsn_oracle as orc


def random_cache(counts, capacity, window, mode, dq, seed, device="cuda", s1_range=(0.5, 3.0), poison=True):
    """A Cache whose sequence (b, h) holds counts[b][h] = (n_quant, n_window) random tokens."""
    import torch

    from calibration_free_vector_b200 import nsn
    B, H = len(counts), len(counts[0])
    rng = np.random.default_rng(seed)
    c = nsn.Cache(B, H, capacity, window, mode, device=device, double_quant=dq)
    put = lambda t, a: t.copy_(torch.from_numpy(np.ascontiguousarray(a)))  # noqa: E731
    put(c.codes, rng.integers(0, 256, c.codes.shape, dtype=np.uint8))
    if c.signs is not None:
        put(c.signs, rng.integers(0, 256, c.signs.shape, dtype=np.uint8))
    nq = np.array([[n for n, _ in row] for row in counts])
    nw = np.array([[w for _, w in row] for row in counts])
    past = (np.arange(capacity) >= nq[..., None]) & poison
    past_block = (np.arange(capacity // 128) * 128 >= nq[..., None]) & poison
    s1 = rng.uniform(*s1_range, past.shape).astype(np.float16)
    s2 = rng.uniform(0.5, 1.5, past.shape).astype(np.float16)
    s1[past] = s2[past] = np.nan
    if dq:
        put(c.norms, s2)
        put(c.s1_levels, rng.integers(0, 256, c.s1_levels.shape, dtype=np.uint8))
        put(c.means, rng.integers(0, 256, c.means.shape, dtype=np.uint8))
        par = np.zeros(c.dq_params.shape, dtype=np.float16)
        par[..., 0] = rng.uniform(0.5, 1.0, par.shape[:-1])
        par[..., 1] = par[..., 0] + rng.uniform(0.1, 2.0, par.shape[:-1])
        par[..., 2] = rng.uniform(-0.6, -0.1, par.shape[:-1])
        par[..., 3] = par[..., 2] + rng.uniform(0.2, 1.2, par.shape[:-1])
        par[past_block] = np.nan
        put(c.dq_params, par)
    else:
        put(c.norms, np.stack([s1, s2], -1))
        o = rng.normal(0.0, 0.3, c.means.shape).astype(np.float16)
        o[past_block] = np.nan
        put(c.means, o)
    if window:
        w = rng.normal(size=c.window_buf.shape).astype(np.float16)
        w[(np.arange(window) >= nw[..., None]) & poison] = np.nan
        put(c.window_buf, w)
    put(c.n_quant, nq.astype(np.int32))
    put(c.n_window, nw.astype(np.int32))
    return c


def rows(cache, b, h, cb, mode):
    """Every token of one (b, h) by the definition in fp64: [n, 128]."""
    g = tl.read_cache(cache, b, h)
    x = orc.dequantize(g["codes"], g["signs"], g["s1"], g["s2"], g["o"], np.asarray(cb, np.float64), mode)
    return np.concatenate([x.reshape(-1, 128), g["window"].reshape(-1, 128)])


def terms(cache, b, h, cb, mode):
    """Sum of the absolute values that the transform adds up for each token of one (b, h): the scale of its rounding."""
    g = tl.read_cache(cache, b, h)
    n = g["codes"].shape[0]
    u = orc.reconstruct_sub(g["codes"].reshape(-1), None if g["signs"] is None else g["signs"].reshape(-1),
                            np.asarray(cb, np.float64), mode).reshape(n, 128)
    o = g["o"][np.arange(n) // 128] if n else np.zeros((0, 128))
    a = ((np.abs(u) * g["s2"][:, None] + np.abs(o)) * np.abs(g["s1"])[:, None]).sum(1) / np.sqrt(128)
    return np.concatenate([a, np.zeros(g["window"].shape[0])])

"""Plain 64-bit references of the MX4 operators and of expert routing, for the tests (numpy, CPU)."""
import math

import numpy as np
import torch

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
EPS32 = 2.0 ** -24  # half a step of fp32, relative


def quantize(x):
    """(codes [..., K/2], scales [..., 4*ceil(K/128)]) of a float array, from the format's definition."""
    x = np.asarray(x, np.float64)
    K = x.shape[-1]
    b = x.reshape(*x.shape[:-1], K // 32, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros((*x.shape[:-1], 4 * ((K + 127) // 128)), np.uint8)
    for at in np.ndindex(b.shape[:-1]):
        v = b[at]
        if not np.isfinite(v).all():
            scales[at] = 255
            continue
        top = np.abs(v).max()
        e = max(math.frexp(top)[1] - 3, -127) if top > 0 else -127
        scales[at] = e + 127
        d = np.abs(np.abs(v)[:, None] / 2.0 ** e - MAGNITUDES[None, :])
        for i in range(32):
            best = np.flatnonzero(d[i] == d[i].min())
            c = best[best % 2 == 0][0] if len(best) > 1 else best[0]  # ties go to the even code
            codes[at][i] = c | (8 if np.signbit(v[i]) else 0)
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales


def values(codes, scales):
    """fp64 values [..., K] of codes and scales (numpy uint8 arrays)."""
    codes = np.asarray(codes)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    K = c.shape[-1]
    s = np.repeat(np.asarray(scales)[..., : K // 32].astype(np.float64), 32, axis=-1)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0) * np.exp2(s - 127)
    return np.where(s == 255, np.nan, v)


def product(x, w):
    """(x w^T, its bound): products are exact and sums of K terms in fp32 are off by at most
    K * 2^-23 of the sum of magnitudes, whatever the order and whether additions round or truncate."""
    y = x @ w.T
    return y, x.shape[-1] * 2 * EPS32 * (np.abs(x) @ np.abs(w).T)


def route(logits, k, renormalize):
    """(ids, weights fp64) of a float64 array of logits."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t, row in enumerate(logits):
        live = [e for e in range(E) if row[e] > -np.inf]  # NaN compares false
        order = sorted(live, key=lambda e: (-row[e], e))[:k]
        if not order:
            continue
        top = row[order[0]]
        w = {e: 1.0 if row[e] == top else math.exp(row[e] - top) for e in live}
        total = sum(w[e] for e in (order if renormalize else live))
        for j, e in enumerate(order):
            ids[t, j], weights[t, j] = e, w[e] / total
    return ids, weights


def moe(x, ids, weights, gate, up, down):
    """(y, its bound) of the experts' products; gate, up [E, I, H] and down [E, H, I] in fp64.

    The bound follows the errors: gate and up carry their product's bound; silu's slope is at most 1.1
    and expf, the division and the two multiplications add under 16 half-steps; the hidden value keeps
    24 bits; the last sum has k * 3 I terms (three planes) and the weights' multiplications."""
    T, H = x.shape
    E, I, _ = gate.shape
    y, b = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            g, bg = product(x[t:t + 1], gate[e])
            u, bu = product(x[t:t + 1], up[e])
            a = g / (1 + np.exp(-g))
            h = a * u
            bh = 1.1 * bg * (np.abs(u) + bu) + np.abs(a) * bu + 18 * EPS32 * np.abs(h)
            y[t] += weights[t, j] * (h @ down[e].T)[0]
            size = (np.abs(h) @ np.abs(down[e]).T)[0]
            b[t] += abs(weights[t, j]) * ((bh @ np.abs(down[e]).T)[0] + (3 * I + 16) * 2 * EPS32 * size)
    return y, b + len(ids[0]) * 2 * EPS32 * np.abs(y)


def random_mx4(shape, seed, device, low=110, high=126):
    """Codes and scales drawn at random (every code, exponents low..high-1), as an Mx4Tensor."""
    from decode_gemv_thinkbit_amd import qlinear as ql

    rng = np.random.default_rng(seed)
    K = shape[-1]
    codes = rng.integers(0, 256, (*shape[:-1], K // 2), dtype=np.uint8)
    scales = rng.integers(low, high, (*shape[:-1], 4 * ((K + 127) // 128)), dtype=np.uint8)
    return ql.Mx4Tensor(torch.from_numpy(codes).to(device), torch.from_numpy(scales).to(device))


def host(t):
    """fp64 values of an Mx4Tensor."""
    return values(t.codes.cpu().numpy(), t.scales.cpu().numpy())

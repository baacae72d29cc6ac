"""The operators between the products (test oracle only), plain numpy in fp64: activations of an epilogue and their
derivatives, layer norm and its gradients, an expert layer."""

from __future__ import annotations

import math

import numpy as np
import torch


def activation_parts(z, act):
    """act(z), act'(z) and the sum of magnitudes that act' is made of."""
    z = np.asarray(z, np.float64)
    if act == "none":
        return z, np.ones_like(z), np.ones_like(z)
    if act == "relu":
        return np.maximum(z, 0), (z > 0) * 1.0, (z > 0) * 1.0
    if act == "gelu":
        t = torch.from_numpy(np.abs(z))
        tail = (0.5 * torch.special.erfcx(t / math.sqrt(2)) * torch.exp(-t * t / 2)).numpy()
        up = np.where(z < 0, tail, 1 - tail)
        zphi = np.where(np.abs(z) > 60, 0.0, z * np.exp(-np.minimum(np.abs(z), 60) ** 2 / 2) / math.sqrt(2 * math.pi))
        return z * up, up + zphi, up + np.abs(zphi) + tail
    if act == "silu":
        f, df = z, np.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        far = np.clip(z, -1e3, 1e3)  # sigma is 0 or 1 there
        f, df = c * far * (1 + 0.044715 * far * far), c * (1 + 3 * 0.044715 * far * far)
    e = np.exp(-np.abs(f))
    s, r = np.where(f >= 0, 1 / (1 + e), e / (1 + e)), np.where(f >= 0, e / (1 + e), 1 / (1 + e))
    bend = np.where(e == 0, 0.0, z * s * r * df)
    return z * s, s + bend, s + np.abs(bend)


def layernorm(h, gamma, beta, eps):
    """(mean [R], rstd [R], y [R, d]) of rows h [R, d]; beta may be None."""
    h = np.asarray(h, np.float64)
    mean = h.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (h - mean) * rstd * np.asarray(gamma, np.float64)
    return mean[:, 0], rstd[:, 0], y if beta is None else y + np.asarray(beta, np.float64)


def layernorm_grad(dy, h, gamma, mean, rstd):
    """(dx, terms of dgamma, terms of dbeta), each [R, d]; the weights' gradients are the sums over the rows."""
    dy, h, gamma = (np.asarray(t, np.float64) for t in (dy, h, gamma))
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (h - mean) * rstd
    g = dy * gamma
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, dy * xh, dy


def moe_layer(x, ids, weights, w1, w2):
    """(out [T, H], bound-making magnitudes [T, H]) of sum_j weights[t,j] w2[e] (silu(g) u), [g | u] = w1[e] x[t];
    w1 [E, 2I, H] and w2 [E, H, I] are the dequantized weights.  The second result is
    sum_j |weights| |w2| (|y| + what y moves by for a relative error of 1 of every sum's magnitudes)."""
    x = np.asarray(x, np.float64)
    out, size = np.zeros_like(x), np.zeros_like(x)
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w1.shape[0]:
                continue
            g, u = np.split(w1[e] @ x[t], 2)
            ga, ua = np.split(np.abs(w1[e]) @ np.abs(x[t]), 2)
            silu, slope, _ = activation_parts(g, "silu")
            moved = np.abs(slope * u) * ga + np.abs(silu) * ua
            out[t] += weights[t, j] * (w2[e] @ (silu * u))
            size[t] += abs(weights[t, j]) * (np.abs(w2[e]) @ (np.abs(silu * u) + moved))
    return out, size

"""4-bit weight tensors and the plain fp64 forms of their operators, for the tests."""
import numpy as np
import torch


def make_w4(shape, group, scale="fp32", zeros=False, seed=0):
    """Random (codes, scales, zeros) of a weight tensor [.., N, K]; all 16 codes occur."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    rows, K = tuple(shape[:-1]), shape[-1]
    groups = -(-K // group)
    codes = torch.randint(0, 256, (*rows, K // 2), generator=g, dtype=torch.uint8)
    scales = 0.005 + 0.02 * torch.rand(*rows, groups, generator=g)
    scales = scales.to({"fp32": torch.float32, "bf16": torch.bfloat16}[scale])
    z = torch.randint(0, 16, (*rows, groups), generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def values(codes, scales, zeros, group):
    """fp64 [.., N, K] of a weight tensor."""
    c = codes.numpy()
    K = 2 * c.shape[-1]
    q = np.empty((*c.shape[:-1], K))
    q[..., 0::2] = c & 15
    q[..., 1::2] = c >> 4
    at = np.arange(K) // group
    z = 8.0 if zeros is None else zeros.numpy().astype(np.float64)[..., at]
    return (q - z) * scales.double().numpy()[..., at]


def matvec(x, v):
    """(x v^T, |x| |v|^T) in fp64: the result and the scale of its rounding errors."""
    x = x.double().numpy()
    return x @ v.T, np.abs(x) @ np.abs(v).T


def sum_bound(K):
    """Relative to the sum of the magnitudes: a product passes at most 12 MMA steps of a
    group, the K/128 group sums of a row and 52 more operations that scale and join
    sums, each off by at most 2^-23 of what it has summed."""
    return (K / 128 + 64) * 2.0 ** -23


BF16 = 2.0 ** -8  # a rounding to bf16, relative to the value


def route(logits, k, renorm):
    l = logits.double().numpy()
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    p = np.exp(l - l.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    w = np.take_along_axis(p, ids, axis=1)
    return ids, w / w.sum(axis=1, keepdims=True) if renorm else w


def layer(x, logits, v13, v2, k, renorm):
    """The layer in fp64: dict(ids, weights, counts, out, mag); mag[t, r] is the sum of
    the magnitudes that make up out[t, r]."""
    x = x.double().numpy()
    T, I = x.shape[0], v2.shape[2]
    ids, w = route(logits, k, renorm)
    out, mag = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            gu = v13[e] @ x[t]
            g, u = gu[:I], gu[I:]
            h = g / (1 + np.exp(-g)) * u
            out[t] += w[t, j] * (v2[e] @ h)
            mag[t] += w[t, j] * (np.abs(v2[e]) @ np.abs(h))
    return dict(ids=ids, weights=w, out=out, mag=mag,
                counts=np.bincount(ids.ravel(), minlength=v13.shape[0]))

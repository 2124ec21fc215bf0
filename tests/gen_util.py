"""Shared helpers of the generation operators' tests: paged caches over
shuffled pages in several layouts, 64-bit values and derived error bounds."""
import math

import numpy as np

import oracle
from bitwise_reproducible_fp32_gb300 import detlib
from gpu_util import torch

F = np.float32
U = 2.0 ** -24          # half a float step, relative


def turns_of(rot, factor=1.0, theta=10000.0):
    """Fixed-point turns of rot / 2 frequencies, as numpy uint64."""
    return detlib.rope_turns(rot, theta, factor, device="cpu").numpy().view(np.uint64)


def rotate64(x, pos, turns, heads, d, half=False, inverse=False):
    """The rotary formula in 64 bits on rows of heads x d."""
    rot = 2 * turns.size
    phase = (np.maximum(pos, 0).astype(np.uint64)[:, None] * turns[None]).astype(np.int64)
    z = np.exp((-1j if inverse else 1j) * phase.astype(np.float64) * (math.pi / 2.0 ** 63))
    z = np.where((pos < 0)[:, None], 1.0, z)[:, None, :]
    X = x.astype(np.float64).reshape(len(x), heads, d)
    out = X.copy()
    i0, i1 = ((slice(0, rot // 2), slice(rot // 2, rot)) if half
              else (slice(0, rot, 2), slice(1, rot, 2)))
    w = (X[..., i0] + 1j * X[..., i1]) * z
    out[..., i0], out[..., i1] = w.real, w.imag
    return out.reshape(len(x), -1)


LAYOUTS = ("token", "head", "packed", "offset")


def make_cache(pages, ps, G, d, layout="token", fill=float("nan")):
    """(k, v) caches pages x ps x G x d on the GPU: token-major, head-major, K and
    V in one tensor with padded rows, or one float past 16-byte alignment."""
    if layout == "token":
        return tuple(torch.full((pages, ps, G, d), fill, device="cuda") for _ in range(2))
    if layout == "head":
        return tuple(torch.full((pages, G, ps, d), fill, device="cuda").transpose(1, 2)
                     for _ in range(2))
    if layout == "packed":
        both = torch.full((pages, 2, ps, G, (d + 3) // 4 * 4 + 4), fill, device="cuda")
        return both[:, 0, :, :, :d], both[:, 1, :, :, :d]
    if layout == "offset":
        return tuple(torch.full((pages * ps * G * d + 1,), fill, device="cuda")[1:]
                     .view(pages, ps, G, d) for _ in range(2))
    raise ValueError(layout)


def fill_cache(lens, ps, G, d, layout, rng, spare=2, K=None, V=None):
    """A cache over shuffled pages holding requests of these lengths: (k, v, table,
    per-request K, per-request V), the slots no token owns left NaN."""
    lens = np.asarray(lens)
    owned = -(-lens // ps)
    total = int(owned.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, int(owned.max()))), -7, np.int32)
    kc, vc = make_cache(total, ps, G, d, layout)
    kh, vh = (np.full((total, ps, G, d), np.nan, F) for _ in range(2))
    Ks, Vs, at = [], [], 0
    for b, n in enumerate(lens):
        ids = perm[at:at + owned[b]]
        at += owned[b]
        table[b, :owned[b]] = ids
        k = rng.standard_normal((n, G, d)).astype(F) if K is None else K[b]
        v = rng.standard_normal((n, G, d)).astype(F) if V is None else V[b]
        j = np.arange(n)
        kh[ids[j // ps], j % ps], vh[ids[j // ps], j % ps] = k, v
        Ks.append(k)
        Vs.append(v)
    kc.copy_(torch.from_numpy(kh))
    vc.copy_(torch.from_numpy(vh))
    return kc, vc, torch.from_numpy(table).cuda(), Ks, Vs


def decode_oracle(q, Ks, Vs, H, scale):
    B = len(Ks)
    G, d = Ks[0].shape[1:]
    out = np.zeros((B, H * d), F)
    for b in range(B):
        for h in range(H):
            g = h // (H // G)
            out[b, h * d:(h + 1) * d] = oracle.decode_attention(
                q[b, h * d:(h + 1) * d], Ks[b][:, g], Vs[b][:, g], scale)
    return out


def decode64(q, K, V, scale):
    """(value, bound) of one head in 64 bits. Score: d fmaf roundings of at most
    U * sum |q k|, one for the scale, one for x - m; each exp within a step (2U); S:
    at most n / 1024 * 4 + 8 adds; 1/S, p: one each; P V: 256 fmaf and one add a
    chunk."""
    n, d = K.shape
    q, K, V = (a.astype(np.float64) for a in (q, K, V))
    s = K @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    ds = scale * (np.abs(K) @ np.abs(q)).max() * (d + 1) * U + 2 * np.abs(s - s.max()).max() * U
    rel = 2 * ds + (2 + 4 * math.ceil(n / 1024) + 8 + 2 + min(n, 256) + math.ceil(n / 256)) * U
    return p @ V, (p @ np.abs(V)) * rel * 1.01 + 1e-37


def logprob64(x, y):
    """(logp, entropy, bounds of both) in 64 bits, rows with finite maxima. d = x - m
    rounds by U |d|, exp within a step (2U): e is off by U (|d| + 2) relative; S:
    at most 4 ceil(V / 1024) + 8 adds; log within a step; T: at most one fmaf for each
    of ceil(V / 4096) elements of a chain, an add a block and 12 adds."""
    x = x.astype(np.float64)
    d = x - x.max(1, keepdims=True)
    e = np.exp(d)
    S = e.sum(1)
    p = e / S[:, None]
    dd = np.where(p > 0, d, 0.0)
    logS = np.log(S)
    dy = d[np.arange(len(x)), np.maximum(y, 0)]
    T = (p * dd).sum(1)
    V = x.shape[1]
    wS = (p * np.abs(dd)).sum(1) + 2 + 4 * math.ceil(V / 1024) + 8
    logp = dy - logS
    b1 = U * (np.abs(dy) + 2 * np.abs(logS) + np.abs(logp) + wS) * 1.01 + 1e-37
    ent = logS - T
    b2 = U * (2 * np.abs(logS) + np.abs(ent) + wS + np.abs(T) * (wS + 2)
              + (p * np.abs(dd) * (2 * np.abs(dd) + 2 + math.ceil(V / 4096)
                                         + math.ceil(V / 16384) + 12)).sum(1)) * 1.01
    return logp, ent, b1, b2 + 1e-37

"""Plain 64-bit forms of the sampled step's operators, for the tests: norm and rotation, drawn paths,
verification. Written from the formulas, a row at a time."""

from __future__ import annotations

import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def turns(positions, frequencies):
    """Angles in turns, exact: the low 64 bits of position * frequency, as a fraction in [-1/2, 1/2)."""
    out = np.zeros((len(positions), len(frequencies)))
    for i, p in enumerate(positions):
        for j, f in enumerate(frequencies):
            t = (int(p) * int(f)) % 2 ** 64
            out[i, j] = (t - 2 ** 64 if t >= 2 ** 63 else t) / 2.0 ** 64
    return torch.from_numpy(out)


def norm_rope(x, weight, eps, angle, interleaved, scale):
    """Normed and rotated heads in 64 bits, x [T, heads, D], angle [T, pairs] turns; and for each value
    what its fp32 error scales with."""
    x = x.detach().cpu().double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.detach().cpu().double()
    y, size = x.clone(), x.abs()
    n = angle.shape[1]
    if n:
        c = torch.cos(2 * math.pi * angle)[:, None] * scale
        s = torch.sin(2 * math.pi * angle)[:, None] * scale
        at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        a, b = x[..., at[0]], x[..., at[1]]
        y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
        size = size.clone()
        size[..., at[0]] = size[..., at[1]] = (a.abs() + b.abs()) * abs(scale)
    return y, size


def close_heads(got, want, size, dtype):
    """fp32 error: the sum of squares of up to 256 values is 16 terms deep in a thread and 4 across,
    so within 2^-19.5, its root within half of that, rsqrt within 2^-22, three products and a
    difference, cos and sin within 2^-22: 2^-19 of the terms' size. Then one rounding: half a step,
    which below the smallest normal number is half of the smallest subnormal one, 2^-134 in bf16 (a value of
    1e-40, say, lies between multiples of 2^-133 = 9.2e-41) and 2^-25 in fp16."""
    got = got.detach().cpu().double()
    tol = want.abs() * UNIT[dtype] + size * 2.0 ** -19 * (1 + UNIT[dtype]) + (
        2.0 ** -24 if dtype == torch.float16 else 2.0 ** -134)
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))


def close_e4m3(got, want, size, scale):
    """A rounding to e4m3 is off by half a step: 2^-4 of the value, 2^-10 below 2^-6; at the top it clamps."""
    v = (want / scale).clamp(-448, 448)
    got = got.detach().cpu().double()
    tol = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + size / scale * 2.0 ** -19
    bad = (got - v).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - v).abs() / tol).max()))


def clamp_uniform(u):
    u = float(u)
    return 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)


def _invert(w, u):
    """The smallest index whose running sum passes u times the sum of all."""
    border, so_far = u * math.fsum(w), 0.0
    last = 0
    for c, v in enumerate(w):
        so_far += v
        if v > 0:
            last = c
        if so_far > border:
            return c
    return last


def sample_path(edges, uniforms, temperatures):
    """(path [R, S], probs [R, S, K])."""
    E = np.asarray(edges.detach().cpu().double())
    u = uniforms.detach().cpu().double().numpy()
    R, S, K, _ = E.shape
    path, probs = np.zeros((R, S), np.int64), np.zeros((R, S, K))
    for r in range(R):
        t, before = float(temperatures[r]), 0
        for p in range(S):
            row = E[r, p, before]
            known = row[~np.isnan(row)]
            top = known.max() if len(known) else -math.inf
            if not t > 0 or math.isinf(top):
                pick = int(np.argmax(row == top)) if len(known) else 0
                probs[r, p, pick] = 1.0
            else:
                z = np.where(np.isnan(row) | (row == -math.inf), -math.inf, (row - top) / t)
                z[row == top] = 0.0
                if math.isinf(t):
                    z = np.where(np.isneginf(z), z, 0.0)
                w = np.exp(z)
                probs[r, p] = w / math.fsum(w)
                pick = _invert(w.tolist(), clamp_uniform(u[r, p]))
            path[r, p] = before = pick
    return path, probs


def target(row, t):
    """Probabilities of a row of logits in 64 bits, or None if it has none."""
    z = row.detach().cpu().double().numpy()
    if np.isnan(z).any() or np.isposinf(z).any() or np.isneginf(z).all():
        return None
    if not t > 0:
        p = np.zeros_like(z)
        p[int(np.argmax(z))] = 1.0
        return p
    with np.errstate(invalid="ignore", over="ignore"):
        d = (z - z.max()) / t if not math.isinf(t) else np.where(np.isneginf(z), -math.inf, 0.0)
    w = np.exp(d)
    return w / math.fsum(w)


def verify(logits, query_start, drafts, accept, sample, ids, probs, temperatures):
    """(tokens [R, S + 1], counts [R], logprobs [R, S + 1])."""
    start = query_start.tolist()
    drafts = drafts.cpu()
    R, S = drafts.shape
    T, V = logits.shape
    tokens, counts = np.full((R, S + 1), -1), np.zeros(R, np.int64)
    logprobs = np.zeros((R, S + 1))
    for r in range(R):
        a, b = start[r], start[r + 1]
        if a < 0 or b < a or b > T or b - a > S + 1:
            continue
        for i in range(b - a):
            p = full = target(logits[a + i], float(temperatures[r]))
            if p is None:
                break
            if i < b - a - 1:
                x = int(drafts[r, i])
                q = np.zeros(V)
                if ids is None:
                    if 0 <= x < V:
                        q[x] = 1.0
                else:
                    for c, v in zip(ids[r, i].tolist(), probs[r, i].double().tolist()):
                        if 0 <= c < V:
                            q[c] += v
                if 0 <= x < V and float(accept[r, i].double()) * q[x] < p[x]:
                    tokens[r, i] = x
                    logprobs[r, i] = math.log(p[x])
                    counts[r] = i + 1
                    continue
                rest = np.maximum(p - q, 0)
                if math.fsum(rest) > 2.0 ** -36:
                    p = rest
            u = clamp_uniform(sample[r].double())
            so_far = np.cumsum(p)
            border = u * so_far[-1]
            above = np.nonzero(so_far > border)[0]
            x = int(above[0]) if len(above) else int(np.nonzero(p)[0][-1])
            tokens[r, i] = x
            logprobs[r, i] = math.log(full[x])
            counts[r] = i + 1
            break
    return tokens, counts, logprobs

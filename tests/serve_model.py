"""Plain models of what include/tb_serve.h promises, in 64 bits or in whole numbers, for the tests."""
import math

import torch

STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
LIMITS = {torch.float16: (-23, 13), torch.bfloat16: (-126, 125)}


def head_bytes(dim):
    return dim // 2 + (dim // 32 + 3) // 4 * 4


def encode(x):
    """x [..., dim] of 16 bits -> uint8 [..., head_bytes(dim)], element by element."""
    dim, (low, high) = x.shape[-1], LIMITS[x.dtype]
    rows = x.reshape(-1, dim).double().tolist()
    out = torch.zeros(len(rows), head_bytes(dim), dtype=torch.uint8)
    for r, row in enumerate(rows):
        for b in range(dim // 32):
            block = row[32 * b:32 * b + 32]
            if not all(math.isfinite(v) for v in block):
                out[r, dim // 2 + b] = 255
                continue
            top = max(abs(v) for v in block)
            e = low
            while e < high and top >= 7 * 2.0 ** e:
                e += 1
            out[r, dim // 2 + b] = e + 127
            for i, v in enumerate(block):
                a = abs(v) / 2.0 ** e
                best = min(range(8), key=lambda c: (abs(STEPS[c] - a), c % 2))
                code = best + (8 if math.copysign(1, v) < 0 else 0)
                out[r, 16 * b + i // 2] |= code << (4 * (i % 2))
    return out.view(*x.shape[:-1], -1)


def decode(raw, dim):
    """What the bytes stand for, float64 [..., dim]."""
    flat = raw.reshape(-1, raw.shape[-1]).long()
    code = torch.stack([flat[:, :dim // 2] & 15, flat[:, :dim // 2] >> 4], 2).view(len(flat), dim)
    value = torch.tensor(STEPS + [-v for v in STEPS], dtype=torch.float64)[code]
    power = flat[:, dim // 2:dim // 2 + dim // 32]
    scale = torch.where(power == 255, math.nan, torch.exp2(power.double() - 127))
    return (value.view(len(flat), -1, 32) * scale[:, :, None]).view(*raw.shape[:-1], dim)


def window_attention(model, layer, q, k, v, seqs, mask=None, nodes=None, scale=None, window=None, sinks=0, depths=None):
    """As cache_model.attention, with a window: (out, lse, A, S, V)."""
    b, t, hq, d = q.shape
    hk = k.shape[2]
    g = hq // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(b, t, hq, d, dtype=torch.float64)
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64)
    a, s, big = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    for i in range(b):
        row = int(seqs[i])
        if not 0 <= row < model.S:
            continue
        count = t if nodes is None else min(max(int(nodes[i]), 0), t)
        n = model.lens[row]
        depth = [u if depths is None else min(max(int(depths[i, u]), 0), count - 1) for u in range(count)]
        for x in range(count):
            at = [j for j in range(n) if window is None or j < sinks or n + depth[x] - j < window]
            sees = [u for u in range(count) if (u <= x if mask is None else int(mask[i, x, u // 64]) >> (u % 64) & 1)]
            if window is not None:
                sees = [u for u in sees if n + depth[u] < sinks or depth[x] - depth[u] < window]
            if not at and not sees:
                continue
            for h in range(hk):
                key = torch.cat([model.context(2 * layer, row, h)[at], k[i, sees, h].double()])
                val = torch.cat([model.context(2 * layer + 1, row, h)[at], v[i, sees, h].double()])
                qq = q[i, x, h * g:(h + 1) * g].double()
                y = qq @ key.T * scale
                z = torch.logsumexp(y, 1)
                w = torch.exp(y - z[:, None])
                out[i, x, h * g:(h + 1) * g] = w @ val
                lse[i, x, h * g:(h + 1) * g] = z
                a[i, x, h * g:(h + 1) * g] = w @ val.abs()
                s[i, x, h * g:(h + 1) * g] = (qq.abs() @ key.abs().T * abs(scale)).amax(1)
                big[i, x, h * g:(h + 1) * g] = val.abs().max()
    return out, lse, a, s, big


def verify(probs, tokens, uniform, parents=None, draft=None, nodes=None):
    """(count, path, token) of each sequence, the walk as the header tells it."""
    b, t, vocab = probs.shape
    found = []
    for i in range(b):
        n = t if nodes is None else min(max(int(nodes[i]), 0), t)
        if n == 0:
            found.append((0, [], -1))
            continue
        path, w, z = [0], probs[i, 0].double().clone(), 1.0
        for u in range(1, n):
            parent = u - 1 if parents is None else int(parents[i, u])
            x = int(tokens[i, u])
            if not 0 <= parent < u or parent != path[-1] or not 0 <= x < vocab:
                continue
            d = 1.0 if draft is None else float(draft[i, parent, x].double())
            if float(uniform[i, u].double()) * d * z < float(w[x]):
                path.append(u)
                w, z = probs[i, u].double().clone(), 1.0
            elif draft is None:
                z -= float(w[x])
                w[x] = 0
            else:
                w = (w - z * draft[i, parent].double()).clamp(min=0)
                z = float(w.sum())
        if not bool((w > 0).any()):
            w = probs[i, path[-1]].double()
        mass = torch.cumsum(w, 0)
        token = int((mass <= float(uniform[i, 0].double()) * float(mass[-1])).sum()) if float(mass[-1]) > 0 else -1
        found.append((len(path), path, token))
    return found

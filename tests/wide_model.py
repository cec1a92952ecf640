"""serve_model.window_attention for many nodes: the same definition in 64 bits, all nodes of a sequence at once."""
import math

import torch


def seen(n, count, mask, window, sinks, depth):
    """[count, n + count]: what each node sees of the n tokens and of the nodes; mask [nodes, words] or None."""
    x = torch.arange(count)
    depth = x if depth is None else depth[:count].long().clamp(0, count - 1)
    at = torch.ones(count, n, dtype=torch.bool)
    if mask is None:
        sees = x[:, None] >= x[None, :]
    else:
        sees = (mask[:count][:, x // 64] >> (x % 64)[None, :] & 1) != 0
    if window is not None:
        j = torch.arange(n)
        at = (j < sinks)[None, :] | (n + depth[:, None] - j[None, :] < window)
        sees = sees & ((n + depth[None, :] < sinks) | (depth[:, None] - depth[None, :] < window))
    return torch.cat([at, sees], 1)


def window_attention(model, layer, q, k, v, seqs, mask=None, nodes=None, scale=None, window=None, sinks=0, depths=None):
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
        if count == 0:
            continue
        sees = seen(model.lens[row], count, None if mask is None else mask[i], window, sinks, None if depths is None else depths[i])
        some = sees.any(1)
        for h in range(hk):
            key = torch.cat([model.context(2 * layer, row, h), k[i, :count, h].double()])
            val = torch.cat([model.context(2 * layer + 1, row, h), v[i, :count, h].double()])
            for x in range(h * g, (h + 1) * g):
                qq = q[i, :count, x].double()
                y = (qq @ key.T * scale).masked_fill(~sees, -math.inf)
                z = torch.logsumexp(y, 1)
                w = torch.where(some[:, None], torch.exp(y - torch.where(some, z, 0.0)[:, None]), 0.0)
                out[i, :count, x] = w @ val
                lse[i, :count, x] = z
                a[i, :count, x] = w @ val.abs()
                s[i, :count, x] = (qq.abs() @ key.abs().T * abs(scale)).masked_fill(~sees, 0.0).amax(1)
                big[i, :count, x] = torch.where(sees, val.abs().amax(1)[None, :], 0.0).amax(1)
    return out, lse, a, s, big

"""Plain CPU references of the layer of experts, in 64 bits, and the inputs of its tests."""
import numpy as np
import torch


def pad(K):
    return -(-K // 256) * 256


def unpack_w4(w):
    """int8 codes [..., 2 * bytes] of packed rows: 32 bytes hold the groups of 16 codes 0, 2, 1, 3; byte j of a
    group's first four holds codes j and 4 + j, of its last four codes 8 + j and 12 + j."""
    b = w.cpu().numpy()
    units = b.reshape(*b.shape[:-1], -1, 4, 2, 4)[..., [0, 2, 1, 3], :, :]
    lo = ((units & 15) ^ 8).astype(np.int8) - 8
    hi = ((units >> 4) ^ 8).astype(np.int8) - 8
    return torch.from_numpy(np.stack([lo, hi], -2).reshape(*b.shape[:-1], -1).astype(np.int8))


def random_weight(E, N, K, seed, dev):
    """(packed rows [E, N, K_pad / 2], scales [E, N]); any bytes are codes (-8 too), columns past K hold some."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 256, (E, N, pad(K) // 2), generator=g, dtype=torch.uint8)
    w = torch.where((w & 15) == 8, w & 240, w)         # -8 is no code of the form
    w = torch.where((w >> 4) == 8, w & 15, w)
    return w.to(dev), (K ** -0.5 * (0.1 + torch.rand(E, N, generator=g))).to(dev)


def random_rows(M, K, seed, dev):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (M, pad(K)), generator=g, dtype=torch.int16).to(torch.int8)
    return q.to(dev), (0.001 + 0.02 * torch.rand(M, generator=g)).to(dev)


def random_choices(T, k, E, seed, dev, none=0.0, repeats=False, skew=1.0):
    """ids [T, k] int32 and weights; some experts are chosen far more often than others."""
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(T, E, generator=g).log().neg().log().neg() + skew * torch.randn(E, generator=g)
    ids = torch.multinomial(torch.softmax(x, 1), k, replacement=True, generator=g) if repeats else x.topk(k, 1).indices
    ids = ids.int()
    if none:
        ids[torch.rand(T, k, generator=g) < none] = -1
    return ids.to(dev), torch.rand(T, k, generator=g).to(dev)


def plan(ids, E, first=0):
    flat = ids.cpu().flatten().tolist()
    rows, offsets = [], [0]
    for e in range(first, first + E):
        rows += [s for s, x in enumerate(flat) if x == e]
        offsets.append(len(rows))
    return offsets, rows + [-1] * (len(flat) - len(rows))


def route(logits, k, bias=None, G=1, top_groups=1, group_sum=2, sigmoid=False, renorm=True, scale=1.0):
    """ids and weights (float64), one row after another."""
    T, E = logits.shape
    L = logits.double().cpu().numpy()
    B = None if bias is None else bias.double().cpu().numpy()
    ids, out = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = L[t]
        ok = l > -np.inf                                # neither -inf nor NaN
        if not ok.any():
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                s = 1 / (1 + np.exp(-l))
            else:
                top = l[ok].max()
                s = np.where(l == top, 1.0, np.exp(l - top))
                s = np.where(ok, s, 0.0)
                s = s / s.sum()
            key = np.where(ok, l if B is None else s + B, -np.inf)
        key[np.isnan(key)] = -np.inf
        if top_groups < G:
            value = np.where(key > -np.inf, s if B is None and group_sum == 2 else key, -np.inf)
            best = []
            for v in value.reshape(G, -1):
                v = np.sort(v[v > -np.inf])[::-1][:group_sum]
                best.append(v.sum() if len(v) else -np.inf)
            order = sorted(range(G), key=lambda g: (-best[g], g))[:top_groups]
            kept = np.repeat(np.isin(np.arange(G), order), E // G)
            key = np.where(kept, key, -np.inf)
        chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:k]
        w = s[chosen] * float(np.float32(scale))
        if renorm:
            total = s[chosen].sum()
            w = w / total if total > 0 else np.zeros_like(w)
        ids[t, :len(chosen)], out[t, :len(chosen)] = chosen, w
    return ids, out


def sums(a, w, offsets, rows, gather):
    """[listed rows, N] int64 sums of the codes in the plan's order."""
    codes, a = unpack_w4(w).double(), a.cpu().double()
    out = []
    for e in range(len(offsets) - 1):
        at = torch.tensor(rows[offsets[e]:offsets[e + 1]], dtype=torch.long) // gather if gather else \
            torch.arange(offsets[e], offsets[e + 1])
        out.append(a[at] @ codes[e].t())                # exact: below 2^53
    return torch.cat(out).long()


def scaled(acc, a_scale, b_scale, bias, offsets, rows, gather):
    """(values, sum of the magnitudes that are added) in float64."""
    n = offsets[-1]
    e = torch.repeat_interleave(torch.arange(len(offsets) - 1), torch.tensor(offsets).diff())
    at = torch.tensor(rows[:n], dtype=torch.long) // gather if gather else torch.arange(n)
    v = acc.double() * a_scale.cpu().double()[at][:, None] * b_scale.cpu().double()[e]
    size = v.abs()
    if bias is not None:
        b = bias.cpu().double()[e]
        v, size = v + b, size + b.abs()
    return v, size


def hadamard():
    m = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(8):
        m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)])
    return m / 16

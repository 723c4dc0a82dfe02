"""Plain 64-bit references of the 8-bit cache's operators, and inputs for their tests."""
import math

import torch

import rotated_bit_linear_amd as rbl
from helpers import dev

F8 = torch.float8_e4m3fn
PAGE = 64
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Batch:
    """A ragged batch (new tokens and cached tokens of each sequence) with shuffled pages."""

    def __init__(self, new, kv, seed=0, spare=2, extra_columns=1):
        self.new, self.kv, self.B, self.T = list(new), list(kv), len(new), sum(new)
        g = torch.Generator().manual_seed(seed)
        need = [-(-k // PAGE) for k in kv]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).int()
        table = torch.full((self.B, max(need + [0]) + extra_columns), -1, dtype=torch.int32)
        at = 0
        for b, p in enumerate(need):
            table[b, :p] = order[at:at + p]
            at += p
        self.table_cpu = table
        self.unused = order[at:].long()
        self.start = [sum(self.new[:b]) for b in range(self.B)]
        self.cu = torch.tensor(self.start + [self.T], dtype=torch.int32).to(dev())
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32).to(dev())
        self.table = table.to(dev())
        self.max_q, self.max_kv = max(self.new + [0]), max(self.kv + [0])

    def page(self, b, p):
        return int(self.table_cpu[b, p])


def random_cache(n_pages, Hkv, D, seed, spread=3):
    """Codes of normal data against power-of-two scales that differ from page to page."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for shape in ((n_pages, Hkv, PAGE, D), (n_pages, Hkv, D, PAGE)):
        x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (n_pages, Hkv, 1, 1), generator=g).float())
        s = torch.ldexp(torch.ones(n_pages, Hkv), torch.frexp(x.abs().amax((2, 3)) / 448).exponent)
        out += [(x / s[..., None, None]).to(F8).view(torch.uint8), s]
    k, ks, v, vs = out
    return rbl.Kv8Cache(k.to(dev()), v.to(dev()), ks.to(dev()), vs.to(dev()))


def dense(cache, batch, b, h):
    """(K, V) [kv, D] of one sequence and head in FP64; pages that the table does not name are NaN."""
    ks, vs = [], []
    for p in range(-(-batch.kv[b] // PAGE)):
        i = batch.page(b, p)
        if 0 <= i < cache.n_pages:
            ks.append(cache.k[i, h].view(F8).double().cpu() * cache.k_scale[i, h].double().cpu())
            vs.append(cache.v[i, h].view(F8).double().cpu().t() * cache.v_scale[i, h].double().cpu())
        else:
            ks.append(torch.full((PAGE, cache.D), math.nan, dtype=torch.float64))
            vs.append(ks[-1])
    if not ks:
        return torch.zeros(0, cache.D, dtype=torch.float64), torch.zeros(0, cache.D, dtype=torch.float64)
    return torch.cat(ks)[: batch.kv[b]], torch.cat(vs)[: batch.kv[b]]


def attention(q, cache, batch, Hq, sm, causal):
    """(out, mean of |v| under the probabilities, largest |v|) [T, Hq, D] in FP64."""
    D, G = cache.D, Hq // cache.Hkv
    qd = q.double().cpu().view(batch.T, Hq, D)
    out, mag = torch.zeros_like(qd), torch.zeros_like(qd)
    top = torch.zeros_like(qd)
    for b in range(batch.B):
        n, kv, at = batch.new[b], batch.kv[b], batch.start[b]
        if n == 0:
            continue
        i, j = torch.arange(n)[:, None], torch.arange(kv)[None]
        see = (j <= kv - n + i) if causal else torch.ones(n, kv, dtype=torch.bool)
        missing = torch.tensor([not 0 <= batch.page(b, int(x) // PAGE) < cache.n_pages for x in range(kv)], dtype=torch.bool)
        see = see & ~missing[None]
        for h in range(cache.Hkv):
            k, v = dense(cache, batch, b, h)
            k, v = torch.where(missing[:, None], 0.0, k), torch.where(missing[:, None], 0.0, v)
            for r in range(h * G, (h + 1) * G):
                s = (qd[at:at + n, r] @ k.T) * sm
                for t in range(n):               # row by row: what a row does not see cannot touch it
                    w = see[t]
                    if not w.any():
                        continue
                    x = s[t, w]
                    p = torch.exp(x - torch.nan_to_num(x, nan=-math.inf).max())
                    out[at + t, r] = (p @ v[w]) / p.sum()
                    mag[at + t, r] = (p @ v[w].abs()) / p.sum()
                    top[at + t, r] = v[w].abs().max()
    return out, mag, top


def rotate(x, pos, freq, axis, interleaved):
    """x [T, H, D] FP64."""
    f = pos.double()[:, axis.long()] * freq
    c, s = f.cos()[:, None], f.sin()[:, None]
    D = x.shape[-1]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., : D // 2], x[..., D // 2:])
    y, z = a * c - b * s, b * c + a * s
    return torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)


def norm(x, w, eps):
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def scale_for(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax.clamp(min=2.0 ** -140) / 448)
    return torch.exp2((e - (m == 0.5).int()).double()).clamp(min=2.0 ** -126)

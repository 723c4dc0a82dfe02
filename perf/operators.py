"""Cases and plain forms of the operators around the quantized linear layers: the RMS norm that
prepares an INT8 activation, the rotary embedding that appends keys and values to the 8-bit
paged cache, and the attention that reads that cache.

`own` selects what run() computes: the plain forms below (elementary torch operations), or the
framework's kernels.  Lengths of ragged batches follow from the case alone (`spread` seeds
them); the values of every input follow from the seed.

The cache: pages of 64 tokens; keys [page, head, token, D] and values [page, head, D, token] as
E4M3 bytes, one FP32 scale for each page and head (a power of two when written by the append).
"""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases ----

def listed():
    return [
        # one token of a text encoder or a decoder step, hidden size of the QKV layer: latency
        dict(name="norm one token", op="norm", M=1, K=5376, dtype="bf16", residual=True),
        # a ragged batch with a hidden size that is no multiple of anything (row stride padded)
        dict(name="norm ragged fp16", op="norm", M=777, K=4111, dtype="fp16", residual=True),
        # the video transformer's block: every token of a clip, before qkv_proj or fc1
        dict(name="norm video", op="norm", M=19989, K=5376, dtype="bf16", residual=True),
        # FP32 rows of the FFN width, no residual
        dict(name="norm wide fp32", op="norm", M=4096, K=14336, dtype="fp32", residual=False),
        # a decoding batch: one new token in each of 64 sequences, grouped heads
        dict(name="append single tokens", op="append", B=64, new=1, past=1000, spread=1, Hq=32, Hkv=8, D=128,
             axes=1, interleaved=False, qk_norm=True, dtype="bf16"),
        # prompts continued in pages that already hold tokens; neighbouring pairs, smaller heads
        dict(name="append ragged prompts", op="append", B=7, new=1500, past=200, spread=2, Hq=24, Hkv=8, D=64,
             axes=1, interleaved=True, qk_norm=False, dtype="fp16"),
        # the video transformer's 56 heads after qkv_proj [21504, 5376]: time, height and width
        dict(name="append video", op="append", B=1, new=19989, past=0, spread=0, Hq=56, Hkv=56, D=128,
             axes=3, interleaved=False, qk_norm=True, dtype="bf16"),
        # one user's decoding step
        dict(name="attention one token", op="attention", B=1, new=1, kv=4097, spread=0, Hq=32, Hkv=8, D=128,
             causal=True, dtype="bf16"),
        # a decoding batch over ragged, long caches
        dict(name="attention single tokens", op="attention", B=64, new=1, kv=32768, spread=3, Hq=32, Hkv=8, D=128,
             causal=True, dtype="bf16"),
        # a chunk of each prompt after ten thousand cached tokens, small heads, no grouping
        dict(name="attention chunk fp16", op="attention", B=3, new=515, kv=10515, spread=4, Hq=12, Hkv=12, D=64,
             causal=True, dtype="fp16"),
        # a batch of ragged prompts
        dict(name="attention prompts", op="attention", B=5, new=4096, kv=4096, spread=5, Hq=32, Hkv=8, D=128,
             causal=True, dtype="bf16"),
        # the video transformer's whole clip, every token sees every other; a quarter of its heads
        dict(name="attention video", op="attention", B=1, new=19989, kv=19989, spread=0, Hq=14, Hkv=14, D=128,
             causal=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attention"])
    if op == "norm":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        K = _log(rng, 200, 20000)
        M = _log(rng, 1, min(40000, 19989 * 5376 * (1 if dtype == "fp32" else 2) // (2 * K)))
        return dict(op=op, M=M, K=K, dtype=dtype, residual=rng.random() < 0.7)
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    Hq = Hkv * rng.choice([1, 1, 2, 4, 7, 8])
    dtype = rng.choice(["bf16", "fp16"])
    B = _log(rng, 1, 48)
    if op == "append":
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(8000, 19989 * 56 * 128 // (B * Hq * D))))
        return dict(op=op, B=B, new=new, past=_log(rng, 1, 1500) - 1, spread=rng.randrange(1, 1 << 20), Hq=Hq,
                    Hkv=Hkv, D=D, axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5,
                    qk_norm=rng.random() < 0.5, dtype=dtype)
    kv = _log(rng, 1, 30000)
    cap = 19989 * 19989 * 14 // (B * Hq * kv * 2)          # scores of the largest listed case
    new = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, min(kv, cap, 6000)))
    return dict(op=op, B=B, new=new, kv=kv, spread=rng.randrange(1, 1 << 20), Hq=Hq, Hkv=Hkv, D=D,
                causal=rng.random() < 0.7, dtype=dtype)


def _lengths(case):
    """(new tokens, cached tokens including the new ones) of each sequence; spread 0: all at the maximum."""
    B, new = case["B"], case["new"]
    if case["op"] == "append":
        if not case["spread"]:
            return [new] * B, [new + case["past"]] * B
        r = random.Random(case["spread"])
        n = [new if new == 1 else r.randint(1, new) for _ in range(B)]
        n[r.randrange(B)] = new
        return n, [k + r.randint(0, case["past"]) for k in n]
    kv = case["kv"]
    if not case["spread"]:
        return [new] * B, [kv] * B
    r = random.Random(case["spread"])
    n = [new if new == 1 else r.randint(1, new) for _ in range(B)]
    total = [max(k, r.randint(1, kv)) if kv > new else k for k in n]
    at = r.randrange(B)
    n[at], total[at] = new, max(new, kv)
    return n, total


def work(case):
    if case["op"] == "norm":
        M, K, e = case["M"], case["K"], 4 if case["dtype"] == "fp32" else 2
        kp = -(-K // 256) * 256
        return {"bytes": M * K * e * (3 if case["residual"] else 1) + M * kp + 4 * M + 4 * K, "flops": M * K * 14}
    n, kv = _lengths(case)
    T, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        pages = sum((b - 1) // PAGE - (b - a) // PAGE + 1 for a, b in zip(n, kv))
        return {"bytes": T * D * (4 * Hq + 6 * Hkv) + 8 * pages * Hkv + 4 * T * case["axes"] + 6 * D,
                "flops": T * D * (Hq + Hkv) * 7}
    seen = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(n, kv))
    cached = sum(b for b in kv)
    return {"bytes": 4 * T * Hq * D + 2 * cached * Hkv * D + 8 * Hkv * sum(-(-b // PAGE) for b in kv),
            "flops": 4 * seen * Hq * D}


# ------------------------------------------------------------------------------ inputs ----

def _rope_table(D, axes, device):
    """Angular frequency and axis of each of the D/2 pairs: the pairs are dealt to the axes in
    runs, the first axis a quarter of them when there are several (time, then height, width)."""
    P = D // 2
    runs = [P] if axes == 1 else [P // 4, P - P // 4] if axes == 2 else [P // 4, (P - P // 4) // 2, P - P // 4 - (P - P // 4) // 2]
    freq, axis = [], []
    for a, n in enumerate(runs):
        freq += [10000.0 ** (-i / n) for i in range(n)]
        axis += [a] * n
    return (torch.tensor(freq, dtype=torch.float64, device=device), torch.tensor(axis, dtype=torch.int32, device=device))


def _fill_cache(g, pages, Hkv, D, dev):
    """A cache that holds tokens already: keys with a few strong channels, values plain."""
    chan = 1.0 + 3.0 * (torch.rand(Hkv, 1, D, generator=g, device=dev) < 0.05).float()
    out = []
    for shape, gain in (((pages, Hkv, PAGE, D), chan), ((pages, Hkv, D, PAGE), 1.0)):
        x = torch.randn(shape, generator=g, device=dev) * gain
        scale = torch.ldexp(torch.ones(pages, Hkv, device=dev), torch.frexp(x.abs().amax((2, 3)) / 448).exponent)
        out += [(x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale]
        del x
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "g": g}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        ld = -(-K // 8) * 8
        def rows():
            t = torch.empty(M, ld, dtype=dt, device=dev)
            t.normal_(generator=g)
            return t[:, :K]
        s["x"] = rows()
        s["x"][:, :: 97] *= 8                    # a few strong channels, as residual streams have
        s["residual"] = rows() if case["residual"] else None
        s["weight"] = 1 + 0.2 * torch.randn(K, generator=g, device=dev)
        return s
    n, kv = _lengths(case)
    B, T, Hq, Hkv, D = case["B"], sum(n), case["Hq"], case["Hkv"], case["D"]
    pages = [-(-b // PAGE) for b in kv]
    order = torch.randperm(sum(pages), generator=g, device=dev).int()
    table = torch.zeros(B, max(pages), dtype=torch.int32, device=dev)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    s |= {"cu": torch.tensor(cu, dtype=torch.int32, device=dev), "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
          "table": table, "max_q": max(n), "max_kv": max(kv)}
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _fill_cache(g, sum(pages), Hkv, D, dev)
    if case["op"] == "append":
        s["qkv"] = torch.empty(T, (Hq + 2 * Hkv) * D, dtype=dt, device=dev).normal_(generator=g)
        pos = torch.empty(T, case["axes"], dtype=torch.int32, device=dev)
        for b in range(B):                       # text: one running index on every axis; video: t, h, w of a grid
            i = torch.arange(kv[b] - n[b], kv[b], dtype=torch.int32, device=dev)
            w = 40
            grid = (i // (w * 24), (i // w) % 24, i % w) if case["axes"] == 3 else (i,) * case["axes"]
            pos[cu[b]:cu[b + 1]] = torch.stack(grid, 1)
        s["pos"] = pos
        s["freq"], s["axis"] = _rope_table(D, case["axes"], dev)
        both = 1 + 0.1 * torch.randn(2, D, generator=g, device=dev)
        s["q_weight"], s["k_weight"] = (both[0], both[1]) if case["qk_norm"] else (None, None)
    else:
        s["q"] = torch.empty(T, Hq * D, dtype=dt, device=dev).normal_(generator=g)
    if own:
        import rotated_bit_linear_amd as rbl
        s["cache"] = rbl.Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attention":
            need = rbl.cr_attn_kv8_workspace_bytes(T, B, s["max_q"], s["max_kv"], Hq, Hkv, D)
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
    return s


# -------------------------------------------------------------------------- one pass ----

def run(s):
    c = s["case"]
    if own:
        import rotated_bit_linear_amd as rbl
        if c["op"] == "norm":
            q, scale, total = rbl.quant_act_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"])
            return {"x_s8": q, "x_scale": scale, "sum": total}
        if c["op"] == "append":
            q = rbl.rope_append_kv8(s["qkv"], s["cache"], s["cu"], s["kv_lens"], s["table"], s["max_q"], c["Hq"],
                                    s["pos"], s["freq"], s["axis"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                    eps=EPS, interleaved=c["interleaved"])
            return {"q": q, **_cache_values(s)}
        return {"out": rbl.attn_kv8(s["q"], s["cache"], s["cu"], s["kv_lens"], s["table"], s["max_q"], s["max_kv"],
                                    c["Hq"], causal=c["causal"], workspace=s["workspace"])}
    return {"norm": _norm, "append": _append, "attention": _attention}[c["op"]](s)


def _cache_values(s):
    # the state's own buffers: the codes as the E4M3 numbers they are, and their scales
    f8 = torch.float8_e4m3fn
    return {"k": s["k"].view(f8), "v": s["v"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------------ plain forms ----

def _norm(s):
    """h = x + residual; y = h rstd weight, rotated in blocks of 256 and held in INT8 with one
    scale a row.  Rotation and codes do not depend on the row's factor rstd, so it goes into the
    scale alone; the products and butterflies are FP32 in the framework's order (stages 1 to 128)."""
    x, w = s["x"], s["weight"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    rstd = torch.rsqrt(f.double().square().mean(1) + EPS).float()
    M, K = f.shape
    z = torch.nn.functional.pad(f * w, (0, -K % 256))
    nb = z.shape[1] // 256
    for step in (1, 2, 4, 8, 16, 32, 64, 128):
        z = z.view(M, nb, 128 // step, 2, step)
        z = torch.stack((z[..., 0, :] + z[..., 1, :], z[..., 0, :] - z[..., 1, :]), 3)
    z = z.reshape(M, nb * 256)
    a = z.abs().amax(1) * 0.0625
    r = (127.0 / a.double()).float() * 0.0625
    r = torch.where(a > 0, r, 0.0)
    q = torch.round(z * r[:, None]).to(torch.int8)
    return {"x_s8": q, "x_scale": (a.double() / 127).float() * rstd, "sum": None if s["residual"] is None else h}


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] by the angles [T, 1, D/2]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _append(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    T = s["qkv"].shape[0]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    if s["q_weight"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_weight"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_weight"]
    angle = s["pos"].double()[:, s["axis"].long()] * s["freq"]           # far positions: in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(q, cos, sin, c["interleaved"]).to(s["qkv"].dtype).view(T, Hq * D)
    k = _rotate(k, cos, sin, c["interleaved"])
    # where each token goes
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    first = kv - (cu[1:] - cu[:-1])
    where = first[b] + t - cu[b]
    page, off = s["table"].long()[b, where // PAGE], where % PAGE
    old_page, old = s["table"].long().gather(1, first[:, None] // PAGE % s["table"].shape[1])[:, 0], first % PAGE
    for x, codes, scale, keys in ((k, s["k"], s["k_scale"], True), (v, s["v"], s["v_scale"], False)):
        amax = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        m, e = torch.frexp(amax)
        need = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126))
        # the first page of each run may hold older tokens: its scale only grows, its codes follow
        held = scale[old_page]
        grown = torch.where(old[:, None] > 0, torch.maximum(held, need[old_page]), need[old_page])
        f = codes[old_page].view(torch.float8_e4m3fn).float()
        f = (f * (held / grown)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        j = torch.arange(PAGE, device=cu.device)
        mask = (j[None] < old[:, None])[:, None]
        mask = mask[..., None] if keys else mask[:, :, None]
        codes[old_page] = torch.where(mask, f, codes[old_page])
        new = need.clone()
        new[old_page] = grown
        y = (x / new[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if keys:
            codes[page, :, off] = y
        else:
            codes[page, :, :, off] = y
        scale[page] = new[page]
    return {"q": q, **_cache_values(s)}


def _attention(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, Nq, Nk = Hq // Hkv, s["max_q"], s["max_kv"]
    f8 = torch.float8_e4m3fn
    cu, kv, table = s["cu"].long(), s["kv_lens"].long(), s["table"].long()
    k = s["k"].view(f8)[table].float() * s["k_scale"][table][..., None, None]      # [B, pages, Hkv, 64, D]
    v = s["v"].view(f8)[table].float() * s["v_scale"][table][..., None, None]      # [B, pages, Hkv, D, 64]
    k = k.permute(0, 2, 4, 1, 3).reshape(B * Hkv, D, -1)[..., :Nk].contiguous()
    v = v.permute(0, 2, 1, 4, 3).reshape(B * Hkv, -1, D)[:, :Nk]
    n = cu[1:] - cu[:-1]
    i, j = torch.arange(Nq, device=cu.device), torch.arange(Nk, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(B, Nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B * Hkv, G * Nq, D)
    v = torch.where(j[None, :, None] < kv.repeat_interleave(Hkv)[:, None, None], v, 0.0)
    x = torch.bmm(q, k).mul_(1 / math.sqrt(D)).view(B, Hkv, G, Nq, Nk)
    last = kv[:, None] - 1 - (n[:, None] - 1 - i if c["causal"] else 0 * i)        # the last key that a row sees
    x.masked_fill_((j > last[..., None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)                                # a row may see nothing
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B * Hkv, G * Nq, Nk), v).view(B, Hkv, G, Nq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, Nq, Hq * D)
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return {"out": o[b, t - cu[b]].to(s["q"].dtype)}


# ------------------------------------------------------------------- 64-bit definition ----

def exact(case, seed):
    s = prepare(case, seed)
    dev = s["g"].device
    if case["op"] == "norm":
        return _exact_norm(s, dev)
    n, kv = _lengths(case)
    if case["op"] == "append":
        return _exact_append(s, n, kv, dev)
    out, at = [], 0
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    f8 = torch.float8_e4m3fn
    for b in range(case["B"]):
        ids = s["table"][b, : -(-kv[b] // PAGE)].long()
        q = s["q"][at:at + n[b]].double().view(n[b], Hq, D)
        at += n[b]
        o = torch.empty(n[b], Hq, D, dtype=torch.float64, device=dev)
        for h in range(Hkv):
            k = (s["k"].view(f8)[ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[: kv[b]]
            v = s["v"].view(f8)[ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)[: kv[b]]
            for r in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                a = torch.mm(q[:, r].contiguous(), k.t().contiguous()) / math.sqrt(D)
                if case["causal"]:
                    hidden = torch.ones(n[b], kv[b], dtype=torch.bool, device=dev).triu(kv[b] - n[b] + 1)
                    a = a.masked_fill(hidden, -math.inf)
                o[:, r] = torch.mm(torch.nan_to_num(torch.softmax(a, -1)), v)
        out.append(o.view(n[b], Hq * D))
    return {"out": torch.cat(out)}


def _hadamard(dev):
    i = torch.arange(256, device=dev)
    x = i[:, None] & i[None]
    for sh in (4, 2, 1):
        x = x ^ (x >> sh)
    return 1.0 - 2.0 * (x & 1).double()


def _exact_norm(s, dev):
    f = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    h = f.to(s["x"].dtype).double()              # the stream is held in its own type
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].double()
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % 256)).view(-1, 256) @ (_hadamard(dev) / 16)
    # the codes are whole numbers; the 64-bit value that they round has none
    return {"x_s8": None, "x_scale": y.view(f.shape[0], -1).abs().amax(1) / 127, "sum": None if s["residual"] is None else f}


def _exact_append(s, n, kv, dev):
    """Codes come as the numbers before their rounding to 8 bits, against the page's scale."""
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = s["qkv"].double().view(-1, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if s["q_weight"] is not None:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / D + EPS) * s["q_weight"].double()
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) / D + EPS) * s["k_weight"].double()
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                        torch.gather(s["pos"].double(), 1, s["axis"].long()[None].expand(x.shape[0], -1)) * s["freq"])[:, None]
    def turn(y):
        z = (torch.complex(y[..., 0::2].contiguous(), y[..., 1::2].contiguous()) if c["interleaved"]
             else torch.complex(y[..., : D // 2].contiguous(), y[..., D // 2:].contiguous())) * phase
        return torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat((z.real, z.imag), -1)
    q, k = turn(q), turn(k)
    f8 = torch.float8_e4m3fn
    out = {"q": q.reshape(-1, Hq * D)}
    for name, y in (("k", k), ("v", v)):
        codes = s[name].view(f8).double() if name == "k" else s[name].view(f8).double().transpose(2, 3).contiguous()
        scale, at = s[name + "_scale"].double(), 0
        for b in range(c["B"]):
            first, end = kv[b] - n[b], kv[b]
            while first < end:
                p, lo = int(s["table"][b, first // PAGE]), first % PAGE
                m = min(PAGE - lo, end - first)
                new = y[at:at + m]
                top = new.abs().amax((0, 2)).clamp(min=2.0 ** -126 * 448)
                m2, e2 = torch.frexp(top / 448)
                to = torch.ldexp(torch.ones_like(top), e2 - (m2 == 0.5).int())
                if lo:
                    to = torch.maximum(to, scale[p])
                    codes[p, :, :lo] *= (scale[p] / to)[:, None, None]
                scale[p] = to
                codes[p, :, lo:lo + m] = (new / to[:, None]).transpose(0, 1)
                first, at = first + m, at + m
        out[name] = codes if name == "k" else codes.transpose(2, 3)
        out[name + "_scale"] = scale
    return out

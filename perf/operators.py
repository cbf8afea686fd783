"""Cases for timing the paged-cache operators: appending rotated keys and values to a paged cache, and attention over a
paged cache held in 8 bits.

Four operators, each reached through kv_cache_quantized_b200.ops (``own``) or written out in elementary torch
operations (the plain form):

* ``append``     ops.append_paged: rotate q and k by their positions, quantize k (and v) with the Lloyd-Max codebook
                 into a paged cache, or store v as fp16;
* ``q8_append``  ops.q8_append_paged: rotate q and k, quantize k and v to 8 bits with one scale for each 16 tokens and
                 head, requantizing a partly filled block whose scale grows;
* ``q8_decode``  ops.q8_attend_paged with one query token per sequence;
* ``q8_prefill`` ops.q8_attend_paged with several query tokens per sequence, causal.

Indices into a codebook and 8-bit integers come back as whole numbers (every rounding step of the definition is a
single IEEE operation in 32 bits, so they are equal, not near); e4m3 codes come back as float8 values.
"""

import math

import numpy as np
import torch

own = False

SB = 16  # tokens of one scale block
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -100  # a scale block whose largest magnitude is below this is held as zeros


# ---- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 8 at the Llama-shaped heads: codes of both tensors, launch latency counts
        dict(name="append step", op="append", B=8, Hq=32, Hkv=8, d=128, bits=4, vq=True, new=1, T=2048, bt=64,
             dtype="bf16", rot=128, interleaved=False),
        # chunks of four prompts going into a cache with fp16 values
        dict(name="append chunks", op="append", B=4, Hq=32, Hkv=8, d=128, bits=4, vq=False, new=2048, T=8192, bt=256,
             dtype="f16", rot=128, interleaved=False),
        # small heads, 3-bit codes that straddle bytes, half of each head rotated in interleaved pairs, fp32 inputs
        dict(name="append d64 b3", op="append", B=3, Hq=12, Hkv=12, d=64, bits=3, vq=True, new=517, T=1024, bt=32,
             dtype="f32", rot=32, interleaved=True),
        # a decode step of a large batch into an 8-bit cache: blocks partly filled, scales that may grow
        dict(name="q8 append step", op="q8_append", B=64, Hq=32, Hkv=8, d=128, kind="i8", new=1, T=1024, bt=16,
             dtype="bf16", rot=128, interleaved=False),
        # whole prompts into an 8-bit cache: streams q, k and v once
        dict(name="q8 append prompts", op="q8_append", B=8, Hq=32, Hkv=8, d=128, kind="e4m3", new=2048, T=2048, bt=64,
             dtype="f16", rot=128, interleaved=False),
        # odd-sized chunks onto sequences that end inside a scale block, few KV heads
        dict(name="q8 append chunks", op="q8_append", B=5, Hq=16, Hkv=2, d=128, kind="i8", new=333, T=1500, bt=128,
             dtype="bf16", rot=64, interleaved=False),
        # the smallest decode call: one sequence, latency counts
        dict(name="q8 decode b1", op="q8_decode", B=1, Hq=32, Hkv=8, d=128, kind="i8", T=4096, bt=64, dtype="f16",
             ragged=False),
        # long-context decode of a batch of 8: bandwidth
        dict(name="q8 decode 32k", op="q8_decode", B=8, Hq=32, Hkv=8, d=128, kind="i8", T=32768, bt=64, dtype="bf16",
             ragged=False),
        # a serving batch of very different lengths, 8 query heads per KV head, the smallest pages
        dict(name="q8 decode ragged", op="q8_decode", B=64, Hq=16, Hkv=2, d=128, kind="e4m3", T=8192, bt=16,
             dtype="bf16", ragged=True),
        # small heads without sharing, fp32 queries and outputs
        dict(name="q8 decode d64 f32", op="q8_decode", B=8, Hq=12, Hkv=12, d=64, kind="i8", T=1024, bt=32, dtype="f32",
             ragged=True),
        # chunked prefill: 2048 new tokens of each of four sequences against up to 8192 cached ones
        dict(name="q8 prefill chunks", op="q8_prefill", B=4, Hq=32, Hkv=8, d=128, kind="i8", new=2048, T=8192, bt=64,
             dtype="bf16", ragged=False),
        # verification of a few drafted tokens per sequence: few rows against a long axis
        dict(name="q8 verify", op="q8_prefill", B=16, Hq=16, Hkv=2, d=128, kind="e4m3", new=5, T=4096, bt=32,
             dtype="f16", ragged=True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "q8_append", "q8_decode", "q8_prefill"])
    Hq, Hkv = rng.choice([(32, 8), (16, 2), (12, 12), (8, 8), (28, 4), (24, 8)])
    d = rng.choice([64, 128, 128])
    bt = rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, bt=bt)
    if op in ("append", "q8_append"):
        case["dtype"] = rng.choice(["f16", "bf16", "f32"])
        case["rot"] = rng.choice([d, d, d // 2])
        case["interleaved"] = rng.random() < 0.3
        case["B"] = log_int(1, 64)
        case["new"] = 1 if rng.random() < 0.4 else log_int(2, max(2, min(2048, 8192 // case["B"])))
        case["T"] = case["new"] + log_int(1, 1024)
        if op == "append":
            case["bits"] = rng.choice([1, 2, 3, 4])
            case["vq"] = rng.random() < 0.5
        else:
            case["kind"] = rng.choice(["i8", "e4m3"])
        return case
    case["kind"] = rng.choice(["i8", "e4m3"])
    case["ragged"] = rng.random() < 0.6
    if op == "q8_decode":
        case["dtype"] = rng.choice(["f16", "bf16", "f32"])
        case["B"] = log_int(1, 64)
        case["T"] = log_int(50, min(32768, 262144 * 8 // (case["B"] * Hkv)))
        return case
    case["dtype"] = rng.choice(["f16", "bf16"])
    case["B"] = log_int(1, 16)
    case["T"] = log_int(64, 8192)
    most = 2048 * 8192 * 4 // (case["B"] * case["T"])  # the listed chunks' score entries at 32 heads
    case["new"] = log_int(2, max(2, min(2048, case["T"], most)))
    return case


def _lengths(case):
    """(new tokens, lengths with them) of each sequence: host integers that the case's sizes alone decide."""
    B, T = case["B"], case["T"]
    g = torch.Generator().manual_seed(1000003 * B + T)
    op = case["op"]
    if op in ("q8_decode", "q8_prefill"):
        new = [1] * B if op == "q8_decode" else [case["new"]] * B
        lens = [T] * B
        if case["ragged"]:
            r = torch.rand(B, generator=g).tolist()
            lens = [max(1, int(T * (0.05 + 0.95 * x))) for x in r]
            if op == "q8_prefill":
                r = torch.rand(B, generator=g).tolist()
                new = [max(1, int(n * (0.5 + 0.5 * x) + 0.5)) for n, x in zip(new, r)]
            lens[0] = T
            new[0] = case["new"] if op == "q8_prefill" else 1
        return [min(n, L) for n, L in zip(new, lens)], lens
    new = [case["new"]] * B
    if case["new"] > 1:  # chunks of somewhat different lengths
        r = torch.rand(B, generator=g).tolist()
        new = [max(1, int(n * (0.8 + 0.2 * x))) for n, x in zip(new, r)]
        new[0] = case["new"]
    past = T - case["new"]
    r = torch.rand(B, generator=g).tolist()
    return new, [n + int(past * (0.3 + 0.7 * x)) for n, x in zip(new, r)]


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _rope_table(n, rot, dev):
    """[n, rot] fp32: cos of each position's rot / 2 angles, then their sines (angles formed in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _codes8(shape, kind, g, dev):
    """8-bit codes as a cache holds them: normal values at the scale their block's largest magnitude sets."""
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.float16)
    if kind == "i8":
        return x.mul_(35.0).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    return x.mul_(90.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    hg = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, Hkv, d, bt = case["B"], case["Hq"], case["Hkv"], case["d"], case["bt"]
    new, lens = _lengths(case)
    n_tok, mb = sum(new), -(-case["T"] // bt)
    need = [-(-L // bt) for L in lens]
    nblocks = sum(need) + 2
    perm = torch.randperm(nblocks, generator=hg).to(torch.int32)
    table = torch.zeros((B, mb), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    s = dict(case=dict(case), table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu=cu.to(dev), n_tok=n_tok, max_new=max(new), T=case["T"])
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("append", "q8_append"):
        # a fused projection's output: q, k and v are slices of one row; a few channels of q and k are large
        qkv = torch.randn((n_tok, (Hq + 2 * Hkv) * d), generator=g, device=dev)
        outlier = torch.ones(d, device=dev)
        outlier[torch.randperm(d, generator=g, device=dev)[:4]] = 5.0
        qkv[:, :(Hq + Hkv) * d].view(n_tok, Hq + Hkv, d).mul_(outlier)
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = (x.view(n_tok, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        s["rope"] = _rope_table(case["T"], case["rot"], dev)
    else:
        s["q"] = torch.randn((n_tok, Hq, d), generator=g, device=dev).to(dt)
    if case["op"] == "append":
        R = d * case["bits"] // 8
        byte = lambda *sh: torch.randint(0, 256, sh, generator=g, device=dev, dtype=torch.uint8)
        norm = lambda *sh: (torch.rand(sh, generator=g, device=dev) * 10 + 5).half()
        s["kcodes"], s["knorms"] = byte(nblocks, Hkv, bt, R), norm(nblocks, Hkv, bt)
        if case["vq"]:
            s["vcodes"], s["vnorms"] = byte(nblocks, Hkv, bt, R), norm(nblocks, Hkv, bt)
        else:
            s["vpool"] = torch.randn((nblocks, Hkv, bt, d), generator=g, device=dev, dtype=torch.float16)
        s["signs"] = (torch.randint(0, 2, (d,), generator=g, device=dev) * 2 - 1).to(torch.int8)
    else:
        top = 127.0 if case["kind"] == "i8" else 448.0
        for name in ("k", "v"):
            s[name + "codes"] = _codes8((nblocks, Hkv, bt, d), case["kind"], g, dev)
            amax = torch.rand((nblocks, Hkv, bt // SB), generator=g, device=dev) * 2 + 2.5
            sc = amax / top
            if case["kind"] == "e4m3":  # powers of two
                sc = torch.exp2(torch.ceil(torch.log2(sc)))
            s[name + "scales"] = sc.contiguous()
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _token_map(s):
    """For each new token: its sequence, its position in the sequence's cache."""
    i = torch.arange(s["n_tok"], device=s["cu"].device)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    new = cu[1:] - cu[:-1]
    pos = s["lens"].long()[b] - new[b] + (i - cu[b])
    return b, pos


def _rotate(x, table, pos, rot, interleaved):
    """Position rotation of x [n, H, d] in 32 bits: pairs (j, j + rot/2), or (2j, 2j + 1) when interleaved."""
    x = x.float()
    h = rot // 2
    cs = table[pos]
    c, sn = cs[:, None, :h], cs[:, None, h:]
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = r[..., :h], r[..., h:]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, rest], -1)


def _lloyd(bits):
    """Thresholds and centroids of the Lloyd-Max quantizer of N(0, 1), 64 bits."""
    L = 1 << bits
    phi = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    Phi = lambda x: 0.5 * math.erfc(-x / math.sqrt(2))
    c = [-2.0 + 4.0 * (k + 0.5) / L for k in range(L)]
    for _ in range(20000):
        t = [-40.0] + [(a + b) / 2 for a, b in zip(c, c[1:])] + [40.0]
        n = [(phi(t[k]) - phi(t[k + 1])) / (Phi(t[k + 1]) - Phi(t[k])) for k in range(L)]
        n = [(a - b) / 2 for a, b in zip(n, reversed(n))]
        move = max(abs(a - b) for a, b in zip(n, c))
        c = n
        if move < 1e-15:
            break
    return [(a + b) / 2 for a, b in zip(c, c[1:])], c


_TAU = {b: _lloyd(b)[0] for b in (1, 2, 3, 4)}


def _fwht(x):
    """Walsh-Hadamard transform (not normalised) of the last axis: butterflies (a + b, a - b), smallest stride first."""
    d, h = x.shape[-1], 1
    while h < d:
        y = x.view(x.shape[:-1] + (d // (2 * h), 2, h))
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack([a + b, a - b], -2).view(x.shape)
        h *= 2
    return x


def _square_sum(x):
    """Sum of squares of the last axis in 32 bits, in a stated order: each run of d / 32 values by fused multiply-adds,
    then pairs of runs at distance 16, 8, 4, 2 and 1.  (A fused step is a product and a sum in 64 bits, rounded.)"""
    x = x.reshape(x.shape[:-1] + (32, x.shape[-1] // 32))
    p = torch.zeros_like(x[..., 0])
    for i in range(x.shape[-1]):
        p = (x[..., i].double() * x[..., i].double() + p.double()).float()
    for m in (16, 8, 4, 2, 1):
        p = p[..., :m] + p[..., m:2 * m]
    return p[..., 0]


def _indices(x, signs, bits):
    """Codebook indices [.., d] and norms [..] of rows x: the thresholds at or below each coordinate of the rotated
    unit vector, counted."""
    n = _square_sum(x).sqrt()
    y = _fwht((x * torch.where(signs < 0, -1.0, 1.0)).contiguous())
    w = torch.where(n[..., None] > 0, y / n[..., None], 0.0)
    tau = torch.tensor(_TAU[bits], dtype=torch.float64, device=x.device).float()
    return torch.bucketize(w, tau, right=True), n


def _pack(idx, bits):
    """Bitstream of b-bit indices, least significant bit first."""
    bit = (idx[..., None] >> torch.arange(bits, device=idx.device)) & 1
    bit = bit.flatten(-2).view(idx.shape[:-1] + (-1, 8))
    return (bit << torch.arange(8, device=idx.device)).sum(-1).to(torch.uint8)


def _plain_append(s):
    c = s["case"]
    b, pos = _token_map(s)
    q = _rotate(s["q"], s["rope"], pos, c["rot"], c["interleaved"])
    k = _rotate(s["k"], s["rope"], pos, c["rot"], c["interleaved"])
    blk, off = s["table"].long()[b, pos // c["bt"]], pos % c["bt"]
    idx, n = _indices(k, s["signs"], c["bits"])
    s["kcodes"][blk, :, off] = _pack(idx, c["bits"])
    s["knorms"][blk, :, off] = n.half()
    if c["vq"]:
        idx, n = _indices(s["v"].float(), s["signs"], c["bits"])
        s["vcodes"][blk, :, off] = _pack(idx, c["bits"])
        s["vnorms"][blk, :, off] = n.half()
    else:
        s["vpool"][blk, :, off] = s["v"].half()
    return q


def _block_map(s):
    """The scale blocks that the new tokens touch, as up to n_tok / 16 + 2 B items: sequence, block, positions [.., 16],
    which of these are new, which are older, and whether the item is in use."""
    dev = s["cu"].device
    cu, lens = s["cu"].long(), s["lens"].long()
    B = lens.numel()
    start = cu[:-1] // SB + 2 * torch.arange(B, device=dev)
    it = torch.arange(s["n_tok"] // SB + 2 * B, device=dev)
    b = torch.searchsorted(start, it, right=True) - 1
    p0 = lens[b] - (cu[1:] - cu[:-1])[b]
    blk = p0 // SB + (it - start[b])
    pos = blk[:, None] * SB + torch.arange(SB, device=dev)
    used = (blk * SB < lens[b]) & (p0 < lens[b])
    is_new = (pos >= p0[:, None]) & (pos < lens[b][:, None]) & used[:, None]
    is_old = (pos < p0[:, None]) & used[:, None]
    tok = (cu[b][:, None] + pos - p0[:, None]).clamp(0, max(s["n_tok"] - 1, 0))
    return b, blk, pos, is_new, is_old, used, tok


def _scale_of(amax, kind):
    if kind == "i8":
        s = amax / torch.full_like(amax, 127.0)
    else:  # the smallest power of two that holds amax within 448 = 0.875 * 2^9
        m, e = torch.frexp(amax)
        e = e - 9 + (m > 0.875).int()
        s = ((e + 127) << 23).view(torch.float32)
    return torch.where(amax >= TINY, s, 0.0)


def _plain_q8_write(s, x, codes, scales):
    c = s["case"]
    kind, bt = c["kind"], c["bt"]
    b, blk, pos, is_new, is_old, used, tok = s["map"]
    cap = s["table"].shape[1] * bt
    page = s["table"].long()[b[:, None], pos.clamp(max=cap - 1) // bt]  # [N, 16]
    off = pos % bt
    xb = torch.where(is_new[:, :, None, None], x[tok], 0.0)
    old = codes[page, :, off]
    oldv = (old.view(torch.int8) if kind == "i8" else old.view(torch.float8_e4m3fn)).float()
    sb = (blk * SB) % bt // SB
    p0 = page[:, 0]
    s_old = torch.where(is_old.any(1)[:, None], scales[p0, :, sb], 0.0)  # [N, Hkv]
    sc = torch.maximum(s_old, _scale_of(xb.abs().amax((1, 3)), kind))
    inv = torch.where(sc > 0, torch.ones_like(sc) / sc, 0.0)
    y = xb * inv[:, None, :, None]
    z = torch.where((sc == s_old)[:, None, :, None], oldv, oldv * (s_old * inv)[:, None, :, None])
    y = torch.where(is_new[:, :, None, None], y, z)
    if kind == "i8":
        y = y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    else:
        y = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    w = is_new | is_old
    codes[page[w], :, off[w]] = y[w]
    scales[p0[used], :, sb[used]] = sc[used]


def _plain_q8_append(s):
    c = s["case"]
    b, pos = _token_map(s)
    q = _rotate(s["q"], s["rope"], pos, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], s["rope"], pos, c["rot"], c["interleaved"])
    s["map"] = _block_map(s)
    _plain_q8_write(s, k, s["kcodes"], s["kscales"])
    _plain_q8_write(s, s["v"].float(), s["vcodes"], s["vscales"])
    return q


def _gathered(s, codes, scales, dtype):
    """The cache of every sequence as values [B, Hkv, T, d]; what no token has written yet is zero."""
    c = s["case"]
    kind = torch.int8 if c["kind"] == "i8" else torch.float8_e4m3fn
    tab = s["table"].long()
    x = codes[tab].view(kind).to(dtype)  # [B, mb, Hkv, bt, d]
    B, mb, H, bt, d = x.shape
    x = (x.view(B, mb, H, bt // SB, SB, d) * scales[tab].to(dtype)[..., None, None]).view(B, mb, H, bt, d)
    x = x.transpose(1, 2).reshape(B, H, mb * bt, d)[:, :, :s["T"]]
    live = torch.arange(x.shape[2], device=x.device)[None] < s["lens"][:, None]
    return torch.where(live[:, None, :, None], x, 0.0)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    G, n = Hq // Hkv, s["max_new"]
    b, pos = _token_map(s)
    i = torch.arange(s["n_tok"], device=b.device) - s["cu"].long()[b]
    k, v = _gathered(s, s["kcodes"], s["kscales"], torch.float32), _gathered(s, s["vcodes"], s["vscales"], torch.float32)
    q = torch.zeros((B, n, Hq, d), device=b.device)
    q[b, i] = s["q"].float()
    last = torch.full((B, n), -1, device=b.device, dtype=torch.long)
    last[b, i] = pos
    q = q.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    sc = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    keep = torch.arange(k.shape[2], device=b.device)[None, None] <= last[:, :, None]  # [B, n, T]
    sc = sc.view(B, Hkv, n, G, -1).masked_fill_(~keep[:, None, :, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, n * G, -1) @ v).view(B, Hkv, n, G, d) / torch.where(l > 0, l, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    return o[b, i].to(s["q"].dtype)


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    ops = None
    if own:
        from kv_cache_quantized_b200 import ops
    if c["op"] == "append":
        if own:
            vals = dict(vcodes=s["vcodes"], vnorms=s["vnorms"]) if c["vq"] else dict(v=s["vpool"])
            q = ops.append_paged(s["k"], s["v"], s["kcodes"], s["knorms"], s["signs"], c["bits"], s["table"],
                                 s["lens"], cu_new=s["cu"], q=s["q"], cos_sin=s["rope"],
                                 interleaved=c["interleaved"], **vals)
        else:
            q = _plain_append(s)
        out = dict(q=q, kcodes=s["kcodes"], knorms=s["knorms"])
        out.update(dict(vcodes=s["vcodes"], vnorms=s["vnorms"]) if c["vq"] else dict(v=s["vpool"]))
        return out
    if c["op"] == "q8_append":
        if own:
            q = ops.q8_append_paged(s["k"], s["v"], s["kcodes"], s["kscales"], s["vcodes"], s["vscales"], s["table"],
                                    s["lens"], kind=c["kind"], cu_new=s["cu"], q=s["q"], cos_sin=s["rope"],
                                    interleaved=c["interleaved"])
        else:
            q = _plain_q8_append(s)
        kind = torch.int8 if c["kind"] == "i8" else torch.float8_e4m3fn
        return dict(q=q, kcodes=s["kcodes"].view(kind), kscales=s["kscales"], vcodes=s["vcodes"].view(kind),
                    vscales=s["vscales"])
    if own:
        return ops.q8_attend_paged(s["q"], s["kcodes"], s["kscales"], s["vcodes"], s["vscales"], s["table"], s["lens"],
                                   kind=c["kind"], cu_q=None if c["op"] == "q8_decode" else s["cu"],
                                   max_q=s["max_new"], T=s["T"])
    return _plain_attend(s)


def work(case):
    """One pass's bytes (each input and output once) and operations."""
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    el = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("append", "q8_append"):
        n_tok = sum(_lengths(case)[0])
        io = n_tok * (Hq + 2 * Hkv) * d * el + n_tok * case["rot"] * 4
        if case["op"] == "append":
            kb = d * case["bits"] / 8 + 2
            return {"bytes": io + n_tok * (Hq * d * 4 + Hkv * (kb + (kb if case["vq"] else 2 * d))),
                    "flops": n_tok * (Hq + 2 * Hkv) * d * 3 + n_tok * Hkv * d * 2 * math.log2(d)}
        return {"bytes": io + n_tok * (Hq * d * el + 2 * Hkv * (d + 4 / SB)), "flops": n_tok * (Hq + 2 * Hkv) * d * 5}
    new, lens = _lengths(case)
    keys = sum(n * (L - (n - 1) / 2) for n, L in zip(new, lens))
    return {"bytes": sum(lens) * Hkv * 2 * (d + 4 / SB) + 2 * sum(new) * Hq * d * el, "flops": 4.0 * keys * Hq * d}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------

def _exact_rows(s):
    """(sequence, cache position) of every new token, in order, from host integers."""
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    return [(b, lens[b] - (cu[b + 1] - cu[b]) + j) for b in range(len(lens)) for j in range(cu[b + 1] - cu[b])]


def _exact_rope(x, s, pos):
    """Complex form of the rotation: each pair, as a complex number, times cos + i sin of the given table."""
    rot, h = s["case"]["rot"], s["case"]["rot"] // 2
    x = x.double().clone()
    tab = s["rope"].double()[pos]
    ph = torch.complex(tab[:, :h], tab[:, h:])[:, None]
    if s["case"]["interleaved"]:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * ph
        x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :h], x[..., h:rot]) * ph
        x[..., :h], x[..., h:rot] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    c, dev = s["case"], s["lens"].device
    if c["op"] in ("append", "q8_append"):
        rows = torch.tensor(_exact_rows(s), device=dev)
        seq, pos = rows[:, 0], rows[:, 1]
        page = s["table"][seq, pos // c["bt"]].long()
        off = pos % c["bt"]
        q, k, v = _exact_rope(s["q"], s, pos), _exact_rope(s["k"], s, pos), s["v"].double()
    if c["op"] == "append":
        out = dict(q=q, kcodes=None, knorms=s["knorms"].double())
        out["knorms"][page, :, off] = k.square().sum(-1).sqrt()
        if c["vq"]:
            out.update(vcodes=None, vnorms=s["vnorms"].double())
            out["vnorms"][page, :, off] = v.square().sum(-1).sqrt()
        else:
            out["v"] = s["vpool"].double()
            out["v"][page, :, off] = v
        return out
    if c["op"] == "q8_append":
        out = dict(q=q)
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        first = torch.tensor([L - (cu[b + 1] - cu[b]) for b, L in enumerate(lens)], device=dev)
        for name, x in (("k", k), ("v", v)):
            scales = s[name + "scales"].double()
            grp = (page * scales.shape[2] + off // SB)  # the block of each token: page, place in the page
            amax = torch.zeros((scales.shape[0] * scales.shape[2], c["Hkv"]), dtype=torch.float64, device=dev)
            amax.scatter_reduce_(0, grp[:, None].expand(-1, c["Hkv"]), x.abs().amax(-1), "amax")
            need = amax / 127.0 if c["kind"] == "i8" else torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
            need = need.view(scales.shape[0], scales.shape[2], c["Hkv"]).transpose(1, 2)
            held = scales.clone()  # a block keeps its scale if older tokens live in it
            fresh = torch.zeros_like(scales, dtype=torch.bool)
            fresh[page, :, off // SB] = ((pos // SB * SB) >= first[seq])[:, None]
            new = torch.where(fresh, need, torch.maximum(held, need))
            touched = torch.zeros_like(fresh)
            touched[page, :, off // SB] = True
            out[name + "scales"] = torch.where(touched, new, held)
            out[name + "codes"] = None
            if c["kind"] == "e4m3":
                codes = s[name + "codes"].view(torch.float8_e4m3fn).double()
                ratio = torch.where(touched & ~fresh, held / new, 1.0)
                codes = codes * ratio.repeat_interleave(SB, 2)[..., None]
                # rows of a touched block that no token has reached keep what they held
                codes_new = x / new[page, :, off // SB][..., None]
                stale = s[name + "codes"].view(torch.float8_e4m3fn).double()
                for b, L in enumerate(lens):
                    last = int(s["table"][b, (L - 1) // c["bt"]])
                    o = (L - 1) % c["bt"] + 1
                    e = -(-o // SB) * SB
                    codes[last, :, o:e] = stale[last, :, o:e]
                codes[page, :, off] = codes_new
                out[name + "codes"] = codes
        return out
    Hkv, G, d = c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.empty((s["n_tok"], c["Hq"], d), dtype=torch.float64, device=dev)
    kind = torch.int8 if c["kind"] == "i8" else torch.float8_e4m3fn
    for b, L in enumerate(lens):
        pages = s["table"][b, :-(-L // c["bt"])].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "codes"][pages].view(kind).double()
            x = x * s[name + "scales"][pages].double().repeat_interleave(SB, 2)[..., None]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, d)[:, :L])
        n = cu[b + 1] - cu[b]
        ahead = torch.arange(L, device=dev)[None] > torch.arange(L - n, L, device=dev)[:, None]
        for h in range(Hkv):
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            w = torch.einsum("ngd,td->ngt", q, kv[0][h]) / math.sqrt(d)
            w = torch.softmax(w.masked_fill(ahead[:, None], float("-inf")), -1)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w, kv[1][h])
    return out

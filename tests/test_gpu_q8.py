"""The paged append (axr_append_paged, axr_q8_append_paged) and attention over the 8-bit cache (axr_q8_attend_paged)
against the oracle: ragged batches, lengths from nothing to several tiles, padding tokens, block edges, strided and
misordered inputs, stale bytes behind the sequences, other streams, captured graphs, refusals."""

import math

import numpy as np
import pytest
import torch

import oracle
from kv_cache_quantized_b200 import _abi, ops
from kv_cache_quantized_b200 import workloads as W
from oracle import q8
from tests import parity

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rope_table(n, rot):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def same(a, b):
    """Equal byte for byte (NaN among them)."""
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


class Batch:
    """A ragged batch: new-token counts and lengths, a shuffled block table, fused projection rows with padding tokens
    behind the last sequence."""

    def __init__(self, counts, lens, Hq, Hkv, d, bt, dtype, seed, pad=3, scale=1.0):
        self.counts, self.lens, self.Hq, self.Hkv, self.d, self.bt = counts, lens, Hq, Hkv, d, bt
        rng = np.random.default_rng(seed)
        self.rng = rng
        B, need = len(lens), [-(-L // bt) for L in lens]
        self.mb = max(max(need), 1) + 1
        self.nb = sum(need) + 2
        perm = rng.permutation(self.nb)
        self.table = np.full((B, self.mb), -7, np.int32)  # entries past a row's blocks are never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.n_tok = int(self.cu[-1]) + pad
        x = rng.normal(size=(self.n_tok, (Hq + 2 * Hkv) * d)) * scale
        qkv = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
        self.qkv = qkv.cuda()
        cut = [Hq * d, Hkv * d, Hkv * d]
        self.q, self.k, self.v = (t.view(self.n_tok, -1, d) for t in self.qkv.split(cut, 1))
        self.qn, self.kn, self.vn = (t.float().numpy().reshape(self.n_tok, -1, d) for t in qkv.split(cut, 1))
        self.t = dict(table=cuda(self.table), lens=cuda(np.array(lens, np.int32)), cu=cuda(self.cu))

    def rows(self, x, b):
        return x[self.cu[b]:self.cu[b + 1]]

    def rotated(self, x, tab, inter, positions=None):
        out = []
        for b, n in enumerate(self.counts):
            r = [q8.rotate(self.rows(x, b)[i], tab, self.lens[b] - n + i if positions is None else
                           int(positions[self.cu[b] + i]), inter) if self.lens[b] - n + i >= 0 else self.rows(x, b)[i]
                 for i in range(n)]
            out.append(np.stack(r) if r else np.zeros((0,) + x.shape[1:], np.float32))
        return out

    def pools8(self, kind):
        """Pools with arbitrary bytes (e4m3 NaN among them) and scales (NaN among them)."""
        codes = self.rng.integers(0, 256, size=(self.nb, self.Hkv, self.bt, self.d)).astype(np.uint8)
        scales = self.rng.uniform(0.01, 0.02, size=(self.nb, self.Hkv, self.bt // 16)).astype(np.float32)
        if kind == "e4m3":
            scales = (2.0 ** np.round(np.log2(scales))).astype(np.float32)
        return codes, scales


def clean_live(bt, codes, scales, kind, batch):
    """Live older rows hold finite codes; stale scales behind the sequences are NaN."""
    live = np.zeros(scales.shape, bool)
    for b, L in enumerate(batch.lens):
        p0 = max(L - batch.counts[b], 0)
        for t in range(p0):
            page = batch.table[b, t // bt]
            live[page, :, t % bt // 16] = True
            row = codes[page, :, t % bt]
            codes[page, :, t % bt] = np.where((row & 127) == 127, 5, row) if kind == "e4m3" else \
                np.where(row == 128, 5, row)
    scales[~live] = np.nan


# counts / lengths: nothing new, one token, whole and partial blocks, more than a tile, an empty sequence, counts above
# the length (their first tokens have no position)
RAGGED = ([0, 1, 5, 16, 17, 40, 0, 3, 33], [7, 1, 20, 16, 50, 300, 0, 2, 64])
STEP = ([1, 1, 1, 1], [1, 16, 17, 130])


@pytest.mark.parametrize("dtype,d,kind,bt,rot,inter", [
    ("f16", 128, "i8", 16, 128, False), ("bf16", 128, "e4m3", 64, 64, False), ("f32", 128, "i8", 128, 128, True),
    ("bf16", 64, "i8", 32, 64, False), ("f16", 64, "e4m3", 16, 16, True), ("f32", 64, "e4m3", 256, 32, False)])
@pytest.mark.parametrize("shape", [RAGGED, STEP])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (15, 5), (9, 9)])
def test_q8_append_is_bit_exact(dtype, d, kind, bt, rot, inter, shape, Hq, Hkv):
    bt_ = Batch(*shape, Hq, Hkv, d, bt, dtype, 11 + d + bt)
    tab = rope_table(400, rot)
    kc, ks = bt_.pools8(kind)
    vc, vs = bt_.pools8(kind)
    clean_live(bt, kc, ks, kind, bt_)
    clean_live(bt, vc, vs, kind, bt_)
    dev = [cuda(x) for x in (kc, ks, vc, vs)]
    qo = torch.full((bt_.n_tok, Hq, d), 777.0, dtype=DT[dtype], device="cuda")
    ops.device_status(clear=True)
    got = ops.q8_append_paged(bt_.k, bt_.v, *dev, bt_.t["table"], bt_.t["lens"], kind=kind, cu_new=bt_.t["cu"],
                              q=bt_.q, cos_sin=cuda(tab), interleaved=inter, q_out=qo)
    assert got is qo and ops.device_status() == 0
    q8.append(bt_.rotated(bt_.kn, tab, inter), kc, ks, bt_.table, bt_.lens, bt_.counts, bt, kind)
    q8.append([bt_.rows(bt_.vn, b) for b in range(len(bt_.lens))], vc, vs, bt_.table, bt_.lens, bt_.counts, bt, kind)
    for name, a, w in zip(("kcodes", "kscales", "vcodes", "vscales"), dev, (kc, ks, vc, vs)):
        a = a.cpu().numpy()
        assert np.array_equal(a.view(np.uint8), w.view(np.uint8)), name
    want = np.full((bt_.n_tok, Hq, d), 777.0, np.float32)
    for b, r in enumerate(bt_.rotated(bt_.qn, tab, inter)):
        ok = max(bt_.counts[b] - bt_.lens[b], 0)  # tokens without a position are left as they were
        want[bt_.cu[b] + ok:bt_.cu[b + 1]] = r[ok:]
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(DT[dtype]))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_q8_append_growth_positions_and_non_finite(kind):
    """Token by token with growing magnitudes, explicit rotation positions, zero and non-finite rows."""
    d, Hkv, bt, n = 128, 3, 32, 37
    tab = rope_table(64, d)
    rng = np.random.default_rng(5)
    x = rng.normal(size=(n, 1, 2 * Hkv, d)).astype(np.float32) * np.linspace(0.1, 4, n, dtype=np.float32)[:, None, None, None]
    x[0] = 0
    x[3, 0, 0, 7] = np.nan
    x[4, 0, 1, 9], x[4, 0, 3, 10] = np.inf, -np.inf
    x[20, 0, 2] *= 2.0 ** -110
    kc, vc = np.zeros((4, Hkv, bt, d), np.uint8), np.zeros((4, Hkv, bt, d), np.uint8)
    ks, vs = np.full((4, Hkv, 2), np.nan, np.float32), np.full((4, Hkv, 2), np.nan, np.float32)
    dev = [cuda(a) for a in (kc, ks, vc, vs)]
    table = np.array([[2, 0]], np.int32)
    for i in range(n):
        pos = np.array([(7 * i) % 64], np.int32)
        k, v = x[i][:, :Hkv], x[i][:, Hkv:]
        ops.q8_append_paged(cuda(k), cuda(v), *dev, cuda(table), cuda(np.array([i + 1], np.int32)), kind=kind,
                            cos_sin=cuda(tab), positions=cuda(pos))
        with np.errstate(invalid="ignore"):
            kr = q8.rotate(k[0], tab, int(pos[0]), False)[None]
        q8.append([kr], kc, ks, table, [i + 1], [1], bt, kind)
        q8.append([v], vc, vs, table, [i + 1], [1], bt, kind)
    for a, w in zip(dev, (kc, ks, vc, vs)):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), w.view(np.uint8))


@pytest.mark.parametrize("d,bits,vq,dtype,bt,rot,inter", [
    (128, 4, True, "bf16", 16, 128, False), (128, 3, True, "f16", 64, 64, True), (128, 2, False, "f32", 32, 128, False),
    (128, 1, True, "f16", 128, 32, False), (64, 4, False, "bf16", 32, 64, True), (64, 3, True, "f32", 16, 64, False),
    (64, 2, True, "f16", 64, 16, False), (64, 1, False, "f16", 16, 48, False)])
def test_append_matches_the_writer_and_the_oracle(d, bits, vq, dtype, bt, rot, inter):
    Hq, Hkv = 15, 5
    bt_ = Batch(*RAGGED, Hq, Hkv, d, bt, dtype, 60 + d + bits)
    tab, s = rope_table(400, rot), W.sign_vector(d, 8)
    R, shape = d * bits // 8, (bt_.nb, Hkv, bt)
    byte = lambda: bt_.rng.integers(0, 256, size=shape + (R,)).astype(np.uint8)
    norm = lambda: bt_.rng.uniform(1, 2, size=shape).astype(np.float16)
    kc, kn, vc, vn = byte(), norm(), byte(), norm()
    vp = bt_.rng.normal(size=shape + (d,)).astype(np.float16)
    dk, dn, dvc, dvn, dvp = (cuda(a) for a in (kc, kn, vc, vn, vp))
    vals = dict(vcodes=dvc, vnorms=dvn) if vq else dict(v=dvp)
    qo = torch.full((bt_.n_tok, Hq, d), 777.0, device="cuda")
    ops.device_status(clear=True)
    got = ops.append_paged(bt_.k, bt_.v, dk, dn, cuda(s), bits, bt_.t["table"], bt_.t["lens"], cu_new=bt_.t["cu"],
                           q=bt_.q, cos_sin=cuda(tab), interleaved=inter, q_out=qo, **vals)
    assert ops.device_status() == 0
    kr, qr = bt_.rotated(bt_.kn, tab, inter), bt_.rotated(bt_.qn, tab, inter)
    want_q = np.full((bt_.n_tok, Hq, d), 777.0, np.float32)
    touched = np.zeros(shape[:1] + shape[2:], bool)
    for b, n in enumerate(bt_.counts):
        for i in range(n):
            pos = bt_.lens[b] - n + i
            if pos < 0:
                continue
            page, off = bt_.table[b, pos // bt], pos % bt
            touched[page, off] = True
            want_q[bt_.cu[b] + i] = qr[b][i]
            # bit for bit what the writer kernel makes of the rotated row
            c, m = ops.write_keys(cuda(kr[b][i]), cuda(s), bits)
            assert torch.equal(dk[page, :, off], c) and torch.equal(dn[page, :, off], m)
            parity.check_indices(c.cpu().numpy(), kr[b][i], s, d, bits) if n > 30 and i == 0 else None
            vrow = bt_.rows(bt_.vn, b)[i]
            if vq:
                c, m = ops.write_keys(cuda(vrow), cuda(s), bits)
                assert torch.equal(dvc[page, :, off], c) and torch.equal(dvn[page, :, off], m)
            else:
                assert np.array_equal(dvp[page, :, off].cpu().numpy(), vrow.astype(np.float16))
    assert np.array_equal(got.cpu().numpy(), want_q)
    keep = np.broadcast_to(~touched[:, None], shape)
    for a, w in ((dk, kc), (dn, kn), (dvc, vc), (dvn, vn), (dvp, vp)):
        assert np.array_equal(a.cpu().numpy()[keep], w[keep])  # every other row keeps its bytes


# ---- attention -------------------------------------------------------------------------------------------------------

def check_attention(got, batch, q, pools, kind, scale, dtype, out_fill=None):
    """|o - ref| <= (2 delta + (T / 16 + 64) 2^-23 + e) A + e |ref|, per coordinate, with A = sum_t p_t |v_t|:
    * delta, the absolute error of a score: fp16 hi and lo planes hold a factor to 2^-22, the d / 16 + 6 roundings of
      the fp32 sum and of its scaling are 2^-23 each (the tensor core truncates), so
      delta <= (2^-22 + (d / 16 + 6) 2^-23) scale sum |q_j k_j|; a weight's relative error is e^(2 delta) - 1, which
      is at most 4 delta for delta <= 0.3, and both the weight and the normaliser carry it at 2 delta each;
    * the value sums: one rounding in each of T / 16 steps, and a constant number around them (weights, splits, merge);
    * e = eps / 2 of a 16-bit output type: the output's rounding, and one of the weights; 0 for fp32;
    * and, beside the relative terms, the floor of the weights' fp16 planes: a weight enters as p vs / vref 2^14 with
      vref < 2 max vs the power of two above the largest value scale met so far, and the lo plane's last step is
      fp16's smallest, 2^-24, so each of at most T weights is off by up to 2^-25 of that, 2^-39 vref < 2^-38 max vs,
      times a code: 2^-38 T max|code| max vs, which only outputs whose A is far below the values' range can notice
      (a coordinate that is zero at every token that matters)."""
    kc, ks, vc, vs = pools
    lens, counts, bt, d = batch.lens, batch.counts, batch.bt, batch.d
    outs, mags, errs = q8.attend(q, kc, ks, vc, vs, batch.table, lens, counts, bt, kind, scale)
    e = torch.finfo(DT[dtype]).eps / 2 if dtype != "f32" else 0.0
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got[:batch.cu[-1]]))
    for b, n in enumerate(counts):
        g = got[batch.cu[b]:batch.cu[b + 1]]
        delta = (2.0 ** -22 + (d / 16 + 6) * 2.0 ** -23) * errs[b][..., None]
        assert n == 0 or delta.max() <= 0.3
        top = (127 if kind == "i8" else 448) * np.nanmax(vs)
        tol = (4 * delta + (lens[b] / 16 + 64) * 2.0 ** -23 + e) * mags[b] + e * np.abs(outs[b])
        tol += 2.0 ** -38 * lens[b] * top + torch.finfo(DT[dtype]).eps * torch.finfo(DT[dtype]).tiny / 2
        bad = np.abs(g - outs[b]) > tol
        assert not bad.any(), (b, float(np.max(np.abs(g - outs[b])[bad])), float(np.max(tol[bad])))
        for i in range(min(n, max(n - lens[b], 0))):
            assert np.all(g[i] == 0)  # a token that sees nothing
    if out_fill is not None:
        assert np.all(got[batch.cu[-1]:] == out_fill)  # rows behind the last sequence


def filled(batch, kind, magnitude=1.0):
    """Pools whose rows below each length hold quantized normal rows; everything else is noise, NaN codes and scales
    included."""
    pools = []
    for _ in range(2):
        codes, scales = batch.pools8(kind)
        scales[:] = np.nan
        if kind == "e4m3":
            codes[:] = 0x7f
        rows = [(batch.rng.normal(size=(L, batch.Hkv, batch.d)) * magnitude *
                 np.exp(batch.rng.normal(size=(L, batch.Hkv, 1)) * 0.5)).astype(np.float32) for L in batch.lens]
        q8.append(rows, codes, scales, batch.table, batch.lens, batch.lens, batch.bt, kind)
        pools += [codes, scales]
    return pools


ATT = [
    # dtype, d, kind, bt, Hq, Hkv
    ("f32", 128, "i8", 16, 8, 2), ("f16", 128, "i8", 64, 8, 2), ("bf16", 128, "e4m3", 32, 16, 2),
    ("f32", 64, "e4m3", 128, 3, 3), ("bf16", 64, "i8", 16, 6, 2), ("f16", 64, "e4m3", 64, 14, 2),
    ("bf16", 128, "i8", 128, 16, 1), ("f16", 128, "e4m3", 16, 12, 1), ("f32", 128, "e4m3", 32, 13, 1)]


@pytest.mark.parametrize("dtype,d,kind,bt,Hq,Hkv", ATT)
def test_q8_decode_matches_the_oracle(dtype, d, kind, bt, Hq, Hkv):
    lens = [1, 0, 16, 17, 700, 333, 2, 95]
    bt_ = Batch([1] * 8, lens, Hq, Hkv, d, bt, dtype, 100 + d + bt, pad=0)
    pools = filled(bt_, kind)
    scale = 1.0 / math.sqrt(d)
    got = ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind)
    check_attention(got, bt_, [bt_.rows(bt_.qn, b) for b in range(8)], pools, kind, scale, dtype)


@pytest.mark.parametrize("dtype,d,kind,bt,Hq,Hkv", ATT)
@pytest.mark.parametrize("max_q", [None, 200])
def test_q8_ragged_queries_match_the_oracle(dtype, d, kind, bt, Hq, Hkv, max_q):
    counts, lens = [0, 1, 5, 16, 17, 129, 0, 3, 1, 70], [7, 1, 20, 16, 50, 300, 0, 2, 400, 70]
    bt_ = Batch(counts, lens, Hq, Hkv, d, bt, dtype, 200 + d + bt)
    pools = filled(bt_, kind)
    out = torch.full((bt_.n_tok, Hq, d), 55.0, dtype=DT[dtype], device="cuda")
    got = ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind,
                              cu_q=bt_.t["cu"], max_q=max_q, T=410, scale=0.2, out=out)
    check_attention(got, bt_, [bt_.rows(bt_.qn, b) for b in range(len(lens))], pools, kind, 0.2, dtype, out_fill=55.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("magnitude", [1e-4, 300.0])
def test_q8_attention_over_a_wide_range_of_scales(dtype, magnitude):
    """Values far below and above one, blocks of one sequence whose scales differ by 2^12, queries to match."""
    d, Hq, Hkv, bt = 128, 4, 1, 32
    bt_ = Batch([1, 9], [200, 150], Hq, Hkv, d, bt, dtype, 31, scale=1.0 / magnitude)
    pools = filled(bt_, "i8", magnitude)
    vs = pools[3]
    vs *= np.where(bt_.rng.random(vs.shape) < 0.5, np.float32(2.0 ** -12), np.float32(1))
    for cu, max_q in ((bt_.t["cu"], None), (bt_.t["cu"], 9)):
        got = ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], cu_q=cu, max_q=max_q)
        check_attention(got, bt_, [bt_.rows(bt_.qn, b) for b in range(2)], pools, "i8", 1 / math.sqrt(d), dtype)


def test_append_then_attend_as_a_server_does():
    """Prompt chunks, then single-token steps, through both calls; the attention output stays near unquantized
    attention, and the cache equals one filled by the oracle."""
    d, Hq, Hkv, bt, kind = 128, 8, 2, 32, "i8"
    tab = rope_table(600, d)
    steps = [([37, 120, 5], [37, 120, 5]), ([60, 1, 1], [97, 121, 6])] + [([1, 1, 1], [98 + i, 122 + i, 7 + i])
                                                                          for i in range(12)]
    final = steps[-1][1]
    pools = [np.zeros((16, Hkv, bt, d), np.uint8), np.zeros((16, Hkv, bt // 16 * 1), np.float32),
             np.zeros((16, Hkv, bt, d), np.uint8), np.zeros((16, Hkv, bt // 16), np.float32)]
    dev = [cuda(p) for p in pools]
    table = np.random.default_rng(3).permutation(15).reshape(3, 5).astype(np.int32)
    hist = [([], []) for _ in final]
    for n, (counts, lens) in enumerate(steps):
        bt_ = Batch(counts, lens, Hq, Hkv, d, bt, "bf16", 900 + n, pad=0)
        bt_.table = table
        tl, cu = bt_.t["lens"], bt_.t["cu"]
        qr = ops.q8_append_paged(bt_.k, bt_.v, *dev, cuda(table), tl, kind=kind, cu_new=cu, q=bt_.q, cos_sin=cuda(tab))
        out = ops.q8_attend_paged(qr, *dev, cuda(table), tl, kind=kind, cu_q=cu, max_q=max(counts))
        kr = bt_.rotated(bt_.kn, tab, False)
        q8.append(kr, pools[0], pools[1], table, lens, counts, bt, kind)
        q8.append([bt_.rows(bt_.vn, b) for b in range(3)], pools[2], pools[3], table, lens, counts, bt, kind)
        for b in range(3):
            hist[b][0].append(kr[b])
            hist[b][1].append(bt_.rows(bt_.vn, b))
        qn = qr.float().cpu().numpy()
        check_attention(out, bt_, [qn[bt_.cu[b]:bt_.cu[b + 1]] for b in range(3)], pools, kind, 1 / math.sqrt(d), "bf16")
    for a, w in zip(dev, pools):
        assert np.array_equal(a.cpu().numpy(), w)
    for b in range(3):  # the last step against unquantized attention
        k, v = np.concatenate(hist[b][0]).astype(np.float64), np.concatenate(hist[b][1]).astype(np.float64)
        s = np.einsum("hd,thd->ht", qn[b].astype(np.float64), np.repeat(k, Hq // Hkv, 1)) / math.sqrt(d)
        p = np.exp(s - s.max(1, keepdims=True))
        ref = np.einsum("ht,thd->hd", p / p.sum(1, keepdims=True), np.repeat(v, Hq // Hkv, 1))
        g = out[b].double().cpu().numpy()
        assert np.linalg.norm(g - ref) <= 0.05 * np.linalg.norm(ref)


def test_append_then_decode_through_the_lloyd_max_pools():
    """append_paged's queries and cache through attend_decode_paged give what the oracle makes of the rotated rows."""
    d, Hq, Hkv, bt, bits = 128, 8, 2, 32, 4
    tab, s = rope_table(300, d), W.sign_vector(d, 4)
    lens = [200, 1, 77]
    bt_ = Batch(lens, lens, Hq, Hkv, d, bt, "f16", 77, pad=0)
    z = lambda *sh, dt: torch.zeros(sh, dtype=dt, device="cuda")
    kc, vc = (z(bt_.nb, Hkv, bt, d // 2, dt=torch.uint8) for _ in range(2))
    kn, vn = (z(bt_.nb, Hkv, bt, dt=torch.float16) for _ in range(2))
    q = ops.append_paged(bt_.k, bt_.v, kc, kn, cuda(s), bits, bt_.t["table"], bt_.t["lens"], cu_new=bt_.t["cu"], q=bt_.q,
                         cos_sin=cuda(tab), vcodes=vc, vnorms=vn)
    last = torch.from_numpy(bt_.cu[1:].astype(np.int64) - 1).cuda()
    out = ops.attend_decode_paged(q[last].contiguous(), kc, kn, cuda(s), bits, bt_.t["table"], seq_lens=bt_.t["lens"],
                                  vcodes=vc, vnorms=vn, T=200).cpu().numpy()
    kr, qr = bt_.rotated(bt_.kn, tab, False), bt_.rotated(bt_.qn, tab, False)
    T = max(lens)
    k, v = np.zeros((3, Hkv, T, d), np.float32), np.zeros((3, Hkv, T, d), np.float32)
    for b, L in enumerate(lens):
        k[b, :, :L], v[b, :, :L] = kr[b].transpose(1, 0, 2), bt_.rows(bt_.vn, b).transpose(1, 0, 2)
    okc, okn = oracle.write(k, s, bits)
    ovc, ovn = oracle.write(v, s, bits)
    want = oracle.decode_attention(np.stack([r[-1] for r in qr]), okc, okn, s, bits, 1 / math.sqrt(d), vcodes=ovc,
                                   vn16=ovn, seq_lens=np.array(lens, np.int32))
    parity.check_outputs(out, want)


def test_q8_on_another_stream_and_in_a_graph():
    """A captured append + attend, replayed on new inputs and lengths, equals the eager calls; so does another stream."""
    d, Hq, Hkv, bt = 128, 8, 2, 32
    bt_ = Batch([1] * 3, [300, 17, 64], Hq, Hkv, d, bt, "bf16", 5, pad=0)
    pools = filled(bt_, "i8")
    tab = cuda(rope_table(400, d))

    def step(dev, q, k, v):
        qr = ops.q8_append_paged(k, v, *dev, bt_.t["table"], bt_.t["lens"], q=q, cos_sin=tab)
        return ops.q8_attend_paged(qr, *dev, bt_.t["table"], bt_.t["lens"], T=320)

    eager = [cuda(p) for p in pools]
    want = step(eager, bt_.q, bt_.k, bt_.v)
    side = [cuda(p) for p in pools]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = step(side, bt_.q, bt_.k, bt_.v)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got, want) and same(side, eager)
    cap = [cuda(p) for p in pools]
    fresh = [p.clone() for p in cap]
    buf = bt_.qkv.clone()
    q, k, v = (t.view(3, -1, d) for t in buf.split([Hq * d, Hkv * d, Hkv * d], 1))
    step(cap, q, k, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(cap, q, k, v)
    for a, b in zip(cap, fresh):
        a.copy_(b)
    g.replay()
    assert torch.equal(out, want) and same(cap, eager)
    buf.mul_(0.5)
    bt_.t["lens"].copy_(torch.tensor([299, 16, 63], dtype=torch.int32))
    for a, b in zip(cap, fresh):
        a.copy_(b)
    g.replay()
    again = [p.clone() for p in fresh]
    assert torch.equal(out, step(again, q, k, v)) and same(cap, again)


def test_q8_results_do_not_depend_on_the_batch_around_them():
    """Two runs are equal bit for bit (no order-dependent atomics)."""
    bt_ = Batch([1] * 4, [900, 10, 333, 64], 8, 2, 128, 32, "f32", 6, pad=0)
    dev = [cuda(p) for p in filled(bt_, "i8")]
    a, b = (ops.q8_attend_paged(bt_.q, *dev, bt_.t["table"], bt_.t["lens"]) for _ in range(2))
    assert torch.equal(a, b)


def test_out_of_range_tables_are_flagged_and_skipped():
    d, Hq, Hkv, bt = 128, 4, 2, 32
    bt_ = Batch([1, 1, 1], [40, 40, 40], Hq, Hkv, d, bt, "f16", 9, pad=0)
    pools = filled(bt_, "i8")
    dev = [cuda(p) for p in pools]
    tab = cuda(rope_table(40, d))
    table = bt_.table.copy()
    table[0, 1], table[1, 1] = -1, bt_.nb
    before = [x.clone() for x in dev]
    ops.device_status(clear=True)
    pos = cuda(np.array([39, 39, 40], np.int32))  # the third is past the rotation table
    qo = torch.full((3, Hq, d), 3.0, dtype=torch.float16, device="cuda")
    ops.q8_append_paged(bt_.k, bt_.v, *dev, cuda(table), bt_.t["lens"], q=bt_.q, cos_sin=tab, positions=pos, q_out=qo)
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX
    assert same(dev, before) and torch.all(qo == 3)
    ops.q8_attend_paged(bt_.q, *dev, cuda(table), bt_.t["lens"])  # in bounds, flagged
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX
    ops.q8_append_paged(bt_.k, bt_.v, *dev, bt_.t["table"], cuda(np.array([40, 97, 40], np.int32)), q=bt_.q,
                        cos_sin=cuda(rope_table(200, d)), q_out=qo)  # 97 is past the table's three blocks
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX
    assert torch.all(qo[1] == 3) and torch.all(qo[0] != 3)
    assert ops.device_status() == 0


def test_more_queries_than_max_q_is_flagged():
    bt_ = Batch([3, 1], [40, 40], 8, 2, 128, 32, "f32", 12)
    dev = [cuda(p) for p in filled(bt_, "i8")]
    ops.device_status(clear=True)
    out = torch.full((bt_.n_tok, 8, 128), 9.0, device="cuda")
    ops.q8_attend_paged(bt_.q, *dev, bt_.t["table"], bt_.t["lens"], cu_q=bt_.t["cu"], max_q=1, out=out)
    assert torch.all(out[:3] == 9) and torch.all(out[3] != 9)
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX


def test_refusals():
    bt_ = Batch([1, 1], [40, 40], 8, 2, 128, 32, "f16", 12, pad=0)
    dev = [cuda(p) for p in filled(bt_, "i8")]
    tab, tl = bt_.t["table"], bt_.t["lens"]
    with pytest.raises(ValueError, match="kind"):
        ops.q8_attend_paged(bt_.q, *dev, tab, tl, kind="int4")
    with pytest.raises(ValueError, match="CUDA"):
        ops.q8_attend_paged(bt_.q.cpu(), *dev, tab, tl)
    with pytest.raises(ValueError, match="contiguous"):
        ops.q8_attend_paged(bt_.q.transpose(1, 2).contiguous().transpose(1, 2), *dev, tab, tl)
    with pytest.raises(ValueError, match="one query token"):
        ops.q8_attend_paged(bt_.q[:1], *dev, tab, tl)
    with pytest.raises(TypeError):
        ops.q8_attend_paged(bt_.q.double(), *dev, tab, tl)
    with pytest.raises(_abi.AxrError):  # a token stride that is no multiple of 16 bytes
        odd = torch.zeros((2, 8 * 128 + 3), dtype=torch.float16, device="cuda")[:, :1024].view(2, 8, 128)
        ops.q8_attend_paged(odd, *dev, tab, tl)
    with pytest.raises(_abi.AxrError) as e:
        ops.q8_attend_paged(torch.zeros((2, 34, 128), device="cuda"), *dev, tab, tl)
    assert e.value.status == 2  # 17 query heads per KV head
    with pytest.raises(_abi.AxrError) as e:
        ops.q8_attend_paged(torch.zeros((2, 8, 128), device="cuda"), *dev, tab, tl, T=4000)
    assert e.value.status == 1
    with pytest.raises(ValueError, match="cos_sin"):
        ops.q8_append_paged(bt_.k, bt_.v, *dev, tab, tl, q=bt_.q)
    with pytest.raises(_abi.AxrError) as e:
        ops.q8_append_paged(bt_.k, bt_.v, *dev, tab, tl, cos_sin=torch.zeros((50, 24), device="cuda"))
    assert e.value.status == 2
    with pytest.raises(ValueError, match="one shape"):
        ops.q8_append_paged(bt_.k, bt_.v[:, :1], *dev, tab, tl)
    with pytest.raises(ValueError, match="exactly one"):
        ops.append_paged(bt_.k, bt_.v, torch.zeros((4, 2, 32, 64), dtype=torch.uint8, device="cuda"),
                         torch.zeros((4, 2, 32), dtype=torch.float16, device="cuda"),
                         torch.ones(128, dtype=torch.int8, device="cuda"), 4, tab, tl)
    # nothing to do
    none = torch.zeros((0, 2, 128), dtype=torch.float16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    ops.q8_append_paged(none, none, *dev, tab, tl, cu_new=cu)
    assert ops.q8_attend_paged(torch.zeros((0, 8, 128), device="cuda"), *dev, tab, tl, cu_q=cu).shape == (0, 8, 128)


# ---- further shapes of a call ----------------------------------------------------------------------------------------

def test_batches_of_more_than_32_sequences():
    """Sequence lookups of several rounds: 75 sequences, empty ones among them, through every entry point."""
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 4, 75).tolist()
    lens = [c + int(x) for c, x in zip(counts, rng.integers(0, 60, 75))]
    lens[40] = counts[40] = 0
    d, Hq, Hkv, bt, kind = 64, 4, 2, 16, "i8"
    bt_ = Batch(counts, lens, Hq, Hkv, d, bt, "f16", 41)
    tab, pools = rope_table(200, d), filled(bt_, kind)
    dev = [cuda(p) for p in pools]
    qr = ops.q8_append_paged(bt_.k, bt_.v, *dev, bt_.t["table"], bt_.t["lens"], kind=kind, cu_new=bt_.t["cu"], q=bt_.q,
                             cos_sin=cuda(tab))
    q8.append(bt_.rotated(bt_.kn, tab, False), pools[0], pools[1], bt_.table, lens, counts, bt, kind)
    q8.append([bt_.rows(bt_.vn, b) for b in range(75)], pools[2], pools[3], bt_.table, lens, counts, bt, kind)
    assert same(dev, [cuda(p) for p in pools])
    qn = qr.float().cpu().numpy()
    for dtype, max_q in (("f16", 3), ("f16", None), ("f32", None)):  # one tile a sequence, tcgen05, flat tiles
        qq = qr.to(DT[dtype])
        out = ops.q8_attend_paged(qq, *dev, bt_.t["table"], bt_.t["lens"], kind=kind, cu_q=bt_.t["cu"], max_q=max_q)
        check_attention(out, bt_, [qn[bt_.cu[b]:bt_.cu[b + 1]] for b in range(75)], pools, kind, 1 / math.sqrt(d), dtype)
    one = Batch([1] * 75, [max(x, 1) for x in lens], Hq, Hkv, d, bt, "bf16", 42, pad=0)
    pools = filled(one, kind)
    out = ops.q8_attend_paged(one.q, *[cuda(p) for p in pools], one.t["table"], one.t["lens"], kind=kind)
    check_attention(out, one, [one.rows(one.qn, b) for b in range(75)], pools, kind, 1 / math.sqrt(d), "bf16")


@pytest.mark.parametrize("dtype,counts,max_q", [("bf16", [1], 1), ("f32", [1], 1), ("f16", [9], 9), ("f16", [40], None),
                                                ("bf16", [300], None), ("f32", [3], None)])
def test_long_axes_split_over_the_gpu(dtype, counts, max_q):
    """One sequence of 20,011 tokens: the axis is cut into many partials, merged."""
    d, Hq, Hkv, bt, kind = 128, 4, 1, 64, "e4m3"
    bt_ = Batch(counts, [20011], Hq, Hkv, d, bt, dtype, 43, pad=2)
    pools = filled(bt_, kind)
    out = torch.full((bt_.n_tok, Hq, d), -3.0, dtype=DT[dtype], device="cuda")
    ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind, cu_q=bt_.t["cu"],
                        max_q=max_q, out=out)
    check_attention(out, bt_, [bt_.rows(bt_.qn, 0)], pools, kind, 1 / math.sqrt(d), dtype, out_fill=-3.0)


@pytest.mark.parametrize("scale", [-0.05, 0.0])
@pytest.mark.parametrize("counts", [[1, 1], [40, 90]])
def test_scales_that_are_not_positive(scale, counts):
    bt_ = Batch(counts, [100, 300], 8, 2, 128, 32, "bf16", 44, pad=0)
    pools = filled(bt_, "i8")
    out = ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], cu_q=bt_.t["cu"], scale=scale)
    check_attention(out, bt_, [bt_.rows(bt_.qn, b) for b in range(2)], pools, "i8", scale, "bf16")


@pytest.mark.parametrize("counts", [[1, 1, 1], [30, 80, 64]])
def test_blocks_of_zero_values_keep_their_weight(counts):
    """Values that are zero for a stretch of tokens (scale 0), tiny or large elsewhere: the zeros count in the
    normaliser."""
    bt_ = Batch(counts, [200, 130, 64], 8, 2, 128, 32, "f16", 45, pad=0)
    kc, ks, vc, vs = filled(bt_, "i8")
    for b in range(3):
        for t in range(0, 64, 16):
            page = bt_.table[b, t // 32]
            vc[page, :, t % 32:t % 32 + 16], vs[page, :, t % 32 // 16] = 0, 0.0
        for t in range(64, bt_.lens[b] - 48, 16):
            vs[bt_.table[b, t // 32], :, t % 32 // 16] *= np.float32(2.0 ** -9)
    pools = [kc, ks, vc, vs]
    out = ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], cu_q=bt_.t["cu"])
    check_attention(out, bt_, [bt_.rows(bt_.qn, b) for b in range(3)], pools, "i8", 1 / math.sqrt(128), "f16")


def test_pools_of_more_than_four_gigabytes():
    """Rows of the last pool blocks: element offsets pass 32 bits (K and V pools of 4.3 GB each)."""
    d, Hq, Hkv, bt, kind = 128, 8, 2, 64, "i8"
    nb = (1 << 32) // (Hkv * bt * d) + 40
    lens, counts = [200, 77, 130], [40, 1, 130]
    bt_ = Batch(counts, lens, Hq, Hkv, d, bt, "bf16", 46, pad=0)
    small = filled(bt_, kind)
    off = nb - bt_.nb
    big = [torch.empty((nb,) + p.shape[1:], dtype=torch.uint8 if p.dtype == np.uint8 else torch.float32, device="cuda")
           for p in small]
    for a, p in zip(big, small):
        a[off:] = cuda(p)
    table = cuda(np.where(bt_.table >= 0, bt_.table + off, -7).astype(np.int32))
    near = [cuda(p) for p in small]
    tab = cuda(rope_table(300, d))
    for tb, pl in ((table, big), (bt_.t["table"], near)):
        qr = ops.q8_append_paged(bt_.k, bt_.v, *pl, tb, bt_.t["lens"], kind=kind, cu_new=bt_.t["cu"], q=bt_.q, cos_sin=tab)
    assert same([a[off:].contiguous() for a in big], near)
    last = torch.from_numpy(bt_.cu[1:].astype(np.int64) - 1).cuda()
    for q, kw in ((qr, dict(cu_q=bt_.t["cu"])), (qr[last].contiguous(), {})):
        assert torch.equal(ops.q8_attend_paged(q, *big, table, bt_.t["lens"], kind=kind, T=256, **kw),
                           ops.q8_attend_paged(q, *near, bt_.t["table"], bt_.t["lens"], kind=kind, T=256, **kw))
    del big
    torch.cuda.empty_cache()


def test_two_graphs_that_share_a_workspace():
    """A decode step and a chunk, each captured with one caller workspace, replayed in turn."""
    d, Hq, Hkv, bt = 128, 8, 2, 32
    a = Batch([1] * 3, [900, 17, 640], Hq, Hkv, d, bt, "bf16", 47, pad=0)
    b = Batch([33, 70], [900, 300], Hq, Hkv, d, bt, "bf16", 48, pad=0)
    pa, pb = [cuda(p) for p in filled(a, "i8")], [cuda(p) for p in filled(b, "i8")]
    need = max(ops.q8_attend_workspace_bytes(3, 1, 3, Hq, Hkv, 960, d),
               ops.q8_attend_workspace_bytes(103, 70, 2, Hq, Hkv, 960, d))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls = [lambda o=None: ops.q8_attend_paged(a.q, *pa, a.t["table"], a.t["lens"], T=960, workspace=ws, out=o),
             lambda o=None: ops.q8_attend_paged(b.q, *pb, b.t["table"], b.t["lens"], cu_q=b.t["cu"], max_q=70, T=960,
                                                workspace=ws, out=o)]
    want = [c() for c in calls]
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for c, o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c(o)
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    with pytest.raises(_abi.AxrError) as e:
        ops.q8_attend_paged(a.q, *pa, a.t["table"], a.t["lens"], T=960, workspace=ws[:64])
    assert e.value.status == 4


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("counts,max_q", [([1, 1, 1], 1), ([30, 80, 64], 80)])
def test_a_query_row_that_is_not_finite_stays_alone(dtype, counts, max_q):
    """NaN and infinite queries give NaN in their own rows and change no others."""
    Hq, Hkv, d, bt = 8, 2, 128, 32
    bt_ = Batch(counts, [500, 81, 300], Hq, Hkv, d, bt, dtype, 77, pad=0)
    pools = [cuda(p) for p in filled(bt_, "i8")]
    args = pools + [bt_.t["table"], bt_.t["lens"]]
    good = ops.q8_attend_paged(bt_.q, *args, cu_q=bt_.t["cu"], max_q=max_q)
    q = bt_.q.clone()
    rows = [(0, 3, 5, math.nan), (bt_.n_tok - 1, 7, 64, math.inf)]
    for i, h, j, x in rows:
        q[i, h, j] = x
    got = ops.q8_attend_paged(q, *args, cu_q=bt_.t["cu"], max_q=max_q)
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    for i, h, _, _ in rows:
        assert torch.isnan(got[i, h]).all(), (i, h)
        keep[i, h] = False
    assert torch.equal(got[keep], good[keep])


@pytest.mark.parametrize("counts", [[1, 1], [40, 90]])
def test_an_axis_of_no_tokens(counts):
    bt_ = Batch(counts, [64, 96], 8, 2, 64, 32, "bf16", 8, pad=0)
    pools = [cuda(p) for p in filled(bt_, "i8")]
    out = ops.q8_attend_paged(bt_.q, *pools, bt_.t["table"], bt_.t["lens"], cu_q=bt_.t["cu"], max_q=max(counts), T=0)
    assert (out == 0).all()


def test_interleaved_takes_a_truth_value():
    bt_ = Batch([1, 1], [40, 40], 8, 2, 128, 32, "f16", 13, pad=0)
    pools = [cuda(p) for p in filled(bt_, "i8")]
    before = [p.clone() for p in pools]
    with pytest.raises(RuntimeError):
        ops.q8_append_paged(bt_.k, bt_.v, *pools, bt_.t["table"], bt_.t["lens"],
                            cos_sin=cuda(rope_table(64, 128)), interleaved=torch.zeros(2))
    torch.cuda.synchronize()
    assert same(pools, before)


@pytest.mark.parametrize("dtype,Hq,Hkv,kind", [("bf16", 8, 2, "i8"), ("f16", 16, 1, "e4m3"), ("f16", 3, 3, "i8")])
@pytest.mark.parametrize("counts", [[1, 1, 90, 0, 2, 1, 3, 1, 8, 9, 17, 1], [129, 100, 1, 90, 120], [1, 300], [300, 1, 2]])
def test_short_sequences_among_long_ones(dtype, Hq, Hkv, kind, counts):
    """Batches that both attention kernels share and batches that one takes, with a workspace of the size asked for."""
    lens = [n + 37 * i % 411 for i, n in enumerate(counts)]
    bt_ = Batch(counts, lens, Hq, Hkv, 128, 32, dtype, 91)
    pools = filled(bt_, kind)
    out = torch.full((bt_.n_tok, Hq, 128), 55.0, dtype=DT[dtype], device="cuda")
    T, mq = max(lens), max(counts)
    need = ops.q8_attend_workspace_bytes(bt_.n_tok, mq, len(lens), Hq, Hkv, T, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ops.device_status(clear=True)
    ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind, cu_q=bt_.t["cu"],
                        max_q=mq, T=T, out=out, workspace=ws)
    assert ops.device_status() == 0
    check_attention(out, bt_, [bt_.rows(bt_.qn, b) for b in range(len(lens))], pools, kind, 1 / math.sqrt(128), dtype,
                    out_fill=55.0)


@pytest.mark.parametrize("dtype,kind", [("bf16", "i8"), ("f16", "e4m3")])
@pytest.mark.parametrize("counts,lens", [
    ([250] + [1] * 30, [1500] + [37 * i % 1400 + 1 for i in range(30)]),   # a split axis, most tiles without work
    ([5] * 12, [1000 + 40 * i for i in range(12)]),                        # one tile a sequence, a split axis
    ([64, 65, 63, 10, 0, 64], [800, 65, 1200, 300, 9, 64])])               # row tiles that end on a token and behind it
def test_long_axes_of_mixed_batches(dtype, kind, counts, lens):
    bt_ = Batch(counts, lens, 8, 2, 128, 64, dtype, 93)
    pools = filled(bt_, kind)
    out = torch.full((bt_.n_tok, 8, 128), 55.0, dtype=DT[dtype], device="cuda")
    ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind, cu_q=bt_.t["cu"],
                        max_q=max(counts), T=max(lens), out=out)
    check_attention(out, bt_, [bt_.rows(bt_.qn, b) for b in range(len(lens))], pools, kind, 1 / math.sqrt(128), dtype,
                    out_fill=55.0)


def test_more_queries_than_max_q_on_a_split_axis_is_flagged():
    bt_ = Batch([7, 9], [4000, 3000], 8, 2, 128, 64, "bf16", 94, pad=0)
    pools = [cuda(p) for p in filled(bt_, "i8")]
    args = pools + [bt_.t["table"], bt_.t["lens"]]
    want = ops.q8_attend_paged(bt_.q, *args, cu_q=bt_.t["cu"], max_q=9)
    assert ops.device_status(clear=True) == 0
    out = torch.full_like(want, 55.0)
    ops.q8_attend_paged(bt_.q, *args, cu_q=bt_.t["cu"], max_q=8, out=out)
    assert ops.device_status(clear=True) == 2
    assert torch.equal(out[:15], want[:15])  # the ninth token of the second sequence may or may not be written
    assert torch.equal(out[15], want[15]) or (out[15] == 55.0).all()

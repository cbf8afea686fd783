"""Attention over the 8-bit cache and the paged appends at the ends of what a call may hold: value scales and queries from
fp32's smallest magnitudes to its largest, lengths and offsets out of range, a split of the token axis beside many single
tokens."""

import math

import numpy as np
import pytest
import torch

from kv_cache_quantized_b200 import _abi, ops
from oracle import q8
from tests.test_gpu_q8 import DT, Batch, cuda, filled, rope_table, same

pytestmark = pytest.mark.gpu

# one query token a sequence (the warp-MMA kernel), flat tiles of the same kernel (fp32), the tcgen05 kernel
FORMS = [("f32", [1, 1, 1]), ("bf16", [1, 1, 1]), ("f16", [1, 1, 1]), ("f32", [30, 40, 64]), ("bf16", [30, 40, 64]),
         ("f16", [30, 40, 64])]


def uses_tcgen05(dtype, counts, G):
    return dtype != "f32" and max(counts) * G > 16


def check(got, bt_, pools, kind, scale, dtype, G, T=None):
    """|o - ref| <= (4 delta + (T / 16 + 64) 2^-23 + e) A + e |ref| + floor, as in check_attention, with the floor of the
    kernel that the call takes.  A weight enters as p vs / vref times a power of two, vref < 2 max vs being the power of
    two at or above the largest value scale met so far:
    * warp-MMA kernel: times 2^14 in fp16 planes whose last step is 2^-24, so a weight is off by up to 2^-25 of that,
      2^-39 vref < 2^-38 max vs, times a code;
    * tcgen05 kernel: times 2^9 in one plane (the running maximum may lag by 2^6), so up to 2^-34 vref < 2^-33 max vs;
    for each of T weights, over a normaliser of at least 1; vref is not below 2^-126.  Beside it, results below fp32's
    normal range are rounded to its step of 2^-149: half a step for each of at most T / 64 + 4 partials and the output."""
    kc, ks, vc, vs = pools
    q = [bt_.rows(bt_.qn, b) for b in range(len(bt_.lens))]
    outs, mags, errs = q8.attend(q, kc, ks, vc, vs, bt_.table, bt_.lens, bt_.counts, bt_.bt, kind, scale, T)
    fi = torch.finfo(DT[dtype])
    e = fi.eps / 2 if dtype != "f32" else 0.0
    step = 2.0 ** -33 if uses_tcgen05(dtype, bt_.counts, G) else 2.0 ** -38
    got = got.double().cpu().numpy()
    for b in range(len(bt_.lens)):
        g = got[bt_.cu[b]:bt_.cu[b + 1]]
        delta = (2.0 ** -22 + (bt_.d / 16 + 6) * 2.0 ** -23) * errs[b][..., None]
        assert bt_.counts[b] == 0 or delta.max() <= 0.3
        L = bt_.lens[b]
        top = (127 if kind == "i8" else 448) * max(np.nanmax(vs.astype(np.float64)), 2.0 ** -127)
        tol = (4 * delta + (L / 16 + 64) * 2.0 ** -23 + e) * mags[b] + e * np.abs(outs[b]) + step * L * top
        tol += fi.eps * fi.tiny / 2 + (L / 64 + 4) * 2.0 ** -150
        bad = ~(np.abs(g - outs[b]) <= tol)
        assert not bad.any(), (b, int(bad.sum()), float(np.abs(g - outs[b])[bad].max()), float(tol[bad].max()))


def attend(bt_, pools, kind="i8", scale=None, **kw):
    one = max(bt_.counts) == 1 and min(bt_.counts) == 1
    return ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], bt_.t["table"], bt_.t["lens"], kind=kind,
                               cu_q=None if one else bt_.t["cu"], max_q=None if one else max(bt_.counts), scale=scale, **kw)


# ---- value scales ----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,counts", FORMS)
@pytest.mark.parametrize("tiny", [9.2e-41, 2.0 ** -126, 2.0 ** -114])
def test_tiny_value_scales_before_ordinary_ones(dtype, counts, tiny):
    """Blocks of zero values that a converted cache holds under a tiny scale, at the start of each sequence."""
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 301, pad=0)
    pools = filled(bt_, "i8")
    for b in range(3):
        for t in range(0, 64, 16):
            page = bt_.table[b, t // 32]
            pools[2][page, :, t % 32:t % 32 + 16] = 0
            pools[3][page, :, t % 32 // 16] = tiny
    check(attend(bt_, pools), bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


@pytest.mark.parametrize("dtype,counts", [f for f in FORMS if f[0] != "f16"])  # (fp16 holds no such outputs)
@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("power", [-149, -140, -126, -114, 106])
def test_value_scales_at_the_ends_of_fp32(dtype, counts, kind, power):
    """Every value scale of one magnitude: 2^power to 2^(power + 4) (outputs below 2^-126 are subnormal)."""
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 302, pad=0)
    pools = filled(bt_, kind)
    vs = pools[3]
    grow = 2.0 ** bt_.rng.integers(0, 5, vs.shape)
    pools[3] = np.where(np.isnan(vs), vs, (2.0 ** power * grow).astype(np.float32)).astype(np.float32)
    assert 2.0 ** (power + 4) * 448 * 300 < 2.0 ** 128  # sums over the cache stay within fp32
    check(attend(bt_, pools, kind), bt_, pools, kind, 1 / math.sqrt(128), dtype, 4)


@pytest.mark.parametrize("dtype,counts", FORMS)
def test_attention_on_blocks_of_small_value_scale(dtype, counts):
    """Rows whose weight lies on blocks with value scales 2^-20 to 2^-26 of another visible block's: held to the floors
    that the kernels state, 2^-38 or 2^-33 of the largest scale."""
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 303, pad=0)
    pools = filled(bt_, "i8")
    kc, ks, vc, vs = pools
    for b in range(3):  # the first block keeps its scale and one value; all other coordinates come from small blocks
        page = bt_.table[b, 0]
        vc[page, :, :16] = 0
        vc[page, :, 0, 0] = 127
        for t in range(16, bt_.lens[b], 16):
            vs[bt_.table[b, t // 32], :, t % 32 // 16] *= np.float32(2.0 ** -bt_.rng.integers(20, 27))
    check(attend(bt_, pools), bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


# ---- appends onto tiny scales ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("old", [9.2e-41, 2.0 ** -130, 2.0 ** -120, 2.0 ** -108, 2.0 ** -107])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -125, 2.0 ** -101, 2.0 ** -99, 1.0])
def test_appends_onto_older_tokens_under_a_tiny_scale(kind, old, size):
    """A converted cache's older tokens under a scale below any that an append sets: the new codes are the formula's, bit
    for bit, where 1 / s overflows (zeros stay zeros) and where x / s passes the largest code."""
    d, Hkv, bt, n = 128, 2, 32, 3
    rng = np.random.default_rng(21)
    k, v = ((rng.uniform(0.5, 1, (n, Hkv, d)) * rng.choice([-1, 0, 1], (n, Hkv, d)) * size).astype(np.float32) for _ in "kv")
    kc, vc = (rng.integers(0, 100, (2, Hkv, bt, d)).astype(np.uint8) for _ in "kv")
    ks, vs = (np.full((2, Hkv, 2), old, np.float32) for _ in "kv")
    dev = [cuda(a) for a in (kc, ks, vc, vs)]
    table, lens = np.array([[1]], np.int32), [8 + n]
    ops.q8_append_paged(cuda(k), cuda(v), *dev, cuda(table), cuda(np.array(lens, np.int32)), kind=kind,
                        cu_new=cuda(np.array([0, n], np.int32)))
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        q8.append([k], kc, ks, table, lens, [n], bt, kind)
        q8.append([v], vc, vs, table, lens, [n], bt, kind)
    for name, a, w in zip(("kcodes", "kscales", "vcodes", "vscales"), dev, (kc, ks, vc, vs)):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), w.view(np.uint8)), name


# ---- queries ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,counts", [f for f in FORMS if f[0] != "f16"])
@pytest.mark.parametrize("power", [-120, -104, 104, 115, 118, 124])
def test_queries_of_extreme_magnitude(dtype, counts, power):
    """Finite queries far from one, key scales to match: the scores are ordinary."""
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 304, pad=0, scale=2.0 ** power)
    pools = filled(bt_, "i8")
    pools[1] = (pools[1] * np.float32(2.0 ** -power)).astype(np.float32)
    check(attend(bt_, pools), bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


# ---- lengths and offsets out of range --------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,counts", FORMS)
@pytest.mark.parametrize("T", [256, 100, 37])
def test_lengths_past_the_bound_keep_their_positions(dtype, counts, T):
    """Keys at or past T are not seen; a token's causal limit stays its own position; the call is flagged."""
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 305, pad=0)
    pools = filled(bt_, "i8")
    ops.device_status(clear=True)
    got = attend(bt_, pools, T=T)
    assert ops.device_status(clear=True) == _abi.STATUS_BAD_INDEX
    check(got, bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4, T)
    got = attend(bt_, pools, T=300)
    assert ops.device_status() == 0
    check(got, bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


@pytest.mark.parametrize("dtype,counts", FORMS)
def test_a_negative_length_is_flagged_and_counts_as_none(dtype, counts):
    bt_ = Batch(counts, [300, 150, 96], 8, 2, 128, 32, dtype, 306, pad=0)
    pools = filled(bt_, "i8")
    bt_.t["lens"][1] = -7
    bt_.lens = [300, 0, 96]
    ops.device_status(clear=True)
    got = attend(bt_, pools)
    assert ops.device_status(clear=True) == _abi.STATUS_BAD_INDEX
    assert torch.all(got[int(bt_.cu[1]):int(bt_.cu[2])] == 0)
    check(got, bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


@pytest.mark.parametrize("dtype,max_q", [("f32", None), ("bf16", None), ("bf16", 3), ("f16", 64)])
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 3, 6, 99], [-2, 3, 6, 8], [90, 91, 92, 93]])
def test_offsets_that_make_no_sense_are_flagged(dtype, max_q, cu):
    """Decreasing, negative or too large offsets: their sequence counts as empty, and the call is flagged, by the attention
    and by both appends, while every other sequence whose tokens are its own is served."""
    good = Batch([3, 3, 2], [40, 50, 60], 8, 2, 128, 32, dtype, 307, pad=0)
    pools = filled(good, "i8")
    bad = cuda(np.array(cu, np.int32))
    dev = [cuda(p) for p in pools]
    ops.device_status(clear=True)
    ops.q8_attend_paged(good.q, *dev, good.t["table"], good.t["lens"], cu_q=bad, max_q=max_q)
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX
    ops.q8_append_paged(good.k, good.v, *dev, good.t["table"], good.t["lens"], cu_new=bad)
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX
    z = lambda *sh, dt: torch.zeros(sh, dtype=dt, device="cuda")
    ops.append_paged(good.k, good.v, z(good.nb, 2, 32, 64, dt=torch.uint8), z(good.nb, 2, 32, dt=torch.float16),
                     torch.ones(128, dtype=torch.int8, device="cuda"), 4, good.t["table"], good.t["lens"], cu_new=bad,
                     v=z(good.nb, 2, 32, 128, dt=torch.float16))
    assert ops.device_status(clear=True) & _abi.STATUS_BAD_INDEX


def test_a_negative_length_is_flagged_by_the_appends():
    bt_ = Batch([3, 3, 2], [40, 50, 60], 8, 2, 128, 32, "f16", 308, pad=0)
    pools = filled(bt_, "i8")
    dev = [cuda(p) for p in pools]
    bt_.t["lens"][:] = torch.tensor([-1, -40, -2 ** 31])
    before = [p.clone() for p in dev]
    qo = torch.full((8, 8, 128), 3.0, dtype=torch.float16, device="cuda")
    ops.device_status(clear=True)
    ops.q8_append_paged(bt_.k, bt_.v, *dev, bt_.t["table"], bt_.t["lens"], cu_new=bt_.t["cu"], q=bt_.q, q_out=qo,
                        cos_sin=cuda(rope_table(64, 128)))
    assert ops.device_status(clear=True) == _abi.STATUS_BAD_INDEX
    assert same(dev, before) and torch.all(qo == 3)
    kc, kn = torch.full((bt_.nb, 2, 32, 64), 9, dtype=torch.uint8, device="cuda"), torch.ones((bt_.nb, 2, 32), device="cuda").half()
    v = torch.ones((bt_.nb, 2, 32, 128), device="cuda").half()
    ops.append_paged(bt_.k, bt_.v, kc, kn, torch.ones(128, dtype=torch.int8, device="cuda"), 4, bt_.t["table"],
                     bt_.t["lens"], cu_new=bt_.t["cu"], v=v)
    assert ops.device_status(clear=True) == _abi.STATUS_BAD_INDEX
    assert torch.all(kc == 9) and torch.all(kn == 1) and torch.all(v == 1)


# ---- one sequence, alone and among others ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,counts", FORMS)
def test_a_sequence_alone_and_among_others(dtype, counts):
    """The other sequences of a batch decide where the token axis is cut, so the bits may differ; both results lie within
    the bound, and the same call gives the same bits."""
    bt_ = Batch(counts, [900, 333, 64], 8, 2, 128, 32, dtype, 309, pad=0)
    pools = filled(bt_, "i8")
    a, b = attend(bt_, pools), attend(bt_, pools)
    assert torch.equal(a, b)
    check(a, bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)
    dev = [cuda(p) for p in pools]
    alone = []
    for s in range(3):
        lo, hi = int(bt_.cu[s]), int(bt_.cu[s + 1])
        cu = cuda(np.array([0, hi - lo], np.int32))
        alone.append(ops.q8_attend_paged(bt_.q[lo:hi], *dev, bt_.t["table"][s:s + 1], bt_.t["lens"][s:s + 1],
                                         cu_q=None if max(counts) == 1 else cu, max_q=hi - lo))
    check(torch.cat(alone), bt_, pools, "i8", 1 / math.sqrt(128), dtype, 4)


# ---- a split axis beside many single tokens --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,kind", [("bf16", "i8"), ("f16", "e4m3")])
def test_a_chunk_on_a_long_axis_beside_many_single_tokens(dtype, kind):
    """A chunk whose token axis is split, among more numbered tiles than SMs; the workspace is of the size asked for, and
    what lies behind it stays as it was."""
    counts = [1] * 100 + [64] + [1] * 99
    lens = [1 + 7 * i % 90 for i in range(100)] + [4100] + [1 + 5 * i % 60 for i in range(99)]
    bt_ = Batch(counts, lens, 16, 8, 64, 64, dtype, 310)
    pools = filled(bt_, kind)
    T = 16384  # a bound that a server with long sequences would give
    table = np.full((200, T // 64), -7, np.int32)
    table[:, :bt_.mb] = bt_.table
    need = ops.q8_attend_workspace_bytes(bt_.n_tok, 64, 200, 16, 8, T, 64)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((bt_.n_tok, 16, 64), 55.0, dtype=DT[dtype], device="cuda")
    ops.device_status(clear=True)
    ops.q8_attend_paged(bt_.q, *[cuda(p) for p in pools], cuda(table), bt_.t["lens"], kind=kind, cu_q=bt_.t["cu"], max_q=64,
                        T=T, out=out, workspace=ws[:need])
    assert ops.device_status() == 0
    assert torch.all(ws[need:] == 77) and torch.all(out[int(bt_.cu[-1]):] == 55.0)
    check(out, bt_, pools, kind, 1 / math.sqrt(64), dtype, 2)

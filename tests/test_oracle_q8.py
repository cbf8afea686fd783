"""Pins of the 8-bit cache oracle (CPU): the e4m3 code against torch's, the rotation against complex arithmetic, the
scale rule, and the bound of a block's codes through growth."""

import numpy as np
import pytest
import torch

from oracle import q8


def test_e4m3_codes_match_the_float_type():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = q8.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    rng = np.random.default_rng(0)
    mid = (q8._POS[1:] + q8._POS[:-1]) / 2
    y = np.concatenate([rng.normal(0, 80, 20000), rng.normal(0, 0.01, 5000), mid, -mid, [448, -448, 460, 0.0, -0.0]])
    y = y.astype(np.float32)
    want = torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q8.to_e4m3(y), want)
    assert q8.to_e4m3(np.float32([np.nan, np.inf, -np.inf])).tolist() == [0, 126, 254]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product(interleaved):
    rng = np.random.default_rng(1)
    d, rot = 64, 32
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    x = rng.normal(size=(3, d)).astype(np.float32)
    y = q8.rotate(x, table, 37, interleaved)
    a, b = (x[:, 0:rot:2], x[:, 1:rot:2]) if interleaved else (x[:, :rot // 2], x[:, rot // 2:rot])
    z = (a + 1j * b) * np.exp(1j * ang[37])
    ya, yb = (y[:, 0:rot:2], y[:, 1:rot:2]) if interleaved else (y[:, :rot // 2], y[:, rot // 2:rot])
    assert np.max(np.abs(ya - z.real)) < 1e-6 and np.max(np.abs(yb - z.imag)) < 1e-6
    assert np.array_equal(y[:, rot:], x[:, rot:])


def test_scale_rule():
    assert q8.need(0.0, "i8") == 0 and q8.need(2.0 ** -101, "e4m3") == 0
    assert q8.need(127.0, "i8") == 1.0
    assert q8.need(448.0, "e4m3") == 1.0 and q8.need(np.nextafter(np.float32(448), np.float32(500)), "e4m3") == 2.0
    assert q8.need(0.875, "e4m3") == 2.0 ** -9


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_appending_one_by_one_stays_within_the_growth_bound(kind):
    """A code is off by at most half a code per rounding of the scale then in force, and scales only grow: with r
    roundings of a row (its write and each later growth), |x - code s| <= r s / 2 (int8); an e4m3 block grows exactly
    (its scales are powers of two), so its error is that of one rounding, half a unit of the last place, but for
    subnormal codes, whose step is 2^-9 s: at most r half steps of it."""
    rng = np.random.default_rng(2)
    d, bt, n = 64, 32, 32
    x = rng.normal(size=(n, 1, d)).astype(np.float32) * np.linspace(0.3, 3, n, dtype=np.float32)[:, None, None]
    codes, scales = np.zeros((1, 1, bt, d), np.uint8), np.full((1, 1, 2), 7.0, np.float32)
    table, growths, prev = [[0]], np.zeros(2, int), None
    for i in range(n):
        before = scales.copy()
        q8.append([x[i:i + 1]], codes, scales, table, [i + 1], [1], bt, kind)
        if i % 16:
            growths += (scales != before)[0, 0]
    v = q8.values(codes[0, 0], kind) * np.repeat(scales[0, 0], 16)[:, None].astype(np.float64)
    err = np.abs(v - x[:, 0])
    s = np.repeat(scales[0, 0], 16)[:, None].astype(np.float64)
    r = np.repeat(growths + 1, 16)[:, None]
    slack = 1 + 2.0 ** -20  # the fp32 roundings of 1 / s and x * (1 / s)
    if kind == "i8":
        assert np.all(err <= r * s / 2 * slack)
    else:
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x[:, 0]), r * s * 2.0 ** -10) * slack)
    assert growths.sum() > 0


FAKE = 0x10000  # never dereferenced: every call below fails validation, or has nothing to do


@pytest.fixture(scope="module")
def L():
    import os

    from kv_cache_quantized_b200 import _abi
    if not os.path.exists(_abi.LIB_PATH):
        from kv_cache_quantized_b200 import build
        build.build()
    return _abi.lib()


def _append8(L, **kw):
    a = dict(dict(q=FAKE, k=FAKE, v=FAKE, dt=1, qs=1024, ks=256, vs=256, cs=FAKE, mp=100, rot=128, inter=0, pos=None,
                  cu=None, lens=FAKE, n=2, B=2, Hq=8, Hkv=2, d=128, kind=0, kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE,
                  tab=FAKE, mb=4, bt=32, nb=9, qo=FAKE), **kw)
    return L.axr_q8_append_paged(*a.values(), None)


def test_q8_append_argument_errors(L):
    assert _append8(L, dt=3) == 1 and _append8(L, kind=2) == 1 and _append8(L, n=-1) == 1
    assert _append8(L, d=96) == 2 and _append8(L, rot=24) == 2 and _append8(L, rot=144) == 2
    assert _append8(L, Hq=7) == 1 and _append8(L, qo=None) == 1 and _append8(L, cs=None) == 1
    assert _append8(L, n=3) == 1 and b"one token per sequence" in L.axr_last_error()
    assert _append8(L, bt=48) == 1 and _append8(L, bt=8) == 1 and _append8(L, nb=0) == 1 and _append8(L, tab=None) == 1
    assert _append8(L, ks=255) == 1 and _append8(L, ks=257) == 1 and _append8(L, k=FAKE + 2) == 1
    assert _append8(L, ks=128) == 1 and _append8(L, kc=None) == 1 and _append8(L, kc=FAKE + 4) == 1
    assert _append8(L, lens=None) == 1 and _append8(L, mp=0) == 1 and _append8(L, mb=(1 << 25) + 1) == 1
    assert _append8(L, n=0, B=0) == 0
    assert _append8(L, n=16385, B=16385) == 2 and b"sequences" in L.axr_last_error()


def test_append_argument_errors(L):
    def call(**kw):
        a = dict(dict(q=FAKE, k=FAKE, v=FAKE, dt=1, qs=1024, ks=256, vs=256, cs=FAKE, mp=100, rot=128, inter=0,
                      pos=None, cu=FAKE, lens=FAKE, n=5, B=2, Hq=8, Hkv=2, d=128, bits=4, s=FAKE, kc=FAKE, kn=FAKE,
                      vk=1, v_=FAKE, vn=FAKE, tab=FAKE, mb=4, bt=32, nb=9, qo=FAKE), **kw)
        return L.axr_append_paged(*a.values(), None)
    assert call(bits=5) == 2 and call(vk=2) == 1 and call(vn=None) == 1 and call(s=None) == 1
    assert call(dt=7) == 1 and call(d=8) == 2 and call(cu=FAKE + 2) == 1 and call(v_=FAKE + 8) == 1
    assert call(n=0) == 0


def test_q8_attend_argument_errors(L):
    def call(**kw):
        a = dict(dict(q=FAKE, dt=1, qs=1024, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, kind=0, tab=FAKE, mb=300, bt=32, nb=9,
                      cu=None, lens=FAKE, n=2, mq=0, B=2, Hq=8, Hkv=2, T=9000, d=128, scale=0.1, out=FAKE, ws=None,
                      wsb=0), **kw)
        return L.axr_q8_attend_paged(*a.values(), None)
    assert call(dt=3) == 1 and call(kind=-1) == 1 and call(T=9601) == 1 and call(Hq=9) == 1
    assert call(d=32) == 2 and call(Hq=34) == 2 and call(n=3) == 1 and call(bt=20) == 1
    assert call(scale=float("nan")) == 1 and call(out=None) == 1 and call(out=FAKE + 8) == 1 and call(qs=1028) == 1
    assert call() == 4 and b"workspace" in L.axr_last_error()
    need = L.axr_q8_attend_workspace_bytes(2, 1, 2, 8, 2, 9000, 128)
    assert need > 0 and call(ws=FAKE, wsb=need - 1) == 4 and call(ws=FAKE + 8, wsb=need) == 1
    assert call(n=0, B=0) == 0
    assert L.axr_q8_attend_workspace_bytes(0, 1, 2, 8, 2, 9000, 128) == 0
    # T = 0 (every sequence cut to nothing) is a call like others, and its workspace is what the call asks for
    need = L.axr_q8_attend_workspace_bytes(2, 1, 2, 8, 2, 0, 128)
    assert need > 0 and call(T=0, ws=FAKE, wsb=need - 1) == 4 and call(T=0, ws=FAKE + 8, wsb=need) == 1
    # large batches and long axes do not multiply
    assert 0 < L.axr_q8_attend_workspace_bytes(16500, 60, 16384, 32, 8, 1 << 20, 128) < 1 << 29
    assert 0 < L.axr_q8_attend_workspace_bytes(4, 4, 1, 32, 2, 1 << 30, 128) < 1 << 29
    assert call(n=16385, B=16385) == 2 and L.axr_q8_attend_workspace_bytes(16385, 1, 16385, 8, 2, 9000, 128) == 0

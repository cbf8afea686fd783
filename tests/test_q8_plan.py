"""The split of the token axis in attention over the 8-bit cache, as its workspace shows it (CPU: no call is made)."""

import os

import pytest


@pytest.fixture(scope="module")
def L():
    from kv_cache_quantized_b200 import _abi
    if not os.path.exists(_abi.LIB_PATH):
        from kv_cache_quantized_b200 import build
        build.build()
    return _abi.lib()


def row_bytes(n_tok, Hq, d):
    """One partial (o, m, l) of every query row."""
    return n_tok * Hq * (d + 2) * 4


@pytest.mark.parametrize("singles", [60, 100, 199])
def test_a_chunk_beside_many_single_tokens_splits_its_axis(L, singles):
    """A chunk of 64 tokens on up to 32768 keys keeps 8 blocks busy (one for each KV head) unless its axis is split, however
    many sequences of one token stand beside it; the workspace holds the rows that exist, not those of every tile."""
    n, B = singles + 64, singles + 1
    need = L.axr_q8_attend_workspace_bytes(n, 64, B, 32, 8, 32768, 128)
    assert 5 * row_bytes(n, 32, 128) <= need <= 64 << 20


@pytest.mark.parametrize("n_tok,max_q,B,Hq,Hkv,T", [
    (16500, 60, 16384, 32, 8, 1 << 20), (4096, 4096, 1, 64, 8, 1 << 30), (40, 40, 1, 16, 1, 1 << 30),
    (20000, 200, 400, 32, 8, 1 << 17), (16384 + 2000, 2001, 16384, 16, 16, 1 << 20)])
def test_the_workspace_is_bounded(L, n_tok, max_q, B, Hq, Hkv, T):
    assert 0 < L.axr_q8_attend_workspace_bytes(n_tok, max_q, B, Hq, Hkv, T, 128) <= 1 << 29


@pytest.mark.parametrize("n_tok,max_q,B,Hq,Hkv,T", [
    (4096, 2048, 2, 32, 8, 8192), (4096, 1024, 4, 32, 8, 8192), (8192, 2048, 4, 32, 8, 8192), (1024, 512, 2, 32, 8, 8192)])
def test_prompt_chunks_that_fill_the_gpu_are_not_split(L, n_tok, max_q, B, Hq, Hkv, T):
    """Partials of full row tiles cost more than an uneven last wave of blocks: a split of these calls took 20 to 40 %
    longer.  (A split would ask for at least two partials of every row, more than the decode kernel's workspace.)"""
    assert L.axr_q8_attend_workspace_bytes(n_tok, max_q, B, Hq, Hkv, T, 128) < 2 * row_bytes(n_tok, Hq, 128)


@pytest.mark.parametrize("n_tok,max_q,B,Hq,Hkv,T,splits", [
    (256, 256, 1, 32, 8, 32768, 4), (512, 512, 1, 32, 8, 8192, 2), (80, 5, 16, 16, 2, 4096, 4)])
def test_few_row_tiles_split_to_one_wave(L, n_tok, max_q, B, Hq, Hkv, T, splits):
    """Calls with fewer row tiles than SMs: as many splits as fill one wave (the measured best)."""
    need = L.axr_q8_attend_workspace_bytes(n_tok, max_q, B, Hq, Hkv, T, 128)
    decode = 148 * 8 * 2 * 16 * 130 * 4  # two partials of 16 rows a warp, which the workspace holds in any case
    assert need == -(-max(splits * row_bytes(n_tok, Hq, 128), decode) // 256) * 256

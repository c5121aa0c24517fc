"""The Python side of rotary positions, dense decode and eviction without a GPU:
how arguments become C values and which are refused."""
import ctypes
import types

import pytest
import torch

import sparse_attention_decode_03_b200 as qsa
from sparse_attention_decode_03_b200 import qsa as Q

STRUCT = Q.qsa_cache_t(0x1000, 0x1000, 0x1000, 0x1000, 10, 2, 4, 2, 0)
CACHE = types.SimpleNamespace(struct=lambda: STRUCT)


def evict_call(n=2, ld=64, budget=16, sink=2, recent=4, ws=4096):
    p = ctypes.c_void_p(0x1000)
    return Q.LaunchCall("qsa_evict", (ctypes.byref(STRUCT), None, p, p, n, p, p, ld, budget, sink, recent, p, p, p, p, ws,
                                      None), (), torch.device("cuda", 0))


def test_integers_that_their_argument_cannot_hold_are_refused():
    """2^32 tokens of sink are not 0 of them."""
    values = [x.value for x in evict_call().args[1:]]
    assert values == [None, 0x1000, 0x1000, 2, 0x1000, 0x1000, 64, 16, 2, 4] + [0x1000] * 4 + [4096, None]
    for k in ("n", "budget", "sink", "recent"):
        for big in (1 << 31, 1 << 32, (1 << 32) + 16, -(1 << 31) - 1, 1 << 64):
            with pytest.raises(ValueError):
                evict_call(**{k: big})
    assert evict_call(ld=1 << 40, ws=1 << 40).args[7].value == 1 << 40
    with pytest.raises(ValueError):
        evict_call(ld=1 << 63)


def test_workspace_sizes_of_counts_beyond_32_bits_are_refused():
    assert qsa.dense_decode_workspace_bytes(CACHE, 1, 16) > 0 and qsa.evict_workspace_bytes(CACHE, 2, 16) > 0
    for call in (lambda x: qsa.dense_decode_workspace_bytes(CACHE, x, 16), lambda x: qsa.evict_workspace_bytes(CACHE, x, 16),
                 lambda x: qsa.dense_decode_workspace_bytes(CACHE, 1, x), lambda x: qsa.evict_workspace_bytes(CACHE, 2, x)):
        for big in ((1 << 32) + 16, -(1 << 32) + 16):
            with pytest.raises(ValueError):
                call(big)
        with pytest.raises(qsa.QSAError):
            call(-1)


def group(**elsewhere):
    """A cache group of CPU tensors, those named on another device."""
    t = dict(kv_pages=torch.empty(1), kc_pages=torch.empty(1), block_table=torch.empty(1))
    t.update({k: torch.empty(1, device="meta") for k in elsewhere})
    return types.SimpleNamespace(struct=lambda: STRUCT, max_pages_per_seq=4, max_seqs=2, **t)


@pytest.mark.parametrize("name", ["kv_pages", "kc_pages", "block_table"])
def test_buffers_of_the_group_on_another_device_are_refused(monkeypatch, name):
    monkeypatch.setattr(Q, "_req", lambda t, *a: t)
    i32, mass, byte = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 64), torch.empty(1 << 24, dtype=torch.uint8)
    cache = group(**{name: True})
    with pytest.raises(ValueError, match=name):
        qsa.bind_evict(cache, i32, i32, mass, mass, 16, 2, 4, i32, i32, i32, byte)
    if name != "kc_pages":      # which dense decode does not read
        q = torch.zeros(2, 4, 256)
        with pytest.raises(ValueError, match=name):
            qsa.bind_dense_decode(cache, q, i32, i32, 1 / 16, q, q, byte)


@pytest.mark.parametrize("nq,hq,hkv", [(1, 16, 1), (1, 128, 8), (9800, 16, 1), (20000, 128, 8), (300000, 4, 4)])
def test_workspace_stays_within_the_stated_bound(nq, hq, hkv):
    """8.5 MB and 8 bytes a (query, KV head) pair; with totals 80 bytes a query, head and page of the table more."""
    st = Q.qsa_cache_t(0x1000, 0x1000, 0x1000, 0x1000, 10, 2, 4, hkv, 0)
    cache = types.SimpleNamespace(struct=lambda: st)
    need, totals = (qsa.dense_decode_workspace_bytes(cache, nq, hq, m) for m in (False, True))
    assert need <= 8_500_000 + 8 * nq * hkv and totals - need <= 80 * nq * hq * 4 + 512

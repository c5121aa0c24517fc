"""Rotary positions, dense decode and eviction without a GPU: what the calls
refuse, the plan objects, and the index arithmetic the kernels share out work
and order their writes by, restated and checked over many sizes."""
import ctypes
import random

import numpy as np
import pytest
import torch

import sparse_attention_decode_03_b200 as qsa
from sparse_attention_decode_03_b200 import qsa as Q
from tests import dense_ref as D

L = Q.LIB
FAKE = ctypes.c_void_p(0x1000)


def cache_struct(hkv=2, mpps=4, kv=0x1000, kc=0x1000, dtype=0):
    return Q.qsa_cache_t(kv, kc, 0x1000, 0x1000, 10, 2, mpps, hkv, dtype)


# ---------------------------------------------------------------- refusals


def test_dense_decode_refuses_bad_arguments_before_any_cuda_call():
    c = cache_struct()
    cp = ctypes.byref(c)
    need = L.qsa_dense_decode_workspace_bytes(cp, 1, 16, 0)
    need_m = L.qsa_dense_decode_workspace_bytes(cp, 1, 16, 1)
    assert 0 < need < need_m == need + 16 * 4 * 4 * 20

    def call(cache=cp, q=FAKE, nq=1, hq=16, seq=FAKE, pos=FAKE, scale=0.0625, out=FAKE, lse=FAKE, mi=None, mo=None,
             ld=0, ws=FAKE, wb=need):
        return L.qsa_dense_decode(cache, q, nq, hq, seq, pos, scale, out, lse, mi, mo, ld, 1.0, ws, wb, None, None)

    assert call(nq=0) == 0 and call(nq=0, q=None, ws=None, wb=0) == 0
    assert call(cache=None) == -1 and call(nq=-1) == -1 and call(hq=0) == -1
    assert call(hq=3) == -1                      # not a multiple of the KV heads
    assert call(hq=64) == -2                     # 32 Q heads per KV head
    for bad in (0.0, -1.0, float("nan")):
        assert call(scale=bad) == -1
    for k in ("q", "seq", "pos", "out", "lse", "ws"):
        assert call(**{k: None}) == -1, k
    assert call(q=ctypes.c_void_p(0x1008)) == -1 and call(out=ctypes.c_void_p(0x1004)) == -1
    assert call(ws=ctypes.c_void_p(0x1080)) == -1 and call(wb=need - 1) == -1
    assert call(mi=FAKE) == -1 and call(mo=FAKE) == -1                  # both or neither
    assert call(mi=FAKE, mo=FAKE, ld=63, wb=need_m) == -1               # rows shorter than the table's blocks
    assert call(mi=FAKE, mo=FAKE, ld=64, wb=need) == -1                 # the weights need more workspace
    kc_only = cache_struct(kv=None)
    assert call(cache=ctypes.byref(kc_only)) == -1
    odd = cache_struct(dtype=7)
    assert call(cache=ctypes.byref(odd)) == -2
    huge = cache_struct(mpps=0x7fffffff // 64 + 1)
    assert call(cache=ctypes.byref(huge)) == -2
    wide = cache_struct(mpps=0x7fffffff // 64)      # 134 million tiles a pair: 8 pairs are 2^30 places, 16 too many
    assert L.qsa_dense_decode_workspace_bytes(ctypes.byref(wide), 4, 16, 0) > 0
    assert L.qsa_dense_decode_workspace_bytes(ctypes.byref(wide), 8, 16, 0) == -2
    assert L.qsa_dense_decode_workspace_bytes(cp, 1, 3, 0) == -1
    assert L.qsa_dense_decode_workspace_bytes(None, 1, 16, 0) == -1


def test_evict_refuses_bad_arguments_before_any_cuda_call():
    c = cache_struct()
    cp = ctypes.byref(c)
    need = L.qsa_evict_workspace_bytes(cp, 2, 16)
    assert need > 0

    def call(cache=cp, dst=None, ids=FAKE, lens=FAKE, n=2, mi=FAKE, mo=FAKE, ld=64, budget=16, sink=2, recent=4,
             keep=FAKE, cnt=FAKE, nl=FAKE, ws=FAKE, wb=need):
        return L.qsa_evict(cache, dst, ids, lens, n, mi, mo, ld, budget, sink, recent, keep, cnt, nl, ws, wb, None,
                           None)

    assert call(n=0) == 0
    assert call(cache=None) == -1 and call(n=-1) == -1
    assert call(budget=0) == -1 and call(budget=(1 << 30) + 1) == -2
    assert call(sink=-1) == -1 and call(recent=-1) == -1
    assert call(sink=10, recent=7) == -1
    assert call(sink=0x7fffffff, recent=0x7fffffff) == -1
    for k in ("ids", "lens", "mi", "mo", "keep", "cnt", "nl", "ws"):
        assert call(**{k: None}) == -1, k
    assert call(ld=63) == -1 and call(wb=need - 1) == -1 and call(ws=ctypes.c_void_p(0x1040)) == -1
    empty = cache_struct(kv=None, kc=None)
    assert call(cache=ctypes.byref(empty)) == -1
    odd = cache_struct(dtype=7)
    assert call(cache=ctypes.byref(odd)) == -2
    assert L.qsa_evict_workspace_bytes(cp, 2, 0) == -1


def rope_tensor(in_=0x1000, out=0x100000, heads=2, dim=256, si=512, so=512):
    return Q.qsa_rope_tensor_t(in_, out, heads, dim, si, so)


def test_rope_refuses_bad_arguments_before_any_cuda_call():
    plan = qsa.RopePlan(64, (12, 10, 10)).struct()

    def call(p=plan, ts=None, nt=None, pos=FAKE, ps=4, n=4):
        ts = [rope_tensor()] if ts is None else ts
        arr = (Q.qsa_rope_tensor_t * max(1, len(ts)))(*ts)
        return L.qsa_rope(None if p is None else ctypes.byref(p), arr, len(ts) if nt is None else nt, pos, ps, n, None)

    def changed(**kw):
        p = Q.qsa_rope_plan_t.from_buffer_copy(plan)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    assert call(n=0) == 0
    assert call(p=None) == -1 and call(n=-1) == -1 and call(nt=0) == -1 and call(nt=5) == -1
    assert call(pos=None) == -1 and call(ps=3) == -1
    for r in (0, 8, 24, 272):
        assert call(p=changed(rot_dim=r)) == -1, r
    assert call(p=changed(num_axes=0)) == -1 and call(p=changed(num_axes=4)) == -1
    assert call(p=changed(num_axes=2)) == -1                            # a pair names axis 2
    p = changed()
    p.freq[31] = float("inf")
    assert call(p=p) == -1
    p.freq[31] = float("nan")
    assert call(p=p) == -1
    assert call(ts=[rope_tensor(in_=None)]) == -1 and call(ts=[rope_tensor(out=None)]) == -1
    assert call(ts=[rope_tensor(heads=0)]) == -1
    for d in (32, 72, 272):
        assert call(ts=[rope_tensor(dim=d)]) == -1, d                   # shorter than rot_dim, odd, too wide
    assert call(ts=[rope_tensor(si=504)]) == -1 and call(ts=[rope_tensor(so=516)]) == -1
    assert call(ts=[rope_tensor(in_=0x1008)]) == -1 and call(ts=[rope_tensor(out=0x100008)]) == -1
    # overlaps: shifted by a row, another tensor's input, two outputs in one place
    assert call(ts=[rope_tensor(out=0x1000 + 1024)]) == -1
    assert call(ts=[rope_tensor(), rope_tensor(in_=0x100000 + 2048, out=0x200000)]) == -1
    assert call(ts=[rope_tensor(), rope_tensor(in_=0x80000)]) == -1
    # columns of one buffer, 1024 elements a row: 256 of q, then 128 of k overlapping q's last ones
    assert call(ts=[rope_tensor(0x1000, 0x1000, 1, 256, 1024, 1024),
                    rope_tensor(0x1000 + 496, 0x1000 + 496, 1, 128, 1024, 1024)]) == -1


def test_bindings_refuse_host_tensors_and_bad_shapes():
    plan = qsa.RopePlan(64)
    pos = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        qsa.bind_rope(plan, pos, [torch.zeros(3, 2, 256, dtype=torch.bfloat16)])
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        qsa.bind_dense_decode(None, torch.zeros(2, 4, 256, dtype=torch.bfloat16), torch.zeros(2, **i32),
                              torch.zeros(2, **i32), 0.0625, None, None, None)
    with pytest.raises(TypeError):
        qsa.bind_dense_decode(None, torch.zeros(2, 4, 256), torch.zeros(2, **i32), torch.zeros(2, **i32), 0.0625,
                              None, None, None)
    with pytest.raises(ValueError):
        qsa.bind_evict(None, torch.zeros(2, **i32), torch.zeros(2, **i32), None, None, 16, 0, 0, None, None, None,
                       None)


def test_rope_plan():
    p = qsa.RopePlan(64, (12, 10, 10), cycled=True)
    assert p.axis[:6] == [0, 1, 2, 0, 1, 2] and p.axis[30:] == [0, 0] and [p.axis.count(a) for a in range(3)] == [
        12, 10, 10]
    p = qsa.RopePlan(64, (12, 10, 10))
    assert p.axis == [0] * 12 + [1] * 10 + [2] * 10
    assert p.freqs[0] == 1.0 and abs(p.freqs[16] - 1e-2) < 1e-12
    assert qsa.RopePlan(128).axis == [0] * 64
    for bad in (dict(rot_dim=40), dict(rot_dim=272), dict(rot_dim=64, sections=(30, 1)),
                dict(rot_dim=64, sections=(8, 8, 8, 8)), dict(rot_dim=64, sections=(33, -1)),
                dict(rot_dim=64, sections=(2, 20, 10), cycled=True), dict(rot_dim=64, freqs=[1.0] * 31),
                dict(rot_dim=64, freqs=[float("inf")] * 32)):
        with pytest.raises(ValueError):
            qsa.RopePlan(**bad)


# ---------------------------------------------------------------- index arithmetic, restated


PIECE_COST, MIN_PLACES = 8, 4


def shares(T, pairs, ctas):
    n = min(ctas, max(pairs, -(-T // MIN_PLACES)))
    base, rem = divmod(T, n)
    return n, [c * base + min(c, rem) for c in range(n + 1)], base, rem


def share_of(base, rem, x):
    cut = rem * (base + 1)
    return x // (base + 1) if x < cut else rem + (x - cut) // base


@pytest.mark.parametrize("seed", range(40))
def test_shares_cover_every_tile_once_and_partials_have_slots_of_their_own(seed):
    """Every tile is in one CTA's walk; a CTA leaves at most two unfinished pairs,
    the one it took over and the one it hands on, each in a slot of its own."""
    rng = random.Random(seed)
    hkv = rng.choice([1, 2, 4])
    lens = [rng.choice([0, 1, 16, 17, rng.randint(0, 50), rng.randint(0, 9000)]) for _ in range(rng.randint(1, 90))]
    pairs, T = [], 0                                   # (first place, tiles, places before them)
    for n in lens:
        for _ in range(hkv if n else 0):
            nt = -(-n // 16)
            pairs.append((T, nt, PIECE_COST if nt > 1 else 1))
            T += pairs[-1][2] + nt
    if T == 0:
        return
    ctas = rng.choice([1, 3, 148, 256])
    n, start, base, rem = shares(T, len(pairs), ctas)
    assert start[0] == 0 and start[n] == T and all(a < b for a, b in zip(start, start[1:]))
    for x in range(0, T, max(1, T // 500)):
        c = share_of(base, rem, x)
        assert start[c] <= x < start[c + 1]
    done, slots = {}, {}
    for c in range(n):                                 # the walk of CTA c
        x0, x1 = start[c], start[c + 1]
        k = next(i for i, (b, nt, cost) in enumerate(pairs) if b <= x0 < b + cost + nt)
        b, nt, cost = pairs[k]
        t0, t1 = max(0, x0 - b - cost), min(nt, x1 - b - cost)
        while t1 > 0:
            for t in range(t0, t1):
                assert (k, t) not in done
                done[k, t] = c
            if t0 == 0:                                # this CTA names the pair's CTAs
                last = c if t1 == nt else share_of(base, rem, b + cost + nt - 1)
                slots.setdefault(k, {})["span"] = (c, last)
            if not (t0 == 0 and t1 == nt):
                s = 2 * c + (1 if t0 == 0 else 0)
                assert all(s not in v.get("slots", {}) for v in slots.values())
                slots.setdefault(k, {}).setdefault("slots", {})[s] = c
            if b + cost + nt >= x1:
                break
            k += 1
            b, nt, cost = pairs[k]
            t0, t1 = 0, min(nt, x1 - b - cost)
    assert len(done) == sum(nt for _, nt, _ in pairs)
    for k, v in slots.items():                         # the join looks for each piece where it was put
        first, last = v["span"]
        if first != last:
            assert v["slots"] == {2 * c + (1 if c == first else 0): c for c in range(first, last + 1)}


@pytest.mark.parametrize("unit", [4, 8])
@pytest.mark.parametrize("seed", range(60))
def test_in_place_moves_never_overwrite_an_unread_block(seed, unit):
    """The eviction's ordering rule: units (of 4 or 8 destination blocks) are
    claimed in order, each reads its blocks, then waits only for the lower units that took
    blocks out of its place, then writes.  Any interleaving of the claimed units
    leaves every kept block in its place, and every wait is for a lower unit."""
    rng = random.Random(seed)
    nb = rng.randint(1, 400)
    ratio = rng.random()
    keep = [b for b in range(nb) if rng.random() < ratio] if rng.random() < 0.8 else list(range(nb))
    tail = rng.random() < 0.5
    slots = list(range(nb + 1)) + [-1] * 16
    moved = keep + ([nb] if tail else [])
    if not moved:
        return
    pages = -(-len(moved) // unit)
    rank = [sum(1 for b in keep if b < unit * p) for p in range(nb // unit + 3)]
    state, data, resident = {}, {}, rng.randint(1, 6)
    claimed, done_read, finished = 0, set(), set()
    while len(finished) < pages:
        running = [p for p in range(claimed) if p not in finished]
        moves = []
        if claimed < pages and len(running) < resident:
            moves.append(("claim", claimed))
        for p in running:
            if p not in done_read:
                moves.append(("read", p))
            else:
                k0, k1 = rank[p], rank[p + 1]
                waits = range(k0 // unit, min(p - 1, (k1 - 1) // unit) + 1) if k1 > k0 else []
                assert all(w < p for w in waits)
                if all(w in done_read for w in waits):
                    moves.append(("write", p))
        assert moves, "a wait that never ends"
        what, p = rng.choice(moves)
        span = range(unit * p, min(unit * p + unit, len(moved)))
        if what == "claim":
            claimed += 1
        elif what == "read":
            data[p] = [slots[moved[k]] for k in span]
            done_read.add(p)
        else:
            for k, x in zip(span, data[p]):
                slots[k] = x
            finished.add(p)
    assert slots[:len(moved)] == moved


UNIT = 8


@pytest.mark.parametrize("seed", range(40))
def test_in_place_tickets_reach_every_unit_that_receives_blocks(seed):
    """Tickets run head, entry, unit; one that finds nothing moves the counter on to
    the next unit that receives blocks, as far as it looks.  Every such unit is
    claimed once, lower units of a sequence first, whatever the warps' order."""
    rng = random.Random(seed)
    n, hkv, look = rng.choice([1, 2, 5, 127, 128, 129, 300]), rng.choice([1, 2, 3]), 128
    units = rng.randint(1, 40)
    totals = [rng.choice([0, 0, 0, 1, rng.randint(0, UNIT * units)]) for _ in range(n)]
    ticket, claimed, pending = 0, [], []
    while True:
        if pending and (len(pending) > rng.randint(0, 8) or ticket >= n * hkv * units):
            t = pending.pop(rng.randrange(len(pending)))       # some warp looks its ticket up
            g, i, unit = t % hkv, t // hkv % n, t // hkv // n
            if unit * UNIT < totals[i]:
                claimed.append((t, i, g, unit))
                continue
            skip = next((s for s in range(look) if totals[(i + 1 + s) % n] > (unit + (i + 1 + s) // n) * UNIT), look)
            over = skip == look and n <= look
            ticket = max(ticket, n * hkv * units if over else (unit * n + i + 1 + skip) * hkv)
        elif ticket < n * hkv * units:
            pending.append(ticket)
            ticket += 1
        else:
            break
    assert sorted(c[1:] for c in claimed) == [(i, g, u) for i in range(n) for g in range(hkv)
                                              for u in range(-(-totals[i] // UNIT))]
    by_ticket = sorted(claimed)
    for i in range(n):
        assert [c[3] for c in by_ticket if c[1] == i] == sorted(c[3] for c in claimed if c[1] == i)


# ---------------------------------------------------------------- the references themselves


def test_reference_dense_is_softmax_attention():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((4, 256)), g.standard_normal((9, 2, 256)), g.standard_normal((9, 2, 256))
    out, lse, w, *_ = D.dense(q, k, v, 1 / 16, False)
    for h in range(4):
        t = torch.softmax(torch.from_numpy(k[:, h // 2] @ q[h]) / 16, 0).numpy()
        assert np.allclose(out[h], t @ v[:, h // 2], atol=1e-12)
    assert abs(w.sum() - 4) < 1e-12
    out, lse, *_ = D.dense(q, k[:0], v[:0], 1 / 16, False)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_reference_keep_blocks():
    nan = float("nan")
    assert D.keep_blocks([5, 1, 1, 9, 1, 2], 24, 6, 0, 0) == [0, 1, 2, 3, 4, 5]
    assert D.keep_blocks([5, 1, 1, 9, 1, 2], 27, 4, 1, 1) == [0, 1, 3, 5]
    assert D.keep_blocks([0, -0.0, 0, nan, -1, 2], 24, 3, 0, 0) == [0, 1, 5]
    assert D.keep_blocks([0, nan, nan, nan], 16, 2, 0, 0) == [0, 1]

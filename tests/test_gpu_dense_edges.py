"""Dense decode, eviction and their classes at the edges of what the calls
accept: alignment, ranges of weights and queries, tables that mix a sequence's
own pages with others, several streams.  References and bounds: dense_ref.py,
and the ones stated beside each test."""
import random

import numpy as np
import pytest
import torch

from tests import dense_ref as D

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_decode_03_b200")

from tests.test_gpu_dense import (  # noqa: E402
    Group, bits, check_dense, i32, masses, queries, snapshot, within)


@pytest.fixture(autouse=True, scope="module")
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


# ---------------------------------------------------------------- alignment of the outputs


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(3, 1), (12, 1), (32, 2)])
def test_dense_decode_writes_outputs_that_are_8_byte_aligned(hq, hkv, fp8):
    """out and lse as slices of packed buffers: pairs of one tile, of several, and of several CTAs."""
    lens = [1, 3, 15, 16, 17, 40, 100, 9000, 2]
    grp = Group(lens, hkv, fp8, seed=hq)
    nq, n = len(lens), len(lens) * hq * 256
    q, q_seq, q_pos = queries(nq, hq, 1).cuda(), i32(list(range(nq))), i32([x - 1 for x in lens])
    ws = torch.empty(qsa.dense_decode_workspace_bytes(grp.cache, nq, hq), dtype=torch.uint8, device="cuda")
    got = []
    for shift in (0, 4):                              # elements: 0 and 8 bytes past a 256-byte boundary
        buf = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        stats = torch.full((nq * hq + 2,), 7.0, device="cuda")
        out, lse = buf[shift:shift + n].view(nq, hq, 256), stats[shift // 4:shift // 4 + nq * hq].view(nq, hq)
        assert out.data_ptr() % 16 == 2 * shift
        qsa.qsa_dense_decode(grp.cache, q, q_seq, q_pos, 1 / 16, out, lse, ws)
        torch.cuda.synchronize()
        got.append((bits(out), bits(lse)))
        assert (buf[:shift] == 7.0).all() and (buf[shift + n:] == 7.0).all()       # nothing beside the rows
        assert (stats[:shift // 4] == 7.0).all() and (stats[shift // 4 + nq * hq:] == 7.0).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---------------------------------------------------------------- one key far above the others


def rewrite(grp, s, k, v):
    """Give sequence s of a group other K and V rows."""
    grp.k[s], grp.v[s] = k.bfloat16(), v.bfloat16()
    grp.append(s, 0, grp.k[s], grp.v[s], grp.ki[s])


def check_rows(grp, q, lens):
    """A tracked step of every sequence against 64 bits.  Bounds: dense_ref's for logits and sums, and for each
    weight half an FP16 step of its own size (an e4m3 cache's; BF16 pairs are finer), however small it is."""
    nq, hq = q.shape[:2]
    dec = qsa.DenseDecoder(grp.cache, hq, nq, track=True)
    out, lse = dec.run(q.cuda(), i32(list(range(nq))), i32([n - 1 for n in lens]))
    torch.cuda.synchronize()
    assert int(dec.dev_status.item()) == 0
    group = hq // grp.hkv
    for s, n in enumerate(lens):
        k, v = (x[:n] for x in grp.rows(s))
        o, l, w, ob, lb, wb = D.dense(q[s].double().numpy(), k, v, 1 / 16, False)
        for h in range(hq):
            z = k[:, h // group] @ q[s, h].double().numpy() / 16
            ob[h] += D.FP16 * (np.exp(z - l[h]) @ np.abs(v[:, h // group]))
        within(out[s].double().cpu().numpy(), o, ob, f"sequence {s}: out")
        within(lse[s].double().cpu().numpy(), l, lb, f"sequence {s}: lse")
        nb = -(-n // 4)
        within(dec.mass[s, :nb].double().cpu().numpy(), D.block_sums(w), D.block_sums(wb) +
               2 * hq * D.FP32 * D.block_sums(w), "totals")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gap", [8, 12, 16, 18, 20, 30, 60])
def test_dense_decode_weights_far_below_one_key_with_no_value(gap, fp8):
    """A key `gap` nats above thousands of others, with V = 0: the output is made of the others' weights alone."""
    lens, hq, hkv = [5000, 33000, 700, 30], 12, 1
    grp = Group(lens, hkv, fp8, seed=gap)
    g = torch.Generator().manual_seed(gap)
    q = torch.empty((len(lens), hq, 256))
    for s, n in enumerate(lens):
        lead = torch.randn(256, generator=g)
        q[s] = lead + 0.2 * torch.randn((hq, 256), generator=g)
        k, v = torch.randn((n, hkv, 256), generator=g), 1.0 + 0.4 * torch.randn((n, hkv, 256), generator=g)
        at = [0, n // 2, n - 1, 5][s]                   # the first, a middle, the last key
        k[at, 0], v[at] = lead * (16 * gap / (lead * lead).sum()), 0.0
        rewrite(grp, s, k, v)
    check_rows(grp, q.bfloat16(), lens)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spread", [2.0, 6.0, 20.0])
def test_dense_decode_weights_of_many_sizes(spread, fp8):
    """Logits spread over tens of nats, so that tiles with and without tiny weights follow one another."""
    lens = [3000, 9001, 64, 17]
    grp = Group(lens, 2, fp8, seed=int(spread))
    for s, n in enumerate(lens):
        rewrite(grp, s, grp.k[s].float(), grp.v[s].float().abs())
    check_rows(grp, queries(len(lens), 16, 5, spread), lens)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gap", [0, 40])
def test_dense_decode_keeps_a_nan_in_its_dims(gap, fp8):
    """A NaN among the values reaches the outputs of its dims and no others, whatever form the weights take."""
    lens, hq = [400, 5, 16], 6
    grp = Group(lens, 1, fp8, seed=1)
    q = queries(len(lens), hq, 2)
    bad = torch.zeros(256, dtype=torch.bool)
    bad[[0, 7, 100, 255]] = True
    for s, n in enumerate(lens):
        k, v = grp.k[s].float(), grp.v[s].float()
        k[0, 0] += q[s].float().mean(0) * gap
        v[n - 1, 0, bad] = float("nan")
        rewrite(grp, s, k, v)
    dec = qsa.DenseDecoder(grp.cache, hq, len(lens))
    out, lse = dec.run(q.cuda(), i32([0, 1, 2]), i32([n - 1 for n in lens]))
    torch.cuda.synchronize()
    assert torch.equal(out.isnan().cpu(), bad.expand(len(lens), hq, 256)) and bool(lse.isfinite().all())


# ---------------------------------------------------------------- queries at the ends of BF16's range


@pytest.mark.parametrize("fp8,gain", [(True, 2.0 ** 118), (True, 2.0 ** 122), (True, 2.0 ** -100), (True, 2.0 ** -120),
                                      (False, 2.0 ** 118)])
def test_dense_decode_queries_at_the_ends_of_their_range(fp8, gain):
    """Rows of |q| near 2^120 or 2^-120 under a scale that leaves ordinary logits; small elements in one row too."""
    grp = Group([333, 40, 7], 1, fp8, seed=4)
    q = queries(3, 6, 8, gain)
    q[0, :, 128:] *= 2.0 ** -20
    check_dense(grp, q, [0, 1, 2], [332, 39, 6], scale=1 / (16 * gain))


# ---------------------------------------------------------------- eviction into tables that mix own pages with others


OWN = {"copy": lambda P, n: True, "fresh then own": lambda P, n: P >= n // 2, "own then fresh": lambda P, n: P < n // 2,
       "alternating": lambda P, n: P % 2 == 0, "one own": lambda P, n: P == n // 3, "every third fresh": lambda P, n: P % 3 != 1}


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("fp8,hkv", [(False, 1), (False, 3), (True, 2)])
@pytest.mark.parametrize("mix", list(OWN))
def test_evict_into_tables_that_mix_own_pages_with_others(mix, fp8, hkv, alias):
    """Rows of dst_table that name the sequence's own page at some places and spare pages at others: every moved
    block, the pages that nothing may write, keep, lengths and totals.  Few units (4 blocks each) and many (8)."""
    for lens, budget, sink, recent in (([2100, 67, 1300, 900], 150, 3, 20), ([9001, 12000, 4097, 30, 8000], 900, 0, 100),
                                       ([7000 + 300 * i for i in range(12)], 1100, 16, 64)):
        rng = random.Random(len(lens))
        grp = Group(lens, hkv, fp8, seed=budget, spare=sum(-(-n // 64) for n in lens))
        c, table = grp.cache, grp.cache.block_table.cpu()
        mass = masses(rng, (len(lens), c.max_pages_per_seq * 16))
        before = snapshot(c, c.block_table, lens)
        dst, at, fresh = table.clone(), 0, set()
        for s, n in enumerate(lens):
            pages = -(-n // 64)
            for P in range(pages):
                if not OWN[mix](P, pages):
                    dst[s, P] = grp.free[at]
                    fresh.add((s, P))
                    at += 1
        spare = grp.free[at:].long().cuda()                     # named by no table
        c.kv_pages.view(torch.uint8)[spare] = 0x5a
        mass_in = mass.cuda()
        mass_out = mass_in if alias else torch.full_like(mass_in, -9.0)
        n = len(lens)
        keep, seq_len = torch.empty((n, budget), dtype=torch.int32, device="cuda"), i32(lens)
        cnt, new_len = torch.empty_like(seq_len), seq_len if alias else torch.empty_like(seq_len)
        ws = torch.full((qsa.evict_workspace_bytes(c, n, budget),), 0xff, dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        qsa.qsa_evict(c, i32(list(range(n))), seq_len, mass_in, mass_out, budget, sink, recent, keep, cnt, new_len, ws,
                      dst_table=dst.cuda(), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert (c.kv_pages.view(torch.uint8)[spare] == 0x5a).all()
        moved = []
        for s, x in enumerate(lens):
            kept = D.keep_blocks(mass[s].tolist(), x, budget, sink, recent)
            assert keep[s].tolist() == kept + [-1] * (budget - len(kept))
            assert int(cnt[s]) == len(kept) and int(new_len[s]) == 4 * len(kept) + x % 4
            moved.append(kept + ([x // 4] if x % 4 else []))
        after = snapshot(c, dst.cuda(), [4 * len(m) for m in moved])
        old = snapshot(c, c.block_table, lens)
        for s, m in enumerate(moved):
            for was, now, left in zip(before[s], after[s], old[s]):
                assert torch.equal(was[m], now), f"sequence {s}: rows differ"
                for b in range(was.shape[0]):                   # places that no block went to keep what they held
                    if (s, b // 16) in fresh or b >= len(m):
                        assert torch.equal(was[b], left[b]), f"sequence {s}: block {b} changed"
            got = mass_out[s].cpu()
            want = torch.zeros(-(-lens[s] // 4))
            want[:len(m)] = mass[s, m]
            assert torch.equal(got[:len(want)].view(torch.int32), want.view(torch.int32))


# ---------------------------------------------------------------- streams of one decoder


def test_dense_decoder_calls_on_several_streams_follow_one_another():
    """Inputs made late on the current stream, a step on one side stream, an eviction on another and a step on the
    current one: as if all were on one stream."""
    lens, hq = [900, 640], 8
    results = []
    for apart in (False, True):
        grp = Group(lens, 1, seed=2)
        dec = qsa.DenseDecoder(grp.cache, hq, 2, track=True)
        q1, q2 = queries(2, hq, 1).cuda(), queries(2, hq, 2).cuda()
        q, seqs, pos = torch.zeros_like(q1), i32([0, 1]), i32([n - 1 for n in lens])
        a, b = (torch.cuda.Stream(), torch.cuda.Stream()) if apart else (None, None)
        torch.cuda.synchronize()
        if apart:
            torch.cuda._sleep(40_000_000)          # about 20 ms: what follows is enqueued long before it runs
        q.copy_(q1)
        dec.run(q, seqs, pos, stream=a)
        new_len, keep, count = dec.evict(seqs, pos + 1, 100, 2, 10, stream=b)
        if apart:
            torch.cuda.current_stream().wait_stream(b)
        out, lse = dec.run(q2, seqs, new_len - 1)
        torch.cuda.synchronize()
        assert int(dec.dev_status.item()) == 0
        results.append([x.clone() for x in (out, lse, dec.mass, new_len, keep, count)])
    for x, y in zip(*results):
        assert torch.equal(bits(x), bits(y))


def test_dense_decoder_runs_inside_a_capture():
    """run and evict captured on a side stream, after calls on another one."""
    lens, hq = [700, 333], 4
    grp = Group(lens, 1, seed=3)
    dec = qsa.DenseDecoder(grp.cache, hq, 2, track=True)
    q, seqs, pos = queries(2, hq, 1).cuda(), i32([0, 1]), i32([n - 1 for n in lens])
    out, lse = (x.clone() for x in dec.run(q, seqs, pos))
    mass = dec.mass.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dec.mass.zero_()
        dec.run(q, seqs, pos)
        totals = dec.mass.clone()
        _, keep, count = dec.evict(seqs, pos + 1, 1000)       # nothing to cut
    dec.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(dec.out), bits(out)) and torch.equal(bits(dec.lse), bits(lse))
    assert torch.equal(bits(totals), bits(mass)) and count.tolist() == [n // 4 for n in lens]


def test_dense_decoder_branches_off_a_capture():
    """A step on a stream of its own inside a capture, after calls outside it: a branch that the caller joins."""
    lens, hq = [700, 333], 4
    grp = Group(lens, 1, seed=3)
    dec = qsa.DenseDecoder(grp.cache, hq, 2)
    q, seqs, pos = queries(2, hq, 1).cuda(), i32([0, 1]), i32([n - 1 for n in lens])
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    out, lse = (x.clone() for x in dec.run(q, seqs, pos))
    dec.run(q, seqs, pos, stream=other)
    torch.cuda.synchronize()
    graph, twice = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        twice.copy_(q)
        dec.run(twice, seqs, pos, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copy = dec.out.clone()
    dec.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(copy), bits(out)) and torch.equal(bits(dec.lse), bits(lse))
    dec.run(q, seqs, pos)
    torch.cuda.synchronize()
    assert torch.equal(bits(dec.out), bits(out))


def test_dense_decoder_keeps_a_side_streams_inputs():
    """Inputs that the caller lets go of right after a call on a side stream are not handed out again before it ran."""
    lens, hq = [900, 640], 8
    results = []
    for apart in (False, True):
        grp = Group(lens, 1, seed=2)
        dec = qsa.DenseDecoder(grp.cache, hq, 2, track=True)
        q, side = queries(2, hq, 1).cuda(), torch.cuda.Stream() if apart else None
        pos, n = i32([n - 1 for n in lens]), i32(lens)
        torch.cuda.synchronize()
        if apart:
            with torch.cuda.stream(side):
                torch.cuda._sleep(40_000_000)
        out, lse = dec.run(q.clone(), i32([0, 1]), pos.clone(), stream=side)
        # what takes the memory that came free: padding ids, which read nothing
        taken = [torch.full((2,), -1, dtype=torch.int32, device="cuda") for _ in range(8)] + [torch.zeros_like(q) for _ in range(4)]
        new_len, keep, count = dec.evict(i32([0, 1]), n.clone(), 100, 2, 10, stream=side)
        taken += [torch.full((2,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert int(dec.dev_status.item()) == 0
        results.append([x.clone() for x in (out, lse, dec.mass, new_len, keep, count)])
    for x, y in zip(*results):
        assert torch.equal(bits(x), bits(y))


# ---------------------------------------------------------------- queries that are not numbers; calls at once


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_dense_decode_keeps_a_bad_query_to_its_head(value, fp8):
    """A NaN or an infinity in one head's query makes that head's row NaN (infinite logits of both signs) and no other."""
    lens, hq, bad = [16, 700, 5000], 12, 5
    grp = Group(lens, 1, fp8, seed=8)
    q = queries(3, hq, 4)
    q[:, bad, 17] = value
    dec = qsa.DenseDecoder(grp.cache, hq, 3)
    out, lse = dec.run(q.cuda(), i32([0, 1, 2]), i32([n - 1 for n in lens]))
    torch.cuda.synchronize()
    good = [h for h in range(hq) if h != bad]
    assert bool(out[:, bad].isnan().all()) and bool(lse[:, bad].isnan().all())
    for s, n in enumerate(lens):
        k, v = grp.rows(s)
        o, l, _, ob, lb, _ = D.dense(q[s, good].double().numpy(), k, v, 1 / 16, fp8)
        within(out[s, good].double().cpu().numpy(), o, ob, f"sequence {s}: out")
        within(lse[s, good].double().cpu().numpy(), l, lb, f"sequence {s}: lse")


@pytest.mark.parametrize("fp8", [False, True])
def test_evictions_and_steps_at_once(fp8):
    """Two evictions in place of different sequences and a step of a third, on three streams with workspaces of their
    own, again and again: the same bytes as one after the other."""
    lens, budget, hq = [9000, 7001, 8003, 5000, 6002], 700, 6
    results = []
    for apart in (False, True):
        grp = Group(lens, 1, fp8, seed=6)
        c = grp.cache
        mass = masses(random.Random(1), (len(lens), c.max_pages_per_seq * 16)).cuda()
        q, decs = queries(1, hq, 3).cuda(), qsa.DenseDecoder(c, hq, 1)
        args = []
        for ids in ([0, 1], [2, 3]):
            n, ws = len(ids), torch.empty(qsa.evict_workspace_bytes(c, 2, budget), dtype=torch.uint8, device="cuda")
            args.append((i32(ids), i32([lens[s] for s in ids]), mass, mass, budget, 3, 40,
                         torch.empty((n, budget), dtype=torch.int32, device="cuda"), *(torch.empty_like(i32(ids)) for _ in range(2)),
                         ws))
        step_args = (q, i32([4]), i32([lens[4] - 1]))
        torch.cuda.synchronize()
        s = [torch.cuda.Stream() for _ in range(3)] if apart else [None] * 3
        out, lse = decs.run(*step_args, stream=s[2])
        for call, st in zip(args, s):
            qsa.qsa_evict(c, *call, stream=st)
        for _ in range(20):
            decs.run(*step_args, stream=s[2])
        torch.cuda.synchronize()
        results.append([bits(x) for x in (c.kv_pages.view(torch.uint8), c.kc_pages, mass, out, lse, args[0][7], args[1][7])])
    for x, y in zip(*results):
        assert torch.equal(x, y)

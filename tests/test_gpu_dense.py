"""Rotary positions, dense paged decode and eviction on the GPU against 64-bit
references (tests/dense_ref.py gives the references and derives the bounds)."""
import math
import random

import numpy as np
import pytest
import torch

from tests import dense_ref as D

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_decode_03_b200")


@pytest.fixture(autouse=True, scope="module")
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), f"{what}: -inf pattern differs"
    fin = ~np.isneginf(want)
    err = np.abs(got[fin] - want[fin])
    lim = np.broadcast_to(bound, want.shape)[fin]
    bad = ~(err <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bounds, worst {np.max(err / lim):.3g} times"


# ---------------------------------------------------------------- rotary positions


@pytest.mark.parametrize("n", [1, 2, 3, 57, 300])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("sections,cycled", [((32,), False), ((12, 10, 10), True), ((8, 4, 12), False), ((0, 64), False),
                                             ((24, 20, 20), True)])
def test_rope_against_64_bits(n, adjacent, sections, cycled):
    g = gen(n)
    rot = 2 * sum(sections)
    plan = qsa.RopePlan(rot, sections, base=1e6, cycled=cycled, adjacent=adjacent)
    pos = torch.randint(-5, 262144, (len(sections), n), generator=g, dtype=torch.int32)
    xs = [torch.randn((n, h, d), generator=g).bfloat16() for h, d in ((6, 256), (1, 256), (8, 128), (3, 128))]
    outs = [torch.full_like(x, 7.0).cuda() for x in xs]
    dev = [x.cuda() for x in xs]
    qsa.qsa_rope(plan, pos.cuda(), dev, outs)
    for x, y, d in zip(xs, outs, dev):
        want, bound = D.rope(x.double().numpy(), pos.numpy(), plan.axis, plan.freqs, adjacent)
        within(y.double().cpu().numpy(), want, bound, f"heads {x.shape[1]} dim {x.shape[2]}")
        assert torch.equal(bits(y[..., rot:]), bits(x[..., rot:]))      # copied as they are
        assert torch.equal(bits(d), bits(x))                           # inputs unchanged
    qsa.qsa_rope(plan, pos.cuda(), dev)                                # in place: the same bits
    for y, d in zip(outs, dev):
        assert torch.equal(bits(y), bits(d))


def test_rope_slices_of_a_fused_projection_in_place_and_odd_widths():
    g = gen(5)
    n, plan = 37, qsa.RopePlan(64, (12, 10, 10))
    buf = torch.randn((n, 6 * 256 + 2 * 256 + 2 * 256 + 144), generator=g).bfloat16().cuda()
    old = buf.clone()
    pos = torch.randint(0, 100000, (3, n), generator=g, dtype=torch.int32).cuda()
    q, k, odd = buf[:, :1536].unflatten(1, (6, 256)), buf[:, 1536:2048].unflatten(1, (2, 256)), \
        buf[:, 2560:].unflatten(1, (1, 144))
    qsa.qsa_rope(plan, pos, [q, k, odd])
    for a, b, h, d in ((0, 1536, 6, 256), (1536, 2048, 2, 256), (2560, 2704, 1, 144)):
        x = old[:, a:b].unflatten(1, (h, d)).double().cpu().numpy()
        want, bound = D.rope(x, pos.cpu().numpy(), plan.axis, plan.freqs, False)
        within(buf[:, a:b].unflatten(1, (h, d)).double().cpu().numpy(), want, bound, f"columns {a}..{b}")
    assert torch.equal(bits(buf[:, 2048:2560]), bits(old[:, 2048:2560]))   # V, between them, untouched


def test_rope_keeps_far_positions_and_turns_relative():
    """q . k after rotation depends on the distance alone, also 2^30 tokens out."""
    g = gen(6)
    plan = qsa.RopePlan(64)
    q, k = (torch.randn((1, 1, 256), generator=g).bfloat16() for _ in range(2))
    dots = []
    for base in (0, 262144, 1 << 30):
        qr, kr = q.cuda(), k.cuda()
        qsa.qsa_rope(plan, i32([[base + 7]]), [qr])
        qsa.qsa_rope(plan, i32([[base]]), [kr])
        dots.append((qr.double() * kr.double()).sum().item())
    mag = (q.abs().double() * k.abs().double())[..., 64:].sum().item() + \
        2 * (q[..., :64].abs().double().sum() * k[..., :64].abs().double().max()).item()
    for d in dots[1:]:
        assert abs(d - dots[0]) <= 4 * D.BF16 * mag


def test_rope_in_a_graph_and_on_another_stream():
    g = gen(7)
    n, plan = 5, qsa.RopePlan(64)
    pos = i32([[3, 1, 4, 1, 5]])
    x, y = torch.randn((n, 4, 256), generator=g).bfloat16().cuda(), torch.empty((n, 4, 256), dtype=torch.bfloat16,
                                                                               device="cuda")
    call = qsa.bind_rope(plan, pos, [x], [y])
    call()
    want = y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = qsa.StepGraph([call], s)
    y.zero_()
    s.wait_stream(torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want))
    y.zero_()
    s.wait_stream(torch.cuda.current_stream())
    qsa.qsa_rope(plan, pos, [x], [y], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want))
    e = torch.empty((0, 4, 256), dtype=torch.bfloat16, device="cuda")
    qsa.qsa_rope(plan, torch.empty((1, 0), dtype=torch.int32, device="cuda"), [e])   # no tokens


# ---------------------------------------------------------------- a cache with known rows


class Group:
    """A cache group, its logical rows on the host, and spare pages."""

    def __init__(self, lens, hkv, fp8=False, seed=0, spare=0, with_kc=True, with_kv=True, mpps=None, lean=0.0,
                 num_pages=None, first_page=0):
        g = gen(seed)
        self.lens, self.hkv, self.fp8 = list(lens), hkv, fp8
        pages = [-(-n // 64) for n in lens]
        width = mpps or max(1, max(pages, default=1))
        total = sum(pages) + spare
        phys = first_page + torch.randperm(total, generator=g).int()
        bt = torch.full((max(1, len(lens)), width), -1, dtype=torch.int32)
        at = 0
        for s, c in enumerate(pages):
            bt[s, :c] = phys[at:at + c]
            at += c
        self.free = phys[at:]
        self.cache = qsa.PagedCache(num_pages or max(1, total), max(1, len(lens)), width, hkv, bt,
                                    kv_dtype=qsa.KV_FP8_E4M3 if fp8 else qsa.KV_BF16, with_kv=with_kv, with_kc=with_kc)
        if with_kv and num_pages is None:   # unwritten rows hold NaN
            self.cache.kv_pages.view(torch.uint8).fill_(0x7f if fp8 else 0xff)
        if with_kc:
            self.cache.kc_pages.fill_(3.0)
        self.k, self.v, self.ki = [], [], []
        for s, n in enumerate(lens):
            self.k.append(torch.randn((n, hkv, 256), generator=g).bfloat16())
            self.v.append(torch.randn((n, hkv, 256), generator=g).bfloat16())
            self.ki.append(torch.randint(-8, 9, (n, 128), generator=g).bfloat16())
            if lean:
                u = torch.randn((hkv, 256), generator=gen(900 + s))
                pick = torch.rand((n, 1, 1), generator=g) < 0.1
                self.k[s] += (lean * pick * u / u.norm(dim=1, keepdim=True)).bfloat16()
            if n:
                self.append(s, 0, self.k[s], self.v[s], self.ki[s])

    def append(self, s, start, k, v, ki):
        n = k.shape[0]
        qsa.qsa_append_kv(self.cache, k.cuda().contiguous(), v.cuda().contiguous(), ki.cuda().contiguous(),
                          torch.full((n,), s, dtype=torch.int32, device="cuda"),
                          torch.arange(start, start + n, dtype=torch.int32, device="cuda"))

    def stored(self, x):
        x = x.float()
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy() if self.fp8 else x.double().numpy()

    def rows(self, s):
        return self.stored(self.k[s]), self.stored(self.v[s])


def queries(nq, hq, seed, scale=1.0):
    return (scale * torch.randn((nq, hq, 256), generator=gen(seed))).bfloat16()


def check_dense(grp, q, q_seq, q_pos, scale=1 / 16, track=False, decay=1.0, mass0=None, status=0, lost=()):
    """Run qsa_dense_decode and compare out, lse (and the totals) with 64 bits."""
    nq, hq = q.shape[:2]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = grp.cache
    out = torch.full((nq, hq, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq, hq), float("nan"), device="cuda")
    ws = torch.full((qsa.dense_decode_workspace_bytes(c, nq, hq, track),), 0xff, dtype=torch.uint8, device="cuda")
    mass_in = mass_out = None
    if track:
        mass_in = mass0.cuda()
        mass_out = torch.full_like(mass_in, -5.0)
    qsa.qsa_dense_decode(c, q.cuda(), i32(q_seq), i32(q_pos), scale, out, lse, ws, mass_in, mass_out, decay, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status, qsa.dev_status_names(int(st.item()))
    mass, mass_b, seen = {}, {}, {}
    for r in range(nq):
        s, p = q_seq[r], q_pos[r]
        n = p + 1 if 0 <= s < c.max_seqs and 0 <= p < c.capacity_tokens else 0
        k, v = grp.rows(s) if n else (np.zeros((0, grp.hkv, 256)),) * 2
        idx = np.array([t for t in range(n) if (s, t // 64) not in lost], dtype=np.int64)
        o, l, w, ob, lb, wb = D.dense(q[r].double().numpy(), k[idx], v[idx], scale, grp.fp8)
        within(out[r].double().cpu().numpy(), o, ob, f"query {r}: out")
        within(lse[r].double().cpu().numpy(), l, lb, f"query {r}: lse")
        if track and n:
            full, fullb = np.zeros(n), np.zeros(n)
            full[idx], fullb[idx] = w, wb
            nb = -(-n // 4)
            if s not in mass or len(mass[s]) < nb:
                pad = nb - len(mass.get(s, []))
                mass[s] = np.pad(mass.get(s, np.zeros(0)), (0, pad))
                mass_b[s] = np.pad(mass_b.get(s, np.zeros(0)), (0, pad))
            mass[s][:nb] += D.block_sums(full)
            mass_b[s][:nb] += D.block_sums(fullb)
    if track:
        got = mass_out.double().cpu().numpy()
        for s in range(c.max_seqs):
            m = mass.get(s, np.zeros(0))
            want = float(np.float32(decay)) * mass0[s, :len(m)].double().numpy() + m
            lim = mass_b.get(s, np.zeros(0)) + 2 * hq * D.FP32 * np.abs(want) + 1e-30
            within(got[s, :len(m)], want, lim, f"sequence {s}: totals")
            assert (got[s, len(m):] == -5.0).all()          # left as they were
    return out, lse


def check_bits(grp, q, q_seq, q_pos):
    nq, hq = q.shape[:2]
    dec = qsa.DenseDecoder(grp.cache, hq, nq)
    o, l = dec.run(q.cuda(), i32(q_seq), i32(q_pos))
    torch.cuda.synchronize()
    assert int(dec.dev_status.item()) == 0
    return o, l


HEADS = [(16, 2), (24, 2), (12, 1), (6, 1), (3, 1), (4, 4), (16, 1), (9, 3)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_dense_decode_ragged_lengths(hq, hkv, fp8):
    lens = [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 127, 129, 200, 700, 1030]
    grp = Group(lens, hkv, fp8, seed=hq + hkv, lean=3.0)
    q_seq = list(range(len(lens))) + [-1, 3, 15, 14]          # padding, no tokens, a second query, a shorter prefix
    q_pos = [n - 1 for n in lens] + [5, -1, 1029, 333]
    q = queries(len(q_seq), hq, 3)
    mass0 = torch.rand((len(lens), grp.cache.max_pages_per_seq * 16), generator=gen(9))
    check_dense(grp, q, q_seq, q_pos, track=True, decay=0.75, mass0=mass0)
    a = check_dense(grp, q, q_seq, q_pos)
    b = check_dense(grp, q, q_seq, q_pos)
    for x, y in zip(a, b):
        assert torch.equal(bits(x), bits(y))                  # same call, same bits


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 16, 128, 129, 4096, 9001])
def test_dense_decode_one_sequence(n, fp8):
    grp = Group([n], 2, fp8, seed=n, lean=4.0)
    mass0 = torch.rand((1, grp.cache.max_pages_per_seq * 16), generator=gen(n))
    check_dense(grp, queries(1, 24, n, 2.0), [0], [n - 1], track=True, mass0=mass0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[60000, 1, 50011, 40], [131072 + 7] + [100] * 90])
def test_dense_decode_long_shares(lens, fp8):
    """Hundreds of tiles per CTA: the ring is reused many times, a share holds several pairs."""
    grp = Group(lens, 2, fp8, seed=len(lens), lean=4.0)
    q_seq = list(range(len(lens)))
    a = check_dense(grp, queries(len(lens), 6, 1), q_seq, [n - 1 for n in lens])
    for _ in range(20):                                       # the same bits, whatever order the copies land in
        b = check_bits(grp, queries(len(lens), 6, 1), q_seq, [n - 1 for n in lens])
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hq,hkv", [([30000], 16, 1), ([9000] + [100] * 7, 16, 1), ([20000] + [40] * 30, 24, 2),
                                         ([20000] + [40] * 150, 32, 2), ([2000 + 7 * i for i in range(60)], 12, 1)])
def test_dense_decode_joins_few_and_many_pieces(lens, hq, hkv, fp8):
    """Pairs of 1 to 148 pieces, heads joined whole or by slices, one or several a block."""
    grp = Group(lens, hkv, fp8, seed=hq)
    mass0 = torch.rand((len(lens), grp.cache.max_pages_per_seq * 16), generator=gen(hq))
    check_dense(grp, queries(len(lens), hq, 3, 2.0), list(range(len(lens))), [n - 1 for n in lens], track=True,
                mass0=mass0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [30000, 1500])
def test_dense_decode_pieces_without_a_token(n, fp8):
    """Runs of missed pages that empty whole CTAs' pieces, the first and the last too."""
    grp = Group([n, 64 * 7], 1, fp8, seed=5)
    pages = -(-n // 64)
    missed = [P for P in range(pages) if P < pages // 5 or pages // 2 <= P < pages // 2 + pages // 6 or P > pages - pages // 8]
    grp.cache.block_table[0, missed] = -1
    mass0 = torch.rand((2, grp.cache.max_pages_per_seq * 16), generator=gen(n))
    check_dense(grp, queries(2, 12, 4, 2.0), [0, 1], [n - 1, 64 * 7 - 1], track=True, mass0=mass0, status=1,
                lost={(0, P) for P in missed})


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gain", [2.0 ** -30, 2.0 ** -14, 30.0, 2.0 ** 18])
def test_dense_decode_small_and_large_queries(gain, fp8):
    """Logits from all but equal to one token taking everything; FP8 operands beyond FP16's range."""
    grp = Group([333, 40], 1, fp8, seed=4)
    q = queries(2, 6, 8, gain)
    # where logits are large, only their own rounding matters: the bounds grow with |z|
    check_dense(grp, q, [0, 1], [332, 39], scale=1 / 16 if gain < 100 else 2.0 ** -20)


def test_dense_decode_many_queries_and_all_empty():
    grp = Group([5 * (i % 41) + 1 for i in range(75)], 1, seed=2)
    check_dense(grp, queries(75, 3, 1), list(range(75)), [n - 1 for n in grp.lens])
    check_dense(grp, queries(75, 3, 1), list(range(75)), [-1] * 75)
    check_dense(grp, queries(40, 3, 1), [-1] * 40, [7] * 40, track=True,
                mass0=torch.zeros((75, grp.cache.max_pages_per_seq * 16)))


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_decode_bad_data_is_masked_and_flagged(fp8):
    grp = Group([500, 300, 64, 20], 2, fp8, seed=6)
    bt = grp.cache.block_table
    bt[0, 2] = grp.cache.num_pages          # a miss in the middle
    bt[1, 4] = -7                            # the last page
    bt[2, 0] = 1 << 30                       # every token
    lost = {(0, 2), (1, 4), (2, 0)}
    q = queries(7, 16, 5)
    mass0 = torch.rand((4, grp.cache.max_pages_per_seq * 16), generator=gen(1))
    cap = grp.cache.capacity_tokens
    check_dense(grp, q, [0, 1, 2, 3, 4, 3, 3], [499, 299, 63, 19, 3, cap, -2], track=True, mass0=mass0,
                status=1 | 2 | 4, lost=lost)


def test_dense_decode_pages_past_four_gigabytes():
    pages = 140000                                            # 32 KiB a page
    grp = Group([700, 90], 1, seed=8, num_pages=pages, first_page=pages - 16)
    assert int(grp.cache.block_table.max()) * 32768 > 1 << 32
    check_dense(grp, queries(2, 12, 2), [0, 1], [699, 89])


def test_dense_decode_graph_streams_and_workspaces():
    grp = Group([1200, 77, 3], 2, seed=3)
    q = [queries(3, 16, s).cuda() for s in (1, 2)]
    q_seq, q_pos = i32([0, 1, 2]), i32([1199, 76, 2])
    decs = [qsa.DenseDecoder(grp.cache, 16, 3, track=True) for _ in range(2)]
    want = []
    for d, x in zip(decs, q):
        o, l = d.run(x, q_seq, q_pos)
        want.append((o.clone(), l.clone(), d.mass.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs = [qsa.StepGraph(d.bind(x, q_seq, q_pos), s) for d, x, s in zip(decs, q, streams)]
    for d in decs:
        d.out.zero_(), d.lse.zero_(), d.mass.zero_()
    torch.cuda.synchronize()
    for _ in range(2):                                        # both graphs at once, each with its own workspace
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for d, (o, l, m) in zip(decs, want):
        assert torch.equal(bits(d.out), bits(o)) and torch.equal(bits(d.lse), bits(l))
        assert torch.equal(bits(d.mass), bits(m + m))         # decay 1: twice the weights
        assert int(d.dev_status.item()) == 0
    q_pos.copy_(i32([700, -1, 0]))                            # a replay reads the lengths of its time
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    o, l = qsa.DenseDecoder(grp.cache, 16, 3).run(q[0], q_seq, q_pos)
    assert torch.equal(bits(decs[0].out), bits(o)) and torch.equal(bits(decs[0].lse), bits(l))
    with pytest.raises(ValueError):
        decs[0].run(queries(4, 16, 0).cuda(), i32([0] * 4), i32([0] * 4))
    with pytest.raises(ValueError):
        qsa.qsa_dense_decode(grp.cache, q[0], q_seq, q_pos, 1 / 16, decs[0].out, decs[0].lse, decs[0].workspace[:512])
    empty = qsa.DenseDecoder(grp.cache, 16, 1)
    o, l = empty.run(q[0][:0], q_seq[:0], q_pos[:0])
    assert o.shape[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_decode_more_queries_than_threads(fp8):
    """Several rounds of the length scan; CTAs whose share spans more queries than they keep lengths of."""
    rng = random.Random(3)
    grp = Group([2000, 333, 64, 1], 1, fp8, seed=14)
    q_seq, q_pos = [], []
    for r in range(1000):
        s = rng.choice([0, 1, 2, 3, -1, -1])
        n = grp.lens[s] if s >= 0 else 10
        q_seq.append(s)
        q_pos.append(-1 if r % 97 > 20 else min(n - 1, rng.choice([0, 3, 16, 40, n - 1])))
    mass0 = torch.rand((4, grp.cache.max_pages_per_seq * 16), generator=gen(1))
    check_dense(grp, queries(1000, 3, 1), q_seq, q_pos, track=True, decay=0.5, mass0=mass0)
    check_dense(grp, queries(1000, 3, 1), [0] * 1000, [15] * 1000)      # one tile each


def test_dense_decode_e4m3_pages_past_four_gigabytes():
    pages = 270000                                            # 16 KiB a page
    grp = Group([700, 90], 1, True, seed=8, num_pages=pages, first_page=pages - 16)
    assert int(grp.cache.block_table.max()) * 16384 > 1 << 32
    check_dense(grp, queries(2, 12, 2), [0, 1], [699, 89])


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_decode_agrees_with_the_sparse_step_that_selects_everything(fp8):
    grp = Group([1999, 500, 3], 2, fp8, seed=15)
    q, q_seq, q_pos = queries(3, 24, 4).cuda(), i32([0, 1, 2]), i32([1998, 499, 2])
    sparse = qsa.Decoder(grp.cache, 24, 3, k=512)
    so, sl = sparse.run(q, torch.ones((3, 8, 128), dtype=torch.bfloat16, device="cuda"),
                        torch.ones((3, 8), device="cuda"), q_seq, q_pos)
    do, dl = qsa.DenseDecoder(grp.cache, 24, 3).run(q, q_seq, q_pos)
    for r in range(3):
        n = int(q_pos[r]) + 1
        k, v = grp.rows(r)
        _, _, _, ob, lb, _ = D.dense(q[r].double().cpu().numpy(), k[:n], v[:n], 1 / 16, fp8)
        within(do[r].double().cpu().numpy(), so[r].double().cpu().numpy(), 2 * ob, "out")   # each within its bound
        within(dl[r].double().cpu().numpy(), sl[r].double().cpu().numpy(), 2 * lb, "lse")


# ---------------------------------------------------------------- eviction


def block_rows(cache, table, s, b, hkv):
    """K/V run of every KV head and the kc row of block b of sequence s, as bytes."""
    page = int(table[s, b // 16])
    kv = bits(cache.kv_pages[page, :, b % 16]) if cache.kv_pages is not None else None
    kc = bits(cache.kc_pages[page, b % 16]) if cache.kc_pages is not None else None
    return kv, kc


def snapshot(cache, table, lens):
    kv = cache.kv_pages.view(torch.uint8).flatten(3).cpu() if cache.kv_pages is not None else None
    kc = cache.kc_pages.view(torch.uint8).cpu() if cache.kc_pages is not None else None
    t = table.cpu().long()
    res = []
    for s, n in enumerate(lens):
        b = torch.arange(-(-n // 4))
        pg = t[s, b // 16]
        res.append((kv[pg, :, b % 16] if kv is not None else None, kc[pg, b % 16] if kc is not None else None))
    return res


def masses(rng, shape):
    g = gen(rng.randint(0, 1 << 30))
    m = torch.rand(shape, generator=g)
    pick = torch.rand(shape, generator=g)
    m = torch.where(pick < 0.2, torch.full_like(m, 0.25), m)       # ties
    m = torch.where((pick > 0.2) & (pick < 0.25), torch.zeros_like(m), m)
    m = torch.where((pick > 0.25) & (pick < 0.3), torch.full_like(m, -0.0), m)
    m = torch.where((pick > 0.3) & (pick < 0.32), torch.full_like(m, float("nan")), m)
    m = torch.where((pick > 0.32) & (pick < 0.34), torch.full_like(m, float("inf")), m)
    return torch.where((pick > 0.34) & (pick < 0.36), torch.full_like(m, -1.5), m)


def same_mass(got, want):
    got, want = got.cpu(), want.cpu()
    return torch.equal(got.view(torch.int32), want.view(torch.int32))


def check_evict(grp, budget, sink, recent, mass, ids=None, lens=None, to_free=False, alias=False, status=0,
                refused=()):
    """Run qsa_evict over a group and compare every moved byte, index and total."""
    c = grp.cache
    ids = list(range(len(grp.lens))) if ids is None else ids
    lens = [grp.lens[s] if 0 <= s < len(grp.lens) else 0 for s in ids] if lens is None else lens
    table = c.block_table.clone()
    before = snapshot(c, table, grp.lens)
    untouched_kv = c.kv_pages.clone() if to_free and c.kv_pages is not None else None
    dst = None
    if to_free:
        dst, at = torch.full_like(table, -1), 0
        free = grp.free.cuda()
        for s, n in zip(ids, lens):
            if s < 0 or s >= c.max_seqs:
                continue
            p = -(-(min(n // 4, budget) * 4 + n % 4) // 64)
            dst[s, :p] = free[at:at + p]
            at += p
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mass_in = mass.cuda()
    mass_out = mass_in if alias else torch.full_like(mass_in, -9.0)
    keep = torch.full((len(ids), budget), 77, dtype=torch.int32, device="cuda")
    cnt, seq_len = torch.full((len(ids),), 77, dtype=torch.int32, device="cuda"), i32(lens)
    new_len = seq_len if alias else torch.full_like(cnt, 77)
    ws = torch.full((qsa.evict_workspace_bytes(c, len(ids), budget),), 0xff, dtype=torch.uint8, device="cuda")
    qsa.qsa_evict(c, i32(ids), seq_len, mass_in, mass_out, budget, sink, recent, keep, cnt, new_len, ws,
                  dst_table=dst, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status, qsa.dev_status_names(int(st.item()))
    where = table if dst is None else dst
    want_mass = mass.clone() if alias else torch.full_like(mass, -9.0)
    result = {}
    for i, (s, n) in enumerate(zip(ids, lens)):
        if i in refused or s < 0:
            assert cnt[i] == 0 and new_len[i] == n and (keep[i] == -1).all()
            continue
        kept = D.keep_blocks(mass[s].tolist(), n, budget, sink, recent)
        assert keep[i].tolist() == kept + [-1] * (budget - len(kept)), f"entry {i}"
        assert int(cnt[i]) == len(kept) and int(new_len[i]) == len(kept) * 4 + n % 4
        src = kept + ([n // 4] if n % 4 else [])
        want_mass[s, :len(src)] = mass[s, src] if src else mass[s, :0]
        want_mass[s, len(src):-(-n // 4)] = 0.0
        result[s] = src
    after = snapshot(c, where, [len(result.get(s, [])) * 4 for s in range(len(grp.lens))])
    for s, src in result.items():
        for old, new in zip(before[s], after[s]):
            if old is not None and src:
                assert torch.equal(old[src], new), f"sequence {s}: rows differ"
    assert same_mass(mass_out, want_mass)
    if untouched_kv is not None:      # the old pages keep their rows
        for old, new in zip(before, snapshot(c, table, grp.lens)):
            for x, y in zip(old, new):
                assert x is None or torch.equal(x, y)
    for s in range(len(grp.lens)):    # sequences that were not listed (or refused) are as they were
        if s not in result:
            for x, y in zip(before[s], snapshot(c, table, grp.lens)[s]):
                assert x is None or torch.equal(x, y)
    return result


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv", [1, 2, 3])
@pytest.mark.parametrize("to_free", [False, True])
def test_evict_moves_every_byte(hkv, fp8, to_free):
    lens = [0, 1, 3, 4, 66, 67, 256, 257, 1000, 2049, 1027, 515]
    for seed, (budget, sink, recent) in enumerate([(64, 4, 8), (100, 0, 0), (17, 17, 0), (16, 0, 16), (1, 0, 0),
                                                    (60, 16, 30), (400, 1, 2)]):
        rng = random.Random(seed * 10 + hkv)
        grp = Group(lens, hkv, fp8, seed=seed, spare=200 if to_free else 0)
        mass = masses(rng, (len(lens), grp.cache.max_pages_per_seq * 16 + 5))
        check_evict(grp, budget, sink, recent, mass, to_free=to_free, alias=bool(seed & 1))


def test_evict_whole_budget_and_full_table():
    grp = Group([256, 255, 130], 1, seed=1, mpps=4)
    mass = masses(random.Random(1), (3, 64))
    check_evict(grp, 64, 10, 10, mass)           # the budget is the table: everything stays
    check_evict(grp, 100, 10, 10, mass)          # or beyond it
    check_evict(grp, 63, 0, 0, mass)


@pytest.mark.parametrize("shape", ["front", "back", "every other", "one in eight", "equal"])
def test_evict_patterns_of_a_long_sequence_in_place(shape):
    """Long moves in place, many units waiting on one another."""
    n = 64 * 400 + 2
    grp = Group([n, n - 7], 2, seed=11)
    nb = -(-n // 4)
    b = torch.arange(401 * 16).float()
    mass = {"front": -b, "back": b, "every other": (b % 2), "one in eight": (b % 8 == 3).float(),
            "equal": torch.ones_like(b)}[shape].expand(2, -1).contiguous()
    check_evict(grp, nb // 3, 5, 40, mass)


@pytest.mark.parametrize("alias", [False, True])
def test_evict_rows_too_long_for_shared_memory(alias):
    """More than 49,152 blocks a CTA: masses are read again and pass through the workspace (128 entries take a CTA each)."""
    lens = [198403, 500] + [1] * 126
    grp = Group(lens, 1, True, seed=13)
    mass = masses(random.Random(5), (128, grp.cache.max_pages_per_seq * 16))
    check_evict(grp, 30000, 3, 100, mass, alias=alias)
    grp = Group(lens[:2], 1, True, seed=13)          # and the same rows shared by clusters
    check_evict(grp, 30000, 3, 100, mass[:2].clone(), alias=alias)


@pytest.mark.parametrize("n", [1, 12, 20, 40, 70])
def test_evict_clusters_of_each_size(n):
    """Rows of a table that may be long: 8, 4, 2 CTAs share a row, or one takes it; short, empty and refused ones among them."""
    rng = random.Random(n)
    lens = [rng.choice([0, 3, 64, 900, 4097, 4 * rng.randint(1, 5000) + rng.randint(0, 3)]) for _ in range(n)]
    lens[0] = 20003
    grp = Group(lens, 1, True, seed=n, mpps=320)
    mass = masses(rng, (n, 320 * 16))
    ids = list(range(n)) + ([0, -1] if n > 1 else [])
    refused = {n} if n > 1 else set()
    check_evict(grp, 800, 5, 90, mass, ids=ids, lens=lens + ([4, 0] if n > 1 else []), refused=refused,
                status=2 if n > 1 else 0, alias=bool(n % 8))


@pytest.mark.parametrize("values", ["one", "two", "close", "nan", "inf", "wide"])
def test_evict_cuts_in_crowded_and_sparse_bins(values):
    """Rows of one value, of two, of neighbouring floats, of NaN, of infinities, and over all exponents."""
    g = gen(4)
    n = 3000
    m = {"one": torch.full((n,), 0.7), "two": torch.where(torch.rand(n, generator=g) < 0.5, 1.0, 2.0),
         "close": (torch.randint(0, 700, (n,), generator=g) + 0x3f800000).int().view(torch.float32),
         "nan": torch.where(torch.rand(n, generator=g) < 0.7, float("nan"), 1.0),
         "inf": torch.where(torch.rand(n, generator=g) < 0.5, float("inf"), -float("inf")),
         "wide": torch.exp2(torch.rand(n, generator=g) * 250 - 125)}[values]
    grp = Group([4 * n], 1, True, seed=16)
    mass = torch.zeros((1, grp.cache.max_pages_per_seq * 16))
    mass[0, :n] = m
    for budget in (1, 700, 1500, 2999):
        check_evict(grp, budget, 0, 0, mass, lens=[4 * n])
        grp = Group([4 * n], 1, True, seed=16)


@pytest.mark.parametrize("seed", range(4))
def test_evict_in_place_random(seed):
    rng = random.Random(seed)
    lens = [rng.randint(1, 12000) for _ in range(7)]
    grp = Group(lens, 1, bool(seed & 1), seed=seed)
    mass = masses(rng, (7, grp.cache.max_pages_per_seq * 16))
    budget = rng.randint(10, 2000)
    check_evict(grp, budget, rng.randint(0, budget // 3), rng.randint(0, budget // 3), mass,
                ids=rng.sample(range(7), 5), alias=True)


@pytest.mark.parametrize("to_free", [False, True])
def test_evict_pages_past_four_gigabytes(to_free):
    pages = 140000                                            # 32 KiB a page
    grp = Group([700, 90], 1, seed=8, num_pages=pages, first_page=pages - 26, spare=13)
    mass = masses(random.Random(3), (2, grp.cache.max_pages_per_seq * 16))
    check_evict(grp, 60, 2, 8, mass, to_free=to_free, alias=True)


@pytest.mark.parametrize("n", [2, 40, 128, 129, 300])
@pytest.mark.parametrize("to_free", [False, True])
def test_evict_many_entries_cut_uncut_and_empty(n, to_free):
    """Most entries have nothing to move, in runs longer and shorter than the search for the next."""
    rng = random.Random(n)
    lens = [rng.choice([0, 3, 40, 90, rng.randint(100, 900)]) if rng.random() < 0.3 or i == n // 2 else rng.choice([0, 5, 70])
            for i in range(n)]
    lens[n // 3] = 2000
    grp = Group(lens, 2, n == 40, seed=n, spare=sum(-(-x // 64) for x in lens) if to_free else 0)
    mass = masses(rng, (n, grp.cache.max_pages_per_seq * 16))
    ids = rng.sample(range(n), n - n // 8) + [-1] * 3
    rng.shuffle(ids)
    check_evict(grp, 30, 2, 5, mass, ids=ids, to_free=to_free, alias=True)


def test_evict_refuses_entries_and_flags_them():
    grp = Group([300, 301, 302, 303], 2, seed=4)
    mass = masses(random.Random(4), (4, grp.cache.max_pages_per_seq * 16))
    cap = grp.cache.capacity_tokens
    # padding, listed twice, out of range, lengths out of range
    check_evict(grp, 20, 2, 4, mass, ids=[0, -1, 0, 4, 2, 3], lens=[300, 9, 200, 50, cap + 1, -1],
                refused={2, 3, 4, 5}, status=2 | 4)
    # the same, short sequences whose open block alone would move
    check_evict(Group([3, 2], 1, seed=5), 4, 0, 0, torch.rand(2, 16), ids=[1, 1, -3], lens=[2, 3, 1], refused={1},
                status=2)


def test_evict_page_misses_lose_their_blocks_only():
    grp = Group([640], 1, seed=6)
    c = grp.cache
    table = c.block_table.clone()
    c.block_table[0, 4] = c.num_pages
    before = snapshot(c, table, [640])[0]
    mass = torch.ones((1, 160))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep, cnt, nl = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((1, 100), (1,), (1,)))
    ws = torch.empty(qsa.evict_workspace_bytes(c, 1, 100), dtype=torch.uint8, device="cuda")
    m = mass.cuda()
    m[0, :40] = 0
    qsa.qsa_evict(c, i32([0]), i32([640]), m, m, 100, 0, 0, keep, cnt, nl, ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 1 and int(nl) == 400
    kept = keep[0].tolist()
    after = snapshot(c, table, [400])[0]
    for k, b in enumerate(kept):
        if b // 16 != 4 and k // 16 != 4:        # neither read from nor written to the missing page
            assert torch.equal(before[0][b], after[0][k]) and torch.equal(before[1][b], after[1][k])
    assert torch.equal(snapshot(c, table, [640])[0][0][64:80], before[0][64:80])   # the page itself is untouched


def test_evict_partial_groups():
    for kw in (dict(with_kc=False), dict(with_kv=False)):
        c = qsa.PagedCache(12, 2, 6, 2, torch.randperm(12, generator=gen(1)).int().view(2, 6), **kw)
        g = torch.Generator(device="cuda").manual_seed(3)
        for t in (c.kv_pages, c.kc_pages):
            if t is not None:
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

        class Bare:
            cache, lens, hkv, free = c, [380, 250], 2, None
        check_evict(Bare, 30, 3, 4, masses(random.Random(2), (2, 96)))


def test_evict_shared_prefix_inside_the_sinks_stays_shared():
    """Two sequences share their first two pages; with those blocks as sinks, evicting one leaves the other whole."""
    grp = Group([64 * 6, 64 * 5], 1, seed=9)
    c = grp.cache
    c.block_table[1, :2] = c.block_table[0, :2]
    before = snapshot(c, c.block_table, grp.lens)[1]
    mass = masses(random.Random(3), (2, c.max_pages_per_seq * 16))
    check_evict_ids = [0]
    keep, cnt, nl = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((1, 60), (1,), (1,)))
    ws = torch.empty(qsa.evict_workspace_bytes(c, 1, 60), dtype=torch.uint8, device="cuda")
    m = mass.cuda()
    qsa.qsa_evict(c, i32(check_evict_ids), i32([384]), m, m, 60, 32, 8, keep, cnt, nl, ws)
    torch.cuda.synchronize()
    for x, y in zip(before, snapshot(c, c.block_table, grp.lens)[1]):
        assert torch.equal(x, y)


def test_evict_in_a_graph():
    grp = Group([2000, 900], 2, seed=12, spare=40)
    c = grp.cache
    mass = masses(random.Random(8), (2, c.max_pages_per_seq * 16)).cuda()
    mass_out = torch.zeros_like(mass)
    dst = torch.full_like(c.block_table, -1)
    dst[0, :7], dst[1, :7] = grp.free[:7].cuda(), grp.free[7:14].cuda()
    keep, cnt, nl = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 100), (2,), (2,)))
    ws = torch.empty(qsa.evict_workspace_bytes(c, 2, 100), dtype=torch.uint8, device="cuda")
    lens = i32([2000, 900])
    call = qsa.bind_evict(c, i32([0, 1]), lens, mass, mass_out, 100, 1, 9, keep, cnt, nl, ws, dst_table=dst)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = qsa.StepGraph([call], s)
    for n in ([2000, 900], [1777, 3], [390, 401]):
        lens.copy_(i32(n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            kept = D.keep_blocks(mass[i].tolist(), n[i], 100, 1, 9)
            assert keep[i, :len(kept)].tolist() == kept and int(nl[i]) == 4 * len(kept) + n[i] % 4
            new = snapshot(c, dst, [4 * len(kept)] * 2)[i][0]
            assert torch.equal(new, snapshot(c, c.block_table, n)[i][0][kept])


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("fp8", [False, True])
def test_rotate_append_attend_evict_as_a_serving_loop_does(fp8):
    """Steps of a layer held to a budget: rotate q and k by (t, h, w), append, attend
    over everything with totals, and evict when a sequence passes its limit."""
    hq, hkv, budget, sink, recent, limit = 6, 1, 24, 2, 6, 128
    plan = qsa.RopePlan(64, (12, 10, 10), cycled=True)
    g = gen(21)
    c = qsa.PagedCache(8, 2, 4, hkv, torch.randperm(8, generator=g).int().view(2, 4),
                       kv_dtype=qsa.KV_FP8_E4M3 if fp8 else qsa.KV_BF16)
    dec = qsa.DenseDecoder(c, hq, 2, track=True, decay=0.95)
    held = [[], []]                                   # (k, v) rows of each sequence, as stored
    total = [np.zeros(0), np.zeros(0)]
    fix = lambda x: (x.float().clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x).double().cpu().numpy()
    lens, evictions = [0, 0], 0
    for step in range(150):
        live = [0, 1] if step % 7 else [step % 2]
        n = len(live)
        q, k, v = (torch.randn((n, h, 256), generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
        ki = torch.randint(-8, 9, (n, 128), generator=g).bfloat16().cuda()
        pos = torch.tensor([[step] * n, [step % 16] * n, [step // 16] * n], dtype=torch.int32, device="cuda")
        qsa.qsa_rope(plan, pos, [q, k])
        at = i32([lens[s] for s in live])
        qsa.qsa_append_kv(c, k, v, ki, i32(live), at)
        out, lse = dec.run(q, i32(live), at)
        for r, s in enumerate(live):
            held[s].append((fix(k[r]), fix(v[r])))
            lens[s] += 1
            K, V = (np.stack([x[i] for x in held[s]]) for i in range(2))
            o, l, w, ob, lb, wb = D.dense(q[r].double().cpu().numpy(), K, V, 1 / 16, fp8)
            within(out[r].double().cpu().numpy(), o, ob, f"step {step} sequence {s}: out")
            within(lse[r].double().cpu().numpy(), l, lb, f"step {step} sequence {s}: lse")
            sums = D.block_sums(w)
            old = np.pad(total[s], (0, len(sums) - len(total[s])))
            total[s] = 0.95 * old + sums
        over = [s for s in (0, 1) if lens[s] >= limit]
        if over:
            evictions += len(over)
            m = dec.mass.double().cpu().numpy()
            new_len, keep, count = dec.evict(i32(over), i32([lens[s] for s in over]), budget, sink, recent)
            for i, s in enumerate(over):
                # totals agree with the reference: each step adds weights within 2 dz of theirs (dz about 3e-4 here, see
                    # tests/dense_ref.py), so do their sums; the cut follows the totals
                assert np.allclose(m[s, :len(total[s])], total[s], rtol=1e-3, atol=1e-5)
                kept = D.keep_blocks(m[s].tolist(), lens[s], budget, sink, recent)
                assert keep[i, :len(kept)].tolist() == kept
                idx = [4 * b + t for b in kept for t in range(4)] + list(range(lens[s] // 4 * 4, lens[s]))
                held[s] = [held[s][j] for j in idx]
                blocks = kept + ([lens[s] // 4] if lens[s] % 4 else [])
                total[s] = total[s][blocks]
                lens[s] = len(held[s])
                assert int(new_len[i]) == lens[s]
    assert evictions >= 2 and int(dec.dev_status.item()) == 0

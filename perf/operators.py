"""Measured cases of the operators around the paged cache group: rotary
positions with several axes, attention of one token over the whole cache, and
eviction by accumulated attention weight.

`run` computes a case either in plain torch operations (32 bits, 64 for the
angles) or, where `own` is true, through the library's calls.  Both read the
same buffers: the cache group's pages in the layout that include/qsa.h states.
"""
import math
import random

import torch

own = False

HEAD_DIM = 256
IDX_HEADS = 8
IDX_DIM = 128
BLOCK = 4           # tokens of a micro-block
PAGE = 64           # tokens of a page
PAGE_BLOCKS = 16
SCALE = 1.0 / 16.0  # 1 / sqrt(HEAD_DIM)
DEV = "cuda"


# ---------------------------------------------------------------- cases


def _rope(name, tokens, hq, hkv, t, h, w, image, cycled, adjacent, fused):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "sec_t": t, "sec_h": h, "sec_w": w,
            "image": image, "cycled": cycled, "adjacent": adjacent, "fused": fused}


def _decode(name, batch, lo, hi, hq, hkv, fp8, track):
    return {"name": name, "op": "decode", "batch": batch, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "fp8": fp8,
            "track": track}


def _evict(name, batch, lo, hi, hkv, budget, sink, recent):
    return {"name": name, "op": "evict", "batch": batch, "lo": lo, "hi": hi, "hkv": hkv, "budget": budget,
            "sink": sink, "recent": recent}


def listed():
    return [
        # one new token of one sequence: q, k and the indexer's q and k of a decode step (latency)
        _rope("rope-step-1", 1, 16, 2, 12, 10, 10, False, True, False, False),
        # a padded decode batch of odd size, rows cut out of one projection's output
        _rope("rope-step-57-fused", 57, 24, 2, 12, 10, 10, False, True, False, True),
        # a prompt chunk of images and text: two sequences' 4,096 new tokens
        _rope("rope-chunk-8192-images", 8192, 24, 2, 12, 10, 10, True, False, False, True),
        # one short chat: a single sequence of 4,096 tokens (latency)
        _decode("decode-b1-4k", 1, 4096, 4096, 16, 2, False, False),
        # many short requests of uneven length, odd head pair
        _decode("decode-b200-short", 200, 1, 700, 3, 1, False, False),
        # a batch of long documents
        _decode("decode-b8-32k", 8, 32768, 32768, 16, 2, False, False),
        # full serving batch at 128K: the largest
        _decode("decode-b32-128k", 32, 131072, 131072, 24, 2, False, False),
        # uneven contexts up to a quarter-million tokens, e4m3 cache
        _decode("decode-b64-ragged-fp8", 64, 16384, 262144, 12, 1, True, False),
        # a batch whose cache is held to a budget: the weights of every micro-block are totalled
        _decode("decode-b16-16k-track", 16, 9000, 16400, 24, 2, False, True),
        # one chat that ran over its budget by a page (latency)
        _evict("evict-b1-4k", 1, 4163, 4163, 2, 1024, 1, 64),
        # many chats a little over the budget: a tenth of the blocks go
        _evict("evict-b48-4k", 48, 4300, 4900, 1, 1024, 16, 128),
        # long documents cut to 32K tokens after the prompt
        _evict("evict-b8-40k", 8, 32769, 50000, 2, 8192, 16, 512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "evict"])
    hq, hkv = rng.choice([(16, 2), (24, 2), (12, 1), (6, 1), (3, 1)])
    if op == "rope":
        h = rng.randint(0, 10)
        w = rng.randint(0, 10)
        return _rope(None, _log_int(rng, 1, 8192), hq, hkv, 32 - h - w, h, w, rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.5, rng.random() < 0.5)
    if op == "decode":
        fp8 = rng.random() < 0.4
        track = rng.random() < 0.4
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, max(2, min(262144, (1 << 23) // (batch * hkv))))
        return _decode(None, batch, rng.randint(1, hi), hi, hq, hkv, fp8, track)
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 64, min(100000, (1 << 19) // (batch * hkv)))
    lo = rng.randint(max(1, hi // 2), hi)
    budget = max(4, int(hi // BLOCK * rng.uniform(0.2, 1.05)))
    sink = rng.randint(0, budget // 4)
    return _evict(None, batch, lo, hi, hkv, budget, sink, rng.randint(0, budget // 2))


def _lengths(case):
    """Tokens each sequence holds: spread over [lo, hi] (over its logarithm when wide), the case's own."""
    rng = random.Random(case["batch"] * 1000003 + case["lo"] * 31 + case["hi"])
    lo, hi = case["lo"], case["hi"]
    if hi > 10 * lo:
        ls = [_log_int(rng, lo, hi) for _ in range(case["batch"])]
    else:
        ls = [rng.randint(lo, hi) for _ in range(case["batch"])]
    ls[0] = hi
    return ls


def work(case):
    if case["op"] == "rope":
        row = (case["hq"] + case["hkv"]) * HEAD_DIM + (IDX_HEADS + 1) * IDX_DIM
        rotated = (case["hq"] + case["hkv"] + IDX_HEADS + 1) * 64
        return {"bytes": case["tokens"] * (2 * 2 * row + 12), "flops": case["tokens"] * rotated * 3}
    ls = _lengths(case)
    if case["op"] == "decode":
        elt = 1 if case["fp8"] else 2
        b = sum(ls) * case["hkv"] * 2 * HEAD_DIM * elt
        b += case["batch"] * (case["hq"] * (HEAD_DIM * 4 + 4) + 8) + 4 * sum(-(-n // PAGE) for n in ls)
        if case["track"]:
            b += 8 * sum(-(-n // BLOCK) for n in ls)
        return {"bytes": b, "flops": 4 * HEAD_DIM * case["hq"] * sum(ls)}
    blk = case["hkv"] * 4096 + 256 + 4
    kept = sum(min(n // BLOCK, case["budget"]) + (1 if n % BLOCK else 0) for n in ls)
    seen = sum(n // BLOCK for n in ls)
    return {"bytes": 2 * kept * blk + 4 * (seen - kept if seen > kept else 0) + 4 * kept, "flops": seen}


# ---------------------------------------------------------------- inputs


def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed((seed * 7919 + salt) & 0x7FFFFFFF)


def _pairs(case):
    """Rotated pairs' axes (0 time, 1 height, 2 width) and angular steps."""
    t, h, w = case["sec_t"], case["sec_h"], case["sec_w"]
    half = t + h + w
    if case["cycled"]:
        axis = [1 if i % 3 == 1 and i < 3 * h else 2 if i % 3 == 2 and i < 3 * w else 0 for i in range(half)]
    else:
        axis = [0] * t + [1] * h + [2] * w
    return axis, [1.0e7 ** (-i / half) for i in range(half)]


def _rope_inputs(case, seed):
    n, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    g = _gen(seed, 1)
    parts = [(hq, HEAD_DIM), (hkv, HEAD_DIM), (IDX_HEADS, IDX_DIM), (1, IDX_DIM)]
    if case["fused"]:  # one projection's output; the values between k and the indexer are V's
        width = sum(a * b for a, b in parts) + hkv * HEAD_DIM
        buf = torch.randn((n, width), generator=g, device=DEV, dtype=torch.bfloat16)
        xs, at = [], 0
        for i, (a, b) in enumerate(parts):
            if i == 2:
                at += hkv * HEAD_DIM
            xs.append(buf[:, at:at + a * b].unflatten(1, (a, b)))
            at += a * b
    else:
        xs = [torch.randn((n, a, b), generator=g, device=DEV, dtype=torch.bfloat16) for a, b in parts]
    rng = random.Random(seed * 17 + n)
    if case["image"]:  # images of 16 to 48 rows and columns with text between them
        pos, at = [], rng.randint(0, 100000)
        while len(pos) < n:
            for _ in range(rng.randint(1, 200)):
                pos.append((at, at, at))
                at += 1
            hh, ww = rng.randint(16, 48), rng.randint(16, 48)
            pos += [(at, at + y, at + x) for y in range(hh) for x in range(ww)]
            at += max(hh, ww)
        pos = torch.tensor(pos[:n], dtype=torch.int32).t().contiguous()
    else:  # one new token each, anywhere in a context of up to a quarter-million tokens
        pos = torch.tensor([rng.randint(0, 262143) for _ in range(n)], dtype=torch.int32).expand(3, n).contiguous()
    return xs, pos.to(DEV)


def _tables(case, lens, pages_used):
    """Random physical pages for every sequence; -1 beyond its end."""
    width = max(pages_used)
    g = torch.Generator().manual_seed(sum(lens) + 5)
    order = torch.randperm(sum(pages_used), generator=g).to(torch.int32)
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(pages_used):
        bt[s, :c] = order[at:at + c]
        at += c
    return bt


def _kv(case, seed, s, n):
    """K and V rows [n][Hkv][256] of sequence s: one key in twenty leans towards a direction that the queries share."""
    hkv = case["hkv"]
    g = _gen(seed, 1000 + s)
    k = torch.randn((n, hkv, HEAD_DIM), generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn((n, hkv, HEAD_DIM), generator=g, device=DEV, dtype=torch.bfloat16)
    lean = torch.rand((n, 1), generator=g, device=DEV) < 0.05
    u = _direction(case, seed, s)
    for h in range(hkv):
        k[:, h] += (3.0 * lean * u[h]).to(torch.bfloat16)
    if case.get("fp8"):
        return k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    return k, v


def _direction(case, seed, s):
    u = torch.randn((case["hkv"], HEAD_DIM), generator=_gen(seed, 500000 + s), device=DEV)
    return u / u.norm(dim=1, keepdim=True)


def _queries(case, seed):
    q = torch.randn((case["batch"], case["hq"], HEAD_DIM), generator=_gen(seed, 2), device=DEV)
    group = case["hq"] // case["hkv"]
    for s in range(case["batch"]):
        q[s] += 8.0 * _direction(case, seed, s).repeat_interleave(group, 0)
    return q.to(torch.bfloat16)


def _mass(case, seed, blocks):
    """Accumulated weights: heavy-tailed, a tenth exact ties, some never attended."""
    g = _gen(seed, 3)
    m = torch.exp(2.0 * torch.randn((case["batch"], blocks), generator=g, device=DEV))
    pick = torch.rand((case["batch"], blocks), generator=g, device=DEV)
    m = torch.where(pick < 0.1, torch.full_like(m, 0.5), m)
    return torch.where(pick > 0.97, torch.zeros_like(m), m)


def _chunk_swap(x):
    """Move chunk c of row r to chunk position c ^ r and back: x [..., 8 rows, 8 chunks, 8]."""
    r = torch.arange(8, device=x.device)
    idx = (r[None, :] ^ r[:, None])[..., None].expand(x.shape[-3:])
    return torch.gather(x, -2, idx.expand(x.shape))


def _to_pages(k, v, fill):
    """K, V [n][Hkv][256] -> [pages][Hkv][16][...] runs; rows behind the last token hold `fill`."""
    n, hkv = k.shape[0], k.shape[1]
    pages = -(-n // PAGE)
    if k.dtype == torch.bfloat16:
        kv = torch.full((pages * PAGE_BLOCKS, 2, BLOCK, hkv, HEAD_DIM), fill, dtype=k.dtype, device=k.device)
    else:
        kv = torch.full((pages * PAGE_BLOCKS, 2, BLOCK, hkv, HEAD_DIM), fill, device=k.device).to(k.dtype)
    whole = n // BLOCK
    raw = kv.view(torch.int16 if k.dtype == torch.bfloat16 else torch.uint8)
    for i, x in enumerate((k, v)):
        x = x.view(raw.dtype)
        raw[:whole, i] = x[:whole * BLOCK].view(whole, BLOCK, hkv, HEAD_DIM)
        if n % BLOCK:
            raw[whole, i, :n % BLOCK] = x[whole * BLOCK:]
    raw = raw.view(pages, PAGE_BLOCKS, 2 * BLOCK, hkv, HEAD_DIM).permute(0, 3, 1, 2, 4)
    if k.dtype != torch.bfloat16:
        return raw.reshape(pages, hkv, PAGE_BLOCKS, 2, BLOCK, HEAD_DIM).contiguous()
    raw = raw.reshape(pages, hkv, PAGE_BLOCKS, 8, 4, 8, 8).permute(0, 1, 2, 4, 3, 5, 6)
    return _chunk_swap(raw.contiguous()).view(pages, hkv, PAGE_BLOCKS, 4, 8, 64)


def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "rope":
        st["x"], st["pos"] = _rope_inputs(case, seed)
        st["out"] = [torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in st["x"]]
        axis, freq = _pairs(case)
        st["axis"] = torch.tensor(axis, device=DEV)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        if own:
            import sparse_attention_decode_03_b200 as qsa
            plan = qsa.RopePlan(64, (case["sec_t"], case["sec_h"], case["sec_w"]), base=1.0e7, cycled=case["cycled"],
                                adjacent=case["adjacent"])
            st["call"] = qsa.bind_rope(plan, st["pos"], st["x"], st["out"])
        return st
    lens, hkv, batch = _lengths(case), case["hkv"], case["batch"]
    used = [-(-n // PAGE) for n in lens]
    st["lens"] = lens
    bt = _tables(case, lens, used)
    width, src_pages = bt.shape[1], sum(used)
    fp8 = bool(case.get("fp8"))
    if case["op"] == "decode":
        total = src_pages
    else:  # the kept blocks go to pages of their own
        kept = [min(n // BLOCK, case["budget"]) * BLOCK + n % BLOCK for n in lens]
        used_to = [-(-n // PAGE) for n in kept]
        dst = torch.full_like(bt, -1)
        at = src_pages
        for s, c in enumerate(used_to):
            dst[s, :c] = torch.arange(at, at + c, dtype=torch.int32)
            at += c
        total = at
    shape = (total, hkv, PAGE_BLOCKS, 2, BLOCK, HEAD_DIM) if fp8 else (total, hkv, PAGE_BLOCKS, 4, 8, 64)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    st["pages"] = torch.zeros(shape, dtype=dt, device=DEV)
    st["bt_host"], st["bt"] = bt, bt.to(DEV)
    raw = torch.uint8 if fp8 else torch.int16
    for s, n in enumerate(lens):
        k, v = _kv(case, seed, s, n)
        st["pages"].view(raw)[st["bt"][s, :used[s]].long()] = _to_pages(k, v, 448.0).view(raw)
    blocks = width * PAGE_BLOCKS
    if case["op"] == "decode":
        st["q"] = _queries(case, seed)
        st["q_seq"] = torch.arange(batch, dtype=torch.int32, device=DEV)
        st["q_pos"] = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
        st["mass"] = _mass(case, seed, blocks) if case["track"] else None
        if own:
            import sparse_attention_decode_03_b200 as qsa
            cache = qsa.PagedCache(1, batch, width, hkv, st["bt"], kv_dtype=qsa.KV_FP8_E4M3 if fp8 else qsa.KV_BF16,
                                   with_kc=False)
            cache.num_pages, cache.kv_pages = total, st["pages"]
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
            st["mass_out"] = torch.zeros_like(st["mass"]) if case["track"] else None
            ws = torch.empty(qsa.dense_decode_workspace_bytes(cache, batch, case["hq"], with_mass=case["track"]),
                             dtype=torch.uint8, device=DEV)
            st["call"] = qsa.bind_dense_decode(cache, st["q"], st["q_seq"], st["q_pos"], SCALE, st["out"], st["lse"],
                                               ws, mass_in=st["mass"], mass_out=st["mass_out"], decay=0.9)
        return st
    st["dst_host"], st["dst"] = dst, dst.to(DEV)
    st["kc"] = torch.zeros((total, PAGE_BLOCKS, IDX_DIM), dtype=torch.bfloat16, device=DEV)
    st["kc"][:src_pages] = torch.randint(-32, 33, (src_pages, PAGE_BLOCKS, IDX_DIM), generator=_gen(seed, 4),
                                         device=DEV).to(torch.bfloat16)
    st["mass"] = _mass(case, seed, blocks)
    st["seq"] = torch.arange(batch, dtype=torch.int32, device=DEV)
    st["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if own:
        import sparse_attention_decode_03_b200 as qsa
        cache = qsa.PagedCache(1, batch, width, hkv, st["bt"])
        cache.num_pages, cache.kv_pages, cache.kc_pages = total, st["pages"], st["kc"]
        st["mass_out"] = torch.zeros_like(st["mass"])
        st["keep"] = torch.empty((batch, case["budget"]), dtype=torch.int32, device=DEV)
        st["count"] = torch.empty((batch,), dtype=torch.int32, device=DEV)
        st["new_len"] = torch.empty((batch,), dtype=torch.int32, device=DEV)
        ws = torch.empty(qsa.evict_workspace_bytes(cache, batch, case["budget"]), dtype=torch.uint8, device=DEV)
        st["call"] = qsa.bind_evict(cache, st["seq"], st["len"], st["mass"], st["mass_out"], case["budget"],
                                    case["sink"], case["recent"], st["keep"], st["count"], st["new_len"], ws,
                                    dst_table=st["dst"])
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    op = st["case"]["op"]
    if own:
        st["call"]()
        if op == "rope":
            return st["out"]
        if op == "decode":
            return [st["out"], st["lse"]] + ([st["mass_out"]] if st["mass"] is not None else [])
        return [st["pages"], st["kc"], st["mass_out"], st["keep"], st["count"], st["new_len"]]
    return {"rope": _plain_rope, "decode": _plain_decode, "evict": _plain_evict}[op](st)


def _plain_rope(st):
    case = st["case"]
    turn = st["pos"].double()[st["axis"]] * st["freq"][:, None]             # [pair][token], radians
    turn = (turn - 2 * math.pi * torch.round(turn / (2 * math.pi))).float().t()
    c, s = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
    half = c.shape[-1]
    outs = []
    for x in st["x"]:
        r = x[..., :2 * half].float()
        a, b = (r[..., 0::2], r[..., 1::2]) if case["adjacent"] else (r[..., :half], r[..., half:])
        y = (a * c - b * s, b * c + a * s)
        y = torch.stack(y, -1).flatten(-2) if case["adjacent"] else torch.cat(y, -1)
        outs.append(torch.cat([y.to(x.dtype), x[..., 2 * half:]], -1))
    return outs


def _rows(st, s, n, h):
    """K and V rows [n][256] of one sequence and KV head in fp32, out of the pages."""
    p = st["pages"][st["bt"][s, :-(-n // PAGE)].long(), h].float()
    if p.dim() == 5 and p.shape[2] == 4:   # BF16: [page][16][4 atoms][8 rows][64]
        p = _chunk_swap(p.unflatten(-1, (8, 8))).flatten(-2)
        p = p.transpose(2, 3).reshape(p.shape[0], PAGE_BLOCKS, 2, BLOCK, HEAD_DIM)
    p = p.transpose(1, 2)                  # [page][K, V][16]... -> rows
    return p[:, 0].reshape(-1, HEAD_DIM)[:n], p[:, 1].reshape(-1, HEAD_DIM)[:n]


def _plain_decode(st):
    case, q = st["case"], st["q"]
    group = case["hq"] // case["hkv"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    mass = torch.zeros_like(st["mass"]) if st["mass"] is not None else None
    for s, n in enumerate(st["lens"]):
        total = 0.0
        for h in range(case["hkv"]):
            k, v = _rows(st, s, n, h)
            z = (q[s, h * group:(h + 1) * group].float() * SCALE) @ k.t()
            m = z.amax(1, keepdim=True)
            e = torch.exp(z - m)
            l = e.sum(1, keepdim=True)
            w = e / l
            out[s, h * group:(h + 1) * group] = (w @ v).to(q.dtype)
            lse[s, h * group:(h + 1) * group] = (m + torch.log(l))[:, 0]
            total = total + w.sum(0)
        if mass is not None:
            nb = -(-n // BLOCK)
            wide = torch.zeros(nb * BLOCK, device=DEV)
            wide[:n] = total
            mass[s, :nb] = 0.9 * st["mass"][s, :nb] + wide.view(nb, BLOCK).sum(1)
    return [out, lse] + ([mass] if mass is not None else [])


def _pick(case, n, mass_row):
    """Kept complete blocks of a sequence of n tokens, ascending."""
    nb, budget, sink, recent = n // BLOCK, case["budget"], case["sink"], case["recent"]
    if nb <= budget:
        return torch.arange(nb, device=mass_row.device)
    mid = mass_row[sink:nb - recent]
    best = torch.sort(mid, descending=True, stable=True).indices[:budget - sink - recent] + sink
    dev = mass_row.device
    return torch.cat([torch.arange(sink, device=dev), torch.sort(best).values,
                      torch.arange(nb - recent, nb, device=dev)])


def _plain_evict(st):
    case = st["case"]
    batch, budget = case["batch"], case["budget"]
    keep = torch.full((batch, budget), -1, dtype=torch.int32, device=DEV)
    mass = torch.zeros_like(st["mass"])
    count, new_len = [], []
    for s, n in enumerate(st["lens"]):
        kept = _pick(case, n, st["mass"][s])
        c = kept.shape[0]
        keep[s, :c] = kept.int()
        count.append(c)
        new_len.append(c * BLOCK + n % BLOCK)
        src = torch.cat([kept, torch.arange(n // BLOCK, -(-n // BLOCK), device=DEV)])
        to = torch.arange(src.shape[0], device=DEV)
        sp, tp = st["bt"][s, src // PAGE_BLOCKS].long(), st["dst"][s, to // PAGE_BLOCKS].long()
        st["pages"][tp, :, to % PAGE_BLOCKS] = st["pages"][sp, :, src % PAGE_BLOCKS]
        st["kc"][tp, to % PAGE_BLOCKS] = st["kc"][sp, src % PAGE_BLOCKS]
        mass[s, :src.shape[0]] = st["mass"][s, src]
    counts = torch.tensor([count, new_len], dtype=torch.int32, device=DEV)
    return [st["pages"], st["kc"], mass, keep, counts[0], counts[1]]


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """What `run` returns for these inputs, from the definitions, in 64 bits."""
    if case["op"] == "rope":
        xs, pos = _rope_inputs(case, seed)
        axis, freq = _pairs(case)
        half = len(axis)
        outs = []
        for x in xs:
            y = x.double()
            for i in range(half):
                a = pos[axis[i]].double()[:, None] * freq[i]
                d0, d1 = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
                x0, x1 = x[..., d0].double(), x[..., d1].double()
                y[..., d0] = x0 * torch.cos(a) - x1 * torch.sin(a)
                y[..., d1] = x1 * torch.cos(a) + x0 * torch.sin(a)
            outs.append(y)
        return outs
    lens = _lengths(case)
    width = -(-max(lens) // PAGE)
    if case["op"] == "decode":
        q = _queries(case, seed).double()
        group = case["hq"] // case["hkv"]
        old = _mass(case, seed, width * PAGE_BLOCKS).double() if case["track"] else None
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
        mass = torch.zeros_like(old) if case["track"] else None
        for s, n in enumerate(lens):
            k, v = _kv(case, seed, s, n)
            got = torch.zeros(n, dtype=torch.float64, device=DEV)
            for h in range(case["hkv"]):
                rows = slice(h * group, (h + 1) * group)
                z = SCALE * (q[s, rows] @ k[:, h].double().t())
                lse[s, rows] = torch.logsumexp(z, 1)
                w = torch.exp(z - lse[s, rows, None])
                out[s, rows] = w @ v[:, h].double()
                got += w.sum(0)
            if case["track"]:
                nb = -(-n // BLOCK)
                mass[s, :nb] = 0.9 * old[s, :nb]
                mass[s].index_add_(0, torch.arange(n, device=DEV) // BLOCK, got)
        return [out, lse] + ([mass] if case["track"] else [])
    # eviction moves bits: which blocks, and their totals (the moved pages have no 64-bit value of their own)
    old = _mass(case, seed, width * PAGE_BLOCKS).cpu()
    batch, budget = case["batch"], case["budget"]
    keep = torch.full((batch, budget), -1, dtype=torch.int32)
    count, new_len = torch.zeros(batch, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    mass = torch.zeros(old.shape, dtype=torch.float64)
    for s, n in enumerate(lens):
        nb, row = n // BLOCK, old[s].tolist()
        chosen = set(range(nb))
        if nb > budget:
            last = nb - case["recent"]
            ranked = sorted(range(case["sink"], last), key=lambda b: (-row[b], b))
            chosen = set(range(case["sink"])) | set(range(last, nb))
            chosen |= set(ranked[:budget - len(chosen)])
        order = sorted(chosen)
        keep[s, :len(order)] = torch.tensor(order, dtype=torch.int32)
        count[s], new_len[s] = len(order), len(order) * BLOCK + n % BLOCK
        if n % BLOCK:
            order.append(nb)
        mass[s, :len(order)] = torch.tensor([row[b] for b in order], dtype=torch.float64)
    return [None, None, mass, keep, count, new_len]

"""Cases for timing and checking attention over a paged key-value cache:

* ``plan``    block tables and slot maps of a step, built on the GPU from the sequences' lengths: pages taken
              from a free list, pages of finished sequences given back;
* ``append``  rows of new keys and values rotated by their positions and written to the cache (bf16, or e4m3
              codes with a power-of-two scale per token and head), the queries rotated beside them;
* ``decode``  attention of one new token per sequence over its cached tokens;
* ``prefill`` causal attention of a chunk's packed rows over the cache that holds them and what came before.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it
calls this package's entry points.  Both work on the same cache bytes, whose layout is that of ``include/moe.h``:
keys [page][head][token / 16][d / C][token % 16][C] and values [page][head][token / T][d][T] with 16-byte cells
(C = T = 16 for e4m3; C = T = 8 for bf16), then a scale byte per page, head and token for each.
"""
import random

import torch

own = False

E4M3_MAX = 448.0
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
# hq, hk: query and key heads; head: their width; page: tokens a page; cache: its type; pattern: the
# random numbers that the sequences' lengths come from.

def listed():
    return [
        # one decode step of a small batch: eight rows, now and then a new page
        dict(name="plan n8 decode", op="plan", n=8, t=8, page=64, longest=4000, kind="decode", pattern=1),
        # a full step of a server: decodes, prompts and finished sequences together, small pages
        dict(name="plan n300 mixed", op="plan", n=300, t=4096, page=16, longest=16000, kind="mixed", pattern=2),
        # one token's key, value and query
        dict(name="append t1", op="append", t=1, n=1, hq=32, hk=8, head=128, rot=128, page=64, cache="bf16", x="bf16",
             longest=4000, pattern=3),
        # a decode batch of odd size into 8-bit pages: every row another page; a part of the head rotated
        dict(name="append t203 q8", op="append", t=203, n=203, hq=16, hk=2, head=256, rot=64, page=32, cache="e4m3",
             x="f32", longest=8000, pattern=4),
        # a full prompt chunk
        dict(name="append t4096", op="append", t=4096, n=5, hq=32, hk=8, head=128, rot=128, page=64, cache="bf16",
             x="bf16", longest=8000, pattern=5),
        # one sequence's next token: latency
        dict(name="decode n1 len1000", op="decode", n=1, hq=32, hk=8, head=128, page=64, cache="bf16", shortest=1000,
             longest=1000, pattern=6),
        # a server's batch of very different lengths on 8-bit pages, few tokens a page
        dict(name="decode n64 ragged q8", op="decode", n=64, hq=40, hk=8, head=128, page=16, cache="e4m3", shortest=1,
             longest=16384, pattern=7),
        # long contexts in a mid batch: the cache does not fit any on-chip memory
        dict(name="decode n32 len16000", op="decode", n=32, hq=32, hk=8, head=128, page=64, cache="bf16",
             shortest=15000, longest=16384, pattern=8),
        # three short prompts of odd lengths in one chunk, nothing cached before
        dict(name="prefill t77 n3", op="prefill", t=77, n=3, hq=14, hk=2, head=64, page=16, cache="bf16", before=0,
             pattern=9),
        # a whole prompt of a full chunk
        dict(name="prefill t4096 n1", op="prefill", t=4096, n=1, hq=32, hk=8, head=128, page=64, cache="bf16", before=0,
             pattern=10),
        # a dozen prompts packed, some of them continued, wide heads
        dict(name="prefill t2500 n12 d256", op="prefill", t=2500, n=12, hq=16, hk=2, head=256, page=32, cache="bf16",
             before=3000, pattern=11),
        # the last piece of a long prompt on 8-bit pages: few rows, many keys
        dict(name="prefill t500 before32000 q8", op="prefill", t=500, n=1, hq=32, hk=8, head=128, page=128,
             cache="e4m3", before=32000, pattern=12),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "prefill", "prefill"])
    page = rng.choice([16, 32, 64, 128, 256])
    pattern = rng.randrange(1 << 30)
    if op == "plan":
        n = _log(rng, 1, 1000)
        kind = rng.choice(["decode", "mixed"])
        return dict(op=op, n=n, t=n if kind == "decode" else _log(rng, n, 4096), page=page,
                    longest=_log(rng, 100, 16000), kind=kind, pattern=pattern)
    head, cache = rng.choice([64, 128, 128, 256]), rng.choice(["bf16", "e4m3"])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    hq = max(hk, min(hq, 8192 // head // hk * hk))
    shape = dict(hq=hq, hk=hk, head=head, page=page, cache=cache, pattern=pattern)
    if op == "append":
        t = _log(rng, 1, 4096)
        t = max(1, min(t, 4096 * 6144 // ((hq + 2 * hk) * head)))
        return dict(op=op, t=t, n=rng.choice([t, _log(rng, 1, t)]), rot=rng.choice([head, head // 2, 32]),
                    x=rng.choice(["bf16", "bf16", "f32"]), longest=_log(rng, 100, 16000), **shape)
    if op == "decode":
        n = _log(rng, 1, 128)
        longest = _log(rng, 16, 32768)
        longest = max(1, min(longest, 2 * 10 ** 9 // (4 * hk * head * n)))
        return dict(op=op, n=n, shortest=rng.choice([1, longest, max(1, longest // 2)]), longest=longest, **shape)
    t = _log(rng, 1, 4096)
    t = max(1, min(t, int((2 ** 37 / (2 * hq * head)) ** 0.5)))
    n = _log(rng, 1, min(t, 32))
    before = rng.choice([0, _log(rng, 16, 32768)])
    before = max(0, min(before, 2 ** 37 // (4 * t * hq * head) - t, 2 ** 30 // (4 * n * hk * head)))
    return dict(op=op, t=t, n=n, before=before, **shape)


def _spread(rnd, total, n):
    """n whole numbers of at least 1 with the given sum, very different from each other."""
    w = [rnd.random() ** 3 + 0.02 for _ in range(n)]
    v = [1 + int((total - n) * x / sum(w)) for x in w]
    v[rnd.randrange(n)] += total - sum(v)
    return v


def _lengths(c):
    """(tokens cached before the step, rows that the step adds; -1 for a finished sequence) of each sequence."""
    rnd = random.Random(c["pattern"])
    n = c["n"]
    if c["op"] == "decode":
        return [_log(rnd, c["shortest"], c["longest"]) - 1 for _ in range(n)], [1] * n
    if c["op"] == "prefill":
        grow = _spread(rnd, c["t"], n)
        one = n == 1
        return [c["before"] if one else int(c["before"] * rnd.choice([0, rnd.random(), 1])) for _ in range(n)], grow
    before = [_log(rnd, 1, c["longest"]) for _ in range(n)]
    if c["op"] == "append":
        return before, _spread(rnd, c["t"], n)
    if c["kind"] == "decode":
        return before, [1] * n
    grow = [rnd.choice([1, 1, 1, 0, -1]) for _ in range(n)]
    free = c["t"] - sum(g > 0 for g in grow)
    for s in range(n):                                  # a few new prompts share what is left of the chunk
        if rnd.random() < 0.1 and free > 0 and grow[s] >= 0:
            before[s] = 0
            more = rnd.randint(1, free)
            grow[s] += more
            free -= more
    return before, grow


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs

def _cells(c):
    """(values a cell, bytes a value) of the cache's type."""
    return (8, 2) if c["cache"] == "bf16" else (16, 1)


def _sections(buf, pages, c):
    """The cache's sections as views of its bytes: keys, values, and their scales (None for bf16)."""
    cell, size = _cells(c)
    count = pages * c["hk"] * c["page"] * c["head"]
    dtype = BF16 if size == 2 else E4M3
    step = -(-count * size // 256) * 256
    k = buf[:count * size].view(dtype).view(pages, c["hk"], c["page"] // 16, c["head"] // cell, 16, cell)
    v = buf[step:step + count * size].view(dtype).view(pages, c["hk"], c["page"] // cell, c["head"], cell)
    if size == 2:
        return k, v, None, None, 2 * step
    rows = pages * c["hk"] * c["page"]
    sstep = -(-rows // 256) * 256
    ks, vs = (buf[2 * step + i * sstep:2 * step + i * sstep + rows].view(pages, c["hk"], c["page"]) for i in (0, 1))
    return k, v, ks, vs, 2 * step + 2 * sstep


def _cache_bytes(pages, c):
    cell, size = _cells(c)
    count = pages * c["hk"] * c["page"]
    step = -(-count * c["head"] * size // 256) * 256
    return 2 * step + (0 if size == 2 else 2 * (-(-count // 256) * 256))


def _tables(before, grow, page, gen, spare=0):
    """Page tables with the pages of the tokens cached before, and the free pages, in random order."""
    have = [_pages(b, page) for b in before]
    want = [_pages(b + max(g, 0), page) for b, g in zip(before, grow)]
    pages = sum(have) + sum(w - h for w, h in zip(want, have)) + spare
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    width = max(want) + 2
    table = torch.full((len(before), width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")
    mine = at[None, :] < torch.tensor(have, device="cuda")[:, None]
    table[mine] = order[:sum(have)]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - sum(have)] = order[sum(have):]
    return table, free, pages, pages - sum(have)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _slots(before, grow, table, page):
    """Positions and slots of the rows that a step adds (the pages already in the table)."""
    seq = torch.repeat_interleave(torch.arange(len(grow), device="cuda"), _ints(grow))
    start = torch.cumsum(_ints(grow), 0) - _ints(grow)
    pos = (torch.arange(seq.numel(), device="cuda") - start[seq] + _ints(before)[seq])
    slot = table[seq, pos // page].long() * page + pos % page
    return pos.int(), slot.int()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    before, grow = _lengths(c)
    st = dict(c=c, before=before, grow=grow)
    page, n = c["page"], c["n"]
    if own:
        import mixture_experts_prefill_amd as mep

        st["mep"] = mep
    if c["op"] == "plan":
        table, free, pages, free_n = _tables(before, grow, page, gen, spare=7)
        st.update(table=table, free=free, pages=pages, free_n=_ints([free_n]), length=_ints(before), rows=_ints(grow))
        # the buffers that a program keeps for the step's plan
        st.update(length_out=torch.empty_like(st["length"]), free_n_out=torch.empty_like(st["free_n"]),
                  starts=torch.empty(n + 1, dtype=torch.int32, device="cuda"), lacking=_ints([0]),
                  positions=torch.empty(c["t"], dtype=torch.int32, device="cuda"),
                  slots=torch.empty(c["t"], dtype=torch.int32, device="cuda"))
        if own:
            st["layout"] = st["mep"].moe_kv_layout_make(pages, page, 8, 128, torch.bfloat16)
        return st
    # the table of a step that has been planned: pages for the new rows too
    table, _, pages, _ = _tables([b + g for b, g in zip(before, grow)], [0] * n, page, gen, spare=3)
    heads, d = c["hk"], c["head"]
    st.update(table=table, pages=pages, length=_ints([b + g for b, g in zip(before, grow)]))
    cache = torch.empty(_cache_bytes(pages, c), dtype=torch.uint8, device="cuda")
    k, v, ks, vs, _ = _sections(cache, pages, c)
    for x, s in ((k, ks), (v, vs)):
        # keys and values of roughly unit variance; as e4m3 the codes of a row reach 224..448 at scales about 2^-7
        step = max(1, pages // 8)
        for at in range(0, pages, step):
            part = torch.randn(x[at:at + step].shape, generator=gen, device="cuda")
            x[at:at + step] = (part if s is None else 100 * part).clamp(-E4M3_MAX, E4M3_MAX).to(x.dtype)
        if s is not None:
            s.copy_(torch.randint(119, 122, s.shape, generator=gen, device="cuda", dtype=torch.uint8))
    st["cache"] = cache
    if own:
        st["layout"] = st["mep"].moe_kv_layout_make(pages, page, heads, d, BF16 if c["cache"] == "bf16" else E4M3)
    if c["op"] == "append":
        t, hq = c["t"], c["hq"]
        dtype = BF16 if c["x"] == "bf16" else torch.float32
        strong = 1 + 6 * (torch.rand((hq + 2 * heads) * d, generator=gen, device="cuda") < 0.01).float()
        # q, k and v are columns of one projection's output
        qkv = (torch.randn((t, (hq + 2 * heads) * d), generator=gen, device="cuda") * strong).to(dtype)
        st["q"], st["k"], st["v"] = qkv.split([hq * d, heads * d, heads * d], dim=1)
        st["q_out"] = torch.empty((t, hq * d), dtype=BF16, device="cuda")
        st["positions"], st["slots"] = _slots(before, grow, table, page)
        half = c["rot"] // 2
        angle = torch.arange(c["longest"] + t, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half))
        st["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return st
    t = n if c["op"] == "decode" else c["t"]
    # queries that pick some keys out: scores of a standard deviation of about 1.5
    st["q"] = (1.5 * torch.randn((t, c["hq"] * d), generator=gen, device="cuda")).to(BF16)
    st["out"] = torch.empty((t, c["hq"] * d), dtype=BF16, device="cuda")
    st["starts"] = _ints([0] + torch.tensor(grow).cumsum(0).tolist())
    if own:
        st["workspace"] = torch.empty(st["mep"].moe_attention_workspace_bytes(t, n, c["hq"], st["layout"]),
                                      dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else globals()["_plain_" + st["c"]["op"]](st)


def _cache_out(st):
    c = st["c"]
    k, v, ks, vs, _ = _sections(st["cache"], st["pages"], c)
    if ks is not None:
        ks, vs = ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu)
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _plan_out(st):
    return {x: st[x] for x in ("table", "free", "free_n_out", "length_out", "starts", "positions", "slots", "lacking")}


def _run_own(st):
    c, mep = st["c"], st["mep"]
    if c["op"] == "plan":
        mep.moe_kv_plan(st["length"], st["rows"], st["layout"], st["table"], st["free"], st["free_n"], st["length_out"],
                        st["free_n_out"], st["starts"], st["positions"], st["slots"], st["lacking"])
        return _plan_out(st)
    if c["op"] == "append":
        mep.moe_kv_append(st["k"], st["v"], st["layout"], st["cache"], st["slots"], positions=st["positions"],
                          rope=st["rope"], q=st["q"], q_out=st["q_out"])
        return dict(q=st["q_out"], **_cache_out(st))
    if c["op"] == "decode":
        mep.moe_attention_decode(st["q"], st["layout"], st["cache"], st["table"], st["length"], c["head"] ** -0.5,
                                 st["out"], st["workspace"])
    else:
        mep.moe_attention_prefill(st["q"], st["starts"], st["layout"], st["cache"], st["table"], st["length"],
                                  c["head"] ** -0.5, st["out"], st["workspace"])
    return dict(out=st["out"])


def _plain_plan(st):
    """Finished sequences' pages go on top of the free list in order, new pages come off its top in order."""
    c, page, table, free = st["c"], st["c"]["page"], st["table"], st["free"]
    n, t, width = c["n"], c["t"], st["table"].shape[1]
    length, rows = st["length"].long(), st["rows"].long()
    done = rows < 0
    back = torch.where(done, (length + page - 1) // page, 0)
    old = torch.where(done, 0, length)
    ends = torch.cumsum(rows.clamp_min(0), 0).clamp_max(t)
    starts = torch.cat([ends.new_zeros(1), ends])
    want = torch.minimum(old + starts[1:] - starts[:-1], torch.full_like(old, width * page))
    have = (old + page - 1) // page
    need = (want + page - 1) // page - have
    free_n = st["free_n"].long()
    at = torch.arange(width, device="cuda")
    given = at[None, :] < back[:, None]
    top = free_n + back.sum()
    free[free_n[0] + torch.arange(int(back.sum()), device="cuda")] = table[given]
    before = torch.cumsum(need, 0) - need
    got = torch.minimum((top - before).clamp_min(0), need)
    st["length_out"].copy_(torch.minimum(want, (have + got) * page))
    st["free_n_out"].copy_(top - got.sum())
    st["starts"].copy_(starts)
    r = torch.arange(t, device="cuda")
    s = torch.searchsorted(ends, r, right=True).clamp_max(n - 1)
    pos = old[s] + r - starts[s]
    real = r < starts[-1]
    placed = real & (pos < st["length_out"][s])
    which = (pos // page).clamp(0, width - 1)
    fresh = placed & (which >= have[s])
    new = free[(top - 1 - (before[s] + which - have[s])).clamp(0, free.numel() - 1)]
    mine = torch.where(fresh, new, table[s, which]).long()
    st["positions"].copy_(torch.where(real, pos, 0))
    st["slots"].copy_(torch.where(placed, mine * page + pos % page, -1))
    table[s[fresh], which[fresh]] = mine[fresh].int()
    st["lacking"].copy_((rows.clamp_min(0).sum() - placed.sum()).reshape(1))
    return _plan_out(st)


def _rotate(x, cos, sin):
    """x [t, heads, head] float32: pairs (i, i + rot / 2) turned by the angle of (position, i)."""
    half = cos.shape[1]
    a, b, rest = x[..., :half].double(), x[..., half:2 * half].double(), x[..., 2 * half:]
    cos, sin = cos[:, None].double(), sin[:, None].double()
    return torch.cat([(a * cos - b * sin).float(), (b * cos + a * sin).float(), rest], -1)


def _quantise(x):
    """Rows [.., head] as e4m3 codes and the byte E + 127 of the smallest 2^E with the largest magnitude <= 448 * 2^E."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    return torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), (e + 127).to(torch.uint8)


def _plain_append(st):
    c = st["c"]
    t, d, page = c["t"], c["head"], c["page"]
    angles = st["rope"][st["positions"].long()]
    cos, sin = angles.chunk(2, dim=1)
    q, k, v = (st[x].float().reshape(t, -1, d) for x in ("q", "k", "v"))
    st["q_out"].copy_(_rotate(q, cos, sin).reshape(t, -1))
    slot = st["slots"].long()
    where, at = slot // page, slot % page
    kc, vc, ks, vs, _ = _sections(st["cache"], st["pages"], c)
    cell, _ = _cells(c)
    k = _rotate(k, cos, sin)
    if ks is None:
        k, v = k.to(BF16), v.to(BF16)
    else:
        (k, k_scale), (v, v_scale) = _quantise(k), _quantise(v)
        ks[where, :, at], vs[where, :, at] = k_scale, v_scale
        k, v, kc, vc = (x.view(torch.uint8) for x in (k, v, kc, vc))
    kc[where, :, at // 16, :, at % 16] = k.view(t, c["hk"], d // cell, cell)
    vc[where, :, at // cell, :, at % cell] = v
    return dict(q=st["q_out"], **_cache_out(st))


def _gathered(st, s, length):
    """Keys and values [heads, length, head] of a sequence in float32."""
    c = st["c"]
    kc, vc, ks, vs, _ = _sections(st["cache"], st["pages"], c)
    p = st["table"][s, :_pages(length, c["page"])].long()
    k = kc[p].float().permute(1, 0, 2, 4, 3, 5).reshape(c["hk"], -1, c["head"])
    v = vc[p].float().permute(1, 0, 2, 4, 3).reshape(c["hk"], -1, c["head"])
    if ks is not None:
        k = torch.ldexp(k, ks[p].int().permute(1, 0, 2).reshape(c["hk"], -1, 1) - 127)
        v = torch.ldexp(v, vs[p].int().permute(1, 0, 2).reshape(c["hk"], -1, 1) - 127)
    return k[:, :length], v[:, :length]


def _softmax(score):
    e = torch.exp(score - score.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_decode(st):
    c = st["c"]
    d, g = c["head"], c["hq"] // c["hk"]
    for s in range(c["n"]):
        k, v = _gathered(st, s, st["before"][s] + 1)
        q = st["q"][s].float().view(c["hk"], g, d)
        p = _softmax(torch.matmul(q, k.transpose(1, 2)) * d ** -0.5)
        st["out"][s] = torch.matmul(p, v).view(-1)
    return dict(out=st["out"])


def _plain_prefill(st):
    c = st["c"]
    d, g = c["head"], c["hq"] // c["hk"]
    r0 = 0
    for s in range(c["n"]):
        rows = st["grow"][s]
        length = st["before"][s] + rows
        k, v = _gathered(st, s, length)
        q = st["q"][r0:r0 + rows].float().view(rows, c["hk"], g, d)
        out = st["out"][r0:r0 + rows].view(rows, c["hk"], g, d)
        at = torch.arange(length, device="cuda")
        later = at[None, :] > torch.arange(length - rows, length, device="cuda")[:, None]
        for h in range(c["hk"]):
            score = torch.matmul(q[:, h].transpose(0, 1).reshape(g * rows, d), k[h].t()).view(g, rows, length) * d ** -0.5
            p = _softmax(score.masked_fill(later, float("-inf")))
            out[:, h] = torch.matmul(p.view(g * rows, length), v[h]).view(g, rows, d).transpose(0, 1)
        r0 += rows
    return dict(out=st["out"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    before, grow = _lengths(c)
    rows = sum(max(g, 0) for g in grow)
    if c["op"] == "plan":
        new = sum(_pages(b + g, c["page"]) - _pages(b, c["page"]) for b, g in zip(before, grow) if g > 0)
        back = sum(_pages(b, c["page"]) for b, g in zip(before, grow) if g < 0)
        # lengths and rows in, lengths and starts out, a position and a slot a row, entries moved
        return {"bytes": 4 * (4 * c["n"] + 1) + 8 * c["t"] + 8 * (new + back), "flops": 4 * rows}
    d, hq, hk = c["head"], c["hq"], c["hk"]
    token = 2 * hk * (2 * d if c["cache"] == "bf16" else d + 1)
    if c["op"] == "append":
        size = 2 if c["x"] == "bf16" else 4
        angles = len({b + i for b, g in zip(before, grow) for i in range(g)})
        return {"bytes": rows * ((hq + 2 * hk) * d * size + 2 * hq * d + token + 8) + 4 * angles * c["rot"],
                "flops": 3 * rows * (hq + hk) * c["rot"]}
    keys = sum(b + g for b, g in zip(before, grow))
    pairs = sum(g * b + g * (g + 1) // 2 for b, g in zip(before, grow))
    return {"bytes": keys * token + 4 * rows * hq * d + 4 * sum(_pages(b + g, c["page"]) for b, g in zip(before, grow)),
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_plan(st):
    """The step taken sequence by sequence and row by row, on the host."""
    c, page = st["c"], st["c"]["page"]
    table, free = st["table"].tolist(), st["free"].tolist()
    top = st["free_n"].item()
    length, starts, positions, slots = [], [0], [], []
    for s, (b, g) in enumerate(zip(st["before"], st["grow"])):
        if g < 0:
            for i in range(_pages(b, page)):
                free[top] = table[s][i]
                top += 1
    lacking = 0
    for s, (b, g) in enumerate(zip(st["before"], st["grow"])):
        held = 0 if g < 0 else b
        for i in range(max(g, 0)):
            if len(slots) == c["t"]:
                lacking += 1
                continue
            at = b + i
            positions.append(at)
            if at % page == 0 and at // page < len(table[s]) and top > 0:
                top -= 1
                table[s][at // page] = free[top]
            elif at % page == 0 or at != held:
                slots.append(-1)
                lacking += 1
                continue
            slots.append(table[s][at // page] * page + at % page)
            held += 1
        length.append(held)
        starts.append(len(slots))
    pad = c["t"] - len(slots)
    out = dict(table=table, free=free, free_n_out=[top], length_out=length, starts=starts,
               positions=positions + [0] * pad, slots=slots + [-1] * pad, lacking=[lacking])
    return {x: _ints(v) for x, v in out.items()}


def _place(tokens, table_row, c):
    """Flat indices of (page, head, token) triples [heads, tokens] for the tokens of one sequence."""
    where = table_row.long()[tokens // c["page"]]
    return (where[None, :] * c["hk"] + torch.arange(c["hk"], device="cuda")[:, None]) * c["page"] + tokens % c["page"]


def _exact_values(st, tokens, table_row):
    """Keys and values [heads, tokens, head] in float64, each element found by its own index."""
    c = st["c"]
    cell, size = _cells(c)
    d = torch.arange(c["head"], device="cuda")
    at = _place(tokens, table_row, c)[..., None]          # (page * heads + head) * page tokens + token in the page
    block, tok = at // c["page"] * (c["page"] * c["head"]), at % c["page"]
    kc, vc, ks, vs, _ = _sections(st["cache"], st["pages"], c)
    ki = block + (tok // 16) * 16 * c["head"] + (d // cell) * 16 * cell + (tok % 16) * cell + d % cell
    vi = block + (tok // cell) * cell * c["head"] + d * cell + tok % cell
    k, v = (x.view(-1).view(torch.uint8 if size == 1 else BF16)[i].view(x.dtype).double() for x, i in ((kc, ki), (vc, vi)))
    if size == 1:
        k = k * torch.exp2(ks.view(-1)[at].double() - 127)
        v = v * torch.exp2(vs.view(-1)[at].double() - 127)
    return k, v


def _exact_append(st):
    c = st["c"]
    t, d, half = c["t"], c["head"], c["rot"] // 2
    cell, size = _cells(c)
    pos, slot = st["positions"].long(), st["slots"].long()
    turn = torch.complex(st["rope"][pos, :half].double(), st["rope"][pos, half:].double())[:, None]

    def turned(x):
        x = x.double().reshape(t, -1, d).clone()
        z = torch.complex(x[..., :half].clone(), x[..., half:2 * half].clone()) * turn
        x[..., :half], x[..., half:2 * half] = z.real, z.imag
        return x

    rows = dict(k=turned(st["k"]), v=st["v"].double().reshape(t, -1, d))
    kc, vc, ks, vs, _ = _sections(st["cache"], st["pages"], c)
    out = dict(q=turned(st["q"]).reshape(t, -1))
    each = torch.arange(d, device="cuda")
    at = ((slot // c["page"])[:, None] * c["hk"] + torch.arange(c["hk"], device="cuda")) * c["page"] + (slot % c["page"])[:, None]
    tok = (slot % c["page"])[:, None, None]
    block = (at // c["page"] * (c["page"] * d))[..., None]
    index = dict(k=block + (tok // 16) * 16 * d + (each // cell) * 16 * cell + (tok % 16) * cell + each % cell,
                 v=block + (tok // cell) * cell * d + each * cell + tok % cell)
    for x, now, s in (("k", kc, ks), ("v", vc, vs)):
        y = rows[x]
        full = now.double().reshape(-1)
        scale = None
        if size == 1:
            e = torch.ceil(torch.log2(y.abs().amax(-1) / E4M3_MAX)).clamp(-127, 127)
            y = y / torch.exp2(e)[..., None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            y = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
            scale = torch.exp2(s.double() - 127).reshape(-1)
            scale[at] = torch.exp2(e)
            scale = scale.view(s.shape)
        full[index[x]] = y
        out[x], out[x + "_scale"] = full.view(now.shape), scale
    return dict(q=out["q"], k=out["k"], v=out["v"], k_scale=out["k_scale"], v_scale=out["v_scale"])


def _exact_attention(st):
    c = st["c"]
    d, g = c["head"], c["hq"] // c["hk"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    r = 0
    for s, (b, rows) in enumerate(zip(st["before"], st["grow"])):
        k, v = _exact_values(st, torch.arange(b + rows, device="cuda"), st["table"][s])
        for r0 in range(0, rows, 512):
            r1 = min(rows, r0 + 512)
            last = b + r1                                  # keys that any of these rows may see
            for h in range(c["hq"]):
                q = st["q"][r + r0:r + r1, h * d:(h + 1) * d].double()
                score = q @ k[h // g, :last].t() / d ** 0.5
                seen = torch.tril(torch.ones_like(score, dtype=torch.bool), diagonal=b + r0)
                weight = torch.where(seen, torch.exp(score - score.where(seen, score.new_tensor(-1e300)).amax(1, True)), 0.0)
                out[r + r0:r + r1, h * d:(h + 1) * d] = weight @ v[h // g, :last] / weight.sum(1, True)
        r += rows
    return dict(out=out)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["c"]["op"]
    return _exact_plan(st) if op == "plan" else _exact_append(st) if op == "append" else _exact_attention(st)

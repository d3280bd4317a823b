"""What the serving operators around the paged cache cost: the cases, their inputs, the
operators' plain forms and the library's calls.

Four operators of one serving step over a paged KV cache are measured:

  tables   block tables, slot map, positions and query offsets of a step, built on the GPU
           from the requests' lengths and a ring of free pages
  rope     rotary positions of the step's query and key rows
  append   the step's K/V rows into a cache held in 8 bits with one scale for each block of
           16 tokens (a page) and kv head
  attn     attention over such a cache: one token per sequence (decode) or a causal chunk
           (prefill)

``own`` selects the form of ``run``: False, elementary torch operations; True, the library.
A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed.
"""
import math

import torch

own = False

PAGE = 16
F32, BF16 = "f32", "bf16"
DEV_BAD_PAGE, DEV_BAD_LEN, DEV_NO_PAGES = 0x1, 0x2, 0x20


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of the batch-256 serving shape: one new token each, a few requests
        # ended, a page boundary crossed by one request in sixteen
        dict(name="tables-decode", op="tables", batch=256, cached=1024, new=1, ended=8, max_blocks=128,
             pool=32768, pad=0, short=False),
        # a mixed step of a large engine: prompt chunks of up to 512 among decode tokens
        # (odd lengths), padded to a captured size, with a pool too small for all of it
        dict(name="tables-mixed", op="tables", batch=511, cached=2048, new=257, ended=31, max_blocks=256,
             pool=131072, pad=1000, short=True),
        # queries and keys of a batch-64 decode step in float, half layout
        dict(name="rope-decode", op="rope", tokens=64, q_heads=9, kv_heads=3, head_dim=64, rotary=64,
             dtype=F32, layout="half", scaling="none", positions=1024, fused_rows=False, transposed=False),
        # a long-context prefill step: bfloat16 rows out of a fused projection, frequencies
        # scaled band by band, positions far past the trained length
        dict(name="rope-prefill", op="rope", tokens=8192, q_heads=12, kv_heads=2, head_dim=128, rotary=128,
             dtype=BF16, layout="half", scaling="bands", positions=1000000, fused_rows=True, transposed=False),
        # a training step's gradient: interleaved pairs over half of each head, odd count
        dict(name="rope-gradient", op="rope", tokens=4095, q_heads=32, kv_heads=4, head_dim=64, rotary=32,
             dtype=BF16, layout="interleaved", scaling="linear", positions=8192, fused_rows=False, transposed=True),
        # one new token for each of 256 sequences, anywhere in its page
        dict(name="append-decode", op="append", batch=256, cached=1024, new=1, kv_heads=4, head_dim=64,
             kv="int8", dtype=F32),
        # prompt chunks of sixteen sequences, starting and ending inside pages
        dict(name="append-prefill", op="append", batch=16, cached=200, new=512, kv_heads=2, head_dim=128,
             kv="fp8", dtype=BF16),
        # one short sequence: the smallest decode call, where latency counts
        dict(name="decode-single", op="decode", batch=1, context=37, ragged=False, q_heads=9, kv_heads=3,
             head_dim=64, kv="fp8", dtype=F32, window=0),
        # the batch-256 serving shape
        dict(name="decode-batch", op="decode", batch=256, context=1024, ragged=False, q_heads=32, kv_heads=4,
             head_dim=64, kv="int8", dtype=F32, window=0),
        # a few sequences of 32k tokens: the context split over the GPU and joined
        dict(name="decode-long", op="decode", batch=4, context=32768, ragged=True, q_heads=12, kv_heads=2,
             head_dim=128, kv="fp8", dtype=BF16, window=0),
        # a short odd chunk behind a short odd prefix
        dict(name="prefill-short", op="prefill", batch=1, prior=41, chunk=37, q_heads=9, kv_heads=3,
             head_dim=64, kv="int8", dtype=F32, window=0),
        # prompt chunks of 512 behind 2048 cached tokens
        dict(name="prefill-chunks", op="prefill", batch=2, prior=2048, chunk=512, q_heads=12, kv_heads=2,
             head_dim=128, kv="fp8", dtype=BF16, window=0),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "decode", "decode", "prefill", "prefill"])
    heads = rng.choice([(9, 3), (12, 2), (32, 4), (8, 8), (16, 1)])
    common = dict(kv_heads=heads[1], head_dim=rng.choice([64, 128]), kv=rng.choice(["int8", "fp8"]),
                  dtype=rng.choice([F32, BF16]))
    if op == "tables":
        batch = _spread(rng, 1, 511)
        return dict(op=op, batch=batch, cached=_spread(rng, 1, 2048), new=rng.choice([1, 1, _spread(rng, 2, 257)]),
                    ended=rng.randrange(0, batch // 8 + 1), max_blocks=256, pool=131072, pad=rng.randrange(0, 300),
                    short=rng.random() < 0.3)
    if op == "rope":
        dim = common["head_dim"]
        return dict(op=op, tokens=_spread(rng, 1, 4096), q_heads=heads[0], kv_heads=heads[1], head_dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, 2 * rng.randrange(1, dim // 2)]), dtype=common["dtype"],
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "bands"]), positions=_spread(rng, 100, 4000000),
                    fused_rows=rng.random() < 0.5, transposed=rng.random() < 0.3)
    if op == "append":
        return dict(op=op, batch=_spread(rng, 1, 100), cached=_spread(rng, 1, 300), new=_spread(rng, 1, 80), **common)
    if op == "decode":
        context = _spread(rng, 1, 32768)
        batch = _spread(rng, 1, max(1, min(300, 65536 // context)))
        return dict(op=op, batch=batch, context=context, ragged=rng.random() < 0.7, q_heads=heads[0],
                    window=rng.choice([0, 0, _spread(rng, 1, 4096)]), **common)
    chunk, batch = _spread(rng, 1, 700), rng.choice([1, 1, 2, 3])
    return dict(op=op, batch=batch, prior=_spread(rng, 1, 2048) - 1, chunk=chunk if batch < 3 else chunk // 2 + 1,
                q_heads=heads[0] if heads[0] < 32 else 16, window=rng.choice([0, 0, _spread(rng, 1, 1500)]), **common)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randint(g, lo, hi, shape):
    """Whole numbers from lo to hi, both included."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda")


def _mixed(g, lo, hi, n):
    """n whole numbers spread evenly from hi down to lo, in random order."""
    some = hi - torch.arange(n, device="cuda") * (hi - lo) // max(1, n - 1)
    return some[torch.randperm(n, generator=g, device="cuda")]


def _type(name):
    return torch.float32 if name == F32 else torch.bfloat16


def _pages(lens):
    return (lens + PAGE - 1) // PAGE


def _paged(lens, max_blocks, perm):
    """Block tables of sequences of these lengths, pages taken from `perm` in order."""
    need = _pages(lens)
    start = need.cumsum(0) - need
    col = torch.arange(max_blocks, device="cuda")[None, :]
    at = (start[:, None] + col).clamp(max=perm.numel() - 1)
    return torch.where(col < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32)


def _codes(x, kv):
    """Random rows as codes in the cache's bytes, with the scale of each block: x is
    [pages, heads, 16, dim]; the bytes keep that order."""
    top = x.abs().amax(dim=(2, 3)).clamp(min=1e-30)
    if kv == "int8":
        scale = top / 127.0
        code = torch.round(x / scale[:, :, None, None]).clamp(-127, 127)
        return (code + 128).to(torch.uint8), scale.contiguous()
    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def _cache(g, pages, heads, dim, kv):
    """A filled cache: K bytes [pages][heads][16][dim], V bytes [pages][heads][dim][16]
    (transposed) and float scales [pages][heads].  Blocks differ in size by a factor of a few,
    as layers' keys and values do."""
    size = torch.exp(0.5 * torch.randn(2, pages, heads, 1, 1, generator=g, device="cuda"))
    k, ks = _codes(torch.randn(pages, heads, PAGE, dim, generator=g, device="cuda") * size[0], kv)
    v, vs = _codes(torch.randn(pages, heads, PAGE, dim, generator=g, device="cuda") * size[1], kv)
    return k, v.transpose(2, 3).contiguous(), ks, vs


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "tables":
        n, mb, pool = case["batch"], case["max_blocks"], case["pool"]
        cached = _randint(g, 0, min(case["cached"], mb * PAGE - case["new"]), (n,))
        new = torch.full((n,), -1, device="cuda")
        live = torch.randperm(n, generator=g, device="cuda")[case["ended"]:]
        new[live] = _mixed(g, 1, case["new"], live.numel())
        perm = torch.randperm(pool, generator=g, device="cuda")
        s["block_tables"] = _paged(cached, mb, perm)
        held = int(_pages(cached).sum())
        rows = new.clamp(min=0)
        need = int((_pages(cached + rows) - _pages(cached)).sum())
        count = need // 2 if case["short"] else min(pool - held, 2 * need + 16)
        head = pool - 5  # the ring's free part wraps around its end
        ring = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(count, device="cuda")) % pool] = perm[held:held + count].to(torch.int32)
        s["ring"], s["pool"] = ring, pool
        s["state0"] = torch.tensor([head, count, 0, 0], dtype=torch.int32, device="cuda")
        s["state"] = s["state0"].clone()
        s["cached"], s["new"] = cached.to(torch.int32), new.to(torch.int32)
        total = int(rows.sum()) + case["pad"]
        i32 = dict(dtype=torch.int32, device="cuda")
        s["context"], s["starts"] = torch.zeros(n, **i32), torch.zeros(n + 1, **i32)
        s["positions"], s["slots"] = torch.zeros(total, **i32), torch.zeros(total, **i32)
        s["status"] = torch.zeros(1, **i32)
        return s
    if op == "rope":
        t, hq, hk, dim, dt = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], _type(case["dtype"])
        if case["fused_rows"]:  # views of one projection's rows: query, key and value heads
            rows = torch.randn(t, hq + 2 * hk, dim, generator=g, device="cuda").to(dt)
            s["q"], s["k"] = rows[:, :hq], rows[:, hq:hq + hk]
        else:
            s["q"] = torch.randn(t, hq, dim, generator=g, device="cuda").to(dt)
            s["k"] = torch.randn(t, hk, dim, generator=g, device="cuda").to(dt)
        s["positions"] = _randint(g, 0, case["positions"], (t,)).to(torch.int32)
        s["q_out"] = torch.empty(t, hq, dim, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(t, hk, dim, dtype=dt, device="cuda")
        return s
    heads, dim, dt = case["kv_heads"], case["head_dim"], _type(case["dtype"])
    if op == "append":
        n = case["batch"]
        cached = _randint(g, 0, case["cached"], (n,))
        new = _mixed(g, 1, case["new"], n)
        mb = -(-(case["cached"] + case["new"]) // PAGE)
        pages = n * mb
        s["k"], s["v"], s["ks"], s["vs"] = _cache(g, pages, heads, dim, case["kv"])
        bt = _paged(cached + new, mb, torch.randperm(pages, generator=g, device="cuda")).long()
        b = torch.repeat_interleave(torch.arange(n, device="cuda"), new)
        pos = cached[b] + torch.arange(b.numel(), device="cuda") - (new.cumsum(0) - new)[b]
        s["slots"] = (bt[b, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
        # new rows a little larger than the blocks they join: some blocks' scales grow
        s["k_new"] = (1.5 * torch.randn(b.numel(), heads, dim, generator=g, device="cuda")).to(dt)
        s["v_new"] = (1.5 * torch.randn(b.numel(), heads, dim, generator=g, device="cuda")).to(dt)
        return s
    n, hq = case["batch"], case["q_heads"]
    if op == "decode":
        top = case["context"]
        lens = _randint(g, max(0, top // 4), top, (n,)) if case["ragged"] else torch.full((n,), top, device="cuda")
        if case["ragged"] and n > 2:
            lens[n // 2] = 0  # a padding row of the batch: nothing to attend to
        s["q"] = torch.randn(n, hq, dim, generator=g, device="cuda").to(dt)
    else:
        top = case["prior"] + case["chunk"]
        prior = _randint(g, case["prior"] // 2, case["prior"], (n,))
        chunk = _mixed(g, (case["chunk"] + 1) // 2, case["chunk"], n)
        lens = prior + chunk
        s["starts"] = torch.cat([chunk.new_zeros(1), chunk.cumsum(0)]).to(torch.int32)
        s["q"] = torch.randn(int(chunk.sum()), hq, dim, generator=g, device="cuda").to(dt)
    mb = max(1, -(-top // PAGE))
    pages = int(_pages(lens).sum()) + 3
    s["k"], s["v"], s["ks"], s["vs"] = _cache(g, pages, heads, dim, case["kv"])
    s["block_tables"] = _paged(lens, mb, torch.randperm(pages, generator=g, device="cuda"))
    s["lens"] = lens.to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["out"] = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_tables(s):
    c, n, bt, ring = s["cached"].long(), s["new"].long(), s["block_tables"].long(), s["ring"].long()
    (num, mb), pool, total = bt.shape, s["pool"], s["slots"].numel()
    head, count = s["state0"][0].long(), s["state0"][1].long()
    ended = n < 0
    rows = n.clamp(min=0)
    end = rows.cumsum(0)
    start = end - rows
    bad = (c < 0) | (c + rows > mb * PAGE) | (~ended & (end > total))
    have = _pages(c)
    need = torch.where(bad | ended, 0, _pages(c + rows) - have)
    cum = need.cumsum(0)
    served = ~bad & ~ended & ((need == 0) | (cum <= count))
    alloc = torch.where(served & (need > 0), cum, 0).amax()
    # the step's rows
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(end, t, right=True)
    live = b < num
    b = b.clamp(max=num - 1)
    pos = c[b] + t - start[b]
    ok = live & served[b]
    page_no = torch.where(ok, pos // PAGE, 0)
    fresh = ok & (page_no >= have[b])
    at = torch.where(fresh, (head + cum[b] - need[b] + page_no - have[b]) % pool, 0)
    page = torch.where(fresh, ring[at], bt[b, page_no])
    good = ok & (page >= 0) & (page < pool)
    slots = torch.where(good, page * PAGE + pos % PAGE, -1)
    positions = torch.where(good, pos, -1)
    # new entries of the block tables, written by each page's first row
    first = fresh & (pos % PAGE == 0)
    flat = torch.cat([bt.reshape(-1), bt.new_zeros(1)])
    flat = flat.scatter(0, torch.where(first, b * mb + page_no, num * mb), torch.where(good, page, -1))
    # pages of ended requests go back, behind the free ones
    held = (torch.arange(mb, device="cuda")[None, :] < have[:, None]) & (ended & ~bad)[:, None]
    back = (held & (bt >= 0) & (bt < pool)).reshape(-1)
    j = back.long().cumsum(0) - 1
    push = back & (j < pool - count + alloc)
    out = torch.cat([ring, ring.new_zeros(1)])
    out = out.scatter(0, torch.where(push, (head + count + j) % pool, pool), bt.reshape(-1))
    wrong = (ok & ~good).any() | (held & (bt >= pool)).any() | (back & ~push).any()
    status = DEV_BAD_LEN * bad.any() + DEV_NO_PAGES * (~bad & ~ended & ~served).any() + DEV_BAD_PAGE * wrong
    state = torch.stack([(head + alloc) % pool, count - alloc + push.sum(), head * 0, head * 0])
    starts = torch.cat([end.new_zeros(1), end]).clamp(max=total)
    made = (flat[:-1].reshape(num, mb), torch.where(served, c + rows, 0), starts, positions, slots, out[:-1], state,
            status.reshape(1))
    return [x.to(torch.int32) for x in made]


_THETA, _FACTOR, _LOW, _HIGH, _TRAINED = 10000.0, 8.0, 1.0, 32.0, 8192


def _plain_freqs(case):
    rd = case["rotary"]
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    theta = _THETA
    if case["scaling"] == "base" and rd > 2:
        theta = _THETA * _FACTOR ** (rd / (rd - 2))
    f = theta ** (-2.0 * i / rd)
    if case["scaling"] == "linear":
        f = f / _FACTOR
    if case["scaling"] == "bands":
        turns = _TRAINED * f / (2 * math.pi)
        keep = ((turns - _LOW) / (_HIGH - _LOW)).clamp(0, 1)
        f = f / _FACTOR * (1 - keep) + f * keep
    return f


def _attention_factor(case):
    return 0.1 * math.log(_FACTOR) + 1.0 if case["scaling"] == "bands" else 1.0


def _plain_turn(x, cos, sin, case):
    """The first `rotary` columns of each head turned, pair by pair, in 32 bits."""
    rd = case["rotary"]
    y = x.float()
    turn, rest = y[..., :rd], y[..., rd:]
    if case["layout"] == "half":
        a, b = turn[..., :rd // 2], turn[..., rd // 2:]
        made = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        made = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([made, rest], dim=-1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    # angles of far positions need 64 bits
    angle = s["positions"].double()[:, None, None] * _plain_freqs(case)
    m = _attention_factor(case)
    cos, sin = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    if case["transposed"]:
        sin = -sin
    return [_plain_turn(s["q"], cos, sin, case), _plain_turn(s["k"], cos, sin, case)]


def _values(x, kv):
    """Codes as numbers, in 32 bits."""
    return x.float() - 128.0 if kv == "int8" else x.view(torch.float8_e4m3fn).float()


def _stored(x, kv):
    """Whole codes (INT8) or scaled rows (E4M3) as the cache's bytes."""
    return (torch.round(x).clamp(-127, 127) + 128).to(torch.uint8) if kv == "int8" else \
        x.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_scale(top, kv):
    """The scale of a block whose largest value is `top`; zero for an empty one."""
    if kv == "int8":
        return top / torch.full_like(top, 127.0)  # a true division in 32 bits
    m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1): 448 = (7/8) 2^9
    power = ((e - 9 + (m > 0.875).int()).clamp(min=-126) + 127).to(torch.int32) << 23
    return torch.where(top > 0, power.view(torch.float32), 0.0)


def _plain_append_one(store, scale, rows, page, off, kv, transposed):
    """One of K and V: the touched blocks' scales grow to hold the new rows, rows before the
    first new one are coded again at the grown scale, and the new rows are stored."""
    heads = rows.shape[1]
    x = rows.float()
    need = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(dim=-1), "amax")
    first = torch.full((scale.shape[0],), PAGE, device="cuda").index_reduce_(0, page, off, "amin")
    touched = (first < PAGE)[:, None]
    need = _plain_scale(need, kv)
    grown = torch.where((first == 0)[:, None], need, torch.maximum(scale, need))
    grown = torch.where(touched, grown, scale)
    kept = touched & (torch.arange(PAGE, device="cuda")[None, :] < first[:, None])
    again = kept[:, None, :] & (grown > scale)[:, :, None]
    by = torch.where(grown > 0, scale / grown, 0.0)[:, :, None, None]
    old = _values(store, kv)
    if transposed:
        old = old.transpose(2, 3)
    bytes_ = store.transpose(2, 3) if transposed else store
    made = torch.where(again[..., None], _stored(old * by, kv), bytes_)
    g = grown[page][..., None]
    fresh = _stored(torch.where(g > 0, x / g, 0.0), kv)
    h = torch.arange(heads, device="cuda")[None, :]
    made = made.index_put((page[:, None], h, off[:, None]), fresh)
    store.copy_(made.transpose(2, 3) if transposed else made)
    scale.copy_(grown)


def _append_out(s):
    """The updated cache.  E4M3 codes come as the values they stand for, up to their block's
    scale; an INT8 code is the whole number byte - 128, which its definition fixes exactly."""
    see = (lambda x: x) if s["case"]["kv"] == "int8" else (lambda x: x.view(torch.float8_e4m3fn))
    return [see(s["k"]), see(s["v"]), s["ks"], s["vs"]]


def _plain_append(s):
    slot, kv = s["slots"].long(), s["case"]["kv"]
    _plain_append_one(s["k"], s["ks"], s["k_new"], slot // PAGE, slot % PAGE, kv, False)
    _plain_append_one(s["v"], s["vs"], s["v_new"], slot // PAGE, slot % PAGE, kv, True)
    return _append_out(s)


def _plain_attention(s):
    """Attention of padded rows [sequences, rows] against every sequence's gathered pages."""
    case, q, bt = s["case"], s["q"], s["block_tables"].long().clamp(min=0)
    kv, heads, dim = case["kv"], case["kv_heads"], case["head_dim"]
    n, mb = bt.shape
    group = case["q_heads"] // heads
    lens = s["lens"].long()
    if "starts" in s:
        starts = s["starts"].long()
        rows = case["chunk"]
        i = torch.arange(rows, device="cuda")[None, :]
        chunk = (starts[1:] - starts[:-1])[:, None]
        there = i < chunk
        at = torch.where(there, starts[:-1, None] + i, 0)
        pos = torch.where(there, lens[:, None] - chunk + i, -1)
        qp = q[at]
    else:
        rows = 1
        pos = lens[:, None] - 1
        qp = q[:, None]
    # [n, heads, rows * group, dim]
    qp = qp.float().reshape(n, rows, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(n, heads, rows * group, dim)
    k = (_values(s["k"], kv) * s["ks"][:, :, None, None])[bt].transpose(1, 2).reshape(n, heads, mb * PAGE, dim)
    v = (_values(s["v"], kv) * s["vs"][:, :, None, None])[bt].permute(0, 2, 1, 4, 3).reshape(n, heads, mb * PAGE, dim)
    score = qp @ k.transpose(2, 3) * s["scale"]
    key = torch.arange(mb * PAGE, device="cuda")
    seen = key <= pos[..., None]
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
    seen = seen[:, None, :, None].expand(n, 1, rows, group, mb * PAGE).reshape(n, 1, rows * group, mb * PAGE)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    out = (p @ v) / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    out = out.reshape(n, heads, rows, group, dim).permute(0, 2, 1, 3, 4).reshape(n, rows, heads * group, dim)
    if "starts" not in s:
        return out[:, 0]
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    return out[b, t - starts[b]]


# ---------------------------------------------------------------------- the library's calls

def _handle(s):
    """What a serving program makes once and keeps: the cache object and the workspace."""
    from paged_kv_attention_09_gb300 import pkv

    case = s["case"]
    if case["op"] == "tables":
        return pkv, pkv.PagePool(s["ring"], s["state"])
    if case["op"] == "rope":
        kind = {"none": {}, "linear": dict(factor=_FACTOR), "base": dict(factor=_FACTOR),
                "bands": dict(factor=_FACTOR, low=_LOW, high=_HIGH, original_len=_TRAINED)}[case["scaling"]]
        return pkv, pkv.RopeParams(case["head_dim"], rotary_dim=case["rotary"], layout=case["layout"], theta=_THETA,
                                   scaling=case["scaling"], attention_factor=_attention_factor(case),
                                   transposed=case["transposed"], **kind)
    kind = pkv.INT8B if case["kv"] == "int8" else pkv.FP8B
    cache = pkv.KVCache(s["k"], s["v"], s["ks"], s["vs"], window=case.get("window", 0), kv_dtype=kind)
    if case["op"] == "append":
        return pkv, cache
    n, mb = s["block_tables"].shape
    if case["op"] == "decode":
        size = pkv.pkv_decode_workspace_size(cache, n, case["q_heads"], mb)
    else:
        size = pkv.pkv_prefill_workspace_size(cache, n, case["q_heads"], case["chunk"], mb)
    return pkv, cache, pkv.workspace_for(size)


def _own(s):
    kept = s.get("kept")
    if kept is None:
        kept = s["kept"] = _handle(s)
    op, pkv, first = s["case"]["op"], kept[0], kept[1]
    if op == "tables":
        s["state"].copy_(s["state0"])  # the pool as it was before the step
        pkv.pkv_batch_tables(first, s["cached"], s["new"], s["block_tables"], s["context"], s["starts"],
                             s["positions"], s["slots"], s["status"])
        return [s["block_tables"], s["context"], s["starts"], s["positions"], s["slots"], s["ring"], s["state"],
                s["status"]]
    if op == "rope":
        pkv.pkv_rope(s["q"], s["k"], s["positions"], first, s["q_out"], s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "append":
        pkv.pkv_append(first, s["k_new"], s["v_new"], s["slots"])
        return _append_out(s)
    if op == "decode":
        pkv.pkv_decode_attn(first, s["q"], s["block_tables"], s["lens"], s["scale"], s["out"], kept[2])
        return s["out"]
    pkv.pkv_prefill_chunk_attn(first, s["q"], s["starts"], s["case"]["chunk"], s["block_tables"], s["lens"],
                               s["scale"], s["out"], kept[2])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tables":
        return _plain_tables(state)
    if op == "rope":
        return _plain_rope(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ---------------------------------------------------------------------------- the work

def work(case):
    """Bytes and operations of one pass: each input read once, each output written once, at
    the case's mean lengths."""
    op = case["op"]
    elt = 4 if case.get("dtype") == F32 else 2
    if op == "tables":
        live = case["batch"] - case["ended"]
        rows = live * (case["new"] + 1) / 2 + case["pad"]
        pages = live * (case["new"] + 1) / 2 / PAGE + case["ended"] * (case["cached"] / 2) / PAGE
        return {"bytes": case["batch"] * 20 + rows * 8 + pages * 8, "flops": rows}
    if op == "rope":
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
        turned = values * case["rotary"] / case["head_dim"]
        return {"bytes": 2 * values * elt + 4 * case["tokens"], "flops": 3 * turned}
    heads, dim = case["kv_heads"], case["head_dim"]
    if op == "append":
        rows = case["batch"] * (1 if case["new"] == 1 else (case["new"] + 1) / 2)
        return {"bytes": rows * (2 * heads * dim * (elt + 1) + 4) + case["batch"] * 16 * heads,
                "flops": 4 * rows * heads * dim}
    if op == "decode":
        length = case["context"] * (0.625 if case["ragged"] else 1.0)
        keys = min(length, case["window"]) if case["window"] else length
        keys *= case["batch"]
        return {"bytes": keys * heads * (2 * dim + 8 / PAGE) + case["batch"] * case["q_heads"] * dim * (elt + 4)
                + 4 * keys / PAGE + 4 * case["batch"], "flops": 4 * keys * case["q_heads"] * dim}
    # one sequence is as long as the case says; prefixes are three quarters of it in the mean
    count = 1 + 0.75 * (case["batch"] - 1)
    chunk, prior = case["chunk"] * count, 0.75 * case["prior"]
    mean = prior + (case["chunk"] + 1) / 2
    if case["window"]:
        mean = min(mean, case["window"])
    keys = prior * case["batch"] + chunk
    return {"bytes": keys * heads * (2 * dim + 8 / PAGE) + chunk * case["q_heads"] * dim * (elt + 4),
            "flops": 4 * chunk * mean * case["q_heads"] * dim}


# ------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    """The operators' definitions, sequence by sequence and head by head in 64 bits."""
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        rd = case["rotary"]
        theta = 10000.0 * (8.0 ** (rd / (rd - 2.0)) if case["scaling"] == "base" and rd > 2 else 1.0)
        m = 1.0 + math.log(8.0) / 10.0 if case["scaling"] == "bands" else 1.0
        turned = [s["q"].double(), s["k"].double()]
        for i in range(rd // 2):
            f = theta ** (-2.0 * i / rd)
            if case["scaling"] == "linear":
                f /= 8.0
            elif case["scaling"] == "bands":
                part = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 31.0))
                f = part * f + (1.0 - part) * f / 8.0
            angle = s["positions"].double()[:, None] * f * (-1.0 if case["transposed"] else 1.0)
            x, y = (i, i + rd // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            for z in turned:
                turn = torch.polar(torch.full_like(angle, m), angle) * torch.complex(z[..., x], z[..., y])
                z[..., x], z[..., y] = turn.real, turn.imag
        return turned
    kv, heads = case["kv"], case["kv_heads"]

    def number(x):
        return x.double() - 128.0 if kv == "int8" else x.view(torch.float8_e4m3fn).double()

    if case["op"] == "append":
        made = []
        slot = s["slots"].long().cpu().tolist()
        pages = {}
        for t, one in enumerate(slot):
            pages.setdefault(one // PAGE, []).append((one % PAGE, t))
        if len(pages) > 3000:
            return None
        for store, scale, rows in ((s["k"], s["ks"], s["k_new"]),
                                   (s["v"].transpose(2, 3), s["vs"], s["v_new"])):
            code, size, x = number(store).cpu(), scale.double().cpu(), rows.double().cpu()
            for page, some in pages.items():
                first = min(off for off, _ in some)
                y = x[[t for _, t in some]]
                top = y.abs().amax(dim=(0, 2))
                if kv == "int8":  # the scale and the quotients are float32 by definition
                    need = (top / 127.0).float().double()
                else:
                    need = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                old = size[page].clone()
                new = need if first == 0 else torch.maximum(old, need)
                for h in range(heads):
                    if first > 0 and new[h] > old[h]:
                        by = (old[h] / new[h]).float().double()
                        again = (code[page, h, :first] * by).float()
                        code[page, h, :first] = torch.round(again).double() if kv == "int8" else \
                            again.to(torch.float8_e4m3fn).double()
                    z = (y[:, h] / new[h]).float()
                    z = torch.round(z).clamp(-127, 127) if kv == "int8" else z.to(torch.float8_e4m3fn)
                    for j, (off, _) in enumerate(some):
                        code[page, h, off] = z[j].double()
                size[page] = new
            made.append((code, size))
        (k, ks), (v, vs) = made
        none = kv == "int8"  # its codes are whole numbers
        return [None if none else k, None if none else v.transpose(2, 3).contiguous(), ks, vs]
    if work(case)["flops"] > 4e11:
        return None
    group = case["q_heads"] // heads
    lens = s["lens"].cpu().tolist()
    starts = s["starts"].cpu().tolist() if "starts" in s else list(range(len(lens) + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        if length == 0 or a == e:
            continue
        page = s["block_tables"][b, :-(-length // PAGE)].long()
        k = number(s["k"][page]) * s["ks"][page].double()[:, :, None, None]
        v = number(s["v"][page]) * s["vs"][page].double()[:, :, None, None]
        k = k.permute(1, 0, 2, 3).reshape(heads, -1, case["head_dim"])[:, :length]
        v = v.permute(1, 0, 3, 2).reshape(heads, -1, case["head_dim"])[:, :length]
        pos = torch.arange(length - (e - a), length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None, :]
        hidden = key > pos
        if case["window"]:
            hidden = hidden | (key <= pos - case["window"])
        for h in range(case["q_heads"]):
            score = s["q"][a:e, h].double() @ k[h // group].T * s["scale"]
            out[a:e, h] = torch.softmax(score.masked_fill(hidden, -math.inf), dim=-1) @ v[h // group]
    return out

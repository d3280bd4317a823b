"""The serving operators' host side without a GPU: argument checks of the C entry points and
the binding, the rotary plan's frequencies, and the reference's own pins."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import pkv


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pkv.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return pkv.load()


def _tables(lib, ring=0x10000, state=0x20000, pages=8, page_size=16, cached=0x30000, new=0x40000, n=2, bt=0x50000,
            mb=4, ctx=0x60000, qsl=0x70000, pos=0x80000, slots=0x90000, rows=5, status=0xA0000, pool=True):
    p = pkv.pkv_page_pool(ring, state, pages, page_size)
    return lib.pkv_batch_tables(ctypes.byref(p) if pool else None, cached, new, n, bt, mb, ctx, qsl, pos, slots, rows,
                                status, None)


def test_batch_tables_refusals(lib):
    assert _tables(lib, pool=False) == 1
    assert _tables(lib, ring=None) == 1 and _tables(lib, state=None) == 1
    assert _tables(lib, page_size=8) == 4
    assert _tables(lib, pages=0) == 2 and _tables(lib, n=-1) == 2 and _tables(lib, mb=0) == 2
    assert _tables(lib, rows=-1) == 2
    assert _tables(lib, pages=0x7fffffff // 16 + 1) == 2 and _tables(lib, mb=0x7fffffff // 16 + 1) == 2
    for name in ("cached", "new", "bt", "ctx", "slots"):
        assert _tables(lib, **{name: None}) == 1, name
    for name in ("cached", "new", "bt", "ctx", "qsl", "pos", "slots", "status", "ring", "state"):
        assert _tables(lib, **{name: 0x30002}) == 5, name
    # lengths overwritten while they are read: the same buffer, or one that overlaps it
    assert _tables(lib, ctx=0x30000) == 7 and _tables(lib, ctx=0x40000) == 7
    assert _tables(lib, ctx=0x30004) == 7 and _tables(lib, ctx=0x3fffc) == 7 and _tables(lib, cached=0x60004) == 7


def _params(**kw):
    d = dict(rotary_dim=64, layout=0, transposed=0, scaling=0, theta=1e4, factor=1.0, low=1.0, high=32.0,
             original_len=4096, attention_factor=1.0)
    d.update(kw)
    return pkv.pkv_rope_params(**d)


def test_rope_plan_refusals(lib):
    plan = pkv.pkv_rope_plan()

    def init(**kw):
        return lib.pkv_rope_plan_init(ctypes.byref(_params(**kw)), ctypes.byref(plan))
    assert init() == 0
    assert lib.pkv_rope_plan_init(None, ctypes.byref(plan)) == 1
    assert lib.pkv_rope_plan_init(ctypes.byref(_params()), None) == 1
    nan, inf = math.nan, math.inf
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-2), dict(layout=2), dict(scaling=4),
                dict(scaling=-1), dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(scaling=1, factor=0.5),
                dict(scaling=2, factor=nan), dict(scaling=3, low=-1.0), dict(scaling=3, high=1.0),
                dict(scaling=3, high=inf), dict(scaling=3, original_len=0), dict(attention_factor=-1.0),
                dict(attention_factor=nan)):
        assert init(**bad) == 2, bad
    assert init(rotary_dim=258) == 7
    # unused fields are not looked at
    assert init(scaling=0, factor=0.0, low=9.0, high=1.0, original_len=0) == 0


def test_rope_call_refusals(lib):
    plan = pkv.pkv_rope_plan()
    assert lib.pkv_rope_plan_init(ctypes.byref(_params()), ctypes.byref(plan)) == 0

    def call(q=0x10000, qo=0x20000, qs=0, qos=0, hq=4, k=0x30000, ko=0x40000, ks=0, kos=0, hk=2, dt=0, n=3, d=64,
             pos=0x50000, p=plan, status=None):
        return lib.pkv_rope(ctypes.byref(p) if p is not None else None, q, qo, qs, qos, hq, k, ko, ks, kos, hk, dt, n, d,
                            pos, status, None)
    assert call(p=None) == 1
    assert call(dt=2) == 3
    assert call(n=-1) == 2 and call(hq=-1) == 2 and call(hk=-1) == 2 and call(hq=65535, hk=1) == 2
    assert call(d=32) == 2           # rotary_dim 64 > head_dim
    assert call(d=512) == 7
    assert call(qs=100) == 2 and call(kos=100) == 2 and call(qs=-512) == 2   # shorter than a row
    assert call(q=None) == 1 and call(ko=None) == 1 and call(pos=None) == 1
    assert call(qo=0x10000, qs=512, qos=1024) == 2   # in place at two strides
    assert call(q=0x10002) == 5 and call(pos=0x50001) == 5 and call(status=0x60002) == 5
    assert call(n=0, q=None, k=None, pos=None) == 0 and call(hq=0, hk=0) == 0


def test_block_formats_are_checked_like_the_others(lib):
    def cache(**kw):
        d = dict(k_cache=0x10000, v_cache=0x20000, k_scale=0x30000, v_scale=0x40000, num_pages=8, page_size=16,
                 num_kv_heads=2, head_dim=64, kv_dtype=pkv.INT8B)
        d.update(kw)
        return pkv.pkv_cache(**d)
    P = None
    for kind in (pkv.INT8B, pkv.FP8B):
        def ap(c, k=0x50000, n=0):
            return lib.pkv_append(ctypes.byref(c), k, 0x60000, pkv.F32, 0x70000, n, P, P)
        assert ap(cache(kv_dtype=kind)) == 0
        assert ap(cache(kv_dtype=kind, k_scale=None)) == 1
        assert ap(cache(kv_dtype=kind, v_scale=0x40008)) == 5
        assert ap(cache(kv_dtype=kind, head_dim=96)) == 7
        c = cache(kv_dtype=kind)
        # the fused step is refused, whatever else is right
        assert lib.pkv_decode_step(ctypes.byref(c), 0x50000, pkv.F32, 0x60000, 0x70000, pkv.F32, 0x80000, P, 1e4, 2, 4,
                                   0x90000, 4, 0xA0000, 0.1, 0xB0000, P, 0, P, P) == 7
    assert lib.pkv_append(ctypes.byref(cache(kv_dtype=7)), 0x50000, 0x60000, pkv.F32, 0x70000, 1, P, P) == 3


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0), dict(scaling="base", factor=8.0),
                                dict(scaling="bands", factor=8.0, low=1.0, high=4.0, original_len=8192),
                                dict(rotary_dim=2, scaling="base", factor=2.0)])
def test_plan_frequencies(lib, kw):
    """Turns per position as fractions of 2^64: pow rounds to a few 2^-53, the division by 2 pi
    and the scalings to 2^-53 each, and the fraction is cut off at 2^-64 (below the value's
    53rd bit for frequencies under 2^-11 of a turn)."""
    rd = kw.get("rotary_dim", 128)
    par = pkv.RopeParams(128, **kw)
    kw = {k: v for k, v in kw.items() if k != "rotary_dim"}
    want = R.freqs(rd, **kw) / (2 * math.pi)
    got = np.array([par._plan.freq[i] / 2.0 ** 64 for i in range(rd // 2)])
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64)
    # the exact fraction of a turn at a far position, from whole numbers
    p = 2**31 - 1
    turns = (p * par._plan.freq[1 % (rd // 2)]) % 2**64 / 2.0 ** 64
    assert abs((turns - p * want[1 % (rd // 2)] + 0.5) % 1 - 0.5) <= p * 2.0 ** -48


def test_binding_refuses_what_it_cannot_pass_on(lib):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        pkv.PagePool(z(4, 2), z(4))
    with pytest.raises(ValueError):
        pkv.PagePool(z(8), z(3))
    pool = pkv.PagePool(z(8), z(4))
    good = dict(cached_lens=z(2), new_lens=z(2), block_tables=z(2, 3), context_lens=z(2), q_start_loc=z(3),
                positions=z(5), slot_mapping=z(5))
    for name, bad in (("new_lens", z(3)), ("cached_lens", z(4)[::2]), ("block_tables", z(3, 3)),
                      ("block_tables", z(3, 2).t()), ("context_lens", z(2).long()), ("q_start_loc", z(2)),
                      ("positions", z(4))):
        with pytest.raises(ValueError):
            pkv.pkv_batch_tables(pool, **dict(good, **{name: bad}), stream=0)
    par = pkv.RopeParams(64)
    q, k, pos = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64), z(5)
    for bad in (dict(q=torch.zeros(5, 4, 32)), dict(positions=z(4)), dict(k=torch.zeros(4, 2, 64)),
                dict(k=k.bfloat16()), dict(q=torch.zeros(4, 5, 64).transpose(0, 1)),
                dict(q_out=torch.zeros(5, 4, 128)[..., ::2]), dict(k_out=torch.zeros(5, 3, 64)),
                dict(positions=pos.long())):
        with pytest.raises(ValueError):
            pkv.pkv_rope(**dict(dict(q=q, k=k, positions=pos, params=par), **bad), stream=0)
    with pytest.raises(pkv.PkvError):
        pkv.RopeParams(64, rotary_dim=128)
    with pytest.raises(KeyError):
        pkv.RopeParams(64, layout="other")


@pytest.mark.parametrize("kv_dtype", [pkv.INT8B, pkv.FP8B])
def test_binding_refuses_rows_that_are_not_dense(lib, kv_dtype):
    cache = pkv.KVCache.allocate(4, 2, 64, kv_dtype, device="cpu")
    slots = torch.zeros(3, dtype=torch.int32)
    rows = torch.zeros(3, 2, 64)
    for k, v in ((rows[:2], rows), (rows, torch.zeros(3, 4, 64)[:, ::2]), (rows, rows.bfloat16()),
                 (torch.zeros(2, 3, 64).transpose(0, 1), rows), (torch.zeros(3, 2, 128), torch.zeros(3, 2, 128))):
        with pytest.raises(ValueError, match="contiguous"):
            pkv.pkv_append(cache, k, v, slots)
    pkv.pkv_append(cache, rows, rows, slots, stream=0, bound=True)
    bt, lens = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    starts = torch.arange(4, dtype=torch.int32)
    q = torch.zeros(3, 4, 64)
    for x, out in ((torch.zeros(4, 3, 64).transpose(0, 1), q), (q, torch.zeros(3, 8, 64)[:, ::2]), (q, q.bfloat16()),
                   (q, q[:2]), (torch.zeros(3, 4, 128), torch.zeros(3, 4, 128))):
        with pytest.raises(ValueError, match="contiguous"):
            pkv.pkv_decode_attn(cache, x, bt, lens, 0.125, out)
        with pytest.raises(ValueError, match="contiguous"):
            pkv.pkv_decode_attn_noalloc(cache, x, bt, lens, 0.125, out)
        with pytest.raises(ValueError, match="contiguous"):
            pkv.pkv_prefill_chunk_attn(cache, x, starts, 1, bt, lens, 0.125, out)
    pkv.pkv_decode_attn(cache, q, bt, lens, 0.125, q.clone(), stream=0, bound=True)


def test_bound_calls_are_not_issued(monkeypatch):
    calls = []

    class Rec:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0
    par = pkv.RopeParams(64)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = pkv.PagePool(z(8), z(4))
    monkeypatch.setattr(pkv, "load", lambda path=pkv.LIB_PATH: Rec())
    a = pkv.pkv_rope(torch.zeros(5, 4, 64), None, z(5), par, stream=0, bound=True)
    b = pkv.pkv_batch_tables(pool, z(2), z(2), z(2, 3), z(2), None, None, z(5), stream=0, bound=True)
    assert calls == []
    a()
    b()
    assert calls == ["pkv_rope", "pkv_batch_tables"]


def test_allocated_caches_and_pools():
    c = pkv.KVCache.allocate(5, 2, 64, pkv.FP8B, device="cpu")
    assert c.k.shape == (5, 2, 16, 64) and c.v.shape == (5, 2, 64, 16) and c.k.dtype == torch.uint8
    assert c.k_scale.shape == (5, 2) and c.clone().kv_dtype == pkv.FP8B
    p = pkv.PagePool.allocate(6, device="cpu")
    assert p.ring.tolist() == list(range(6)) and p.state.tolist() == [0, 6, 0, 0]


# ------------------------------------------------------------------- the reference's pins

def test_reference_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(R.E4M3, nan=1e9))
    rng = np.random.default_rng(0)
    mags = R.E4M3[:127]
    x = np.concatenate([rng.standard_normal(20000) * 10, rng.standard_normal(2000) * 1e-2, (mags[1:] + mags[:-1]) / 2,
                        mags]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_code(x), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_reference_block_scale_and_append(fp8):
    rng = np.random.default_rng(1)
    for top in [448.0, 448.0001, 1.75, 1.7500001, 3.5, 2.0 ** -130, 3e38] + list(np.exp(rng.standard_normal(50) * 5)):
        s = float(R.block_scale(np.float32(top), fp8))
        t = float(np.float32(top))
        if fp8:
            assert math.log2(s) == round(math.log2(s)) and t / s <= 448
            assert s == 2.0 ** -126 or t / (s / 2) > 448
        else:
            assert abs(s * 127 / t - 1) <= 2.0 ** -23 or t < 1e-36
    # appended one by one without growth: the same bytes as all at once
    x = rng.standard_normal((16, 1, 64)).astype(np.float32)
    x[0] *= 4
    a, b = R.BlockCache(1, 1, 64, fp8), R.BlockCache(1, 1, 64, fp8)
    a.append(x, x, list(range(16)))
    for t in range(16):
        b.append(x[t:t + 1], x[t:t + 1], [t])
    if np.abs(x[0]).max() >= np.abs(x).max():
        assert np.array_equal(a.k, b.k) and np.array_equal(a.v, b.v) and np.array_equal(a.ks, b.ks)
    k, v = a.rows(0, [0], 16)
    assert np.array_equal(k, v) and np.abs(k - x[:, 0]).max() <= (0.04 if not fp8 else 2.0 ** -4) * np.abs(x).max()


def test_reference_tables_by_hand():
    w = R.tables([4, 5, 6, 7, 0, 1, 2, 3], [6, 4, 0, 0], [15, 16, 3], [2, 1, -1], [[3, -1], [2, -1], [1, -1]], 5)
    assert w["bt"] == [[3, 2], [2, 3], [1, -1]]
    assert w["context"] == [17, 17, 0] and w["starts"] == [0, 2, 3, 3]
    assert w["positions"] == [15, 16, 16, -1, -1] and w["slots"] == [3 * 16 + 15, 2 * 16, 3 * 16, -1, -1]
    assert w["state"][:2] == [0, 3] and w["ring"][2] == 1 and w["status"] == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_rope_pins(layout):
    """Complex multiplication, and scores that depend on the distance alone."""
    rng = np.random.default_rng(2)
    f = R.freqs(16)
    x, y = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    i = np.arange(8)
    a, b = (i, i + 8) if layout == "half" else (2 * i, 2 * i + 1)
    z = (x[0, 0, a] + 1j * x[0, 0, b]) * np.exp(1j * 5 * f)
    r = R.rope(x, [5], 16, layout, f)[0, 0]
    assert np.allclose(r[a], z.real) and np.allclose(r[b], z.imag)
    s1 = (R.rope(x, [105], 16, layout, f) * R.rope(y, [100], 16, layout, f)).sum()
    s2 = (R.rope(x, [5], 16, layout, f) * R.rope(y, [0], 16, layout, f)).sum()
    assert abs(s1 - s2) < 1e-10
    assert np.allclose(R.rope(R.rope(x, [7], 16, layout, f), [7], 16, layout, f, transposed=True), x)

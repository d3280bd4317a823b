"""Caches held in 8 bits with one scale for each block of 16 tokens and kv head (INT8B,
FP8B): append, decode and chunked prefill on the GPU against the definitions in 64 bits.

Append is compared bit for bit, whole cache.

Attention tolerance.  Operands are exact in FP16 (queries to 2^-22), sums are FP32.  With A
the largest sum of |q_i k_i| of a row's keys in log2 units (computed beside the reference), a
score is off by at most A (16 2^-23 + 2^-22) (its FP32 sum in at most 16 steps, and the
queries), the exponent's argument by 2 A 2^-24 more, so a probability by ln 2 times that,
relative, and 2^-20 for exp2, the two FP16 parts and the V scale's logarithm.  Numerator and
sum both carry that (factor 2).  Accumulating over at most n = 2 pages steps adds n 2^-23, the
merges 2^-20.  All relative to the row's sum of |p v|, at most max|v|."""
import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import pkv

pytestmark = pytest.mark.gpu


def tol(bc, tables, A):
    n = 2 * tables.shape[1]
    p = np.log(2) * A * (18 * 2.0 ** -23 + 2.0 ** -23) + 2.0 ** -20
    return (2 * p + n * 2.0 ** -23 + 2.0 ** -20) * vmax(bc)

FORMATS = [False, True]
IDS = ["int8b", "fp8b"]


def rounded(x, dtype):
    return torch.from_numpy(x).to(dtype).float().numpy() if dtype == torch.bfloat16 else x


def append(cache, k, v, slots, dtype, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_append(cache, torch.from_numpy(k).to(dtype).cuda(), torch.from_numpy(v).to(dtype).cuda(),
                   torch.tensor(slots, dtype=torch.int32, device="cuda"), status, **kw)
    torch.cuda.synchronize()
    return int(status.item())


def draw_rows(rng, T, H, D, dtype, spread=1.0):
    """New K and V rows whose sizes differ from token to token (blocks' scales grow)."""
    size = np.exp(spread * rng.standard_normal((2, T, H, 1)))
    x = (rng.standard_normal((2, T, H, D)) * size).astype(np.float32)
    return rounded(x[0], dtype), rounded(x[1], dtype)


def token_slots(table, a, b):
    return [int(table[t // 16]) * 16 + t % 16 for t in range(a, b)]


def built(rng, lens, H, D, fp8, P=None, MB=None, spread=0.7, size=(1.0, 1.0)):
    """A cache that holds sequences of these lengths (values through the reference's append,
    in pieces), everything else filled with NaN codes and NaN scales."""
    need = sum(R.pages(n) for n in lens)
    P = need + 3 if P is None else P
    MB = max([R.pages(n) for n in lens] + [1]) + 1 if MB is None else MB
    perm = rng.permutation(P)
    bc = R.BlockCache(P, H, D, fp8, fill=0x7f)
    tables = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        tables[b, :R.pages(n)] = perm[at:at + R.pages(n)]
        at += R.pages(n)
        k, v = draw_rows(rng, n, H, D, torch.float32, spread)
        cut = n // 3
        for lo, hi in ((0, cut), (cut, n)):
            if hi > lo:
                assert bc.append(k[lo:hi] * np.float32(size[0]), v[lo:hi] * np.float32(size[1]),
                                 token_slots(tables[b], lo, hi)) == 0
    return bc, tables


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def vmax(bc):
    v = R.block_values(bc.v, bc.fp8) * bc.vs[:, :, None, None]
    return float(np.nanmax(np.abs(v))) if np.isfinite(v).any() else 1.0


# ------------------------------------------------------------------------------- append

@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_token_by_token_and_in_chunks(fp8, D, dtype):
    """Chunks that start and end anywhere in pages, then tokens one by one: the whole cache
    bit for bit, bytes that no row owns included."""
    rng = np.random.default_rng(D)
    H, P = 3, 24
    bc = R.BlockCache(P, H, D, fp8, fill=0x55)
    dev = bc.device(pkv)
    table = rng.permutation(P)
    at = [0, 0, 0]
    for step, lens in enumerate([(37, 1, 16), (11, 20, 0), (1, 1, 1), (1, 1, 1), (5, 3, 30)]):
        slots, n = [], sum(lens)
        for s, m in enumerate(lens):
            slots += token_slots(table[8 * s:8 * s + 8], at[s], at[s] + m)
            at[s] += m
        slots += [-1, -1]
        k, v = draw_rows(rng, n + 2, H, D, dtype, 1.0)
        assert append(dev, k, v, slots, dtype) == bc.append(k, v, slots) == 0
        assert bc.same_as(dev), step


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_append_values_at_the_edges(fp8):
    """All-zero rows, exact ties, exact powers of two, the type's largest and smallest
    values, growth from an all-zero block, growth by a factor of 2^60."""
    rng = np.random.default_rng(1)
    D, H = 64, 1
    rows = [np.zeros(D), np.full(D, 1e-30), np.linspace(-127, 127, D), np.linspace(-63.5, 63.5, D) * 2,
            np.full(D, 448.0), np.full(D, 448.1), np.full(D, -2.0 ** 40), np.full(D, 3e38), np.full(D, 1e-42),
            rng.standard_normal(D)]
    x = np.array(rows, dtype=np.float32)[:, None]
    bc = R.BlockCache(4, H, D, fp8, fill=0)
    dev = bc.device(pkv)
    for t in range(len(rows)):  # one by one into page 2: each growth codes the page again
        a, b = x[t:t + 1], x[::-1][t:t + 1].copy()
        assert append(dev, a, b, [32 + t], torch.float32) == bc.append(a, b, [32 + t]) == 0
        assert bc.same_as(dev), t


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_append_reports_bad_slots(fp8):
    rng = np.random.default_rng(2)
    bc = R.BlockCache(4, 2, 64, fp8, fill=0)
    dev = bc.device(pkv)
    slots = [64, 5, 4, 17, 18, 20, 2**31 - 1, -7, 40, 40]
    k, v = draw_rows(rng, len(slots), 2, 64, torch.float32)
    for page in range(4):  # scales that the rows before offset 0 of a run can be read at
        bc.ks[page] = bc.vs[page] = 0.25
    dev = bc.device(pkv)
    assert append(dev, k, v, slots, torch.float32) == bc.append(k, v, slots) == R.BAD_SLOT
    assert bc.same_as(dev)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_recoded_rows_stay_near_the_values_given(fp8):
    """Sixteen rows appended one by one, each larger than the last: every growth codes the
    rows before it again.  INT8B: each coding is off by at most half a step of its scale and
    the last one is the largest: 16 halves of it bound the sum (8 steps).  FP8B scales are powers
    of two, so only codes that leave the normal range round again: 2^-4 of the value from the
    first rounding, and at most half of 2^-9 steps of each later scale, which sum to less than
    2^-9 of the last."""
    rng = np.random.default_rng(3)
    bc = R.BlockCache(1, 1, 64, fp8)
    dev = bc.device(pkv)
    x = (rng.standard_normal((16, 1, 64)) * (1 + np.arange(16))[:, None, None]).astype(np.float32)
    for t in range(16):
        append(dev, x[t:t + 1], x[t:t + 1], [t], torch.float32)
        bc.append(x[t:t + 1], x[t:t + 1], [t])
    assert bc.same_as(dev)
    k, _ = bc.rows(0, [0], 16)
    s = float(bc.ks[0, 0])
    err = np.abs(k - x[:, 0].astype(np.float64))
    if fp8:
        assert np.all(err <= np.abs(x[:, 0]) * 2.0 ** -4 + s * 2.0 ** -9)
    else:
        assert np.all(err <= 8 * s)


# ------------------------------------------------------------------------------- decode

def run_decode(bc, tables, lens, q, window=0, split=0, noalloc=False):
    cache = bc.device(pkv, window=window)
    B, Hq, D = q.shape
    out = torch.full((B, Hq, D), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bt, ln = i32(tables), i32(lens)
    scale = 1 / np.sqrt(D)
    if noalloc:
        pkv.pkv_decode_attn_noalloc(cache, q, bt, ln, scale, out, status, split_pages=split)
    else:
        n = pkv.pkv_decode_workspace_size(cache, B, Hq, bt.shape[1], split)
        pkv.pkv_decode_attn(cache, q, bt, ln, scale, out, pkv.workspace_for(n), status, split_pages=split)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), int(status.item())


LENS = [0, 1, 15, 16, 17, 33, 100, 257, 400]


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("Hq,H,D", [(9, 3, 64), (12, 2, 128), (32, 4, 64), (4, 4, 128), (20, 1, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 40])
def test_decode_against_the_definition(fp8, Hq, H, D, dtype, window):
    rng = np.random.default_rng(Hq + D)
    bc, tables = built(rng, LENS, H, D, fp8)
    q = torch.from_numpy(rng.standard_normal((len(LENS), Hq, D)).astype(np.float32)).to(dtype).cuda()
    want, A = R.decode(bc, q.float().cpu().numpy(), tables, LENS, 1 / np.sqrt(D), window)
    for split in (0, 1, 3, 8):
        got, status = run_decode(bc, tables, LENS, q, window, split)
        assert status == 0
        assert np.abs(got - want).max() <= tol(bc, tables, A), split
    same, status = run_decode(bc, tables, LENS, q, window, 3, noalloc=True)
    assert status == 0
    again, _ = run_decode(bc, tables, LENS, q, window, 3)
    assert np.array_equal(same, again)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("Hq,H,D", [(8, 4, 64), (6, 2, 128)])
@pytest.mark.parametrize("window", [0, 21])
def test_decode_of_more_sequences_than_one_wave_of_wide_blocks(fp8, Hq, H, D, window):
    """Batches past that take blocks of fewer warps; split or not, rows depend on their own
    sequence only."""
    rng = np.random.default_rng(D + window)
    lens = [int(n) for n in rng.integers(0, 70, 240)]
    bc, tables = built(rng, lens, H, D, fp8)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)).astype(np.float32)).cuda()
    want, A = R.decode(bc, q.cpu().numpy(), tables, lens, 1 / np.sqrt(D), window)
    for split in (0, 1, 2):
        got, status = run_decode(bc, tables, lens, q, window, split)
        assert status == 0
        assert np.abs(got - want).max() <= tol(bc, tables, A), split


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("Hq,H,D", [(8, 1, 64), (3, 1, 64), (6, 1, 128)])
def test_decode_of_many_splits(fp8, Hq, H, D):
    """Up to 157 partials, joined in batches by all or half of a block's threads."""
    rng = np.random.default_rng(Hq)
    lens = [2500, 7, 1290]
    bc, tables = built(rng, lens, H, D, fp8, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    want, A = R.decode(bc, q.float().cpu().numpy(), tables, lens, 1 / np.sqrt(D))
    for split in (0, 1, 2, 5, 9):
        got, status = run_decode(bc, tables, lens, q, split=split)
        assert status == 0
        assert np.abs(got - want).max() <= tol(bc, tables, A), split


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("size", [(1.0, 1e-6), (1.0, 1e6), (1e5, 1.0), (1e-5, 1e-12), (3.0, 1e30)])
def test_decode_and_prefill_over_the_range_of_values(fp8, size):
    """V (and K) of very small and very large values: nothing leaves FP16's range inside.
    Scores grow with K: the softmax scale is divided by K's size."""
    rng = np.random.default_rng(5)
    bc, tables = built(rng, [300, 47], 2, 64, fp8, size=size, spread=1.5)
    q = torch.from_numpy(rng.standard_normal((2, 8, 64)).astype(np.float32)).cuda()
    cache = bc.device(pkv)
    scale = float(np.float32(0.125 / size[0]))
    want, A = R.decode(bc, q.cpu().numpy(), tables, [300, 47], scale)
    out = torch.empty(2, 8, 64, device="cuda")
    n = pkv.pkv_decode_workspace_size(cache, 2, 8, tables.shape[1])
    pkv.pkv_decode_attn(cache, q, i32(tables), i32([300, 47]), scale, out, pkv.workspace_for(n))
    assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A)
    qs = torch.from_numpy(rng.standard_normal((50, 8, 64)).astype(np.float32)).cuda()
    starts = [0, 33, 50]
    want, A = R.prefill(bc, qs.cpu().numpy(), starts, tables, [300, 47], scale)
    out = torch.empty(50, 8, 64, device="cuda")
    n = pkv.pkv_prefill_workspace_size(cache, 2, 8, 33, tables.shape[1])
    pkv.pkv_prefill_chunk_attn(cache, qs, i32(starts), 33, i32(tables), i32([300, 47]), scale, out,
                               pkv.workspace_for(n))
    assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_decode_blocks_of_zeros(fp8):
    """A page whose K (or V) is all zero has scale 0: its keys still count in the softmax."""
    rng = np.random.default_rng(6)
    bc, tables = built(rng, [64], 1, 64, fp8)
    for page, (a, s) in ((0, (bc.k, bc.ks)), (1, (bc.v, bc.vs)), (2, (bc.k, bc.ks)), (2, (bc.v, bc.vs))):
        a[tables[0, page]] = 0 if fp8 else 128
        s[tables[0, page]] = 0
    q = torch.from_numpy(rng.standard_normal((1, 4, 64)).astype(np.float32)).cuda()
    want, A = R.decode(bc, q.cpu().numpy(), tables, [64], 1 / 8)
    got, status = run_decode(bc, tables, [64], q)
    assert status == 0 and np.abs(got - want).max() <= tol(bc, tables, A)
    got, status = run_prefill(bc, tables, [64], q, [0, 1])
    assert status == 0 and np.abs(got - want).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_decode_reports_bad_pages_and_lengths(fp8):
    rng = np.random.default_rng(7)
    lens = [40, 50, 60, 20]
    bc, tables = built(rng, lens, 2, 64, fp8)
    q = torch.from_numpy(rng.standard_normal((4, 4, 64)).astype(np.float32)).cuda()
    want, A = R.decode(bc, q.cpu().numpy(), tables, lens, 1 / 8)
    tables[1, 2] = bc.P
    tables[2, 0] = -1
    got, status = run_decode(bc, tables, [40, 50, 60, 16 * tables.shape[1] + 1], q)
    assert status == R.BAD_PAGE | R.BAD_LEN
    assert np.isnan(got[1:]).all() and np.abs(got[0] - want[0]).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_decode_is_the_same_under_any_page_order(fp8):
    rng = np.random.default_rng(8)
    bc, tables = built(rng, [333, 90], 2, 128, fp8)
    q = torch.from_numpy(rng.standard_normal((2, 12, 128)).astype(np.float32)).cuda()
    a, _ = run_decode(bc, tables, [333, 90], q, split=4)
    perm = rng.permutation(bc.P)
    inv = np.argsort(perm)
    for name in ("k", "v", "ks", "vs"):
        setattr(bc, name, getattr(bc, name)[perm])
    moved = np.where(tables >= 0, inv[np.maximum(tables, 0)], -1).astype(np.int32)
    b, _ = run_decode(bc, moved, [333, 90], q, split=4)
    assert np.array_equal(a, b)


# ------------------------------------------------------------------------------ prefill

def run_prefill(bc, tables, lens, q, starts, window=0, key_split=0, max_q=None):
    cache = bc.device(pkv, window=window)
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    top = max_q or max(1, int(np.diff(starts).max()))
    n = pkv.pkv_prefill_workspace_size(cache, len(lens), Hq, top, tables.shape[1], key_split)
    ws = pkv.workspace_for(n)
    for _ in range(2):  # the workspace is ready for the next call
        pkv.pkv_prefill_chunk_attn(cache, q, i32(starts), top, i32(tables), i32(lens), 1 / np.sqrt(D), out, ws,
                                   status, key_split=key_split)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), int(status.item())


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("Hq,H,D", [(9, 3, 64), (12, 2, 128), (4, 4, 128), (20, 1, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 50])
def test_prefill_against_the_definition(fp8, Hq, H, D, dtype, window):
    """(prior, chunk) pairs: empty chunk, single tokens, chunk without a prefix, ragged ends
    inside pages and tiles, several row tiles."""
    rng = np.random.default_rng(Hq + D + window)
    shapes = [(41, 37), (7, 0), (0, 1), (129, 1), (0, 65), (200, 23), (63, 16)]
    lens = [a + b for a, b in shapes]
    starts = np.concatenate([[0], np.cumsum([b for _, b in shapes])])
    bc, tables = built(rng, lens, H, D, fp8)
    q = torch.from_numpy(rng.standard_normal((starts[-1], Hq, D)).astype(np.float32)).to(dtype).cuda()
    want, A = R.prefill(bc, q.float().cpu().numpy(), starts, tables, lens, 1 / np.sqrt(D), window)
    for key_split in (0, 1, 2, 3):
        got, status = run_prefill(bc, tables, lens, q, starts, window, key_split)
        assert status == 0
        assert np.abs(got - want).max() <= tol(bc, tables, A), key_split


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_prefill_long_prefix(fp8):
    rng = np.random.default_rng(11)
    bc, tables = built(rng, [1500], 1, 128, fp8, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((30, 6, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    want, A = R.prefill(bc, q.float().cpu().numpy(), [0, 30], tables, [1500], 1 / np.sqrt(128))
    for key_split in (1, 3):
        got, status = run_prefill(bc, tables, [1500], q, [0, 30], key_split=key_split)
        assert status == 0 and np.abs(got - want).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_reads_from_cold_memory(fp8, D, dtype):
    """With the cache out of L2 the softmax can be three tiles ahead of the values: every call
    gives the same bits, over one to fourteen key tiles and their shares."""
    rng = np.random.default_rng(D)
    lens, chunk = [100, 230, 380, 500, 640, 1290, 1700], 24
    starts = np.arange(len(lens) + 1) * chunk
    bc, tables = built(rng, lens, 1, D, fp8, spread=0.5)
    q = torch.from_numpy(rng.standard_normal((starts[-1], 5, D)).astype(np.float32)).to(dtype).cuda()
    want, A = R.prefill(bc, q.float().cpu().numpy(), starts, tables, lens, 1 / np.sqrt(D))
    other = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    cache = bc.device(pkv)
    for key_split in (1, 2, 3):
        n = pkv.pkv_prefill_workspace_size(cache, len(lens), 5, chunk, tables.shape[1], key_split)
        ws = pkv.workspace_for(n)
        first = None
        for _ in range(8):
            out = torch.full(q.shape, 7.0, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            other.add_(1)
            pkv.pkv_prefill_chunk_attn(cache, q, i32(starts), chunk, i32(tables), i32(lens), 1 / np.sqrt(D), out, ws,
                                       status, key_split=key_split)
            assert int(status.item()) == 0
            if first is None:
                first = out
                assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A), key_split
            assert torch.equal(out, first)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_scores_and_values_that_rise(fp8, D, dtype):
    """The running maximum and the gain on the values change in the middle and at the ends of
    the segments that one accumulator takes: what came before keeps its weight."""
    rng = np.random.default_rng(D + 1)
    levels = [0, 0, 0, 9, 18, 18, 18, 18, 27.5, 36, 36, 36, 36, 45, 45]  # log2 units, by 128 keys
    rises = [1, 1, 1, 1, 300, 300, 1, 1e4, 1e4, 1e4, 1e4, 1, 3e5, 3e5, 3e5]
    n, rows = 128 * len(levels) - 37, 9
    bc, tables = built(rng, [1], 1, D, fp8, P=R.pages(n) + 2, MB=R.pages(n) + 1)
    tables[0, :R.pages(n)] = rng.permutation(bc.P)[:R.pages(n)]
    way = rng.choice([-1.0, 1.0], D)
    level = np.repeat(levels, 128)[:n, None, None] + 0.5 * rng.standard_normal((n, 1, 1))
    k = (way * level * np.log(2) / np.sqrt(D)).astype(np.float32)
    v = (np.repeat(rises, 128)[:n, None, None] * rng.standard_normal((n, 1, D))).astype(np.float32)
    for t in range(0, n, 16):
        assert bc.append(k[t:t + 16], v[t:t + 16], token_slots(tables[0], t, min(t + 16, n))) == 0
    q = torch.from_numpy(np.tile(way, (rows, 4, 1)).astype(np.float32)).to(dtype).cuda()
    for length in (128 * 5 - 3, 128 * 9 + 30, n):
        want, A = R.prefill(bc, q.float().cpu().numpy(), [0, rows], tables, [length], 1 / np.sqrt(D))
        seen = R.block_values(bc.v, bc.fp8) * bc.vs[:, :, None, None]
        bound = tol(bc, tables, A) / vmax(bc) * np.nanmax(np.abs(seen[tables[0, :R.pages(length)]]))
        for key_split in (1, 2, 3):
            got, status = run_prefill(bc, tables, [length], q, [0, rows], key_split=key_split)
            assert status == 0 and np.abs(got - want).max() <= bound, (length, key_split)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
@pytest.mark.parametrize("key_split", [1, 3])
def test_prefill_reports_errors(fp8, key_split):
    rng = np.random.default_rng(12)
    lens = [100, 90, 80, 20]
    bc, tables = built(rng, lens, 2, 64, fp8)
    starts = [0, 10, 20, 30, 55]
    q = torch.from_numpy(rng.standard_normal((55, 4, 64)).astype(np.float32)).cuda()
    want, A = R.prefill(bc, q[:10].cpu().numpy(), [0, 10], tables[:1], lens[:1], 1 / 8)
    tables[1, 1], tables[2, 4] = bc.P + 5, -1
    got, status = run_prefill(bc, tables, lens, q, starts, key_split=key_split)
    assert status == R.BAD_PAGE | R.BAD_CHUNK
    assert np.isnan(got[10:]).all() and np.abs(got[:10] - want).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_prefill_rows_behind_the_last_sequence_are_left_alone(fp8):
    rng = np.random.default_rng(13)
    bc, tables = built(rng, [30], 1, 64, fp8)
    q = torch.from_numpy(rng.standard_normal((12, 2, 64)).astype(np.float32)).cuda()
    got, status = run_prefill(bc, tables, [30], q, [0, 7], max_q=300)
    assert status == 0 and (got[7:] == 7).all() and not (got[:7] == 7).any()


def test_prefill_query_range():
    """Query rows of very different sizes, an all-zero row, and rows of 1e30 and 1e-30 with a
    softmax scale to match: each row is brought to FP16's range by its own power of two."""
    rng = np.random.default_rng(14)
    bc, tables = built(rng, [70], 1, 64, True)
    x = rng.standard_normal((20, 4, 64)).astype(np.float32)
    x[3] = 0
    for size in (1e30, 1.0, 1e-30):
        q = (x * np.float32(size)).astype(np.float32)
        cache = bc.device(pkv)
        out = torch.empty(20, 4, 64, device="cuda")
        scale = float(np.float32(0.125 / size))
        want, A = R.prefill(bc, q, [0, 20], tables, [70], scale)
        pkv.pkv_prefill_chunk_attn(cache, torch.from_numpy(q).cuda(), i32([0, 20]), 20, i32(tables), i32([70]), scale,
                                   out, pkv.workspace_for(pkv.pkv_prefill_workspace_size(cache, 1, 4, 20, tables.shape[1])))
        assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_softmax_scale_of_zero_averages(fp8):
    """scale 0: every visible key weighs the same, in masked and unmasked pages alike."""
    rng = np.random.default_rng(17)
    bc, tables = built(rng, [37], 1, 64, fp8)
    cache = bc.device(pkv)
    q = torch.from_numpy(rng.standard_normal((5, 4, 64)).astype(np.float32)).cuda()
    out = torch.empty(5, 4, 64, device="cuda")
    want, A = R.prefill(bc, q.cpu().numpy(), [0, 5], tables, [37], 0.0)
    pkv.pkv_prefill_chunk_attn(cache, q, i32([0, 5]), 5, i32(tables), i32([37]), 0.0, out,
                               pkv.workspace_for(pkv.pkv_prefill_workspace_size(cache, 1, 4, 5, tables.shape[1])))
    assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A)
    pkv.pkv_decode_attn(cache, q[4:], i32(tables), i32([37]), 0.0, out,
                        pkv.workspace_for(pkv.pkv_decode_workspace_size(cache, 1, 4, tables.shape[1])))
    assert np.abs(out[:1].cpu().numpy() - want[4:]).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_negative_softmax_scale(fp8):
    rng = np.random.default_rng(18)
    bc, tables = built(rng, [100], 1, 64, fp8)
    cache = bc.device(pkv)
    q = torch.from_numpy(rng.standard_normal((5, 4, 64)).astype(np.float32)).cuda()
    out = torch.empty(5, 4, 64, device="cuda")
    want, A = R.prefill(bc, q.cpu().numpy(), [0, 5], tables, [100], -0.125)
    pkv.pkv_prefill_chunk_attn(cache, q, i32([0, 5]), 5, i32(tables), i32([100]), -0.125, out,
                               pkv.workspace_for(pkv.pkv_prefill_workspace_size(cache, 1, 4, 5, tables.shape[1])))
    assert np.abs(out.cpu().numpy() - want).max() <= tol(bc, tables, A)
    pkv.pkv_decode_attn(cache, q[4:], i32(tables), i32([100]), -0.125, out,
                        pkv.workspace_for(pkv.pkv_decode_workspace_size(cache, 1, 4, tables.shape[1])))
    assert np.abs(out[:1].cpu().numpy() - want[4:]).max() <= tol(bc, tables, A)


@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_offsets_past_32_bits(fp8):
    """Pages at the far end of a pool whose K alone is larger than 4 GiB: byte offsets of 33
    bits in append, decode and prefill."""
    P, H, D = 160000, 16, 128  # 160000 * 16 * 2048 bytes = 5.2 GB for K and as much for V
    cache = pkv.KVCache.allocate(P, H, D, pkv.FP8B if fp8 else pkv.INT8B)
    rng = np.random.default_rng(19)
    table = [P - 1, 3, P - 7]
    n = 40
    k, v = draw_rows(rng, n, H, D, torch.float32, 0.3)
    slots = token_slots(np.array(table), 0, n)
    assert append(cache, k, v, slots, torch.float32) == 0
    small = R.BlockCache(3, H, D, fp8)
    assert small.append(k, v, list(range(n))) == 0
    for i, page in enumerate(table):
        assert np.array_equal(cache.k[page].cpu().numpy(), small.k[i]) and np.array_equal(cache.v[page].cpu().numpy(), small.v[i])
    bt = np.array([table], dtype=np.int32)
    order = np.array([[0, 1, 2]], dtype=np.int32)
    q = torch.from_numpy(rng.standard_normal((2, H, D)).astype(np.float32)).cuda()
    want, A = R.prefill(small, q.cpu().numpy(), [0, 2], order, [n], D ** -0.5)
    out = torch.empty(2, H, D, device="cuda")
    pkv.pkv_prefill_chunk_attn(cache, q, i32([0, 2]), 2, i32(bt), i32([n]), D ** -0.5, out,
                               pkv.workspace_for(pkv.pkv_prefill_workspace_size(cache, 1, H, 2, 3)))
    assert np.abs(out.cpu().numpy() - want).max() <= tol(small, order, A)
    pkv.pkv_decode_attn(cache, q[1:], i32(bt), i32([n]), D ** -0.5, out,
                        pkv.workspace_for(pkv.pkv_decode_workspace_size(cache, 1, H, 3)))
    assert np.abs(out[:1].cpu().numpy() - want[1:]).max() <= tol(small, order, A)


# ------------------------------------------------------------------- graphs and refusals

@pytest.mark.parametrize("fp8", FORMATS, ids=IDS)
def test_decode_graph_runs_append_and_attention(fp8):
    """The bucketed executor over a block-scaled layer: bit for bit the direct calls."""
    rng = np.random.default_rng(15)
    lens = [37, 16, 1, 70]
    bc, tables = built(rng, lens, 2, 64, fp8)
    k, v = draw_rows(rng, 4, 2, 64, torch.float32)
    slots = [token_slots(tables[b], n - 1, n)[0] for b, n in enumerate(lens)]
    q = torch.from_numpy(rng.standard_normal((4, 8, 64)).astype(np.float32)).cuda()
    kd, vd, bt, ln, sl = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i32(tables), i32(lens), i32(slots)
    a, b = bc.device(pkv), bc.device(pkv)
    out_a, out_b = torch.empty_like(q), torch.empty_like(q)
    pkv.pkv_append(a, kd, vd, sl)
    n = pkv.pkv_decode_workspace_size(a, 4, 8, bt.shape[1])
    pkv.pkv_decode_attn(a, q, bt, ln, 0.125, out_a, pkv.workspace_for(n))
    g = pkv.DecodeGraph([pkv.GraphLayer(b, q, out_b, kd, vd)], bt, ln, 0.125, [4], slot_mapping=sl)
    g.launch(4)
    torch.cuda.synchronize()
    g.close()
    assert torch.equal(out_a, out_b) and torch.equal(a.k, b.k) and \
        torch.equal(a.v_scale.view(torch.int32), b.v_scale.view(torch.int32))  # (unused blocks hold NaN)
    with pytest.raises(pkv.PkvError) as e:  # no fused step over these formats
        pkv.DecodeGraph([pkv.GraphLayer(b, q, out_b, kd, vd)], bt, ln, 0.125, [4], slot_mapping=sl, fused=True)
    assert e.value.code == 7


def test_two_captured_graphs_share_a_workspace():
    """A split decode and a split prefill captured with one workspace, replayed in turn."""
    rng = np.random.default_rng(16)
    bc, tables = built(rng, [900], 1, 64, True, spread=0.5)
    cache = bc.device(pkv)
    q = torch.from_numpy(rng.standard_normal((20, 8, 64)).astype(np.float32)).cuda()
    bt, ln, st = i32(tables), i32([900]), i32([0, 20])
    n = max(pkv.pkv_decode_workspace_size(cache, 1, 8, bt.shape[1], 4),
            pkv.pkv_prefill_workspace_size(cache, 1, 8, 20, bt.shape[1], 3))
    ws = pkv.workspace_for(n)
    a, b = torch.empty(1, 8, 64, device="cuda"), torch.empty(20, 8, 64, device="cuda")

    def decode():
        pkv.pkv_decode_attn(cache, q[:1], bt, ln, 0.125, a, ws, split_pages=4)

    def prefill():
        pkv.pkv_prefill_chunk_attn(cache, q, st, 20, bt, ln, 0.125, b, ws, key_split=3)
    decode()
    want_a = a.clone()
    ws.zero_()
    prefill()
    want_b = b.clone()
    ws.zero_()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        decode()
    with torch.cuda.graph(gb):
        prefill()
    for _ in range(3):
        a.zero_(), b.zero_()
        ga.replay()
        ws[:64].zero_()  # (the two calls keep their counters in different layouts)
        gb.replay()
        ws[:64].zero_()
        torch.cuda.synchronize()
        assert torch.equal(a, want_a) and torch.equal(b, want_b)

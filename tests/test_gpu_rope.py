"""pkv_rope on the GPU against the definition in 64 bits.

Tolerance.  cos and sin come from sincospif (2 units in the last place: 2^-22 relative, on
values up to 1) of an angle that is exact but for its rounding to float (2^-25 of a value up
to 1, times pi: 2^-23 absolute); frequencies rounded to 2^-53 move the angle of position p by
p 2^-52 turns at most (2^-21 turns = 3e-6 at 2^31).  An output a c - b s then differs by at
most (|a| + |b|) (2^-22 + 2^-23 + 2^-24 + 2 pi p 2^-52), and is rounded once to its type."""
import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import pkv

pytestmark = pytest.mark.gpu


def rows(g, T, H, D, dtype):
    return torch.randn(T, H, D, generator=g, device="cuda").to(dtype)


def f64(x):
    return x.double().cpu().numpy()


def check(got, x, pos, rd, layout, f, m=1.0, transposed=False):
    want = R.rope(f64(x), pos, rd, layout, f, m, transposed)
    half = torch.finfo(x.dtype).eps / 2 if x.dtype != torch.float32 else 2.0 ** -24
    big = np.abs(f64(x)).max()
    p = max(1, int(np.max(pos)))
    tol = m * 2 * big * (2.0 ** -22 + 2.0 ** -23 + 2.0 ** -24 + 2 * np.pi * p * 2.0 ** -52) + half * np.abs(want)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (err.max(), (err - tol).max())


KINDS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
         dict(scaling="bands", factor=8.0, low=1.0, high=32.0, original_len=4096)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rd", [(64, 64), (128, 128), (64, 32), (128, 48), (64, 2), (128, 30), (80, 80), (6, 4),
                                  (256, 256)])
def test_layouts_sizes_and_types(dtype, layout, D, rd):
    g = torch.Generator(device="cuda").manual_seed(D + rd)
    T, Hq, Hk = 37, 5, 2
    q, k = rows(g, T, Hq, D, dtype), rows(g, T, Hk, D, dtype)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    par = pkv.RopeParams(D, rotary_dim=rd, layout=layout)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pkv.pkv_rope(q, k, pos, par, qo, ko)
    f = R.freqs(rd)
    p = pos.cpu().numpy()
    check(qo, q, p, rd, layout, f)
    check(ko, k, p, rd, layout, f)
    assert torch.equal(qo[..., rd:], q[..., rd:])
    # in place: the same bits
    q2, k2 = q.clone(), k.clone()
    pkv.pkv_rope(q2, k2, pos, par)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("T", [1, 2, 255, 4097])
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k.get("scaling", "none"))
def test_scalings_and_lengths(T, kind):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k = rows(g, T, 12, 128, torch.bfloat16), rows(g, T, 2, 128, torch.bfloat16)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.pkv_rope(q, k, pos, pkv.RopeParams(128, attention_factor=1.2, **kind), qo, ko)
    f = R.freqs(128, **kind)
    check(qo, q, pos.cpu().numpy(), 128, "half", f, m=float(np.float32(1.2)))
    check(ko, k, pos.cpu().numpy(), 128, "half", f, m=float(np.float32(1.2)))


def test_far_positions():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = rows(g, 64, 3, 64, torch.float32)
    pos = torch.randint(2**31 - 100000, 2**31 - 1, (64,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2**31 - 1
    qo = torch.empty_like(q)
    pkv.pkv_rope(q, None, pos, pkv.RopeParams(64), qo)
    check(qo, q, pos.cpu().numpy(), 64, "half", R.freqs(64))


def test_negative_positions_are_padding():
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = rows(g, 33, 4, 64, torch.float32), rows(g, 33, 2, 64, torch.float32)
    pos = torch.arange(33, device="cuda", dtype=torch.int32)
    pos[5:9] = -1
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pkv.pkv_rope(q, k, pos, pkv.RopeParams(64, rotary_dim=32), qo, ko)
    assert (qo[5:9] == 7).all() and (ko[5:9] == 7).all()
    keep = [i for i in range(33) if not 5 <= i < 9]
    check(qo[keep], q[keep], pos[keep].cpu().numpy(), 32, "half", R.freqs(32))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_views_of_a_fused_projection(layout, dtype, shift):
    """Any token stride and any element alignment; only the rows' own elements change."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, Hq, Hk, D = 29, 4, 2, 64
    width = (Hq + 2 * Hk) * D + shift
    flat = torch.randn(T * width + shift, generator=g, device="cuda").to(dtype)
    row = flat[shift:].view(T, width)
    q = row[:, :Hq * D].unflatten(1, (Hq, D))
    k = row[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    before = flat.clone()
    pos = torch.randint(0, 999, (T,), generator=g, device="cuda", dtype=torch.int32)
    q0, k0 = q.clone(), k.clone()
    pkv.pkv_rope(q, k, pos, pkv.RopeParams(D, layout=layout))
    f = R.freqs(D)
    check(q, q0, pos.cpu().numpy(), D, layout, f)
    check(k, k0, pos.cpu().numpy(), D, layout, f)
    mask = torch.ones_like(flat, dtype=torch.bool)
    mask[shift:].view(T, width)[:, :(Hq + Hk) * D] = False
    assert torch.equal(flat[mask], before[mask])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_transposed_is_the_gradient(layout):
    """Against the formula's gradient and against differences: y is linear in x, so the
    difference quotient of sum(w y) in direction d is exactly sum(d * turn^T(w)), up to the
    two sides' roundings (512 terms of magnitude ~1 with 2^-22 each)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w, d = (rows(g, 17, 4, 64, torch.float32) for _ in range(3))
    pos = torch.randint(0, 10000, (17,), generator=g, device="cuda", dtype=torch.int32)
    kw = dict(rotary_dim=48, layout=layout, scaling="linear", factor=2.0, attention_factor=1.1)
    fwd, bwd = pkv.RopeParams(64, **kw), pkv.RopeParams(64, transposed=True, **kw)
    grad = torch.empty_like(w)
    pkv.pkv_rope(w, None, pos, bwd, grad)
    m = float(np.float32(1.1))
    check(grad, w, pos.cpu().numpy(), 48, layout, R.freqs(48, scaling="linear", factor=2.0), m=m, transposed=True)
    ya, yb = torch.empty_like(x), torch.empty_like(x)
    pkv.pkv_rope(x + d, None, pos, fwd, ya)
    pkv.pkv_rope(x - d, None, pos, fwd, yb)
    diff = float(((ya.double() - yb.double()) / 2 * w.double()).sum())
    want = float((d.double() * grad.double()).sum())
    terms = float((d.abs().double() * grad.abs().double()).sum() + (w.abs().double() * (x.abs() + d.abs()).double()).sum() * 4)
    assert abs(diff - want) <= terms * 2.0 ** -21


def test_graph_other_stream_and_bound():
    g = torch.Generator(device="cuda").manual_seed(5)
    q = rows(g, 50, 9, 64, torch.float32)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    par = pkv.RopeParams(64)
    want = torch.empty_like(q)
    pkv.pkv_rope(q, None, pos, par, want)
    out = torch.zeros_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call = pkv.pkv_rope(q, None, pos, par, out, stream=st, bound=True)
    assert not out.any()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pkv.pkv_rope(q, None, pos, par, out)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_agrees_with_the_fused_step_rotation():
    """The half layout over the whole head is what pkv_decode_step turns by: its stored key
    row (float cache) against this call's, within both roundings (each at most
    2 |x| 2^-22 from the definition)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = pkv.KVCache.allocate(4, 2, 64, pkv.F32)
    q, k, v = rows(g, 1, 4, 64, torch.float32), rows(g, 1, 2, 64, torch.float32), rows(g, 1, 2, 64, torch.float32)
    slot, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 777, dtype=torch.int32, device="cuda")
    bt, lens = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.empty(1, 4, 64, device="cuda")
    pkv.pkv_decode_step(cache, q, k, v, slot, pos, 10000.0, bt, lens, 0.125, out)
    turned = torch.empty_like(k)
    pkv.pkv_rope(k, None, pos, pkv.RopeParams(64), turned)
    err = (cache.k[0, :, 0] - turned[0]).abs().max().item()
    assert err <= 4 * k.abs().max().item() * 2.0 ** -22 * 2

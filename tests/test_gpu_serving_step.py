"""A serving loop as a user writes it: each step's tables from the lengths, rotary positions,
append into a paged cache, attention, for prompt chunks and single tokens, requests that end
and requests that take over their pages.  Everything is compared with dense attention in 64
bits over the keys and values that each request was given (rotated in 64 bits, and coded as
the cache codes them)."""
import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import pkv

pytestmark = pytest.mark.gpu

HQ, HKV, D, MB, N = 6, 2, 64, 12, 40


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    def __init__(self, kind, B, layout, seed):
        self.kind, self.B = kind, B
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = pkv.PagePool.allocate(N)
        self.cache = pkv.KVCache.allocate(N, HKV, D, kind)
        self.bt = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cached = [0] * B
        self.rope = dict(rotary_dim=48, layout=layout, scaling="bands", factor=4.0, original_len=64)
        self.params = pkv.RopeParams(D, **self.rope)
        self.f = R.freqs(48, scaling="bands", factor=4.0, original_len=64)
        self.layout = layout
        # what each request was given: rotated keys and values, float64, and their runs
        self.keys = [np.zeros((0, HKV, D)) for _ in range(B)]
        self.values = [np.zeros((0, HKV, D)) for _ in range(B)]
        self.runs = [[] for _ in range(B)]

    def step(self, new, pad=3):
        B, T = self.B, sum(max(n, 0) for n in new)
        context, starts = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda")
        pos, slots = torch.empty(T + pad, dtype=torch.int32, device="cuda"), torch.empty(T + pad, dtype=torch.int32, device="cuda")
        cached = i32(self.cached)
        pkv.pkv_batch_tables(self.pool, cached, i32(new), self.bt, context, starts, pos, slots, self.status)
        rows = torch.randn(T + pad, HQ + 2 * HKV, D, generator=self.g, device="cuda")
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]
        k0, q0 = k.double().cpu().numpy(), q.double().cpu().numpy()
        qr, kr = torch.zeros(T + pad, HQ, D, device="cuda"), torch.zeros(T + pad, HKV, D, device="cuda")
        pkv.pkv_rope(q, k, pos, self.params, qr, kr)
        pkv.pkv_append(self.cache, kr, v.contiguous(), slots, self.status)
        out = torch.full((T + pad, HQ, D), 7.0, device="cuda")
        top = max(new)
        if top == 1 and all(n == 1 for n in new):
            n = pkv.pkv_decode_workspace_size(self.cache, B, HQ, MB)
            pkv.pkv_decode_attn(self.cache, qr[:B], self.bt, context, D ** -0.5, out, pkv.workspace_for(n), self.status)
        else:
            n = pkv.pkv_prefill_workspace_size(self.cache, B, HQ, top, MB)
            pkv.pkv_prefill_chunk_attn(self.cache, qr, starts, top, self.bt, context, D ** -0.5, out, pkv.workspace_for(n),
                                       self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        assert (out[T:] == 7).all()
        # the definition
        at = 0
        vr = v.double().cpu().numpy()
        want = np.zeros((T, HQ, D))
        for b in range(B):
            if new[b] < 0:
                self.cached[b], self.runs[b] = 0, []
                self.keys[b] = self.values[b] = np.zeros((0, HKV, D))
                continue
            n, c = new[b], self.cached[b]
            p = np.arange(c, c + n)
            krow = R.rope(k0[at:at + n], p, 48, self.layout, self.f)
            qrow = R.rope(q0[at:at + n], p, 48, self.layout, self.f)
            self.keys[b] = np.concatenate([self.keys[b], krow])
            self.values[b] = np.concatenate([self.values[b], vr[at:at + n]])
            for h in range(HQ):
                g = h // (HQ // HKV)
                for i in range(n):
                    want[at + i, h] = R.attend(qrow[i, h], self.keys[b][:, g], self.values[b][:, g], D ** -0.5, 0, c + i)
            at += n
            self.cached[b] = c + n
        return out[:T].double().cpu().numpy(), want


def tolerance(kind):
    """Attention over coded keys and values against the uncoded ones.  With a value error of at
    most e_v and a score error of at most e_s (in natural units) the output moves by at most
    e_v + (exp(2 e_s) - 1) max|v|; e_s = sum|q||k's error| / 8 at random over 64 columns.  Blocks
    reach |x| = 5: INT8B errs by half a step a coding, 5 / 127 / 2 = 0.02, at most twice that
    after growths; FP8B by 2^-4 of a value, 0.04 rms of which is a quarter of the step; BF16 2^-8.
    Scores then move by about |q| e sqrt(64) / 8 = |q| e.  The bounds are those, with |q| = 2.5
    and max|v| = 5 averaged over at least the few keys that a row sees."""
    return {pkv.BF16: 0.15, pkv.INT8B: 0.35, pkv.FP8B: 1.2, pkv.F32: 1e-4}[kind]


@pytest.mark.parametrize("kind", [pkv.BF16, pkv.INT8B, pkv.FP8B], ids=["bf16", "int8b", "fp8b"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_serving_loop(kind, layout):
    loop = Loop(kind, 4, layout, 5)
    steps = [[37, 5, 1, 64], [1, 1, 1, 1], [1, 20, 1, 1], [1, 1, 1, 1], [-1, 1, 30, 1], [50, 1, 1, -1], [1, 1, 1, 40],
             [1, 1, 1, 1]]
    used, most = set(), 0
    for i, new in enumerate(steps):
        got, want = loop.step(new)
        err = np.abs(got - want).max()
        assert err <= tolerance(kind), (i, err)
        rms = np.sqrt(((got - want) ** 2).mean())
        assert rms <= tolerance(kind) / 8, (i, rms)
        count = int(loop.pool.state[1].item())
        held = sum(R.pages(c) for c in loop.cached)
        assert count == N - held
        most = max(most, held)
        used |= set(loop.bt[loop.bt >= 0].tolist())
    assert len(used) > most  # returned pages wait behind the free ones


def test_serving_loop_float_decode():
    """Float keys and values: single tokens only (prefill takes BF16 and block-scaled caches),
    at the tolerance of the float attention."""
    loop = Loop(pkv.F32, 3, "half", 6)
    for _ in range(40):
        got, want = loop.step([1, 1, 1])
        assert np.abs(got - want).max() <= tolerance(pkv.F32)

"""The block-scaled prefill kernel's waits, when they give up: the call reports
PKV_DEV_TIMEOUT with NaN rows, every copy and product in flight is drained, and the next
call on the same buffers and workspace is exact.  As for the other kernels, a test build of
the library (PKV_TEST_HOOKS, never the product library) lets the softmax threads' first wait
for scores give up at once; the other roles' waits run out on their own limits."""
import ctypes
import os

import numpy as np
import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import _build, pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks(tmp_path_factory):
    d = tmp_path_factory.mktemp("hooks")
    path = _build.build(defines=["-DPKV_TEST_HOOKS"], lib=os.path.join(str(d), "libpkv_hooks.so"),
                        obj=os.path.join(str(d), "obj"))
    lib = pkv.bind(path)
    lib.pkv_test_prefill_blk_fail_first_wait.argtypes = [ctypes.c_int]
    lib.pkv_test_prefill_blk_fail_first_wait.restype = ctypes.c_int
    yield lib
    lib.pkv_test_prefill_blk_fail_first_wait(0)


@pytest.mark.parametrize("fp8,dtype,key_split", [(True, torch.bfloat16, 1), (False, torch.float32, 3)])
def test_wait_that_gives_up(hooks, fp8, dtype, key_split):
    rng = np.random.default_rng(20)
    n, chunk = 700, 40
    bc = R.BlockCache(R.pages(n), 1, 64, fp8)
    k, v = (rng.standard_normal((n, 1, 64)).astype(np.float32) for _ in range(2))
    bc.append(k, v, list(range(n)))
    table = np.arange(R.pages(n), dtype=np.int32)[None]
    q = torch.from_numpy(rng.standard_normal((chunk, 4, 64)).astype(np.float32)).to(dtype).cuda()
    want, _ = R.prefill(bc, q.float().cpu().numpy(), [0, chunk], table, [n], 0.125)
    cache = bc.device(pkv)
    bt = torch.from_numpy(table).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
    need = pkv.pkv_prefill_workspace_size(cache, 1, 4, chunk, bt.shape[1], key_split)
    ws = pkv.workspace_for(need)
    out = torch.empty(chunk, 4, 64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        status.zero_()
        out.fill_(7.0)
        c = cache.struct()
        opts = pkv.pkv_prefill_opts(key_split)
        rc = hooks.pkv_prefill_chunk_attn_ex(
            ctypes.byref(c), q.data_ptr(), pkv._CODE[dtype], 1, 4, starts.data_ptr(), chunk, bt.data_ptr(), bt.shape[1],
            lens.data_ptr(), 0.125, out.data_ptr(), None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * 4, ctypes.byref(opts), status.data_ptr(), None)
        assert rc == 0
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), int(status.item())
    good, s = call()
    assert s == 0 and np.abs(good - want).max() <= 1e-3  # (the product library's tests hold the tolerance)
    assert hooks.pkv_test_prefill_blk_fail_first_wait(1) == 0
    bad, s = call()
    assert s == pkv.DEV_TIMEOUT and np.isnan(bad).all()
    assert hooks.pkv_test_prefill_blk_fail_first_wait(0) == 0
    again, s = call()
    assert s == 0 and np.array_equal(again, good)


def test_product_library_has_no_hook():
    assert not hasattr(pkv.load(), "pkv_test_prefill_blk_fail_first_wait")

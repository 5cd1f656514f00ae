"""GPU tests of the decode step's operators where a wait runs out: the copies
that a kernel waits for are left out (test hook), the limit is short, the call
ends with the error status and the next one is right again.  The workspace is
filled with bytes that name no place in it, as an uninitialised one may be."""

import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

ROW_WORKERS, PREFIX = 1, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(mattn.LIB_PATH):
        from block_sparse_attention_masked_gb300 import build

        build.build()
    mattn.lib()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _times_out(run, workspace, what):
    """run() with the hook set; then without: the results of a call before."""
    hook = mattn.lib().mattn_internal_decode_wait_selftest
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    assert mattn.device_status()[0] == 0
    for fill in (0x7F, 0xFF, 0x55):
        workspace.fill_(fill)
        mattn.set_wait_timeout_ns(50_000_000)  # 50 ms
        assert hook(what) == 0
        try:
            run()
            torch.cuda.synchronize()
            rc, word = mattn.device_status()
        finally:
            hook(0)
            mattn.set_wait_timeout_ns(0)
        assert rc == mattn.ERR_TIMEOUT, hex(word)
        workspace.fill_(fill)
        for a, b in zip(run(), want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        rc, word = mattn.device_status()
        assert rc == 0, hex(word)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("P,what", [(0, ROW_WORKERS), (300, ROW_WORKERS), (300, PREFIX)])
@pytest.mark.parametrize("B", [3, 70])
def test_shared_prefix_waits_run_out(d, P, what, B):
    H, Hkv, L = 8, 2, 90
    x = _randn(1, B, H, d), _randn(2, Hkv, P, d), _randn(3, Hkv, P, d), _randn(4, B, Hkv, L, d), _randn(5, B, Hkv, L, d)
    lens = torch.arange(B, dtype=torch.int32, device="cuda") % (L + 1)
    ws = mattn.decode_shared_workspace(B, H, Hkv, P, L, d)
    _times_out(lambda: mattn.decode_shared(*x, seq_lens=lens, workspace=ws), ws, what)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("top_k", [5, 1100])
def test_block_list_waits_run_out(d, top_k):
    """Clusters (short lists) and equal shares with the merge (long ones)."""
    B, H, Hkv, L, block = 3, 8, 2, 200, 16
    q, k, v = _randn(1, B, H, d), _randn(2, B, Hkv, L, d), _randn(3, B, Hkv, L, d)
    ids = torch.arange(top_k, dtype=torch.int32, device="cuda").expand(B, Hkv, top_k).contiguous()
    ws = mattn.decode_blocks_workspace(B, H, Hkv, top_k, block, d)
    _times_out(lambda: mattn.decode_blocks(q, k, v, ids, block, workspace=ws), ws, ROW_WORKERS)

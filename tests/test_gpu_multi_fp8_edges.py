"""Corners of pa_decode_multi_fp8 at which its two kernels (runs of few rows, runs
of many) have to say the same: bad blocks, a NaN scale."""
import numpy as np
import pytest
import torch

from test_gpu_multi_fp8 import (_clean_error_word, assert_close, batch, dequantised,  # noqa: F401
                                gpu_multi)

pytestmark = pytest.mark.gpu


def attend_64(b, s, bad=()):
    """The rows of sequence s in 64 bits over the keys that no bad block holds;
    zero for a row without keys."""
    k, v = (x.double().numpy() for x in dequantised(b))
    qs, L = b.meta["query_start"], int(b.seq_lens[s])
    n = qs[s + 1] - qs[s]
    H, Hkv = b.q.shape[1], b.num_kv_heads
    blocks = np.where(np.isin(np.arange((L + 15) // 16), bad), 0, b.block_tables[s, :(L + 15) // 16])
    held = ~np.isin(np.arange(L) // 16, bad)
    out = np.zeros((n, H, b.q.shape[2]))
    q = b.q[qs[s]:qs[s + 1]].double().cpu().numpy()
    for h in range(H):
        kh, vh = (x[blocks, h * Hkv // H].reshape(-1, x.shape[-1])[:L] for x in (k, v))
        for i in range(n):
            sees = held & (np.arange(L) <= L - n + i)
            if sees.any():
                x = b.scale * (kh[sees] @ q[i, h])
                w = np.exp(x - x.max())
                out[i, h] = w @ vh[sees] / w.sum()
    return out


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("n", [2, 8, 9, 50])       # 8, 32, 36 and 200 rows a KV head
@pytest.mark.parametrize("ctx,bad", [(100, [0]), (100, [3]), (150, [2, 3, 4, 5, 9]), (2000, [0, 7, 63, 64, 65])])
def test_bad_blocks_are_left_out(cuda_lib, ctx, bad, n, D, dtype):
    """The rows of a sequence with bad block ids attend over its other blocks."""
    b = batch(900 + ctx + n, num_seqs=3, min_ctx=ctx, max_ctx=ctx + 9, n_new=n, num_heads=8,
              num_kv_heads=2, head_dim=D, dtype=dtype)
    qs = b.meta["query_start"]
    good = gpu_multi(cuda_lib, b)
    for ids in (-5, b.num_blocks):
        bt = b.block_tables.copy()
        bt[1, bad] = ids
        out = gpu_multi(cuda_lib, b, block_tables=bt)
        assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_BLOCK_ID
        assert_close(out[qs[1]:qs[2]], attend_64(b, 1, bad), f"without {bad}")
        assert torch.equal(out[:qs[1]], good[:qs[1]]) and torch.equal(out[qs[2]:], good[qs[2]:])


@pytest.mark.parametrize("n", [8, 9, 50, 300])
def test_rows_that_see_bad_blocks_alone_are_zero(cuda_lib, n):
    """Nothing before the new tokens, and their first blocks bad."""
    b = batch(920 + n, num_seqs=2, min_ctx=0, max_ctx=0, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    bad = list(range((n + 31) // 32))
    bt = b.block_tables.copy()
    bt[:, bad] = b.num_blocks + 3
    out = gpu_multi(cuda_lib, b, block_tables=bt)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_BLOCK_ID
    qs = b.meta["query_start"]
    for s in range(2):
        assert (out[qs[s]:qs[s] + min(n, 16 * len(bad))] == 0).all()
        assert_close(out[qs[s]:qs[s + 1]], attend_64(b, s, bad), "no keys")


@pytest.mark.parametrize("n", [2, 50])
@pytest.mark.parametrize("ctx", [40, 3000])
def test_nan_key_scale(cuda_lib, ctx, n):
    """A KV head whose scale is NaN has NaN scores; the others keep their rows."""
    b = batch(930, num_seqs=2, min_ctx=ctx, max_ctx=ctx, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    good = gpu_multi(cuda_lib, b)
    b.meta["k_scale"] = b.meta["k_scale"].clone()
    b.meta["k_scale"][1] = float("nan")
    out = gpu_multi(cuda_lib, b)
    assert out[:, 4:].isnan().all() and torch.equal(out[:, :4], good[:, :4])

"""Corners of pa_decode_multi_fp8 at which its two kernels (runs of few rows, runs
of many) have to say the same: bad blocks, a NaN scale, weights that f16 rounds,
waits that run out."""
import math
import time

import numpy as np
import pytest
import torch

from test_gpu_multi_fp8 import (_clean_error_word, assert_close, batch, dequantised,  # noqa: F401
                                gpu_multi, oracle_multi)

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


def one_key_above(pa, S, L, n, D, v_first, v_rest, v_scales, B=1):
    """Every row's first key scores S above the others in log2, all others 0, over L
    keys and n tokens of 4 heads a KV head; the values are v_first and v_rest.  B
    sequences have the same blocks.  Returns the rows [B, n, Hkv, 4, D] in 64 bits
    and the number of other keys of each token."""
    Hkv, nb = len(v_scales), (L + 15) // 16
    code = lambda x: int(torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8))  # noqa: E731
    kc = torch.zeros(nb, Hkv, 16, D, dtype=torch.uint8, device="cuda")
    kc[0, :, 0, 0] = code(1.0)
    vc = torch.full((nb, Hkv, 16, D), code(v_rest), dtype=torch.uint8, device="cuda")
    vc[0, :, 0] = code(v_first)
    q = torch.zeros(B * n, 4 * Hkv, D, device="cuda", dtype=torch.float16)
    q[:, :, 0] = 1
    out = torch.full_like(q, float("nan"))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pa.pa_decode_multi_fp8(out, q, kc, vc, torch.ones(Hkv, device="cuda"),
                           torch.tensor(v_scales, dtype=torch.float32, device="cuda"),
                           torch.arange(nb, dtype=torch.int32, device="cuda")[None].repeat(B, 1),
                           i32([L] * B), i32([n * s for s in range(B + 1)]), n, S * math.log(2), Hkv)
    torch.cuda.synchronize()
    return out.double().cpu().numpy().reshape(B, n, Hkv, 4, D), (L - n + np.arange(n)).astype(float)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 8, 9, 100])
def test_equal_values_come_back_whatever_the_weights(cuda_lib, n, D):
    """All values of a head equal v: the result is v.  With S = -log2(0.50024) the
    other keys' weight lies just below the middle of two f16 numbers and loses
    4.8e-4 of itself in P, which the sum has to lose too.  What is left: the
    output's half step 2^-11 |v|, V's scale and the division (4 of 2^-24), and
    the accumulation of 4000 keys sixteen at a time, 2^-23 each."""
    vs = np.float32(1 + 1.2e-4 * np.arange(8))
    out, _ = one_key_above(cuda_lib, -math.log2(0.50024), 4000, n, D, 1.0, 1.0, vs.tolist())
    v = vs.astype(float)[None, :, None, None]
    assert (np.abs(out - v) <= v * (2.0**-11 + 4 * 2.0**-24 + 4000 / 16 * 2.0**-23)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n", [(1, 2), (1, 8), (1, 9), (1, 100), (600, 2), (76, 64)])
@pytest.mark.parametrize("S", [24.9, 25.2, 27.0])
def test_one_key_above_a_long_tail(cuda_lib, S, B, n, D):
    """60000 keys 2^-S below one: together 1.9e-3 (S = 24.9) to 4.5e-4 of its weight,
    in few pieces (many sequences) or many.  The result is v (1 - x) / (1 + x), x
    the tail's share, for values v and -v.  Allowed: the output's half step 2^-11,
    the accumulation of the keys sixteen at a time (2^-23 each), a tail off by
    half of a 16th (its weights are f16 numbers of four bits at the least), which
    moves the result by 2 x / 32.

    Where S > 25 the tail may be missing from the products' sum: that is kept in
    binary32 with the first key's weight in it, 1 + 2^-S is 1 there (the last bit
    of 1 is 2^-23, half of it 2^-24), and the matrix instructions align every
    product to the sum on its own.  (1 - x) / (1 + x) becomes 1 / (1 + x): x more."""
    L = 60000
    out, others = one_key_above(cuda_lib, S, L, n, D, 1.0, -1.0, [1.0, 0.5], B)
    x = others * 2.0**-S
    want = ((1 - x) / (1 + x))[:, None, None, None] * np.array([1.0, 0.5])[None, :, None, None]
    tol = 2.0**-11 + L / 16 * 2.0**-23 + 2 * x.max() / 32 + (x.max() if S > 25 else 0)
    assert (np.abs(out - want) <= tol * np.abs(want)).all(), np.abs(out / want - 1).max()


@pytest.mark.parametrize("seqs,n", [(38, 64), (15, 64), (1, 64), (1, 3)])
def test_long_runs_that_wait_too_long(cuda_lib, seqs, n):
    """Keys that never arrive, for runs of many rows in items of one, two and four
    blocks: the call ends with PA_DEVERR_TIMEOUT, and the next one is right."""
    b = batch(940 + seqs, num_seqs=seqs, min_ctx=100, max_ctx=700, n_new=n, num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="bf16")
    ref = oracle_multi(b)
    assert_close(gpu_multi(cuda_lib, b), ref, "before")
    t0 = time.perf_counter()
    cuda_lib.pa_test_stall_next_decode()
    gpu_multi(cuda_lib, b)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_TIMEOUT
    assert time.perf_counter() - t0 < 30
    assert_close(gpu_multi(cuda_lib, b), ref, "after the timeout")

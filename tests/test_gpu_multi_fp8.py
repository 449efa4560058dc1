"""Multi-token queries over an E4M3 cache (pa_decode_multi_fp8) against the fp64
oracle's causal attention over the dequantised cache.

Tolerances as for the 16-bit paths: max |err| <= 2e-2 and relative L2 error <=
5e-3.  The codes convert exactly to f16, so what is rounded is P (f16, half a
step 2^-11, weights that the running sum holds too) and the output (bf16 half
a step 2^-8: for values spread evenly over a binade that is 2^-8 / sqrt(3) of
the value at most, 2.3e-3 relative L2; f16 2^-11)."""
import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from paged_kv_cache_151_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

TOL_ABS = 2e-2
TOL_REL_L2 = 5e-3


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


def assert_close(gpu, ref, what=""):
    g = gpu.detach().double().cpu().numpy()
    assert g.shape == ref.shape, (g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    if not g.size:
        return
    err = np.abs(g - ref).max()
    rel = np.linalg.norm(g - ref) / max(np.linalg.norm(ref), 1e-30)
    assert err <= TOL_ABS, f"{what}: max abs err {err:.3g}"
    assert rel <= TOL_REL_L2, f"{what}: rel L2 err {rel:.3g}"


def batch(seed, **kw):
    b = wl.multi_query_batch(seed, device="cuda", keep_seq=False, **kw)
    return wl.with_fp8_pool(b, seed=seed)


def gpu_multi(pa, b, max_query_len=None, k_cache=None, v_cache=None, seq_lens=None,
              block_tables=None, query_start=None, out=None, q=None, stream=None):
    qs = b.meta["query_start"] if query_start is None else query_start
    mq = int(np.diff(qs).max()) if max_query_len is None else max_query_len
    as_t = lambda x: torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    q = b.q if q is None else q
    out = torch.full(q.shape, float("nan"), device="cuda", dtype=q.dtype) if out is None else out
    torch.cuda.synchronize()
    pa.pa_decode_multi_fp8(out, q, b.k_cache if k_cache is None else k_cache,
                           b.v_cache if v_cache is None else v_cache, b.meta["k_scale"],
                           b.meta["v_scale"],
                           as_t(b.block_tables if block_tables is None else block_tables),
                           as_t(b.seq_lens if seq_lens is None else seq_lens), as_t(qs), mq,
                           b.scale, b.num_kv_heads, stream=stream)
    torch.cuda.synchronize()
    return out


def dequantised(b):
    v = [torch.from_numpy(po.e4m3_values(c.cpu().numpy()).astype(np.float32))
         * b.meta[s].cpu()[None, :, None, None]
         for c, s in ((b.k_cache, "k_scale"), (b.v_cache, "v_scale"))]
    return [torch.nan_to_num(x, nan=0.0) for x in v]   # canaries of rows that no token holds


def oracle_multi(b, seq_lens=None, query_start=None):
    k, v = dequantised(b)
    return oracle.decode_multi(b.q.float().cpu(), k, v, b.block_tables,
                               b.seq_lens if seq_lens is None else seq_lens,
                               b.meta["query_start"] if query_start is None else query_start,
                               b.scale, b.num_kv_heads, "f32")


CASES = [(dtype, D, G, Hkv) for dtype in ("bf16", "f16") for D in (64, 128)
         for G, Hkv in ((1, 4), (2, 2), (4, 2), (8, 1))]
IDS = [f"{c[0]}-d{c[1]}-g{c[2]}" for c in CASES]


@pytest.mark.parametrize("dtype,D,G,Hkv", CASES, ids=IDS)
def test_short_runs(cuda_lib, dtype, D, G, Hkv):
    """1..7 new tokens over 0..300 cached ones: every row of a 16-row tile, its
    ragged tail, and several tiles."""
    b = batch(600 + D + G, num_seqs=11, min_ctx=0, max_ctx=300, n_new=(1, 7), num_heads=G * Hkv,
              num_kv_heads=Hkv, head_dim=D, dtype=dtype)
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"{dtype} d{D} g{G}")


@pytest.mark.parametrize("dtype,D,G,Hkv", CASES, ids=IDS)
def test_chunks(cuda_lib, dtype, D, G, Hkv):
    """Prompt chunks of odd lengths beside short runs, one of them with nothing
    before it."""
    b = batch(620 + D + G, num_seqs=6, min_ctx=0, max_ctx=400, n_new=[200, 1, 77, 3, 131, 64],
              num_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D, dtype=dtype)
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"chunks {dtype} d{D} g{G}")


@pytest.mark.parametrize("G", [1, 4, 8])
def test_whole_sequence_is_new(cuda_lib, G):
    """Row i sees positions 0..i; the first row returns its own value."""
    Hkv = 2
    b = batch(640 + G, num_seqs=5, min_ctx=0, max_ctx=0, n_new=(1, 150), num_heads=G * Hkv,
              num_kv_heads=Hkv, head_dim=128, dtype="bf16")
    out = gpu_multi(cuda_lib, b)
    assert_close(out, oracle_multi(b), f"prefill g{G}")
    qs, v = b.meta["query_start"], dequantised(b)[1]
    for s in range(b.num_seqs):
        v0 = v[int(b.block_tables[s, 0]), :, 0].repeat_interleave(G, dim=0)
        # one weight of 1: the output's rounding and V's scale product (2^-24)
        assert (out[qs[s]].float().cpu() - v0).abs().le(2.0 ** -8 * v0.abs() * 1.0001).all()


def test_every_length_remainder(cuda_lib):
    """Contexts 0..79 with chunks and runs: blocks that end inside a tile, steps
    that end inside a block."""
    n = [(37 * i) % 90 + 1 for i in range(80)]
    b = batch(650, num_seqs=80, min_ctx=0, max_ctx=79, n_new=n, num_heads=4, num_kv_heads=1,
              head_dim=128, dtype="bf16")
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "remainders")


def test_one_token_matches_decode(cuda_lib):
    b = batch(660, num_seqs=40, min_ctx=0, max_ctx=600, n_new=1, num_heads=32, num_kv_heads=8,
              head_dim=128, dtype="bf16")
    ref = oracle_multi(b)
    assert_close(gpu_multi(cuda_lib, b), ref, "multi")
    out = torch.empty_like(b.q)
    bt, sl, _ = b.torch_tables("cuda")
    cuda_lib.pa_decode_fp8(out, b.q, b.k_cache, b.v_cache, b.meta["k_scale"], b.meta["v_scale"],
                           bt, sl, b.scale, b.num_kv_heads)
    torch.cuda.synchronize()
    assert_close(out, ref, "decode")


@pytest.mark.parametrize("ctx,n", [(9000, 4), (6000, 300), (20000, 1)])
def test_long_contexts(cuda_lib, ctx, n):
    b = batch(670 + n, num_seqs=2, min_ctx=ctx, max_ctx=ctx + 33, n_new=n, num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="bf16")
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"ctx {ctx} n {n}")


@pytest.mark.parametrize("n", [(1, 4), (40, 90)])
def test_block_permutation_bit_identical(cuda_lib, n):
    b = batch(680, num_seqs=9, min_ctx=0, max_ctx=500, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    p = wl.permute_blocks(b, seed=5)
    p.meta.update({k: b.meta[k] for k in ("query_start", "k_scale", "v_scale")})
    assert torch.equal(gpu_multi(cuda_lib, b), gpu_multi(cuda_lib, p))


@pytest.mark.parametrize("n", [(1, 4), (40, 90)])
def test_nan_in_rows_that_no_token_holds(cuda_lib, n):
    """NaN codes in every row past a sequence's end and in every block that no
    table names, and padding entries in the tables: no output changes."""
    b = batch(690, num_seqs=7, min_ctx=0, max_ctx=200, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    used = np.zeros((b.num_blocks, 16), dtype=bool)
    for s, L in enumerate(b.seq_lens):
        pos = np.arange(L)
        used[b.block_tables[s][pos // 16], pos % 16] = True
    idle = torch.from_numpy(~used).cuda()
    out = []
    for fill in (0x00, 0x7F):
        kc, vc = b.k_cache.clone(), b.v_cache.clone()
        for c in (kc, vc):
            c.view(torch.uint8).transpose(1, 2)[idle] = fill
        out.append(gpu_multi(cuda_lib, b, k_cache=kc, v_cache=vc,
                             block_tables=wl.tables_with_padding(b, b.block_tables.shape[1] + 3)))
    assert torch.equal(out[0], out[1])
    assert_close(out[0], oracle_multi(b), "nan rows")


@pytest.mark.parametrize("n", [2, 50])
def test_rows_past_the_last_sequence_stay(cuda_lib, n):
    """Sequences without rows, rows behind the last sequence: left as they were."""
    b = batch(700, num_seqs=5, min_ctx=3, max_ctx=100, n_new=[n, 0, n, 0, 1], num_heads=8,
              num_kv_heads=2, head_dim=64, dtype="bf16")
    rows = b.q.shape[0]
    q = torch.cat([b.q, torch.randn(6, 8, 64, device="cuda").bfloat16()])
    out = torch.full(q.shape, 3.5, device="cuda", dtype=torch.bfloat16)
    gpu_multi(cuda_lib, b, q=q, out=out)
    assert (out[rows:] == 3.5).all()
    assert_close(out[:rows], oracle_multi(b), "rows")


@pytest.mark.parametrize("n", [3, 60])
def test_strided_queries(cuda_lib, n):
    b = batch(710, num_seqs=4, min_ctx=3, max_ctx=100, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="f16")
    wide = torch.zeros(b.q.shape[0], 12, 128, device="cuda", dtype=torch.float16)
    wide[:, :8] = b.q
    assert torch.equal(gpu_multi(cuda_lib, b, q=wide[:, :8],
                                 out=torch.empty_like(b.q)), gpu_multi(cuda_lib, b))


@pytest.mark.parametrize("n", [2, 50])
def test_bad_ranges_are_skipped_and_flagged(cuda_lib, n):
    b = batch(720, num_seqs=4, min_ctx=60, max_ctx=100, n_new=n, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    good = gpu_multi(cuda_lib, b)
    qs = b.meta["query_start"]
    sl = b.seq_lens.copy()
    sl[1] = n - 1                                  # fewer tokens than rows
    out = gpu_multi(cuda_lib, b, seq_lens=sl)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN
    assert out[qs[1]:qs[2]].isnan().all()
    # the rows of the others, whatever the split of their work
    assert_close(out[qs[2]:], good[qs[2]:].double().cpu().numpy(), "others")
    bt = b.block_tables.copy()
    bt[2, 0] = b.num_blocks + 7
    out = gpu_multi(cuda_lib, b, block_tables=bt)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_BLOCK_ID
    assert_close(out[qs[3]:], good[qs[3]:].double().cpu().numpy(), "others")
    gpu_multi(cuda_lib, b, max_query_len=n - 1)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN


def test_more_sequences_than_one_sort(cuda_lib):
    b = batch(730, num_seqs=4200, min_ctx=0, max_ctx=30, n_new=[(i % 3) + (60 if i % 700 == 5 else 0)
                                                                for i in range(4200)],
              num_heads=4, num_kv_heads=1, head_dim=128, dtype="bf16")
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "4200 sequences")


def test_large_scores(cuda_lib):
    """Scores of some hundred: one key takes nearly all the weight."""
    b = batch(740, num_seqs=3, min_ctx=100, max_ctx=300, n_new=[3, 70, 130], num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="bf16")
    b.q.mul_(60)
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "large scores")


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scale_zero_and_negative(cuda_lib, scale):
    """A scale of 0 is the mean of the visible values; a negative one turns the
    scores round."""
    b = batch(760, num_seqs=4, min_ctx=10, max_ctx=200, n_new=[3, 70, 300, 1], num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="bf16")
    b.scale = scale
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"scale {scale}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [31, 32, 33, 127, 128, 129, 255, 256, 257])
def test_rows_around_the_tiles(cuda_lib, D, rows):
    """One query head per KV head, so a token is a row: the sizes at which a run
    changes kernel, tile and item, over a context that several blocks share."""
    b = batch(770 + rows, num_seqs=2, min_ctx=1000, max_ctx=1100, n_new=[rows, rows + 1],
              num_heads=2, num_kv_heads=2, head_dim=D, dtype="bf16")
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"rows {rows}")


@pytest.mark.parametrize("seqs,n", [(1, 64), (3, 200), (20, 300), (60, 100)])
def test_items_shared_by_none_two_and_four_blocks(cuda_lib, seqs, n):
    """Few items to many; contexts of less than one step a block too."""
    b = batch(780 + seqs, num_seqs=seqs, min_ctx=0, max_ctx=700, n_new=n, num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="f16")
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), f"{seqs} x {n}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", [50, 52])
def test_items_without_steps_for_some_blocks(cuda_lib, seqs, D):
    """Around a hundred items of one or two steps, shared by four blocks: most
    blocks have no step of most items, several items in a row."""
    b = batch(785 + seqs, num_seqs=seqs, min_ctx=0, max_ctx=70, n_new=(9, 16), num_heads=8,
              num_kv_heads=2, head_dim=D, dtype="bf16")
    ref = oracle_multi(b)
    for _ in range(20):
        assert_close(gpu_multi(cuda_lib, b), ref, f"{seqs} short items")


@pytest.mark.parametrize("n", [4, 100])
@pytest.mark.parametrize("ctx", [50, 3000])
def test_nan_keys(cuda_lib, n, ctx):
    """A NaN key makes the rows that see it NaN, whatever blocks or warps share
    their keys, and no row before it."""
    b = batch(790, num_seqs=1, min_ctx=ctx, max_ctx=ctx, n_new=n, num_heads=4, num_kv_heads=1,
              head_dim=128, dtype="bf16")
    ref = gpu_multi(cuda_lib, b)
    L = int(b.seq_lens[0])
    for at, rows in ((L - 1, n - 1), (L - 2, n - 2), (7, 0)):      # position, first row that sees it
        kc = b.k_cache.clone()
        kc[int(b.block_tables[0, at // 16]), :, at % 16] = 0x7F
        out = gpu_multi(cuda_lib, b, k_cache=kc)
        assert torch.equal(out[:rows], ref[:rows]) and out[rows:].isnan().all()
    kc = torch.full_like(b.k_cache, 0x7F)          # nothing but NaN
    assert gpu_multi(cuda_lib, b, k_cache=kc).isnan().all()


@pytest.mark.parametrize("n", [4, 90])
def test_many_blocks_past_32_bits_of_cache(cuda_lib, n):
    """A pool of more than 2^31 codes: the blocks used lie at its end."""
    b = batch(800, num_seqs=2, min_ctx=100, max_ctx=300, n_new=n, num_heads=8, num_kv_heads=8,
              head_dim=128, dtype="bf16")
    N = 135_000                                    # x 8 x 16 x 128 codes = 2.2e9 each
    out = gpu_multi(cuda_lib, b)
    shift = N - b.num_blocks
    big = [torch.empty(N, 8, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for dst, src in zip(big, (b.k_cache, b.v_cache)):
        dst[shift:] = src
    tables = np.where(b.block_tables < b.num_blocks, b.block_tables + shift, b.block_tables)
    assert torch.equal(gpu_multi(cuda_lib, b, k_cache=big[0], v_cache=big[1],
                                 block_tables=tables), out)


def test_wait_that_runs_out(cuda_lib):
    """A copy that never completes: the call ends with PA_DEVERR_TIMEOUT, and
    the next one is right."""
    b = batch(810, num_seqs=8, min_ctx=100, max_ctx=300, n_new=4, num_heads=8, num_kv_heads=2,
              head_dim=128, dtype="bf16")
    cuda_lib.pa_test_stall_next_decode()
    gpu_multi(cuda_lib, b)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_TIMEOUT
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "after the timeout")


def test_on_another_stream(cuda_lib):
    b = batch(750, num_seqs=5, min_ctx=0, max_ctx=300, n_new=(1, 90), num_heads=8,
              num_kv_heads=2, head_dim=128, dtype="bf16")
    assert torch.equal(gpu_multi(cuda_lib, b, stream=torch.cuda.Stream()), gpu_multi(cuda_lib, b))


@pytest.mark.slow
def test_spec_verify_fp8_full(cuda_lib):
    """256 sequences of the serving mix's lengths, four rows each."""
    b = wl.with_fp8_pool(wl.spec_verify(device="cuda"), seed=3)
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "spec_verify")


@pytest.mark.slow
def test_chunked_prefill_mix_fp8_full(cuda_lib):
    b = wl.with_fp8_pool(wl.chunked_prefill_mix(device="cuda"), seed=4)
    assert_close(gpu_multi(cuda_lib, b), oracle_multi(b), "chunked_prefill_mix")

"""Verification of drafted tokens (pa_verify_drafts) against the 64-bit form of
plain_ops.py: every output is a whole number and has to be equal."""
import numpy as np
import pytest
import torch

import plain_ops as po
from paged_kv_cache_151_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


def gpu_verify(pa, target, draft, tokens, au, su, qs, width=None):
    B = len(qs) - 1
    width = int(np.diff(qs).max()) if width is None else width
    out = torch.full((B, width), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    as_t = lambda x, dt: torch.as_tensor(np.ascontiguousarray(x), dtype=dt, device="cuda")  # noqa: E731
    pa.pa_verify_drafts(out, acc, target, draft, as_t(tokens, torch.int32),
                        as_t(au, torch.float32), as_t(su, torch.float32),
                        as_t(qs, torch.int32), width)
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy()


def check(pa, target, draft, tokens, au, su, qs, width=None):
    width = int(np.diff(qs).max()) if width is None else width
    got = gpu_verify(pa, target, draft, tokens, au, su, qs, width)
    want = po.verify(target.float().cpu().numpy(),
                     None if draft is None else draft.float().cpu().numpy(),
                     np.asarray(tokens), np.float32(au), np.float32(su), qs, width)
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])
    return want


def inputs(seed, n, V, dtype="f32", blur=0.8, pad=0):
    """n[s] rows per sequence; a draft model near the target, rows V + pad apart."""
    r = np.random.default_rng(seed)
    rows = int(np.sum(n))
    logits = 3 * r.standard_normal((rows, V))
    soft = lambda x: np.exp(x - x.max(1, keepdims=True)) / np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)  # noqa: E731
    behind = np.roll(logits, 1, 0) + blur * r.standard_normal((rows, V))
    tokens = (behind + r.gumbel(size=(rows, V))).argmax(1).astype(np.int32)

    def on_gpu(p):
        wide = torch.full((rows, V + pad), 9.0, dtype=wl.DTYPES[dtype], device="cuda")
        wide[:, :V] = torch.from_numpy(p).cuda().to(wl.DTYPES[dtype])
        return wide[:, :V]
    return (on_gpu(soft(logits)), on_gpu(soft(behind)), tokens, r.random(rows, dtype=np.float32),
            r.random(len(n), dtype=np.float32), np.concatenate([[0], np.cumsum(n)]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099, 50021])
def test_verify_sizes(cuda_lib, V, dtype):
    n = np.random.default_rng(V).integers(0, 9, 12)
    n[0] = 1                                       # no drafts at all
    t, d, tok, au, su, qs = inputs(V, n, V, dtype)
    check(cuda_lib, t, d, tok, au, su, qs)
    check(cuda_lib, t, None, tok, au, su, qs, width=11)


@pytest.mark.parametrize("B", [1, 3, 40, 160, 700])
def test_verify_batches(cuda_lib, B):
    """Every cluster size, each with accepted, rejected and bonus tokens."""
    t, d, tok, au, su, qs = inputs(B, np.full(B, 4), 5003)
    out, acc = check(cuda_lib, t, d, tok, au, su, qs)
    if B >= 40:
        assert set(acc) == {0, 1, 2, 3}


def test_verify_many_drafts(cuda_lib):
    """More drafts than a warp's lanes, accepted far into the run."""
    t, d, tok, au, su, qs = inputs(5, [100, 1, 65, 33, 34], 300, blur=0.0)
    au[:] = 0.0
    au[qs[0] + 70] = 1.0
    d = t.roll(1, 0)
    tok = d.argmax(1).cpu().numpy().astype(np.int32)
    out, acc = check(cuda_lib, t, d.contiguous(), tok, au, su, qs)
    assert acc.tolist()[1:] == [0, 64, 32, 33]


def test_verify_strided_rows(cuda_lib):
    t, d, tok, au, su, qs = inputs(6, [3, 2, 5], 1001, pad=6)
    assert t.stride(0) == 1007
    check(cuda_lib, t, d, tok, au, su, qs)
    t, d, tok, au, su, qs = inputs(6, [3, 2, 5], 1001, "bf16", pad=7)
    check(cuda_lib, t, d, tok, au, su, qs)


@pytest.mark.parametrize("V", [64, 3000, 40000])
def test_verify_uniform_on_a_border(cuda_lib, V):
    """Weights that are multiples of 2^-20, so every sum is exact and u W falls on
    a border: the token behind it is drawn; u = 0 and 1 take the first and
    the last weight."""
    r = np.random.default_rng(V)
    w = np.zeros((9, V), dtype=np.float64)
    k = 2**16                                      # of 2^-16 each: W = 1
    for i in range(9):
        w[i] = np.bincount(r.integers(V // 8, V - V // 8, k), minlength=V) / k
    c = np.cumsum(w, 1)
    su = np.array([0.0, 1.0, 0.5, 2.0**-16, 1 - 2.0**-16, 0, 0, 0, 0])
    su[5:] = c[np.arange(5, 9), r.integers(V // 4, V // 2, 4)]
    t = torch.from_numpy(w).float().cuda()
    out, acc = check(cuda_lib, t, None, np.zeros(9), np.zeros(9), su, np.arange(10))
    assert out[0, 0] == np.flatnonzero(w[0])[0] and out[1, 0] == np.flatnonzero(w[1])[-1]


def test_verify_greedy_rows(cuda_lib):
    """One-hot targets: drafts are kept while they are the target's token, and the
    token after them is the target's."""
    V, qs = 777, np.array([0, 4, 8])
    best = np.array([5, 9, 700, 3, 1, 2, 776, 0])
    t = torch.zeros(8, V, device="cuda")
    t[torch.arange(8), torch.from_numpy(best).cuda()] = 1
    tok = np.array([50, 5, 9, 700, 50, 1, 3, 0])   # the second sequence's second draft is wrong
    for d in (None, torch.roll(t, 1, 0).contiguous()):
        out, acc = check(cuda_lib, t, d, tok, np.full(8, 0.999), [0.3, 0.9], qs)
        assert acc.tolist() == [3, 1]
        assert out.tolist() == [[5, 9, 700, 3], [1, 2, -1, -1]]


def test_verify_nothing_left_and_odd_entries(cuda_lib):
    """p == q with a draft of probability 0: nothing is left, the target's row
    is drawn from.  NaN, negative and infinite entries, a row without weight,
    uniforms outside [0, 1] and NaN."""
    t, d, tok, au, su, qs = inputs(8, [2] * 12, 500)
    d = torch.roll(t, 1, 0).contiguous()
    nan, inf = float("nan"), float("inf")
    t[0, 7] = d[1, 7] = 0
    tok[1] = 7                                     # 0: nothing left
    t[2, 5:90] = nan
    tok[3], au[3] = 6, 0.0                         # 1: a NaN token is rejected
    t[4, 3:480] = -0.25
    d[5, 100:] = nan                               # 2
    t[6] = 0                                       # 3: no weight in the first row
    t[8] = nan                                     # 4
    t[10, 11] = inf
    tok[11] = 11                                   # 5: an infinite token is rejected
    d[13, 20] = inf
    au[13] = 1.0                                   # 6
    su[7], su[8], su[9] = -3.0, nan, 2.5
    t[22, :-1] = 0
    out, acc = check(cuda_lib, t, d, tok, au, su, qs)
    assert out[3, 0] == -1 and out[4, 0] == -1 and acc[1] == 0 and acc[5] == 0


def test_verify_bad_token_and_rows(cuda_lib):
    t, d, tok, au, su, qs = inputs(9, [3, 3, 3, 3], 400)
    tok[1], tok[4], tok[8] = 400, -1, 2**31 - 1
    tok[2] = 10**9                                 # behind a rejection: not looked at
    au[:] = 0.0
    t[6:8] = d[7:9] = 1 / 400
    for dr in (d, None):
        out, acc = check(cuda_lib, t, dr, tok, au, su, qs)
        assert acc.tolist()[:3] == [0, 0, 1]
        assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_TOKEN
    tok[:] = 3
    bad = np.array([0, 3, 2, 99, 12])              # decreasing, past the rows, negative length
    out, acc = check(cuda_lib, t, d, tok, au, su, bad, width=3)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN
    assert (out[1:] == -1).all()
    out, acc = check(cuda_lib, t, d, tok, au, su, qs, width=2)    # longer than the width
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN
    assert (out == -1).all() and (acc == 0).all()


def test_verify_no_rows(cuda_lib):
    t, d, tok, au, su, qs = inputs(10, [1, 2], 50)
    out, acc = gpu_verify(cuda_lib, t[:0], None, tok[:0], au[:0], su, np.array([0, 0, 0]), 3)
    assert (out == -1).all() and (acc == 0).all()


def test_verify_row_offsets_past_32_bits(cuda_lib):
    """Rows more than 2^31 elements into the probabilities (8.6 GB)."""
    V, rows = 131071, 16400
    t = torch.zeros(rows, V, device="cuda")
    t[-1, 100_000] = 0.5
    t[-1, 7] = 0.25
    t[-2, 42] = 1.0
    tok = np.zeros(rows, dtype=np.int32)
    tok[-1] = 42
    out, acc = gpu_verify(cuda_lib, t, None, tok, np.full(rows, 0.5), [0.9],
                          np.array([rows - 2, rows]))
    assert acc.tolist() == [1] and out.tolist() == [[42, 100_000]]


def test_verify_same_answer_every_time(cuda_lib):
    t, d, tok, au, su, qs = inputs(11, [4] * 30, 20011, "bf16")
    first = gpu_verify(cuda_lib, t, d, tok, au, su, qs)
    for _ in range(5):
        again = gpu_verify(cuda_lib, t, d, tok, au, su, qs)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])

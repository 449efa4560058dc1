"""Processed logits against a 64-bit form."""
import numpy as np
import pytest
import torch

import plain_serving as ps
from plain_ops import HALF, TINY

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def f32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.float32, device="cuda")


def packed(allow):
    T, V = allow.shape
    wide = np.zeros((T, -(-V // 32) * 32), np.uint8)
    wide[:, :V] = allow
    return np.packbits(wide, axis=1, bitorder="little").view(np.int32)


class Case:
    def __init__(self, seed, n, V, dtype="f32", out="f32", history=50, bias=6, masked=True,
                 penalties=True, probs=True, greedy=False, pad=2):
        r = np.random.default_rng(seed)
        B = len(n)
        self.starts = np.concatenate([[0], np.cumsum(n)])
        self.rows = int(self.starts[-1])
        T = self.rows + pad                            # rows behind the last sequence
        self.x = torch.from_numpy(4 * r.standard_normal((T, V)).astype(np.float32)).to(DT[dtype])
        self.dtype, self.out_t, self.probs, self.V, self.T = dtype, out, probs, V, T
        self.kw = dict(tokens=r.integers(0, V, T) // 3)
        if penalties:
            h = (V * r.random((B, history)) ** 3).astype(int)
            hl = r.integers(0, history + 1, B)
            self.kw.update(history=h, history_lens=hl, prompt_lens=(hl * r.random(B)).astype(int),
                           repetition=(1 + 0.5 * r.random(B)).astype(np.float32),
                           frequency=(0.4 * r.random(B)).astype(np.float32),
                           presence=r.random(B).astype(np.float32))
        self.bias = None
        if bias:
            self.bias = [[(int(r.integers(0, V)), np.float32(3 * r.standard_normal()))
                          for _ in range(r.integers(0, bias + 1))] for _ in range(B)]
            if B > 1:                                  # a token named three times
                self.bias[1] = [(V - 1, np.float32(b)) for b in (0.1, 1e3, -1e3)] + self.bias[1]
        self.allowed = None
        if masked:
            self.allowed = r.random((T, V)) < r.choice([0.02, 0.5, 1.0], T)[:, None]
            self.allowed[0] = False                    # a row that allows nothing
            self.x[:, 0] = float("nan")                # and NaN where nobody may look
            self.allowed[:, 0] = False
        self.tau = (0.4 + r.random(B)).astype(np.float32)
        if greedy:
            self.tau[::2] = 0

    def run(self, pa, out=None, x=None):
        x = self.x.cuda() if x is None else x
        out = torch.full((self.T, self.V), 5.0, dtype=DT[self.out_t], device="cuda") if out is None else out
        kw = {k: (f32 if v.dtype == np.float32 else i32)(v) for k, v in self.kw.items()}
        if self.bias is not None:
            kw["bias_start"] = i32(np.concatenate([[0], np.cumsum([len(b) for b in self.bias])]))
            kw["bias_tokens"] = i32([v for b in self.bias for v, _ in b])
            kw["bias_values"] = f32([y for b in self.bias for _, y in b])
        if self.allowed is not None:
            kw["allowed"] = torch.from_numpy(packed(self.allowed)).cuda()
        pa.pa_process_logits(out, x, i32(self.starts), temperature=f32(self.tau), probs=self.probs, **kw)
        return out

    def want(self):
        return ps.logits(self.x.float().numpy(), self.starts, bias=self.bias, allowed=self.allowed,
                         temperature=self.tau, probs=self.probs, **self.kw)

    def check(self, out):
        """With logits, the terms c, b and x of one element add up to what it may be
        off by in fp32: 12 roundings (three products or quotients with a rounded
        reciprocal, the sums) of the terms' sizes, here below S = 4096 in all (the
        biases of 1e3 among them), usually far below.  A probability is off by that
        much in its logarithm, for itself and the sum, by exp2 of a scaled argument
        (|x| < 2^7 log2 units: 2^-24 2^8) and by the sum (2^-20)."""
        ref = self.want()[:self.rows]
        got = out[:self.rows].double().cpu().numpy()
        hist = self.kw.get("history")
        size = np.abs(np.nan_to_num(self.x[:self.rows].float().numpy().astype(np.float64))).max() + 8
        if hist is not None:
            size += 0.4 * (hist.shape[1] + 10) + 1
        if self.bias is not None:
            size += max((sum(abs(float(y)) for _, y in b) for b in self.bias), default=0)
        size = size * 1.5 / min(0.4, *[t for t in self.tau if t > 0]) if (self.tau > 0).any() else size
        off = 12 * 2.0 ** -24 * size
        half, tiny = HALF[self.out_t], TINY[self.out_t]
        assert np.array_equal(np.isinf(got), np.isinf(ref) if not self.probs else np.zeros_like(got, bool))
        fin = np.isfinite(ref)
        if self.probs:
            rel = 2 * off + 2.0 ** -16 + 2.0 ** -20
            bound = rel * ref + half * ref * (1 + rel) + tiny + 2.0 ** -126   # exp2 flushes below
        else:
            bound = off + half * np.abs(ref) * (1 + 2.0 ** -10) + tiny
        err, bound = np.abs(got[fin] - ref[fin]), bound[fin]
        assert (err <= bound).all(), (err / bound).max()
        assert (out[self.rows:] == 5).all()            # rows of no sequence


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


@pytest.mark.parametrize("probs", [True, False], ids=["probs", "logits"])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("f16", "f16")])
@pytest.mark.parametrize("V", [1, 31, 33, 1000, 5003])
def test_rows(cuda_lib, probs, dtype, out, V):
    c = Case(V, [1, 4, 0, 2], V, dtype, out, probs=probs)
    c.check(c.run(cuda_lib))


@pytest.mark.parametrize("n,V", [([1] * 40, 4096), ([5], 32000), ([2, 3], 50021), ([1], 131071), ([3], 262144),
                                 ([2], 300001), ([1] * 400, 700)])
def test_vocabularies_and_batches(cuda_lib, n, V):
    for probs in (True, False):
        c = Case(V, n, V, "bf16", probs=probs)
        c.check(c.run(cuda_lib))


@pytest.mark.parametrize("what", [dict(penalties=False), dict(bias=0), dict(masked=False),
                                  dict(penalties=False, bias=0, masked=False), dict(history=5000),
                                  dict(bias=200)], ids=str)
def test_parts(cuda_lib, what):
    c = Case(5, [2, 3, 1], 3001, **what)
    c.check(c.run(cuda_lib))


def test_greedy_takes_the_first_largest(cuda_lib):
    c = Case(6, [1, 2, 1, 3], 40001, "bf16", penalties=False, bias=0, greedy=True)
    c.x[3:, 7] = 100.0                                 # ties, far apart
    c.x[3:, 39000] = 100.0
    c.x[3:, 30] = 100.0
    c.allowed[3:, :8] = False
    c.check(c.run(cuda_lib))


def test_in_place(cuda_lib):
    for V in (5003, 300001):
        c = Case(7, [2, 2], V, pad=0)
        want = c.run(cuda_lib)
        x = c.x.cuda()
        assert torch.equal(c.run(cuda_lib, out=x, x=x), want)


def test_rows_of_wider_tensors(cuda_lib):
    """Rows that start elsewhere: their sums are taken in another order, so the bound
    of check holds and not equality."""
    c = Case(8, [2, 3], 1001, pad=0)
    x = torch.full((5, 1313), float("nan"), device="cuda")
    out = torch.full((5, 1237), 3.0, device="cuda")
    x[:, 5:1006] = c.x.cuda()
    c.run(cuda_lib, out=out[:, 7:1008], x=x[:, 5:1006])
    c.check(out[:, 7:1008])
    assert (out[:, :7] == 3).all() and (out[:, 1008:] == 3).all()


def test_infinities_and_nan(cuda_lib):
    c = Case(9, [1] * 4, 900, penalties=False, bias=0, masked=False, pad=0)
    c.x[0, 5] = float("-inf")
    c.x[1, :] = float("-inf")
    c.x[2, 8] = float("nan")
    c.x[3, 8] = float("inf")
    out = c.run(cuda_lib)
    assert out[0, 5] == 0 and abs(out[0].sum().item() - 1) < 1e-5
    assert (out[1] == 0).all()
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()


def test_neutral_values_change_nothing(cuda_lib):
    x = torch.randn(3, 777, device="cuda")
    out = torch.empty_like(x)
    cuda_lib.pa_process_logits(out, x, i32([0, 1, 3]), probs=False)
    assert torch.equal(out, x)
    h = i32([[1, 2, 3], [4, 5, 6]])
    one, zero = torch.ones(2, device="cuda"), torch.zeros(2, device="cuda")
    cuda_lib.pa_process_logits(out, x, i32([0, 1, 3]), tokens=i32([1, 2, 3]), history=h,
                               history_lens=i32([3, 3]), repetition=one, frequency=zero, presence=zero,
                               temperature=one, probs=False)
    assert torch.equal(out, x)


def test_only_drafts_count_without_a_history(cuda_lib):
    x = torch.zeros(4, 50, device="cuda")
    out = torch.empty_like(x)
    cuda_lib.pa_process_logits(out, x, i32([0, 4]), tokens=i32([9, 7, 7, 8]),
                               frequency=torch.ones(1, device="cuda"), probs=False)
    want = torch.zeros(4, 50)
    want[1, 7], want[2, 7], want[3, 7], want[3, 8] = -1, -2, -2, -1
    assert torch.equal(out.cpu(), want)


def test_bad_tokens_and_lengths_are_flagged(cuda_lib):
    pa = cuda_lib
    x = torch.zeros(1, 50, device="cuda")
    out = torch.empty_like(x)
    one = torch.ones(1, device="cuda")
    pa.pa_process_logits(out, x, i32([0, 1]), history=i32([[3, 50, -1, 3]]), history_lens=i32([4]),
                         frequency=one, probs=False)
    assert pa.pa_device_error(clear=True) == pa.PA_DEVERR_TOKEN
    assert out[0, 3] == -2 and out.sum() == -2
    for hl, pl in ((9, 0), (-2, 0), (2, 3), (2, -1)):
        pa.pa_process_logits(out, x, i32([0, 1]), history=i32([[3, 4, 5, 6]]), history_lens=i32([hl]),
                             prompt_lens=i32([pl]), frequency=one, probs=False)
        assert pa.pa_device_error(clear=True) == pa.PA_DEVERR_SEQ_LEN
    for bs in ([0, 9], [2, 1], [-1, 1]):
        pa.pa_process_logits(out, x, i32([0, 1]), bias_start=i32(bs), bias_tokens=i32([1, 2]),
                             bias_values=f32([1, 1]), probs=False)
        assert pa.pa_device_error(clear=True) == pa.PA_DEVERR_SEQ_LEN
        assert (out == 0).all()
    pa.pa_process_logits(out, x, i32([0, 1]), bias_start=i32([0, 2]), bias_tokens=i32([50, 2]),
                         bias_values=f32([1, 1]), probs=False)
    assert pa.pa_device_error(clear=True) == pa.PA_DEVERR_TOKEN
    assert out[0, 2] == 1 and out.sum() == 1


def test_row_ranges_that_decrease_or_leave_the_rows(cuda_lib):
    x = torch.randn(4, 50, device="cuda")
    out = torch.full_like(x, 5.0)
    cuda_lib.pa_process_logits(out, x, i32([1, 3, 90]), probs=False)
    assert (out[0] == 5).all() and torch.equal(out[1:], x[1:])
    out.fill_(5.0)
    cuda_lib.pa_process_logits(out, x, i32([-5, 2, 1, 3]), probs=False)     # stays inside
    torch.cuda.synchronize()

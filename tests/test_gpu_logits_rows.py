"""Logits of many rows: blocks that take one row after the other, the next one's data
fetched ahead."""
import numpy as np
import pytest
import torch

from test_gpu_logits import Case, DT, HALF, TINY, _clean_error_word, f32, i32      # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probs", [True, False], ids=["probs", "logits"])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("f16", "f16")])
@pytest.mark.parametrize("n,V", [([1] * 90 + [0, 7, 4], 50021), ([3] * 210, 9001)], ids=["cluster", "block"])
def test_many_rows(cuda_lib, probs, dtype, out, n, V):
    c = Case(V + len(n), n, V, dtype, out, probs=probs, greedy=True)
    c.check(c.run(cuda_lib))


@pytest.mark.parametrize("probs", [True, False], ids=["probs", "logits"])
def test_the_largest_run(cuda_lib, probs):
    """Blocks of 512 threads; histories that one pass of loads does not hold."""
    c = Case(3, [1, 5, 0, 2] * 8, 131071, "bf16", "f32", history=2500, bias=40, probs=probs)
    c.check(c.run(cuda_lib))


@pytest.mark.parametrize("parts", [dict(penalties=False), dict(bias=0), dict(masked=False),
                                   dict(penalties=False, bias=0, masked=False)],
                         ids=["no-penalties", "no-bias", "no-mask", "plain"])
def test_parts_of_many_rows(cuda_lib, parts):
    c = Case(4, [2] * 50, 50021, "f16", "f32", **parts)
    c.check(c.run(cuda_lib))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_in_wider_tensors(cuda_lib, dtype):
    """Rows at odd distances, the tensor's first and last bytes at odd addresses."""
    c = Case(5, [2] * 60, 40003, dtype, dtype, pad=0)
    wide = torch.full((c.T * 40010 + 9,), 7.0, dtype=DT[dtype], device="cuda")
    rows = wide[3:3 + c.T * 40010].view(c.T, 40010)[:, :40003]
    rows.copy_(c.x)
    c.check(c.run(cuda_lib, out=rows, x=rows))
    assert (wide[:3] == 7).all() and (wide[3 + c.T * 40010:] == 7).all()
    assert (wide[3:3 + c.T * 40010].view(c.T, 40010)[:, 40003:] == 7).all()


@pytest.mark.parametrize("probs", [True, False], ids=["probs", "logits"])
def test_more_rows_than_a_block_looks_up_at_once(cuda_lib, probs):
    """Rows of no sequence in front and behind; each sequence's history is its own number
    twice, its temperature 1/2."""
    R, V, B = 26000, 4203, 8000
    x = torch.randn(R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).bfloat16()
    first = 1000
    qs = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 3 + first
    out = torch.full((R, V), 5.0, device="cuda")
    own = (torch.arange(B, device="cuda", dtype=torch.int32) % V)[:, None].repeat(1, 2).contiguous()
    cuda_lib.pa_process_logits(out, x, qs, history=own, history_lens=torch.full((B,), 2, dtype=torch.int32,
                               device="cuda"), frequency=torch.full((B,), 0.5, device="cuda"),
                               temperature=torch.full((B,), 0.5, device="cuda"), probs=probs)
    last = first + 3 * B
    assert (out[:first] == 5).all() and (out[last:] == 5).all()
    for a in range(0, B, 1000):
        rows = slice(first + 3 * a, first + 3 * (a + 1000))
        z = x[rows].double()
        z.scatter_add_(1, own[a:a + 1000, :1].long().repeat_interleave(3, 0),
                       torch.full((3000, 1), -1.0, dtype=torch.float64, device="cuda"))
        z = z * 2
        want = torch.softmax(z, 1) if probs else z
        # roundings of a difference and of products below 16; exp2 and the sum 2^-16
        bound = want * (2 * 3 * 2.0 ** -24 * 16 + 2.0 ** -15) if probs else want.abs() * 2.0 ** -23 + 2.0 ** -22
        assert ((out[rows].double() - want).abs() <= bound + 1e-37).all()


def test_on_two_streams_and_replayed(cuda_lib):
    c = [Case(s, [2] * 60, 50021, "bf16", "f32") for s in (7, 8)]
    want = [x.run(cuda_lib) for x in c]
    torch.cuda.synchronize()
    got = []
    for x in c:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(x.run(cuda_lib))
    torch.cuda.synchronize()
    assert all(torch.equal(a.nan_to_num(9), b.nan_to_num(9)) for a, b in zip(got, want))
    x, out = c[0].x.cuda(), torch.full_like(want[0], 5.0)
    qs, tau = i32(c[0].starts), f32(c[0].tau)
    kw = {k: (f32 if v.dtype == np.float32 else i32)(v) for k, v in c[0].kw.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.pa_process_logits(out, x, qs, temperature=tau, **kw)
    g.replay()
    first = out.clone()
    out.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(9), first.nan_to_num(9))

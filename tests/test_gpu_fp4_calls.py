"""Calls of the 4-bit functions: other streams, waits that run out, rows at any
16-byte distance, scales at the type's edges."""
import time

import numpy as np
import pytest
import torch

import plain_serving as ps
from test_gpu_fp4 import Batch, DT, _clean_error_word, i32      # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 5, 60], ids=["decode", "rows", "chunk"])
def test_on_another_stream(cuda_lib, n):
    lens = [70, 200, 1000]
    b = Batch(5, lens, [n] * 3, 16, 2, 128, "bf16")
    run = b.decode if n == 1 else b.multi
    want = run(cuda_lib)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = run(cuda_lib)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 5, 60], ids=["decode", "rows", "chunk"])
def test_wait_that_runs_out(cuda_lib, n):
    """A copy that never completes: the call ends with PA_DEVERR_TIMEOUT, and the next
    one is right."""
    b = Batch(6, [100, 300, 64, 90], [n] * 4, 16, 2, 128, "bf16")
    run = b.decode if n == 1 else b.multi
    cuda_lib.pa_test_stall_next_decode()
    t0 = time.perf_counter()
    run(cuda_lib)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_TIMEOUT
    assert time.perf_counter() - t0 < 30
    b.check(run(cuda_lib))


@pytest.mark.parametrize("lens", [[16000], [9000, 30, 8000]], ids=["one", "three"])
def test_wait_that_runs_out_in_large_clusters(cuda_lib, lens):
    b = Batch(7, lens, [1] * len(lens), 32, 8, 128, "bf16")
    cuda_lib.pa_test_stall_next_decode()
    b.decode(cuda_lib)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_TIMEOUT
    b.check(b.decode(cuda_lib))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [16, 48])
def test_rows_at_any_16_byte_distance(cuda_lib, dtype, shift):
    """Rows that start 16 but not 32 bytes aligned are written and read as others are."""
    T, Hkv, D, N = 70, 3, 80, 9
    size = DT[dtype].itemsize
    r = np.random.default_rng(shift)
    wide = Hkv * D + 16 // size * 3                    # an odd number of 16 bytes more
    flat = torch.from_numpy(r.standard_normal(T * wide + 64).astype(np.float32)).to(DT[dtype]).cuda()
    x = flat[shift // size:shift // size + T * wide].view(T, wide)[:, :Hkv * D].view(T, Hkv, D)
    s = torch.tensor([0.5, 1.0, 3e-3], device="cuda")
    slots = torch.from_numpy(r.permutation(N * 16)[:T]).cuda()
    kc = torch.zeros(N, Hkv, 9, D, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    cuda_lib.pa_reshape_and_cache_fp4(x, x.contiguous(), kc, vc, s, s, slots)
    want = ps.fp4_write(np.zeros(kc.shape, np.uint8), x.float().cpu().numpy(), s.cpu().numpy(),
                        slots.cpu().numpy())
    assert np.array_equal(kc.cpu().numpy(), want) and torch.equal(kc, vc)
    back = torch.full_like(flat, 7.0)
    y = back[shift // size:shift // size + T * wide].view(T, wide)[:, :Hkv * D].view(T, Hkv, D)
    z = torch.empty(T, Hkv, D, dtype=DT[dtype], device="cuda")
    cuda_lib.pa_gather_cache_fp4(y, z, kc, vc, s, s, slots)
    assert torch.equal(y, z)
    assert int((back != 7).sum()) == int((z != 7).sum())     # nothing between the rows


def test_two_tokens_with_one_slot_touch_only_it(cuda_lib):
    """Such tokens race, so that a group may hold codes of one and the scale of the
    other (1 has the scale 0.171875, the E4M3 next to 1/6, -2 twice that; all codes are
    6): values of either size or sign, and nothing elsewhere."""
    D = 64
    x = torch.stack([torch.full((1, D), 1.0), torch.full((1, D), -2.0)]).cuda()
    kc = torch.zeros(2, 1, 9, D, dtype=torch.uint8, device="cuda")
    vc, s = kc.clone(), torch.ones(1, device="cuda")
    cuda_lib.pa_reshape_and_cache_fp4(x, x, kc, vc, s, s, torch.tensor([5, 5], device="cuda"))
    v = ps.fp4_cache_values(kc.cpu().numpy(), np.ones(1))[:, 0]
    assert np.isin(np.abs(v[0, 5]), [1.03125, 2.0625]).all()
    v[0, 5] = 0
    assert (v == 0).all()


def test_captured_and_replayed_over_growing_lengths(cuda_lib):
    b = Batch(8, [900, 40, 700], [1] * 3, 16, 4, 128, "f16")
    full = b.lens.copy()
    out, g = b.out(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.decode(cuda_lib, out)
    for f in (0.0, 0.01, 0.3, 1.0):
        b.lens = (full * f).astype(np.int64)
        b.g["sl"].copy_(i32(b.lens))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert (out[torch.from_numpy(b.lens == 0).cuda()] == 0).all()
        b.check(out)

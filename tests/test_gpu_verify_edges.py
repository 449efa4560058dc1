"""Corners of pa_verify_drafts: blocks that have next to nothing to do before they
meet their cluster, accept products on a border below binary32, uniforms of 1."""
import numpy as np
import pytest
import torch

from test_gpu_verify import _clean_error_word, check, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 19, 37, 38, 75, 76, 151, 152, 153, 400])
def test_no_work_before_the_cluster_meets(cuda_lib, B):
    """A handful of tokens and no drafts, every size of a cluster; sequences
    without rows, whose blocks leave at once, between them."""
    r = np.random.default_rng(B)
    for V in (1, 3, 40):
        n = r.integers(0, 2, B)
        n[0] = 1
        t, d, tok, au, su, qs = inputs(B + V, n, V)
        for _ in range(4):
            check(cuda_lib, t, d, tok, au, su, qs, width=2)


def test_accept_products_next_to_the_target(cuda_lib):
    """p is u q rounded to binary32, or a neighbour of that: the product decides
    by what it is exactly, down to where its low half is no binary32 number."""
    r = np.random.default_rng(3)
    B = 6000
    u, q = (np.ldexp(1 + r.integers(0, 2**23, B) / 2**23, -r.integers(1, 64, B)) for _ in range(2))
    # 2^-59 (1 + 2^-23) times 2^-59 (1 - 2^-23) is 2^-118 (1 - 2^-46)
    u[:4], q[:4] = 2.0**-59 * (1 + 2.0**-23), 2.0**-59 * (1 - 2.0**-23)
    near = (u * q).astype(np.float32)
    p = np.where(np.arange(B) % 3 == 0, near,
                 np.nextafter(near, np.where(np.arange(B) % 3 == 1, np.float32(1), np.float32(0))))
    want = u * q < p.astype(np.float64)            # 48 bits: exact in binary64
    assert want[0] and 0.3 < want.mean() < 0.7
    t = torch.zeros(2 * B, 4, device="cuda")
    t[:, 0] = 0.5
    d = torch.zeros_like(t)
    t[0::2, 1] = torch.from_numpy(p).cuda()
    d[1::2, 1] = torch.from_numpy(q.astype(np.float32)).cuda()
    au = np.zeros(2 * B)
    au[1::2] = u
    out, acc = check(cuda_lib, t, d, np.ones(2 * B, dtype=np.int32), au, np.full(B, 0.5),
                     np.arange(0, 2 * B + 1, 2))
    assert np.array_equal(acc, want)


@pytest.mark.parametrize("V", [64, 3000, 40000])
@pytest.mark.parametrize("B", [1, 9, 60, 200])
def test_uniform_of_one_takes_the_last_weight(cuda_lib, B, V):
    """Peaked rows, whose last weights are far below the last bit of their sum."""
    r = np.random.default_rng(V + B)
    logits = 12 * r.standard_normal((B, V))
    w = np.exp(logits - logits.max(1, keepdims=True)).astype(np.float32)
    w[:, V - V // 8:] = 0                          # no weight at the end of the row
    t = torch.from_numpy(w).cuda()
    out, acc = check(cuda_lib, t, None, np.zeros(B), np.zeros(B),
                     np.where(np.arange(B) % 2 == 0, 1.0, 2.5), np.arange(B + 1))
    assert np.array_equal(out[:, 0], [np.flatnonzero(x)[-1] for x in w])

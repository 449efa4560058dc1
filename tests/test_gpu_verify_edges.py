"""Corners of pa_verify_drafts: blocks that have next to nothing to do before they
meet their cluster, accept products on a border below binary32, uniforms of 1."""
import numpy as np
import pytest

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

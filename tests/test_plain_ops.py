"""The 64-bit forms that the GPU tests compare with, held to worked examples and
to the oracle; refusals of the operators' entry points that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from paged_kv_cache_151_gb300 import build as pabuild
from paged_kv_cache_151_gb300 import pa


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.load()


def test_rotation_of_a_quarter_turn():
    """cos 0, sin 1: (a, b) becomes (-b, a), in halves and in neighbours."""
    x = np.arange(1.0, 33).reshape(1, 1, 32)
    table = np.concatenate([np.zeros(8), np.ones(8)])[None].astype(np.float32)
    y, size = po.rotated(x, table, [0], False)
    assert np.array_equal(y[0, 0, :8], -x[0, 0, 8:16]) and np.array_equal(y[0, 0, 8:16], x[0, 0, :8])
    assert np.array_equal(y[0, 0, 16:], x[0, 0, 16:])
    assert size[0, 0, 0] == 1 + 9 and size[0, 0, 20] == 21
    y, _ = po.rotated(x, table, [0], True)
    assert y[0, 0, :4].tolist() == [-2, 1, -4, 3] and np.array_equal(y[0, 0, 16:], x[0, 0, 16:])


def test_norm_of_a_known_head():
    y = po.normed(np.full((1, 1, 16), 3.0), np.full(16, 2.0), 0.0)
    assert np.allclose(y, 2.0, rtol=1e-15)
    assert np.array_equal(po.normed(np.zeros((1, 1, 16)), np.ones(16), 1e-6), np.zeros((1, 1, 16)))


def test_e4m3_of_plain_ops_is_the_oracles():
    x = np.concatenate([np.linspace(-500, 500, 4001), np.ldexp(1.0, np.arange(-14, 9)),
                        3 * np.ldexp(1.0, np.arange(-14, 7))]).astype(np.float32)
    assert np.array_equal(po.e4m3_codes(x), oracle.e4m3_encode(x))
    c = np.arange(256, dtype=np.uint8)
    assert np.array_equal(po.e4m3_values(c), oracle.e4m3_decode(c), equal_nan=True)


def test_verify_by_hand():
    t = np.array([[.5, .25, .25, 0], [0, .5, 0, .5], [.25, .25, .25, .25]], np.float32)
    d = np.array([[0, 0, 0, 0], [.25, .5, .25, 0], [0, .25, .75, 0]], np.float32)
    run = lambda tok, au, su, dr=d: po.verify(t, dr, tok, au, [su], [0, 3], 4)  # noqa: E731
    # u q < p: .9 * .25 < .5 keeps token 0, .9 * .25 < .5 keeps token 1, then the last row
    out, acc = run([9, 0, 1], [0, .9, .9], .5)
    assert out.tolist() == [[0, 1, 2, -1]] and acc[0] == 2
    # .6 * .5 >= .25 rejects token 1; max(p - q, 0) is (.25, 0, 0, 0)
    out, acc = run([9, 1, 1], [0, .6, 0], .99)
    assert out.tolist() == [[0, -1, -1, -1]] and acc[0] == 0
    # the second draft: p (0, .5, 0, .5) - q (0, .25, .75, 0) leaves (0, .25, 0, .5)
    out, acc = run([9, 0, 2], [0, 0, 0], 1 / 3 - 1e-6)
    assert out.tolist() == [[0, 1, -1, -1]] and acc[0] == 1
    out, acc = run([9, 0, 2], [0, 0, 0], .34)
    assert out.tolist() == [[0, 3, -1, -1]]
    # without draft probabilities: u < p keeps, a rejected token is left out
    out, acc = run([9, 1, 1], [0, .25, 0], .999, None)
    assert out.tolist() == [[2, -1, -1, -1]] and acc[0] == 0


def test_verify_keeps_the_targets_distribution():
    """Accepting with p/q and drawing from max(p - q, 0) gives tokens of the
    target: the mean over a grid of uniforms is its distribution."""
    p, q = np.array([.5, .2, .3]), np.array([.2, .6, .2])
    got = np.zeros(3)
    grid = (np.arange(64) + .5) / 64
    for x in range(3):
        for u in grid:
            for su in grid:
                t = np.stack([p, p]).astype(np.float32)
                d = np.stack([q, q]).astype(np.float32)
                out, _ = po.verify(t, d, [0, x], [0, u], [su], [0, 2], 2)
                got[out[0, 0]] += q[x] / len(grid) ** 2
    # each of two thresholds moves by at most half a step of its grid
    assert np.abs(got - p).max() <= 2 / 64


# ---- refusals ----------------------------------------------------------------

def _rope(lib, fp8=False, **kw):
    a = dict(q_out=16, q=16, k=16, v=16, k_cache=16, v_cache=16, k_scale=16, v_scale=16,
             q_weight=16, k_weight=16, eps=1e-6, table=16, npos=100, rot=64, inter=0,
             positions=16, slots=16, T=4, H=8, Hkv=2, D=64, qs=512, qos=512, ks=128, vs=128, N=10,
             bs=16, dtype=1)
    a.update(kw)
    scales = [a["k_scale"], a["v_scale"]] if fp8 else []
    f = lib.pa_rope_and_cache_fp8 if fp8 else lib.pa_rope_and_cache
    return f(a["q_out"], a["q"], a["k"], a["v"], a["k_cache"], a["v_cache"], *scales,
             a["q_weight"], a["k_weight"], a["eps"], a["table"], a["npos"], a["rot"], a["inter"],
             a["positions"], a["slots"], a["T"], a["H"], a["Hkv"], a["D"], a["qs"], a["qos"],
             a["ks"], a["vs"], a["N"], a["bs"], a["dtype"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=0, k=None), 0), (dict(T=-1), -1), (dict(H=-1), -1), (dict(Hkv=0), -1),
    (dict(D=0), -1), (dict(D=72), -2), (dict(D=272, qs=9999, ks=9999, vs=9999), -2),
    (dict(rot=-16), -1), (dict(rot=80), -1), (dict(rot=24), -2), (dict(npos=-1), -1),
    (dict(dtype=3), -2), (dict(dtype=9), -2), (dict(bs=32), -2), (dict(N=-1), -1),
    (dict(N=2**31), -2), (dict(T=2**31), -2), (dict(H=65536, qs=2**30, qos=2**30), -2),
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1),
    (dict(slots=None), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(table=None), -1),
    (dict(positions=None), -1), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1),
    (dict(eps=math.inf), -1), (dict(qs=504), -1), (dict(qos=504), -1), (dict(ks=120), -1),
    (dict(vs=120), -1), (dict(qs=516), -1), (dict(qos=516), -1), (dict(ks=132), -1),
    (dict(vs=132), -1), (dict(q=8), -1), (dict(q_out=8), -1), (dict(k=8), -1), (dict(v=8), -1),
    (dict(k_cache=8), -1), (dict(v_cache=24 + 4), -1), (dict(q_weight=8), -1),
    (dict(k_weight=8), -1), (dict(table=8), -1)])
def test_append_refusals(lib, fp8, kw, status):
    assert _rope(lib, fp8, **kw) == status


@pytest.mark.parametrize("kw", [
    dict(qs=640), dict(qos=640),                   # in place, one stride
    dict(q_out=32, qs=504), dict(q_out=32, qos=504), dict(q_out=32, qs=516),
    dict(q_out=32, qos=516)])
def test_append_strides_in_place_and_apart(lib, kw):
    assert _rope(lib, **kw) == _rope(lib, True, **kw) == -1


def test_append_fp8_needs_scales(lib):
    assert _rope(lib, True, k_scale=None) == -1 and _rope(lib, True, v_scale=None) == -1


def _verify(lib, **kw):
    a = dict(out=16, acc=16, target=16, draft=16, tokens=16, au=16, su=16, qs=16, B=3, T=9, mq=4,
             V=100, ts=100, ds=100, dtype=0)
    a.update(kw)
    return lib.pa_verify_drafts(a["out"], a["acc"], a["target"], a["draft"], a["tokens"], a["au"],
                                a["su"], a["qs"], a["B"], a["T"], a["mq"], a["V"], a["ts"],
                                a["ds"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 0), (dict(B=0, out=None, qs=None), 0), (dict(B=-1), -1), (dict(T=-1), -1),
    (dict(mq=-1), -1), (dict(V=0), -1), (dict(V=-5), -1), (dict(dtype=3), -2), (dict(out=None), -1),
    (dict(acc=None), -1), (dict(target=None), -1), (dict(tokens=None), -1), (dict(au=None), -1),
    (dict(su=None), -1), (dict(qs=None), -1), (dict(ts=99), -1), (dict(ds=99), -1),
    (dict(target=18), -1), (dict(draft=18), -1), (dict(target=17, dtype=1), -1)])
def test_verify_refusals(lib, kw, status):
    assert _verify(lib, **kw) == status


def _multi(lib, **kw):
    a = dict(out=16, q=16, k_cache=16, v_cache=16, k_scale=16, v_scale=16, block_tables=16,
             seq_lens=16, query_start=16, num_seqs=4, num_q_rows=12, max_query_len=3, num_heads=8,
             num_kv_heads=2, head_dim=64, num_blocks=10, block_size=16, max_blocks=4,
             q_row_stride=512, scale=0.125, dtype=1)
    a.update(kw)
    return lib.pa_decode_multi_fp8(*list(a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -2), (dict(dtype=3), -2), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
    (dict(query_start=None), -1), (dict(num_q_rows=-1), -1), (dict(max_query_len=-1), -1),
    (dict(q=8), -1), (dict(out=8), -1), (dict(q_row_stride=516), -1), (dict(head_dim=96), -2),
    (dict(block_size=32), -2), (dict(num_heads=6, num_kv_heads=2), -2), (dict(num_heads=7), -1),
    (dict(scale=math.nan), -1), (dict(k_cache=8), -1), (dict(num_seqs=0), 0),
    (dict(num_q_rows=0), 0), (dict(max_query_len=0), 0), (dict(num_seqs=65536), -2)])
def test_multi_fp8_refusals(lib, kw, status):
    assert _multi(lib, **kw) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64)
    c = torch.zeros(3, 2, 16, 64)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(x, x, x, x, c, c, None, None, i)
    with pytest.raises(ValueError):
        pa.pa_verify_drafts(i, i, x[0], None, i, x, x, i, 2)
    with pytest.raises(TypeError):
        pa.pa_decode_multi_fp8(None, x, c, c, x, x, i, i, i, 2, 0.1, 2)
    assert ctypes.sizeof(ctypes.c_void_p) == 8

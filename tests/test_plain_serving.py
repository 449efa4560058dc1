"""The 64-bit forms of the 4-bit cache, step building and logits against worked
examples and library conversions; the C ABI's and the binding's refusals (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import plain_serving as ps
from paged_kv_cache_151_gb300 import build as pabuild
from paged_kv_cache_151_gb300 import pa

P = 16                                             # any 16-byte aligned address


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.load()


# ---- the forms ------------------------------------------------------------------

def test_e4m3_values_are_the_library_types():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = ps.e4m3_values()
    assert np.array_equal(np.isnan(v), np.isnan(t)) and np.array_equal(v[~np.isnan(v)], t[~np.isnan(t)])


def test_nearest_takes_the_even_code_on_ties():
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert ps.E2M1[ps.nearest(ties, ps.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4]
    assert ps.E2M1[ps.nearest(np.nextafter(ties, 9), ps.E2M1)].tolist() == [0.5, 1, 1.5, 2, 3, 4, 6]
    x = np.linspace(0, 448, 20011)
    t = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ps.nearest(x.astype(np.float32), ps.e4m3_values()[:127]), t)


def test_a_group_by_hand():
    x = np.zeros((1, 1, 16), np.float32)
    x[0, 0, :8] = [12, -6, 3, 1, 0.5, 0.4, -0.1, 9]
    codes, sc = ps.fp4_quantise(x, np.array([1.0]))
    assert ps.e4m3_values()[sc[0, 0, 0]] == 2      # 12 / 6
    v = ps.fp4_values(codes, sc, np.array([1.0]))[0, 0, :8]
    assert v.tolist() == [12, -6, 3, 1, 0, 0, 0, 8]    # 0.25 goes to 0, 4.5 to 4
    codes, sc = ps.fp4_quantise(np.full((1, 1, 16), np.inf, np.float32), np.array([2.0]))
    assert (ps.fp4_values(codes, sc, np.array([2.0])) == 6 * 448 * 2).all()
    x[0, 0, 3] = np.nan
    assert np.isnan(ps.fp4_values(*ps.fp4_quantise(x, np.array([1.0])), np.array([1.0]))).all()


def test_rounding_is_within_half_a_step():
    r = np.random.default_rng(0)
    x = r.standard_normal((50, 2, 64)).astype(np.float32)
    s = np.array([0.3, 0.7], np.float32)
    y = ps.fp4_values(*ps.fp4_quantise(x, s), s)
    top = np.abs(x.reshape(50, 2, -1, 16)).max(-1, keepdims=True)
    # a scale is off by at most 2^-4 of itself: the largest is cut to at least 6 / 6.375
    # of it, and half the widest step is 1 of 6.375
    assert (np.abs(y - x).reshape(50, 2, -1, 16) <= top * (1 / 6 + 2.0 ** -4)).all()


def test_a_planted_mistake_is_seen():
    """Ties away from zero, a scale of the largest over 7, the nibbles swapped: each
    changes the bytes of ordinary rows."""
    r = np.random.default_rng(1)
    x = (r.integers(-24, 25, (40, 1, 32)) / 4).astype(np.float32)
    cache = np.zeros((3, 1, 9, 32), np.uint8)
    good = ps.fp4_write(cache, x, np.ones(1), np.arange(40))
    codes, sc = ps.fp4_unpack(good)
    swapped = good.copy()
    swapped[:, :, :8] = (good[:, :, :8] >> 4) | (good[:, :, :8] << 4)
    assert not np.array_equal(swapped, good)
    assert not np.array_equal(ps.fp4_write(cache, x * np.float32(6 / 7), np.ones(1), np.arange(40)), good)
    z = np.abs(x[:40, 0].reshape(40, 2, 16)) / ps.e4m3_values()[sc.transpose(0, 2, 1, 3)[..., 0, :].reshape(48, 2)[:40]][..., None]
    ties = np.isin(z, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert ties.any()                              # the rows do have ties


def test_a_step_by_hand():
    st = dict(request_tables=np.full((3, 4), -1), request_blocks=np.array([1, 0, 2]),
              free_blocks=np.array([7, 3, 9, 0]), free_count=np.array([3]))
    st["request_tables"][0, 0], st["request_tables"][2, :2] = 5, [1, 2]
    o = ps.build_step(st, [2, 0], [30, 16], [3, 1], 4, 6, 10)
    # request 2: 33 tokens, a third block (9, the last of three); request 0: 17, block 3
    assert o["tables"].tolist() == [[1, 2, 9, -7], [5, 3, -7, -7]]
    assert o["lens"].tolist() == [33, 17] and o["starts"].tolist() == [0, 3, 4]
    assert o["positions"].tolist() == [30, 31, 32, 16, 0, 0]
    assert o["slots"].tolist() == [46, 47, 144, 48, -1, -1]
    assert st["free_count"][0] == 1 and st["request_blocks"].tolist() == [2, 0, 3]
    assert ps.trim(st, [2, 0], [31, 0]) == 0       # one block of 2 back, then all of 0's
    assert st["request_blocks"].tolist() == [0, 0, 2]
    assert st["free_blocks"][:4].tolist() == [7, 3, 5, 9]


def test_logits_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.0], [2.0, -2.0, 1.0, 0.0]], np.float32)
    z = ps.logits(x, [0, 2], tokens=[9, 1], history=[[0, 1, 2]], prompt_lens=[1], history_lens=[3],
                  repetition=[2.0], frequency=[0.25], presence=[0.5], bias=[[(3, 1.0), (3, 2.0)]],
                  allowed=np.array([[1, 1, 1, 1], [1, 0, 1, 1]], bool), temperature=[0.5], probs=False)
    # row 0: 0 is in the prompt, 1 and 2 once in the output; row 1: 1 twice, not allowed
    assert z[0].tolist() == [2.0, (-4 - 0.75) * 2, (0.5 - 0.75) * 2, 6.0]
    assert z[1].tolist() == [2.0, -np.inf, (0.5 - 0.75) * 2, 6.0]
    t = torch.tensor([[1.0, 3.0, 3.0]])
    assert ps.logits(t.numpy(), [0, 1], temperature=[0.0]).tolist() == [[0, 1, 0]]
    p = ps.logits(t.numpy(), [0, 1], temperature=[2.0])
    assert np.allclose(p, torch.softmax(t.double() / 2, 1).numpy(), rtol=1e-14)


# ---- refusals of the C ABI ----------------------------------------------------------

def test_fp4_write_checks(lib):
    args = [P, P, P, P, P, P, P, 4, 2, 64, 128, 128, 10, 16, 1, None]
    for f in (lib.pa_reshape_and_cache_fp4, lib.pa_gather_cache_fp4):
        def status(**kw):
            a = list(args)
            for k, v in kw.items():
                a[int(k[1:])] = v
            return f(*a)
        assert status(_7=0) == 0                   # nothing to do
        assert status(_7=-1) == -1 and status(_8=0) == -1 and status(_12=-1) == -1
        assert status(_9=40) == -2 and status(_9=1040, _10=2080, _11=2080) == -2
        assert status(_13=32) == -2 and status(_14=7) == -2
        for i in (0, 1, 2, 3, 4, 5, 6):
            assert status(**{f"_{i}": None}) == -1
        for i in (0, 1, 2, 3):
            assert status(**{f"_{i}": 8}) == -1    # not 16-byte aligned
        assert status(_10=100) == -1 and status(_10=132) == -1     # short; 264 bytes
        assert status(_7=2**31) == -2


def test_fp4_decode_checks(lib):
    dec = [P, P, P, P, P, P, P, P, 4, 8, 2, 64, 10, 16, 4, 512, 0.125, 1, None]
    def status(f=lib.pa_decode_fp4, base=dec, **kw):
        a = list(base)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    assert status(_8=0) == 0
    assert status(_17=0) == -2 and status(_17=3) == -2 and status(_17=4) == -2   # q in fp32, codes
    for i in range(8):
        assert status(**{f"_{i}": None}) == -1
    assert status(_0=8) == -1 and status(_1=8) == -1 and status(_2=8) == -1
    assert status(_11=96) == -2 and status(_13=32) == -2 and status(_9=7) == -1
    assert status(_9=32, _15=2048) == -2           # 16 heads a group
    assert status(_15=516) == -1 and status(_16=float("nan")) == -1
    ws = ctypes.c_void_p(256)
    part = dec[:-1] + [512, 64, ws, 1 << 30, None]
    assert status(lib.pa_decode_partitioned_fp4, part, _18=100) == -1
    assert status(lib.pa_decode_partitioned_fp4, part, _21=16) == -3
    assert status(lib.pa_decode_partitioned_fp4, part, _20=ctypes.c_void_p(128)) == -3
    multi = [P] * 9 + [4, 12, 3, 8, 2, 64, 10, 16, 4, 512, 0.125, 1, None]
    f = lib.pa_decode_multi_fp4
    assert status(f, multi, _9=0) == 0 and status(f, multi, _10=0) == 0 and status(f, multi, _11=0) == 0
    assert status(f, multi, _8=None) == -1 and status(f, multi, _10=-1) == -1
    assert status(f, multi, _20=0) == -2


def test_step_checks(lib):
    b = [P] * 12 + [4, 9, 6, 6, 20, 50, 40, 16, None]
    def status(f, base, **kw):
        a = list(base)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    f = lib.pa_build_step
    for i in range(12, 19):
        assert status(f, b, **{f"_{i}": -1}) == -1
    assert status(f, b, _19=32) == -2 and status(f, b, _12=65536) == -2 and status(f, b, _18=2**31) == -2
    assert status(f, b, _13=2**19 + 1) == -2
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 10, 11):     # not request_ids and new_lens
        assert status(f, b, **{f"_{i}": None}) == -1
    t = [P] * 6 + [4, 9, 6, 50, 16, None]
    f = lib.pa_trim_blocks
    assert status(f, t, _6=0) == 0
    for i in (6, 7, 8, 9):
        assert status(f, t, **{f"_{i}": -1}) == -1
    for i in (0, 1, 3, 4, 5):
        assert status(f, t, **{f"_{i}": None}) == -1
    assert status(f, t, _10=8) == -2 and status(f, t, _7=2**19 + 1) == -2


def test_logits_checks(lib):
    # out logits start tokens history prompt hist_lens rep freq pres bias_start bias_tok bias_val allowed temp
    b = [P] * 15 + [2, 5, 100, 100, 100, 30, 4, 6, 1, 1, 0, None]
    b[0] = 32
    def status(**kw):
        a = list(b)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.pa_process_logits(*a)
    assert status(_15=0) == 0 and status(_16=0) == 0
    assert status(_17=0) == -1 and status(_17=2**30 + 1) == -2 and status(_15=-1) == -1
    assert status(_24=7) == -2 and status(_25=2) == -2 and status(_24=0, _25=1) == -2
    for i in (0, 1, 2, 6, 11, 12):
        assert status(**{f"_{i}": None}) == -1
    assert status(_18=99) == -1 and status(_19=99) == -1 and status(_21=3) == -1
    assert status(_0=30) == -1                     # not a multiple of 4
    assert status(_1=32) == -1                     # in place in another type
    assert status(_1=32, _24=0, _19=104) == -1     # in place at another distance


# ---- refusals of the binding -----------------------------------------------------------

def test_the_binding_refuses_host_tensors_and_other_things():
    t = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="out must be a CUDA tensor"):
        pa.pa_process_logits(t, t, t)
    with pytest.raises(TypeError, match="k must be a torch.Tensor"):
        pa.pa_reshape_and_cache_fp4(None, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="come together"):
        pa.pa_build_step(*[t] * 10, t, None, 5)
    with pytest.raises(ValueError, match="needs history_lens"):
        pa.pa_process_logits(t, t, t, history=t)
    with pytest.raises(ValueError, match="come together"):
        pa.pa_process_logits(t, t, t, bias_start=t)


def test_descriptions_of_tensors():
    pa.load()
    Spec = pa._tensors.Spec
    for bad in ("a:i32[B", "a", "a:[B]", "a:i32[B]!", "a:abcd[B]"):
        with pytest.raises(ValueError, match="not a description"):
            Spec(bad)
    s = Spec("a:i32[B] b:f32[B+1]?")
    with pytest.raises(TypeError):
        s(0, None)
    with pytest.raises(TypeError, match="a must be a torch.Tensor"):
        s(0, None, None)
    with pytest.raises(ValueError, match="a must be a CUDA tensor"):
        s(-1, torch.zeros(3, dtype=torch.int32), None)

"""The cache write with per-head norms and rotation (pa_rope_and_cache and its
E4M3 form) against the 64-bit forms of plain_ops.py.  Tolerances:
plain_ops.stored_error_bound (a stored key or query), bit equality (values,
and everything a call must leave alone)."""
import numpy as np
import pytest
import torch

import plain_ops as po
from paged_kv_cache_151_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


class Case:
    """Inputs of one call; tokens of `lens` sequences at random positions."""

    def __init__(self, seed, T, H, Hkv, D, R, dtype="bf16", fp8=False, norm=True,
                 interleaved=False, padding=0, npos=5000, fused=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        dt = wl.DTYPES[dtype]
        self.dtype, self.fp8, self.interleaved, self.T, self.D = dtype, fp8, interleaved, T, D
        if fused:                                  # views of one projection's output
            x = torch.randn(T, (H + 2 * Hkv) * D, device="cuda", generator=g).mul_(1.5).to(dt)
            self.q = x[:, :H * D].view(T, H, D)
            self.k = x[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
            self.v = x[:, (H + Hkv) * D:].view(T, Hkv, D)
        else:
            self.q, self.k, self.v = (torch.randn(T, h, D, device="cuda", generator=g).to(dt)
                                      for h in (H, Hkv, Hkv))
        N = (T + 15) // 16 + 5
        slots = r.permutation(N * 16)[:T]
        slots[r.permutation(T)[:padding]] = -1 - r.integers(0, 5)
        self.slots = torch.from_numpy(slots).cuda()
        self.positions = torch.from_numpy(r.integers(0, npos, T)).cuda()
        self.table = None
        if R:
            ang = np.arange(npos)[:, None] * 1e4 ** (-np.arange(R // 2) / (R // 2))[None]
            self.table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)
                                          .astype(np.float32)).cuda()
        self.q_w = self.k_w = None
        if norm:
            self.q_w = (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dt)
            self.k_w = (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dt)
        shape = (N, Hkv, 16, D)
        self.ks = self.vs = None
        if fp8:
            self.kc = torch.randint(0, 127, shape, device="cuda", generator=g, dtype=torch.uint8)
            self.vc = torch.randint(0, 127, shape, device="cuda", generator=g, dtype=torch.uint8)
            self.ks = torch.linspace(0.004, 0.02, Hkv, device="cuda")   # small ones saturate
            self.vs = torch.linspace(0.03, 0.003, Hkv, device="cuda")
        else:
            self.kc = torch.randn(shape, device="cuda", generator=g).to(dt)
            self.vc = torch.randn(shape, device="cuda", generator=g).to(dt)

    def run(self, pa, q_out=None, stream=None):
        kc, vc = self.kc.clone(), self.vc.clone()
        if q_out is None:
            q_out = torch.full(self.q.shape, float("nan"), device="cuda", dtype=self.q.dtype)
        torch.cuda.synchronize()
        kw = dict(q_weight=self.q_w, k_weight=self.k_w, eps=EPS, interleaved=self.interleaved,
                  stream=stream)
        if self.fp8:
            pa.pa_rope_and_cache_fp8(q_out, self.q, self.k, self.v, kc, vc, self.ks, self.vs,
                                     self.table, self.positions, self.slots, **kw)
        else:
            pa.pa_rope_and_cache(q_out, self.q, self.k, self.v, kc, vc, self.table,
                                 self.positions, self.slots, **kw)
        torch.cuda.synchronize()
        return q_out, kc, vc

    def check(self, q_out, kc, vc, skip=()):
        """skip: tokens that must leave everything alone."""
        host = lambda t: None if t is None else t.detach().double().cpu().numpy()  # noqa: E731
        pos = self.positions.cpu().numpy().copy()
        pos[list(skip)] = 0
        live = np.ones(self.T, bool)
        live[list(skip)] = False
        table = None if self.table is None else self.table.cpu().numpy()
        y, size = po.rotated(po.normed(host(self.q), host(self.q_w), EPS), table, pos,
                             self.interleaved)
        err = np.abs(host(q_out) - y)[live]
        assert (err <= po.stored_error_bound(y, size, self.dtype)[live]).all(), err.max()
        y, size = po.rotated(po.normed(host(self.k), host(self.k_w), EPS), table, pos,
                             self.interleaved)
        slots = self.slots.cpu().numpy()
        put = live & (slots >= 0) & (slots < self.kc.shape[0] * 16)
        b, row = slots[put] // 16, slots[put] % 16
        # everything else in the caches is as it was
        for new, old in ((kc, self.kc), (vc, self.vc)):
            same = (new.view(torch.uint8) == old.view(torch.uint8)).view(*new.shape, -1).all(-1)
            same = same.cpu().numpy()
            same[b, :, row] = True
            assert same.all()
        got_k = kc.cpu()[torch.from_numpy(b), :, torch.from_numpy(row)]
        got_v = vc.cpu()[torch.from_numpy(b), :, torch.from_numpy(row)]
        want_v = self.v.cpu()[torch.from_numpy(put)]
        if self.fp8:
            ks = self.ks.double().cpu().numpy()[:, None]
            z, zs = y[put] / ks, 33 * 2.0 ** -24 * size[put] / ks     # one more: the quotient
            assert po.e4m3_between(got_k.numpy(), z, zs).all()
            q32 = want_v.float().numpy() / self.vs.cpu().numpy()[:, None]
            assert np.array_equal(got_v.numpy(), po.e4m3_codes(q32))
        else:
            err = np.abs(host(got_k) - y[put])
            assert (err <= po.stored_error_bound(y, size, self.dtype)[put]).all(), err.max()
            assert torch.equal(got_v.contiguous().view(torch.uint8),
                               want_v.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T", [1, 2, 37, 300])
@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f16", False), ("f32", False),
                                       ("bf16", True), ("f16", True), ("f32", True)])
def test_append_types(cuda_lib, dtype, fp8, T):
    c = Case(T, T, 8, 2, 128, 128, dtype=dtype, fp8=fp8, padding=T // 9)
    c.check(*c.run(cuda_lib))


@pytest.mark.parametrize("H,Hkv,D,R", [(32, 8, 128, 128), (8, 8, 64, 64), (16, 1, 64, 32),
                                       (3, 1, 96, 48), (5, 3, 16, 16), (4, 4, 48, 16),
                                       (7, 7, 256, 128), (2, 1, 208, 208), (9, 2, 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_shapes(cuda_lib, H, Hkv, D, R, interleaved, norm, fp8):
    c = Case(H + D + R, 45, H, Hkv, D, R, fp8=fp8, norm=norm, interleaved=interleaved, padding=4)
    c.check(*c.run(cuda_lib))


@pytest.mark.parametrize("T", [5000, 20000])
def test_append_many_tokens(cuda_lib, T):
    c = Case(7, T, 8, 2, 64, 64, fp8=True, padding=100)
    c.check(*c.run(cuda_lib))


def test_append_one_norm_only(cuda_lib):
    for which in ("q_w", "k_w"):
        c = Case(11, 33, 8, 2, 128, 64)
        setattr(c, which, None)
        c.check(*c.run(cuda_lib))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_in_place(cuda_lib, dtype):
    """q_out may be q, inside the projection's output."""
    c = Case(12, 70, 16, 4, 128, 128, dtype=dtype)
    apart = c.run(cuda_lib)
    k0, v0 = c.k.clone(), c.v.clone()
    q0 = c.q.clone()
    got = c.run(cuda_lib, q_out=c.q)
    assert torch.equal(c.q, apart[0]) and torch.equal(got[1], apart[1])
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)       # the neighbours in the buffer
    assert not torch.equal(c.q, q0)


def test_append_q_out_strided(cuda_lib):
    c = Case(13, 21, 4, 2, 64, 64)
    wide = torch.zeros(21, 6, 64, device="cuda", dtype=torch.bfloat16)
    q_out, kc, vc = c.run(cuda_lib, q_out=wide[:, 1:5])
    c.check(q_out, kc, vc)
    assert not wide[:, 0].any() and not wide[:, 5].any()


def test_append_without_queries(cuda_lib):
    c = Case(14, 50, 4, 2, 128, 128)
    want = c.run(cuda_lib)
    kc, vc = c.kc.clone(), c.vc.clone()
    cuda_lib.pa_rope_and_cache(None, None, c.k, c.v, kc, vc, c.table, c.positions, c.slots,
                               k_weight=c.k_w, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(kc, want[1]) and torch.equal(vc, want[2])


def test_append_no_tokens(cuda_lib):
    c = Case(15, 4, 4, 2, 64, 64)
    kc, vc = c.kc.clone(), c.vc.clone()
    cuda_lib.pa_rope_and_cache(c.q[:0], c.q[:0], c.k[:0], c.v[:0], kc, vc, c.table,
                               c.positions[:0], c.slots[:0])
    torch.cuda.synchronize()
    assert torch.equal(kc, c.kc) and torch.equal(vc, c.vc)


def test_append_bad_slot_and_position(cuda_lib):
    """A slot past the pool: the query row only.  A position outside the table:
    nothing of the token.  A padding token with such a position: nothing, and
    no error."""
    c = Case(16, 40, 4, 2, 128, 128)
    N = c.kc.shape[0] * 16
    c.slots[3], c.slots[5] = N, N + 2**40
    c.check(*c.run(cuda_lib))
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SLOT
    c = Case(17, 40, 4, 2, 128, 128)
    c.positions[7], c.positions[8] = c.table.shape[0], -1
    got = c.run(cuda_lib)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_POSITION
    c.check(*got, skip=[7, 8])
    assert got[0][[7, 8]].isnan().all()
    c = Case(18, 40, 4, 2, 128, 128)
    c.positions[7], c.slots[7] = -1, -1
    got = c.run(cuda_lib)
    c.check(*got, skip=[7])
    assert got[0][7].isnan().all()


def test_append_infinities_stay_in_their_place(cuda_lib):
    """Without norms an infinite or NaN element reaches its pair's elements and
    no other; elements past rot_dim pass."""
    c = Case(19, 3, 2, 1, 128, 64, norm=False, fused=False)
    c.q[1, 0, 3], c.q[1, 1, 100], c.v[2, 0, 9] = float("inf"), float("nan"), float("inf")
    q_out, kc, vc = c.run(cuda_lib)
    bad = ~torch.isfinite(q_out)
    assert set(map(tuple, bad.nonzero().tolist())) == {(1, 0, 3), (1, 0, 35), (1, 1, 100)}
    assert torch.isfinite(kc).all() and (~torch.isfinite(vc)).sum() == 1


def test_append_zero_heads_normalise_to_zero(cuda_lib):
    c = Case(20, 9, 4, 2, 128, 128)
    c.q[4].zero_()
    c.k[4].zero_()
    c.check(*c.run(cuda_lib))


def test_append_far_positions_past_32_bits_of_table(cuda_lib):
    """A table of more than 2^31 elements (9 GB): row offsets are 64-bit."""
    P, R = 17_000_000, 128
    c = Case(21, 6, 2, 1, 128, 0, norm=False)
    c.table = torch.zeros(P, R, device="cuda")
    c.positions = torch.tensor([P - 1, P - 2, 16_777_216, 5, 16_777_215, 0], device="cuda")
    for i, p in enumerate(c.positions.tolist()):
        ang = np.linspace(0.1, 3.0, R // 2) * (i + 1)
        c.table[p] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)])).float()
    q_out, kc, vc = c.run(cuda_lib)
    rows = c.table[c.positions].clone()
    c.table, c.positions = rows, torch.arange(6, device="cuda")   # the same rows, small
    c.check(q_out, kc, vc)


def test_append_on_another_stream(cuda_lib):
    c = Case(22, 100, 8, 2, 128, 128, fp8=True)
    s = torch.cuda.Stream()
    c.check(*c.run(cuda_lib, stream=s))

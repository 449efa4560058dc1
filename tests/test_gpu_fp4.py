"""The 4-bit cache on the GPU: writes and read-back equal to the format's
definition, attention within derived bounds of a 64-bit form."""
import numpy as np
import pytest
import torch

import plain_serving as ps
from plain_ops import HALF, TINY

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAD = 2**31 - 1


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def pool(N, Hkv, D, seed, nan_outside=None):
    """Random tiles; with nan_outside (a bool mask [N, 16] of rows in use) the rows
    outside it get scales that are NaN."""
    r = np.random.default_rng(seed)
    c = r.integers(0, 256, (N, Hkv, 9, D), dtype=np.uint8)
    sc = r.integers(40, 72, (N, Hkv, 16, D // 16), dtype=np.uint8)     # 2^-2 .. 3.5
    if nan_outside is not None:
        sc = np.where(nan_outside[:, None, :, None], sc, np.uint8(127))
    c[:, :, 8] = sc.reshape(N, Hkv, D)
    return c


# ---- the write and the read-back --------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 16), (5, 2, 64), (37, 8, 128), (300, 3, 96), (33, 1, 256)])
def test_write_and_gather(cuda_lib, dtype, T, Hkv, D):
    r = np.random.default_rng(T + D)
    N = T // 8 + 3
    x = torch.from_numpy(r.standard_normal((T, 2 * Hkv + 1, D)).astype(np.float32) *
                         np.exp(r.uniform(-6, 6, (T, 2 * Hkv + 1, 1))).astype(np.float32)).to(DT[dtype])
    x[0, 0, :] = 0                                     # a group of zeros
    if T > 4:
        x[1, 0, 3], x[2, Hkv, 5], x[3, 0, 0] = np.inf, -np.inf, np.nan
        x[4, 0, :16] = 2.0 ** -14                      # a scale below the least E4M3 number
    ks, vs = r.uniform(0.5, 2, Hkv).astype(np.float32), r.uniform(0.01, 0.1, Hkv).astype(np.float32)
    slots = r.permutation(N * 16)[:T].astype(np.int64)
    slots[T // 2::7] = -1
    kc, vc = pool(N, Hkv, D, 1), pool(N, Hkv, D, 2)
    xg = x.cuda()
    k, v = xg[:, :Hkv], xg[:, Hkv:2 * Hkv]             # rows of a wider tensor
    dk, dv = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    tks, tvs, ts = (torch.from_numpy(a).cuda() for a in (ks, vs, slots))
    cuda_lib.pa_reshape_and_cache_fp4(k, v, dk, dv, tks, tvs, ts)
    wk = ps.fp4_write(kc, x[:, :Hkv].float().numpy(), ks, slots)
    wv = ps.fp4_write(vc, x[:, Hkv:2 * Hkv].float().numpy(), vs, slots)
    for got, want in ((dk, wk), (dv, wv)):
        codes, sc = ps.fp4_unpack(got.cpu().numpy())
        wcodes, wsc = ps.fp4_unpack(want)
        assert np.array_equal(sc, wsc)
        assert np.array_equal(codes, wcodes)           # signs of zeros too
    ko, vo = (torch.full((T, Hkv, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    cuda_lib.pa_gather_cache_fp4(ko, vo, dk, dv, tks, tvs, ts)
    for got, cache, s in ((ko, wk, ks), (vo, wv, vs)):
        val = ps.fp4_cache_values(cache, s)            # the product with s, rounded to binary32
        live = slots >= 0
        with np.errstate(invalid="ignore"):
            want = torch.from_numpy(val[slots[live] // 16, :, slots[live] % 16].astype(np.float32))
        assert torch.equal(got[torch.from_numpy(live).cuda()].cpu().nan_to_num(9e9),
                           want.to(DT[dtype]).nan_to_num(9e9))
        assert (got[torch.from_numpy(~live).cuda()] == 7).all()


def test_every_quotient_near_a_border_rounds_as_defined(cuda_lib):
    """Elements around every border of E2M1 and scales around those of E4M3, under a
    scale that is no power of two."""
    D, rows = 64, []
    base = np.float32(0.37)
    for top in np.concatenate([6 * ps.e4m3_values()[1:126], 6 * (ps.e4m3_values()[1:125] +
                                                                ps.e4m3_values()[2:126]) / 2]):
        for nudge in (-1, 0, 1):
            t = np.float32(top)
            t = np.nextafter(t, np.float32(nudge * 1e9)) if nudge else t
            mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]) * top / 6
            g = np.concatenate([[t], mids[:7], -mids, ]).astype(np.float32)[:16]
            rows.append(g * base)
    rows = np.array(rows, np.float32)
    T = len(rows) // 4
    x = rows[:4 * T].reshape(T, 1, D)
    N = T // 16 + 1
    kc = torch.zeros(N, 1, 9, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    s = torch.full((1,), float(base), device="cuda")
    slots = torch.arange(T, device="cuda")
    xg = torch.from_numpy(x).cuda()
    cuda_lib.pa_reshape_and_cache_fp4(xg, xg, kc, vc, s, s, slots)
    want = ps.fp4_write(np.zeros((N, 1, 9, D), np.uint8), x, np.array([base]), np.arange(T))
    assert np.array_equal(kc.cpu().numpy(), want)
    assert torch.equal(kc, vc)


def test_slots_past_the_pool_are_flagged(cuda_lib):
    D, N = 64, 2
    kc = torch.full((N, 2, 9, D), 3, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    x = torch.ones(3, 2, D, device="cuda")
    s = torch.ones(2, device="cuda")
    slots = torch.tensor([N * 16, 2**40, -5], device="cuda")
    cuda_lib.pa_reshape_and_cache_fp4(x, x, kc, vc, s, s, slots)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SLOT
    assert (kc == 3).all() and (vc == 3).all()
    y = torch.full_like(x, 5.0)
    cuda_lib.pa_gather_cache_fp4(y, y.clone(), kc, vc, s, s, slots)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SLOT
    assert (y == 5).all()


# ---- attention ----------------------------------------------------------------

class Batch:
    """Sequences of n[s] rows over lens[s] tokens, blocks dealt from a permutation;
    rows of the pool outside the sequences have NaN scales."""

    def __init__(self, seed, lens, n, H, Hkv, D, dtype, kscale=0.3):
        r = np.random.default_rng(seed)
        self.lens, self.n = np.asarray(lens), np.asarray(n)
        self.H, self.Hkv, self.D, self.dtype = H, Hkv, D, dtype
        nb = (self.lens + 15) // 16
        N = int(nb.sum()) + 3
        perm = r.permutation(N)
        self.tables = np.full((len(lens), max(1, int(nb.max(initial=0)))), PAD, np.int64)
        used = np.zeros((N, 16), bool)
        at = 0
        for s, L in enumerate(self.lens):
            self.tables[s, :nb[s]] = perm[at:at + nb[s]]
            for i in range(nb[s]):
                used[perm[at + i], :min(16, L - 16 * i)] = True
            at += nb[s]
        self.kc, self.vc = pool(N, Hkv, D, seed + 1, used), pool(N, Hkv, D, seed + 2, used)
        self.ks = r.uniform(0.5, 1.5, Hkv).astype(np.float32) * np.float32(kscale)
        self.vs = r.uniform(0.5, 1.5, Hkv).astype(np.float32)
        self.starts = np.concatenate([[0], np.cumsum(self.n)])
        T = int(self.starts[-1])
        self.q = torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).to(DT[dtype]).cuda()
        self.scale = D ** -0.5
        cu = lambda a: torch.from_numpy(a).cuda()      # noqa: E731
        self.g = dict(kc=cu(self.kc), vc=cu(self.vc), ks=cu(self.ks), vs=cu(self.vs),
                      bt=i32(self.tables), sl=i32(self.lens), qs=i32(self.starts))

    def out(self):
        return torch.full_like(self.q, float("nan"))

    def decode(self, pa, out=None):
        out = self.out() if out is None else out
        g = self.g
        pa.pa_decode_fp4(out, self.q, g["kc"], g["vc"], g["ks"], g["vs"], g["bt"], g["sl"],
                         self.scale, self.Hkv)
        return out

    def partitioned(self, pa, part, most=None):
        g, out = self.g, self.out()
        most = int(self.lens.max()) if most is None else most
        ws = torch.empty(pa.pa_decode_partitioned_workspace_size(len(self.lens), self.H, self.D, most,
                                                                 part), dtype=torch.uint8, device="cuda")
        pa.pa_decode_partitioned_fp4(out, self.q, g["kc"], g["vc"], g["ks"], g["vs"], g["bt"], g["sl"],
                                     self.scale, self.Hkv, part, most, ws)
        return out, ws

    def multi(self, pa, most=None):
        g, out = self.g, self.out()
        pa.pa_decode_multi_fp4(out, self.q, g["kc"], g["vc"], g["ks"], g["vs"], g["bt"], g["sl"],
                               g["qs"], int(self.n.max()) if most is None else most, self.scale, self.Hkv)
        return out

    def check(self, out):
        """Every element against 64 bits.  The codes times their scales are exact
        and so is q as f16; a weight is off by e1 of itself: its rounding to f16
        (2^-11), exp2 and its argument (2^-20), and the score's sum of D + 8 terms
        in fp32 and its two scalings, (D + 16) 2^-24 of the sum of the terms' sizes.
        With such weights in numerator and denominator the result is off by e1 (A +
        |out|), A = sum of w |v|.  fp32 sums of L products lose at most L 2^-24 of
        the same, and the result is rounded.  f16 holds weights below 2^-14 in steps
        of 2^-24, off by 2^-25 however small they are, while a row's largest weight
        is at least 2^7 (its level is set 7 log2 units below a score): L keys of no
        weight to speak of may so add L 2^-32 of the largest value, which counts
        where the keys that have the weight hold a 0.  With scores of thousands e1
        is no longer small: exp(e1) - 1 and 1 / (1 - that) in its place."""
        G = self.H // self.Hkv
        kv = [torch.from_numpy(np.nan_to_num(ps.fp4_cache_values(c, s))).cuda()
              for c, s in ((self.kc, self.ks), (self.vc, self.vs))]
        for s, L in enumerate(self.lens.tolist()):
            a, b = int(self.starts[s]), int(self.starts[s + 1])
            if a == b or L == 0:
                continue
            blocks = torch.from_numpy(self.tables[s, :-(-L // 16)]).cuda()
            k, v = (c[blocks].permute(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, :L] for c in kv)
            q = self.q[a:b].double().unflatten(1, (self.Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)
            x = torch.matmul(q, k.transpose(1, 2)) * self.scale       # [Hkv, G * n, L]
            size = torch.matmul(q.abs(), k.abs().transpose(1, 2)).amax(-1, keepdim=True) * self.scale
            pos = torch.arange(L - (b - a), L, device="cuda").repeat(G)[:, None]
            x = torch.where(torch.arange(L, device="cuda") <= pos, x, -np.inf)
            w = torch.softmax(x, -1) if L else x
            ref, A = torch.matmul(w, v), torch.matmul(w, v.abs())
            e1 = 2.0 ** -11 + 2.0 ** -20 + (self.D + 16) * 2.0 ** -24 * size
            e1 = torch.expm1(e1 + L * 2.0 ** -24)
            e1 = e1 / (1 - e1)
            bound = 1.01 * e1 * (A + ref.abs()) + HALF[self.dtype] * ref.abs() * (1.01 + e1)
            bound = bound + L * 2.0 ** -32 * v.abs().amax((1, 2), keepdim=True)
            bound = bound + TINY[self.dtype]
            got = out[a:b].double().unflatten(1, (self.Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)
            bad = ~((got - ref).abs() <= bound)
            assert not bad.any(), (s, L, int(bad.sum()), float(((got - ref).abs() / bound).max()))


LENS = [[1], [15, 16, 17], [0, 1, 33, 0, 250, 1000], [5000, 3, 700]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 64), (8, 4, 128), (8, 2, 64), (8, 2, 128), (16, 2, 128),
                                     (16, 2, 64)])
@pytest.mark.parametrize("lens", LENS, ids=["one", "edges", "empty", "long"])
def test_decode(cuda_lib, dtype, H, Hkv, D, lens):
    b = Batch(len(lens) + D, lens, [1] * len(lens), H, Hkv, D, dtype)
    out = b.decode(cuda_lib)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
    for s, L in enumerate(lens):
        if L == 0:
            assert (out[s] == 0).all()
    b.check(out)


@pytest.mark.parametrize("B", [130, 300, 700])
def test_decode_batches(cuda_lib, B):
    r = np.random.default_rng(B)
    b = Batch(B, r.integers(0, 200, B), [1] * B, 8, 2, 64, "bf16")
    b.check(b.decode(cuda_lib))


@pytest.mark.parametrize("dtype,H,Hkv,D,part", [("bf16", 32, 8, 128, 512), ("f16", 8, 1, 64, 16),
                                                ("bf16", 4, 4, 128, 96)])
def test_partitioned(cuda_lib, dtype, H, Hkv, D, part):
    b = Batch(3, [700, 1, 0, 513, 2000], [1] * 5, H, Hkv, D, dtype)
    out, ws = b.partitioned(cuda_lib, part)
    torch.cuda.synchronize()
    assert (out[2] == 0).all()
    b.check(out)
    # the statistics: level 7 to 15 log2 units below the largest score
    o, m, l = cuda_lib.workspace_views(ws, 5, H, D, 2000, part)
    k = torch.from_numpy(np.nan_to_num(ps.fp4_cache_values(b.kc, b.ks))).cuda()
    for s, L in ((0, 700), (3, 513)):
        keys = k[torch.from_numpy(b.tables[s, :-(-L // 16)]).cuda()].permute(1, 0, 2, 3)
        keys = keys.reshape(Hkv, -1, D)[:, :L].repeat_interleave(H // Hkv, 0)
        x = torch.einsum("hd,hld->hl", b.q[s].double(), keys) * b.scale
        for p in range(-(-L // part)):
            y = x[:, p * part:(p + 1) * part]
            below = (y.amax(1) - m[s, :, p].double()) / np.log(2)
            assert (below > 6.99).all() and (below < 15.01).all()
            want = (y - m[s, :, p].double()[:, None]).exp().sum(1)
            assert ((l[s, :, p].double() - want).abs() <= 2.0 ** -9 * want).all()


ROWS = [([1], [1]), ([5], [5]), ([700, 33, 16], [4, 4, 1]), ([90, 0, 64, 300], [8, 0, 3, 9]),
        ([200, 500, 40], [130, 7, 40]), ([1500], [600]), ([65, 64, 63], [65, 64, 63])]


@pytest.mark.parametrize("dtype,H,Hkv,D", [("bf16", 32, 8, 128), ("f16", 8, 2, 64), ("bf16", 8, 8, 64),
                                           ("f16", 16, 2, 128), ("bf16", 4, 2, 128)])
@pytest.mark.parametrize("lens,n", ROWS, ids=[str(i) for i in range(len(ROWS))])
def test_multi(cuda_lib, dtype, H, Hkv, D, lens, n):
    b = Batch(len(lens) + D, lens, n, H, Hkv, D, dtype)
    out = b.multi(cuda_lib)
    torch.cuda.synchronize()
    b.check(out)


def test_one_row_per_sequence_is_decode(cuda_lib):
    b = Batch(11, [40, 1, 555, 16, 2100], [1] * 5, 8, 2, 128, "bf16")
    b.check(b.decode(cuda_lib))
    b.check(b.multi(cuda_lib))
    b.check(b.partitioned(cuda_lib, 64)[0])


def test_rows_of_a_wider_tensor(cuda_lib):
    b = Batch(12, [300, 50], [1, 1], 8, 2, 64, "f16")
    want = b.decode(cuda_lib)
    wide = torch.randn(2, 24, 64, device="cuda").half()
    wide[:, 8:16] = b.q
    b.q = wide[:, 8:16]
    out = torch.empty(2, 8, 64, device="cuda", dtype=torch.float16)
    assert torch.equal(b.decode(cuda_lib, out), want)


def test_large_and_tiny_scores(cuda_lib):
    """Scores of some thousands, where one key takes a row, and of nearly zero."""
    for kscale in (300.0, 1e-6):
        b = Batch(13, [400, 60], [1, 1], 8, 2, 128, "bf16", kscale)
        b.check(b.decode(cuda_lib))
        b = Batch(13, [400, 60], [5, 50], 8, 2, 128, "bf16", kscale)
        b.check(b.multi(cuda_lib))


@pytest.mark.parametrize("n", [[3, 2], [3, 80]], ids=["short", "long"])
def test_blocks_outside_the_pool_are_left_out(cuda_lib, n):
    b = Batch(14, [100, 90], n, 8, 2, 128, "bf16")
    lost = b.tables.copy()
    b.g["bt"] = i32(np.where(np.arange(lost.shape[1]) == 2, 10**6, lost))
    out = b.multi(cuda_lib)
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_BLOCK_ID
    # the same sequences without tokens 32..47, rows that stand behind them
    for s in range(2):
        first = int(b.lens[s]) - n[s]
        behind = [i for i in range(n[s]) if first + i >= 48]
        c = Batch(14, [int(b.lens[s]) - 16], [len(behind)], 8, 2, 128, "bf16")
        c.kc, c.vc, c.ks, c.vs = b.kc, b.vc, b.ks, b.vs
        c.tables = np.delete(lost[s:s + 1], 2, 1)
        rows = [int(b.starts[s]) + i for i in behind]
        c.q = b.q[rows]
        c.check(out[rows])


def test_nan_in_a_key_reaches_the_rows_that_see_it(cuda_lib):
    b = Batch(15, [200, 100], [1, 1], 8, 2, 128, "bf16")
    c = b.g["kc"].clone()
    blk = int(b.tables[0, 3])
    c[blk, 1, 8, :8] = 127                             # row 0 of that block, KV head 1
    b.g["kc"] = c
    out = b.decode(cuda_lib)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()
    out, _ = b.partitioned(cuda_lib, 32)
    assert torch.isnan(out[0, 4:]).all() and torch.isfinite(out[0, :4]).all()


def test_results_do_not_depend_on_the_placement(cuda_lib):
    b = Batch(16, [1000, 77, 300], [4, 60, 1], 8, 2, 128, "f16")
    want = b.multi(cuda_lib)
    N = b.kc.shape[0]
    perm = np.random.default_rng(1).permutation(N)
    back = np.argsort(perm)
    b.g["kc"], b.g["vc"] = b.g["kc"][torch.from_numpy(perm).cuda()], b.g["vc"][torch.from_numpy(perm).cuda()]
    b.g["bt"] = i32(np.where(b.tables == PAD, PAD, back[np.minimum(b.tables, N - 1)]))
    assert torch.equal(b.multi(cuda_lib), want)


def test_offsets_past_32_bits(cuda_lib):
    """A pool of more than 2^32 bytes, the sequence in its last blocks."""
    D, Hkv = 128, 8
    N = (1 << 32) // (Hkv * 9 * D) + 50
    small = Batch(17, [100], [1], 8, Hkv, D, "bf16")
    n = small.kc.shape[0]
    big = []
    for c in (small.kc, small.vc):
        x = torch.empty(N, Hkv, 9, D, dtype=torch.uint8, device="cuda")
        x[N - n:] = torch.from_numpy(c).cuda()
        big.append(x)
    want = small.decode(cuda_lib)
    small.g["kc"], small.g["vc"] = big
    small.g["bt"] = i32(small.tables + N - n)
    assert torch.equal(small.decode(cuda_lib), want)
    # and rows written and read there
    x = torch.randn(2, Hkv, D, device="cuda").bfloat16()
    slots = torch.tensor([N * 16 - 1, N * 16 - 17], device="cuda")
    cuda_lib.pa_reshape_and_cache_fp4(x, x, *big, small.g["ks"], small.g["vs"], slots)
    y, z = torch.empty_like(x), torch.empty_like(x)
    cuda_lib.pa_gather_cache_fp4(y, z, *big, small.g["ks"], small.g["vs"], slots)
    # half a step of E2M1 at the largest of 16 (1 of 6) and the scale's rounding
    # (2^-4) bound an element's error by a third of the group's largest
    big16 = x.float().unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True)
    assert ((y.float() - x.float()).unflatten(-1, (-1, 16)).abs() <= big16 / 3).all()


@pytest.mark.parametrize("lens,n", [([3000], [1]), ([9000, 5], [1, 1]), ([20000], [1]), ([70000], [1]),
                                    ([4100], [4]), ([9000, 40, 2500], [3, 1, 8]), ([30000], [7])])
def test_few_long_sequences_over_large_clusters(cuda_lib, lens, n):
    """Few units and long tables: clusters of up to 16 blocks share a unit's keys."""
    for H, Hkv, D in ((8, 2, 128), (8, 1, 64), (4, 4, 128)):
        b = Batch(lens[0] + D, lens, n, H, Hkv, D, "bf16")
        b.check(b.decode(cuda_lib) if max(n) == 1 else b.multi(cuda_lib))

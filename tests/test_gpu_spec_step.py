"""One speculative serving step as it is used: the new queries and keys
normalised, rotated and written (pa_rope_and_cache_fp8), attention of every
row (pa_decode_multi_fp8), a projection to the vocabulary, and the verification
of the drafts (pa_verify_drafts) -- eager, captured in a CUDA graph and
replayed on new inputs, and beside another step on a second stream."""
import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from paged_kv_cache_151_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

H, HKV, D, V = 8, 2, 128, 701


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


class Step:
    """The buffers of a step of B sequences, n[s] rows each (padded to T rows
    with padding tokens), over a pool with room for their contexts."""

    def __init__(self, seed, n, ctx, pad=3):
        r = np.random.default_rng(seed)
        n, ctx = np.asarray(n), np.asarray(ctx)
        self.B, self.T, rows = len(n), int(n.sum()) + pad, int(n.sum())
        L = n + ctx
        nb = (L + 15) // 16
        N = int(nb.sum()) + 4
        perm = r.permutation(N)
        self.tables = np.full((self.B, int(nb.max()) + 1), wl.PAD, dtype=np.int32)
        at = np.concatenate([[0], np.cumsum(nb)])
        for s in range(self.B):
            self.tables[s, :nb[s]] = perm[at[s]:at[s + 1]]
        self.qs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        s_of = np.repeat(np.arange(self.B), n)
        pos = ctx[s_of] + np.arange(rows) - self.qs[s_of]
        slots = self.tables[s_of, pos // 16].astype(np.int64) * 16 + pos % 16
        self.positions = torch.from_numpy(np.concatenate([pos, np.zeros(pad, np.int64)])).cuda()
        self.slots = torch.from_numpy(np.concatenate([slots, np.full(pad, -1)])).cuda()
        self.L, self.n = L, n
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bt, self.sl, self.qst = i32(self.tables), i32(L), i32(self.qs)
        ang = np.arange(int(L.max()))[:, None] * 1e4 ** (-np.arange(D // 2) / (D // 2))[None]
        self.table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)
                                      .astype(np.float32)).cuda()
        self.qkv = torch.empty(self.T, (H + 2 * HKV) * D, device="cuda", dtype=torch.bfloat16)
        self.w = (1 + 0.2 * torch.randn(D, device="cuda")).bfloat16()
        self.ks = torch.full((HKV,), 0.01, device="cuda")
        self.vs = torch.full((HKV,), 0.012, device="cuda")
        self.kc, self.vc = ((torch.randn(N, HKV, 16, D, device="cuda") / 0.01).clamp(-448, 448)
                            .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
        self.q = torch.empty(self.T, H, D, device="cuda", dtype=torch.bfloat16)
        self.o = torch.zeros_like(self.q)
        self.head = torch.randn(H * D, V, device="cuda").bfloat16() / 4
        self.probs = torch.empty(self.T, V, device="cuda")
        self.draft = torch.empty(self.T, V, device="cuda")
        self.tokens = torch.zeros(self.T, device="cuda", dtype=torch.int32)
        self.au = torch.empty(self.T, device="cuda")
        self.su = torch.empty(self.B, device="cuda")
        self.out = torch.empty(self.B, int(n.max()), device="cuda", dtype=torch.int32)
        self.acc = torch.empty(self.B, device="cuda", dtype=torch.int32)
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv.copy_(torch.randn(self.qkv.shape, device="cuda", generator=g))
        self.draft.copy_((2 * torch.randn(self.T, V, device="cuda", generator=g)).softmax(-1))
        self.tokens.copy_(self.draft.argmax(-1))
        self.au.copy_(torch.rand(self.T, device="cuda", generator=g) / 16)
        self.su.copy_(torch.rand(self.B, device="cuda", generator=g))

    def run(self, pa):
        q, k, v = (x.view(self.T, -1, D) for x in self.qkv.split([H * D, HKV * D, HKV * D], 1))
        pa.pa_rope_and_cache_fp8(self.q, q, k, v, self.kc, self.vc, self.ks, self.vs, self.table,
                                 self.positions, self.slots, q_weight=self.w, k_weight=self.w)
        pa.pa_decode_multi_fp8(self.o, self.q, self.kc, self.vc, self.ks, self.vs, self.bt, self.sl,
                               self.qst, int(self.n.max()), D ** -0.5, HKV)
        torch.softmax((self.o.flatten(1) @ self.head).float(), -1, out=self.probs)
        pa.pa_verify_drafts(self.out, self.acc, self.probs, self.draft, self.tokens, self.au,
                            self.su, self.qst, self.out.shape[1])

    def results(self):
        return [x.clone() for x in (self.q, self.kc, self.vc, self.o, self.probs, self.out, self.acc)]

    def check(self):
        rows = int(self.qs[-1])
        host = lambda t: t.double().cpu().numpy()  # noqa: E731
        x = host(self.qkv).reshape(self.T, -1, D)
        y, size = po.rotated(po.normed(x[:, :H], host(self.w), 1e-6), self.table.cpu().numpy(),
                             self.positions.cpu().numpy(), False)
        assert (np.abs(host(self.q) - y) <= po.stored_error_bound(y, size, "bf16")).all()
        y, size = po.rotated(po.normed(x[:, H:H + HKV], host(self.w), 1e-6),
                             self.table.cpu().numpy(), self.positions.cpu().numpy(), False)
        slots = self.slots.cpu().numpy()[:rows]
        codes = self.kc.cpu().numpy()[slots // 16, :, slots % 16]
        scale = self.ks.double().cpu().numpy()[:, None]
        assert po.e4m3_between(codes, (y / scale)[:rows], (33 * 2.0 ** -24 * size / scale)[:rows]).all()
        kv = [torch.from_numpy(po.e4m3_values(c.cpu().numpy()).astype(np.float32)) * float(s[0])
              for c, s in ((self.kc, self.ks), (self.vc, self.vs))]
        ref = oracle.decode_multi(self.q[:rows].float().cpu(), *kv, self.tables, self.L, self.qs,
                                  D ** -0.5, HKV, "f32")
        got = host(self.o)[:rows]
        assert np.abs(got - ref).max() <= 2e-2
        assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
        out, acc = po.verify(self.probs.cpu().numpy(), self.draft.cpu().numpy(),
                             self.tokens.cpu().numpy(), self.au.cpu().numpy(),
                             self.su.cpu().numpy(), self.qs, self.out.shape[1])
        assert np.array_equal(self.out.cpu().numpy(), out)
        assert np.array_equal(self.acc.cpu().numpy(), acc)


SHAPES = [([4] * 12, range(5, 600, 50)), ([1], [0]), ([3, 90, 1, 5], [17, 300, 0, 250]),
          ([1, 0, 7], [31, 40, 500])]


@pytest.mark.parametrize("n,ctx", SHAPES, ids=["drafts", "one-token", "chunk", "idle"])
def test_step(cuda_lib, n, ctx):
    st = Step(1, n, list(ctx))
    st.run(cuda_lib)
    torch.cuda.synchronize()
    st.check()


def test_steps_back_to_back_see_their_own_writes(cuda_lib):
    """Attention starts early behind the cache write: the same results as with
    a synchronisation between the calls."""
    st = Step(2, [4] * 40, [37 * i for i in range(40)])
    for seed in range(20):
        st.fill(seed)
        torch.cuda.synchronize()
        st.run(cuda_lib)
        got = st.results()
        q, k, v = (x.view(st.T, -1, D) for x in st.qkv.split([H * D, HKV * D, HKV * D], 1))
        cuda_lib.pa_rope_and_cache_fp8(st.q, q, k, v, st.kc, st.vc, st.ks, st.vs, st.table,
                                       st.positions, st.slots, q_weight=st.w, k_weight=st.w)
        torch.cuda.synchronize()
        st.run(cuda_lib)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, st.results()))


def test_queries_rotated_in_place_reach_the_attention(cuda_lib):
    """q rotated inside the projection's output, then attention on that view at
    once: the same as with a synchronisation between."""
    st = Step(6, [4] * 30, [41 * i for i in range(30)])
    q, k, v = (x.view(st.T, -1, D) for x in st.qkv.split([H * D, HKV * D, HKV * D], 1))
    for seed in range(20):
        got = []
        for wait in (False, True):
            st.fill(seed)
            torch.cuda.synchronize()
            cuda_lib.pa_rope_and_cache_fp8(q, q, k, v, st.kc, st.vc, st.ks, st.vs, st.table,
                                           st.positions, st.slots, q_weight=st.w, k_weight=st.w)
            if wait:
                torch.cuda.synchronize()
            cuda_lib.pa_decode_multi_fp8(st.o, q, st.kc, st.vc, st.ks, st.vs, st.bt, st.sl,
                                         st.qst, 4, D ** -0.5, HKV)
            got.append(st.o.clone())
        assert torch.equal(*got)


@pytest.mark.parametrize("n,ctx", [SHAPES[0], SHAPES[2]], ids=["drafts", "chunk"])
def test_step_captured_and_replayed(cuda_lib, n, ctx):
    st = Step(3, n, list(ctx))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        st.run(cuda_lib)                           # the libraries' first use, outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run(cuda_lib)
    for seed in (11, 12):
        st.fill(seed)
        g.replay()
        torch.cuda.synchronize()
        got = st.results()
        st.check()
        st.run(cuda_lib)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, st.results()))


def test_two_steps_at_once(cuda_lib):
    """Two steps with buffers of their own on two streams."""
    a, b = Step(4, [4] * 12, range(5, 600, 50)), Step(5, [3, 90, 1, 5], [17, 300, 0, 250])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for st, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                st.run(cuda_lib)
    torch.cuda.synchronize()
    a.check()
    b.check()

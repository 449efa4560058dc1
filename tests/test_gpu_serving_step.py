"""The 4-bit cache, the step building, the logits and the drafts' verification run
together as a serving loop runs them, every step against the 64-bit forms."""
import numpy as np
import pytest
import torch

import plain_serving as ps
from test_gpu_fp4 import Batch, DT, HALF

pytestmark = pytest.mark.gpu

H, HKV, D, V, WIDTH, HIST = 8, 2, 64, 203, 12, 120


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Server:
    """R requests, of which the batch names some, each with a fixed number of rows a
    step; an entry without rows pads the batch, and so do `pad` rows.  All of a step
    runs on the device; sequences alternate between greedy and drawn tokens."""

    def __init__(self, pa, seed, ids, new, R, dtype="bf16", steps=8, pad=3):
        r = np.random.default_rng(seed)
        self.pa, self.ids, self.new, self.dtype, self.r = pa, np.asarray(ids), np.asarray(new), dtype, r
        B, self.T = len(ids), int(sum(new)) + pad
        self.ctx = np.where(self.ids < 0, 0, r.integers(1, 70, B))
        held = np.zeros(R, np.int64)
        held[self.ids[self.ids >= 0]] = -(-self.ctx // 16)[self.ids >= 0]
        N = int(held.sum()) + 6 * B
        perm = r.permutation(N)
        tables, at = np.zeros((R, WIDTH), np.int64), 0
        for i in range(R):
            tables[i, :held[i]] = perm[at:at + held[i]]
            at += held[i]
        self.st = dict(request_tables=tables, request_blocks=held,
                       free_blocks=np.concatenate([perm[at:], np.zeros(at, np.int64)]),
                       free_count=np.array([N - at]))
        self.N = N
        self.ks, self.vs = (r.uniform(0.02, 0.04, HKV).astype(np.float32) for _ in range(2))
        # the tokens in the cache at the start
        self.kc, self.vc = np.zeros((N, HKV, 9, D), np.uint8), np.zeros((N, HKV, 9, D), np.uint8)
        slots = [int(tables[self.ids[s], p // 16]) * 16 + p % 16 for s in range(B) for p in range(self.ctx[s])]
        for c, sc in ((self.kc, self.ks), (self.vc, self.vs)):
            c[:] = ps.fp4_write(c, r.standard_normal((len(slots), HKV, D)).astype(np.float32), sc, np.array(slots))
        hl = np.where(self.ids < 0, 0, r.integers(3, 20, B))
        self.hist, self.hl, self.pl = r.integers(0, V, (B, HIST)), hl, hl // 2
        self.tau = np.where(np.arange(B) % 2 == 0, 0, 0.8).astype(np.float32)
        self.rep = np.full(B, 1.3, np.float32)
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()    # noqa: E731
        # inputs of every step: the model's stand-ins
        S = steps
        self.k, self.v = (torch.from_numpy(r.standard_normal((S, self.T, HKV, D)).astype(np.float32))
                          .to(DT[dtype]).cuda() for _ in range(2))
        self.q = torch.from_numpy(r.standard_normal((S, self.T, H, D)).astype(np.float32)).to(DT[dtype]).cuda()
        self.x = torch.from_numpy(3 * r.standard_normal((S, self.T, V)).astype(np.float32)).to(DT[dtype]).cuda()
        self.row_seq = np.concatenate([np.repeat(np.arange(B), new), np.zeros(pad, int)]).astype(int)
        first = np.concatenate([[0], np.cumsum(new)])[:-1]
        self.row_off = np.arange(self.T) - first[self.row_seq]
        # a draft is what the row before it likes best, three times of four
        best = self.x.float().argmax(-1).cpu().numpy()
        drafts = np.roll(best, 1, 1)
        self.drafts = cu(np.where(r.random(drafts.shape) < 0.75, drafts, r.integers(0, V, drafts.shape)))
        self.ua, self.us = cu(r.random((S, self.T)).astype(np.float32)), cu(r.random((S, B)).astype(np.float32))
        self.allow = r.random((S, self.T, V)) < 0.9
        words = np.zeros((S, self.T, -(-V // 32) * 32), np.uint8)
        words[:, :, :V] = self.allow
        self.mask = cu(np.packbits(words, axis=-1, bitorder="little").view(np.int32))
        self.most = max(new)
        self.B = B
        self.now = dict(k=self.k[0].clone(), v=self.v[0].clone(), q=self.q[0].clone(), x=self.x[0].clone(),
                        drafts=self.drafts[0].clone(), ua=self.ua[0].clone(), us=self.us[0].clone(),
                        mask=self.mask[0].clone())
        self.all = dict(k=self.k, v=self.v, q=self.q, x=self.x, drafts=self.drafts, ua=self.ua, us=self.us,
                        mask=self.mask)
        z = lambda *shape, dt=torch.int32: torch.zeros(*shape, dtype=dt, device="cuda")    # noqa: E731
        self.g = dict(tables=z(B, WIDTH), lens=z(B), starts=z(B + 1), pos=z(self.T, dt=torch.int64),
                      slots=z(self.T, dt=torch.int64), out=torch.zeros_like(self.q[0]),
                      probs=z(self.T, V, dt=torch.float32), tok=z(B, self.most), acc=z(B),
                      ctx=i32(self.ctx), new=i32(self.new), ids=i32(self.ids), hist=i32(self.hist),
                      hl=i32(self.hl), pl=i32(self.pl), kc=cu(self.kc), vc=cu(self.vc), ks=cu(self.ks),
                      vs=cu(self.vs), tau=cu(self.tau), rep=cu(self.rep), tokens=z(self.T),
                      row_seq=cu(self.row_seq), row_off=cu(self.row_off), cols=torch.arange(HIST, device="cuda"),
                      **{k: i32(v) for k, v in self.st.items()})
        # the hole that a refused or padded entry leaves in its history's index
        self.step_no = 0

    def load(self, i):
        for k, v in self.now.items():
            v.copy_(self.all[k][i])

    def step(self):
        """One step's calls, all on the current stream."""
        pa, g, n = self.pa, self.g, self.now
        pa.pa_build_step(g["tables"], g["lens"], g["starts"], g["pos"], g["slots"], g["request_tables"],
                         g["request_blocks"], g["ids"], g["ctx"], g["new"], g["free_blocks"],
                         g["free_count"], self.N)
        last = g["hist"].gather(1, (g["hl"] - 1).clamp(min=0).long()[:, None])[:, 0]
        g["tokens"].copy_(torch.where(g["row_off"] == 0, last[g["row_seq"]].long(), n["drafts"]))
        pa.pa_reshape_and_cache_fp4(n["k"], n["v"], g["kc"], g["vc"], g["ks"], g["vs"], g["slots"])
        pa.pa_decode_multi_fp4(g["out"], n["q"], g["kc"], g["vc"], g["ks"], g["vs"], g["tables"], g["lens"],
                               g["starts"], self.most, D ** -0.5, HKV)
        pa.pa_process_logits(g["probs"], n["x"], g["starts"], tokens=g["tokens"], history=g["hist"],
                             prompt_lens=g["pl"], history_lens=g["hl"], repetition=g["rep"],
                             allowed=n["mask"], temperature=g["tau"])
        pa.pa_verify_drafts(g["tok"], g["acc"], g["probs"], None, g["tokens"], n["ua"], n["us"], g["starts"],
                            self.most)
        grown = torch.where(g["new"] > 0, g["acc"] + 1, 0)
        at = g["cols"][None] - g["hl"][:, None]        # column of the step's tokens
        fresh = g["tok"].gather(1, at.clamp(0, self.most - 1))
        g["hist"].copy_(torch.where((at >= 0) & (at < grown[:, None]), fresh, g["hist"]))
        g["hl"].add_(grown)
        g["ctx"].add_(grown)
        pa.pa_trim_blocks(g["request_tables"], g["request_blocks"], g["ids"], g["ctx"], g["free_blocks"],
                          g["free_count"])

    def check(self, i):
        """What step i left, against the forms."""
        o = ps.build_step(self.st, self.ids, self.ctx, self.new, WIDTH, self.T, self.N)
        assert o["flags"] == 0
        g = {k: v.cpu() for k, v in self.g.items()}
        written = o["tables"] != -7
        assert np.array_equal(g["tables"].numpy()[written], o["tables"][written])
        for a, b in (("lens", "lens"), ("starts", "starts"), ("pos", "positions"), ("slots", "slots")):
            assert np.array_equal(g[a].numpy(), o[b]), a
        for c, x, s, name in ((self.kc, self.k, self.ks, "kc"), (self.vc, self.v, self.vs, "vc")):
            c[:] = ps.fp4_write(c, x[i].float().cpu().numpy(), s, o["slots"])
            assert np.array_equal(g[name].numpy(), c), name
        b = Batch.__new__(Batch)
        b.lens, b.n, b.H, b.Hkv, b.D, b.dtype = o["lens"], self.new, H, HKV, D, self.dtype
        b.tables, b.kc, b.vc, b.ks, b.vs = np.maximum(o["tables"], 0), self.kc, self.vc, self.ks, self.vs
        b.starts, b.q, b.scale = o["starts"], self.q[i], D ** -0.5
        b.check(self.g["out"])
        starts, tokens = o["starts"], g["tokens"].numpy()
        last = [self.hist[s, max(self.hl[s] - 1, 0)] for s in range(self.B)]
        want_tokens = np.where(self.row_off == 0, np.array(last)[self.row_seq], self.drafts[i].cpu().numpy())
        assert np.array_equal(tokens, want_tokens)
        p = ps.logits(self.x[i].float().cpu().numpy(), starts, tokens=tokens, history=self.hist,
                      prompt_lens=self.pl, history_lens=self.hl, repetition=self.rep,
                      allowed=self.allow[i], temperature=self.tau)
        got = g["probs"].double().numpy()
        rows = starts[-1]
        # four roundings of terms below 16 / 0.8, and the exponential's and sum's 2^-16
        assert (np.abs(got[:rows] - p[:rows]) <= (2 * 6 * 2.0 ** -24 * 20 + 2.0 ** -15) * p[:rows] + 1e-37).all()
        assert (got[rows:] == 0).all()
        tok, acc = g["tok"].numpy(), g["acc"].numpy()
        for s in range(self.B):
            n, a = int(self.new[s]), int(acc[s])
            if n == 0:
                assert a == 0 and (tok[s] == -1).all()
                continue
            first = int(starts[s])
            if self.tau[s] == 0:                       # a draft is kept while it is the largest
                best = p[first:first + n].argmax(-1)
                want = 0
                while want < n - 1 and tokens[first + want + 1] == best[want]:
                    want += 1
                assert a == want and tok[s, a] == best[a]
            assert np.array_equal(tok[s, :a], tokens[first + 1:first + 1 + a])
            assert 0 <= tok[s, a] < V and p[first + a, tok[s, a]] > 0
            self.hist[s, self.hl[s]:self.hl[s] + a + 1] = tok[s, :a + 1]
            self.hl[s] += a + 1
            self.ctx[s] += a + 1
        assert np.array_equal(g["hist"].numpy(), self.hist)
        assert ps.trim(self.st, self.ids, self.ctx) == 0
        for k, v in self.st.items():
            assert np.array_equal(g[k].numpy(), v), k

    def results(self):
        return {k: v.clone() for k, v in self.g.items()}


def server(pa, seed, dtype="bf16", steps=8):
    return Server(pa, seed, ids=[4, 0, -1, 7, 2, 9, 1], new=[4, 1, 0, 3, 6, 2, 4], R=11, dtype=dtype, steps=steps)


@pytest.fixture(autouse=True)
def _clean_error_word(cuda_lib):
    cuda_lib.pa_device_error(clear=True)
    yield
    flags = cuda_lib.pa_device_error(clear=True)
    assert flags == 0, f"device error word set: {flags:#x}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_steps_one_by_one(cuda_lib, dtype):
    s = server(cuda_lib, 1, dtype)
    for i in range(8):
        s.load(i)
        s.step()
        s.check(i)


def test_a_captured_step_replayed(cuda_lib):
    s = server(cuda_lib, 2)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.step()
    for i in range(8):
        s.load(i)
        g.replay()
        s.check(i)


def test_back_to_back_and_on_two_streams_at_once(cuda_lib):
    """Eight steps without a wait, then two servers at once, each on a stream of its
    own: the same bits."""
    want = []
    for seed in (3, 4):
        s = server(cuda_lib, seed)
        for i in range(8):
            s.load(i)
            s.step()
        want.append(s.results())
    both = [server(cuda_lib, seed) for seed in (3, 4)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for i in range(8):
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s.load(i)
                s.step()
    torch.cuda.synchronize()
    for s, w in zip(both, want):
        for k, v in s.results().items():
            assert torch.equal(v, w[k]), k


def test_a_prompt_in_chunks_then_decode(cuda_lib):
    """A prompt of 90 tokens in runs of 40, 40 and 10 next to sequences in decode."""
    pa = cuda_lib
    ref = None
    for runs in ([90], [40, 40, 10]):
        s = Server(pa, 5, ids=[3, 1], new=[1, 1], R=4, steps=1, pad=0)
        k, v, q = (torch.randn(90, h, D, generator=torch.Generator().manual_seed(h)).bfloat16().cuda()
                   for h in (HKV, HKV + 1, H))
        v = v[:, :HKV].contiguous()
        done, outs, g = 0, [], s.g
        for n in runs:
            o = [torch.zeros(1, WIDTH, dtype=torch.int32, device="cuda"), i32([0]), i32([0, 0]),
                 torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")]
            pa.pa_build_step(*o, g["request_tables"], g["request_blocks"], i32([2]), i32([done]), i32([n]),
                             g["free_blocks"], g["free_count"], s.N)
            r = slice(done, done + n)
            pa.pa_reshape_and_cache_fp4(k[r], v[r], g["kc"], g["vc"], g["ks"], g["vs"], o[4])
            out = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
            pa.pa_decode_multi_fp4(out, q[r], g["kc"], g["vc"], g["ks"], g["vs"], o[0], o[1], o[2], n,
                                   D ** -0.5, HKV)
            outs.append(out)
            done += n
        got = torch.cat(outs).double()
        if ref is None:
            ref = got
            back = [torch.zeros_like(k), torch.zeros_like(v)]
            pa.pa_gather_cache_fp4(*back, g["kc"], g["vc"], g["ks"], g["vs"], o[4])
        else:
            # both within the attention's bound, about a rounding to bf16 and two of weights
            assert ((got - ref).abs() <= 2 * (HALF["bf16"] + 2.0 ** -9) * ref.abs().amax()).all()
    assert torch.isfinite(back[0].float()).all()

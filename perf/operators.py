"""The operators of a speculative serving step over a paged KV cache, in their
plain form and through the library's entry points.

* ``append``: the step's new queries and keys normalised per head (optional),
  rotated by their positions, the keys and values written into their cache
  slots (``pa_rope_and_cache``, and ``pa_rope_and_cache_fp8`` into E4M3);
* ``attend``: several new query tokens per sequence, causal among themselves,
  over an E4M3 paged cache (``pa_decode_multi_fp8``);
* ``verify``: the drafted tokens accepted or rejected against the target's
  probabilities with given uniforms, and the token after them drawn
  (``pa_verify_drafts``).

Each case has an ``op`` and the sizes of one call.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
PAD = 2**31 - 1                    # block-table padding, never a valid block id
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


def listed():
    return [
        # one request, one token: the latency of a step's append
        dict(name="append_one_token", op="append", seqs=1, tokens=1, far=4000, heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, norm=True, padding=0, dtype="bf16", cache="bf16",
             len_seed=1),
        # a decode step of the serving mix: 256 sequences, four rows each (one
        # token and three drafts)
        dict(name="append_verify_batch", op="append", seqs=256, tokens=1024, far=4096, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, norm=True, padding=13, dtype="bf16",
             cache="e4m3", len_seed=2),
        # prompt chunks of odd lengths, rotation of half the head in
        # neighbouring pairs, no norms
        dict(name="append_chunks_odd", op="append", seqs=5, tokens=4099, far=30000, heads=16,
             kv_heads=4, dim=64, rot=32, interleaved=True, norm=False, padding=29, dtype="f16",
             cache="f16", len_seed=3),
        # a prefill step of long prompts
        dict(name="append_prompts_long", op="append", seqs=8, tokens=32768, far=60000, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, norm=True, padding=0, dtype="bf16",
             cache="e4m3", len_seed=4),
        # one request verifying four drafts: latency
        dict(name="attend_one_request", op="attend", seqs=1, rows_lo=5, rows_hi=5, ctx="range",
             ctx_lo=900, ctx_hi=1100, heads=32, kv_heads=8, dim=128, dtype="bf16", len_seed=5),
        # the serving mix with three drafts each
        dict(name="attend_verify_batch", op="attend", seqs=256, rows_lo=4, rows_hi=4, ctx="mix",
             ctx_lo=1, ctx_hi=4092, heads=32, kv_heads=8, dim=128, dtype="bf16", len_seed=6),
        # prompt chunks of odd lengths over contexts of odd lengths
        dict(name="attend_chunks_odd", op="attend", seqs=3, rows_lo=200, rows_hi=500, ctx="range",
             ctx_lo=37, ctx_hi=6000, heads=16, kv_heads=2, dim=64, dtype="f16", len_seed=7),
        # a long prompt's later chunk
        dict(name="attend_chunk_long", op="attend", seqs=1, rows_lo=2048, rows_hi=2048, ctx="range",
             ctx_lo=14000, ctx_hi=14336, heads=32, kv_heads=8, dim=128, dtype="bf16", len_seed=8),
        # one request, four drafts, a small vocabulary: latency
        dict(name="verify_one_request", op="verify", seqs=1, drafts_lo=4, drafts_hi=4, vocab=32000,
             draft_probs=True, dtype="f32", len_seed=9),
        # a batch with 0 to 6 drafts each over a large odd vocabulary
        dict(name="verify_batch", op="verify", seqs=64, drafts_lo=0, drafts_hi=6, vocab=131071,
             draft_probs=True, dtype="f32", len_seed=10),
        # drafts without probabilities (copied from the prompt), probabilities in 16 bits
        dict(name="verify_copied_drafts", op="verify", seqs=256, drafts_lo=3, drafts_hi=3,
             vocab=50021, draft_probs=False, dtype="bf16", len_seed=11),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "verify"])
    seed = rng.randrange(1, 10**6)
    heads, kv_heads = rng.choice([(32, 8), (16, 2), (8, 8), (16, 8), (64, 8), (8, 2)])
    if op == "append":
        dim = rng.choice([64, 128, 96, 256])
        tokens = _log(rng, 1, 12000 if dim * (heads + 2 * kv_heads) <= 7000 else 4000)
        rot = rng.choice([dim, dim, dim // 2, 32])
        dtype = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 300)), tokens=tokens,
                    far=_log(rng, 16, 60000), heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                    padding=rng.choice([0, 0, tokens // 7]), dtype=dtype,
                    cache=rng.choice([dtype, "e4m3"]), len_seed=seed)
    if op == "attend":
        dim = rng.choice([64, 128])
        many = rng.random() < 0.5
        if many:                                   # a batch verifying drafts
            lo = _log(rng, 1, 4)
            return dict(op=op, seqs=_log(rng, 1, 200), rows_lo=lo, rows_hi=lo + rng.randrange(0, 6),
                        ctx="mix", ctx_lo=0, ctx_hi=4000, heads=heads, kv_heads=kv_heads, dim=dim,
                        dtype=rng.choice(["bf16", "f16"]), len_seed=seed)
        lo = _log(rng, 17, 900)                    # prompt chunks
        ctx = _log(rng, 16, 8000)
        hi = lo + rng.randrange(0, lo)
        most = 2048 * 14000 * 32 * 128 // (hi * (ctx + hi) * heads * dim)
        return dict(op=op, seqs=max(1, min(rng.randrange(1, 5), most)), rows_lo=lo, rows_hi=hi,
                    ctx="range", ctx_lo=ctx // 3, ctx_hi=ctx, heads=heads, kv_heads=kv_heads,
                    dim=dim, dtype=rng.choice(["bf16", "f16"]), len_seed=seed)
    lo = rng.randrange(0, 6)
    vocab, dtype = _log(rng, 1000, 131071), rng.choice(["f32", "f32", "bf16", "f16"])
    most = 64 * 131071 * 4 // (vocab * SIZE[dtype])
    return dict(op=op, seqs=min(_log(rng, 1, 200), most), drafts_lo=lo,
                drafts_hi=lo + rng.randrange(0, 4), vocab=vocab, draft_probs=rng.random() < 0.7,
                dtype=dtype, len_seed=seed)


# ---- the lengths of a case (they belong to the case, not to the inputs' seed) ----

def _append_lens(c):
    """(tokens, first position) of each sequence; tokens adds up to c["tokens"]."""
    r = np.random.RandomState(c["len_seed"])
    S, T = c["seqs"], c["tokens"]
    n = np.full(S, T // S, dtype=np.int64)
    n[: T % S] += 1
    shift = r.randint(0, max(1, n.min()), S)       # ragged: take from one, give to the next
    n = n - shift + np.roll(shift, 1)
    return n, r.randint(0, c["far"] + 1, S).astype(np.int64)


def _attend_lens(c):
    """(rows, context before them) of each sequence."""
    r = np.random.RandomState(c["len_seed"])
    S = c["seqs"]
    n = r.randint(c["rows_lo"], c["rows_hi"] + 1, S).astype(np.int64)
    if c["ctx"] == "mix":                          # lognormal, median 350, sigma 1
        ctx = np.clip(np.round(np.exp(r.randn(S) + math.log(350.0))), c["ctx_lo"], c["ctx_hi"])
    else:
        ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, S)
    return n, ctx.astype(np.int64)


def _verify_lens(c):
    r = np.random.RandomState(c["len_seed"])
    return r.randint(c["drafts_lo"], c["drafts_hi"] + 1, c["seqs"]).astype(np.int64)


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)])


def work(case):
    c = case
    if c["op"] == "append":
        T, P = c["tokens"], c["padding"]
        row, kv = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        es, cs = SIZE[c["dtype"]], SIZE[c["cache"]]
        nbytes = T * (2 * row * es + 16 + 4 * c["rot"]) + (T - P) * 2 * kv * (es + cs)
        if c["norm"]:
            nbytes += 2 * c["dim"] * es
        return {"bytes": nbytes, "flops": T * (row + kv) * (4 * c["norm"] + 3)}
    if c["op"] == "attend":
        n, ctx = _attend_lens(c)
        D, H, Hkv = c["dim"], c["heads"], c["kv_heads"]
        seen = n * ctx + n * (n + 1) // 2          # (row, key) pairs of one head
        nbytes = (int((n + ctx).sum()) * 2 * Hkv * D + int(n.sum()) * 2 * H * D * SIZE[c["dtype"]]
                  + 4 * int(((n + ctx + 15) // 16).sum()) + 8 * c["seqs"])
        return {"bytes": nbytes, "flops": 4 * D * H * int(seen.sum())}
    n = _verify_lens(c)
    es = SIZE[c["dtype"]]
    # the rows that the drawn token needs: one of the target, and one of the
    # drafts where a draft is rejected (about a third of them are)
    rows = float(c["seqs"])
    if c["draft_probs"]:
        rows += float((1 - (2 / 3) ** n).sum())
    return {"bytes": rows * c["vocab"] * es + 8 * int((n + 1).sum()), "flops": 3 * rows * c["vocab"]}


# ---- inputs ----------------------------------------------------------------

def _tensor(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def _codes(shape, scale, g):
    """E4M3 codes of standard normal keys or values, scale[j] for KV head j."""
    x = torch.randn(shape, device="cuda", generator=g, dtype=torch.float16)
    return (x / scale.half()[None, :, None, None]).clamp_(-448, 448).to(E4M3)


def _prepare_append(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    T, H, Hkv, D, R = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    dt = TYPES[c["dtype"]]
    n, first = _append_lens(c)
    start = _starts(n)
    s_of = np.repeat(np.arange(len(n)), n)
    pos = first[s_of] + np.arange(T) - start[s_of]
    # the blocks that the new tokens fall in, dealt out of a shuffled pool
    blocks = (first + n + BLOCK - 1) // BLOCK - first // BLOCK
    blocks[n == 0] = 0
    off = _starts(blocks)
    N = int(off[-1]) + int(off[-1]) // 4 + 8
    phys = r.permutation(N)
    block = phys[off[s_of] + pos // BLOCK - first[s_of] // BLOCK]
    slots = block * BLOCK + pos % BLOCK
    if c["padding"]:                               # padding tokens of a padded batch
        at = r.permutation(T)[: c["padding"]]
        slots[at] = -1
    P = int(pos.max()) + 1 + r.randint(0, 64)
    angle = np.arange(P)[:, None] * (1e4 ** (-np.arange(R // 2) / (R // 2)))[None, :]
    table = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
    qkv = torch.randn(T, (H + 2 * Hkv) * D, device="cuda", generator=g).mul_(1.7).to(dt)
    st = dict(case=c, qkv=qkv, table=_tensor(table), positions=_tensor(pos), slots=_tensor(slots),
              q=qkv[:, : H * D].view(T, H, D), k=qkv[:, H * D : (H + Hkv) * D].view(T, Hkv, D),
              v=qkv[:, (H + Hkv) * D :].view(T, Hkv, D), q_w=None, k_w=None,
              q_out=torch.zeros(T, H, D, device="cuda", dtype=dt))
    if c["norm"]:
        st["q_w"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
        st["k_w"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
    shape = (N, Hkv, BLOCK, D)
    if c["cache"] == "e4m3":
        st["k_s"] = torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01
        st["v_s"] = torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01
        st["kc"], st["vc"] = _codes(shape, st["k_s"], g), _codes(shape, st["v_s"], g)
    else:
        st["kc"] = torch.randn(shape, device="cuda", generator=g).to(TYPES[c["cache"]])
        st["vc"] = torch.randn(shape, device="cuda", generator=g).to(TYPES[c["cache"]])
    return st


def _prepare_attend(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    n, ctx = _attend_lens(c)
    L = n + ctx
    blocks = (L + BLOCK - 1) // BLOCK
    off = _starts(blocks)
    N = int(off[-1]) + int(off[-1]) // 8 + 4
    phys = r.permutation(N)
    col = np.arange(int(blocks.max()))[None, :]
    at = np.minimum(off[:-1, None] + col, N - 1)
    tables = np.where(col < blocks[:, None], phys[at], PAD).astype(np.int32)
    k_s = torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01
    v_s = torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01
    rows = int(n.sum())
    q = torch.randn(rows, H, D, device="cuda", generator=g).to(TYPES[c["dtype"]])
    return dict(case=c, q=q, out=torch.zeros_like(q), k_s=k_s, v_s=v_s,
                kc=_codes((N, Hkv, BLOCK, D), k_s, g), vc=_codes((N, Hkv, BLOCK, D), v_s, g),
                tables=_tensor(tables), lens=_tensor(L, torch.int32),
                starts=_tensor(_starts(n), torch.int32), most=int(n.max()), scale=D**-0.5,
                host_lens=L, host_starts=_starts(n))


def _prepare_verify(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = _verify_lens(c) + 1
    start = _starts(n)
    rows, V, dt = int(start[-1]), c["vocab"], TYPES[c["dtype"]]
    logits = torch.randn(rows, V, device="cuda", generator=g).mul_(3.0)
    target = logits.softmax(-1)
    gumbel = torch.rand(rows, V, device="cuda", generator=g).clamp_min_(1e-30).log_().neg_().log_().neg_()
    # row r of the target stands behind the draft of row r + 1
    logits = logits.roll(1, 0)
    if c["draft_probs"]:                           # the draft model: a blurred target
        logits.add_(torch.randn(rows, V, device="cuda", generator=g), alpha=0.8)
    tokens = (logits + gumbel).argmax(-1).to(torch.int32)
    draft = logits.softmax(-1).to(dt) if c["draft_probs"] else None
    return dict(case=c, target=target.to(dt), draft=draft, tokens=tokens,
                accept_u=torch.rand(rows, device="cuda", generator=g),
                sample_u=torch.rand(c["seqs"], device="cuda", generator=g),
                starts=_tensor(start, torch.int32), most=int(n.max()),
                out=torch.zeros(c["seqs"], int(n.max()), device="cuda", dtype=torch.int32),
                accepted=torch.zeros(c["seqs"], device="cuda", dtype=torch.int32))


def prepare(case, seed):
    return {"append": _prepare_append, "attend": _prepare_attend,
            "verify": _prepare_verify}[case["op"]](case, seed)


# ---- one pass --------------------------------------------------------------

def _rotated(x, w, st):
    """Heads of x [T, h, D] normalised and rotated, in 32 bits."""
    c = st["case"]
    R = c["rot"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    row = st["table"][st["positions"]][:, None, :]
    cos, sin = row[..., : R // 2], row[..., R // 2 :]
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _written(cache, rows, slots):
    """The rows written into their slots; a padding token repeats the write of
    the first token that has one."""
    ok = slots >= 0
    at = torch.where(ok, torch.arange(len(slots), device=slots.device), ok.int().argmax())
    slots, raw = slots[at], cache.view(torch.uint8) if cache.dtype == E4M3 else cache
    rows = rows.view(torch.uint8) if rows.dtype == E4M3 else rows
    raw[slots // BLOCK, :, slots % BLOCK] = rows[at]
    return cache


def _plain_append(st):
    dt = st["q"].dtype
    k, v = _rotated(st["k"], st["k_w"], st), st["v"]
    if st["case"]["cache"] == "e4m3":
        k = (k / st["k_s"][:, None]).clamp(-448, 448).to(E4M3)
        v = (v.float() / st["v_s"][:, None]).clamp(-448, 448).to(E4M3)
    q = _rotated(st["q"], st["q_w"], st).to(dt)
    kc, vc = _written(st["kc"], k.to(st["kc"].dtype), st["slots"]), _written(st["vc"], v, st["slots"])
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _gathered(cache, tables, scale):
    """[seqs, kv_heads, positions, dim] in 32 bits of every sequence's blocks."""
    t = tables.clamp(max=cache.shape[0] - 1)
    x = cache.view(torch.uint8)[t].view(E4M3).float() * scale[:, None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(st):
    c = st["case"]
    G, rows = c["heads"] // c["kv_heads"], st["q"].shape[0]
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(st["most"], device="cuda")
    at = (starts[:-1, None] + i).clamp(max=rows - 1)               # [S, most]
    q = st["q"][at].float().unflatten(2, (c["kv_heads"], G))       # [S, most, Hkv, G, D]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                     # [S, Hkv, G * most, D]
    k = _gathered(st["kc"], st["tables"], st["k_s"])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"])
    del k
    seen = (lens - n)[:, None] + i + 1                             # keys that a row sees
    key = torch.arange(x.shape[-1], device="cuda")
    hide = key >= seen[:, :, None]                                 # [S, most, keys]
    x = x.unflatten(2, (G, st["most"])).masked_fill_(hide[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True))
    o = torch.matmul(x.flatten(2, 3), _gathered(st["vc"], st["tables"], st["v_s"]))
    o = o.unflatten(2, (G, st["most"])).permute(0, 3, 1, 2, 4).flatten(2, 3)   # [S, most, H, D]
    r = torch.arange(rows, device="cuda")
    s = torch.searchsorted(starts, r, right=True) - 1
    return o[s, r - starts[s]].to(st["q"].dtype)


def _plain_verify(st):
    c = st["case"]
    starts, rows = st["starts"].long(), st["tokens"].shape[0]
    n = starts[1:] - starts[:-1]
    i = torch.arange(1, st["most"], device="cuda")
    at = (starts[:-1, None] + i).clamp(max=rows - 1)               # the drafts' rows
    tok = st["tokens"][at].long()
    p = st["target"][at - 1, tok].double()
    q = st["draft"][at, tok].double() if c["draft_probs"] else torch.ones_like(p)
    ok = (st["accept_u"][at].double() * q < p) & (i < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    rejected = a + 1 < n
    row = starts[:-1] + a
    p = st["target"][row].float()
    behind = (row + 1).clamp(max=rows - 1)
    if c["draft_probs"]:
        left = (p - st["draft"][behind].float()).clamp_min(0)
    else:
        left = p.scatter(1, st["tokens"][behind].long()[:, None], 0.0)
    w = torch.where(rejected[:, None], left, p)
    w = torch.where((w.amax(1) > 0)[:, None], w, p).double()
    total = w.sum(1, keepdim=True)
    drawn = (w.cumsum(1) <= st["sample_u"].double()[:, None] * total).sum(1)
    last = c["vocab"] - 1 - (w.flip(1) > 0).int().argmax(1)
    drawn = torch.minimum(drawn, last)
    j = torch.arange(st["most"], device="cuda")
    shifted = st["tokens"][(starts[:-1, None] + j + 1).clamp(max=rows - 1)].long()
    out = torch.where(j < a[:, None], shifted, torch.where(j == a[:, None], drawn[:, None], -1))
    return {"tokens": out.to(torch.int32), "accepted": a.to(torch.int32)}


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[c["op"]](st)
    from paged_kv_cache_151_gb300 import pa
    if c["op"] == "append":
        kw = dict(q_weight=st["q_w"], k_weight=st["k_w"], eps=EPS, interleaved=c["interleaved"])
        if c["cache"] == "e4m3":
            pa.pa_rope_and_cache_fp8(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                                     st["k_s"], st["v_s"], st["table"], st["positions"],
                                     st["slots"], **kw)
        else:
            pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                                 st["table"], st["positions"], st["slots"], **kw)
        return {"q": st["q_out"], "k_cache": st["kc"], "v_cache": st["vc"]}
    if c["op"] == "attend":
        pa.pa_decode_multi_fp8(st["out"], st["q"], st["kc"], st["vc"], st["k_s"], st["v_s"],
                               st["tables"], st["lens"], st["starts"], st["most"], st["scale"],
                               c["kv_heads"])
        return st["out"]
    pa.pa_verify_drafts(st["out"], st["accepted"], st["target"], st["draft"], st["tokens"],
                        st["accept_u"], st["sample_u"], st["starts"], st["most"])
    return {"tokens": st["out"], "accepted": st["accepted"]}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_append(st):
    c = st["case"]
    D, R = c["dim"], c["rot"]
    half = R // 2
    angle = st["table"].double()[st["positions"]]                  # [T, R]
    # the rotation as a sum of two products, x * A + swap(x) * B
    A = torch.ones(len(angle), 1, D, device="cuda", dtype=torch.float64)
    B = torch.zeros_like(A)
    j = torch.arange(half, device="cuda")
    lo, hi = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    A[:, 0, lo], A[:, 0, hi] = angle[:, :half], angle[:, :half]
    B[:, 0, lo], B[:, 0, hi] = -angle[:, half:], angle[:, half:]
    swap = torch.arange(D, device="cuda")
    swap[lo], swap[hi] = hi, lo

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        return x * A + x[..., swap] * B

    kc, vc = st["kc"].double(), st["vc"].double()
    live = (st["slots"] >= 0).nonzero().flatten()
    slot = st["slots"][live]
    k, v = turned(st["k"], st["k_w"])[live], st["v"].double()[live]
    if c["cache"] == "e4m3":
        k = (k / st["k_s"].double()[:, None]).clamp(-448, 448)
        v = (v / st["v_s"].double()[:, None]).clamp(-448, 448)
    kc[slot // BLOCK, :, slot % BLOCK] = k
    vc[slot // BLOCK, :, slot % BLOCK] = v
    return {"q": turned(st["q"], st["q_w"]), "k_cache": kc, "v_cache": vc}


def exact(case, seed):
    if case["op"] == "verify":
        return None                                # whole numbers
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    # one sequence and one head at a time
    c, G = case, case["heads"] // case["kv_heads"]
    out = torch.empty(st["q"].shape, device="cuda", dtype=torch.float64)
    for s, L in enumerate(st["host_lens"].tolist()):
        a, b = int(st["host_starts"][s]), int(st["host_starts"][s + 1])
        blocks = st["tables"][s, : -(-L // BLOCK)].long()
        k = st["kc"].view(torch.uint8)[blocks].view(E4M3).double() * st["k_s"].double()[:, None, None]
        v = st["vc"].view(torch.uint8)[blocks].view(E4M3).double() * st["v_s"].double()[:, None, None]
        k = k.permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, c["dim"])[:, :L]
        v = v.permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, c["dim"])[:, :L]
        sees = torch.arange(L, device="cuda") <= torch.arange(L - (b - a), L, device="cuda")[:, None]
        for h in range(c["heads"]):
            x = st["q"][a:b, h].double() @ k[h // G].T * st["scale"]
            x = torch.where(sees, x, -math.inf)
            out[a:b, h] = torch.softmax(x, -1) @ v[h // G]
    return out

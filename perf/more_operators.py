"""The operators of a serving step whose cache is held in 4 bits and whose
bookkeeping stays on the GPU, in their plain form and through the library's
entry points.

* ``write``: new keys and values into a cache of 4-bit floats, E2M1 codes with an
  E4M3 scale for every 16 of them (``pa_reshape_and_cache_fp4``), and the rows as
  the cache then holds them (``pa_gather_cache_fp4``);
* ``attend``: attention over that cache -- one token per sequence
  (``pa_decode_fp4``), split into partitions for long contexts
  (``pa_decode_partitioned_fp4``), several new tokens per sequence
  (``pa_decode_multi_fp4``);
* ``step``: block tables, sequence lengths, row ranges, positions and cache slots
  of a step built from the requests' lengths, blocks taken from a free list on
  the device (``pa_build_step``), and the blocks past a length given back, as
  after rejected drafts (``pa_trim_blocks``);
* ``logits``: penalties for repeated tokens, biases, masks of allowed tokens and
  temperature on logits, as probabilities or as logits (``pa_process_logits``).

Each case has an ``op`` and the sizes of one call.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
PAD = 2**31 - 1                    # block-table padding, never a valid block id
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # the cache write of a decode step of 256 sequences
        dict(name="write_decode_batch", op="write", seqs=256, tokens=256, far=4096, kv_heads=8,
             dim=128, padding=5, dtype="bf16", len_seed=1),
        # the cache write of long prompts
        dict(name="write_prompts", op="write", seqs=7, tokens=32001, far=60000, kv_heads=8,
             dim=128, padding=0, dtype="bf16", len_seed=2),
        # one request, one token: the latency of a step's attention
        dict(name="decode_one_request", op="attend", form="decode", seqs=1, rows_lo=1, rows_hi=1,
             ctx="range", ctx_lo=900, ctx_hi=1100, heads=32, kv_heads=8, dim=128, dtype="bf16",
             len_seed=3),
        # a decode step of the serving mix: lognormal context lengths
        dict(name="decode_serving_mix", op="attend", form="decode", seqs=256, rows_lo=1, rows_hi=1,
             ctx="mix", ctx_lo=1, ctx_hi=4095, heads=32, kv_heads=8, dim=128, dtype="bf16",
             len_seed=4),
        # long contexts, split into partitions of 512 tokens
        dict(name="decode_long_context", op="attend", form="partitioned", seqs=8, rows_lo=1,
             rows_hi=1, ctx="range", ctx_lo=32768, ctx_hi=131071, heads=64, kv_heads=8, dim=128,
             dtype="bf16", len_seed=5),
        # the serving mix verifying three drafts each
        dict(name="attend_verify_batch", op="attend", form="multi", seqs=256, rows_lo=4, rows_hi=4,
             ctx="mix", ctx_lo=1, ctx_hi=4092, heads=32, kv_heads=8, dim=128, dtype="bf16",
             len_seed=6),
        # prompt chunks of odd lengths over contexts of odd lengths
        dict(name="attend_chunks_odd", op="attend", form="multi", seqs=3, rows_lo=700, rows_hi=1500,
             ctx="range", ctx_lo=37, ctx_hi=16000, heads=32, kv_heads=8, dim=128, dtype="f16",
             len_seed=7),
        # a decode step's maps, five rows a sequence
        dict(name="step_decode_batch", op="step", seqs=256, new_lo=5, new_hi=5, ctx="mix",
             ctx_lo=0, ctx_hi=4000, width=256, short=False, spare=40, len_seed=8),
        # a step of prompts and decodes over many requests
        dict(name="step_many_requests", op="step", seqs=3001, new_lo=1, new_hi=21, ctx="mix",
             ctx_lo=0, ctx_hi=8000, width=512, short=True, spare=0, len_seed=9),
        # one request, four drafts, a small vocabulary: latency
        dict(name="logits_one_request", op="logits", seqs=1, rows_lo=5, rows_hi=5, vocab=32000,
             history=1500, bias=0, masked=False, penalties=True, probs=True, dtype="bf16",
             out="f32", len_seed=10),
        # a batch with 0 to 6 drafts each over a large odd vocabulary, grammar masks
        dict(name="logits_verify_batch", op="logits", seqs=64, rows_lo=1, rows_hi=7, vocab=131071,
             history=4000, bias=20, masked=True, penalties=True, probs=True, dtype="bf16",
             out="f32", len_seed=11),
        # one token each, processed logits in 32 bits
        dict(name="logits_decode_batch", op="logits", seqs=256, rows_lo=1, rows_hi=1, vocab=50021,
             history=600, bias=40, masked=True, penalties=True, probs=False, dtype="f32",
             out="f32", len_seed=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "step", "logits", "logits"])
    seed = rng.randrange(1, 10**6)
    heads, kv_heads = rng.choice([(32, 8), (16, 2), (8, 8), (16, 8), (64, 8), (8, 2)])
    if op == "write":
        tokens = _log(rng, 1, 30000)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 300)), tokens=tokens,
                    far=_log(rng, 16, 60000), kv_heads=rng.choice([1, 2, 8]),
                    dim=rng.choice([64, 96, 128]), padding=rng.choice([0, 0, tokens // 7]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), len_seed=seed)
    if op == "attend":
        dim, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "f16"])
        form = rng.choice(["decode", "partitioned", "multi", "multi"])
        c = dict(op=op, form=form, seqs=1, rows_lo=1, rows_hi=1, ctx="mix", ctx_lo=0, ctx_hi=4000,
                 heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, len_seed=seed)
        if form == "decode":
            c.update(seqs=_log(rng, 1, 250))
        elif form == "partitioned":
            hi = _log(rng, 600, 120000)
            c.update(seqs=rng.randrange(1, 8), ctx="range", ctx_lo=hi // 4, ctx_hi=hi)
        elif rng.random() < 0.5:                   # a batch verifying drafts
            lo = _log(rng, 1, 4)
            c.update(seqs=_log(rng, 1, 200), rows_lo=lo, rows_hi=lo + rng.randrange(0, 6))
        else:                                      # prompt chunks
            lo, ctx = _log(rng, 17, 700), _log(rng, 16, 8000)
            hi = lo + rng.randrange(0, lo)
            most = 3 * 1100 * 9000 * 32 * 128 // (hi * (ctx + hi) * heads * dim)
            c.update(seqs=max(1, min(rng.randrange(1, 5), most)), rows_lo=lo, rows_hi=hi,
                     ctx="range", ctx_lo=ctx // 3, ctx_hi=ctx)
        return c
    if op == "step":
        lo = rng.randrange(0, 3)
        return dict(op=op, seqs=_log(rng, 1, 2800), new_lo=lo, new_hi=lo + _log(rng, 1, 20),
                    ctx="mix", ctx_lo=0, ctx_hi=_log(rng, 100, 7000), width=500,
                    short=rng.random() < 0.3, spare=rng.randrange(0, 60), len_seed=seed)
    lo = rng.randrange(1, 5)
    vocab, dtype = _log(rng, 1000, 131071), rng.choice(["f32", "bf16", "f16"])
    hi = lo + rng.randrange(0, 4)
    return dict(op=op, seqs=max(1, min(_log(rng, 1, 200), 200 * 131071 // (vocab * hi))),
                rows_lo=lo, rows_hi=hi, vocab=vocab, history=_log(rng, 1, 5000),
                bias=rng.choice([0, 0, 30]), masked=rng.random() < 0.5,
                penalties=rng.random() < 0.8, probs=rng.random() < 0.7, dtype=dtype,
                out=rng.choice(["f32", dtype]), len_seed=seed)


# ---- the lengths of a case (they belong to the case, not to the inputs' seed) ----

def _write_lens(c):
    """(tokens, first position) of each sequence; tokens adds up to c["tokens"]."""
    r = np.random.RandomState(c["len_seed"])
    S, T = c["seqs"], c["tokens"]
    n = np.full(S, T // S, dtype=np.int64)
    n[: T % S] += 1
    shift = r.randint(0, max(1, n.min()), S)       # ragged: take from one, give to the next
    return n - shift + np.roll(shift, 1), r.randint(0, c["far"] + 1, S).astype(np.int64)


def _lens(c, lo, hi):
    """(rows, context before them) of each sequence."""
    r = np.random.RandomState(c["len_seed"])
    S = c["seqs"]
    n = r.randint(c[lo], c[hi] + 1, S).astype(np.int64)
    if c["ctx"] == "mix":                          # lognormal, median 350, sigma 1
        ctx = np.clip(np.round(np.exp(r.randn(S) + math.log(350.0))), c["ctx_lo"], c["ctx_hi"])
    else:
        ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, S)
    return n, ctx.astype(np.int64)


def _logits_lens(c):
    """(rows, tokens of the history, of these the prompt's) of each sequence."""
    r = np.random.RandomState(c["len_seed"])
    S = c["seqs"]
    n = r.randint(c["rows_lo"], c["rows_hi"] + 1, S).astype(np.int64)
    total = r.randint(1, c["history"] + 1, S).astype(np.int64)
    return n, total, (total * r.rand(S)).astype(np.int64)


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)])


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    c = case
    if c["op"] == "write":
        kv, live = c["kv_heads"] * c["dim"], c["tokens"] - c["padding"]
        return {"bytes": live * 2 * kv * (2 * SIZE[c["dtype"]] + 9 / 16) + 8 * c["tokens"],
                "flops": 4 * live * 2 * kv}
    if c["op"] == "attend":
        n, ctx = _lens(c, "rows_lo", "rows_hi")
        D, H, Hkv = c["dim"], c["heads"], c["kv_heads"]
        seen = n * ctx + n * (n + 1) // 2          # (row, key) pairs of one head
        nbytes = (int((n + ctx).sum()) * 2 * Hkv * D * 9 / 16 + int(n.sum()) * 2 * H * D * 2
                  + 4 * int(_blocks(n + ctx).sum()) + 8 * c["seqs"])
        return {"bytes": nbytes, "flops": 4 * D * H * int(seen.sum())}
    if c["op"] == "step":
        n, ctx = _lens(c, "new_lo", "new_hi")
        have = int(_blocks(ctx).sum())
        new = int(_blocks(n + ctx).sum()) - have
        # tables read and written, blocks from the free list into both tables and
        # back, a row's position and slot, a sequence's lengths, blocks and ids
        return {"bytes": 8 * have + 20 * new + 16 * (int(n.sum()) + c["spare"]) + 40 * c["seqs"],
                "flops": 4 * int(n.sum())}
    n, total, _ = _logits_lens(c)
    rows, V = int(n.sum()), c["vocab"]
    nbytes = rows * V * (SIZE[c["dtype"]] + SIZE[c["out"]] + c["masked"] / 8)
    nbytes += 4 * int(total.sum()) * c["penalties"] + 8 * c["bias"] * c["seqs"] + 40 * c["seqs"]
    return {"bytes": nbytes, "flops": 5 * rows * V}


# ---- inputs ----------------------------------------------------------------

def _tensor(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def _fp4_pool(N, Hkv, D, g):
    """Tiles of a 4-bit cache: codes of 16 rows (every magnitude about as likely,
    as normal values scaled by the largest of 16 have it), then their scales."""
    pool = torch.randint(0, 256, (N, Hkv, 9, D), device="cuda", generator=g, dtype=torch.uint8)
    size = torch.rand((N, Hkv, D), device="cuda", generator=g).mul_(0.9).add_(0.6)
    pool[:, :, 8] = size.to(E4M3).view(torch.uint8)
    return pool


def _prepare_write(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    T, Hkv, D = c["tokens"], c["kv_heads"], c["dim"]
    n, first = _write_lens(c)
    start = _starts(n)
    s_of = np.repeat(np.arange(len(n)), n)
    pos = first[s_of] + np.arange(T) - start[s_of]
    # the blocks that the new tokens fall in, dealt out of a shuffled pool
    blocks = _blocks(first + n) - first // BLOCK
    blocks[n == 0] = 0
    off = _starts(blocks)
    N = int(off[-1]) + int(off[-1]) // 4 + 8
    slots = r.permutation(N)[off[s_of] + pos // BLOCK - first[s_of] // BLOCK] * BLOCK + pos % BLOCK
    if c["padding"]:                               # padding tokens of a padded batch
        slots[r.permutation(T)[: c["padding"]]] = -1
    kv = torch.randn(T, 2 * Hkv * D, device="cuda", generator=g)
    # a few channels of the keys are far larger, as real keys have them
    kv[:, : Hkv * D] *= 1 + 6 * (torch.rand(Hkv * D, device="cuda", generator=g) < 0.03)
    kv = kv.to(TYPES[c["dtype"]])
    return dict(case=c, k=kv[:, : Hkv * D].view(T, Hkv, D), v=kv[:, Hkv * D :].view(T, Hkv, D),
                slots=_tensor(slots), kc=_fp4_pool(N, Hkv, D, g), vc=_fp4_pool(N, Hkv, D, g),
                k_s=torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01,
                v_s=torch.rand(Hkv, device="cuda", generator=g) * 0.01 + 0.01,
                k_out=torch.zeros(T, Hkv, D, device="cuda", dtype=kv.dtype),
                v_out=torch.zeros(T, Hkv, D, device="cuda", dtype=kv.dtype))


def _prepare_attend(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    n, ctx = _lens(c, "rows_lo", "rows_hi")
    L = n + ctx
    blocks = _blocks(L)
    off = _starts(blocks)
    N = int(off[-1]) + int(off[-1]) // 8 + 4
    phys = r.permutation(N)
    col = np.arange(int(blocks.max()))[None, :]
    at = np.minimum(off[:-1, None] + col, N - 1)
    tables = np.where(col < blocks[:, None], phys[at], PAD).astype(np.int32)
    rows = int(n.sum())
    q = torch.randn(rows, H, D, device="cuda", generator=g).to(TYPES[c["dtype"]])
    st = dict(case=c, q=q, out=torch.zeros_like(q),
              k_s=torch.rand(Hkv, device="cuda", generator=g) * 0.15 + 0.25,
              v_s=torch.rand(Hkv, device="cuda", generator=g) * 0.15 + 0.25,
              kc=_fp4_pool(N, Hkv, D, g), vc=_fp4_pool(N, Hkv, D, g), tables=_tensor(tables),
              lens=_tensor(L, torch.int32), starts=_tensor(_starts(n), torch.int32),
              most=int(n.max()), longest=int(L.max()), scale=D**-0.5, host_lens=L,
              host_starts=_starts(n))
    if own and c["form"] == "partitioned":
        from paged_kv_cache_151_gb300 import pa
        nbytes = pa.pa_decode_partitioned_workspace_size(c["seqs"], H, D, st["longest"], 512)
        st["workspace"] = torch.empty(nbytes, device="cuda", dtype=torch.uint8)
    return st


def _prepare_step(c, seed):
    r = np.random.RandomState(seed)
    S, W = c["seqs"], c["width"]
    n, ctx = _lens(c, "new_lo", "new_hi")
    R = S + S // 3 + 2                             # requests, of which the step runs S
    ids = r.permutation(R)[:S]
    held = np.zeros(R, dtype=np.int64)
    held[ids] = _blocks(ctx)
    idle = np.setdiff1d(np.arange(R), ids)
    held[idle] = np.arange(len(idle)) % 20
    off = _starts(held)
    need = int((_blocks(ctx + n) - _blocks(ctx)).sum())
    spare = need // 2 if c["short"] else need + 30   # a pool too small for all, or large enough
    N = int(off[-1]) + spare
    phys = r.permutation(N)
    col = np.arange(W)[None, :]
    tables = np.where(col < held[:, None], phys[np.minimum(off[:-1, None] + col, N - 1)], -1)
    T = int(n.sum()) + c["spare"]
    i32 = torch.int32
    free = np.concatenate([phys[off[-1] :], np.full(N - spare, -1)])   # room for every block
    return dict(case=c, num_blocks=N, request_tables=_tensor(tables, i32),
                request_blocks=_tensor(held, i32), ids=_tensor(ids, i32), ctx=_tensor(ctx, i32),
                new=_tensor(n, i32), free_blocks=_tensor(free, i32),
                free_count=_tensor([spare], i32),
                tables=torch.full((S, W), PAD, device="cuda", dtype=i32),
                lens=torch.zeros(S, device="cuda", dtype=i32),
                starts=torch.zeros(S + 1, device="cuda", dtype=i32),
                positions=torch.zeros(T, device="cuda", dtype=torch.int64),
                slots=torch.zeros(T, device="cuda", dtype=torch.int64))


def _prepare_logits(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed)
    S, V = c["seqs"], c["vocab"]
    n, total, prompt = _logits_lens(c)
    starts = _starts(n)
    rows = int(starts[-1])
    logits = torch.randn(rows, V, device="cuda", generator=g).mul_(3.0).to(TYPES[c["dtype"]])
    # tokens of a text repeat: a few frequent ones, many rare ones
    text = (V * r.rand(S, c["history"]) ** 4).astype(np.int64)
    st = dict(case=c, logits=logits, starts=_tensor(starts, torch.int32), host_starts=starts,
              tokens=_tensor((V * r.rand(rows) ** 4).astype(np.int64), torch.int32),
              host=(text, total, prompt), history=None, prompt_lens=None, history_lens=None,
              repetition=None, frequency=None, presence=None, bias_start=None, bias_tokens=None,
              bias_values=None, allowed=None, temperature=None,
              out=torch.zeros(rows, V, device="cuda", dtype=TYPES[c["out"]]))
    if c["penalties"]:
        st.update(history=_tensor(text, torch.int32), prompt_lens=_tensor(prompt, torch.int32),
                  history_lens=_tensor(total, torch.int32),
                  repetition=_tensor(1 + 0.4 * r.rand(S), torch.float32),
                  frequency=_tensor(0.5 * r.rand(S), torch.float32),
                  presence=_tensor(0.8 * r.rand(S), torch.float32))
    if c["bias"]:
        m = r.randint(0, c["bias"] + 1, S)
        k = int(m.sum())
        st.update(bias_start=_tensor(_starts(m), torch.int32),
                  bias_tokens=_tensor(r.randint(0, V, k), torch.int32),
                  bias_values=_tensor(4 * r.randn(k), torch.float32))
    if c["masked"]:
        # a grammar allows a few tokens here, most of them there, now and then nothing
        share = r.choice([0.0, 0.001, 0.05, 0.9, 1.0], rows, p=[0.02, 0.25, 0.25, 0.28, 0.2])
        share = _tensor(share, torch.float32)[:, None]
        words = torch.zeros(rows, (V + 31) // 32, device="cuda", dtype=torch.int32)
        for bit in range(32):
            allow = torch.rand(words.shape, device="cuda", generator=g) < share
            words |= allow.int() << bit
        st["allowed"] = words
    tau = np.where(r.rand(S) < 0.1, 0.0, 0.5 + r.rand(S))   # some requests are greedy
    if not c["probs"]:
        tau = np.maximum(tau, 0.5)
    st["temperature"] = _tensor(tau, torch.float32)
    return st


def prepare(case, seed):
    return {"write": _prepare_write, "attend": _prepare_attend, "step": _prepare_step,
            "logits": _prepare_logits}[case["op"]](case, seed)


# ---- one pass --------------------------------------------------------------

def _fp4_of(x, scale):
    """Codes (0 to 15) and scales (as floats) of x [T, Hkv, D]: E2M1 of what the
    head's scale and an E4M3 scale for every 16 elements leave."""
    y = (x.float() / scale[:, None]).unflatten(-1, (-1, 16))
    top = y.abs().amax(-1, keepdim=True)
    size = (top / torch.full_like(top, 6.0)).clamp(max=448).to(E4M3).float()
    z = torch.where(size > 0, y / size, 0.0)
    a = z.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5))
    return (code + 8 * torch.signbit(z).int()).flatten(-2), size.squeeze(-1)


def _plain_write(st):
    live = (st["slots"] >= 0).nonzero().flatten()
    slot = st["slots"][live]
    block, row = slot // BLOCK, slot % BLOCK
    out = {}
    for name in ("k", "v"):
        x, cache, scale = st[name], st[name + "c"], st[name + "_s"]
        N, Hkv, _, D = cache.shape
        code, size = _fp4_of(x[live], scale)
        codes, sizes = cache[:, :, :8].view(N, Hkv, -1), cache[:, :, 8]   # 16 rows of each
        col, head = torch.arange(D // 2, device="cuda"), torch.arange(Hkv, device="cuda")[:, None]
        at = (block[:, None, None], head)
        codes[(*at, row[:, None, None] * (D // 2) + col)] = (code[..., ::2] + 16 * code[..., 1::2]).byte()
        col = torch.arange(D // 16, device="cuda")
        sizes[(*at, row[:, None, None] * (D // 16) + col)] = size.to(E4M3).view(torch.uint8)
        # the rows as they are held now
        lut = torch.tensor(E2M1 + [-m for m in E2M1], device="cuda")
        y = (lut[code.long()].unflatten(-1, (-1, 16)) * size[..., None]).flatten(-2) * scale[:, None]
        out[name] = st[name + "_out"].index_copy_(0, live, y.to(x.dtype))
    return out


def _gathered(cache, tables, scale):
    """[seqs, kv_heads, positions, dim] in 32 bits of every sequence's blocks."""
    D = cache.shape[-1]
    t = cache[tables.clamp(max=cache.shape[0] - 1)]                # [S, blocks, Hkv, 9, D]
    codes = t[:, :, :, :8].reshape(*t.shape[:3], BLOCK, D // 2)
    size = t[:, :, :, 8].contiguous().view(E4M3).float().unflatten(-1, (BLOCK, D // 16))
    lut = torch.tensor(E2M1 + [-x for x in E2M1], device="cuda")
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    x = x.unflatten(-1, (D // 16, 16)).mul_(size.mul_(scale[:, None, None])[..., None]).flatten(-2)
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


def _plain_step(st):
    ids, ctx, new = st["ids"].long(), st["ctx"].long(), st["new"].long()
    S, W = st["tables"].shape
    T = st["slots"].shape[0]
    rt, held, count = st["request_tables"], st["request_blocks"][ids].long(), st["free_count"].long()
    starts = torch.cat([ids.new_zeros(1), new.cumsum(0)])
    want = _blocks(ctx + new)
    need = (want - held).clamp_min(0)
    end = need.cumsum(0)
    granted = (need == 0) | (end <= count)
    taken = torch.where(granted, need, 0)
    # entry held + i of a request takes the (blocks before it + i)-th from the
    # list's end
    col = torch.arange(W, device="cuda")
    table = rt[ids].long()
    i = col - held[:, None]
    take = (i >= 0) & (i < taken[:, None])
    at = (count - 1 - (end - need)[:, None] - i).clamp(0, st["free_blocks"].shape[0] - 1)
    table = torch.where(take, st["free_blocks"].long()[at], table)
    rt[ids] = table.int()
    shown = (col < want[:, None]) & granted[:, None]
    st["tables"].copy_(torch.where(shown, table, st["tables"]))
    st["lens"].copy_(torch.where(granted, ctx + new, 0))
    st["starts"].copy_(starts)
    row = torch.arange(T, device="cuda")
    s = (torch.searchsorted(starts, row, right=True) - 1).clamp(max=S - 1)
    live = row < starts[-1]
    pos = torch.where(live, ctx[s] + row - starts[s], 0)
    slot = table[s, (pos // BLOCK).clamp(max=W - 1)] * BLOCK + pos % BLOCK
    st["positions"].copy_(pos)
    st["slots"].copy_(torch.where(live & granted[s], slot, -1))
    # blocks past the context go back, the first sequence's first one last
    held = held + taken
    keep = torch.minimum(held, _blocks(ctx))
    back = held - keep
    count = count - taken.sum()
    i = col - keep[:, None]
    give = (i >= 0) & (i < back[:, None])
    at = count + back.sum() - 1 - (back.cumsum(0) - back)[:, None] - i
    st["free_blocks"][at[give]] = table[give].int()
    st["free_count"].copy_(count + back.sum())
    st["request_blocks"][ids] = keep.int()
    return _step_outputs(st)


def _step_outputs(st):
    return {k: st[k] for k in ("tables", "lens", "starts", "positions", "slots", "request_tables",
                               "request_blocks", "free_blocks", "free_count")}


def _plain_logits(st):
    c = st["case"]
    rows, V = st["logits"].shape
    starts = st["starts"].long()
    row = torch.arange(rows, device="cuda")
    s = torch.searchsorted(starts, row, right=True) - 1
    x = st["logits"].float()
    if c["penalties"]:
        text = st["history"].long()
        i = torch.arange(text.shape[1], device="cuda")
        there = i < st["history_lens"][:, None]
        prompt = i < st["prompt_lens"][:, None]
        said = torch.zeros(len(text), V, device="cuda")
        said.scatter_add_(1, text, (there & ~prompt).float())
        asked = torch.zeros(len(text), V, device="cuda")
        asked.scatter_add_(1, text, (there & prompt).float())
        count, seen = said[s], asked[s] > 0
        for back in range(c["rows_hi"] - 1):       # a row counts the drafts before it
            at = row - back
            mine = (at > starts[s]).float()[:, None]
            count.scatter_add_(1, st["tokens"].long()[at.clamp_min(0)][:, None], mine)
        seen = seen | (count > 0)
        theta = st["repetition"][s][:, None]
        x = torch.where(seen, torch.where(x > 0, x / theta, x * theta), x)
        x = x - st["frequency"][s][:, None] * count - st["presence"][s][:, None] * (count > 0)
    if c["bias"]:
        b = torch.zeros(c["seqs"], V, device="cuda")
        e = torch.arange(len(st["bias_tokens"]), device="cuda")
        of = torch.searchsorted(st["bias_start"].long(), e, right=True) - 1
        b.index_put_((of, st["bias_tokens"].long()), st["bias_values"], accumulate=True)
        x = x + b[s]
    if c["masked"]:
        v = torch.arange(V, device="cuda")
        allow = (st["allowed"][:, v // 32] >> (v % 32)) & 1
        x = torch.where(allow == 1, x, -math.inf)
    tau = st["temperature"][s][:, None]
    x = torch.where(tau > 0, x / tau.clamp_min(1e-30), x)
    if not c["probs"]:
        return x.to(st["out"].dtype)
    top = x.amax(1, keepdim=True)
    e = (x - torch.where(top > -math.inf, top, 0.0)).exp()
    p = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    first = torch.where(x == top, torch.arange(V, device="cuda"), V).amin(1, keepdim=True)
    best = (torch.arange(V, device="cuda") == first) & (top > -math.inf)
    return torch.where(tau > 0, p, best.float()).to(st["out"].dtype)


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"write": _plain_write, "attend": _plain_attend, "step": _plain_step,
                "logits": _plain_logits}[c["op"]](st)
    from paged_kv_cache_151_gb300 import pa
    if c["op"] == "write":
        pa.pa_reshape_and_cache_fp4(st["k"], st["v"], st["kc"], st["vc"], st["k_s"], st["v_s"],
                                    st["slots"])
        pa.pa_gather_cache_fp4(st["k_out"], st["v_out"], st["kc"], st["vc"], st["k_s"], st["v_s"],
                               st["slots"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if c["op"] == "attend":
        args = (st["out"], st["q"], st["kc"], st["vc"], st["k_s"], st["v_s"], st["tables"],
                st["lens"])
        if c["form"] == "decode":
            pa.pa_decode_fp4(*args, st["scale"], c["kv_heads"])
        elif c["form"] == "partitioned":
            pa.pa_decode_partitioned_fp4(*args, st["scale"], c["kv_heads"], 512, st["longest"],
                                         st["workspace"])
        else:
            pa.pa_decode_multi_fp4(*args, st["starts"], st["most"], st["scale"], c["kv_heads"])
        return st["out"]
    if c["op"] == "step":
        pa.pa_build_step(st["tables"], st["lens"], st["starts"], st["positions"], st["slots"],
                         st["request_tables"], st["request_blocks"], st["ids"], st["ctx"],
                         st["new"], st["free_blocks"], st["free_count"], st["num_blocks"])
        pa.pa_trim_blocks(st["request_tables"], st["request_blocks"], st["ids"], st["ctx"],
                          st["free_blocks"], st["free_count"])
        return _step_outputs(st)
    pa.pa_process_logits(st["out"], st["logits"], st["starts"], tokens=st["tokens"],
                         history=st["history"], prompt_lens=st["prompt_lens"],
                         history_lens=st["history_lens"], repetition=st["repetition"],
                         frequency=st["frequency"], presence=st["presence"],
                         bias_start=st["bias_start"], bias_tokens=st["bias_tokens"],
                         bias_values=st["bias_values"], allowed=st["allowed"],
                         temperature=st["temperature"], probs=c["probs"])
    return st["out"]


# ---- the definition in 64 bits ----------------------------------------------

def _exact_write(st):
    """Nearest of the representable values, found among them all; the scale of a
    group is the cache's own E4M3 number of the 32-bit quotient, as defined."""
    out = {}
    grid = torch.tensor(sorted({s * m for m in E2M1 for s in (1, -1)}), device="cuda",
                        dtype=torch.float64)
    for name in ("k", "v"):
        scale = st[name + "_s"]
        y = (st[name].float() / scale[:, None]).unflatten(-1, (-1, 16))
        six = torch.full_like(y[..., :1], 6.0)
        size = torch.minimum(y.abs().amax(-1, keepdim=True) / six, six * 0 + 448).to(E4M3).double()
        z = (y / size.float()).nan_to_num(0.0, 6.0, -6.0).double()
        mid = (grid[1:] + grid[:-1]) / 2
        at = torch.searchsorted(mid, z)            # ties go down here ...
        tie = (at < len(mid)) & (mid[at.clamp(max=len(mid) - 1)] == z)
        low = grid[at]
        up = grid[(at + 1).clamp(max=len(grid) - 1)]
        # ... and to the neighbour with the even code
        odd = (low.abs() == 0.5) | (low.abs() == 1.5) | (low.abs() == 3) | (low.abs() == 6)
        value = torch.where(tie & odd, up, low) * size
        value = torch.where(size > 0, value, 0.0).flatten(-2) * scale.double()[:, None]
        live = (st["slots"] >= 0)[:, None, None]
        out[name] = torch.where(live, value, st[name + "_out"].double())
    return out


def _exact_rows(cache, blocks, scale, L):
    """[kv_heads, L, dim] of one sequence."""
    N, Hkv, _, D = cache.shape
    raw = cache[blocks]
    codes = raw[:, :, :8].reshape(-1, Hkv, BLOCK, D // 2).permute(1, 0, 2, 3).reshape(Hkv, -1, D // 2)
    size = raw[:, :, 8].contiguous().view(E4M3).double()
    size = size.reshape(-1, Hkv, BLOCK, D // 16).permute(1, 0, 2, 3).reshape(Hkv, -1, D // 16)
    x = torch.empty(Hkv, codes.shape[1], D, device="cuda", dtype=torch.float64)
    for half, code in enumerate((codes.int() % 16, codes.int() // 16)):
        e, m = (code % 8) // 2, (code % 2).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double())
        x[..., half::2] = torch.where(code >= 8, -mag, mag)
    return (x * size.repeat_interleave(16, -1) * scale.double()[:, None, None])[:, :L]


def _exact_attend(st):
    # one sequence and one head at a time
    c = st["case"]
    G = c["heads"] // c["kv_heads"]
    out = torch.empty(st["q"].shape, device="cuda", dtype=torch.float64)
    for s, L in enumerate(st["host_lens"].tolist()):
        a, b = int(st["host_starts"][s]), int(st["host_starts"][s + 1])
        blocks = st["tables"][s, : -(-L // BLOCK)].long()
        k = _exact_rows(st["kc"], blocks, st["k_s"], L)
        v = _exact_rows(st["vc"], blocks, st["v_s"], L)
        sees = torch.arange(L, device="cuda") <= torch.arange(L - (b - a), L, device="cuda")[:, None]
        for h in range(c["heads"]):
            x = st["q"][a:b, h].double() @ k[h // G].T * st["scale"]
            x = torch.where(sees, x, -math.inf)
            out[a:b, h] = torch.softmax(x, -1) @ v[h // G]
    return out


def _exact_logits(st):
    """One row at a time."""
    c = st["case"]
    V = c["vocab"]
    text, total, prompt = st["host"]
    tokens = st["tokens"].cpu().numpy()
    out = torch.empty(st["logits"].shape, device="cuda", dtype=torch.float64)
    f = {k: None if st[k] is None else st[k].double().cpu().numpy()
         for k in ("repetition", "frequency", "presence", "bias_values", "temperature")}
    if c["bias"]:
        bs, bt = st["bias_start"].cpu().numpy(), st["bias_tokens"].cpu().numpy()
    if c["masked"]:
        bits = st["allowed"].cpu().numpy().view(np.uint32)
    for s in range(c["seqs"]):
        for r in range(int(st["host_starts"][s]), int(st["host_starts"][s + 1])):
            add = np.zeros(V)
            if c["penalties"]:
                drafts = tokens[int(st["host_starts"][s]) + 1 : r + 1]
                said = np.concatenate([text[s, prompt[s] : total[s]], drafts])
                n = np.bincount(said, minlength=V)
                seen = n + np.bincount(text[s, : prompt[s]], minlength=V) > 0
                add -= f["frequency"][s] * n + f["presence"][s] * (n > 0)
            if c["bias"]:
                np.add.at(add, bt[bs[s] : bs[s + 1]], f["bias_values"][bs[s] : bs[s + 1]])
            x = st["logits"][r].double()
            if c["penalties"]:
                by = torch.where(x > 0, 1 / f["repetition"][s], f["repetition"][s])
                x = x * torch.where(_tensor(seen), by, 1.0)
            x = x + _tensor(add)
            if c["masked"]:
                allow = np.unpackbits(bits[r].view(np.uint8), bitorder="little")[:V]
                x[~_tensor(allow.astype(bool))] = -math.inf
            if f["temperature"][s] > 0:
                x = x / f["temperature"][s]
            if c["probs"]:
                if not bool((x > -math.inf).any()):
                    x = torch.zeros_like(x)
                elif f["temperature"][s] > 0:
                    x = torch.softmax(x, 0)
                else:
                    first = int((x == x.max()).nonzero()[0])
                    x = torch.zeros_like(x)
                    x[first] = 1
            out[r] = x
    return out


def exact(case, seed):
    if case["op"] == "step":
        return None                                # whole numbers
    return {"write": _exact_write, "attend": _exact_attend,
            "logits": _exact_logits}[case["op"]](prepare(case, seed))

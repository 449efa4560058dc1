"""Block tables and maps of a step built on the GPU, and blocks given back, equal to
a sequential form."""
import numpy as np
import pytest
import torch

import plain_serving as ps

pytestmark = pytest.mark.gpu


class State:
    def __init__(self, seed, R, width, held, spare, capacity=None):
        r = np.random.default_rng(seed)
        held = np.asarray(held)
        total = int(held.sum()) + spare
        phys = r.permutation(total)
        self.st = dict(request_tables=np.full((R, width), -3, np.int64), request_blocks=held.copy(),
                       free_blocks=np.concatenate([phys[held.sum():], np.full(total - spare if capacity
                                                   is None else capacity - spare, -9)]),
                       free_count=np.array([spare]))
        at = 0
        for i in range(R):
            self.st["request_tables"][i, :held[i]] = phys[at:at + held[i]]
            at += held[i]
        self.num_blocks = total
        self.g = {k: torch.as_tensor(v, dtype=torch.int32, device="cuda") for k, v in self.st.items()}

    def same(self):
        for k, v in self.st.items():
            assert np.array_equal(self.g[k].cpu().numpy(), v), k


def i32(x):
    return None if x is None else torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def both(pa, S, ids, ctx, new, width, num_rows, free=True, flags=0):
    """The call and the plain form on the same state; everything equal."""
    B = len(ctx)
    o = dict(tables=torch.full((B, width), -7, dtype=torch.int32, device="cuda"),
             lens=torch.full((B,), 99, dtype=torch.int32, device="cuda"),
             starts=torch.full((B + 1,), 99, dtype=torch.int32, device="cuda"),
             positions=torch.full((num_rows,), 99, dtype=torch.int64, device="cuda"),
             slots=torch.full((num_rows,), 99, dtype=torch.int64, device="cuda"))
    g = S.g
    pa.pa_device_error(clear=True)
    pa.pa_build_step(o["tables"], o["lens"], o["starts"], o["positions"], o["slots"],
                     g["request_tables"], g["request_blocks"], i32(ids), i32(ctx), i32(new),
                     g["free_blocks"] if free else None, g["free_count"] if free else None,
                     S.num_blocks)
    st = S.st if free else dict(S.st, free_blocks=None)
    want = ps.build_step(st, ids, ctx, new, width, num_rows, S.num_blocks)
    for k in o:
        assert np.array_equal(o[k].cpu().numpy(), want[k]), k
    S.same()
    assert pa.pa_device_error(clear=True) == want["flags"]
    assert want["flags"] & flags == flags
    return o


@pytest.mark.parametrize("B", [1, 2, 31, 300, 1025, 5000])
def test_build_and_trim(cuda_lib, B):
    r = np.random.default_rng(B)
    R, width = B + B // 3 + 1, 40
    ids = r.permutation(R)[:B]
    ctx, new = r.integers(0, 500, B), r.integers(0, 30, B)
    held = r.integers(0, 5, R)
    held[ids] = -(-ctx // 16) + (r.random(B) < 0.2)    # some hold one more: drafts were rejected
    S = State(B, R, width, held, int(3 * B + 5))
    before = {k: v.copy() for k, v in S.st.items()}
    both(cuda_lib, S, ids, ctx, new, 34, int(new.sum()) + 9)
    # trimmed to what was accepted
    keep = ctx + r.integers(0, 30, B) % (new + 1)
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], i32(ids), i32(keep),
                            S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, ids, keep) == 0
    S.same()
    # nothing is lost or named twice
    st = S.st
    owned = [int(b) for i in range(R) for b in st["request_tables"][i, :st["request_blocks"][i]]]
    free = [int(b) for b in st["free_blocks"][:st["free_count"][0]]]
    assert sorted(owned + free) == list(range(S.num_blocks))
    assert before["request_tables"].shape == st["request_tables"].shape
    assert cuda_lib.pa_device_error(clear=True) == 0


def test_a_step_trimmed_to_its_context_leaves_the_list(cuda_lib):
    ctx, new = np.array([0, 16, 17, 250]), np.array([40, 1, 16, 100])
    S = State(1, 4, 30, -(-ctx // 16), 30)
    free = S.st["free_blocks"].copy()
    both(cuda_lib, S, None, ctx, new, 30, 200)
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], None, i32(ctx),
                            S.g["free_blocks"], S.g["free_count"])
    ps.trim(S.st, None, ctx)
    S.same()
    assert np.array_equal(S.st["free_blocks"], free) and S.st["free_count"][0] == 30


def test_one_row_each_by_default(cuda_lib):
    ctx = np.array([0, 15, 16, 31, 32])
    both(cuda_lib, State(2, 5, 4, -(-ctx // 16), 10), None, ctx, None, 4, 5)


def test_long_tables_and_long_prompts(cuda_lib):
    """Tables past what one warp copies, a prompt of thousands of rows."""
    ctx, new = np.array([40000, 3, 9000, 0]), np.array([1, 5000, 700, 0])
    S = State(3, 6, 2600, [2500, 1, 563, 0, 7, 0], 600)
    both(cuda_lib, S, [0, 1, 2, 5], ctx, new, 2550, 6000)


def test_a_list_too_short_refuses_those_that_need_more(cuda_lib):
    ctx = np.array([16, 30, 16, 5, 16, 0])
    new = np.array([1, 1, 40, 1, 1, 1])                # need 1, 0, 3, 0, 1, 1
    S = State(4, 6, 10, -(-ctx // 16), 3)
    o = both(cuda_lib, S, None, ctx, new, 10, 50, flags=cuda_lib.PA_DEVERR_NO_BLOCKS)
    assert o["lens"].tolist() == [17, 31, 0, 6, 0, 0]


def test_complete_tables_without_a_list(cuda_lib):
    ctx = np.array([20, 16, 100])
    S = State(5, 3, 10, [2, 1, 8], 0)
    o = both(cuda_lib, S, None, ctx, [5, 1, 20], 10, 26, free=False, flags=cuda_lib.PA_DEVERR_NO_BLOCKS)
    assert o["lens"].tolist() == [25, 0, 120]


def test_bad_ids_and_lengths_are_refused(cuda_lib):
    ctx = np.array([5, -1, 5, 5, 170, 5, 5])
    new = np.array([1, 1, -4, 1, 1, 1, 3])
    S = State(6, 8, 10, [1, 1, 1, 1, 9, 1, 1, 0], 20)
    both(cuda_lib, S, [0, 1, 2, 8, 4, -1, 6], ctx, new, 10, 12, flags=cuda_lib.PA_DEVERR_SEQ_LEN)
    S.st["request_blocks"][3] = 11                     # more than a table holds
    S.g["request_blocks"][3] = 11
    both(cuda_lib, S, [3, 0], [5, 6], [1, 1], 10, 12, flags=cuda_lib.PA_DEVERR_SEQ_LEN)


def test_rows_past_the_arrays_are_refused(cuda_lib):
    S = State(7, 3, 10, [1, 1, 1], 9)
    both(cuda_lib, S, None, [3, 4, 5], [4, 4, 1], 10, 7, flags=cuda_lib.PA_DEVERR_SEQ_LEN)


def test_bad_blocks_are_flagged(cuda_lib):
    S = State(8, 2, 4, [1, 1], 2)
    for t, v in ((S.st["request_tables"], 77), (S.g["request_tables"], 77)):
        t[1, 0] = v
    both(cuda_lib, S, None, [3, 4], [2, 2], 4, 4, flags=cuda_lib.PA_DEVERR_BLOCK_ID)


def test_bad_counts_touch_nothing_outside(cuda_lib):
    pa = cuda_lib
    for count in (-5, 1000):
        S = State(9, 2, 4, [1, 1], 2)
        S.g["free_count"].fill_(count)
        pa.pa_device_error(clear=True)
        pa.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], None, i32([0, 0]),
                          S.g["free_blocks"], S.g["free_count"])
        assert pa.pa_device_error(clear=True) == pa.PA_DEVERR_BLOCK_ID
        assert S.g["free_count"].item() == count
        S.g["free_count"].fill_(2)
        S.same()


def test_blocks_that_do_not_fit_stay(cuda_lib):
    S = State(10, 2, 8, [5, 4], 3, capacity=9)
    cuda_lib.pa_device_error(clear=True)
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], None, i32([0, 0]),
                            S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, None, [0, 0]) == 0x1
    S.same()
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_BLOCK_ID


def test_trim_with_bad_entries(cuda_lib):
    S = State(11, 4, 8, [5, 4, 2, 1], 3)
    cuda_lib.pa_device_error(clear=True)
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], i32([0, 9, 2, -1, 1]),
                            i32([17, 0, -3, 0, 0]), S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, [0, 9, 2, -1, 1], [17, 0, -3, 0, 0]) == 0x2
    S.same()
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN


@pytest.mark.parametrize("B", [3, 900, 3000])
def test_a_request_named_twice_refuses_the_call(cuda_lib, B):
    """Else its blocks would be taken, or given back, twice."""
    r = np.random.default_rng(B)
    ids = r.permutation(B + 5)[:B]
    S = State(14, B + 5, 6, r.integers(0, 4, B + 5), 4 * B)
    ids[B - 1] = ids[B // 3]
    o = both(cuda_lib, S, ids, r.integers(0, 40, B), r.integers(0, 3, B), 6, 3 * B,
             flags=cuda_lib.PA_DEVERR_SEQ_LEN)
    assert not o["lens"].any() and (o["slots"] == -1).all()
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], i32(ids), i32(np.zeros(B)),
                            S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, ids, np.zeros(B)) == 0x2
    S.same()
    assert cuda_lib.pa_device_error(clear=True) == cuda_lib.PA_DEVERR_SEQ_LEN


@pytest.mark.parametrize("B", [4, 2000])
def test_padded_entries(cuda_lib, B):
    r = np.random.default_rng(B)
    ids = np.where(np.arange(B) % 4 == 1, -1, np.arange(B))
    S = State(15, B, 6, np.full(B, 2), 4 * B)
    o = both(cuda_lib, S, ids, r.integers(17, 33, B), np.where(ids < 0, 0, r.integers(1, 5, B)), 6, 5 * B)
    assert (o["lens"].cpu().numpy()[ids < 0] == 0).all()
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], i32(ids), i32(np.full(B, 16)),
                            S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, ids, np.full(B, 16)) == 0
    S.same()
    assert cuda_lib.pa_device_error(clear=True) == 0


def test_the_most_sequences_and_requests(cuda_lib):
    """65535 sequences of 2^19 requests: the largest records and map of named ones."""
    R, B = 1 << 19, 65535
    r = np.random.default_rng(16)
    held = np.zeros(R, int)
    ids = r.permutation(R)[:B]
    held[ids] = r.integers(0, 3, B)
    S = State(16, R, 3, held, B)
    ctx = np.maximum(held[ids] * 16 - r.integers(0, 16, B), 0)
    new = (r.random(B) < 0.5).astype(int)
    both(cuda_lib, S, ids, ctx, new, 3, B)
    cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], i32(ids), i32(ctx),
                            S.g["free_blocks"], S.g["free_count"])
    assert ps.trim(S.st, ids, ctx) == 0
    S.same()


def test_an_empty_step(cuda_lib):
    S = State(12, 2, 4, [1, 1], 2)
    both(cuda_lib, S, np.zeros(0, int), np.zeros(0, int), np.zeros(0, int), 4, 5)


def test_a_loop_of_steps_captured_and_replayed(cuda_lib):
    """Contexts grow on the device by what a step accepts; one graph, many replays."""
    B, width = 40, 30
    r = np.random.default_rng(13)
    ctx = r.integers(0, 60, B)
    S = State(13, B, width, -(-ctx // 16), 900)
    new = np.full(B, 5)
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    dctx, dnew = i32(ctx), i32(new)
    o = [torch.zeros(B, width, dtype=torch.int32, device="cuda"),
         torch.zeros(B, dtype=torch.int32, device="cuda"),
         torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
         torch.zeros(5 * B, dtype=torch.int64, device="cuda"),
         torch.zeros(5 * B, dtype=torch.int64, device="cuda")]

    def step():
        cuda_lib.pa_build_step(*o, S.g["request_tables"], S.g["request_blocks"], None, dctx, dnew,
                               S.g["free_blocks"], S.g["free_count"], S.num_blocks)
        dctx.add_(acc)
        cuda_lib.pa_trim_blocks(S.g["request_tables"], S.g["request_blocks"], None, dctx,
                                S.g["free_blocks"], S.g["free_count"])

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for _ in range(25):
        a = r.integers(1, 6, B)
        acc.copy_(i32(a))
        g.replay()
        torch.cuda.synchronize()
        want = ps.build_step(S.st, None, ctx, new, width, 5 * B, S.num_blocks)
        assert want["flags"] == 0
        for got, k in zip(o[1:], ("lens", "starts", "positions", "slots")):
            assert np.array_equal(got.cpu().numpy(), want[k]), k
        ctx = ctx + a
        ps.trim(S.st, None, ctx)
        S.same()
    assert cuda_lib.pa_device_error(clear=True) == 0

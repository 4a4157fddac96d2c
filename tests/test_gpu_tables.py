"""Block tables grown and shortened on the GPU against the oracle: whole
numbers, so every output is equal."""
import numpy as np
import pytest
import torch

from oracle import tables as T
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def make_tables(rng, lens, W, extra):
    """A table over the lengths, the free stack behind it and the pool's size."""
    need = [-(-int(L) // 16) for L in lens]
    N = sum(need) + extra
    perm = rng.permutation(N).astype(np.int32)
    table = np.full((len(lens), W), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].copy(), N


def run_extend(pq, lens, new, table, stack, count, N, num_tokens, in_place=False, **kw):
    sl, bt = dev(lens), dev(table)
    fc = dev([count])
    slo, fco = (sl, fc) if in_place else (torch.full_like(sl, -7), torch.full_like(fc, -7))
    slots = torch.full((num_tokens,), -9, dtype=torch.int64, device="cuda")
    pos = torch.full((num_tokens,), -9, dtype=torch.int32, device="cuda")
    off = torch.full((len(lens) + 1,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pq.extend_block_tables(sl, dev(new), bt, dev(stack), fc, N, slo, fco, slots, pos, off,
                           status=status, **kw)
    return slo, fco, bt, slots, pos, off, status


def check_extend(pq, lens, new, table, stack, count, N, num_tokens, in_place=False):
    got = run_extend(pq, lens, new, table, stack, count, N, num_tokens, in_place)
    want = T.extend(lens, new, table, stack, count, N, num_tokens)
    names = ("seq_lens", "free_count", "block_table", "slots", "positions", "offsets", "status")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w), name
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,cached,new,pad", [
    (1, 1, 1, 0), (1, 0, 1, 63), (1, 16, 1, 0), (3, 40, 5, 1), (8, 3000, 1, 0), (33, 500, 8, 27),
    (511, 100, 17, 5), (513, 60, 40, 0), (2048, 70, 5, 11), (7, 0, 3001, 100)])
def test_extend(B, cached, new, pad, in_place):
    pq = require_gpu()
    rng = np.random.default_rng(B * 31 + new)
    lens = rng.integers(0, cached, B, endpoint=True)
    add = rng.integers(0, new, B, endpoint=True)
    add[0] = new
    W = -(-int((lens + add).max()) // 16) + 1
    need = int((-(-(lens + add) // 16) - -(-lens // 16)).sum())
    table, stack, N = make_tables(rng, lens, W, need + 3)
    want = check_extend(pq, lens, add, table, stack, len(stack), N, int(add.sum()) + pad, in_place)
    assert want[-1] == 0 and want[1] == 3


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("count", [0, 1, 40, 200])
def test_the_stack_runs_out(count, in_place):
    pq = require_gpu()
    rng = np.random.default_rng(count)
    lens = rng.integers(0, 60, 150)
    add = rng.integers(0, 50, 150)
    table, stack, N = make_tables(rng, lens, 9, 400)
    want = check_extend(pq, lens, add, table, stack, count, N, int(add.sum()) + 9, in_place)
    assert want[-1] == T.SLOT_RANGE and (want[3] >= 0).any()


def test_extend_with_nothing_to_do():
    pq = require_gpu()
    table, stack, N = make_tables(np.random.default_rng(0), [5, 0, 16], 2, 4)
    check_extend(pq, [5, 0, 16], [0, 0, 0], table, stack, 4, N, 6)       # only padding
    check_extend(pq, [5, 0, 16], [0, 0, 0], table, stack, 4, N, 0)       # no tokens at all
    check_extend(pq, [5, 0, 16], [1, 0, 1], table, stack, 4, N, 2)
    check_extend(pq, [], [], np.zeros((0, 2), np.int32), stack, 4, N, 3)  # no requests


@pytest.mark.parametrize("in_place", [False, True])
def test_bad_lengths_are_reported_and_left(in_place):
    pq = require_gpu()
    rng = np.random.default_rng(5)
    lens = np.array([10, 20, 30, 40, 31, 7])
    table, stack, N = make_tables(rng, lens, 4, 20)
    big = 2 ** 31 - 1
    for s, L, n in [(0, -1, 3), (1, 20, -1), (2, 60, 5), (3, 65, 0), (4, 31, big), (5, big, big),
                    (0, -big - 1, -big - 1)]:
        sl, add = lens.copy(), np.array([3, 3, 3, 3, 3, 3])
        sl[s], add[s] = L, n
        want = check_extend(pq, sl, add, table, stack, 20, N, 15, in_place)
        assert want[-1] == T.SEQ_RANGE
        assert want[0][s] == L
    # the step's batch is too small for the last requests
    want = check_extend(pq, lens, [3] * 6, table, stack, 20, N, 13, in_place)
    assert want[-1] == T.SEQ_RANGE and want[0].tolist() == [13, 23, 33, 43, 31, 7]
    # every length at its largest: the token sums pass 32 bits
    want = check_extend(pq, lens, [big] * 6, table, stack, 20, N, 13, in_place)
    assert want[-1] == T.SEQ_RANGE and (want[3] == -1).all()


def test_bad_counts_and_pages_are_reported():
    pq = require_gpu()
    lens = np.array([15, 30, 8])
    table, stack, N = make_tables(np.random.default_rng(6), lens, 4, 6)
    for count in (-3, 7, 2 ** 31 - 1):
        want = check_extend(pq, lens, [20, 1, 1], table, stack, count, N, 30)
        assert want[-1] == T.SLOT_RANGE
    for bad in (-1, N, 2 ** 31 - 1):
        st = stack.copy()
        st[5] = bad                                    # the top of the stack: taken by request 0
        want = check_extend(pq, lens, [20, 1, 1], table, st, 6, N, 30)
        assert want[-1] == T.PAGE_RANGE
        tb = table.copy()
        tb[2, 0] = bad                                 # a page begun earlier
        want = check_extend(pq, lens, [20, 1, 1], tb, stack, 6, N, 30)
        assert want[-1] == T.PAGE_RANGE


def check_truncate(pq, lens, keep, table, stack, count, owned=None, in_place=0):
    sl, kp, fc, fp = dev(lens), dev(keep), dev([count]), dev(stack)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slo = {0: torch.full_like(sl, -7), 1: sl, 2: kp}[in_place]     # 2: over keep_lens
    fco = fc if in_place else torch.full_like(fc, -7)
    bt = dev(table)
    pq.truncate_block_tables(sl, kp, bt, fp, fc, slo, fco,
                             owned_pages=None if owned is None else dev(owned), status=status)
    want = T.truncate(lens, keep, table, stack, count, owned)
    for name, g, w in zip(("seq_lens", "free_count", "free_pages", "status"),
                          (slo, fco, fp, status), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w), name
    assert np.array_equal(bt.cpu().numpy(), table)
    return want


@pytest.mark.parametrize("in_place", [0, 1, 2])
@pytest.mark.parametrize("B,cached,drop,owned", [
    (1, 16, 16, False), (1, 17, 1, False), (5, 100, 30, True), (300, 90, 5, False),
    (2048, 200, 200, True), (9, 30000, 30000, True)])
def test_truncate(B, cached, drop, owned, in_place):
    pq = require_gpu()
    rng = np.random.default_rng(B + drop)
    lens = rng.integers(0, cached, B, endpoint=True)
    keep = np.maximum(lens - rng.integers(0, drop, B, endpoint=True), 0)
    keep[0], lens[0] = 0, cached
    table, free, N = make_tables(rng, lens, -(-cached // 16), 5)
    stack = np.full(N, -1, np.int32)
    stack[:5] = free
    own = rng.integers(-1, 4, B) if owned else None
    want = check_truncate(pq, lens, keep, table, stack, 5, own, in_place)
    assert want[-1] == 0


def test_truncate_reports_bad_arguments():
    pq = require_gpu()
    lens = np.array([40, 64, 20])
    table, free, N = make_tables(np.random.default_rng(8), lens, 4, 2)
    stack = np.full(N, -1, np.int32)
    for L, keep in [([40, 64, 20], [-1, 1, 1]), ([40, 64, 20], [10, 65, 1]), ([65, 64, 20], [1, 1, 1]),
                    ([-5, 64, 20], [-5, 0, 0]), ([2 ** 31 - 1, 64, 20], [0, 0, 0])]:
        assert check_truncate(pq, L, keep, table, stack, 2)[-1] == T.SEQ_RANGE
    # no room for every page, and counts outside the stack
    want = check_truncate(pq, lens, [0, 0, 0], table, np.full(5, -1, np.int32), 2)
    assert want[-1] == T.SLOT_RANGE and want[1] == 5
    for count in (-1, N + 1):
        assert check_truncate(pq, lens, [0, 0, 0], table, stack, count)[-1] & T.SLOT_RANGE


def test_steps_of_extend_and_truncate_keep_every_page_once():
    """Verify steps in place on one stream: 5 tokens in, some of them taken
    back, requests ending and others starting in their row."""
    pq = require_gpu()
    rng = np.random.default_rng(11)
    B, W, N, T_cap = 37, 6, 160, 256
    sl, fc = dev(np.zeros(B)), dev([N])
    bt, fp = dev(np.full((B, W), -1)), dev(rng.permutation(N))
    slots = torch.empty(T_cap, dtype=torch.int64, device="cuda")
    lens, count, stack, table = np.zeros(B, np.int32), N, fp.cpu().numpy(), bt.cpu().numpy()
    for step in range(25):
        new = np.where(lens == 0, rng.integers(1, 30, B), 5) if step % 3 else np.full(B, 5)
        new = np.minimum(new, 16 * W - lens)
        new = new * (np.cumsum(new) <= T_cap)
        pq.extend_block_tables(sl, dev(new), bt, fp, fc, N, sl, fc, slots)
        lens, count, table, want, *_ = T.extend(lens, new, table, stack, count, N, T_cap)
        assert np.array_equal(slots.cpu().numpy(), want)
        keep = np.maximum(lens - rng.integers(0, 5, B), 0)
        keep[rng.random(B) < 0.1] = 0
        pq.truncate_block_tables(sl, dev(keep), bt, fp, fc, sl, fc)
        lens, count, stack, _ = T.truncate(lens, keep, table, stack, count)
        assert np.array_equal(sl.cpu().numpy(), lens) and int(fc.item()) == count
        held = [int(table[s, j]) for s in range(B) for j in range(-(-int(lens[s]) // 16))]
        assert sorted(held + fp.cpu().numpy()[:count].tolist()) == list(range(N))


def test_captured_steps_and_another_stream():
    """A captured extend/truncate pair replayed in place, and the same calls on
    a side stream, go on from the state they find."""
    pq = require_gpu()
    B, W, N, T_cap = 70, 300, 9000, 1024
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 100, B).astype(np.int32)
    table, free, _ = make_tables(rng, lens, W, N - int((-(-lens // 16)).sum()))
    stack = np.full(N, -1, np.int32)
    stack[:len(free)] = free
    count = len(free)
    sl, bt, fp, fc = dev(lens), dev(table), dev(stack), dev([count])
    new, keep = dev(np.full(B, 9)), torch.empty(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(T_cap, dtype=torch.int64, device="cuda")

    def step():
        pq.extend_block_tables(sl, new, bt, fp, fc, N, sl, fc, slots)
        torch.sub(sl, 2, out=keep)
        pq.truncate_block_tables(sl, keep, bt, fp, fc, sl, fc)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for k in range(6):
        if k % 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        lens, count, table, want, *_ = T.extend(lens, np.full(B, 9), table, stack, count, N, T_cap)
        lens, count, stack, _ = T.truncate(lens, lens - 2, table, stack, count)
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want)
        assert np.array_equal(sl.cpu().numpy(), lens) and int(fc.item()) == count
        assert np.array_equal(fp.cpu().numpy()[:count], stack[:count])
        assert np.array_equal(bt.cpu().numpy(), table)


def test_the_slots_feed_the_append():
    """extend -> kv_append_quant: every token lands in its request's page, and a
    refused request's tokens are skipped."""
    pq = require_gpu()
    lens, add = np.array([3, 30, 0, 16]), np.array([20, 5, 40, 2])
    table, stack, N = make_tables(np.random.default_rng(1), lens, 4, 5)
    slo, fco, bt, slots, pos, off, status = run_extend(pq, lens, add, table, stack, 3, N, 70)
    assert int(status.item()) == T.SLOT_RANGE            # request 2 needs three pages of one
    pages = pq.new_pages(N, 2, pq.FP16, "cuda", fill=0.0)
    k = torch.arange(1, 71, device="cuda", dtype=torch.float16)[:, None, None].expand(70, 2, 128)
    pq.kv_append_quant(k.contiguous(), k.contiguous(), slots, pq.FP16, None, None, pages)
    want = np.zeros((N, 16))
    for t, (s, q) in enumerate([(0, 3 + i) for i in range(20)] + [(1, 30 + i) for i in range(5)]):
        want[int(bt[s, q // 16]), q % 16] = t + 1
    assert np.array_equal(pages[:, 0, 0, :, 0].float().cpu().numpy(), want)


def test_the_binding_refuses_mismatches():
    pq = require_gpu()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    ok = dict(seq_lens=z(2), new_tokens=z(2), block_table=z(2, 4), free_pages=z(9), free_count=z(1),
              num_pages=9, seq_lens_out=z(2), free_count_out=z(1), slot_mapping=slots)
    pq.extend_block_tables(**ok)
    for name, bad in [("seq_lens", z(3)), ("new_tokens", z(2).long()), ("block_table", z(2, 8)[:, ::2]),
                      ("free_pages", z(9).cpu()), ("free_count", z(2)), ("seq_lens_out", z(1)),
                      ("free_count_out", z(1).float()), ("slot_mapping", slots.int()),
                      ("positions", z(5)), ("token_offsets", z(2)), ("status", slots)]:
        with pytest.raises(ValueError):
            pq.extend_block_tables(**{**ok, name: bad})
    with pytest.raises(ValueError):
        pq.truncate_block_tables(z(2), z(2), z(2, 4), z(9), z(1), z(2), z(1), owned_pages=z(3))

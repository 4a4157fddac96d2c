"""Attention over shared prefixes against the float64 definition of each
sequence's own attention, at the sizes where the split can go wrong."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.helpers import require_gpu
from tests.shared_case import NAN_FILL, SharedCase

pytestmark = pytest.mark.gpu

FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW]
HEADS = [(8, 1, 1), (32, 8, 1), (16, 4, 5), (8, 2, 8), (6, 2, 3), (4, 4, 2), (32, 2, 1), (10, 2, 6)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,q_len", HEADS)
def test_one_group(fmt, hq, hkv, q_len):
    rng = np.random.default_rng(hq * 100 + q_len)
    c = SharedCase([(177, (q_len + rng.integers(0, 60, 5)).tolist())], hq, hkv, q_len, fmt, seed=hq,
                   per_head=True)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 3, 7, 13, 33, 70])
def test_batch_sizes(fmt, n):
    """From one sequence to rows that pass several row tiles."""
    rng = np.random.default_rng(n)
    c = SharedCase([(130, (5 + rng.integers(0, 40, n)).tolist())], 8, 2, 5, fmt, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 32, 127, 128, 129, 143, 144, 255, 256, 272,
                                    1025, 4096, 5003])
def test_prefix_lengths(fmt, prefix):
    c = SharedCase([(prefix, [1, 16, 17, 40])], 8, 2, 1, fmt, seed=prefix)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_groups_of_all_kinds(fmt):
    """Several groups: one without a prefix, one of a single sequence, empty
    ones in front, between and behind, prefixes that end inside a page."""
    groups = [(50, []), (333, [5, 6, 90]), (0, [5, 33]), (64, []), (64, [7]), (15, [8, 8]),
              (200, [20] * 19), (48, [])]
    c = SharedCase(groups, 16, 4, 5, fmt, seed=3)
    c.check(c.run())
    c.check(c.run(max_seq_len=int(c.lens.max()), max_prefix_len=333), "with bounds")


@pytest.mark.parametrize("bounds", [dict(max_prefix_len=15), dict(max_prefix_len=160),
                                    dict(max_prefix_len=16, max_seq_len=1),
                                    dict(max_seq_len=100), dict(max_seq_len=1 << 30)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_bounds_that_do_not_hold_change_no_result(fmt, bounds):
    c = SharedCase([(333, [5, 6, 90]), (0, [33]), (700, [20] * 9)], 16, 4, 5, fmt, seed=30)
    c.check(c.run(**bounds))


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_groups_of_every_size(fmt):
    """More groups than CTAs: a CTA's share spans several of them."""
    rng = np.random.default_rng(31)
    groups = [(int(rng.integers(0, 200)), (2 + rng.integers(0, 30, rng.integers(0, 4))).tolist())
              for _ in range(400)]
    c = SharedCase(groups, 4, 2, 2, fmt, seed=31)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_sequences_of_one_page_beside_a_long_one(fmt):
    """Shares of the private keys that hold many segments, one segment, and none."""
    c = SharedCase([(64, [1] * 150 + [3000] + [1] * 49)], 8, 8, 1, fmt, seed=32)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_private_parts(fmt):
    c = SharedCase([(96, [2000, 1, 700]), (640, [3, 1500])], 8, 2, 1, fmt, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_prefix_given_up_to_the_end(fmt):
    """prefix_lens may reach the sequences' ends: the new tokens stay private."""
    pq = require_gpu()
    for q_len, prefix, priv in [(1, 64, [1, 5]), (5, 64, [5, 9]), (8, 47, [8, 20])]:
        c = SharedCase([(prefix, priv)], 8, 2, q_len, fmt, seed=q_len)
        c.upload()
        full = int(c.lens.min())
        n = full // 16
        c.bt[1:, :n] = c.bt[0, :n]                  # the rows agree over the whole given prefix
        c.g["block_table"].copy_(torch.from_numpy(c.bt))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        given = torch.full((1,), full, dtype=torch.int32, device="cuda")
        c.check(c.run(prefix_lens=given, status=status), "q_len %d" % q_len)
        assert int(status.item()) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_lengths_and_groups_are_reported_and_harmless(fmt):
    pq = require_gpu()
    c = SharedCase([(100, [5, 6, 40]), (64, [7, 8])], 8, 2, 5, fmt, seed=6)
    c.upload()
    for name, bad in [("prefix_lens", [-1, 64]), ("prefix_lens", [2 ** 31 - 1, 64]),
                      ("prefix_lens", [100, -2 ** 31]), ("group_offsets", [1, 3, 5]),
                      ("group_offsets", [0, 4, 3]), ("group_offsets", [0, 3, 6]),
                      ("group_offsets", [0, 2 ** 31 - 1, 5]), ("group_offsets", [-5, 3, 5]),
                      ("group_offsets", [0, 3, 4])]:
        if bad[0] == 2 ** 31 - 1:
            c2 = SharedCase([(100, [5])], 8, 2, 5, fmt, seed=6)   # alone: any prefix is its own
            c2.upload()
            use, bad = c2, bad[:1]
        else:
            use = c
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        arg = torch.tensor(bad, dtype=torch.int32, device="cuda")
        use.check(use.run(**{name: arg, "status": status}), "%s %s" % (name, bad))
        assert pq.status_bits(status) == ["seq_len out of range"], (name, bad)
    # lengths beyond the row or below q_len are clamped, as in paged_attention
    for L in (2, -7, 2 ** 31 - 1):
        lens = c.g["seq_lens"].clone()
        lens[1] = L
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(seq_lens=lens, status=status)
        assert pq.status_bits(status)[0] == "seq_len out of range"
        c.check(got, "L %d" % L, seqs=[0, 2, 3, 4])


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_outside_the_pool_read_as_zeros(fmt):
    pq = require_gpu()
    for where in (2, 9):                            # a shared page, a private one
        for bad in (-1, None, 2 ** 31 - 1):
            c = SharedCase([(100, [60, 70])], 8, 2, 1, fmt, seed=8)
            c.upload()
            bt = c.bt.copy()
            bt[:, where] = c.pool.shape[0] if bad is None else bad
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = c.run(block_table=torch.from_numpy(bt).cuda(), status=status)
            assert pq.status_bits(status) == ["block-table page id out of range"]
            # the oracle reads a page of zeros there, one that no row names
            spare = (set(range(c.pool.shape[0])) - set(c.bt.ravel().tolist())).pop()
            c.pool[spare] = 0
            if fmt == W.INT8_ROW:
                c.pool_ks[spare] = c.pool_vs[spare] = 0
            c.bt[:, where] = spare
            c.check(got, "page %d = %s" % (where, bad))


def test_bad_scales_are_reported():
    pq = require_gpu()
    c = SharedCase([(100, [6, 7])], 8, 2, 1, W.FP8_E4M3)
    c.upload()
    for v in (0.0, -1.0, float("inf"), float("nan")):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.run(k_scale=torch.full((1,), v, device="cuda"), status=status)
        assert pq.status_bits(status) == ["bad scale"]


def test_the_result_is_paged_attentions_and_reproducible():
    pq = require_gpu()
    for fmt in FORMATS:
        c = SharedCase([(1000, [5, 6, 200, 31] * 4), (500, [9, 10])], 32, 8, 5, fmt, seed=9)
        a = c.run()
        b = torch.empty_like(a)
        pq.paged_attention(c.g["q"], c.g["pages"], c.g["block_table"], c.g["seq_lens"], 5, fmt,
                           c.g["k_scale"], c.g["v_scale"], b)
        want, tol = c.expected(seqs=[0, 2, 17], heads=[0, 7])
        sel = ~np.isnan(want)
        for x in (a, b):                          # both round where the bound says
            assert (np.abs(x.double().cpu().numpy()[sel] - want[sel]) <= tol[sel]).all()
        for _ in range(3):
            assert torch.equal(c.run(), a)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,q_len,prefix", [(64, 5, 20000), (250, 1, 12000), (24, 8, 40000)])
def test_long_prefixes_of_many_rows_repeat_and_match(fmt, B, q_len, prefix):
    """Several row tiles read the same keys out of L2, so that copies are fast and every
    wait of the pipeline is met; every run gives the same bits, and paged_attention's
    result.  Both round the probabilities and the output to fp16: at most 4 halves of
    a step of the largest |V|."""
    pq = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(B)
    hq, hkv, own = 32, 8, 40
    shared, width = prefix // 16, -(-(prefix + own) // 16)
    N = shared + B * (width - shared)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    pages = pq.new_pages(N, hkv, fmt, "cuda")
    x = torch.randn(pages.shape, generator=gen, device="cuda")
    x *= 1 + 4 * (torch.rand(pages.shape, generator=gen, device="cuda") < 0.01)
    ks = vs = None
    if fmt == W.FP16:
        pages.copy_(x)
    elif fmt == W.FP8_E4M3:
        ks = vs = torch.full((1,), 1 / 16, device="cuda")
        pages.copy_((x * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        pages.copy_((x * 5).round().clamp(-127, 127).to(torch.int8).view(torch.uint8))
        ks = vs = torch.full((1,), 1 / 5, device="cuda")
        if fmt == W.INT8_ROW:
            pq.row_scales(pages).copy_(0.2 * (1 + torch.rand(pq.row_scales(pages).shape,
                                                             generator=gen, device="cuda")))
    bt = torch.empty((B, width), dtype=torch.int32, device="cuda")
    perm = torch.randperm(N, generator=gen, device="cuda").int()
    bt[:, :shared] = perm[:shared]
    bt[:, shared:] = perm[shared:].view(B, -1)
    q = torch.randn((B * q_len, hq, 128), generator=gen, device="cuda").half()
    sl = prefix + q_len + torch.randint(0, own - q_len, (B,), generator=gen, device="cuda").int()
    want = pq.paged_attention(q, pages, bt, sl, q_len, fmt, ks, vs, torch.empty_like(q))
    first = None
    for k in range(6):
        out = torch.full_like(q, float("nan"))
        pq.paged_attention_shared_prefix(q, pages, bt, sl, i32([0, B]), i32([prefix]), q_len, fmt,
                                         ks, vs, out)
        first = out if first is None else first
        assert torch.equal(out, first), "run %d differs" % k
    top = float(x[:, :, 1].abs().max()) * (2 if fmt == W.INT8_ROW else 1) + 1
    assert float((first.float() - want.float()).abs().max()) <= 4 * 2.0 ** -11 * top


def test_large_scores_and_values():
    """Scores far apart (a running maximum that keeps moving, probabilities
    that vanish) and values near the format's end."""
    for fmt in FORMATS:
        c = SharedCase([(700, [40, 80, 16])], 8, 2, 1, fmt, seed=12, outliers=True, v_amp=20.0)
        c.q = (c.q.astype(np.float32) * 30).astype(np.float16)
        c.check(c.run(), "format %d" % fmt)


def test_many_sequences():
    c = SharedCase([(48, (1 + np.arange(1500) % 20).tolist()), (16, [3] * 548)], 4, 1, 1, W.FP8_E4M3,
                   seed=13)
    c.check(c.run())


def test_wide_heads():
    c = SharedCase([(300, [9, 20, 33])], 64, 64, 2, W.INT8, seed=14, per_head=True)
    c.check(c.run())


def test_a_captured_call_follows_its_inputs():
    """Replays after the lengths, the prefix and the groups change, beside eager
    calls with other workspaces."""
    pq = require_gpu()
    c = SharedCase([(320, [40, 50, 60]), (320, [41, 9])], 8, 2, 5, W.FP8_E4M3, seed=15)
    c.upload()
    out = torch.empty_like(c.g["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(out=out)
    for prefix, offsets, cut in [([320, 320], [0, 3, 5], 0), ([100, 0], [0, 3, 5], 3),
                                 ([320, 16], [0, 1, 5], 2), ([0, 0], [0, 5, 5], 0)]:
        lens = np.maximum(c.lens - cut, 5)
        if offsets[1] == 1:                       # the second group mixes two prefixes: share none
            prefix = [320, 0]
        c.g["seq_lens"].copy_(torch.from_numpy(lens))
        c.g["prefix_lens"].copy_(torch.tensor(prefix, dtype=torch.int32))
        c.g["group_offsets"].copy_(torch.tensor(offsets, dtype=torch.int32))
        out.fill_(float("nan"))
        if offsets[1] == 5:
            c.g["prefix_lens"].zero_()
        graph.replay()
        eager = c.run()
        torch.cuda.synchronize()
        c.check(out, "replay %s" % prefix, lens=lens)
        assert torch.equal(out, eager)


def test_two_streams_at_once():
    """Calls on two streams, without a workspace of their own, do not meet."""
    pq = require_gpu()
    cases = [SharedCase([(600, [30] * 9)], 8, 2, 5, f, seed=20 + f) for f in (W.FP8_E4M3, W.FP16)]
    want = [c.run().clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(w, float("nan")) for _ in range(20)] for w in want]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for k in range(20):
        for c, s, o in zip(cases, streams, outs):
            c.run(out=o[k], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for x in o:
            assert torch.equal(x, w)


def test_a_given_workspace_may_hold_anything():
    pq = require_gpu()
    c = SharedCase([(500, [30, 5, 77])], 16, 4, 5, W.INT8, seed=30)
    c.upload()
    need = pq.shared_prefix_workspace_size(3, 1, 5, 16, 4)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    a = c.run(workspace=ws)
    c.check(a)
    assert torch.equal(c.run(workspace=ws), a)
    with pytest.raises(pq.PqkvError, match="workspace"):
        c.run(workspace=ws[:need - 256])
    with pytest.raises(ValueError):
        c.run(workspace=ws.cpu())


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn on one stream, neither finds what the other left."""
    pq = require_gpu()
    cases = [SharedCase([(400, [30, 50]), (0, [9])], 8, 2, 5, W.INT8, seed=33),
             SharedCase([(96, [3] * 40)], 16, 2, 1, W.INT8_ROW, seed=34)]
    need = max(pq.shared_prefix_workspace_size(len(c.lens), len(c.prefix), c.q_len, c.hq, c.hkv)
               for c in cases)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for c in cases:
        out = torch.empty_like(c.upload()["q"])
        c.run(out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(out=out, workspace=ws)
        outs.append(out)
        graphs.append(graph)
    for _ in range(3):
        for out, graph in zip(outs, graphs):
            out.fill_(float("nan"))
            graph.replay()
    for c, out in zip(cases, outs):
        c.check(out)


@pytest.mark.parametrize("fmt", [W.FP16, W.INT8_ROW])
def test_pages_past_four_gigabytes(fmt):
    pq = require_gpu()
    c = SharedCase([(150, [20, 33, 5]), (40, [7])], 16, 8, 2, fmt, seed=35)
    g = c.upload()
    n, page = g["pages"].shape[0], g["pages"][0].numel() * g["pages"].element_size()
    top = (1 << 32) // page + 5                       # pages in front of the case's own
    big = pq.new_pages(top + n, 8, fmt, "cuda")
    big[top:].copy_(g["pages"])
    if fmt == W.INT8_ROW:
        pq.row_scales(big)[top:].copy_(pq.row_scales(g["pages"]))
    c.check(c.run(pages=big, block_table=torch.where(g["block_table"] >= 0, g["block_table"] + top,
                                                     g["block_table"])))


def test_an_empty_batch_and_the_longest_row():
    pq = require_gpu()
    c = SharedCase([(100, [6, 7])], 8, 2, 1, W.FP8_E4M3, seed=36)
    g = c.upload()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = c.run(q=g["q"][:0], out=g["q"][:0].clone(), seq_lens=none, prefix_lens=none,
                block_table=g["block_table"][:0], group_offsets=torch.zeros_like(g["seq_lens"][:1]))
    assert out.shape[0] == 0
    wide = torch.full((2, 524288 // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :g["block_table"].shape[1]] = g["block_table"]
    c.check(c.run(block_table=wide))


def test_rows_behind_the_batch_are_left():
    """q and out may be the leading rows of larger buffers."""
    c = SharedCase([(200, [9, 8, 30])], 8, 2, 5, W.FP8_E4M3, seed=31)
    c.upload()
    big = torch.full((40, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    c.check(c.run(out=big[:15]))
    assert (big[15:] == 7.0).all()


def test_a_step_from_lengths_to_attention():
    """The operators together: prompts on a shared prefix, then verify steps --
    pages taken, tokens appended, attention over the shared prefix, rejected
    drafts given back -- all state on the device."""
    pq = require_gpu()
    fmt, hq, hkv, q_len = W.FP8_E4M3, 8, 2, 5
    rng = np.random.default_rng(40)
    B, W_, N, P = 6, 24, 120, 70                       # a 70-token prefix: 4 whole pages shared
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    ks = vs = torch.full((1,), 6.0 / 448, device="cuda")
    pages = pq.new_pages(N, hkv, fmt, "cuda", fill=NAN_FILL[fmt])
    bt = torch.full((B, W_), -1, dtype=torch.int32, device="cuda")
    fp, fc = i32(rng.permutation(N).tolist()), i32([N])
    sl = i32([0] * B)
    dense = [None] * B                                  # each sequence's fp16 K and V
    tokens = lambda n: torch.randn((2, n, hkv, 128), device="cuda").half()   # noqa: E731

    def append(new, kv):
        slots = torch.empty(sum(new) + 3, dtype=torch.int64, device="cuda")
        status = i32([0])
        pq.extend_block_tables(sl, i32(new), bt, fp, fc, N, sl, fc, slots, status=status)
        pad = torch.cat([kv, tokens(3)], 1)
        pq.kv_append_quant(pad[0], pad[1], slots, fmt, ks, vs, pages, status=status)
        assert int(status.item()) == 0

    # the first request brings the prefix; the others start behind its whole pages
    prefix = tokens(P)
    append([P] + [0] * (B - 1), prefix)
    bt[1:, :P // 16] = bt[0, :P // 16]
    sl[1:] = P // 16 * 16
    owned = i32([0] + [P // 16] * (B - 1))
    rest = [0] + [P % 16 + int(x) for x in rng.integers(1, 60, B - 1)]
    kv = tokens(sum(rest))
    append(rest, kv)
    at = 0
    for s in range(B):
        tail = kv[:, at:at + rest[s]]
        at += rest[s]
        dense[s] = prefix if s == 0 else torch.cat([prefix[:, :P // 16 * 16], tail], 1)
    for step in range(4):
        q = torch.randn((B * q_len, hq, 128), device="cuda").half()
        kv = tokens(B * q_len)
        append([q_len] * B, kv)
        dense = [torch.cat([d, kv[:, s * q_len:(s + 1) * q_len]], 1) for s, d in enumerate(dense)]
        out = torch.empty_like(q)
        pq.paged_attention_shared_prefix(q, pages, bt, sl, i32([0, B]), i32([P]), q_len, fmt, ks,
                                         vs, out)
        for s in range(B):
            n = dense[s].shape[1]
            assert n == int(sl[s].item())
            x = dense[s].float() / (6.0 / 448)
            x = x.clamp(-448, 448).to(torch.float8_e4m3fn).double() * float(ks.item())
            K, V = (y.repeat_interleave(hq // hkv, 1) for y in x)
            z = torch.einsum("ihd,nhd->hin", q[s * q_len:(s + 1) * q_len].double(), K) / 128 ** 0.5
            see = torch.arange(n, device="cuda")[None] <= n - q_len + torch.arange(
                q_len, device="cuda")[:, None]
            want = torch.einsum("hin,nhd->ihd", torch.softmax(z.masked_fill(~see, -np.inf), -1), V)
            err = (out[s * q_len:(s + 1) * q_len].double() - want).abs().max().item()
            # |V| <= 6: roundings of p and out, 2^-11 each of at most 6
            assert err <= 6 * (2.0 ** -10 + 2.0 ** -12)
        keep = sl - i32(rng.integers(0, q_len, B).tolist())
        pq.truncate_block_tables(sl, keep, bt, fp, fc, sl, fc, owned_pages=owned)
        dense = [d[:, :int(k)] for d, k in zip(dense, keep.tolist())]
    pq.truncate_block_tables(sl, torch.zeros_like(sl), bt, fp, fc, sl, fc, owned_pages=owned)
    assert sorted(fp.tolist()) == list(range(N)) and int(fc.item()) == N


def test_the_binding_refuses_mismatches():
    pq = require_gpu()
    c = SharedCase([(100, [6, 7])], 8, 2, 1, W.FP8_E4M3)
    g = c.upload()
    for name, bad in [("seq_lens", g["seq_lens"].long()), ("seq_lens", g["seq_lens"].cpu()),
                      ("block_table", g["block_table"][:1]), ("block_table", g["block_table"].t()),
                      ("group_offsets", g["seq_lens"][:1]), ("prefix_lens", g["seq_lens"]),
                      ("q", g["q"].float()), ("q", g["q"][:1]), ("out", g["q"][:1]),
                      ("q_len", 2), ("k_scale", g["k_scale"].double()), ("max_seq_len", -1),
                      ("max_prefix_len", -1), ("kv_dtype", W.FP16)]:
        with pytest.raises(ValueError):
            c.run(**{name: bad})

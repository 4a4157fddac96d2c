"""Shared-prefix attention over a 4-bit pool against each sequence's own attention in 64 bits.

The bounds are those of paged_attention (int4_case.allowance): the two key sets' parts
round their probabilities by the same steps, the products of codes and scales are exact,
and the merge of the parts is fp32."""
import numpy as np
import pytest
import torch

import oracle
from tests.helpers import require_gpu
from tests.int4_case import F, allowance, assert_within, rows

pytestmark = pytest.mark.gpu


class Shared:
    """Groups [(prefix, [private lengths])] in a 4-bit pool whose unwritten bytes are NaN scales."""

    def __init__(self, groups, hq, hkv, q_len, seed):
        rng = np.random.default_rng(seed)
        self.q_len, self.hkv = q_len, hkv
        self.lens = [pre // 16 * 16 + max(n, q_len) for pre, priv in groups for n in priv]
        self.offsets = np.cumsum([0] + [len(priv) for _, priv in groups]).astype(np.int32)
        self.prefix = np.array([pre for pre, _ in groups], np.int32)
        shared = [pre // 16 if priv else 0 for pre, priv in groups]
        need = [-(-L // 16) for L in self.lens]
        n_pages = sum(shared) + sum(n - shared[g] for g, (a, b) in enumerate(
            zip(self.offsets, self.offsets[1:])) for n in need[a:b]) + 3
        perm, at = rng.permutation(n_pages).astype(np.int32), 0
        self.bt = np.full((len(self.lens), max(need + [1])), -1, np.int32)
        own = []                                    # slots of all tokens, once each
        for g, (a, b) in enumerate(zip(self.offsets, self.offsets[1:])):
            pages = perm[at:at + shared[g]]
            at += shared[g]
            if a < b:
                own.append((pages[:, None].astype(np.int64) * 16 + np.arange(16)).ravel())
            for s in range(a, b):
                n = need[s] - shared[g]
                self.bt[s, :need[s]] = np.concatenate([pages, perm[at:at + n]])
                at += n
                t = np.arange(16 * shared[g], self.lens[s])
                own.append(self.bt[s, t // 16].astype(np.int64) * 16 + t % 16)
        self.spare = int(perm[-1])
        own = np.concatenate(own)
        self.pages = oracle.kv_append_quant(
            rows(rng, len(own), hkv), rows(rng, len(own), hkv), own, F, None, None,
            oracle.new_pool(n_pages, hkv, 128, F, fill=0xFF))
        self.q = rng.normal(size=(len(self.lens) * q_len, hq, 128)).astype(np.float16)

    def args(self):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return [d(self.q), d(self.pages), d(self.bt), d(np.array(self.lens, np.int32)),
                d(self.offsets), d(self.prefix)]

    def run(self, args=None, status_bits=0, **kw):
        pq = require_gpu()
        # (a prefix that is longer than a sequence of its group is reported, and clamped)
        for pre, a, b in zip(self.prefix, self.offsets, self.offsets[1:]):
            if min(self.lens[a:b], default=pre) < pre:
                status_bits |= 2
        args = args or self.args()
        out = torch.full(self.q.shape, float("nan"), dtype=torch.float16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        pq.paged_attention_shared_prefix(*args, self.q_len, "int4_group", None, None, out,
                                         status=st, **kw)
        assert int(st.item()) == status_bits, pq.status_bits(st)
        return out

    def check(self, out, seqs=None, bt=None, pages=None, what=""):
        seqs = list(range(len(self.lens)) if seqs is None else seqs)
        at = np.concatenate([np.arange(s * self.q_len, (s + 1) * self.q_len) for s in seqs])
        ref, bound = allowance(self.q[at], self.pages if pages is None else pages,
                               (self.bt if bt is None else bt)[seqs],
                               [self.lens[s] for s in seqs], self.q_len)
        assert_within(out.cpu().numpy()[at].astype(np.float64), ref, bound, what)


@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (32, 8, 1), (16, 4, 5), (8, 2, 8), (6, 2, 3),
                                          (4, 4, 2), (32, 2, 1), (10, 2, 6)])
def test_heads_of_one_group(hq, hkv, q_len):
    rng = np.random.default_rng(hq)
    c = Shared([(177, rng.integers(1, 60, 5).tolist())], hq, hkv, q_len, seed=hq + q_len)
    c.check(c.run())


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 32, 127, 128, 129, 144, 255, 272, 1025, 5003])
def test_prefix_lengths(prefix):
    c = Shared([(prefix, [1, 16, 17, 40])], 8, 2, 1, seed=prefix)
    c.check(c.run())


@pytest.mark.parametrize("n", [1, 2, 7, 13, 33, 70])
def test_batch_sizes(n):
    """From one sequence to rows that pass several row tiles."""
    rng = np.random.default_rng(n)
    c = Shared([(400, rng.integers(1, 40, n).tolist())], 8, 2, 5, seed=n)
    c.check(c.run())


def test_groups_of_all_kinds():
    c = Shared([(50, []), (333, [5, 6, 90]), (0, [5, 33]), (64, []), (64, [7]), (15, [8, 8]),
                (200, [20] * 19), (48, [])], 16, 4, 5, seed=3)
    c.check(c.run())
    c.check(c.run(max_seq_len=max(c.lens), max_prefix_len=333), what="with bounds")
    c.check(c.run(max_prefix_len=160), what="a bound that does not hold")


def test_long_private_parts():
    c = Shared([(96, [2000, 1, 700]), (640, [3, 1500])], 8, 2, 1, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("where", [2, 9])                   # a shared page, a private one
@pytest.mark.parametrize("bad", [-1, "n", 2 ** 31 - 1])
def test_a_page_outside_the_pool_reads_zeros(where, bad):
    c = Shared([(100, [60, 70])], 8, 2, 1, seed=8)
    zeros = c.pages.copy()
    zeros[c.spare] = 0
    ref = c.bt.copy()
    seqs = slice(None) if where == 2 else slice(0, 1)
    ref[seqs, where] = c.spare
    c.bt[seqs, where] = c.pages.shape[0] if bad == "n" else bad
    c.check(c.run(status_bits=16), bt=ref, pages=zeros)


@pytest.mark.parametrize("B,q_len,prefix", [(64, 5, 20000), (250, 1, 12000), (24, 8, 40000)])
def test_long_prefixes_of_many_rows(B, q_len, prefix):
    """Many key tiles a block; the same bits every time; and paged_attention's result."""
    pq = require_gpu()
    c = Shared([(prefix, [q_len + s % 50 for s in range(B)])], 16, 4, q_len, seed=B)
    args = c.args()
    out = c.run(args)
    for _ in range(5):
        assert torch.equal(c.run(args), out)
    c.check(out, seqs=[0, B // 2, B - 1])
    whole = torch.empty_like(out)
    pq.paged_attention(args[0], args[1], args[2], args[3], q_len, "int4_group", None, None, whole)
    # each is within 1.5 * 2^-11 A and its own half step of the same rows: A <= max |V|,
    # and a value is 20 * 5 sigmas at most here
    assert (out.float() - whole.float()).abs().max().item() < 2 * 1.75 * 2.0 ** -11 * 100


def test_scores_that_rise_far():
    """Queries along keys: references are raised on the way, probabilities pass 2^15."""
    c = Shared([(1500, [30, 40, 50])], 8, 2, 5, seed=11)
    # N(0, 4): scores have a deviation of about 4.5 (allowance counts |q| |K| for 1), so the
    # bound's share of the scores' rounding is taken four times
    c.q = (4 * c.q.astype(np.float32)).astype(np.float16)
    out = c.run().cpu().numpy().astype(np.float64)
    ref, bound = allowance(c.q, c.pages, c.bt, c.lens, c.q_len)
    A = 0
    for h in range(2):
        for s, L in enumerate(c.lens):
            A = max(A, np.abs(oracle.gather_kv(c.pages, c.bt[s], L, h, F, None, None)[1]).max())
    assert_within(out, ref, bound + 3 * 2.0 ** -13 * A)


def test_a_captured_call_follows_its_inputs():
    pq = require_gpu()
    c = Shared([(300, [20, 35, 17]), (64, [9, 40])], 8, 2, 5, seed=12)
    d = Shared([(300, [20, 35, 17]), (64, [9, 40])], 8, 2, 5, seed=13)
    args, other = c.args(), d.args()
    out = torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    ws = torch.empty(pq.shared_prefix_workspace_size(len(c.lens), 2, 5, 8, 2), dtype=torch.uint8,
                     device="cuda")
    call = lambda: pq.paged_attention_shared_prefix(*args, 5, "int4_group", None, None, out,
                                                    workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    c.check(out)
    for a, b in zip(args, other):
        a.copy_(b)
    graph.replay()
    d.check(out)

"""Measured cases of the serving-step operators around the paged KV pool.

Three operators, each in its plain form (elementary torch operations in 32 or
64 bits) and as the library's own call:

  extend_block_tables    admit each request's new tokens: take pages from the
                         free stack, write them into the block tables, and
                         give every token its pool slot and position
  truncate_block_tables  shorten requests (rejected draft tokens, finished
                         requests) and push their pages back on the stack
  paged_attention_shared_prefix
                         decode / verify attention of a batch whose sequences
                         share a long prefix, the prefix's keys read once

Lengths are a function of the case alone, so that work() is exact; values,
page numbers and the order of the free stack come from the seed.
"""
import json
import math
import zlib

import numpy as np
import torch

own = False

PAGE = 16
DIM = 128
FORMATS = {"fp16": 0, "fp8_e4m3": 1, "int8": 2, "int8_row": 3}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _extend(batch, cached, new, fixed):
    return {"op": "extend", "batch": batch, "cached": cached, "new": new, "fixed": fixed}


def _truncate(batch, cached, drop, release):
    return {"op": "truncate", "batch": batch, "cached": cached, "drop": drop, "release": release}


def _shared(fmt, batch, groups, hq, hkv, q_len, prefix, suffix):
    return {"op": "shared", "format": fmt, "batch": batch, "groups": groups, "hq": hq, "hkv": hkv,
            "q_len": q_len, "prefix": prefix, "suffix": suffix}


def listed():
    return [
        # one decode step of 8 requests: nothing but latency
        dict(_extend(8, 32768, 1, True), name="extend_decode_b8"),
        # one verify step (1 committed + 4 draft tokens) of the largest batch
        dict(_extend(2048, 4096, 5, True), name="extend_verify_b2048"),
        # many ragged prompts admitted at once onto partly filled tables
        dict(_extend(777, 2000, 2600, False), name="extend_prompts_b777"),
        # rejected drafts of a verify step given back
        dict(_truncate(2048, 4096, 5, False), name="truncate_drafts_b2048"),
        # a third of the long requests of a batch end and release their pages
        dict(_truncate(96, 131072, 5, True), name="truncate_release_b96"),
        # the smallest attention: short contexts, one kv-head, fp16 pool
        dict(_shared("fp16", 4, 1, 8, 1, 1, 1024, 64), name="shared_fp16_tiny"),
        # 8 concurrent requests behind one system prompt, plain decode
        dict(_shared("fp8_e4m3", 8, 1, 32, 8, 1, 32768, 2048), name="shared_e4m3_decode_b8"),
        # 64 requests behind one long document, verify with 4 draft tokens
        dict(_shared("fp8_e4m3", 64, 1, 32, 8, 5, 32768, 1024), name="shared_e4m3_verify_b64"),
        # a long shared context with per-head INT8 scales, plain decode
        dict(_shared("int8", 61, 1, 32, 8, 1, 131072, 512), name="shared_int8_decode_b61"),
        # several system prompts in one batch, run-time row scales, odd sizes
        dict(_shared("int8_row", 45, 4, 32, 8, 5, 9001, 777), name="shared_int8_row_verify_g4"),
        # a wide decode batch with short private parts
        dict(_shared("fp8_e4m3", 256, 2, 32, 8, 1, 16384, 300), name="shared_e4m3_decode_b256"),
        # the widest verify (8 positions, 32 rows a kv-head) on an fp16 pool
        dict(_shared("fp16", 32, 1, 32, 8, 8, 16384, 1500), name="shared_fp16_verify_b32"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "truncate", "shared", "shared", "shared", "shared"])
    if op == "extend":
        batch = _log(rng, 1, 2048)
        if rng.random() < 0.5:
            return _extend(batch, _log(rng, 16, 32768 if batch <= 256 else 4096), rng.randint(1, 8),
                           True)
        return _extend(batch, _log(rng, 16, 4096), _log(rng, 9, min(8192, 2000000 // batch)), False)
    if op == "truncate":
        batch = _log(rng, 1, 2048)
        return _truncate(batch, _log(rng, 64, min(131072, 12000000 // batch)), rng.randint(1, 8),
                         rng.random() < 0.4)
    fmt = rng.choice(sorted(FORMATS))
    hq, hkv = rng.choice([(32, 8), (32, 8), (8, 1), (16, 4), (24, 8), (16, 16), (64, 8)])
    q_len = rng.choice([q for q in (1, 1, 2, 3, 5, 5, 8) if q * hq // hkv <= 32])
    batch = _log(rng, 2, 256)
    groups = rng.choice([1, 1, 1, 2, 3, 5])
    # at most the largest listed case's work: rows x prefix, and the private keys
    prefix = _log(rng, 64, 131072)
    prefix = max(64, min(prefix, int(2.0e8 / (batch * q_len * hq / 32.0) / 32)))
    suffix = _log(rng, 16, max(32, min(2048, 65536 // batch)))
    return _shared(fmt, batch, min(groups, batch), hq, hkv, q_len, prefix, max(suffix, q_len + 1))


def _case_rng(case):
    plain = {k: v for k, v in case.items() if k != "name"}
    return np.random.default_rng(zlib.crc32(json.dumps(plain, sort_keys=True).encode()))


def _pages(n):
    return -(-n // PAGE)


def _extend_lengths(case):
    r = _case_rng(case)
    B = case["batch"]
    lens = r.integers(0 if not case["fixed"] else 1, case["cached"], B, endpoint=True)
    new = np.full(B, case["new"]) if case["fixed"] else r.integers(0, case["new"], B, endpoint=True)
    if not case["fixed"]:
        new[B // 2] = max(1, new[B // 2])
    return lens.astype(np.int64), new.astype(np.int64)


def _truncate_lengths(case):
    r = _case_rng(case)
    B = case["batch"]
    lens = r.integers(case["cached"] // 2, case["cached"], B, endpoint=True)
    keep = np.maximum(lens - r.integers(0, case["drop"], B), 0)
    owned = r.integers(0, np.maximum(keep // PAGE // 4, 1), B)
    if case["release"]:
        keep[::3] = 0
    return lens.astype(np.int64), keep.astype(np.int64), owned.astype(np.int64)


def _shared_lengths(case):
    """(group offsets, prefix length of each group, length of each sequence)."""
    r = _case_rng(case)
    B, n = case["batch"], case["groups"]
    cuts = np.sort(r.choice(np.arange(1, B), n - 1, replace=False)) if n > 1 else np.array([], int)
    offsets = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    prefix = r.integers(max(16, 3 * case["prefix"] // 4), case["prefix"], n, endpoint=True)
    prefix[0] = case["prefix"]
    own_part = r.integers(case["q_len"], case["suffix"], B, endpoint=True)
    lens = np.repeat(prefix, np.diff(offsets)) + own_part
    return offsets, prefix.astype(np.int64), lens.astype(np.int64)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=torch.int32)


def _perm(n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _tables(lens, width, perm):
    """Block tables of requests of these lengths on the pages of `perm`, -1
    behind each request's last page; and how many pages they take."""
    need = _pages(lens)
    start = np.concatenate([[0], np.cumsum(need)])
    j = torch.arange(width, device="cuda")[None]
    at = torch.from_numpy(start[:-1]).cuda()[:, None] + j
    live = j < torch.from_numpy(need).cuda()[:, None]
    table = torch.where(live, perm[at.clamp(max=perm.numel() - 1)], torch.full_like(perm[:1], -1))
    return table.contiguous(), int(start[-1])


def _prepare_extend(case, seed):
    lens, new = _extend_lengths(case)
    B = case["batch"]
    width = int(_pages(lens + new).max())
    used = int(_pages(lens).sum())
    need = int((_pages(lens + new) - _pages(lens)).sum())
    num_pages = used + need + 64
    perm = _perm(num_pages, seed)
    table, _ = _tables(lens, width, perm)
    total = max(64, -(-int(new.sum()) // 64) * 64)       # the step's token bucket
    return {"case": case, "seq_lens": _i32(lens), "new_tokens": _i32(new), "block_table": table,
            "free_pages": perm[used:].contiguous(), "free_count": _i32([num_pages - used]),
            "num_pages": num_pages, "num_tokens": total,
            "seq_lens_out": torch.empty(B, dtype=torch.int32, device="cuda"),
            "free_count_out": torch.empty(1, dtype=torch.int32, device="cuda"),
            "slot_mapping": torch.empty(total, dtype=torch.int64, device="cuda"),
            "positions": torch.empty(total, dtype=torch.int32, device="cuda"),
            "token_offsets": torch.empty(B + 1, dtype=torch.int32, device="cuda")}


def _prepare_truncate(case, seed):
    lens, keep, owned = _truncate_lengths(case)
    B = case["batch"]
    used = int(_pages(lens).sum())
    num_pages = used + 64
    perm = _perm(num_pages, seed)
    table, _ = _tables(lens, int(_pages(lens).max()), perm)
    free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free[:64] = perm[used:]
    return {"case": case, "seq_lens": _i32(lens), "keep_lens": _i32(keep), "block_table": table,
            "owned_pages": _i32(owned), "free_pages": free, "free_count": _i32([64]),
            "seq_lens_out": torch.empty(B, dtype=torch.int32, device="cuda"),
            "free_count_out": torch.empty(1, dtype=torch.int32, device="cuda")}


def _values(shape, gen):
    """N(0, 1) with about 1% outliers twenty times as large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x * (1.0 + 19.0 * (torch.rand(shape, generator=gen, device="cuda") < 0.01))


def _prepare_pool(fmt, num_pages, hkv, gen):
    """A pool [num_pages, hkv, 2, 16, 128] of encoded values with its scales."""
    shape = (num_pages, hkv, 2, PAGE, DIM)
    kinds = {"fp16": torch.float16}
    n = num_pages * hkv * 2 * PAGE * DIM
    extra = num_pages * hkv * 2 * PAGE * 2 if fmt == "int8_row" else 0
    flat = torch.empty(n + extra, dtype=kinds.get(fmt, torch.uint8), device="cuda")
    pages = flat[:n].view(shape)
    amax = 90.0
    if fmt == "fp8_e4m3":
        ks = torch.full((1,), amax / 448.0, device="cuda")
        vs = torch.full((1,), 0.9 * amax / 448.0, device="cuda")
    elif fmt == "int8":
        ks = amax / 127.0 * torch.linspace(0.8, 1.0, hkv, device="cuda")
        vs = amax / 127.0 * torch.linspace(1.0, 0.9, hkv, device="cuda")
    else:
        ks = vs = torch.ones(1, device="cuda")
    row = flat[n:].view(torch.float16).view(num_pages, hkv, 8, 2, 2) if extra else None
    step = max(1, (1 << 26) // (hkv * 2 * PAGE * DIM))
    for a in range(0, num_pages, step):
        b = min(num_pages, a + step)
        x = _values((b - a,) + shape[1:], gen)
        if fmt == "fp16":
            pages[a:b] = x.half()
        elif fmt == "int8_row":
            x = x.half().float()
            r = (x.abs().amax(-1) / 127.0).half()                  # [n, hkv, 2, 16]
            pages[a:b] = (x / r.float()[..., None]).round().clamp(-127, 127).to(torch.int8).view(
                torch.uint8)
            # the stored order: [page][head][row % 8][K or V][row // 8]
            row[a:b] = r.view(b - a, hkv, 2, 2, 8).permute(0, 1, 4, 2, 3)
        else:
            both = torch.stack([ks.expand(hkv), vs.expand(hkv)], 1)[None, :, :, None, None]
            x = x / both
            pages[a:b] = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                          if fmt == "fp8_e4m3" else
                          x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8))
    return flat, pages, row, ks, vs


def _prepare_shared(case, seed):
    offsets, prefix, lens = _shared_lengths(case)
    B, hq, hkv, q_len = case["batch"], case["hq"], case["hkv"], case["q_len"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    shared = prefix // PAGE                                # whole pages are shared
    per_seq = np.repeat(shared, np.diff(offsets))
    private = _pages(lens) - per_seq
    num_pages = int(shared.sum() + private.sum()) + 7
    perm = _perm(num_pages, seed + 1)
    width = int(_pages(lens).max())
    heads, used = _tables(shared * PAGE, int(max(shared.max(), 1)), perm)
    tails, _ = _tables(private * PAGE, int(private.max()), perm[used:])
    j = torch.arange(width, device="cuda")[None]
    cut = torch.from_numpy(per_seq).cuda()[:, None]
    group = torch.from_numpy(np.repeat(np.arange(len(prefix)), np.diff(offsets))).cuda()
    table = torch.where(j < cut, heads[group][:, j[0].clamp(max=heads.shape[1] - 1)],
                        tails.gather(1, (j - cut).clamp(0, tails.shape[1] - 1)))
    flat, pages, row, ks, vs = _prepare_pool(case["format"], num_pages, hkv, gen)
    q = torch.randn((B * q_len, hq, DIM), generator=gen, device="cuda").half()
    return {"case": case, "q": q, "flat": flat, "pages": pages, "row_scales": row, "k_scale": ks,
            "v_scale": vs, "block_table": table.contiguous(), "seq_lens": _i32(lens),
            "group_offsets": _i32(offsets), "prefix_lens": _i32(prefix),
            "max_seq_len": int(lens.max()), "max_prefix_len": int(prefix.max()),
            "largest_group": int(np.diff(offsets).max()), "out": torch.empty_like(q)}


def prepare(case, seed):
    return {"extend": _prepare_extend, "truncate": _prepare_truncate,
            "shared": _prepare_shared}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_extend(s):
    L, n = s["seq_lens"].long(), s["new_tokens"].long()
    table, free, fc = s["block_table"], s["free_pages"], s["free_count"].long()
    B, width = table.shape
    T = s["num_tokens"]
    offsets = torch.cat([torch.zeros_like(fc), n.cumsum(0)])
    fits = (L + n <= width * PAGE) & (offsets[1:] <= T)
    have = (L + PAGE - 1) // PAGE
    need = torch.where(fits, (L + n + PAGE - 1) // PAGE - have, torch.zeros_like(n))
    upto = need.cumsum(0)
    granted = fits & ((need == 0) | (upto <= fc))
    taken = torch.where(granted, need, torch.zeros_like(need))
    j = torch.arange(width, device=L.device)[None]
    fresh = (j >= have[:, None]) & (j < (have + taken)[:, None])
    at = fc - 1 - (upto - need)[:, None] - (j - have[:, None])
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(T, device=L.device)
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = L[r] + t - offsets[r]
    page = table[r, (pos // PAGE).clamp(0, width - 1)].long()
    live = (t < offsets[-1]) & granted[r] & (page >= 0) & (page < s["num_pages"])
    none = torch.full_like(pos, -1)
    return {"seq_lens": torch.where(granted, L + n, L).int(),
            "free_count": (fc - taken.sum()).int(), "block_table": table,
            "slot_mapping": torch.where(live, page * PAGE + pos % PAGE, none),
            "positions": torch.where(live, pos, none).int(),
            "token_offsets": offsets.clamp(max=T).int()}


def _plain_truncate(s):
    L, keep = s["seq_lens"].long(), s["keep_lens"].long()
    table, free, fc = s["block_table"], s["free_pages"], s["free_count"].long()
    first = torch.maximum((keep + PAGE - 1) // PAGE, s["owned_pages"].long())
    last = (L + PAGE - 1) // PAGE
    j = torch.arange(table.shape[1], device=L.device)[None]
    gone = (j >= first[:, None]) & (j < last[:, None])
    rank = gone.reshape(-1).long().cumsum(0).view(gone.shape) - 1
    at = torch.where(gone, fc + rank, torch.full_like(rank, free.numel()))
    spare = torch.cat([free, free[:1]])                 # one place behind for what stays
    spare = spare.scatter(0, at.reshape(-1), table.reshape(-1))[:-1]
    return {"seq_lens": keep.int(), "free_count": (fc + gone.sum()).int(), "free_pages": spare}


def _decode(s, ids, h, kv):
    """fp32 rows [..., 128] of one kv-head's K (kv 0) or V (kv 1) of these pages."""
    fmt = s["case"]["format"]
    x = s["pages"][ids, h, kv]
    if fmt == "fp16":
        x = x.float()
    elif fmt == "fp8_e4m3":
        x = x.view(torch.float8_e4m3fn).float() * (s["v_scale"] if kv else s["k_scale"])
    elif fmt == "int8":
        x = x.view(torch.int8).float() * (s["v_scale"] if kv else s["k_scale"])[h]
    else:
        r = s["row_scales"][ids, h][..., kv, :]                     # [..., 8, 2]
        x = x.view(torch.int8).float() * r.transpose(-1, -2).reshape(x.shape[:-1])[..., None].float()
    return x.flatten(-3, -2)


def _plain_shared(s):
    case = s["case"]
    B, hq, hkv, q_len = case["batch"], case["hq"], case["hkv"], case["q_len"]
    G = hq // hkv
    q, table, L = s["q"], s["block_table"].long(), s["seq_lens"].long()
    offsets, plen = s["group_offsets"].long(), s["prefix_lens"].long()
    ids = torch.arange(B, device=q.device)
    group = torch.searchsorted(offsets[1:].contiguous(), ids, right=True)
    place = ids - offsets[group]
    shared = plen // PAGE                                           # pages read once a group
    n, most = plen.numel(), max(1, s["max_prefix_len"] // PAGE)
    heads = table[offsets[:-1]][:, :most].clamp(min=0)
    room = _pages(case["suffix"]) + 1                               # private pages at most
    j = torch.arange(room, device=q.device)[None]
    tails = table.gather(1, (shared[group][:, None] + j).clamp(max=table.shape[1] - 1)).clamp(min=0)
    in_prefix = torch.arange(most * PAGE, device=q.device)[None] < (shared * PAGE)[:, None]
    pos = (shared[group] * PAGE)[:, None] + torch.arange(room * PAGE, device=q.device)[None]
    last = L[:, None] - q_len + torch.arange(q_len, device=q.device)[None]
    seen = pos[:, None, :] <= last[:, :, None]                      # [B, q_len, keys]
    live = (pos < L[:, None])[..., None]
    no = torch.full((), -math.inf, device=q.device)
    scale = 1.0 / math.sqrt(DIM)
    out = torch.empty_like(q).view(B, q_len, hkv, G, DIM)
    for h in range(hkv):
        rows = q.view(B, q_len, hkv, G, DIM)[:, :, h].float() * scale
        wide = rows.new_zeros((n, s["largest_group"], q_len * G, DIM))
        wide[group, place] = rows.reshape(B, q_len * G, DIM)
        wide = wide.view(n, -1, DIM)
        a = wide @ _decode(s, heads, h, 0).transpose(1, 2)          # [n, rows, prefix keys]
        a = torch.where(in_prefix[:, None], a, no)
        b = rows.reshape(B, q_len * G, DIM) @ _decode(s, tails, h, 0).transpose(1, 2)
        b = torch.where(seen.repeat_interleave(G, 1), b, no)
        ma = a.amax(-1).view(n, -1, q_len * G)
        m = torch.maximum(ma[group, place], b.amax(-1))             # [B, q_len * G]
        back = torch.zeros_like(ma)
        back[group, place] = m
        pa = torch.exp(a - back.view(n, -1)[..., None])
        pb = torch.exp(b - m[..., None])
        oa = (pa @ _decode(s, heads, h, 1)).view(n, -1, q_len * G, DIM)[group, place]
        la = pa.sum(-1).view(n, -1, q_len * G)[group, place]
        ob = pb @ torch.where(live, _decode(s, tails, h, 1), torch.zeros((), device=q.device))
        o = (oa + ob) / (la + pb.sum(-1))[..., None]
        out[:, :, h] = o.view(B, q_len, G, DIM).half()
    return out.view(B * q_len, hq, DIM)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"extend": _plain_extend, "truncate": _plain_truncate,
                "shared": _plain_shared}[op](state)
    import paged_quantized_kv_append_gb300 as pq
    s = state
    if op == "extend":
        pq.extend_block_tables(s["seq_lens"], s["new_tokens"], s["block_table"], s["free_pages"],
                               s["free_count"], s["num_pages"], s["seq_lens_out"],
                               s["free_count_out"], s["slot_mapping"], s["positions"],
                               s["token_offsets"])
        return {"seq_lens": s["seq_lens_out"], "free_count": s["free_count_out"],
                "block_table": s["block_table"], "slot_mapping": s["slot_mapping"],
                "positions": s["positions"], "token_offsets": s["token_offsets"]}
    if op == "truncate":
        pq.truncate_block_tables(s["seq_lens"], s["keep_lens"], s["block_table"], s["free_pages"],
                                 s["free_count"], s["seq_lens_out"], s["free_count_out"],
                                 owned_pages=s["owned_pages"])
        return {"seq_lens": s["seq_lens_out"], "free_count": s["free_count_out"],
                "free_pages": s["free_pages"]}
    return pq.paged_attention_shared_prefix(
        s["q"], s["pages"], s["block_table"], s["seq_lens"], s["group_offsets"], s["prefix_lens"],
        s["case"]["q_len"], FORMATS[s["case"]["format"]], s["k_scale"], s["v_scale"], s["out"],
        max_seq_len=s["max_seq_len"], max_prefix_len=s["max_prefix_len"])


def work(case):
    B = case["batch"]
    if case["op"] == "extend":
        lens, new = _extend_lengths(case)
        fresh = int((_pages(lens + new) - _pages(lens)).sum())
        tokens = max(64, -(-int(new.sum()) // 64) * 64)
        started = int(((lens % PAGE > 0) & (new > 0)).sum())     # table entries read
        return {"bytes": B * 4 * 4 + 4 * 3 + fresh * 8 + started * 4 + tokens * 12, "flops": 0}
    if case["op"] == "truncate":
        lens, keep, owned = _truncate_lengths(case)
        gone = int(np.maximum(_pages(lens) - np.maximum(_pages(keep), owned), 0).sum())
        return {"bytes": B * 4 * 4 + 8 + gone * 8, "flops": 0}
    offsets, prefix, lens = _shared_lengths(case)
    hq, hkv, q_len = case["hq"], case["hkv"], case["q_len"]
    shared = prefix // PAGE * PAGE
    per_seq = np.repeat(shared, np.diff(offsets))
    keys = int(shared.sum() + (lens - per_seq).sum())
    key_bytes = {"fp16": 512, "fp8_e4m3": 256, "int8": 256, "int8_row": 260}[case["format"]]
    seen = int((lens * q_len - q_len * (q_len - 1) // 2).sum())    # keys seen, over all queries
    return {"bytes": keys * hkv * key_bytes + 2 * B * q_len * hq * DIM * 2
            + (_pages(keys) + 2 * B) * 4, "flops": 4 * seen * hq * DIM}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "shared":
        return None                                          # whole numbers only
    s = _prepare_shared(case, seed)
    hq, hkv, q_len, fmt = case["hq"], case["hkv"], case["q_len"], case["format"]
    G = hq // hkv
    _, _, lens = _shared_lengths(case)
    if 4.0 * lens.sum() * q_len * hq * DIM > 4e12:           # at about 0.5 TFLOP/s
        return None
    out = torch.empty((len(lens) * q_len, hq, DIM), dtype=torch.float64, device="cuda")
    # the value of every code of a format, from its definition
    code = torch.arange(256, device="cuda")
    if fmt == "fp8_e4m3":
        e, m = (code >> 3) & 15, (code & 7).double()
        mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7).double())
        value = torch.where(code < 128, mag, -mag)
    else:
        value = torch.where(code < 128, code, code - 256).double()
    for i, n in enumerate(lens.tolist()):
        ids = s["block_table"][i, :_pages(n)].long()
        sees = torch.arange(n, device="cuda")[None] <= (
            n - q_len + torch.arange(q_len, device="cuda"))[:, None]
        for h in range(hkv):
            kv = s["pages"][ids, h]                          # [pages, 2, 16, 128]
            kv = kv.double() if fmt == "fp16" else value[kv.long()]
            K = kv[:, 0].reshape(-1, DIM)[:n]
            V = kv[:, 1].reshape(-1, DIM)[:n]
            if fmt == "int8_row":
                t = torch.arange(n, device="cuda")
                pg, r = ids[t // PAGE], t % PAGE
                K = K * s["row_scales"][pg, h, r % 8, 0, r // 8].double()[:, None]
                V = V * s["row_scales"][pg, h, r % 8, 1, r // 8].double()[:, None]
            elif fmt != "fp16":
                hh = h if s["k_scale"].numel() > 1 else 0
                K = K * s["k_scale"][hh].double()
                V = V * s["v_scale"][hh].double()
            x = s["q"][i * q_len:(i + 1) * q_len, h * G:(h + 1) * G].double()
            z = torch.einsum("igd,nd->ign", x, K) / DIM ** 0.5
            z = z.masked_fill(~sees[:, None], -math.inf)
            out[i * q_len:(i + 1) * q_len, h * G:(h + 1) * G] = torch.einsum(
                "ign,nd->igd", torch.softmax(z, -1), V)
    return out

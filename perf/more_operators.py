"""Measured cases of a KV pool held in 4 bits, and of reading a pool back.

Three operators, each in its plain form (elementary torch operations in 32
bits) and as the library's own calls:

  kv_append_quant  ("int4_group")  new K/V rows quantised to 4 bits, with an
                   fp16 scale per 32 values found as they are written; what
                   was written is read back, since a prompt's next chunk
                   attends to it
  paged_attention  ("int4_group")  decode, verify and sliding-window attention
                   over a 4-bit pool
  kv_read          the tokens of requests out of a pool of any format, as
                   contiguous fp16 rows

A 4-bit pool is uint8 [num_pages, num_kv_heads, 2, 16, 72]: the 1152 bytes of a
K (or V) tile are 1024 bytes of codes, then fp16 scales [4 groups][16 rows].
Of the codes, line i (128 bytes) holds rows 2 i and 2 i + 1: the 16 bytes of
group c of row r are chunk (4 (r % 2) + c) ^ (0, 5, 2, 7)[i % 4].  In them, word
w (32 bits) holds values 8 w .. 8 w + 7; value 8 w + 2 f + e is in half e, as
code + 8 rotated left by (6, 2, 10, 14)[f] bits within the half's 16.

Lengths are a function of the case alone, so that work() is exact; values and
page numbers come from the seed.
"""
import json
import math
import zlib

import numpy as np
import torch

own = False

PAGE = 16
DIM = 128
GROUP = 32                       # values that share a scale in a 4-bit pool
MOST_SCALE = 2720.0              # its largest scale
ROW_BYTES = {"fp16": 256, "fp8_e4m3": 128, "int8": 128, "int8_row": 130, "int4_group": 72}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(batch, hkv, cached, new, fixed, context):
    return {"op": "append", "batch": batch, "hkv": hkv, "cached": cached, "new": new,
            "fixed": fixed, "context": context}


def _attend(batch, hq, hkv, q_len, shortest, longest, window):
    return {"op": "attend", "batch": batch, "hq": hq, "hkv": hkv, "q_len": q_len,
            "shortest": shortest, "longest": longest, "window": window}


def _read(fmt, batch, hkv, longest, part):
    return {"op": "read", "format": fmt, "batch": batch, "hkv": hkv, "longest": longest,
            "part": part}


def listed():
    return [
        # four prompts' chunks written and read back for the dense attention over them
        dict(_append(4, 8, 0, 2048, True, False), name="append_prompt_b4"),
        # one token of each request of the largest batch: a decode step's write
        dict(_append(2048, 8, 4096, 1, True, False), name="append_decode_b2048"),
        # ragged chunks of prompts behind cached ones, the whole context read back
        dict(_append(24, 8, 4096, 513, False, True), name="append_context_b24"),
        # the smallest attention: short contexts, one kv-head
        dict(_attend(4, 8, 1, 1, 512, 1024, 0), name="attend_tiny"),
        # 8 concurrent requests of ragged contexts, plain decode
        dict(_attend(8, 32, 8, 1, 2048, 32768, 0), name="attend_decode_b8"),
        # the same batch at 128K tokens each, verify of 4 draft tokens
        dict(_attend(8, 32, 8, 5, 131072, 131072, 0), name="attend_verify_b8_131k"),
        # the drafter's sliding-window layers over the same caches
        dict(_attend(8, 32, 8, 5, 131072, 131072, 2048), name="attend_window_b8_131k"),
        # one request at the longest context, 32 query rows a kv-head
        dict(_attend(1, 64, 8, 4, 524288, 524288, 0), name="attend_verify_512k"),
        # a wide decode batch of a model whose every query head has its own kv-head
        dict(_attend(256, 16, 16, 1, 64, 4096, 0), name="attend_mha_b256"),
        # a long request taken out of its pool (moved to another one, or to the host)
        dict(_read("fp8_e4m3", 1, 8, 131072, False), name="read_e4m3_131k"),
        # the cached context of many prompts, from odd positions on
        dict(_read("int4_group", 45, 8, 9001, True), name="read_int4_b45"),
        # a few short contexts of one kv-head: nothing but latency
        dict(_read("fp16", 4, 1, 1024, False), name="read_fp16_tiny"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_ROWS = 8 * 131072 * 8       # (token, kv-head) rows of the largest listed case


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "read"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    if op == "append":
        batch = _log(rng, 1, 2048)
        cached = rng.choice([0, _log(rng, 16, 8192)])
        if rng.random() < 0.4:
            return _append(batch, hkv, cached, rng.randint(1, 8), True, False)
        new = _log(rng, 9, max(16, min(8192, 65536 // batch)))
        context = (cached + new) * batch <= 262144 and rng.random() < 0.5
        return _append(batch, hkv, cached, new, False, context)
    if op == "attend":
        hq, hkv = rng.choice([(32, 8), (32, 8), (8, 1), (16, 4), (24, 8), (16, 16), (64, 8)])
        q_len = rng.choice([q for q in (1, 1, 2, 3, 5, 5, 8) if q * hq // hkv <= 32])
        batch = _log(rng, 1, 256)
        longest = _log(rng, 64, max(128, min(524288, MOST_ROWS // hkv // batch)))
        window = rng.choice([0, 0, 0, _log(rng, 16, longest)])
        return _attend(batch, hq, hkv, q_len, max(q_len, longest // rng.choice([1, 2, 20])),
                       longest, window)
    batch = _log(rng, 1, 256)
    longest = _log(rng, 16, max(64, min(131072, MOST_ROWS // 8 // hkv // batch)))
    return _read(rng.choice(sorted(ROW_BYTES)), batch, hkv, longest, rng.random() < 0.5)


def _case_rng(case):
    plain = {k: v for k, v in case.items() if k != "name"}
    return np.random.default_rng(zlib.crc32(json.dumps(plain, sort_keys=True).encode()))


def _pages(n):
    return -(-n // PAGE)


def _append_lengths(case):
    """(cached tokens, new tokens, first token that is read back) of each request."""
    r = _case_rng(case)
    B = case["batch"]
    lens = r.integers(case["cached"] // 2, case["cached"], B, endpoint=True)
    new = np.full(B, case["new"]) if case["fixed"] else r.integers(0, case["new"], B, endpoint=True)
    if not case["fixed"]:
        new[B // 2] = max(1, new[B // 2])
    first = np.zeros(B, np.int64) if case["context"] else lens
    return lens.astype(np.int64), new.astype(np.int64), first.astype(np.int64)


def _attend_lengths(case):
    r = _case_rng(case)
    return r.integers(case["shortest"], case["longest"], case["batch"], endpoint=True)


def _read_lengths(case):
    """(tokens, first token read, tokens read) of each request."""
    r = _case_rng(case)
    B = case["batch"]
    lens = r.integers(case["longest"] // 2, case["longest"], B, endpoint=True)
    if not case["part"]:
        lens[0] = case["longest"]
        return lens, np.zeros(B, np.int64), lens
    first = r.integers(0, np.maximum(lens // 3, 1), B)
    return lens, first, np.maximum(r.integers(lens // 2, lens, B, endpoint=True) - first, 0)


# ---------------------------------------------------------------------------
# a 4-bit pool's bytes
# ---------------------------------------------------------------------------
def _places(row):
    """Bytes of a K (or V) tile that row `row` (a tensor) takes: 64 of codes, 8 of scales."""
    line = (row // 2)[..., None, None]
    turn = torch.tensor([0, 5, 2, 7], device=row.device)[line % 4]
    chunk = (row % 2 * 4)[..., None, None] + torch.arange(4, device=row.device)[:, None]
    codes = line * 128 + (chunk ^ turn) * 16 + torch.arange(16, device=row.device)
    scales = 1024 + 2 * (torch.arange(4, device=row.device)[:, None] * 16 + row[..., None, None])
    scales = scales + torch.arange(2, device=row.device)
    return torch.cat([codes.flatten(-2), scales.flatten(-2)], -1)


def _turns(device):
    return torch.tensor([6, 2, 10, 14], dtype=torch.int32, device=device)


def _row_values(rows):
    """fp32 values [..., 128] of rows of 72 bytes, in the order of _places."""
    words = rows[..., :64].contiguous().view(torch.int32)                  # [..., 16]
    half = torch.stack([words & 0xFFFF, (words >> 16) & 0xFFFF], -1)       # [..., 16, e]
    half = (half | (half << 16))[..., None, :]
    code = ((half >> _turns(rows.device)[:, None]) & 15) - 8               # [..., 16, f, e]
    scale = rows[..., 64:].contiguous().view(torch.float16).float()
    return (code.flatten(-3).unflatten(-1, (4, GROUP)).float() * scale[..., None]).flatten(-2)


def _row_bytes(x):
    """Rows of 72 bytes, in the order of _places, of fp16 rows [..., 128]."""
    x = x.float().unflatten(-1, (4, GROUP))
    # (divided by a tensor: by a number it would be a product with the rounded 1 / 7)
    scale = (x.abs().amax(-1) / x.new_full((), 7.0)).bfloat16().half().clamp(max=MOST_SCALE)
    s = scale.float()[..., None]
    code = torch.where(s > 0, (x / s).round().clamp(-7, 7), torch.zeros_like(x)).int() + 8
    code = code.flatten(-2).unflatten(-1, (16, 4, 2))                      # [..., word, f, e]
    wide = code << _turns(x.device)[:, None]
    half = ((wide & 0xFFFF) | (wide >> 16)).sum(-2, dtype=torch.int32)     # [..., word, e]
    codes = half.to(torch.int16).view(torch.uint8).flatten(-2)
    return torch.cat([codes, scale.contiguous().view(torch.uint8)], -1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=torch.int32)


def _tables(lens, num_pages, seed):
    """Block tables of requests of these lengths on shuffled pages, -1 behind
    each request's last page."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    need = _pages(lens)
    start = np.concatenate([[0], np.cumsum(need)])[:-1]
    j = torch.arange(max(1, int(need.max())), device="cuda")[None]
    at = torch.from_numpy(start).cuda()[:, None] + j
    live = j < torch.from_numpy(need).cuda()[:, None]
    return torch.where(live, perm[at.clamp(max=num_pages - 1)], torch.full_like(perm[:1], -1))


def _values(shape, gen):
    """N(0, 1) with about 1% outliers twenty times as large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x * (1.0 + 19.0 * (torch.rand(shape, generator=gen, device="cuda") < 0.01))


def _pool(fmt, num_pages, hkv, gen):
    """A pool of encoded values with its scales, as a dict."""
    n = num_pages * hkv * 2 * PAGE * DIM
    tiles = (num_pages, hkv, 2, PAGE, DIM)
    ks = vs = torch.ones(1, device="cuda")
    row = None
    if fmt == "int4_group":
        pages = torch.empty((num_pages, hkv, 2, PAGE, 72), dtype=torch.uint8, device="cuda")
        flat = pages.view(num_pages, hkv, 2, PAGE * 72)
        at = _places(torch.arange(PAGE, device="cuda"))
        back = torch.argsort(at.flatten())
    else:
        extra = num_pages * hkv * 2 * PAGE * 2 if fmt == "int8_row" else 0
        whole = torch.empty(n + extra, device="cuda",
                            dtype=torch.float16 if fmt == "fp16" else torch.uint8)
        pages = whole[:n].view(tiles)
        row = whole[n:].view(torch.float16).view(num_pages, hkv, 8, 2, 2) if extra else None
    if fmt == "fp8_e4m3":
        ks, vs = torch.full((1,), 90.0 / 448, device="cuda"), torch.full((1,), 81.0 / 448, device="cuda")
    elif fmt == "int8":
        ks = 90.0 / 127 * torch.linspace(0.8, 1.0, hkv, device="cuda")
        vs = 90.0 / 127 * torch.linspace(1.0, 0.9, hkv, device="cuda")
    step = max(1, (1 << 26) // (hkv * 2 * PAGE * DIM))
    for a in range(0, num_pages, step):
        b = min(num_pages, a + step)
        x = _values((b - a,) + tiles[1:], gen)
        if fmt == "int4_group":
            flat[a:b] = _row_bytes(x.half()).flatten(-2)[..., back]
        elif fmt == "fp16":
            pages[a:b] = x.half()
        elif fmt == "int8_row":
            x = x.half().float()
            r = (x.abs().amax(-1) / 127.0).half()                  # [n, hkv, 2, 16]
            pages[a:b] = (x / r.float()[..., None]).round().clamp(-127, 127).to(torch.int8).view(
                torch.uint8)
            # the stored order: [page][head][row % 8][K or V][row // 8]
            row[a:b] = r.view(b - a, hkv, 2, 2, 8).permute(0, 1, 4, 2, 3)
        else:
            x = x / torch.stack([ks.expand(hkv), vs.expand(hkv)], 1)[None, :, :, None, None]
            pages[a:b] = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                          if fmt == "fp8_e4m3" else
                          x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8))
    return {"pages": pages, "row_scales": row, "k_scale": ks, "v_scale": vs}


def _offsets(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]))


def _prepare_append(case, seed):
    lens, new, first = _append_lengths(case)
    hkv = case["hkv"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    num_pages = int(_pages(lens + new).sum()) + 7
    table = _tables(lens + new, num_pages, seed + 1)
    s = _pool("int4_group", num_pages, hkv, gen)
    T = int(new.sum())
    # K and V are column slices of one projection's output
    qkv = _values((T, 2 * hkv * DIM), gen).half()
    seq = torch.from_numpy(np.repeat(np.arange(len(new)), new)).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(a, a + n) for a, n in zip(lens, new)])).cuda()
    slots = table[seq, pos // PAGE].long() * PAGE + pos % PAGE
    back = int((lens + new - first).sum())
    s.update(case=case, k=qkv[:, :hkv * DIM].view(T, hkv, DIM), v=qkv[:, hkv * DIM:].view(T, hkv, DIM),
             slots=slots, block_table=table, first=_i32(first), offsets=_offsets(lens + new - first),
             k_out=torch.empty((back, hkv, DIM), dtype=torch.float16, device="cuda"),
             v_out=torch.empty((back, hkv, DIM), dtype=torch.float16, device="cuda"))
    return s


def _prepare_attend(case, seed):
    lens = _attend_lengths(case)
    B, hq, hkv, q_len = case["batch"], case["hq"], case["hkv"], case["q_len"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    num_pages = int(_pages(lens).sum()) + 7
    s = _pool("int4_group", num_pages, hkv, gen)
    q = torch.randn((B * q_len, hq, DIM), generator=gen, device="cuda").half()
    s.update(case=case, q=q, out=torch.empty_like(q), block_table=_tables(lens, num_pages, seed + 1),
             seq_lens=_i32(lens), max_seq_len=int(lens.max()))
    return s


def _prepare_read(case, seed):
    lens, first, n = _read_lengths(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    num_pages = int(_pages(lens).sum()) + 7
    s = _pool(case["format"], num_pages, case["hkv"], gen)
    shape = (int(n.sum()), case["hkv"], DIM)
    s.update(case=case, block_table=_tables(lens, num_pages, seed + 1), first=_i32(first),
             offsets=_offsets(n), k_out=torch.empty(shape, dtype=torch.float16, device="cuda"),
             v_out=torch.empty(shape, dtype=torch.float16, device="cuda"))
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "attend": _prepare_attend,
            "read": _prepare_read}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_read(s, fmt):
    """fp16 K and V of the tokens first[i] .. first[i] + offsets[i + 1] - offsets[i] - 1."""
    offsets = s["offsets"].long()
    t = torch.arange(s["k_out"].shape[0], device=offsets.device)
    seq = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    pos = s["first"].long()[seq] + t - offsets[seq]
    page, row = s["block_table"].long()[seq, pos // PAGE], pos % PAGE
    if fmt == "int4_group":
        tiles = s["pages"].flatten(-2)                                     # [pages, H, 2, 1152]
        H = tiles.shape[1]
        rows = tiles[page[:, None, None, None], torch.arange(H, device=t.device)[:, None, None],
                     torch.arange(2, device=t.device)[:, None], _places(row)[:, None, None, :]]
        x = _row_values(rows)
    else:
        x = s["pages"][page, :, :, row]                                    # [T, H, 2, 128]
        if fmt == "fp8_e4m3":
            x = x.view(torch.float8_e4m3fn).float()
        else:
            x = x.float() if fmt == "fp16" else x.view(torch.int8).float()
        if fmt == "int8_row":
            x = x * s["row_scales"][page, :, row % 8, :, row // 8].float()[..., None]
        elif fmt != "fp16":
            H = x.shape[1]
            x = x * torch.stack([s["k_scale"].expand(H), s["v_scale"].expand(H)], 1)[..., None]
    x = x.half()
    return {"k": x[:, :, 0], "v": x[:, :, 1]}


def _plain_append(s):
    rows = torch.stack([_row_bytes(s["k"]), _row_bytes(s["v"])], 2)        # [T, H, 2, 72]
    tiles = s["pages"].flatten(-2)
    page, row = s["slots"] // PAGE, s["slots"] % PAGE
    H = tiles.shape[1]
    tiles[page[:, None, None, None], torch.arange(H, device=page.device)[:, None, None],
          torch.arange(2, device=page.device)[:, None], _places(row)[:, None, None, :]] = rows
    return _plain_read(s, "int4_group")


def _plain_attend(s):
    case = s["case"]
    B, hq, hkv, q_len = case["batch"], case["hq"], case["hkv"], case["q_len"]
    G = hq // hkv
    L = s["seq_lens"].long()
    ids = s["block_table"].long().clamp(min=0)                             # [B, width]
    at = _places(torch.arange(PAGE, device=ids.device))
    pos = torch.arange(ids.shape[1] * PAGE, device=ids.device)
    last = L[:, None] - q_len + torch.arange(q_len, device=ids.device)     # [B, q_len]
    sees = pos <= last[..., None]
    if case["window"]:
        sees &= pos > last[..., None] - case["window"]
    q = s["q"].view(B, q_len, hkv, G, DIM).permute(0, 2, 1, 3, 4).float() / math.sqrt(DIM)

    def rows(kv):
        tile = s["pages"].flatten(-2)[ids, :, kv]                          # [B, width, H, 1152]
        x = _row_values(tile[..., at])                                     # [B, width, H, 16, 128]
        return x.permute(0, 2, 1, 3, 4).flatten(2, 3)

    z = q.flatten(2, 3) @ rows(0).transpose(-1, -2)                        # [B, H, q_len * G, keys]
    z = z.masked_fill(~sees.repeat_interleave(G, 1)[:, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    o = p @ rows(1) / p.sum(-1, keepdim=True)
    o = o.unflatten(2, (q_len, G)).permute(0, 2, 1, 3, 4)
    return o.reshape(B * q_len, hq, DIM).half()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "read":
            return _plain_read(s, case["format"])
        return {"append": _plain_append, "attend": _plain_attend}[case["op"]](s)
    import paged_quantized_kv_append_gb300 as pq
    if case["op"] == "attend":
        return pq.paged_attention(s["q"], s["pages"], s["block_table"], s["seq_lens"], case["q_len"],
                                  "int4_group", None, None, s["out"], max_seq_len=s["max_seq_len"],
                                  window=case["window"])
    fmt = "int4_group"
    if case["op"] == "append":
        pq.kv_append_quant(s["k"], s["v"], s["slots"], fmt, None, None, s["pages"])
    else:
        fmt = case["format"]
    pq.kv_read(s["pages"], s["block_table"], s["first"], s["offsets"], fmt, s["k_scale"],
               s["v_scale"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _table_entries(first, n):
    """Block-table entries that cover the tokens first .. first + n - 1."""
    return int(np.where(n > 0, _pages(first + n) - first // PAGE, 0).sum())


def work(case):
    B, hkv = case["batch"], case["hkv"]
    if case["op"] == "append":
        lens, new, first = _append_lengths(case)
        T, back = int(new.sum()), int((lens + new - first).sum())
        return {"bytes": T * hkv * 2 * (2 * DIM + 72) + T * 8
                + back * hkv * 2 * (72 + 2 * DIM) + 4 * _table_entries(first, lens + new - first)
                + 4 * (2 * B + 1), "flops": 0}
    if case["op"] == "read":
        lens, first, n = _read_lengths(case)
        return {"bytes": int(n.sum()) * hkv * 2 * (ROW_BYTES[case["format"]] + 2 * DIM)
                + 4 * _table_entries(first, n) + 4 * (2 * B + 1), "flops": 0}
    lens = _attend_lengths(case)
    hq, q_len, window = case["hq"], case["q_len"], case["window"]
    last = lens[:, None] - q_len + np.arange(q_len)
    begin = np.maximum(last - window + 1, 0) if window else np.zeros_like(last)
    keys = lens - begin[:, 0]
    return {"bytes": int(keys.sum()) * hkv * 2 * 72 + 2 * B * q_len * hq * DIM * 2
            + 4 * _table_entries(begin[:, 0], keys) + 4 * B,
            "flops": 4 * int((last - begin + 1).sum()) * hq * DIM}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_codes():
    """The four codes of every 16-bit half of a word: [65536, 4]."""
    h = np.arange(65536)
    bits = [(h >> 6) & 15, (h >> 2) & 15, (h >> 10) & 15, (h >> 14) + 4 * (h & 3)]
    return torch.from_numpy(np.stack(bits, -1) - 8.0).cuda()


def _exact_rows(s, fmt, table, kv, h, pos):
    """64-bit rows [len(pos), 128] of K (0) or V (1) of one request's positions."""
    page, r = table[pos // PAGE].long(), pos % PAGE
    tile = s["pages"][page, h, kv]                                   # [n, 16, row]
    at = torch.arange(len(pos), device="cuda")
    if fmt == "int4_group":
        tile = tile.reshape(len(pos), PAGE * 72)
        turn = torch.tensor([[0], [5], [2], [7]], device="cuda")[r // 2 % 4]
        chunk = r[:, None] // 2 * 8 + ((r[:, None] % 2 * 4 + torch.arange(4, device="cuda")) ^ turn)
        halves = tile[:, :1024].contiguous().view(torch.int16).view(len(pos), 64, 8)
        halves = halves[at[:, None], chunk].long() & 0xFFFF          # [n, group, 8 halves]
        code = _exact_codes()[halves].view(len(pos), 4, 4, 2, 4).transpose(-1, -2)
        scale = tile[:, 1024:].contiguous().view(torch.float16).view(len(pos), 4, 16)[at, :, r]
        return (code.reshape(len(pos), 4, GROUP) * scale.double()[..., None]).view(len(pos), DIM)
    x = tile[at, r]
    if fmt == "fp16":
        return x.double()
    if fmt == "fp8_e4m3":
        c = torch.arange(256, device="cuda")
        e, m = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7).double())
        x = torch.where(c < 128, mag, -mag)[x.long()]
    else:
        x = x.long()
        x = torch.where(x < 128, x, x - 256).double()
    if fmt == "int8_row":
        return x * s["row_scales"][page, h, r % 8, kv, r // 8].double()[:, None]
    scale = s["v_scale"] if kv else s["k_scale"]
    return x * scale[h if scale.numel() > 1 else 0].double()


def _exact_quantised(x):
    """What 4 bits hold of rows [..., 128], in 64 bits."""
    x = x.double().unflatten(-1, (4, GROUP))
    s = x.abs().amax(-1, keepdim=True) / 7
    # 8 significant bits (52 - 7 of the mantissa's are dropped), then a multiple of 2^-24
    bits = s.view(torch.int64)
    s = ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) & -(1 << 45)).view(torch.float64)
    s = torch.clamp(torch.round(s * 2.0 ** 24) / 2.0 ** 24, max=MOST_SCALE)
    c = torch.where(s > 0, torch.round(x / s.clamp(min=2.0 ** -24)).clamp(-7, 7), 0 * x)
    return (c * s).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    hkv = case["hkv"]
    if case["op"] == "attend":
        lens = _attend_lengths(case)
        hq, q_len, window = case["hq"], case["q_len"], case["window"]
        G = hq // hkv
        if 4.0 * lens.sum() * q_len * hq * DIM > 2e12 or len(lens) * hkv > 8192:
            return None
        out = torch.empty((len(lens) * q_len, hq, DIM), dtype=torch.float64, device="cuda")
        for i, n in enumerate(lens.tolist()):
            begin = max(0, n - q_len - window + 1) if window else 0
            pos = torch.arange(begin, n, device="cuda")
            last = n - q_len + torch.arange(q_len, device="cuda")[:, None]
            sees = pos <= last
            if window:
                sees &= pos > last - window
            for h in range(hkv):
                x = s["q"][i * q_len:(i + 1) * q_len, h * G:(h + 1) * G].double()
                K = _exact_rows(s, "int4_group", s["block_table"][i], 0, h, pos)
                z = torch.einsum("igd,nd->ign", x, K) / DIM ** 0.5
                z = z.masked_fill(~sees[:, None], -math.inf)
                V = _exact_rows(s, "int4_group", s["block_table"][i], 1, h, pos)
                out[i * q_len:(i + 1) * q_len, h * G:(h + 1) * G] = torch.einsum(
                    "ign,nd->igd", torch.softmax(z, -1), V)
        return out
    if case["op"] == "append":
        lens, new, first = _append_lengths(case)
        n, fmt = lens + new - first, "int4_group"
    else:
        lens, first, n = _read_lengths(case)
        fmt = case["format"]
    if len(n) * hkv > 2048 * 16:
        return None
    out = {x: torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for x in "kv"}
    ends, news = np.cumsum(n), np.cumsum(new) if case["op"] == "append" else None
    for kv, name in enumerate("kv"):
        fresh = _exact_quantised(s[name]) if case["op"] == "append" else None
        for i in range(len(n)):
            a, b = int(ends[i] - n[i]), int(ends[i])
            old = int(lens[i] - first[i]) if fresh is not None else int(n[i])
            pos = int(first[i]) + torch.arange(old, device="cuda")
            if old:
                for h in range(hkv):
                    out[name][a:a + old, h] = _exact_rows(s, fmt, s["block_table"][i], kv, h, pos)
            if fresh is not None:
                out[name][a + old:b] = fresh[int(news[i] - new[i]):int(news[i])]
    return out

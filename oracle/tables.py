"""Oracle: block tables grown and shortened from the requests' lengths.

TEST INFRASTRUCTURE ONLY.  Plain Python, one request, page and token at a time.

A stack holds the free pages (its top is entry free_count - 1).  ``extend``
serves the requests in order; each takes ceil((L + n) / 16) - ceil(L / 16)
pages off the top.  Once a request finds too few pages no later one gets any;
requests that need none are still served.  ``truncate`` pushes the pages that a
shortened request no longer needs.
"""
from __future__ import annotations

import numpy as np

PAGE_SIZE = 16

SLOT_RANGE, SEQ_RANGE, PAGE_RANGE = 1, 2, 16


def _pages(tokens):
    return (tokens + PAGE_SIZE - 1) // PAGE_SIZE


def extend(seq_lens, new_tokens, block_table, free_pages, free_count, num_pages, num_tokens):
    """Returns (seq_lens, free_count, block_table, slots, positions, offsets,
    status bits) after the step."""
    lens = [int(x) for x in seq_lens]
    table = np.array(block_table, copy=True)
    slots = np.full(num_tokens, -1, np.int64)
    positions = np.full(num_tokens, -1, np.int32)
    offsets = []
    cap = table.shape[1] * PAGE_SIZE
    count = int(free_count)
    bits = 0
    if not 0 <= count <= len(free_pages):
        bits |= SLOT_RANGE
        count = min(max(count, 0), len(free_pages))
    out_of_pages = False
    at = 0
    for s, n in enumerate(int(x) for x in new_tokens):
        L = lens[s]
        offsets.append(min(at, num_tokens))
        first = at
        at += max(n, 0)
        if L < 0 or n < 0 or L + n > cap or (n > 0 and at > num_tokens):
            bits |= SEQ_RANGE
            continue
        need = _pages(L + n) - _pages(L)
        if need > 0 and (out_of_pages or need > count):
            out_of_pages = True
            bits |= SLOT_RANGE
            continue
        for j in range(need):
            count -= 1
            table[s, _pages(L) + j] = free_pages[count]
        for i in range(n):
            pos = L + i
            page = int(table[s, pos // PAGE_SIZE])
            if 0 <= page < num_pages:
                slots[first + i] = page * PAGE_SIZE + pos % PAGE_SIZE
                positions[first + i] = pos
            else:
                bits |= PAGE_RANGE
        lens[s] = L + n
    offsets.append(min(at, num_tokens))
    return (np.array(lens, np.int32), count, table, slots, positions,
            np.array(offsets, np.int32), bits)


def truncate(seq_lens, keep_lens, block_table, free_pages, free_count, owned_pages=None):
    """Returns (seq_lens, free_count, free_pages, status bits)."""
    lens = [int(x) for x in seq_lens]
    stack = np.array(free_pages, copy=True)
    cap = block_table.shape[1] * PAGE_SIZE
    count = int(free_count)
    bits = 0
    if not 0 <= count <= len(stack):
        bits |= SLOT_RANGE
        count = min(max(count, 0), len(stack))
    for s, keep in enumerate(int(x) for x in keep_lens):
        L = lens[s]
        if keep < 0 or keep > L or L > cap:
            bits |= SEQ_RANGE
            continue
        owned = 0 if owned_pages is None else max(int(owned_pages[s]), 0)
        for j in range(max(_pages(keep), owned), _pages(L)):
            if count == len(stack):
                bits |= SLOT_RANGE
                break
            stack[count] = block_table[s, j]
            if stack[count] < 0:
                bits |= PAGE_RANGE
            count += 1
        lens[s] = keep
    return np.array(lens, np.int32), count, stack, bits

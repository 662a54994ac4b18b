"""The step operators in plain Python and numpy fp64 (the oracle of include/fi_step.h)."""
from __future__ import annotations

import math

import numpy as np


def rates(rot_dim, theta, scaling="none", s=1.0, L=0, low=1.0, high=4.0):
    """Radians per position of each pair and the amplitude, from the definitions."""
    if scaling == "ntk":
        theta = theta * s ** (rot_dim / (rot_dim - 2))
    out = []
    for i in range(rot_dim // 2):
        f = math.exp(-2.0 * i / rot_dim * math.log(theta))
        if scaling == "linear":
            f = f / s
        elif scaling == "by_parts":
            turns = L * f / (2 * math.pi)
            if turns <= low:
                f = f / s
            elif turns < high:
                g = (turns - low) / (high - low)
                f = g * f + (1 - g) * f / s
        elif scaling == "yarn":
            def d(r):
                return rot_dim * math.log(L / (2 * math.pi * r)) / (2 * math.log(theta))
            a, b = max(0, math.floor(d(high))), min(rot_dim - 1, math.ceil(d(low)))
            g = min(1.0, max(0.0, (i - a) / (b - a if b > a else 1e-3)))
            f = (1 - g) * f + g * f / s
        out.append(f)
    return np.array(out), 0.1 * math.log(s) + 1 if scaling == "yarn" else 1.0


def rotate(x, positions, f, amp, rot_dim, interleaved):
    """x [tokens, heads, dim] fp64, its first rot_dim dims turned pair by pair."""
    y = np.array(x, dtype=np.float64)
    for t, pos in enumerate(positions):
        for i, rate in enumerate(f):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
            # reduced to one turn in integers times the rate, as far as fp64 goes
            c, s = amp * math.cos(pos * rate), amp * math.sin(pos * rate)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def tables(qo_lens, kv_lens, block_table, page_size, free_pages, free_head, max_pages, max_tokens):
    """dict of the arrays of fi_build_step_tables (kv_indices without its unwritten end), or the status."""
    width = len(block_table[0]) if len(block_table) else 0
    pages = [-(-kv // page_size) for kv in kv_lens]
    had = [-(-(kv - q) // page_size) for q, kv in zip(qo_lens, kv_lens)]
    if any(q < 0 or q > kv or kv > width * page_size for q, kv in zip(qo_lens, kv_lens)):
        return 1
    taken = sum(pages) - sum(had)
    if sum(qo_lens) > max_tokens or sum(pages) > max_pages or free_head < 0 or free_head + taken > len(free_pages):
        return 3
    table = [list(r) for r in block_table]
    at = free_head
    ids, positions, slots, qp, kp, last = [], [], [], [0], [0], []
    for b, (q, kv) in enumerate(zip(qo_lens, kv_lens)):
        for p in range(had[b], pages[b]):
            table[b][p] = free_pages[at]
            at += 1
        ids += table[b][:pages[b]]
        for pos in range(kv - q, kv):
            positions.append(pos)
            slots.append(table[b][pos // page_size] * page_size + pos % page_size)
        qp.append(qp[-1] + q)
        kp.append(kp[-1] + pages[b])
        last.append(kv - (pages[b] - 1) * page_size if pages[b] else 0)
    pad = max_tokens - len(positions)
    return dict(qo_indptr=qp, kv_indptr=kp, last_page_len=last, kv_indices=ids, positions=positions + [0] * pad,
                slots=slots + [-1] * pad, table=table, counts=[qp[-1], kp[-1], taken, at, 0, 0, 0, 0])

"""fp64 NumPy oracle of the paged attention path: the page plan, the rotary append and the
attention over the paged cache, each written step by step from its definition in include/gdn.h.
Used by the tests only; it shares no code with the CUDA path."""
import math

import numpy as np


def kv_plan(seq_len, n_pages, table, free_list, free_count, T, page, commit=None, add=None, block=None):
    """One call of gdn_kv_plan, sequence by sequence. Returns a dict of everything it writes, and
    the status bits."""
    B, max_pages = table.shape
    seq, held, table, free = seq_len.copy(), n_pages.copy(), table.copy(), free_list.copy()
    count, status = int(free_count), 0
    kv, ql = np.zeros(B, np.int32), np.zeros(B, np.int32)
    slots = np.full((B, T), -1, np.int64)
    plans = []
    for b in range(B):
        s, h = int(seq[b]), int(held[b])
        if s < 0 or h < 0 or h > max_pages or s > h * page:
            status |= 4
            plans.append((None, h, 0))
            continue
        c = 0 if commit is None else int(commit[b])
        if block is not None:
            c = min(c, int(block[b]))
        if c < 0 or s + c > h * page:
            status |= 1
            c = 0
        a = T if add is None else int(add[b])
        if a < -1 or a > T:
            status |= 4
            a = 0
        length, a = (0, 0) if a == -1 else (s + c, a)
        want = -(-(length + a) // page)
        if want > max_pages:
            status |= 16
            want, a = h, 0
        plans.append((length, want, a))
    for b, (_, want, _) in enumerate(plans):
        for i in range(want, int(held[b])):
            free[count] = table[b, i]
            count += 1
    dry = False
    for b, (length, want, a) in enumerate(plans):
        if length is None:
            continue
        h = int(held[b])
        dry = dry or want - h > count
        if want > h and dry:
            status |= 16
            want, a = h, 0
        for i in range(h, want):
            count -= 1
            table[b, i] = free[count]
        seq[b], held[b], kv[b], ql[b] = length, want, length + a, a
        for t in range(a):
            slots[b, t] = int(table[b, (length + t) // page]) * page + (length + t) % page
    return dict(seq_len=seq, n_pages=held, table=table, free=free, free_count=count, kv_len=kv, q_len=ql, slots=slots,
                status=status)


def pair_axis(i, sections, interleaved):
    """The axis of rotated pair i."""
    A = len(sections)
    if interleaved:
        return i % A if i < A * sections[i % A] else 0
    for a in range(A):
        if i < sections[a]:
            return a
        i -= sections[a]
    raise ValueError("pair outside the sections")


def rotate(x, w, pos, inv_freq, sections, axes_interleaved, pairs_interleaved, eps):
    """Heads x [H, d] of one token at positions pos [axes], normalised and rotated."""
    x = np.asarray(x, np.float64).copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    half = len(inv_freq)
    for i in range(half):
        ang = float(pos[pair_axis(i, sections, axes_interleaved)]) * float(inv_freq[i])
        lo, hi = (2 * i, 2 * i + 1) if pairs_interleaved else (i, i + half)
        a, b = x[:, lo].copy(), x[:, hi].copy()
        x[:, lo] = a * math.cos(ang) - b * math.sin(ang)
        x[:, hi] = a * math.sin(ang) + b * math.cos(ang)
    return x


def rope_append(q, k, v, inv_freq, k_cache, v_cache, slots, positions, sections, axes_interleaved=False,
                pairs_interleaved=False, q_norm=None, k_norm=None, eps=1e-6, q_out=None):
    """fp64 q_out, k_cache, v_cache after the call (positions [axes, B, T])."""
    B, T = slots.shape
    page = k_cache.shape[1]
    q_out = np.zeros(q.shape) if q_out is None else np.asarray(q_out, np.float64).copy()
    kc, vc = np.asarray(k_cache, np.float64).copy(), np.asarray(v_cache, np.float64).copy()
    for b in range(B):
        for t in range(T):
            s = int(slots[b, t])
            if not 0 <= s < k_cache.shape[0] * page:
                continue
            at = (positions[:, b, t], inv_freq, sections, axes_interleaved, pairs_interleaved, eps)
            q_out[b, t] = rotate(q[b, t], q_norm, *at)
            kc[s // page, s % page] = rotate(k[b, t], k_norm, *at)
            vc[s // page, s % page] = v[b, t]
    return q_out, kc, vc


def paged_attention(q, k_cache, v_cache, table, kv_len, q_len=None, scale=None, window=0):
    """fp64 (o, lse, seen): seen[b, t] says which rows the call writes."""
    B, T, Hq, d = q.shape
    pages, page, Hk, _ = k_cache.shape
    scale = d ** -0.5 if scale is None else scale
    o, lse, written = np.zeros(q.shape), np.full((B, T, Hq), -np.inf), np.zeros((B, T), bool)
    for b in range(B):
        n, m = int(kv_len[b]), T if q_len is None else int(q_len[b])
        if not (0 <= n <= table.shape[1] * page and 0 <= m <= T):
            continue
        for t in range(m):
            written[b, t] = True
            p = n - m + t
            cells = [(int(table[b, j // page]), j % page) for j in range(max(0, p - window + 1) if window else 0, p + 1)]
            cells = [c for c in cells if 0 <= c[0] < pages]
            if not cells:
                continue
            ids, off = np.array(cells).T
            for h in range(Hq):
                g = h // (Hq // Hk)
                s = scale * (np.asarray(k_cache[ids, off, g], np.float64) @ np.asarray(q[b, t, h], np.float64))
                top = s.max()
                w = np.exp(s - top)
                o[b, t, h] = w @ np.asarray(v_cache[ids, off, g], np.float64) / w.sum()
                lse[b, t, h] = top + math.log(w.sum())
    return o, lse, written

"""The paged attention path beside the Gated DeltaNet mixer: what is measured, and its plain forms.

A hybrid stack runs attention layers between its Gated DeltaNet layers, and a speculative
round takes the same block of tokens through both. Three operators carry such an attention
layer from the accept counts of one verify block to the outputs of the next:

  plan     block tables and slot maps from the requests' lengths: the previous block's accept
           counts are committed, pages are handed back and out, every new token gets its slot;
  append   the block's queries and keys normalised and rotated (positions with one to four
           axes), keys and values written into their slots of the paged cache;
  attn     attention of the block's rows (one new token, or a verify block) over the paged cache.

Layouts are those of the library: q [B, T, H_q, d], k and v [B, T, H_kv, d], caches
[pages, page, H_kv, d] (any order in memory with the last axis contiguous), block tables
[B, max_pages], one slot (page * page size + offset) per token and -1 where there is none.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NORM_EPS = 1e-6
ROPE_BASE = 1e6


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # One sequence's verify block (7 drafts and the anchor) at 32K context: pure latency.
        dict(name="plan_one", op="plan", B=1, T=8, page=64, max_len=32768, prompt=False),
        # A serving batch between two verify blocks; some requests end and give their pages back.
        dict(name="plan_serve", op="plan", B=256, T=8, page=16, max_len=8192, prompt=False),
        # Admission of a batch of ragged prompts: every slot of every prompt token.
        dict(name="plan_prompts", op="plan", B=32, T=8192, page=64, max_len=16384, prompt=True),
        # One sequence's verify block, partial rotation, head norms, text positions.
        dict(name="append_one", op="append", B=1, T=8, H_q=24, H_kv=4, d=256, rot=64, axes=1, axes_interleaved=False,
             pairs_interleaved=False, norm=True, dtype="bf16", page=64, text=True, ragged=False),
        # Two long prompts with images: time, height and width positions, ragged ends.
        dict(name="append_image_prompts", op="append", B=2, T=16384, H_q=32, H_kv=8, d=128, rot=128, axes=3,
             axes_interleaved=True, pairs_interleaved=False, norm=True, dtype="bf16", page=64, text=False, ragged=True),
        # A batch of verify blocks in 32 bits, two axes, neighbouring pairs, no norm, odd pages.
        dict(name="append_f32", op="append", B=64, T=8, H_q=16, H_kv=4, d=64, rot=64, axes=2, axes_interleaved=False,
             pairs_interleaved=True, norm=False, dtype="f32", page=24, text=False, ragged=True),
        # One new token of one short chat: latency.
        dict(name="attn_one_1k", op="attn", B=1, T=1, H_q=32, H_kv=8, d=128, dtype="bf16", page=16, min_len=1023,
             max_len=1023, window=0, ragged=False, heads_first=False),
        # One sequence's verify block at 32K context (the single-sequence round's attention layer).
        dict(name="attn_one_32k", op="attn", B=1, T=8, H_q=24, H_kv=4, d=256, dtype="bf16", page=64, min_len=32768,
             max_len=32768, window=0, ragged=False, heads_first=False),
        # Plain decoding of a batch with lengths of every size.
        dict(name="attn_decode", op="attn", B=64, T=1, H_q=32, H_kv=8, d=128, dtype="bf16", page=16, min_len=500,
             max_len=16384, window=0, ragged=False, heads_first=False),
        # A batch of verify blocks, some shorter than the block, pages stored head by head.
        dict(name="attn_verify", op="attn", B=32, T=8, H_q=24, H_kv=4, d=256, dtype="bf16", page=64, min_len=100,
             max_len=8192, window=0, ragged=True, heads_first=True),
        # One head for each key head (no sharing), many short requests.
        dict(name="attn_unshared", op="attn", B=128, T=1, H_q=16, H_kv=16, d=128, dtype="bf16", page=32, min_len=1,
             max_len=2048, window=0, ragged=False, heads_first=False),
        # 32-bit cache, sliding window, odd pages, short blocks; the shortest requests have fewer
        # positions than rows.
        dict(name="attn_f32_window", op="attn", B=16, T=4, H_q=16, H_kv=4, d=64, dtype="f32", page=24, min_len=1,
             max_len=4096, window=1000, ragged=True, heads_first=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    page = rng.choice([16, 24, 32, 64, 128])
    if op == "plan":
        if rng.random() < 0.3:
            T = _log_int(rng, 17, 8192)
            return dict(op=op, B=_log_int(rng, 1, max(1, min(64, 262144 // T))), T=T, page=page, max_len=16384, prompt=True)
        return dict(op=op, B=_log_int(rng, 1, 512), T=rng.randint(1, 16), page=page, max_len=_log_int(rng, 200, 8192),
                    prompt=False)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 256])
    H_kv = rng.choice([1, 2, 4, 8])
    H_q = H_kv * rng.choice([1, 2, 3, 4, 6, 8])
    if op == "append":
        axes = rng.randint(1, 4)
        rot = rng.choice([r for r in (32, 64, 128, 256) if r <= d])
        T = _log_int(rng, 1, 16384)
        most = 24576 * 48 * 128 // ((H_q + 2 * H_kv) * d * (2 if dtype == "f32" else 1))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(256, most // T))), T=min(T, most), H_q=H_q, H_kv=H_kv, d=d, rot=rot,
                    axes=axes, axes_interleaved=rng.random() < 0.5, pairs_interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, dtype=dtype, page=page, text=axes == 1 and rng.random() < 0.5,
                    ragged=rng.random() < 0.5)
    max_len = _log_int(rng, 1, 32768)
    # at most the cached elements and the scores of the largest listed case
    most = 32 * 16384 * 8 * 128 // (max_len * H_kv * d * (2 if dtype == "f32" else 1))
    B = _log_int(rng, 1, max(1, min(128, most)))
    T = rng.choice([1, 1, 1, rng.randint(2, 16), 8])
    while T > 1 and B * T * H_q * max_len > 64 * 32 * 16384:
        T -= 1
    return dict(op=op, B=B, T=T, H_q=H_q, H_kv=H_kv, d=d, dtype=dtype, page=page, min_len=max(1, max_len // rng.choice([1, 4, 100])),
                max_len=max_len, window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), ragged=T > 1 and rng.random() < 0.5,
                heads_first=rng.random() < 0.3)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randint(g, lo, hi, n):
    """n whole numbers in lo..hi (both included), int32."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _spread(lo, hi, n):
    """n lengths from hi down to lo, evenly apart (one: hi)."""
    return [hi] if n == 1 else [hi - (hi - lo) * i // (n - 1) for i in range(n)]


def _shuffled(g, values):
    v = torch.tensor(values, dtype=torch.int32, device=DEV)
    return v[torch.randperm(len(values), generator=g, device=DEV)]


def _max_pages(c):
    return -(-(c["max_len"] + c["T"]) // c["page"])


def _prepare_plan(c, g):
    B, T, P = c["B"], c["T"], c["page"]
    width = _max_pages(c)
    if c["prompt"]:
        seq_len = torch.zeros(B, dtype=torch.int32, device=DEV)
        held_to = seq_len
        commit = None
        add = _shuffled(g, _spread(1, T, B))
    else:
        # the previous block held T tokens behind seq_len; commit of them were accepted
        seq_len = _randint(g, 0, max(0, c["max_len"] - T), B)
        held_to = seq_len + T
        commit = _randint(g, 0, T, B)
        add = torch.full((B,), T, dtype=torch.int32, device=DEV)
        pick = torch.randperm(B, generator=g, device=DEV)
        add[pick[: B // 16]] = -1                       # requests that have ended
        add[pick[B // 16: B // 8]] = T // 2             # requests near their end
    n_pages = (held_to + P - 1) // P
    n = B * width                                       # the pool: enough for every sequence at its longest
    ids = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(n_pages, 0) - n_pages)[:, None] + col
    table = torch.where(col < n_pages[:, None], ids[at.clamp(max=n - 1)], torch.full_like(at, -1, dtype=torch.int32))
    used = int(n_pages.sum())
    free = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    free[: n - used] = ids[used:]
    e = lambda *s, dtype=torch.int32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    return dict(c=c, seq_len=seq_len, n_pages=n_pages.to(torch.int32), commit=commit, add=add, table=table.contiguous(), free=free,
                free_count=torch.tensor([n - used], dtype=torch.int32, device=DEV), seq_len_out=e(B), n_pages_out=e(B),
                free_count_out=e(1), kv_len=e(B), q_len=e(B), slots=e(B, T, dtype=torch.int64))


def _sections(c):
    """Rotated pairs of each axis: the later axes an equal share, the first the rest."""
    half = c["rot"] // 2
    share = half // (c["axes"] + 1) if c["axes"] > 1 else 0
    return [half - share * (c["axes"] - 1)] + [share] * (c["axes"] - 1)


def _append_rows(c):
    """Tokens of each sequence; in a large ragged batch some have none."""
    lo = c["T"] if not c["ragged"] else 0 if c["B"] > 8 else max(1, c["T"] // 2)
    return _spread(lo, c["T"], c["B"])


def _prepare_append(c, g):
    B, T, Hq, Hk, d, P = c["B"], c["T"], c["H_q"], c["H_kv"], c["d"], c["page"]
    dt = DTYPES[c["dtype"]]
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=g, device=DEV, dtype=torch.float32).to(dt)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
    base = _randint(g, 0, 32768 - 1, B)
    rows = _shuffled(g, _append_rows(c))
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    off = (base % P)[:, None] + t                            # within the sequence's pages touched here
    per = (T + P - 1) // P + 1
    pages = torch.randperm(B * per, generator=g, device=DEV).view(B, per)
    slots = torch.gather(pages, 1, (off // P).long()) * P + off % P
    slots = torch.where(t < rows[:, None], slots, torch.full_like(slots, -1))
    positions = None
    if not c["text"]:
        # a patch grid of 32 x 24 in every 768 tokens: axis 0 its frame, axes 1 and 2 row and column
        step = [t // 768, (t % 768) // 32, t % 32, t // 2][: c["axes"]]
        positions = torch.stack([base[:, None] + s for s in step]).contiguous()
    inv_freq = (ROPE_BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).to(torch.float32).to(DEV)
    w = lambda: (0.5 + torch.rand(d, generator=g, device=DEV)) if c["norm"] else None  # noqa: E731
    # one page more than the pool: the plain form sends the rows without a slot there
    cache = lambda: torch.zeros(B * per + 1, P, Hk, d, dtype=dt, device=DEV)  # noqa: E731
    return dict(c=c, q=q, k=k, v=v, slots=slots.contiguous(), positions=positions, kv_len=base + rows, q_len=rows, inv_freq=inv_freq,
                q_norm=w(), k_norm=w(), k_pool=cache(), v_pool=cache(), q_out=torch.zeros(B, T, Hq, d, dtype=dt, device=DEV))


def _lens(c):
    return _spread(c["min_len"], c["max_len"], c["B"])


def _rows(c):
    return [1 + (i * 5) % c["T"] if c["ragged"] else c["T"] for i in range(c["B"])]


def _prepare_attn(c, g):
    B, T, Hq, Hk, d, P = c["B"], c["T"], c["H_q"], c["H_kv"], c["d"], c["page"]
    dt = DTYPES[c["dtype"]]
    order = torch.randperm(B, generator=g, device=DEV)
    kv_len = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[order]
    q_len = torch.tensor(_rows(c), dtype=torch.int32, device=DEV)[order]
    n_pages = (kv_len + P - 1) // P
    width = -(-c["max_len"] // P)
    n = sum(-(-m // P) for m in _lens(c)) + 3
    ids = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    at = (torch.cumsum(n_pages, 0) - n_pages)[:, None] + col
    table = torch.where(col < n_pages[:, None], ids[at.clamp(max=n - 1)], torch.full_like(at, -1, dtype=torch.int32))
    shape = (n, Hk, P, d) if c["heads_first"] else (n, P, Hk, d)
    cache = [torch.randn(shape, generator=g, device=DEV, dtype=dt) for _ in range(2)]
    if c["heads_first"]:
        cache = [x.transpose(1, 2) for x in cache]
    q = torch.randn(B, T, Hq, d, generator=g, device=DEV, dtype=torch.float32).to(dt)
    s = dict(c=c, q=q, k_cache=cache[0], v_cache=cache[1], table=table.contiguous(), kv_len=kv_len, q_len=q_len,
             o=torch.zeros_like(q), lse=torch.zeros(B, T, Hq, dtype=torch.float32, device=DEV))
    if own:   # the workspace that a user's program keeps for the call
        from gated_deltanet_mixer_verify_b200 import gdn
        s["workspace"] = torch.empty(gdn.paged_attention_workspace_bytes(B, T, Hq, Hk, d, dt), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn}[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------------------ plain forms

def _plain_plan(s):
    c, T, P = s["c"], s["c"]["T"], s["c"]["page"]
    table, free = s["table"], s["free"]
    width, n = table.shape[1], free.numel()
    held = s["n_pages"].long()
    length = s["seq_len"].long() + (s["commit"].long() if s["commit"] is not None else 0)
    add = s["add"].long()
    ended = add < 0
    want = torch.where(ended, 0, (length + add + P - 1) // P)
    # pages handed back, in the order of the sequences, onto the top of the free list
    back = (held - want).clamp(min=0)
    have = s["free_count"].long() + back.sum()
    col = torch.arange(width, device=DEV)[None, :]
    at = s["free_count"].long() + (torch.cumsum(back, 0) - back)[:, None] + (col - want[:, None])
    gives = (col >= want[:, None]) & (col < held[:, None])
    longer = torch.cat([free, free.new_zeros(1)])
    longer.scatter_(0, torch.where(gives, at, n).view(-1), table.reshape(-1))
    free.copy_(longer[:n])
    # pages handed out, in the order of the sequences, from the top
    fits = want <= width
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (upto <= have))
    now = torch.where(granted, want, held)
    k = (upto - need)[:, None] + (col - held[:, None])
    takes = (col >= held[:, None]) & (col < now[:, None])
    table.copy_(torch.where(takes, free[(have - 1 - k).clamp(0, n - 1)], table))
    length = torch.where(ended, 0, length)
    q_len = torch.where(granted & ~ended, add, 0)
    t = torch.arange(T, device=DEV)[None, :]
    pos = length[:, None] + t
    page = torch.gather(table, 1, (pos // P).clamp(max=width - 1)).long()
    slots = torch.where(t < q_len[:, None], page * P + pos % P, -1)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(seq_len=i32(length), n_pages=i32(now), free_count=i32(have - (need * granted).sum()), kv_len=i32(length + q_len),
                q_len=i32(q_len), slots=slots, table=table, free=free)


def _pair_axes(c):
    """The axis of each rotated pair: blocks one after the other, or the axes in turn while their
    sections last and the first axis in the rest."""
    sec, half, A = _sections(c), c["rot"] // 2, c["axes"]
    i = torch.arange(half, device=DEV)
    if not c["axes_interleaved"]:
        return torch.bucketize(i, torch.cumsum(torch.tensor(sec, device=DEV), 0), right=True)
    return torch.where(i < A * torch.tensor(sec, device=DEV)[i % A], i % A, 0)


def _plain_rotate(c, x, w, cos, sin):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS) * w
    r, half = c["rot"], c["rot"] // 2
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["pairs_interleaved"] else (x[..., :half], x[..., half:r])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if c["pairs_interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(s):
    c, T = s["c"], s["c"]["T"]
    t = torch.arange(T, device=DEV)
    if s["positions"] is None:
        pos = ((s["kv_len"] - s["q_len"])[:, None] + t)[None]
    else:
        pos = s["positions"]
    # angles of far positions keep nothing in 32 bits
    angle = pos.double()[_pair_axes(c)].permute(1, 2, 0) * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, :, None, :] for f in (torch.cos, torch.sin))
    dt = DTYPES[c["dtype"]]
    there = s["slots"] >= 0
    s["q_out"].copy_(torch.where(there[:, :, None, None], _plain_rotate(c, s["q"], s["q_norm"], cos, sin).to(dt), s["q_out"]))
    pool = s["k_pool"]
    spare = (pool.shape[0] - 1) * pool.shape[1]
    to = torch.where(there, s["slots"], spare).view(-1)
    pool.view(-1, *pool.shape[2:])[to] = _plain_rotate(c, s["k"], s["k_norm"], cos, sin).to(dt).flatten(0, 1)
    s["v_pool"].view(-1, *pool.shape[2:])[to] = s["v"].flatten(0, 1)
    return dict(q=s["q_out"], k_cache=pool[:-1], v_cache=s["v_pool"][:-1])


def _plain_attn(s):
    c, B, T, Hq, Hk, d = s["c"], *(s["c"][n] for n in ("B", "T", "H_q", "H_kv", "d"))
    G = Hq // Hk
    at = s["table"].clamp(min=0)
    k = s["k_cache"][at].flatten(1, 2).permute(0, 2, 3, 1).float()                       # [B, H_kv, d, S]
    j = torch.arange(k.shape[-1], device=DEV)
    written = j < s["kv_len"][:, None]
    t = torch.arange(T, device=DEV)
    p = (s["kv_len"] - s["q_len"])[:, None] + t                                          # [B, T]
    seen = (j <= p[..., None]) & written[:, None, :]
    if c["window"]:
        seen &= j > (p - c["window"])[..., None]
    seen = seen[:, None, :, None, :]                                                     # [B, 1, T, 1, S]
    q = s["q"].float().view(B, T, Hk, G, d).permute(0, 2, 1, 3, 4)
    x = (q.reshape(B, Hk, T * G, d) @ k).view(B, Hk, T, G, -1) * d ** -0.5
    del k
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = s["v_cache"][at].flatten(1, 2).transpose(1, 2).float()
    v = torch.where(written[:, None, :, None], v, 0.0)
    o = (x.view(B, Hk, T * G, -1) @ v).view(B, Hk, T, G, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d).to(s["o"].dtype)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hq)
    there = t < s["q_len"][:, None]
    s["o"].copy_(torch.where(there[..., None, None], o, s["o"]))
    s["lse"].copy_(torch.where(there[..., None], lse, s["lse"]))
    return dict(o=s["o"], lse=s["lse"])


# ------------------------------------------------------------------------------ the framework's calls

def _own_plan(s):
    from gated_deltanet_mixer_verify_b200 import gdn
    gdn.kv_plan(s["seq_len"], s["n_pages"], s["table"], s["free"], s["free_count"], s["c"]["T"], s["c"]["page"],
                commit_len=s["commit"], add_len=s["add"], seq_len_out=s["seq_len_out"], n_pages_out=s["n_pages_out"],
                free_count_out=s["free_count_out"], kv_len=s["kv_len"], q_len=s["q_len"], slot_map=s["slots"])
    return dict(seq_len=s["seq_len_out"], n_pages=s["n_pages_out"], free_count=s["free_count_out"], kv_len=s["kv_len"],
                q_len=s["q_len"], slots=s["slots"], table=s["table"], free=s["free"])


def _own_append(s):
    from gated_deltanet_mixer_verify_b200 import gdn
    c = s["c"]
    k_cache, v_cache = s["k_pool"][:-1], s["v_pool"][:-1]
    gdn.rope_append(s["q"], s["k"], s["v"], s["inv_freq"], k_cache, v_cache, s["slots"], positions=s["positions"], kv_len=s["kv_len"],
                    q_len=s["q_len"], sections=_sections(c), axes_interleaved=c["axes_interleaved"],
                    pairs_interleaved=c["pairs_interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=NORM_EPS,
                    q_out=s["q_out"])
    return dict(q=s["q_out"], k_cache=k_cache, v_cache=v_cache)


def _own_attn(s):
    from gated_deltanet_mixer_verify_b200 import gdn
    gdn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], q_len=s["q_len"], window=s["c"]["window"],
                        o=s["o"], lse=s["lse"], workspace=s["workspace"])
    return dict(o=s["o"], lse=s["lse"])


def run(state):
    op = state["c"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "attn": _own_attn}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    B, T = c["B"], c["T"]
    if c["op"] == "plan":
        # four counts in and four out for each sequence, one slot for each row, the table entries
        # behind the slots and the pages that change hands (read and written)
        tokens = sum(_spread(1, T, B)) if c["prompt"] else B * T
        pages = tokens // c["page"] + B
        return {"bytes": 32 * B + 8 * B * T + 4 * pages + (8 * pages if c["prompt"] else 0), "flops": 8 * B + 4 * B * T}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        rows = sum(_append_rows(c))
        width = (c["H_q"] + 2 * c["H_kv"]) * c["d"]
        turned = (c["H_q"] + c["H_kv"]) * c["d"]
        return {"bytes": 2 * rows * width * es + 8 * B * T + (0 if c["text"] else 4 * rows * c["axes"]),
                "flops": rows * (turned * 3 + (turned * 4 if c["norm"] else 0) + 20 * c["rot"])}
    read, pairs = 0, 0
    for n, m in zip(_lens(c), _rows(c)):
        first = max(0, n - m - c["window"] + 1) if c["window"] else 0
        read += n - first
        for i in range(m):
            p = n - m + i
            pairs += max(0, min(p + 1, c["window"]) if c["window"] else p + 1)
    rows = sum(_rows(c)) * c["H_q"]
    return {"bytes": 2 * read * c["H_kv"] * c["d"] * es + 2 * rows * c["d"] * es + 4 * rows, "flops": 4 * pairs * c["H_q"] * c["d"]}


# ------------------------------------------------------------------------------ the definitions, in 64 bits

def _exact_append(s):
    """Each pair as one complex number, turned by e^(i position frequency)."""
    c = s["c"]
    B, T, d, half = c["B"], c["T"], c["d"], c["rot"] // 2
    sec, A = _sections(c), c["axes"]
    ends = [sum(sec[: a + 1]) for a in range(A)]
    axis = []
    for i in range(half):
        if c["axes_interleaved"]:
            axis.append(i % A if i < A * sec[i % A] else 0)
        else:
            axis.append(next(a for a in range(A) if i < ends[a]))
    if s["positions"] is None:
        start = (s["kv_len"].double() - s["q_len"].double()).view(B, 1)
        at = [(start + torch.arange(T, device=DEV, dtype=torch.float64))] * A
    else:
        at = list(s["positions"].double())
    freq = s["inv_freq"].double()

    def turn(x, w, rows):
        x = x[rows].double()                                # [n, heads, d]
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt() * w.double()
        out = x.clone()
        for i in range(half):
            lo, hi = (2 * i, 2 * i + 1) if c["pairs_interleaved"] else (i, i + half)
            angle = (at[axis[i]][rows] * freq[i])[:, None]
            z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(angle), angle)
            out[..., lo], out[..., hi] = z.real, z.imag
        return out

    rows = s["slots"] >= 0
    where = s["slots"][rows]
    q = s["q_out"].double()
    q[rows] = turn(s["q"], s["q_norm"], rows)
    k, v = (s[n][:-1].double() for n in ("k_pool", "v_pool"))
    k.view(-1, *k.shape[2:])[where] = turn(s["k"], s["k_norm"], rows)
    v.view(-1, *v.shape[2:])[where] = s["v"][rows].double()
    return dict(q=q, k_cache=k, v_cache=v)


def _exact_attn(s):
    """Sequence by sequence and row by row of the block, over exactly the positions that the row sees."""
    c, d = s["c"], s["c"]["d"]
    G, P = c["H_q"] // c["H_kv"], c["page"]
    o, lse = s["o"].double(), s["lse"].double()
    table = s["table"].cpu()
    for b, (n, m) in enumerate(zip(s["kv_len"].tolist(), s["q_len"].tolist())):
        ids = table[b, : -(-n // P)].long().to(DEV)
        k, v = (x[ids].reshape(-1, c["H_kv"], d)[:n].double() for x in (s["k_cache"], s["v_cache"]))
        for t in range(m):
            last = n - m + t
            first = max(0, last - c["window"] + 1) if c["window"] else 0
            if last < 0:
                o[b, t], lse[b, t] = 0.0, -math.inf
                continue
            kk, vv = k[first: last + 1], v[first: last + 1]
            x = torch.einsum("hgd,nhd->hgn", s["q"][b, t].double().view(-1, G, d), kk) / math.sqrt(d)
            lse[b, t] = torch.logsumexp(x, -1).view(-1)
            o[b, t] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), vv).reshape(-1, d)
    return dict(o=o, lse=lse)


def exact(case, seed):
    if case["op"] == "plan":
        return None                                        # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)

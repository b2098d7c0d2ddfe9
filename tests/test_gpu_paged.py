"""The paged attention path on the GPU against the fp64 oracle: the page plan, the rotary append
and the attention over the paged cache, each at the sizes, layouts and masks where it can go wrong,
then the three together as a verify loop runs them.

Tolerances, per element, derived before the first run (a rounding is half a step of its type:
bf16 2^-8, fp32 2^-24, relative):
  append, fp32: the head norm's sum of d <= 256 squares runs through 8 + 5 additions (13 2^-24, half
    of it in the root), the angle is off by 2e-7 at most (2^-24 of half a turn), cosine and sine by
    2 2^-24, the products and the sum by 3 2^-24 more: below 1.5e-6 of the larger element of the
    pair; 2e-6 of the head's largest element is allowed. bf16 adds half a step, 2^-8 of the result.
  attention: a score is a sum of d products, each within 2^-21 of exact for split fp32 operands
    (bf16 products are exact), added in fp32; with |q.k| scale summed over its terms at most A = 12
    for these inputs (d = 256 terms of mean 0.64 / 16) that is 12 (2^-21 + 8 2^-24) = 1.2e-5. A weight is
    off by that, by 2^-22 in its exponential and by 2^-17 as two bf16 terms (fp32: 2^-21), the
    sum of the weights likewise; so o is off by at most 2 (1.2e-5 + 2^-22 + 2^-17) max|v| = 4e-5 max|v|
    for bf16, 3e-5 max|v| for fp32, and the logarithm of the sum by 1.2e-5 + 2^-23 |lse|, allowed 2e-5 + 2^-22 |lse|.
    An o stored as bf16 adds 2^-8 of itself."""
import numpy as np
import pytest
import torch

from gdn_helpers import launched_kernels
from oracle import paged

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn(cuda_device):
    from gated_deltanet_mixer_verify_b200 import build, gdn as g
    build.build()
    return g


def _f64(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ the page plan

def _plan_state(rng, B, T, page, width, spare, ended=0.1):
    """A state between two blocks: lengths, pages held for a block behind them, a shuffled pool."""
    seq = rng.integers(0, max(1, width * page - 2 * T), B).astype(np.int32)
    held = -(-(seq + T) // page)
    n = int(held.sum()) + spare
    ids = rng.permutation(n).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : held[b]] = ids[at: at + held[b]]
        at += held[b]
    free = np.full(n, -1, np.int32)
    free[: n - at] = ids[at:]
    add = rng.integers(0, T + 1, B).astype(np.int32)
    add[rng.random(B) < ended] = -1
    return dict(seq=seq, held=held.astype(np.int32), table=table, free=free, count=n - at,
                commit=rng.integers(0, T + 1, B).astype(np.int32), add=add)


def _run_plan(gdn, s, T, page, in_place, commit=True, add=True, block=None):
    st = _status()
    d = {k: _i32(v) for k, v in s.items() if k != "count"}
    count = _i32([s["count"]])
    out = {} if in_place else dict(seq_len_out=torch.full_like(d["seq"], 77), n_pages_out=torch.full_like(d["held"], 77),
                                   free_count_out=torch.full_like(count, 77))
    rows = None if block is None else _i32(block)
    kv, ql, slots = gdn.kv_plan(d["seq"], d["held"], d["table"], d["free"], count, T, page, commit_len=d["commit"] if commit else None,
                                add_len=d["add"] if add else None, block_len=rows, q_len=rows if in_place else None, status_word=st,
                                **out)
    torch.cuda.synchronize()
    if not in_place:
        assert np.array_equal(d["seq"].cpu(), s["seq"]) and np.array_equal(d["held"].cpu(), s["held"]) and int(count) == s["count"]
    got = dict(seq_len=out.get("seq_len_out", d["seq"]), n_pages=out.get("n_pages_out", d["held"]), table=d["table"], free=d["free"],
               free_count=out.get("free_count_out", count)[0], kv_len=kv, q_len=ql, slots=slots)
    ref = paged.kv_plan(s["seq"], s["held"], s["table"], s["free"], s["count"], T, page, s["commit"] if commit else None,
                        s["add"] if add else None, block)
    assert int(st) == ref["status"]
    for k, v in got.items():
        if k == "free":       # behind the last free page the list is scratch
            v, ref[k] = v[: ref["free_count"]], ref[k][: ref["free_count"]]
        assert np.array_equal(v.cpu().numpy(), ref[k]), k
    return ref


@pytest.mark.parametrize("B,T,page,width", [(1, 1, 1, 4), (1, 8, 64, 520), (3, 16, 7, 40), (33, 8, 16, 64), (512, 5, 16, 9),
                                            (513, 8, 3, 30), (1300, 2, 24, 5), (2, 20000, 64, 700), (40, 700, 5, 300), (5, 300, 512, 2)])
def test_plan(gdn, B, T, page, width):
    rng = np.random.default_rng([B, T, page])
    for in_place in (True, False):
        _run_plan(gdn, _plan_state(rng, B, T, page, width, spare=B * (T // page + 2)), T, page, in_place)
        s = _plan_state(rng, B, T, page, width, spare=B * (T // page + 2))
        _run_plan(gdn, s, T, page, in_place, block=rng.integers(0, T + 1, B).astype(np.int32))
    _run_plan(gdn, _plan_state(rng, B, T, page, width, spare=B * (T // page + 2)), T, page, True, commit=False, add=False)


@pytest.mark.parametrize("B", [9, 600])
def test_plan_pool_runs_dry(gdn, B):
    # few free pages, and some sequences return theirs in the same call; then all of them grow by
    # four pages with room for some of them only
    rng = np.random.default_rng(B)
    for spare in (0, 3, B // 3):
        _run_plan(gdn, _plan_state(rng, B, 16, 4, 64, spare, ended=0.05), 16, 4, True)
        s = _plan_state(rng, B, 16, 4, 64, spare)
        s["commit"][:] = s["add"][:] = 16
        ref = _run_plan(gdn, s, 16, 4, True)
        assert ref["status"] == 16 and ref["free_count"] < 4 and (ref["q_len"] > 0).sum() == spare // 4


def test_plan_counts_that_cannot_be(gdn):
    rng = np.random.default_rng(8)
    s = _plan_state(rng, 12, 8, 4, 10, 40)
    s["seq"][0], s["held"][1], s["held"][2] = -1, -3, 11
    s["seq"][3] = s["held"][3] * 4 + 1
    s["commit"][4], s["commit"][5] = -2, 1000
    s["add"][6], s["add"][7] = -2, 9
    s["seq"][8], s["held"][8], s["commit"][8], s["add"][8] = 36, 10, 0, 8        # would need an eleventh page
    ref = _run_plan(gdn, s, 8, 4, False)
    assert ref["status"] == 1 | 4 | 16


def test_plan_free_count_that_cannot_be(gdn):
    # a count outside the pool counts as an empty or a full list
    for count, want in ((-3, 0), (99, 7)):
        st, c = _status(), _i32([count])
        gdn.kv_plan(_i32([0]), _i32([0]), _i32([[-1] * 4]), _i32(range(7)), c, 2, 16, add_len=_i32([0]), status_word=st)
        assert int(st) == 4 and int(c) == want


@pytest.mark.parametrize("T", [5, 9000])
@pytest.mark.parametrize("bad", [-1, -3, 40, (1 << 31) - 1, -(1 << 31)])
def test_plan_pages_that_cannot_be(gdn, bad, T):
    # ids outside the pool, in a page that is held and among the free: their tokens have no slot (a negative id would
    # make a negative slot, which means none, without a word), all others theirs
    page, pages = 16, 40
    width = -(-(T + 20) // page) + 1
    table = np.full((2, width), -1, np.int32)
    table[0, 0], table[1, 0] = bad, 7
    free = np.arange(8, 40, dtype=np.int32)
    free[31] = bad                                   # the first to be handed out
    for slots_in in (4, 12):
        st = _status()
        add = min(T, 20)
        tb, fr = _i32(table), _i32(np.concatenate([free, np.zeros(8, np.int32)]))
        kv, ql, slots = gdn.kv_plan(_i32([slots_in, slots_in]), _i32([1, 1]), tb, fr, _i32([32]), T, page, add_len=_i32([add, add]), status_word=st)
        tb, slots = tb.cpu().numpy(), slots.cpu().numpy()
        assert int(st) == 8 and kv.tolist() == [slots_in + add] * 2 and ql.tolist() == [add] * 2
        for b in range(2):
            for t in range(T):
                pos = slots_in + t
                ok = t < add and 0 <= tb[b, pos // page] < pages
                assert slots[b, t] == (int(tb[b, pos // page]) * page + pos % page if ok else -1), (b, t)


@pytest.mark.parametrize("B", [2, 1500])
def test_plan_more_pages_back_than_there_are(gdn, B):
    # pages returned onto a list that is full already: they are dropped, and it is said
    count, st = _i32([6]), _status()
    free = _i32([3, 1, 4, 0, 5, 2, -9])
    held = np.zeros(B, np.int32)
    held[-1] = 2
    table = np.full((B, 4), -1, np.int32)
    table[-1, :2] = 6, 3
    gdn.kv_plan(_i32([0] * B), _i32(held), _i32(table), free, count, 2, 16, add_len=_i32([-1] * B), status_word=st)
    assert int(st) == 4 and int(count) == 7 and free.tolist() == [3, 1, 4, 0, 5, 2, 6]


def test_plan_empty_batch_and_zero_adds(gdn):
    e = lambda *sh, dt=torch.int32: torch.empty(sh, dtype=dt, device="cuda")  # noqa: E731
    count = _i32([5])
    gdn.kv_plan(e(0), e(0), e(0, 4), _i32(range(7)), count, 3, 16)
    assert int(count) == 5
    s = _plan_state(np.random.default_rng(1), 4, 3, 16, 8, 9)
    s["add"][:] = 0
    assert (_run_plan(gdn, s, 3, 16, True)["slots"] == -1).all()


# ------------------------------------------------------------------------------ the rotary append

def _append(gdn, B, T, Hq, Hk, d, rot, sections, dt, page=16, ai=False, pi=False, norm=True, fused=True, in_place=False,
            text=False, far=1 << 20, layout="tokens", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if fused:
        qkv = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=g, device="cuda").to(dt)
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
    else:
        q, k, v = (torch.randn(B, T, h, d, generator=g, device="cuda").to(dt) for h in (Hq, Hk, Hk))
    pages = B * T // page + 3
    slots = rng.permutation(pages * page)[: B * T].reshape(B, T)
    slots[rng.random((B, T)) < 0.2] = -1
    if layout == "tokens":
        kc, vc = torch.full((2, pages, page, Hk, d), 9.0, dtype=dt, device="cuda")
    elif layout == "heads":
        kc, vc = torch.full((2, pages, Hk, page, d), 9.0, dtype=dt, device="cuda").transpose(2, 3)
    else:                                                        # keys and values side by side in one allocation
        both = torch.full((pages, page, Hk, 2, d + 8), 9.0, dtype=dt, device="cuda")
        kc, vc = both[..., 0, :d], both[..., 1, :d]
    pos = rng.integers(-5, far, (len(sections), B, T)).astype(np.int32)
    kv, ql = rng.integers(T, far, B).astype(np.int32), rng.integers(0, T + 1, B).astype(np.int32)
    if text:
        pos = np.broadcast_to((kv - ql)[None, :, None] + np.arange(T), pos.shape)
    f = torch.tensor(1e6 ** (-np.arange(0, rot, 2) / rot), dtype=F32, device="cuda")
    qw, kw = ((0.5 + torch.rand(2, d, generator=g, device="cuda")) if norm else (None, None))
    ref = paged.rope_append(_f64(q), _f64(k), _f64(v), _f64(f), _f64(kc), _f64(vc), slots, pos, sections, ai, pi,
                            None if qw is None else _f64(qw), None if kw is None else _f64(kw), 1e-6,
                            _f64(q) if in_place else np.full(q.shape, 9.0))
    q_out = q if in_place else torch.full((B, T, Hq, d), 9.0, dtype=dt, device="cuda")
    st = _status()
    out = gdn.rope_append(q, k, v, f, kc, vc, torch.as_tensor(slots).cuda(), positions=None if text else _i32(pos), kv_len=_i32(kv),
                          q_len=_i32(ql), sections=sections, axes_interleaved=ai, pairs_interleaved=pi, q_norm=qw, k_norm=kw,
                          q_out=q_out, status_word=st)
    torch.cuda.synchronize()
    assert out is q_out and int(st) == 0
    step = 2.0 ** -8 if dt == BF else 0.0
    for name, x, r in (("q", q_out, ref[0]), ("k", kc, ref[1])):
        bound = step * np.abs(r) + 2e-6 * np.abs(r).max(-1, keepdims=True)
        assert (np.abs(_f64(x) - r) <= bound).all(), (name, np.max(np.abs(_f64(x) - r) / np.maximum(bound, 1e-300)))
    assert np.array_equal(_f64(vc), ref[2])
    if layout == "side":
        assert bool((both[..., d:] == 9.0).all())                # nothing outside the heads
    return q_out, kc, vc


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 64), (256, 256)])
@pytest.mark.parametrize("pi", [False, True])
def test_append_sizes(gdn, dt, d, rot, pi):
    _append(gdn, 3, 5, 6, 2, d, rot, [rot // 2], dt, pi=pi, seed=d + rot)


@pytest.mark.parametrize("sections,ai", [([32], False), ([10, 22], False), ([16, 8, 8], False), ([0, 0, 0, 32], False), ([16, 8, 8], True),
                                         ([22, 10], True), ([8, 8, 8, 8], True), ([32, 0, 0], True), ([30, 1, 1, 0], True)])
def test_append_axes(gdn, sections, ai):
    _append(gdn, 2, 7, 4, 1, 64, 64, sections, F32, ai=ai, norm=False, seed=len(sections))
    _append(gdn, 2, 7, 4, 1, 64, 64, sections, BF, ai=ai, pi=True, seed=len(sections))


@pytest.mark.parametrize("B,T,Hq,Hk,page,layout,fused,in_place,text",
                         [(1, 1, 1, 1, 1, "tokens", True, False, True), (1, 1, 24, 4, 64, "heads", True, True, False),
                          (2, 300, 3, 3, 7, "side", False, True, True), (200, 1, 16, 2, 16, "heads", False, False, False),
                          (40, 8, 40, 8, 24, "side", True, True, True), (5, 33, 13, 1, 128, "tokens", True, False, False)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_append_layouts(gdn, B, T, Hq, Hk, page, layout, fused, in_place, text, dt):
    _append(gdn, B, T, Hq, Hk, 128, 64, [16, 8, 8] if not text else [32], dt, page=page, layout=layout, fused=fused, in_place=in_place,
            text=text, seed=B + T)


@pytest.mark.parametrize("B,T,Hq,Hk,d", [(3, 2100, 2, 1, 64), (1, 6151, 9, 3, 128)])
def test_append_prompts(gdn, B, T, Hq, Hk, d):
    # so many tokens that a CTA takes sixteen of them, and the last CTA fewer
    _append(gdn, B, T, Hq, Hk, d, 16, [8], BF, seed=d)


def test_append_far_positions(gdn):
    # angles of up to 2^31 radians: what is left of a turn would be gone in 32 bits
    _append(gdn, 2, 64, 2, 1, 64, 64, [32], F32, far=(1 << 31) - 1, norm=False, seed=3)


def test_append_bad_slots_write_nothing(gdn):
    q, k, v = (torch.randn(1, 3, 2, 64, device="cuda") for _ in range(3))
    kc, vc = torch.zeros(2, 4, 16, 2, 64, device="cuda")
    q_out, st = torch.full_like(q, 5.0), _status()
    slots = torch.tensor([[64, 1 << 40, -7]], device="cuda")
    gdn.rope_append(q, k, v, torch.ones(32, device="cuda"), kc, vc, slots, kv_len=_i32([3]), q_len=_i32([3]), q_out=q_out, status_word=st)
    assert int(st) == 8 and bool((q_out == 5).all()) and not kc.any() and not vc.any()


def test_append_far_into_a_large_pool(gdn):
    # the last page starts behind element 2^31 of the cache
    page, Hk, d = 256, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 2
    kc, vc = torch.empty(pages, page, Hk, d, dtype=BF, device="cuda"), torch.empty(pages, page, Hk, d, dtype=BF, device="cuda")
    kc[-1], vc[-1] = 0, 0
    q, k, v = (torch.randn(1, 2, Hk, d, device="cuda").to(BF) for _ in range(3))
    slots = torch.tensor([[(pages - 1) * page + 3, pages * page - 1]], device="cuda")
    gdn.rope_append(q, k, v, torch.zeros(64, device="cuda"), kc, vc, slots, kv_len=_i32([2]), q_len=_i32([2]))
    assert torch.equal(kc[-1, 3], k[0, 0]) and torch.equal(kc[-1, 255], k[0, 1]) and torch.equal(vc[-1, 255], v[0, 1])
    assert not kc[-1, 4:255].any() and not kc[-1, :3].any()


# ------------------------------------------------------------------------------ the attention

# The kernel goes by what the block tables can hold. Every test of it runs with tables as wide as
# its lengths (the streaming kernel), and with tables so wide that the tensor-memory kernel takes what it can.
WIDE = False


@pytest.fixture(params=["narrow", "wide"])
def tables(request):
    global WIDE
    WIDE = request.param == "wide"
    yield request.param
    WIDE = False


def _cache(g, pages, page, Hk, d, dt, layout="tokens"):
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    if layout == "tokens":
        return r(pages, page, Hk, d), r(pages, page, Hk, d)
    if layout == "heads":
        return r(pages, Hk, page, d).transpose(1, 2), r(pages, Hk, page, d).transpose(1, 2)
    both = r(pages, page, Hk, 2, d + 8)
    return both[..., 0, :d], both[..., 1, :d]


def _attn_case(T, Hq, Hk, d, dt, page, lens, q_len=None, layout="tokens", seed=0, extra=0, stale=float("nan")):
    """Inputs with every slot behind a sequence's length, and every page of nobody, full of `stale`."""
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = [-(-max(0, x) // page) for x in lens]
    width = max(1, max(n) + extra)
    if WIDE:
        width = max(width, (1 << 23) // (B * Hk * d * page) + 1)
    ids = np.random.default_rng(seed).permutation(sum(n) + 2)
    kc, vc = _cache(g, sum(n) + 2, page, Hk, d, dt, layout)
    table = np.full((B, width), -1, np.int32)
    used = np.zeros((sum(n) + 2, page), bool)
    at = 0
    for b in range(B):
        table[b, : n[b]] = ids[at: at + n[b]]
        for j in range(lens[b]):
            used[table[b, j // page], j % page] = True
        at += n[b]
    if stale is not None:
        m = torch.as_tensor(~used).cuda()
        kc[m], vc[m] = stale, stale
    q = torch.randn(B, T, Hq, d, generator=g, device="cuda").to(dt)
    return dict(q=q, kc=kc, vc=vc, table=table, kv=np.asarray(lens, np.int32), ql=None if q_len is None else np.asarray(q_len, np.int32))


def _check_attn(x, o, lse, window=0, scale=None, keep=5.0):
    r, rl, written = paged.paged_attention(_f64(x["q"]), _f64(x["kc"]), _f64(x["vc"]), x["table"], x["kv"], x["ql"], scale, window)
    o64, l64 = _f64(o), _f64(lse)
    assert (o64[~written] == keep).all() and (l64[~written] == keep).all()
    top = np.nanmax(np.abs(np.where(np.isfinite(_f64(x["vc"])), _f64(x["vc"]), 0))) if x["vc"].numel() else 1.0
    bound = (4e-5 if x["q"].dtype == BF else 3e-5) * top + (2.0 ** -8 * np.abs(r) if o.dtype == BF else 0)
    r, rl, o64, l64 = r[written], rl[written], o64[written], l64[written]
    bound = np.broadcast_to(bound, written.shape + o.shape[2:])[written]
    assert np.array_equal(np.isneginf(rl), np.isneginf(l64))
    ok = np.isfinite(rl)
    l64, rl = l64[ok], rl[ok]
    assert (np.abs(l64 - rl) <= 2e-5 + 2.0 ** -22 * np.abs(rl)).all(), np.abs(l64 - rl).max()
    assert (np.abs(o64 - r) <= bound).all(), float(np.nanmax(np.abs(o64 - r) / bound))


def _run_attn(gdn, x, window=0, scale=None, out_dtype=None, status=0, workspace=None, table=None, check=True):
    out_dtype = out_dtype or x["q"].dtype
    o = torch.full(x["q"].shape, 5.0, dtype=out_dtype, device="cuda")
    lse, st = torch.full(x["q"].shape[:3], 5.0, device="cuda"), _status()
    gdn.paged_attention(x["q"], x["kc"], x["vc"], _i32(x["table"]), _i32(x["kv"]), q_len=None if x["ql"] is None else _i32(x["ql"]),
                        scale=scale, window=window, o=o, lse=lse, workspace=workspace, status_word=st)
    torch.cuda.synchronize()
    assert int(st) == status
    if check:
        _check_attn(x, o, lse, window, scale)
    return o, lse


# heads shared 1, 2, 3, 6, 8, 16 and 40 ways; 1 to 640 rows for one key head
@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 4, 4, 64), (1, 8, 1, 128), (1, 16, 1, 256), (2, 6, 2, 64), (8, 24, 4, 256), (8, 6, 1, 128),
                                       (16, 8, 1, 64), (16, 32, 2, 128), (3, 40, 1, 64), (16, 40, 1, 128), (5, 3, 3, 256), (11, 8, 4, 128)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_heads(gdn, tables, T, Hq, Hk, d, dt):
    x = _attn_case(T, Hq, Hk, d, dt, 16, [T, 100, 257], seed=T + Hq + d)
    _run_attn(gdn, x)


@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("page,layout", [(1, "tokens"), (7, "side"), (16, "heads"), (24, "tokens"), (64, "side"), (128, "heads"), (400, "tokens")])
def test_attention_pages_and_lengths(gdn, tables, T, d, dt, page, layout):
    lens = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300, 5]
    _run_attn(gdn, _attn_case(T, 4, 2, d, dt, page, lens, layout=layout, seed=page + T))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("window", [1, 3, 64, 100, 1000])
def test_attention_window(gdn, tables, window, dt):
    lens = [0, 1, 5, 64, 100, 101, 163, 450]
    for T, Hq in ((1, 2), (6, 12)):
        _run_attn(gdn, _attn_case(T, Hq, 2, 128, dt, 16, lens, seed=window), window=window)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq", [(4, 2), (8, 12), (16, 16)])
def test_attention_short_blocks(gdn, tables, T, Hq, dt):
    # rows behind a sequence's q_len stay as they were; a block longer than the sequence has rows
    # that see nothing
    lens, ql = [3, 40, 0, 200, 7, 9, 1], [T, 1, 2, 3, 0, min(4, T), T]
    for window in (0, 2):
        _run_attn(gdn, _attn_case(T, Hq, 2, 64, dt, 16, lens, q_len=ql, seed=T), window=window)


def test_attention_output_type_and_scale(gdn, tables):
    x = _attn_case(8, 12, 2, 128, BF, 16, [50, 333], seed=1)
    _run_attn(gdn, x, out_dtype=F32, scale=0.03)
    _run_attn(gdn, x, out_dtype=F32, scale=0.0)
    _run_attn(gdn, x, scale=-0.06)
    for window in (1 << 30, (1 << 31) - 1):
        _run_attn(gdn, x, window=window)
    y = _attn_case(1, 12, 2, 128, F32, 16, [50, 333], seed=1)
    _run_attn(gdn, y, out_dtype=BF)


@pytest.mark.parametrize("T,Hq,Hk,d,dt", [(1, 8, 2, 128, BF), (8, 24, 4, 256, BF), (8, 12, 2, 128, BF), (16, 8, 1, 64, BF), (1, 4, 2, 64, F32)])
def test_attention_long(gdn, tables, T, Hq, Hk, d, dt):
    # many pieces for one row: one long sequence, and one beside short ones
    _run_attn(gdn, _attn_case(T, Hq, Hk, d, dt, 64, [20011], seed=2))
    _run_attn(gdn, _attn_case(T, Hq, Hk, d, dt, 16, [5, 9000, 0, 64, 1], seed=2))


@pytest.mark.parametrize("T,Hq", [(1, 3), (8, 12)])
def test_attention_many_sequences(gdn, tables, T, Hq):
    rng = np.random.default_rng(T)
    _run_attn(gdn, _attn_case(T, Hq, 3, 64, BF, 16, rng.integers(0, 40, 700).tolist(), seed=T))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq", [(4, 2), (8, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_unseen_infinities(gdn, tables, T, Hq, dt, bad):
    # the last draft's key and value are not numbers: the rows before it do not see them
    x = _attn_case(T, Hq, 2, 64, dt, 16, [70, T, 130], seed=4)
    clean = _run_attn(gdn, x)
    for b, n in enumerate(x["kv"]):
        page, slot = x["table"][b, (n - 1) // 16], (n - 1) % 16
        x["kc"][page, slot], x["vc"][page, slot, :, 3] = bad, bad
    o, lse = _run_attn(gdn, x, check=False)
    assert torch.equal(o[:, :-1], clean[0][:, :-1]) and torch.equal(lse[:, :-1], clean[1][:, :-1])
    # and with a window, the rows that have left a position behind do not see it
    x = _attn_case(T, Hq, 2, 64, dt, 16, [70, 90], seed=5)
    clean = _run_attn(gdn, x, window=20)
    for b, n in enumerate(x["kv"]):
        j = n - T - 20 + 1                       # the first row's oldest position
        page, slot = x["table"][b, j // 16], j % 16
        x["vc"][page, slot, :, 1] = bad
    o, _ = _run_attn(gdn, x, window=20, check=False)
    assert torch.equal(o[:, 1:], clean[0][:, 1:])
    assert not bool(torch.isfinite(o[:, 0, :, 1]).any()) and torch.equal(o[:, 0, :, 2:], clean[0][:, 0, :, 2:])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 48])
def test_attention_unseen_values_by_place(gdn, tables, d, page):
    # a value that only the last row sees and one that only the first row sees, in any column of any tile
    T, W = 8, 150
    rng = np.random.default_rng(d + page)
    x = _attn_case(T, 12, 2, d, BF, page, [T, 128, 136, 260, 300, 517, 640], seed=d)
    clean = _run_attn(gdn, x, window=W)
    expect = clean[0].clone()
    for b, n in enumerate(x["kv"]):
        for pos, row in ((n - 1, T - 1), (n - T - W + 1, 0)):
            if pos < 0:
                continue
            h, col = int(rng.integers(2)), int(rng.integers(d))
            x["vc"][x["table"][b, pos // page], pos % page, h, col] = float("inf")
            expect[b, row, 6 * h:6 * h + 6, col] = float("inf")
    o, _ = _run_attn(gdn, x, window=W, check=False)
    assert torch.equal(o, expect)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq,d", [(8, 12, 64), (8, 12, 128), (16, 12, 256)])
def test_attention_rows_behind_the_block_change_nothing(gdn, tables, T, Hq, d, dt):
    # q's rows from q_len on are nobody's: the same bits whatever stands there
    rng = np.random.default_rng(d)
    lens = rng.integers(T, 900, 40).tolist()
    x = _attn_case(T, Hq, 2, d, dt, 16, lens, q_len=rng.integers(0, T + 1, 40), seed=d)
    behind = torch.arange(T, device="cuda")[None] >= _i32(x["ql"])[:, None]
    want = None
    for junk in (0.0, 1e4, float("nan"), float("-inf"), torch.finfo(dt).max):
        x["q"][behind] = junk
        got = _run_attn(gdn, x, check=want is None)
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), junk


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_stale_slots_cost_nothing(gdn, d):
    # what a page holds behind a sequence's length may be anything, and is looked at only there: a call over slots
    # full of NaN takes as long as one over zeros (each the best of five, so a factor of 1.5 is noise enough; walking
    # the items in search of such values took 4 to 6 times as long)
    def us(x):
        kv, table, o = _i32(x["kv"]), _i32(x["table"]), torch.empty_like(x["q"])
        ws = torch.empty(gdn.paged_attention_workspace_bytes(*x["q"].shape[:3], 4, d), dtype=torch.uint8, device="cuda")
        call = lambda: gdn.paged_attention(x["q"], x["kc"], x["vc"], table, kv, o=o, workspace=ws)  # noqa: E731
        call()
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best, o

    lens = [100 + 8000 * i // 31 for i in range(32)]
    (clean, o0), (nan, o1) = (us(_attn_case(8, 24, 4, d, BF, 64, lens, seed=1, stale=s)) for s in (0.0, float("nan")))
    assert torch.equal(o0, o1) and nan <= 1.5 * clean, (clean, nan)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,window", [(8, 0), (16, 5), (8, 700)])
def test_attention_seen_infinities_item_by_item(gdn, tables, d, T, window):
    # a visible infinity in some sequences only, among many that one CTA works through: the ones behind it are as they
    # were, and it reaches exactly the rows that see it
    rng = np.random.default_rng([d, T])
    lens = rng.integers(T, 300, 200).tolist()
    x = _attn_case(T, 24, 4, d, BF, 8, lens, seed=d)
    clean, _ = _run_attn(gdn, x, window=window)
    expect = clean.clone()
    for b in range(0, 200, 3):
        n, h, col = lens[b], int(rng.integers(4)), int(rng.integers(d))
        t = int(rng.integers(T))
        pos = n - T + t                              # row t's own position: the rows from t on see it
        x["vc"][x["table"][b, pos // 8], pos % 8, h, col] = float("inf")
        last = T if window == 0 else min(T, t + window)
        expect[b, t:last, 6 * h:6 * h + 6, col] = float("inf")
    o, _ = _run_attn(gdn, x, window=window, check=False)
    assert torch.equal(o, expect)


def _same_with_non_numbers(x, o, lse, window=0):
    """_check_attn where the definition gives infinities and NaN: those have to be the same, the rest within its bounds."""
    with np.errstate(all="ignore"):
        r, rl, written = paged.paged_attention(_f64(x["q"]), _f64(x["kc"]), _f64(x["vc"]), x["table"], x["kv"], x["ql"], None, window)
    o64, l64 = _f64(o), _f64(lse)
    for got, ref in ((o64[written], r[written]), (l64[written], rl[written])):
        for kind in (np.isnan, np.isposinf, np.isneginf):
            assert np.array_equal(kind(got), kind(ref)), kind
    ok = written[..., None, None] & np.isfinite(r)
    top = np.abs(_f64(x["vc"]))
    top = top[np.isfinite(top) & (top < 1e30)].max()
    bound = (4e-5 if x["q"].dtype == BF else 3e-5) * top + (2.0 ** -8 * np.abs(r) if o.dtype == BF else 0)
    assert (np.abs(o64[ok] - r[ok]) <= np.broadcast_to(bound, r.shape)[ok]).all()
    ok = written[..., None] & np.isfinite(rl)
    assert (np.abs(l64[ok] - rl[ok]) <= 2e-5 + 2.0 ** -22 * np.abs(rl[ok])).all()
    assert np.isfinite(r[written]).any() and not np.isfinite(r[written]).all()


def _put(x, b, pos, h, col, val, what="vc"):
    page = x["kc"].shape[1]
    x[what][x["table"][b, pos // page], pos % page, h, col] = val


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 4, 2, 128), (8, 12, 2, 64), (8, 12, 2, 128), (8, 6, 1, 256), (16, 16, 2, 64)])
def test_attention_seen_values_that_are_no_numbers(gdn, tables, T, Hq, Hk, d, dt):
    # where every row sees them, wherever they stand: infinities stay infinities, in their column, whether their item
    # is one CTA's or many's; a NaN, or both infinities, give NaN
    inf, nan = float("inf"), float("nan")
    for lens in ([300, 40, 700, 129], [5000, 333]):
        x = _attn_case(T, Hq, Hk, d, dt, 16, lens, seed=d + T)
        rng = np.random.default_rng(d + T)
        cols = rng.permutation(d)
        for b, n in enumerate(lens):
            for i, vals in enumerate(([inf], [-inf], [nan], [inf, -inf], [inf, inf, inf], [-inf, -inf], [inf, nan])):
                for v in vals:
                    _put(x, b, int(rng.integers(0, n - T)) if i else 0, int(rng.integers(Hk)) if len(vals) == 1 else 0, cols[i], v)
        for window in (0, 64):
            o, lse = _run_attn(gdn, x, window=window, check=False)
            _same_with_non_numbers(x, o, lse, window)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 4, 2, 128), (8, 12, 2, 64), (8, 12, 2, 128), (3, 6, 1, 256), (16, 16, 2, 64)])
def test_attention_keys_that_are_no_numbers(gdn, tables, T, Hq, Hk, d, dt):
    # an infinite element of a key is a score of plus or minus infinity by the query's sign: the row is NaN, or as if
    # the position were not there; so is an infinite element of a query, and a NaN is a NaN
    lens = [300, 40, 2500, 129]
    for which in range(3):
        x = _attn_case(T, Hq, Hk, d, dt, 16, lens, seed=d + T)
        if which == 0:
            for b, n in enumerate(lens):
                _put(x, b, n // 2, b % Hk, 7 * b, float("-inf") if b % 2 else float("inf"), "kc")
        elif which == 1:
            _put(x, 1, 20, 0, 3, float("nan"), "kc")
            _put(x, 2, 2490, 0, 5, float("-inf"), "kc")
        else:
            x["q"][0, T - 1, Hq - 1, 9] = float("inf")
            x["q"][3, 0, 0, 1] = float("nan")
        o, lse = _run_attn(gdn, x, check=False)
        _same_with_non_numbers(x, o, lse)


@pytest.mark.parametrize("T,Hq,dt", [(1, 4, BF), (8, 16, BF), (2, 4, F32)])
def test_attention_scores_of_minus_infinity(gdn, tables, T, Hq, dt):
    # keys that shut out all positions but some, and then all
    x = _attn_case(T, Hq, 2, 128, dt, 16, [500, 64, 90], seed=3)
    x["q"].abs_()
    clean = {k: v.clone() for k, v in x.items() if k in ("kc", "vc")}
    shut = np.ones(500, bool)
    shut[[3, 77, 140, 299, 471]] = False
    for pos in np.nonzero(shut)[0]:
        _put(x, 0, pos, slice(None), 11, float("-inf"), "kc")
    o, lse = _run_attn(gdn, x, check=False)
    k, v = (_f64(clean[n])[x["table"][0]].reshape(-1, 2, 128)[:500] for n in ("kc", "vc"))
    for t in range(T):
        see = [p for p in (3, 77, 140, 299, 471) if p <= 500 - T + t]
        for h in range(Hq):
            g = h * 2 // Hq
            s = k[see][:, g] @ _f64(x["q"])[0, t, h] / 128 ** 0.5
            w = np.exp(s - s.max())
            ref = w @ v[see][:, g] / w.sum()
            assert (np.abs(_f64(o)[0, t, h] - ref) <= 4e-5 * 6 + 2.0 ** -8 * np.abs(ref)).all()
            assert abs(float(lse[0, t, h]) - s.max() - np.log(w.sum())) <= 2e-5 + 2.0 ** -22 * 12
    x["kc"][..., 11] = float("-inf")
    o, lse = _run_attn(gdn, x, check=False)
    assert not o.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("T,Hq", [(4, 2), (8, 16)])
@pytest.mark.parametrize("bad", [float("-inf"), torch.finfo(F32).max, torch.finfo(F32).min])
def test_attention_unseen_largest_numbers(gdn, T, Hq, bad):
    # fp32 slots behind the sequences, and the last draft's key and value, full of a type's largest or lowest number
    x = _attn_case(T, Hq, 2, 64, F32, 16, [70, T, 130], seed=4, stale=0.0)
    clean = _run_attn(gdn, x)
    y = _attn_case(T, Hq, 2, 64, F32, 16, [70, T, 130], seed=4, stale=bad)
    o, lse = _run_attn(gdn, y)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
    for b, n in enumerate(y["kv"]):
        _put(y, b, n - 1, slice(None), slice(None), bad, "kc")
        _put(y, b, n - 1, slice(None), 3, bad)
    o, lse = _run_attn(gdn, y, check=False)
    assert torch.equal(o[:, :-1], clean[0][:, :-1]) and torch.equal(lse[:, :-1], clean[1][:, :-1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_long_fp32_sums_do_not_drift(gdn, d):
    # With values of one, an output is its weights' sum over the same sum: 1 but for roundings. Those of 64
    # additions that round have a deviation of sqrt(64) 2^-25 = 2.4e-7 at most, and their mean over 1024 rows one
    # of 7.5e-9; sums that are cut instead of rounded all lose, 64 2^-25 = 1.9e-6 on average. 2^-22 lies between.
    x = _attn_case(1, 16, 4, d, F32, 16, [4096] * 64, seed=d)
    x["vc"].fill_(1.0)
    o = torch.empty_like(x["q"])
    gdn.paged_attention(x["q"], x["kc"], x["vc"], _i32(x["table"]), _i32(x["kv"]), o=o)
    o = o.double()
    assert float((o - 1).abs().max()) <= 2e-5 and abs(float((o - 1).mean())) <= 2.0 ** -22


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,T", [(16, 8), (20, 8), (20, 1)])
def test_attention_long_bf16_sums_do_not_drift(gdn, d, page, T):
    # As above, of a bf16 cache: 160 items of 65,536 positions (all over the same pages), so that a CTA holds whole ones, on the
    # tensor-memory kernel (page 16) and the streaming one. A product of 16 positions cuts its sum by less than
    # 2^-23 of it; 2 of them go into each sum of the streaming kernel, 128 into each of the other's (256 are allowed for), whose
    # first half of growth counts half: 2^-22 and 2^-16 at most, however long the sequence; the additions that put those
    # together round to either side (2^-24 each, 2^-22 in the mean is allowed). Sums formed in the units all along
    # lose 8e-5 and 1e-5 here.
    S, Hq, Hk = 65536, 12, 2
    n = -(-S // page)
    kc = torch.randn(n, page, Hk, d, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda").to(BF)
    q = torch.randn(80, T, Hq, d, device="cuda").to(BF)
    table = torch.arange(n, dtype=torch.int32, device="cuda").repeat(80, 1)
    o = gdn.paged_attention(q, kc, torch.ones_like(kc), table, _i32([S] * 80), out_dtype=F32).double()
    assert abs(float((o - 1).mean())) <= (2.0 ** -16 if page == 16 else 2.0 ** -22) + 2.0 ** -22, float((o - 1).mean())


@pytest.mark.parametrize("d", [128, 256])
def test_attention_many_items_for_each_cta(gdn, tables, d):
    rng = np.random.default_rng(d)
    _run_attn(gdn, _attn_case(8, 12, 2, d, BF, 8, rng.integers(0, 400, 260).tolist(), seed=d))


@pytest.mark.parametrize("T,Hq", [(1, 4), (8, 16)])
def test_attention_extreme_scores(gdn, tables, T, Hq):
    # one key far ahead of all others, then all scores very negative, then equal
    x = _attn_case(T, Hq, 2, 128, BF, 16, [600], seed=6)
    x["kc"][x["table"][0, 20], 3] = x["q"][0, 0, 0] * 40
    _run_attn(gdn, x, check=False)
    x = _attn_case(T, Hq, 2, 128, BF, 16, [600], seed=6)
    x["kc"].copy_(-torch.ones_like(x["kc"]) * 64)
    x["q"].copy_(torch.ones_like(x["q"]) * 64)
    o, lse = _run_attn(gdn, x, check=False)      # every score is -64 64 sqrt(128), exactly representable products
    assert torch.allclose(lse[0, -1], torch.full_like(lse[0, -1], -4096 * 128 ** 0.5 + np.log(600)), rtol=2e-6)
    assert bool(torch.isfinite(o).all())


@pytest.mark.parametrize("T,Hq,dt", [(1, 4, BF), (8, 16, BF), (2, 4, F32)])
def test_attention_bad_lengths_and_pages(gdn, tables, T, Hq, dt):
    x = _attn_case(T, Hq, 2, 64, dt, 16, [40, 50, 60, 70, 33], q_len=[T] * 5, seed=7)
    x["kv"][1], x["kv"][2] = -1, x["table"].shape[1] * 16 + 1
    x["ql"][3], x["ql"][4] = T + 1, -1
    _run_attn(gdn, x, status=4)
    pages = x["kc"].shape[0]
    for bad in (-1, pages, 1 << 30, -(1 << 31)):
        x = _attn_case(T, Hq, 2, 64, dt, 16, [100, 40], seed=8)
        x["table"][0, 2], x["table"][1, 2] = bad, bad
        _run_attn(gdn, x, status=8)
    x["table"][:] = -5                            # nothing left to see
    o, lse = _run_attn(gdn, x, status=8)
    assert not o.any() and bool(torch.isneginf(lse).all())


def test_attention_far_into_a_large_pool(gdn):
    page, Hk, d = 256, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 3
    kc, vc = torch.empty(pages, page, Hk, d, dtype=BF, device="cuda"), torch.empty(pages, page, Hk, d, dtype=BF, device="cuda")
    kc[-2:], vc[-2:] = torch.randn(2, 2, page, Hk, d, device="cuda").to(BF)
    for T, Hq, width in ((1, 16, 2), (8, 48, 2), (8, 48, 40)):
        table = np.full((1, width), -1, np.int32)
        table[0, :2] = pages - 1, pages - 2
        q = torch.randn(1, T, Hq, d, device="cuda").to(BF)
        o, lse = gdn.paged_attention(q, kc, vc, _i32(table), _i32([300]), lse=(l := torch.empty(1, T, Hq, device="cuda"))), l
        torch.cuda.synchronize()
        _check_attn(dict(q=q, kc=kc[-2:], vc=vc[-2:], table=np.array([[1, 0]]), kv=[300], ql=None), o, lse)


def test_attention_streams_graphs_and_repeats(gdn, tables):
    # the same bits from a side stream, from two captured graphs (a workspace each), and again
    cases = [_attn_case(8, 24, 4, 128, BF, 16, [3000, 17, 800], seed=9), _attn_case(1, 8, 4, 64, BF, 16, [900, 1, 64], seed=10)]
    want = [_run_attn(gdn, x) for x in cases]
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for x in cases:
        B, T, Hq, d = x["q"].shape
        ws = torch.full((gdn.paged_attention_workspace_bytes(B, T, Hq, x["kc"].shape[2], d),), 255, dtype=torch.uint8, device="cuda")
        o, lse = torch.zeros_like(x["q"]), torch.zeros(B, T, Hq, device="cuda")
        args = (x["q"], x["kc"], x["vc"], _i32(x["table"]), _i32(x["kv"]))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            gdn.paged_attention(*args, o=o, lse=lse, workspace=ws)
        s.synchronize()
        outs.append((o, lse, args, ws))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gdn.paged_attention(*args, o=o, lse=lse, workspace=ws)
        graphs.append(graph)
    for (o, lse, _, _), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
        o.zero_()
    for _ in range(2):
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for (o, lse, _, _), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("T,Hq,d,page", [(8, 12, 64, 16), (8, 12, 128, 16), (8, 12, 256, 16), (16, 12, 64, 16), (16, 12, 256, 16), (8, 12, 128, 20), (1, 4, 256, 16)])
def test_attention_maxima_that_grow_along_a_sequence(gdn, T, Hq, d, page):
    # Rows whose best score so far is left behind by 2^16 and more, again and again, in tiles far into an item, each row
    # at places of its own; a CTA holds some twenty tiles of an item. Scores of up to 80 (1.1 times that in sums of their
    # terms' sizes, A): 16 steps of a product cut 2^-23 each, so a weight is off by 2e-6 A, o by twice that and the
    # 4e-5 of other scores, of max|v|. A row one of whose keys is 40 ahead of all others is that key's value.
    B, Hk = 64, 2
    rng = np.random.default_rng([T, d, page])
    lens = rng.integers(2500, 3300, B).tolist()
    x = _attn_case(T, Hq, Hk, d, BF, page, lens, seed=d + T)
    q = _f64(x["q"])
    final = {}
    for b, n in enumerate(lens):
        for i, pos in enumerate(np.sort(rng.choice(n - T, 8, replace=False))):
            t, h = int(rng.integers(T)), int(rng.integers(Hq))
            score = 12.0 + 9.0 * i if (b % 4) else 80.0 - 8.0 * i           # growing, or the greatest first
            key = q[b, t, h] * score * d ** 0.5 / (q[b, t, h] ** 2).sum()
            x["kc"][x["table"][b, pos // page], pos % page, h * Hk // Hq] = torch.as_tensor(key).to(BF).cuda()
        t, h, pos = int(rng.integers(T)), int(rng.integers(Hq)), int(rng.integers(n // 2, n - T))
        key = q[b, t, h] * 140.0 * d ** 0.5 / (q[b, t, h] ** 2).sum()
        if b % 2:
            x["kc"][x["table"][b, pos // page], pos % page, h * Hk // Hq] = torch.as_tensor(key).to(BF).cuda()
            final[b] = (t, h, pos)
    o, lse = _run_attn(gdn, x, check=False)
    for b, (t, h, pos) in final.items():
        assert torch.equal(o[b, t, h], x["vc"][x["table"][b, pos // page], pos % page, h * Hk // Hq]), b
    few = [0, 1, 2, 4, 7, 62]
    r, rl, _ = paged.paged_attention(q[few], _f64(x["kc"]), _f64(x["vc"]), x["table"][few], x["kv"][few], None, None, 0)
    top = float(np.nanmax(np.abs(_f64(x["vc"]))))
    A = 160.0
    assert (np.abs(_f64(o)[few] - r) <= (2 * 2e-6 * A + 4e-5) * top + 2.0 ** -8 * np.abs(r)).all()
    assert (np.abs(_f64(lse)[few] - rl) <= 2e-6 * A + 2e-5 + 2.0 ** -22 * np.abs(rl)).all()


def test_attention_kernel_choice(gdn):
    # each branch of the rule, on both of its sides
    def name(B, T, Hq, Hk, d, dt, page, capacity):
        x = _attn_case(T, Hq, Hk, d, dt, page, [20] * B, extra=capacity // page - -(-20 // page), seed=1)
        _, names = launched_kernels(lambda: _run_attn(gdn, x, check=False))
        return any("attention_tc_kernel" in n for n in names)

    assert not name(1, 8, 24, 4, 64, BF, 16, 4096) and name(1, 8, 24, 4, 64, BF, 16, 8192)
    assert not name(8, 4, 32, 4, 64, BF, 16, 8192) and name(8, 5, 32, 4, 64, BF, 16, 8192)
    assert not name(1, 8, 24, 4, 128, BF, 16, 2048) and name(1, 8, 24, 4, 128, BF, 16, 4096)
    assert not name(8, 2, 32, 4, 128, BF, 16, 4096) and name(8, 3, 32, 4, 128, BF, 16, 4096)
    assert not name(1, 8, 24, 4, 256, BF, 16, 2048) and name(1, 8, 24, 4, 256, BF, 16, 4096)
    assert not name(1, 1, 24, 4, 256, BF, 16, 4096) and name(1, 1, 24, 4, 256, BF, 16, 8192)
    assert not name(8, 8, 24, 4, 128, F32, 16, 8192) and not name(8, 8, 24, 4, 128, BF, 20, 8200)


def test_attention_empty_batch(gdn):
    q = torch.empty(0, 1, 4, 64, dtype=BF, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, dtype=BF, device="cuda")
    assert gdn.paged_attention(q, kc, kc.clone(), _i32(np.zeros((0, 3))), _i32([])).shape == (0, 1, 4, 64)


# ------------------------------------------------------------------------------ together

def test_a_stack_of_mixers_and_attention_layers(gdn):
    """verify (a programmatic dependent) -> append -> attention, layer upon layer on one stream, over shared scratch, as a
    hybrid stack runs them: the results of the same calls one by one, eagerly and from a graph."""
    from gated_deltanet_mixer_verify_b200.inputs import make_inputs, workload
    from gdn_helpers import to_dev
    w = workload("single_seq_verify")
    L0 = make_inputs(w, layer=0)["accept_len"].numpy()
    mix = [to_dev(make_inputs(w, layer=i, accept_len=L0, gates="gentle")) for i in range(4)]
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    B, T, Hq, Hk, d, page, past = 1, mix[0]["q"].shape[1], 24, 4, 256, 64, 9000
    pages = -(-(past + T) // page) + 400
    layers = [dict(q=r(B, T, Hq, d), k=r(B, T, Hk, d), v=r(B, T, Hk, d), kc=r(pages, page, Hk, d), vc=r(pages, page, Hk, d)) for _ in mix]
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
    kv, ql = _i32([past + T]), _i32([T])
    pos = torch.arange(past, past + T, device="cuda")
    slots = (table[0, pos // page].long() * page + pos % page).view(B, T)
    freq = torch.tensor(1e6 ** (-np.arange(0, 64, 2) / 64), dtype=F32, device="cuda")
    q_out, ws = torch.empty(B, T, Hq, d, dtype=BF, device="cuda"), torch.empty(gdn.paged_attention_workspace_bytes(B, T, Hq, Hk, d), dtype=torch.uint8,
                                                                               device="cuda")

    def run(states, caches, outs, one_by_one=False):
        for m, a, st, (kc, vc), (om, oa) in zip(mix, layers, states, caches, outs):
            gdn.verify_step(m["q"], m["k"], m["v"], m["a"], m["b"], m["A_log"], m["dt_bias"], st, st, m["accept_len"], om, pdl=not one_by_one)
            if one_by_one:
                torch.cuda.synchronize()
            gdn.rope_append(a["q"], a["k"], a["v"], freq, kc, vc, slots, kv_len=kv, q_len=ql, q_out=q_out)
            if one_by_one:
                torch.cuda.synchronize()
            gdn.paged_attention(q_out, kc, vc, table, kv, q_len=ql, o=oa, workspace=ws)
            if one_by_one:
                torch.cuda.synchronize()

    def fresh():
        return ([m["S0"].clone() for m in mix], [(a["kc"].clone(), a["vc"].clone()) for a in layers],
                [(torch.zeros(m["v"].shape, device="cuda"), torch.zeros(B, T, Hq, d, dtype=BF, device="cuda")) for m in mix])

    want = fresh()
    run(*want, one_by_one=True)
    flat = lambda x: [*x[0], *(t for p in x[1] + x[2] for t in p)]  # noqa: E731
    for _ in range(3):
        got = fresh()
        torch.cuda.synchronize()
        run(*got)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))
    got = fresh()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(*got)
    for a, b in zip(flat(got), flat(fresh())):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))


@pytest.mark.parametrize("dt", [BF, F32])
def test_verify_loop(gdn, dt):
    """Four rounds of plan -> append -> attention -> greedy acceptance, the accept counts of one
    round committed by the next one's plan, nothing read on the host in between; every round's
    outputs against dense fp64 attention over the accepted tokens and the block, in tokens' order."""
    B, T, Hq, Hk, d, page, V = 5, 8, 6, 2, 64, 16, 64
    rng = np.random.default_rng(11)
    g = torch.Generator(device="cuda").manual_seed(11)
    width, pages = 8, 30
    seq, held, table = _i32([0] * B), _i32([0] * B), _i32(np.full((B, width), -1))
    free, count = _i32(rng.permutation(pages)), _i32([pages])
    kc = torch.full((pages, page, Hk, d), float("nan"), dtype=dt, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    f = torch.tensor(1e4 ** (-np.arange(0, d, 2) / d), dtype=F32, device="cuda")
    accepted, last, prompt = None, None, [3, 0, 17, 30, 1]
    st = _status()
    past = [[] for _ in range(B)]            # (k, v) rows of each sequence, as given, in order
    rounds = []
    for r in range(5):
        n = 32 if r == 0 else T              # the prompts first, ragged
        add = _i32(prompt) if r == 0 else _i32([T] * (B - 1) + [T if r < 3 else -1])
        kv, ql, slots = gdn.kv_plan(seq, held, table, free, count, n, page, commit_len=accepted, add_len=add, block_len=last,
                                     status_word=st)
        last = ql
        qkv = torch.randn(B, n, (Hq + 2 * Hk) * d, generator=g, device="cuda").to(dt)
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
        qr = gdn.rope_append(q, k, v, f, kc, vc, slots, kv_len=kv, q_len=ql, q_out=torch.zeros(B, n, Hq, d, dtype=dt, device="cuda"),
                             status_word=st)
        if r == 0:
            accepted = ql                    # a prompt is kept whole
            rounds.append((q, k, v, None, kv.clone(), ql.clone(), None))
            continue
        o = gdn.paged_attention(qr, kc, vc, table, kv, q_len=ql, o=torch.zeros_like(qr), status_word=st)
        tokens = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
        logits = torch.randn(B, T, V, generator=g, device="cuda")
        logits[:, :-1].scatter_add_(2, tokens[:, 1:, None].long(), 3 + torch.rand(B, T - 1, 1, generator=g, device="cuda"))
        accepted, _ = gdn.accept(logits, tokens)
        rounds.append((q, k, v, o, kv.clone(), ql.clone(), accepted.clone()))
    torch.cuda.synchronize()
    assert int(st) == 0
    inv = _f64(f)
    for r, (q, k, v, o, kv, ql, acc) in enumerate(rounds):
        kv, ql = kv.cpu().numpy(), ql.cpu().numpy()
        for b in range(B):
            if r >= 3 and b == B - 1:
                assert kv[b] == 0 and ql[b] == 0 and not o[b].any()
                continue
            assert kv[b] - ql[b] == len(past[b])
            rows = past[b] + [(_f64(k[b, t]), _f64(v[b, t])) for t in range(ql[b])]
            if r > 0:
                K = np.stack([paged.rotate(x, None, [j], inv, [d // 2], False, False, 0.0) for j, (x, _) in enumerate(rows)])
                W = np.stack([y for _, y in rows])
                if dt == BF:                 # the cache and the queries hold rounded values
                    K = _f64(torch.tensor(K).to(BF))
                for t in range(ql[b]):
                    p = kv[b] - ql[b] + t
                    Q = paged.rotate(_f64(q[b, t]), None, [p], inv, [d // 2], False, False, 0.0)
                    if dt == BF:
                        Q = _f64(torch.tensor(Q).to(BF))
                    for h in range(Hq):
                        s = K[: p + 1, h // 3] @ Q[h] / 8
                        w = np.exp(s - s.max())
                        ref = w @ W[: p + 1, h // 3] / w.sum()
                        # bf16: a key or query element near a border of its type may be stored one
                        # step off (its fp32 value differs in the last bits), 2^-7 of it: sqrt(d) such
                        # steps of |q k| / 8 below 6 would be 2^-7 6 / 8 in a score at worst, so 0.05 max|v|
                        tol = 5e-5 * np.abs(W).max() if dt == F32 else 2.0 ** -8 * np.abs(ref) + 0.05 * np.abs(W).max()
                        assert (np.abs(_f64(o[b, t, h]) - ref) <= tol).all(), (r, b, t, h)
            keep = ql[b] if acc is None else int(acc[b])
            past[b] = rows[: len(past[b]) + keep]
    # every page is somebody's or free, once
    held, table, n = held.cpu().numpy(), table.cpu().numpy(), int(count)
    assert sorted([table[b, i] for b in range(B) for i in range(held[b])] + free.cpu().numpy()[:n].tolist()) == list(range(pages))

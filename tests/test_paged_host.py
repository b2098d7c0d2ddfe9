"""Refusals of the paged attention calls, made on the host before any launch (no GPU needed:
nothing here is ever launched)."""
import pytest
import torch

from gated_deltanet_mixer_verify_b200 import build as gbuild

INVALID, UNSUP, WORKSPACE = -1, -2, -4
F32, BF16 = 0, 1
FAKE = 0x100000


@pytest.fixture(scope="module")
def gdn():
    gbuild.build()
    from gated_deltanet_mixer_verify_b200 import gdn as g
    return g


def _shape(gdn, **kw):
    f = dict(B=2, T=8, H_q=24, H_kv=4, d=128, dtype=BF16, out_dtype=BF16, page_size=16, num_pages=100, max_pages=8,
             page_stride=16 * 4 * 128, slot_stride=4 * 128, head_stride=128, status_word=0)
    f.update(kw)
    return gdn._pack_kv_shape(*f.values())


def _err(gdn):
    return gdn.lib().gdn_last_error().decode()


def test_plan_refusals(gdn):
    lib = gdn.lib()
    names = ["seq_in", "seq_out", "commit", "block", "add", "held_in", "held_out", "table", "free", "count_in", "count_out", "kv", "ql",
             "slots"]

    def call(shape=None, **kw):
        # one region per array, 1 MiB apart; the counts in place
        at = {n: FAKE * (i + 1) for i, n in enumerate(names)}
        at.update(seq_out=at["seq_in"], held_out=at["held_in"], count_out=at["count_in"])
        at.update(kw)
        return lib.gdn_kv_plan(shape or _shape(gdn), *[at[n] for n in names], None)

    assert lib.gdn_kv_plan(None, *([FAKE] * 14), None) == INVALID
    for bad in (dict(B=-1), dict(T=0), dict(page_size=0), dict(num_pages=0), dict(max_pages=0)):
        assert call(_shape(gdn, **bad)) == INVALID and "positive" in _err(gdn), bad
    for bad in (dict(B=65536), dict(T=(1 << 20) + 1), dict(page_size=65537), dict(max_pages=1 << 27)):
        assert call(_shape(gdn, **bad)) == UNSUP, bad
    assert call(_shape(gdn, status_word=FAKE + 2)) == INVALID and "status_word" in _err(gdn)
    for n in names:
        if n not in ("commit", "block", "add"):
            assert call(**{n: None}) == INVALID and "is NULL" in _err(gdn), n
        assert call(**{n: FAKE * 40 + 8}) == INVALID and "16-byte aligned" in _err(gdn), n
    assert call(kv=FAKE) == INVALID and "an output overlaps an input" in _err(gdn)
    assert call(block=FAKE * 12) == INVALID and "an output overlaps an input" in _err(gdn)      # kv_len
    assert call(kv=FAKE * 30, ql=FAKE * 30) == INVALID and "two outputs overlap" in _err(gdn)
    assert call(slots=FAKE * 8) == INVALID and "two outputs overlap" in _err(gdn)
    assert call(commit=FAKE * 12) == INVALID and "an output overlaps" in _err(gdn)


def test_append_refusals(gdn):
    lib = gdn.lib()
    def rope(**kw):
        f = dict(dict(rot=128, n_axes=3, sections=(32, 16, 16, 0), ai=0, pi=0, eps=1e-6, q=24 * 128, k=4 * 128, v=4 * 128,
                      o=24 * 128), **kw)
        return gdn._pack_rope(f["rot"], f["n_axes"], *f["sections"], *list(f.values())[3:])

    def call(shape=None, r=None, **kw):
        names = ["q", "k", "v", "inv_freq", "positions", "kv_len", "q_len", "slots", "q_norm", "k_norm", "q_out", "k_cache",
                 "v_cache"]
        at = {n: FAKE * (i + 1) for i, n in enumerate(names)}
        at.update(kw)
        return lib.gdn_rope_append(shape or _shape(gdn), r or rope(), *[at[n] for n in names], None)

    assert call(_shape(gdn, H_q=23)) == INVALID and "multiple of H_kv" in _err(gdn)
    assert call(_shape(gdn, d=96)) == UNSUP and "not built" in _err(gdn)
    assert call(_shape(gdn, dtype=7)) == INVALID and "dtype 7" in _err(gdn)
    assert call(_shape(gdn, T=(1 << 20) + 1)) == UNSUP
    for s in ("page_stride", "slot_stride", "head_stride"):
        assert call(_shape(gdn, **{s: 64})) == INVALID and s in _err(gdn)            # less than d
        assert call(_shape(gdn, **{s: 4 * 128 + 4})) == INVALID and s in _err(gdn)   # not 16 bytes
    sec = lambda *v: v  # noqa: E731
    for bad in (dict(rot=8), dict(rot=24), dict(rot=144), dict(n_axes=0), dict(n_axes=5), dict(sections=sec(32, 16, 15, 0)),
                dict(sections=sec(80, -16, 0, 0)), dict(ai=2), dict(pi=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(ai=1, sections=sec(2, 30, 32, 0)), dict(q=24 * 128 - 8), dict(k=4 * 128 + 4), dict(v=0), dict(o=128)):
        assert call(r=rope(**bad)) == INVALID, bad
    assert lib.gdn_rope_append(_shape(gdn), None, *([FAKE] * 13), None) == INVALID
    for n in ("q", "k", "v", "inv_freq", "slots", "q_out", "k_cache", "v_cache"):
        assert call(**{n: None}) == INVALID and "is NULL" in _err(gdn), n
    assert call(positions=None, kv_len=None) == INVALID and "kv_len is NULL" in _err(gdn)
    assert call(positions=None, q_len=None) == INVALID and "q_len is NULL" in _err(gdn)
    assert call(v_cache=FAKE + 8) == INVALID and "16-byte aligned" in _err(gdn)
    assert call(q_out=FAKE, r=rope(o=25 * 128)) == INVALID and "in place" in _err(gdn)
    assert call(q_out=FAKE + 16) == INVALID and "overlaps" in _err(gdn)
    assert call(q_out=FAKE * 2) == INVALID and "overlaps" in _err(gdn)
    assert call(_shape(gdn, B=0), q=None, q_out=None) == 0


def test_attention_refusals(gdn):
    lib = gdn.lib()

    def call(shape=None, scale=0.1, window=0, nbytes=1 << 40, **kw):
        names = ["q", "k", "v", "table", "kv_len", "q_len", "o", "lse", "ws"]
        at = {n: FAKE * (i + 1) for i, n in enumerate(names)}
        at.update(kw)
        return lib.gdn_paged_attention(shape or _shape(gdn), scale, window, *[at[n] for n in names], nbytes, None)

    for bad, want in ((dict(T=17), UNSUP), (dict(T=0), INVALID), (dict(B=65536), UNSUP), (dict(d=80), UNSUP), (dict(H_q=25), INVALID),
                      (dict(dtype=3), INVALID), (dict(out_dtype=3), INVALID), (dict(max_pages=0), INVALID),
                      (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=1 << 17), UNSUP),
                      (dict(max_pages=1 << 28), UNSUP), (dict(head_stride=64), INVALID), (dict(slot_stride=129), INVALID),
                      (dict(status_word=FAKE + 1), INVALID)):
        assert call(_shape(gdn, **bad)) == want, bad
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(window=-1) == INVALID and "window" in _err(gdn)
    for n in ("q", "k", "v", "table", "kv_len", "o"):
        assert call(**{n: None}) == INVALID and "is NULL" in _err(gdn), n
        assert call(**{n: FAKE * 40 + 8}) == INVALID and "16-byte aligned" in _err(gdn), n
    assert call(o=FAKE + 16) == INVALID and "o overlaps q" in _err(gdn)
    need = gdn.paged_attention_workspace_bytes(2, 8, 24, 4, 128)
    if need:
        assert call(nbytes=need - 1) == WORKSPACE and str(need) in _err(gdn)
        assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 8) == INVALID and "workspace not 16-byte aligned" in _err(gdn)
    assert gdn.paged_attention_workspace_bytes(2, 17, 24, 4, 128) == 0
    assert gdn.paged_attention_workspace_bytes(2, 8, 24, 5, 128) == 0
    assert call(_shape(gdn, B=0), q=None) == 0


def test_attention_refuses_what_it_writes_over_what_it_uses(gdn):
    names = ["q", "k", "v", "table", "kv_len", "q_len", "o", "lse", "ws"]
    at = {n: FAKE * 64 * (i + 1) for i, n in enumerate(names)}
    need = gdn.paged_attention_workspace_bytes(2, 8, 24, 4, 128)
    size = dict(q=2 * 8 * 24 * 128 * 2, o=2 * 8 * 24 * 128 * 2, lse=2 * 8 * 24 * 4, ws=need, table=2 * 8 * 4, kv_len=8, q_len=8)
    call = lambda **kw: gdn.lib().gdn_paged_attention(_shape(gdn), 0.1, 0, *dict(at, **kw).values(), need, None)  # noqa: E731
    for out in ("o", "lse", "ws"):
        for other in size:
            if other == out:
                continue
            for p in (at[other], at[other] + (size[other] - 1) // 16 * 16, at[other] - (size[out] - 1) // 16 * 16):
                assert call(**{out: p}) == INVALID and "overlaps" in _err(gdn), (out, other)


def test_attention_selftest_refusals(gdn):
    at = [FAKE * (i + 1) for i in range(9)]
    call = lambda polls, *p: gdn.lib().gdn_selftest_attention_wait(_shape(gdn), 0.1, 0, *(p or at), 1 << 40, polls, None)  # noqa: E731
    for polls in (0, (1 << 20) + 1):
        assert call(polls) == INVALID and "polls" in _err(gdn)
    assert call(16, None, *at[1:]) == INVALID and _err(gdn).startswith("gdn_selftest_attention_wait: q is NULL")


def test_binding_refusals(gdn):
    # raised before any pointer is taken, so CPU tensors suffice
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    plan = lambda **kw: gdn.kv_plan(**dict(dict(seq_len=i32(2), n_pages=i32(2), block_table=i32(2, 4), free_list=i32(9),  # noqa: E731
                                                free_count=i32(1), T=8, page_size=16), **kw))
    for kw, msg in ((dict(seq_len=i32(2).long()), "seq_len must be int32"), (dict(add_len=i32(2).float()), "add_len must be int32"),
                    (dict(slot_map=i32(2, 8)), "slot_map must be int64"), (dict(status_word=i32(1).long()), "status_word")):
        with pytest.raises(TypeError, match=msg):
            plan(**kw)
    for kw, msg in ((dict(n_pages=i32(3)), "n_pages must be"), (dict(commit_len=i32(1)), "commit_len must be"),
                    (dict(free_list=i32(3, 3)), "free_list"), (dict(free_count=i32(2)), "free_count"),
                    (dict(slot_map=torch.zeros(2, 7, dtype=torch.int64)), "slot_map must be")):
        with pytest.raises(ValueError, match=msg):
            plan(**kw)

    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    app = lambda **kw: gdn.rope_append(**dict(dict(q=bf(2, 8, 6, 64), k=bf(2, 8, 2, 64), v=bf(2, 8, 2, 64), inv_freq=torch.zeros(32),  # noqa: E731
                                                   k_cache=bf(5, 16, 2, 64), v_cache=bf(5, 16, 2, 64),
                                                   slot_map=torch.zeros(2, 8, dtype=torch.int64), kv_len=i32(2), q_len=i32(2)), **kw))
    for kw, msg in ((dict(k=bf(2, 8, 2, 64).float()), "share a dtype"), (dict(k_cache=bf(5, 16, 2, 64).float()), "dtype of q"),
                    (dict(inv_freq=torch.zeros(32).double()), "inv_freq must be float32"), (dict(slot_map=i32(2, 8)), "slot_map must be int64"),
                    (dict(q_norm=bf(64)), "q_norm must be float32"), (dict(positions=torch.zeros(1, 2, 8)), "positions must be int32"),
                    (dict(q_out=bf(2, 8, 6, 64).float()), "q_out must have")):
        with pytest.raises(TypeError, match=msg):
            app(**kw)
    wide = bf(2, 8, 12, 64)
    for kw, msg in ((dict(v=bf(2, 8, 3, 64)), "disagree"), (dict(k_cache=bf(5, 16, 3, 64)), "k_cache and v_cache must be"),
                    (dict(v_cache=bf(5, 2, 16, 64).transpose(1, 2)), "same strides"), (dict(q=wide[:, :, ::2]), "contiguous heads"),
                    (dict(q=bf(8, 2, 6, 64).transpose(0, 1)), "one stride from token to token"),
                    (dict(sections=[8] * 5), "one to four"), (dict(positions=i32(2, 2, 8)), "positions must be"),
                    (dict(q_norm=torch.zeros(32)), "q_norm must be"), (dict(kv_len=i32(3)), "kv_len must be"),
                    (dict(), "expected a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            app(**kw)

    attn = lambda **kw: gdn.paged_attention(**dict(dict(q=bf(2, 8, 6, 64), k_cache=bf(5, 16, 2, 64), v_cache=bf(5, 16, 2, 64),  # noqa: E731
                                                        block_table=i32(2, 3), kv_len=i32(2)), **kw))
    for kw, msg in ((dict(q=bf(2, 8, 6, 64).half()), "dtype"), (dict(v_cache=bf(5, 16, 2, 64).float()), "dtype of q"),
                    (dict(kv_len=i32(2).long()), "kv_len must be int32"), (dict(lse=bf(2, 8, 6)), "lse must be float32"),
                    (dict(o=bf(2, 8, 6, 64), out_dtype=torch.float32), "out_dtype")):
        with pytest.raises(TypeError, match=msg):
            attn(**kw)
    for kw, msg in ((dict(o=bf(2, 8, 6, 32)), "o must be"), (dict(block_table=i32(3, 3)), "block_table"),
                    (dict(q_len=i32(1)), "q_len must be"), (dict(lse=torch.zeros(2, 6, 8)), "lse must be"),
                    (dict(k_cache=bf(5, 16, 128)), "k_cache and v_cache must be"), (dict(), "expected a CUDA tensor")):
        with pytest.raises(ValueError, match=msg):
            attn(**kw)


def test_native_checks_agree_with_the_slow_ones(gdn):
    # the native look answers exactly where the tensor-by-tensor one does, with the same pointers
    spec = (("a", torch.int32, (0, 1)), ("b", torch.float32, (1,)), ("c", torch.int64, (0,)))
    a, b, c = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3), torch.zeros(2, dtype=torch.int64)
    native = gdn._native().pointers
    slow = lambda *t: tuple(gdn._want(n, x, dt, tuple((2, 3)[i] for i in ax), -1) for (n, dt, ax), x in zip(spec, t))  # noqa: E731
    assert native(spec, -1, (2, 3), a, b, None) == slow(a, b, None) == (a.data_ptr(), b.data_ptr(), None)
    assert gdn._pointers(spec, -1, (2, 3), a, b, c) == slow(a, b, c)
    for bad in ((a.long(), b, c), (a.t(), b, c), (a[:1], b, c), (a, b[:2], c), (a, b.double(), c), (a, b, c[:, None]),
                (torch.zeros(3, 2, dtype=torch.int32).t(), b, c), (a, b, 5)):
        assert native(spec, -1, (2, 3), *bad) is None
    assert native(spec, 0, (2, 3), a, b, c) is None
    for wrong in ((), (spec,), (spec, -1, (2, 3), a), (spec, -1, [2, 3], a, b, c)):
        with pytest.raises(TypeError):
            native(*wrong)
    with pytest.raises(TypeError, match="a must be int32"):
        gdn._pointers(spec, -1, (2, 3), b, b, c)

    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    wide, k, v = bf(2, 5, 12, 64), bf(3, 2, 16, 64).transpose(1, 2), bf(3, 2, 16, 64).transpose(1, 2)
    q = wide[:, :, 2:8]
    assert gdn._native().tokens(torch.bfloat16, -1, 2, 5, 64, q, 6) == (gdn._token_stride("q", q, 2, 5, 6, 64), q.data_ptr())
    for one in (bf(4, 1, 6, 64), bf(1, 1, 6, 64), wide[:1, :1, :6], wide[:, :1, :6]):
        assert gdn._native().tokens(torch.bfloat16, -1, one.shape[0], 1, 64, one, 6)[0] == gdn._token_stride("q", one, one.shape[0], 1, 6, 64)
    for t in (wide[:, :, ::2], wide[:, ::2, :6], wide[:, :, :6].float(), wide[..., :32], bf(5, 2, 6, 64).transpose(0, 1)):
        assert gdn._native().tokens(torch.bfloat16, -1, 2, 5, 64, t, 6) is None
    assert gdn._native().caches(k, v, torch.bfloat16, -1, 2, 64) == (16, 3, 2048, 64, 1024, k.data_ptr(), v.data_ptr())
    for pair in ((k, v.contiguous()), (k.float(), v), (k[:2], v), (k[..., :32], v[..., :32]), (k[0], v[0])):
        assert gdn._native().caches(*pair, torch.bfloat16, -1, 2, 64) is None

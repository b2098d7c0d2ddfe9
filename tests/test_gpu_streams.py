"""Calls launched on a stream that is not the current one: what they make themselves is not handed out again while their
kernels still run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def gdn(cuda_device):
    from gated_deltanet_mixer_verify_b200 import build, gdn as g
    build.build()
    return g


def _calls(gdn):
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s, dt=BF: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    B, T, Hq, Hk, d, page = 3, 8, 12, 2, 128, 16
    width = 188
    table = torch.randperm(B * width, generator=g, device="cuda").to(I32).view(B, width)
    q, kc, vc = r(B, T, Hq, d), r(B * width, page, Hk, d), r(B * width, page, Hk, d)
    kv = torch.tensor([3000, 17, 800], dtype=I32, device="cuda")
    logits, tokens = r(16, T, 4096), torch.randint(0, 4096, (16, T), generator=g, device="cuda", dtype=I32)
    n = 300
    k, v = r(B, T, Hk, d), r(B, T, Hk, d)
    slots = torch.randperm(page * B * width, generator=g, device="cuda")[: B * T].view(B, T)
    freq, mid, rows = r(64, dt=F32), i(B) + 100, i(B) + T
    plans = [(i(B), i(B), i(B, 4), torch.arange(40, dtype=I32, device="cuda"), i(1) + 40) for _ in range(5)]
    n_th = iter(range(5))
    x = dict(q=r(1, n, 2, 128), k=r(1, n, 2, 128), v=r(1, n, 4, 128), a=r(1, n, 4), b=r(1, n, 4), A_log=r(4, dt=F32), dt_bias=r(4, dt=F32))
    caches = [torch.zeros_like(kc), torch.zeros_like(vc)]
    return {"paged_attention": lambda **o: gdn.paged_attention(q, kc, vc, table, kv, **o),
            "accept": lambda **o: gdn.accept(logits, tokens, **o),
            "chunk_prefill": lambda **o: gdn.chunk_prefill(**x, **o),
            "rope_append": lambda **o: gdn.rope_append(q, k, v, freq, *caches, slots, kv_len=mid, q_len=rows, **o),
            # the tables are updated in place: each call has its own
            "kv_plan": lambda **o: gdn.kv_plan(*plans[next(n_th)], T, page, **o)}


@pytest.mark.parametrize("name", ["paged_attention", "accept", "chunk_prefill", "rope_append", "kv_plan"])
@pytest.mark.parametrize("handle", [False, True])
def test_stream_argument_beside_a_busy_current_stream(gdn, name, handle):
    call = _calls(gdn)[name]                         # (its inputs live as long as it does)
    side = torch.cuda.Stream()
    flat = lambda r: r if isinstance(r, tuple) else (r,)  # noqa: E731
    want = [t.clone() for t in flat(call())]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(4):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)             # a millisecond: the call below is still to come on the GPU
        got = flat(call(stream=side.cuda_stream if handle else side))
        # what the call dropped (its workspace) must not be among what the current stream is given now
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (64, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 22) for _ in range(8)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del junk, got
    # and its bytes come from that stream's pool
    assert any(s["stream"] == side.cuda_stream for s in torch.cuda.memory_snapshot())

"""The failure path of the bounded waits, on the GPU, without a fault: a wait on an mbarrier
that nothing completes, and the acceptance draw kernel's wait on a sequence flag that nothing
raises, each give up after their poll limit, report the wait-timeout bit in the status word
and return; the context stays usable (a verify call after them is still exact)."""
import pytest
import torch

from gated_deltanet_mixer_verify_b200.inputs import make_inputs, workload
from gdn_helpers import TOL, gpu_verify, oracle_verify, rel_err, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn(cuda_device):
    from gated_deltanet_mixer_verify_b200 import build, gdn as g
    build.build()
    return g


def test_bounded_wait_reports_timeout_and_context_survives(gdn):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.selftest_bounded_wait(status, polls=1024)
    torch.cuda.synchronize()
    assert int(status.item()) == 2
    # the context still computes: a verify call afterwards matches the oracle
    w = workload("batched_verify", B=2, seed=95)
    x = make_inputs(w)
    st2 = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = gpu_verify(gdn, to_dev(x), x["accept_len"].numpy(), status=st2)
    o_ref, S_ref, _ = oracle_verify(x, x["accept_len"].numpy())
    assert rel_err(o, o_ref) <= TOL and rel_err(S, S_ref) <= TOL and int(st2.item()) == 0


def test_accept_flag_wait_reports_timeout_and_context_survives(gdn):
    # The acceptance draw kernel alone, its sequence's flag never raised: every CTA gives up,
    # reports the wait-timeout bit and writes next token 0; nothing else is touched.
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nt = torch.full((1,), 12345, dtype=torch.int32, device="cuda")
    gdn.selftest_accept_wait(status, nt, polls=256)
    torch.cuda.synchronize()
    assert int(status.item()) == 2 and int(nt.item()) == 0
    # the context still computes: a verify call afterwards matches the oracle
    w = workload("batched_verify", B=2, seed=96)
    x = make_inputs(w)
    st2 = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = gpu_verify(gdn, to_dev(x), x["accept_len"].numpy(), status=st2)
    o_ref, S_ref, _ = oracle_verify(x, x["accept_len"].numpy())
    assert rel_err(o, o_ref) <= TOL and rel_err(S, S_ref) <= TOL and int(st2.item()) == 0


@pytest.mark.parametrize("d,Hk,T,lens", [(64, 2, 8, [40000, 300, 9000, 1]), (128, 4, 8, [700] * 60), (256, 2, 16, [5000, 17, 20000])])
def test_attention_waits_report_timeout_and_write_nothing_by_halves(gdn, d, Hk, T, lens):
    # The tensor-memory attention kernel with waits of a few polls only: some give up in some CTAs, all of them with
    # one poll. Every row of o and lse is then as it was, or as the call without a limit leaves it.
    g = torch.Generator(device="cuda").manual_seed(d)
    B, Hq, page = len(lens), 6 * Hk, 16
    width = max(-(-max(lens) // page), (1 << 23) // (B * Hk * d * page) + 1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    n = sum(-(-x // page) for x in lens)
    kc, vc, q = r(n, page, Hk, d), r(n, page, Hk, d), r(B, T, Hq, d)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(lens):
        m = -(-x // page)
        table[b, :m] = torch.arange(at, at + m)
        at += m
    table, kv = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want, want_lse = torch.empty_like(q), torch.empty(B, T, Hq, device="cuda")
    gdn.paged_attention(q, kc, vc, table, kv, o=want, lse=want_lse)
    ws = torch.full((gdn.paged_attention_workspace_bytes(B, T, Hq, Hk, d),), 255, dtype=torch.uint8, device="cuda")
    missed = 0
    for polls in (1, 2, 5, 20, 100, 1 << 20, 3, 50):
        o, lse = torch.full_like(q, 5.0), torch.full_like(want_lse, 5.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.selftest_attention_wait(q, kc, vc, table, kv, o, lse, ws, status, polls=polls)
        torch.cuda.synchronize()
        same = (o == want).all(-1) & (lse == want_lse)
        kept = (o == 5.0).all(-1) & (lse == 5.0)
        assert bool((same | kept).all()), polls
        assert int(status.item()) == (2 if bool(kept.any()) else 0) or (int(status.item()) == 2 and polls < (1 << 20)), polls
        if polls == 1:
            assert int(status.item()) == 2 and bool(kept.any())
        if polls == 1 << 20:
            assert bool(same.all()) and int(status.item()) == 0
        missed += int(kept.sum())
    assert missed > 0
    # and the context computes on
    o, lse = torch.empty_like(q), torch.empty_like(want_lse)
    gdn.paged_attention(q, kc, vc, table, kv, o=o, lse=lse, workspace=ws)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)

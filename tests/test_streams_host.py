"""Where the binding allocates what a call makes itself: on the stream that the call is launched on, not on the
current one, whose allocator would hand the same bytes out again while the kernels still run (no GPU needed: CPU
tensors, so every call ends at its refusal, which comes after the allocations)."""
import contextlib

import pytest
import torch

from gated_deltanet_mixer_verify_b200 import build as gbuild

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HANDLE = 0x7000


@pytest.fixture(scope="module")
def gdn():
    gbuild.build()
    from gated_deltanet_mixer_verify_b200 import gdn as g
    return g


def _mixer(T=8):
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    return dict(q=z(2, T, 2, 128), k=z(2, T, 2, 128), v=z(2, T, 4, 128), a=z(2, T, 4), b=z(2, T, 4), A_log=z(4, dt=F32),
                dt_bias=z(4, dt=F32))


def _state():
    return torch.zeros(2, 4, 128, 128)


def _calls():
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=I32)  # noqa: E731
    x = _mixer()
    heads = dict(q=z(2, 8, 6, 64), k_cache=z(5, 16, 2, 64), v_cache=z(5, 16, 2, 64))
    # name, arguments, tensors that the call makes
    return [("verify_step", dict(x, state_in=_state(), accept_len=i(2)), 1),
            ("commit_and_verify", dict(x, state=_state(), prev_stash=z(8, dt=F32), prev_accept_len=i(2), prev_T=8, accept_len=i(2)), 1),
            ("verify_step_gated", dict(x, state_in=_state(), state_out=_state(), accept_len=i(2), norm_z=x["v"], norm_w=z(128, dt=F32)), 1),
            ("gated_rmsnorm", dict(x=x["v"], z=x["v"], w=z(128, dt=F32)), 1),
            ("accept", dict(target=z(2, 8, 64), tokens=i(2, 8)), 3),
            ("short_conv", dict(q=x["q"], k=x["k"], v=x["v"], conv_w=z(1024, 4, dt=F32), hist_in=z(2, 3, 1024)), 3),
            ("decode_step", dict(_mixer(1), state=_state()), 1),
            ("chunk_prefill", x, 3),
            ("chunk_prefill_scan", dict(v=x["v"], workspace=z(64, dt=torch.uint8), H_k=2), 2),
            ("chunk_prefill_noalloc", x, 2),
            ("kv_plan", dict(seq_len=i(2), n_pages=i(2), block_table=i(2, 4), free_list=i(9), free_count=i(1), T=8, page_size=16), 3),
            ("rope_append", dict(heads, k=z(2, 8, 2, 64), v=z(2, 8, 2, 64), inv_freq=z(32, dt=F32),
                                 slot_map=torch.zeros(2, 8, dtype=torch.int64), kv_len=i(2), q_len=i(2)), 1),
            # (its workspace is made behind the output, and its device is refused behind both)
            ("paged_attention", dict(heads, block_table=i(2, 3), kv_len=i(2)), 2)]


@pytest.mark.parametrize("case", _calls(), ids=lambda c: c[0])
def test_own_tensors_are_made_on_the_launch_stream(gdn, monkeypatch, case):
    name, kw, made = case
    inside, where = [None], []

    @contextlib.contextmanager
    def on(stream):
        inside[0] = stream
        yield
        inside[0] = None

    def watch(real):
        def make(*a, **k):
            where.append(inside[0])
            return real(*a, **k)
        return make

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch, "empty", watch(torch.empty))
    monkeypatch.setattr(torch, "empty_like", watch(torch.empty_like))
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        getattr(gdn, name)(**kw, stream=HANDLE)
    assert where == [("external", HANDLE)] * made
    # without a stream the current one serves, as it is
    where.clear()
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        getattr(gdn, name)(**kw)
    assert where == [None] * made


def test_the_stream_that_a_handle_names(gdn, monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")

    class Other:                                   # another library's stream object
        cuda_stream = HANDLE

    assert gdn._torch_stream(Other(), None) == gdn._torch_stream(HANDLE, None) == ("external", HANDLE)
    assert gdn._torch_stream(0, None) == gdn._torch_stream(1, None) == "default"     # both are the legacy default stream

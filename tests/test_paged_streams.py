"""The streams that the paged-cache calls run on when one is given: torch
stream objects, raw handles, and the handles that name the default stream."""
import contextlib

import pytest
import torch

from nvfp4_block_scaled_22_b200 import binding as nb

DEV = "cuda"


class FakeStream:
    """In place of torch.cuda.Stream: a stream of device 0 unless said otherwise."""

    def __init__(self, name="given", index=0):
        self.name, self.device_index, self.device = name, index, torch.device("cuda", index)


@pytest.fixture
def made_current(monkeypatch):
    """The names of the streams that are made current, without a GPU."""
    seen = []

    @contextlib.contextmanager
    def current(stream):
        seen.append(stream.name)
        yield

    def external(handle, device=None):
        assert handle not in (0, 1), "torch takes a stream of its own pool for a null handle"
        return FakeStream(f"external {handle}", 0)

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream("default", 0))
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(nb, "_current_device", lambda: 0)
    return seen


@pytest.mark.parametrize("stream,name", [(0, "default"), (1, "default"), (2, "external 2"), (0x7F00, "external 32512"), (FakeStream(), "given")])
def test_the_stream_that_a_handle_names(made_current, stream, name):
    """0 is the legacy default stream in the C ABI, as 1 (cudaStreamLegacy) is."""
    with nb._switched(torch.device("cuda", 0), stream):
        pass
    assert made_current == [name]


def test_a_stream_of_another_device_is_refused(made_current):
    """Made current, it would leave the call on the tensors' own device's current stream."""
    with pytest.raises(ValueError, match="stream is not on cuda:0"):
        with nb._switched(torch.device("cuda", 0), FakeStream(index=1)):
            raise AssertionError("the call would have run")
    with nb._switched(torch.device("cuda"), FakeStream(index=0)):       # the current device
        pass
    assert made_current == ["given"]


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1])
def test_handle_of_the_default_stream_keeps_the_order_of_its_work(handle):
    """x, a slot and a page table are written on the default stream behind a
    wait of some milliseconds; calls given its handle from within another
    stream see what was written."""
    heads, dim, n = 2, 64, 16
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(dim), 64, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    new = torch.randn(n, heads, dim, device=DEV).bfloat16()
    kc, vc = (nb.NVFP4Tensor(torch.zeros(n, heads * dim // 2, dtype=torch.uint8, device=DEV), torch.zeros(n * heads * dim // 16, dtype=torch.uint8, device=DEV),
                             torch.full((1,), 448.0, device=DEV), n, heads * dim, nb.SF_LINEAR) for _ in range(2))
    pages, lens = torch.arange(n, dtype=torch.int32, device=DEV)[None], torch.full((1,), n, dtype=torch.int32, device=DEV)
    q = new[:1].clone()
    nb.default_workspace()
    want = nb.nvfp4_rope(new, pos, table)
    nb.nvfp4_kv_write(want, new, pos, kc, vc)
    rows = [t.clone() for t in nb.nvfp4_kv_read(kc, vc, pos)]
    o = nb.nvfp4_attention_decode_paged(q, kc, vc, heads, pages, lens, 1)
    for t in (kc, vc):
        t.codes.zero_()
        t.scales.zero_()
    x = torch.zeros_like(new)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                                        # 10 ms
    x.copy_(new)
    with torch.cuda.stream(torch.cuda.Stream()):
        y = nb.nvfp4_rope(x, pos, table, stream=handle)
        nb.nvfp4_kv_write(y, x, pos, kc, vc, stream=handle)
        got = nb.nvfp4_kv_read(kc, vc, pos, stream=handle)
        z = nb.nvfp4_attention_decode_paged(q, kc, vc, heads, pages, lens, 1, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1]) and torch.equal(z, o)
    assert nb.nvfp4_check_status() == 0


@pytest.mark.parametrize("capturing", [False, True])
def test_the_default_workspace_is_filled_before_it_is_handed_out(monkeypatch, capturing):
    """Its zeros are written on the stream of the first call; a later call on
    another stream is not ordered behind them.  Inside of a capture there is
    nothing to wait for."""
    done = []

    class Stream:
        def synchronize(self):
            assert done == ["filled on cuda:0"] and not nb._default_ws
            done.append("waited")

    monkeypatch.setattr(nb, "_default_ws", {})
    monkeypatch.setattr(nb, "Workspace", lambda device: done.append(f"filled on {device}") or object())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    ws = nb.default_workspace(torch.device("cuda", 0))
    assert done == ["filled on cuda:0"] + ["waited"] * (not capturing)
    assert nb.default_workspace(torch.device("cuda", 0)) is ws and len(done) == 2 - capturing


@pytest.mark.gpu
def test_an_error_recorded_behind_a_first_call_on_a_busy_stream_is_kept(monkeypatch):
    monkeypatch.setattr(nb, "_default_ws", {})
    table = nb.nvfp4_rope_table(nb.nvfp4_rope_inv_freq(64), 16, device=DEV)
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    good, bad = (torch.full((4,), p, dtype=torch.int32, device=DEV) for p in (3, 99))
    busy = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(20_000_000)                                    # 10 ms
        nb.nvfp4_rope(x, good, table)                                    # makes the default workspace here
    nb.nvfp4_rope(x, bad, table)
    torch.cuda.synchronize()
    assert nb.nvfp4_check_status() == 1
    assert nb.nvfp4_check_status() == 0

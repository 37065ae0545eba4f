"""How the bindings ask torch for the current stream and device: directly where torch has the calls,
by its public interface where it has not."""
import importlib.util
import sys

import pytest
import torch

import rht_bit_block_amd as U


def without_direct_calls(monkeypatch):
    """The bindings as they are imported by a torch that lacks the direct calls."""
    spec = importlib.util.spec_from_file_location("bindings_again", U.__file__, submodule_search_locations=list(U.__path__))
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, "bindings_again", module)
    with monkeypatch.context() as at_import:
        for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
            at_import.delattr(torch._C, name, raising=False)
        spec.loader.exec_module(module)
    return module


def test_public_calls_where_torch_has_no_others(monkeypatch):
    class Stream:
        def __init__(self, dev):
            self.cuda_stream = 1000 + dev

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    m = without_direct_calls(monkeypatch)
    assert m._raw_stream(2) == 1002 and m._current_device() == 3


@pytest.mark.gpu
def test_both_ways_are_the_same(monkeypatch):
    x = torch.randn(32, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    cfg = lambda m: m.make_cfg(U.UFP4_INT4, U.UFP4_RTNE, U.UFP4_SCALE_F32, 1, 32, 32, sign_seed=5)  # noqa: E731
    q, starts = x.view(32, 1, 64), torch.tensor([0, 32], dtype=torch.int32, device="cuda")
    want = U.ufp4_rht_quant(x, 0, cfg(U))[0].codes, U.ufp4_attn_fwd(q, q, q, starts)[0]
    torch.cuda.synchronize()
    m = without_direct_calls(monkeypatch)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert m._stream(x) == m._raw_stream(0) == side.cuda_stream == U._stream(x)
        got = m.ufp4_rht_quant(x, 0, cfg(m))[0].codes, m.ufp4_attn_fwd(q, q, q, starts)[0]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

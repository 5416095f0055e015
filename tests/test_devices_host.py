"""Calls whose tensors or stream are not of the current device are refused before anything is
launched (stand-ins for the tensors and the library: no GPU)."""
import types

import pytest
import torch

from gated_delta_rule_43_gb300 import inputs, kda
from tests import la_util as U


class On:
    """A CPU tensor that says it lives on a GPU."""

    def __init__(self, t, device):
        self._t, self._device = t, device

    is_cuda = True

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


class Library:
    """Takes every call, launches nothing."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                return 256
            self.launched.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(kda, "_lib", fake)
    monkeypatch.setattr(kda, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kda, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(kda, "_new",
                        lambda like, shape, dtype, stream: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0))
    kda._la_workspace_size.cache_clear()
    yield fake
    kda._la_workspace_size.cache_clear()


def every_call(device, stream=None):
    """Each entry point once, its tensors on `device`."""
    def on(*ts):
        return [On(t, device) for t in ts]
    q, k, v, g, cu, h0 = on(*U.make([5, 3], 4, 2, 32, 64, torch.float32))
    pos, freq = on(torch.zeros(8, dtype=torch.int32), torch.ones(16))
    i, = on(torch.arange(2, dtype=torch.int32))
    idx, = on(torch.arange(8, dtype=torch.int32))
    pool, live = on(torch.zeros(8, 4, 32, 64), torch.ones(8, dtype=torch.bool))
    kw = dict(stream=stream)
    yield lambda: kda.la_chunk_fwd(q, k, v, g, cu, h0, **kw)
    yield lambda: kda.la_decode_step(q, k, v, g, pool, **kw)
    yield lambda: kda.la_decode_step_indexed(q, k, v, g, pool, idx, **kw)
    yield lambda: kda.qk_norm_rope(q, k, pos, freq, **kw)
    yield lambda: kda.state_pool_copy(pool, i, i, **kw)
    yield lambda: kda.state_pool_compact(pool, live, **kw)


def delta_rule_calls(device):
    d = {n: On(t, device) if torch.is_tensor(t) else t
         for n, t in inputs.make_prefill([5, 3], H=2, dk=32, dv=32, dtype="f32", seed=1).items()}
    a = [d[n] for n in ("q", "k", "v", "z", "beta", "A_log")]
    state, = [On(torch.zeros(8, 2, 32, 32), device)]
    idx = On(torch.arange(8, dtype=torch.int32), device)
    yield lambda: kda.chunk_fwd(*a, d["cu_seqlens"])
    yield lambda: kda.chunk_fwd_segmented(*a, d["cu_seqlens"], segments=2)
    yield lambda: kda.decode_step(*a, state)
    yield lambda: kda.decode_step_indexed(*a, state, idx)
    yield lambda: kda.gate_cumsum(d["z"], d["A_log"], d["cu_seqlens"])
    yield lambda: kda.query_status(On(torch.zeros(256, dtype=torch.uint8), device))


def test_another_device_than_the_current_one(lib):
    for call in (*every_call(1), *delta_rule_calls(1)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert lib.launched == []


def test_a_stream_of_another_device(lib):
    stream = types.SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1))
    for call in every_call(0, stream):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call()
    assert lib.launched == []


def test_tensors_on_two_devices(lib):
    d = {n: On(t, 0) if torch.is_tensor(t) else t
         for n, t in inputs.make_prefill([5, 3], H=2, dk=32, dv=32, dtype="f32", seed=1).items()}
    d["k"] = On(d["k"]._t, 1)
    with pytest.raises(ValueError, match="one CUDA device"):
        kda.chunk_fwd(*(d[n] for n in ("q", "k", "v", "z", "beta", "A_log")), d["cu_seqlens"])
    assert lib.launched == []


def test_the_current_device_passes(lib):
    for call in (*every_call(0), *delta_rule_calls(0)):
        call()
    assert len(lib.launched) == 12

"""Which stream the cache operators' own buffers belong to: the one the call
runs on, whether it is given as a Stream or as a raw handle."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from kv_cache_early_art_b200 import build
from tests import cache_ref as ref


@pytest.fixture(scope="module")
def binding():
    build.build_library()
    from kv_cache_early_art_b200 import binding
    return binding


# ---- host: torch's stream calls replaced, any device ------------------------

class FakeStream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device = handle, device


@pytest.fixture
def streams(monkeypatch):
    """torch.cuda's streams as plain objects; `set` gets what was made current."""
    made = []
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0, device))

    @contextlib.contextmanager
    def stream(s):
        made.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    return made


CUDA0, CUDA1 = torch.device("cuda:0"), torch.device("cuda:1")


@pytest.mark.parametrize("given,handle", [(0, 0), (1, 0), (0x7f00, 0x7f00), (FakeStream(0x7f00, CUDA1), 0x7f00),
                                          (FakeStream(0, CUDA0), 0)])
def test_buffers_belong_to_the_given_stream_on_the_tensors_device(binding, streams, given, handle):
    """The default stream's handle, its other name, a raw handle with another
    device current, a Stream, and another device's default stream (whose handle
    the kernels take for their own device's)."""
    with binding._allocating(given, SimpleNamespace(is_cuda=True, device=CUDA1)):
        pass
    assert [(s.cuda_stream, s.device) for s in streams] == [(handle, CUDA1)]


def test_a_stream_with_cpu_tensors_is_refused(binding):
    z, i32 = torch.zeros, torch.int32
    with pytest.raises(ValueError):
        binding.art_decode_attention_split(z(1, 4, 64), z(9, 2, 16, 64), z(9, 2, 16, 64), z(1, 2, dtype=i32), z(1, dtype=i32),
                                           stream=0x7f00)


# ---- on the GPU -------------------------------------------------------------

def owner(address):
    """The stream whose memory the caching allocator gave out at an address."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["zero", "handle", "stream", "default"])
def test_owner_of_every_buffer(cuda_lib, binding, monkeypatch, how):
    """q_out, out, lse, the workspace, the new lengths and the kept rows, called while another stream is current."""
    art, dev, page, Hq, Hkv, d, n = cuda_lib, "cuda", 64, 8, 2, 128, 3000
    side = torch.cuda.Stream()
    given = {"zero": 0, "handle": side.cuda_stream, "stream": side, "default": torch.cuda.default_stream()}[how]
    want = 0 if how in ("zero", "default") else side.cuda_stream
    k, v, table = ref.paged([n], page, Hkv, d, "bf16", 1, stale=0.0, width=n // page + 2)
    g = torch.Generator().manual_seed(2)
    k, v, table = k.to(dev), v.to(dev), table.to(dev)
    q, kn, vn = (torch.randn(1, h, d, generator=g).to(dev, torch.bfloat16) for h in (Hq, Hkv, Hkv))
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    mass = torch.zeros(1, Hkv, table.shape[1] * page, device=dev)
    seen = {}
    run = binding._run

    def spy(name, stream, tensors, others, tail):
        seen[name] = [t.data_ptr() for t in others if t is not None and t.numel()]
        return run(name, stream, tensors, others, tail)

    monkeypatch.setattr(binding, "_run", spy)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        x = binding.art_rope_append(art.art_rope_init(d), q, kn, vn, k, v, table, lens, mass=mass, stream=given)
        o, e = binding.art_decode_attention_split(x, k, v, table, lens, mass=mass, stream=given)
        nl, kept = binding.art_cache_evict(k, v, table, lens, mass, 100, stream=given)
    torch.cuda.synchronize()
    workspace = seen["art_decode_attention_split"]
    assert len(workspace) == 1                       # long enough to need one
    assert {owner(p) for p in [t.data_ptr() for t in (x, o, e, nl, kept)] + workspace} == {want}

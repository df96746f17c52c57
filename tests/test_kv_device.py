"""Which device is current while the cache's binding calls the library, on the CPU: the library
and torch's device switch are stand-ins that note it."""
import contextlib
import types

import pytest
import torch


@pytest.fixture
def omq():
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


class Tensor:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, device, True
        n, st = 1, []
        for d in reversed(shape):
            st.insert(0, n)
            n *= d
        self.st, self.n = tuple(st), n

    def is_contiguous(self):
        return True

    def stride(self):
        return self.st

    def numel(self):
        return self.n

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("current,theirs", [(0, 1), (1, 0), (2, 2)])
def test_workspace_is_sized_under_the_tensors_device(omq, monkeypatch, current, theirs):
    now, seen = [current], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(omq, "_lib", types.SimpleNamespace(
        omq_kv_attn_workspace_bytes=lambda a: seen.append(("size", now[0])) or 0,
        omq_kv_attn=lambda a, ws, n, stream: seen.append(("attn", now[0], stream)) or 0))
    dev = torch.device("cuda", theirs)
    q = Tensor((3, 2, 128), torch.float16, dev)
    ints = lambda *s: Tensor(s, torch.int32, dev)  # noqa: E731
    pool = Tensor((4, 1, 1, 2304), torch.uint8, dev)
    out = omq.kv_attn(q, pool, ints(2, 2), ints(2), ints(3), 3, out=Tensor((3, 2, 128), torch.float16, dev))
    assert out.shape == q.shape and now == [current]
    assert seen == [("size", theirs), ("attn", theirs, 100 + theirs)]


class Entered(Exception):
    pass


@pytest.mark.parametrize("device,theirs", [("cuda", 1), (torch.device("cuda"), 1), ("cuda:1", 1), (torch.device("cuda", 0), 0)])
def test_rope_table_takes_the_stream_s_device(omq, monkeypatch, device, theirs):
    """A device without a number is the stream's, however it is written."""
    def stream_context(s):
        raise Entered(s.device)

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(Entered if theirs == 1 else ValueError):
        omq.rope_table(8, 64, device=device, stream=stream)

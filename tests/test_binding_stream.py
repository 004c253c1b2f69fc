"""The stream of a call that is given none: the current torch stream, asked for
at each call, by whichever query this torch has."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def test_the_query_follows_the_current_stream(m, monkeypatch):
    """On stand-ins for torch's queries (no GPU is asked)."""
    now = {"device": 0, (0): 11, (1): 22}
    monkeypatch.setattr(m, "_current_stream", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert m._stream(None) is None and m._current_stream is None          # asked again at the next call
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["device"])
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=now[now["device"]]))
    for raw in (lambda device: now[device], None):
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
        monkeypatch.setattr(m, "_current_stream", None)
        for device, handle in ((0, 11), (1, 22), (0, 33)):
            now["device"], now[device] = device, handle
            assert m._stream(None) == handle
    assert m._stream(44) == 44 and m._stream(types.SimpleNamespace(cuda_stream=55)) == 55


@pytest.mark.gpu
def test_the_query_agrees_with_torch(m):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")

    def agree():
        return (m._stream(None) or 0) == torch.cuda.current_stream().cuda_stream

    assert agree()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        with torch.cuda.stream(s):
            assert agree() and m._stream(None) == s.cuda_stream
            with torch.cuda.stream(side[0]):
                assert agree() and m._stream(None) == side[0].cuda_stream
            assert agree()
    x = torch.zeros(8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1)
        captured = m._stream(None), torch.cuda.current_stream().cuda_stream
    assert captured[0] == captured[1] != 0
    assert agree()

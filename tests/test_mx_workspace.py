"""Memory that a product makes for its launch stays its own until the launch is enqueued:
the foreign call releases the interpreter's lock, so that another thread may allocate, or
empty the allocator's cache, before that."""
import types
import weakref

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz


@pytest.mark.parametrize("grouped", [False, True])
def test_workspace_lives_until_the_launch(grouped, monkeypatch):
    """On the host: what was allocated is followed, the library is a stand-in."""
    made, seen = [], []

    def empty(*a, **k):
        t = real(*a, **k)
        made.append((t.data_ptr(), weakref.ref(t)))
        return t

    def launch(*args):
        space, size = args[-3:-1]
        seen.append([ref() is not None for at, ref in made if at == space])
        assert size == 4096
        return rz.RAZER_OK

    real, mx = torch.empty, rz.mx
    x, w = rz.MxTensor(4, 64, "cpu"), rz.MxTensor(8, 64, "cpu")
    x._index = w._index = 0
    stand_in = types.SimpleNamespace(razer_mx_gemm=launch, razer_mx_gemm_grouped=launch, razer_mx_workspace_bytes=lambda *a: 4096)
    monkeypatch.setattr(mx, "lib", lambda: stand_in)
    monkeypatch.setattr(mx, "_stream", lambda index: 0)
    monkeypatch.setattr(mx, "_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(mx, "_check_buffer", lambda *a: None)
    monkeypatch.setattr(torch, "empty", empty)
    if grouped:
        mx.razer_mx_gemm_grouped(x, w, torch.zeros(3, dtype=torch.int32))
    else:
        mx.razer_mx_gemm(x, w)
    assert seen == [[True]]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_workspace_is_not_handed_out_before_the_launch(monkeypatch):
    """An allocation in front of the launch gets other memory, and the product is right."""
    m, n, k = 300, 256, 16384
    x, w = (rz.razer_mx_quantize(torch.randn(r, k, device="cuda")) for r in (m, n))
    size = rz.razer_mx_workspace_bytes(m, n, k)
    assert size > 0
    want = rz.razer_mx_gemm(x, w)
    real, others = rz.lib(), []

    def launch(*args):
        others.append(torch.zeros(size, dtype=torch.uint8, device="cuda"))
        assert others[-1].data_ptr() != args[-3] and args[-2] == size
        return real.razer_mx_gemm(*args)

    monkeypatch.setattr(rz.mx, "lib", lambda: types.SimpleNamespace(razer_mx_gemm=launch))
    for _ in range(3):
        assert torch.equal(rz.razer_mx_gemm(x, w), want)
    assert all((t == 0).all() for t in others)

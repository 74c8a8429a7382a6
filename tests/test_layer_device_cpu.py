"""The layers' launches on CPU, with the library calls recorded: the layer's
device is current for each, whichever was."""
import pytest

torch = pytest.importorskip("torch")

import block_scaled_fp4_sigmoid_gb300 as fm  # noqa: E402
from block_scaled_fp4_sigmoid_gb300 import layer as L  # noqa: E402


class Gpu1:
    """A device object of index 1 on which allocations land in host memory."""
    index, type = 1, "cuda"


@pytest.fixture
def seen(monkeypatch):
    current, log = [0], []

    class device:
        def __init__(self, d):
            self.d = getattr(d, "index", d)

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *exc):
            current[0] = self.before

    class stream:
        cuda_stream = 0

    empty, zeros = torch.empty, torch.zeros
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: stream)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    for name in ("forward", "forward_cols", "forward_w8a8", "forward_nvfp4_emulated", "check_scales", "get_status",
                 "pack_scales", "pack_weights", "pack_gateup_scales", "pack_gateup_weights", "mxfp4_to_fp8_rowscale"):
        monkeypatch.setattr(L, name, lambda *a, _n=name: (log.append((_n, current[0])), (0, 0))[1])
    for name in ("packed_weights_bytes", "packed_scales_bytes", "emulation_workspace_size", "workspace_size"):
        monkeypatch.setattr(L, name, lambda *a: 256)
    monkeypatch.setattr(L, "workspace_layout", lambda d: None)
    return log


def moe_layer(fmt):
    """A layer of few experts whose device says GPU 1."""
    E, H, I, T = 2, 256, 128, 4
    blk = 16 if fmt == fm.NVFP4 else 32
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731

    class Held(torch.Tensor):
        device = Gpu1

        def contiguous(self):
            return self

    layer = L.MoELayer(fm.make_dims(T, H, I, E, 2, fmt=fmt), u8(E, 2 * I, H // 2).as_subclass(Held), u8(E, 2 * I, H // blk),
                       u8(E, H, I // 2), u8(E, H, I // blk), torch.zeros((E, H), dtype=torch.bfloat16), torch.zeros(E),
                       *([torch.ones(E), torch.ones(E)] if fmt == fm.NVFP4 else []))
    return layer, torch.zeros((T, H), dtype=torch.bfloat16)


def test_every_launch_of_a_layer_has_its_device_current(seen):
    layer, x = moe_layer(fm.MXFP4)
    layer.forward(x)
    layer.forward_cols(x, 0, 256)
    L.W8A8Layer(layer).forward(x)
    nv, x = moe_layer(fm.NVFP4)
    nv.forward_emulated(x)
    names = {n for n, _ in seen}
    assert {"forward", "forward_cols", "forward_w8a8", "forward_nvfp4_emulated", "check_scales", "mxfp4_to_fp8_rowscale",
            "pack_gateup_weights", "pack_gateup_scales", "get_status"} <= names
    assert {d for _, d in seen} == {1}, sorted({(n, d) for n, d in seen if d != 1})
    assert torch.cuda.current_device() == 0

"""The tensor functions of the block-scaled FP8 operators up to the launch, on
CPU tensors: the library calls are replaced by recorders and the device index
of CPU tensors (-1) stands for a GPU other than the current one."""
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_sigmoid_gb300 import build  # noqa: E402

CALLS = ("_add_rmsnorm", "_swiglu", "_linear", "_experts", "_route")


class Launches:
    """What would have been launched: the call's name, its arguments and the current device."""

    def __init__(self, current):
        self.current, self.seen = current, []

    def record(self, name):
        return lambda *args: self.seen.append((name, args, self.current))


@pytest.fixture
def fb(monkeypatch):
    build.build_library()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    monkeypatch.setattr(fp8_block, "_device", lambda t: t.get_device())
    monkeypatch.setattr(fp8_block, "_stream", lambda device: 1000 + device)
    return fp8_block


@pytest.fixture
def launches(fb, monkeypatch):
    """Current device 0; torch.cuda.device(d) makes d current while it lasts."""
    rec = Launches(0)

    class device:
        def __init__(self, d):
            self.d = d if isinstance(d, int) else d.index

        def __enter__(self):
            self.before, rec.current = rec.current, self.d

        def __exit__(self, *exc):
            rec.current = self.before

    monkeypatch.setattr(fb, "_current_device", lambda: rec.current, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: rec.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in CALLS:
        monkeypatch.setattr(fb, name, rec.record(name))
    return rec


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(shape)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def expert_args(T=2, H=256, I=128, E=4, k=2):
    return [u8(T, H), f32(T, H // 128), torch.zeros((T, k), dtype=torch.int32), f32(T, k), u8(E, 2 * I, H),
            f32(E, 2 * I // 128, H // 128), u8(E, H, I), f32(E, H // 128, I // 128)]


def linear_args(T=4, K=256, N=128):
    return [u8(T, K), f32(T, K // 128), u8(N, K), f32(-(-N // 128), K // 128)]


def call_all(fb):
    fb.add_rmsnorm_fp8(bf16(3, 256), None, bf16(256), 1e-6)
    fb.swiglu_fp8(bf16(3, 512))
    fb.linear_fp8_block(*linear_args())
    fb.experts_fp8_block(*expert_args(), out=bf16(2, 256))


@pytest.mark.parametrize("current", [0, -1])
def test_every_launch_has_its_tensors_device_current(fb, launches, current):
    """A launch goes to the current device, and the default stream's handle is the same number on
    every device: with the tensors' device not current it would run elsewhere on their addresses."""
    launches.current = current
    call_all(fb)
    assert [n for n, _, _ in launches.seen] == ["_add_rmsnorm", "_swiglu", "_linear", "_experts"]
    for name, args, device in launches.seen:
        assert device == -1, name
        assert args[-1] == 999, name  # the stream of that device
    assert launches.current == current


def moe(fb, T=2, H=256, I=128, E=4, k=2, **kw):
    import block_scaled_fp4_sigmoid_gb300 as fm
    dims = fm.make_dims(T, H, I, E, k, fmt=fm.FP8)
    return fb.Fp8BlockMoE(dims, bf16(H), bf16(E, H), f32(E), *expert_args(T, H, I, E, k)[4:], **kw)


def test_the_router_refuses_rows_of_another_device_than_its_weights(fb, launches, monkeypatch):
    layer = moe(fb)
    y = bf16(2, 256)
    assert layer.route(y)[0].shape == (2, 2)

    class Elsewhere:
        """y as a tensor of device 3."""
        shape, dtype, device = y.shape, y.dtype, "cuda:3"
        get_device, is_contiguous, data_ptr = (lambda self: 3), (lambda self: True), (lambda self: 64)

    with pytest.raises(ValueError, match="y: "):
        layer.route(Elsewhere())
    assert len(launches.seen) == 1


class OnHost:
    """A CPU workspace, for calls whose tensors' device (-1 here) would be a GPU."""
    dtype, shape = torch.uint8, torch.Size([1 << 20])
    get_device, is_contiguous, data_ptr = (lambda self: -2), (lambda self: True), (lambda self: 64)
    device, stride, numel, dim = "cpu", (lambda self: (1,)), (lambda self: 1 << 20), (lambda self: 1)


BAD_WORKSPACES = {
    "on another device": lambda: OnHost(),
    "expanded from one byte": lambda: u8(1).expand(1 << 20),
    "every second byte": lambda: u8(1 << 20)[::2],
    "of another type": lambda: torch.zeros(1 << 20, dtype=torch.int32),
}


@pytest.mark.parametrize("kind", BAD_WORKSPACES)
def test_workspaces_that_do_not_hold_their_bytes_are_refused(fb, launches, kind):
    """The kernels write to the workspace: one on the host, or with fewer bytes behind it than it
    counts, is written past its end."""
    ws = BAD_WORKSPACES[kind]()
    with pytest.raises(ValueError, match="ws: "):
        fb.linear_fp8_block(*linear_args(), ws=ws)
    with pytest.raises(ValueError, match="ws: "):
        fb.experts_fp8_block(*expert_args(), out=bf16(2, 256), ws=ws)
    assert not launches.seen


def test_workspaces_of_any_shape_are_taken(fb, launches):
    for ws in (u8(1 << 16), u8(256, 256), u8(1 << 17)[256:]):
        fb.linear_fp8_block(*linear_args(), ws=ws)
        fb.experts_fp8_block(*expert_args(), out=bf16(2, 256), ws=ws)
        for name, args, _ in launches.seen[-2:]:
            assert args[-3:-1] == (ws.data_ptr(), ws.numel()), name


def test_a_layer_object_keeps_nothing_that_its_calls_write(fb, launches, monkeypatch):
    """Two streams may call one layer: each call's scratch is its own, from the allocator."""
    monkeypatch.setattr(fb, "_out", lambda name, t, shape, dtypes, device: torch.empty(shape, dtype=dtypes[0]))
    layer = moe(fb)
    layer.forward(bf16(2, 256))
    kept = [t for v in vars(layer).values() for t in (v if isinstance(v, tuple) else [v]) if torch.is_tensor(t)]
    weights = [layer.gamma, layer.w_router, layer.bias, *layer.weights]
    scratch = [a[-3] for n, a, _ in launches.seen if n in ("_route", "_experts")]
    assert len(scratch) == 2
    for t in kept:
        inside = [p for p in scratch if t.data_ptr() <= p < t.data_ptr() + t.numel() * t.element_size()]
        assert not inside or any(t is w for w in weights)
    with pytest.raises(Exception, match="UNSUPPORTED|unsupported"):
        moe(fb, T=17)  # refused when the layer is made, as before


def test_an_empty_product_leaves_a_clear_status(fb, launches):
    """A call clears the status word of its workspace, one without tokens as well."""
    ws = torch.full((256,), 0xA5, dtype=torch.uint8)
    out = fb.linear_fp8_block(*linear_args(T=0), out=bf16(0, 128), ws=ws)
    assert out.shape == (0, 128) and not launches.seen
    assert not ws[:64].any() and bool((ws[64:] == 0xA5).all())

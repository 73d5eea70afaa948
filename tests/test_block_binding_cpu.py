"""The Python path of the MoE block's binding without a GPU: stand-ins for CUDA tensors, streams and
the library, so that what a call allocates where, and what it hands over, can be looked at."""

import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
import moe_lora_virtual_gb300 as mol  # noqa: E402
from moe_lora_virtual_gb300 import block  # noqa: E402

bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32


class Cuda(torch.Tensor):
    """A host tensor that says that it is on the GPU."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return getattr(self, "on", 0)


def cuda(*shape, dtype=bf16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Cuda)


class Stream:
    """A stream that is only a handle (nothing is created)."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def binding(monkeypatch):
    """The calls that reach the library, and (stream, shape) of what is allocated."""
    seen = SimpleNamespace(calls=[], made=[], at=None)

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.calls.append((name, args))
                return {"mol_moe_workspace_bytes": 4096, "mol_workspace_bytes": 4096,
                        "mol_align_capacity": 64}.get(name, 0)
            return call

    @contextlib.contextmanager
    def on(stream):
        before, seen.at = seen.at, stream
        try:
            yield
        finally:
            seen.at = before

    real = torch.empty

    def empty(shape, *more, dtype=None, device=None):
        shape = (shape, *more) if isinstance(shape, int) else tuple(shape)
        seen.made.append((seen.at, shape))
        return real(shape, dtype=dtype).as_subclass(Cuda)

    monkeypatch.setattr(block, "_native", None)
    monkeypatch.setattr(mol, "_lib", Library())
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return seen


def calls(stream):
    """Every call of the block with nothing passed in that it would allocate."""
    T, k, E, H, I = 5, 2, 4, 64, 32
    x, ids, w = cuda(T, H), cuda(T, k, dtype=i32), cuda(T, k, dtype=f32)
    gu, dn = cuda(E, 2 * I, H), cuda(E, H, I)
    head = mol.W4(cuda(7, 128, dtype=torch.uint8), cuda(7, 8), H, 32)
    return {
        "norm": (lambda: mol.mol_block_norm(x, x, cuda(H), stream=stream), 2),
        "route": (lambda: mol.mol_moe_route(cuda(T, E, dtype=f32), k, stream=stream), 2),
        "gate_up": (lambda: mol.mol_moe_gate_up(x, ids, gu, stream=stream), 1),
        "down": (lambda: mol.mol_moe_down(cuda(T * k, I), ids, w, dn, stream=stream), 2),
        "forward": (lambda: mol.mol_moe_forward(x, ids, w, gu, dn, stream=stream), 3),
        "linear": (lambda: mol.mol_w4_linear(x, head, stream=stream), 1),
    }


NAMES = ["norm", "route", "gate_up", "down", "forward", "linear"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_and_scratch_are_the_streams_own(binding, name):
    """Memory of the current stream would be handed out again, or still be in use there, while the
    kernels on the call's stream write it."""
    side = Stream(0x1230)
    call, tensors = calls(side)[name]
    call()
    assert len(binding.made) == tensors
    assert all(at is side for at, _ in binding.made), binding.made
    assert binding.calls[-1][1][-1] == 0x1230 and binding.at is None


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_the_current_one_is_used(binding, name, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x77)
    call, tensors = calls(None)[name]
    call()
    assert [at for at, _ in binding.made] == [None] * tensors
    assert binding.calls[-1][1][-1] == 0x77


def test_raw_stream_handles(binding, monkeypatch):
    """A handle as an integer: the stream itself; 0 and 1 name the default stream."""
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: made.append(raw) or "external")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    for handle, stream in ((0, "default"), (1, "default"), (0x5550, "external")):
        binding.made.clear()
        calls(handle)["forward"][0]()
        assert [at for at, _ in binding.made] == [stream] * 3
        assert binding.calls[-1][1][-1] == handle
    assert made == [0x5550] * 3


@pytest.mark.parametrize("group", [0, 32])
def test_an_odd_number_of_gate_and_up_rows_is_refused(binding, group):
    """17 rows are no gate and up halves: the second expert's would be read one row too early."""
    T, k, E, H = 5, 2, 4, 64
    gu = cuda(E, 17, H)
    if group:
        gu = mol.W4(cuda(E, 17, 128, dtype=torch.uint8), cuda(E, 17, 256 // group), H, group)
    x, ids = cuda(T, H), cuda(T, k, dtype=i32)
    with pytest.raises(ValueError):
        mol.mol_moe_gate_up(x, ids, gu, stream=Stream(0))
    with pytest.raises(ValueError):
        mol.mol_moe_forward(x, ids, cuda(T, k, dtype=f32), gu, cuda(E, H, 8), stream=Stream(0))
    assert not [c for c in binding.calls if c[0] != "mol_moe_workspace_bytes"]


@pytest.mark.parametrize("stream", [None, Stream(0x40)])
def test_operands_on_another_device_are_refused(binding, stream, monkeypatch):
    """Each operand in turn on a device that is not the current one: nothing is enqueued."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x77)
    T, k, E, H, I = 40, 2, 4, 64, 32
    x, y, vec, ids = cuda(T, H), cuda(T, H), cuda(H), cuda(T, k, dtype=i32)
    w, gu, dn = cuda(T, k, dtype=f32), cuda(E, 2 * I, H), cuda(E, H, I)
    q, s = cuda(7, 128, dtype=torch.uint8), cuda(7, 8)
    act, dgu, ddn = cuda(T * k, I), cuda(T * k, 2 * I), cuda(T * k, H)
    out, ws = cuda(T, H), cuda(4096, dtype=torch.uint8)
    logits, out7 = cuda(T, E, dtype=f32), cuda(T, 7)

    def norm(x, y, v, p, gate, out, normed):
        mol.mol_block_norm(x, y, v, post_weight=p, gate=gate, residual_out=out, normed=normed,
                           stream=stream)

    def gate_up(x, ids, gu, delta, act):
        mol.mol_moe_gate_up(x, ids, gu, act=act, delta=delta, stream=stream)

    def down(act, ids, w, dn, delta, out, ws):
        mol.mol_moe_down(act, ids, w, dn, out=out, delta=delta, workspace=ws, stream=stream)

    def forward(x, ids, w, gu, dn, out, act, ws):
        mol.mol_moe_forward(x, ids, w, gu, dn, out=out, act=act, workspace=ws, stream=stream)

    def route(logits, ids, w):
        mol.mol_moe_route(logits, k, topk_ids=ids, topk_weights=w, stream=stream)

    def linear(x, q, s, out):
        mol.mol_w4_linear(x, mol.W4(q, s, H, 32), out=out, stream=stream)

    for call, operands in [(norm, (x, y, vec, cuda(H), cuda(T, H), out, cuda(T, H))),
                           (route, (logits, ids, w)), (gate_up, (x, ids, gu, dgu, act)),
                           (down, (act, ids, w, dn, ddn, out, ws)),
                           (forward, (x, ids, w, gu, dn, out, act, ws)), (linear, (x, q, s, out7))]:
        call(*operands)  # (all on the current device)
        for t in operands:
            binding.calls.clear()
            t.on = 1
            with pytest.raises(ValueError, match="current device"):
                call(*operands)
            del t.on
            assert not [c for c in binding.calls if c[0] != "mol_moe_workspace_bytes"]


def test_calls_of_the_lora_path_allocate_on_their_stream(binding, monkeypatch):
    """The routing buffers, the align's workspace, copies that make ids contiguous: as above."""
    side = Stream(0x1230)
    real = torch.Tensor.contiguous
    copies = []
    monkeypatch.setattr(Cuda, "contiguous", lambda self: copies.append(binding.at) or real(self))
    monkeypatch.setattr(torch, "empty_like", lambda t: torch.empty(t.shape, dtype=t.dtype))
    ids, lora = cuda(5, 4, dtype=i32)[:, :2], cuda(5, dtype=i32)
    vid = mol.mol_virtual_topk(ids, lora, 8, 4, stream=side)
    assert copies == [side, side] and [at for at, _ in binding.made] == [side]
    for align in (mol.mol_align_block_size, mol.mol_align_block_size_noalloc):
        binding.made.clear()
        routing = align(vid, 32, 16, stream=side)
        assert len(binding.made) >= 3 and all(at is side for at, _ in binding.made)
    binding.made.clear()
    mol.mol_lora_shrink(cuda(5, 64), 2, cuda(32, 8, 64), 1, routing, stream=side)
    mol.mol_token_lora_ids(cuda(2, dtype=i32), cuda(3, dtype=i32), 5, 4, stream=side)
    assert [at for at, _ in binding.made] == [side, side] and binding.at is None


@pytest.mark.parametrize("dtype", [f32, bf16, torch.complex64])
def test_pack_refuses_what_is_no_integer(dtype):
    """3.7 would be packed as 3."""
    with pytest.raises(TypeError):
        mol.w4_pack(torch.full((2, 64), 3.7).to(dtype), torch.ones(2, 2), 32)
    q = torch.full((2, 64), 3, dtype=torch.int16)
    assert torch.equal(mol.w4_unpack(mol.w4_pack(q, torch.ones(2, 2), 32)), torch.full((2, 64), -5.0))


@pytest.mark.parametrize("low,high,step", [(-8.0, 7.0, 1.0), (-8.5, 7.0, 1.0625), (-7.5, 7.0, 1.0), (-1.0, 14.0, 2.0)])
def test_quantize_steps(low, high, step):
    """The least step that keeps a group's values within -8 and 7 of them."""
    w = torch.linspace(low, high, 64).unsqueeze(0)
    p = mol.w4_quantize(w, 64)
    assert p.scales[0, 0].item() == step
    assert bool(((mol.w4_unpack(p) - w).abs() <= step / 2).all())

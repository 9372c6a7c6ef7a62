"""What the binding of the operators around the block hands to the library: workspaces, devices, sizes. Needs no GPU."""
import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw


class _OnGpu:
    """Stands for a contiguous GPU tensor, with an address that is never read."""

    def __init__(self, shape, dtype=torch.float32, index=0, contiguous=True):
        self.shape, self.dtype, self.index, self.contiguous = torch.Size(shape), dtype, index, contiguous
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x100000


def test_workspace_has_to_be_device_memory_in_one_piece():
    """Its size is what the library is told: a host tensor's address, or the bytes that an expanded or strided tensor
    does not hold, would be written by a kernel."""
    x = _OnGpu((4, 64))
    with pytest.raises(ValueError, match="ws must be on the GPU"):
        tw._workspace(torch.empty(4096, dtype=torch.uint8), 1024, x, None)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        tw._workspace(_OnGpu((4096,), torch.uint8, contiguous=False), 1024, x, None)
    with pytest.raises(ValueError, match="ws must be on cuda:0"):
        tw._workspace(_OnGpu((4096,), torch.uint8, index=1), 1024, x, None)
    ws = _OnGpu((4096,), torch.uint8)
    assert tw._workspace(ws, 1024, x, None)[:2] == (0x100000, 4096)
    assert tw._workspace(None, 0, x, None)[:2] == (None, 0)


class _Library:
    """Stands for the library: notes which calls are made, and on which current device and stream."""

    def __init__(self, current):
        self.current, self.calls = current, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current[0], args[-1]))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    """The binding on a machine of two GPUs, device 0 current, whose current streams are 1000 and 1001."""
    current = [0]

    class _Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    made = _Library(current)
    monkeypatch.setattr(tw, "lib", lambda: made)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    return made


U8, F32, BF = torch.uint8, torch.float32, torch.bfloat16


def _calls():
    """(function, its tensors by name) for every operator; the tensors are made on the device index given."""
    def t(*shape, dtype=F32):
        return lambda index: _OnGpu(shape, dtype, index)

    rows, cols, units = 4, 64, 8
    mx_x = dict(codes=t(rows, 64, dtype=U8), scales=t(rows, 16, dtype=U8))
    mx_w = dict(w_codes=t(units, 64, dtype=U8), w_scales=t(units, 16, dtype=U8))
    return [
        (lambda v, **k: tw.add_rms_norm(v["residual"], v["weight"], delta=v["delta"],
                                        out=[v[n] for n in ("r", "o", "q", "s", "rstd")], **k),
         dict(residual=t(rows, cols), weight=t(cols), delta=t(rows, cols, dtype=BF), r=t(rows, cols), o=t(rows, cols),
              q=t(rows, cols, dtype=U8), s=t(rows), rstd=t(rows))),
        (lambda v, **k: tw.add_rms_norm_bwd(v["d_out"], v["residual"], v["rstd"], v["weight"], v["d_residual"],
                                            out=(v["dr"], v["dw"]), ws=v["ws"], **k),
         dict(d_out=t(rows, cols), residual=t(rows, cols), rstd=t(rows), weight=t(cols), d_residual=t(rows, cols),
              dr=t(rows, cols), dw=t(cols), ws=t(64, dtype=U8))),
        (lambda v, **k: tw.quantize_mx4(v["a"], out=(v["codes"], v["scales"]), **k), dict(a=t(rows, cols), **mx_x)),
        (lambda v, **k: tw.dequantize_mx4(v["codes"], v["scales"], cols, out=v["out"], **k), dict(out=t(rows, cols), **mx_x)),
        (lambda v, **k: tw.matmul_mx4(v["codes"], v["scales"], v["w_codes"], v["w_scales"], cols, out=v["y"], ws=v["ws"],
                                      **k), dict(y=t(rows, units), ws=t(64, dtype=U8), **mx_x, **mx_w)),
        (lambda v, **k: tw.linear_mx4(v["x"], v["w_codes"], v["w_scales"], out=v["y"], ws=v["ws"], **k),
         dict(x=t(rows, cols), y=t(rows, units), ws=t(64, dtype=U8), **mx_w)),
    ]


@pytest.mark.parametrize("which", range(6))
def test_tensors_of_different_devices_are_refused(which, library):
    call, tensors = _calls()[which]
    call({n: make(0) for n, make in tensors.items()})
    assert len(library.calls) == 1
    for other in tensors:
        with pytest.raises(ValueError, match="must be on cuda:"):
            call({n: make(1 if n == other else 0) for n, make in tensors.items()})
    assert len(library.calls) == 1


@pytest.mark.parametrize("which", range(6))
def test_calls_run_on_the_device_of_their_tensors(which, library):
    """A launch goes to the current device, whatever its stream's: that of the tensors has to be current."""
    call, tensors = _calls()[which]
    for index in (0, 1):
        call({n: make(index) for n, make in tensors.items()})
        assert library.calls[-1][1:] == (index, 1000 + index)
        assert library.current == [0]  # the caller's device is left as it was


class _Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


@pytest.mark.parametrize("which", range(6))
def test_a_stream_of_another_device_is_refused(which, library):
    call, tensors = _calls()[which]
    call({n: make(1) for n, make in tensors.items()}, stream=_Stream(1))
    assert library.calls[-1][1:] == (1, 77)
    with pytest.raises(ValueError, match="stream"):
        call({n: make(1) for n, make in tensors.items()}, stream=_Stream(0))
    assert len(library.calls) == 1


def test_serving_block_runs_on_the_device_of_its_buffers(library):
    """All launches of a forward, those of the gate and the projections among them, go to the device of the buffers."""
    class _Serve(tw.TwellServe):
        def __init__(self, gate, index):
            N, D, F = 4, 64, 128
            self.dims, self.gate, self.eps, self.stream_dtype = tw.make_dims(N, D, F, 64, 64), gate, 1e-6, BF
            make = lambda *shape, dtype=F32: _OnGpu(shape, dtype, index)  # noqa: E731
            self.x, self.y, self.g, self.ws_gate = make(N, D, dtype=BF), make(N, D), make(N, F), make(64, dtype=U8)
            self.x_q, self.x_scale = (make(N, D, dtype=U8), make(N)) if gate == "fp8" else (None, None)
            self.pack, self.ws_fwd = None, make(64, dtype=U8)

    seen = []
    note = lambda *a, **k: seen.append(library.current[0])  # noqa: E731
    with pytest.MonkeyPatch.context() as mp:
        for name in ("ffn_forward", "ffn_forward_fp8", "pack_preact", "ffn_fwd"):
            mp.setattr(tw, name, note)
        for index in (0, 1):
            make = lambda *shape, dtype=F32: _OnGpu(shape, dtype, index)  # noqa: E731
            gates = {"bf16": make(128, 64, dtype=BF), "fp8": (make(128, 64, dtype=U8), make(128)),
                     "mx4": (make(128, 64, dtype=U8), make(128, 16, dtype=U8))}
            for gate, w in gates.items():
                first, before = len(seen), len(library.calls)
                up = make(128, 64, dtype=BF)
                _Serve(gate, index).forward(make(4, 64, dtype=BF), make(4, 64), make(64), w, up, up, make(4))
                assert len(seen) > first and all(i == index for i in seen[first:])
                assert [c[1] for c in library.calls[before:]] == [index] * (2 if gate == "mx4" else 1)
                with pytest.raises(ValueError, match="must be on cuda:"):
                    _Serve(gate, 1 - index).forward(make(4, 64, dtype=BF), make(4, 64), make(64), w, up, up, make(4))
    assert library.current == [0]


def test_sizes_beyond_32_bits_are_refused(library):
    """The library takes columns and units as 32-bit numbers; 2^32 + 64 of them must not pass for 64."""
    far = (1 << 32) + 64
    t = lambda *shape, dtype=F32: _OnGpu(shape, dtype)  # noqa: E731
    mx = lambda rows, cols: [t(*shape, dtype=U8) for shape in tw.mx4_shapes(rows, cols)]  # noqa: E731
    long, short, y, ws = mx(2, far), mx(2, 64), t(2, 2), t(64, dtype=U8)
    norm = [t(2, far), t(2, far), None, None, t(2)]
    for call in (lambda: tw.add_rms_norm(t(2, far), t(far), out=norm),
                 lambda: tw.add_rms_norm_bwd(t(2, far), t(2, far), t(2), t(far), out=(t(2, far), t(far)), ws=ws),
                 lambda: tw.quantize_mx4(t(2, far), out=long),
                 lambda: tw.dequantize_mx4(*long, far, out=t(2, far)),
                 lambda: tw.matmul_mx4(*long, *long, far, out=y, ws=ws),
                 lambda: tw.matmul_mx4(*short, *mx(far, 64), 64, out=t(2, far), ws=ws),
                 lambda: tw.linear_mx4(t(2, far), *long, out=y, ws=ws),
                 lambda: tw.linear_mx4(t(2, 64), *mx(far, 64), out=t(2, far), ws=ws)):
        with pytest.raises(tw.TwellError, match="UNSUPPORTED"):
            call()
    assert not library.calls


def test_workspaces_of_sizes_beyond_32_bits_are_refused():
    far = (1 << 32) + 64
    for call in (lambda: tw.add_rms_norm_bwd_ws(600, far), lambda: tw.matmul_mx4_ws(100, far, 64),
                 lambda: tw.matmul_mx4_ws(100, 64, far), lambda: tw.linear_mx4_ws(100, far, 64),
                 lambda: tw.linear_mx4_ws(100, 64, far)):
        with pytest.raises(tw.TwellError, match="UNSUPPORTED"):
            call()

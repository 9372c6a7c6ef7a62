"""The operators around the block as programs use them: a captured step that adds its own y, views that begin
anywhere."""
from __future__ import annotations

import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.mark.parametrize("gate", ["bf16", "fp8", "mx4"])
def test_capture_keeps_the_pending_delta(gate):
    """y is the delta of the next call: recording that call neither uses y up nor changes it, and every replay adds the
    y of the one before, as a chain of eager calls does."""
    require_gpu()
    N, D, F = 4, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dims = tw.make_dims(N, D, F, 64, 64, 0, 8, 0)
    w = (rnd(F, D) / D ** 0.5).to(BF)
    w = {"bf16": lambda: w, "fp8": lambda: tw.quantize_e4m3(w), "mx4": lambda: tw.quantize_mx4(w)}[gate]()
    weights = ((1 + 0.2 * rnd(D)).to(BF), w, (rnd(F, D) / D ** 0.5).to(BF), (rnd(F, D) / F ** 0.5).to(BF),
               torch.full((N,), 1.15, device="cuda"))
    stream, delta = rnd(N, D).to(BF), rnd(N, D)
    want_stream = stream.clone()
    serve, eager = tw.TwellServe(dims, gate, EPS), tw.TwellServe(dims, gate, EPS)
    y, want = serve.forward(stream, delta, *weights), eager.forward(want_stream, delta, *weights)
    graph = serve.capture(stream, y, *weights)
    torch.cuda.synchronize()
    assert torch.equal(stream, want_stream) and torch.equal(y, want)  # nothing has run yet
    for _ in range(4):
        graph.replay()
        want = eager.forward(want_stream, want, *weights)
        torch.cuda.synchronize()
        assert torch.equal(stream, want_stream) and torch.equal(y, want)

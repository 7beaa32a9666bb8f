"""GPU tests of the training operators where a caller's streams, buffers and
values are out of the ordinary. Tolerances as in test_training_gpu.py: U is the
unit roundoff of the output type, E = 2^-24 that of fp32 arithmetic."""
import math

import pytest
import torch

from newton_schulz_quintic_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from newton_schulz_quintic_gb300 import build
    build.build()
    api.load_library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, g, dtype=F32, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


# ------------------------------------------------------------------ embedding
def test_sliced_ids_on_another_stream():
    # the ids of a batch without its last column are not contiguous: their copy has to run on the call's stream, which
    # waits for nothing here, and must not be handed out again while the call still reads it
    g = gen(1)
    vocab, dim = 5000, 64
    table = normal((vocab, dim), g, BF16)
    batch = torch.randint(0, vocab, (16, 2049), device="cuda", generator=g)
    dout = normal((16 * 2048, dim), g, BF16)
    ids = batch[:, :-1]
    flat = ids.reshape(-1)
    looked_up, grad = api.embed_lookup(table, flat), api.embed_grad(dout, flat, vocab=vocab)
    other = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream
        for s in other:
            a = api.embed_lookup(table, ids, stream=s)
            b = api.embed_grad(dout, ids, vocab=vocab, stream=s)
            torch.full((16, 2048), -1, device="cuda")  # what takes the memory that the current stream has free
            s.synchronize()  # the current stream still sleeps
            assert torch.equal(a.cpu().view(-1, dim), looked_up.cpu()) and torch.equal(b.cpu(), grad.cpu())
    torch.cuda.synchronize()

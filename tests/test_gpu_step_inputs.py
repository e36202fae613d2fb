"""What an EdgeStep names as its inputs is what its step reads."""

import pytest
import torch

import oracle
from speculative_decoding_verification_padding_gb300 import build
from test_gpu_step_edges import _edge_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0.7, 0.0])
def test_a_step_on_copied_inputs_is_the_step_on_the_originals(T):
    build.build()
    oracle.build()
    a, b = (_edge_step(n_req=6, ctx_scale=0.01, temperature=T) for _ in range(2))
    for x in b.inputs():
        if x.is_floating_point():
            x.zero_()  # projections and logits come with the inputs alone
    for x, y in zip(a.inputs(), b.inputs(), strict=True):
        assert x.shape == y.shape and x.dtype == y.dtype
        y.copy_(x)
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        assert s.dev_status.item() == 0
    for x, y in zip((*a.outputs(), a.target, a.kv.cache_lens), (*b.outputs(), b.target, b.kv.cache_lens)):
        assert torch.equal(x, y)
    assert len(a.inputs()) == (8 if T > 0 else 7)

"""Shards from weights of another type than fp32: a base whose weights come in
bf16 is stored as the same values in fp32 are."""
import numpy as np
import pytest
import torch

import soup_synth as ss

pytestmark = pytest.mark.gpu


class Rounded:
    """A weight source's projections rounded to bf16, handed out as `dtype`."""

    def __init__(self, source, dtype):
        self.source, self.dtype = source, dtype

    def __getattr__(self, name):
        return getattr(self.source, name)

    def layer(self, l):
        return {k: v.to(torch.bfloat16).to(self.dtype) if not k.startswith("norm") else v
                for k, v in self.source.layer(l).items()}


@pytest.mark.parametrize("kind", ["nf4", "mxfp4", "bf16"])
def test_bf16_weights_are_stored_as_their_values(kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_streamed_qlora_b200 import model as M
    from tests.model_fixture import NumpyWeights
    cfg = M.ModelConfig(hidden=512, n_q_heads=4, n_kv_heads=2, head_dim=128, intermediate=1024, rank=16, alpha=32.0,
                        vocab=512, n_layers=2, kind=kind)
    w = NumpyWeights(cfg, 0)
    ids = torch.from_numpy(ss.uniform_ids(1, "ids", (2, 64), cfg.vocab).astype(np.int32))
    got = []
    for dtype in (torch.float32, torch.bfloat16):
        m = M.StreamedLoRAModel(cfg, 2, 64, n_buffers=2, weights=Rounded(w, dtype), head_chunk=48)
        try:
            m.set_ids(ids)
            loss = float(m.sft_step().item())
            got.append((loss, m.grad_flat.clone(), [h.clone() for h in m.host_layers]))
        finally:
            m.close()
    assert got[0][0] == got[1][0] and torch.equal(got[0][1], got[1][1])
    assert all(torch.equal(a, b) for a, b in zip(got[0][2], got[1][2]))

"""The storages of the frozen base that a model configuration can name."""
import dataclasses

import pytest


def test_unknown_storages_are_refused():
    from layer_streamed_qlora_b200 import _lib as L, model as M
    cfg = M.ModelConfig(hidden=512, n_q_heads=4, n_kv_heads=2, head_dim=128, intermediate=1024, rank=16, alpha=32.0,
                        vocab=512, n_layers=1)
    kinds = {"nf4": L.SOUP_WEIGHT_NF4, "mxfp4": L.SOUP_WEIGHT_MXFP4, "bf16": L.SOUP_WEIGHT_BF16}
    for k, v in kinds.items():
        assert dataclasses.replace(cfg, kind=k).weight_kind == v
    for k in ("MXFP4", "mx4", "fp4", "", None):
        with pytest.raises(ValueError, match="kind must be"):
            dataclasses.replace(cfg, kind=k)

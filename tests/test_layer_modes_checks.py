"""What PoetxLinear and Int8Linear do on the host around the C calls: refusals
that leave a layer as it was, where their scratch comes from and on which
stream and device the calls run.  The C calls are stood in for, so no GPU is
needed."""
import pytest
import torch

import orthogonal_equivalence_b200 as px
from orthogonal_equivalence_b200 import layer as layer_py

BF = torch.bfloat16


@pytest.mark.parametrize("scratch,match", [(torch.empty(128 * 192 - 1, dtype=BF), "elements"),
                                           (torch.empty(128 * 192), "scratch: dtype"),
                                           (torch.empty(128, 192, dtype=BF), "scratch: shape")])
def test_a_refused_scratch_leaves_the_layer_as_it_was(monkeypatch, scratch, match):
    monkeypatch.setattr(layer_py, "poetx_weight_quantize", lambda *a: None)
    L = px.PoetxLinear(128, 192, 64, px.POETX_BF16, device="cpu")
    W = L.W
    with pytest.raises(ValueError, match=match):
        L.quantize_weight(scratch)
    assert L.W is W and L.Wq is None and L.Wscale is None

"""What colibri_moe_decode says to a caller whose layer it does not run."""
import pytest
import torch

import sparse_expert_ffn_router_b200 as colibri


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", [colibri.COLIBRI_I8, colibri.COLIBRI_I4, colibri.COLIBRI_I8A8])
def test_quantised_layers_are_sent_to_forward(wdt):
    layer = colibri.MoELayer(128, 128, 4, 2, 0, colibri.COLIBRI_BF16, wdt, max_tokens=4)
    x = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(colibri.ColibriError) as ei:
        layer.decode(x, x, None, x, x)
    assert ei.value.status == -3
    said = colibri.colibri_last_error(layer.ctx)
    # true of every one of these types; how many launches forward takes differs between them
    assert "colibri_moe_forward" in said and "launch" not in said

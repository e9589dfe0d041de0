"""Host-side tests of the layers that forward_attn refuses (no GPU, the operators mocked)."""
import enum
from unittest import mock

import pytest
import torch

import hybrid_model_linear_amd as gdn
from hybrid_model_linear_amd import attention
from test_attn_host import _batch, _layer


class Kind(enum.Enum):
    DECODER = "decoder"
    DECODER_BIDIRECTIONAL = "decoder_bidirectional"
    ENCODER_ONLY = "encoder_only"


def _call(mode, **layer):
    x = torch.zeros(2, 4 * 64), torch.zeros(2, 2 * 64), torch.zeros(2, 2 * 64)
    with mock.patch.object(attention, "kv_store"), mock.patch.object(attention, "attn_decode") as de, \
            mock.patch.object(attention, "attn_extend") as ex:
        de.return_value = ex.return_value = torch.zeros(2, 4, 64)
        gdn.forward_attn(_layer(**layer), _batch(mode), *x)


@pytest.mark.parametrize("mode", ["decode", "extend", "target_verify"])
@pytest.mark.parametrize("layer,word", [
    (dict(is_cross_attention=True), "cross"), (dict(attn_type="encoder_only"), "encoder_only"),
    (dict(attn_type=Kind.ENCODER_ONLY), "ENCODER_ONLY"), (dict(attn_type=Kind.DECODER_BIDIRECTIONAL), "BIDIRECTIONAL"),
    (dict(v_head_dim=32), "v_head_dim 32"), (dict(v_head_dim=0), "v_head_dim 0")])
def test_other_attentions_are_refused(mode, layer, word):
    with pytest.raises(ValueError, match=word):
        _call(mode, **layer)


@pytest.mark.parametrize("layer", [dict(is_cross_attention=False), dict(attn_type="decoder"), dict(attn_type=Kind.DECODER),
                                   dict(attn_type=None), dict(v_head_dim=64), dict(v_head_dim=-1), dict(v_head_dim=None)])
def test_decoder_layers_are_taken(layer):
    for mode in ("decode", "extend"):
        _call(mode, **layer)

"""Workspaces and phases that are not on the device of the tensors described, or not in one piece, are
refused before anything runs."""

import pytest
import torch

import activation_sparse_tiered_amd as spax
from tests.test_layer_ops_descriptions import _attention


@pytest.mark.parametrize("ws,says", [
    (torch.zeros(1 << 20, dtype=torch.uint8), "workspace is on cpu"),
    (torch.zeros(1 << 20, dtype=torch.uint8, device="meta"), "workspace is on meta"),
])
def test_a_workspace_of_another_device_is_refused(ws, says):
    a = spax._on(_attention(), torch.device("cuda", 0))
    with pytest.raises(ValueError, match=says):
        spax.spax_paged_attention(a, ws)
    layers = spax._on((spax.DecoderLayer * 1)(), torch.device("cuda", 0))
    with pytest.raises(ValueError, match=says):
        spax.spax_decode_layers(layers, ws)


def test_a_workspace_in_pieces_is_refused():
    a = _attention()
    with pytest.raises(ValueError, match="contiguous"):
        spax.spax_paged_attention(a, torch.zeros(64, 64)[:, ::2])


def test_phases_of_another_device_are_refused():
    x = torch.zeros(1, 64)
    norm = spax.make_residual_norm(x, None, None, x.half())
    glu = spax.make_glu(x, x.clone(), x.half())
    attention = _attention()
    cache = attention._keep[1][0]
    q = torch.zeros(1, 4, 64, dtype=torch.float16)
    append = spax.make_kv_append(cache, q, q[:, :2], q[:, 2:], torch.zeros(1, dtype=torch.int32),
                                 q.clone())
    L = spax.spax_layout_init(256, [256])

    def phase(device):
        t = [torch.zeros(1, device=device) for _ in range(7)]
        return spax.make_phase(L, t[0], t[1], spax.topk_params(8, 8), *t[2:])

    here, there = phase("cpu"), phase("meta")
    spax.make_layer(here, append, attention, here, norm, here, glu, here, norm)
    for at in range(4):
        p = [here] * 4
        p[at] = there
        with pytest.raises(ValueError, match="different devices"):
            spax.make_layer(p[0], append, attention, p[1], norm, p[2], glu, p[3], norm)

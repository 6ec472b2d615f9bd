"""What the refusals of whole layers say: always the layer and the part, never the number of a
phase that the caller has not numbered (host-side checks, no GPU work)."""

import pytest

import activation_sparse_tiered_amd as spax
from activation_sparse_tiered_amd import _lib
from tests.test_layer_ops_abi import FAKE, _layer, _run_layers, needs_no_gpu

PARTS = ("qkv", "o", "gate_up", "down")


def _said(status, layers, **kw):
    assert _run_layers(layers, **kw) == status
    return _lib.lib.spax_last_error().decode()


@needs_no_gpu
@pytest.mark.parametrize("part", PARTS)
@pytest.mark.parametrize("fields,status,says", [
    (dict(packed=0), _lib.SPAX_ERR_NULL, "a required pointer is NULL"),
    (dict(full_idx=0), _lib.SPAX_ERR_NULL, "full_idx, approx_idx and counts are required"),
    (dict(counts=FAKE + 2), _lib.SPAX_ERR_ALIGN, "aligned"),
    (dict(layout=None), _lib.SPAX_ERR_NULL, "layout is NULL"),
    (dict(params=spax.topk_params(-1, 8)), _lib.SPAX_ERR_PARAM, ""),
])
def test_a_phase_is_named_by_layer_and_part(part, fields, status, says):
    good, buf = _layer(0)
    bad, _ = _layer(1, x=buf(22), **{part: fields})
    said = _said(status, [good, bad])
    assert said.startswith(f"layer 1, {part}: ") and says in said and "phase" not in said, said


@needs_no_gpu
@pytest.mark.parametrize("part,at", [("o", 17), ("gate_up", 20), ("down", 21)])
def test_a_workspace_on_a_buffer_names_its_layer(part, at):
    good, buf = _layer(0)
    other, buf1 = _layer(1, x=buf(22))
    need = spax.spax_layers_workspace_bytes((spax.DecoderLayer * 2)(good, other))
    said = _said(_lib.SPAX_ERR_PARAM, [good, other], ws=buf1(at), ws_bytes=need,
                 flags=spax.STEP_DETERMINISTIC)
    assert "layer 1" in said and "phase" not in said, said


@needs_no_gpu
def test_the_step_itself_still_numbers_its_phases():
    p = _layer(0)[0]._keep[0]
    arr = (spax.Phase * 2)(p["qkv"], p["o"])
    arr[1].packed = 0
    step = spax.Step()
    step.n_phases, step.phases = 2, arr
    assert _lib.lib.spax_decode_step_projections(step, 0) == _lib.SPAX_ERR_NULL
    assert _lib.lib.spax_last_error().startswith(b"phase 1: ")

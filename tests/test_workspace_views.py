"""A given workspace must own its bytes: the library writes on from its first
element, so an expanded or strided view would be written past. Checked where
no GPU is, with the device check out of the way."""

import os

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from newton_schulz_matrix_amd import operators as ops

pytestmark = pytest.mark.skipif(not os.path.exists(nsmi.LIB_PATH), reason="libnsmi.so not built")

BYTES = 64 << 20


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("host tensors: only where nothing can be launched")
    for module in (nsmi, ops):
        monkeypatch.setattr(module, "_device_tensor", lambda t, name: t)
    monkeypatch.setattr(nsmi, "_stream_ptr", lambda t: 0)
    monkeypatch.setattr(ops, "_stream_of", lambda dev: 0)


def _calls():
    m = [torch.zeros(64, 64) for _ in range(3)]
    ids, w, rstd = torch.zeros(64, dtype=torch.int64), torch.zeros(64), torch.zeros(64)
    logits, labels = torch.zeros(2, 3, 8), torch.zeros((2, 3), dtype=torch.int64)
    return {
        "ns_batched": lambda ws: nsmi.ns_batched([m[0]], workspace=ws),
        "ns_gram": lambda ws: nsmi.ns_gram(m[0], workspace=ws),
        "ns_direct": lambda ws: nsmi.ns_direct(m[0], workspace=ws),
        "ns_muon_step": lambda ws: nsmi.ns_muon_step([m[0]], [m[1]], [m[2]], 0.9, 0.1, workspace=ws),
        "ns_embedding_grad": lambda ws: nsmi.ns_embedding_grad(m[0], ids, 9, workspace=ws),
        "ns_rms_norm_grad": lambda ws: nsmi.ns_rms_norm_grad(m[0], m[1], w, rstd, workspace=ws),
        "ns_preference_loss": lambda ws: nsmi.ns_preference_loss(logits, labels, torch.zeros(2),
                                                                 workspace=ws),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_views_that_do_not_own_their_bytes(name):
    call = _calls()[name]
    one = torch.zeros(1, dtype=torch.uint8)
    for view in (one.expand(BYTES), torch.empty(2 * BYTES, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(view)
    # one that is too small is replaced, whatever it is; a dense one reaches the device check
    for ws in (one, one.expand(2), None, torch.empty(BYTES, dtype=torch.uint8)):
        with pytest.raises(nsmi.NsError) as e:
            call(ws)
        assert e.value.status in (nsmi.NS_ERR_UNSUPPORTED, nsmi.NS_ERR_WORKSPACE)

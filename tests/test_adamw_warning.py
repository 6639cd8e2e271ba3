"""A bf16 second moment with an average too slow for it is not taken without a
word (the calls end at the device check: there is no GPU here)."""

import os
import warnings

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from newton_schulz_matrix_amd import operators as ops

pytestmark = pytest.mark.skipif(not os.path.exists(nsmi.LIB_PATH), reason="libnsmi.so not built")


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("host tensors: only where nothing can be launched")
    for module in (nsmi, ops):
        monkeypatch.setattr(module, "_device_tensor", lambda t, name: t)
    monkeypatch.setattr(ops, "_stream_of", lambda dev: 0)


def _step(v_dtype, beta2):
    p = [torch.zeros(8), torch.zeros(4)]
    with pytest.raises(nsmi.NsError) as e:
        nsmi.ns_adamw_step(p, [t.clone() for t in p], [t.clone() for t in p],
                           [torch.zeros(8), torch.zeros(4, dtype=v_dtype)], 1, 0.1, betas=(0.9, beta2))
    assert e.value.status == nsmi.NS_ERR_UNSUPPORTED


@pytest.mark.parametrize("beta2", [0.999, 0.9999, 0.9962])
def test_warns_where_the_moment_would_stand_still(beta2):
    with pytest.warns(RuntimeWarning, match="exp_avg_sq"):
        _step(torch.bfloat16, beta2)


@pytest.mark.parametrize("dtype,beta2", [(torch.bfloat16, 0.99), (torch.bfloat16, 1 - 2.0 ** -8),
                                         (torch.float32, 0.9999)])
def test_says_nothing_else(dtype, beta2):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _step(dtype, beta2)

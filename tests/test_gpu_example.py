"""The example trains, quantizes and serves: the pieces work together."""
import os
import sys

import pytest

from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu


def test_train_quantize_serve():
    require_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_quantize_serve

    r = train_quantize_serve.main(steps=60, tokens=16)
    # from log(1000) for an untrained head; 0.3 of the targets cannot be learned
    assert r["first_loss"] > 6 and r["last_loss"] < 4 and r["logp_bf16"] > -1.5
    # int8 codes of weights and activations: logits of magnitude 10 off by less than 1 %
    assert r["drift"] < 0.1 and abs(r["logp_int8"] - r["logp_bf16"]) < 0.1
    assert r["greedy_right"] > 0.9

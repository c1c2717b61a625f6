"""The example of a whole GRPO step runs, and its stages agree with one another."""
import importlib.util
from pathlib import Path

import pytest
import torch

from oracle import rollout as ref

pytestmark = pytest.mark.gpu


def test_grpo_step_example():
    path = Path(__file__).resolve().parents[1] / "examples" / "grpo_step.py"
    spec = importlib.util.spec_from_file_location("grpo_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(prompt_len=700, members=3, steps=5, hidden=256, vocab=1001, verbose=False)
    # each value row is rounded by at most 2^-4 of itself and each key by as much, so that scores of a
    # few units move by a few hundredths: far below a tenth of the result, far above zero
    assert 0 < out["off"] < 0.1
    h, w, t = (out[n].cpu() for n in ("h", "w", "targets"))
    logp, *_ = ref.vocab_logprob(h, w, t, 1.0, -100)
    assert torch.allclose(out["logp"].cpu().double(), logp, atol=1e-4)
    dh, dw, _, _ = ref.vocab_gradients(h, w, t, out["d_logp"].cpu(), 1.0, -100)
    for got, want in ((out["dh"], dh), (out["dw"], dw)):
        assert (got.cpu().double() - want).norm() <= 2 ** -7 * want.norm()
    for mem in out["group"]:
        for name in ("o", "dq", "dk", "dv"):
            assert mem[name].isfinite().all()

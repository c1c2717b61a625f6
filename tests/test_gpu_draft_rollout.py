"""The example of a rollout with drafted tokens runs, and what it leaves is what a rollout without drafts would have."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = Path(__file__).resolve().parents[1] / "examples" / "draft_rollout.py"
    spec = importlib.util.spec_from_file_location("draft_rollout", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompt_len,members,new_tokens,drafts", [(70, 3, 40, 3), (97, 1, 33, 5), (33, 4, 10, 0)])
def test_rollout_with_drafts(example, prompt_len, members, new_tokens, drafts):
    out = example.main(prompt_len, members, new_tokens, drafts, verbose=False)
    assert [len(t) for t in out["tokens"]] == [new_tokens] * members == [len(x) for x in out["logps"]]
    assert out["offered"] > out["taken"] > 0 if drafts else out["offered"] == 0
    # The same tokens one by one through a server of their own give the same log-probabilities: pages, rows and states
    # after accepted and rejected drafts are those of a rollout without any.  The attention of one token and of four, and
    # what follows in bf16, round differently: some six roundings of 2^-9 relative to hidden rows whose logits have a
    # deviation of 3, an rms of 0.02, and the logits' own 2^-9 of up to 12; a lost row or a stale state moves them by 1.
    server = example.Server(out["model"], members, prompt_len + new_tokens + drafts, torch.device("cuda"))
    server.capture(out["prompt"][:-1])
    last = [int(out["prompt"][-1])] * members
    for i in range(new_tokens):
        logits, _, _, commit = server.step([[t] for t in last], None)
        commit(server.ints([1] * members))
        last = [t[i] for t in out["tokens"]]
        want = torch.log_softmax(logits.float(), 1)[range(members), last]
        got = torch.tensor([x[i] for x in out["logps"]], device="cuda")
        assert (want - got).abs().max() <= 0.15
    # the pool: the prompt's pages alone, at its front, in order
    used = -(-(prompt_len - 1) // example.PAGE)
    s = out["server"]
    assert s.refs.tolist() == [1] * used + [0] * (len(s.refs) - used)
    assert sorted(s.table[0, :used].tolist()) == list(range(used))
    assert s.kv_len.tolist() == [prompt_len - 1] + [0] * members

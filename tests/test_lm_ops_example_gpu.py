"""The speculative step of examples/, its pieces against the 64-bit forms of each operator."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from tests import lm_ops_reference as ref
from tests.test_lm_ops_gpu import close

pytestmark = pytest.mark.gpu


def load_example():
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    module = importlib.util.module_from_spec(spec)
    sys.modules["speculative_step"] = module
    spec.loader.exec_module(module)
    return module


def test_speculative_step_runs_the_operators_together():
    example = load_example()
    model = example.Model(batch=3, seed=5)
    model.attend(model.states(3 * 21), 21)
    for _ in range(2):
        drafts, logits, scored = example.speculative_step(model, model.states(3))
    assert model.lengths.tolist() == [23] * 3 and model.cache.read_errors() == 0
    want = ref.logprobs(logits, drafts, 1.0, 5)
    for name, (value, tol) in want.items():
        got = getattr(scored, name)
        assert torch.equal(got.cpu().long(), value.long()) if tol is None else close(got, value, tol, name) is None
    assert ((drafts >= 0) & (drafts < 8192)).all() and logits.abs().max() < 30


def test_speculative_step_as_a_program(capsys):
    load_example().main()
    assert "loss" in capsys.readouterr().out


def test_results_behind_one_another():
    """Operators launched back to back on one stream, each reading what the one ahead has just written, and the
    masked head between them: the same bits as with a wait after every call."""
    example = load_example()
    outs = []
    for wait in (False, True):
        model = example.Model(batch=4, seed=9)
        model.attend(model.states(4 * 40), 40)
        results = []
        for _ in range(4):
            hidden = model.states(4)
            state = model.attend(hidden, 1)
            if wait:
                torch.cuda.synchronize()
            drafts, best = example.mtp.mtp_masked_topk_tokens(model.head, state)
            if wait:
                torch.cuda.synchronize()
            logits = example.mtp.mtp_q4_matvec(model.verifier, state)
            if wait:
                torch.cuda.synchronize()
            scored = example.mtp.mtp_token_logprobs(logits, drafts, top=3)
            if wait:
                torch.cuda.synchronize()
            grad = example.mtp.mtp_token_logprobs_backward(logits, drafts, scored.lse, scored.entropy, scored.logprob)
            results += [state, drafts, best, logits, grad, *scored]
        torch.cuda.synchronize()
        outs.append([t.clone() for t in results])
    assert all(torch.equal(a, b) for a, b in zip(*outs))

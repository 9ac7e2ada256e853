"""The measured cases' calls of the library (perf/operators.py, own = True) give
what the cases' definitions say, where a call and a definition could part: the
loss of scored tokens some of which carry none."""
import importlib.util
import os

import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def cases():
    spec = importlib.util.spec_from_file_location("measured_cases",
                                                  os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


@pytest.mark.parametrize("ignored", [0.0, 0.2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,vocab", [(7, 300), (41, 1000), (130, 777)])
def test_scored_tokens(cases, tokens, vocab, dtype, ignored):
    """Loss, each token's loss, and every token's log-sum-exp, those of tokens
    without a loss among them."""
    case = dict(op="linear_xent", tokens=tokens, d_model=72, vocab=vocab, dtype=dtype,
                ignored=ignored, train=False)
    s = cases.prepare(case, 5)
    mean, token, lse = cases.run(s)
    x, w, target = s["x"], s["weight"], s["target"]
    loss, tok, _ = R.xent(x, w, target, x.dtype, "mean", ignore=cases.IGNORE)
    _, _, every = R.xent(x, w, target.clamp(min=0), x.dtype, "none", ignore=cases.IGNORE)
    # (the mean's own sum may be fp32: gamma of its terms)
    count = max(1, int((target != cases.IGNORE).sum()))
    R.within(mean, loss[0], loss[1] + R.gamma(tokens) * tok[0].abs().sum() / count, "loss")
    R.within(token, *tok, "token")
    R.within(lse, *every, "lse")

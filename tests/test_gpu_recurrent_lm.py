"""The example model runs the operators around the scan together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VOCAB = 97


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("recurrent_lm", os.path.join(ROOT, "examples", "recurrent_lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def model(lm):
    torch.manual_seed(3)
    return lm.RecurrentLM(VOCAB, width=64, lanes=96, dtype=torch.float32).cuda()


# fp32 throughout, two blocks: each path sums at most 200 terms of order one a
# value, in another order; 2^-24 * 200 a sum, a few sums one after another
TOL = 5e-4


def close(got, ref):
    assert torch.isfinite(got).all()
    assert (got - ref).abs().max() <= TOL * max(1.0, ref.abs().max().item())


def test_packed_documents_are_apart(lm, model):
    ids, pos = (t.cuda() for t in lm.corpus(VOCAB, 3, 150, torch.Generator().manual_seed(1)))
    with torch.no_grad():
        packed = model(ids, pos)
        for b in range(3):
            starts = (pos[b] == 0).nonzero().flatten().tolist() + [150]
            for s, e in zip(starts, starts[1:]):
                close(packed[b, s:e], model(ids[b:b + 1, s:e])[0])


def test_steps_continue_a_prompt(lm, model):
    ids = torch.randint(0, VOCAB, (3, 40), generator=torch.Generator().manual_seed(2)).cuda()
    lengths = [17, 1, 30]  # a prompt shorter than the convolution's window among them
    with torch.no_grad():
        whole = model(ids)
    server = lm.Server(model, slots=5)
    order = [4, 0, 2]
    for b, (s, n) in enumerate(zip(order, lengths)):
        close(server.prefill(s, ids[b, :n]), whole[b, n - 1])
    untouched = [t[[1, 3]].clone() for t in server.states]
    for k in range(9):
        at = [n + k for n in lengths]
        tokens = torch.stack([ids[b, t] for b, t in enumerate(at)] + [ids[0, 0]])
        slots = torch.tensor(order + [-1], dtype=torch.int32, device="cuda")  # the last row is no request
        got = server.step(tokens, slots)
        for b, t in enumerate(at):
            close(got[b], whole[b, t])
    for before, after in zip(untouched, server.states):
        assert torch.equal(before, after[[1, 3]])


def test_training_lowers_the_loss(lm):
    torch.manual_seed(4)
    m = lm.RecurrentLM(VOCAB, width=64, lanes=128).cuda()
    losses = lm.train(m, VOCAB, 60, rows=4, tokens=192, generator=torch.Generator().manual_seed(5))
    # ln 97 = 4.57 at chance; a document's next token follows from its last two
    assert losses[0] > 3.5 and losses[-1] < 0.75 * losses[0]
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in m.parameters())

"""The example's two paths, in graphs too, against 64 bits on the same quantized operands."""
import os
import sys

import numpy as np
import pytest

import layer_ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import score_prompt

    return score_prompt


def host(t):
    return t.detach().float().cpu().numpy()


def test_prompt_logits_and_scores(ex):
    """Each step against 64 bits from the step before's own output, so that no rounding is compounded."""
    bqm = ex.bqm
    m = ex.Model(512, 3001, DEV, seed=3)
    tokens = torch.randint(0, 3001, (40,), device=DEV)
    x = m.embedding[tokens[:-1]]
    xq, xs, _ = bqm.bqm_add_rmsnorm_e4m3_blk(x, None, m.gains[0], ex.EPS)
    out = bqm.bqm_e4m3_blk_gemm(m.w8, m.w8_grid, xq, xs)
    y_ref, T = oracle.e4m3_blk_matmul(m.w8.cpu().numpy(), host(m.w8_grid), xq.cpu().numpy(), host(xs))
    # the block GEMM's bound: groups of eight products cut 13 bits below the largest
    assert (np.abs(host(out) - y_ref) <= (7 * 2.0 ** -13 + 2.0 ** -19) * T).all()
    y, h = bqm.bqm_add_rmsnorm(out, x, m.gains[1], ex.EPS)
    ref, s = layer_ref.rmsnorm(host(out), host(x), host(m.gains[1]), ex.EPS)
    assert np.allclose(host(y), ref, rtol=32 * 2.0 ** -24, atol=0) and np.allclose(host(h), s, rtol=2.0 ** -24, atol=0)
    yq, ys = bqm.bqm_mxfp4_quantize(y)
    logits = m.prompt_logits(tokens[:-1])
    ref, T = layer_ref.mxfp4_matmul(m.head.cpu().numpy(), m.head_scales.cpu().numpy(),
                                    layer_ref.mxfp4_values(yq.cpu().numpy(), ys.cpu().numpy()))
    assert (np.abs(host(logits) - ref) <= (3 * 512 / 64 + 2) * 2.0 ** -23 * T).all()
    logp, entropy, ids, top = ex.score(m, tokens)
    r = layer_ref.logprobs(host(logits).astype(np.float64), tokens[1:, None].cpu().numpy(), 5)
    assert np.allclose(host(logp), r[0][:, 0], rtol=1e-5, atol=1e-5) and np.allclose(host(entropy), r[2], atol=1e-4)
    assert np.array_equal(ids.cpu().numpy(), r[3])


def test_decode_step_replayed_from_a_graph(ex):
    """The decode path captured once and replayed on new tokens gives the eager bits, every time."""
    bqm = ex.bqm
    m = ex.Model(512, 70001, DEV, seed=4)
    token = torch.zeros((), dtype=torch.long, device=DEV)
    for _ in range(3):
        ex.continue_greedily(m, token, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        logits = m.token_logits(token)
        got = bqm.bqm_logprobs(logits, None, 20)
    for t in (5, 69999, 1234, 5):
        token.fill_(t)
        g.replay()
        torch.cuda.synchronize()
        replayed = [logits.clone()] + [v.clone() for v in got]
        eager_logits = m.token_logits(torch.tensor(t, device=DEV))
        eager = [eager_logits] + list(bqm.bqm_logprobs(eager_logits, None, 20))
        torch.cuda.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b), t


def test_prompt_path_replayed_from_a_graph(ex):
    bqm = ex.bqm
    m = ex.Model(1024, 5000, DEV, seed=5)
    tokens = torch.randint(0, 5000, (200,), device=DEV)
    ex.score(m, tokens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ex.score(m, tokens, 3)
    for seed in range(4):
        tokens.copy_(torch.randint(0, 5000, (200,), generator=torch.Generator().manual_seed(seed)).to(DEV))
        g.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in got]
        eager = ex.score(m, tokens, 3)
        torch.cuda.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b), seed


def test_greedy_tokens_are_the_arguments_of_the_maximum(ex):
    m = ex.Model(256, 2000, DEV, seed=6)
    token = torch.tensor(7, device=DEV)
    for chosen, logp in ex.continue_greedily(m, token, 4):
        logits = host(m.token_logits(token)).astype(np.float64)[0]
        assert chosen == int(np.argmax(logits))
        lse = logits.max() + np.log(np.exp(logits - logits.max()).sum())
        assert abs(logp - (logits[chosen] - lse)) < 1e-5
        token = torch.tensor(chosen, device=DEV)

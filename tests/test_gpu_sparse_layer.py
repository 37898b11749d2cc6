"""The sparse layer's two paths: each step against 64 bits from the step before's own output, in graphs, and on two
streams at once."""
import os
import sys

import numpy as np
import pytest

import groups_ref
import layer_ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

DEV = "cuda:0"
WIDTH, INNER, EXPERTS, TOP, ADAPTERS, RANK = 512, 160, 12, 3, 4, 16


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_layer

    return sparse_layer


@pytest.fixture(scope="module")
def layer(ex):
    return ex.Layer(WIDTH, INNER, EXPERTS, TOP, ADAPTERS, RANK, DEV, seed=3)


def host(t):
    return t.detach().double().cpu().numpy()


def inputs(m, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((m, WIDTH), generator=g).to(DEV), torch.randint(-1, ADAPTERS, (m,), generator=g, dtype=torch.int32).to(DEV))


def close(got, want, tol):
    return (np.abs(host(got) - want) <= tol).all()


def check_lora(layer, y, before, after, ids):
    """The adapters' sum: h's 16 steps of three products, 16 / 8 a wave and part of k, then y's (see test_gpu_lora)."""
    x, a, b, i = host(y), host(layer.a), host(layer.b), ids.cpu().numpy()
    want, tol = host(before), 2.0 ** -24 * np.abs(host(before))
    for e in range(ADAPTERS):
        at, s = np.nonzero(i == e)[0], float(layer.scale[e])
        want[at] += s * ((x[at] @ a[e].T) @ b[e].T)
        total = (np.abs(x[at]) @ np.abs(a[e]).T) @ np.abs(b[e]).T
        tol[at] += s * total * (1.02 * (8 * 3 * 2 + 8 + 8 * 3) + 1) * 2.0 ** -23
    assert close(after, want, tol + 2.0 ** -24 * np.abs(want))


def check_route(layer, logits, ids, weights):
    want_ids, want, steps = groups_ref.route(host(logits), TOP, True)
    assert np.array_equal(ids.cpu().numpy(), want_ids) and close(weights, want, steps * 2.0 ** -24 * want + 2.0 ** -148)


def combined(outer, weights, h):
    terms = host(outer).reshape(len(h), TOP, WIDTH) * host(weights)[:, :, None]
    return terms.sum(1) + host(h), (TOP + 1) * 2.0 ** -24 * (np.abs(terms).sum(1) + np.abs(host(h)))


@pytest.mark.parametrize("m", [1, 7, 200])
def test_prompt_steps(ex, layer, m):
    bqm = ex.bqm
    x, adapters = inputs(m, m)
    plan = layer.plan(adapters)
    y, _ = bqm.bqm_add_rmsnorm(x, None, layer.gains[0], ex.EPS)
    out = bqm.bqm_f16_gemm(layer.w16, bqm.bqm_f16_cvt(y))
    with_lora = bqm.bqm_lora_add(y, layer.a, layer.b, *plan, scale=layer.scale, res=out)
    check_lora(layer, y, out, with_lora, adapters)
    y, h = bqm.bqm_add_rmsnorm(with_lora, x, layer.gains[1], ex.EPS)
    logits = bqm.bqm_f16_gemm(layer.router, bqm.bqm_f16_cvt(y))
    ids, weights = layer.route(y)
    check_route(layer, logits, ids, weights)
    flat = ids.cpu().numpy().reshape(-1)
    offsets, order = bqm.bqm_group_rows(ids, EXPERTS)
    want_offsets, want_order = groups_ref.group_rows(flat, EXPERTS)
    assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(order.cpu().numpy(), want_order)

    def half(v):
        return groups_ref.half_step(np.abs(v), 2.0 ** -7, 2.0 ** -133)

    yq, ys = bqm.bqm_mxfp4_quantize(y)
    inner = bqm.bqm_mxfp4_grouped_gemm(layer.up, layer.up_scales, yq, ys, offsets, order, glu=True, out_dtype=torch.bfloat16)
    p, total = groups_ref.expert_products(layer.up.cpu().numpy(), layer.up_scales.cpu().numpy(),
                                          layer_ref.mxfp4_values(yq.cpu().numpy(), ys.cpu().numpy()), flat, TOP)
    want, tol = groups_ref.gated(p, (3 * WIDTH / 64 + 2) * 2.0 ** -23 * total)
    assert close(inner, want, tol + half(np.abs(want) + tol))
    uq, us = bqm.bqm_mxfp4_quantize(inner)
    outer = bqm.bqm_mxfp4_grouped_gemm(layer.down, layer.down_scales, uq, us, offsets, order, out_dtype=torch.bfloat16)
    p, total = groups_ref.expert_products(layer.down.cpu().numpy(), layer.down_scales.cpu().numpy(),
                                          layer_ref.mxfp4_values(uq.cpu().numpy(), us.cpu().numpy()), flat, 1)
    tol = (3 * INNER / 64 + 2) * 2.0 ** -23 * total
    assert close(outer, p, tol + half(np.abs(p) + tol))
    want, tol = combined(outer, weights, h)
    got = layer.prompt(x, plan)
    assert close(got, want, tol)


@pytest.mark.parametrize("m", [1, 6, 15])
def test_decode_steps(ex, layer, m):
    bqm = ex.bqm
    x, adapters = inputs(m, 50 + m)
    plan = layer.plan(adapters)
    y, _ = bqm.bqm_add_rmsnorm(x, None, layer.gains[0], ex.EPS)
    out = bqm.bqm_q8_0_gemv(layer.w, *bqm.bqm_q8_1_quantize(y))
    q, d = oracle.q8_1_quantize(y.cpu().numpy())
    ref, total = oracle.q8_0_matmul(layer.w.cpu().numpy(), q, d, WIDTH)
    assert close(out, ref, 1e-5 * total)
    with_lora = bqm.bqm_lora_add(y, layer.a, layer.b, *plan, scale=layer.scale, res=out)
    check_lora(layer, y, out, with_lora, adapters)
    y, h = bqm.bqm_add_rmsnorm(with_lora, x, layer.gains[1], ex.EPS)
    ids, weights = layer.route(y)
    check_route(layer, bqm.bqm_f16_gemm(layer.router, bqm.bqm_f16_cvt(y)), ids, weights)
    flat = ids.cpu().numpy().reshape(-1)
    inner = bqm.bqm_mxfp4_expert_gemv(layer.up, layer.up_scales, y, ids, glu=True)
    p, total = groups_ref.expert_products(layer.up.cpu().numpy(), layer.up_scales.cpu().numpy(), host(y), flat, TOP)
    want, tol = groups_ref.gated(p, (8 * 16 + 8 + 4) * 2.0 ** -23 * total)
    assert close(inner, want, tol)
    outer = bqm.bqm_mxfp4_expert_gemv(layer.down, layer.down_scales, inner, ids)
    p, total = groups_ref.expert_products(layer.down.cpu().numpy(), layer.down_scales.cpu().numpy(), host(inner), flat, 1)
    assert close(outer, p, (8 * 16 + 8 + 4) * 2.0 ** -23 * total)
    want, tol = combined(outer, weights, h)
    assert close(layer.decode(x, plan), want, tol)


@pytest.mark.parametrize("path,m", [("decode", 1), ("decode", 15), ("prompt", 33), ("prompt", 300)])
def test_paths_replayed_from_a_graph(layer, path, m):
    """Captured once with its plan, replayed on new rows, adapters and so experts, with eager work in between."""
    step = getattr(layer, path)
    x, adapters = inputs(m, 1)
    for _ in range(2):
        step(x, layer.plan(adapters))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(x, layer.plan(adapters))
    for seed in range(4):
        new_x, new_adapters = inputs(m, 10 + seed)
        x.copy_(new_x)
        adapters.copy_(new_adapters)
        g.replay()
        torch.cuda.synchronize()
        replayed = got.clone()
        eager = step(new_x, layer.plan(new_adapters))
        torch.cuda.synchronize()
        assert torch.equal(replayed, eager), seed


def test_two_graphs_share_buffers_and_workspaces(ex, layer):
    """Two captured graphs of different sizes on the same workspaces and outputs, replayed in turn."""
    bqm = ex.bqm
    work = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    ids = {m: torch.randint(-1, 9, (m,), generator=torch.Generator().manual_seed(m), dtype=torch.int32).to(DEV) for m in (5000, 9000)}
    x = {m: inputs(40 if m == 5000 else 25, m)[0] for m in ids}
    plans, graphs, outs = {}, {}, {}

    def run(m):
        rows = len(x[m])
        offsets, order = bqm.bqm_group_rows(ids[m], 8, workspace=work)
        plan = bqm.bqm_group_rows(ids[m][:rows], ADAPTERS)
        return offsets, order, bqm.bqm_lora_add(x[m], layer.a, layer.b, *plan, workspace=work)

    for m in ids:
        plans[m] = [v.clone() for v in run(m)]
    torch.cuda.synchronize()
    for m in ids:
        graphs[m] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[m]):
            outs[m] = run(m)
    for _ in range(3):
        for m in ids:
            graphs[m].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[m], plans[m]):
                assert torch.equal(a, b), m
            work.fill_(0x77)


def test_two_streams_at_once_match_serial(layer):
    work = [(inputs(15, 3), "decode"), (inputs(260, 4), "prompt")]
    serial = [getattr(layer, path)(x, layer.plan(a)) for (x, a), path in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        out = []
        for s, ((x, a), path) in zip(streams, work):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                out.append(getattr(layer, path)(x, layer.plan(a)))
        for s in streams:
            s.synchronize()
        for a, b in zip(out, serial):
            assert torch.equal(a, b)


def test_example_runs(ex, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["sparse_layer.py", "--tokens", "40", "--width", "512", "--inner", "128", "--experts", "8",
                                      "--top", "2", "--adapters", "3"])
    ex.main()
    assert "40 rows" in capsys.readouterr().out

"""The 8-bit head and sampling together, as a program answers with them: a head
quantised once, hidden states projected against it, a token drawn for each
row; alone, on two streams at once, inside a captured graph, and through the
bounds-checking build."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import output_projection_kl_amd as fkl
from oracle import decode_oracle as oracle
from output_projection_kl_amd.build import DEBUG_LIB_PATH

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
import decode_cases  # noqa: E402
from decode_cases import answer, make_head  # noqa: E402

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


@pytest.mark.parametrize("N", [1, 3, 40, 200])
def test_answering_with_a_quantised_head(N):
    """Against the oracle, each step on the GPU's own inputs of that step; and the 8-bit logits stay
    within the two roundings' bound of the bf16 head's: the levels are off by at most half a step each, so a
    row's sum by at most K (127 + 127 + 1/2) / 2 steps' product."""
    dev = _dev()
    K, V = 200, 3001
    h, W, head, scale, u = make_head(fkl, torch, dev, N, K, V, N)
    logits, token, logprob = answer(fkl, h, head, scale, u, temperature=0.9, top_k=100, top_p=0.97)
    torch.cuda.synchronize()
    rq, rs = oracle.quantize(W.float().cpu().numpy())
    np.testing.assert_array_equal(head.cpu().numpy(), rq)
    qa, sa = oracle.quantize(h.float().cpu().numpy())
    want, prod = oracle.project(qa, sa, rq, rs)
    got = logits.double().cpu().numpy()
    assert (np.abs(got - want) <= 1.01 * (3 * 2.0 ** -24 * np.abs(prod) + (2.0 ** -24 + 2.0 ** -8) * np.abs(want))).all()
    exact = h.double().cpu().numpy() @ W.double().cpu().numpy().T
    step = sa.astype(np.float64)[:, None] * rs.astype(np.float64)[None, :]
    assert (np.abs(want - exact) <= 1.01 * K * (127 + 127 + 0.5) / 2 * step).all()
    rt, rl = oracle.sample(got, u.cpu().numpy(), 0.9, 100, 0.97)
    np.testing.assert_array_equal(token.cpu().numpy(), rt)
    assert (np.abs(logprob.double().cpu().numpy() - rl) <= 1.01 * 2.0 ** -24 * np.abs(rl) + 1e-11).all()


def test_labels_drawn_from_a_teacher_cache_feed_the_loss():
    """topk's lists -> one token drawn from each -> the loss's hard labels."""
    dev = _dev()
    h, W, _, _, u = make_head(fkl, torch, dev, 60, 64, 2000, 8)
    t_idx, t_logit = fkl.topk(h, W, 50)
    label, _ = fkl.sample(t_logit, u, top_p=0.9, ids=t_idx)
    assert fkl.validate_terms(60, 2000, label=label) == 0
    loss, lse = fkl.forward(h, W, t_idx, t_logit, label=label, label_weight=1.0)
    torch.cuda.synchronize()
    z = h.double().cpu() @ W.double().cpu().T
    ce = torch.nn.functional.cross_entropy(z, label.cpu().long())
    assert abs(loss.item() - ce.item()) <= 1e-3 * abs(ce.item())


def test_two_streams_match_one():
    dev = _dev()
    jobs = [(make_head(fkl, torch, dev, 70, 136, 9000, 1), dict(top_p=0.9)),
            (make_head(fkl, torch, dev, 9, 500, 40000, 2), dict(temperature=1.5, top_k=700, top_p=0.95))]

    def run(j):
        (h, _, head, scale, u), s = jobs[j]
        return answer(fkl, h, head, scale, u, **s)

    ref = [[t.cpu() for t in run(j)] for j in (0, 1)]
    cur, streams = torch.cuda.current_stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        print(f"[decode] two streams, round {rep}", flush=True)
        outs = []
        for j in (0, 1):
            streams[j].wait_stream(cur)
            with torch.cuda.stream(streams[j]):
                outs.append(run(j))
        for s in streams:
            cur.wait_stream(s)
        torch.cuda.synchronize()
        for r, o in zip(ref, outs):
            assert all(torch.equal(a, b.cpu()) for a, b in zip(r, o))


def test_captured_and_replayed():
    """Every launch is a kernel on the caller's stream: the chain is captured
    once and replayed on changed inputs, two graphs with a workspace each, with
    eager calls on other sizes in between."""
    dev = _dev()
    made = []
    for seed, (N, K, V), s in ((3, (5, 1024, 30001), dict(top_k=50, top_p=0.95)),
                               (4, (130, 72, 5000), dict(temperature=1.4, top_p=0.9))):
        h, _, head, scale, u = make_head(fkl, torch, dev, N, K, V, seed)
        need = fkl.project_workspace_size(N, V, K, a_dtype=torch.bfloat16, ldb=head.stride(0))
        ws = {"project": torch.empty(max(need, 256), dtype=torch.uint8, device=dev),
              "sample": torch.empty(fkl.sample_workspace_size(N, V, torch.bfloat16), dtype=torch.uint8, device=dev)}
        outs = {"logits": torch.empty((N, V), dtype=torch.bfloat16, device=dev),
                "token": torch.empty(N, dtype=torch.int32, device=dev), "logprob": torch.empty(N, device=dev)}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            answer(fkl, h, head, scale, u, ws, outs, **s)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            answer(fkl, h, head, scale, u, ws, outs, **s)
        made.append((graph, h, head, scale, u, outs, s))
    for rep in range(4):
        print(f"[decode] replay {rep}", flush=True)
        for graph, h, head, scale, u, outs, s in made:
            h.copy_(torch.randn(h.shape, generator=torch.Generator().manual_seed(rep)))
            u.copy_(torch.rand(u.shape, generator=torch.Generator().manual_seed(rep)))
            outs["token"].fill_(-7)
            outs["logprob"].fill_(float("nan"))
        for graph, *_ in made:
            graph.replay()
        torch.cuda.synchronize()
        got = [[m[5][k].clone() for k in ("logits", "token", "logprob")] for m in made]
        for m, g in zip(made, got):
            want = answer(fkl, m[1], m[2], m[3], m[4], **m[6])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(g, want))
        x = torch.randn((3, 50000 + rep), device=dev)
        fkl.sample(x, torch.rand(3, device=dev), top_p=0.99)


def test_debug_build_reports_nothing_and_gives_the_same(tmp_path):
    if not os.path.exists(DEBUG_LIB_PATH):
        pytest.fail(f"{DEBUG_LIB_PATH} is missing: __graft_entry__.build() builds it")
    _dev()
    out = tmp_path / "debug.npz"
    r = subprocess.run([sys.executable, "-u", os.path.join(HERE, "decode_cases.py"), str(out)],
                       env=dict(os.environ, FKL_LIBRARY=DEBUG_LIB_PATH), capture_output=True, text=True, timeout=100)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0, r.stderr[-3000:]
    dbg = dict(np.load(out))
    rel = decode_cases.run_all()
    assert set(rel) == set(dbg)
    for k in sorted(rel):
        if k.startswith("sample") and k.endswith("/1") or k == "answer/2":  # log-probabilities, in fp32
            np.testing.assert_allclose(rel[k], dbg[k], rtol=2.0 ** -22, atol=1e-10, err_msg=k)
        else:
            np.testing.assert_array_equal(rel[k], dbg[k], err_msg=k)


@pytest.mark.parametrize("call,error", [
    (lambda x, q, s, u: fkl.quantize(x.int()), TypeError),
    (lambda x, q, s, u: fkl.quantize(x.t()), ValueError),
    (lambda x, q, s, u: fkl.quantize(x[0]), ValueError),
    (lambda x, q, s, u: fkl.quantize(x, q=q[:, :8]), ValueError),
    (lambda x, q, s, u: fkl.quantize(x, scale=s[:1]), ValueError),
    (lambda x, q, s, u: fkl.quantize(x[:1].expand(4, 64)), ValueError),
    (lambda x, q, s, u: fkl.project(q, q, s), ValueError),
    (lambda x, q, s, u: fkl.project(x, q, s, a_scale=s), ValueError),
    (lambda x, q, s, u: fkl.project(x, x, s), TypeError),
    (lambda x, q, s, u: fkl.project(x, q[:, :32], s), ValueError),
    (lambda x, q, s, u: fkl.project(x, q, s.double()), TypeError),
    (lambda x, q, s, u: fkl.project(x, q, s, bias=s[:3]), ValueError),
    (lambda x, q, s, u: fkl.project(x, q, s, out_dtype=torch.int8), TypeError),
    (lambda x, q, s, u: fkl.project(x, q, s, out=x), ValueError),
    (lambda x, q, s, u: fkl.project(x, q.cpu(), s), ValueError),
    (lambda x, q, s, u: fkl.sample(x.int(), u), TypeError),
    (lambda x, q, s, u: fkl.sample(x, u[:2]), ValueError),
    (lambda x, q, s, u: fkl.sample(x, u.double()), TypeError),
    (lambda x, q, s, u: fkl.sample(x, u, temperature=-1.0), fkl.FklError),
    (lambda x, q, s, u: fkl.sample(x, u, top_p=float("nan")), fkl.FklError),
    (lambda x, q, s, u: fkl.sample(x, u, top_k=u), TypeError),
    (lambda x, q, s, u: fkl.sample(x, u, temperature=u[:3]), ValueError),
    (lambda x, q, s, u: fkl.sample(x, u, ids=q), ValueError),
    (lambda x, q, s, u: fkl.sample(x, u, token=u), TypeError),
    (lambda x, q, s, u: fkl.sample(x.t(), u), ValueError),
])
def test_refusals_of_the_binding(call, error):
    dev = _dev()
    x = torch.randn((4, 64), device=dev)
    q, s = fkl.quantize(x)
    with pytest.raises(error):
        call(x, q, s, torch.rand(4, device=dev))

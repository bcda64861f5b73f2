"""GPU parity of sampling (fkl.sample) with the fp64 oracle: tokens equal, and
log-probabilities to the rounding of the result to fp32 (2^-24 of its value)
plus 1e-11 for the 64-bit sums and exponentials on both sides."""

import numpy as np
import pytest
import torch

import output_projection_kl_amd as fkl
from oracle import decode_oracle as oracle

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [1, 2, 7, 63, 64, 65, 100, 255, 1000, 1024, 1025, 2048, 4097, 8185, 8186, 8191, 20000, 50257, 131075]


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def _np(v):
    return v.cpu().numpy() if isinstance(v, torch.Tensor) else v


def _check(x, u, T=1.0, k=0, p=1.0, q=0.0, ids=None, **kw):
    token, logprob = fkl.sample(x, u, temperature=T, top_k=k, top_p=p, min_p=q, ids=ids, **kw)
    torch.cuda.synchronize()
    rt, rl = oracle.sample(x.double().cpu().numpy(), u.cpu().numpy(), _np(T), _np(k), _np(p), _np(q),
                           None if ids is None else ids.cpu().numpy())
    np.testing.assert_array_equal(token.cpu().numpy(), rt)
    got = logprob.double().cpu().numpy()
    assert (np.isneginf(got) == np.isneginf(rl)).all()
    live = np.isfinite(rl)
    assert (np.abs(got[live] - rl[live]) <= 1.01 * 2.0 ** -24 * np.abs(rl[live]) + 1e-11).all()
    return token, logprob


def _logits(N, V, seed, dtype, dev, std=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, V), generator=g) * std
    at = torch.randint(0, V, (N, 5), generator=g)
    x.scatter_(1, at, 4.0 + 8.0 * torch.rand((N, 5), generator=g))
    return x.to(dtype).to(dev), torch.rand(N, generator=g).to(dev)


SETTINGS = [
    dict(),
    dict(T=0.7),
    dict(T=0.0),
    dict(k=1),
    dict(T=0.9, k=40),
    dict(k=900),
    dict(p=0.9),
    dict(T=1.5, p=0.95),
    dict(p=0.3, k=7),
    dict(q=0.05),
    dict(T=1.3, p=0.99, q=1e-4),
    dict(T=0.8, k=50, p=0.95, q=0.02),
    dict(T=3.0, k=3000, p=0.9),
    dict(q=1.0),
    dict(p=1e-9),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", SIZES)
def test_sample_settings(V, dtype):
    dev = _dev()
    N = 6 if V > 5000 else 19
    x, u = _logits(N, V, V, dtype, dev)
    for i, s in enumerate(SETTINGS):
        print(f"[sample] N={N} V={V} {dtype} {s}", flush=True)
        _check(x, torch.roll(u, i), **s)


@pytest.mark.parametrize("N,V", [(1, 201088), (300, 700), (64, 30000), (1025, 100), (260, 5000), (70, 70001)])
def test_sample_settings_for_each_row(N, V):
    dev = _dev()
    x, u = _logits(N, V, N + V, torch.float32, dev)
    g = torch.Generator().manual_seed(9)
    T = (torch.rand(N, generator=g) * 1.5).masked_fill(torch.rand(N, generator=g) < 0.2, 0.0).to(dev)
    k = torch.randint(-3, 2 * min(V, 300), (N,), generator=g, dtype=torch.int32).to(dev)
    p = (torch.rand(N, generator=g) * 1.2).to(dev)
    q = (torch.rand(N, generator=g) * 0.2 - 0.1).to(dev)
    print(f"[sample] per-row settings N={N} V={V}", flush=True)
    _check(x, u, T=T, k=k, p=p, q=q)
    _check(x, u, T=T, k=20, p=p)
    _check(x, u, k=k, q=q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [5, 200, 3000, 40000])
def test_sample_ties(V, dtype):
    """Few distinct logits: every border falls inside a group of equal entries,
    which is kept up to a position; -0 and +0 are equal."""
    dev = _dev()
    N = 12
    g = torch.Generator().manual_seed(V)
    x = torch.randint(-2, 2, (N, V), generator=g).float()
    x[:, ::3] *= -1.0  # zeros of both signs
    x[0] = 0.0
    x[1] = 1.5
    x, u = x.to(dtype).to(dev), torch.rand(N, generator=g).to(dev)
    for s in (dict(), dict(k=1), dict(k=3), dict(k=V // 2 + 1), dict(p=0.5), dict(p=0.01), dict(p=0.999), dict(q=0.2),
              dict(k=V - 1, p=0.7), dict(T=0.0), dict(T=0.01, p=0.6), dict(k=V // 3 + 1, p=0.5, q=0.1)):
        print(f"[sample] ties V={V} {dtype} {s}", flush=True)
        _check(x, u, **s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [3, 100, 1500, 33000])
def test_sample_masked_entries(V, dtype):
    """-inf and NaN are never drawn; rows of nothing else give -1; the type's
    lowest value is a number; +inf takes all of the mass."""
    dev = _dev()
    N = 16
    x, u = _logits(N, V, V + 1, torch.float32, dev)
    g = torch.Generator().manual_seed(1)
    mask = (torch.rand((N, V), generator=g) < 0.8).to(dev)
    x = x.masked_fill(mask, float("-inf"))
    x = x.masked_fill((torch.rand((N, V), generator=g) < 0.1).to(dev), float("nan"))
    x = x.to(dtype)
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2] = torch.finfo(dtype).min
    x[3, V // 2] = float("inf")
    x[4, 0] = x[4, V - 1] = float("inf")
    x[5] = float("-inf")
    x[5, V - 1] = 0.0
    x[6] = torch.finfo(dtype).min
    x[6, V // 3] = torch.finfo(dtype).max
    for s in (dict(), dict(k=5), dict(p=0.9), dict(q=0.1), dict(T=0.0), dict(T=2.0, k=10, p=0.8, q=0.01), dict(k=V - 1)):
        print(f"[sample] masked V={V} {dtype} {s}", flush=True)
        token, logprob = _check(x, u, **s)
        assert token[0] == -1 and token[1] == -1 and torch.isneginf(logprob[:2]).all()
        assert token[5] == V - 1


@pytest.mark.parametrize("V", [1, 50, 5000])
def test_sample_random_numbers_at_the_ends(V):
    dev = _dev()
    x, _ = _logits(8, V, 3, torch.float32, dev)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), 0.5, 2.0 ** -126], device=dev)
    for s in (dict(), dict(k=10), dict(p=0.7), dict(T=0.0)):
        _check(x, u, **s)


@pytest.mark.parametrize("V", [40, 3000])
def test_sample_extreme_temperatures_and_settings(V):
    dev = _dev()
    x, u = _logits(6, V, 4, torch.float32, dev)
    for s in (dict(T=1e-30), dict(T=1e-44), dict(T=1e30), dict(T=3e38, p=0.5), dict(p=0.0), dict(p=-1.0), dict(p=7.0),
              dict(q=2.0), dict(q=-3.0), dict(k=-5), dict(k=2 ** 31 - 1), dict(T=1e-3, q=1e-30, p=0.999999)):
        print(f"[sample] extremes V={V} {s}", flush=True)
        _check(x, u, **s)
    x[:, ::2] = float("-inf")
    for s in (dict(T=1e30, p=0.5), dict(T=3e38, p=0.9), dict(T=3e38), dict(T=1e-30, p=0.5), dict(T=1e37, k=V // 4)):
        print(f"[sample] extremes V={V} {s}, half masked", flush=True)
        _check(x, u, **s)
    x = torch.nan_to_num(x, neginf=-3.0)
    bad = torch.tensor([-1.0, float("nan"), float("inf"), 1.0, 0.0, float("-inf")], device=dev)
    token, logprob = _check(x, u, T=bad)
    assert token[[0, 1, 2, 5]].tolist() == [-1] * 4 and (token[[3, 4]] >= 0).all()
    nan = torch.full((6,), float("nan"), device=dev)
    _check(x, u, p=nan, q=nan)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [30, 100, 1024, 6001])
def test_sample_strided_rows_ids_and_given_outputs(V, dtype):
    """Rows that are slices of a wider matrix, aligned and not, with lists of
    indices of another stride; only the rows' own outputs are written."""
    dev = _dev()
    N = 11
    wide, u = _logits(N, V + 40, V, dtype, dev)
    lists = torch.randint(0, 2 ** 31 - 1, (N, V + 3), dtype=torch.int32, device=dev)
    for lo in (0, 1, 8):
        for ids in (None, lists[:, :V], lists[:, 3:]):
            store = torch.full((N + 4,), 77, dtype=torch.int32, device=dev)
            lp = torch.full((N + 4,), 77.0, device=dev)
            _check(wide[:, lo:lo + V], u, T=0.9, k=60, p=0.97, ids=ids, token=store[2:N + 2], logprob=lp[2:N + 2])
            assert (store[[0, 1, N + 2, N + 3]] == 77).all() and (lp[[0, 1, N + 2, N + 3]] == 77).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [262135, 262136, 262137, 262144, 300001, 524280, 524281, 1048568, 1048569])
def test_sample_the_longest_rows(V, dtype):
    """Around the row lengths at which the groups, chunks and the route change, from aligned and unaligned rows."""
    dev = _dev()
    wide, u = _logits(3, V + 8, V, dtype, dev)
    for lo in (0, 7):
        x = wide[:, lo:lo + V]
        for s in (dict(), dict(k=60), dict(k=5000, p=0.9), dict(p=0.9), dict(T=2.5, p=0.95), dict(q=0.01), dict(T=0.0)):
            print(f"[sample] V={V} lo={lo} {dtype} {s}", flush=True)
            _check(x, u, **s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(3, 60000), (40, 30000), (600, 20000), (3, 262000)])
def test_sample_flat_rows(N, V, dtype):
    """Rows in which top-p keeps tens of thousands of entries, and rows whose
    entries nearly all weigh the same."""
    dev = _dev()
    g = torch.Generator().manual_seed(N)
    x = (torch.randn((N, V), generator=g) * torch.tensor([2.0, 1.0, 1e-3])[torch.arange(N) % 3][:, None] + 3.0).to(dtype)
    x, u = x.to(dev), torch.rand(N, generator=g).to(dev)
    rows = slice(0, 9)
    for s in (dict(p=0.9), dict(p=0.999), dict(T=1.7, p=0.5), dict(p=0.95, q=1e-3), dict(k=6000), dict(k=V - 5, p=0.8)):
        print(f"[sample] flat N={N} V={V} {dtype} {s}", flush=True)
        token, logprob = fkl.sample(x, u, temperature=s.get("T", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                                    min_p=s.get("q", 0.0))
        _check(x[rows], u[rows], **s)
        few, few_logprob = fkl.sample(x[rows], u[rows], temperature=s.get("T", 1.0), top_k=s.get("k", 0),
                                      top_p=s.get("p", 1.0), min_p=s.get("q", 0.0))
        torch.cuda.synchronize()
        assert torch.equal(token[rows], few) and torch.allclose(logprob[rows], few_logprob, rtol=1e-6, atol=1e-10)


def test_sample_from_a_teacher_cache():
    """topk() lists, one entry drawn from each: the tokens are the lists' own indices."""
    dev = _dev()
    h = torch.randn((70, 64), device=dev).to(torch.bfloat16)
    W = torch.randn((3000, 64), device=dev).to(torch.bfloat16)
    t_idx, t_logit = fkl.topk(h, W, 100)
    u = torch.rand(70, device=dev)
    token, _ = _check(t_logit, u, T=2.0, p=0.95, ids=t_idx)
    assert (t_idx == token[:, None]).any(dim=1).all()


def test_sample_no_rows():
    dev = _dev()
    token, logprob = fkl.sample(torch.empty((0, 50), device=dev), torch.empty(0, device=dev))
    assert token.shape == (0,) and logprob.shape == (0,)


def test_sample_frequencies():
    """Draws over a fine grid of random numbers fall on each entry in proportion
    to its weight: with u = (i + 1/2) / n every count is within one of n p."""
    dev = _dev()
    n, V = 4096, 37
    row = torch.randn(V, generator=torch.Generator().manual_seed(2)) * 2
    x = row.to(dev).expand(n, V).contiguous()
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().to(dev)
    token, _ = fkl.sample(x, u, temperature=0.8, top_p=0.98)
    pos, w = oracle.kept_entries(row.double().numpy(), np.float32(0.8), 0, np.float32(0.98), 0)
    want = np.zeros(V)
    want[pos] = w / w.sum() * n
    assert np.abs(np.bincount(token.cpu().numpy(), minlength=V) - want).max() <= 1.0


# Rows that keep thousands of entries, their logits moved so that the border
# lies among positive, negative and zero ones; each with as many rows as two
# workgroups on a CU take, and with few.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [4, 258])
@pytest.mark.parametrize("shift", [-40.0, -1.5, 0.0, 30.0])
def test_sample_wide_borders_of_either_sign(shift, N, dtype):
    dev = _dev()
    V = 9001
    g = torch.Generator().manual_seed(N + int(shift * 2))
    x = (torch.randn((N, V), generator=g) * 1.2 + shift).to(dtype).to(dev)
    u = torch.rand(N, generator=g).to(dev)
    _check(x, u, p=0.8)
    _check(x, u, T=2.0, p=0.9)
    _check(x, u, k=3500)
    _check(x, u, q=0.002)


@pytest.mark.parametrize("dtype,N,V", [(torch.float32, 600, 120001), (torch.bfloat16, 1030, 150016), (torch.float32, 1200, 60001)])
def test_sample_logits_larger_than_the_cache(dtype, N, V):
    """Logits that are streamed past the last-level cache: the same draws as from their halves, which are not."""
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(V)
    x = (2.0 * torch.randn((N, V), generator=g, device=dev)).to(dtype)
    u = torch.rand(N, generator=g, device=dev)
    assert x.nbytes > 1 << 28 > x.nbytes * 11 // 20
    half = (N + 1) // 2
    for s in (dict(temperature=0.8), dict(top_k=40, top_p=0.9), dict(top_p=0.9), dict(top_p=0.9, min_p=0.01)):
        token, logprob = fkl.sample(x, u, **s)
        parts = [fkl.sample(x[r:r + half], u[r:r + half], **s) for r in (0, half)]
        assert torch.equal(token, torch.cat([p[0] for p in parts]))
        assert torch.allclose(logprob, torch.cat([p[1] for p in parts]), rtol=2.0 ** -22, atol=1e-11)
    _check(x[:6], u[:6], p=0.9)

"""GPU parity of the 8-bit head (fkl.quantize, fkl.project) with the fp64 oracle.

Levels and scales must equal the oracle's bit for bit (the rounding is that of
the real quotient). The product's sum is exact; the fp32 steps after it are
the sum's conversion, the product with a_scale, the fused product with b_scale
and addition of the bias, and the rounding to the output type, each off by at
most half a step of its type: |error| <= 2 * 2^-24 |product| + 2^-24 |result|
+ eps / 2 |result|, taken 1% wider for the products of those terms, and one
more 2^-24 |product| where the call quantises the rows (a_scale is rounded).
"""

import numpy as np
import pytest
import torch

import output_projection_kl_amd as fkl
from oracle import decode_oracle as oracle

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def _check_levels(x, q, scale):
    rq, rs = oracle.quantize(x.float().cpu().numpy())
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(scale.cpu().numpy(), rs)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (2, 63), (7, 64), (4, 1000), (33, 2880), (2, 8192), (3, 8200),
                                 (2, 40000), (1, 131071)])
def test_quantize_levels(M, K, dtype):
    dev = _dev()
    g = torch.Generator().manual_seed(M * 131 + K)
    x = (torch.randn((M, K), generator=g) * torch.exp(2 * torch.randn((M, 1), generator=g))).to(dtype).to(dev)
    print(f"[quantize] M={M} K={K} {dtype}", flush=True)
    q, s = fkl.quantize(x)
    torch.cuda.synchronize()
    assert q.shape == (M, K) and q.stride(0) % 16 == 0 and s.dtype == torch.float32
    _check_levels(x, q, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_halves_and_extremes(dtype):
    """Quotients that are halves exactly (ties to even), the type's largest and
    smallest numbers, a row of zeros, negative zeros."""
    dev = _dev()
    half = torch.arange(-254, 255, dtype=torch.float64) / 2  # q + 1/2 for every q where the maximum is 127
    rows = [half, half * 2.0 ** -6, half / 127, torch.zeros_like(half), -torch.zeros_like(half)]
    info = torch.finfo(dtype)
    rows += [half / 127 * info.max, half / 127 * info.tiny, half * info.smallest_normal * info.eps]
    x = torch.stack(rows).to(dtype).to(dev)
    print(f"[quantize] halves {dtype}", flush=True)
    q, s = fkl.quantize(x)
    torch.cuda.synchronize()
    _check_levels(x, q, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_rows_that_are_not_finite(dtype):
    dev = _dev()
    x = torch.randn((5, 72)).to(dtype)
    x[1, 3], x[2, 70], x[3, 0] = float("inf"), float("nan"), float("-inf")
    x = x.to(dev)
    q, s = fkl.quantize(x)
    torch.cuda.synchronize()
    assert torch.isnan(s[1:4]).all() and (q[1:4] == 0).all() and torch.isfinite(s[[0, 4]]).all()
    _check_levels(x[[0, 4]], q[[0, 4]], s[[0, 4]])


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strided_rows_write_only_their_columns(dtype):
    dev = _dev()
    big = torch.randn((9, 300), device=dev).to(dtype)
    for lo, hi in ((0, 64), (3, 100), (8, 136), (1, 2)):
        x = big[1:8, lo:hi]
        store = torch.full((9, 400), 99, dtype=torch.int8, device=dev)
        q = store[1:8, lo:hi]
        scale = torch.empty(7, device=dev)
        out, _ = fkl.quantize(x, q=q, scale=scale)
        torch.cuda.synchronize()
        assert out.data_ptr() == q.data_ptr()
        _check_levels(x, q, scale)
        store[1:8, lo:hi] = 99
        assert (store == 99).all()


def _rows(M, K, g, dev, padded=True):
    w = -(-K // 16) * 16 if padded else K
    return torch.randint(-128, 128, (M, w), generator=g, dtype=torch.int8).to(dev)[:, :K]


def _check_product(out, a, sa, b, sb, bias, quantised=False):
    want, prod = oracle.project(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy(),
                                None if bias is None else bias.cpu().numpy())
    half = torch.finfo(out.dtype).eps / 2
    tol = 1.01 * ((3 if quantised else 2) * 2.0 ** -24 * np.abs(prod) + (2.0 ** -24 + half) * np.abs(want))
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))


SIZES = [(1, 1, 1), (1, 16, 64), (2, 3, 5), (1, 257, 2880), (3, 1000, 64), (5, 100, 63), (15, 129, 130), (16, 64, 128),
         (17, 300, 65), (31, 33, 1000), (32, 520, 320), (33, 70, 129), (48, 777, 512), (64, 64, 64), (65, 255, 191),
         (100, 256, 256), (128, 130, 513), (129, 257, 64), (200, 500, 72), (256, 256, 128), (257, 300, 1000),
         (511, 513, 200), (700, 1025, 2887)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_project_int8_rows(M, N, K, out):
    dev = _dev()
    g = torch.Generator().manual_seed(M * 7919 + N * 31 + K)
    a, b = _rows(M, K, g, dev), _rows(N, K, g, dev)
    sa = (torch.rand(M, generator=g) + 0.5).to(dev) / 127
    sb = (torch.rand(N, generator=g) + 0.5).to(dev) / (127 * K ** 0.5)
    bias = torch.randn(N, generator=g).to(dev) if (M + N) % 2 else None
    print(f"[project] M={M} N={N} K={K} {out} bias={bias is not None}", flush=True)
    got = fkl.project(a, b, sb, a_scale=sa, bias=bias, out_dtype=out)
    torch.cuda.synchronize()
    assert got.dtype == out and got.shape == (M, N)
    _check_product(got, a, sa, b, sb, bias)


# One size and more for every layout of the product, under the names of the
# library's trace; ragged in every dimension.
LAYOUTS = [(5, 70, 500, "project_16x16"), (85, 706, 417, "project_16x16"), (9, 30001, 1000, "project_16x64"),
           (25, 30001, 1000, "project_32x64"),
           (60, 40001, 1030, "project_64x64"), (38, 56217, 335, "project_64x128"), (117, 31149, 1090, "project_128x128"),
           (139, 19627, 2383, "project_128x256"), (201, 32003, 2887, "project_256x128"),
           (1030, 20003, 700, "project_256x256"), (505, 323, 7071, "project_split"), (3, 16, 9000, "project_split"),
           (100, 65, 20011, "project_split")]


@pytest.mark.parametrize("M,N,K,layout", LAYOUTS)
def test_project_every_layout(M, N, K, layout):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(M + N + K)
    a = torch.randint(-128, 128, (M, -(-K // 16) * 16), generator=g, dtype=torch.int8, device=dev)[:, :K]
    b = torch.randint(-128, 128, (N, -(-K // 16) * 16), generator=g, dtype=torch.int8, device=dev)[:, :K]
    sa = (torch.rand(M, generator=g, device=dev) + 0.5) / 127
    sb = (torch.rand(N, generator=g, device=dev) + 0.5) / (127 * K ** 0.5)
    bias = torch.randn(N, generator=g, device=dev)
    print(f"[project] {layout} M={M} N={N} K={K}", flush=True)
    fkl.trace_read()
    fkl.trace_enable(True)
    half = fkl.project(a, b, sb, a_scale=sa, bias=bias, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    fkl.trace_enable(False)
    assert [k["name"] for k in fkl.trace_read()] == [layout]
    outs = [half] + [fkl.project(a, b, sb, a_scale=sa, bias=bias, out_dtype=t) for t in TYPES]
    torch.cuda.synchronize()
    # fp64 products of int8 sums are exact; the oracle's steps on the GPU
    prod = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    want = prod + bias.double()
    for out in outs:
        tol = 1.01 * (2 * 2.0 ** -24 * prod.abs() + (2.0 ** -24 + torch.finfo(out.dtype).eps / 2) * want.abs()) + 2.0 ** -25
        assert ((out.double() - want).abs() <= tol).all(), out.dtype
    assert torch.equal(half, outs[1 + TYPES.index(torch.bfloat16)])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 300, 2880), (1, 17, 3), (7, 129, 1000), (40, 257, 72), (130, 200, 2887), (300, 300, 64)])
def test_project_floating_rows_are_quantised_first(M, N, K, dtype):
    """Equal, bit for bit, to quantize() followed by the product of its rows."""
    dev = _dev()
    g = torch.Generator().manual_seed(M + N + K)
    a = torch.randn((M, K), generator=g).to(dtype).to(dev)
    b, sb = _rows(N, K, g, dev), (torch.rand(N, generator=g) + 0.5).to(dev) / 127
    print(f"[project-float] M={M} N={N} K={K} {dtype}", flush=True)
    got = fkl.project(a, b, sb, out_dtype=torch.float32)
    q, s = fkl.quantize(a)
    two = fkl.project(q, b, sb, a_scale=s, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got, two)
    rq, rs = oracle.quantize(a.float().cpu().numpy())
    _check_product(got, torch.from_numpy(rq), torch.from_numpy(rs), b, sb, None, quantised=True)


@pytest.mark.parametrize("M", [1, 5, 40, 140, 300])
def test_project_largest_sums_are_exact(M):
    """Every product 128 * 128 or its negative, at the largest K."""
    dev = _dev()
    K = 131071
    a = torch.full((M, K), -128, dtype=torch.int8, device=dev)
    b = torch.full((3, K), -128, dtype=torch.int8, device=dev)
    b[1] = 127
    b[2, ::2] = 127
    print(f"[project] largest sums M={M}", flush=True)
    got = fkl.project(a, b, torch.ones(3, device=dev), a_scale=torch.ones(M, device=dev), out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = (a[:1].cpu().numpy().astype(np.int64) @ b.cpu().numpy().astype(np.int64).T).astype(np.float32)
    assert (got.cpu().numpy() == want).all()


@pytest.mark.parametrize("M", [1, 20, 150, 300])
@pytest.mark.parametrize("ka,kb,lo", [(80, 80, 3), (96, 112, 16), (83, 90, 0), (75, 80, 5)])
def test_project_strided_and_unaligned_operands(M, ka, kb, lo):
    """Operands that are column slices of wider matrices (their neighbours hold
    other values), aligned and not, and an output that is one: nothing outside
    the slice is written."""
    dev = _dev()
    K, N = 70, 150
    g = torch.Generator().manual_seed(ka * kb + M)
    a = torch.randint(-128, 128, (M, lo + ka), generator=g, dtype=torch.int8).to(dev)[:, lo:lo + K]
    b = torch.randint(-128, 128, (N, lo + kb), generator=g, dtype=torch.int8).to(dev)[:, lo:lo + K]
    sa, sb = torch.rand(M, generator=g).to(dev), torch.rand(N, generator=g).to(dev) / 127
    for out_type in TYPES:
        store = torch.full((M + 2, N + 9), 7.0, dtype=out_type, device=dev)
        out = store[1:M + 1, 4:4 + N]
        got = fkl.project(a, b, sb, a_scale=sa, out=out)
        torch.cuda.synchronize()
        assert got is out
        _check_product(out.clone(), a, sa, b, sb, None)
        store[1:M + 1, 4:4 + N] = 7.0
        assert (store == 7.0).all()


def test_project_no_rows_and_rows_that_are_not_finite():
    dev = _dev()
    b, sb = torch.ones((40, 64), dtype=torch.int8, device=dev), torch.ones(40, device=dev)
    assert fkl.project(torch.empty((0, 64), dtype=torch.bfloat16, device=dev), b, sb).shape == (0, 40)
    q, s = fkl.quantize(torch.empty((0, 64), device=dev))
    assert q.shape == (0, 64) and s.shape == (0,)
    a = torch.ones((3, 64), device=dev)
    a[1, 5] = float("nan")
    out = fkl.project(a, b, sb, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()


@pytest.mark.parametrize("M", [1, 24, 100, 400])
def test_project_uses_the_given_workspace_and_stream(M):
    """On a side stream, into given memory, the same workspace used call after call."""
    dev = _dev()
    g = torch.Generator().manual_seed(5)
    K, N = 264, 333
    a = torch.randn((M, K), generator=g).to(torch.bfloat16).to(dev)
    b, sb = _rows(N, K, g, dev, padded=False), torch.rand(N, generator=g).to(dev)
    want = fkl.project(a, b, sb)
    flags = 0
    ws = torch.full((fkl.project_workspace_size(M, N, K, a_dtype=torch.bfloat16, flags=flags) + 1024,), 255,
                    dtype=torch.uint8, device=dev)
    need = ws.numel() - 1024
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            fkl.project(a, b, sb, out=out, workspace=ws[:need])
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (ws[need:] == 255).all()
    with pytest.raises(ValueError):
        fkl.project(a, b, sb, out=out, workspace=ws[:need - 1])


# A head larger than the last-level cache is read once, by hints or by whole
# lines, in tiles that follow the rows: the same sums as those of its parts,
# which are small enough to be read otherwise. Rows that start at every multiple
# of 16 bytes of a 128-byte line, alike and each its own; one stage and several,
# with every remainder of the last one.
@pytest.mark.parametrize("M,N,K,ldb,first", [
    (1, 120011, 2304, 2304, 0), (16, 140003, 1921, 1936, 16), (9, 2500003, 100, 112, 0), (2, 2200019, 128, 128, 48),
    (17, 101009, 2880, 2880, 64), (32, 110017, 2500, 2560, 112), (31, 130003, 2177, 2192, 32), (29, 2400011, 112, 112, 96),
    (64, 120011, 2304, 2304, 0), (40, 100003, 2880, 2880, 0), (65, 100003, 2816, 2816, 0), (128, 100003, 2833, 2848, 80),
    (129, 95003, 2944, 2944, 0), (250, 100003, 2700, 2704, 0)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_project_heads_larger_than_the_cache(M, N, K, ldb, first, out):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(M + N + K)
    store = torch.empty(N * ldb + 256, dtype=torch.int8, device=dev)
    store.random_(-128, 128, generator=g)
    assert N * ldb > 1 << 28 and store.data_ptr() % 128 == 0
    b = torch.as_strided(store, (N, K), (ldb, 1), first)
    a = torch.randint(-128, 128, (M, -(-K // 16) * 16), generator=g, dtype=torch.int8, device=dev)[:, :K]
    sa = torch.rand(M, generator=g, device=dev)
    sb = torch.rand(N, generator=g, device=dev)
    got = fkl.project(a, b, sb, a_scale=sa, out_dtype=out)
    part = (200 << 20) // ldb  # rows
    for n in range(0, N, part):
        want = fkl.project(a, b[n:n + part], sb[n:n + part], a_scale=sa, out_dtype=out)
        assert torch.equal(got[:, n:n + part], want), (n, N)
    # and some columns from the formula
    at = torch.randint(0, N, (64,), generator=g, device=dev)
    at[0], at[1] = 0, N - 1
    exact = (a.double() @ b[at].double().T).to(torch.float32) * sa[:, None]
    want = (exact.double() * sb[at].double()).float().to(out)
    err = (got[:, at].double() - want.double()).abs()
    # the same roundings to fp32 and to out: at most a step of out apart
    assert (err <= want.double().abs() * torch.finfo(out).eps).all()


@pytest.mark.parametrize("dtype,M,K", [(torch.bfloat16, 50021, 2881), (torch.float32, 20011, 4096)])
def test_quantize_more_than_the_cache_holds(dtype, M, K):
    """Rows streamed past the last-level cache: the same levels as those of their halves, which are not."""
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn((M, K), generator=g, device=dev).to(dtype)
    assert x.nbytes > 1 << 28 > x.nbytes * 11 // 20
    q, scale = fkl.quantize(x)
    half = (M + 1) // 2
    for r in (0, half):
        q1, scale1 = fkl.quantize(x[r:r + half])
        assert torch.equal(q[r:r + half], q1) and torch.equal(scale[r:r + half], scale1)
    _check_levels(x[-70:], q[-70:], scale[-70:])

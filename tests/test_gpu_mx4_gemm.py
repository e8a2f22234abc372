"""MXFP4 grouped products against fp64 sums of the values that the codes stand for.

Tolerance: products of two e2m1 values and two powers of two are exact in fp32, so the error is
that of the fp32 sums: at most K 2^-24 of the sum of the products' magnitudes if every addition
rounds alone, and this test allows 2^-22 sqrt(K) of their Euclidean norm (roundings of
independent sign, with a factor of four to spare) plus 2^-22 of the result.  bf16 outputs add half
a unit in the last place.  Sums of small integers must be exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_expert_layer_07_gb300 as moe
from oracle import mx4

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


def _values(codes, scales):
    return torch.tensor(mx4.dequantize(codes.cpu().numpy(), scales.cpu().numpy()), device="cuda")


def _problem(counts, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, rows = len(counts), sum(counts)
    spread = torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
    a, a_s = moe.mx4_quantize(torch.randn(rows, K, device="cuda", generator=g) * spread)
    w, w_s = moe.mx4_quantize(torch.randn(G, N, K, device="cuda", generator=g) * 0.02)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return a, a_s, w, w_s, off


def _sums(counts, a, a_s, w, w_s):
    """(sums, Euclidean norms of the products) in fp64."""
    va, lo, s, n = _values(a, a_s), 0, [], []
    for g, c in enumerate(counts):
        vw = _values(w[g], w_s[g])
        s.append(va[lo:lo + c] @ vw.t())
        n.append((va[lo:lo + c].square() @ vw.square().t()).sqrt())
        lo += c
    return torch.cat(s), torch.cat(n)


def _half_ulp(ref):
    return torch.exp2(torch.frexp(ref)[1].double() - 9)


CASES = [([1], 128, 128), ([5, 0, 130, 1], 256, 128), ([0, 0, 3], 384, 256), ([128], 256, 384),
         ([97, 33, 31, 64], 640, 1408), ([300, 1, 0, 129], 512, 2048), ([2] * 40, 256, 7168),
         ([1000], 7168, 256)]


@pytest.mark.parametrize("counts,N,K", CASES)
def test_product(lib, counts, N, K):
    a, a_s, w, w_s, off = _problem(counts, N, K, K + N)
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    rows = sum(counts)
    ref, norm = _sums(counts, a, a_s, w, w_s)
    bound = 2.0 ** -22 * (K ** 0.5 * norm + ref.abs())
    for kind, dt in ((moe.OUT_F32, torch.float32), (moe.OUT_BF16, torch.bfloat16)):
        # a guard row before and after the rows of the groups
        c = torch.full((rows + 2, N), 7.0, dtype=dt, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.mx4_grouped_gemm(len(counts), N, K, rows, a, a_s, off, wt, wt_s, c[1:-1], kind, st)
        assert int(st) == 0 and bool((c[0] == 7.0).all()) and bool((c[-1] == 7.0).all())
        lim = bound + (_half_ulp(ref) if dt == torch.bfloat16 else 0.0)
        err = (c[1:-1].double() - ref).abs()
        assert bool((err <= lim).all()), float((err / lim).max())


def test_integers_are_exact(lib):
    """Codes of whole numbers with scales of one: every partial sum is a whole number below 2^24."""
    g = torch.Generator().manual_seed(3)
    whole = torch.tensor([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15], dtype=torch.uint8)

    def codes(*shape):
        lo, hi = (whole[torch.randint(0, 11, shape, generator=g)] for _ in range(2))
        return (lo | (hi << 4)).cuda()

    K, N, rows = 1024, 512, 200
    a, w = codes(rows, K // 2), codes(1, N, K // 2)
    a_s = torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
    w_s = torch.full((1, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    c = torch.empty(rows, N, device="cuda")
    moe.mx4_grouped_gemm(1, N, K, rows, a, a_s, off, wt, wt_s, c, moe.OUT_F32)
    assert torch.equal(c.double(), _values(a, a_s) @ _values(w[0], w_s[0]).t())


def test_each_scale_meets_its_block(lib):
    """One row and one weight row at a time carry a large scale in one block: a scale that is read
    for a wrong row, or a wrong block of K, changes the result by its whole size."""
    K, N, rows = 512, 256, 128
    one = torch.full((rows, K // 2), 0x22, dtype=torch.uint8, device="cuda")        # all ones
    wone = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(K // 32, device="cuda")[None, :]
    n = torch.arange(N, device="cuda")[:, None]
    a_s = (127 + (r * 7 + b * 3) % 5).to(torch.uint8)
    w_s = (127 - (n * 3 + b * 5) % 7).to(torch.uint8)[None]
    wt, wt_s = moe.pack_mx4_weights(wone, w_s.contiguous())
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    c = torch.empty(rows, N, device="cuda")
    moe.mx4_grouped_gemm(1, N, K, rows, one, a_s.contiguous(), off, wt, wt_s, c, moe.OUT_F32)
    ref = _values(one, a_s) @ _values(wone[0], w_s[0]).t()
    assert torch.equal(c.double(), ref)


@pytest.mark.parametrize("counts,I,K", [([1], 128, 128), ([5, 0, 130, 1], 256, 384),
                                        ([97, 33, 31, 64], 1408, 2048), ([2] * 20, 384, 7168)])
def test_swiglu(lib, counts, I, K):
    """Each stored h against fp64: no further from it than the nearest MXFP4 value, but for 2e-5 of
    its block's largest (the fp32 sums above, a fast exponential and division)."""
    a, a_s, w, w_s, off = _problem(counts, 2 * I, K, K + I)
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    rows = sum(counts)
    h = torch.zeros(rows, I // 2, dtype=torch.uint8, device="cuda")
    h_s = torch.zeros(rows, I // 32, dtype=torch.uint8, device="cuda")
    moe.mx4_grouped_gemm_swiglu(len(counts), I, K, rows, a, a_s, off, wt, wt_s, h, h_s)
    o, _ = _sums(counts, a, a_s, w, w_s)
    ref = o[:, :I] / (1 + torch.exp(-o[:, :I])) * o[:, I:]
    near = (torch.tensor(mx4.dequantize(*mx4.quantize(ref.cpu().numpy())), device="cuda") - ref).abs()
    amax = ref.abs().view(rows, -1, 32).amax(-1).repeat_interleave(32, 1)
    off_by = (_values(h, h_s) - ref).abs() - near
    assert bool((off_by <= 2e-5 * amax).all()), float((off_by / amax).max())
    # codes and scales are those of the same values quantised alone, but for blocks next to a boundary
    c, s = mx4.quantize(ref.cpu().numpy())
    assert float(np.mean(h_s.cpu().numpy() != s)) < 1e-3
    assert float(np.mean(h.cpu().numpy() != c)) < 1e-3


def test_rows_with_nan_stay_alone(lib):
    a, a_s, w, w_s, off = _problem([140], 256, 512, 1)
    a_s[3, 5] = 255
    a_s[139, 0] = 255
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    c = torch.empty(140, 256, device="cuda")
    moe.mx4_grouped_gemm(1, 256, 512, 140, a, a_s, off, wt, wt_s, c, moe.OUT_F32)
    bad = torch.isnan(c)
    assert bool(bad[3].all()) and bool(bad[139].all()) and int(bad.any(-1).sum()) == 2


def test_offsets_that_are_wrong_or_leave_rows_out(lib):
    a, a_s, w, w_s, _ = _problem([10, 10], 256, 256, 2)
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = torch.full((20, 256), 7.0, device="cuda")
    for bad in ([0, 12, 21], [5, 3, 20], [-1, 3, 20]):
        st.zero_()
        moe.mx4_grouped_gemm(2, 256, 256, 20, a, a_s, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                             wt, wt_s, c, moe.OUT_F32, st)
        assert int(st) == moe.DEV_BAD_OFFSETS and bool((c == 7.0).all())
    st.zero_()
    moe.mx4_grouped_gemm(2, 256, 256, 20, a, a_s, torch.tensor([3, 8, 15], dtype=torch.int32, device="cuda"),
                         wt, wt_s, c, moe.OUT_F32, st)
    assert int(st) == 0 and bool((c[:3] == 7.0).all()) and bool((c[15:] == 7.0).all())
    assert not bool((c[3:15] == 7.0).any(-1).all())


def test_repeatable(lib):
    counts = [130, 7, 260, 0, 64]
    a, a_s, w, w_s, off = _problem(counts, 512, 1024, 4)
    wt, wt_s = moe.pack_mx4_weights(w, w_s)
    c = [torch.empty(461, 512, device="cuda") for _ in range(2)]
    for o in c:
        moe.mx4_grouped_gemm(5, 512, 1024, 461, a, a_s, off, wt, wt_s, o, moe.OUT_F32)
    assert torch.equal(*c)


# Groups of more than 128 rows on average run on pairs of CTAs, 256 rows to a tile: one row past a
# CTA's, exactly full tiles, a tile with nothing for the second CTA, an odd number of weight blocks
# (the second CTA has none) and of K blocks, more tiles than pairs.
PAIRS = [([129], 128, 128), ([256], 256, 256), ([257, 256, 255, 0], 384, 384), ([700, 1, 0, 300], 640, 1408),
         ([1300, 20], 1024, 2304), ([6000], 896, 640)]


@pytest.mark.parametrize("counts,N,K", PAIRS)
def test_product_on_pairs(lib, counts, N, K):
    test_product(lib, counts, N, K)


@pytest.mark.parametrize("counts,I,K", [([129], 128, 128), ([257, 256, 255, 0], 384, 384),
                                        ([700, 1, 0, 300], 640, 1408), ([3000, 130], 1024, 2304)])
def test_swiglu_on_pairs(lib, counts, I, K):
    test_swiglu(lib, counts, I, K)


def test_each_scale_meets_its_block_on_pairs(lib):
    """As above with rows, and weight rows, in both CTAs."""
    K, N, rows = 768, 384, 300
    one = torch.full((rows, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    wone = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(K // 32, device="cuda")[None, :]
    n = torch.arange(N, device="cuda")[:, None]
    a_s = (127 + (r * 7 + b * 3) % 5).to(torch.uint8)
    w_s = (127 - (n * 3 + b * 5) % 7).to(torch.uint8)[None]
    wt, wt_s = moe.pack_mx4_weights(wone, w_s.contiguous())
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    c = torch.empty(rows, N, device="cuda")
    moe.mx4_grouped_gemm(1, N, K, rows, one, a_s.contiguous(), off, wt, wt_s, c, moe.OUT_F32)
    assert torch.equal(c.double(), _values(one, a_s) @ _values(wone[0], w_s[0]).t())

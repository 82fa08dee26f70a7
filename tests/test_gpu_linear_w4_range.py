"""4-bit products of bf16 without zero points at the ends of x's range.  The sums may be those of
the codes with 8 times the sum of x taken off; what the definition gives, code - 8 times x, must
come out all the same where x is infinite or missing, so large that only the codes' sums pass
fp32's range, or subnormal."""
import numpy as np
import pytest
import torch

from block_cases import BF, U, gen, group_offsets, n64, randn, sum_err
from mixture_experts_layer_dispatch_amd import binding as B
from oracle import around

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# (M, N, K, experts' rows, group): streams of 16, 32 and 64 columns, dense and grouped; tiles, whole and
# split reductions, dense and grouped
SIZES = [(5, 72, 256, None, 64), (20, 72, 96, None, 32), (9, 16384, 256, None, 128), (5, 65536, 128, None, 32),
         (30, 136, 384, [9, 0, 20], 128), (80, 520, 256, None, 32), (130, 72, 128, None, 128), (100, 136, 4096, None, 64),
         (90, 136, 8192, None, 128), (200, 264, 320, [70, 1, 120], 64), (300, 72, 4096, [170, 100], 32)]


def call(wc, x, codes, scales, bias, off, residual=None):
    y = torch.full((wc.M, wc.N), 7.0, dtype=BF, device="cuda") if residual is None else residual.clone()
    B.moe_linear_w4_forward(wc, x, codes, scales, y, B.alloc_linear_w4_workspace(wc), bias=bias,
                            residual=None if residual is None else y, offsets=off)
    return y


def case(M, N, K, counts, group, seed, act="none"):
    g = gen(seed)
    wc = B.LinearW4Config(M=M, N=N, K=K, E=len(counts) if counts else 0, group=group, act=act)
    cs, ss = wc.shapes
    codes = torch.randint(0, 256, cs, generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(ss, generator=g, device="cuda") + 0.5) * K ** -0.5).to(BF)
    off = group_offsets(counts) if counts else None
    rows = sum(counts) if counts else M
    return g, wc, randn(g, (M, K), BF), codes, scales, off, rows


def definition(wc, x, codes, scales, off, rows):
    """(sums by the definition, with IEEE's rules for infinities; magnitudes of the codes' sums; the largest
    sum of magnitudes of a group as the definition sums it)"""
    off = [0, rows] if off is None else off.tolist()
    w = around.w4_weights(codes.cpu().numpy(), np.ones_like(n64(scales)))
    s = n64(scales)
    w, s = (w[None], s[None]) if wc.E == 0 else (w, s)
    x = n64(x)
    z, mag, most = (np.zeros((rows, wc.N)) for _ in range(3))
    G = wc.group
    with np.errstate(invalid="ignore", over="ignore"):
        for e in range(len(w)):
            r = slice(off[e], off[e + 1])
            for i in range(wc.K // G):
                k = slice(i * G, (i + 1) * G)
                p = x[r, k] @ w[e][:, k].T
                # (a product of 0 and an infinity, or infinities of both signs, is NaN in any order)
                bad = ~np.isfinite(x[r, k]).all(1)
                if bad.any():
                    p[bad] = (x[r, k][bad][:, None, :] * w[e][None, :, k]).sum(2)
                m = np.abs(x[r, k]) @ np.abs(w[e][:, k]).T
                most[r] = np.maximum(most[r], m)
                z[r] += p * s[e][i]
                mag[r] += np.abs(np.where(np.isfinite(x[r, k]), x[r, k], 0)).sum(1)[:, None] * 16 * np.abs(s[e][i])
    return z, mag, most


def compare(y, z, mag, most, wc):
    """mag: of all that is summed."""
    y = n64(y)
    nan, inf = np.isnan(z), np.isinf(z)
    assert (np.isnan(y) == nan).all()
    assert (y[inf] == z[inf]).all()
    ok = ~nan & ~inf & (most < 2.0 ** 127)
    err = np.abs(np.where(ok, y, 0) - np.where(ok, z, 0))
    # the codes' sums, the sums of x, the groups; then bf16
    tol = sum_err(2 * wc.K + wc.K // wc.group + 4, mag)
    tol = (tol + U[BF] * np.abs(z) + 2.0 ** -134) * (1 + 2 * U[BF])
    assert (err <= np.where(ok, tol, INF)).all(), float((err - tol)[ok].max())
    return ok


@pytest.mark.parametrize("M,N,K,counts,group", SIZES)
def test_infinite_and_missing_x(M, N, K, counts, group):
    """x of +-inf where codes are 8 nowhere, then somewhere; NaN; rows beside them keep their bits."""
    g, wc, x, codes, scales, off, rows = case(M, N, K, counts, group, M + K)
    codes[..., 5] = torch.where(codes[..., 5] & 15 == 8, codes[..., 5] + 1, codes[..., 5])      # input 10: no code of 8
    good = call(wc, x, codes, scales, None, off)
    x2 = x.clone()
    x2[0, 10], x2[rows - 1, 10], x2[1, K - 1], x2[2, 3] = INF, -INF, INF, float("nan")
    bad = call(wc, x2, codes, scales, None, off)
    z, mag, most = definition(wc, x2, codes, scales, off, rows)
    assert np.isinf(z[0]).all() and np.isinf(z[rows - 1]).all()
    compare(bad[:rows], z, mag, np.where(np.isfinite(most), most, 0), wc)
    rest = [i for i in range(rows) if i not in (0, 1, 2, rows - 1)]
    assert torch.equal(good[rest], bad[rest])
    assert (bad[rows:] == 7).all()


@pytest.mark.parametrize("M,N,K,counts,group", SIZES)
def test_sums_of_codes_past_the_range(M, N, K, counts, group):
    """Two and three x of 2^124 in a group: 8 times their sum passes fp32's largest number, the sum of their
    code - 8 not everywhere."""
    g, wc, x, codes, scales, off, rows = case(M, N, K, counts, group, M + N)
    x[0] = 0
    x[0, 0] = x[0, group // 2] = 2.0 ** 124
    x[rows - 1] = 0
    x[rows - 1, K - group] = x[rows - 1, K - 2] = x[rows - 1, K - 1] = -2.0 ** 124
    r = torch.full((M, N), 3.0, dtype=BF, device="cuda")
    y = call(wc, x, codes, scales, None, off, residual=r)
    z, mag, most = definition(wc, x, codes, scales, off, rows)
    ok = compare(y[:rows], z + 3, mag + 3, most, wc)
    assert ok[0].any() and ok[rows - 1].any()
    assert (y[rows:] == 3).all()


@pytest.mark.parametrize("M,N,K,counts,group", SIZES)
def test_subnormal_x(M, N, K, counts, group):
    g, wc, x, codes, scales, off, rows = case(M, N, K, counts, group, N + K)
    x = (torch.randint(-127, 128, (M, K), generator=g, device="cuda").double() * 2.0 ** -133).to(BF)
    assert (x.float().abs() < 2.0 ** -126).all() and x.any()
    x[rows - 1] = torch.randint(1, 128, (K,), generator=g, device="cuda").double().mul(2.0 ** -133).to(BF)
    scales = (scales.float() * 2.0 ** 60).to(BF)
    y = call(wc, x, codes, scales, None, off)
    z, mag, most = definition(wc, x, codes, scales, off, rows)
    compare(y[:rows], z, mag, most, wc)


@pytest.mark.parametrize("M,N,K,counts,group", SIZES)
def test_rows_of_a_padded_batch(M, N, K, counts, group):
    """Rows that were never written: whatever bits. A NaN anywhere makes a row NaN, beside rows with infinities,
    and the others keep their bits."""
    g, wc, x, codes, scales, off, rows = case(M, N, K, counts, group, M * 3 + K)
    good = call(wc, x, codes, scales, None, off)
    x2 = x.clone()
    x2[rows // 2:].view(torch.int16).random_(-32768, 32767, generator=g)
    x2[rows // 2:, ::9] = float("nan")
    x2[0, K - 1], x2[1, 0] = float("nan"), INF
    x2[1, 1:].clamp_(-1, 1)
    bad = call(wc, x2, codes, scales, None, off)
    assert bad[0].isnan().all() and bad[rows // 2:rows].isnan().all()
    z, mag, most = definition(wc, x2[:2], codes if not wc.E else codes[:1], scales if not wc.E else scales[:1],
                              None if not wc.E else torch.tensor([0, 2]), 2)
    compare(bad[:2], z, mag, np.where(np.isfinite(most), most, 0), wc)
    assert torch.equal(good[2:rows // 2], bad[2:rows // 2])
    assert (bad[rows:] == 7).all()

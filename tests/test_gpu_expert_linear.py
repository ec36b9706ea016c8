"""expert_linear against its formula in 64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
# a product loses less than 2^-13 of the largest of its group of eight: 7 2^-13 of the sum
TILED = 2.0 ** -10


def case(seed, counts, T, K, N, bits, gather, gap=(0, 0)):
    """x, w (quantized), offsets and rows for segments of those lengths, with `gap` rows
    before and behind them."""
    g = torch.Generator().manual_seed(seed)
    E, R = len(counts), sum(counts) + sum(gap)
    T = T if gather else max(T, R)
    x = M.quantize(torch.randn(T, K, generator=g, dtype=torch.float64))
    w = M.quantize(torch.randn(E, N, K, generator=g, dtype=torch.float64) * K ** -0.5, bits)
    offsets = gap[0] + torch.tensor([0] + counts).cumsum(0)
    rows = torch.randint(0, T, (R,), generator=g, dtype=torch.int32) if gather else None
    return x, w, offsets.to(torch.int32), rows


def cuda(t):
    return tuple(v.cuda() for v in t) if isinstance(t, tuple) else None if t is None else t.cuda()


TILES = ["tile32", "tile64", "tile256"]


def check(x, w, offsets, rows, swiglu, out, what, kernel="auto"):
    R = x[0].shape[0] if rows is None else rows.shape[0]
    outs = w[0].shape[1] // (2 if swiglu else 1)
    if out == "bf16":
        y = torch.full((R, outs), 7.0, dtype=torch.bfloat16, device="cuda")
        ys = None
    else:
        y = torch.full((R, outs), 7, dtype=torch.uint8, device="cuda").view(M.E4M3)
        ys = torch.full((R, outs // 32), 7, dtype=torch.uint8, device="cuda").view(M.E8M0)
    got = tr.expert_linear(cuda(x), cuda(w), cuda(offsets), rows=cuda(rows), swiglu=swiglu, out=out, y=y, ys=ys,
                           kernel=kernel)
    want, err, inside = M.products(M.value(*x), M.value(*w), offsets, rows, swiglu,
                                   0.0 if kernel == "rows" else TILED)
    if out == "bf16":
        assert got is y
        M.check_rows(y, want, err, inside, what)
        assert (y.cpu()[~inside] == 7.0).all(), f"{what}: rows outside the segments"
    else:
        M.check_blocks((y[inside.cuda()], ys[inside.cuda()]), want[inside], err[inside], what)
        for t in (y, ys):
            assert (t.cpu().view(torch.uint8)[~inside] == 7).all(), f"{what}: rows outside the segments"
    return got


FORMS = [(False, "bf16"), (True, "bf16"), (False, "mx8"), (True, "mx8")]


@pytest.mark.parametrize("counts,T,K,N", [
    ([1], 1, 32, 64), ([0, 1, 0], 3, 96, 128), ([1, 1, 1, 1], 2, 512, 192), ([16, 15, 17, 1], 9, 160, 64),
    ([33, 0, 64, 5], 20, 256, 448), ([63, 65], 128, 1024, 64), ([2, 31, 32], 40, 2880, 192),
    ([100, 3, 260, 0, 1], 90, 384, 320), ([300], 300, 640, 512), ([129, 128, 127], 200, 224, 576),
    ([513, 0, 0, 70], 600, 288, 64), ([5, 0, 9], 14, 1024, 128), ([16], 7, 2880, 192), ([1], 1, 8480, 64),
    ([3, 4], 9, 544, 320), ([40, 24], 64, 768, 192),
])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("swiglu,out", FORMS)
def test_products(counts, T, K, N, bits, swiglu, out):
    """By every kernel that takes the sizes."""
    say(f"experts {counts} T={T} K={K} N={N} bits={bits} swiglu={swiglu} {out}")
    for gather in (False, True):
        x, w, offsets, rows = case(K + N, counts, T, K, N, bits, gather)
        for kernel in ["auto", "rows"] + (TILES if K >= 256 else []):
            check(x, w, offsets, rows, swiglu, out, f"gather={gather} {kernel}", kernel)


@pytest.mark.parametrize("counts,K,N,swiglu,out", [
    ([700], 256, 16384, False, "bf16"), ([300, 257, 0, 100], 320, 8192, True, "mx8"),
    ([90, 33, 200, 64], 512, 1024, True, "bf16"),
])
@pytest.mark.parametrize("bits", [8, 4])
def test_many_tiles(counts, K, N, swiglu, out, bits):
    """More than one tile a CU; what the rule chooses."""
    say(f"experts many {counts} K={K} N={N} bits={bits}")
    x, w, offsets, rows = case(K + N, counts, 90, K, N, bits, True)
    for kernel in ["auto"] + TILES:
        check(x, w, offsets, rows, swiglu, out, kernel, kernel)


def test_a_kernel_that_does_not_take_the_sizes():
    x, w, offsets, rows = case(1, [3], 3, 224, 64, 8, False)
    for kernel in TILES:
        with pytest.raises(tr.TopReduceError, match="does not take"):
            tr.expert_linear(cuda(x), cuda(w), cuda(offsets), kernel=kernel)
    with pytest.raises(ValueError):
        tr.expert_linear(cuda(x), cuda(w), cuda(offsets), kernel="other")


@pytest.mark.parametrize("N", [1, 2, 7, 30, 66, 250, 1001])
@pytest.mark.parametrize("counts", [[3, 0, 18], [5, 150]])
def test_odd_outputs(N, counts):
    for swiglu in (False, True):
        if N % 2 and swiglu:
            continue
        for K in (96, 320):
            x, w, offsets, rows = case(N, counts, 30, K, N, 8, True)
            for kernel in ["rows"] + (TILES if K >= 256 else []):
                check(x, w, offsets, rows, swiglu, "bf16", f"N={N} {kernel}", kernel)


@pytest.mark.parametrize("counts", [[4, 0, 9], [2, 200, 80]])
@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_rows_outside_the_segments_stay(counts, out):
    for gather in (False, True):
        x, w, offsets, rows = case(5, counts, 50, 256, 96, 8, gather, gap=(3, 40))
        for kernel in ["rows"] + TILES:
            check(x, w, offsets, rows, False, out, f"gather={gather} {kernel}", kernel)


@pytest.mark.parametrize("n", [6, 20, 300])
def test_offsets_and_rows_out_of_range_are_held_inside(n):
    x, w, _, rows = case(6, [n, n], 40, 256, 64, 8, True)
    rows[3], rows[7], rows[n] = -5, 1 << 30, 40
    for offsets in ([-9, n, 1 << 30], [0, n, n - 4], [2 * n, 2 * n, 2 * n], [5, 5, 9]):
        for kernel in ["rows"] + TILES:
            check(x, w, torch.tensor(offsets, dtype=torch.int32), rows, False, "bf16", f"{offsets} {kernel}", kernel)


@pytest.mark.parametrize("n", [5, 200])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kernel", ["rows"] + TILES)
def test_what_is_not_a_number_stays_in_its_row(n, bits, kernel):
    x, w, offsets, rows = case(7, [n, n], n, 288, 96, bits, True)
    args = cuda(w), cuda(offsets)
    clean = tr.expert_linear(cuda(x), *args, rows=cuda(rows), kernel=kernel).cpu()
    q = x[0].clone()
    q[2, 100] = float("nan")
    s = x[1].clone().view(torch.uint8)
    s[3, 1] = 255
    got = tr.expert_linear((q.cuda(), s.view(M.E8M0).cuda()), *args, rows=cuda(rows), kernel=kernel).cpu()
    bad = (rows == 2) | (rows == 3)
    assert bad.any() and torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])
    # a weight row: its output column, of its expert only
    ws = w[1].clone().view(torch.uint8)
    ws[1, 40, 3] = 255
    got = tr.expert_linear(cuda(x), (cuda(w)[0], ws.view(M.E8M0).cuda()), cuda(offsets), rows=cuda(rows),
                           kernel=kernel).cpu()
    hit = torch.zeros(2 * n, 96, dtype=torch.bool)
    hit[n:, 40] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("counts", [[1, 7], [90, 300]])
@pytest.mark.parametrize("kernel", ["rows"] + TILES)
def test_scales_of_any_size(counts, kernel):
    """Blocks whose scales lie 2^60 apart, and the same product scaled."""
    x, w, offsets, rows = case(8, counts, 60, 416, 64, 8, True)
    s = x[1].view(torch.uint8).clone()
    s[:, 1] -= 60
    x = (x[0], s.view(M.E8M0))
    y = check(x, w, offsets, rows, False, "bf16", "wide scales", kernel)
    up = ((x[1].view(torch.uint8) + 100).view(M.E8M0), (w[1].view(torch.uint8) - 90).view(M.E8M0))
    far = tr.expert_linear(cuda((x[0], up[0])), cuda((w[0], up[1])), cuda(offsets), rows=cuda(rows), kernel=kernel)
    assert torch.equal(far.double(), y.double() * 2.0 ** 10)


def test_nothing_to_do():
    x, w, offsets, _ = case(9, [0, 0, 0], 4, 64, 64, 8, False)
    y = torch.full((4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    tr.expert_linear(cuda(x), cuda(w), cuda(offsets), y=y)
    assert (y == 3).all()
    empty = (x[0][:0].cuda(), x[1][:0].cuda())
    assert tr.expert_linear(empty, cuda(w), cuda(offsets)).shape == (0, 64)


@pytest.mark.parametrize("counts", [[3, 1, 8], [200, 20, 70]])
@pytest.mark.parametrize("kernel", ["rows"] + TILES)
def test_order_of_rows_keeps_their_bits(counts, kernel):
    x, w, offsets, rows = case(10, counts, 64, 256, 128, 4, True)
    y = tr.expert_linear(cuda(x), cuda(w), cuda(offsets), rows=cuda(rows), kernel=kernel)
    perm = torch.cat([o + torch.randperm(n) for o, n in zip(offsets.tolist(), counts)])
    z = tr.expert_linear(cuda(x), cuda(w), cuda(offsets), rows=cuda(rows[perm]), kernel=kernel)
    assert torch.equal(z, y[perm.cuda()])

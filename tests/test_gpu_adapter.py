"""The shared projection with adapters (adapter_linear) against its formula in
64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(seed, T, H, N, R, A, dtype, run=1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, A + 1, (-(-T // run),), generator=g, dtype=torch.int32)  # -1 and A: none
    ids = ids.repeat_interleave(run)[:T].contiguous()
    return (S.inputs(g, T, H, dtype=dtype), S.inputs(g, N, H, dtype=dtype, std=H ** -0.5),
            S.inputs(g, A, R, H, dtype=dtype, std=H ** -0.5),
            S.inputs(g, A, N, R, dtype=dtype, std=R ** -0.5), ids,
            torch.rand(A, generator=g) * 2 - 0.5)


@pytest.mark.parametrize("T,H,N,R,A,run,dtype", [
    (1, 8, 1, 1, 1, 1, BF), (1, 3584, 512, 16, 8, 1, BF), (8, 264, 1000, 8, 3, 1, BF),
    (16, 256, 256, 12, 16, 1, BF), (17, 1032, 33, 64, 40, 1, BF), (33, 40, 130, 7, 5, 2, BF),
    (63, 512, 515, 100, 4, 5, BF), (64, 512, 256, 256, 64, 1, BF), (64, 136, 17, 33, 2, 64, BF),
    (65, 136, 17, 33, 2, 64, BF), (65, 256, 256, 16, 70, 1, BF), (130, 264, 129, 12, 3, 7, BF),
    (257, 512, 512, 32, 5, 50, BF), (300, 1032, 250, 64, 8, 1, BF), (512, 128, 260, 65, 9, 128, BF),
    (513, 2880, 1001, 256, 4, 100, BF), (1024, 512, 768, 16, 4, 300, BF),
    (1, 256, 128, 8, 8, 1, F32), (9, 264, 77, 5, 3, 1, F32), (64, 72, 256, 64, 9, 3, F32),
    (65, 40, 130, 3, 2, 9, F32), (200, 1448, 301, 12, 5, 40, F32), (256, 256, 256, 256, 3, 1, F32),
])
def test_against_the_formula(T, H, N, R, A, run, dtype):
    say(f"adapter T={T} H={H} N={N} R={R} A={A} run={run} {dtype}")
    x, w, a, b, ids, scales = make(T + N, T, H, N, R, A, dtype, run)
    for s in (scales, None):
        y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(),
                              scales=None if s is None else s.cuda())
        ref, bound = S.adapter(x, w, a, b, ids, s)
        S.check(y, ref, bound, f"scales {s is not None}")


@pytest.mark.parametrize("T,H,N,R,A,run", [
    (4096, 128, 8192, 8, 5, 1000), (4090, 256, 8192, 16, 3, 256), (8191, 128, 4096, 40, 6, 333),
    (16385, 256, 2048, 64, 40, 1), (8000, 384, 4352, 24, 2, 31), (33000, 128, 1024, 256, 4, 5000),
])
def test_large_tiles_against_the_formula(T, H, N, R, A, run):
    """Shapes of the 256 x 256 tiles: row blocks of one adapter, of several, of
    none, and a short last tile. Checked on the first and last rows, on the rows
    around every 256th, and on some others."""
    say(f"adapter tiles T={T} H={H} N={N} R={R} A={A} run={run}")
    x, w, a, b, ids, scales = make(T + N, T, H, N, R, A, BF, run)
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    rows = {0, 1, T - 2, T - 1} | {t + d for t in range(256, T - 1, 1792) for d in (-1, 0, 31, 32, 127)}
    g = torch.Generator().manual_seed(T)
    rows |= set(torch.randint(0, T, (150,), generator=g).tolist())
    rows = torch.tensor(sorted(t for t in rows if t < T))
    # (the row sample is past 64 rows, so the bound has the low-rank product's rounding)
    ref, bound = S.adapter(x[rows], w, a, b, ids[rows], scales)
    S.check(y[rows.cuda()], ref, bound, "y")


@pytest.mark.parametrize("T", [5, 64, 100, 700])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_adapters_that_no_row_names_are_not_read(T, dtype):
    x, w, a, b, ids, scales = make(3, T, 256, 256, 16, 6, dtype)
    ids[ids == 2] = -7
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    a[2], b[2], scales[2] = float("nan"), float("nan"), float("nan")
    y2 = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    assert torch.equal(y, y2)
    # and one that some rows name reaches those rows only
    b[3] = float("nan")
    y3 = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    mine = (ids == 3).cuda()
    assert torch.equal(y[~mine], y3[~mine]) and torch.isnan(y3[mine]).all()


@pytest.mark.parametrize("run", [1, 50, 300])
def test_an_adapter_of_infinities_in_the_large_tiles(run):
    T, H, N, R, A = 4100, 128, 8192, 16, 4
    x, w, a, b, ids, scales = make(run, T, H, N, R, A, BF, run)
    call = lambda: tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda())  # noqa: E731
    y = call()
    b[1], a[2] = float("inf"), float("nan")
    y2 = call()
    theirs = ((ids == 1) | (ids == 2)).cuda()
    assert torch.equal(y[~theirs], y2[~theirs])
    assert not torch.isfinite(y2[theirs]).any()


@pytest.mark.parametrize("T", [20, 200])
def test_rows_with_nan_and_infinity_stay_apart(T):
    x, w, a, b, ids, scales = make(4, T, 264, 130, 20, 3, BF, run=3)
    call = lambda v: tr.adapter_linear(v.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda())  # noqa: E731
    y = call(x)
    bad = x.clone()
    bad[3, 7], bad[T - 1, 0] = float("nan"), float("inf")
    y2 = call(bad)
    assert torch.equal(y[4:T - 1], y2[4:T - 1]) and torch.equal(y[:3], y2[:3])
    assert torch.isnan(y2[3]).all() and not torch.isfinite(y2[T - 1]).any()


@pytest.mark.parametrize("T", [1, 30, 64, 90, 600])
def test_no_adapter_is_the_plain_projection(T):
    x, w, a, b, ids, _ = make(5, T, 512, 384, 16, 2, BF)
    none = torch.full_like(ids, -1)
    nan = torch.full_like(a, float("nan")), torch.full_like(b, float("nan"))
    y = tr.adapter_linear(x.cuda(), w.cuda(), nan[0].cuda(), nan[1].cuda(), none.cuda())
    ref, bound = S.adapter(x, w, a, b, none)
    S.check(y, ref, bound, "y")


@pytest.mark.parametrize("T", [12, 300])
def test_same_bits_in_a_dirty_workspace_on_another_stream_and_in_a_graph(T):
    x, w, a, b, ids, scales = (t.cuda() for t in make(6, T, 512, 512, 24, 5, BF, run=4))
    y = tr.adapter_linear(x, w, a, b, ids, scales=scales)
    ws = torch.full((tr.adapter_workspace_size(T, 512, 512, 24, 5),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.empty_like(y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tr.adapter_linear(x, w, a, b, ids, scales=scales, y=out, ws=ws, stream=s)
    s.synchronize()
    assert got is out and torch.equal(out, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tr.adapter_linear(x, w, a, b, ids, scales=scales, y=out, ws=ws)
    for _ in range(4):
        x.copy_(torch.randn(T, 512, device="cuda").to(BF))
        want = tr.adapter_linear(x, w, a, b, ids, scales=scales)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_outputs_past_four_gigabytes():
    """Rows of y past 2^32 bytes and elements past 2^31."""
    T, H, N, R, A = 70000, 64, 32768, 8, 2
    x, w, a, b, ids, scales = make(7, T, H, N, R, A, BF, run=1000)
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    rows = torch.tensor([0, 1, 32767, 65535, 65536, 65537, 69998, 69999])
    ref, bound = S.adapter(x[rows], w, a, b, ids[rows], scales)
    low, _ = S.adapter(x[rows], torch.zeros_like(w), a, b, ids[rows], scales)
    mag = (x[rows].double().abs() @ a.double().abs().amax(0).t()) @ b.double().abs().amax(0).t()
    S.check(y[rows.cuda()], ref, bound + S.U[BF] * mag * 2, "y")


@pytest.mark.parametrize("N", [256, 250])
def test_x_past_two_gigabytes(N):
    """Rows too far apart for 32-bit offsets: taken in their own order."""
    T, H, R, A = 300_007, 3584, 16, 3
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=BF)      # 2.15 GB
    _, w, a, b, _, scales = make(9, 1, H, N, R, A, BF)
    ids = (torch.arange(T) // 37 % (A + 1)).to(torch.int32) - 1
    y = tr.adapter_linear(x, w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    rows = torch.cat([torch.arange(40), torch.arange(T - 80, T), torch.randint(0, T, (60,))])
    ref, bound = S.adapter(x[rows.cuda()], w, a, b, ids[rows], scales)
    S.check(y[rows.cuda()], ref, bound, "y")


def test_rows_do_not_depend_on_their_order():
    """A shuffled batch gives the shuffled rows: requests' tokens may be mixed."""
    T, H, N, R, A = 5000, 256, 8192, 24, 7
    x, w, a, b, ids, scales = (t.cuda() for t in make(12, T, H, N, R, A, BF, run=60))
    y = tr.adapter_linear(x, w, a, b, ids, scales=scales)
    at = torch.randperm(T, generator=torch.Generator().manual_seed(5)).cuda()
    y2 = tr.adapter_linear(x[at].contiguous(), w, a, b, ids[at].contiguous(), scales=scales)
    assert torch.equal(y[at], y2)


@pytest.mark.parametrize("A", [3, 1023, 1024, 5000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_mixed_rows_of_few_and_of_many_adapters(A, dtype):
    T, H, N, R = 2100, 64, 1030, 8
    x, w, a, b, ids, scales = make(A, T, H, N, R, A, dtype, run=1)
    ids[5], ids[2099], ids[2047], ids[2048] = A, A - 1, A - 1, -7
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    ref, bound = S.adapter(x, w, a, b, ids, scales)
    S.check(y, ref, bound, "y")


@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("H,N,dtype", [(7168, 7160, BF), (7176, 6001, BF), (4104, 8200, F32)])
def test_few_tokens_of_long_weights(T, H, N, dtype):
    R, A = 20, 3
    x, w, a, b, ids, scales = make(T, T, H, N, R, A, dtype, run=1)
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    ref, bound = S.adapter(x, w, a, b, ids, scales)
    S.check(y, ref, bound, "y")


def test_adapters_past_four_gigabytes():
    """The last adapter's rows of b lie past 2^32 bytes."""
    T, H, N, R, A = 3, 64, 4096, 256, 2100
    g = torch.Generator().manual_seed(8)
    x, w = S.inputs(g, T, H, dtype=BF), S.inputs(g, N, H, dtype=BF, std=H ** -0.5)
    a1, b1 = S.inputs(g, R, H, dtype=BF, std=H ** -0.5), S.inputs(g, N, R, dtype=BF, std=R ** -0.5)
    a = torch.zeros(A, R, H, dtype=BF, device="cuda")
    b = torch.zeros(A, N, R, dtype=BF, device="cuda")      # 4.4 GB
    a[A - 1], b[A - 1] = a1.cuda(), b1.cuda()
    for rows in (T, 100):
        xs = x.repeat(rows // T + 1, 1)[:rows].contiguous()
        ids = torch.full((rows,), A - 1, dtype=torch.int32)
        y = tr.adapter_linear(xs.cuda(), w.cuda(), a, b, ids.cuda())
        ref, bound = S.adapter(xs, w, a1[None], b1[None], ids - (A - 1))
        S.check(y, ref, bound, f"{rows} rows")


def test_no_rows():
    x, w, a, b, ids, _ = make(1, 1, 64, 32, 4, 2, BF)
    y = tr.adapter_linear(x[:0].cuda(), w.cuda(), a.cuda(), b.cuda(), ids[:0].cuda())
    assert y.shape == (0, 32)


def test_refusals():
    x, w, a, b, ids, scales = (t.cuda() for t in make(1, 4, 64, 64, 4, 2, BF))
    with pytest.raises(tr.TopReduceError):
        tr.adapter_linear(x, w, a, b, ids, y=x)      # y over x
    with pytest.raises(tr.TopReduceError):
        tr.adapter_linear(x, w, a, b, ids, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    big = torch.zeros(2, 257, 64, dtype=BF, device="cuda")
    with pytest.raises(tr.TopReduceError):
        tr.adapter_linear(x, w, big, torch.zeros(2, 64, 257, dtype=BF, device="cuda"), ids)
    with pytest.raises(TypeError):
        tr.adapter_linear(x, w, a, b, ids.long())
    with pytest.raises(TypeError):
        tr.adapter_linear(x, w.float(), a, b, ids)
    with pytest.raises(ValueError):
        tr.adapter_linear(x, w, a, b[:, :32].contiguous(), ids)
    with pytest.raises(ValueError):
        tr.adapter_linear(x, w, a, b, ids[:3])
    with pytest.raises(ValueError):
        tr.adapter_linear(x, w, a, b, ids, scales=scales[:1])
    with pytest.raises(ValueError):
        tr.adapter_linear(x, w, a.transpose(1, 2).contiguous().transpose(1, 2), b, ids)

"""moe_grouped_gemm and moe_grouped_gemm_wgrad against float64 products."""
import pytest
import torch

from tests import ops_ref as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_mixture_experts_prefix_amd")
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def normal(shape, seed, std=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def offsets_of(sizes, start=0):
    o = [start]
    for n in sizes:
        o.append(o[-1] + n)
    return o


def e4m3(shape, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    w = torch.randn(shape, generator=g)
    scale = w.abs().amax(-1) / 448
    codes = (w / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def check_grouped(sizes, N, K, transposed=False, fp8=False, out=torch.float32, start=0, tail=0, seed=0):
    G = len(sizes)
    off = offsets_of(sizes, start)
    R = off[-1] + tail
    x = normal((R, K), seed)
    scale = None
    if fp8:
        w, scale = e4m3((G, N, K), seed + 1)
    else:
        w = normal((G, K, N) if transposed else (G, N, K), seed + 1, 0.05)
    y0, s = ref.grouped(x, off, w, transposed, scale)
    x[:start] = float("nan")  # rows of no group are not read
    if tail:
        x[off[-1]:] = float("inf")
    buf = torch.full((R + 2, N), -7.0, dtype=out, device=DEV)
    y = buf[1:R + 1]
    moe.moe_grouped_gemm(x.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), w.to(DEV),
                         w_scale=None if scale is None else scale.to(DEV), transposed=transposed, y=y)
    torch.cuda.synchronize()
    got = buf.cpu()
    inside = ~y0.isnan()
    outside = torch.cat([torch.ones((1, N), dtype=torch.bool), ~inside, torch.ones((1, N), dtype=torch.bool)])
    assert (got[outside] == -7).all(), "rows of no group were written"
    bound = ref.product_bound(s, K, y0 if out == torch.bfloat16 else None)
    if fp8:
        bound = bound + ref.U32 * y0.abs()  # the scale's product
    ref.assert_within(got[1:R + 1][inside], y0[inside], bound[inside],
                      "sizes %s N %d K %d" % (sizes, N, K))


SIZES = [
    [1], [0, 1, 0], [3, 0, 5, 1], [16, 17, 1, 0, 15], [20] * 8, [33, 31, 48, 32], [64, 65, 63],
    [100, 0, 255, 1], [256, 257], [288, 289, 0, 512], [700, 3, 0, 290], [1500],
]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("form", ["nk", "kn", "e4m3"])
def test_group_sizes(sizes, form):
    check_grouped(sizes, 264, 328, transposed=form == "kn", fp8=form == "e4m3", seed=len(sizes))


@pytest.mark.parametrize("N,K", [(8, 8), (16, 64), (8, 1024), (1032, 8), (520, 136), (256, 256), (64, 2880)])
@pytest.mark.parametrize("form", ["nk", "kn", "e4m3"])
@pytest.mark.parametrize("rows", [5, 40, 300])
def test_widths(N, K, form, rows):
    check_grouped([rows, 0, 2 * rows + 1], N, K, transposed=form == "kn", fp8=form == "e4m3", seed=rows)


@pytest.mark.parametrize("form", ["nk", "kn", "e4m3"])
@pytest.mark.parametrize("sizes", [[3, 4], [40, 30], [300, 1, 70]], ids=str)
def test_bf16_rows(form, sizes):
    check_grouped(sizes, 272, 192, transposed=form == "kn", fp8=form == "e4m3", out=torch.bfloat16)


@pytest.mark.parametrize("form", ["nk", "kn", "e4m3"])
@pytest.mark.parametrize("sizes", [[3, 0, 4], [40, 30], [300, 0, 70]], ids=str)
def test_rows_of_no_group_stay(form, sizes):
    for out in (torch.float32, torch.bfloat16):
        check_grouped(sizes, 72, 80, transposed=form == "kn", fp8=form == "e4m3", out=out, start=3, tail=37)


def test_many_groups():
    g = torch.Generator()
    g.manual_seed(3)
    for top in (2, 9, 120):
        sizes = torch.randint(0, top, (256,), generator=g).tolist()
        for form in ("nk", "kn", "e4m3"):
            check_grouped(sizes, 24, 72, transposed=form == "kn", fp8=form == "e4m3", seed=top)


@pytest.mark.parametrize("form", ["nk", "kn", "e4m3"])
def test_one_group_holds_all_rows_of_a_few_row_call(form):
    """Mean rows per group say few-row tiles, one group has them all."""
    check_grouped([0] * 20 + [390] + [0] * 11, 136, 264, transposed=form == "kn", fp8=form == "e4m3")
    check_grouped([1200] + [0] * 31, 136, 264, transposed=form == "kn", fp8=form == "e4m3")


def test_few_tiles_and_a_long_sum():
    """Few output tiles over a long K (the tiles are cut along K)."""
    for form in ("nk", "kn", "e4m3"):
        check_grouped([256, 130], 512, 4160, transposed=form == "kn", fp8=form == "e4m3")


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-4, 4, 9, 9], [0, 4, 99, 12], [9, 2, 2, 2],
                                     [2 ** 31 - 1, -2 ** 31, 3, 2 ** 31 - 1]], ids=str)
@pytest.mark.parametrize("rows", [12, 600])
def test_offsets_are_clamped(offsets, rows):
    """Offsets outside [0, R] or descending stay inside the tensors; groups that do
    not overlap another are right, and the rows of no group untouched."""
    N, K, G = 40, 64, 3
    off = [o * rows // 12 if abs(o) < 1000 else o for o in offsets]
    x, w = normal((rows, K), 1), normal((G, N, K), 2)
    y0, s = ref.grouped(x, off, w)
    count = torch.zeros(rows, dtype=torch.int64)
    for g in range(G):
        a, b = ref.rows_of(off, g, rows)
        count[a:b] += 1
    for transposed in (False, True):
        buf = torch.full((rows + 2, N), -7.0, device=DEV)
        wd = w.transpose(1, 2).contiguous() if transposed else w
        moe.moe_grouped_gemm(x.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), wd.to(DEV),
                             transposed=transposed, y=buf[1:rows + 1])
        got = buf.cpu()
        assert (got[0] == -7).all() and (got[-1] == -7).all()
        assert (got[1:-1][count == 0] == -7).all()
        one = count == 1
        ref.assert_within(got[1:-1][one], y0[one], ref.product_bound(s, K)[one])


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_wgrad_group_sizes(sizes):
    check_wgrad(sizes, 264, 136, seed=len(sizes))


@pytest.mark.parametrize("N,K", [(8, 8), (16, 600), (1032, 8), (256, 256), (520, 264)])
def test_wgrad_widths(N, K):
    check_wgrad([70, 0, 131, 1], N, K)


def check_wgrad(sizes, N, K, start=2, tail=5, seed=0):
    off = offsets_of(sizes, start)
    R = off[-1] + tail
    dy, x = normal((R, N), seed, 0.1), normal((R, K), seed + 1)
    dw0, s, n = ref.grouped_wgrad(dy, x, off)
    for t in (dy, x):  # rows of no group are not read
        t[:start] = float("nan")
        t[off[-1]:] = float("inf")
    buf = torch.full((len(sizes) * N * K + 16,), -7.0, device=DEV)
    dw = buf[8:-8].view(len(sizes), N, K)
    moe.moe_grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), dw=dw)
    torch.cuda.synchronize()
    assert (buf[:8] == -7).all() and (buf[-8:] == -7).all()
    for g, rows in enumerate(n):
        if rows == 0:
            assert (dw[g] == 0).all()
        ref.assert_within(dw[g], dw0[g], ref.product_bound(s[g], rows), "group %d" % g)


def test_wgrad_many_groups():
    g = torch.Generator()
    g.manual_seed(5)
    check_wgrad(torch.randint(0, 9, (256,), generator=g).tolist(), 24, 40)


@pytest.mark.parametrize("sizes,N,K", [([2000], 264, 136), ([1500, 0, 701, 33], 72, 520), ([1, 640, 129], 136, 136),
                                       ([300] * 9, 1032, 1032), ([513, 0, 129, 777], 1544, 1544)])
def test_wgrad_few_and_many_tiles(sizes, N, K):
    """Both sides of the choice of tiles by how many there are, over many rows."""
    check_wgrad(sizes, N, K, seed=N)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = normal((2, 32, 64), 0).to(DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert moe.moe_grouped_gemm(x, off, w).shape == (0, 32)
    dy = torch.empty((0, 32), dtype=torch.bfloat16, device=DEV)
    assert (moe.moe_grouped_gemm_wgrad(dy, x, off) == 0).all()


@pytest.mark.parametrize("sizes", [[2, 3, 0, 1], [300, 0, 40]], ids=str)
def test_gradients_are_the_differences(sizes):
    """y is linear in x and in w: with values on a coarse grid every product and sum
    is exact, and differences of <dy, y> equal the gradients' products exactly."""
    g = torch.Generator()
    g.manual_seed(9)
    N, K, G = 72, 80, len(sizes)
    off = torch.tensor(offsets_of(sizes), dtype=torch.int32, device=DEV)
    R = int(off[-1])

    def grid(shape):
        return (torch.randint(-4, 5, shape, generator=g).float() / 8).to(torch.bfloat16).to(DEV)

    x, w, dy, ex, ew = grid((R, K)), grid((G, N, K)), grid((R, N)), grid((R, K)), grid((G, N, K))
    dx = moe.moe_grouped_gemm(dy, off, w, transposed=True)
    dw = moe.moe_grouped_gemm_wgrad(dy, x, off)

    def loss(xx, ww):
        return (moe.moe_grouped_gemm(xx, off, ww).double() * dy.double()).sum()

    assert loss(x + ex, w) - loss(x - ex, w) == 2 * (dx.double() * ex.double()).sum()
    assert loss(x, w + ew) - loss(x, w - ew) == 2 * (dw.double() * ew.double()).sum()


@pytest.mark.parametrize("sizes", [[5, 0, 9], [300, 0, 260, 31]], ids=str)
def test_repeats_are_bitwise_equal(sizes):
    """Also with a workspace full of NaN patterns, and on another stream."""
    off = torch.tensor(offsets_of(sizes), dtype=torch.int32, device=DEV)
    R, N, K = int(off[-1]), 520, 1096
    x, dy = normal((R, K), 1).to(DEV), normal((R, N), 2).to(DEV)
    w = normal((len(sizes), N, K), 3).to(DEV)
    wt = w.transpose(1, 2).contiguous()
    n = moe.moe_grouped_gemm_workspace_size(x, w)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((max(n, 1),), fill, dtype=torch.uint8, device=DEV)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            out = (moe.moe_grouped_gemm(x, off, w, workspace=ws),
                   moe.moe_grouped_gemm(x, off, wt, transposed=True, workspace=ws.clone()),
                   moe.moe_grouped_gemm_wgrad(dy, x, off))
        torch.cuda.synchronize()
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("rows", [12, 700])
def test_graph_replays_match_eager(rows):
    """The offsets are read on the device: a replay follows new ones."""
    G, N, K = 4, 264, 640
    x, dy, w = normal((rows, K), 1).to(DEV), normal((rows, N), 2).to(DEV), normal((G, N, K), 3).to(DEV)
    off = torch.tensor([0, 1, 2, 3, rows], dtype=torch.int32, device=DEV)
    ws = torch.empty(max(moe.moe_grouped_gemm_workspace_size(x, w), 1), dtype=torch.uint8, device=DEV)
    y, dx = torch.empty((rows, N), device=DEV), torch.empty((rows, K), device=DEV)
    wsx = torch.empty(max(moe.moe_grouped_gemm_workspace_size(dy, w, transposed=True), 1), dtype=torch.uint8,
                      device=DEV)
    dw = torch.empty((G, N, K), device=DEV)

    def step(y, dx, dw, ws, wsx):
        moe.moe_grouped_gemm(x, off, w, y=y, workspace=ws)
        moe.moe_grouped_gemm(dy, off, w, transposed=True, y=dx, workspace=wsx)
        moe.moe_grouped_gemm_wgrad(dy, x, off, dw=dw)

    step(y, dx, dw, ws, wsx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(y, dx, dw, ws, wsx)
    for r in range(3):
        x.copy_(normal((rows, K), 10 + r).to(DEV))
        cuts = [0, rows // (r + 3), rows // 2, rows // 2, rows]
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e = [torch.empty_like(t) for t in (y, dx, dw)]
        step(*e, torch.empty_like(ws), torch.empty_like(wsx))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), e)), r


def test_no_rows_fill_more_than_a_grid_of_threads():
    """A call without rows writes zeros over all of dw, also past 2^32 elements."""
    G, N, K = 9, 23160, 23160
    dw = torch.ones((G, N, K), device=DEV)
    e = torch.empty((0, N), dtype=torch.bfloat16, device=DEV), torch.empty((0, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_wgrad(*e, torch.zeros(G + 1, dtype=torch.int32, device=DEV), dw=dw)
    assert all(not dw[g].any() for g in range(G))

"""moe_lora_forward and moe_lora_backward against float64 products."""
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


def make(T, D, N, L, r, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)

    def normal(shape, std):
        return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)

    return dict(x=normal((T, D), 1.0), w=normal((N, D), 0.05), a=normal((L, r, D), D ** -0.5),
                b=normal((L, N, r), 0.1), scale=torch.rand(L, generator=g) + 0.5, dy=normal((T, N), 0.1))


def adapters(kind, T, L, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    t = torch.arange(T)
    if kind == "one":
        ad = torch.full((T,), L - 1)
    elif kind == "none":
        ad = torch.full((T,), -1)
    elif kind == "mixed":  # every row its own draw, some without, some ids past the last
        ad = torch.randint(-1, L + 1, (T,), generator=g)
        ad[torch.rand(T, generator=g) < 0.05] = 2 ** 31 - 1
        ad[torch.rand(T, generator=g) < 0.05] = -2 ** 31
    else:  # runs of rows
        ad = torch.randint(-1, L, ((T + 36) // 37,), generator=g).repeat_interleave(37)[:T]
    return ad.to(torch.int32) + 0 * t.to(torch.int32)


def check(T, D, N, L, r, kind, out=torch.bfloat16, scale=True, seed=0, backward=True):
    m = make(T, D, N, L, r, seed)
    ad = adapters(kind, T, L, seed + 1)
    sc = m["scale"] if scale else None
    want = ref.lora(m["x"], m["w"], m["a"], m["b"], ad, sc)
    used = {int(v) for v in ad.tolist()}
    a, b = m["a"].clone(), m["b"].clone()
    for l in range(L):
        if l not in used:  # adapters that no row names are not read
            a[l], b[l] = float("nan"), float("inf")
    d = {k: v.to(DEV) for k, v in dict(x=m["x"], w=m["w"], a=a, b=b, ad=ad, dy=m["dy"]).items()}
    dsc = None if sc is None else sc.to(DEV)
    buf = torch.full((T + 2, N), -7.0, dtype=out, device=DEV)
    xa = torch.full((T, r), float("nan"), device=DEV)
    moe.moe_lora_forward(d["x"], d["w"], d["a"], d["b"], d["ad"], dsc, y=buf[1:T + 1], xa=xa)
    assert (buf[0] == -7).all() and (buf[-1] == -7).all()
    bound = ref.product_bound(want["s"], D + 2 * r) + want["parts"]
    if out == torch.bfloat16:
        bound = bound + ref.HALF_BF16 * (want["y"].abs() + bound)
    ref.assert_within(buf[1:T + 1], want["y"], bound, "y")
    ref.assert_within(xa, want["xa"], ref.product_bound(want["sxa"], D), "xa")
    y2 = moe.moe_lora_forward(d["x"], d["w"], d["a"], d["b"], d["ad"], dsc, out_dtype=out)
    assert torch.equal(y2, buf[1:T + 1])  # the same without keeping xa
    if not backward:
        return
    g0 = ref.lora_backward(m["x"], m["w"], m["a"], m["b"], ad, sc, m["dy"], xa)
    g = moe.moe_lora_backward(d["x"], d["w"], d["a"], d["b"], d["ad"], d["dy"], xa, dsc, out_dtype=out)
    dxb = g0["dx_bound"]
    if out == torch.bfloat16:
        dxb = dxb + ref.HALF_BF16 * (g0["dx"].abs() + dxb)
    ref.assert_within(g["dx"], g0["dx"], dxb, "dx")
    ref.assert_within(g["da"], g0["da"], g0["da_bound"], "da")
    ref.assert_within(g["db"], g0["db"], g0["db_bound"], "db")
    for l in range(L):
        if l not in used:
            assert (g["da"][l] == 0).all() and (g["db"][l] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 48, 64, 65, 100, 257, 300, 700])
@pytest.mark.parametrize("kind", ["one", "none", "mixed", "runs"])
def test_rows(T, kind):
    check(T, 328, 264, 5, 16, kind, seed=T)


@pytest.mark.parametrize("T,L,r", [(65, 6, 128), (66, 2, 8), (128, 5, 64), (129, 4, 120), (193, 30, 40),
                                   (255, 30, 128), (256, 5, 16), (256, 4, 64), (256, 4, 72)])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_more_rows_than_a_tile_of_64(T, L, r, kind):
    """Both sides of the choice between the few rows' launches and the 256-row tiles."""
    check(T, 1096, 264, L, r, kind, seed=r)
    check(T, 264, 1096, L, r, kind, out=torch.float32, seed=T)


@pytest.mark.parametrize("T,L,r", [(257, 30, 120), (300, 30, 128), (513, 6, 64), (600, 30, 64), (1024, 5, 32),
                                   (1025, 5, 32), (1100, 256, 8), (1100, 40, 16)])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_many_adapters_in_a_tile_of_256_rows(T, L, r, kind):
    """Both sides of that choice for more rows; tiles that hold 2 to 256 adapters."""
    check(T, 136, 264, L, r, kind, seed=r)
    check(T, 264, 136, L, r, kind, out=torch.float32, seed=T)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("T", [9, 300])
def test_ranks(T, r):
    check(T, 264, 392, 4, r, "mixed", seed=r)
    check(T, 264, 392, 4, r, "runs", out=torch.float32, seed=r)


@pytest.mark.parametrize("D,N", [(8, 8), (8, 1032), (1032, 8), (64, 64), (2880, 72), (72, 2880), (136, 520)])
@pytest.mark.parametrize("T", [3, 70, 270])
def test_widths(T, D, N):
    check(T, D, N, 3, 8, "mixed", out=torch.float32)


@pytest.mark.parametrize("T", [7, 40, 290])
def test_no_scale(T):
    check(T, 128, 136, 3, 16, "runs", scale=False)


@pytest.mark.parametrize("T", [1, 20, 100, 300])
def test_nothing_of_an_unnamed_adapter_is_read(T):
    """Not its scale either: gradients of adapters without rows are zeros."""
    D, N, L, r = 72, 136, 6, 8
    m = {k: v.to(DEV) for k, v in make(T, D, N, L, r).items()}
    ad = (torch.arange(T, dtype=torch.int32, device=DEV) % 3) * 2  # 0, 2, 4
    for l in range(L):
        if l not in set(ad.tolist()):
            m["a"][l] = m["b"][l] = m["scale"][l] = float("nan")
    xa = torch.empty((T, r), device=DEV)
    y = moe.moe_lora_forward(m["x"], m["w"], m["a"], m["b"], ad, m["scale"], xa=xa)
    g = moe.moe_lora_backward(m["x"], m["w"], m["a"], m["b"], ad, m["dy"], xa, m["scale"])
    assert all(torch.isfinite(v).all() for v in (y, xa, g["dx"], g["da"], g["db"]))
    for l in range(L):
        if l not in set(ad.tolist()):
            assert (g["da"][l] == 0).all() and (g["db"][l] == 0).all()


@pytest.mark.parametrize("T", [64, 600])
def test_many_adapters(T):
    check(T, 72, 80, 256, 8, "mixed", out=torch.float32)
    check(T, 72, 80, 3000, 8, "mixed", backward=False)


def test_few_tiles_and_a_long_sum():
    check(300, 4160, 520, 3, 32, "runs", out=torch.float32)


@pytest.mark.parametrize("T", [16, 64, 300, 600])
def test_an_adapter_with_nan_reaches_its_own_rows_only(T):
    D, N, L, r = 136, 264, 4, 16
    m = make(T, D, N, L, r)
    ad = adapters("mixed", T, L, 3)
    clean = moe.moe_lora_forward(*[m[k].to(DEV) for k in "xwab"], ad.to(DEV), m["scale"].to(DEV))
    xa = torch.zeros((T, r), device=DEV)
    moe.moe_lora_forward(*[m[k].to(DEV) for k in "xwab"], ad.to(DEV), m["scale"].to(DEV), xa=xa)
    g_clean = moe.moe_lora_backward(*[m[k].to(DEV) for k in "xwab"], ad.to(DEV), m["dy"].to(DEV), xa,
                                    m["scale"].to(DEV))
    m["a"][2] = float("nan")
    m["b"][2] = float("inf")
    y = moe.moe_lora_forward(*[m[k].to(DEV) for k in "xwab"], ad.to(DEV), m["scale"].to(DEV))
    g = moe.moe_lora_backward(*[m[k].to(DEV) for k in "xwab"], ad.to(DEV), m["dy"].to(DEV), xa,
                              m["scale"].to(DEV))
    others = (ad != 2).to(DEV)
    assert torch.equal(y[others], clean[others])
    assert torch.equal(g["dx"][others], g_clean["dx"][others])
    for name in ("da", "db"):
        assert torch.equal(g[name][[0, 1, 3]], g_clean[name][[0, 1, 3]])


def test_no_rows():
    m = make(0, 64, 72, 2, 8)
    d = [m[k].to(DEV) for k in "xwab"]
    ad = torch.empty(0, dtype=torch.int32, device=DEV)
    assert moe.moe_lora_forward(*d, ad).shape == (0, 72)
    g = moe.moe_lora_backward(*d, ad, m["dy"].to(DEV), torch.empty((0, 8), device=DEV))
    assert (g["da"] == 0).all() and (g["db"] == 0).all() and g["dx"].shape == (0, 64)


@pytest.mark.parametrize("T", [12, 300])
def test_gradients_are_the_differences(T):
    """With values on a coarse grid the sums are exact: <dy, y> is linear in A, in B
    and in x, and its differences equal the gradients' products."""
    g = torch.Generator()
    g.manual_seed(11)
    D, N, L, r = 40, 48, 3, 8

    def grid(shape):
        return (torch.randint(-2, 3, shape, generator=g).float() / 4).to(torch.bfloat16).to(DEV)

    x, w, a, b, dy = grid((T, D)), grid((N, D)), grid((L, r, D)), grid((L, N, r)), grid((T, N))
    ex, ea, eb = grid((T, D)), grid((L, r, D)), grid((L, N, r))
    ad = adapters("mixed", T, L, 4).to(DEV)
    sc = torch.tensor([0.5, 2.0, -1.0], device=DEV)
    xa = torch.empty((T, r), device=DEV)
    moe.moe_lora_forward(x, w, a, b, ad, sc, xa=xa)
    gr = moe.moe_lora_backward(x, w, a, b, ad, dy, xa, sc)

    def loss(x=x, a=a, b=b):
        return (moe.moe_lora_forward(x, w, a, b, ad, sc, out_dtype=torch.float32).double() * dy.double()).sum()

    for name, e, plus, minus in (("dx", ex, dict(x=x + ex), dict(x=x - ex)), ("da", ea, dict(a=a + ea), dict(a=a - ea)),
                                 ("db", eb, dict(b=b + eb), dict(b=b - eb))):
        assert loss(**plus) - loss(**minus) == 2 * (gr[name].double() * e.double()).sum(), name


@pytest.mark.parametrize("T", [20, 64, 400])
def test_repeats_are_bitwise_equal(T):
    D, N, L, r = 1096, 520, 6, 24
    m = make(T, D, N, L, r)
    d = [m[k].to(DEV) for k in "xwab"]
    ad, sc, dy = adapters("runs", T, L).to(DEV), m["scale"].to(DEV), m["dy"].to(DEV)
    n, nb = moe.moe_lora_workspace_size(*d[:3]), moe.moe_lora_backward_workspace_size(*d[:3])
    first = None
    for fill in (0, 255, 127):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            xa = torch.empty((T, r), device=DEV)
            y = moe.moe_lora_forward(*d, ad, sc, xa=xa,
                                     workspace=torch.full((max(n, 1),), fill, dtype=torch.uint8, device=DEV))
            g = moe.moe_lora_backward(*d, ad, dy, xa, sc,
                                      workspace=torch.full((max(nb, 1),), fill, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        out = (y, xa, g["dx"], g["da"], g["db"])
        first = first or out
        assert all(torch.equal(p, q) for p, q in zip(first, out))


@pytest.mark.parametrize("T", [20, 400])
def test_graph_replays_match_eager(T):
    """The adapters are read on the device: a replay follows new ones."""
    D, N, L, r = 264, 328, 5, 16
    m = make(T, D, N, L, r)
    x, w, a, b = [m[k].to(DEV) for k in "xwab"]
    ad, sc, dy = adapters("runs", T, L).to(DEV), m["scale"].to(DEV), m["dy"].to(DEV)

    def bufs():
        return dict(y=torch.empty((T, N), dtype=torch.bfloat16, device=DEV), xa=torch.empty((T, r), device=DEV),
                    ws=torch.empty(max(moe.moe_lora_workspace_size(x, w, a), 1), dtype=torch.uint8, device=DEV),
                    wb=torch.empty(max(moe.moe_lora_backward_workspace_size(x, w, a), 1), dtype=torch.uint8, device=DEV),
                    g=dict(dx=torch.empty((T, D), device=DEV), da=torch.empty((L, r, D), device=DEV),
                           db=torch.empty((L, N, r), device=DEV)))

    def step(q):
        moe.moe_lora_forward(x, w, a, b, ad, sc, y=q["y"], xa=q["xa"], workspace=q["ws"])
        moe.moe_lora_backward(x, w, a, b, ad, dy, q["xa"], sc, grads=q["g"], workspace=q["wb"])

    q = bufs()
    step(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q)
    for i in range(3):
        ad.copy_(adapters(["mixed", "runs", "one"][i], T, L, 20 + i).to(DEV))
        x.copy_(make(T, D, N, L, r, 30 + i)["x"].to(DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e = bufs()
        step(e)
        torch.cuda.synchronize()
        assert torch.equal(q["y"], e["y"]) and torch.equal(q["xa"], e["xa"]), i
        assert all(torch.equal(q["g"][k], e["g"][k]) for k in e["g"]), i

"""moe_orthogonalize against float64 Newton-Schulz steps.

Bars: RMS_BAR and MAX_BAR of tests/test_ops_tolerances.py, where the kernel's
roundings are emulated on matrices whose elements are a few times their RMS.  An
element far above the RMS also has its own roundings: half a bf16 step of its
value, 2^-8, and in each of five steps Q's half fp16 step (|Q| <= 2.81: 5 * 2.81 *
2^-12 < 2^-8)."""
import pytest
import torch

from tests import ops_ref as ref
from tests.test_ops_tolerances import MAX_BAR, RMS_BAR, gradients

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_mixture_experts_prefix_amd")
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def check(g, steps=5, eps=1e-7):
    want = ref.orthogonalize(g, steps, eps)
    E, M, N = g.shape
    buf = torch.full((E * M * N + 16,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:-8].view(E, M, N)
    moe.moe_orthogonalize(g.to(DEV), steps=steps, eps=eps, out=out)
    torch.cuda.synchronize()
    assert (buf[:8] == -7).all() and (buf[-8:] == -7).all()
    for e in range(E):
        rms = want[e].square().mean().sqrt()
        err = (out[e].cpu().double() - want[e]).abs()
        if rms == 0:
            assert err.max() == 0
            continue
        assert err.square().mean().sqrt() <= RMS_BAR * rms, (e, float(err.square().mean().sqrt() / rms))
        assert (err <= MAX_BAR * rms + 2 * ref.HALF_BF16 * want[e].abs()).all(), (e, float(err.max() / rms))
    return out


@pytest.mark.parametrize("kind", ["random", "low_rank", "rank8", "decay"])
@pytest.mark.parametrize("M,N", [(64, 64), (128, 256), (256, 128), (264, 264), (520, 72)])
def test_kinds(kind, M, N):
    check(gradients(kind, 3, M, N))


@pytest.mark.parametrize("M,N", [(8, 8), (8, 1024), (1024, 8), (16, 40), (72, 136), (320, 336), (640, 264),
                                 (257 * 8, 24), (24, 257 * 8), (512, 768)])
def test_sizes(M, N):
    check(gradients("random", 2, M, N))


def test_one_matrix_of_few_tiles_and_a_long_side():
    check(gradients("low_rank", 1, 300 // 4 * 8, 4160))
    check(gradients("low_rank", 1, 4160, 300 // 4 * 8))


@pytest.mark.parametrize("steps", [1, 2, 6, 16])
def test_steps(steps):
    check(gradients("random", 2, 96, 160), steps=steps)


def test_many_matrices_and_both_input_types():
    g = gradients("random", 40, 40, 24)
    check(g)
    check(g.to(torch.bfloat16))


def test_zeros_and_scales():
    """A stack of unlike sizes: zeros (an expert without tokens) stay zeros, and the
    result does not depend on a gradient's scale, down to 1e-30 and up to 1e30."""
    g = gradients("random", 6, 128, 96)
    g[1] = 0
    g[2] *= 1e-27
    g[3] *= 1e33
    out = check(g, eps=0.0)
    assert (out[1] == 0).all()
    base = gradients("random", 6, 128, 96)
    one = moe.moe_orthogonalize((base[2:3] * 2.0 ** -80).to(DEV), eps=0.0)
    two = moe.moe_orthogonalize(base[2:3].to(DEV), eps=0.0)
    assert torch.equal(one, two)


def test_one_element_holds_the_norm():
    g = torch.zeros((1, 64, 128))
    g[0, 5, 7] = 3.0
    check(g)


def test_eps():
    check(gradients("random", 1, 64, 64) * 1e-6, eps=1e-3)


def test_a_matrix_with_nan_does_not_reach_the_others():
    g = gradients("random", 4, 136, 72)
    clean = moe.moe_orthogonalize(g.to(DEV))
    g[2, 3, 4] = float("nan")
    out = moe.moe_orthogonalize(g.to(DEV))
    assert torch.equal(out[[0, 1, 3]], clean[[0, 1, 3]])


def test_no_matrices():
    assert moe.moe_orthogonalize(torch.empty((0, 64, 64), device=DEV)).shape == (0, 64, 64)


def test_the_steps_orthogonalise():
    """The singular values of a well conditioned matrix come out near 1."""
    q = torch.linalg.qr(gradients("random", 1, 256, 128)[0].double())[0]
    g = (q * torch.linspace(0.3, 1.0, 128, dtype=torch.float64)).float()[None].contiguous()
    s = torch.linalg.svdvals(moe.moe_orthogonalize(g.to(DEV))[0].cpu().double())
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("M,N", [(264, 520), (520, 264), (64, 64)])
def test_repeats_are_bitwise_equal(M, N):
    g = gradients("random", 5, M, N).to(DEV)
    n = moe.moe_orthogonalize_workspace_size(g)
    first = None
    for fill in (0, 255, 127):
        out = moe.moe_orthogonalize(g, workspace=torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        first = out if first is None else first
        assert torch.equal(first, out)


def test_graph_replays_match_eager():
    g = gradients("random", 4, 264, 136).to(DEV)
    ws = torch.empty(moe.moe_orthogonalize_workspace_size(g), dtype=torch.uint8, device=DEV)
    out = torch.empty(g.shape, dtype=torch.bfloat16, device=DEV)
    moe.moe_orthogonalize(g, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out=out, workspace=ws)
    for i in range(3):
        g.copy_(gradients("low_rank", 4, 264, 136, seed=i).to(DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.moe_orthogonalize(g)), i

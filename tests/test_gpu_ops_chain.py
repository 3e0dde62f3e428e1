"""The operators together, as a training step uses them: a routing, the experts'
products over its rows and their gradients, orthogonalised updates of those, and a
projection of the result with every row's adapter.  Every part is compared where its
inputs are known exactly: the layer and its weight gradients with the oracle, the
updates and the adapters with float64 of the tensors they were given.

The chain rounds what the layer rounds (h, dy, dg and du to bf16, once each; the
routing weight multiplies h before its rounding, which then carries it), so the
layer's bars Y_TOL, GRAD_RMS_TOL and GRAD_MAX_TOL hold for it as they are.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests import ops_ref as ref
from tests import tolerances as TL
from tests.parity import y_error
from tests.test_ops_tolerances import MAX_BAR, RMS_BAR

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_mixture_experts_prefix_amd")
DEV = torch.device("cuda:0")
L, RANK, N_OUT = 3, 16, 136


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    moe.load_library()


def rows_of_routing(ids, E):
    """(token, slot of topk) of every expert-sorted row, and the experts' offsets."""
    al = moe.moe_align(ids, E, 1)
    order = al["sorted_assign"].long()
    return order, al["offsets"]


def step(t, ids, p):
    """One step; t: dict of GPU tensors.  Returns a dict of its results."""
    T, k = ids.shape
    E, F2, D = t["w_gate_up"].shape
    F = F2 // 2
    order, off = rows_of_routing(ids, E)
    token, weight = order // k, p.flatten()[order][:, None]
    xs, dys = t["x"][token], t["dy"].to(torch.bfloat16)[token]
    # forward
    gu = moe.moe_grouped_gemm(xs, off, t["w_gate_up"])
    g, u = gu[:, :F], gu[:, F:]
    sig = torch.sigmoid(g)
    h = weight * (g * sig * u)
    h16 = h.to(torch.bfloat16)
    rows = torch.empty((T * k, D), device=DEV)
    rows[order] = moe.moe_grouped_gemm(h16, off, t["w_down"])
    y = rows.view(T, k, D).sum(1)
    # backward
    dh = weight * moe.moe_grouped_gemm(dys, off, t["w_down"], transposed=True)
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1).to(torch.bfloat16)
    dx = torch.empty((T * k, D), device=DEV)
    dx[order] = moe.moe_grouped_gemm(dgu, off, t["w_gate_up"], transposed=True)
    dw_gate_up = moe.moe_grouped_gemm_wgrad(dgu, xs, off)
    dw_down = moe.moe_grouped_gemm_wgrad(dys, h16, off)
    # updates, and the adapters on the layer's output
    out = dict(y=y, dx=dx.view(T, k, D).sum(1), dw_gate_up=dw_gate_up, dw_down=dw_down,
               up_gate_up=moe.moe_orthogonalize(dw_gate_up), up_down=moe.moe_orthogonalize(dw_down))
    y16 = y.to(torch.bfloat16)
    xa = torch.empty((T, RANK), device=DEV)
    z = moe.moe_lora_forward(y16, t["w_out"], t["a"], t["b"], t["adapter"], t["scale"],
                             out_dtype=torch.float32, xa=xa)
    gr = moe.moe_lora_backward(y16, t["w_out"], t["a"], t["b"], t["adapter"], t["dz"], xa, t["scale"])
    out.update(y16=y16, xa=xa, z=z, dy16=gr["dx"], da=gr["da"], db=gr["db"])
    return out


def make(T, D, E, k, F, seed):
    s = W.Shape(T=T, D=D, E=E, k=k, F=F)
    inp = W.make_inputs(s, seed=seed)
    ids, p, _, _ = oracle.route(inp.x, inp.w_g, None, k)
    g = torch.Generator()
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)

    t = dict(x=inp.x, w_gate_up=inp.w_gate_up, w_down=inp.w_down, dy=W.normal_f32((T, D), seed, 99, 1.0),
             w_out=normal(N_OUT, D, std=0.05), a=normal(L, RANK, D, std=D ** -0.5), b=normal(L, N_OUT, RANK, std=0.1),
             adapter=torch.randint(-1, L, (T,), generator=g).to(torch.int32),
             scale=torch.rand(L, generator=g) + 0.5, dz=normal(T, N_OUT, std=0.1))
    return inp, ids, p, {n: v.to(DEV) for n, v in t.items()}


SIZES = [(40, 264, 8, 2, 136), (300, 200, 4, 2, 264), (1, 64, 8, 2, 72)]


@pytest.mark.parametrize("T,D,E,k,F", SIZES)
def test_a_training_step(T, D, E, k, F):
    inp, ids, p, t = make(T, D, E, k, F, seed=T)
    p32 = p.astype(np.float32)
    gi, gp = torch.from_numpy(ids).to(DEV), torch.from_numpy(p32).to(DEV)
    got = step(t, gi, gp)
    torch.cuda.synchronize()
    want = oracle.experts(inp, ids, p32.astype(np.float64))
    assert y_error(got["y"].cpu().numpy(), want)[0] <= TL.Y_TOL
    grads = oracle.backward(inp, ids, p32.astype(np.float64), t["dy"].cpu().numpy())
    for name in ("dw_gate_up", "dw_down"):
        r, m = TL.grad_error(got[name].cpu().numpy(), grads[name])
        print("T=%d %s: RMS err %.3g, max err %.3g" % (T, name, r, m))
        assert r <= TL.GRAD_RMS_TOL and m <= TL.GRAD_MAX_TOL, name
    # the layer's own call takes the same rows
    y = moe.moe_forward_routed(t["x"], t["w_gate_up"], t["w_down"], gi, gp)
    assert y_error(got["y"].cpu().numpy(), y.cpu().double().numpy())[0] <= 2 * TL.Y_TOL
    for name, dw in (("up_gate_up", "dw_gate_up"), ("up_down", "dw_down")):
        for got_e, want_e in zip(got[name].cpu().double(), ref.orthogonalize(got[dw])):
            rms = want_e.square().mean().sqrt()
            err = (got_e - want_e).abs()
            assert err.square().mean().sqrt() <= RMS_BAR * rms
            assert (err <= MAX_BAR * rms + 2 * ref.HALF_BF16 * want_e.abs()).all()
    args = [t["w_out"], t["a"], t["b"], t["adapter"], t["scale"]]
    fwd = ref.lora(got["y16"], *args)
    ref.assert_within(got["z"], fwd["y"], ref.product_bound(fwd["s"], D + 2 * RANK) + fwd["parts"], "z")
    bwd = ref.lora_backward(got["y16"], *args, t["dz"], got["xa"])
    for name, key in (("dx", "dy16"), ("da", "da"), ("db", "db")):
        ref.assert_within(got[key], bwd[name], bwd[name + "_bound"], name)


@pytest.mark.parametrize("T,D,E,k,F", SIZES[:2])
def test_the_step_as_a_graph(T, D, E, k, F):
    """A captured step follows new tokens, weights and routings, beside eager steps."""
    _, ids, p, t = make(T, D, E, k, F, seed=1)
    gi, gp = torch.from_numpy(ids).to(DEV), torch.from_numpy(p.astype(np.float32)).to(DEV)
    al = moe.moe_align(gi, E, 1)  # captured steps keep the buffers of the rows' order
    order, off = al["sorted_assign"].long(), al["offsets"].clone()
    xs, dys = t["x"][order // k].clone(), t["dy"].to(torch.bfloat16)[order // k].clone()
    wd = t["w_down"]
    R = T * k

    def products():
        gu = moe.moe_grouped_gemm(xs, off, t["w_gate_up"], out_dtype=torch.bfloat16)
        h = gu[:, :F].contiguous()
        y = moe.moe_grouped_gemm(h, off, wd, out_dtype=torch.bfloat16)
        xa = torch.empty((R, RANK), device=DEV)
        ad = t["adapter"].repeat(k)
        z = moe.moe_lora_forward(y, t["w_out"], t["a"], t["b"], ad, t["scale"], xa=xa)
        g = moe.moe_lora_backward(y, t["w_out"], t["a"], t["b"], ad, z, xa, t["scale"], out_dtype=torch.bfloat16)
        dh = moe.moe_grouped_gemm(g["dx"], off, wd, transposed=True, out_dtype=torch.bfloat16)
        dw = moe.moe_grouped_gemm_wgrad(g["dx"], h, off)
        return [gu, y, z, xa, g["dx"], g["da"], g["db"], dh, dw, moe.moe_orthogonalize(dw),
                moe.moe_orthogonalize(dw.transpose(1, 2).contiguous())]

    products()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = products()
    for r in range(4):
        gen = torch.Generator()
        gen.manual_seed(50 + r)
        xs.copy_(torch.randn(xs.shape, generator=gen).to(torch.bfloat16))
        cuts = torch.randint(0, R + 1, (E - 1,), generator=gen).sort().values.tolist()
        off.copy_(torch.tensor([0] + cuts + [R], dtype=torch.int32))
        t["adapter"].copy_(torch.randint(-1, L, (T,), generator=gen).to(torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = products()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, eager)), r


def test_two_streams_at_once():
    """Steps queued on two streams, each with its own results, equal the same steps alone."""
    made = [make(*SIZES[i], seed=20 + i) for i in range(2)]
    routing = [(torch.from_numpy(i).to(DEV), torch.from_numpy(p.astype(np.float32)).to(DEV)) for _, i, p, _ in made]
    alone = [step(m[3], *r) for m, r in zip(made, routing)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for s, m, r, out in zip(streams, made, routing, got):
            with torch.cuda.stream(s):
                out.append(step(m[3], *r))
    torch.cuda.synchronize()
    for first, outs in zip(alone, got):
        for out in outs:
            for name, v in out.items():
                assert torch.equal(v, first[name]), name

"""The grouped products, the low-rank adapters and the orthogonalised update as
measured calls: their cases, inputs, plain forms and 64-bit definitions.

Three operators, each in every direction it has:
 - grouped products: y[r] = W[g] x[r] for the rows offsets[g] <= r < offsets[g+1]
   (weights [G, N, K] as bf16 or as E4M3 codes with a scale per row, or stored
   transposed, [G, K, N], which is the gradient of x), and the gradient of the
   weights, dW[g] = sum of dy[r] x[r]^T over the group's rows;
 - adapters: y[t] = W x[t] + s[a] B[a] (A[a] x[t]) with a = adapter[t] (-1: no
   adapter), and its backward pass for x and the adapters (W is frozen);
 - orthogonalised update: five Newton-Schulz steps X <- aX + (bA + cAA)X,
   A = X X^T, on every matrix of a stack of gradients, each divided by its norm.

Sizes are those of the layers this repository runs (widths 128, 2880, 4096 and
7168, hidden widths 256, 2048, 2880 and 14336) or generic ones around them.
"""
import math

import torch

own = False

NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a decode step: its four experts' down projection, 4 of 32 experts touched
        dict(name="grouped_one_token", op="grouped", R=4, G=32, busy=4, N=2880, K=2880, fmt="bf16",
             transposed=False, out="f32"),
        # a decode batch of 64 tokens over every expert, E4M3 weights, gate and up rows
        dict(name="grouped_decode_e4m3", op="grouped", R=256, G=32, busy=32, N=5760, K=2880, fmt="e4m3",
             transposed=False, out="f32"),
        # a prompt's rows on eight wide experts, ragged loads, bf16 rows out
        dict(name="grouped_prompt", op="grouped", R=8192, G=8, busy=8, N=4096, K=14336, fmt="bf16",
             transposed=False, out="bf16"),
        # the gradient of x for many narrow experts, some without rows, an odd row count
        dict(name="grouped_grad_x", op="grouped", R=10007, G=64, busy=61, N=7168, K=2048, fmt="bf16",
             transposed=True, out="f32"),
        # the gradient of the weights of the same kind of layer, again with idle experts
        dict(name="grouped_grad_w", op="wgrad", R=10007, G=64, busy=61, N=2048, K=4096),
        # one decode step of 16 requests, 11 different adapters among them, beside a square projection
        dict(name="adapters_decode", op="lora", T=16, N=4096, D=4096, L=32, live=11, r=16, run=1, out="bf16"),
        # a full decode batch, nearly every request with its own adapter of a higher rank
        dict(name="adapters_decode_wide", op="lora", T=64, N=5760, D=2880, L=64, live=48, r=64, run=1, out="bf16"),
        # prompts of several requests packed into one batch, runs of rows with one adapter each
        dict(name="adapters_prompt", op="lora", T=4096, N=8192, D=4096, L=8, live=7, r=32, run=400, out="bf16"),
        # a training batch of adapters beside a frozen projection, odd row count
        dict(name="adapters_backward", op="lora_bwd", T=4101, N=4096, D=4096, L=4, live=4, r=16, run=512, out="f32"),
        # the update of a small layer's experts
        dict(name="update_small", op="orth", E=8, M=256, N=128),
        # the update of 32 square experts
        dict(name="update_square", op="orth", E=32, M=2880, N=2880),
        # the update of two wide experts, the tall orientation of their input projections
        dict(name="update_tall", op="orth", E=2, M=14336, N=4096),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "lora", "lora", "lora_bwd", "orth"])
    if op == "grouped":
        G = _log_int(rng, 1, 64)
        N, K = _log_int(rng, 128, 8192, 8), _log_int(rng, 128, 8192, 8)
        R = _log_int(rng, 1, 12000)
        fmt = rng.choice(["bf16", "bf16", "e4m3"])
        return dict(op=op, R=R, G=G, busy=rng.randint(1, min(G, R)), N=N, K=K, fmt=fmt,
                    transposed=fmt == "bf16" and rng.random() < 0.4, out=rng.choice(["f32", "bf16"]))
    if op == "wgrad":
        G, R = _log_int(rng, 1, 64), _log_int(rng, 1, 12000)
        return dict(op=op, R=R, G=G, busy=rng.randint(1, min(G, R)), N=_log_int(rng, 128, 5760, 8),
                    K=_log_int(rng, 128, 5760, 8))
    if op in ("lora", "lora_bwd"):
        T, L = _log_int(rng, 1, 6000), _log_int(rng, 1, 64)
        run = 1 if T <= 64 else _log_int(rng, 1, 512)
        live = rng.randint(0, min(L, (T + run - 1) // run))
        return dict(op=op, T=T, N=_log_int(rng, 128, 8192, 8), D=_log_int(rng, 128, 7168, 8), L=L, live=live,
                    r=rng.choice([8, 16, 24, 32, 64, 128]), run=run, out=rng.choice(["f32", "bf16"]))
    return dict(op=op, E=_log_int(rng, 1, 16), M=_log_int(rng, 64, 4096, 8), N=_log_int(rng, 64, 4096, 8))


# ---------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, std=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _ragged(R, G, busy, seed):
    """Rows per group: `busy` groups of uneven loads, at least a row each, the others empty."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 17)
    chosen = torch.randperm(G, generator=g)[:busy]
    p = torch.softmax(0.5 * torch.randn(busy, generator=g), 0)
    extra = torch.multinomial(p, R - busy, replacement=True, generator=g) if R > busy else torch.empty(0, dtype=torch.int64)
    sizes = torch.zeros(G, dtype=torch.int64)
    sizes[chosen] = 1 + torch.bincount(extra, minlength=busy)
    return sizes.tolist()


def _adapters(case, seed):
    """Adapter of every row: requests of `run` rows each, `live` adapters among them, one row in
    sixteen requests without one (all of them when live is 0)."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 23)
    T, L, live, run = case["T"], case["L"], case["live"], case["run"]
    reqs = (T + run - 1) // run
    if live == 0:
        return torch.full((T,), -1, dtype=torch.int32)
    names = torch.randperm(L, generator=g)[:live]
    of = names[torch.randint(0, live, (reqs,), generator=g)]
    of[torch.rand(reqs, generator=g) < 1 / 16] = -1
    of[torch.randperm(reqs, generator=g)[:live]] = names  # every one of them takes part
    return of.repeat_interleave(run)[:T].to(torch.int32)


def _weights(case, g):
    G, N, K = case["G"], case["N"], case["K"]
    shape = (G, K, N) if case["transposed"] else (G, N, K)
    if case["fmt"] == "bf16":
        return _normal(shape, g, 0.02), None
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((G, N), dtype=torch.float32, device="cuda")
    for e in range(G):
        w = _normal((N, K), g, 0.02, torch.float32)
        scale[e] = w.abs().amax(1) / 448.0
        codes[e] = (w / scale[e][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def _dtype(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op in ("grouped", "wgrad"):
        sizes = _ragged(case["R"], case["G"], case["busy"], seed)
        s["sizes"] = sizes
        s["offsets"] = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        s["x"] = _normal((case["R"], case["K"]), g)
        if op == "wgrad":
            s["dy"] = _normal((case["R"], case["N"]), g, 0.1)
        else:
            s["w"], s["w_scale"] = _weights(case, g)
    elif op in ("lora", "lora_bwd"):
        T, N, D, L, r = (case[k] for k in ("T", "N", "D", "L", "r"))
        s["x"] = _normal((T, D), g)
        s["w"] = _normal((N, D), g, 0.02)
        s["lora_a"] = _normal((L, r, D), g, 1 / math.sqrt(D))
        s["lora_b"] = _normal((L, N, r), g, 0.05)
        s["scale"] = torch.rand(L, generator=g, device="cuda") + 0.5
        s["adapter"] = _adapters(case, seed).to("cuda")
        if op == "lora_bwd":
            s["dy"] = _normal((T, N), g, 0.1)
            # the forward's A[a] x, which a training step keeps
            s["xa"] = _per_adapter(s["x"].float(), s["lora_a"].float(), s["adapter"])
    else:
        # a gradient: few strong directions over a weak floor
        E, M, N = case["E"], case["M"], case["N"]
        k = min(32, M, N)
        s["g"] = torch.empty((E, M, N), dtype=torch.float32, device="cuda")
        decay = torch.logspace(0, -2, k, device="cuda")
        for e in range(E):
            u, v = _normal((M, k), g, 1e-3, torch.float32), _normal((k, N), g, 1.0, torch.float32)
            s["g"][e] = (u * decay) @ v + _normal((M, N), g, 1e-4, torch.float32)
    if own:
        _plan(s)
    return s


def _plan(s):
    """Outputs and workspaces that a program keeps from call to call."""
    import sparse_mixture_experts_prefix_amd as moe
    case, op = s["case"], s["case"]["op"]

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "grouped":
        s["y"] = new((case["R"], case["N"]), _dtype(case))
        s["ws"] = new(moe.moe_grouped_gemm_workspace_size(s["x"], s["w"], transposed=case["transposed"]), torch.uint8)
    elif op == "wgrad":
        s["dw"] = new((case["G"], case["N"], case["K"]), torch.float32)
    elif op == "lora":
        s["y"] = new((case["T"], case["N"]), _dtype(case))
        s["ws"] = new(moe.moe_lora_workspace_size(s["x"], s["w"], s["lora_a"]), torch.uint8)
    elif op == "lora_bwd":
        s["out"] = dict(dx=new((case["T"], case["D"]), _dtype(case)),
                        da=new(tuple(s["lora_a"].shape), torch.float32), db=new(tuple(s["lora_b"].shape), torch.float32))
        s["ws"] = new(moe.moe_lora_backward_workspace_size(s["x"], s["w"], s["lora_a"]), torch.uint8)
    else:
        s["update"] = new(tuple(s["g"].shape), torch.bfloat16)
        s["ws"] = new(moe.moe_orthogonalize_workspace_size(s["g"]), torch.uint8)


# ---------------------------------------------------------------- the passes
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import sparse_mixture_experts_prefix_amd as moe
    case, op = s["case"], s["case"]["op"]
    if op == "grouped":
        return moe.moe_grouped_gemm(s["x"], s["offsets"], s["w"], w_scale=s["w_scale"],
                                    transposed=case["transposed"], y=s["y"], workspace=s["ws"])
    if op == "wgrad":
        return moe.moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], dw=s["dw"])
    if op == "lora":
        return moe.moe_lora_forward(s["x"], s["w"], s["lora_a"], s["lora_b"], s["adapter"], s["scale"],
                                    y=s["y"], workspace=s["ws"])
    if op == "lora_bwd":
        return moe.moe_lora_backward(s["x"], s["w"], s["lora_a"], s["lora_b"], s["adapter"], s["dy"], s["xa"],
                                     s["scale"], grads=s["out"], workspace=s["ws"])
    return moe.moe_orthogonalize(s["g"], steps=NS_STEPS, eps=NS_EPS, out=s["update"], workspace=s["ws"])


def _plain_grouped(s):
    case = s["case"]
    y = torch.empty((case["R"], case["N"]), dtype=_dtype(case), device="cuda")
    r0 = 0
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        if s["w_scale"] is None:
            w = s["w"][e].float()
        else:
            w = s["w"][e].view(torch.float8_e4m3fn).float() * s["w_scale"][e][:, None]
        x = s["x"][r0:r0 + n].float()
        y[r0:r0 + n] = (x @ w if case["transposed"] else x @ w.t()).to(y.dtype)
        r0 += n
    return y


def _plain_wgrad(s):
    case = s["case"]
    dw = torch.zeros((case["G"], case["N"], case["K"]), dtype=torch.float32, device="cuda")
    r0 = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            dw[e] = s["dy"][r0:r0 + n].float().t() @ s["x"][r0:r0 + n].float()
        r0 += n
    return dw


def _member(adapter, L):
    """[T, L]: 1 where the row has that adapter."""
    return (adapter[:, None] == torch.arange(L, device=adapter.device)[None, :]).float()


def _per_adapter(x, a, adapter):
    """[T, r]: A[adapter[t]] x[t], zero rows without an adapter."""
    L, r, D = a.shape
    all_a = (x @ a.reshape(L * r, D).t()).reshape(-1, L, r)
    return (all_a * _member(adapter, L)[:, :, None]).sum(1)


def _spread(v, adapter, L):
    """[T, L r]: row t holds v[t] in its adapter's columns."""
    return (v[:, None, :] * _member(adapter, L)[:, :, None]).reshape(v.shape[0], -1)


def _row_scale(s):
    a = s["adapter"].long()
    return torch.where(a >= 0, s["scale"][a.clamp(min=0)], torch.zeros((), device="cuda"))[:, None]


def _plain_lora(s):
    case = s["case"]
    L, r, D = s["lora_a"].shape
    x = s["x"].float()
    v = _per_adapter(x, s["lora_a"].float(), s["adapter"]) * _row_scale(s)
    b = s["lora_b"].float().permute(0, 2, 1).reshape(L * r, case["N"])
    return (x @ s["w"].float().t() + _spread(v, s["adapter"], L) @ b).to(_dtype(case))


def _plain_lora_bwd(s):
    case = s["case"]
    L, r, D = s["lora_a"].shape
    N = case["N"]
    x, dy = s["x"].float(), s["dy"].float()
    sdy = dy * _row_scale(s)
    a, b = s["lora_a"].float(), s["lora_b"].float()
    u = _spread(_per_adapter(sdy, b.permute(0, 2, 1).contiguous(), s["adapter"]), s["adapter"], L)
    dx = dy @ s["w"].float() + u @ a.reshape(L * r, D)
    da = (u.t() @ x).reshape(L, r, D)
    db = (_spread(s["xa"], s["adapter"], L).t() @ sdy).reshape(L, r, N).permute(0, 2, 1).contiguous()
    return dict(dx=dx.to(_dtype(case)), da=da, db=db)


def _plain_orth(s):
    a, b, c = NS_COEFFS
    g = s["g"]
    out = torch.empty(g.shape, dtype=torch.bfloat16, device="cuda")
    for e in range(g.shape[0]):
        x = g[e] / (g[e].square().sum().sqrt() + NS_EPS)
        tall = x.shape[0] > x.shape[1]
        if tall:
            x = x.t().contiguous()
        for _ in range(NS_STEPS):
            p = x @ x.t()
            x = a * x + (b * p + c * (p @ p)) @ x
        out[e] = x.t() if tall else x
    return out


_PLAIN = dict(grouped=_plain_grouped, wgrad=_plain_wgrad, lora=_plain_lora, lora_bwd=_plain_lora_bwd, orth=_plain_orth)


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op == "grouped":
        R, N, K = case["R"], case["N"], case["K"]
        w = N * K + 4 * N if case["fmt"] == "e4m3" else 2 * N * K
        return dict(bytes=2 * R * K + case["busy"] * w + R * N * (4 if case["out"] == "f32" else 2), flops=2 * R * N * K)
    if op == "wgrad":
        R, N, K = case["R"], case["N"], case["K"]
        return dict(bytes=2 * R * (N + K) + 4 * case["G"] * N * K, flops=2 * R * N * K)
    if op in ("lora", "lora_bwd"):
        T, N, D, L, r, live = (case[k] for k in ("T", "N", "D", "L", "r", "live"))
        o = 4 if case["out"] == "f32" else 2
        ab = 2 * live * r * (N + D)
        if op == "lora":
            return dict(bytes=2 * T * D + 2 * N * D + ab + o * T * N, flops=2 * T * N * D + 2 * T * r * (N + D))
        return dict(bytes=2 * T * (D + N) + 4 * T * r + 2 * N * D + ab + o * T * D + 4 * L * r * (N + D),
                    flops=2 * T * N * D + 4 * T * r * (N + D))
    E, m, n = case["E"], min(case["M"], case["N"]), max(case["M"], case["N"])
    # a symmetric product needs one triangle of its result
    return dict(bytes=E * m * n * 6, flops=NS_STEPS * E * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n))


# -------------------------------------------------- the definitions in 64 bits
def _e4m3_value(codes):
    """The value of E4M3 codes (bias 7, no infinities) from their bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, c & 7
    mag = torch.where(e > 0, torch.ldexp((8 + m).double(), e - 10), torch.ldexp(m.double(), torch.full_like(e, -9)))
    return torch.where(c >= 128, -mag, mag)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "grouped":
        y = torch.empty((case["R"], case["N"]), dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(case["G"]):
            if off[e] == off[e + 1]:
                continue
            if case["fmt"] == "e4m3":
                w = _e4m3_value(s["w"][e]) * s["w_scale"][e].double().unsqueeze(1)
            else:
                w = s["w"][e].double()
            wt = w if case["transposed"] else w.t().contiguous()
            torch.mm(s["x"][off[e]:off[e + 1]].double(), wt, out=y[off[e]:off[e + 1]])
        return y
    if op == "wgrad":
        off = s["offsets"].tolist()
        return torch.stack([torch.mm(s["dy"][i:j].double().t().contiguous(), s["x"][i:j].double())
                            for i, j in zip(off, off[1:])])
    if op in ("lora", "lora_bwd"):
        x, w = s["x"].double(), s["w"].double()
        rows = [(torch.nonzero(s["adapter"] == l).flatten(), s["scale"][l].double(), s["lora_a"][l].double(),
                 s["lora_b"][l].double()) for l in range(case["L"])]
        if op == "lora":
            y = x @ w.t()
            for t, sc, a, b in rows:
                y[t] += sc * ((x[t] @ a.t()) @ b.t())
            return y
        dy = s["dy"].double()
        dx, da, db = dy @ w, [], []
        for t, sc, a, b in rows:
            u = sc * (dy[t] @ b)
            dx[t] += u @ a
            da.append(u.t() @ x[t])
            db.append(sc * (dy[t].t() @ s["xa"][t].double()))
        return dict(dx=dx, da=torch.stack(da), db=torch.stack(db))
    ca, cb, cc = NS_COEFFS
    out = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        x = s["g"][e].double()
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        short = x.shape[0] <= x.shape[1]
        for _ in range(NS_STEPS):
            p = (x @ x.t()) if short else (x.t() @ x)
            q = cb * p + cc * (p @ p)
            q.diagonal().add_(ca)
            x = q @ x if short else x @ q
        out[e] = x
    return out

"""What the operators around and inside the routed experts compute, and what is measured of them.

Five operators of the block that holds the experts:

- norm_in: the norm before the block (RMS or layer norm of the residual stream), forward and
  backward, and its form for serving, which also writes the rows in 8 bits;
- norm_out: the norm after the block with the block's gate, the residual add and its scales, and
  in the same pass the next block's norm; forward and backward;
- quantize: rows (gathered by token) to e4m3 with a scale for each 128 columns of a row, and
  weights with a scale for each 128 x 128 block;
- matmul: the product of such rows with such weights, dense or by expert;
- gated: both projections, the clamped SwiGLU and the rounding of its result to e4m3.

`run` gives their plain form (elementary operations in 32 bits) where `own` is false, and makes
the library's calls where it is true. Sizes are those of the benchmark's layers (d = 1024, 2048,
4096; f = 768, 1536, 2048; 128 and 256 experts), of the tests' ragged layers, and odd ones.
"""
import math

import numpy as np
import torch

own = False

F32, BF16, F16, E4M3 = 0, 1, 2, 3  # the library's dtype codes
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": F32, "bf16": BF16, "f16": F16}
GATES = {"none": 0, "channel": 1, "token": 2}
KINDS = {"none": 0, "rms": 1, "layer": 2}
EPS, LIMIT, QMAX, SMIN = 1e-6, 7.0, 448.0, 2.0 ** -126


def ceil128(n):
    return (n + 127) // 128


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # a token being written: the norm before the experts, bf16 rows and 8-bit rows in one pass
        dict(name="norm_in_token", op="norm_in", T=1, d=4096, kind="rms", stream="f32", block="bf16", train=False),
        # a training step of the 4096-token layer: forward and backward
        dict(name="norm_in_step", op="norm_in", T=4096, d=2048, kind="rms", stream="bf16", block="bf16", train=True),
        # eight tokens being written: post norm, gate, residual, and the next block's norm
        dict(name="norm_out_tokens", op="norm_out", T=8, d=4096, kind="rms", gate="channel", bias=False,
             stream="f32", block="bf16", train=False),
        # a training step of the 8192-token layer with one gate value a token and layer norm
        dict(name="norm_out_step", op="norm_out", T=8192, d=1024, kind="layer", gate="token", bias=True,
             stream="f32", block="bf16", train=True),
        # the rows of a 4096-token prompt, each to its 8 experts, as the experts' products take them
        dict(name="quantize_rows", op="quantize", T=4096, k=8, K=2048, src="bf16", weights=False),
        # loading: a few experts' weights, given [K, N] as the bf16 layer has them
        dict(name="quantize_weights", op="quantize", E=16, K=2048, N=768, src="bf16", weights=True, transposed=True),
        # one token through a dense projection
        dict(name="matmul_token", op="matmul", T=1, k=1, E=1, K=4096, N=1536, out="bf16"),
        # a dense projection of a prompt
        dict(name="matmul_prompt", op="matmul", T=4096, k=1, E=1, K=4096, N=4096, out="bf16"),
        # the down projection of the 128-expert prompt layer, gate weights applied
        dict(name="matmul_experts", op="matmul", T=4096, k=8, E=128, K=768, N=2048, out="f16"),
        # the experts of one token: 8 of 256
        dict(name="gated_token", op="gated", T=1, k=8, E=256, K=4096, N=1536, out="e4m3"),
        # the 128-expert prompt layer
        dict(name="gated_experts", op="gated", T=4096, k=8, E=128, K=2048, N=768, out="e4m3"),
        # ragged sizes: rows, a last block of K and a last block of columns that are all partial
        dict(name="gated_ragged", op="gated", T=333, k=3, E=6, K=1040, N=1000, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_in", "norm_out", "quantize", "matmul", "gated"])
    if op in ("norm_in", "norm_out"):
        train = rng.random() < 0.5
        d = rng.choice([_log(rng, 64, 4096), 8 * _log(rng, 8, 512), 128 * rng.randint(1, 32)])
        case = dict(op=op, T=_log(rng, 1, 8192), d=d, kind=rng.choice(["rms", "layer"]),
                    stream=rng.choice(["f32", "bf16", "f16"]), block=rng.choice(["bf16", "f16", "f32"]), train=train)
        if op == "norm_in" and not train:
            case["d"] = 16 * max(1, d // 16)  # rows in 8 bits start on 16 bytes
        if op == "norm_out":
            case.update(gate=rng.choice(["none", "channel", "token"]), bias=rng.random() < 0.3)
        return case
    K, N = 16 * _log(rng, 4, 256), 8 * _log(rng, 4, 512)
    if op == "quantize":
        if rng.random() < 0.5:
            return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 8), K=min(K, 2048),
                        src=rng.choice(["bf16", "f16", "f32"]), weights=False)
        return dict(op=op, E=rng.randint(1, 8), K=min(K, 2048), N=min(N, 1536), src=rng.choice(["bf16", "f32"]),
                    weights=True, transposed=rng.random() < 0.5)
    E = rng.choice([1, 1, rng.randint(2, 128)])
    k = 1 if E == 1 else rng.randint(1, min(8, E))
    T = _log(rng, 1, 4096)
    K, N = min(K, 2048), min(N, 2048 if op == "matmul" else 1024)
    if E > 1:  # by expert: smaller projections, so that the largest listed case stays the largest
        K, N, T = min(K, 1536), min(N, 768), min(T, 2048)
    if op == "matmul":
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, out=rng.choice(["bf16", "f16", "f32"]))
    return dict(op=op, T=T, k=k, E=E, K=K, N=16 * max(1, N // 16), out=rng.choice(["e4m3", "e4m3", "bf16", "f16"]))


# ------------------------------------------------------------------------------ inputs

def _counts(case, rng):
    """Rows of each expert: T tokens, k distinct experts each, popular experts much fuller than others."""
    T, k, E = case["T"], case["k"], case["E"]
    bias = 3.0 * (1.0 - np.log(rng.permutation(E) + 1.0) / math.log(max(2, E)))
    pick = np.argsort(-(rng.gumbel(size=(T, E)) + bias), axis=1)[:, :k]
    return pick


def _weights(g, dev, E, N, K):
    """Weights of normal values in e4m3 with a scale for each 128 x 128 block."""
    nb, kb = ceil128(N), ceil128(K)
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty(E, nb, kb, dtype=torch.float32, device=dev)
    for e0 in range(0, E, 32):
        e1 = min(E, e0 + 32)
        w = torch.randn(e1 - e0, N, K, generator=g, device=dev) * 0.02
        w = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(e1 - e0, nb, 128, kb, 128)
        sc = (w.abs().amax(dim=(2, 4)) / QMAX).clamp(min=SMIN)
        w = (w / sc[:, :, None, :, None]).clamp(-QMAX, QMAX)
        q[e0:e1] = w.view(e1 - e0, nb * 128, kb * 128)[:, :N, :K].to(torch.float8_e4m3fn)
        s[e0:e1] = sc
    return q, s


def _rows(g, dev, R, K):
    """Rows of normal values of several sizes in e4m3, with scales [ceil(K/128), R]."""
    kb = ceil128(K)
    x = torch.randn(R, K, generator=g, device=dev) * torch.exp(0.5 * torch.randn(R, 1, generator=g, device=dev))
    x = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(R, kb, 128)
    sc = (x.abs().amax(dim=2) / QMAX).clamp(min=SMIN)
    q = (x / sc[:, :, None]).clamp(-QMAX, QMAX).view(R, kb * 128)[:, :K].to(torch.float8_e4m3fn).contiguous()
    return q, sc.t().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.default_rng([int(seed), 77])
    op, s = case["op"], dict(case)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dtype)

    if op in ("norm_in", "norm_out"):
        T, d, st, bl = case["T"], case["d"], DT[case["stream"]], DT[case["block"]]
        s["ws"] = None
        s["weight"] = normal(d, std=0.1, mean=1.0)
        # a residual stream: sizes differ between tokens, a few channels are large
        size = torch.exp(0.5 * normal(T, 1)) * torch.where(torch.rand(d, generator=g, device=dev) < 0.01, 8.0, 1.0)
        s["mean"], s["rstd"] = torch.empty(T, device=dev), torch.empty(T, device=dev)
        if op == "norm_in":
            s["x"] = (normal(T, d) * size).to(st)
            s["y"] = torch.empty(T, d, dtype=bl, device=dev)
            if case["train"]:
                s["dy"], s["dres"] = normal(T, d, dtype=bl), normal(T, d, dtype=st)
                s["dx"], s["dw"] = torch.empty(T, d, dtype=st, device=dev), torch.empty(d, device=dev)
            else:
                s["q8"] = torch.empty(T, d, dtype=torch.float8_e4m3fn, device=dev)
                s["s8"] = torch.empty(ceil128(d), T, device=dev)
        else:
            s["resid"], s["block_out"] = (normal(T, d) * size).to(st), (normal(T, d) * size).to(bl)
            s["bias_t"] = normal(d, std=0.1) if case["bias"] else None
            s["gate_t"] = {"none": None, "channel": normal(d, std=0.5), "token": normal(T, std=0.5)}[case["gate"]]
            s["next_weight"] = normal(d, std=0.1, mean=1.0)
            s["alpha"], s["beta"] = 0.9, 0.5
            s["out"], s["x_next"] = torch.empty(T, d, dtype=st, device=dev), torch.empty(T, d, dtype=bl, device=dev)
            if case["train"]:
                s["dout"] = normal(T, d, dtype=st)
                s["dresid"], s["dy"] = torch.empty(T, d, dtype=st, device=dev), torch.empty(T, d, dtype=bl, device=dev)
                s["dw"] = torch.empty(d, device=dev)
                s["db"] = torch.empty(d, device=dev) if case["bias"] else None
                s["dgate"] = {"none": None, "channel": torch.empty(d, device=dev),
                              "token": torch.empty(T, device=dev)}[case["gate"]]
        if case["train"]:
            s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
        return s
    if op == "quantize":
        if case["weights"]:
            E, K, N = case["E"], case["K"], case["N"]
            s["w"] = normal(*((E, K, N) if case["transposed"] else (E, N, K)), dtype=DT[case["src"]], std=0.02)
            s["q"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=dev)
            s["s"] = torch.empty(E, ceil128(N), ceil128(K), device=dev)
        else:
            T, k, K = case["T"], case["k"], case["K"]
            s["x"] = (normal(T, K) * torch.exp(0.5 * normal(T, 1))).to(DT[case["src"]])
            order = rng.permutation(T * k) // k
            s["index"] = torch.from_numpy(order.astype(np.int32)).to(dev)
            s["q"] = torch.empty(T * k, K, dtype=torch.float8_e4m3fn, device=dev)
            s["s"] = torch.empty(ceil128(K), T * k, device=dev)
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
        return s
    T, k, E, K, N = case["T"], case["k"], case["E"], case["K"], case["N"]
    R = T * k
    s["a"], s["a_scale"] = _rows(g, dev, R, K)
    s["offsets"] = s["sorted_pair"] = s["topk_w"] = None
    if E > 1:
        pick = _counts(case, rng)
        counts = np.bincount(pick.reshape(-1), minlength=E)
        s["most"] = int(counts.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
        if op == "matmul":  # the gate weight of each row's (token, choice) pair
            pairs = np.argsort(pick.reshape(-1), kind="stable").astype(np.int32)
            s["sorted_pair"] = torch.from_numpy(pairs).to(dev)
            s["topk_w"] = torch.softmax(normal(T, k), dim=1).contiguous()
    s["ws"] = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
    if op == "matmul":
        s["w"], s["w_scale"] = _weights(g, dev, E, N, K)
        s["c"] = torch.zeros(R, N, dtype=DT[case["out"]], device=dev)
    else:
        s["w_gate"], s["s_gate"] = _weights(g, dev, E, N, K)
        s["w_up"], s["s_up"] = _weights(g, dev, E, N, K)
        if case["out"] == "e4m3":
            s["h"] = torch.zeros(R, N, dtype=torch.float8_e4m3fn, device=dev)
            s["h_scale"] = torch.zeros(ceil128(N), R, device=dev)
        else:
            s["h"], s["h_scale"] = torch.zeros(R, N, dtype=DT[case["out"]], device=dev), None
    return s


# ------------------------------------------------------------------------------ plain forms

def _norm(x, kind):
    """The normalised rows of x (32 bits) and what the backward pass needs of them."""
    mean = x.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + EPS)
    return c * rstd, rstd


def _norm_backward(xhat, rstd, g, kind):
    t = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if kind == "layer":
        t = t - g.mean(dim=1, keepdim=True)
    return t * rstd


def _round_rows(x):
    """Rows of x (32 bits) in e4m3 and the scales of each 128 columns, [ceil(K/128), R]."""
    R, K = x.shape
    kb = ceil128(K)
    x = torch.nn.functional.pad(x, (0, kb * 128 - K)).view(R, kb, 128)
    sc = (x.abs().amax(dim=2) / QMAX).clamp(min=SMIN)
    q = (x / sc[:, :, None]).clamp(-QMAX, QMAX).view(R, kb * 128)[:, :K].to(torch.float8_e4m3fn)
    return q, sc.t()


def _values(a, a_scale):
    return a.float() * a_scale.t().repeat_interleave(128, dim=1)[:, :a.shape[1]]


def _weight_values(q, s):
    N, K = q.shape[1], q.shape[2]
    return q.float() * s.repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]


def _products(a, offsets, most, weights):
    """Each row's product with its expert's weights [N, K]; rows behind the last expert's give nothing of use."""
    if offsets is None:
        return [a @ _weight_values(q, s)[0].t() for q, s in weights]
    R, E = a.shape[0], offsets.numel() - 1
    r = torch.arange(R, device=a.device)
    e = torch.searchsorted(offsets[1:].contiguous(), r.to(torch.int32), right=True).clamp(max=E - 1)
    if R <= E:  # a few rows: the weights of each row's expert
        return [torch.bmm(_weight_values(q.view(torch.uint8)[e].view(q.dtype), s[e]), a[:, :, None])[:, :, 0]
                for q, s in weights]
    at = (offsets[:-1, None] + torch.arange(most, device=a.device)).clamp(max=R - 1)  # [E, most] rows
    pos = (r - offsets[e]).clamp(0, most - 1)
    rect = a[at.long()]
    return [torch.bmm(rect, _weight_values(q, s).transpose(1, 2))[e, pos] for q, s in weights]


def _plain(s):
    op = s["op"]
    if op == "norm_in":
        x = s["x"].float()
        xhat, rstd = _norm(x, s["kind"])
        y = xhat * s["weight"]
        if not s["train"]:
            q, sc = _round_rows(y)
            return {"y": y.to(s["y"].dtype), "q8": q, "s8": sc}
        dy = s["dy"].float()
        dx = s["dres"].float() + _norm_backward(xhat, rstd, dy * s["weight"], s["kind"])
        return {"y": y.to(s["y"].dtype), "dx": dx.to(s["dx"].dtype), "dw": (dy * xhat).sum(dim=0)}
    if op == "norm_out":
        b, gate, bias = s["block_out"].float(), s["gate_t"], s["bias_t"]
        gate = 1.0 if gate is None else gate[:, None] if s["gate"] == "token" else gate
        bhat, rstd = _norm(b, s["kind"])
        n = bhat * s["weight"] + (0.0 if bias is None else bias)
        out = (s["alpha"] * s["resid"].float() + s["beta"] * gate * n).to(s["out"].dtype)
        x_next = _norm(out.float(), s["kind"])[0] * s["next_weight"]
        got = {"out": out, "x_next": x_next.to(s["x_next"].dtype)}
        if s["train"]:
            dout = s["dout"].float()
            dn = s["beta"] * gate * dout
            got["dresid"] = (s["alpha"] * dout).to(s["dresid"].dtype)
            got["dy"] = _norm_backward(bhat, rstd, dn * s["weight"], s["kind"]).to(s["dy"].dtype)
            got["dw"] = (dn * bhat).sum(dim=0)
            if bias is not None:
                got["db"] = dn.sum(dim=0)
            if s["gate_t"] is not None:
                got["dgate"] = (s["beta"] * dout * n).sum(dim=1 if s["gate"] == "token" else 0)
        return got
    if op == "quantize":
        if not s["weights"]:
            q, sc = _round_rows(s["x"].float()[s["index"].long()])
            return {"q": q, "s": sc}
        w = s["w"].float()
        w = w.transpose(1, 2) if s["transposed"] else w
        E, N, K = w.shape
        nb, kb = ceil128(N), ceil128(K)
        w = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).reshape(E, nb, 128, kb, 128)
        sc = (w.abs().amax(dim=(2, 4)) / QMAX).clamp(min=SMIN)
        q = (w / sc[:, :, None, :, None]).clamp(-QMAX, QMAX).view(E, nb * 128, kb * 128)[:, :N, :K]
        return {"q": q.to(torch.float8_e4m3fn), "s": sc}
    a = _values(s["a"], s["a_scale"])
    if op == "matmul":
        (c,) = _products(a, s["offsets"], s.get("most"), [(s["w"], s["w_scale"])])
        if s["topk_w"] is not None:
            c = c * s["topk_w"].view(-1)[s["sorted_pair"].long()][:, None]
        return {"c": c.to(s["c"].dtype)}
    g, u = _products(a, s["offsets"], s.get("most"), [(s["w_gate"], s["s_gate"]), (s["w_up"], s["s_up"])])
    g, u = g.clamp(-LIMIT, LIMIT), u.clamp(-LIMIT, LIMIT)
    h = g / (1.0 + torch.exp(-g)) * u
    if s["out"] == "e4m3":
        q, sc = _round_rows(h)
        return {"h": q, "h_scale": sc}
    return {"h": h.to(s["h"].dtype)}


# ------------------------------------------------------------------------------ the library's calls

def _library(s):
    from mixture_experts_routed_04_b200 import binding as b
    op = s["op"]
    if op == "norm_in":
        T, d = s["x"].shape
        p = b.norm_params(T, d, kind=KINDS[s["kind"]], eps=EPS, stream_dtype=CODE[s["stream"]],
                          block_dtype=CODE[s["block"]])
        if not s["train"]:
            b.norm_forward(p, s["x"], s["y"], weight=s["weight"], q8=s["q8"], s8=s["s8"])
            return {"y": s["y"], "q8": s["q8"], "s8": s["s8"]}
        b.norm_forward(p, s["x"], s["y"], weight=s["weight"], mean=s["mean"], rstd=s["rstd"])
        b.norm_backward(p, s["x"], s["dy"], s["mean"], s["rstd"], s["dx"], s["ws"], weight=s["weight"],
                        dres=s["dres"], dw=s["dw"])
        return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    if op == "norm_out":
        T, d = s["resid"].shape
        p = b.norm_params(T, d, kind=KINDS[s["kind"]], next_kind=KINDS[s["kind"]], eps=EPS,
                          stream_dtype=CODE[s["stream"]], block_dtype=CODE[s["block"]], gate_kind=GATES[s["gate"]],
                          alpha=s["alpha"], beta=s["beta"])
        b.norm_residual_forward(p, s["resid"], s["block_out"], s["out"], weight=s["weight"], bias=s["bias_t"],
                                gate=s["gate_t"], mean=s["mean"], rstd=s["rstd"], next_weight=s["next_weight"],
                                x_next=s["x_next"])
        got = {"out": s["out"], "x_next": s["x_next"]}
        if s["train"]:
            b.norm_residual_backward(p, s["block_out"], s["dout"], s["mean"], s["rstd"], s["dy"], s["ws"],
                                     weight=s["weight"], bias=s["bias_t"], gate=s["gate_t"], dresid=s["dresid"],
                                     dw=s["dw"], db=s["db"], dgate=s["dgate"])
            got.update({n: s[n] for n in ("dresid", "dy", "dw", "db", "dgate") if s[n] is not None})
        return got
    if op == "quantize":
        if s["weights"]:
            b.quantize_f8_weights(s["w"], s["q"], s["s"], transposed=s["transposed"])
        else:
            b.quantize_f8(s["x"], s["q"], s["s"], s["ws"], row_index=s["index"])
        return {"q": s["q"], "s": s["s"]}
    R, K, N, E = s["a"].shape[0], s["K"], s["N"], s["E"]
    p = b.f8_params(R, K, N, E=E, out_dtype=E4M3 if s["out"] == "e4m3" else CODE[s["out"]], swiglu_limit=LIMIT)
    if op == "matmul":
        b.matmul_f8(p, s["a"], s["a_scale"], s["w"], s["w_scale"], s["c"], s["ws"], offsets=s["offsets"],
                    sorted_pair=s["sorted_pair"], topk_w=s["topk_w"])
        return {"c": s["c"]}
    b.gated_f8(p, s["a"], s["a_scale"], s["w_gate"], s["s_gate"], s["w_up"], s["s_up"], s["h"], s["ws"],
               h_scale=s["h_scale"], offsets=s["offsets"])
    return {"h": s["h"]} if s["h_scale"] is None else {"h": s["h"], "h_scale": s["h_scale"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
    if op in ("norm_in", "norm_out"):
        n, st, bl = case["T"] * case["d"], size[case["stream"]], size[case["block"]]
        if op == "norm_in":  # x in, y out; then dy, x and the residual's gradient in, dx out
            b = n * (st + bl) + (n * (bl + 3 * st) if case["train"] else n)
            return {"bytes": b, "flops": n * (18 if case["train"] else 8)}
        b = n * (2 * st + 2 * bl) + (n * (2 * st + 2 * bl) if case["train"] else 0)
        return {"bytes": b, "flops": n * (30 if case["train"] else 14)}
    if op == "quantize":
        if case["weights"]:
            n = case["E"] * case["K"] * case["N"]
            return {"bytes": n * (size[case["src"]] + 1), "flops": 3 * n}
        n = case["T"] * case["K"]
        return {"bytes": n * size[case["src"]] + n * case["k"] * (1 + 4 / 128), "flops": 3 * n * case["k"]}
    R, E, K, N = case["T"] * case["k"], case["E"], case["K"], case["N"]
    touched, mats = min(E, R), 1 if op == "matmul" else 2
    out = R * N * size[case["out"]] + (R * N / 32 if case["out"] == "e4m3" else 0)
    return {"bytes": R * K * (1 + 4 / 128) + mats * touched * N * K + out, "flops": 2.0 * R * N * K * mats}


# ------------------------------------------------------------------------------ definitions in 64 bits

def _e4m3_64(v):
    """The nearest e4m3 value (ties to even), from the format's definition: 3 bits of fraction, 2^-6 the least exponent."""
    a = v.abs().clamp(max=QMAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(a / step) * step * torch.sign(v)


def _by_128_64(v):
    """Columns of v (64 bits) in groups of 128: the values in units of each group's scale, and the scales."""
    K = v.shape[1]
    q, sc = torch.empty_like(v), []
    for k0 in range(0, K, 128):
        blk = v[:, k0:k0 + 128]
        s = (blk.abs().max(dim=1).values / QMAX).float().double().clamp(min=SMIN)
        q[:, k0:k0 + 128] = _e4m3_64(blk / s[:, None])
        sc.append(s)
    return q, torch.stack(sc)


def _stats_64(v, kind):
    m = v.sum(dim=1, keepdim=True) / v.shape[1] if kind == "layer" else 0.0
    var = ((v - m) ** 2).sum(dim=1, keepdim=True) / v.shape[1]
    return (v - m) * (var + EPS) ** -0.5, (var + EPS) ** -0.5


def _grad_64(vhat, rstd, g, kind):
    d = vhat.shape[1]
    inner = (g * vhat).sum(dim=1, keepdim=True) / d
    centre = g.sum(dim=1, keepdim=True) / d if kind == "layer" else 0.0
    return rstd * (g - centre - vhat * inner)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_in":
        x, w = s["x"].double(), s["weight"].double()
        xh, rstd = _stats_64(x, s["kind"])
        if not s["train"]:
            q, sc = _by_128_64(xh * w)
            return {"y": xh * w, "q8": q, "s8": sc}
        dy = s["dy"].double()
        return {"y": xh * w, "dx": s["dres"].double() + _grad_64(xh, rstd, dy * w, s["kind"]),
                "dw": (dy * xh).sum(dim=0)}
    if op == "norm_out":
        r, v, w = s["resid"].double(), s["block_out"].double(), s["weight"].double()
        vh, rstd = _stats_64(v, s["kind"])
        n = vh * w + (s["bias_t"].double() if s["bias_t"] is not None else 0.0)
        gate = torch.ones(1, device=v.device, dtype=v.dtype) if s["gate_t"] is None else s["gate_t"].double()
        gate = gate[:, None] if s["gate"] == "token" else gate[None, :]
        out = s["alpha"] * r + s["beta"] * gate * n
        got = {"out": out, "x_next": None, "dresid": None, "dy": None, "dw": None, "db": None, "dgate": None}
        # the next norm reads the stream as it is stored
        got["x_next"] = _stats_64(out.to(s["out"].dtype).double(), s["kind"])[0] * s["next_weight"].double()
        if s["train"]:
            do = s["dout"].double()
            dn = do * gate * s["beta"]
            got.update(dresid=s["alpha"] * do, dy=_grad_64(vh, rstd, dn * w, s["kind"]), dw=(dn * vh).sum(dim=0))
            if s["bias_t"] is not None:
                got["db"] = dn.sum(dim=0)
            if s["gate_t"] is not None:
                got["dgate"] = (do * n).sum(dim=1 if s["gate"] == "token" else 0) * s["beta"]
        return got
    if op == "quantize":
        if not s["weights"]:
            q, sc = _by_128_64(s["x"].double()[s["index"].long()])
            return {"q": q, "s": sc}
        w = s["w"].double()
        w = w.transpose(1, 2) if s["transposed"] else w
        q, sc = torch.empty(w.shape, dtype=torch.float64, device=w.device), torch.empty(s["s"].shape, device=w.device).double()
        for i in range(sc.shape[1]):
            for j in range(sc.shape[2]):
                blk = w[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                sc[:, i, j] = (blk.abs().amax(dim=(1, 2)) / QMAX).float().double().clamp(min=SMIN)
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _e4m3_64(blk / sc[:, i, j, None, None])
        return {"q": q, "s": sc}

    def product(q, sc):
        """By expert and block of 128 along K, each with its scales."""
        off = [0, s["a"].shape[0]] if s["offsets"] is None else s["offsets"].tolist()
        c = torch.zeros(s["a"].shape[0], case["N"], dtype=torch.float64, device=s["a"].device)
        block = torch.arange(case["N"], device=c.device) // 128
        for e in range(len(off) - 1):
            r0, r1 = off[e], off[e + 1]
            if r0 == r1:
                continue
            for j in range(sc.shape[2]):
                left = s["a"][r0:r1, 128 * j:128 * j + 128].double() * s["a_scale"][j, r0:r1, None].double()
                right = q[e, :, 128 * j:128 * j + 128].double() * sc[e, block, j, None].double()
                c[r0:r1] += left @ right.t()
        return c

    if op == "matmul":
        c = product(s["w"], s["w_scale"])
        if s["topk_w"] is not None:
            c = c * s["topk_w"].double().reshape(-1)[s["sorted_pair"].long(), None]
        return {"c": c}
    g = product(s["w_gate"], s["s_gate"]).clamp(-LIMIT, LIMIT)
    u = product(s["w_up"], s["s_up"]).clamp(-LIMIT, LIMIT)
    h = g * torch.sigmoid(g) * u
    if case["out"] != "e4m3":
        return {"h": h}
    q, sc = _by_128_64(h)
    return {"h": q, "h_scale": sc}

"""The block's operators as they are used, one after the other.

Serving: norm -> router -> permutation -> rows to e4m3 by token -> gated experts -> down with the
gate weights -> combine -> post norm, gate, residual and the next block's norm, with a capacity drop.
Every stage is checked against the fp64 oracle on what the stage before it really wrote, with that
stage's own tolerance (see the operators' tests), and the whole once more from a replayed graph.

Training: the norm after a block and the next block's norm, whose gradients meet in the residual
stream, against torch's double-precision autograd of the whole.
"""
import numpy as np
import pytest
import torch

import oracle
from mixture_experts_routed_04_b200 import binding as b
from oracle import block as o

pytestmark = pytest.mark.gpu

U, U2 = 2.0 ** -24, 2.0 ** -23
EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def within(got, ref, tol, what):
    excess = np.abs(np.asarray(got) - ref) - tol
    assert (excess <= 0).all(), f"{what}: worst by {excess.max():.3e}"


class Layer:
    """A block with its experts in e4m3 and every buffer it needs."""

    def __init__(self, T, d, f, E, k, cf, seed=0):
        rng = np.random.default_rng(seed)
        dev = dict(device="cuda")
        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k
        n = lambda *s, std=1.0, mean=0.0: torch.from_numpy(rng.normal(mean, std, s).astype(np.float32)).cuda()  # noqa: E731
        self.resid, self.logits = n(T, d, std=2.0), n(T, E)
        self.w1, self.w2, self.w3 = n(d, std=0.1, mean=1.0), n(d, std=0.1, mean=1.0), n(d, std=0.1, mean=1.0)
        self.gate = n(T, std=0.5)
        self.wts = {}
        for name, N, K in (("gate", f, d), ("up", f, d), ("down", d, f)):
            q, s = torch.empty(E, N, K, dtype=torch.uint8, **dev), torch.empty(E, (N + 127) // 128, (K + 127) // 128, **dev)
            b.quantize_f8_weights(n(E, K, N, std=0.08), q, s, transposed=True)  # given [E, K, N], as the bf16 layer's
            self.wts[name] = (q, s)
        self.mp = b.params(T, d, f, E, k, capacity_factor=cf, swiglu_limit=7.0)
        self.np1 = b.norm_params(T, d, b.NORM_RMS, eps=EPS, block_dtype=b.DT_BF16)
        self.np2 = b.norm_params(T, d, b.NORM_RMS, b.NORM_RMS, eps=EPS, block_dtype=b.DT_F32, gate_kind=b.GATE_TOKEN, alpha=0.9, beta=0.5)
        R = self.R = b.max_rows(self.mp)
        self.gp = b.f8_params(R, d, f, E, out_dtype=b.DT_E4M3, swiglu_limit=7.0)
        self.dp = b.f8_params(R, f, d, E, out_dtype=b.DT_F16)
        i32, f32, u8 = dict(dtype=torch.int32, **dev), dict(dtype=torch.float32, **dev), dict(dtype=torch.uint8, **dev)
        self.x = torch.empty(T, d, dtype=torch.bfloat16, **dev)
        self.idx, self.tw = torch.empty(T, k, **i32), torch.empty(T, k, **f32)
        self.counts, self.kept, self.off = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.st, self.sp, self.pr = torch.zeros(R, **i32), torch.zeros(R, **i32), torch.empty(T * k, **i32)
        self.xq, self.xs = torch.zeros(R, d, **u8), torch.zeros((d + 127) // 128, R, **f32)
        self.hq, self.hs = torch.zeros(R, f, **u8), torch.zeros((f + 127) // 128, R, **f32)
        self.y = torch.zeros(R, d, dtype=torch.float16, **dev)
        self.blk, self.out, self.xn = torch.empty(T, d, **f32), torch.empty(T, d, **f32), torch.empty(T, d, **f32)
        self.ws = b.workspace(self.mp, b.WS_FORWARD)
        self.ws8 = b.f8_workspace(self.gp)

    def run(self):
        b.norm_forward(self.np1, self.resid, self.x, weight=self.w1)
        b.route(self.mp, self.logits, self.idx, self.tw, self.ws)
        b.permute(self.mp, self.idx, self.counts, self.kept, self.off, self.st, self.sp, self.pr, self.ws)
        b.quantize_f8(self.x, self.xq, self.xs, self.ws8, row_index=self.st, n_rows=self.off[self.E:])
        b.gated_f8(self.gp, self.xq, self.xs, *self.wts["gate"], *self.wts["up"], self.hq, self.ws8, h_scale=self.hs, offsets=self.off)
        b.matmul_f8(self.dp, self.hq, self.hs, *self.wts["down"], self.y, self.ws8, offsets=self.off, sorted_pair=self.sp, topk_w=self.tw)
        b.combine(self.mp, self.y, self.pr, self.off, self.blk, self.ws)
        b.norm_residual_forward(self.np2, self.resid, self.blk, self.out, weight=self.w2, gate=self.gate, next_weight=self.w3, x_next=self.xn)

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("x", "xq", "xs", "hq", "hs", "y", "blk", "out", "xn")}


@pytest.mark.parametrize("T,d,f,E,k,cf", [(1, 256, 192, 8, 2, 0.0), (96, 256, 192, 8, 2, 0.9), (300, 1088, 320, 6, 3, 0.0),
                                          (700, 512, 384, 16, 4, 1.1)])
def test_serving(T, d, f, E, k, cf):
    L = Layer(T, d, f, E, k, cf)
    L.run()
    assert b.get_error(L.ws) == 0 and b.get_error(L.ws8) == 0
    off = L.off.cpu().numpy()
    n = int(off[-1])
    assert n == T * k or cf > 0
    # the norm
    r = f64(L.resid)
    ref = o.norm(r, "rms", EPS, f64(L.w1))
    within(f64(L.x), ref, 2.0 ** -8 * np.abs(ref) + 128 * U * np.abs(ref), "x")
    # 8-bit rows, gathered: as the library defines them, bit for bit
    rq, rs = o.quantize_rows(L.x.float().cpu().numpy()[L.st.cpu().numpy()[:n]])
    assert np.array_equal(o.e4m3_values(bits(L.xq)[:n]), rq) and np.array_equal(L.xs.cpu().numpy()[:, :n], rs)
    # the gated experts
    W = {}
    for name, (q, s) in L.wts.items():
        qs, ss = bits(q), s.cpu().numpy()
        W[name] = [o.dequantize_weights(o.e4m3_values(qs[e]), ss[e]) for e in range(E)]
    A = np.zeros((L.R, d))
    A[:n] = o.dequantize_rows(rq, rs)
    g, u = (o.matmul(A, off, lambda e: W[m][e])[:n] for m in ("gate", "up"))
    dg, du = ((132 + d // 128 + 1) * U2 * o.matmul(np.abs(A), off, lambda e: np.abs(W[m][e]))[:n] for m in ("gate", "up"))
    h = o.gated(g, u, 7.0)
    gc, uc = np.clip(g, -7, 7), np.clip(u, -7, 7)
    th = 1.1 * np.abs(uc) * dg + np.abs(o.gated(gc, 1.0, 0.0)) * du + 1.1 * dg * du + 2.0 ** -19 * np.abs(h)
    hs = L.hs.cpu().numpy()[:, :n]
    got = o.dequantize_rows(o.e4m3_values(bits(L.hq)[:n]), hs)
    step = np.repeat(hs.astype(np.float64), 128, 0)[:f].T
    within(got, h, th + 2.0 ** -4 * (np.abs(h) + th) + 2.0 ** -10 * step, "h")
    # down, weighted, from the h that was written
    H = np.zeros((L.R, f))
    H[:n] = got
    pair = L.sp.cpu().numpy()[:n]
    w = f64(L.tw).reshape(-1)[pair][:, None]
    y = o.matmul(H, off, lambda e: W["down"][e])[:n] * w
    ty = (133 + f // 128 + 1) * U2 * o.matmul(np.abs(H), off, lambda e: np.abs(W["down"][e]))[:n] * w
    within(f64(L.y)[:n], y, ty + 2.0 ** -11 * (np.abs(y) + ty) + 2.0 ** -25, "y")
    # the combine and the post norm, from what was written
    blk = oracle.combine(f64(L.y), L.pr.cpu().numpy().reshape(-1), np.ones((T, k)), T, k)
    within(f64(L.blk), blk, k * U * oracle.combine(np.abs(f64(L.y)), L.pr.cpu().numpy().reshape(-1), np.ones((T, k)), T, k), "combine")
    v = f64(L.blk)
    gt = f64(L.gate)[:, None]
    ref = o.norm_residual(r, v, "rms", EPS, f64(L.w2), None, 0.0, gt, 0.9, 0.5)
    part = np.abs(0.5 * gt * o.norm(v, "rms", EPS, f64(L.w2)))
    within(f64(L.out), ref, U * 8 * (np.abs(0.9 * r) + np.abs(ref)) + 320 * U * part, "out")
    nref = o.norm(f64(L.out), "rms", EPS, f64(L.w3))
    within(f64(L.xn), nref, 128 * U * np.abs(nref), "x_next")
    # the same from a graph, twice
    first = L.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    for t in (L.x, L.xq, L.hq, L.y, L.blk, L.out, L.xn):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for name, t in L.outputs().items():
        assert torch.equal(t, first[name]), name


def test_training():
    """L = <c1, x_next> + <c2, out>, out = alpha r + beta gate N(y), x_next = N2(out), all in fp32. The two
    backward calls run in turn, the second's result joining the stream's gradient. Each adds at most the
    rounding that its own test allows (160 * 2^-24 of sums of magnitudes); over both, and with sums of
    256 tokens, 1e-4 of the gradient's largest entry is above that by more than ten times."""
    T, d = 256, 320
    rng = np.random.default_rng(3)
    n = lambda *s, std=1.0, mean=0.0: torch.from_numpy(rng.normal(mean, std, s).astype(np.float32)).cuda()  # noqa: E731
    r, y, w, bias, gate, w2 = n(T, d), n(T, d), n(d, mean=1.0, std=0.2), n(d), n(d), n(d, mean=1.0, std=0.2)
    c1, c2 = n(T, d), n(T, d)
    f32 = dict(stream_dtype=b.DT_F32, block_dtype=b.DT_F32)
    p = b.norm_params(T, d, b.NORM_LAYER, b.NORM_RMS, eps=EPS, gate_kind=b.GATE_CHANNEL, alpha=0.8, beta=1.5, **f32)
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    out, xn, m, rs, m2, rs2 = e(T, d), e(T, d), e(T), e(T), e(T), e(T)
    b.norm_residual_forward(p, r, y, out, weight=w, bias=bias, gate=gate, mean=m, rstd=rs, next_weight=w2, x_next=xn, next_mean=m2, next_rstd=rs2)
    p2 = b.norm_params(T, d, b.NORM_RMS, eps=EPS, **f32)
    dout, dw2 = e(T, d), e(d)
    b.norm_backward(p2, out, c1, m2, rs2, dout, b.norm_workspace(p2), weight=w2, dres=c2, dw=dw2)
    dr, dy, dw, db, dgate = e(T, d), e(T, d), e(d), e(d), e(d)
    b.norm_residual_backward(p, y, dout, m, rs, dy, b.norm_workspace(p), weight=w, bias=bias, gate=gate, dresid=dr, dw=dw, db=db, dgate=dgate)

    v = {k: t.double().requires_grad_() for k, t in dict(r=r, y=y, w=w, b=bias, g=gate, w2=w2).items()}
    hat = torch.nn.functional.layer_norm(v["y"], (d,), v["w"], v["b"], EPS)
    o64 = 0.8 * v["r"] + 1.5 * v["g"] * hat
    x64 = o64 / torch.sqrt((o64 * o64).mean(1, keepdim=True) + EPS) * v["w2"]
    (x64 * c1.double()).sum().add((o64 * c2.double()).sum()).backward()
    for got, name in ((dr, "r"), (dy, "y"), (dw, "w"), (db, "b"), (dgate, "g"), (dw2, "w2")):
        ref = v[name].grad
        assert float((got.double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()), name


def test_two_streams_at_once():
    """Two layers, each with its own buffers, running on two streams at the same time, give what each gives alone."""
    A, B = Layer(96, 256, 192, 8, 2, 0.0, seed=1), Layer(200, 512, 256, 16, 4, 0.0, seed=2)
    want = []
    for L in (A, B):
        L.run()
        want.append(L.outputs())
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L, st in zip((A, B), s):
            with torch.cuda.stream(st):
                L.run()
    torch.cuda.synchronize()
    for L, w in zip((A, B), want):
        for name, t in L.outputs().items():
            assert torch.equal(t, w[name]), name


def test_launches():
    """One launch a call, two for a backward call with sums over tokens."""
    L = Layer(96, 256, 192, 8, 2, 0.0)
    L.run()
    T, d = 96, 256
    bp = b.norm_params(T, d, block_dtype=b.DT_F32)
    rs, dx, dw = torch.ones(T, device="cuda"), torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
    ws = b.norm_workspace(bp)
    b.norm_backward(bp, L.resid, L.blk, None, rs, dx, ws, weight=L.w1, dw=dw)
    torch.cuda.synchronize()
    b.profile_collect()
    b.profile_enable(True)
    try:
        L.run()
        b.norm_backward(bp, L.resid, L.blk, None, rs, dx, ws, weight=L.w1, dw=dw)
        b.norm_backward(bp, L.resid, L.blk, None, rs, dx, weight=L.w1)
        torch.cuda.synchronize()
        n = {k: c for k, (_, c) in b.profile_collect().items() if c}
    finally:
        b.profile_enable(False)
    assert n["norm"] == 2 and n["quant_f8"] == 1 and n.get("tc_f8", 0) + n.get("stream_f8", 0) == 2 and n["norm_bwd"] == 3

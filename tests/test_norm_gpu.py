"""The norms before and after a block (moe_norm_*), forward and backward, against the fp64 oracle.

Tolerances, element by element, from arithmetic. An output rounds once: half a step of its dtype
(eps/2 of the value; fp16 below 2^-14 half of 2^-24). Before that everything is fp32 with
relative error 2^-24 an operation. A row's sum of d <= 8192 terms runs through at most 32 terms a
thread, 5 shuffles and 8 warps (45 roundings), rstd takes half of that and a few more, xhat that
and two more: below 64 * 2^-24 of |xhat| + rstd mean|x| (the second term: the mean's own error).
Gradients add two more such sums and their products: 160 * 2^-24 of the sums of magnitudes. Sums
over tokens run through at most T / groups rows, groups / 32 partial sums and 5 shuffles, below
160 roundings for the sizes here.
"""
import numpy as np
import pytest
import torch

from mixture_experts_routed_04_b200 import binding as b
from oracle import block as o

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KIND = {"none": b.NORM_NONE, "rms": b.NORM_RMS, "layer": b.NORM_LAYER}
GATE = {"none": b.GATE_NONE, "channel": b.GATE_CHANNEL, "token": b.GATE_TOKEN}
DT = {"f32": (b.DT_F32, torch.float32), "bf16": (b.DT_BF16, torch.bfloat16), "f16": (b.DT_F16, torch.float16)}
EPS = 1e-6


def half_step(ref, dtype):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all(), f"{what}: not finite"
    excess = np.abs(got - ref) - tol
    assert (excess <= 0).all(), f"{what}: {int((excess > 0).sum())} of {excess.size} off, worst by {excess.max():.3e}"


def make(rng, shape, dtype, std=1.0, mean=0.0):
    return torch.from_numpy(rng.normal(mean, std, shape).astype(np.float32)).to("cuda").to(dtype)


def rows_of(t, ld, shift=0):
    """t's rows in a larger buffer: ld elements from row to row, the base `shift` elements in."""
    T, d = t.shape
    buf = torch.full((T * ld + shift + 16,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:shift + T * ld].view(T, ld)[:, :d]
    v.copy_(t)
    return v


# T, d, stride and shift of the rows (0, 0: dense), mean of x, weight offset
SIZES = [(1, 1, 0, 0, 0.0, 0.0), (1, 8, 0, 0, 0.0, 1.0), (3, 7, 0, 0, 0.0, 0.0), (5, 128, 0, 0, 4.0, 0.0),
         (37, 129, 0, 0, 0.0, 0.0), (9, 255, 300, 0, 0.0, 1.0), (33, 256, 264, 8, 0.0, 0.0), (17, 1000, 0, 1, 0.0, 0.0),
         (300, 1024, 0, 0, 30.0, 0.0), (64, 2048, 0, 0, 0.0, 0.0), (2, 4096, 0, 0, 0.0, 1.0), (3, 4100, 0, 0, 0.0, 0.0),
         (2, 8192, 0, 0, 0.0, 0.0), (2, 8191, 0, 0, 1.0, 0.0), (1700, 320, 0, 0, 0.0, 0.0),
         # many rows: the rows ahead pass through shared memory, with 1, 2, 4 and 8 warps a row
         (1201, 248, 0, 0, 0.0, 0.0), (1251, 1024, 1032, 8, 0.0, 0.0), (613, 2048, 0, 0, 2.0, 0.0), (301, 4096, 0, 0, 0.0, 1.0),
         (151, 8192, 0, 0, 0.0, 0.0), (601, 2040, 0, 0, 0.0, 0.0), (1300, 1023, 0, 0, 0.0, 0.0), (160, 8185, 0, 0, 0.0, 0.0)]


def tol_norm(x, kind, w, bias, offset):
    mean, rstd = o.norm_stats(x, kind, EPS)
    xa = np.abs((x - mean) * rstd) + rstd * np.mean(np.abs(x), axis=1, keepdims=True) if kind != "none" else np.abs(x)
    wm = 1.0 if w is None else np.abs(w + offset)
    return xa, 64 * U * (xa * wm + (0.0 if bias is None else np.abs(bias)))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream,block,par", [("f32", "bf16", "f32"), ("bf16", "bf16", "bf16"), ("f16", "f32", "f16")])
@pytest.mark.parametrize("size", SIZES)
def test_before(size, stream, block, par, kind):
    T, d, ld, shift, mean, off = size
    rng = np.random.default_rng([T, d])
    (sc, st), (bc, bl), (pc, pt) = DT[stream], DT[block], DT[par]
    ld = ld or d
    x = rows_of(make(rng, (T, d), st, 2.0, mean), ld, shift)
    w, bias = make(rng, (d,), pt, 0.3, 1.0), make(rng, (d,), pt)
    p = b.norm_params(T, d, KIND[kind], eps=EPS, weight_offset=off, stream_dtype=sc, block_dtype=bc, param_dtype=pc,
                      ld_stream=ld, ld_block=ld)
    y = rows_of(torch.zeros(T, d, dtype=bl, device="cuda"), ld, shift)
    m, r = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    b.norm_forward(p, x, y, weight=w, bias=bias, mean=m, rstd=r)
    xr, wr, br = f64(x), f64(w), f64(bias)
    ref = o.norm(xr, kind, EPS, wr, br, off)
    xa, tol = tol_norm(xr, kind, wr, br, off)
    close(y, ref, half_step(ref, bl) + tol, "y")
    mean_r, rstd_r = o.norm_stats(xr, kind, EPS)
    close(r, rstd_r[:, 0], 64 * U * rstd_r[:, 0], "rstd")
    close(m, mean_r[:, 0], 64 * U * np.mean(np.abs(xr), axis=1), "mean")

    dy, dres = rows_of(make(rng, (T, d), bl), ld, shift), rows_of(make(rng, (T, d), st), ld, shift)
    dx = rows_of(torch.zeros(T, d, dtype=st, device="cuda"), ld, shift)
    dw, db = torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
    ws = b.norm_workspace(p)
    b.norm_backward(p, x, dy, m, r, dx, ws, weight=w, dres=dres, dw=dw, db=db)
    dyr, dresr = f64(dy), f64(dres)
    rdx, rdw, rdb = o.norm_backward(xr, dyr, kind, EPS, wr, off)
    g = np.abs(dyr * (wr + off))
    mag = rstd_r * (g + g.mean(axis=1, keepdims=True) + xa * np.mean(g * xa, axis=1, keepdims=True))
    close(dx, dresr + rdx, half_step(dresr + rdx, st) + 160 * U * (np.abs(dresr) + mag), "dx")
    close(dw, rdw, 160 * U * np.sum(np.abs(dyr) * xa, axis=0), "dw")
    close(db, rdb, 160 * U * np.sum(np.abs(dyr), axis=0), "db")
    # without the residual's gradient and the weights' sums: no workspace, the same rows
    dx2 = torch.empty(T, d, dtype=st, device="cuda") if ld == d else rows_of(torch.zeros(T, d, dtype=st, device="cuda"), ld)
    b.norm_backward(p, x, dy, m, r, dx2, weight=w)
    close(dx2, rdx, half_step(rdx, st) + 160 * U * mag, "dx alone")


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("stream,block", [("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("size", [(1, 3, 0, 0), (5, 64, 0, 0), (37, 129, 0, 0), (9, 1000, 1008, 8), (130, 1024, 0, 0),
                                  (3, 4096, 0, 0), (21, 2047, 2100, 3), (2, 8192, 0, 0), (2, 6001, 0, 0),
                                  (1251, 512, 0, 0), (620, 2048, 2056, 0), (303, 4096, 0, 0), (152, 8192, 0, 0), (640, 1999, 0, 0)])
def test_after(size, stream, block, gate, kind):
    T, d, ld, shift = size
    rng = np.random.default_rng([T, d, 1])
    (sc, st), (bc, bl) = DT[stream], DT[block]
    ld, alpha, beta = ld or d, 0.75, -1.5
    resid, y = rows_of(make(rng, (T, d), st, 3.0), ld, shift), rows_of(make(rng, (T, d), bl, 2.0, 0.5), ld, shift)
    par = kind != "none"
    w = make(rng, (d,), torch.float32, 0.3, 1.0) if par else None
    bias = make(rng, (d,), torch.float32) if par else None
    gt = {"none": None, "channel": make(rng, (d,), torch.float32), "token": make(rng, (T,), torch.float32)}[gate]
    nw, nb = make(rng, (d,), torch.float32, 0.3, 1.0), make(rng, (d,), torch.float32)
    p = b.norm_params(T, d, KIND[kind], b.NORM_RMS, eps=EPS, stream_dtype=sc, block_dtype=bc, gate_kind=GATE[gate],
                      alpha=alpha, beta=beta, ld_stream=ld, ld_block=ld)
    out = rows_of(torch.zeros(T, d, dtype=st, device="cuda"), ld, shift)
    xn = rows_of(torch.zeros(T, d, dtype=bl, device="cuda"), ld, shift)
    m, r = (torch.empty(T, device="cuda"), torch.empty(T, device="cuda")) if par else (None, None)
    b.norm_residual_forward(p, resid, y, out, weight=w, bias=bias, gate=gt, mean=m, rstd=r, next_weight=nw,
                            next_bias=nb, x_next=xn)
    rr, yr, nwr, nbr = f64(resid), f64(y), f64(nw), f64(nb)
    wr, br = (f64(w), f64(bias)) if par else (None, None)
    gr = None if gt is None else f64(gt) if gate == "channel" else f64(gt)[:, None]
    gm = abs(beta) * (1.0 if gr is None else np.abs(gr))
    ref = o.norm_residual(rr, yr, kind, EPS, wr, br, 0.0, gr, alpha, beta)
    xa, tol = tol_norm(yr, kind, wr, br, 0.0)
    close(out, ref, half_step(ref, st) + gm * tol + 4 * U * (np.abs(alpha * rr) + np.abs(ref)) + 4 * gm * tol, "out")
    outr = f64(out)  # the next norm takes out as it is stored
    nref = o.norm(outr, "rms", EPS, nwr, nbr)
    close(xn, nref, half_step(nref, bl) + tol_norm(outr, "rms", nwr, nbr, 0.0)[1], "x_next")
    # in place, and without the next norm
    p1 = b.norm_params(T, d, KIND[kind], eps=EPS, stream_dtype=sc, block_dtype=bc, gate_kind=GATE[gate], alpha=alpha,
                       beta=beta, ld_stream=ld, ld_block=ld)
    same = rows_of(resid, ld, shift)
    b.norm_residual_forward(p1, same, y, same, weight=w, bias=bias, gate=gt)
    assert torch.equal(same, out)

    dout = rows_of(make(rng, (T, d), st), ld, shift)
    dr, dy = rows_of(torch.zeros(T, d, dtype=st, device="cuda"), ld, shift), rows_of(torch.zeros(T, d, dtype=bl, device="cuda"), ld, shift)
    nan = float("nan")
    dw, db = (torch.full((d,), nan, device="cuda"), torch.full((d,), nan, device="cuda")) if par else (None, None)
    dg = None if gt is None else torch.full(gt.shape, nan, device="cuda")
    b.norm_residual_backward(p, y, dout, m, r, dy, b.norm_workspace(p), weight=w, bias=bias, gate=gt, dresid=dr, dw=dw,
                             db=db, dgate=dg)
    do = f64(dout)
    rdr, rdy, rdw, rdb, rdg = o.norm_residual_backward(yr, do, kind, EPS, wr, br, 0.0, gr, alpha, beta)
    close(dr, rdr, half_step(rdr, st) + 2 * U * np.abs(rdr), "dr")
    D = gm * np.abs(do)
    g = D if wr is None else D * np.abs(wr)
    rstd = o.norm_stats(yr, kind, EPS)[1]
    mag = rstd * (g + (0 if kind == "none" else g.mean(axis=1, keepdims=True) + xa * np.mean(g * xa, axis=1, keepdims=True)))
    close(dy, rdy, half_step(rdy, bl) + 160 * U * mag, "dy")
    if par:
        close(dw, rdw, 160 * U * np.sum(D * xa, axis=0), "dw")
        close(db, rdb, 160 * U * np.sum(D * np.ones_like(do), axis=0), "db")
    nmag = xa * (1.0 if wr is None else np.abs(wr)) + (0.0 if br is None else np.abs(br))
    if gate == "channel":
        close(dg, rdg.sum(axis=0), 160 * U * np.sum(abs(beta) * np.abs(do) * nmag, axis=0), "dgate")
    if gate == "token":
        close(dg, rdg.sum(axis=1), 160 * U * np.sum(abs(beta) * np.abs(do) * nmag, axis=1), "dgate")


def test_gradients_against_differences():
    """The kernels' gradients of L = sum(c * out) against central differences of the kernels' own
    forward in fp32: a step h gives a truncation error of order h^2 and a rounding error of
    eps * sum|c out| / h; with h = 2^-6 and values of order one both are below 2e-3."""
    T, d = 4, 48
    rng = np.random.default_rng(9)
    f32 = dict(stream_dtype=b.DT_F32, block_dtype=b.DT_F32)
    p = b.norm_params(T, d, b.NORM_LAYER, eps=1e-2, gate_kind=b.GATE_TOKEN, alpha=0.5, beta=2.0, **f32)
    v = {n: make(rng, s, torch.float32, 1.0, m) for n, s, m in (("resid", (T, d), 0), ("y", (T, d), 0), ("weight", (d,), 1),
                                                                ("bias", (d,), 0), ("gate", (T,), 1))}
    c = make(rng, (T, d), torch.float32)

    def loss(**over):
        a = {**v, **over}
        out = torch.empty(T, d, device="cuda")
        b.norm_residual_forward(p, a["resid"], a["y"], out, weight=a["weight"], bias=a["bias"], gate=a["gate"])
        return float((out.double() * c.double()).sum())

    m, r, out = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, d, device="cuda")
    b.norm_residual_forward(p, v["resid"], v["y"], out, weight=v["weight"], bias=v["bias"], gate=v["gate"], mean=m, rstd=r)
    got = dict(resid=torch.empty(T, d, device="cuda"), y=torch.empty(T, d, device="cuda"), weight=torch.empty(d, device="cuda"),
               bias=torch.empty(d, device="cuda"), gate=torch.empty(T, device="cuda"))
    b.norm_residual_backward(p, v["y"], c, m, r, got["y"], b.norm_workspace(p), weight=v["weight"], bias=v["bias"],
                             gate=v["gate"], dresid=got["resid"], dw=got["weight"], db=got["bias"], dgate=got["gate"])
    h = 2.0 ** -6
    for name, t in v.items():
        for i in rng.choice(t.numel(), 4, replace=False):
            up, dn = t.clone(), t.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            assert abs(num - float(got[name].view(-1)[i])) <= 2e-3 * max(1.0, abs(num)), (name, i)


@pytest.mark.parametrize("d", [16, 128, 144, 1000 // 16 * 16, 4096, 8192])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_rows_in_8_bits(T, d):
    """q8, s8 are what moe_quantize_f8 makes of the fp32 result: with the result stored as fp32,
    bit for bit. A row of zeros gives zeros with the least scale."""
    rng = np.random.default_rng([T, d, 3])
    x, w = make(rng, (T, d), torch.float32, 2.0), make(rng, (d,), torch.float32, 0.3, 1.0)
    x[T // 2, :128] = 0
    p = b.norm_params(T, d, b.NORM_RMS, eps=EPS, block_dtype=b.DT_F32)
    y, q, s = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty((d + 127) // 128, T, device="cuda")
    b.norm_forward(p, x, y, weight=w, q8=q, s8=s)
    rq, rs = o.quantize_rows(y.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(o.e4m3_values(q.cpu().numpy()), rq)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    b.norm_forward(p, x, None, weight=w, q8=q2, s8=s2)  # 8-bit rows alone
    assert torch.equal(q, q2) and torch.equal(s, s2)
    # after the block, of the next norm's result
    pj = b.norm_params(T, d, b.NORM_NONE, b.NORM_RMS, eps=EPS, block_dtype=b.DT_F32)
    out, xn = torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda")
    b.norm_residual_forward(pj, x, y, out, next_weight=w, x_next=xn, q8=q, s8=s)
    rq, rs = o.quantize_rows(xn.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(o.e4m3_values(q.cpu().numpy()), rq)


def test_empty_batch_and_zero_gradients():
    d = 96
    w = torch.ones(d, device="cuda")
    p = b.norm_params(0, d, gate_kind=b.GATE_NONE)
    e32, e16 = torch.empty(0, d, device="cuda"), torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    b.norm_forward(p, e32, e16, weight=w)
    dw, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    b.norm_backward(p, e32, e16, None, None, e32, b.norm_workspace(p), weight=w, dw=dw, db=db)
    pg = b.norm_params(0, d, gate_kind=b.GATE_CHANNEL)
    dg = torch.full((d,), 7.0, device="cuda")
    b.norm_residual_backward(pg, e16, e32, None, None, e16, b.norm_workspace(pg), weight=w, gate=w, dgate=dg)
    torch.cuda.synchronize()
    assert float(dw.abs().sum() + db.abs().sum() + dg.abs().sum()) == 0.0


def test_same_bits_streams_and_graphs():
    """Two calls give the same bits; so do another stream and a replayed graph of forward and backward."""
    T, d = 777, 640
    rng = np.random.default_rng(4)
    x, w, dy = make(rng, (T, d), torch.bfloat16), make(rng, (d,), torch.float32, 0.3, 1.0), make(rng, (T, d), torch.bfloat16)
    p = b.norm_params(T, d, b.NORM_LAYER, stream_dtype=b.DT_BF16)

    def step(v):
        b.norm_forward(p, x, v["y"], weight=w, mean=v["m"], rstd=v["r"])
        b.norm_backward(p, x, dy, v["m"], v["r"], v["dx"], v["ws"], weight=w, dw=v["dw"], db=v["db"])

    def bufs():
        f = dict(device="cuda")
        return dict(y=torch.zeros(T, d, dtype=torch.bfloat16, **f), m=torch.zeros(T, **f), r=torch.zeros(T, **f),
                    dx=torch.zeros(T, d, dtype=torch.bfloat16, **f), dw=torch.zeros(d, **f), db=torch.zeros(d, **f),
                    ws=b.norm_workspace(p))
    one, two, three = bufs(), bufs(), bufs()
    step(one)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(two)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(three)
    for n in ("y", "dx", "dw", "db"):
        three[n].zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for n in ("y", "m", "r", "dx", "dw", "db"):
        assert torch.equal(one[n], two[n]) and torch.equal(one[n], three[n]), n


def test_an_infinity_stays_in_its_row():
    T, d = 6, 256
    x = torch.randn(T, d, device="cuda")
    x[2, 5], x[4, 7] = float("inf"), float("nan")
    p = b.norm_params(T, d, block_dtype=b.DT_F32)
    y, q, s = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(2, T, device="cuda")
    b.norm_forward(p, x, y, q8=q, s8=s)
    back = torch.from_numpy(o.dequantize_rows(o.e4m3_values(q.cpu().numpy()), s.cpu().numpy()))
    for r in range(T):
        assert bool(torch.isfinite(y[r]).all()) == (r not in (2, 4))
        assert bool(torch.isfinite(back[r]).all()) == (r not in (2, 4))


def test_tensors_that_do_not_fit_are_refused():
    T, d = 4, 64
    p = b.norm_params(T, d)
    x, y = torch.randn(T, d, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(b.MoeError):
        b.norm_forward(p, x[:, :32], y)
    with pytest.raises(b.MoeError):
        b.norm_forward(p, x.t().contiguous().t(), y)  # columns are not neighbours
    with pytest.raises(b.MoeError):
        b.norm_forward(p, x, y.float())
    with pytest.raises(b.MoeError):
        b.norm_forward(p, x.cpu(), y)
    with pytest.raises(b.MoeError):  # 8-bit rows of a length that is no multiple of 16
        b.norm_forward(b.norm_params(T, 24), x[:, :24].contiguous(), y[:, :24].contiguous(),
                       q8=torch.empty(T, 24, dtype=torch.uint8, device="cuda"), s8=torch.empty(1, T, device="cuda"))
    with pytest.raises(b.MoeError):  # a workspace that is too small
        b.norm_backward(p, x, y, torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x),
                        torch.zeros(256, dtype=torch.uint8, device="cuda"), dw=torch.empty(d, device="cuda"),
                        weight=torch.ones(d, device="cuda"))


# Many rows of 8 bits: copied ahead, several rows a block, the last block of rows not full (rows a block:
# 8, 4, 2 or 1 by d). 256 to 4096 are whole numbers of the layout's groups, the others end inside one.
@pytest.mark.parametrize("T,d", [(1201, 256), (1185, 512), (1203, 512), (593, 1024), (1001, 1024), (301, 2048), (613, 2048),
                                 (303, 4096), (4095, 256), (1201, 240), (613, 2032), (303, 4080), (151, 8192)])
@pytest.mark.parametrize("stream,kind", [("f32", "rms"), ("bf16", "layer"), ("f16", "rms")])
def test_many_rows_in_8_bits(T, d, stream, kind):
    rng = np.random.default_rng([T, d, 4])
    sc, st = DT[stream]
    x = make(rng, (T, d), st, 2.0)
    w, bias, gate = make(rng, (d,), torch.float32, 0.3, 1.0), make(rng, (d,), torch.float32), make(rng, (T,), torch.float32)

    def rows8():
        return (torch.full((T, d), 77, dtype=torch.uint8, device="cuda"), torch.full(((d + 127) // 128, T), -5.0, device="cuda"))

    def same(q, s, y, what):
        rq, rs = o.quantize_rows(y.cpu().numpy())
        gs, gq = s.cpu().numpy(), o.e4m3_values(q.cpu().numpy())
        assert np.array_equal(gs[:, 0], rs[:, 0]) and np.array_equal(gq[0], rq[0]), f"{what}: row 0"
        assert np.array_equal(gs, rs) and np.array_equal(gq, rq), what
    p = b.norm_params(T, d, KIND[kind], eps=EPS, stream_dtype=sc, block_dtype=b.DT_F32)
    y, (q, s) = torch.empty(T, d, device="cuda"), rows8()
    b.norm_forward(p, x, y, weight=w, bias=bias, q8=q, s8=s)
    same(q, s, y, "before the block")
    q2, s2 = rows8()
    b.norm_forward(p, x, None, weight=w, bias=bias, q8=q2, s8=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    pj = b.norm_params(T, d, KIND[kind], KIND[kind], eps=EPS, stream_dtype=sc, block_dtype=b.DT_F32, gate_kind=b.GATE_TOKEN,
                       alpha=0.75, beta=-1.5)
    out, xn, (q, s) = torch.empty(T, d, dtype=st, device="cuda"), torch.empty(T, d, device="cuda"), rows8()
    b.norm_residual_forward(pj, x, y, out, weight=w, bias=bias, gate=gate, next_weight=w, next_bias=bias, x_next=xn, q8=q, s8=s)
    same(q, s, xn, "after the block")

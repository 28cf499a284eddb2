"""Products in 8-bit floating point (moe_quantize_f8, moe_matmul_f8, moe_gated_f8) against the fp64 oracle.

Rounding to e4m3 is defined in fp32 operations and compared bit for bit. A product's error, from
arithmetic: products of e4m3 values are exact; a sum of 128 of them in fp32, however ordered, is
off by at most 128 * 2^-23 of the sum of magnitudes (2^-23: truncation, not rounding, is allowed
for); its two scales and the sum over the KB blocks add KB + 3 roundings: (131 + KB) * 2^-23 of
sum |a b| in all (call it d). A gate weight adds one. The output rounds once, half a step of its
dtype. gated: |h| moves by at most 1.1 |u| dg + |silu(g)| du (|silu'| < 1.1) and its own fast
exponential and division by 2^-19 of |h|; an e4m3 result is within half a step (2^-4 of the value,
2^-10 scales near zero) of what was rounded.
"""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_routed_04_b200 import binding as b
from oracle import block as o

pytestmark = pytest.mark.gpu

U2 = 2.0 ** -23
DT = {"f32": (b.DT_F32, torch.float32), "bf16": (b.DT_BF16, torch.bfloat16), "f16": (b.DT_F16, torch.float16)}
VARIANTS = {"auto": b.VARIANT_AUTO, "tensor": b.VARIANT_TENSOR, "stream": b.VARIANT_STREAM}


def ws256():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ rounding

@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,K,ld,shift", [(1, 16, 0, 0), (1, 4096, 0, 0), (3, 128, 0, 0), (37, 144, 160, 8), (20, 1040, 1041, 1),
                                          (300, 2048, 0, 0), (5, 1008, 0, 4)])
def test_rows(T, K, ld, shift, dt):
    rng = np.random.default_rng([T, K])
    ld = ld or K
    buf = torch.full((T * ld + shift + 16,), float("nan"), dtype=DT[dt][1], device="cuda")
    x = buf[shift:shift + T * ld].view(T, ld)[:, :K]
    v = rng.normal(0, 1, (T, K)) * np.exp(rng.normal(0, 2, (T, 1)))
    v[:, :16] = 0
    v[T // 2] *= 1e-7 if dt == "f16" else 1e-41  # denormals
    x.copy_(torch.from_numpy(v.astype(np.float32)).to(DT[dt][1]))
    q, s = torch.empty(T, K, dtype=torch.uint8, device="cuda"), torch.empty((K + 127) // 128, T, device="cuda")
    b.quantize_f8(x, q, s, ws256())
    rq, rs = o.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(o.e4m3_values(bits(q)), rq)
    # torch's own rounding of the same quotients
    pad = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(T, -1, 128) / s.t()[:, :, None]
    tq = pad.clamp(-448, 448).view(T, -1)[:, :K].to(torch.float8_e4m3fn)
    assert torch.equal(tq.view(torch.uint8), q)


def test_rows_every_quotient():
    """All bf16 mantissas against scales of several sizes: the three-instruction quotient is the division's."""
    rng = np.random.default_rng(5)
    R = 4096
    x = (rng.normal(0, 1, (R, 128)) * np.exp2(rng.integers(-100, 100, (R, 1)))).astype(np.float32)
    x[:, 1:] *= np.exp2(-rng.integers(0, 14, (R, 127))).astype(np.float32)
    xd = torch.from_numpy(x).cuda()
    q, s = torch.empty(R, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, R, device="cuda")
    b.quantize_f8(xd, q, s, ws256())
    rq, rs = o.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(o.e4m3_values(bits(q)), rq)


def test_rows_gathered_with_a_row_count():
    T, K, R = 50, 384, 200
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(0, 1, (T, K)).astype(np.float32)).cuda().bfloat16()
    idx = rng.integers(0, T, R).astype(np.int32)
    idx[7], idx[9] = -1, T  # reported, their rows left alone
    q, s = torch.full((R, K), 77, dtype=torch.uint8, device="cuda"), torch.full((3, R), -5.0, device="cuda")
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    ws = ws256()
    b.quantize_f8(x, q, s, ws, row_index=torch.from_numpy(idx).cuda(), n_rows=n)
    assert b.get_error(ws) == b.DEVERR_BOUNDS
    rq, rs = o.quantize_rows(x.float().cpu().numpy()[np.clip(idx, 0, T - 1)])
    keep = np.ones(R, bool)
    keep[[7, 9]] = False
    keep[150:] = False
    assert np.array_equal(o.e4m3_values(bits(q))[keep], rq[keep]) and np.array_equal(s.cpu().numpy()[:, keep], rs[:, keep])
    assert (bits(q)[~keep] == 77).all() and (s.cpu().numpy()[:, ~keep] == -5).all()


@pytest.mark.parametrize("R,K,n,bad", [(19001, 144, 19001, []), (19000, 4240, 18997, []), (18950, 1040, 18950, [0, 9, 18949]),
                                       (20000, 128, 3, [])])
def test_many_rows(R, K, n, bad):
    """Enough rows for a warp to take eight of them; a last group of fewer, left rows, bad indices."""
    rng = np.random.default_rng([R, K])
    x = torch.from_numpy(rng.normal(0, 1, (61, K)).astype(np.float32)).cuda().bfloat16()
    idx = rng.integers(0, 61, R).astype(np.int32)
    for i in bad:
        idx[i] = 61
    q, s = torch.full((R, K), 77, dtype=torch.uint8, device="cuda"), torch.full(((K + 127) // 128, R), -5.0, device="cuda")
    ws = ws256()
    b.quantize_f8(x, q, s, ws, row_index=torch.from_numpy(idx).cuda(), n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert b.get_error(ws) == (b.DEVERR_BOUNDS if bad else 0)
    one, so = torch.empty(61, K, dtype=torch.uint8, device="cuda"), torch.empty((K + 127) // 128, 61, device="cuda")
    b.quantize_f8(x, one, so, ws256())
    rq, rs = o.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(so.cpu().numpy(), rs) and np.array_equal(o.e4m3_values(bits(one)), rq)
    keep = np.ones(R, bool)
    keep[n:] = False
    keep[bad] = False
    want_q, want_s = bits(one)[np.minimum(idx, 60)], so.cpu().numpy()[:, np.minimum(idx, 60)]
    want_q[~keep], want_s[:, ~keep] = 77, -5
    assert np.array_equal(bits(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_infinities_and_nan_make_their_block_nan():
    x = torch.randn(3, 256, device="cuda")
    x[0, 3], x[1, 200] = float("inf"), float("nan")
    q, s = torch.empty(3, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 3, device="cuda")
    b.quantize_f8(x, q, s, ws256())
    v = o.dequantize_rows(o.e4m3_values(bits(q)), s.cpu().numpy())
    bad = np.zeros((3, 256), bool)
    bad[0, :128] = bad[1, 128:] = True
    assert np.isnan(v[bad]).all() and np.isfinite(v[~bad]).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("E,N,K,shift", [(1, 8, 16, 0), (2, 128, 128, 0), (3, 200, 144, 0), (1, 264, 400, 1), (2, 1000, 272, 0)])
def test_weights(E, N, K, shift, turned, dt):
    rng = np.random.default_rng([E, N, K])
    w = rng.normal(0, 0.02, (E, N, K)).astype(np.float32)
    w[0, :8, :16] *= 50
    src = torch.from_numpy(np.ascontiguousarray(w.transpose(0, 2, 1)) if turned else w)
    buf = torch.zeros(E * N * K + 16, dtype=DT[dt][1], device="cuda")
    wd = buf[shift:shift + E * N * K].view(src.shape)
    wd.copy_(src)
    q, s = torch.empty(E, N, K, dtype=torch.uint8, device="cuda"), torch.empty(E, (N + 127) // 128, (K + 127) // 128, device="cuda")
    b.quantize_f8_weights(wd, q, s, transposed=turned)
    given = wd.float().cpu().numpy()
    given = given.transpose(0, 2, 1) if turned else given
    for e in range(E):
        rq, rs = o.quantize_weights(given[e])
        assert np.array_equal(s[e].cpu().numpy(), rs) and np.array_equal(o.e4m3_values(bits(q[e])), rq)


# ------------------------------------------------------------------ products

def rows8(rng, R, K):
    x = (rng.normal(0, 1, (R, K)) * np.exp(rng.normal(0, 1, (R, 1)))).astype(np.float32)
    q, s = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty((K + 127) // 128, R, device="cuda")
    b.quantize_f8(torch.from_numpy(x).cuda(), q, s, ws256())
    return q, s


def weights8(rng, E, N, K, std=0.05):
    w = torch.from_numpy((rng.normal(0, std, (E, N, K)) * np.exp(rng.normal(0, 0.5, (E, N, 1)))).astype(np.float32)).cuda()
    q, s = torch.empty(E, N, K, dtype=torch.uint8, device="cuda"), torch.empty(E, (N + 127) // 128, (K + 127) // 128, device="cuda")
    b.quantize_f8_weights(w, q, s)
    return q, s


def values(q, s):
    q = o.e4m3_values(bits(q))
    return o.dequantize_rows(q, s.cpu().numpy())


def weight_values(q, s):
    qs, ss = bits(q), s.cpu().numpy()
    return [o.dequantize_weights(o.e4m3_values(qs[e]), ss[e]) for e in range(qs.shape[0])]


def split(rng, R, E, tail=0):
    """Offsets of R - tail rows over E experts, several of them empty."""
    cut = np.sort(rng.integers(0, R - tail + 1, E - 1)) if E > 1 else np.array([], int)
    cut[:E // 4] = 0
    return np.concatenate([[0], cut, [R - tail]]).astype(np.int32)


# R, K, N, E, rows behind the last expert's
SHAPES = [(1, 16, 8, 1, 0), (1, 4096, 1536, 1, 0), (2, 128, 128, 1, 0), (7, 272, 200, 1, 0), (8, 1040, 264, 1, 0), (9, 512, 16, 1, 0),
          (130, 384, 392, 1, 0), (257, 1040, 520, 1, 0), (600, 2048, 768, 1, 0), (8, 256, 256, 256, 0), (40, 144, 328, 6, 3),
          (333, 1040, 1000, 6, 0), (700, 320, 192, 9, 50), (1000, 768, 256, 128, 11), (130, 128, 64, 3, 130)]


def check_matmul(R, K, N, E, tail, out, variant, weighted):
    rng = np.random.default_rng([R, K, N, E])
    a, sa = rows8(rng, R, K)
    w, sw = weights8(rng, E, N, K)
    off = split(rng, R, E, tail)
    use = R - tail
    code, dt = DT[out]
    p = b.f8_params(R, K, N, E, out_dtype=code, variant=VARIANTS[variant])
    c = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    sp = tw = None
    wr = np.ones(R)
    if weighted:
        sp = rng.permutation(R).astype(np.int32)
        sp[::5] = -1
        tw = rng.random(R).astype(np.float32)
        wr = np.where(sp >= 0, tw[np.maximum(sp, 0)], 1.0).astype(np.float64)
        sp, tw = torch.from_numpy(sp).cuda(), torch.from_numpy(tw).cuda()
    ws = b.f8_workspace(p)
    offs = None if E == 1 and tail == 0 else torch.from_numpy(off).cuda()
    b.matmul_f8(p, a, sa, w, sw, c, ws, offsets=offs, sorted_pair=sp, topk_w=tw)
    assert b.get_error(ws) == 0
    got = c.double().cpu().numpy()
    assert (got[use:] == 7.0).all(), "rows behind the last expert's were written"
    if use == 0:
        return
    A, W = values(a, sa), weight_values(w, sw)
    ref = o.matmul(A, off, lambda e: W[e])[:use] * wr[:use, None]
    mag = o.matmul(np.abs(A), off, lambda e: np.abs(W[e]))[:use] * wr[:use, None]
    tol = (132 + (K + 127) // 128) * U2 * mag + torch.finfo(dt).eps / 2 * np.abs(ref) + (2.0 ** -25 if out == "f16" else 0)
    err = np.abs(got[:use] - ref) - tol
    assert (err <= 0).all(), f"{int((err > 0).sum())} of {err.size} off, worst by {err.max():.3e}"


@pytest.mark.parametrize("variant", list(VARIANTS))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_matmul(shape, variant):
    check_matmul(*shape, "f32", variant, False)


# Dense products of more tiles than SMs: several tiles a block, the last ones nearly empty, ragged, full.
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1300, 1040, 4104, 1, 0), (1537, 272, 3592, 1, 0), (5001, 128, 2048, 1, 0)], ids=str)
def test_matmul_many_tiles(shape, out):
    check_matmul(*shape, out, "tensor", out == "bf16")


@pytest.mark.parametrize("variant", ["tensor", "stream"])
@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(5, 272, 200, 1, 0), (333, 272, 1000, 6, 9), (260, 768, 64, 1, 0)], ids=str)
def test_matmul_weighted_16_bits(shape, out, variant):
    check_matmul(*shape, out, variant, True)


@pytest.mark.parametrize("variant", list(VARIANTS))
@pytest.mark.parametrize("out", ["e4m3", "f32", "bf16"])
@pytest.mark.parametrize("limit", [0.0, 2.0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated(shape, limit, out, variant):
    if out == "e4m3" and shape[2] % 16:
        pytest.skip("rows in 8 bits are multiples of 16")
    if out == "bf16" and limit:
        pytest.skip("covered by the others")
    check_gated(shape, limit, out, variant)


@pytest.mark.parametrize("out", ["e4m3", "f32", "bf16"])
@pytest.mark.parametrize("shape", [(1300, 1040, 1872, 1, 0), (2047, 256, 1296, 1, 0)], ids=str)
def test_gated_many_tiles(shape, out):
    check_gated(shape, 2.0, out, "tensor")


def check_gated(shape, limit, out, variant):
    R, K, N, E, tail = shape
    rng = np.random.default_rng([R, K, N, E, 5])
    a, sa = rows8(rng, R, K)
    wg, sg = weights8(rng, E, N, K)
    wu, su = weights8(rng, E, N, K)
    off = split(rng, R, E, tail)
    use = R - tail
    p = b.f8_params(R, K, N, E, out_dtype=b.DT_E4M3 if out == "e4m3" else DT[out][0], swiglu_limit=limit,
                    variant=VARIANTS[variant])
    ws = b.f8_workspace(p)
    offs = None if E == 1 and tail == 0 else torch.from_numpy(off).cuda()
    if out == "e4m3":
        h, hs = torch.full((R, N), 77, dtype=torch.uint8, device="cuda"), torch.full(((N + 127) // 128, R), -5.0, device="cuda")
    else:
        h, hs = torch.full((R, N), 7.0, dtype=DT[out][1], device="cuda"), None
    b.gated_f8(p, a, sa, wg, sg, wu, su, h, ws, h_scale=hs, offsets=offs)
    assert b.get_error(ws) == 0
    if out == "e4m3":
        assert (bits(h)[use:] == 77).all() and (hs.cpu().numpy()[:, use:] == -5).all()
    else:
        assert bool((h[use:] == 7.0).all())
    if use == 0:
        return
    A, G, V = values(a, sa), weight_values(wg, sg), weight_values(wu, su)
    g, u = (o.matmul(A, off, lambda e: w[e])[:use] for w in (G, V))
    dg, du = ((132 + (K + 127) // 128) * U2 * o.matmul(np.abs(A), off, lambda e: np.abs(w[e]))[:use] for w in (G, V))
    ref = o.gated(g, u, limit)
    lim = limit if limit > 0 else np.inf
    uc, gc = np.clip(u, -lim, lim), np.clip(g, -lim, lim)
    tol = 1.1 * np.abs(uc) * dg + np.abs(o.gated(gc, 1.0, 0.0)) * du + 1.1 * dg * du + 2.0 ** -19 * np.abs(ref)
    if out == "e4m3":
        s = np.repeat(hs.cpu().numpy().astype(np.float64), 128, 0)[:N].T[:use]
        got = o.e4m3_values(bits(h)[:use]) * s
        amax = np.stack([np.abs(ref[:, j:j + 128]).max(1) for j in range(0, N, 128)])
        tmax = np.stack([tol[:, j:j + 128].max(1) for j in range(0, N, 128)])
        assert (np.abs(hs.cpu().numpy()[:, :use] * 448.0 - amax) <= tmax + 2 * U2 * amax + 2.0 ** -117).all()
        tol = tol + 2.0 ** -4 * (np.abs(ref) + tol) + 2.0 ** -10 * s
    else:
        got = h[:use].double().cpu().numpy()
        tol = tol + torch.finfo(DT[out][1]).eps / 2 * np.abs(ref)
    err = np.abs(got - ref) - tol
    assert (err <= 0).all(), f"{int((err > 0).sum())} of {err.size} off, worst by {err.max():.3e}"


@pytest.mark.parametrize("variant", ["tensor", "stream"])
def test_nan_stays_in_its_row(variant):
    """A row whose block reads back as NaN gives a NaN row; the others are untouched. Gated too."""
    R, K, N = 20, 256, 256
    rng = np.random.default_rng(3)
    a, sa = rows8(rng, R, K)
    w, sw = weights8(rng, 1, N, K)
    sa[1, 11] = float("nan")
    p = b.f8_params(R, K, N, out_dtype=b.DT_F32, swiglu_limit=7.0, variant=VARIANTS[variant])
    c, h = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    b.matmul_f8(p, a, sa, w, sw, c, b.f8_workspace(p))
    b.gated_f8(p, a, sa, w, sw, w, sw, h, b.f8_workspace(p))
    for t in (c, h):
        n = torch.isnan(t).all(1).cpu().numpy()
        assert n[11] and n.sum() == 1 and bool(torch.isfinite(t[torch.arange(R) != 11]).all())


@pytest.mark.parametrize("variant", ["tensor", "stream"])
def test_fp16_range_is_flagged(variant):
    R, K, N = 12, 128, 64
    a, w = torch.full((R, K), 0x7E, dtype=torch.uint8, device="cuda"), torch.full((1, N, K), 0x7E, dtype=torch.uint8, device="cuda")
    sa, sw = torch.ones(1, R, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    p = b.f8_params(R, K, N, out_dtype=b.DT_F16, variant=VARIANTS[variant])
    c, ws = torch.empty(R, N, dtype=torch.float16, device="cuda"), b.f8_workspace(p)
    b.matmul_f8(p, a, sa, w, sw, c, ws)
    assert b.get_error(ws) == b.DEVERR_RANGE


@pytest.mark.parametrize("variant", ["tensor", "stream"])
def test_bad_offsets_are_reported_and_not_followed(variant):
    R, K, N, E = 64, 128, 64, 4
    rng = np.random.default_rng(8)
    a, sa = rows8(rng, R, K)
    w, sw = weights8(rng, E, N, K)
    off = torch.tensor([0, 10, 200, 210, 64], dtype=torch.int32, device="cuda")  # experts 1 and 2 reach past the rows
    p = b.f8_params(R, K, N, E, out_dtype=b.DT_F32, variant=VARIANTS[variant])
    c, ws = torch.full((R, N), 7.0, device="cuda"), b.f8_workspace(p)
    b.matmul_f8(p, a, sa, w, sw, c, ws, offsets=off)
    assert b.get_error(ws) & b.DEVERR_BOUNDS
    assert bool((c[10:] == 7.0).all()) and bool((c[:10] != 7.0).any())


@pytest.mark.parametrize("variant", ["tensor", "stream"])
def test_same_bits_streams_and_graphs(variant):
    R, K, N, E = 300, 640, 384, 7
    rng = np.random.default_rng(11)
    a, sa = rows8(rng, R, K)
    wg, sg = weights8(rng, E, N, K)
    wu, su = weights8(rng, E, N, K)
    wd, sd = weights8(rng, E, 512, N)
    off = torch.from_numpy(split(rng, R, E)).cuda()
    p1 = b.f8_params(R, K, N, E, out_dtype=b.DT_E4M3, swiglu_limit=7.0, variant=VARIANTS[variant])
    p2 = b.f8_params(R, N, 512, E, variant=VARIANTS[variant])

    def bufs():
        return dict(h=torch.zeros(R, N, dtype=torch.uint8, device="cuda"), s=torch.zeros((N + 127) // 128, R, device="cuda"),
                    y=torch.zeros(R, 512, dtype=torch.bfloat16, device="cuda"), ws=b.f8_workspace(p1))

    def step(v):
        b.gated_f8(p1, a, sa, wg, sg, wu, su, v["h"], v["ws"], h_scale=v["s"], offsets=off)
        b.matmul_f8(p2, v["h"], v["s"], wd, sd, v["y"], v["ws"], offsets=off)
    one, two, three = bufs(), bufs(), bufs()
    step(one)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(two)
        step(two)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(three)
    three["y"].zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for n in ("h", "s", "y"):
        assert torch.equal(one[n], two[n]) and torch.equal(one[n], three[n]), n


def test_no_rows():
    p = b.f8_params(0, 128, 64, 3)
    w, sw = torch.zeros(3, 64, 128, dtype=torch.uint8, device="cuda"), torch.ones(3, 1, 1, device="cuda")
    a, sa = torch.zeros(0, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 0, device="cuda")
    b.matmul_f8(p, a, sa, w, sw, torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), b.f8_workspace(p),
                offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


def test_waits_that_run_out_are_reported():
    """With every wait limited to 1 ns the tile kernels give up, report it and leave the context usable."""
    R, K, N = 300, 1024, 512
    rng = np.random.default_rng(2)
    a, sa = rows8(rng, R, K)
    w, sw = weights8(rng, 1, N, K)
    p = b.f8_params(R, K, N, out_dtype=b.DT_F32, variant=b.VARIANT_TENSOR)
    c, ws = torch.zeros(R, N, device="cuda"), b.f8_workspace(p)
    b.set_wait_limit_ns(1)
    try:
        b.matmul_f8(p, a, sa, w, sw, c, ws)
        err = b.get_error(ws)
    finally:
        b.set_wait_limit_ns(0)
    assert err in (0, b.DEVERR_TIMEOUT)
    b.clear_error(ws)
    check_matmul(R, K, N, 1, 0, "f32", "tensor", False)


def test_buffers_elsewhere_are_refused():
    x, q, s = torch.zeros(4, 64, device="cuda"), torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(1, 4, device="cuda")
    with pytest.raises(b.MoeError):
        b.quantize_f8(x, q, s, torch.zeros(256, dtype=torch.uint8))            # the host's memory
    with pytest.raises(b.MoeError):
        b.quantize_f8(x, q, s, torch.zeros(256, device="cuda"))                # not bytes
    with pytest.raises(b.MoeError):
        b.quantize_f8(x, q, s, ws256(), n_rows=torch.empty(0, dtype=torch.int32, device="cuda"))
    p = b.norm_params(4, 64)
    st = torch.empty(4, device="cuda")
    with pytest.raises(b.MoeError):
        b.norm_backward(p, x, x.bfloat16(), st, st, torch.empty_like(x), torch.zeros(1 << 20, dtype=torch.uint8),
                        weight=torch.ones(64, device="cuda"), dw=torch.empty(64, device="cuda"))


@pytest.mark.parametrize("out", ["e4m3", "bf16"])
def test_tiles_with_tiny_wait_limit_report_and_recover(out):
    rng = np.random.default_rng(11)
    R, K, N, E = 700, 1040, 528, 5
    a, sa = rows8(rng, R, K)
    wg, sg = weights8(rng, E, N, K)
    wu, su = weights8(rng, E, N, K)
    off = torch.from_numpy(split(rng, R, E)).cuda()
    p = b.f8_params(R, K, N, E, out_dtype=b.DT_E4M3 if out == "e4m3" else b.DT_BF16, variant=b.VARIANT_TENSOR)
    h = torch.empty(R, N, dtype=torch.uint8 if out == "e4m3" else torch.bfloat16, device="cuda")
    hs = torch.empty((N + 127) // 128, R, device="cuda") if out == "e4m3" else None
    pm = b.f8_params(R, K, N, E, out_dtype=b.DT_F32, variant=b.VARIANT_TENSOR)
    c = torch.empty(R, N, device="cuda")
    ws = b.f8_workspace(p)
    b.set_wait_limit_ns(1)
    try:
        for _ in range(3):
            b.gated_f8(p, a, sa, wg, sg, wu, su, h, ws, h_scale=hs, offsets=off)
            b.matmul_f8(pm, a, sa, wg, sg, c, ws, offsets=off)
        torch.cuda.synchronize()
    finally:
        b.set_wait_limit_ns(0)
    err = b.get_error(ws)
    assert err & ~b.DEVERR_TIMEOUT == 0, f"unexpected error bits {err:#x}"
    check_gated((R, K, N, E, 0), 0.0, out, "tensor")
    check_matmul(R, K, N, E, 0, "f32", "tensor", False)


# One token's rows to e4m3: one strip of columns a block up to ceil(N / 128) * 8 * chunks of 3 blocks an SM, above it
# two; the chunks are the rows by 8, or as many as the rows may make of the experts.
@pytest.mark.parametrize("shape", [(1, 512, 128, 1, 0), (1, 4096, 1536, 1, 0), (8, 1040, 144, 1, 0), (17, 256, 1536, 1, 0),
                                   (8, 2048, 128, 8, 0), (8, 512, 768, 8, 0), (8, 512, 1536, 8, 0), (8, 128, 272, 256, 0),
                                   (70, 384, 1536, 1, 0)], ids=str)
def test_gated_strips(shape):
    check_gated(shape, 7.0, "e4m3", "stream")


@pytest.mark.parametrize("variant", ["tensor", "stream"])
@pytest.mark.parametrize("out", ["f32", "e4m3"])
def test_gated_of_large_projections(variant, out):
    """Without a limit, h = silu(g) u where g u alone would pass fp32's largest value: one row with a single 1, column n's
    g and u are its block's scales. At g = -80 the exponential's argument in powers of two, 116, rounds by 2^-18, which
    moves h by ln 2 of that; three roundings and the reciprocal stay below the rest of 2^-18. e4m3: half a step more."""
    gu = [(-50.0, 1e38), (-1e20, 1e20), (-80.0, -3e37), (30.0, 1e37), (1e-20, 1e38), (-1e38, 1e-38)]
    R, K, N = 3, 16, 128 * len(gu)
    a = torch.zeros(R, K, dtype=torch.uint8, device="cuda")
    a[1, 5] = 0x38  # 1.0
    w = torch.full((1, N, K), 0x38, dtype=torch.uint8, device="cuda")
    sa = torch.ones(1, R, device="cuda")
    sg, su = (torch.tensor([v[i] for v in gu], device="cuda").view(1, -1, 1).contiguous() for i in (0, 1))
    p = b.f8_params(R, K, N, out_dtype=b.DT_E4M3 if out == "e4m3" else b.DT_F32, variant=VARIANTS[variant])
    h = torch.empty(R, N, dtype=torch.uint8 if out == "e4m3" else torch.float32, device="cuda")
    hs = torch.empty(len(gu), R, device="cuda") if out == "e4m3" else None
    b.gated_f8(p, a, sa, w, sg, w, su, h, b.f8_workspace(p), h_scale=hs)
    got = values(h, hs) if out == "e4m3" else h.double().cpu().numpy()
    g, u = (np.repeat(s.double().cpu().numpy().reshape(-1), 128) for s in (sg, su))
    ref = np.zeros((R, N))
    with np.errstate(under="ignore"):
        ref[1] = o.gated(g, u, 0.0)
    assert np.isfinite(got).all()
    tol = (2.0 ** -18 + (2.0 ** -4 if out == "e4m3" else 0.0)) * np.abs(ref) + 2.0 ** -126
    assert (np.abs(got - ref) <= tol).all()


ROWS_MOST = 2 ** 31 - 1
needs_room = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[0] < 120 << 30,
                                reason="2^31 - 1 rows take 90 GB")


def periodic(table, got):
    """Row r of got is table's row r % 5: compared 5 * 2^24 rows at a time."""
    step = 5 << 24
    want = table.repeat(1 << 24, 1)
    for r in range(0, got.shape[0], step):
        part = got[r:r + step]
        if not torch.equal(part, want[:part.shape[0]]):
            return False
    return True


@needs_room
def test_most_rows_rounded():
    x = torch.randn(5, 16, device="cuda").bfloat16()
    q, s = torch.zeros(ROWS_MOST, 16, dtype=torch.uint8, device="cuda"), torch.zeros(1, ROWS_MOST, device="cuda")
    idx = torch.arange(ROWS_MOST, dtype=torch.int32, device="cuda").remainder_(5)
    b.quantize_f8(x, q, s, ws256(), row_index=idx)
    one, so = torch.empty(5, 16, dtype=torch.uint8, device="cuda"), torch.empty(1, 5, device="cuda")
    b.quantize_f8(x, one, so, ws256())
    assert periodic(one, q) and periodic(so.t(), s.t())
    del q, s, idx
    torch.cuda.empty_cache()


@needs_room
@pytest.mark.parametrize("variant", ["tensor", "stream"])
def test_most_rows_multiplied(variant):
    rng = np.random.default_rng(6)
    one, so = rows8(rng, 5, 16)
    w, sw = weights8(rng, 1, 8, 16)
    ref = torch.empty(5, 8, dtype=torch.bfloat16, device="cuda")
    b.matmul_f8(b.f8_params(5, 16, 8, variant=VARIANTS[variant]), one, so, w, sw, ref, ws256())
    a = one.repeat((ROWS_MOST + 4) // 5, 1)[:ROWS_MOST]
    sa = so.repeat(1, (ROWS_MOST + 4) // 5)[:, :ROWS_MOST].contiguous()
    c = torch.zeros(ROWS_MOST, 8, dtype=torch.bfloat16, device="cuda")
    p = b.f8_params(ROWS_MOST, 16, 8, variant=VARIANTS[variant])
    ws = b.f8_workspace(p)
    b.matmul_f8(p, a, sa, w, sw, c, ws, offsets=torch.tensor([0, ROWS_MOST], dtype=torch.int32, device="cuda"))
    assert b.get_error(ws) == 0 and periodic(ref, c)
    del a, sa, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("blocks", [0, 1, 3, 5, 7])
def test_tiles_whose_copies_stop_report_it(blocks, gated):
    """No wait of a product that runs as it should lasts the 64 polls between two looks at the clock (0.3 ms), so that a
    short limit alone makes none run out. Here the copies stop: every CTA's waits run out, and the next calls are right."""
    ws = torch.zeros(b.F8_SELFTEST_BYTES, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b.f8_wait_selftest(gated, blocks, 1_000_000, ws)  # 1 ms
        assert b.get_error(ws) == b.DEVERR_TIMEOUT
        b.clear_error(ws)
        assert b.get_error(ws) == 0
    check_gated((300, 1024, 256, 1, 0), 7.0, "e4m3", "tensor")
    check_matmul(300, 1024, 256, 1, 0, "f32", "tensor", False)

"""GPU tests of the seam between two blocks of linears (poet_block_norm_fwd / _bwd) against the float64 formulas of
tests/token_ref.py, with its bounds: every combination of its parts and types, single tokens, odd dimensions, pitches
and misaligned bases, gates shared by runs of tokens, in-place residuals, streams, graphs and far offsets."""
import numpy as np
import pytest

from tests import token_ref as R
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def B():
    from orthogonal_reparameterized_amd import binding
    return binding


def tdt(dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


def mat(a, dt, pad=0, skew=0):
    """(view, float64 values) of a's values at pitch d + pad, skew elements into a buffer of NaN."""
    a = torch.as_tensor(np.asarray(a), dtype=torch.float32)
    T, d = a.shape
    buf = torch.full((skew + T * (d + pad),), float("nan"), dtype=tdt(dt), device="cuda")
    v = buf.as_strided((T, d), (d + pad, 1), skew)
    v.copy_(a)
    return v, v.double().cpu().numpy()


def out(T, d, dt, pad=0, skew=0):
    buf = torch.full((skew + T * (d + pad),), 9.0, dtype=tdt(dt), device="cuda")
    return buf.as_strided((T, d), (d + pad, 1), skew), buf


def intact(v, buf):
    """Nothing but the view was written."""
    v.fill_(9.0)
    assert (buf == 9.0).all()


def close(got, ref, bound, dt, what):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape, what
    off, b = np.abs(g - ref), bound + R.HALF[dt] * np.abs(ref) * 1.01 + 1e-38
    assert (off <= b).all(), (what, float((off - b).max()), int((off > b).sum()), float(off.max()))


def f32(a):
    t = torch.as_tensor(np.asarray(a), dtype=torch.float32).cuda()
    return t, t.double().cpu().numpy()


def run(T, d, res, act, has_y=True, gate=1, post=True, pre=True, dh_in=True, scale=0.5, pads=(0, 0, 0, 0), skew=0, seed=0,
        eps=1e-6, inplace=False, zero_rows=False):
    announce(f"block norm T={T} d={d} res={res} act={act} y={has_y} gate={gate} post={post} pre={pre} dh={dh_in} pads={pads} skew={skew}")
    rng = np.random.default_rng([T, d, seed])
    ph, py, pg, px = pads
    hv = rng.standard_normal((T, d)) * 2
    yv = rng.standard_normal((T, d)) * 0.7
    if zero_rows:
        hv[0] = 0.0
        yv[0] = 0.0
    h, h64 = mat(hv, res, ph, skew)
    y, y64 = mat(yv, act, py, skew) if has_y else (None, None)
    G, G64 = mat(rng.standard_normal((-(-T // gate), d)), act, pg, skew) if gate and has_y else (None, None)
    wq, wq64 = f32(1 + 0.2 * rng.standard_normal(d)) if post and has_y else (None, None)
    wp, wp64 = f32(1 + 0.2 * rng.standard_normal(d)) if pre else (None, None)
    rstd = torch.full((T, 2), 9.0, device="cuda")
    ho, hob = (h, None) if inplace else out(T, d, res, ph, skew) if has_y else (None, None)
    x, xb = out(T, d, act, px, skew) if pre else (None, None)
    gt = gate or 1
    B().poet_block_norm_fwd(h, rstd, y=y, gate=G, w_post=wq, w_pre=wp, h_out=ho, x=x, res_scale=scale, eps=eps, gate_tokens=gt)
    torch.cuda.synchronize()
    rnd = lambda v: torch.as_tensor(v).to(tdt(res)).double().numpy()  # noqa: E731
    got_h = ho.double().cpu().numpy() if has_y else h64
    eps32 = float(np.float32(eps))
    # x and r_h are of the residual stream as it is kept: the reference takes the kept values
    rh_, eh, rx, ex, ry, rh = R.norm_fwd(h64, y64, G64, wq64, wp64, float(np.float32(scale)), eps32, gt, lambda v: got_h if has_y else rnd(v))
    if has_y:
        close(ho, rh_, eh, res, "h_out")
    S = (3 * R.U + R.U * (np.log2(d) + d / 64 + 8)) / 2 + 4 * R.U
    r = rstd.double().cpu().numpy()
    assert (np.abs(r[:, :1] - ry) <= S * ry).all(), "r_y"
    if pre:
        close(x, rx, ex, act, "x")
        assert (np.abs(r[:, 1:] - rh) <= S * rh).all(), "r_h"
    else:
        assert (r[:, 1] == 0).all()
    # backward
    dx, dx64 = mat(rng.standard_normal((T, d)), act, px, skew) if pre else (None, None)
    dh_in = dh_in or not pre
    dho, dho64 = mat(rng.standard_normal((T, d)) * 0.3, res, ph, skew) if dh_in else (None, None)
    dh, dhb = (dho, None) if inplace and dh_in else out(T, d, res, ph, skew)
    dy, dyb = out(T, d, act, py, skew) if has_y else (None, None)
    dg, dgb = out(-(-T // gt), d, act, pg, skew) if G is not None else (None, None)
    dwq = torch.full((d,), 9.0, device="cuda") if wq is not None else None
    dwp = torch.full((d,), 9.0, device="cuda") if pre else None
    # without post norm and gate the backward does not need y
    yb = y if G is not None or wq is not None else None
    hb = (ho if has_y else h) if pre else None

    def bwd():
        B().poet_block_norm_bwd(hb, rstd, y=yb, gate=G, w_post=wq, w_pre=wp, dh_out=dho, dx=dx, dh=dh, dy=dy, dgate=dg,
                                dw_post=dwq, dw_pre=dwp, res_scale=scale if has_y else 1.0, gate_tokens=gt)
        torch.cuda.synchronize()
    bwd()
    first = [None if t is None else t.clone() for t in (dh, dy, dg, dwq, dwp)]
    if not (inplace and dh_in):
        bwd()
        assert all(a is None or torch.equal(a, b) for a, b in zip(first, (dh, dy, dg, dwq, dwp)))
    ref = R.norm_bwd(got_h if pre else None, y64, G64, wq64, wp64, ry, rh, dho64, dx64, float(np.float32(scale)) if has_y else 1.0,
                     gt, min(T, 512) + 64) if has_y else R.norm_bwd(h64, np.zeros((T, d)), None, None, wp64, ry, rh, dho64, dx64, 1.0, 1, min(T, 512) + 64)
    S2 = 2 * S  # the kept r_y and r_h differ from the reference's by S: every term holds at most two of them
    for name, t, dt in (("dh", dh, res), ("dy", dy, act), ("dgate", dg, act), ("dw_post", dwq, "f32"), ("dw_pre", dwp, "f32")):
        if t is not None:
            v, e = ref[name]
            mag = {"dh": np.abs(v), "dy": np.abs(v)}.get(name, np.abs(v))
            extra = S2 * (mag + e / (4 * R.U))  # e / 4u bounds the sum of the terms' magnitudes
            close(t, v, e + extra, dt, name)
    for v, b in ((ho, hob), (x, xb), (dh, dhb), (dy, dyb), (dg, dgb)):
        if b is not None:
            intact(v, b)


DIMS = [1, 2, 7, 63, 64, 65, 100, 511, 512, 513, 1000, 1377, 2048, 2560, 4095, 5461, 6848, 8192, 8200, 16384]


@pytest.mark.parametrize("res,act", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("d", DIMS)
def test_dimensions(d, res, act):
    pads, skew = [((0, 0, 0, 0), 0), ((8, 16, 8, 24), 0), ((1, 3, 0, 5), 1), ((0, 8, 1, 0), 8)][d % 4]
    run(5, d, res, act, pads=pads, skew=skew, seed=1)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("has_y,gate,post,pre,dh_in", [
    (True, 1, True, True, True), (True, 1, True, True, False), (True, 1, True, False, True), (True, 1, False, True, True),
    (True, 0, True, True, True), (True, 0, False, True, True), (True, 0, False, True, False), (True, 0, False, False, True),
    (True, 1, False, False, True), (True, 0, True, False, True), (False, 0, False, True, True), (False, 0, False, True, False)])
@pytest.mark.parametrize("T,d", [(1, 200), (13, 1024), (67, 2049)])
def test_parts(T, d, has_y, gate, post, pre, dh_in, act):
    run(T, d, "f32", act, has_y, gate, post, pre, dh_in, seed=2)
    run(T, d, "bf16", act, has_y, gate, post, pre, dh_in, seed=3)


@pytest.mark.parametrize("T,gate", [(1, 5), (7, 7), (100, 3), (100, 33), (101, 100), (700, 2), (700, 699), (2500, 1000),
                                    (3000, 7), (3001, 3001), (3001, 5000)])
@pytest.mark.parametrize("d", [96, 515])
def test_gate_runs(T, gate, d):
    run(T, d, "f32", "bf16", gate=gate, seed=4)
    run(T, d, "f32", "f32", gate=gate, post=False, seed=5)


@pytest.mark.parametrize("res,act", [("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,d", [(1, 2048), (300, 513), (2049, 256)])
def test_in_place_residual(T, d, res, act):
    run(T, d, res, act, seed=6, inplace=True)


def test_rows_of_zeros_and_scales():
    run(9, 300, "f32", "f32", seed=7, zero_rows=True, eps=1e-6)
    run(9, 300, "bf16", "bf16", seed=8, zero_rows=True, eps=1e-3)
    run(9, 300, "f32", "f32", seed=9, scale=0.0)
    run(9, 300, "f32", "f32", seed=10, scale=-1.5)


@pytest.mark.parametrize("T,d", [(1024, 2048), (4100, 640)])
def test_many_tokens(T, d):
    run(T, d, "bf16", "bf16", gate=1, seed=11)
    run(T, d, "f32", "bf16", gate=512, seed=12)


def test_gradients_against_differences():
    """The backward against central differences of the float64 formula of the forward along random directions."""
    T, d, gt, a, eps, e = 6, 37, 2, 0.7, 1e-3, 1e-5
    announce("block norm gradients against differences")
    rng = np.random.default_rng(0)
    (h, h64), (y, y64) = mat(rng.standard_normal((T, d)), "f32"), mat(rng.standard_normal((T, d)), "f32")
    G, G64 = mat(rng.standard_normal((3, d)), "f32")
    (wq, wq64), (wp, wp64) = f32(1 + 0.2 * rng.standard_normal(d)), f32(1 + 0.2 * rng.standard_normal(d))
    (gh, gh64), (gx, gx64) = mat(rng.standard_normal((T, d)), "f32"), mat(rng.standard_normal((T, d)), "f32")
    new = lambda like: torch.empty_like(like)  # noqa: E731
    rstd, ho, x = torch.empty((T, 2), device="cuda"), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    B().poet_block_norm_fwd(h, rstd, y=y, gate=G, w_post=wq, w_pre=wp, h_out=ho, x=x, res_scale=a, eps=eps, gate_tokens=gt)
    g = dict(dh=new(gh), dy=new(gh), dgate=torch.empty((3, d), device="cuda"), dw_post=new(wq), dw_pre=new(wp))
    B().poet_block_norm_bwd(ho, rstd, y=y, gate=G, w_post=wq, w_pre=wp, dh_out=gh, dx=gx, res_scale=a, gate_tokens=gt, **g)
    torch.cuda.synchronize()

    def value(h, y, G, wq, wp):
        o, _, xx, _, _, _ = R.norm_fwd(h, y, G, wq, wp, float(np.float32(a)), float(np.float32(eps)), gt, lambda v: v)
        return (o * gh64).sum() + (xx * gx64).sum()
    at = [h64, y64, G64, wq64, wp64]
    for i, name in enumerate(("dh", "dy", "dgate", "dw_post", "dw_pre")):
        gr = g[name].double().cpu().numpy()
        for r in range(2):
            u = np.random.default_rng([i, r]).standard_normal(at[i].shape)
            up, dn = list(at), list(at)
            up[i], dn[i] = at[i] + e * u, at[i] - e * u
            diff = (value(*up) - value(*dn)) / (2 * e)
            assert abs((gr * u).sum() - diff) <= 2e-5 * (np.abs(gr * u).sum() + 1.0), name


def test_offsets_past_32_bits():
    T, d, ld = 3, 700, 1_200_000_008
    announce("block norm offsets past 32 bits")
    buf = torch.empty((T - 1) * ld + d, dtype=torch.bfloat16, device="cuda")
    y = buf.as_strided((T, d), (ld, 1), 0)
    v = np.random.default_rng(1).standard_normal((T, d))
    y.copy_(torch.as_tensor(v))
    y64 = y.double().cpu().numpy()
    h, h64 = mat(v[::-1].copy(), "f32")
    ho, x, rstd = torch.empty((T, d), device="cuda"), torch.empty((T, d), dtype=torch.bfloat16, device="cuda"), torch.empty((T, 2), device="cuda")
    wp, wp64 = f32(np.ones(d))
    B().poet_block_norm_fwd(h, rstd, y=y, w_pre=wp, h_out=ho, x=x)
    torch.cuda.synchronize()
    ref, eh, rx, ex, _, _ = R.norm_fwd(h64, y64, None, None, wp64, 1.0, 1e-6, 1, lambda q: ho.double().cpu().numpy())
    close(ho, ref, eh, "f32", "h_out")
    close(x, rx, ex, "bf16", "x")
    dy = y  # the gradient of y, far apart as well
    dx = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    dh, dwp = torch.empty((T, d), device="cuda"), torch.empty(d, device="cuda")
    B().poet_block_norm_bwd(ho, rstd, w_pre=wp, dx=dx, dh=dh, dy=dy, dw_pre=dwp)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(dy.float().cpu().numpy(), dh.to(torch.bfloat16).float().cpu().numpy())


def test_empty_batch():
    z = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    B().poet_block_norm_fwd(z(0, 8), z(0, 2), y=z(0, 8), gate=z(0, 8), w_post=z(8), w_pre=z(8), h_out=z(0, 8), x=z(0, 8))
    dwq, dwp = torch.full((8,), 9.0, device="cuda"), torch.full((8,), 9.0, device="cuda")
    B().poet_block_norm_bwd(z(0, 8), z(0, 2), y=z(0, 8), w_post=z(8), w_pre=z(8), dx=z(0, 8), dh=z(0, 8), dy=z(0, 8),
                            dw_post=dwq, dw_pre=dwp)
    torch.cuda.synchronize()
    assert (dwq == 0).all() and (dwp == 0).all()


def test_interleaved_gradients():
    """y and its gate as the two halves of one linear's output, and their gradients alike."""
    T, d = 11, 264
    announce("block norm interleaved halves")
    both = torch.randn((T, 2 * d), device="cuda")
    h, wp, wq = torch.randn((T, d), device="cuda"), torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
    dx, dho = torch.randn((T, d), device="cuda"), torch.randn((T, d), device="cuda")
    res = []
    for joined in (True, False):
        y, G = both[:, :d], both[:, d:]
        db = torch.empty((T, 2 * d), device="cuda")
        dy, dg = db[:, :d], db[:, d:]
        if not joined:
            y, G, dy, dg = y.contiguous(), G.contiguous(), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
        rstd, ho, x = torch.empty((T, 2), device="cuda"), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
        dh, a, b = torch.empty((T, d), device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        B().poet_block_norm_fwd(h, rstd, y=y, gate=G, w_post=wq, w_pre=wp, h_out=ho, x=x)
        B().poet_block_norm_bwd(ho, rstd, y=y, gate=G, w_post=wq, w_pre=wp, dh_out=dho, dx=dx, dh=dh, dy=dy, dgate=dg,
                                dw_post=a, dw_pre=b)
        res.append([t.clone() for t in (ho, x, dh, dy, dg, a, b)])
    assert all(torch.equal(p, q) for p, q in zip(*res))


@pytest.mark.parametrize("T,d", [(1, 512), (1500, 320)])
def test_two_streams_and_graph_replay(T, d):
    announce(f"block norm streams and graph T={T} d={d}")
    r = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    h, y, G = r(T, d), r(T, d).to(bf), r(-(-T // 100), d).to(bf)
    wq, wp, dho, dx = r(d), r(d), r(T, d), r(T, d).to(bf)
    need = max(1, B().poet_block_norm_workspace_bytes(T, d, 100))

    def outs():
        e = torch.empty_like
        return dict(rstd=r(T, 2), h_out=e(h), x=e(y), dh=e(h), dy=e(y), dgate=e(G), dw_post=e(wq), dw_pre=e(wp),
                    ws=torch.empty(need, dtype=torch.uint8, device="cuda"))

    def call(o, stream=None):
        B().poet_block_norm_fwd(h, o["rstd"], y=y, gate=G, w_post=wq, w_pre=wp, h_out=o["h_out"], x=o["x"], gate_tokens=100,
                                stream=stream)
        B().poet_block_norm_bwd(o["h_out"], o["rstd"], y=y, gate=G, w_post=wq, w_pre=wp, dh_out=dho, dx=dx, gate_tokens=100,
                                stream=stream, **{k: o[k] for k in ("dh", "dy", "dgate", "dw_post", "dw_pre", "ws")})
    names = ("rstd", "h_out", "x", "dh", "dy", "dgate", "dw_post", "dw_pre")
    ref = outs()
    call(ref)
    want = [ref[k].clone() for k in names]
    streams, bufs = [torch.cuda.Stream(), torch.cuda.Stream()], [outs(), outs()]
    torch.cuda.synchronize()
    for s, b in zip(streams, bufs):
        call(b, s)
    torch.cuda.synchronize()
    for b in bufs:
        assert all(torch.equal(w, b[k]) for w, k in zip(want, names))
    b = outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(b)
    for _ in range(3):
        for k in names:
            b[k].fill_(3)
        call(ref)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w, b[k]) for w, k in zip(want, names))

"""GPU tests of the operators on rows of logits (poet_token_logprobs, poet_distill and their backwards) against the
float64 formulas of tests/token_ref.py, with its bounds: odd and ragged sizes, pitches and misaligned bases, masked
vocabularies and empty rows, NaN and infinities, ties, absent and repeated entries, in-place gradients, other streams,
graph replays and offsets past 32 bits."""
import numpy as np
import pytest

from tests import token_ref as R
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def B():
    from orthogonal_reparameterized_amd import binding
    return binding


def tdt(dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


def rows(a, dt, pad=0, skew=0, fill=None):
    """A GPU tensor of a's values at pitch V + pad whose base is skew elements into its buffer; (view, float64 values).
    The buffer around the view holds `fill` (a NaN by default: a read of it would show)."""
    a = torch.as_tensor(np.asarray(a), dtype=torch.float32)
    T, V = a.shape
    buf = torch.full((skew + T * (V + pad),), float("nan") if fill is None else fill, dtype=tdt(dt), device="cuda")
    v = buf.as_strided((T, V), (V + pad, 1), skew)
    v.copy_(a)
    return v, v.double().cpu().numpy(), buf


def f32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.float32).cuda()


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def close(got, ref, bound, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    ref, bound = np.broadcast_arrays(ref, bound)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fin = np.isfinite(ref)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    inf = ~fin & ~np.isnan(ref)
    np.testing.assert_array_equal(got[inf], ref[inf], err_msg=what)
    off = np.abs(got[fin] - ref[fin])
    bad = off > bound[fin]
    assert not bad.any(), (what, int(bad.sum()), float(off[bad].max()), float(bound[fin][bad][off[bad].argmax()]))


def gauss(T, V, seed, scale=3.0):
    return np.random.default_rng([T, V, seed]).standard_normal((T, V)) * scale


def check_logprobs(zt, z, ids, s=1.0, K=0, gl=None, gh=None, entropy=True, dt="f32", dz=None, ws=None):
    """One forward (with the gradient when gl or gh is given) against the reference; then the backward by itself."""
    T, V = z.shape
    logp, H = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda") if entropy else None
    stats = torch.full((T, 4), 7.0, device="cuda")
    ti = torch.full((T, K), -5, dtype=torch.int32, device="cuda") if K else None
    tl = torch.full((T, K), 7.0, device="cuda") if K else None
    grads = {}
    if gl is not None or gh is not None:
        dz = torch.full((T, V), 7.0, dtype=zt.dtype, device="cuda") if dz is None else dz
        grads = dict(dlogp=None if gl is None else f32(gl), dentropy=None if gh is None else f32(gh))
    B().poet_token_logprobs(zt, i32(ids), logp, stats, inv_temp=s, entropy=H, top_ids=ti, top_logp=tl, ws=ws,
                            dlogits=dz if grads else None, **grads)
    torch.cuda.synchronize()
    lp, p, ref_h = R.logprobs(z, s)
    has = (ids >= 0) & (ids < V)
    ref = np.where(has, lp[np.arange(T), np.where(has, ids, 0)], 0.0)
    bound = lambda r: R.DZ + 4 * R.U * np.abs(np.where(np.isfinite(r), r, 0))  # noqa: E731
    close(logp, ref, bound(ref), "logp")
    if entropy:
        close(H, ref_h, R.entropy_bound(z, s), "entropy")
    if K:
        at = R.top(z, K)
        np.testing.assert_array_equal(ti.cpu().numpy(), at)
        r = np.take_along_axis(lp, at, 1)
        close(tl, r, bound(r), "top_logp")
    if grads:
        ref, err = R.logprobs_grad(z, s, ids, gl, gh)
        err = err + R.HALF[dt] * np.abs(ref) * 1.01 + 1e-38
        close(dz, ref, err, "dlogits")
        again = torch.full((T, V), 3.0, dtype=zt.dtype, device="cuda")
        if dz.data_ptr() != zt.data_ptr():
            B().poet_token_logprobs_bwd(zt, i32(ids), stats, grads["dlogp"], again, inv_temp=s, dentropy=grads["dentropy"])
            torch.cuda.synchronize()
            close(again, ref, err, "dlogits of the backward")
    return stats, dz


SIZES = [(1, 1), (1, 2), (3, 7), (2, 63), (5, 64), (4, 65), (3, 127), (2, 1000), (3, 2047), (2, 2049), (1, 4099),
         (2, 8192), (2, 16411), (2, 32000), (3, 33333), (2, 50001), (1, 65537), (1, 131071), (2, 131073), (1, 262147)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_logprobs_sizes(T, V, dt):
    pad, skew = [(0, 0), (1, 0), (3, 1), (0, 5)][V % 4]
    announce(f"logprobs T={T} V={V} {dt} pad={pad} skew={skew}")
    zt, z, buf = rows(gauss(T, V, 1), dt, pad, skew)
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, T)
    check_logprobs(zt, z, ids, K=min(V, 20), dt=dt)
    check_logprobs(zt, z, ids, s=0.7, K=min(V, 128), gl=rng.standard_normal(T), gh=rng.standard_normal(T), dt=dt)
    check_logprobs(zt, z, ids, s=2.5, gl=rng.standard_normal(T), entropy=False, dt=dt)
    check_logprobs(zt, z, ids, gh=rng.standard_normal(T), dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(9, 1001), (300, 4097), (1030, 515)])
def test_logprobs_many_rows_masks_and_missing_tokens(T, V, dt):
    announce(f"logprobs masked T={T} V={V} {dt}")
    rng = np.random.default_rng(T)
    z = gauss(T, V, 2)
    z[:, rng.random(V) < 0.7] = -INF
    z[T // 2] = -INF                                    # a row whose mask leaves nothing
    z[T // 3, 1:] = -INF                                # a row that it leaves one token
    z[T // 4] = np.where(rng.random(V) < 0.9, -3.3e38, z[T // 4])  # masked by a lowest value instead
    z[T - 1] = -3.3e38                                  # ... everywhere: all tokens alike
    zt, z, _ = rows(z, dt, 3)
    ids = rng.integers(-1, V + 1, T)
    ids[0], ids[1] = -100, V
    check_logprobs(zt, z, ids, K=30, gl=rng.standard_normal(T), gh=rng.standard_normal(T), dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logprobs_nan_and_infinity(dt):
    announce(f"logprobs nan {dt}")
    z = gauss(6, 777, 3)
    z[0, 5] = np.nan
    z[1, 700] = INF
    z[2, :] = -INF
    z[2, 9] = np.nan
    z[3, 20] = z[3, 600] = INF
    z[4, 13] = -INF
    zt, z, _ = rows(z, dt)
    T, V = z.shape
    logp, H, stats = (torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros((T, 4), device="cuda"))
    ti, tl = torch.zeros((T, 9), dtype=torch.int32, device="cuda"), torch.zeros((T, 9), device="cuda")
    dz = torch.zeros((T, V), dtype=zt.dtype, device="cuda")
    B().poet_token_logprobs(zt, i32([3, 4, 5, 6, 7, 8]), logp, stats, entropy=H, top_ids=ti, top_logp=tl,
                            dlogp=f32(np.ones(T)), dlogits=dz)
    torch.cuda.synchronize()
    for t in range(4):
        assert np.isnan(float(logp[t])) and np.isnan(float(H[t])) and tl[t].isnan().all() and dz[t].isnan().all()
    for t in (4, 5):
        assert np.isfinite(float(logp[t])) and np.isfinite(float(H[t])) and dz[t].isfinite().all()
    np.testing.assert_array_equal(ti.cpu().numpy(), R.top(z, 9))
    # no upstream gradient: zeros, whatever the row holds
    B().poet_token_logprobs_bwd(zt, i32([-1] * T), stats, f32(np.ones(T)), dz)
    assert (dz == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "up", "down", "period", "zeros", "few", "blocks"])
@pytest.mark.parametrize("V", [1, 100, 2048, 5000, 40961, 140001])
def test_top_order_of_ties_and_runs(V, kind, dt):
    """Rows whose best tokens are many equal ones, sit side by side or at one distance from each other."""
    K = min(V, 33)
    announce(f"top {kind} V={V} {dt}")
    j = np.arange(V)
    z = {"equal": np.full(V, 1.25), "up": np.minimum(j, 30000) * 2.0 ** -7, "down": -np.minimum(j, 30000) * 2.0 ** -7,
         "period": np.where(j % 2048 < 8, 100.0 + j % 5, 0.0), "zeros": np.where(j % 3 == 0, -0.0, 0.0),
         "few": np.where(j % 997 == 5, 3.0, -INF), "blocks": (j // 1024 % 7).astype(float)}[kind]
    zt, z, _ = rows(np.stack([z, z[::-1]]), dt, 1)
    check_logprobs(zt, z, np.array([0, V - 1]), K=K, dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [999, 33000, 140001])
def test_gradient_in_place_and_apart(V, dt):
    """dlogits = logits; and dlogits of another pitch and alignment, whose surroundings stay as they were."""
    T = 5
    announce(f"in place V={V} {dt}")
    rng = np.random.default_rng(V)
    ids, gl, gh = rng.integers(0, V, T), rng.standard_normal(T), rng.standard_normal(T)
    zt, z, buf = rows(gauss(T, V, 4), dt, 3, 1, fill=5.0)
    out = torch.full((T * (V + 6) + 2,), 5.0, dtype=tdt(dt), device="cuda")
    dz = out.as_strided((T, V), (V + 6, 1), 2)
    check_logprobs(zt, z, ids, gl=gl, gh=gh, dt=dt, dz=dz)
    apart = dz.clone()
    dz.fill_(5.0)
    assert (out == 5.0).all()
    check_logprobs(zt, z, ids, gl=gl, gh=gh, dt=dt, dz=zt)
    assert torch.equal(zt, apart)
    zt.fill_(5.0)
    assert (buf == 5.0).all()
    # the distillation's gradient the same ways
    zt.copy_(torch.as_tensor(z))
    t_ids = rng.integers(-1, V, (T, 17))
    t_z, w = rng.standard_normal((T, 17)), rng.standard_normal(T)
    loss, stats = torch.empty(T, device="cuda"), torch.empty((T, 4), device="cuda")
    for mode in (0, 1):
        zt.copy_(torch.as_tensor(z))
        lse = f32(np.full(T, 4.0)) if mode else None
        B().poet_distill(zt, i32(t_ids), f32(t_z), loss, stats, mode=mode, t_lse=lse, dloss=f32(w), dlogits=dz)
        apart = dz.clone()
        dz.fill_(5.0)
        assert (out == 5.0).all()
        B().poet_distill(zt, i32(t_ids), f32(t_z), loss, stats, mode=mode, t_lse=lse, dloss=f32(w), dlogits=zt)
        assert torch.equal(zt, apart)
        zt.copy_(torch.as_tensor(z))
        B().poet_distill_bwd(zt, i32(t_ids), f32(t_z), stats, f32(w), zt, mode=mode, t_lse=lse)
        ref, err = R.distill(z, 1.0, t_ids, f32(t_z).double().cpu().numpy(), 1.0, bool(mode),
                             np.full(T, 4.0) if mode else None, f32(w).double().cpu().numpy())[2:]
        close(zt, ref, err + R.HALF[dt] * np.abs(ref) * 1.01 + 1e-38, "distill in place")
        zt.fill_(5.0)
        assert (buf == 5.0).all()


def check_distill(zt, z, t_ids, t_z, s=1.0, ts=1.0, tail=False, lse=None, w=None, dt="f32", ws=None):
    T, V = z.shape
    tz, tl = f32(t_z), None if lse is None else f32(lse)
    loss, stats = torch.full((T,), 7.0, device="cuda"), torch.full((T, 4), 7.0, device="cuda")
    wd = None if w is None else f32(w)
    dz = None if w is None else torch.full((T, V), 7.0, dtype=zt.dtype, device="cuda")
    kw = dict(mode=int(tail), inv_temp=s, t_inv_temp=ts, t_lse=tl)
    B().poet_distill(zt, i32(t_ids), tz, loss, stats, dloss=wd, dlogits=dz, ws=ws, **kw)
    torch.cuda.synchronize()
    ref, err, dref, derr = R.distill(z, s, t_ids, tz.double().cpu().numpy(), float(np.float32(ts)), tail,
                                     None if lse is None else tl.double().cpu().numpy(),
                                     None if w is None else wd.double().cpu().numpy())
    close(loss, ref, err + 2 * R.U * np.abs(np.where(np.isfinite(ref), ref, 0)), "loss")
    if w is not None:
        b = derr + R.HALF[dt] * np.abs(dref) * 1.01 + 1e-38
        close(dz, dref, b, "dlogits")
        again = torch.full((T, V), 3.0, dtype=zt.dtype, device="cuda")
        B().poet_distill_bwd(zt, i32(t_ids), tz, stats, wd, again, **kw)
        torch.cuda.synchronize()
        close(again, dref, b, "dlogits of the backward")
    return loss, dz


def teacher(z, K, seed):
    """A teacher near the student: the K best of z plus noise, and the log of its whole sum."""
    t = z + np.random.default_rng(seed).standard_normal(z.shape)
    ids = np.argsort(-t, axis=1, kind="stable")[:, :K]
    m = t.max(1, keepdims=True)
    return ids, np.take_along_axis(t, ids, 1), (m + np.log(np.exp(t - m).sum(1, keepdims=True)))[:, 0]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_distill_sizes(T, V, dt, tail):
    pad, skew = [(0, 0), (1, 0), (3, 1), (0, 5)][V % 4]
    K = min(V, 1 + V % 128)
    announce(f"distill T={T} V={V} K={K} {dt} tail={tail}")
    zt, z, _ = rows(gauss(T, V, 5), dt, pad, skew)
    ids, t, lse = teacher(z, K, V)
    w = np.random.default_rng(V).standard_normal(T)
    check_distill(zt, z, ids, t, tail=tail, lse=lse if tail else None, w=w, dt=dt)
    check_distill(zt, z, ids, t, tail=tail, lse=lse if tail else None, dt=dt)
    ids, t, lse = teacher(z * 0.5, K, V + 1)
    check_distill(zt, z, ids, t, s=0.5, ts=2.0, tail=tail, lse=2.0 * lse + 0.5 if tail else None, w=w, dt=dt)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [130, 1023, 20001, 140001])
def test_distill_lists(V, dt, tail):
    """Absent, repeated and foreign ids, whole rows of them, entries of no mass, masked students, a list that covers
    the whole vocabulary or leaves tokens of almost no mass, a zero weight."""
    T, K = 12, 128
    announce(f"distill lists V={V} {dt} tail={tail}")
    rng = np.random.default_rng(V)
    z = gauss(T, V, 6)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    t = rng.standard_normal((T, K)) - 6.0
    ids[0, ::3] = -1
    ids[1] = -1                                   # no teacher
    ids[2] = rng.integers(0, 4, K)                # repeated ids
    t[2] -= 1.0
    ids[3, :5] = [V, V + 7, -100, 2 ** 31 - 1, -2 ** 31]
    t[4, ::2] = -INF                              # entries of no mass
    z[5, ids[5]] = -INF                           # the student cannot give them
    t[5, ::2] = -INF
    z[6] = -INF                                   # a student row that its mask leaves nothing
    z[7] -= 200.0                                 # all unlisted tokens far below the listed ones
    z[7, ids[7]] += 200.0
    z[8, rng.random(V) < 0.5] = -INF
    z[8, ids[8]] = 1.0
    ids[9, 1:] = -1                               # one entry
    t[9, 0] = -0.001 if tail else 3.0
    t[10] = -INF                                  # a list without mass
    if not tail:
        t[10, 3] = 0.0
    zt, z, _ = rows(z, dt, 1)
    w = rng.standard_normal(T)
    w[11] = 0.0
    check_distill(zt, z, ids, t, tail=tail, w=w, dt=dt)
    if V == 130 and tail:                         # the list covers every token: nothing is left on either side
        full = np.tile(np.arange(V)[:K], (T, 1))
        z2 = z.copy()
        z2[:, K:] = -INF
        z2[5:7] = gauss(2, V, 8)
        z2[5:7, K:] = -INF
        zt2, z2, _ = rows(z2, dt)
        lq, _, _ = R.logprobs(gauss(T, K, 9))
        check_distill(zt2, z2, full, lq + 1e-3, tail=True, w=w, dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [90, 700, 1500, 3000, 7000, 15001, 30000])
def test_many_rows(V, dt):
    """Enough rows that each gets the smallest workgroup that holds it."""
    T, K = 530, 17
    announce(f"many rows V={V} {dt}")
    rng = np.random.default_rng(V)
    z = gauss(T, V, 12)
    z[:, rng.random(V) < 0.05] = -INF
    z[7] = -INF
    z[8, 3:] = -INF
    z[9] = np.round(z[9])
    zt, z, _ = rows(z, dt, 1 if V % 2 else 0)
    ids = rng.integers(-1, V, T)
    check_logprobs(zt, z, ids, K=K, gl=rng.standard_normal(T), gh=rng.standard_normal(T), dt=dt)
    check_logprobs(zt, z, ids, s=1.5, gl=rng.standard_normal(T), dt=dt)
    t_ids, t_z, lse = teacher(np.where(np.isfinite(z), z, -50.0), K, V)
    t_ids[5, 4:9] = t_ids[5, 0]
    t_ids[6] = -1
    w = rng.standard_normal(T)
    for tail in (False, True):
        check_distill(zt, z, t_ids, t_z, tail=tail, lse=lse + 0.2 if tail else None, w=w, dt=dt)


@pytest.mark.parametrize("V,dt,pad", [(65541, "f32", 0), (70001, "f32", 3), (131080, "bf16", 0), (140001, "bf16", 1)])
def test_many_long_rows(V, dt, pad):
    """Rows longer than a workgroup holds, enough of them that each is taken whole in parts: masks that empty a part or
    all of a row, a maximum in the first or the last part, lists over both; in place and apart."""
    T, K = 203, 21
    announce(f"many long rows V={V} {dt}")
    rng = np.random.default_rng(V)
    z = gauss(T, V, 15)
    z[0, : V // 2 + 100] = -INF
    z[1, V // 2 - 100:] = -INF
    z[2] = -INF
    z[3, 7], z[4, V - 1] = 40.0, 40.0
    z[5, : V // 2 + 100] -= 300.0
    zt, z, _ = rows(z, dt, pad)
    ids = rng.integers(-1, V, T)
    ids[3], ids[4], ids[6], ids[7] = 7, V - 1, 0, V // 2
    gl, gh = rng.standard_normal(T), rng.standard_normal(T)
    _, apart = check_logprobs(zt, z, ids, s=0.8, gl=gl, gh=gh, dt=dt, dz=torch.empty((T, V + 5), dtype=zt.dtype, device="cuda")[:, :V])
    apart = apart.clone()
    check_logprobs(zt, z, ids, s=0.8, gl=gl, gh=gh, dt=dt, dz=zt)
    assert torch.equal(zt, apart)
    zt.copy_(torch.as_tensor(z))
    t_ids = rng.integers(0, V, (T, K))
    t_ids[8, 1:6] = t_ids[8, 0]
    t_ids[9] = -1
    t_ids[10, :3] = [0, V - 1, V // 2]
    t_z, w = rng.standard_normal((T, K)) - 4.0, rng.standard_normal(T)
    for tail in (False, True):
        check_distill(zt, z, t_ids, t_z, tail=tail, w=w, dt=dt)


@pytest.mark.parametrize("T", [515, 640])
@pytest.mark.parametrize("V,dt,pad", [(65541, "f32", 0), (131071, "f32", 1), (140001, "bf16", 1)])
def test_long_rows_whole(V, dt, pad, T):
    """The same for the log-probabilities with more rows still (some of them are held to the formula), in numbers that go
    in segments and whole."""
    H = 12
    announce(f"long rows T={T} V={V} {dt}")
    rng = np.random.default_rng(V)
    head, tail = gauss(H, V, 16), gauss(3, V, 17)
    head[0, : V // 2 + 100] = -INF
    head[1, V // 2 - 100:] = -INF
    head[2] = -INF
    head[3, 7], head[4, V - 1] = 40.0, 40.0
    head[5, : V // 2 + 100] -= 300.0
    zt = torch.empty((T, V + pad), dtype=tdt(dt), device="cuda")[:, :V]
    zt.normal_()
    zt[:H], zt[T - 3:] = torch.as_tensor(head).to(tdt(dt)), torch.as_tensor(tail).to(tdt(dt))
    sel = np.r_[0:H, T - 3:T]
    z = zt[torch.as_tensor(sel).cuda()].double().cpu().numpy()
    ids = rng.integers(-1, V, T)
    ids[3], ids[4], ids[6], ids[7] = 7, V - 1, 0, V // 2
    gl, gh = f32(rng.standard_normal(T)), f32(rng.standard_normal(T))
    logp, Hd, st = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty((T, 4), device="cuda")
    apart = torch.empty((T, V + 3), dtype=zt.dtype, device="cuda")[:, :V]
    for dz in (apart, zt):
        B().poet_token_logprobs(zt, i32(ids), logp, st, inv_temp=0.8, entropy=Hd, dlogp=gl, dentropy=gh, dlogits=dz)
        torch.cuda.synchronize()
        lp, _, H64 = R.logprobs(z, 0.8)
        has = ids[sel] >= 0
        ref = np.where(has, lp[np.arange(len(sel)), np.where(has, ids[sel], 0)], 0.0)
        at = torch.as_tensor(sel).cuda()
        close(logp[at], ref, R.DZ + 4 * R.U * np.abs(np.where(np.isfinite(ref), ref, 0)), "logp")
        close(Hd[at], H64, R.entropy_bound(z, 0.8), "entropy")
        ref, err = R.logprobs_grad(z, 0.8, ids[sel], gl.double().cpu().numpy()[sel], gh.double().cpu().numpy()[sel])
        close(dz[at], ref, err + R.HALF[dt] * np.abs(ref) * 1.01 + 1e-38, "dlogits")
    assert torch.equal(zt, apart)


@pytest.mark.parametrize("dt,V", [("bf16", v) for v in (504, 1000, 1024, 2040, 4096, 8192, 16376, 32744, 32768)] +
                         [("f32", v) for v in (255, 512, 2047, 4096, 8180, 16384)])
def test_rows_that_fill_a_workgroup(dt, V):
    """Rows of as many 16-byte steps as a workgroup has places, or a few less, at every place in a line of memory: those
    that have room start at a line's beginning, the others do not."""
    T, K = 520, 9
    announce(f"rows that fill a workgroup V={V} {dt}")
    rng = np.random.default_rng(V)
    pad = {"bf16": 8, "f32": 4}[dt] if V % 8 == 0 else 1  # the next row starts one step later, or anywhere
    zt, z, _ = rows(gauss(T, V, 18), dt, pad, skew=pad)
    ids = rng.integers(-1, V, T)
    ids[:4] = [0, 1, V - 1, V - 2]
    check_logprobs(zt, z, ids, K=K, gl=rng.standard_normal(T), gh=rng.standard_normal(T), dt=dt,
                   dz=torch.empty((T, V + pad), dtype=zt.dtype, device="cuda")[:, :V])
    t_ids, t_z, _ = teacher(z, K, V)
    t_ids[:, :2] = [0, V - 1]
    check_distill(zt, z, t_ids, t_z, tail=bool(V & 8), w=rng.standard_normal(T), dt=dt)


@pytest.mark.parametrize("V,dt,pad", [(16411, "f32", 0), (40001, "f32", 3), (33333, "bf16", 1), (65536, "bf16", 8)])
def test_rows_in_segments(V, dt, pad):
    """Rows of 64 to 256 KB without a gradient, more of them than fit a workgroup each: masks that empty a segment or all
    of a row, equal logits across segments, a NaN; the same numbers as for the rows one at a time, to the bounds."""
    T, K = 260, 40
    announce(f"rows in segments V={V} {dt}")
    rng = np.random.default_rng(V)
    z = gauss(T, V, 19)
    z[0, : V // 2 + 100] = -INF
    z[1, V // 2 - 100:] = -INF
    z[2] = -INF
    z[3, 5:] = -INF
    z[4], z[5] = np.round(z[4]), 1.5
    z[6, V - 3] = float("nan")
    zt, z, _ = rows(z, dt, pad)
    ids = rng.integers(-1, V, T)
    check_logprobs(zt, z, ids, s=1.3, K=K, dt=dt)
    few = slice(0, 9)
    check_logprobs(zt[few], z[few], ids[few], s=1.3, K=K, dt=dt)
    t_ids, t_z, lse = teacher(np.where(np.isfinite(z), z, -50.0), K, V)
    t_ids[9, 4:9] = t_ids[9, 0]
    t_ids[10] = -1
    for tail in (False, True):
        lt = lse + 0.2 if tail else None
        check_distill(zt, z, t_ids, t_z, tail=tail, lse=lt, dt=dt)
        check_distill(zt[few], z[few], t_ids[few], t_z[few], tail=tail, lse=lt[few] if tail else None, dt=dt)


@pytest.mark.parametrize("V,dt,pad", [(65541, "f32", 3), (140001, "bf16", 1)])
def test_distill_gradient_of_segments(V, dt, pad):
    """The distillation's gradient after segments, for numbers of rows that do not fill the CUs (some of the rows are held
    to the formula): lists over several segments, repeated and absent entries, masks; in place and apart, and the backward
    alone, which reads the list again."""
    T, K, H = 260, 30, 14
    announce(f"distillation gradient of segments V={V} {dt}")
    rng = np.random.default_rng(V)
    head = gauss(H, V, 21)
    head[0, : V // 2 + 100] = -INF
    head[1] = -INF
    head[2, V - 1] = 40.0
    zt = torch.empty((T, V + pad), dtype=tdt(dt), device="cuda")[:, :V]
    zt.normal_()
    zt[:H] = torch.as_tensor(head).to(tdt(dt))
    keep = zt.clone()
    z = zt[:H].double().cpu().numpy()
    t_ids = rng.integers(0, V, (T, K))
    t_ids[3, 1:6] = t_ids[3, 0]
    t_ids[4] = -1
    t_ids[5, :4] = [0, V - 1, V // 2, -100]
    t_z, w = rng.standard_normal((T, K)) - 4.0, rng.standard_normal(T)
    w[6] = 0.0
    ids, tz, wd = i32(t_ids), f32(t_z), f32(w)
    loss, st = torch.empty(T, device="cuda"), torch.empty((T, 4), device="cuda")
    for mode in (0, 1):
        got = []
        for dz in (torch.empty((T, V + 2), dtype=zt.dtype, device="cuda")[:, :V], zt):
            B().poet_distill(zt, ids, tz, loss, st, mode=mode, dloss=wd, dlogits=dz)
            got.append(dz.clone())
        zt.copy_(keep)
        B().poet_distill_bwd(zt, ids, tz, st, wd, zt, mode=mode)
        got.append(zt.clone())
        zt.copy_(keep)
        ref, err, dref, derr = R.distill(z, 1.0, t_ids[:H], tz.double().cpu().numpy()[:H], 1.0, bool(mode), None,
                                         wd.double().cpu().numpy()[:H])
        close(loss[:H], ref, err + 2 * R.U * np.abs(np.where(np.isfinite(ref), ref, 0)), "loss")
        for g in got:
            close(g[:H], dref, derr + R.HALF[dt] * np.abs(dref) * 1.01 + 1e-38, "dlogits")
        assert torch.equal(got[0], got[1])


def test_more_rows_than_workgroups():
    """More rows than one launch has workgroups."""
    T, V, P = 1_100_003, 9, 7
    announce("more rows than workgroups")
    base, t = gauss(P, V, 13), torch.arange(T, device="cuda") % P
    zt = torch.as_tensor(base, dtype=torch.float32).cuda()[t].contiguous()
    ids = (t % V).to(torch.int32)
    one = torch.ones(T, device="cuda")
    o = dict(logp=torch.empty(T, device="cuda"), stats=torch.empty((T, 4), device="cuda"), entropy=torch.empty(T, device="cuda"),
             top_ids=torch.empty((T, 3), dtype=torch.int32, device="cuda"), top_logp=torch.empty((T, 3), device="cuda"),
             dlogits=torch.empty_like(zt))
    B().poet_token_logprobs(zt, ids, dlogp=one, dentropy=one, **o)
    d = dict(loss=torch.empty(T, device="cuda"), stats=torch.empty((T, 4), device="cuda"), dlogits=torch.empty_like(zt))
    B().poet_distill(zt, o["top_ids"], o["top_logp"], mode=1, dloss=one, **d)
    again = torch.empty_like(zt)
    B().poet_token_logprobs_bwd(zt, ids, o["stats"], one, again, dentropy=one)
    torch.cuda.synchronize()
    assert torch.equal(again, o["dlogits"])
    # rows of an odd pitch lie at four alignments, where their sums are taken in different orders: every row is held to
    # the formula with the bounds of tests/token_ref.py
    z64, n, t = zt[:P].double().cpu().numpy(), np.arange(P), t.cpu().numpy()
    lp, _, H = R.logprobs(z64)
    bound = lambda r: R.DZ + 4 * R.U * np.abs(r)  # noqa: E731
    idp = ids.cpu().numpy()
    close(o["logp"], lp[t, idp], bound(lp[t, idp]), "logp")
    close(o["entropy"], H[t], R.entropy_bound(z64)[t], "entropy")
    at = R.top(z64, 3)
    np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), at[t])
    tl = np.take_along_axis(lp, at, 1)
    close(o["top_logp"], tl[t], bound(tl)[t], "top_logp")
    for k in range(V):  # the gradients of the rows whose token is k
        sel = np.flatnonzero(idp == k)[:1000]
        ref, err = R.logprobs_grad(z64[t[sel]], 1.0, idp[sel], np.ones(len(sel)), np.ones(len(sel)))
        close(o["dlogits"][torch.as_tensor(sel).cuda()], ref, err + R.U * np.abs(ref) + 1e-38, "dlogits")
    sel = np.r_[0:500, T - 500:T]
    ref, err, dref, derr = R.distill(z64[t[sel]], 1.0, at[t[sel]], o["top_logp"].double().cpu().numpy()[sel], 1.0, True, None,
                                     np.ones(len(sel)))
    close(d["loss"][torch.as_tensor(sel).cuda()], ref, err + 2 * R.U * np.abs(ref), "loss")
    close(d["dlogits"][torch.as_tensor(sel).cuda()], dref, derr + R.U * np.abs(dref) + 1e-38, "dlogits of the distillation")


@pytest.mark.parametrize("s", [1e-30, 1e-3, 300.0, 1e30])
def test_extreme_temperatures_and_gradients(s):
    """Temperatures at the ends of their range, upstream gradients of 1e20, masked logits: finite, and the formula's."""
    T, V = 4, 600
    announce(f"temperature {s}")
    rng = np.random.default_rng(3)
    z = gauss(T, V, 14)
    z[:, ::3] = -INF
    z[1, ::3] = -3e38
    zt, z, _ = rows(z, "f32")
    big = 1e20 if s < 1e10 else 1.0
    gl, gh = f32(big * rng.standard_normal(T)), f32(big * rng.standard_normal(T))
    check_logprobs(zt, z, np.array([1, 2, 4, -1]), s=float(np.float32(s)), gl=gl.double().cpu().numpy(),
                   gh=gh.double().cpu().numpy())


def test_gradients_against_differences():
    """Both gradients against central differences of the float64 formulas along random directions."""
    T, V, K, s, e = 4, 61, 9, 0.8, 1e-5
    announce("gradients against differences")
    rng = np.random.default_rng(0)
    zt, z, _ = rows(gauss(T, V, 7), "f32")
    ids, gl, gh = rng.integers(0, V, T), rng.standard_normal(T), rng.standard_normal(T)
    gl, gh = np.float32(gl).astype(float), np.float32(gh).astype(float)
    _, dz = check_logprobs(zt, z, ids, s=s, gl=gl, gh=gh)

    def value(x):
        lp, _, H = R.logprobs(x, s)
        return (gl * lp[np.arange(T), ids]).sum() + (gh * H).sum()
    t_ids, t_z, lse = teacher(z, K, 1)
    t_z, lse = np.float32(t_z).astype(float), np.float32(lse + 0.3).astype(float)
    for tail in (None, False, True):
        if tail is not None:
            _, dz = check_distill(zt, z, t_ids, t_z, s=s, tail=tail, lse=lse if tail else None, w=gl)
            value = lambda x: (gl * R.distill(x, s, t_ids, t_z, 1.0, tail, lse if tail else None)[0]).sum()  # noqa: E731,B023
        g = dz.double().cpu().numpy()
        for r in range(3):
            u = np.random.default_rng(r).standard_normal((T, V))
            diff = (value(z + e * u) - value(z - e * u)) / (2 * e)
            # second-order term of the difference: e^2 times a third derivative of order 1; rounding 1e-16 / e
            assert abs((g * u).sum() - diff) <= 2e-5 * (np.abs(g * u).sum() + 1.0), (tail, r)


def test_offsets_past_32_bits():
    """Row offsets beyond 2^31 elements and 2^32 bytes."""
    T, V, ld = 3, 1000, 1_200_000_008
    announce("offsets past 32 bits")
    buf = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    zt = buf.as_strided((T, V), (ld, 1), 0)
    zt.copy_(torch.as_tensor(gauss(T, V, 10)))
    z = zt.double().cpu().numpy()
    ids = np.array([1, 2, 999])
    rng = np.random.default_rng(1)
    check_logprobs(zt, z, ids, K=5, gl=rng.standard_normal(T), gh=rng.standard_normal(T), dt="bf16", dz=zt)
    zt.copy_(torch.as_tensor(z))
    t_ids, t_z, lse = teacher(z, 8, 2)
    check_distill(zt, z, t_ids, t_z, tail=True, lse=lse, w=rng.standard_normal(T), dt="bf16")


def test_empty_batch():
    z = torch.empty((0, 50), device="cuda")
    e, st = torch.empty(0, device="cuda"), torch.empty((0, 4), device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    B().poet_token_logprobs(z, i, e, st, entropy=e, dlogp=e, dlogits=torch.empty_like(z))
    B().poet_token_logprobs_bwd(z, i, st, e, torch.empty_like(z))
    ti, tz = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    B().poet_distill(z, ti, tz, e, st, dloss=e, dlogits=torch.empty_like(z))
    B().poet_distill_bwd(z, ti, tz, st, e, torch.empty_like(z))
    torch.cuda.synchronize()


def test_rows_behind_the_last_stay():
    """Outputs larger rows would fall into are left alone: the rows after T of every output buffer."""
    T, V, K = 3, 4097, 6
    announce("rows behind the last")
    big = torch.full((T + 2, V), 9.0, device="cuda")
    z = torch.randn((T, V), device="cuda")
    lg, H = torch.full((T + 2,), 9.0, device="cuda"), torch.full((T + 2,), 9.0, device="cuda")
    st, tl = torch.full((T + 2, 4), 9.0, device="cuda"), torch.full((T + 2, K), 9.0, device="cuda")
    ti = torch.full((T + 2, K), 9, dtype=torch.int32, device="cuda")
    B().poet_token_logprobs(z, i32([1, 2, 3]), lg[:T], st[:T], entropy=H[:T], top_ids=ti[:T], top_logp=tl[:T],
                            dlogp=f32([1, 1, 1]), dlogits=big[:T])
    B().poet_distill(z, ti[:T], tl[:T], lg[:T], st[:T], dloss=f32([1, 1, 1]), dlogits=big[:T])
    for t in (big, lg, H, st, tl, ti):
        assert (t[T:] == 9).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 140001), (700, 3001), (3, 32000)])
def test_two_streams_and_graph_replay(T, V, dt):
    """The same calls on two streams at once (each with its own workspace and outputs) and replayed from a graph with
    eager work between the replays: the same bits every time."""
    announce(f"streams and graph T={T} V={V} {dt}")
    K = 10
    zt, z, _ = rows(gauss(T, V, 11), dt, 1)
    ids = i32(np.random.default_rng(0).integers(0, V, T))
    one = torch.ones(T, device="cuda")
    dtc = B().POET_BF16 if dt == "bf16" else B().POET_F32
    need = max(B().poet_token_logprobs_workspace_bytes(T, V, dtc, K), B().poet_distill_workspace_bytes(T, V, dtc), 1)

    def outs():
        o = dict(logp=torch.empty(T, device="cuda"), stats=torch.empty((T, 4), device="cuda"),
                 entropy=torch.empty(T, device="cuda"), top_ids=torch.empty((T, K), dtype=torch.int32, device="cuda"),
                 top_logp=torch.empty((T, K), device="cuda"), dlogits=torch.empty((T, V), dtype=zt.dtype, device="cuda"))
        d = dict(loss=torch.empty(T, device="cuda"), stats=torch.empty((T, 4), device="cuda"),
                 dlogits=torch.empty((T, V), dtype=zt.dtype, device="cuda"))
        return o, d, torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(bufs, stream=None):
        o, d, ws = bufs
        B().poet_token_logprobs(zt, ids, dlogp=one, dentropy=one, ws=ws, stream=stream, **o)
        B().poet_distill(zt, o["top_ids"], o["top_logp"], mode=1, dloss=one, ws=ws, stream=stream, **d)

    def flat(bufs):
        return [t.clone() for part in bufs[:2] for t in part.values()]
    ref = outs()
    call(ref)
    want = flat(ref)
    streams, bufs = [torch.cuda.Stream(), torch.cuda.Stream()], [outs(), outs()]
    torch.cuda.synchronize()
    for s, b in zip(streams, bufs):
        call(b, s)
    torch.cuda.synchronize()
    for b in bufs:
        assert all(torch.equal(x, y) for x, y in zip(want, flat(b)))
    b = outs()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(b)
    for _ in range(3):
        for part in b[:2]:
            for t in part.values():
                t.fill_(3)
        call(ref)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, flat(b)))

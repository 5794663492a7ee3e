"""A whole training step of a small POET model on the GPU through the C ABI, as a program makes it: the norm before a
block, its linear, the seam with gate and residual behind it, a head linear, the token loss with entropy bonus and the
distillation loss on a teacher's best alternatives, and all of it backwards to the skew parameters and the norms'
weights, against the same chain in float64 (the oracle's linears, tests/token_ref.py's norms and losses).

Tolerance: float32 linears are held to 1e-5 by their own tests; two forward and two backward ones stand on the longest
path (4e-5), the norms and losses add their bounds (below 1e-6), and the losses' gradients turn a relative error of the
logits (of magnitude about 3) into one of p: 1e-4 covers the sum, relative to the norm of each result."""
import numpy as np
import pytest

import oracle as O
import poet_inputs as PI
from tests import token_ref as R
from tests.gpu_util import announce, make_linear, rel

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
T, D, V, K, GT, A, EPS, S = 37, 96, 203, 12, 5, 0.7, 1e-5, 1.0
TOL = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Model:
    """One block and a head, their buffers, and one step of them."""

    def __init__(self, dt=PI.DT_F32, path="weight"):
        from orthogonal_reparameterized_amd import binding as B
        from orthogonal_reparameterized_amd.layer import PoetLinear
        self.B, self.dt, self.path = B, dt, path
        rng = np.random.default_rng(5)
        f32 = lambda a: torch.as_tensor(np.asarray(a, np.float32)).cuda()  # noqa: E731
        act = torch.float32 if dt == PI.DT_F32 else torch.bfloat16
        self.specs, self.lins, self.host = [], [], []
        for i, (m, n) in enumerate(((D, D), (V, D))):
            spec = make_linear(f"step{i}", m, n, T, PI.MODE_BS, 32, 32, 3, dt, linear_id=i)
            W0, tR, tP, _, _ = PI.gen_linear(60 + i, 0, spec, theta_std=0.02)
            self.specs.append(spec)
            self.host.append((W0, tR, tP))
            self.lins.append(PoetLinear(m, n, T, B.side_of(spec.R), B.side_of(spec.P), dt, W0, tR, tP, path=path,
                                        ldw=PI.pad_ld(n, 8), ldx=PI.pad_ld(n, 8), ldy=PI.pad_ld(m, 8)))
        self.h0 = f32(rng.standard_normal((T, D)) * 2)
        self.gate = f32(rng.standard_normal((-(-T // GT), D))).to(act)
        self.w0, self.wq, self.w1 = (f32(1 + 0.1 * rng.standard_normal(D)) for _ in range(3))
        self.ids = torch.as_tensor(rng.integers(0, V, T), dtype=torch.int32).cuda()
        self.ids[3] = -100
        self.wl, self.wh, self.wd = f32(-rng.random(T)), f32(0.1 * rng.standard_normal(T)), f32(rng.random(T))
        self.teacher = f32(rng.standard_normal((T, V)) * 2)
        new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.x0, self.x1 = new(T, D, dtype=act), new(T, D, dtype=act)
        self.y, self.ldv = new(T, D, dtype=act), PI.pad_ld(V, 8)
        self.z_buf = new(T, self.ldv, dtype=act)
        self.r0, self.r1, self.h1 = new(T, 2), new(T, 2), new(T, D)
        self.logp, self.H, self.st, self.loss, self.std = new(T), new(T), new(T, 4), new(T), new(T, 4)
        self.t_ids, self.t_lp, self.t_st = new(T, K, dtype=torch.int32), new(T, K), new(T, 4)
        self.dz_buf, self.dz2 = new(T, self.ldv, dtype=act), new(T, V, dtype=act)
        self.dx1, self.dx0, self.dy = new(T, D, dtype=act), new(T, D, dtype=act), new(T, D, dtype=act)
        self.dh1, self.dh0, self.dgate = new(T, D), new(T, D), torch.zeros_like(self.gate)
        self.dw0, self.dwq, self.dw1 = new(D), new(D), new(D)
        self.ws = torch.empty(max(1, B.poet_block_norm_workspace_bytes(T, D, GT), B.poet_block_norm_workspace_bytes(T, D)),
                              dtype=torch.uint8, device="cuda")
        self.keep = [lin.alloc_act(T, lin.L.ldy) if path == "act" else lin.alloc_W() for lin in self.lins]

    def linear(self, i, X, Y):
        lin = self.lins[i]
        lin.forward_act(X, Y, self.keep[i]) if self.path == "act" else lin.forward(X, Y, W_out=self.keep[i])

    def linear_bwd(self, i, X, dY, dX):
        lin = self.lins[i]
        if self.path == "act":
            lin.backward_act(X, self.keep[i], dY, dX)
        else:
            lin.backward(X, dY, dX, W=self.keep[i])

    def step(self):
        B = self.B
        z, dz = self.z_buf[:, :V], self.dz_buf[:, :V]
        for lin in self.lins:
            lin.build()
        # the teacher's answer: its best alternatives and their log-probabilities
        B.poet_token_logprobs(self.teacher, None, None, self.t_st, top_ids=self.t_ids, top_logp=self.t_lp)
        B.poet_block_norm_fwd(self.h0, self.r0, w_pre=self.w0, x=self.x0, eps=EPS)
        self.linear(0, self.x0, self.y)
        B.poet_block_norm_fwd(self.h0, self.r1, y=self.y, gate=self.gate, w_post=self.wq, w_pre=self.w1, h_out=self.h1,
                              x=self.x1, res_scale=A, eps=EPS, gate_tokens=GT)
        self.linear(1, self.x1, self.z_buf)
        B.poet_token_logprobs(z, self.ids, self.logp, self.st, entropy=self.H, dlogp=self.wl, dentropy=self.wh, dlogits=dz)
        B.poet_distill(z, self.t_ids, self.t_lp, self.loss, self.std, mode=B.POET_DISTILL_TAIL, dloss=self.wd,
                       dlogits=self.dz2)
        dz += self.dz2
        self.linear_bwd(1, self.x1, self.dz_buf, self.dx1)
        B.poet_block_norm_bwd(self.h1, self.r1, y=self.y, gate=self.gate, w_post=self.wq, w_pre=self.w1, dx=self.dx1,
                              dh=self.dh1, dy=self.dy, dgate=self.dgate, dw_post=self.dwq, dw_pre=self.dw1, res_scale=A,
                              gate_tokens=GT, ws=self.ws)
        self.linear_bwd(0, self.x0, self.dy, self.dx0)
        B.poet_block_norm_bwd(self.h0, self.r0, w_pre=self.w0, dh_out=self.dh1, dx=self.dx0, dh=self.dh0, dw_pre=self.dw0,
                              ws=self.ws)

    def results(self):
        r = {k: getattr(self, k) for k in ("logp", "H", "loss", "dh0", "dgate", "dw0", "dwq", "dw1")}
        for i, lin in enumerate(self.lins):
            r[f"dthetaR{i}"], r[f"dthetaP{i}"] = lin.dthetaR, lin.dthetaP
        return r

    def reference(self):
        n = lambda t: t.double().cpu().numpy()  # noqa: E731
        ident = lambda v: v  # noqa: E731
        g = {k: n(getattr(self, k)) for k in ("h0", "gate", "w0", "wq", "w1", "wl", "wh", "wd", "teacher")}
        ids = self.ids.cpu().numpy()
        side = [(O.Side.of(s.R), O.Side.of(s.P)) for s in self.specs]
        _, _, x0, _, _, rh0 = R.norm_fwd(g["h0"], None, None, None, g["w0"], 1.0, EPS, 1, ident)
        y = O.linear_fwd(*side[0], *self.host[0], None, None, x0)["Y"]
        h1, _, x1, _, ry1, rh1 = R.norm_fwd(g["h0"], y, g["gate"], g["wq"], g["w1"], A, EPS, GT, ident)
        z = O.linear_fwd(*side[1], *self.host[1], None, None, x1)["Y"]
        lp, _, H = R.logprobs(z, S)
        has = (ids >= 0) & (ids < V)
        dz, _ = R.logprobs_grad(z, S, ids, g["wl"], g["wh"])
        tlp = R.logprobs(g["teacher"])[0]
        t_ids = R.top(g["teacher"], K)
        loss, _, dzd, _ = R.distill(z, S, t_ids, np.take_along_axis(tlp, t_ids, 1), 1.0, True, None, g["wd"])
        b1 = O.linear_bwd(*side[1], *self.host[1], None, None, x1, dz + dzd)
        s1 = R.norm_bwd(h1, y, g["gate"], g["wq"], g["w1"], ry1, rh1, None, b1["dX"], A, GT, T)
        b0 = O.linear_bwd(*side[0], *self.host[0], None, None, x0, s1["dy"][0])
        s0 = R.norm_bwd(g["h0"], np.zeros((T, D)), None, None, g["w0"], 1.0, rh0, s1["dh"][0], b0["dX"], 1.0, 1, T)
        return dict(logp=np.where(has, lp[np.arange(T), np.where(has, ids, 0)], 0.0), H=H, loss=loss, dh0=s0["dh"][0],
                    dgate=s1["dgate"][0], dw0=s0["dw_pre"][0], dwq=s1["dw_post"][0], dw1=s1["dw_pre"][0],
                    dthetaR0=b0["dthetaR"], dthetaP0=b0["dthetaP"], dthetaR1=b1["dthetaR"], dthetaP1=b1["dthetaP"])


def test_step_against_float64():
    announce("training step float32")
    m = Model()
    m.step()
    torch.cuda.synchronize()
    ref, got = m.reference(), m.results()
    errs = {k: rel(got[k].double().cpu().numpy(), ref[k]) for k in ref}
    assert all(e <= TOL for e in errs.values()), errs


@pytest.mark.parametrize("path", ["weight", "act"])
def test_bf16_step_replayed_from_a_graph(path):
    """The bf16 step on either path of the linears, captured and replayed with eager work between the replays: the eager
    step's bits every time, and finite gradients of everything that learns."""
    announce(f"training step bf16 path={path}")
    m = Model(PI.DT_BF16, path)
    m.step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in m.results().items()}
    assert all(v.float().isfinite().all() and v.float().abs().max() > 0 for v in want.values())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step()
    for _ in range(3):
        for v in m.results().values():
            v.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], v) for k, v in m.results().items())
        m.step()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], v) for k, v in m.results().items())

"""Measured cases of the operators around a stack of POET linears: what the trained model answers with and is trained
on (token log-probabilities with entropy and top alternatives, distillation from a teacher's top logits) and the
norm-gate-residual seam between two blocks of linears.

A case is one call as a training or evaluation program makes it. ``own`` false: the operator in elementary torch
operations, 32 bits inside, rounded once; ``own`` true: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
NO_TOKEN = -100  # a position that scores no token (padding, prompt)


# ---- cases ----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decoding loop: the chosen token's log-probability and 20 alternatives (latency)
        dict(name="score 1x32000 bf16", op="logprobs", do="score", T=1, V=32000, pad=0, dtype="bf16", K=20, temp=1.0,
             masked=0.0, entropy=True),
        # evaluation of 8192 positions (32 sequences of 256), with what an evaluation logs
        dict(name="score 8192x32000 bf16", op="logprobs", do="score", T=8192, V=32000, pad=0, dtype="bf16", K=20,
             temp=1.0, masked=0.0, entropy=True),
        # a ragged batch in float32, odd vocabulary without padding, a constrained vocabulary (half masked), tempered
        dict(name="score 1000x50001 f32 masked", op="logprobs", do="score", T=1000, V=50001, pad=0, dtype="f32", K=5,
             temp=0.7, masked=0.5, entropy=True),
        # the loss of a pretraining step: weights of the positions are known, the gradient comes with the loss
        dict(name="train 16384x32000 bf16", op="logprobs", do="train", T=16384, V=32000, pad=0, dtype="bf16", K=0,
             temp=1.0, masked=0.0, entropy=False),
        # the backward alone, after a loss that needs the log-probabilities first (a policy ratio), entropy bonus
        dict(name="bwd 4095x50001 f32", op="logprobs", do="bwd", T=4095, V=50001, pad=7, dtype="f32", K=0, temp=1.0,
             masked=0.0, entropy=True),
        # distillation of a short batch on the teacher's 64 best tokens (loss only: validation)
        dict(name="distill loss 255x32000 bf16", op="distill", do="loss", T=255, V=32000, pad=0, dtype="bf16", K=64,
             temp=1.0, tail=False),
        # a distillation training step, the teacher's remaining mass as one more outcome
        dict(name="distill train 8192x32000 bf16", op="distill", do="train", T=8192, V=32000, pad=0, dtype="bf16",
             K=64, temp=2.0, tail=True),
        # the same in float32 on a large odd vocabulary, 100 entries, renormalized
        dict(name="distill train 511x131071 f32", op="distill", do="train", T=511, V=131071, pad=1, dtype="f32",
             K=100, temp=1.0, tail=False),
        # the seam before a block while one token is decoded (latency)
        dict(name="seam fwd 1x2048 bf16", op="seam", do="fwd", T=1, d=2048, res="bf16", act="bf16", post=True,
             gate_tokens=1, scale=1.0),
        # the seam of a training step at LLaMA-1.3B's width, gated per token
        dict(name="seam fwd 16384x2048 bf16", op="seam", do="fwd", T=16384, d=2048, res="bf16", act="bf16", post=True,
             gate_tokens=1, scale=0.5),
        # its backward at LLaMA-3B's width and tokens (64 sequences of 512), one gate a sequence, float32 residual
        dict(name="seam bwd 32768x2560 bf16", op="seam", do="bwd", T=32768, d=2560, res="f32", act="bf16", post=True,
             gate_tokens=512, scale=0.5),
        # the backward of a plain residual add and norm, an odd width, a ragged number of tokens, float32
        dict(name="seam bwd 1001x1377 f32", op="seam", do="bwd", T=1001, d=1377, res="f32", act="f32", post=False,
             gate_tokens=0, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "distill", "distill", "seam", "seam"])
    if op == "seam":
        d = _log(rng, 64, 8192)
        T = _log(rng, 1, min(32768, 40_000_000 // d))
        return dict(op=op, do=rng.choice(["fwd", "bwd"]), T=T, d=d, res=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["bf16", "bf16", "f32"]), post=rng.random() < 0.7,
                    gate_tokens=rng.choice([0, 1, 1, rng.randint(2, 700)]), scale=rng.choice([1.0, 0.5, 0.18]))
    V = _log(rng, 1000, 131072)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    T = _log(rng, 1, min(16384, (260_000_000 if dtype == "bf16" else 130_000_000) // V))
    pad = rng.choice([0, 0, 1, 24])
    temp = rng.choice([1.0, 1.0, 0.7, 2.0])
    if op == "logprobs":
        do = rng.choice(["score", "train", "bwd"])
        return dict(op=op, do=do, T=T, V=V, pad=pad, dtype=dtype, K=rng.choice([0, 1, 5, 20, 64]) if do == "score" else 0,
                    temp=temp, masked=rng.choice([0.0, 0.0, 0.9]), entropy=rng.random() < 0.5)
    return dict(op=op, do=rng.choice(["loss", "train"]), T=T, V=V, pad=pad, dtype=dtype, K=rng.choice([1, 8, 20, 64, 128]),
                temp=temp, tail=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _rows(T, n, pad, dtype):
    """T rows of n values at a row pitch of n + pad."""
    return torch.empty((T, n + pad), dtype=dtype, device=DEV)[:, :n]


def _logits(c, g):
    """Logits as a trained head gives them: a broad background and one likely token a row."""
    T, V = c["T"], c["V"]
    z = torch.randn((T, V), generator=g, device=DEV) * 2.0
    likely = torch.randint(0, V, (T, 1), generator=g, device=DEV)
    z.scatter_add_(1, likely, 12.0 * torch.rand((T, 1), generator=g, device=DEV))
    if c.get("masked"):
        z.masked_fill_(torch.rand((1, V), generator=g, device=DEV) < c["masked"], -math.inf)
    out = _rows(T, V, c["pad"], _dt(c["dtype"]))
    out.copy_(z)
    return out, likely[:, 0].to(torch.int32)


def _prepare_logprobs(c, g):
    T, V, f32 = c["T"], c["V"], dict(dtype=torch.float32, device=DEV)
    z, likely = _logits(c, g)
    ids = torch.where(torch.rand(T, generator=g, device=DEV) < 0.6, likely,
                      torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32))
    if T > 1:
        ids = torch.where(torch.rand(T, generator=g, device=DEV) < 0.1, torch.full_like(ids, NO_TOKEN), ids)
    s = dict(case=c, z=z, ids=ids, logp=torch.empty(T, **f32), stats=torch.empty((T, 4), **f32), ws=None)
    s["H"] = torch.empty(T, **f32) if c["entropy"] else None
    s["top_ids"] = torch.empty((T, c["K"]), dtype=torch.int32, device=DEV) if c["K"] else None
    s["top_logp"] = torch.empty((T, c["K"]), **f32) if c["K"] else None
    if c["do"] != "score":
        s["dlogp"] = -torch.rand(T, generator=g, device=DEV)
        s["dH"] = 0.3 * torch.randn(T, generator=g, device=DEV) if c["entropy"] else None
        s["dz"] = _rows(T, V, c["pad"], z.dtype)
    if c["do"] == "bwd":  # what the forward left for the backward: row maximum, log of the sum, entropy
        w = z.float()
        m = w.amax(1)
        d = (w - m[:, None]) / c["temp"]
        e = d.exp()
        Z = e.sum(1)
        H = Z.log() - (e * d.clamp_min(-1e30)).sum(1) / Z
        s["stats"].copy_(torch.stack([m, Z.log(), H, torch.zeros_like(H)], 1))
    return s


def _prepare_distill(c, g):
    T, V, K, f32 = c["T"], c["V"], c["K"], dict(dtype=torch.float32, device=DEV)
    z, _ = _logits(c, g)
    # the teacher agrees with the student up to noise; its K best tokens and the log of its sum, as it answered
    t = z.float() + torch.randn((T, V), generator=g, device=DEV)
    top = t.topk(K, dim=1)
    s = dict(case=c, z=z, t_ids=top.indices.to(torch.int32), t_z=top.values.contiguous(),
             t_lse=torch.logsumexp(t / c["temp"], 1) if c["tail"] else None, loss=torch.empty(T, **f32),
             stats=torch.empty((T, 4), **f32), ws=None)
    if T > 2:  # a position without a teacher, and one whose list is short
        s["t_ids"][T // 2] = -1
        s["t_ids"][T // 3, K // 2:] = -1
    if c["do"] != "loss":
        s["dloss"] = torch.rand(T, generator=g, device=DEV) + 0.1
        s["dz"] = _rows(T, V, c["pad"], z.dtype)
    return s


def _prepare_seam(c, g):
    T, d, res, act = c["T"], c["d"], _dt(c["res"]), _dt(c["act"])
    def randn(rows, dt, k=1.0):
        return (torch.randn((rows, d), generator=g, device=DEV) * k).to(dt)
    weight = lambda: 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)  # noqa: E731
    gt = c["gate_tokens"]
    s = dict(case=c, y=randn(T, act, 0.7), gate=randn(-(-T // gt), act) if gt else None,
             w_post=weight() if c["post"] else None, w_pre=weight(), ws=None,
             rstd=torch.empty((T, 2), dtype=torch.float32, device=DEV))
    if c["do"] == "fwd":
        s.update(h=randn(T, res, 2.0), h_out=torch.empty((T, d), dtype=res, device=DEV),
                 x=torch.empty((T, d), dtype=act, device=DEV))
        return s
    s.update(h_out=randn(T, res, 2.0), dh_out=randn(T, res, 0.3), dx=randn(T, act),
             dh=torch.empty((T, d), dtype=res, device=DEV), dy=torch.empty((T, d), dtype=act, device=DEV),
             dgate=None if s["gate"] is None else torch.empty_like(s["gate"]),
             dw_post=torch.empty(d, device=DEV) if c["post"] else None, dw_pre=torch.empty(d, device=DEV))
    s["rstd"][:, 0] = (s["y"].float().square().mean(1) + EPS).rsqrt() if c["post"] else 1.0
    s["rstd"][:, 1] = (s["h_out"].float().square().mean(1) + EPS).rsqrt()
    return s


EPS = 1e-6


def prepare(case, seed):
    g = _gen(seed)
    return {"logprobs": _prepare_logprobs, "distill": _prepare_distill, "seam": _prepare_seam}[case["op"]](case, g)


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _top(w, K):
    """The K largest values' places in each row, equal values by the lower place."""
    i = (w + 0.0).view(torch.int32).long()  # + 0.0: one zero
    key = (torch.where(i < 0, i ^ 0x7FFFFFFF, i) << 32) + (w.shape[1] - torch.arange(w.shape[1], device=w.device))
    return key.topk(K, dim=1, sorted=True).indices


def _token(ids, V):
    has = (ids >= 0) & (ids < V)
    return has, torch.where(has, ids, torch.zeros_like(ids)).long()[:, None]


def _plain_logprobs(s):
    c, z, it = s["case"], s["z"], 1.0 / s["case"]["temp"]
    w = z.float()
    has, at = _token(s["ids"], c["V"])
    if c["do"] == "bwd":
        m, logZ, H = s["stats"][:, 0:1], s["stats"][:, 1:2], s["stats"][:, 2]
        lp = (w - m) * it - logZ
    else:
        d = (w - w.amax(1, keepdim=True)) * it
        e = d.exp()
        Z = e.sum(1, keepdim=True)
        logZ = Z.log()
        lp = d - logZ
        H = logZ[:, 0] - (e * d.clamp_min(-1e30)).sum(1) / Z[:, 0] if c["entropy"] else None
    out = {}
    if c["do"] != "bwd":
        out["logp"] = torch.where(has, lp.gather(1, at)[:, 0], torch.zeros_like(lp[:, 0]))
        if c["entropy"]:
            out["entropy"] = H
    if c["K"]:
        top = _top(w, c["K"])
        out["top_ids"], out["top_logp"] = top.to(torch.int32), lp.gather(1, top)
    if c["do"] != "score":
        p, gl = lp.exp(), torch.where(has, s["dlogp"], torch.zeros_like(s["dlogp"]))
        k = -gl[:, None]
        if c["entropy"]:
            k = k - s["dH"][:, None] * (lp.clamp_min(-1e30) + H[:, None])
        dz = p * k
        dz.scatter_add_(1, at, gl[:, None])
        out["dlogits"] = (dz * it).to(z.dtype)
    return out


def _plain_distill(s):
    c, z, it = s["case"], s["z"], 1.0 / s["case"]["temp"]
    w = z.float()
    has, V = (s["t_ids"] >= 0) & (s["t_ids"] < c["V"]), c["V"]
    at = torch.where(has, s["t_ids"], torch.zeros_like(s["t_ids"])).long()
    some = has.any(1)
    zero = torch.zeros((), device=z.device)
    # the list's few terms in 64 bits: the loss is the small difference of the teacher's and the student's logarithms
    t = torch.where(has, s["t_z"].double() * it, torch.full((), -math.inf, dtype=torch.float64, device=z.device))
    if c["tail"]:
        lq = t - s["t_lse"].double()[:, None]
        q = lq.exp()
        qt = torch.where(some, (1.0 - q.sum(1)).clamp_min(0.0), zero.double())
    else:
        tm = torch.where(some, t.amax(1), zero.double())[:, None]
        q = (t - tm).exp()
        Q = torch.where(some, q.sum(1), torch.ones_like(tm[:, 0]))[:, None]
        lq, q = t - tm - Q.log(), q / Q
    d = (w - w.amax(1, keepdim=True)) * it
    e = d.exp()
    Z = e.sum(1, keepdim=True)
    ls = ((w.gather(1, at).double() - w.amax(1, keepdim=True)) * it) - Z.double().log()
    loss = torch.where(q > 0, q * (lq - ls), zero.double()).sum(1)
    if c["tail"]:  # what the list leaves, as one more outcome of both
        inlist = torch.zeros(w.shape, dtype=torch.bool, device=w.device)
        inlist.scatter_(1, torch.where(has, at, at[:, :1]), has | has[:, :1])
        mt = d.masked_fill(inlist, -math.inf).amax(1, keepdim=True)
        Zt = (d - mt).masked_fill(inlist, -math.inf).exp().sum(1, keepdim=True)
        lpt = (Zt.double().log() + mt - Z.double().log())[:, 0]
        loss = loss + torch.where(qt > 0, qt * (qt.log() - lpt), zero.double())
    out = {"loss": torch.where(some, loss, zero.double()).float()}
    if c["do"] != "loss":
        dz = e / Z
        if c["tail"]:
            dz = torch.where(inlist, dz, dz - (d - mt - Zt.log()).exp() * qt.float()[:, None])
        dz.scatter_add_(1, at, -torch.where(has, q, zero.double()).float())
        dz = dz * torch.where(some, s["dloss"] * it, zero)[:, None]
        out["dlogits"] = dz.to(z.dtype)
    return out


def _gate_of_tokens(s, T):
    gt = s["case"]["gate_tokens"]
    return s["gate"].float().repeat_interleave(gt, 0)[:T] if gt else None


def _plain_seam(s):
    c, y = s["case"], s["y"].float()
    T = y.shape[0]
    G = _gate_of_tokens(s, T)
    if c["do"] == "fwd":
        r = y
        if c["post"]:
            r = y * (y.square().mean(1, keepdim=True) + EPS).rsqrt() * s["w_post"]
        if G is not None:
            r = r * G
        h = (s["h"].float() * c["scale"] + r).to(s["h"].dtype)
        w = h.float()
        x = w * (w.square().mean(1, keepdim=True) + EPS).rsqrt() * s["w_pre"]
        return {"h_out": h, "x": x.to(s["x"].dtype)}
    ry, rh = s["rstd"][:, 0:1], s["rstd"][:, 1:2]
    n, dx = s["h_out"].float() * rh, s["dx"].float()
    u = dx * s["w_pre"]
    dt = s["dh_out"].float() + rh * (u - n * (u * n).mean(1, keepdim=True))
    m = y * ry if c["post"] else y
    v = dt if G is None else dt * G
    out = {"dh": (dt * c["scale"]).to(s["dh"].dtype), "dw_pre": (dx * n).sum(0)}
    if G is not None:
        dg = dt * m * s["w_post"] if c["post"] else dt * m
        gt = c["gate_tokens"]
        if gt > 1:
            short = -T % gt
            dg = torch.cat([dg, dg.new_zeros((short, dg.shape[1]))]) if short else dg
            dg = dg.view(-1, gt, dg.shape[1]).sum(1)
        out["dgate"] = dg.to(s["dgate"].dtype)
    if c["post"]:
        out["dw_post"] = (v * m).sum(0)
        v = v * s["w_post"]
        v = ry * (v - m * (v * m).mean(1, keepdim=True))
    out["dy"] = v.to(s["dy"].dtype)
    return out


# ---- the framework's calls ------------------------------------------------------------------------------------------

def _own_logprobs(s):
    from orthogonal_reparameterized_amd import binding as B
    c, it = s["case"], 1.0 / s["case"]["temp"]
    if s["ws"] is None:  # kept by the program for all calls of this size
        n = B.poet_token_logprobs_workspace_bytes(c["T"], c["V"], B.POET_BF16 if c["dtype"] == "bf16" else B.POET_F32, c["K"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    if c["do"] == "bwd":
        B.poet_token_logprobs_bwd(s["z"], s["ids"], s["stats"], s["dlogp"], s["dz"], inv_temp=it, dentropy=s["dH"])
        return {"dlogits": s["dz"]}
    train = {} if c["do"] == "score" else dict(dlogp=s["dlogp"], dentropy=s["dH"], dlogits=s["dz"])
    B.poet_token_logprobs(s["z"], s["ids"], s["logp"], s["stats"], inv_temp=it, entropy=s["H"], top_ids=s["top_ids"],
                          top_logp=s["top_logp"], ws=s["ws"], **train)
    out = {"logp": s["logp"]}
    if c["entropy"]:
        out["entropy"] = s["H"]
    if c["K"]:
        out["top_ids"], out["top_logp"] = s["top_ids"], s["top_logp"]
    if train:
        out["dlogits"] = s["dz"]
    return out


def _own_distill(s):
    from orthogonal_reparameterized_amd import binding as B
    c, it = s["case"], 1.0 / s["case"]["temp"]
    if s["ws"] is None:
        n = B.poet_distill_workspace_bytes(c["T"], c["V"], B.POET_BF16 if c["dtype"] == "bf16" else B.POET_F32)
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    train = {} if c["do"] == "loss" else dict(dloss=s["dloss"], dlogits=s["dz"])
    B.poet_distill(s["z"], s["t_ids"], s["t_z"], s["loss"], s["stats"],
                   mode=B.POET_DISTILL_TAIL if c["tail"] else B.POET_DISTILL_RENORM, inv_temp=it, t_inv_temp=it,
                   t_lse=s["t_lse"], ws=s["ws"], **train)
    return {"loss": s["loss"], "dlogits": s["dz"]} if train else {"loss": s["loss"]}


def _own_seam(s):
    from orthogonal_reparameterized_amd import binding as B
    c = s["case"]
    if c["do"] == "fwd":
        B.poet_block_norm_fwd(s["h"], s["rstd"], y=s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
                              h_out=s["h_out"], x=s["x"], res_scale=c["scale"], eps=EPS, gate_tokens=c["gate_tokens"] or 1)
        return {"h_out": s["h_out"], "x": s["x"]}
    if s["ws"] is None:
        n = B.poet_block_norm_workspace_bytes(c["T"], c["d"], c["gate_tokens"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    B.poet_block_norm_bwd(s["h_out"], s["rstd"], y=s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
                          dh_out=s["dh_out"], dx=s["dx"], dh=s["dh"], dy=s["dy"], dgate=s["dgate"],
                          dw_post=s["dw_post"], dw_pre=s["dw_pre"], res_scale=c["scale"],
                          gate_tokens=c["gate_tokens"] or 1, ws=s["ws"])
    return {k: s[k] for k in ("dh", "dw_pre", "dgate", "dw_post", "dy") if s[k] is not None}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"logprobs": _own_logprobs, "distill": _own_distill, "seam": _own_seam}[op](state)
    return {"logprobs": _plain_logprobs, "distill": _plain_distill, "seam": _plain_seam}[op](state)


# ---- the work of one pass -------------------------------------------------------------------------------------------

def work(case):
    c, T = case, case["T"]
    size = lambda n: 2 if n == "bf16" else 4  # noqa: E731
    if c["op"] == "seam":
        d, r, a = c["d"], size(c["res"]), size(c["act"])
        rows = -(-T // c["gate_tokens"]) if c["gate_tokens"] else 0
        if c["do"] == "fwd":  # h, y, gate in; h_out, x out
            return {"bytes": T * d * (2 * r + 2 * a) + rows * d * a + 8 * d + 8 * T, "flops": 10 * T * d}
        # h_out, dh_out, y, dx, gate in; dh, dy, dgate out
        return {"bytes": T * d * (3 * r + 3 * a) + 2 * rows * d * a + 16 * d + 8 * T, "flops": 25 * T * d}
    V, e = c["V"], size(c["dtype"])
    grad = c["do"] in ("train", "bwd")
    n = T * V * e * (2 if grad else 1) + 24 * T
    f = T * V * (9 if grad else 6)
    return {"bytes": n + 8 * T * c["K"], "flops": f}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------

def _exact_logprobs(c, s):
    V, T = c["V"], c["T"]
    parts = []
    for lo in range(0, T, max(1, 60_000_000 // V)):  # some rows at a time
        hi = min(T, lo + max(1, 60_000_000 // V))
        a = s["z"][lo:hi].double() / c["temp"]
        lse = torch.logsumexp(a, 1, keepdim=True)
        lp = a - lse
        p = torch.exp(lp)
        ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
        ids = s["ids"][lo:hi].tolist()
        rows = [i for i, j in enumerate(ids) if 0 <= j < V]
        cols = [ids[i] for i in rows]
        o = {}
        if c["do"] != "bwd":
            got = torch.zeros(hi - lo, dtype=torch.float64, device=DEV)
            got[rows] = lp[rows, cols]
            o["logp"] = got
            if c["entropy"]:
                o["entropy"] = ent
        if c["K"]:
            order = torch.sort(s["z"][lo:hi].double(), dim=1, descending=True, stable=True).indices[:, :c["K"]]
            o["top_ids"], o["top_logp"] = order.to(torch.int32), torch.take_along_dim(lp, order, 1)
        if c["do"] != "score":
            gl = torch.zeros(hi - lo, dtype=torch.float64, device=DEV)
            gl[rows] = s["dlogp"][lo:hi].double()[rows]
            dz = -gl[:, None] * p
            dz[rows, cols] += gl[rows]
            if c["entropy"]:
                dz -= s["dH"][lo:hi].double()[:, None] * torch.where(p > 0, p * (lp + ent[:, None]), torch.zeros_like(p))
            o["dlogits"] = dz / c["temp"]
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def _exact_distill(c, s):
    V, T = c["V"], c["T"]
    parts = []
    for lo in range(0, T, max(1, 60_000_000 // V)):
        hi = min(T, lo + max(1, 60_000_000 // V))
        a = torch.log_softmax(s["z"][lo:hi].double() / c["temp"], 1)
        ids = s["t_ids"][lo:hi].long()
        ok = (ids >= 0) & (ids < V)
        tv = torch.where(ok, s["t_z"][lo:hi].double() / c["temp"], torch.full((), -math.inf, dtype=torch.float64, device=DEV))
        lse = s["t_lse"][lo:hi].double() if c["tail"] else torch.logsumexp(tv, 1)
        lq = torch.where(ok, tv - lse[:, None], torch.full_like(tv, -math.inf))
        q = torch.exp(lq)
        full = torch.zeros((hi - lo, V + 1), dtype=torch.float64, device=DEV)  # the teacher over all tokens; last: no token
        full.scatter_add_(1, torch.where(ok, ids, torch.full_like(ids, V)), q)
        listed_ = torch.zeros((hi - lo, V + 1), dtype=torch.bool, device=DEV)
        listed_.scatter_(1, torch.where(ok, ids, torch.full_like(ids, V)), True)
        full, listed_ = full[:, :V], listed_[:, :V]
        la = torch.gather(a, 1, ids.clamp(0, V - 1))
        loss = torch.where(q > 0, q * (lq - la), torch.zeros_like(q)).sum(1)
        g = torch.exp(a) - full
        some = ok.any(1)
        if c["tail"]:
            rest = torch.logsumexp(a.masked_fill(listed_, -math.inf), 1)
            qr = (1.0 - q.sum(1)).clamp_min(0.0)
            loss = loss + torch.where(qr > 0, qr * (torch.log(qr) - rest), torch.zeros_like(qr))
            g = torch.where(listed_, g, torch.exp(a) - qr[:, None] * torch.exp(a - rest[:, None]))
        o = {"loss": torch.where(some, loss, torch.zeros_like(loss))}
        if c["do"] != "loss":
            o["dlogits"] = torch.where(some[:, None], g * (s["dloss"][lo:hi].double()[:, None] / c["temp"]), torch.zeros_like(g))
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def _exact_seam(c, s):
    T, d = c["T"], c["d"]
    token_gate = torch.arange(T, device=DEV) // c["gate_tokens"] if c["gate_tokens"] else None
    gate = torch.ones((1, d), dtype=torch.float64, device=DEV) if token_gate is None else s["gate"].double()[token_gate]
    wp = s["w_post"].double() if c["post"] else torch.ones(d, dtype=torch.float64, device=DEV)
    y = s["y"].double()
    ry = 1.0 / torch.sqrt((y * y).sum(1, keepdim=True) / d + EPS) if c["post"] else torch.ones((T, 1), dtype=torch.float64, device=DEV)
    if c["do"] == "fwd":
        h = c["scale"] * s["h"].double() + gate * wp * (ry * y)
        hr = h.to(s["h"].dtype).double()  # the norm reads the residual stream as it is kept
        return {"h_out": h, "x": s["w_pre"].double() * hr / torch.sqrt((hr * hr).sum(1, keepdim=True) / d + EPS)}
    h, dx, w = s["h_out"].double(), s["dx"].double(), s["w_pre"].double()
    rh = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / d + EPS)
    dh = s["dh_out"].double() + rh * dx * w - h * rh ** 3 * (dx * w * h).sum(1, keepdim=True) / d
    e = dh * gate * wp
    o = {"dh": c["scale"] * dh, "dw_pre": (dx * h * rh).sum(0)}
    if c["post"]:
        o["dw_post"] = (dh * gate * y * ry).sum(0)
        o["dy"] = ry * e - y * ry ** 3 * (e * y).sum(1, keepdim=True) / d
    else:
        o["dy"] = e
    if token_gate is not None:
        o["dgate"] = torch.zeros(s["gate"].shape, dtype=torch.float64, device=DEV).index_add_(0, token_gate, dh * wp * (ry * y))
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "distill": _exact_distill, "seam": _exact_seam}[case["op"]](case, s)

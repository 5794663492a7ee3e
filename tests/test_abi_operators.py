"""Host-only checks of the operators on rows of logits and of the block norm seam: workspace sizes, and every invalid
argument refused with its status before anything is launched (no GPU needed); the binding's own refusals of tensors."""
import ctypes

import pytest

from orthogonal_reparameterized_amd import binding as B

torch = pytest.importorskip("torch")
BIG = 1 << 40


def ptr(k):
    """Never dereferenced addresses, 2^40 bytes apart: every call below fails validation first."""
    return ctypes.c_void_p(0x10000000 + k * BIG)


Z, D, IDS, LP, ST, TI, TL, GL, H, WS = (ptr(k) for k in range(1, 11))


def _logits(**over):
    kw = dict(T=7, V=1000, ld=1008, dtype=B.POET_BF16, inv_temp=1.0)
    kw.update(over)
    return B.poet_logits(**kw)


def _fwd(L=None, z=Z, ids=IDS, K=0, dlogp=None, dent=None, logp=LP, ent=H, ti=None, tl=None, st=ST, dz=None, ldd=1008):
    return B.lib().poet_token_logprobs(ctypes.byref(L or _logits()), z, ids, K, dlogp, dent, logp, ent, ti, tl, st, dz, ldd,
                                       None, 0, None)


def _bwd(L=None, z=Z, ids=IDS, st=ST, dlogp=GL, dent=None, dz=D, ldd=1008):
    return B.lib().poet_token_logprobs_bwd(ctypes.byref(L or _logits()), z, ids, st, dlogp, dent, dz, ldd, None)


def _dis(L=None, K=5, mode=0, tit=1.0, z=Z, ti=TI, tz=TL, lse=None, w=None, loss=LP, st=ST, dz=None, ldd=1008):
    t = B.poet_teacher(K, mode, tit)
    return B.lib().poet_distill(ctypes.byref(L or _logits()), ctypes.byref(t), z, ti, tz, lse, w, loss, st, dz, ldd, None, 0,
                                None)


def _dis_bwd(L=None, K=5, mode=0, tit=1.0, z=Z, ti=TI, tz=TL, lse=None, st=ST, w=GL, dz=D, ldd=1008):
    t = B.poet_teacher(K, mode, tit)
    return B.lib().poet_distill_bwd(ctypes.byref(L or _logits()), ctypes.byref(t), z, ti, tz, lse, st, w, dz, ldd, None)


BAD_LOGITS = [(dict(T=-1), B.POET_E_SHAPE), (dict(V=0), B.POET_E_SHAPE), (dict(ld=999), B.POET_E_SHAPE),
              (dict(V=B.POET_MAX_VOCAB + 1, ld=1 << 25), B.POET_E_UNSUPPORTED), (dict(ld=1 << 47), B.POET_E_UNSUPPORTED),
              (dict(dtype=2), B.POET_E_DTYPE), (dict(inv_temp=0.0), B.POET_E_ARG), (dict(inv_temp=-1.0), B.POET_E_ARG),
              (dict(inv_temp=float("nan")), B.POET_E_ARG), (dict(inv_temp=float("inf")), B.POET_E_ARG),
              (dict(inv_temp=2e30), B.POET_E_ARG), (dict(inv_temp=5e-31), B.POET_E_ARG)]


@pytest.mark.parametrize("over,status", BAD_LOGITS)
def test_bad_logits_are_refused(over, status):
    L = _logits(**over)
    for st in (_fwd(L), _bwd(L), _dis(L), _dis_bwd(L)):
        assert st == status
        assert B.poet_last_error() != ""


def test_null_descriptions():
    assert B.lib().poet_token_logprobs(None, Z, IDS, 0, None, None, LP, None, None, None, ST, None, 0, None, 0, None) == B.POET_E_ARG
    assert B.lib().poet_distill(ctypes.byref(_logits()), None, Z, TI, TL, None, None, LP, ST, None, 0, None, 0, None) == B.POET_E_ARG
    assert B.lib().poet_block_norm_fwd(None, Z, None, None, None, GL, None, D, ST, None) == B.POET_E_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(K=-1), B.POET_E_SHAPE), (dict(K=129, ti=TI, tl=TL), B.POET_E_SHAPE), (dict(K=3), B.POET_E_ARG),
    (dict(K=3, ti=TI), B.POET_E_ARG), (dict(ti=TI, tl=TL), B.POET_E_ARG), (dict(z=None), B.POET_E_ARG),
    (dict(st=None), B.POET_E_ARG), (dict(ids=None), B.POET_E_ARG), (dict(dz=D), B.POET_E_ARG), (dict(dlogp=GL), B.POET_E_ARG),
    (dict(dent=GL), B.POET_E_ARG), (dict(dlogp=GL, dz=D, ids=None, logp=None), B.POET_E_ARG),
    (dict(dlogp=GL, dz=D, ldd=999), B.POET_E_SHAPE), (dict(z=ctypes.c_void_p(Z.value + 1)), B.POET_E_ARG),
    (dict(dlogp=GL, dz=ctypes.c_void_p(D.value + 1)), B.POET_E_ARG),
    (dict(dlogp=GL, dz=Z, ldd=1009), B.POET_E_ARG), (dict(dlogp=GL, dz=ctypes.c_void_p(Z.value + 2)), B.POET_E_ARG),
    (dict(dlogp=GL, dz=ctypes.c_void_p(Z.value + 2 * 6 * 1008)), B.POET_E_ARG)])
def test_logprobs_refusals(kw, status):
    assert _fwd(**kw) == status
    assert B.poet_last_error() != ""


def test_more_alternatives_than_tokens():
    assert _fwd(_logits(V=4, ld=4), K=5, ti=TI, tl=TL, ldd=4) == B.POET_E_SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), B.POET_E_ARG), (dict(ids=None), B.POET_E_ARG), (dict(st=None), B.POET_E_ARG),
    (dict(dlogp=None), B.POET_E_ARG), (dict(dz=None), B.POET_E_ARG), (dict(ldd=1), B.POET_E_SHAPE),
    (dict(dz=Z, ldd=2000), B.POET_E_ARG)])
def test_logprobs_bwd_refusals(kw, status):
    assert _bwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), B.POET_E_SHAPE), (dict(K=129), B.POET_E_SHAPE), (dict(mode=2), B.POET_E_ARG), (dict(tit=0.0), B.POET_E_ARG),
    (dict(tit=float("nan")), B.POET_E_ARG), (dict(lse=GL), B.POET_E_ARG), (dict(z=None), B.POET_E_ARG),
    (dict(ti=None), B.POET_E_ARG), (dict(tz=None), B.POET_E_ARG), (dict(st=None), B.POET_E_ARG)])
def test_distill_refusals(kw, status):
    assert _dis(**kw) == status
    assert _dis_bwd(**kw) == status


def test_distill_gradient_refusals():
    assert _dis(loss=None) == B.POET_E_ARG
    assert _dis(w=GL) == B.POET_E_ARG and _dis(dz=D) == B.POET_E_ARG
    assert _dis(w=GL, dz=ctypes.c_void_p(Z.value + 4)) == B.POET_E_ARG
    assert _dis_bwd(w=None) == B.POET_E_ARG and _dis_bwd(dz=None) == B.POET_E_ARG


def test_workspace_sizes():
    lib = B.lib()
    for T, V, dt, K in ((1, 1, 0, 1), (16384, 32000, 1, 20), (1, B.POET_MAX_VOCAB, 0, 128), (0, 5, 0, 0)):
        assert lib.poet_token_logprobs_workspace_bytes(T, V, dt, K) < (1 << 36)
        assert lib.poet_distill_workspace_bytes(T, V, dt) < (1 << 36)
    assert lib.poet_token_logprobs_workspace_bytes(-1, 5, 0, 0) == 0 and B.poet_last_error() != ""
    assert lib.poet_token_logprobs_workspace_bytes(1, 5, 0, 6) == 0 and B.poet_last_error() != ""
    assert lib.poet_block_norm_workspace_bytes(0, 5, 0) == 0
    assert lib.poet_block_norm_workspace_bytes(5, 0, 0) == 0 and B.poet_last_error() != ""
    assert lib.poet_block_norm_workspace_bytes(5, B.POET_MAX_NORM + 1, 0) == 0
    assert lib.poet_block_norm_workspace_bytes(5, 8, -1) == 0
    for T, d, g in ((1, 1, 0), (32768, 2560, 512), (7, B.POET_MAX_NORM, 1), (100000, 64, 3)):
        assert 0 < lib.poet_block_norm_workspace_bytes(T, d, g) < (1 << 32)


def _norm(**over):
    kw = dict(T=6, d=100, ldh=104, ldy=104, ldg=104, ldx=104, res_dtype=0, act_dtype=1, gate_tokens=2, res_scale=1.0, eps=1e-6)
    kw.update(over)
    return B.poet_norm(**kw)


N_H, N_Y, N_G, N_WQ, N_WP, N_HO, N_X, N_R, N_DH, N_DY, N_DG, N_DQ, N_DP, N_DHO, N_DX = (ptr(k) for k in range(20, 35))


def _nf(N=None, **over):
    a = dict(h=N_H, y=N_Y, gate=N_G, w_post=N_WQ, w_pre=N_WP, h_out=N_HO, x=N_X, rstd=N_R)
    a.update(over)
    return B.lib().poet_block_norm_fwd(ctypes.byref(N or _norm()), *a.values(), None)


def _nb(N=None, ws_bytes=BIG, **over):
    a = dict(h_out=N_HO, y=N_Y, gate=N_G, w_post=N_WQ, w_pre=N_WP, rstd=N_R, dh_out=N_DHO, dx=N_DX, dh=N_DH, dy=N_DY,
             dgate=N_DG, dw_post=N_DQ, dw_pre=N_DP)
    a.update(over)
    return B.lib().poet_block_norm_bwd(ctypes.byref(N or _norm()), *a.values(), WS, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), B.POET_E_SHAPE), (dict(d=0), B.POET_E_SHAPE), (dict(d=16385, ldh=20000), B.POET_E_UNSUPPORTED),
    (dict(ldh=99), B.POET_E_SHAPE), (dict(ldy=99), B.POET_E_SHAPE), (dict(ldg=0), B.POET_E_SHAPE), (dict(ldx=1), B.POET_E_SHAPE),
    (dict(ldh=1 << 47), B.POET_E_SHAPE), (dict(res_dtype=2), B.POET_E_DTYPE), (dict(act_dtype=-1), B.POET_E_DTYPE),
    (dict(gate_tokens=0), B.POET_E_SHAPE), (dict(eps=0.0), B.POET_E_ARG), (dict(eps=float("nan")), B.POET_E_ARG),
    (dict(res_scale=float("inf")), B.POET_E_ARG)])
def test_bad_norms_are_refused(over, status):
    assert _nf(_norm(**over)) == status
    assert _nb(_norm(**over)) == status
    assert B.poet_last_error() != ""


@pytest.mark.parametrize("over", [
    dict(h=None), dict(rstd=None), dict(h_out=None), dict(y=None), dict(w_pre=None), dict(x=None),
    dict(y=None, gate=None, w_post=None), dict(y=None, gate=None, w_post=None, h_out=None, w_pre=None, x=None),
    dict(x=N_Y), dict(x=N_G), dict(h_out=N_Y), dict(x=N_HO), dict(h_out=ctypes.c_void_p(N_H.value + 4)),
    dict(x=ctypes.c_void_p(N_X.value + 1))])
def test_norm_forward_refusals(over):
    assert _nf(**over) == B.POET_E_ARG


@pytest.mark.parametrize("over", [
    dict(w_post=None), dict(dw_post=None), dict(w_pre=None), dict(dw_pre=None), dict(dx=None), dict(dgate=None),
    dict(gate=None), dict(y=None), dict(dy=None), dict(dh=None), dict(rstd=None), dict(h_out=None),
    dict(dh_out=None, dx=None, w_pre=None, dw_pre=None), dict(dy=N_Y), dict(dy=N_DX), dict(dh=N_HO), dict(dgate=N_G),
    dict(dy=N_DG), dict(dh=N_DX), dict(dh=ctypes.c_void_p(N_DHO.value + 4))])
def test_norm_backward_refusals(over):
    assert _nb(**over) == B.POET_E_ARG


def test_norm_backward_workspace():
    assert _nb(ws_bytes=16) == B.POET_E_WORKSPACE


def test_binding_refuses_tensors_off_the_gpu_and_of_other_types():
    z, i, v, st = torch.zeros((3, 8)), torch.zeros(3, dtype=torch.int32), torch.zeros(3), torch.zeros((3, 4))
    with pytest.raises(ValueError, match="GPU"):
        B.poet_token_logprobs(z, i, v, st)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        B.poet_token_logprobs(z.half(), i, v, st)
    with pytest.raises(ValueError, match="2-D"):
        B.poet_token_logprobs(v, i, v, st)
    with pytest.raises(ValueError, match="GPU"):
        B.poet_distill(z, torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)), v, st)
    with pytest.raises(ValueError, match="GPU"):
        B.poet_block_norm_fwd(z, st, w_pre=torch.zeros(8), x=z)
    with pytest.raises(ValueError, match="nothing to compute"):
        B.poet_block_norm_fwd(z, st)
    with pytest.raises(ValueError, match="gate_tokens"):
        B.poet_block_norm_fwd(z, st, y=z, gate=z, gate_tokens=0)
    with pytest.raises(ValueError, match="dh must"):
        B.poet_block_norm_bwd(z, st)

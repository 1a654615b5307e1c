"""Refusals of the training-step operators, on the host and before any launch (no GPU)."""
import ctypes

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
from moe_expert_ffn_top_gb300 import _build

FAKE = 1 << 20  # aligned, never dereferenced: every call below is rejected before any CUDA work


@pytest.fixture(scope="module")
def L():
    _build.build()
    return m.lib()


def _norm(**kw):
    a = dict(rows=8, ldx=0, ldy=0, lddx=0, lddres=0, n=64, dtype=1, wdtype=0, eps=1e-5)
    a.update(kw)
    return m.Norm(*(a[n] for n, _ in m.Norm._fields_))


@pytest.mark.parametrize("code,norm,over", [
    (-5, dict(dtype=3), {}), (-5, dict(wdtype=-1), {}), (-2, dict(rows=-1), {}), (-2, dict(n=0), {}),
    (-2, dict(n=(1 << 24) + 1), {}), (-2, dict(ldx=63), {}), (-2, dict(ldy=-64), {}), (-2, dict(eps=0.0), {}),
    (-2, dict(eps=float("nan")), {}), (-1, {}, dict(x=None)), (-1, {}, dict(y=None)), (-1, {}, dict(rstd=None)),
    (-3, {}, dict(x=FAKE + 8)), (-3, {}, dict(gamma=FAKE + 2)), (-3, {}, dict(beta=FAKE + 4)),
    (-3, {}, dict(mean=FAKE + 4))])
def test_norm_forward_rejections(L, code, norm, over):
    a = dict(x=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, mean=FAKE, rstd=FAKE)
    a.update(over)
    assert L.moe_lora_layernorm_forward(_norm(**norm), a["x"], a["gamma"], a["beta"], a["y"], a["mean"], a["rstd"],
                                        None) == code


@pytest.mark.parametrize("code,norm,over", [
    (-5, dict(dtype=7), {}), (-2, dict(lddx=10), {}), (-2, dict(lddres=63), {}), (-1, {}, dict(mean=None)),
    (-1, {}, dict(rstd=None)), (-1, {}, dict(dx=None)), (-1, {}, dict(dy=None)), (-1, {}, dict(scratch=None)),
    (-3, {}, dict(scratch=FAKE + 8)), (-3, {}, dict(dres=FAKE + 2)), (-3, {}, dict(dgamma=FAKE + 4)),
    (-4, {}, dict(bytes=64))])
def test_norm_backward_rejections(L, code, norm, over):
    a = dict(x=FAKE, gamma=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, dres=FAKE, dx=FAKE, dgamma=FAKE, dbeta=FAKE,
             scratch=FAKE, bytes=1 << 40)
    a.update(over)
    assert L.moe_lora_layernorm_backward(_norm(**norm), *(a[n] for n in ("x", "gamma", "mean", "rstd", "dy", "dres",
                                                                         "dx", "dgamma", "dbeta", "scratch", "bytes")),
                                         None) == code


def test_norm_backward_of_wide_rows_needs_scratch(L):
    """Beyond 8,192 columns also without weight gradients."""
    for n, code in ((8192, None), (8193, -1)):
        nm = _norm(n=n)
        rc = L.moe_lora_layernorm_backward(nm, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, None, None, None, 0, None)
        assert rc == -1  # mean is NULL in both
        if code:
            assert L.moe_lora_layernorm_backward(nm, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, None, None, 0,
                                                 None) == code
            assert L.moe_lora_layernorm_backward(nm, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, None, FAKE, 64,
                                                 None) == -4


def test_norm_scratch_sizes(L):
    assert L.moe_lora_layernorm_scratch_bytes(_norm()) >= 8 * 64
    assert L.moe_lora_layernorm_scratch_bytes(_norm(n=0)) == 0
    assert L.moe_lora_layernorm_scratch_bytes(None) == 0


def _dims(**kw):
    a = dict(T=256, H=64, I=64, E=16, k=2, r=8)
    a.update(kw)
    return m.make_dims(**a)


@pytest.mark.parametrize("code,dims,over", [
    (-2, dict(k=0), {}), (-5, dict(E=1025), {}), (-5, {}, dict(dtype=3)), (-2, {}, dict(ld=15)), (-2, {}, dict(ld=-1)),
    (-1, {}, dict(logits=None)), (-1, {}, dict(ids=None)), (-1, {}, dict(loss=None)), (-1, {}, dict(counts=None)),
    (-1, {}, dict(prob=None)), (-1, {}, dict(scratch=None)), (-3, {}, dict(logits=FAKE + 4)),
    (-3, {}, dict(dlogits=FAKE + 4)), (-3, {}, dict(dloss=FAKE + 4)), (-4, {}, dict(bytes=16)),
    (-1, dict(A=2), {}), (-2, dict(A=2), dict(offs=(0, 100, 256))), (-2, dict(A=2), dict(offs=(0, 128, 200)))])
def test_balance_rejections(L, code, dims, over):
    a = dict(logits=FAKE, dtype=0, ld=0, ids=FAKE, offs=None, dloss=FAKE, loss=FAKE, counts=FAKE, prob=FAKE,
             dlogits=FAKE, scratch=FAKE, bytes=1 << 40)
    a.update(over)
    offs = None if a["offs"] is None else (ctypes.c_int64 * 3)(*a["offs"])
    assert L.moe_lora_balance_loss(_dims(**dims), a["logits"], a["dtype"], a["ld"], a["ids"], offs, 0.01, a["dloss"],
                                   a["loss"], a["counts"], a["prob"], a["dlogits"], a["scratch"], a["bytes"],
                                   None) == code


def test_balance_scratch_sizes(L):
    assert m.moe_lora_workspace_bytes(_dims(), m.MOE_LORA_WS_BALANCE_SCRATCH) > 0
    assert m.moe_lora_workspace_bytes(_dims(E=1025), m.MOE_LORA_WS_BALANCE_SCRATCH) == 0


def test_router_backward_aux_rejections(L):
    d = _dims()
    call = lambda aux, dw: L.moe_lora_router_backward_aux(d, FAKE, FAKE, None, FAKE, FAKE, dw, aux, None, FAKE, FAKE,  # noqa: E731
                                                          FAKE, 1 << 40, None)
    assert call(FAKE + 4, FAKE) == -3
    assert call(FAKE, None) == -1


def _tensor(**kw):
    t = m.AdamWTensor(p=FAKE, master=FAKE, g=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, numel=100, p_dtype=1,
                      g_dtype=0, state=1, lr=1e-3, weight_decay=0.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("code,opt,over", [
    (-2, dict(step=0), {}), (-2, dict(beta1=1.0), {}), (-2, dict(beta2=-0.1), {}), (-2, dict(eps=0.0), {}),
    (-2, dict(eps=float("nan")), {}), (-2, dict(eps=1e-60), {}), (-2, dict(eps=1e-39), {}), (-3, dict(grad_scale=FAKE + 2), {}), (-2, {}, dict(numel=-1)),
    (-5, {}, dict(p_dtype=4)), (-5, {}, dict(g_dtype=-1)), (-5, {}, dict(state=2)), (-5, {}, dict(p_dtype=0)),
    (-2, {}, dict(lr=float("nan"))), (-2, {}, dict(weight_decay=float("inf"))), (-1, {}, dict(p=None)),
    (-1, {}, dict(g=None)), (-1, {}, dict(m=None)), (-1, {}, dict(v=None)), (-1, {}, dict(m_scale=None)),
    (-1, {}, dict(v_scale=None)), (-3, {}, dict(p=FAKE + 2)), (-3, {}, dict(master=FAKE + 4)),
    (-3, {}, dict(g=FAKE + 8)), (-3, {}, dict(m=FAKE + 1)), (-3, {}, dict(v_scale=FAKE + 2)), (-3, {}, dict(m_scale=FAKE + 1))])
def test_adamw_rejections(L, code, opt, over):
    o = dict(beta1=0.9, beta2=0.999, eps=1e-8, step=1, grad_scale=None)
    o.update(opt)
    table = (m.AdamWTensor * 2)(_tensor(), _tensor(**over))  # a bad tensor anywhere refuses the whole call
    assert L.moe_lora_adamw_step(m.AdamW(*(o[n] for n, _ in m.AdamW._fields_)), table, 2, None) == code


def test_adamw_null_and_negative(L):
    o = m.AdamW(0.9, 0.999, 1e-8, 1, None)
    assert L.moe_lora_adamw_step(None, None, 0, None) == -1
    assert L.moe_lora_adamw_step(o, None, 1, None) == -1
    assert L.moe_lora_adamw_step(o, None, -1, None) == -2


def test_binding_rejections():
    """What the binding alone can see: host tensors, shapes, types and layouts."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora_layernorm_forward(x, None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        m.AdamWTensors([dict(p=x, g=x, m=x, v=x)])
    with pytest.raises(ValueError, match="elements"):
        m._vec(x, 31, "g")
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        m._dtype(x.double(), "x")
    with pytest.raises(ValueError, match="come together"):
        m.AdamWTensors([dict(p=x, g=x, m=x, v=x, m_scale=x)])

"""Refusals of the post-training operators, on the host and before any launch (no GPU)."""
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


def _struct(cls, base, kw):
    a = dict(base)
    a.update(kw)
    return cls(*(a[n] for n, _ in cls._fields_))


def _rows(**kw):
    return _struct(m.Rows, dict(rows=8, ld=0, ldd=0, n=100, dtype=1, inv_temp=1.0), kw)


BAD_ROWS = [(-5, dict(dtype=3)), (-5, dict(dtype=-1)), (-2, dict(rows=-1)), (-2, dict(rows=(1 << 26) + 1)), (-2, dict(n=0)),
            (-5, dict(n=(1 << 19) + 1)), (-2, dict(ld=99)), (-2, dict(ldd=99)), (-2, dict(ld=-100)), (-2, dict(inv_temp=0.0)),
            (-2, dict(inv_temp=-1.0)), (-2, dict(inv_temp=float("nan"))), (-2, dict(inv_temp=float("inf")))]


def _forward(L, rows=(), **over):
    a = dict(logits=FAKE, targets=FAKE, logp=FAKE, lse=FAKE, entropy=FAKE, err=None)
    a.update(over)
    return L.moe_lora_token_logp_forward(_rows(**dict(rows)), *a.values(), None)


@pytest.mark.parametrize("code,rows,over", [(c, r, {}) for c, r in BAD_ROWS] + [
    (-1, {}, dict(logits=None)), (-1, {}, dict(targets=None)), (-1, {}, dict(logp=None, lse=None, entropy=None)),
    (-3, {}, dict(logits=FAKE + 8)), (-3, {}, dict(targets=FAKE + 4)), (-3, {}, dict(logp=FAKE + 4)), (-3, {}, dict(lse=FAKE + 8)),
    (-3, {}, dict(entropy=FAKE + 2)), (-3, {}, dict(err=FAKE + 2))])
def test_token_logp_rejections(L, code, rows, over):
    assert _forward(L, rows, **over) == code


def test_no_rows_is_a_no_op(L):
    assert _forward(L, dict(rows=0), logits=None, targets=None) == 0
    assert L.moe_lora_token_logp_backward(_rows(rows=0), None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("code,rows,over", [(c, r, {}) for c, r in BAD_ROWS] + [
    (-1, {}, dict(logits=None)), (-1, {}, dict(targets=None)), (-1, {}, dict(lse=None)), (-1, {}, dict(dlogp=None)),
    (-1, {}, dict(dlogits=None)), (-3, {}, dict(dlogits=FAKE + 2)), (-3, {}, dict(dlogp=FAKE + 4)), (-3, {}, dict(err=FAKE + 1))])
def test_token_logp_backward_rejections(L, code, rows, over):
    a = dict(logits=FAKE, targets=FAKE, lse=FAKE, dlogp=FAKE, dlogits=2 * FAKE, err=None)
    a.update(over)
    assert L.moe_lora_token_logp_backward(_rows(**rows), *a.values(), None) == code


def _policy(L, rows=(), opt=(), offs=None, **over):
    a = dict(logits=FAKE, targets=FAKE, adv=FAKE, old=FAKE, ref=FAKE, weight=FAKE, offs=offs, dloss=FAKE, loss=FAKE, stats=FAKE,
             logp=FAKE, dlogits=2 * FAKE, err=None, scratch=FAKE, bytes=1 << 40)
    if offs is not None:
        a["offs"] = (ctypes.c_int64 * len(offs))(*offs)
    a.update(over)
    o = _struct(m.Policy, dict(clip_low=0.2, clip_high=0.2, kl_coef=0.1, adapters=1), dict(opt))
    return L.moe_lora_policy_loss(_rows(**dict(rows)), o, *a.values(), None)


@pytest.mark.parametrize("code,rows,kw", [(c, r, {}) for c, r in BAD_ROWS] + [
    (-2, {}, dict(opt=dict(clip_low=-0.1))), (-2, {}, dict(opt=dict(clip_low=1.5))), (-2, {}, dict(opt=dict(clip_high=-0.1))),
    (-2, {}, dict(opt=dict(clip_high=float("inf")))), (-2, {}, dict(opt=dict(kl_coef=float("nan")))), (-2, {}, dict(opt=dict(adapters=0))),
    (-2, {}, dict(opt=dict(adapters=65))), (-1, {}, dict(opt=dict(adapters=2))), (-2, {}, dict(opt=dict(adapters=2), offs=(0, 9, 8))),
    (-2, {}, dict(opt=dict(adapters=2), offs=(1, 4, 8))), (-2, {}, dict(opt=dict(adapters=2), offs=(0, 4, 7))),
    (-2, {}, dict(opt=dict(adapters=3), offs=(0, 5, 4, 8))), (-1, {}, dict(logits=None)), (-1, {}, dict(targets=None)), (-1, {}, dict(adv=None)),
    (-1, {}, dict(old=None)), (-1, {}, dict(loss=None)), (-1, {}, dict(stats=None)), (-1, {}, dict(scratch=None)),
    (-3, {}, dict(ref=FAKE + 4)), (-3, {}, dict(weight=FAKE + 4)), (-3, {}, dict(dloss=FAKE + 4)), (-3, {}, dict(dlogits=FAKE + 4)),
    (-3, {}, dict(logp=FAKE + 4)), (-3, {}, dict(err=FAKE + 1)), (-4, {}, dict(bytes=64))])
def test_policy_rejections(L, code, rows, kw):
    assert _policy(L, rows, **kw) == code


def test_gradient_in_place_of_the_logits_needs_their_stride(L):
    assert _policy(L, dict(ld=104, ldd=112), dlogits=FAKE) == -2
    assert L.moe_lora_token_logp_backward(_rows(ldd=104), FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == -2


def _pref(L, opt=(), offs=None, **over):
    a = dict(logp=FAKE, targets=FAKE, seq=FAKE, ref=FAKE, offs=offs, dloss=FAKE, loss=FAKE, stats=FAKE, seq_logp=FAKE, dlogp=FAKE, err=None,
             scratch=FAKE, bytes=1 << 40)
    if offs is not None:
        a["offs"] = (ctypes.c_int64 * len(offs))(*offs)
    a.update(over)
    o = _struct(m.Preference, dict(tokens=100, pairs=4, beta=0.1, margin=0.0, label_smoothing=0.0, kind=0, average=0, adapters=1), dict(opt))
    return L.moe_lora_preference_loss(o, *a.values(), None)


@pytest.mark.parametrize("code,kw", [
    (-5, dict(opt=dict(kind=3))), (-5, dict(opt=dict(kind=-1))), (-2, dict(opt=dict(tokens=-1))), (-2, dict(opt=dict(pairs=-1))),
    (-2, dict(opt=dict(beta=0.0))), (-2, dict(opt=dict(beta=float("nan")))), (-2, dict(opt=dict(beta=float("inf")))),
    (-2, dict(opt=dict(margin=float("inf")))), (-2, dict(opt=dict(label_smoothing=0.6))), (-2, dict(opt=dict(label_smoothing=-0.1))),
    (-2, dict(opt=dict(adapters=0))), (-1, dict(opt=dict(adapters=2))), (-2, dict(opt=dict(adapters=2), offs=(0, 5, 4))),
    (-2, dict(opt=dict(adapters=2), offs=(0, 2, 3))), (-1, dict(logp=None)), (-1, dict(targets=None)), (-1, dict(seq=None)), (-1, dict(loss=None)),
    (-1, dict(stats=None)), (-1, dict(scratch=None)), (-3, dict(seq=FAKE + 8)), (-3, dict(ref=FAKE + 4)), (-3, dict(dlogp=FAKE + 4)),
    (-3, dict(seq_logp=FAKE + 4)), (-3, dict(dloss=FAKE + 4)), (-3, dict(err=FAKE + 2)), (-4, dict(bytes=16))])
def test_preference_rejections(L, code, kw):
    assert _pref(L, **kw) == code


def test_null_options(L):
    assert L.moe_lora_token_logp_forward(None, FAKE, FAKE, FAKE, None, None, None, None) == -1
    assert L.moe_lora_policy_loss(_rows(), None, *[FAKE] * 14, 1 << 40, None) == -1
    assert L.moe_lora_preference_loss(None, *[FAKE] * 12, 1 << 40, None) == -1


def test_scratch_sizes(L):
    assert L.moe_lora_policy_scratch_bytes(100, 2) >= 5 * 4 * 100
    assert L.moe_lora_policy_scratch_bytes(-1, 1) == 0 and L.moe_lora_policy_scratch_bytes(1, 65) == 0
    assert L.moe_lora_preference_scratch_bytes(0) > 0 and L.moe_lora_preference_scratch_bytes(-1) == 0


def test_binding_rejections():
    """What the binding alone can see."""
    x, t, v = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora_token_logp_forward(x, t, v)
    with pytest.raises(ValueError, match="kind"):
        m.moe_lora_preference_loss(v, t, torch.zeros(3, dtype=torch.int64), None, v, v, x, kind="other")
    with pytest.raises(ValueError, match="2 \\* pairs"):
        m.moe_lora_preference_loss(v, t, torch.zeros(4, dtype=torch.int64), None, v, v, x)
    with pytest.raises(ValueError, match="entries"):
        m._host_offsets([0, 4], 2, "adapter_offsets")


def _muon_tensor(**kw):
    t = m.MuonTensor(p=FAKE, master=FAKE, g=FAKE, m=FAKE, batch=3, rows=64, cols=100, p_dtype=1, g_dtype=0, lr=1e-3, weight_decay=0.0,
                     scale=1.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("code,opt,over", [
    (-5, dict(steps=0), {}), (-5, dict(steps=6), {}), (-2, dict(momentum=1.0), {}), (-2, dict(momentum=-0.1), {}), (-2, dict(eps=0.0), {}),
    (-2, dict(eps=float("nan")), {}), (-2, dict(eps=2.0), {}), (-2, dict(a=9.0), {}), (-2, dict(b=float("nan")), {}), (-2, dict(c=-17.0), {}),
    (-3, dict(grad_scale=FAKE + 2), {}), (-2, {}, dict(batch=-1)), (-2, {}, dict(rows=0)), (-2, {}, dict(cols=0)), (-5, {}, dict(rows=129, cols=129)),
    (-2, {}, dict(batch=1 << 33)), (-2, {}, dict(batch=1 << 30, cols=1 << 30)), (-5, {}, dict(p_dtype=3)), (-5, {}, dict(g_dtype=-1)), (-5, {}, dict(p_dtype=0)),
    (-2, {}, dict(lr=float("nan"))), (-2, {}, dict(weight_decay=float("inf"))), (-2, {}, dict(scale=float("nan"))), (-1, {}, dict(p=None)),
    (-1, {}, dict(g=None)), (-1, {}, dict(m=None)), (-3, {}, dict(p=FAKE + 2)), (-3, {}, dict(master=FAKE + 4)), (-3, {}, dict(g=FAKE + 8)),
    (-3, {}, dict(m=FAKE + 4))])
def test_muon_rejections(L, code, opt, over):
    o = dict(momentum=0.95, eps=1e-7, a=3.4445, b=-4.775, c=2.0315, nesterov=1, steps=5, grad_scale=None)
    table = (m.MuonTensor * 2)(_muon_tensor(), _muon_tensor(**over))  # a bad tensor anywhere refuses the whole call
    assert L.moe_lora_muon_step(_struct(m.Muon, o, opt), table, 2, FAKE, 1 << 50, None) == code


def test_muon_scratch_and_null(L):
    o = m.Muon(0.95, 1e-7, 3.4445, -4.775, 2.0315, 1, 5, None)
    table = (m.MuonTensor * 1)(_muon_tensor())
    need = L.moe_lora_muon_scratch_bytes(table, 1)
    assert need >= 4 * 3 * 64 * 100
    assert L.moe_lora_muon_step(o, table, 1, FAKE, need - 1, None) == -4
    assert L.moe_lora_muon_step(o, table, 1, None, need, None) == -1
    assert L.moe_lora_muon_step(o, table, 1, FAKE + 8, need, None) == -3
    assert L.moe_lora_muon_step(None, table, 1, FAKE, need, None) == -1
    assert L.moe_lora_muon_step(o, None, 1, FAKE, need, None) == -1
    assert L.moe_lora_muon_step(o, None, -1, FAKE, need, None) == -2
    assert L.moe_lora_muon_scratch_bytes(table, -1) == 0 and L.moe_lora_muon_scratch_bytes(None, 1) == 0
    assert L.moe_lora_muon_scratch_bytes((m.MuonTensor * 1)(_muon_tensor(rows=200, cols=200)), 1) == 0
    assert L.moe_lora_muon_get_error(None, None) == -1


def test_muon_binding_rejections():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="two axes"):
        m.MuonTensors([dict(p=torch.zeros(4), g=torch.zeros(4), m=torch.zeros(4))])
    with pytest.raises(ValueError, match="must be \\(4, 8\\)"):
        m.MuonTensors([dict(p=x, g=torch.zeros(8, 4), m=x)])
    with pytest.raises(ValueError, match="CUDA"):
        m.MuonTensors([dict(p=x, g=x, m=x)])

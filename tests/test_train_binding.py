"""What the training calls of the binding pass to the library, without a GPU: the library is replaced by a
recorder of its arguments, so nothing is launched whatever a test passes."""

import ctypes

import pytest
import torch

from segmented_gather_gemm_lora_gb300 import binding as B


class Recorder:
    """Stands for the library: every call succeeds and leaves its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return B.LORA_OK

        return call


@pytest.fixture
def calls(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(B, "lib", lambda: r)
    return r.calls


def rows(T):
    return torch.zeros(T, dtype=torch.int32), torch.zeros(T), torch.zeros(T)


def options(args, kind):
    """The structure of options among a call's arguments, as it is now."""
    for a in args:
        if hasattr(a, "_obj") and isinstance(a._obj, kind):
            return a._obj
    raise AssertionError("no options")


def policy(**kw):
    lab, f, g = rows(4)
    x = torch.zeros(4, 8)
    B.lora_policy_loss(x, lab, f, g, f.clone(), g.clone(), None, None, ref_logp=f, stream=0, **kw)


def preference(**kw):
    lab, f, g = rows(4)
    B.lora_preference_loss(torch.zeros(4, 8), lab, torch.tensor([0, 2, 4], dtype=torch.int32), f[:1], None, None,
                           torch.zeros(64, dtype=torch.uint8), stream=0, **kw)


@pytest.mark.parametrize("name", ["clip_low", "clip_high", "kl_coef", "grad_scale"])
def test_a_policy_option_held_in_a_tensor_is_read_at_each_call(calls, name):
    value = torch.tensor(0.25, dtype=torch.float64)
    for v in (0.25, 0.5, 0.125):
        value.fill_(v)
        policy(**{name: value})
        assert getattr(options(calls[-1][1], B.lora_policy_opts_t), name) == v


@pytest.mark.parametrize("name", ["beta", "label_smoothing", "margin", "grad_scale"])
def test_a_preference_option_held_in_a_tensor_is_read_at_each_call(calls, name):
    value = torch.tensor(0.25)
    for v in (0.25, 0.5, 0.125):
        value.fill_(v)
        preference(**{name: value})
        assert getattr(options(calls[-1][1], B.lora_pref_opts_t), name) == v
    kind = torch.tensor(B.LORA_PREF_HINGE)
    preference(kind=kind)
    kind.fill_(B.LORA_PREF_IPO)
    preference(kind=kind)
    assert options(calls[-1][1], B.lora_pref_opts_t).kind == B.LORA_PREF_IPO


def strided(T, V, stride, dtype=torch.float32):
    return torch.zeros(max(1, (T - 1) * stride + V), dtype=dtype).as_strided((T, V), (stride, 1))


def loss_calls(x, d):
    T = x.shape[0]
    lab, f, g = rows(T)
    ws = torch.zeros(256, dtype=torch.uint8)
    out = [lambda: B.lora_policy_loss(x, lab, f, g, f.clone(), g.clone(), None, d, stream=0),
           lambda: B.lora_preference_loss(x, lab, torch.tensor([0, 1, T], dtype=torch.int32), f[:1], None, d, ws, stream=0)]
    return out + ([lambda: B.lora_token_logprobs(x, lab, f, stream=0)] if d is None else [])


@pytest.mark.parametrize("stride", [0, 1, 8, 15])
def test_rows_closer_than_their_length_are_refused(calls, stride):
    """Broadcast and overlapping rows: their buffer is shorter than T rows of V."""
    for call in loss_calls(strided(4, 16, stride), None) + loss_calls(torch.zeros(4, 16), strided(4, 16, stride)):
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_the_stride_of_rows_reaches_the_library(calls):
    for T, V, stride, ld in [(4, 16, 16, 16), (4, 16, 19, 19), (1, 16, 0, 16), (1, 16, 5, 16), (1, 16, 40, 40), (0, 16, 0, 16), (3, 1, 1, 1)]:
        B.lora_token_logprobs(strided(T, V, stride), *rows(T)[:2], stream=0)
        assert calls[-1][1][1] == ld


def proj_arrays(e4m3=False, n=512):
    """A view's worth of state arrays for TrainProj, by name."""
    a = dict(grad=torch.zeros(n), m=torch.zeros(n), v=torch.zeros(n), master=torch.zeros(n))
    if e4m3:
        a.update(m=torch.zeros(n, dtype=torch.uint8), v=torch.zeros(n, dtype=torch.uint8).view(torch.float8_e4m3fn),
                 m_scale=torch.zeros(n // 64, dtype=torch.bfloat16), v_scale=torch.zeros(n // 64, dtype=torch.bfloat16))
    return a


def view(n=512):
    return B.PoolView(torch.zeros(n // 64, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32),
                      torch.zeros(2, 4, dtype=torch.int32), 64, 4, 64, 64)


@pytest.mark.parametrize("e4m3", [False, True])
def test_state_arrays_of_another_type_are_refused(e4m3):
    good = proj_arrays(e4m3)
    assert B.TrainProj(view(), **good).state == (B.LORA_STATE_E4M3 if e4m3 else B.LORA_STATE_F32)
    assert B.TrainProj(view(), **dict(good, master=None)).c.master is None
    wrong = {"grad": (torch.int32,), "master": (torch.int32,), "m": (torch.int8, torch.float8_e5m2) if e4m3 else (torch.int32,),
             "m_scale": (torch.float16, torch.int16) if e4m3 else ()}
    wrong["v"], wrong["v_scale"] = wrong["m"], wrong["m_scale"]
    for name, types in wrong.items():
        for t in types:
            with pytest.raises(ValueError, match=name):
                B.TrainProj(view(), **dict(good, **{name: good[name].view(t)}))
    for name in good:
        with pytest.raises(ValueError, match=name):  # short, and not contiguous
            B.TrainProj(view(), **dict(good, **{name: good[name][:-1]}))
        with pytest.raises(ValueError, match=name):
            B.TrainProj(view(), **dict(good, **{name: torch.empty(2 * good[name].numel(), dtype=good[name].dtype)[::2]}))


def test_both_scales_or_none():
    a = proj_arrays(True)
    for name in ("m_scale", "v_scale"):
        with pytest.raises(ValueError, match="scale"):
            B.TrainProj(view(), **dict(a, **{name: None}))

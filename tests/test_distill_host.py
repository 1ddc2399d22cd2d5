"""Distillation without a GPU: the plain form's gradient against differences, and the refusals that happen on
the host before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch

import distill_ref as R
from segmented_gather_gemm_lora_gb300 import binding as B


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
def test_plain_gradient_against_differences(kind, tail):
    if kind == "reverse" and not tail:
        pytest.skip("reverse needs a tail")
    rng = np.random.default_rng(0)
    T, V, k = 5, 9, 4
    x = rng.normal(size=(T, V))
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(T)])
    values = rng.normal(size=(T, k))
    ids[1, 2], values[2, 0] = -1, -np.inf
    labels = np.array([0, 3, 8, -1, 2])
    args = dict(ids=ids, values=values, tail=rng.normal(size=T) if tail else None, labels=labels, weight=rng.uniform(0.5, 1, T),
                kind=kind, mix=0.3, temperature=1.7, kd_weight=2.0, ce_weight=0.5)
    g = R.distill(x, **args)["grad"]
    h = 1e-5  # third derivatives stay below 10
    for t in range(T):
        for v in range(V):
            d = np.zeros_like(x)
            d[t, v] = h
            num = (R.distill(x + d, **args)["loss"].sum() - R.distill(x - d, **args)["loss"].sum()) / (2 * h)
            assert abs(num - g[t, v]) <= 2e-9 + 1e-8


def test_plain_topk_orders_ties_by_index():
    ids, values, tail = R.topk(np.array([[1.0, 3.0, 3.0, -np.inf, 0.0], [-np.inf] * 5]), 4, 1.0)
    assert ids.tolist() == [[1, 2, 0, 4], [-1] * 4] and tail.tolist() == [-np.inf, -np.inf]


FAKE = 1 << 20  # an address that no call here gets as far as using


def topk(logits=FAKE, ld=100, dtype=0, labels=None, T=4, V=100, k=5, temperature=1.0, ids=FAKE, values=FAKE, tail=None):
    return B.lib().lora_topk_logits(logits, ld, dtype, labels, T, V, k, temperature, ids, values, tail, None, None)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=FAKE + 1), dict(ld=99), dict(dtype=2), dict(T=-1), dict(V=0), dict(k=0),
                                dict(k=101), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
                                dict(temperature=float("inf")), dict(ids=None), dict(values=None), dict(values=FAKE + 2),
                                dict(tail=FAKE + 2), dict(labels=FAKE + 2), dict(dtype=1, logits=FAKE + 2), dict(ld=1 << 41)])
def test_topk_refuses_bad_arguments(kw):
    assert topk(**kw) == B.LORA_ERR_INVALID_ARG


def test_topk_refuses_longer_lists_and_takes_no_rows():
    assert topk(ld=1000, V=1000, k=257) == B.LORA_ERR_UNSUPPORTED
    assert topk(T=0, logits=None, ids=None, values=None) == B.LORA_OK


OPTS = dict(kind=0, temperature=1.0, mix=0.5, kd_weight=1.0, ce_weight=0.0, grad_scale=1.0)


def loss(logits=FAKE, ld=100, dtype=0, ids=FAKE, values=FAKE, tail=FAKE, k=5, labels=FAKE, weight=None, T=4, V=100, out=FAKE, kd=None,
         ce=None, dlogits=None, ldd=0, opts=True, **kw):
    o = B.lora_distill_opts_t(**dict(OPTS, **kw))
    return B.lib().lora_distill_loss(logits, ld, dtype, ids, values, tail, k, labels, weight, T, V, ctypes.byref(o) if opts else None,
                                     out, kd, ce, dlogits, ldd, None, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=FAKE + 1), dict(ld=99), dict(dtype=2), dict(T=-1), dict(V=0), dict(k=0),
                                dict(ids=None), dict(values=None), dict(out=None), dict(ids=FAKE + 1), dict(values=FAKE + 2),
                                dict(out=FAKE + 2), dict(tail=FAKE + 1), dict(weight=FAKE + 1), dict(kd=FAKE + 1), dict(ce=FAKE + 1),
                                dict(labels=FAKE + 1), dict(opts=False), dict(kind=3), dict(kind=-1), dict(temperature=0.0),
                                dict(temperature=NAN), dict(temperature=INF), dict(kind=2, mix=0.0), dict(kind=2, mix=1.0),
                                dict(kind=2, mix=NAN), dict(kd_weight=-1.0), dict(kd_weight=NAN), dict(ce_weight=-1.0),
                                dict(ce_weight=NAN), dict(kind=1, tail=None), dict(ce_weight=1.0, labels=None),
                                dict(dlogits=FAKE, ldd=99), dict(dlogits=FAKE + 200, ldd=101), dict(dlogits=FAKE + 1, ldd=100),
                                dict(ld=1 << 41)])
def test_loss_refuses_bad_arguments(kw):
    assert loss(**kw) == B.LORA_ERR_INVALID_ARG


def test_loss_refuses_longer_lists_and_takes_no_rows():
    assert loss(ld=1000, V=1000, k=257) == B.LORA_ERR_UNSUPPORTED
    assert loss(T=0, logits=None, ids=None, values=None, out=None) == B.LORA_OK


# ------------------------------------------------------------------ the binding --

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
    monkeypatch.setattr(B, "_one_device", lambda *a: None)
    return r.calls


def lists(T=4, k=3):
    return torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)


def test_options_held_in_tensors_are_read_at_each_call(calls):
    x, (ids, values), f = torch.zeros(4, 8), lists(), torch.zeros(4)
    for name in ("mix", "temperature", "kd_weight", "ce_weight", "grad_scale"):
        value = torch.tensor(0.25)
        for v in (0.25, 0.5):
            value.fill_(v)
            B.lora_distill_loss(x, ids, values, f, None, None, stream=0, **{name: value})
            o = [a._obj for a in calls[-1][1] if hasattr(a, "_obj")][0]
            assert getattr(o, name) == v


def test_binding_refuses_arrays_of_another_shape_or_type(calls):
    x, (ids, values), f = torch.zeros(4, 8), lists(), torch.zeros(4)
    i = torch.zeros(4, dtype=torch.int32)
    bad = [dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.view(-1)), dict(ids=torch.zeros(3, 4, dtype=torch.int32).t()),
           dict(values=values.double()), dict(values=values[:, :2]), dict(tail=f[:3]), dict(labels=f), dict(labels=i[:2]),
           dict(weight=i), dict(loss=f[:3]), dict(kd=i), dict(ce=f[:1]), dict(dlogits=torch.zeros(4, 9)),
           dict(dlogits=torch.zeros(4, 8, dtype=torch.bfloat16)), dict(logits=x.half()), dict(logits=x.t()),
           dict(logits=x[:1].expand(4, 8)), dict(err=f)]
    for kw in bad:
        args = dict(logits=x, ids=ids, values=values, loss=f, kd=None, dlogits=None, **{})
        args.update(kw)
        with pytest.raises(ValueError):
            B.lora_distill_loss(**args, stream=0)
    for kw in [b for b in bad if set(b) <= {"ids", "values", "tail", "labels", "logits", "err"}]:
        args = dict(logits=x, ids=ids, values=values)
        args.update(kw)
        with pytest.raises(ValueError):
            B.lora_topk_logits(**args, stream=0)
    assert not calls


def test_binding_refuses_tensors_off_the_device():
    x, (ids, values), f = torch.zeros(4, 8), lists(), torch.zeros(4)
    for stream in (None, 0):
        with pytest.raises(ValueError):
            B.lora_topk_logits(x, ids, values, stream=stream)
        with pytest.raises(ValueError):
            B.lora_distill_loss(x, ids, values, f, None, None, stream=stream)

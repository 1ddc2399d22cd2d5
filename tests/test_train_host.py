"""Training operators without a GPU: the plain forms' gradients against differences, the layout of
the structures, and the refusals that happen on the host before anything is launched."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import train_ref as R
from segmented_gather_gemm_lora_gb300 import binding as B
from test_abi_host import fake_view

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def small_batch(seed, T=9, V=7):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, V)) * 2
    labels = rng.integers(0, V, T)
    labels[2] = -1
    return rng, x, labels


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_against_differences(kind, average):
    rng, x, labels = small_batch(1)
    ref = R.logprobs(x, labels)[0] + 0.2 * rng.normal(size=9)
    args = (labels, ref, [0, 3, 5, 5, 8], kind, 0.7, 0.1, 0.05, average, 1.0)
    g = R.preference(x, *args)[2]
    # central differences: the third derivatives here stay below 10, so h^2 / 6 * 10 is the error
    h = 1e-5
    for t, v in [(0, 0), (0, int(labels[0])), (2, 1), (3, 4), (6, 2), (8, 3)]:
        d = np.zeros_like(x)
        d[t, v] = h
        num = (R.preference(x + d, *args)[0].sum() - R.preference(x - d, *args)[0].sum()) / (2 * h)
        assert abs(num - g[t, v]) <= 1e-9 + 1e-8


def test_policy_gradient_against_differences():
    rng, x, labels = small_batch(2)
    lp = R.logprobs(x, labels)[0]
    old, ref = lp + rng.choice([-0.5, 0.05, 0.5], 9), lp + 0.3 * rng.normal(size=9)
    adv, weight = rng.normal(size=9), rng.uniform(0.5, 1, 9)
    args = (labels, old, adv, ref, weight, 0.2, 0.3, 0.1, 1.0)
    g = R.policy(x, *args)[3]
    h = 1e-5
    for t in range(9):
        for v in (0, 3, max(0, int(labels[t]))):
            d = np.zeros_like(x)
            d[t, v] = h
            num = (R.policy(x + d, *args)[1].sum() - R.policy(x - d, *args)[1].sum()) / (2 * h)
            assert abs(num - g[t, v]) <= 1e-9 + 1e-8


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [B.lora_pref_opts_t, B.lora_policy_opts_t, B.lora_train_proj_t, B.lora_adamw_hyper_t]
    lines = []
    for s in structs:
        n = s.__name__
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (n, n))
        for f, _ in s._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (n, f, n, f))
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"lora_train.h\"\nint main(void) {\n%s\nreturn 0;\n}\n"
                   % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True, capture_output=True)
    got = dict(line.rsplit(" ", 1) for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                              text=True).stdout.splitlines())
    for s in structs:
        assert int(got[s.__name__]) == ctypes.sizeof(s)
        for f, _ in s._fields_:
            assert int(got["%s.%s" % (s.__name__, f)]) == getattr(s, f).offset, (s.__name__, f)


def vp(x):
    return ctypes.c_void_p(x)


LOGITS = dict(logits=0x10000000, ld=104, dtype=0, labels=0x1000, T=10, V=100)


def call_logprobs(**kw):
    a = dict(LOGITS, logp=0x2000, lse=0)
    a.update(kw)
    return B.lib().lora_token_logprobs(vp(a["logits"]), a["ld"], a["dtype"], vp(a["labels"]), a["T"], a["V"],
                                       vp(a["logp"]), vp(a["lse"]), None, None)


def call_preference(**kw):
    a = dict(LOGITS, ref=0, indptr=0x3000, n=2, opts=(0, 0, 0.1, 0.0, 0.0, 1.0), loss=0x4000, seq=0, d=0x20000000,
             ldd=104, ws=0x5000, wsb=1 << 20)
    a.update(kw)
    return B.lib().lora_preference_loss(vp(a["logits"]), a["ld"], a["dtype"], vp(a["labels"]), vp(a["ref"]),
                                        vp(a["indptr"]), a["n"], a["T"], a["V"],
                                        None if a["opts"] is None else ctypes.byref(B.lora_pref_opts_t(*a["opts"])),
                                        vp(a["loss"]), vp(a["seq"]), vp(a["d"]), a["ldd"], vp(a["ws"]), a["wsb"], None, None)


def call_policy(**kw):
    a = dict(LOGITS, old=0x3000, ref=0x3400, adv=0x3800, weight=0, opts=(0.2, 0.2, 0.1, 1.0), logp=0x4000, loss=0x4400,
             kl=0, d=0x20000000, ldd=104)
    a.update(kw)
    return B.lib().lora_policy_loss(vp(a["logits"]), a["ld"], a["dtype"], vp(a["labels"]), vp(a["old"]), vp(a["ref"]),
                                    vp(a["adv"]), vp(a["weight"]), a["T"], a["V"],
                                    None if a["opts"] is None else ctypes.byref(B.lora_policy_opts_t(*a["opts"])),
                                    vp(a["logp"]), vp(a["loss"]), vp(a["kl"]), vp(a["d"]), a["ldd"], None, None)


BAD_LOGITS = [dict(logits=0), dict(logits=0x10000001), dict(dtype=2), dict(ld=99), dict(T=-1), dict(V=0), dict(labels=0),
              dict(labels=0x1002), dict(ld=1 << 41), dict(dtype=1, logits=0x10000002)]


@pytest.mark.parametrize("bad", BAD_LOGITS + [dict(logp=0), dict(logp=0x2002), dict(lse=0x2001)])
def test_logprobs_refusals(bad):
    assert call_logprobs(**bad) == B.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad,want", [(b, B.LORA_ERR_INVALID_ARG) for b in BAD_LOGITS + [
    dict(n=-1), dict(opts=None), dict(opts=(3, 0, 0.1, 0, 0, 1)), dict(opts=(0, 2, 0.1, 0, 0, 1)),
    dict(opts=(0, 0, 0.0, 0, 0, 1)), dict(opts=(0, 0, float("nan"), 0, 0, 1)), dict(opts=(0, 0, 0.1, 1.5, 0, 1)),
    dict(opts=(0, 0, 0.1, -0.1, 0, 1)), dict(indptr=0), dict(loss=0), dict(ref=0x3002), dict(seq=0x3002),
    dict(d=0x20000001), dict(ldd=99), dict(d=0x10000000, ldd=112), dict(d=0x10000000 + 2 * 104), dict(ws=0),
    dict(ws=0x5004)]] + [(dict(wsb=100), B.LORA_ERR_WORKSPACE)])
def test_preference_refusals(bad, want):
    assert call_preference(**bad) == want


@pytest.mark.parametrize("bad", BAD_LOGITS + [
    dict(old=0), dict(adv=0), dict(logp=0), dict(loss=0), dict(kl=0x4002), dict(weight=0x4001), dict(ref=0),
    dict(opts=None), dict(opts=(-0.1, 0.2, 0.1, 1)), dict(opts=(1.1, 0.2, 0.1, 1)), dict(opts=(0.2, -0.2, 0.1, 1)),
    dict(opts=(0.2, 0.2, -0.1, 1)), dict(opts=(0.2, float("nan"), 0.1, 1)), dict(ldd=99), dict(d=0x10000000 + 2)])
def test_policy_refusals(bad):
    assert call_policy(**bad) == B.LORA_ERR_INVALID_ARG


def test_no_rows_is_a_no_op_without_launch():
    before = B.launch_count()
    assert call_logprobs(T=0) == B.LORA_OK
    assert call_policy(T=0) == B.LORA_OK
    assert call_preference(T=0, n=0) == B.LORA_OK
    assert B.launch_count() == before


def fake_proj(**kw):
    d = dict(grad=0x1000000, master=0, m=0x2000000, v=0x3000000, m_scale=0, v_scale=0)
    view = kw.pop("view", None) or fake_view()
    d.update(kw)
    return B.lora_train_proj_t(view, *(d[k] for k in ("grad", "master", "m", "v", "m_scale", "v_scale")))


def call_step(projs=None, n=1, state=0, ids=0x1000, n_ids=3, hyper=0x2000, sumsq=0, flags=0):
    arr = (B.lora_train_proj_t * max(1, n))(*(projs or [fake_proj()]))
    return B.lib().lora_adamw_step(arr, n, state, vp(ids), n_ids, vp(hyper), vp(sumsq), flags, None, None)


def test_step_refusals():
    bad = B.LORA_ERR_INVALID_ARG
    assert call_step(n=0) == bad
    assert call_step(state=2) == bad
    assert call_step(ids=0) == bad
    assert call_step(n_ids=-1) == bad
    assert call_step(n_ids=B.LORA_MAX_ADAPTERS + 1) == B.LORA_ERR_UNSUPPORTED
    assert call_step(hyper=0) == bad
    assert call_step(hyper=0x2002) == bad
    assert call_step(sumsq=0x2002) == bad
    assert call_step(flags=2) == bad
    assert call_step([fake_proj(view=fake_view(pool=0x10008))]) == bad
    assert call_step([fake_proj(view=fake_view(max_rank=65))]) == B.LORA_ERR_UNSUPPORTED
    assert call_step([fake_proj(), fake_proj(view=fake_view(n_adapters=5))], n=2) == bad
    for k in ("grad", "m", "v"):
        assert call_step([fake_proj(**{k: 0})]) == bad
        assert call_step([fake_proj(**{k: 0x1000008})]) == bad
    assert call_step([fake_proj(master=0x4000004)]) == bad
    assert call_step([fake_proj(m=0x1000010)]) == bad  # overlaps grad
    assert call_step([fake_proj(master=0x2000000)]) == bad  # overlaps m
    assert call_step([fake_proj(m_scale=0x5000000)]) == bad  # scales belong to the 8-bit state
    assert call_step(state=B.LORA_STATE_E4M3) == bad
    assert call_step([fake_proj(m_scale=0x5000001, v_scale=0x6000000)], state=B.LORA_STATE_E4M3) == bad
    before = B.launch_count()
    assert call_step(n_ids=0) == B.LORA_OK
    assert B.launch_count() == before


def test_sumsq_and_init_refusals():
    L = B.lib()
    arr = (B.lora_train_proj_t * 1)(fake_proj())
    need = L.lora_grad_sumsq_workspace_bytes(arr, 1, 3)
    assert need >= 3 * 2 * 4
    assert L.lora_grad_sumsq_workspace_bytes(arr, 0, 3) == 0
    assert L.lora_grad_sumsq_workspace_bytes(arr, 1, -1) == 0

    def call(ids=0x1000, n_ids=3, sumsq=0x2000, ws=0x3000, bytes_=need):
        return L.lora_grad_sumsq(arr, 1, vp(ids), n_ids, 0, vp(sumsq), vp(ws), bytes_, None, None)

    assert call(ids=0) == B.LORA_ERR_INVALID_ARG
    assert call(sumsq=0) == B.LORA_ERR_INVALID_ARG
    assert call(sumsq=0x2002) == B.LORA_ERR_INVALID_ARG
    assert call(ws=0) == B.LORA_ERR_INVALID_ARG
    assert call(ws=0x3004) == B.LORA_ERR_INVALID_ARG
    assert call(bytes_=need - 1) == B.LORA_ERR_WORKSPACE
    assert call(n_ids=0, ids=0) == B.LORA_OK
    assert L.lora_adamw_init(arr, 1, 2, vp(0x1000), 3, None, None) == B.LORA_ERR_INVALID_ARG
    assert L.lora_adamw_init(arr, 1, 0, vp(0), 3, None, None) == B.LORA_ERR_INVALID_ARG
    assert L.lora_adamw_init(arr, 1, 0, vp(0), 0, None, None) == B.LORA_OK


def test_binding_refusals():
    x = torch.zeros(4, 8, dtype=torch.float16)
    lab, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError):
        B.lora_token_logprobs(x, lab, f, stream=0)
    x = x.float()
    with pytest.raises(ValueError):
        B.lora_token_logprobs(x.t(), lab, f, stream=0)
    with pytest.raises(ValueError):
        B.lora_token_logprobs(x, lab.long(), f, stream=0)
    with pytest.raises(ValueError):
        B.lora_token_logprobs(x, lab[:3], f, stream=0)
    with pytest.raises(ValueError):
        B.lora_policy_loss(x, lab, f, f, f.clone(), f.clone(), None, torch.zeros(4, 9), stream=0)
    with pytest.raises(ValueError):
        B.lora_preference_loss(x, lab, lab, torch.zeros(1), None, None, torch.zeros(64, dtype=torch.uint8), stream=0)


def test_hyper_holds_each_adapters_settings():
    h = B.adamw_hyper(3, step=[1, 5, 9], lr=[1e-3, 2e-3, 3e-3], max_norm=1.5, device="cpu")
    assert h.view(torch.int32)[:, 0].tolist() == [1, 5, 9]
    one = B.lora_adamw_hyper_t.from_buffer_copy(h.numpy().tobytes()[32:64])
    assert one.step == 5 and abs(one.lr - 2e-3) < 1e-9 and one.max_norm == 1.5 and one.grad_scale == 1.0


def sized_proj(d_in=4096, d_out=4096, max_rank=64, **kw):
    return fake_proj(view=fake_view(d_in=d_in, d_out=d_out, max_rank=max_rank), **kw)


@pytest.mark.parametrize("shapes,max_rank", [([(4096, 4096)] * 4 + [(4096, 11008)] * 2 + [(11008, 4096)], 64),
                                             ([(2048, 2048)], 8), ([(8, 8)], 1), ([(5120, 13824)] * 20, 16)])
def test_a_norm_workspace_for_many_adapters_serves_fewer(shapes, max_rank):
    """The size grows with the list, and a byte less than a list's own size is refused."""
    L = B.lib()
    arr = (B.lora_train_proj_t * len(shapes))(*(sized_proj(a, b, max_rank) for a, b in shapes))
    need = [L.lora_grad_sumsq_workspace_bytes(arr, len(shapes), n) for n in range(B.LORA_MAX_ADAPTERS + 1)]
    assert all(0 < a <= b for a, b in zip(need, need[1:]))
    for n in (1, 2, 5, 15, 16, 17, 31, 32, 200, 1000):
        status = L.lora_grad_sumsq(arr, len(shapes), vp(0x1000), n, 0, vp(0x2000), vp(0x3000), need[n] - 1, None, None)
        assert status == B.LORA_ERR_WORKSPACE


def test_gradient_rows_between_the_logits_rows_are_accepted():
    """Halves of one buffer whose rows take turns do not overlap; shifted into each other they do."""
    big = dict(ld=256, ldd=256, ws=0x5000, wsb=16, T=10, V=100)  # stops at the workspace, after the checks of the rows
    base = 0x10000000
    for shift in (100, 128, 156):
        assert call_preference(**big, d=base + 2 * shift) == B.LORA_ERR_WORKSPACE
        assert call_preference(**big, d=base - 2 * shift) == B.LORA_ERR_WORKSPACE
    for shift in (1, 99, 157, 255, 256, 256 + 99, 9 * 256 - 1):
        assert call_preference(**big, d=base + 2 * shift) == B.LORA_ERR_INVALID_ARG
        assert call_preference(**big, d=base - 2 * shift) == B.LORA_ERR_INVALID_ARG
    # other strides: their ranges must not meet
    assert call_preference(**dict(big, ldd=300), d=base + 2 * 128) == B.LORA_ERR_INVALID_ARG
    assert call_preference(**dict(big, ldd=300), d=base + 2 * 2404) == B.LORA_ERR_WORKSPACE

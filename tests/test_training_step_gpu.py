"""The operators together, as examples/training_step.py runs them: its
gradients against autograd in 64 bits, and a few steps that have to raise the
likelihood of what is rewarded. And the operators' kernels in a debug build,
whose stores are all checked against their buffers."""
import importlib.util
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from newton_schulz_quintic_gb300 import api

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from newton_schulz_quintic_gb300 import build
    build.build()
    api.load_library()
    spec = importlib.util.spec_from_file_location("training_step", os.path.join(ROOT, "examples", "training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def batch(model, n, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, model.table.shape[0], (n,), device="cuda", generator=g)
    targets = (ids * 7 + 1) % model.table.shape[0]
    targets[: n // 4] = -100
    return ids, targets, torch.randn(n, device="cuda", generator=g) + 1, (targets >= 0).float() / n


def test_gradients_of_a_step(example):
    model = example.Model(vocab=301, dim=64, ffn=96)
    ids, targets, adv, w = batch(model, 333)
    logits, kept = model.forward(ids)
    out = api.policy_loss(logits, targets, adv, w)
    got = model.backward(out.dlogits, kept)
    p = [t.double().requires_grad_() for t in (model.table, model.w_gu, model.w_down)]
    table, w_gu, w_down = p
    x = table[ids] * model.scale
    gate, up = (x @ w_gu.t()).chunk(2, 1)
    y = x + (gate * torch.sigmoid(gate) * up) @ w_down.t()
    lp = torch.log_softmax(y @ table.t() / model.scale, -1)
    live = targets >= 0
    lp = lp[torch.arange(len(ids), device="cuda"), targets.clamp(min=0)]
    # on-policy: the gradient of -A r at r = 1
    loss = -(w.double() * adv.double() * torch.exp(lp - lp.detach()) * live).sum()
    loss.backward()
    for name, a, b in zip(("table", "w_gu", "w_down"), got, p):
        err = float((a.double() - b.grad).norm() / b.grad.norm())
        # 8 bits: about 0.7 % of a value each (half a unit of 1/128 .. 1/64 of its block's largest, uniform), bf16
        # activations and products 0.4 %: a handful of such independent errors in a row, below 3 %
        assert err < 0.03, (name, err)


def test_steps_raise_what_is_rewarded(example):
    model = example.Model(vocab=301, dim=64, ffn=96, seed=1)
    ids, targets, _, w = batch(model, 1024)
    adv = torch.ones(1024, device="cuda")
    live = targets >= 0
    seen = [float(model.step(ids, targets, adv, w).logp[live].mean()) for _ in range(12)]
    assert seen[-1] > seen[0] + 0.1, seen
    assert api.get_status() == 0


CHILD = textwrap.dedent("""
    import os, sys
    import torch
    sys.path.insert(0, %r)
    from newton_schulz_quintic_gb300 import build, api
    os.environ["NS_LIBRARY_PATH"] = build.build()
    api.load_library()
    assert api.selftest_bounds_check() == 0
    assert api.get_status() == -8 and api.get_status() == 0
    bf16, f32 = torch.bfloat16, torch.float32
    for dt in (bf16, f32):
        for n, vocab, dim in ((100, 501, 33), (3000, 700, 64)):
            ids = torch.randint(-1, vocab, (n,), device="cuda")
            table, dout = torch.randn(vocab, dim, device="cuda").to(dt), torch.randn(n, dim, device="cuda").to(dt)
            api.embed_lookup(table, ids)
            for gd in (bf16, f32):
                g = api.embed_grad(dout, ids, vocab=vocab, dtype=gd)
                api.embed_grad(dout, ids, grad=g, accumulate=True)
        for n, vocab in ((3, 40000), (70, 1001), (500, 256)):
            x, y = torch.randn(n, vocab, device="cuda").to(dt), torch.randint(-1, vocab, (n,), device="cuda")
            api.token_logprobs(x, y)
            api.policy_loss(x, y, torch.randn(n, device="cuda"), torch.ones(n, device="cuda"), kl_coef=0.1,
                            ref_logp=torch.zeros(n, device="cuda"))
        for n, m in ((5, 31), (70, 1024), (33, 4112)):
            gu, dh = torch.randn(n, 2 * m, device="cuda").to(dt), torch.randn(n, m, device="cuda").to(dt)
            h, a, b = api.gated_forward(gu[:, :m], gu[:, m:])
            api.gated_backward(dh, a, b)
            api.checkpoint_load(api.checkpoint_store(dh), dtype=dt)
        for t, n, k, groups in ((300, 200, 333, 1), (2000, 100, 64, 1), (700, 300, 512, 3)):
            dy, ck = torch.randn(t, n, device="cuda").to(dt), api.checkpoint_store(torch.randn(t, k, device="cuda"))
            off = torch.tensor([0, t // 3, t // 2, t], dtype=torch.int32, device="cuda") if groups == 3 else None
            g = api.checkpoint_wgrad(dy, ck, offsets=off)
            api.checkpoint_wgrad(dy, ck, offsets=off, grad=g, accumulate=True)
    assert api.get_status() == 0, "a bounds check fired"
    print("debug-bounds ok")
""") % ROOT


def test_debug_build_checks_the_operators():
    env = dict(os.environ, NS_BUILD_TAG="debugbounds", NS_EXTRA_NVCC_FLAGS="-DNS_DEBUG_BOUNDS")
    env.pop("NS_LIBRARY_PATH", None)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=1200, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug-bounds ok" in r.stdout

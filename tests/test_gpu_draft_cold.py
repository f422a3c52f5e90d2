"""Verification of drafted tokens at temperatures down to the smallest f32 and for logits up to the largest: whole numbers, equal
to the plain definition's (oracle/draft.py), which takes differences before anything else."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from test_gpu_draft import _check_verify
from test_gpu_serve8 import TYPES, Batch

pytestmark = pytest.mark.gpu

COLD = [1e-5, 1e-7, 1e-10, 1e-12, 1e-13, 1e-14, 1e-15, 1e-17, 1e-20, 1e-30, 1e-38, 1.5e-45]


def _near(rng, T, vocab, xt, size):
    """Logits about `size`, several of them the largest or a few steps of the type below it."""
    x = torch.from_numpy(rng.normal(size=(T, vocab)) * size * 0.2 + size * 0.1).to(TYPES[xt])
    top = x.double().abs().amax(1) * 1.25
    eps = torch.finfo(TYPES[xt]).eps
    for r in range(T):
        at = torch.from_numpy(rng.permutation(vocab)[:12])
        x[r, at] = (top[r] * (1 - eps * torch.tensor([0, 0, 0, 1, 1, 2, 3, 4, 5, 8, 16, 32], dtype=torch.float64))).to(TYPES[xt])
    return x


def _run(rng, target, draft, temps, n):
    """Chains by the draft's probabilities, and trees and chains of chosen tokens."""
    b = Batch([(n, n + 5)] * len(temps), 1, 64, 16, 1)
    d = draft.double().numpy()
    tokens = np.zeros(b.T, np.int64)
    for r in range(1, b.T):
        if r % n:
            tokens[r] = od.pick(od.chance(d[r - 1], float(temps[r // n])), rng.random())
    sample, accept = (rng.random(b.T).astype(np.float32) for _ in "sa")
    target, draft = target.cuda(), draft.cuda()
    got = _check_verify(b, tokens, target, draft=draft, temps=temps, sample=sample, accept=accept)
    assert got[1].min() >= 0
    best = target.double().argmax(1).cpu().numpy()
    tokens[1:] = np.where(rng.random(b.T - 1) < 0.5, best[:-1], tokens[1:])
    par = np.concatenate([np.arange(-1, n - 1)] * len(temps)).astype(np.int32)
    for parents in (None, par):
        got = _check_verify(b, tokens, target, temps=temps, sample=sample, parents=parents)
        assert got[1].min() >= 0


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
def test_cold(xt):
    rng = np.random.default_rng(5)
    temps = np.repeat(np.array(COLD, np.float32), 4)
    print(f"verify cold {xt}", flush=True)
    for vocab in (700, 3000):
        target = _near(rng, 3 * len(temps), vocab, xt, 12.3)
        draft = _near(rng, 3 * len(temps), vocab, xt, 30.0)
        # half of the time what the target holds largest is the draft's largest too
        for r in range(0, len(target), 2):
            at = target[r].double().argmax()
            draft[r, at] = draft[r].max()
        _run(rng, target, draft, temps, 3)


@pytest.mark.parametrize("size", [1e4, 1e9, 1e12, 1e15, 1e19, 1e25, 1e37, -1e15, -1e30])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_large_logits(xt, size):
    rng = np.random.default_rng(6)
    print(f"verify large logits {xt} {size}", flush=True)
    temps = np.array([1.0, 0.5, 2.0, 1e-3, 1e3, 1e-30, 3e38, size if size > 0 else 1.0], np.float32)
    target, draft = (_near(rng, 3 * len(temps), 2500, xt, abs(size)) * (1 if size > 0 else -1) for _ in "td")
    draft[::2] = target[::2]
    _run(rng, target, draft, temps, 3)


def test_large_trees_cold():
    """Batches whose first rows go before the others."""
    rng = np.random.default_rng(7)
    n, temps = 60, np.array(COLD * 3, np.float32)
    assert n * len(temps) * 10 >= 20000
    target = _near(rng, n * len(temps), 9500, "f32", 12.3)
    b = Batch([(n, n + 5)] * len(temps), 1, 64, 16, 1)
    best = target.argmax(1).numpy()
    tokens = rng.integers(0, 9500, b.T)
    tokens[1:] = np.where(rng.random(b.T - 1) < 0.9, best[:-1], tokens[1:])
    par = np.concatenate([np.arange(-1, n - 1)] * len(temps)).astype(np.int32)
    got = _check_verify(b, tokens, target.cuda(), parents=par, temps=temps, sample=rng.random(b.T).astype(np.float32))
    assert got[1].min() >= 0


@pytest.mark.parametrize("temp", [1e-10, 1e-14, 1e-15, 1e-18, 1e-30, 1e-45])
def test_halves(temp):
    """A token that the target gives a half and the draft all, by largest logits of different sizes: it stays below a half."""
    target = torch.full((4, 1500), -3.0)
    target[:, 7] = target[:, 1111] = 12.3
    draft = torch.full((4, 1500), 1.0)
    draft[:, 1111] = 250.7
    b = Batch([(2, 9), (2, 9)], 1, 64, 16, 1)
    tokens = np.array([0, 1111, 0, 1111])
    temps = np.full(2, temp, np.float32)
    got = _check_verify(b, tokens, target.cuda(), draft=draft.cuda(), temps=temps, sample=np.full(4, 0.6, np.float32),
                        accept=np.array([0, 0.49, 0, 0.51], np.float32))
    assert got[0].tolist() == [1, 0] and got[1].tolist() == [1111, 7]

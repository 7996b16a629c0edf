"""The gradient-list oracle against independent derivations (CPU)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import grads as og


@pytest.mark.parametrize("n", [0, 1, 2, 33, 1000])
def test_norms_of_one_list(n):
    x = np.random.default_rng(n).standard_normal(n).astype(np.float32)
    s = og.sums([(x, False)], "2", [0.0, 0.0], 0)
    norm, scale, bad = og.finalize(s, "2", 1.0, 1.0)
    assert norm == pytest.approx(math.hypot(*x.tolist()) if n else 0.0, rel=1e-15)
    assert scale == min(1.0, 1.0 / (norm + 1e-6)) and not bad
    top, _, _ = og.finalize(og.sums([(x, True)], "inf", [0.0, 0.0], 0), "inf", 1.0, 1.0)
    assert top == (torch.from_numpy(x).abs().max().item() if n else 0.0)


def test_finalize_agrees_with_the_flat_norms():
    """At loss scale 1 both norms are the same."""
    s = [3.0, 4.0, 9.0]
    norm, scale, bad = og.finalize(s, "2", 1.0, 1.0)
    n0, _, s0, b0 = oracle.grad_norm_finalize(s[:2], s[2], 1.0)
    assert (norm, np.float32(scale), bad) == (n0, np.float32(s0), b0)


def test_loss_scale_is_taken_out_of_the_norm():
    """Gradients 1024 times as large under a loss scale of 1024: the same norm, and a
    scale that is 1024 times smaller."""
    x = np.array([3.0, 4.0], np.float32)
    n0, s0, _ = og.finalize(og.sums([(x, False)], "2", [0, 0], 0), "2", 2.0, 1.0)
    n1, s1, _ = og.finalize(og.sums([(1024 * x, False)], "2", [0, 0], 0), "2", 2.0, 1024.0)
    assert n0 == n1 == 5.0 and s1 == s0 / 1024


def test_groups_and_peers():
    a, b = np.array([1.0, 2.0], np.float32), np.array([3.0], np.float32)
    assert og.sums([(a, False), (b, True)], "2", [10.0, 20.0, 30.0], 1) == [10.0, 5.0, 9.0]
    assert og.sums([(a, False), (b, True)], "inf", [10.0, 20.0, 30.0], 0) == [2.0, 20.0, 3.0]


@pytest.mark.parametrize("kind", ["2", "inf"])
def test_values_that_are_not_finite(kind):
    for x, want in (([1.0, np.inf], math.inf), ([-np.inf], math.inf), ([np.nan, np.inf], math.nan)):
        norm, scale, bad = og.finalize(og.sums([(np.array(x, np.float32), False)], kind, [0, 0], 0), kind, 1.0, 1.0)
        assert bad and math.isnan(scale) and (norm == want or (math.isnan(norm) and math.isnan(want)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_clip_is_a_product_and_a_cast(dtype):
    x = np.random.default_rng(5).standard_normal(1000).astype(np.float32)
    y = torch.from_numpy(x) * torch.tensor(0.3, dtype=torch.float32)
    t = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    got = og.clip(x, 0.3, dtype)
    want = y.to(t)
    want = want.numpy() if dtype == "fp32" else want.view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, want)


def test_accumulation_is_rounded_once():
    rng = np.random.default_rng(6)
    x, acc = (rng.standard_normal(500).astype(np.float32) for _ in range(2))
    f = 1 / 3
    got = og.accumulate(acc, x, f, False)
    ff = Fraction(float(np.float32(f)))
    for a, v, g in zip(acc, x, got):
        exact = ff * Fraction(float(v)) + Fraction(float(a))
        below, above = np.nextafter(g, np.float32(-np.inf)), np.nextafter(g, np.float32(np.inf))
        d = abs(Fraction(float(g)) - exact)
        assert d <= abs(Fraction(float(below)) - exact) and d <= abs(Fraction(float(above)) - exact)
    assert np.array_equal(og.accumulate(np.full(500, np.nan, np.float32), x, f, True), (np.float32(f) * x).astype(np.float32))

"""Adapters, probabilities and verification on the GPU where one path ends and the next begins, against fp64 and whole numbers.

Tolerances beyond those of the entry points' other tests:
* lora, fp16, rows of x with one element that is not 0: down x is exact in fp32 (22 bits), so what is left is the result's rounding
  2^-11 |out| (2^-25 where it is subnormal), s as two fp16 parts, 2^-22 a with a = sum_r |up s|, and fp32 sums of 2 R products, each
  step of which may cut off one last place: (2 R + 16) 2^-23 a.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import requests_oracle_np as orc
from tests.test_gpu_requests import _check_lora, _lora_inputs, _up, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("M,run", [(20, 1), (300, 60), (1500, 1), (2500, 700), (2500, 2500), (9000, 3000)])
def test_lora_fp16_keeps_the_first_products_precision(env, M, run, R):  # noqa: F811
    """Bases that the adapters' results cancel: what is left shows the bits of down x beyond fp16."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + R)
    K, N = 208, 264
    x, _, down, up, _, scales, adapter = _lora_inputs(rng, M, K, N, R, 5, "f16", without=0)
    adapter[:] = np.arange(M) // run % 5
    at = rng.integers(0, K, M)
    one = x[np.arange(M), at]
    x[:] = 0
    x[np.arange(M), at] = one
    base = (-orc.lora(x, down, up, None, scales, adapter, None)[0]).astype(np.float16)
    want, a, _ = orc.lora(x, down, up, None, scales, adapter, base)
    xd, bd, dd, ud, sd, ad = _up(torch, dev, x, base, down, up, scales, adapter)
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud, scales=sd), ad, base=bd).cpu().numpy().astype(np.float64)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -22 * a + (2 * R + 16) * 2.0 ** -23 * a
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())
    mnb.mnb_check_device_status()

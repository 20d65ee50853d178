"""Adapters, probabilities and verification of drafted tokens: checks that need no GPU (oracle, refusals)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from oracle import requests_oracle_np as orc

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from gemm_mnb_gemv_gb300 import _build
    try:
        _build.build()
    except RuntimeError as e:  # no nvcc in this environment
        pytest.skip(str(e))
    import gemm_mnb_gemv_gb300 as mnb
    return mnb.load_library()


@pytest.mark.parametrize("lookup", [False, True])
def test_oracle_draws_from_the_target(lookup):
    """Over a grid of random numbers, what comes first is distributed as the target, whatever the draft was."""
    p = np.float32([0.5, 0.0, 0.125, 0.25, 0.125])
    q = np.float32([0.125, 0.25, 0.25, 0.25, 0.125])
    n = 32
    grid = (np.arange(n, dtype=np.float32) + 0.5) / n
    count = np.zeros(5)
    for tok, weight in enumerate(q):
        u, v = (g.reshape(-1) for g in np.meshgrid(grid, grid))
        B = len(u)
        tokens, _ = orc.verify(np.tile(p, (2 * B, 1)), None if lookup else np.tile(q, (B, 1)), np.full(B, tok), np.arange(B + 1), u, v)
        count += weight * np.bincount(tokens[::2], minlength=5) / B
    np.testing.assert_allclose(count, p, atol=2 / n)


def test_oracle_lora_against_dense_products():
    rng = np.random.default_rng(1)
    x, down, up = rng.standard_normal((5, 16)), rng.standard_normal((3, 8, 16)), rng.standard_normal((3, 4, 8))
    adapter = np.array([2, -1, 0, 2, 7])
    out, _, _ = orc.lora(x, down, up, [8, 8, 3], [2.0, 1.0, 0.5], adapter, None)
    np.testing.assert_allclose(out[0], 0.5 * up[2, :, :3] @ (down[2, :3] @ x[0]), rtol=1e-12)
    np.testing.assert_allclose(out[2], 2.0 * up[0] @ (down[0] @ x[2]), rtol=1e-12)
    assert not out[1].any() and not out[4].any()


@pytest.mark.parametrize("change,expect,word", [
    (dict(dtype=2), 1, "dtype"),
    (dict(M=-1), 1, "M=-1"),
    (dict(M=(1 << 20) + 1), 1, "M="),
    (dict(K=0), 1, "K=0"),
    (dict(K=40), 1, "K=40"),
    (dict(N=0), 1, "N=0"),
    (dict(count=0), 1, "count"),
    (dict(rank=12), 1, "max_rank"),
    (dict(rank=136), 1, "max_rank"),
    (dict(x=None), 1, "x is NULL"),
    (dict(x=8), 3, "x is not"),
    (dict(x_stride=40), 1, "x_stride"),
    (dict(x_stride=52), 3, "x_stride"),
    (dict(down=None), 1, "down"),
    (dict(up=24), 3, "up"),
    (dict(ranks=4), 3, "ranks"),
    (dict(scales=4), 3, "scales"),
    (dict(adapter=None), 1, "adapter"),
    (dict(base=4), 3, "base"),
    (dict(base_stride=6), 1, "base_stride"),
    (dict(base=96, out=96, base_stride=9), 1, "out_stride"),
    (dict(out=None), 1, "out is NULL"),
    (dict(out_stride=6), 1, "out_stride"),
    (dict(M=1300, ws_bytes=1300 * 24 + 15), 1, "workspace"),
    (dict(M=1300, workspace=None), 1, "workspace"),
    (dict(M=1300, workspace=72), 3, "workspace"),
])
def test_lora_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(x=64, dtype=0, M=3, K=48, x_stride=48, down=64, up=64, ranks=None, scales=None, count=2, rank=16, adapter=64, base=64,
             base_stride=7, N=7, workspace=64, ws_bytes=1 << 40, out=128, out_stride=7)
    a.update(change)
    pool = mnb.MnbLoraPoolArg(a["down"], a["up"], a["ranks"], a["scales"], a["count"], a["rank"])
    st = lib.mnb_lora(P(a["x"]), a["dtype"], a["M"], a["K"], a["x_stride"], pool, P(a["adapter"]), P(a["base"]), a["base_stride"],
                      a["N"], P(a["workspace"]), a["ws_bytes"], P(a["out"]), a["out_stride"], None)
    assert st == expect, mnb.mnb_last_error()
    assert mnb.mnb_last_error().startswith("mnb_lora") and word in mnb.mnb_last_error()


@pytest.mark.parametrize("change,expect,word", [
    (dict(dtype=-1), 1, "dtype"),
    (dict(rows=-1), 1, "rows=-1"),
    (dict(V=0), 1, "V=0"),
    (dict(V=(1 << 24) + 1), 1, "V="),
    (dict(logits=None), 1, "logits"),
    (dict(logits=2), 3, "logits"),
    (dict(stride=9), 1, "stride"),
    (dict(temperature=4), 3, "temperature"),
    (dict(out=None), 1, "out"),
    (dict(rows=77, V=16378, stride=16378, ws_bytes=77 * 7 * 16 - 1, workspace=64), 1, "workspace"),
    (dict(rows=77, V=16378, stride=16378, ws_bytes=1 << 30), 1, "workspace"),
    (dict(rows=1 << 20, V=1 << 23, stride=1 << 23, ws_bytes=1 << 50, workspace=64), 2, "more than"),
])
def test_softmax_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(logits=64, dtype=0, rows=2, V=10, stride=10, temperature=None, workspace=None, ws_bytes=0, out=64)
    a.update(change)
    st = lib.mnb_softmax(P(a["logits"]), a["dtype"], a["rows"], a["V"], a["stride"], P(a["temperature"]),
                         P(a["workspace"]), a["ws_bytes"], P(a["out"]), None)
    assert st == expect, mnb.mnb_last_error()
    assert mnb.mnb_last_error().startswith("mnb_softmax") and word in mnb.mnb_last_error()


@pytest.mark.parametrize("change,expect,word", [
    (dict(batch=-1), 1, "batch=-1"),
    (dict(drafted=-1), 1, "drafted=-1"),
    (dict(batch=0), 1, "drafted"),
    (dict(V=0), 1, "V=0"),
    (dict(target=None), 1, "target"),
    (dict(target=4), 3, "target"),
    (dict(target_stride=9), 1, "target_stride"),
    (dict(draft=4), 3, "draft"),
    (dict(draft_stride=9), 1, "draft_stride"),
    (dict(tokens_in=None), 1, "draft_tokens"),
    (dict(start=None), 1, "draft_start"),
    (dict(u=None), 1, "u_accept"),
    (dict(v=None), 1, "u_next"),
    (dict(tokens=None), 1, "tokens"),
    (dict(accepted=8), 3, "accepted"),
    (dict(batch=600, ws_bytes=600 * 64 - 1), 1, "workspace"),
    (dict(batch=600, workspace=None), 1, "workspace"),
    (dict(batch=1 << 20, V=1 << 23, target_stride=1 << 23, draft_stride=1 << 23), 2, "more than"),
])
def test_verify_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(target=64, target_stride=10, draft=64, draft_stride=10, tokens_in=64, start=64, u=64, v=64, batch=2, drafted=3, V=10,
             workspace=64, ws_bytes=1 << 50, tokens=64, accepted=64)
    a.update(change)
    st = lib.mnb_verify(P(a["target"]), a["target_stride"], P(a["draft"]), a["draft_stride"], P(a["tokens_in"]), P(a["start"]),
                        P(a["u"]), P(a["v"]), a["batch"], a["drafted"], a["V"], P(a["workspace"]),
                        a["ws_bytes"], P(a["tokens"]), P(a["accepted"]), None)
    assert st == expect, mnb.mnb_last_error()
    assert mnb.mnb_last_error().startswith("mnb_verify") and word in mnb.mnb_last_error()


def test_lora_workspace_bytes(lib):
    assert [lib.mnb_lora_workspace_bytes(M) for M in (-1, 0, 1, 256, 257, 1 << 20, (1 << 20) + 1)] == [
        0, 0, 0, 0, 16 + 24 * 257, 16 + 24 * (1 << 20), 0]


def test_draft_workspace_bytes(lib):
    """16 and 64 bytes for each part of a row; a part has 256 to 2048 chunks of 8 elements, or
    512 to 4096 of 4, and the rows have 608 where possible; few rows and few sequences need none."""
    soft, ver = lib.mnb_softmax_workspace_bytes, lib.mnb_verify_workspace_bytes
    assert [soft(*a) for a in [(0, 9), (3, 0), (3, 16377), (76, 16378), (77, 16378), (320, 128256), (1, (1 << 24) + 1)]] == [
        0, 0, 0, 0, 77 * 7 * 16, 320 * 8 * 16, 0]
    assert [ver(*a) for a in [(0, 9), (3, 0), (512, 1), (513, 1), (513, 4096), (64, 128256), (65, 128256), (1, 262141), (1, 262142),
                              (1, (1 << 24) + 1)]] == [0, 0, 0, 513 * 64, 513 * 64, 0, 65 * 9 * 64, 0, 129 * 64, 0]


def test_no_rows_is_valid(lib):
    import gemm_mnb_gemv_gb300 as mnb
    pool = mnb.MnbLoraPoolArg(None, None, None, None, 1, 8)
    assert lib.mnb_lora(None, 0, 0, 16, 16, pool, None, None, 0, 1, None, 0, None, 1, None) == 0
    assert lib.mnb_softmax(None, 0, 0, 1, 1, None, None, 0, None, None) == 0
    assert lib.mnb_verify(None, 0, None, 0, None, None, None, None, 0, 0, 1, None, 0, None, None, None) == 0


def test_host_tensors_are_refused():
    import torch

    import gemm_mnb_gemv_gb300 as mnb
    x = torch.zeros(2, 16)
    with pytest.raises(TypeError, match="down must be a CUDA tensor"):
        mnb.MnbLoraPool(torch.zeros(1, 8, 16, dtype=torch.float16), torch.zeros(1, 4, 8, dtype=torch.float16))
    with pytest.raises(TypeError, match="logits must be a CUDA tensor"):
        mnb.mnb_softmax(x)
    with pytest.raises(TypeError, match="logits must be a CUDA tensor"):
        mnb.mnb_softmax(None)
    with pytest.raises(TypeError, match="target must be a CUDA tensor"):
        mnb.mnb_verify(x, None, None, None, None, None)

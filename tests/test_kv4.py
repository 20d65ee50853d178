"""Paged 4-bit key/value cache: checks that need no GPU (oracle, sizes, refusals)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from oracle import kv4_oracle_np as orc


@pytest.fixture(scope="module")
def lib():
    from gemm_mnb_gemv_gb300 import _build
    try:
        _build.build()
    except RuntimeError as e:  # no nvcc in this environment
        pytest.skip(str(e))
    import gemm_mnb_gemv_gb300 as mnb
    return mnb.load_library()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_block_places_are_a_bijection(D):
    """Every (row, element) has a nibble of its own, and the codes fill the first 16 D bytes."""
    for place, base in ((orc.k_place, 0), (orc.v_place, 8 * D)):
        seen = {place(D, r, d) for r in range(16) for d in range(D)}
        assert seen == {(base + b, bit) for b in range(8 * D) for bit in (0, 4)}


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 128), (256, 64)])
def test_parameter_places_fill_the_rest(D, group):
    seen = {orc.param_place(D, group, r, g, v) for r in range(16) for g in range(D // group) for v in (False, True)}
    assert seen == set(range(16 * D, orc.block_bytes(D, group), 4))


def test_quantise_rounding_error_is_half_a_step():
    """|x - value| <= scale / 2 plus what the fp16 roundings of scale and offset allow: the code grid moves by at
    most |offset| 2^-11 + 15 scale 2^-11."""
    x = np.random.default_rng(1).standard_normal((50, 3, 128)).astype(np.float32) * 3
    code, scale, offset = orc.quantise(x, 32)
    s, o = (np.repeat(a.astype(np.float64), 32, axis=-1) for a in (scale, offset))
    err = np.abs(o + code * s - x)
    assert np.all(err <= s / 2 + np.abs(o) * 2.0 ** -11 + 15 * s * 2.0 ** -11 + 1e-7)
    const = np.full((1, 1, 64), 0.7, dtype=np.float32)
    code, scale, offset = orc.quantise(const, 64)
    assert not code.any() and not scale.any() and offset[0, 0, 0] == np.float16(0.7)


def test_oracle_attention_against_differences_of_lse():
    """d lse / d q = scale * sum_j p_j k_j: the oracle's probabilities against central differences."""
    rng = np.random.default_rng(2)
    D, group, ps = 64, 64, 16
    k, v = rng.standard_normal((2, 20, 1, D)).astype(np.float32)
    pages = np.zeros((2, 1, orc.block_bytes(D, group)), np.uint8)
    pages = orc.append(pages, k, v, None, None, None, False, np.arange(20), ps, group).reshape(pages.shape)
    K, V = orc.read(pages, np.arange(20), ps, 1, D, group, np.float64)
    q = rng.standard_normal((1, 1, D))
    args = (pages, [0, 1], [20], np.array([[0, 1]]), ps, 1, group, 0.125, True, 0)
    out, lse, _, _ = orc.attention(q, *args)
    p = np.exp(0.125 * (K[:, 0] @ q[0, 0]) - lse[0, 0])
    np.testing.assert_allclose(p.sum(), 1, rtol=1e-12)
    np.testing.assert_allclose(out[0, 0], p @ V[:, 0], rtol=1e-10, atol=1e-12)
    h = 1e-5
    for d in (0, 17, 63):
        up, dn = q.copy(), q.copy()
        up[..., d] += h
        dn[..., d] -= h
        diff = (orc.attention(up, *args)[1] - orc.attention(dn, *args)[1])[0, 0] / (2 * h)
        np.testing.assert_allclose(diff, 0.125 * (p @ K[:, 0, d]), rtol=1e-6, atol=1e-9)


def test_cache_bytes(lib):
    for pages, ps, H, D, group in [(1, 16, 1, 64, 64), (7, 48, 3, 128, 32), (2, 4096, 8, 256, 128)]:
        assert lib.mnb_kv4_cache_bytes(pages, ps, H, D, group) == pages * H * (ps // 16) * orc.block_bytes(D, group)
    for bad in [(0, 16, 1, 64, 64), (1, 24, 1, 64, 64), (1, 8192, 1, 64, 64), (1, 16, 0, 64, 64), (1, 16, 1, 96, 32),
                (1, 16, 1, 64, 128), (1, 16, 1, 128, 16)]:
        assert lib.mnb_kv4_cache_bytes(*bad) == 0
    # more than 2^32 bytes
    assert lib.mnb_kv4_cache_bytes(1 << 20, 16, 8, 128, 128) == (1 << 23) * 2176


P = ctypes.c_void_p


def _cache(mnb, pages=64, num_pages=4, page_size=16, kv_heads=2, head_dim=128, group=64):
    return mnb.MnbKv4CacheArg(pages, num_pages, page_size, kv_heads, head_dim, group)


@pytest.mark.parametrize("change,expect,word", [
    (dict(cache=dict(head_dim=96)), 1, "head_dim"),
    (dict(cache=dict(page_size=20)), 1, "page_size"),
    (dict(cache=dict(group=16)), 1, "group_size"),
    (dict(cache=dict(pages=None)), 1, "pages"),
    (dict(cache=dict(pages=72)), 3, "pages"),
    (dict(dtype=2), 1, "dtype"),
    (dict(T=-1), 1, "T=-1"),
    (dict(T=(1 << 20) + 1), 1, "T="),
    (dict(q=None), 1, "q_heads"),
    (dict(q_heads=0), 1, "q_heads"),
    (dict(q_out=None), 1, "q_out"),
    (dict(k=None), 1, "k is NULL"),
    (dict(v=24), 3, "v is not"),
    (dict(k_stride=255), 1, "k_stride"),
    (dict(v_stride=260), 3, "v_stride"),
    (dict(q_stride=511), 1, "q_stride"),
    (dict(slots=None), 1, "slots"),
    (dict(rot=24), 1, "rot_dim"),
    (dict(rot=144), 1, "rot_dim"),
    (dict(rows=0), 1, "rows"),
    (dict(cos=None), 1, "cos"),
    (dict(positions=None), 1, "positions"),
])
def test_append_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(q=64, k=64, v=64, dtype=0, T=3, q_heads=4, q_stride=512, k_stride=256, v_stride=256, positions=64, cos=64,
             rows=10, rot=64, slots=64, q_out=64, cache={})
    a.update(change)
    rope = mnb.MnbRope(a["cos"], 64, a["rows"], a["rot"], 0)
    st = lib.mnb_kv4_append(P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], a["T"], a["q_heads"], a["q_stride"],
                            a["k_stride"], a["v_stride"], P(a["positions"]), rope, P(a["slots"]),
                            _cache(mnb, **a["cache"]), P(a["q_out"]), None)
    assert st == expect, mnb.mnb_last_error()
    assert mnb.mnb_last_error().startswith("mnb_kv4_append") and word in mnb.mnb_last_error()


@pytest.mark.parametrize("change,expect,word", [
    (dict(cache=dict(num_pages=0)), 1, "num_pages"),
    (dict(dtype=-1), 1, "dtype"),
    (dict(q_heads=3), 1, "q_heads"),
    (dict(q_heads=0), 1, "q_heads"),
    (dict(q_stride=256), 1, "q_stride"),
    (dict(q_stride=516), 3, "q_stride"),
    (dict(batch=0), 1, "batch"),
    (dict(table_stride=0), 1, "table_stride"),
    (dict(table_stride=(1 << 26) + 1), 1, "table_stride"),
    (dict(window=-1), 1, "window"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(q=None), 1, "q is NULL"),
    (dict(q_start=None), 1, "q_start"),
    (dict(kv_len=8), 3, "kv_len"),
    (dict(page_table=None), 1, "page_table"),
    (dict(out=None), 1, "out"),
    (dict(lse=4), 3, "lse"),
])
def test_attention_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(q=64, dtype=0, T=3, q_heads=4, q_stride=512, cache={}, q_start=64, kv_len=64, page_table=64, batch=2,
             table_stride=5, scale=0.1, window=0, out=64, lse=None)
    a.update(change)
    st = lib.mnb_kv4_attention(P(a["q"]), a["dtype"], a["T"], a["q_heads"], a["q_stride"], _cache(mnb, **a["cache"]),
                               P(a["q_start"]), P(a["kv_len"]), P(a["page_table"]), a["batch"], a["table_stride"],
                               a["scale"], 1, a["window"], P(64), 1 << 40, P(a["out"]), P(a["lse"]), None)
    assert st == expect, mnb.mnb_last_error()
    assert mnb.mnb_last_error().startswith("mnb_kv4_attention") and word in mnb.mnb_last_error()


def test_attention_workspace_is_checked(lib):
    import gemm_mnb_gemv_gb300 as mnb
    need = mnb.mnb_kv4_attention_workspace_bytes(3, 2, 4, 2, 128)
    for bad in [(0, 2, 4, 2, 128), (3, 0, 4, 2, 128), (3, 2, 3, 2, 128), (3, 2, 4, 2, 100)]:
        assert mnb.mnb_kv4_attention_workspace_bytes(*bad) == 0
    if need:
        st = lib.mnb_kv4_attention(P(64), 0, 3, 4, 512, _cache(mnb), P(64), P(64), P(64), 2, 5, 0.1, 1, 0, P(64),
                                   need - 1, P(64), None, None)
        assert st == mnb.MNB_ERR_INVALID_ARG and "workspace" in mnb.mnb_last_error()


def test_no_tokens_is_valid(lib):
    import gemm_mnb_gemv_gb300 as mnb
    c = _cache(mnb)
    assert lib.mnb_kv4_append(None, None, None, 0, 0, 0, 0, 0, 0, None, mnb.MnbRope(), None, c, None, None) == 0
    assert lib.mnb_kv4_read(c, None, 0, 0, None, None, None) == 0
    assert lib.mnb_kv4_attention(None, 0, 0, 4, 512, c, None, None, None, 0, 5, 0.1, 1, 0, None, 0, None, None,
                                 None) == 0


@pytest.mark.parametrize("change,expect,word", [
    (dict(T=-1), 1, "T=-1"), (dict(dtype=5), 1, "dtype"), (dict(slots=None), 1, "slots"), (dict(k=None), 1, "k_out"),
    (dict(v=8), 3, "v_out"),
])
def test_read_refusals(lib, change, expect, word):
    import gemm_mnb_gemv_gb300 as mnb
    a = dict(T=2, dtype=0, slots=64, k=64, v=64)
    a.update(change)
    st = lib.mnb_kv4_read(_cache(mnb), P(a["slots"]), a["T"], a["dtype"], P(a["k"]), P(a["v"]), None)
    assert st == expect and word in mnb.mnb_last_error()


def test_rows_of_the_tcgen05_kernel_own_their_bytes(tmp_path):
    """A row's chunks lie in bytes of that row alone: q and the results that pass through the same places belong to the
    warp of the row, whichever piece of work each warp is at."""
    import os
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "places.cpp"
    src.write_text('#define __host__\n#define __device__\n#include "kv4.cuh"\n#include <cstdio>\nint main() {\n'
                   '  for (int r = 0; r < 128; ++r)\n    for (int c = 0; c < 16; ++c)\n'
                   '      std::printf("%d\\n", mnb::kv4::tile_row_byte(r, c));\n}\n')
    exe = tmp_path / "places"
    subprocess.run([gxx, "-std=c++17", "-I", os.path.join(root, "gemm_mnb_gemv_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    at = np.array(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split(), int).reshape(128, 16)
    assert sorted(at.reshape(-1)) == list(range(0, 128 * 256, 16))
    np.testing.assert_array_equal(at % 16384 // 128, np.repeat(np.arange(128)[:, None], 16, 1))
    np.testing.assert_array_equal(at // 16384, np.repeat(np.arange(16)[None] // 8, 128, 0))
    # the kernel keeps q and stages its results through these places alone
    kernel = open(os.path.join(root, "gemm_mnb_gemv_gb300", "csrc", "kv4_tile.cu")).read()
    used = [line for line in kernel.splitlines() if "room +" in line]
    assert used and all("room + tile_row_byte(" in line for line in used)


def test_dequantisers_stop_together():
    """They meet at a named barrier, which has no limit: a warp whose wait gave up has to come to it, so the only way out of
    the loop over tiles is behind the barrier, on what all four were told there."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    kernel = open(os.path.join(root, "gemm_mnb_gemv_gb300", "csrc", "kv4_tile.cu")).read()
    assert len(re.findall(r"bar\.sync|barrier\.(?:cta\.)?sync", kernel)) == 1
    role = kernel[kernel.index("- dequantisers -"):kernel.index("- softmax -")]
    loop = role[role.index("for (int tile = "):role.index("next_piece(here)")]
    loop = re.sub(r"\[\]\([^)]*\) \{[^}]*\}", "", loop)  # lambdas
    before, after = loop.split("bar.sync 1, 128;")
    assert not re.search(r"\b(break|return|goto)\b", before)
    outs = re.findall(r"(if \([^;{]*\) \{\s*ok = false;\s*)?\b(?:break|return|goto)\b", after)
    assert len(outs) == 1 and outs[0].startswith("if (ksize == kLate)")


class _Recorder:
    """Stands for the library: keeps what the binding hands to an entry point."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def binding(lib, monkeypatch):
    """The binding on tensors that say they lie on GPU `dev`, and a library that keeps the calls."""
    import torch

    import gemm_mnb_gemv_gb300 as mnb

    class OnGpu(torch.Tensor):
        dev = 0
        is_cuda = property(lambda self: True)

        def get_device(self):
            return self.dev

    def tensor(*shape, dtype=torch.float16, dev=0):
        t = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
        t.dev = dev
        return t

    recorder = _Recorder(lib)
    monkeypatch.setattr(mnb, "load_library", lambda *a: recorder)
    monkeypatch.setattr(mnb, "_raw_stream", lambda *a, **k: 77)
    monkeypatch.setattr(mnb, "_new", lambda shape, dtype, device, stream: tensor(*(shape if isinstance(shape, tuple) else (shape,)),
                                                                                 dtype=dtype))
    monkeypatch.setattr(mnb, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(mnb, "_gpu_count", lambda: 2, raising=False)
    return mnb, torch, tensor, recorder


def _binding_cache(binding, **kw):
    mnb, torch, tensor, _ = binding
    return mnb.MnbKv4Cache(tensor(4, 2, 1280, dtype=torch.uint8, **kw), 16, 64, 32)


def _binding_attention(binding, cache=None, **kw):
    mnb, torch, tensor, _ = binding
    i32 = torch.int32
    a = dict(q=tensor(3, 4, 64), cache=cache or _binding_cache(binding), q_start=tensor(3, dtype=i32), kv_len=tensor(2, dtype=i32),
             page_table=tensor(2, 5, dtype=i32), scale=0.1)
    a.update(kw)
    return mnb.mnb_kv4_attention(**a)


@pytest.mark.parametrize("window,handed_on", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                              (2 ** 32, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1)])
def test_a_window_beyond_32_bits_is_not_cut(binding, window, handed_on):
    _binding_attention(binding, window=window)
    name, args = binding[3].calls[-1]
    assert name == "mnb_kv4_attention" and args[13] == handed_on


@pytest.mark.parametrize("window", [-1, -2 ** 32, -2 ** 32 + 9, -2 ** 40])
def test_a_negative_window_stays_negative(binding, window):
    _binding_attention(binding, window=window)
    assert -2 ** 31 <= binding[3].calls[-1][1][13] < 0  # the library refuses it


def test_sizes_beyond_32_bits_are_refused(binding):
    mnb, torch, tensor, _ = binding
    for bad in [(2 ** 32 + 4, 16, 2, 64, 32), (4, 2 ** 32 + 16, 2, 64, 32), (4, 16, 2, 2 ** 32 + 64, 32), (4, 16, 2, 64, 32 - 2 ** 32)]:
        assert mnb.mnb_kv4_cache_bytes(*bad) == 0
    with pytest.raises(mnb.MnbError):
        mnb.MnbKv4Cache(tensor(4, 2, 1280, dtype=torch.uint8), 2 ** 32 + 16, 64, 32)
    assert mnb.mnb_kv4_attention_workspace_bytes(2 ** 32 + 3, 2, 4, 2, 64) == 0


def _binding_append(binding, cache=None, **kw):
    mnb, torch, tensor, _ = binding
    a = dict(cache=cache or _binding_cache(binding), k=tensor(3, 2, 64), v=tensor(3, 2, 64), slots=tensor(3, dtype=torch.int64),
             q=tensor(3, 4, 64), positions=tensor(3, dtype=torch.int32), cos=tensor(9, 32, dtype=torch.float32),
             sin=tensor(9, 32, dtype=torch.float32))
    a.update(kw)
    return mnb.mnb_kv4_append(**a)


@pytest.mark.parametrize("missing", ["k", "v", "slots", "positions", "sin", "cos"])
def test_append_says_what_is_missing(binding, missing):
    _binding_append(binding)
    calls = len(binding[3].calls)
    with pytest.raises(TypeError, match=missing):
        _binding_append(binding, **{missing: None})
    assert len(binding[3].calls) == calls


@pytest.mark.parametrize("missing", ["q", "q_start", "kv_len", "page_table"])
def test_attention_says_what_is_missing(binding, missing):
    with pytest.raises((TypeError, ValueError), match=missing):
        _binding_attention(binding, **{missing: None})
    assert not binding[3].calls


def test_wrong_dimensions_are_named(binding):
    mnb, torch, tensor, _ = binding
    with pytest.raises(ValueError, match="cos"):
        _binding_append(binding, cos=tensor(9, dtype=torch.float32))
    with pytest.raises(ValueError, match="kv_len"):
        _binding_attention(binding, kv_len=tensor(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="kv_len"):
        _binding_attention(binding, kv_len=torch.tensor(3))
    with pytest.raises(ValueError, match="page_table"):
        _binding_attention(binding, page_table=tensor(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="slots"):
        mnb.mnb_kv4_read(_binding_cache(binding), None)
    assert not binding[3].calls


APPEND = ["k", "v", "slots", "q", "positions", "cos", "sin", "q_out"]
ATTENTION = ["q", "q_start", "kv_len", "page_table", "out", "lse", "workspace"]
READ = ["slots", "k_out", "v_out"]


def _tensors(binding, dev):
    """Arguments of the three entry points on GPU `dev`."""
    _, torch, tensor, _ = binding
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    t = lambda *s, d=torch.float16: tensor(*s, dtype=d, dev=dev)  # noqa: E731
    return (dict(k=t(3, 2, 64), v=t(3, 2, 64), slots=t(3, d=i64), q=t(3, 4, 64), positions=t(3, d=i32), cos=t(9, 32, d=f32),
                 sin=t(9, 32, d=f32), q_out=t(3, 4, 64)),
            dict(q=t(3, 4, 64), q_start=t(3, d=i32), kv_len=t(2, d=i32), page_table=t(2, 5, d=i32), out=t(3, 4, 64),
                 lse=t(3, 4, d=f32), workspace=t(1 << 20, d=torch.uint8)),
            dict(slots=t(3, d=i64), k_out=t(3, 2, 64), v_out=t(3, 2, 64)))


@pytest.mark.parametrize("call,name", [(i, n) for i, names in enumerate((APPEND, ATTENTION, READ)) for n in names])
def test_tensors_of_another_gpu_are_refused(binding, call, name):
    mnb, torch, tensor, recorder = binding
    cache = _binding_cache(binding)
    fn = (mnb.mnb_kv4_append, mnb.mnb_kv4_attention, mnb.mnb_kv4_read)[call]
    own, other = _tensors(binding, 0)[call], _tensors(binding, 1)[call]
    more = dict(scale=0.1) if call == 1 else {}
    fn(cache=cache, **own, **more)
    assert len(recorder.calls) == 1
    with pytest.raises(ValueError, match=f"{name} is on .*the cache on cuda:0"):
        fn(cache=cache, **{**own, name: other[name]}, **more)
    assert len(recorder.calls) == 1


@pytest.mark.parametrize("call", [0, 1, 2])
def test_calls_run_on_the_gpu_of_their_cache(binding, call, monkeypatch):
    """The library launches on the current device: it is the cache's during the call, and no other call changes it."""
    import contextlib
    mnb, torch, tensor, recorder = binding
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append((index, len(recorder.calls)))
        yield
        entered.append(("left", len(recorder.calls)))

    monkeypatch.setattr(torch.cuda, "device", device)
    fn = (mnb.mnb_kv4_append, mnb.mnb_kv4_attention, mnb.mnb_kv4_read)[call]
    more = dict(scale=0.1) if call == 1 else {}
    fn(cache=_binding_cache(binding, dev=1), **_tensors(binding, 1)[call], **more)
    assert entered == [(1, 0), ("left", 1)]
    fn(cache=_binding_cache(binding), **_tensors(binding, 0)[call], **more)
    assert len(entered) == 2 and len(recorder.calls) == 2


def test_a_stream_of_another_gpu_is_refused(lib):
    from types import SimpleNamespace

    import gemm_mnb_gemv_gb300 as mnb
    stream = SimpleNamespace(device=SimpleNamespace(index=1), cuda_stream=5)
    assert mnb._raw_stream(1, stream) == 5
    with pytest.raises(ValueError, match="stream"):
        mnb._raw_stream(0, stream)

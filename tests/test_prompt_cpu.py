"""Rotary positions, prompt chunks, gathered weights and eviction: refusals before any device access, the binding's
checks, struct layouts and the frequency helpers (no GPU)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from sparse_attention_indexer_spin_gb300 import spin

A = ctypes.c_void_p(256)    # an aligned address that is never read
ODD = ctypes.c_void_p(258)
HALF = ctypes.c_void_p(264)


def err():
    return spin.lib().spin_last_error_string().decode()


def kv_cfg(**kw):
    f = dict(n_req=2, max_slots=100, max_rows=2, n_heads=8, kv_heads=2, head_dim=64, dtype="bf16")
    f.update(kw)
    return spin.make_kv_config(**f)


# ----------------------------------------------------------------------------------- rotary positions

def rope_call(code, word, cfg=None, rows=None, n_rows=None, T=4, positions=A, turns=A, **kw):
    f = dict(head_dim=64, dtype="bf16")
    f.update(kw)
    cfg = cfg or spin.make_rope_config(**f)
    rows = [(256, 1 << 20, 512, 512, 8)] if rows is None else rows
    arr = (spin.SpinRopeRows * max(1, len(rows)))(*[spin.SpinRopeRows(*r) for r in rows])
    rc = spin.lib().spin_rope(ctypes.byref(cfg), arr, len(rows) if n_rows is None else n_rows, T, positions, turns, None)
    assert rc == code, (rc, err())
    assert word in err()


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 1, 1), ("head_dim", 1025, 1), ("rot_dim", 0, 1), ("rot_dim", 3, 1), ("rot_dim", 66, 1),
    ("rot_first", -1, 1), ("rot_first", 2, 1), ("layout", 2, 1), ("dtype", 2, 4), ("dtype", 7, 4),
    ("magnitude", float("nan"), 1), ("magnitude", float("inf"), 1)])
def test_rope_config(spin_lib, field, value, code):
    cfg = spin.make_rope_config(64, "bf16")
    setattr(cfg, field, value)
    rope_call(code, "", cfg)
    assert err()


def test_rope_refusals(spin_lib):
    L = spin.lib()
    assert L.spin_rope(None, None, 1, 1, A, A, None) == 1 and "cfg" in err()
    cfg = spin.make_rope_config(64, "bf16")
    assert L.spin_rope(ctypes.byref(cfg), None, 1, 1, A, A, None) == 1 and "rows" in err()
    rope_call(1, "n_rows", rows=[], n_rows=0)
    rope_call(1, "n_rows", rows=[(256, 256, 512, 512, 8)] * 5)
    rope_call(1, "heads", rows=[(256, 256, 512, 512, 0)])
    rope_call(1, "heads", rows=[(256, 256, 1 << 20, 1 << 20, 1025)])
    rope_call(2, "strides", rows=[(256, 256, 511, 512, 8)])
    rope_call(2, "strides", rows=[(256, 256, 512, 511, 8)])
    rope_call(2, "strides", rows=[(256, 256, (1 << 30) + 1, 512, 8)])
    rope_call(1, "non-NULL", rows=[(None, 256, 512, 512, 8)])
    rope_call(1, "non-NULL", rows=[(256, None, 512, 512, 8)])
    rope_call(1, "aligned", rows=[(257, 257, 512, 512, 8)])
    rope_call(1, "aligned", dtype="f32", rows=[(258, 258, 512, 512, 8)])
    rope_call(3, "n_tokens", T=-1)
    rope_call(3, "n_tokens", T=1 << 31)
    rope_call(1, "non-NULL", positions=None)
    rope_call(1, "non-NULL", turns=None)
    rope_call(1, "aligned", positions=ODD)
    rope_call(1, "aligned", turns=ctypes.c_void_p(260))
    # overlaps: a token's row is 1024 bytes here, four tokens of it
    rope_call(1, "overlaps", rows=[(4096, 4096 + 1024, 512, 512, 8)])
    rope_call(1, "overlaps", rows=[(4096, 4096, 512, 1024, 8)])
    rope_call(1, "overlaps", rows=[(4096, 1 << 20, 512, 512, 8), (1 << 21, (1 << 20) + 2, 512, 512, 8)])
    rope_call(1, "overlaps", rows=[(4096, 4096, 512, 512, 8), (4096, 1 << 20, 512, 512, 8)])
    # side by side in one buffer is fine until the second reaches into the next token's first
    rope_call(1, "overlaps", rows=[(4096, 4096, 1024, 1024, 8), (5120, 5120, 1024, 1024, 9)])
    rope_call(1, "overlaps", rows=[(5120, 5120, 1024, 1024, 9), (4096, 4096, 1024, 1024, 8)])
    assert L.spin_rope(ctypes.byref(cfg), (spin.SpinRopeRows * 1)(spin.SpinRopeRows(None, None, 512, 512, 8)), 1, 0, None,
                       None, None) == 0


def test_rope_binding(spin_lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    cfg, x = spin.make_rope_config(64, "bf16"), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    p, t = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    for bad in ([x], [x.float()], [x[:2]], [x[:, 0]]):
        with pytest.raises(spin.SpinError):
            spin.rope(cfg, bad, p, t)
    with pytest.raises(spin.SpinError, match="as many"):
        spin.rope(cfg, [x], p, t, [])


def test_struct_layouts(tmp_path):
    """The binding's structs have the C structs' sizes and offsets."""
    src, want = ["#include <stdio.h>", "#include <stddef.h>", '#include "spin.h"', "int main(void) {"], []
    for c, s in (("spin_rope_config", spin.SpinRopeConfig), ("spin_rope_rows", spin.SpinRopeRows)):
        src.append('printf("%%zu ", sizeof(%s));' % c)
        want.append(ctypes.sizeof(s))
        for name, _ in s._fields_:
            src.append('printf("%%zu ", offsetof(%s, %s));' % (c, name.rstrip("_")))
            want.append(getattr(s, name).offset)
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(spin.HEADER), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want


def test_rope_frequencies():
    f, m = spin.rope_frequencies(64, 1e4)
    assert m == 1.0 and f.dtype is torch.float64 and f.shape == (32,)
    assert torch.allclose(f, torch.tensor([1e4 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64), rtol=1e-14)
    g, _ = spin.rope_frequencies(64, 1e4, "linear", 4.0)
    assert torch.allclose(g, f / 4, rtol=1e-14)
    g, _ = spin.rope_frequencies(64, 1e4, "base", 4.0)
    assert g[0] == 1.0 and math.isclose(float(g[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    g, m = spin.rope_frequencies(64, 1e4, "parts", 8.0, original=4096)
    turns = f * 4096 / (2 * math.pi)
    ratio = g / f
    assert (ratio[turns > 40] == 1.0).all() and torch.allclose(ratio[turns < 0.9], torch.tensor(0.125, dtype=torch.float64))
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all() and math.isclose(m, 0.1 * math.log(8) + 1)
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, theta=0.0), dict(rot_dim=8, factor=2.0),
                dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, scaling="none"),
                dict(rot_dim=8, scaling="parts", factor=2.0), dict(rot_dim=8, scaling="parts", original=9, fast=1.0)):
        with pytest.raises(spin.SpinError):
            spin.rope_frequencies(**bad)


@pytest.mark.parametrize("original,fast,slow", [(4, 32.0, 1.0), (6, 2.0, 1.0), (6.2, 32.0, 1.0), (100, 64.0, 16.0), (4096, 32.0, 1.0), (200, 64.0, 31.0)])
def test_rope_frequencies_by_parts_at_the_ends(original, fast, slow):
    """Pairs that turn `slow` times or less within the original context are divided, the first one among them."""
    f, _ = spin.rope_frequencies(64, 1e4)
    g, _ = spin.rope_frequencies(64, 1e4, "parts", 8.0, original=original, fast=fast, slow=slow)
    turns = f * original / (2 * math.pi)
    assert torch.allclose((g / f)[turns <= slow], torch.tensor(0.125, dtype=torch.float64), rtol=1e-14)
    assert (g[turns >= fast] == f[turns >= fast]).all()


def test_rope_frequencies_of_no_meaning():
    for bad in (dict(theta=math.inf), dict(theta=math.nan), dict(scaling="linear", factor=math.inf), dict(scaling="base", factor=math.nan),
                dict(theta=0.5, scaling="parts", factor=2.0, original=4096), dict(scaling="parts", factor=2.0, original=math.inf)):
        with pytest.raises(spin.SpinError):
            spin.rope_frequencies(8, **bad)


def test_rope_turns():
    t = spin.rope_turns(torch.tensor([0.0, math.pi, 2 * math.pi, -math.pi / 2, 1.0], dtype=torch.float64), "cpu")
    u = [x % (1 << 64) for x in t.tolist()]
    assert u[0] == 0 and abs(u[1] - (1 << 63)) < 1 << 12 and min(u[2], (1 << 64) - u[2]) < 1 << 13
    assert abs(u[3] - 3 * (1 << 62)) < 1 << 12
    assert abs(u[4] / 2.0 ** 64 * 2 * math.pi - 1.0) < 1e-15
    for bad in (torch.zeros(3), torch.zeros((2, 2), dtype=torch.float64), torch.tensor([math.inf], dtype=torch.float64)):
        with pytest.raises(spin.SpinError):
            spin.rope_turns(bad, "cpu")


# ------------------------------------------------------------------------------ chunks of new tokens

WS = 1 << 50


def prefill_call(code, word, cfg=None, **kw):
    a = dict(q=A, T=4, start=A, max_new=4, before=A, k=A, v=A, ks=A, vs=A, n_pages=4, bt=A, stride=2, out=A, lse=A, ws=A,
             bytes=WS, status=None)
    a.update(kw)
    rc = spin.lib().spin_kv_prefill(ctypes.byref(cfg or kv_cfg()), *a.values(), None)
    assert rc == code and word in err(), (rc, err())


def weigh_call(code, word, cfg=None, **kw):
    a = dict(q=A, lse=A, T=4, start=A, max_new=4, before=A, k=A, ks=A, n_pages=4, bt=A, stride=2, decay=1.0, weight=A, ws=A,
             bytes=WS, status=None)
    a.update(kw)
    rc = spin.lib().spin_kv_weigh(ctypes.byref(cfg or kv_cfg()), *a.values(), None)
    assert rc == code and word in err(), (rc, err())


@pytest.mark.parametrize("field,value,code", [
    ("n_req", 0, 1), ("max_slots", 0, 3), ("block", 32, 1), ("n_heads", 129, 1), ("kv_heads", 3, 2), ("head_dim", 72, 1),
    ("dtype", 2, 4), ("softmax_scale", float("nan"), 1), ("reserved", 1, 1)])
def test_chunk_config(spin_lib, field, value, code):
    cfg = kv_cfg()
    setattr(cfg, field, value)
    size = ctypes.c_size_t(0)
    for f in (spin.lib().spin_kv_prefill_workspace_size, spin.lib().spin_kv_weigh_workspace_size):
        assert f(ctypes.byref(cfg), 4, 4, ctypes.byref(size)) == code and err()
    prefill_call(code, "", cfg)
    weigh_call(code, "", cfg)


def test_chunk_refusals(spin_lib):
    for call, words, wide in ((prefill_call, ("start", "before", "bt", "lse", "ks", "vs"), ("q", "out", "k", "v")),
                              (weigh_call, ("start", "before", "bt", "lse", "ks", "weight"), ("q", "k"))):
        for name in (*words, *wide):
            if not (call is prefill_call and name == "lse"):
                call(1, "NULL", **{name: None})
        for name in words:
            call(1, "4-byte aligned", **{name: ODD})
        call(1, "4-byte aligned", status=ODD)
        for name in wide:
            call(1, "16-byte aligned", **{name: HALF})
        call(3, "n_tokens", T=-1)
        call(3, "n_tokens", T=(1 << 24) + 1)
        call(3, "n_heads", T=1 << 24, cfg=kv_cfg(n_heads=128))
        call(1, "max_new", max_new=-1)
        call(1, "max_new", max_new=101)
        call(3, "n_pages", n_pages=-1)
        call(2, "bt_stride", stride=1)
        call(1, "workspace", ws=None)
        call(1, "workspace", bytes=0)
        call(1, "256-byte aligned", ws=HALF)
    for bad in (float("nan"), float("inf")):
        weigh_call(1, "decay", decay=bad)
    for f in (spin.lib().spin_kv_prefill_workspace_size, spin.lib().spin_kv_weigh_workspace_size):
        assert f(ctypes.byref(kv_cfg()), 4, 4, None) == 1 and "bytes" in err()


def test_chunk_binding(spin_lib, monkeypatch):
    """Tensors of other types, shapes or devices are refused before the call."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    cfg = kv_cfg()
    q, i = torch.zeros((4, 8, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(spin.SpinError):
        spin.kv_prefill(cfg, q, i, 4, i[:2], q, q, q, q, q, q, None, torch.zeros(1), None)
    with pytest.raises(spin.SpinError):
        spin.kv_weigh(cfg, q, q, i, 4, i[:2], q, q, q, 1.0, q, torch.zeros(1), None)


def test_prompt_run_refusals(spin_lib, monkeypatch):
    """A chunk of run_prompt is refused before its first launch."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)   # (a host tensor's device number)
    R, T, W, h, kvh, d = 2, 6, 3, 8, 2, 64
    cfg = spin.make_kv_config(R, 64 * W, 1, h, kvh, d, "bf16")
    cache = spin.KvCache(5, kvh, d, device="cpu")
    freq, _ = spin.rope_frequencies(d)
    core = spin.PromptAttention(cfg, cache, 8, 4, spin.make_rope_config(d, "bf16"), spin.rope_turns(freq, device="cpu"), device="cpu")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kv = (torch.zeros((T, x, d), dtype=torch.bfloat16) for x in (h, kvh))
    good = dict(q=q, k=kv, v=kv, positions=i32(T), new_start=i32(R + 1), max_new=3, n_before=i32(R), block_table=i32(R, W),
                status=i32(1), weight=torch.zeros((R, 64 * W)))
    core.check(**good)
    core.check(**{**good, "weight": None, "status": None})
    for name, bad in (("q", q.float()), ("q", q[:5]), ("q", torch.zeros((9, h, d), dtype=torch.bfloat16)), ("k", q), ("k", kv[1:]),
                      ("v", kv[:, :1]), ("positions", None), ("positions", i32(T + 1)), ("positions", i32(T).long()),
                      ("new_start", i32(R)), ("max_new", 5), ("max_new", -1), ("n_before", i32(R + 1)), ("block_table", i32(R, W - 1)),
                      ("block_table", i32(R + 1, W)), ("status", i32(2)), ("weight", torch.zeros((R, 64))),
                      ("weight", torch.zeros((R, 64 * W)).double())):
        with pytest.raises(spin.SpinError):
            core.check(**{**good, name: bad})
    plain = spin.PromptAttention(cfg, cache, 8, 4, device="cpu")
    plain.check(**{**good, "positions": None})
    with pytest.raises(spin.SpinError):
        plain.check(**good)
    for rope in (spin.make_rope_config(32, "bf16"), spin.make_rope_config(d, "f32")):
        with pytest.raises(spin.SpinError):
            spin.PromptAttention(cfg, cache, 8, 4, rope, core.turns, device="cpu")
    with pytest.raises(spin.SpinError):
        spin.PromptAttention(cfg, cache, 8, 4, core.rope, device="cpu")
    with pytest.raises(spin.SpinError):
        spin.PromptAttention(cfg, cache, -1, 4, device="cpu")


@pytest.mark.parametrize("decay", [float("nan"), float("inf"), -float("inf"), 1e39, None])
def test_prompt_run_refuses_a_decay_before_it_writes(spin_lib, monkeypatch, decay):
    """The last step's argument is looked at before the first step; a decay that no step reads is not."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    called = []
    for name in ("rope", "kv_append", "kv_prefill", "kv_weigh"):
        monkeypatch.setattr(spin, name, lambda *a, name=name: called.append(name))
    cfg = spin.make_kv_config(1, 64, 1, 2, 1, 16, "bf16")
    core = spin.PromptAttention(cfg, spin.KvCache(2, 1, 16, device="cpu"), 4, 4, device="cpu")
    q, kv = (torch.zeros((4, h, 16), dtype=torch.bfloat16) for h in (2, 1))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    call = lambda **kw: spin.run_prompt(core, q, kv, kv, i32(0, 4), 4, i32(0), i32(0)[None], None, **kw)  # noqa: E731
    with pytest.raises((spin.SpinError, TypeError)):
        call(weight=torch.zeros((1, 64)), decay=decay)
    assert not called
    call(decay=decay)
    call(weight=torch.zeros((1, 64)), decay=-2.0)
    assert called == ["kv_append", "kv_prefill"] * 2 + ["kv_weigh"]


def test_prompt_run_refuses_buffers_elsewhere(spin_lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    cfg = spin.make_kv_config(1, 64, 1, 2, 1, 16, "bf16")
    core = spin.PromptAttention(cfg, spin.KvCache(2, 1, 16, device="cpu"), 4, 4, device="cpu")
    q, kv = (torch.zeros((4, h, 16), dtype=torch.bfloat16) for h in (2, 1))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    args = (q, kv, kv, None, i32(0, 4), 4, i32(0), i32(0)[None], None, None)
    core.check(*args)
    core.out = core.out.to("meta")      # (a device of another number)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda x: 1 if x.is_meta else -1)
    with pytest.raises(spin.SpinError, match="buffers"):
        core.check(*args)


# ------------------------------------------------------------------------------------------- eviction

def evict_call(code, word, **kw):
    a = dict(R=2, n_pages=4, table=A, stride=3, n=A, w=ctypes.c_void_p(1 << 20), out=ctypes.c_void_p(1 << 21), keep=A, first=1,
             last=1, ref=A, kept=A, ws=A, bytes=WS, status=None)
    a.update(kw)
    rc = spin.lib().spin_pages_evict(*a.values(), None)
    assert rc == code and word in err(), (rc, err())


def test_evict_refusals(spin_lib):
    for name in ("table", "n", "w", "out", "keep", "ref", "kept"):
        evict_call(1, "non-NULL", **{name: None})
    for name in ("table", "n", "keep", "ref", "kept", "status"):
        evict_call(1, "4-byte aligned", **{name: ODD})
    for name in ("w", "out"):
        evict_call(1, "16-byte aligned", **{name: HALF})
    evict_call(1, "n_req", R=0)
    evict_call(1, "n_req", R=65536)
    evict_call(3, "n_pages", n_pages=0)
    evict_call(3, "bt_stride", stride=0)
    evict_call(3, "bt_stride", stride=(1 << 18) + 1)
    evict_call(1, "n_first", first=-1)
    evict_call(1, "n_last", last=0)
    evict_call(1, "overlap", out=ctypes.c_void_p((1 << 20) + 16))
    evict_call(1, "overlap", out=ctypes.c_void_p(1 << 20))
    evict_call(1, "workspace", ws=None)
    evict_call(1, "workspace", bytes=0)
    evict_call(1, "256-byte aligned", ws=HALF)
    size = ctypes.c_size_t(0)
    f = spin.lib().spin_pages_evict_workspace_size
    assert f(0, 3, ctypes.byref(size)) == 1 and f(2, 0, ctypes.byref(size)) == 3 and f(2, 3, None) == 1
    assert f(2, 3, ctypes.byref(size)) == 0 and size.value >= 24


def test_evict_binding(spin_lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    i = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(spin.SpinError):
        spin.pages_evict(i, i[:, 0], i, i, i[:, 0], 1, 1, i[0], i, torch.zeros(1), None)
    with pytest.raises(spin.SpinError):
        spin.pages_evict(i[0], i[:, 0], i, i, i[:, 0], 1, 1, i[0], i, torch.zeros(1), None)

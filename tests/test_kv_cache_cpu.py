"""KV-cache and page calls: refusals before any device access, the binding's checks, and the
oracle's encoder against torch's conversion (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin


def cfg_of(**kw):
    f = dict(n_req=2, max_slots=100, max_rows=2, n_heads=8, kv_heads=2, head_dim=64, dtype="bf16")
    f.update(kw)
    return spin.make_kv_config(**f)


def err():
    return spin.lib().spin_last_error_string().decode()


A = ctypes.c_void_p(256)    # an aligned address that is never read


@pytest.mark.parametrize("field,value,code", [
    ("n_req", 0, 1), ("n_req", 65536, 1), ("max_slots", 0, 3), ("max_slots", (1 << 24) + 1, 3), ("max_rows", 0, 1),
    ("max_rows", 9, 1), ("block", 32, 1), ("n_heads", 0, 1), ("n_heads", 129, 1), ("kv_heads", 3, 2),
    ("kv_heads", 0, 2), ("kv_heads", 16, 2), ("head_dim", 0, 1), ("head_dim", 72, 1), ("head_dim", 272, 1),
    ("dtype", 2, 4), ("dtype", 4, 4), ("softmax_scale", float("nan"), 1), ("softmax_scale", float("inf"), 1),
    ("reserved", 1, 1)])
def test_config_validation(spin_lib, field, value, code):
    cfg = cfg_of()
    setattr(cfg, field, value)
    size = ctypes.c_size_t(0)
    L = spin.lib()
    assert L.spin_kv_workspace_size(ctypes.byref(cfg), 1, 0, ctypes.byref(size)) == code and err()
    assert L.spin_kv_attend(ctypes.byref(cfg), A, A, A, A, A, 1, A, 2, A, 1, None, 0, A, None, A, 1 << 40, None,
                            None) == code
    assert L.spin_kv_append(ctypes.byref(cfg), A, A, 1, A, 1, A, A, A, A, A, 1, A, 2, None, None) == code


def test_null_config(spin_lib):
    assert spin.lib().spin_kv_workspace_size(None, 1, 0, None) == 1 and "cfg" in err()


def test_attend_refusals(spin_lib):
    cfg, L = cfg_of(), spin.lib()
    ws = 1 << 40

    def call(code, word, **kw):
        a = dict(q=A, k=A, v=A, ks=A, vs=A, n_pages=4, bt=A, stride=2, n=A, rows=1, idx=None, top_k=0, out=A, ws=A,
                 bytes=ws)
        a.update(kw)
        assert L.spin_kv_attend(ctypes.byref(cfg), a["q"], a["k"], a["v"], a["ks"], a["vs"], a["n_pages"], a["bt"],
                                a["stride"], a["n"], a["rows"], a["idx"], a["top_k"], a["out"], None, a["ws"],
                                a["bytes"], None, None) == code
        assert word in err()

    odd = ctypes.c_void_p(264)
    for name in ("q", "k", "v", "ks", "vs", "bt", "n", "out"):
        call(1, "non-NULL", **{name: None})
    for name in ("q", "out", "k", "v"):
        call(1, "16-byte aligned", **{name: odd})
    call(1, "4-byte aligned", ks=ctypes.c_void_p(258))
    call(2, "rows", rows=0)
    call(2, "rows", rows=3)
    call(2, "bt_stride", stride=1)
    call(1, "top_k", top_k=-1)
    call(1, "top_k", top_k=16385, idx=A)
    call(1, "go together", top_k=5)
    call(1, "go together", idx=A)
    call(3, "n_pages", n_pages=-1)
    call(3, "n_pages", n_pages=(1 << 30) + 1)
    call(1, "workspace", ws=None)
    call(1, "workspace", bytes=0)
    call(1, "256-byte aligned", ws=odd)


def test_append_refusals(spin_lib):
    cfg, L = cfg_of(), spin.lib()

    def call(code, word, **kw):
        a = dict(x=A, y=A, T=1, start=A, max_new=1, before=A, k=A, v=A, ks=A, vs=A, n_pages=4, bt=A, stride=2)
        a.update(kw)
        assert L.spin_kv_append(ctypes.byref(cfg), a["x"], a["y"], a["T"], a["start"], a["max_new"], a["before"],
                                a["k"], a["v"], a["ks"], a["vs"], a["n_pages"], a["bt"], a["stride"], None,
                                None) == code
        assert word in err()

    for name in ("x", "y", "start", "before", "k", "v", "ks", "vs", "bt"):
        call(1, "NULL", **{name: None})
    call(1, "16-byte aligned", x=ctypes.c_void_p(264))
    call(3, "n_tokens", T=-1)
    call(3, "n_tokens", T=1 << 31)
    call(1, "max_new", max_new=-1)
    call(1, "max_new", max_new=101)
    call(2, "bt_stride", stride=1)


def test_page_refusals(spin_lib):
    L = spin.lib()
    pool = (spin.SpinPagePool * 1)(spin.SpinPagePool(256, 16))
    ws = 1 << 40

    def calls(n_req=1, n_pages=4, table=A, stride=2, ref=A):
        yield L.spin_pages_fork(n_req, n_pages, ctypes.c_void_p(1 << 30), stride, A, table, ref, None, None)
        yield L.spin_pages_free(n_req, n_pages, table, stride, A, ref, None, None)
        yield L.spin_pages_reserve(n_req, n_pages, table, stride, A, A, ref, pool, 1, A, A, ws, None, None)
        yield L.spin_pages_compact(n_req, n_pages, table, stride, ref, pool, 1, A, A, ws, None, None)

    for kw, code in (({"n_req": 0}, 1), ({"n_req": 65536}, 1), ({"n_pages": 0}, 3), ({"n_pages": (1 << 30) + 1}, 3),
                     ({"stride": 0}, 3), ({"stride": (1 << 18) + 1}, 3), ({"table": None}, 1), ({"ref": None}, 1),
                     ({"ref": ctypes.c_void_p(257)}, 1)):
        for rc in calls(**kw):
            assert rc == code and err()
    # tables that overlap without being the same
    assert L.spin_pages_fork(4, 4, ctypes.c_void_p(256), 2, A, ctypes.c_void_p(272), A, None, None) == 1
    assert "overlap" in err()
    assert L.spin_pages_fork(1, 4, None, 2, A, A, A, None, None) == 1
    assert L.spin_pages_fork(1, 4, A, 2, None, A, A, None, None) == 1
    assert L.spin_pages_free(1, 4, A, 2, None, A, None, None) == 1

    def reserve(pools, n, w=A, b=ws, granted=A):
        return L.spin_pages_reserve(1, 4, A, 2, A, A, A, pools, n, granted, w, b, None, None)

    def compact(pools, n, w=A, b=ws, live=A):
        return L.spin_pages_compact(1, 4, A, 2, A, pools, n, live, w, b, None, None)

    for f in (reserve, compact):
        assert f(None, 1) == 1 and f(pool, -1) == 1 and f(pool, 17) == 1
        for data, nbytes in ((None, 16), (258, 16), (256, 0), (256, 6), (256, (1 << 30) + 4)):
            assert f((spin.SpinPagePool * 1)(spin.SpinPagePool(data, nbytes)), 1) == 1 and "pool 0" in err()
        assert f(pool, 1, w=None) == 1 and f(pool, 1, b=8) == 1 and f(pool, 1, w=ctypes.c_void_p(260)) == 1
        assert f(pool, 1, A, ws, None) == 1
    size = ctypes.c_size_t(0)
    assert L.spin_pages_workspace_size(0, 4, ctypes.byref(size)) == 1
    assert L.spin_pages_workspace_size(1, 0, ctypes.byref(size)) == 3
    assert L.spin_pages_workspace_size(1, 4, None) == 1
    assert L.spin_pages_workspace_size(3, 1000, ctypes.byref(size)) == 0 and size.value >= 4 * 3000


def test_struct_layouts(spin_lib, tmp_path):
    """The binding's structs have the C structs' size and offsets."""
    import os
    import subprocess
    want, lines = [], []
    for name, cls in (("spin_kv_config", spin.SpinKvConfig), ("spin_page_pool", spin.SpinPagePool)):
        lines.append('printf("%%zu ", sizeof(%s));' % name)
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append('printf("%%zu ", offsetof(%s, %s));' % (name, f))
            want.append(getattr(cls, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spin.h"\nint main(void) {\n%s\nreturn 0;\n}\n'
                   % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(spin.HEADER), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def test_binding_refuses_wrong_tensors():
    """Shapes, types, devices and layouts are checked before an address is taken."""
    t = torch.zeros((4, 6), dtype=torch.int32)
    for bad in (dict(dtype=torch.float32), dict(shape=(4, 5)), dict(device=0), dict(t=t.t().contiguous().t())):
        kw = dict(t=t, dtype=torch.int32, shape=(4, 6), device=-1)
        kw.update(bad)
        with pytest.raises(spin.SpinError):
            spin._arg("x", **kw)
    assert spin._arg("x", t, torch.int32, (4, 6), -1) == t.data_ptr()
    with pytest.raises(spin.SpinError):
        spin.PagePools(t)              # not on a GPU


def test_oracle_e4m3_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, o.E4M3, equal_nan=True)
    x = np.random.default_rng(0).normal(size=20000) * 10.0 ** np.random.default_rng(1).uniform(-4, 2.6, 20000)
    x = np.concatenate([x, o.E4M3[:127], (o.E4M3[:126] + o.E4M3[1:127]) / 2, [-0.0, 447.9]]).clip(-448, 448)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.e4m3_encode(x.astype(np.float32)), want)
    assert o.e4m3_encode([np.inf, -np.inf, np.nan, 1e9]).tolist() == [126, 254, 127, 126]


def test_oracle_scale_rule():
    assert o.pow2_scale(448.0) == 1.0 and o.pow2_scale(448.1) == 2.0 and o.pow2_scale(0.0) == 0.0
    assert o.pow2_scale(2.0 ** -149) == 2.0 ** -126 and o.pow2_scale(1.0) == 2.0 ** -8


def test_oracle_pages_by_hand():
    table = np.array([[0, 1], [2, -1], [3, -1]], np.int32)
    ref = np.array([1, 1, 1, 1, 0, 0], np.int32)
    t, r = o.fork(table, [0, 0, -1], ref)
    assert t.tolist() == [[0, 1], [0, 1], [-1, -1]] and r.tolist() == [2, 2, 0, 0, 0, 0]
    pool = np.arange(6)[:, None].copy()
    # both sharers of the partly filled page 1 get copies; the page itself becomes free
    t, r, g = o.reserve(t, [70, 70, 0], [1, 1, 1], r, [pool])
    assert t.tolist() == [[0, 2], [0, 3], [4, -1]] and r.tolist() == [2, 0, 1, 1, 1, 0] and g.tolist() == [1, 1, 1]
    assert pool[:, 0].tolist() == [0, 1, 1, 1, 4, 5]
    t, r = o.free(t, [64, -1, 0], r)
    assert t.tolist() == [[0, -1], [0, 3], [-1, -1]] and r.tolist() == [2, 0, 0, 1, 0, 0]
    t, r, n = o.compact(t, r, [pool])
    assert t.tolist() == [[0, -1], [0, 1], [-1, -1]] and r.tolist() == [2, 1, 0, 0, 0, 0] and n == 2


def test_oracle_attention_by_hand():
    """One head, two slots with equal keys: the mean of their values, lse = s + ln 2."""
    k = np.zeros((2, 64, 1, 16), np.uint8)
    v = np.zeros((2, 64, 1, 16), np.uint8)
    k[1, :2] = 0x38                    # code of 1.0
    v[1, 0], v[1, 1] = 0x38, 0x40      # 1.0 and 2.0
    q = np.ones((1, 1, 1, 16))
    ks, vs = np.full((2, 1), 0.5, np.float32), np.full((2, 1), 2.0, np.float32)
    out, lse, info = o.attend(q, k, v, ks, vs, np.array([[1]]), np.array([[2]]), 0.25)
    assert np.allclose(out, 3.0) and np.allclose(lse, 0.25 * 0.5 * 16 + np.log(2))
    out, lse, _ = o.attend(q, k, v, ks, vs, np.array([[1]]), np.array([[2]]), 0.25, np.array([[[1, -1]]]))
    assert np.allclose(out, 4.0)
    out, lse, _ = o.attend(q, k, v, ks, vs, np.array([[1]]), np.array([[0]]), 0.25)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_oracle_appends_infinities_beside_nothing_finite():
    """Saturated under a scale of 0, and gone with the page's next finite value."""
    pool, scale = np.zeros((1, 64, 1, 16), np.uint8), np.zeros((1, 1), np.float32)
    x = np.zeros((1, 1, 16))
    x[0, 0, :3] = np.inf, -np.inf, np.nan
    o.append(x, [0, 1], [0], pool, scale, np.zeros((1, 1), np.int32))
    assert pool[0, 0, 0].tolist() == [126, 254, 127] + [0] * 13 and scale[0, 0] == 0
    o.append(np.ones((1, 1, 16)), [0, 1], [1], pool, scale, np.zeros((1, 1), np.int32))
    assert (pool[0, 0, 0] & 127).tolist() == [0, 0, 127] + [0] * 13 and scale[0, 0] == 2.0 ** -8


def test_page_copy_refusals(spin_lib):
    L, pool, ws = spin.lib(), (spin.SpinPagePool * 1)(spin.SpinPagePool(256, 16)), 1 << 40

    def copy(n_req=1, n_pages=4, pools=pool, n=1, w=A, b=ws):
        return L.spin_pages_copy(n_req, n_pages, pools, n, w, b, None, None)

    for kw, code in (({"n_req": 0}, 1), ({"n_req": 65536}, 1), ({"n_pages": 0}, 3), ({"n_pages": (1 << 30) + 1}, 3),
                     ({"pools": None}, 1), ({"n": -1}, 1), ({"n": 17}, 1), ({"w": None}, 1), ({"b": 8}, 1),
                     ({"w": ctypes.c_void_p(260)}, 1)):
        assert copy(**kw) == code and err()
    for data, nbytes in ((None, 16), (258, 16), (256, 0), (256, 6), (256, (1 << 30) + 4)):
        assert copy(pools=(spin.SpinPagePool * 1)(spin.SpinPagePool(data, nbytes))) == 1 and "pool 0" in err()


def test_run_step_refuses_a_core_attention_without_queries(monkeypatch):
    """As an error of the binding, before anything is launched."""
    for name in ("select_blocks", "indexer_score", "topk", "update_ema"):
        monkeypatch.setattr(spin, name, lambda *a, **k: pytest.fail("launched"))
    core, buf = object.__new__(spin.CoreAttention), object.__new__(spin.StepBuffers)
    buf.rows = 1
    with pytest.raises(spin.SpinError, match="core_q"):
        spin.run_step(None, None, buf, None, None, None, None, 0, None, None, None, core=core)


def test_words_at_odd_addresses_are_refused(spin_lib):
    """Every array of 4-byte words, one at a time (an odd address would fault on the device)."""
    L, cfg, odd, ws = spin.lib(), cfg_of(), ctypes.c_void_p(258), 1 << 40
    pool = (spin.SpinPagePool * 1)(spin.SpinPagePool(256, 16))
    far = ctypes.c_void_p(1 << 30)

    def attend(n=A, idx=A, lse=A, status=A):
        return L.spin_kv_attend(cfg, A, A, A, A, A, 4, A, 2, n, 1, idx, 1, A, lse, A, ws, status, None)

    def append(start=A, before=A, status=A):
        return L.spin_kv_append(cfg, A, A, 1, start, 1, before, A, A, A, A, 4, A, 2, status, None)

    def fork(table_in=far, parent=A, status=A):
        return L.spin_pages_fork(1, 4, table_in, 2, parent, A, A, status, None)

    def free(keep=A, status=A):
        return L.spin_pages_free(1, 4, A, 2, keep, A, status, None)

    def reserve(n=A, new=A, granted=A, status=A):
        return L.spin_pages_reserve(1, 4, A, 2, n, new, A, pool, 1, granted, A, ws, status, None)

    def compact(live=A, status=A):
        return L.spin_pages_compact(1, 4, A, 2, A, pool, 1, live, A, ws, status, None)

    def copy(status=A):
        return L.spin_pages_copy(1, 4, pool, 1, A, ws, status, None)

    for f in (attend, append, fork, free, reserve, compact, copy):
        names = f.__code__.co_varnames[:f.__code__.co_argcount]
        for name in names:
            at = ctypes.c_void_p((1 << 30) + 2) if name == "table_in" else odd
            assert f(**{name: at}) == 1 and "4-byte aligned" in err(), (f.__name__, name)


def test_page_calls_refuse_tables_and_counts_of_other_dimensions():
    t, ref, x = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for table, r in ((t[0], ref), (t[None], ref), (t, ref[None])):
        for call in (lambda: spin.pages_fork(table, x, table, r, None), lambda: spin.pages_free(table, x, r, None),
                     lambda: spin.pages_reserve(table, x, x, r, None, x, x, None),
                     lambda: spin.pages_compact(table, r, None, x, x, None)):
            with pytest.raises(spin.SpinError, match="block table"):
                call()

"""The paged cache without a GPU: refusals of the C entry points, the bindings' structs, the oracle's own pins."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT
from oracle import pages as op


_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


class Chunks(ctypes.Structure):
    _fields_ = [("q_start", _P), ("rows", _P), ("n_seqs", _I), ("total_q", _I)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_token_stride", _L), ("k_head_stride", _L), ("v_token_stride", _L),
                ("v_head_stride", _L), ("q", _P), ("q_out", _P), ("q_token_stride", _L), ("q_head_stride", _L),
                ("q_out_token_stride", _L), ("q_out_head_stride", _L), ("n_q_heads", _I), ("rope", _P), ("positions", _P),
                ("pos_stride", _L)]


class AttendArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("out", _P), ("lse", _P), ("q_token_stride", _L), ("q_head_stride", _L), ("out_token_stride", _L),
                ("out_head_stride", _L), ("n_q_heads", _I), ("causal", _I), ("max_q_len", _I), ("scale", ctypes.c_float)]


@pytest.fixture(scope="module")
def paged():
    import tiered_quantize_evict_gb300 as qe
    pytest.importorskip("torch")
    if not os.path.exists(qe.LIB_PATH):
        from tiered_quantize_evict_gb300.build import build_library
        build_library()
    from tiered_quantize_evict_gb300 import paged
    return paged


@pytest.fixture()
def env(paged):
    """Valid arguments (addresses are never followed: every call here is refused, or has nothing to do)."""
    import tiered_quantize_evict_gb300 as qe
    class E:
        lib = qe.load_library()
        pages = paged._Pages(4096, 8192, 0, 0, 2, 10, 2, 16, 64, 20480, 2048, 1024, 64, 16)
        table = paged._Table(4096, 4096, 4096, 8, 4, 8)
        chunks = Chunks(4096, None, 2, 5)
        append = AppendArgs(4096, 4096, 128, 64, 128, 64, 4096, 4096, 256, 64, 256, 64, 4, None, None, 0)
        attend = AttendArgs(4096, 4096, None, 256, 64, 256, 64, 4, 1, 0, 0.125)
        rope = paged._Rope(64, 0, 1)

        def run(self, what, layer=0, ws=4096, nb=1 << 40, n=3, null=()):
            r = lambda x: None if x in null else ctypes.byref(getattr(self, x))  # noqa: E731
            g, t, c = r("pages"), r("table"), r("chunks")
            if what == "append":
                st = self.lib.qe_pages_append(g, layer, t, c, r("append"), None)
            elif what == "attend":
                st = self.lib.qe_pages_attend(g, layer, t, c, r("attend"), ws, nb, None)
            elif what in ("resize", "fork"):
                st = getattr(self.lib, "qe_pages_" + what)(g, t, 4096, 4096, n, ws, nb, None)
            elif what == "compact":
                st = self.lib.qe_pages_compact(g, t, None, None, None, ws, nb, None)
            elif what == "copy":
                st = self.lib.qe_pages_copy(g, 4096, 4096, n, None)
            else:
                st = self.lib.qe_pages_gather(g, layer, t, None, 2, 0, n, 4096, 4096, None)
            return st, self.lib.qe_last_error(None).decode()
    return E()


ALL = ["append", "attend", "resize", "fork", "compact", "copy", "gather"]


def refused(env, what, text, **kw):
    import tiered_quantize_evict_gb300 as qe
    st, msg = env.run(what, **kw)
    assert st == qe.QE_ERR_INVALID_ARG and text in msg, (what, st, msg)


@pytest.mark.parametrize("field,value,text", [
    ("k", None, "null"), ("v", 8200, "aligned"), ("dtype", 2, "dtype"), ("device", -1, "device"), ("n_layers", 0, "n_layers"),
    ("n_pages", 0, "n_pages"), ("n_kv_heads", 0, "n_kv_heads"), ("page_size", 8, "page_size"), ("page_size", 48, "page_size"),
    ("page_size", 512, "page_size"), ("head_dim", 96, "head_dim"), ("layer_stride", 0, "strides"), ("page_stride", -2048, "strides"),
    ("head_stride", 1028, "strides"), ("token_stride", 32, "strides"), ("err", 18, "err")])
def test_pool_is_checked_by_every_call(env, field, value, text):
    setattr(env.pages, field, value)
    for what in ALL:
        refused(env, what, text)


@pytest.mark.parametrize("field,value,text", [
    ("table", None, "null"), ("kv_len", None, "null"), ("kv_len", 4098, "aligned"), ("n_rows", 0, "n_rows"), ("max_pages", 0, "max_pages"),
    ("row_stride", 7, "row_stride")])
def test_table_is_checked(env, field, value, text):
    setattr(env.table, field, value)
    for what in ALL:
        if what != "copy":
            refused(env, what, text)


def test_refs_are_needed_where_pages_are_managed(env):
    env.table.refs = None
    for what in ("resize", "fork", "compact"):
        refused(env, what, "refs")


def test_managed_tables_are_counted_in_32_bits(env):
    env.table.n_rows, env.table.max_pages, env.table.row_stride = 2 ** 15, 2 ** 16, 2 ** 16
    for what in ("resize", "fork", "compact"):
        refused(env, what, "too large")


@pytest.mark.parametrize("field,value,text", [("q_start", None, "q_start"), ("n_seqs", -1, "n_seqs"), ("n_seqs", 65537, "n_seqs"),
                                              ("total_q", -1, "total_q"), ("total_q", 2 ** 30 + 1, "total_q"), ("rows", 4098, "aligned")])
def test_chunks_are_checked(env, field, value, text):
    setattr(env.chunks, field, value)
    refused(env, "append", text)
    refused(env, "attend", text)


@pytest.mark.parametrize("field,value,text", [
    ("q", None, "q is null"), ("out", None, "out is null"), ("q", 4100, "q must be 16-byte"), ("q_token_stride", 4, "q: strides"),
    ("out_head_stride", 68, "out: strides"), ("n_q_heads", 3, "multiple"), ("n_q_heads", 0, "multiple"), ("n_q_heads", 258, "multiple"),
    ("scale", 0.0, "scale"), ("scale", -1.0, "scale"), ("scale", math.inf, "scale"), ("scale", math.nan, "scale"), ("max_q_len", -1, "max_q_len"),
    ("lse", 4098, "lse")])
def test_attend_arguments(env, field, value, text):
    setattr(env.attend, field, value)
    refused(env, "attend", text)


def test_attend_workspace(env):
    import tiered_quantize_evict_gb300 as qe
    n = ctypes.c_size_t(7)
    ask = lambda: env.lib.qe_pages_attend_workspace(ctypes.byref(env.pages), ctypes.byref(env.table), ctypes.byref(n))  # noqa: E731
    assert ask() == qe.QE_OK and n.value == 0       # 8 pages of 16 tokens: never split
    env.table.max_pages, env.table.row_stride = 1000, 1000
    assert ask() in (qe.QE_OK, qe.QE_ERR_CUDA)      # else its size goes by the device
    assert env.lib.qe_pages_attend_workspace(ctypes.byref(env.pages), ctypes.byref(env.table), None) == qe.QE_ERR_INVALID_ARG
    refused(env, "resize", "workspace", nb=64)
    refused(env, "fork", "workspace", ws=None)
    refused(env, "compact", "aligned", ws=4100)


@pytest.mark.parametrize("field,value,text", [
    ("k", None, "k is null"), ("v", 4100, "v must be"), ("k_token_stride", 60, "k: strides"), ("v_head_stride", 0, "v: strides"),
    ("q_out", None, "q_out is null"), ("n_q_heads", 0, "n_q_heads"), ("q", None, "q_out without q"), ("positions", 4096, "without rope")])
def test_append_arguments(env, field, value, text):
    setattr(env.append, field, value)
    refused(env, "append", text)


@pytest.mark.parametrize("field,value,text", [("rot_dim", 66, "rot_dim"), ("rot_dim", 7, "rot_dim"), ("rot_dim", -2, "rot_dim"),
                                              ("n_axes", 0, "n_axes"), ("n_axes", 9, "n_axes")])
def test_rope_arguments(env, field, value, text):
    setattr(env.rope, field, value)
    env.append.rope = ctypes.addressof(env.rope)
    refused(env, "append", text)


def test_rope_pairs(env):
    env.append.rope = ctypes.addressof(env.rope)
    env.rope.axis[5] = 1
    refused(env, "append", "axis of pair 5")
    env.rope.axis[5] = 0
    env.rope.inv_freq[3] = math.nan
    refused(env, "append", "inv_freq of pair 3")
    env.rope.inv_freq[3] = 0.0
    env.rope.halves, env.rope.rot_dim = 1, 24
    refused(env, "append", "multiple of 16")
    env.rope.halves, env.rope.rot_dim, env.rope.n_axes = 0, 64, 2
    env.append.positions, env.append.pos_stride = 4096, 4
    refused(env, "append", "pos_stride")


@pytest.mark.parametrize("what", ["append", "attend", "gather"])
@pytest.mark.parametrize("layer", [-1, 2])
def test_layer_range(env, what, layer):
    refused(env, what, "layer", layer=layer)


def test_compact_outputs_go_together(env):
    import tiered_quantize_evict_gb300 as qe
    for t, r in ((4096, None), (None, 4096)):
        assert env.lib.qe_pages_compact(ctypes.byref(env.pages), ctypes.byref(env.table), t, r, None, 4096, 1 << 40, None) == qe.QE_ERR_INVALID_ARG
        assert b"together" in env.lib.qe_last_error(None)


def test_null_structs(env):
    for what in ALL:
        refused(env, what, "null", null=("pages",))
    for what in ("append", "attend"):
        refused(env, what, "null", null=("chunks",))
        refused(env, what, "null", null=(what,))


def test_nothing_to_do(env):
    """Empty calls are fine and touch nothing."""
    import tiered_quantize_evict_gb300 as qe
    env.chunks.total_q = 0
    assert env.run("append")[0] == env.run("attend")[0] == qe.QE_OK
    env.chunks.total_q, env.chunks.n_seqs = 5, 0
    assert env.run("append")[0] == env.run("attend")[0] == qe.QE_OK
    for what in ("resize", "fork", "copy", "gather"):
        assert env.run(what, n=0)[0] == qe.QE_OK
        refused(env, what, "", n=-1)


def test_structs_match_the_header(paged, tmp_path):
    """Sizes and offsets of the ctypes structs are the C ones."""
    names = {"qe_pages": paged._Pages, "qe_page_table": paged._Table, "qe_rope": paged._Rope, "qe_chunks": Chunks,
             "qe_pages_append_args": AppendArgs, "qe_pages_attend_args": AttendArgs}
    body = "".join(f'printf("{n} %zu", sizeof({n}));' + "".join(f'printf(" %zu", offsetof({n}, {f[0]}));' for f in c._fields_) + 'printf("\\n");'
                   for n, c in names.items())
    (tmp_path / "s.c").write_text('#include <stdio.h>\n#include "qe.h"\nint main(void) {' + body + "return 0;}")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    for line in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.splitlines():
        n, *nums = line.split()
        c = names[n]
        if n in ("qe_chunks", "qe_pages_append_args", "qe_pages_attend_args"):   # what the binding packs has the same layout
            packed = {"qe_chunks": paged._CHUNKS, "qe_pages_append_args": paged._APPEND, "qe_pages_attend_args": paged._ATTEND}[n]
            vals = [0.5 * i if f[1] is ctypes.c_float else i + 1 for i, f in enumerate(c._fields_)]
            assert packed.size == ctypes.sizeof(c)
            got = c.from_buffer_copy(packed.pack(*vals))
            assert [getattr(got, f[0]) for f in c._fields_] == vals
        assert [int(x) for x in nums] == [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_], n


def test_python_refusals(paged):
    import torch
    from tiered_quantize_evict_gb300 import QEError
    x = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(QEError, match="CUDA"):
        paged.PagePool(x, x)
    t = torch.zeros(3, 4, dtype=torch.int32)
    for bad in (t.long(), t[0], t.T):
        with pytest.raises(QEError):
            paged.PageTable(bad, torch.zeros(3, dtype=torch.int32))
    for n in (torch.zeros(2, dtype=torch.int32), torch.zeros(3)):
        with pytest.raises(QEError):
            paged.PageTable(t, n)
    for kw in (dict(rot_dim=65), dict(rot_dim=130), dict(sections=[10, 10]), dict(sections=[32, 32], axis=[0] * 64), dict(axis=[0] * 63),
               dict(theta=-1.0), dict(inv_freq=[1.0]), dict(axis=[-1] * 64), dict(axis=[8] * 64)):
        with pytest.raises(QEError):
            paged.Rope(128, **kw)
    assert paged.Rope(128, sections=[16, 24, 24]).n_axes == 3 and paged.Rope(64, rot_dim=0).n_axes == 1


# ------------------------------------------------------------------------------ the oracle's own pins

def test_oracle_attention_is_the_textbook_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    out, lse, _, _ = op.attend(q, k, v, 1, 0.5, True)
    for j in range(3):
        for h in range(2):
            e = np.exp(0.5 * (k[: 3 + j, 0] @ q[j, h]))
            assert np.allclose(out[j, h], (e[:, None] * v[: 3 + j, 0]).sum(0) / e.sum()) and np.isclose(lse[j, h], np.log(e.sum()))
    out, lse, _, _ = op.attend(q, k[:1], v[:1], 1, 0.5, True)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(out[2], v[0])


def test_oracle_rotation_matches_the_single_axis_one():
    from oracle.rope import apply_rope
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((6, 1, 16)), rng.integers(0, 1000, 6)
    f = [1e4 ** (-2 * i / 16) for i in range(8)]
    assert np.allclose(op.rotate(x, [pos], [0] * 8, f, 16, False)[:, 0], apply_rope(x[:, 0], pos, 1e4))
    y = np.concatenate([x[..., 0::2], x[..., 1::2]], -1)      # halves are the same pairs in another order
    r, z = op.rotate(x, [pos], [0] * 8, f, 16, False), op.rotate(y, [pos], [0] * 8, f, 16, True)
    assert np.allclose(np.concatenate([r[..., 0::2], r[..., 1::2]], -1), z)


def test_oracle_books():
    o = op.Pages(4, 4, 8, 16)
    assert o.resize([0], [40]) == [] and o.table[0] == [0, 1, 2, -1] and o.refs[:4] == [1, 1, 1, 0]
    assert o.fork([0, 0], [1, 2]) == [(2, 3, 8), (2, 4, 8)]
    assert o.table[1] == [0, 1, 3, -1] and o.refs[:5] == [3, 3, 1, 1, 1]
    assert o.resize([1], [20]) == [(1, 5, 4)] and o.table[1] == [0, 5, -1, -1] and o.refs[1] == 2   # its own copy of a shared page
    assert o.resize([3], [64]) is None and o.kv_len[3] == 0      # 3 pages free, 4 needed
    assert o.resize([0], [0]) == [] and o.refs == [2, 1, 0, 0, 1, 1, 0, 0]
    assert o.compact() == ([(4, 2, 16), (5, 3, 16)], 4) and o.table[1][:2] == [0, 3] and o.table[2][:3] == [0, 1, 2]

"""Windows, shared prefixes and dropped pages without a GPU: refusals of the C entry points, the bindings' structs, the oracle's pins."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT
from oracle import pages as op
from test_pages_cpu import _I, _P, env, paged  # noqa: F401


class Groups(ctypes.Structure):
    _fields_ = [("group_start", _P), ("prefix_len", _P), ("n_groups", _I), ("max_group_len", _I)]


@pytest.fixture()
def call(env):  # noqa: F811
    env.groups = Groups(4096, 4096, 2, 0)

    def run(what, layer=0, window=8, sinks=0, ws=4096, nb=1 << 40, n=3, rows=4096, null=()):
        r = lambda x: None if x in null else ctypes.byref(getattr(env, x))  # noqa: E731
        g, t, c, a = r("pages"), r("table"), r("chunks"), r("attend")
        if what == "window":
            st = env.lib.qe_pages_attend_window(g, layer, t, c, a, window, sinks, ws, nb, None)
        elif what == "shared":
            st = env.lib.qe_pages_attend_shared(g, layer, t, c, a, r("groups"), ws, nb, None)
        else:
            st = env.lib.qe_pages_drop(g, t, rows, n, window, sinks, None)
        return st, env.lib.qe_last_error(None).decode()
    return run


def refused(call, what, text, **kw):
    import tiered_quantize_evict_gb300 as qe
    st, msg = call(what, **kw)
    assert st == qe.QE_ERR_INVALID_ARG and text in msg, (what, st, msg)


@pytest.mark.parametrize("field,value,text", [("k", None, "null"), ("dtype", 2, "dtype"), ("page_size", 48, "page_size"), ("head_dim", 96, "head_dim"),
                                              ("page_stride", -2048, "strides"), ("err", 18, "err")])
def test_pool(env, call, field, value, text):  # noqa: F811
    setattr(env.pages, field, value)
    for what in ("window", "shared", "drop"):
        refused(call, what, text)


@pytest.mark.parametrize("field,value,text", [("table", None, "null"), ("kv_len", 4098, "aligned"), ("n_rows", 0, "n_rows"), ("row_stride", 7, "row_stride")])
def test_table(env, call, field, value, text):  # noqa: F811
    setattr(env.table, field, value)
    for what in ("window", "shared", "drop"):
        refused(call, what, text)


@pytest.mark.parametrize("field,value,text", [("q_start", None, "q_start"), ("n_seqs", 65537, "n_seqs"), ("total_q", -1, "total_q"), ("rows", 4098, "aligned")])
def test_chunks(env, call, field, value, text):  # noqa: F811
    setattr(env.chunks, field, value)
    for what in ("window", "shared"):
        refused(call, what, text)


@pytest.mark.parametrize("field,value,text", [("q", None, "q is null"), ("out", 4100, "out must be"), ("q_token_stride", 4, "q: strides"), ("n_q_heads", 3, "multiple"),
                                              ("scale", 0.0, "scale"), ("max_q_len", -1, "max_q_len"), ("lse", 4098, "lse")])
def test_arguments(env, call, field, value, text):  # noqa: F811
    setattr(env.attend, field, value)
    for what in ("window", "shared"):
        refused(call, what, text)


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (4, -1), (-2 ** 31, 5)])
def test_windows(call, window, sinks):
    for what in ("window", "drop"):
        refused(call, what, "window", window=window, sinks=sinks)


def test_a_window_is_causal(env, call):  # noqa: F811
    env.attend.causal = 0
    refused(call, "window", "causal")


@pytest.mark.parametrize("field,value,text", [("group_start", None, "null"), ("prefix_len", None, "null"), ("group_start", 4098, "aligned"), ("prefix_len", 4097, "aligned"),
                                              ("n_groups", -1, "n_groups"), ("n_groups", 65537, "n_groups"), ("n_groups", 0, "no group"),
                                              ("max_group_len", -1, "max_group_len")])
def test_groups(env, call, field, value, text):  # noqa: F811
    setattr(env.groups, field, value)
    refused(call, "shared", text)


def test_tables_too_large_for_shared_prefixes(env, call):  # noqa: F811
    """(2 sequences + 1) * max_pages * 16 tokens are counted in 32 bits."""
    env.table.max_pages = env.table.row_stride = 2 ** 31 // (3 * 16) + 1
    refused(call, "shared", "too large")


def test_other_refusals(env, call):  # noqa: F811
    for what in ("window", "shared", "drop"):
        refused(call, what, "null", null=("pages",))
        refused(call, what, "null", null=("table",))
    for what in ("window", "shared"):
        refused(call, what, "layer", layer=2)
        refused(call, what, "null", null=("attend",))
        refused(call, what, "null", null=("chunks",))
    refused(call, "shared", "null", null=("groups",))
    refused(call, "drop", "rows", rows=None)
    refused(call, "drop", "rows", rows=4098)
    refused(call, "drop", "n must be", n=-1)
    refused(call, "drop", "n must be", n=2 ** 24 + 1)
    assert env.lib.qe_pages_attend_shared_workspace(ctypes.byref(env.pages), None) == 1
    env.table.refs = None
    refused(call, "drop", "refs")


def test_nothing_to_do(env, call):  # noqa: F811
    import tiered_quantize_evict_gb300 as qe
    assert call("drop", n=0)[0] == qe.QE_OK
    env.chunks.total_q = 0
    env.groups.n_groups = 0
    assert call("window")[0] == call("shared")[0] == qe.QE_OK
    refused(call, "window", "window", window=0)


def test_structs_match_the_header(paged, tmp_path):  # noqa: F811
    body = 'printf("%zu", sizeof(qe_groups));' + "".join(f'printf(" %zu", offsetof(qe_groups, {f[0]}));' for f in Groups._fields_)
    body += 'printf(" %d", QE_PAGES_DROPPED);'
    (tmp_path / "s.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qe.h"\nint main(void) {' + body + "return 0;}")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    nums = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert nums == [ctypes.sizeof(Groups)] + [getattr(Groups, f[0]).offset for f in Groups._fields_] + [paged.QE_PAGES_DROPPED]
    got = Groups.from_buffer_copy(paged._GROUPS.pack(1, 2, 3, 4))
    assert paged._GROUPS.size == ctypes.sizeof(Groups) and [getattr(got, f[0]) for f in Groups._fields_] == [1, 2, 3, 4]


# ------------------------------------------------------------------------------ the oracle's own pins

def test_oracle_windows():
    assert op.window_seen(3, 6, 2, 1) == [[0, 2, 3], [0, 3, 4], [0, 4, 5]]
    assert op.window_seen(2, 1, 5, 0) == [[], [0]]
    assert op.window_seen(1, 4, 1, 3) == [[0, 1, 2, 3]]


def test_oracle_attends_to_what_is_seen():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    full = op.attend(q, k, v, 2, 0.5, True)
    for a, b in zip(full, op.attend_seen(q, k, v, 2, 0.5, op.window_seen(2, 9, 9, 0))):
        assert np.array_equal(a, b)
    some = op.attend_seen(q, k, v, 2, 0.5, [[0, 7], []])
    for a, b in zip(some, op.attend(q[:1], k[[0, 7]], v[[0, 7]], 2, 0.5, False)):
        assert np.allclose(a[:1], b)
    assert not some[0][1].any() and np.isneginf(some[1][1]).all()


def test_oracle_drops():
    o = op.Pages(2, 6, 10, 16)
    o.resize([0], [70])
    o.fork([0], [1])
    o.drop([0], 20, 5)      # the next token sees keys from 51 on: pages 1 and 2 go, page 0 has sinks
    assert o.table[0] == [0, -2, -2, 3, 4, -1] and o.refs[:6] == [2, 1, 1, 2, 1, 1]
    o.drop([0, 1], 20, 0)
    assert o.table[0][:3] == [-2] * 3 and o.refs[:6] == [0, 0, 0, 2, 1, 1]
    o.drop([0], 55, 0)      # a wider window takes nothing back
    assert o.table[0][:4] == [-2, -2, -2, 3]
    o.resize([0], [0])
    assert o.table[0] == [-1] * 6 and o.refs[:6] == [0, 0, 0, 1, 0, 1]

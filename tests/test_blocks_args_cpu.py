"""The refusals of the block operators: every bad argument is answered on the host,
before any launch and without a GPU."""
import ctypes

import pytest
import torch

import sparse_mla_attention_02_gb300 as smla
from sparse_mla_attention_02_gb300 import build

A = 1 << 12                      # a plausible address; never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return smla.load()


def P(x):
    return None if x is None else ctypes.c_void_p(x)


def ptrs(x):
    return None if x is None else (ctypes.c_void_p * len(x))(*x)


def pool(a):
    return (ptrs(a["kv"]), ptrs(a["scale"]), a["L"], a["fmt"], a["d"], a["S"], a["block"],
            a["rows"])


POOL = dict(kv=[A, A], scale=[A, A], L=2, fmt=0, d=576, S=640, block=64, rows=0)
TABLE = dict(table=A, table_out=A, R=2, stride=4, ref=A, ref_out=A, NB=10)


def tables(a):
    return (P(a["table"]), P(a["table_out"]), a["R"], a["stride"], P(a["ref"]), P(a["ref_out"]),
            a["NB"])


def copy(lib, **kw):
    a = {**POOL, **dict(src=A, dst=A, n=3), **kw}
    return lib.smla_cache_copy(*pool(a), P(a["src"]), P(a["dst"]), a["n"], None)


def fork(lib, **kw):
    a = {**POOL, **TABLE, **dict(parents=A, children=A, room=A, n=3, lens=A, lens_out=A,
                                 missing=A, ws=None, ws_n=0), **kw}
    return lib.smla_cache_fork(P(a["parents"]), P(a["children"]), P(a["room"]), a["n"],
                               P(a["lens"]), P(a["lens_out"]), *tables(a), *pool(a),
                               P(a["missing"]), P(a["ws"]), a["ws_n"], None)


def free(lib, **kw):
    a = {**TABLE, **dict(rows=A, begin=A, end=A, n=3, block=64), **kw}
    return lib.smla_cache_free(P(a["rows"]), P(a["begin"]), P(a["end"]), a["n"], *tables(a),
                               a["block"], None)


def compact(lib, **kw):
    a = {**POOL, **TABLE, **dict(map=A, live=A, ws=None, ws_n=0), **kw}
    return lib.smla_cache_compact(*tables(a), *pool(a), P(a["map"]), P(a["live"]), P(a["ws"]),
                                  a["ws_n"], None)


POOL_BAD = [(dict(L=0), 1), (dict(block=0), 1), (dict(S=63), 1), (dict(S=0), 1),
            (dict(rows=63), 1), (dict(rows=-1), 1), (dict(d=128), 2), (dict(S=1 << 31), 2),
            (dict(fmt=6), 2), (dict(fmt=-1), 2), (dict(fmt=3, d=512), 2), (dict(fmt=4, d=512), 2),
            (dict(kv=None), 1), (dict(kv=[A, None]), 1), (dict(kv=[A, A + 8]), 1),
            (dict(fmt=2, scale=None), 1), (dict(fmt=4, scale=[A, None]), 1),
            (dict(fmt=5, scale=[A + 2, A]), 1)]
TABLE_BAD = [(dict(R=0), 1), (dict(stride=0), 1), (dict(NB=0), 1), (dict(R=(1 << 24) + 1), 2),
             (dict(stride=(1 << 24) + 1), 2),
             (dict(table=None), 1), (dict(table_out=None), 1), (dict(ref=None), 1),
             (dict(ref_out=None), 1), (dict(table=A + 2), 1), (dict(table_out=A + 1), 1),
             (dict(ref=A + 2), 1), (dict(ref_out=A + 2), 1)]


@pytest.mark.parametrize("kw,code", POOL_BAD + [(dict(n=-1), 1), (dict(src=None), 1),
                                                (dict(dst=A + 2), 1)])
def test_copy_refusals(lib, kw, code):
    assert copy(lib, **kw) == code


@pytest.mark.parametrize("kw,code", POOL_BAD + TABLE_BAD + [
    (dict(n=-1), 1), (dict(NB=11), 1), (dict(lens=None), 1), (dict(lens_out=None), 1),
    (dict(lens=A + 2), 1), (dict(missing=A + 2), 1), (dict(children=None), 1),
    (dict(children=A + 2), 1), (dict(parents=A + 2), 1), (dict(room=A + 1), 1),
    (dict(n=1 << 30), 2), (dict(n=65537), 2), (dict(n=65536, stride=1 << 15), 2), (dict(), 6), (dict(ws=A, ws_n=8), 6),
    (dict(ws=A + 4, ws_n=1 << 20), 1)])
def test_fork_refusals(lib, kw, code):
    assert fork(lib, **kw) == code


@pytest.mark.parametrize("kw,code", TABLE_BAD + [
    (dict(block=0), 1), (dict(n=-1), 1), (dict(rows=None), 1), (dict(rows=A + 2), 1),
    (dict(begin=A + 2), 1), (dict(end=A + 2), 1), (dict(n=65537), 2)])
def test_free_refusals(lib, kw, code):
    assert free(lib, **kw) == code


@pytest.mark.parametrize("kw,code", POOL_BAD + TABLE_BAD + [
    (dict(NB=11), 1), (dict(map=None), 1), (dict(map=A + 2), 1), (dict(live=A + 2), 1),
    (dict(), 6), (dict(ws=A, ws_n=8), 6), (dict(ws=A + 4, ws_n=1 << 20), 1)])
def test_compact_refusals(lib, kw, code):
    assert compact(lib, **kw) == code


def test_nothing_to_do_and_sizes(lib):
    assert copy(lib, n=0, src=None, dst=None) == 0
    size = lib.smla_cache_fork_workspace_size
    assert size(0, 4, 10) == size(3, 0, 10) == size(3, 4, 0) == size(65537, 4, 10) == 0
    assert size(3, 4, 10) > 3 * 4 * 4 and size(3, 4, 10) % 16 == 0
    assert lib.smla_cache_compact_workspace_size(0) == 0
    assert lib.smla_cache_compact_workspace_size(10) >= 2 * 4 * 5


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros((128, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        smla.smla_cache_copy(kv, 0, None, i, i, 64)
    with pytest.raises(ValueError):
        smla.smla_cache_fork(i, i, i, i, i.view(2, 1), i, 64, kv, 0)
    with pytest.raises(ValueError):
        smla.smla_cache_free(i, None, None, i.view(2, 1), i, 64)
    with pytest.raises(ValueError):
        smla.smla_cache_compact(i.view(2, 1), i, 64, kv, 0)

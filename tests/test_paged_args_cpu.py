"""The refusals of smla_cache_append and smla_fwd_window: every bad argument
is answered on the host, before any launch and without a GPU."""
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


def append(lib, **kw):
    a = dict(kv_c=A, kv_s=512, k_pe=A, pe_s=64, cs=A, cs_rows=10, inter=1, q_pe=None, q_t=64,
             q_h=64, q_out=None, qo_t=64, qo_h=64, h=4, start=A, lens=A, table=A, R=2, stride=4,
             block=64, rows=0, N=4, d=576, fmt=0, S=512, cache=A, scale=None, kpe=1.0)
    a.update(kw)
    return lib.smla_cache_append(
        P(a["kv_c"]), a["kv_s"], P(a["k_pe"]), a["pe_s"], P(a["cs"]), a["cs_rows"], a["inter"],
        P(a["q_pe"]), a["q_t"], a["q_h"], P(a["q_out"]), a["qo_t"], a["qo_h"], a["h"],
        P(a["start"]), P(a["lens"]), P(a["table"]), a["R"], a["stride"], a["block"], a["rows"],
        a["N"], a["d"], a["fmt"], a["S"], P(a["cache"]), P(a["scale"]), a["kpe"], None)


def window(lib, **kw):
    a = dict(q=A, kv=A, fmt=0, scale=None, start=A, lens=A, table=A, R=2, stride=4, block=64,
             rows=0, window=0, sinks=0, limit=0, T=4, h=16, d=576, dv=512, S=512, sm=0.1, out=A,
             lse=None, ws=None, ws_n=0)
    a.update(kw)
    return lib.smla_fwd_window(
        P(a["q"]), P(a["kv"]), a["fmt"], P(a["scale"]), P(a["start"]), P(a["lens"]), P(a["table"]),
        a["R"], a["stride"], a["block"], a["rows"], a["window"], a["sinks"], a["limit"], a["T"],
        a["h"], a["d"], a["dv"], a["S"], a["sm"], P(a["out"]), P(a["lse"]), P(a["ws"]), a["ws_n"],
        None)


BATCH = [(dict(R=0), 1), (dict(stride=0), 1), (dict(block=0), 1), (dict(rows=63), 1),
         (dict(rows=-1), 1), (dict(S=0), 1), (dict(S=1 << 31), 2), (dict(start=None), 1),
         (dict(lens=None), 1), (dict(table=None), 1), (dict(start=A + 2), 1), (dict(lens=A + 1), 1),
         (dict(table=A + 2), 1)]


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(N=-1), 1), (dict(d=128), 2), (dict(fmt=6), 2), (dict(fmt=-1), 2),
    (dict(kv_c=None), 1), (dict(kv_c=A + 8), 1), (dict(kv_s=504), 1), (dict(kv_s=516), 1),
    (dict(cache=None), 1), (dict(cache=A + 4), 1),
    (dict(k_pe=None), 1), (dict(cs=None), 1), (dict(cs=A + 8), 1), (dict(cs_rows=0), 1),
    (dict(k_pe=A + 2), 1), (dict(pe_s=60), 1), (dict(pe_s=68), 1),
    (dict(d=512), 1), (dict(d=512, k_pe=None), 1), (dict(d=512, cs=None), 1),
    (dict(d=512, fmt=3, k_pe=None, cs=None), 2), (dict(d=512, fmt=4, k_pe=None, cs=None), 2),
    (dict(fmt=1), 1), (dict(fmt=2), 1), (dict(fmt=4), 1), (dict(fmt=5), 1),
    (dict(fmt=5, scale=A + 2), 1),
    (dict(q_pe=A), 1), (dict(q_pe=A, q_out=A, h=0), 1), (dict(q_pe=A, q_out=A, h=129), 2),
    (dict(q_pe=A + 4, q_out=A), 1), (dict(q_pe=A, q_out=A + 8), 1),
    (dict(q_pe=A, q_out=A, q_h=32), 1), (dict(q_pe=A, q_out=A, qo_t=100), 1),
    (dict(d=512, k_pe=None, cs=None, q_pe=A, q_out=A), 1),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(T=-1), 1), (dict(h=0), 1), (dict(h=129), 2), (dict(d=192), 2), (dict(dv=128), 2),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(T=1 << 27), 2),
    (dict(fmt=2, scale=A), 2), (dict(fmt=3), 2), (dict(fmt=4, scale=A), 2), (dict(fmt=6), 2),
    (dict(fmt=-1), 2), (dict(fmt=1), 1), (dict(fmt=5), 1), (dict(fmt=5, scale=A + 1), 1),
    (dict(q=None), 1), (dict(q=A + 8), 1), (dict(kv=None), 1), (dict(kv=A + 8), 1),
    (dict(out=None), 1), (dict(out=A + 8), 1), (dict(lse=A + 2), 1),
])
def test_window_refusals(lib, kw, code):
    assert window(lib, **kw) == code


def test_nothing_to_do(lib):
    assert append(lib, N=0, start=None, cache=None) == 0
    assert window(lib, T=0, q=None, out=None, start=None) == 0
    size = lib.smla_fwd_window_workspace_size
    for kw in ((0, 4, 16, 576, 512, 0, 4, 64, 0, 0, 0), (2, 0, 16, 576, 512, 0, 4, 64, 0, 0, 0),
               (2, 4, 16, 576, 512, 2, 4, 64, 0, 0, 0), (2, 4, 16, 576, 512, 0, 4, 64, -1, 0, 0)):
        assert size(*kw) == 0


def test_sparse_entry_points_do_not_take_block_scales(lib):
    fwd = lib.smla_fwd
    assert fwd(P(A), P(A), 5, P(A), P(A), None, 4, 16, 576, 512, 64, 256, 0.1, P(A), None,
               None) == smla_unsupported()


def smla_unsupported():
    return [k for k, v in smla.STATUS_NAMES.items() if v == "SMLA_ERR_UNSUPPORTED"][0]


def test_binding_refuses_host_tensors():
    q = torch.zeros((1, 1, 576), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        smla.smla_fwd_window(q, q[0], 0, None, i, i[:1], i.view(1, 2), 64, 0.1)
    with pytest.raises(ValueError):
        smla.smla_cache_append(q[0, :, :512], None, None, i, i[:1], i.view(1, 2), 64, q[0], 0)

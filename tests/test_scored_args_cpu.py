"""The refusals of smla_fwd_scored, on the host and without a GPU."""
import pytest

from tests.test_paged_args_cpu import BATCH, A, P, lib  # noqa: F401


def scored(lib, **kw):  # noqa: F811
    a = dict(q=A, kv=A, fmt=0, scale=None, start=A, lens=A, table=A, R=2, stride=4, block=64,
             rows=0, window=0, sinks=0, limit=0, T=4, h=16, d=576, dv=512, S=512, sm=0.1, cap=1.0,
             slopes=A, first=A, last=A, out=A, lse=None, ws=None, ws_n=0)
    a.update(kw)
    return lib.smla_fwd_scored(
        P(a["q"]), P(a["kv"]), a["fmt"], P(a["scale"]), P(a["start"]), P(a["lens"]), P(a["table"]),
        a["R"], a["stride"], a["block"], a["rows"], a["window"], a["sinks"], a["limit"], a["T"],
        a["h"], a["d"], a["dv"], a["S"], a["sm"], a["cap"], P(a["slopes"]), P(a["first"]),
        P(a["last"]), P(a["out"]), P(a["lse"]), P(a["ws"]), a["ws_n"], None)


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(T=-1), 1), (dict(h=0), 1), (dict(h=129), 2), (dict(d=192), 2), (dict(dv=128), 2),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(T=1 << 27), 2), (dict(fmt=2, scale=A), 2),
    (dict(fmt=3), 2), (dict(fmt=1), 1), (dict(fmt=5, scale=A + 1), 1), (dict(q=None), 1),
    (dict(kv=A + 8), 1), (dict(out=None), 1), (dict(lse=A + 2), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(cap=1e-31), 1),
    (dict(cap=2e30), 1), (dict(slopes=A + 2), 1),
    (dict(first=A + 1), 1), (dict(last=A + 2), 1)])
def test_refusals(lib, kw, code):  # noqa: F811
    assert scored(lib, **kw) == code


def test_nothing_to_do(lib):  # noqa: F811
    assert scored(lib, T=0, q=None, out=None, start=None, first=None, last=None, slopes=None) == 0

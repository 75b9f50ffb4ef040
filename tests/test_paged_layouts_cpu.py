"""smla_cache_append's layouts of rotated queries that no launch may see: rows of q_out
that overlap, and rotation in place with other strides."""
import pytest

from tests.test_paged_args_cpu import A, append, lib  # noqa: F401

Q = dict(q_pe=A, q_out=A + (1 << 20), h=4, N=4)


@pytest.mark.parametrize("kw", [
    dict(qo_t=64, qo_h=64),                            # every (token, head) on its neighbour's
    dict(qo_t=192, qo_h=64),                           # the last head on the next token's first
    dict(qo_t=64, qo_h=192),
    dict(qo_t=128, qo_h=128),
    dict(qo_t=248, qo_h=64),
    dict(q_out=A, q_t=256, q_h=64, qo_t=64, qo_h=256),             # in place, transposed
    dict(q_out=A, q_t=256, q_h=64, qo_t=512, qo_h=64),
])
def test_refused(lib, kw):  # noqa: F811
    assert append(lib, **{**Q, **dict(q_t=256, q_h=64), **kw}) == 1


@pytest.mark.parametrize("kw", [
    dict(q_t=256, q_h=64, qo_t=256, qo_h=64), dict(q_t=256, q_h=64, qo_t=64, qo_h=256),
    dict(q_t=64, q_h=64, qo_t=768, qo_h=192), dict(q_out=A, q_t=768, q_h=192, qo_t=768, qo_h=192),
    dict(N=1, q_t=64, q_h=64, qo_t=64, qo_h=64), dict(h=1, q_t=64, q_h=64, qo_t=64, qo_h=64),
    dict(N=1, q_out=A, q_t=64, q_h=64, qo_t=128, qo_h=64),
])
def test_not_refused(lib, kw):  # noqa: F811
    """(Without a GPU such a call ends at the device query; with one it would launch, so
    it is made on the CPU only.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    assert append(lib, **{**Q, **kw}) == 3

"""The entry points of decoding refuse strides with which the last row or page would lie beyond 2^63 bytes (CPU: refused
before anything is enqueued)."""

import pytest
import torch

from test_decode_abi import _append, _attend, _compact, _fork, _select

FAR = 1 << 40                                        # the largest stride of a few rows


@pytest.mark.parametrize("call,kw", [
    (_append, dict(pages=1 << 24, ks=FAR)), (_append, dict(pages=(1 << 20) + 1, vs=FAR)), (_append, dict(s=1 << 24, ldk=FAR)),
    (_append, dict(s=1 << 24, ldv=FAR)),
    (_attend, dict(pages=1 << 24, ks=FAR)), (_attend, dict(pages=1 << 24, vs=FAR)),
    (_fork, dict(pages=1 << 24, step=(FAR,))), (_compact, dict(pages=1 << 24, step=(FAR,))),
    (_select, dict(n=1 << 20, beams=4, ld=FAR)), (_select, dict(n=1 << 20, ldh=FAR)), (_select, dict(n=1 << 20, ldho=FAR))])
def test_far_rows_are_refused(call, kw):
    assert call(**kw) == -1


def test_a_large_stride_of_few_rows_is_not():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is present: the calls would run")
    assert _append(pages=9, ks=FAR, vs=FAR, ldk=FAR, ldv=FAR, ldt=FAR) == -2
    assert _append(n=1 << 20, ldt=FAR) == -2         # 2^60 elements
    assert _attend(ldq=FAR, ldo=FAR, ks=FAR, vs=FAR) == -2 and _fork(step=(FAR,), ldto=FAR) == -2
    assert _compact(step=(FAR,)) == -2 and _select(ld=FAR, ldh=FAR, ldho=FAR) == -2

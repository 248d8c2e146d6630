"""The choice of tokens on the CPU: the oracle's own pins and what the entry
point refuses before any HIP call."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import sparse_weight_only_amd as sg
from oracle import decode as odec
from sparse_weight_only_amd import _build, decode as D
from sparse_weight_only_amd.sgemv import SGEMV_EALIGN, SGEMV_EINVAL, SGEMV_ESIZE
from test_decode_host import BASE

torch = pytest.importorskip("torch")
NO = -math.inf


def test_oracle_by_hand():
    x = np.log([4.0, 1.0, 2.0, 1.0])
    pick = lambda u, **kw: odec.sample(x, u, **kw)[0]                      # noqa: E731
    # shares .5 .125 .25 .125
    assert [pick(u) for u in (0.0, 0.49, 0.51, 0.62, 0.63, 0.87, 0.88, 0.999, 1.0, 7.0, -1.0, math.nan)] == [0, 0, 1, 1, 2, 2, 3, 3, 3, 3, 0, 0]
    assert [pick(u, temperature=0.0) for u in (0.0, 0.99)] == [0, 0]
    # squared: 16 1 4 1 of 22
    assert [pick(u, temperature=0.5) for u in (0.72, 0.73, 0.78, 0.97)] == [0, 1, 2, 3]
    assert [pick(u, top_k=2) for u in (0.66, 0.67)] == [0, 2]
    assert [pick(u, top_k=3) for u in (0.57, 0.58, 0.72)] == [0, 1, 2]     # of 1 and 3, equal, the lower id
    assert [pick(u, top_p=0.7) for u in (0.66, 0.67)] == [0, 2]
    assert [pick(u, top_p=0.76) for u in (0.57, 0.58, 0.72)] == [0, 1, 2]
    assert pick(0.99, top_p=0.0) == 0 and pick(0.99, top_p=0.4) == 0
    assert [pick(u, min_p=0.3) for u in (0.66, 0.67)] == [0, 2]
    assert [pick(u, top_k=3, top_p=0.8) for u in (0.66, 0.67)] == [0, 2]   # 4/7, 6/7 reaches it
    token, share, far = odec.sample(x, 0.6, top_k=2)
    assert token == 0 and abs(share - math.log(2 / 3)) < 1e-15 and abs(far - (2 / 3 - 0.6)) < 1e-15


def test_oracle_special_values():
    assert odec.sample([NO, NO], 0.5)[:2] == (-1, NO) and odec.sample([math.nan], 0.5)[0] == -1
    assert odec.sample([math.nan, 1.0, NO], 0.9)[:2] == (1, 0.0)
    assert odec.sample([math.inf, 1.0, math.inf], 0.6)[0] == 2 and odec.sample([math.inf, 1.0, math.inf], 0.4)[0] == 0
    assert odec.sample([0.0, -0.0, 0.0], 0.9, top_k=2)[0] == 1 and odec.sample([-1.0, 3.0, 3.0], 0.1, temperature=0.0)[0] == 1


def test_bound_of_top_k_under_sanitizers():
    """What is listed for top_k stays near k, whatever a row's length leaves without a logit, and whatever masks do."""
    from sparse_weight_only_amd import _build_san
    exe = _build_san.BOUND_CHECK
    newest = max(os.path.getmtime(f) for f in [_build_san.BOUND_SRC] + [os.path.join(_build.CSRC, h) for h in ("sample_bound.hpp", "decode_index.hpp")])
    if not os.path.exists(exe) or os.path.getmtime(exe) < newest:
        _build_san.build_index_check()
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-3000:]


def args(**kw):
    a = dict(x=BASE, x_stride=100, uniform=BASE, ids=BASE, rows=3, vocab=100, dtype=D.F32)
    a.update(kw)
    return D.Sampling(**a)


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), SGEMV_EINVAL), (dict(vocab=0), SGEMV_EINVAL), (dict(vocab=-5), SGEMV_EINVAL), (dict(dtype=3), SGEMV_EINVAL), (dict(dtype=-1), SGEMV_EINVAL),
    (dict(x=0), SGEMV_EINVAL), (dict(uniform=0), SGEMV_EINVAL), (dict(ids=0), SGEMV_EINVAL), (dict(x_stride=-100), SGEMV_EINVAL),
    (dict(rows=65536), SGEMV_ESIZE), (dict(vocab=(1 << 20) + 1), SGEMV_ESIZE), (dict(x=BASE + 2), SGEMV_EALIGN), (dict(x=BASE + 1, dtype=D.F16), SGEMV_EALIGN),
    (dict(uniform=BASE + 2), SGEMV_EALIGN), (dict(ids=BASE + 1), SGEMV_EALIGN), (dict(logprob=BASE + 3), SGEMV_EALIGN), (dict(top_k=BASE + 2), SGEMV_EALIGN),
    (dict(temperature=BASE + 2), SGEMV_EALIGN), (dict(top_p=BASE + 2), SGEMV_EALIGN), (dict(min_p=BASE + 2), SGEMV_EALIGN)])
def test_refused(bad, want):
    assert sg.lib().sgemv_sample(ctypes.byref(args(**bad)), None) == want


def test_nothing_to_do_is_no_launch():
    assert sg.lib().sgemv_sample(None, None) == SGEMV_EINVAL
    assert sg.lib().sgemv_sample(ctypes.byref(args(rows=0, x=0, uniform=0, ids=0)), None) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    x, u = torch.zeros(3, 50), torch.zeros(3)
    i = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(x=x[0]), dict(x=x.t()), dict(uniform=u.double()), dict(uniform=u[:2]), dict(uniform=u[:, None]), dict(temperature=i), dict(top_k=u),
               dict(top_p=torch.zeros(6)[::2]), dict(min_p=u.half()), dict(out=i.long()), dict(logprob=i), dict(x=x.double()), dict(x=x.int())):
        with pytest.raises(ValueError):
            sg.sample(**{**dict(x=x, uniform=u), **kw})
    with pytest.raises(ValueError, match="not on a GPU"):
        sg.sample(x, u, temperature=u, top_k=i, top_p=u, min_p=u, out=i, logprob=u)

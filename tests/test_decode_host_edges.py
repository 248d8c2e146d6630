"""The decode-step operators on the CPU where they can go wrong between the
cases of the other host tests."""
import os
import subprocess

import numpy as np
import pytest

import sparse_weight_only_amd as sg
from oracle import decode as odec
from sparse_weight_only_amd import _build
from sparse_weight_only_amd.sgemv import SGEMV_EINVAL

torch = pytest.importorskip("torch")


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_a_mask_table_without_masks_is_refused():
    """An empty tensor's address is null, which the library takes for no masks."""
    for kw in (dict(masks=ints(0, 2)), dict(masks=ints(0, 2), mask_row=ints(2))):
        with pytest.raises(ValueError, match="no mask"):
            sg.adjust_logits(torch.zeros(2, 50), **kw)


def test_oracle_candidates_below_slot_zero():
    """Three candidates in a context of two: the first has no slot and sees nothing, whatever its bits."""
    v = np.arange(16.0).reshape(1, 8, 1, 2)
    q = np.zeros((3, 1, 2))
    out, _, _, keys = odec.attend(q, np.zeros_like(v), v, [0, 3], [2], np.array([[0]]), 1.0, tree=np.array([[7], [6], [2]]))
    # new token 1 is slot 0 (values 0, 1), token 2 is slot 1 (values 2, 3)
    assert keys.ravel().tolist() == [0, 2, 1]
    assert out[:, 0].tolist() == [[0.0, 0.0], [1.0, 2.0], [0.0, 1.0]]


def test_visible_keys_under_sanitizers():
    from sparse_weight_only_amd import _build_san
    exe = _build_san.VISIBLE_CHECK
    newest = max(os.path.getmtime(f) for f in (_build_san.VISIBLE_SRC, os.path.join(_build.CSRC, "decode_index.hpp")))
    if not os.path.exists(exe) or os.path.getmtime(exe) < newest:
        _build_san.build_index_check()
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-3000:]


@pytest.mark.parametrize("args", [(128, 1e-320), (8, 1e-300, 1e-300), (8, 1e4, 2.0, 1e3, -1e308, 1e308), (64, 1e-320, 1.0, 10.0)])
def test_rope_table_refuses_frequencies_that_are_not_finite(args):
    """Finite arguments whose powers, quotients or differences overflow: every angle would be NaN."""
    with pytest.raises(sg.SgemvError) as e:
        sg.rope_table(*args)
    assert e.value.code == SGEMV_EINVAL


@pytest.mark.parametrize("args", [(8, 1e-300), (256, 1e300), (8, 1e4, 1e300), (8, 1e4, 2.0, 1e300)])
def test_rope_table_takes_extreme_arguments(args):
    got = sg.rope_table(*args)
    assert np.isfinite(got).all() and np.all(got >= 0)

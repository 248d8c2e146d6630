"""The decode-step operators on the CPU where they can go wrong between the
cases of the other host tests."""
import os
import subprocess

import numpy as np
import pytest

import sparse_weight_only_amd as sg
from oracle import decode as odec
from sparse_weight_only_amd import _build

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

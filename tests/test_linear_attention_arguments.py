"""CPU tests of arguments of the linear attention and the layer norm that are refused, or answered, before a GPU is
asked."""
import ctypes

import pytest

from nonlinear_rnn_pararnn_b200 import _lib
from test_linear_attention_boundary import E, _cfg


@pytest.mark.parametrize("bad", [{"debug_fault": -1}, {"wait_limit_us": -1}])
def test_wait_settings(bad):
    size = _lib.load().slstm_linear_attention_workspace_size
    assert size(ctypes.byref(_cfg(**bad)), 2, 100, 0, 0) == 0
    assert size(ctypes.byref(_cfg(**{n: 5 for n in bad})), 2, 100, 0, 0) == size(ctypes.byref(_cfg()), 2, 100, 0, 0)
    p = ctypes.c_void_p(0x10000)
    assert _lib.load().slstm_linear_attention_step(p, p, p, p, None, p, p, ctypes.byref(_cfg(**bad)), 2, None) == E

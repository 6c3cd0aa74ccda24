"""CPU tests of arguments of the linear attention and the layer norm that are refused, or answered, before a GPU is
asked."""
import ctypes

import pytest
import torch

from nonlinear_rnn_pararnn_b200 import _lib, api
from test_linear_attention_boundary import E, _cfg


@pytest.mark.parametrize("bad", [{"debug_fault": -1}, {"wait_limit_us": -1}])
def test_wait_settings(bad):
    size = _lib.load().slstm_linear_attention_workspace_size
    assert size(ctypes.byref(_cfg(**bad)), 2, 100, 0, 0) == 0
    assert size(ctypes.byref(_cfg(**{n: 5 for n in bad})), 2, 100, 0, 0) == size(ctypes.byref(_cfg()), 2, 100, 0, 0)
    p = ctypes.c_void_p(0x10000)
    assert _lib.load().slstm_linear_attention_step(p, p, p, p, None, p, p, ctypes.byref(_cfg(**bad)), 2, None) == E


def test_workspaces_of_repeated_or_strided_bytes():
    """A view may count more bytes than its memory has: refused."""
    cpu = torch.device("cpu")
    fields = (4, 2, 64, 64, _lib.SLSTM_BF16, _lib.SLSTM_DECAY_TOKEN, 1.0, 128, 128, 256)
    n = api._la_bytes(fields, 2, 100, False, False)
    assert api._la_workspace(fields, 2, 100, False, False, torch.empty(n, dtype=torch.uint8), cpu).numel() == n
    for ws in (torch.empty(1, dtype=torch.uint8).expand(n), torch.empty(2 * n, dtype=torch.uint8)[::2],
               torch.empty(n - 1, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="ws must hold"):
            api._la_workspace(fields, 2, 100, False, False, ws, cpu)
        with pytest.raises(ValueError, match="ws must hold"):
            api._bytes_on(ws, n, cpu)

"""Arguments of the packed scan and the norms that a call could not use are refused,
not passed over (CPU: the checks come before the library)."""
import pytest
import torch

import gated_delta_rule_decay_amd as g


def test_packed_calls_need_offsets():
    x = torch.zeros(1, 8, 16)
    with pytest.raises(ValueError, match="cu_seqlens"):
        g.gated_scan_fwd_varlen(x, x, None)
    with pytest.raises(ValueError, match="cu_seqlens"):
        g.gated_scan_bwd_varlen(x, x, x, torch.zeros(1, 1, 16), None)


def test_what_belongs_to_a_missing_k():
    q, f = torch.zeros(2, 8, 3, 16), torch.zeros(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="k_out"):
        g.rotary_fwd(q, None, f, k_out=q.clone())
    with pytest.raises(ValueError, match="dk"):
        g.rotary_bwd(q, None, f, dk=q.clone())
    with pytest.raises(ValueError, match="k_out"):
        g.qk_norm_rotary_fwd(q, None, freq=f, k_out=q.clone())
    with pytest.raises(ValueError, match="d_k_out"):
        g.qk_norm_rotary_bwd(q, q, q, None, freq=f)


def test_missing_tensors_are_named():
    x, q = torch.zeros(2, 8, 16), torch.zeros(2, 8, 3, 16)
    f = torch.zeros(8, dtype=torch.float64)
    marks = torch.zeros(2, 1, 16)
    with pytest.raises(TypeError, match="x "):
        g.gated_scan_fwd(None, x)
    with pytest.raises(TypeError, match="log_decay"):
        g.gated_scan_fwd(x, None)
    with pytest.raises(TypeError, match="marks"):
        g.gated_scan_bwd(x, x, x, None)
    with pytest.raises(TypeError, match="dy"):
        g.gated_scan_bwd(None, x, x, marks)
    with pytest.raises(TypeError, match="state"):
        g.gated_scan_step(x[0], x[0], None)
    with pytest.raises(TypeError, match="q "):
        g.rotary_fwd(None, q, f)
    with pytest.raises(TypeError, match="d_q_out "):
        g.rotary_bwd(None, q, f)

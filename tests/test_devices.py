"""The kernels run on the current device: tensors of another one are refused."""
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for stream in (gdn._stream, gdn._raw_stream):
        with pytest.raises(gdn.GdnError, match="current device"):
            stream(torch.device("cuda", 1))


def test_a_workspace_elsewhere_is_refused():
    """The kernels would write to its address."""
    cpu, cuda = torch.device("cpu"), torch.device("cuda", 0)
    given = torch.empty(64, dtype=torch.uint8)
    for x, device in ((given, cuda), (given[::2], cpu)):
        with pytest.raises(gdn.GdnError, match="workspace"):
            gdn._workspace(16, x, device)
    assert gdn._workspace(16, given, cpu) is given
    assert gdn._workspace(65, given, cpu) is not given


@pytest.mark.gpu
def test_calls_refuse_another_current_device(monkeypatch):
    """Every call asks for its stream, and that refuses; nothing is launched."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, x, w, n = z(1, 4, 2, 64), z(3, 64), z(64, dt=torch.float32), z(3, dt=torch.float32)
    lse, lens = z(1, 2, 4, dt=torch.float32), z(1, dt=torch.int32)
    g = z(1, 4, 2, dt=torch.float32)
    kc = z(1, 9, 2, 64)
    calls = (lambda: gdn.attn_fwd(q, q, q), lambda: gdn.attn_bwd(q, q, q, q, lse, q), lambda: gdn.attention(q, q, q),
             lambda: gdn.attn_decode(q, q, q, kc, kc.clone(), lens), lambda: gdn.layer_norm_fwd(x, w),
             lambda: gdn.layer_norm_bwd(x, w, n, n, x), lambda: gdn.layer_norm(x, w), lambda: gdn.gdn_fwd(q, q, q, g, g))
    with gdn.KernelTimer() as t:
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
        for call in calls:
            with pytest.raises(gdn.GdnError, match="current device"):
                call()
        monkeypatch.undo()
    assert t.launches == 0
